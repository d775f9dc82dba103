// The product of two matrices in 4-bit MX form, grouped by expert.
#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kRowTile = 16, kColTile = 64;
constexpr int kMaxGroups = kMaxE + 1;

struct Params {
  const uint8_t *xc, *xs;
  int x_rows;
  moe_mx4_matrix w;
  bool grouped;
  const int32_t *n_uniq, *uniq_offset, *uniq_slot, *pair_token;
  const float* pair_gate;
  int n_pairs, T, max_uniq, shared_slot;
  bool gather, gate;
  void* out;
  long long ld;
  int* status;
};

// The groups' row tiles, laid end to end: group i's first is prefix[i].
struct Schedule {
  int n_groups;
  int prefix[kMaxGroups + 1];
  int scan[kThreads];
};

// Rows of group i: the used experts in order, then the shared one.
__device__ __forceinline__ void group_rows(const Params& P, int i, int n_uniq, int& first, int& n, int& slot) {
  if (!P.grouped) {
    first = 0, n = P.x_rows, slot = 0;
  } else if (i < n_uniq) {
    first = min(max(__ldg(P.uniq_offset + i), 0), P.n_pairs);
    n = max(min(__ldg(P.uniq_offset + i + 1), P.n_pairs) - first, 0);
    slot = __ldg(P.uniq_slot + i);
  } else {
    first = P.n_pairs, n = P.T, slot = P.shared_slot;
  }
}

__device__ void build_schedule(const Params& P, Schedule& S) {
  const int nu = P.grouped ? min(max(__ldg(P.n_uniq), 0), P.max_uniq) : 0;
  const int ng = P.grouped ? nu + (P.shared_slot >= 0 ? 1 : 0) : 1;
  const int per = (ng + kThreads - 1) / kThreads;
  int mine = 0;
  for (int i = threadIdx.x * per; i < min(ng, (int(threadIdx.x) + 1) * per); ++i) {
    int first, n, slot;
    group_rows(P, i, nu, first, n, slot);
    if (slot < 0 || slot >= P.w.n_slots) {
      if (blockIdx.x == 0) report(P.status, kDevBadSlot, first);
      n = 0;
    }
    S.prefix[i] = mine;
    mine += (n + kRowTile - 1) / kRowTile;
  }
  S.scan[threadIdx.x] = mine;
  __syncthreads();
  int base = 0;
  for (int i = 0; i < threadIdx.x; ++i) base += S.scan[i];
  for (int i = threadIdx.x * per; i < min(ng, (int(threadIdx.x) + 1) * per); ++i) S.prefix[i] += base;
  if (threadIdx.x == kThreads - 1) {
    S.n_groups = ng;
    S.prefix[ng] = base + mine;
  }
  __syncthreads();
}

__device__ __forceinline__ float level(uint32_t code) {
  const uint32_t m = code & 7;
  const float a = m < 4 ? 0.5f * m : m == 7 ? 6.f : static_cast<float>(m - 2);
  return (code & 8) ? -a : a;
}

__device__ __forceinline__ float scale_of(uint32_t s) {
  return __uint_as_float(s == 0 ? 0x00400000u : s == 255 ? 0x7fffffffu : s << 23);
}

template <typename T>
__device__ __forceinline__ void store(void* out, long long i, float v);
template <>
__device__ __forceinline__ void store<float>(void* out, long long i, float v) { static_cast<float*>(out)[i] = v; }
template <>
__device__ __forceinline__ void store<__nv_bfloat16>(void* out, long long i, float v) {
  static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ void store<__half>(void* out, long long i, float v) {
  static_cast<__half*>(out)[i] = __float2half_rn(v);
}

template <typename T, bool SWIGLU>
__global__ void __launch_bounds__(kThreads) mx4_product_kernel(const Params P) {
  __shared__ Schedule S;
  __shared__ float xt[kRowTile][33], wt[kColTile][33];
  build_schedule(P, S);
  const int m_tiles = (P.w.rows + kColTile - 1) / kColTile;
  const int K = P.w.cols, pitch = mx4_pitch(K);
  const int nu = S.n_groups - (P.grouped && P.shared_slot >= 0 ? 1 : 0);
  const long long total = static_cast<long long>(S.prefix[S.n_groups]) * m_tiles;
  const int r = threadIdx.x / 8, n0 = (threadIdx.x % 8) * 8;
  for (long long item = blockIdx.x; item < total; item += gridDim.x) {
    const int tile = static_cast<int>(item / m_tiles), m = static_cast<int>(item % m_tiles);
    int lo = 0, hi = S.n_groups;  // the last group whose first tile is at most `tile` and that has tiles
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (S.prefix[mid] <= tile) lo = mid; else hi = mid;
    }
    int first, n, slot;
    group_rows(P, lo, nu, first, n, slot);
    const int row0 = first + (tile - S.prefix[lo]) * kRowTile, rows = min(kRowTile, first + n - row0);
    const uint8_t* wc = P.w.codes + static_cast<size_t>(slot) * P.w.code_stride;
    const uint8_t* ws = P.w.scales + static_cast<size_t>(slot) * P.w.scale_stride;
    float acc[8] = {};
    for (int k0 = 0; k0 < K; k0 += 32) {
      __syncthreads();
      for (int i = threadIdx.x; i < kRowTile * 16; i += kThreads) {
        const int row = i / 16, b = i % 16, p = row0 + row;
        uint32_t c = 0, s = 0;
        if (row < rows) {
          int src = p;
          if (P.gather) src = p < P.n_pairs ? __ldg(P.pair_token + p) : p - P.n_pairs;
          if (src < 0 || src >= P.x_rows) {
            report(P.status, kDevBadExpert, p);
          } else {
            c = P.xc[static_cast<size_t>(src) * (K / 2) + k0 / 2 + b];
            s = P.xs[static_cast<size_t>(src) * pitch + k0 / 32];
          }
        }
        xt[row][2 * b] = level(c & 15) * scale_of(s);
        xt[row][2 * b + 1] = level(c >> 4) * scale_of(s);
      }
      for (int i = threadIdx.x; i < kColTile * 16; i += kThreads) {
        const int row = i / 16, b = i % 16, wr = m * kColTile + row;
        uint32_t c = 0, s = 0;
        if (wr < P.w.rows) {
          c = wc[static_cast<size_t>(wr) * (K / 2) + k0 / 2 + b];
          s = ws[static_cast<size_t>(wr) * pitch + k0 / 32];
        }
        wt[row][2 * b] = level(c & 15) * scale_of(s);
        wt[row][2 * b + 1] = level(c >> 4) * scale_of(s);
      }
      __syncthreads();
#pragma unroll 8
      for (int k = 0; k < 32; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = fmaf(xt[r][k], wt[n0 + j][k], acc[j]);
    }
    if (r >= rows) continue;
    const int p = row0 + r;
    const float g = P.gate && p < P.n_pairs ? __ldg(P.pair_gate + p) : 1.f;
    const int wr = m * kColTile + n0;
    if (wr >= P.w.rows) continue;
#pragma unroll
    for (int j = 0; j < 8; j += SWIGLU ? 2 : 1) {
      if (SWIGLU)
        store<T>(P.out, p * P.ld + (wr + j) / 2, acc[j] / (1.f + expf(-acc[j])) * acc[j + 1] * g);
      else
        store<T>(P.out, p * P.ld + wr + j, acc[j] * g);
    }
  }
}

}  // namespace

cudaError_t mx4_product_init(const Ctx& ctx) {
  (void)ctx;
  return cudaSuccess;
}

cudaError_t launch_mx4_product(const Ctx& ctx, const Mx4Args& a, cudaStream_t s) {
  Params P{};
  P.xc = a.x_codes;
  P.xs = a.x_scales;
  P.x_rows = a.x_rows;
  P.w = a.w;
  P.grouped = a.g != nullptr;
  if (a.g != nullptr) {
    P.n_uniq = a.g->n_uniq;
    P.uniq_offset = a.g->uniq_offset;
    P.uniq_slot = a.g->uniq_slot;
    P.pair_token = a.g->pair_token;
    P.pair_gate = a.g->pair_gate;
    P.n_pairs = a.g->n_pairs;
    P.T = a.g->T;
    P.max_uniq = a.g->n_pairs < a.g->E ? a.g->n_pairs : a.g->E;
  }
  P.shared_slot = a.shared_slot;
  P.gather = a.gather;
  P.gate = a.gate;
  P.out = a.out;
  P.ld = static_cast<long long>(a.ld);
  P.status = ctx.d_status;
  const int grid = 8 * ctx.num_sms;
#define MOE_MX4_CASE(T)                                                    \
  if (a.swiglu)                                                            \
    mx4_product_kernel<T, true><<<grid, kThreads, 0, s>>>(P);              \
  else                                                                     \
    mx4_product_kernel<T, false><<<grid, kThreads, 0, s>>>(P);
  if (a.out_type == MOE_TYPE_BF16) {
    MOE_MX4_CASE(__nv_bfloat16)
  } else if (a.out_type == MOE_TYPE_FP16) {
    MOE_MX4_CASE(__half)
  } else {
    MOE_MX4_CASE(float)
  }
#undef MOE_MX4_CASE
  return cudaGetLastError();
}

}  // namespace moe

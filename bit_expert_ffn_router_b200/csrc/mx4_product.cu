// The product of two matrices in 4-bit MX form, grouped by expert, on the
// block-scaled tensor cores:
//
//   out[r, n] = sum_b 2^(sx[r,b] + sw[n,b] - 254) sum_{i<32} x[r,32b+i] w[n,32b+i]
//
// tcgen05.mma kind::mxf4 takes both 4-bit operands from shared memory and both
// scales from tensor memory, one scale byte per 32 K values, so nothing is
// unpacked: codes go from global memory to the tensor cores by TMA, and only
// the scales (one byte in 17) pass through registers.
//
// The weight rows are the M side (128 per tile, TMEM lanes), the x rows the N
// side (16 to kBN per tile, in steps of 16). A group's rows are cut into equal
// tiles, so a ragged expert wastes at most 15 rows per tile, one decoded token
// costs N = 16, and an expert of up to kBN rows reads its weights once.
//
// One persistent CTA per SM, ten warps:
//   warp 0     codes: a stage's 128 weight rows x 256 K values by one TMA box,
//              the x rows by gather loads of four rows each (the rows that the
//              tokens name, or consecutive ones);
//   warp 1     TMEM allocation; one lane issues the scale copies
//              (shared -> tensor memory) and the MMAs;
//   warps 2-5  scales: thread r loads weight row r's and x rows r's and r +
//              128's scale bytes, 16 K blocks ahead, and stores them in the
//              order the tensor memory wants: 512-byte pieces of 128 rows x 4
//              blocks, row r at (r % 32) * 16 + (r / 32) * 4;
//   warps 6-9  epilogue: accumulators from tensor memory (two buffers, so that
//              the next item's MMAs overlap), SwiGLU or gate, one rounding,
//              stores of 64 to 128 consecutive bytes per row and warp.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "moe_internal.cuh"
#include "ptx.cuh"
#include "tc.cuh"

namespace moe {
namespace {

constexpr int kThreads = 576;
constexpr int kBM = 128;                      // weight rows per tile
constexpr int kBN = 208;                      // x rows per tile, at most
constexpr int kBK = 256;                      // K values per stage: 128 bytes of codes per row
constexpr int kStages = 4;
constexpr int kMaxGroups = kMaxE + 1;
constexpr int kAcc = kBN;                     // TMEM columns of one accumulator
constexpr int kSfCols = 24;                   // TMEM columns of a stage's scales: w 2 x 4, x 2 x 8
static_assert(2 * kAcc + kStages * kSfCols <= 512, "tensor memory budget");
constexpr int kScaleThreads = 128;
constexpr int kEpiThreads = 256;
constexpr int kGatherThreads = 128;
constexpr int kGatherRows = kBN / (kGatherThreads / 8);  // rows of a stage per gather thread
constexpr int kGatherLag = 2;                            // stages between issuing a copy and announcing it
constexpr int kBoxA = 64, kBoxB = 16;                    // x rows of the two TMA boxes

struct Smem {
  static constexpr int kA = 0;                          // kBM rows x 128 bytes, 128B-swizzled
  static constexpr int kB = kBM * 128;                  // kBN rows x 128 bytes
  static constexpr int kSfA = kB + kBN * 128;           // 2 pieces of 512 bytes (K 0..127, 128..255)
  static constexpr int kSfB = kSfA + 1024;              // 2 x 2 pieces (K half, rows 0..127 / 128..255)
  static constexpr int kStage = kSfB + 2048;
  static constexpr int kTable = kStages * kStage;
};
static_assert(Smem::kStage % 1024 == 0, "swizzle atoms start on 1024 bytes");

// The groups' row tiles, laid end to end: group i's first is prefix[i].
struct Table {
  uint64_t full[kStages];      // TMA (tx), scale warps, gather warps: a stage is complete
  uint64_t empty[kStages];     // MMA commit: codes and scales read
  uint64_t d_full[2];          // MMA commit: accumulator complete
  uint64_t d_empty[2];         // epilogue (count 256)
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort_flag;
  int n_groups;
  int scan[kThreads / 32];
  int prefix[kMaxGroups + 1];
  int first[kMaxGroups];
  int rows[kMaxGroups];
  int slot[kMaxGroups];
};
constexpr int kSmemBytes = Smem::kTable + static_cast<int>(sizeof(Table)) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");

struct Params {
  const uint8_t *xc, *xs, *ws;  // x codes; scales
  size_t ws_stride;
  int x_rows, w_rows, n_slots, K, pitch, m_tiles;
  bool grouped;
  const int32_t *n_uniq, *uniq_offset, *uniq_slot, *pair_token;
  const float* pair_gate;
  int n_pairs, T, max_uniq, shared_slot;
  bool gather, gate;
  bool pack;               // 32-bit stores of two neighbouring 16-bit results
  void* out;
  long long ld;
  int* status;
  unsigned long long timeout_ns;
};

__device__ __forceinline__ bool aborted(const Table* B) {
  return *reinterpret_cast<const volatile int*>(&B->abort_flag) != 0;
}

// Waits at most the context's limit; on expiry records the place and raises
// the CTA's abort flag, on which every role leaves its loop.
__device__ __forceinline__ bool wait_bar(Table* B, uint64_t* bar, uint32_t parity, const Params& P, int where) {
  if (mbar_test(bar, parity)) return true;
  if (aborted(B)) return false;
  if (mbar_wait(bar, parity, global_timer_ns() + P.timeout_ns)) return true;
  report(P.status, kDevTimeout, 200 + where);
  *reinterpret_cast<volatile int*>(&B->abort_flag) = 1;
  return false;
}

// Lane 0 waits; every lane takes the same path afterwards.
__device__ __forceinline__ bool wait_warp(Table* B, uint64_t* bar, uint32_t parity, const Params& P, int where) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = wait_bar(B, bar, parity, P, where) ? 1 : 0;
  ok = __shfl_sync(0xffffffffu, ok, 0);
  return ok != 0;
}

__device__ __forceinline__ int tiles_of(int rows) { return (rows + kBN - 1) / kBN; }

__device__ void build_table(const Params& P, Table& S) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nu = P.grouped ? min(max(__ldg(P.n_uniq), 0), P.max_uniq) : 0;
  const int ng = P.grouped ? nu + (P.shared_slot >= 0 ? 1 : 0) : 1;
  const int per = (ng + kThreads - 1) / kThreads;
  const int i0 = min(tid * per, ng), i1 = min(i0 + per, ng);
  int mine = 0;
  for (int i = i0; i < i1; ++i) {
    int first, n, slot;
    if (!P.grouped) {
      first = 0, n = P.x_rows, slot = 0;
    } else if (i < nu) {  // bounds hold even where the grouping's arrays do not make sense
      first = min(max(__ldg(P.uniq_offset + i), 0), P.n_pairs);
      n = max(min(__ldg(P.uniq_offset + i + 1), P.n_pairs) - first, 0);
      slot = __ldg(P.uniq_slot + i);
    } else {
      first = P.n_pairs, n = P.T, slot = P.shared_slot;
    }
    if (slot < 0 || slot >= P.n_slots) {
      if (blockIdx.x == 0) report(P.status, kDevBadSlot, first);
      n = 0;
    }
    S.first[i] = first;
    S.rows[i] = n;
    S.slot[i] = slot;
    S.prefix[i] = mine;
    mine += tiles_of(n);
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) S.scan[warp] = incl;
  __syncthreads();
  int base = incl - mine;
  for (int w = 0; w < warp; ++w) base += S.scan[w];
  for (int i = i0; i < i1; ++i) S.prefix[i] += base;
  if (tid == kThreads - 1) {
    S.n_groups = ng;
    S.prefix[ng] = base + mine;
  }
}

struct Item {
  int m, row0, rows, slot, n16;
};

// Item w: tile w / m_tiles of weight tile w % m_tiles. The group is the last
// one whose first tile is at most the tile (empty groups share the next
// one's); its rows are cut into equal tiles of a multiple of 16.
__device__ __forceinline__ Item item_at(const Params& P, const Table& S, int w) {
  const int tile = w / P.m_tiles;
  int lo = 0, hi = S.n_groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (S.prefix[mid] <= tile)
      lo = mid;
    else
      hi = mid;
  }
  const int n = S.rows[lo], nt = tiles_of(n), j = tile - S.prefix[lo];
  const int tr = ((n + nt - 1) / nt + 15) & ~15;
  Item it;
  it.m = w - tile * P.m_tiles;
  it.row0 = S.first[lo] + j * tr;
  it.rows = min(tr, n - j * tr);
  it.slot = S.slot[lo];
  it.n16 = (it.rows + 15) & ~15;
  return it;
}

// x row of output row p; out-of-range tokens are clamped (and reported by the
// scale threads).
__device__ __forceinline__ int source_row(const Params& P, int p) {
  if (!P.gather) return p;
  const int t = p < P.n_pairs ? __ldg(P.pair_token + p) : p - P.n_pairs;
  return min(max(t, 0), P.x_rows - 1);
}

// 16 bytes to shared memory without passing through registers; zeros where
// `live` is false.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

// 32 rows of 16 bytes, to four 32-bit columns of every lane quarter.
__device__ __forceinline__ void tc_copy_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Descriptor of such a piece: no swizzle, cores of 8 rows x 16 bytes, 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(const void* p) {
  uint64_t d = (static_cast<uint64_t>(smem_u32(p)) >> 4) & 0x3FFFull;
  d |= uint64_t(128 >> 4) << 16;
  d |= uint64_t(128 >> 4) << 32;
  d |= uint64_t(1) << 46;
  return d;
}

// kind::mxf4: A and B e2m1, scales ue8m0, both K-major, M = 128, N = n. Bits
// 29-30 and 4-5 pick the byte of the scale columns: 0 for the first 64 K
// values of a 128, 2 for the second.
__device__ __forceinline__ uint32_t instr_desc_mxf4(int n, uint32_t half) {
  return (half << 5) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>(128 >> 7) << 27) | (half << 30);
}

__device__ __forceinline__ void tc_mma_mxf4(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                            uint32_t sfb, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
          d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(sfa), "r"(sfb)
      : "memory");
}

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Every lane's shared-memory writes, made visible to the asynchronous units
// that read them, then one arrival for the warp.
__device__ __forceinline__ void arrive_warp(uint64_t* bar) {
  fence_async_smem();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// The scale bytes of blocks 16 pair .. 16 pair + 15 of one row as four words
// (blocks past the row's end read as 0).
__device__ __forceinline__ uint4 load_scales(const uint8_t* row, int pair, int blocks) {
  uint4 v = __ldg(reinterpret_cast<const uint4*>(row) + pair);
  const int left = blocks - 16 * pair;  // bytes that are scales
  if (left < 16) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = min(max(left - 4 * i, 0), 4);
      w[i] = n == 4 ? w[i] : w[i] & ((1u << (8 * n)) - 1u);
    }
  }
  return v;
}

__device__ __forceinline__ void put_scales(uint8_t* piece, int row, uint32_t word) {
  *reinterpret_cast<uint32_t*>(piece + (row & 31) * 16 + (row >> 5) * 4) = word;
}

template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half narrow<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  T v[2] = {narrow<T>(a), narrow<T>(b)};
  uint32_t r;
  memcpy(&r, v, 4);
  return r;
}

// 16 accumulator columns (output rows p0 .. p0 + 15, `left` of them real) of
// weight row wr in v; lane i holds the gate of row p0 + i % 16.
template <typename T, bool SWIGLU>
__device__ __forceinline__ void store16(const Params& P, const float* v, int wr, long long p0, int left, float gate_l) {
  const bool live = wr < P.w_rows;
  T* out = static_cast<T*>(P.out) + p0 * P.ld;
  if constexpr (!SWIGLU && sizeof(T) == 4) {
    float o[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = P.gate ? v[i] * __shfl_sync(0xffffffffu, gate_l, i) : v[i];
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (live && i < left) out[i * P.ld + wr] = narrow<T>(o[i]);
  } else {
    // Neighbouring lanes hold rows 2c and 2c + 1 of w; of every two columns the
    // even lane takes the first with both rows, the odd lane the second.
    const int odd = threadIdx.x & 1;
    float a[8], b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float other = __shfl_xor_sync(0xffffffffu, odd ? v[2 * i] : v[2 * i + 1], 1);
      a[i] = odd ? other : v[2 * i];
      b[i] = odd ? v[2 * i + 1] : other;
      // h is rounded to 16 bits or summed in fp32 far above these errors: the
      // fast exponential and division (2 + 1.2 |a| steps, 2 steps)
      if (SWIGLU) a[i] = __fdividef(a[i], 1.f + __expf(-a[i])) * b[i];
      if (P.gate) {
        const float g = __shfl_sync(0xffffffffu, gate_l, 2 * i + odd);
        a[i] *= g, b[i] *= g;
      }
    }
    out += odd * P.ld + (SWIGLU ? wr >> 1 : wr & ~1);
    left -= odd;
    if (SWIGLU) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (live && 2 * i < left) out[2 * i * P.ld] = narrow<T>(a[i]);
    } else if (P.pack) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (live && 2 * i < left) *reinterpret_cast<uint32_t*>(out + 2 * i * P.ld) = pack2<T>(a[i], b[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (live && 2 * i < left) {
          out[2 * i * P.ld] = narrow<T>(a[i]);
          out[2 * i * P.ld + 1] = narrow<T>(b[i]);
        }
    }
  }
}

template <typename T, bool SWIGLU>
__global__ void __launch_bounds__(kThreads, 1)
    mx4_product_kernel(const __grid_constant__ CUtensorMap tW, const __grid_constant__ CUtensorMap tXa,
                       const __grid_constant__ CUtensorMap tXb, const Params P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Table* B = reinterpret_cast<Table*>(smem + Smem::kTable);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&B->full[i], 1 + kScaleThreads / 32 + (P.gather ? kGatherThreads / 32 : 0));
      mbar_init(&B->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B->d_full[i], 1);
      mbar_init(&B->d_empty[i], kEpiThreads);
    }
    mbar_init(&B->mma_done, 1);
    B->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&B->tmem_base, 512);
  grid_dep_wait();  // codes, scales and grouping come from the kernels before this one
  build_table(P, *B);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B->tmem_base;
  const int total = B->prefix[B->n_groups] * P.m_tiles;
  const int n_k = (P.K + kBK - 1) / kBK;
  const int G = gridDim.x;

  if (warp == 0) {
    // ---------------------------------------------------------- codes
    int g = 0;
    if (lane == 0) {
      bool ok = true;
      for (int w = blockIdx.x; w < total && ok; w += G) {
        const Item it = item_at(P, *B, w);
        const uint32_t tx = static_cast<uint32_t>(kBM + (P.gather ? 0 : it.n16)) * 128u;
        for (int k = 0; k < n_k; ++k, ++g) {
          const int st = g % kStages;
          if (g >= kStages && !wait_bar(B, &B->empty[st], ((g / kStages) - 1) & 1, P, 1)) {
            ok = false;
            break;
          }
          uint8_t* stage = smem + st * Smem::kStage;
          mbar_arrive_expect_tx(&B->full[st], tx);
          tma_load_3d(stage + Smem::kA, &tW, k * (kBK / 2), it.m * kBM, it.slot, &B->full[st]);
          if (P.gather) continue;
          int r = 0;  // n16 rows: boxes of 64, the rest in boxes of 16
          for (; r + kBoxA <= it.n16; r += kBoxA)
            tma_load_2d(stage + Smem::kB + r * 128, &tXa, k * (kBK / 2), it.row0 + r, &B->full[st]);
          for (; r < it.n16; r += kBoxB)
            tma_load_2d(stage + Smem::kB + r * 128, &tXb, k * (kBK / 2), it.row0 + r, &B->full[st]);
        }
      }
    }
    // every copy this warp issued lands before the CTA may exit (bounded wait)
    if (lane == 0) {
      const uint64_t drain = global_timer_ns() + P.timeout_ns;
      for (int n = max(0, g - kStages); n < g; ++n) mbar_wait(&B->full[n % kStages], (n / kStages) & 1, drain);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issue
    // The whole warp walks the loop and one lane issues: the operands then stay
    // in uniform registers, and a stage costs the issuer less than its MMAs take.
    const uint64_t da0 = smem_desc(smem + Smem::kA), db0 = smem_desc(smem + Smem::kB);
    const uint64_t sa0 = scale_desc(smem + Smem::kSfA), sb0 = scale_desc(smem + Smem::kSfB);
    int st = 0, i = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int w = blockIdx.x; w < total && ok; w += G, ++i) {
      const Item it = item_at(P, *B, w);
      const uint32_t id0 = instr_desc_mxf4(it.n16, 0), id1 = instr_desc_mxf4(it.n16, 1);
      const bool wide = it.n16 > 128;
      const int acc = i & 1;
      if (i >= 2 && !wait_bar(B, &B->d_empty[acc], ((i >> 1) - 1) & 1, P, 2)) break;
      tc_fence_after();
      const uint32_t d_tmem = tmem + static_cast<uint32_t>(acc * kAcc);
      for (int k = 0; k < n_k; ++k) {
        if (!wait_bar(B, &B->full[st], ph, P, 3)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t off = static_cast<uint64_t>(st * (Smem::kStage >> 4));
        const uint32_t sf = tmem + static_cast<uint32_t>(2 * kAcc + st * kSfCols);
        const int steps = P.K - k * kBK;  // K values left
        if (elect_one()) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h == 1 && steps <= 128) break;
            tc_copy_scales(sf + 4 * h, sa0 + off + 32 * h);
            tc_copy_scales(sf + 8 + 8 * h, sb0 + off + 64 * h);
            if (wide) tc_copy_scales(sf + 12 + 8 * h, sb0 + off + 64 * h + 32);
          }
#pragma unroll
          for (int s = 0; s < 4; ++s)  // K = 64 per MMA: 32 bytes of a row
            if (64 * s < steps)
              tc_mma_mxf4(d_tmem, da0 + off + 2 * s, db0 + off + 2 * s, (s & 1) ? id1 : id0, sf + 4 * (s >> 1),
                          sf + 8 + 8 * (s >> 1), (k > 0 || s > 0) ? 1u : 0u);
          tc_commit(&B->empty[st]);
          if (k == n_k - 1) tc_commit(&B->d_full[acc]);
        }
        __syncwarp();
        if (++st == kStages) {
          st = 0;
          ph ^= 1;
        }
      }
    }
    // everything issued above completes before the tensor memory is freed
    if (elect_one()) tc_commit(&B->mma_done);
    __syncwarp();
    if (lane == 0) mbar_wait(&B->mma_done, 0, global_timer_ns() + P.timeout_ns);
    __syncwarp();
  } else if (warp < 6) {
    // ---------------------------------------------------------- scales
    const int r = threadIdx.x - 64;
    const int blocks = P.K / kBlock;
    int g = 0;
    bool ok = true;
    for (int w = blockIdx.x; w < total && ok; w += G) {
      const Item it = item_at(P, *B, w);
      const int wr = it.m * kBM + r;
      const uint8_t* rows[3] = {nullptr, nullptr, nullptr};
      if (wr < P.w_rows)
        rows[0] = P.ws + static_cast<size_t>(it.slot) * P.ws_stride + static_cast<size_t>(wr) * P.pitch;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = r + 128 * h;
        if (i >= it.rows) continue;
        const int p = it.row0 + i;
        if (P.gather && it.m == 0 && p < P.n_pairs &&
            static_cast<unsigned>(__ldg(P.pair_token + p)) >= static_cast<unsigned>(P.x_rows))
          report(P.status, kDevBadExpert, p);
        rows[1 + h] = P.xs + static_cast<size_t>(source_row(P, p)) * P.pitch;
      }
      uint4 next[3];
#pragma unroll
      for (int j = 0; j < 3; ++j) next[j] = rows[j] != nullptr ? load_scales(rows[j], 0, blocks) : make_uint4(0, 0, 0, 0);
      for (int pair = 0; 2 * pair < n_k && ok; ++pair) {
        uint4 cur[3];
#pragma unroll
        for (int j = 0; j < 3; ++j) {
          cur[j] = next[j];
          if (rows[j] != nullptr && 2 * pair + 2 < n_k) next[j] = load_scales(rows[j], pair + 1, blocks);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (2 * pair + s >= n_k) break;
          const int st = g % kStages;
          if (g >= kStages && !wait_warp(B, &B->empty[st], ((g / kStages) - 1) & 1, P, 5)) {
            ok = false;
            break;
          }
          uint8_t* stage = smem + st * Smem::kStage;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t wa = s == 0 ? (h == 0 ? cur[0].x : cur[0].y) : (h == 0 ? cur[0].z : cur[0].w);
            const uint32_t w1 = s == 0 ? (h == 0 ? cur[1].x : cur[1].y) : (h == 0 ? cur[1].z : cur[1].w);
            const uint32_t w2 = s == 0 ? (h == 0 ? cur[2].x : cur[2].y) : (h == 0 ? cur[2].z : cur[2].w);
            put_scales(stage + Smem::kSfA + 512 * h, r, wa);
            put_scales(stage + Smem::kSfB + 1024 * h, r, w1);
            if (it.n16 > 128) put_scales(stage + Smem::kSfB + 1024 * h + 512, r, w2);
          }
          arrive_warp(&B->full[st]);  // the stores above are read by the asynchronous scale copies
          ++g;
        }
      }
    }
  } else if (warp >= 14) {
    // ---------------------------------------------------------- gathered x rows
    // Thread i copies 16-byte chunk i % 8 of rows i / 8, i / 8 + 16, ... of a
    // stage to its swizzled place (chunk ^ row % 8).
    if (P.gather) {
      const int c = threadIdx.x & 7, r0 = (threadIdx.x - 448) >> 3;
      const uint32_t dst0 = smem_u32(smem + Smem::kB) + static_cast<uint32_t>(r0 * 128 + ((c ^ (r0 & 7)) << 4));
      const int row_b = P.K / 2;
      int g = 0, told = 0;
      bool ok = true;
      for (int w = blockIdx.x; w < total && ok; w += G) {
        const Item it = item_at(P, *B, w);
        int src[kGatherRows];
#pragma unroll
        for (int j = 0; j < kGatherRows; ++j) {
          const int r = r0 + 16 * j;
          src[j] = r < it.n16 ? source_row(P, it.row0 + min(r, it.rows - 1)) : 0;
        }
        for (int k = 0; k < n_k; ++k, ++g) {
          const int st = g % kStages;
          if (g >= kStages && !wait_warp(B, &B->empty[st], ((g / kStages) - 1) & 1, P, 8)) {
            ok = false;
            break;
          }
          const int col = k * (kBK / 2) + c * 16;
          const bool live = col < row_b;
          const uint8_t* base = P.xc + (live ? col : 0);
          const uint32_t dst = dst0 + static_cast<uint32_t>(st * Smem::kStage);
#pragma unroll
          for (int j = 0; j < kGatherRows; ++j)
            if (r0 + 16 * j < it.n16)
              copy16(dst + j * 16 * 128, base + static_cast<size_t>(src[j]) * row_b, live);
          asm volatile("cp.async.commit_group;" ::: "memory");
          if (g - told >= kGatherLag) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kGatherLag) : "memory");
            arrive_warp(&B->full[told % kStages]);
            ++told;
          }
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      for (; told < g; ++told) arrive_warp(&B->full[told % kStages]);
    }
  } else {
    // ---------------------------------------------------------- epilogue
    const int q = warp & 3;           // TMEM lane quarter of this warp
    const int half = (warp - 6) >> 2;  // takes the 16-column chunks of this parity
    int i = 0;
    for (int w = blockIdx.x; w < total; w += G, ++i) {
      const Item it = item_at(P, *B, w);
      const int acc = i & 1;
      if (!wait_warp(B, &B->d_full[acc], (i >> 1) & 1, P, 6)) break;
      tc_fence_after();
      const uint32_t base = tmem + static_cast<uint32_t>(acc * kAcc) + (static_cast<uint32_t>(q * 32) << 16);
      const int wr = it.m * kBM + q * 32 + lane;
      for (int c0 = 16 * half; c0 < it.rows; c0 += 32) {
        float gate_l = 1.f;
        if (P.gate) {
          const int c = c0 + (lane & 15), p = it.row0 + c;
          if (c < it.rows && p < P.n_pairs) gate_l = __ldg(P.pair_gate + p);
        }
        __syncwarp();
        float v[16];
        tmem_ld16(base + c0, v);
        store16<T, SWIGLU>(P, v, wr, static_cast<long long>(it.row0) + c0, it.rows - c0, gate_l);
      }
      tc_fence_before();
      mbar_arrive(&B->d_empty[acc]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ tensor maps (host)
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    const cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q);
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p)
                                                               : nullptr;
  }();
  return fn;
}

// Bytes [slots][rows][row_bytes] in boxes of box_rows rows of 128 bytes, 128B-swizzled;
// bytes past a row's end read as 0.
bool map_codes(CUtensorMap* m, const uint8_t* base, int row_bytes, int rows, int slots, size_t stride, int dims,
               int box_rows) {
  const cuuint64_t d[3] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(rows),
                           static_cast<cuuint64_t>(slots)};
  const cuuint64_t s[2] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(stride)};
  const cuuint32_t box[3] = {128u, static_cast<cuuint32_t>(box_rows), 1u};
  const cuuint32_t es[3] = {1u, 1u, 1u};
  return encoder()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, dims, const_cast<uint8_t*>(base), d, s, box, es,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T>
const void* kernel_of(bool swiglu) {
  return swiglu ? reinterpret_cast<const void*>(mx4_product_kernel<T, true>)
                : reinterpret_cast<const void*>(mx4_product_kernel<T, false>);
}

const void* kernel_of(int type, bool swiglu) {
  return type == MOE_TYPE_BF16   ? kernel_of<__nv_bfloat16>(swiglu)
         : type == MOE_TYPE_FP16 ? kernel_of<__half>(swiglu)
                                 : kernel_of<float>(swiglu);
}

}  // namespace

cudaError_t mx4_product_init(const Ctx& ctx) {
  (void)ctx;
  for (int type = MOE_TYPE_BF16; type <= MOE_TYPE_FP32; ++type)
    for (int swiglu = 0; swiglu < 2; ++swiglu) {
      const cudaError_t e = cudaFuncSetAttribute(kernel_of(type, swiglu != 0),
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
      if (e != cudaSuccess) return e;
    }
  return cudaSuccess;
}

cudaError_t launch_mx4_product(const Ctx& ctx, const Mx4Args& a, cudaStream_t s) {
  if (encoder() == nullptr) return cudaErrorNotSupported;
  Params P{};
  P.xc = a.x_codes;
  P.xs = a.x_scales;
  P.ws = a.w.scales;
  P.ws_stride = a.w.n_slots > 1 ? a.w.scale_stride : 0;
  P.x_rows = a.x_rows;
  P.w_rows = a.w.rows;
  P.n_slots = a.w.n_slots;
  P.K = a.w.cols;
  P.pitch = mx4_pitch(a.w.cols);
  P.m_tiles = (a.w.rows + kBM - 1) / kBM;
  P.grouped = a.g != nullptr;
  long long groups = 1, rows = a.x_rows;  // at most
  if (a.g != nullptr) {
    P.n_uniq = a.g->n_uniq;
    P.uniq_offset = a.g->uniq_offset;
    P.uniq_slot = a.g->uniq_slot;
    P.pair_token = a.g->pair_token;
    P.pair_gate = a.g->pair_gate;
    P.n_pairs = a.g->n_pairs;
    P.T = a.g->T;
    P.max_uniq = a.g->n_pairs < a.g->E ? a.g->n_pairs : a.g->E;
    groups = P.max_uniq + 1;
    rows = static_cast<long long>(P.n_pairs) + P.T;
  }
  P.shared_slot = a.shared_slot;
  P.gather = a.gather;
  P.gate = a.gate;
  P.pack = a.ld % 2 == 0 && reinterpret_cast<uintptr_t>(a.out) % 4 == 0;
  P.out = a.out;
  P.ld = static_cast<long long>(a.ld);
  P.status = ctx.d_status;
  P.timeout_ns = ctx.timeout_ns;
  const long long items = (rows / kBN + groups) * P.m_tiles;
  if (items > 0x7fffffff) return cudaErrorNotSupported;

  const int row_b = a.w.cols / 2;
  CUtensorMap tw, txa, txb;
  const size_t stride = a.w.n_slots > 1 ? a.w.code_stride : static_cast<size_t>(a.w.rows) * row_b;
  if (!map_codes(&tw, a.w.codes, row_b, a.w.rows, a.w.n_slots, stride, 3, kBM)) return cudaErrorInvalidValue;
  if (a.gather)
    txa = txb = tw;  // not used: the x rows are copied one by one
  else if (!map_codes(&txa, a.x_codes, row_b, a.x_rows, 1, 0, 2, kBoxA) ||
           !map_codes(&txb, a.x_codes, row_b, a.x_rows, 1, 0, 2, kBoxB))
    return cudaErrorInvalidValue;

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items < ctx.num_sms ? items : ctx.num_sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {&tw, &txa, &txb, &P};
  return cudaLaunchKernelExC(&cfg, kernel_of(a.out_type, a.swiglu), args);
}

}  // namespace moe

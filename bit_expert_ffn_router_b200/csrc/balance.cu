// The router's balance loss with its per-expert counts, and the gradient of
// the router's logits.
//
// Over the n tokens that count (mask byte set, at least one logit above
// -infinity), with p_t = softmax(l_t) over the E logits, c_e the (token, j)
// choices of expert e and S_e = sum_t p_te:
//   balance = E / (k n) * sum_e c_e * S_e / n,     z = sum_t lse_t^2 / n,
//   lse_t = log sum_e exp(l_te).
// The counts are whole numbers and take no gradient, so with the upstream
// gradients a of balance and b of z
//   d l_te = p_te * (a E / (k n^2) * (c_e - sum_i c_i p_ti) + b 2/n lse_t)
//            + the gates' part.
// Gates g_j over the k choices (softmax over the chosen logits, renorm) give
// g_j (dg_j - sum_i g_i dg_i) at the chosen experts; gates read from the full
// softmax give g_j dg_j there and -p_te sum_i g_i dg_i at every expert.
//
// Each direction reads the logits once (a token's row lives in the registers
// of a lane group: its maximum, sum and weighted sum are shuffles) and the
// backward pass writes the gradient once; p is recomputed rather than kept,
// since an exponential costs less than eight more bytes per logit. Rows: 4 to
// 32 lanes, 1 to 8 float4 per lane, so short rows share a warp. While a row
// is worked on, the next one's logits, choices and gates are on their way (the
// choices loaded where they are used: forward 38 against 31 us, backward 55
// against 48 us at 65521 tokens x 512 experts).
//
// What bounds it, at 65521 x 512: neither unit is full. The rows' kernel forward
// takes 28 us of the pass's 32 (137 MB, 4.9 TB/s: DRAM 62%, issue slots 68%), the
// backward kernel 47 us (276 MB, 5.8 TB/s: 58% and 64%). A row that does not
// count saves its bytes but not its instructions: with none, 20% and 50% masked
// 32, 31 and 29 us forward, 48, 46 and 42 backward. x 1024: 54 and 90 us (5.0 and 6.0
// TB/s). At 8192 x 512 (13 and 10 us) the start of two launches and the two
// reductions of the forward pass.
//
// Sums over tokens: a lane adds its own experts' p over its rows in fp32 (T /
// 3552 of them at 512 experts), the CTA adds its lane groups in a fixed order, and the finish
// adds the CTAs' partial sums in fp64, in a fixed order too: results do not
// depend on the timing. The counts are integer atomics in shared memory.
#include <type_traits>

#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

// Threads of a CTA, one per SM, by a lane's float4s: 80 registers for a row of up
// to 4 and the next one's loads, 128 for one of 6, 144 (forward) or 168 for one
// of 8. 65521 rows with 768 threads, which spill, then with these:
// 1024 forward 86 and 53 us (384 threads: 61), backward 168 and 89 (448: 96); 768
// forward 74 and 41 (8 slots: 60), backward 130 and 68 (75).
constexpr int row_threads(int slots, bool forward) { return slots > 6 ? (forward ? 448 : 384) : slots > 4 ? 512 : 768; }
constexpr int row_warps(int slots, bool forward) { return row_threads(slots, forward) / 32; }
constexpr int slots_of(int E) { return E > 768 ? 8 : E > 512 ? 6 : 4; }  // at most
constexpr int kFinExperts = 32;  // experts of a CTA of the finish
constexpr int kFinThreads = 256;
static_assert(kMaxE <= 32 * kFinExperts, "a warp adds up the finish's CTAs");

struct BalanceRows {
  const float* logits;
  const int32_t* idx;
  const float* gate;
  const uint8_t* mask;  // or null
  int T, E, k;
  int* status;
};

struct BalanceOut {
  float* stats;     // balance, z, tokens, largest load
  int32_t* counts;  // [E]
  float* prob;      // [E]
};

__device__ __forceinline__ float ex2(float x) {  // 2^x within 2 steps; 0 below the normal range
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kFar = 65536.f;  // below it the sum is scaled by 2^(2^-9) at most

// A token's row in a lane group: slot (i, c) of lane s holds expert
// (i * LANES + s) * 4 + c, or (4 i + c) * LANES + s where rows are read and
// written by single values, so that a warp's are neighbours (65521 x 509
// backward 58 -> 50 us, x 101 22 -> 17; up to 32 experts, whose rows are a few
// sectors either way, it is slower: x 13 5.8 -> 6.8); slots past E hold -infinity.
template <int LANES, int SLOTS, bool VEC>
struct Row {
  float v[SLOTS * 4];

  static constexpr bool kQuads = VEC || LANES * SLOTS <= 8;
  __device__ __forceinline__ static int expert(int i, int c, int sub) {
    return kQuads ? (i * LANES + sub) * 4 + c : (4 * i + c) * LANES + sub;
  }

  __device__ __forceinline__ void load(const float* p, int E, int sub) {
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      if (VEC) {
        const int e = expert(i, 0, sub);
        float4 a = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (e < E) a = ld_plain(reinterpret_cast<const float4*>(p + e));
        v[4 * i] = a.x, v[4 * i + 1] = a.y, v[4 * i + 2] = a.z, v[4 * i + 3] = a.w;
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int e = expert(i, c, sub);
          v[4 * i + c] = e < E ? ld_plain(p + e) : -INFINITY;
        }
      }
    }
  }

  // exp(x - m) as 2^(x log2(e) - m log2(e)), one multiply-add: what the second
  // product is rounded by is the same for the whole row and leaves p alone. It
  // does scale the row's sum by 2^r, |r| <= 2^-25 |m log2(e)|, so rows that lie
  // far out take the difference first: past 1e10 the sum would leave fp32's
  // range, and a row would count as empty.
  struct Exp {
    float m, off;
    bool far;
    __device__ __forceinline__ explicit Exp(float m_) : m(m_ == -INFINITY ? 0.f : m_), off(-m * kLog2e), far(!(fabsf(off) < kFar)) {}
    __device__ __forceinline__ float operator()(float x) const {
      return far ? ex2((x - m) * kLog2e) : ex2(fmaf(x, kLog2e, off));
    }
  };

  // v <- exp(v - max); returns the sum (0: nothing above -infinity; NaN if
  // the row holds one) and the maximum.
  __device__ __forceinline__ float exp_sum(float& m) {
    m = v[0];
#pragma unroll
    for (int i = 1; i < SLOTS * 4; ++i) m = fmaxf(m, v[i]);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const Exp e(m);
    float s = 0.f;
    if (!e.far) {
#pragma unroll
      for (int i = 0; i < SLOTS * 4; ++i) v[i] = ex2(fmaf(v[i], kLog2e, e.off));
    } else {
#pragma unroll
      for (int i = 0; i < SLOTS * 4; ++i) v[i] = e(v[i]);
    }
#pragma unroll
    for (int i = 0; i < SLOTS * 4; ++i) s += v[i];
    return group_sum(s, LANES);
  }
};

// What the CTAs of the rows' kernel leave behind, and the finish's scalars.
struct Partials {
  int pitch;
  float* sum;    // [n][pitch]: pitch = E rounded up to 4
  int32_t* cnt;  // [n][pitch]
  double* z;     // [n]
  int32_t* tok;  // [n]
  double* dot;   // [finish CTAs]
  int32_t* top;
  int32_t* ticket;
};

// Sum over a CTA of WARPS warps, in every thread.
template <int WARPS>
__device__ __forceinline__ double block_sum(double v, double* scratch) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < WARPS ? scratch[threadIdx.x & 31] : 0.0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int WARPS>
__device__ __forceinline__ int block_max(int v, int* scratch) {
  v = __reduce_max_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_max_sync(0xffffffffu, (threadIdx.x & 31) < WARPS ? scratch[threadIdx.x & 31] : 0);
}

// One of a row's choices: choice `sub` in lane `sub` of the row's group.
struct Choice {
  int e;
  float gate, d_gate;
};

// The rows of a lane group, first + stride * i: the row at hand, the next one's
// logits and choices on their way, and the flag (the mask's byte; 0 past the
// end) of the one after it. A row that does not count is not read: row 0
// stands in (the launchers see to it that there is one).
template <int LANES, int SLOTS, bool VEC>
struct Walk {
  const BalanceRows& R;
  const float* d_gate;  // or null: no gates are loaded
  int t, stride, sub;
  uint32_t in, ahead, later;
  Row<LANES, SLOTS, VEC> row, next;
  Choice choice, next_choice;

  __device__ __forceinline__ uint32_t flag(int at) const {
    uint32_t f = at < R.T ? 1u : 0u;
    if (f != 0 && R.mask != nullptr) f = ld_plain(R.mask + at);
    return f;
  }
  __device__ __forceinline__ void fetch(int at, uint32_t f) {
    const size_t r = f != 0 ? at : 0;
    next.load(R.logits + r * R.E, R.E, sub);
    next_choice = {-1, 0.f, 0.f};
    if (sub < R.k) {
      next_choice.e = ld_plain(R.idx + r * R.k + sub);
      if (d_gate != nullptr) {
        next_choice.gate = ld_plain(R.gate + r * R.k + sub);
        next_choice.d_gate = ld_plain(d_gate + r * R.k + sub);
      }
    }
  }
  __device__ __forceinline__ Walk(const BalanceRows& rows, const float* d_gate_, int first, int stride_, int sub_)
      : R(rows), d_gate(d_gate_), t(first - stride_), stride(stride_), sub(sub_) {
    ahead = flag(first);
    later = flag(first + stride);
    fetch(first, ahead);
  }
  __device__ __forceinline__ void step() {
    t += stride;
    in = ahead;
    ahead = later;
    row = next;
    choice = next_choice;
    // A choice that names no expert takes no part, whatever its gate holds.
    // (Asked here; at the sum of the gates it costs registers: 65521 x 256
    // backward 31 -> 33 us, or x 1024 90 -> 105, by the form.)
    if (static_cast<unsigned>(choice.e) >= static_cast<unsigned>(R.E)) choice.gate = choice.d_gate = 0.f;
    fetch(t + stride, ahead);
    later = flag(t + 2 * stride);
  }
};

// stats from the sums over all experts; one thread.
__device__ __forceinline__ void write_stats(float* stats, double dot, double z, int n, int top, int E, int k) {
  const double m = n > 0 ? n : 1;
  stats[0] = static_cast<float>(dot * E / (k * m * m));
  stats[1] = static_cast<float>(z / m);
  stats[2] = static_cast<float>(n);
  stats[3] = static_cast<float>(static_cast<double>(top) * E / (k * m));
}

template <int LANES, int SLOTS, bool VEC>
__global__ void __launch_bounds__(row_threads(SLOTS, true)) balance_rows_kernel(BalanceRows R, Partials P, BalanceOut O) {
  using R_ = Row<LANES, SLOTS, VEC>;
  constexpr int kThreads = row_threads(SLOTS, true), kWarps = row_warps(SLOTS, true);
  extern __shared__ float sums[];  // [kWarps][E]
  __shared__ int hist[kMaxE];
  __shared__ double scratch[kWarps];
  __shared__ int iscratch[kWarps];
  constexpr int kRows = 32 / LANES;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % LANES;
  const int E = R.E, k = R.k;
  for (int e = threadIdx.x; e < E; e += kThreads) hist[e] = 0;
  grid_dep_wait();
  grid_dep_launch();  // the finish sets up meanwhile; it waits for this grid's end
  __syncthreads();

  float acc[SLOTS * 4];
#pragma unroll
  for (int i = 0; i < SLOTS * 4; ++i) acc[i] = 0.f;
  double z = 0;
  int n = 0;
  const int stride = gridDim.x * kWarps * kRows;
  Walk<LANES, SLOTS, VEC> walk(R, nullptr, (blockIdx.x * kWarps + warp) * kRows + lane / LANES, stride, sub);
  // every lane of a warp makes the same number of turns: the shuffles are warp-wide
  for (int t0 = (blockIdx.x * kWarps + warp) * kRows; t0 < R.T; t0 += stride) {
    walk.step();
    const int t = walk.t;
    R_& row = walk.row;
    float m;
    const float s = row.exp_sum(m);
    if (walk.in == 0 || s == 0.f) continue;
    const float r = 1.f / s;
#pragma unroll
    for (int i = 0; i < SLOTS * 4; ++i) acc[i] += row.v[i] * r;
    if (sub == 0) {
      const float lse = m + logf(s);
      z += static_cast<double>(lse) * lse;
      ++n;
    }
    for (int j = sub; j < k; j += LANES) {
      const int e = j == sub ? walk.choice.e : ld_plain(R.idx + static_cast<size_t>(t) * k + j);
      if (static_cast<unsigned>(e) < static_cast<unsigned>(E))
        atomicAdd(&hist[e], 1);
      else
        report(R.status, kDevBadExpert, t * k + j);
    }
  }
  // lane groups of a warp, then the warps
#pragma unroll
  for (int i = 0; i < SLOTS * 4; ++i) {
#pragma unroll
    for (int o = LANES; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    const int e = R_::expert(i / 4, i % 4, sub);
    if (lane < LANES && e < E) sums[warp * E + e] = acc[i];
  }
  z = block_sum<kWarps>(z, scratch);  // its barriers also publish sums and hist
  n = static_cast<int>(block_sum<kWarps>(static_cast<double>(n), scratch));
  if (gridDim.x > 1) {
    for (int e = threadIdx.x; e < E; e += kThreads) {
      float s = 0.f;
      for (int w = 0; w < kWarps; ++w) s += sums[w * E + e];
      P.sum[blockIdx.x * P.pitch + e] = s;
      P.cnt[blockIdx.x * P.pitch + e] = hist[e];
    }
    if (threadIdx.x == 0) {
      if (blockIdx.x == 0) *P.ticket = 0;
      P.z[blockIdx.x] = z;
      P.tok[blockIdx.x] = n;
    }
    return;
  }
  // all rows were this CTA's: finish here
  double dot = 0;
  int top = 0;
  for (int e = threadIdx.x; e < E; e += kThreads) {
    double s = 0;
    for (int w = 0; w < kWarps; ++w) s += sums[w * E + e];
    dot += s * hist[e];
    top = max(top, hist[e]);
    O.prob[e] = static_cast<float>(s / max(n, 1));
    O.counts[e] = hist[e];
  }
  dot = block_sum<kWarps>(dot, scratch);
  top = block_max<kWarps>(top, iscratch);
  if (threadIdx.x == 0) write_stats(O.stats, dot, z, n, top, E, k);
}

// The finish over n_parts CTAs' sums: a CTA takes kFinExperts experts, a thread
// four of them over every 32nd part with all its loads under way at once. The
// CTA that comes last (the rows' kernel set the counter to 0) adds the CTAs'
// scalars, in the CTAs' order whichever it is. Bound by latency, not by its
// bytes: with one load at a time it took 16 us of a 22 us forward call.
__global__ void __launch_bounds__(kFinThreads) balance_finish_kernel(Partials P, BalanceOut O, int n_parts, int E, int k) {
  constexpr int kAcross = kFinExperts / 4, kSlices = kFinThreads / kAcross;
  constexpr int kEach = (kBalanceMaxCtas + kSlices - 1) / kSlices;
  __shared__ double part[kSlices][kFinExperts];
  __shared__ int partc[kSlices][kFinExperts];
  __shared__ bool last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = tid % kAcross, slice = tid / kAcross, e = blockIdx.x * kFinExperts + 4 * c;
  grid_dep_wait();
  double s[4] = {0, 0, 0, 0};
  int n4[4] = {0, 0, 0, 0};
  float4 a[kEach];
  int4 b[kEach];
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    a[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    b[j] = make_int4(0, 0, 0, 0);
    const int i = slice + j * kSlices;
    if (i < n_parts && e < P.pitch) {
      a[j] = *reinterpret_cast<const float4*>(P.sum + i * P.pitch + e);
      b[j] = *reinterpret_cast<const int4*>(P.cnt + i * P.pitch + e);
    }
  }
  int n = 0;  // tokens that count: every warp adds them up for itself
  for (int i = lane; i < n_parts; i += 32) n += P.tok[i];
  n = __reduce_add_sync(0xffffffffu, n);
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    s[0] += a[j].x, s[1] += a[j].y, s[2] += a[j].z, s[3] += a[j].w;
    n4[0] += b[j].x, n4[1] += b[j].y, n4[2] += b[j].z, n4[3] += b[j].w;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    part[slice][4 * c + q] = s[q];
    partc[slice][4 * c + q] = n4[q];
  }
  __syncthreads();
  if (warp == 0) {
    double t = 0;
    int m = 0;
#pragma unroll
    for (int w = 0; w < kSlices; ++w) {
      t += part[w][lane];
      m += partc[w][lane];
    }
    const int x = blockIdx.x * kFinExperts + lane;
    if (x < E) {
      O.prob[x] = static_cast<float>(t / max(n, 1));
      O.counts[x] = m;
    } else {
      t = 0;
      m = 0;
    }
    double dot = t * m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) {
      P.dot[blockIdx.x] = dot;
      P.top[blockIdx.x] = m;
      __threadfence();
      last = atomicAdd(P.ticket, 1) == static_cast<int>(gridDim.x) - 1;
    }
    __syncwarp();
    if (!last) return;
    __threadfence();
    double d = lane < gridDim.x ? __ldcg(P.dot + lane) : 0.0, z = 0;
    m = lane < gridDim.x ? __ldcg(P.top + lane) : 0;
    for (int i = lane; i < n_parts; i += 32) z += P.z[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      d += __shfl_xor_sync(0xffffffffu, d, o);
      z += __shfl_xor_sync(0xffffffffu, z, o);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) write_stats(O.stats, d, z, n, m, E, k);
  }
}

template <int LANES, int SLOTS, bool VEC>
__global__ void __launch_bounds__(row_threads(SLOTS, false))
    balance_backward_kernel(BalanceRows R, const float* stats, const int32_t* counts, const float* d_loss,
                            const float* d_gate, bool renorm,
                            float* __restrict__ d_logits) {
  using R_ = Row<LANES, SLOTS, VEC>;
  constexpr int kRows = 32 / LANES, kWarps = row_warps(SLOTS, false);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % LANES;
  const int E = R.E, k = R.k;
  grid_dep_wait();
  const float n = fmaxf(ld_plain(stats + 2), 1.f);
  const float ca = ld_plain(d_loss) * (static_cast<float>(E) / k) / n / n;
  const float cz = ld_plain(d_loss + 1) * 2.f / n;
  float c[SLOTS * 4];  // ca * counts of this lane's experts
#pragma unroll
  for (int i = 0; i < SLOTS * 4; ++i) {
    const int e = R_::expert(i / 4, i % 4, sub);
    c[i] = e < E ? ca * ld_plain(counts + e) : 0.f;
  }
  const int stride = gridDim.x * kWarps * kRows;
  Walk<LANES, SLOTS, VEC> walk(R, d_gate, (blockIdx.x * kWarps + warp) * kRows + lane / LANES, stride, sub);
  for (int t0 = (blockIdx.x * kWarps + warp) * kRows; t0 < R.T; t0 += stride) {
    walk.step();
    const bool live = walk.t < R.T, in = walk.in != 0;
    const size_t at = live ? walk.t : 0;
    R_& row = walk.row;
    const int32_t* ti = R.idx + at * k;
    const float* tg = R.gate + at * k;
    const float* td = d_gate + at * k;
    const int mine = walk.choice.e;
    const float g = walk.choice.gate, gd = g * walk.choice.d_gate;
    float m;
    const float s = row.exp_sum(m);
    const bool keep = in && s != 0.f;
    const float r = 1.f / s;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < SLOTS * 4; ++i) dot = fmaf(row.v[i], c[i], dot);
    dot = group_sum(dot, LANES) * r;
    // the gates' weighted sum
    float gs = 0.f;
    if (d_gate != nullptr) {
      gs = gd;
      if (LANES < 32)
#pragma unroll 1  // unrolled, 56 bytes a thread spill (65521 x 256 31 -> 38 us)
        for (int j = sub + LANES; j < k; j += LANES) {
          const float more = fmaf(ld_plain(tg + j), ld_plain(td + j), gs);
          if (static_cast<unsigned>(ld_plain(ti + j)) < static_cast<unsigned>(E)) gs = more;
        }
      gs = group_sum(gs, LANES);
    }
    // every expert: p * (c_e + base); a z gradient of 0 leaves an infinite lse out
    const float base = (cz != 0.f ? cz * (m + logf(s)) : 0.f) - dot - (renorm ? 0.f : gs);
    float* out = d_logits + at * E;
    if (live) {
      const float rb = base * r;
#pragma unroll
      for (int i = 0; i < SLOTS; ++i) {
        float o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = keep ? row.v[4 * i + q] * fmaf(c[4 * i + q], r, rb) : 0.f;
        if (VEC) {
          const int e = R_::expert(i, 0, sub);
          if (e < E) *reinterpret_cast<float4*>(out + e) = make_float4(o[0], o[1], o[2], o[3]);
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int e = R_::expert(i, q, sub);
            if (e < E) out[e] = o[q];
          }
        }
      }
    }
    if (d_gate == nullptr) continue;
    __syncwarp();  // the stores above come before the chosen experts' below
    const typename R_::Exp ex(m);
    const float gr = renorm ? gs : 0.f;
    // An expert that a row names more than once takes the sum of its parts, in
    // rank order, from each of the lanes that store it.
    bool again = LANES < 32;
    if (LANES == 32) {  // the lanes without a choice share one value: a match takes time by their number
      const unsigned same = __match_any_sync(0xffffffffu, mine);
      again = __any_sync(0xffffffffu, mine >= 0 && (same & (same - 1)) != 0);
    }
    if (keep) {
      for (int j = sub; j < k; j += LANES) {
        const int e = j == sub ? mine : ld_plain(ti + j);
        if (static_cast<unsigned>(e) >= static_cast<unsigned>(E)) continue;
        float part = gd - g * gr;
        if (again) {
          part = 0.f;
          for (int i = 0; i < k; ++i)
            if (ld_plain(ti + i) == e) part += ld_plain(tg + i) * (ld_plain(td + i) - gr);
        }
        const float p = ex(ld_plain(R.logits + at * E + e)) * r;
        out[e] = fmaf(p, fmaf(ca, static_cast<float>(ld_plain(counts + e)), base), part);
      }
    }
    __syncwarp();
  }
}

bool rows_vec(const void* p, int E) { return E % 4 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Lanes of a row. With few lanes and many values each, a row's shuffles and
// choices are shared by more rows of the warp: 65521 x 128 forward 22 us with 32
// lanes, 14 with 8, backward 33 and 15; 65521 x 64 with 16 and 8 lanes 14.5 and
// 11.8, 17.5 and 10.7. Where a warp has one row at most (3552 on 148 SMs), its
// time alone counts and more lanes are faster. Forward + backward with 8 or 16
// lanes against 32: 300 x 128 7.2 + 5.2 and 7.4 + 3.3 us; at 3552 rows x 128 9.5 +
// 5.3 and 8.2 + 3.5, x 256 10.3 + 5.6 and 8.7 + 3.9; just past them, at 4200, x 80
// 8.9 + 5.0 and 9.5 + 4.7, x 128 9.1 + 5.3 and 9.4 + 4.7, x 256 10.5 + 5.5 and 9.3 +
// 5.3; at 8192 x 128 10.2 + 5.4 and 10.7 + 6.0, x 256 10.8 + 8.2 and 10.9 + 7.0; at
// 20000 x 128 10.2 + 7.8 and 12.0 + 10.1, x 256 11.6 + 10.7 and 13.5 + 11.3. So 256
// experts would gain by a border nearer 12000 rows, by 1.4 us at most.
int lanes_of(const Ctx& ctx, int E, int T) {
  if (E <= 16) return 4;
  if (E <= 64) return 8;
  if (E > 256 || T <= ctx.num_sms * row_warps(slots_of(E), true)) return 32;
  return E <= 128 ? 8 : 16;
}

template <typename F>
cudaError_t by_experts(int E, int lanes_per_row, bool vec, F f) {
  auto with = [&](auto lanes, auto slots) { return vec ? f(lanes, slots, std::true_type()) : f(lanes, slots, std::false_type()); };
  using std::integral_constant;
  switch (lanes_per_row) {
    case 4: return with(integral_constant<int, 4>(), integral_constant<int, 1>());
    case 8:
      if (E <= 32) return with(integral_constant<int, 8>(), integral_constant<int, 1>());
      if (E <= 64) return with(integral_constant<int, 8>(), integral_constant<int, 2>());
      return with(integral_constant<int, 8>(), integral_constant<int, 4>());
    case 16: return with(integral_constant<int, 16>(), integral_constant<int, 4>());
  }
  if (E <= 128) return with(integral_constant<int, 32>(), integral_constant<int, 1>());
  if (E <= 256) return with(integral_constant<int, 32>(), integral_constant<int, 2>());
  if (E <= 512) return with(integral_constant<int, 32>(), integral_constant<int, 4>());
  if (E <= 768) return with(integral_constant<int, 32>(), integral_constant<int, 6>());
  return with(integral_constant<int, 32>(), integral_constant<int, 8>());
}

// One CTA while each of its lane groups has at most kOneCta rows, else up to
// one per SM and the finish. One CTA against several, forward: at 3 rows a group
// 5.0 and 6.9 us (16 experts), 7.2 and 8.8 (512), 7.8 and 8.9 (1024); at 4 rows 5.7 and
// 6.5, 8.2 and 8.7, 9.0 and 8.9; at 6 rows 7.0 and 7.5, 10.1 and 8.3, 11.3 and 8.9.
constexpr int kOneCta = 4;

int balance_ctas(const Ctx& ctx, int E, int lanes, int T) {
  const int per_cta = row_warps(slots_of(E), true) * (32 / lanes);
  if (T <= per_cta * kOneCta) return 1;
  const int want = (T + per_cta - 1) / per_cta;
  const int most = ctx.num_sms < kBalanceMaxCtas ? ctx.num_sms : kBalanceMaxCtas;
  return want < most ? want : most;
}

}  // namespace

size_t balance_ws_bytes(int E) {
  return static_cast<size_t>(kBalanceMaxCtas) * (static_cast<size_t>(E + 3) / 4 * 4 * 8 + 16) + 1024;
}

cudaError_t balance_init(const Ctx& ctx) {
  (void)ctx;
  const void* fns[6] = {reinterpret_cast<const void*>(balance_rows_kernel<32, 4, true>),
                        reinterpret_cast<const void*>(balance_rows_kernel<32, 4, false>),
                        reinterpret_cast<const void*>(balance_rows_kernel<32, 6, true>),
                        reinterpret_cast<const void*>(balance_rows_kernel<32, 6, false>),
                        reinterpret_cast<const void*>(balance_rows_kernel<32, 8, true>),
                        reinterpret_cast<const void*>(balance_rows_kernel<32, 8, false>)};
  for (const void* fn : fns) {
    const cudaError_t e =
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, row_warps(8, true) * kMaxE * 4);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_balance(const Ctx& ctx, const moe_layer_cfg& c, const float* logits, const int32_t* idx,
                           const uint8_t* mask, int T, float* stats, int32_t* counts, float* prob, void* ws,
                           cudaStream_t s) {
  const int E = c.E;
  if (T == 0) {  // no row 0 to stand in for the rows that do not count: logits and idx may be null
    cudaError_t e = cudaMemsetAsync(stats, 0, 4 * sizeof(float), s);
    if (e == cudaSuccess) e = cudaMemsetAsync(counts, 0, E * sizeof(int32_t), s);
    return e == cudaSuccess ? cudaMemsetAsync(prob, 0, E * sizeof(float), s) : e;
  }
  const int lanes_per_row = lanes_of(ctx, E, T), n = balance_ctas(ctx, E, lanes_per_row, T);
  const BalanceRows R{logits, idx, nullptr, mask, T, E, c.k, ctx.d_status};
  const BalanceOut O{stats, counts, prob};
  char* b = static_cast<char*>(ws);
  Partials P;
  P.pitch = (E + 3) / 4 * 4;
  P.z = reinterpret_cast<double*>(b);
  P.sum = reinterpret_cast<float*>(P.z + kBalanceMaxCtas + 32);
  P.cnt = reinterpret_cast<int32_t*>(P.sum + static_cast<size_t>(kBalanceMaxCtas) * P.pitch);
  P.dot = P.z + kBalanceMaxCtas;
  P.tok = P.cnt + static_cast<size_t>(kBalanceMaxCtas) * P.pitch;
  P.top = P.tok + kBalanceMaxCtas;
  P.ticket = P.top + 32;
  const cudaError_t e = by_experts(E, lanes_per_row, rows_vec(logits, E), [&](auto lanes, auto slots, auto vec) {
    return launch_dependent(balance_rows_kernel<lanes.value, slots.value, vec.value>, n, row_threads(slots.value, true),
                            static_cast<size_t>(row_warps(slots.value, true)) * E * 4, s, R, P, O);
  });
  if (e != cudaSuccess || n == 1) return e;
  return launch_dependent(balance_finish_kernel, (E + kFinExperts - 1) / kFinExperts, kFinThreads, 0, s, P, O, n, E, c.k);
}

cudaError_t launch_balance_backward(const Ctx& ctx, const moe_layer_cfg& c, const float* logits, const int32_t* idx,
                                    const float* gate, const uint8_t* mask, int T, const float* stats,
                                    const int32_t* counts, const float* d_loss, const float* d_gate, float* d_logits,
                                    cudaStream_t s) {
  const int E = c.E, lanes_per_row = lanes_of(ctx, E, T);
  const BalanceRows R{logits, idx, gate, mask, T, E, c.k, ctx.d_status};
  const int per_cta = row_warps(slots_of(E), false) * (32 / lanes_per_row);
  const int want = (T + per_cta - 1) / per_cta;
  const int n = want < ctx.num_sms ? want : ctx.num_sms;
  return by_experts(E, lanes_per_row, rows_vec(logits, E) && rows_vec(d_logits, E), [&](auto lanes, auto slots, auto vec) {
    return launch_dependent(balance_backward_kernel<lanes.value, slots.value, vec.value>, n,
                            row_threads(slots.value, false), 0, s, R, stats, counts, d_loss, d_gate, c.renorm != 0,
                            d_logits);
  });
}

}  // namespace moe

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
// The x rows are the M side (a row per tensor-memory lane, so that a thread of
// the epilogue owns an output row and finds gate and up of a channel in
// neighbouring columns), the weight rows the N side, 192 per tile. A group's
// rows are cut into equal tiles of at most 128; where tokens are few, the MMAs'
// unused rows cost nothing beside the weights' way from memory (64 x 128 tiles
// with two stages more: 1 token 8.5 against 9.0 us up and 7.8 against 6.8 down,
// 64 tokens 92.5 against 90.7 and 55.8 against 49.8). With the weight rows on the M side instead, gate and up
// sit in neighbouring lanes, and the exchange, the selects and the short stores
// kept the epilogue four times as long (gate/up of 8192 tokens over 512 experts:
// 374 us at that step, 289 us after it).
//
// One persistent CTA per SM; a ring of stages of 256 K values:
//   warp 0       the weight rows' codes, one TMA box per stage, and the x rows'
//                in boxes of 64 and 16 where they follow each other;
//   warp 1       allocates the tensor memory; copies a stage's scales there and
//                issues its four MMAs;
//   warps 2-7    scales, to shared memory in the order the copies want: pieces
//                of 128 rows x 4 blocks, row r at (r % 32) * 16 + (r / 32) * 4;
//   warps 8-15   epilogue: accumulators from tensor memory (two of them, so that
//                the next item's MMAs overlap), SwiGLU or gate, one rounding;
//   warps 16-19  the x rows that tokens name, 16 bytes per copy (TMA gather loads
//                of four rows took 105 cycles each: 858 us in the place of 626).
//
// What bounds it. With few rows per expert, the weights: 64 tokens over 512
// experts read 613 MB in 91 us. Down products are written at the memory's pace
// (8192 tokens x 10 experts + shared: 1.19 GB in 203 us, 5.9 TB/s). Elsewhere no
// unit is full, and the ring is what is waited for: a stage's way round it takes
// 400 to 530 ns, its MMAs 210, and there are four. Counters:
//   gate/up, 8192 tokens, 512 experts   228 us  L2 to SM 2.50 GB (11.0 TB/s, L2 45%)  tensor 43%  DRAM 55%
//   gate/up, 7919 tokens, 16 experts     98 us           1.11 GB (11.3 TB/s,    41%)         39%       13%
//   7696 x 1536 x 8192, one matrix       67 us           0.72 GB (10.8 TB/s,    36%)         35%        8%
//   8190 x 1536 x 2048, one matrix       24 us           0.18 GB ( 7.8 TB/s,    24%)         25%        5%
// In the last, 3.46 waves of tiles take the time of 4: 4 items x 8 stages x 400 ns
// are 13 us; the other 11 are the launch, the table, the first fill and the last
// epilogue, which have not been told apart. In gate/up of 8192 tokens about 35 ns
// of a stage's 530 are the gathered rows (16-byte copies by the load-store units,
// again for each of the 8 weight tiles) and 30 the epilogue. Where the rows follow
// each other, 16 experts' worth takes 82 us (3.6 PFLOP/s), gathered 96.
//
// Tried and no faster for gate/up of 8192 tokens over 512 experts, about 160 rows
// each and gathered (other cases were not tried): a pair of CTAs on one tile (cta_group::2: half
// the weight traffic, but a stage waits for both, 266 us), x rows that stay for
// all weight tiles of their row tile (three stages of weight rows are left: 238
// us), scale copies in a warp of their own (their completion lands behind the
// MMAs in the queue: 309 against 248 us), a gather warp per stage (372 us), twice
// the gather warps, 128 weight rows per tile with a stage more (277 us), one
// arrival per warp a stage late (260 us).
#include <cuda.h>
#include <cudaTypedefs.h>

#include "moe_internal.cuh"
#include "ptx.cuh"
#include "tc.cuh"

namespace moe {
namespace {

// warps by role
constexpr int kWarpScales = 2, kScaleParts = 3, kScaleWarps = 2 * kScaleParts;
constexpr int kWarpEpi = kWarpScales + kScaleWarps, kEpiWarps = 8;
constexpr int kWarpGather = kWarpEpi + kEpiWarps, kGatherWarps = 4;
constexpr int kThreads = 32 * (kWarpGather + kGatherWarps);
constexpr int kBK = 256;                      // K values per stage: 128 bytes of codes per row
constexpr int kMaxGroups = kMaxE + 1;
constexpr int kList = 256;                    // items of a CTA worked out at its start
constexpr int kGatherThreads = 32 * kGatherWarps;
constexpr uint32_t kTryNs = 20000;            // sleep of one try of a wait
constexpr unsigned long long kDrainNs = 2000000;  // what copies and MMAs in flight get to end, at least
constexpr int kBoxA = 64, kBoxB = 16;         // x rows of the two TMA boxes
constexpr int kBM = 128, kBN = 192;           // x rows and weight rows per tile, at most
constexpr int kStages = 4;
constexpr int kAcc = kBN;                     // TMEM columns of one accumulator
constexpr int kPieces = (kBN + 127) / 128;    // of 128 weight rows
constexpr int kSfCols = 8 + 8 * kPieces;      // TMEM columns of a stage's scales
constexpr int kGatherRows = kBM / (kGatherThreads / 8);  // rows of a stage per gather thread
static_assert(2 * kAcc + kStages * kSfCols <= 512, "tensor memory budget");
static_assert(kScaleParts == 1 + kPieces, "a part for the x rows' scales and one for each piece of weight rows");

// The groups' row tiles, laid end to end: group i's first is prefix[i].
struct Table {
  uint64_t full[kStages];   // TMA (tx), scale warps: a stage is complete
  uint64_t x_full[kStages];  // gather threads (count 128), waited on by the x rows' scale warp
  uint64_t empty[kStages];  // MMA commit: codes and scales read
  uint64_t d_full[2];          // MMA commit: accumulator complete
  uint64_t d_empty[2];         // epilogue warps
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort_flag;
  int n_groups;
  int scan[kThreads / 32];
  int prefix[kMaxGroups + 1];
  int first[kMaxGroups];
  int rows[kMaxGroups];
  int slot[kMaxGroups];
  alignas(16) int4 list[kList];
};

// Shared memory: the stages, the epilogue's staging, the table. (A fifth stage
// does not fit beside the table, in the place of the staging either.)
struct Smem {
  // within a stage
  static constexpr int kX = 0;                 // kBM rows x 128 bytes, 128B-swizzled
  static constexpr int kW = kBM * 128;         // kBN rows x 128 bytes
  static constexpr int kSfX = kW + kBN * 128;  // 2 pieces of 512 bytes (K 0..127, 128..255)
  static constexpr int kSfW = kSfX + 1024;     // 2 x kPieces pieces (K half, 128 weight rows)
  static constexpr int kStage = kSfW + 1024 * kPieces;
  static constexpr int kOut = kStages * kStage;  // 32 rows x 128 bytes for each epilogue warp
  static constexpr int kTable = kOut + kEpiWarps * 4096;
  static constexpr int kBytes = kTable + static_cast<int>(sizeof(Table)) + 1024;
  static_assert(kStage % 1024 == 0 && kW % 1024 == 0, "swizzle atoms start on 1024 bytes");
  static_assert(kBytes <= 227 * 1024, "shared memory budget");
};

struct Params {
  const uint8_t *xc, *xs, *ws;  // x codes; scales
  size_t ws_stride;
  int x_rows, w_rows, n_slots, K, pitch, w_tiles;
  bool grouped;
  const int32_t *n_uniq, *uniq_offset, *uniq_slot, *pair_token;
  const float* pair_gate;
  int n_pairs, T, max_uniq, shared_slot;
  bool gather, gate;
  int vec;                 // bytes that every output row is aligned to: 32, 16 or less
  void* out;
  long long ld;
  int* status;
  unsigned long long timeout_ns;
};

__device__ __forceinline__ bool aborted(const Table* B) {
  return *reinterpret_cast<const volatile int*>(&B->abort_flag) != 0;
}

// Whether a wait that has failed so often should go on: until the context's
// limit has passed or another role has given up; then the place is recorded and
// the CTA's abort flag raised, on which every role leaves its loop.
struct Patience {
  uint64_t deadline = 0;
  int tries = 0;
  __device__ __forceinline__ bool more(Table* B, const Params& P, int where) {
    if (++tries < 8) return true;  // each try sleeps on the barrier for a while
    if (deadline == 0) deadline = global_timer_ns() + P.timeout_ns;
    if (aborted(B)) return false;
    if (global_timer_ns() < deadline) return true;
    report(P.status, kDevTimeout, 200 + where);
    *reinterpret_cast<volatile int*>(&B->abort_flag) = 1;
    return false;
  }
};

__device__ __forceinline__ bool wait_bar(Table* B, uint64_t* bar, uint32_t parity, const Params& P, int where) {
  Patience p;
  while (!mbar_try_wait(bar, parity, kTryNs))
    if (!p.more(B, P, where)) return false;
  return true;
}

// The same for a whole warp, every lane taking the same path afterwards.
__device__ __forceinline__ bool wait_warp(Table* B, uint64_t* bar, uint32_t parity, const Params& P, int where) {
  Patience p;
  while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity, kTryNs)))
    if (!__all_sync(0xffffffffu, p.more(B, P, where))) return false;
  return true;
}

__device__ __forceinline__ int tiles_of(int rows) { return (rows + kBM - 1) / kBM; }

__device__ void build_table(const Params& P, Table& S) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // The groups' entries are loaded before their number is known (the arrays
  // have max_uniq of them): one round trip to memory instead of two.
  const int most = P.grouped ? P.max_uniq + 1 : 1;
  const int per = (most + kThreads - 1) / kThreads;
  const int i0 = tid * per;
  constexpr int kPer = (kMaxGroups + kThreads - 1) / kThreads;
  int from[kPer + 1], slots[kPer];
#pragma unroll
  for (int j = 0; j <= kPer; ++j)
    if (P.grouped && j <= per && i0 + j <= P.max_uniq) {
      from[j] = ld_plain(P.uniq_offset + i0 + j);
      if (j < kPer && i0 + j < P.max_uniq) slots[j] = ld_plain(P.uniq_slot + i0 + j);
    }
  const int nu = P.grouped ? min(max(ld_plain(P.n_uniq), 0), P.max_uniq) : 0;
  const int ng = P.grouped ? nu + (P.shared_slot >= 0 ? 1 : 0) : 1;
  int mine = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = i0 + j;
    if (j >= per || i >= ng) break;
    int first, n, slot;
    if (!P.grouped) {
      first = 0, n = P.x_rows, slot = 0;
    } else if (i < nu) {  // bounds hold even where the grouping's arrays do not make sense
      first = min(max(from[j], 0), P.n_pairs);
      n = max(min(from[j + 1], P.n_pairs) - first, 0);
      slot = slots[j];
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
  for (int i = i0; i < min(i0 + per, ng); ++i) S.prefix[i] += base;
  if (tid == kThreads - 1) {
    S.n_groups = ng;
    S.prefix[ng] = base + mine;
  }
}

struct Item {
  int n0, row0, rows, slot;  // first weight row; first output row and their number; pool slot
  __device__ __forceinline__ int rows16() const { return (rows + 15) & ~15; }
};

// Item w: row tile w / w_tiles with weight tile w % w_tiles. The group is the
// last one whose first tile is at most the tile (empty groups share the next
// one's); its rows are cut into equal tiles of a multiple of 16.
__device__ Item work_out(const Params& P, const Table& S, int w) {
  const int tile = w / P.w_tiles;
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
  it.n0 = (w - tile * P.w_tiles) * kBN;
  it.row0 = S.first[lo] + j * tr;
  it.rows = min(tr, n - j * tr);
  it.slot = S.slot[lo];
  return it;
}

// This CTA's i-th item, blockIdx.x + i * gridDim.x.
__device__ __forceinline__ Item item_at(const Params& P, const Table& S, int i) {
  if (i >= kList) return work_out(P, S, blockIdx.x + i * gridDim.x);
  const int4 v = S.list[i];
  return {v.x, v.y, v.z, v.w};
}

// x row of output row p as the grouping names it; clamp_row makes it one of
// x's (out-of-range tokens are reported by the scale warps). The two are apart,
// and the load is a predicated one, so that its latency is not waited for where
// it is issued.
__device__ __forceinline__ int source_row(const Params& P, int p) {
  int t = P.gather && p >= P.n_pairs ? p - P.n_pairs : p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %2, 0;\n\t"
      "@p ld.global.b32 %0, [%1];\n\t}"
      : "+r"(t)
      : "l"(P.pair_token + p), "r"(P.gather && p < P.n_pairs ? 1 : 0));
  return t;
}
__device__ __forceinline__ int clamp_row(const Params& P, int t) { return min(max(t, 0), P.x_rows - 1); }

// 16 bytes to shared memory without passing through registers; zeros where
// `live` is false.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

// One arrival on `bar` (counted in its initial number) once every copy16 this
// thread has issued is complete.
__device__ __forceinline__ void copy16_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// 32 rows of 16 bytes, to four 32-bit columns of every lane quarter.
__device__ __forceinline__ void tc_copy_scales(uint32_t taddr, uint32_t desc, uint32_t desc_hi) {
  asm volatile(
      "{\n\t.reg .b64 d;\n\t"
      "mov.b64 d, {%1, %2};\n\t"
      "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d;\n\t}" ::"r"(taddr),
      "r"(desc), "r"(desc_hi)
      : "memory");
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

// a, b: low words of the operands' descriptors, whose high words are the same.
__device__ __forceinline__ void tc_mma_mxf4(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc,
                                            uint32_t sfa, uint32_t sfb, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 da, {%1, %3};\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, %4, [%6], [%7], p;\n\t}" ::"r"(
          d_tmem),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(acc), "r"(sfa), "r"(sfb)
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

// The bytes of four K blocks (word i of 16) that are scales of a row with
// `left` blocks from the first word's on; the others 0.
__device__ __forceinline__ uint32_t mask_scales(uint32_t w, int i, int left) {
  const int n = min(max(left - 4 * i, 0), 4);
  return n == 4 ? w : w & ((1u << (8 * n)) - 1u);
}

template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half narrow<__half>(float v) { return __float2half_rn(v); }

// 1 / x of x in [1, infinity], within a step (0 above 2^126).
__device__ __forceinline__ float fast_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  T v[2] = {narrow<T>(a), narrow<T>(b)};
  uint32_t r;
  memcpy(&r, v, 4);
  return r;
}

// Words 8i .. 8i + 7 as one 32-byte store, a whole sector of this lane's row.
__device__ __forceinline__ void store32(uint32_t* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// 16 accumulator columns of one output row (weight rows n .. n + 15) in v to
// `words` 32-bit words of results.
template <typename T, bool SWIGLU>
__device__ __forceinline__ void results16(const float* v, float gate, uint32_t* words) {
  constexpr int kN = SWIGLU ? 8 : 16;
  float o[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    // h is rounded to 16 bits or summed in fp32 far above these errors: the
    // fast exponential and reciprocal (2 + 1.2 |v| steps, 1 step)
    if (SWIGLU)
      o[i] = v[2 * i] * fast_rcp(1.f + __expf(-v[2 * i])) * v[2 * i + 1] * gate;
    else
      o[i] = v[i] * gate;
  }
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < kN; ++i) words[i] = __float_as_uint(o[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) words[i] = pack2<T>(o[2 * i], o[2 * i + 1]);
  }
}

// N words to p, aligned to `vec` bytes.
template <typename T, int N>
__device__ __forceinline__ void store_words(T* p, const uint32_t* w, int vec) {
  if (N % 8 == 0 && vec >= 32) {
#pragma unroll
    for (int i = 0; i < N; i += 8) store32(reinterpret_cast<uint32_t*>(p) + i, w + i);
  } else if (vec >= 16) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *reinterpret_cast<uint4*>(reinterpret_cast<uint32_t*>(p) + i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  } else {
    T v[N * 4 / sizeof(T)];
    memcpy(v, w, N * 4);
#pragma unroll
    for (int i = 0; i < static_cast<int>(N * 4 / sizeof(T)); ++i) p[i] = v[i];
  }
}

// A lane's own row, without staging: `valid` of N words.
template <typename T, int N>
__device__ __forceinline__ void store_row(T* p, const uint32_t* w, int valid, int vec) {
  if (valid == N)
    store_words<T, N>(p, w, vec);
  else
    store_words<T, N / 2>(p, w, vec);
}

// 32 rows of `valid` of N words (lane l has row l's, `rows` rows are real) to
// p, ld elements from row to row, through the warp's shared memory, so that a
// store covers 64 or 128 bytes of a row by neighbouring lanes (16 bytes each;
// the units are swizzled against bank conflicts). With a row per lane instead,
// the fp32 rows of a down product of 8192 tokens took 305 us, staged 238 us.
template <typename T, int N>
__device__ __forceinline__ void store_staged(uint4* stage, const uint32_t* w, T* p, long long ld, int rows, int valid) {
  constexpr int kUnits = N / 4, kRowsAtOnce = 32 / kUnits;
  const int lane = threadIdx.x & 31, u = lane % kUnits;
  auto place = [&](int row, int unit) {
    return stage + row * kUnits + (unit ^ (kUnits == 8 ? row & 7 : (row >> 1) & (kUnits - 1)));
  };
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kUnits; ++i) *place(lane, i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  __syncwarp();
  p += (lane / kUnits) * ld + u * (16 / static_cast<int>(sizeof(T)));
#pragma unroll
  for (int k = 0; k < kUnits; ++k, p += kRowsAtOnce * ld) {
    const int row = k * kRowsAtOnce + lane / kUnits;
    if (row < rows && 4 * u < valid) *reinterpret_cast<uint4*>(p) = *place(row, u);
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
      mbar_init(&B->full[i], 1 + kScaleParts);
      mbar_init(&B->x_full[i], kGatherThreads);
      mbar_init(&B->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B->d_full[i], 1);
      mbar_init(&B->d_empty[i], kEpiWarps);
    }
    mbar_init(&B->mma_done, 1);
    B->abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == 32 * kWarpEpi) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tW) : "memory");
    if (!P.gather) asm volatile("prefetch.tensormap [%0];" ::"l"(&tXa) : "memory");
    if (!P.gather) asm volatile("prefetch.tensormap [%0];" ::"l"(&tXb) : "memory");
  }
  // The x rows that no item fills stay zero: the MMAs take 128 rows whatever an
  // item has, and on zeros they draw less power (8192 tokens, up to 112 rows a
  // tile, long runs under the power cap: 303 -> 288 us a pass).
  if (P.gather) {
    for (int i = threadIdx.x; i < kStages * kBM * 8; i += kThreads)
      reinterpret_cast<uint4*>(smem + i / (kBM * 8) * Smem::kStage + Smem::kX)[i % (kBM * 8)] = make_uint4(0, 0, 0, 0);
    fence_async_smem();
  }
  if (warp == 1) tmem_alloc(&B->tmem_base, 512);
  grid_dep_wait();  // codes, scales and grouping come from the kernels before this one
  build_table(P, *B);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B->tmem_base;
  const int total = B->prefix[B->n_groups] * P.w_tiles;
  const int n_items = total > static_cast<int>(blockIdx.x) ? (total - 1 - blockIdx.x) / gridDim.x + 1 : 0;
  for (int i = threadIdx.x; i < min(n_items, kList); i += kThreads) {
    const Item it = work_out(P, *B, blockIdx.x + i * gridDim.x);
    B->list[i] = make_int4(it.n0, it.row0, it.rows, it.slot);
  }
  __syncthreads();
  const int n_k = (P.K + kBK - 1) / kBK;

  if (warp == 0) {
    // ---------------------------------------------------------- codes
    int g = 0;
    if (lane == 0) {
      bool ok = true;
      for (int i = 0; i < n_items && ok; ++i) {
        const Item it = item_at(P, *B, i);
        const uint32_t tx = static_cast<uint32_t>(kBN + (P.gather ? 0 : it.rows16())) * 128u;
        for (int k = 0; k < n_k; ++k, ++g) {
          const int st = g % kStages;
          if (g >= kStages && !wait_bar(B, &B->empty[st], ((g / kStages) - 1) & 1, P, 1)) {
            ok = false;
            break;
          }
          uint8_t* stage = smem + st * Smem::kStage;
          mbar_arrive_expect_tx(&B->full[st], tx);
          tma_load_3d(stage + Smem::kW, &tW, k * (kBK / 2), it.n0, it.slot, &B->full[st]);
          if (P.gather) continue;
          int r = 0;  // boxes of 64 rows, the rest in boxes of 16
          for (; r + kBoxA <= it.rows16(); r += kBoxA)
            tma_load_2d(stage + Smem::kX + r * 128, &tXa, k * (kBK / 2), it.row0 + r, &B->full[st]);
          for (; r < it.rows16(); r += kBoxB)
            tma_load_2d(stage + Smem::kX + r * 128, &tXb, k * (kBK / 2), it.row0 + r, &B->full[st]);
        }
      }
    }
    // every copy this warp issued lands before the CTA may exit (bounded wait)
    if (lane == 0) {
      const uint64_t drain = global_timer_ns() + max(P.timeout_ns, kDrainNs);
      for (int n = max(0, g - kStages); n < g; ++n) mbar_wait(&B->full[n % kStages], (n / kStages) & 1, drain);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issue
    // The whole warp walks the loop and one lane issues: the operands then stay
    // in uniform registers. Issued by one lane of a diverged warp, a stage took
    // 500 ns whatever its N; now about 310 ns, its MMAs alone 210 ns.
    const uint64_t da0 = smem_desc(smem + Smem::kX), db0 = smem_desc(smem + Smem::kW);
    const uint32_t hi = static_cast<uint32_t>(da0 >> 32);
    const uint32_t a0 = static_cast<uint32_t>(da0), b0 = static_cast<uint32_t>(db0);
    const uint64_t dsx = scale_desc(smem + Smem::kSfX), dsw = scale_desc(smem + Smem::kSfW);
    const uint32_t hs = static_cast<uint32_t>(dsx >> 32);
    const uint32_t sx = static_cast<uint32_t>(dsx), sw = static_cast<uint32_t>(dsw);
    int st = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int i = 0; i < n_items && ok; ++i) {
      const int n = min(kBN, P.w_rows - item_at(P, *B, i).n0);
      const uint32_t id0 = instr_desc_mxf4(n, 0), id1 = instr_desc_mxf4(n, 1);
      const int acc = i & 1;
      if (i >= 2 && !wait_warp(B, &B->d_empty[acc], ((i >> 1) - 1) & 1, P, 2)) break;
      tc_fence_after();
      const uint32_t d_tmem = tmem + static_cast<uint32_t>(acc * kAcc);
      int left = P.K;  // K values
      for (int k = 0; k < n_k; ++k, left -= kBK) {
        if (!wait_warp(B, &B->full[st], ph, P, 3)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t off = static_cast<uint32_t>(st * (Smem::kStage >> 4));
        const uint32_t sf = tmem + static_cast<uint32_t>(2 * kAcc + st * kSfCols);
        if (elect_one()) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            tc_copy_scales(sf + 4 * h, sx + off + 32 * h, hs);
#pragma unroll
            for (int j = 0; j < kPieces; ++j)
              tc_copy_scales(sf + 8 + 4 * (kPieces * h + j), sw + off + 32 * (kPieces * h + j), hs);
          }
#pragma unroll
          for (int s = 0; s < 4; ++s)  // K = 64 per MMA: 32 bytes of a row
            if (s == 0 || 64 * s < left)
              tc_mma_mxf4(d_tmem, a0 + off + 2 * s, b0 + off + 2 * s, hi, (s & 1) ? id1 : id0, sf + 4 * (s >> 1),
                          sf + 8 + 4 * kPieces * (s >> 1), (k > 0 || s > 0) ? 1u : 0u);
          tc_commit(&B->empty[st]);
          if (left <= kBK) tc_commit(&B->d_full[acc]);
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
    if (lane == 0) mbar_wait(&B->mma_done, 0, global_timer_ns() + max(P.timeout_ns, kDrainNs));
    __syncwarp();
  } else if (warp < kWarpEpi) {
    // ---------------------------------------------------------- scales
    // Part 0: the x rows'; part 1 and 2: weight rows 0 .. 127 and 128 .. 191 (a piece
    // has 128, the last 64 repeat the matrix's last row or hold the next tile's: not read).
    // Lane l loads the scales of rows l, l + 32, l + 64, l + 96 for 16 K blocks
    // (two stages) and stores, for each piece of 4 blocks, the four rows' words
    // side by side.
    // Two warps per part take turns, 16 blocks each. Loads run one turn ahead,
    // over the item's end too, and the tokens one item ahead.
    const int part = (warp - kWarpScales) % kScaleParts, turn = (warp - kWarpScales) / kScaleParts;
    const int blocks = P.K / kBlock, n_pairs_k = (n_k + 1) / 2;
    // Rows past the item's end take its last row: nobody reads their results.
    int tok[4];  // x rows of the item that comes next
    auto tokens_of = [&](int i) {
      if (part > 0 || i >= n_items) return;
      const Item it = item_at(P, *B, i);
#pragma unroll
      for (int j = 0; j < 4; ++j) tok[j] = source_row(P, it.row0 + min(lane + 32 * j, it.rows - 1));
    };
    const uint8_t* rows[4];
    auto rows_of = [&](int i) {
      const Item it = item_at(P, *B, i);
      if (part == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = lane + 32 * j;
          if (it.n0 == 0 && r < it.rows && static_cast<unsigned>(tok[j]) >= static_cast<unsigned>(P.x_rows))
            report(P.status, kDevBadExpert, it.row0 + r);
          rows[j] = P.xs + static_cast<size_t>(clamp_row(P, tok[j])) * P.pitch;
        }
      } else {
        const uint8_t* base = P.ws + static_cast<size_t>(it.slot) * P.ws_stride;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          rows[j] = base + static_cast<size_t>(min(it.n0 + 128 * (part - 1) + lane + 32 * j, P.w_rows - 1)) * P.pitch;
      }
    };
    uint4 next[4];
    auto load = [&](int pair) {
#pragma unroll
      for (int j = 0; j < 4; ++j) next[j] = ld_plain(reinterpret_cast<const uint4*>(rows[j]) + pair);
    };
    // this warp's turns: every second one of the items' n_pairs_k each
    const int stride = n_pairs_k >= 2 ? 1 : 2;  // items from one that it meets to the next
    int i = turn / n_pairs_k, pair = turn % n_pairs_k;
    bool ok = true;
    if (i < n_items) {
      tokens_of(i);
      rows_of(i);
      load(pair);
      tokens_of(i + stride);
    }
    while (i < n_items && ok) {
      uint4 cur[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) cur[j] = next[j];
      const int left = blocks - 16 * pair;
      if (left < 16) {  // the row's end: bytes past it are not scales
#pragma unroll
        for (int j = 0; j < 4; ++j)
          cur[j] = make_uint4(mask_scales(cur[j].x, 0, left), mask_scales(cur[j].y, 1, left),
                              mask_scales(cur[j].z, 2, left), mask_scales(cur[j].w, 3, left));
      }
      int i2 = i, pair2 = pair + 2;
      while (pair2 >= n_pairs_k) {
        pair2 -= n_pairs_k;
        ++i2;
      }
      if (i2 < n_items) {
        if (i2 != i) rows_of(i2);
        load(pair2);
        if (i2 != i) tokens_of(i2 + stride);
      }
      int g = i * n_k + 2 * pair;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (2 * pair + s >= n_k) break;
        const int st = g % kStages;
        if (g >= kStages && !wait_warp(B, &B->empty[st], ((g / kStages) - 1) & 1, P, 5)) {
          ok = false;
          break;
        }
        uint8_t* stage = smem + st * Smem::kStage;
        uint4* p0 = reinterpret_cast<uint4*>(stage + (part == 0 ? Smem::kSfX : Smem::kSfW + 512 * (part - 1))) + lane;
        uint4* p1 = p0 + (part == 0 ? 512 : 512 * kPieces) / 16;
        if (s == 0) {
          *p0 = make_uint4(cur[0].x, cur[1].x, cur[2].x, cur[3].x);
          *p1 = make_uint4(cur[0].y, cur[1].y, cur[2].y, cur[3].y);
        } else {
          *p0 = make_uint4(cur[0].z, cur[1].z, cur[2].z, cur[3].z);
          *p1 = make_uint4(cur[0].w, cur[1].w, cur[2].w, cur[3].w);
        }
        // the gathered rows' writes are announced with this warp's own
        if (part == 0 && P.gather && !wait_warp(B, &B->x_full[st], (g / kStages) & 1, P, 7)) {
          ok = false;
          break;
        }
        arrive_warp(&B->full[st]);  // the stores are read by the asynchronous scale copies
        ++g;
      }
      i = i2;
      pair = pair2;
    }
  } else if (warp >= kWarpGather) {
    // ---------------------------------------------------------- gathered x rows
    // Thread i copies 16-byte chunk i % 8 of rows i / 8, i / 8 + 16, ... of a
    // stage to its swizzled place (chunk ^ row % 8).
    if (P.gather) {
      const int c = threadIdx.x & 7, r0 = (threadIdx.x - 32 * kWarpGather) >> 3;
      const uint32_t dst0 = smem_u32(smem + Smem::kX) + static_cast<uint32_t>(r0 * 128 + ((c ^ (r0 & 7)) << 4));
      const int row_b = P.K / 2;
      int g = 0;
      bool ok = true;
      int src[kGatherRows], ahead[kGatherRows];  // this item's rows, the next one's
      auto rows_of = [&](int i) {
        if (i >= n_items) return;
        const Item it = item_at(P, *B, i);
#pragma unroll
        for (int j = 0; j < kGatherRows; ++j) ahead[j] = source_row(P, it.row0 + min(r0 + 16 * j, it.rows - 1));
      };
      rows_of(0);
      for (int i = 0; i < n_items && ok; ++i) {
        const Item it = item_at(P, *B, i);
#pragma unroll
        for (int j = 0; j < kGatherRows; ++j) src[j] = clamp_row(P, ahead[j]);
        rows_of(i + 1);
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
            if (r0 + 16 * j < it.rows)
              copy16(dst + j * 16 * 128, base + static_cast<size_t>(src[j]) * row_b, live);
          copy16_arrive(&B->x_full[st]);
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");  // nothing in flight when the CTA exits
    }
  } else {
    // ---------------------------------------------------------- epilogue
    // A thread has one output row; two warps share a lane quarter, 32 columns in turn.
    const int q = warp & 3;                   // TMEM lane quarter of this warp
    const int half = (warp - kWarpEpi) >> 2;
    const int r = q * 32 + lane;
    constexpr int kOut = SWIGLU ? 2 : 1;      // weight rows per result
    constexpr int kWords = 32 / kOut * sizeof(T) / 4;  // of a row's 32 columns
    uint4* stage_out = reinterpret_cast<uint4*>(smem + Smem::kOut) + 256 * (warp - kWarpEpi);
    for (int i = 0; i < n_items; ++i) {
      const Item it = item_at(P, *B, i);
      const int acc = i & 1, p = it.row0 + r;
      const bool live = r < it.rows;
      const float gate = P.gate && live && p < P.n_pairs ? ld_plain(P.pair_gate + p) : 1.f;
      if (!wait_warp(B, &B->d_full[acc], (i >> 1) & 1, P, 6)) break;
      if (q * 32 < it.rows) {
        tc_fence_after();
        const uint32_t base = tmem + static_cast<uint32_t>(acc * kAcc) + (static_cast<uint32_t>(q * 32) << 16);
        const int n = min(kBN, P.w_rows - it.n0);
        for (int c0 = 32 * half; c0 < n; c0 += 64) {
          float v[32];
          uint32_t words[kWords];
          tmem_ld16(base + c0, v);
          if (c0 + 16 < n) tmem_ld16(base + c0 + 16, v + 16);
          results16<T, SWIGLU>(v, gate, words);
          results16<T, SWIGLU>(v + 16, gate, words + kWords / 2);
          T* dst = static_cast<T*>(P.out) + (it.n0 + c0) / kOut;  // the chunk's place in row 0
          const int valid = c0 + 16 < n ? kWords : kWords / 2;
          if (kWords >= 16 && P.vec >= 16)
            store_staged<T, kWords>(stage_out, words, dst + (it.row0 + q * 32) * P.ld, P.ld, it.rows - q * 32, valid);
          else if (live)
            store_row<T, kWords>(dst + p * P.ld, words, valid, P.vec);
          __syncwarp();
        }
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&B->d_empty[acc]);
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
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, Smem::kBytes);
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
  const size_t mix = reinterpret_cast<uintptr_t>(a.out) | (a.ld * (a.out_type == MOE_TYPE_FP32 ? 4 : 2));
  P.vec = mix % 32 == 0 ? 32 : mix % 16 == 0 ? 16 : 0;
  P.out = a.out;
  P.ld = static_cast<long long>(a.ld);
  P.status = ctx.d_status;
  P.timeout_ns = ctx.timeout_ns;
  P.w_tiles = (a.w.rows + kBN - 1) / kBN;
  const long long items = (rows / kBM + groups) * P.w_tiles;
  if (items > 0x7fffffff) return cudaErrorNotSupported;

  const int row_b = a.w.cols / 2;
  CUtensorMap tw, txa, txb;
  const size_t stride = a.w.n_slots > 1 ? a.w.code_stride : static_cast<size_t>(a.w.rows) * row_b;
  if (!map_codes(&tw, a.w.codes, row_b, a.w.rows, a.w.n_slots, stride, 3, kBN)) return cudaErrorInvalidValue;
  if (a.gather)
    txa = txb = tw;  // not used: the x rows are copied one by one
  else if (!map_codes(&txa, a.x_codes, row_b, a.x_rows, 1, 0, 2, kBoxA) ||
           !map_codes(&txb, a.x_codes, row_b, a.x_rows, 1, 0, 2, kBoxB))
    return cudaErrorInvalidValue;

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items < ctx.num_sms ? items : ctx.num_sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Smem::kBytes;
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

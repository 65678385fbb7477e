// pa_prefill_kernel.cuh -- the kernel of pa_prefill and pa_decode_cascade (pa_prefill.cu)
// and, with changed scores, of pa_prefill_masked (pa_prefill_masked.cu): multi-token
// query over the paged KV cache on the 5th-generation tensor cores (tcgen05): a chunk of new
// tokens per sequence attends to its cached prefix and, causally, to itself.  This is the prefill
// that automatic prefix caching leaves to compute: the second request sharing
// a cached prompt computes only its new tokens
// ("LLM推理优化：vLLM PagedAttention深度解析与工程实践" §4.2;
// "KVcache-learning" s08), attention as §二 of the former page states it.
//
// A query tile packs TQ = 128 / G query tokens x the G query heads of one kv
// head (row m = token m / G, head m % G), so every K/V byte loaded serves the
// whole GQA group.  One CTA holds two such tiles (A and B) and plays four
// roles with its 10 warps (11 with MOD >= 0, below):
//   warp 8      TMA: Q once, then 128-token K and V tiles (one box per block
//               and 64-column half) into rings of 3 (K) and 2 (V) stages, K
//               running one tile ahead of V;
//   warp 9      MMA: one elected lane issues every tcgen05.mma --
//               S_x = Q_x K^T (M 128, N 128, K = head_dim; both operands in
//               shared memory) into TMEM, and O_x += P_x V (N = head_dim, P
//               read from TMEM, V MN-major from the TMA tile), in the order
//               PV_A(j), S_A(j+1), PV_B(j), S_B(j+1), so the tensor core works
//               on one tile while the other tile's softmax runs;
//   warps 0-3   softmax of tile A, warps 4-7 of tile B: each thread owns one
//               row -- tcgen05.ld of its 128 S columns, causal mask, online sum
//               in the log2 domain against a base that moves only when the row
//               max jumps by more than 8 (then O is rescaled in TMEM), P
//               (16-bit; bf16 as a high and a low part) written back over the
//               S columns it has read, where the PV product takes it from.
//               Its FP32 work runs as packed f32x2 instructions (two results
//               each) and its maxima as 3-input max: the softmax is bound by
//               instruction issue, not by the 16 exponentials per clock of the
//               special-function unit (moving a share of them to a polynomial
//               on the FMA pipe made it slower).
// 128-token tiles (the MOD builds take them in 64-token steps) halve the hand-offs a token.
// P over S needs one order the hardware does not give by itself: S_x(j+1)
// may overwrite P_x(j) only once PV_x(j) has completed, so the MMA thread
// waits for PV_x(j)'s commit before it issues S_x(j+1).
// Hand-offs are mbarriers (TMA transaction counts, tcgen05.commit, thread
// arrivals).  Every wait is bounded: one that runs out sets a CTA-wide abort
// flag that ends every role; the CTA then lets its copies and MMAs finish,
// reports PA_DEVERR_TIMEOUT, writes zeros and frees TMEM.
//
// In shared-prefix (cascade) mode the rows are every sequence's decode query and
// they all attend, without a causal mask, to the prefix the sequences share: the
// prefix's K/V are read once per kv head instead of once per sequence, and the
// kernel leaves (o / l, m, l) partials that the decode of each sequence's own
// tokens merges (pa_decode_cascade).  The prefix's KV tiles may be split over
// blockIdx.z so that a batch of few query tiles still fills the GPU; each split
// leaves its own partial.
//
// MOD >= 0 (pa_prefill_masked; bit 0: tanh cap, bit 1: bias by distance): every row sees
// its own span [lo, hi) of tokens, the CTA takes the KV tiles of the spans' union, and
// the scores are changed in registers between tcgen05.ld and the running maximum.
// * Steps of 64 tokens, S apart from P in TMEM: the next step's S is computed while this
//   one's softmax runs, where P over S made each tile's softmax, P V and S one chain
//   (7.5k clocks a 128-token tile; a 64-token step takes 2.8 to 3.5k).  S and P V are
//   issued by a warp each: one warp spent as long on its waits as the tensor core on
//   the products.
// * The cap is a polynomial on the FMA pipe where the row's scores allow it.  The softmax's own
//   exponential already keeps the special-function unit (4 results a clock and SM
//   quarter: 2048 clocks per 128 tokens of both query tiles) nearly as busy as the
//   products keep the tensor core (3584); tanh through ex2 and rcp would triple it.
// * Where few query tiles would leave SMs idle, up to 8 CTAs of a cluster share a query
//   tile's KV tiles; each leaves O and (m, l) in its shared memory, and the cluster merges
//   them row by row through distributed shared memory (no workspace, a fixed order).
// * P goes in as two parts for fp16 too: one part's rounding alone is as large as the
//   output's.  (bf16's two are 16 bits, 0.2% of the outputs round the other way than from P
//   in 32 bits, with no larger error; fp16's are 22.)
// * V rows that no row of the CTA sees are zeroed; a row that comes out non-finite (a
//   V row that other rows see holds infinities or NaN: 0 * inf in the product) is computed
//   again from its own tokens alone.
// Bound: the softmax's instructions and the tensor core about evenly (issue 55%, tensor
// pipe 47%, ALU 47%, FMA 39% busy on the capped bf16 case).  8 x (4096 cached + 512 new),
// 64/8 heads, bf16, cap: 1.02 ms, 575 TFLOP/s (one launch alone, off the power cap, 0.96); 2 x
// 4096 whole prompts, fp16, prefix and bias: 0.96 ms, 608 TFLOP/s (0.88).
#pragma once

#include <cooperative_groups.h>
#include <cudaTypedefs.h>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_score.cuh"
#include "pa_tile.cuh"
#include "pa_umma.cuh"
#include "pa_write.cuh"

namespace pa {
namespace {

constexpr int kRows = 128;                 // rows per query tile (tokens x heads)
constexpr int kQTiles = 2;                 // query tiles per CTA (A, B)
constexpr int kBN = 128;                   // KV tokens per tile (N of the S product)
constexpr int kD = 128;                    // head_dim
constexpr int kKst = 3, kVst = 2;          // K and V ring stages
constexpr int kQHalf = 16384;              // 128 rows x 128 bytes (one 64-column half)
constexpr int kKvHalf = 16384;             // 128 tokens x 128 bytes
constexpr int kKvTile = 2 * kKvHalf;       // one K or V tile: two 64-column halves
constexpr int kQOff = 0;
constexpr int kKOff = kQTiles * 2 * kQHalf;
constexpr int kVOff = kKOff + kKst * kKvTile;
constexpr int kSmemBytes = kVOff + kVst * kKvTile + 1024;   // + alignment slack
constexpr uint32_t kTmemCols = 512;        // S_A, S_B, O_A, O_B: 128 columns each
constexpr int kThreads = 320;
constexpr int kTmaWarp = 8, kMmaWarp = 9;
constexpr int kPvWarp = 10;                // MOD >= 0: a warp of its own issues P V
template <int MOD>
__host__ __device__ constexpr int prefill_threads() { return MOD >= 0 ? kThreads + 32 : kThreads; }
// MOD >= 0: the KV tiles' two 64-token halves are steps of their own, with S and P apart
// in TMEM (S_A, S_B, P_A, P_B: 64 columns each, O_A, O_B: 128), so that the next step's S
// can be computed while this one's softmax runs.
constexpr int kSub = 64;
// MOD >= 0: the order of the CTAs.  Query tiles go out from the last one on, as a causal
// row's work grows with its position and a long CTA that starts last runs alone; a group
// of up to 16 neighbours stays together, for their common K and V in L2.
constexpr int kTileGroup = 16;
constexpr int kMaxSplit = 8;               // MOD >= 0: CTAs that share one query tile's KV tiles

// bf16 keeps 8 significant bits: P goes in as a high and a low bf16 part (two
// PV products, ~16 bits); fp16's 11 bits need one.  P of 128 tokens takes 64
// TMEM columns per part.
template <typename QT, int MOD>
__host__ __device__ constexpr int p_parts() {
  return MOD >= 0 || std::is_same<QT, __nv_bfloat16>::value ? 2 : 1;
}

// ---- packed f32x2 arithmetic: two FP32 results per instruction
__device__ __forceinline__ uint64_t f2pack(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 f2unpack(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t f2fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2sub(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2splat(float v) { return f2pack(v, v); }
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The largest magnitude of three (an fabsf of an asm operand would be an instruction).
__device__ __forceinline__ float fmax3_abs(float a, float b, float c) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

enum {
  kBarQ = 0, kBarKFull = 1, kBarKEmpty = kBarKFull + kKst, kBarVFull = kBarKEmpty + kKst,
  kBarVEmpty = kBarVFull + kVst, kBarSFull = kBarVEmpty + kVst, kBarPFull = kBarSFull + 2,
  kBarODone = kBarPFull + 2, kBarDrain = kBarODone + 2,
  kBarSFree = kBarDrain + 1,                 // MOD >= 0: S is in the softmax's registers
  kBarDrainPv = kBarSFree + 2, kNumBars
};

// MOD >= 0: y -> factor * tanh(y) as factor * y * Q(y^2), Q interpolating tanh(y) / y at the
// Chebyshev points of y^2: of degree 4 for |y| <= 0.625 (1e-7 relative), of degree 6 for
// |y| <= 1 (4e-8).  Evaluated in 32 bits both are 2e-7 off, relative to the score, so the cap
// costs no precision however large it is (degree 4 over all of [0, 1], 7e-6, moved weights
// by 2e-4 at cap 50).  N = 7 holds either: the shorter one's last terms are zero and leave
// its bits alone.
constexpr float kCapNear = 0.625f;
template <int N>
struct CapPoly {
  uint64_t c[N];
  __device__ __forceinline__ explicit CapPoly(float factor, bool near = true) {
    constexpr float kn[7] = {0.9999998807907104f, -0.33331942558288574f, 0.1330437958240509f,
                             -0.05181591212749481f, 0.015043356455862522f, 0.f, 0.f};
    constexpr float kw[7] = {0.9999999403953552f, -0.3333282768726349f, 0.13325075805187225f,
                             -0.053451646119356155f, 0.02027970738708973f, -0.0061943246982991695f,
                             0.0010380251333117485f};
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = f2splat(factor * (N == 5 || near ? kn[i] : kw[i]));
  }
  __device__ __forceinline__ uint64_t operator()(uint64_t y, uint64_t add) const {
    const uint64_t z = f2mul(y, y);
    uint64_t q = c[N - 1];
#pragma unroll
    for (int i = N - 2; i >= 0; --i) q = f2fma(q, z, c[i]);
    return f2fma(q, y, add);
  }
};

// One (query row, head) from its own tokens alone, by a whole warp (MOD >= 0, the
// non-finite rows): lanes split head_dim, one token at a time.
template <typename QT>
__device__ __noinline__ void masked_row(const PrefillArgs& a, const int32_t* table, int row, int h,
                                        int kvh, int pos, int lo, int hi) {
  constexpr int NE = kD / 32;
  const int lane = threadIdx.x & 31, BS = a.block_size;
  const QT* kc = static_cast<const QT*>(a.k_cache);
  const QT* vc = static_cast<const QT*>(a.v_cache);
  const size_t qrow = (static_cast<size_t>(row) * a.num_heads + h) * kD;
  const float slope = a.slopes ? a.slopes[h] * kLog2e : 0.f;
  float q[NE], acc[NE], m2 = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < NE; ++e) {
    q[e] = to_f32<QT>(static_cast<const QT*>(a.q)[qrow + lane + 32 * e]);
    acc[e] = 0.f;
  }
  for (int t = lo; t < hi; ++t) {
    const int blk = table[t / BS];
    const bool ok = blk >= 0 && blk < a.num_blocks;      // else read as zeros
    const size_t at = ok ? ((static_cast<size_t>(blk) * BS + t % BS) * a.num_kv_heads + kvh) * kD : 0;
    float x = 0.f, v[NE];
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      x = ok ? fmaf(q[e], to_f32<QT>(kc[at + lane + 32 * e]), x) : 0.f;
      v[e] = ok ? to_f32<QT>(vc[at + lane + 32 * e]) : 0.f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    x = a.cap_in != 0.f ? a.cap_log2 * tanh_f32(x * a.cap_in) : x * a.scale_log2;
    x = fmaf(-slope, fabsf(static_cast<float>(pos - t)), x);
    const float mn = fmaxf(m2, x);
    const float al = mn == -INFINITY ? 1.f : fast_exp2(m2 - mn);
    const float p = x == -INFINITY ? 0.f : fast_exp2(x - mn);   // NaN stays NaN, the first too
    l = l * al + p;
#pragma unroll
    for (int e = 0; e < NE; ++e) acc[e] = fmaf(p, v[e], acc[e] * al);
    m2 = mn;
  }
#pragma unroll
  for (int e = 0; e < NE; ++e) {
    const float o = l == 0.f ? 0.f : acc[e] / l;
    static_cast<QT*>(a.out)[qrow + lane + 32 * e] = static_cast<QT>(o);
  }
}

__device__ __forceinline__ void prefetch_l1(const void* p) {
  asm volatile("prefetch.global.L1 [%0];" ::"l"(p));
}

// BSC: tokens per block, 0: a.block_size.
template <typename QT, int BSC, int MOD = -1>
__global__ void __launch_bounds__(prefill_threads<MOD>(), 1)
    prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PrefillArgs a) {
  constexpr bool MASK = MOD >= 0, CAP = MASK && (MOD & 1), BIAS = MASK && (MOD & 2);
  const int BS = BSC > 0 ? BSC : a.block_size;
  const int BOXH = BS < 16 ? BS : 16;
  const int NBOX = kBN / BOXH;             // boxes per 64-column half
  constexpr bool kBf16 = std::is_same<QT, __nv_bfloat16>::value;
  constexpr int PARTS = p_parts<QT, MOD>();
  constexpr uint32_t FULL = 0xffffffffu;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kNumBars];
  __shared__ uint32_t tmem_base_slot;
  __shared__ int abort_flag;
  __shared__ int span_lo[8], span_hi[8];     // MASK: the union of each softmax warp's spans

  int tile2 = blockIdx.x, kvh = blockIdx.y, seq = blockIdx.z;
  int nsplit = 1, rank = 0;                  // MASK: CTAs that share the KV tiles of one query tile
  if constexpr (MASK) {                      // grid (splits x tile group x kv heads, sequences, groups)
    nsplit = static_cast<int>(cooperative_groups::this_cluster().num_blocks());
    rank = blockIdx.x % nsplit;
    const int ng = gridDim.x / (nsplit * a.num_kv_heads), bx = blockIdx.x / nsplit;
    kvh = bx / ng;
    seq = blockIdx.y;
    tile2 = static_cast<int>((gridDim.z - blockIdx.z) * ng - 1 - bx % ng);
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = a.num_heads / a.num_kv_heads;
  const int TQ = kRows / G;

  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  if (tid == kTmaWarp * 32) {
    for (int i = 0; i < kNumBars; ++i) {
      const bool from_threads = (i >= kBarPFull && i < kBarPFull + 2) ||
                                (i >= kBarSFree && i < kBarSFree + 2);
      mbar_init(bar(i), from_threads ? kRows : 1);
    }
    abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }

  // Wait first, then release the dependent grid: a kernel launched behind this
  // one may then read whatever the kernels before this one wrote.
  griddep_wait();
  griddep_launch_dependents();

  const bool cascade = a.cascade_rows > 0;   // shared-prefix partials, no causal mask
  const int q0 = cascade ? 0 : a.query_start[seq];
  const int q_len = cascade ? a.cascade_rows : a.query_start[seq + 1] - q0;
  const int L = cascade ? a.cascade_len : a.seq_lens[seq];
  const bool bad_rows = MASK && (q0 < 0 || q_len < 0 || q0 > a.total_q - q_len);
  const bool bad_len = q_len < 0 || bad_rows || (!cascade && L < q_len) || L < 0 ||
                       static_cast<long long>(L) > static_cast<long long>(a.max_blocks) * BS;
  if (bad_len) {
    if (tid == 0 && a.err_flag) report_error(a.err_flag, kErrSeqLen);
    return;
  }
  const int row0 = tile2 * kQTiles * TQ;     // first query token of tile A
  if (row0 >= q_len) return;                 // this sequence has fewer query tiles
  const int row_end = min(row0 + kQTiles * TQ, q_len);
  const int pos_last = cascade ? L - 1 : L - q_len + row_end - 1;
  int t_lo = 0;                              // first KV tile of this CTA
  int ntiles = pos_last >= 0 ? pos_last / kBN + 1 : 0;
  // MASK: this thread's row and the tokens it sees; the union of the CTA's rows
  int row_lo = 0, row_hi = 0, row_pos = -1, u_lo = 0, u_hi = 0;
  if constexpr (MASK) {
    if (warp < 8) {
      const int r = (tid % kRows) / G, tok = row0 + (warp / 4) * TQ + r;
      if (r < TQ && tok < q_len) {
        row_pos = L - q_len + tok;
        const Span sp = seen_span(a.kv_start ? a.kv_start[q0 + tok] : 0, row_pos, a.window,
                                  a.prefix_lens ? a.prefix_lens[seq] : 0, L);
        if (sp.lo < sp.hi) {
          row_lo = sp.lo;
          row_hi = sp.hi;
        }
      }
      const int wl = __reduce_min_sync(FULL, row_lo < row_hi ? row_lo : INT_MAX);
      const int wh = __reduce_max_sync(FULL, row_hi);
      if (lane == 0) {
        span_lo[warp] = wl;
        span_hi[warp] = wh;
      }
    }
  }
  if (cascade && a.cascade_splits > 1) {     // the prefix split over blockIdx.z
    const int per = (ntiles + a.cascade_splits - 1) / a.cascade_splits;
    t_lo = min(ntiles, seq * per);
    ntiles = min(ntiles - t_lo, per);
  }

  const uint32_t sraw = smem_u32(smem_raw);
  const uint32_t sbase = (sraw + 1023u) & ~1023u;
  auto q_s = [&](int x) { return sbase + kQOff + static_cast<uint32_t>(x * 2 * kQHalf); };
  auto k_s = [&](int st) { return sbase + kKOff + static_cast<uint32_t>(st * kKvTile); };
  auto v_s = [&](int st) { return sbase + kVOff + static_cast<uint32_t>(st * kKvTile); };
  const int32_t* table = a.block_tables + (cascade ? 0 : static_cast<size_t>(seq) * a.max_blocks);
  volatile int* abort = &abort_flag;

  // the first table entries come while the spans do
  if (MASK && warp == kTmaWarp && 32 * lane < a.max_blocks) prefetch_l1(table + 32 * lane);
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&tmem_base_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = tmem_base_slot;
  if constexpr (MASK) {
    u_lo = span_lo[0];
    u_hi = span_hi[0];
    for (int w = 1; w < 8; ++w) {
      u_lo = min(u_lo, span_lo[w]);
      u_hi = max(u_hi, span_hi[w]);
    }
    t_lo = u_lo < u_hi ? u_lo / kBN : 0;
    ntiles = u_lo < u_hi ? (u_hi - 1) / kBN + 1 - t_lo : 0;
    const int per = (ntiles + nsplit - 1) / nsplit, skip = min(ntiles, rank * per);
    t_lo += skip;
    ntiles = min(ntiles - skip, per);
  }
  // MASK: steps [i0, i1) of 64 tokens, counted from the first KV tile
  const int i0 = MASK && ntiles > 0 ? max(0, u_lo / kSub - t_lo * (kBN / kSub)) : 0;
  const int i1 = MASK && ntiles > 0
                     ? min((u_hi - 1) / kSub + 1 - t_lo * (kBN / kSub), ntiles * (kBN / kSub))
                     : i0;
  // S_x (f32) and, over it once read, P_x (16-bit pairs per column; bf16's low
  // part in columns 64..127)
  auto t_s = [&](int x) { return tmem + static_cast<uint32_t>((MASK ? kSub : 128) * x); };
  auto t_p = [&](int x) { return tmem + static_cast<uint32_t>(2 * kSub + kSub * x); };   // MASK
  auto t_o = [&](int x) { return tmem + 256u + static_cast<uint32_t>(128 * x); };

  // softmax state (warps 0-7), kept here for the epilogue
  const int x_me = warp < 8 ? warp / 4 : 0;
  const int row_me = tid % kRows;
  const int r_tok = row_me / G;
  const int tok_me = row0 + x_me * TQ + r_tok;          // query token within the chunk
  const bool row_valid = warp < 8 && tok_me < q_len && (!MASK || r_tok < TQ);
  float m_run = -INFINITY, l_run = 0.f;
  int armed_k[kKst], armed_v[kVst];          // TMA warp: last tile issued into each stage
#pragma unroll
  for (int i = 0; i < kKst; ++i) armed_k[i] = -1;
#pragma unroll
  for (int i = 0; i < kVst; ++i) armed_v[i] = -1;

  if (warp == kTmaWarp) {
    // ------------------------------------------------------------ TMA producer
    const uint64_t pol = policy_evict_first();
    if (lane == 0) {
      mbar_arrive_expect_tx(bar(kBarQ), kQTiles * 2 * (MASK ? TQ * G * 128 : kQHalf));
      for (int x = 0; x < kQTiles; ++x)        // rows past the chunk: zero-filled or unused
        for (int h = 0; h < 2; ++h)
          tma_load_3d(q_s(x) + h * kQHalf, &tm_q, h * 64, kvh * G, q0 + row0 + x * TQ,
                      bar(kBarQ), pol);
    }
    // one tile's cache rows, lane b holding box b's (past the cache: the box
    // is zero-filled, as is one that no row of the CTA sees, whose block may be gone)
    auto tile_rows = [&](int j) {
      int row = a.num_blocks * BS;
      if (lane < NBOX) {
        const int t0 = (t_lo + j) * kBN + lane * BOXH;
        if (t0 < L && (!MASK || (t0 + BOXH > u_lo && t0 < u_hi))) {
          const int blk = __ldg(table + t0 / BS);
          if (blk >= 0 && blk < a.num_blocks) row = blk * BS + t0 % BS;
          else if (a.err_flag) report_error(a.err_flag, kErrBlockId);
        }
      }
      return row;
    };
    // lane b loads box b (one lane for all of them took ~100 clocks a box, which kept V
    // from arriving in time)
    auto load_tile = [&](const CUtensorMap* map, uint32_t dst, int row, uint32_t full) {
      if (lane == 0) mbar_arrive_expect_tx(full, kKvTile);
      __syncwarp();
      if (lane < NBOX) {
        for (int h = 0; h < 2; ++h)
          tma_load_3d(dst + static_cast<uint32_t>(h * kKvHalf + lane * BOXH * 128), map, h * 64,
                      kvh, row, full, pol);
      }
      __syncwarp();
    };
    // K(j), then V(j - 1): the S product of a tile comes one step before its PV
    int row_prev = 0;
    for (int j = 0; j <= ntiles; ++j) {
      int row = 0;
      if (j < ntiles) {
        const int ks = j % kKst;
        if (j >= kKst) {
          bool ok = true;
          if (lane == 0) ok = mbar_wait_abortable(bar(kBarKEmpty + ks), ((j / kKst) - 1) & 1,
                                                  a.timeout_ns, abort);
          if (!__shfl_sync(FULL, ok, 0)) break;
        }
        row = tile_rows(j);
        if (!(a.inject == 1 && j == 0)) {    // test hook: K(0) never arrives
          armed_k[ks] = j;
          load_tile(&tm_k, k_s(ks), row, bar(kBarKFull + ks));
        }
      }
      if (j >= 1) {
        const int jv = j - 1, vs = jv % kVst;
        if (jv >= kVst) {
          bool ok = true;
          if (lane == 0) ok = mbar_wait_abortable(bar(kBarVEmpty + vs), ((jv / kVst) - 1) & 1,
                                                  a.timeout_ns, abort);
          if (!__shfl_sync(FULL, ok, 0)) break;
        }
        armed_v[vs] = jv;
        load_tile(&tm_v, v_s(vs), row_prev, bar(kBarVFull + vs));
      }
      row_prev = row;
    }
  } else if (warp == kMmaWarp || warp == kPvWarp) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t idesc_s = umma_idesc_f16(kBf16, false, kRows, kBN);
    const uint32_t idesc_o = umma_idesc_f16(kBf16, true, kRows, kD);
    auto wait1 = [&](int b, uint32_t parity) {   // the vote keeps the control flow uniform
      return __all_sync(FULL, mbar_wait_abortable(bar(b), parity, a.timeout_ns, abort)) != 0;
    };
    // operand descriptors of the first stage / tile; a K slice, stage or tile
    // moves only the start-address field (bytes >> 4), which no offset here
    // carries out of
    const uint64_t dq0 = umma_desc_sw128(q_s(0), 16, 1024);
    const uint64_t dk0 = umma_desc_sw128(k_s(0), 16, 1024);
    const uint64_t dv0 = umma_desc_sw128(v_s(0), kKvHalf, 1024);
    auto issue_s = [&](int x, int j) {       // S_x = Q_x K_j^T
      tc_fence_after_sync();
      const uint64_t qd = dq0 + static_cast<uint64_t>(x * (2 * kQHalf >> 4));
      const uint64_t kd = dk0 + static_cast<uint64_t>((j % kKst) * (kKvTile >> 4));
#pragma unroll
      for (int kk = 0; kk < kD / 16; ++kk) {
        const uint32_t qoff = static_cast<uint32_t>(((kk >> 2) * kQHalf + (kk & 3) * 32) >> 4);
        const uint32_t koff = static_cast<uint32_t>(((kk >> 2) * kKvHalf + (kk & 3) * 32) >> 4);
        umma_f16_ss_warp(t_s(x), qd + qoff, kd + koff, idesc_s, kk > 0);
      }
      umma_commit_warp(bar(kBarSFull + x));
    };
    auto issue_pv = [&](int x, int j) {      // O_x += P_x V_j, P from TMEM
      tc_fence_after_sync();
      const uint64_t vd = dv0 + static_cast<uint64_t>((j % kVst) * (kKvTile >> 4));
#pragma unroll
      for (int part = 0; part < PARTS; ++part) {
#pragma unroll
        for (int kk = 0; kk < kBN / 16; ++kk)
          umma_f16_ts_warp(t_o(x), t_s(x) + static_cast<uint32_t>(part * 64 + kk * 8),
                           vd + static_cast<uint32_t>(kk * 16 * 128 >> 4), idesc_o,
                           j > 0 || part > 0 || kk > 0);
      }
      umma_commit_warp(bar(kBarODone + x));
    };
    if constexpr (MASK) {
      const uint32_t idesc_s64 = umma_idesc_f16(kBf16, false, kRows, kSub);
      auto sub_s = [&](int x, int i) {       // S_x = Q_x K^T over step i's 64 tokens
        tc_fence_after_sync();
        const uint64_t qd = dq0 + static_cast<uint64_t>(x * (2 * kQHalf >> 4));
        const uint64_t kd = dk0 + static_cast<uint64_t>((((i >> 1) % kKst) * kKvTile +
                                                         (i & 1) * kSub * 128) >> 4);
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk) {
          const uint32_t qoff = static_cast<uint32_t>(((kk >> 2) * kQHalf + (kk & 3) * 32) >> 4);
          const uint32_t koff = static_cast<uint32_t>(((kk >> 2) * kKvHalf + (kk & 3) * 32) >> 4);
          umma_f16_ss_warp(t_s(x), qd + qoff, kd + koff, idesc_s64, kk > 0);
        }
        umma_commit_warp(bar(kBarSFull + x));
      };
      auto sub_pv = [&](int x, int i) {      // O_x += P_x V: high parts, then low parts
        tc_fence_after_sync();
        const uint64_t vd = dv0 + static_cast<uint64_t>((((i >> 1) % kVst) * kKvTile +
                                                         (i & 1) * kSub * 128) >> 4);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
#pragma unroll
          for (int kk = 0; kk < kSub / 16; ++kk)
            umma_f16_ts_warp(t_o(x), t_p(x) + static_cast<uint32_t>(part * 32 + kk * 8),
                             vd + static_cast<uint32_t>(kk * 16 * 128 >> 4), idesc_o,
                             i > i0 || part > 0 || kk > 0);
        }
        umma_commit_warp(bar(kBarODone + x));
      };
      // S and P V each from a warp of its own: one warp for both spent as long on its
      // waits as the tensor core on the products
      if (warp == kMmaWarp) {
        bool ok = wait1(kBarQ, 0);
        for (int i = i0; ok && i < i1; ++i) {
          const int j = i >> 1, n = i - i0;
          if ((i == i0 || !(i & 1)) && !(ok = wait1(kBarKFull + j % kKst, (j / kKst) & 1))) break;
          if (n > 0 && !(ok = wait1(kBarSFree + 0, (n - 1) & 1))) break;
          sub_s(0, i);
          if (n > 0 && !(ok = wait1(kBarSFree + 1, (n - 1) & 1))) break;
          sub_s(1, i);
          if ((i & 1) || i + 1 == i1) umma_commit_warp(bar(kBarKEmpty + j % kKst));
        }
      } else {
        bool ok = true;
        for (int i = i0; ok && i < i1; ++i) {
          const int j = i >> 1, vs = j % kVst, n = i - i0;
          if (i == i0 || !(i & 1)) {         // the tile's V, at its first step
            if (!(ok = wait1(kBarVFull + vs, (j / kVst) & 1))) break;
            const int first = max(0, u_lo - (t_lo + j) * kBN), last = min(kBN, u_hi - (t_lo + j) * kBN);
            if (first > 0 || last < kBN) {   // rows that no row of the CTA sees: zeros
              for (int idx = lane; idx < kBN * 16; idx += 32) {
                const int row = idx / 16, ch = idx % 16;
                if (row >= first && row < last) continue;
                const uint32_t addr = v_s(vs) + (ch >> 3) * kKvHalf + row * 128 + (ch & 7) * 16;
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0u) : "memory");
              }
              fence_proxy_async_smem();
              __syncwarp();
            }
          }
          if (!(ok = wait1(kBarPFull + 0, n & 1))) break;
          sub_pv(0, i);
          if (!(ok = wait1(kBarPFull + 1, n & 1))) break;
          sub_pv(1, i);
          if ((i & 1) || i + 1 == i1) umma_commit_warp(bar(kBarVEmpty + vs));
        }
      }
    }
    bool ok = !MASK && wait1(kBarQ, 0);
    if (ok && ntiles > 0) {
      ok = wait1(kBarKFull, 0);
      if (ok) {
        issue_s(0, 0);
        issue_s(1, 0);
        umma_commit_warp(bar(kBarKEmpty));                  // K(0) is read by now
      }
    }
    for (int j = 0; ok && j < ntiles; ++j) {
      const int vs = j % kVst;
      if (!(ok = wait1(kBarVFull + vs, (j / kVst) & 1))) break;
      if ((t_lo + j) * kBN + kBN > L) {
        // V rows at or past the sequence end: zero them so that poisoned or
        // stale slots cannot turn 0 * x into NaN inside the MMA
        const int first = max(0, L - (t_lo + j) * kBN);
        for (int idx = lane; idx < (kBN - first) * 16; idx += 32) {
          const int row = first + idx / 16, ch = idx % 16;
          const uint32_t addr = v_s(vs) + (ch >> 3) * kKvHalf + row * 128 + (ch & 7) * 16;
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0u) : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (!(ok = wait1(kBarPFull + 0, j & 1))) break;
      issue_pv(0, j);
      if (j + 1 < ntiles) {
        if (!(ok = wait1(kBarKFull + (j + 1) % kKst, ((j + 1) / kKst) & 1))) break;
        if (!(ok = wait1(kBarODone + 0, j & 1))) break;   // P_A(j) consumed
        issue_s(0, j + 1);
      }
      if (!(ok = wait1(kBarPFull + 1, j & 1))) break;
      issue_pv(1, j);
      umma_commit_warp(bar(kBarVEmpty + vs));               // V(j) is read by now
      if (j + 1 < ntiles) {
        if (!(ok = wait1(kBarODone + 1, j & 1))) break;   // P_B(j) consumed
        issue_s(1, j + 1);
        umma_commit_warp(bar(kBarKEmpty + (j + 1) % kKst));  // K(j+1) read
      }
    }
  } else {
    // ------------------------------------------------------------ softmax (tile x_me)
    const int x = x_me;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int pos = !row_valid ? -1 : (cascade ? L - 1 : L - q_len + tok_me);
    float slope = 0.f;
    if (BIAS && row_valid) slope = a.slopes[kvh * G + row_me % G] * kLog2e;
    if constexpr (MASK) {
      constexpr int NC = kSub;
      for (int i = i0; i < i1; ++i) {
        const int n = i - i0;
        if (!mbar_wait_abortable(bar(kBarSFull + x), n & 1, a.timeout_ns, abort)) break;
        tc_fence_after_sync();
        float sv[NC];
#pragma unroll
        for (int q = 0; q < NC / 32; ++q) {
          float v[32];
          tmem_ld32(t_s(x) + lane_off + 32 * q, v);
#pragma unroll
          for (int e = 0; e < 32; ++e) sv[32 * q + e] = v[e];
        }
        tmem_wait_ld();
        tc_fence_before_sync();
        mbar_arrive(bar(kBarSFree + x));     // the next step's S may come

        const int t_base = t_lo * kBN + i * kSub;            // the token of column 0
        // every column seen by every row of the warp; else a bit per seen column (a test
        // of two bounds per element would cost as much as the rest of the softmax)
        const bool off = row_lo >= row_hi;   // this row sees nothing
        const bool full = __all_sync(FULL, !row_valid || (row_lo <= t_base && row_hi >= t_base + NC));
        uint32_t bits[NC / 32];
#pragma unroll
        for (int q = 0; q < NC / 32; ++q) {
          const int from = max(0, min(32, row_lo - t_base - 32 * q));
          const int to = max(0, min(32, row_hi - t_base - 32 * q));
          bits[q] = from < to ? (FULL >> (32 - (to - from))) << from : 0u;
        }
        auto seen = [&](int c) { return ((bits[c / 32] >> (c % 32)) & 1u) != 0; };

        // The scores.  The cap as a polynomial where every |score| that the row sees is within
        // its range (it grows with the score, so the maximum can be taken before it and
        // the polynomial left to the pass that makes P), else tanh over its whole range: each
        // row's own choice, so that its bits do not depend on what other rows see.  Warps
        // whose rows all take the short polynomial run it alone.  The bias by packed adds
        // where all of the step is on one side of pos.
        float factor = a.scale_log2;         // what turns sv into scores in log2 units
        bool near = false, own = false;      // this row: the short polynomial; one of the two
        bool poly = false;                   // the short one in every row of the warp
        if constexpr (CAP) {
          float big[2] = {0.f, 0.f};
          if (!full) {                       // what the row does not see has no say
#pragma unroll
            for (int c = 0; c < NC; ++c) sv[c] = seen(c) ? sv[c] : 0.f;
          }
#pragma unroll
          for (int c = 0; c < NC; c += 2)
            big[(c >> 1) & 1] = fmax3_abs(big[(c >> 1) & 1], sv[c], sv[c + 1]);
          const float most = off ? 0.f : fmaxf(big[0], big[1]) * fabsf(a.cap_in);
          near = most <= kCapNear;
          own = most <= 1.f;
          poly = __all_sync(FULL, near);
          factor = a.cap_in;
          if (!own) {
#pragma unroll
            for (int c = 0; c < NC; ++c) sv[c] = a.cap_log2 * tanh_f32(sv[c] * a.cap_in);
            factor = 1.f;
          }
        }
        if constexpr (BIAS) {
          const int d0 = t_base - row_pos;   // column c is at distance |c + d0|
          const bool before = d0 + NC - 1 <= 0;
          if (__all_sync(FULL, off || before) || __all_sync(FULL, off || d0 >= 0)) {
            const uint64_t f2 = f2splat(factor);
            const float sg = before ? slope : -slope;
            const uint64_t step = f2splat(2.f * sg);
#pragma unroll
            for (int c32 = 0; c32 < NC; c32 += 32) {
              const float b0 = sg * static_cast<float>(d0 + c32);
              uint64_t b = f2pack(b0, b0 + sg);
              if (CAP && poly) {
                const CapPoly<5> cap(a.cap_log2);
#pragma unroll
                for (int c = c32; c < c32 + 32; c += 2) {
                  const float2 y = f2unpack(cap(f2mul(f2pack(sv[c], sv[c + 1]), f2), b));
                  sv[c] = y.x;
                  sv[c + 1] = y.y;
                  b = f2add(b, step);
                }
              } else {
                const CapPoly<7> cap(a.cap_log2, near);
#pragma unroll
                for (int c = c32; c < c32 + 32; c += 2) {
                  const uint64_t s2 = f2pack(sv[c], sv[c + 1]);
                  float2 y = f2unpack(f2fma(s2, f2, b));
                  if constexpr (CAP) {
                    const float2 yc = f2unpack(cap(f2mul(s2, f2), b));
                    y = own ? yc : y;
                  }
                  sv[c] = y.x;
                  sv[c + 1] = y.y;
                  b = f2add(b, step);
                }
              }
            }
          } else {
            const float d = static_cast<float>(d0);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const float y = CAP && own ? a.cap_log2 * tanh_f32(sv[c] * factor) : sv[c] * factor;
              sv[c] = fmaf(-slope, fabsf(d + static_cast<float>(c)), y);
            }
          }
          own = poly = false;
          factor = 1.f;
        }

        float mx[2] = {-INFINITY, -INFINITY};
        if (full && (CAP ? a.cap_in : a.scale_log2) >= 0.f) {     // so is every row's factor
#pragma unroll
          for (int c = 0; c < NC; c += 2)
            mx[(c >> 1) & 1] = fmax3(mx[(c >> 1) & 1], sv[c], sv[c + 1]);
        } else {
          const float sg = factor >= 0.f ? 1.f : -1.f;       // (bits cover a whole step too)
#pragma unroll
          for (int c = 0; c < NC; ++c)
            mx[c & 1] = fmaxf(mx[c & 1], seen(c) ? sg * sv[c] : -INFINITY);
        }
        const float rmax = fmaxf(mx[0], mx[1]);
        float tmax = rmax;
        if (rmax != -INFINITY) {
          tmax = rmax * fabsf(factor);
          if (CAP && own) tmax = a.cap_log2 * tanh_f32(tmax);
        }
        // the exponent base moves only when the step's maximum exceeds it by more than 8
        const float m_new = tmax > m_run + 8.f ? tmax : m_run;
        const float base = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = m_new == m_run ? 1.f : fast_exp2(m_run - base);
        m_run = m_new;

        // P and O are free to be written once the last step's PV is done
        if (n > 0 && !mbar_wait_abortable(bar(kBarODone + x), (n - 1) & 1, a.timeout_ns, abort)) break;
        tc_fence_after_sync();
        uint64_t ps2[2];
        auto emit = [&](auto cap_now, auto whole) {
          constexpr bool POLY = decltype(cap_now)::value;    // the cap is still to be taken
          constexpr bool WHOLE = decltype(whole)::value;     // every column is seen
          const CapPoly<POLY ? 5 : 7> cap(a.cap_log2, near);
          const uint64_t sc2 = f2splat(factor), nb2 = f2splat(-base);
          ps2[0] = ps2[1] = f2splat(0.f);
#pragma unroll
          for (int q = 0; q < NC / 32; ++q) {
            uint32_t hw[16], lw[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int c = 32 * q + 2 * e;
              const uint64_t s2 = f2pack(sv[c], sv[c + 1]);
              float2 xx = f2unpack(POLY ? cap(f2mul(s2, sc2), nb2) : f2fma(s2, sc2, nb2));
              if constexpr (CAP && !BIAS && !POLY) {     // rows of the warp differ
                const float2 xc = f2unpack(cap(f2mul(s2, sc2), nb2));
                xx = own ? xc : xx;
              }
              float2 p = make_float2(fast_exp2(xx.x), fast_exp2(xx.y));
              if constexpr (!WHOLE) {
                p.x = seen(c) ? p.x : 0.f;
                p.y = seen(c + 1) ? p.y : 0.f;
              }
              const uint64_t p2 = f2pack(p.x, p.y);
              ps2[e & 1] = f2add(ps2[e & 1], p2);
              hw[e] = pack2<QT>(p.x, p.y);
              const float2 f = unpack2<QT>(hw[e]);
              const float2 rest = f2unpack(f2sub(p2, f2pack(f.x, f.y)));
              lw[e] = pack2<QT>(rest.x, rest.y);
            }
            tmem_st16(t_p(x) + lane_off + 16 * q, hw);
            tmem_st16(t_p(x) + lane_off + 32 + 16 * q, lw);
          }
        };
        using Yes = std::true_type;
        using No = std::false_type;
        if (CAP && poly) full ? emit(Yes{}, Yes{}) : emit(Yes{}, No{});
        else full ? emit(No{}, Yes{}) : emit(No{}, No{});
        const float2 s0 = f2unpack(ps2[0]), s1 = f2unpack(ps2[1]);
        l_run = l_run * alpha + ((s0.x + s0.y) + (s1.x + s1.y));
        if (n > 0 && __any_sync(FULL, alpha != 1.f)) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float v[32];
            tmem_ld32(t_o(x) + lane_off + 32 * q, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] *= alpha;
            tmem_st32(t_o(x) + lane_off + 32 * q, v);
          }
        }
        tmem_wait_st();
        tc_fence_before_sync();
        mbar_arrive(bar(kBarPFull + x));
      }
      if (i0 < i1)
        mbar_wait_abortable(bar(kBarODone + x), (i1 - i0 - 1) & 1, a.timeout_ns, abort);
    } else {
      for (int j = 0; j < ntiles; ++j) {
        // S_x(j) complete also means PV_x(j-1) is: its MMA waited for that
        if (!mbar_wait_abortable(bar(kBarSFull + x), j & 1, a.timeout_ns, abort)) break;
        tc_fence_after_sync();
        float sv[kBN];
#pragma unroll
        for (int i = 0; i < kBN / 32; ++i) {
          float v[32];
          tmem_ld32(t_s(x) + lane_off + 32 * i, v);
#pragma unroll
          for (int e = 0; e < 32; ++e) sv[32 * i + e] = v[e];
        }
        tmem_wait_ld();

        // the row max of scale * s (log2 units), taken on the raw dot products:
        // the largest for scale >= 0, the smallest otherwise; four independent
        // chains; no per-element mask on a tile that lies wholly inside this
        // row's causal window
        const int t_base = (t_lo + j) * kBN;
        const bool full = t_base + kBN - 1 <= pos;
        const int nvalid = full ? kBN : max(0, pos - t_base + 1);
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (full && a.scale_log2 >= 0.f) {
#pragma unroll
          for (int c = 0; c < kBN; c += 2)
            mx[(c >> 1) & 3] = fmax3(mx[(c >> 1) & 3], sv[c], sv[c + 1]);
        } else if (full) {
#pragma unroll
          for (int c = 0; c < kBN; c += 2)
            mx[(c >> 1) & 3] = fmax3(mx[(c >> 1) & 3], -sv[c], -sv[c + 1]);
        } else {
          const float sg = a.scale_log2 >= 0.f ? 1.f : -1.f;
#pragma unroll
          for (int c = 0; c < kBN; ++c) mx[c & 3] = fmaxf(mx[c & 3], c < nvalid ? sg * sv[c] : -INFINITY);
        }
        const float rmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        // the exponent base moves only when the tile's max exceeds it by more
        // than 8 (log2 units): p <= 2^8 stays exact enough in 16 bits, O and l
        // share the base, and O / l is unchanged
        const float tmax = rmax == -INFINITY ? -INFINITY : rmax * fabsf(a.scale_log2);
        const float m_new = tmax > m_run + 8.f ? tmax : m_run;
        const float base = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = m_new == m_run ? 1.f : fast_exp2(m_run - base);
        // P = 2^(scale * s - base) over the S columns just read (masked
        // columns 0), pairs in packed f32x2 arithmetic: 32 tokens per
        // 16-column store
        const uint64_t sc2 = f2splat(a.scale_log2), nb2 = f2splat(-base);
        uint64_t ps2[2] = {f2splat(0.f), f2splat(0.f)};
#pragma unroll
        for (int c32 = 0; c32 < kBN / 32; ++c32) {
          uint32_t hw[16], lw[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int c = 32 * c32 + 2 * e;
            const uint64_t x2 = f2fma(f2pack(sv[c], sv[c + 1]), sc2, nb2);
            const float2 xx = f2unpack(x2);
            float2 p = make_float2(fast_exp2(xx.x), fast_exp2(xx.y));
            if (!full) {
              p.x = c < nvalid ? p.x : 0.f;
              p.y = c + 1 < nvalid ? p.y : 0.f;
            }
            ps2[e & 1] = f2add(ps2[e & 1], f2pack(p.x, p.y));
            hw[e] = pack2<QT>(p.x, p.y);
            if constexpr (PARTS == 2) {
              const float2 f = unpack2<QT>(hw[e]);
              lw[e] = pack2<QT>(p.x - f.x, p.y - f.y);
            }
          }
          tmem_st16(t_s(x) + lane_off + 16 * c32, hw);
          if constexpr (PARTS == 2) tmem_st16(t_s(x) + lane_off + 64 + 16 * c32, lw);
        }
        const float2 s0 = f2unpack(ps2[0]), s1 = f2unpack(ps2[1]);
        l_run = l_run * alpha + ((s0.x + s0.y) + (s1.x + s1.y));
        m_run = m_new;
        if (j > 0 && __any_sync(FULL, alpha != 1.f)) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v[32];
            tmem_ld32(t_o(x) + lane_off + 32 * i, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] *= alpha;
            tmem_st32(t_o(x) + lane_off + 32 * i, v);
          }
        }
        tmem_wait_st();
        tc_fence_before_sync();
        mbar_arrive(bar(kBarPFull + x));
      }
    }
    if (!MASK && ntiles > 0)
      mbar_wait_abortable(bar(kBarODone + x), (ntiles - 1) & 1, a.timeout_ns, abort);
  }

  tc_fence_before_sync();
  __syncthreads();                           // every role is done issuing and waiting
  if (*abort && (lane == 0 || warp == kMmaWarp || warp == kPvWarp)) {
    if (warp == kTmaWarp) {                  // let the copies in flight land
      for (int st = 0; st < kKst; ++st)
        if (armed_k[st] >= 0)
          mbar_wait_bounded(bar(kBarKFull + st), (armed_k[st] / kKst) & 1, kDrainLimitNs);
      for (int st = 0; st < kVst; ++st)
        if (armed_v[st] >= 0)
          mbar_wait_bounded(bar(kBarVFull + st), (armed_v[st] / kVst) & 1, kDrainLimitNs);
    } else if (warp == kMmaWarp) {           // let the MMAs in flight finish
      if (lane == 0) report_error(a.err_flag, kErrTimeout);
      __syncwarp();
      umma_commit_warp(bar(kBarDrain));
      mbar_wait_bounded(bar(kBarDrain), 0, kDrainLimitNs);
    } else if (warp == kPvWarp) {
      umma_commit_warp(bar(kBarDrainPv));
      mbar_wait_bounded(bar(kBarDrainPv), 0, kDrainLimitNs);
    }
  }
  __syncthreads();                           // drains done
  tc_fence_after_sync();
  const bool dead = *abort;
  const bool empty = ntiles == 0;            // an empty split: m = -inf, l = 0, o = 0
  if (MASK && nsplit > 1) {
    // ---- the cluster's CTAs share the rows out and merge them from each other's shared
    // memory: O (not yet divided) in Q's and K's place, (m, l) in V's.  Every product and
    // copy of this CTA is done, or it is dead and its memory is not read.
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    float4* po = reinterpret_cast<float4*>(smem_raw + (sbase - sraw));      // [256][32], swizzled
    float2* pml = reinterpret_cast<float2*>(smem_raw + (sbase - sraw) + kVOff);
    if (warp < 8 && !dead) {
      pml[tid] = empty ? make_float2(-INFINITY, 0.f) : make_float2(m_run, l_run);
      if (!empty) {
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v[32];
          tmem_ld32(t_o(x_me) + lane_off + 32 * i, v);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e)
            po[32 * tid + ((8 * i + e) ^ lane)] =
                make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        }
      }
    }
    tc_fence_before_sync();
    cluster.sync();
    if (warp < 8) {
      bool lost = false;                     // a CTA whose wait ran out: zeros
      for (int c = 0; c < nsplit; ++c) lost = lost || *cluster.map_shared_rank(&abort_flag, c) != 0;
      const int share = kQTiles * kRows / nsplit;
      for (int row = rank * share + warp; row < (rank + 1) * share; row += 8) {
        const int r = (row % kRows) / G, tok = row0 + row / kRows * TQ + r;
        if (r >= TQ || tok >= q_len) continue;
        float m = -INFINITY, l = 0.f;
        if (lane < nsplit && !lost) {
          const float2 ml = cluster.map_shared_rank(pml, lane)[row];
          m = ml.x;
          l = ml.y;
        }
        float M = l == 0.f ? -INFINITY : m;
#pragma unroll
        for (int o = kMaxSplit / 2; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL, M, o));
        const float w = l == 0.f || M == -INFINITY ? 0.f : fast_exp2(m - M);
        float sum = w * l;
#pragma unroll
        for (int o = kMaxSplit / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 0; c < nsplit; ++c) {
          const float wc = __shfl_sync(FULL, w, c);
          if (wc == 0.f) continue;           // nothing seen there: its O is not read
          const float4 v = cluster.map_shared_rank(po, c)[32 * row + (lane ^ (row & 31))];
          acc.x = fmaf(wc, v.x, acc.x);
          acc.y = fmaf(wc, v.y, acc.y);
          acc.z = fmaf(wc, v.z, acc.z);
          acc.w = fmaf(wc, v.w, acc.w);
        }
        sum = __shfl_sync(FULL, sum, 0);
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        const int pos = L - q_len + tok, h = kvh * G + row % kRows % G;
        const Span sp = seen_span(a.kv_start ? a.kv_start[q0 + tok] : 0, pos, a.window,
                                  a.prefix_lens ? a.prefix_lens[seq] : 0, L);
        const float s = fmaf(0.f, acc.x, fmaf(0.f, acc.y, fmaf(0.f, acc.z, 0.f * acc.w)));
        const bool odd = !(s == 0.f) || !(sum < INFINITY) || (sp.lo < sp.hi && !(sum > 0.f));
        if (__any_sync(FULL, odd) && !lost) {
          masked_row<QT>(a, table, q0 + tok, h, kvh, pos, sp.lo, sp.hi);
          continue;
        }
        uint2 pk;
        pk.x = pack2<QT>(acc.x * inv, acc.y * inv);
        pk.y = pack2<QT>(acc.z * inv, acc.w * inv);
        reinterpret_cast<uint2*>(static_cast<QT*>(a.out) +
                                 (static_cast<size_t>(q0 + tok) * a.num_heads + h) * kD)[lane] = pk;
      }
    }
    cluster.sync();                          // nobody reads this CTA's memory any more
  } else if (warp < 8) {
    // ---- epilogue: out row = O / l (cascade: the partial o / l, m, l)
    const int x = x_me;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    bool odd = false;                        // MASK: a non-finite value in this row
    const float inv = (!dead && l_run > 0.f) ? 1.f / l_run : 0.f;
    const int h = kvh * G + row_me % G;
    const size_t orow_idx = static_cast<size_t>(q0 + tok_me) * a.num_heads + h;
    // this warp's 32 output rows, 16 chunks of 16 bytes each, in Q's place (every product
    // that read it is done); chunk c of row r at c ^ (r & 15), free of bank conflicts
    uint4* stage = reinterpret_cast<uint4*>(smem_raw + (sbase - sraw) + kQOff) + 512 * warp;
    const size_t split_rows = cascade ? static_cast<size_t>(seq) * q_len * a.num_heads : 0;
    if (cascade && row_valid) {
      a.part_m[split_rows + orow_idx] = (dead || empty) ? -INFINITY : m_run;
      a.part_l[split_rows + orow_idx] = (dead || empty) ? 0.f : l_run;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[32];
      tmem_ld32(t_o(x) + lane_off + 32 * i, v);
      tmem_wait_ld();
      if (!row_valid) continue;
      if (dead || empty) {                   // TMEM may hold anything: write plain zeros
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = 0.f;
      }
      if constexpr (MASK) {
        float s = 0.f;                       // 0 * inf and 0 * NaN are NaN
#pragma unroll
        for (int e = 0; e < 32; ++e) s = fmaf(0.f, v[e], s);
        odd = odd || !(s == 0.f) || !(l_run < INFINITY) || (row_lo < row_hi && !(l_run > 0.f));
      }
      if (cascade) {
        float4* dst = reinterpret_cast<float4*>(a.part_o + (split_rows + orow_idx) * kD + 32 * i);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          dst[e] = make_float4(v[4 * e] * inv, v[4 * e + 1] * inv, v[4 * e + 2] * inv,
                               v[4 * e + 3] * inv);
      } else {
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          uint4 w;
          w.x = pack2<QT>(v[e] * inv, v[e + 1] * inv);
          w.y = pack2<QT>(v[e + 2] * inv, v[e + 3] * inv);
          w.z = pack2<QT>(v[e + 4] * inv, v[e + 5] * inv);
          w.w = pack2<QT>(v[e + 6] * inv, v[e + 7] * inv);
          if (dead || empty)                 // a copy may still be on its way to shared memory
            *reinterpret_cast<uint4*>(reinterpret_cast<QT*>(a.out) + orow_idx * kD + 32 * i + e) = w;
          else
            stage[16 * lane + ((4 * i + e / 8) ^ (lane & 15))] = w;
        }
      }
    }
    if (!cascade && !dead && !empty) {
      // the warp's rows go out two at a time, 512 bytes a store (a thread per row stores 16
      // bytes to each of 32 lines: 4k clocks a CTA longer)
      __syncwarp();
      const long long mine = row_valid ? static_cast<long long>(orow_idx) : -1;
#pragma unroll 4
      for (int r = 0; r < 32; r += 2) {
        const int src = r + (lane >> 4), ch = lane & 15;
        const long long to = __shfl_sync(FULL, mine, src);
        if (to >= 0)
          reinterpret_cast<uint4*>(static_cast<QT*>(a.out) + to * kD)[ch] =
              stage[16 * src + (ch ^ (src & 15))];
      }
      __syncwarp();
    }
    if constexpr (MASK) {                    // the rows that came out non-finite, once more
      uint32_t again = __ballot_sync(FULL, odd && !dead && row_valid);
      while (again) {
        const int src = __ffs(again) - 1;
        again &= again - 1;
        masked_row<QT>(a, table, __shfl_sync(FULL, q0 + tok_me, src), __shfl_sync(FULL, h, src), kvh,
                       __shfl_sync(FULL, row_pos, src), __shfl_sync(FULL, row_lo, src),
                       __shfl_sync(FULL, row_hi, src));
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

cudaError_t make_q_map(CUtensorMap* map, const void* q, int total_q, int num_heads, int G) {
  auto fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(kD), static_cast<cuuint64_t>(num_heads),
                        static_cast<cuuint64_t>(total_q)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(kD) * 2,
                           static_cast<cuuint64_t>(num_heads) * kD * 2};
  cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(kRows / G)};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  CUresult rc = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(q), dims, strides,
                   box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return rc == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace
}  // namespace pa

// pa_decode_kernel.cuh -- the per-partition kernel of paged decode attention
// (pa_decode_v1, pa_decode_v2_partition, pa_append_decode_v1; pa_decode.cu) and, with
// changed scores, of pa_decode_masked (pa_masked.cu).
#pragma once

#include <cudaTypedefs.h>

#include <climits>
#include <mutex>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_score.cuh"
#include "pa_tile.cuh"
#include "pa_write.cuh"

namespace pa {

// A v2 partition of a sequence whose seq_len failed the bounds check: written
// as empty (m = -inf, l = 0, o = 0) so the merge skips it and outputs zeros.
__device__ __forceinline__ void write_empty_partial(const DecodeArgs& a, int seq, int kvh,
                                                    int part, int G, int D) {
  for (int idx = threadIdx.x; idx < G * D; idx += blockDim.x) {
    const int g = idx / D, d = idx % D;
    const size_t row =
        (static_cast<size_t>(seq) * a.num_heads + kvh * G + g) * a.max_parts + part;
    a.tmp_out[row * D + d] = 0.f;
    if (d == 0) {
      a.max_logits[row] = -INFINITY;
      a.exp_sums[row] = 0.f;
    }
  }
}

// 8-bit caches: at most 128 registers, so two CTAs of up to 8 warps fit an SM
// (the 8-bit path is issue- and latency-bound: more resident warps help).
//
// MASK (pa_decode_masked): the v1 pass with changed scores, over the tiles from the
// 16-token boundary at or before the sequence's first seen token (a block that ends before
// that token is not looked up: it may be gone).  With running scores
// asked for, the scores x go to the workspace and, once the CTA has merged its warps and
// knows every head's log-sum-exp, come back as weights: the CTA holds the whole
// (sequence, kv head), so no second launch is needed.
template <typename QT, int KIND, int D, int BS, bool MASK = false>
__global__ void __launch_bounds__(kMaxWarps * 32, KIND == kKind16 ? 0 : 2)
    decode_tc_kernel(const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ DecodeArgs a) {
  using T = Tr<KIND, D, BS>;
  using CT = mma_type<QT, KIND, MASK>;        // MMA operand type
  constexpr bool WIDE = !std::is_same<CT, QT>::value;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kMaxWarps * kMaxStages];
  __shared__ int stage_ok[kMaxWarps * kMaxStages];

  const int part = blockIdx.x, kvh = blockIdx.y, seq = blockIdx.z;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
  const int r = lane >> 2, c = lane & 3;
  const int G = a.num_heads / a.num_kv_heads;
  const int S = a.stages;
  const bool check = a.err_flag != nullptr;
  const bool v1 = MASK || a.partition_size == 0;
  constexpr uint32_t FULL = 0xffffffffu;

  griddep_launch_dependents();
  // mode 2 first reads lens / tables; mode 3 (cascade suffix) waits only for the
  // prior partial its epilogue merges
  if (a.pdl != 2 && a.pdl != 3) griddep_wait();

  int len = a.seq_lens[seq];
  bool bad = false;                               // MASK
  if (check) {
    const long long cap = static_cast<long long>(a.max_blocks) * BS;
    if (len < 0 || len > cap) {
      if (threadIdx.x == 0) report_error(a.err_flag, kErrSeqLen);
      len = 0;                                    // skip the sequence: its output is zeros
      bad = true;
      if (!MASK && !v1) {
        griddep_wait();
        write_empty_partial(a, seq, kvh, part, G, D);
        return;
      }
    }
  }
  int t_begin = v1 ? min(a.t_offset, len) : 0, t_end = len;
  int lo = 0;                                     // MASK: first seen token
  if constexpr (MASK) {
    lo = seen_span(a.kv_start ? a.kv_start[seq] : 0, len - 1, a.window, 0, len).lo;
    t_begin = lo < len ? lo & ~15 : len;
  }
  if (!MASK && !v1) {
    t_begin = part * a.partition_size;
    t_end = min(len, t_begin + a.partition_size);
    if (t_begin >= t_end) return;                 // empty partition: nothing to write
  }

  const uint32_t sraw = smem_u32(smem_raw);
  const uint32_t sbase = (sraw + 1023u) & ~1023u;
  const uint32_t wbase = sbase + static_cast<uint32_t>(warp * S * T::STAGE);
  const uint32_t bar0 = smem_u32(&bars[warp * kMaxStages]);
  int* ok_slot = &stage_ok[warp * kMaxStages];

  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init(bar0 + 8u * s, 1);
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (threadIdx.x == 0) {
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  __syncwarp();

  const int ntok = t_end - t_begin;
  const int ntiles = (ntok + 15) / 16;
  const int nmine = ntiles > warp ? (ntiles - warp + nwarps - 1) / nwarps : 0;
  const int nblk_seq = (len + BS - 1) / BS;
  const int32_t* table = a.block_tables + static_cast<size_t>(seq) * a.max_blocks;
  constexpr int kBeyond = INT_MIN;

  // Block ids of this warp's tiles, 32 tiles per window, one tile per lane.
  int ids_cur[T::NBOX], ids_nxt[T::NBOX];
  auto load_window = [&](int wdx, int (&ids)[T::NBOX]) {
    const int i = wdx * 32 + lane;
    const int t0 = t_begin + 16 * (warp + i * nwarps);
#pragma unroll
    for (int b = 0; b < T::NBOX; ++b) {
      const int tb = t0 + b * T::BOXH, lb = tb / BS;
      const bool use = i < nmine && lb < nblk_seq && (!MASK || tb + T::BOXH > lo);
      ids[b] = use ? __ldg(table + lb) : kBeyond;
    }
  };
#pragma unroll
  for (int b = 0; b < T::NBOX; ++b) ids_cur[b] = ids_nxt[b] = kBeyond;
  if (nmine > 0) load_window(0, ids_cur);
  if (nmine > 32) load_window(1, ids_nxt);
  int win_cur = 0;
  uint32_t armed = 0;                             // stages with a completion pending

  // PDL mode 2: fetch this warp's first tiles into L2 while the preceding grid
  // finishes (lane i prefetches tile i of window 0)
  if (a.pdl == 2 && lane < min(a.prefetch, nmine)) {
    const int ob = BS > 16 ? (t_begin + 16 * (warp + lane * nwarps)) % BS : 0;
    prefetch_tile<KIND, D, BS>(&tm_k, &tm_v, a.k_scale, a.v_scale, a.num_kv_heads, a.num_blocks,
                               kvh, ids_cur, ob);
  }

  const uint64_t pol = policy_evict_first();

  const int never = a.inject == 1 ? 0 : MASK && a.inject == 3 && nmine > 2 ? nmine - 1 : -1;

  // Issue the loads of this warp's i-th tile into stage s (whole warp calls).
  auto issue = [&](int i, int s) {
    const int wdx = i >> 5;
    if (wdx != win_cur) {
#pragma unroll
      for (int b = 0; b < T::NBOX; ++b) ids_cur[b] = ids_nxt[b];
      win_cur = wdx;
      if ((wdx + 1) * 32 < nmine) load_window(wdx + 1, ids_nxt);
    }
    int blk[T::NBOX];
#pragma unroll
    for (int b = 0; b < T::NBOX; ++b) blk[b] = __shfl_sync(FULL, ids_cur[b], i & 31);
    if (i == never) return;                       // test hook: this stage never arrives
    armed |= 1u << s;
    if (lane == 0) {
      const uint32_t st = wbase + static_cast<uint32_t>(s * T::STAGE);
      const uint32_t bar = bar0 + 8u * s;
      const int ob = BS > 16 ? (t_begin + 16 * (warp + i * nwarps)) % BS : 0;
      int okm = 0;
#pragma unroll
      for (int b = 0; b < T::NBOX; ++b) {
        if (blk[b] == kBeyond) continue;
        if (check && (blk[b] < 0 || blk[b] >= a.num_blocks)) {
          report_error(a.err_flag, kErrBlockId);
          continue;
        }
        okm |= 1 << b;
      }
      ok_slot[s] = okm;
      fence_proxy_async_smem();
      mbar_arrive_expect_tx(bar, tile_bytes<KIND, D, BS>(okm));
      issue_tile_copies<KIND, D, BS>(st, bar, &tm_k, &tm_v, a.k_scale, a.v_scale,
                                     a.num_kv_heads, kvh, blk, okm, ob, pol);
    }
  };

  if (a.pdl == 2) griddep_wait();                 // q and the caches may come from it

  // With a fused cache write, this CTA's range ends at the sequence's last
  // token, and the warp owning that tile writes the token before it loads the
  // tile: its prologue copy of that tile (if any) waits for the write.
  const bool writes = !MASK && a.new_k != nullptr && t_end == len && ntok > 0;
  const int w_last = writes ? (ntiles - 1) % nwarps : -1;
  const int i_last = writes ? (ntiles - 1) / nwarps : -1;
  const bool writer = warp == w_last;

  const int npro = min(S, nmine);
  for (int i = 0; i < npro; ++i)
    if (!(writer && i == i_last)) issue(i, i);
  if (writer) {
    const int64_t slot = a.new_slots[seq];
    // debug mode: the slot must be where the table puts token len - 1 (a slot in an
    // earlier tile would be written while another warp may be loading that tile)
    bool slot_ok = slot >= 0 && slot < static_cast<int64_t>(a.num_blocks) * BS;
    if (check && slot >= 0) {
      const int64_t want = static_cast<int64_t>(table[(len - 1) / BS]) * BS + (len - 1) % BS;
      slot_ok = slot_ok && slot == want;
    }
    if (slot_ok) {
      constexpr int MODE = KIND == kKind16 ? kWriteCopy : (KIND == kKindI8 ? kWriteInt8 : kWriteFp8);
      const int64_t blk = slot / BS;
      const int off = static_cast<int>(slot % BS);
      const size_t src_row = (static_cast<size_t>(seq) * a.num_kv_heads + kvh) * D;
      const size_t dst_row = ((static_cast<size_t>(blk) * BS + off) * a.num_kv_heads + kvh) * D;
      const size_t sidx = (static_cast<size_t>(blk) * a.num_kv_heads + kvh) * BS + off;
      write_kv_row<QT, MODE, D>(static_cast<const QT*>(a.new_k) + src_row, a.wk_cache, dst_row,
                                MODE ? a.wk_scale + sidx : nullptr, lane);
      write_kv_row<QT, MODE, D>(static_cast<const QT*>(a.new_v) + src_row, a.wv_cache, dst_row,
                                MODE ? a.wv_scale + sidx : nullptr, lane);
      fence_proxy_async_global();
    } else if (slot >= 0 && lane == 0) {
      report_error(a.err_flag, kErrSlot);         // past the pool or off the table: nothing written
    }
    __syncwarp();
    if (i_last < npro) issue(i_last, i_last);
  }

  WarpAttn<CT, KIND, D, BS> wa;
  wa.reset();
  const QT* qrow = reinterpret_cast<const QT*>(a.q) +
                   (static_cast<size_t>(seq) * a.num_heads + static_cast<size_t>(kvh) * G + r) * D;
  ScoreMod mod;
  if constexpr (WIDE) wa.load_q_wide(qrow, r < G, c, mod.qs);
  else wa.load_q_global(qrow, r < G, c);

  if constexpr (MASK) {
    mod.cap_in = a.cap_in;
    mod.cap_log2 = a.cap_log2;
    mod.G = G;
    mod.slope[0] = a.slopes && 2 * c < G ? a.slopes[kvh * G + 2 * c] * kLog2e : 0.f;
    mod.slope[1] = a.slopes && 2 * c + 1 < G ? a.slopes[kvh * G + 2 * c + 1] * kLog2e : 0.f;
    mod.logits = nullptr;
  }
  const size_t unit = static_cast<size_t>(seq) * a.num_kv_heads + kvh;

  int si = 0;
  uint32_t ph = 0;
  bool dead = false;
  for (int i = 0; i < nmine; ++i) {
    const uint32_t st = wbase + static_cast<uint32_t>(si * T::STAGE);
    const bool arrived = __all_sync(FULL, mbar_wait_bounded(bar0 + 8u * si, ph, a.timeout_ns));
    if (!arrived) {
      // Stop consuming; let every copy this warp still has in flight land (each
      // wait again bounded), so none targets shared memory after the CTA exits.
      for (int k = 0; k < S; ++k) {
        const int s2 = (si + k) % S;
        if ((armed >> s2) & 1u)
          mbar_wait_bounded(bar0 + 8u * s2, ph ^ ((si + k) >= S ? 1u : 0u), kDrainLimitNs);
      }
      dead = true;
      break;
    }
    armed &= ~(1u << si);
    const int j = warp + i * nwarps;
    const int nv = min(16, ntok - j * 16);
    const int okm = ok_slot[si];
    TileFrag<KIND, D, BS> fr;
    load_tile<CT, KIND, D, BS>(fr, st, lane);
    __syncwarp();
    if (i + S < nmine) issue(i + S, si);          // refill the stage right away
    if constexpr (MASK) {
      const int t0 = t_begin + 16 * j;
      mod.back = len - 1 - t0;
      mod.lo = lo - t0;
      mod.room = a.score_stride - t0;
      if (a.scores_out) mod.logits = a.logits + (unit * a.score_stride + t0) * G;
      tile_compute<CT, KIND, D, BS, true, WIDE>(wa, fr, nv, okm, a.scale_log2, lane, mod);
    } else {
      tile_compute<QT, KIND, D, BS>(wa, fr, nv, okm, a.scale_log2, lane);
    }
    if (++si == S) {
      si = 0;
      ph ^= 1u;
    }
  }

  if (dead) {
    if (lane == 0) report_error(a.err_flag, kErrTimeout);
    wa.reset();
  } else {
    wa.template finish<MASK, WIDE>();
  }

  // ---- merge the warps of the CTA through shared memory
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    wa.lsum[0] += __shfl_xor_sync(FULL, wa.lsum[0], off);
    wa.lsum[1] += __shfl_xor_sync(FULL, wa.lsum[1], off);
  }
  // every warp is done with its stages; MASK: a warp lost tiles, and with them the unit
  bool lost = false;
  if constexpr (MASK) lost = __syncthreads_or(dead) != 0;
  else __syncthreads();
  constexpr int OP = D + 4;
  float* ored = reinterpret_cast<float*>(smem_raw + (sbase - sraw));
  float* mred = ored + nwarps * 8 * OP;
  float* lred = mred + nwarps * 8;
#pragma unroll
  for (int mt = 0; mt < T::NMT; ++mt) {
    const int d0 = out_dim<KIND>(mt, r, 0), d1 = out_dim<KIND>(mt, r, 1);
    float* o0 = ored + (warp * 8 + 2 * c) * OP;
    float* o1 = o0 + OP;
    o0[d0] = wa.oacc[mt][0];
    o1[d0] = wa.oacc[mt][1];
    o0[d1] = wa.oacc[mt][2];
    o1[d1] = wa.oacc[mt][3];
  }
  if (r == 0) {
    mred[warp * 8 + 2 * c] = wa.m2[0];
    mred[warp * 8 + 2 * c + 1] = wa.m2[1];
    lred[warp * 8 + 2 * c] = wa.lsum[0];
    lred[warp * 8 + 2 * c + 1] = wa.lsum[1];
  }
  __syncthreads();

  constexpr int NCH = D / 8;
  if (!MASK && a.prior_o != nullptr && a.pdl == 3) griddep_wait();   // the prior partial's producer
  for (int idx = threadIdx.x; idx < G * NCH; idx += blockDim.x) {
    const int g = idx / NCH, d0 = (idx % NCH) * 8;
    float M = -INFINITY;
    for (int w = 0; w < nwarps; ++w) M = fmaxf(M, mred[w * 8 + g]);
    float L = 0.f;
    float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    // MASK: a row whose scores are all NaN has no maximum, but is NaN
    if (MASK || M != -INFINITY) {
      const float ms = MASK && M == -INFINITY ? 0.f : M;
      for (int w = 0; w < nwarps; ++w) {
        const float f = fast_exp2(mred[w * 8 + g] - ms);
        L += lred[w * 8 + g] * f;
        const float* src = ored + (w * 8 + g) * OP + d0;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] += src[e] * f;
      }
    }
    const int h = kvh * G + g;
    if (!MASK && v1 && a.prior_o != nullptr) {
      // merge the prior partials (o_p / l_p, m_p, l_p) by log-sum-exp
      const size_t rows = static_cast<size_t>(a.num_seqs) * a.num_heads;
      const size_t pr = static_cast<size_t>(seq) * a.num_heads + h;
      for (int k = 0; k < a.prior_splits; ++k) {
        const float mp = a.prior_m[k * rows + pr], lp = a.prior_l[k * rows + pr];
        if (mp == -INFINITY) continue;         // an empty split
        const float M2 = fmaxf(M, mp);
        const float f1 = M == -INFINITY ? 0.f : fast_exp2(M - M2);
        const float f2 = fast_exp2(mp - M2) * lp;
        const float4* op = reinterpret_cast<const float4*>(a.prior_o + (k * rows + pr) * D + d0);
        const float4 p0 = op[0], p1 = op[1];
        const float pv[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = o[e] * f1 + pv[e] * f2;
        L = L * f1 + f2;
        M = M2;
      }
    }
    const float inv = L > 0.f && !lost ? 1.f / L : 0.f;
    if (MASK && lost) {
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = 0.f;
    }
    if (v1) {
      uint4 pk;
      pk.x = pack2<QT>(o[0] * inv, o[1] * inv);
      pk.y = pack2<QT>(o[2] * inv, o[3] * inv);
      pk.z = pack2<QT>(o[4] * inv, o[5] * inv);
      pk.w = pack2<QT>(o[6] * inv, o[7] * inv);
      *reinterpret_cast<uint4*>(reinterpret_cast<QT*>(a.out) +
                                (static_cast<size_t>(seq) * a.num_heads + h) * D + d0) = pk;
    } else {
      const size_t row = (static_cast<size_t>(seq) * a.num_heads + h) * a.max_parts + part;
      float4* dst = reinterpret_cast<float4*>(a.tmp_out + row * D + d0);
      dst[0] = make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
      dst[1] = make_float4(o[4] * inv, o[5] * inv, o[6] * inv, o[7] * inv);
      if (d0 == 0) {
        a.max_logits[row] = M == -INFINITY ? -INFINITY : M * 0.69314718055994530942f;
        a.exp_sums[row] = L;
      }
    }
  }
  if constexpr (MASK) {
    if (!a.scores_out || bad || lost) return;     // a skipped or lost unit keeps its scores
    __shared__ float lse[kMaxGroup];
    if (threadIdx.x < kMaxGroup) {
      float M = -INFINITY, L = 0.f;
      for (int w = 0; w < nwarps; ++w) M = fmaxf(M, mred[w * 8 + threadIdx.x]);
      const float ms = M == -INFINITY ? 0.f : M;
      for (int w = 0; w < nwarps; ++w)
        L += lred[w * 8 + threadIdx.x] * fast_exp2(mred[w * 8 + threadIdx.x] - ms);
      lse[threadIdx.x] = threadIdx.x < G ? weight_lse(M, L) : INFINITY;
    }
    __syncthreads();                              // the scores x are this CTA's own writes
    for (int t = threadIdx.x; t < min(len, a.score_stride); t += blockDim.x) {
      const size_t i = unit * a.score_stride + t;
      const float before = a.scores_in ? a.scores_in[i] : 0.f;
      float x[8];
      load_scores(a.logits + i * G, t >= lo, G, x);
      a.scores_out[i] = before + (t >= lo ? token_weight(x, lse) : 0.f);
    }
  }
}

template <typename QT, int KIND, int D, int BS, bool MASK>
cudaError_t launch_tc(const DecodeArgs& a, const DecodeShape& sh, cudaStream_t stream) {
  using T = Tr<KIND, D, BS>;
  CUtensorMap mk, mv;
  cudaError_t e = make_cache_map<KIND, D, BS>(&mk, a.k_cache, a.num_kv_heads, a.num_blocks);
  if (e != cudaSuccess) return e;
  e = make_cache_map<KIND, D, BS>(&mv, a.v_cache, a.num_kv_heads, a.num_blocks);
  if (e != cudaSuccess) return e;
  const int ring = sh.warps * a.stages * T::STAGE;
  const int epi = sh.warps * 8 * (D + 4) * 4 + sh.warps * 16 * 4;   // the warps' merge
  const int smem = (ring > epi ? ring : epi) + 1024;
  auto kern = decode_tc_kernel<QT, KIND, D, BS, MASK>;
  static int configured[64] = {0};
  e = opt_in_smem(reinterpret_cast<const void*>(kern), smem, configured);
  if (e != cudaSuccess) return e;
  dim3 grid(sh.grid_x, a.num_kv_heads, a.num_seqs);
  return launch_kernel(kern, grid, dim3(sh.warps * 32), smem, stream, a.pdl != 0, mk, mv, a);
}

}  // namespace pa

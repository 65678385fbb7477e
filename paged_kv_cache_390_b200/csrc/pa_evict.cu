// pa_evict.cu -- eviction from the paged cache by accumulated attention weight
// (pa_evict) for sm_100a: per (sequence, kv head) the num_recent newest tokens and the
// highest-scored others stay, num_keep in all, and move to fresh blocks in their order.
//
// Which tokens stay is a selection of the r-th largest of up to max_blocks * block_size
// fp32 scores (r = num_keep - num_recent): scores become unsigned keys of the same
// order, and up to four passes of 8 bits count digits in shared memory and narrow the
// threshold's digits, most significant first, until all the keys that begin with them
// stay (spread scores: mostly after two or three).  Tokens above the threshold stay, and of
// those equal to it the first ones until r are found; a token's place is the number of
// tokens before it that are above the threshold plus that of equal ones, as far as they
// stay.  Whole-number counts, so the same tokens every time.
//
// One cluster of 1 to 8 CTAs per (sequence, kv head), one launch: each CTA takes an equal
// run of the tokens, its keys read once into shared memory, and the CTAs add up their
// digit counts through distributed shared memory; then the cluster's threads copy the
// kept rows, 16 bytes a thread, eight rows' loads before their stores.  Bound: the rows'
// bytes once the tokens are selected.  8 x 16k tokens to 4096, 8 kv heads, bf16 (275 MB):
// 66 us, of them ~45 at 6.2 TB/s for the rows and ~16 for the selection (the scores' load,
// digits at ~2 us, the places); 16 x 640 to 256: 14.2 us, ~7 for the rows.  (The first form, one CTA per
// (sequence, kv head) and a second launch to move, took 144.)
#include <cooperative_groups.h>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_tile.cuh"

namespace pa {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kKeys = 8192;                    // keys a CTA holds; longer runs are read again
constexpr int kMaxCluster = 8;
constexpr int kMove = 8;                       // rows in flight per thread

// Unsigned key with the order of the scores; NaN counts as lowest, -0 as 0.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0u;
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ void prefetch_l1(const void* p) {
  asm volatile("prefetch.global.L1 [%0];" ::"l"(p));
}

// Sequence length if its tokens lie inside the table and the scores and what stays
// fits the new table and the outputs, else -1 (always checked).
__device__ __forceinline__ int checked_len(const EvictArgs& a, int s) {
  const int len = a.seq_lens[s];
  const long long cap = static_cast<long long>(a.max_src_blocks) * a.block_size;
  if (len < 0 || len > cap || len > a.score_stride) return -1;
  return min(len, a.num_keep) > a.max_kept ? -1 : len;
}

__global__ void __launch_bounds__(kThreads, 2)
    evict_kernel(const __grid_constant__ EvictArgs a) {
  constexpr uint32_t FULL = 0xffffffffu;
  __shared__ __align__(8) uint32_t keys[kKeys];
  // Digit counts of this CTA, the highest digit first.  Three in turn: pass p fills one
  // and clears the next, which was last read in pass p - 2, so before everybody came to
  // pass p - 1's barrier.
  __shared__ __align__(16) uint32_t hist[3][256];
  __shared__ uint32_t found[3];                // threshold so far, keys wanted of it, its keys
  __shared__ uint32_t counts[2];               // this CTA's keys above / equal to the threshold
  __shared__ uint32_t wcount[2][kWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = blockIdx.x, nc = gridDim.x, kvh = blockIdx.y, s = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_launch_dependents();
  if (tid < 256) hist[0][tid] = 0;
  __syncthreads();
  griddep_wait();
  const size_t unit = static_cast<size_t>(s) * a.num_kv_heads + kvh;
  const float* sc = a.scores + unit * a.score_stride;
  const int32_t* stab = a.src_tables + static_cast<size_t>(s) * a.max_src_blocks;
  const int32_t* dtab = a.dst_tables + static_cast<size_t>(s) * a.max_dst_blocks;
  // the first scores and table entries come while the length does
  if (nc == 1 && tid < 128 && 32 * tid < a.score_stride) prefetch_l1(sc + 32 * tid);
  if (warp < kWarps / 2) {
    if (32 * tid < a.max_src_blocks) prefetch_l1(stab + 32 * tid);
  } else if (32 * (tid - kThreads / 2) < a.max_dst_blocks) {
    prefetch_l1(dtab + 32 * (tid - kThreads / 2));
  }
  const int len = checked_len(a, s);
  int* kept = a.kept + unit * a.kept_stride;
  if (len < 0) {                               // skipped (the whole cluster): nothing kept
    if (tid == 0 && kvh == 0 && rank == 0) {
      report_error(a.err_flag, kErrSeqLen);
      a.new_lens[s] = 0;
    }
    for (int i = rank * kThreads + tid; i < a.kept_stride; i += nc * kThreads) kept[i] = -1;
    return;
  }
  float* nsc = a.new_scores ? a.new_scores + unit * a.new_score_stride : nullptr;
  const int m = min(len, a.num_keep);
  const int old = max(0, len - a.num_recent);  // tokens that compete by score
  const int r = m - (len - old);               // how many of them stay
  auto sync = [&]() {
    if (nc > 1) cluster.sync();
    else __syncthreads();
  };
  auto put = [&](int place, int t) {
    if (place >= m) return;                    // scores that change meanwhile stay harmless
    kept[place] = t;
  };
  if (r > 0 && r < old) {
    // this CTA's run of tokens, in whole warps of 32 for each of its warps
    const int per_warp = ((old + nc * kWarps - 1) / (nc * kWarps) + 31) / 32 * 32;
    const int run = per_warp * kWarps;
    const int t_lo = min(old, rank * run), t_hi = min(old, t_lo + run);
    const bool held = run <= kKeys;
    auto key = [&](int t) { return held ? keys[t - t_lo] : score_key(sc[t]); };
    // Keys, and the first digit on the way: sign and exponent, so a warp's keys share a few
    // digits and equal ones are counted by one lane (32 lanes on one counter take 32 turns).
    // Four loads of a thread in flight.
#pragma unroll 1
    for (int t0 = t_lo + tid; t0 < t_hi; t0 += 4 * kThreads) {
      float x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (t0 + u * kThreads < t_hi) x[u] = sc[t0 + u * kThreads];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int t = t0 + u * kThreads;
        if (t >= t_hi) break;
        const uint32_t k = score_key(x[u]);
        if (held) keys[t - t_lo] = k;
        const uint32_t d = 255u - (k >> 24);
        const uint32_t same = __match_any_sync(__activemask(), d);
        if (lane == __ffs(same) - 1) atomicAdd(&hist[0][d], __popc(same));
      }
    }
    uint32_t thr = 0, mask = 0, want = static_cast<uint32_t>(r);
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = 24 - 8 * pass, buf = pass % 3;
      if (tid < 256) hist[(pass + 1) % 3][tid] = 0;
      if (pass > 0) {
        for (int t = t_lo + tid; t < t_hi; t += kThreads) {
          const uint32_t k = key(t);
          if ((k & mask) == thr) atomicAdd(&hist[buf][255u - ((k >> shift) & 255u)], 1u);
        }
      }
      sync();
      // Warp 0 finds the digit; lane l holds digits 255 - 8l .. 248 - 8l.
      if (warp == 0) {
        uint32_t c[8] = {};
#pragma unroll
        for (int cta = 0; cta < kMaxCluster; ++cta) {
          if (cta < nc) {
            const uint32_t* from = nc > 1 ? cluster.map_shared_rank(&hist[buf][0], cta) : hist[buf];
            const uint4 c0 = reinterpret_cast<const uint4*>(from)[2 * lane];
            const uint4 c1 = reinterpret_cast<const uint4*>(from)[2 * lane + 1];
            c[0] += c0.x; c[1] += c0.y; c[2] += c0.z; c[3] += c0.w;
            c[4] += c1.x; c[5] += c1.y; c[6] += c1.z; c[7] += c1.w;
          }
        }
        uint32_t sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += c[i];
        uint32_t incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t v = __shfl_up_sync(FULL, incl, o);
          if (lane >= o) incl += v;
        }
        uint32_t before = incl - sum;
        if (before < want && incl >= want) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (before < want && before + c[i] >= want) {
              found[0] = thr | ((255u - 8 * lane - i) << shift);
              found[1] = want - before;
              found[2] = c[i];
              break;
            }
            before += c[i];
          }
        }
      }
      __syncthreads();
      thr = found[0];
      want = found[1];
      mask |= 255u << shift;
      // everything that begins with these digits stays: they are the threshold (zeros
      // after them), the further digits do not matter
      if (found[2] == want) {
        want = ~0u;
        break;
      }
    }
    // `want` of the tokens equal to the threshold stay, the first ones
    const int w_lo = min(t_hi, t_lo + warp * per_warp), w_hi = min(t_hi, w_lo + per_warp);
    uint32_t above = 0, equal = 0;
    for (int t0 = w_lo; t0 < w_hi; t0 += 32) {
      const uint32_t k = t0 + lane < w_hi ? key(t0 + lane) : 0u;
      const bool in = t0 + lane < w_hi;
      above += __popc(__ballot_sync(FULL, in && k > thr));
      equal += __popc(__ballot_sync(FULL, in && k == thr));
    }
    if (lane == 0) {
      wcount[0][warp] = above;
      wcount[1][warp] = equal;
    }
    __syncthreads();
    if (tid < 2) {
      uint32_t sum = 0;
      for (int w = 0; w < kWarps; ++w) sum += wcount[tid][w];
      counts[tid] = sum;
    }
    sync();
    above = equal = 0;                         // before this warp's first token
    for (int c = 0; c < rank; ++c) {
      const uint32_t* other = cluster.map_shared_rank(&counts[0], c);
      above += other[0];
      equal += other[1];
    }
    for (int w = 0; w < warp; ++w) {
      above += wcount[0][w];
      equal += wcount[1][w];
    }
    const uint32_t below = (1u << lane) - 1u;
    for (int t0 = w_lo; t0 < w_hi; t0 += 32) {
      const int t = t0 + lane;
      const uint32_t k = t < w_hi ? key(t) : 0u;
      const uint32_t ba = __ballot_sync(FULL, t < w_hi && k > thr);
      const uint32_t be = __ballot_sync(FULL, t < w_hi && k == thr);
      const uint32_t eq_before = equal + __popc(be & below);
      const uint32_t place = above + __popc(ba & below) + min(eq_before, want);
      if (((ba >> lane) & 1u) || (((be >> lane) & 1u) && eq_before < want))
        put(static_cast<int>(place), t);
      above += __popc(ba);
      equal += __popc(be);
    }
  } else if (r > 0) {                          // all of them stay
    for (int t = rank * kThreads + tid; t < old; t += nc * kThreads) put(t, t);
  }
  for (int t = old + rank * kThreads + tid; t < len; t += nc * kThreads) put(r + t - old, t);
  for (int i = m + rank * kThreads + tid; i < a.kept_stride; i += nc * kThreads) kept[i] = -1;
  if (tid == 0 && kvh == 0 && rank == 0) a.new_lens[s] = m;
  // every place is written (the barrier orders the cluster's global writes too), and
  // nobody reads this CTA's shared memory any more
  sync();

  // ---- copy the kept rows: this CTA takes a run of places; their source and destination
  // slots go to shared memory first (in place of the keys), so that a row's copy waits
  // for one load, not for the place, the table and the row one after another
  const int vshift = a.vec_shift;                          // 2 * row_vecs = 1 << vshift
  const int bsh = a.block_shift, bmask = (1 << bsh) - 1;
  const int v = tid & ((1 << vshift) - 1), rows = kThreads >> vshift;
  const bool is_v = v >= a.row_vecs;
  const size_t pitch = static_cast<size_t>(a.num_kv_heads) * a.row_vecs;
  uint4* pool = static_cast<uint4*>(is_v ? a.v_cache : a.k_cache) +
                static_cast<size_t>(kvh) * a.row_vecs + (is_v ? v - a.row_vecs : v);
  int2* moves = reinterpret_cast<int2*>(keys);             // (source, destination) slots
  const int per = (m + nc - 1) / nc;
  const int end = min(m, (rank + 1) * per);
  for (int base = rank * per; base < end; base += kKeys / 2) {
    const int n = min(end - base, kKeys / 2);
    for (int i = tid; i < n; i += kThreads) {
      const int j = base + i, t = __ldcg(kept + j);
      if (t < 0 || t >= len) {                 // a place left open by scores that changed
        moves[i] = make_int2(-1, -1);
        continue;
      }
      const int sb = stab[t >> bsh], db = dtab[j >> bsh];
      if (nsc) nsc[j] = sc[t];
      const bool ok = sb >= 0 && sb < a.num_blocks && db >= 0 && db < a.num_blocks;
      const int from = (sb << bsh) + (t & bmask), to = (db << bsh) + (j & bmask);
      if (!ok) report_error(a.err_flag, kErrBlockId);      // not copied
      moves[i] = ok ? make_int2(from, to) : make_int2(-1, -1);
      if (ok && a.k_scale) {
        const size_t f = ((static_cast<size_t>(sb) * a.num_kv_heads + kvh) << bsh) + (t & bmask);
        const size_t g = ((static_cast<size_t>(db) * a.num_kv_heads + kvh) << bsh) + (j & bmask);
        a.k_scale[g] = a.k_scale[f];
        a.v_scale[g] = a.v_scale[f];
      }
    }
    __syncthreads();
    for (int i0 = tid >> vshift; i0 < n; i0 += kMove * rows) {
      uint4 x[kMove];
      int to[kMove];
#pragma unroll
      for (int u = 0; u < kMove; ++u) {
        const int i = i0 + u * rows;
        const int2 mv = i < n ? moves[i] : make_int2(-1, -1);
        to[u] = mv.y;
        if (mv.y >= 0) x[u] = pool[mv.x * pitch];
      }
#pragma unroll
      for (int u = 0; u < kMove; ++u)
        if (to[u] >= 0) pool[to[u] * pitch] = x[u];
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a0, cudaStream_t stream) {
  EvictArgs a = a0;
  a.vec_shift = 0;
  while ((1 << a.vec_shift) < 2 * a.row_vecs) ++a.vec_shift;   // row_vecs and the block size
  a.block_shift = 0;                                           // are powers of two
  while ((1 << a.block_shift) < a.block_size) ++a.block_shift;
  int sms = 0;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  // CTAs per (sequence, kv head): until every SM has one, while each has 1024 tokens to
  // look at (a cluster's barriers and remote reads cost ~1 us a digit)
  const long long cap = static_cast<long long>(a.max_src_blocks) * a.block_size;
  const long long width = cap < a.score_stride ? cap : a.score_stride;
  const long long units = static_cast<long long>(a.num_seqs) * a.num_kv_heads;
  unsigned nc = 1;
  while (nc < kMaxCluster && units * nc < sms && width >= 2048LL * nc) nc *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(nc, a.num_kv_heads, a.num_seqs);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = nc;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_mode() != 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, evict_kernel, a);
}

}  // namespace pa

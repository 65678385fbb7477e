// pa_evict.cu -- eviction from the paged cache by accumulated attention weight
// (pa_evict) for sm_100a: per (sequence, kv head) the num_recent newest tokens and the
// highest-scored others stay, num_keep in all, and move to fresh blocks in their order.
//
// Which tokens stay is a selection of the r-th largest of up to max_blocks * block_size
// fp32 scores (r = num_keep - num_recent): scores become unsigned keys of the same
// order, and four passes of 8 bits count digits in shared memory and narrow the
// threshold's digits, most significant first.  Tokens above the threshold stay, and of
// those equal to it the first ones until r are found: whole-number counts, so the same
// tokens every time.  A block scan over the tokens in their order gives each kept one
// its place.
#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_tile.cuh"

namespace pa {
namespace {

constexpr int kSelThreads = 1024;

// Unsigned key with the order of the scores; NaN counts as lowest, -0 as 0.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0u;
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Sequence length if its tokens lie inside the table and the scores and what stays
// fits the new table and the outputs, else -1 (always checked).
__device__ __forceinline__ int checked_len(const EvictArgs& a, int s) {
  const int len = a.seq_lens[s];
  const long long cap = static_cast<long long>(a.max_src_blocks) * a.block_size;
  if (len < 0 || len > cap || len > a.score_stride) return -1;
  return min(len, a.num_keep) > a.max_kept ? -1 : len;
}

__global__ void __launch_bounds__(kSelThreads)
    evict_select_kernel(const __grid_constant__ EvictArgs a) {
  constexpr uint32_t FULL = 0xffffffffu;
  __shared__ uint32_t hist[256];
  __shared__ uint32_t pick[2];                 // digit, how many to take inside it
  __shared__ uint32_t wsum[2][32];
  const int kvh = blockIdx.x, s = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_launch_dependents();
  griddep_wait();
  const int len = checked_len(a, s);
  int* kept = a.kept + (static_cast<size_t>(s) * a.num_kv_heads + kvh) * a.kept_stride;
  if (len < 0) {                               // skipped: nothing kept
    if (tid == 0 && kvh == 0) {
      report_error(a.err_flag, kErrSeqLen);
      a.new_lens[s] = 0;
    }
    for (int i = tid; i < a.kept_stride; i += kSelThreads) kept[i] = -1;
    return;
  }
  const float* sc = a.scores + (static_cast<size_t>(s) * a.num_kv_heads + kvh) * a.score_stride;
  const int m = min(len, a.num_keep);
  const int old = max(0, len - a.num_recent);  // tokens that compete by score
  const int r = m - (len - old);               // how many of them stay
  uint32_t thr = 0, eq = 0;                    // key of the r-th largest, how many equal to it stay
  if (r > 0 && r < old) {
    uint32_t mask = 0, want = static_cast<uint32_t>(r);
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int t = tid; t < old; t += kSelThreads) {
        const uint32_t k = score_key(sc[t]);
        if ((k & mask) == thr) atomicAdd(&hist[(k >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (warp == 0) {                         // lane l: digits 255 - 8l .. 248 - 8l
        uint32_t c[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          c[i] = hist[255 - 8 * lane - i];
          sum += c[i];
        }
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
              pick[0] = 255 - 8 * lane - i;
              pick[1] = want - before;
            }
            before += c[i];
          }
        }
      }
      __syncthreads();
      thr |= pick[0] << shift;
      want = pick[1];
      mask |= 255u << shift;
      __syncthreads();
    }
    eq = want;
  }
  const bool all = r >= old, none = r <= 0;

  // ---- the kept ones in their order: chunks of one token per thread, two counts a
  // chunk (equal to the threshold, kept)
  uint32_t n_eq = 0, n_kept = 0;
  for (int base = 0; base < len; base += kSelThreads) {
    const int t = base + tid;
    const uint32_t k = t < old ? score_key(sc[t]) : 0u;
    const bool is_eq = !all && !none && t < old && k == thr;
    const uint32_t be = __ballot_sync(FULL, is_eq);
    if (lane == 0) wsum[0][warp] = __popc(be);
    __syncthreads();
    uint32_t rank = n_eq + __popc(be & ((1u << lane) - 1u)), tot = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) rank += wsum[0][w];
      tot += wsum[0][w];
    }
    n_eq += tot;
    const bool stay = t < len && (t >= old || all || (!none && (k > thr || (is_eq && rank < eq))));
    const uint32_t bk = __ballot_sync(FULL, stay);
    if (lane == 0) wsum[1][warp] = __popc(bk);
    __syncthreads();
    uint32_t at = n_kept + __popc(bk & ((1u << lane) - 1u));
    tot = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) at += wsum[1][w];
      tot += wsum[1][w];
    }
    n_kept += tot;
    if (stay) {
      kept[at] = t;
      if (a.new_scores)
        a.new_scores[(static_cast<size_t>(s) * a.num_kv_heads + kvh) * a.new_score_stride + at] = sc[t];
    }
    __syncthreads();
  }
  for (int i = m + tid; i < a.kept_stride; i += kSelThreads) kept[i] = -1;
  if (tid == 0 && kvh == 0) a.new_lens[s] = m;
}

// Move the kept rows: one warp per (place, kv head), a row's K and V by 16-byte vectors.
__global__ void __launch_bounds__(256)
    evict_move_kernel(const __grid_constant__ EvictArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int s = blockIdx.z, kvh = blockIdx.y;
  const int j = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (j >= a.max_kept) return;
  const int t = a.kept[(static_cast<size_t>(s) * a.num_kv_heads + kvh) * a.kept_stride + j];
  if (t < 0) return;
  const int bs = a.block_size;
  const int sb = a.src_tables[static_cast<size_t>(s) * a.max_src_blocks + t / bs];
  const int db = a.dst_tables[static_cast<size_t>(s) * a.max_dst_blocks + j / bs];
  if (sb < 0 || sb >= a.num_blocks || db < 0 || db >= a.num_blocks) {
    if (lane == 0) report_error(a.err_flag, kErrBlockId);
    return;
  }
  const size_t src = ((static_cast<size_t>(sb) * bs + t % bs) * a.num_kv_heads + kvh) * a.row_vecs;
  const size_t dst = ((static_cast<size_t>(db) * bs + j % bs) * a.num_kv_heads + kvh) * a.row_vecs;
  for (int i = lane; i < 2 * a.row_vecs; i += 32) {
    uint4* c = static_cast<uint4*>(i < a.row_vecs ? a.k_cache : a.v_cache);
    const int v = i < a.row_vecs ? i : i - a.row_vecs;
    c[dst + v] = c[src + v];
  }
  if (a.k_scale && lane < 2) {
    float* sc = lane == 0 ? a.k_scale : a.v_scale;
    sc[(static_cast<size_t>(db) * a.num_kv_heads + kvh) * bs + j % bs] =
        sc[(static_cast<size_t>(sb) * a.num_kv_heads + kvh) * bs + t % bs];
  }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
  const bool pdl = pdl_mode() != 0;
  cudaError_t e = launch_kernel(evict_select_kernel, dim3(a.num_kv_heads, a.num_seqs),
                                dim3(kSelThreads), 0, stream, pdl, a);
  if (e != cudaSuccess) return e;
  return launch_kernel(evict_move_kernel, dim3((a.max_kept + 7) / 8, a.num_kv_heads, a.num_seqs),
                       dim3(256), 0, stream, pdl, a);
}

}  // namespace pa

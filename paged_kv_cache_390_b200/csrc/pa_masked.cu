// pa_masked.cu -- paged attention with changed scores (pa_decode_masked,
// pa_prefill_masked): per query row at position pos of its sequence
//   x_t = cap * tanh(scale * q.K_t / cap)  (cap 0: scale * q.K_t)  - slope_h * |pos - t|
// over the tokens lo <= t < hi that the row sees,
//   lo = max(kv_start, pos - window + 1),  hi = min(len, max(pos + 1, prefix_len)),
//   out = softmax(x) V; a row that sees nothing gets zeros.
// pa_decode_masked also adds each cached token's weight, summed over the query heads of
// its kv head, to a running score: the attention leaves its scores x in the workspace and
// they come back as weights once the log-sum-exps are known, so K is not read twice (32
// bytes a token and kv head at 8 query heads, against 512 of K and V at 16 bits).
//
// Here: the CUDA-core form (fp32 caches; prefills that the tcgen05 kernel does not take),
// the second launch of the persistent decode, and the choice of form.  The tensor-core
// forms are the MASK builds of pa_decode_kernel.cuh and pa_fused_kernel.cuh and the MOD
// builds of pa_prefill_kernel.cuh.  Decode is bound by the cache's bytes: 8 x 32k tokens,
// bf16, with scores (1.04 GB) 202 us, 172 of them in the attention launch (6.0 TB/s);
// 32 x 640, fp16, capped (85 MB) 18.8 us; 64 windows of 4096, bf16 over FP8 (552 MB) 146 us,
// there by the widening of the codes (ALU pipe 58% busy).  The CUDA-core form is bound by
// its one chain of loads and exponentials per row and head: 1.3 to 2.4 TFLOP/s in prefill, and
// 29 ms for 8 x 32k tokens in fp32, 5 times the plain fp32 decode.
#include "pa_decode_kernel.cuh"
#include "pa_fused_kernel.cuh"
#include "pa_write.cuh"

namespace pa {
namespace {

template <typename KT, int NE>
__device__ __forceinline__ void load_row(const void* cache, size_t row, float scale, int lane,
                                         float (&x)[NE]) {
#pragma unroll
  for (int e = 0; e < NE; ++e) {
    const size_t i = row + lane + 32 * e;
    if constexpr (std::is_same<KT, int8_t>::value)
      x[e] = static_cast<float>(static_cast<const int8_t*>(cache)[i]) * scale;
    else if constexpr (std::is_same<KT, __nv_fp8_e4m3>::value)
      x[e] = static_cast<float>(static_cast<const __nv_fp8_e4m3*>(cache)[i]) * scale;
    else
      x[e] = to_f32<KT>(static_cast<const KT*>(cache)[i]);
  }
}

// One CTA per (query row, kv head, sequence); its warps take the group's query heads in
// turn, lanes split head_dim, one token at a time.
template <typename QT, typename KT, int D>
__global__ void __launch_bounds__(256)
    masked_rows_kernel(const __grid_constant__ MaskedArgs a) {
  constexpr int NE = D / 32;
  constexpr uint32_t FULL = 0xffffffffu;
  constexpr bool QUANT = sizeof(KT) == 1;
  const int r = blockIdx.x, kvh = blockIdx.y, s = blockIdx.z;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
  const int G = a.num_heads / a.num_kv_heads, BS = a.block_size;
  const bool prefill = a.query_start != nullptr;
  griddep_launch_dependents();
  griddep_wait();
  int len = a.seq_lens[s];
  const bool bad = len < 0 || static_cast<long long>(len) > static_cast<long long>(a.max_blocks) * BS;
  int row = s, pos = len - 1;
  if (prefill) {
    const int q0 = a.query_start[s], n = a.query_start[s + 1] - q0;
    if (bad || n < 0 || n > len || q0 < 0 || q0 > a.total_q - n) {
      if (r == 0 && threadIdx.x == 0 && a.err_flag) report_error(a.err_flag, kErrSeqLen);
      return;                                     // skipped
    }
    if (r >= n) return;
    row = q0 + r;
    pos = len - n + r;
  } else if (bad && a.err_flag) {
    if (threadIdx.x == 0) report_error(a.err_flag, kErrSeqLen);
    len = 0;                                      // skipped: zeros
    pos = -1;
  }
  const Span sp = seen_span(a.kv_start ? a.kv_start[row] : 0, pos, a.window,
                            a.prefix_lens ? a.prefix_lens[s] : 0, len);
  const int32_t* table = a.block_tables + static_cast<size_t>(s) * a.max_blocks;
  for (int g = warp; g < G; g += nwarps) {
    const int h = kvh * G + g;
    const size_t qrow = (static_cast<size_t>(row) * a.num_heads + h) * D;
    const float slope = a.slopes ? a.slopes[h] : 0.f;
    float q[NE], acc[NE];
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      q[e] = to_f32<QT>(static_cast<const QT*>(a.q)[qrow + lane + 32 * e]);
      acc[e] = 0.f;
    }
    float m2 = -INFINITY, l = 0.f;
    for (int t = sp.lo; t < sp.hi; ++t) {
      const int blk = table[t / BS];
      bool zero = false;
      float* lg = a.logits && t < a.score_stride
                      ? a.logits + ((static_cast<size_t>(s) * a.num_kv_heads + kvh) * a.score_stride + t) * G + g
                      : nullptr;
      if ((prefill || a.err_flag) && (blk < 0 || blk >= a.num_blocks)) {
        if (lane == 0 && a.err_flag) report_error(a.err_flag, kErrBlockId);
        if (!prefill) {                           // its tokens are dropped
          if (lg && lane == 0) *lg = -INFINITY;
          continue;
        }
        zero = true;                              // read as zeros
      }
      float k[NE], v[NE];
      if (zero) {
#pragma unroll
        for (int e = 0; e < NE; ++e) k[e] = v[e] = 0.f;
      } else {
        const size_t at = ((static_cast<size_t>(blk) * BS + t % BS) * a.num_kv_heads + kvh) * D;
        const size_t si = (static_cast<size_t>(blk) * a.num_kv_heads + kvh) * BS + t % BS;
        load_row<KT, NE>(a.k_cache, at, QUANT ? a.k_scale[si] : 1.f, lane, k);
        load_row<KT, NE>(a.v_cache, at, QUANT ? a.v_scale[si] : 1.f, lane, v);
      }
      float x = 0.f;
#pragma unroll
      for (int e = 0; e < NE; ++e) x = fmaf(q[e], k[e], x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(FULL, x, o);
      x *= a.scale;
      if (a.softcap > 0.f) x = a.softcap * tanhf(x / a.softcap);
      x = (x - slope * fabsf(static_cast<float>(pos - t))) * kLog2e;
      if (lg && lane == 0) *lg = x;
      const float mn = fmaxf(m2, x);
      const float al = mn == -INFINITY ? 1.f : exp2f(m2 - mn);
      const float p = x == -INFINITY ? 0.f : exp2f(x - mn);     // NaN stays NaN, the first too
      l = l * al + p;
#pragma unroll
      for (int e = 0; e < NE; ++e) acc[e] = fmaf(p, v[e], acc[e] * al);
      m2 = mn;
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // NaN stays NaN
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      const float o = acc[e] * inv;
      if constexpr (std::is_same<QT, float>::value)
        static_cast<float*>(a.out)[qrow + lane + 32 * e] = o;
      else if constexpr (std::is_same<QT, __half>::value)
        static_cast<__half*>(a.out)[qrow + lane + 32 * e] = __float2half_rn(o);
      else
        static_cast<__nv_bfloat16*>(a.out)[qrow + lane + 32 * e] = __float2bfloat16_rn(o);
    }
    if (a.lse && lane == 0)
      a.lse[static_cast<size_t>(s) * a.num_heads + h] = weight_lse(m2, l);
  }
}

// After the persistent form, per (sequence, kv head): CTA x = 0 merges the unit's records
// by log-sum-exp into out (a unit that one warp had to itself is already there), the
// others add the weights to the running scores, kTokens cached tokens each, from
// log-sum-exps that every CTA takes from the records' (m, l) for itself.  That takes five
// loads one after another, so a CTA has many tokens and four fit an SM (1024 tokens, two
// per SM: 37 us for 8 x 32k tokens).
// One warp per query head of the kv head; a merge keeps 8 records' loads in flight.
// The prefix and the records are the preceding launch's writes, which this one may overlap:
// their pointers carry no __restrict__, which would let the compiler take them for constant
// and load them on the read-only path or before griddepcontrol.wait.
constexpr int kFinish = 256, kTokens = 4096;

template <typename QT, int D>
__global__ void __launch_bounds__(kFinish, 4)
    masked_finish_kernel(const __grid_constant__ MaskedArgs a, const int* prefix,
                         const float* records, int warps) {
  constexpr uint32_t FULL = 0xffffffffu;
  constexpr int REC = 8 * D + 32;
  __shared__ float lse[kMaxGroup];
  griddep_launch_dependents();
  griddep_wait();
  const int kvh = blockIdx.y, s = blockIdx.z;
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int G = a.num_heads / a.num_kv_heads;
  const size_t row = static_cast<size_t>(s) * a.num_heads + kvh * G + g;
  // the split of pa_fused_kernel.cuh, in 32 bits (fewer than 2^31 tiles): its 64-bit
  // divisions, in every CTA here, were a third of this launch
  const unsigned total = prefix[a.num_seqs];
  const unsigned W = static_cast<unsigned>(masked_warps_used(total, warps));
  const unsigned c0 = prefix[s], nt = (prefix[s + 1] - c0) / a.num_kv_heads;
  const unsigned q = total / W, rem = total - q * W;
  auto range_start = [&](unsigned w) { return w * q + min(w, rem); };
  auto warp_of = [&](unsigned t) {
    return t < (q + 1) * rem ? t / (q + 1) : rem + (t - (q + 1) * rem) / q;
  };
  const unsigned start = c0 + kvh * nt;
  const unsigned wf = nt > 0 ? warp_of(start) : 0, wl = nt > 0 ? warp_of(start + nt - 1) : 0;
  const int n = nt > 0 ? static_cast<int>(wl - wf + 1) : 0;      // records (1: none was left)
  const int slot_f = nt > 0 && range_start(wf) == start ? 0 : 1;
  auto record = [&](int t) {
    return records + static_cast<size_t>(2 * (wf + t) + (t == 0 ? slot_f : 0)) * REC;
  };
  // a score CTA's own loads first: they do not depend on the log-sum-exps
  const int len = a.seq_lens[s];
  const bool bad = len < 0 ||
                   static_cast<long long>(len) > static_cast<long long>(a.max_blocks) * a.block_size;
  const int lo = seen_span(a.kv_start ? a.kv_start[s] : 0, len - 1, a.window, 0, len).lo;
  const int have = min(len, a.score_stride);
  const int from = (static_cast<int>(blockIdx.x) - 1) * kTokens;
  const size_t unit = (static_cast<size_t>(s) * a.num_kv_heads + kvh) * a.score_stride;
  constexpr int NT = 2;                           // tokens a thread has in flight
  float x[NT][kMaxGroup], before[NT];
  auto load = [&](int t0) {
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      const int t = t0 + u * kFinish + threadIdx.x;
      before[u] = t < have && a.scores_in ? a.scores_in[unit + t] : 0.f;
      load_scores(a.logits + (unit + t) * G, t >= lo && t < have, G, x[u]);
    }
  };
  if (blockIdx.x > 0) {
    if (bad || from >= have) return;              // a skipped sequence keeps its scores
    load(from);
  }
  // a unit that lost tiles to a wait that ran out: a marked record, or its own mark
  bool lost = n == 1 && a.lse && g < G && a.lse[row] == -INFINITY;
  float M = -INFINITY, L = 0.f;
  if (n > 1 && g < G) {
    for (int t = lane; t < n; t += 32) lost = lost || record(t)[kLostAt<D>] != 0.f;
    lost = __any_sync(FULL, lost);
    for (int t = lane; t < n; t += 32) M = fmaxf(M, record(t)[8 * D + g]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL, M, o));
    const float ms = M == -INFINITY ? 0.f : M;    // then L is 0, or NaN where all scores are
    for (int t = lane; t < n; t += 32)
      L += record(t)[8 * D + 8 + g] * fast_exp2(record(t)[8 * D + g] - ms);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(FULL, L, o);
  }
  if (blockIdx.x == 0) {
    if (n <= 1 || g >= G) return;
    constexpr int L4 = D / 4, PER = 32 / L4;     // lanes of a row, rows a warp takes at once
    const int d4 = lane % L4, sub = lane / L4;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int t0 = sub; t0 < n; t0 += 8 * PER) {
      float m[8];
      float4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int t = t0 + u * PER;
        m[u] = t < n ? record(t)[8 * D + g] : -INFINITY;
        v[u] = t < n ? reinterpret_cast<const float4*>(record(t) + g * D)[d4]
                     : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float w = M == -INFINITY ? 0.f : fast_exp2(m[u] - M);
        acc.x = fmaf(w, v[u].x, acc.x);
        acc.y = fmaf(w, v[u].y, acc.y);
        acc.z = fmaf(w, v[u].z, acc.z);
        acc.w = fmaf(w, v[u].w, acc.w);
      }
    }
    if constexpr (PER == 2) {
      acc.x += __shfl_xor_sync(FULL, acc.x, 16);
      acc.y += __shfl_xor_sync(FULL, acc.y, 16);
      acc.z += __shfl_xor_sync(FULL, acc.z, 16);
      acc.w += __shfl_xor_sync(FULL, acc.w, 16);
    }
    float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);        // NaN stays NaN
    if (lost) {
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
      inv = 0.f;
    }
    if (sub == 0) {
      uint2 pk;
      pk.x = pack2<QT>(acc.x * inv, acc.y * inv);
      pk.y = pack2<QT>(acc.z * inv, acc.w * inv);
      *reinterpret_cast<uint2*>(static_cast<QT*>(a.out) + row * D + 4 * d4) = pk;
    }
    return;
  }
  if (lane == 0) lse[g] = g >= G ? INFINITY : (n == 1 ? a.lse[row] : weight_lse(M, L));
  if (__syncthreads_or(lost)) return;             // its scores stay
  const int end = min(have, from + kTokens);
  for (int t0 = from; t0 < end; t0 += NT * kFinish) {
    float sum[NT];
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      const int t = t0 + u * kFinish + threadIdx.x;
      sum[u] = before[u] + (t >= lo ? token_weight(x[u], lse) : 0.f);
    }
    if (t0 + NT * kFinish < end) load(t0 + NT * kFinish);
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      const int t = t0 + u * kFinish + threadIdx.x;
      if (t < have) a.scores_out[unit + t] = sum[u];
    }
  }
}

// fp32 caches' running scores: one thread per (token, kv head, sequence).
__global__ void __launch_bounds__(256)
    masked_scores_kernel(const __grid_constant__ MaskedArgs a) {
  __shared__ float lse[kMaxGroup];
  griddep_launch_dependents();
  griddep_wait();
  const int kvh = blockIdx.y, s = blockIdx.z;
  const int len = a.seq_lens[s];
  if (len < 0 || static_cast<long long>(len) > static_cast<long long>(a.max_blocks) * a.block_size)
    return;                                       // a skipped sequence keeps its scores
  const int n = min(len, a.score_stride);
  if (blockIdx.x * 256 >= n) return;
  const int G = a.num_heads / a.num_kv_heads;
  if (threadIdx.x < kMaxGroup)
    lse[threadIdx.x] = threadIdx.x < G
                           ? a.lse[static_cast<size_t>(s) * a.num_heads + kvh * G + threadIdx.x]
                           : INFINITY;
  __syncthreads();
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t >= n) return;
  const Span sp = seen_span(a.kv_start ? a.kv_start[s] : 0, len - 1, a.window, 0, len);
  const size_t i = (static_cast<size_t>(s) * a.num_kv_heads + kvh) * a.score_stride + t;
  const float before = a.scores_in ? a.scores_in[i] : 0.f;
  float x[kMaxGroup];
  load_scores(a.logits + i * G, t >= sp.lo, G, x);
  a.scores_out[i] = before + (t >= sp.lo ? token_weight(x, lse) : 0.f);
}

template <typename QT, typename KT>
cudaError_t launch_rows(const MaskedArgs& a, int D, int rows, cudaStream_t s) {
  const int G = a.num_heads / a.num_kv_heads;
  const dim3 grid(rows, a.num_kv_heads, a.num_seqs), block(32 * (G < 8 ? G : 8));
  const bool pdl = pdl_mode() != 0;
  return D == 128 ? launch_kernel(masked_rows_kernel<QT, KT, 128>, grid, block, 0, s, pdl, a)
                  : launch_kernel(masked_rows_kernel<QT, KT, 64>, grid, block, 0, s, pdl, a);
}

template <typename QT>
cudaError_t launch_q(const MaskedArgs& a, int cache_dtype, int D, int rows, cudaStream_t s) {
  if (cache_dtype == PA_INT8) return launch_rows<QT, int8_t>(a, D, rows, s);
  if (cache_dtype == PA_FP8E4M3) return launch_rows<QT, __nv_fp8_e4m3>(a, D, rows, s);
  return launch_rows<QT, QT>(a, D, rows, s);
}

cudaError_t launch_attention(const MaskedArgs& a, int q_dtype, int cache_dtype, int D, int rows,
                             cudaStream_t s) {
  switch (q_dtype) {
    case PA_F32: return launch_rows<float, float>(a, D, rows, s);
    case PA_F16: return launch_q<__half>(a, cache_dtype, D, rows, s);
    case PA_BF16: return launch_q<__nv_bfloat16>(a, cache_dtype, D, rows, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

namespace {

template <typename QT, int KIND>
cudaError_t masked_shape(const FusedArgs& a, int D, int BS, size_t ws, cudaStream_t s,
                         const DecodeArgs* v1, const DecodeShape& sh, int* grid) {
#define PA_CASE(DD, BB) \
  if (D == DD && BS == BB)                                                             \
    return v1 ? launch_tc<QT, KIND, DD, BB, true>(*v1, sh, s)                          \
              : launch_fused_t<QT, KIND, DD, BB, true>(a, ws, s, grid);
  PA_CASE(128, 16)
  PA_CASE(128, 8)
  PA_CASE(128, 32)
  PA_CASE(64, 16)
  PA_CASE(64, 8)
  PA_CASE(64, 32)
#undef PA_CASE
  return cudaErrorInvalidValue;
}

// The persistent form, or with v1 the one-CTA-per-(sequence, kv head) form.
cudaError_t launch_masked_tc(const FusedArgs& a, int q_dtype, int cache_dtype, int D, int BS,
                             size_t ws, cudaStream_t s, const DecodeArgs* v1,
                             const DecodeShape& sh, int* grid) {
  const bool qh = q_dtype == PA_F16;
  switch (cache_dtype) {
    case PA_F16: return masked_shape<__half, kKind16>(a, D, BS, ws, s, v1, sh, grid);
    case PA_BF16: return masked_shape<__nv_bfloat16, kKind16>(a, D, BS, ws, s, v1, sh, grid);
    case PA_INT8:
      return qh ? masked_shape<__half, kKindI8>(a, D, BS, ws, s, v1, sh, grid)
                : masked_shape<__nv_bfloat16, kKindI8>(a, D, BS, ws, s, v1, sh, grid);
    case PA_FP8E4M3:
      return qh ? masked_shape<__half, kKindE4M3>(a, D, BS, ws, s, v1, sh, grid)
                : masked_shape<__nv_bfloat16, kKindE4M3>(a, D, BS, ws, s, v1, sh, grid);
  }
  return cudaErrorInvalidValue;
}

// Warps per CTA of the one-CTA form, as pa_decode_v1 chooses them.
int masked_warps(int cache_dtype) {
  return cache_dtype == PA_INT8 || cache_dtype == PA_FP8E4M3 ? kMaxWarps : kDefaultWarps;
}

// One CTA per (sequence, kv head), or the persistent form, which spreads long or few units
// over every SM at the price of a second launch.  By the most tiles a unit can have
// (table width or window); device times, one CTA / persistent, lengths even in [L/2, L]:
//   16-bit, 64/8 heads   L 768: 8.8 / 12.1 us (2 sequences), 17.7 / 22.4 (32), 32.1 / 34.6 (64)
//                        L 1500: 20.5 / 14.2 (2), 24.9 / 24.3 (19), 30.0 / 32.0 (32)
//                        L 3000: 38.3 / 20.4 (2), 45.5 / 35.7 (19), 97.2 / 97.6 (64)
//   FP8, 32/8 heads      L 512: 9.4 / 9.4 (2), L 1500: 16.1 / 14.3 (2), 51.3 / 53.5 (64)
// Under a window the lengths are alike and the CTAs even: 64 sequences, window 4096, FP8:
// 144.8 / 156.4.
bool pick_one_cta(const MaskedArgs& a, int cache_dtype, int num_sms) {
  long long most = static_cast<long long>(a.max_blocks) * a.block_size;   // tokens a row sees
  const bool even = a.window > 0 && a.window + 15LL < most;
  if (even) most = a.window + 15LL;
  const long long tiles = (most + 15) / 16;
  const long long units = static_cast<long long>(a.num_seqs) * a.num_kv_heads;
  return tiles <= 8 * masked_warps(cache_dtype) ||
         (2 * units >= 3LL * num_sms && tiles <= (even ? 288 : 192));
}

size_t lse_bytes(int num_seqs, int num_heads) {
  return (static_cast<size_t>(num_seqs) * num_heads * sizeof(float) + 255) / 256 * 256;
}
}  // namespace

// The persistent decode's workspace (the tile prefix, then the records), then lse, then
// the scores x of every cached token.
size_t masked_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                              int score_width, int num_sms) {
  return fused_workspace_bytes(num_seqs + 1, num_kv_heads, head_dim, num_sms) +
         lse_bytes(num_seqs, num_heads) +
         static_cast<size_t>(num_seqs) * num_heads * score_width * sizeof(float);
}

cudaError_t launch_decode_masked(const MaskedArgs& a0, int q_dtype, int cache_dtype, int head_dim,
                                 void* workspace, int num_sms, cudaStream_t s) {
  MaskedArgs a = a0;
  if (a.scores_out) {
    char* ws = static_cast<char*>(workspace) +
               fused_workspace_bytes(a.num_seqs + 1, a.num_kv_heads, head_dim, num_sms);
    a.lse = reinterpret_cast<float*>(ws);
    a.logits = reinterpret_cast<float*>(ws + lse_bytes(a.num_seqs, a.num_heads));
  }
  cudaError_t e;
  if (cache_dtype == PA_F32) {
    e = launch_rows<float, float>(a, head_dim, 1, s);
  } else {
    FusedArgs f{};
    f.out = a.out;
    f.q = a.q;
    f.k_cache = a.k_cache;
    f.v_cache = a.v_cache;
    f.k_scale = a.k_scale;
    f.v_scale = a.v_scale;
    f.block_tables = a.block_tables;
    f.seq_lens = a.seq_lens;
    f.err_flag = a.err_flag;
    f.counters = static_cast<int*>(workspace);
    f.max_blocks = a.max_blocks;
    f.num_seqs = a.num_seqs;
    f.num_heads = a.num_heads;
    f.num_kv_heads = a.num_kv_heads;
    f.num_blocks = a.num_blocks;
    f.stages = 2;
    f.scale_log2 = a.scale * kLog2e;
    f.timeout_ns = a.timeout_ns;
    f.inject = a.inject;
    f.pdl = pdl_mode() != 0 ? 1 : 0;         // kv_start is read with the lengths: after the wait
    f.slopes = a.slopes;
    f.kv_start = a.kv_start;
    f.cap_in = a.softcap > 0.f ? a.scale / a.softcap : 0.f;
    f.cap_log2 = a.softcap * kLog2e;
    f.window = a.window;
    f.lse = a.lse;
    f.logits = a.logits;
    f.score_stride = a.score_stride;
    DecodeShape sh{};
    const bool one_cta = pick_one_cta(a, cache_dtype, num_sms);
    DecodeArgs d{};
    if (one_cta) {
      sh.warps = masked_warps(cache_dtype);
      sh.grid_x = 1;
      d.out = a.out;
      d.q = a.q;
      d.k_cache = a.k_cache;
      d.v_cache = a.v_cache;
      d.k_scale = a.k_scale;
      d.v_scale = a.v_scale;
      d.block_tables = a.block_tables;
      d.seq_lens = a.seq_lens;
      d.err_flag = a.err_flag;
      d.max_blocks = a.max_blocks;
      d.num_seqs = a.num_seqs;
      d.num_heads = a.num_heads;
      d.num_kv_heads = a.num_kv_heads;
      d.num_blocks = a.num_blocks;
      d.stages = default_stages(cache_dtype, head_dim, a.block_size, sh.warps, 96);
      d.scale_log2 = f.scale_log2;
      d.timeout_ns = a.timeout_ns;
      d.inject = a.inject;
      d.pdl = f.pdl;
      d.slopes = a.slopes;
      d.kv_start = a.kv_start;
      d.cap_in = f.cap_in;
      d.cap_log2 = f.cap_log2;
      d.window = a.window;
      d.scores_in = a.scores_in;
      d.scores_out = a.scores_out;
      d.logits = a.logits;
      d.score_stride = a.score_stride;
    }
    int ctas = 0;
    e = launch_masked_tc(f, q_dtype, cache_dtype, head_dim, a.block_size,
                         fused_workspace_bytes(a.num_seqs + 1, a.num_kv_heads, head_dim, num_sms), s,
                         one_cta ? &d : nullptr, sh, &ctas);
    if (one_cta || e != cudaSuccess) return e;   // its CTAs add the running scores themselves
    const float* records = reinterpret_cast<const float*>(
        static_cast<char*>(workspace) + fused_counter_bytes(a.num_seqs + 1, a.num_kv_heads));
    const int* prefix = static_cast<const int*>(workspace);
    int chunks = 0;
    if (a.scores_out) {
      const long long cap = static_cast<long long>(a.max_blocks) * a.block_size;
      chunks = static_cast<int>(((cap < a.score_stride ? cap : a.score_stride) + kTokens - 1) / kTokens);
    }
    const dim3 grid(1 + chunks, a.num_kv_heads, a.num_seqs);
    const bool pdl = pdl_mode() != 0, wide = head_dim == 128;
    auto kern = q_dtype == PA_BF16 ? (wide ? masked_finish_kernel<__nv_bfloat16, 128>
                                           : masked_finish_kernel<__nv_bfloat16, 64>)
                                   : (wide ? masked_finish_kernel<__half, 128>
                                           : masked_finish_kernel<__half, 64>);
    return launch_kernel(kern, grid, dim3(kFinish), 0, s, pdl, a, prefix, records,
                         ctas * kFusedWarps);
  }
  if (e != cudaSuccess || !a.scores_out) return e;
  const long long cap = static_cast<long long>(a.max_blocks) * a.block_size;
  const int width = static_cast<int>(cap < a.score_stride ? cap : a.score_stride);
  return launch_kernel(masked_scores_kernel, dim3((width + 255) / 256, a.num_kv_heads, a.num_seqs),
                       dim3(256), 0, s, pdl_mode() != 0, a);
}

cudaError_t launch_prefill_masked(const MaskedArgs& a, int q_dtype, int cache_dtype, int head_dim,
                                  int max_query_len, cudaStream_t s) {
  if (max_query_len > a.total_q) max_query_len = a.total_q;     // longer ones are skipped
  if (head_dim != 128 || cache_dtype != q_dtype || q_dtype == PA_F32)
    return launch_attention(a, q_dtype, cache_dtype, head_dim, max_query_len, s);
  PrefillArgs p{};
  p.out = a.out;
  p.q = a.q;
  p.k_cache = a.k_cache;
  p.v_cache = a.v_cache;
  p.block_tables = a.block_tables;
  p.seq_lens = a.seq_lens;
  p.query_start = a.query_start;
  p.err_flag = a.err_flag;
  p.max_blocks = a.max_blocks;
  p.num_seqs = a.num_seqs;
  p.num_heads = a.num_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.num_blocks = a.num_blocks;
  p.scale_log2 = a.scale * kLog2e;
  p.timeout_ns = a.timeout_ns;
  p.inject = a.inject;
  p.slopes = a.slopes;
  p.kv_start = a.kv_start;
  p.prefix_lens = a.prefix_lens;
  p.cap_in = a.softcap > 0.f ? a.scale / a.softcap : 0.f;
  p.cap_log2 = a.softcap * kLog2e;
  p.window = a.window;
  p.total_q = a.total_q;
  p.block_size = a.block_size;
  return launch_prefill_masked_tc(p, q_dtype, max_query_len, s);
}

}  // namespace pa

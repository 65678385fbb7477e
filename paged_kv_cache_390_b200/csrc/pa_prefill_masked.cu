// pa_prefill_masked.cu -- launches of pa_prefill_masked's tcgen05 form (the kernel is in
// pa_prefill_kernel.cuh).
#include "pa_prefill_kernel.cuh"

namespace pa {
namespace {

template <int BS>
cudaError_t kv_maps(CUtensorMap* mk, CUtensorMap* mv, const PrefillArgs& a) {
  cudaError_t e = make_cache_map<kKind16, kD, BS>(mk, a.k_cache, a.num_kv_heads, a.num_blocks);
  if (e != cudaSuccess) return e;
  return make_cache_map<kKind16, kD, BS>(mv, a.v_cache, a.num_kv_heads, a.num_blocks);
}

template <typename QT, int MOD>
cudaError_t launch_mod(const PrefillArgs& a, int max_query_len, cudaStream_t stream) {
  const int G = a.num_heads / a.num_kv_heads;
  CUtensorMap mq, mk, mv;
  cudaError_t e = make_q_map(&mq, a.q, a.total_q, a.num_heads, G);
  if (e != cudaSuccess) return e;
  switch (a.block_size) {
    case 8: e = kv_maps<8>(&mk, &mv, a); break;
    case 16: e = kv_maps<16>(&mk, &mv, a); break;
    default: e = kv_maps<32>(&mk, &mv, a); break;
  }
  if (e != cudaSuccess) return e;
  auto kern = prefill_kernel<QT, 0, MOD>;
  static int configured[64] = {0};
  e = opt_in_smem(reinterpret_cast<const void*>(kern), kSmemBytes, configured);
  if (e != cudaSuccess) return e;
  const int rows_per_cta = kQTiles * (kRows / G);
  const int tiles = (max_query_len + rows_per_cta - 1) / rows_per_cta;
  const int ng = tiles < kTileGroup ? tiles : kTileGroup;
  // Few query tiles over long contexts: the CTAs of a cluster share a tile's KV tiles, two
  // at least each, while that leaves every cluster its own SMs.  fp16, cap, prefix, one CTA
  // a tile / shared: 20 rows over 1.5k tokens, 8/1 heads 60.5 / 29.8 us; 64 rows over 16k,
  // 32/8 heads 570 / 83; 4 x 64 over 4k, 32/4 heads 155 / 55; 256 over 1k, 32/4 heads 55 / 32.
  int sms = 0;
  e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  long long seen = static_cast<long long>(a.max_blocks) * a.block_size;   // tokens a CTA may see
  if (a.window > 0 && !a.prefix_lens && a.window + 1LL * rows_per_cta < seen)
    seen = a.window + 1LL * rows_per_cta;
  const long long kv_tiles = (seen + kBN - 1) / kBN;
  const long long ctas = static_cast<long long>(tiles) * a.num_kv_heads * a.num_seqs;
  unsigned nsplit = 1;
  while (nsplit < kMaxSplit && 2 * nsplit * ctas <= sms && kv_tiles >= 4 * nsplit) nsplit *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ng * a.num_kv_heads * nsplit, a.num_seqs, (tiles + ng - 1) / ng);
  cfg.blockDim = dim3(prefill_threads<MOD>());
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  if (nsplit > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = nsplit;
    attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (pdl_mode() != 0) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  return cudaLaunchKernelEx(&cfg, kern, mq, mk, mv, a);
}

template <typename QT>
cudaError_t launch_q(const PrefillArgs& a, int max_query_len, cudaStream_t s) {
  switch ((a.cap_in != 0.f ? 1 : 0) | (a.slopes ? 2 : 0)) {
    case 0: return launch_mod<QT, 0>(a, max_query_len, s);
    case 1: return launch_mod<QT, 1>(a, max_query_len, s);
    case 2: return launch_mod<QT, 2>(a, max_query_len, s);
  }
  return launch_mod<QT, 3>(a, max_query_len, s);
}

}  // namespace

cudaError_t launch_prefill_masked_tc(const PrefillArgs& a, int q_dtype, int max_query_len,
                                     cudaStream_t s) {
  return q_dtype == PA_BF16 ? launch_q<__nv_bfloat16>(a, max_query_len, s)
                            : launch_q<__half>(a, max_query_len, s);
}

}  // namespace pa

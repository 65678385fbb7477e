// pa_score.cuh -- the changed scores of pa_decode_masked / pa_prefill_masked: the tanh cap,
// the bias by distance and the span of tokens a query row sees.
#pragma once

#include <stdint.h>

namespace pa {

constexpr float kLog2e = 1.4426950408889634f;

// Tokens [lo, hi) that a row at position pos sees.
struct Span {
  int lo, hi;
};

__device__ __forceinline__ Span seen_span(int start, int pos, int window, int prefix, int len) {
  Span s;
  s.lo = max(start, 0);
  if (window > 0) s.lo = max(s.lo, pos - window + 1);
  s.hi = min(len, max(pos + 1, prefix));
  return s;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh(y) to ~2 ulp.  Below 0.625 an odd polynomial y + y z Q(z), z = y^2, with Q of
// degree 4 interpolating (tanh(y) / y - 1) / z at the Chebyshev points of [0, 0.625^2]
// (2e-8 relative); above, 1 - 2 / (1 + e^(2|y|)), whose error is absolute (2^-23) and so
// relative there.  (Near 0 that form alone would lose the digits of a small score, and
// a score carries into its weight absolutely: cap 50 would leave 1e-5 on every weight.)
__device__ __forceinline__ float tanh_f32(float y) {
  const float a = fabsf(y), z = y * y;
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(a * (2.f * kLog2e)));
  const float big = copysignf(fmaf(-2.f, rcp_approx(e + 1.f), 1.f), y);
  float q = fmaf(z, -0.006096714176237583f, 0.020997179672122f);
  q = fmaf(z, q, -0.05385090783238411f);
  q = fmaf(z, q, 0.1333276927471161f);
  q = fmaf(z, q, -0.333333283662796f);
  return a < 0.625f ? fmaf(y * z, q, y) : big;
}

// Warps that share out `tiles` 16-token tiles: all of them, but at least 4 tiles each (a
// record to write and merge costs about as much as a tile or two).
__host__ __device__ __forceinline__ long long masked_warps_used(long long tiles, long long warps) {
  const long long most = (tiles + 3) / 4;
  return most < 1 ? 1 : (most < warps ? most : warps);
}

// A cached token's scores x under the G (up to 8) query heads of its kv head, log2 units;
// -inf where it is not seen.
__device__ __forceinline__ void load_scores(const float* p, bool seen, int G, float (&x)[8]) {
  if ((G & 3) == 0) {
#pragma unroll
    for (int g = 0; g < 8; g += 4) {
      float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (seen && g < G) v = *reinterpret_cast<const float4*>(p + g);
      x[g] = v.x;
      x[g + 1] = v.y;
      x[g + 2] = v.z;
      x[g + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int g = 0; g < 8; ++g) x[g] = seen && g < G ? p[g] : -INFINITY;
  }
}

// A head's log-sum-exp (log2 units) from its maximum and sum; +inf, which makes every
// weight 0, where its row saw nothing.
__device__ __forceinline__ float weight_lse(float M, float L) {
  return L > 0.f || L != L ? M + log2f(L) : INFINITY;
}

// A seen token's weight, summed over the heads (lse: 8 of them, +inf past G).  Not for
// others: where a head's row is NaN, -inf would give NaN too.
__device__ __forceinline__ float token_weight(const float (&x)[8], const float* lse) {
  float w = 0.f;
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    float p;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(x[g] - lse[g]));
    w += p;
  }
  return w;
}

}  // namespace pa

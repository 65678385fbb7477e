"""The rotary cache write, masked attention and cache eviction in plain 64-bit torch on
the CPU, from their definitions (no code of the library), and the tolerances.

A result rounded to a type T is off by at most half a step, eps(T) / 2 relative.  The
kernels round once at the end and hold everything else in 32 bits (and P of the
attention in 16 bits, see `attention_tol`)."""
import math

import torch


def half_step(dt):
    return torch.finfo(dt).eps / 2


def rope(x, positions, inv_freq, pair_axis, interleaved):
    """x [T, heads, D] turned, in 64 bits."""
    x = x.double().clone()
    T, _, D = x.shape
    pairs = inv_freq.numel()
    for i in range(pairs):
        ax = int(pair_axis[i])
        if not 0 <= ax < positions.shape[0]:
            continue
        ang = positions[ax].double() * inv_freq[i].double()
        c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        a, b = x[:, :, ia].clone(), x[:, :, ib].clone()
        x[:, :, ia] = a * c - b * s
        x[:, :, ib] = a * s + b * c
    return x


def rope_tol(x64, dt):
    """Elementwise bound on a turned row in dtype dt: half a step of dt at the value,
    plus the 32-bit arithmetic: sine and cosine to 2 ulp of the reduced angle in 32 bits
    (4 * 2^-24 absolute in all) and three roundings, on |a| + |b| <= 2 max|row|."""
    mag = x64.abs().amax(-1, keepdim=True)
    tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    return half_step(dt) * x64.abs() * (1 + 2.0 ** -10) + 2 * mag * (4 + 3) * 2.0 ** -24 + tiny


def evict(scores, lens, num_keep, num_recent):
    """Kept token lists [S][H_kv], from the definition."""
    out = []
    for s, n in enumerate(lens):
        per = []
        for h in range(scores.shape[1]):
            row = scores[s, h].tolist()
            new = list(range(max(0, n - num_recent), n))
            old = [i for i in range(max(0, n - num_recent))]
            val = {i: (-math.inf if math.isnan(row[i]) else row[i]) for i in old}
            # NaN below every number, then by score, then the earlier token
            old.sort(key=lambda i: (math.isnan(row[i]), -val[i], i))
            m = min(n, num_keep)
            per.append(sorted(new + old[:m - len(new)]))
        out.append(per)
    return out


# ---------------------------------------------------------------------- attention

def attend(q, k, v, scale, lo, hi, pos, softcap=0.0, slopes=None):
    """One sequence, rows of one call: q [R, H, D], k, v [n, Hkv, D] (64-bit values), lo, hi,
    pos per row.  Only seen tokens enter (unseen ones may hold anything).  Returns out
    [R, H, D], weights [R, H, n], bound terms: dx [R, H] (how far a score may be off in
    32-bit arithmetic) and wv [R, H, D] = sum w |v|."""
    R, H, D = q.shape
    n, Hkv, _ = k.shape
    G = H // Hkv
    out, w = torch.zeros(R, H, D, dtype=torch.float64), torch.zeros(R, H, n, dtype=torch.float64)
    dx, wv = torch.zeros(R, H, dtype=torch.float64), torch.zeros(R, H, D, dtype=torch.float64)
    q = q.double()
    for r in range(R):
        a, b = int(lo[r]), int(hi[r])
        if a >= b:
            continue
        kk = k[a:b].repeat_interleave(G, dim=1)                 # [m, H, D]
        vv = v[a:b].repeat_interleave(G, dim=1)
        x = torch.einsum("hd,mhd->hm", q[r], kk) * scale
        size = torch.einsum("hd,mhd->hm", q[r].abs(), kk.abs()) * abs(scale)
        if softcap:
            x = softcap * torch.tanh(x / softcap)
        bias = torch.zeros_like(x)
        if slopes is not None:
            dist = (int(pos[r]) - torch.arange(a, b)).abs().double()
            bias = slopes.double()[:, None] * dist
        x = x - bias
        p = torch.softmax(x, dim=1)
        w[r, :, a:b] = p
        out[r] = torch.einsum("hm,mhd->hd", p, vv)
        wv[r] = torch.einsum("hm,mhd->hd", p, vv.abs())
        # D products summed (each step to 2 ulp: matrix units may truncate), the cap's tanh
        # to 4 ulp of the cap, the bias to 2, and 8 more on the score and exponent itself;
        # only tokens whose weight counts (a score off by e moves its weight by w * e)
        off = 2.0 ** -23 * ((D + 8) * size + 4 * softcap + 2 * bias + 8 * (x.abs() + 1))
        dx[r] = torch.where(p > 2.0 ** -30, off, torch.zeros_like(off)).amax(1)
    return out, w, dx, wv


def attention_tol(out, dx, wv, dt, cache, n, vmax, smax=0.0):
    """Elementwise bound on an attention output: half a step of dt; scores off by dx move
    every weight and the sum by a factor exp(+-dx) each (2 dx); the running sums' 32-bit
    rescaling, 2^-18; P in 16 bits: fp16 half a step 2^-11 and 2^-25 absolute below
    its normal range (n tokens), bf16 as two parts 2^-16; INT8 under fp16: codes enter
    as 1152 + c, whose sum is held in 32 bits (n / 16 + 8 roundings)."""
    p_err = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -16, torch.float32: 0.0}[dt]
    tol = half_step(dt) * out.abs() * (1 + 2.0 ** -9) + (p_err + 2 * dx[..., None] + 2.0 ** -18) * wv
    tol = tol + n * 2.0 ** -25 * vmax
    if cache == "int8" and dt == torch.float16:
        tol = tol + (n / 16 + 8) * 2.0 ** -24 * 1152 * smax
    return tol + 2.0 ** -24 * torch.finfo(dt).smallest_normal


def scores_tol(scores, w_sum, dx):
    """Bound on running scores [.., n]: w off by a factor exp(2 dx) and 2^-19 (exponentials
    and log-sum-exp in 32 bits), one rounding of the sum over the group and one of the
    total."""
    return w_sum * (2 * dx + 2.0 ** -19) + 2.0 ** -23 * scores.abs() + 2.0 ** -40

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

"""pa_decode_masked and pa_prefill_masked where single bits, infinities and NaN, missing
blocks or waits that run out decide: against plain 64-bit arithmetic, with tolerances that
count each rounding."""
import pytest
import torch

import _plain64 as p64
from test_masked import DT, Batch, _close, _decode, _prefill, _wide

HEADS = 8


def _scores_near(dt, cap, tops, n, seed):
    """Sequences of n tokens whose scores (before the cap) are known without error and lie
    within a few units below tops[s] * cap: K holds a score as two numbers of `dt`, q adds
    them up.  V is zero but for two tokens per (head, dim), whose products with the weights
    nearly cancel, so that the output shows the weights' ratio and not its own rounding."""
    g = torch.Generator().manual_seed(seed)
    t, D = DT[dt], 128
    b = Batch(dt, dt, [n] * len(tops), [2] * len(tops), HEADS, HEADS, D, 16, seed, softcap=cap)
    b.scale = 1.0
    b.q = torch.zeros_like(b.q)
    b.q[..., :2] = 1.0
    for s, top in enumerate(tops):
        x = top * cap - 6.0 * torch.rand((n, HEADS), generator=g, dtype=torch.float64)
        hi = x.to(t).double()
        lo = (x - hi).to(t).double()
        w = torch.softmax(cap * torch.tanh((hi + lo) / cap), dim=0)        # [n, heads]
        pair = torch.stack([torch.randperm(n - 1, generator=g)[:2] for _ in range(HEADS * D)])
        pair = pair.view(HEADS, D, 2)
        k = torch.zeros(n, HEADS, D, dtype=torch.float64)
        v = torch.zeros(n, HEADS, D, dtype=torch.float64)
        k[..., 0], k[..., 1] = hi, lo
        for h in range(HEADS):
            i, j = pair[h, :, 0], pair[h, :, 1]
            d = torch.arange(D)
            v[i, h, d] = 1.0
            v[j, h, d] = -(w[i, h] / w[j, h])
        at = [b.at(s, i) for i in range(n)]
        for x64, val, pool in zip((k, v), b.val, b.kv):
            pool.flatten(0, 1)[at] = x64.to(t)
            val.flatten(0, 1)[at] = x64.to(t).double()
    return b


def _ratio_tol(b, want, wv, top, wmax):
    """Half a step of the output's type; P in two 16-bit parts: 2^-16, and for fp16 2^-25 of
    the largest weight below its normal range, times the largest V (e^6, two tokens); two
    weights, whose scores are each off by 6 units of the score in 2^-24 (the tanh to 4, its
    product with the cap, scale / cap) and 24 of the exponent (16 or less) and the
    exponential; sums 2^-18."""
    dx = 2.0 ** -24 * (6 * min(top, 1.0) * b.softcap + 24)
    floor = 2 * 2.0 ** -25 * 404 * wmax if b.dt == torch.float16 else 0.0
    tiny = 2.0 ** -25 if b.dt == torch.float16 else 0.0           # fp16's step near 0
    return (p64.half_step(b.dt) * want.abs() * (1 + 2.0 ** -9)
            + (2.0 ** -16 + 2 * dx + 2.0 ** -18) * wv + floor + tiny)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("alibi", [False, True])
@pytest.mark.parametrize("cap", [50.0, 300.0, 3000.0])
def test_weights_under_any_cap(pa, dt, alibi, cap):
    """Scores over the whole unit range of the cap and past it (where a row of the same
    warp needs more than the polynomial): prefill and decode to the 32-bit arithmetic's
    error, whatever the cap is."""
    tops = (0.3, 0.6, 0.9, 1.0, 1.3)
    b = _scores_near(dt, cap, tops, 90, 3)
    if alibi:                                          # a bias of zero: the biased build
        b.slopes = torch.zeros(HEADS)
    pre = _prefill(pa, b).cpu().double()
    last = [2 * s + 1 for s in range(len(tops))]
    b1 = Batch.__new__(Batch)
    b1.__dict__.update(b.__dict__, q=b.q[last].contiguous())
    dec = _decode(pa, b1).cpu().double()
    for s, top in enumerate(tops):
        n = b.lens[s]
        at = [b.at(s, t) for t in range(n)]
        k, v = (x.flatten(0, 1)[at] for x in b.val)
        lo, hi, pos = b.rows[s]
        o, w, _, wv = p64.attend(b.q[2 * s:2 * s + 2], k, v, 1.0, lo, hi, pos, cap, b.slopes)
        tol = _ratio_tol(b, o, wv, top, float(w.max()))
        assert ((pre[2 * s:2 * s + 2] - o).abs() <= tol).all(), \
            (s, float(((pre[2 * s:2 * s + 2] - o).abs() / tol).max()))
        assert ((dec[s] - o[1]).abs() <= tol[1]).all(), (s, float(((dec[s] - o[1]).abs() / tol[1]).max()))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("alibi", [False, True])
@pytest.mark.parametrize("H,Hkv", [(8, 8), (8, 2)])
def test_unseen_keys_leave_every_bit_alone(pa, dt, alibi, H, Hkv):
    """Rows of several documents: the keys of one document small or a hundred times larger
    (past the polynomial's range); the rows of the others do not see them, and come out
    the same in every bit."""
    n = 200
    starts = [0 if p < 70 else (70 if p < 130 else 130) for p in range(n)]
    outs = []
    for mul in (1.0, 100.0):
        b = Batch(dt, dt, [n, 40], [n, 40], H, Hkv, 128, 16, 12, softcap=8.0, alibi=alibi,
                  starts=starts + [0] * 40)
        for t in range(70, 130):
            b.kv[0].flatten(0, 1)[b.at(0, t)] *= mul
        for t in range(40, 48):                        # behind the end of sequence 1
            b.kv[0].flatten(0, 1)[b.at(1, t)] = mul
        outs.append(_prefill(pa, b).cpu())
    assert torch.equal(outs[0][:70], outs[1][:70]) and torch.equal(outs[0][130:], outs[1][130:])
    assert torch.isfinite(outs[1]).all() and not torch.equal(outs[0][70:130], outs[1][70:130])


def _v_scales(b, how):
    """Sequence by sequence, a factor on each token's V scale (a power of two), sign included
    for "signs"."""
    for s, n in enumerate(b.lens):
        for t in range(n):
            f = {"spikes": 2.0 ** 24 if t % 16 == 3 and t < n - 40 else 1.0,
                 "spikes 2^60": 2.0 ** 60 if t % 16 == 3 and t < n - 100 else 1.0,
                 "first": 2.0 ** 20 if t < 32 else 1.0,
                 "falling": 2.0 ** (40 - 40 * t // max(1, n)),
                 "rising": 2.0 ** (40 * t // max(1, n) - 40),
                 "signs": -1.0 if t % 3 == 0 else 1.0,
                 "tiny": 2.0 ** -16}[how]
            blk, off = divmod(b.at(s, t), b.bs)
            b.sc[1][blk, :, off] *= f
            b.val[1][blk, off] *= f


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True], ids=["one-cta", "persistent"])
@pytest.mark.parametrize("cd", ["int8", "fp8"])
@pytest.mark.parametrize("how", ["spikes", "spikes 2^60", "first", "falling", "rising", "signs", "tiny"])
@pytest.mark.parametrize("slope", [1.0, 0.125, 0.0])
def test_decode_bf16_v_scales_by_their_weight(pa, cd, how, slope, wide):
    """V scales that differ by many powers of two: tokens with the largest ones and a
    vanishing weight take nothing from the others, as the maximum of the scores rises
    token by token (a steep bias) or not."""
    b = Batch("bf16", cd, [300, 40, 150], [1] * 3, 8, 2, 64, 16, 41)
    b.slopes = slope * torch.linspace(1.0, 1.5, 8)
    _v_scales(b, how)
    if wide:
        _wide(b)
    got = _decode(pa, b).cpu().double()
    for s, n in enumerate(b.lens):
        k, v = (x.flatten(0, 1)[[b.at(s, t) for t in range(n)]] for x in b.val)
        lo, hi, pos = b.rows[s]
        o, w, dx, wv = p64.attend(b.q[s:s + 1], k, v, b.scale, lo, hi, pos, 0.0, b.slopes)
        # P times the V scale in two fp16 parts: 2^-22, and 2^-26 of the largest such product
        # for each token (times the largest code); weights 2 dx, sums 2^-18
        top = v.abs().amax(-1).repeat_interleave(4, dim=1).T              # [H, n]
        peak = (w[0] * top).amax(1)[None, :, None]
        tol = (p64.half_step(torch.bfloat16) * o.abs() * (1 + 2.0 ** -9)
               + (2.0 ** -22 + 2 * dx[..., None] + 2.0 ** -18) * wv + n * 2.0 ** -26 * peak)
        assert torch.isfinite(got[s]).all()
        assert ((got[s] - o[0]).abs() <= tol[0]).all(), (s, float(((got[s] - o[0]).abs() / tol[0]).max()))


def _drop_unseen_blocks(b):
    """-1 in place of every block that ends before the first token that its sequence sees."""
    for s, (lo, hi, _) in enumerate(b.rows):
        seen = lo[lo < hi]
        first = int(seen.min()) if len(seen) else b.lens[s]
        b.table[s, :first // b.bs] = -1


@pytest.mark.gpu
@pytest.mark.parametrize("flagged", [True, False], ids=["checked", "unchecked"])
@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("dt,cd", [("f16", "f16"), ("bf16", "bf16"), ("f32", "f32"), ("f16", "int8"),
                                   ("bf16", "int8"), ("f16", "fp8"), ("bf16", "fp8")])
def test_blocks_before_the_window_may_be_gone(pa, dt, cd, bs, flagged):
    """A window, or a document's start, whose earlier blocks were given back: their entries
    are not looked up, wherever in a tile the first seen token lies."""
    flag = torch.zeros(1, dtype=torch.int32, device="cuda") if flagged else None
    for wide in (False, True):
        for kw in (dict(window=45), dict(starts=[8 * i + 7 * (i % 3) for i in range(12)])):
            lens = [60 + 9 * i for i in range(12)]
            b = Batch(dt, cd, lens, [1] * 12, 8, 2, 128, bs, bs, **kw)
            if wide:
                _wide(b)
            _drop_unseen_blocks(b)
            sc = torch.zeros((12, 2, max(lens)), device="cuda")
            per = _close(_decode(pa, b, scores_out=sc, err_flag=flag), b, str(kw))
            for s, n in enumerate(lens):
                w, dx = per[s]
                assert ((sc[s, :, :n].cpu().double() - w).abs() <= p64.scores_tol(w, w, dx)).all()
    # prefill: few rows (a shared tile), many, and a document that starts inside a block
    for lens, q_lens in (([700], [9]), ([333, 200], [5, 130]), ([500], [150])):
        b = Batch(dt, cd, lens, q_lens, 8, 1 if bs == 8 else 2, 128, bs, 7, window=45, softcap=20.0)
        _drop_unseen_blocks(b)
        _close(_prefill(pa, b, err_flag=flag), b, str(lens))
        b = Batch(dt, cd, lens, q_lens, 8, 2, 128, bs, 8, alibi=True,
                  starts=[n - m - 20 for n, m in zip(lens, q_lens) for _ in range(m)])
        _drop_unseen_blocks(b)
        _close(_prefill(pa, b, err_flag=flag), b, str(lens))
    assert flag is None or int(flag) == 0
    assert pa.get_device_error(clear=True) == 0


NAN = float("nan")
ALL = [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f16", "int8"), ("f16", "fp8"),
       ("bf16", "int8"), ("bf16", "fp8")]


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["plain", "cap", "alibi"])
@pytest.mark.parametrize("dt,cd,D", [(*p, 128) for p in ALL] + [("f16", "f16", 64)])
def test_prefill_nan_wherever_it_stands(pa, dt, cd, D, form):
    """A NaN score makes the rows that see it NaN, the first seen token's as well as a later
    one's, and so does a NaN query; the other rows stay exact."""
    kw = dict(plain={}, cap=dict(softcap=20.0), alibi=dict(alibi=True))[form]
    for lens, q_lens, first in (([150], [150], 40), ([700], [12], 600)):
        n, m = lens[0], q_lens[0]
        half = n - m // 2                                  # the first rows' document ends here
        starts = [first if p < half else half for p in range(n - m, n)]
        for at in (first, first + 3, half - 1):
            b = Batch(dt, cd, lens, q_lens, 8, 1, D, 16, 5, starts=starts, **kw)
            want, tol, _ = b.want()
            blk, off = divmod(b.at(0, at), 16)
            if cd in DT:
                b.kv[0][blk, off] = NAN
            else:
                b.sc[0][blk, :, off] = NAN
            b.q[-2, 3] = NAN
            got = _prefill(pa, b).cpu().double()
            sees = torch.zeros(m, 8, D, dtype=torch.bool)
            for r, p in enumerate(range(n - m, n)):
                sees[r] = starts[r] <= at <= p
            sees[-2, 3] = True
            assert torch.isnan(got[sees]).all(), (lens, at)
            assert ((got - want).abs() <= tol)[~sees].all(), (lens, at)


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True], ids=["one-cta", "persistent"])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("dt,cd", ALL)
def test_decode_nan_wherever_it_stands(pa, dt, cd, softcap, wide):
    """Decode in both forms: a NaN query, a NaN in the only, the first or a later seen token."""
    lens = [1, 90, 300, 200, 200]
    b = Batch(dt, cd, lens, [1] * 5, 8, 2, 128, 16, 9, softcap=softcap, starts=[0, 5, 0, 33, 0])
    if wide:
        _wide(b)
    want, tol, _ = b.want()
    for s, t in ((0, 0), (1, 5), (2, 150)):
        blk, off = divmod(b.at(s, t), 16)
        if cd in DT:
            b.kv[0][blk, off, 1] = NAN
        else:
            b.sc[0][blk, 1, off] = NAN
    b.q[3, 2] = NAN
    sees = torch.zeros(want.shape, dtype=torch.bool)
    sees[:3, 4:] = True                                    # the heads of kv head 1
    sees[3, 2] = True
    got = _decode(pa, b).cpu().double()
    assert torch.isnan(got[sees]).all()
    assert ((got - want).abs() <= tol)[~sees].all()


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True], ids=["one-cta", "persistent"])
@pytest.mark.parametrize("dt,cd", [("f32", "f32"), ("f16", "f16"), ("bf16", "int8")])
def test_running_scores_of_rows_that_are_nan(pa, dt, cd, wide):
    """Tokens that the row does not see keep their scores though its weights are NaN, and
    so do the scores of the other kv head."""
    lens, starts = [200, 90], [77, 40]
    b = Batch(dt, cd, lens, [1, 1], 8, 2, 128, 16, 9, starts=starts)
    if wide:
        _wide(b)
    _, _, per = b.want()
    for s, t in ((0, 77), (1, 80)):
        blk, off = divmod(b.at(s, t), 16)
        if cd in DT:
            b.kv[0][blk, off, 1] = NAN
        else:
            b.sc[0][blk, 1, off] = NAN
    before = torch.rand((2, 2, 210), generator=torch.Generator().manual_seed(1))
    sc = before.cuda()
    _decode(pa, b, scores_in=sc, scores_out=sc)
    sc = sc.cpu()
    for s, n in enumerate(lens):
        lo = starts[s]
        assert torch.equal(sc[s, :, :lo], before[s, :, :lo])
        assert torch.equal(sc[s, :, n:], before[s, :, n:])
        assert torch.isnan(sc[s, 1, lo:n]).all()
        w, dx = per[s]
        total = before[s, 0, :n].double() + w[0]
        assert ((sc[s, 0, :n].double() - total).abs() <= p64.scores_tol(total, w[0], dx[0])).all()


WAIT_LENS = [90, 200, 700, 16, 40, 333, 1, 512]


def _wait_batch(pa, dt, cd, wide):
    b = Batch(dt, cd, WAIT_LENS, [1] * len(WAIT_LENS), 8, 2, 128, 16, 19, softcap=20.0)
    if wide:
        _wide(b)
    g = b.gpu()
    ws = pa.MaskedWorkspace(len(WAIT_LENS), 8, 2, 128, 700)
    ws.buf.fill_(0x7E)                                     # 8e37 wherever a float is read
    before = torch.rand((len(WAIT_LENS), 2, 700), generator=torch.Generator().manual_seed(1))
    return b, g, ws, before


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True], ids=["one-cta", "persistent"])
@pytest.mark.parametrize("dt,cd", [("bf16", "bf16"), ("f16", "int8"), ("bf16", "fp8")])
def test_decode_tiles_that_never_arrive(pa, dt, cd, wide):
    """Zeros, and the running scores as they were, whatever the workspace held."""
    b, g, ws, before = _wait_batch(pa, dt, cd, wide)
    sc = before.cuda()
    try:
        pa.set_fault_injection(1)
        pa.set_wait_limit_ns(1_000_000)
        out = _decode(pa, b, g, scores_in=sc, scores_out=sc, workspace=ws)
        torch.cuda.synchronize()
        assert pa.get_device_error(clear=True) & pa.DEVERR_TIMEOUT
    finally:
        pa.set_fault_injection(0)
        pa.set_wait_limit_ns(0)
    assert not out.any() and torch.equal(sc.cpu(), before)
    _close(_decode(pa, b, g, scores_in=sc, scores_out=sc, workspace=ws), b)


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True], ids=["one-cta", "persistent"])
@pytest.mark.parametrize("dt,cd", [("bf16", "bf16"), ("f16", "int8"), ("bf16", "fp8")])
@pytest.mark.parametrize("mode,limit", [(3, 1_000_000), (0, 1)], ids=["last tiles", "no wait"])
def test_decode_some_tiles_that_never_arrive(pa, dt, cd, wide, mode, limit):
    """Each (sequence, kv head) is right, scores and all, or is zeros with its scores as they
    were."""
    b, g, ws, before = _wait_batch(pa, dt, cd, wide)
    want, tol, per = b.want()
    results = []
    try:
        pa.set_fault_injection(mode)
        pa.set_wait_limit_ns(limit)
        for scored in (True, False):
            ws.buf.fill_(0x7E)
            sc = before.cuda() if scored else None
            out = _decode(pa, b, g, scores_in=sc, scores_out=sc, workspace=ws)
            torch.cuda.synchronize()
            results.append((out.cpu().double(), sc.cpu() if scored else None,
                            bool(pa.get_device_error(clear=True) & pa.DEVERR_TIMEOUT)))
    finally:
        pa.set_fault_injection(0)
        pa.set_wait_limit_ns(0)
    for out, sc, flag in results:
        lost = 0
        for i, n in enumerate(b.lens):
            for k in range(2):
                x = slice(4 * k, 4 * k + 4)
                if not out[i, x].any():
                    lost += 1
                    assert sc is None or torch.equal(sc[i, k], before[i, k])
                    continue
                assert ((out[i, x] - want[i, x]).abs() <= tol[i, x]).all(), (i, k)
                if sc is not None:
                    w, dx = per[i]
                    total = before[i, k, :n].double() + w[k]
                    assert ((sc[i, k, :n].double() - total).abs()
                            <= p64.scores_tol(total, w[k], dx[k])).all(), (i, k)
                    assert torch.equal(sc[i, k, n:], before[i, k, n:])
        assert flag == (lost > 0)
        assert mode == 0 or 0 < lost < 2 * len(b.lens), lost


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True], ids=["one-cta", "persistent"])
@pytest.mark.parametrize("cd", ["int8", "fp8"])
@pytest.mark.parametrize("vs", [1.0, 2.0 ** -6, 2.0 ** -9, 2.0 ** 8])
@pytest.mark.parametrize("slope", [0.0, 0.125])
def test_decode_f16_v_scales_of_any_size(pa, cd, vs, slope, wide):
    """fp16 queries over 8-bit caches: values of a few hundredths or thousandths, or of
    hundreds, to the output's rounding."""
    lens = [300, 40, 900]
    b = Batch("f16", cd, lens, [1] * 3, 8, 2, 64, 16, 43, qmul=0.5)
    b.slopes = slope * torch.linspace(1.0, 1.5, 8)
    b.sc[1] *= vs
    b.val[1] = b.val[1] * vs
    if wide:
        _wide(b)
    got = _decode(pa, b).cpu().double()
    for s, n in enumerate(lens):
        k, v = (x.flatten(0, 1)[[b.at(s, t) for t in range(n)]] for x in b.val)
        lo, hi, pos = b.rows[s]
        o, w, dx, wv = p64.attend(b.q[s:s + 1], k, v, b.scale, lo, hi, pos, 0.0, b.slopes)
        # as above, and half of fp16's step near 0
        peak = (w[0] * v.abs().amax(-1).repeat_interleave(4, dim=1).T).amax(1)[None, :, None]
        tol = (p64.half_step(torch.float16) * o.abs() * (1 + 2.0 ** -9) + 2.0 ** -25
               + (2.0 ** -22 + 2 * dx[..., None] + 2.0 ** -18) * wv + n * 2.0 ** -26 * peak)
        assert ((got[s] - o[0]).abs() <= tol[0]).all(), (s, float(((got[s] - o[0]).abs() / tol[0]).max()))


def _parts_batch(cd, prefill):
    if prefill:
        return Batch("f16", cd, [300, 90, 520], [40, 90, 130], 8, 2, 128, 16, 51, softcap=30.0)
    return Batch("f16", cd, [100, 333, 640, 700], [1] * 4, 32, 4, 128, 16, 52, softcap=30.0)


def _off(out, want):
    return float((out - want).norm() / want.norm())


@pytest.mark.gpu
@pytest.mark.parametrize("form,cd", [(f, c) for f in ("one-cta", "persistent")
                                     for c in ("f16", "int8", "fp8")] + [("prefill", "f16")])
def test_fp16_weights_go_in_as_two_parts(pa, form, cd):
    """The result is off by little more than its own rounding: the weights' two fp16 parts are
    2^-22 (one alone is as far off as the output, see below), 32-bit arithmetic and INT8's
    bias a few 2^-18, against a rounding of about 2^-12 in the mean."""
    b = _parts_batch(cd, form == "prefill")
    if form == "persistent":
        _wide(b)
    want, _, _ = b.want()
    got = (_prefill if form == "prefill" else _decode)(pa, b).cpu().double()
    assert _off(got, want) <= 1.05 * _off(want.half().double(), want) + 5e-6


@pytest.mark.parametrize("prefill", [False, True])
def test_that_bound_tells_one_part_from_two(prefill):
    b = _parts_batch("f16", prefill)
    want, _, _ = b.want()
    one, two, r = [], [], 0
    for s, (n, m) in enumerate(zip(b.lens, b.q_lens)):
        k, v = (x.flatten(0, 1)[[b.at(s, t) for t in range(n)]] for x in b.val)
        lo, hi, pos = b.rows[s]
        _, w, _, _ = p64.attend(b.q[r:r + m], k, v, b.scale, lo, hi, pos, b.softcap)
        p = w / w.amax(-1, keepdim=True)                   # as the kernels hold it
        vv = v.repeat_interleave(b.H // b.Hkv, dim=1)
        h = p.half().double()
        for parts, to in ((h, one), (h + (p - h).half().double(), two)):
            to.append(torch.einsum("rhn,nhd->rhd", parts, vv) / p.sum(-1, keepdim=True))
        r += m
    bound = 1.05 * _off(want.half().double(), want) + 5e-6
    assert _off(torch.cat(two).half().double(), want) <= bound
    # one part: each weight off by up to 2^-12 of its binade, as the output is once more; over
    # many weights that adds 2^-11 / sqrt(12) / 1.4 = 1.0e-4 to the rounding's 2.0e-4, as
    # sqrt(2.0^2 + 1.0^2) = 2.24, which is past 1.05 * 2.0
    assert _off(torch.cat(one).half().double(), want) > bound


@pytest.mark.gpu
@pytest.mark.parametrize("dt,cd", [("f16", "int8"), ("f16", "fp8"), ("f16", "f16"), ("bf16", "int8")])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_long_contexts_to_the_rounding(pa, dt, cd, D):
    """Tens of thousands of tokens, weights spread over all of them: the mean error is the
    output's rounding and little more.  (Two 16-bit parts of the weights 2^-22, for bf16
    under an 8-bit cache too; sums in 32 bits.)"""
    b = Batch(dt, cd, [30000, 9001], [1, 1], 4, 1, D, 16, 61)
    got = _decode(pa, b).cpu().double()
    want, _, _ = b.want()
    for s in range(2):
        rounded = want[s].to(b.dt).double()
        assert _off(got[s], want[s]) <= 1.05 * _off(rounded, want[s]) + 5e-6

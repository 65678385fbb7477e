"""pa_decode_masked and pa_prefill_masked -- paged attention with capped scores, a bias by
distance, documents, windows and prefixes, and running scores of the cached tokens --
against plain 64-bit arithmetic over the tokens that each row sees.  Every slot that no
row sees holds NaN."""
import ctypes

import pytest
import torch

import _plain64 as p64

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
PAIRS = [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f16", "int8"), ("f16", "fp8"),
         ("bf16", "int8"), ("bf16", "fp8")]


class Batch:
    """Sequences of given lengths in a shuffled paged pool, and what each row sees."""

    def __init__(self, dt, cd, lens, q_lens, H, Hkv, D, bs, seed, softcap=0.0, alibi=False,
                 starts=None, prefix=None, window=0, qmul=2.0):
        g = torch.Generator().manual_seed(seed)
        self.dt, self.cd, self.lens, self.q_lens, self.bs = DT[dt], cd, lens, q_lens, bs
        self.H, self.Hkv, self.D, self.softcap, self.window = H, Hkv, D, softcap, window
        self.scale = D ** -0.5
        counts = [-(-n // bs) for n in lens]
        nb = sum(counts) + 3
        shape = (nb, bs, Hkv, D)
        self.sc = None
        if cd in DT:
            self.kv = [torch.randn(shape, generator=g).to(DT[cd]) for _ in range(2)]
            self.val = [x.double() for x in self.kv]
        else:
            self.kv, self.sc, self.val = [], [], []
            for _ in range(2):
                x = torch.randn(shape, generator=g)
                s = x.abs().amax(-1) / (127.0 if cd == "int8" else 448.0)
                y = x / s[..., None]
                c = y.round().to(torch.int8) if cd == "int8" else y.to(torch.float8_e4m3fn)
                self.kv.append(c)
                self.sc.append(s.transpose(1, 2).contiguous())
                self.val.append(c.float().double() * s.double()[..., None])
        perm = torch.randperm(nb, generator=g).to(torch.int32)
        self.table = torch.full((len(lens), max(counts + [1]) + 1), -1, dtype=torch.int32)
        at = 0
        for s, c in enumerate(counts):
            self.table[s, :c] = perm[at:at + c]
            at += c
        rows = sum(q_lens)
        self.q = (qmul * torch.randn((rows, H, D), generator=g)).to(self.dt)
        self.slopes = torch.tensor([2.0 ** (-8 * (h + 1) / H) for h in range(H)]) if alibi else None
        self.starts = None if starts is None else torch.tensor(starts, dtype=torch.int32)
        self.prefix = None if prefix is None else torch.tensor(prefix, dtype=torch.int32)
        self.begin = torch.tensor([0] + list(torch.tensor(q_lens).cumsum(0)), dtype=torch.int32)
        self.rows = []                                    # per sequence: lo, hi, pos
        r = 0
        for s, (n, m) in enumerate(zip(lens, q_lens)):
            pos = torch.arange(n - m, n)
            lo = torch.zeros(m, dtype=torch.long) if starts is None else \
                self.starts[r:r + m].long().clamp(min=0)
            if window:
                lo = torch.maximum(lo, pos - window + 1)
            hi = pos + 1 if prefix is None else (pos + 1).clamp(min=min(max(prefix[s], 0), n))
            self.rows.append((lo, hi.clamp(max=n), pos))
            r += m
        self.poison()

    def at(self, s, t):
        return int(self.table[s, t // self.bs]) * self.bs + t % self.bs

    def poison(self):
        seen = torch.zeros(self.kv[0].shape[0] * self.bs, dtype=torch.bool)
        for s, (lo, hi, _) in enumerate(self.rows):
            for a, b in set(zip(lo.tolist(), hi.tolist())):
                for t in range(a, b):
                    seen[self.at(s, t)] = True
        for x in self.kv:
            f = x.flatten(0, 1)
            if self.cd in DT:
                f[~seen] = float("nan")
            elif self.cd == "int8":
                f[~seen] = 127
            else:
                f.view(torch.uint8)[~seen] = 0x7F          # the NaN code
        if self.sc:
            for x in self.sc:
                x.transpose(1, 2).reshape(-1, self.Hkv)    # scales of unseen slots: NaN too
                y = x.transpose(1, 2).contiguous().flatten(0, 1)
                y[~seen] = float("nan")
                x.copy_(y.view(x.shape[0], self.bs, self.Hkv).transpose(1, 2))

    def want(self):
        """out, tolerance [rows, H, D]; per sequence: weights summed over groups of the last
        row [Hkv, n], its dx."""
        out, tol, per = [], [], []
        r = 0
        for s, (n, m) in enumerate(zip(self.lens, self.q_lens)):
            slots = torch.tensor([self.at(s, t) for t in range(n)], dtype=torch.long)
            k, v = (x.flatten(0, 1)[slots] for x in self.val)
            lo, hi, pos = self.rows[s]
            o, w, dx, wv = p64.attend(self.q[r:r + m], k, v, self.scale, lo, hi, pos, self.softcap,
                                      self.slopes)
            out.append(o)
            vmax = float(v.abs().max()) if n else 0.0
            smax = float(self.sc[1].nan_to_num(0).max()) if self.sc else 0.0
            tol.append(p64.attention_tol(o, dx, wv, self.dt, self.cd, n, vmax, smax))
            if m:
                G = self.H // self.Hkv
                per.append((w[-1].view(self.Hkv, G, n).sum(1),
                            dx[-1].view(self.Hkv, G).amax(1)[:, None]))
            r += m
        return torch.cat(out), torch.cat(tol), per

    def gpu(self):
        c = lambda x: None if x is None else x.cuda()      # noqa: E731
        kv = [x.view(torch.uint8).cuda() if self.cd == "fp8" else x.cuda() for x in self.kv]
        sc = [None, None] if self.sc is None else [x.cuda() for x in self.sc]
        return dict(q=c(self.q), kv=kv, sc=sc, table=c(self.table), begin=c(self.begin),
                    lens=torch.tensor(self.lens, dtype=torch.int32).cuda(), slopes=c(self.slopes),
                    starts=c(self.starts), prefix=c(self.prefix))


def _decode(pa, b, g=None, **kw):
    g = g or b.gpu()
    return pa.decode_masked(g["q"], *g["kv"], g["table"], g["lens"], b.scale, softcap=b.softcap,
                            alibi_slopes=g["slopes"], kv_start=g["starts"], window=b.window,
                            cache_dtype=b.cd, k_scale=g["sc"][0], v_scale=g["sc"][1], **kw)


def _prefill(pa, b, g=None, **kw):
    g = g or b.gpu()
    return pa.prefill_masked(g["q"], *g["kv"], g["table"], g["lens"], g["begin"], b.scale,
                             softcap=b.softcap, alibi_slopes=g["slopes"], kv_start=g["starts"],
                             prefix_lens=g["prefix"], window=b.window, cache_dtype=b.cd,
                             k_scale=g["sc"][0], v_scale=g["sc"][1], **kw)


def _close(out, b, what=""):
    want, tol, per = b.want()
    got = out.detach().cpu().double()
    bad = (got - want).abs() > tol
    assert not bad.any() and torch.isfinite(got).all(), \
        (what, int(bad.sum()), float(((got - want).abs() / tol).max()))
    return per


FORMS = {
    "plain": dict(),
    "cap": dict(softcap=5.0),
    "alibi": dict(alibi=True),
    "window": dict(window=37),
    "all": dict(softcap=30.0, alibi=True, window=150),
}
LENS = [1, 15, 16, 17, 33, 100, 255, 300, 0, 700]


def _wide(b, tokens=1024):
    """A table for more tokens than any sequence has: the persistent form."""
    b.table = torch.nn.functional.pad(b.table, (0, tokens // b.bs), value=-1)


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True], ids=["one-cta", "persistent"])
@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("dt,cd", PAIRS)
def test_decode(pa, dt, cd, form, wide):
    b = Batch(dt, cd, LENS, [1] * len(LENS), 16, 2, 128, 16, 11, **FORMS[form])
    if wide:
        _wide(b)
    b.rows[8] = (torch.zeros(1, dtype=torch.long), torch.zeros(1, dtype=torch.long), torch.tensor([-1]))
    _close(_decode(pa, b), b, form)


@pytest.mark.gpu
@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("wide", [False, True], ids=["one-cta", "persistent"])
@pytest.mark.parametrize("dt,cd", PAIRS)
def test_decode_documents_and_scores(pa, dt, cd, D, bs, wide):
    """Document starts everywhere in a tile and past the end (a row that sees nothing), with
    running scores; scores past each length stay as they are.  A wide table (the most
    tokens a sequence could have) takes the persistent form."""
    lens = [1, 16, 40, 64, 100, 129, 300, 50, 31]
    starts = [0, 15, 17, 16, -4, 127, 250, 50, 90]
    b = Batch(dt, cd, lens, [1] * len(lens), 12, 4, D, bs, D + bs, softcap=20.0, starts=starts)
    if wide:
        _wide(b)
    width = 310
    g = torch.Generator().manual_seed(3)
    before = torch.rand((len(lens), 4, width), generator=g)
    sin, sout = before.cuda(), torch.full_like(before, -5.0).cuda()
    per = _close(_decode(pa, b, scores_in=sin, scores_out=sout), b)
    got = sout.cpu().double()
    for s, n in enumerate(lens):
        w, dx = per[s]
        total = before[s, :, :n].double() + w
        assert ((got[s, :, :n] - total).abs() <= p64.scores_tol(total, w, dx)).all(), s
        assert (got[s, :, n:] == -5.0).all()
    assert torch.equal(sin.cpu(), before)
    # in place, and without a start: the same bits
    out2 = _decode(pa, b, scores_in=sin, scores_out=sin)
    fresh = torch.zeros_like(sout)
    _decode(pa, b, scores_out=fresh)
    for s, n in enumerate(lens):
        assert torch.equal(sin.cpu()[s, :, :n], sout.cpu()[s, :, :n])
        w, dx = per[s]
        assert ((fresh.cpu()[s, :, :n].double() - w).abs() <= p64.scores_tol(w, w, dx)).all()
    assert torch.isfinite(out2).all()


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hkv", [(1, 1), (8, 8), (14, 2), (8, 1), (5, 1)])
def test_decode_head_groups(pa, H, Hkv):
    lens = [3, 90, 400, 17]
    b = Batch("f16", "f16", lens, [1] * 4, H, Hkv, 128, 16, H, alibi=True, window=64)
    sc = torch.zeros((4, Hkv, 401), device="cuda")
    per = _close(_decode(pa, b, scores_out=sc), b)
    for s, n in enumerate(lens):
        w, dx = per[s]
        assert ((sc[s, :, :n].cpu().double() - w).abs() <= p64.scores_tol(w, w, dx)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dt,cd", [("bf16", "bf16"), ("f16", "int8"), ("f32", "f32")])
def test_decode_long_and_window_of_one(pa, dt, cd):
    lens = [5000, 1, 2049]
    b = Batch(dt, cd, lens, [1] * 3, 8, 2, 64, 16, 77, softcap=10.0, alibi=True)
    sc = torch.zeros((3, 2, 5000), device="cuda")
    per = _close(_decode(pa, b, scores_out=sc), b)
    for s, n in enumerate(lens):
        w, dx = per[s]
        assert ((sc[s, :, :n].cpu().double() - w).abs() <= p64.scores_tol(w, w, dx)).all()
    b = Batch(dt, cd, lens, [1] * 3, 8, 2, 64, 16, 78, window=1)
    _close(_decode(pa, b), b)


@pytest.mark.gpu
def test_decode_large_logits_under_the_cap(pa):
    """Scores far past the cap: the tanh is flat there and every score is near +-cap."""
    b = Batch("bf16", "bf16", [70, 200], [1, 1], 8, 2, 128, 16, 5, softcap=8.0, qmul=60.0)
    _close(_decode(pa, b), b)


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True], ids=["one-cta", "persistent"])
@pytest.mark.parametrize("cd", ["int8", "fp8"])
@pytest.mark.parametrize("kv,qm", [(2.0 ** 40, 2.0 ** -60), (2.0 ** -40, 2.0 ** 30), (1.0, 2.0 ** -20)])
def test_decode_bf16_range_over_8_bit_caches(pa, cd, kv, qm, wide):
    """bf16's range, which fp16 lacks, on both sides: huge or tiny K and V scales and
    queries, and a V scale that grows by 2^30 in the middle of a sequence."""
    b = Batch("bf16", cd, [300, 40], [1, 1], 8, 2, 64, 16, 17)
    grow = torch.ones(b.sc[1].shape)
    blk = [int(x) for x in b.table[0] if x >= 0]
    grow[blk[9]:blk[9] + 1] = 2.0 ** 30
    for i in range(2):
        b.sc[i] = b.sc[i] * kv * (grow if i else 1.0)
        b.val[i] = b.val[i] * kv * (grow.transpose(1, 2)[..., None].double() if i else 1.0)
    b.q = (b.q.float() * qm).to(torch.bfloat16)
    b.scale = b.scale / (kv * qm)
    if wide:
        _wide(b)
    want, tol, _ = b.want()
    got = _decode(pa, b).cpu().double()
    # the tolerance's floor for tiny values scales with the values
    tol = tol + 300 * 2.0 ** -25 * want.abs().amax(-1, keepdim=True)
    assert torch.isfinite(got).all() and ((got - want).abs() <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [-0.1, 0.0])
@pytest.mark.parametrize("form", ["plain", "cap", "alibi", "all"])
def test_negative_and_zero_scales(pa, form, scale):
    for dt, cd in (("bf16", "bf16"), ("f16", "int8"), ("f32", "f32")):
        b = Batch(dt, cd, [200, 33], [1, 1], 8, 2, 64, 16, 23, **FORMS[form])
        b.scale = scale
        _close(_decode(pa, b), b, "decode")
    for dt in ("f16", "bf16"):
        b = Batch(dt, dt, [200, 33], [150, 20], 8, 2, 128, 16, 24, **FORMS[form])
        b.scale = scale
        _close(_prefill(pa, b), b, "prefill")


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_prefill_large_logits_and_steep_biases(pa, dt):
    """Scores past the polynomial's range (tanh over its whole range), and a slope so
    steep that the largest product is not the largest score."""
    b = Batch(dt, dt, [300], [200], 8, 2, 128, 16, 5, softcap=8.0, qmul=20.0)
    _close(_prefill(pa, b), b)
    b = Batch(dt, dt, [300], [200], 8, 2, 128, 16, 6, alibi=True, prefix=[250], qmul=4.0)
    b.slopes = torch.tensor([3.0, 1.0, 0.5, 0.0, -0.01, 2.0, 0.25, 1.5])
    _close(_prefill(pa, b), b)


@pytest.mark.gpu
def test_decode_scores_narrower_than_the_sequences(pa):
    lens = [100, 20]
    b = Batch("f16", "f16", lens, [1, 1], 8, 2, 128, 16, 6)
    sc = torch.zeros((2, 2, 64), device="cuda")
    per = _close(_decode(pa, b, scores_out=sc), b)
    for s, n in enumerate((64, 20)):
        w, dx = per[s]
        assert ((sc[s, :, :n].cpu().double() - w[:, :n]).abs() <= p64.scores_tol(w[:, :n], w[:, :n], dx)).all()
        assert not sc[s, :, n:].any()


@pytest.mark.gpu
def test_decode_repeats_streams_and_graphs(pa):
    """One workspace over calls of different batches; a captured and replayed call; a call on
    another stream: the same bits each time."""
    b = Batch("bf16", "bf16", [900, 30, 2000], [1] * 3, 16, 2, 128, 16, 9, softcap=30.0, alibi=True)
    g = b.gpu()
    ws = pa.MaskedWorkspace(3, 16, 2, 128, 2000)
    sc = [torch.zeros((3, 2, 2000), device="cuda") for _ in range(4)]
    a = _decode(pa, b, g, scores_out=sc[0], workspace=ws)
    again = _decode(pa, b, g, scores_out=sc[1], workspace=ws)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    other = _decode(pa, b, g, scores_out=sc[2], stream=st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = _decode(pa, b, g, scores_out=sc[3], workspace=ws)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for o, x in ((again, sc[1]), (other, sc[2]), (cap, sc[3])):
        assert torch.equal(a, o) and torch.equal(sc[0], x)


@pytest.mark.gpu
@pytest.mark.parametrize("dt,cd", [("f16", "f16"), ("f32", "f32"), ("f16", "int8")])
def test_decode_bad_blocks_and_lengths(pa, dt, cd):
    lens = [64, 64, 64]
    b = Batch(dt, cd, lens, [1] * 3, 8, 2, 128, 16, 13)
    g = b.gpu()
    good = _decode(pa, b, g)
    g["table"][0, 1] = 10 ** 6
    g["lens"][1] = 5000
    sc = torch.zeros((3, 2, 64), device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = _decode(pa, b, g, scores_out=sc, err_flag=flag)
    assert int(flag) == pa.DEVERR_BLOCK_ID | pa.DEVERR_SEQ_LEN
    pa.get_device_error(clear=True)
    assert torch.isfinite(out).all() and not out[1].any() and torch.equal(out[2], good[2])
    assert not sc[1].any() and not sc[0, :, 16:32].any()
    assert torch.allclose(sc[0].sum(-1), torch.full((2,), 4.0, device="cuda"), atol=1e-4)


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True], ids=["one-cta", "persistent"])
@pytest.mark.parametrize("dt,cd", [("bf16", "bf16"), ("f16", "int8")])
def test_decode_wait_that_runs_out(pa, dt, cd, wide):
    """A stage that never arrives: the bounded wait ends, the error is reported, and the
    next call is right again (the workspace needs no clearing)."""
    b = Batch(dt, cd, [90, 200], [1, 1], 8, 2, 128, 16, 19)
    if wide:
        _wide(b)
    g = b.gpu()
    ws = pa.MaskedWorkspace(2, 8, 2, 128, 200)
    sc = torch.zeros((2, 2, 200), device="cuda")
    try:
        pa.set_fault_injection(1)
        pa.set_wait_limit_ns(1_000_000)
        _decode(pa, b, g, scores_out=sc, workspace=ws)
        torch.cuda.synchronize()
        assert pa.get_device_error(clear=True) & pa.DEVERR_TIMEOUT
    finally:
        pa.set_fault_injection(0)
        pa.set_wait_limit_ns(0)
    _close(_decode(pa, b, g, scores_out=sc, workspace=ws), b)
    assert pa.get_device_error(clear=True) == 0


@pytest.mark.gpu
def test_empty_batches(pa):
    b = Batch("f16", "f16", [20], [1], 8, 2, 128, 16, 1)
    g = b.gpu()
    none = dict(q=g["q"][:0], kv=g["kv"], sc=g["sc"], table=g["table"][:0], lens=g["lens"][:0],
                begin=g["begin"][:1], slopes=None, starts=None, prefix=None)
    assert _decode(pa, b, none).shape == (0, 8, 128)
    assert _prefill(pa, b, none).shape == (0, 8, 128)
    kept, lens, sc = pa.evict(*g["kv"], g["table"][:0], g["lens"][:0], g["table"][:0],
                              torch.zeros((0, 2, 20), device="cuda"), 8, 2)
    assert kept.shape == (0, 2, 8) and lens.shape == (0,)


@pytest.mark.gpu
def test_workspaces_that_are_too_small_are_refused(pa):
    b = Batch("f16", "f16", [20, 30], [1, 1], 8, 2, 128, 16, 1)
    sc = torch.zeros((2, 2, 30), device="cuda")
    with pytest.raises(pa.PAError) as e:
        _decode(pa, b, scores_out=sc, workspace=pa.MaskedWorkspace(2, 8, 2, 128, 29))
    assert e.value.status == pa.PA_ERR_INVALID_ARG
    with pytest.raises(ValueError, match="contiguous"):
        _decode(pa, b, dict(b.gpu(), q=b.q.cuda().transpose(0, 1).contiguous().transpose(0, 1)))


# ---------------------------------------------------------------------- prefill

PFORMS = dict(FORMS, docs=dict(), prefix=dict(softcap=15.0), mixed=dict(alibi=True, window=90))


def _prefill_batch(dt, cd, form, H, Hkv, D, bs, seed, lens=(5, 140, 300, 257, 64),
                   q_lens=(5, 33, 300, 1, 40), **over):
    g = torch.Generator().manual_seed(seed)
    kw = dict(PFORMS[form], **over)
    if form in ("docs", "mixed"):
        starts = []
        for n, m in zip(lens, q_lens):
            for pos in range(n - m, n):
                starts.append(int(torch.randint(-3, pos + 3, (1,), generator=g)) if pos % 11 == 0
                              else max(0, pos - pos % 53))
        kw["starts"] = starts
    if form in ("prefix", "mixed"):
        kw["prefix"] = [3, 120, 200, 400, 0][:len(lens)]
    return Batch(dt, cd, list(lens), list(q_lens), H, Hkv, D, bs, seed, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("form", sorted(PFORMS))
@pytest.mark.parametrize("dt,cd,D", [("f16", "f16", 128), ("bf16", "bf16", 128), ("f32", "f32", 64),
                                     ("f16", "f16", 64), ("bf16", "int8", 128), ("f16", "fp8", 64)])
def test_prefill(pa, dt, cd, D, form):
    b = _prefill_batch(dt, cd, form, 8, 2, D, 16, 5)
    _close(_prefill(pa, b), b, form)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (6, 2), (8, 1), (16, 1), (12, 4)])
def test_prefill_head_groups_and_blocks(pa, dt, bs, H, Hkv):
    b = _prefill_batch(dt, dt, "mixed", H, Hkv, 128, bs, H + bs, lens=(1, 190, 129), q_lens=(1, 130, 7))
    _close(_prefill(pa, b), b)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("H,Hkv,most", [(64, 1, None), (32, 2, None), (48, 1, 600), (8, 8, 2**31 - 1)])
def test_prefill_many_query_tiles(pa, dt, H, Hkv, most):
    """More query tiles than are kept together in the order of the CTAs, chunks of different
    lengths, a max_query_len far above them."""
    b = _prefill_batch(dt, dt, "mixed", H, Hkv, 128, 16, H, lens=(300, 5, 310), q_lens=(290, 3, 77))
    _close(_prefill(pa, b, max_query_len=most), b)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("form", sorted(PFORMS))
@pytest.mark.parametrize("lens,q_lens", [((1500,), (20,)), ((2300, 100, 900), (40, 100, 1)),
                                         ((513,), (513,)), ((600, 3), (1, 3))])
def test_prefill_few_rows_over_long_contexts(pa, dt, form, lens, q_lens):
    """Few query tiles: several CTAs share one tile's KV tiles and merge; some of them see
    nothing.  Twice the same, captured and replayed too."""
    b = _prefill_batch(dt, dt, form, 8, 1, 128, 16, 21, lens=lens, q_lens=q_lens)
    g = b.gpu()
    out = _prefill(pa, b, g)
    _close(out, b, form)
    again = torch.empty_like(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _prefill(pa, b, g, max_query_len=max(q_lens), out=again)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, out)


@pytest.mark.gpu
def test_prefill_few_rows_and_a_wait_that_runs_out(pa):
    """Every CTA of the cluster gives up: zeros, and the next call is whole."""
    b = _prefill_batch("f16", "f16", "prefix", 8, 1, 128, 16, 22, lens=(1500,), q_lens=(20,))
    g = b.gpu()
    try:
        pa.set_fault_injection(1)
        pa.set_wait_limit_ns(1_000_000)
        out = _prefill(pa, b, g)
        torch.cuda.synchronize()
        assert pa.get_device_error(clear=True) & pa.DEVERR_TIMEOUT
        assert not out.any()
    finally:
        pa.set_fault_injection(0)
        pa.set_wait_limit_ns(0)
    _close(_prefill(pa, b, g), b)
    assert pa.get_device_error(clear=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_prefill_few_rows_and_unseen_infinities(pa, dt):
    """The row repair behind a merge: NaN in V of a token that other rows of the tile see."""
    lens, q_lens = [1200], [16]
    starts = [1184 if i % 2 else 0 for i in range(16)]
    b = Batch(dt, dt, lens, q_lens, 8, 2, 128, 16, 33, starts=starts, softcap=20.0)
    want, tol, _ = b.want()
    b.kv[1].flatten(0, 1)[b.at(0, 700)] = float("nan")
    got = _prefill(pa, b).cpu().double()
    assert ((got - want).abs() <= tol)[1::2].all()
    assert not torch.isfinite(got[::2]).any()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_prefill_rows_that_see_nothing(pa, dt):
    """Documents that start behind their row, a window of one, an empty chunk: zeros."""
    lens, q_lens = [200, 50, 30], [140, 0, 30]
    starts = [n - m + i + (5 if i % 3 == 0 else 0) for n, m in zip(lens, q_lens) for i in range(m)]
    b = Batch(dt, dt, lens, q_lens, 8, 1, 128, 16, 3, starts=starts, softcap=9.0)
    out = _prefill(pa, b)
    _close(out, b)
    assert not out[0].any() and out[1].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_prefill_unseen_infinities_stay_out_of_a_row(pa, dt, bad):
    """A token's V (and another's K) holds NaN or infinity; the rows of other documents see
    neither and stay exact, the rows that see it are not finite."""
    lens, q_lens = [300], [300]
    starts = [0 if p < 100 else (100 if p < 170 else 170) for p in range(300)]
    b = Batch(dt, dt, lens, q_lens, 8, 2, 128, 16, 31, starts=starts, alibi=True)
    want, tol, _ = b.want()
    b.kv[1].flatten(0, 1)[b.at(0, 130), 0, 5] = bad        # V of token 130, kv head 0
    b.kv[0].flatten(0, 1)[b.at(0, 40), 1, 7] = bad         # K of token 40, kv head 1
    got = _prefill(pa, b).cpu().double()
    sees_v = torch.zeros(300, 8, 128, dtype=torch.bool)
    sees_v[130:170, :4, 5] = True
    sees_k = torch.zeros(300, 8, 128, dtype=torch.bool)
    sees_k[40:100, 4:] = True
    clean = ~(sees_v | sees_k)
    assert torch.isfinite(got[clean]).all() and ((got - want).abs() <= tol)[clean].all()
    assert not torch.isfinite(got[sees_v]).any()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_prefill_equals_decode_and_plain_prefill(pa, dt):
    """The last row of a chunk is the decode of that token; without changes to the scores it
    is pa_prefill's attention."""
    b = _prefill_batch(dt, dt, "plain", 8, 2, 128, 16, 8, lens=(700, 90), q_lens=(300, 90))
    g = b.gpu()
    out = _prefill(pa, b, g)
    ref = pa.prefill(g["q"], *g["kv"], g["table"], g["lens"], g["begin"], b.scale)
    _, tol, _ = b.want()
    assert ((out - ref).abs().cpu().double() <= 2 * tol).all()
    last = (g["begin"][1:] - 1).long()
    d = pa.decode_masked(g["q"][last].contiguous(), *g["kv"], g["table"], g["lens"], b.scale)
    assert ((out[last] - d).abs().cpu().double() <= 2 * tol[last.cpu()]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dt,cd,D", [("bf16", "bf16", 128), ("f16", "f16", 64)])
def test_prefill_bad_sequences_are_skipped(pa, dt, cd, D):
    b = Batch(dt, cd, [64, 64, 64, 64], [16] * 4, 8, 2, D, 16, 2)
    g = b.gpu()
    good = _prefill(pa, b, g)
    g["lens"][1] = 9000
    g["lens"][2] = 8                                       # fewer than its query rows
    g["table"][3, 0] = -9
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(good, 3.0)
    _prefill(pa, b, g, out=out, err_flag=flag)
    assert int(flag) == pa.DEVERR_SEQ_LEN | pa.DEVERR_BLOCK_ID
    pa.get_device_error(clear=True)
    assert torch.equal(out[:16], good[:16]) and (out[16:48] == 3.0).all()
    assert torch.isfinite(out).all()


@pytest.mark.gpu
def test_prefill_query_rows_past_the_batch_are_skipped(pa):
    """A query_start that reaches past the query rows: that sequence is skipped."""
    b = Batch("f16", "f16", [64, 64], [16, 16], 8, 2, 128, 16, 2)
    g = b.gpu()
    good = _prefill(pa, b, g)
    g["begin"][2] = 48
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(good, 3.0)
    _prefill(pa, b, g, out=out, err_flag=flag, max_query_len=32)
    assert int(flag) == pa.DEVERR_SEQ_LEN
    pa.get_device_error(clear=True)
    assert torch.equal(out[:16], good[:16]) and (out[16:] == 3.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_prefill_wait_that_runs_out(pa, dt):
    b = Batch(dt, dt, [300, 90], [140, 20], 8, 2, 128, 16, 19, softcap=9.0)
    g = b.gpu()
    try:
        pa.set_fault_injection(1)
        pa.set_wait_limit_ns(1_000_000)
        out = _prefill(pa, b, g)
        torch.cuda.synchronize()
        assert pa.get_device_error(clear=True) & pa.DEVERR_TIMEOUT
        assert not out.any()                               # abandoned tiles write zeros
    finally:
        pa.set_fault_injection(0)
        pa.set_wait_limit_ns(0)
    _close(_prefill(pa, b, g), b)
    assert pa.get_device_error(clear=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_prefill_side_stream_and_graph(pa, dt):
    b = _prefill_batch(dt, dt, "mixed", 8, 2, 128, 16, 4)
    g = b.gpu()
    a = _prefill(pa, b, g, max_query_len=300)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    o = _prefill(pa, b, g, max_query_len=300, stream=st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = _prefill(pa, b, g, max_query_len=300)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, o) and torch.equal(a, c)


# ---------------------------------------------------------------------- the set together

@pytest.mark.gpu
@pytest.mark.parametrize("cd", ["bf16", "fp8"])
def test_a_serving_run(pa, cd):
    """What a user does with the set: turn and cache a prompt, decode with running scores,
    evict through the block manager, and decode on over what stayed -- each attention
    checked against 64 bits over the rows that the cache holds."""
    from paged_kv_cache_390_b200.block_manager import BlockManager
    H, Hkv, D, bs, keep, recent, n0 = 8, 2, 128, 16, 48, 16, [90, 61]
    g = torch.Generator().manual_seed(2)
    with BlockManager(64, bs) as bm:
        pool = torch.full((64, bs, Hkv, D), 0x7F, dtype=torch.uint8, device="cuda")
        kc = pool.clone() if cd == "fp8" else torch.full(pool.shape, float("nan"),
                                                         dtype=torch.bfloat16, device="cuda")
        vc = kc.clone()
        ks = torch.full((64, Hkv, bs), float("nan"), device="cuda") if cd == "fp8" else None
        vs = None if ks is None else ks.clone()
        kw = dict(cache_dtype=cd, k_scale=ks, v_scale=vs)
        inv, axis = pa.rope_inv_freq(D, 1e6), pa.rope_pair_axis((16, 24, 24))
        mk = lambda n, h: torch.randn((n, h, D), generator=g).to(torch.bfloat16).cuda()  # noqa: E731
        slots = torch.cat([torch.from_numpy(bm.add_sequence(i, range(n))[0]) for i, n in enumerate(n0)])
        pos = torch.cat([torch.arange(n) for n in n0]).repeat(3, 1).cuda()
        pa.rope_and_cache(mk(sum(n0), H), mk(sum(n0), Hkv), mk(sum(n0), Hkv), pos, inv, axis, kc, vc,
                          slots.cuda(), **kw)
        scores = torch.zeros((2, Hkv, 128), device="cuda")
        true_pos = list(n0)

        def values(table, s, n):
            out = []
            for c, sc in ((kc, ks), (vc, vs)):
                x = (c.view(torch.float8_e4m3fn) if cd == "fp8" else c).float().double().cpu()
                if sc is not None:
                    x = x * sc.double().cpu().transpose(1, 2)[..., None]
                ids = torch.tensor([int(table[s, t // bs]) * bs + t % bs for t in range(n)])
                out.append(x.flatten(0, 1)[ids])
            return out

        def step(scores):
            sl, cow = bm.append_batch([0, 1], [7, 8])
            assert len(cow) == 0
            p = torch.tensor(true_pos).repeat(3, 1).cuda()
            q = pa.rope_and_cache(mk(2, H), mk(2, Hkv), mk(2, Hkv), p, inv, axis, kc, vc,
                                  torch.from_numpy(sl).cuda(), **kw)
            for i in range(2):
                true_pos[i] += 1
            tab, lens = bm.build_batch([0, 1])
            before = scores.clone()
            out = pa.decode_masked(q, kc, vc, torch.from_numpy(tab).cuda(),
                                   torch.from_numpy(lens).cuda(), D ** -0.5, softcap=20.0,
                                   scores_in=scores, scores_out=scores, **kw)
            for s, n in enumerate(lens.tolist()):
                k, v = values(tab, s, n)
                o, w, dx, wv = p64.attend(q[s:s + 1].cpu(), k, v, D ** -0.5, [0], [n], [n - 1], 20.0)
                tol = p64.attention_tol(o, dx, wv, torch.bfloat16, cd, n, float(v.abs().max()))
                assert ((out[s:s + 1].cpu().double() - o).abs() <= tol).all()
                ws = w[0].view(Hkv, H // Hkv, n).sum(1)
                total = before[s, :, :n].cpu().double() + ws
                assert ((scores[s, :, :n].cpu().double() - total).abs()
                        <= p64.scores_tol(total, ws, dx[0].view(Hkv, -1).amax(1)[:, None])).all()
            return tab, lens

        for _ in range(3):
            tab, lens = step(scores)
        old_k = [values(tab, s, int(n)) for s, n in enumerate(lens)]
        new_tab = bm.evict([0, 1], keep)
        kept, new_lens, ns = pa.evict(kc, vc, torch.from_numpy(tab).cuda(),
                                      torch.from_numpy(lens).cuda(), torch.from_numpy(new_tab).cuda(),
                                      scores, keep, recent, new_scores=torch.zeros_like(scores), **kw)
        want = p64.evict(scores.cpu(), lens.tolist(), keep, recent)
        assert new_lens.tolist() == [keep, keep]
        for s in range(2):
            k, v = values(new_tab, s, keep)
            for h in range(Hkv):
                assert kept[s, h].tolist() == want[s][h]
                assert torch.equal(k[:, h], old_k[s][0][want[s][h], h])
                assert torch.equal(v[:, h], old_k[s][1][want[s][h], h])
        for _ in range(2):
            _, lens = step(ns)
        assert lens.tolist() == [keep + 2, keep + 2]


# ---------------------------------------------------------------------- refusals (CPU)

@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_390_b200 import build, pa
    build.build()
    return pa.lib()


def _cdecode(lib, **over):
    fake, f2 = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 21)
    d = dict(out=fake, q=fake, qd=1, k=fake, v=fake, cd=1, ks=None, vs=None, bt=fake, mb=4, sl=fake,
             S=2, H=8, Hkv=2, D=128, bs=16, nb=10, scale=0.1, cap=0.0, sp=None, st=None, win=0,
             si=None, so=None, ss=0, ws=f2, wsb=1 << 40)
    d.update(over)
    return lib.pa_decode_masked(*[d[k] for k in ("out", "q", "qd", "k", "v", "cd", "ks", "vs", "bt",
                                                 "mb", "sl", "S", "H", "Hkv", "D", "bs", "nb",
                                                 "scale", "cap", "sp", "st", "win", "si", "so", "ss",
                                                 "ws", "wsb")], None, None)


@pytest.mark.parametrize("over,status", [
    (dict(S=0), 0), (dict(S=0, cap=-1.0), 1), (dict(S=0, window=0, win=-1), 1),
    (dict(S=0, cap=float("inf")), 1), (dict(S=0, cap=float("nan")), 1), (dict(S=0, cap=1e-9), 1),
    (dict(S=0, cap=1e30), 1), (dict(S=0, cap=1e30, scale=0.0), 0),
    (dict(q=None), 1), (dict(D=96), 2), (dict(H=18, Hkv=2), 2), (dict(cd=3), 1), (dict(ws=None), 1),
    (dict(ws=ctypes.c_void_p((1 << 20) + 16)), 1), (dict(wsb=100), 1),
    (dict(si=ctypes.c_void_p(1 << 20)), 1), (dict(so=ctypes.c_void_p(1 << 20)), 1),
    (dict(so=ctypes.c_void_p((1 << 20) + 2), ss=8), 1), (dict(sp=ctypes.c_void_p((1 << 20) + 2)), 1),
    (dict(so=ctypes.c_void_p(1 << 20), ss=64, wsb=200000), 1), (dict(S=9000), 2)])
def test_decode_host_checks(lib, over, status):
    over.pop("window", None)
    assert _cdecode(lib, **over) == status


def _cprefill(lib, **over):
    fake = ctypes.c_void_p(1 << 20)
    d = dict(out=fake, q=fake, qd=1, qs=fake, tq=8, mq=4, k=fake, v=fake, cd=1, ks=None, vs=None,
             bt=fake, mb=4, sl=fake, S=2, H=8, Hkv=2, D=128, bs=16, nb=10, scale=0.1, cap=0.0,
             sp=None, st=None, pl=None, win=0)
    d.update(over)
    return lib.pa_prefill_masked(*[d[k] for k in ("out", "q", "qd", "qs", "tq", "mq", "k", "v", "cd",
                                                  "ks", "vs", "bt", "mb", "sl", "S", "H", "Hkv", "D",
                                                  "bs", "nb", "scale", "cap", "sp", "st", "pl",
                                                  "win")], None, None)


@pytest.mark.parametrize("over,status", [
    (dict(S=0), 0), (dict(tq=0), 0), (dict(mq=0), 0), (dict(out=None), 1), (dict(qs=None), 1),
    (dict(cap=-2.0), 1), (dict(win=-3), 1), (dict(H=7), 1), (dict(H=260, Hkv=2), 2), (dict(D=32), 2),
    (dict(qd=1, cd=2), 2), (dict(cd=4), 1), (dict(Hkv=0), 1), (dict(tq=-1), 1),
    (dict(pl=ctypes.c_void_p((1 << 20) + 1)), 1), (dict(scale=float("nan")), 1)])
def test_prefill_host_checks(lib, over, status):
    assert _cprefill(lib, **over) == status


def test_workspace_sizes(lib):
    base = lib.pa_decode_masked_workspace_bytes(4, 16, 2, 128, 0)
    assert base >= lib.pa_decode_fused_workspace_bytes(4, 2, 128, 148) + 4 * 16 * 4
    assert lib.pa_decode_masked_workspace_bytes(4, 16, 2, 128, 1000) == base + 4 * 16 * 1000 * 4
    assert lib.pa_decode_masked_workspace_bytes(0, 16, 2, 128, 0) == 0
    assert lib.pa_decode_masked_workspace_bytes(4, 16, 2, 128, -1) == 0


def test_binding_refusals(lib):
    from paged_kv_cache_390_b200 import pa
    q, kc = torch.zeros(2, 8, 64), torch.zeros(4, 16, 2, 64)
    tab, lens = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)       # noqa: E731
    sc = torch.zeros(2, 2, 10)
    for kw in (dict(alibi_slopes=torch.zeros(7)), dict(alibi_slopes=torch.zeros(8).double()),
               dict(kv_start=i32(3)), dict(kv_start=lens.long()), dict(scores_in=sc),
               dict(scores_out=sc[:, :1]), dict(scores_out=sc, scores_in=sc[..., :5]),
               dict(out=torch.zeros(2, 8, 32)), dict()):
        with pytest.raises(ValueError):
            pa.decode_masked(q, kc, kc, tab, lens, 0.1, **kw)
    begin = i32(3)
    for kw in (dict(kv_start=i32(3)), dict(prefix_lens=i32(1)), dict(out=q.half()), dict()):
        with pytest.raises(ValueError):
            pa.prefill_masked(q, kc, kc, tab, lens, begin, 0.1, max_query_len=1, **kw)
    with pytest.raises(ValueError):
        pa.prefill_masked(q, kc, kc, tab, lens, i32(2), 0.1, max_query_len=1)

"""pa_rope_and_cache -- rotary positions with several axes and the cache write -- against
plain 64-bit arithmetic, and against pa_reshape_and_cache for the rows it writes."""
import ctypes

import pytest
import torch

import _plain64 as p64

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _inputs(dt, T, H, Hkv, D, bs, axes, far, seed, fused=False):
    g = torch.Generator().manual_seed(seed)
    rows = torch.randn((T, H + 2 * Hkv, D), generator=g).to(DT[dt])
    q, k, v = rows[:, :H], rows[:, H:H + Hkv], rows[:, H + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pos = torch.randint(0, far, (axes, T), generator=g)
    nb = -(-max(T, 1) // bs) + 2
    slots = torch.randperm(nb * bs, generator=g)[:T]
    return rows, q, k, v, pos, slots, nb


def _on_gpu(rows, H, Hkv, fused):
    r = rows.cuda()
    q, k, v = r[:, :H], r[:, H:H + Hkv], r[:, H + Hkv:]
    return (q, k, v) if fused else (q.contiguous(), k.contiguous(), v.contiguous())


def _pool(cd, nb, bs, Hkv, D):
    if cd in DT:
        kc = torch.full((nb, bs, Hkv, D), float("nan"), dtype=DT[cd], device="cuda")
        return kc, kc.clone(), None, None
    kc = torch.full((nb, bs, Hkv, D), 127, dtype=torch.int8 if cd == "int8" else torch.uint8,
                    device="cuda")
    sc = torch.full((nb, Hkv, bs), float("nan"), device="cuda")
    return kc, kc.clone(), sc, sc.clone()


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,rot,sections,spread", [
    (128, 128, (16, 24, 24), False), (128, 128, (24, 20, 20), True), (128, 96, (48,), False),
    (64, 64, (16, 16), False), (64, 16, (8,), False), (128, 32, (5, 11), True)])
def test_rows_match_64_bits(pa, dt, D, rot, sections, spread, interleaved):
    T, H, Hkv, bs = 37, 6, 2, 16
    rows, q, k, v, pos, slots, nb = _inputs(dt, T, H, Hkv, D, bs, len(sections), 1 << 20, D + rot,
                                            fused=True)
    slots[5] = -1
    inv = pa.rope_inv_freq(rot, 1e6)
    axis = pa.rope_pair_axis(sections, spread)
    gq, gk, gv = _on_gpu(rows, H, Hkv, True)
    kc, vc, _, _ = _pool(dt, nb, bs, Hkv, D)
    out = pa.rope_and_cache(gq, gk, gv, pos.cuda(), inv, axis, kc, vc, slots.cuda(),
                            interleaved=interleaved)
    want_q = p64.rope(q, pos, inv.cpu(), axis.cpu(), interleaved)
    want_k = p64.rope(k, pos, inv.cpu(), axis.cpu(), interleaved)
    assert ((out.cpu().double() - want_q).abs() <= p64.rope_tol(want_q, DT[dt])).all()
    ok = slots >= 0
    got_k = kc.flatten(0, 1).cpu()[slots[ok]]
    assert ((got_k.double() - want_k[ok]).abs() <= p64.rope_tol(want_k[ok], DT[dt])).all()
    assert torch.equal(vc.flatten(0, 1).cpu()[slots[ok]], v[ok])
    rest = torch.ones(nb * bs, dtype=torch.bool)
    rest[slots[ok]] = False                              # every other slot as it was
    assert kc.flatten(0, 1).cpu()[rest].isnan().all() and vc.flatten(0, 1).cpu()[rest].isnan().all()


@pytest.mark.gpu
@pytest.mark.parametrize("cd", ["int8", "fp8"])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_quantised_rows_are_the_cache_writes(pa, dt, cd, D):
    """Turned keys in fp32 (positions of 0 turn nothing, so the rows are exact) quantise to
    the bits that pa_reshape_and_cache writes; turned ones to within a code's half step."""
    T, H, Hkv, bs = 50, 4, 3, 8
    rows, q, k, v, pos, slots, nb = _inputs(dt, T, H, Hkv, D, bs, 1, 5000, 3)
    gq, gk, gv = _on_gpu(rows, H, Hkv, False)
    inv, axis = pa.rope_inv_freq(D), pa.rope_pair_axis((D // 2,))
    a, b = _pool(cd, nb, bs, Hkv, D), _pool(cd, nb, bs, Hkv, D)
    gs = slots.cuda()
    pa.reshape_and_cache(gk, gv, a[0], a[1], gs, cache_dtype=cd, k_scale=a[2], v_scale=a[3])
    out = pa.rope_and_cache(gq, gk, gv, torch.zeros(T, dtype=torch.int64, device="cuda"), inv, axis,
                            b[0], b[1], gs, cache_dtype=cd, k_scale=b[2], v_scale=b[3])
    assert torch.equal(out, gq)
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.uint8) if x.dtype != torch.float32 else x.view(torch.int32),
                           y.view(torch.uint8) if y.dtype != torch.float32 else y.view(torch.int32))
    pa.rope_and_cache(gq, gk, gv, pos.cuda(), inv, axis, b[0], b[1], gs, cache_dtype=cd,
                      k_scale=b[2], v_scale=b[3])
    want = p64.rope(k, pos, inv.cpu(), axis.cpu(), False)
    blk, off = slots // bs, slots % bs
    sc = b[2].cpu().double()[blk, :, off]                # [T, Hkv]
    top = 127.0 if cd == "int8" else 448.0
    amax = want.abs().amax(-1)
    assert ((sc * top - amax).abs() <= amax * 16 * 2.0 ** -24).all()
    codes = b[0].flatten(0, 1)[gs]
    codes = (codes if cd == "int8" else codes.view(torch.float8_e4m3fn)).to(torch.float32).cpu().double()
    got = codes * sc[..., None]
    # half a code step (INT8: s / 2; E4M3: 2^-4 of the value, at least half a subnormal
    # step 2^-10 s), plus the 32-bit arithmetic of the row
    step = sc[..., None] / 2 if cd == "int8" else \
        torch.maximum(want.abs() * 2.0 ** -4, sc[..., None] * 2.0 ** -10)
    assert ((got - want).abs() <= step * (1 + 2.0 ** -12) + amax[..., None] * 16 * 2.0 ** -24).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 2, 333])
def test_in_place_and_token_counts(pa, T):
    rows, q, k, v, pos, slots, nb = _inputs("bf16", T, 8, 2, 128, 16, 3, 4096, T)
    gq, gk, gv = _on_gpu(rows, 8, 2, False)
    inv, axis = pa.rope_inv_freq(128), pa.rope_pair_axis((16, 24, 24))
    kc, vc, _, _ = _pool("bf16", nb, 16, 2, 128)
    a = pa.rope_and_cache(gq, gk, gv, pos.cuda(), inv, axis, kc, vc, slots.cuda())
    b = gq.clone()
    pa.rope_and_cache(b, gk, gv, pos.cuda(), inv, axis, kc, vc, slots.cuda(), out=b)
    assert torch.equal(a, b)
    want = p64.rope(q, pos, inv.cpu(), axis.cpu(), False)
    assert ((a.cpu().double() - want).abs() <= p64.rope_tol(want, torch.bfloat16)).all()


@pytest.mark.gpu
def test_far_and_negative_positions(pa):
    T = 16
    rows, q, k, v, _, slots, nb = _inputs("f32", T, 2, 2, 64, 16, 1, 10, 9)
    pos = torch.tensor([0, 1, -1, -5000, 2 ** 20 + 1, 2 ** 24 + 3, 2 ** 31 - 1, -2 ** 31] * 2)[None]
    gq, gk, gv = _on_gpu(rows, 2, 2, False)
    inv, axis = pa.rope_inv_freq(64), pa.rope_pair_axis((32,))
    kc, vc, _, _ = _pool("f32", nb, 16, 2, 64)
    out = pa.rope_and_cache(gq, gk, gv, pos.cuda(), inv, axis, kc, vc, slots.cuda())
    want = p64.rope(q, pos, inv.cpu(), axis.cpu(), False)
    # the angle's own 64-bit rounding at |position| 2^31: 3 * 2^-53 * 2^31 more
    tol = p64.rope_tol(want, torch.float32) + want.abs().amax() * 3 * 2.0 ** -22
    assert ((out.cpu().double() - want).abs() <= tol).all()


@pytest.mark.gpu
def test_slots_past_the_pool_and_foreign_axes(pa):
    T = 5
    rows, q, k, v, pos, slots, nb = _inputs("f16", T, 2, 1, 64, 16, 2, 100, 4)
    gq, gk, gv = _on_gpu(rows, 2, 1, False)
    slots[1], slots[3] = nb * 16, -7
    axis = torch.tensor([0, 1, 2, -1] * 8, dtype=torch.int32, device="cuda")
    inv = pa.rope_inv_freq(64)
    kc, vc, _, _ = _pool("f16", nb, 16, 1, 64)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pa.rope_and_cache(gq, gk, gv, pos.cuda(), inv, axis, kc, vc, slots.cuda(), err_flag=flag)
    assert int(flag) == pa.DEVERR_SLOT
    pa.get_device_error(clear=True)
    want = p64.rope(q, pos, inv.cpu(), axis.cpu(), False)
    assert ((out.cpu().double() - want).abs() <= p64.rope_tol(want, torch.float16)).all()
    written = (~kc.flatten(0, 1).isnan()).all(-1).all(-1).sum()
    assert int(written) == 3


@pytest.mark.gpu
def test_side_stream_and_graph(pa):
    T = 20
    rows, q, k, v, pos, slots, nb = _inputs("f16", T, 4, 2, 128, 16, 1, 9999, 12)
    gq, gk, gv = _on_gpu(rows, 4, 2, False)
    inv, axis = pa.rope_inv_freq(128), pa.rope_pair_axis((64,))
    args = (gq, gk, gv, pos.cuda(), inv, axis)
    pools = [_pool("f16", nb, 16, 2, 128) for _ in range(3)]
    gs = slots.cuda()
    a = pa.rope_and_cache(*args, pools[0][0], pools[0][1], gs)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    b = pa.rope_and_cache(*args, pools[1][0], pools[1][1], gs, stream=st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c = pa.rope_and_cache(*args, pools[2][0], pools[2][1], gs)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)
    for p in pools[1:]:
        assert torch.equal(p[0].view(torch.int16), pools[0][0].view(torch.int16))


# ---------------------------------------------------------------------- refusals (CPU)

@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_390_b200 import build, pa
    build.build()
    return pa.lib()


def _call(lib, **over):
    fake = ctypes.c_void_p(1 << 20)
    d = dict(out=fake, q=fake, k=fake, v=fake, dt=1, qs=512, ks=256, vs=256, pos=fake, axes=3,
             inv=fake, ax=fake, rot=128, il=0, kc=fake, vc=fake, cd=1, ksc=None, vsc=None,
             slots=fake, T=4, H=4, Hkv=2, D=128, bs=16, nb=10)
    d.update(over)
    return lib.pa_rope_and_cache(d["out"], d["q"], d["k"], d["v"], d["dt"], d["qs"], d["ks"],
                                 d["vs"], d["pos"], d["axes"], d["inv"], d["ax"], d["rot"], d["il"],
                                 d["kc"], d["vc"], d["cd"], d["ksc"], d["vsc"], d["slots"], d["T"],
                                 d["H"], d["Hkv"], d["D"], d["bs"], d["nb"], None, None)


@pytest.mark.parametrize("over,status", [
    (dict(T=0), 0), (dict(T=0, q=None), 0), (dict(T=-1), 1), (dict(q=None), 1), (dict(pos=None), 1),
    (dict(slots=None), 1), (dict(axes=0), 1), (dict(rot=24), 1), (dict(rot=0), 1),
    (dict(rot=144), 1), (dict(D=96), 2), (dict(bs=12), 1), (dict(cd=2), 2), (dict(cd=3), 1),
    (dict(qs=511), 1), (dict(qs=504), 1), (dict(ks=128), 1), (dict(vs=260), 1), (dict(il=2), 1),
    (dict(q=ctypes.c_void_p((1 << 20) + 2)), 1), (dict(kc=ctypes.c_void_p((1 << 20) + 8)), 1),
    (dict(dt=3), 1), (dict(H=0), 1), (dict(nb=0), 1)])
def test_host_checks(lib, over, status):
    assert _call(lib, **over) == status


def test_binding_refuses_cpu_tensors_and_wrong_shapes(lib):
    from paged_kv_cache_390_b200 import pa
    q, k = torch.zeros(3, 4, 128), torch.zeros(3, 2, 128)
    kc = torch.zeros(4, 16, 2, 128)
    pos, slots = torch.zeros(1, 3, dtype=torch.int64), torch.zeros(3, dtype=torch.int64)
    inv, axis = pa.rope_inv_freq(128, device="cpu"), pa.rope_pair_axis((64,), device="cpu")
    ok = (q, k, k, pos, inv, axis, kc, kc, slots)
    with pytest.raises(ValueError, match="CUDA"):
        pa.rope_and_cache(*ok)
    for i, bad in ((1, k[:2]), (3, pos.int()), (3, pos[:, :2]), (4, inv.float()), (5, axis.long()),
                   (8, slots.int()), (7, kc.half()), (2, k.half())):
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError):
            pa.rope_and_cache(*args)


def test_pair_axis_layouts(lib):
    from paged_kv_cache_390_b200 import pa
    assert pa.rope_pair_axis((2, 1, 3), device="cpu").tolist() == [0, 0, 1, 2, 2, 2]
    assert pa.rope_pair_axis((2, 1, 3), spread=True, device="cpu").tolist() == [0, 1, 2, 0, 2, 2]
    f = pa.rope_inv_freq(8, 100.0, device="cpu")
    assert f.dtype == torch.float64 and torch.allclose(f, torch.tensor([1, 100 ** -0.25, 0.1, 100 ** -0.75], dtype=torch.float64), rtol=1e-15)

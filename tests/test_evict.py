"""pa_evict and pa_bm_evict -- cutting cached sequences by accumulated attention weight --
against the definition: whole numbers and copied bits, so every comparison is exact."""
import ctypes

import numpy as np
import pytest
import torch

import _plain64 as p64

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _case(lens, Hkv, D, bs, cd, keep, seed, width=None):
    g = torch.Generator().manual_seed(seed)
    counts = [-(-n // bs) for n in lens]
    spare = [-(-min(n, keep) // bs) for n in lens]
    nb = sum(counts) + sum(spare) + 2
    shape = (nb, bs, Hkv, D)
    if cd in DT:
        kc, vc = (torch.randn(shape, generator=g).to(DT[cd]) for _ in range(2))
        ks = vs = None
    else:
        kc, vc = (torch.randint(0, 256, shape, generator=g, dtype=torch.uint8) for _ in range(2))
        if cd == "int8":
            kc, vc = kc.view(torch.int8), vc.view(torch.int8)
        ks, vs = (torch.rand((nb, Hkv, bs), generator=g) for _ in range(2))
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    tab = torch.full((len(lens), max(counts + [1])), -1, dtype=torch.int32)
    new = torch.full((len(lens), max(spare + [1])), -1, dtype=torch.int32)
    at = 0
    for t, cs in ((tab, counts), (new, spare)):
        for s, c in enumerate(cs):
            t[s, :c] = perm[at:at + c]
            at += c
    L = width or max(max(lens), 1)
    scores = torch.exp(torch.randn((len(lens), Hkv, L), generator=g))
    return kc, vc, ks, vs, tab, new, scores


def _run(pa, case, lens, keep, recent, cd, **kw):
    kc, vc, ks, vs, tab, new, scores = (x.cuda() if x is not None else None for x in case)
    gl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    res = pa.evict(kc, vc, tab, gl, new, scores, keep, recent, cache_dtype=cd, k_scale=ks,
                   v_scale=vs, **kw)
    torch.cuda.synchronize()
    return (kc, vc, ks, vs), res


def _check(case, lens, keep, recent, pools, res, bs):
    kc, vc, ks, vs, tab, new, scores = case
    want = p64.evict(scores, lens, keep, recent)
    kept, new_lens, new_scores = (x.cpu() for x in res)
    Hkv = kc.shape[2]
    assert new_lens.tolist() == [min(n, keep) for n in lens]
    wk, wv = kc.clone(), vc.clone()
    wks, wvs = (None, None) if ks is None else (ks.clone(), vs.clone())
    for s, n in enumerate(lens):
        m = min(n, keep)
        for h in range(Hkv):
            idx = want[s][h]
            assert kept[s, h, :m].tolist() == idx, (s, h)
            assert (kept[s, h, m:] == -1).all()
            a, b = new_scores[s, h, :m], scores[s, h, idx]
            assert torch.equal(a.view(torch.int32), b.view(torch.int32))
            j = torch.arange(m)
            t = torch.tensor(idx, dtype=torch.long)
            db, sb = new[s].long()[j // bs], tab[s].long()[t // bs]
            wk[db, j % bs, h], wv[db, j % bs, h] = kc[sb, t % bs, h], vc[sb, t % bs, h]
            if ks is not None:
                wks[db, h, j % bs], wvs[db, h, j % bs] = ks[sb, h, t % bs], vs[sb, h, t % bs]
    for got, w in zip(pools, (wk, wv, wks, wvs)):
        if w is not None:                       # moved rows, and every other slot as it was
            assert torch.equal(got.cpu().contiguous().view(torch.uint8), w.view(torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("cd", ["f32", "f16", "bf16", "int8", "fp8"])
@pytest.mark.parametrize("D,bs,Hkv", [(128, 16, 2), (64, 8, 3), (64, 32, 1)])
def test_matches_the_definition(pa, cd, D, bs, Hkv):
    lens, keep, recent = [1, 40, 41, 300, 0, 17, 39], 40, 8
    case = _case(lens, Hkv, D, bs, cd, keep, D + bs)
    pools, res = _run(pa, case, lens, keep, recent, cd)
    _check(case, lens, keep, recent, pools, res, bs)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,keep,recent", [
    ([5000, 1, 1025, 2048], 700, 0), ([3000, 4097], 1, 0), ([3000, 4097], 1, 1),
    ([2500, 1024, 1023], 1024, 1024), ([9000], 8999, 13), ([1500] * 3, 5000, 100),
    ([33000], 20000, 1)])
def test_sizes(pa, lens, keep, recent):
    case = _case(lens, 2, 64, 16, "bf16", keep, sum(lens))
    pools, res = _run(pa, case, lens, keep, recent, "bf16")
    _check(case, lens, keep, recent, pools, res, 16)


@pytest.mark.gpu
def test_ties_zeros_infinities_and_nan(pa):
    lens, keep, recent = [600, 600, 600, 600], 200, 20
    case = _case(lens, 2, 64, 16, "f16", keep, 5)
    sc = case[6]
    sc[0] = 1.0                                    # all equal: the first ones
    sc[1] = torch.randint(0, 4, sc[1].shape).float()
    sc[1][sc[1] == 0] = -0.0                       # -0 ties with 0
    sc[1, :, ::7] = 0.0
    sc[2, :, ::3] = float("inf")
    sc[2, :, 1::3] = float("-inf")
    sc[3, :, ::2] = float("nan")                   # more NaN than places: the first numbers, then NaN
    sc[3, :, 1::4] = float("-inf")
    pools, res = _run(pa, case, lens, keep, recent, "f16")
    _check(case, lens, keep, recent, pools, res, 16)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [600, 9000])
@pytest.mark.parametrize("digit", [0, 1, 2, 3])
@pytest.mark.parametrize("more", [-1, 0, 1])
def test_a_digit_that_decides_alone(pa, n, digit, more):
    """keep - recent + more tokens share the score's first digits (8 bits each) up to
    `digit` and differ behind it; the others are lower in that digit."""
    keep, recent, Hkv = 200, 20, 2
    case = _case([n], Hkv, 64, 16, "f16", keep, 31)
    g = torch.Generator().manual_seed(1000 * digit + more)
    top = 0x4B4B4B4B
    shift = 24 - 8 * digit
    low = torch.randint(0, 1 << shift, (Hkv, n), generator=g) if shift else torch.zeros(Hkv, n, dtype=torch.long)
    high = torch.full((Hkv, n), (top >> shift) - 1)
    for h in range(Hkv):
        high[h, torch.randperm(n - recent, generator=g)[:keep - recent + more]] += 1
    case[6][0, :, :n] = ((high << shift) + low).to(torch.int32).view(torch.float32)
    pools, res = _run(pa, case, [n], keep, recent, "f16")
    _check(case, [n], keep, recent, pools, res, 16)


@pytest.mark.gpu
def test_wide_outputs_keep_their_tails_and_repeat(pa):
    """Outputs wider than needed: kept is filled with -1, new_scores past the new length
    stays; two runs on one input give the same bits; captured and replayed alike."""
    lens, keep, recent = [100, 37], 30, 4
    case = _case(lens, 2, 128, 16, "bf16", keep, 8, width=150)
    ns = torch.full((2, 2, 64), 7.0, device="cuda")
    kept = torch.full((2, 2, 50), 99, dtype=torch.int32, device="cuda")
    pools, res = _run(pa, case, lens, keep, recent, "bf16", new_scores=ns, kept=kept)
    _check(case, lens, keep, recent, pools, (kept, res[1], ns), 16)
    assert (ns[:, :, 30:] == 7.0).all()
    dev = [x.cuda() if x is not None else None for x in case]
    gl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    k2, l2, s2 = torch.zeros_like(kept), torch.zeros_like(res[1]), torch.zeros_like(ns)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.evict(dev[0], dev[1], dev[4], gl, dev[5], dev[6], keep, recent, kept=k2, new_lens=l2,
                 new_scores=s2)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(k2, kept) and torch.equal(l2, res[1])
    assert torch.equal(dev[0].view(torch.int16), pools[0].view(torch.int16))


@pytest.mark.gpu
def test_bad_lengths_and_blocks_are_skipped(pa):
    lens, keep, recent = [64, 64, 64, 64], 32, 8
    case = _case(lens, 2, 64, 16, "f16", keep, 21)
    kc, vc, _, _, tab, new, scores = case
    bad_tab, bad_new = tab.clone(), new.clone()
    bad_tab[2, :] = kc.shape[0] + 3                # every source block outside the pool
    bad_new[3, 1] = -5                             # the second half of sequence 3 has no place
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    pools, res = _run(pa, (kc, vc, None, None, bad_tab, bad_new, scores), [64, 65, 64, 64], keep,
                      recent, "f16", err_flag=flag)
    assert int(flag) == pa.DEVERR_SEQ_LEN | pa.DEVERR_BLOCK_ID
    assert pa.get_device_error(clear=True) == pa.DEVERR_SEQ_LEN | pa.DEVERR_BLOCK_ID
    assert res[1].tolist() == [32, 0, 32, 32]
    assert (res[0][1] == -1).all()
    want, wv = kc.clone(), vc.clone()
    keep_idx = p64.evict(scores, [64, 0, 64, 64], keep, recent)
    for s, places in ((0, 32), (3, 16)):
        for h in range(2):
            j = torch.arange(places)
            t = torch.tensor(keep_idx[s][h])[:places]
            want[new[s].long()[j // 16], j % 16, h] = kc[tab[s].long()[t // 16], t % 16, h]
    assert torch.equal(pools[0].cpu(), want)


@pytest.mark.gpu
def test_room_for_what_stays_is_checked(pa):
    lens, keep = [64, 20], 32
    case = _case(lens, 1, 64, 16, "f16", keep, 2)
    narrow = (*case[:5], case[5][:, :1].contiguous(), case[6])       # 16 places only
    pools, res = _run(pa, narrow, lens, keep, 0, "f16")
    assert res[1].tolist() == [0, 0] and (res[0] == -1).all()
    assert torch.equal(pools[0].cpu(), case[0])
    assert pa.get_device_error(clear=True) == pa.DEVERR_SEQ_LEN


# ---------------------------------------------------------------------- CPU

@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_390_b200 import build, pa
    build.build()
    return pa.lib()


def _call(lib, **over):
    fake, fake2 = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 21)
    d = dict(kc=fake, vc=fake, cd=1, ks=None, vs=None, tab=fake, mb=8, sl=fake, new=fake2, mnb=4,
             sc=fake, ss=128, keep=32, recent=8, kept=fake, kst=32, ns=fake2, nst=32, nl=fake2, S=2,
             Hkv=2, D=128, bs=16, nb=20)
    d.update(over)
    return lib.pa_evict(d["kc"], d["vc"], d["cd"], d["ks"], d["vs"], d["tab"], d["mb"], d["sl"],
                        d["new"], d["mnb"], d["sc"], d["ss"], d["keep"], d["recent"], d["kept"],
                        d["kst"], d["ns"], d["nst"], d["nl"], d["S"], d["Hkv"], d["D"], d["bs"],
                        d["nb"], None, None)


@pytest.mark.parametrize("over,status", [
    (dict(S=0), 0), (dict(S=-1), 1), (dict(kc=None), 1), (dict(keep=0), 1), (dict(recent=33), 1),
    (dict(recent=-1), 1), (dict(bs=12), 1), (dict(D=80), 2), (dict(cd=4), 1), (dict(cd=5), 1),
    (dict(ss=0), 1), (dict(kst=0), 1), (dict(nst=0), 1), (dict(mnb=0), 1), (dict(kept=None), 1),
    (dict(nl=ctypes.c_void_p(1 << 20)), 1), (dict(ns=ctypes.c_void_p(1 << 20)), 1),
    (dict(new=ctypes.c_void_p(1 << 20)), 1), (dict(kc=ctypes.c_void_p((1 << 20) + 4)), 1),
    (dict(sc=None), 1), (dict(S=70000), 2)])
def test_host_checks(lib, over, status):
    assert _call(lib, **over) == status


def test_binding_refusals(lib):
    from paged_kv_cache_390_b200 import pa
    kc = torch.zeros(4, 16, 2, 64)
    tab, lens = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    sc = torch.zeros(2, 2, 48)
    for args in ((kc, kc, tab, lens, tab, sc.double()), (kc, kc, tab.long(), lens, tab, sc),
                 (kc, kc, tab, lens[:1], tab, sc), (kc, kc, tab, lens, tab, sc[:, :1]),
                 (kc, kc.half(), tab, lens, tab, sc), (kc, kc, tab, lens, tab, sc)):
        with pytest.raises(ValueError):
            pa.evict(*args, 8, 2)


def _manager(n=20, bs=4, prefix=False, cpu=4):
    from paged_kv_cache_390_b200.block_manager import BlockManager
    return BlockManager(n, bs, cpu, prefix)


def test_manager_hands_out_fresh_blocks(lib):
    from paged_kv_cache_390_b200 import pa
    m = _manager()
    m.add_sequence(1, range(14))
    m.add_sequence(2, range(6))
    m.add_sequence(3, range(3))
    old, _ = m.build_batch([1, 2, 3])
    free = m.free_gpu_blocks
    new = m.evict([1, 2, 3], 7)
    assert new.shape == (3, 2)
    assert (new[0] >= 0).all() and (new[1] >= 0).all() and new[2, 0] >= 0 and new[2, 1] == -1
    ids = [b for b in new.ravel().tolist() if b >= 0]
    assert len(set(ids)) == 5 and not set(ids) & {b for b in old.ravel().tolist() if b >= 0}
    assert [m.block_table(s)[1] for s in (1, 2, 3)] == [7, 6, 3]
    assert m.free_gpu_blocks == free - 5 + 7
    slot, src, dst = m.append_token(1, 99)               # goes on at place 7
    assert slot == new[0, 1] * 4 + 3 and src == dst == -1
    with pytest.raises(pa.PAError):
        m.evict([1, 1], 4)
    with pytest.raises(pa.PAError):
        m.evict([9], 4)
    with pytest.raises(pa.PAError):
        m.evict([1], 0)
    for s in (1, 2, 3):
        m.free_sequence(s)
    assert m.free_gpu_blocks == 20


def test_manager_needs_room_before_it_changes_anything(lib):
    from paged_kv_cache_390_b200 import pa
    m = _manager(n=6)
    m.add_sequence(1, range(16))
    with pytest.raises(pa.PAError) as e:
        m.evict([1], 12)                                  # three fresh blocks, two free
    assert e.value.status == pa.PA_ERR_NO_SPACE
    assert m.block_table(1)[1] == 16 and m.free_gpu_blocks == 2
    m.swap_out([1])
    with pytest.raises(pa.PAError):
        m.evict([1], 4)                                   # swapped out
    assert m.evict([], 4).shape == (0, 1)


def test_manager_shared_and_cached_blocks_survive(lib):
    m = _manager(prefix=True)
    prompt = list(range(100, 113))
    m.add_sequence(1, prompt)
    m.fork(1, 2)
    kept = m.block_table(2)[0].tolist()
    m.evict([1], 6)
    assert m.block_table(2)[0].tolist() == kept           # the fork still has them
    _, cached = m.add_sequence(3, prompt)                 # and the prefix cache too
    assert cached == 12 and m.block_table(3)[0].tolist()[:3] == kept[:3]
    # what the cut sequence fills is never offered: its blocks hold mixed tokens
    for t in range(10):
        m.append_token(1, 500 + t)
    _, cached = m.add_sequence(4, prompt[:6] + [500 + t for t in range(10)] + [1])
    assert cached == 4                                    # only the prompt's own first block
    for s in (1, 2, 3, 4):
        m.free_sequence(s)
    assert m.free_gpu_blocks == 20

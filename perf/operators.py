"""What the masked attention, the rotary cache write and the cache eviction have to do,
as measurable cases: the inputs a serving program holds, one pass of each operator in
elementary torch operations (``own = False``) or through this package (``own = True``),
and the same results in 64 bits.

Operators (``case["op"]``):

* ``rope``: rotary positions with several axes (time, height, width) on the query and key
  rows of new tokens; the rotated keys and the values go into the paged cache.
* ``decode``: one new token per sequence over the paged cache, the scores capped by a
  tanh, with a bias by distance (one slope per head), a sliding window and the start of
  the token's document; optionally every cached token's attention weight is added to a
  running score.
* ``prefill``: several new tokens per sequence over the paged cache with the same
  changes to the scores, causal, with a document start per row and a prefix that sees
  itself whole.
* ``evict``: of every kv head of a sequence keep the newest tokens and the ones with the
  highest running score, and move them to fresh blocks in their order.
"""
import math
import random

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NEG = float("-inf")


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------

def _rope(name, tokens, H, Hkv, D, bs, dtype, sections, spread, interleaved, fused_qkv, far, pads):
    return dict(name=name, op="rope", tokens=tokens, H=H, Hkv=Hkv, D=D, bs=bs, dtype=dtype,
                sections=sections, spread=spread, interleaved=interleaved, fused_qkv=fused_qkv,
                far=far, pads=pads)


def _decode(name, seqs, lo, hi, H, Hkv, D, bs, dtype, cache, cap, alibi, docs, window, scores):
    return dict(name=name, op="decode", seqs=seqs, lo=lo, hi=hi, H=H, Hkv=Hkv, D=D, bs=bs,
                dtype=dtype, cache=cache, cap=cap, alibi=alibi, docs=docs, window=window,
                scores=scores)


def _prefill(name, seqs, q_lo, q_hi, cached, H, Hkv, bs, dtype, cap, alibi, doc, prefix, window):
    return dict(name=name, op="prefill", seqs=seqs, q_lo=q_lo, q_hi=q_hi, cached=cached, H=H,
                Hkv=Hkv, D=128, bs=bs, dtype=dtype, cap=cap, alibi=alibi, doc=doc,
                prefix=prefix, window=window)


def _evict(name, seqs, lo, hi, Hkv, D, bs, cache, keep, recent):
    return dict(name=name, op="evict", seqs=seqs, lo=lo, hi=hi, Hkv=Hkv, D=D, bs=bs,
                cache=cache, keep=keep, recent=recent)


def listed():
    return [
        # one decode step of a batch of 32: a token each, positions far into the text
        _rope("rope_step_f16", 32, 64, 8, 128, 16, "f16", "16,24,24", False, False, False, 32768, 0),
        # a prompt of text and images: the three axes differ, the rows are slices of one
        # fused projection, axes taken in turn over the frequencies
        _rope("rope_prompt_bf16", 8191, 64, 8, 128, 16, "bf16", "24,20,20", True, False, True, 32768, 0),
        # a small fp32 model in the pairs-side-by-side form, two axes (an image grid), a
        # padded batch, and positions past a million
        _rope("rope_grid_f32", 1500, 4, 4, 64, 16, "f32", "16,16", False, True, False, 1 << 20, 37),
        # a few short sequences with documents, 8-bit cache, one query head per kv head:
        # the smallest call, where launches count
        _decode("decode_short_int8", 3, 1, 100, 8, 8, 64, 16, "f16", "int8", 0.0, True, True, 0, True),
        # the 32-sequence serving batch with capped scores
        _decode("decode_cap_f16", 32, 512, 768, 64, 8, 128, 16, "f16", "f16", 50.0, False, False, 0, False),
        # long contexts, a bias by distance, weights added to the running scores
        _decode("decode_alibi_scores_bf16", 8, 30000, 32768, 64, 8, 128, 16, "bf16", "bf16", 0.0, True, False, 0, True),
        # a sliding window over an 8-bit cache, capped
        _decode("decode_window_fp8", 64, 3000, 16384, 32, 8, 128, 32, "bf16", "fp8", 30.0, False, False, 4096, False),
        # short ragged chunks of packed documents
        _prefill("prefill_docs_f16", 3, 100, 700, 130, 32, 8, 16, "f16", 0.0, False, 150, False, 0),
        # eight requests with 4096 cached tokens and 512 new ones, capped
        _prefill("prefill_cap_bf16", 8, 512, 512, 4096, 64, 8, 16, "bf16", 50.0, False, 0, False, 0),
        # whole prompts whose first part sees itself in both directions, a bias by distance
        _prefill("prefill_prefix_alibi_f16", 2, 4000, 4096, 0, 64, 8, 16, "f16", 0.0, True, 0, True, 0),
        # a batch of short conversations cut to 256 tokens
        _evict("evict_f16", 16, 500, 768, 8, 128, 16, "f16", 256, 64),
        # long contexts cut to a quarter
        _evict("evict_long_bf16", 8, 15000, 16384, 8, 128, 16, "bf16", 4096, 512),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "decode", "decode", "prefill", "evict"])
    H, Hkv = rng.choice([(64, 8), (32, 8), (8, 8), (8, 1), (12, 4), (4, 4)])
    bs = rng.choice([8, 16, 32])
    if op == "rope":
        D = rng.choice([64, 128])
        sections = rng.choice({64: ["32", "16,16", "8,12,12"], 128: ["64", "16,24,24", "24,20,20"]}[D])
        tokens = _log_int(rng, 1, 8191)
        return _rope(None, tokens, H, Hkv, D, bs, rng.choice(["f16", "bf16", "f32"]), sections,
                     rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.5,
                     _log_int(rng, 256, 1 << 20), rng.randrange(0, 1 + tokens // 4))
    if op == "decode":
        seqs = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, min(32768, 262144 // seqs))
        dtype = rng.choice(["f16", "bf16"])
        cache = rng.choice([dtype, dtype, "int8", "fp8"])
        return _decode(None, seqs, rng.randint(1, hi), hi, H, Hkv, rng.choice([64, 128]), bs, dtype,
                       cache, rng.choice([0.0, 30.0, 50.0]), rng.random() < 0.5,
                       rng.random() < 0.4, rng.choice([0, 0, _log_int(rng, 1, 8192)]),
                       rng.random() < 0.5)
    if op == "prefill":
        seqs = rng.randint(1, 6)
        q_hi = _log_int(rng, 1, 1500)
        return _prefill(None, seqs, rng.randint(1, q_hi), q_hi, _log_int(rng, 1, 2500) - 1, H, Hkv, bs,
                        rng.choice(["f16", "bf16"]), rng.choice([0.0, 30.0, 50.0]),
                        rng.random() < 0.5, rng.choice([0, 0, 40, 300]), rng.random() < 0.4,
                        rng.choice([0, 0, _log_int(rng, 1, 2000)]))
    seqs = _log_int(rng, 1, 16)
    hi = _log_int(rng, 64, min(16384, 131072 // seqs))
    keep = _log_int(rng, 1, max(1, hi // 2))
    return _evict(None, seqs, rng.randint(1, hi), hi, Hkv, rng.choice([64, 128]), bs,
                  rng.choice(["f16", "bf16", "int8", "fp8"]), keep, rng.randint(0, keep))


# ---------------------------------------------------------------------------------------
# lengths and inputs
# ---------------------------------------------------------------------------------------

def _key(case):
    return ",".join("%s=%s" % (k, case[k]) for k in sorted(case) if k != "name")


def _lengths(case):
    """Cached tokens per sequence (new ones included), and new tokens per sequence."""
    rng = random.Random(_key(case))
    if case["op"] == "prefill":
        q = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(case["seqs"])]
        return [n + case["cached"] for n in q], q
    n = [rng.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    return n, [1] * case["seqs"]


def _starts(case, lens, q_lens):
    """The first token of the document of every new token, row by row."""
    rng = random.Random(_key(case) + "docs")
    out = []
    for n, m in zip(lens, q_lens):
        if case["op"] == "decode":
            out.append(rng.randint(0, n - 1) if case["docs"] else 0)
            continue
        bounds, at = [0], 0
        while case["doc"] and at < n:
            at += rng.randint(1, 2 * case["doc"])
            bounds.append(at)
        k = 0
        for pos in range(n - m, n):
            while k + 1 < len(bounds) and bounds[k + 1] <= pos:
                k += 1
            out.append(bounds[k])
    return out


def _slopes(H):
    return [2.0 ** (-8.0 * (h + 1) / H) for h in range(H)]


def _prefixes(case, lens):
    rng = random.Random(_key(case) + "prefix")
    return [rng.randint(0, n // 2) for n in lens]


def _pool(case, blocks, gen, dev):
    """A pool's keys and values (and scales): every slot holds some token's row."""
    shape = (blocks, case["bs"], case["Hkv"], case["D"])
    out = {}
    for w in ("k", "v"):
        if case["cache"] in DT:
            out[w] = torch.randn(shape, generator=gen, device=dev, dtype=DT[case["cache"]])
            out[w + "_scale"] = None
            continue
        x = torch.randn(shape, generator=gen, device=dev, dtype=torch.float16).float()
        s = x.abs().amax(-1, keepdim=True) / (127.0 if case["cache"] == "int8" else 448.0)
        y = x / s
        out[w] = (y.round().to(torch.int8) if case["cache"] == "int8"
                  else y.to(torch.float8_e4m3fn).view(torch.uint8))
        out[w + "_scale"] = s[..., 0].transpose(1, 2).contiguous()
    return out


def _tables(counts, blocks, gen, dev, first=0):
    """Block tables cut from one permutation, padded with -1."""
    perm = torch.randperm(blocks, generator=gen, device=dev).to(torch.int32)
    t = torch.full((len(counts), max(1, max(counts))), -1, dtype=torch.int32, device=dev)
    at = first
    for s, c in enumerate(counts):
        t[s, :c] = perm[at:at + c]
        at += c
    return t, perm[at:]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    op, bs, Hkv, D = case["op"], case["bs"], case["Hkv"], case["D"]
    st = {"case": case}
    if op == "rope":
        T, H, dt = case["tokens"], case["H"], DT[case["dtype"]]
        rows = torch.randn((T, H + 2 * Hkv, D), generator=gen, device=dev, dtype=dt)
        q, k, v = rows[:, :H], rows[:, H:H + Hkv], rows[:, H + Hkv:]
        if not case["fused_qkv"]:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        sec = [int(x) for x in case["sections"].split(",")]
        pairs, axes = sum(sec), len(sec)
        axis = [a for a, n in enumerate(sec) for _ in range(n)]
        if case["spread"]:                      # the axes in turn, until each has its share
            left, axis = list(sec), []
            while len(axis) < pairs:
                for a in range(axes):
                    if left[a]:
                        left[a] -= 1
                        axis.append(a)
        base = torch.arange(T, device=dev) + int(torch.randint(0, case["far"], (1,), generator=gen, device=dev))
        pos = base.repeat(axes, 1)
        if axes > 1:                            # images: rows and columns of a grid
            grid = torch.randint(0, 64, (axes, T), generator=gen, device=dev)
            image = (torch.arange(T, device=dev) // 97) % 2 == 1
            pos = torch.where(image, base - torch.arange(T, device=dev) % 97 + grid, pos)
        blocks = -(-T // bs) + 2
        slots = torch.randperm(blocks * bs, generator=gen, device=dev)[:T]
        written = torch.arange(T, device=dev)
        if case["pads"]:                        # a padded batch: rows without a slot
            perm = torch.randperm(T, generator=gen, device=dev)
            slots[perm[:case["pads"]]] = -1
            written = perm[case["pads"]:].sort().values
        shape = (blocks, bs, Hkv, D)
        st.update(q=q, k=k, v=v, pos=pos.contiguous(), slots=slots.contiguous(), written=written,
                  inv_freq=torch.tensor([1e6 ** (-i / pairs) for i in range(pairs)],
                                        dtype=torch.float64, device=dev),
                  pair_axis=torch.tensor(axis, dtype=torch.int32, device=dev),
                  kc=torch.randn(shape, generator=gen, device=dev, dtype=dt),
                  vc=torch.randn(shape, generator=gen, device=dev, dtype=dt))
        return st
    lens, q_lens = _lengths(case)
    counts = [-(-n // bs) for n in lens]
    spare = [-(-min(n, case["keep"]) // bs) for n in lens] if op == "evict" else []
    blocks = sum(counts) + sum(spare) + 3
    full = dict(case, cache=case.get("cache", case.get("dtype")))
    pool = _pool(full, blocks, gen, dev)
    table, rest = _tables(counts, blocks, gen, dev)
    st.update(kc=pool["k"], vc=pool["v"], ks=pool["k_scale"], vs=pool["v_scale"], table=table,
              lens=torch.tensor(lens, dtype=torch.int32, device=dev), max_len=max(lens))
    S = case["seqs"]
    if op == "evict":
        t2 = torch.full((S, max(spare)), -1, dtype=torch.int32, device=dev)
        at = 0
        for s, c in enumerate(spare):
            t2[s, :c] = rest[at:at + c]
            at += c
        # running scores: a few tokens draw most of the weight, some were never looked at
        sc = torch.exp(2.0 * torch.randn((S, Hkv, max(lens)), generator=gen, device=dev))
        sc = torch.where(torch.rand(sc.shape, generator=gen, device=dev) < 0.1, 0.0, sc)
        width = max(spare) * bs
        st.update(new_table=t2, scores=sc,
                  new_scores=torch.zeros((S, Hkv, width), device=dev),
                  kept=torch.full((S, Hkv, width), -1, dtype=torch.int32, device=dev),
                  new_lens=torch.zeros(S, dtype=torch.int32, device=dev))
        return st
    H, rows = case["H"], sum(q_lens)
    # queries whose logits spread as a trained model's do (a few units either way)
    st.update(q=2.0 * torch.randn((rows, H, D), generator=gen, device=dev, dtype=DT[case["dtype"]]),
              scale=1.0 / math.sqrt(D),
              slopes=torch.tensor(_slopes(H), device=dev) if case["alibi"] else None, start=None)
    if case.get("docs") or case.get("doc"):
        st["start"] = torch.tensor(_starts(case, lens, q_lens), dtype=torch.int32, device=dev)
    if op == "decode":
        if case["scores"]:
            st["scores"] = torch.exp(torch.randn((S, Hkv, max(lens)), generator=gen, device=dev))
            st["scores_out"] = st["scores"].clone()
        return st
    begin = [0]
    for n in q_lens:
        begin.append(begin[-1] + n)
    st.update(begin=torch.tensor(begin, dtype=torch.int32, device=dev), max_q=max(q_lens),
              prefix=(torch.tensor(_prefixes(case, lens), dtype=torch.int32, device=dev)
                      if case["prefix"] else None))
    return st


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------

def run(state):
    return {"rope": _run_rope, "decode": _run_decode, "prefill": _run_prefill,
            "evict": _run_evict}[state["case"]["op"]](state)


def _run_rope(st):
    if own:
        from paged_kv_cache_390_b200 import pa
        q = pa.rope_and_cache(st["q"], st["k"], st["v"], st["pos"], st["inv_freq"], st["pair_axis"],
                              st["kc"], st["vc"], st["slots"],
                              interleaved=st["case"]["interleaved"])
        return {"q": q, "k_cache": st["kc"], "v_cache": st["vc"]}
    angle = st["pos"].double()[st["pair_axis"].long()] * st["inv_freq"][:, None]     # [pairs, T]
    cos, sin = angle.cos().float().T[:, None], angle.sin().float().T[:, None]        # [T, 1, pairs]

    def turn(x):
        x = x.float()
        if st["case"]["interleaved"]:
            a, b = x[..., 0::2], x[..., 1::2]
            return torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
        a, b = x.chunk(2, dim=-1)
        return torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)

    dt = st["q"].dtype
    at = st["slots"][st["written"]]
    st["kc"].flatten(0, 1)[at] = turn(st["k"]).to(dt)[st["written"]]
    st["vc"].flatten(0, 1)[at] = st["v"][st["written"]]
    return {"q": turn(st["q"]).to(dt), "k_cache": st["kc"], "v_cache": st["vc"]}


def _rows_of(st, which, dtype):
    """Every sequence's cached rows [S, max_len, Hkv, D], in `dtype`; padding reads block 0."""
    bs = st["case"]["bs"]
    t = torch.arange(st["max_len"], device=st["lens"].device)
    blk = st["table"].long().clamp(min=0)[:, t // bs]                                # [S, L]
    x = st["kc" if which == "k" else "vc"]
    s = st["ks" if which == "k" else "vs"]
    if x.dtype == torch.uint8:
        x = x.view(torch.float8_e4m3fn)
    rows = x[blk, t % bs].to(dtype) if x.dtype != torch.float8_e4m3fn else \
        x.view(torch.uint8)[blk, t % bs].view(torch.float8_e4m3fn).to(dtype)
    if s is not None:
        rows = rows * s.transpose(1, 2)[blk, t % bs].to(dtype)[..., None]
    return rows


def _run_decode(st):
    case = st["case"]
    if own:
        from paged_kv_cache_390_b200 import pa
        S, H, D = st["q"].shape
        width = st["scores"].shape[2] if case["scores"] else 0
        if "workspace" not in st:               # kept by the program, zeroed once
            st["workspace"] = pa.MaskedWorkspace(S, H, case["Hkv"], D, width)
        out = pa.decode_masked(st["q"], st["kc"], st["vc"], st["table"], st["lens"], st["scale"],
                               softcap=case["cap"], alibi_slopes=st["slopes"],
                               kv_start=st["start"], window=case["window"],
                               scores_in=st.get("scores"), scores_out=st.get("scores_out"),
                               k_scale=st["ks"], v_scale=st["vs"], workspace=st["workspace"])
        return {"out": out, "scores": st["scores_out"]} if case["scores"] else {"out": out}
    S, H, D = st["q"].shape
    G = H // case["Hkv"]
    k, v = _rows_of(st, "k", torch.float32), _rows_of(st, "v", torch.float32)
    x = torch.einsum("skgd,stkd->skgt", st["q"].float().view(S, case["Hkv"], G, D), k) * st["scale"]
    if case["cap"]:
        x = case["cap"] * torch.tanh(x / case["cap"])
    t = torch.arange(st["max_len"], device=x.device)
    pos = (st["lens"] - 1)[:, None]
    if case["alibi"]:
        x = x - st["slopes"].view(case["Hkv"], G, 1) * (pos - t).abs().float()[:, None, None]
    seen = t < st["lens"][:, None]
    if st["start"] is not None:
        seen = seen & (t >= st["start"][:, None])
    if case["window"]:
        seen = seen & (pos - t < case["window"])
    x = x.masked_fill(~seen[:, None, None], NEG)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    w = p / p.sum(-1, keepdim=True)
    out = torch.einsum("skgt,stkd->skgd", w, v).reshape(S, H, D).to(st["q"].dtype)
    if not case["scores"]:
        return {"out": out}
    st["scores_out"].copy_(st["scores"] + w.sum(2))
    return {"out": out, "scores": st["scores_out"]}


def _run_prefill(st):
    case = st["case"]
    if own:
        from paged_kv_cache_390_b200 import pa
        return pa.prefill_masked(st["q"], st["kc"], st["vc"], st["table"], st["lens"], st["begin"],
                                 st["scale"], softcap=case["cap"], alibi_slopes=st["slopes"],
                                 kv_start=st["start"], prefix_lens=st["prefix"],
                                 window=case["window"], max_query_len=st["max_q"])
    rows, H, D = st["q"].shape
    G, S = H // case["Hkv"], case["seqs"]
    begin = st["begin"].long()
    r = torch.arange(st["max_q"], device=begin.device)
    q_len = (begin[1:] - begin[:-1])[:, None]
    at = (begin[:-1, None] + r).clamp(max=rows - 1)                                  # [S, R]
    q = st["q"].float()[at].view(S, st["max_q"], case["Hkv"], G, D)
    k, v = _rows_of(st, "k", torch.float32), _rows_of(st, "v", torch.float32)
    x = torch.einsum("srkgd,stkd->skgrt", q, k)
    x *= st["scale"]
    if case["cap"]:
        x = torch.tanh(x.div_(case["cap"])).mul_(case["cap"])
    t = torch.arange(st["max_len"], device=x.device)
    pos = (st["lens"][:, None] - q_len + r)[..., None]                               # [S, R, 1]
    if case["alibi"]:
        x -= st["slopes"].view(case["Hkv"], G, 1, 1) * (pos - t).abs().float()[:, None, None]
    seen = t <= pos
    if st["prefix"] is not None:
        seen = seen | (t < st["prefix"][:, None, None])
    seen = seen & (t < st["lens"][:, None, None])
    if st["start"] is not None:
        seen = seen & (t >= st["start"].long()[at][..., None])
    if case["window"]:
        seen = seen & (pos - t < case["window"])
    x.masked_fill_(~seen[:, None, None], NEG)
    p = torch.exp(x.sub_(x.amax(-1, keepdim=True)))
    total = p.sum(-1)
    out = torch.einsum("skgrt,stkd->srkgd", p, v) / total.permute(0, 3, 1, 2)[..., None]
    flat = out.reshape(S * st["max_q"], H, D).to(st["q"].dtype)
    row = torch.arange(rows, device=begin.device)
    s = torch.searchsorted(begin, row, right=True) - 1
    return flat[s * st["max_q"] + row - begin[s]]


def _run_evict(st):
    case = st["case"]
    if own:
        from paged_kv_cache_390_b200 import pa
        pa.evict(st["kc"], st["vc"], st["table"], st["lens"], st["new_table"], st["scores"],
                 case["keep"], case["recent"], new_scores=st["new_scores"], kept=st["kept"],
                 new_lens=st["new_lens"], k_scale=st["ks"], v_scale=st["vs"])
    else:
        bs, keep = case["bs"], case["keep"]
        lens = st["lens"].long()[:, None, None]
        S, Hkv, L = st["scores"].shape
        t = torch.arange(L, device=lens.device)
        # the newest first, then by score (equal scores: the lower index), then the padding
        rank = torch.where(t >= lens, NEG, torch.where(t >= lens - case["recent"], math.inf, st["scores"]))
        order = torch.sort(rank, dim=-1, descending=True, stable=True).indices
        place = torch.empty_like(order).scatter_(2, order, t.expand(S, Hkv, L).contiguous())
        stays = (place < keep) & (t < lens)
        width = st["kept"].shape[2]
        first = torch.sort(torch.where(stays, t, L), dim=-1).values                   # in their order
        first = torch.cat([first, first.new_full((S, Hkv, max(0, width - L)), L)], -1)[..., :width]
        there = first < L
        st["kept"].copy_(torch.where(there, first, -1).int())
        st["new_lens"].copy_(lens[:, 0, 0].clamp(max=keep))
        src = torch.where(there, first, 0)
        st["new_scores"].copy_(torch.where(there, st["scores"].gather(2, src), st["new_scores"]))
        j = torch.arange(width, device=lens.device)
        dst_blk = st["new_table"].long()[:, j // bs].clamp(min=0)[:, None].expand(S, Hkv, width)
        src_blk = st["table"].long().gather(1, (src // bs).view(S, -1)).view(S, Hkv, width).clamp(min=0)
        head = torch.arange(Hkv, device=lens.device)[:, None].expand(S, Hkv, width)
        # places past the end: the first place's row once more, to the first place
        dst_off = (j % bs).expand(S, Hkv, width)
        src_blk = torch.where(there, src_blk, src_blk[..., :1])
        src_off = torch.where(there, src % bs, src[..., :1] % bs)
        dst_blk = torch.where(there, dst_blk, dst_blk[..., :1])
        dst_off = torch.where(there, dst_off, dst_off[..., :1])
        for x in (st["kc"], st["vc"]):
            x[dst_blk, dst_off, head] = x[src_blk, src_off, head]
        for x in (st["ks"], st["vs"]):
            if x is not None:
                x[dst_blk, head, dst_off] = x[src_blk, head, src_off]
    res = {"kept": st["kept"], "new_lens": st["new_lens"], "new_scores": st["new_scores"],
           "k_cache": st["kc"], "v_cache": st["vc"]}
    if st["ks"] is not None:
        res.update(k_scale=st["ks"], v_scale=st["vs"])
    return res


# ---------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------

def _es(name):
    return {"f32": 4, "f16": 2, "bf16": 2}.get(name, 1)


def work(case):
    op, Hkv, D = case["op"], case["Hkv"], case["D"]
    if op == "rope":
        T, H, es = case["tokens"], case["H"], _es(case["dtype"])
        axes, pairs = case["sections"].count(",") + 1, sum(map(int, case["sections"].split(",")))
        w = T - case["pads"]
        return {"bytes": 2 * T * H * D * es + 4 * w * Hkv * D * es + T * 8 * (axes + 1) + 12 * pairs,
                "flops": 3 * (T * H + w * Hkv) * D}
    lens, q_lens = _lengths(case)
    cache = case.get("cache", case.get("dtype"))
    row = 2 * D * _es(cache) + (0 if cache in DT else 8)       # a token's K and V of one kv head
    table = sum(-(-n // case["bs"]) for n in lens) * 4
    if op == "evict":
        kept = sum(min(n, case["keep"]) for n in lens)
        b = 4 * Hkv * sum(lens) + 2 * kept * Hkv * row + 8 * kept * Hkv + table
        return {"bytes": b, "flops": Hkv * sum(lens)}
    H = case["H"]
    starts, at, pairs, span = _starts(case, lens, q_lens), 0, 0, 0
    prefix = _prefixes(case, lens) if case.get("prefix") else [0] * len(lens)
    for n, m, pre in zip(lens, q_lens, prefix):
        first, last = n, 0
        for i in range(m):
            pos = n - m + i
            lo = starts[at + i]
            if case["window"]:
                lo = max(lo, pos - case["window"] + 1)
            hi = max(pos + 1, pre)
            pairs += max(0, hi - lo)
            first, last = min(first, lo), max(last, hi)
        at += m
        span += max(0, last - first)
    b = 2 * sum(q_lens) * H * D * _es(case["dtype"]) + span * Hkv * row + table
    if case.get("scores"):
        b += 8 * Hkv * sum(lens)
    return {"bytes": b, "flops": 4 * pairs * H * D}


# ---------------------------------------------------------------------------------------
# the same in 64 bits
# ---------------------------------------------------------------------------------------

def _plain_rows(st, s, which, n):
    """Sequence s's n cached rows [n, Hkv, D] as 64-bit values."""
    bs = st["case"]["bs"]
    ids = st["table"][s, :-(-n // bs)].long()
    x = st[which + "c"][ids]
    if x.dtype == torch.uint8:
        x = x.view(torch.float8_e4m3fn).to(torch.float32)
    x = x.double()
    if st[which + "s"] is not None:
        x = x * st[which + "s"][ids].double().permute(0, 2, 1).unsqueeze(3)
    return x.flatten(0, 1)[:n]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        T, half = case["tokens"], st["inv_freq"].numel()
        turn = torch.zeros((T, half), dtype=torch.complex128, device="cuda")
        for i in range(half):
            a = st["pos"][int(st["pair_axis"][i])].double() * st["inv_freq"][i]
            turn[:, i] = torch.polar(torch.ones_like(a), a)

        def rotate(x):
            x = x.double()
            even = slice(0, None, 2) if case["interleaved"] else slice(0, half)
            odd = slice(1, None, 2) if case["interleaved"] else slice(half, None)
            z = torch.complex(x[..., even].contiguous(), x[..., odd].contiguous()) * turn[:, None]
            out = torch.empty_like(x)
            out[..., even], out[..., odd] = z.real, z.imag
            return out

        k, v = st["kc"].double().flatten(0, 1), st["vc"].double().flatten(0, 1)
        ok = st["slots"] >= 0
        k[st["slots"][ok]] = rotate(st["k"])[ok]
        v[st["slots"][ok]] = st["v"].double()[ok]
        return {"q": rotate(st["q"]), "k_cache": k.view(st["kc"].shape),
                "v_cache": v.view(st["vc"].shape)}
    lens, q_lens = _lengths(case)
    if op == "evict":
        return _exact_evict(case, st, lens)
    H, Hkv, D = case["H"], case["Hkv"], case["D"]
    G = H // Hkv
    starts = _starts(case, lens, q_lens)
    prefix = _prefixes(case, lens) if case.get("prefix") else [0] * len(lens)
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    scores = st["scores"].double() if case.get("scores") else None
    at = 0
    for s, (n, m) in enumerate(zip(lens, q_lens)):
        k, v = _plain_rows(st, s, "k", n), _plain_rows(st, s, "v", n)
        pos = torch.arange(n - m, n, device="cuda")
        t = torch.arange(n, device="cuda")
        lo = torch.tensor(starts[at:at + m], device="cuda")
        if case["window"]:
            lo = torch.maximum(lo, pos - case["window"] + 1)
        hi = torch.clamp(pos + 1, min=prefix[s])
        hidden = (t[None] < lo[:, None]) | (t[None] >= hi[:, None])
        for h in range(H):
            x = st["q"][at:at + m, h].double() @ k[:, h // G].T * st["scale"]
            if case["cap"]:
                x = case["cap"] * torch.tanh(x / case["cap"])
            if case["alibi"]:
                x = x - float(st["slopes"][h]) * (pos[:, None] - t[None]).abs().double()
            w = torch.softmax(x.masked_fill(hidden, NEG), dim=-1)
            out[at:at + m, h] = w @ v[:, h // G]
            if scores is not None:
                scores[s, h // G, :n] += w[0]
        at += m
    if op == "prefill":
        return out
    return {"out": out} if scores is None else {"out": out, "scores": scores}


def _exact_evict(case, st, lens):
    bs, keep, recent = case["bs"], case["keep"], case["recent"]
    value = st["scores"].double().cpu().numpy()
    table, fresh = st["table"].tolist(), st["new_table"].tolist()
    kept, sc = st["kept"].cpu(), st["new_scores"].double().cpu()
    src, dst, heads = [], [], []
    for s, n in enumerate(lens):
        m = min(n, keep)
        for h in range(case["Hkv"]):
            old = list(range(max(0, n - recent)))
            old.sort(key=lambda i: (-value[s, h, i], i))
            new = list(range(max(0, n - recent), n))
            chosen = sorted(new[:m] + old[:max(0, m - len(new))])
            kept[s, h, :m] = torch.tensor(chosen, dtype=torch.int32)
            sc[s, h, :m] = torch.from_numpy(value[s, h, chosen])
            src += [table[s][i // bs] * bs + i % bs for i in chosen]
            dst += [fresh[s][j // bs] * bs + j % bs for j in range(m)]
            heads += [h] * m
    src, dst = torch.tensor(src, device="cuda"), torch.tensor(dst, device="cuda")
    heads = torch.tensor(heads, device="cuda")
    res = {"kept": kept, "new_lens": torch.tensor([min(n, keep) for n in lens], dtype=torch.int32),
           "new_scores": sc}
    for name, x in (("k_cache", st["kc"]), ("v_cache", st["vc"])):
        y = x.clone().flatten(0, 1)
        y[dst, heads] = y[src, heads]
        y = y.view(x.shape)
        res[name] = y if x.dtype in (torch.int8, torch.uint8) else y.double()
    if st["ks"] is not None:
        for name, x in (("k_scale", st["ks"]), ("v_scale", st["vs"])):
            y = x.double()
            y[dst // bs, heads, dst % bs] = y[src // bs, heads, src % bs]
            res[name] = y
    return res

"""The measured cases of the paged-cache operators, with their plain forms.

Five operators that serve a paged FP8 KV cache with positions on several axes:

  rope        rotary positions with several axes (time, height, width): the
              dimension pairs of a head are divided among the axes, each pair
              turned by its axis' position; forward, and the gradient (the
              turn back)
  write       new tokens into the cache's pages: K turned, K and V quantised
              to E4M3 with one power-of-two scale per token and head
  attend      attention of each sequence's new tokens over its pages
  accumulate  the attention weight that every cached token received
  evict       per sequence and head, the `keep` tokens with the most weight
              (the last `recent` always) copied, in order, to new pages

Page layouts, shared by all of them (P = tokens of a page):
  kcodes [pages][kv_heads][P][head_dim]   E4M3
  vcodes [pages][kv_heads][head_dim][P]   E4M3 (V transposed)
  kscale, vscale [pages][kv_heads][P]     E8M0: byte b stands for 2^(b - 127)
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one chunk of a video model: the 757 tokens' queries of 48 heads turned by (time, height, width)
        {"name": "rope chunk", "op": "rope", "n": 757, "heads": 48, "dim": 128, "axes": 3, "dtype": "bf16", "back": False},
        # the gradient through the turn for a training clip of 45 such chunks, gradients kept in 32 bits
        {"name": "rope clip gradient", "op": "rope", "n": 34065, "heads": 16, "dim": 128, "axes": 3, "dtype": "f32", "back": True},
        # one decode step of 64 chat sequences: a token each
        {"name": "write 64 single tokens", "op": "write", "seqs": 64, "new_min": 1, "new_max": 1, "kv_min": 40, "kv_max": 4093,
         "kv_heads": 8, "dim": 128, "page": 16, "axes": 1},
        # one chunk of the video model into its cache
        {"name": "write chunk", "op": "write", "seqs": 1, "new_min": 757, "new_max": 757, "kv_min": 5788, "kv_max": 5788,
         "kv_heads": 48, "dim": 128, "page": 64, "axes": 3},
        # the shortest call: one token of one young sequence, where latency is all
        {"name": "attend one token", "op": "attend", "seqs": 1, "new_min": 1, "new_max": 1, "kv_min": 337, "kv_max": 337,
         "heads": 16, "kv_heads": 2, "dim": 64, "page": 16, "causal": True},
        # a decode step of 32 sequences of very different ages, six query heads to a key head
        {"name": "attend 32 single tokens", "op": "attend", "seqs": 32, "new_min": 1, "new_max": 1, "kv_min": 61, "kv_max": 16381,
         "heads": 48, "kv_heads": 8, "dim": 128, "page": 64, "causal": True},
        # the video model's call: 757 queries see the whole cache of 5,788 tokens
        {"name": "attend chunk", "op": "attend", "seqs": 1, "new_min": 757, "new_max": 757, "kv_min": 5788, "kv_max": 5788,
         "heads": 48, "kv_heads": 48, "dim": 128, "page": 64, "causal": False},
        # chunked prefill of four prompts at different stages
        {"name": "attend prefill", "op": "attend", "seqs": 4, "new_min": 259, "new_max": 2701, "kv_min": 1031, "kv_max": 6143,
         "heads": 48, "kv_heads": 8, "dim": 128, "page": 64, "causal": True},
        # the weights of a decode step, kept up for a later eviction
        {"name": "accumulate single tokens", "op": "accumulate", "seqs": 16, "new_min": 1, "new_max": 1, "kv_min": 509, "kv_max": 8191,
         "heads": 48, "kv_heads": 8, "dim": 128, "page": 64, "causal": True},
        # the weights of the video model's chunk
        {"name": "accumulate chunk", "op": "accumulate", "seqs": 1, "new_min": 757, "new_max": 757, "kv_min": 5788, "kv_max": 5788,
         "heads": 48, "kv_heads": 48, "dim": 128, "page": 64, "causal": False},
        # one sequence over its budget by half
        {"name": "evict one sequence", "op": "evict", "seqs": 1, "kv_min": 1021, "kv_max": 1021, "keep": 512, "recent": 32,
         "kv_heads": 8, "dim": 128, "page": 16},
        # a batch of long sequences cut to one budget
        {"name": "evict batch", "op": "evict", "seqs": 8, "kv_min": 9001, "kv_max": 32749, "keep": 8192, "recent": 256,
         "kv_heads": 8, "dim": 128, "page": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        case = _draw(rng)
        if _cost(case) <= most:
            return case


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def _draw(rng):
    op = rng.choice(["rope", "write", "attend", "attend", "accumulate", "evict"])
    dim = rng.choice([64, 128, 128])
    if op == "rope":
        return {"op": op, "n": _log(rng, 1, 34065), "heads": rng.randint(1, 16), "dim": dim, "axes": rng.randint(1, 4),
                "dtype": rng.choice(["bf16", "f32"]), "back": rng.random() < 0.5}
    page = rng.choice([16, 32, 64, 128])
    if op == "evict":
        kv = _log(rng, 16, 30000)
        keep = rng.randint(1, min(kv, 8192))
        return {"op": op, "seqs": rng.randint(1, 6), "kv_min": max(1, int(kv * rng.uniform(0.2, 1.0))), "kv_max": kv, "keep": keep,
                "recent": rng.randint(0, keep), "kv_heads": rng.randint(1, 8), "dim": dim, "page": page}
    shape = rng.choice(["single", "few", "chunk"])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    if shape == "single":
        seqs, new, kv = _log(rng, 1, 32), 1, _log(rng, 1, 16381)
    elif shape == "few":
        seqs, new, kv = rng.randint(1, 8), rng.randint(2, 33), _log(rng, 40, 16381)
    else:
        seqs, new, kv = rng.randint(1, 3), _log(rng, 40, 1500), _log(rng, 1501, 6143)
    case = {"op": op, "seqs": seqs, "new_min": rng.randint(1, new), "new_max": new, "kv_min": rng.randint(min(new, kv), kv), "kv_max": kv,
            "kv_heads": kv_heads, "dim": dim, "page": page}
    if op == "write":
        return dict(case, axes=rng.randint(1, 4))
    return dict(case, heads=kv_heads * rng.choice([1, 1, 2, 4, 6, 8]), causal=rng.random() < 0.7)


# ------------------------------------------------------------------ sizes of a case
def _spread(lo, hi, seqs):
    """`seqs` lengths from lo to hi, the longest first, the shortest second, and so on inwards."""
    v = [hi - (hi - lo) * i // max(1, seqs - 1) for i in range(seqs)]
    return [v[i // 2] if i % 2 == 0 else v[seqs - 1 - i // 2] for i in range(seqs)]


def _lengths(case):
    """Per sequence: new tokens, cached tokens (the new ones included)."""
    kv = _spread(case["kv_min"], case["kv_max"], case["seqs"])
    new = _spread(case.get("new_min", 0), case.get("new_max", 0), case["seqs"])
    return [min(a, b) for a, b in zip(new, kv)], kv


def _sections(dim, axes):
    """Pairs of each axis: as even as they go, the first axis (time) with what is left over."""
    pairs = dim // 2
    even = pairs // axes
    return [pairs - even * (axes - 1)] + [even] * (axes - 1)


def _seen(new, kv, causal):
    """Pairs of a query token and a cached token that it sees."""
    return sum(n * k - (n * (n - 1) // 2 if causal else 0) for n, k in zip(new, kv))


def work(case):
    op, dim = case["op"], case["dim"]
    if op == "rope":
        size = 4 if case["dtype"] == "f32" else 2
        values = case["n"] * case["heads"] * dim
        return {"bytes": 2 * size * values + 4 * case["axes"] * case["n"], "flops": 3 * values}
    new, kv = _lengths(case)
    hk = case["kv_heads"]
    if op == "write":
        t = sum(new)
        return {"bytes": t * (hk * (2 * (2 * dim) + 2 * (dim + 1)) + 4 * case["axes"]), "flops": 7 * t * hk * dim}
    token = hk * (dim + 1)  # one token's codes and scales, K or V, of all heads
    if op == "evict":
        kept = sum(min(k, case["keep"]) for k in kv)
        return {"bytes": 2 * 2 * kept * token + 4 * hk * (sum(kv) + 2 * kept), "flops": hk * sum(kv)}
    t, hq = sum(new), case["heads"]
    pairs = _seen(new, kv, case["causal"]) * hq
    if op == "attend":
        return {"bytes": 2 * sum(kv) * token + t * hq * (2 * 2 * dim + 4), "flops": pairs * 4 * dim}
    return {"bytes": sum(kv) * (token + 2 * 4 * hk) + t * hq * (2 * dim + 4), "flops": pairs * 2 * dim}


# ------------------------------------------------------------------ inputs
def _quantise(x):
    """E4M3 codes (as bytes) and E8M0 bytes of rows x [..., dim] in 32 bits: the scale is the
    smallest power of two 2^e with max|x| <= 448 * 2^e (e in -124..7; 1 for a row of zeros)."""
    amax = x.abs().amax(-1)
    mant, e = torch.frexp(amax / 448)  # amax / 448 = mant * 2^e with mant in [0.5, 1)
    e = torch.where(mant == 0.5, e - 1, e).clamp(-124, 7)
    e = torch.where(amax == 0, torch.zeros_like(e), e)
    codes = torch.ldexp(x, -e[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), (e + 127).to(torch.uint8)


def _pool(case, g, kv, fill=True):
    """Pages for sequences of `kv` tokens, their ids scattered over the pool, and what they hold."""
    hk, dim, p = case["kv_heads"], case["dim"], case["page"]
    need = [-(-k // p) for k in kv]
    pages = sum(need) + 3
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(kv), max(need)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = ids[at:at + n]
        at += n
    pool = {"table": table, "kv_len": torch.tensor(kv, dtype=torch.int32, device=DEV)}
    for name, shape in (("k", (pages, hk, p, dim)), ("v", (pages, hk, p, dim))):
        x = torch.randn(shape, generator=g, device=DEV)
        # every channel has a spread of its own (a few of them large), every token a size of its own
        x *= torch.exp(0.5 * torch.randn((1, hk, 1, dim), generator=g, device=DEV)) * torch.exp(0.3 * torch.randn((pages, hk, p, 1), generator=g, device=DEV))
        codes, scale = _quantise(x)
        if name == "v":
            codes = codes.transpose(2, 3).contiguous()
        pool[name + "codes"], pool[name + "scale"] = codes, scale
        del x
    return pool


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, dim = case["op"], case["dim"]
    st = {"op": op, "case": case}
    if op == "rope":
        dtype = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        st["x"] = torch.randn((case["n"], case["heads"], dim), generator=g, device=DEV).to(dtype)
        st["y"] = torch.empty_like(st["x"])
        st["pos"] = _positions(case, case["n"], g)
        return st
    new, kv = _lengths(case)
    hk, t = case["kv_heads"], sum(new)
    if op == "evict":
        p, keep = case["page"], case["keep"]
        kept = [min(k, keep) for k in kv]
        st.update(_pool(case, g, kv + kept))
        st["dst"], st["table"] = st["table"][len(kv):, :-(-max(kept) // p)].contiguous(), st["table"][:len(kv), :-(-max(kv) // p)].contiguous()
        st["kv_len"] = st["kv_len"][:len(kv)].contiguous()
        # attention weight: few tokens have most of it, and a part of them none at all
        w = torch.randn((len(kv), hk, max(kv)), generator=g, device=DEV).mul(2).exp()
        st["scores"] = w * (torch.rand(w.shape, generator=g, device=DEV) > 0.2)
        st["kept"] = torch.full((len(kv), hk, keep), -1, dtype=torch.int32, device=DEV)
        st["scores_out"] = torch.zeros((len(kv), hk, keep), device=DEV)
        st["len_out"] = torch.zeros(len(kv), dtype=torch.int32, device=DEV)
        st["max_kv"] = max(kv)
        return st
    st.update(_pool(case, g, kv))
    st["q_start"] = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device=DEV)
    st["tokens"], st["max_new"], st["max_kv"] = t, max(new), max(kv)
    if op == "write":
        for name in "kv":
            x = torch.randn((t, hk, dim), generator=g, device=DEV) * torch.exp(0.5 * torch.randn((1, hk, dim), generator=g, device=DEV))
            st[name] = x.to(torch.bfloat16)
        st["pos"] = _positions(case, t, g)
        return st
    hq = case["heads"]
    st["q"] = torch.randn((t, hq, dim), generator=g, device=DEV).to(torch.bfloat16)
    if op == "attend":
        st["out"] = torch.zeros((t, hq, dim), dtype=torch.bfloat16, device=DEV)
        st["lse"] = torch.zeros((t, hq), device=DEV)
        return st
    st["lse"] = _lse(st)
    st["scores"] = torch.rand((len(kv), hk, max(kv)), generator=g, device=DEV)
    st["scores_out"] = torch.zeros_like(st["scores"])
    return st


def _positions(case, n, g):
    """[axes][n]: the first axis counts frames far into a session, the others run over a picture."""
    at = torch.arange(n, device=DEV)
    pos = [at // 7 + 190000] + [torch.randint(0, 90, (n,), generator=g, device=DEV) for _ in range(case["axes"] - 1)]
    return torch.stack(pos).to(torch.int32)


# ------------------------------------------------------------------ the plain forms
def _turn(x, pos, sections, sign):
    """x [n][heads][dim] in 32 bits, pairs (2i, 2i + 1) turned by sign * position * frequency."""
    axis = torch.repeat_interleave(torch.arange(len(sections), device=x.device), torch.tensor(sections, device=x.device))
    width = torch.tensor(sections, device=x.device)[axis]
    first = torch.tensor([sum(sections[:i]) for i in range(len(sections))], device=x.device)[axis]
    rank = torch.arange(axis.numel(), device=x.device) - first
    angle = pos[axis].t().double() * torch.pow(10000.0, -rank.double() / width)
    c, s = torch.cos(angle).float()[:, None], sign * torch.sin(angle).float()[:, None]
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)


def _slots(st):
    """Of every new token: its page and its place in the page."""
    p = st["case"]["page"]
    new = st["q_start"][1:] - st["q_start"][:-1]
    seq = torch.repeat_interleave(torch.arange(new.numel(), device=DEV), new.long(), output_size=st["tokens"])
    index = torch.arange(st["tokens"], device=DEV) - st["q_start"][seq] + st["kv_len"][seq] - new[seq]
    return st["table"][seq, index // p].long(), index % p


def _values(st, name, table):
    """What the pages of `table` hold, in 32 bits: [seqs][kv_heads][tokens][dim]."""
    at = table.clamp(min=0).long()
    codes = st[name + "codes"].view(torch.float8_e4m3fn)[at].float()  # [seqs][pages][heads][..]
    if name == "v":
        codes = codes.transpose(3, 4)
    byte = st[name + "scale"][at].int()
    scale = torch.ldexp(torch.ones(byte.shape, device=DEV), byte - 127)
    return (codes * scale[..., None]).transpose(1, 2).flatten(2, 3)


def _logits(st):
    """Scores of the padded queries [seqs][kv_heads][group * max_new][tokens] (-inf where a query sees nothing),
    and where the padded queries are."""
    case = st["case"]
    hk, hq, dim, m = case["kv_heads"], case["heads"], case["dim"], st["max_new"]
    new = (st["q_start"][1:] - st["q_start"][:-1]).long()
    i = torch.arange(m, device=DEV)
    valid = i[None] < new[:, None]
    row = (st["q_start"][:-1, None].long() + i).clamp(max=st["tokens"] - 1)
    q = st["q"].float()[row]  # [seqs][m][hq][dim]
    q = q.unflatten(2, (hk, hq // hk)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    k = _values(st, "k", st["table"])
    x = (q @ k.transpose(-1, -2)).mul_(1 / math.sqrt(dim)).unflatten(2, (hq // hk, m))
    j = torch.arange(k.shape[2], device=DEV)
    kv = st["kv_len"].long()[:, None, None]
    sees = (j < kv) & valid[..., None]
    if case["causal"]:
        sees = sees & (j <= kv - new[:, None, None] + i[:, None])
    return x.masked_fill_(~sees[:, None, None], -math.inf), row, valid


def _unpad(x, valid):
    """[seqs][kv_heads][group][max_new][...] of the padded queries -> [tokens][heads][...]."""
    x = x.flatten(1, 2).transpose(1, 2)
    return x[valid]


def _lse(st):
    x, _, valid = _logits(st)
    return _unpad(torch.logsumexp(x, -1), valid)


def _attend(st):
    x, _, valid = _logits(st)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    v = _values(st, "v", st["table"])
    # a page's places behind a sequence's end hold whatever they hold: they have no part in the sum
    v = torch.where((torch.arange(v.shape[2], device=DEV) < st["kv_len"][:, None])[:, None, :, None], v, 0.0)
    o = (x.flatten(2, 3) @ v).unflatten(2, x.shape[2:4]) / torch.where(total == 0, 1.0, total)
    lse = top[..., 0] + torch.log(total[..., 0])
    n = st["q_start"][-1:]
    here = torch.arange(st["tokens"], device=DEV) < n
    st["out"][here] = _unpad(o, valid).to(torch.bfloat16)
    st["lse"][here] = _unpad(lse, valid)
    return {"out": st["out"], "lse": st["lse"]}


def _accumulate(st):
    x, row, valid = _logits(st)
    hk, group = x.shape[1:3]
    lse = st["lse"][row].unflatten(2, (hk, group)).permute(0, 2, 3, 1)[..., None]
    x = torch.where(x == -math.inf, x, x.sub_(torch.where(lse == -math.inf, math.inf, lse)))
    weight = x.exp_().sum((2, 3))
    st["scores_out"][:] = st["scores"] + weight[..., :st["max_kv"]]
    return st["scores_out"]


def _write(st):
    case = st["case"]
    page, place = _slots(st)
    codes, scale = _quantise(_turn(st["k"].float(), st["pos"], _sections(case["dim"], case["axes"]), 1.0))
    st["kcodes"][page, :, place], st["kscale"][page, :, place] = codes, scale
    codes, scale = _quantise(st["v"].float())
    st["vcodes"][page, :, :, place], st["vscale"][page, :, place] = codes, scale
    return _held(st)


def _held(st):
    """The pages as the 8-bit values that they hold."""
    return {"kcodes": st["kcodes"].view(torch.float8_e4m3fn), "vcodes": st["vcodes"].view(torch.float8_e4m3fn),
            "kscale": st["kscale"].view(torch.float8_e8m0fnu), "vscale": st["vscale"].view(torch.float8_e8m0fnu)}


def _evict(st):
    case = st["case"]
    p, keep, recent = case["page"], case["keep"], case["recent"]
    kv = st["kv_len"].long()[:, None, None]
    j = torch.arange(st["max_kv"], device=DEV)
    key = torch.where(j < kv - recent, st["scores"], torch.where(j < kv, math.inf, -math.inf))  # the last ones first, none behind the end
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    order = torch.nn.functional.pad(order, (0, max(0, keep - st["max_kv"])), value=st["max_kv"])[..., :keep]
    order = torch.where(order < kv, order, torch.full_like(order, 1 << 30)).sort(-1).values
    live = order < kv
    st["kept"][:] = torch.where(live, order, -1)
    st["len_out"][:] = st["kv_len"].clamp(max=keep)
    st["scores_out"][:] = torch.where(live, st["scores"].gather(2, torch.where(live, order, 0)), 0.0)
    s, h, i = torch.nonzero(live, as_tuple=True)
    at = order[s, h, i]
    page, place = st["table"][s, at // p].long(), at % p
    to, spot = st["dst"][s, i // p].long(), i % p
    st["kcodes"][to, h, spot] = st["kcodes"][page, h, place]
    st["kscale"][to, h, spot] = st["kscale"][page, h, place]
    st["vcodes"][to, h, :, spot] = st["vcodes"][page, h, :, place]
    st["vscale"][to, h, spot] = st["vscale"][page, h, place]
    return dict(_held(st), kept=st["kept"], kv_len=st["len_out"], scores=st["scores_out"])


def run(st):
    if own:
        return _run_own(st)
    op = st["op"]
    if op == "rope":
        case = st["case"]
        st["y"].copy_(_turn(st["x"].float(), st["pos"], _sections(case["dim"], case["axes"]), -1.0 if case["back"] else 1.0))
        return st["y"]
    return {"write": _write, "attend": _attend, "accumulate": _accumulate, "evict": _evict}[op](st)


# ------------------------------------------------------------------ the framework's calls
def _run_own(st):
    import fp8_ring_kv_cache_gb300 as rc

    op, case = st["op"], st["case"]
    if "rope" not in st and "axes" in case:  # a user's program makes its handles once and keeps them
        st["rope"] = rc.RopeAxes(_sections(case["dim"], case["axes"]), base=10000.0)
    if op == "rope":
        rc.rc_rope_axes(st["x"], st["pos"], st["rope"], out=st["y"], inverse=case["back"])
        return st["y"]
    if "cache" not in st:
        st["cache"] = rc.PagedKVCache(st["kcodes"], st["vcodes"], st["kscale"], st["vscale"])
        st["batch"] = rc.PagedBatch(st["table"], st["kv_len"], st.get("q_start"), tokens=st.get("tokens", 0),
                                    max_new=st.get("max_new", 0), max_kv=st["max_kv"])
    cache, batch = st["cache"], st["batch"]
    if op == "write":
        cache.write(batch, st["k"], st["v"], st["pos"], st["rope"])
        return _held(st)
    if op == "attend":
        cache.attend(batch, st["q"], st["out"], lse=st["lse"], causal=case["causal"])
        return {"out": st["out"], "lse": st["lse"]}
    if op == "accumulate":
        cache.accumulate(batch, st["q"], st["lse"], st["scores"], out=st["scores_out"], causal=case["causal"])
        return st["scores_out"]
    cache.evict(batch, st["scores"], keep=case["keep"], recent=case["recent"], dst_table=st["dst"], kept=st["kept"],
                kv_len_out=st["len_out"], scores_out=st["scores_out"])
    return dict(_held(st), kept=st["kept"], kv_len=st["len_out"], scores=st["scores_out"])


# ------------------------------------------------------------------ in 64 bits
_E4M3 = [(-1.0 if c & 128 else 1.0) * (math.nan if c & 127 == 127 else (c & 7) * 2.0 ** -9 if c & 120 == 0 else (8 + (c & 7)) * 2.0 ** ((c >> 3 & 15) - 10))
         for c in range(256)]


def _nearest_codes(y):
    """The E4M3 code nearest to each y, ties to the even code, magnitudes over 448 cut to it."""
    mags = torch.tensor(_E4M3[:127], dtype=torch.float64, device=y.device)
    mid = (mags[1:] + mags[:-1]) / 2
    up = torch.searchsorted(mid, y.abs().contiguous())  # codes whose midpoint above is under |y|
    tie = (up < mid.numel()) & (mid[up.clamp(max=mid.numel() - 1)] == y.abs()) & (up % 2 == 1)
    return ((up + tie.long()) + 128 * torch.signbit(y).long()).to(torch.uint8)


def _exact_turn(x, pos, sections, sign):
    y = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    pair = 0
    for a, width in enumerate(sections):
        for r in range(width):
            angle = sign * pos[a].double() * 10000.0 ** (-r / width)
            z = torch.complex(x[..., 2 * pair].double(), x[..., 2 * pair + 1].double()) * torch.polar(torch.ones_like(angle), angle)[:, None]
            y[..., 2 * pair], y[..., 2 * pair + 1] = z.real, z.imag
            pair += 1
    return y


def _exact_rows(y):
    """Codes and scale bytes of rows in 64 bits."""
    top = y.abs().amax(-1)
    e = torch.zeros_like(top)
    some = top > 0
    e[some] = torch.ceil(torch.log2(top[some] / 448))
    e = torch.where(some & (top > 448 * torch.exp2(e)), e + 1, torch.where(some & (top <= 448 * torch.exp2(e - 1)), e - 1, e))
    e = e.clamp(-124, 7)
    return _nearest_codes(y * torch.exp2(-e)[..., None]), (e + 127).to(torch.uint8)


def _exact_tokens(st, name, s, h, count):
    """The first `count` tokens of sequence s, head h, in 64 bits: [count][dim]."""
    p = st["case"]["page"]
    table = torch.tensor(_E4M3, dtype=torch.float64, device=DEV)
    at = st["table"][s, :-(-count // p)].long()
    rows = table[st[name + "codes"][at, h].long()]
    rows = (rows if name == "k" else rows.transpose(1, 2)) * torch.exp2(st[name + "scale"][at, h].double() - 127)[..., None]
    return rows.reshape(-1, rows.shape[-1])[:count]


def exact(case, seed):
    st = prepare(case, seed)
    op, dim = case["op"], case["dim"]
    if op == "rope":
        return _exact_turn(st["x"], st["pos"], _sections(dim, case["axes"]), -1.0 if case["back"] else 1.0)
    new, kv = _lengths(case)
    hk, p = case["kv_heads"], case["page"]
    if op == "write":
        rows = {"k": _exact_rows(_exact_turn(st["k"], st["pos"], _sections(dim, case["axes"]), 1.0)), "v": _exact_rows(st["v"].double())}
        at = 0
        for s, n in enumerate(new):
            for i in range(n):
                page, place = int(st["table"][s, (kv[s] - n + i) // p]), (kv[s] - n + i) % p
                st["kcodes"][page, :, place], st["kscale"][page, :, place] = rows["k"][0][at], rows["k"][1][at]
                st["vcodes"][page, :, :, place], st["vscale"][page, :, place] = rows["v"][0][at], rows["v"][1][at]
                at += 1
        table = torch.tensor(_E4M3, dtype=torch.float64, device=DEV)
        return {"kcodes": table[st["kcodes"].long()], "vcodes": table[st["vcodes"].long()],
                "kscale": torch.exp2(st["kscale"].double() - 127), "vscale": torch.exp2(st["vscale"].double() - 127)}
    if op == "evict":
        return None  # copies and whole numbers: nothing is computed
    group = case["heads"] // hk
    out = torch.zeros((sum(new), case["heads"], dim), dtype=torch.float64, device=DEV)
    lse = torch.zeros((sum(new), case["heads"]), dtype=torch.float64, device=DEV)
    scores = st["scores"].double() if op == "accumulate" else None
    for s, n in enumerate(new):
        t0 = sum(new[:s])
        j = torch.arange(kv[s], device=DEV)
        hidden = j[None] > kv[s] - n + torch.arange(n, device=DEV)[:, None] if case["causal"] else torch.zeros((n, kv[s]), dtype=torch.bool, device=DEV)
        for h in range(hk):
            k, v = _exact_tokens(st, "k", s, h, kv[s]), _exact_tokens(st, "v", s, h, kv[s])
            for q in range(h * group, (h + 1) * group):
                x = st["q"][t0:t0 + n, q].double() @ k.t() / math.sqrt(dim)
                x.masked_fill_(hidden, -math.inf)
                if op == "attend":
                    lse[t0:t0 + n, q] = torch.logsumexp(x, 1)
                    out[t0:t0 + n, q] = torch.softmax(x, 1) @ v
                else:
                    scores[s, h, :kv[s]] += torch.exp(x - st["lse"][t0:t0 + n, q].double()[:, None]).sum(0)
    return {"out": out, "lse": lse} if op == "attend" else scores

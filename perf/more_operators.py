"""The measured cases of the 4-bit paged cache and of the rotary forms, with their plain forms.

Three operators that serve a paged cache held in 4 bits:

  rope    rotary positions in the forms that models have: neighbouring pairs or
          halves, the whole head or a part of it, one axis or several,
          frequencies scaled for long contexts, a gain; forward, and the gradient
  write   new tokens into the cache's pages: K turned, K and V quantised to
          E2M1 with one scale per token, head and 16 dims
  attend  attention of each sequence's new tokens over its pages

Page layouts, shared by both (P = tokens of a page):
  kcodes [pages][kv_heads][P][head_dim / 2]   two E2M1 codes a byte, the lower dim in the low bits
  vcodes [pages][kv_heads][head_dim][P / 2]   V transposed, the earlier token in the low bits
  kscale, vscale [pages][kv_heads][head_dim / 16][P]   5 bits of exponent and 3 of fraction:
          byte b stands for the fp16 number with the bits b << 7
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the queries of one decode step of 32 sequences, turned as a model with a context stretched by parts does
        {"name": "rope decode step", "op": "rope", "n": 32, "heads": 48, "dim": 128, "first": 0, "rot": 128, "layout": "halves", "axes": 1,
         "scaling": "parts", "dtype": "bf16", "back": False},
        # a prompt, three quarters of each head turned
        {"name": "rope prompt, part of the head", "op": "rope", "n": 6143, "heads": 48, "dim": 128, "first": 0, "rot": 96, "layout": "halves", "axes": 1,
         "scaling": "linear", "dtype": "bf16", "back": False},
        # heads of an odd width of which a small part turns: pieces that no vector load fits
        {"name": "rope narrow part", "op": "rope", "n": 4093, "heads": 16, "dim": 80, "first": 0, "rot": 20, "layout": "halves", "axes": 1,
         "scaling": "none", "dtype": "bf16", "back": False},
        # the gradient through a video clip's turn by (time, height, width), gradients kept in 32 bits
        {"name": "rope clip gradient, halves", "op": "rope", "n": 34065, "heads": 16, "dim": 128, "first": 0, "rot": 128, "layout": "halves", "axes": 3,
         "scaling": "base", "dtype": "f32", "back": True},
        # one decode step of 64 young chat sequences: a token each
        {"name": "write 64 single tokens", "op": "write", "seqs": 64, "new_min": 1, "new_max": 1, "kv_min": 5, "kv_max": 93,
         "kv_heads": 8, "dim": 128, "page": 16, "first": 0, "rot": 128, "layout": "halves", "axes": 1, "scaling": "parts"},
        # the first chunk of the video model into its cache
        {"name": "write chunk", "op": "write", "seqs": 1, "new_min": 757, "new_max": 757, "kv_min": 757, "kv_max": 757,
         "kv_heads": 48, "dim": 128, "page": 64, "first": 0, "rot": 128, "layout": "pairs", "axes": 3, "scaling": "none"},
        # the shortest call: one token of one young sequence, where latency is all
        {"name": "attend one token", "op": "attend", "seqs": 1, "new_min": 1, "new_max": 1, "kv_min": 337, "kv_max": 337,
         "heads": 16, "kv_heads": 2, "dim": 64, "page": 16, "causal": True},
        # a decode step of 32 sequences of very different ages, six query heads to a key head
        {"name": "attend 32 single tokens", "op": "attend", "seqs": 32, "new_min": 1, "new_max": 1, "kv_min": 61, "kv_max": 16381,
         "heads": 48, "kv_heads": 8, "dim": 128, "page": 64, "causal": True},
        # four guessed tokens of each of nine sequences checked at once, four query heads to a key head
        {"name": "attend guessed tokens", "op": "attend", "seqs": 9, "new_min": 4, "new_max": 4, "kv_min": 1021, "kv_max": 12007,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 32, "causal": True},
        # the video model's call: 757 queries see the whole cache of 5,788 tokens
        {"name": "attend chunk", "op": "attend", "seqs": 1, "new_min": 757, "new_max": 757, "kv_min": 5788, "kv_max": 5788,
         "heads": 48, "kv_heads": 48, "dim": 128, "page": 64, "causal": False},
        # chunked prefill of four prompts at different stages
        {"name": "attend prefill", "op": "attend", "seqs": 4, "new_min": 259, "new_max": 2701, "kv_min": 1031, "kv_max": 6143,
         "heads": 48, "kv_heads": 8, "dim": 128, "page": 64, "causal": True},
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


def _form_of(rng, dim):
    rot = dim if rng.random() < 0.5 else 2 * rng.randint(1, dim // 2)
    return {"first": 2 * rng.randint(0, (dim - rot) // 2) if rng.random() < 0.3 else 0, "rot": rot, "layout": rng.choice(["halves", "halves", "pairs"]),
            "axes": rng.randint(1, min(4, rot // 2)), "scaling": rng.choice(["none", "linear", "base", "parts"])}


def _draw(rng):
    op = rng.choice(["rope", "rope", "write", "attend", "attend", "attend"])
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
        return dict({"op": op, "n": _log(rng, 1, 34065), "heads": rng.randint(1, 16), "dim": dim}, **_form_of(rng, dim),
                    dtype=rng.choice(["bf16", "f32"]), back=rng.random() < 0.5)
    dim, page, kv_heads = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128]), rng.choice([1, 2, 3, 4, 8])
    shape = rng.choice(["single", "few", "chunk"])
    if op == "write":
        seqs, new = (_log(rng, 1, 64), 1) if shape == "single" else (rng.randint(1, 8), rng.randint(2, 33)) if shape == "few" else (rng.randint(1, 3), _log(rng, 40, 1500))
        kv = new + rng.randint(0, 100)
        return dict({"op": op, "seqs": seqs, "new_min": rng.randint(1, new), "new_max": new, "kv_min": rng.randint(new, kv), "kv_max": kv,
                     "kv_heads": kv_heads, "dim": dim, "page": page}, **_form_of(rng, dim))
    if shape == "single":
        seqs, new, kv = _log(rng, 1, 32), 1, _log(rng, 1, 16381)
    elif shape == "few":
        seqs, new, kv = rng.randint(1, 8), rng.randint(2, 33), _log(rng, 40, 16381)
    else:
        seqs, new, kv = rng.randint(1, 3), _log(rng, 40, 1500), _log(rng, 1501, 6143)
    return {"op": op, "seqs": seqs, "new_min": rng.randint(1, new), "new_max": new, "kv_min": rng.randint(min(new, kv), kv), "kv_max": kv,
            "heads": kv_heads * rng.choice([1, 1, 2, 4, 6, 8]), "kv_heads": kv_heads, "dim": dim, "page": page, "causal": rng.random() < 0.7}


# ------------------------------------------------------------------ sizes of a case
def _spread(lo, hi, seqs):
    """`seqs` lengths from lo to hi, the longest first, the shortest second, and so on inwards."""
    v = [hi - (hi - lo) * i // max(1, seqs - 1) for i in range(seqs)]
    return [v[i // 2] if i % 2 == 0 else v[seqs - 1 - i // 2] for i in range(seqs)]


def _lengths(case):
    """Per sequence: new tokens, cached tokens (the new ones included)."""
    kv = _spread(case["kv_min"], case["kv_max"], case["seqs"])
    new = _spread(case["new_min"], case["new_max"], case["seqs"])
    return [min(a, b) for a, b in zip(new, kv)], kv


def _sections(case):
    """Pairs of each axis: as even as they go, the first axis (time) with what is left over."""
    pairs, axes = case["rot"] // 2, case["axes"]
    even = pairs // axes
    return [pairs - even * (axes - 1)] + [even] * (axes - 1)


# what each kind of scaling is used with: the context that the model was trained for, how far it is stretched, the turns
# between which a frequency goes over from stretched to not, and the gain that comes with it
_SCALING = {"none": {"factor": 1.0, "context": 0, "low": 1.0, "high": 32.0, "gain": 1.0},
            "linear": {"factor": 4.0, "context": 0, "low": 1.0, "high": 32.0, "gain": 1.0},
            "base": {"factor": 8.0, "context": 0, "low": 1.0, "high": 32.0, "gain": 1.0},
            "parts": {"factor": 16.0, "context": 4096, "low": 1.0, "high": 32.0, "gain": 1.25}}


def work(case):
    op, dim = case["op"], case["dim"]
    if op == "rope":
        size = 4 if case["dtype"] == "f32" else 2
        values = case["n"] * case["heads"] * dim
        return {"bytes": 2 * size * values + 4 * case["axes"] * case["n"], "flops": 3 * case["n"] * case["heads"] * case["rot"]}
    new, kv = _lengths(case)
    hk = case["kv_heads"]
    token = hk * (dim // 2 + dim // 16)  # one token's codes and scales, K or V, of all heads
    if op == "write":
        return {"bytes": sum(new) * (2 * 2 * hk * dim + 2 * token + 4 * case["axes"]), "flops": 7 * sum(new) * hk * dim}
    t, hq = sum(new), case["heads"]
    pairs = sum(n * k - (n * (n - 1) // 2 if case["causal"] else 0) for n, k in zip(new, kv)) * hq
    return {"bytes": 2 * sum(kv) * token + t * hq * (2 * 2 * dim + 4), "flops": pairs * 4 * dim}


# ------------------------------------------------------------------ inputs
def _scale_values(device, dtype):
    """What the scale bytes 0 .. 226 stand for (226: 10240, the largest that a row gets)."""
    return (torch.arange(227, device=device).to(torch.int16) * 128).view(torch.float16).to(dtype)


def _quantise(x):
    """E2M1 codes and scale bytes of rows x [..., dim], blocks of 16: the smallest scale s with max|x| <= 6 s, the nearest
    code to x / s (ties to the even one), found without a division."""
    y = x.unflatten(-1, (-1, 16))
    scales = _scale_values(x.device, x.dtype)
    byte = torch.searchsorted(6 * scales, y.abs().amax(-1)).clamp(max=226)
    s, a = scales[byte][..., None], y.abs()
    # the middles between neighbouring codes: one that is met goes to the even code
    code = sum(((a > m * s) if i % 2 == 0 else (a >= m * s)).to(torch.uint8) for i, m in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)))
    code = torch.where(s == 0, torch.zeros_like(code), code)
    return (code + 8 * torch.signbit(y).to(torch.uint8)).flatten(-2), byte.to(torch.uint8)


def _pack(codes):
    """Neighbouring codes of the last dimension in a byte, the first in the low bits."""
    return codes[..., 0::2] | codes[..., 1::2] << 4


def _pool(case, g, kv):
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
    codes = torch.empty((2, pages * hk * p * dim // 2), dtype=torch.uint8, device=DEV)
    scale = torch.empty((2, pages * hk * p * dim // 16), dtype=torch.uint8, device=DEV)
    pool["codes"], pool["scale"] = codes, scale
    shapes = {"k": (pages, hk, p, dim // 2), "v": (pages, hk, dim, p // 2)}
    for i, name in enumerate("kv"):
        pool[name + "codes"], pool[name + "scale"] = codes[i].view(shapes[name]), scale[i].view(pages, hk, dim // 16, p)
        # every channel has a spread of its own (a few of them large), every token a size of its own
        channel = torch.exp(0.5 * torch.randn((1, hk, 1, dim), generator=g, device=DEV))
        for a in range(0, pages, 512):
            n = min(512, pages - a)
            x = torch.randn((n, hk, p, dim), generator=g, device=DEV) * channel * torch.exp(0.3 * torch.randn((n, hk, p, 1), generator=g, device=DEV))
            c, b = _quantise(x)
            pool[name + "codes"][a:a + n] = _pack(c if name == "k" else c.transpose(2, 3))
            pool[name + "scale"][a:a + n] = b.transpose(2, 3)
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
    st.update(_pool(case, g, kv))
    st["q_start"] = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device=DEV)
    st["tokens"], st["max_new"], st["max_kv"] = t, max(new), max(kv)
    if op == "write":
        for name in "kv":
            x = torch.randn((t, hk, dim), generator=g, device=DEV) * torch.exp(0.5 * torch.randn((1, hk, dim), generator=g, device=DEV))
            st[name] = x.to(torch.bfloat16)
        st["pos"] = _positions(case, t, g)
        # what a byte of codes stands for, two bf16 numbers, and a scale byte, an fp16 one
        st["pairs"] = _byte_values(torch.bfloat16).view(torch.int32).flatten()
        return st
    st["q"] = torch.randn((t, case["heads"], dim), generator=g, device=DEV).to(torch.bfloat16)
    st["out"] = torch.zeros((t, case["heads"], dim), dtype=torch.bfloat16, device=DEV)
    st["lse"] = torch.zeros((t, case["heads"]), device=DEV)
    return st


def _positions(case, n, g):
    """[axes][n]: the first axis counts far into a session, the others run over a picture."""
    at = torch.arange(n, device=DEV)
    pos = [at + 60000] + [torch.randint(0, 90, (n,), generator=g, device=DEV) for _ in range(case["axes"] - 1)]
    return torch.stack(pos).to(torch.int32)


# ------------------------------------------------------------------ the plain forms
def _byte_values(dtype):
    """[256][2]: the two values of a byte of codes."""
    mags = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
    values = torch.cat([mags, -mags]).to(dtype)
    b = torch.arange(256, device=DEV)
    return torch.stack([values[b & 15], values[b >> 4]], -1)


def _frequencies(case):
    """Of each pair: its axis and its frequency, in 64 bits."""
    width = torch.tensor(_sections(case), device=DEV)
    axis = torch.repeat_interleave(torch.arange(len(width), device=DEV), width)
    rank = torch.arange(axis.numel(), device=DEV) - (torch.cumsum(width, 0) - width)[axis]
    w, s = width[axis].double(), _SCALING[case["scaling"]]
    base = torch.full_like(w, 10000.0)
    if case["scaling"] == "base":
        base = torch.where(w > 1, base * s["factor"] ** (w / (w - 1).clamp(min=1)), base)
    theta = torch.pow(base, -rank / w)
    if case["scaling"] == "linear":
        theta = theta / s["factor"]
    if case["scaling"] == "parts":
        keep = ((s["context"] * theta / (2 * math.pi) - s["low"]) / (s["high"] - s["low"])).clamp(0, 1)
        theta = theta * (keep + (1 - keep) / s["factor"])
    return axis, theta


def _turn(x, case, pos, sign):
    """The turned part of x [n][heads][dim] by sign * position * frequency, times the gain; the rest as it is."""
    axis, theta = _frequencies(case)
    angle = pos[axis].t().double() * theta
    gain = _SCALING[case["scaling"]]["gain"]
    c, s = (gain * torch.cos(angle)).to(x.dtype)[:, None], (sign * gain * torch.sin(angle)).to(x.dtype)[:, None]
    first, rot = case["first"], case["rot"]
    part = x[..., first:first + rot]
    if case["layout"] == "halves":
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        turned = torch.cat([a * c - b * s, a * s + b * c], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    return torch.cat([x[..., :first], turned, x[..., first + rot:]], -1)


def _slots(st):
    """Of every new token: its page and its place in the page."""
    p = st["case"]["page"]
    new = st["q_start"][1:] - st["q_start"][:-1]
    seq = torch.repeat_interleave(torch.arange(new.numel(), device=DEV), new.long(), output_size=st["tokens"])
    index = torch.arange(st["tokens"], device=DEV) - st["q_start"][seq] + st["kv_len"][seq] - new[seq]
    return st["table"][seq, index // p].long(), index % p


def _write(st):
    case = st["case"]
    page, place = _slots(st)
    # (in 64 bits: a value next to the middle between two codes may go to either in 32)
    codes, scale = _quantise(_turn(st["k"].double(), case, st["pos"], 1.0))
    st["kcodes"][page, :, place], st["kscale"][page, :, :, place] = _pack(codes), scale
    codes, scale = _quantise(st["v"].double())
    st["vscale"][page, :, :, place] = scale
    # (two tokens share a byte of V)
    tokens = torch.stack([st["vcodes"] & 15, st["vcodes"] >> 4], -1).flatten(-2)
    tokens[page, :, :, place] = codes
    st["vcodes"][:] = _pack(tokens)
    return _held(st)


def _held(st):
    """What the pages hold, as values: of the codes, then of the scales."""
    values = st["pairs"].index_select(0, st["codes"].flatten().int()).view(torch.bfloat16)
    return {"codes": values, "scale": (st["scale"].to(torch.int16) * 128).view(torch.float16)}


def _values(st, name):
    """What the pages of the table hold, in 32 bits: [seqs][kv_heads][tokens][dim]."""
    at = st["table"].clamp(min=0).long()
    values = _byte_values(torch.float32)[st[name + "codes"][at].int()].flatten(-2)  # [seqs][pages][heads][..]
    if name == "v":
        values = values.transpose(3, 4)
    scale = (st[name + "scale"][at].to(torch.int16) * 128).view(torch.float16).float().transpose(3, 4)
    return (values.unflatten(-1, (-1, 16)) * scale[..., None]).flatten(-2).transpose(1, 2).flatten(2, 3)


def _attend(st):
    case = st["case"]
    hk, hq, dim, m = case["kv_heads"], case["heads"], case["dim"], st["max_new"]
    new = (st["q_start"][1:] - st["q_start"][:-1]).long()
    i = torch.arange(m, device=DEV)
    valid = i[None] < new[:, None]
    row = (st["q_start"][:-1, None].long() + i).clamp(max=st["tokens"] - 1)
    q = st["q"].float()[row].unflatten(2, (hk, hq // hk)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # padded queries
    k = _values(st, "k")
    x = (q @ k.transpose(-1, -2)).mul_(1 / math.sqrt(dim)).unflatten(2, (hq // hk, m))
    j = torch.arange(k.shape[2], device=DEV)
    kv = st["kv_len"].long()[:, None, None]
    sees = (j < kv) & valid[..., None]
    if case["causal"]:
        sees = sees & (j <= kv - new[:, None, None] + i[:, None])
    x = x.masked_fill_(~sees[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    # a page's places behind a sequence's end hold whatever they hold: they have no part in the sum
    v = torch.where((j < st["kv_len"][:, None])[:, None, :, None], _values(st, "v"), 0.0)
    o = (x.flatten(2, 3) @ v).unflatten(2, x.shape[2:4]) / torch.where(total == 0, 1.0, total)
    lse = top[..., 0] + torch.log(total[..., 0])
    st["out"][:] = o.flatten(1, 2).transpose(1, 2)[valid].to(torch.bfloat16)
    st["lse"][:] = lse.flatten(1, 2).transpose(1, 2)[valid]
    return {"out": st["out"], "lse": st["lse"]}


def run(st):
    if own:
        return _run_own(st)
    case = st["case"]
    if st["op"] == "rope":
        st["y"].copy_(_turn(st["x"].float(), case, st["pos"], -1.0 if case["back"] else 1.0))
        return st["y"]
    return _write(st) if st["op"] == "write" else _attend(st)


# ------------------------------------------------------------------ the framework's calls
def _run_own(st):
    import fp8_ring_kv_cache_gb300 as rc

    op, case = st["op"], st["case"]
    if "form" not in st and "rot" in case:  # a user's program makes its handles once and keeps them
        s = _SCALING[case["scaling"]]
        st["form"] = rc.RopeForm(case["dim"], sections=_sections(case), first=case["first"], layout=case["layout"], base=10000.0,
                                 scaling=None if case["scaling"] == "none" else case["scaling"], factor=s["factor"],
                                 context=s["context"], low=s["low"], high=s["high"], gain=s["gain"])
    if op == "rope":
        rc.rc_rope_turn(st["x"], st["pos"], st["form"], out=st["y"], back=case["back"])
        return st["y"]
    if "cache" not in st:
        st["cache"] = rc.PagedKVCache4(st["kcodes"], st["vcodes"], st["kscale"], st["vscale"])
        st["batch"] = rc.PagedBatch(st["table"], st["kv_len"], st["q_start"], tokens=st["tokens"], max_new=st["max_new"], max_kv=st["max_kv"])
    if op == "write":
        st["cache"].write(st["batch"], st["k"], st["v"], st["pos"], st["form"])
        return _held(st)
    st["cache"].attend(st["batch"], st["q"], st["out"], lse=st["lse"], causal=case["causal"])
    return {"out": st["out"], "lse": st["lse"]}


# ------------------------------------------------------------------ in 64 bits
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]
_SCALES = [b * 2.0 ** -17 if b < 8 else (8 + b % 8) * 2.0 ** (b // 8 - 18) for b in range(256)]


def _exact_turn(x, case, pos, sign):
    """Pair by pair, as complex numbers."""
    y = x.double().clone()
    s, half, pair = _SCALING[case["scaling"]], case["rot"] // 2, 0
    for a, width in enumerate(_sections(case)):
        base = 10000.0 * s["factor"] ** (width / (width - 1)) if case["scaling"] == "base" and width > 1 else 10000.0
        for r in range(width):
            theta = base ** (-r / width)
            if case["scaling"] == "linear":
                theta /= s["factor"]
            elif case["scaling"] == "parts":
                turns = s["context"] * theta / (2 * math.pi)
                keep = min(1.0, max(0.0, (turns - s["low"]) / (s["high"] - s["low"])))
                theta = theta * keep + theta / s["factor"] * (1 - keep)
            i, j = (pair, pair + half) if case["layout"] == "halves" else (2 * pair, 2 * pair + 1)
            i, j = i + case["first"], j + case["first"]
            angle = sign * pos[a].double() * theta
            z = torch.complex(x[..., i].double(), x[..., j].double()) * torch.polar(torch.full_like(angle, s["gain"]), angle)[:, None]
            y[..., i], y[..., j] = z.real, z.imag
            pair += 1
    return y


def _exact_rows(y):
    """What the codes and the scales of rows y [..., dim] stand for, by distances to every code."""
    blocks = y.unflatten(-1, (-1, 16))
    top = blocks.abs().amax(-1)
    # 8 .. 15 eighths of a power of two from 2^-14 on, eighths of 2^-14 below
    _, e = torch.frexp((top / 6).clamp(2.0 ** -14, 2.0 ** 14))
    power = torch.tensor([2.0 ** (k - 17) for k in range(29)], dtype=torch.float64, device=y.device)[e.long() + 13]
    scale = torch.ceil(top / 6 / power) * power
    scale = torch.where(6 * (scale - power) >= top, scale - power, torch.where(6 * scale < top, scale + power, scale)).clamp(max=10240.0)
    q = blocks.abs() / torch.where(scale == 0, 1.0, scale)[..., None]
    mags = torch.tensor(_E2M1[:8], dtype=torch.float64, device=y.device)
    order = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7], device=y.device)  # the first of the nearest: an even one of two
    nearest = order[(q[..., None] - mags[order]).abs().argmin(-1)]
    return torch.copysign(mags[nearest], blocks).flatten(-2), scale


def _exact_tokens(st, name, s, h, count):
    """The first `count` tokens of sequence s, head h, in 64 bits: [count][dim]."""
    p, dim = st["case"]["page"], st["case"]["dim"]
    table = torch.tensor(_E2M1, dtype=torch.float64, device=DEV)
    at = st["table"][s, :-(-count // p)].long()
    codes = st[name + "codes"][at, h].long()
    rows = torch.empty(codes.shape[:-1] + (2 * codes.shape[-1],), dtype=torch.float64, device=DEV)
    rows[..., 0::2], rows[..., 1::2] = table[codes % 16], table[codes // 16]
    if name == "v":
        rows = rows.transpose(1, 2)
    byte = st[name + "scale"][at, h].long()
    scale = torch.tensor(_SCALES, dtype=torch.float64, device=DEV)[byte]
    return (rows * scale.transpose(1, 2).repeat_interleave(16, -1)).reshape(-1, dim)[:count]


def exact(case, seed):
    st = prepare(case, seed)
    op, dim = case["op"], case["dim"]
    if op == "rope":
        return _exact_turn(st["x"], case, st["pos"], -1.0 if case["back"] else 1.0)
    new, kv = _lengths(case)
    hk, p = case["kv_heads"], case["page"]
    if op == "write":
        rows = {"k": _exact_rows(_exact_turn(st["k"], case, st["pos"], 1.0)), "v": _exact_rows(st["v"].double())}
        table = torch.tensor(_E2M1, dtype=torch.float64, device=DEV)
        held = []
        for name in "kv":
            codes = st[name + "codes"].long()
            values = torch.stack([table[codes % 16], table[codes // 16]], -1).flatten(-2)
            byte = st[name + "scale"].long()
            scale = torch.tensor(_SCALES, dtype=torch.float64, device=DEV)[byte]
            at = 0
            for s, n in enumerate(new):
                for i in range(n):
                    page, place = int(st["table"][s, (kv[s] - n + i) // p]), (kv[s] - n + i) % p
                    if name == "k":
                        values[page, :, place] = rows[name][0][at]
                    else:
                        values[page, :, :, place] = rows[name][0][at]
                    scale[page, :, :, place] = rows[name][1][at]
                    at += 1
            held.append((values.flatten(), scale.flatten()))
        return {"codes": torch.cat([v for v, _ in held]), "scale": torch.stack([s for _, s in held])}
    group = case["heads"] // hk
    out = torch.zeros((sum(new), case["heads"], dim), dtype=torch.float64, device=DEV)
    lse = torch.zeros((sum(new), case["heads"]), dtype=torch.float64, device=DEV)
    for s, n in enumerate(new):
        t0 = sum(new[:s])
        j = torch.arange(kv[s], device=DEV)
        hidden = j[None] > kv[s] - n + torch.arange(n, device=DEV)[:, None] if case["causal"] else torch.zeros((n, kv[s]), dtype=torch.bool, device=DEV)
        for h in range(hk):
            k, v = _exact_tokens(st, "k", s, h, kv[s]), _exact_tokens(st, "v", s, h, kv[s])
            for q in range(h * group, (h + 1) * group):
                x = st["q"][t0:t0 + n, q].double() @ k.t() / math.sqrt(dim)
                x.masked_fill_(hidden, -math.inf)
                lse[t0:t0 + n, q] = torch.logsumexp(x, 1)
                out[t0:t0 + n, q] = torch.softmax(x, 1) @ v
    return {"out": out, "lse": lse}

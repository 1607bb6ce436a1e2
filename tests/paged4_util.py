"""The rotary forms and the 4-bit paged cache from their definitions, in 64 bits on the CPU, for the tests."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
MIDDLES = (E2M1[1:] + E2M1[:-1]) / 2
# what each scale byte stands for: 5 bits of exponent (bias 15), 3 of fraction, subnormals below 8; NaN from 248 on
SCALES = np.array([b * 2.0 ** -17 if b < 8 else (8 + b % 8) * 2.0 ** (b // 8 - 18) if b < 248 else np.nan for b in range(256)])
TOP = 226


def frequencies(sections, base=10000.0, shared=False, scaling=None, factor=1.0, context=0.0, low=1.0, high=32.0):
    """(axis, frequency) of every pair."""
    out, pairs = [], sum(sections)
    for a, width in enumerate(sections):
        for r in range(width):
            w, k = (pairs, len(out)) if shared else (width, r)
            b = base * factor ** (w / (w - 1)) if scaling == "base" and w > 1 else base
            theta = b ** (-k / w)
            if scaling == "linear":
                theta /= factor
            elif scaling == "parts":
                turns = context * theta / (2 * np.pi)
                keep = min(1.0, max(0.0, (turns - low) / (high - low)))
                theta *= keep + (1 - keep) / factor
            out.append((a, theta))
    return out


def pair_of(first, dims, layout, i):
    return (first + i, first + i + dims // 2) if layout == "halves" else (first + 2 * i, first + 2 * i + 1)


def turn(x, pos, sections, first=0, layout="pairs", gain=1.0, sign=1.0, **kw):
    """x [n][heads][dim], pos [axes][n] -> float64; and gain (|a| + |b|) of each value's pair (0 where nothing turns: outside
    the part, at position 0)."""
    x = np.asarray(x, np.float64)
    y, reach, dims = x.copy(), np.zeros_like(x), 2 * sum(sections)
    for i, (a, theta) in enumerate(frequencies(sections, **kw)):
        p, q = pair_of(first, dims, layout, i)
        angle = sign * pos[a].astype(np.float64) * theta
        c, s = gain * np.cos(angle)[:, None], gain * np.sin(angle)[:, None]
        y[..., p], y[..., q] = x[..., p] * c - x[..., q] * s, x[..., p] * s + x[..., q] * c
        reach[..., p] = reach[..., q] = gain * (np.abs(x[..., p]) + np.abs(x[..., q])) * (pos[a] != 0)[:, None]
    return y, reach


def quantise(x):
    """Codes [..., dim] (0 .. 15) and scale bytes [..., dim / 16] of rows in float64."""
    x = np.asarray(x, np.float64)
    fine = np.isfinite(x).all(-1)
    xx = np.where(fine[..., None], x, 0.0).reshape(x.shape[:-1] + (-1, 16))
    byte = np.minimum(np.searchsorted(6 * SCALES[:TOP + 1], np.abs(xx).max(-1)), TOP)
    s = SCALES[byte][..., None]
    a = np.abs(xx)
    code = np.zeros(xx.shape, np.int64)
    for i, m in enumerate(MIDDLES):  # one that is met goes to the even code
        code += (a > m * s) if i % 2 == 0 else (a >= m * s)
    code = np.where(s == 0, 0, code) + 8 * np.signbit(xx)
    code = np.where(fine[..., None, None], code, 0).reshape(x.shape)
    return code.astype(np.uint8), np.where(fine[..., None], byte, 255).astype(np.uint8)


def near_border(x, err):
    """Of rows x [..., dim]: whether a value within err of x can have another code or scale."""
    xx, rr = x.reshape(x.shape[:-1] + (-1, 16)), err.reshape(x.shape[:-1] + (-1, 16))
    a, top = np.abs(xx), np.abs(xx).max(-1)
    scale = np.searchsorted(6 * SCALES[:TOP + 1], (a - rr).max(-1)) != np.searchsorted(6 * SCALES[:TOP + 1], (a + rr).max(-1))
    s = SCALES[np.minimum(np.searchsorted(6 * SCALES[:TOP + 1], top), TOP)][..., None]
    code = np.zeros(xx.shape, bool)
    for m in MIDDLES:
        code |= np.abs(a - m * s) <= rr
    code |= a <= rr  # the sign
    return (code & (rr > 0)).reshape(x.shape), np.broadcast_to(scale[..., None], xx.shape).reshape(x.shape)


def pack(codes):
    return (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)


def unpack(b):
    return np.stack([b & 15, b >> 4], -1).reshape(b.shape[:-1] + (-1,))


def values(codes):
    return np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7]


def put(pool, name, page, h, place, codes, scale):
    """One row's codes and scale bytes into a page."""
    if name == "k":
        pool["kcodes"][page, h, place] = pack(codes)
    else:
        low = place % 2 == 0
        old = pool["vcodes"][page, h, :, place // 2]
        pool["vcodes"][page, h, :, place // 2] = (old & 0xf0 | codes) if low else (old & 0x0f | codes << 4)
    pool[name + "scale"][page, h, :, place] = scale


def tokens_of(pool, name, table_row, h, count):
    """The first `count` cached tokens of a sequence, head h: float64 [count][dim]."""
    scale = pool[name + "scale"]
    p, d = scale.shape[3], 16 * scale.shape[2]
    rows = []
    for i in range(-(-count // p)):
        page = table_row[i]
        v = values(unpack(pool[name + "codes"][page, h]))
        s = np.repeat(SCALES[scale[page, h]], 16, 0)  # [dim][P]
        rows.append((v if name == "k" else v.T) * s.T)
    return np.concatenate(rows)[:count] if rows else np.zeros((0, d))


def attend_head(q, k, v, n, causal):
    """q [n][dim] of one head, its sequence's k, v [kv][dim]: (out, lse, weights, scores' reach)."""
    kv = len(k)
    with np.errstate(invalid="ignore", over="ignore"):
        x = q @ k.T / np.sqrt(q.shape[1])
        big = (np.abs(q) @ np.abs(np.nan_to_num(k)).T / np.sqrt(q.shape[1])).max(initial=0.0)
    see = np.ones((n, kv), bool)
    if causal:
        see = np.arange(kv)[None] <= kv - n + np.arange(n)[:, None]
    out, lse, w = np.zeros((n, v.shape[1])), np.full(n, -np.inf), np.zeros((n, kv))
    for i in range(n):
        if not see[i].any():
            continue
        xs = x[i][see[i]]
        m = xs.max()
        with np.errstate(invalid="ignore"):
            e = np.exp(xs - m)
            lse[i] = m + np.log(e.sum())
            w[i, see[i]] = e / e.sum()
            out[i] = w[i, see[i]] @ v[see[i]]
    return out, lse, w, big


def make(seqs, kv_heads, dim, page, rng, spare=2, spread=1.0):
    """A pool for sequences [(new, kv), ...] with scattered pages, and the metadata, as numpy arrays."""
    need = [-(-kv // page) for _, kv in seqs]
    pages = sum(need) + spare
    ids = rng.permutation(pages).astype(np.int32)
    table = np.full((len(seqs), max(max(need), 1)), -1, np.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = ids[at:at + n]
        at += n
    pool = {}
    for name in "kv":
        x = rng.standard_normal((pages, kv_heads, page, dim)) * np.exp(spread * rng.standard_normal((pages, kv_heads, page, 1)))
        codes, scale = quantise(x)
        pool[name + "codes"] = pack(codes) if name == "k" else pack(codes.transpose(0, 1, 3, 2))
        pool[name + "scale"] = np.ascontiguousarray(scale.transpose(0, 1, 3, 2))
    new = [n for n, _ in seqs]
    meta = {"table": table, "kv_len": np.array([kv for _, kv in seqs], np.int32),
            "q_start": np.concatenate([[0], np.cumsum(new)]).astype(np.int32)}
    return pool, meta

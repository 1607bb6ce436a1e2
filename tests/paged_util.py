"""The paged-cache operators from their definitions, in 64 bits on the CPU, for the tests."""
import numpy as np

# the value of every E4M3 code
E4M3 = np.array([(-1.0 if c & 128 else 1.0) * (np.nan if c & 127 == 127 else (c & 7) * 2.0 ** -9 if c & 120 == 0
                                               else (8 + (c & 7)) * 2.0 ** ((c >> 3 & 15) - 10)) for c in range(256)])
MAGS = E4M3[:127]


def turn(x, pos, sections, base=10000.0, shared=False, sign=1.0):
    """x [n][heads][dim], pos [axes][n] -> float64."""
    x = np.asarray(x, np.float64)
    y = np.empty_like(x)
    i = 0
    for a, w in enumerate(sections):
        for r in range(w):
            theta = base ** (-2.0 * i / x.shape[2]) if shared else base ** (-r / w)
            z = (x[..., 2 * i] + 1j * x[..., 2 * i + 1]) * np.exp(1j * sign * pos[a].astype(np.float64) * theta)[:, None]
            y[..., 2 * i], y[..., 2 * i + 1] = z.real, z.imag
            i += 1
    return y


def nearest_code(y):
    """E4M3 code nearest to each y (ties to even, cut at 448)."""
    y = np.asarray(y, np.float64)
    a = np.minimum(np.abs(y), 448.0)
    up = np.clip(np.searchsorted(MAGS, a), 0, 126)
    lo = np.maximum(up - 1, 0)
    dl, du = a - MAGS[lo], MAGS[up] - a
    code = np.where((dl < du) | ((dl == du) & (lo % 2 == 0)), lo, up)
    return (code + 128 * np.signbit(y)).astype(np.uint8)


def quantise(x):
    """Codes and scale bytes of rows x [..., dim] in float64."""
    x = np.asarray(x, np.float64)
    fine = np.isfinite(x).all(-1)
    xx = np.where(fine[..., None], x, 0.0)
    amax = np.abs(xx).max(-1)
    e = np.zeros(amax.shape, np.int64)
    some = amax > 0
    e[some] = np.ceil(np.log2(amax[some] / 448.0)).astype(np.int64)
    e = np.where(some & (amax > 448.0 * 2.0 ** e), e + 1, e)
    e = np.where(some & (amax <= 448.0 * 2.0 ** (e - 1.0)), e - 1, e)
    e = np.clip(e, -124, 7)
    codes = nearest_code(xx * 2.0 ** -e[..., None].astype(np.float64))
    return np.where(fine[..., None], codes, 0).astype(np.uint8), np.where(fine, e + 127, 255).astype(np.uint8)


def scale_value(b):
    b = np.asarray(b)
    return np.where(b == 255, np.nan, 2.0 ** (b.astype(np.float64) - 127.0))


def tokens_of(pool, name, table_row, h, count):
    """The first `count` cached tokens of a sequence, head h: float64 [count][dim]."""
    codes, scale = pool[name + "codes"], pool[name + "scale"]
    p = scale.shape[2]
    rows = []
    for i in range(-(-count // p)):
        page = table_row[i]
        c = E4M3[codes[page, h]]
        rows.append((c if name == "k" else c.T) * scale_value(scale[page, h])[:, None])
    d = codes.shape[3] if name == "k" else codes.shape[2]
    return np.concatenate(rows)[:count] if rows else np.zeros((0, d))


def logits(pool, meta, q, s, h, head, causal):
    """Scores [n][kv] of sequence s for one query head, -inf where nothing is seen."""
    q0, q1, kv = meta["q_start"][s], meta["q_start"][s + 1], meta["kv_len"][s]
    n = q1 - q0
    k = tokens_of(pool, "k", meta["table"][s], h, kv)
    with np.errstate(invalid="ignore"):
        x = np.asarray(q[q0:q1, head], np.float64) @ k.T / np.sqrt(q.shape[2])
    if causal:
        x = np.where(np.arange(kv)[None] <= kv - n + np.arange(n)[:, None], x, -np.inf)
    return x


def reach(pool, meta, q, s, h, head):
    """The largest sum of |q_d k_d| / sqrt(dim) of a query and a key: what the rounding of a score is relative to."""
    q0, q1, kv = meta["q_start"][s], meta["q_start"][s + 1], meta["kv_len"][s]
    k = tokens_of(pool, "k", meta["table"][s], h, kv)
    x = np.abs(np.asarray(q[q0:q1, head], np.float64)) @ np.abs(np.nan_to_num(k)).T / np.sqrt(q.shape[2])
    return x.max(initial=0.0)


def attend(pool, meta, q, causal):
    """(out, lse) float64; rows outside every sequence are NaN-free zeros marked in `touched`."""
    t, hq, d = q.shape
    hk = pool["kcodes"].shape[1]
    out, lse, touched = np.zeros((t, hq, d)), np.zeros((t, hq)), np.zeros(t, bool)
    for s in range(len(meta["kv_len"])):
        q0, q1, kv = meta["q_start"][s], meta["q_start"][s + 1], meta["kv_len"][s]
        touched[q0:q1] = True
        for h in range(hk):
            v = tokens_of(pool, "v", meta["table"][s], h, kv)
            for head in range(h * hq // hk, (h + 1) * hq // hk):
                x = logits(pool, meta, q, s, h, head, causal)
                for i in range(q1 - q0):
                    see = x[i] != -np.inf
                    if not see.any():
                        lse[q0 + i, head] = -np.inf
                        continue
                    xs = x[i][see]
                    m = xs.max()
                    w = np.exp(xs - m)
                    lse[q0 + i, head] = m + np.log(w.sum())
                    out[q0 + i, head] = (w / w.sum()) @ v[see]
    return out, lse, touched


def accumulate(pool, meta, q, lse, scores, causal):
    out = np.array(scores, np.float64)
    hk, hq = pool["kcodes"].shape[1], q.shape[1]
    for s in range(len(meta["kv_len"])):
        q0, q1, kv = meta["q_start"][s], meta["q_start"][s + 1], meta["kv_len"][s]
        for h in range(hk):
            for head in range(h * hq // hk, (h + 1) * hq // hk):
                x = logits(pool, meta, q, s, h, head, causal)
                z = np.asarray(lse[q0:q1, head], np.float64)[:, None]
                with np.errstate(invalid="ignore"):
                    w = np.where((x == -np.inf) | (z == -np.inf), 0.0, np.exp(x - z))
                out[s, h, :kv] += w.sum(0)
    return out


def evict(scores, kv, keep, recent):
    """The kept indices of one row of scores, ascending."""
    if kv <= keep:
        return list(range(kv))
    recent = min(recent, kv)
    cand = kv - recent
    key = [(0 if scores[j] != scores[j] else 1, -scores[j] if scores[j] == scores[j] else 0.0, j) for j in range(cand)]
    return sorted(j for _, _, j in sorted(key)[:keep - recent]) + list(range(cand, kv))


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
        pool[name + "codes"] = codes if name == "k" else np.ascontiguousarray(codes.transpose(0, 1, 3, 2))
        pool[name + "scale"] = scale
    new = [n for n, _ in seqs]
    meta = {"table": table, "kv_len": np.array([kv for _, kv in seqs], np.int32),
            "q_start": np.concatenate([[0], np.cumsum(new)]).astype(np.int32)}
    return pool, meta

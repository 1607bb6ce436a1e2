"""The rotary forms and the 4-bit paged cache on the GPU, against their definitions in 64 bits (tests/paged4_util.py).

Tolerances, from the roundings that the operators make (half a step: bf16 2^-8 of the value, fp16 2^-11, fp32 2^-24):
  turn    fp32 products of magnitude r = gain (|a| + |b|): cos, sin and the position's fraction of a turn are each within
          3 * 2^-24 + 2^-32 * 2 pi, the gain, the two products and their sum add 4 * 2^-24: 2^-20 r covers them; a bf16
          result is rounded once more.  What does not turn is equal bit for bit.
  write   codes and scales are those of the exact turn, which the kernel knows to 2^-25 r and the definition here to
          2^-52 |pos| r: equal except where that reaches another code or scale.  V is not computed with: equal.
  attend  a score is an fp32 sum of at most 128 products: off by 128 * 2^-24 = 2^-17 of b = sum |q_d k_d| / sqrt(dim),
          and its exponent's argument by 2^-23 of itself: 2^-17 (1 + b) in all.  Weights are rounded to fp16: 2^-11
          each, and those under 2^-21 of the largest to 2^-32 of it; n of them are summed in fp32 (2^-23 an addition);
          the output is rounded to bf16: |error| <= 2^-8 |out| + (2^-11 + 2^-16 (1 + b) + n 2^-23) sum w |v| + 2^-32 max w sum |v|
  lse     2^-17 (1 + b) + 2^-20 |lse|
"""
import numpy as np
import pytest
import torch

import paged4_util as pu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rc():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import __graft_entry__
    __graft_entry__.build()
    import fp8_ring_kv_cache_gb300 as rc
    return rc


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bf16(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16)


# ------------------------------------------------------------------ rotary forms
FORMS = [  # head_dim, first, sections, layout, scaling and gain
    (64, 0, (32,), "halves", {}),
    (64, 0, (32,), "pairs", {"scaling": "linear", "factor": 3.5}),
    (128, 0, (64,), "halves", {"scaling": "parts", "factor": 16.0, "context": 4096.0, "gain": 1.25}),
    (128, 0, (22, 21, 21), "halves", {"scaling": "base", "factor": 8.0}),
    (128, 32, (24, 24), "halves", {"gain": 0.1}),
    (128, 10, (1, 0, 30, 6), "pairs", {"shared": True}),
    (80, 0, (10,), "halves", {"scaling": "parts", "factor": 4.0, "context": 2048.0, "low": 1.0, "high": 4.0}),
    (80, 6, (9,), "halves", {}),
    (96, 2, (13,), "pairs", {"scaling": "base", "factor": 2.0, "gain": 2.0}),
    (8, 0, (1,), "halves", {"scaling": "base", "factor": 2.0}),
    (8, 2, (3,), "halves", {}),
    (192, 128, (32,), "pairs", {}),
    (256, 0, (128,), "halves", {"shared": True, "scaling": "linear", "factor": 2.0}),
    (256, 0, (64, 64), "pairs", {}),
]


def make_form(rc, form):
    dim, first, sections, layout, kw = form
    kw = dict(kw)
    return rc.RopeForm(dim, sections=sections, first=first, layout=layout, shared_freqs=kw.pop("shared", False), **kw)


def want_turn(form, x, pos, sign=1.0):
    dim, first, sections, layout, kw = form
    return pu.turn(x, pos, sections, first=first, layout=layout, sign=sign, **kw)


def check_turn(form, x, pos, got, sign):
    want, reach = want_turn(form, x.double().numpy(), pos, sign)
    got = got.detach().cpu()
    # the definition's own angle is rounded to 2^-53 of itself: up to 2^-22 at the farthest positions
    tol = (2.0 ** -20 + np.abs(pos.astype(np.float64)).max(initial=0) * 2.0 ** -52) * reach + 2.0 ** -23 * np.abs(want)
    if x.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(want)
    err = np.abs(got.double().numpy() - want)
    assert (err <= tol).all(), (form, (err - tol).max())
    dim, first, sections = form[:3]
    for a, b in ((0, first), (first + 2 * sum(sections), dim)):
        assert torch.equal(got[..., a:b], x[..., a:b])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,heads", [(1, 1), (1, 48), (37, 5), (1301, 3)])
def test_rope_turn(rc, form, dtype, n, heads):
    rng = np.random.default_rng(n + form[0])
    x = torch.from_numpy(rng.standard_normal((n, heads, form[0])).astype(np.float32)).to(dtype)
    axes = len(form[2])
    pos = rng.integers(-2 ** 31, 2 ** 31, (axes, n)).astype(np.int32)
    pos[:, : n // 2] = rng.integers(-1000, 200000, (axes, n // 2))
    f = make_form(rc, form)
    for sign, back in ((1.0, False), (-1.0, True)):
        got = rc.rc_rope_turn(x.cuda(), dev(pos), f, back=back)
        assert got.dtype == dtype
        check_turn(form, x, pos, got, sign)
        here = x.cuda()
        assert rc.rc_rope_turn(here, dev(pos), f, out=here, back=back) is here
        assert torch.equal(here, got)


def test_rope_turn_is_rope_axes_where_both_are(rc):
    rng = np.random.default_rng(3)
    x, pos = bf16(rng, 57, 6, 128).cuda(), dev(rng.integers(0, 100000, (3, 57)).astype(np.int32))
    a = rc.rc_rope_axes(x, pos, rc.RopeAxes((22, 21, 21)))
    assert torch.equal(a, rc.rc_rope_turn(x, pos, rc.RopeForm(128, sections=(22, 21, 21))))


@pytest.mark.parametrize("form", [FORMS[2], FORMS[6], FORMS[5]])
def test_rope_turn_strides_and_values_that_stay(rc, form):
    """A slice of a fused projection's rows into another's, positions from a longer table; what lies beside keeps its bits,
    and numbers outside the part, NaN and infinities among them, are copied."""
    rng = np.random.default_rng(5)
    n, heads, dim = 83, 6, form[0]
    wide = bf16(rng, n, 3 * heads, dim).cuda()
    first, turned = form[1], 2 * sum(form[2])
    if turned < dim:
        outside = [d for d in range(dim) if not first <= d < first + turned]
        wide[3, heads, outside[0]], wide[4, heads, outside[-1]] = float("nan"), float("inf")
    table = dev(rng.integers(0, 5000, (len(form[2]), 200)).astype(np.int32))
    pos, x = table[:, 50:50 + n], wide[:, heads:2 * heads]
    to = torch.full((n, 2 * heads, dim), 9.0, dtype=torch.bfloat16, device="cuda")
    rc.rc_rope_turn(x, pos, make_form(rc, form), out=to[:, heads:])
    assert (to[:, :heads] == 9.0).all()
    plain = rc.rc_rope_turn(x.contiguous(), pos.contiguous(), make_form(rc, form))
    assert torch.equal(to[:, heads:].contiguous().view(torch.int16), plain.view(torch.int16))


@pytest.mark.parametrize("form", [FORMS[2], FORMS[3], FORMS[8]])
def test_rope_turn_gradient(rc, form):
    """Against the transposed turn, against differences, and twice."""
    rng = np.random.default_rng(8)
    n, heads, dim = 19, 3, form[0]
    x = torch.from_numpy(rng.standard_normal((n, heads, dim)).astype(np.float32))
    dy = torch.from_numpy(rng.standard_normal((n, heads, dim)).astype(np.float32))
    pos = rng.integers(0, 50000, (len(form[2]), n)).astype(np.int32)
    f = make_form(rc, form)
    leaf = x.cuda().requires_grad_()
    y = rc.rc_rope_turn(leaf, dev(pos), f)
    (grad,) = torch.autograd.grad(y, leaf, dy.cuda(), create_graph=False, retain_graph=True)
    check_turn(form, dy, pos, grad, -1.0)
    # the turn is linear: <dy, f(x + e) - f(x)> is <grad, e> to rounding
    e = torch.from_numpy(rng.standard_normal((n, heads, dim)).astype(np.float32))
    a, b = want_turn(form, (x + e).double().numpy(), pos)[0], want_turn(form, x.double().numpy(), pos)[0]
    left, right = (dy.double().numpy() * (a - b)).sum(), (grad.double().cpu().numpy() * e.double().numpy()).sum()
    size = np.abs(dy.double().numpy()).sum() * 4 * f.gain * float((x.abs().max() + e.abs().max()))
    assert abs(left - right) <= 2.0 ** -20 * size
    y.sum().backward()  # a broadcast gradient
    check_turn(form, torch.ones(n, heads, dim), pos, leaf.grad, -1.0)
    with pytest.raises(RuntimeError):
        rc.rc_rope_turn(leaf, dev(pos), f, out=torch.empty_like(leaf))


def test_rope_turn_streams_and_graph(rc):
    rng = np.random.default_rng(9)
    form = FORMS[2]
    x, pos, f = bf16(rng, 40, 8, 128), rng.integers(0, 9000, (1, 40)).astype(np.int32), make_form(rc, form)
    xd, pd, out = x.cuda(), dev(pos), torch.empty(40, 8, 128, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = rc.rc_rope_turn(xd, pd, f, stream=side)
    side.synchronize()
    check_turn(form, x, pos, got, 1.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rc.rc_rope_turn(xd, pd, f, out=out)
    for seed in (1, 2):
        pos = np.random.default_rng(seed).integers(0, 9000, (1, 40)).astype(np.int32)
        pd.copy_(dev(pos))
        graph.replay()
        torch.cuda.synchronize()
        check_turn(form, x, pos, out, 1.0)


# ------------------------------------------------------------------ the cache
class Setup:
    """A pool, its metadata and the handles, on both sides."""

    def __init__(self, rc, seqs, hk, dim, page, seed, spread=1.0, tokens=None, max_kv=None, max_new=None):
        self.rc = rc
        self.rng = np.random.default_rng(seed)
        self.pool, self.meta = pu.make(seqs, hk, dim, page, self.rng, spread=spread)
        self.tokens = tokens if tokens is not None else int(self.meta["q_start"][-1])
        self.max_kv = max_kv if max_kv is not None else int(self.meta["kv_len"].max())
        self.max_new = max_new if max_new is not None else int(np.diff(self.meta["q_start"]).max())
        self.upload()

    def upload(self):
        rc = self.rc
        self.cache = rc.PagedKVCache4(*[dev(self.pool[k]) for k in ("kcodes", "vcodes", "kscale", "vscale")])
        self.table, self.kv_len, self.q_start = dev(self.meta["table"]), dev(self.meta["kv_len"]), dev(self.meta["q_start"])
        self.batch = rc.PagedBatch(self.table, self.kv_len, self.q_start, tokens=self.tokens, max_new=self.max_new,
                                   max_kv=self.max_kv)

    def held(self):
        return {k: getattr(self.cache, k).cpu().numpy() for k in ("kcodes", "vcodes", "kscale", "vscale")}

    # ---- write
    def write(self, K, V, pos, form, stream=None):
        self.cache.write(self.batch, K, V, None if pos is None else dev(pos), None if form is None else make_form(self.rc, form),
                         stream=stream)
        self.cache.sync(stream)

    def want_write(self, K, V, pos, form):
        """The pages after a write, and where K's codes (as the pages have them) and scales may be another's."""
        want = {k: v.copy() for k, v in self.pool.items()}
        kx = K.double().numpy()
        if form is None:
            y, reach = kx, np.zeros_like(kx)
        else:
            with np.errstate(invalid="ignore", over="ignore"):
                y, reach = want_turn(form, kx, pos)
            y = np.where(np.isfinite(kx).all(-1)[..., None], y, np.nan)
        far = 0.0 if pos is None else np.abs(pos.astype(np.float64)).max(0)[:, None, None]
        fine = np.isfinite(y).all(-1)[..., None]
        loose, open_ = pu.near_border(np.where(fine, y, 0.0), np.where(fine, reach * (2.0 ** -24 + far * 2.0 ** -52), 0.0))
        kc, ks = pu.quantise(y)
        vc, vs = pu.quantise(V.double().numpy())
        p = self.pool["kscale"].shape[3]
        may = []  # (page, head, place, dim) whose code may differ, (page, head, place, block) whose scale may
        for s in range(len(self.meta["kv_len"])):
            q0, q1, kv = self.meta["q_start"][s], self.meta["q_start"][s + 1], self.meta["kv_len"][s]
            for t in range(q0, q1):
                j = kv - (q1 - q0) + t - q0
                page, place = self.meta["table"][s, j // p], j % p
                for h in range(K.shape[1]):
                    pu.put(want, "k", page, h, place, kc[t, h], ks[t, h])
                    pu.put(want, "v", page, h, place, vc[t, h], vs[t, h])
                    for d in np.nonzero(loose[t, h] | open_[t, h])[0]:
                        may.append((page, h, place, int(d), bool(open_[t, h, d])))
        return want, may

    def check_write(self, K, V, pos, form):
        want, may = self.want_write(K, V, pos, form)
        got = self.held()
        assert np.array_equal(got["vcodes"], want["vcodes"]) and np.array_equal(got["vscale"], want["vscale"])
        a, b = pu.unpack(got["kcodes"]).copy(), pu.unpack(want["kcodes"])
        sa = got["kscale"].copy()
        for page, h, place, d, scale_too in may:
            if scale_too:
                assert abs(int(sa[page, h, d // 16, place]) - int(want["kscale"][page, h, d // 16, place])) <= 1
                sa[page, h, d // 16, place] = want["kscale"][page, h, d // 16, place]
            a[page, h, place, d] = b[page, h, place, d]
        if form is not None:  # (the sign of a sum that is 0 is anyone's)
            a[a == 8], b[b == 8] = 0, 0
        assert np.array_equal(sa, want["kscale"]) and np.array_equal(a, b)
        assert len(may) <= 32 + K.numel() // 1000  # (few values are so near a border)

    # ---- attend
    def attend(self, q, causal, stream=None):
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full(q.shape[:2], 7.0, device="cuda")
        self.cache.attend(self.batch, q, out, lse=lse, causal=causal, stream=stream)
        self.cache.sync(stream)
        return out, lse

    def check_attend(self, q, causal, got=None, heads=None, queries=None):
        """heads, queries: of which heads and of how many queries of a sequence (its first and last ones) to look at."""
        out, lse = got if got is not None else self.attend(q.cuda(), causal)
        qn = q.double().cpu().numpy()
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        hk, hq = self.pool["kcodes"].shape[1], q.shape[1]
        touched = np.zeros(len(qn), bool)
        for s in range(len(self.meta["kv_len"])):
            q0, q1, kv = self.meta["q_start"][s], self.meta["q_start"][s + 1], self.meta["kv_len"][s]
            touched[q0:q1] = True
            for head in (range(hq) if heads is None else heads):
                h = head * hk // hq
                k, v = (pu.tokens_of(self.pool, x, self.meta["table"][s], h, kv) for x in "kv")
                want, rlse, w, big = pu.attend_head(qn[q0:q1, head], k, v, q1 - q0, causal)
                g, gl = out[q0:q1, head], lse[q0:q1, head]
                empty = rlse == -np.inf
                assert (gl[empty] == -np.inf).all() and (g[empty] == 0).all()
                nan = np.isnan(want)
                assert np.isnan(g[nan]).all() and np.array_equal(np.isnan(gl), np.isnan(rlse))
                ok = ~nan & ~empty[:, None]
                assert np.isfinite(g[ok]).all()
                av = np.abs(np.nan_to_num(v))
                w = np.nan_to_num(w)
                tol = 2.0 ** -8 * np.abs(np.nan_to_num(want)) + (2.0 ** -11 + 2.0 ** -16 * (1 + big) + kv * 2.0 ** -23) * (w @ av) + \
                    2.0 ** -32 * w.max(-1, initial=0.0)[:, None] * av.sum(0) + 1e-30
                err = np.abs(np.where(ok, g - want, 0.0))
                assert (err <= tol).all(), (s, head, (err / tol).max())
                le = np.abs(np.where(np.isfinite(rlse), gl - rlse, 0.0))
                assert (le <= 2.0 ** -17 * (1 + big) + 2.0 ** -20 * np.abs(np.where(np.isfinite(rlse), rlse, 0.0))).all()
        assert (out[~touched] == 7.0).all() and (lse[~touched] == 7.0).all(), "a row of no sequence was written"
        return out, lse


WRITE_FORMS = {64: [FORMS[0], (64, 6, (9,), "halves", {}), None], 128: [FORMS[2], FORMS[3], FORMS[4], FORMS[5], (128, 2, (41,), "halves", {"gain": 3.0}), None]}


@pytest.mark.parametrize("dim,form", [(d, f) for d in (64, 128) for f in WRITE_FORMS[d]])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("seqs", [[(1, 1)], [(1, 40), (1, 7), (1, 16), (1, 33)], [(5, 9), (0, 12), (40, 40), (17, 70), (2, 131)]])
def test_write(rc, dim, form, page, seqs):
    s = Setup(rc, seqs, 3, dim, page, seed=dim + page + len(seqs))
    t = s.tokens
    K, V = bf16(s.rng, t, 3, dim), bf16(s.rng, t, 3, dim)
    pos = None if form is None else s.rng.integers(0, 200000, (len(form[2]), t)).astype(np.int32)
    s.write(K.cuda(), V.cuda(), pos, form)
    s.check_write(K, V, pos, form)


def test_write_many_heads_and_strides(rc):
    """Blocks of four heads and fewer at the end; rows of a fused projection; positions far away and zero (no turn at all:
    ties are then exact)."""
    form = FORMS[3]
    s = Setup(rc, [(757, 800), (3, 3)], 7, 128, 64, seed=5)
    t = s.tokens
    qkv = bf16(s.rng, t, 21, 128)
    pos = s.rng.integers(-2 ** 31, 2 ** 31, (3, t)).astype(np.int32)
    pos[:, ::3] = s.rng.integers(0, 90, (3, len(pos[0, ::3])))
    pos[1:, ::6] = 0
    pos[:, 5] = 0
    dq = qkv.cuda()
    s.write(dq[:, 7:14], dq[:, 14:], pos, form)
    s.check_write(qkv[:, 7:14], qkv[:, 14:], pos, form)


def test_write_values(rc):
    """Zeros, subnormal scales, ties, the largest numbers, infinities and NaN."""
    s = Setup(rc, [(16, 20)], 2, 64, 16, seed=6)
    K = bf16(s.rng, 16, 2, 64)
    V = K.clone()
    for x in (K, V):
        x[0] = 0.0
        x[1] *= 2.0 ** -15
        x[2] *= 2.0 ** -30
        x[3] *= 2.0 ** 13
        x[4] *= 2.0 ** 100
        x[5, 0, 3] = float("inf")
        x[6, 1, 60] = float("nan")
        x[7, :, :] = 6.0
        x[7, :, 1::2] = 0.25
        x[8] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 8).to(torch.bfloat16)
        x[9] = -x[8] * 1.125
        x[10, :, 16:] = 0.0
        x[11] *= torch.exp(torch.linspace(-20, 20, 64))
        x[12, 0, 0] = -0.0
        x[13] = 3e38
        x[13, :, ::2] = -3e38
    V[14] = 61440.0
    V[15] = 2.0 ** -18
    for form, pos in ((None, None), (FORMS[0], np.zeros((1, 16), np.int32))):
        s.upload()
        s.write(K.cuda(), V.cuda(), pos, form)
        s.check_write(K, V, pos, form)
    # turned: rows that are not numbers are 255 throughout, the largest saturate
    form, pos = (64, 0, (32,), "halves", {"gain": 16.0}), np.arange(16, dtype=np.int32)[None] * 1000
    s.upload()
    s.write(K.cuda(), V.cuda(), pos, form)
    s.check_write(K, V, pos, form)


ROW_CASES = [  # sequences (new, kv), heads, kv_heads
    ([(1, 1)], 1, 1), ([(1, 337)], 16, 2), ([(1, 64), (1, 65), (1, 1000), (1, 3)], 8, 1), ([(1, 700), (0, 5), (2, 300)], 12, 2),
    ([(3, 3), (8, 90), (1, 2049)], 2, 2), ([(16, 500)], 1, 1), ([(2, 8200)], 7, 1),
]


@pytest.mark.parametrize("seqs,hq,hk", ROW_CASES)
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 32), (128, 64), (64, 128), (128, 16)])
@pytest.mark.parametrize("causal", [True, False])
def test_attend_few_rows(rc, seqs, hq, hk, dim, page, causal):
    s = Setup(rc, seqs, hk, dim, page, seed=dim + page)
    s.check_attend(bf16(s.rng, s.tokens, hq, dim), causal)


@pytest.mark.parametrize("seqs,hq,hk", [([(4, 300), (1, 70), (0, 5), (3, 3)], 8, 1), ([(4, 5000), (2, 40), (1, 3000)], 16, 2), ([(32, 50)], 1, 1),
                                        ([(3, 700)] * 9, 16, 2)])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (128, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_attend_two_row_tiles(rc, seqs, hq, hk, dim, page, causal):
    s = Setup(rc, seqs, hk, dim, page, seed=dim + page)
    s.check_attend(bf16(s.rng, s.tokens, hq, dim), causal)


TILE_CASES = [
    ([(17, 17)], 1, 1), ([(40, 300), (1, 129), (0, 9), (90, 90)], 2, 1), ([(130, 257)], 3, 1), ([(300, 700), (5, 1200)], 4, 2),
    ([(33, 4000)], 2, 2),
]


@pytest.mark.parametrize("seqs,hq,hk", TILE_CASES)
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 32), (128, 64), (64, 128), (128, 16)])
@pytest.mark.parametrize("causal", [True, False])
def test_attend_many_rows(rc, seqs, hq, hk, dim, page, causal):
    s = Setup(rc, seqs, hk, dim, page, seed=dim + page)
    s.check_attend(bf16(s.rng, s.tokens, hq, dim), causal)


@pytest.mark.parametrize("seqs,hq,hk", [([(1, 90), (1, 7)], 4, 1), ([(2, 90), (30, 200)], 3, 1)])
@pytest.mark.parametrize("dim", [64, 128])
def test_attend_spread_of_sizes(rc, seqs, hq, hk, dim):
    """Tokens whose sizes are far apart, and query rows far from 1."""
    s = Setup(rc, seqs, hk, dim, 32, seed=3, spread=4.0)
    q = bf16(s.rng, s.tokens, hq, dim)
    q[0] *= 2.0 ** -60
    q[1] *= 2.0 ** -3
    s.check_attend(q, True)


@pytest.mark.parametrize("seqs,hq,hk", [([(1, 90), (1, 1), (1, 1500)], 4, 1), ([(3, 700), (1, 2)], 12, 2), ([(1, 20000)], 8, 1), ([(30, 500), (1, 1)], 3, 1),
                                        ([(200, 1000), (90, 90)], 4, 2)])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("size", [2.0 ** 16, 2.0 ** 20, 2.0 ** 24, 2.0 ** 27, 2.0 ** 32, 2.0 ** 60, 2.0 ** 110, -(2.0 ** 26), 2.0])
def test_attend_large_scores(rc, seqs, hq, hk, dim, page, size):
    """Scores far over what weights can be told apart by (size 2: rows of Q under 16, K with the largest scale): every result is finite, and where the largest score leads the others
    by 30 and more than what rounding may be (2^-17 (1 + b) each), it is that token's V and its score; with two tokens of the
    same K it is the mean of both their V."""
    s = Setup(rc, seqs, hk, dim, page, seed=dim + page, spread=0.3)
    if size == 2.0:
        s.pool["kscale"][:] = pu.TOP
    for i, (new, kv) in enumerate(seqs):  # the last token's K is the first one's too
        first, last = (s.meta["table"][i, j // page] for j in (0, kv - 1))
        s.pool["kcodes"][first, :, 0] = s.pool["kcodes"][last, :, (kv - 1) % page]
        s.pool["kscale"][first, :, :, 0] = s.pool["kscale"][last, :, :, (kv - 1) % page]
    s.upload()
    q = bf16(s.rng, s.tokens, hq, dim) * size
    for t in s.meta["q_start"][1:] - 1:  # the last query of a sequence looks for its last token
        i = int(np.searchsorted(s.meta["q_start"], t, side="right")) - 1
        kv = int(s.meta["kv_len"][i])
        for head in range(hq):
            k = pu.tokens_of(s.pool, "k", s.meta["table"][i], head * hk // hq, kv)[-1]
            q[t, head] = torch.from_numpy((7.96 * k / np.abs(k).max()).astype(np.float32)).to(torch.bfloat16) * size
    out, lse = s.attend(q.cuda(), True)
    out, lse, qn = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().numpy()
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    sure = twice = 0
    for i, (new, kv) in enumerate(seqs):
        q0 = s.meta["q_start"][i]
        for head in range(hq):
            k, v = (pu.tokens_of(s.pool, x, s.meta["table"][i], head * hk // hq, kv) for x in "kv")
            for t in range(new):
                see = kv - new + t + 1
                x = k[:see] @ qn[q0 + t, head] / np.sqrt(dim)
                off = 2.0 ** -17 * (1 + (np.abs(k[:see]) @ np.abs(qn[q0 + t, head]) / np.sqrt(dim)).max())
                top = x.max()
                lead = np.nonzero(x >= top - 2 * off - 30)[0]
                g, tol = out[q0 + t, head], off + 2.0 ** -20 * abs(top)
                # (what is behind has weights under e^-30 each)
                if len(lead) == 1:
                    sure += 1
                    assert (np.abs(g - v[lead[0]]) <= 2.0 ** -8 * np.abs(v[lead[0]]) + see * np.exp(-30.0) * np.abs(v[:see]).max()).all(), (i, head, t)
                    assert abs(lse[q0 + t, head] - top) <= tol + see * np.exp(-30.0)
                elif len(lead) == 2 and lead[0] == 0 and lead[1] == kv - 1 == see - 1:
                    twice += 1
                    want = (v[0] + v[-1]) / 2
                    # (two weights rounded to fp16 each, the result to bf16)
                    assert (np.abs(g - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + see * np.exp(-30.0)) * np.abs(v[:see]).max()).all(), (i, head, t)
                    assert abs(lse[q0 + t, head] - top - np.log(2.0)) <= tol + see * np.exp(-30.0)
                else:
                    low, high = v[lead].min(0), v[lead].max(0)
                    reach = 2.0 ** -8 * np.abs(g) + (2.0 ** -10 + see * np.exp(-30.0)) * np.abs(v[:see]).max()
                    assert (g >= low - reach).all() and (g <= high + reach).all(), (i, head, t)
    assert sure + twice > 0 and (size < 2.0 ** 20 or twice > 0) and (size != 2.0 or np.abs(qn).max() < 16.0)


@pytest.mark.parametrize("rows", [1, 5, 40])
def test_attend_rows_that_see_nothing(rc, rows):
    """More new tokens than cached ones: the first rows see no token; a sequence without any."""
    s = Setup(rc, [(rows, max(0, rows - 3)), (rows, 0), (rows, rows + 20)], 2, 128, 16, seed=rows)
    s.check_attend(bf16(s.rng, s.tokens, 4, 128), True)


@pytest.mark.parametrize("new,hq", [(1, 2), (6, 2), (40, 2), (200, 2)])
def test_attend_what_is_behind_the_end(rc, new, hq):
    """Places behind a sequence's end, and pages that no sequence has, hold NaN scales: nothing of them is seen."""
    s = Setup(rc, [(new, new + 30), (new, new + 55)], 1, 128, 64, seed=new)
    used = np.zeros(s.pool["kscale"].shape[0] * 64, bool)
    for i in range(2):
        for j in range(s.meta["kv_len"][i]):
            used[s.meta["table"][i, j // 64] * 64 + j % 64] = True
    for name in ("kscale", "vscale"):
        a = s.pool[name].transpose(0, 3, 1, 2).reshape(-1, 1, 8)
        a[~used] = 255
        s.pool[name] = np.ascontiguousarray(a.reshape(-1, 64, 1, 8).transpose(0, 2, 3, 1))
    s.upload()
    out, lse = s.check_attend(bf16(s.rng, s.tokens, hq, 128), True)
    assert np.isfinite(out).all() and np.isfinite(lse).all()


@pytest.mark.parametrize("new,hq,hk", [(6, 2, 1), (40, 2, 2), (260, 1, 1)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("name", ["k", "v"])
def test_attend_tokens_that_are_not_numbers(rc, new, hq, hk, dim, name):
    """Rows that see such a token get NaN, the others do not."""
    s = Setup(rc, [(new, new + 70)], hk, dim, 16, seed=new + dim)
    j = new + 70 - 3
    s.pool[name + "codes"] = s.pool[name + "codes"].copy()
    pu.put(s.pool, name, s.meta["table"][0, j // 16], 0, j % 16, np.zeros(dim, np.uint8), np.full(dim // 16, 255, np.uint8))
    s.upload()
    out, _ = s.check_attend(bf16(s.rng, s.tokens, hq, dim), True)
    assert np.isnan(out[-3:, 0]).all() and np.isfinite(out[:-3]).all()


def test_attend_long_sequence(rc):
    s = Setup(rc, [(1, 40001), (1, 5)], 1, 64, 128, seed=2)
    s.check_attend(bf16(s.rng, 2, 8, 64), True)
    s = Setup(rc, [(20, 20001)], 1, 64, 128, seed=3)
    s.check_attend(bf16(s.rng, 20, 2, 64), True)


def test_attend_strides_rows_of_nobody_and_repeats(rc):
    s = Setup(rc, [(1, 500), (9, 60)], 2, 128, 32, seed=4, tokens=14, max_new=30, max_kv=512)
    s.meta["table"] = np.concatenate([s.meta["table"]] * 2, 1)
    s.upload()
    wide = bf16(s.rng, 14, 3 * 8, 128).cuda()
    out = torch.full((14, 16, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((14, 8), 7.0, device="cuda")
    for _ in range(2):
        s.cache.attend(s.batch, wide[:, 8:16], out[:, 8:], lse=lse)
    s.cache.sync()
    assert (out[:, :8] == 7.0).all()
    s.check_attend(wide[:, 8:16].cpu(), True, got=(out[:, 8:], lse))
    again = s.attend(wide[:, 8:16], True)
    assert torch.equal(again[0][:10], out[:10, 8:]) and torch.equal(again[1][:10], lse[:10])


def test_bad_metadata_is_left_out_and_reported(rc):
    """Lengths, rows and pages out of bounds: nothing of them is read or written, the call's status says so."""
    for new in (1, 40):
        s = Setup(rc, [(new, new + 20), (new, new + 40)], 2, 64, 16, seed=new)
        good = s.attend(bf16(np.random.default_rng(1), s.tokens, 2, 64).cuda(), True)
        q = bf16(np.random.default_rng(1), s.tokens, 2, 64).cuda()
        before = s.held()
        for what in ("page", "kv", "rows"):
            s.upload()
            if what == "page":
                s.table[1, 0] = 10 ** 6
            elif what == "kv":
                s.kv_len[1] = s.max_kv + 1
            else:
                s.q_start[2] = s.tokens + 5
            out = torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda")
            s.cache.attend(s.batch, q, out)
            with pytest.raises(rc.RcError) as e:
                s.cache.sync()
            assert e.value.status == rc.RC_ERR_ARG
            s.cache.sync()  # said once
            assert torch.equal(out[:new], good[0][:new])
            if what != "page":
                s.cache.write(s.batch, q, q)
                with pytest.raises(rc.RcError):
                    s.cache.sync()
                table, p = s.meta["table"], 16
                other = [int(x) for x in table[1] if x >= 0]
                for k, v in s.held().items():
                    assert np.array_equal(v[other], before[k][other])


def test_a_layers_step(rc):
    """Queries turned, keys and values written, attention over both, a prompt and then single tokens, as a model calls them;
    the steps captured into a graph that is replayed as the lengths grow."""
    form = FORMS[2]
    f, rng = make_form(rc, form), np.random.default_rng(12)
    hk, hq, dim, page, steps = 2, 8, 128, 32, 5
    prompts = [37, 5]
    cache = rc.PagedKVCache4.empty(pages=8, kv_heads=hk, head_dim=dim, page_tokens=page)
    table = np.array([[3, 1, 6], [0, 5, 2]], np.int32)
    ref = {k: getattr(cache, k).cpu().numpy() for k in ("kcodes", "vcodes", "kscale", "vscale")}

    def step(new, kv, q, k, v, pos, batch, out, lse, qt):
        rc.rc_rope_turn(q, pos, f, out=qt)
        cache.write(batch, k, v, pos, f)
        cache.attend(batch, qt, out, lse=lse)

    s = Setup.__new__(Setup)
    s.rc, s.pool, s.cache = rc, ref, cache

    def check(meta, q, k, v, pos, qt, out, lse):
        s.meta, s.tokens = meta, len(q)
        s.check_write(k, v, pos, form)
        s.pool = s.held()
        check_turn(form, q, pos, qt, 1.0)
        s.check_attend(qt.cpu(), True, got=(out, lse))

    def rows(t):
        return bf16(rng, t, hq, dim), bf16(rng, t, hk, dim), bf16(rng, t, hk, dim)

    # the prompts
    t = sum(prompts)
    q, k, v = rows(t)
    pos = np.concatenate([np.arange(n) for n in prompts]).astype(np.int32)[None]
    meta = {"table": table, "kv_len": np.array(prompts, np.int32), "q_start": np.array([0, prompts[0], t], np.int32)}
    batch = rc.PagedBatch(dev(table), dev(meta["kv_len"]), dev(meta["q_start"]), tokens=t, max_new=max(prompts), max_kv=96)
    out, lse, qt = torch.empty(t, hq, dim, dtype=torch.bfloat16, device="cuda"), torch.empty(t, hq, device="cuda"), torch.empty(t, hq, dim, dtype=torch.bfloat16, device="cuda")
    step(None, None, q.cuda(), k.cuda(), v.cuda(), dev(pos), batch, out, lse, qt)
    cache.sync()
    check(meta, q, k, v, pos, qt, out, lse)
    # single tokens: direct once, then replayed
    q, k, v = (x.cuda() for x in rows(2))
    kv_len, q_start, posd = dev(np.array(prompts, np.int32)), dev(np.array([0, 1, 2], np.int32)), dev(np.array([prompts], np.int32))
    batch = rc.PagedBatch(dev(table), kv_len, q_start, tokens=2, max_new=1, max_kv=96)
    out, lse, qt = torch.empty(2, hq, dim, dtype=torch.bfloat16, device="cuda"), torch.empty(2, hq, device="cuda"), torch.empty(2, hq, dim, dtype=torch.bfloat16, device="cuda")
    graph = None
    for i in range(steps):
        for x, y in zip((q, k, v), rows(2)):
            x.copy_(y)
        kv_len += 1
        pos = (kv_len.cpu().numpy() - 1)[None].astype(np.int32)
        posd.copy_(dev(pos))
        if i == 1:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step(None, None, q, k, v, posd, batch, out, lse, qt)
        if graph is None:
            step(None, None, q, k, v, posd, batch, out, lse, qt)
        else:
            graph.replay()
        cache.sync()
        meta = {"table": table, "kv_len": kv_len.cpu().numpy(), "q_start": np.array([0, 1, 2], np.int32)}
        check(meta, q.cpu(), k.cpu(), v.cpu(), pos, qt, out, lse)


def test_streams_of_their_own(rc):
    """Two caches on two streams at once, each with its workspace."""
    caches = [Setup(rc, [(1, 900), (1, 77)], 2, 128, 64, seed=i) for i in range(2)]
    qs = [bf16(c.rng, 2, 8, 128) for c in caches]
    streams, outs = [torch.cuda.Stream() for _ in caches], []
    torch.cuda.synchronize()
    for c, q, st in zip(caches, qs, streams):
        out, lse = torch.empty(2, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 8, device="cuda")
        qd = q.cuda()
        torch.cuda.synchronize()
        for _ in range(20):
            c.cache.attend(c.batch, qd, out, lse=lse, stream=st)
        outs.append((out, lse))
    torch.cuda.synchronize()
    for c, q, got in zip(caches, qs, outs):
        c.check_attend(q, True, got=got)


def test_a_workspace_for_both_kinds_of_cache(rc):
    """Calls on an FP8 cache and on a 4-bit one that share a workspace, one after another on one stream."""
    s = Setup(rc, [(1, 3000)], 1, 128, 64, seed=9)
    fp8 = rc.PagedKVCache.empty(pages=48, kv_heads=1, head_dim=128, page_tokens=64, workspace=s.cache.workspace)
    table, kv_len, q_start = dev(np.arange(48, dtype=np.int32)[None]), dev(np.array([3000], np.int32)), dev(np.array([0, 1], np.int32))
    batch = rc.PagedBatch(table, kv_len, q_start, tokens=1, max_new=1, max_kv=3000)
    q = bf16(s.rng, 1, 4, 128)
    out8 = torch.full((1, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    want = None
    for _ in range(3):
        fp8.attend(batch, q.cuda(), out8)
        got = s.attend(q.cuda(), True)
        assert (out8 == 0).all()  # pages of zeros
        s.check_attend(q, True, got=got)
        assert want is None or torch.equal(want, got[0])
        want = got[0]


@pytest.mark.parametrize("new,hq", [(1, 6), (3, 5), (4, 8)])
def test_a_line_of_many_lists(rc, new, hq):
    """More sequences than a block has threads, of lengths from none to thousands, some without new tokens: equal stretches
    of work, which begin and end anywhere.  The same twice, bit for bit."""
    rng = np.random.default_rng(new)
    seqs = [(int(rng.integers(0, new + 1)), int(np.exp(rng.uniform(0, np.log(2500))))) for _ in range(300)]
    seqs[7], seqs[8], seqs[299] = (new, 0), (0, 0), (new, 3000)
    s = Setup(rc, seqs, 2, 64, 32, seed=new)
    q = bf16(s.rng, s.tokens, 2 * hq, 64)
    got = s.check_attend(q, True, heads=[0, hq, 2 * hq - 1])
    again = s.attend(q.cuda(), True)
    assert np.array_equal(got[0], again[0].double().cpu().numpy()) and np.array_equal(got[1], again[1].double().cpu().numpy())


@pytest.mark.parametrize("new,hq", [(1, 2), (2, 8), (5, 8)])
def test_a_graph_over_growing_lengths(rc, new, hq):
    """One captured call, replayed as the lengths on the device change from a few tokens to thousands and back."""
    s = Setup(rc, [(new, 4000 + 40 * i) for i in range(40)], 2, 64, 128, seed=new, max_kv=8192)
    s.meta["table"] = np.concatenate([s.meta["table"], np.zeros((40, 64 - s.meta["table"].shape[1]), np.int32)], 1)
    s.upload()
    q = bf16(s.rng, s.tokens, hq, 64)
    qd, out, lse = q.cuda(), torch.empty(q.shape, dtype=torch.bfloat16, device="cuda"), torch.empty(q.shape[:2], device="cuda")
    s.cache.attend(s.batch, qd, out, lse=lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.cache.attend(s.batch, qd, out, lse=lse)
    full = s.meta["kv_len"].copy()
    for share in (0.0, 0.1, 1.0, 0.01):
        s.meta["kv_len"] = np.maximum((full * share).astype(np.int32), new if share else 0)
        s.kv_len.copy_(dev(s.meta["kv_len"]))
        graph.replay()
        s.cache.sync()
        s.check_attend(q, True, got=(out, lse), heads=[0, hq - 1])


@pytest.mark.parametrize("new,hq", [(1, 4), (3, 8), (20, 4)])
def test_pages_far_into_a_large_pool(rc, new, hq):
    """Codes past 2^32 bytes and scales past 2^31 of their pool."""
    dim, page, hk = 128, 64, 1
    s = Setup(rc, [(new, 700), (new, 90)], hk, dim, page, seed=new)
    pages, small = (1 << 32) // (page * dim // 2) + 4096 * 900, s.pool["kcodes"].shape[0]
    cache = rc.PagedKVCache4.empty(pages=pages, kv_heads=hk, head_dim=dim, page_tokens=page)
    assert cache.kcodes.numel() > 1 << 34 and cache.kscale.numel() > 1 << 31
    at = dev(np.linspace(pages - 1, pages // 2, small).astype(np.int64))
    for k, v in s.pool.items():
        getattr(cache, k)[at] = dev(v)
    table = s.meta["table"]
    far = np.where(table < 0, -1, at.cpu().numpy()[np.maximum(table, 0)]).astype(np.int32)
    batch = rc.PagedBatch(dev(far), s.kv_len, s.q_start, tokens=s.tokens, max_new=s.max_new, max_kv=s.max_kv)
    q = bf16(s.rng, s.tokens, hq, dim)
    out, lse = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda"), torch.empty(q.shape[:2], device="cuda")
    cache.attend(batch, q.cuda(), out, lse=lse)
    cache.sync()
    s.check_attend(q, True, got=(out, lse))
    K, V = bf16(s.rng, s.tokens, hk, dim), bf16(s.rng, s.tokens, hk, dim)
    cache.write(batch, K.cuda(), V.cuda())
    cache.sync()
    want, _ = s.want_write(K, V, None, None)
    for k, v in want.items():
        assert np.array_equal(getattr(cache, k)[at].cpu().numpy(), v), k


@pytest.mark.parametrize("dim", [64, 128])
def test_pages_on_a_16_byte_boundary(rc, dim):
    """Pages whose address is a multiple of 16 bytes but not of 32 give the same bits."""
    s = Setup(rc, [(3, 200), (150, 600)], 2, dim, 16, seed=95)
    small = Setup(rc, [(1, 300), (2, 90)], 2, dim, 16, seed=96)

    def moved(t):
        flat = torch.zeros(t.numel() + 64, dtype=torch.uint8, device="cuda")
        at = 16 + (-flat.data_ptr()) % 32
        new = flat[at:at + t.numel()].view(t.shape)
        assert new.data_ptr() % 32 == 16
        return new.copy_(t)

    for x in (s, small):
        q, K = bf16(x.rng, x.tokens, 4, dim).cuda(), bf16(x.rng, x.tokens, 2, dim).cuda()
        a = x.attend(q, True)
        x.cache.write(x.batch, K, K)
        pages = x.held()
        x.upload()
        x.cache = rc.PagedKVCache4(*[moved(getattr(x.cache, k)) for k in ("kcodes", "vcodes", "kscale", "vscale")])
        b = x.attend(q, True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        x.cache.write(x.batch, K, K)
        for k, v in x.held().items():
            assert np.array_equal(v, pages[k])


def test_a_wait_that_runs_out_is_reported(rc):
    s = Setup(rc, [(200, 900), (30, 400)], 2, 128, 64, seed=11)
    q = bf16(s.rng, s.tokens, 4, 128).cuda()
    good = s.attend(q, True)
    rc.rc_paged_set_wait_limit(0)
    try:
        s.cache.attend(s.batch, q, torch.zeros_like(q))
        with pytest.raises(rc.RcError) as e:
            s.cache.sync()
    finally:
        rc.rc_paged_set_wait_limit(2_000_000_000)
    assert e.value.status == rc.RC_ERR_TIMEOUT
    s.cache.sync()
    again = s.attend(q, True)
    assert torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])


@pytest.mark.parametrize("seqs,hq,hk", [([(200, 900), (30, 400)], 4, 2), ([(40, 3000)], 2, 1), ([(300, 2500)], 2, 2), ([(33, 1100)] * 40, 2, 2)])
@pytest.mark.parametrize("dim", [64, 128])
def test_waits_that_run_out_at_any_time(rc, seqs, hq, hk, dim):
    """Limits from nothing to what a call takes: a wait runs out early, late, at some warps only or nowhere.  Each call ends,
    says so if one did, has its result if none did, and leaves nothing behind for the next."""
    s = Setup(rc, seqs, hk, dim, 64, seed=dim + hq)
    q = bf16(s.rng, s.tokens, hq, dim).cuda()
    good = s.attend(q, False)
    for limit in [0, 1, 100, 300, 1000, 2000, 4000, 8000, 16000, 32000] * 4:
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
        rc.rc_paged_set_wait_limit(limit)
        try:
            s.cache.attend(s.batch, q, out, lse=lse, causal=False)
        finally:
            rc.rc_paged_set_wait_limit(2_000_000_000)
        try:
            s.cache.sync()
        except rc.RcError as e:
            assert e.status == rc.RC_ERR_TIMEOUT
        else:
            assert torch.equal(out, good[0]) and torch.equal(lse, good[1])
    again = s.attend(q, False)
    assert torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])


def test_new_tokens_that_the_length_does_not_count(rc):
    s = Setup(rc, [(5, 4), (3, 9)], 2, 64, 16, seed=12)
    K = bf16(s.rng, s.tokens, 2, 64)
    before = s.held()
    s.cache.write(s.batch, K.cuda(), K.cuda())
    with pytest.raises(rc.RcError) as e:
        s.cache.sync()
    assert e.value.status == rc.RC_ERR_ARG
    first = int(s.meta["table"][0, 0])
    got = s.held()
    for k in got:
        assert np.array_equal(got[k][first], before[k][first])
    assert not np.array_equal(got["kcodes"], before["kcodes"])  # (the other sequence's tokens are there)


def test_refusals_of_tensors(rc):
    s = Setup(rc, [(3, 20)], 2, 64, 16, seed=13)
    form = rc.RopeForm(64)
    K, q = bf16(s.rng, 3, 2, 64).cuda(), bf16(s.rng, 3, 4, 64).cuda()
    pos, out = torch.zeros(1, 3, dtype=torch.int32, device="cuda"), torch.empty(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    c, b = s.cache, s.batch
    for bad in (lambda: c.write(b, K, K, pos), lambda: c.write(b, K, K, pos, rc.RopeForm(128)), lambda: c.write(b, K[:2], K, pos, form),
                lambda: c.write(b, K, K.transpose(1, 2).contiguous().transpose(1, 2), pos, form), lambda: c.write(b, K, K, pos[:, :2], form),
                lambda: c.attend(b, q[0], out), lambda: c.attend(b, q, out[:, :2]), lambda: c.attend(b, q, out, lse=torch.empty(3, 3, device="cuda")),
                lambda: rc.rc_rope_turn(q, pos, rc.RopeForm(128)), lambda: rc.rc_rope_turn(q, pos[0], form),
                lambda: rc.rc_rope_turn(q[:2], pos[:, :2], form, out=q[1:]), lambda: rc.rc_rope_turn(q[0], pos, form)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: c.write(b, K, K, None, form), lambda: c.write(b, K.float(), K, pos, form), lambda: c.attend(b, q.cpu(), out),
                lambda: c.attend(b, q, out.float()), lambda: rc.rc_rope_turn(q.half(), pos, form), lambda: rc.rc_rope_turn(q.cpu(), pos, form),
                lambda: rc.rc_rope_turn(q, pos.long(), form), lambda: rc.PagedKVCache4(c.kcodes.cpu(), c.vcodes, c.kscale, c.vscale),
                lambda: rc.PagedKVCache4(c.kcodes, c.vcodes.float(), c.kscale, c.vscale)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(ValueError):
        rc.PagedKVCache4(c.kcodes, c.kcodes, c.kscale, c.vscale)
    with pytest.raises(ValueError):
        rc.PagedKVCache4(c.kcodes, c.vcodes, c.kscale[:, :, :2], c.vscale)
    with pytest.raises(rc.RcError) as e:  # queries and results in one place
        c.attend(b, q, q)
    assert e.value.status == rc.RC_ERR_ARG
    with pytest.raises(rc.RcError) as e:  # heads that the KV heads do not divide
        c.attend(b, bf16(s.rng, 3, 3, 64).cuda(), torch.empty(3, 3, 64, dtype=torch.bfloat16, device="cuda"))
    assert e.value.status == rc.RC_ERR_ARG
    c.sync()


def test_rope_turn_gradient_in_a_graph_and_on_another_stream(rc):
    """Forward and backward captured together, replayed on other inputs; and recorded on a stream of the caller's."""
    form = FORMS[3]
    f, rng = make_form(rc, form), np.random.default_rng(20)
    pos = rng.integers(0, 50000, (3, 12)).astype(np.int32)
    pd, dy = dev(pos), torch.from_numpy(rng.standard_normal((12, 2, 128)).astype(np.float32))
    leaf = torch.zeros(12, 2, 128, device="cuda", requires_grad=True)
    dyd = dy.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            (grad,) = torch.autograd.grad(rc.rc_rope_turn(leaf, pd, f), leaf, dyd)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = rc.rc_rope_turn(leaf, pd, f)
        (grad,) = torch.autograd.grad(y, leaf, dyd)
    for seed in (1, 2):
        x = torch.from_numpy(np.random.default_rng(seed).standard_normal((12, 2, 128)).astype(np.float32))
        leaf.data.copy_(x)
        dy = torch.from_numpy(np.random.default_rng(seed + 9).standard_normal((12, 2, 128)).astype(np.float32))
        dyd.copy_(dy)
        graph.replay()
        torch.cuda.synchronize()
        check_turn(form, x, pos, y, 1.0)
        check_turn(form, dy, pos, grad, -1.0)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    y = rc.rc_rope_turn(leaf, pd, f, stream=other)
    torch.cuda.current_stream().wait_stream(other)
    (grad,) = torch.autograd.grad(y, leaf, dyd)
    torch.cuda.synchronize()
    check_turn(form, dy, pos, grad, -1.0)


MIXED = [  # single and few new tokens next to long ones; rows at, one under and one over what a single token's tile holds
    ([(1, 900)] * 5 + [(130, 400)], 6, 1), ([(300, 300)] + [(1, 2000), (2, 50), (3, 70), (0, 4), (1, 0)] * 2, 8, 2),
    ([(8, 600), (9, 600), (7, 33), (1, 1), (60, 90), (2, 0)], 1, 1), ([(1, 500), (2, 300), (1, 5000), (40, 41)], 16, 1),
    ([(1, 500), (2, 300), (1, 600), (40, 100)], 17, 1), ([(1, 300), (1, 90), (9, 300)], 33, 1), ([(1, 6000), (20, 6000)], 8, 4),
    ([(1, 700)] * 70 + [(64, 3000)] + [(1, 40)] * 70, 4, 1),
]


@pytest.mark.parametrize("seqs,hq,hk", MIXED)
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_attend_short_and_long_sequences_in_one_call(rc, seqs, hq, hk, dim, page, causal):
    s = Setup(rc, seqs, hk, dim, page, seed=dim + len(seqs))
    q = bf16(s.rng, s.tokens, hq, dim)
    first = s.check_attend(q, causal)
    again = s.attend(q.cuda(), causal)
    assert np.array_equal(first[0], again[0].double().cpu().numpy(), equal_nan=True)
    assert np.array_equal(first[1], again[1].double().cpu().numpy(), equal_nan=True)


def test_a_graph_in_which_sequences_become_short_and_long(rc):
    """One captured call over 9 sequences whose new tokens change on the device: all short, mixed, and rows of nobody."""
    s = Setup(rc, [(1, 700 + 90 * i) for i in range(8)] + [(40, 1500)], 2, 64, 32, seed=11, tokens=120, max_new=40)
    q = bf16(s.rng, 120, 12, 64)
    qd = q.cuda()
    out, lse = torch.empty((120, 12, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((120, 12), device="cuda")
    s.cache.attend(s.batch, qd, out, lse=lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.cache.attend(s.batch, qd, out, lse=lse)
    for new in ([1] * 9, [1] * 8 + [40], [40, 1, 0, 2, 1, 1, 40, 0, 1], [13] * 9):
        s.meta["q_start"] = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        s.q_start.copy_(dev(s.meta["q_start"]))
        n = sum(new)
        out.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        s.cache.sync()
        s.check_attend(q, True, got=(out, lse), heads=[0, 11])
        assert (out[n:] == 7.0).all() and (lse[n:] == 7.0).all()


def test_many_short_and_long_sequences_in_one_call(rc):
    """More sequences than a block of the tiles' kernel has threads, tiles of lengths that end anywhere, a bad length among them
    (which is left out and reported; the others are as they were)."""
    rng = np.random.default_rng(5)
    seqs = [(1, int(rng.integers(1, 200))) for _ in range(700)]
    for i in (0, 13, 14, 333, 639, 640, 699):
        seqs[i] = (int(rng.integers(60, 400)), int(rng.integers(1, 500)))
    seqs[20], seqs[641] = (0, 3), (1, 0)
    s = Setup(rc, seqs, 1, 64, 16, seed=6)
    q = bf16(s.rng, s.tokens, 5, 64)
    s.check_attend(q, True, heads=[0, 4])
    good, _ = s.attend(q.cuda(), True)
    s.kv_len[333] = s.max_kv + 1
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    s.cache.attend(s.batch, q.cuda(), out)
    with pytest.raises(rc.RcError):
        s.cache.sync()
    a, b = int(s.meta["q_start"][333]), int(s.meta["q_start"][334])
    assert (out[a:b] == 7.0).all()
    assert torch.equal(out[:a], good[:a]) and torch.equal(out[b:], good[b:])

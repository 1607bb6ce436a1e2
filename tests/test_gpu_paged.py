"""The paged-cache operators and the several-axes rotary positions on the GPU, against their definitions in 64 bits
(tests/paged_util.py).

Tolerances, from the roundings that the operators make (half a step: bf16 2^-8 of the value, fp32 2^-24):
  turn        fp32 products of magnitude r (the pair's length): cos, sin and the position's fraction of a turn are
              each within 3 * 2^-24 + 2^-32 * 2 pi, the two products and their sum add 3 * 2^-24: 2^-20 r covers
              them; a bf16 result is rounded once more
  write       scales equal to the definition's except where the row's largest magnitude is within 2^-20 of a power-of-two
              border; codes of K within one step (a product within 2^-20 r of a border between two codes can fall on
              either side); V is not computed with: its codes and scales are equal
  attend      a score is an fp32 sum of at most 128 products: off by 128 * 2^-24 = 2^-17 of b = sum |q_d k_d| / sqrt(dim),
              and its exponent's argument by 2^-23 of itself: 2^-17 (1 + b) in all.  Weights are rounded to bf16 (2^-8
              each), the output is rounded to bf16: |error| <= 2^-8 |out| + (2^-8 + 2 * 2^-17 (1 + b)) sum w |v|
  lse         2^-17 (1 + b) + 2^-20 |lse|
  accumulate  each weight relative 2 * 2^-17 (1 + b), each of the n additions 2^-24 of the sum
"""
import numpy as np
import pytest
import torch

import paged_util as pu

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


class Setup:
    """A pool, its metadata and the handles, on both sides."""

    def __init__(self, rc, seqs, hk, dim, page, seed, spread=1.0, tokens=None, max_kv=None, max_new=None):
        self.rng = np.random.default_rng(seed)
        self.pool, self.meta = pu.make(seqs, hk, dim, page, self.rng, spread=spread)
        self.tokens = tokens if tokens is not None else int(self.meta["q_start"][-1])
        self.max_kv = max_kv if max_kv is not None else int(self.meta["kv_len"].max())
        self.max_new = max_new if max_new is not None else int(np.diff(self.meta["q_start"]).max())
        self.upload(rc)

    def upload(self, rc):
        self.cache = rc.PagedKVCache(*[dev(self.pool[k]) for k in ("kcodes", "vcodes", "kscale", "vscale")])
        self.table, self.kv_len, self.q_start = dev(self.meta["table"]), dev(self.meta["kv_len"]), dev(self.meta["q_start"])
        self.batch = rc.PagedBatch(self.table, self.kv_len, self.q_start, tokens=self.tokens, max_new=self.max_new,
                                   max_kv=self.max_kv)

    def attend(self, q, causal, stream=None):
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full(q.shape[:2], 7.0, device="cuda")
        self.cache.attend(self.batch, q, out, lse=lse, causal=causal, stream=stream)
        self.cache.sync(stream)
        return out, lse

    def check_attend(self, q, causal, got=None):
        out, lse = got if got is not None else self.attend(q.cuda(), causal)
        qn = q.float().cpu().numpy()
        ref, rlse, touched = pu.attend(self.pool, self.meta, qn, causal)
        out, lse = out.float().cpu().numpy(), lse.cpu().numpy()
        assert (out[~touched] == 7.0).all() and (lse[~touched] == 7.0).all(), "a row of no sequence was written"
        hk, hq = self.pool["kcodes"].shape[1], q.shape[1]
        for s in range(len(self.meta["kv_len"])):
            q0, q1, kv = self.meta["q_start"][s], self.meta["q_start"][s + 1], self.meta["kv_len"][s]
            for head in range(hq):
                h = head * hk // hq
                x = pu.logits(self.pool, self.meta, qn, s, h, head, causal)
                v = pu.tokens_of(self.pool, "v", self.meta["table"][s], h, kv)
                big = pu.reach(self.pool, self.meta, qn, s, h, head)
                for i in range(q1 - q0):
                    r, g, want = rlse[q0 + i, head], lse[q0 + i, head], ref[q0 + i, head]
                    if r == -np.inf:
                        assert g == -np.inf and (out[q0 + i, head] == 0).all()
                        continue
                    see = x[i] != -np.inf
                    if np.isnan(want).any():
                        assert np.isnan(out[q0 + i, head][np.isnan(want)]).all()
                        assert np.isnan(g) == np.isnan(r)
                        continue
                    assert np.isfinite(out[q0 + i, head]).all()
                    w = np.exp(x[i][see] - r)
                    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -16 * (1 + big)) * (w @ np.abs(v[see])) + 1e-30
                    err = np.abs(out[q0 + i, head] - want)
                    assert (err <= tol).all(), (s, head, i, (err / tol).max())
                    assert abs(g - r) <= 2.0 ** -17 * (1 + big) + 2.0 ** -20 * abs(r)
        return out, lse


# ------------------------------------------------------------------ rotary positions
@pytest.mark.parametrize("dim,sections", [(64, (32,)), (64, (11, 11, 10)), (128, (64,)), (128, (22, 21, 21)),
                                          (128, (0, 40, 24)), (128, (16, 16, 16, 16))])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,heads", [(1, 1), (1, 48), (37, 5), (1301, 3)])
def test_rope_axes(rc, dim, sections, dtype, n, heads):
    rng = np.random.default_rng(n + dim + len(sections))
    x = torch.from_numpy(rng.standard_normal((n, heads, dim)).astype(np.float32)).to(dtype)
    pos = rng.integers(-2 ** 31, 2 ** 31, (len(sections), n)).astype(np.int32)
    pos[:, : n // 2] = rng.integers(-1000, 200000, (len(sections), n // 2))
    for shared in (False, True):
        rope = rc.RopeAxes(sections, base=10000.0, shared_freqs=shared)
        for sign, inverse in ((1.0, False), (-1.0, True)):
            got = rc.rc_rope_axes(x.cuda(), dev(pos), rope, inverse=inverse)
            assert got.dtype == dtype
            want = pu.turn(x.double().numpy(), pos, sections, shared=shared, sign=sign)
            r = np.abs(x.double().numpy())
            r = np.repeat(r[..., 0::2] + r[..., 1::2], 2, -1)
            # the definition's own angle is rounded to 2^-53 of itself: up to 2^-22 at the farthest positions
            tol = (2.0 ** -20 + np.abs(pos).max() * 2.0 ** -52) * r + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0)
            assert (np.abs(got.double().cpu().numpy() - want) <= tol).all()


def test_rope_axes_one_axis_is_the_caches_rope(rc):
    import oracle
    rng = np.random.default_rng(3)
    x = rng.standard_normal((9, 2, 128)).astype(np.float32)
    pos = np.array([[0, 1, 2, 757, 5788, 200000, -40, 77, 12345]], np.int32)
    got = rc.rc_rope_axes(dev(x), dev(pos), rc.RopeAxes((64,))).cpu().numpy()
    for t in range(9):
        for h in range(2):
            want = oracle.rope_rows(x[t:t + 1, h].astype(np.float64), [int(pos[0, t])])[0]
            assert np.abs(got[t, h] - want).max() <= 2.0 ** -20 * 2 * np.abs(x[t, h]).max()


def test_rope_axes_strides_in_place_and_streams(rc):
    rng = np.random.default_rng(5)
    n, heads, dim = 83, 6, 128
    rope = rc.RopeAxes((24, 20, 20))
    fused = bf16(rng, n, 3 * heads, dim).cuda()       # q, k and v of a fused projection side by side
    pos = dev(rng.integers(0, 5000, (3, 200)).astype(np.int32))[:, 50:50 + n]  # a slice of a longer table
    want = rc.rc_rope_axes(fused[:, :heads].contiguous(), pos.contiguous(), rope)
    keep = fused.clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    rc.rc_rope_axes(fused[:, :heads], pos, rope, out=fused[:, :heads], stream=stream)
    stream.synchronize()
    assert torch.equal(fused[:, :heads], want)
    assert torch.equal(fused[:, heads:], keep[:, heads:])
    back = rc.rc_rope_axes(rc.rc_rope_axes(want.float(), pos, rope, inverse=True), pos, rope)
    assert (back - want.float()).abs().max() <= 2.0 ** -18 * want.float().abs().max()


def test_rope_axes_gradient_against_differences(rc):
    """dx = inverse turn of dy: the loss <dy, R x> is linear in x, so its central difference along any direction
    is exact up to the rounding of the two losses (fp32 values summed in 64 bits: 2^-20 of the terms)."""
    rng = np.random.default_rng(6)
    x, dy = (dev(rng.standard_normal((5, 3, 64)).astype(np.float32)) for _ in range(2))
    pos = dev(rng.integers(0, 90, (3, 5)).astype(np.int32))
    rope = rc.RopeAxes((12, 10, 10))
    dx = rc.rc_rope_axes(dy, pos, rope, inverse=True)
    for k in range(4):
        v = dev(rng.standard_normal((5, 3, 64)).astype(np.float32))
        f = [float((dy.double() * rc.rc_rope_axes(x + e * v, pos, rope).double()).sum()) for e in (1.0, -1.0)]
        assert abs((f[0] - f[1]) / 2 - float((dx.double() * v.double()).sum())) <= 2.0 ** -20 * 4 * float(
            (dy.abs().double() * (x.abs() + v.abs()).double()).sum()) * 2


# ------------------------------------------------------------------ write
def check_write(got, pool, meta, k, v, pos, sections):
    """Pool `pool` after the write of k, v (float64 values of the bf16 inputs)."""
    want = {n: a.copy() for n, a in pool.items()}
    p = pool["kscale"].shape[2]
    kt = pu.turn(k, pos, sections)
    kc, ks = pu.quantise(kt)
    vc, vs = pu.quantise(v)
    loose = []
    for s in range(len(meta["kv_len"])):
        q0, q1, kv = meta["q_start"][s], meta["q_start"][s + 1], meta["kv_len"][s]
        for i in range(q1 - q0):
            j = kv - (q1 - q0) + i
            page, place = meta["table"][s][j // p], j % p
            want["kcodes"][page, :, place], want["kscale"][page, :, place] = kc[q0 + i], ks[q0 + i]
            want["vcodes"][page, :, :, place], want["vscale"][page, :, place] = vc[q0 + i], vs[q0 + i]
            loose.append((page, place, q0 + i))
    assert np.array_equal(got["vcodes"], want["vcodes"]) and np.array_equal(got["vscale"], want["vscale"])
    same = got["kscale"] == want["kscale"]
    for page, place, t in loose:
        for h in range(k.shape[1]):
            if not np.isfinite(k[t, h]).all():
                assert got["kscale"][page, h, place] == 255 and (got["kcodes"][page, h, place] == 0).all()
                continue
            if not same[page, h, place]:
                m = np.abs(kt[t, h]).max() / 448.0
                near = 2.0 ** np.round(np.log2(m))
                assert abs(m / near - 1) <= 2.0 ** -20 and abs(int(got["kscale"][page, h, place]) - int(want["kscale"][page, h, place])) == 1
                continue
            a, b = got["kcodes"][page, h, place].astype(int), want["kcodes"][page, h, place].astype(int)
            oa, ob = np.where(a & 128, -(a & 127), a & 127), np.where(b & 128, -(b & 127), b & 127)
            off = np.abs(oa - ob)
            assert off.max() <= 1
            y = np.abs(kt[t, h]) * 2.0 ** (127.0 - want["kscale"][page, h, place])
            r = np.abs(k[t, h]) * 2.0 ** (127.0 - want["kscale"][page, h, place])
            r = np.repeat(r[0::2] + r[1::2], 2)
            mid = (pu.MAGS[np.minimum(np.abs(oa), np.abs(ob))] + pu.MAGS[np.maximum(np.abs(oa), np.abs(ob))]) / 2
            assert (np.abs(y - mid)[off == 1] <= (2.0 ** -20 * r)[off == 1]).all()
            got["kcodes"][page, h, place] = want["kcodes"][page, h, place]
    ok = same.copy()
    for page, place, _ in loose:
        ok[page, :, place] = True
    assert ok.all(), "a scale of an older token changed"
    touched = np.zeros(got["kscale"].shape, bool)
    for page, place, _ in loose:
        touched[page, :, place] = True
    assert np.array_equal(got["kcodes"][~touched], want["kcodes"][~touched]), "an older token's codes changed"


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("seqs", [[(1, 1)], [(1, 16), (1, 17), (0, 5), (1, 33)], [(16, 16), (15, 31), (17, 49)],
                                  [(37, 200), (1, 129), (64, 64), (130, 131)]])
def test_write(rc, dim, page, seqs):
    st = Setup(rc, seqs, 3, dim, page, seed=len(seqs) + page + dim)
    n = st.tokens
    sections = (dim // 2 - 2 * (dim // 6), dim // 6, dim // 6)
    k, v = bf16(st.rng, n, 3, dim), bf16(st.rng, n, 3, dim)
    k *= torch.from_numpy(np.exp2(st.rng.integers(-12, 12, (n, 3, 1))).astype(np.float32)).to(torch.bfloat16)
    v *= torch.from_numpy(np.exp2(st.rng.integers(-12, 12, (n, 3, 1))).astype(np.float32)).to(torch.bfloat16)
    if n > 2:
        k[1, 0] = 0            # a row of zeros
        v[1, 2] = 0
        v[2, 1, 5] = float("inf")   # a row that is not finite
        k[2, 2, 7] = float("nan")
        v[0, 0] = 60000.0      # over the largest scale: cut to 448 * 2^7
        v[0, 1] = 2.0 ** -133  # the smallest bf16
    pos = st.rng.integers(0, 200000, (3, n)).astype(np.int32)
    st.cache.write(st.batch, k.cuda(), v.cuda(), dev(pos), rc.RopeAxes(sections))
    st.cache.sync()
    got = {x: getattr(st.cache, x).cpu().numpy() for x in st.pool}
    check_write(got, st.pool, st.meta, k.double().numpy(), v.double().numpy(), pos, sections)


def test_write_takes_strided_rows(rc):
    st = Setup(rc, [(20, 50), (7, 7)], 2, 64, 16, seed=9)
    n, rope = st.tokens, rc.RopeAxes((32,))
    fused = bf16(st.rng, n, 10, 64).cuda()
    pos = dev(st.rng.integers(0, 99, (1, n)).astype(np.int32))
    st.cache.write(st.batch, fused[:, 6:8], fused[:, 8:], pos, rope)
    a = [getattr(st.cache, x).clone() for x in st.pool]
    st.upload(rc)
    st.cache.write(st.batch, fused[:, 6:8].contiguous(), fused[:, 8:].contiguous(), pos, rope)
    assert all(torch.equal(x, getattr(st.cache, y)) for x, y in zip(a, st.pool))


# ------------------------------------------------------------------ attend
SHAPES = [
    # (new, kv) of each sequence: single tokens at the borders of chunks, pages and splits
    [(1, 1)], [(1, 15), (1, 16), (1, 17), (1, 63), (1, 64), (1, 65)], [(1, 255), (1, 256), (1, 257), (1, 1500)],
    # few tokens, empty sequences among them
    [(5, 5), (0, 40), (3, 700), (2, 2), (0, 0), (8, 129)],
    # chunks
    [(17, 17), (33, 300)], [(129, 640), (1, 2000)], [(255, 255)],
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("seqs", SHAPES)
@pytest.mark.parametrize("dim,page,hk,group", [(64, 16, 2, 1), (128, 64, 1, 6), (128, 32, 2, 3), (64, 128, 1, 8), (128, 16, 1, 1)])
def test_attend(rc, seqs, causal, dim, page, hk, group):
    st = Setup(rc, seqs, hk, dim, page, seed=sum(k for _, k in seqs) + group)
    st.check_attend(bf16(st.rng, st.tokens, hk * group, dim), causal)


@pytest.mark.parametrize("group", [1, 2, 5, 16, 17, 24])
def test_attend_head_groups(rc, group):
    st = Setup(rc, [(1, 300), (3, 77)], 2, 64, 32, seed=group)
    st.check_attend(bf16(st.rng, st.tokens, 2 * group, 64), True)


def test_attend_many_splits_is_exactly_repeatable(rc):
    st = Setup(rc, [(1, 9001)], 2, 128, 64, seed=1)
    q = bf16(st.rng, 1, 16, 128)
    first = st.attend(q.cuda(), True)
    st.check_attend(q, True, first)
    for _ in range(5):
        again = st.attend(q.cuda(), True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_attend_queries_before_the_first_token_see_nothing(rc):
    """More new tokens than cached ones, causal: the first of them see nothing."""
    for new, kv in ((5, 2), (40, 3), (3, 0), (300, 129)):
        st = Setup(rc, [(new, kv), (1, 9)], 1, 64, 16, seed=new)
        st.check_attend(bf16(st.rng, st.tokens, 2, 64), True)


def test_attend_large_scores(rc):
    """Scores of some hundreds: weights of 0 and 1, maxima that move late."""
    st = Setup(rc, [(1, 500), (40, 500)], 2, 64, 16, seed=2, spread=1.0)
    st.check_attend(bf16(st.rng, st.tokens, 4, 64) * 30, True)


def test_attend_tokens_that_are_not_numbers(rc):
    """A cached token that is not finite reaches the queries that see it and no other; what lies behind a
    sequence's end in its last page reaches none."""
    for new, group in ((6, 1), (150, 1), (150, 4)):
        st = Setup(rc, [(new, new + 90)], 1, 64, 64, seed=new)
        p = 64
        j = new + 90 - new // 2          # a new token: the earlier ones do not see it
        page = st.meta["table"][0]
        for name in ("kscale", "vscale"):
            st.pool[name][page[-1], 0, (new + 90) % p:] = 255        # behind the end
        for name in ("kcodes", "vcodes"):
            x = st.pool[name]
            (x[page[-1], 0, (new + 90) % p:] if name == "kcodes" else x[page[-1], 0, :, (new + 90) % p:])[...] = 0x7f
        for name in ("kscale", "vscale"):
            keep = st.pool[name].copy()
            st.pool[name][page[j // p], 0, j % p] = 255
            codes = st.pool[name[0] + "codes"]
            old = codes.copy()
            if name == "kscale":
                codes[page[j // p], 0, j % p] = 0
            else:
                codes[page[j // p], 0, :, j % p] = 0
            st.upload(rc)
            out, _ = st.check_attend(bf16(st.rng, new, group, 64), True)
            assert np.isnan(out).any() and not np.isnan(out).all()
            st.pool[name][...], codes[...] = keep, old


def test_attend_strided_queries_and_outputs(rc):
    st = Setup(rc, [(9, 200), (140, 300)], 2, 64, 32, seed=12)
    fused = bf16(st.rng, st.tokens, 12, 64).cuda()
    out, lse = st.attend(fused[:, :8].contiguous(), True)
    wide = torch.zeros((st.tokens, 16, 64), dtype=torch.bfloat16, device="cuda")
    st.cache.attend(st.batch, fused[:, :8], wide[:, 4:12], causal=True)
    st.cache.sync()
    assert torch.equal(wide[:, 4:12], out) and not wide[:, :4].any() and not wide[:, 12:].any()


def test_attend_looser_bounds_and_rows_of_no_sequence(rc):
    """max_new, max_kv and tokens are bounds: larger ones give the same; rows outside the sequences stay."""
    st = Setup(rc, [(3, 50), (20, 170)], 2, 64, 16, seed=4, tokens=40, max_kv=176, max_new=33)
    st.check_attend(bf16(st.rng, 40, 4, 64), True)


# ------------------------------------------------------------------ accumulate
def check_scores(st, q, causal, scores=None, in_place=False):
    hk = st.pool["kcodes"].shape[1]
    width = st.max_kv + 5
    if scores is None:
        scores = st.rng.random((len(st.meta["kv_len"]), hk, width)).astype(np.float32)
    _, lse = st.attend(q.cuda(), causal)
    lse = lse.clone()
    lse[st.meta["q_start"][-1]:] = 0
    sd = dev(scores)
    out = sd if in_place else torch.full_like(sd, 7.0)
    st.cache.accumulate(st.batch, q.cuda(), lse, sd, out=None if in_place else out, causal=causal)
    st.cache.sync()
    want = pu.accumulate(st.pool, st.meta, q.float().numpy(), lse.cpu().numpy(), scores, causal)
    got = out.cpu().numpy().astype(np.float64)
    past = 7.0 if not in_place else scores[..., st.max_kv:]
    assert (got[..., st.max_kv:] == past).all(), "entries past max_kv were written"
    big = max(pu.reach(st.pool, st.meta, q.float().numpy(), s, head * hk // q.shape[1], head)
              for s in range(len(st.meta["kv_len"])) for head in range(q.shape[1]))
    n = int(np.diff(st.meta["q_start"]).max()) * q.shape[1] // hk
    tol = 2.0 ** -16 * (1 + big) * (want - scores) + 2.0 ** -24 * (n + 8) * want + 1e-30
    err = np.abs(got - want)[..., :st.max_kv]
    assert (err <= tol[..., :st.max_kv]).all(), (err / tol[..., :st.max_kv]).max()
    return out


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("seqs", SHAPES)
@pytest.mark.parametrize("dim,page,hk,group", [(64, 16, 2, 1), (128, 64, 1, 6), (128, 128, 2, 2)])
def test_accumulate(rc, seqs, causal, dim, page, hk, group):
    st = Setup(rc, seqs, hk, dim, page, seed=sum(k for _, k in seqs) + group + 1)
    check_scores(st, bf16(st.rng, st.tokens, hk * group, dim), causal, in_place=group == 6)


def test_accumulate_weights_of_a_row_add_up_to_one(rc):
    st = Setup(rc, [(150, 700), (3, 90)], 2, 64, 32, seed=8)
    q = bf16(st.rng, st.tokens, 6, 64).cuda()
    _, lse = st.attend(q, True)
    sc = torch.zeros((2, 2, st.max_kv), device="cuda")
    st.cache.accumulate(st.batch, q, lse, sc, causal=True)
    total = sc.double().sum(-1).cpu().numpy()
    assert np.abs(total[0] / (150 * 3) - 1).max() < 1e-5 and np.abs(total[1] / 9 - 1).max() < 1e-5


def test_accumulate_rows_that_saw_nothing_and_repeats(rc):
    st = Setup(rc, [(40, 3), (200, 900)], 1, 128, 64, seed=3)
    q = bf16(st.rng, st.tokens, 4, 128)
    a = check_scores(st, q, True, scores=np.zeros((2, 1, 905), np.float32))
    b = check_scores(st, q, True, scores=np.zeros((2, 1, 905), np.float32))
    assert torch.equal(a, b)


# ------------------------------------------------------------------ evict
def check_evict(rc, lens, keep, recent, page, hk=2, dim=64, scores=None, seed=0, with_scores=True):
    rng = np.random.default_rng(seed)
    kept_n = [min(k, keep) for k in lens]
    pool, meta = pu.make([(0, k) for k in lens + kept_n], hk, dim, page, rng)
    n, max_kv = len(lens), max(lens)
    table = meta["table"][:n, :max(1, -(-max_kv // page))]
    dst = np.ascontiguousarray(meta["table"][n:, :max(1, -(-max(kept_n) // page))])
    cache = rc.PagedKVCache(*[dev(pool[k]) for k in ("kcodes", "vcodes", "kscale", "vscale")])
    batch = rc.PagedBatch(dev(table), dev(np.array(lens, np.int32)), max_kv=max_kv)
    if scores is None:
        scores = rng.exponential(size=(n, hk, max_kv + 3)).astype(np.float32)
        scores[rng.random(scores.shape) < 0.3] = 0
    kept = torch.full((n, hk, keep), 99, dtype=torch.int32, device="cuda")
    sout = torch.full((n, hk, keep), 99.0, device="cuda") if with_scores else None
    length = torch.full((n,), 99, dtype=torch.int32, device="cuda")
    cache.evict(batch, dev(scores), keep=keep, recent=recent, dst_table=dev(dst), kept=kept, kv_len_out=length, scores_out=sout)
    cache.sync()
    want = {k: a.copy() for k, a in pool.items()}
    kept = kept.cpu().numpy()
    assert list(length.cpu().numpy()) == kept_n
    for s in range(n):
        for h in range(hk):
            w = pu.evict(scores[s, h], lens[s], keep, recent)
            assert list(kept[s, h]) == w + [-1] * (keep - len(w)), (s, h)
            if with_scores:
                got = sout[s, h].cpu().numpy()
                assert np.array_equal(got[:len(w)], scores[s, h][w], equal_nan=True) and (got[len(w):] == 0).all()
            for i, j in enumerate(w):
                a, b, c, d = table[s][j // page], j % page, dst[s][i // page], i % page
                for x in ("kcodes", "kscale", "vscale"):
                    want[x][c, h, d] = pool[x][a, h, b]
                want["vcodes"][c, h, :, d] = pool["vcodes"][a, h, :, b]
    for x in pool:
        assert np.array_equal(getattr(cache, x).cpu().numpy(), want[x]), x


@pytest.mark.parametrize("lens,keep,recent", [([1], 1, 0), ([1], 1, 1), ([2, 1], 1, 1), ([17, 0, 40], 16, 4), ([100, 64, 65], 64, 64),
                                              ([100, 300], 64, 0), ([1000, 33, 2049], 500, 20), ([90], 200, 10)])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_evict(rc, lens, keep, recent, page):
    check_evict(rc, lens, keep, recent, page, seed=keep + page)


def test_evict_wide_head_and_no_scores_out(rc):
    check_evict(rc, [700, 300], 256, 32, 32, hk=3, dim=128, with_scores=False)


@pytest.mark.parametrize("kind", ["equal", "zeros", "negative", "nan", "steps", "infinite"])
def test_evict_scores_of_every_kind(rc, kind):
    rng = np.random.default_rng(4)
    sc = rng.standard_normal((2, 2, 1500)).astype(np.float32)
    if kind == "equal":
        sc[:] = 0.25
    elif kind == "zeros":
        sc = np.where(rng.random(sc.shape) < 0.5, np.float32(-0.0), np.float32(0.0))
    elif kind == "nan":
        sc[rng.random(sc.shape) < 0.1] = np.nan
    elif kind == "steps":
        sc = rng.integers(0, 5, sc.shape).astype(np.float32)
    elif kind == "infinite":
        sc[rng.random(sc.shape) < 0.2] = np.inf
        sc[rng.random(sc.shape) < 0.2] = -np.inf
    check_evict(rc, [1500, 1203], 400, 30, 16, scores=sc)


def test_evict_more_scores_than_shared_memory_holds(rc):
    check_evict(rc, [50000], 777, 7, 128, hk=1)


# ------------------------------------------------------------------ together, graphs, refusals
def test_a_session(rc):
    """Prompts written and attended, weights kept up over decode steps, a cut, and further steps on the new pages,
    against the definitions fed with the same pages."""
    rng = np.random.default_rng(11)
    hk, group, dim, page, rope = 2, 3, 64, 16, rc.RopeAxes((12, 10, 10))
    cache = rc.PagedKVCache.empty(64, hk, dim, page)
    ids = list(rng.permutation(64))
    tables = np.full((2, 12), -1, np.int32)
    lens = [0, 0]
    scores = torch.zeros((2, hk, 192), device="cuda")

    def step(new):
        for s, n in enumerate(new):
            have = -(-lens[s] // page)
            lens[s] += n
            for i in range(have, -(-lens[s] // page)):
                tables[s, i] = ids.pop()
        t = sum(new)
        k, v, q = bf16(rng, t, hk, dim), bf16(rng, t, hk, dim), bf16(rng, t, hk * group, dim)
        pos = np.stack([np.concatenate([np.arange(n) + lens[s] - n for s, n in enumerate(new)])] * 3).astype(np.int32)
        meta = {"table": tables.copy(), "kv_len": np.array(lens, np.int32), "q_start": np.array([0, new[0], t], np.int32)}
        batch = rc.PagedBatch(dev(tables), dev(meta["kv_len"]), dev(meta["q_start"]), tokens=t, max_new=max(new), max_kv=max(lens))
        before = {x: getattr(cache, x).cpu().numpy() for x in ("kcodes", "vcodes", "kscale", "vscale")}
        cache.write(batch, k.cuda(), v.cuda(), dev(pos), rope)
        qd = rc.rc_rope_axes(q.cuda(), dev(pos), rope)
        out, lse = torch.zeros_like(qd), torch.zeros((t, hk * group), device="cuda")
        cache.attend(batch, qd, out, lse=lse)
        old = scores.cpu().numpy()
        cache.accumulate(batch, qd, lse, scores)
        cache.sync()
        pool = {x: getattr(cache, x).cpu().numpy() for x in before}
        check_write({x: a.copy() for x, a in pool.items()}, before, meta, k.double().numpy(), v.double().numpy(), pos, rope.sections)
        ref, rlse, _ = pu.attend(pool, meta, qd.float().cpu().numpy(), True)
        assert np.abs(out.float().cpu().numpy() - ref).max() <= 2.0 ** -7 * np.abs(ref).max() + 2.0 ** -6
        assert np.abs(lse.cpu().numpy() - rlse).max() <= 1e-4
        want = pu.accumulate(pool, meta, qd.float().cpu().numpy(), lse.cpu().numpy(), old, True)
        assert np.abs(scores.cpu().numpy() - want).max() <= 1e-4 * (1 + want.max())

    step([90, 33])
    for _ in range(3):
        step([1, 1])
    # cut to 40 tokens, the last 8 always
    keep = 40
    dst = np.array([[ids.pop() for _ in range(3)] for _ in range(2)], np.int32)
    kept = torch.zeros((2, hk, keep), dtype=torch.int32, device="cuda")
    length = torch.zeros(2, dtype=torch.int32, device="cuda")
    sout = torch.zeros((2, hk, keep), device="cuda")
    host = scores.cpu().numpy()
    cache.evict(rc.PagedBatch(dev(tables), dev(np.array(lens, np.int32)), max_kv=max(lens)), scores, keep=keep, recent=8,
                dst_table=dev(dst), kept=kept, kv_len_out=length, scores_out=sout)
    cache.sync()
    for s in range(2):
        for h in range(hk):
            w = pu.evict(host[s, h], lens[s], keep, 8)
            assert list(kept[s, h].cpu().numpy()[:len(w)]) == w
    lens = [int(x) for x in length.cpu()]
    assert lens == [40, 36]
    tables[:] = -1
    tables[:, :3] = dst
    scores.zero_()
    scores[..., :keep] = sout
    step([1, 1])
    step([20, 5])


def test_captured_calls_follow_the_metadata(rc):
    """Two graphs on one workspace, captured once, replayed in turn with other lengths and other inputs in the same tensors."""
    st = Setup(rc, [(1, 900), (1, 33)], 2, 128, 64, seed=21, max_kv=960)
    q = bf16(st.rng, 2, 12, 128).cuda()
    out, lse = torch.zeros_like(q), torch.zeros((2, 12), device="cuda")
    sc = torch.zeros((2, 2, 960), device="cuda")
    st.cache.attend(st.batch, q, out, lse=lse)
    st.cache.accumulate(st.batch, q, lse, sc)
    big = Setup(rc, [(150, 400)], 2, 128, 64, seed=22)
    big.cache = rc.PagedKVCache(big.cache.kcodes, big.cache.vcodes, big.cache.kscale, big.cache.vscale, workspace=st.cache.workspace)
    qb = bf16(big.rng, 150, 12, 128).cuda()
    ob, lb = torch.zeros_like(qb), torch.zeros((150, 12), device="cuda")
    big.cache.attend(big.batch, qb, ob, lse=lb)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        st.cache.attend(st.batch, q, out, lse=lse)
        st.cache.accumulate(st.batch, q, lse, sc)
    with torch.cuda.graph(g2):
        big.cache.attend(big.batch, qb, ob, lse=lb)
    for lens in ([900, 33], [1, 960 - 64], [257, 2], [0, 64]):
        need = [-(-x // 64) for x in lens]
        if lens[1] > 33:
            st.meta["table"][[0, 1]] = st.meta["table"][[1, 0]]
        st.meta["kv_len"][:] = lens
        st.table.copy_(dev(st.meta["table"]))
        st.kv_len.copy_(dev(st.meta["kv_len"]))
        ok = all((st.meta["table"][s][:need[s]] >= 0).all() for s in range(2))
        assert ok
        qn = bf16(st.rng, 2, 12, 128)
        q.copy_(qn)
        sc.zero_()
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        st.check_attend(qn, True, (out, lse))
        want = pu.accumulate(st.pool, st.meta, qn.float().numpy(), lse.cpu().numpy(), np.zeros((2, 2, 960)), True)
        assert np.abs(sc.cpu().numpy() - want).max() <= 1e-4
        if lens[1] > 33:
            st.meta["table"][[0, 1]] = st.meta["table"][[1, 0]]
    big.check_attend(qb.cpu(), True, (ob, lb))
    st.cache.sync()


def test_bad_metadata_is_reported_and_the_rest_is_right(rc):
    """Lengths and pages out of the bounds: found on the device, nothing is touched outside, other sequences are right."""
    st = Setup(rc, [(2, 70), (3, 90), (1, 64)], 2, 64, 16, seed=31)
    q = bf16(st.rng, st.tokens, 4, 64).cuda()
    good, glse = st.attend(q, True)
    sc = torch.zeros((3, 2, st.max_kv), device="cuda")
    for what, value in (("kv_len", 91), ("kv_len", -1), ("q_start", 7), ("table", 10 ** 6), ("table", -5)):
        t = {"kv_len": st.kv_len, "q_start": st.q_start, "table": st.table}[what]
        old = t.clone()
        if what == "table":
            t[1, 2] = value
        else:
            t[1] = value
        out, lse = torch.zeros_like(q), torch.zeros((st.tokens, 4), device="cuda")
        st.cache.attend(st.batch, q, out, lse=lse)
        with pytest.raises(rc.RcError) as e:
            st.cache.sync()
        assert e.value.status == rc.RC_ERR_ARG
        assert torch.equal(out[5], good[5])
        st.cache.accumulate(st.batch, q, glse, sc)
        with pytest.raises(rc.RcError):
            st.cache.sync()
        if what == "table":
            kept, length = torch.zeros((3, 2, 8), dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
            before = st.cache.kcodes.clone()
            bad = torch.full((3, 1), 10 ** 6, dtype=torch.int32, device="cuda")
            st.cache.evict(st.batch, sc, keep=8, recent=2, dst_table=bad, kept=kept, kv_len_out=length)
            with pytest.raises(rc.RcError):
                st.cache.sync()
            assert torch.equal(before, st.cache.kcodes)
        t.copy_(old)
        st.cache.sync()
    out, lse = st.attend(q, True)
    assert torch.equal(out, good)
    # a write of more tokens than the sequence has
    k = bf16(st.rng, st.tokens, 2, 64).cuda()
    before = st.cache.kcodes.clone()
    st.kv_len[:] = 0
    st.cache.write(st.batch, k, k, torch.zeros((1, st.tokens), dtype=torch.int32, device="cuda"), rc.RopeAxes((32,)))
    with pytest.raises(rc.RcError):
        st.cache.sync()
    assert torch.equal(before, st.cache.kcodes)


def test_a_call_on_another_stream(rc):
    st = Setup(rc, [(1, 3000), (1, 10)], 2, 64, 16, seed=41)
    q = bf16(st.rng, 2, 4, 64)
    stream = torch.cuda.Stream()
    qd = q.cuda()
    stream.wait_stream(torch.cuda.current_stream())
    st.check_attend(q, True, st.attend(qd, True, stream=stream))


def test_pools_past_32_bit_offsets(rc):
    """Pages whose codes lie over 4 GB into the pool."""
    pages, hk, page, dim = 36000, 8, 128, 128
    cache = rc.PagedKVCache.empty(pages, hk, dim, page)
    rng = np.random.default_rng(51)
    ids = np.array([[pages - 1, 0, pages - 2]], np.int32)
    n = 300
    k, v, q = bf16(rng, n, hk, dim).cuda(), bf16(rng, n, hk, dim).cuda(), bf16(rng, n, hk, dim).cuda()
    pos = torch.arange(n, dtype=torch.int32, device="cuda")[None]
    rope = rc.RopeAxes((64,))
    batch = rc.PagedBatch(dev(ids), dev(np.array([n], np.int32)), dev(np.array([0, n], np.int32)), tokens=n, max_new=n, max_kv=n)
    small = rc.PagedKVCache.empty(8, hk, dim, page)
    sb = rc.PagedBatch(dev(np.array([[3, 1, 2]], np.int32)), dev(np.array([n], np.int32)), dev(np.array([0, n], np.int32)), tokens=n,
                       max_new=n, max_kv=n)
    res = []
    for c, b, to in ((cache, batch, [[pages - 3]]), (small, sb, [[5]])):
        c.write(b, k, v, pos, rope)
        out, lse, sc = torch.zeros_like(q), torch.zeros((n, hk), device="cuda"), torch.zeros((1, hk, n), device="cuda")
        c.attend(b, q, out, lse=lse)
        c.accumulate(b, q, lse, sc)
        kept, length = torch.zeros((1, hk, 100), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        c.evict(b, sc, keep=100, recent=10, dst_table=dev(np.array(to, np.int32)), kept=kept, kv_len_out=length)
        c.sync()
        res.append((out, lse, sc, kept, c.kcodes[to[0][0]].clone(), c.vcodes[to[0][0]].clone(), c.vscale[to[0][0]].clone()))
    assert all(torch.equal(a, b) for a, b in zip(*res))
    assert res[0][4].any()


def test_injected_launch_failure_changes_nothing(rc, monkeypatch):
    st = Setup(rc, [(1, 40)], 1, 64, 16, seed=61)
    q = bf16(st.rng, 1, 2, 64).cuda()
    out = torch.full_like(q, 7.0)
    monkeypatch.setenv("RC_FAULT_INJECT", "launch")
    with pytest.raises(rc.RcError) as e:
        st.cache.attend(st.batch, q, out)
    assert e.value.status == rc.RC_ERR_CUDA
    monkeypatch.delenv("RC_FAULT_INJECT")
    torch.cuda.synchronize()
    assert (out == 7).all()
    st.cache.attend(st.batch, q, out)
    st.cache.sync()


def test_refused_tensors(rc):
    st = Setup(rc, [(2, 40)], 2, 64, 16, seed=71)
    q = bf16(st.rng, 2, 4, 64).cuda()
    out = torch.zeros_like(q)
    with pytest.raises(TypeError):
        st.cache.attend(st.batch, q.float(), out)
    with pytest.raises(TypeError):
        st.cache.attend(st.batch, q.cpu(), out)
    with pytest.raises(ValueError):
        st.cache.attend(st.batch, q[:1], out)
    with pytest.raises(ValueError):
        st.cache.attend(st.batch, q.transpose(0, 1).contiguous().transpose(0, 1), out)
    with pytest.raises(rc.RcError):     # 3 query heads on 2 KV heads
        st.cache.attend(st.batch, q[:, :3].contiguous(), out[:, :3].contiguous())
    flat = torch.zeros(2 * 4 * 64 + 1, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(rc.RcError):     # not 16-byte aligned
        st.cache.attend(st.batch, flat[1:].view(2, 4, 64), out)
    rope = rc.RopeAxes((32,))
    pos = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        rc.rc_rope_axes(q, pos.long(), rope)
    with pytest.raises(ValueError):
        rc.rc_rope_axes(q, pos, rc.RopeAxes((64,)))
    wide = torch.zeros((3, 4, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):     # shifted over itself
        rc.rc_rope_axes(wide[:2], pos, rope, out=wide[1:])
    st.cache.sync()


# ------------------------------------------------------------------ borders of the kernels' shares of the work
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [1, 7, 8, 9, 16])
@pytest.mark.parametrize("kv", [512, 513, 1279, 4351, 8193])
def test_attend_few_rows_splits(rc, kv, group, dim):
    st = Setup(rc, [(1, kv)], 1, dim, 64, seed=kv + group)
    st.check_attend(bf16(st.rng, 1, group, dim), True)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("seqs,group", [([(40, 3000)], 1), ([(17, 513), (17, 4097)], 1), ([(100, 2500)], 3), ([(257, 1300), (1, 5)], 1)])
def test_attend_some_rows_splits(rc, seqs, group, dim, causal):
    st = Setup(rc, seqs, 1, dim, 32, seed=sum(k for _, k in seqs) + group)
    st.check_attend(bf16(st.rng, st.tokens, group, dim), causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim,seqs,group", [
    (64, [(8, 300)], 4), (128, [(33, 300)], 1), (128, [(16, 257), (3, 700)], 3),   # 32, 33 and 48 rows
    (64, [(500, 700)], 2), (128, [(385, 385)], 1), (128, [(431, 1100), (33, 33)], 2),  # several blocks of rows
])
def test_accumulate_many_rows(rc, seqs, group, dim, causal):
    st = Setup(rc, seqs, 1, dim, 16, seed=sum(k for _, k in seqs) + group + 2)
    check_scores(st, bf16(st.rng, st.tokens, group, dim), causal, in_place=dim == 64)


def test_two_caches_on_the_same_pages_at_once(rc):
    """Two streams, each with a workspace of its own, read one pool's pages at the same time."""
    st = Setup(rc, [(1, 6000), (60, 900), (1, 77)], 2, 128, 32, seed=81)
    other = rc.PagedKVCache(st.cache.kcodes, st.cache.vcodes, st.cache.kscale, st.cache.vscale)
    q = bf16(st.rng, st.tokens, 6, 128).cuda()
    want, wlse = st.attend(q, True)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    res = []
    for i in range(8):
        cache = (st.cache, other)[i % 2]
        out, lse = torch.zeros_like(want), torch.zeros_like(wlse)
        streams[i % 2].wait_stream(torch.cuda.current_stream())
        cache.attend(st.batch, q, out, lse=lse, stream=streams[i % 2])
        res.append((out, lse))
    for cache, stream in zip((st.cache, other), streams):
        cache.sync(stream=stream)
    torch.cuda.synchronize()
    n = st.meta["q_start"][-1]
    assert all(torch.equal(o[:n], want[:n]) and torch.equal(x[:n], wlse[:n]) for o, x in res)


def test_a_wait_that_runs_out_is_reported_and_forgotten(rc):
    """With a limit of 0 the first wait that is not already over gives up: the call reports RC_ERR_TIMEOUT, frees what
    it holds and the next call with the limit restored is right."""
    st = Setup(rc, [(300, 2000)], 2, 128, 64, seed=91)
    q = bf16(st.rng, st.tokens, 4, 128)
    good, lse = st.attend(q.cuda(), True)
    sc = torch.zeros((1, 2, st.max_kv), device="cuda")
    st.cache.accumulate(st.batch, q.cuda(), lse, sc)
    st.cache.sync()
    for call in (lambda: st.cache.attend(st.batch, q.cuda(), torch.zeros_like(good)),
                 lambda: st.cache.accumulate(st.batch, q.cuda(), lse, sc, out=torch.zeros_like(sc))):
        rc.rc_paged_set_wait_limit(0)
        try:
            call()
            with pytest.raises(rc.RcError) as e:
                st.cache.sync()
        finally:
            rc.rc_paged_set_wait_limit(2_000_000_000)
        assert e.value.status == rc.RC_ERR_TIMEOUT
        st.cache.sync()
        again, lse2 = st.attend(q.cuda(), True)
        assert torch.equal(again, good) and torch.equal(lse2, lse)
        sc2 = torch.zeros_like(sc)
        st.cache.accumulate(st.batch, q.cuda(), lse, sc2)
        st.cache.sync()
        assert torch.equal(sc2, sc)


@pytest.mark.parametrize("dim", [64, 128])
def test_pages_on_a_16_byte_boundary(rc, dim):
    """Pages whose address is a multiple of 16 bytes but not of 32 give the same bits."""
    st = Setup(rc, [(3, 200), (150, 600)], 2, dim, 16, seed=95)
    q = bf16(st.rng, st.tokens, 4, dim).cuda()

    def moved(t):
        flat = torch.zeros(t.numel() + 64, dtype=torch.uint8, device="cuda")
        at = 16 + (-flat.data_ptr()) % 32
        new = flat[at:at + t.numel()].view(t.shape)
        assert new.data_ptr() % 32 == 16
        return new.copy_(t)

    res = []
    for cache in (st.cache, rc.PagedKVCache(*(moved(getattr(st.cache, x)) for x in ("kcodes", "vcodes", "kscale", "vscale")))):
        out, lse = torch.zeros_like(q), torch.zeros((st.tokens, 4), device="cuda")
        sc = torch.zeros((2, 2, st.max_kv), device="cuda")
        cache.attend(st.batch, q, out, lse=lse)
        cache.accumulate(st.batch, q, lse, sc)
        k = bf16(np.random.default_rng(1), st.tokens, 2, dim).cuda()
        cache.write(st.batch, k, k, torch.zeros((1, st.tokens), dtype=torch.int32, device="cuda"), rc.RopeAxes((dim // 2,)))
        cache.sync()
        res.append((out, lse, sc, cache.kcodes, cache.vcodes, cache.kscale, cache.vscale))
    assert all(torch.equal(a, b) for a, b in zip(*res))


@pytest.mark.parametrize("dim,sections", [(128, (22, 21, 21)), (64, (32,))])
def test_write_codes_are_those_of_the_exact_turn(rc, dim, sections):
    """cos and sin are good to 2^-25.6, all else to far less: a code may be the neighbour's only where the exact value is
    within 2^-25 (|a| + |b|) of the middle between the two (with fp32 sums that is 2^-22)."""
    st = Setup(rc, [(900, 900)], 6, dim, 32, seed=97)
    k = bf16(st.rng, 900, 6, dim)
    pos = st.rng.integers(0, 200000, (len(sections), 900)).astype(np.int32)
    st.cache.write(st.batch, k.cuda(), k.cuda(), dev(pos), rc.RopeAxes(sections))
    st.cache.sync()
    table = st.meta["table"][0]
    at = np.arange(900)
    got = st.cache.kcodes.cpu().numpy()[table[at // 32], :, at % 32].astype(int)
    scale = st.cache.kscale.cpu().numpy()[table[at // 32], :, at % 32]
    x = k.double().numpy()
    y = pu.turn(x, pos, sections)
    want, wscale = pu.quantise(y)
    assert np.array_equal(scale, wscale)
    off = np.nonzero(got != want)
    factor = 2.0 ** (127.0 - wscale[off[:2]])
    r = (np.abs(x[..., 0::2]) + np.abs(x[..., 1::2])).repeat(2, -1)[off] * factor
    mid = (pu.E4M3[got[off]] + pu.E4M3[want[off].astype(int)]) / 2
    assert (np.abs(y[off] * factor - mid) <= 2.0 ** -25 * r).all()


def test_write_at_the_ends_of_the_positions(rc):
    """Negative positions and those at the ends of int32: K's codes are those of rc_rope_axes' fp32 rows, but for roundings
    (fp32 sums are within 2^-22 (|a| + |b|) and rounded to 2^-24 once more: two codes at most one step apart)."""
    st = Setup(rc, [(64, 64)], 2, 128, 16, seed=98)
    pos = st.rng.integers(-2 ** 31, 2 ** 31, (3, 64)).astype(np.int32)
    pos[:, 0], pos[:, 1], pos[:, 2] = -2 ** 31, 2 ** 31 - 1, -1
    k, rope = bf16(st.rng, 64, 2, 128), rc.RopeAxes((22, 21, 21))
    st.cache.write(st.batch, k.cuda(), k.cuda(), dev(pos), rope)
    st.cache.sync()
    y = rc.rc_rope_axes(k.float().cuda(), dev(pos), rope).cpu().double().numpy()
    table, at = st.meta["table"][0], np.arange(64)
    got = pu.E4M3[st.cache.kcodes.cpu().numpy()[table[at // 16], :, at % 16]]
    scale = pu.scale_value(st.cache.kscale.cpu().numpy()[table[at // 16], :, at % 16])[..., None]
    # half a step of E4M3 (2^-4 relative, 2^-10 at least) and the fp32 rounding
    assert (np.abs(got * scale - y) <= np.maximum(np.abs(y) * 2.0 ** -4, scale * 2.0 ** -10) * (1 + 2.0 ** -12) + 2.0 ** -21 * np.abs(
        k.double().numpy()).max()).all()


def test_calls_from_two_threads(rc):
    """Each thread its own stream and workspace, on one pool's pages."""
    import threading
    st = Setup(rc, [(1, 3000), (70, 500)], 2, 64, 16, seed=99)
    q = bf16(st.rng, st.tokens, 4, 64).cuda()
    want, wlse = st.attend(q, True)
    sc = torch.zeros((2, 2, st.max_kv), device="cuda")
    st.cache.accumulate(st.batch, q, wlse, sc)
    torch.cuda.synchronize()
    n, bad = st.meta["q_start"][-1], []

    def work():
        try:
            cache = rc.PagedKVCache(st.cache.kcodes, st.cache.vcodes, st.cache.kscale, st.cache.vscale)
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(30):
                    out, lse, s2 = torch.zeros_like(want), torch.zeros_like(wlse), torch.zeros_like(sc)
                    cache.attend(st.batch, q, out, lse=lse)
                    cache.accumulate(st.batch, q, wlse, s2)
                    cache.sync()
                    if not (torch.equal(out[:n], want[:n]) and torch.equal(lse[:n], wlse[:n]) and torch.equal(s2, sc)):
                        bad.append("results differ")
        except Exception as e:  # noqa: BLE001 (reported below)
            bad.append(repr(e))

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad[:3]


FIRST_IN_A_GRAPH = """
import torch, fp8_ring_kv_cache_gb300 as rc
c = rc.PagedKVCache.empty(20, 2, 64, 16)
q = torch.randn(70, 4, 64, device="cuda").to(torch.bfloat16)
i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
pos, rope = torch.arange(70, dtype=torch.int32, device="cuda")[None], rc.RopeAxes((32,))
one = rc.PagedBatch(i32(*range(10))[None], i32(1), i32(0, 1), tokens=1, max_new=1, max_kv=160)
c.write(one, q[:1, :2], q[:1, 2:], pos[:, :1], rope)     # one token: other kernels than below
out, lse, sc = torch.zeros_like(q), torch.zeros(70, 4, device="cuda"), torch.zeros(1, 2, 160, device="cuda")
c.attend(one, q[:1], out[:1], lse=lse[:1])
c.sync()
many = rc.PagedBatch(i32(*range(10))[None], i32(70), i32(0, 70), tokens=70, max_new=70, max_kv=160)
kept, n, dst = torch.zeros(1, 2, 40, dtype=torch.int32, device="cuda"), i32(0), i32(10, 11, 12)[None]
def run():
    sc.zero_()
    c.write(many, q[:, :2], q[:, 2:], pos, rope)
    c.attend(many, q, out, lse=lse)
    c.accumulate(many, q, lse, sc)
    c.evict(many, sc, keep=40, recent=4, dst_table=dst, kept=kept, kv_len_out=n)
s = torch.cuda.Stream()
g = torch.cuda.CUDAGraph()
with torch.cuda.stream(s):
    with torch.cuda.graph(g, stream=s):
        run()
g.replay()
c.sync()
torch.cuda.synchronize()
a = [x.clone() for x in (out, lse, sc, kept, n, c.kcodes, c.vcodes)]
run()
c.sync()
assert all(torch.equal(x, y) for x, y in zip(a, (out, lse, sc, kept, n, c.kcodes, c.vcodes)))
print("ok")
"""


def test_kernels_first_used_inside_a_graph(rc):
    """A process whose first call of many rows, and of accumulate and evict, is a captured one."""
    import pathlib
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", FIRST_IN_A_GRAPH], cwd=pathlib.Path(__file__).parents[1], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "ok" in r.stdout, r.stderr[-2000:]

"""Edges of the paged-cache calls on the GPU: streams other than the current one, tensors that share memory, rows that are
switched off, borders of a row's scale.  Tolerances and definitions are those of tests/test_gpu_paged.py and
tests/paged_util.py."""
import gc

import numpy as np
import pytest
import torch

import paged_util as pu
from test_gpu_paged import Setup, bf16, check_scores, dev, rc  # noqa: F401 (rc: the fixture)

pytestmark = pytest.mark.gpu


BUSY = 200_000_000  # cycles that a stream is kept busy for: about a tenth of a second


# ------------------------------------------------------------------ streams
def test_a_new_cache_is_ready_for_any_stream(rc):  # noqa: F811
    """The workspace of a cache built while the current stream is busy, in a block of memory that was used before, is
    zeroed before the constructor returns: a split call on another stream, which nothing orders behind the fill, is right."""
    st = Setup(rc, [(1, 6000), (1, 3000)], 2, 128, 64, seed=1)
    q = bf16(st.rng, 2, 12, 128).cuda()
    want, wlse = st.attend(q, True)
    out, lse = torch.zeros_like(want), torch.zeros_like(wlse)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    gc.collect()
    torch.cuda.empty_cache()  # the only free block of the size is the one that follows
    junk = torch.full((rc.RC_PAGED_WORKSPACE_BYTES,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    at = junk.data_ptr()
    del junk
    torch.cuda._sleep(BUSY)
    cache = rc.PagedKVCache(st.cache.kcodes, st.cache.vcodes, st.cache.kscale, st.cache.vscale)
    assert cache.workspace.data_ptr() == at, "the block was not used again: the test shows nothing"
    cache.attend(st.batch, q, out, lse=lse, stream=stream)
    cache.sync(stream)
    assert torch.equal(out, want) and torch.equal(lse, wlse)


def test_empty_pages_are_ready_for_any_stream(rc):  # noqa: F811
    """The pages of `empty` keep what another stream writes right after."""
    st = Setup(rc, [(70, 70), (16, 16)], 2, 64, 16, seed=2)
    k, rope = bf16(st.rng, 86, 2, 64).cuda(), rc.RopeAxes((32,))
    pos = torch.arange(86, dtype=torch.int32, device="cuda")[None]
    pages = st.cache.pages
    plain = rc.PagedKVCache.empty(pages, 2, 64, 16)
    plain.write(st.batch, k, k, pos, rope)
    plain.sync()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    cache = rc.PagedKVCache.empty(pages, 2, 64, 16)
    cache.write(st.batch, k, k, pos, rope, stream=stream)
    torch.cuda.synchronize()
    for x in ("kcodes", "vcodes", "kscale", "vscale"):
        assert torch.equal(getattr(cache, x), getattr(plain, x)), x


def test_layers_share_a_workspace(rc):  # noqa: F811
    """Caches of `empty` with one workspace, called in turn on one stream, and ready for any: the bits of separate ones."""
    st = Setup(rc, [(1, 5000), (90, 700)], 2, 64, 16, seed=10)
    n, pages, rope = st.tokens, st.cache.pages, rc.RopeAxes((32,))
    k, q = bf16(st.rng, n, 2, 64).cuda(), bf16(st.rng, n, 4, 64).cuda()
    pos = torch.arange(n, dtype=torch.int32, device="cuda")[None]
    stream = torch.cuda.Stream()
    keys = [k * (layer + 1) for layer in range(3)]
    res = []
    for shared in (False, True):
        caches = []
        torch.cuda.synchronize()
        for layer in range(3):
            torch.cuda._sleep(BUSY // 10)
            caches.append(rc.PagedKVCache.empty(pages, 2, 64, 16, workspace=caches[0].workspace if shared and caches else None))
            caches[-1].write(st.batch, keys[layer], k, pos, rope, stream=stream)
            torch.cuda.synchronize()
        assert len({c.workspace.data_ptr() for c in caches}) == (1 if shared else 3)
        for c in caches:
            out, lse = torch.zeros_like(q), torch.zeros((n, 4), device="cuda")
            c.attend(st.batch, q, out, lse=lse)
            res.append((c.kcodes, c.vcodes, out, lse))
        torch.cuda.synchronize()
    for a, b in zip(res[:3], res[3:]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    with pytest.raises(ValueError):
        rc.PagedKVCache.empty(4, 2, 64, 16, workspace=caches[0].workspace[1:])


def test_a_cache_built_inside_a_capture(rc):  # noqa: F811
    """Its fill is a part of the graph."""
    st = Setup(rc, [(1, 3000)], 2, 64, 16, seed=3)
    q = bf16(st.rng, 1, 4, 64).cuda()
    want, wlse = st.attend(q, True)
    out, lse = torch.zeros_like(want), torch.zeros_like(wlse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache = rc.PagedKVCache(st.cache.kcodes, st.cache.vcodes, st.cache.kscale, st.cache.vscale)
        cache.attend(st.batch, q, out, lse=lse)
    for _ in range(2):
        out.zero_()
        graph.replay()
        cache.sync()
        assert torch.equal(out, want) and torch.equal(lse, wlse)


def turned(rc):  # noqa: F811
    rng = np.random.default_rng(4)
    x = bf16(rng, 4096, 8, 128).cuda()
    pos = torch.arange(4096, dtype=torch.int32, device="cuda")[None]
    rope = rc.RopeAxes((64,))
    want = rc.rc_rope_axes(x, pos, rope, out=torch.empty_like(x))
    torch.cuda.synchronize()
    gc.collect()
    torch.cuda.empty_cache()
    return x, pos, rope, want


@pytest.mark.parametrize("handle", [False, True])
def test_rope_axes_result_on_another_stream_while_the_current_one_is_busy(rc, handle):  # noqa: F811
    """The result's memory is not a block that the current stream has still to write."""
    x, pos, rope, want = turned(rc)
    stream = torch.cuda.Stream()
    junk = torch.empty_like(want)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    junk.fill_(7)
    del junk
    out = rc.rc_rope_axes(x, pos, rope, stream=stream.cuda_stream if handle else stream)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_rope_axes_result_that_is_dropped(rc):  # noqa: F811
    """Its memory is not handed out again on the current stream while the call's kernel has still to write it, nor on the
    call's stream while the current one has still to read it."""
    x, pos, rope, want = turned(rc)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(BUSY)
    out = rc.rc_rope_axes(x, pos, rope, stream=stream)
    del out
    other = torch.full_like(want, 3.0)
    torch.cuda.synchronize()
    assert (other == 3).all()
    out = rc.rc_rope_axes(x, pos, rope, stream=stream)
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda._sleep(BUSY)
    copy = out.clone()
    del out
    with torch.cuda.stream(stream):
        again = torch.full_like(want, 5.0)
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and (again == 5).all()


def test_rope_axes_result_on_the_default_streams_handle(rc):  # noqa: F811
    x, pos, rope, want = turned(rc)
    assert torch.equal(rc.rc_rope_axes(x, pos, rope, stream=torch.cuda.default_stream().cuda_stream), want)


# ------------------------------------------------------------------ tensors that share memory
def test_rope_axes_from_one_slice_of_the_rows_to_another(rc):  # noqa: F811
    """Queries of a fused projection's rows turned into the place next to them: no element is shared, and none but the
    result's changes.  One that does share some is refused."""
    rng = np.random.default_rng(7)
    n, heads = 61, 4
    rope, pos = rc.RopeAxes((24, 20, 20)), dev(rng.integers(0, 9000, (3, n)).astype(np.int32))
    fused = bf16(rng, n, 3 * heads, 128).cuda()
    before = fused.clone()
    want = rc.rc_rope_axes(fused[:, :heads].contiguous(), pos, rope)
    rc.rc_rope_axes(fused[:, :heads], pos, rope, out=fused[:, 2 * heads:])
    assert torch.equal(fused[:, 2 * heads:], want) and torch.equal(fused[:, :2 * heads], before[:, :2 * heads])
    flat = fused.view(-1)
    apart = flat[:n * 2 * heads * 128].view(n, 2 * heads, 128)[:, :heads]   # rows at another distance, over the same memory
    for out in (fused[:, heads - 1:2 * heads - 1], apart):
        with pytest.raises(ValueError):
            rc.rc_rope_axes(fused[:, :heads], pos, rope, out=out)
    assert torch.equal(fused[:, 2 * heads:], want) and torch.equal(fused[:, :2 * heads], before[:, :2 * heads])


def test_scores_and_results_between_each_others_rows(rc):  # noqa: F811
    """Queries and results that alternate in one buffer are as good as separate ones; over each other they are refused."""
    st = Setup(rc, [(1, 300), (40, 200)], 2, 64, 16, seed=8)
    n, heads = st.tokens, 4
    both = torch.zeros((n, 2 * heads, 64), dtype=torch.bfloat16, device="cuda")
    both[:, :heads] = bf16(st.rng, n, heads, 64).cuda()
    want, lse = st.attend(both[:, :heads].contiguous(), True)
    st.cache.attend(st.batch, both[:, :heads], both[:, heads:])
    st.cache.sync()
    assert torch.equal(both[:, heads:], want)
    scores = torch.zeros((4, 2, st.max_kv), device="cuda")
    kept, length = torch.zeros((2, 2, 8), dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    dst = torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    for call in (lambda: st.cache.attend(st.batch, both[:, :heads], both[:, heads - 1:2 * heads - 1]),
                 lambda: st.cache.accumulate(st.batch, both[:, :heads], lse, scores[:2], out=scores[1:3]),
                 lambda: st.cache.evict(st.batch, scores[:2], keep=8, recent=2, dst_table=dst, kept=kept, kv_len_out=length,
                                        scores_out=scores.view(-1)[:32].view(2, 2, 8))):
        with pytest.raises(rc.RcError) as e:
            call()
        assert e.value.status == rc.RC_ERR_ARG
    st.cache.accumulate(st.batch, both[:, :heads], lse, scores[:2], out=scores[2:])
    st.cache.sync()
    assert scores[2:].any() and not scores[:2].any()


@pytest.mark.parametrize("lens,keep", [([5000, 40, 0, 3000], 700), ([33, 20], 64), ([0, 0], 5), ([60000], 50)])
def test_evict_shortens_the_lengths_in_place(rc, lens, keep):  # noqa: F811
    """kv_len_out may be the batch's kv_len: every head selects among the tokens that there were."""
    hk, page, n = 16, 32, len(lens)
    rng = np.random.default_rng(5)
    left = [min(x, keep) for x in lens]
    pool, meta = pu.make([(0, x) for x in lens + left], hk, 64, page, rng)
    table, dst = meta["table"][:n], np.ascontiguousarray(meta["table"][n:, :max(1, -(-max(left) // page))])
    scores = dev(rng.exponential(size=(n, hk, max(lens) + 1)).astype(np.float32))
    res = []
    for shared in (False, True):
        cache = rc.PagedKVCache(*(dev(pool[x]) for x in ("kcodes", "vcodes", "kscale", "vscale")))
        kv_len = dev(np.array(lens, np.int32))
        batch = rc.PagedBatch(dev(table), kv_len, max_kv=max(lens))
        kept = torch.full((n, hk, keep), 99, dtype=torch.int32, device="cuda")
        out = kv_len if shared else torch.full_like(kv_len, 99)
        cache.evict(batch, scores, keep=keep, recent=min(keep, 16), dst_table=dev(dst), kept=kept, kv_len_out=out)
        cache.sync()
        assert out.tolist() == left
        res.append((kept, cache.kcodes, cache.vcodes, cache.kscale, cache.vscale))
    assert all(torch.equal(a, b) for a, b in zip(*res))
    for s in range(n):
        w = pu.evict(scores[s, hk - 1].cpu().numpy(), lens[s], keep, min(keep, 16))
        assert res[0][0][s, hk - 1].tolist() == w + [-1] * (keep - len(w))


def test_evict_with_bad_lengths_in_place(rc):  # noqa: F811
    """A length out of bounds is reported and becomes 0; the other sequences are cut."""
    st = Setup(rc, [(0, 90), (0, 70), (0, 80)], 2, 64, 16, seed=6, max_kv=90)
    st.kv_len[1] = 91
    kept = torch.zeros((3, 2, 20), dtype=torch.int32, device="cuda")
    scores = torch.rand((3, 2, 90), device="cuda")
    dst = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")  # no page of the pool: nothing is copied
    st.cache.evict(st.batch, scores, keep=20, recent=4, dst_table=dst, kept=kept, kv_len_out=st.kv_len)
    with pytest.raises(rc.RcError):
        st.cache.sync()
    assert st.kv_len.tolist() == [20, 0, 20] and (kept[1] == -1).all() and (kept[0] >= 0).all()


# ------------------------------------------------------------------ accumulate: rows that are switched off
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows", [8, 16, 24, 48, 1000])
def test_accumulate_rows_switched_off_add_nothing(rc, rows, dim, causal):  # noqa: F811
    """A row whose lse is -infinity adds nothing, whatever its query holds (NaN, infinities) and whatever it would see (a
    cached token that is not a number): every entry is what the other rows make it.  Three sequences: some rows off; all
    rows off; all off, with cached tokens that are not numbers.  With a token that is not a number and a row that sees it,
    its entry is NaN and no other."""
    group = 2
    n = rows // group
    st = Setup(rc, [(n, n + 150), (n, n + 90), (n, n + 40)], 2, dim, 16, seed=rows + dim)
    q = bf16(st.rng, st.tokens, 2 * group, dim)
    off = st.rng.random((st.tokens, 2 * group)) < 0.4
    off[n:] = True
    bad = [(0, 20), (0, n + 149), (2, 7), (2, n + 3), (2, n + 39)]  # (sequence, cached token)
    for s, j in bad:
        page = st.meta["table"][s][j // 16]
        st.pool["kscale"][page, :, j % 16] = 255
        st.pool["kcodes"][page, :, j % 16] = 0
    st.upload(rc)
    # the rows that are on: any finite lse (the weights then do not add up to 1)
    lse = (3 + st.rng.random((st.tokens, 2 * group))).astype(np.float32)
    lse[off] = -np.inf
    q[torch.from_numpy(off)] = torch.tensor([float("nan"), float("inf"), float("-inf"), 3e38])[
        torch.from_numpy(st.rng.integers(0, 4, (int(off.sum()), dim)))].to(torch.bfloat16)
    scores = st.rng.random((3, 2, st.max_kv)).astype(np.float32)
    out = torch.full((3, 2, st.max_kv), 7.0, device="cuda")
    st.cache.accumulate(st.batch, q.cuda(), dev(lse), dev(scores), out=out, causal=causal)
    st.cache.sync()
    got = out.cpu().numpy()
    qn = np.where(off[..., None], 0.0, q.float().numpy())
    assert np.array_equal(got[1], scores[1]) and np.array_equal(got[2], scores[2])
    want = pu.accumulate(st.pool, st.meta, qn, lse, scores, causal)[0]
    kv = n + 150
    nan = np.isnan(want)
    # (the last token is seen by the last row alone when causal)
    for h in range(2):
        assert nan[h, 20] and nan[h].sum() == 1 + (not causal or not off[n - 1, h * group:(h + 1) * group].all())
    assert np.array_equal(np.isnan(got[0]), nan)
    big = max(pu.reach(st.pool, st.meta, qn, 0, head // group, head) for head in range(2 * group))
    tol = 2.0 ** -16 * (1 + big) * (want - scores[0]) + 2.0 ** -24 * (rows + 8) * want
    past = want > np.finfo(np.float32).max  # weights of exp(100) and more: over what fp32 holds, which rounds to infinity
    assert (got[0][past] == np.inf).all()
    over = np.argwhere(~nan & ~past & ~(np.abs(got[0] - want) <= tol))
    assert not len(over), [(tuple(i), got[0][tuple(i)], want[tuple(i)], scores[0][tuple(i)], tol[tuple(i)]) for i in over[:5]]
    assert np.array_equal(got[0][:, kv:], scores[0][:, kv:])


@pytest.mark.parametrize("causal", [True, False])
def test_accumulate_rows_switched_off_in_some_blocks_of_rows(rc, causal):  # noqa: F811
    """3,000 rows are brought in four blocks of 768: rows are off in the second and the fourth of them, or in the first."""
    for where in ((800, 900, 2400, 2500), (10, 11)):
        st = Setup(rc, [(1500, 1600)], 1, 64, 16, seed=len(where))
        q = bf16(st.rng, 1500, 2, 64)
        _, lse = st.attend(q.cuda(), causal)
        off = np.zeros(3000, bool)
        for a, b in zip(where[::2], where[1::2]):
            off[a:b] = True
        off = torch.from_numpy(off.reshape(1500, 2))
        lse[off.cuda()] = -np.inf
        q[off] = float("nan")
        sc = torch.zeros((1, 1, 1600), device="cuda")
        st.cache.accumulate(st.batch, q.cuda(), lse, sc, causal=causal)
        st.cache.sync()
        qn = np.where(off.numpy()[..., None], 0.0, q.float().numpy())
        want = pu.accumulate(st.pool, st.meta, qn, lse.cpu().numpy(), np.zeros((1, 1, 1600), np.float32), causal)
        big = max(pu.reach(st.pool, st.meta, qn, 0, 0, head) for head in range(2))
        tol = 2.0 ** -16 * (1 + big) * want + 2.0 ** -24 * 3008 * want + 1e-30
        assert (np.abs(sc.cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("seqs", [[(3000, 3000)], [(2500, 3001), (40, 40)]])
def test_accumulate_row_blocks_that_see_nothing_of_a_range(rc, seqs):  # noqa: F811
    """A long prompt's last cached tokens, which the first blocks of 768 query rows do not see."""
    st = Setup(rc, seqs, 1, 64, 16, seed=11)
    check_scores(st, bf16(st.rng, st.tokens, 2, 64), True)


# ------------------------------------------------------------------ accumulate: scores that no cached token has
@pytest.mark.parametrize("new", [1, 4, 12, 24, 200])
def test_accumulate_copies_what_is_behind_the_end_unchanged(rc, new):  # noqa: F811
    """Entries kv_len .. max_kv - 1 are copied bit for bit, -0 and NaNs among them."""
    st = Setup(rc, [(new, new + 70), (new, new + 300), (0, 33)], 2, 64, 16, seed=new, max_kv=560)
    st.meta["table"] = np.concatenate([st.meta["table"], np.full((3, 35), -1, np.int32)], 1)
    st.upload(rc)
    q = bf16(st.rng, st.tokens, 4, 64).cuda()
    _, lse = st.attend(q, True)
    bits = st.rng.integers(0, 2 ** 32, (3, 2, 560), dtype=np.uint32)  # any bits: NaNs with payloads, subnormals
    bits[st.rng.random(bits.shape) < 0.5] = 0x80000000
    scores = bits.view(np.int32)
    for in_place in (False, True):
        sd = dev(scores).view(torch.float32)
        out = sd if in_place else torch.zeros_like(sd)
        st.cache.accumulate(st.batch, q, lse, sd, out=None if in_place else out)
        st.cache.sync()
        got = out.view(torch.int32).cpu().numpy()
        for s, kv in enumerate((new + 70, new + 300, 33)):
            assert np.array_equal(got[s, :, kv:], scores[s, :, kv:]), s
        assert np.array_equal(got[2], scores[2])  # (no new tokens: nothing is added)


# ------------------------------------------------------------------ write: the row scale next to its border
# (position, 256 a, 256 b) of the pair with frequency 1: the larger of the turned pair lies within 2.5e-7 of 1.75 * 2^k,
# the border of a scale, but more than 2^-25 (a + b) from it, and its fp32 sum falls on the other side of it
BORDER = [(322, 296, 900), (1956, 316, 360), (3677, 872, 206), (3688, 872, 206), (5606, 406, 980), (5976, 274, 936),
          (6133, 344, 306), (7257, 430, 245), (7844, 916, 224), (11456, 147, 884), (13237, 432, 181), (14577, 450, 196),
          (15429, 280, 908), (16507, 932, 162), (18909, 378, 334), (19036, 151, 584), (19620, 376, 876), (20062, 416, 197),
          (20389, 154, 888), (22540, 272, 356), (23047, 288, 384)]


@pytest.mark.parametrize("dim", [64, 128])
def test_write_scales_are_those_of_the_exact_turn(rc, dim):  # noqa: F811
    """Rows whose largest magnitude is next to the border between two scales have the exact turn's scale and codes."""
    n = len(BORDER)
    st = Setup(rc, [(n, n)], 3, dim, 16, seed=dim)
    k = torch.zeros((n, 3, dim), dtype=torch.float64)
    for t, (_, a, b) in enumerate(BORDER):
        for h, f in enumerate((1 / 256, -(2.0 ** 9), 2.0 ** -40)):
            k[t, h, 0], k[t, h, 1] = a * f, b * f
    k[:, :, 2:] = 2.0 ** -6 * bf16(st.rng, n, 3, dim - 2).double() * k[:, :, :1].abs()
    k = k.to(torch.bfloat16)
    pos = np.array([[p for p, _, _ in BORDER]], np.int32)
    st.cache.write(st.batch, k.cuda(), k.cuda(), dev(pos), rc.RopeAxes((dim // 2,)))
    st.cache.sync()
    y = pu.turn(k.double().numpy(), pos, (dim // 2,))
    x = np.abs(k.double().numpy())
    top = np.abs(y).max(-1)
    border = 1.75 * 2.0 ** np.round(np.log2(top / 1.75))
    assert (np.abs(top - border) > 2.0 ** -25 * (x[..., 0] + x[..., 1])).all() and (np.abs(top / border - 1) < 2.5e-7).all()
    codes, scale = pu.quantise(y)
    table, at = st.meta["table"][0], np.arange(n)
    assert np.array_equal(st.cache.kscale.cpu().numpy()[table[at // 16], :, at % 16], scale)
    assert np.array_equal(st.cache.kcodes.cpu().numpy()[table[at // 16], :, at % 16], codes)


# ------------------------------------------------------------------ rotary positions: the gradient
def rope_case(rc, dtype=torch.float32, n=19, heads=3):  # noqa: F811
    rng = np.random.default_rng(9)
    rope = rc.RopeAxes((12, 10, 10))
    x = torch.from_numpy(rng.standard_normal((n, heads, 64)).astype(np.float32)).to(dtype).cuda().requires_grad_()
    pos = rng.integers(0, 5000, (3, n)).astype(np.int32)
    return rng, rope, x, pos, dev(pos)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_axes_gradient_by_autograd(rc, dtype, inverse):  # noqa: F811
    """The gradient that autograd finds is the definition's adjoint (2^-20 of a pair's size, and bf16's half step), and
    the hand call's bit for bit."""
    rng, rope, x, pos, pd = rope_case(rc, dtype)
    dy = torch.from_numpy(rng.standard_normal(x.shape).astype(np.float32)).to(dtype).cuda()
    y = rc.rc_rope_axes(x, pd, rope, inverse=inverse)
    assert y.requires_grad and torch.equal(y.detach(), rc.rc_rope_axes(x.detach(), pd, rope, inverse=inverse))
    (dx,) = torch.autograd.grad(y, x, dy)
    assert torch.equal(dx, rc.rc_rope_axes(dy, pd, rope, inverse=not inverse))
    g = dy.double().cpu().numpy()
    want = pu.turn(g, pos, rope.sections, sign=1.0 if inverse else -1.0)
    r = np.repeat(np.abs(g)[..., 0::2] + np.abs(g)[..., 1::2], 2, -1)
    tol = 2.0 ** -20 * r + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0)
    assert (np.abs(dx.double().cpu().numpy() - want) <= tol).all()


def test_rope_axes_gradient_against_differences_of_a_loss(rc):  # noqa: F811
    """sum((R x)^3) along a direction: the central difference with step e is the gradient's product with the direction
    but for e^2 sum (R v)^3 exactly (the loss is a cubic), and the roundings of the values, 2^-20 of their sizes."""
    rng, rope, x, _, pd = rope_case(rc)
    y = rc.rc_rope_axes(x, pd, rope)
    (dx,) = torch.autograd.grad((y.double() ** 3).sum(), x)
    v = dev(rng.standard_normal(x.shape).astype(np.float32))
    with torch.no_grad():
        e = 0.5
        f = [(rc.rc_rope_axes(x + s * e * v, pd, rope).double() ** 3).sum() for s in (1, -1)]
        rv = rc.rc_rope_axes(v, pd, rope).double()
        size = ((x.abs() + v.abs()).double().sum(-1, keepdim=True) ** 3).sum() * 3
    assert abs((f[0] - f[1]) / (2 * e) - e * e * (rv ** 3).sum() - (dx.double() * v.double()).sum()) <= 2.0 ** -20 * 4 * size


def test_rope_axes_gradients_of_every_kind(rc):  # noqa: F811
    """A broadcast gradient, one that is not aligned, strided x, x used twice, the gradient of a gradient, none at all."""
    rng, rope, x, _, pd = rope_case(rc)
    ones = torch.ones_like(x)
    back = rc.rc_rope_axes(ones, pd, rope, inverse=True)
    (dx,) = torch.autograd.grad(rc.rc_rope_axes(x, pd, rope).sum(), x)
    assert torch.equal(dx, back)
    flat = torch.ones(x.numel() + 1, device="cuda")[1:].view(x.shape)
    assert flat.data_ptr() % 16
    (dx,) = torch.autograd.grad(rc.rc_rope_axes(x, pd, rope), x, flat)
    assert torch.equal(dx, back)
    fused = torch.zeros((x.shape[0], 8, 64), device="cuda", requires_grad=True)
    rc.rc_rope_axes(fused[:, 2:5], pd, rope).sum().backward()
    assert torch.equal(fused.grad[:, 2:5], back) and not fused.grad[:, :2].any() and not fused.grad[:, 5:].any()
    (dx,) = torch.autograd.grad(rc.rc_rope_axes(x, pd, rope).sum() + rc.rc_rope_axes(x, pd, rope).sum(), x)
    assert torch.equal(dx, 2 * back)
    y = rc.rc_rope_axes(x, pd, rope)
    (dx,) = torch.autograd.grad((y * y).sum() / 2, x, create_graph=True)   # x itself, but for roundings
    (ddx,) = torch.autograd.grad(dx.sum(), x)
    assert (ddx - 1).abs().max() <= 2.0 ** -18
    with torch.no_grad():
        assert not rc.rc_rope_axes(x, pd, rope).requires_grad
    assert not rc.rc_rope_axes(x.detach(), pd, rope).requires_grad


def test_rope_axes_gradient_on_another_stream_and_in_a_graph(rc):  # noqa: F811
    rng, rope, x, _, pd = rope_case(rc, n=4000, heads=8)
    dy = dev(rng.standard_normal(x.shape).astype(np.float32))
    back = rc.rc_rope_axes(dy, pd, rope, inverse=True)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    y = rc.rc_rope_axes(x, pd, rope, stream=stream)
    torch.cuda.current_stream().wait_stream(stream)
    (dx,) = torch.autograd.grad(y, x, dy)
    torch.cuda.synchronize()
    assert torch.equal(dx, back)
    del y, dx
    leaf = x.detach().clone().requires_grad_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (dx,) = torch.autograd.grad(rc.rc_rope_axes(leaf, pd, rope), leaf, dy)
    dy.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dx, 2 * back)


def test_rope_axes_refuses_to_lose_a_gradient(rc):  # noqa: F811
    _, rope, x, _, pd = rope_case(rc)
    out = torch.zeros_like(x)
    for a, b in ((x, out.detach()), (x.detach(), out.detach().requires_grad_()), (x * 1, None)):
        with pytest.raises(RuntimeError):
            y = a if b is None else b
            rc.rc_rope_axes(a, pd, rope, out=y)
    with torch.no_grad():
        rc.rc_rope_axes(x, pd, rope, out=out)
    pos = pd.clone()
    y = rc.rc_rope_axes(x, pos, rope)
    pos += 1  # the positions of the turn back: autograd notices
    with pytest.raises(RuntimeError):
        y.sum().backward()

"""Edges of the paged-cache calls on the GPU: streams other than the current one, tensors that share memory, rows that are
switched off, borders of a row's scale.  Tolerances and definitions are those of tests/test_gpu_paged.py and
tests/paged_util.py."""
import gc

import pytest
import torch

from test_gpu_paged import Setup, bf16, rc  # noqa: F401 (rc: the fixture)

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

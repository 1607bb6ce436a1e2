"""Edges of the paged-cache calls on the GPU: streams other than the current one, tensors that share memory, rows that are
switched off, borders of a row's scale.  Tolerances and definitions are those of tests/test_gpu_paged.py and
tests/paged_util.py."""
import gc

import numpy as np
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

"""Which tensors of a paged call may share memory: the host's checks, without a GPU (the addresses are never read)."""
import ctypes
import itertools
import pathlib
import subprocess

import pytest

from test_paged_cpu import A, calls, good_plan, rc, structs  # noqa: F401 (rc: the fixture)

MEET = """
#include "rc_paged_bounds.h"
extern "C" int meet(uint64_t a, int64_t sa, int64_t na, int64_t wa, uint64_t b, int64_t sb, int64_t nb, int64_t wb) {
    return paged_rows_meet(a, sa, na, wa, b, sb, nb, wb);
}
"""


@pytest.fixture(scope="module")
def meet(tmp_path_factory):
    d = tmp_path_factory.mktemp("meet")
    (d / "m.cpp").write_text(MEET)
    csrc = pathlib.Path(__file__).parents[1] / "fp8_ring_kv_cache_gb300" / "csrc"
    subprocess.run(["g++", "-O1", "-shared", "-fPIC", "-fsanitize=undefined", "-fsanitize-undefined-trap-on-error", f"-I{csrc}",
                    str(d / "m.cpp"), "-o", str(d / "m.so")], check=True)
    f = ctypes.CDLL(str(d / "m.so")).meet
    f.argtypes = [ctypes.c_uint64, *[ctypes.c_int64] * 3] * 2
    return f


def brute(a, sa, na, wa, b, sb, nb, wb):
    mine = {a + i * sa + k for i in range(na) for k in range(wa)}
    return any(b + j * sb + k in mine for j in range(nb) for k in range(wb))


def test_rows_that_meet(rc, meet):  # noqa: F811
    """Every small arrangement of two sets of rows against the sets of their bytes, and the Python form of the same."""
    from fp8_ring_kv_cache_gb300._paged import _rows_meet
    at = 1000
    for (wa, ga), (wb, gb), na, nb in itertools.product(((1, 0), (2, 0), (2, 1), (3, 4), (4, 7)), ((1, 0), (2, 1), (3, 4), (5, 2)),
                                                        (1, 2, 4), (1, 3, 5)):
        sa, sb = wa + ga, wb + gb
        for b in range(at - nb * sb - 2, at + na * sa + 3):
            want = brute(at, sa, na, wa, b, sb, nb, wb)
            assert bool(meet(at, sa, na, wa, b, sb, nb, wb)) == want, (sa, na, wa, b - at, sb, nb, wb)
            assert bool(meet(b, sb, nb, wb, at, sa, na, wa)) == want
    for w, n, sa, sb in itertools.product((1, 2, 3), (1, 2, 5), (3, 4, 7), (3, 5, 9)):
        for b in range(at - n * sb - 2, at + n * sa + 3):
            assert _rows_meet(at, sa, b, sb, n, w) == brute(at, sa, n, w, b, sb, n, w), (sa, b - at, sb, n, w)


def test_rows_that_meet_far_apart(meet):
    """Spans past 64 bits do not wrap."""
    top = 2 ** 63 - 1
    assert not meet(2 ** 20, 2 ** 57, 2 ** 31, 64, 2 ** 20 + 64, 2 ** 57, 2 ** 31, 64)
    assert meet(2 ** 20, 2 ** 57, 2 ** 31, 64, 2 ** 20 + 63, 2 ** 57, 2 ** 31, 64)
    assert not meet(2 ** 20, top, 2 ** 40, 16, 2 ** 20 + 16, top, 2 ** 40, 16)
    assert meet(2 ** 56, 16, 1, 16, 2 ** 56 - 2 ** 40 + 8, 2 ** 40, 2, 16)


def test_rope_axes_refuses_what_overlaps(rc):  # noqa: F811
    p = good_plan(rc)._ptr
    # 5 tokens of 4 heads x 64, bf16: rows of 512 bytes
    for x, xs, out, os in ((A, 256, A + 512, 256), (A, 512, A + 256, 512), (A, 512, A + 496, 512), (A + 2048, 256, A, 264), (A, 512, A, 256)):
        assert rc.lib.rc_rope_axes(p, x, xs, out, os, 0, 5, 4, A, 5, 0, None) == rc.RC_ERR_ARG, (x - A, xs, out - A, os)


def test_attend_refuses_results_over_its_queries(rc):  # noqa: F811
    v, b = structs(rc)  # 5 tokens of 4 heads x 64: rows of 512 bytes
    for q, qs, out, os in ((A, 256, A, 256), (A, 256, A + 16, 256), (A, 512, A + 496, 512), (A, 512, A, 256), (A + 2048, 256, A, 264)):
        assert calls(rc, v, b, q=q, qs=qs, out=out, os=os)["attend"]() == rc.RC_ERR_ARG, (q - A, qs, out - A, os)


def test_accumulate_refuses_scores_over_each_other(rc):  # noqa: F811
    v, b = structs(rc)  # 3 sequences x 2 heads, rows of 60 scores
    for out, stride in ((A + 4, 60), (A + 236, 119), (A - 4, 60), (A + 4 * 60, 60), (A - 4 * 299, 60)):
        assert calls(rc, v, b, scores=A, out=out, stride=stride)["accumulate"]() == rc.RC_ERR_ARG, (out - A, stride)


def test_evict_refuses_scores_over_each_other(rc):  # noqa: F811
    v, b = structs(rc)  # 3 sequences x 2 heads: rows of 60 scores, 48 of the kept ones in all
    vp, bp = ctypes.addressof(v), ctypes.addressof(b)
    for out, stride in ((A, 60), (A + 4 * 359, 60), (A - 4 * 47, 60), (A + 4 * 60, 100)):
        assert rc.lib.rc_paged_evict(vp, bp, A, stride, 8, 2, A, 1, A, A, out, None) == rc.RC_ERR_ARG, (out - A, stride)


def test_calls_that_take_more_blocks_than_a_grid_has(rc):  # noqa: F811
    """65,535 sequences of which one may have all the rows."""
    most = 2 ** 31 - 1
    v, b = structs(rc, None, dict(seqs=65535, tokens=most, max_new=most))
    assert calls(rc, v, b, ps=most)["write"]() == rc.RC_ERR_UNSUPPORTED
    assert calls(rc, v, b, out=A + (1 << 45), heads=2, qs=128, os=128)["attend"]() == rc.RC_ERR_UNSUPPORTED   # rows of a head
    v, b = structs(rc, dict(kv_heads=1024), dict(seqs=65535, tokens=1 << 20, max_new=1 << 14))
    assert calls(rc, v, b, out=A + (1 << 45), heads=1024, qs=65536, os=65536)["attend"]() == rc.RC_ERR_UNSUPPORTED

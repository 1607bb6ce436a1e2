"""The paged-cache entry points without a GPU: the rotary plan's numbers, and every refusal of the C ABI's argument
checks, which come before any device work (the addresses here are never read)."""
import ctypes
import functools
import math
from fractions import Fraction

import numpy as np
import pytest

import paged_util as pu


@pytest.fixture(scope="module")
def rc():
    import __graft_entry__
    __graft_entry__.build()
    import fp8_ring_kv_cache_gb300 as rc
    return rc


def test_plan_frequencies(rc):
    from fractions import Fraction
    for sections, shared in (((64,), False), ((22, 21, 21), False), ((22, 21, 21), True), ((0, 32), False), ((8, 8, 8, 8), True)):
        plan = rc.RopeAxes(sections, base=10000.0, shared_freqs=shared).plan
        i = 0
        for a, w in enumerate(sections):
            for r in range(w):
                theta = 10000.0 ** (-2.0 * i / (2 * sum(sections))) if shared else 10000.0 ** (-r / w)
                assert plan.axis[i] == a
                # 2 pi to 64 bits
                two_pi = Fraction(6283185307179586476925286766559, 10 ** 30)
                want = Fraction(theta) / two_pi * 2 ** 64
                assert abs(plan.turns[i] - want) <= 1 + want * Fraction(1, 2 ** 52)
                i += 1


def test_plan_turns_far_positions_exactly(rc):
    """position * frequency mod 1 turn in 64-bit integers, at the farthest positions, against exact rationals."""
    from fractions import Fraction
    plan = rc.RopeAxes((22, 21, 21)).plan
    two_pi = Fraction(6283185307179586476925286766559, 10 ** 30)
    for i, (a, r, w) in enumerate([(0, r, 22) for r in range(22)]):
        for pos in (1, 757, 200000, 2 ** 31 - 1, -2 ** 31):
            frac = Fraction((pos * plan.turns[i]) % 2 ** 64, 2 ** 64)
            want = Fraction(10000.0 ** (-r / w)) * pos / two_pi % 1
            off = abs(frac - want)
            off = min(off, 1 - off)
            assert off <= Fraction(abs(pos), 2 ** 52)  # pow()'s own rounding, carried by the position


@pytest.mark.parametrize("sections,base,flags", [((33,), 1e4, 0), ((31,), 1e4, 0), ((33, -1), 1e4, 0), ((32,), 1.0, 0),
                                                 ((32,), float("nan"), 0), ((32,), 1e10, 0), ((32,), 1e4, 2),
                                                 ((8, 8, 8, 4, 4), 1e4, 0), ((), 1e4, 0)])
def test_plan_refusals(rc, sections, base, flags):
    from fp8_ring_kv_cache_gb300 import _paged
    plan = _paged.rc_rope_plan()
    arr = (ctypes.c_int * max(1, len(sections)))(*sections)
    st = rc.lib.rc_rope_plan_init(ctypes.addressof(plan), 64, len(sections), arr, base, flags)
    assert st == rc.RC_ERR_ARG


def test_plan_unsupported_head_dim(rc):
    with pytest.raises(rc.RcError) as e:
        rc.RopeAxes((48,))
    assert e.value.status == rc.RC_ERR_UNSUPPORTED
    assert rc.lib.rc_rope_plan_init(None, 64, 1, (ctypes.c_int * 1)(32), 1e4, 0) == rc.RC_ERR_ARG


A = 1 << 20  # an aligned address that nobody reads


def structs(rc, view=None, batch=None):
    from fp8_ring_kv_cache_gb300 import _paged
    v = _paged.rc_paged_view(A, A, A, A, A, 10, 2, 64, 16)
    b = _paged.rc_paged_batch(A, A, A, 3, 4, 5, 2, 60)
    for k, x in (view or {}).items():
        setattr(v, k, x)
    for k, x in (batch or {}).items():
        setattr(b, k, x)
    return v, b


@functools.cache
def good_plan(rc):
    return rc.RopeAxes((32,))


def calls(rc, v, b, q=A, qs=256, heads=4, out=A, os=256, lse=A, scores=A, stride=60, keep=8, recent=2, dst=A, dst_pages=1,
          kept=A, length=A, k=A, ks=128, pos=A, ps=5, plan=None):
    if plan is None:
        plan = good_plan(rc)._ptr
    vp, bp = ctypes.addressof(v) if v is not None else None, ctypes.addressof(b) if b is not None else None
    return {"write": lambda: rc.lib.rc_paged_write(vp, bp, k, ks, k, ks, pos, ps, plan, None),
            "attend": lambda: rc.lib.rc_paged_attend(vp, bp, q, qs, heads, out, os, lse, 1, None),
            "accumulate": lambda: rc.lib.rc_paged_accumulate(vp, bp, q, qs, heads, lse, scores, out, stride, 1, None),
            "evict": lambda: rc.lib.rc_paged_evict(vp, bp, scores, stride, keep, recent, dst, dst_pages, kept, length, None, None)}


ALL = ("write", "attend", "accumulate", "evict")


@pytest.mark.parametrize("view", [dict(kcodes=0), dict(vcodes=0), dict(kscale=0), dict(vscale=0), dict(workspace=0), dict(kcodes=A + 8),
                                  dict(vscale=A + 4), dict(workspace=A + 128), dict(pages=0), dict(kv_heads=0), dict(kv_heads=1025)])
def test_refused_pools(rc, view):
    v, b = structs(rc, view)
    for name, call in calls(rc, v, b).items():
        assert call() == rc.RC_ERR_ARG, name


@pytest.mark.parametrize("view", [dict(head_dim=96), dict(head_dim=0), dict(page_tokens=8), dict(page_tokens=48), dict(page_tokens=256),
                                  dict(page_tokens=0)])
def test_unsupported_pools(rc, view):
    v, b = structs(rc, view)
    for name, call in calls(rc, v, b).items():
        assert call() == rc.RC_ERR_UNSUPPORTED, name


@pytest.mark.parametrize("batch", [dict(page_table=0), dict(kv_len=0), dict(seqs=0), dict(seqs=65536), dict(table_pages=-1), dict(tokens=-1),
                                   dict(max_new=-1), dict(max_kv=-1), dict(max_kv=65), dict(max_kv=(1 << 24) + 1, table_pages=1 << 22)])
def test_refused_batches(rc, batch):
    v, b = structs(rc, None, batch)
    for name, call in calls(rc, v, b, stride=1 << 25, dst_pages=1 << 22).items():
        assert call() == rc.RC_ERR_ARG, name


def test_null_structs_and_q_start(rc):
    v, b = structs(rc)
    for name in ALL:
        assert calls(rc, None, b)[name]() == rc.RC_ERR_ARG
        assert calls(rc, v, None)[name]() == rc.RC_ERR_ARG
    b.q_start = 0
    for name in ("write", "attend", "accumulate"):
        assert calls(rc, v, b)[name]() == rc.RC_ERR_ARG
    assert rc.lib.rc_paged_status(None, None) == rc.RC_ERR_ARG
    assert rc.lib.rc_paged_set_wait_limit(60_000_000_001) == rc.RC_ERR_ARG


@pytest.mark.parametrize("name,args", [
    ("attend", dict(q=0)), ("attend", dict(out=0)), ("attend", dict(q=A + 2)), ("attend", dict(out=A + 8)), ("attend", dict(heads=3)),
    ("attend", dict(heads=0)), ("attend", dict(qs=255)), ("attend", dict(qs=252)), ("attend", dict(qs=260)), ("attend", dict(os=128)),
    ("attend", dict(heads=-2)), ("accumulate", dict(q=0)), ("accumulate", dict(lse=0)), ("accumulate", dict(scores=0)),
    ("accumulate", dict(out=0)), ("accumulate", dict(stride=59)), ("accumulate", dict(heads=5)), ("accumulate", dict(qs=8)),
    ("write", dict(k=0)), ("write", dict(k=A + 4)), ("write", dict(ks=64)), ("write", dict(ks=132)), ("write", dict(pos=0)),
    ("write", dict(ps=4)), ("evict", dict(keep=0)), ("evict", dict(recent=-1)), ("evict", dict(recent=9)), ("evict", dict(dst=0)),
    ("evict", dict(keep=17, dst_pages=1)), ("evict", dict(dst_pages=-1)), ("evict", dict(kept=0)), ("evict", dict(length=0)),
    ("evict", dict(scores=0)), ("evict", dict(stride=59))])
def test_refused_arguments(rc, name, args):
    v, b = structs(rc)
    assert calls(rc, v, b, **args)[name]() == rc.RC_ERR_ARG


def test_refused_plans(rc):
    v, b = structs(rc)
    wide = rc.RopeAxes((64,))
    assert calls(rc, v, b, plan=wide._ptr)["write"]() == rc.RC_ERR_ARG
    from fp8_ring_kv_cache_gb300 import _paged
    blank = _paged.rc_rope_plan()
    assert calls(rc, v, b, plan=ctypes.addressof(blank))["write"]() == rc.RC_ERR_ARG
    turn = rc.lib.rc_rope_axes
    p = good_plan(rc)._ptr
    good = [p, A, 256, A, 256, 0, 5, 4, A, 5, 0, None]
    for at, value in ((0, None), (0, ctypes.addressof(blank)), (1, None), (1, A + 8), (2, 128), (2, 260), (3, None), (4, 255), (5, 2),
                      (6, -1), (7, 0), (8, None), (9, 4)):
        args = list(good)
        args[at] = value
        assert turn(*args) == rc.RC_ERR_ARG, (at, value)


def test_empty_calls_do_nothing(rc):
    v, b = structs(rc, None, dict(tokens=0, max_new=0))
    c = calls(rc, v, b, q=0, out=0, k=0)
    assert c["write"]() == rc.RC_OK and c["attend"]() == rc.RC_OK
    assert rc.lib.rc_rope_axes(good_plan(rc)._ptr, None, 0, None, 0, 0, 0, 4, None, 0, 0, None) == rc.RC_OK


def test_the_tests_own_definitions():
    """E4M3 rounding and the row scale of tests/paged_util.py against torch's cast and by the definition."""
    import torch
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(20000) * 2.0 ** rng.integers(-12, 9, 20000), pu.E4M3[np.r_[0:127, 128:255]],
                        (pu.MAGS[1:] + pu.MAGS[:-1]) / 2]).clip(-448, 448)
    want = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(pu.nearest_code(x.astype(np.float32)), want)
    rows = rng.standard_normal((500, 8)) * 2.0 ** rng.integers(-130, 20, (500, 1))
    rows[3] = 0
    rows[4] = 448 * 2.0 ** -5
    codes, scale = pu.quantise(rows)
    s = pu.scale_value(scale)
    amax = np.abs(rows).max(-1)
    inside = (scale > 3) & (scale < 134)
    assert (amax[inside] <= 448 * s[inside]).all() and (amax[inside & (amax > 0)] > 224 * s[inside & (amax > 0)]).all()
    assert scale[3] == 127 and scale[4] == 127 - 5 and scale.min() >= 3 and scale.max() <= 134
    assert pu.quantise(np.array([[1.0, np.inf]]))[1][0] == 255


@pytest.mark.parametrize("base,sections,shared", [(10000.0, (64,), False), (10000.0, (24, 20, 20), False),
                                                  (500000.0, (32,), False), (1e9, (64,), False), (10000.0, (12, 10, 10), True)])
def test_plan_turns_are_the_rounded_frequencies(rc, base, sections, shared):
    """turns = frequency / 2 pi * 2^64: within half a unit of the last place (and the constant's own 2^-12) of the double."""
    plan = rc.RopeAxes(sections, base=base, shared_freqs=shared).plan
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582")
    i = 0
    for axis, w in enumerate(sections):
        for r in range(w):
            theta = math.pow(base, -2.0 * i / (2 * sum(sections))) if shared else math.pow(base, -r / w)
            assert abs(plan.turns[i] - Fraction(theta) * 2 ** 64 / two_pi) <= Fraction(1, 2) + Fraction(1, 2 ** 12)
            assert plan.axis[i] == axis
            i += 1


BOUNDS = """
#include "rc_paged_bounds.h"
extern "C" int seq_ok(int kv, int q0, int end, int tokens, int max_new, int max_kv) {
    return paged_seq_ok(kv, q0, end, tokens, max_new, max_kv);
}
extern "C" int len_ok(int kv, int max_kv) { return paged_len_ok(kv, max_kv); }
extern "C" int page_ok(int page, int pages) { return paged_page_ok(page, pages); }
"""


def test_device_side_bounds(tmp_path):
    """The checks that the kernels make of lengths, rows and pages: every mix of ordinary and extreme values against the
    same conditions on Python's integers; signed overflow would trap."""
    import itertools
    import pathlib
    import subprocess
    src, so = tmp_path / "b.cpp", tmp_path / "b.so"
    src.write_text(BOUNDS)
    csrc = pathlib.Path(__file__).parents[1] / "fp8_ring_kv_cache_gb300" / "csrc"
    subprocess.run(["g++", "-O1", "-shared", "-fPIC", "-fsanitize=undefined", "-fsanitize-undefined-trap-on-error", f"-I{csrc}",
                    str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    values = (-2 ** 31, -1, 0, 1, 5, 6, 100, 101, 2 ** 31 - 1)
    for kv, q0, end in itertools.product(values, repeat=3):
        for tokens, max_new, max_kv in ((0, 0, 0), (5, 5, 100), (100, 6, 5), (2 ** 31 - 1, 2 ** 31 - 1, 1 << 24)):
            want = 0 <= kv <= max_kv and 0 <= q0 <= end <= tokens and end - q0 <= max_new
            assert bool(lib.seq_ok(kv, q0, end, tokens, max_new, max_kv)) == want, (kv, q0, end, tokens, max_new, max_kv)
    for a in values:
        for b in (0, 1, 6, 2 ** 31 - 1):
            assert bool(lib.len_ok(a, b)) == (0 <= a <= b) and bool(lib.page_ok(a, b)) == (0 <= a < b)

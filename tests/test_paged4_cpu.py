"""The rotary forms and the 4-bit paged cache without a GPU: the forms' numbers, and every refusal of the C ABI's argument
checks, which come before any device work (the addresses here are never read)."""
import copy
import ctypes
import functools
import os
import pickle
import re
from fractions import Fraction

import numpy as np
import pytest

import paged4_util as pu


@pytest.fixture(scope="module")
def rc():
    import __graft_entry__
    __graft_entry__.build()
    import fp8_ring_kv_cache_gb300 as rc
    return rc


TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582")


@pytest.mark.parametrize("dim,sections,kw", [
    (128, (64,), {}), (128, (22, 21, 21), {"scaling": "linear", "factor": 3.7}), (64, (1, 31), {"scaling": "base", "factor": 8.0}),
    (256, (128,), {"scaling": "parts", "factor": 40.0, "context": 4096.0}), (96, (10, 0, 3), {"shared_freqs": True, "scaling": "base", "factor": 2.0}),
    (80, (10,), {"scaling": "parts", "factor": 8.0, "context": 8192.0, "low": 1.0, "high": 4.0, "base": 500000.0}),
    (128, (64,), {"scaling": "linear", "factor": 1e6, "base": 1e9}), (8, (1,), {"scaling": "base", "factor": 1e6})])
def test_form_frequencies(rc, dim, sections, kw):
    form = rc.RopeForm(dim, sections=sections, **kw).form
    kw = dict(kw)
    shared = kw.pop("shared_freqs", False)
    want = pu.frequencies(sections, shared=shared, **kw)
    for i, (axis, theta) in enumerate(want):
        exact = Fraction(theta) / TWO_PI * 2 ** 64
        # (some roundings of 2^-53 on the way to the frequency, the power's among them, here and there)
        assert abs(form.turns[i] - exact) <= 1 + exact * Fraction(1, 2 ** 48), (i, theta)
        assert form.axis[i] == axis


def test_form_scalings_at_their_ends(rc):
    """By parts: fast pairs are kept, slow ones divided by the factor; by base: the fastest kept, the slowest divided."""
    plain = rc.RopeForm(128, sections=(64,)).form.turns
    parts = rc.RopeForm(128, sections=(64,), scaling="parts", factor=16.0, context=4096.0).form.turns
    assert parts[0] == plain[0] and abs(parts[63] * 16 - plain[63]) <= 16 + plain[63] * 2 ** -48
    base = rc.RopeForm(128, sections=(64,), scaling="base", factor=16.0).form.turns
    assert base[0] == plain[0] and abs(base[63] * 16 - plain[63]) <= 16 + plain[63] * 2 ** -45
    assert all(plain[i] >= parts[i] >= plain[i] // 16 for i in range(64))


def test_form_defaults(rc):
    f = rc.RopeForm(96)
    assert (f.dims, f.sections, f.axes, f.gain) == (96, (48,), 1, 1.0)
    f = rc.RopeForm(96, first=32)
    assert (f.dims, f.sections) == (64, (32,))
    f = rc.RopeForm(96, dims=40, layout="halves", gain=0.5)
    assert (f.dims, f.sections, f.form.layout, f.form.gain) == (40, (20,), 1, 0.5)


@pytest.mark.parametrize("kw", [
    dict(first=-2), dict(first=1), dict(first=66), dict(dims=0), dict(dims=66), dict(dims=7), dict(first=32, dims=34), dict(sections=(31,), dims=64),
    dict(sections=(33, -1)), dict(base=1.0), dict(base=float("nan")), dict(base=2e9), dict(scaling="linear", factor=0.5),
    dict(scaling="base", factor=float("inf")), dict(scaling="parts", factor=2.0), dict(scaling="parts", factor=2.0, context=100.0, low=5.0, high=5.0),
    dict(scaling="parts", factor=2.0, context=100.0, low=-1.0), dict(scaling="parts", factor=2.0, context=float("nan")),
    dict(gain=0.0), dict(gain=-1.0), dict(gain=17.0), dict(gain=float("nan")), dict(first=2 ** 31 - 2, dims=64)])
def test_refused_forms(rc, kw):
    with pytest.raises(rc.RcError) as e:
        rc.RopeForm(64, **kw)
    assert e.value.status == rc.RC_ERR_ARG


@pytest.mark.parametrize("dim", [0, 4, 12, 100, 264, -8])
def test_unsupported_heads(rc, dim):
    with pytest.raises(rc.RcError) as e:
        rc.RopeForm(dim, dims=2)
    assert e.value.status == rc.RC_ERR_UNSUPPORTED


def test_refused_forms_in_python(rc):
    for kw in (dict(layout="thirds"), dict(scaling="more"), dict(sections=()), dict(sections=(8, 8, 8, 4, 4))):
        with pytest.raises(ValueError):
            rc.RopeForm(64, **kw)
    from fp8_ring_kv_cache_gb300 import _paged4
    form, spec = _paged4.rc_rope_form(), _paged4.rc_rope_spec()
    init = rc.lib.rc_rope_form_init
    assert init(None, ctypes.addressof(spec)) == rc.RC_ERR_ARG and init(ctypes.addressof(form), None) == rc.RC_ERR_ARG
    for field, value in (("layout", 2), ("layout", -1), ("axes", 0), ("axes", 5), ("flags", 2), ("scaling", 4), ("scaling", -1)):
        spec = _paged4.rc_rope_spec(head_dim=64, dims=64, axes=1, base=1e4, gain=1.0)
        spec.sections[0] = 32
        assert init(ctypes.addressof(form), ctypes.addressof(spec)) == rc.RC_OK
        setattr(spec, field, value)
        assert init(ctypes.addressof(form), ctypes.addressof(spec)) == rc.RC_ERR_ARG, (field, value)


A = 1 << 20  # an aligned address that nobody reads


def structs(rc, view=None, batch=None):
    from fp8_ring_kv_cache_gb300 import _paged, _paged4
    v = _paged4.rc_paged4_view(A, A, A, A, A, 10, 2, 64, 16)
    b = _paged.rc_paged_batch(A, A, A, 3, 4, 5, 2, 60)
    for k, x in (view or {}).items():
        setattr(v, k, x)
    for k, x in (batch or {}).items():
        setattr(b, k, x)
    return v, b


@functools.cache
def good_form(rc):
    return rc.RopeForm(64, layout="halves")


def calls(rc, v, b, q=A, qs=256, heads=4, out=A + (1 << 30), os=256, lse=A, k=A, ks=128, v2=A, vs=128, pos=A, ps=5, form=-1):
    form = good_form(rc)._ptr if form == -1 else form
    vp, bp = ctypes.addressof(v) if v is not None else None, ctypes.addressof(b) if b is not None else None
    return {"write": lambda: rc.lib.rc_paged4_write(vp, bp, k, ks, v2, vs, pos, ps, form, None),
            "attend": lambda: rc.lib.rc_paged4_attend(vp, bp, q, qs, heads, out, os, lse, 1, None)}


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


@pytest.mark.parametrize("batch", [dict(page_table=0), dict(kv_len=0), dict(q_start=0), dict(seqs=0), dict(seqs=65536), dict(table_pages=-1),
                                   dict(tokens=-1), dict(max_new=-1), dict(max_kv=-1), dict(max_kv=65), dict(max_kv=(1 << 24) + 1, table_pages=1 << 22)])
def test_refused_batches(rc, batch):
    v, b = structs(rc, None, batch)
    for name, call in calls(rc, v, b).items():
        assert call() == rc.RC_ERR_ARG, name


def test_null_structs(rc):
    v, b = structs(rc)
    for name in ("write", "attend"):
        assert calls(rc, None, b)[name]() == rc.RC_ERR_ARG
        assert calls(rc, v, None)[name]() == rc.RC_ERR_ARG
    assert rc.lib.rc_paged4_status(None, None) == rc.RC_ERR_ARG
    v.workspace = 0
    assert rc.lib.rc_paged4_status(ctypes.addressof(v), None) == rc.RC_ERR_ARG


@pytest.mark.parametrize("name,args", [
    ("attend", dict(q=0)), ("attend", dict(out=0)), ("attend", dict(q=A + 2)), ("attend", dict(out=A + 8)), ("attend", dict(heads=3)),
    ("attend", dict(heads=0)), ("attend", dict(heads=-2)), ("attend", dict(qs=255)), ("attend", dict(qs=252)), ("attend", dict(qs=260)),
    ("attend", dict(os=128)), ("attend", dict(out=A)), ("attend", dict(out=A + 16)), ("attend", dict(out=A + 2032)),
    ("write", dict(k=0)), ("write", dict(v2=0)), ("write", dict(k=A + 4)), ("write", dict(v2=A + 8)), ("write", dict(ks=64)), ("write", dict(vs=132)),
    ("write", dict(pos=0)), ("write", dict(ps=4))])
def test_refused_arguments(rc, name, args):
    v, b = structs(rc)
    assert calls(rc, v, b, **args)[name]() == rc.RC_ERR_ARG


def test_refused_form_of_a_call(rc):
    from fp8_ring_kv_cache_gb300 import _paged4
    v, b = structs(rc)
    wide = rc.RopeForm(128)
    blank = _paged4.rc_rope_form()
    bad = rc.RopeForm(64, sections=(20, 12))
    bad.form.axis[31] = 2  # an axis that the form does not have
    for form in (wide._ptr, ctypes.addressof(blank), bad._ptr):
        assert calls(rc, v, b, form=form)["write"]() == rc.RC_ERR_ARG
    turn, p = rc.lib.rc_rope_turn, good_form(rc)._ptr
    good = [p, A, 256, A, 256, 0, 5, 4, A, 5, 0, None]
    for at, value in ((0, None), (0, ctypes.addressof(blank)), (0, bad._ptr), (1, None), (1, A + 8), (2, 128), (2, 260), (3, None), (3, A + 512),
                      (4, 255), (4, 264), (5, 2), (6, -1), (7, 0), (8, None), (9, 4)):
        args = list(good)
        args[at] = value
        assert turn(*args) == rc.RC_ERR_ARG, (at, value)
    args = list(good)
    args[6], args[9] = 1 << 31, 1 << 31
    assert turn(*args) == rc.RC_ERR_UNSUPPORTED


def test_empty_calls_do_nothing(rc):
    v, b = structs(rc, None, dict(tokens=0, max_new=0))
    c = calls(rc, v, b, q=0, out=0, k=0, v2=0, pos=0)
    assert c["write"]() == rc.RC_OK and c["attend"]() == rc.RC_OK
    assert rc.lib.rc_rope_turn(good_form(rc)._ptr, None, 0, None, 0, 0, 0, 4, None, 0, 0, None) == rc.RC_OK


def test_calls_that_take_more_blocks_than_a_grid_has(rc):
    most = 2 ** 31 - 1
    v, b = structs(rc, None, dict(seqs=65535, tokens=most, max_new=most))
    assert calls(rc, v, b, ps=most)["write"]() == rc.RC_ERR_UNSUPPORTED
    assert calls(rc, v, b, out=A + (1 << 45), heads=2, qs=128, os=128)["attend"]() == rc.RC_ERR_UNSUPPORTED


def test_the_tests_own_definitions():
    """Codes and scales of tests/paged4_util.py against a search of all codes and all scales."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((300, 16)) * 2.0 ** rng.integers(-20, 16, (300, 1))
    x[0] = 0
    x[1] = 6 * pu.SCALES[100] * np.array([1, 0.25, 0.5, 0.125, 1 / 24, 1 / 8, 5 / 24, 7 / 24, 5 / 12, 7 / 12, 5 / 6, -1 / 24, -1 / 8, 0, 1, 1])
    x[2] = 1e9
    codes, scale = pu.quantise(x)
    for row, c, (b,) in zip(x, codes, scale):
        top = np.abs(row).max()
        fits = [i for i in range(pu.TOP + 1) if top <= 6 * pu.SCALES[i]]
        assert b == (fits[0] if fits else pu.TOP)
        s = pu.SCALES[b]
        for value, code in zip(row, c):
            d = np.abs(np.abs(value) - pu.E2M1 * s)
            best = [i for i in range(8) if d[i] == d.min()]
            if s > 0:
                assert (code & 7) in best and ((code & 7) % 2 == 0 or len(best) == 1)
            assert (code >> 3) == np.signbit(value)
    assert scale[0, 0] == 0 and scale[2, 0] == pu.TOP and scale[1, 0] == 100
    bad = np.ones((1, 32))
    bad[0, 20] = np.nan
    c, b = pu.quantise(bad)
    assert (c == 0).all() and (b == 255).all()
    assert np.array_equal(pu.unpack(pu.pack(codes)), codes)
    # every code times every scale is an exact bf16 and fp16 number
    import torch
    every = torch.from_numpy(pu.E2M1[:, None] * pu.SCALES[None, :pu.TOP + 1])
    assert torch.equal(every.to(torch.bfloat16).double(), every) and torch.equal(every.half().double(), every)


@pytest.mark.parametrize("make", [lambda rc: rc.RopeForm(128, layout="halves", gain=1.25), lambda rc: rc.RopeAxes((22, 21, 21))])
@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, lambda f: pickle.loads(pickle.dumps(f))])
def test_a_copy_of_a_form_has_numbers_of_its_own(rc, make, how):
    """What a call is given is the address of numbers that live as long as the copy, whatever happens to the original."""
    form = make(rc)
    numbers = lambda f: f.form if hasattr(f, "form") else f.plan
    want = bytes(numbers(form))
    other = how(form)
    assert other._ptr == ctypes.addressof(numbers(other))
    assert bytes(numbers(other)) == want


def test_shared_arrays_lie_on_the_boundaries_of_their_accesses():
    """Shared arrays that the kernels' sources read or write as vectors are declared with the vectors' alignment."""
    here = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_ring_kv_cache_gb300", "csrc")
    size = {"uint2": 8, "float2": 8, "uint4": 16, "float4": 16, "int4": 16}
    checked = 0
    for name in sorted(os.listdir(here)):
        with open(os.path.join(here, name)) as f:
            text = f.read()
        for align, kind, array in re.findall(r"__shared__\s+(?:__align__\((\d+)\)\s+)?(\w+)\s+(\w+)\s*\[", text):
            for access in re.findall(r"reinterpret_cast<(?:const )?(\w+)\s*\*>\(\s*&?" + array + r"\b", text):
                if access in size:
                    checked += 1
                    assert max(int(align or 1), size.get(kind, 1)) >= size[access], (name, array, access)
    assert checked >= 2

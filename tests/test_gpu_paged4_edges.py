"""Edges of the rotary forms and of the 4-bit paged cache on the GPU: tangents, blocks of many heads.  Tolerances and definitions are
those of tests/test_gpu_paged4.py and tests/paged4_util.py."""
import numpy as np
import pytest
import torch
from torch.autograd import forward_ad

from test_gpu_paged4 import FORMS, Setup, bf16, check_turn, dev, make_form, rc  # noqa: F401 (rc: the fixture)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ tangents
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("back", [False, True])
def test_turns_of_dual_tensors_have_tangents(rc, dtype, back):  # noqa: F811
    """The turn is linear: its tangent is the tangent's turn, of the definition's and bit for bit the call's, with and without
    recorded gradients, for a broadcast tangent, on the caller's stream, and through the turn back."""
    rng = np.random.default_rng(31)
    form = FORMS[3]
    pos = rng.integers(0, 50000, (3, 21)).astype(np.int32)
    pd, f = dev(pos), make_form(rc, form)
    x, t = (torch.from_numpy(rng.standard_normal((21, 4, 128)).astype(np.float32)).to(dtype) for _ in range(2))
    xd, td = x.cuda(), t.cuda()
    axes = rc.RopeAxes((22, 21, 21))
    turns = [lambda y, **kw: rc.rc_rope_turn(y, pd, f, back=back, **kw), lambda y, **kw: rc.rc_rope_axes(y, pd, axes, inverse=back, **kw)]
    stream = torch.cuda.Stream()
    for i, turn in enumerate(turns):
        value, want = turn(xd), turn(td)
        if i == 0:
            check_turn(form, t, pos, want, -1.0 if back else 1.0)
        with forward_ad.dual_level():
            assert forward_ad.unpack_dual(turn(xd)).tangent is None
            for leaf in (xd, xd.clone().requires_grad_()):
                y = forward_ad.unpack_dual(turn(forward_ad.make_dual(leaf, td)))
                assert torch.equal(y.primal, value) and torch.equal(y.tangent, want) and y.primal.requires_grad == leaf.requires_grad
            with torch.no_grad():
                y = forward_ad.unpack_dual(turn(forward_ad.make_dual(xd, td)))
                assert torch.equal(y.primal, value) and torch.equal(y.tangent, want)
            one = torch.ones((), dtype=dtype, device="cuda").expand(xd.shape)
            y = forward_ad.unpack_dual(turn(forward_ad.make_dual(xd, one)))
            assert torch.equal(y.tangent, turn(one.contiguous()))
            stream.wait_stream(torch.cuda.current_stream())
            y = forward_ad.unpack_dual(turn(forward_ad.make_dual(xd, td), stream=stream))
            stream.synchronize()
            assert torch.equal(y.primal, value) and torch.equal(y.tangent, want)
            for a, out in ((forward_ad.make_dual(xd, td), torch.empty_like(xd)), (xd, forward_ad.make_dual(torch.empty_like(xd), td))):
                with pytest.raises(RuntimeError):
                    turn(a, out=out)
            dt = td.clone().requires_grad_()  # the gradient of a tangent
            y = forward_ad.unpack_dual(turn(forward_ad.make_dual(xd, dt)))
            (g,) = torch.autograd.grad(y.tangent, dt, td)
            assert torch.equal(g, rc.rc_rope_turn(td, pd, f, back=not back) if i == 0 else rc.rc_rope_axes(td, pd, axes, inverse=not back))


# ------------------------------------------------------------------ blocks of six heads
SIX_FORMS = [(64, FORMS[0]), (64, FORMS[1]), (64, (64, 6, (9,), "halves", {})), (64, None), (128, FORMS[2]), (128, FORMS[5]),
             (128, (128, 2, (41,), "halves", {"gain": 3.0})), (128, None)]


@pytest.mark.parametrize("dim,form,heads,page,many", [(d, f, h, p, True) for d, f in SIX_FORMS for h, p in ((6, 64), (7, 16), (9, 128), (11, 32))] +
                         [(d, f, h, p, False) for d, f in SIX_FORMS[1:7:2] for h, p in ((7, 32), (11, 64))])
def test_write_blocks_of_six_heads(rc, dim, form, heads, page, many):  # noqa: F811
    """Writes that are large enough for blocks of six heads, and fewer in the last ones: many sequences of one to three tokens, or two
    long ones; they begin and end inside a run of 16 tokens, next to tokens that keep their bits."""
    seqs = [(1 + i % 3, 1 + i % 3 + (7 * i) % 43) for i in range(160)] if many else [(1300, 1307), (1291, 1300)]
    runs = (max(n for n, _ in seqs) + 14) // 16 + 1
    assert len(seqs) * runs * -(-heads // 6) >= 2 * 152  # (the rule of the launch)
    s = Setup(rc, seqs, heads, dim, page, seed=dim + heads + page)
    t = s.tokens
    qkv = bf16(s.rng, t, 3 * heads, dim)
    pos = None if form is None else s.rng.integers(0, 200000, (len(form[2]), t)).astype(np.int32)
    dq = qkv.cuda()
    s.write(dq[:, heads:2 * heads], dq[:, 2 * heads:], pos, form)
    s.check_write(qkv[:, heads:2 * heads], qkv[:, 2 * heads:], pos, form)


def test_write_neighbouring_pairs_of_narrow_heads(rc):  # noqa: F811
    for form in (FORMS[1], (64, 4, (5, 0, 20), "pairs", {"gain": 0.3})):
        for page in (16, 64):
            s = Setup(rc, [(5, 9), (0, 12), (40, 40), (1, 70), (2, 131)], 3, 64, page, seed=page)
            K, V = bf16(s.rng, s.tokens, 3, 64), bf16(s.rng, s.tokens, 3, 64)
            pos = s.rng.integers(0, 200000, (len(form[2]), s.tokens)).astype(np.int32)
            s.write(K.cuda(), V.cuda(), pos, form)
            s.check_write(K, V, pos, form)

"""Edges of the rotary forms and of the 4-bit paged cache on the GPU: tangents.  Tolerances and definitions are
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

"""Grads clipped in place that an autograd graph has saved."""
import pytest
import torch

import fsdp_sharded_mixed_flatparameter_gb300 as pkg

pytestmark = pytest.mark.gpu


def saved():
    """A grad that the graph of its own derivative needs: g = 3 w^2, whose square has the derivative 2 g 6 w."""
    w = torch.full((300,), 2.0, device="cuda", requires_grad=True)
    (g,) = torch.autograd.grad((w ** 3).sum(), w, create_graph=True)
    return w, g, (g * g).sum()


@pytest.mark.parametrize("how", ["function", "launch", "out"])
def test_a_graph_that_saved_a_clipped_grad_refuses_it(how):
    w, g, second = saved()
    x = torch.ones(300, device="cuda")
    if how == "function":
        pkg.clip_grad_norm_([None, g.detach()], 1.0)
    elif how == "launch":
        pkg.GradClip([300, 300], max_norm=1.0).launch([x, g.detach()])
    else:
        pkg.GradClip([300], max_norm=1.0).launch([x], out=[g.detach()])
    assert float(g.detach()[0]) < 1.0
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        second.backward()


def test_norms_and_other_destinations_leave_it_usable():
    w, g, second = saved()
    y = torch.zeros(300, device="cuda")
    c = pkg.GradClip([300], max_norm=1.0)
    c.launch_norms([g.detach()])
    c.launch([g.detach()], out=[y])
    c.launch([g.detach()], out=[None])
    second.backward()
    assert torch.equal(w.grad, torch.full_like(w, 2 * 12.0 * 12.0)) and y._version == 1


def test_inference_tensors_have_no_version():
    with torch.inference_mode():
        x = torch.full((4,), 2.0, device="cuda")
        assert float(pkg.clip_grad_norm_([x], 1.0)) == 4.0
        assert torch.allclose(x, torch.full_like(x, 0.5))

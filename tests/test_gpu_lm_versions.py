"""What a call writes in place counts as modified: a graph that kept a tensor from before refuses its backward."""
import pytest
import torch

from linear_recurrence_sequence_amd import autograd, lm
from tests.helpers import say

pytestmark = pytest.mark.gpu
bf = torch.bfloat16


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("step", [1, 1.0], ids=["quick", "checked"])
def test_a_step_between_forward_and_backward(bits, step):
    say(f"[lm] a step between forward and backward, bits={bits}")
    g = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn(20, 64, generator=g, device="cuda").to(bf).requires_grad_()
    w = torch.randn(90, 64, generator=g, device="cuda").to(bf).requires_grad_()
    t = torch.randint(0, 90, (20,), generator=g, device="cuda")
    s = lm.adamw_state(w, bits)
    more = dict(m_scales=[s["m_scale"]], v_scales=[s["v_scale"]]) if bits == 8 else {}
    loss = autograd.linear_ce(h, w, t)[0].sum()
    grad = torch.ones_like(w)
    lm.adamw_step([w], [grad], [s["m"]], [s["v"]], step=step, lr=1e-3, **more)
    assert grad._version == 0
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_outputs_given():
    say("[lm] outputs given")
    x, k = torch.randn(6, 64, device="cuda"), torch.ones(64, device="cuda", requires_grad=True)
    kept = (x * k).sum()                                     # keeps x
    lm.block_norm_fwd(x, x.clone(), None, None, None, k, r=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        kept.backward()
    h, w, t = x.to(bf), torch.randn(9, 64, device="cuda").to(bf), torch.zeros(6, dtype=torch.int64, device="cuda")
    outs = dict(loss=torch.empty(6, device="cuda"), lse=torch.empty(6, device="cuda"))
    lm.linear_ce_fwd(h, w, t, **outs)
    grads = dict(dh=torch.empty_like(h), dw=torch.empty_like(w))
    lm.linear_ce_bwd(h, w, t, outs["lse"], outs["loss"], **grads)
    assert all(a._version == 1 for a in (*outs.values(), *grads.values())) and w._version == 0
    with torch.inference_mode():                             # these have no versions
        y = torch.randn(6, 64, device="cuda")
        s = lm.adamw_state(y)
        lm.block_norm_fwd(y, y.clone(), None, None, None, k, r=y)
        lm.adamw_step([y], [y.clone()], [s["m"]], [s["v"]], step=1, lr=1e-3)
        lm.adamw_step([y], [y.clone()], [s["m"]], [s["v"]], step=2.0, lr=1e-3)

"""Tensors of another device than the current one are refused: a launch and its stream are the current device's.

One device is enough: the binding is told that another one is current."""
import pytest
import torch

from linear_recurrence_sequence_amd import lm
from tests.helpers import say

pytestmark = pytest.mark.gpu
bf = torch.bfloat16


def test_another_device_is_current(monkeypatch):
    say("[lm] another device is current")
    x, k = torch.randn(4, 64, device="cuda"), torch.ones(64, device="cuda")
    h, w, t = x.to(bf), torch.randn(90, 64, device="cuda").to(bf), torch.zeros(4, dtype=torch.int64, device="cuda")
    st = lm.adamw_state(x)
    r, n, stats = lm.block_norm_fwd(x, x, None, None, None, k)
    loss, lse = lm.linear_ce_fwd(h, w, t)
    calls = [lambda: lm.block_norm_fwd(x, x, None, None, None, k), lambda: lm.block_norm_bwd(x, x, None, None, None, k, stats, r, n),
             lambda: lm.linear_ce_fwd(h, w, t), lambda: lm.linear_ce_bwd(h, w, t, lse, loss),
             lambda: lm.adamw_step([x], [x.clone()], [st["m"]], [st["v"]], step=1, lr=0.0)]
    for f in calls:
        f()
    torch.cuda.synchronize()
    bind = lm._native()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    bind.setup(lambda: 1, torch._C._cuda_getCurrentRawStream)
    try:
        for f in calls:
            with pytest.raises(ValueError, match="the current device is cuda:1"):
                f()
    finally:
        bind.setup(torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)
    monkeypatch.undo()
    for f in calls:
        f()
    torch.cuda.synchronize()


def test_a_stream_given_to_adamw():
    """A step that is no integer goes by the Python checks."""
    say("[adamw] a stream given")
    p = [torch.randn(300, device="cuda") for _ in range(3)]
    g = [torch.randn(300, device="cuda") for _ in p]
    want, got = [t.clone() for t in p], [t.clone() for t in p]
    state = [[lm.adamw_state(t) for t in p] for _ in range(2)]
    lm.adamw_step(want, g, [s["m"] for s in state[0]], [s["v"] for s in state[0]], step=3, lr=1e-3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    lm.adamw_step(got, g, [s["m"] for s in state[1]], [s["v"] for s in state[1]], step=3.0, lr=1e-3, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))

"""Groups of b and c of one channel each: what one channel holds stays out of its neighbours' group."""
import pytest
import torch

from tests.helpers import say
from tests.test_gpu_ssm_scan import check, inputs, run

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("width,n", [(2, 4), (3, 16), (5, 20), (4, 40)])
def test_groups_of_one_channel(dtype, width, n):
    say(f"[ssm] groups of one channel {dtype} width={width} n={n}")
    length = 40
    k, dy, dh = inputs(2, length, width, n, width, dtype, seed=width)
    clean = run(k, dy, dh)
    check(clean, k, dy, dh, {}, dtype, length)
    for channel in range(width):
        others = [i for i in range(width) if i != channel]
        for name in ("dt", "u", "h0", "z", "dy"):
            m, my = {x: t.clone() for x, t in k.items()}, dy.clone()
            if name == "h0":
                m["h0"][:, channel] = float("nan")
            elif name == "dy":
                my[:, 7, channel] = float("nan")
            else:
                m[name][:, 7, channel] = float("nan")
            got = run(m, my, dh)
            for x, t in got.items():
                at = others if x in ("da", "dd", "ddt_bias") else (slice(None), others) if x in ("h", "dh0") else (slice(None), slice(None), others)
                assert torch.equal(t[at], clean[x][at]), (name, channel, x)

"""Block norms with r written over x: the results are those of a call with outputs of its own."""
import pytest
import torch

from linear_recurrence_sequence_amd import lm
from tests.helpers import say
from tests.test_gpu_lm_norm import EPS, make

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("st,br", [(f32, bf), (bf, f32)], ids=["fb", "bf"])
@pytest.mark.parametrize("full", [True, False], ids=["full", "plain"])
@pytest.mark.parametrize("d", [3, 63, 129, 255, 1021, 1537, 4099, 8195])
def test_rows_in_place(d, full, st, br):
    """r over x: where the width is no multiple of four, the lane at a row's end reads columns that its neighbour writes."""
    for rows in (1, 45, 700):
        say(f"[norm] in place {rows}x{d} full={full} {st}")
        a = make(rows, d, st, br, "silu", full, d)
        w = [a[k] for k in ("x", "y", "gate", "w_post", "scale", "w_pre")]
        r, n, stats = lm.block_norm_fwd(*w, eps=EPS, gate_act="silu")
        x = a["x"].clone()
        r2, n2, s2 = lm.block_norm_fwd(x, *w[1:], eps=EPS, gate_act="silu", r=x)
        assert r2.data_ptr() == x.data_ptr()
        assert torch.equal(r2, r) and torch.equal(n2, n) and torch.equal(s2, stats)

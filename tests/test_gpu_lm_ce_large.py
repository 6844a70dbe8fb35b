"""Linear cross entropy where a launch of one workgroup a tile would pass the threads that one may have.

The vocabulary is one block of entries many times over: lse is the block's and the logarithm of their number, the gradients
follow from the block's.  Tolerances are those of test_gpu_lm_ce.py, for the block."""
import math

import pytest
import torch

from linear_recurrence_sequence_amd import lm
from tests.helpers import say
from tests.test_gpu_lm_ce import exact, make, within

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


def test_a_vocabulary_beyond_one_launch():
    n, d, block, times = 4, 8, 1 << 20, 1025
    say(f"[ce] n={n} d={d} v={block * times}")
    a = make(n, d, block, 21)
    ref = exact(a, 0.0, a["dlse"])
    on = a["t"] >= 0
    w = a["w"].repeat(times, 1)
    t = torch.where(on, a["t"] + block * (times - 1), a["t"])          # the targets lie in the last block
    loss, lse = lm.linear_ce_fwd(a["h"], w, t)
    more = math.log(times)
    within(lse, ref["lse"] + more, ref["ez"] + 1e-6 * (ref["lse"].abs() + more), "lse")
    within(loss, torch.where(on, ref["loss"] + more, torch.zeros_like(ref["loss"])), 2 * ref["ez"] + 1e-6 * (ref["lse"].abs() + more + ref["picked"].abs()), "loss")
    g = lm.linear_ce_bwd(a["h"], w, t, lse, a["dloss"], a["dlse"])
    within(g["dh"], ref["dh"], ref["tol_h"], "dh")
    off = dict(a, t=torch.full_like(t, -1))
    c = torch.where(on, a["dloss"], torch.zeros_like(a["dloss"])) + a["dlse"]
    rest = exact(off, 0.0, c)                                          # a block without targets: all weight as lse's cotangent
    for first in (0, 500):
        within(g["dw"][first * block:(first + 1) * block], rest["dw"] / times, rest["tol_w"] / times, "dw")
    hot = torch.zeros(block, d, dtype=torch.float64, device="cuda")
    hot.index_add_(0, a["t"][on], -(a["dloss"][on].double()[:, None] * a["h"][on].double()))
    size = torch.zeros_like(hot).index_add_(0, a["t"][on], a["dloss"][on].double()[:, None] * a["h"][on].double().abs())
    within(g["dw"][-block:], rest["dw"] / times + hot, rest["tol_w"] / times + (2.0 ** -8 + 2 * float(ref["ez"].max()) + 1e-5) * size, "dw")


def test_no_tokens_and_a_large_head():
    v, d = 1 << 20, 4104
    say(f"[ce] no tokens, v={v} d={d}")
    h, w = torch.zeros(0, d, dtype=bf, device="cuda"), torch.empty(v, d, dtype=bf, device="cuda")
    t, none = torch.zeros(0, dtype=torch.int64, device="cuda"), torch.zeros(0, device="cuda")
    dw = torch.ones(v, d, device="cuda")
    lm.linear_ce_bwd(h, w, t, none, none, dw=dw, dh=torch.empty(0, d, device="cuda"))
    assert float(dw.abs().max()) == 0

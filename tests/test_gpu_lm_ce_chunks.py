"""Linear cross entropy of few tokens over several chunks of the vocabulary, against the definition in 64 bits.

Tolerances are those of test_gpu_lm_ce.py: dz rounded to BF16 (2^-8 of the term) and the error of a logit through exp."""
import pytest
import torch

from linear_recurrence_sequence_amd import lm
from tests.helpers import say
from tests.test_gpu_lm_ce import exact, make, within

pytestmark = pytest.mark.gpu
f32 = torch.float32


@pytest.mark.parametrize("n,d,v", [(141, 72, 557087), (200, 64, 589826), (65, 8, 1100001), (17, 16, 4194304 + 257)])
def test_few_tokens_over_several_chunks(n, d, v):
    """The last chunk is shorter than the first and may not be cut into more ranges of dh's sum; the workspace holds NaN."""
    say(f"[ce] few tokens, several chunks n={n} d={d} v={v}")
    a = make(n, d, v, n)
    lse = lm.linear_ce_fwd(a["h"], a["w"], a["t"])[1]
    need = lm.lib().lm_linear_ce_workspace_bytes(n, d, v, 1)
    ws = torch.full((need // 4,), float("nan"), device="cuda").view(torch.uint8)
    g = lm.linear_ce_bwd(a["h"], a["w"], a["t"], lse, a["dloss"], a["dlse"], grad_dtype=f32, workspace=ws)
    ref = exact(a, 0.0, a["dlse"])
    within(lse, ref["lse"], ref["ez"] + 1e-6 * ref["lse"].abs(), "lse")
    within(g["dh"], ref["dh"], ref["tol_h"], "dh")
    within(g["dw"], ref["dw"], ref["tol_w"], "dw")

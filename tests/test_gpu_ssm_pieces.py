"""The selective scan with segments of several chunks, and the causal convolution with pieces of more than eight tokens, as rows of
real sizes have them.  What the plans give is read off the workspaces' sizes, so that another plan cannot drop these cases unnoticed."""
import pytest
import torch

from linear_recurrence_sequence_amd import ssm
from tests import test_gpu_ssm_conv as conv
from tests import test_gpu_ssm_scan as scan
from tests.helpers import say

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


def segments_of(batch, length, d, n, groups, backward):
    """Segments of a row: the number for which the workspace's parts (rounded to 256 bytes each) add up to its size."""
    size = ssm.lib().ssm_scan_workspace_bytes(batch, length, d, n, groups, int(backward))
    ng = next(g for g in (2, 4, 8, 16) if 4 * g >= n)
    blocks = -(-(-(-(d // groups) // (128 // ng))) // 4)

    def take(floats):
        return (4 * floats + 255) // 256 * 256

    for s in range(1, 65):
        parts = batch * s
        need = take(parts * 2 * n * d if s > 1 else 0)
        if backward:
            need += take(groups * blocks * batch * length * 8 * ng) + take(parts * n * d) + take(parts * 2 * d)
        if max(need, 256) == size:
            return s
    raise AssertionError("no number of segments fits the workspace")


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("batch,length,d,n,groups,several,gate,packed,ragged", [
    (16, 104, 4096, 8, 1, True, True, False, False), (15, 100, 4097, 3, 1, True, False, True, True), (40, 57, 4096, 8, 1, False, True, True, False),
    (8, 112, 4096, 16, 1, True, True, False, False), (8, 101, 4090, 13, 2, True, False, True, False), (8, 97, 4095, 16, 1, True, True, True, True),
    (20, 70, 4096, 16, 4, False, False, False, True), (4, 108, 4096, 32, 1, True, True, True, True), (4, 100, 4084, 20, 4, True, False, False, False),
    (2, 110, 4096, 64, 1, True, True, False, True), (2, 97, 3999, 40, 3, True, False, True, False), (5, 66, 4096, 64, 1, False, True, True, True),
])
def test_segments_of_several_chunks(dtype, batch, length, d, n, groups, several, gate, packed, ragged):
    """several: rows of two or more segments of three chunks or more each (but the last); else one segment of all."""
    say(f"[ssm] segments {dtype} batch={batch} length={length} d={d} n={n} groups={groups} gate={gate} packed={packed} ragged={ragged}")
    chunks = -(-length // 16)
    for backward in (False, True):
        s = segments_of(batch, length, d, n, groups, backward)
        assert (s > 1) is several and -(-chunks // s) >= 3, (backward, s)
    k, dy, dh = scan.inputs(batch, length, d, n, groups, dtype, seed=length, gate=gate)
    kw = {}
    if packed:
        kw["reset"] = scan.flags(batch, length, 1, 0.03)
    if ragged:
        kw["lengths"] = torch.linspace(0, length, batch, device="cuda").to(torch.int32).flip(0)
    scan.check(scan.run(k, dy, dh, **kw), k, dy, dh, kw, dtype, length)


@pytest.mark.parametrize("batch,length,d,n", [(1, 2500, 64, 8), (2, 2300, 24, 33)])
def test_long_narrow_rows(batch, length, d, n):
    """Rows cut into many segments of several chunks each."""
    say(f"[ssm] long and narrow batch={batch} length={length} d={d} n={n}")
    s = segments_of(batch, length, d, n, 1, True)
    assert s > 20 and -(-length // 16) / s >= 2
    k, dy, dh = scan.inputs(batch, length, d, n, 1, bf, seed=length, scale=0.3)
    kw = dict(reset=scan.flags(batch, length, 2, 0.002), lengths=torch.tensor([length - 100, length][:batch], dtype=torch.int32, device="cuda"))
    scan.check(scan.run(k, dy, dh, **kw), k, dy, dh, kw, bf, length)


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("batch,length,d,width,act,tokens", [(3, 1407, 2050, 4, "silu", 24), (2, 5003, 1701, 3, "none", 40), (1, 33001, 1031, 4, "silu", 64),
                                                             (4, 16411, 1028, 2, "silu", 64)])
def test_pieces_of_the_convolution(dtype, batch, length, d, width, act, tokens):
    """The backward's pieces are of `tokens`; the forward's are half as long, or as long where that is the most."""
    say(f"[conv] pieces {dtype} batch={batch} length={length} d={d} width={width} {act}")
    pieces = ssm.lib().ssm_conv_bwd_workspace_bytes(batch, length, d, width) // (batch * (width + 1) * d * 4)
    assert -(-length // tokens) == pieces
    k, dy, do = conv.inputs(batch, length, d, width, dtype, seed=length)
    g = torch.Generator(device="cuda").manual_seed(width)
    kw = dict(reset=(torch.rand(batch, length, generator=g, device="cuda") < 0.01).to(torch.uint8),
              lengths=torch.tensor([length - 777, length, length - 1, length // 3][:batch], dtype=torch.int32, device="cuda"))
    conv.check(conv.run(k, dy, do, act, **kw), k, dy, do, act, kw, dtype)

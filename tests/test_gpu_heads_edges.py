"""Rotary positions, norms and appends in calls that their documentation allows
and that are out of the ordinary: through the C entry points, and at positions
far from zero."""
import math
from fractions import Fraction

import pytest
import torch

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("d", [64, 90])
@pytest.mark.parametrize("kind", [1, 2])
def test_no_weights_have_no_stride(gpu_lib, d, kind):
    """a null weight is a factor left out, whatever its stride: in 16-byte pieces
    (d 64) and element by element (d 90)"""
    lib, rows, Hq, Hk = gpu_lib.load(), 21, 4, 2
    x = torch.randn(rows, Hq + Hk, d, generator=gen(1)).bfloat16().cuda()
    w = (torch.rand(Hk, d, generator=gen(2)) + 0.5).bfloat16().cuda()
    pos, f = ints(list(range(rows))), torch.rand(8, generator=gen(3)).cuda()
    got = []
    for head in (0, d):
        q, k = (torch.full((rows, H, d), float("nan"), dtype=torch.bfloat16, device="cuda")
                for H in (Hq, Hk))
        code = lib.gdn_qk_norm_rope(
            x.data_ptr(), (Hq + Hk) * d, d, x.data_ptr() + 2 * Hq * d, (Hq + Hk) * d, d, 1, kind, 1e-6,
            0.0, None, head, w.data_ptr(), d, 1, pos.data_ptr(), None, 1, f.data_ptr(), 16, 0, 1.0,
            q.data_ptr(), Hq * d, d, k.data_ptr(), Hk * d, d, rows, Hq, Hk, d,
            torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert code == 0
        got.append((q, k))
    for a, b in zip(*got):
        assert torch.isfinite(a).all() and torch.equal(a, b)

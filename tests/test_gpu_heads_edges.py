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


# 2 pi to 80 digits
TWO_PI = 2 * Fraction(int("31415926535897932384626433832795028841971693993751058209749445923078164062862089"),
                      10 ** 79)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d", [64, 42])
def test_far_positions_are_as_good_as_near_ones(gpu_lib, d, layout):
    """cos and sin themselves, of positions up to 2^32 at frequencies near 1.

    The angle, in half turns between -1 and 1, is rounded to fp32 once: half a
    step there is at most 2^-25, or pi 2^-25 in radians, which neither cos nor
    sin enlarges.  Their own error is two steps of numbers up to 1, 2 * 2^-24; a
    turn of (1, 0) adds nothing."""
    tol = math.pi * 2.0 ** -25 + 2 * 2.0 ** -24
    f = torch.rand(16, generator=gen(5)) * 0.2 + 0.8
    i = torch.arange(16)
    a, b = (i, i + 16) if layout == "half" else (2 * i, 2 * i + 1)
    for low, base in ((0, 0), (2 ** 28, 0), (2 ** 31 - 2 ** 24, 0), (2 ** 31 - 2 ** 24, 2 ** 31 - 1),
                      (-2 ** 31, -2 ** 31)):
        at = torch.randint(low, low + 2 ** 24, (400,), generator=gen(6))
        x = torch.zeros(1, 400, 1, d)
        x[..., a] = 1
        got = gpu_lib.rope(x.cuda(), None, at.int()[None].cuda(), f.cuda(), layout=layout,
                           base=ints([base]))[0][0, :, 0].cpu().double()
        angle = torch.tensor([[float((p + base) * Fraction(y) % TWO_PI) for y in f.tolist()]
                              for p in at.tolist()], dtype=torch.float64)
        off = max((got[:, a] - angle.cos()).abs().max(), (got[:, b] - angle.sin()).abs().max())
        print(low, base, float(off), flush=True)
        assert off <= tol, (low, base)

"""Biases by the thousand: more of them in one wave's tokens than its list holds
(432), where the sequence's are gone over instead.  Values are exact in fp32 as
in the other tests of the logits (sums of 4096 eighths up to 30 need 18 bits), so
results are equal to the 64-bit ones bit for bit."""
import numpy as np
import pytest
import torch

from test_gpu_logits import DT, ints, make, reference, same, upload

pytestmark = pytest.mark.gpu


def biased(batch, n, V, dtype, seed, tokens, mask="one"):
    """a case with these bias tokens [m] in every sequence, each in an order of its own"""
    x = make(batch, n, V, dtype, seed, bias=len(tokens), mask=mask)
    rng = np.random.default_rng(seed + 1)
    x["bias"] = (np.stack([rng.permutation(tokens) for _ in range(batch)]), x["bias"][1])
    return x


def check(lib, x, out):
    ref, best, _ = reference(x)
    z, kw = upload(x)
    st = ints([-1] * x["batch"])
    assert torch.equal(lib.adjust_logits(z, status=st, **kw).cpu().long(), best)
    assert not st.any()
    o = torch.full(z.shape, float("nan"), dtype=DT[out], device="cuda")
    assert torch.equal(lib.adjust_logits(z, out=o, **kw).cpu().long(), best)
    same(o, ref, DT[out])


@pytest.mark.parametrize("m", [432, 433, 1000, 4096])
@pytest.mark.parametrize("batch,n,V,dtype", [
    (1, 1, 32000, "bf16"),            # a slice a wave
    (2, 40, 5003, "fp32"),
    (16, 128, 13001, "bf16"),         # many slices a wave: touched tokens put off
    (50, 128, 4500, "fp16"),          # one wave a node
])
@pytest.mark.parametrize("spread", [7, 300, 4000])
def test_more_biases_than_a_wave_lists(gpu_lib, m, batch, n, V, dtype, spread):
    """all in one slice, with repeats, or in the wave's first eight; some outside the
    vocabulary"""
    rng = np.random.default_rng(m + spread)
    tokens = rng.integers(0, spread, m)
    if m > 433:
        tokens[::50] = rng.choice([-1, V, V + 5, 2 ** 31 - 1, -2 ** 31], len(tokens[::50]))
    check(gpu_lib, biased(batch, n, V, dtype, 51, tokens), "fp32")


@pytest.mark.parametrize("batch,n", [(1, 1), (16, 128), (50, 128)])
@pytest.mark.parametrize("m", [433, 2000])
def test_some_waves_list_theirs_and_some_cannot(gpu_lib, batch, n, m):
    """the first tokens have m biases, the others a few a slice; the row's last slice
    is cut"""
    V = 13001
    rng = np.random.default_rng(m)
    tokens = np.concatenate([rng.integers(0, 200, m), rng.integers(0, V, 300), [V - 1, V, V + 500]])
    check(gpu_lib, biased(batch, n, V, "bf16", 53, tokens, mask="node"), "bf16")


@pytest.mark.parametrize("m", [9, 64, 65, 432, 433, 4096])
@pytest.mark.parametrize("batch,n", [(1, 1), (16, 128)])
def test_biases_of_a_token_add_up_in_order(gpu_lib, m, batch, n):
    """arbitrary values on 20 tokens: every sum is rounded, one after the other"""
    V = 13001
    rng = np.random.default_rng(m)
    tok = rng.integers(0, 20, (batch, m)) * 25
    val = rng.standard_normal((batch, m)).astype(np.float32)
    want = np.zeros((batch, V), dtype=np.float32)
    for b in range(batch):
        for t, y in zip(tok[b], val[b]):
            want[b, t] += y
    want = torch.from_numpy(want)[:, None].expand(batch, n, V)
    z = torch.zeros(batch, n, V, device="cuda")
    bias = (ints(tok), torch.from_numpy(val).cuda())
    o = torch.full_like(z, float("nan"))
    best = gpu_lib.adjust_logits(z, bias=bias, out=o)
    assert torch.equal(o.cpu(), want)
    assert torch.equal(best.cpu().long(), want.argmax(-1))
    assert torch.equal(gpu_lib.adjust_logits(z, bias=bias), best)

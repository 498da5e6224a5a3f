"""The rotary serving example against a plain 64-bit form of its model, token by
token: rotated and normalised queries and keys, the attention that reads them,
and the penalised logits.

The bounds count roundings.  The plain form rounds to bf16 where the example does:
the DeltaNet layer's queries, keys and values, the projections of the attention
layer, its queries and keys once more after norm and rotation, and its output.
What is left is what fp32 sums may flip: the queries, keys and values of either
side round to neighbouring numbers here and there, and the softmax weights round,
at most half a step of bf16 (2^-8) each, independent over keys and elements.
Four of them, 4 * 2^-8 of the attention layer's part of a token's logits in the
2-norm, leave room for all; a penalty makes a difference at most REPETITION times
as large.  Mistakes are planted in the plain form, on the CPU: every one has to
pass the bound by far.
"""
import importlib.util
import math
import os

import pytest

torch = pytest.importorskip("torch")

BOUND = 4 * 2.0 ** -8


def example(device):
    folder = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")
    spec = importlib.util.spec_from_file_location("serve_rotary_" + device,
                                                  os.path.join(folder, "serve_rotary.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def bf16(x):
    return x.float().bfloat16().double()


def delta_net(ex, w, seq, first, rounded):
    """the DeltaNet layer's output of every token; its values are rounded to bf16 for
    the first tokens, and for the others where asked for (single tokens; trees keep fp32)"""
    H, DK = ex.base.HEADS, ex.base.DK
    x = w["embed"][seq]
    q, k, v = (x @ w["w_qkv"]).unflatten(-1, (3, H, DK)).unbind(1)
    q, k = (bf16(y / y.norm(dim=-1, keepdim=True)) for y in (q, k))
    v, gate = bf16(v), x @ w["w_gate"]
    alpha = torch.exp(-torch.nn.functional.softplus(gate[:, :H] - 2))
    beta = torch.sigmoid(gate[:, H:])
    S, o = torch.zeros(H, DK, DK, dtype=torch.float64), []
    for t in range(len(seq)):
        S = alpha[t][:, None, None] * S
        u = beta[t][:, None] * (v[t] - (S * k[t][..., None]).sum(-2))
        S = S + k[t][..., None] * u[:, None, :]
        o.append((S * q[t][..., None]).sum(-2))
    o = torch.stack(o)
    o = torch.cat([bf16(o[:first]), bf16(o[first:]) if rounded else o[first:]])
    return x + o.flatten(1) @ w["w_out"]


def normed(x, weight):
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight


def turned(x, pos, f, scale):
    """the first half of each head by complex products, pairs (i, i + D / 4)"""
    r = len(f)
    z = torch.complex(x[..., :r], x[..., r:2 * r])
    a = pos.double()[:, None] * f
    z = z * torch.polar(torch.full_like(a, scale), a)[:, None]
    return torch.cat([z.real, z.imag, x[..., 2 * r:]], -1)


def plain(ex, weights, prompt, tokens, rounded, mistake=None):
    """the penalised logits of `tokens` after `prompt`, and the attention layer's part
    of the logits"""
    w, q_weight, k_weight, f, scale = weights
    seq, first = torch.cat([prompt, tokens]).cpu().long(), len(prompt)
    n = len(seq)
    h = delta_net(ex, w, seq, first, rounded)
    q, k, v = bf16(h @ w["a_qkv"]).unflatten(-1, (-1, ex.D)).split(
        (ex.QHEADS, ex.KVHEADS, ex.KVHEADS), dim=1)
    pos = torch.arange(n)
    late = pos >= first
    q_pos, k_pos = pos.clone(), pos.clone()
    if mistake == "queries from the prompt's end":
        q_pos[late] -= first
    if mistake == "queries and keys from the prompt's end":
        q_pos[late] -= first
        k_pos[late] -= first
    if mistake == "queries a token late":
        q_pos[late] += 1
    if mistake == "keys of a chunk from its start":
        k_pos = torch.where(late, pos, pos % 16)
    if mistake == "no magnitude":
        scale = 1.0
    if mistake == "plain frequencies":
        f = 10000.0 ** (-torch.arange(len(f), dtype=torch.float64) / len(f))
    if mistake == "weights exchanged":
        q_weight, k_weight = k_weight, q_weight
    q = normed(q, 1.0 if mistake == "no weights" else q_weight)
    k = normed(k, 1.0 if mistake == "no weights" else k_weight)
    q, k = turned(q, q_pos, f, scale), turned(k, k_pos, f, scale)
    if mistake == "turned backwards":
        k = turned(turned(k, -pos, f, 1.0 / scale), -pos, f, scale)
    q, k = bf16(q), bf16(k)
    k, v = (y.repeat_interleave(ex.QHEADS // ex.KVHEADS, 1) for y in (k, v))
    z = (q.transpose(0, 1) @ k.transpose(0, 1).transpose(1, 2)) * ex.D ** -0.5
    see = torch.ones(n, n, dtype=torch.bool).tril()
    if mistake == "a key not appended" and n > first + 1:
        see[first + 1:, first] = False
    p = torch.softmax(z.masked_fill(~see, -math.inf), -1)
    a = bf16((p @ v.transpose(0, 1)).transpose(0, 1))
    if mistake == "no attention output":
        a = torch.zeros_like(a)
    part = (a.flatten(1) @ w["a_out"] @ w["embed"].t())[first:]
    logits = (h @ w["embed"].t())[first:] + part
    said, asked = torch.zeros(ex.VOCAB, dtype=torch.float64), torch.zeros(ex.VOCAB, dtype=torch.bool)
    asked[seq[:first]] = mistake != "prompt not marked"
    out = []
    for t, y in zip(seq[first:], logits):
        if mistake != "own token not counted":
            said[t] += 1
        y = torch.where(asked | (said > 0), torch.where(y > 0, y / ex.REPETITION, y * ex.REPETITION), y)
        out.append(y - torch.where(said > 0, ex.PRESENCE + ex.FREQUENCY * said, 0.0))
        if mistake == "own token not counted":
            said[t] += 1
    return torch.stack(out), part


def off(ex, got, ref, part):
    """the largest of the tokens' distances, relative to the attention's part"""
    return float(((got.cpu().double() - ref).norm(dim=-1) / part.norm(dim=-1)).max()) / ex.REPETITION


def weights_of(model, q_weight, k_weight, f, scale):
    w = {n: getattr(model, n).cpu().double()
         for n in ("embed", "w_qkv", "w_out", "w_gate", "a_qkv", "a_out")}
    return w, q_weight.cpu().double(), k_weight.cpu().double(), f.cpu().double(), scale


@pytest.mark.gpu
@pytest.mark.parametrize("prompt_len", [1, 16, 150])
def test_example_follows_its_model(prompt_len):
    ex = example("cuda")
    r = ex.serve(prompt_len=prompt_len, rounds=4, seed=3)
    s = r["server"]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    prompt = torch.randint(ex.VOCAB, (prompt_len,), generator=gen, device="cuda")
    weights = weights_of(r["model"], s.q_weight, s.k_weight, s.inv_freq, s.magnitude)
    tokens = torch.tensor(r["emitted"][0])
    for got, rounded in ((r["logits"], False), (r["again"], True)):
        ref, part = plain(ex, weights, prompt.cpu(), tokens, rounded)
        assert got.shape == ref.shape
        print(prompt_len, rounded, off(ex, got, ref, part), BOUND, flush=True)
        assert off(ex, got, ref, part) <= BOUND


MISTAKES = ["queries from the prompt's end", "queries a token late",
            "queries and keys from the prompt's end", "no magnitude", "plain frequencies",
            "no weights", "turned backwards", "a key not appended", "no attention output",
            "prompt not marked", "own token not counted"]


# a prompt of one chunk has its keys in place, and weights of random signs next to
# 1 take many keys to tell apart
@pytest.mark.parametrize("mistake,prompt_len", [(m, n) for m in MISTAKES for n in (1, 16, 150)] + [
    ("keys of a chunk from its start", 150), ("weights exchanged", 150)])
def test_the_bound_catches_mistakes(mistake, prompt_len, monkeypatch):
    """the plain form with a mistake against itself"""
    ex = example("cpu")
    monkeypatch.setattr(ex.base, "DEV", "cpu")
    gen = torch.Generator()
    gen.manual_seed(6)
    q_weight, k_weight = (1 + 0.1 * torch.randn(ex.D, generator=gen) for _ in range(2))
    f, scale = ex.g.rope_frequencies(ex.D // 2, scaling="yarn", factor=4, original=64, low=1, high=8,
                                     device="cpu")
    weights = weights_of(ex.base.Model(5), q_weight, k_weight, f, scale)
    prompt = torch.randint(ex.VOCAB, (prompt_len,), generator=gen)
    tokens = torch.randint(ex.VOCAB, (8,), generator=gen)
    for rounded in (False, True):
        ref, part = plain(ex, weights, prompt, tokens, rounded)
        got, _ = plain(ex, weights, prompt, tokens, rounded, mistake)
        print(mistake, prompt_len, rounded, off(ex, got, ref, part), flush=True)
        assert off(ex, got, ref, part) > 3 * BOUND

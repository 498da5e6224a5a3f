"""The serving example against a plain 64-bit form of its model, token by token.

The bounds count roundings.  An attention output differs by the rounding of its
weights and its own, at most half a step of bf16 (2^-8) each, independent over
keys and elements; the queries, keys and values of either side may round to
neighbouring bf16 numbers where fp32 sums differ.  Four of them, 4 * 2^-8 of the
attention layer's part of a token's logits in the 2-norm, leave room for all.  Fp32 sums
of 128 terms are off by about 2^-20.5 and flip a bf16 rounding with a
probability of 2^-11.5: states, linear in rounded values, differ by 2^-8 of a
flipped one, 2^-13.75 of the whole in the 2-norm; eight of these bound them.
Mistakes are planted in the plain form, on the CPU: every one has to pass the
bounds by far.
"""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

LOGITS = 4 * 2.0 ** -8
STATES = 8 * 2.0 ** -13.75


def example(device):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "serve_tree.py")
    spec = importlib.util.spec_from_file_location("serve_tree_" + device, path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.DEV = device
    return mod


def bf16(x):
    return x.float().bfloat16().double()


def plain(ex, model, prompt, tokens, rounded, mistake=None):
    """logits of `tokens` after `prompt`, the attention layer's part of them,
    and the DeltaNet state at the end.  rounded: the tokens' DeltaNet outputs
    are rounded to bf16, as the prompt's are (single tokens; trees keep fp32)."""
    w = {n: getattr(model, n).cpu().double()
         for n in ("embed", "w_qkv", "w_out", "w_gate", "a_qkv", "a_out")}
    seq, first = torch.cat([prompt, tokens]).cpu().long(), len(prompt)
    n, H, DK = len(seq), ex.HEADS, ex.DK
    x = w["embed"][seq]
    q, k, v = (x @ w["w_qkv"]).unflatten(-1, (3, H, DK)).unbind(1)
    q, k = (bf16(y / y.norm(dim=-1, keepdim=True)) for y in (q, k))
    v, gate = bf16(v), x @ w["w_gate"]
    alpha = torch.exp(-torch.nn.functional.softplus(gate[:, :H] - 2))
    beta = torch.sigmoid(gate[:, H:])
    if mistake == "gates of the token before":
        alpha[first:], beta[first:] = alpha[first - 1:-1].clone(), beta[first - 1:-1].clone()
    S, o = torch.zeros(H, DK, DK, dtype=torch.float64), torch.zeros(n, H, DK, dtype=torch.float64)
    for t in range(n):
        if mistake == "state not forked" and t == first:
            S = torch.zeros_like(S)
        M = alpha[t][:, None, None] * S
        u = beta[t][:, None] * (v[t] - (M * k[t][..., None]).sum(-2))
        M = M + k[t][..., None] * u[:, None, :]
        o[t] = (M * q[t][..., None]).sum(-2)
        if not (mistake == "a token not committed" and t == first):
            S = M
    o = torch.cat([bf16(o[:first]), bf16(o[first:]) if rounded else o[first:]])
    if mistake == "no DeltaNet output":
        o = torch.zeros_like(o)
    h = x + o.flatten(1) @ w["w_out"]
    G = ex.QHEADS // ex.KVHEADS
    aq, ak, av = bf16(h @ w["a_qkv"]).unflatten(-1, (-1, ex.D)).split(
        (ex.QHEADS, ex.KVHEADS, ex.KVHEADS), dim=1)
    ak, av = (y.repeat_interleave(G, 1) for y in (ak, av))
    z = (aq.transpose(0, 1) @ ak.transpose(0, 1).transpose(1, 2)) * ex.D ** -0.5
    see = torch.ones(n, n, dtype=torch.bool).tril()
    if mistake == "keys not appended":
        see[first:, first:] = torch.eye(n - first, dtype=torch.bool)
    if mistake == "nodes see each other":
        see[first:, first:] = True
    p = torch.softmax(z.masked_fill(~see, float("-inf")), -1)
    a = bf16((p @ av.transpose(0, 1)).transpose(0, 1))
    if mistake == "no attention output":
        a = torch.zeros_like(a)
    part = a.flatten(1) @ w["a_out"] @ w["embed"].t()
    return (h @ w["embed"].t() + part)[first:], part[first:], S


def logits_off(got, ref, part):
    """the largest of the tokens' distances, relative to the attention's part"""
    return float(((got.cpu().double() - ref).norm(dim=-1) / part.norm(dim=-1)).max())


def state_off(got, ref):
    return float((got.cpu().double() - ref).norm() / ref.norm())


@pytest.mark.gpu
@pytest.mark.parametrize("prompt_len", [1, 16, 150])
def test_example_follows_its_model(prompt_len):
    ex = example("cuda")
    r = ex.serve(prompt_len=prompt_len, rounds=4, seed=3)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    prompt = torch.randint(ex.VOCAB, (prompt_len,), generator=gen, device="cuda")
    tokens = torch.tensor(r["emitted"][0])
    s = r["server"]
    for got, slot, rounded in ((r["logits"], 0, False), (r["again"], s.replay, True)):
        ref, part, S = plain(ex, r["model"], prompt.cpu(), tokens, rounded)
        assert got.shape == ref.shape
        print(prompt_len, rounded, logits_off(got, ref, part), state_off(s.S[slot], S), flush=True)
        assert logits_off(got, ref, part) <= LOGITS
        assert state_off(s.S[slot], S) <= STATES
    # the two ways leave the same state, their inputs rounded alike
    assert state_off(s.S[0], s.S[s.replay].cpu().double()) <= STATES


@pytest.mark.parametrize("prompt_len", [1, 16, 150])
@pytest.mark.parametrize("mistake,state", [
    ("no DeltaNet output", False), ("no attention output", False), ("state not forked", True),
    ("a token not committed", True), ("gates of the token before", True),
    ("keys not appended", False), ("nodes see each other", False),
])
def test_bounds_catch_mistakes(mistake, state, prompt_len):
    """the plain form with a mistake against itself: past the logits' bound, and
    past the state's where the mistake is in the state"""
    ex = example("cpu")
    model = ex.Model(5)
    gen = torch.Generator()
    gen.manual_seed(6)
    prompt = torch.randint(ex.VOCAB, (prompt_len,), generator=gen)
    tokens = torch.randint(ex.VOCAB, (8,), generator=gen)
    for rounded in (False, True):
        ref, part, S = plain(ex, model, prompt, tokens, rounded)
        got, _, wrong = plain(ex, model, prompt, tokens, rounded, mistake)
        assert logits_off(got, ref, part) > 3 * LOGITS
        if state:
            assert state_off(wrong, S) > 3 * STATES

"""The rotary serving example: tree decoding and token-by-token decoding of the
same tokens through the operators between projections, attention, cache and
acceptance."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "serve_rotary.py")
    spec = importlib.util.spec_from_file_location("serve_rotary", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("prompt_len", [1, 16, 150])
def test_trees_and_single_tokens_agree(example, prompt_len):
    r = example.serve(prompt_len=prompt_len, rounds=4)
    m, s = r["model"], r["server"]
    # Either way rounds queries, keys and values to bf16 where fp32 sums may
    # differ, queries and keys once more after norm and rotation, the softmax
    # weights, and the attention output.  Each is at most a half step, 2^-8, of a
    # value no larger than the largest |v| (scores move weights by as much
    # again): ten of them, summed over the output matrix and the embedding
    # without any cancellation.  A penalty makes a difference at most 1.3 times
    # as large.
    v = s.cache[1].abs().max().float()
    gain = (m.a_out @ m.embed.t()).abs().sum(0).max()
    bound = example.REPETITION * 10 * 2.0 ** -8 * float(v * gain)
    assert r["logits"].shape == r["again"].shape
    assert float((r["logits"] - r["again"]).abs().max()) <= bound
    # the greedy tokens of either way, where no other token is as near as that
    top = r["again"].topk(2, dim=-1).values
    clear = (top[:, 0] - top[:, 1] > 2 * bound).tolist()
    for picked, best, sure in zip(r["picked"], r["best"], clear):
        assert picked == best or not sure
    assert all(len(e) >= 4 for e in r["emitted"])
    want = [prompt_len + len(e) for e in r["emitted"]]
    assert s.length[:s.users].tolist() == want and int(s.length[s.prompt]) == prompt_len


def test_both_ways_leave_the_same_counts(example):
    r = example.serve(prompt_len=40, rounds=5, seed=7)
    s = r["server"]
    assert torch.equal(s.counts[0], s.counts[s.replay])
    for u, tokens in enumerate(r["emitted"]):
        said = torch.bincount(torch.tensor(tokens), minlength=example.VOCAB)
        assert torch.equal((s.counts[u].int() & 32767).cpu(), said.int())
    asked = s.counts[s.prompt] < 0
    assert torch.equal(s.counts[0] < 0, asked) and 0 < int(asked.sum()) <= 40
    assert not (s.counts[s.prompt].int() & 32767).any()


def test_both_ways_leave_the_same_keys(example):
    """kv_commit of rotated tree keys, kv_append of raw ones: the same cells but
    for the two roundings of a key, at most half a step each on either side"""
    r = example.serve(prompt_len=30, rounds=4, seed=3)
    s, page = r["server"], example.PAGE
    n = int(s.length[0])
    assert int(s.length[s.replay]) == n
    cells = lambda row, c: torch.cat([s.cache[c][int(p)].transpose(0, 1) for p in s.table[
        row, : (n + page - 1) // page]])[:n].float()
    for c in (0, 1):
        a, b = cells(0, c), cells(s.replay, c)
        assert torch.equal(a[:30], b[:30])
        # a pair turns as a whole: an element moves by roundings of its head's size
        size = a.norm(dim=-1, keepdim=True)
        assert ((a - b).abs() <= 4 * 2.0 ** -8 * size).all()

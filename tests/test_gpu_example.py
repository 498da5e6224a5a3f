"""The serving example: tree decoding and token-by-token decoding of the same
tokens through all serving operators."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "serve_tree.py")
    spec = importlib.util.spec_from_file_location("serve_tree", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("prompt_len", [1, 16, 150])
def test_trees_and_single_tokens_agree(example, prompt_len):
    r = example.serve(prompt_len=prompt_len, rounds=4)
    m, s = r["model"], r["server"]
    # The two paths round differently at three places: keys, values and
    # queries (neighbouring bf16 numbers where the DeltaNet outputs differ in
    # fp32's last places), the softmax weights, and the attention output.  Each
    # is at most a half step, 2^-8, of a value no larger than the largest |v|
    # (scores move weights by as much again), on either side: 8 of them, summed
    # over the output matrix and the embedding without any cancellation.
    v = s.cache[1].abs().max().float()
    gain = (m.a_out @ m.embed.t()).abs().sum(0).max()
    bound = 8 * 2.0 ** -8 * float(v * gain)
    assert r["logits"].shape == r["again"].shape
    assert float((r["logits"] - r["again"]).abs().max()) <= bound
    assert all(len(e) >= 4 for e in r["emitted"])           # a token a round at least
    assert r["dense"] and r["kept"]
    want = int(s.length.sum())
    assert want == prompt_len + sum(prompt_len + len(e) for i, e in enumerate(r["emitted"])
                                    if i != 1)

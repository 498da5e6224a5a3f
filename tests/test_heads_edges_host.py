"""Calls of the operators between projections and attention, cache and
acceptance that their documentation allows and that are out of the ordinary.
Nothing here reaches a GPU."""
import os
import subprocess
import sys

import pytest

import gated_deltanet_tree_verify_amd as g

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Tensors inside torch.vmap look like ordinary ones and raise when they are asked
# for their address.  Whole calls leave them to Python, whose calls raise.
WITHOUT_STORAGE = """
import sys
import torch
import gated_deltanet_tree_verify_amd as g
from torch._subclasses.fake_tensor import FakeTensorMode

native = g._native()
native.streams(lambda: 0, lambda device: 0)
torch._C._cuda_getDevice = lambda: 0
torch._C._cuda_getCurrentRawStream = lambda device: 0
case = sys.argv[1]
with FakeTensorMode():
    e = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device="cuda")
    i = lambda *s: e(*s, dtype=torch.int32)
    f, w, c16, best = e(32, dtype=torch.float32), e(64), e(4, 100, dtype=torch.int16), i(2, 3)
    cache, room = e(8, 2, 16, 64), e(1 << 20, dtype=torch.uint8)
    none = [None] * 8
    calls = {
        "rope": (e(3, 5, 2, 64), lambda x: native.heads_call(
                     0, x, None, None, None, i(5), None, f, 0.0, 0.0, 0, 1.0, x, None, None),
                 lambda x: g.rope(x, None, i(5), f, q_out=x)),
        "norm": (e(3, 5, 2, 64), lambda x: native.heads_call(
                     1, x, None, w, None, i(5), None, f, 0.0, 0.0, 0, 1.0, x, None, None),
                 lambda x: g.qk_norm_rope(x, None, w, None, i(5), f, q_out=x)),
        "append": (e(3, 5, 2, 64), lambda x: native.append_call(
                       cache, cache, i(5, 4), i(5), i(5), x, x, None, f, 0, 1.0, None, 0, 0.0, 0.0,
                       None, None, None, None, None, None, None),
                   lambda x: g.kv_append(cache, cache, i(5, 4), i(5), i(5), x, x, inv_freq=f)),
        "prompt": (i(3, 9), lambda x: native.count_prompt_call(c16, i(2), i(3), x, None, None),
                   lambda x: g.count_prompt(c16, i(2), i(3), x)),
        "commit": (i(3, 2, 9),
                   lambda x: native.count_commit_call(c16, i(2), x, i(2, 4), i(2), None, None),
                   lambda x: g.count_commit(c16, i(2), x, i(2, 4), i(2))),
        "logits": (e(3, 2, 3, 100), lambda x: native.logits_call(
                       x, *none, None, None, None, best, None, None, room),
                   lambda x: g.adjust_logits(x, best=best)),
    }
    x, whole, public = calls[case]

    def run(x):
        assert whole(x) is None
        try:
            public(x)
        except RuntimeError as error:
            assert "storage" in str(error), error
            print("raised")
        return x

    torch.vmap(run)(x)
"""


@pytest.mark.parametrize("case", ["rope", "norm", "append", "prompt", "commit", "logits"])
def test_a_tensor_without_an_address_raises(case):
    """and leaves the process alive: the exception is raised while the interpreter is held"""
    pytest.importorskip("torch")
    if not os.path.exists(g.lib_path()):
        g.build()
    done = subprocess.run([sys.executable, "-c", WITHOUT_STORAGE, case], cwd=ROOT, text=True,
                          capture_output=True, timeout=300)
    assert done.returncode == 0 and done.stdout.strip() == "raised", (done.returncode, done.stdout,
                                                                      done.stderr[-2000:])

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


# ---------------------------------------------------------------------------
# What a call does not use is not looked at.  So many rows that the launch is
# refused (-2), after all arguments have been accepted: nothing runs.
# ---------------------------------------------------------------------------
FAKE = 0x10000          # an aligned address that is never dereferenced
ODD = 0x10001
ROWS = 1 << 30


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(g.lib_path()):
        g.build()
    return g.load()


def norm(lib, kind=1, Hq=4, Hk=2, wq=FAKE, wq_head=0, wk=FAKE, wk_head=0, w_dtype=1, pos=FAKE, base=None,
         base_rows=1, f=FAKE, rot=64, rows=ROWS):
    return lib.gdn_qk_norm_rope(FAKE, 384, 64, FAKE, 384, 64, 1, kind, 1e-6, 0.0, wq, wq_head, wk,
                                wk_head, w_dtype, pos, base, base_rows, f, rot, 0, 1.0, FAKE, 256, 64,
                                FAKE, 128, 64, rows, Hq, Hk, 64, None)


def append(lib, kind=1, Hq=4, wq=FAKE, wq_head=0, wk=FAKE, wk_head=0, w_dtype=1, pos=FAKE, f=FAKE,
           rot=64, rows=ROWS):
    return lib.gdn_kv_append(FAKE, FAKE, 2 * 16 * 64, FAKE, FAKE, FAKE, FAKE, FAKE, 512, 64, FAKE, 512,
                             64, FAKE, 512, 64, 1, kind, 1e-6, 0.0, wq, wq_head, wk, wk_head, w_dtype,
                             pos, f, rot, 0, 1.0, FAKE, 256, 64, None, 0, 0, 3, rows, Hq, 2, 64, 4, 4, 8,
                             16, None, None)


def test_all_in_order_but_the_rows(lib):
    assert norm(lib) == -2 and append(lib) == -2
    assert norm(lib, wq=ODD) == -1 and append(lib, wk=ODD) == -1


def test_weights_of_a_part_without_heads_are_not_looked_at(lib):
    """its pointers are ignored, and so is the type that only they would have"""
    stale = dict(w_dtype=2, wq_head=7)
    assert norm(lib, wk=None, **stale) == -1                  # queries have heads: another type
    for q in (FAKE, ODD):
        assert norm(lib, Hq=0, wq=q, wk=None, **stale) == -2
        assert append(lib, Hq=0, wq=q, wk=None, **stale) == -2
        assert norm(lib, Hk=0, wk=q, wq=None, w_dtype=2, wk_head=7) == -2


def test_positions_without_a_rotation_are_not_looked_at(lib):
    for fn in (norm, append):
        for kw in (dict(pos=ODD), dict(f=ODD)):
            assert fn(lib, **kw) == -1
            assert fn(lib, rot=0, **kw) == -2
        assert fn(lib, rot=0, pos=None, f=None) == -2
    assert norm(lib, base=ODD) == -1 and norm(lib, base=FAKE, base_rows=0) == -1
    assert norm(lib, rot=0, base=ODD) == -2 and norm(lib, rot=0, base=FAKE, base_rows=0) == -2


def test_weights_without_a_norm_are_not_looked_at(lib):
    """GDN_NORM_NONE is gdn_rope, which has none"""
    for fn in (norm, append):
        for kw in (dict(wq=ODD), dict(wk=ODD), dict(wq_head=7), dict(wk_head=7)):
            assert fn(lib, **kw) == -1
            assert fn(lib, kind=0, **kw) == -2


@pytest.mark.parametrize("rot", [2 ** 32 + 64, 2 ** 31, 2 ** 40 + 2, 258, -2 ** 32 + 64, -2, 0, 63])
def test_frequencies_of_sizes_that_no_head_has(rot):
    """refused, whatever their low 32 bits are"""
    pytest.importorskip("torch")
    with pytest.raises(g.GdnError):
        g.rope_frequencies(rot, device="cpu")

"""Refusals of the serving operators: arguments that the C entry points and
the binding turn down before any launch.  Nothing here reaches a GPU."""
import os
import subprocess
import sys

import pytest

import gated_deltanet_tree_verify_amd as g

FAKE = 0x10000          # an aligned address that is never dereferenced
ODD = 0x10004


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(g.lib_path()):
        g.build()
    return g.load()


def prefill(lib, null=None, odd=None, dtype=1, out_dtype=0, batch=1, rows=64, slots=2, H=4, Hk=2,
            dk=64, dv=64, ws=FAKE, ws_bytes=1 << 40):
    p = [FAKE] * 10      # q k v alpha beta cu S src dst out
    if null is not None:
        p[null] = None
    if odd is not None:
        p[odd] = ODD
    q, k, v, al, be, cu, S, src, dst, out = p
    return lib.gdn_prefill(q, k, v, dtype, al, be, cu, S, src, dst, out, out_dtype, batch, rows,
                           slots, H, Hk, dk, dv, ws, ws_bytes, None, None)


@pytest.mark.parametrize("i", range(10))
def test_prefill_pointers(lib, i):
    assert prefill(lib, null=i) == -1
    assert prefill(lib, odd=i) == -1


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), -1), (dict(out_dtype=2), -1), (dict(batch=0), -1), (dict(rows=-1), -1),
    (dict(slots=0), -1), (dict(H=3), -2), (dict(Hk=0), -1), (dict(dk=12), -2), (dict(dk=136), -2),
    (dict(dv=0), -1), (dict(dv=4), -2), (dict(ws=ODD), -1), (dict(rows=1 << 30, H=64), -2),
])
def test_prefill_refuses(lib, kw, code):
    assert prefill(lib, **kw) == code


def test_rule_refuses_more_threads_than_a_launch_has(lib):
    big = dict(dk=8, dv=8, H=1024, Hk=1024, slots=8)
    assert prefill(lib, batch=8192, rows=8192, **big) == -2        # 2^23 workgroups of 512
    assert prefill(lib, batch=1, rows=1 << 20, **big) == -2        # 2^24 of 256
    assert prefill(lib, batch=8191, rows=0, ws=None, **big) == -1  # these pass: the workspace lacks
    assert prefill(lib, batch=1, rows=(1 << 20) - 65, ws=None, **big) == -1
    step = lambda batch: lib.gdn_step(FAKE, FAKE, FAKE, 1, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0,
                                      batch, 8, 1024, 1024, 8, 8, None, None)
    assert step(1 << 14) == -2


def test_prefill_workspace(lib):
    need = lib.gdn_prefill_workspace(1, 3, 1000, 4, 2, 128, 128)
    assert need >= 0
    if need > 0:
        assert prefill(lib, rows=1000, batch=3, dk=128, dv=128, ws_bytes=need - 1) == -1
        assert prefill(lib, rows=1000, batch=3, dk=128, dv=128, ws=None) == -1
    assert lib.gdn_prefill_workspace(1, 0, 10, 4, 2, 128, 128) == 0
    assert lib.gdn_prefill_workspace(1, 1, 10, 4, 3, 128, 128) == 0


def test_step_refuses(lib):
    def step(q=FAKE, S=FAKE, dtype=1, batch=2, slots=2, H=4, Hk=2, dk=64, dv=64, status=None):
        return lib.gdn_step(q, FAKE, FAKE, dtype, FAKE, FAKE, S, FAKE, FAKE, FAKE, 0, batch, slots,
                            H, Hk, dk, dv, status, None)
    assert step(q=None) == -1 and step(S=ODD) == -1 and step(status=ODD) == -1
    assert step(batch=0) == -1 and step(slots=0) == -1 and step(dtype=5) == -1
    assert step(Hk=3) == -2 and step(dk=20) == -2 and step(dv=256) == -2


def attention(lib, null=None, odd=None, dtype=1, groups=0, start=None, shared=None, stride=None,
              batch=1, n=4, Hq=4, Hkv=2, d=64, page=16, num=8, width=4, ws=FAKE, ws_bytes=1 << 40,
              status=None):
    p = [FAKE] * 9       # q k v parent kc vc pages length out
    if null is not None:
        p[null] = None
    if odd is not None:
        p[odd] = ODD
    q, k, v, par, kc, vc, pages, length, out = p
    return lib.gdn_tree_attention(q, k, v, dtype, par, kc, vc,
                                  Hkv * page * d if stride is None else stride, pages, length,
                                  start, shared, groups, 0.1, out, batch, n, Hq, Hkv, d, page, num,
                                  width, ws, ws_bytes, status, None)


@pytest.mark.parametrize("i", range(9))
def test_attention_pointers(lib, i):
    assert attention(lib, null=i) == -1
    assert attention(lib, odd=i) == -1


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=0), -1), (dict(dtype=3), -1), (dict(groups=-1), -1), (dict(groups=1), -1),
    (dict(groups=1, start=FAKE), -1), (dict(groups=1, start=FAKE, shared=ODD), -1),
    (dict(batch=0), -1), (dict(n=0), -1), (dict(n=129), -2), (dict(Hq=3), -2), (dict(d=60), -2),
    (dict(d=264), -2), (dict(page=0), -1), (dict(page=24), -2), (dict(num=0), -1),
    (dict(width=0), -1), (dict(stride=8), -1), (dict(stride=2 * 16 * 64 + 4), -1),
    (dict(batch=513), -2), (dict(groups=513, start=FAKE, shared=FAKE), -2),
    (dict(width=1 << 27), -2), (dict(ws=None), -1), (dict(ws_bytes=16), -1), (dict(ws=ODD), -1),
    (dict(status=ODD), -1),
])
def test_attention_refuses(lib, kw, code):
    assert attention(lib, **kw) == code


def test_attention_workspace(lib):
    size = lib.gdn_tree_attention_workspace
    need = size(2, 4, 8, 2, 64, 16, 10, 0)
    assert need > 0 and size(2, 4, 8, 2, 64, 16, 10, 1) > need
    assert attention(lib, batch=2, Hq=8, width=10, ws_bytes=need - 1) == -1
    assert size(0, 4, 8, 2, 64, 16, 10, 0) == 0 and size(2, 4, 8, 2, 64, 24, 10, 0) == 0


def test_pages_refuse(lib):
    P = FAKE

    def table(fn, a=P, b=P, c=P, t=P, m=2, seqs=4, width=4, pool=8, page=16, status=None):
        return fn(t, P, P, a, b, c, m, seqs, width, pool, page, status, None)
    for fn in (lib.gdn_page_fork, lib.gdn_page_extend):
        assert table(fn, a=None) == -1 and table(fn, b=None) == -1 and table(fn, c=None) == -1
        assert table(fn, t=None) == -1 and table(fn, t=ODD) == -1 and table(fn, c=ODD) == -1
        assert table(fn, m=-1) == -1 and table(fn, m=4097) == -2 and table(fn, page=24) == -2
        assert table(fn, page=0) == -1 and table(fn, seqs=0) == -1 and table(fn, pool=0) == -1
        assert table(fn, width=1 << 28) == -2 and table(fn, status=ODD) == -1
        assert table(fn, m=0) == 0                     # nothing to do, nothing launched
    free = lambda t=P, done=P, m=1, page=16: lib.gdn_page_free(t, P, P, done, m, 4, 4, 8, page,
                                                               None, None)
    assert free(t=None) == -1 and free(done=None) == -1 and free(done=ODD) == -1
    assert free(page=3) == -2 and free(m=0) == 0
    pack = lambda copies=P, count=P, ws=P, pool=8: lib.gdn_page_compact(P, P, P, copies, count, ws,
                                                                        4, 4, pool, 16, None)
    assert pack(copies=None) == -1 and pack(count=None) == -1 and pack(ws=None) == -1
    assert pack(ws=ODD) == -1 and pack(pool=0) == -1
    copy = lambda cache=P, copies=P, m=1, planes=2, pool=8, size=64: lib.gdn_page_copy(
        cache, copies, None, m, planes, pool, size, None)
    assert copy(cache=None) == -1 and copy(copies=None) == -1 and copy(size=24) == -1
    assert copy(planes=0) == -1 and copy(pool=0) == -1 and copy(planes=1 << 20) == -2
    assert copy(m=0) == 0 and copy(cache=ODD) == -1

    def rows(kc=P, k=P, stride=2 * 16 * 64, m=1, n=4, max_path=4, Hkv=2, d=64, size=2, page=16):
        return lib.gdn_kv_commit(kc, P, stride, P, P, P, k, P, P, P, m, n, max_path, Hkv, d, size,
                                 4, 4, 8, page, None, None)
    assert rows(kc=None) == -1 and rows(k=ODD) == -1 and rows(size=3) == -1 and rows(n=0) == -1
    assert rows(d=60) == -2 and rows(page=24) == -2 and rows(stride=64) == -1 and rows(m=0) == 0


def test_binding_refuses_what_the_gpu_calls_cannot_take():
    torch = pytest.importorskip("torch")
    z = torch.zeros
    i = lambda *s: z(*s, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU tensor"):
        g.step(z(1, 2, 64), z(1, 2, 64), z(1, 2, 64), z(1, 2), z(1, 2), z(2, 2, 64, 64), i(1), i(1))
    with pytest.raises(ValueError, match="GPU tensor"):
        g.prefill(z(1, 2, 64), z(1, 2, 64), z(1, 2, 64), z(1, 2), z(1, 2), i(2), z(2, 2, 64, 64),
                  i(1), i(1))
    h = lambda *s: z(*s, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU tensor"):
        g.tree_attention(h(1, 1, 2, 64), h(1, 1, 1, 64), h(1, 1, 1, 64), i(1, 1), h(4, 1, 16, 64),
                         h(4, 1, 16, 64), i(1, 2), i(1), 0.1)
    with pytest.raises(TypeError):
        g.page_fork(None, i(4), i(8), i(1), i(1), 16)
    with pytest.raises(ValueError, match="GPU tensor"):
        g.page_free(i(4, 4), i(4), i(8), i(1), 16)
    with pytest.raises(ValueError, match="GPU tensor"):
        g.page_copy(h(2, 8, 64), i(1, 2))
    with pytest.raises(ValueError, match="GPU tensor"):
        g.kv_commit(h(8, 1, 16, 64), h(8, 1, 16, 64), i(4, 4), i(1), i(1), h(1, 1, 1, 64),
                    h(1, 1, 1, 64), i(1, 1), i(1))


def test_native_calls_check_their_arguments():
    pytest.importorskip("torch")
    native = g._native()
    ok = (FAKE, FAKE, FAKE, FAKE, 0, 4, 4, 8, 16, None, None)
    assert native.gdn_page_free(*ok) == 0              # no rows: nothing launched
    assert native.gdn_page_free(None, *ok[1:]) == -1
    with pytest.raises(TypeError):
        native.gdn_page_free(*ok[:-1])
    with pytest.raises(TypeError):
        native.gdn_page_free("table", *ok[1:])
    with pytest.raises(TypeError):
        native.gdn_page_free(*ok[:4], 1.5, *ok[5:])
    for big in (1 << 31, -(1 << 31) - 1, 1 << 70):
        with pytest.raises(OverflowError):
            native.gdn_page_free(*ok[:4], big, *ok[5:])


def test_native_check_says_what_is_wrong():
    torch = pytest.importorskip("torch")
    need = g._native().need
    x = torch.zeros(2, 3)
    with pytest.raises(ValueError, match="x must be a GPU tensor"):
        need(x, "x", (torch.float32,), (2, 3))
    with pytest.raises(TypeError, match="x must be a torch.Tensor"):
        need([0.0], "x", (torch.float32,))
    with pytest.raises(TypeError):
        need(x, "x")


ODD_TENSORS = r"""
import torch
import gated_deltanet_tree_verify_amd as g
from torch._subclasses.fake_tensor import FakeTensorMode
from torch.fx.experimental.symbolic_shapes import ShapeEnv

class Raises(torch.Tensor):
    @staticmethod
    def __new__(cls, shape):
        return torch.Tensor._make_wrapper_subclass(
            cls, shape, device="cuda", dtype=torch.float32, dispatch_sizes_strides_policy="strides")

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise LookupError("this tensor has no " + str(func))

native, f32 = g._native(), (torch.float32,)
mode = FakeTensorMode(shape_env=ShapeEnv(), allow_non_fake_inputs=True)
with mode:
    size = mode.shape_env.create_unbacked_symint()
    unknown = torch.empty(size, 3, device="cuda")
    unknown4 = torch.empty(size, 2, 16, 8, device="cuda")
    fake = torch.empty(2, 3, device="cuda")
    fake4 = torch.empty(6, 2, 16, 8, device="cuda")

def tells(f, *kinds):
    try:
        f()
    except kinds as e:
        print(type(e).__name__, str(e).splitlines()[0][:60])
    else:
        raise SystemExit("accepted")

native.need(fake, "x", f32, (2, 3))
assert native.cache(fake4, f32, 2, 8) == (6, 16, 256)
tells(lambda: native.need(Raises((2, 3)), "x", f32, (2, 3)), LookupError)
tells(lambda: native.need(unknown, "x", f32, (2, 3)), ValueError, RuntimeError)
tells(lambda: g._need(Raises((2, 3)), "x", f32), LookupError)
assert native.cache(Raises((6, 2, 16, 8)), f32, 2, 8) is None
assert native.cache(unknown4, f32, 2, 8) is None
tells(lambda: g._need_cache(Raises((6, 2, 16, 8)), fake4, f32, 2, 8), LookupError)
# the older entry points check theirs with the same code
tells(lambda: g.accept(unknown, fake, fake), TypeError, RuntimeError, ValueError)
print("alive")
"""


def test_tensors_whose_metadata_raises_do_not_end_the_process():
    """exceptions of a tensor's own checks come out as Python exceptions"""
    pytest.importorskip("torch")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", ODD_TENSORS], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.endswith("alive\n"), (r.returncode, r.stdout, r.stderr)


def test_cache_strides_that_say_nothing():
    """dimensions of one may have any stride; others are refused as before"""
    torch = pytest.importorskip("torch")
    from torch._subclasses.fake_tensor import FakeTensorMode
    native, bf16 = g._native(), (torch.bfloat16,)
    with FakeTensorMode():
        x = torch.empty(9, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
        y = torch.empty(9, 2, 1, 64, dtype=torch.bfloat16, device="cuda")
        z = torch.empty(1, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
        for t, strides, heads, want in (
                (x, (1024, 24, 64, 1), 1, (9, 16, 1024)), (x, (2048, 0, 64, 1), 1, (9, 16, 2048)),
                (y, (128, 64, 7, 1), 2, (9, 1, 128)), (z, (5, 1024, 64, 1), 2, (1, 16, 2048))):
            u = t.as_strided(t.shape, strides)
            assert native.cache(u, bf16, heads, 64) == want
            assert g._need_cache(u, u, bf16, heads, 64) == want
        for t, strides, heads in ((x, (1024, 1024, 65, 1), 1), (y, (128, 65, 64, 1), 2),
                                  (z, (2048, 1000, 64, 1), 2), (z, (2048, 1024, 64, 2), 2)):
            u = t.as_strided(t.shape, strides)
            assert native.cache(u, bf16, heads, 64) is None
            with pytest.raises(ValueError, match="the pages of k_cache must be contiguous"):
                g._need_cache(u, u, bf16, heads, 64)


def test_pages_refuse_more_threads_than_a_launch_has(lib):
    """before anything is launched: page_compact changes the counts in its
    first kernel, and the second is the one that would not fit"""
    P = FAKE
    free = lambda m: lib.gdn_page_free(P, P, P, P, m, 4, 4, 8, 16, None, None)
    assert free(1 << 26) == -2                              # workgroups of 64
    pack = lambda seqs: lib.gdn_page_compact(P, P, P, P, P, P, seqs, 1, 8, 16, None)
    assert pack(1 << 26) == -2
    copy = lambda m, size: lib.gdn_page_copy(P, P, None, m, 2, 8, size, None)
    assert copy(1 << 24, 16) == -2                          # workgroups of 256, 16 KiB each
    assert copy(1 << 14, 1 << 24) == -2 and copy(1 << 14, (1 << 24) - 16) == -2
    assert copy(1, 1 << 38) == -2 and copy(0x7fffffff, 0x7ffffffffffffff0) == -2
    rows = lambda m, max_path: lib.gdn_kv_commit(P, P, 2048, P, P, P, P, P, P, P, m, 4, max_path, 2,
                                                 64, 2, 4, 4, 8, 16, None, None)
    assert rows(1 << 24, 1) == -2                           # workgroups of 256, 8 tokens each
    assert rows(1 << 20, 128) == -2 and rows(1 << 20, 121) == -2
    assert rows(0x7fffffff, 0x7fffffff) == -2 and rows(1, 0x7fffffff) == -2


def test_pages_refuse_counts_past_32_bits(lib):
    """loops over tokens and pages step past their end: 2^30 and more of either
    are refused before anything is launched"""
    P, most = FAKE, (1 << 30) - 1
    for fn in (lib.gdn_page_fork, lib.gdn_page_extend):
        call = lambda m, width, pool, page: fn(P, P, P, P, P, P, m, 4, width, pool, page, None, None)
        assert call(1, 4, most + 1, 16) == -2 and call(1, 1 << 26, 8, 16) == -2
        assert call(0, 4, most, 16) == 0 and call(0, (1 << 26) - 1, 8, 16) == 0
    free = lambda m, width, pool: lib.gdn_page_free(P, P, P, P, m, 4, width, pool, 1, None, None)
    assert free(1, 1 << 30, 8) == -2 and free(1, 4, most + 1) == -2 and free(0, most, most) == 0
    pack = lambda width, pool: lib.gdn_page_compact(P, P, P, P, P, P, 4, width, pool, 1, None)
    assert pack(1 << 30, 8) == -2 and pack(4, 0x7fffffff) == -2

    def rows(width=4, Hkv=2, d=64, page=16):
        return lib.gdn_kv_commit(P, P, Hkv * page * d, P, P, P, P, P, P, P, 1, 4, 4, Hkv, d, 2, 4,
                                 width, 8, page, None, None)
    assert rows(width=1 << 26) == -2 and rows(Hkv=1 << 18) == -2 and rows(Hkv=1 << 21, d=1024) == -2


WITHOUT_NATIVE = r"""
import sys, types
import torch
import gated_deltanet_tree_verify_amd as g
name = "gated_deltanet_tree_verify_amd._binding"
kind = sys.argv[1]
if kind == "missing":
    sys.modules[name] = None
else:
    sys.modules[name] = g._binding = types.ModuleType(name)
    if kind == "older":
        g._binding.ABI_VERSION = g.ABI_VERSION - 1
    g._binding.need = g._binding.explain = None

def tells(f, kind, text):
    try:
        f()
    except kind as e:
        assert text in str(e), e
    else:
        raise SystemExit("accepted")

z = torch.zeros
i = lambda *s: z(*s, dtype=torch.int32)
for _ in range(2):
    tells(lambda: g.verify(z(1, 2, 1, 64), z(1, 2, 1, 64), z(1, 2, 1, 64), z(1, 2, 1), z(1, 2, 1),
                           i(1, 2), z(1, 1, 64, 64)), ValueError, "q must be a GPU tensor")
    tells(lambda: g.accept([0], i(1, 2), i(1, 2)), TypeError, "parent must be a torch.Tensor")
    tells(lambda: g.page_free(i(4, 4), i(4), i(8), i(1), 16), RuntimeError, "build()")
    tells(lambda: g.step(z(1, 2, 64), z(1, 2, 64), z(1, 2, 64), z(1, 2), z(1, 2), z(2, 2, 64, 64),
                         i(1), i(1)), RuntimeError, "native part")
print("done")
"""


@pytest.mark.parametrize("kind", ["missing", "older", "unversioned"])
def test_tree_calls_need_the_library_alone(lib, kind):
    """without the binding's native part, or with one of another ABI version,
    the tree calls check their arguments as ever and the serving operators raise"""
    pytest.importorskip("torch")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", WITHOUT_NATIVE, kind], cwd=root, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and r.stdout == "done\n", (r.returncode, r.stdout, r.stderr)


def test_native_part_has_the_headers_version(lib):
    pytest.importorskip("torch")
    assert g._native().ABI_VERSION == g.ABI_VERSION == lib.gdn_tree_abi_version()


def test_step_says_what_is_wrong_with_q():
    torch = pytest.importorskip("torch")
    i = torch.zeros(1, dtype=torch.int32)
    for q in (None, [0.0], 1):
        with pytest.raises(TypeError, match="q must be a torch.Tensor"):
            g.step(q, q, q, q, q, q, i, i)
    with pytest.raises(ValueError, match="q must be a GPU tensor"):
        g.step(torch.tensor(1.0), i, i, i, i, i, i, i)

"""Refusals of the operators between projections and attention, cache and
acceptance, before any launch, and the frequencies of rotary positions, which
are computed on the host.  Nothing here reaches a GPU."""
import ctypes
import math
import os

import pytest

import gated_deltanet_tree_verify_amd as g

FAKE = 0x10000          # an aligned address that is never dereferenced
ODD = 0x10001


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(g.lib_path()):
        g.build()
    return g.load()


def norm(lib, q=FAKE, k=FAKE, dtype=1, kind=1, w=FAKE, w_head=0, w_dtype=1, pos=FAKE, base=None,
         base_rows=1, f=FAKE, rot=64, layout=0, q_out=FAKE, k_out=FAKE, rows=4, Hq=4, Hk=2, d=64,
         row=384, head=64, out_row=256, out_head=64, k_row=128):
    return lib.gdn_qk_norm_rope(q, row, head, k, row, head, dtype, kind, 1e-6, 0.0, w, w_head, w,
                                w_head, w_dtype, pos, base, base_rows, f, rot, layout, 1.0, q_out,
                                out_row, out_head, k_out, k_row, out_head, rows, Hq, Hk, d, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(q=ODD), -1), (dict(k=ODD), -1), (dict(w=ODD), -1),
    (dict(dtype=3), -1), (dict(dtype=-1), -1), (dict(kind=3), -1), (dict(kind=-1), -1),
    (dict(w_dtype=2), -1), (dict(w_head=32), -1), (dict(pos=None), -1), (dict(pos=ODD), -1),
    (dict(f=None), -1), (dict(f=ODD), -1), (dict(base=FAKE, base_rows=0), -1), (dict(base=ODD), -1),
    (dict(rot=63), -1), (dict(rot=66), -1), (dict(rot=-2), -1), (dict(layout=2), -1),
    (dict(q_out=None), -1), (dict(k_out=None), -1), (dict(q_out=ODD), -1), (dict(rows=-1), -1),
    (dict(Hq=-1), -1), (dict(Hq=0, Hk=0), -1), (dict(d=0, rot=0), -1), (dict(d=257), -2),
    (dict(row=-1), -1), (dict(head=-1), -1), (dict(row=1 << 41), -1),
    (dict(out_row=255), -1), (dict(out_row=0), -1), (dict(out_head=0), -1), (dict(out_head=63), -1),
    (dict(k_row=64), -1), (dict(Hq=65536, out_row=1 << 30), -2),
    (dict(rows=1 << 30), -2),
])
def test_norm_refuses(lib, kw, code):
    assert norm(lib, **kw) == code


def test_strides_beyond_64_bits_are_weighed(lib):
    """rows times a row's stride would not fit: heads inside such rows are fine, rows
    between such heads are not"""
    far = 1 << 40
    assert norm(lib, rows=(1 << 25), out_row=far, out_head=far, k_row=far, Hk=0) == -1
    assert norm(lib, rows=(1 << 30), out_row=far, out_head=far, Hk=0) == -1
    assert norm(lib, rows=(1 << 25), out_row=64, out_head=(1 << 30), Hq=2, Hk=0) == -1


def test_nothing_to_do_is_no_error(lib):
    assert norm(lib, rows=0) == 0
    assert norm(lib, rows=0, q=None, k=None) == 0


def test_rope_refuses(lib):
    def rope(q=FAKE, k=FAKE, pos=FAKE, f=FAKE, rot=64, rows=4, Hk=2, k_out=FAKE):
        return lib.gdn_rope(q, 384, 64, k, 384, 64, 0, pos, None, 1, f, rot, 0, 1.0, FAKE, 256, 64,
                            k_out, 128, 64, rows, 4, Hk, 64, None)
    assert rope(q=None) == -1 and rope(k=None) == -1 and rope(k_out=None) == -1
    assert rope(pos=None) == -1 and rope(f=None) == -1 and rope(rot=3) == -1
    assert rope(rows=0) == 0
    # fp32 rows have to lie on four bytes
    assert rope(q=0x10002) == -1 and rope(k_out=0x10002) == -1


def append(lib, kc=FAKE, vc=FAKE, stride=2 * 16 * 64, table=FAKE, dst=FAKE, begin=FAKE, cu=FAKE,
           q=FAKE, k=FAKE, v=FAKE, dtype=1, q_out=FAKE, k_out=None, m=3, rows=9, Hq=4, Hkv=2, d=64,
           rot=64, f=FAKE, pos=None, seqs=4, width=4, pool=8, page=16, status=None, row=512,
           k_out_row=128):
    return lib.gdn_kv_append(kc, vc, stride, table, dst, begin, cu, q, row, 64, k, row, 64, v, row,
                             64, dtype, 0, 0.0, 0.0, None, 0, None, 0, 0, pos, f, rot, 0, 1.0, q_out,
                             256, 64, k_out, k_out_row, 64, m, rows, Hq, Hkv, d, seqs, width, pool,
                             page, status, None)


@pytest.mark.parametrize("kw,code", [
    (dict(kc=None), -1), (dict(vc=None), -1), (dict(kc=0x10008), -1), (dict(table=None), -1),
    (dict(dst=None), -1), (dict(begin=None), -1), (dict(table=ODD), -1), (dict(dst=ODD), -1),
    (dict(begin=ODD), -1), (dict(cu=ODD), -1), (dict(status=ODD), -1), (dict(cu=None), -1),
    (dict(k=None), -1), (dict(v=None), -1), (dict(q=None), -1), (dict(q_out=None), -1),
    (dict(v=ODD), -1), (dict(k=ODD), -1), (dict(k_out=ODD), -1), (dict(k_out=FAKE, k_out_row=1), -1),
    (dict(dtype=3), -1), (dict(m=-1), -1), (dict(rows=-1), -1), (dict(Hkv=0), -1), (dict(Hq=-1), -1),
    (dict(d=60, rot=60), -2), (dict(d=264), -2), (dict(rot=3), -1), (dict(f=None), -1),
    (dict(seqs=0), -1), (dict(width=0), -1), (dict(pool=0), -1), (dict(page=0), -1),
    (dict(page=24), -2), (dict(stride=64), -1), (dict(stride=2 * 16 * 64 + 4), -1),
    (dict(width=1 << 27), -2), (dict(pool=(1 << 30)), -2), (dict(m=4097), -2),
    (dict(rows=1 << 30), -2), (dict(row=-1), -1),
])
def test_append_refuses(lib, kw, code):
    assert append(lib, **kw) == code


def test_append_of_nobody(lib):
    assert append(lib, m=0) == 0
    assert append(lib, m=0, rows=0, cu=None, k=None, q=None, v=None) == 0


def test_counts_refuse(lib):
    def prompt(c=FAKE, stride=100, slot=FAKE, cu=FAKE, tok=FAKE, m=2, rows=5, slots=4, V=100,
               status=None):
        return lib.gdn_count_prompt(c, stride, slot, cu, tok, m, rows, slots, V, status, None)

    def commit(c=FAKE, stride=100, slot=FAKE, tok=FAKE, path=FAKE, add=FAKE, m=2, n=4, max_path=4,
               slots=4, V=100, status=None):
        return lib.gdn_count_commit(c, stride, slot, tok, path, add, m, n, max_path, slots, V,
                                    status, None)
    for fn in (prompt, commit):
        assert fn(c=None) == -1 and fn(c=ODD) == -1 and fn(slot=None) == -1 and fn(slot=ODD) == -1
        assert fn(stride=99) == -1 and fn(m=-1) == -1 and fn(slots=0) == -1 and fn(V=0) == -1
        assert fn(status=ODD) == -1 and fn(tok=None) == -1 and fn(tok=ODD) == -1
        assert fn(V=(1 << 24) + 1, stride=1 << 25) == -2 and fn(m=4097) == -2
        assert fn(stride=(1 << 40) + 1) == -2
        assert fn(m=0) == 0
    assert prompt(cu=None) == -1 and prompt(cu=ODD) == -1 and prompt(rows=-1) == -1
    assert prompt(rows=0, tok=None, m=0) == 0
    assert commit(path=None) == -1 and commit(add=None) == -1 and commit(n=0) == -1
    assert commit(max_path=0) == -1 and commit(max_path=1 << 30) == -2 and commit(add=ODD) == -1


def logits(lib, z=FAKE, dtype=1, stride=100, counts=FAKE, c_stride=100, slot=FAKE, slots=4,
           tokens=FAKE, parent=FAKE, rep=FAKE, bias_tok=FAKE, bias=FAKE, biases=3, mask=FAKE,
           mask_rows=1, out=FAKE, out_dtype=0, out_stride=100, best=FAKE, batch=2, n=3, V=100,
           ws=FAKE, size=1 << 40, status=None):
    return lib.gdn_adjust_logits(z, dtype, stride, counts, c_stride, slot, slots, tokens, parent, rep,
                                 None, None, bias_tok, bias, biases, mask, mask_rows, out, out_dtype,
                                 out_stride, best, batch, n, V, ws, size, status, None)


@pytest.mark.parametrize("kw,code", [
    (dict(z=None), -1), (dict(z=ODD), -1), (dict(out=None, best=None), -1), (dict(dtype=3), -1),
    (dict(out_dtype=2), -1), (dict(out_dtype=3), -1), (dict(out=0x10002), -1), (dict(batch=0), -1),
    (dict(n=0), -1), (dict(V=0), -1), (dict(biases=-1), -1), (dict(stride=-1), -1),
    (dict(tokens=None), -1), (dict(parent=None), -1), (dict(bias=None), -1), (dict(bias_tok=None), -1),
    (dict(slots=0), -1), (dict(c_stride=99), -1), (dict(counts=ODD), -1), (dict(slot=ODD), -1),
    (dict(mask_rows=2), -1), (dict(mask_rows=0), -1), (dict(mask=ODD), -1), (dict(out_stride=99), -1),
    (dict(best=ODD), -1), (dict(status=ODD), -1), (dict(rep=ODD), -1), (dict(ws=0x10004), -1),
    (dict(n=129, mask_rows=1), -2),
    (dict(V=(1 << 24) + 1, stride=1 << 25, c_stride=1 << 25, out_stride=1 << 25), -2),
    (dict(biases=4097), -2), (dict(batch=1 << 26), -2), (dict(stride=(1 << 40) + 1), -2),
    (dict(batch=1 << 20, n=64, V=1 << 20, stride=1 << 20, c_stride=1 << 20, out_stride=1 << 20,
          mask_rows=1, size=1 << 62), -2),
])
def test_logits_refuse(lib, kw, code):
    assert logits(lib, **kw) == code


def test_logits_workspace(lib):
    size = lib.gdn_adjust_logits_workspace
    big = dict(V=100000, stride=100000, c_stride=100000, out_stride=100000)
    need = size(2, 3, 100000)
    assert need > 0 and logits(lib, size=need - 1, **big) == -1 and logits(lib, ws=None, **big) == -1
    assert size(0, 3, 100) == 0 and size(1, 129, 100) == 0 and size(1, 1, 0) == 0


# ---------------------------------------------------------------------------
# frequencies
# ---------------------------------------------------------------------------
def frequencies(lib, rot, base, kind=0, factor=1.0, original=0.0, low=1.0, high=32.0):
    out, m = (ctypes.c_float * max(1, rot // 2))(), ctypes.c_float()
    code = lib.gdn_rope_frequencies(rot, base, kind, factor, original, low, high,
                                    ctypes.addressof(out), ctypes.addressof(m))
    return code, list(out), m.value


def single(x):
    return ctypes.c_float(x).value


@pytest.mark.parametrize("rot", [2, 6, 64, 128, 256])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_frequencies(lib, rot, base):
    """the closed forms, each rounded once; a last place of the 64-bit power may
    move a rounding, so one step of fp32 is allowed"""
    t = [base ** (-2 * i / rot) for i in range(rot // 2)]
    near = lambda got, want: all(abs(a - b) <= 2.0 ** -23 * b for a, b in zip(got, want))
    code, f, m = frequencies(lib, rot, base)
    assert code == 0 and m == 1.0 and near(f, t)
    code, f, m = frequencies(lib, rot, base, 1, 4.0)
    assert code == 0 and m == 1.0 and near(f, [x / 4 for x in t])
    if rot > 2:
        code, f, m = frequencies(lib, rot, base, 2, 8.0)
        b = base * 8 ** (rot / (rot - 2))
        assert code == 0 and m == 1.0 and near(f, [b ** (-2 * i / rot) for i in range(rot // 2)])
        # the fastest stays, the slowest is divided by the factor
        assert f[0] == 1.0 and abs(f[-1] * 8 / t[-1] - 1) < 1e-6
    want = []
    for x in t:
        n = 4096 * x / (2 * math.pi)
        share = min(max((n - 1) / 31, 0), 1)
        want.append(share * x + (1 - share) * x / 16)
    for kind, magnitude in ((3, 1.0), (4, single(0.1 * math.log(16) + 1))):
        code, f, m = frequencies(lib, rot, base, kind, 16.0, 4096.0)
        assert code == 0 and m == magnitude and near(f, want)


@pytest.mark.parametrize("args", [
    (0, 1e4), (3, 1e4), (-2, 1e4), (64, 1.0), (64, 0.0), (64, math.inf), (64, math.nan),
    (64, 1e4, 5), (64, 1e4, -1), (64, 1e4, 1, 0.5), (64, 1e4, 1, math.nan), (64, 1e4, 1, math.inf),
    (2, 1e4, 2, 4.0), (64, 1e4, 3, 4.0, 0.0), (64, 1e4, 4, 4.0, 4096.0, 32.0, 1.0),
    (64, 1e4, 4, 4.0, 4096.0, 1.0, math.inf), (64, 1e4, 3, 4.0, math.nan),
])
def test_frequencies_refuse(lib, args):
    assert frequencies(lib, *args)[0] == -1


def test_frequencies_refuse_more(lib):
    assert frequencies(lib, 258, 1e4)[0] == -2
    m = ctypes.c_float()
    assert lib.gdn_rope_frequencies(64, 1e4, 0, 1.0, 0.0, 0.0, 0.0, None, ctypes.addressof(m)) == -1


def test_binding_of_frequencies():
    torch = pytest.importorskip("torch")
    f, m = g.rope_frequencies(64, scaling="yarn", factor=4, original=2048, device="cpu")
    assert f.shape == (32,) and f.dtype == torch.float32 and abs(m - 1.1386294) < 1e-6
    with pytest.raises(ValueError, match="scaling"):
        g.rope_frequencies(64, scaling="dynamic", device="cpu")
    with pytest.raises(g.GdnError):
        g.rope_frequencies(63, device="cpu")


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------
def test_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    h = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    f = torch.zeros(32)
    for call in (
            lambda: g.rope(h(2, 4, 64), h(2, 1, 64), i(2), f),
            lambda: g.qk_norm_rope(h(2, 4, 64), None, None, None),
            lambda: g.kv_append(h(4, 1, 16, 64), h(4, 1, 16, 64), i(2, 2), i(2), i(2), h(2, 1, 64),
                                h(2, 1, 64)),
            lambda: g.count_prompt(torch.zeros(2, 9, dtype=torch.int16), i(1), i(2), i(3)),
            lambda: g.count_commit(torch.zeros(2, 9, dtype=torch.int16), i(1), i(1, 2), i(1, 2), i(1)),
            lambda: g.adjust_logits(torch.zeros(1, 1, 9))):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    for call in (lambda: g.rope(None, None, i(2), f), lambda: g.adjust_logits([0.0]),
                 lambda: g.count_prompt(3, i(1), i(2), i(3))):
        with pytest.raises(TypeError, match="must be a torch.Tensor"):
            call()


def fake(torch, shape, dtype, strides=None):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    return t if strides is None else t.as_strided(shape, strides)


def test_rows_of_strided_tensors():
    """which leading dimensions are one, and what their stride is"""
    torch = pytest.importorskip("torch")
    from torch._subclasses.fake_tensor import FakeTensorMode
    rows, bf16 = g._native().rows, (torch.bfloat16,)
    with FakeTensorMode():
        big = torch.empty(3, 5, 8, 64, dtype=torch.bfloat16, device="cuda")
        assert rows(big, bf16, 2) == (15, 512, 8, 64, 64)
        assert rows(big, bf16, 1) == (120, 64, 64)
        assert rows(big[:, :, 2:5], bf16, 2) == (15, 512, 3, 64, 64)
        assert rows(big[:, 1], bf16, 2) == (3, 2560, 8, 64, 64)
        assert rows(big[:, :4], bf16, 2) is None                     # two strides
        assert rows(big[:1, :4], bf16, 2) == (4, 512, 8, 64, 64)
        assert rows(big.transpose(1, 2), bf16, 2) is None
        assert rows(big[0].transpose(0, 1), bf16, 2) == (8, 64, 5, 512, 64)
        assert rows(big[..., ::2], bf16, 2) is None                  # d not adjacent
        assert rows(big[..., :1], bf16, 2) == (15, 512, 8, 64, 1)
        assert rows(big[0, 0], bf16, 2) == (1, 512, 8, 64, 64)
        assert rows(big[0, 0, :1], bf16, 2) == (1, 64, 1, 64, 64)
        assert rows(big[0, 0, 0], bf16, 2) is None
        assert rows(big.expand(2, 3, 5, 8, 64), bf16, 2) is None
        assert rows(big[:1, :1].expand(3, 5, 8, 64), bf16, 2) == (15, 0, 8, 64, 64)
        assert rows(big, (torch.float32,), 2) is None
        assert rows(torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda"), bf16,
                    2) == (0, 256, 4, 64, 64)
        for lead in ((2, 0), (0, 2), (3, 0, 2)):
            none = torch.empty(*lead, 4, 64, dtype=torch.bfloat16, device="cuda")
            assert rows(none, bf16, 2)[0] == 0
        assert g._native().on_device(0, big, None, 3) and not g._native().on_device(1, big)
    assert rows(torch.empty(3, 4, 64, dtype=torch.bfloat16), bf16, 2) is None
    with pytest.raises(TypeError):
        rows(None, bf16)


def test_binding_says_what_is_wrong(monkeypatch):
    torch = pytest.importorskip("torch")
    from torch._subclasses.fake_tensor import FakeTensorMode
    g._native()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    b16, i32, f32 = torch.bfloat16, torch.int32, torch.float32

    def refuses(kind, text, call):
        with pytest.raises(kind, match=text):
            call()

    with FakeTensorMode():
        e = lambda *s, dtype=b16: torch.empty(*s, dtype=dtype, device="cuda")
        q, k, pos, f = e(2, 3, 4, 64), e(2, 3, 2, 64), e(2, 3, dtype=i32), e(32, dtype=f32)
        refuses(TypeError, "dtype", lambda: g.rope(q.long(), k, pos, f))
        refuses(TypeError, "k has dtype", lambda: g.rope(q, k.float(), pos, f))
        refuses(ValueError, "leading dimensions and d", lambda: g.rope(q, k[:1], pos, f))
        refuses(ValueError, "leading dimensions and d", lambda: g.rope(q, k[..., :32], pos, f))
        refuses(ValueError, "pos has shape", lambda: g.rope(q, k, pos[:1], f))
        refuses(TypeError, "pos has dtype", lambda: g.rope(q, k, pos.long(), f))
        refuses(ValueError, "base has shape", lambda: g.rope(q, k, pos, f, base=e(3, dtype=i32)))
        refuses(ValueError, "inv_freq must be", lambda: g.rope(q, k, pos, e(33, dtype=f32)))
        refuses(ValueError, "q_out has shape", lambda: g.rope(q, k, pos, f, q_out=k))
        refuses(TypeError, "k_out has dtype", lambda: g.rope(q, k, pos, f, k_out=k.float()))
        refuses(ValueError, "k_out without k", lambda: g.rope(q, None, pos, f, k_out=k))
        refuses(ValueError, "layout must be", lambda: g.rope(q, k, pos, f, layout="pairs"))
        refuses(ValueError, "last dimension", lambda: g.rope(q[..., ::2], k[..., ::2], pos, f))
        refuses(ValueError, "single stride", lambda: g.rope(e(3, 2, 4, 64).transpose(0, 1), k, pos, f))
        refuses(ValueError, "norm must be", lambda: g.qk_norm_rope(q, k, None, None, norm="layer"))
        refuses(ValueError, "weights belong", lambda: g.qk_norm_rope(q, k, e(64), None, norm=None))
        refuses(ValueError, "q_weight has shape", lambda: g.qk_norm_rope(q, k, e(32), None))
        refuses(ValueError, "k_weight has shape", lambda: g.qk_norm_rope(q, k, None, e(4, 64)))
        refuses(TypeError, "share a dtype",
                lambda: g.qk_norm_rope(q, k, e(64), e(64, dtype=f32)))
        refuses(ValueError, "without inv_freq", lambda: g.qk_norm_rope(q, k, None, None, pos=pos))
        c = e(8, 2, 16, 64)
        table, two = e(4, 4, dtype=i32), e(2, dtype=i32)
        six = e(6, dtype=i32)
        put = lambda k_=k, v_=k, dst=six, begin=six, **kw: g.kv_append(c, c, table, dst, begin, k_,
                                                                      v_, **kw)
        refuses(ValueError, "v must have", lambda: put(v_=k[:1]))
        refuses(ValueError, "dst has shape", lambda: put(dst=two))
        refuses(ValueError, "dst has shape", lambda: put(cu=two))
        refuses(ValueError, "begin has shape", lambda: put(begin=two))
        refuses(ValueError, "cu must be", lambda: put(cu=e(0, dtype=i32)))
        refuses(ValueError, r"k_cache must be \[pages\]", lambda: put(e(6, 4, 64), e(6, 4, 64)))
        refuses(ValueError, "without q", lambda: put(q_out=q))
        refuses(ValueError, "without q", lambda: put(q_weight=e(64)))
        refuses(ValueError, "q must be", lambda: put(q=q[:1]))
        refuses(ValueError, "without inv_freq", lambda: put(pos=pos))
        refuses(ValueError, "weights belong", lambda: put(k_weight=e(64)))
        z = e(2, 3, 100)
        adjust = lambda **kw: g.adjust_logits(z, **kw)
        refuses(ValueError, "logits must be", lambda: g.adjust_logits(z[0]))
        refuses(ValueError, "counts must be", lambda: adjust(counts=e(4, 99, dtype=torch.int16)))
        refuses(ValueError, "slot without", lambda: adjust(slot=two))
        refuses(ValueError, "belong together", lambda: adjust(tokens=e(2, 3, dtype=i32)))
        refuses(ValueError, "repetition has shape", lambda: adjust(repetition=e(3, dtype=f32)))
        refuses(ValueError, "bias tokens must be", lambda: adjust(bias=(e(3, 4, dtype=i32), f)))
        refuses(ValueError, "bias values has shape", lambda: adjust(bias=(e(2, 4, dtype=i32), f)))
        refuses(ValueError, "mask must be", lambda: adjust(mask=e(2, 2, 4, dtype=i32)))
        refuses(ValueError, "mask must be", lambda: adjust(mask=e(2, 4, dtype=i32)))
        refuses(ValueError, "out must be", lambda: adjust(out=z[:1]))
        refuses(TypeError, "out has dtype", lambda: adjust(out=z.half()))
        refuses(ValueError, "best has shape", lambda: adjust(best=e(3, 2, dtype=i32)))
        n16 = e(4, 100, dtype=torch.int16)
        refuses(ValueError, "cu has shape", lambda: g.count_prompt(n16, two, two, six))
        refuses(ValueError, "tokens must be", lambda: g.count_commit(n16, two, six, table, two))
        refuses(ValueError, "path must be",
                lambda: g.count_commit(n16, two, e(2, 3, dtype=i32), table, two))
        refuses(TypeError, "counts has dtype", lambda: g.count_prompt(table, two, six[:3], six))


def test_calls_stay_on_the_current_device(monkeypatch):
    """tensors of another GPU are refused before anything is launched"""
    torch = pytest.importorskip("torch")
    from torch._subclasses.fake_tensor import FakeTensorMode
    g._native()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    with FakeTensorMode():
        z = torch.empty(1, 1, 9, device="cuda:0")
        with pytest.raises(ValueError, match="current device, cuda:1"):
            g.adjust_logits(z)

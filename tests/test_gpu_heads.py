"""Rotary positions, norms of queries and keys, and both on the way into the
paged cache, against plain 64-bit implementations.

Tolerances.  A result is rounded once, by at most half a step h = eps / 2 of its
type (below the smallest normal number, half of that type's smallest step).
Before that fp32: an angle is off by 2^-24 of half a turn, cos and sin by two
steps more, the two products and their sum by one each, which is less than
8 * 2^-23 of |x| + |y| of the pair; a norm by at most 8 roundings of its sum
(four squares a lane, six steps across lanes or fewer, the mean, eps), halved by
the root, which is one more of two steps, and the two products: less than
16 * 2^-24.  F = 32 * 2^-24 of |x| + |y| (of |x| alone past the rotated
elements) bounds both together.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
F = 32 * 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
NAN = float("nan")


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def frequencies(rot):
    return (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float()


def heads_ref(x, pos, inv_freq, layout, scale=1.0, norm=None, eps=0.0, weight=None, offset=0.0):
    """(result, the magnitude that its error is relative to) in 64 bits; x
    [rows][heads][d], pos [rows] python integers"""
    y = x.double()
    d = y.shape[-1]
    if norm:
        s = y.square().sum(-1, keepdim=True)
        y = y / torch.sqrt((s / d if norm == "rms" else s) + eps)
        if weight is not None:
            y = y * (offset + weight.double())
    rot = 0 if inv_freq is None else 2 * len(inv_freq)
    out, mag = y.clone(), y.abs()
    if rot:
        # the angle of position p: p f mod 2 pi, from an integer and a dyadic
        # number without any rounding before the reduction
        angle = np.array([[math.fmod(int(p) * float(f), 2 * math.pi) if abs(int(p)) < 1 << 28 else
                           _far(int(p), float(f)) for f in inv_freq.tolist()] for p in pos])
        angle = torch.from_numpy(angle).reshape(len(pos), rot // 2)[:, None]
        i = torch.arange(rot // 2)
        a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
        c, s = torch.cos(angle) * scale, torch.sin(angle) * scale
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
        mag[..., a] = mag[..., b] = abs(scale) * (y[..., a].abs() + y[..., b].abs())
    return out, mag


def _far(p, f):
    """p f mod 2 pi for large p: the product is an exact fraction"""
    from fractions import Fraction
    turns = Fraction(p) * Fraction(f) / Fraction(math.pi)      # pi to 2^-53: its error is
    return float(turns % 2) * math.pi + _pi_rest(p, f)         # put right to first order


def _pi_rest(p, f):
    # pi = math.pi + 1.2246467991473532e-16: p f / pi changes by -p f rest / pi^2
    return -p * f / math.pi * 1.2246467991473532e-16


def close(got, ref_mag, what=""):
    ref, mag = ref_mag
    t, got = got.dtype, got.double().cpu()
    assert got.shape == ref.shape, what
    h = torch.finfo(t).eps / 2
    tol = h * ref.abs() + F * (1 + h) * mag + torch.finfo(t).smallest_normal * h
    off = (got - ref).abs()
    assert torch.isfinite(got).all(), what
    assert (off <= tol).all(), (what, (off / tol).max().item())


def projection(lead, Hq, Hk, d, dtype, seed, fused):
    """q, k, v of these leading dimensions, views of one tensor where fused"""
    rows = math.prod(lead)
    x = (torch.randn(rows, Hq + 2 * Hk, d, generator=gen(seed)) * 1.5).to(DT[dtype])
    parts = x.split((Hq, Hk, Hk), 1)
    if fused:
        dev = x.cuda().split((Hq, Hk, Hk), 1)
    else:
        dev = [p.contiguous().cuda() for p in parts]
    return parts, [p.unflatten(0, lead) for p in dev]


ROPE = [
    # lead, Hq, Hk, d, rot, layout, dtype, fused, positions
    ((1,), 1, 1, 2, 2, "half", "fp32", False, [7]),
    ((3,), 2, 1, 8, 4, "interleaved", "bf16", False, [0, 1, -1]),
    ((2, 3), 4, 2, 64, 64, "half", "bf16", True, range(6)),
    ((5,), 32, 8, 128, 128, "half", "bf16", True, [0, 1, 63, 4095, 131071]),
    ((7,), 8, 2, 128, 128, "interleaved", "fp16", True, range(100000, 100007)),
    ((4,), 3, 3, 128, 32, "half", "fp32", False, [5, 2 ** 20, -2 ** 20, 0]),
    ((4,), 16, 2, 256, 64, "half", "bf16", True, [2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 3]),
    ((3,), 5, 1, 256, 256, "interleaved", "fp32", True, [1, 10 ** 6, 10 ** 9]),
    ((9,), 5, 2, 80, 20, "half", "bf16", True, range(9)),
    ((9,), 5, 2, 90, 90, "half", "fp16", True, range(50, 59)),
    ((9,), 2, 1, 7, 6, "interleaved", "fp32", True, range(9)),
    ((2,), 3, 2, 1, 0, "half", "bf16", False, [4, 5]),
    ((2,), 3, 2, 72, 0, "half", "bf16", False, [4, 5]),
    ((6,), 3, 2, 72, 48, "half", "fp16", True, range(6)),
    ((6,), 3, 2, 248, 240, "half", "bf16", True, range(6)),
    ((6,), 3, 2, 40, 24, "interleaved", "bf16", True, range(6)),
    ((6,), 11, 2, 96, 96, "half", "fp32", True, range(6)),
    ((700,), 6, 2, 64, 32, "half", "bf16", True, range(3, 703)),
    # pieces that turn in part
    ((5,), 9, 2, 80, 20, "half", "bf16", True, range(7, 12)),
    ((5,), 9, 2, 96, 24, "half", "fp32", True, range(7, 12)),
    ((5,), 3, 2, 256, 250, "half", "fp16", True, range(7, 12)),
    ((5,), 3, 2, 256, 254, "interleaved", "bf16", True, range(7, 12)),
    ((5,), 17, 3, 8, 6, "half", "bf16", False, range(7, 12)),
    ((5,), 17, 3, 8, 2, "interleaved", "bf16", False, range(7, 12)),
    ((600,), 5, 1, 72, 72, "half", "bf16", True, range(7, 607)),
    ((600,), 5, 1, 104, 50, "interleaved", "fp32", True, range(7, 607)),
]


@pytest.mark.parametrize("lead,Hq,Hk,d,rot,layout,dtype,fused,at", ROPE)
def test_rope(gpu_lib, lead, Hq, Hk, d, rot, layout, dtype, fused, at):
    print("rope", lead, Hq, Hk, d, rot, layout, dtype, fused, flush=True)
    (q, k, _), (dq, dk, _) = projection(lead, Hq, Hk, d, dtype, 3, fused)
    f = frequencies(rot)
    pos = ints(list(at)).reshape(lead)
    a, b = gpu_lib.rope(dq, dk, pos, f.cuda(), layout=layout, scale=1.25)
    torch.cuda.synchronize()
    assert a.shape == dq.shape and b.shape == dk.shape and a.is_contiguous()
    close(a.flatten(0, -3), heads_ref(q, at, f, layout, 1.25), "q")
    close(b.flatten(0, -3), heads_ref(k, at, f, layout, 1.25), "k")
    if rot == 0:
        assert torch.equal(a.cpu().flatten(0, -3), q)


NORM = [
    # lead, Hq, Hk, d, rot, layout, dtype, fused, norm, weight, offset, eps
    ((1,), 32, 8, 128, 128, "half", "bf16", True, "rms", "same", 0.0, 1e-6),
    ((2, 4), 4, 2, 128, 128, "half", "bf16", True, "rms", "heads", 0.0, 1e-6),
    ((9,), 16, 2, 256, 64, "half", "bf16", True, "rms", "wide", 1.0, 1e-6),
    ((5,), 4, 4, 64, 64, "interleaved", "fp16", True, "rms", "same", 1.0, 1e-5),
    ((33,), 4, 2, 128, 0, "half", "bf16", False, "l2", None, 0.0, 1e-6),
    ((33,), 4, 2, 64, 0, "half", "fp32", True, "l2", "wide heads", 0.5, 1e-6),
    ((13,), 8, 4, 90, 22, "half", "fp32", False, "l2", "same", 0.0, 1e-6),
    ((13,), 3, 1, 80, 40, "interleaved", "bf16", True, "rms", "heads", 0.0, 0.5),
    ((3,), 1, 1, 1, 0, "half", "fp32", False, "rms", None, 0.0, 1e-6),
    ((6,), 3, 5, 24, 16, "half", "fp16", True, "rms", "wide", 0.0, 1e-6),
    ((6,), 3, 5, 16, 16, "half", "bf16", True, "l2", "same", 0.0, 1e-6),
    ((600,), 7, 2, 128, 96, "half", "bf16", True, "rms", "same", 0.0, 1e-6),
    ((600,), 7, 2, 80, 20, "half", "bf16", True, "rms", "heads", 0.0, 1e-6),
    ((9,), 7, 2, 96, 36, "half", "fp16", True, "l2", "wide", 1.0, 1e-6),
    ((9,), 7, 2, 88, 44, "interleaved", "bf16", True, "rms", "same", 0.0, 1e-6),
]


@pytest.mark.parametrize("lead,Hq,Hk,d,rot,layout,dtype,fused,norm,weight,offset,eps", NORM)
def test_qk_norm_rope(gpu_lib, lead, Hq, Hk, d, rot, layout, dtype, fused, norm, weight, offset,
                      eps):
    print("norm", lead, Hq, Hk, d, rot, layout, dtype, norm, weight, flush=True)
    (q, k, _), (dq, dk, _) = projection(lead, Hq, Hk, d, dtype, 5, fused)
    rows = math.prod(lead)
    at = [1000 + 3 * i for i in range(rows)]
    w = []
    for H in (Hq, Hk):
        shape = (H, d) if weight and "heads" in weight else (d,)
        x = torch.randn(shape, generator=gen(7 + H)) * 0.3 + 1
        w.append(None if weight is None else x.to(DT["fp32" if "wide" in weight else dtype]))
    f = frequencies(rot) if rot else None
    kw = dict(pos=ints(at).reshape(lead), inv_freq=f.cuda(), layout=layout) if rot else {}
    a, b = gpu_lib.qk_norm_rope(dq, dk, *(x if x is None else x.cuda() for x in w), norm=norm,
                                eps=eps, offset=offset, **kw)
    torch.cuda.synchronize()
    for got, x, y in ((a, q, w[0]), (b, k, w[1])):
        close(got.flatten(0, -3), heads_ref(x, at, f, layout, 1.0, norm, eps, y, offset))


def test_base_counts_positions_from_lengths(gpu_lib):
    (q, k, _), (dq, dk, _) = projection((3, 5), 4, 2, 128, "bf16", 11, True)
    depth = [[0, 1, 1, 2, 3], [0, 1, 2, 3, 4], [0, 0, 1, 1, 2]]
    base = [100, 0, -7]
    f = frequencies(128)
    a, b = gpu_lib.rope(dq, dk, ints(depth), f.cuda(), base=ints(base))
    at = [x + y for row, y in zip(depth, base) for x in row]
    close(a.flatten(0, 1), heads_ref(q, at, f, "half"))
    close(b.flatten(0, 1), heads_ref(k, at, f, "half"))
    # past 32 bits: the sum is not cut
    a, _ = gpu_lib.rope(dq, dk, ints([[2 ** 31 - 1] * 5] * 3), f.cuda(), base=ints([2 ** 31 - 1] * 3))
    close(a.flatten(0, 1), heads_ref(q, [2 ** 32 - 2] * 15, f, "half"))


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (90, "fp32"), (64, "fp16")])
def test_in_place_and_strided_outputs(gpu_lib, d, dtype):
    (q, k, v), (dq, dk, dv) = projection((37,), 6, 2, d, dtype, 13, True)
    f = frequencies(d).cuda()
    pos = ints(list(range(37)))
    want = gpu_lib.rope(dq, dk, pos, f)
    # heads before rows: [heads][rows][d]
    turned = torch.full((6, 37, d), NAN, dtype=DT[dtype], device="cuda").transpose(0, 1)
    a, b = gpu_lib.rope(dq, dk, pos, f, q_out=turned, k_out=dk)
    assert a is turned and b is dk
    gpu_lib.rope(dq, None, pos, f, q_out=dq)
    torch.cuda.synchronize()
    for got in (a, dq):
        assert torch.equal(got, want[0])
    assert torch.equal(dk, want[1]) and torch.equal(dv.cpu(), v)
    # and the input [heads][rows][d], each rounded on its own
    x = q.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    assert torch.equal(gpu_lib.rope(x, None, pos, f)[0], want[0])
    # the same heads for every row: a stride of zero
    same = dv[:1].expand(37, 2, d)
    got = gpu_lib.rope(same, None, pos, f)[0]
    close(got, heads_ref(v[:1].expand(37, 2, d), range(37), f.cpu(), "half"))


def test_turning_back(gpu_lib):
    """-p undoes p, up to the roundings of two results of the pair's size"""
    (q, _, _), (dq, _, _) = projection((50,), 4, 1, 128, "fp32", 17, False)
    f = frequencies(128).cuda()
    pos = ints([i * 977 for i in range(50)])
    there = gpu_lib.rope(dq, None, pos, f)[0]
    back = gpu_lib.rope(there, None, -pos, f)[0].cpu()
    pair = q.double().abs().reshape(50, 4, 2, 64).sum(-2).repeat(1, 1, 2)
    assert ((back.double() - q.double()).abs() <= 4 * F * pair).all()


@pytest.mark.parametrize("layout,rot", [("half", 20), ("interleaved", 20), ("half", 64),
                                        ("interleaved", 48)])
def test_values_not_finite_do_not_reach_what_is_copied(gpu_lib, layout, rot):
    """also where a piece turns in part"""
    q = torch.randn(3, 4, 80, generator=gen(37)).bfloat16()
    q[1, 2, rot:] = float("inf")
    q[2, 1, rot + 1] = NAN
    got = gpu_lib.rope(q.cuda(), None, ints([5, 6, 7]), frequencies(rot).cuda(), layout=layout)[0]
    got = got.cpu()
    assert torch.isfinite(got[..., :rot]).all()
    assert torch.equal(got[..., rot:].view(torch.int16), q[..., rot:].view(torch.int16))
    q[1, 2, 0] = float("inf")
    got = gpu_lib.rope(q.cuda(), None, ints([5, 6, 7]), frequencies(rot).cuda(), layout=layout)[0]
    mate = rot // 2 if layout == "half" else 1
    bad = ~torch.isfinite(got[1, 2, :rot].cpu())
    assert bad.tolist() == [i in (0, mate) for i in range(rot)]


def test_values_not_finite_stay_in_their_heads(gpu_lib):
    (q, k, _), (dq, dk, _) = projection((8,), 8, 2, 128, "bf16", 19, True)
    f = frequencies(64).cuda()
    pos = ints(list(range(8)))
    w = torch.ones(128, device="cuda")
    want = gpu_lib.qk_norm_rope(dq, dk, w, w, pos, f)
    dq[3, 5, 70], dk[2, 1, 0] = float("inf"), NAN
    got = gpu_lib.qk_norm_rope(dq, dk, w, w, pos, f)
    hit = [torch.zeros(8, 8, dtype=torch.bool), torch.zeros(8, 2, dtype=torch.bool)]
    hit[0][3, 5] = hit[1][2, 1] = True
    for g_, w_, h_ in zip(got, want, hit):
        assert torch.equal(g_[~h_], w_[~h_])
    assert torch.isnan(got[1][2, 1]).all()
    # without a norm they reach their own pair alone
    got = gpu_lib.rope(dq, dk, pos, f)[0][3, 5].cpu()
    assert not torch.isfinite(got[70]) and torch.isfinite(got[:64]).all()
    # zeros have no direction: eps keeps them zero
    z = torch.zeros(2, 3, 128, dtype=torch.bfloat16, device="cuda")
    assert not gpu_lib.qk_norm_rope(z, None, w, None, ints([1, 2]), f)[0].any()


def test_no_rows(gpu_lib):
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    a, b = gpu_lib.rope(q, q, ints([]), frequencies(64).cuda())
    assert a.shape == q.shape and b.shape == q.shape
    for lead in ((2, 0), (0, 2)):
        q, f = torch.empty(*lead, 4, 64, dtype=torch.float16, device="cuda"), frequencies(64).cuda()
        pos, base = torch.empty(lead, dtype=torch.int32, device="cuda"), ints([3] * lead[0])
        for given in (None, q):
            a, b = gpu_lib.qk_norm_rope(q, q, None, None, pos, f, base=base, q_out=given, k_out=given)
            assert a.shape == q.shape and b.shape == q.shape


# ---------------------------------------------------------------------------
# rope_frequencies
# ---------------------------------------------------------------------------
def test_frequencies_on_the_gpu(gpu_lib):
    f, m = gpu_lib.rope_frequencies(64, 10000.0)
    assert f.is_cuda and m == 1.0
    assert torch.equal(f.cpu(), frequencies(64))


# ---------------------------------------------------------------------------
# kv_append
# ---------------------------------------------------------------------------
def cache_of(num, Hkv, page, d, dtype, seed, pad=0):
    """[2][num][Hkv][page][d]; pad: elements between pages that nothing may touch"""
    x = torch.randn(2, num, Hkv * page * d + pad, generator=gen(seed)).to(DT[dtype])
    return x


def view(x, Hkv, page, d):
    return x[..., : Hkv * page * d].unflatten(-1, (Hkv, page, d))


def place(lens, begin, page, seed, extra=3):
    """table, rows of the requests, and the number of pages"""
    rng = np.random.default_rng(seed)
    m = len(lens)
    pages = [-(-(b + n) // page) if b >= 0 else 1 for b, n in zip(begin, lens)]
    order = [int(x) for x in rng.permutation(sum(pages) + extra)]
    dst = [int(x) for x in rng.permutation(m + 2)[:m]]
    width = max(pages + [1]) + 1
    table = np.full((m + 2, width), -1, dtype=np.int32)
    for r, p in zip(dst, pages):
        for c in range(p):
            table[r, c] = order.pop()
    return table, dst, len(order) + sum(pages)


APPEND = [
    # lens, begin, Hq, Hkv, d, rot, page, dtype, layout, norm, cu, k_out, pad
    ([1], [0], 4, 1, 64, 64, 16, "bf16", "half", "rms", False, True, 0),
    ([1], [1000], 32, 8, 128, 128, 16, "bf16", "half", "rms", False, True, 0),
    ([1] * 70, [3 * i for i in range(70)], 4, 2, 64, 32, 16, "fp16", "half", None, False, False, 24),
    ([3, 0, 70, 1, 0], [0, 5, 30, 15, 0], 4, 2, 128, 128, 16, "bf16", "half", "rms", True, True, 0),
    ([0, 0, 17], [1, 2, 3], 0, 3, 72, 24, 8, "fp32", "interleaved", "l2", True, True, 8),
    ([65, 64, 63], [64, 63, 65], 2, 2, 256, 64, 64, "bf16", "interleaved", None, True, False, 0),
    ([300], [0], 3, 1, 8, 8, 4, "bf16", "half", "l2", True, False, 0),
    ([5, 6], [7, 0], 2, 1, 16, 0, 1, "fp16", "half", None, True, True, 0),
    ([2, 9] * 100, [1, 31] * 100, 2, 2, 64, 64, 32, "bf16", "half", "rms", True, True, 16),
    ([2, 9, 31], [1, 31, 0], 5, 2, 80, 20, 16, "bf16", "half", "rms", True, True, 0),
    ([2, 9, 31], [1, 31, 0], 5, 2, 88, 22, 16, "fp32", "interleaved", None, True, True, 0),
]


def append_case(lens, begin, Hq, Hkv, d, rot, page, dtype, layout, norm, pad, before=0, after=0,
                seed=23, fused=True):
    rows = before + sum(lens) + after
    (q, k, v), dev = projection((rows,), Hq, Hkv, d, dtype, seed, fused)
    table, dst, num = place(lens, begin, page, seed)
    raw = cache_of(num, Hkv, page, d, dtype, seed + 1, pad)
    w = torch.randn(2, d, generator=gen(seed + 2)) * 0.2 + 1
    f = frequencies(rot) if rot else None
    cu = [before + sum(lens[:i]) for i in range(len(lens) + 1)]
    return dict(q=q, k=k, v=v, dev=dev, table=table, dst=dst, num=num, raw=raw, w=w, f=f, cu=cu,
                lens=lens, begin=begin, Hq=Hq, Hkv=Hkv, d=d, page=page, layout=layout, norm=norm)


def append_ref(x, served=None, pos=None):
    """cache, q and k in 64 bits with their magnitudes, row by row"""
    c, page = view(x["raw"], x["Hkv"], x["page"], x["d"]).double(), x["page"]
    cache, mag = c.clone(), torch.zeros_like(c)
    qk = [x["q"].double().clone(), x["k"].double().clone()]
    qm = [torch.zeros_like(qk[0]), torch.zeros_like(qk[1])]
    for r, (n, b) in enumerate(zip(x["lens"], x["begin"])):
        rows = slice(x["cu"][r], x["cu"][r] + n)
        if n == 0:
            continue
        if served is not None and not served[r]:
            qk[0][rows] = qk[1][rows] = NAN
            continue
        at = range(b, b + n) if pos is None else pos[rows]
        for j, name in enumerate(("q", "k")):
            if x[name].shape[1]:
                qk[j][rows], qm[j][rows] = heads_ref(
                    x[name][rows], at, x["f"], x["layout"], 1.0, x["norm"], 1e-6,
                    x["w"][j] if x["norm"] else None, 0.0)
        for t in range(n):
            p = x["table"][x["dst"][r], (b + t) // page]
            off = (b + t) % page
            cache[0, p, :, off], mag[0, p, :, off] = qk[1][rows][t], qm[1][rows][t]
            cache[1, p, :, off] = x["v"][rows][t].double()
    return cache, mag, qk, qm


def run_append(lib, x, cu=True, k_out=True, status=None, pos=None, stream=None, raw=None, **kw):
    raw = x["raw"].cuda() if raw is None else raw
    c = view(raw, x["Hkv"], x["page"], x["d"])
    q, k, v = x["dev"]
    w = [y.cuda() if x["norm"] else None for y in x["w"]]
    args = dict(cu=ints(x["cu"]) if cu else None,
                inv_freq=None if x["f"] is None else x["f"].cuda(), layout=x["layout"],
                norm=x["norm"], k_weight=w[1], status=status, stream=stream,
                pos=None if pos is None else ints(pos))
    if x["Hq"]:
        args.update(q=q, q_weight=w[0])
    if k_out is True:
        args["k_out"] = torch.zeros(k.shape, dtype=k.dtype, device="cuda")
    elif k_out is not False:
        args["k_out"] = k_out
    args.update(kw)
    got = lib.kv_append(c[0], c[1], ints(x["table"].tolist()), ints(x["dst"]), ints(x["begin"]), k,
                        v, **args)
    return raw, got


def check_append(x, raw, got, ref, rows=None):
    cache, mag, qk, qm = ref
    n = x["Hkv"] * x["page"] * x["d"]
    after = raw.cpu()
    assert torch.equal(after[..., n:], x["raw"][..., n:])             # between the pages
    c = view(after, x["Hkv"], x["page"], x["d"])
    close(c[0], (cache[0], mag[0]), "keys")
    assert torch.equal(c[1].double(), cache[1])
    for g_, y, m in zip(got, qk, qm):
        if g_ is None or not g_.shape[1]:
            continue
        g_, y, m = (g_.cpu(), y, m) if rows is None else (g_.cpu()[rows], y[rows], m[rows])
        fine = torch.isfinite(y)
        assert torch.equal(torch.isnan(g_), torch.isnan(y))
        close(g_[fine], (y[fine], m[fine]))


@pytest.mark.parametrize("lens,begin,Hq,Hkv,d,rot,page,dtype,layout,norm,cu,k_out,pad", APPEND)
def test_kv_append(gpu_lib, lens, begin, Hq, Hkv, d, rot, page, dtype, layout, norm, cu, k_out, pad):
    print("append", lens[:6], begin[:6], Hq, Hkv, d, rot, page, dtype, layout, norm, flush=True)
    x = append_case(lens, begin, Hq, Hkv, d, rot, page, dtype, layout, norm, pad)
    st = ints([-1] * len(lens))
    raw, got = run_append(gpu_lib, x, cu, k_out, st)
    torch.cuda.synchronize()
    assert st.tolist() == [0] * len(lens)
    assert (got[0] is None) == (Hq == 0) and (got[1] is None) == (not k_out)
    check_append(x, raw, got, append_ref(x))


@pytest.mark.parametrize("d,fused", [(8, True), (24, False)])
def test_kv_append_many_requests(gpu_lib, d, fused):
    """a thousand requests, several rows a wave, some requests not served"""
    rng = np.random.default_rng(9)
    lens = [int(n) for n in rng.integers(0, 17, 1100)]
    begin = [int(b) if b % 7 else -1 for b in rng.integers(0, 40, 1100)]
    x = append_case(lens, begin, 1, 1, d, 8, 16, "bf16", "half", "rms", 0, 3, 2, fused=fused)
    assert sum(lens) > 2 * 4096
    st = ints([-1] * len(lens))
    q_out = torch.full((sum(lens) + 5, 1, d), 7.0, dtype=torch.bfloat16, device="cuda")
    k_out = torch.full_like(q_out, 7.0)
    raw, got = run_append(gpu_lib, x, status=st, q_out=q_out, k_out=k_out)
    torch.cuda.synchronize()
    assert st.tolist() == [0] * len(lens)
    check_append(x, raw, got, append_ref(x, [b >= 0 for b in begin]), slice(3, 3 + sum(lens)))
    for y in got:
        assert (y[:3] == 7).all() and (y[-2:] == 7).all()


def test_kv_append_leaves_rows_of_nobody(gpu_lib):
    x = append_case([4, 0, 9], [3, 0, 20], 4, 2, 64, 64, 16, "bf16", "half", "rms", 0, 5, 6)
    q, k, _ = x["dev"]
    q_out, k_out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda"), torch.full(
        k.shape, 7.0, dtype=k.dtype, device="cuda")
    raw, got = run_append(gpu_lib, x, q_out=q_out, k_out=k_out)
    torch.cuda.synchronize()
    check_append(x, raw, got, append_ref(x), slice(5, 18))
    for y in got:
        assert (y[:5] == 7).all() and (y[18:] == 7).all()


def test_kv_append_own_positions_and_in_place(gpu_lib):
    """positions that are not places: a cache whose oldest tokens went"""
    x = append_case([40, 3], [10, 0], 4, 2, 64, 64, 16, "fp32", "half", None, 0)
    pos = [500 + 2 * i for i in range(43)]
    ref = append_ref(x, pos=pos)
    q, k, _ = x["dev"]
    raw, got = run_append(gpu_lib, x, pos=pos, q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert got[0] is q and got[1] is k
    check_append(x, raw, got, ref)


@pytest.mark.parametrize("cu", [True, False])
def test_kv_append_faults(gpu_lib, cu):
    g = gpu_lib
    lens = [5, 1, 7, 20, 3, 4] if cu else [1] * 6
    x = append_case(lens, [0, 10, 30, 4, -1, 9], 4, 2, 64, 64, 16, "bf16", "half", "rms", 0)
    x["dst"][1] = 8                                       # outside the table
    x["begin"][2] = x["table"].shape[1] * 16 - lens[2] + 1     # one past the row's end
    x["table"][x["dst"][3], (4 + lens[3] - 1) // 16] = x["num"]          # its last page
    st = ints([-1] * 6)
    raw, got = run_append(g, x, cu=cu, status=st)
    torch.cuda.synchronize()
    assert st.tolist() == [0, g.FAULT_BAD_SLOT, g.FAULT_BAD_LENGTH, g.FAULT_BAD_PAGE, 0, 0]
    check_append(x, raw, got, append_ref(x, [True, False, False, False, False, True]))
    x["begin"][0] = -2
    x["table"][x["dst"][5], 0] = -1
    raw, got = run_append(g, x, cu=cu, status=st)
    torch.cuda.synchronize()
    assert st.tolist() == [g.FAULT_BAD_LENGTH, g.FAULT_BAD_SLOT, g.FAULT_BAD_LENGTH,
                           g.FAULT_BAD_PAGE, 0, g.FAULT_BAD_PAGE]
    assert torch.equal(raw.cpu(), x["raw"])


@pytest.mark.parametrize("cu", [[0, 3, 2, 8], [-1, 3, 4, 8], [0, 3, 4, 9], [3, 0, 0, 0]])
def test_kv_append_rows_that_do_not_ascend(gpu_lib, cu):
    x = append_case([3, 1, 4], [0, 10, 30], 4, 2, 64, 64, 16, "bf16", "half", "rms", 0)
    x["cu"] = cu
    st = ints([-1] * 3)
    q_out = torch.full((8, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    raw, got = run_append(gpu_lib, x, status=st, q_out=q_out)
    torch.cuda.synchronize()
    assert st.tolist() == [gpu_lib.FAULT_BAD_LENGTH] * 3
    assert torch.equal(raw.cpu(), x["raw"]) and (got[0] == 5).all() and not got[1].any()


def test_kv_append_past_32_bits(gpu_lib):
    """pages whose elements lie past 2^32 bytes and past 2^31 elements"""
    d, page, Hkv, num = 128, 64, 8, 33000
    cache = torch.zeros(num, Hkv, page, d, dtype=torch.bfloat16, device="cuda")     # 4.3 GB
    (q, k, v), (_, dk, dv) = projection((70,), 1, Hkv, d, "bf16", 29, True)
    f = frequencies(d)
    table = ints([[5, num - 1]])
    gpu_lib.kv_append(cache, cache.clone(), table, ints([0]), ints([30]), dk, dv, cu=ints([0, 70]),
                      inv_freq=f.cuda())
    torch.cuda.synchronize()
    ref, mag = heads_ref(k, range(30, 100), f, "half")
    got = torch.cat([cache[5, :, 30:], cache[num - 1, :, :36]], 1).transpose(0, 1)
    close(got, (ref, mag))
    assert not cache[5, :, :30].any() and not cache[num - 1, :, 36:].any()
    assert not cache[6:num - 1].any()


def test_kv_append_does_what_kv_commit_does(gpu_lib):
    """without norm and rotation: the same bytes in the same places"""
    lens, begin = [9, 1, 30], [0, 40, 5]
    x = append_case(lens, begin, 0, 2, 64, 0, 16, "bf16", "half", None, 0, fused=False)
    raw, _ = run_append(gpu_lib, x)
    c = view(x["raw"].cuda(), 2, 16, 64)
    n = 30
    k, v = (torch.zeros(3, n, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for r, m in enumerate(lens):
        k[r, :m] = x["dev"][1][x["cu"][r]:x["cu"][r] + m]
        v[r, :m] = x["dev"][2][x["cu"][r]:x["cu"][r] + m]
    gpu_lib.kv_commit(c[0], c[1], ints(x["table"].tolist()), ints(x["dst"]), ints(begin), k, v,
                      ints([list(range(n))] * 3), ints(lens))
    torch.cuda.synchronize()
    assert torch.equal(view(raw, 2, 16, 64), c)


# ---------------------------------------------------------------------------
# streams, graphs, prepared launches
# ---------------------------------------------------------------------------
def test_another_stream_and_prepared(gpu_lib):
    x = append_case([5, 1, 40], [0, 9, 30], 4, 2, 128, 128, 16, "bf16", "half", "rms", 0)
    want, (wq, wk) = run_append(gpu_lib, x)
    s = torch.cuda.Stream()
    raw = x["raw"].cuda()
    torch.cuda.synchronize()
    _, got = run_append(gpu_lib, x, stream=s, raw=raw)
    s.synchronize()
    assert torch.equal(raw, want) and torch.equal(got[0], wq) and torch.equal(got[1], wk)
    raw = x["raw"].cuda()
    _, launch = run_append(gpu_lib, x, raw=raw, prepare=True)
    assert isinstance(launch, gpu_lib.Launch)
    for _ in range(2):
        a, b = launch()
    torch.cuda.synchronize()
    assert torch.equal(raw, want) and torch.equal(a, wq) and torch.equal(b, wk)


def test_in_a_graph(gpu_lib):
    """captured once, replayed on changing inputs, lengths and pages"""
    x = append_case([5, 1, 40], [0, 9, 30], 4, 2, 128, 128, 16, "bf16", "half", "rms", 0)
    q, k, v = (y.contiguous() for y in x["dev"])
    w, f = x["w"].cuda(), x["f"].cuda()
    c = view(x["raw"].cuda(), 2, 16, 128)
    table, dst, begin = ints(x["table"].tolist()), ints(x["dst"]), ints(x["begin"])
    cu, pos, st = ints(x["cu"]), ints(list(range(46))), ints([-1] * 3)
    outs = [torch.empty_like(y) for y in (q, k, q, k)]

    def step(cache, o, status):
        gpu_lib.qk_norm_rope(q, k, w[0], w[1], pos, f, q_out=o[0], k_out=o[1])
        gpu_lib.kv_append(cache[0], cache[1], table, dst, begin, k, v, cu=cu, inv_freq=f,
                          norm="rms", k_weight=w[1], q=q, q_weight=w[0], q_out=o[2], k_out=o[3],
                          status=status)

    step(c, outs, st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(c, outs, st)
    for i in range(4):
        k.copy_(torch.randn(k.shape, generator=gen(40 + i)).to(k.dtype))
        begin.copy_(ints([i, 9 + i, 30 - i]))
        table[int(dst[1]), 0] = -1 if i == 2 else int(x["table"][x["dst"][1], 0])
        eager_c, eager_o, eager_st = c.clone(), [torch.empty_like(y) for y in outs], ints([-1] * 3)
        step(eager_c, eager_o, eager_st)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c, eager_c) and st.tolist() == eager_st.tolist()
        assert st.tolist()[1] == (gpu_lib.FAULT_BAD_PAGE if i == 2 else 0)
        for a, b in zip(outs, eager_o):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))


# ---------------------------------------------------------------------------
# the two ways to the entry points: with outputs given the native part checks
# and calls, without, or where it finds something unusual, Python does
# ---------------------------------------------------------------------------
def test_both_ways_give_the_same(gpu_lib):
    (q, k, v), (dq, dk, dv) = projection((2, 7), 6, 2, 64, "bf16", 31, True)
    f, w = frequencies(32).cuda(), torch.rand(64, device="cuda")
    pos, base = ints([list(range(7))] * 2), ints([5, 900])
    out = lambda: (torch.full(dq.shape, NAN, dtype=dq.dtype, device="cuda"),
                   torch.full(dk.shape, NAN, dtype=dk.dtype, device="cuda"))
    wq = torch.rand(6, 64, device="cuda")
    for fn, args, kw in (
            (gpu_lib.rope, (dq, dk, pos, f), dict(base=base, scale=1.5, layout="interleaved")),
            (gpu_lib.rope, (dq, dk, pos, f), {}),
            (gpu_lib.qk_norm_rope, (dq, dk, wq, w, pos, f), dict(base=base, norm="l2", offset=0.5)),
            (gpu_lib.qk_norm_rope, (dq, dk, w.bfloat16(), None, pos, f), dict(eps=0.1)),
            (gpu_lib.qk_norm_rope, (dq, dk, None, None), dict(norm="l2"))):
        a, b = out()
        got = fn(*args, q_out=a, k_out=b, **kw)
        assert got[0] is a and got[1] is b
        want = fn(*args, **kw)
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
        assert torch.equal(fn(args[0], None, *([args[2], None] if fn is gpu_lib.qk_norm_rope else []),
                              *args[4 if fn is gpu_lib.qk_norm_rope else 2:], q_out=out()[0],
                              **kw)[0], want[0])


def test_native_calls_leave_the_unusual_to_python(gpu_lib):
    """None, and nothing written, for every argument out of order"""
    native = gpu_lib._native()
    q, k = (torch.randn(3, H, 64, device="cuda").bfloat16() for H in (4, 2))
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    w, pos, f = torch.ones(64, device="cuda").bfloat16(), ints([1, 2, 3]), torch.ones(32, device="cuda")
    good = [1, q, k, w, w, pos, None, f, 1e-6, 0.0, 0, 1.0, qo, ko, None]

    def refused(call, args, at, value):
        x = list(args)
        x[at] = value
        assert call(*x) is None, (at, value if not torch.is_tensor(value) else value.shape)

    host = torch.zeros(3, dtype=torch.int32)
    for at, value in (
            (0, None), (0, 3), (0, -1), (1, None), (1, q.cpu()), (1, q.double()), (1, q[:2]),
            (1, q[..., ::2]), (2, k.float()), (2, k[:2]), (2, k[..., :32]), (2, None), (3, w.half()),
            (3, w[:32]), (3, w.float()), (4, torch.ones(4, 64, device="cuda").bfloat16()), (5, None),
            (5, pos.long()), (5, pos[:2]), (5, host), (5, pos[None]), (6, ints([1])), (7, f.double()),
            (7, torch.ones(33, device="cuda")), (7, f[None]), (8, "x"), (9, None), (10, None), (10, 2),
            (11, None), (12, None), (12, ko), (12, qo.float()), (13, None), (13, qo), (14, "s")):
        refused(native.heads_call, good, at, value)
    assert not qo.any() and not ko.any()
    rope = [0, q, k, None, None, pos, None, f, 0.0, 0.0, 0, 1.0, qo, ko, None]
    refused(native.heads_call, rope, 3, w)
    refused(native.heads_call, rope, 7, None)
    assert not qo.any()
    cache = torch.zeros(2, 4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    table, dst, begin = ints([[0, 1]] * 3), ints([0, 1, 2]), ints([0, 16, 3])
    good = [cache[0], cache[1], table, dst, begin, k, k, None, f, 0, 1.0, None, 1, 1e-6, 0.0, w, q, w,
            qo, ko, None, None]
    for at, value in (
            (0, cache[0].float()), (0, cache[0][:, :1]), (0, cache[0][:2]), (1, cache[1, :, :, :8]),
            (0, cache[0].transpose(0, 1)), (2, table[0]), (2, table.long()), (3, dst[:2]),
            (4, begin.cpu()), (5, k[:2]), (6, k[:2]), (6, k.float()), (7, ints([0, 1])), (7, host),
            (8, torch.ones(33, device="cuda")), (9, 5), (10, None), (11, ints([1, 2])), (12, 7),
            (15, w[:9]), (16, None), (16, q[:2]), (17, w.float()), (18, None), (18, ko), (19, qo),
            (20, ints([0])), (21, "s")):
        refused(native.append_call, good, at, value)
    assert not cache.any() and not qo.any() and not ko.any()
    assert native.append_call(*good) == 0
    torch.cuda.synchronize()
    assert cache.any() and qo.any() and ko.any()

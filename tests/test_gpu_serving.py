"""The serving operators on the GPU against plain 64-bit implementations:
prefill and step of the gated delta rule, attention of a draft tree over a
paged cache with shared prefixes, page bookkeeping.

Tolerances.  A rounding is off by at most half a step h(t) = finfo(t).eps / 2.
Rule outputs and states (fp32): operands enter products exactly or in parts
exact to 2^-24; a contraction of up to 128 terms and the few that follow one
another per chunk stay within 64 roundings of 2^-24 in the 2-norm.  A bf16
output adds its own rounding, elementwise.  Attention: each weight is rounded
once to the operand type, so with A = sum p |v| an output is off by at most
h A, its own rounding by h |out|, and fp32 scores and sums by less than
1e-4 A.  Whole numbers are equal.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

F32 = 64 * 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def half_step(t):
    return torch.finfo(t).eps / 2


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


# ---------------------------------------------------------------------------
# the gated delta rule
# ---------------------------------------------------------------------------
def rule_inputs(lens, H, Hk, dk, dv, dtype, slots, seed):
    g = gen(seed)
    rows = sum(lens)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    r = lambda *s: torch.randn(*s, generator=g)
    x = dict(q=unit(r(rows, Hk, dk)).to(DT[dtype]), k=unit(r(rows, Hk, dk)).to(DT[dtype]),
             v=r(rows, H, dv).to(DT[dtype]),
             alpha=torch.exp(-torch.exp(torch.rand(rows, H, generator=g) * 6.9 - 6.9)),
             beta=torch.sigmoid(r(rows, H)), S=r(slots, H, dk, dv) * dk ** -0.5)
    x["cu"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32)
    return x


def rule_ref(x, cu, src, dst):
    """token by token in 64 bits"""
    H, Hk = x["v"].shape[1], x["q"].shape[1]
    q, k = (x[n].double().repeat_interleave(H // Hk, dim=1) for n in ("q", "k"))
    v, a, b = x["v"].double(), x["alpha"].double(), x["beta"].double()
    S0 = x["S"].double()
    S, out = S0.clone(), torch.zeros(v.shape, dtype=torch.float64)
    for i in range(len(cu) - 1):
        M = S0[src[i]].clone() if src[i] >= 0 else torch.zeros_like(S0[0])
        for t in range(cu[i], cu[i + 1]):
            M = M * a[t][:, None, None]
            u = b[t][:, None] * (v[t] - (M * k[t][..., None]).sum(-2))
            M = M + k[t][..., None] * u[:, None, :]
            out[t] = (M * q[t][..., None]).sum(-2)
        S[dst[i]] = M
    return out, S


def near(got, ref, what):
    got, ref = got.double().cpu(), ref
    assert torch.isfinite(got).all(), what
    if got.numel() == 0:
        return
    err = (got - ref).norm() / max(ref.norm().item(), 1e-300)
    assert err <= F32, (what, err.item())


def near_out(got, ref, what):
    if got.dtype == torch.float32:
        return near(got, ref, what)
    rms = ref.square().mean().sqrt().item() if ref.numel() else 0.0
    off = (got.double().cpu() - ref).abs()
    # fp32 error before the rounding: F32 of the 2-norm, at one element at
    # most eight times its root mean square
    assert (off <= half_step(got.dtype) * ref.abs() + 8 * F32 * rms).all(), (what, off.max())


RULE = [
    # lens, H, Hk, dk, dv, dtype, out
    ([1], 1, 1, 8, 8, "fp32", "fp32"),
    ([1, 2, 0, 5], 2, 1, 16, 24, "fp32", "fp32"),
    ([3, 0, 64, 1], 4, 2, 64, 48, "bf16", "fp32"),
    ([63, 64, 65, 66], 2, 2, 128, 128, "bf16", "fp32"),
    ([130, 1, 31, 33], 4, 1, 128, 64, "bf16", "bf16"),
    ([257], 2, 2, 72, 120, "bf16", "fp32"),
    ([200, 7], 3, 3, 40, 128, "fp32", "bf16"),
    ([96, 97], 2, 1, 128, 128, "fp32", "fp32"),
    ([15, 16, 17, 48, 49], 2, 2, 128, 16, "bf16", "fp32"),
    ([1000], 1, 1, 128, 128, "bf16", "fp32"),
    ([0, 0], 2, 2, 64, 64, "bf16", "fp32"),
]


@pytest.mark.parametrize("lens,H,Hk,dk,dv,dtype,out", RULE)
def test_prefill(gpu_lib, lens, H, Hk, dk, dv, dtype, out):
    print("prefill", lens, H, Hk, dk, dv, dtype, out, flush=True)
    batch = len(lens)
    x = rule_inputs(lens, H, Hk, dk, dv, dtype, 2 * batch + 1, 7)
    # from a slot, from zero, in place
    src = [[i, -1, batch + i][i % 3] for i in range(batch)]
    dst = [batch + i for i in range(batch)]
    d = {n: t.cuda() for n, t in x.items()}
    o = torch.full((sum(lens), H, dv), float("nan"), dtype=DT[out], device="cuda")
    st = ints([-1] * batch)
    r = gpu_lib.prefill(d["q"], d["k"], d["v"], d["alpha"], d["beta"], d["cu"], d["S"], ints(src),
                        ints(dst), out=o, status=st)
    torch.cuda.synchronize()
    assert r is o and st.tolist() == [0] * batch
    ro, rS = rule_ref(x, x["cu"].tolist(), src, dst)
    near_out(o, ro, "out")
    near(d["S"], rS, "S")
    untouched = [i for i in range(2 * batch + 1) if i not in dst]
    assert torch.equal(d["S"].cpu()[untouched], x["S"][untouched])


def check_prefill(lib, lens, H, Hk, dk, dv, dtype, out, seed):
    batch = len(lens)
    x = rule_inputs(lens, H, Hk, dk, dv, dtype, 2 * batch, seed)
    src = [i if i % 3 else -1 for i in range(batch)]
    dst = [batch + i for i in range(batch)]
    d = {n: t.cuda() for n, t in x.items()}
    o = torch.full((sum(lens), H, dv), float("nan"), dtype=DT[out], device="cuda")
    st = ints([-1] * batch)
    lib.prefill(d["q"], d["k"], d["v"], d["alpha"], d["beta"], d["cu"], d["S"], ints(src),
                ints(dst), out=o, status=st)
    torch.cuda.synchronize()
    assert st.tolist() == [0] * batch
    ro, rS = rule_ref(x, x["cu"].tolist(), src, dst)
    near_out(o, ro, "out")
    near(d["S"], rS, "S")
    assert torch.equal(d["S"].cpu()[:batch], x["S"][:batch])


@pytest.mark.parametrize("H,Hk,dk,dv,dtype,out", [
    (32, 16, 128, 128, "bf16", "fp32"), (32, 32, 64, 72, "bf16", "bf16"),
    (32, 8, 128, 40, "fp32", "fp32"), (64, 64, 48, 64, "fp32", "bf16"),
])
def test_prefill_many_sequences(gpu_lib, H, Hk, dk, dv, dtype, out):
    """enough (sequence, head) pairs that a workgroup takes 64 columns"""
    print("prefill many", H, Hk, dk, dv, dtype, out, flush=True)
    check_prefill(gpu_lib, [1, 64, 0, 65, 3, 130, 17, 63], H, Hk, dk, dv, dtype, out, 11)


@pytest.mark.parametrize("batch", [1023, 1024, 1025, 1100])
def test_prefill_thousand_sequences(gpu_lib, batch):
    """around the number of sequences that are ordered by length"""
    print("prefill", batch, "sequences", flush=True)
    check_prefill(gpu_lib, [i * 7 % 4 for i in range(batch - 1)] + [70], 1, 1, 8, 8, "fp32",
                  "fp32", 13)


def test_prefill_keeps_values_that_are_not_finite_in_their_sequence(gpu_lib):
    lens = [70, 200, 40]
    x = rule_inputs(lens, 2, 1, 64, 64, "bf16", 3, 17)
    bad = {n: t.clone() for n, t in x.items()}
    bad["v"][70 + 130, 0, 5] = float("nan")          # chunk 2 of sequence 1, head 0
    bad["alpha"][70 + 130, 1] = -0.5
    got = []
    for y in (x, bad):
        d = {n: t.cuda() for n, t in y.items()}
        o = gpu_lib.prefill(d["q"], d["k"], d["v"], d["alpha"], d["beta"], d["cu"], d["S"],
                            ints([0, 1, 2]), ints([0, 1, 2]),
                            out=torch.empty(310, 2, 64, device="cuda"))
        got.append((o.cpu(), d["S"].cpu()))
    (o, S), (ob, Sb) = got
    assert torch.equal(ob[:70 + 128], o[:70 + 128]) and torch.equal(ob[270:], o[270:])
    assert torch.equal(Sb[[0, 2]], S[[0, 2]])
    assert torch.isnan(ob[200:270, 0, 5]).all() and torch.isnan(ob[200:270, 1]).all()
    assert torch.equal(ob[198:270, 0, 16:], o[198:270, 0, 16:])      # other columns of the state
    assert torch.isnan(Sb[1, 0, :, 5]).all() and torch.isnan(Sb[1, 1]).all()


def test_prefill_cleared_and_saturated_gates(gpu_lib):
    """alpha = 0 clears the state, alpha = 1 keeps it, beta = 0 writes nothing"""
    lens = [150, 70]
    x = rule_inputs(lens, 2, 2, 64, 64, "bf16", 4, 3)
    x["alpha"][40, 0] = 0.0
    x["alpha"][41, 0] = 0.0
    x["alpha"][100, 1] = 0.0
    x["alpha"][150:, :] = 1.0
    x["alpha"][5:20, 1] = 1e-30
    x["beta"][60:70] = 0.0
    d = {n: t.cuda() for n, t in x.items()}
    o = gpu_lib.prefill(d["q"], d["k"], d["v"], d["alpha"], d["beta"], d["cu"], d["S"],
                        ints([0, 1]), ints([2, 3]), out=torch.empty(220, 2, 64, device="cuda"))
    ro, rS = rule_ref(x, [0, 150, 220], [0, 1], [2, 3])
    near(o, ro, "out")
    near(d["S"], rS, "S")


def test_prefill_continues_where_it_stopped(gpu_lib):
    """a prompt in two calls gives the state and outputs of one"""
    x = rule_inputs([333], 2, 1, 128, 128, "bf16", 3, 5)
    d = {n: t.cuda() for n, t in x.items()}
    one = gpu_lib.prefill(d["q"], d["k"], d["v"], d["alpha"], d["beta"], d["cu"], d["S"],
                          ints([-1]), ints([0]), out=torch.empty(333, 2, 128, device="cuda"))
    two = torch.empty_like(one)
    for a, b, s in ((0, 100, -1), (100, 333, 1)):
        gpu_lib.prefill(d["q"][a:b], d["k"][a:b], d["v"][a:b], d["alpha"][a:b].contiguous(),
                        d["beta"][a:b].contiguous(), ints([0, b - a]), d["S"], ints([s]),
                        ints([1]), out=two[a:b])
    torch.cuda.synchronize()
    assert (one - two).norm() <= 2 * F32 * one.norm()
    assert (d["S"][0] - d["S"][1]).norm() <= 2 * F32 * d["S"][0].norm()


def test_prefill_faults(gpu_lib):
    """bad row offsets and slots are reported, nothing of theirs is written"""
    lens = [10, 20, 30, 5]
    x = rule_inputs(lens, 2, 1, 64, 64, "bf16", 8, 9)
    d = {n: t.cuda() for n, t in x.items()}
    S0 = d["S"].clone()
    cu = ints([0, 10, 30, 60, 1 << 30])            # the last one passes the rows
    o = torch.full((65, 2, 64), 7.0, device="cuda")
    st = ints([-1] * 4)
    gpu_lib.prefill(d["q"], d["k"], d["v"], d["alpha"], d["beta"], cu, d["S"],
                    ints([8, -2, 0, 1]), ints([4, 5, 8, 7]), out=o, status=st)
    torch.cuda.synchronize()
    assert st.tolist() == [gpu_lib.FAULT_BAD_SLOT] * 3 + [gpu_lib.FAULT_BAD_LENGTH]
    assert torch.isnan(o[:60]).all() and (o[60:] == 7.0).all()
    assert torch.equal(d["S"], S0)
    for bad in ([5, 3, 30, 60, 65], [-4, 10, 30, 60, 65]):
        gpu_lib.prefill(d["q"], d["k"], d["v"], d["alpha"], d["beta"], ints(bad), d["S"],
                        ints([-1] * 4), ints([4, 5, 6, 7]), out=o, status=st)
        torch.cuda.synchronize()
        assert st.tolist()[0] == gpu_lib.FAULT_BAD_LENGTH and st.tolist()[2:] == [0, 0]


@pytest.mark.parametrize("batch,H,Hk,dk,dv,dtype,out", [
    (1, 32, 16, 128, 128, "bf16", "bf16"), (1, 1, 1, 8, 8, "fp32", "fp32"),
    (5, 4, 1, 64, 48, "bf16", "fp32"), (3, 6, 3, 72, 40, "fp32", "bf16"),
    (7, 2, 2, 128, 120, "fp32", "fp32"), (64, 2, 2, 16, 128, "bf16", "fp32"),
])
def test_step(gpu_lib, batch, H, Hk, dk, dv, dtype, out):
    print("step", batch, H, Hk, dk, dv, dtype, out, flush=True)
    x = rule_inputs([1] * batch, H, Hk, dk, dv, dtype, 2 * batch, 11)
    src = [-1 if i % 5 == 4 else i // 4 for i in range(batch)]      # shared sources
    dst = [batch + i for i in range(batch)]
    d = {n: t.cuda() for n, t in x.items()}
    st = ints([-1] * batch)
    o = torch.empty(batch, H, dv, dtype=DT[out], device="cuda")
    gpu_lib.step(d["q"], d["k"], d["v"], d["alpha"], d["beta"], d["S"], ints(src), ints(dst), out=o,
                 status=st)
    torch.cuda.synchronize()
    ro, rS = rule_ref(x, list(range(batch + 1)), src, dst)
    assert st.tolist() == [0] * batch
    near_out(o, ro, "out")
    near(d["S"], rS, "S")


def test_step_in_place_and_faults(gpu_lib):
    x = rule_inputs([1] * 4, 2, 2, 64, 64, "bf16", 4, 13)
    d = {n: t.cuda() for n, t in x.items()}
    st = ints([-1] * 4)
    o = gpu_lib.step(d["q"], d["k"], d["v"], d["alpha"], d["beta"], d["S"], ints([0, 1, 2, 4]),
                     ints([0, 1, -1, 3]), out=torch.empty(4, 2, 64, device="cuda"), status=st)
    torch.cuda.synchronize()
    bad = gpu_lib.FAULT_BAD_SLOT
    assert st.tolist() == [0, 0, bad, bad]
    ro, rS = rule_ref(x, [0, 1, 2], [0, 1], [0, 1])
    near(o[:2], ro[:2], "out")
    near(d["S"], rS, "S")
    assert torch.isnan(o[2:]).all() and torch.equal(d["S"][2:].cpu(), x["S"][2:])


# ---------------------------------------------------------------------------
# attention of a draft tree
# ---------------------------------------------------------------------------
def tree(rng, n):
    return [-1] + [int(rng.integers(max(-1, i - 6), i)) for i in range(1, n)]


def attention_inputs(lengths, n, Hq, Hkv, d, page, dtype, seed, groups=None):
    """groups: list of (first, last + 1, shared tokens); the members' rows name
    the same pages there.  Unused cache rows hold NaN."""
    rng = np.random.default_rng(seed)
    g = gen(seed)
    batch = len(lengths)
    width = max(1, max(-(-x // page) for x in lengths)) + 1
    rows = -np.ones((batch, width), np.int64)
    ids = list(rng.permutation(sum(-(-x // page) for x in lengths) + 3))
    for b, x in enumerate(lengths):
        for c in range(-(-x // page)):
            rows[b, c] = ids.pop()
    for lo, hi, tokens in groups or []:
        full = max(range(lo, hi), key=lambda b: lengths[b])
        for b in range(lo, hi):
            upto = -(-min(tokens, lengths[b]) // page)
            rows[b, :upto] = rows[full, :upto]
        # the first member's row is the one that is read
        upto = -(-min(tokens, lengths[full]) // page)
        rows[lo, :upto] = rows[full, :upto]
    pool = int(rows.max()) + 3
    r = lambda *s: torch.randn(*s, generator=g).to(DT[dtype])
    x = dict(q=r(batch, n, Hq, d), k=r(batch, n, Hkv, d), v=r(batch, n, Hkv, d),
             kc=r(pool, Hkv, page, d), vc=r(pool, Hkv, page, d))
    used = torch.zeros(pool, page, dtype=torch.bool)
    for b, n_b in enumerate(lengths):
        for t in range(n_b):
            used[rows[b, t // page], t % page] = True
    for c in ("kc", "vc"):
        x[c] = torch.where(used[:, None, :, None], x[c], torch.tensor(float("nan"), dtype=DT[dtype]))
    x["parent"] = torch.tensor([tree(rng, n) for _ in range(batch)], dtype=torch.int32)
    x["pages"] = torch.tensor(rows, dtype=torch.int32)
    x["length"] = torch.tensor(lengths, dtype=torch.int32)
    return x


def attention_ref(x, scale):
    """(out, sum p |v|) in 64 bits, row by row over the keys it sees"""
    batch, n, Hq, d = x["q"].shape
    G = Hq // x["k"].shape[2]
    page = x["kc"].shape[2]
    out = torch.zeros(batch, n, Hq, d, dtype=torch.float64)
    mag = torch.zeros_like(out)
    for b in range(batch):
        L = int(x["length"][b])
        at = x["pages"][b, : -(-L // page)].long()
        kc, vc = (x[c][at].transpose(1, 2).reshape(-1, Hq // G, d)[:L].double()
                  for c in ("kc", "vc"))
        for i in range(n):
            chain, j = [], i
            while j >= 0:
                chain.append(j)
                j = int(x["parent"][b, j])
            K = torch.cat([kc, x["k"][b, chain].double()]).repeat_interleave(G, 1)
            V = torch.cat([vc, x["v"][b, chain].double()]).repeat_interleave(G, 1)
            p = torch.softmax(scale * torch.einsum("hd,jhd->hj", x["q"][b, i].double(), K), -1)
            out[b, i] = torch.einsum("hj,jhd->hd", p, V)
            mag[b, i] = torch.einsum("hj,jhd->hd", p, V.abs())
    return out, mag


def attention_near(got, ref, mag, what=""):
    h = half_step(got.dtype)
    off = (got.double().cpu() - ref).abs()
    tol = h * ref.abs() + (h + 1e-4) * mag
    assert torch.isfinite(got).all(), what
    assert (off <= tol).all(), (what, (off / tol).max().item())


def attend(lib, x, scale, shared=None, **kw):
    d = {n: t.cuda() for n, t in x.items()}
    return lib.tree_attention(d["q"], d["k"], d["v"], d["parent"], d["kc"], d["vc"], d["pages"],
                              d["length"], scale, shared=shared, **kw)


ATTENTION = [
    # lengths, n, Hq, Hkv, d, page, dtype, groups
    ([0], 1, 1, 1, 64, 16, "bf16", None),
    ([1], 1, 4, 1, 128, 16, "fp16", None),
    ([17, 0, 128, 129], 1, 8, 2, 128, 16, "bf16", None),
    ([1000], 1, 8, 8, 128, 16, "bf16", None),
    ([300, 5], 33, 4, 2, 64, 32, "bf16", None),
    ([255, 256, 257], 7, 6, 2, 128, 64, "fp16", None),
    ([40, 700], 128, 2, 1, 128, 16, "bf16", None),
    ([90], 64, 8, 1, 256, 16, "bf16", None),
    ([90, 33], 9, 2, 2, 72, 8, "fp16", None),
    ([50], 3, 2, 1, 8, 1, "bf16", None),
    ([200, 200, 200], 1, 40, 1, 128, 16, "bf16", None),
    ([400, 390, 300, 260], 1, 8, 2, 128, 16, "bf16", [(0, 4, 256)]),
    ([400, 390, 300, 260, 100], 5, 4, 1, 64, 32, "fp16", [(0, 2, 320), (2, 4, 250)]),
    ([130, 50, 131, 0], 20, 2, 2, 128, 16, "bf16", [(0, 4, 128)]),     # shorter than shared
    ([600] * 9, 16, 8, 2, 128, 64, "bf16", [(0, 1, 512), (1, 8, 512)]),
    ([64, 64], 2, 2, 1, 256, 64, "bf16", [(0, 2, 64)]),                # nothing of their own
    ([300] * 40, 1, 16, 1, 64, 16, "fp16", [(3, 37, 272)]),            # rows over many units
]


@pytest.mark.parametrize("lengths,n,Hq,Hkv,d,page,dtype,groups", ATTENTION)
def test_tree_attention(gpu_lib, lengths, n, Hq, Hkv, d, page, dtype, groups):
    print("attention", lengths[:6], n, Hq, Hkv, d, page, dtype, groups, flush=True)
    x = attention_inputs(lengths, n, Hq, Hkv, d, page, dtype, 17, groups)
    ref, mag = attention_ref(x, d ** -0.5)
    st = ints([-1] * len(lengths))
    plain = attend(gpu_lib, x, d ** -0.5, status=st)
    torch.cuda.synchronize()
    assert st.tolist() == [0] * len(lengths)
    attention_near(plain, ref, mag, "no groups")
    if groups:
        shared = (ints([groups[0][0]] + [g[1] for g in groups]), ints([g[2] for g in groups]))
        st.fill_(-1)
        got = attend(gpu_lib, x, d ** -0.5, shared=shared, status=st)
        torch.cuda.synchronize()
        assert st.tolist() == [0] * len(lengths)
        attention_near(got, ref, mag, "groups")


@pytest.mark.parametrize("scale", [-0.1, 0.0, 3.0])
def test_tree_attention_scales(gpu_lib, scale):
    """negative, zero and sharp scales"""
    x = attention_inputs([200, 77], 5, 4, 2, 64, 16, "bf16", 19)
    ref, mag = attention_ref(x, scale)
    attention_near(attend(gpu_lib, x, scale), ref, mag)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_tree_attention_keeps_masked_values_out(gpu_lib, dtype):
    """infinities and NaN in nodes that are no ancestors, and in shared tokens
    past a member's length, do not reach the others; in an ancestor they do"""
    x = attention_inputs([100, 30], 6, 4, 2, 128, 16, dtype, 23, [(0, 2, 96)])
    x["parent"][:] = torch.tensor([-1, 0, 0, 1, 2, 4])
    ref, mag = attention_ref(x, 0.1)
    x["v"][:, 3] = float("inf")                    # leaf 3: seen by itself alone
    x["k"][:, 3] = float("nan")
    x["v"][:, 5, :, ::7] = float("nan")
    page, off = int(x["pages"][0, 4]), 3           # token 67: past sequence 1
    x["vc"][page, :, off, 5] = float("-inf")
    got = attend(gpu_lib, x, 0.1, shared=(ints([0, 2]), ints([96])))
    torch.cuda.synchronize()
    got = got.cpu()
    keep = [0, 1, 2, 4]
    attention_near(got[1, keep], ref[1, keep], mag[1, keep])
    cols = [c for c in range(128) if c != 5]
    attention_near(got[0, keep][..., cols], ref[0, keep][..., cols], mag[0, keep][..., cols])
    assert (got[0, keep][..., 5] == float("-inf")).all()
    assert not torch.isfinite(got[:, 3]).any()
    assert torch.isnan(got[:, 5, :, ::7]).all()


def test_tree_attention_peaked_rows(gpu_lib):
    """scores far apart and all equal: the running maximum moves"""
    x = attention_inputs([500], 4, 2, 1, 64, 16, "bf16", 29)
    x["q"][0, 1] *= 40
    x["q"][0, 2] = 0
    ref, mag = attention_ref(x, 0.125)
    attention_near(attend(gpu_lib, x, 0.125), ref, mag)


def test_tree_attention_page_strides(gpu_lib):
    """keys and values interleaved page by page"""
    x = attention_inputs([333, 64], 3, 4, 2, 128, 32, "bf16", 31)
    ref, mag = attention_ref(x, 0.09)
    both = torch.stack([x["kc"], x["vc"]], 1).cuda()             # [pages][2][...]
    d = {n: t.cuda() for n, t in x.items()}
    got = gpu_lib.tree_attention(d["q"], d["k"], d["v"], d["parent"], both[:, 0], both[:, 1],
                                 d["pages"], d["length"], 0.09)
    attention_near(got, ref, mag)


def test_tree_attention_faults(gpu_lib):
    """a sequence with a bad parent, length, page or group gives NaN and its
    flag; the others are as before"""
    L = [100, 100, 100, 100, 100]
    x = attention_inputs(L, 4, 2, 1, 64, 16, "bf16", 37)
    ref, mag = attention_ref(x, 0.1)
    x["parent"][0, 2] = 2
    x["length"][1] = 100000
    x["pages"][2, 3] = 1 << 20
    x["pages"][3, 0] = -1
    st = ints([-1] * 5)
    got = attend(gpu_lib, x, 0.1, status=st)
    torch.cuda.synchronize()
    assert st.tolist() == [gpu_lib.FAULT_BAD_PARENT, gpu_lib.FAULT_BAD_LENGTH,
                           gpu_lib.FAULT_BAD_PAGE, gpu_lib.FAULT_BAD_PAGE, 0]
    assert torch.isnan(got[:4]).all()
    attention_near(got[4:], ref[4:], mag[4:])
    # groups: rows that differ within the shared tokens; offsets out of order
    x = attention_inputs(L, 4, 2, 1, 64, 16, "bf16", 37)
    got = attend(gpu_lib, x, 0.1, shared=(ints([0, 2]), ints([32])), status=st)
    torch.cuda.synchronize()
    assert st.tolist() == [0, gpu_lib.FAULT_BAD_GROUP, 0, 0, 0]
    assert torch.isnan(got[1]).all()
    attention_near(got[[0, 2, 3, 4]], ref[[0, 2, 3, 4]], mag[[0, 2, 3, 4]])
    for start in ([3, 1], [0, 6], [-1, 2]):
        got = attend(gpu_lib, x, 0.1, shared=(ints(start), ints([32])), status=st)
        torch.cuda.synchronize()
        assert st.tolist() == [gpu_lib.FAULT_BAD_GROUP] * 5 and torch.isnan(got).all()


# ---------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------
class Pages:
    """the page table in plain Python, one request after the other"""

    def __init__(self, rng, seqs, width, pool, page, lengths):
        self.page, self.width = page, width
        self.table = -np.ones((seqs, width), np.int64)
        self.length = np.zeros(seqs, np.int64)
        self.ref = np.zeros(pool, np.int64)
        ids = list(rng.permutation(pool))
        for s, x in lengths.items():
            self.length[s] = x
            for c in range(-(-x // page)):
                self.table[s, c] = ids.pop()
                self.ref[self.table[s, c]] += 1

    def up(self):
        return ints(self.table.tolist()), ints(self.length.tolist()), ints(self.ref.tolist())

    def free(self):
        return int((self.ref == 0).sum())

    def take(self):
        p = int(np.argmax(self.ref == 0))
        self.ref[p] = 1
        return p

    def fork(self, src, dst):
        copies = []
        ask = 0
        avail = self.free()
        for s, d in zip(src, dst):
            whole, part = divmod(int(self.length[s]), self.page)
            ask += part > 0
            if part and ask > avail:
                copies.append([-1, -1])
                continue
            self.table[d] = -1
            self.table[d, :whole] = self.table[s, :whole]
            self.ref[self.table[s, :whole]] += 1
            if part:
                self.table[d, whole] = self.take()
                copies.append([int(self.table[s, whole]), int(self.table[d, whole])])
            else:
                copies.append([-1, -1])
            self.length[d] = self.length[s]
        return copies

    def extend(self, dst, add):
        begin, asked, avail = [], 0, self.free()
        for d, m in zip(dst, add):
            old = int(self.length[d])
            have, want = -(-old // self.page), -(-(old + m) // self.page)
            asked += want - have
            if asked > avail:
                begin.append(-1)
                continue
            for c in range(have, want):
                self.table[d, c] = self.take()
            begin.append(old)
            self.length[d] = old + m
        return begin

    def release(self, done):
        for d in done:
            for c in range(-(-int(self.length[d]) // self.page)):
                self.ref[self.table[d, c]] -= 1
            self.table[d] = -1
            self.length[d] = 0

    def compact(self):
        used = int((self.ref > 0).sum())
        moves = [p for p in range(used, len(self.ref)) if self.ref[p]]
        holes = [p for p in range(used) if not self.ref[p]]
        to = np.arange(len(self.ref))
        for p, q in zip(moves, holes):
            to[p] = q
            self.ref[q], self.ref[p] = self.ref[p], 0
        for s in range(len(self.length)):
            n = -(-int(self.length[s]) // self.page)
            self.table[s, :n] = to[self.table[s, :n]]
        return [[p, int(to[p])] for p in moves]

    def same(self, table, length, ref):
        assert table.cpu().numpy().tolist() == self.table.tolist()
        assert length.tolist() == self.length.tolist()
        assert ref.tolist() == self.ref.tolist()


@pytest.mark.parametrize("seqs,width,pool,page,live,forks", [
    (4, 3, 9, 4, 1, 2), (40, 12, 300, 16, 10, 30), (200, 9, 1500, 64, 40, 130),
    (3000, 4, 6000, 1, 700, 2200), (20, 40, 90, 16, 5, 15),
])
def test_page_life(gpu_lib, seqs, width, pool, page, live, forks):
    """fork, extend, free, compact against the plain table, request by request"""
    print("pages", seqs, width, pool, page, flush=True)
    rng = np.random.default_rng(seqs)
    top = width * page
    lengths = {}
    left = pool
    for s in range(live):
        x = int(rng.integers(0, top - page + 1))
        if -(-x // page) <= left:
            lengths[s] = x
            left -= -(-x // page)
    P = Pages(rng, seqs, width, pool, page, lengths)
    table, length, ref = P.up()
    st = ints([-1] * forks)
    src = [int(rng.integers(0, live)) for _ in range(forks)]
    dst = [int(x) for x in rng.choice(np.arange(live, seqs), forks, replace=False)]
    copies = gpu_lib.page_fork(table, length, ref, ints(src), ints(dst), page, status=st)
    want = P.fork(src, dst)
    torch.cuda.synchronize()
    assert copies.tolist() == want
    P.same(table, length, ref)
    refused = [int(c == [-1, -1] and P.length[s] % page != 0) for c, s in zip(want, src)]
    assert st.tolist() == [gpu_lib.FAULT_NO_PAGE * r for r in refused]

    add = [int(rng.integers(0, 2 * page + 1)) for _ in range(forks)]
    add = [min(a, top - int(P.length[d])) for a, d in zip(add, dst)]
    begin = gpu_lib.page_extend(table, length, ref, ints(dst), ints(add), page, status=st)
    want = P.extend(dst, add)
    torch.cuda.synchronize()
    assert begin.tolist() == want
    P.same(table, length, ref)
    assert st.tolist() == [gpu_lib.FAULT_NO_PAGE * (w < 0) for w in want]

    done = [int(x) for x in rng.choice(seqs, max(1, seqs // 3), replace=False)]
    gpu_lib.page_free(table, length, ref, ints(done + done[:2]), page)     # two named twice
    P.release(done)
    torch.cuda.synchronize()
    P.same(table, length, ref)

    copies, count = gpu_lib.page_compact(table, length, ref, page)
    want = P.compact()
    torch.cuda.synchronize()
    assert int(count) == len(want) and copies[: len(want)].tolist() == want
    P.same(table, length, ref)
    # a second time there is nothing to move
    copies, count = gpu_lib.page_compact(table, length, ref, page)
    torch.cuda.synchronize()
    assert int(count) == 0
    P.same(table, length, ref)


def test_page_requests_that_cannot_be(gpu_lib):
    """bad rows, rows in use, repeated rows, lengths and ids: reported, and
    nothing changes for them"""
    rng = np.random.default_rng(1)
    P = Pages(rng, 8, 4, 20, 4, {0: 10, 1: 16, 2: 3})
    P.table[2, 0] = 25                                    # outside the pool
    table, length, ref = P.up()
    bad, page, none = (gpu_lib.FAULT_BAD_SLOT, gpu_lib.FAULT_BAD_PAGE, 0)
    src, dst = [0, 9, 0, 0, 2, 1, 1, 0], [4, 5, -1, 1, 6, 6, 6, 0]
    st = ints([-1] * 8)
    copies = gpu_lib.page_fork(table, length, ref, ints(src), ints(dst), 4, status=st)
    torch.cuda.synchronize()
    assert st.tolist() == [none, bad, bad, bad, page, none, bad, bad]
    want = P.fork([0, 1], [4, 6])
    assert copies.tolist() == [want[0]] + [[-1, -1]] * 7
    P.same(table, length, ref)
    st = ints([-1] * 5)
    begin = gpu_lib.page_extend(table, length, ref, ints([4, 4, 1, 8, 0]), ints([3, 1, 1, 1, -1]),
                                4, status=st)
    torch.cuda.synchronize()
    size = gpu_lib.FAULT_BAD_LENGTH
    assert st.tolist() == [none, bad, size, bad, size]
    assert begin.tolist() == P.extend([4], [3]) + [-1] * 4
    P.same(table, length, ref)
    st = ints([-1] * 3)
    gpu_lib.page_free(table, length, ref, ints([4, -1, 8]), 4, status=st)
    P.release([4])
    torch.cuda.synchronize()
    assert st.tolist() == [none, bad, bad]
    P.same(table, length, ref)


@pytest.mark.parametrize("shape,dtype", [((1, 7, 3, 2, 8), "fp32"), ((2, 9, 4, 16, 64), "bf16"),
                                         ((4, 5, 8, 64, 128), "fp16")])
def test_page_copy(gpu_lib, shape, dtype):
    cache = torch.randn(*shape).to(DT[dtype])
    copies = [[0, 3], [-1, -1], [1, 4], [2, 99], [77, 1], [2, 2]]
    for count in (None, 0, 1, 3):
        got = cache.cuda()
        gpu_lib.page_copy(got, ints(copies), None if count is None else ints([count]))
        want = cache.clone()
        for f, t in copies[:count]:
            if 0 <= f < shape[1] and 0 <= t < shape[1]:
                want[:, t] = cache[:, f]
        torch.cuda.synchronize()
        assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("Hkv,d,page,n,dtype", [(1, 8, 1, 3, "fp32"), (2, 72, 16, 40, "fp16"),
                                                (8, 128, 64, 64, "bf16")])
def test_kv_commit(gpu_lib, Hkv, d, page, n, dtype):
    rng = np.random.default_rng(3)
    m, seqs, width = 5, 6, -(-3 * n // page) + 1
    table = rng.permutation(seqs * width).reshape(seqs, width)
    pool = seqs * width
    kc, vc = (torch.randn(pool, Hkv, page, d).to(DT[dtype]) for _ in range(2))
    k, v = (torch.randn(m, n, Hkv, d).to(DT[dtype]) for _ in range(2))
    dst, begin = [3, 0, 5, 1, 2], [0, n, -1, 2 * n, 5]
    add = [n, 1, 3, 0, n // 2 + 1]
    path = [sorted(rng.choice(n, n, replace=True).tolist()) for _ in range(m)]
    wk, wv = kc.clone(), vc.clone()
    for r in range(m):
        for j in range(add[r] if begin[r] >= 0 else 0):
            c, o = divmod(begin[r] + j, page)
            wk[table[dst[r], c], :, o] = k[r, path[r][j]]
            wv[table[dst[r], c], :, o] = v[r, path[r][j]]
    # as one cache [2][pool], and as pages that hold keys and values
    for caches in ((kc.cuda(), vc.cuda()), torch.stack([kc, vc], 1).cuda().unbind(1)):
        st = ints([-1] * m)
        gpu_lib.kv_commit(*caches, ints(table.tolist()), ints(dst), ints(begin), k.cuda(), v.cuda(),
                          ints(path), ints(add), status=st)
        torch.cuda.synchronize()
        assert torch.equal(caches[0].cpu(), wk) and torch.equal(caches[1].cpu(), wv)
        assert st.tolist() == [0] * m


def test_kv_commit_faults(gpu_lib):
    kc, vc = torch.zeros(6, 1, 4, 8).cuda(), torch.zeros(6, 1, 4, 8).cuda()
    k = torch.ones(5, 3, 1, 8).cuda()
    table = ints([[0, 1], [2, 6], [3, -1]])
    st = ints([-1] * 5)
    # row outside, node outside, add past the path, pages outside, past the row
    gpu_lib.kv_commit(kc, vc, table, ints([3, 0, 0, 1, 0]), ints([0, 0, 0, 3, 6]), k, k,
                      ints([[0, 1, 2], [0, 3, 1], [0, 1, 2], [0, 1, 2], [0, 1, 2]]),
                      ints([1, 2, 4, 2, 3]), status=st)
    torch.cuda.synchronize()
    assert st.tolist() == [gpu_lib.FAULT_BAD_SLOT, gpu_lib.FAULT_BAD_PATH, gpu_lib.FAULT_BAD_PATH,
                           gpu_lib.FAULT_BAD_PAGE, gpu_lib.FAULT_BAD_LENGTH]
    assert not kc.any() and not vc.any()


# ---------------------------------------------------------------------------
# streams and graphs
# ---------------------------------------------------------------------------
def serving_step(lib, x, d, r, out, P):
    """one decoded token: the rule's step, room and rows for it, attention"""
    table, length, ref = P
    lib.step(r["q"], r["k"], r["v"], r["alpha"], r["beta"], r["S"], r["src"], r["src"],
             out=out["rule"])
    lib.tree_attention(d["q"], d["k"], d["v"], d["parent"], d["kc"], d["vc"], table, length, 0.1,
                       shared=d["shared"], out=out["attention"])
    begin = lib.page_extend(table, length, ref, d["rows"], d["ones"], 16)
    lib.kv_commit(d["kc"], d["vc"], table, d["rows"], begin, d["k"], d["v"], d["path"], d["ones"])


def serving_state():
    L = [100, 90, 79, 64]
    x = attention_inputs(L, 1, 4, 2, 64, 16, "bf16", 41, [(0, 4, 64)])
    x["kc"], x["vc"] = (torch.cat([torch.nan_to_num(x[c]), torch.zeros(16, *x[c].shape[1:],
                                                                       dtype=x[c].dtype)])
                        for c in ("kc", "vc"))
    x["pages"] = torch.cat([x["pages"], torch.full((4, 4), -1, dtype=torch.int32)], 1)
    ref = torch.zeros(x["kc"].shape[0], dtype=torch.int32)
    for b, n in enumerate(L):
        for c in range(-(-n // 16)):
            ref[x["pages"][b, c]] += 1
    d = {n: t.cuda() for n, t in x.items()}
    d["shared"] = (ints([0, 4]), ints([64]))
    d["rows"], d["ones"], d["path"] = ints([0, 1, 2, 3]), ints([1] * 4), ints([[0]] * 4)
    r = {n: t.cuda() for n, t in rule_inputs([1] * 4, 4, 2, 64, 64, "bf16", 4, 43).items()}
    r["src"] = ints([0, 1, 2, 3])
    out = dict(rule=torch.empty(4, 4, 64, dtype=torch.bfloat16, device="cuda"),
               attention=torch.empty_like(d["q"]))
    return x, d, r, out, (d["pages"], d["length"], ref.cuda())


def test_serving_step_in_a_graph(gpu_lib):
    """every replay of a captured decode step equals the eager steps"""
    x, d, r, out, P = serving_state()
    start = [t.clone() for t in (*P, r["S"], d["kc"], d["vc"])]
    want = []
    for _ in range(4):
        serving_step(gpu_lib, x, d, r, out, P)
        torch.cuda.synchronize()
        want.append([t.cpu().clone() for t in (out["rule"], out["attention"], *P, r["S"], d["kc"],
                                               d["vc"])])

    def reset():
        for t, s in zip((*P, r["S"], d["kc"], d["vc"]), start):
            t.copy_(s)

    reset()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        serving_step(gpu_lib, x, d, r, out, P)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        serving_step(gpu_lib, x, d, r, out, P)
    reset()
    torch.cuda.synchronize()
    for i in range(4):
        graph.replay()
        torch.cuda.synchronize()
        got = [t.cpu() for t in (out["rule"], out["attention"], *P, r["S"], d["kc"], d["vc"])]
        for a, b in zip(got, want[i]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i
        torch.randn(1000, device="cuda").sum().item()        # work between the replays


def test_another_stream(gpu_lib):
    """stream=: the work and its workspace run there"""
    x = attention_inputs([300, 20], 4, 4, 2, 64, 16, "bf16", 47)
    ref, mag = attention_ref(x, 0.1)
    d = {n: t.cuda() for n, t in x.items()}
    out = torch.empty_like(d["q"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        out.zero_()
        torch.cuda.synchronize()
        gpu_lib.tree_attention(d["q"], d["k"], d["v"], d["parent"], d["kc"], d["vc"], d["pages"],
                               d["length"], 0.1, out=out, stream=s)
        junk = [torch.full((1 << 20,), 9, dtype=torch.uint8, device="cuda") for _ in range(4)]
        side.synchronize()
        attention_near(out, ref, mag)
        del junk


def test_prepared_launches(gpu_lib):
    """prepare=True: the same results, call after call"""
    x = attention_inputs([77, 20], 3, 4, 2, 64, 16, "bf16", 53)
    want = attend(gpu_lib, x, 0.1)
    go = attend(gpu_lib, x, 0.1, prepare=True)
    for _ in range(3):
        go.result.zero_()
        got = go()
        torch.cuda.synchronize()
        assert torch.equal(got, want)

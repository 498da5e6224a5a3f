"""Penalties, biases and grammar masks on logits, greedy tokens of tree nodes,
and the table of counts, against plain 64-bit implementations.

Most cases take values whose every step is exact in fp32 (logits in eighths, a
repetition penalty of 2, the others in eighths): results and greedy tokens, ties
among them, are then equal to the 64-bit ones bit for bit.  With arbitrary values
the steps' roundings count: the quotient or product, freq c, its sum with pres,
the bracket and the last sum, each half a step 2^-24 of its result, and the
result's own rounding.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
INF, NAN = float("inf"), float("nan")


def ints(x):
    return torch.tensor(np.asarray(x, dtype=np.int64), dtype=torch.int32, device="cuda")


def tree(rng, n):
    return [-1] + [max(0, i - 1 - int(rng.exponential(3))) for i in range(1, n)]


def make(batch, n, V, dtype, seed, exact=True, bias=5, mask="node", slots=None, pad=0):
    rng = np.random.default_rng(seed)
    z = rng.integers(-40, 41, (batch, n, V)) / 8 if exact else rng.standard_normal((batch, n, V)) * 3
    x = dict(batch=batch, n=n, V=V, pad=pad)
    x["z"] = torch.tensor(z, dtype=torch.float32).to(DT[dtype])
    slots = batch + 2 if slots is None else slots
    x["slot"] = rng.permutation(slots)[:batch]
    c = rng.integers(0, 4, (slots, V)) * (rng.random((slots, V)) < 0.3)
    c = np.where(rng.random((slots, V)) < 0.2, c - 32768, c)
    x["counts"] = c.astype(np.int16)
    x["parent"] = np.array([tree(rng, n) for _ in range(batch)])
    x["tokens"] = rng.integers(0, max(1, V // 3), (batch, n))        # many of a kind
    some = lambda lo, hi: rng.integers(lo, hi, batch) / 8 if exact else rng.uniform(lo, hi, batch) / 8
    x["repetition"] = np.where(rng.random(batch) < 0.7, 2.0, 0.5) if exact else rng.uniform(
        0.8, 1.5, batch)
    x["presence"], x["frequency"] = some(0, 12), some(0, 6)
    tok = rng.integers(-1, min(V, 40) + 1, (batch, bias))            # several of a kind, some outside
    x["bias"] = (tok, rng.integers(-30, 31, (batch, bias)) / 8 if exact
                 else rng.standard_normal((batch, bias)))
    rows = {"node": n, "one": 1, "none": 0}[mask]
    x["mask"] = rng.integers(0, 1 << 32, (batch, rows, (V + 31) // 32), dtype=np.uint64)
    return x


def reference(x, skip=()):
    """z' and its greedy tokens in 64 bits, and the sum of the steps' sizes"""
    batch, n, V = x["batch"], x["n"], x["V"]
    out, size = x["z"].double().numpy().copy(), np.zeros((batch, n, V))
    best = np.full((batch, n), -1)
    for b in range(batch):
        row = x["counts"][x["slot"][b]].astype(np.int64) if "counts" not in skip else np.zeros(V, int)
        prompt, said = row < 0, row & 32767
        bias = np.zeros(V)
        if "bias" not in skip:
            for t, y in zip(*(y[b] for y in x["bias"])):
                if 0 <= t < V:
                    bias[t] += y
        rep, pres, freq = ((x[k][b] if k not in skip else d) for k, d in
                           (("repetition", 1.0), ("presence", 0.0), ("frequency", 0.0)))
        for i in range(n):
            c, j = said.copy(), i
            while j >= 0 and "tokens" not in skip:
                if 0 <= x["tokens"][b, j] < V:
                    c[x["tokens"][b, j]] += 1
                j = x["parent"][b, j]
            z = out[b, i]
            seen = (c > 0) | prompt
            with np.errstate(invalid="ignore", over="ignore"):
                z1 = np.where(seen, np.where(z > 0, z / rep, z * rep), z)
                less = np.where(c > 0, freq * c + pres, 0.0)
                y = z1 + (bias - less)
                size[b, i] = np.abs(z1) + np.abs(bias) + 3 * np.abs(less) + np.abs(y)
            if x["mask"].shape[1] and "mask" not in skip:
                words = x["mask"][b, i if x["mask"].shape[1] > 1 else 0]
                bits = (words[np.arange(V) // 32] >> (np.arange(V) % 32).astype(np.uint64)) & 1
                y = np.where(bits == 1, y, -INF)
            out[b, i] = y
            fine = np.where(np.isnan(y), -INF, y)
            if fine.max() > -INF:
                best[b, i] = int(np.argmax(fine == fine.max()))
    return torch.from_numpy(out), torch.from_numpy(best), torch.from_numpy(size)


def padded(t, pad):
    """t on the GPU, rows `pad` elements longer"""
    if not pad:
        return t.cuda().contiguous()
    room = torch.full((*t.shape[:-1], t.shape[-1] + pad), 3, dtype=t.dtype, device="cuda")
    room[..., : t.shape[-1]] = t.cuda()
    return room[..., : t.shape[-1]]


def upload(x, skip=()):
    f = lambda y: torch.tensor(y, dtype=torch.float32, device="cuda")
    kw = {}
    if "counts" not in skip:
        kw.update(counts=padded(torch.from_numpy(x["counts"]), x["pad"]), slot=ints(x["slot"]))
    if "tokens" not in skip:
        kw.update(tokens=ints(x["tokens"]), parent=ints(x["parent"]))
    for k in ("repetition", "presence", "frequency"):
        if k not in skip:
            kw[k] = f(x[k])
    if "bias" not in skip and x["bias"][0].shape[1]:
        kw["bias"] = (ints(x["bias"][0]), f(x["bias"][1]))
    if "mask" not in skip and x["mask"].shape[1]:
        kw["mask"] = torch.from_numpy(x["mask"].astype(np.uint32).view(np.int32)).cuda()
    return padded(x["z"], x["pad"]), kw


def same(got, ref, dtype):
    """equal to the 64-bit result, rounded once"""
    assert torch.equal(torch.isnan(got.cpu()), torch.isnan(ref))
    want = ref.to(dtype)
    ok = (got.cpu() == want) | torch.isnan(ref)
    assert ok.all(), (got.cpu()[~ok][:5], want[~ok][:5])


CASES = [
    # batch, n, V, dtype, out, mask, bias, pad
    (1, 1, 1, "fp32", "fp32", "none", 0, 0),
    (1, 1, 31, "bf16", "fp32", "one", 2, 0),
    (2, 3, 33, "fp16", "fp16", "node", 5, 0),
    (3, 4, 511, "bf16", "bf16", "node", 5, 1),
    (2, 2, 512, "bf16", "fp32", "one", 70, 0),
    (2, 5, 513, "fp32", "fp32", "node", 5, 3),
    (1, 64, 1000, "bf16", "fp32", "node", 5, 0),
    (2, 128, 1024, "fp16", "fp32", "none", 0, 8),
    (1, 128, 2049, "bf16", "bf16", "one", 130, 0),
    (5, 7, 4096, "bf16", "fp32", "node", 300, 0),
    (3, 1, 32000, "bf16", "bf16", "one", 16, 0),
    (70, 1, 5003, "fp16", "fp32", "node", 3, 0),
    (40, 33, 1536, "bf16", "fp32", "node", 9, 0),
    (300, 2, 520, "fp32", "fp32", "one", 9, 0),
    (1, 9, 100003, "bf16", "fp32", "node", 5, 5),
    (2, 17, 65544, "fp32", "fp32", "one", 5, 0),
    (3, 1, 70000, "bf16", "fp32", "none", 65, 0),
    (600, 1, 1025, "bf16", "bf16", "node", 3, 0),
]


@pytest.mark.parametrize("batch,n,V,dtype,out,mask,bias,pad", CASES)
def test_adjust_logits(gpu_lib, batch, n, V, dtype, out, mask, bias, pad):
    print("logits", batch, n, V, dtype, out, mask, bias, pad, flush=True)
    x = make(batch, n, V, dtype, 3, bias=bias, mask=mask, pad=pad)
    ref, best, _ = reference(x)
    z, kw = upload(x)
    o = padded(torch.full(z.shape, NAN, dtype=DT[out]), pad)
    st = ints([-1] * batch)
    got = gpu_lib.adjust_logits(z, out=o, status=st, **kw)
    torch.cuda.synchronize()
    assert st.tolist() == [0] * batch
    assert torch.equal(got.cpu().long(), best)
    same(o, ref, DT[out])
    if pad:
        assert (o._base[..., V:] == 3).all() and (z._base[..., V:] == 3).all()
    # the greedy tokens alone, given (checked and called natively) or not, and in place
    assert torch.equal(gpu_lib.adjust_logits(z, **kw), got)
    mine = torch.full_like(got, -7)
    assert gpu_lib.adjust_logits(z, best=mine, status=st, **kw) is mine and torch.equal(mine, got)
    again = torch.full_like(o, NAN)
    gpu_lib.adjust_logits(z, best=mine, out=again, **kw)
    same(again, ref, DT[out])
    assert gpu_lib.adjust_logits(z, out=z, best=False, **kw) is None
    same(z, ref, z.dtype)


ABSENT = ["counts", "tokens", "repetition", "presence", "frequency", "bias", "mask"]


@pytest.mark.parametrize("skip", [[a] for a in ABSENT] + [ABSENT, ["counts", "tokens"]])
def test_what_is_left_out(gpu_lib, skip):
    x = make(3, 6, 777, "bf16", 5, mask="node")
    ref, best, _ = reference(x, skip)
    z, kw = upload(x, skip)
    o = torch.empty(z.shape, device="cuda")
    got = gpu_lib.adjust_logits(z, out=o, **kw)
    assert torch.equal(got.cpu().long(), best)
    same(o, ref, torch.float32)


def test_slots_by_row(gpu_lib):
    x = make(4, 1, 600, "bf16", 7, slots=4)
    x["slot"] = np.arange(4)
    ref, best, _ = reference(x)
    z, kw = upload(x)
    del kw["slot"]
    assert torch.equal(gpu_lib.adjust_logits(z, **kw).cpu().long(), best)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_arbitrary_values(gpu_lib, dtype):
    x = make(4, 20, 3001, dtype, 9, exact=False, bias=40)
    ref, best, size = reference(x)
    z, kw = upload(x)
    o = torch.empty(z.shape, device="cuda")
    got = gpu_lib.adjust_logits(z, out=o, **kw).cpu().long()
    off = (o.cpu().double() - ref).abs()
    off[torch.isinf(ref)] = 0
    assert torch.equal(torch.isinf(o.cpu()), torch.isinf(ref))
    # the quotient is of fp32 values of the penalties: half a step of each more;
    # biases of one token (3 or fewer here) add up with a rounding each
    assert (off <= 4 * 2.0 ** -24 * size).all(), (off / size.clamp(min=1e-300)).max()
    top = ref.amax(-1)
    at = ref.gather(-1, got[..., None])[..., 0]
    slack = 8 * 2.0 ** -24 * size.amax(-1)
    assert (at >= top - slack).all()
    assert torch.equal(got, torch.where(at == top, best, got))


@pytest.mark.parametrize("spread", [40, 600, 30000])
@pytest.mark.parametrize("batch,n", [(1, 1), (3, 40)])
def test_many_biases(gpu_lib, spread, batch, n):
    """hundreds of them, on few tokens (which then add up to 20 in order) or on many"""
    x = make(batch, n, 40000, "fp32", 25, bias=300, mask="none")
    x["bias"] = (np.random.default_rng(26).integers(-2, spread, (batch, 300)), x["bias"][1])
    ref, best, _ = reference(x)
    z, kw = upload(x)
    o = torch.empty(z.shape, device="cuda")
    assert torch.equal(gpu_lib.adjust_logits(z, out=o, **kw).cpu().long(), best)
    same(o, ref, torch.float32)


def test_values_not_finite(gpu_lib):
    x = make(1, 6, 900, "bf16", 11, mask="none")
    x["z"][0, 1, 7] = INF
    x["z"][0, 2, :] = -INF
    x["z"][0, 3, 5] = NAN
    x["z"][0, 4, :] = NAN
    x["z"][0, 5, :] = -INF
    x["z"][0, 5, 640] = float(torch.finfo(torch.bfloat16).min)
    x["frequency"][:] = x["presence"][:] = 0
    x["bias"][1][:] = 0
    x["repetition"][:] = 0.5
    ref, best, _ = reference(x)
    z, kw = upload(x)
    o = torch.empty(z.shape, device="cuda")
    got = gpu_lib.adjust_logits(z, out=o, **kw)
    assert torch.equal(got.cpu().long(), best)
    assert got[0].tolist()[1] == 7 and got[0].tolist()[2] == -1 and got[0].tolist()[4:] == [-1, 640]
    same(o, ref, torch.float32)


@pytest.mark.parametrize("dtype,bits", [("bf16", 0x7f81), ("bf16", -0x7f), ("fp16", 0x7c01),
                                        ("fp32", 0x7f800001), ("fp32", -0x7fffff)])
def test_nan_of_every_kind_is_never_the_largest(gpu_lib, dtype, bits):
    """signalling ones too, at every place of a lane's eight tokens"""
    V = 1024
    z = torch.zeros(1, 8, V, dtype=DT[dtype], device="cuda")
    raw = z.view(torch.int32 if dtype == "fp32" else torch.int16)
    for i in range(8):
        z[0, i, 8 * i + (i + 3) % 8] = 3.0
        raw[0, i, 8 * i + i] = bits
        raw[0, i, 512:] = bits
    assert torch.isnan(z[0, 0, 0])
    assert gpu_lib.adjust_logits(z)[0].tolist() == [8 * i + (i + 3) % 8 for i in range(8)]


def test_masks_that_leave_nothing_or_one(gpu_lib):
    x = make(2, 4, 70, "fp32", 13, mask="node")
    x["mask"][0, 0] = 0
    x["mask"][0, 1] = 0
    x["mask"][0, 1, 2] = 1 << 5                                  # token 69, the last
    x["mask"][1, 2] = 0
    x["mask"][1, 2, 2] = 0xffffffff << 6 & 0xffffffff            # past the vocabulary
    ref, best, _ = reference(x)
    z, kw = upload(x)
    got = gpu_lib.adjust_logits(z, **kw).cpu()
    assert torch.equal(got.long(), best)
    assert got[0, :2].tolist() == [-1, 69] and got[1, 2] == -1


def test_ties_take_the_lowest_token(gpu_lib):
    for V in (64, 600, 5000, 70001):
        z = torch.zeros(1, 3, V, dtype=torch.bfloat16, device="cuda")
        z[0, 1, V // 2:] = 1
        z[0, 2, -1] = z[0, 2, V - 7] = 2
        assert gpu_lib.adjust_logits(z)[0].tolist() == [0, V // 2, V - 7]
        z[0, 0] = -0.0
        z[0, 0, 5] = 0.0                                         # equal to -0
        assert gpu_lib.adjust_logits(z)[0, 0] == 0


@pytest.mark.parametrize("dtype,bias,spread,mask,ties", [
    ("bf16", 5, 40, "node", False), ("fp16", 300, 30, "node", False), ("fp32", 300, 30000, "one", False),
    ("bf16", 5, 40, "none", True), ("fp16", 70, 13001, "node", True)])
def test_many_nodes(gpu_lib, dtype, bias, spread, mask, ties):
    """so many that a wave goes over many slices of a row, dense counts among them:
    the greedy tokens alone, and with an output, equal those in 64 bits.  With three
    values of logits the largest is there dozens of times a slice, with counts and
    without."""
    batch, n, V = 16, 128, 13001
    x = make(batch, n, V, dtype, 31, bias=bias, mask=mask)
    rng = np.random.default_rng(32)
    x["bias"] = (rng.integers(-1, spread, (batch, bias)), x["bias"][1])
    if ties:
        x["z"] = torch.from_numpy(rng.integers(-1, 2, (batch, n, V)) / 8).to(DT[dtype])
        x["repetition"][:] = 1
        x["presence"][:] = x["frequency"][:] = 0
        x["bias"][1][:] = 0
    x["z"][:, 3, 9000:] = NAN
    x["z"][:, 4, 100:] = -INF
    x["z"][:, 5, :] = -INF
    ref, best, _ = reference(x)
    z, kw = upload(x)
    got = gpu_lib.adjust_logits(z, **kw)
    assert torch.equal(got.cpu().long(), best)
    assert (got[:, 5] == -1).all()
    o = torch.empty(z.shape, dtype=torch.float32, device="cuda")
    assert torch.equal(gpu_lib.adjust_logits(z, out=o, **kw), got)
    same(o, ref, torch.float32)


@pytest.mark.parametrize("density", [0.02, 0.06, 0.3, 1.0])
@pytest.mark.parametrize("spread", [40, 13001])
def test_many_nodes_by_density(gpu_lib, density, spread):
    """few or all tokens of a slice counted, hundreds of biases, with a path and without"""
    batch, n, V = 16, 128, 13001
    x = make(batch, n, V, "bf16", 41, bias=300, mask="one")
    rng = np.random.default_rng(42)
    x["counts"] = np.where(rng.random(x["counts"].shape) < density,
                           rng.choice([1, 2, 7, -32768, -32765], x["counts"].shape), 0).astype(np.int16)
    x["bias"] = (rng.integers(-1, spread, (batch, 300)), x["bias"][1])
    for skip in ([], ["tokens"], ["counts"], ["counts", "tokens"]):
        _, best, _ = reference(x, skip)
        z, kw = upload(x, skip)
        assert torch.equal(gpu_lib.adjust_logits(z, **kw).cpu().long(), best), skip


def test_many_nodes_with_faults(gpu_lib):
    x = make(16, 128, 13001, "bf16", 33)
    x["slot"][2] = 99
    x["parent"][5, 7] = 7
    z, kw = upload(x)
    st = ints([-1] * 16)
    got = gpu_lib.adjust_logits(z, status=st, **kw)
    assert [i for i, f in enumerate(st.tolist()) if f] == [2, 5]
    assert (got[[2, 5]] == -1).all() and (got[[0, 1, 3, 4, 6]] >= 0).all()


def test_a_chain_counts_every_node_once(gpu_lib):
    """128 nodes in a row with the same token: its count is the depth + 1"""
    V = 1000
    z = torch.zeros(2, 128, V, device="cuda")
    parent = ints([list(range(-1, 127))] * 2)
    tokens = ints([[511] * 128, [512] * 64 + [-5] * 32 + [V] * 32])
    o = torch.empty_like(z)
    one = torch.ones(2, device="cuda")
    gpu_lib.adjust_logits(z, tokens=tokens, parent=parent, frequency=one, presence=one * 0.5, out=o)
    depth = torch.arange(1, 129, device="cuda")
    assert torch.equal(o[0, :, 511], -(depth + 0.5))
    assert torch.equal(o[1, :, 512], -(depth.clamp(max=64) + 0.5))
    o[0, :, 511] = o[1, :, 512] = 0
    assert not o.any()


def test_faults(gpu_lib):
    x = make(5, 6, 700, "bf16", 15)
    x["parent"][1, 3] = 3
    x["parent"][4, 2] = -2
    x["slot"][2], x["slot"][4] = 7, -1
    ref, best, _ = reference({**x, "slot": x["slot"] % 7, "parent": np.array([tree(
        np.random.default_rng(1), 6) if b in (1, 4) else p for b, p in enumerate(x["parent"])])})
    z, kw = upload(x)
    o = torch.zeros(z.shape, device="cuda")
    st = ints([-1] * 5)
    got = gpu_lib.adjust_logits(z, out=o, status=st, **kw).cpu().long()
    P, S = gpu_lib.FAULT_BAD_PARENT, gpu_lib.FAULT_BAD_SLOT
    assert st.tolist() == [0, P, S, 0, P | S]
    for b in range(5):
        if b in (0, 3):
            assert torch.equal(got[b], best[b])
            same(o[b], ref[b], torch.float32)
        else:
            assert (got[b] == -1).all() and torch.isnan(o[b]).all()


# ---------------------------------------------------------------------------
# counts
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("V,pad", [(1, 0), (31, 0), (1000, 1), (32768, 0), (70001, 3)])
def test_count_prompt(gpu_lib, V, pad):
    rng = np.random.default_rng(17)
    slots, lens = 9, [5, 0, 300, 1, 2000]
    c = rng.integers(-32768, 32768, (slots, V)).astype(np.int16)
    tokens = rng.integers(-3, V + 3, sum(lens) + 4)
    tokens[:3] = V - 1
    cu = [2 + sum(lens[:i]) for i in range(len(lens) + 1)]
    slot = [3, 0, 8, 4, 1]
    want = c.copy()
    for s, a, b in zip(slot, cu, cu[1:]):
        want[s] = 0
        want[s, [t for t in tokens[a:b] if 0 <= t < V]] = -32768
    counts = padded(torch.from_numpy(c), pad)
    st = ints([-1] * 5)
    assert gpu_lib.count_prompt(counts, ints(slot), ints(cu), ints(tokens), status=st) is counts
    torch.cuda.synchronize()
    assert st.tolist() == [0] * 5
    assert torch.equal(counts.cpu(), torch.from_numpy(want))
    if pad:
        assert (counts._base[:, V:] == 3).all()


def test_count_prompt_faults(gpu_lib):
    c = torch.full((6, 100), 9, dtype=torch.int16, device="cuda")
    st = ints([-1] * 7)
    #         fine  outside  again  outside  falls  fine  too far
    slot, cu = [2, 6, 2, -1, 4, 5, 0], [0, 3, 6, 9, 12, 10, 13, 99]
    gpu_lib.count_prompt(c, ints(slot), ints(cu), ints(list(range(20))), status=st)
    torch.cuda.synchronize()
    S, L = gpu_lib.FAULT_BAD_SLOT, gpu_lib.FAULT_BAD_LENGTH
    assert st.tolist() == [0, S, S, S, L, 0, L]
    want = torch.full((6, 100), 9, dtype=torch.int16)
    want[2] = want[5] = 0
    want[2, :3] = want[5, 10:13] = -32768
    assert torch.equal(c.cpu(), want)
    gpu_lib.count_prompt(c, ints([]), ints([0]), ints([]))       # nobody


@pytest.mark.parametrize("n,max_path,pad", [(1, 1, 0), (8, 5, 1), (64, 64, 0), (128, 128, 3),
                                            (300, 200, 0)])
def test_count_commit(gpu_lib, n, max_path, pad):
    rng = np.random.default_rng(19)
    V, slots, m = 50, 7, 5
    c = rng.integers(0, 5, (slots, V)) - 32768 * (rng.random((slots, V)) < 0.5)
    c[0, :] = 32766
    c[1, :] = -1                                                # the most, and in the prompt
    slot, add = [0, 1, 4, 2, 6], [max_path, max_path, 0, max_path // 2, max_path]
    tokens = rng.integers(-2, V + 2, (m, n))
    tokens[4] = 7
    path = rng.integers(0, n, (m, max_path))
    want = c.copy()
    for r in range(m):
        for j in range(add[r]):
            t = tokens[r, path[r, j]]
            if 0 <= t < V and want[slot[r], t] & 32767 != 32767:
                want[slot[r], t] += 1
    path[3, max_path // 2:] = -1
    counts = padded(torch.from_numpy(c.astype(np.int16)), pad)
    st = ints([-1] * m)
    assert gpu_lib.count_commit(counts, ints(slot), ints(tokens), ints(path), ints(add),
                                status=st) is counts
    torch.cuda.synchronize()
    assert st.tolist() == [0] * m
    assert torch.equal(counts.cpu().long(), torch.from_numpy(want))


def test_count_commit_faults(gpu_lib):
    c = torch.zeros(4, 30, dtype=torch.int16, device="cuda")
    st = ints([-1] * 7)
    slot, add = [1, 4, 1, 0, 2, 3, -1], [2, 2, 2, 3, -1, 2, 1]
    path = [[0, 1], [0, 1], [0, 1], [0, 1], [0, 1], [0, 5], [0, 0]]
    gpu_lib.count_commit(c, ints(slot), ints([[3, 4, 5]] * 7), ints(path), ints(add), status=st)
    torch.cuda.synchronize()
    S, P = gpu_lib.FAULT_BAD_SLOT, gpu_lib.FAULT_BAD_PATH
    assert st.tolist() == [0, S, S, P, P, P, S]
    want = torch.zeros(4, 30, dtype=torch.int16)
    want[1, 3] = want[1, 4] = 1
    assert torch.equal(c.cpu(), want)


# ---------------------------------------------------------------------------
# streams, graphs, workspaces
# ---------------------------------------------------------------------------
def test_in_a_graph_and_on_another_stream(gpu_lib):
    """a round's end: counts of the accepted branch, the next greedy tokens"""
    x = make(3, 8, 5000, "bf16", 21)
    z, kw = upload(x)
    path, add = ints([[0, 1, 2, -1]] * 3), ints([3, 0, 1])
    table, best = kw["counts"], ints(np.zeros((3, 8)))

    def step(counts, out):
        gpu_lib.count_commit(counts, kw["slot"], kw["tokens"], path, add)
        return gpu_lib.adjust_logits(z, best=out, **{**kw, "counts": counts})

    step(table.clone(), best)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(table, best)
    s = torch.cuda.Stream()
    for i in range(4):
        z.copy_(z.roll(i + 1, -1))
        eager = table.clone()
        want = step(eager, None)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(best, want) and torch.equal(table, eager)
        other = gpu_lib.adjust_logits(z, stream=s, **kw)
        s.synchronize()
        assert torch.equal(other, want)


def test_given_workspace_and_prepared(gpu_lib):
    x = make(2, 3, 150000, "fp16", 23)
    z, kw = upload(x)
    want = gpu_lib.adjust_logits(z, **kw)
    room = torch.full((1 << 16,), 255, dtype=torch.uint8, device="cuda")
    launch = gpu_lib.adjust_logits(z, workspace=room, prepare=True, **kw)
    for _ in range(3):
        room.fill_(255)
        assert torch.equal(launch(), want)
    need = gpu_lib.load().gdn_adjust_logits_workspace(2, 3, 150000)
    assert 0 < need <= room.numel()
    with pytest.raises(gpu_lib.GdnError):
        gpu_lib.adjust_logits(z, workspace=room[:need - 1], **kw)


def test_native_calls_leave_the_unusual_to_python(gpu_lib):
    """None, and nothing written, for every argument out of order"""
    native = gpu_lib._native()
    z = torch.randn(2, 3, 100, device="cuda").bfloat16()
    c = torch.zeros(4, 100, dtype=torch.int16, device="cuda")
    slot, six, one = ints([0, 1]), ints([[1, 2, 3]] * 2), torch.ones(2, device="cuda")
    parent, mask = ints([[-1, 0, 1]] * 2), ints(np.zeros((2, 1, 4)))
    best, room = ints([[7] * 3] * 2), torch.empty(64, dtype=torch.uint8, device="cuda")
    good = [z, c, slot, six, parent, one, one, one, six, torch.ones(2, 3, device="cuda"), mask, None,
            best, None, None, room]

    def refused(call, args, at, value):
        x = list(args)
        x[at] = value
        assert call(*x) is None, (at, value if not torch.is_tensor(value) else value.shape)

    for at, value in (
            (0, None), (0, z.cpu()), (0, z[0]), (0, z.double()), (0, z[..., ::2]), (0, z[:1]),
            (0, z[..., :99]), (1, None), (1, c[:, :99]), (1, c.int()), (1, c[0]), (2, slot[:1]),
            (2, slot.long()), (3, None), (3, six[:1]), (4, None), (4, parent.cpu()), (5, one[:1]),
            (6, one.double()), (7, one.cpu()), (8, None), (8, six[0]), (9, six.float()[:1]), (9, six),
            (10, mask[:, 0]), (10, mask[..., :3]), (10, ints(np.zeros((2, 2, 4)))), (11, z[:1]),
            (11, z.half()), (11, z.double()), (12, None), (12, best[:1]), (12, best.long()),
            (13, slot[:1]), (14, "s"), (15, None), (15, room.int())):
        refused(native.logits_call, good, at, value)
    torch.cuda.synchronize()
    assert (best == 7).all()
    assert native.logits_call(*good) == 0
    torch.cuda.synchronize()
    assert (best == -1).all()
    cu, tok = ints([0, 2, 3]), ints([1, 2, 3])
    good = [c, slot, cu, tok, None, None]
    for at, value in ((0, None), (0, c.int()), (0, c[0]), (1, slot[None]), (1, slot.cpu()), (2, cu[:2]),
                      (3, tok.long()), (3, None), (4, slot[:1]), (5, "s")):
        refused(native.count_prompt_call, good, at, value)
    path = ints([[0, 1]] * 2)
    commit = [c, slot, six, path, slot, None, None]
    for at, value in ((0, c.int()), (1, slot[None]), (2, six[0]), (2, six[:1]), (3, path[:1]),
                      (3, path.cpu()), (4, slot[:1]), (5, slot[:1]), (6, "s")):
        refused(native.count_commit_call, commit, at, value)
    torch.cuda.synchronize()
    assert not c.any()
    assert native.count_prompt_call(*good) == 0 and native.count_commit_call(*commit) == 0
    torch.cuda.synchronize()
    assert c.any()

"""The serving operators at the edges of their contracts: values that are not
finite at the end of a shared part, groups whose members differ in length,
weights far below a row's largest, requests that cannot be served, caches whose
strides say nothing.  Plain 64-bit implementations and tolerances as in
test_gpu_serving.py.
"""
import numpy as np
import pytest
import torch

from test_gpu_serving import (DT, Pages, attend, attention_inputs, attention_near, attention_ref,
                              gen, half_step, ints)

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def group(first, last, tokens):
    return ints([first, last]), ints([tokens])


def cell(x, b, t):
    """page and offset of sequence b's token t"""
    page = x["kc"].shape[2]
    return int(x["pages"][b, t // page]), t % page


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("shared,lengths,n,dtype", [
    (96, [100, 100], 1, "bf16"), (144, [150, 160, 150], 3, "fp16"), (200, [200, 200], 2, "bf16"),
    (33, [40, 40], 1, "bf16"), (128, [130, 130], 1, "bf16"), (90, [90, 64, 77], 2, "bf16"),
])
def test_values_not_finite_at_the_end_of_a_shared_part(gpu_lib, shared, lengths, n, dtype):
    """they reach every row that sees them, wherever the shared part ends"""
    print("shared", shared, lengths, n, dtype, flush=True)
    x = attention_inputs(lengths, n, 4, 2, 64, 16, dtype, 61, [(0, len(lengths), shared)])
    ref, mag = attention_ref(x, 0.1)
    for t, col, value in ((shared - 1, 5, INF), (max(0, shared - 1) // 64 * 64, 9, NAN),
                          (shared // 2, 13, -INF)):
        page, off = cell(x, 0, t)
        x["vc"][page, :, off, col] = value
        ref[[b for b, L in enumerate(lengths) if L > t], ..., col] = value
    got = attend(gpu_lib, x, 0.1, shared=group(0, len(lengths), shared)).cpu()
    torch.cuda.synchronize()
    for col in (5, 9, 13):
        assert torch.equal(torch.isnan(got[..., col]), torch.isnan(ref[..., col])), col
        for sign in (INF, -INF):
            assert torch.equal(got[..., col] == sign, ref[..., col] == sign), col
    fine = torch.isfinite(ref)
    assert torch.isfinite(got[fine]).all()
    attention_near(got[fine], ref[fine], mag[fine])


def test_values_not_finite_under_weights_that_are_zero(gpu_lib):
    """scores of -inf give weights of exactly zero, and 0 * inf is NaN: also
    where they fill a part of the softmax by themselves"""
    x = attention_inputs([200, 200], 1, 4, 2, 64, 16, "bf16", 67, [(0, 2, 144)])
    x["q"][..., 0] = 1.0
    for t in range(128, 144):
        page, off = cell(x, 0, t)
        x["kc"][page, :, off, 0] = -INF
    ref, mag = attention_ref(x, 0.1)
    page, off = cell(x, 0, 131)
    x["vc"][page, :, off, 5] = INF
    got = attend(gpu_lib, x, 0.1, shared=group(0, 2, 144)).cpu()
    assert not torch.isfinite(got[..., 5]).any()
    cols = [c for c in range(64) if c != 5]
    attention_near(got[..., cols], ref[..., cols], mag[..., cols])


def test_values_not_finite_beside_a_member_that_does_not_fit(gpu_lib):
    """a member whose length passes its table does not hide what the others see"""
    x = attention_inputs([200, 200, 200], 2, 4, 2, 64, 16, "bf16", 71, [(0, 3, 128)])
    ref, mag = attention_ref(x, 0.1)
    page, off = cell(x, 0, 70)
    x["vc"][page, :, off, 5] = INF
    for length in (100000, -3):
        x["length"][2] = length
        st = ints([-1] * 3)
        got = attend(gpu_lib, x, 0.1, shared=group(0, 3, 128), status=st).cpu()
        assert st.tolist() == [0, 0, gpu_lib.FAULT_BAD_LENGTH]
        assert torch.isnan(got[2]).all()
        assert (got[:2, ..., 5] == INF).all(), length
        cols = [c for c in range(64) if c != 5]
        attention_near(got[:2][..., cols], ref[:2][..., cols], mag[:2][..., cols])


SHORT = [
    # lengths, n, page, groups
    ([50, 130], 1, 16, [(0, 2, 128)]),                    # the first member is short
    ([0, 130, 131], 3, 16, [(0, 3, 128)]),                # and empty
    ([130, 50, 200, 0, 200], 2, 16, [(0, 5, 192)]),       # the longest is in the middle, twice
    ([40, 60], 1, 16, [(0, 2, 128)]),                     # nobody has the whole of it
    ([0, 0], 4, 32, [(0, 2, 64)]),
    ([10, 70, 30, 300, 290], 1, 8, [(0, 2, 64), (2, 5, 280)]),
    ([5] + [300] * 70, 1, 16, [(0, 71, 256)]),            # rows over several units
]


@pytest.mark.parametrize("lengths,n,page,groups", SHORT)
def test_groups_with_members_shorter_than_the_shared_part(gpu_lib, lengths, n, page, groups):
    """entries past a length are not read, whichever member it is"""
    print("short members", lengths[:6], n, page, groups, flush=True)
    x = attention_inputs(lengths, n, 8, 2, 64, page, "bf16", 73, groups)
    for b, L in enumerate(lengths):
        x["pages"][b, -(-L // page):] = -1
    ref, mag = attention_ref(x, 0.125)
    st = ints([-1] * len(lengths))
    shared = (ints([groups[0][0]] + [g[1] for g in groups]), ints([g[2] for g in groups]))
    got = attend(gpu_lib, x, 0.125, shared=shared, status=st)
    torch.cuda.synchronize()
    assert st.tolist() == [0] * len(lengths)
    attention_near(got, ref, mag)


def test_short_members_with_other_pages(gpu_lib):
    """a member is held against the longest one, within its own tokens"""
    x = attention_inputs([30, 130, 70], 1, 2, 1, 64, 16, "bf16", 79, [(0, 3, 128)])
    x["pages"][0, 2:] = -1
    x["pages"][2, 4] = (x["pages"][2, 4] + 1) % x["kc"].shape[0]
    ref, mag = attention_ref({n: torch.nan_to_num(t) if n in ("kc", "vc") else t
                              for n, t in x.items()}, 0.125)
    st = ints([-1] * 3)
    got = attend(gpu_lib, x, 0.125, shared=group(0, 3, 128), status=st)
    torch.cuda.synchronize()
    assert st.tolist() == [0, 0, gpu_lib.FAULT_BAD_GROUP]
    assert torch.isnan(got[2]).all()
    attention_near(got[:2], ref[:2], mag[:2])


@pytest.mark.parametrize("below", [25.3, 30.0])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_keys_far_below_the_largest(gpu_lib, below, dtype):
    """every 32nd key is large and has no value, the others are 2^-below of it.
    fp16 weights are relative to 2^12 at least, so that one is off by half a
    step of its own or by 2^-25 / 2^12 of the largest, 31 of them to each
    large one."""
    x = attention_inputs([4096], 1, 1, 1, 64, 128, dtype, 83)
    for n in ("q", "kc", "k"):
        x[n].zero_()
    x["vc"].copy_((torch.nan_to_num(x["vc"]).abs() + 0.5) * 4096)
    x["q"][..., 0] = below * np.log(2) / 4
    x["kc"][:, :, ::32, 0] = 4
    x["vc"][:, :, ::32] = 0
    ref, mag = attention_ref(x, 1.0)
    got = attend(gpu_lib, x, 1.0).cpu()
    floor = 32 * 2.0 ** -37 * float(x["vc"].max()) if dtype == "fp16" else 0.0
    h = half_step(DT[dtype])
    tol = h * ref.abs() + (h + 1e-4) * mag + floor + torch.finfo(DT[dtype]).smallest_normal * h
    off = (got.double() - ref).abs()
    assert (off <= tol).all(), ((off / tol).max().item(), ref.max(), got.max())


def loose(t, *dims):
    """t, with strides that mean nothing in the given dimensions of size one"""
    strides = list(t.stride())
    for i in dims:
        assert t.shape[i] == 1
        strides[i] = 24
    return t.as_strided(t.shape, strides)


@pytest.mark.parametrize("Hkv,page,dims", [(1, 16, (1,)), (2, 1, (2,)), (1, 1, (1, 2))])
def test_strides_of_dimensions_of_one(gpu_lib, Hkv, page, dims):
    x = attention_inputs([33, 5], 2, 2, Hkv, 64, page, "bf16", 89)
    d = {n: t.cuda() for n, t in x.items()}
    want = attend(gpu_lib, x, 0.1)
    odd = {n: loose(d[n], *dims) for n in ("kc", "vc")}
    got = gpu_lib.tree_attention(d["q"], d["k"], d["v"], d["parent"], odd["kc"], odd["vc"],
                                 d["pages"], d["length"], 0.1)
    assert torch.equal(got, want)
    plain = [d["kc"].clone(), d["vc"].clone()]
    args = (d["pages"], ints([0, 1]), ints([3, 0]), d["k"], d["v"], ints([[0, 1], [1, 1]]),
            ints([2, 1]))
    gpu_lib.kv_commit(*plain, *args)
    gpu_lib.kv_commit(odd["kc"], odd["vc"], *args)
    for a, b in zip(plain, (d["kc"], d["vc"])):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


# ---------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------
def test_page_free_changes_nothing_for_a_bad_row(gpu_lib):
    """an id outside the pool, or a page that nobody is counted for: the row,
    its length and every count stay, and a repaired row is freed whole"""
    rng = np.random.default_rng(5)
    P = Pages(rng, 6, 4, 20, 4, {0: 10, 1: 16, 2: 3, 3: 9, 4: 8})
    kept = P.table.copy()
    P.table[1, 2] = 25                                   # outside the pool
    P.table[3, 1] = -1
    P.table[4, 1] = int(np.argmax(P.ref == 0))           # free
    table, length, ref = P.up()
    st = ints([-1] * 8)
    done = [0, 1, 3, 1, 4, 0, 2, 5]
    gpu_lib.page_free(table, length, ref, ints(done), 4, status=st)
    P.release([0, 2])
    torch.cuda.synchronize()
    bad = gpu_lib.FAULT_BAD_PAGE
    assert st.tolist() == [0, bad, bad, bad, bad, 0, 0, 0]
    P.same(table, length, ref)
    for r in (1, 3, 4):
        P.table[r] = kept[r]
    table.copy_(ints(P.table.tolist()))
    gpu_lib.page_free(table, length, ref, ints(done), 4, status=st)
    P.release([1, 3, 4])
    torch.cuda.synchronize()
    assert st.tolist() == [0] * 8 and not ref.any()
    P.same(table, length, ref)


def test_page_free_many_named_twice(gpu_lib):
    """rows that share pages, each named twice: every count goes down once"""
    rng = np.random.default_rng(6)
    P = Pages(rng, 600, 30, 100, 4, {s: 100 for s in range(3)})
    table, length, ref = P.up()
    src, dst = [i % 3 for i in range(3, 600)], list(range(3, 600))
    gpu_lib.page_fork(table, length, ref, ints(src), ints(dst), 4)
    P.fork(src, dst)
    P.same(table, length, ref)
    done = [int(x) for x in rng.permutation(600)[:500]]
    st = ints([-1] * 1000)
    gpu_lib.page_free(table, length, ref, ints(done + done[::-1]), 4, status=st)
    P.release(done)
    assert st.tolist() == [0] * 1000
    P.same(table, length, ref)


def test_page_fork_from_a_row_of_the_same_call(gpu_lib):
    """a row that an earlier request of the call writes cannot be read; one
    that a later request writes is read as it was, empty"""
    rng = np.random.default_rng(8)
    P = Pages(rng, 10, 4, 20, 4, {0: 10, 1: 16})
    table, length, ref = P.up()
    src, dst = [0, 4, 7, 1, 5], [4, 5, 6, 7, 8]
    st = ints([-1] * 5)
    copies = gpu_lib.page_fork(table, length, ref, ints(src), ints(dst), 4, status=st)
    want = P.fork([0, 1], [4, 7])
    torch.cuda.synchronize()
    bad = gpu_lib.FAULT_BAD_SLOT
    assert st.tolist() == [0, bad, 0, 0, bad]
    assert copies.tolist() == [want[0], [-1, -1], [-1, -1], want[1], [-1, -1]]
    P.same(table, length, ref)


def test_page_extend_totals_past_32_bits(gpu_lib):
    """requests for whole rows of half a million pages: more than 2^31 pages
    are asked for, 100 are there"""
    seqs, width = 4096, (1 << 19) + 1
    table = torch.empty(seqs, width, dtype=torch.int32, device="cuda")      # 8 GiB
    table[:3] = -1
    length = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    ref = ints([0] * 100)
    add = torch.full((seqs,), width, dtype=torch.int32, device="cuda")
    add[0], add[1] = 50, 30
    st = torch.full((seqs,), -1, dtype=torch.int32, device="cuda")
    begin = gpu_lib.page_extend(table, length, ref, torch.arange(seqs, dtype=torch.int32,
                                                                 device="cuda"), add, 1, status=st)
    torch.cuda.synchronize()
    none = gpu_lib.FAULT_NO_PAGE
    assert st.tolist() == [0, 0] + [none] * (seqs - 2)
    assert begin.tolist() == [0, 0] + [-1] * (seqs - 2)
    assert length.tolist() == [50, 30] + [0] * (seqs - 2)
    assert table[0, :51].tolist() == list(range(50)) + [-1]
    assert table[1, :31].tolist() == list(range(50, 80)) + [-1]
    assert (table[2] == -1).all() and ref.tolist() == [1] * 80 + [0] * 20


def test_page_copy_of_a_single_page(gpu_lib):
    """a pool of one page, whose stride says nothing: nothing to copy"""
    cache = torch.randn(2, 1, 4, 8, device="cuda")
    odd = cache.as_strided(cache.shape, (32, 3, 8, 1))
    assert odd.is_contiguous()
    want = cache.clone()
    assert gpu_lib.page_copy(odd, ints([[0, 0], [-1, -1]])) is odd
    torch.cuda.synchronize()
    assert torch.equal(cache, want)

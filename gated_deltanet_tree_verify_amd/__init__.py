"""Rollback-free tree verification and commit for Gated DeltaNet on MI355X.

Thin Python binding over the C ABI of libgdntree.so (include/gdn_tree.h).
Every function here only marshals arguments: it checks torch tensors, takes
their device pointers and the current HIP stream, and calls the entry point
of the same name.  All computation runs in the library's HIP kernels; there
is no CPU or PyTorch fallback, and a missing library raises.

    verify(q, k, v, alpha, beta, parent, S0)        -> out   (gdn_tree_verify)
    branch_verify(q, k, v, alpha, beta, parent, S0) -> out   (gdn_branch_verify, baseline)
    commit(S, path, path_len, k, v, alpha, beta, parent)     (gdn_tree_commit, in place)
    commit_verify(S, path, path_len, prev, q, k, v, alpha, beta, parent)
                                                    -> out   (gdn_tree_commit_verify)
    build_tree(cand_logp, cand_tok, root_tok, width, max_depth)
                                                    -> (parent, token, score, n_built)
    accept(parent, draft_tok, verify_tok)           -> (accepted, accept_len, bonus_tok)
    path(parent, accepted, max_path)                -> (path, path_len)
    index(parent)                                   -> (depth, anc)

Serving operators next to the tree calls:

    prefill(q, k, v, alpha, beta, cu, S, src, dst)  -> out   (gdn_prefill)
    step(q, k, v, alpha, beta, S, src, dst)         -> out   (gdn_step)
    tree_attention(q, k, v, parent, k_cache, v_cache, pages, length, scale)
                                                    -> out   (gdn_tree_attention)
    page_fork(table, length, ref, src, dst, page)   -> copies
    page_extend(table, length, ref, dst, add, page) -> begin
    page_free(table, length, ref, done, page)
    page_compact(table, length, ref, page)          -> (copies, count)
    page_copy(cache, copies, count)
    kv_commit(k_cache, v_cache, table, dst, begin, k, v, path, add)
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

__all__ = ["load", "lib_path", "verify", "branch_verify", "commit", "commit_verify", "build_tree", "accept", "path", "Launch", "index", "status_string",
           "prefill", "step", "tree_attention", "page_fork", "page_extend", "page_free",
           "page_compact", "page_copy", "kv_commit",
           "FAULT_BAD_SLOT", "FAULT_BAD_LENGTH", "FAULT_BAD_PAGE", "FAULT_BAD_GROUP",
           "FAULT_NO_PAGE",
           "GdnError", "FAULT_BAD_PARENT", "FAULT_BAD_PATH", "DTYPE_F32", "DTYPE_BF16",
           "MAX_NODES", "MAX_DIM", "ABI_VERSION", "build"]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libgdntree.so"

FAULT_BAD_PARENT = 1
FAULT_BAD_PATH = 2
FAULT_BAD_SLOT = 4
FAULT_BAD_LENGTH = 8
FAULT_BAD_PAGE = 16
FAULT_BAD_GROUP = 32
FAULT_NO_PAGE = 64
DTYPE_F32 = 0
DTYPE_BF16 = 1
DTYPE_F16 = 2     # pseudo-values of commit_verify, tree_attention
MAX_NODES = 128
MAX_DIM = 128
MAX_CANDIDATES = 32
# GDN_TREE_ABI_VERSION of include/gdn_tree.h that the signatures below follow
ABI_VERSION = 9

_lock = threading.Lock()
_lib = None


class GdnError(RuntimeError):
    """A negative gdn_status returned by the library."""

    def __init__(self, fn: str, code: int, text: str):
        super().__init__(f"{fn}: {text} (status {code})")
        self.code = code


def lib_path() -> str:
    return os.path.join(_PKG, _LIB_NAME)


def build(verbose: bool = False) -> str:
    """Compile libgdntree.so in-tree (hipcc, gfx950)."""
    from . import _build as _b
    return _b.build(verbose=verbose)


def load() -> ctypes.CDLL:
    """Load libgdntree.so from the package directory (raises if absent)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = lib_path()
        if not os.path.exists(p):
            raise RuntimeError(f"{p} is not built; run gated_deltanet_tree_verify_amd.build()")
        lib = ctypes.CDLL(p)
        P, I = ctypes.c_void_p, ctypes.c_int
        lib.gdn_tree_verify.argtypes = [P, P, P, I, P, P, P, P, P, I, I, I, I, I, P, P]
        lib.gdn_tree_verify.restype = I
        lib.gdn_branch_verify.argtypes = [P, P, P, I, P, P, P, P, P, I, I, I, I, I, P, P]
        lib.gdn_branch_verify.restype = I
        lib.gdn_tree_commit.argtypes = [P, P, P, I, P, P, I, P, P, P, I, I, I, I, I, P, P]
        lib.gdn_tree_commit.restype = I
        lib.gdn_tree_commit_verify.argtypes = [P, P, P, I, P, P, P, P, P, P, I, P, P, P, I, P, P,
                                               P, P, P, I, I, I, I, I, I, P, P]
        lib.gdn_tree_commit_verify.restype = I
        lib.gdn_tree_build.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, P]
        lib.gdn_tree_build.restype = I
        lib.gdn_tree_accept.argtypes = [P, P, P, P, P, P, I, I, P, P]
        lib.gdn_tree_accept.restype = I
        lib.gdn_tree_path.argtypes = [P, P, P, P, I, I, I, P, P]
        lib.gdn_tree_path.restype = I
        lib.gdn_tree_index.argtypes = [P, P, P, I, I, P, P]
        lib.gdn_tree_index.restype = I
        L, F = ctypes.c_int64, ctypes.c_float
        lib.gdn_prefill_workspace.argtypes = [I] * 7
        lib.gdn_prefill_workspace.restype = L
        lib.gdn_prefill.argtypes = [P, P, P, I, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, P, L,
                                    P, P]
        lib.gdn_step.argtypes = [P, P, P, I, P, P, P, P, P, P, I, I, I, I, I, I, I, P, P]
        lib.gdn_tree_attention_workspace.argtypes = [I] * 8
        lib.gdn_tree_attention_workspace.restype = L
        lib.gdn_tree_attention.argtypes = [P, P, P, I, P, P, P, L, P, P, P, P, I, F, P, I, I, I, I,
                                           I, I, I, I, P, L, P, P]
        lib.gdn_page_fork.argtypes = [P, P, P, P, P, P, I, I, I, I, I, P, P]
        lib.gdn_page_extend.argtypes = [P, P, P, P, P, P, I, I, I, I, I, P, P]
        lib.gdn_page_free.argtypes = [P, P, P, P, I, I, I, I, I, P, P]
        lib.gdn_page_compact.argtypes = [P, P, P, P, P, P, I, I, I, I, P]
        lib.gdn_page_copy.argtypes = [P, P, P, I, I, I, L, P]
        lib.gdn_kv_commit.argtypes = [P, P, L, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, I,
                                      P, P]
        for fn in (lib.gdn_prefill, lib.gdn_step, lib.gdn_tree_attention, lib.gdn_page_fork,
                   lib.gdn_page_extend, lib.gdn_page_free, lib.gdn_page_compact,
                   lib.gdn_page_copy, lib.gdn_kv_commit):
            fn.restype = I
        lib.gdn_status_string.argtypes = [I]
        lib.gdn_status_string.restype = ctypes.c_char_p
        lib.gdn_tree_abi_version.argtypes = []
        lib.gdn_tree_abi_version.restype = I
        got = lib.gdn_tree_abi_version()
        if got != ABI_VERSION:
            raise RuntimeError(f"{p} has ABI version {got}, this binding expects {ABI_VERSION}; "
                               "rebuild with gated_deltanet_tree_verify_amd.build()")
        _lib = lib
        return lib


def status_string(code: int) -> str:
    return load().gdn_status_string(int(code)).decode()


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------
_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


_native_module = None


def _native():
    """csrc/binding.cpp: argument checks and calls of the serving operators"""
    global _native_module
    if _native_module is None:
        load()
        _torch()
        try:
            from . import _binding
        except ImportError as e:
            raise RuntimeError("the binding's native part cannot be loaded; run "
                               "gated_deltanet_tree_verify_amd.build()") from e
        got = getattr(_binding, "ABI_VERSION", None)
        if got != ABI_VERSION:
            raise RuntimeError(f"the binding's native part has ABI version {got}, this package "
                               f"expects {ABI_VERSION}; rebuild with "
                               "gated_deltanet_tree_verify_amd.build()")
        _binding.explain(_explain)
        _native_module = _binding
    return _native_module


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    torch = _torch()
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn, code):
    if code != 0:
        raise GdnError(fn, code, status_string(code))


class Launch:
    """One entry-point call with its arguments already checked and marshalled
    (device pointers, sizes, stream).  Calling it re-issues the same launch
    with no per-call checks, for launch loops where those checks would cost
    more host time than the kernel takes on the GPU.  It keeps references to
    its tensors; `result` is what the eager call returns."""

    __slots__ = ("_fn", "_name", "_args", "_keep", "result")

    def __init__(self, name, fn, args, keep, result):
        self._name, self._fn, self._args, self._keep, self.result = name, fn, args, keep, result

    def __call__(self):
        rc = self._fn(*self._args)
        if rc != 0:
            _check(self._name, rc)
        return self.result


def _issue(name, fn, args, keep, result, prepare):
    if prepare:
        return Launch(name, fn, args, keep, result)
    _check(name, fn(*args))
    return result


def _explain(t, name, dtypes, shape=None):
    """raises what is wrong with an argument"""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _need(t, name, dtypes, shape=None):
    """a contiguous GPU tensor of one of the dtypes, of this shape if given;
    from the first call on this name is the native check itself.  The tree
    calls need libgdntree.so alone: without the native part they are checked
    in Python (the serving operators ask for it first, and raise)."""
    global _need
    try:
        _need = _native().need
    except RuntimeError:
        load()
        _need = _explain
    _need(t, name, dtypes, shape)


def _qkv_dtype(q):
    torch = _torch()
    return DTYPE_BF16 if q.dtype == torch.bfloat16 else DTYPE_F32


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------
def _verify_like(name, q, k, v, alpha, beta, parent, S0, out, status, stream, prepare):
    torch = _torch()
    lib = load()
    qk = (torch.bfloat16, torch.float32)
    _need(q, "q", qk)
    batch, n, H, dk = q.shape
    _need(k, "k", (q.dtype,), q.shape)
    _need(v, "v", (q.dtype,))
    if tuple(v.shape[:3]) != (batch, n, H):
        raise ValueError("v must be [batch][n][H][d_v]")
    dv = v.shape[3]
    _need(alpha, "alpha", (torch.float32,), (batch, n, H))
    _need(beta, "beta", (torch.float32,), (batch, n, H))
    _need(parent, "parent", (torch.int32,), (batch, n))
    _need(S0, "S0", (torch.float32,), (batch, H, dk, dv))
    if out is None:
        out = torch.empty((batch, n, H, dv), dtype=torch.float32, device=q.device)
    _need(out, "out", (torch.float32,), (batch, n, H, dv))
    if status is not None:
        _need(status, "status", (torch.int32,), (batch,))
    args = (_ptr(q), _ptr(k), _ptr(v), _qkv_dtype(q), _ptr(alpha), _ptr(beta), _ptr(parent),
            _ptr(S0), _ptr(out), batch, n, H, dk, dv, _ptr(status), _stream(stream))
    return _issue(name, getattr(lib, name), args,
                  (q, k, v, alpha, beta, parent, S0, out, status), out, prepare)


def verify(q, k, v, alpha, beta, parent, S0, out=None, status=None, stream=None, prepare=False):
    """gdn_tree_verify: fp32 out [batch][n][H][d_v]; S0 is never written.
    prepare=True returns a Launch instead of launching."""
    return _verify_like("gdn_tree_verify", q, k, v, alpha, beta, parent, S0, out, status, stream,
                        prepare)


def branch_verify(q, k, v, alpha, beta, parent, S0, out=None, status=None, stream=None,
                  prepare=False):
    """gdn_branch_verify: the single-branch recurrent baseline, same result
    as verify()."""
    return _verify_like("gdn_branch_verify", q, k, v, alpha, beta, parent, S0, out, status,
                        stream, prepare)


def commit(S, path, path_len, k, v, alpha, beta, parent, status=None, stream=None,
           prepare=False):
    """gdn_tree_commit: advances S [batch][H][d_k][d_v] in place; returns S.
    prepare=True returns a Launch instead of launching."""
    torch = _torch()
    lib = load()
    _need(k, "k", (torch.bfloat16, torch.float32))
    batch, n, H, dk = k.shape
    _need(v, "v", (k.dtype,))
    dv = v.shape[3]
    _need(S, "S", (torch.float32,), (batch, H, dk, dv))
    _need(path, "path", (torch.int32,))
    if path.dim() != 2 or path.shape[0] != batch:
        raise ValueError("path must be [batch][max_path]")
    _need(path_len, "path_len", (torch.int32,), (batch,))
    _need(alpha, "alpha", (torch.float32,), (batch, n, H))
    _need(beta, "beta", (torch.float32,), (batch, n, H))
    _need(parent, "parent", (torch.int32,), (batch, n))
    if status is not None:
        _need(status, "status", (torch.int32,), (batch,))
    args = (_ptr(S), _ptr(path), _ptr(path_len), int(path.shape[1]), _ptr(k), _ptr(v),
            _qkv_dtype(k), _ptr(alpha), _ptr(beta), _ptr(parent), batch, n, H, dk, dv,
            _ptr(status), _stream(stream))
    return _issue("gdn_tree_commit", lib.gdn_tree_commit, args,
                  (S, path, path_len, k, v, alpha, beta, parent, status), S, prepare)


def commit_verify(S, path, path_len, prev, q, k, v, alpha, beta, parent, out=None,
                  status=None, stream=None, prepare=False, u_prev=None, u_out=None):
    """gdn_tree_commit_verify: commit the previous tree's accepted path into S
    (in place), then verify the new tree from the committed S.

    prev = (k_prev, v_prev, alpha_prev, beta_prev, parent_prev): the tensors
    of the tree the path was accepted from.  u_out ([batch][n][H][d_v], fp32
    or fp16) receives the new tree's pseudo-values; u_prev, the previous
    call's u_out on this same S (same dtype), lets the commit skip its
    solve.  Returns out [batch][n][H][d_v] (prepare=True: a Launch instead
    of launching).
    """
    torch = _torch()
    lib = load()
    k_prev, v_prev, alpha_prev, beta_prev, parent_prev = prev
    qk = (torch.bfloat16, torch.float32)
    _need(q, "q", qk)
    batch, n, H, dk = q.shape
    _need(k, "k", (q.dtype,), q.shape)
    _need(v, "v", (q.dtype,))
    if tuple(v.shape[:3]) != (batch, n, H):
        raise ValueError("v must be [batch][n][H][d_v]")
    dv = v.shape[3]
    _need(alpha, "alpha", (torch.float32,), (batch, n, H))
    _need(beta, "beta", (torch.float32,), (batch, n, H))
    _need(parent, "parent", (torch.int32,), (batch, n))
    _need(k_prev, "k_prev", (q.dtype,))
    if k_prev.dim() != 4 or k_prev.shape[0] != batch or tuple(k_prev.shape[2:]) != (H, dk):
        raise ValueError("k_prev must be [batch][n_prev][H][d_k]")
    n_prev = k_prev.shape[1]
    _need(v_prev, "v_prev", (q.dtype,), (batch, n_prev, H, dv))
    _need(alpha_prev, "alpha_prev", (torch.float32,), (batch, n_prev, H))
    _need(beta_prev, "beta_prev", (torch.float32,), (batch, n_prev, H))
    _need(parent_prev, "parent_prev", (torch.int32,), (batch, n_prev))
    udt = (torch.float32, torch.float16)
    if u_prev is not None:
        _need(u_prev, "u_prev", udt, (batch, n_prev, H, dv))
    _need(S, "S", (torch.float32,), (batch, H, dk, dv))
    _need(path, "path", (torch.int32,))
    if path.dim() != 2 or path.shape[0] != batch:
        raise ValueError("path must be [batch][max_path]")
    _need(path_len, "path_len", (torch.int32,), (batch,))
    if out is None:
        out = torch.empty((batch, n, H, dv), dtype=torch.float32, device=q.device)
    _need(out, "out", (torch.float32,), (batch, n, H, dv))
    if u_out is not None:
        _need(u_out, "u_out", udt, (batch, n, H, dv))
    if u_prev is not None and u_out is not None and u_prev.dtype != u_out.dtype:
        raise ValueError("u_prev and u_out must share a dtype")
    u_given = u_out if u_out is not None else u_prev
    u_dtype = DTYPE_F16 if (u_given is not None and u_given.dtype == torch.float16) else 0
    if status is not None:
        _need(status, "status", (torch.int32,), (batch,))
    args = (_ptr(S), _ptr(path), _ptr(path_len), int(path.shape[1]), _ptr(k_prev),
            _ptr(v_prev), _ptr(alpha_prev), _ptr(beta_prev), _ptr(parent_prev), _ptr(u_prev),
            n_prev, _ptr(q), _ptr(k), _ptr(v), _qkv_dtype(q), _ptr(alpha), _ptr(beta),
            _ptr(parent), _ptr(out), _ptr(u_out), u_dtype, batch, n, H, dk, dv, _ptr(status),
            _stream(stream))
    return _issue("gdn_tree_commit_verify", lib.gdn_tree_commit_verify, args,
                  (S, path, path_len, *prev, u_prev, q, k, v, alpha, beta, parent, out, u_out,
                   status), out, prepare)


def build_tree(cand_logp, cand_tok, root_tok, width, max_depth, stream=None, prepare=False):
    """gdn_tree_build: (parent, token, score, n_built) from a candidate table
    cand_logp fp32 [batch][n][K], cand_tok int32 [batch][n][K]; root_tok
    int32 [batch] or None."""
    torch = _torch()
    lib = load()
    _need(cand_logp, "cand_logp", (torch.float32,))
    if cand_logp.dim() != 3:
        raise ValueError("cand_logp must be [batch][n][K]")
    batch, n, K = cand_logp.shape
    _need(cand_tok, "cand_tok", (torch.int32,), (batch, n, K))
    if root_tok is not None:
        _need(root_tok, "root_tok", (torch.int32,), (batch,))
    dev = cand_logp.device
    parent = torch.empty((batch, n), dtype=torch.int32, device=dev)
    token = torch.empty((batch, n), dtype=torch.int32, device=dev)
    score = torch.empty((batch, n), dtype=torch.float32, device=dev)
    n_built = torch.empty((batch,), dtype=torch.int32, device=dev)
    args = (_ptr(cand_logp), _ptr(cand_tok), _ptr(root_tok), _ptr(parent), _ptr(token),
            _ptr(score), _ptr(n_built), batch, n, K, int(width), int(max_depth), _stream(stream))
    return _issue("gdn_tree_build", lib.gdn_tree_build, args,
                  (cand_logp, cand_tok, root_tok, parent, token, score, n_built),
                  (parent, token, score, n_built), prepare)


def accept(parent, draft_tok, verify_tok, status=None, stream=None, prepare=False):
    """gdn_tree_accept: (accepted, accept_len, bonus_tok), int32 [batch] each."""
    torch = _torch()
    lib = load()
    _need(parent, "parent", (torch.int32,))
    batch, n = parent.shape
    _need(draft_tok, "draft_tok", (torch.int32,), (batch, n))
    _need(verify_tok, "verify_tok", (torch.int32,), (batch, n))
    acc = torch.empty((batch,), dtype=torch.int32, device=parent.device)
    alen = torch.empty((batch,), dtype=torch.int32, device=parent.device)
    bonus = torch.empty((batch,), dtype=torch.int32, device=parent.device)
    if status is not None:
        _need(status, "status", (torch.int32,), (batch,))
    args = (_ptr(parent), _ptr(draft_tok), _ptr(verify_tok), _ptr(acc), _ptr(alen), _ptr(bonus),
            batch, n, _ptr(status), _stream(stream))
    return _issue("gdn_tree_accept", lib.gdn_tree_accept, args,
                  (parent, draft_tok, verify_tok, acc, alen, bonus, status), (acc, alen, bonus),
                  prepare)


def path(parent, accepted, max_path, out=None, path_len=None, status=None, stream=None,
         prepare=False):
    """gdn_tree_path: (path int32 [batch][max_path], path_len int32 [batch])."""
    torch = _torch()
    lib = load()
    _need(parent, "parent", (torch.int32,))
    batch, n = parent.shape
    _need(accepted, "accepted", (torch.int32,), (batch,))
    if out is None:
        out = torch.empty((batch, max_path), dtype=torch.int32, device=parent.device)
    if path_len is None:
        path_len = torch.empty((batch,), dtype=torch.int32, device=parent.device)
    _need(out, "path", (torch.int32,), (batch, max_path))
    _need(path_len, "path_len", (torch.int32,), (batch,))
    if status is not None:
        _need(status, "status", (torch.int32,), (batch,))
    args = (_ptr(parent), _ptr(accepted), _ptr(out), _ptr(path_len), batch, n, int(max_path),
            _ptr(status), _stream(stream))
    return _issue("gdn_tree_path", lib.gdn_tree_path, args,
                  (parent, accepted, out, path_len, status), (out, path_len), prepare)


def index(parent, status=None, stream=None):
    """gdn_tree_index: (depth int32 [batch][n], anc int32 bit patterns [batch][n][ceil(n/32)])."""
    torch = _torch()
    lib = load()
    _need(parent, "parent", (torch.int32,))
    batch, n = parent.shape
    W = (n + 31) // 32
    depth = torch.empty((batch, n), dtype=torch.int32, device=parent.device)
    anc = torch.empty((batch, n, W), dtype=torch.int32, device=parent.device)
    if status is not None:
        _need(status, "status", (torch.int32,), (batch,))
    rc = lib.gdn_tree_index(_ptr(parent), _ptr(depth), _ptr(anc), batch, n, _ptr(status),
                            _stream(stream))
    _check("gdn_tree_index", rc)
    return depth, anc


# ---------------------------------------------------------------------------
# serving operators
# ---------------------------------------------------------------------------
@functools.lru_cache(maxsize=1024)
def _workspace_bytes(name, *sizes):
    return max(16, int(getattr(load(), name)(*sizes)))


def _empty(shape, dtype, device, stream):
    """Device memory from torch's allocator, ordered on the current stream:
    where the call runs on another one, that waits for whatever may have used
    the block just before, and keeps the block until it is done with it."""
    torch = _torch()
    t = torch.empty(shape, dtype=dtype, device=device)
    if stream is not None:
        other = torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream
        other.wait_stream(torch.cuda.current_stream(device))
        t.record_stream(other)
    return t


def _rule_shapes(q, k, v, alpha, beta, S, src, dst, out, batch, status, stream):
    torch = _torch()
    _need(q, "q", (torch.bfloat16, torch.float32))
    if q.dim() != 3:
        raise ValueError("q must be [rows][key heads][d_k]")
    rows, Hk, dk = q.shape
    _need(k, "k", (q.dtype,), q.shape)
    _need(v, "v", (q.dtype,))
    if v.dim() != 3 or v.shape[0] != rows:
        raise ValueError("v must be [rows][heads][d_v]")
    H, dv = v.shape[1], v.shape[2]
    if batch is None:
        batch = rows
    _need(alpha, "alpha", (torch.float32,), (rows, H))
    _need(beta, "beta", (torch.float32,), (rows, H))
    _need(S, "S", (torch.float32,))
    if S.dim() != 4 or tuple(S.shape[1:]) != (H, dk, dv):
        raise ValueError("S must be [slots][heads][d_k][d_v]")
    _need(src, "src", (torch.int32,), (batch,))
    _need(dst, "dst", (torch.int32,), (batch,))
    if out is None:
        out = _empty((rows, H, dv), q.dtype, q.device, stream)
    _need(out, "out", (torch.bfloat16, torch.float32), (rows, H, dv))
    if status is not None:
        _need(status, "status", (torch.int32,), (batch,))
    return rows, Hk, dk, H, dv, out


def prefill(q, k, v, alpha, beta, cu, S, src, dst, out=None, status=None, stream=None,
            workspace=None, prepare=False):
    """gdn_prefill: the gated delta rule over the prompts of a ragged batch.

    q, k [rows][Hk][d_k], v [rows][H][d_v] (bf16 or fp32), alpha, beta
    [rows][H] fp32; sequence i owns rows cu[i] .. cu[i+1] (cu int32
    [batch + 1], on the GPU).  It starts from state slot src[i] of S
    [slots][H][d_k][d_v] (-1: zero) and leaves its state in slot dst[i].
    Returns out [rows][H][d_v] (bf16 or fp32, q's type by default); S is
    updated in place.  workspace: a uint8 tensor of prefill_workspace bytes;
    one is allocated when None.  prepare=True returns a Launch.
    """
    torch = _torch()
    native = _native()
    _need(cu, "cu", (torch.int32,))
    if cu.dim() != 1 or cu.shape[0] < 2:
        raise ValueError("cu must be [batch + 1]")
    batch = cu.shape[0] - 1
    rows, Hk, dk, H, dv, out = _rule_shapes(q, k, v, alpha, beta, S, src, dst, out, batch, status,
                                        stream)
    dt = _qkv_dtype(q)
    need = _workspace_bytes("gdn_prefill_workspace", dt, batch, rows, H, Hk, dk, dv)
    if workspace is None:
        workspace = _empty(need, torch.uint8, q.device, stream)
    else:
        _need(workspace, "workspace", (torch.uint8,))
    args = (q, k, v, dt, alpha, beta, cu, S, src,
            dst, out, _qkv_dtype(out), batch, rows, S.shape[0], H, Hk, dk, dv,
            workspace, workspace.numel(), status, _stream(stream))
    return _issue("gdn_prefill", native.gdn_prefill, args,
                  (q, k, v, alpha, beta, cu, S, src, dst, out, workspace, status), out, prepare)


def step(q, k, v, alpha, beta, S, src, dst, out=None, status=None, stream=None, prepare=False):
    """gdn_step: one token for every sequence (row i: sequence i); arguments
    as for prefill without cu.  Returns out; S is updated in place."""
    native = _native()
    rows, Hk, dk, H, dv, out = _rule_shapes(q, k, v, alpha, beta, S, src, dst, out, None,
                                            status, stream)
    args = (q, k, v, _qkv_dtype(q), alpha, beta, S, src,
            dst, out, _qkv_dtype(out), rows, S.shape[0], H, Hk, dk, dv, status,
            _stream(stream))
    return _issue("gdn_step", native.gdn_step, args,
                  (q, k, v, alpha, beta, S, src, dst, out, status), out, prepare)


def _need_cache(k_cache, v_cache, dtypes, Hkv, d):
    """Caches [pages][Hkv][page][d] whose pages are contiguous (the stride
    between pages is free); returns (pages, page, page stride)."""
    native = _native()
    got = native.cache(k_cache, dtypes, Hkv, d)
    if got is None or native.cache(v_cache, dtypes, Hkv, d) != got:
        _explain_caches(k_cache, v_cache, dtypes, Hkv, d)
    return got


def _explain_caches(k_cache, v_cache, dtypes, Hkv, d):
    torch = _torch()
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor")
        if t.dtype not in dtypes:
            raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
        if t.dim() != 4 or t.shape[1] != Hkv or t.shape[3] != d:
            raise ValueError(f"{name} must be [pages][{Hkv}][page][{d}]")
        if any(t.shape[i] != 1 and t.stride(i) != s
               for i, s in ((1, t.shape[2] * d), (2, d), (3, 1))):
            raise ValueError(f"the pages of {name} must be contiguous")
    raise ValueError("k_cache and v_cache must have the same pages and strides")


def tree_attention(q, k, v, parent, k_cache, v_cache, pages, length, scale, shared=None, out=None,
                   status=None, stream=None, workspace=None, prepare=False):
    """gdn_tree_attention: softmax attention of a draft tree (n = 1: one
    token) over a paged cache and the tree's own ancestors.

    q [batch][n][Hq][d], k, v [batch][n][Hkv][d] (bf16 or fp16); parent int32
    [batch][n]; k_cache, v_cache [pages][Hkv][page][d]; pages int32
    [batch][max_pages]; length int32 [batch].  shared = (start [groups + 1],
    tokens [groups]), int32: sequences start[g] .. start[g+1]-1 have their
    first tokens[g] tokens in the same pages, which are then read once for
    all of them.  Returns out [batch][n][Hq][d].  prepare=True: a Launch.
    """
    torch = _torch()
    native = _native()
    _need(q, "q", (torch.bfloat16, torch.float16))
    if q.dim() != 4:
        raise ValueError("q must be [batch][n][Hq][d]")
    batch, n, Hq, d = q.shape
    _need(k, "k", (q.dtype,))
    if k.dim() != 4 or k.shape[0] != batch or k.shape[1] != n or k.shape[3] != d:
        raise ValueError("k must be [batch][n][Hkv][d]")
    Hkv = k.shape[2]
    _need(v, "v", (q.dtype,), k.shape)
    _need(parent, "parent", (torch.int32,), (batch, n))
    num, page, stride = _need_cache(k_cache, v_cache, (q.dtype,), Hkv, d)
    _need(pages, "pages", (torch.int32,))
    if pages.dim() != 2 or pages.shape[0] != batch:
        raise ValueError("pages must be [batch][max_pages]")
    _need(length, "length", (torch.int32,), (batch,))
    start = tokens = None
    groups = 0
    if shared is not None:
        start, tokens = shared
        _need(tokens, "shared tokens", (torch.int32,))
        groups = tokens.numel()
        _need(tokens, "shared tokens", (torch.int32,), (groups,))
        _need(start, "group starts", (torch.int32,), (groups + 1,))
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    _need(out, "out", (q.dtype,), q.shape)
    if status is not None:
        _need(status, "status", (torch.int32,), (batch,))
    width = pages.shape[1]
    need = _workspace_bytes("gdn_tree_attention_workspace", batch, n, Hq, Hkv, d, page, width,
                            groups)
    if workspace is None:
        workspace = _empty(need, torch.uint8, q.device, stream)
    else:
        _need(workspace, "workspace", (torch.uint8,))
    args = (q, k, v, DTYPE_BF16 if q.dtype == torch.bfloat16 else DTYPE_F16,
            parent, k_cache, v_cache, stride, pages, length,
            start, tokens, groups, float(scale), out, batch, n, Hq, Hkv, d, page,
            num, width, workspace, workspace.numel(), status, _stream(stream))
    return _issue("gdn_tree_attention", native.gdn_tree_attention, args,
                  (q, k, v, parent, k_cache, v_cache, pages, length, start, tokens, out, workspace,
                   status), out, prepare)


def _need_table(table, length, ref):
    torch = _torch()
    _need(table, "table", (torch.int32,))
    if table.dim() != 2:
        raise ValueError("table must be [seqs][max_pages]")
    _need(length, "length", (torch.int32,), (table.shape[0],))
    _need(ref, "ref", (torch.int32,))
    if ref.dim() != 1:
        raise ValueError("ref must be [pool]")
    return table.shape[0], table.shape[1], ref.shape[0]


def page_fork(table, length, ref, src, dst, page, copies=None, status=None, stream=None,
              prepare=False):
    """gdn_page_fork: the empty rows dst become continuations of the rows src
    of the page table; returns copies int32 [m][2], the partial pages that
    page_copy has to move ({-1, -1}: none)."""
    torch = _torch()
    native = _native()
    seqs, width, pool = _need_table(table, length, ref)
    _need(src, "src", (torch.int32,))
    m = src.numel()
    _need(dst, "dst", (torch.int32,), src.shape)
    if copies is None:
        copies = _empty((m, 2), torch.int32, table.device, stream)
    _need(copies, "copies", (torch.int32,), (m, 2))
    if status is not None:
        _need(status, "status", (torch.int32,), (m,))
    args = (table, length, ref, src, dst, copies, m, seqs,
            width, pool, int(page), status, _stream(stream))
    return _issue("gdn_page_fork", native.gdn_page_fork, args,
                  (table, length, ref, src, dst, copies, status), copies, prepare)


def page_extend(table, length, ref, dst, add, page, begin=None, status=None, stream=None,
                prepare=False):
    """gdn_page_extend: room for add[r] more tokens in row dst[r]; returns
    begin int32 [m], the lengths before (-1: not enough free pages)."""
    torch = _torch()
    native = _native()
    seqs, width, pool = _need_table(table, length, ref)
    _need(dst, "dst", (torch.int32,))
    m = dst.numel()
    _need(add, "add", (torch.int32,), dst.shape)
    if begin is None:
        begin = _empty(dst.shape, torch.int32, dst.device, stream)
    _need(begin, "begin", (torch.int32,), dst.shape)
    if status is not None:
        _need(status, "status", (torch.int32,), (m,))
    args = (table, length, ref, dst, add, begin, m, seqs,
            width, pool, int(page), status, _stream(stream))
    return _issue("gdn_page_extend", native.gdn_page_extend, args,
                  (table, length, ref, dst, add, begin, status), begin, prepare)


def page_free(table, length, ref, done, page, status=None, stream=None, prepare=False):
    """gdn_page_free: the rows `done` give their pages back and become empty."""
    torch = _torch()
    native = _native()
    seqs, width, pool = _need_table(table, length, ref)
    _need(done, "done", (torch.int32,))
    if status is not None:
        _need(status, "status", (torch.int32,), (done.numel(),))
    args = (table, length, ref, done, done.numel(), seqs, width, pool,
            int(page), status, _stream(stream))
    return _issue("gdn_page_free", native.gdn_page_free, args, (table, length, ref, done, status),
                  None, prepare)


def page_compact(table, length, ref, page, copies=None, count=None, workspace=None, stream=None,
                 prepare=False):
    """gdn_page_compact: the used pages become the lowest ids (table and ref
    follow); returns (copies int32 [pool // 2][2], count int32 []): what
    page_copy has to move."""
    torch = _torch()
    native = _native()
    seqs, width, pool = _need_table(table, length, ref)
    if copies is None:
        copies = _empty((pool // 2, 2), torch.int32, table.device, stream)
    _need(copies, "copies", (torch.int32,), (pool // 2, 2))
    if count is None:
        count = _empty((), torch.int32, table.device, stream)
    _need(count, "count", (torch.int32,), ())
    if workspace is None:
        workspace = _empty(4 * pool, torch.uint8, table.device, stream)
    _need(workspace, "workspace", (torch.uint8,))
    if workspace.numel() < 4 * pool:
        raise ValueError("workspace must hold 4 bytes for every page of the pool")
    args = (table, length, ref, copies, count, workspace, seqs,
            width, pool, int(page), _stream(stream))
    return _issue("gdn_page_compact", native.gdn_page_compact, args,
                  (table, length, ref, copies, count, workspace), (copies, count), prepare)


def page_copy(cache, copies, count=None, stream=None, prepare=False):
    """gdn_page_copy: cache [planes][pool][...], page `to` <- page `from` in
    every plane for the first count (default: all) of copies [m][2]."""
    torch = _torch()
    native = _native()
    _need(cache, "cache", (torch.bfloat16, torch.float16, torch.float32, torch.uint8))
    if cache.dim() < 3:
        raise ValueError("cache must be [planes][pool][...]")
    _need(copies, "copies", (torch.int32,))
    if copies.dim() != 2 or copies.shape[1] != 2:
        raise ValueError("copies must be [m][2]")
    if count is not None:
        _need(count, "count", (torch.int32,))
        if count.numel() != 1:
            raise ValueError("count must hold one number")
    planes, pool = cache.shape[0], cache.shape[1]
    nbytes = cache.element_size()              # of a page; a pool of one may have any stride
    for n in cache.shape[2:]:
        nbytes *= n
    args = (cache, copies, count, copies.shape[0], planes, pool, nbytes,
            _stream(stream))
    return _issue("gdn_page_copy", native.gdn_page_copy, args, (cache, copies, count), cache, prepare)


def kv_commit(k_cache, v_cache, table, dst, begin, k, v, path, add, status=None, stream=None,
              prepare=False):
    """gdn_kv_commit: the accepted branches' key and value rows (rows
    path[r][: add[r]] of k, v [m][n][Hkv][d]) become tokens begin[r] .. of the
    table's rows dst[r]."""
    torch = _torch()
    native = _native()
    kinds = (torch.bfloat16, torch.float16, torch.float32)
    _need(k, "k", kinds)
    if k.dim() != 4:
        raise ValueError("k must be [m][n][Hkv][d]")
    m, n, Hkv, d = k.shape
    _need(v, "v", (k.dtype,), k.shape)
    num, page, stride = _need_cache(k_cache, v_cache, (k.dtype,), Hkv, d)
    _need(table, "table", (torch.int32,))
    if table.dim() != 2:
        raise ValueError("table must be [seqs][max_pages]")
    _need(dst, "dst", (torch.int32,), (m,))
    _need(begin, "begin", (torch.int32,), (m,))
    _need(add, "add", (torch.int32,), (m,))
    _need(path, "path", (torch.int32,))
    if path.dim() != 2 or path.shape[0] != m:
        raise ValueError("path must be [m][max_path]")
    if status is not None:
        _need(status, "status", (torch.int32,), (m,))
    args = (k_cache, v_cache, stride, table, dst, begin, k,
            v, path, add, m, n, path.shape[1], Hkv, d, k.element_size(),
            table.shape[0], table.shape[1], num, page, status, _stream(stream))
    return _issue("gdn_kv_commit", native.gdn_kv_commit, args,
                  (k_cache, v_cache, table, dst, begin, k, v, path, add, status), None, prepare)

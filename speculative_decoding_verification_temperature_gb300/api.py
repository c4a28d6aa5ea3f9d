"""Thin torch binding over libsdverify.so (the C ABI of include/sd_verify.h).

Only argument marshalling happens here: shapes and dtypes are checked, raw
device pointers and the current CUDA stream are passed through ctypes, and
outputs are allocated with torch.  Every step of the verify path runs in the
library's CUDA kernels; there is no other implementation behind these
functions, and they raise if the library cannot be loaded.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

SD_OK, SD_ERR_INVALID_ARG, SD_ERR_UNSUPPORTED, SD_ERR_CUDA = 0, 1, 2, 3
SD_F32, SD_BF16, SD_F16 = 0, 1, 2
DEV_BAD_TOKEN, DEV_NONFINITE, DEV_BAD_PARENT, DEV_ZERO_MASS = 1, 2, 4, 8
DEV_TIMEOUT = 16
DEV_BAD_LENGTH, DEV_BAD_PAGE, DEV_BAD_POSITION = 32, 64, 128

_lock = threading.Lock()
_lib = None
_get_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


class SdError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__("sd_verify error %d: %s" % (code, msg))
        self.code = code


def lib() -> ctypes.CDLL:
    """Load libsdverify.so (compiling it first if it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            # SDV_LIB selects another build of the same library
            path = os.environ.get("SDV_LIB") or _build.build()
            if not os.path.exists(path):
                raise RuntimeError("libsdverify.so is missing: run "
                                   "__graft_entry__.build()")
            L = ctypes.CDLL(path)
            _declare(L)
            _lib = L
    return _lib


def _declare(L):
    P, I, F, D, Z = (ctypes.c_void_p, ctypes.c_int, ctypes.c_float,
                     ctypes.c_double, ctypes.c_size_t)
    LL = ctypes.c_longlong
    sig = {
        "sd_version": ([], ctypes.c_char_p),
        "sd_last_error": ([], ctypes.c_char_p),
        "sd_verify_linear_workspace": ([I, I, I, I], Z),
        "sd_verify_linear": ([P, P, I, P, P, I, I, I, F, P, P, P, P, P, P, P,
                              Z, P], I),
        "sd_verify_kcand_workspace": ([I, I, I, I, I], Z),
        "sd_verify_kcand": ([P, P, I, P, P, I, I, I, I, F, P, P, P, P, P, P,
                             P, Z, P], I),
        "sd_verify_kcand_trie_workspace": ([I, I, I, I, I], Z),
        "sd_verify_kcand_trie": ([P, P, I, P, P, I, I, I, I, F, P, P, P, P,
                                  P, P, Z, P], I),
        "sd_presto_init": ([I, I, I, P, P, P, P, P, P, P], I),
        "sd_presto_expand_workspace": ([I, I, I, I, I], Z),
        "sd_presto_expand": ([P, ctypes.c_longlong, P, I, I, I, I, F, F, I,
                              I, P, P, P, P, P, P, P, P, Z, P], I),
        "sd_branch_fork_workspace": ([I, I, I, I], Z),
        "sd_branch_fork": ([P, I, P, I, I, F, I, P, P, P, P, Z, P], I),
        "sd_verify_tree_workspace": ([I, I, I, I], Z),
        "sd_verify_tree": ([P, P, I, P, P, P, I, I, I, F, P, P, P, P, P, P,
                            Z, P], I),
        "sd_verify_tree_det_workspace": ([I, I, I, I], Z),
        "sd_verify_tree_det": ([P, I, P, P, P, I, I, I, F, P, P, P, P, P, P,
                                Z, P], I),
        "sd_fanout_schedule": ([I, I, D, D, P], I),
        "sd_fanout_topk_workspace": ([I, I, I, I], Z),
        "sd_fanout_topk": ([P, I, I, I, I, P, P, P, P, P, Z, P], I),
        "sd_verify_linear_static": ([P, P, I, P, P, I, I, I, F, P, P, P, P,
                                     P, P, P], I),
        "sd_fanout_hits": ([P, P, P, I, I, P, P, P], I),
        "sd_verify_linear_filtered_workspace": ([I, I, I, I], Z),
        "sd_verify_linear_filtered": ([P, P, I, P, P, I, I, I, F, I, F, P, P,
                                       P, P, P, P, Z, P], I),
        "sd_verify_linear_fanout_workspace": ([I, I, I, I], Z),
        "sd_verify_linear_fanout": ([P, P, I, P, P, I, I, I, F, P, P, P, P,
                                     P, P, P, P, Z, P], I),
        "sd_kv_append": ([P, P, LL, P, LL, P, LL, I, P, P, P, P, I, I, I, I,
                          I, P, P, P], I),
        "sd_paged_attention_workspace": ([I, I, I, I], Z),
        "sd_paged_attention": ([P, LL, I, P, P, P, P, I, I, I, I, F, P, P, P,
                                P, Z, P], I),
        "sd_distill_topk": ([P, LL, I, P, P, P, I, I, I, F, P, P, P, P], I),
        "sd_distill_topk_backward": ([P, LL, I, P, P, P, P, P, I, I, I, F, P,
                                      LL, P, P], I),
        "sd_distill_topk_step": ([P, LL, I, P, P, P, P, I, I, I, F, P, P, P,
                                  LL, P, P], I),
        "sd_tune_set": ([I, I], I),
        "sd_selftest_bounded_wait": ([I, P, P, P], I),
        "sd_tune_get": ([I], I),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res


def version() -> str:
    return lib().sd_version().decode()


TUNE = {"cluster": 0, "no_tma": 1, "allrows": 2, "spec": 3, "fused": 4,
        "kcand_ring": 5, "fanout_cluster": 6, "fanout_ldg": 7,
        "fanout_maxc": 8, "fanout_l2_first": 9, "helpers": 10}
"""Tuning switches of sd_tune_set, by name (see include/sd_verify.h)."""


def tune_get(name: str) -> int:
    return lib().sd_tune_get(TUNE[name])


def tune_set(name: str, value: int) -> None:
    _check(lib().sd_tune_set(TUNE[name], int(value)))


class tuned:
    """Context manager: set tuning switches (name=value) for the block and
    restore the previous values after it."""

    def __init__(self, **switches):
        self.switches = switches

    def __enter__(self):
        self.saved = {k: tune_get(k) for k in self.switches}
        for k, v in self.switches.items():
            tune_set(k, v)
        return self

    def __exit__(self, *exc):
        for k, v in self.saved.items():
            tune_set(k, v)
        return False


def _check(rc):
    if rc != SD_OK:
        raise SdError(rc, lib().sd_last_error().decode())


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SD_F32
    if t.dtype == torch.bfloat16:
        return SD_BF16
    raise TypeError("logits must be float32 or bfloat16, got %s" % t.dtype)


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dev(t, device, name, dtype=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (there is no CPU path)"
                         % name)
    if t.device != device:
        raise ValueError("%s must live on %s" % (name, device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s" % (name, dtype))
    return t


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _raw_stream(device):
    """The current stream's handle (without a Stream object around it where
    torch has a call for that: 2 us less)."""
    if _get_raw_stream is not None and device.index is not None:
        return _get_raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


class Workspace:
    """Scratch buffers of the calls that need one (work-queue counters, the
    records and partial sums that one kernel of a call leaves to the next).

    Each device, stream and host thread has its own, so calls on several
    streams or from several threads share nothing; the default that calls
    without ``workspace`` use is one of these.  A buffer that becomes too
    small is kept beside the larger one, so that a captured CUDA graph never
    writes to memory that something else has.  Graphs captured on one stream
    by one thread do share a buffer: give those that are replayed at the same
    time, or beside other calls on the capture's stream, a Workspace each."""

    def __init__(self):
        self._buf = {}
        self._outgrown = []

    def get(self, device, nbytes):
        key = device, _raw_stream(device), threading.get_ident()
        b = self._buf.get(key)
        if b is None or b.numel() < nbytes:
            if b is not None:  # doubled: what is kept stays below what is used
                self._outgrown.append(b)
                nbytes = max(nbytes, 2 * b.numel())
            b = torch.empty(max(nbytes, 256), dtype=torch.uint8,
                            device=device)
            self._buf[key] = b
        return b


_default_ws = Workspace()


def verify_linear(target, draft, tokens, uniforms, T, *, want_accept=False,
                  want_resid=False, status=None, workspace=None, out=None):
    """Linear verify (sd_verify_linear).

    target [B, gamma+1, V], draft [B, gamma, V] (may be None when T == 0),
    both float32 or bfloat16 on one CUDA device; tokens [B, gamma] int32;
    uniforms [B, gamma+1] float32.  Returns a dict with n [B], tokens
    [B, gamma+1], prob [B] (and accept [B, gamma], resid [B, V] on request).
    ``status``: optional int32 [1] device tensor OR-ed with SD_DEV_* bits.
    """
    dev = target.device
    _dev(target, dev, "target")
    B, G1, V = target.shape
    gamma = G1 - 1
    if draft is not None:
        _dev(draft, dev, "draft", target.dtype)
        if draft.shape[0] != B or draft.shape[2] != V or \
                draft.shape[1] != gamma:
            raise ValueError("draft must be [B, gamma, V]")
    tokens = _dev(tokens, dev, "tokens", torch.int32)
    uniforms = _dev(uniforms, dev, "uniforms", torch.float32)
    if out is None:
        out = {}
    n = out.get("n")
    if n is None:
        n = torch.empty(B, dtype=torch.int32, device=dev)
    toks = out.get("tokens")
    if toks is None:
        toks = torch.empty((B, G1), dtype=torch.int32, device=dev)
    prob = out.get("prob")
    if prob is None:
        prob = torch.empty(B, dtype=torch.float32, device=dev)
    acc = torch.empty((B, max(gamma, 1)), dtype=torch.float32,
                      device=dev) if want_accept else None
    res = torch.empty((B, V), dtype=torch.float32,
                      device=dev) if want_resid else None
    L = lib()
    nbytes = L.sd_verify_linear_workspace(B, gamma, V, _dt(target))
    ws = (workspace or _default_ws).get(dev, nbytes)
    _check(L.sd_verify_linear(
        _p(target), _p(draft), _dt(target), _p(tokens), _p(uniforms), B,
        gamma, V, float(T), _p(n), _p(toks), _p(prob), _p(acc), _p(res),
        _p(status), _p(ws), ws.numel(), _stream(dev)))
    r = {"n": n, "tokens": toks, "prob": prob}
    if want_accept:
        r["accept"] = acc[:, :gamma]
    if want_resid:
        r["resid"] = res
    return r


def verify_linear_static(target, draft, tokens, uniforms, T, *,
                         want_accept=False, status=None):
    """Linear verify with the library's static per-device scratch instead of
    a workspace (sd_verify_linear_static): same arguments and results as
    verify_linear.  Calls that overlap on the GPU race on that scratch."""
    dev = target.device
    _dev(target, dev, "target")
    B, G1, V = target.shape
    gamma = G1 - 1
    if draft is not None:
        _dev(draft, dev, "draft", target.dtype)
        if tuple(draft.shape) != (B, gamma, V):
            raise ValueError("draft must be [B, gamma, V]")
    tokens = _dev(tokens, dev, "tokens", torch.int32)
    uniforms = _dev(uniforms, dev, "uniforms", torch.float32)
    n = torch.empty(B, dtype=torch.int32, device=dev)
    toks = torch.empty((B, G1), dtype=torch.int32, device=dev)
    prob = torch.empty(B, dtype=torch.float32, device=dev)
    acc = torch.empty((B, max(gamma, 1)), dtype=torch.float32,
                      device=dev) if want_accept else None
    _check(lib().sd_verify_linear_static(
        _p(target), _p(draft), _dt(target), _p(tokens), _p(uniforms), B,
        gamma, V, float(T), _p(n), _p(toks), _p(prob), _p(acc), None,
        _p(status), _stream(dev)))
    r = {"n": n, "tokens": toks, "prob": prob}
    if want_accept:
        r["accept"] = acc[:, :gamma]
    return r


def verify_linear_filtered(target, draft, tokens, uniforms, T, top_k,
                           top_p=1.0, *, want_keep=False, status=None,
                           workspace=None):
    """Linear verify with top_k / top_p filtered sampling applied to p and q
    before the ratio (sd_verify_linear_filtered); same shapes as
    verify_linear; top_k >= V keeps every token.  Returns n, tokens, prob
    (and keep [B, 2 gamma + 1]: the kept count of each row read, -1 for the
    rest, when want_keep)."""
    dev = target.device
    _dev(target, dev, "target")
    B, G1, V = target.shape
    gamma = G1 - 1
    if draft is not None:
        _dev(draft, dev, "draft", target.dtype)
        if tuple(draft.shape) != (B, gamma, V):
            raise ValueError("draft must be [B, gamma, V]")
    tokens = _dev(tokens, dev, "tokens", torch.int32)
    uniforms = _dev(uniforms, dev, "uniforms", torch.float32)
    n = torch.empty(B, dtype=torch.int32, device=dev)
    toks = torch.empty((B, G1), dtype=torch.int32, device=dev)
    prob = torch.empty(B, dtype=torch.float32, device=dev)
    keep = torch.empty((B, 2 * gamma + 1), dtype=torch.int32,
                       device=dev) if want_keep else None
    L = lib()
    nbytes = L.sd_verify_linear_filtered_workspace(B, gamma, V, _dt(target))
    ws = (workspace or _default_ws).get(dev, nbytes)
    _check(L.sd_verify_linear_filtered(
        _p(target), _p(draft), _dt(target), _p(tokens), _p(uniforms), B,
        gamma, V, float(T), int(top_k), float(top_p), _p(n), _p(toks),
        _p(prob), _p(keep), _p(status), _p(ws), ws.numel(), _stream(dev)))
    r = {"n": n, "tokens": toks, "prob": prob}
    if want_keep:
        r["keep"] = keep
    return r


def verify_kcand(target, draft, tokens, uniforms, T, *, status=None,
                 workspace=None):
    """K-candidate verify with longest-streak selection (sd_verify_kcand).

    target [B, K, gamma+1, V], draft [B, gamma, V] shared marginals, tokens
    [B, K, gamma] int32, uniforms [B, K, gamma+1] float32.  Returns n, k,
    tokens [B, gamma+1], n_per_cand [B, K], prob."""
    dev = target.device
    _dev(target, dev, "target")
    B, K, G1, V = target.shape
    gamma = G1 - 1
    _dev(draft, dev, "draft", target.dtype)
    if tuple(draft.shape) != (B, gamma, V):
        raise ValueError("draft must be [B, gamma, V]")
    tokens = _dev(tokens, dev, "tokens", torch.int32)
    uniforms = _dev(uniforms, dev, "uniforms", torch.float32)
    n = torch.empty(B, dtype=torch.int32, device=dev)
    ks = torch.empty(B, dtype=torch.int32, device=dev)
    toks = torch.empty((B, G1), dtype=torch.int32, device=dev)
    npc = torch.empty((B, K), dtype=torch.int32, device=dev)
    prob = torch.empty(B, dtype=torch.float32, device=dev)
    L = lib()
    nbytes = L.sd_verify_kcand_workspace(B, K, gamma, V, _dt(target))
    ws = (workspace or _default_ws).get(dev, nbytes)
    _check(L.sd_verify_kcand(
        _p(target), _p(draft), _dt(target), _p(tokens), _p(uniforms), B, K,
        gamma, V, float(T), _p(n), _p(ks), _p(toks), _p(npc), _p(prob),
        _p(status), _p(ws), ws.numel(), _stream(dev)))
    return {"n": n, "k": ks, "tokens": toks, "n_per_cand": npc, "prob": prob}


def verify_kcand_trie(target, draft, tokens, uniforms, T, *, status=None,
                      workspace=None):
    """K candidates verified as one token tree (sd_verify_kcand_trie).
    Arguments as verify_kcand (draft may be None when T == 0).  Returns n,
    k (the candidate that created the last accepted node), tokens
    [B, gamma+1], prob."""
    dev = target.device
    _dev(target, dev, "target")
    B, K, G1, V = target.shape
    gamma = G1 - 1
    if draft is not None:
        _dev(draft, dev, "draft", target.dtype)
        if tuple(draft.shape) != (B, gamma, V):
            raise ValueError("draft must be [B, gamma, V]")
    tokens = _dev(tokens, dev, "tokens", torch.int32)
    uniforms = _dev(uniforms, dev, "uniforms", torch.float32)
    n = torch.empty(B, dtype=torch.int32, device=dev)
    ks = torch.empty(B, dtype=torch.int32, device=dev)
    toks = torch.empty((B, G1), dtype=torch.int32, device=dev)
    prob = torch.empty(B, dtype=torch.float32, device=dev)
    L = lib()
    nbytes = L.sd_verify_kcand_trie_workspace(B, K, gamma, V, _dt(target))
    ws = (workspace or _default_ws).get(dev, nbytes)
    _check(L.sd_verify_kcand_trie(
        _p(target), _p(draft), _dt(target), _p(tokens), _p(uniforms), B, K,
        gamma, V, float(T), _p(n), _p(ks), _p(toks), _p(prob), _p(status),
        _p(ws), ws.numel(), _stream(dev)))
    return {"n": n, "k": ks, "tokens": toks, "prob": prob}


def verify_tree(target, draft, parent, node_tokens, uniforms, T, *,
                status=None, workspace=None):
    """Token-tree verify (sd_verify_tree).  target, draft [B, N, V]; parent,
    node_tokens [B, N] int32; uniforms [B, N] float32.  Returns n, tokens
    [B, N], nodes [B, N], prob."""
    dev = target.device
    _dev(target, dev, "target")
    B, N, V = target.shape
    _dev(draft, dev, "draft", target.dtype)
    if tuple(draft.shape) != (B, N, V):
        raise ValueError("draft must be [B, N, V]")
    parent = _dev(parent, dev, "parent", torch.int32)
    node_tokens = _dev(node_tokens, dev, "node_tokens", torch.int32)
    uniforms = _dev(uniforms, dev, "uniforms", torch.float32)
    n = torch.empty(B, dtype=torch.int32, device=dev)
    toks = torch.empty((B, N), dtype=torch.int32, device=dev)
    nodes = torch.empty((B, N), dtype=torch.int32, device=dev)
    prob = torch.empty(B, dtype=torch.float32, device=dev)
    L = lib()
    nbytes = L.sd_verify_tree_workspace(B, N, V, _dt(target))
    ws = (workspace or _default_ws).get(dev, nbytes)
    _check(L.sd_verify_tree(
        _p(target), _p(draft), _dt(target), _p(parent), _p(node_tokens),
        _p(uniforms), B, N, V, float(T), _p(n), _p(toks), _p(nodes),
        _p(prob), _p(status), _p(ws), ws.numel(), _stream(dev)))
    return {"n": n, "tokens": toks, "nodes": nodes, "prob": prob}


def verify_tree_det(target, parent, node_tokens, uniforms, T, *,
                    status=None, workspace=None):
    """Token-tree verify with deterministic drafts (sd_verify_tree_det):
    child v accepted with the current p(t_v), a rejected token removed from
    p.  target [B, N, V]; the rest as verify_tree."""
    dev = target.device
    _dev(target, dev, "target")
    B, N, V = target.shape
    parent = _dev(parent, dev, "parent", torch.int32)
    node_tokens = _dev(node_tokens, dev, "node_tokens", torch.int32)
    uniforms = _dev(uniforms, dev, "uniforms", torch.float32)
    n = torch.empty(B, dtype=torch.int32, device=dev)
    toks = torch.empty((B, N), dtype=torch.int32, device=dev)
    nodes = torch.empty((B, N), dtype=torch.int32, device=dev)
    prob = torch.empty(B, dtype=torch.float32, device=dev)
    L = lib()
    nbytes = L.sd_verify_tree_det_workspace(B, N, V, _dt(target))
    ws = (workspace or _default_ws).get(dev, nbytes)
    _check(L.sd_verify_tree_det(
        _p(target), _dt(target), _p(parent), _p(node_tokens), _p(uniforms),
        B, N, V, float(T), _p(n), _p(toks), _p(nodes), _p(prob), _p(status),
        _p(ws), ws.numel(), _stream(dev)))
    return {"n": n, "tokens": toks, "nodes": nodes, "prob": prob}


class PrestoTree:
    """Device state of PRESTO trees under construction (sd_presto_init):
    node arrays [B, budget], frontier [B, W]."""

    def __init__(self, B, W, budget, device):
        if torch.device(device).type != "cuda":
            raise ValueError("PrestoTree must live on a CUDA device (there "
                             "is no CPU path)")
        self.B, self.W, self.budget = B, W, budget
        i32 = dict(dtype=torch.int32, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        self.n_nodes = torch.empty(B, **i32)
        self.parent = torch.empty((B, budget), **i32)
        self.node_tokens = torch.empty((B, budget), **i32)
        self.node_score = torch.empty((B, budget), **f32)
        self.frontier_node = torch.empty((B, W), **i32)
        self.frontier_score = torch.empty((B, W), **f32)
        _check(lib().sd_presto_init(
            B, W, budget, _p(self.n_nodes), _p(self.parent),
            _p(self.node_tokens), _p(self.node_score),
            _p(self.frontier_node), _p(self.frontier_score),
            _stream(torch.device(device))))


def presto_expand(tree, q_logits, log_rho, T, lam, b_top, *, status=None,
                  workspace=None):
    """One depth of PRESTO's beam construction (sd_presto_expand) on `tree`
    (a PrestoTree, updated in place).  q_logits [B, V] (rows may be strided,
    e.g. q[:, d] of a [B, D, V] tensor); log_rho [B, W, V] (None when
    lam == 0)."""
    dev = q_logits.device
    B, V = q_logits.shape
    if not q_logits.is_cuda or q_logits.stride(1) != 1:
        raise ValueError("q_logits must be CUDA rows with unit stride")
    if log_rho is not None:
        _dev(log_rho, dev, "log_rho", q_logits.dtype)
        if tuple(log_rho.shape) != (B, tree.W, V):
            raise ValueError("log_rho must be [B, W, V]")
    L = lib()
    nbytes = L.sd_presto_expand_workspace(B, tree.W, V, int(b_top),
                                          _dt(q_logits))
    ws = (workspace or _default_ws).get(dev, nbytes)
    _check(L.sd_presto_expand(
        _p(q_logits), q_logits.stride(0), _p(log_rho), _dt(q_logits), B,
        tree.W, V, float(T), float(lam), int(b_top), tree.budget,
        _p(tree.n_nodes), _p(tree.parent), _p(tree.node_tokens),
        _p(tree.node_score), _p(tree.frontier_node), _p(tree.frontier_score),
        _p(status), _p(ws), ws.numel(), _stream(dev)))
    return tree


def branch_fork(draft, x_b, T, k_max, *, status=None, workspace=None):
    """SpecBranch fork (sd_branch_fork): k = max(1, floor(k_max (1 -
    q(x_b)))) (capped at V) and the top-k tokens of each row.  draft
    [B, V]; x_b [B].  Returns k [B], tokens [B, k_max]."""
    dev = draft.device
    _dev(draft, dev, "draft")
    B, V = draft.shape
    x_b = _dev(x_b, dev, "x_b", torch.int32)
    k = torch.empty(B, dtype=torch.int32, device=dev)
    toks = torch.empty((B, k_max), dtype=torch.int32, device=dev)
    L = lib()
    nbytes = L.sd_branch_fork_workspace(B, V, int(k_max), _dt(draft))
    ws = (workspace or _default_ws).get(dev, nbytes)
    _check(L.sd_branch_fork(_p(draft), _dt(draft), _p(x_b), B, V, float(T),
                            int(k_max), _p(k), _p(toks), _p(status), _p(ws),
                            ws.numel(), _stream(dev)))
    return {"k": k, "tokens": toks}


def selftest_bounded_wait(polls, device="cuda"):
    """The failure-path self-test (sd_selftest_bounded_wait): a wait that
    can never complete, bounded by `polls` polls.  Returns (status word,
    threads whose wait gave up, 1 if the kernel ran to its end)."""
    dev = torch.device(device)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    out = torch.zeros(2, dtype=torch.int32, device=dev)
    _check(lib().sd_selftest_bounded_wait(int(polls), _p(st), _p(out),
                                          _stream(dev)))
    torch.cuda.synchronize(dev)
    o = out.tolist()
    return int(st.item()), o[0], o[1]


def fanout_schedule(K, budget, a, r):
    """Geometric fan-out F[0..K] (sd_fanout_schedule, host only)."""
    F = (ctypes.c_int32 * (K + 1))()
    _check(lib().sd_fanout_schedule(int(K), int(budget), float(a), float(r),
                                    ctypes.cast(F, ctypes.c_void_p)))
    return [int(x) for x in F]


def fanout_topk(draft, F, *, want_logit=False, status=None, workspace=None):
    """Top-F_k tokens per lookahead row (sd_fanout_topk).  draft [B, K+1, V];
    F a list of K+1 ints.  Returns tokens [B, sum F] (and logit)."""
    dev = draft.device
    _dev(draft, dev, "draft")
    B, K1, V = draft.shape
    F = [int(x) for x in F]
    if len(F) != K1:
        raise ValueError("F must have K+1 entries")
    Fh = (ctypes.c_int32 * K1)(*F)
    total = sum(F)
    toks = torch.empty((B, max(total, 1)), dtype=torch.int32, device=dev)
    lg = torch.empty((B, max(total, 1)), dtype=torch.float32,
                     device=dev) if want_logit else None
    L = lib()
    nbytes = L.sd_fanout_topk_workspace(B, K1 - 1, V, _dt(draft))
    ws = (workspace or _default_ws).get(dev, nbytes)
    _check(L.sd_fanout_topk(
        _p(draft), _dt(draft), B, K1 - 1, V, ctypes.cast(Fh, ctypes.c_void_p),
        _p(toks), _p(lg), _p(status), _p(ws), ws.numel(), _stream(dev)))
    r = {"tokens": toks[:, :total]}
    if want_logit:
        r["logit"] = lg[:, :total]
    return r


def fanout_hits(n, tokens, fan_tokens, F):
    """Saguaro cache hit of each sequence's verification outcome
    (sd_fanout_hits): 1 if tokens[b, n[b]] is among the F[n[b]] fan-out
    tokens of position n[b], 0 if not, -1 where n[b] < 0.  n [B], tokens
    [B, K+1] and fan_tokens [B, sum F] int32 on one CUDA device."""
    dev = n.device
    n = _dev(n, dev, "n", torch.int32)
    tokens = _dev(tokens, dev, "tokens", torch.int32)
    F = [int(x) for x in F]
    B, K1 = tokens.shape
    if len(F) != K1:
        raise ValueError("F must have K+1 entries")
    fan_tokens = _dev(fan_tokens, dev, "fan_tokens", torch.int32)
    if tuple(fan_tokens.shape) != (B, sum(F)):
        raise ValueError("fan_tokens must be [B, sum F]")
    Fh = (ctypes.c_int32 * K1)(*F)
    hit = torch.empty(B, dtype=torch.int32, device=dev)
    _check(lib().sd_fanout_hits(_p(n), _p(tokens), _p(fan_tokens), B, K1 - 1,
                                ctypes.cast(Fh, ctypes.c_void_p), _p(hit),
                                _stream(dev)))
    return hit


def verify_linear_fanout(target, draft, tokens, uniforms, T, F, *,
                         status=None, workspace=None):
    """Linear verify fused with the fan-out of the same draft logits
    (sd_verify_linear_fanout).  draft [B, gamma+1, V] (K == gamma)."""
    dev = target.device
    _dev(target, dev, "target")
    B, G1, V = target.shape
    gamma = G1 - 1
    _dev(draft, dev, "draft", target.dtype)
    if tuple(draft.shape) != (B, gamma + 1, V):
        raise ValueError("draft must be [B, gamma+1, V]")
    tokens = _dev(tokens, dev, "tokens", torch.int32)
    uniforms = _dev(uniforms, dev, "uniforms", torch.float32)
    F = [int(x) for x in F]
    if len(F) != gamma + 1:
        raise ValueError("F must have gamma+1 entries")
    Fh = (ctypes.c_int32 * (gamma + 1))(*F)
    total = sum(F)
    n = torch.empty(B, dtype=torch.int32, device=dev)
    toks = torch.empty((B, G1), dtype=torch.int32, device=dev)
    prob = torch.empty(B, dtype=torch.float32, device=dev)
    ftok = torch.empty((B, max(total, 1)), dtype=torch.int32, device=dev)
    flog = torch.empty((B, max(total, 1)), dtype=torch.float32, device=dev)
    L = lib()
    nbytes = L.sd_verify_linear_fanout_workspace(B, gamma, V, _dt(target))
    ws = (workspace or _default_ws).get(dev, nbytes)
    _check(L.sd_verify_linear_fanout(
        _p(target), _p(draft), _dt(target), _p(tokens), _p(uniforms), B,
        gamma, V, float(T), ctypes.cast(Fh, ctypes.c_void_p), _p(n),
        _p(toks), _p(prob), _p(ftok), _p(flog), _p(status), _p(ws),
        ws.numel(), _stream(dev)))
    return {"n": n, "tokens": toks, "prob": prob,
            "fan_tokens": ftok[:, :total], "fan_logit": flog[:, :total]}


class _PagedKVStruct(ctypes.Structure):
    """sd_paged_kv of include/sd_verify.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("dt", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("heads", ctypes.c_int),
                ("head_dim", ctypes.c_int),
                ("page_stride", ctypes.c_longlong),
                ("token_stride", ctypes.c_longlong),
                ("head_stride", ctypes.c_longlong),
                ("block_table", ctypes.c_void_p),
                ("max_pages", ctypes.c_int)]


_CACHE_DT = {torch.bfloat16: SD_BF16, torch.float16: SD_F16}


class PagedKV:
    """A paged cache of keys and values (sd_paged_kv).

    k, v [num_pages, page_size, heads, head_dim], bfloat16 or float16, the
    last dimension contiguous and the others strided alike in both (a
    head-major page is ``t.transpose(1, 2)`` of [num_pages, heads,
    page_size, head_dim]); block_table [B, max_pages] int32, the page of
    each page_size keys of a sequence.  The tensors are kept, not copied:
    the program may change what they hold between calls.  Other tensors want
    another PagedKV (k, v and block_table cannot be assigned)."""

    k = property(lambda self: self._k)
    v = property(lambda self: self._v)
    block_table = property(lambda self: self._block_table)

    def __init__(self, k, v, block_table):
        dev = k.device
        for t, name in ((k, "k"), (v, "v")):
            if not t.is_cuda:
                raise ValueError("%s must be a CUDA tensor (there is no CPU "
                                 "path)" % name)
            if t.dtype not in _CACHE_DT:
                raise TypeError("%s must be bfloat16 or float16, got %s" %
                                (name, t.dtype))
            if t.dim() != 4 or t.stride(3) != 1:
                raise ValueError("%s must be [pages, page_size, heads, "
                                 "head_dim] with a contiguous last dimension"
                                 % name)
        if v.device != dev or v.dtype != k.dtype or v.shape != k.shape or \
                v.stride() != k.stride():
            raise ValueError("k and v must have one device, dtype, shape and "
                             "strides")
        _dev(block_table, dev, "block_table", torch.int32)
        if block_table.dim() != 2:
            raise ValueError("block_table must be [B, max_pages]")
        self._k, self._v, self._block_table = k, v, block_table
        n, page, heads, dim = k.shape
        self.B, self.heads, self.head_dim = block_table.shape[0], heads, dim
        self.device, self.dtype = dev, k.dtype
        self._struct = _PagedKVStruct(
            k.data_ptr(), v.data_ptr(), _CACHE_DT[k.dtype], n, page, heads,
            dim, k.stride(0), k.stride(1), k.stride(2),
            block_table.data_ptr(), block_table.shape[1])
        self._addr = ctypes.addressof(self._struct)


# The checks below look at each property once: a call on a few tokens takes
# less time on the GPU than its checks can take here.

def _rows(t, cache, name, heads=None):
    """Packed rows [total, heads, head_dim] of the cache's type, a row's
    heads contiguous; returns their number, the heads and the row stride."""
    d, shape, st = cache.head_dim, t.shape, t.stride()
    if t.dtype is cache.dtype and t.device == cache.device and \
            len(shape) == 3 and shape[2] == d and st[2] == 1:
        n, h, _ = shape
        if (st[1] == d or h == 1) and (h == heads or heads is None):
            return n, h, st[0] if n > 1 else h * d
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (there is no CPU path)"
                         % name)
    if t.device != cache.device:
        raise ValueError("%s must live on %s" % (name, cache.device))
    if t.dtype != cache.dtype:
        raise TypeError("%s must be %s" % (name, cache.dtype))
    raise ValueError("%s must be [total, %s, %d] with a row's heads "
                     "contiguous" % (name, heads or "heads", d))


def _vec(t, device, dtype, name):
    """A contiguous tensor of this type and device; returns its address."""
    if t.dtype is not dtype or t.device != device or not t.is_contiguous():
        _dev(t, device, name, dtype)
    return t.data_ptr()


def _lengths(cache, q_start, kv_len):
    qp = _vec(q_start, cache.device, torch.int32, "q_start")
    kp = _vec(kv_len, cache.device, torch.int32, "kv_len")
    B = kv_len.numel()
    if q_start.numel() != B + 1:
        raise ValueError("q_start must have one entry more than kv_len")
    if B > cache.B:
        raise ValueError("block_table has %d rows for %d sequences" %
                         (cache.B, B))
    return B, qp, kp


def _ptr(t):
    return None if t is None else t.data_ptr()


def _status(status, device):
    """The address of the status word (None without one)."""
    if status is None:
        return None
    if status.numel() < 1:
        raise ValueError("status must hold one int32")
    return _vec(status, device, torch.int32, "status")


def kv_append(cache, k, v, q_start, kv_len, *, q=None, cos_sin=None,
              positions=None, interleaved=False, status=None):
    """Append new tokens' keys and values to a PagedKV, rotated by position
    (sd_kv_append).

    k, v [total, heads, D] and q [total, q_heads, D] (optional), rows may be
    strided; q_start [B+1] and kv_len [B] int32 (kv_len counts the new
    tokens); cos_sin [max_pos, rot_dim] float32, cosines then sines (None:
    no rotation); positions [total] int32 (None: the index in the sequence).
    Returns the rotated queries (None without q)."""
    dev, D = cache.device, cache.head_dim
    total, _, ks = _rows(k, cache, "k", cache.heads)
    nv, _, vs = _rows(v, cache, "v", cache.heads)
    if nv != total:
        raise ValueError("k and v must have the same number of rows")
    B, start, lens = _lengths(cache, q_start, kv_len)
    qs = Hq = max_pos = rot = 0
    qp = op = cp = pp = out = None
    if q is not None:
        nq, Hq, qs = _rows(q, cache, "q")
        if nq != total:
            raise ValueError("q and k must have the same number of rows")
        out = torch.empty((total, Hq, D), dtype=cache.dtype, device=dev)
        qp, op = q.data_ptr(), out.data_ptr()
    if cos_sin is not None:
        cp = _vec(cos_sin, dev, torch.float32, "cos_sin")
        max_pos, rot = cos_sin.shape
    if positions is not None:
        pp = _vec(positions, dev, torch.int32, "positions")
        if positions.numel() != total:
            raise ValueError("positions must be [total]")
    rc = lib().sd_kv_append(
        cache._addr, k.data_ptr(), ks, v.data_ptr(), vs, qp, qs, Hq, start,
        lens, pp, cp, max_pos, rot, 1 if interleaved else 0, B, total, op,
        _status(status, dev), _raw_stream(dev))
    if rc != SD_OK:
        _check(rc)
    return out


def paged_attention(q, cache, q_start, kv_len, *, max_q=None, scale=None,
                    tree_mask=None, want_lse=False, status=None,
                    workspace=None):
    """Attention of a chunk of new tokens per sequence over a PagedKV
    (sd_paged_attention); their keys and values are appended before.

    q [total, q_heads, D], rows may be strided; q_start [B+1], kv_len [B]
    int32.  tree_mask [total, words] int32 (None: causal): the tokens of its
    own chunk that each token sees, as bits.  max_q: the longest chunk, a
    hint that picks the tile shape (default: the mean chunk), and with it
    whether weights are rounded to the type before they multiply the values
    (max_q x q_heads / heads above 128) or keep twice its bits.  scale
    defaults to D ** -0.5.  workspace: scratch between the call's two kernels
    (default: the current stream's and thread's own).  Returns out [total,
    q_heads, D] (and lse [total, q_heads] float32 when want_lse)."""
    dev, D = cache.device, cache.head_dim
    total, Hq, qs = _rows(q, cache, "q")
    B, start, lens = _lengths(cache, q_start, kv_len)
    words, mp = 0, None
    if tree_mask is not None:
        mp = _vec(tree_mask, dev, torch.int32, "tree_mask")
        if tree_mask.dim() != 2 or tree_mask.shape[0] != total:
            raise ValueError("tree_mask must be [total, words]")
        words = tree_mask.shape[1]
    if max_q is None:
        max_q = -(-total // max(B, 1))
    out = torch.empty((total, Hq, D), dtype=cache.dtype, device=dev)
    lse = torch.empty((total, Hq), dtype=torch.float32,
                      device=dev) if want_lse else None
    L = lib()
    nbytes = L.sd_paged_attention_workspace(Hq, cache.heads, D, max_q)
    ws = (workspace or _default_ws).get(dev, nbytes)
    rc = L.sd_paged_attention(
        q.data_ptr(), qs, Hq, cache._addr, start, lens, mp, words, B, total,
        max_q, D ** -0.5 if scale is None else scale, out.data_ptr(),
        _ptr(lse), _status(status, dev), ws.data_ptr(), ws.numel(),
        _raw_stream(dev))
    if rc != SD_OK:
        _check(rc)
    return {"out": out, "lse": lse} if want_lse else {"out": out}


_LOGIT_DT = {torch.float32: SD_F32, torch.bfloat16: SD_BF16}


def _distill_rows(student, logit, ids, lse):
    """Checks the rows; returns the arguments that every call shares."""
    dev = student.device
    if dev.type != "cuda":
        raise ValueError("student must be a CUDA tensor (there is no CPU "
                         "path)")
    shape, st = student.shape, student.stride()
    if len(shape) != 2 or st[1] != 1:
        raise ValueError("student must be [N, V] rows with unit stride")
    dt = _LOGIT_DT.get(student.dtype)
    if dt is None:
        dt = _dt(student)
    N, V = shape
    lp = _vec(logit, dev, torch.float32, "teacher_logit")
    ip = _vec(ids, dev, torch.int32, "teacher_id")
    if logit.dim() != 2 or logit.shape[0] != N or ids.shape != logit.shape:
        raise ValueError("teacher_logit and teacher_id must be [N, K]")
    tp = None if lse is None else _row_vector(lse, dev, "teacher_lse", N)
    return dev, N, V, logit.shape[1], dt, st[0] if N > 1 else V, lp, ip, tp


def _row_vector(t, dev, name, N):
    p = _vec(t, dev, torch.float32, name)
    if t.numel() != N:
        raise ValueError("%s must be [N]" % name)
    return p


def _grad_out(out, student, dev, N, V):
    """The gradient's buffer and row stride (a new one without `out`)."""
    if out is None:
        return torch.empty((N, V), dtype=student.dtype, device=dev), V
    if out.device != dev or out.dtype != student.dtype \
            or tuple(out.shape) != (N, V) or out.stride(1) != 1:
        raise ValueError("out must be [N, V] rows with unit stride, of the "
                         "student's type and device")
    return out, out.stride(0) if N > 1 else V


def distill_topk(student, teacher_logit, teacher_id, T=1.0, *,
                 teacher_lse=None, status=None):
    """KL from the target's top-K logits to the drafter's softmax
    (sd_distill_topk): student [N, V] float32 or bfloat16 (rows may be
    strided), teacher_logit [N, K] float32, teacher_id [N, K] int32 (-1:
    padding), teacher_lse [N] float32 (None: the K probabilities are
    normalised among themselves).  Returns loss [N] and lse [N] (log sum
    exp(student / T), which the backward call takes).  Neither is part of
    torch's graph: the gradient is distill_topk_backward's."""
    dev, N, V, K, dt, rs, lp, ip, tp = _distill_rows(
        student, teacher_logit, teacher_id, teacher_lse)
    loss = torch.empty(N, dtype=torch.float32, device=dev)
    lse = torch.empty(N, dtype=torch.float32, device=dev)
    rc = lib().sd_distill_topk(
        student.data_ptr(), rs, dt, lp, ip, tp, N, V, K, T, loss.data_ptr(),
        lse.data_ptr(), _status(status, dev), _raw_stream(dev))
    if rc != SD_OK:
        _check(rc)
    return {"loss": loss, "lse": lse}


def distill_topk_backward(student, lse, teacher_logit, teacher_id, grad_loss,
                          T=1.0, *, teacher_lse=None, out=None, status=None):
    """Gradient of sum_n grad_loss[n] loss[n] of distill_topk with respect to
    the student's logits (sd_distill_topk_backward); lse as distill_topk
    returned it.  ``out`` may be the student itself; torch does not see that
    write (no version is counted, so nothing that autograd saved of the student
    may be used after it).  Returns grad [N, V] of the student's type."""
    dev, N, V, K, dt, rs, lp, ip, tp = _distill_rows(
        student, teacher_logit, teacher_id, teacher_lse)
    sp = _row_vector(lse, dev, "lse", N)
    wp = _row_vector(grad_loss, dev, "grad_loss", N)
    grad, gs = _grad_out(out, student, dev, N, V)
    rc = lib().sd_distill_topk_backward(
        student.data_ptr(), rs, dt, sp, lp, ip, tp, wp, N, V, K, T,
        grad.data_ptr(), gs, _status(status, dev), _raw_stream(dev))
    if rc != SD_OK:
        _check(rc)
    return grad


def distill_topk_step(student, teacher_logit, teacher_id, grad_loss, T=1.0,
                      *, teacher_lse=None, out=None, status=None):
    """distill_topk and its gradient in one call (sd_distill_topk_step), for
    a training step that knows the rows' weights beforehand; ``out`` as in
    distill_topk_backward.  Returns loss, lse and grad."""
    dev, N, V, K, dt, rs, lp, ip, tp = _distill_rows(
        student, teacher_logit, teacher_id, teacher_lse)
    wp = _row_vector(grad_loss, dev, "grad_loss", N)
    loss = torch.empty(N, dtype=torch.float32, device=dev)
    lse = torch.empty(N, dtype=torch.float32, device=dev)
    grad, gs = _grad_out(out, student, dev, N, V)
    rc = lib().sd_distill_topk_step(
        student.data_ptr(), rs, dt, lp, ip, tp, wp, N, V, K, T,
        loss.data_ptr(), lse.data_ptr(), grad.data_ptr(), gs,
        _status(status, dev), _raw_stream(dev))
    if rc != SD_OK:
        _check(rc)
    return {"loss": loss, "lse": lse, "grad": grad}

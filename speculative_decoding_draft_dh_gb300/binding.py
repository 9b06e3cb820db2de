"""ctypes binding of libdh (include/dh.h).  Argument marshalling only: every step of the path runs
in the CUDA library.  torch supplies device memory and the current stream.

The library is loaded on first use from this package directory; if it is missing or cannot be
loaded the call raises (there is no fallback).
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdh.so")

DH_OK = 0
STATUS = {0: "DH_OK", 1: "DH_ERR_INVALID_ARG", 2: "DH_ERR_UNSUPPORTED", 3: "DH_ERR_WORKSPACE",
          4: "DH_ERR_CUDA", 5: "DH_ERR_TIMEOUT", 6: "DH_ERR_BAD_INPUT"}
F32, BF16 = 0, 1

EXPORTS = ["dh_status_string", "dh_version", "dh_last_error", "dh_lowrank_topk_workspace", "dh_lowrank_topk",
           "dh_exact_rescore_workspace", "dh_exact_rescore", "dh_draft_head_workspace", "dh_draft_head",
           "dh_expand_children",
           "dh_tree_accept_workspace",
           "dh_tree_accept", "dh_tree_accept_noalloc", "dh_workspace_status", "dh_selftest_wait_timeout", "dh_prof_enable", "dh_prof_read",
           "dh_set_tuning", "dh_verify_chain_workspace", "dh_verify_chain", "dh_size_level",
           "dh_lowrank_topk_shard", "dh_merge_topk", "dh_exact_rescore_shard_workspace", "dh_exact_rescore_shard",
           "dh_combine_softmax",
           "dh_distill_topk_workspace", "dh_distill_topk", "dh_distill_topk_backward",
           "dh_distill_topk_step_workspace", "dh_distill_topk_step", "dh_selftest_distill_timeout",
           "dh_beam_select_workspace", "dh_beam_select", "dh_reorder_states"]

MAX_K, MAX_BEAMS, MAX_BEAM_OUT, MAX_SLOTS = 1024, 128, 256, 1024  # DH_MAX_*

_lib = None
_lock = threading.Lock()


class DhError(RuntimeError):
    def __init__(self, status: int, what: str, detail: str = ""):
        msg = f"{what} failed: {STATUS.get(status, status)}"
        super().__init__(msg + (f" ({detail})" if detail else ""))
        self.status = status


def load_library(path: str | None = None):
    """Load libdh.so and declare the C signatures (raises if the library is missing)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    with _lock:
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"libdh.so not found at {p}: build it with "
                               "`python -m speculative_decoding_draft_dh_gb300.build`")
        lib = ctypes.CDLL(p)
        P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        lib.dh_status_string.argtypes = [I]
        lib.dh_status_string.restype = ctypes.c_char_p
        lib.dh_version.restype = I
        lib.dh_last_error.restype = ctypes.c_char_p
        lib.dh_lowrank_topk_workspace.argtypes = [I, I, I, I, I, I]
        lib.dh_lowrank_topk_workspace.restype = Z
        lib.dh_lowrank_topk.argtypes = [P, P, P, I, I, I, I, I, I, P, P, P, Z, P]
        lib.dh_lowrank_topk.restype = I
        lib.dh_exact_rescore_workspace.argtypes = [I, I, I, I, I]
        lib.dh_exact_rescore_workspace.restype = Z
        lib.dh_exact_rescore.argtypes = [P, P, P, I, I, I, I, I, P, P, P, Z, P]
        lib.dh_exact_rescore.restype = I
        lib.dh_draft_head_workspace.argtypes = [I, I, I, I, I, I]
        lib.dh_draft_head_workspace.restype = Z
        lib.dh_draft_head.argtypes = [P, P, P, P, I, I, I, I, I, I, P, P, P, P, P, Z, P]
        lib.dh_draft_head.restype = I
        lib.dh_expand_children.argtypes = [P, P, P, I, I, I, ctypes.c_float, P, P, P, P]
        lib.dh_expand_children.restype = I
        lib.dh_tree_accept_workspace.argtypes = [I, I, I]
        lib.dh_tree_accept_workspace.restype = Z
        lib.dh_tree_accept.argtypes = [P, P, P, I, I, I, I, P, P, P, P, P, P, Z, P]
        lib.dh_tree_accept.restype = I
        lib.dh_tree_accept_noalloc.argtypes = [P, P, P, I, I, I, I, P, P, P, P, P, P]
        lib.dh_tree_accept_noalloc.restype = I
        lib.dh_workspace_status.argtypes = [P, P, P]
        lib.dh_workspace_status.restype = I
        lib.dh_selftest_wait_timeout.argtypes = [I, I, P, Z, P]
        lib.dh_selftest_wait_timeout.restype = I
        lib.dh_prof_enable.argtypes = [I]
        lib.dh_prof_enable.restype = I
        lib.dh_prof_read.argtypes = [P, I, P, P, I]
        lib.dh_prof_read.restype = I
        lib.dh_verify_chain_workspace.argtypes = [I, I, I, I]
        lib.dh_verify_chain_workspace.restype = Z
        lib.dh_verify_chain.argtypes = [P, P, P, P, P, P, I, I, I, I, I, ctypes.c_float, P, P, P, Z, P]
        lib.dh_verify_chain.restype = I
        lib.dh_size_level.argtypes = [P, P, P, I, I, I, P, P, I, I, I, ctypes.c_float, P, P, P, P, P]
        lib.dh_size_level.restype = I
        lib.dh_lowrank_topk_shard.argtypes = [P, P, P, I, I, I, I, I, I, I, P, P, P, Z, P]
        lib.dh_lowrank_topk_shard.restype = I
        lib.dh_merge_topk.argtypes = [P, P, I, I, I, P, P, P]
        lib.dh_merge_topk.restype = I
        lib.dh_exact_rescore_shard_workspace.argtypes = [I, I, I, I, I]
        lib.dh_exact_rescore_shard_workspace.restype = Z
        lib.dh_exact_rescore_shard.argtypes = [P, P, P, I, I, I, I, I, I, P, P, P, Z, P]
        lib.dh_exact_rescore_shard.restype = I
        lib.dh_combine_softmax.argtypes = [P, P, I, I, I, P, P, P]
        lib.dh_combine_softmax.restype = I
        L, F = ctypes.c_int64, ctypes.c_float
        lib.dh_distill_topk_workspace.argtypes = [I, I, I]
        lib.dh_distill_topk_workspace.restype = Z
        lib.dh_distill_topk.argtypes = [P, L, P, P, P, I, I, I, I, F, P, P, P, Z, P]
        lib.dh_distill_topk.restype = I
        lib.dh_distill_topk_backward.argtypes = [P, L, P, P, P, P, P, I, I, I, I, F, P, L, P]
        lib.dh_distill_topk_backward.restype = I
        lib.dh_distill_topk_step_workspace.argtypes = [I, I, I, I]
        lib.dh_distill_topk_step_workspace.restype = Z
        lib.dh_distill_topk_step.argtypes = [P, L, P, P, P, P, I, I, I, I, F, P, P, L, P, Z, P]
        lib.dh_distill_topk_step.restype = I
        lib.dh_selftest_distill_timeout.argtypes = [I, I, I, P, L, P, P, P, I, I, I, F, P, P, L, P, Z, P]
        lib.dh_selftest_distill_timeout.restype = I
        lib.dh_beam_select_workspace.argtypes = [I, I, I, I]
        lib.dh_beam_select_workspace.restype = Z
        lib.dh_beam_select.argtypes = [P, L, L, P, P, I, I, I, I, I, F, I, P, P, P, P, Z, P]
        lib.dh_beam_select.restype = I
        lib.dh_reorder_states.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, L, P]
        lib.dh_reorder_states.restype = I
        lib.dh_set_tuning.argtypes = [ctypes.c_char_p, ctypes.c_char_p]
        lib.dh_set_tuning.restype = I
        if path is None:
            _lib = lib
        return lib


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t.dtype}: use torch.bfloat16 or torch.float32")


def _dev(t: torch.Tensor, name: str) -> torch.Tensor:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


class Workspace:
    """Zero-initialised device workspaces, grown on demand: one buffer per (device, call kind), so
    one object can serve all three calls.  Calls using the same object must not overlap in time."""

    def __init__(self):
        self.buf = {}

    def get(self, nbytes: int, device, kind: str, stream=None) -> torch.Tensor | None:
        """The buffer for one call kind, at least nbytes long; a new one is zeroed on `stream` (the
        call's stream, else the current one), so that the call that follows finds it zeroed."""
        if nbytes == 0:
            return None
        key = (torch.device(device), kind)
        cur = self.buf.get(key)
        if cur is None or cur.numel() < nbytes:
            with torch.cuda.stream(torch.cuda.current_stream(key[0]) if stream is None else stream):
                cur = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=key[0])
            self.buf[key] = cur
        return cur


_default_ws = Workspace()


def _check(status, what):
    if status != DH_OK:
        detail = ""
        if status == 4 and _lib is not None:
            detail = (_lib.dh_last_error() or b"").decode(errors="replace")
        raise DhError(status, what, detail)


def lowrank_topk(h, U, V, K, *, idx_out=None, score_out=None, workspace=None, stream=None):
    """Stage 1: the K best low-rank scores per row.  Returns (idx int32 [B,K], score fp32 [B,K])."""
    lib = load_library()
    _dev(h, "h"), _dev(U, "U"), _dev(V, "V")
    B, d = h.shape
    r, vocab = V.shape
    dt = _dtype_code(h)
    if U.dtype != h.dtype or V.dtype != h.dtype or U.shape != (d, r):
        raise ValueError("h, U, V must share a dtype and have shapes [B,d], [d,r], [r,vocab]")
    if idx_out is None:
        idx_out = torch.empty(B, K, dtype=torch.int32, device=h.device)
    if score_out is None:
        score_out = torch.empty(B, K, dtype=torch.float32, device=h.device)
    nbytes = lib.dh_lowrank_topk_workspace(B, d, r, vocab, K, dt)
    ws = (workspace or _default_ws).get(nbytes, h.device, "topk", stream)
    _check(lib.dh_lowrank_topk(_ptr(h), _ptr(U), _ptr(V), B, d, r, vocab, K, dt, _ptr(idx_out),
                               _ptr(score_out), _ptr(ws), nbytes, _stream(stream)), "dh_lowrank_topk")
    return idx_out, score_out


def exact_rescore(h, W, idx, *, with_probs=True, logits_out=None, probs_out=None, workspace=None,
                  stream=None):
    """Stage 2: exact logits of the candidates and (optionally) their softmax."""
    lib = load_library()
    _dev(h, "h"), _dev(W, "W"), _dev(idx, "idx")
    B, d = h.shape
    vocab = W.shape[0]
    K = idx.shape[1]
    dt = _dtype_code(h)
    if W.dtype != h.dtype or W.shape[1] != d or idx.dtype != torch.int32 or idx.shape[0] != B:
        raise ValueError("h [B,d], W [vocab,d] share a dtype; idx is int32 [B,K]")
    if logits_out is None:
        logits_out = torch.empty(B, K, dtype=torch.float32, device=h.device)
    if with_probs and probs_out is None:
        probs_out = torch.empty(B, K, dtype=torch.float32, device=h.device)
    nbytes = lib.dh_exact_rescore_workspace(B, d, vocab, K, dt)
    ws = (workspace or _default_ws).get(nbytes, h.device, "rescore", stream)
    _check(lib.dh_exact_rescore(_ptr(h), _ptr(W), _ptr(idx), B, d, vocab, K, dt, _ptr(logits_out),
                                _ptr(probs_out if with_probs else None), _ptr(ws), nbytes,
                                _stream(stream)), "dh_exact_rescore")
    return logits_out, (probs_out if with_probs else None)


def draft_head(h, U, V, W, K, *, with_probs=True, idx_out=None, score_out=None, logits_out=None,
               probs_out=None, workspace=None, stream=None):
    """Both stages in one call (dh_draft_head: the outputs of lowrank_topk followed by
    exact_rescore, with selection and rescoring fused into one cluster kernel for small batches:
    up to 32 rows of 64 candidates on a GB300).  Returns (idx int32 [B,K], score fp32 [B,K],
    logits fp32 [B,K], probs fp32 [B,K] or None)."""
    lib = load_library()
    _dev(h, "h"), _dev(U, "U"), _dev(V, "V"), _dev(W, "W")
    B, d = h.shape
    r, vocab = V.shape
    dt = _dtype_code(h)
    if U.dtype != h.dtype or V.dtype != h.dtype or W.dtype != h.dtype or U.shape != (d, r) \
            or W.shape != (vocab, d):
        raise ValueError("h, U, V, W must share a dtype and have shapes [B,d], [d,r], [r,vocab], [vocab,d]")
    dev = h.device
    if idx_out is None:
        idx_out = torch.empty(B, K, dtype=torch.int32, device=dev)
    if score_out is None:
        score_out = torch.empty(B, K, dtype=torch.float32, device=dev)
    if logits_out is None:
        logits_out = torch.empty(B, K, dtype=torch.float32, device=dev)
    if with_probs and probs_out is None:
        probs_out = torch.empty(B, K, dtype=torch.float32, device=dev)
    nbytes = lib.dh_draft_head_workspace(B, d, r, vocab, K, dt)
    ws = (workspace or _default_ws).get(nbytes, dev, "head", stream)
    _check(lib.dh_draft_head(_ptr(h), _ptr(U), _ptr(V), _ptr(W), B, d, r, vocab, K, dt, _ptr(idx_out),
                             _ptr(score_out), _ptr(logits_out), _ptr(probs_out if with_probs else None),
                             _ptr(ws), nbytes, _stream(stream)), "dh_draft_head")
    return idx_out, score_out, logits_out, (probs_out if with_probs else None)


def expand_children(probs, idx, w, *, parent_prob=None, min_benefit=0.0, child_token=None, child_prob=None,
                    n_keep=None, stream=None):
    """The w children of each frontier node by exact probability.  Returns (child_token int32
    [B,w], child_prob fp32 [B,w], n_keep int32 [B])."""
    lib = load_library()
    _dev(probs, "probs"), _dev(idx, "idx")
    if probs.dtype != torch.float32 or idx.dtype != torch.int32 or probs.shape != idx.shape:
        raise ValueError("probs fp32 [B,K] and idx int32 [B,K]")
    B, K = probs.shape
    dev = probs.device
    if parent_prob is not None:
        _dev(parent_prob, "parent_prob")
        if parent_prob.dtype != torch.float32 or parent_prob.shape != (B,):
            raise ValueError("parent_prob must be fp32 [B]")
    if child_token is None:
        child_token = torch.empty(B, w, dtype=torch.int32, device=dev)
    if child_prob is None:
        child_prob = torch.empty(B, w, dtype=torch.float32, device=dev)
    if n_keep is None:
        n_keep = torch.empty(B, dtype=torch.int32, device=dev)
    _check(lib.dh_expand_children(_ptr(probs), _ptr(idx), _ptr(parent_prob), B, K, w, float(min_benefit),
                                  _ptr(child_token), _ptr(child_prob), _ptr(n_keep), _stream(stream)),
           "dh_expand_children")
    return child_token, child_prob, n_keep


def tree_accept(logits, parent, token, *, with_argmax=True, workspace=None, stream=None):
    """Greedy acceptance over draft trees.  Returns dict(argmax, path, len, bonus, err)."""
    lib = load_library()
    _dev(logits, "logits"), _dev(parent, "parent"), _dev(token, "token")
    B, N, vocab = logits.shape
    dt = _dtype_code(logits)
    if parent.dtype != torch.int32 or token.dtype != torch.int32 or parent.shape != (B, N) \
            or token.shape != (B, N):
        raise ValueError("parent and token must be int32 [B,N]")
    dev = logits.device
    out = {"argmax": torch.empty(B, N, dtype=torch.int32, device=dev) if with_argmax else None,
           "path": torch.empty(B, N, dtype=torch.int32, device=dev),
           "len": torch.empty(B, dtype=torch.int32, device=dev),
           "bonus": torch.empty(B, dtype=torch.int32, device=dev),
           "err": torch.empty(B, dtype=torch.int32, device=dev)}
    nbytes = lib.dh_tree_accept_workspace(B, N, vocab)
    ws = (workspace or _default_ws).get(nbytes, dev, "tree", stream)
    _check(lib.dh_tree_accept(_ptr(logits), _ptr(parent), _ptr(token), B, N, vocab, dt,
                              _ptr(out["argmax"]), _ptr(out["path"]), _ptr(out["len"]),
                              _ptr(out["bonus"]), _ptr(out["err"]), _ptr(ws), nbytes,
                              _stream(stream)), "dh_tree_accept")
    return out


def lowrank_topk_shard(h, U, V_shard, K, vocab_offset, *, idx_out=None, score_out=None, workspace=None,
                       stream=None):
    """Stage 1 on one vocabulary shard (V_shard [r, n] holds the columns vocab_offset .. + n):
    the shard's K best (global id, score) per row."""
    lib = load_library()
    _dev(h, "h"), _dev(U, "U"), _dev(V_shard, "V_shard")
    B, d = h.shape
    r, n = V_shard.shape
    dt = _dtype_code(h)
    if U.dtype != h.dtype or V_shard.dtype != h.dtype or U.shape != (d, r):
        raise ValueError("h, U, V_shard must share a dtype and have shapes [B,d], [d,r], [r,n]")
    if idx_out is None:
        idx_out = torch.empty(B, K, dtype=torch.int32, device=h.device)
    if score_out is None:
        score_out = torch.empty(B, K, dtype=torch.float32, device=h.device)
    nbytes = lib.dh_lowrank_topk_workspace(B, d, r, n, K, dt)
    ws = (workspace or _default_ws).get(nbytes, h.device, "topk", stream)
    _check(lib.dh_lowrank_topk_shard(_ptr(h), _ptr(U), _ptr(V_shard), B, d, r, n, int(vocab_offset), K, dt,
                                     _ptr(idx_out), _ptr(score_out), _ptr(ws), nbytes, _stream(stream)),
           "dh_lowrank_topk_shard")
    return idx_out, score_out


def merge_topk(idx_parts, score_parts, *, idx_out=None, score_out=None, stream=None):
    """The K best of P shard lists per row (dh_merge_topk).  idx_parts int32 / score_parts fp32
    [P, B, K]."""
    lib = load_library()
    _dev(idx_parts, "idx_parts"), _dev(score_parts, "score_parts")
    P, B, K = idx_parts.shape
    if idx_parts.dtype != torch.int32 or score_parts.dtype != torch.float32 or score_parts.shape != (P, B, K):
        raise ValueError("idx_parts int32 and score_parts fp32 [P, B, K]")
    dev = idx_parts.device
    if idx_out is None:
        idx_out = torch.empty(B, K, dtype=torch.int32, device=dev)
    if score_out is None:
        score_out = torch.empty(B, K, dtype=torch.float32, device=dev)
    _check(lib.dh_merge_topk(_ptr(idx_parts), _ptr(score_parts), P, B, K, _ptr(idx_out), _ptr(score_out),
                             _stream(stream)), "dh_merge_topk")
    return idx_out, score_out


def exact_rescore_shard(h, W_shard, idx, vocab_offset, *, logits_out=None, stats_out=None, workspace=None,
                        stream=None):
    """Stage 2 on one shard: logits of the candidates this shard owns (-inf elsewhere) and the row's
    (max, sum of exp) pair [B, 2]."""
    lib = load_library()
    _dev(h, "h"), _dev(W_shard, "W_shard"), _dev(idx, "idx")
    B, d = h.shape
    n = W_shard.shape[0]
    K = idx.shape[1]
    dt = _dtype_code(h)
    if W_shard.dtype != h.dtype or W_shard.shape[1] != d or idx.dtype != torch.int32 or idx.shape[0] != B:
        raise ValueError("h [B,d], W_shard [n,d] share a dtype; idx is int32 [B,K]")
    if logits_out is None:
        logits_out = torch.empty(B, K, dtype=torch.float32, device=h.device)
    if stats_out is None:
        stats_out = torch.empty(B, 2, dtype=torch.float32, device=h.device)
    nbytes = lib.dh_exact_rescore_shard_workspace(B, d, n, K, dt)
    ws = (workspace or _default_ws).get(nbytes, h.device, "rescore_shard", stream)
    _check(lib.dh_exact_rescore_shard(_ptr(h), _ptr(W_shard), _ptr(idx), B, d, n, int(vocab_offset), K, dt,
                                      _ptr(logits_out), _ptr(stats_out), _ptr(ws), nbytes, _stream(stream)),
           "dh_exact_rescore_shard")
    return logits_out, stats_out


def combine_softmax(logits_parts, stats_parts, *, with_probs=True, logits_out=None, probs_out=None, stream=None):
    """Each candidate's logit from its owner shard and the softmax over the K candidates
    (dh_combine_softmax).  logits_parts [P, B, K], stats_parts [P, B, 2] fp32."""
    lib = load_library()
    _dev(logits_parts, "logits_parts"), _dev(stats_parts, "stats_parts")
    P, B, K = logits_parts.shape
    if logits_parts.dtype != torch.float32 or stats_parts.dtype != torch.float32 or stats_parts.shape != (P, B, 2):
        raise ValueError("logits_parts [P, B, K] and stats_parts [P, B, 2], fp32")
    dev = logits_parts.device
    if logits_out is None:
        logits_out = torch.empty(B, K, dtype=torch.float32, device=dev)
    if with_probs and probs_out is None:
        probs_out = torch.empty(B, K, dtype=torch.float32, device=dev)
    _check(lib.dh_combine_softmax(_ptr(logits_parts), _ptr(stats_parts), P, B, K, _ptr(logits_out),
                                  _ptr(probs_out if with_probs else None), _stream(stream)), "dh_combine_softmax")
    return logits_out, (probs_out if with_probs else None)


def size_level(child_prob, child_token, cost, bin_batch, batch, theta, *, n_valid=None, out=None, stream=None):
    """Width and children of the next draft level per request (dh_size_level).  child_prob fp32 /
    child_token int32 [R, F, Wc]; cost fp32 [n_bins, wmax+1] and bin_batch int32 [n_bins] on the
    device.  Returns dict(width int32 [R], parent, token int32 [R, wmax], prob fp32 [R, wmax])."""
    lib = load_library()
    _dev(child_prob, "child_prob"), _dev(child_token, "child_token"), _dev(cost, "cost"), _dev(bin_batch, "bin_batch")
    R, F, Wc = child_prob.shape
    n_bins, w1 = cost.shape
    wmax = w1 - 1
    if child_prob.dtype != torch.float32 or child_token.dtype != torch.int32 or child_token.shape != (R, F, Wc) \
            or cost.dtype != torch.float32 or bin_batch.dtype != torch.int32 or bin_batch.shape != (n_bins,):
        raise ValueError("child_prob fp32 / child_token int32 [R,F,Wc], cost fp32 [n_bins,wmax+1], "
                         "bin_batch int32 [n_bins]")
    if n_valid is not None:
        _dev(n_valid, "n_valid")
    dev = child_prob.device
    if out is None:
        out = {"width": torch.empty(R, dtype=torch.int32, device=dev),
               "parent": torch.empty(R, wmax, dtype=torch.int32, device=dev),
               "token": torch.empty(R, wmax, dtype=torch.int32, device=dev),
               "prob": torch.empty(R, wmax, dtype=torch.float32, device=dev)}
    _check(lib.dh_size_level(_ptr(child_prob), _ptr(child_token), _ptr(n_valid), R, F, Wc, _ptr(cost), _ptr(bin_batch),
                             n_bins, wmax, int(batch), float(theta), _ptr(out["width"]), _ptr(out["parent"]),
                             _ptr(out["token"]), _ptr(out["prob"]), _stream(stream)), "dh_size_level")
    return out


def verify_chain(logits, cand_idx, cand_prob, draft_token, u_accept, u_sample, *, temperature=1.0,
                 n_accept_out=None, token_out=None, workspace=None, stream=None):
    """Speculative sampling over a chain of L drafted tokens per request (dh_verify_chain).
    logits [B, L+1, vocab] (bf16 or fp32); cand_idx int32 / cand_prob fp32 [B, L, K]; draft_token
    int32 / u_accept fp32 [B, L]; u_sample fp32 [B].  Returns (n_accept int32 [B], token int32 [B])."""
    lib = load_library()
    _dev(logits, "logits"), _dev(u_sample, "u_sample")
    B, L1, vocab = logits.shape
    L = L1 - 1
    K = cand_idx.shape[2] if L > 0 else 0
    for t, name, dt in ((cand_idx, "cand_idx", torch.int32), (cand_prob, "cand_prob", torch.float32),
                        (draft_token, "draft_token", torch.int32), (u_accept, "u_accept", torch.float32)):
        if L > 0:
            _dev(t, name)
            if t.dtype != dt:
                raise ValueError(f"{name} must be {dt}")
    if u_sample.dtype != torch.float32 or u_sample.shape != (B,):
        raise ValueError("u_sample must be fp32 [B]")
    dev = logits.device
    if n_accept_out is None:
        n_accept_out = torch.empty(B, dtype=torch.int32, device=dev)
    if token_out is None:
        token_out = torch.empty(B, dtype=torch.int32, device=dev)
    dt = _dtype_code(logits)
    nbytes = lib.dh_verify_chain_workspace(B, L, vocab, dt)
    ws = (workspace or _default_ws).get(nbytes, dev, "verify", stream)
    _check(lib.dh_verify_chain(_ptr(logits), _ptr(cand_idx if L > 0 else None), _ptr(cand_prob if L > 0 else None),
                               _ptr(draft_token if L > 0 else None), _ptr(u_accept if L > 0 else None),
                               _ptr(u_sample), B, L, vocab, K, dt, float(temperature), _ptr(n_accept_out),
                               _ptr(token_out), _ptr(ws), nbytes, _stream(stream)), "dh_verify_chain")
    return n_accept_out, token_out


# ---------------------------------------------------------------- training, search and state operators
#
# These calls take strided rows and run on the device of their tensors, whichever is current.  Their
# scratch needs no zeroing, so without `workspace` each call takes its own from the caching allocator
# on its stream: calls on different streams, and graphs captured from them, share nothing.  With an
# explicit `stream` the results belong to that stream, and the inputs are kept from being reused by
# the allocator until the stream has passed the call (the caller orders the stream behind whatever
# wrote the inputs).  They are outside of autograd (distill.distill_loss is the differentiable form):
# results have no graph, whether or not the inputs require grad.  Tensors of the caller's that a call
# writes count as modified, so that autograd notices where it saved them.


# The current stream's handle (torch.cuda.current_stream(index).cuda_stream without the object).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _elsewhere(stream, dev, tensors, call):
    """call() with `dev` current and, if given, `stream`; the tensors (some may be None) are kept for
    the stream."""
    if stream is None:
        with torch.cuda.device(dev):
            return call()
    if stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
    with torch.cuda.stream(stream):
        out = call()
        if not torch.cuda.is_current_stream_capturing():
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
    return out


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(query, *sizes):
    return getattr(load_library(), query)(*sizes)


def _scratch(nbytes, workspace, kind, dev):
    """nbytes of device memory, not zeroed: the caller's workspace object's, else fresh (None: 0 bytes)."""
    if workspace is not None:
        return workspace.get(nbytes, dev, kind)
    return torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None


def _addr(t):
    return None if t is None else t.data_ptr()


_bump = torch.autograd.graph.increment_version


def _written(*tensors):
    """Raises the version of the caller's tensors (None: not given) that a call has written."""
    for t in tensors:
        if t is not None:
            _bump((t,))


def _typed(t, name, dtype, shape, index):
    """Checks a contiguous tensor of one dtype and shape on CUDA device `index`."""
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} {list(shape)}, not {t.dtype} {list(t.shape)}")
    if t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and on CUDA device {index}, not on {t.device}")


_INT_MAX = (1 << 31) - 1  # larger sizes would be cut off on their way to the library


def _rows(t, name):
    """Checks a [.., vocab] CUDA tensor of logits whose elements of a row are adjacent; its dtype's
    code and its device's index."""
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    code = _dtype_code(t)
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: the elements of a row must be adjacent (last stride 1)")
    return code, index


def _distill_inputs(logits, idx, teacher, n_valid):
    if logits.dim() != 2 or idx.dim() != 2:
        raise ValueError("logits must be [N, vocab] and idx [N, K]")
    dt, index = _rows(logits, "logits")
    N, vocab = logits.shape
    K = idx.shape[1]
    if N > _INT_MAX or vocab > _INT_MAX or K > _INT_MAX:
        raise ValueError("logits and idx: N, vocab and K have to fit 32 bits")
    _typed(idx, "idx", torch.int32, (N, K), index)
    _typed(teacher, "teacher", torch.float32, (N, K), index)
    if n_valid is not None:
        _typed(n_valid, "n_valid", torch.int32, (N,), index)
    return dt, index, N, vocab, K


def _grad_rows(logits, grad_out, index):
    """grad_out checked, or memory for the gradient: rows that lie like those of `logits` on 16 bytes, the
    first one and the distance between them, which is theirs where that takes at most an eighth more memory.
    Rows that share memory get packed ones."""
    N, vocab = logits.shape
    if grad_out is None:
        ld = logits.stride(0)
        if ld <= vocab or N <= 1:
            ld = vocab
        elif ld - vocab > vocab // 8:
            ld = vocab + (ld - vocab) % (16 // logits.element_size())
        beside = logits.data_ptr() & 15
        if beside:
            first = beside // logits.element_size()
            rows = torch.empty(N * ld + first, dtype=logits.dtype, device=logits.device)[first:].view(N, ld)
        else:
            rows = torch.empty((N, ld), dtype=logits.dtype, device=logits.device)
        return rows if ld == vocab else rows[:, :vocab]
    if grad_out.dtype != logits.dtype or grad_out.shape != logits.shape:
        raise ValueError("grad_out must have the logits' dtype and shape")
    if _rows(grad_out, "grad_out")[1] != index:
        raise ValueError(f"grad_out must be on CUDA device {index}")
    if N > 1 and grad_out.stride(0) < vocab:
        raise ValueError("the rows of grad_out must not overlap")
    return grad_out


def _out(t, name, dtype, shape, dev):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _typed(t, name, dtype, shape, dev.index)
    return t


def distill_topk(logits, idx, teacher, *, n_valid=None, temperature=1.0, loss_out=None, stats_out=None, workspace=None,
                 stream=None):
    """The loss of a student's logits [N, vocab] (bf16 or fp32, rows may be strided) against a
    teacher's top logits: ids idx int32 and values teacher fp32 [N, K], of which the first n_valid
    int32 [N] count (dh_distill_topk).  Returns (loss fp32 [N], stats fp32 [N, 2]: each row's
    maximum and sum of exp((z - max) / T), which the gradient takes)."""
    lib = load_library()
    dt, index, N, vocab, K = _distill_inputs(logits, idx, teacher, n_valid)
    dev = logits.device
    if stream is not None or index != torch.cuda.current_device():
        return _elsewhere(stream, dev, (logits, idx, teacher, n_valid, loss_out, stats_out), lambda: distill_topk(
            logits, idx, teacher, n_valid=n_valid, temperature=temperature, loss_out=loss_out, stats_out=stats_out,
            workspace=workspace))
    loss = _out(loss_out, "loss_out", torch.float32, (N,), dev)
    stats = _out(stats_out, "stats_out", torch.float32, (N, 2), dev)
    nbytes = _workspace_bytes("dh_distill_topk_workspace", N, vocab, dt)
    ws = _scratch(nbytes, workspace, "distill", dev)
    _check(lib.dh_distill_topk(logits.data_ptr(), logits.stride(0), idx.data_ptr(), teacher.data_ptr(), _addr(n_valid),
                               N, vocab, K, dt, float(temperature), loss.data_ptr(), stats.data_ptr(), _addr(ws),
                               nbytes, _raw_stream(index)), "dh_distill_topk")
    if loss_out is not None or stats_out is not None:
        _written(loss_out, stats_out)
    return loss, stats


def distill_topk_backward(logits, idx, teacher, stats, grad_loss, *, n_valid=None, temperature=1.0, grad_out=None,
                          stream=None):
    """The gradient of sum(grad_loss * loss) with respect to the logits, from the stats that
    distill_topk returned for the same inputs (dh_distill_topk_backward).  grad_out may be the
    logits themselves.  Returns it, in the logits' dtype."""
    lib = load_library()
    dt, index, N, vocab, K = _distill_inputs(logits, idx, teacher, n_valid)
    _typed(stats, "stats", torch.float32, (N, 2), index)
    _typed(grad_loss, "grad_loss", torch.float32, (N,), index)
    if stream is not None or index != torch.cuda.current_device():
        return _elsewhere(stream, logits.device, (logits, idx, teacher, n_valid, stats, grad_loss, grad_out),
                          lambda: distill_topk_backward(logits, idx, teacher, stats, grad_loss, n_valid=n_valid,
                                                        temperature=temperature, grad_out=grad_out))
    grad = _grad_rows(logits, grad_out, index)
    _check(lib.dh_distill_topk_backward(logits.data_ptr(), logits.stride(0), idx.data_ptr(), teacher.data_ptr(),
                                        _addr(n_valid), stats.data_ptr(), grad_loss.data_ptr(), N, vocab, K, dt,
                                        float(temperature), grad.data_ptr(), grad.stride(0), _raw_stream(index)),
           "dh_distill_topk_backward")
    if grad_out is not None:
        _written(grad_out)
    return grad


def distill_topk_step(logits, idx, teacher, grad_loss, *, n_valid=None, temperature=1.0, loss_out=None, grad_out=None,
                      workspace=None, stream=None):
    """distill_topk and distill_topk_backward in one call, for rows whose weights grad_loss fp32 [N]
    are known beforehand (dh_distill_topk_step).  grad_out may be the logits themselves.  A wait of the
    kernel that gives up shows as NaN losses and gradients, with `workspace` also in workspace_status.
    Returns (loss fp32 [N], gradient)."""
    lib = load_library()
    dt, index, N, vocab, K = _distill_inputs(logits, idx, teacher, n_valid)
    _typed(grad_loss, "grad_loss", torch.float32, (N,), index)
    dev = logits.device
    if stream is not None or index != torch.cuda.current_device():
        return _elsewhere(stream, dev, (logits, idx, teacher, n_valid, grad_loss, loss_out, grad_out),
                          lambda: distill_topk_step(logits, idx, teacher, grad_loss, n_valid=n_valid,
                                                    temperature=temperature, loss_out=loss_out, grad_out=grad_out,
                                                    workspace=workspace))
    loss = _out(loss_out, "loss_out", torch.float32, (N,), dev)
    grad = _grad_rows(logits, grad_out, index)
    nbytes = _workspace_bytes("dh_distill_topk_step_workspace", N, vocab, K, dt)
    ws = _scratch(nbytes, workspace, "distill_step", dev)
    _check(lib.dh_distill_topk_step(logits.data_ptr(), logits.stride(0), idx.data_ptr(), teacher.data_ptr(),
                                    _addr(n_valid), grad_loss.data_ptr(), N, vocab, K, dt, float(temperature),
                                    loss.data_ptr(), grad.data_ptr(), grad.stride(0), _addr(ws), nbytes,
                                    _raw_stream(index)), "dh_distill_topk_step")
    if loss_out is not None or grad_out is not None:
        _written(loss_out, grad_out)
    return loss, grad


def beam_select(logits, score, M, *, finished=None, pad_token=0, temperature=1.0, parent_out=None, token_out=None,
                score_out=None, workspace=None, stream=None):
    """The M best continuations of each request's beams over the whole vocabulary (dh_beam_select).
    logits [R, W, vocab] (bf16 or fp32, beams and requests may be strided or shared); score fp32
    [R, W], -inf for unused beams; finished int32 [R, W].  Returns (parent int32 [R, M], token int32
    [R, M], score fp32 [R, M])."""
    lib = load_library()
    if logits.dim() != 3:
        raise ValueError("logits must be [R, W, vocab]")
    dt, index = _rows(logits, "logits")
    R, W, vocab = logits.shape
    _typed(score, "score", torch.float32, (R, W), index)
    if finished is not None:
        _typed(finished, "finished", torch.int32, (R, W), index)
    M = int(M)
    pad_token = int(pad_token)
    if R > _INT_MAX or W > _INT_MAX or vocab > _INT_MAX or abs(M) > _INT_MAX or abs(pad_token) > _INT_MAX:
        raise ValueError("R, W, vocab, M and pad_token have to fit 32 bits")
    dev = logits.device
    if stream is not None or index != torch.cuda.current_device():
        return _elsewhere(stream, dev, (logits, score, finished, parent_out, token_out, score_out), lambda: beam_select(
            logits, score, M, finished=finished, pad_token=pad_token, temperature=temperature, parent_out=parent_out,
            token_out=token_out, score_out=score_out, workspace=workspace))
    size = (R, max(M, 0))
    parent = _out(parent_out, "parent_out", torch.int32, size, dev)
    token = _out(token_out, "token_out", torch.int32, size, dev)
    best = _out(score_out, "score_out", torch.float32, size, dev)
    nbytes = _workspace_bytes("dh_beam_select_workspace", R, W, vocab, dt)
    ws = _scratch(nbytes, workspace, "beam", dev)
    _check(lib.dh_beam_select(logits.data_ptr(), logits.stride(0), logits.stride(1), score.data_ptr(), _addr(finished),
                              R, W, vocab, M, dt, float(temperature), pad_token, parent.data_ptr(),
                              token.data_ptr(), best.data_ptr(), _addr(ws), nbytes, _raw_stream(index)),
           "dh_beam_select")
    if parent_out is not None or token_out is not None or score_out is not None:
        _written(parent_out, token_out, score_out)
    return parent, token, best


def _copy_dims(dims, unit):
    """(size, source stride, target stride) of the free dimensions, outer to inner, with those that
    lie next to each other in both tensors made one; the innermost ones that are contiguous become
    part of the unit (bytes).  Returns (unit, dims)."""
    dims = [d for d in dims if d[0] != 1]
    while dims and dims[-1][1] == unit and dims[-1][2] == unit:
        unit *= dims.pop()[0]
    out = []
    for d in dims:
        if out and out[-1][1] == d[0] * d[1] and out[-1][2] == d[0] * d[2]:
            out[-1] = (out[-1][0] * d[0], d[1], d[2])
        else:
            out.append(d)
    return unit, out


@functools.lru_cache(maxsize=256)
def _reorder_plan(shape, stride, out_shape, out_stride, size, request_dim, slot_dim, out_slot_dim, length_dim):
    """What the library is told of a layout: (A, R, source slots, target slots, H, T, unit bytes, byte
    strides of the source, of the target).  Goes by shapes and strides alone."""
    n = len(shape)
    if len(out_shape) != n:
        raise ValueError("out must have the number of dimensions of states")
    for name, d in (("request_dim", request_dim), ("slot_dim", slot_dim), ("out_slot_dim", out_slot_dim),
                    ("length_dim", 0 if length_dim is None else length_dim)):
        if not 0 <= d < n:
            raise ValueError(f"{name} must be in [0, {n})")
    if len({request_dim, slot_dim, length_dim}) != 3 or out_slot_dim == request_dim:
        raise ValueError("the request, slot and length dimensions must differ")
    free = [d for d in range(n) if d not in (request_dim, slot_dim)]
    out_free = [d for d in range(n) if d not in (request_dim, out_slot_dim)]
    if [shape[d] for d in free] != [out_shape[d] for d in out_free] or out_shape[request_dim] != shape[request_dim]:
        raise ValueError("states and out differ in more than their slots")
    reach = 0
    for st, s in sorted((st, s) for st, s in zip(out_stride, out_shape) if s > 1):
        if st <= reach:
            raise ValueError("the elements of out must be distinct (it is expanded or overlaps itself)")
        reach += st * (s - 1)
    dims = [(shape[a], stride[a] * size, out_stride[b] * size) for a, b in zip(free, out_free)]
    T, ts, td = 1, 0, 0
    if length_dim is not None:
        at = free.index(length_dim)
        T, ts, td = dims[at]
        unit, rest = _copy_dims(dims[at + 1:], size)
        outer = _copy_dims(dims[:at] + rest, None)[1]  # nothing more joins the unit
    else:
        unit, outer = _copy_dims(dims, size)
    if len(outer) > 2:
        raise ValueError("states: more than two separate dimensions besides requests, slots, positions and the "
                         "contiguous part; make the inner ones contiguous")
    (A, sa, da), (H, sh, dh) = [(1, 0, 0)] * (2 - len(outer)) + outer
    if max(A, H, T, shape[request_dim], shape[slot_dim], out_shape[out_slot_dim]) > _INT_MAX:
        raise ValueError("states: a dimension, or dimensions that lie together, of 2^31 elements or more")
    ss = (ctypes.c_int64 * 5)(sa, stride[request_dim] * size, stride[slot_dim] * size, sh, ts)
    ds = (ctypes.c_int64 * 5)(da, out_stride[request_dim] * size, out_stride[out_slot_dim] * size, dh, td)
    return A, shape[request_dim], shape[slot_dim], out_shape[out_slot_dim], H, T, unit, ss, ds


def reorder_states(states, idx, *, out=None, lengths=None, length_dim=None, src_base=None, dst_base=None, request_dim=1,
                   slot_dim=2, out_slot_dim=None, stream=None):
    """Slot dst_base[r] + j of request r takes slot src_base[r] + idx[r, j] (dh_reorder_states):
    beams' states after a selection, or an accepted path's states appended to the committed ones.

    states: any dtype, any dimensions among them requests (request_dim) and slots (slot_dim), e.g.
    [layers, R, beams, heads, positions, head size].  idx int32 [R, M]; negative entries and slots
    that do not exist are passed over.  lengths int32 [R] with length_dim: only the first lengths[r]
    entries of that dimension (the positions that a cache holds) are moved.  out: the tensor written
    (None: `states` itself, in place), whose slots are dimension out_slot_dim (slot_dim if not given)
    and whose other dimensions are those of `states`; what is not a target stays as it was.  Returns
    out."""
    lib = load_library()
    dst = states if out is None else out
    index = states.get_device()
    if index < 0:
        raise ValueError("states must be a CUDA tensor")
    if dst is not states and (dst.dtype != states.dtype or dst.is_neg() != states.is_neg()
                              or (dst.is_complex() and dst.is_conj() != states.is_conj())):
        raise ValueError("out must have the dtype of states (and be a conjugate or negated view only if they are)")
    if (states.requires_grad or dst.requires_grad) and torch.is_grad_enabled():
        raise ValueError("states are moved outside of autograd: detach them, or call under torch.no_grad()")
    if (lengths is None) != (length_dim is None):
        raise ValueError("lengths and length_dim come together")
    plan = _reorder_plan(states.shape, states.stride(), dst.shape, dst.stride(), states.element_size(), request_dim,
                         slot_dim, slot_dim if out_slot_dim is None else out_slot_dim, length_dim)
    A, R, slots, out_slots, H, T, unit, ss, ds = plan
    if idx.dim() != 2:
        raise ValueError("idx must be [R, M]")
    M = idx.shape[1]
    if M > _INT_MAX:
        raise ValueError("idx: M has to fit 32 bits")
    _typed(idx, "idx", torch.int32, (R, M), index)
    n = sb = db = None
    if lengths is not None:
        _typed(lengths, "lengths", torch.int32, (R,), index)
        n = lengths.data_ptr()
    if src_base is not None:
        _typed(src_base, "src_base", torch.int32, (R,), index)
        sb = src_base.data_ptr()
    if dst_base is not None:
        _typed(dst_base, "dst_base", torch.int32, (R,), index)
        db = dst_base.data_ptr()
    if dst is not states and dst.get_device() != index:
        raise ValueError(f"out must be on {states.device}")
    if stream is not None or index != torch.cuda.current_device():
        return _elsewhere(stream, states.device, (states, dst, idx, lengths, src_base, dst_base),
                          lambda: reorder_states(states, idx, out=out, lengths=lengths, length_dim=length_dim,
                                                 src_base=src_base, dst_base=dst_base, request_dim=request_dim,
                                                 slot_dim=slot_dim, out_slot_dim=out_slot_dim))
    _check(lib.dh_reorder_states(states.data_ptr(), ss, dst.data_ptr(), ds, idx.data_ptr(), n, sb, db, A, R, slots,
                                 out_slots, M, H, T, unit, _raw_stream(index)), "dh_reorder_states")
    _bump((dst,))
    return dst


def workspace_status(workspace: "Workspace | None" = None, device=None, stream=None) -> int:
    """Read and clear the device status words of a workspace object (OR over its buffers)."""
    lib = load_library()
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    status = 0
    for (d, _kind), ws in (workspace or _default_ws).buf.items():
        if d != dev:
            continue
        out = ctypes.c_int(0)
        _check(lib.dh_workspace_status(_ptr(ws), _stream(stream), ctypes.byref(out)), "dh_workspace_status")
        status |= out.value
    return status


def selftest_wait_timeout(limit_us: int = 50000, stream=None) -> int:
    """Run the bounded-wait self-test (an mbarrier wait that nothing completes) on a fresh workspace
    and return the status word it left (expected: 1 << DH_ERR_TIMEOUT)."""
    lib = load_library()
    with torch.cuda.stream(torch.cuda.current_stream() if stream is None else stream):
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    _check(lib.dh_selftest_wait_timeout(0, limit_us, _ptr(ws), 256, _stream(stream)),
           "dh_selftest_wait_timeout")
    out = ctypes.c_int(0)
    _check(lib.dh_workspace_status(_ptr(ws), _stream(stream), ctypes.byref(out)), "dh_workspace_status")
    return out.value


def selftest_distill_timeout(mode, row, limit_us, logits, idx, teacher, grad_loss):
    """distill_topk_step on fp32 rows with something held back from row `row` on and its waits limited to
    limit_us (dh_selftest_distill_timeout).  Returns (loss, gradient, status word; expected 1 <<
    DH_ERR_TIMEOUT where a wait gave up)."""
    lib = load_library()
    dt, index, N, vocab, K = _distill_inputs(logits, idx, teacher, None)
    _typed(grad_loss, "grad_loss", torch.float32, (N,), index)
    if dt != F32:
        raise TypeError("the self-test takes fp32 logits")
    dev = logits.device
    if index != torch.cuda.current_device():
        return _elsewhere(None, dev, (), lambda: selftest_distill_timeout(mode, row, limit_us, logits, idx, teacher,
                                                                          grad_loss))
    nbytes = lib.dh_distill_topk_step_workspace(N, vocab, K, dt)
    loss, grad = torch.empty(N, device=dev), _grad_rows(logits, None, index)
    ws = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=dev)
    _check(lib.dh_selftest_distill_timeout(mode, row, limit_us, logits.data_ptr(), logits.stride(0), idx.data_ptr(),
                                           teacher.data_ptr(), grad_loss.data_ptr(), N, vocab, K, 1.0, loss.data_ptr(),
                                           grad.data_ptr(), grad.stride(0), ws.data_ptr(), nbytes, _raw_stream(index)),
           "dh_selftest_distill_timeout")
    out = ctypes.c_int(0)
    _check(lib.dh_workspace_status(_ptr(ws), ctypes.c_void_p(_raw_stream(index)), ctypes.byref(out)),
           "dh_workspace_status")
    return loss, grad, out.value


def set_tuning(name: str, value: str | None):
    """Set one test or tuning switch (kernel choice only; None restores the default)."""
    lib = load_library()
    _check(lib.dh_set_tuning(name.encode(), None if value is None else str(value).encode()), "dh_set_tuning")


def prof_enable(on: bool):
    load_library().dh_prof_enable(1 if on else 0)


def prof_read(max_kernels: int = 64) -> dict:
    """{kernel name: (total ms, launches)} recorded since the last read (waits for the events)."""
    lib = load_library()
    L = 64
    names = ctypes.create_string_buffer(L * max_kernels)
    tot = (ctypes.c_double * max_kernels)()
    cnt = (ctypes.c_int * max_kernels)()
    n = lib.dh_prof_read(names, L, tot, cnt, max_kernels)
    if n < 0:
        raise DhError(4, "dh_prof_read")
    out = {}
    for k in range(min(n, max_kernels)):
        nm = names.raw[k * L:(k + 1) * L].split(b"\0", 1)[0].decode()
        out[nm] = (tot[k], cnt[k])
    return out

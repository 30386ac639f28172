"""ctypes binding of libpctree.so (argument marshalling only).

Every step of the hot path runs in the library's CUDA kernels; this module only
checks shapes, allocates outputs and workspace with torch on the inputs' device,
and passes raw pointers plus the current CUDA stream. If the shared library is
missing it raises instead of falling back to anything else.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpctree.so")

PCT_OK, PCT_EINVAL, PCT_EWORKSPACE, PCT_ECUDA, PCT_EDEVICE, PCT_ETIMEOUT, PCT_EUNSUPPORTED = range(7)
PCT_F32, PCT_BF16 = 0, 1
DEV_BAD_PARENT, DEV_BAD_TOKEN, DEV_BAD_COUNT, DEV_DEPTH_OVERFLOW, DEV_BAD_COST, DEV_TIMEOUT = (
    1, 2, 4, 8, 16, 32)
DEV_BAD_PAGE, DEV_NO_PAGE, DEV_BAD_LENGTH, DEV_BAD_PATH = 64, 128, 256, 512
_NAMES = {0: "PCT_OK", 1: "PCT_EINVAL", 2: "PCT_EWORKSPACE", 3: "PCT_ECUDA", 4: "PCT_EDEVICE",
          5: "PCT_ETIMEOUT", 6: "PCT_EUNSUPPORTED"}

EXPORTED = [
    "pct_tree_build_workspace", "pct_tree_build", "pct_score_parents_workspace",
    "pct_score_parents", "cadd_tree_grow_workspace", "cadd_tree_grow", "tree_ancestor_mask",
    "tree_verify_accept_workspace", "tree_verify_accept", "pct_trace_enable", "pct_trace_reset",
    "pct_trace_read", "pct_version", "tree_verify_accept_noalloc", "tree_verify_walk",
    "tree_accept_sim",
    "cadd_cost_fit", "pct_tree_build_seeded", "cadd_tree_grow_topk", "pct_markov_rank_pad",
    "pct_markov_transpose", "kv_pages_resize", "kv_tree_slots", "kv_append",
    "tree_attention_workspace", "tree_attention", "kv_commit",
]


class PctError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what} returned {_NAMES.get(code, code)}")
        self.code = code


class BuildDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("depth", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("rank", ctypes.c_int32), ("k", ctypes.c_int32), ("beam", ctypes.c_int32),
                ("n_nodes", ctypes.c_int32), ("logits_dtype", ctypes.c_int32),
                ("markov_dtype", ctypes.c_int32)]


class CaddDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("depth", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("n_max", ctypes.c_int32), ("logits_dtype", ctypes.c_int32),
                ("C_d", ctypes.c_float), ("a", ctypes.c_float), ("b", ctypes.c_float),
                ("c", ctypes.c_float), ("e", ctypes.c_float)]


class KvCacheDesc(ctypes.Structure):
    _fields_ = [("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("heads_kv", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("page_stride", ctypes.c_int64), ("slot_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libpctree.so from the package directory (raises if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing; build it with "
                          "`python -m speculative_decoding_draft_07_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    bd, cd = ctypes.POINTER(BuildDesc), ctypes.POINTER(CaddDesc)
    kd = ctypes.POINTER(KvCacheDesc)
    sig = {
        "pct_tree_build_workspace": (sz, [bd]),
        "pct_tree_build": (i32, [bd, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "pct_score_parents_workspace": (sz, [bd, i32]),
        "pct_score_parents": (i32, [bd, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "cadd_tree_grow_workspace": (sz, [cd]),
        "cadd_tree_grow": (i32, [cd, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "tree_ancestor_mask": (i32, [i32, i32, vp, vp, vp, vp, vp]),
        "tree_verify_accept_workspace": (sz, [i32, i32]),
        "tree_verify_accept": (i32, [i32, i32, i32, i32, vp, vp, vp, vp, i32, vp, vp, vp, vp,
                                     vp, vp, sz, vp]),
        "pct_trace_enable": (i32, [i32]),
        "pct_trace_reset": (i32, []),
        "pct_trace_read": (i32, [ctypes.c_char_p, i32, vp, vp, i32]),
        "pct_version": (ctypes.c_char_p, []),
        "tree_verify_accept_noalloc": (i32, [i32, i32, i32, i32, vp, vp, vp, vp, i32, vp, vp, vp,
                                             vp, vp, vp]),
        "tree_verify_walk": (i32, [i32, i32, i32, i32, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp]),
        "tree_accept_sim": (i32, [i32, i32, i32, vp, vp, vp, ctypes.c_int64, ctypes.c_uint64, vp,
                                  vp, vp]),
        "cadd_cost_fit": (i32, [ctypes.c_int64, vp, vp, vp, vp, vp, vp]),
        "pct_tree_build_seeded": (i32, [bd, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                        sz, vp]),
        "pct_markov_rank_pad": (i32, [i32]),
        "pct_markov_transpose": (i32, [i32, i32, vp, vp, vp]),
        "cadd_tree_grow_topk": (i32, [cd, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                      sz, vp]),
        "kv_pages_resize": (i32, [i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp]),
        "kv_tree_slots": (i32, [i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp]),
        "kv_append": (i32, [kd, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp]),
        "tree_attention_workspace": (sz, [kd, i32, i32, i32]),
        "tree_attention": (i32, [kd, i32, i32, i32, ctypes.c_float, vp, vp, vp, vp, vp, vp, vp, vp,
                                 vp, vp, vp, vp, sz, vp]),
        "kv_commit": (i32, [kd, i32, i32, ctypes.c_int64, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                            vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype, f.argtypes = res, args
    _lib = L
    return L


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return PCT_BF16
    if t.dtype == torch.float32:
        return PCT_F32
    raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")


def _check(t: torch.Tensor, name: str, dev: torch.device, shape=None, dtype=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")


def _workspace(nbytes: int, dev, ws: Optional[torch.Tensor]):
    if nbytes == 0:
        return None, 0
    if ws is not None:
        if ws.numel() * ws.element_size() < nbytes:
            raise ValueError(f"workspace has {ws.numel() * ws.element_size()} bytes, needs {nbytes}")
        return ws, ws.numel() * ws.element_size()
    return torch.empty(nbytes, dtype=torch.uint8, device=dev), nbytes


def _raise(code: int, what: str):
    if code != PCT_OK:
        raise PctError(code, what)


@dataclass
class TreeOut:
    tok: torch.Tensor
    parent: torch.Tensor
    depth: torch.Tensor
    score: torch.Tensor
    count: torch.Tensor
    status: torch.Tensor
    phi: Optional[torch.Tensor] = None


def build_desc(batch, depth, vocab, rank, k, beam, n_nodes, logits_dtype, markov_dtype) -> BuildDesc:
    return BuildDesc(batch, depth, vocab, rank, k, beam, n_nodes, logits_dtype, markov_dtype)


def pct_tree_build_workspace(desc: BuildDesc) -> int:
    return int(lib().pct_tree_build_workspace(ctypes.byref(desc)))


def pct_tree_build(L: torch.Tensor, anchor: torch.Tensor, E: torch.Tensor, W: torch.Tensor,
                   k: int, beam: int, n_nodes: int, out: Optional[TreeOut] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None,
                   seeds: Optional[torch.Tensor] = None,
                   Wt: Optional[torch.Tensor] = None) -> TreeOut:
    """PCTree for a batch of requests. L [batch][D][V], anchor [batch] int32,
    E [V][r], W [r][V]; returns node tables [batch][N] in canonical BFS order.
    seeds [batch][D][k] int32 (optional): the columns that seed each row's top-k
    gate (pct_tree_build_seeded), e.g. cadd_tree_grow's top_tok for the same L;
    the result does not depend on them. Wt (optional, with seeds):
    markov_transpose(W), read for the seeds' W columns."""
    dev = L.device
    batch, D, V = L.shape
    r = E.shape[1]
    _check(L, "L", dev)
    _check(anchor, "anchor", dev, (batch,), torch.int32)
    _check(E, "E", dev, (V, r))
    _check(W, "W", dev, (r, V), E.dtype)
    desc = build_desc(batch, D, V, r, k, beam, n_nodes, _code(L), _code(E))
    if out is None:
        out = TreeOut(*(torch.empty((batch, n_nodes), dtype=torch.int32, device=dev) for _ in range(3)),
                      torch.empty((batch, n_nodes), dtype=torch.float32, device=dev),
                      torch.empty(batch, dtype=torch.int32, device=dev),
                      torch.empty(batch, dtype=torch.int32, device=dev))
    nbytes = pct_tree_build_workspace(desc)
    if nbytes == 0:
        _raise(PCT_EINVAL, "pct_tree_build_workspace")
    ws, wsb = _workspace(nbytes, dev, workspace)
    if seeds is not None:
        _check(seeds, "seeds", dev, (batch, D, k), torch.int32)
        if Wt is not None:
            _check(Wt, "Wt", dev, (V, int(lib().pct_markov_rank_pad(r))), torch.bfloat16)
        code = lib().pct_tree_build_seeded(ctypes.byref(desc), _p(L), _p(anchor), _p(E), _p(W),
                                           _p(Wt), _p(seeds), _p(out.tok), _p(out.parent),
                                           _p(out.depth), _p(out.score), _p(out.count),
                                           _p(out.status), _p(ws), wsb, _stream(stream))
        _raise(code, "pct_tree_build_seeded")
        return out
    code = lib().pct_tree_build(ctypes.byref(desc), _p(L), _p(anchor), _p(E), _p(W), _p(out.tok),
                                _p(out.parent), _p(out.depth), _p(out.score), _p(out.count),
                                _p(out.status), _p(ws), wsb, _stream(stream))
    _raise(code, "pct_tree_build")
    return out


def markov_transpose(W: torch.Tensor, stream=None) -> torch.Tensor:
    """Wt [V][r_pad] bf16: W [r][V] bf16 transposed, zero past r (once per model)."""
    dev = W.device
    r, V = W.shape
    _check(W, "W", dev, dtype=torch.bfloat16)
    r_pad = int(lib().pct_markov_rank_pad(r))
    if r_pad == 0:
        _raise(PCT_EINVAL, "pct_markov_rank_pad")
    Wt = torch.empty((V, r_pad), dtype=torch.bfloat16, device=dev)
    _raise(lib().pct_markov_transpose(V, r, _p(W), _p(Wt), _stream(stream)), "pct_markov_transpose")
    return Wt


def pct_score_parents(L_row: torch.Tensor, parent_tok: torch.Tensor, E: torch.Tensor,
                      W: torch.Tensor, k: int, stream=None):
    """One depth of batched parent scoring: returns (lse [b][p], top_tok [b][p][k],
    top_logpi [b][p][k], status [b])."""
    dev = L_row.device
    batch, V = L_row.shape
    n_par = parent_tok.shape[1]
    r = E.shape[1]
    _check(L_row, "L_row", dev)
    _check(parent_tok, "parent_tok", dev, (batch, n_par), torch.int32)
    _check(E, "E", dev, (V, r))
    _check(W, "W", dev, (r, V), E.dtype)
    desc = build_desc(batch, 1, V, r, k, 1, 1, _code(L_row), _code(E))
    nbytes = int(lib().pct_score_parents_workspace(ctypes.byref(desc), n_par))
    if nbytes == 0:
        _raise(PCT_EINVAL, "pct_score_parents_workspace")
    ws, wsb = _workspace(nbytes, dev, None)
    lse = torch.empty((batch, n_par), dtype=torch.float32, device=dev)
    tt = torch.empty((batch, n_par, k), dtype=torch.int32, device=dev)
    tl = torch.empty((batch, n_par, k), dtype=torch.float32, device=dev)
    st = torch.empty(batch, dtype=torch.int32, device=dev)
    code = lib().pct_score_parents(ctypes.byref(desc), n_par, _p(L_row), _p(parent_tok), _p(E),
                                   _p(W), _p(lse), _p(tt), _p(tl), _p(st), _p(ws), wsb,
                                   _stream(stream))
    _raise(code, "pct_score_parents")
    return lse, tt, tl, st


def cadd_desc(batch, depth, vocab, n_max, logits_dtype, C_d, a, b, c, e) -> CaddDesc:
    return CaddDesc(batch, depth, vocab, n_max, logits_dtype, C_d, a, b, c, e)


def cadd_tree_grow(L: torch.Tensor, anchor: torch.Tensor, ctx_len: torch.Tensor, n_max: int,
                   C_d: float, a: float, b: float, c: float, e: float,
                   out: Optional[TreeOut] = None, workspace: Optional[torch.Tensor] = None,
                   stream=None, top_tok: Optional[torch.Tensor] = None) -> TreeOut:
    """CaDDTree for a batch of requests. L [batch][D][V] marginal logits,
    anchor [batch] int32, ctx_len [batch] int64; node tables [batch][n_max].
    top_tok [batch][D][top_k] int32 (optional, top_k 1..32): also written with
    each row's top_k tokens by logit (value desc, token asc), cadd_tree_grow_topk."""
    dev = L.device
    batch, D, V = L.shape
    _check(L, "L", dev)
    _check(anchor, "anchor", dev, (batch,), torch.int32)
    _check(ctx_len, "ctx_len", dev, (batch,), torch.int64)
    desc = cadd_desc(batch, D, V, n_max, _code(L), C_d, a, b, c, e)
    if out is None:
        out = TreeOut(*(torch.empty((batch, n_max), dtype=torch.int32, device=dev) for _ in range(3)),
                      torch.empty((batch, n_max), dtype=torch.float32, device=dev),
                      torch.empty(batch, dtype=torch.int32, device=dev),
                      torch.empty(batch, dtype=torch.int32, device=dev),
                      torch.empty(batch, dtype=torch.float32, device=dev))
    nbytes = int(lib().cadd_tree_grow_workspace(ctypes.byref(desc)))
    if nbytes == 0:
        _raise(PCT_EINVAL, "cadd_tree_grow_workspace")
    ws, wsb = _workspace(nbytes, dev, workspace)
    if top_tok is not None:
        if top_tok.dim() != 3:
            raise ValueError("top_tok must be [batch][D][top_k]")
        _check(top_tok, "top_tok", dev, (batch, D, top_tok.shape[2]), torch.int32)
        code = lib().cadd_tree_grow_topk(ctypes.byref(desc), _p(L), _p(anchor), _p(ctx_len),
                                         int(top_tok.shape[2]), _p(out.tok), _p(out.parent),
                                         _p(out.depth), _p(out.score), _p(out.count), _p(out.phi),
                                         _p(top_tok), _p(out.status), _p(ws), wsb, _stream(stream))
        _raise(code, "cadd_tree_grow_topk")
        return out
    code = lib().cadd_tree_grow(ctypes.byref(desc), _p(L), _p(anchor), _p(ctx_len), _p(out.tok),
                                _p(out.parent), _p(out.depth), _p(out.score), _p(out.count),
                                _p(out.phi), _p(out.status), _p(ws), wsb, _stream(stream))
    _raise(code, "cadd_tree_grow")
    return out


def tree_ancestor_mask(parent: torch.Tensor, count: torch.Tensor, mask: Optional[torch.Tensor] = None,
                       status: Optional[torch.Tensor] = None, stream=None):
    """Self-plus-ancestor bitmask [batch][n_stride][ceil(n_stride/32)] (int32 view of uint32)."""
    dev = parent.device
    batch, n_stride = parent.shape
    _check(parent, "parent", dev, dtype=torch.int32)
    _check(count, "count", dev, (batch,), torch.int32)
    words = (n_stride + 31) // 32
    if mask is None:
        mask = torch.empty((batch, n_stride, words), dtype=torch.int32, device=dev)
    if status is None:
        status = torch.empty(batch, dtype=torch.int32, device=dev)
    code = lib().tree_ancestor_mask(batch, n_stride, _p(parent), _p(count), _p(mask), _p(status),
                                    _stream(stream))
    _raise(code, "tree_ancestor_mask")
    return mask, status


@dataclass
class VerifyOut:
    argmax: torch.Tensor
    accept_len: torch.Tensor
    accept_path: torch.Tensor
    correction: torch.Tensor
    status: torch.Tensor


def tree_verify_accept(tok: torch.Tensor, parent: torch.Tensor, count: torch.Tensor,
                       target: torch.Tensor, max_depth: int, out: Optional[VerifyOut] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> VerifyOut:
    """Greedy verification of node tables against target logits [batch][n_stride][V]."""
    dev = tok.device
    batch, n_stride = tok.shape
    V = target.shape[2]
    _check(tok, "tok", dev, dtype=torch.int32)
    _check(parent, "parent", dev, (batch, n_stride), torch.int32)
    _check(count, "count", dev, (batch,), torch.int32)
    _check(target, "target", dev, (batch, n_stride, V))
    if out is None:
        out = VerifyOut(torch.empty((batch, n_stride), dtype=torch.int32, device=dev),
                        torch.empty(batch, dtype=torch.int32, device=dev),
                        torch.empty((batch, max_depth), dtype=torch.int32, device=dev),
                        torch.empty(batch, dtype=torch.int32, device=dev),
                        torch.empty(batch, dtype=torch.int32, device=dev))
    nbytes = int(lib().tree_verify_accept_workspace(batch, n_stride))
    ws, wsb = _workspace(nbytes, dev, workspace)
    code = lib().tree_verify_accept(batch, n_stride, V, max_depth, _p(tok), _p(parent), _p(count),
                                    _p(target), _code(target), _p(out.argmax), _p(out.accept_len),
                                    _p(out.accept_path), _p(out.correction), _p(out.status),
                                    _p(ws), wsb, _stream(stream))
    _raise(code, "tree_verify_accept")
    return out


def tree_verify_walk(tok: torch.Tensor, parent: torch.Tensor, count: torch.Tensor,
                     target: torch.Tensor, max_depth: int, out: Optional[VerifyOut] = None,
                     stream=None) -> VerifyOut:
    """Greedy verification reading only the rows the walk reaches: the same
    accept_len, accept_path and correction as tree_verify_accept; argmax holds
    the walked rows' argmax and -1 elsewhere."""
    dev = tok.device
    batch, n_stride = tok.shape
    V = target.shape[2]
    _check(tok, "tok", dev, dtype=torch.int32)
    _check(parent, "parent", dev, (batch, n_stride), torch.int32)
    _check(count, "count", dev, (batch,), torch.int32)
    _check(target, "target", dev, (batch, n_stride, V))
    if out is None:
        out = VerifyOut(torch.empty((batch, n_stride), dtype=torch.int32, device=dev),
                        torch.empty(batch, dtype=torch.int32, device=dev),
                        torch.empty((batch, max_depth), dtype=torch.int32, device=dev),
                        torch.empty(batch, dtype=torch.int32, device=dev),
                        torch.empty(batch, dtype=torch.int32, device=dev))
    code = lib().tree_verify_walk(batch, n_stride, V, max_depth, _p(tok), _p(parent), _p(count),
                                  _p(target), _code(target), _p(out.argmax), _p(out.accept_len),
                                  _p(out.accept_path), _p(out.correction), _p(out.status),
                                  _stream(stream))
    _raise(code, "tree_verify_walk")
    return out


def tree_accept_sim(parent: torch.Tensor, count: torch.Tensor, p_child: torch.Tensor,
                    trials: int, seed: int, max_depth: int, stream=None):
    """Monte Carlo walks of greedy verification: (hist [batch][max_depth + 1]
    int64 walks per accepted length, status [batch])."""
    dev = parent.device
    batch, n_stride = parent.shape
    _check(parent, "parent", dev, dtype=torch.int32)
    _check(count, "count", dev, (batch,), torch.int32)
    _check(p_child, "p_child", dev, (batch, n_stride), torch.float32)
    hist = torch.empty((batch, max_depth + 1), dtype=torch.int64, device=dev)
    status = torch.empty(batch, dtype=torch.int32, device=dev)
    code = lib().tree_accept_sim(batch, n_stride, max_depth, _p(parent), _p(count), _p(p_child),
                                 int(trials), int(seed) & ((1 << 64) - 1), _p(hist), _p(status),
                                 _stream(stream))
    _raise(code, "tree_accept_sim")
    return hist, status


def cadd_cost_fit(n: torch.Tensor, ell: torch.Tensor, lat: torch.Tensor, stream=None):
    """Non-negative fit of C_v(n; l) = a + b l + c n + e n^2 to latency samples:
    (out float64 [5] = a, b, c, e, rms; status [1])."""
    dev = n.device
    m = n.numel()
    _check(n, "n", dev, (m,), torch.float32)
    _check(ell, "ell", dev, (m,), torch.float32)
    _check(lat, "lat", dev, (m,), torch.float32)
    out = torch.empty(5, dtype=torch.float64, device=dev)
    status = torch.empty(1, dtype=torch.int32, device=dev)
    code = lib().cadd_cost_fit(m, _p(n), _p(ell), _p(lat), _p(out), _p(status), _stream(stream))
    _raise(code, "cadd_cost_fit")
    return out, status


# ---------------------------------------------------------------------------
# Paged key-value cache. Unlike the calls above, these take strided views where
# the ABI does, make the tensors' device current for the call when it is not,
# and allocate their outputs and workspace on the stream they run on. Several run
# once a layer or a round with little GPU work behind them, so the checks take one
# fast look first, and what follows from shapes and strides alone (descriptors,
# stride arrays, workspace sizes) is worked out once per combination.
_HERE_ALREADY = contextlib.nullcontext()
_I32, _I64, _F32 = torch.int32, torch.int64, torch.float32


def _on(t: torch.Tensor, name: str, stream):
    """(device, stream handle, context to allocate and launch in) for work on t's device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dev, index = t.device, t.get_device()
    if not t.is_cuda:
        raise ValueError(f"{name} is on {dev}, expected a CUDA device")
    if stream is None:
        if index == torch._C._cuda_getDevice():
            return dev, torch._C._cuda_getCurrentRawStream(index), _HERE_ALREADY
        stream = torch.cuda.current_stream(dev)
    elif stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, {name} on {dev}")
    return dev, stream.cuda_stream, torch.cuda.stream(stream)


def _want(t: torch.Tensor, name: str, dev: torch.device, shape, dtype):
    """_check, with the common case first (dev is a CUDA device)."""
    try:
        if (t.dtype is dtype and t.get_device() == dev.index and t.shape == shape
                and t.is_contiguous()):
            return
    except AttributeError:
        pass
    _check(t, name, dev, shape, dtype)


def _given(t: Optional[torch.Tensor], name: str, dev: torch.device, shape, dtype) -> torch.Tensor:
    """The caller's output tensor, checked, or a new one."""
    if t is None:   # (sizes one by one: taken apart faster than a tuple)
        return torch.empty(*shape, dtype=dtype, device=dev)
    _want(t, name, dev, shape, dtype)
    return t


def _rows(t: torch.Tensor, name: str, dev: torch.device, dtype):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-dimensional tensor")
    if not (t.dtype is dtype and t.device == dev and t.is_contiguous()):
        _check(t, name, dev, dtype=dtype)
    return t.shape


@functools.lru_cache(maxsize=1024)
def _strides(shape, stride, name: str):
    """The element strides of all but the last axis of a view whose last axis is
    contiguous (0 for an axis of one entry, which is never stepped over), as an array."""
    if stride[-1] != 1 and shape[-1] != 1:
        raise ValueError(f"{name} must be contiguous along its last axis")
    st = [0 if n == 1 else x for n, x in zip(shape[:-1], stride[:-1])]
    return (ctypes.c_int64 * len(st))(*st)


def _view(t: torch.Tensor, name: str, dev: torch.device, shape, dtype):
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.device == dev):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    return _strides(t.shape, t.stride(), name)


@functools.lru_cache(maxsize=1024)
def _cache_desc(shape, stride, code: int, max_pages: int):
    """(descriptor, a reference to it, layer stride) of a cache's shape and strides."""
    st = list(_strides(shape, stride, "k_cache"))
    d = KvCacheDesc(*shape[-4:-2], max_pages, *shape[-2:], code, *st[-3:])
    return d, ctypes.byref(d), st[0] if len(shape) == 5 else 0


def _cache(k_cache: torch.Tensor, v_cache: torch.Tensor, dev: torch.device, max_pages: int,
           layered: bool = False):
    """_cache_desc of K and V caches [layers][n_pages][page_size][heads][head_dim] (no layer
    axis unless `layered`)."""
    _same_caches(k_cache, v_cache, dev, 5 if layered else 4)
    return _cache_desc(k_cache.shape, k_cache.stride(), _code(k_cache), max_pages)


def _same_caches(k_cache: torch.Tensor, v_cache: torch.Tensor, dev: torch.device, dims: int):
    """K and V caches of `dims` axes on dev, of a supported dtype, laid out alike."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != dims:
        raise ValueError("k_cache must be a %d-dimensional tensor" % dims)
    if k_cache.device != dev:
        raise ValueError(f"k_cache is on {k_cache.device}, expected {dev}")
    _code(k_cache)
    shape, stride = k_cache.shape, k_cache.stride()
    if not (isinstance(v_cache, torch.Tensor) and v_cache.dtype is k_cache.dtype
            and v_cache.get_device() == dev.index and v_cache.shape == shape
            and v_cache.stride() == stride):
        st = _view(v_cache, "v_cache", dev, shape, k_cache.dtype)
        if list(st) != list(_strides(shape, stride, "k_cache")):
            raise ValueError("k_cache and v_cache must have the same strides")


def kv_pages_resize(ctx_len: torch.Tensor, block_table: torch.Tensor, held: torch.Tensor,
                    free_pages: torch.Tensor, free_count: torch.Tensor, page_size: int,
                    count: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """Block tables [batch][max_pages] int32 grown and shrunk in place to
    ceil((ctx_len + count) / page_size) pages a request, with pages from and back to
    free_pages[:free_count] (int32 [n_pages] and [1]); held [batch] int32 counts each
    request's pages. ctx_len [batch] int64, count [batch] int32. Returns status [batch]."""
    dev, s, ctx = _on(block_table, "block_table", stream)
    batch, max_pages = _rows(block_table, "block_table", dev, _I32)
    _want(ctx_len, "ctx_len", dev, (batch,), _I64)
    _want(held, "held", dev, (batch,), _I32)
    if not isinstance(free_pages, torch.Tensor) or free_pages.dim() != 1:
        raise ValueError("free_pages must be a 1-dimensional tensor")
    _want(free_pages, "free_pages", dev, free_pages.shape, _I32)
    _want(free_count, "free_count", dev, (1,), _I32)
    if count is not None:
        _want(count, "count", dev, (batch,), _I32)
    with ctx:
        status = _given(status, "status", dev, (batch,), _I32)
        code = lib().kv_pages_resize(batch, page_size, max_pages, free_pages.shape[0],
                                     ctx_len.data_ptr(),
                                     None if count is None else count.data_ptr(),
                                     block_table.data_ptr(), held.data_ptr(),
                                     free_pages.data_ptr(), free_count.data_ptr(),
                                     status.data_ptr(), s)
    _raise(code, "kv_pages_resize")
    return status


def kv_tree_slots(ctx_len: torch.Tensor, count: torch.Tensor, block_table: torch.Tensor,
                  n_stride: int, page_size: int, n_pages: int,
                  depth: Optional[torch.Tensor] = None, slot: Optional[torch.Tensor] = None,
                  pos: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                  stream=None):
    """(slot, pos, status): cache slots and positions [batch][n_stride] int64 of the
    count[b] tokens after ctx_len[b]; depth [batch][n_stride] int32 (a tree's node
    depths) makes siblings share a position, None is a chain."""
    dev, s, ctx = _on(block_table, "block_table", stream)
    batch, max_pages = _rows(block_table, "block_table", dev, _I32)
    _want(ctx_len, "ctx_len", dev, (batch,), _I64)
    _want(count, "count", dev, (batch,), _I32)
    if depth is not None:
        _want(depth, "depth", dev, (batch, n_stride), _I32)
    with ctx:
        slot = _given(slot, "slot", dev, (batch, n_stride), _I64)
        pos = _given(pos, "pos", dev, (batch, n_stride), _I64)
        status = _given(status, "status", dev, (batch,), _I32)
        code = lib().kv_tree_slots(batch, n_stride, page_size, max_pages, n_pages,
                                   ctx_len.data_ptr(), count.data_ptr(),
                                   None if depth is None else depth.data_ptr(),
                                   block_table.data_ptr(), slot.data_ptr(), pos.data_ptr(),
                                   status.data_ptr(), s)
    _raise(code, "kv_tree_slots")
    return slot, pos, status


def kv_append(k_new: torch.Tensor, v_new: torch.Tensor, slot: torch.Tensor, k_cache: torch.Tensor,
              v_cache: torch.Tensor, status: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """Rows k_new, v_new [batch][n_stride][heads][head_dim] (views with a contiguous
    last axis and equal strides) into the caches [n_pages][page_size][heads][head_dim] at
    slot [batch][n_stride] int64 (negative: skipped). Returns status [batch]."""
    dev, s, ctx = _on(k_cache, "k_cache", stream)
    desc, ref, _ = _cache(k_cache, v_cache, dev, 1)
    batch, n = _rows(slot, "slot", dev, _I64)
    shape = (batch, n, desc.heads_kv, desc.head_dim)
    st = _view(k_new, "k_new", dev, shape, k_cache.dtype)
    st_v = _view(v_new, "v_new", dev, shape, k_cache.dtype)
    if st_v is not st and list(st_v) != list(st):
        raise ValueError("k_new and v_new must have the same strides")
    with ctx:
        status = _given(status, "status", dev, (batch,), _I32)
        code = lib().kv_append(ref, batch, n, k_new.data_ptr(), v_new.data_ptr(), st,
                               slot.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                               status.data_ptr(), s)
    _raise(code, "kv_append")
    return status


@dataclass
class AttnOut:
    out: torch.Tensor
    lse: torch.Tensor
    status: torch.Tensor


@functools.lru_cache(maxsize=1024)
def _attn_workspace(shape, stride, code: int, max_pages: int, batch: int, n_stride: int,
                    heads_q: int, device: int) -> int:
    ref = _cache_desc(shape, stride, code, max_pages)[1]
    with torch.cuda.device(device):   # the pieces of the work follow that device's size
        return int(lib().tree_attention_workspace(ref, batch, n_stride, heads_q))


@functools.lru_cache(maxsize=1024)
def _attn_plan(q_shape, q_stride, shape, stride, dtype, max_pages: int, device: int):
    """(reference to the cache's descriptor, query strides, workspace bytes) of an attention
    call, which the shapes and strides of its tensors alone decide."""
    code = PCT_BF16 if dtype is torch.bfloat16 else PCT_F32
    _, ref, _ = _cache_desc(shape, stride, code, max_pages)
    batch, n, hq, _ = q_shape
    nbytes = _attn_workspace(shape, stride, code, max_pages, batch, n, hq, device)
    if nbytes == 0:
        _raise(PCT_EINVAL, "tree_attention_workspace")
    return ref, _strides(q_shape, q_stride, "q"), nbytes


def tree_attention_workspace(k_cache: torch.Tensor, v_cache: torch.Tensor, max_pages: int,
                             batch: int, n_stride: int, heads_q: int) -> int:
    """Workspace bytes tree_attention needs for these shapes on the caches' device."""
    dev, _, _ = _on(k_cache, "k_cache", None)
    _cache(k_cache, v_cache, dev, max_pages)
    return _attn_workspace(k_cache.shape, k_cache.stride(), _code(k_cache), max_pages, batch,
                           n_stride, heads_q, k_cache.get_device())


def tree_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   block_table: torch.Tensor, ctx_len: torch.Tensor,
                   count: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
                   scale: Optional[float] = None, out: Optional[AttnOut] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> AttnOut:
    """Attention of a tree's nodes over the paged cache. q [batch][n_stride][heads_q][head_dim]
    (a view with a contiguous last axis), caches [n_pages][page_size][heads_kv][head_dim] that
    hold the nodes' K and V as tokens ctx_len + i, block_table [batch][max_pages] int32,
    ctx_len [batch] int64, count [batch] int32 (None: n_stride for all), mask the words of
    tree_ancestor_mask [batch][n_stride][ceil(n_stride / 32)] int32 (None: a causal chain; a
    decode step with n_stride = 1). scale defaults to head_dim ** -0.5. Rows at or past count
    are 0, their lse -inf. bf16 inputs: the softmax's weights are rounded to bf16 for the product
    with V (off by at most 2^-8 each; sums and lse are fp32); fp32 inputs are not rounded. With
    out given, out.lse may be None. Outputs and workspace do not overlap inputs."""
    dev, s, ctx = _on(q, "q", stream)
    if q.dim() != 4:
        raise ValueError("q must be [batch][n_stride][heads_q][head_dim]")
    batch, n, hq, d = q.shape
    rows, max_pages = _rows(block_table, "block_table", dev, _I32)
    if rows != batch:
        raise ValueError(f"block_table has {rows} rows, expected {batch}")
    _same_caches(k_cache, v_cache, dev, 4)
    if q.dtype is not k_cache.dtype or k_cache.shape[3] != d:
        _view(q, "q", dev, (batch, n, hq, k_cache.shape[3]), k_cache.dtype)
    ref, st, nbytes = _attn_plan(q.shape, q.stride(), k_cache.shape, k_cache.stride(), q.dtype,
                                 max_pages, q.get_device())
    _want(ctx_len, "ctx_len", dev, (batch,), _I64)
    if count is not None:
        _want(count, "count", dev, (batch,), _I32)
    if mask is not None:
        _want(mask, "mask", dev, (batch, n, (n + 31) // 32), _I32)
    with ctx:
        if out is None:
            out = AttnOut(torch.empty(batch, n, hq, d, dtype=q.dtype, device=dev),
                          torch.empty(batch, n, hq, dtype=_F32, device=dev),
                          torch.empty(batch, dtype=_I32, device=dev))
        else:
            _want(out.out, "out.out", dev, (batch, n, hq, d), q.dtype)
            if out.lse is not None:
                _want(out.lse, "out.lse", dev, (batch, n, hq), _F32)
            _want(out.status, "out.status", dev, (batch,), _I32)
        if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()):
            raise ValueError(f"workspace must be contiguous on {dev}")
        ws, wsb = _workspace(nbytes, dev, workspace)
        code = lib().tree_attention(ref, batch, n, hq, d ** -0.5 if scale is None else scale,
                                    q.data_ptr(), st, k_cache.data_ptr(), v_cache.data_ptr(),
                                    block_table.data_ptr(), ctx_len.data_ptr(),
                                    None if count is None else count.data_ptr(),
                                    None if mask is None else mask.data_ptr(), out.out.data_ptr(),
                                    None if out.lse is None else out.lse.data_ptr(),
                                    out.status.data_ptr(), ws.data_ptr(), wsb, s)
    _raise(code, "tree_attention")
    return out


def kv_commit(k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
              ctx_len: torch.Tensor, count: torch.Tensor, accept_len: torch.Tensor,
              accept_path: torch.Tensor, new_len: Optional[torch.Tensor] = None,
              status: Optional[torch.Tensor] = None, stream=None):
    """(new_len [batch] int64, status): the accepted nodes' K and V (accept_len [batch],
    accept_path [batch][max_depth] int32, as tree_verify_accept writes them) move behind the
    root in every layer of the caches [layers][n_pages][page_size][heads][head_dim] (or one
    layer without that axis), in place; new_len = ctx_len + 1 + accept_len."""
    dev, s, ctx = _on(k_cache, "k_cache", stream)
    batch, max_pages = _rows(block_table, "block_table", dev, _I32)
    layered = k_cache.dim() == 5
    _, ref, layer_stride = _cache(k_cache, v_cache, dev, max_pages, layered)
    _want(ctx_len, "ctx_len", dev, (batch,), _I64)
    _want(count, "count", dev, (batch,), _I32)
    _want(accept_len, "accept_len", dev, (batch,), _I32)
    rows, max_depth = _rows(accept_path, "accept_path", dev, _I32)
    if rows != batch:
        raise ValueError(f"accept_path has {rows} rows, expected {batch}")
    with ctx:
        new_len = _given(new_len, "new_len", dev, (batch,), _I64)
        if new_len.data_ptr() == ctx_len.data_ptr():
            raise ValueError("new_len must not be ctx_len")
        status = _given(status, "status", dev, (batch,), _I32)
        code = lib().kv_commit(ref, batch, k_cache.shape[0] if layered else 1, layer_stride,
                               max_depth, k_cache.data_ptr(), v_cache.data_ptr(),
                               block_table.data_ptr(), ctx_len.data_ptr(), count.data_ptr(),
                               accept_len.data_ptr(), accept_path.data_ptr(), new_len.data_ptr(),
                               status.data_ptr(), s)
    _raise(code, "kv_commit")
    return new_len, status


def trace_enable(on: bool = True) -> bool:
    return bool(lib().pct_trace_enable(1 if on else 0))


def trace_reset():
    lib().pct_trace_reset()


def trace_read(max_entries: int = 64) -> dict:
    """{kernel name: (launches, total ms)} for the launches recorded since the last reset."""
    stride = 64
    names = ctypes.create_string_buffer(stride * max_entries)
    launches = (ctypes.c_int64 * max_entries)()
    ms = (ctypes.c_double * max_entries)()
    n = lib().pct_trace_read(names, stride, ctypes.cast(launches, ctypes.c_void_p),
                             ctypes.cast(ms, ctypes.c_void_p), max_entries)
    if n < 0:
        raise PctError(PCT_ECUDA, "pct_trace_read")
    out = {}
    for i in range(n):
        nm = names.raw[i * stride:(i + 1) * stride].split(b"\0", 1)[0].decode()
        out[nm] = (int(launches[i]), float(ms[i]))
    return out


def version() -> str:
    return lib().pct_version().decode()

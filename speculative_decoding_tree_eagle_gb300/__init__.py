"""GB300 tree-verify hot path for EAGLE-2-style speculative decoding (Python binding).

Thin ctypes binding over ``libtreespec.so`` (C ABI in ``include/treespec.h``).  The
functions below only check tensor metadata, allocate outputs with torch and pass raw
device pointers plus torch's current CUDA stream; every step of the computation runs in
the library's CUDA kernels.  There is no CPU fallback: without the built library, or
without a CUDA device, every call raises.

    tree_build(draft_logp, root_tokens, k, depth, m)      -> dict(tokens, parents, depth, mask, values)
    tree_attention(q, k_cache, v_cache, block_table, prefix_len, mask, ...) -> (out, lse)
    tree_accept(logits, tokens, parents)                  -> dict(argmax, accept_len, accept_path, bonus)

The rows after the path: ``kv_commit`` (keep the accepted path's K/V rows, release the
rejected pages), ``lm_head_argmax`` / ``tree_accept_hidden`` (target LM head with the argmax in
its GEMM epilogue), ``efficient_head`` / ``tree_build_from_topk`` (the draft's two-stage head
and the tree from its lists), ``tree_accept_sample`` (acceptance at temperature T > 0) and
``tree_prune`` (cost-aware pruning before verification).

Long contexts: ``kv_page_bounds`` (per-page bounds of the keys), ``page_select`` (the pages each
node attends to) and ``tree_attention_sparse`` (tree attention over them).  A cache in 8 bits, e4m3
codes beside a scale for each block of tokens and head: ``kv_write_fp8``, ``kv_read_fp8``,
``kv_commit_fp8`` and ``tree_attention_fp8``.  The page pool:
``kv_reserve`` (room for the next tokens), ``kv_fork`` (fork, reorder and drop sequences) and
``kv_compact`` (move the pages in use together).  These ten run on the tensors' device, which need
not be the current one, on that device's current stream, and take their workspace from torch's
allocator call by call, so calls on several streams or in several captured graphs share none.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading
from typing import Dict, List, Optional, Tuple

import torch

__all__ = [
    "TreeSpecError", "library", "library_path", "launch_count", "status_string",
    "tree_build", "tree_attention", "tree_accept", "kv_commit", "lm_head_argmax", "tree_accept_hidden",
    "efficient_head", "tree_build_from_topk", "tree_accept_sample", "tree_prune",
    "kv_page_bounds", "page_select", "tree_attention_sparse", "kv_reserve", "kv_fork", "kv_compact",
    "kv_write_fp8", "kv_read_fp8", "kv_commit_fp8", "tree_attention_fp8",
    "new_status", "check_status",
    "tree_build_workspace", "tree_attention_workspace", "tree_accept_workspace", "tree_attention_plan",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_PKG, "libtreespec.so")

TS_F32, TS_BF16 = 0, 1
_lib = None
_lock = threading.Lock()


class TreeSpecError(RuntimeError):
    pass


def library():
    """Load libtreespec.so (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(library_path):
            raise TreeSpecError(f"{library_path} is missing: build it with "
                                "`python -m speculative_decoding_tree_eagle_gb300.build`")
        L = ctypes.CDLL(library_path)
        P, I, S, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
        L.ts_status_string.restype = ctypes.c_char_p
        L.ts_status_string.argtypes = [I]
        L.ts_version.restype = I
        L.ts_launch_count.restype = ctypes.c_uint64
        L.ts_tree_build_workspace.restype = S
        L.ts_tree_build_workspace.argtypes = [I, I, I, I, I]
        L.ts_tree_build.restype = I
        L.ts_tree_build.argtypes = [P, P, I, I, I, I, I, P, P, P, P, P, P, P, S, P, P]
        L.ts_tree_attention_workspace.restype = S
        L.ts_tree_attention_workspace.argtypes = [I, I, I, I, I, I, I]
        L.ts_tree_attention.restype = I
        L.ts_tree_attention.argtypes = [P, P, P, I, I, I, P, I, P, I, P, I, I, I, I, I, F, P, P, P, S, P, P]
        L.ts_tree_attention_plan.restype = I
        L.ts_tree_attention_plan.argtypes = [I, I, I, I, I, I, I, I, P]
        L.ts_tree_attention_plan_for_sms.restype = I
        L.ts_tree_attention_plan_for_sms.argtypes = [I, I, I, I, I, I, I, I, I, P]
        L.ts_tree_accept_workspace.restype = S
        L.ts_tree_accept_workspace.argtypes = [I, I, I, I]
        L.ts_tree_accept.restype = I
        L.ts_tree_accept.argtypes = [P, I, P, P, I, I, I, P, P, P, P, P, S, P, P]
        L.ts_lm_head_argmax_workspace.restype = S
        L.ts_lm_head_argmax_workspace.argtypes = [I, I, I]
        L.ts_lm_head_argmax.restype = I
        L.ts_lm_head_argmax.argtypes = [P, P, I, I, I, P, P, P, S, P, P]
        L.ts_tree_accept_hidden_workspace.restype = S
        L.ts_tree_accept_hidden_workspace.argtypes = [I, I, I, I]
        L.ts_tree_accept_hidden.restype = I
        L.ts_tree_accept_hidden.argtypes = [P, P, P, P, I, I, I, I, P, P, P, P, P, S, P, P]
        L.ts_efficient_head_candidates.restype = I
        L.ts_efficient_head_candidates.argtypes = [I, I, I]
        L.ts_efficient_head_workspace.restype = S
        L.ts_efficient_head_workspace.argtypes = [I, I, I, I, I, I]
        L.ts_efficient_head.restype = I
        L.ts_efficient_head.argtypes = [P, P, P, P, I, I, I, I, I, I, I, P, P, P, P, S, P, P]
        L.ts_tree_build_from_topk.restype = I
        L.ts_tree_build_from_topk.argtypes = [P, P, P, I, I, I, I, P, P, P, P, P, P, P, P]
        L.ts_tree_accept_sample_workspace.restype = S
        L.ts_tree_accept_sample_workspace.argtypes = [I, I, I]
        L.ts_tree_accept_sample.restype = I
        L.ts_tree_accept_sample.argtypes = [P, I, P, P, P, P, P, I, I, I, I, F, I, P, P, P, P, S, P, P]
        L.ts_tree_prune_workspace.restype = S
        L.ts_tree_prune_workspace.argtypes = [I, I]
        L.ts_tree_prune.restype = I
        D = ctypes.c_double
        L.ts_tree_prune.argtypes = [P, P, P, P, P, I, I, D, D, D, P, P, P, P, P, P, P, P, P, P, S, P, P]
        L.ts_selftest_bounded_wait.restype = I
        L.ts_selftest_bounded_wait.argtypes = [I, P, P, P]
        L.ts_kv_commit.restype = I
        L.ts_kv_commit.argtypes = [P, P, I, I, I, I, I, P, I, P, P, P, I, I, P, P, P, P]
        L.ts_kv_page_bounds.restype = I
        L.ts_kv_page_bounds.argtypes = [P, I, I, I, I, I, P, I, P, P, I, P, P, P]
        L.ts_page_select_workspace.restype = S
        L.ts_page_select_workspace.argtypes = [I, I, I, I, I, I, I]
        L.ts_page_select.restype = I
        L.ts_page_select.argtypes = [P, I, P, I, I, P, I, P, I, I, I, I, I, I, I, I, I, P, P, P, P, S, P, P]
        L.ts_tree_attention_sparse_workspace.restype = S
        L.ts_tree_attention_sparse_workspace.argtypes = [I, I, I, I, I, I, I, I]
        L.ts_tree_attention_sparse.restype = I
        L.ts_tree_attention_sparse.argtypes = [P, P, P, I, I, I, P, I, P, P, P, P, P, I, I, I, I, I, I, F, P, P, P, S, P, P]
        L.ts_kv_reserve_workspace.restype = S
        L.ts_kv_reserve_workspace.argtypes = [I, I, I, I]
        L.ts_kv_reserve.restype = I
        L.ts_kv_reserve.argtypes = [P, P, I, I, I, I, I, P, I, P, P, I, I, P, I, P, P, P, P, S, P, P]
        L.ts_kv_fork.restype = I
        L.ts_kv_fork.argtypes = [P, I, P, P, I, I, I, P, I, P, P, P, P, P]
        L.ts_kv_reserve_fp8.restype = I
        L.ts_kv_reserve_fp8.argtypes = [P, P, P, P, I, I, I, I, I, P, I, P, P, I, I, P, I, P, P, P, P, S, P, P]
        L.ts_kv_compact_fp8.restype = I
        L.ts_kv_compact_fp8.argtypes = [P, P, P, P, I, I, I, I, I, P, I, P, I, P, P, P, P, P, S, P, P]
        L.ts_kv_compact_workspace.restype = S
        L.ts_kv_compact_workspace.argtypes = [I]
        L.ts_kv_compact.restype = I
        L.ts_kv_compact.argtypes = [P, P, I, P, I, I, I, I, P, I, P, I, P, P, P, P, P, S, P, P]
        L.ts_kv_write_fp8.restype = I
        L.ts_kv_write_fp8.argtypes = [P, P, I, P, P, P, P, P, P, I, I, I, I, I, P, I, P, P, I, I, P, P]
        L.ts_kv_read_fp8.restype = I
        L.ts_kv_read_fp8.argtypes = [P, P, P, P, I, I, I, I, I, P, I, P, P, I, I, P, P, I, P, P]
        L.ts_kv_commit_fp8.restype = I
        L.ts_kv_commit_fp8.argtypes = [P, P, P, P, I, I, I, I, I, P, I, P, P, P, I, I, P, P, P, P, P, P]
        L.ts_tree_attention_fp8_workspace.restype = S
        L.ts_tree_attention_fp8_workspace.argtypes = [I, I, I, I, I, I, I, I]
        L.ts_tree_attention_fp8.restype = I
        L.ts_tree_attention_fp8.argtypes = [P, I, P, P, P, P, I, I, I, P, I, P, I, P, I, I, I, I, I, F, P, P, P, S, P, P]
        _lib = L
    return _lib


def status_string(code: int) -> str:
    return library().ts_status_string(int(code)).decode()


def launch_count() -> int:
    """Kernels launched by the library in this process so far."""
    return int(library().ts_launch_count())


def _check(rc: int) -> None:
    if rc != 0:
        raise TreeSpecError(status_string(rc))


def _p(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def _need_cuda(name: str, t: torch.Tensor, dtype=None) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return TS_F32
    if t.dtype == torch.bfloat16:
        return TS_BF16
    raise ValueError(f"unsupported dtype {t.dtype} (fp32 or bf16)")


_ws_cache: Dict[int, torch.Tensor] = {}


def _workspace(nbytes: int, device: torch.device, ws: Optional[torch.Tensor]) -> torch.Tensor:
    if ws is not None:
        if ws.numel() * ws.element_size() < nbytes:
            raise ValueError("workspace too small")
        return ws
    idx = device.index if device.index is not None else torch.cuda.current_device()
    cur = _ws_cache.get(idx)
    if cur is None or cur.numel() < nbytes:
        cur = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
        _ws_cache[idx] = cur
    return cur


def new_status(device=None) -> torch.Tensor:
    """A zeroed int32 device word for the kernels' device-side error codes."""
    return torch.zeros(1, dtype=torch.int32, device=device or "cuda")


def check_status(status: torch.Tensor) -> None:
    """Synchronise and raise if a kernel reported a device-side error."""
    code = int(status.item())
    if code != 0:
        raise TreeSpecError(status_string(code))


def tree_build_workspace(B: int, V: int, k: int, depth: int, m: int) -> int:
    return int(library().ts_tree_build_workspace(B, V, k, depth, m))


def tree_attention_workspace(dtype: torch.dtype, B: int, m: int, Hq: int, Hkv: int, d: int,
                             max_prefix: int) -> int:
    dt = TS_F32 if dtype == torch.float32 else TS_BF16
    return int(library().ts_tree_attention_workspace(dt, B, m, Hq, Hkv, d, max_prefix))


def tree_attention_plan(dtype: torch.dtype, B: int, m: int, Hq: int, Hkv: int, d: int, max_prefix: int,
                        block_size: int, num_sms: Optional[int] = None) -> Dict[str, int]:
    """The launch plan tree_attention uses for these sizes on the current device, or, with
    ``num_sms``, for that many SMs (multicast and the in-cluster merge still depend on what the
    current device can co-schedule; with no device present neither is chosen)."""
    dt = TS_F32 if dtype == torch.float32 else TS_BF16
    out = (ctypes.c_int * 6)()
    if num_sms is None:
        _check(library().ts_tree_attention_plan(dt, B, m, Hq, Hkv, d, max_prefix, block_size, out))
    else:
        _check(library().ts_tree_attention_plan_for_sms(dt, B, m, Hq, Hkv, d, max_prefix, block_size,
                                                        int(num_sms), out))
    modes = {0: "one chunk", 1: "cluster merge", 2: "workspace merge"}
    return {"path": "tensor-core" if out[0] else "cuda-core", "row_groups": out[1], "chunks": out[2],
            "tiles_per_chunk": out[3], "split": modes.get(out[4], str(out[4])), "multicast": out[5]}


def tree_accept_workspace(dtype: torch.dtype, B: int, m: int, V: int) -> int:
    dt = TS_F32 if dtype == torch.float32 else TS_BF16
    return int(library().ts_tree_accept_workspace(dt, B, m, V))


def tree_build(draft_logp: torch.Tensor, root_tokens: torch.Tensor, k: int, depth: int, m: int, *,
               out: Optional[Dict[str, torch.Tensor]] = None, with_values: bool = True,
               workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """EAGLE-2 dynamic draft tree: draft_logp [B, 1+(depth-1)k, V] fp32 log-probs, root_tokens [B] int32."""
    L = library()
    _need_cuda("draft_logp", draft_logp, torch.float32)
    _need_cuda("root_tokens", root_tokens, torch.int32)
    B, R, V = draft_logp.shape
    if R != 1 + (depth - 1) * k:
        raise ValueError(f"draft_logp must have {1 + (depth - 1) * k} rows per sequence, got {R}")
    dev = draft_logp.device
    W = (m + 63) // 64
    if out is None:
        out = dict(tokens=torch.empty(B, m, dtype=torch.int32, device=dev),
                   parents=torch.empty(B, m, dtype=torch.int32, device=dev),
                   depth=torch.empty(B, m, dtype=torch.int32, device=dev),
                   mask=torch.empty(B, m, W, dtype=torch.int64, device=dev))
        if with_values:
            out["values"] = torch.empty(B, m, dtype=torch.float64, device=dev)
        out["node_row"] = torch.empty(B, m, dtype=torch.int32, device=dev)
    need = L.ts_tree_build_workspace(B, V, k, depth, m)
    if need == 0:
        raise TreeSpecError("invalid tree_build sizes")
    ws = _workspace(need, dev, workspace)
    _check(L.ts_tree_build(_p(draft_logp), _p(root_tokens), B, V, k, depth, m, _p(out["tokens"]),
                           _p(out["parents"]), _p(out["depth"]), _p(out["mask"]), _p(out.get("values")),
                           _p(out.get("node_row")), _p(ws), ws.numel() * ws.element_size(), _p(status), _stream()))
    return out


def tree_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                   prefix_len: torch.Tensor, mask: torch.Tensor, *, max_prefix: int,
                   scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                   lse: Optional[torch.Tensor] = None, with_lse: bool = True,
                   workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None):
    """Tree attention.  q [B,m,Hq,d]; caches [num_blocks,Hkv,block_size,d]; block_table [B,max_blocks]
    int32; prefix_len [B] int32; mask [B,m,ceil(m/64)] (int64 view of uint64 words)."""
    L = library()
    for name, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache)):
        _need_cuda(name, t, q.dtype)
    _need_cuda("block_table", block_table, torch.int32)
    _need_cuda("prefix_len", prefix_len, torch.int32)
    _need_cuda("mask", mask, torch.int64)
    B, m, Hq, d = q.shape
    NB, Hkv, bs, d2 = k_cache.shape
    if d2 != d or tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("cache shapes do not match q")
    if mask.shape != (B, m, (m + 63) // 64):
        raise ValueError("mask must be [B, m, ceil(m/64)]")
    dt = _dt(q)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and with_lse:
        lse = torch.empty(B, m, Hq, dtype=torch.float32, device=q.device)
    need = L.ts_tree_attention_workspace(dt, B, m, Hq, Hkv, d, max_prefix)
    ws = _workspace(max(need, 256), q.device, workspace)
    _check(L.ts_tree_attention(_p(q), _p(k_cache), _p(v_cache), dt, NB, bs, _p(block_table),
                               block_table.shape[1], _p(prefix_len), int(max_prefix), _p(mask), B, m, Hq,
                               Hkv, d, float(scale), _p(out), _p(lse), _p(ws),
                               ws.numel() * ws.element_size(), _p(status), _stream()))
    return out, lse


def tree_accept(logits: torch.Tensor, tokens: torch.Tensor, parents: torch.Tensor, *,
                out: Optional[Dict[str, torch.Tensor]] = None, workspace: Optional[torch.Tensor] = None,
                status: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """Per-node argmax of logits [B,m,V] and the longest matching root path."""
    L = library()
    _need_cuda("logits", logits)
    _need_cuda("tokens", tokens, torch.int32)
    _need_cuda("parents", parents, torch.int32)
    B, m, V = logits.shape
    dt = _dt(logits)
    dev = logits.device
    if out is None:
        out = dict(argmax=torch.empty(B, m, dtype=torch.int32, device=dev),
                   accept_len=torch.empty(B, dtype=torch.int32, device=dev),
                   accept_path=torch.empty(B, m, dtype=torch.int32, device=dev),
                   bonus=torch.empty(B, dtype=torch.int32, device=dev))
    need = L.ts_tree_accept_workspace(dt, B, m, V)
    if need == 0:
        raise TreeSpecError("invalid tree_accept sizes")
    ws = _workspace(need, dev, workspace)
    _check(L.ts_tree_accept(_p(logits), dt, _p(tokens), _p(parents), B, m, V, _p(out["argmax"]),
                            _p(out["accept_len"]), _p(out["accept_path"]), _p(out["bonus"]), _p(ws),
                            ws.numel() * ws.element_size(), _p(status), _stream()))
    return out


Q_MODES = {"point": 0, "draft": 1}


def tree_accept_sample(logits: torch.Tensor, tokens: torch.Tensor, parents: torch.Tensor, uniforms: torch.Tensor,
                       temperature: float, *, q_mode: str = "point", draft_logp: Optional[torch.Tensor] = None,
                       node_row: Optional[torch.Tensor] = None, out: Optional[Dict[str, torch.Tensor]] = None,
                       workspace: Optional[torch.Tensor] = None,
                       status: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """Verification at temperature T > 0 by multi-round rejection sampling: logits [B,m,V],
    tokens/parents [B,m] int32, uniforms [B,m] float32 in [0, 1).  q_mode "point" (a unit mass
    per candidate) or "draft" (the draft rows draft_logp [B,R,V] named by node_row [B,m]).
    Returns accept_len [B], accept_path [B,m] and bonus [B] (the drawn token)."""
    L = library()
    _need_cuda("logits", logits)
    _need_cuda("tokens", tokens, torch.int32)
    _need_cuda("parents", parents, torch.int32)
    _need_cuda("uniforms", uniforms, torch.float32)
    if q_mode not in Q_MODES:
        raise TreeSpecError("q_mode is 'point' or 'draft'")
    B, m, V = logits.shape
    R = 0
    if q_mode == "draft":
        if draft_logp is None or node_row is None:
            raise TreeSpecError("q_mode 'draft' needs draft_logp and node_row")
        _need_cuda("draft_logp", draft_logp, torch.float32)
        _need_cuda("node_row", node_row, torch.int32)
        R = draft_logp.shape[1]
    dev = logits.device
    if out is None:
        out = dict(accept_len=torch.empty(B, dtype=torch.int32, device=dev),
                   accept_path=torch.empty(B, m, dtype=torch.int32, device=dev),
                   bonus=torch.empty(B, dtype=torch.int32, device=dev))
    need = L.ts_tree_accept_sample_workspace(B, V, Q_MODES[q_mode])
    ws = _workspace(need, dev, workspace) if need > 0 else None
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(L.ts_tree_accept_sample(_p(logits), _dt(logits), _p(tokens), _p(parents), _p(uniforms), _p(draft_logp),
                                   _p(node_row), R, B, m, V, float(temperature), Q_MODES[q_mode],
                                   _p(out["accept_len"]), _p(out["accept_path"]), _p(out["bonus"]), _p(ws), nbytes,
                                   _p(status), _stream()))
    return out


def tree_prune(tree: Dict[str, torch.Tensor], t_draft: float, t_fixed: float, t_node: float, *,
               workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
               sync: bool = True) -> Dict[str, torch.Tensor]:
    """Cost-aware pruning before verification of a tree from tree_build (``tokens``, ``parents``,
    ``depth`` int32 and ``values`` float64 [B,m]; ``node_row`` optional).  One node count n for
    the batch maximises expected tokens per unit of round time (t_draft + t_fixed + t_node*B*n).
    Returns ``n`` (a device int32 [1]) and the pruned tree: ``tokens``, ``parents``, ``depth``,
    ``kept`` (old flat indices), ``node_row`` int32 and ``values`` [B,n], ``mask`` int64
    [B,n,ceil(n/64)], ``expected`` float32 [B].  With ``sync`` (default) the host reads n and
    the outputs are views of shape [B,n]; without it they are the flat buffers (row stride n)."""
    L = library()
    for name, dt in (("tokens", torch.int32), ("parents", torch.int32), ("depth", torch.int32),
                     ("values", torch.float64)):
        _need_cuda(name, tree[name], dt)
    nr = tree.get("node_row")
    if nr is not None:
        _need_cuda("node_row", nr, torch.int32)
    B, m = tree["tokens"].shape
    dev = tree["tokens"].device
    W = (m + 63) // 64
    buf = dict(n=torch.empty(1, dtype=torch.int32, device=dev),
               tokens=torch.empty(B * m, dtype=torch.int32, device=dev),
               parents=torch.empty(B * m, dtype=torch.int32, device=dev),
               depth=torch.empty(B * m, dtype=torch.int32, device=dev),
               kept=torch.empty(B * m, dtype=torch.int32, device=dev),
               values=torch.empty(B * m, dtype=torch.float64, device=dev),
               mask=torch.empty(B * m * W, dtype=torch.int64, device=dev),
               expected=torch.empty(B, dtype=torch.float32, device=dev))
    if nr is not None:
        buf["node_row"] = torch.empty(B * m, dtype=torch.int32, device=dev)
    need = L.ts_tree_prune_workspace(B, m)
    if need == 0:
        raise TreeSpecError("invalid tree_prune sizes")
    ws = _workspace(need, dev, workspace)
    _check(L.ts_tree_prune(_p(tree["tokens"]), _p(tree["parents"]), _p(tree["depth"]), _p(tree["values"]), _p(nr),
                           B, m, float(t_draft), float(t_fixed), float(t_node), _p(buf["n"]), _p(buf["tokens"]),
                           _p(buf["parents"]), _p(buf["depth"]), _p(buf["mask"]), _p(buf["values"]),
                           _p(buf.get("node_row")), _p(buf["kept"]), _p(buf["expected"]), _p(ws),
                           ws.numel() * ws.element_size(), _p(status), _stream()))
    if not sync:
        return buf
    n = int(buf["n"].item())
    Wn = (n + 63) // 64
    out = {"n": buf["n"], "expected": buf["expected"]}
    for k in ("tokens", "parents", "depth", "kept", "values", "node_row"):
        if k in buf:
            out[k] = buf[k][: B * n].view(B, n)
    out["mask"] = buf["mask"][: B * n * Wn].view(B, n, Wn)
    return out


def kv_commit(k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
              prefix_len: torch.Tensor, accept_path: torch.Tensor, accept_len: torch.Tensor, *,
              out: Optional[Dict[str, torch.Tensor]] = None,
              status: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """Keep the accepted path's K/V rows and release the rejected scratch pages, in place on
    k_cache/v_cache [num_blocks,Hkv,bs,d], block_table [B,max_blocks] and prefix_len [B];
    returns freed_blocks [B,max_blocks] (-1 padded) and freed_count [B]."""
    L = library()
    _need_cuda("k_cache", k_cache)
    _need_cuda("v_cache", v_cache, k_cache.dtype)
    _need_cuda("block_table", block_table, torch.int32)
    _need_cuda("prefix_len", prefix_len, torch.int32)
    _need_cuda("accept_path", accept_path, torch.int32)
    _need_cuda("accept_len", accept_len, torch.int32)
    nb, hkv, bs, d = k_cache.shape
    B, max_blocks = block_table.shape
    m = accept_path.shape[1]
    dev = k_cache.device
    if out is None:
        out = dict(freed_blocks=torch.empty(B, max_blocks, dtype=torch.int32, device=dev),
                   freed_count=torch.empty(B, dtype=torch.int32, device=dev))
    _check(L.ts_kv_commit(_p(k_cache), _p(v_cache), _dt(k_cache), nb, bs, hkv, d, _p(block_table), max_blocks,
                          _p(prefix_len), _p(accept_path), _p(accept_len), B, m, _p(out["freed_blocks"]),
                          _p(out["freed_count"]), _p(status), _stream()))
    return out


def lm_head_argmax(hidden: torch.Tensor, weight: torch.Tensor, *, out: Optional[Dict[str, torch.Tensor]] = None,
                   workspace: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """Per-row argmax (first index) and max of hidden [M,K] @ weight[N,K]^T (bf16), logits kept on chip."""
    L = library()
    _need_cuda("hidden", hidden, torch.bfloat16)
    _need_cuda("weight", weight, torch.bfloat16)
    M, K = hidden.shape
    N, K2 = weight.shape
    if K2 != K:
        raise ValueError("hidden and weight disagree on K")
    dev = hidden.device
    if out is None:
        out = dict(argmax=torch.empty(M, dtype=torch.int32, device=dev),
                   max_logit=torch.empty(M, dtype=torch.float32, device=dev))
    need = L.ts_lm_head_argmax_workspace(M, N, K)
    if need == 0:
        raise TreeSpecError("invalid lm_head_argmax sizes")
    ws = _workspace(need, dev, workspace)
    _check(L.ts_lm_head_argmax(_p(hidden), _p(weight), M, N, K, _p(out["argmax"]), _p(out.get("max_logit")), _p(ws),
                               ws.numel() * ws.element_size(), _p(status), _stream()))
    return out


def tree_accept_hidden(hidden: torch.Tensor, weight: torch.Tensor, tokens: torch.Tensor, parents: torch.Tensor, *,
                       out: Optional[Dict[str, torch.Tensor]] = None, workspace: Optional[torch.Tensor] = None,
                       status: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """tree_accept from the target's final hidden states [B,m,K] and its LM head [V,K] (bf16)."""
    L = library()
    _need_cuda("hidden", hidden, torch.bfloat16)
    _need_cuda("weight", weight, torch.bfloat16)
    _need_cuda("tokens", tokens, torch.int32)
    _need_cuda("parents", parents, torch.int32)
    B, m, K = hidden.shape
    V = weight.shape[0]
    dev = hidden.device
    if out is None:
        out = dict(argmax=torch.empty(B, m, dtype=torch.int32, device=dev),
                   accept_len=torch.empty(B, dtype=torch.int32, device=dev),
                   accept_path=torch.empty(B, m, dtype=torch.int32, device=dev),
                   bonus=torch.empty(B, dtype=torch.int32, device=dev))
    need = L.ts_tree_accept_hidden_workspace(B, m, V, K)
    if need == 0:
        raise TreeSpecError("invalid tree_accept_hidden sizes")
    ws = _workspace(need, dev, workspace)
    _check(L.ts_tree_accept_hidden(_p(hidden), _p(weight), _p(tokens), _p(parents), B, m, V, K, _p(out["argmax"]),
                                   _p(out["accept_len"]), _p(out["accept_path"]), _p(out["bonus"]), _p(ws),
                                   ws.numel() * ws.element_size(), _p(status), _stream()))
    return out


def efficient_head(hidden: torch.Tensor, lr_b: torch.Tensor, lr_a: torch.Tensor, weight: torch.Tensor, *,
                   tile_tokens: int, k_tile: int, k: int, with_candidates: bool = False,
                   workspace: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """Two-stage draft head: hidden [M,d], lr_b [rank,d], lr_a [V,rank], weight [V,d] (bf16) ->
    top_tok [M,k], top_logp [M,k] (log-probs over the candidates), optionally candidates [M,C]."""
    L = library()
    for n, t in (("hidden", hidden), ("lr_b", lr_b), ("lr_a", lr_a), ("weight", weight)):
        _need_cuda(n, t, torch.bfloat16)
    M, d = hidden.shape
    rank = lr_b.shape[0]
    V = weight.shape[0]
    dev = hidden.device
    C = L.ts_efficient_head_candidates(V, tile_tokens, k_tile)
    out = dict(top_tok=torch.empty(M, k, dtype=torch.int32, device=dev),
               top_logp=torch.empty(M, k, dtype=torch.float32, device=dev))
    if with_candidates:
        out["candidates"] = torch.empty(M, max(C, 1), dtype=torch.int32, device=dev)
    need = L.ts_efficient_head_workspace(M, V, d, rank, tile_tokens, k_tile)
    if need == 0:
        raise TreeSpecError("invalid efficient_head sizes")
    ws = _workspace(need, dev, workspace)
    _check(L.ts_efficient_head(_p(hidden), _p(lr_b), _p(lr_a), _p(weight), M, V, d, rank, tile_tokens, k_tile, k,
                               _p(out["top_tok"]), _p(out["top_logp"]), _p(out.get("candidates")), _p(ws),
                               ws.numel() * ws.element_size(), _p(status), _stream()))
    return out


def tree_build_from_topk(row_tok: torch.Tensor, row_logp: torch.Tensor, root_tokens: torch.Tensor, k: int,
                         depth: int, m: int, *, out: Optional[Dict[str, torch.Tensor]] = None,
                         status: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """tree_build from per-row top-k lists row_tok [B,R,k] int32 / row_logp [B,R,k] fp32."""
    L = library()
    _need_cuda("row_tok", row_tok, torch.int32)
    _need_cuda("row_logp", row_logp, torch.float32)
    _need_cuda("root_tokens", root_tokens, torch.int32)
    B = row_tok.shape[0]
    dev = row_tok.device
    W = (m + 63) // 64
    if out is None:
        out = dict(tokens=torch.empty(B, m, dtype=torch.int32, device=dev),
                   parents=torch.empty(B, m, dtype=torch.int32, device=dev),
                   depth=torch.empty(B, m, dtype=torch.int32, device=dev),
                   mask=torch.empty(B, m, W, dtype=torch.int64, device=dev),
                   values=torch.empty(B, m, dtype=torch.float64, device=dev),
                   node_row=torch.empty(B, m, dtype=torch.int32, device=dev))
    _check(L.ts_tree_build_from_topk(_p(row_tok), _p(row_logp), _p(root_tokens), B, k, depth, m, _p(out["tokens"]),
                                     _p(out["parents"]), _p(out["depth"]), _p(out["mask"]), _p(out.get("values")),
                                     _p(out.get("node_row")), _p(status), _stream()))
    return out


# The calls below check each tensor once (device, type, shape, layout) and run on the tensors' own device.

_raw_stream = torch._C._cuda_getCurrentRawStream  # current_stream(i).cuda_stream without building a Stream object
_INVALID = -1
_I32, _I64, _BF16, _F32 = torch.int32, torch.int64, torch.bfloat16, torch.float32
_E4M3 = torch.float8_e4m3fn


def _refuse(name: str, t: torch.Tensor, index: int, dtype, shape) -> None:
    _need_cuda(name, t, dtype)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} is on {t.device}, the other tensors on cuda:{index}")


def _arg(name: str, t: torch.Tensor, index: int, dtype, shape) -> int:
    """The address of a contiguous tensor of this type and shape on device ``index``."""
    if t.get_device() != index or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _refuse(name, t, index, dtype, shape)
    return t.data_ptr()


def _out_args(out: Dict[str, torch.Tensor], index: int, made: bool, **want) -> List[int]:
    """The addresses of the outputs; those of the caller's making are checked."""
    if made:
        return [out[name].data_ptr() for name in want]
    return [_arg(name, out[name], index, dtype, shape) for name, (dtype, shape) in want.items()]


def _status_arg(status: Optional[torch.Tensor], index: int) -> Optional[int]:
    return None if status is None else _arg("status", status, index, _I32, (1,))


def _index_of(name: str, t: torch.Tensor, dims: int) -> int:
    """Device index of the tensor that decides where the call runs."""
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {list(t.shape)}")
    return index


def _scratch(nbytes: int, like: torch.Tensor, ws: Optional[torch.Tensor]):
    """(address, bytes) of the caller's workspace, or of one of this call's own, and what keeps it."""
    if ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=like.device)
        return ws.data_ptr(), nbytes, ws
    _need_cuda("workspace", ws)
    if ws.device != like.device:
        raise ValueError(f"workspace is on {ws.device}, the other tensors on {like.device}")
    size = ws.numel() * ws.element_size()
    if size < nbytes:
        raise ValueError("workspace too small")
    return ws.data_ptr(), size, ws


def _apart(out: Dict[str, torch.Tensor], may_be_same: Tuple[str, ...], **inputs: Optional[torch.Tensor]) -> None:
    """Name the outputs that share memory with an input or with one another; those in ``may_be_same`` may be the very
    buffer of the input of their name.  (The library refuses such calls; this says why.)"""
    def memory(t):
        at = t.data_ptr()
        return at, at + t.numel() * t.element_size()

    outs = [(f"out[{name!r}]", name, *memory(t)) for name, t in out.items()]
    ins = [(name, name, *memory(t)) for name, t in inputs.items() if t is not None]
    for i, (label, name, a0, a1) in enumerate(outs):
        for other, theirs, b0, b1 in ins + outs[i + 1:]:
            if a0 < b1 and b0 < a1 and not (theirs == name and name in may_be_same and a0 == b0 and a1 == b1):
                raise ValueError(f"{label} shares memory with {other}")


def kv_page_bounds(k_cache: torch.Tensor, block_table: torch.Tensor, prefix_len: torch.Tensor, *,
                   start_len: Optional[torch.Tensor] = None, bounds: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Bounds of the keys of the pages complete at prefix_len [B] that were not at start_len [B]
    (default: at 0), into bounds [num_blocks,Hkv,2,d] bf16 (largest, smallest), which is returned.
    Other pages' bounds stay; without ``bounds`` a tensor of zeros is made."""
    L = library()
    ix = _index_of("k_cache", k_cache, 4)
    if ix != torch.cuda.current_device():
        with torch.cuda.device(ix):
            return kv_page_bounds(k_cache, block_table, prefix_len, start_len=start_len, bounds=bounds, status=status)
    dt = _dt(k_cache)
    NB, Hkv, bs, d = shape = k_cache.shape
    B, width = block_table.shape
    if bounds is None:
        bounds = torch.zeros((NB, Hkv, 2, d), dtype=_BF16, device=k_cache.device)
    _check(L.ts_kv_page_bounds(_arg("k_cache", k_cache, ix, k_cache.dtype, shape), dt, NB, bs, Hkv, d,
                               _arg("block_table", block_table, ix, _I32, (B, width)), width,
                               _arg("prefix_len", prefix_len, ix, _I32, (B,)),
                               None if start_len is None else _arg("start_len", start_len, ix, _I32, (B,)), B,
                               _arg("bounds", bounds, ix, _BF16, (NB, Hkv, 2, d)), _status_arg(status, ix), _raw_stream(ix)))
    return bounds


def page_select(q: torch.Tensor, bounds: torch.Tensor, block_table: torch.Tensor, prefix_len: torch.Tensor, n_pages: int, *,
                block_size: int, max_prefix: int, first: int = 1, recent: int = 1,
                out: Optional[Dict[str, torch.Tensor]] = None, workspace: Optional[torch.Tensor] = None,
                status: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """The complete prefix pages each node of q [B,m,Hq,d] attends to: the first ``first``, the last
    ``recent`` and the best by the bounds [num_blocks,Hkv,2,d] of its scores, n_pages in all, per KV head.
    Returns pages [B,Hkv,C] (logical pages that any node keeps, ascending, -1 behind them), count
    [B,Hkv] and node_mask [B,Hkv,C,ceil(m/64)] (bit i: node i keeps the page), C = max(1, max_prefix //
    block_size): the selection that ``tree_attention_sparse`` takes."""
    L = library()
    ix = _index_of("q", q, 4)
    if ix != torch.cuda.current_device():
        with torch.cuda.device(ix):
            return page_select(q, bounds, block_table, prefix_len, n_pages, block_size=block_size, max_prefix=max_prefix,
                               first=first, recent=recent, out=out, workspace=workspace, status=status)
    dt = _dt(q)
    B, m, Hq, d = shape = q.shape
    NB, Hkv = bounds.shape[:2]
    width = block_table.shape[1]
    W = (m + 63) // 64
    need = L.ts_page_select_workspace(B, m, Hq, Hkv, d, max_prefix, block_size)
    if need == 0:
        raise TreeSpecError("invalid page_select sizes")
    C = max(1, max_prefix // block_size)
    made = out is None
    if made:
        dev = q.device
        out = dict(pages=torch.empty((B, Hkv, C), dtype=_I32, device=dev), count=torch.empty((B, Hkv), dtype=_I32, device=dev),
                   node_mask=torch.empty((B, Hkv, C, W), dtype=_I64, device=dev))
    ws, ws_bytes, keep = _scratch(need, q, workspace) if need > 256 else (None, 0, None)
    _check(L.ts_page_select(_arg("q", q, ix, q.dtype, shape), dt, _arg("bounds", bounds, ix, _BF16, (NB, Hkv, 2, d)), NB,
                            block_size, _arg("block_table", block_table, ix, _I32, (B, width)), width,
                            _arg("prefix_len", prefix_len, ix, _I32, (B,)), max_prefix, B, m, Hq, Hkv, d, n_pages, first,
                            recent,
                            *_out_args(out, ix, made, pages=(_I32, (B, Hkv, C)), count=(_I32, (B, Hkv)),
                                       node_mask=(_I64, (B, Hkv, C, W))), ws, ws_bytes,
                            _status_arg(status, ix), _raw_stream(ix)))
    return out


def tree_attention_sparse(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                          prefix_len: torch.Tensor, mask: torch.Tensor, selection: Dict[str, torch.Tensor], *,
                          scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                          lse: Optional[torch.Tensor] = None, with_lse: bool = True,
                          workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None):
    """Tree attention over chosen pages: each node of q [B,m,Hq,d] attends to the pages that
    ``selection`` (pages, count and node_mask of ``page_select``) gives it, to the prefix rows of the page
    that is not complete yet and to its ancestors (mask).  Returns (out, lse) like ``tree_attention``."""
    L = library()
    ix = _index_of("q", q, 4)
    if ix != torch.cuda.current_device():
        with torch.cuda.device(ix):
            return tree_attention_sparse(q, k_cache, v_cache, block_table, prefix_len, mask, selection, scale=scale, out=out,
                                         lse=lse, with_lse=with_lse, workspace=workspace, status=status)
    dtype, dt = q.dtype, _dt(q)
    B, m, Hq, d = shape = q.shape
    NB, Hkv, bs, d2 = cache = k_cache.shape
    if d2 != d:
        raise ValueError("cache shapes do not match q")
    pages = selection["pages"]
    W, C, width = (m + 63) // 64, pages.shape[-1], block_table.shape[1]
    # (given ones are checked, new ones are not)
    out_at = None if out is None else _arg("out", out, ix, dtype, shape)
    lse_at = None if lse is None else _arg("lse", lse, ix, _F32, (B, m, Hq))
    if out is None:
        out = torch.empty_like(q)
        out_at = out.data_ptr()
    if lse is None and with_lse:
        lse = torch.empty((B, m, Hq), dtype=_F32, device=q.device)
        lse_at = lse.data_ptr()
    need = L.ts_tree_attention_sparse_workspace(dt, B, m, Hq, Hkv, d, C, bs)
    ws, ws_bytes, keep = _scratch(need, q, workspace) if need > 256 else (None, 0, None)
    _check(L.ts_tree_attention_sparse(_arg("q", q, ix, dtype, shape), _arg("k_cache", k_cache, ix, dtype, cache),
                                      _arg("v_cache", v_cache, ix, dtype, cache), dt, NB, bs,
                                      _arg("block_table", block_table, ix, _I32, (B, width)), width,
                                      _arg("prefix_len", prefix_len, ix, _I32, (B,)),
                                      _arg("mask", mask, ix, _I64, (B, m, W)), _arg("pages", pages, ix, _I32, (B, Hkv, C)),
                                      _arg("count", selection["count"], ix, _I32, (B, Hkv)),
                                      _arg("node_mask", selection["node_mask"], ix, _I64, (B, Hkv, C, W)), C, B, m, Hq, Hkv,
                                      d, 1.0 / math.sqrt(d) if scale is None else scale, out_at, lse_at, ws, ws_bytes,
                                      _status_arg(status, ix), _raw_stream(ix)))
    return out, lse


def _pool_cache(name: str, k_cache, v_cache, k_scale, v_scale, ix):
    """The entry point of the pool for this cache, in bf16 or fp32 or with its scales in 8 bits, and its cache arguments."""
    if (k_scale is None) != (v_scale is None):
        raise ValueError("a cache in 8 bits has k_scale and v_scale")
    if k_scale is not None:
        at, sizes = _fp8_cache(k_cache, v_cache, k_scale, v_scale, ix)
        return getattr(library(), name + "_fp8"), [*at, *sizes]
    dtype, dt = k_cache.dtype, _dt(k_cache)
    NB, Hkv, bs, d = cache = k_cache.shape
    return getattr(library(), name), [_arg("k_cache", k_cache, ix, dtype, cache), _arg("v_cache", v_cache, ix, dtype, cache), dt,
                                      NB, bs, Hkv, d]


def kv_reserve(k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor, prefix_len: torch.Tensor,
               refs: torch.Tensor, n: int, *, freed: Optional[torch.Tensor] = None,
               k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
               out: Optional[Dict[str, torch.Tensor]] = None, workspace: Optional[torch.Tensor] = None,
               status: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """Pages for the next n tokens of every sequence: the pages in ``freed`` (any shape, -1 skipped; such as
    kv_commit's freed_blocks) lose a reference each, missing pages are handed out, and a half-filled last page
    that others hold too is replaced by a copy (its rows move in k_cache / v_cache).  Returns the new
    block_table and refs and granted [B] (fresh pages per sequence, -1 where the pool ran short and the sequence
    stays as it was).  A cache in 8 bits is given with its k_scale and v_scale; the copied rows' scales go with them.
    In ``out``, block_table and refs may be the input tensors themselves, for an update in place;
    otherwise the outputs lie apart from the inputs and from one another."""
    L = library()
    ix = _index_of("k_cache", k_cache, 4)
    if ix != torch.cuda.current_device():
        with torch.cuda.device(ix):
            return kv_reserve(k_cache, v_cache, block_table, prefix_len, refs, n, freed=freed, k_scale=k_scale,
                              v_scale=v_scale, out=out, workspace=workspace, status=status)
    call, cache_args = _pool_cache("ts_kv_reserve", k_cache, v_cache, k_scale, v_scale, ix)
    NB, Hkv, bs, d = k_cache.shape
    B, width = table = block_table.shape
    need = L.ts_kv_reserve_workspace(NB, bs, B, n)
    if need == 0:
        raise TreeSpecError("invalid kv_reserve sizes")
    args = [*cache_args, _arg("block_table", block_table, ix, _I32, table), width, _arg("prefix_len", prefix_len, ix, _I32, (B,)),
            _arg("refs", refs, ix, _I32, (NB,)), B, n]
    nfreed = 0 if freed is None else freed.numel()
    freed_at = _arg("freed", freed, ix, _I32, freed.shape) if nfreed else None
    made = out is None
    if made:
        out = dict(block_table=torch.empty_like(block_table), refs=torch.empty_like(refs),
                   granted=torch.empty_like(prefix_len))
    ws, ws_bytes, keep = _scratch(need, refs, workspace)
    rc = call(*args, freed_at, nfreed,
              *_out_args(out, ix, made, block_table=(_I32, table), refs=(_I32, (NB,)), granted=(_I32, (B,))), ws, ws_bytes,
              _status_arg(status, ix), _raw_stream(ix))
    if rc == _INVALID and not made:
        _apart(out, ("block_table", "refs"), block_table=block_table, refs=refs, prefix_len=prefix_len, freed=freed,
               k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale)
    _check(rc)
    return out


def kv_fork(block_table: torch.Tensor, prefix_len: torch.Tensor, refs: torch.Tensor, src: torch.Tensor, block_size: int, *,
            out: Optional[Dict[str, torch.Tensor]] = None, status: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """New sequences from old ones: row r continues row src[r] (int32, any number of rows; -1: an empty row).
    Returns the new block_table, prefix_len and refs, which replace the old ones: pages are shared, not
    copied, and those of rows that nobody continues are let go.  ``out["refs"]`` may be ``refs`` itself; otherwise the
    outputs lie apart from the inputs and from one another."""
    L = library()
    ix = _index_of("block_table", block_table, 2)
    if ix != torch.cuda.current_device():
        with torch.cuda.device(ix):
            return kv_fork(block_table, prefix_len, refs, src, block_size, out=out, status=status)
    B, width = table = block_table.shape
    R, NB = src.shape[0], refs.shape[0]
    args = [_arg("block_table", block_table, ix, _I32, table), width, _arg("prefix_len", prefix_len, ix, _I32, (B,)),
            _arg("refs", refs, ix, _I32, (NB,)), NB, block_size, B, _arg("src", src, ix, _I32, (R,)), R]
    made = out is None
    if made:
        out = dict(block_table=torch.empty((R, width), dtype=_I32, device=refs.device), prefix_len=torch.empty_like(src),
                   refs=torch.empty_like(refs))
    rc = L.ts_kv_fork(*args, *_out_args(out, ix, made, block_table=(_I32, (R, width)), prefix_len=(_I32, (R,)),
                                        refs=(_I32, (NB,))), _status_arg(status, ix), _raw_stream(ix))
    if rc == _INVALID and not made:
        _apart(out, ("refs",), block_table=block_table, prefix_len=prefix_len, refs=refs, src=src)
    _check(rc)
    return out


def kv_compact(k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor, refs: torch.Tensor, *,
               bounds: Optional[torch.Tensor] = None, k_scale: Optional[torch.Tensor] = None,
               v_scale: Optional[torch.Tensor] = None, out: Optional[Dict[str, torch.Tensor]] = None,
               workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """Move the pages in use (refs > 0) to the lowest ids, in place on k_cache / v_cache (and bounds; a cache in 8 bits is
    given with its k_scale and v_scale, which move too, and has no bounds).  Returns the new block_table and refs, remap
    [num_blocks] (a page's new id, -1 for a free one) and live [1] (pages in use).  In ``out``, block_table and refs may be
    the input tensors themselves, for an update in place; otherwise the outputs lie apart from the inputs and from one
    another."""
    L = library()
    ix = _index_of("k_cache", k_cache, 4)
    if ix != torch.cuda.current_device():
        with torch.cuda.device(ix):
            return kv_compact(k_cache, v_cache, block_table, refs, bounds=bounds, k_scale=k_scale, v_scale=v_scale, out=out,
                              workspace=workspace, status=status)
    call, cache_args = _pool_cache("ts_kv_compact", k_cache, v_cache, k_scale, v_scale, ix)
    NB, Hkv, bs, d = k_cache.shape
    if k_scale is None:
        cache_args.insert(3, None if bounds is None else _arg("bounds", bounds, ix, _BF16, (NB, Hkv, 2, d)))
    elif bounds is not None:
        raise ValueError("bounds belong to a cache in bf16 or fp32")
    B, width = table = block_table.shape
    args = [*cache_args, _arg("block_table", block_table, ix, _I32, table), width, _arg("refs", refs, ix, _I32, (NB,)), B]
    made = out is None
    if made:
        out = dict(block_table=torch.empty_like(block_table), refs=torch.empty_like(refs), remap=torch.empty_like(refs),
                   live=torch.empty((1,), dtype=_I32, device=refs.device))
    ws, ws_bytes, keep = _scratch(L.ts_kv_compact_workspace(NB), refs, workspace)
    rc = call(*args, *_out_args(out, ix, made, block_table=(_I32, table), refs=(_I32, (NB,)), remap=(_I32, (NB,)),
                                live=(_I32, (1,))), ws, ws_bytes, _status_arg(status, ix), _raw_stream(ix))
    if rc == _INVALID and not made:
        _apart(out, ("block_table", "refs"), block_table=block_table, refs=refs, k_cache=k_cache, v_cache=v_cache, bounds=bounds,
               k_scale=k_scale, v_scale=v_scale)
    _check(rc)
    return out


def _fp8_cache(k_cache, v_cache, k_scale, v_scale, ix):
    """Addresses and sizes of an 8-bit cache: codes [num_blocks,Hkv,bs,d] e4m3, scales [num_blocks,Hkv,bs/sb] fp32."""
    NB, Hkv, bs, d = cache = k_cache.shape
    if k_scale.dim() != 3 or k_scale.shape[2] < 1 or bs % k_scale.shape[2]:
        raise ValueError(f"k_scale must have shape [{NB}, {Hkv}, a divisor of {bs}], got {list(k_scale.shape)}")
    scales = (NB, Hkv, k_scale.shape[2])
    at = [_arg("k_cache", k_cache, ix, _E4M3, cache), _arg("v_cache", v_cache, ix, _E4M3, cache),
          _arg("k_scale", k_scale, ix, _F32, scales), _arg("v_scale", v_scale, ix, _F32, scales)]
    return at, (NB, bs, bs // scales[2], Hkv, d)


def _rows_arg(name: str, t: torch.Tensor, ix: int, dtype, shape):
    """The address and strides (sequences, rows, heads) of a tensor whose head rows are contiguous."""
    if t.get_device() != ix or t.dtype is not dtype or t.shape != shape:
        _refuse(name, t.contiguous(), ix, dtype, shape)
    if t.stride(3) != 1 and shape[3] != 1:
        raise ValueError(f"{name} must have contiguous head rows, got strides {list(t.stride())}")
    return t.data_ptr(), (ctypes.c_int64 * 3)(*t.stride()[:3])


def kv_write_fp8(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                 v_scale: torch.Tensor, block_table: torch.Tensor, start_len: torch.Tensor, *,
                 length: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None) -> None:
    """Quantise rows of k, v [B,n,Hkv,d] (bf16 or fp32; strides are free but for contiguous head rows) into the cache, in
    place: codes k_cache, v_cache [num_blocks,Hkv,bs,d] float8_e4m3fn and scales k_scale, v_scale [num_blocks,Hkv,bs/sb]
    fp32, one for every sb tokens of a page and head.  Row t of sequence b becomes position start_len[b] + t, t < length[b]
    (default: n).  A block's scale is the smallest power of two (2^-40 to 2^40) that brings its rows, those below start_len
    and the new ones, to at most 448; the sequence ends behind the write."""
    L = library()
    ix = _index_of("k_cache", k_cache, 4)
    if ix != torch.cuda.current_device():
        with torch.cuda.device(ix):
            return kv_write_fp8(k, v, k_cache, v_cache, k_scale, v_scale, block_table, start_len, length=length, status=status)
    cache, sizes = _fp8_cache(k_cache, v_cache, k_scale, v_scale, ix)
    B, width = block_table.shape
    if k.dim() != 4:
        raise ValueError(f"k must have 4 dimensions, got {list(k.shape)}")
    dt, shape = _dt(k), (B, k.shape[1], *k_cache.shape[1::2])
    k_at, k_strides = _rows_arg("k", k, ix, k.dtype, shape)
    v_at, v_strides = _rows_arg("v", v, ix, k.dtype, shape)
    _check(L.ts_kv_write_fp8(k_at, v_at, dt, k_strides, v_strides, *cache, *sizes,
                             _arg("block_table", block_table, ix, _I32, (B, width)), width,
                             _arg("start_len", start_len, ix, _I32, (B,)),
                             None if length is None else _arg("length", length, ix, _I32, (B,)), B, shape[1],
                             _status_arg(status, ix), _raw_stream(ix)))


def kv_read_fp8(k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                block_table: torch.Tensor, prefix_len: torch.Tensor, n: int, *, start_len: Optional[torch.Tensor] = None,
                dtype: torch.dtype = torch.bfloat16, out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                status: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The values k, v [B,n,Hkv,d] (bf16, in which they are exact, or fp32) of positions start_len[b] .. start_len[b] + n - 1
    (default: from 0); rows at and behind prefix_len[b] are 0."""
    L = library()
    ix = _index_of("k_cache", k_cache, 4)
    if ix != torch.cuda.current_device():
        with torch.cuda.device(ix):
            return kv_read_fp8(k_cache, v_cache, k_scale, v_scale, block_table, prefix_len, n, start_len=start_len, dtype=dtype,
                               out=out, status=status)
    cache, sizes = _fp8_cache(k_cache, v_cache, k_scale, v_scale, ix)
    B, width = block_table.shape
    shape = (B, n, *k_cache.shape[1::2])
    if out is None:
        k, v = (torch.empty(shape, dtype=dtype, device=k_cache.device) for _ in range(2))
    else:
        k, v = out
        dtype = k.dtype
    dt = _dt(k)
    _check(L.ts_kv_read_fp8(*cache, *sizes, _arg("block_table", block_table, ix, _I32, (B, width)), width,
                            _arg("prefix_len", prefix_len, ix, _I32, (B,)),
                            None if start_len is None else _arg("start_len", start_len, ix, _I32, (B,)), B, n,
                            _arg("k", k, ix, dtype, shape), _arg("v", v, ix, dtype, shape), dt, _status_arg(status, ix),
                            _raw_stream(ix)))
    return k, v


def kv_commit_fp8(k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                  block_table: torch.Tensor, prefix_len: torch.Tensor, accept_path: torch.Tensor, accept_len: torch.Tensor, *,
                  out: Optional[Dict[str, torch.Tensor]] = None,
                  status: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """kv_commit on an 8-bit cache: the accepted path's rows move in the caches (in place, quantised again with the block they
    move to).  Returns the new block_table and prefix_len, freed_blocks [B,max_blocks] (-1 padded) and freed_count [B].
    In ``out``, block_table and prefix_len may be the input tensors themselves; otherwise the outputs lie apart from the
    inputs and from one another."""
    L = library()
    ix = _index_of("k_cache", k_cache, 4)
    if ix != torch.cuda.current_device():
        with torch.cuda.device(ix):
            return kv_commit_fp8(k_cache, v_cache, k_scale, v_scale, block_table, prefix_len, accept_path, accept_len, out=out,
                                 status=status)
    cache, sizes = _fp8_cache(k_cache, v_cache, k_scale, v_scale, ix)
    B, width = table = block_table.shape
    m = accept_path.shape[1]
    args = [*cache, *sizes, _arg("block_table", block_table, ix, _I32, table), width,
            _arg("prefix_len", prefix_len, ix, _I32, (B,)), _arg("accept_path", accept_path, ix, _I32, (B, m)),
            _arg("accept_len", accept_len, ix, _I32, (B,)), B, m]
    made = out is None
    if made:
        out = dict(block_table=torch.empty_like(block_table), prefix_len=torch.empty_like(prefix_len),
                   freed_blocks=torch.empty_like(block_table), freed_count=torch.empty_like(prefix_len))
    rc = L.ts_kv_commit_fp8(*args, *_out_args(out, ix, made, block_table=(_I32, table), prefix_len=(_I32, (B,)),
                                              freed_blocks=(_I32, table), freed_count=(_I32, (B,))), _status_arg(status, ix),
                            _raw_stream(ix))
    if rc == _INVALID and not made:
        _apart(out, ("block_table", "prefix_len"), block_table=block_table, prefix_len=prefix_len, accept_path=accept_path,
               accept_len=accept_len, k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale)
    _check(rc)
    return out


def tree_attention_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                       v_scale: torch.Tensor, block_table: torch.Tensor, prefix_len: torch.Tensor, mask: torch.Tensor, *,
                       max_prefix: int, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                       lse: Optional[torch.Tensor] = None, with_lse: bool = True, workspace: Optional[torch.Tensor] = None,
                       status: Optional[torch.Tensor] = None):
    """Tree attention over an 8-bit cache (codes float8_e4m3fn and scales fp32, as kv_write_fp8 fills them).  q
    [B,m,Hq,d] bf16 or fp32; the rest as ``tree_attention``.  Returns (out, lse)."""
    L = library()
    ix = _index_of("q", q, 4)
    if ix != torch.cuda.current_device():
        with torch.cuda.device(ix):
            return tree_attention_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, prefix_len, mask, max_prefix=max_prefix,
                                      scale=scale, out=out, lse=lse, with_lse=with_lse, workspace=workspace, status=status)
    dtype, dt = q.dtype, _dt(q)
    B, m, Hq, d = shape = q.shape
    _index_of("k_cache", k_cache, 4)
    cache, (NB, bs, sb, Hkv, d2) = _fp8_cache(k_cache, v_cache, k_scale, v_scale, ix)
    if d2 != d:
        raise ValueError("cache shapes do not match q")
    width = block_table.shape[1]
    # (given ones are checked, new ones are not)
    out_at = None if out is None else _arg("out", out, ix, dtype, shape)
    lse_at = None if lse is None else _arg("lse", lse, ix, _F32, (B, m, Hq))
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        out_at = out.data_ptr()
    if lse is None and with_lse:
        lse = torch.empty((B, m, Hq), dtype=_F32, device=q.device)
        lse_at = lse.data_ptr()
    need = L.ts_tree_attention_fp8_workspace(dt, B, m, Hq, Hkv, d, max_prefix, bs)
    if need == 0:
        raise TreeSpecError("invalid tree_attention_fp8 sizes")
    ws, ws_bytes, keep = _scratch(need, q, workspace) if need > 256 else (None, 0, None)
    _check(L.ts_tree_attention_fp8(_arg("q", q, ix, dtype, shape), dt, *cache, NB, bs, sb,
                                   _arg("block_table", block_table, ix, _I32, (B, width)), width,
                                   _arg("prefix_len", prefix_len, ix, _I32, (B,)), max_prefix,
                                   _arg("mask", mask, ix, _I64, (B, m, (m + 63) // 64)), B, m, Hq, Hkv, d,
                                   1.0 / math.sqrt(d) if scale is None else scale, out_at, lse_at, ws, ws_bytes,
                                   _status_arg(status, ix), _raw_stream(ix)))
    return out, lse

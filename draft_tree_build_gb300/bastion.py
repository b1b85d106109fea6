"""Python binding of the C ABI in ``include/bastion.h`` and
``include/bastion_cache.h`` (ctypes; argument checks and marshalling, the paged cache's also in C, csrc/marshal.c).
Every function takes CUDA tensors, passes their device
pointers and the current stream to ``libbastion.so``, and raises on a negative
return code.  All computation happens in the library's kernels; there is no
fallback path: if the library cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import struct
import warnings
from dataclasses import dataclass

import torch

from . import _build

BASTION_F32 = 0
BASTION_BF16 = 1
BASTION_F16 = 2

STATUS_NONFINITE = 1
STATUS_EMPTY_ROW = 2
STATUS_BAD_COST = 4
STATUS_KV_OVERFLOW = 8
STATUS_BAD_TREE = 16
STATUS_BAD_WEIGHT = 32
STATUS_BAD_PAGE = 64
STATUS_BAD_ROW = 128
STATUS_TIMEOUT = 1 << 30

# the exported C symbols, in header order
SYMBOLS = (
    "bastion_version", "bastion_status_string",
    "bastion_topk_marginals_workspace_bytes", "bastion_topk_marginals",
    "bastion_lm_head_topk_workspace_bytes", "bastion_lm_head_topk",
    "bastion_build_tree", "bastion_build_tree_mixture_workspace_bytes", "bastion_build_tree_mixture",
    "bastion_calibrate_cost",
    "bastion_tree_attention_workspace_bytes", "bastion_tree_attention",
    "bastion_verify_greedy_workspace_bytes", "bastion_verify_greedy",
    "bastion_verify_sample_workspace_bytes", "bastion_verify_sample",
    "bastion_verify_greedy_noalloc",
)

# the exported C symbols of the paged cache (include/bastion_cache.h), in header order
CACHE_SYMBOLS = (
    "bastion_paged_append_workspace_bytes", "bastion_paged_append",
    "bastion_paged_attention_workspace_bytes", "bastion_paged_attention",
    "bastion_paged_evict_workspace_bytes", "bastion_paged_evict",
)


class BastionError(RuntimeError):
    pass


# bastion_paged_cache of include/bastion_cache.h: k_pool, v_pool, n_pages, stride_page, stride_slot, stride_head,
# page_table, dtype, B, Hkv, D, page_size, max_pages
_PAGED_CACHE = struct.Struct("@PPqqqqPiiiiii")


_lib = None
_marshal = None  # the paged cache's short way past ctypes (csrc/marshal.c), loaded with the library


def _load_marshal(L):
    loader = importlib.machinery.ExtensionFileLoader("bastion_marshal", _build.MARSHAL)
    m = importlib.util.module_from_spec(importlib.util.spec_from_loader("bastion_marshal", loader))
    loader.exec_module(m)
    address = lambda f: ctypes.cast(f, ctypes.c_void_p).value  # noqa: E731
    m.init(torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.uint8, torch._C._cuda_getDevice,
           torch._C._cuda_getCurrentRawStream, address(L.bastion_paged_append), address(L.bastion_paged_attention),
           address(L.bastion_paged_evict))
    return m


def _short_way(L):
    """The compiled short way, or None where it is not there or cannot be loaded: the binding's own checks and ctypes
    do the same then, a few microseconds a call later."""
    if not _build.marshal_up_to_date():
        return None
    try:
        return _load_marshal(L)
    except (ImportError, OSError, AttributeError) as e:  # AttributeError: a torch without CUDA has no current stream
        warnings.warn(f"the paged cache's calls take the way through ctypes: {e}")
        return None


def library_path() -> str:
    return _build.LIB


def lib(build_if_missing: bool = True):
    """Load libbastion.so (building it in-tree first if it is missing or stale)."""
    global _lib, _marshal
    if _lib is not None:
        return _lib
    if build_if_missing:
        _build.build()
    if not os.path.exists(_build.LIB):
        raise BastionError(f"libbastion.so not found at {_build.LIB}; run __graft_entry__.build()")
    L = ctypes.CDLL(_build.LIB)
    vp, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    L.bastion_version.restype = ctypes.c_char_p
    L.bastion_version.argtypes = []
    L.bastion_status_string.restype = ctypes.c_char_p
    L.bastion_status_string.argtypes = [i32]
    L.bastion_topk_marginals_workspace_bytes.restype = sz
    L.bastion_topk_marginals_workspace_bytes.argtypes = [i32, i32, i32, i32]
    L.bastion_topk_marginals.restype = i32
    L.bastion_topk_marginals.argtypes = [vp, i32, i32, i32, i32, i64, i32, vp, vp, vp, vp, vp, sz, vp, vp]
    L.bastion_lm_head_topk_workspace_bytes.restype = sz
    L.bastion_lm_head_topk_workspace_bytes.argtypes = [i32, i32, i32, i32]
    L.bastion_lm_head_topk.restype = i32
    L.bastion_lm_head_topk.argtypes = [vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp, vp]
    L.bastion_build_tree.restype = i32
    L.bastion_build_tree.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, i32, vp] + [vp] * 11 + [vp]
    L.bastion_build_tree_mixture_workspace_bytes.restype = sz
    L.bastion_build_tree_mixture_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    L.bastion_build_tree_mixture.restype = i32
    L.bastion_build_tree_mixture.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, i32,
                                             vp] + [vp] * 9 + [vp, sz, vp, vp]
    L.bastion_calibrate_cost.restype = i32
    L.bastion_calibrate_cost.argtypes = [vp, vp, i32] + [ctypes.c_double] * 7 + [i32, vp, vp, vp, vp]
    L.bastion_tree_attention_workspace_bytes.restype = sz
    L.bastion_tree_attention_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i64]
    L.bastion_tree_attention.restype = i32
    L.bastion_tree_attention.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32, i64, vp, vp, vp, f32,
                                         vp, vp, sz, vp, vp]
    L.bastion_verify_greedy_workspace_bytes.restype = sz
    L.bastion_verify_greedy_workspace_bytes.argtypes = [i32, i32, i32]
    L.bastion_verify_greedy.restype = i32
    L.bastion_verify_greedy.argtypes = [vp, i32, i32, i32, i32, i64, i32, vp, vp, vp, vp, vp, vp, vp,
                                        vp, sz, vp, vp]
    L.bastion_verify_sample_workspace_bytes.restype = sz
    L.bastion_verify_sample_workspace_bytes.argtypes = [i32, i32, i32]
    L.bastion_verify_sample.restype = i32
    L.bastion_verify_sample.argtypes = [vp, i32, i32, i32, i32, i64, i32, f32, vp, vp, vp, vp, vp, vp,
                                        vp, vp, vp, sz, vp, vp]
    L.bastion_verify_greedy_noalloc.restype = i32
    L.bastion_verify_greedy_noalloc.argtypes = [vp, i32, i32, i32, i32, i64, i32, vp, vp, vp, vp, vp,
                                                vp, vp, vp, vp]
    L.bastion_paged_append_workspace_bytes.restype = sz
    L.bastion_paged_append_workspace_bytes.argtypes = [i32]
    L.bastion_paged_append.restype = i32
    L.bastion_paged_append.argtypes = [vp, vp, vp, i32, i64, i64, i64, vp, i32, vp, vp, vp, vp, vp, vp, vp,
                                       vp, sz, vp, vp]
    L.bastion_paged_attention_workspace_bytes.restype = sz
    L.bastion_paged_attention_workspace_bytes.argtypes = [i32, i32, i32, i32, i64, i32]
    L.bastion_paged_attention.restype = i32
    L.bastion_paged_attention.argtypes = [vp, vp, i32, i64, vp, f32, vp, vp, vp, vp, vp, sz, vp, vp]
    L.bastion_paged_evict_workspace_bytes.restype = sz
    L.bastion_paged_evict_workspace_bytes.argtypes = [i32, i32, i64]
    L.bastion_paged_evict.restype = i32
    L.bastion_paged_evict.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, vp, vp, vp, vp, sz, vp, vp]
    _marshal = _short_way(L)
    _lib = L
    return L


def _p(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise BastionError("tensor must live on a CUDA device")
    return ctypes.c_void_p(t.data_ptr())


def _p_rows(t):
    """Target logits: a device tensor, or a pinned (page-locked) host tensor, which
    the verify kernels read in place over the host link (only the rows of the
    tree's nodes cross it)."""
    if t.is_cuda or (t.device.type == "cpu" and t.is_pinned()):
        return ctypes.c_void_p(t.data_ptr())
    raise BastionError("target logits must live on a CUDA device or in pinned host memory")


def _s(stream):
    st = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(st.cuda_stream)


def _dtype(t) -> int:
    if t.dtype == torch.float32:
        return BASTION_F32
    if t.dtype == torch.bfloat16:
        return BASTION_BF16
    raise BastionError(f"logits must be float32 or bfloat16, got {t.dtype}")


def _check(rc: int, name: str):
    if rc != 0:
        raise BastionError(f"{name}: {bastion_status_string(rc)} ({rc})")


def _rows_view(x, dims):
    """Row stride (elements) of a [B, n, V] tensor whose last dim is contiguous and
    whose B*n rows are evenly strided."""
    if x.dim() != dims:
        raise BastionError(f"expected {dims} dims, got {tuple(x.shape)}")
    if x.stride(-1) != 1:
        raise BastionError("last dimension must be contiguous")
    ld = x.stride(-2)
    if x.shape[0] > 1 and x.stride(0) != ld * x.shape[1]:
        raise BastionError("rows must be evenly strided")
    return ld


# --------------------------------------------------------------------------- C ABI mirrors

def bastion_version() -> str:
    return lib().bastion_version().decode()


def bastion_status_string(code: int) -> str:
    return lib().bastion_status_string(int(code)).decode()


def bastion_topk_marginals_workspace_bytes(B: int, b: int, V: int, K: int) -> int:
    return int(lib().bastion_topk_marginals_workspace_bytes(B, b, V, K))


def bastion_topk_marginals(logits, K, topk_logq, topk_logit, topk_tok, lse, workspace, status,
                           stream=None):
    """logits [B, b, V] (fp32/bf16, last dim contiguous); outputs [B, b, K] / [B, b]."""
    B, b, V = logits.shape
    ld = _rows_view(logits, 3)
    rc = lib().bastion_topk_marginals(_p(logits), _dtype(logits), B, b, V, ld, int(K), _p(topk_logq),
                                      _p(topk_logit), _p(topk_tok), _p(lse), _p(workspace),
                                      workspace.numel() * workspace.element_size(), _p(status), _s(stream))
    _check(rc, "bastion_topk_marginals")


def bastion_lm_head_topk_workspace_bytes(B: int, b: int, V: int, K: int) -> int:
    return int(lib().bastion_lm_head_topk_workspace_bytes(B, b, V, K))


def bastion_lm_head_topk(hidden, weight, K, topk_logq, topk_logit, topk_tok, lse, workspace, status,
                         stream=None):
    """hidden [B, b, H] and weight [V, H], contiguous bfloat16; outputs as
    bastion_topk_marginals for the logits hidden . weight^T."""
    for name, t in (("hidden", hidden), ("weight", weight)):
        if t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise BastionError(f"lm head: {name} must be contiguous bfloat16")
    B, b, H = hidden.shape
    V = weight.shape[0]
    if weight.dim() != 2 or weight.shape[1] != H:
        raise BastionError("lm head: weight must be [V, H] with the hidden size of hidden")
    rc = lib().bastion_lm_head_topk(_p(hidden), _p(weight), B, b, H, V, int(K), _p(topk_logq),
                                    _p(topk_logit), _p(topk_tok), _p(lse), _p(workspace),
                                    workspace.numel() * workspace.element_size(), _p(status), _s(stream))
    _check(rc, "bastion_lm_head_topk")


def bastion_build_tree(topk_logit, topk_tok, lse, n_max, root_token, ctx_len, cost_ms, l_ar,
                       n_nodes, parent, depth, pos_id, token, rank, log_rho, a_hat, speedup,
                       anc_mask, status, stream=None):
    B, b, K = topk_logit.shape
    per_req = 1 if (cost_ms.dim() == 2 and cost_ms.shape[0] == B and B > 1) else 0
    rc = lib().bastion_build_tree(_p(topk_logit), _p(topk_tok), _p(lse), B, b, K, int(n_max),
                                  _p(root_token), _p(ctx_len), _p(cost_ms), per_req, _p(l_ar),
                                  _p(n_nodes), _p(parent), _p(depth), _p(pos_id), _p(token), _p(rank),
                                  _p(log_rho), _p(a_hat), _p(speedup), _p(anc_mask), _p(status), _s(stream))
    _check(rc, "bastion_build_tree")


def bastion_build_tree_mixture_workspace_bytes(B: int, Z: int, b: int, K: int, n_max: int) -> int:
    return int(lib().bastion_build_tree_mixture_workspace_bytes(B, Z, b, K, n_max))


def bastion_build_tree_mixture(topk_logit, topk_tok, lse, pi, n_max, root_token, ctx_len, cost_ms, l_ar,
                               n_nodes, parent, depth, pos_id, token, log_rho, a_hat, speedup, anc_mask,
                               workspace, status, stream=None):
    """topk_logit/tok [B, Z, b, K], lse [B, Z, b] float64, pi [B, Z] float64 (contiguous);
    workspace: bastion_build_tree_mixture_workspace_bytes(B, Z, b, K, n_max) bytes."""
    B, Z, b, K = topk_logit.shape
    for t in (topk_logit, topk_tok, lse, pi):
        if not t.is_contiguous():
            raise BastionError("mixture tree inputs must be contiguous")
    # the library reads these bytes as the stated types; a wrong dtype would be read as garbage
    for name, t, dt in (("topk_logit", topk_logit, torch.float32), ("topk_tok", topk_tok, torch.int32),
                        ("lse", lse, torch.float64), ("pi", pi, torch.float64)):
        if t.dtype != dt:
            raise BastionError(f"mixture tree: {name} must be {dt}, got {t.dtype}")
    if tuple(topk_tok.shape) != (B, Z, b, K) or tuple(lse.shape) != (B, Z, b) or tuple(pi.shape) != (B, Z):
        raise BastionError("mixture tree: topk_tok [B,Z,b,K], lse [B,Z,b] and pi [B,Z] must match topk_logit")
    if cost_ms.numel() not in (n_max + 1, B * (n_max + 1)):
        raise BastionError("mixture tree: cost_ms must hold n_max + 1 entries, or n_max + 1 per request")
    per_req = 1 if (cost_ms.dim() == 2 and cost_ms.shape[0] == B and B > 1) else 0
    rc = lib().bastion_build_tree_mixture(_p(topk_logit), _p(topk_tok), _p(lse), _p(pi), B, Z, b, K,
                                          int(n_max), _p(root_token), _p(ctx_len), _p(cost_ms), per_req,
                                          _p(l_ar), _p(n_nodes), _p(parent), _p(depth), _p(pos_id),
                                          _p(token), _p(log_rho), _p(a_hat), _p(speedup), _p(anc_mask),
                                          _p(workspace), workspace.numel() * workspace.element_size(),
                                          _p(status), _s(stream))
    _check(rc, "bastion_build_tree_mixture")


def bastion_calibrate_cost(sample_n, sample_ms, roofline: dict, t_draft, n_max, cost_ms, params, status,
                           stream=None):
    """sample_n / sample_ms [n] float32 on the device; cost_ms [n_max + 1], params [2] float32.
    roofline: bytes0, bytes1, flops0, flops1, bw, peak (roof(N) in ms)."""
    r = roofline
    rc = lib().bastion_calibrate_cost(_p(sample_n), _p(sample_ms), int(sample_n.numel()), r["bytes0"],
                                      r["bytes1"], r["flops0"], r["flops1"], r["bw"], r["peak"],
                                      float(t_draft), int(n_max), _p(cost_ms), _p(params), _p(status),
                                      _s(stream))
    _check(rc, "bastion_calibrate_cost")


def bastion_tree_attention_workspace_bytes(B, n_max, Hq, Hkv, D, L_cap) -> int:
    return int(lib().bastion_tree_attention_workspace_bytes(B, n_max, Hq, Hkv, D, L_cap))


def bastion_tree_attention(q, k_cache, v_cache, ctx_len, n_nodes, anc_mask, scale, out, workspace,
                           status, stream=None):
    """q/out [B, n_max, Hq, D], k/v [B, L_cap, Hkv, D], bf16 contiguous."""
    B, n_max, Hq, D = q.shape
    L_cap, Hkv = k_cache.shape[1], k_cache.shape[2]
    for t in (q, k_cache, v_cache, out):
        if t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise BastionError("attention tensors must be contiguous bfloat16")
    rc = lib().bastion_tree_attention(_p(q), _p(k_cache), _p(v_cache), B, n_max, Hq, Hkv, D, L_cap,
                                      _p(ctx_len), _p(n_nodes), _p(anc_mask), float(scale), _p(out),
                                      _p(workspace), workspace.numel() * workspace.element_size(),
                                      _p(status), _s(stream))
    _check(rc, "bastion_tree_attention")


def bastion_verify_greedy_workspace_bytes(B: int, n_max: int, V: int) -> int:
    return int(lib().bastion_verify_greedy_workspace_bytes(B, n_max, V))


def bastion_verify_greedy(target_logits, b, n_nodes, parent, token, argmax, accept_len,
                          accept_nodes, out_tokens, workspace, status, stream=None):
    """target_logits [B, n_max, V] (fp32/bf16, last dim contiguous), on the device or in
    pinned host memory."""
    B, n_max, V = target_logits.shape
    ld = _rows_view(target_logits, 3)
    rc = lib().bastion_verify_greedy(_p_rows(target_logits), _dtype(target_logits), B, n_max, V, ld, int(b),
                                     _p(n_nodes), _p(parent), _p(token), _p(argmax), _p(accept_len),
                                     _p(accept_nodes), _p(out_tokens), _p(workspace),
                                     workspace.numel() * workspace.element_size(), _p(status), _s(stream))
    _check(rc, "bastion_verify_greedy")


def bastion_verify_sample_workspace_bytes(B: int, n_max: int, V: int) -> int:
    return int(lib().bastion_verify_sample_workspace_bytes(B, n_max, V))


def bastion_verify_sample(target_logits, b, temperature, uniforms, n_nodes, parent, token, sampled,
                          accept_len, accept_nodes, out_tokens, workspace, status, stream=None):
    """target_logits [B, n_max, V] (fp32/bf16, last dim contiguous); uniforms [B, n_max] float64."""
    B, n_max, V = target_logits.shape
    ld = _rows_view(target_logits, 3)
    if uniforms.dtype != torch.float64 or not uniforms.is_contiguous():
        raise BastionError("uniforms must be a contiguous float64 tensor")
    rc = lib().bastion_verify_sample(_p_rows(target_logits), _dtype(target_logits), B, n_max, V, ld, int(b),
                                     float(temperature), _p(uniforms), _p(n_nodes), _p(parent), _p(token),
                                     _p(sampled), _p(accept_len), _p(accept_nodes), _p(out_tokens),
                                     _p(workspace), workspace.numel() * workspace.element_size(),
                                     _p(status), _s(stream))
    _check(rc, "bastion_verify_sample")


def bastion_verify_greedy_noalloc(target_logits, b, n_nodes, parent, token, argmax, accept_len,
                                  accept_nodes, out_tokens, status, stream=None):
    """Same as bastion_verify_greedy without a workspace argument, for callers that
    cannot allocate device memory: the library uses a fixed 128 KiB scratch array
    of its own (B <= 4096, B * n_max <= 16384).  Calls that overlap on the GPU race
    on that array."""
    B, n_max, V = target_logits.shape
    ld = _rows_view(target_logits, 3)
    rc = lib().bastion_verify_greedy_noalloc(_p_rows(target_logits), _dtype(target_logits), B, n_max, V, ld,
                                             int(b), _p(n_nodes), _p(parent), _p(token), _p(argmax),
                                             _p(accept_len), _p(accept_nodes), _p(out_tokens), _p(status),
                                             _s(stream))
    _check(rc, "bastion_verify_greedy_noalloc")


# --------------------------------------------------------------------------- paged cache

# These calls take a few microseconds on the GPU, so that what the host spends on one counts: a call whose arguments
# are right goes through csrc/marshal.c, which checks them and calls the library; any other comes back here, where the
# same checks say what is wrong.

_CACHE_DTYPES = {torch.bfloat16: BASTION_BF16, torch.float16: BASTION_F16}


def _need(names, dev, dtype, shape, *tensors):
    """Contiguous tensors (None: left out) of one type and shape on device dev: the library reads their bytes as
    such.  names: a text, split when one fails."""
    for i, t in enumerate(tensors):
        if t is not None and (t.dtype is not dtype or t.shape != shape or t.get_device() != dev
                              or not t.is_contiguous()):
            name = names.split()[i]
            if t.get_device() != dev:
                raise BastionError(f"paged cache: {name} is on {t.device}, the page table on another device")
            raise BastionError(f"paged cache: {name} must be contiguous {dtype} {list(shape)}, got {t.dtype} "
                               f"{list(t.shape)}, strides {t.stride()}")


def _launch_on(dev, stream, workspace):
    """Checks the workspace and that dev is the current CUDA device, where the launches go; the stream's handle."""
    if workspace.dtype is not torch.uint8 or workspace.get_device() != dev or not workspace.is_contiguous():
        raise BastionError("paged cache: the workspace must be contiguous uint8 (bastion.workspace) on the tensors' "
                           "device")
    if dev < 0:
        raise BastionError("tensor must live on a CUDA device")
    if dev != torch.cuda.current_device():
        raise BastionError(f"paged cache: the tensors are on cuda:{dev}, the current device is "
                           f"cuda:{torch.cuda.current_device()}")
    # the current stream's handle without a Stream object, which costs 3 us to make
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _same_strides(a, b):
    """Of two tensors of one shape: the stride of a dimension of length 1 says nothing."""
    x, y = a.stride(), b.stride()
    return x == y or all(n == 1 or i == j for n, i, j in zip(a.shape, x, y))


def _cache(k_pool, v_pool, page_table):
    """Checks the cache; (device, B, Hkv, D, slots of a request, the struct's bytes, which ctypes passes by address).
    Pools [n_pages, page_size, Hkv, D] of any strides (a head-major pool is a transposed view), page_table
    [B, max_pages] int32."""
    shape, st, dev = k_pool.shape, k_pool.stride(), page_table.get_device()
    if len(shape) != 4 or shape != v_pool.shape or k_pool.dtype is not v_pool.dtype:
        raise BastionError("paged cache: the pools must be [n_pages, page_size, Hkv, D], of one shape and dtype")
    dt = _CACHE_DTYPES.get(k_pool.dtype)
    if dt is None:
        raise BastionError(f"paged cache: the pools must be bfloat16 or float16, got {k_pool.dtype}")
    if st[3] != 1 or not _same_strides(k_pool, v_pool):
        raise BastionError("paged cache: the pools must have equal strides and a contiguous last dimension")
    table = page_table.shape
    if len(table) != 2 or page_table.dtype is not torch.int32 or not page_table.is_contiguous():
        raise BastionError("paged cache: page_table must be contiguous int32 [B, max_pages]")
    if k_pool.get_device() != dev or v_pool.get_device() != dev:
        raise BastionError(f"paged cache: pools on {k_pool.device} and {v_pool.device}, page_table on "
                           f"{page_table.device}")
    n_pages, page, Hkv, D = shape
    B, max_pages = table
    return dev, B, Hkv, D, max_pages * page, _PAGED_CACHE.pack(
        k_pool.data_ptr(), v_pool.data_ptr(), n_pages, st[0], st[1], st[2], page_table.data_ptr(), dt, B, Hkv, D, page,
        max_pages)


def _ptr(t):
    return None if t is None else t.data_ptr()


def bastion_paged_append_workspace_bytes(B: int) -> int:
    return int(lib().bastion_paged_append_workspace_bytes(B))


def bastion_paged_append(k_new, v_new, k_pool, v_pool, page_table, seq_len, seq_len_out, workspace, status,
                         rows=None, n_new=None, acc=None, pos=None, n_seen=None, n_seen_out=None, stream=None):
    """k_new/v_new [B, n_rows, Hkv, D] (equal strides, last dim contiguous) enter the cache's next slots: the
    rows listed in rows [B, m] (a negative entry ends a list; Verify.accept_nodes fits), or the first n_new [B].
    seq_len_out may be seq_len, n_seen_out n_seen."""
    if _marshal is not None:
        rc = _marshal.append(k_new, v_new, k_pool, v_pool, page_table, seq_len, seq_len_out, workspace, status, rows,
                             n_new, acc, pos, n_seen, n_seen_out, stream)
        if rc is not None:
            return _check(rc, "bastion_paged_append")
    dev, B, Hkv, D, cap, cache = _cache(k_pool, v_pool, page_table)
    new, st, dtype = k_new.shape, k_new.stride(), k_pool.dtype
    if len(new) != 4 or new != v_new.shape or new[0] != B or new[2] != Hkv or new[3] != D \
            or k_new.dtype is not dtype or v_new.dtype is not dtype:
        raise BastionError("paged append: k_new and v_new must be [B, n_rows, Hkv, D] of the pools' dtype")
    if st[3] != 1 or not _same_strides(k_new, v_new):
        raise BastionError("paged append: k_new and v_new must have equal strides and a contiguous last dimension")
    if k_new.get_device() != dev or v_new.get_device() != dev:
        raise BastionError("paged append: k_new and v_new must be on the pools' device")
    m = n_rows = new[1]
    if rows is not None:
        if rows.dim() != 2:
            raise BastionError("paged append: rows must be [B, m]")
        m = rows.shape[1]
        _need("rows", dev, torch.int32, (B, m), rows)
    _need("seq_len seq_len_out status n_new n_seen n_seen_out", dev, torch.int32, (B,), seq_len, seq_len_out, status,
          n_new, n_seen, n_seen_out)
    if acc is not None or pos is not None:
        _need("acc", dev, torch.float32, (B, Hkv, cap), acc)
        _need("pos", dev, torch.int32, (B, Hkv, cap), pos)
    st_cuda = _launch_on(dev, stream, workspace)
    rc = lib().bastion_paged_append(cache, k_new.data_ptr(), v_new.data_ptr(), n_rows, st[0], st[1], st[2],
                                    _ptr(rows), m, _ptr(n_new), seq_len.data_ptr(), seq_len_out.data_ptr(),
                                    _ptr(n_seen), _ptr(n_seen_out), _ptr(acc), _ptr(pos), workspace.data_ptr(),
                                    workspace.numel(), status.data_ptr(), st_cuda)
    _check(rc, "bastion_paged_append")


def bastion_paged_attention_workspace_bytes(B: int, Hq: int, Hkv: int, D: int, cap: int, weights: bool) -> int:
    """cap: max_pages * page_size."""
    return int(lib().bastion_paged_attention_workspace_bytes(B, Hq, Hkv, D, cap, int(bool(weights))))


def bastion_paged_attention(q, k_pool, v_pool, page_table, seq_len, scale, out, workspace, status, lse=None,
                            acc=None, acc_out=None, stream=None):
    """q [B, Hq, D] (heads contiguous, any stride between requests), out [B, Hq, D] contiguous, lse [B, Hq]
    float32 or None; acc/acc_out [B, Hkv, max_pages * page_size] float32 or None (acc_out may be acc)."""
    if _marshal is not None:
        rc = _marshal.attention(q, k_pool, v_pool, page_table, seq_len, scale, out, workspace, status, lse, acc, acc_out,
                                stream)
        if rc is not None:
            return _check(rc, "bastion_paged_attention")
    dev, B, Hkv, D, cap, cache = _cache(k_pool, v_pool, page_table)
    qs, st, dtype = q.shape, q.stride(), q.dtype
    if len(qs) != 3 or dtype is not k_pool.dtype or qs[0] != B or qs[2] != D:
        raise BastionError("paged attention: q must be [B, Hq, D] of the pools' dtype")
    Hq = qs[1]
    if st[2] != 1 or (Hq > 1 and st[1] != D):
        raise BastionError("paged attention: the heads of q must be contiguous")
    if q.get_device() != dev:
        raise BastionError("paged attention: q must be on the pools' device")
    _need("out", dev, dtype, qs, out)
    _need("seq_len status", dev, torch.int32, (B,), seq_len, status)
    if lse is not None:
        _need("lse", dev, torch.float32, (B, Hq), lse)
    if acc is not None or acc_out is not None:
        _need("acc acc_out", dev, torch.float32, (B, Hkv, cap), acc, acc_out)
    st_cuda = _launch_on(dev, stream, workspace)
    rc = lib().bastion_paged_attention(cache, q.data_ptr(), Hq, st[0], seq_len.data_ptr(), scale, out.data_ptr(),
                                       _ptr(lse), _ptr(acc), _ptr(acc_out), workspace.data_ptr(), workspace.numel(),
                                       status.data_ptr(), st_cuda)
    _check(rc, "bastion_paged_attention")


def bastion_paged_evict_workspace_bytes(B: int, Hkv: int, cap: int) -> int:
    return int(lib().bastion_paged_evict_workspace_bytes(B, Hkv, cap))


def bastion_paged_evict(k_pool, v_pool, page_table, seq_len, n_seen, acc, pos, budget, n_sink, n_recent,
                        seq_len_out, acc_out, pos_out, workspace, status, stream=None):
    """Every request and KV head keeps budget slots: those of the n_sink first and n_recent last tokens, then the
    largest acc.  acc/pos [B, Hkv, max_pages * page_size]; each output may be its input."""
    if _marshal is not None:
        rc = _marshal.evict(k_pool, v_pool, page_table, seq_len, n_seen, acc, pos, budget, n_sink, n_recent, seq_len_out,
                            acc_out, pos_out, workspace, status, stream)
        if rc is not None:
            return _check(rc, "bastion_paged_evict")
    dev, B, Hkv, _, cap, cache = _cache(k_pool, v_pool, page_table)
    if not all(-(1 << 31) <= x < 1 << 31 for x in (budget, n_sink, n_recent)):  # ctypes would cut it to 32 bits
        raise BastionError("paged evict: budget, n_sink and n_recent must fit 32 bits")
    _need("seq_len n_seen seq_len_out status", dev, torch.int32, (B,), seq_len, n_seen, seq_len_out, status)
    _need("acc acc_out", dev, torch.float32, (B, Hkv, cap), acc, acc_out)
    _need("pos pos_out", dev, torch.int32, (B, Hkv, cap), pos, pos_out)
    st_cuda = _launch_on(dev, stream, workspace)
    rc = lib().bastion_paged_evict(cache, seq_len.data_ptr(), n_seen.data_ptr(), acc.data_ptr(), pos.data_ptr(),
                                   budget, n_sink, n_recent, seq_len_out.data_ptr(), acc_out.data_ptr(),
                                   pos_out.data_ptr(), workspace.data_ptr(), workspace.numel(), status.data_ptr(),
                                   st_cuda)
    _check(rc, "bastion_paged_evict")


# --------------------------------------------------------------------------- buffers

def workspace(nbytes: int, device) -> torch.Tensor:
    """A zero-filled, 256-byte aligned workspace (torch allocations are)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


@dataclass
class TopK:
    logq: torch.Tensor
    logit: torch.Tensor
    tok: torch.Tensor
    lse: torch.Tensor


@dataclass
class Tree:
    n_nodes: torch.Tensor
    parent: torch.Tensor
    depth: torch.Tensor
    pos_id: torch.Tensor
    token: torch.Tensor
    rank: torch.Tensor
    log_rho: torch.Tensor
    a_hat: torch.Tensor
    speedup: torch.Tensor
    anc_mask: torch.Tensor


@dataclass
class Verify:
    argmax: torch.Tensor
    accept_len: torch.Tensor
    accept_nodes: torch.Tensor
    out_tokens: torch.Tensor


def alloc_topk(B, b, K, device) -> TopK:
    return TopK(torch.empty(B, b, K, dtype=torch.float32, device=device),
                torch.empty(B, b, K, dtype=torch.float32, device=device),
                torch.empty(B, b, K, dtype=torch.int32, device=device),
                torch.empty(B, b, dtype=torch.float64, device=device))


def alloc_tree(B, n_max, device) -> Tree:
    W = (n_max + 31) // 32
    i = lambda: torch.full((B, n_max), -7, dtype=torch.int32, device=device)  # noqa: E731
    f = lambda: torch.full((B, n_max), float("nan"), dtype=torch.float32, device=device)  # noqa: E731
    return Tree(torch.zeros(B, dtype=torch.int32, device=device), i(), i(), i(), i(), i(), f(), f(), f(),
                torch.zeros(B, n_max, W, dtype=torch.int32, device=device))


def alloc_verify(B, n_max, b, device) -> Verify:
    return Verify(torch.full((B, n_max), -7, dtype=torch.int32, device=device),
                  torch.zeros(B, dtype=torch.int32, device=device),
                  torch.zeros(B, b + 1, dtype=torch.int32, device=device),
                  torch.zeros(B, b + 1, dtype=torch.int32, device=device))


class TreeStep:
    """One tree step (top-K marginals -> best-first tree -> greedy verify) over
    preallocated device buffers; ``capture()`` records the launches in a CUDA
    graph so a step replays with one host call."""

    def __init__(self, B, b, V, K, n_max, device, root_token, ctx_len, cost_ms, l_ar):
        self.B, self.b, self.V, self.K, self.n_max = B, b, V, K, n_max
        self.device = device
        self.topk = alloc_topk(B, b, K, device)
        self.tree = alloc_tree(B, n_max, device)
        self.ver = alloc_verify(B, n_max, b, device)
        self.status = torch.zeros(B, dtype=torch.int32, device=device)
        self.ws_topk = workspace(bastion_topk_marginals_workspace_bytes(B, b, V, K), device)
        self.ws_verify = workspace(bastion_verify_greedy_workspace_bytes(B, n_max, V), device)
        self.root_token = root_token.to(device=device, dtype=torch.int32)
        self.ctx_len = ctx_len.to(device=device, dtype=torch.int32)
        self.cost_ms = cost_ms.to(device=device, dtype=torch.float32)
        self.l_ar = l_ar.to(device=device, dtype=torch.float32)
        self.graph = None

    def draft(self, drafter_logits, stream=None):
        """Steps 1-3: marginals, then the tree (its size decides which target rows exist)."""
        t, tr = self.topk, self.tree
        bastion_topk_marginals(drafter_logits, self.K, t.logq, t.logit, t.tok, t.lse, self.ws_topk,
                               self.status, stream)
        bastion_build_tree(t.logit, t.tok, t.lse, self.n_max, self.root_token, self.ctx_len,
                           self.cost_ms, self.l_ar, tr.n_nodes, tr.parent, tr.depth, tr.pos_id,
                           tr.token, tr.rank, tr.log_rho, tr.a_hat, tr.speedup, tr.anc_mask,
                           self.status, stream)

    def set_sampling(self, temperature, uniforms):
        """Verify at temperature T > 0 with the uniforms [B, n_max] (float64 in
        [0, 1), refreshed by the caller between steps); T = 0 returns to greedy."""
        self.temperature = float(temperature)
        if self.temperature > 0:
            self.uniforms = uniforms.to(device=self.device, dtype=torch.float64).contiguous()
            self.ws_sample = workspace(bastion_verify_sample_workspace_bytes(self.B, self.n_max, self.V),
                                       self.device)

    def verify(self, target_logits, stream=None):
        """Step 4: verification of the tree against the target's logits (greedy,
        or sampled at the temperature set by set_sampling)."""
        tr, v = self.tree, self.ver
        if getattr(self, "temperature", 0.0) > 0:
            bastion_verify_sample(target_logits, self.b, self.temperature, self.uniforms, tr.n_nodes,
                                  tr.parent, tr.token, v.argmax, v.accept_len, v.accept_nodes,
                                  v.out_tokens, self.ws_sample, self.status, stream)
            return
        bastion_verify_greedy(target_logits, self.b, tr.n_nodes, tr.parent, tr.token, v.argmax,
                              v.accept_len, v.accept_nodes, v.out_tokens, self.ws_verify,
                              self.status, stream)

    def run(self, drafter_logits, target_logits, stream=None):
        self.draft(drafter_logits, stream)
        self.verify(target_logits, stream)

    def run_chunked(self, drafter_logits, target_logits, chunks):
        """The same step with the batch split into request chunks on their own
        streams (forked from and joined to the current stream).  A chunk's
        top-K starts after the previous chunk's top-K, so one chunk's tree build
        (a serial chain per request) overlaps the other chunks' sweeps.
        Requests are independent, so the results equal run()'s."""
        B = self.B
        chunks = max(1, min(chunks, B))
        bounds = [B * c // chunks for c in range(chunks + 1)]
        if getattr(self, "_chunk_state", None) is None or len(self._chunk_state) != chunks:
            self._chunk_state = []
            for c in range(chunks):
                nb = bounds[c + 1] - bounds[c]
                self._chunk_state.append((torch.cuda.Stream(device=self.device),
                                          workspace(bastion_verify_greedy_workspace_bytes(nb, self.n_max, self.V),
                                                    self.device)))
        main = torch.cuda.current_stream(self.device)
        t, tr, v = self.topk, self.tree, self.ver
        per_req_cost = self.cost_ms.dim() == 2 and self.cost_ms.shape[0] == B and B > 1
        prev = None
        for c in range(chunks):
            c0, c1 = bounds[c], bounds[c + 1]
            st, ws_v = self._chunk_state[c]
            st.wait_stream(main)
            if prev is not None:
                st.wait_event(prev)
            with torch.cuda.stream(st):
                bastion_topk_marginals(drafter_logits[c0:c1], self.K, t.logq[c0:c1], t.logit[c0:c1],
                                       t.tok[c0:c1], t.lse[c0:c1], self.ws_topk, self.status[c0:c1], st)
                prev = torch.cuda.Event()
                prev.record(st)
                cost = self.cost_ms[c0:c1] if per_req_cost else self.cost_ms
                bastion_build_tree(t.logit[c0:c1], t.tok[c0:c1], t.lse[c0:c1], self.n_max,
                                   self.root_token[c0:c1], self.ctx_len[c0:c1], cost, self.l_ar[c0:c1],
                                   tr.n_nodes[c0:c1], tr.parent[c0:c1], tr.depth[c0:c1], tr.pos_id[c0:c1],
                                   tr.token[c0:c1], tr.rank[c0:c1], tr.log_rho[c0:c1], tr.a_hat[c0:c1],
                                   tr.speedup[c0:c1], tr.anc_mask[c0:c1], self.status[c0:c1], st)
                bastion_verify_greedy(target_logits[c0:c1], self.b, tr.n_nodes[c0:c1], tr.parent[c0:c1],
                                      tr.token[c0:c1], v.argmax[c0:c1], v.accept_len[c0:c1],
                                      v.accept_nodes[c0:c1], v.out_tokens[c0:c1], ws_v,
                                      self.status[c0:c1], st)
        for c in range(chunks):
            main.wait_stream(self._chunk_state[c][0])

    def capture(self, drafter_logits, target_logits, chunks=1):
        """Records one step in a CUDA graph (chunks > 1: run_chunked)."""
        def step():
            if chunks > 1:
                self.run_chunked(drafter_logits, target_logits, chunks)
            else:
                self.run(drafter_logits, target_logits)
        s = torch.cuda.Stream(device=self.device)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()  # warm (sets kernel attributes, creates the chunk streams)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize(self.device)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        self.graph = g
        return g


class PagedCache:
    """The paged key-value cache of one target layer for B requests, over preallocated device buffers (nothing
    is allocated after construction, so a step that uses it can be captured in a CUDA graph).

    page_table None: request r owns pages r * max_pages .. (r + 1) * max_pages - 1, i.e. the pools are a
    contiguous cache [B, max_pages * page_size, Hkv, D], which ``contiguous()`` gives to bastion_tree_attention.
    weights: keep the accumulated attention weight and the position of every slot, which evict() needs.
    After STATUS_TIMEOUT in status, zero ws_attend before the next attend()."""

    def __init__(self, B, Hq, Hkv, D, page_size, max_pages, device, dtype=torch.bfloat16, page_table=None,
                 n_pages=None, weights=False):
        self.B, self.Hq, self.Hkv, self.D, self.page_size, self.max_pages = B, Hq, Hkv, D, page_size, max_pages
        self.cap, self.device = max_pages * page_size, device
        self.identity = page_table is None
        if page_table is None:
            n_pages = B * max_pages
            page_table = torch.arange(n_pages, dtype=torch.int32).view(B, max_pages)
        elif n_pages is None:
            raise BastionError("paged cache: a page_table needs n_pages")
        self.page_table = page_table.to(device=device, dtype=torch.int32).contiguous()
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=device)  # noqa: E731
        self.k_pool = torch.zeros(n_pages, page_size, Hkv, D, dtype=dtype, device=device)
        self.v_pool = torch.zeros_like(self.k_pool)
        self.seq_len, self.n_seen, self.status = i32(B), i32(B), i32(B)
        self.acc = torch.zeros(B, Hkv, self.cap, device=device) if weights else None
        self.pos = i32(B, Hkv, self.cap) if weights else None
        self.ws_append = workspace(bastion_paged_append_workspace_bytes(B), device)
        self.ws_attend = workspace(bastion_paged_attention_workspace_bytes(B, Hq, Hkv, D, self.cap, weights), device)
        self.ws_evict = workspace(bastion_paged_evict_workspace_bytes(B, Hkv, self.cap), device) if weights else None

    def contiguous(self):
        """(k, v) [B, cap, Hkv, D]: the same memory as a contiguous cache."""
        if not self.identity:
            raise BastionError("paged cache: its pages are not in order")
        shape = (self.B, self.cap, self.Hkv, self.D)
        return self.k_pool.view(shape), self.v_pool.view(shape)

    def append(self, k_new, v_new, rows=None, n_new=None, stream=None):
        """The rows of k_new/v_new [B, n_rows, Hkv, D] (all, the first n_new, or those listed in rows) enter the
        next slots; rows = Verify.accept_nodes commits the accepted path of a verified tree."""
        bastion_paged_append(k_new, v_new, self.k_pool, self.v_pool, self.page_table, self.seq_len, self.seq_len,
                             self.ws_append, self.status, rows, n_new, self.acc, self.pos, self.n_seen, self.n_seen,
                             stream)

    def attend(self, q, scale, out, lse=None, stream=None):
        """out [B, Hq, D] = attention of q over the used slots; adds the weights to acc where they are kept."""
        bastion_paged_attention(q, self.k_pool, self.v_pool, self.page_table, self.seq_len, scale, out,
                                self.ws_attend, self.status, lse, self.acc, self.acc, stream)

    def evict(self, budget, n_sink=0, n_recent=0, stream=None):
        """Keeps budget slots per request and KV head."""
        if self.acc is None:
            raise BastionError("paged cache: evict needs weights=True")
        bastion_paged_evict(self.k_pool, self.v_pool, self.page_table, self.seq_len, self.n_seen, self.acc, self.pos,
                            budget, n_sink, n_recent, self.seq_len, self.acc, self.pos, self.ws_evict, self.status,
                            stream)

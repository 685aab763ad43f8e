"""GB300-native one-pass tree verification for EAGLE-style speculative decoding.

A thin ctypes binding over ``libspecverify.so``, whose C ABI is declared in
``include/specverify.h``. The functions here only check tensor shapes, dtypes,
devices and contiguity and pass raw device pointers and the current CUDA
stream; every step of the computation runs in the library's CUDA kernels.
There is no CPU path: calling with a tensor that is not on a CUDA device, or
without the built library, raises.

    anc, depth, status = tree_mask_build(parent)
    out, lse, status   = tree_verify_attn(q, k_cache, v_cache, page_table, seq_lens, anc)
    res                = spec_accept(target_logits, draft_logits, tokens, parent,
                                     u_accept, u_bonus)
"""

from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libspecverify.so")

SVF_F32, SVF_BF16 = 0, 1
SVF_OK, SVF_ERR_ARG, SVF_ERR_UNSUPPORTED, SVF_ERR_LAUNCH, SVF_ERR_WORKSPACE = 0, -1, -2, -3, -4
SVF_ERR_SCRATCH_LIMIT = -5
SVF_DEV_BAD_PARENT, SVF_DEV_BAD_TOKEN, SVF_DEV_BAD_PAGE, SVF_DEV_BAD_LENGTH, SVF_DEV_TIMEOUT = (
    1, 2, 4, 8, 16)
SVF_DEV_BAD_PATH, SVF_DEV_BAD_CLUSTER, SVF_DEV_NO_PAGES, SVF_DEV_BAD_ADAPTER = 32, 64, 128, 256
SVF_DEV_BAD_ROW = 512

EXPORTED = [
    "svf_tree_mask_build",
    "svf_tree_verify_attn_workspace_size",
    "svf_tree_verify_attn",
    "svf_tree_mask_attn",
    "svf_spec_accept_workspace_size",
    "svf_spec_accept",
    "svf_spec_accept_noalloc",
    "svf_lm_head",
    "svf_debug_set_attn_wait_ns",
    "svf_debug_set_attn_splits",
    "svf_debug_set_attn_kernel",
    "svf_debug_set_lora_wait_ns",
    "svf_debug_lora_plan",
    "svf_spec_accept_lmhead",
    "svf_kv_commit",
    "svf_selftest_wait_timeout",
    "svf_spec_accept_bf16",
    "svf_spec_accept_greedy",
    "svf_spec_accept_onehot",
    "svf_spec_accept_greedy_bf16",
    "svf_spec_accept_onehot_bf16",
    "svf_eagle2_init",
    "svf_eagle2_expand",
    "svf_eagle2_finalize",
    "svf_page_pool_init",
    "svf_page_reserve",
    "svf_page_release",
    "svf_page_fork",
    "svf_page_copy",
    "svf_page_release_shared",
    "svf_rope_kv_write",
    "svf_norm_rope_kv_write",
    "svf_chunk_attn_workspace_size",
    "svf_chunk_attn",
    "svf_debug_set_chunk_wait_ns",
    "svf_lora_proj_workspace_size",
    "svf_lora_proj",
    "svf_status_string",
    "svf_version",
]

_lib = None


class SpecVerifyError(RuntimeError):
    pass


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libspecverify.so and declare its signatures (no GPU needed)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise SpecVerifyError(
            f"{path} is missing: build it with speculative_decoding_tree_03_gb300.build.build()")
    lib = ctypes.CDLL(path)
    P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.svf_tree_mask_build.argtypes = [P, I, I, P, P, P, P]
    lib.svf_tree_mask_build.restype = I
    lib.svf_tree_verify_attn_workspace_size.argtypes = [I, I, I, I, I, I, I, I]
    lib.svf_tree_verify_attn_workspace_size.restype = Z
    lib.svf_tree_verify_attn.argtypes = [P, P, P, I, I, P, I, P, P, I, I, I, I, I, I, F, P, P, P,
                                         Z, P, P]
    lib.svf_tree_verify_attn.restype = I
    lib.svf_tree_mask_attn.argtypes = [P, P, P, P, P, P, P, I, I, P, I, P, I, I, I, I, I, I, F,
                                       P, P, P, Z, P, P]
    lib.svf_tree_mask_attn.restype = I
    lib.svf_spec_accept_workspace_size.argtypes = [I, I, I]
    lib.svf_spec_accept_workspace_size.restype = Z
    lib.svf_spec_accept.argtypes = [P, P, P, P, P, P, I, I, I, P, P, P, P, P, Z, P, P]
    lib.svf_spec_accept.restype = I
    lib.svf_spec_accept_noalloc.argtypes = [P, P, P, P, P, P, I, I, I, P, P, P, P, P, P]
    lib.svf_spec_accept_noalloc.restype = I
    lib.svf_spec_accept_bf16.argtypes = [P, P, P, P, P, P, I, I, I, P, P, P, P, P, P]
    lib.svf_spec_accept_bf16.restype = I
    lib.svf_spec_accept_greedy.argtypes = [P, P, P, I, I, I, P, P, P, P, P]
    lib.svf_spec_accept_greedy.restype = I
    lib.svf_spec_accept_onehot.argtypes = [P, P, P, P, P, I, I, I, P, P, P, P, P, P]
    lib.svf_spec_accept_onehot.restype = I
    lib.svf_spec_accept_greedy_bf16.argtypes = [P, P, P, I, I, I, P, P, P, P, P]
    lib.svf_spec_accept_greedy_bf16.restype = I
    lib.svf_spec_accept_onehot_bf16.argtypes = [P, P, P, P, P, I, I, I, P, P, P, P, P, P]
    lib.svf_spec_accept_onehot_bf16.restype = I
    lib.svf_eagle2_init.argtypes = [P, I, I, P, P, P, P, P, P]
    lib.svf_eagle2_init.restype = I
    lib.svf_eagle2_expand.argtypes = [P, I, I, I, I, P, I, P, P, P, P, P, P, P, P]
    lib.svf_eagle2_expand.restype = I
    lib.svf_eagle2_finalize.argtypes = [I, I, P, P, P, P, P, I, P, P, P, P, P, P]
    lib.svf_eagle2_finalize.restype = I
    lib.svf_selftest_wait_timeout.argtypes = [P, ctypes.c_longlong, P]
    lib.svf_selftest_wait_timeout.restype = I
    lib.svf_kv_commit.argtypes = [P, P, I, ctypes.c_longlong, I, I, P, I, P, P, P, I, I, I, I,
                                  I, P, P, I, P, P, P]
    lib.svf_kv_commit.restype = I
    lib.svf_lm_head.argtypes = [P, P, I, I, I, P, P, P]
    lib.svf_lm_head.restype = I
    lib.svf_spec_accept_lmhead.argtypes = [P, P, P, P, P, P, P, I, I, I, I, P, P, P, P, P, P, P,
                                           P]
    lib.svf_spec_accept_lmhead.restype = I
    lib.svf_debug_set_attn_wait_ns.argtypes = [ctypes.c_longlong]
    lib.svf_debug_set_attn_wait_ns.restype = I
    lib.svf_debug_set_attn_splits.argtypes = [I]
    lib.svf_debug_set_attn_splits.restype = I
    lib.svf_debug_set_attn_kernel.argtypes = [I]
    lib.svf_debug_set_attn_kernel.restype = I
    lib.svf_debug_set_lora_wait_ns.argtypes = [ctypes.c_longlong]
    lib.svf_debug_set_lora_wait_ns.restype = I
    lib.svf_debug_lora_plan.argtypes = [I, I, I, I, I, I, P]
    lib.svf_debug_lora_plan.restype = I
    L = ctypes.c_longlong
    lib.svf_page_pool_init.argtypes = [P, P, I, P]
    lib.svf_page_pool_init.restype = I
    lib.svf_page_reserve.argtypes = [P, I, I, P, P, I, P, P, I, I, P, P, P, P, P, P]
    lib.svf_page_reserve.restype = I
    lib.svf_page_release.argtypes = [P, I, I, P, P, I, P, P, I, P, P, P]
    lib.svf_page_release.restype = I
    lib.svf_rope_kv_write.argtypes = [P, P, P, L, L, L, I, I, I, I, I, P, I, I, I, P, P, P, P, P,
                                      I, P, P]
    lib.svf_rope_kv_write.restype = I
    lib.svf_page_fork.argtypes = [P, I, I, P, P, I, P, P, I, P, P, I, P, P, P, P, P]
    lib.svf_page_fork.restype = I
    lib.svf_page_copy.argtypes = [P, P, I, L, I, I, P, P, P, I, I, I, I, P, P]
    lib.svf_page_copy.restype = I
    lib.svf_page_release_shared.argtypes = [P, I, I, P, P, I, P, P, P, I, P, P, P]
    lib.svf_page_release_shared.restype = I
    lib.svf_norm_rope_kv_write.argtypes = [P, P, P, L, L, L, I, I, I, I, I, P, P, F, P, I, I, I, P,
                                           I, P, P, P, P, P, I, P, P]
    lib.svf_norm_rope_kv_write.restype = I
    lib.svf_chunk_attn_workspace_size.argtypes = [I, I, I, I, I, I]
    lib.svf_chunk_attn_workspace_size.restype = Z
    lib.svf_chunk_attn.argtypes = [P, P, P, I, I, P, I, P, P, I, I, I, I, I, I, F, P, P, P, Z, P, P]
    lib.svf_chunk_attn.restype = I
    lib.svf_debug_set_chunk_wait_ns.argtypes = [L]
    lib.svf_debug_set_chunk_wait_ns.restype = I
    lib.svf_lora_proj_workspace_size.argtypes = [I, I]
    lib.svf_lora_proj_workspace_size.restype = Z
    lib.svf_lora_proj.argtypes = [P, L, P, P, P, P, P, I, I, I, I, I, I, P, L, P, Z, P, P]
    lib.svf_lora_proj.restype = I
    lib.svf_status_string.argtypes = [I]
    lib.svf_status_string.restype = ctypes.c_char_p
    lib.svf_version.argtypes = []
    lib.svf_version.restype = I
    _lib = lib
    _load_fastcall(lib)
    return lib


_fast = None


def _load_fastcall(lib) -> None:
    """The compiled checks of the short calls, if they were built from these sources
    for this interpreter and torch."""
    global _fast
    import importlib.machinery
    import importlib.util

    from . import build as _build

    try:
        path = _build.fastcall_path()
        if not os.path.exists(path):
            return
        loader = importlib.machinery.ExtensionFileLoader("_fastcall", path)
        mod = importlib.util.module_from_spec(
            importlib.util.spec_from_loader("_fastcall", loader))
        loader.exec_module(mod)
    except (ImportError, OSError):
        return
    mod.bind(*(ctypes.cast(fn, ctypes.c_void_p).value for fn in
               (lib.svf_page_reserve, lib.svf_page_release, lib.svf_rope_kv_write,
                lib.svf_lora_proj, lib.svf_page_release_shared, lib.svf_page_fork,
                lib.svf_page_copy, lib.svf_norm_rope_kv_write, lib.svf_chunk_attn)))
    _fast = mod


def status_string(code: int) -> str:
    return load_library().svf_status_string(int(code)).decode()


def _check(rc: int, what: str) -> None:
    if rc != SVF_OK:
        raise SpecVerifyError(f"{what}: {status_string(rc)} ({rc})")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dev(t: torch.Tensor, name: str, dtype=None, shape=None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise SpecVerifyError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise SpecVerifyError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise SpecVerifyError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise SpecVerifyError(f"{name} must be contiguous")
    return t


_ZEROED_WS = {}


def _zeroed_workspace(need: int, dev: torch.device, stream=None, of="tree") -> torch.Tensor:
    """The attention workspace used when the caller passes none: zero-filled
    once, on the stream of the call that makes it, and kept per device and
    operator (every call leaves zero what has to be); the chunk attention's per
    stream too, so that its calls on two streams never meet in one. Tree calls that may
    overlap on the GPU should pass workspaces of their own. A captured call gets
    one of the graph's memory, filled in every replay: the kept one goes when a
    larger shape comes, and one made in a capture would begin at zero only in
    the replays."""
    with _on(stream, dev):
        if torch.cuda.is_current_stream_capturing():
            return torch.zeros((need,), dtype=torch.uint8, device=dev)
        key = (dev.type, dev.index if dev.index is not None else torch.cuda.current_device(), of)
        if of == "chunk":
            key += (torch.cuda.current_stream(dev).cuda_stream,)
        ws = _ZEROED_WS.get(key)
        if ws is None or ws.numel() < need:
            ws = torch.zeros((need,), dtype=torch.uint8, device=dev)
            _ZEROED_WS[key] = ws
        return ws


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float32:
        return SVF_F32
    if dt == torch.bfloat16:
        return SVF_BF16
    raise SpecVerifyError(f"unsupported dtype {dt}")


# ---------------------------------------------------------------------------
# tree_mask_build
# ---------------------------------------------------------------------------

def tree_mask_build(parent: torch.Tensor, anc: Optional[torch.Tensor] = None,
                    depth: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                    stream=None):
    """Ancestor bitmasks of BFS-flattened trees: parent [B, N] int32 ->
    (anc [B, N, ceil(N/64)] int64 bit patterns, depth [B, N] int32, status [B] int32)."""
    lib = load_library()
    _dev(parent, "parent", torch.int32)
    B, N = parent.shape
    W = max(1, (N + 63) // 64)
    dev = parent.device
    if anc is None:
        anc = torch.empty((B, N, W), dtype=torch.int64, device=dev)
    if depth is None:
        depth = torch.empty((B, N), dtype=torch.int32, device=dev)
    if status is None:
        status = torch.empty((B,), dtype=torch.int32, device=dev)
    _dev(anc, "anc", torch.int64, (B, N, W))
    _dev(depth, "depth", torch.int32, (B, N))
    _dev(status, "status", torch.int32, (B,))
    rc = lib.svf_tree_mask_build(_ptr(parent), B, N, _ptr(anc), _ptr(depth), _ptr(status),
                                 _stream(stream))
    _check(rc, "svf_tree_mask_build")
    return anc, depth, status


# ---------------------------------------------------------------------------
# tree_verify_attn
# ---------------------------------------------------------------------------

def tree_verify_attn_workspace_size(B, N, Hq, Hkv, D, dtype, max_pages, page_size) -> int:
    return int(load_library().svf_tree_verify_attn_workspace_size(
        B, N, Hq, Hkv, D, _dtype_code(dtype) if isinstance(dtype, torch.dtype) else int(dtype),
        max_pages, page_size))


def tree_verify_attn(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                     page_table: torch.Tensor, seq_lens: torch.Tensor, anc: torch.Tensor,
                     sm_scale: float = 0.0, out: Optional[torch.Tensor] = None,
                     lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                     status: Optional[torch.Tensor] = None, want_lse: bool = True, stream=None):
    """Tree attention against a paged KV cache.

    q [B, N, Hq, D]; k_cache, v_cache [num_pages, page_size, Hkv, D] (same dtype,
    float32 or bfloat16); page_table [B, max_pages] int32; seq_lens [B] int32
    (prefix length, tree excluded); anc [B, N, 1] int64 from tree_mask_build.
    Returns (out [B, N, Hq, D], lse [B, N, Hq] float32 or None, status [B] int32).
    """
    lib = load_library()
    _dev(q, "q")
    B, N, Hq, D = q.shape
    dt = q.dtype
    _dev(k_cache, "k_cache", dt)
    num_pages, page_size, Hkv, Dk = k_cache.shape
    if Dk != D:
        raise SpecVerifyError("k_cache head_dim differs from q")
    _dev(v_cache, "v_cache", dt, k_cache.shape)
    _dev(page_table, "page_table", torch.int32)
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise SpecVerifyError("page_table must be [B, max_pages]")
    max_pages = page_table.shape[1]
    _dev(seq_lens, "seq_lens", torch.int32, (B,))
    _dev(anc, "anc", torch.int64)
    if anc.shape[0] != B or anc.shape[1] != N:
        raise SpecVerifyError("anc must be [B, N, W]")
    dev = q.device
    if out is None:
        out = torch.empty_like(q)
    _dev(out, "out", dt, q.shape)
    if lse is None and want_lse:
        lse = torch.empty((B, N, Hq), dtype=torch.float32, device=dev)
    if lse is not None:
        _dev(lse, "lse", torch.float32, (B, N, Hq))
    if status is None:
        status = torch.empty((B,), dtype=torch.int32, device=dev)
    _dev(status, "status", torch.int32, (B,))
    code = _dtype_code(dt)
    need = int(lib.svf_tree_verify_attn_workspace_size(B, N, Hq, Hkv, D, code, max_pages,
                                                       page_size))
    if workspace is None and need > 0:
        workspace = _zeroed_workspace(need, dev, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.svf_tree_verify_attn(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), num_pages, page_size, _ptr(page_table), max_pages,
        _ptr(seq_lens), _ptr(anc), B, N, Hq, Hkv, D, code, float(sm_scale), _ptr(out), _ptr(lse),
        _ptr(workspace), ws_bytes, _ptr(status), _stream(stream))
    _check(rc, "svf_tree_verify_attn")
    return out, lse, status


def tree_mask_attn(parent: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                   v_cache: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
                   sm_scale: float = 0.0, anc: Optional[torch.Tensor] = None,
                   depth: Optional[torch.Tensor] = None,
                   mask_status: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None, want_lse: bool = True, stream=None):
    """tree_mask_build and tree_verify_attn in one call (one kernel for
    bfloat16). Returns (out, lse, status, anc, depth, mask_status)."""
    lib = load_library()
    _dev(q, "q")
    B, N, Hq, D = q.shape
    dt = q.dtype
    _dev(parent, "parent", torch.int32, (B, N))
    _dev(k_cache, "k_cache", dt)
    num_pages, page_size, Hkv, Dk = k_cache.shape
    if Dk != D:
        raise SpecVerifyError("k_cache head_dim differs from q")
    _dev(v_cache, "v_cache", dt, k_cache.shape)
    _dev(page_table, "page_table", torch.int32)
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise SpecVerifyError("page_table must be [B, max_pages]")
    max_pages = page_table.shape[1]
    _dev(seq_lens, "seq_lens", torch.int32, (B,))
    dev = q.device
    if anc is None:
        anc = torch.empty((B, N, 1), dtype=torch.int64, device=dev)
    _dev(anc, "anc", torch.int64, (B, N, 1))
    if depth is None:
        depth = torch.empty((B, N), dtype=torch.int32, device=dev)
    _dev(depth, "depth", torch.int32, (B, N))
    if mask_status is None:
        mask_status = torch.empty((B,), dtype=torch.int32, device=dev)
    _dev(mask_status, "mask_status", torch.int32, (B,))
    if out is None:
        out = torch.empty_like(q)
    _dev(out, "out", dt, q.shape)
    if lse is None and want_lse:
        lse = torch.empty((B, N, Hq), dtype=torch.float32, device=dev)
    if lse is not None:
        _dev(lse, "lse", torch.float32, (B, N, Hq))
    if status is None:
        status = torch.empty((B,), dtype=torch.int32, device=dev)
    _dev(status, "status", torch.int32, (B,))
    code = _dtype_code(dt)
    need = int(lib.svf_tree_verify_attn_workspace_size(B, N, Hq, Hkv, D, code, max_pages,
                                                       page_size))
    if workspace is None and need > 0:
        workspace = _zeroed_workspace(need, dev, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.svf_tree_mask_attn(
        _ptr(parent), _ptr(anc), _ptr(depth), _ptr(mask_status), _ptr(q), _ptr(k_cache),
        _ptr(v_cache), num_pages, page_size, _ptr(page_table), max_pages, _ptr(seq_lens), B, N,
        Hq, Hkv, D, code, float(sm_scale), _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes,
        _ptr(status), _stream(stream))
    _check(rc, "svf_tree_mask_attn")
    return out, lse, status, anc, depth, mask_status


# ---------------------------------------------------------------------------
# spec_accept
# ---------------------------------------------------------------------------

def spec_accept_workspace_size(B, N, V) -> int:
    return int(load_library().svf_spec_accept_workspace_size(B, N, V))


def spec_accept(target_logits: torch.Tensor, draft_logits: torch.Tensor, tokens: torch.Tensor,
                parent: torch.Tensor, u_accept: torch.Tensor, u_bonus: torch.Tensor,
                want_ratio: bool = True, workspace: Optional[torch.Tensor] = None,
                outputs: Optional[dict] = None, stream=None) -> dict:
    """Acceptance walk. Returns a dict of device tensors: accept_len [B], path [B, N],
    out_tokens [B, N], ratio [B, N] (or None), status [B]. Logits are float32 or
    bfloat16 (both the same dtype)."""
    lib = load_library()
    _dev(target_logits, "target_logits")
    if target_logits.dtype not in (torch.float32, torch.bfloat16):
        raise SpecVerifyError("logits must be float32 or bfloat16")
    B, N, V = target_logits.shape
    _dev(draft_logits, "draft_logits", target_logits.dtype, (B, N, V))
    _dev(tokens, "tokens", torch.int32, (B, N))
    _dev(parent, "parent", torch.int32, (B, N))
    _dev(u_accept, "u_accept", torch.float32, (B, N))
    _dev(u_bonus, "u_bonus", torch.float32, (B,))
    dev = target_logits.device
    o = outputs if outputs is not None else {}
    if "accept_len" not in o:
        o["accept_len"] = torch.empty((B,), dtype=torch.int32, device=dev)
        o["path"] = torch.empty((B, N), dtype=torch.int32, device=dev)
        o["out_tokens"] = torch.empty((B, N), dtype=torch.int32, device=dev)
        o["ratio"] = torch.empty((B, N), dtype=torch.float32, device=dev) if want_ratio else None
        o["status"] = torch.empty((B,), dtype=torch.int32, device=dev)
    if target_logits.dtype == torch.bfloat16:
        rc = lib.svf_spec_accept_bf16(
            _ptr(target_logits), _ptr(draft_logits), _ptr(tokens), _ptr(parent), _ptr(u_accept),
            _ptr(u_bonus), B, N, V, _ptr(o["accept_len"]), _ptr(o["path"]),
            _ptr(o["out_tokens"]), _ptr(o.get("ratio")), _ptr(o["status"]), _stream(stream))
        _check(rc, "svf_spec_accept_bf16")
        return o
    need = int(lib.svf_spec_accept_workspace_size(B, N, V))
    if workspace is None:
        workspace = torch.empty((max(need, 1),), dtype=torch.uint8, device=dev)
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = lib.svf_spec_accept(
        _ptr(target_logits), _ptr(draft_logits), _ptr(tokens), _ptr(parent), _ptr(u_accept),
        _ptr(u_bonus), B, N, V, _ptr(o["accept_len"]), _ptr(o["path"]), _ptr(o["out_tokens"]),
        _ptr(o.get("ratio")), _ptr(workspace), ws_bytes, _ptr(o["status"]), _stream(stream))
    _check(rc, "svf_spec_accept")
    return o


def _variant_outputs(o, B, N, dev, want_ratio):
    if "accept_len" not in o:
        o["accept_len"] = torch.empty((B,), dtype=torch.int32, device=dev)
        o["path"] = torch.empty((B, N), dtype=torch.int32, device=dev)
        o["out_tokens"] = torch.empty((B, N), dtype=torch.int32, device=dev)
        o["ratio"] = torch.empty((B, N), dtype=torch.float32, device=dev) if want_ratio else None
        o["status"] = torch.empty((B,), dtype=torch.int32, device=dev)
    return o


def spec_accept_greedy(target_logits: torch.Tensor, tokens: torch.Tensor, parent: torch.Tensor,
                       outputs: Optional[dict] = None, stream=None) -> dict:
    """Temperature-0 acceptance (argmax matching) on float32 or bfloat16
    logits. Returns a dict of device tensors: accept_len [B], path [B, N],
    out_tokens [B, N], status [B]."""
    lib = load_library()
    if target_logits.dtype not in (torch.float32, torch.bfloat16):
        raise SpecVerifyError("target_logits must be float32 or bfloat16")
    _dev(target_logits, "target_logits")
    bf = target_logits.dtype == torch.bfloat16
    B, N, V = target_logits.shape
    _dev(tokens, "tokens", torch.int32, (B, N))
    _dev(parent, "parent", torch.int32, (B, N))
    o = _variant_outputs(outputs if outputs is not None else {}, B, N, target_logits.device,
                         False)
    fn = lib.svf_spec_accept_greedy_bf16 if bf else lib.svf_spec_accept_greedy
    rc = fn(_ptr(target_logits), _ptr(tokens), _ptr(parent), B, N, V, _ptr(o["accept_len"]),
            _ptr(o["path"]), _ptr(o["out_tokens"]), _ptr(o["status"]), _stream(stream))
    _check(rc, "svf_spec_accept_greedy" + ("_bf16" if bf else ""))
    return o


def spec_accept_onehot(target_logits: torch.Tensor, tokens: torch.Tensor, parent: torch.Tensor,
                       u_accept: torch.Tensor, u_bonus: torch.Tensor, want_ratio: bool = True,
                       outputs: Optional[dict] = None, stream=None) -> dict:
    """The sampling rule with q = one-hot(candidate) for every child, on
    float32 or bfloat16 logits. Returns accept_len, path, out_tokens, ratio
    (or None) and status."""
    lib = load_library()
    if target_logits.dtype not in (torch.float32, torch.bfloat16):
        raise SpecVerifyError("target_logits must be float32 or bfloat16")
    _dev(target_logits, "target_logits")
    bf = target_logits.dtype == torch.bfloat16
    B, N, V = target_logits.shape
    _dev(tokens, "tokens", torch.int32, (B, N))
    _dev(parent, "parent", torch.int32, (B, N))
    _dev(u_accept, "u_accept", torch.float32, (B, N))
    _dev(u_bonus, "u_bonus", torch.float32, (B,))
    o = _variant_outputs(outputs if outputs is not None else {}, B, N, target_logits.device,
                         want_ratio)
    fn = lib.svf_spec_accept_onehot_bf16 if bf else lib.svf_spec_accept_onehot
    rc = fn(_ptr(target_logits), _ptr(tokens), _ptr(parent), _ptr(u_accept), _ptr(u_bonus), B,
            N, V, _ptr(o["accept_len"]), _ptr(o["path"]), _ptr(o["out_tokens"]),
            _ptr(o.get("ratio")), _ptr(o["status"]), _stream(stream))
    _check(rc, "svf_spec_accept_onehot" + ("_bf16" if bf else ""))
    return o


# ---------------------------------------------------------------------------
# LM head (target logits from hidden states) and the walk fed by it
# ---------------------------------------------------------------------------

def lm_head(hidden: torch.Tensor, weight: torch.Tensor, logits: Optional[torch.Tensor] = None,
            status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """logits[..., v] = hidden[..., :] . weight[v, :] for bf16 hidden [..., H]
    and weight [V, H], as fp32 [..., V]."""
    lib = load_library()
    _dev(hidden, "hidden", torch.bfloat16)
    H = hidden.shape[-1]
    _dev(weight, "weight", torch.bfloat16)
    if weight.dim() != 2 or weight.shape[1] != H:
        raise SpecVerifyError("weight must be [V, H] with H = hidden.shape[-1]")
    V = weight.shape[0]
    R = hidden.numel() // H if H > 0 else 0
    shape = tuple(hidden.shape[:-1]) + (V,)
    if logits is None:
        logits = torch.empty(shape, dtype=torch.float32, device=hidden.device)
    _dev(logits, "logits", torch.float32, shape)
    if status is not None:
        _dev(status, "status", torch.int32)
    rc = lib.svf_lm_head(_ptr(hidden), _ptr(weight), R, H, V, _ptr(logits), _ptr(status),
                         _stream(stream))
    _check(rc, "svf_lm_head")
    return logits


def spec_accept_lmhead(hidden: torch.Tensor, weight: torch.Tensor, draft_logits: torch.Tensor,
                       tokens: torch.Tensor, parent: torch.Tensor, u_accept: torch.Tensor,
                       u_bonus: torch.Tensor, want_ratio: bool = True,
                       outputs: Optional[dict] = None, stream=None) -> dict:
    """The acceptance walk with target rows from the LM head: hidden [B, N, H]
    bf16, weight [V, H] bf16, draft logits [B, N, V] fp32. Returns
    spec_accept's outputs plus "target_logits" [B, N, V] fp32 and
    "lm_status" [1]."""
    lib = load_library()
    _dev(hidden, "hidden", torch.bfloat16)
    B, N, H = hidden.shape
    _dev(weight, "weight", torch.bfloat16)
    V = weight.shape[0]
    if weight.dim() != 2 or weight.shape[1] != H:
        raise SpecVerifyError("weight must be [V, H] with H = hidden.shape[-1]")
    _dev(draft_logits, "draft_logits", torch.float32, (B, N, V))
    _dev(tokens, "tokens", torch.int32, (B, N))
    _dev(parent, "parent", torch.int32, (B, N))
    _dev(u_accept, "u_accept", torch.float32, (B, N))
    _dev(u_bonus, "u_bonus", torch.float32, (B,))
    dev = hidden.device
    o = outputs if outputs is not None else {}
    if "accept_len" not in o:
        o["accept_len"] = torch.empty((B,), dtype=torch.int32, device=dev)
        o["path"] = torch.empty((B, N), dtype=torch.int32, device=dev)
        o["out_tokens"] = torch.empty((B, N), dtype=torch.int32, device=dev)
        o["ratio"] = torch.empty((B, N), dtype=torch.float32, device=dev) if want_ratio else None
        o["status"] = torch.empty((B,), dtype=torch.int32, device=dev)
        o["target_logits"] = torch.empty((B, N, V), dtype=torch.float32, device=dev)
        o["lm_status"] = torch.zeros((1,), dtype=torch.int32, device=dev)
    rc = lib.svf_spec_accept_lmhead(
        _ptr(hidden), _ptr(weight), _ptr(draft_logits), _ptr(tokens), _ptr(parent),
        _ptr(u_accept), _ptr(u_bonus), B, N, H, V, _ptr(o["target_logits"]),
        _ptr(o["accept_len"]), _ptr(o["path"]), _ptr(o["out_tokens"]), _ptr(o.get("ratio")),
        _ptr(o["lm_status"]), _ptr(o["status"]), _stream(stream))
    _check(rc, "svf_spec_accept_lmhead")
    return o


# ---------------------------------------------------------------------------
# EAGLE-2 tree construction
# ---------------------------------------------------------------------------

def eagle2_init(pool: dict, root_tokens: torch.Tensor, stream=None) -> dict:
    """Reset ``pool`` to the roots alone (a new build in the same arrays)."""
    lib = load_library()
    _dev(root_tokens, "root_tokens", torch.int32)
    B, C = pool["parent"].shape
    if root_tokens.shape != (B,):
        raise SpecVerifyError("root_tokens must be [B]")
    rc = lib.svf_eagle2_init(_ptr(root_tokens), B, C, _ptr(pool["parent"]),
                             _ptr(pool["depth"]), _ptr(pool["token"]), _ptr(pool["value"]),
                             _ptr(pool["count"]), _stream(stream))
    _check(rc, "svf_eagle2_init")
    return pool


def eagle2_pool(root_tokens: torch.Tensor, capacity: int, stream=None) -> dict:
    """A node pool per sequence holding only the root (device tensors)."""
    _dev(root_tokens, "root_tokens", torch.int32)
    B = root_tokens.shape[0]
    dev = root_tokens.device
    pool = {"parent": torch.empty((B, capacity), dtype=torch.int32, device=dev),
            "depth": torch.empty((B, capacity), dtype=torch.int32, device=dev),
            "token": torch.empty((B, capacity), dtype=torch.int32, device=dev),
            "value": torch.empty((B, capacity), dtype=torch.float64, device=dev),
            "count": torch.empty((B,), dtype=torch.int32, device=dev)}
    return eagle2_init(pool, root_tokens, stream)


def eagle2_expand(pool: dict, draft_rows: torch.Tensor, frontier: torch.Tensor, k: int,
                  next_frontier: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One expansion round in place; returns the next frontier [B, k].
    ``status`` [B] int32, when given, gets 0 or SVF_DEV_TIMEOUT per sequence."""
    lib = load_library()
    _dev(draft_rows, "draft_rows", torch.float32)
    B, R, V = draft_rows.shape
    _dev(frontier, "frontier", torch.int32, (B, R))
    C = pool["parent"].shape[1]
    if next_frontier is None:
        next_frontier = torch.empty((B, k), dtype=torch.int32, device=draft_rows.device)
    if status is not None:
        _dev(status, "status", torch.int32, (B,))
    rc = lib.svf_eagle2_expand(_ptr(draft_rows), B, R, V, k, _ptr(frontier), C,
                               _ptr(pool["parent"]), _ptr(pool["depth"]), _ptr(pool["token"]),
                               _ptr(pool["value"]), _ptr(pool["count"]), _ptr(next_frontier),
                               None if status is None else _ptr(status), _stream(stream))
    _check(rc, "svf_eagle2_expand")
    return next_frontier


def eagle2_finalize(pool: dict, n_nodes: int, outputs: Optional[dict] = None,
                    stream=None) -> dict:
    """Rerank and flatten: parent [B, n], tokens, values, cids, n_out."""
    lib = load_library()
    B, C = pool["parent"].shape
    dev = pool["parent"].device
    out = outputs if outputs is not None else {}
    if "parent" not in out:
        out.update({"parent": torch.empty((B, n_nodes), dtype=torch.int32, device=dev),
                    "tokens": torch.empty((B, n_nodes), dtype=torch.int32, device=dev),
                    "values": torch.empty((B, n_nodes), dtype=torch.float64, device=dev),
                    "cids": torch.empty((B, n_nodes), dtype=torch.int32, device=dev),
                    "n_out": torch.empty((B,), dtype=torch.int32, device=dev)})
    rc = lib.svf_eagle2_finalize(B, C, _ptr(pool["parent"]), _ptr(pool["depth"]),
                                 _ptr(pool["token"]), _ptr(pool["value"]), _ptr(pool["count"]),
                                 n_nodes, _ptr(out["parent"]), _ptr(out["tokens"]),
                                 _ptr(out["values"]), _ptr(out["cids"]), _ptr(out["n_out"]),
                                 _stream(stream))
    _check(rc, "svf_eagle2_finalize")
    return out


def selftest_wait_timeout(deadline_s: float = 0.02, device="cuda", stream=None) -> dict:
    """Run the bounded-wait diagnostic; returns the statuses and elapsed
    times (seconds) of a CTA wait and a cluster wait that nothing completes."""
    lib = load_library()
    res = torch.zeros((4,), dtype=torch.int32, device=device)
    rc = lib.svf_selftest_wait_timeout(_ptr(res), int(deadline_s * 1e9), _stream(stream))
    _check(rc, "svf_selftest_wait_timeout")
    r = res.cpu().tolist()
    return {"cta_status": r[0], "cta_elapsed_s": r[1] * 1e-6,
            "cluster_status": r[2], "cluster_elapsed_s": r[3] * 1e-6}


# ---------------------------------------------------------------------------
# kv_commit
# ---------------------------------------------------------------------------

def kv_commit(k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
              seq_lens: torch.Tensor, path: torch.Tensor, accept_len: torch.Tensor,
              max_free: Optional[int] = None, outputs: Optional[dict] = None,
              stream=None) -> dict:
    """Keep the accepted path's K/V in place, in path order after the prefix.

    k_cache, v_cache [layers, num_pages, page_size, Hkv, D] (or without the
    layer axis), float32 or bfloat16, each layer contiguous; page_table
    [B, max_pages], seq_lens [B], path [B, N], accept_len [B] int32. Returns a
    dict of device tensors: new_seq_lens [B], freed [B, max_free] (page ids, -1
    padded), n_freed [B], status [B]."""
    lib = load_library()
    _dev(k_cache, "k_cache")
    if k_cache.dim() == 4:
        layers, (num_pages, page_size, Hkv, D) = 1, k_cache.shape
        stride = 0
    elif k_cache.dim() == 5:
        layers, num_pages, page_size, Hkv, D = k_cache.shape
        stride = k_cache.stride(0)
    else:
        raise SpecVerifyError("k_cache must be [layers,] num_pages, page_size, Hkv, D")
    if not (k_cache[0] if k_cache.dim() == 5 else k_cache).is_contiguous():
        raise SpecVerifyError("each layer of k_cache must be contiguous")
    _dev(v_cache, "v_cache", k_cache.dtype, k_cache.shape)
    if v_cache.stride() != k_cache.stride():
        raise SpecVerifyError("v_cache must have k_cache's strides")
    _dev(page_table, "page_table", torch.int32)
    B, max_pages = page_table.shape
    _dev(seq_lens, "seq_lens", torch.int32, (B,))
    _dev(path, "path", torch.int32)
    if path.dim() != 2 or path.shape[0] != B:
        raise SpecVerifyError("path must be [B, N]")
    N = path.shape[1]
    _dev(accept_len, "accept_len", torch.int32, (B,))
    if max_free is None:
        max_free = (N + page_size - 1) // page_size
    dev = k_cache.device
    o = outputs if outputs is not None else {}
    if "status" not in o:
        o["new_seq_lens"] = torch.empty((B,), dtype=torch.int32, device=dev)
        o["freed"] = torch.empty((B, max(max_free, 1)), dtype=torch.int32, device=dev)
        o["n_freed"] = torch.empty((B,), dtype=torch.int32, device=dev)
        o["status"] = torch.empty((B,), dtype=torch.int32, device=dev)
    rc = lib.svf_kv_commit(
        _ptr(k_cache), _ptr(v_cache), layers, stride, num_pages, page_size, _ptr(page_table),
        max_pages, _ptr(seq_lens), _ptr(path), _ptr(accept_len), B, N, Hkv, D,
        _dtype_code(k_cache.dtype), _ptr(o["new_seq_lens"]), _ptr(o["freed"]), max_free,
        _ptr(o["n_freed"]), _ptr(o["status"]), _stream(stream))
    _check(rc, "svf_kv_commit")
    return o


# ---------------------------------------------------------------------------
# The operators around the verify pass: pages, rotary K/V write, projections
# with per-request adapters. Their calls are short: the compiled checks
# (fastcall.cpp) take a call that is all in order; the checks here take any
# other, a call's tensors in one expression, and where that is false each by
# itself for the message.
# ---------------------------------------------------------------------------

def _device_of(t, name: str) -> int:
    dev = t.get_device() if isinstance(t, torch.Tensor) else -1
    if dev < 0:
        raise SpecVerifyError(f"{name} must be a CUDA tensor")
    return dev


def _bad(t, name: str, dtype, shape, dev: int):
    if isinstance(t, torch.Tensor) and t.get_device() >= 0 and t.get_device() != dev:
        raise SpecVerifyError(f"{name} must be on cuda:{dev}, got {t.device}")
    _dev(t, name, dtype, shape)
    raise SpecVerifyError(f"{name} is not a usable tensor")


def _p(t, name: str, dtype, shape, dev: int) -> int:
    """The address of a contiguous tensor of this dtype, shape and device."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == dev and t.is_contiguous()):
        return t.data_ptr()
    _bad(t, name, dtype, shape, dev)


def _current_stream(dev: int) -> int:
    """The handle of the device's current stream (the stream object that the
    public call makes costs a microsecond)."""
    return torch.cuda.current_stream(dev).cuda_stream


_current_device = torch.cuda.current_device
if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    _current_stream = torch._C._cuda_getCurrentRawStream


def _call(fn, what: str, dev: int, stream, *args) -> None:
    """fn(*args, stream) with ``dev`` current; the default stream is the
    current one of that device."""
    if dev != _current_device():
        with torch.cuda.device(dev):
            return _call(fn, what, dev, stream, *args)
    for v, c in zip(args, fn.argtypes):  # ctypes would cut them to 32 bits
        if c is ctypes.c_int and not -(1 << 31) <= v < 1 << 31:
            raise SpecVerifyError(f"{what}: {v} does not fit into 32 bits")
    rc = fn(*args, _current_stream(dev) if stream is None else stream.cuda_stream)
    if rc != SVF_OK:
        _check(rc, what)


def _on(stream, device):
    """Where a call allocates for itself: memory of the stream that it runs on,
    so that nothing on the current one uses it before or after the call."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
    return torch.cuda.stream(stream)


def _outs(o: dict, dtype, like: torch.Tensor, dev: int, stream, **shapes) -> None:
    """Allocate the outputs that ``o`` lacks, check the ones that it has."""
    for key, shape in shapes.items():
        if o.get(key) is None:
            with _on(stream, like.device):
                o[key] = torch.empty(shape, dtype=dtype, device=like.device)
        else:
            _p(o[key], key, dtype, shape, dev)


def page_pool(num_pages: int, device="cuda", stream=None, shared: bool = False) -> dict:
    """A pool of ``num_pages`` pages, all free: ``free`` [num_pages] int32 (a
    stack of page ids) and ``state`` [4] int32 (state[0] free pages). With
    ``shared`` also ``shares`` [num_pages] int32, how many sequences besides one
    hold a page, for page_fork; page_release then goes by it."""
    if num_pages < 1:
        raise SpecVerifyError("num_pages must be at least 1")
    with _on(stream, device):
        pool = {"free": torch.empty((num_pages,), dtype=torch.int32, device=device),
                "state": torch.empty((4,), dtype=torch.int32, device=device)}
        if shared:
            pool["shares"] = torch.zeros((num_pages,), dtype=torch.int32, device=device)
    free, state = pool["free"], pool["state"]
    _call(load_library().svf_page_pool_init, "svf_page_pool_init", _device_of(free, "device"),
          stream, free.data_ptr(), state.data_ptr(), num_pages)
    return pool


def _page_args(pool: dict, page_table, lens_a, name_a: str, lens_b, name_b: str):
    """Check what the two calls on a pool and a table share; (dev, B, max_pages)."""
    dev = _device_of(page_table, "page_table")
    if page_table.dim() != 2:
        raise SpecVerifyError("page_table must be [B, max_pages]")
    B, max_pages = page_table.shape
    free, state, i32, row = pool["free"], pool["state"], torch.int32, (B,)
    try:
        fine = (page_table.dtype is i32 and page_table.is_contiguous()
                and free.dtype is i32 and free.get_device() == dev and free.dim() == 1
                and free.is_contiguous()
                and state.dtype is i32 and state.get_device() == dev and state.shape == (4,)
                and state.is_contiguous()
                and lens_a.dtype is i32 and lens_a.get_device() == dev and lens_a.shape == row
                and lens_a.is_contiguous()
                and lens_b.dtype is i32 and lens_b.get_device() == dev and lens_b.shape == row
                and lens_b.is_contiguous())
    except AttributeError:
        fine = False
    if not fine:
        _p(page_table, "page_table", i32, (B, max_pages), dev)
        _p(free, "pool['free']", i32, (free.numel(),), dev)
        _p(state, "pool['state']", i32, (4,), dev)
        _p(lens_a, name_a, i32, row, dev)
        _p(lens_b, name_b, i32, row, dev)
    return dev, B, max_pages


def page_reserve(pool: dict, page_table: torch.Tensor, seq_lens: torch.Tensor,
                 new_lens: torch.Tensor, page_size: int, rows: int,
                 depth: Optional[torch.Tensor] = None, outputs: Optional[dict] = None,
                 stream=None) -> dict:
    """Pages and slots for ``new_lens`` [B] more tokens of sequences of
    ``seq_lens`` [B] tokens (int32), in place in ``page_table`` [B, max_pages]
    int32 and the pool. ``rows`` is the capacity of the row arrays: sequence
    b's new tokens are rows row_offsets[b] .. row_offsets[b + 1]. ``depth``
    (int32, ``rows`` values in any shape, e.g. tree_mask_build's) makes a
    row's position seq_lens + depth instead of seq_lens + i. Returns device
    tensors slots [rows], positions [rows], row_offsets [B + 1], status [B]."""
    lib = _lib or load_library()
    if _fast is not None and outputs is not None:
        rc = _fast.page_reserve(pool, page_table, seq_lens, new_lens, page_size, rows, depth,
                                outputs, stream)
        if rc is not None:
            _check(rc, "svf_page_reserve")
            return outputs
    dev, B, max_pages = _page_args(pool, page_table, seq_lens, "seq_lens", new_lens, "new_lens")
    free, i32 = pool["free"], torch.int32
    o = outputs if outputs is not None else {}
    try:
        slots, positions, offsets, status = (o["slots"], o["positions"], o["row_offsets"],
                                             o["status"])
        fine = (slots.dtype is i32 and slots.get_device() == dev and slots.shape == (rows,)
                and slots.is_contiguous()
                and positions.dtype is i32 and positions.get_device() == dev
                and positions.shape == (rows,) and positions.is_contiguous()
                and offsets.dtype is i32 and offsets.get_device() == dev
                and offsets.shape == (B + 1,) and offsets.is_contiguous()
                and status.dtype is i32 and status.get_device() == dev
                and status.shape == (B,) and status.is_contiguous())
    except (KeyError, AttributeError):
        fine = False
    if not fine:
        if rows < 0:
            raise SpecVerifyError("rows must not be negative")
        _outs(o, i32, page_table, dev, stream, slots=(rows,), positions=(rows,),
              row_offsets=(B + 1,), status=(B,))
        slots, positions, offsets, status = (o["slots"], o["positions"], o["row_offsets"],
                                             o["status"])
    d = None
    if depth is not None:
        if depth.numel() != rows:
            raise SpecVerifyError("depth must hold one value per row")
        d = _p(depth, "depth", i32, depth.shape, dev)
    if B == 0:  # all rows are behind the last sequence
        with _on(stream, page_table.device):
            slots.fill_(-1)
            positions.zero_()
            offsets.zero_()
        return o
    _call(lib.svf_page_reserve, "svf_page_reserve", dev, stream, page_table.data_ptr(), max_pages,
          page_size, free.data_ptr(), pool["state"].data_ptr(), free.numel(), seq_lens.data_ptr(),
          new_lens.data_ptr(), B, rows, d, slots.data_ptr(), positions.data_ptr(),
          offsets.data_ptr(), status.data_ptr())
    return o


def page_release(pool: dict, page_table: torch.Tensor, old_lens: torch.Tensor,
                 keep_lens: torch.Tensor, page_size: int, outputs: Optional[dict] = None,
                 stream=None) -> dict:
    """Give the pages past the first ``keep_lens`` [B] of ``old_lens`` [B]
    tokens back to the pool (after kv_commit: seq_lens + N and new_seq_lens;
    for finished requests keep 0). In a pool with ``shares`` a page goes back
    when its last holder leaves it. Returns n_released [B], status [B]."""
    lib = _lib or load_library()
    shares = pool.get("shares")
    if _fast is not None and outputs is not None:
        fn = _fast.page_release if shares is None else _fast.page_release_shared
        rc = fn(pool, page_table, old_lens, keep_lens, page_size, outputs, stream)
        if rc is not None:
            _check(rc, "svf_page_release" if shares is None else "svf_page_release_shared")
            return outputs
    dev, B, max_pages = _page_args(pool, page_table, old_lens, "old_lens", keep_lens, "keep_lens")
    free, i32 = pool["free"], torch.int32
    o = outputs if outputs is not None else {}
    try:
        n_released, status = o["n_released"], o["status"]
        fine = (n_released.dtype is i32 and n_released.get_device() == dev
                and n_released.shape == (B,) and n_released.is_contiguous()
                and status.dtype is i32 and status.get_device() == dev
                and status.shape == (B,) and status.is_contiguous())
    except (KeyError, AttributeError):
        fine = False
    if not fine:
        _outs(o, i32, page_table, dev, stream, n_released=(B,), status=(B,))
        n_released, status = o["n_released"], o["status"]
    if shares is not None:
        _call(lib.svf_page_release_shared, "svf_page_release_shared", dev, stream,
              page_table.data_ptr(), max_pages, page_size, free.data_ptr(),
              pool["state"].data_ptr(), free.numel(),
              _p(shares, "pool['shares']", i32, free.shape, dev), old_lens.data_ptr(),
              keep_lens.data_ptr(), B, n_released.data_ptr(), status.data_ptr())
        return o
    _call(lib.svf_page_release, "svf_page_release", dev, stream, page_table.data_ptr(), max_pages,
          page_size, free.data_ptr(), pool["state"].data_ptr(), free.numel(), old_lens.data_ptr(),
          keep_lens.data_ptr(), B, n_released.data_ptr(), status.data_ptr())
    return o


def page_fork(pool: dict, page_table: torch.Tensor, seq_lens: torch.Tensor, src: torch.Tensor,
              dst: torch.Tensor, page_size: int, outputs: Optional[dict] = None,
              stream=None) -> dict:
    """Rows ``dst`` [F] of ``page_table`` become sequences of the tokens of rows
    ``src`` [F] (int32): full pages are shared, the tokens behind them get a page
    of the pool, which page_copy fills. The pool has ``shares``
    (page_pool(..., shared=True)); page_table, seq_lens and the pool are updated in
    place. Returns device tensors copy_src, copy_dst, copy_len, status [F]."""
    lib = _lib or load_library()
    if _fast is not None and outputs is not None:
        rc = _fast.page_fork(pool, page_table, seq_lens, src, dst, page_size, outputs, stream)
        if rc is not None:
            _check(rc, "svf_page_fork")
            return outputs
    if "shares" not in pool:
        raise SpecVerifyError("the pool has no 'shares': make it with page_pool(..., shared=True)")
    dev, B, max_pages = _page_args(pool, page_table, seq_lens, "seq_lens", seq_lens, "seq_lens")
    i32, free = torch.int32, pool["free"]
    shares = _p(pool["shares"], "pool['shares']", i32, free.shape, dev)
    F = src.shape[0] if isinstance(src, torch.Tensor) and src.dim() == 1 else -1
    if F < 0:
        raise SpecVerifyError("src must be [F]")
    sp, dp = _p(src, "src", i32, (F,), dev), _p(dst, "dst", i32, (F,), dev)
    o = outputs if outputs is not None else {}
    _outs(o, i32, page_table, dev, stream, copy_src=(F,), copy_dst=(F,), copy_len=(F,),
          status=(F,))
    _call(lib.svf_page_fork, "svf_page_fork", dev, stream, page_table.data_ptr(), max_pages,
          page_size, free.data_ptr(), pool["state"].data_ptr(), free.numel(), shares,
          seq_lens.data_ptr(), B, sp, dp, F, o["copy_src"].data_ptr(), o["copy_dst"].data_ptr(),
          o["copy_len"].data_ptr(), o["status"].data_ptr())
    return o


def _layered(k_cache, v_cache):
    """(layers, layer stride, pages, page size, Hkv, D) of a pair of caches."""
    dev = _device_of(k_cache, "k_cache")
    if k_cache.dim() == 4:
        layers, (num_pages, page_size, Hkv, D), stride = 1, k_cache.shape, 0
    elif k_cache.dim() == 5:
        layers, num_pages, page_size, Hkv, D = k_cache.shape
        stride = k_cache.stride(0)
    else:
        raise SpecVerifyError("k_cache must be [layers,] num_pages, page_size, Hkv, D")
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype != k_cache.dtype \
                or t.shape != k_cache.shape:
            _bad(t, name, k_cache.dtype, k_cache.shape, dev)
        if layers and not (t[0] if t.dim() == 5 else t).is_contiguous():
            raise SpecVerifyError(f"each layer of {name} must be contiguous")
    if v_cache.stride() != k_cache.stride():
        raise SpecVerifyError("v_cache must have k_cache's strides")
    return dev, layers, stride, num_pages, page_size, Hkv, D


def page_copy(k_cache: torch.Tensor, v_cache: torch.Tensor, src: torch.Tensor, dst: torch.Tensor,
              lens: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """The first ``lens`` [n] tokens (None: all) of pages ``src`` [n] over those of
    pages ``dst`` [n] (int32; -1, -1 leaves an entry out), in place, in every layer of
    k_cache and v_cache [layers, num_pages, page_size, Hkv, D] (or without the layer
    axis). Returns status [n]."""
    lib = _lib or load_library()
    if _fast is not None and status is not None:
        rc = _fast.page_copy(k_cache, v_cache, src, dst, lens, status, stream)
        if rc is not None:
            _check(rc, "svf_page_copy")
            return status
    dev, layers, stride, num_pages, page_size, Hkv, D = _layered(k_cache, v_cache)
    i32 = torch.int32
    n = src.shape[0] if isinstance(src, torch.Tensor) and src.dim() == 1 else -1
    if n < 0:
        raise SpecVerifyError("src must be [n]")
    sp, dp = _p(src, "src", i32, (n,), dev), _p(dst, "dst", i32, (n,), dev)
    lp = None if lens is None else _p(lens, "lens", i32, (n,), dev)
    if status is None:
        with _on(stream, k_cache.device):
            status = torch.empty((n,), dtype=i32, device=k_cache.device)
    _call(lib.svf_page_copy, "svf_page_copy", dev, stream, k_cache.data_ptr(), v_cache.data_ptr(),
          layers, stride, num_pages, page_size, sp, dp, lp, n, Hkv, D, _dtype_code(k_cache.dtype),
          _p(status, "status", i32, (n,), dev))
    return status


def _row_stride(t, name: str, dtype, shape, dev: int) -> int:
    """Elements between the rows of [T, heads, D] with dense heads."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == dev):
        _bad(t, name, dtype, shape, dev)
    s0, s1, s2 = t.stride()
    if (s2 != 1 and shape[2] > 1) or (s1 != shape[2] and shape[1] > 1):
        raise SpecVerifyError(f"{name} must have dense heads (strides [row, D, 1])")
    return s0 if shape[0] > 1 else shape[1] * shape[2]


def rope_kv_write(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, rope: torch.Tensor,
                  positions: torch.Tensor, slots: torch.Tensor, k_cache: torch.Tensor,
                  v_cache: torch.Tensor, q_out: Optional[torch.Tensor] = None,
                  interleaved: bool = False, status: Optional[torch.Tensor] = None, stream=None):
    """Rotary positions of q and k rows, and the K/V write into the cache.

    q [T, Hq, D], k and v [T, Hkv, D] float32 or bfloat16, heads dense, rows
    any distance apart (slices of a fused projection); rope [max_pos, rot]
    float32, cosines then sines; positions, slots [T] int32 (page_reserve's;
    slot -1 leaves a row out); k_cache, v_cache [num_pages, page_size, Hkv, D].
    Returns (q_out [T, Hq, D], status [T] int32). Rows that are left out keep
    what q_out held (a new q_out: undefined)."""
    lib = _lib or load_library()
    if _fast is not None:
        rc = _fast.rope_kv_write(q, k, v, rope, positions, slots, k_cache, v_cache, q_out,
                                 interleaved, status, stream)
        if rc is not None:
            _check(rc, "svf_rope_kv_write")
            return q_out, status
    dev = _device_of(q, "q")
    if q.dim() != 3 or k.dim() != 3 or k_cache.dim() != 4 or rope.dim() != 2:
        raise SpecVerifyError("q and k must be [T, heads, D], the caches [pages, page_size, Hkv, "
                              "D], rope [max_pos, rot]")
    T, Hq, D = q.shape
    Hkv, dt, i32 = k.shape[1], q.dtype, torch.int32
    qs, ks, vs = (_row_stride(q, "q", dt, (T, Hq, D), dev), _row_stride(k, "k", dt, (T, Hkv, D), dev),
                  _row_stride(v, "v", dt, (T, Hkv, D), dev))
    max_pos, rot = rope.shape
    pages, ps = k_cache.shape[:2]
    cache, row = (pages, ps, Hkv, D), (T,)
    if q_out is None or status is None:
        with _on(stream, q.device):
            if q_out is None:
                q_out = torch.empty((T, Hq, D), dtype=dt, device=q.device)
            if status is None:
                status = torch.empty(row, dtype=i32, device=q.device)
    try:
        fine = (rope.dtype is torch.float32 and rope.get_device() == dev and rope.is_contiguous()
                and positions.dtype is i32 and positions.get_device() == dev
                and positions.shape == row and positions.is_contiguous()
                and slots.dtype is i32 and slots.get_device() == dev and slots.shape == row
                and slots.is_contiguous()
                and q_out.dtype is dt and q_out.get_device() == dev and q_out.shape == (T, Hq, D)
                and q_out.is_contiguous()
                and k_cache.dtype is dt and k_cache.get_device() == dev
                and k_cache.shape == cache and k_cache.is_contiguous()
                and v_cache.dtype is dt and v_cache.get_device() == dev
                and v_cache.shape == cache and v_cache.is_contiguous()
                and status.dtype is i32 and status.get_device() == dev and status.shape == row
                and status.is_contiguous())
    except AttributeError:
        fine = False
    if not fine:
        for t, name, dtype, shape in (
                (rope, "rope", torch.float32, (max_pos, rot)), (positions, "positions", i32, row),
                (slots, "slots", i32, row), (q_out, "q_out", dt, (T, Hq, D)),
                (k_cache, "k_cache", dt, cache), (v_cache, "v_cache", dt, cache),
                (status, "status", i32, row)):
            _p(t, name, dtype, shape, dev)
    _call(lib.svf_rope_kv_write, "svf_rope_kv_write", dev, stream, q.data_ptr(), k.data_ptr(),
          v.data_ptr(), qs, ks, vs, T, Hq, Hkv, D, _dtype_code(dt), rope.data_ptr(), rot, max_pos,
          1 if interleaved else 0, positions.data_ptr(), slots.data_ptr(), q_out.data_ptr(),
          k_cache.data_ptr(), v_cache.data_ptr(), pages * ps, status.data_ptr())
    return q_out, status


def norm_rope_kv_write(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                       q_norm: Optional[torch.Tensor], k_norm: Optional[torch.Tensor],
                       rope: torch.Tensor, positions: torch.Tensor, slots: torch.Tensor,
                       k_cache: torch.Tensor, v_cache: torch.Tensor, eps: float = 1e-6,
                       pair_axis: Optional[torch.Tensor] = None,
                       q_out: Optional[torch.Tensor] = None, interleaved: bool = False,
                       status: Optional[torch.Tensor] = None, stream=None):
    """rope_kv_write with a norm of every q and k head before it, and positions on
    several axes.

    q_norm, k_norm [D] of q's dtype (None: no norm); positions [T], or [axes, T] with
    ``pair_axis`` [rot / 2] int32, the axis that turns each pair. The other arguments,
    the results and the rows that are left out are rope_kv_write's."""
    lib = _lib or load_library()
    if _fast is not None and q_out is not None:
        rc = _fast.norm_rope_kv_write(q, k, v, q_norm, k_norm, rope, positions, slots, k_cache,
                                      v_cache, eps, pair_axis, q_out, interleaved, status, stream)
        if rc is not None:
            _check(rc, "svf_norm_rope_kv_write")
            return q_out, status
    dev = _device_of(q, "q")
    if q.dim() != 3 or k.dim() != 3 or k_cache.dim() != 4 or rope.dim() != 2:
        raise SpecVerifyError("q and k must be [T, heads, D], the caches [pages, page_size, Hkv, "
                              "D], rope [max_pos, rot]")
    T, Hq, D = q.shape
    Hkv, dt, i32 = k.shape[1], q.dtype, torch.int32
    qs, ks, vs = (_row_stride(q, "q", dt, (T, Hq, D), dev), _row_stride(k, "k", dt, (T, Hkv, D), dev),
                  _row_stride(v, "v", dt, (T, Hkv, D), dev))
    max_pos, rot = rope.shape
    pages, ps = k_cache.shape[:2]
    if positions.dim() == 2:
        axes = positions.shape[0]
        if axes > 1 and pair_axis is None:
            raise SpecVerifyError("positions on several axes need pair_axis")
        pos = _p(positions, "positions", i32, (axes, T), dev)
    else:
        axes, pos = 1, _p(positions, "positions", i32, (T,), dev)
    axis = None if pair_axis is None else _p(pair_axis, "pair_axis", i32, (rot // 2,), dev)
    wq = None if q_norm is None else _p(q_norm, "q_norm", dt, (D,), dev)
    wk = None if k_norm is None else _p(k_norm, "k_norm", dt, (D,), dev)
    if q_out is None or status is None:
        with _on(stream, q.device):
            if q_out is None:
                q_out = torch.empty((T, Hq, D), dtype=dt, device=q.device)
            if status is None:
                status = torch.empty((T,), dtype=i32, device=q.device)
    cache = (pages, ps, Hkv, D)
    _call(lib.svf_norm_rope_kv_write, "svf_norm_rope_kv_write", dev, stream, q.data_ptr(),
          k.data_ptr(), v.data_ptr(), qs, ks, vs, T, Hq, Hkv, D, _dtype_code(dt), wq, wk,
          float(eps), _p(rope, "rope", torch.float32, (max_pos, rot), dev), rot, max_pos,
          1 if interleaved else 0, pos, axes, axis, _p(slots, "slots", i32, (T,), dev),
          _p(q_out, "q_out", dt, (T, Hq, D), dev), _p(k_cache, "k_cache", dt, cache, dev),
          _p(v_cache, "v_cache", dt, cache, dev), pages * ps, _p(status, "status", i32, (T,), dev))
    return q_out, status


# ---------------------------------------------------------------------------
# Attention of chunks of new tokens over the paged cache
# ---------------------------------------------------------------------------

def chunk_attn_workspace_size(rows, B, Hq, Hkv, D, dtype) -> int:
    return int((_lib or load_library()).svf_chunk_attn_workspace_size(
        rows, B, Hq, Hkv, D, _dtype_code(dtype) if isinstance(dtype, torch.dtype) else int(dtype)))


def chunk_attn(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
               page_table: torch.Tensor, seq_lens: torch.Tensor, row_offsets: torch.Tensor,
               sm_scale: float = 0.0, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               status: Optional[torch.Tensor] = None, want_lse: bool = True, stream=None):
    """Causal attention of chunks of new tokens over the paged cache.

    q [rows, Hq, D]; k_cache, v_cache [num_pages, page_size, Hkv, D] (same dtype,
    float32 or bfloat16), the chunks' own K/V already in it; page_table [B, max_pages],
    seq_lens [B] (tokens before the chunk), row_offsets [B + 1] int32 (page_reserve's:
    sequence b's tokens are rows row_offsets[b] .. row_offsets[b + 1]). A row sees the
    tokens up to its own. ``workspace``: chunk_attn_workspace_size bytes, zero-filled
    once; calls that may overlap need workspaces of their own (without one, the binding
    keeps one per stream). Returns (out [rows, Hq, D], lse [rows, Hq] float32 or None,
    status [B] int32); rows behind the last sequence keep what out and lse held (new
    ones: undefined)."""
    lib = _lib or load_library()
    if _fast is not None and workspace is not None and (lse is not None or not want_lse):
        rc = _fast.chunk_attn(q, k_cache, v_cache, page_table, seq_lens, row_offsets, sm_scale, out,
                              lse, workspace, status, stream)
        if rc is not None:
            _check(rc, "svf_chunk_attn")
            return out, lse, status
    dev = _device_of(q, "q")
    if q.dim() != 3 or k_cache.dim() != 4 or page_table.dim() != 2:
        raise SpecVerifyError("q must be [rows, Hq, D], k_cache [pages, page_size, Hkv, D], "
                              "page_table [B, max_pages]")
    rows, Hq, D = q.shape
    dt, i32, f32 = q.dtype, torch.int32, torch.float32
    num_pages, page_size, Hkv = k_cache.shape[:3]
    B, max_pages = page_table.shape
    cache = (num_pages, page_size, Hkv, D)
    code = _dtype_code(dt)
    args = (_p(q, "q", dt, (rows, Hq, D), dev), _p(k_cache, "k_cache", dt, cache, dev),
            _p(v_cache, "v_cache", dt, cache, dev), num_pages, page_size,
            _p(page_table, "page_table", i32, (B, max_pages), dev), max_pages,
            _p(seq_lens, "seq_lens", i32, (B,), dev),
            _p(row_offsets, "row_offsets", i32, (B + 1,), dev), B, rows, Hq, Hkv, D, code,
            float(sm_scale))
    if out is None or status is None or (lse is None and want_lse):
        with _on(stream, q.device):
            if out is None:
                out = torch.empty((rows, Hq, D), dtype=dt, device=q.device)
            if lse is None and want_lse:
                lse = torch.empty((rows, Hq), dtype=f32, device=q.device)
            if status is None:
                status = torch.empty((B,), dtype=i32, device=q.device)
    op = _p(out, "out", dt, (rows, Hq, D), dev)
    lp = None if lse is None else _p(lse, "lse", f32, (rows, Hq), dev)
    st = _p(status, "status", i32, (B,), dev)
    if workspace is None:
        need = int(lib.svf_chunk_attn_workspace_size(rows, B, Hq, Hkv, D, code))
        if need:
            with torch.cuda.device(dev):
                workspace = _zeroed_workspace(need, q.device, stream, "chunk")
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise SpecVerifyError("workspace must be a contiguous tensor on q's device")
    _call(lib.svf_chunk_attn, "svf_chunk_attn", dev, stream, *args, op, lp,
          None if workspace is None else workspace.data_ptr(),
          0 if workspace is None else workspace.nbytes, st)
    return out, lse, status


def lora_proj_workspace_size(R: int, rank: int) -> int:
    return int((_lib or load_library()).svf_lora_proj_workspace_size(R, rank))


def lora_proj(x: torch.Tensor, weight: torch.Tensor, lora_a: torch.Tensor, lora_b: torch.Tensor,
              ids: torch.Tensor, scales: Optional[torch.Tensor] = None,
              out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
              status: Optional[torch.Tensor] = None, stream=None):
    """out = x weight^T + scales[a] (x lora_a[a]^T) lora_b[a]^T with one adapter
    a = ids[g] per group of rows (-1: none).

    x [..., H] bfloat16 of R rows (2-D: rows any multiple of 8 elements apart),
    weight [O, H], lora_a [adapters, rank, H], lora_b [adapters, O, rank]
    bfloat16; ids [G] int32, group g being the R / G rows from g R / G on
    (x [B, N, H] with ids [B]: one adapter per request); scales [adapters]
    float32. Returns (out [..., O] bfloat16, status [G] int32)."""
    lib = _lib or load_library()
    if _fast is not None:
        rc = _fast.lora_proj(x, weight, lora_a, lora_b, ids, scales, out, workspace, status, stream)
        if rc is not None:
            _check(rc, "svf_lora_proj")
            return out, status
    dev = _device_of(x, "x")
    bf = torch.bfloat16
    if weight.dim() != 2 or lora_a.dim() != 3:
        raise SpecVerifyError("weight must be [O, H] and lora_a [adapters, rank, H]")
    O, H = weight.shape
    adapters, rank = lora_a.shape[:2]
    if x.dtype is not bf or x.dim() < 1 or x.shape[-1] != H:
        raise SpecVerifyError("x must be bfloat16 [..., H] with weight's H")
    if x.is_contiguous():
        xs = H
    elif x.dim() == 2 and x.stride(1) == 1:
        xs = x.stride(0)
    else:
        raise SpecVerifyError("x must be contiguous, or 2-D with dense rows")
    R = x.numel() // H if H > 0 else 0
    G = ids.shape[0] if ids.dim() == 1 else 0
    if R > 0 and (G < 1 or R % G):
        raise SpecVerifyError("ids must be [G] with G dividing the rows of x")
    shape = x.shape[:-1] + (O,)
    i32 = torch.int32
    if out is None or status is None or workspace is None:
        with _on(stream, x.device):
            if out is None:
                out = torch.empty(shape, dtype=bf, device=x.device)
            if status is None:
                status = torch.empty((G,), dtype=i32, device=x.device)
            if workspace is None:
                workspace = torch.empty((lora_proj_workspace_size(R, rank),), dtype=torch.uint8,
                                        device=x.device)
    if out.dim() == 2 and out.shape[0] > 1 and not out.is_contiguous():
        if out.stride(1) != 1 or out.shape != shape or out.dtype is not bf \
                or out.get_device() != dev:
            raise SpecVerifyError("out must be bfloat16 [..., O] with dense rows")
        op, os_ = out.data_ptr(), out.stride(0)
    else:
        op, os_ = _p(out, "out", bf, shape, dev), O
    try:
        fine = (weight.dtype is bf and weight.get_device() == dev and weight.is_contiguous()
                and lora_a.dtype is bf and lora_a.get_device() == dev
                and lora_a.shape[2] == H and lora_a.is_contiguous()
                and lora_b.dtype is bf and lora_b.get_device() == dev
                and lora_b.shape == (adapters, O, rank) and lora_b.is_contiguous()
                and ids.dtype is i32 and ids.get_device() == dev and ids.is_contiguous()
                and (scales is None
                     or (scales.dtype is torch.float32 and scales.get_device() == dev
                         and scales.shape == (adapters,) and scales.is_contiguous()))
                and status.dtype is i32 and status.get_device() == dev and status.shape == (G,)
                and status.is_contiguous()
                and workspace.get_device() == dev and workspace.is_contiguous())
    except AttributeError:
        fine = False
    if not fine:
        _p(weight, "weight", bf, (O, H), dev)
        _p(lora_a, "lora_a", bf, (adapters, rank, H), dev)
        _p(lora_b, "lora_b", bf, (adapters, O, rank), dev)
        _p(ids, "ids", i32, (G,), dev)
        if scales is not None:
            _p(scales, "scales", torch.float32, (adapters,), dev)
        _p(status, "status", i32, (G,), dev)
        raise SpecVerifyError("workspace must be a contiguous tensor on x's device")
    if R == 0:
        with _on(stream, x.device):
            status.zero_()
        return out, status
    _call(lib.svf_lora_proj, "svf_lora_proj", dev, stream, x.data_ptr(), xs, weight.data_ptr(),
          lora_a.data_ptr(), lora_b.data_ptr(), None if scales is None else scales.data_ptr(),
          ids.data_ptr(), R // G if G else 1, R, H, O, adapters, rank, op, os_,
          workspace.data_ptr(), workspace.nbytes, status.data_ptr())
    return out, status


# ---------------------------------------------------------------------------
# One verify step: mask -> attention -> acceptance
# ---------------------------------------------------------------------------

def verify_step(parent, tokens, q, k_cache, v_cache, page_table, seq_lens, target_logits,
                draft_logits, u_accept, u_bonus, stream=None, buffers: Optional[dict] = None):
    """The whole hot path on device tensors: ancestor masks and tree attention
    of one layer (one fused call), then the acceptance walk. ``buffers``
    (optional) holds preallocated outputs and workspaces and is filled on the
    first call."""
    bufs = buffers if buffers is not None else {}
    ws = bufs.get("attn_ws")
    if ws is None:
        B, N, Hq, D = q.shape
        need = tree_verify_attn_workspace_size(B, N, Hq, k_cache.shape[2], D, q.dtype,
                                               page_table.shape[1], k_cache.shape[1])
        with _on(stream, q.device):  # the attention's counters begin at zero
            ws = torch.zeros((max(need, 1),), dtype=torch.uint8, device=q.device)
            if not torch.cuda.is_current_stream_capturing():
                bufs["attn_ws"] = ws  # (one of a graph does so in its replays only)
    out, lse, astatus, anc, depth, mstatus = tree_mask_attn(
        parent, q, k_cache, v_cache, page_table, seq_lens, anc=bufs.get("anc"),
        depth=bufs.get("depth"), mask_status=bufs.get("mask_status"), out=bufs.get("attn_out"),
        lse=bufs.get("lse"), workspace=ws, status=bufs.get("attn_status"),
        stream=stream)
    bufs["anc"], bufs["depth"], bufs["mask_status"] = anc, depth, mstatus
    bufs["attn_out"], bufs["lse"], bufs["attn_status"] = out, lse, astatus
    if "acc_ws" not in bufs:
        B, N, V = target_logits.shape
        bufs["acc_ws"] = torch.empty((spec_accept_workspace_size(B, N, V),), dtype=torch.uint8,
                                     device=q.device)
    res = spec_accept(target_logits, draft_logits, tokens, parent, u_accept, u_bonus,
                      workspace=bufs["acc_ws"], outputs=bufs.get("accept"), stream=stream)
    bufs["accept"] = res
    return out, lse, res, bufs

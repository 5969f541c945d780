"""Torch-facing wrappers of the paged KV cache's entry points (argument
marshalling only, as in ``ops``)."""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .ops import CAUSAL_BOTTOM_RIGHT, LAYOUT_BHSD, LAYOUT_BSHD, _check_lengths, _check_tensor, _stream_handle


def _check_ints(name, t, shape, device):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32:
        raise TypeError(f"{name} must be an int32 tensor")
    if tuple(t.shape) != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {list(shape)} tensor on {device}, got {tuple(t.shape)}")


def _check_pages(name, t):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be a torch.bfloat16 tensor")
    if t.dim() != 4:
        raise ValueError(f"{name} must have 4 dims, got {t.dim()}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    _, s1, s2, d = t.shape
    if t.stride()[1:] != (s2 * d, d, 1):
        raise ValueError(f"{name} must be dense inside a page")


def _paged_cache(k_pages, v_pages, layout, device, block_table=None):
    """(attn_paged_cache_t, Hkv, d) of two page pools [N, Hkv, P, d] ([N, P, Hkv, d] for
    LAYOUT_BSHD), dense inside a page and of one stride between pages."""
    _check_pages("k_pages", k_pages)
    _check_pages("v_pages", v_pages)
    if layout == LAYOUT_BSHD:
        N, P, Hkv, d = k_pages.shape
    elif layout == LAYOUT_BHSD:
        N, Hkv, P, d = k_pages.shape
    else:
        raise ValueError(f"unknown layout {layout}")
    if v_pages.shape != k_pages.shape or (N > 1 and v_pages.stride(0) != k_pages.stride(0)):
        raise ValueError("k_pages and v_pages must have one shape and one page stride")
    if k_pages.device != device or v_pages.device != device:
        raise ValueError(f"k_pages and v_pages must be on {device}")
    c = _lib.PagedCache()
    c.k_pages = k_pages.data_ptr()
    c.v_pages = v_pages.data_ptr()
    c.page_stride = k_pages.stride(0) if N > 1 else 0
    c.num_pages = N
    c.page_size = P
    c.layout = int(layout)
    if block_table is not None:
        c.block_table = block_table.data_ptr()
        c.max_pages = int(block_table.shape[1])
    return c, Hkv, d


def _check_table(block_table, B, device):
    if not isinstance(block_table, torch.Tensor) or block_table.dtype != torch.int32 or block_table.dim() != 2:
        raise TypeError("block_table must be an int32 tensor [B, max_pages]")
    if block_table.shape[0] != B or block_table.device != device or not block_table.is_contiguous():
        raise ValueError(f"block_table must be a contiguous [{B}, max_pages] tensor on {device}")


def _outputs(q, lse_shape, out, lse, return_lse):
    if out is None:
        out = torch.zeros_like(q)
    else:
        _check_tensor("out", out, torch.bfloat16, q.dim())
        if out.shape != q.shape or out.device != q.device:
            raise ValueError("out must have the shape of q, on q's device")
    if lse is None:
        if return_lse:
            lse = torch.zeros(lse_shape, dtype=torch.float32, device=q.device)
    else:
        _check_tensor("lse", lse, torch.float32, len(lse_shape))
        if tuple(lse.shape) != lse_shape or lse.device != q.device:
            raise ValueError(f"lse must be {list(lse_shape)} on q's device")
    return out, lse


def _check_workspace(workspace, device):
    if not isinstance(workspace, torch.Tensor) or workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous buffer on q's device")


def attn_page_plan(past_lens, new_lens, block_table, free_pages, free_range, page_size: int, num_tokens: int,
                   cu_new=None, total_lens=None, positions=None, slot_map=None, free_range_out=None):
    """Block tables and slot maps of the next step, built on the device (``attn_page_plan``).

    Request b holds ``past_lens[b]`` keys and brings ``new_lens[b]`` tokens (int32 [B]);
    ``block_table`` [B, max_pages] int32 gets the entries of its new pages in place.  The
    entries ``free_range[0]`` .. ``free_range[1] - 1`` of ``free_pages`` (int32) are the free
    pages.  ``num_tokens`` is the size of the ragged batch's buffers; tokens behind the last
    request are padding.  Returns (cu_new [B+1], total_lens [B], positions [num_tokens],
    slot_map [num_tokens], free_range_out [2]), all int32; ``total_lens`` may be ``past_lens``
    or ``new_lens`` and ``free_range_out`` may be ``free_range``.  Refused requests are
    reported by check_device_error (ATTN_ERR_PAGE).
    """
    if not isinstance(past_lens, torch.Tensor) or past_lens.dim() != 1:
        raise TypeError("past_lens must be an int32 tensor [B]")
    if not past_lens.is_cuda:
        raise ValueError("past_lens must be a CUDA tensor")
    B, dev = past_lens.shape[0], past_lens.device
    _check_lengths("past_lens", past_lens, B, dev)
    _check_lengths("new_lens", new_lens, B, dev)
    _check_table(block_table, B, dev)
    if not isinstance(free_pages, torch.Tensor) or free_pages.dim() != 1:
        raise TypeError("free_pages must be an int32 tensor [num_free]")
    _check_ints("free_pages", free_pages, (free_pages.shape[0],), dev)
    _check_ints("free_range", free_range, (2,), dev)
    T = int(num_tokens)
    if T < 0:
        raise ValueError("num_tokens must not be negative")
    outs = []
    for name, t, n in (("cu_new", cu_new, B + 1), ("total_lens", total_lens, B), ("positions", positions, T),
                       ("slot_map", slot_map, T), ("free_range_out", free_range_out, 2)):
        if t is None:
            t = torch.empty(n, dtype=torch.int32, device=dev)
        else:
            _check_ints(name, t, (n,), dev)
        outs.append(t)
    lib = _lib.get()
    with torch.cuda.device(dev):
        st = lib.attn_page_plan(past_lens.data_ptr(), new_lens.data_ptr(), block_table.data_ptr(),
                                free_pages.data_ptr(), free_range.data_ptr(), outs[0].data_ptr(), outs[1].data_ptr(),
                                outs[2].data_ptr(), outs[3].data_ptr(), outs[4].data_ptr(), B,
                                int(block_table.shape[1]), int(free_pages.shape[0]), int(page_size), T,
                                _stream_handle(dev))
    _lib.check(st, "attn_page_plan")
    return tuple(outs)


def attn_rope_append_paged(packed_qkv, cos, sin, positions, slot_map, k_pages, v_pages, Hq: int, Hkv: int,
                           layout: int = LAYOUT_BHSD, q_out=None):
    """``attn_rope_append`` for a ragged batch and a paged cache (``attn_rope_append_paged``).

    packed_qkv [T, (Hq + 2*Hkv) * d] bf16; cos, sin [max_pos, d/2] fp32; positions and slot_map
    [T] int32 as from attn_page_plan; k_pages, v_pages [N, Hkv, P, d] bf16 ([N, P, Hkv, d] for
    LAYOUT_BSHD), updated in place.  Returns q [T, Hq, d]; rows of tokens with a negative slot
    are not written (a new ``q_out`` is zero-filled).
    """
    _check_tensor("packed_qkv", packed_qkv, torch.bfloat16, 2)
    _check_tensor("cos", cos, torch.float32, 2)
    _check_tensor("sin", sin, torch.float32, 2)
    T, width = packed_qkv.shape
    dev = packed_qkv.device
    cache, pages_hkv, d = _paged_cache(k_pages, v_pages, layout, dev)
    if pages_hkv != Hkv or Hq <= 0 or width != (Hq + 2 * Hkv) * d:
        raise ValueError("packed_qkv's last dim must be (Hq + 2*Hkv) * d of pages with Hkv heads")
    if cos.shape != sin.shape or cos.shape[1] != d // 2 or cos.device != dev or sin.device != dev:
        raise ValueError("cos and sin must both be [max_pos, d/2] on packed_qkv's device")
    _check_ints("positions", positions, (T,), dev)
    _check_ints("slot_map", slot_map, (T,), dev)
    if q_out is None:
        q_out = torch.zeros((T, Hq, d), dtype=torch.bfloat16, device=dev)
    else:
        _check_tensor("q_out", q_out, torch.bfloat16, 3)
        if tuple(q_out.shape) != (T, Hq, d) or q_out.device != dev:
            raise ValueError(f"q_out must be {(T, Hq, d)} on packed_qkv's device")
    lib = _lib.get()
    with torch.cuda.device(dev):
        st = lib.attn_rope_append_paged(packed_qkv.data_ptr(), cos.data_ptr(), sin.data_ptr(), int(cos.shape[0]),
                                        positions.data_ptr(), slot_map.data_ptr(), q_out.data_ptr(),
                                        ctypes.byref(cache), T, Hq, Hkv, d, _stream_handle(dev))
    _lib.check(st, "attn_rope_append_paged")
    return q_out


def fwd_paged_workspace_size(T, Hq, Hkv, d) -> int:
    """Bytes of workspace ``attn_fwd_paged`` needs."""
    return int(_lib.get().attn_fwd_paged_workspace_size(T, Hq, Hkv, d))


def decode_paged_workspace_size(B, Hq, Hkv, Sq, d) -> int:
    """Bytes of workspace ``attn_decode_splitkv_paged`` needs."""
    return int(_lib.get().attn_decode_paged_workspace_size(B, Hq, Hkv, Sq, d))


def _pages_hkv(k_pages, layout):
    return k_pages.shape[2] if layout == LAYOUT_BSHD else k_pages.shape[1]


def fwd_paged_workspace(q, k_pages, layout: int = LAYOUT_BHSD) -> torch.Tensor:
    """A caller-owned workspace buffer for ``attn_fwd_paged`` with this q [T, Hq, d]."""
    T, Hq, d = q.shape
    with torch.cuda.device(q.device):
        n = fwd_paged_workspace_size(T, Hq, _pages_hkv(k_pages, layout), d)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=q.device)


def decode_paged_workspace(q, k_pages, layout: int = LAYOUT_BHSD) -> torch.Tensor:
    """A caller-owned workspace buffer for ``attn_decode_splitkv_paged`` with this q [B, Sq, Hq, d]."""
    B, Sq, Hq, d = q.shape
    with torch.cuda.device(q.device):
        n = decode_paged_workspace_size(B, Hq, _pages_hkv(k_pages, layout), Sq, d)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=q.device)


def attn_fwd_paged(q, k_pages, v_pages, cu_q, seqlens_k, block_table, causal: int = CAUSAL_BOTTOM_RIGHT,
                   scale: float = 0.0, layout: int = LAYOUT_BHSD, workspace=None, out=None, lse=None,
                   return_lse: bool = True):
    """Attention of ragged chunks of new tokens over a paged cache (``attn_fwd_paged``).

    q [T, Hq, d] bf16, sequence b's tokens at cu_q[b] .. cu_q[b+1]-1 (int32 [B+1]);
    k_pages, v_pages [N, Hkv, P, d] bf16 ([N, P, Hkv, d] for LAYOUT_BSHD); seqlens_k [B] int32
    keys per sequence; block_table [B, max_pages] int32.  Returns (o [T, Hq, d], lse [Hq, T]
    fp32); rows behind cu_q[B] are not written (new buffers are zero-filled).
    """
    _check_tensor("q", q, torch.bfloat16, 3)
    T, Hq, d = q.shape
    dev = q.device
    if not isinstance(seqlens_k, torch.Tensor) or seqlens_k.dim() != 1:
        raise TypeError("seqlens_k must be an int32 tensor [B]")
    B = seqlens_k.shape[0]
    _check_lengths("seqlens_k", seqlens_k, B, dev)
    _check_ints("cu_q", cu_q, (B + 1,), dev)
    _check_table(block_table, B, dev)
    cache, Hkv, dk = _paged_cache(k_pages, v_pages, layout, dev, block_table)
    if dk != d:
        raise ValueError(f"head_dim of q ({d}) and of the pages ({dk}) differ")
    out, lse = _outputs(q, (Hq, T), out, lse, return_lse)
    if workspace is None:
        workspace = fwd_paged_workspace(q, k_pages, layout)
    _check_workspace(workspace, dev)
    lib = _lib.get()
    with torch.cuda.device(dev):
        st = lib.attn_fwd_paged(q.data_ptr(), ctypes.byref(cache), cu_q.data_ptr(), seqlens_k.data_ptr(),
                                out.data_ptr(), lse.data_ptr() if lse is not None else None, B, T, Hq, Hkv, d,
                                float(scale), int(causal), workspace.data_ptr(),
                                workspace.numel() * workspace.element_size(), _stream_handle(dev))
    _lib.check(st, "attn_fwd_paged")
    return out, lse


def attn_decode_splitkv_paged(q, k_pages, v_pages, seqlens_k, block_table, causal: int = CAUSAL_BOTTOM_RIGHT,
                              scale: float = 0.0, layout: int = LAYOUT_BHSD, workspace=None, out=None, lse=None,
                              return_lse: bool = True):
    """Split-KV decode over a paged cache (``attn_decode_splitkv_paged``).

    q [B, Sq, Hq, d] bf16 (token-major, as attn_rope_append_paged writes it); pages, lengths and
    table as for attn_fwd_paged.  Returns (o [B, Sq, Hq, d], lse [B, Hq, Sq] fp32).
    """
    _check_tensor("q", q, torch.bfloat16, 4)
    B, Sq, Hq, d = q.shape
    dev = q.device
    _check_lengths("seqlens_k", seqlens_k, B, dev)
    _check_table(block_table, B, dev)
    cache, Hkv, dk = _paged_cache(k_pages, v_pages, layout, dev, block_table)
    if dk != d:
        raise ValueError(f"head_dim of q ({d}) and of the pages ({dk}) differ")
    out, lse = _outputs(q, (B, Hq, Sq), out, lse, return_lse)
    if workspace is None:
        workspace = decode_paged_workspace(q, k_pages, layout)
    _check_workspace(workspace, dev)
    lib = _lib.get()
    with torch.cuda.device(dev):
        st = lib.attn_decode_splitkv_paged(q.data_ptr(), ctypes.byref(cache), seqlens_k.data_ptr(), out.data_ptr(),
                                           lse.data_ptr() if lse is not None else None, B, Hq, Hkv, Sq, d,
                                           float(scale), int(causal), workspace.data_ptr(),
                                           workspace.numel() * workspace.element_size(), _stream_handle(dev))
    _lib.check(st, "attn_decode_splitkv_paged")
    return out, lse

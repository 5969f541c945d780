"""Torch-facing wrappers of the paged KV cache's entry points (argument
marshalling only, as in ``ops``).

A decode step's kernels take a few microseconds, so what a wrapper does before
the launch counts: each property of a tensor is read once, a device is compared
by its index, and the device context is entered only where it changes something.
"""
from __future__ import annotations

import torch

from . import _lib
from .ops import CAUSAL_BOTTOM_RIGHT, LAYOUT_BHSD, LAYOUT_BSHD, _stream_handle

_BF16, _INT32, _FP32 = torch.bfloat16, torch.int32, torch.float32
_Tensor = torch.Tensor
# the current device, and the current stream of one as an integer (without a Stream object), where torch
# offers them directly
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or _stream_handle


def _is_tensor(t):
    return type(t) is _Tensor or isinstance(t, _Tensor)  # isinstance alone asks torch's metaclass


def _call(fn, name, index, *args):
    """One entry point on the current stream of device `index`."""
    if _current_device() == index:
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, _raw_stream(index))
    if st:
        _lib.check(st, name)


def _tensor(name, t, dtype, ndim):
    """The device index of a contiguous CUDA tensor of this type."""
    if not _is_tensor(t):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")
    index = t.get_device()  # -1: not on a GPU
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return index


def _ints(name, t, n, index):
    """The address of a contiguous int32 tensor [n] on device `index`."""
    if not _is_tensor(t) or t.dtype is not _INT32 or t.dim() != 1:
        raise TypeError(f"{name} must be an int32 tensor [{n}]")
    if t.numel() != n or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [{n}] tensor on cuda:{index}, got {tuple(t.shape)}")
    return t.data_ptr()


def _table(t, B, index):
    """(address, entries per row) of a block table."""
    if not _is_tensor(t) or t.dtype is not _INT32 or t.dim() != 2:
        raise TypeError("block_table must be an int32 tensor [B, max_pages]")
    rows, width = t.shape
    if rows != B or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"block_table must be a contiguous [{B}, max_pages] tensor on cuda:{index}")
    return t.data_ptr(), width


def _pages(k_pages, v_pages, layout, index, table=0, max_pages=0):
    """(attn_paged_cache_t as bytes, Hkv, d) of two page pools [N, Hkv, P, d] ([N, P, Hkv, d] for
    LAYOUT_BSHD), dense inside a page and of one stride between pages."""
    if not _is_tensor(k_pages) or not _is_tensor(v_pages) or k_pages.dtype is not _BF16 or v_pages.dtype is not _BF16:
        raise TypeError("k_pages and v_pages must be torch.bfloat16 tensors")
    shape = k_pages.shape
    if len(shape) != 4 or v_pages.shape != shape:
        raise ValueError("k_pages and v_pages must have one shape of 4 dims")
    if k_pages.get_device() != index or v_pages.get_device() != index:
        raise ValueError(f"k_pages and v_pages must be on cuda:{index}")
    N, s1, s2, d = shape
    stride, s1_stride, s2_stride, s3_stride = strides = k_pages.stride()
    other = v_pages.stride()
    if s3_stride != 1 or s2_stride != d or s1_stride != s2 * d or (other != strides and other[1:] != strides[1:]):
        raise ValueError("k_pages and v_pages must be dense inside a page")
    if N < 2:
        stride = 0
    elif other[0] != stride or stride == 0:  # (0: all pages in one place, which a call would take for dense ones)
        raise ValueError("k_pages and v_pages must have one page stride, and pages that do not overlap")
    if layout == LAYOUT_BHSD:
        Hkv, P = s1, s2
    elif layout == LAYOUT_BSHD:
        P, Hkv = s1, s2
    else:
        raise ValueError(f"unknown layout {layout}")
    return _lib.pack_paged_cache(k_pages.data_ptr(), v_pages.data_ptr(), table, stride, N, P, max_pages,
                                 layout), Hkv, d


def _outputs(q, lse_shape, out, lse, return_lse, index):
    if out is None:
        out = torch.zeros_like(q)
    elif _tensor("out", out, _BF16, q.dim()) != index or out.shape != q.shape:
        raise ValueError("out must have the shape of q, on q's device")
    if lse is None:
        if return_lse:
            lse = torch.zeros(lse_shape, dtype=_FP32, device=q.device)
    elif _tensor("lse", lse, _FP32, len(lse_shape)) != index or lse.shape != lse_shape:
        raise ValueError(f"lse must be {list(lse_shape)} on q's device")
    return out, lse


def _workspace(t, index):
    """(address, bytes) of a workspace."""
    if not _is_tensor(t) or t.get_device() != index or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous buffer on q's device")
    return t.data_ptr(), t.numel() * t.element_size()


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
    index = _tensor("past_lens", past_lens, _INT32, 1)
    B = past_lens.shape[0]
    new = _ints("new_lens", new_lens, B, index)
    table, width = _table(block_table, B, index)
    if not _is_tensor(free_pages) or free_pages.dim() != 1:
        raise TypeError("free_pages must be an int32 tensor [num_free]")
    num_free = free_pages.shape[0]
    free = _ints("free_pages", free_pages, num_free, index)
    frange = _ints("free_range", free_range, 2, index)
    T = int(num_tokens)
    if T < 0:
        raise ValueError("num_tokens must not be negative")
    if cu_new is None or total_lens is None or positions is None or slot_map is None or free_range_out is None:
        def new_ints(t, n):
            return torch.empty(n, dtype=_INT32, device=past_lens.device) if t is None else t
        cu_new, total_lens = new_ints(cu_new, B + 1), new_ints(total_lens, B)
        positions, slot_map = new_ints(positions, T), new_ints(slot_map, T)
        free_range_out = new_ints(free_range_out, 2)
    _call(_lib.get().attn_page_plan, "attn_page_plan", index, past_lens.data_ptr(), new, table, free, frange,
          _ints("cu_new", cu_new, B + 1, index), _ints("total_lens", total_lens, B, index),
          _ints("positions", positions, T, index), _ints("slot_map", slot_map, T, index),
          _ints("free_range_out", free_range_out, 2, index), B, width, num_free, int(page_size), T)
    return cu_new, total_lens, positions, slot_map, free_range_out


def attn_rope_append_paged(packed_qkv, cos, sin, positions, slot_map, k_pages, v_pages, Hq: int, Hkv: int,
                           layout: int = LAYOUT_BHSD, q_out=None):
    """``attn_rope_append`` for a ragged batch and a paged cache (``attn_rope_append_paged``).

    packed_qkv [T, (Hq + 2*Hkv) * d] bf16; cos, sin [max_pos, d/2] fp32; positions and slot_map
    [T] int32 as from attn_page_plan; k_pages, v_pages [N, Hkv, P, d] bf16 ([N, P, Hkv, d] for
    LAYOUT_BSHD), updated in place.  Returns q [T, Hq, d]; rows of tokens with a negative slot
    are not written (a new ``q_out`` is zero-filled).
    """
    index = _tensor("packed_qkv", packed_qkv, _BF16, 2)
    T, width = packed_qkv.shape
    cache, pages_hkv, d = _pages(k_pages, v_pages, layout, index)
    if pages_hkv != Hkv or Hq <= 0 or width != (Hq + 2 * Hkv) * d:
        raise ValueError("packed_qkv's last dim must be (Hq + 2*Hkv) * d of pages with Hkv heads")
    if _tensor("cos", cos, _FP32, 2) != index or _tensor("sin", sin, _FP32, 2) != index or cos.shape != sin.shape \
            or cos.shape[1] != d // 2:
        raise ValueError("cos and sin must both be [max_pos, d/2] on packed_qkv's device")
    pos, slot = _ints("positions", positions, T, index), _ints("slot_map", slot_map, T, index)
    if q_out is None:
        q_out = torch.zeros((T, Hq, d), dtype=_BF16, device=packed_qkv.device)
    elif _tensor("q_out", q_out, _BF16, 3) != index or q_out.shape != (T, Hq, d):
        raise ValueError(f"q_out must be {(T, Hq, d)} on packed_qkv's device")
    _call(_lib.get().attn_rope_append_paged, "attn_rope_append_paged", index, packed_qkv.data_ptr(), cos.data_ptr(),
          sin.data_ptr(), cos.shape[0], pos, slot, q_out.data_ptr(), cache, T, Hq, Hkv, d)
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
    index = _tensor("q", q, _BF16, 3)
    T, Hq, d = q.shape
    if not _is_tensor(seqlens_k) or seqlens_k.dim() != 1:
        raise TypeError("seqlens_k must be an int32 tensor [B]")
    B = seqlens_k.shape[0]
    lens, cu = _ints("seqlens_k", seqlens_k, B, index), _ints("cu_q", cu_q, B + 1, index)
    cache, Hkv, dk = _pages(k_pages, v_pages, layout, index, *_table(block_table, B, index))
    if dk != d:
        raise ValueError(f"head_dim of q ({d}) and of the pages ({dk}) differ")
    out, lse = _outputs(q, (Hq, T), out, lse, return_lse, index)
    if workspace is None:
        workspace = fwd_paged_workspace(q, k_pages, layout)
    ws, ws_bytes = _workspace(workspace, index)
    _call(_lib.get().attn_fwd_paged, "attn_fwd_paged", index, q.data_ptr(), cache, cu, lens,
          out.data_ptr(), None if lse is None else lse.data_ptr(), B, T, Hq, Hkv, d, float(scale),
          int(causal), ws, ws_bytes)
    return out, lse


def attn_decode_splitkv_paged(q, k_pages, v_pages, seqlens_k, block_table, causal: int = CAUSAL_BOTTOM_RIGHT,
                              scale: float = 0.0, layout: int = LAYOUT_BHSD, workspace=None, out=None, lse=None,
                              return_lse: bool = True):
    """Split-KV decode over a paged cache (``attn_decode_splitkv_paged``).

    q [B, Sq, Hq, d] bf16 (token-major, as attn_rope_append_paged writes it); pages, lengths and
    table as for attn_fwd_paged.  Returns (o [B, Sq, Hq, d], lse [B, Hq, Sq] fp32).
    """
    index = _tensor("q", q, _BF16, 4)
    B, Sq, Hq, d = q.shape
    lens = _ints("seqlens_k", seqlens_k, B, index)
    cache, Hkv, dk = _pages(k_pages, v_pages, layout, index, *_table(block_table, B, index))
    if dk != d:
        raise ValueError(f"head_dim of q ({d}) and of the pages ({dk}) differ")
    out, lse = _outputs(q, (B, Hq, Sq), out, lse, return_lse, index)
    if workspace is None:
        workspace = decode_paged_workspace(q, k_pages, layout)
    ws, ws_bytes = _workspace(workspace, index)
    _call(_lib.get().attn_decode_splitkv_paged, "attn_decode_splitkv_paged", index, q.data_ptr(),
          cache, lens, out.data_ptr(), None if lse is None else lse.data_ptr(), B, Hq, Hkv, Sq, d,
          float(scale), int(causal), ws, ws_bytes)
    return out, lse

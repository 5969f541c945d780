"""Refusals of the paged cache's entry points on the host (no GPU), and the plain plan."""
import ctypes
import os
import re

import pytest
import torch

from scaled_dot_product_fa2_b200 import _lib, build, paged
from tests import paged_ref

P = 1 << 20  # a fake, well-aligned device address: every call here fails before it is used
NULL, SHAPE, GQA, HEADDIM, ALIGN, CAUSAL, WORKSPACE, SCALE, PAGE = 1, 2, 3, 4, 5, 6, 7, 11, 14


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.get()


def cache(**kw):
    c = _lib.PagedCache(P, P, P, 0, 100, 16, 8, 0)
    for name, value in kw.items():
        setattr(c, name, value)
    return ctypes.byref(c)


def plan(lib, past=P, new=P, table=P, free=P, rng=P, cu=P, total=P, pos=P, slot=P, out=P, B=3, max_pages=8,
         num_free=10, page=16, T=20):
    return lib.attn_page_plan(past, new, table, free, rng, cu, total, pos, slot, out, B, max_pages, num_free, page,
                              T, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), SHAPE), (dict(max_pages=-1), SHAPE), (dict(num_free=-1), SHAPE), (dict(T=-1), SHAPE),
    (dict(B=16385), SHAPE), (dict(T=(1 << 30) + 1), SHAPE), (dict(max_pages=(1 << 26) + 1), SHAPE),
    (dict(page=8), PAGE), (dict(page=24), PAGE), (dict(page=512), PAGE), (dict(page=0), PAGE),
    (dict(past=None), NULL), (dict(new=None), NULL), (dict(table=None), NULL), (dict(free=None), NULL),
    (dict(rng=None), NULL), (dict(cu=None), NULL), (dict(total=None), NULL), (dict(pos=None), NULL),
    (dict(slot=None), NULL), (dict(out=None), NULL),
    (dict(past=P + 2), ALIGN), (dict(slot=P + 1), ALIGN), (dict(table=P + 3), ALIGN), (dict(out=P + 2), ALIGN),
])
def test_plan_rejects_bad_arguments_on_host(lib, kw, status):
    assert plan(lib, **kw) == status


def append(lib, packed=P, cos=P, sin=P, max_pos=64, pos=P, slot=P, q=P, c=None, T=4, Hq=4, Hkv=2, d=64):
    return lib.attn_rope_append_paged(packed, cos, sin, max_pos, pos, slot, q, c if c is not None else cache(), T, Hq,
                                      Hkv, d, None)


def fwd(lib, q=P, c=None, cu=P, lens=P, o=P, lse=P, B=2, T=8, Hq=4, Hkv=2, d=64, scale=0.0, causal=2, ws=P, n=None):
    if n is None:
        n = lib.attn_fwd_paged_workspace_size(8, 4, 2, 64)
    return lib.attn_fwd_paged(q, c if c is not None else cache(), cu, lens, o, lse, B, T, Hq, Hkv, d, scale, causal,
                              ws, n, None)


def decode(lib, q=P, c=None, lens=P, o=P, lse=P, B=2, Hq=4, Hkv=2, Sq=1, d=64, scale=0.0, causal=2, ws=P, n=None):
    if n is None:
        n = lib.attn_decode_paged_workspace_size(2, 4, 2, 1, 64)
    return lib.attn_decode_splitkv_paged(q, c if c is not None else cache(), lens, o, lse, B, Hq, Hkv, Sq, d, scale,
                                         causal, ws, n, None)


@pytest.mark.parametrize("call", [append, fwd, decode])
@pytest.mark.parametrize("kw,status", [
    (dict(Hq=0), SHAPE), (dict(Hkv=0), SHAPE), (dict(Hq=3), GQA), (dict(d=96), HEADDIM), (dict(q=None), NULL),
    (dict(q=P + 8), ALIGN),
    (dict(c=dict(num_pages=-1)), SHAPE), (dict(c=dict(layout=2)), SHAPE), (dict(c=dict(page_size=48)), PAGE),
    (dict(c=dict(page_size=8)), PAGE), (dict(c=dict(page_size=512)), PAGE),
    (dict(c=dict(num_pages=(1 << 27) + 1)), SHAPE),
    (dict(c=dict(page_stride=2 * 16 * 64 - 8)), PAGE), (dict(c=dict(page_stride=2 * 16 * 64 + 4)), PAGE),
    (dict(c=dict(page_stride=1 << 38)), SHAPE),
    (dict(c=dict(k_pages=None)), NULL), (dict(c=dict(v_pages=None)), NULL), (dict(c=dict(v_pages=P + 8)), ALIGN),
])
def test_paged_calls_reject_bad_arguments_on_host(lib, call, kw, status):
    kw = dict(kw)
    if "c" in kw:
        kw["c"] = cache(**kw["c"])
    assert call(lib, **kw) == status


@pytest.mark.parametrize("call", [fwd, decode])
@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), SHAPE), (dict(lens=None), NULL), (dict(lens=P + 2), ALIGN), (dict(o=None), NULL),
    (dict(o=P + 4), ALIGN), (dict(lse=P + 2), ALIGN), (dict(causal=3), CAUSAL), (dict(scale=-1.0), SCALE),
    (dict(scale=float("nan")), SCALE), (dict(scale=float("inf")), SCALE),
    (dict(ws=None), WORKSPACE), (dict(ws=P + 8), WORKSPACE), (dict(n=0), WORKSPACE),
    (dict(c=dict(max_pages=-1)), SHAPE), (dict(c=dict(max_pages=(1 << 26) + 1)), SHAPE),
    (dict(c=dict(block_table=None)), NULL), (dict(c=dict(block_table=P + 2)), ALIGN),
])
def test_paged_attention_rejects_bad_arguments_on_host(lib, call, kw, status):
    kw = dict(kw)
    if "c" in kw:
        kw["c"] = cache(**kw["c"])
    assert call(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SHAPE), (dict(max_pos=0), SHAPE), (dict(packed=None), NULL), (dict(cos=None), NULL),
    (dict(pos=None), NULL), (dict(slot=None), NULL), (dict(packed=P + 8), ALIGN), (dict(sin=P + 4), ALIGN),
    (dict(pos=P + 1), ALIGN),
])
def test_paged_append_rejects_bad_arguments_on_host(lib, kw, status):
    assert append(lib, **kw) == status


def test_fwd_rejects_bad_row_offsets_on_host(lib):
    assert fwd(lib, cu=None) == NULL
    assert fwd(lib, cu=P + 2) == ALIGN
    assert fwd(lib, T=-1) == SHAPE


def test_packed_cache_has_the_layout_of_the_struct():
    c = _lib.PagedCache(1, 2, 3, 4, 5, 6, 7, 1)
    assert _lib.pack_paged_cache(1, 2, 3, 4, 5, 6, 7, 1) == bytes(c)


def test_null_cache_is_refused(lib):
    assert append(lib, c=ctypes.POINTER(_lib.PagedCache)()) == NULL
    assert fwd(lib, c=ctypes.POINTER(_lib.PagedCache)()) == NULL
    assert decode(lib, c=ctypes.POINTER(_lib.PagedCache)()) == NULL


def test_empty_batches_need_no_pointers(lib):
    assert fwd(lib, B=0, q=None, o=None, cu=None, lens=None, ws=None, n=0) == 0
    assert fwd(lib, T=0, q=None, o=None, cu=None, lens=None, ws=None, n=0) == 0
    assert decode(lib, B=0, q=None, o=None, lens=None, ws=None, n=0) == 0
    assert decode(lib, Sq=0, q=None, o=None, lens=None, ws=None, n=0) == 0
    assert append(lib, T=0, packed=None, cos=None, sin=None, pos=None, slot=None, q=None) == 0


def test_workspace_sizes_of_unsupported_shapes_are_zero(lib):
    assert lib.attn_fwd_paged_workspace_size(8, 4, 3, 64) == 0
    assert lib.attn_fwd_paged_workspace_size(8, 4, 2, 96) == 0
    assert lib.attn_fwd_paged_workspace_size(-1, 4, 2, 64) == 0
    assert lib.attn_decode_paged_workspace_size(2, 4, 3, 1, 64) == 0
    assert lib.attn_decode_paged_workspace_size(2, 4, 2, -1, 64) == 0
    assert lib.attn_fwd_paged_workspace_size(8, 4, 2, 64) > 0
    assert lib.attn_decode_paged_workspace_size(2, 4, 2, 1, 64) > 0


def test_status_string_of_the_page_error(lib):
    assert b"page" in lib.attn_status_string(PAGE)


def test_plain_plan_by_hand():
    # page 4: request 0 holds 3 keys and brings 2 (one new page), request 1 starts with 9 (three
    # pages, one too many), request 2 brings one token into its page's last row
    out, refused = paged_ref.plan([3, 0, 7], [2, 9, 1], [[5, -1], [-1] * 2, [6, 8]], [1, 9, 2, 3, 4], [1, 4], 4, 14,
                                  4)
    assert refused
    assert out[0] == [[5, 9], [-1, -1], [6, 8]]
    assert out[1] == [0, 2, 11, 12]
    assert out[2] == [5, 0, 8]
    assert out[3] == [3, 4] + list(range(9)) + [7, -1, -1]
    assert out[4] == [23, 36] + [-1] * 9 + [35, -1, -1]
    assert out[5] == [2, 4]


def test_warps_of_the_paged_kernels_meet_as_whole_warps():
    """A piece's entries are given back by the warp that read them, all of its lanes: which lanes happen to be
    active after a spin-wait says nothing about the others."""
    csrc = os.path.join(os.path.dirname(build.__file__), "csrc")
    for name in ("paged.cuh", "paged_decode.cuh", "paged_fwd.cuh", "page_plan.cuh", "piece_steps.h"):
        with open(os.path.join(csrc, name)) as f:
            assert "__activemask" not in f.read(), name


def test_programmatic_dependents_read_with_ordinary_loads():
    """A kernel whose blocks are resident before the grid before it ends reads what that grid writes (lengths,
    tables, slots, q) with ordinary loads: a non-coherent one may be answered from before the wait."""
    csrc = os.path.join(os.path.dirname(build.__file__), "csrc")
    for name in ("page_plan.cuh", "paged.cuh", "paged_decode.cuh", "paged_fwd.cuh"):
        with open(os.path.join(csrc, name)) as f:
            code = "\n".join(line.split("//")[0] for line in f.read().splitlines())
        assert "__ldg" not in code and ".nc" not in code, name
    with open(os.path.join(csrc, "decode.cuh")) as f:
        assert not re.search(r"__ldg\((p\.)?seqlens", f.read())
    with open(os.path.join(csrc, "rope.cuh")) as f:
        assert not re.search(r"__ldg\((p\.(slots|positions)|src|cr|sr)", f.read())


@pytest.mark.parametrize("layout", [0, 1])
def test_pools_whose_pages_overlap_are_refused(layout):
    """One page's memory for all of them (a stride of 0) is no pool: the C call takes 0 for dense pages."""
    one = torch.zeros((1, 2, 16, 64) if layout == 0 else (1, 16, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        paged._pages(one.expand(5, -1, -1, -1), one.expand(5, -1, -1, -1), layout, -1)
    both = torch.zeros((5, 2, *one.shape[1:]), dtype=torch.bfloat16)
    for k, v in ((one, one), (both[:, 0], both[:, 1]), (both[:1, 0], both[:1, 1]), (both[:, 0].clone(), both[:, 1].clone())):
        packed, Hkv, d = paged._pages(k, v, layout, -1)
        assert (Hkv, d) == (2, 64)

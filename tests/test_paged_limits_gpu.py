"""Limits of the paged entry points that a plain batch does not come near."""
import pytest
import torch

from scaled_dot_product_fa2_b200 import _lib, inputs
from tests import paged_ref
from tests.paged_ref import BHSD, BSHD, TL, Batch, check

pytestmark = pytest.mark.gpu

PAGE = 14


@pytest.fixture(scope="module")
def sdpa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from scaled_dot_product_fa2_b200 import build
    build.build()
    import scaled_dot_product_fa2_b200 as m
    return m


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("lens,Sq", [([5000, 300, 3, 1, 0], 3), ([9000], 1), ([700, 20], 70)])
def test_top_left_decode_reads_the_keys_that_its_tokens_see(sdpa, lens, Sq):
    """Token i sees keys 0 .. i: table entries behind the last token's key are not looked at."""
    page = 16
    bt = Batch([(L, Sq) for L in lens], 8, 2, 128, page, BHSD, seed=Sq)
    bt.table[:, paged_ref.pages_of(Sq, page):] = paged_ref.NOT_AN_ENTRY
    B = len(lens)
    o, lse = sdpa.attn_decode_splitkv_paged(bt.q.view(B, Sq, 8, 128), bt.k, bt.v, bt.seqlens, bt.table, causal=TL)
    sdpa.check_device_error()
    check(o.view(B * Sq, 8, 128), lse.transpose(0, 1).reshape(8, B * Sq), bt.reference(TL))


def test_top_left_decode_reports_lengths_out_of_range(sdpa):
    bt = Batch([(300, 2), (40, 2)], 8, 2, 128, 16, BHSD, seed=1)
    for lens in ([bt.table.shape[1] * 16 + 1, 40], [300, -1]):
        sdpa.attn_decode_splitkv_paged(bt.q.view(2, 2, 8, 128), bt.k, bt.v, ints(lens), bt.table, causal=TL)
        with pytest.raises(_lib.AttnError) as e:
            sdpa.check_device_error()
        assert e.value.status == 13
    sdpa.check_device_error()


def test_plan_of_the_largest_number_of_tokens(sdpa):
    """T = 2^30, its limit: a request whose tokens end behind the buffers is refused there as anywhere."""
    T, page = 1 << 30, 256
    free_mem, _ = torch.cuda.mem_get_info()
    if free_mem < 12 << 30:
        pytest.skip("two buffers of 4 GB")
    pages = T // page
    table = torch.full((2, pages), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(pages + 3, dtype=torch.int32, device="cuda").flip(0).contiguous()
    cu, total, pos, slot, rng = sdpa.attn_page_plan(ints([0, 5]), ints([T, 300]), table, free, ints([0, pages + 3]),
                                                    page, T)
    with pytest.raises(_lib.AttnError) as e:
        sdpa.check_device_error()
    assert e.value.status == PAGE
    assert cu.tolist() == [0, T, T] and total.tolist() == [T, 5] and rng.tolist() == [pages, pages + 3]
    assert (table[1] == -1).all() and torch.equal(table[0], free[:pages])
    at = torch.tensor([0, 255, 256, T // 2 + 77, T - 257, T - 1], device="cuda")
    assert torch.equal(pos[at].long(), at)
    assert torch.equal(slot[at].long(), free[at // page].long() * page + at % page)
    sdpa.check_device_error()


@pytest.mark.parametrize("layout", [BHSD, BSHD])
def test_pools_of_more_elements_than_32_bits_count(sdpa, layout):
    """Keys appended to the last pages of two pools of 4.6 * 10^9 elements, and read from there."""
    Hq, Hkv, d, page, N = 8, 8, 128, 64, 70000
    free_mem, _ = torch.cuda.mem_get_info()
    if free_mem < 24 << 30:
        pytest.skip("two pools of 9 GB")
    shape = (N, Hkv, page, d) if layout == BHSD else (N, page, Hkv, d)
    k, v = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gen = torch.Generator(device="cuda").manual_seed(layout)
    L, n = 300, 300
    free = torch.tensor([N - 1, 3, N - 2, 40000, 65536, 32768, N - 7], dtype=torch.int32, device="cuda")
    table = torch.zeros((1, 6), dtype=torch.int32, device="cuda")
    cos, sin = (t.cuda() for t in inputs.rope_tables(400, d))
    packed = torch.randn((n, (Hq + 2 * Hkv) * d), generator=gen, device="cuda").bfloat16()
    cu, lens, pos, slot, _ = sdpa.attn_page_plan(ints([0]), ints([n]), table, free, ints([0, 7]), page, n)
    q = sdpa.attn_rope_append_paged(packed, cos, sin, pos, slot, k, v, Hq, Hkv, layout=layout)
    o, lse = sdpa.attn_fwd_paged(q, k, v, cu, lens, table, layout=layout)
    od, lsed = sdpa.attn_decode_splitkv_paged(q[-1:].view(1, 1, Hq, d), k, v, lens, table, layout=layout)
    sdpa.check_device_error()
    x = packed.double().view(n, Hq + 2 * Hkv, d)
    a, b = x[:, :Hq + Hkv, :d // 2], x[:, :Hq + Hkv, d // 2:]
    c, s = cos[:n, None].double(), sin[:n, None].double()
    rot = torch.cat([a * c - b * s, b * c + a * s], -1)
    pair = (a.abs() + b.abs()).repeat(1, 1, 2)
    bound = paged_ref.EPS_BF16 * rot.abs() + 2.0 ** -22 * pair  # (see the append's own test)
    rows = k[table[0, :5].long()]
    rows = (rows.transpose(1, 2) if layout == BHSD else rows).reshape(-1, Hkv, d)[:n]
    assert ((rows.double() - rot[:, Hq:]).abs() <= bound[:, Hq:]).all()
    bt = Batch([(L, n)], Hq, Hkv, d, page, layout)
    bt.q_host, bt.k_seq, bt.v_seq = q.cpu(), [rows.cpu()], [packed.cpu().view(n, -1, d)[:, Hq + Hkv:]]
    check(o, lse, bt.reference(paged_ref.BR))
    bt = Batch([(L, 1)], Hq, Hkv, d, page, layout)
    bt.q_host, bt.k_seq, bt.v_seq = q[-1:].cpu(), [rows.cpu()], [packed.cpu().view(n, -1, d)[:, Hq + Hkv:]]
    check(od.view(1, Hq, d), lsed.view(1, Hq).transpose(0, 1).contiguous(), bt.reference(paged_ref.BR))


@pytest.mark.parametrize("L,Sq,d,page", [(131072, 1, 128, 16), (100003, 3, 64, 64), (32769, 1, 128, 128)])
def test_decode_of_one_very_long_sequence(sdpa, L, Sq, d, page):
    bt = Batch([(L, Sq), (77, Sq)], 8, 2, d, page, BSHD, seed=d)
    o, lse = sdpa.attn_decode_splitkv_paged(bt.q.view(2, Sq, 8, d), bt.k, bt.v, bt.seqlens, bt.table, layout=BSHD)
    sdpa.check_device_error()
    check(o.view(2 * Sq, 8, d), lse.transpose(0, 1).reshape(8, 2 * Sq), bt.reference(paged_ref.BR))
    o, lse = sdpa.attn_fwd_paged(bt.q, bt.k, bt.v, bt.cu, bt.seqlens, bt.table, layout=BSHD)
    sdpa.check_device_error()
    check(o, lse, bt.reference(paged_ref.BR))

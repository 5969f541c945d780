"""Limits of the paged entry points that a plain batch does not come near."""
import pytest
import torch

from scaled_dot_product_fa2_b200 import _lib
from tests import paged_ref
from tests.paged_ref import BHSD, TL, Batch, check

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

"""The paged forward's thin units (chunks with rows in one tile, whose key tiles the two MMA issuers take in
turn) on the GPU, element by element against 64 bits, many calls one after the other."""
import random

import pytest
import torch

from tests.paged_ref import BHSD, BR, BSHD, Batch, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sdpa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from scaled_dot_product_fa2_b200 import build
    build.build()
    import scaled_dot_product_fa2_b200 as m
    return m


@pytest.mark.parametrize("d,page,layout", [(128, 16, BSHD), (128, 128, BHSD), (64, 32, BHSD)])
def test_thin_units_in_a_row_over_large_caches(sdpa, d, page, layout):
    """Copies of pages far apart land in any order; caches that do not fit the L2 together keep them slow.  Thin
    units of every parity of key tiles, alone, cut, and with pairs behind and before them."""
    rng = random.Random(d + page)
    sets = []
    for i in range(2):
        seqs = [(rng.randrange(4000, 8000) * 128 // d, rng.choice((5, 9, 17, 31, 32))) for _ in range(20)]
        seqs += [(3000, 80), (129 * 3, 9), (640, 640), (5000, 9), (100, 20)]
        bt = Batch(seqs, 8, 2, d, page, layout, seed=50 + i)
        ws = sdpa.fwd_paged_workspace(bt.q, bt.k, layout)
        args = dict(q=bt.q, k_pages=bt.k, v_pages=bt.v, cu_q=bt.cu, seqlens_k=bt.seqlens, block_table=bt.table,
                    layout=layout, workspace=ws)
        first = sdpa.attn_fwd_paged(**args)
        check(*first, bt.reference(BR), f"set {i}")
        sets.append((args, first))
    same = torch.ones((), dtype=torch.bool, device="cuda")
    for i in range(200):
        args, (o0, lse0) = sets[i % 2]
        o, lse = sdpa.attn_fwd_paged(**args)
        same &= (o == o0).all() & (lse == lse0).all()
    assert same.item()
    sdpa.check_device_error()


@pytest.mark.parametrize("n", [5, 9, 31, 32])
@pytest.mark.parametrize("tiles", [1, 2, 3, 4, 5, 6, 7, 11, 12])
def test_thin_units_of_every_length(sdpa, n, tiles):
    for L in (tiles * 128 - 127, tiles * 128):
        if L < n:
            continue
        bt = Batch([(L, n)], 8, 2, 128, 64, BHSD, seed=tiles)
        check(*sdpa.attn_fwd_paged(bt.q, bt.k, bt.v, bt.cu, bt.seqlens, bt.table), bt.reference(BR), f"L={L}")
    sdpa.check_device_error()

"""The paged KV cache's operators on the GPU against plain implementations (``paged_ref``): the page
plan exactly, the append against the 64-bit rotation, the attentions element by element within the
bound that ``Batch.reference`` derives."""
import random

import pytest
import torch

from scaled_dot_product_fa2_b200 import _lib, inputs
from tests import paged_ref
from tests.paged_ref import BHSD, BR, BSHD, NONE, TL, Batch, check

pytestmark = pytest.mark.gpu

SEQLEN, PAGE = 13, 14


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


def reported(sdpa, status):
    with pytest.raises(_lib.AttnError) as e:
        sdpa.check_device_error()
    assert e.value.status == status
    sdpa.check_device_error()


# ------------------------------------------------------------------------------- plan
def plan_case(past, new, page, extra_free=3, pad=0, max_pages=None, skip=1, seed=0, short=None):
    rng = random.Random(seed)
    if max_pages is None:
        max_pages = max([paged_ref.pages_of(max(p, 0) + max(n, 0), page) for p, n in zip(past, new)] + [1])
    held = [paged_ref.pages_of(max(p, 0), page) for p in past]
    need = sum(paged_ref.pages_of(max(p, 0) + max(n, 0), page) - h for p, n, h in zip(past, new, held))
    free = need + extra_free if short is None else short
    ids = rng.sample(range(sum(held) + free + 5), sum(held) + free)
    table = []
    for h in held:
        row = [ids.pop() for _ in range(min(h, max_pages))]
        table.append(row + [-7] * (max_pages - len(row)))
    T = sum(max(n, 0) for n in new) + pad
    return dict(past=past, new=new, table=table, free=[-1] * skip + ids, rng=[skip, skip + free], page=page, T=T,
                max_pages=max_pages)


def run_plan(sdpa, c, **kw):
    B = len(c["past"])
    table = ints(c["table"]).reshape(B, c["max_pages"])
    out = sdpa.attn_page_plan(ints(c["past"]), ints(c["new"]), table, ints(c["free"]), ints(c["rng"]), c["page"],
                              c["T"], **kw)
    return (table, *out)


def check_plan(sdpa, c, **kw):
    got = run_plan(sdpa, c, **kw)
    want, refused = paged_ref.plan(c["past"], c["new"], c["table"], c["free"], c["rng"], c["page"], c["T"],
                                   c["max_pages"])
    for name, g, w in zip(("table", "cu_new", "total_lens", "positions", "slot_map", "free_range"), got, want):
        assert g.cpu().tolist() == w, name
    if refused:
        reported(sdpa, PAGE)
    else:
        sdpa.check_device_error()


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("past,new", [
    ([0], [1]), ([15], [1]), ([16], [1]), ([17], [0]), ([0], [0]),
    ([0, 5, 256, 1000], [300, 0, 1, 17]),
    ([255] * 9, [1, 2] * 4 + [258]),
])
def test_plan_matches_the_plain_one(sdpa, page, past, new):
    for pad in (0, 3):
        check_plan(sdpa, plan_case(past, new, page, pad=pad))


@pytest.mark.parametrize("B,hi,page", [(1, 9000, 16), (700, 3, 16), (513, 60, 32), (2500, 9, 16), (64, 2000, 128)])
def test_plan_of_large_batches(sdpa, B, hi, page):
    rng = random.Random(B)
    past = [rng.randrange(3000) for _ in range(B)]
    new = [rng.randrange(hi) for _ in range(B)]
    check_plan(sdpa, plan_case(past, new, page, pad=rng.randrange(9), seed=B))
    check_plan(sdpa, plan_case(past, new, page, seed=B, short=B // 3))


def test_plan_without_requests(sdpa):
    c = dict(past=[], new=[], table=[], free=[3, 4], rng=[0, 2], page=16, T=5, max_pages=4)
    check_plan(sdpa, c)


def test_plan_refuses_and_reports(sdpa):
    # pages run out; one that needs none is served all the same
    check_plan(sdpa, plan_case([0, 20, 3, 8, 40], [33, 12, 100, 1, 1], 16, short=4))
    # negative lengths, a sequence longer than the table
    check_plan(sdpa, plan_case([4, -3, 2, 9], [5, 4, -6, 5], 16))
    check_plan(sdpa, plan_case([4, 60, 2], [5, 10, 6], 16, max_pages=4))
    # more tokens than the batch's buffers hold
    c = plan_case([0, 10, 20, 5], [10, 30, 5, 0], 16)
    c["T"] = 30
    check_plan(sdpa, c)
    # an empty list, and one whose range runs out of it
    check_plan(sdpa, plan_case([0, 3], [2, 1], 16, short=0))
    c = plan_case([0, 3], [2, 1], 16)
    got = run_plan(sdpa, {**c, "rng": [-5, 1000]})
    reported(sdpa, PAGE)
    assert got[5].cpu().tolist()[1] == len(c["free"])


def test_plan_advances_in_place(sdpa):
    c = plan_case([15, 0, 31], [2, 40, 1], 16, pad=2)
    want, _ = paged_ref.plan(c["past"], c["new"], c["table"], c["free"], c["rng"], c["page"], c["T"], c["max_pages"])
    for into in ("past", "new"):
        past, new, rng = ints(c["past"]), ints(c["new"]), ints(c["rng"])
        table = ints(c["table"])
        out = sdpa.attn_page_plan(past, new, table, ints(c["free"]), rng, 16, c["T"],
                                  total_lens=past if into == "past" else new, free_range_out=rng)
        sdpa.check_device_error()
        assert (past if into == "past" else new).cpu().tolist() == want[2]
        assert rng.cpu().tolist() == want[5]
        assert out[3].cpu().tolist() == want[4]


def test_plan_in_place_of_a_large_batch(sdpa):
    # several thread blocks read the lengths that one of them overwrites
    rng = random.Random(5)
    past = [rng.randrange(500) for _ in range(900)]
    new = [rng.randrange(60) for _ in range(900)]
    c = plan_case(past, new, 16)
    want, _ = paged_ref.plan(c["past"], c["new"], c["table"], c["free"], c["rng"], c["page"], c["T"], c["max_pages"])
    for _ in range(5):
        dev, fr, table = ints(past), ints(c["rng"]), ints(c["table"])
        out = sdpa.attn_page_plan(dev, ints(new), table, ints(c["free"]), fr, 16, c["T"], total_lens=dev,
                                  free_range_out=fr)
        assert dev.cpu().tolist() == want[2] and fr.cpu().tolist() == want[5]
        assert out[2].cpu().tolist() == want[3] and out[3].cpu().tolist() == want[4]
        assert table.cpu().tolist() == want[0]
    sdpa.check_device_error()


def test_plan_into_unaligned_buffers(sdpa):
    c = plan_case([15, 0, 31], [2, 40, 1], 16, pad=3)
    buf = torch.full((2 * c["T"] + 3,), -9, dtype=torch.int32, device="cuda")
    check_plan(sdpa, c, positions=buf[1:1 + c["T"]], slot_map=buf[c["T"] + 2:2 * c["T"] + 2])
    assert buf[0].item() == -9 and buf[c["T"] + 1].item() == -9 and buf[-1].item() == -9


# ----------------------------------------------------------------------------- append
@pytest.mark.parametrize("layout", [BHSD, BSHD])
@pytest.mark.parametrize("T,Hq,Hkv,d,page", [(1, 1, 1, 64, 16), (9, 8, 2, 128, 16), (37, 6, 2, 64, 32),
                                             (130, 32, 8, 128, 64), (5, 40, 40, 64, 256)])
def test_append_matches_the_rotation(sdpa, T, Hq, Hkv, d, page, layout):
    gen = torch.Generator().manual_seed(T + d)
    N, max_pos = paged_ref.pages_of(T, page) + 3, 5000
    packed = torch.randn((T, (Hq + 2 * Hkv) * d), generator=gen).bfloat16()
    slots = torch.randperm(N * page, generator=gen)[:T].int()
    pos = torch.randint(0, max_pos, (T,), generator=gen).int()
    skipped = torch.arange(T) % 4 == 3
    slots[skipped] = -1
    pos[skipped] = -1
    cos, sin = inputs.rope_tables(max_pos, d)
    inner = (page, Hkv, d) if layout == BSHD else (Hkv, page, d)
    both = torch.randn((N, 2, *inner), generator=gen).bfloat16().cuda()
    before = both.clone()
    q = torch.full((T, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    sdpa.attn_rope_append_paged(packed.cuda(), cos.cuda(), sin.cuda(), pos.cuda(), slots.cuda(), both[:, 0],
                                both[:, 1], Hq, Hkv, layout=layout, q_out=q)
    sdpa.check_device_error()
    live = ~skipped
    x = packed[live].double().view(-1, Hq + 2 * Hkv, d)
    c, s = cos[pos[live].long()].double()[:, None], sin[pos[live].long()].double()[:, None]
    a, b = x[..., :d // 2], x[..., d // 2:]
    rot = torch.cat([a * c - b * s, b * c + a * s], -1)
    pair = (a.abs() + b.abs()).repeat(1, 1, 2)
    # products and sum in fp32 (2^-22 of the operands), one rounding to bf16
    bound = paged_ref.EPS_BF16 * rot.abs() + 2.0 ** -22 * pair

    def rows(pool):
        p = pool if layout == BSHD else pool.transpose(1, 2)
        return p.reshape(N * page, Hkv, d).cpu()

    where = slots[live].long()
    assert ((q.cpu()[live].double() - rot[:, :Hq]).abs() <= bound[:, :Hq]).all()
    assert (q.cpu()[skipped] == 7).all()
    k, v = rows(both[:, 0]), rows(both[:, 1])
    assert ((k[where].double() - rot[:, Hq:Hq + Hkv]).abs() <= bound[:, Hq:Hq + Hkv]).all()
    assert torch.equal(v[where], packed[live].view(-1, Hq + 2 * Hkv, d)[:, Hq + Hkv:])
    other = torch.ones(N * page, dtype=torch.bool)
    other[where] = False
    assert torch.equal(k[other], rows(before[:, 0])[other])
    assert torch.equal(v[other], rows(before[:, 1])[other])


def test_append_skips_and_reports_bad_places(sdpa):
    Hq, Hkv, d, page, N = 2, 1, 64, 16, 3
    packed = torch.randn((4, (Hq + 2 * Hkv) * d), device="cuda").bfloat16()
    cos, sin = (t.cuda() for t in inputs.rope_tables(10, d))
    for pos, slot, status in (([0, 10, 1, 2], [0, 1, 2, 3], SEQLEN), ([0, -1, 1, 2], [0, 1, 2, 3], SEQLEN),
                              ([0, 1, 2, 3], [0, N * page, 2, 3], PAGE), ([0, 1, 2, 3], [0, 2 ** 31 - 1, 2, 3], PAGE)):
        k = torch.zeros((N, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
        v = torch.zeros_like(k)
        q = sdpa.attn_rope_append_paged(packed, cos, sin, ints(pos), ints(slot), k, v, Hq, Hkv)
        reported(sdpa, status)
        assert (q[1] == 0).all() and (q[2] != 0).any()
        assert k.count_nonzero().item() == 3 * d and v.count_nonzero().item() == 3 * d


# ------------------------------------------------------------------------- attention
def run_fwd(sdpa, bt, causal, scale=0.0, **kw):
    o = torch.full((bt.T, bt.Hq, bt.d), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((bt.Hq, bt.T), float("nan"), dtype=torch.float32, device="cuda")
    sdpa.attn_fwd_paged(bt.q, bt.k, bt.v, bt.cu, bt.seqlens, bt.table, causal=causal, scale=scale, layout=bt.layout,
                        out=o, lse=lse, **kw)
    live = bt.cu_list[-1]
    assert torch.isnan(o[live:]).all() and torch.isnan(lse[:, live:]).all(), "rows behind the last sequence written"
    o[live:] = 0
    lse[:, live:] = -float("inf")
    return o, lse


def check_fwd(sdpa, bt, causal=BR, scale=0.0):
    got = run_fwd(sdpa, bt, causal, scale)
    sdpa.check_device_error()
    check(*got, bt.reference(causal, scale), f"fwd causal={causal}")


HEADS = [(8, 2, 64), (4, 4, 128), (6, 2, 128), (5, 5, 64), (8, 1, 128), (16, 2, 64), (20, 1, 64)]
RAGGED = [(0, 0), (1, 1), (17, 3), (300, 7), (129, 129), (64, 1), (0, 2), (3, 5), (128, 0), (256, 128), (400, 260)]


@pytest.mark.parametrize("layout", [BHSD, BSHD])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("Hq,Hkv,d", HEADS)
def test_fwd_ragged_batch(sdpa, Hq, Hkv, d, page, layout):
    bt = Batch(RAGGED, Hq, Hkv, d, page, layout, seed=Hq + page, pad=5)
    check_fwd(sdpa, bt)


@pytest.mark.parametrize("causal", [NONE, TL, BR])
@pytest.mark.parametrize("page", [32, 128])
def test_fwd_masks(sdpa, page, causal):
    bt = Batch(RAGGED, 8, 2, 128, page, seed=page, pad=1, interleaved=True)
    check_fwd(sdpa, bt, causal, scale=0.11)


@pytest.mark.parametrize("seqs,Hq,Hkv,d", [
    ([(5000, 1)], 32, 8, 128), ([(5000, 1)], 1, 1, 64), ([(4097, 130)], 8, 2, 128), ([(3001, 33)], 4, 4, 64),
    ([(2048, 2048)], 4, 2, 128), ([(1500, 1200), (9000, 1), (10, 10)], 8, 2, 128), ([(0, 700)], 2, 2, 64),
    ([(200, 700)], 2, 1, 64), ([(1, 1)], 1, 1, 128), ([(700, 3)], 160, 1, 64), ([(700, 200)], 132, 1, 128),
])
def test_fwd_long_and_lone_sequences(sdpa, seqs, Hq, Hkv, d):
    bt = Batch(seqs, Hq, Hkv, d, 64, BSHD, seed=len(seqs) + d, pad=2)
    check_fwd(sdpa, bt)


def test_fwd_of_many_single_tokens_beside_chunks(sdpa):
    rng = random.Random(3)
    seqs = [(rng.randrange(1, 900), 1) for _ in range(70)] + [(700, 300)] + [(rng.randrange(0, 300), 1)
                                                                             for _ in range(75)] + [(513, 64)]
    check_fwd(sdpa, Batch(seqs, 8, 2, 128, 16, BSHD, seed=1))


def run_decode(sdpa, bt, Sq, causal, scale=0.0, **kw):
    B = len(bt.lens)
    q = bt.q[:B * Sq].view(B, Sq, bt.Hq, bt.d)
    o = torch.full_like(q, float("nan"))
    lse = torch.full((B, bt.Hq, Sq), float("nan"), dtype=torch.float32, device="cuda")
    sdpa.attn_decode_splitkv_paged(q, bt.k, bt.v, bt.seqlens, bt.table, causal=causal, scale=scale, layout=bt.layout,
                                   out=o, lse=lse, **kw)
    return o.view(B * Sq, bt.Hq, bt.d), lse.transpose(0, 1).reshape(bt.Hq, B * Sq)


def check_decode(sdpa, lens, Sq, Hq, Hkv, d, page, layout=BHSD, causal=BR, seed=0, scale=0.0, **kw):
    bt = Batch([(L, Sq) for L in lens], Hq, Hkv, d, page, layout, seed=seed, **kw)
    got = run_decode(sdpa, bt, Sq, causal, scale)
    sdpa.check_device_error()
    check(*got, bt.reference(causal, scale), f"decode Sq={Sq} causal={causal}")


DECODE_LENS = [0, 1, 3, 64, 517, 65, 1000, 16]


@pytest.mark.parametrize("layout", [BHSD, BSHD])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("Hq,Hkv,d", HEADS)
def test_decode_matches_the_plain_one(sdpa, Hq, Hkv, d, page, layout):
    for Sq in (1, 4):
        check_decode(sdpa, DECODE_LENS, Sq, Hq, Hkv, d, page, layout, seed=page + Sq)


@pytest.mark.parametrize("causal", [NONE, TL, BR])
def test_decode_masks(sdpa, causal):
    check_decode(sdpa, DECODE_LENS, 3, 8, 2, 128, 32, causal=causal, seed=causal, scale=0.07, interleaved=True)


@pytest.mark.parametrize("lens,Sq,Hq,Hkv,d", [
    ([700], 1, 32, 8, 128), ([20000], 1, 4, 1, 128), ([1], 1, 1, 1, 64), ([3000, 1], 5, 2, 1, 64),
    ([100], 40, 2, 2, 64), ([4000] * 3, 2, 16, 16, 64), ([300], 7, 160, 1, 64),
])
def test_decode_sizes(sdpa, lens, Sq, Hq, Hkv, d):
    check_decode(sdpa, lens, Sq, Hq, Hkv, d, 16, BSHD, seed=d)


def test_decode_of_a_large_mixed_batch(sdpa):
    rng = random.Random(8)
    check_decode(sdpa, [int(2 ** rng.uniform(0, 11)) for _ in range(200)], 1, 8, 2, 128, 16, BSHD)
    check_decode(sdpa, [rng.randrange(0, 40) for _ in range(700)], 1, 4, 4, 64, 32)


def test_shared_pages_and_unused_entries(sdpa):
    # two sequences with one prefix in the same pages
    bt = Batch([(128, 1), (131, 1)], 8, 2, 128, 64, seed=4)
    bt.table[1, :2] = bt.table[0, :2]
    bt.k_seq[1] = torch.cat([bt.k_seq[0], bt.k_seq[1][128:]])
    bt.v_seq[1] = torch.cat([bt.v_seq[0], bt.v_seq[1][128:]])
    check(*run_decode(sdpa, bt, 1, BR), bt.reference(BR))
    check(*run_fwd(sdpa, bt, BR), bt.reference(BR))
    sdpa.check_device_error()


@pytest.mark.parametrize("entry", [-1, -(2 ** 31), 2 ** 31 - 1, "N"])
def test_a_bad_page_reads_as_zeros_and_is_reported(sdpa, entry):
    bt = Batch([(200, 3), (300, 3)], 8, 2, 128, 64, seed=5)
    bt.table[1, 2] = bt.N if entry == "N" else entry
    for seq in (bt.k_seq[1], bt.v_seq[1]):
        seq[128:192] = 0
    ref = bt.reference(BR)
    got = run_decode(sdpa, bt, 3, BR)
    reported(sdpa, PAGE)
    check(*got, ref)
    got = run_fwd(sdpa, bt, BR)
    reported(sdpa, PAGE)
    check(*got, ref)


def test_bad_lengths_are_clamped_and_reported(sdpa):
    bt = Batch([(200, 2), (128, 2), (64, 2)], 8, 2, 128, 64, seed=6)
    bt.table = bt.table[:, :4].contiguous()
    bt.table[1] = bt.table[0]
    cap = 4 * 64
    bt.k[bt.table[0, 3].long(), :, 8:] = 0  # every row up to the table's end is a number
    bt.v[bt.table[0, 3].long(), :, 8:] = 0
    zeros = torch.zeros((56, 2, 128), dtype=torch.bfloat16)
    bt.k_seq[1] = torch.cat([bt.k_seq[0], zeros])
    bt.v_seq[1] = torch.cat([bt.v_seq[0], zeros])
    bt.seqlens = ints([200, cap + 1, -5])
    bt.lens = [200, cap, 0]
    for run in (lambda: run_decode(sdpa, bt, 2, BR), lambda: run_fwd(sdpa, bt, BR)):
        got = run()
        reported(sdpa, SEQLEN)
        check(*got, bt.reference(BR))


def test_without_pages_every_row_is_empty(sdpa):
    k = torch.zeros((0, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.randn((3, 4, 64), device="cuda").bfloat16()
    table = torch.zeros((3, 0), dtype=torch.int32, device="cuda")
    o, lse = sdpa.attn_fwd_paged(q, k, k, ints([0, 1, 2, 3]), ints([0, 0, 0]), table)
    assert (o == 0).all() and (lse == -float("inf")).all()
    o, lse = sdpa.attn_decode_splitkv_paged(q.view(3, 1, 4, 64), k, k, ints([0, 0, 0]), table)
    assert (o == 0).all() and (lse == -float("inf")).all()
    sdpa.check_device_error()


def test_lse_is_optional(sdpa):
    bt = Batch([(200, 3), (70, 3)], 8, 2, 64, 16, seed=9)
    o, lse = sdpa.attn_fwd_paged(bt.q, bt.k, bt.v, bt.cu, bt.seqlens, bt.table, return_lse=False)
    assert lse is None
    o2, lse = sdpa.attn_decode_splitkv_paged(bt.q.view(2, 3, 8, 64), bt.k, bt.v, bt.seqlens, bt.table,
                                             return_lse=False)
    assert lse is None
    sdpa.check_device_error()
    ref = bt.reference(BR)
    check(o, ref[1], ref)
    check(o2.view(6, 8, 64), ref[1], ref)


def test_results_do_not_depend_on_the_run(sdpa):
    bt = Batch([(3000, 40), (900, 1), (700, 300)], 8, 2, 128, 16, seed=10)
    first = run_fwd(sdpa, bt, BR)
    dec = Batch([(L, 2) for L in (1, 5000, 40, 900)], 8, 2, 128, 16, seed=11)
    first_d = run_decode(sdpa, dec, 2, BR)
    for _ in range(5):
        for a, b in ((first, run_fwd(sdpa, bt, BR)), (first_d, run_decode(sdpa, dec, 2, BR))):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_wrapper_refusals(sdpa):
    bt = Batch([(40, 2), (20, 2)], 4, 2, 64, 16, seed=12)
    ok = dict(q=bt.q, k_pages=bt.k, v_pages=bt.v, cu_q=bt.cu, seqlens_k=bt.seqlens, block_table=bt.table)
    sdpa.attn_fwd_paged(**ok)
    for bad, err in ((dict(q=bt.q.float()), TypeError), (dict(k_pages=bt.k.float()), TypeError),
                     (dict(cu_q=bt.cu.long()), TypeError), (dict(cu_q=bt.cu[:2]), ValueError),
                     (dict(block_table=bt.table.long()), TypeError), (dict(block_table=bt.table[:1]), ValueError),
                     (dict(block_table=bt.table[:, ::2]), ValueError), (dict(v_pages=bt.v[:-1]), ValueError),
                     (dict(k_pages=bt.k.transpose(1, 2)), ValueError), (dict(q=bt.q.cpu()), ValueError),
                     (dict(k_pages=bt.k.cpu()), ValueError), (dict(seqlens_k=bt.seqlens.long()), TypeError),
                     (dict(out=torch.empty_like(bt.q)[:2]), ValueError),
                     (dict(workspace=torch.empty(0, dtype=torch.uint8, device="cuda")), _lib.AttnError),
                     (dict(layout=2), ValueError), (dict(causal=7), _lib.AttnError)):
        with pytest.raises(err):
            sdpa.attn_fwd_paged(**{**ok, **bad})
    sdpa.check_device_error()


# ----------------------------------------------------------------------- the whole step
class Server:
    """Sequences kept in a paged cache by the operators, and in plain 64-bit tensors beside them."""

    def __init__(self, sdpa, B, Hq, Hkv, d, page, layout, seed):
        self.m, self.B, self.Hq, self.Hkv, self.d, self.page, self.layout = sdpa, B, Hq, Hkv, d, page, layout
        self.gen = torch.Generator().manual_seed(seed)
        N = 60
        inner = (page, Hkv, d) if layout == BSHD else (Hkv, page, d)
        self.k = torch.full((N, *inner), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.v = self.k.clone()
        self.table = torch.full((B, 20), paged_ref.NOT_AN_ENTRY, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(N, generator=self.gen).int().cuda()
        self.range = ints([0, N])
        self.lens = ints([0] * B)
        self.cos, self.sin = (t.cuda() for t in inputs.rope_tables(400, d))
        self.bt = Batch([(0, 0)] * B, Hq, Hkv, d, page, layout)

    def tokens(self, T):
        return torch.randn((T, (self.Hq + 2 * self.Hkv) * self.d), generator=self.gen).bfloat16().cuda()

    def append(self, packed, new):
        T = packed.shape[0]
        cu, _, pos, slot, _ = self.m.attn_page_plan(self.lens, new, self.table, self.free, self.range, self.page, T,
                                                    total_lens=self.lens, free_range_out=self.range)
        q = self.m.attn_rope_append_paged(packed, self.cos, self.sin, pos, slot, self.k, self.v, self.Hq, self.Hkv,
                                          layout=self.layout)
        return q, cu

    def remember(self, packed, new, q):
        """The plain side: q, k, v rows of the step, rotated to their positions (k as the cache holds
        it: its rounding is the append's, tested above)."""
        bt, at = self.bt, 0
        past, bt.cu_list = list(bt.lens), [0]
        slots = []
        for b, n in enumerate(new):
            bt.lens[b] += n
            bt.cu_list.append(bt.cu_list[-1] + n)
            slots += [(b, past[b] + i) for i in range(n)]
        table = self.table.cpu()
        k = (self.k if self.layout == BSHD else self.k.transpose(1, 2)).cpu()
        x = packed.cpu().view(-1, self.Hq + 2 * self.Hkv, self.d)
        for t, (b, p) in enumerate(slots):
            row = k[table[b, p // self.page], p % self.page]
            bt.k_seq[b] = torch.cat([bt.k_seq[b], row[None]])
            bt.v_seq[b] = torch.cat([bt.v_seq[b], x[t, self.Hq + self.Hkv:][None]])
            pos = torch.tensor(float(p))
            c, s = self.cos[p].double().cpu(), self.sin[p].double().cpu()
            a, z = x[t, self.Hq:self.Hq + self.Hkv, :self.d // 2].double(), \
                x[t, self.Hq:self.Hq + self.Hkv, self.d // 2:].double()
            want = torch.cat([a * c - z * s, z * c + a * s], -1)
            assert (row.double() - want).abs().max() < 0.05, (pos, "k row in the wrong place")
        bt.new, bt.T, bt.q_host = list(new), packed.shape[0], q.cpu()

    def check(self, o, lse):
        check(o, lse, self.bt.reference(BR))


@pytest.mark.parametrize("Hq,Hkv,d,page,layout", [(8, 2, 128, 16, BHSD), (4, 4, 64, 32, BSHD)])
def test_prompts_then_chunks_then_decode_steps(sdpa, Hq, Hkv, d, page, layout):
    s = Server(sdpa, 4, Hq, Hkv, d, page, layout, seed=d)
    for new in ([37, 1, 130, 5], [1, 64, 0, 20], [1, 1, 1, 1]):
        pad = 3
        packed = s.tokens(sum(new) + pad)
        q, cu = s.append(packed, ints(new))
        o, lse = sdpa.attn_fwd_paged(q, s.k, s.v, cu, s.lens, s.table, layout=layout)
        sdpa.check_device_error()
        s.remember(packed, new, q)
        assert s.lens.cpu().tolist() == s.bt.lens
        lse[:, sum(new):] = -float("inf")
        s.check(o, lse)
    for _ in range(20):  # over a page border
        packed = s.tokens(4)
        q, _ = s.append(packed, ints([1] * 4))
        o, lse = sdpa.attn_decode_splitkv_paged(q.view(4, 1, Hq, d), s.k, s.v, s.lens, s.table, layout=layout)
        s.remember(packed, [1] * 4, q)
    sdpa.check_device_error()
    s.check(o.view(4, Hq, d), lse.view(4, Hq).transpose(0, 1).contiguous())
    used = sum(paged_ref.pages_of(L, page) for L in s.bt.lens)
    assert s.range.cpu().tolist() == [used, 60]


def test_a_captured_decode_step_replays(sdpa):
    """One step (plan, append, decode) captured once, replayed with new tokens; an eager chunk of
    other sequences runs between the replays on the same cache."""
    Hq, Hkv, d, page = 8, 2, 128, 16
    s = Server(sdpa, 3, Hq, Hkv, d, page, BHSD, seed=1)
    packed = s.tokens(60)
    q, cu = s.append(packed, ints([33, 20, 7]))
    s.remember(packed, [33, 20, 7], q)
    one = ints([1, 1, 1])
    static = torch.zeros((3, packed.shape[1]), dtype=torch.bfloat16, device="cuda")
    q0 = torch.zeros((3, 1, Hq, d), dtype=torch.bfloat16, device="cuda")
    ws = sdpa.decode_paged_workspace(q0, s.k)
    lens, table, rng = s.lens.clone(), s.table.clone(), s.range.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        q, _ = s.append(static, one)
        o, lse = sdpa.attn_decode_splitkv_paged(q.view(3, 1, Hq, d), s.k, s.v, s.lens, s.table, workspace=ws)
        return q, o, lse

    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    s.lens.copy_(lens)
    s.table.copy_(table)
    s.range.copy_(rng)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q, o, lse = step()
    for i in range(30):
        packed = s.tokens(3)
        static.copy_(packed)
        g.replay()
        torch.cuda.synchronize()
        s.remember(packed, [1, 1, 1], q)
        s.check(o.view(3, Hq, d), lse.view(3, Hq).transpose(0, 1).contiguous())
        if i == 12:
            new = [0, 40, 3]
            packed = s.tokens(43)
            qe, cu = s.append(packed, ints(new))
            oe, le = sdpa.attn_fwd_paged(qe, s.k, s.v, cu, s.lens, s.table)
            s.remember(packed, new, qe)
            s.check(oe, le)
    sdpa.check_device_error()


def test_two_streams_with_a_workspace_each(sdpa):
    bts = [Batch([(900 + 100 * i, 20), (3000, 1), (60, 60)], 8, 2, 128, 16, seed=20 + i) for i in range(2)]
    refs = [bt.reference(BR) for bt in bts]
    streams = [torch.cuda.Stream() for _ in bts]
    ws = [sdpa.fwd_paged_workspace(bt.q, bt.k) for bt in bts]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(sdpa.attn_fwd_paged(bts[i].q, bts[i].k, bts[i].v, bts[i].cu, bts[i].seqlens,
                                                   bts[i].table, workspace=ws[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in outs[i]:
            check(o, lse, refs[i])
    sdpa.check_device_error()


@pytest.mark.parametrize("page,d", [(64, 128), (16, 64)])
def test_many_decodes_in_a_row_over_large_caches(sdpa, page, d):
    """Back-to-back calls over caches that do not fit the L2 together: copies land in any order, and
    each call's first copies are in flight while the call before it ends."""
    B, Hq, Hkv, L = 8, 32, 8, 8192
    N, W = B * L // page, L // page
    gen = torch.Generator(device="cuda").manual_seed(page)
    sets = []
    for _ in range(3):
        k, v = (torch.randn((N, Hkv, page, d), generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        table = torch.randperm(N, generator=gen, device="cuda").int().view(B, W)
        q = torch.randn((B, 1, Hq, d), generator=gen, device="cuda", dtype=torch.bfloat16)
        sets.append((q, k, v, ints([L - 13 * i for i in range(B)]), table, sdpa.decode_paged_workspace(q, k)))
    first = []
    for q, k, v, lens, table, ws in sets:
        o, lse = sdpa.attn_decode_splitkv_paged(q, k, v, lens, table, workspace=ws)
        keys = k[table[3, :].long()].transpose(1, 2).reshape(-1, Hkv, d)[:lens[3].item()].double()
        s = torch.einsum("hgd,khd->hgk", q[3, 0].double().view(Hkv, Hq // Hkv, d), keys) / d ** 0.5
        assert (torch.logsumexp(s, -1).flatten() - lse[3, :, 0].double()).abs().max() < 1e-4
        first.append((o, lse))
    for i in range(600):
        q, k, v, lens, table, ws = sets[i % 3]
        o, lse = sdpa.attn_decode_splitkv_paged(q, k, v, lens, table, workspace=ws)
        if i % 50 >= 47:
            assert torch.equal(o, first[i % 3][0]) and torch.equal(lse, first[i % 3][1])
    sdpa.check_device_error()


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (4, 4, 64)])
def test_lengths_around_what_is_split(sdpa, Hq, Hkv, d):
    """Tables that hold no more than the keys that stay in one piece, and just more than that."""
    for L in (128, 255, 256, 257, 320, 384, 385, 513):
        lens = [L, 1, L - 1]
        check_decode(sdpa, lens, 1, Hq, Hkv, d, 64, seed=L)
        bt = Batch([(L, min(L, 70)), (L, 1), (L, L)], Hq, Hkv, d, 64, seed=L)
        check_fwd(sdpa, bt)
        exact = -(-L // 64)  # a table without a spare entry
        bt.table = bt.table[:, :exact].contiguous()
        check_fwd(sdpa, bt)


def test_fwd_of_more_sequences_than_threads(sdpa):
    rng = random.Random(21)
    seqs = [(rng.randrange(0, 90), rng.choice((0, 1, 1, 1, 5, 40))) for _ in range(900)]
    check_fwd(sdpa, Batch(seqs, 4, 2, 64, 32, seed=2, pad=3))
    check_fwd(sdpa, Batch([(3, 0)] * 500 + [(70, 33)] + [(9, 0)] * 300 + [(40, 1)] + [(0, 0)] * 90, 8, 1, 128, 16))


@pytest.mark.parametrize("n", [4, 5, 31, 32, 33, 63, 64, 65, 67, 68, 69, 128, 132, 133])
def test_fwd_around_the_borders_of_its_tiles(sdpa, n):
    # 4 heads per KV head: 32 tokens a tile, 64 a unit, 4 left over are the decode's work
    for L in (n, n + 300):
        check_fwd(sdpa, Batch([(L, n)], 8, 2, 128, 16, BSHD, seed=n))


@pytest.mark.parametrize("seqs,Hq,Hkv,d,causal", [
    ([(700, 700)] * 13, 8, 2, 128, BR),                           # 286 equal units in all: two each and a rest
    ([(1300, 1300)], 32, 8, 128, BR),                             # one prompt, units of every weight
    ([(1300, 1300)], 32, 8, 64, NONE),
    ([(900 - 37 * i, 300 - 13 * i) for i in range(20)] + [(0, 0), (5, 0), (0, 9)], 8, 2, 64, BR),
    ([(100 * i, 90 + i) for i in range(24)], 16, 2, 128, TL),     # ends in one tile, rows that see nothing
    ([(600, 16 * 24 * 2)], 128, 1, 64, BR),                       # a unit per thread that ranks them, and one more
    ([(600, 16 * 24 * 2 + 2)], 128, 1, 64, BR),
    ([(700, 379)] * 24 + [(300, 256)], 64, 8, 64, BR),            # 16 units a processor on 148, and more
    ([(700, 379)] * 24 + [(300, 290)], 64, 8, 64, BR),
    ([(400, 400)] * 3 + [(500 + 7 * i, 1) for i in range(30)], 32, 8, 128, BR),
])
def test_fwd_of_units_that_are_dealt_whole(sdpa, seqs, Hq, Hkv, d, causal):
    check_fwd(sdpa, Batch(seqs, Hq, Hkv, d, 64, BSHD, seed=len(seqs) + d, pad=1), causal)


def test_bad_row_offsets_are_clamped_and_reported(sdpa):
    bt = Batch([(200, 30), (100, 20), (50, 10)], 8, 2, 128, 64, seed=30)
    T = bt.T
    for cu, starts in (([0, 30, 50, T + 7], None), ([-4, 30, 50, T], None)):
        bt.cu = ints(cu)
        got = run_fwd(sdpa, bt, BR)
        reported(sdpa, SEQLEN)
        check(*got, bt.reference(BR))  # clamped to what it should have been
    bt.cu = ints([0, 30, 10, T])  # decreasing: no fault, no row outside the batch, and it is told
    o, lse = sdpa.attn_fwd_paged(bt.q, bt.k, bt.v, bt.cu, bt.seqlens, bt.table)
    reported(sdpa, SEQLEN)
    bt.cu = ints([2 ** 31 - 1, -(2 ** 31), 0, 2 ** 31 - 1])
    sdpa.attn_fwd_paged(bt.q, bt.k, bt.v, bt.cu, bt.seqlens, bt.table)
    reported(sdpa, SEQLEN)


def test_any_workspace_contents_do(sdpa):
    bt = Batch([(3000, 40), (900, 1), (700, 300)], 8, 2, 128, 16, seed=31)
    dec = Batch([(L, 2) for L in (1, 5000, 40, 900)], 8, 2, 128, 16, seed=32)
    ref, dec_ref = bt.reference(BR), dec.reference(BR)
    ws = sdpa.fwd_paged_workspace(bt.q, bt.k)
    dec_ws = sdpa.decode_paged_workspace(dec.q.view(4, 2, 8, 128), dec.k)
    for fill in (0, 255, 127):
        ws.fill_(fill)
        dec_ws.fill_(fill)
        check(*run_fwd(sdpa, bt, BR, workspace=ws), ref)
        check(*run_decode(sdpa, dec, 2, BR, workspace=dec_ws), dec_ref)
    sdpa.check_device_error()


def test_two_captured_forwards_share_a_workspace(sdpa):
    bts = [Batch([(900, 20), (3000 + i, 1), (600, 600)], 8, 2, 128, 16, seed=40 + i) for i in range(2)]
    refs = [bt.reference(BR) for bt in bts]
    ws = sdpa.fwd_paged_workspace(bts[0].q, bts[0].k)
    outs, graphs = [], []
    for bt in bts:
        o, lse = torch.zeros_like(bt.q), torch.zeros((8, bt.T), device="cuda")
        args = (bt.q, bt.k, bt.v, bt.cu, bt.seqlens, bt.table)
        sdpa.attn_fwd_paged(*args, workspace=ws, out=o, lse=lse)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sdpa.attn_fwd_paged(*args, workspace=ws, out=o, lse=lse)
        outs.append((o, lse))
        graphs.append(g)
    for _ in range(5):
        for g, (o, lse) in zip(graphs, outs):
            o.fill_(float("nan"))
            g.replay()
    torch.cuda.synchronize()
    for (o, lse), ref in zip(outs, refs):
        check(o, lse, ref)
    sdpa.check_device_error()


@pytest.mark.parametrize("d,page", [(128, 16), (64, 128)])
def test_many_forwards_in_a_row_over_large_caches(sdpa, d, page):
    """As for the decode: back-to-back calls, whose copies land in any order."""
    rng = random.Random(d)
    Hq, Hkv = 32, 8
    seqs = [(8000, 700)] + [(rng.randrange(1, 8000), 1) for _ in range(24)] + [(5000, 130), (3000, 9)]
    used = sum(-(-L // page) for L, _ in seqs)
    T = sum(n for _, n in seqs)
    sets = []
    gen = torch.Generator(device="cuda").manual_seed(d)
    for _ in range(3):
        k, v = (torch.randn((used, page, Hkv, d), generator=gen, device="cuda", dtype=torch.bfloat16)
                for _ in range(2))
        perm = torch.randperm(used, generator=gen, device="cuda").int()
        table = torch.zeros((len(seqs), -(-8000 // page)), dtype=torch.int32, device="cuda")
        at = 0
        for b, (L, _) in enumerate(seqs):
            m = -(-L // page)
            table[b, :m] = perm[at:at + m]
            at += m
        q = torch.randn((T, Hq, d), generator=gen, device="cuda", dtype=torch.bfloat16)
        cu = ints([sum(n for _, n in seqs[:b]) for b in range(len(seqs) + 1)])
        sets.append((q, k, v, cu, ints([L for L, _ in seqs]), table))
    ws = [sdpa.fwd_paged_workspace(s[0], s[1], BSHD) for s in sets]
    first = []
    for s, w in zip(sets, ws):
        o, lse = sdpa.attn_fwd_paged(*s, layout=BSHD, workspace=w)
        q, k, v, cu, lens, table = s
        for b, t in ((0, 0), (0, 699), (3, 702), (25, T - 10)):  # one row's sum, in 64 bits
            L, n = seqs[b]
            seen = L - (cu[b + 1].item() - 1 - t)
            keys = k[table[b, :-(-L // page)].long()].reshape(-1, Hkv, d)[:seen].double()
            x = torch.einsum("hgd,khd->hgk", q[t].double().view(Hkv, Hq // Hkv, d), keys) / d ** 0.5
            assert (torch.logsumexp(x, -1).flatten() - lse[:, t].double()).abs().max() < 1e-4, (b, t)
        first.append((o, lse))
    for i in range(300):
        o, lse = sdpa.attn_fwd_paged(*sets[i % 3], layout=BSHD, workspace=ws[i % 3])
        if i % 50 >= 47:
            assert torch.equal(o, first[i % 3][0]) and torch.equal(lse, first[i % 3][1])
    sdpa.check_device_error()


def test_plan_of_the_largest_batches(sdpa):
    rng = random.Random(9)
    for B, hi in ((4096, 12), (4097, 12), (16384, 3)):
        past = [rng.randrange(300) for _ in range(B)]
        new = [rng.randrange(hi) for _ in range(B)]
        check_plan(sdpa, plan_case(past, new, 16, pad=1, seed=B))

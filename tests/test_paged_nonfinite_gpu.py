"""Keys and queries that are not finite, over a paged cache.  A row that sees a NaN score, or one of +infinity, has
o = NaN and an lse that is not finite either, whether its keys are walked in one piece or in many; one of -infinity
has no weight; every other row is what it is without them, within the bound of ``paged_ref``."""
import math

import pytest
import torch

from tests import paged_ref
from tests.paged_ref import BHSD, BR, NONE, Batch

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def sdpa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from scaled_dot_product_fa2_b200 import build
    build.build()
    import scaled_dot_product_fa2_b200 as m
    return m


def poison_key(bt, b, j, value):
    """Element 5 of key j of sequence b, for every head."""
    bt.k_seq[b][j, :, 5] = value
    bt.k[bt.table_list[b][j // bt.page], :, j % bt.page, 5] = value


def poison_query(bt, t, h, value):
    bt.q_host[t, h, 7] = value
    bt.q[t, h, 7] = value


def check(bt, o, lse, causal, what):
    """o [T, Hq, d], lse [Hq, T] against the formula in 64 bits."""
    d, G = bt.d, bt.Hq // bt.Hkv
    sc = 1 / math.sqrt(d)
    counted = [0, 0]
    for b, (L, n) in enumerate(zip(bt.lens, bt.new)):
        c0 = bt.cu_list[b]
        if n == 0 or L == 0:
            continue
        key, tok = torch.arange(L, device="cuda")[None], torch.arange(n, device="cuda")[:, None]
        seen = key <= (tok + L - n if causal == BR else L)
        for h in range(bt.Hq):
            q = bt.q_host[c0:c0 + n, h].double().cuda()
            k, v = (s[b][:, h // G].double().cuda() for s in (bt.k_seq, bt.v_seq))
            x = (q[:, None, :] * k[None]).sum(-1) * sc
            x = x.masked_fill(~seen, -INF)
            lost = (torch.isnan(x) | (x == INF)).any(1)
            z = torch.logsumexp(torch.where(lost[:, None], 0.0, x), 1)
            empty = ~lost & (z == -INF)
            p = torch.where(x > -INF, (x - z[:, None]).exp(), 0.0)
            p[lost | empty] = 0
            finite = x.abs() < INF
            mag = torch.where(finite, (q[:, None, :] * k[None]).abs().sum(-1) * sc, 0.0).amax(1)
            e = (d + 2) * 2.0 ** -24 * mag + 2.0 ** -22 * (torch.where(finite, x, 0.0).abs().amax(1) + 4)
            out = p @ v
            bound = (paged_ref.EPS_BF16 * 1.01 + 2 * e[:, None]) * (p @ v.abs()) \
                + paged_ref.EPS_BF16 * 1.01 * out.abs() + 1e-30
            go, gl = o[c0:c0 + n, h].double(), lse[h, c0:c0 + n].double()
            at = f"{what}: sequence {b}, head {h}"
            assert torch.isnan(go[lost]).all(), f"{at}: rows that see a lost score are numbers"
            assert (torch.isnan(gl[lost]) | (gl[lost] == INF)).all(), f"{at}: their lse {gl[lost][:4]}"
            assert (gl[empty] == -INF).all() and (go[empty] == 0).all(), f"{at}: empty rows"
            ok = ~lost & ~empty
            assert ((go - out).abs() <= bound)[ok].all(), f"{at}: o"
            assert ((gl - z).abs() <= e + 2.0 ** -21 * (z.abs() + 4))[ok].all(), f"{at}: lse"
            counted[0] += lost.sum().item()
            counted[1] += ok.sum().item()
    return counted


# cut pairs, cut thin units, rows of the units' rest, units that stay whole, a table that allows no cut
SEQS = {"pair": [(5000, 40)], "thin": [(5000, 20)], "rows": [(5000, 3), (300, 1)],
        "whole": [(700, 200)] * 6, "short": [(240, 40), (200, 20), (90, 3)], "mixed": [(3000, 70), (2000, 1), (150, 9)]}


def run(sdpa, bt, causal, form):
    if form == "fwd":
        return sdpa.attn_fwd_paged(bt.q, bt.k, bt.v, bt.cu, bt.seqlens, bt.table, causal=causal)
    B, Sq = len(bt.lens), bt.new[0]
    o, lse = sdpa.attn_decode_splitkv_paged(bt.q.view(B, Sq, bt.Hq, bt.d), bt.k, bt.v, bt.seqlens, bt.table,
                                            causal=causal)
    return o.view(B * Sq, bt.Hq, bt.d), lse.transpose(0, 1).reshape(bt.Hq, B * Sq)


@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name", SEQS)
def test_fwd_with_a_key_that_is_not_finite(sdpa, name, d, value):
    for at in (0.0, 0.4, 1.0):
        for causal in (BR, NONE):
            bt = Batch(SEQS[name], 8, 2, d, 16, BHSD, seed=d)
            for b, L in enumerate(bt.lens):
                if b % 2 == 0:
                    poison_key(bt, b, int(at * (L - 1)), value)
            lost, ok = check(bt, *run(sdpa, bt, causal, "fwd"), causal, f"{name} at {at} causal={causal}")
            assert lost > 0 and (ok > 0 or value != value)
    sdpa.check_device_error()


@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("name", SEQS)
def test_fwd_with_a_query_that_is_not_finite(sdpa, name, value):
    bt = Batch(SEQS[name], 8, 2, 128, 16, BHSD, seed=1)
    poison_query(bt, 0, 3, value)
    poison_query(bt, bt.T - 1, 6, value)
    lost, ok = check(bt, *run(sdpa, bt, BR, "fwd"), BR, name)
    assert lost == 2 and ok > 0
    sdpa.check_device_error()


@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,Sq", [([5000], 1), ([9000, 700], 3), ([240, 200, 60], 2), ([700] * 40, 1),
                                     ([20000], 5)])
def test_decode_with_a_key_that_is_not_finite(sdpa, lens, Sq, d, value):
    for at in (0.0, 0.4, 1.0):
        bt = Batch([(L, Sq) for L in lens], 8, 2, d, 16, BHSD, seed=d)
        for b, L in enumerate(lens):
            if b % 2 == 0:
                poison_key(bt, b, int(at * (L - 1)), value)
        lost, _ = check(bt, *run(sdpa, bt, BR, "decode"), BR, f"at {at}")
        assert lost > 0
    sdpa.check_device_error()


@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("lens,Sq", [([5000], 1), ([9000, 700], 3), ([240, 200, 60], 2)])
def test_decode_with_a_query_that_is_not_finite(sdpa, lens, Sq, value):
    bt = Batch([(L, Sq) for L in lens], 8, 2, 128, 16, BHSD, seed=2)
    poison_query(bt, 0, 1, value)
    lost, ok = check(bt, *run(sdpa, bt, BR, "decode"), BR, "query")
    assert lost == 1 and ok > 0
    sdpa.check_device_error()


def test_a_lone_key_of_minus_infinity_leaves_the_row_empty(sdpa):
    for form in ("fwd", "decode"):
        bt = Batch([(1, 1), (40, 1)], 4, 2, 64, 16, BHSD, seed=3)
        bt.q_host[0, :, 5] = 1.0
        bt.q[0, :, 5] = 1.0
        poison_key(bt, 0, 0, -INF)
        o, lse = run(sdpa, bt, BR, form)
        assert (lse[:, 0] == -INF).all() and (o[0] == 0).all()
        check(bt, o, lse, BR, form)
    sdpa.check_device_error()

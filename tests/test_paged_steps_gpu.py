"""Whole steps over a paged cache without a host wait between the calls: each kernel starts while the one before
it still runs and reads what that one writes, the lengths that the plan advances in place among it."""
import random

import pytest
import torch

from scaled_dot_product_fa2_b200 import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sdpa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from scaled_dot_product_fa2_b200 import build
    build.build()
    import scaled_dot_product_fa2_b200 as m
    return m


def steps(sdpa, B, Hq, Hkv, d, page, seed, wait):
    """Outputs of a run of steps over fresh sequences; `wait` is called behind every call."""
    rng = random.Random(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    pages, width = 4096 // page * B, 4096 // page
    k, v = (torch.zeros((pages, Hkv, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.zeros((B, width), dtype=torch.int32, device="cuda")
    free = torch.randperm(pages, generator=gen, device="cuda").int()
    free_range = torch.tensor([0, pages], dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    cos, sin = (t.cuda() for t in inputs.rope_tables(4096, d))
    plans = []
    for i in range(24):
        new = [1] * B if i % 3 else [rng.choice((0, 1, 1, 9, 70, 200)) for _ in range(B)]
        packed = torch.randn((sum(new) + 2, (Hq + 2 * Hkv) * d), generator=gen, device="cuda").bfloat16()
        plans.append((packed, torch.tensor(new, dtype=torch.int32, device="cuda"), i % 3 == 1))
    q_like = torch.zeros((B, 1, Hq, d), dtype=torch.bfloat16, device="cuda")
    most = max(p.shape[0] for p, _, _ in plans)
    fwd_ws = sdpa.fwd_paged_workspace(torch.zeros((most, Hq, d), dtype=torch.bfloat16, device="cuda"), k)
    dec_ws = sdpa.decode_paged_workspace(q_like, k)
    torch.cuda.synchronize()
    outs = []
    for packed, new, decode in plans:
        T = packed.shape[0]
        cu, _, pos, slot, _ = sdpa.attn_page_plan(lens, new, table, free, free_range, page, T, total_lens=lens,
                                                  free_range_out=free_range)
        wait()
        q = sdpa.attn_rope_append_paged(packed, cos, sin, pos, slot, k, v, Hq, Hkv)
        wait()
        if decode:
            o, lse = sdpa.attn_decode_splitkv_paged(q[:B].view(B, 1, Hq, d), k, v, lens, table, workspace=dec_ws)
        else:
            o, lse = sdpa.attn_fwd_paged(q, k, v, cu, lens, table, workspace=fwd_ws)
        wait()
        outs += [cu, pos, slot, q, o, lse]
    sdpa.check_device_error()
    return outs + [lens, table, free_range, k, v]


@pytest.mark.parametrize("B,Hq,Hkv,d,page", [(3, 8, 2, 128, 16), (40, 4, 4, 64, 32), (150, 8, 1, 128, 64)])
def test_steps_in_a_row_are_those_with_waits_between(sdpa, B, Hq, Hkv, d, page):
    want = steps(sdpa, B, Hq, Hkv, d, page, B, torch.cuda.synchronize)
    for _ in range(5):
        got = steps(sdpa, B, Hq, Hkv, d, page, B, lambda: None)
        for g, w in zip(got, want):
            assert torch.equal(g, w)


def test_lengths_that_the_plan_advances_before_a_contiguous_decode(sdpa):
    B, Hq, Hkv, d, cap = 40, 8, 2, 128, 2048
    gen = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn((B, Hq, 1, d), generator=gen, device="cuda").bfloat16()
    k, v = (torch.randn((B, Hkv, cap, d), generator=gen, device="cuda").bfloat16() for _ in range(2))
    new = torch.randint(0, 150, (B,), generator=gen, device="cuda").int()

    def run(wait):
        lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        table = torch.zeros((B, cap // 16), dtype=torch.int32, device="cuda")
        free = torch.arange(B * cap // 16, dtype=torch.int32, device="cuda")
        free_range = torch.tensor([0, free.numel()], dtype=torch.int32, device="cuda")
        outs = []
        for _ in range(10):
            sdpa.attn_page_plan(lens, new, table, free, free_range, 16, 150 * B, total_lens=lens,
                                free_range_out=free_range)
            wait()
            outs += sdpa.attn_decode_splitkv_varlen(q, k, v, lens)
            wait()
        sdpa.check_device_error()
        return outs

    want = run(torch.cuda.synchronize)
    for _ in range(5):
        for g, w in zip(run(lambda: None), want):
            assert torch.equal(g, w)

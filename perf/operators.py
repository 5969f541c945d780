"""Cases of the paged KV cache's operators: the page plan, the rotary append into pages, the
attention of ragged chunks of new tokens over the pages, and the split-KV decode over them.

``run`` makes one pass through an operator: the framework's own call where ``own`` is true, else
the same operator written out in elementary torch operations (32-bit, rounded once at the end).
"""
from __future__ import annotations

import math
import random

import torch

own = False

_DEV = "cuda"
_BF16 = torch.bfloat16


# --------------------------------------------------------------------------- cases
def _case(op, **kw):
    c = {"op": op, "lens_seed": 1}
    c.update(kw)
    return c


def listed():
    dec = dict(op="decode", causal=True, lens_seed=1)
    fwd = dict(op="fwd", causal=True, lens_seed=1)
    return [
        # one user's next token, a short conversation: launch latency and little else
        _case(**dec, name="decode_one_short", B=1, Sq=1, Hq=32, Hkv=8, d=128, page=16, token_major=False,
              lo=700, hi=700),
        # eight caches filled to 8192 keys, one new token each: the whole pass is the cache's bytes
        _case(**dec, name="decode_b8_full", B=8, Sq=1, Hq=32, Hkv=8, d=128, page=64, token_major=False,
              lo=8192, hi=8192),
        # a serving batch in steady state: many sequences of every age, small pages, tokens outermost
        _case(**dec, name="decode_b64_mixed", B=64, Sq=1, Hq=32, Hkv=8, d=128, page=16, token_major=True,
              lo=20, hi=8192),
        # four drafted tokens to check per sequence, no shared heads, 64-wide heads
        _case(**dec, name="decode_sq4_d64", B=7, Sq=4, Hq=16, Hkv=16, d=64, page=32, token_major=False,
              lo=300, hi=5000),
        # short prompts of different lengths that arrive together
        _case(**fwd, name="chunk_short_ragged", B=5, ones=0, new_lo=3, new_hi=150, past_lo=0, past_hi=40, Hq=8,
              Hkv=2, d=64, page=16, token_major=True),
        # one prompt's chunk scheduled with the next tokens of 40 running sequences
        _case(**fwd, name="chunk_mixed_batch", B=41, ones=40, new_lo=2000, new_hi=2000, past_lo=100, past_hi=8192,
              Hq=32, Hkv=8, d=128, page=16, token_major=True),
        # a short turn at the end of a long document: few query rows, a long axis to split
        _case(**fwd, name="chunk_long_past", B=1, ones=0, new_lo=129, new_hi=129, past_lo=32639, past_hi=32639,
              Hq=32, Hkv=8, d=128, page=64, token_major=False),
        # the longest prompt in one piece
        _case(**fwd, name="chunk_prompt_16384", B=1, ones=0, new_lo=16384, new_hi=16384, past_lo=0, past_hi=0,
              Hq=32, Hkv=8, d=128, page=64, token_major=False),
        # the page plan of one decode step of eight sequences, and of a large mixed batch
        _case("plan", name="plan_step_b8", B=8, ones=8, new_lo=1, new_hi=1, past_lo=0, past_hi=8192, page=16, pad=0,
              short=False),
        _case("plan", name="plan_b512_chunks", B=512, ones=480, new_lo=300, new_hi=2048, past_lo=0, past_hi=8192,
              page=16, pad=100, short=False),
        # the append of one decode step, and of prompts' chunks with decode tokens beside them in a
        # padded buffer
        _case("append", name="append_step_b8", B=8, ones=8, new_lo=1, new_hi=1, past_lo=100, past_hi=2000, Hq=32,
              Hkv=8, d=128, page=16, token_major=False, pad=0),
        _case("append", name="append_chunk_8192", B=24, ones=20, new_lo=1500, new_hi=2048, past_lo=0, past_hi=500,
              Hq=32, Hkv=8, d=128, page=16, token_major=True, pad=28),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _key_budget(heads):
    """Cached keys of all sequences together that are no more than the largest listed cache."""
    return (64 << 20) // (heads["Hkv"] * heads["d"])


def draw(rng):
    op = rng.choice(("decode", "decode", "fwd", "fwd", "plan", "append"))
    seed = rng.randrange(1 << 30)
    page = rng.choice((16, 32, 64, 128))
    heads = dict(zip(("Hq", "Hkv"), rng.choice(((32, 8), (16, 16), (8, 2), (6, 2), (4, 4), (16, 2), (5, 5), (8, 1)))))
    heads.update(d=rng.choice((64, 128)), page=page, token_major=rng.random() < 0.5)
    if op == "decode":
        hi = _log(rng, 1, 8192)
        b = max(1, min(_log(rng, 1, 64), _key_budget(heads) // hi))
        return _case(op, lens_seed=seed, B=b, Sq=rng.choice((1, 1, 1, 2, 3, 4)), causal=rng.random() < 0.9,
                     lo=rng.choice((0, 1, hi)) if hi > 1 else 1, hi=hi, **heads)
    if op == "fwd":
        new = _log(rng, 2, 4096)
        past = rng.choice((0, _log(rng, 1, 8192)))
        b = max(1, min(_log(rng, 1, 40), _key_budget(heads) // (past + new)))
        ones = rng.randrange(b)
        while (b - ones) * new > 16384:
            ones += 1
        return _case(op, lens_seed=seed, B=b, ones=ones, new_lo=rng.choice((0, max(1, new // 3))), new_hi=new,
                     past_lo=0, past_hi=past, causal=rng.random() < 0.9, **heads)
    b = _log(rng, 1, 512 if op == "plan" else 64)
    new = _log(rng, 1, 2048)
    ones = rng.randrange(b + 1)
    while (b - ones) * new > (65536 if op == "plan" else 8192):
        ones += 1
    c = dict(lens_seed=seed, B=b, ones=ones, new_lo=rng.choice((0, new)), new_hi=new, past_lo=0,
             past_hi=_log(rng, 1, 8192 if op == "plan" else 2000), pad=rng.choice((0, rng.randrange(1, 64))))
    if op == "plan":
        return _case(op, page=page, short=rng.random() < 0.2, **c)
    return _case(op, **c, **heads)


def _between(rng, lo, hi):
    """Spread over the logarithm where the range spans more than a factor of ten."""
    if hi <= lo:
        return lo
    if hi > 10 * max(lo, 1):
        return min(hi, lo + _log(rng, 1, hi - lo + 1) - 1)
    return rng.randint(lo, hi)


def _lens(case):
    """(past, new) of every sequence; the first one is the longest of the range."""
    rng = random.Random(case["lens_seed"] * 7919 + case["B"])
    if case["op"] == "decode":
        total = [_between(rng, case["lo"], case["hi"]) for _ in range(case["B"])]
        total[0] = case["hi"]
        return total, [case["Sq"]] * case["B"]
    past, new = [], []
    for b in range(case["B"]):
        chunk = b < case["B"] - case["ones"]
        past.append(_between(rng, case["past_lo"], case["past_hi"]))
        new.append(_between(rng, case["new_lo"], case["new_hi"]) if chunk else 1)
    if case["B"] > case["ones"]:
        new[0] = case["new_hi"]
    return past, new


def _pages(n, page):
    return (n + page - 1) // page


# --------------------------------------------------------------------------- inputs
def _ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=_DEV)


def _table(case, totals, gen, spare=3):
    """A block table over randomly placed pages, and the number of pages in the pool."""
    width = max(1, max(_pages(t, case["page"]) for t in totals)) + 1
    used = sum(_pages(t, case["page"]) for t in totals)
    pool = used + spare
    perm = torch.randperm(pool, generator=gen, device=_DEV).to(torch.int32)
    table = torch.zeros((case["B"], width), dtype=torch.int32, device=_DEV)
    at = 0
    for b, t in enumerate(totals):
        n = _pages(t, case["page"])
        table[b, :n] = perm[at:at + n]
        at += n
    return table, pool, perm[at:]


def _page_shape(case, pool):
    if case["token_major"]:
        return (pool, case["page"], case["Hkv"], case["d"])
    return (pool, case["Hkv"], case["page"], case["d"])


def prepare(case, seed):
    gen = torch.Generator(device=_DEV)
    gen.manual_seed(int(seed))
    st = {"case": case}

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=_DEV, dtype=_BF16)

    op = case["op"]
    past, new = _lens(case)
    if op == "plan":
        P = case["page"]
        tot = [p + n for p, n in zip(past, new)]
        width = max(1, max(_pages(t, P) for t in tot))
        held = [_pages(p, P) for p in past]
        need = sum(_pages(t, P) - h for t, h in zip(tot, held))
        free = max(1, need // 2) if case["short"] else need + 5
        perm = torch.randperm(sum(held) + free, generator=gen, device=_DEV).to(torch.int32)
        table = torch.full((case["B"], width), -1, dtype=torch.int32, device=_DEV)
        at = 0
        for b, h in enumerate(held):
            table[b, :h] = perm[at:at + h]
            at += h
        skip = 2  # pages at the head of the list that earlier steps took
        fl = torch.cat([torch.full((skip,), -1, dtype=torch.int32, device=_DEV), perm[at:]]).contiguous()
        T = sum(new) + case["pad"]
        st.update(past=_ints(past), new=_ints(new), table=table, free=fl, range=_ints([skip, skip + free]), T=max(T, 1),
                  outs=(_ints([0] * (case["B"] + 1)), _ints([0] * case["B"]),
                        torch.empty(max(T, 1), dtype=torch.int32, device=_DEV),
                        torch.empty(max(T, 1), dtype=torch.int32, device=_DEV), _ints([0, 0])))
        return st
    if op == "append":
        P, d = case["page"], case["d"]
        tot = [p + n for p, n in zip(past, new)]
        table, pool, _ = _table(case, tot, gen)
        T = max(1, sum(new) + case["pad"])
        host = table.cpu().tolist()
        pos, slot = [], []
        for b in range(case["B"]):
            for i in range(past[b], tot[b]):
                pos.append(i)
                slot.append(host[b][i // P] * P + i % P)
        st["n"] = len(pos)
        pos += [-1] * (T - len(pos))
        slot += [-1] * (T - len(slot))
        half = torch.arange(d // 2, dtype=torch.float64, device=_DEV)
        ang = torch.arange(max(tot) + 1, dtype=torch.float64, device=_DEV)[:, None] * 10000.0 ** (-2.0 * half / d)
        st.update(packed=normal(T, (case["Hq"] + 2 * case["Hkv"]) * d), cos=ang.cos().float(), sin=ang.sin().float(),
                  pos=_ints(pos), slot=_ints(slot), k=normal(*_page_shape(case, pool)),
                  v=normal(*_page_shape(case, pool)),
                  q=torch.zeros((T, case["Hq"], d), dtype=_BF16, device=_DEV))
        return st
    totals = past if op == "decode" else [p + n for p, n in zip(past, new)]
    table, pool, _ = _table(case, totals, gen)
    st.update(table=table, k=normal(*_page_shape(case, pool)), v=normal(*_page_shape(case, pool)), lens=_ints(totals),
              totals=totals, new=new)
    if op == "decode":
        q = normal(case["B"], case["Sq"], case["Hq"], case["d"])
        lse = torch.zeros((case["B"], case["Hq"], case["Sq"]), dtype=torch.float32, device=_DEV)
    else:
        T = max(1, sum(new))
        q = normal(T, case["Hq"], case["d"])
        lse = torch.zeros((case["Hq"], T), dtype=torch.float32, device=_DEV)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        st["cu"] = _ints(cu)
    st.update(q=q, o=torch.zeros_like(q), lse=lse)
    if own:
        import scaled_dot_product_fa2_b200 as sdpa
        mode = dict(layout=sdpa.LAYOUT_BSHD if case["token_major"] else sdpa.LAYOUT_BHSD)
        make = sdpa.decode_paged_workspace if op == "decode" else sdpa.fwd_paged_workspace
        st["workspace"] = make(q, st["k"], **mode)
    return st


# --------------------------------------------------------------------------- one pass
def run(st):
    return _own(st) if own else _plain(st)


def _own(st):
    import scaled_dot_product_fa2_b200 as sdpa
    case = st["case"]
    op = case["op"]
    if op == "plan":
        cu, tot, pos, slot, rng = st["outs"]
        sdpa.attn_page_plan(st["past"], st["new"], st["table"], st["free"], st["range"], case["page"], st["T"],
                            cu_new=cu, total_lens=tot, positions=pos, slot_map=slot, free_range_out=rng)
        return (st["table"], *st["outs"])
    layout = sdpa.LAYOUT_BSHD if case["token_major"] else sdpa.LAYOUT_BHSD
    if op == "append":
        sdpa.attn_rope_append_paged(st["packed"], st["cos"], st["sin"], st["pos"], st["slot"], st["k"], st["v"],
                                    case["Hq"], case["Hkv"], layout=layout, q_out=st["q"])
        return st["q"], st["k"], st["v"]
    causal = sdpa.CAUSAL_BOTTOM_RIGHT if case["causal"] else sdpa.CAUSAL_NONE
    if op == "decode":
        return sdpa.attn_decode_splitkv_paged(st["q"], st["k"], st["v"], st["lens"], st["table"], causal=causal,
                                              layout=layout, workspace=st["workspace"], out=st["o"], lse=st["lse"])
    return sdpa.attn_fwd_paged(st["q"], st["k"], st["v"], st["cu"], st["lens"], st["table"], causal=causal,
                               layout=layout, workspace=st["workspace"], out=st["o"], lse=st["lse"])


def _plain(st):
    op = st["case"]["op"]
    if op == "plan":
        return _plain_plan(st)
    if op == "append":
        return _plain_append(st)
    return _plain_attention(st)


def _plain_plan(st):
    P, past, new, table = st["case"]["page"], st["past"].long(), st["new"].long(), st["table"]
    B, T = past.shape[0], st["T"]
    held = (past + P - 1) // P
    need = (past + new + P - 1) // P - held
    cum = need.cumsum(0)
    head = st["range"][0].long()
    free = st["range"][1].long() - head
    fits = (need == 0) | (cum <= free)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=_DEV), new.cumsum(0)])
    t = torch.arange(T, device=_DEV)
    b = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=B - 1)
    live = (t < cu[B]) & fits[b]
    pos = past[b] + t - cu[b]
    page_i = pos // P
    fresh = page_i >= held[b]
    at = head + cum[b] - need[b] + page_i - held[b]
    taken = st["free"][at.clamp(0, st["free"].shape[0] - 1)].long()
    old = table[b, page_i.clamp(max=table.shape[1] - 1)].long()
    page = torch.where(fresh, taken, old)
    slot = torch.where(live, page * P + pos % P, -1)
    # the block table's new entries: entry j of sequence b is page j - held[b] of its share
    j = torch.arange(table.shape[1], device=_DEV)[None, :]
    mine = (j >= held[:, None]) & (j < (held + need)[:, None]) & fits[:, None]
    src = (head + (cum - need)[:, None] + j - held[:, None]).clamp(0, st["free"].shape[0] - 1)
    table.copy_(torch.where(mine, st["free"][src], table))
    used = torch.where(fits, need, 0).sum()
    return (table, cu.int(), torch.where(fits, past + new, past).int(),
            torch.where(t < cu[B], pos, -1).int(), slot.int(), torch.stack([head + used, head + free]).int())


def _plain_append(st):
    c, n = st["case"], st["n"]
    Hq, Hkv, d, P = c["Hq"], c["Hkv"], c["d"], c["page"]
    x = st["packed"][:n].view(n, Hq + 2 * Hkv, d)
    pos, slot = st["pos"][:n].long(), st["slot"][:n].long()
    cos, sin = st["cos"][pos][:, None, :], st["sin"][pos][:, None, :]
    f = x[:, :Hq + Hkv].float()
    a, b = f[..., :d // 2], f[..., d // 2:]
    r = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1).to(_BF16)
    st["q"][:n] = r[:, :Hq]
    page, row = slot // P, slot % P
    if c["token_major"]:
        st["k"][page, row] = r[:, Hq:]
        st["v"][page, row] = x[:, Hq + Hkv:]
    else:
        st["k"][page, :, row] = r[:, Hq:]
        st["v"][page, :, row] = x[:, Hq + Hkv:]
    return st["q"], st["k"], st["v"]


def _plain_attention(st):
    c = st["case"]
    Hq, Hkv, d, P, G = c["Hq"], c["Hkv"], c["d"], c["page"], c["Hq"] // c["Hkv"]
    scale = 1.0 / math.sqrt(d)
    decode = c["op"] == "decode"
    o = st["o"].view(-1, Hq, d)
    q = st["q"].view(-1, Hq, d)
    t0 = 0
    for b, (L, n) in enumerate(zip(st["totals"], st["new"])):
        if n == 0:
            continue
        ids = st["table"][b, :_pages(L, P)].long()
        k, v = st["k"][ids], st["v"][ids]
        if not c["token_major"]:
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        k = k.reshape(-1, Hkv, d)[:L].float()
        v = v.reshape(-1, Hkv, d)[:L].float()
        k, v = k.transpose(0, 1), v.transpose(0, 1)  # [Hkv, L, d]
        rows = max(1, (1 << 29) // max(1, L * Hq))  # query tokens whose scores are held at a time
        for i0 in range(0, n, rows):
            i1 = min(n, i0 + rows)
            m = i1 - i0
            last = (L - n if c["causal"] else L) + torch.arange(i0, i1, device=_DEV)
            seen = (torch.arange(L, device=_DEV)[None, :] <= last[:, None]).repeat_interleave(G, dim=0)
            qs = q[t0 + i0:t0 + i1].float().view(m, Hkv, G, d).transpose(0, 1).reshape(Hkv, m * G, d)
            x = torch.matmul(qs, k.transpose(1, 2)) * scale  # [Hkv, tokens * G, L]
            x = torch.where(seen, x, -math.inf)
            if L > 0:
                top = x.max(dim=-1, keepdim=True).values
            else:
                top = torch.full((Hkv, m * G, 1), -math.inf, device=_DEV)
            base = torch.where(top == -math.inf, 0.0, top)
            e = torch.exp(x - base)
            den = e.sum(dim=-1, keepdim=True)
            out = torch.matmul(e, v) / torch.where(den == 0, 1.0, den)
            o[t0 + i0:t0 + i1] = out.view(Hkv, m, G, d).transpose(0, 1).reshape(m, Hq, d).to(_BF16)
            lse = (base + torch.log(den)).view(Hkv, m, G).transpose(1, 2).reshape(Hq, m)
            if decode:
                st["lse"][b, :, i0:i1] = lse
            else:
                st["lse"][:, t0 + i0:t0 + i1] = lse
        t0 += n
    return st["o"], st["lse"]


# --------------------------------------------------------------------------- 64-bit definition
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return _exact_plan(st)
    if op == "append":
        return _exact_append(st)
    return _exact_attention(st)


def _exact_plan(st):
    P, T = st["case"]["page"], st["T"]
    past, new, table = st["past"].tolist(), st["new"].tolist(), st["table"].tolist()
    free, (head, tail) = st["free"].tolist(), st["range"].tolist()
    cu, total, pos, slot = [0], [], [-1] * T, [-1] * T
    asked = used = 0
    for b, (p, n) in enumerate(zip(past, new)):
        held, want = _pages(p, P), _pages(p + n, P)
        asked += want - held
        ok = want == held or asked <= tail - head
        if ok:
            for j in range(held, want):
                table[b][j] = free[head + used]
                used += 1
        for i in range(n):
            pos[cu[b] + i] = p + i
            if ok:
                slot[cu[b] + i] = table[b][(p + i) // P] * P + (p + i) % P
        cu.append(cu[b] + n)
        total.append(p + n if ok else p)
    return tuple(_ints(x) for x in (table, cu, total, pos, slot, [head + used, tail]))


def _exact_append(st):
    c = st["case"]
    Hq, Hkv, d, P = c["Hq"], c["Hkv"], c["d"], c["page"]
    q, k, v = st["q"].double(), st["k"].double(), st["v"].double()
    pos = st["pos"][:st["n"]].long()
    slot = st["slot"][:st["n"]].long()
    z = st["packed"][:st["n"]].double().view(-1, Hq + 2 * Hkv, 2, d // 2)
    turn = torch.complex(st["cos"][pos].double(), st["sin"][pos].double())[:, None]
    w = torch.complex(z[:, :, 0], z[:, :, 1]) * turn
    rot = torch.stack([w.real, w.imag], dim=2).flatten(2)
    q[:st["n"]] = rot[:, :Hq]
    # one row per (page, row in page), heads next to each other
    kk = k if c["token_major"] else k.transpose(1, 2)
    vv = v if c["token_major"] else v.transpose(1, 2)
    kk[slot // P, slot % P] = rot[:, Hq:Hq + Hkv]
    vv[slot // P, slot % P] = z[:, Hq + Hkv:].flatten(2)
    return q, k, v


def _exact_attention(st):
    c = st["case"]
    Hq, Hkv, d, P = c["Hq"], c["Hkv"], c["d"], c["page"]
    G = Hq // Hkv
    o = st["o"].double()
    lse = st["lse"].double()
    flat_o, flat_q = o.view(-1, Hq, d), st["q"].view(-1, Hq, d)
    swap = (lambda x: x) if c["token_major"] else (lambda x: x.transpose(1, 2))
    kp, vp = swap(st["k"]), swap(st["v"])
    start = 0
    for b, (L, n) in enumerate(zip(st["totals"], st["new"])):
        key = torch.arange(L, device=_DEV)
        page, row = st["table"][b].long()[key // P], key % P
        for hq in range(Hq if n else 0):
            kh, vh = kp[page, row, hq // G].double(), vp[page, row, hq // G].double()
            for i in range(0, n, 4096):
                j = min(n, i + 4096)
                s = flat_q[start + i:start + j, hq].double() @ kh.T / d ** 0.5
                if c["causal"]:
                    hidden = key[None] > torch.arange(i, j, device=_DEV)[:, None] + (L - n)
                    s = s.masked_fill(hidden, -math.inf)
                z = torch.logsumexp(s, 1)
                p = (s - z[:, None]).exp()
                p[z == -math.inf] = 0
                flat_o[start + i:start + j, hq] = p @ vh
                if c["op"] == "decode":
                    lse[b, hq, i:j] = z
                else:
                    lse[hq, start + i:start + j] = z
        start += n
    return o, lse


# --------------------------------------------------------------------------- floors
def work(case):
    past, new = _lens(case)
    B, op = case["B"], case["op"]
    if op == "plan":
        P = case["page"]
        T = max(1, sum(new) + case["pad"])
        fresh = sum(_pages(p + n, P) - _pages(p, P) for p, n in zip(past, new))
        held = sum(1 for p, n in zip(past, new) if n and p % P)
        return {"bytes": 4 * (2 * B + 2 + 2 * fresh + held + (B + 1) + B + 2 * T + 2), "flops": 0}
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if op == "append":
        n = sum(new)
        rows = len({i for p, m in zip(past, new) for i in range(p, p + m)})
        T = max(1, n + case["pad"])
        return {"bytes": 2 * 2 * n * (Hq + 2 * Hkv) * d + rows * 4 * d + 8 * T, "flops": 3 * n * (Hq + Hkv) * d}
    totals = past if op == "decode" else [p + n for p, n in zip(past, new)]
    keys = rows = pairs = table = 0
    for L, n in zip(totals, new):
        if n == 0:
            continue
        rows += n
        table += _pages(L, case["page"])
        keys += L
        if case["causal"]:
            first = max(0, n - L)  # rows before it see no key
            m = n - first
            pairs += m * (L - n + first + 1) + m * (m - 1) // 2
        else:
            pairs += n * L
    return {"bytes": 2 * 2 * keys * Hkv * d + rows * Hq * (2 * 2 * d + 4) + 4 * (table + 2 * B),
            "flops": 4 * pairs * Hq * d}

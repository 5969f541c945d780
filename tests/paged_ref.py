"""Plain implementations (Python integers, 64-bit floats) of the paged cache's operators, and the
batches the tests run them on."""
from __future__ import annotations

import math

import torch

BHSD, BSHD = 0, 1
NONE, TL, BR = 0, 1, 2
EPS_BF16 = torch.finfo(torch.bfloat16).eps / 2  # one rounding to bf16, relative
NOT_AN_ENTRY = 1 << 29  # fills the table entries a call must not look at


def pages_of(n, page):
    return -(-n // page)


def plan(past, new, table, free_pages, free_range, page, T, max_pages):
    """attn_page_plan on Python lists: (table, cu, total, positions, slots, range), any refused."""
    table = [list(r) for r in table]
    head, tail = free_range
    cu, total, positions, slots = [0], [], [-1] * T, [-1] * T
    asked = used = tokens = 0
    refused = False
    for b, (p, n) in enumerate(zip(past, new)):
        ok = p >= 0 and n >= 0 and p + n <= max_pages * page
        held, want = pages_of(p, page), pages_of(p + n, page)
        if ok:
            asked += want - held
        tokens += max(n, 0)
        ok = ok and tokens <= T and (want == held or asked <= tail - head)
        if ok:
            for j in range(held, want):
                table[b][j] = free_pages[head + used]
                used += 1
        for t in range(cu[-1], min(tokens, T)):
            i = p + t - cu[-1]
            positions[t] = i
            if ok:
                slots[t] = table[b][i // page] * page + i % page
        cu.append(min(tokens, T))
        total.append(p + n if ok else p)
        refused = refused or not ok
    return (table, cu, total, positions, slots, [head + used, tail]), refused


class Batch:
    """Sequences of L keys, of which n are new, in a paged cache.  Everything a call must not read is
    NaN (rows of the pages behind a sequence's last key) or NOT_AN_ENTRY (table entries)."""

    def __init__(self, seqs, Hq, Hkv, d, page, layout=BHSD, seed=0, pad=0, interleaved=False, device="cuda"):
        self.Hq, self.Hkv, self.d, self.page, self.layout = Hq, Hkv, d, page, layout
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.new = [s[0] for s in seqs], [s[1] for s in seqs]
        self.T = sum(self.new) + pad
        used = sum(pages_of(L, page) for L in self.lens)
        self.N = used + 2
        width = max([pages_of(L, page) for L in self.lens] + [1]) + 1
        perm = torch.randperm(self.N, generator=gen).tolist()
        table = [[NOT_AN_ENTRY] * width for _ in seqs]
        inner = (page, Hkv, d) if layout == BSHD else (Hkv, page, d)
        if interleaved:
            both = torch.full((self.N, 2, *inner), float("nan"), dtype=torch.bfloat16)
            k, v = both[:, 0], both[:, 1]
        else:
            k = torch.full((self.N, *inner), float("nan"), dtype=torch.bfloat16)
            v = k.clone()
        self.k_seq, self.v_seq = [], []
        at = 0
        for b, L in enumerate(self.lens):
            ks = torch.randn((L, Hkv, d), generator=gen).bfloat16()
            vs = torch.randn((L, Hkv, d), generator=gen).bfloat16()
            self.k_seq.append(ks)
            self.v_seq.append(vs)
            for j in range(pages_of(L, page)):
                table[b][j] = perm[at]
                rows = slice(j * page, min(L, (j + 1) * page))
                m = rows.stop - rows.start
                for pool, seq in ((k, ks), (v, vs)):
                    if layout == BSHD:
                        pool[perm[at], :m] = seq[rows]
                    else:
                        pool[perm[at], :, :m] = seq[rows].transpose(0, 1)
                at += 1
        self.table_list = table
        self.q_host = torch.randn((self.T, Hq, d), generator=gen).bfloat16()
        cu = [0]
        for n in self.new:
            cu.append(cu[-1] + n)
        self.cu_list = cu

        def ints(x):
            return torch.tensor(x, dtype=torch.int32, device=device)

        if interleaved:
            both = both.to(device)
            self.k, self.v = both[:, 0], both[:, 1]
        else:
            self.k, self.v = k.to(device), v.to(device)
        self.q = self.q_host.to(device)
        self.cu, self.seqlens, self.table = ints(cu), ints(self.lens), ints(table)

    def reference(self, causal, scale=0.0, device="cuda"):
        """(o [T, Hq, d], lse [Hq, T], bound on |o error|, bound on |lse error|) in 64 bits.

        The kernels round each probability to bf16 (relative 2^-8), the output to bf16 (2^-8) and
        hold all else in fp32.  A score is a sum of d products: its error is at most (d + 2) 2^-24
        of the sum of the products' magnitudes, plus 2^-22 of its own size in the exponent's
        argument (two roundings of the running maximum times the scale, one of the sum); exp2's
        is 2^-22 relative.  With A = sum_j p_j |v_j|, an error e of every score changes o by at
        most 2 e A.
        """
        d, G = self.d, self.Hq // self.Hkv
        sc = scale if scale else 1 / math.sqrt(d)
        o = torch.zeros((self.T, self.Hq, d), dtype=torch.float64, device=device)
        lse = torch.full((self.Hq, self.T), -math.inf, dtype=torch.float64, device=device)
        ob, lb = torch.zeros_like(o), torch.zeros_like(lse)
        for b, (L, n) in enumerate(zip(self.lens, self.new)):
            c0 = self.cu_list[b]
            if L == 0 or n == 0:
                continue
            key = torch.arange(L, device=device)
            tok = torch.arange(n, device=device)
            last = {NONE: torch.full_like(tok, L), TL: tok, BR: tok + L - n}[causal]
            seen = key[None] <= last[:, None]
            for hk in range(self.Hkv):
                k = self.k_seq[b][:, hk].double().to(device)
                v = self.v_seq[b][:, hk].double().to(device)
                for hq in range(hk * G, hk * G + G):
                    q = self.q_host[c0:c0 + n, hq].double().to(device)
                    x = (q @ k.T * sc).masked_fill(~seen, -math.inf)
                    mag = (q.abs() @ k.abs().T * sc).masked_fill(~seen, 0.0).amax(1)
                    z = torch.logsumexp(x, 1)
                    p = torch.where(seen, (x - z[:, None]).exp(), 0.0)
                    p[z == -math.inf] = 0
                    top = x.masked_fill(~seen, 0.0).abs().amax(1)
                    e = (d + 2) * 2.0 ** -24 * mag + 2.0 ** -22 * (top + 4)
                    A = p @ v.abs()
                    out = p @ v
                    o[c0:c0 + n, hq] = out
                    lse[hq, c0:c0 + n] = z
                    ob[c0:c0 + n, hq] = (EPS_BF16 * 1.01 + 2 * e[:, None]) * A + EPS_BF16 * 1.01 * out.abs() + 1e-30
                    lb[hq, c0:c0 + n] = e + 2.0 ** -21 * torch.where(z == -math.inf, 0.0, z.abs() + 4)
        return o, lse, ob, lb


def check(got_o, got_lse, ref, what=""):
    o, lse, ob, lb = ref
    err = (got_o.double() - o).abs()
    assert not torch.isnan(err).any(), f"{what}: NaN"
    over = (err - ob).max().item() if err.numel() else 0.0
    assert (err <= ob).all(), f"{what}: o off by {over:.3e} above its bound"
    empty = lse == -math.inf
    assert torch.equal(got_lse.double() == -math.inf, empty), f"{what}: pattern of empty rows"
    lerr = torch.where(empty, 0.0, got_lse.double() - lse).abs()
    assert (lerr <= lb).all(), f"{what}: lse off by {(lerr - lb).max().item():.3e} above its bound"

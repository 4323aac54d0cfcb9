"""Plumbing of the attention tests: a step of sequences on the device, the library's calls on it, and their results
against the 64-bit oracle."""
from __future__ import annotations

import numpy as np
import torch

import rank_adapter_gb300 as ra
from oracle import attn_oracle

EPS = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative to the value


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Step:
    """Sequences with `new` rows and `before` tokens in the cache ahead of them; q, k and v are column ranges of one
    packed matrix. Everything a kernel must not use holds NaN: rows past the last sequence, unused slots of pages
    and unused pages."""

    def __init__(self, heads, kv_heads, head_dim, new, before=None, dtype=torch.bfloat16, causal=True, page=16, scale=None,
                 seed=0, pad_rows=0, spread=2.0, layout="page", spare_pages=3):
        g = torch.Generator().manual_seed(seed)
        self.H, self.K, self.D, self.new, self.causal, self.dtype, self.page = heads, kv_heads, head_dim, list(new), causal, dtype, page
        self.before = list(before) if before is not None else [0] * len(self.new)
        self.start = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.used, self.T = int(self.start[-1]), int(self.start[-1]) + pad_rows
        self.kv = np.array([a + b for a, b in zip(self.new, self.before)], np.int32)
        qkv = torch.randn(self.T, (heads + 2 * kv_heads) * head_dim, generator=g)
        qkv[:, :heads * head_dim] *= spread
        qkv[self.used:] = float("nan")
        self.qkv = qkv.to(dtype).cuda()
        self.q, self.k, self.v = self.qkv.split([heads * head_dim, kv_heads * head_dim, kv_heads * head_dim], 1)
        self.out = torch.full((self.T, heads * head_dim), 7.0, dtype=dtype, device="cuda")
        self.lse = torch.full((self.T, heads), 7.0, device="cuda")
        self.att = ra.Attention(heads, kv_heads, head_dim, scale=scale, causal=causal,
                                dtype=ra.LORA_BF16 if dtype == torch.bfloat16 else ra.LORA_F32)
        self.q_start = torch.from_numpy(self.start).cuda()
        self.kv_len = torch.from_numpy(self.kv).cuda()
        if before is None:
            self.seqs = ra.SeqMeta(self.att, self.T, len(self.new))
            self.seqs.prepare(self.T, self.q_start)
            return
        need = [-(-int(x) // page) for x in self.kv]
        self.most_pages = max(1, max(need))
        pool = sum(need) + spare_pages
        perm = torch.randperm(pool, generator=g).tolist()
        table = np.full((len(self.new), self.most_pages), 1 << 30, np.int32)   # entries past a sequence's pages are not to be read
        for b, n in enumerate(need):
            table[b, :n] = [perm.pop() for _ in range(n)]
        self.table = torch.from_numpy(table).cuda()
        shape = {"page": (pool, page, kv_heads, head_dim), "head": (pool, kv_heads, page, head_dim),
                 "both": (pool, 2, page, kv_heads, head_dim)}[layout]
        make = lambda: torch.full(shape, float("nan"), dtype=dtype, device="cuda")  # noqa: E731
        if layout == "both":
            both = make()
            self.kc, self.vc = both[:, 0], both[:, 1]
        else:
            self.kc, self.vc = make(), make()
            if layout == "head":
                self.kc, self.vc = self.kc.transpose(1, 2), self.vc.transpose(1, 2)
        self.cache = ra.KVCache(self.kc, self.vc)
        for b, n in enumerate(self.before):                                     # what earlier steps wrote
            x = torch.randn(2, n, kv_heads, head_dim, generator=g).to(dtype).cuda()
            j = np.arange(n)
            page_of, slot = torch.from_numpy(table[b][j // page]).long().cuda(), torch.from_numpy(j % page).cuda()
            self.kc[page_of, slot], self.vc[page_of, slot] = x[0], x[1]
        self.seqs = ra.SeqMeta(self.att, self.T, len(self.new), page, self.most_pages)
        self.seqs.prepare(self.T, self.q_start, self.kv_len, self.table)

    def write(self, **kw):
        ra.kv_write(self.seqs, self.cache, self.k, self.v, **kw)

    def prompt(self, **kw):
        ra.attn_prompt(self.seqs, self.q, self.k, self.v, self.out, lse=self.lse, **kw)

    def paged(self, **kw):
        ra.attn_paged(self.seqs, self.cache, self.q, self.out, lse=self.lse, **kw)

    def oracle(self, keys=None, values=None):
        """keys, values: per sequence; by default the packed rows (a prompt), or the pages."""
        if keys is None:
            if hasattr(self, "cache"):
                table = self.table.cpu().numpy()
                keys = attn_oracle.paged_rows(f64(self.kc), table, self.kv)
                values = attn_oracle.paged_rows(f64(self.vc), table, self.kv)
            else:
                split = lambda t: [f64(t)[a:b].reshape(b - a, self.K, self.D) for a, b in zip(self.start, self.start[1:])]  # noqa: E731
                keys, values = split(self.k), split(self.v)
        return attn_oracle.attention(f64(self.q), keys, values, self.start, self.kv, self.H, self.K, self.D,
                                     float(np.float32(self.att.scale)), self.causal)

    def check(self, want=None, status=0):
        torch.cuda.synchronize()
        assert ra.lora_query_seqs(self.seqs.c)[0] == status
        out, lse, spread, reach = want or self.oracle()
        eps = EPS[self.dtype]
        tol, tol_lse = attn_oracle.tolerance(out, lse, spread, reach, self.D, max(1, int(self.kv.max())),
                                             eps if self.dtype == torch.bfloat16 else 0.0, eps)
        got, got_lse = f64(self.out).reshape(self.T, self.H, self.D), f64(self.lse)
        n = self.used
        bad = ~(np.abs(got[:n] - out[:n]) <= tol[:n])
        assert not bad.any(), (f"{bad.sum()} of {bad.size} outputs off, first (row, head, element) {np.argwhere(bad)[0]}: "
                               f"{got[:n][bad][0]} for {out[:n][bad][0]}, bound {tol[:n][bad][0]}")
        none = np.isneginf(lse[:n])
        assert np.array_equal(np.isneginf(got_lse[:n]), none)
        bad = ~none & ~(np.abs(np.where(none, 0, got_lse[:n]) - np.where(none, 0, lse[:n])) <= tol_lse[:n])
        assert not bad.any(), f"lse: first off at (row, head) {np.argwhere(bad)[0]}: {got_lse[:n][bad][0]} for {lse[:n][bad][0]}"
        assert (got[n:] == 7.0).all() and (got_lse[n:] == 7.0).all(), "rows behind the last sequence were written"

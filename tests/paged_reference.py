"""Plain 64-bit forms of the paged cache's operations, request by request, and
random inputs for them."""
from __future__ import annotations

import numpy as np
import torch

E4M3_MAX = 448.0


def two(e):
    """2^e in 64 bits, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def held(x, e4m3):
    """What a cache holds for bf16 rows x [..., D]: x, or its rounding to the
    e4m3 grid under the row's power-of-two scale (non-finite becomes NaN)."""
    x = x.double().cpu()
    if not e4m3:
        return x
    fin = torch.isfinite(x)
    top = torch.where(fin, x, 0.0).abs().amax(-1, keepdim=True)
    mant, power = torch.frexp(top)                                  # top = mant 2^power, mant in [1/2, 1)
    e = torch.where(mant <= 0.875, power - 9, power - 8).clamp(-110, 119)
    y = (x * two(-e)).clamp(-E4M3_MAX, E4M3_MAX)
    ymant, ypower = torch.frexp(y.abs())
    step = two((ypower - 1).clamp(min=-6) - 3)
    q = torch.round(y / step) * step * two(e)
    return torch.where(fin, q, torch.nan)


class Setup:
    """A pool of pages in random order with lengths w (windows) and ctx, filled
    with `fill` wherever no request has a token."""

    def __init__(self, w, ctx, G, D, page, e4m3, seed=0, spare=3, fill=float("nan"), device="cuda"):
        from speculative_decoding_markov_gb300 import binding as sdm
        self.w, self.ctx_list, self.G, self.D, self.page, self.e4m3 = list(w), list(ctx), G, D, page, e4m3
        R = len(w)
        g = torch.Generator().manual_seed(seed)
        self.gen = g
        need = [(a + b + page - 1) // page for a, b in zip(w, ctx)]
        n_pages = sum(need) + spare
        order = torch.randperm(n_pages, generator=g).to(torch.int32)
        table = torch.zeros((R, max(max(need), 1) + 1), dtype=torch.int32)
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n]
            at += n
        self.table_cpu = table
        # every token's keys and values [tokens, G, D], as the bf16 rows that were written
        self.kv = [{n: torch.randn((a + b, G, D), generator=g).to(torch.bfloat16) for n in "kv"}
                   for a, b in zip(w, ctx)]
        dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
        self.cache = sdm.PagedCache.empty(n_pages, G, page, D, table.to(device), dtype)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(w)]), dtype=torch.int32, device=device)
        self.ctx = torch.tensor(ctx, dtype=torch.int32, device=device)
        self.rows = int(sum(w))
        self.status = sdm.new_status()
        self.fill_pools(fill)

    def fill_pools(self, fill):
        c = self.cache
        if self.e4m3:
            code = torch.full((1,), fill).to(torch.float8_e4m3fn).view(torch.uint8).item()
            c.k.view(torch.uint8).fill_(code)
            c.v.view(torch.uint8).fill_(code)
        else:
            c.k.fill_(fill)
            c.v.fill_(fill)

    def packed(self, name):
        """The windows' rows of "k" or "v" [rows, G, D] (cuda)."""
        parts = [kv[name][c:] for kv, c in zip(self.kv, self.ctx_list)]
        return torch.cat(parts).cuda() if self.rows else torch.zeros((0, self.G, self.D), dtype=torch.bfloat16).cuda()

    def write_all(self):
        """Writes contexts and windows through the library, in two calls."""
        from speculative_decoding_markov_gb300 import binding as sdm
        zero = torch.zeros_like(self.ctx)
        R = len(self.w)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(self.ctx_list)]), dtype=torch.int32, device="cuda")
        if int(cu[-1]) > 0:
            rows = {n: torch.cat([self.kv[i][n][:self.ctx_list[i]] for i in range(R)]).cuda() for n in "kv"}
            sdm.cache_write(self.cache, rows["k"], rows["v"], cu, zero, dev_status=self.status)
        if self.rows:
            sdm.cache_write(self.cache, self.packed("k"), self.packed("v"), self.cu, self.ctx, dev_status=self.status)

    def held(self, i, name):
        return held(self.kv[i][name], self.e4m3)


def visible(w, ctx, window=0, sinks=0, mask=None):
    """[w, ctx + w] bool: whether window row p sees token j (mask: int32 words
    [nodes, words] of the request's tree, or None)."""
    n = ctx + w
    key = np.arange(n)[None]
    if mask is None:
        pos = ctx + np.arange(w)[:, None]
        see = key <= pos
        if window > 0:
            see &= (pos - key < window) | (key < sinks)
        return see
    bits = ((mask[:w, :, None].astype(np.int64) >> np.arange(32)) & 1).reshape(w, -1).astype(bool)
    pos = ctx + np.maximum(0, bits.sum(1) - 1)[:, None]
    see = np.ones((w, n), bool)
    if window > 0:
        see &= (pos - key < window) | (key < sinks)
    see[:, ctx:] = bits[:, :w]
    return see


def attend(q, k, v, see, scale):
    """q [w, H, D], k, v [n, G, D] (64 bits), see [w, n]: out [w, H, D], lse
    [w, H] and sum_j p_j |v_j| (the scale of the weights' rounding).  Tokens
    that a row does not see take no part, whatever they hold."""
    w, H, D = q.shape
    G = k.shape[1]
    rep = H // G
    out, lse, size = (np.zeros((w, H, D)), np.full((w, H), -np.inf), np.zeros((w, H, D)))
    q, k, v = (t.double().cpu().numpy() for t in (q, k, v))
    for p in range(w):
        at = np.nonzero(see[p])[0]
        if at.size == 0:
            continue
        for g in range(G):
            s = scale * (q[p, g * rep:(g + 1) * rep] @ k[at, g].T)
            with np.errstate(invalid="ignore"):
                m = s.max(-1, keepdims=True)
                e = np.exp(s - m)
                l = e.sum(-1, keepdims=True)
                out[p, g * rep:(g + 1) * rep] = (e / l) @ v[at, g]
                size[p, g * rep:(g + 1) * rep] = (e / l) @ np.abs(v[at, g])
                lse[p, g * rep:(g + 1) * rep] = (m + np.log(l))[:, 0]
    return out, lse, size


def random_trees(R, S, depth, rng, vocab=1000):
    """Draft trees in rank order: tok, parent [R, S], mask words, n_nodes."""
    tok, parent = np.zeros((R, S), np.int32), np.full((R, S), -1, np.int32)
    anc = np.zeros((R, S, S), bool)
    for i in range(R):
        d = np.zeros(S, int)
        tok[i] = rng.permutation(vocab)[:S]
        anc[i, 0, 0] = True
        for c in range(1, S):
            p = int(rng.integers(0, c))
            while d[p] >= depth:
                p = int(rng.integers(0, c))
            parent[i, c], d[c] = p, d[p] + 1
            anc[i, c] = anc[i, p]
            anc[i, c, c] = True
    words = (S + 31) // 32
    bits = np.zeros((R, S, words * 32), np.uint64)
    bits[:, :, :S] = anc
    mask = (bits.reshape(R, S, words, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32).view(np.int32)
    return dict(tok=tok, parent=parent, mask=mask, n_nodes=np.full((R,), S, np.int32))

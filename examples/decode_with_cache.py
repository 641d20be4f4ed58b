"""Speculative decoding of a small attention model, three ways, on one GPU.

    python examples/decode_with_cache.py

The target is one attention layer over a paged key/value cache: a token's
embedding gives its query, key and value, the attention's output plus the
embedding gives its logits.  Its greedy continuation is decoded

  one     a token at a time (windows of one row),
  chain   with the Markov head's chain drafts: draft_chain, pack_ragged,
          cache_write, attend over the ragged windows, verify,
  tree    with PCTree drafts: draft_tree, cache_write, attend under the
          tree's ancestor mask, verify_tree, cache_commit,

and the three must agree, since speculative decoding changes the speed and
not the result.  The cache is bf16 or (--cache e4m3) 8-bit.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from speculative_decoding_markov_gb300 import binding as sdm  # noqa: E402

R, V, RANK = 6, 4096, 64                 # requests, vocabulary, the Markov head's rank
H, KV, D, PAGE = 8, 2, 64, 16            # query heads, kv heads, head dim, tokens per page
B = 5                                    # drafts per chain; levels of a tree


class Model:
    """The target's weights and the drafter's Markov tables and backbone."""

    def __init__(self, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        hidden = H * D
        self.embed = (rnd(V, hidden)).to(torch.bfloat16)
        self.qkv = (rnd(hidden, (H + 2 * KV) * D) / hidden ** 0.5).to(torch.bfloat16)
        self.out = (rnd(hidden, V) / hidden ** 0.5).to(torch.bfloat16)
        # The drafter: a token's likely successors, learnt from the target alone
        # (without attention), as logits that depend on the last token only.
        self.U = (rnd(V, RANK) / RANK).to(torch.bfloat16)
        self.W = (rnd(RANK, V) / RANK).to(torch.bfloat16)

    def project(self, tok):
        """Queries, keys and values of tokens [n]: slices of one product."""
        x = (self.embed[tok.long()] @ self.qkv).view(-1, H + 2 * KV, D)
        return x[:, :H], x[:, H:H + KV], x[:, H + KV:]

    def logits(self, tok, attention):
        return (self.embed[tok.long()] + attention.reshape(-1, H * D)) @ self.out

    def backbone(self, anchor, noise):
        """Draft logits [R, B, V]: the target's own logits without attention,
        for the anchor, with noise (a drafter is right some of the time)."""
        base = (self.embed[anchor.long()] @ self.out).float()
        return (base[:, None] + noise).to(torch.bfloat16)


class State:
    def __init__(self, first, tokens, dtype):
        pages = (tokens + PAGE - 1) // PAGE
        table = torch.randperm(R * pages, device="cuda").to(torch.int32).view(R, pages).contiguous()
        self.cache = sdm.PagedCache.empty(R * pages, KV, PAGE, D, table, dtype)
        self.length = torch.zeros(R, dtype=torch.int32, device="cuda")     # tokens in the cache
        self.last = first.clone()                                          # the next token, not in it yet
        self.status = sdm.new_status()
        self.text = [[int(t)] for t in first.tolist()]

    def committed(self, out_tok, n_out):
        for i, (row, n) in enumerate(zip(out_tok.tolist(), n_out.tolist())):
            self.text[i] += row[:n]
        self.last = out_tok.gather(1, (n_out.long() - 1)[:, None])[:, 0].contiguous()


def attend_window(m, s, tok, cu, longest, tree_mask=None):
    """The target forward of packed windows: writes their keys and values,
    attends, returns the logits."""
    q, k, v = m.project(tok)
    sdm.cache_write(s.cache, k, v, cu, s.length, dev_status=s.status)
    o = sdm.attend(s.cache, q, cu, s.length, longest, tree_mask=tree_mask, dev_status=s.status)
    return m.logits(tok, o["out"])


def step_one(m, s):
    cu = torch.arange(R + 1, dtype=torch.int32, device="cuda")
    nxt = attend_window(m, s, s.last, cu, 1).float().argmax(-1).to(torch.int32)
    s.length += 1
    s.committed(nxt[:, None], torch.ones_like(nxt))


def step_chain(m, s, noise, tiers):
    L = m.backbone(s.last, noise)
    drafts = sdm.draft_chain(L, m.U, m.W, s.last)["tokens"]
    budget = torch.full((R,), B, dtype=torch.int32, device="cuda")
    budget[::2] = B - 2                                                    # ragged windows
    pk = sdm.pack_ragged(s.last, drafts, budget, tiers)
    rows = int(pk["cu_seqlens"][-1])
    logits = attend_window(m, s, pk["packed_tok"][:rows], pk["cu_seqlens"], B + 1)
    got = sdm.verify(sdm.COMPACT, sdm.GREEDY, logits.contiguous(), pk["cu_seqlens"], s.last, drafts)
    s.length += got["n_out"]             # the root and the accepted drafts: a prefix of the window
    s.committed(got["out_tok"], got["n_out"])


def step_tree(m, s, noise):
    N = 20
    L = m.backbone(s.last, noise)
    t = sdm.draft_tree(L, m.U, m.W, s.last, k=4, P=8, N=N)
    cu = torch.arange(R + 1, dtype=torch.int32, device="cuda") * (N + 1)
    logits = attend_window(m, s, t["tok"].clamp(min=0).view(-1), cu, N + 1, tree_mask=t["mask"])
    got = sdm.verify_tree(logits.view(R, N + 1, V), t["tok"], t["parent"], t["n_nodes"], B)
    done = sdm.cache_commit(s.cache, t["tok"], t["parent"], t["n_nodes"], got["out_tok"], got["accept"], s.length,
                            dev_status=s.status)
    s.length = done["length"]
    s.committed(got["out_tok"], got["n_out"])


def main(tokens=48, cache="bf16", seed=0):
    """Decodes `tokens` tokens per request each way; returns the texts and the
    steps that each way took."""
    dtype = torch.bfloat16 if cache == "bf16" else torch.float8_e4m3fn
    m = Model(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    first = torch.randint(0, V, (R,), generator=g, device="cuda", dtype=torch.int32)
    tiers = torch.tensor([16, 32, 64], dtype=torch.int32, device="cuda")
    texts, steps = {}, {}
    for way in ("one", "chain", "tree"):
        s = State(first, tokens + 32, dtype)
        steps[way] = 0
        while min(len(t) for t in s.text) <= tokens:
            # requests that are ahead go on: their text is cut at the end
            if max(int(x) for x in s.length) + 32 > s.cache.table.shape[1] * PAGE:
                break
            noise = torch.randn((R, B, V), generator=g, device="cuda") * 0.2
            if way == "one":
                step_one(m, s)
            elif way == "chain":
                step_chain(m, s, noise, tiers)
            else:
                step_tree(m, s, noise)
            steps[way] += 1
        if s.status.item():
            raise RuntimeError(f"device status {s.status.item()}")
        texts[way] = s.text
    return texts, steps


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=48)
    p.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    a = p.parse_args()
    texts, steps = main(a.tokens, a.cache)
    for way in texts:
        n = [min(len(t), len(u)) for t, u in zip(texts[way], texts["one"])]
        same = all(t[:k] == u[:k] for t, u, k in zip(texts[way], texts["one"], n))
        print(f"{way:6s} {steps[way]:4d} steps for {min(n) - 1} tokens of every request, "
              f"{'the same text' if same else 'ANOTHER TEXT'}")

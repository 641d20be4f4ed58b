"""The paged key/value cache operators: what is timed, on which inputs, and what they compute.

Three operators over one cache (keys and values in pages of `page` tokens, [pages, kv heads, page, head dim], held in
bf16 or in 8-bit floating point (e4m3) with one power-of-two scale per token and kv head):

  attend  attention of each request's window of new tokens over its cached context and the window itself: causal or by
          a draft tree's ancestor mask, optionally over a sliding window of positions and a few first tokens
  cache   new keys and values written into the pages (quantised as they are written), then tokens read back
  commit  a draft tree's keys and values written, then those of the accepted path moved to follow the context

A case fixes every length (`mix` seeds their spread); a seed fixes the values, the page order and the trees.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
EXP_LO, EXP_HI = -110, 119      # the scale exponents that a cache row may have
VOCAB = 151936


def listed():
    base = dict(op="attend", tree=False, window=0, sinks=0, read="", mix=1)
    return [
        # decoding one token of one short conversation: nothing but latency
        dict(base, name="attend_one_token", R=1, w_lo=1, w_hi=1, c_lo=500, c_hi=500, H=32, G=8, D=128, page=16,
             cache="bf16"),
        # the headline cycle's verification: 64 requests, windows of a root and up to 7 drafts, uneven contexts
        dict(base, name="attend_verify_64", R=64, w_lo=1, w_hi=8, c_lo=300, c_hi=8000, H=32, G=8, D=128, page=64,
             cache="bf16"),
        # the mixed traffic's verification: 256 requests, a root and up to 8 drafts, an 8-bit cache, 7 heads share one
        dict(base, name="attend_verify_256_e4m3", R=256, w_lo=1, w_hi=9, c_lo=200, c_hi=4000, H=28, G=4, D=128,
             page=32, cache="e4m3"),
        # the drafting tree's verification: 32 requests, a root and 64 nodes under the ancestor mask
        dict(base, name="attend_tree_32", R=32, w_lo=65, w_hi=65, c_lo=500, c_hi=4000, H=32, G=8, D=128, page=64,
             cache="bf16", tree=True),
        # one token each of two long documents, an 8-bit cache: few rows, a long axis
        dict(base, name="attend_long_e4m3", R=2, w_lo=1, w_hi=1, c_lo=150001, c_hi=199999, H=28, G=4, D=128,
             page=128, cache="e4m3"),
        # a chunk of a long prompt in a model with sliding windows and kept first tokens, 64-wide heads
        dict(base, name="attend_chunk_sinks", R=1, w_lo=4001, w_hi=4001, c_lo=6007, c_hi=6007, H=64, G=8, D=64,
             page=16, cache="bf16", window=1024, sinks=4),
        # chunks of several prompts at once, on contexts of very different lengths, an 8-bit cache
        dict(base, name="attend_chunks_e4m3", R=5, w_lo=37, w_hi=1500, c_lo=0, c_hi=4000, H=32, G=8, D=128, page=64,
             cache="e4m3"),
        # a whole prompt of 8192 tokens at once: the largest product
        dict(base, name="attend_prompt_8192", R=1, w_lo=8192, w_hi=8192, c_lo=0, c_hi=0, H=32, G=8, D=128, page=128,
             cache="bf16"),
        # what one decode cycle of 64 requests writes in one layer
        dict(base, name="cache_step_64", op="cache", read="new", R=64, w_lo=1, w_hi=8, c_lo=300, c_hi=8000, H=32, G=8,
             D=128, page=64, cache="bf16"),
        # prompts' chunks written in 8 bits and the whole prefixes read back (to hand them to another worker)
        dict(base, name="cache_prefix_e4m3", op="cache", read="all", R=6, w_lo=1, w_hi=8192, c_lo=100, c_hi=30000,
             H=32, G=8, D=128, page=64, cache="e4m3"),
        # the accepted paths of four small trees in an 8-bit cache
        dict(base, name="commit_tree_4_e4m3", op="commit", R=4, w_lo=17, w_hi=17, c_lo=100, c_hi=900, H=28, G=4,
             D=128, page=16, cache="e4m3", tree=True),
        # the accepted paths of the drafting tree's 32 requests
        dict(base, name="commit_tree_32", op="commit", R=32, w_lo=65, w_hi=65, c_lo=500, c_hi=4000, H=32, G=8, D=128,
             page=64, cache="bf16", tree=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the same ranges: single tokens, verify windows, trees, chunks of prompts; writes and commits."""
    cap = 1.0e9                                                # the largest listed case's cost in bytes, or less
    for _ in range(1000):
        H, G, D = rng.choice([(32, 8, 128), (28, 4, 128), (16, 16, 64), (64, 8, 64), (12, 2, 64), (8, 1, 128),
                              (40, 8, 128), (4, 4, 128)])
        c = dict(op=rng.choice(["attend", "attend", "attend", "cache", "commit"]), tree=False, window=0, sinks=0,
                 read="", mix=rng.randrange(1, 1 << 20), H=H, G=G, D=D, page=rng.choice([16, 32, 64, 128]),
                 cache=rng.choice(["bf16", "e4m3"]))
        kind = "tree" if c["op"] == "commit" else rng.choice(["one", "verify", "tree", "chunk"])
        if kind == "one":
            c.update(R=_log(rng, 1, 256), w_lo=1, w_hi=1)
            hi = _log(rng, 16, 200000)
        elif kind == "verify":
            c.update(R=_log(rng, 1, 256), w_lo=1, w_hi=rng.randrange(2, 18))
            hi = _log(rng, 16, 60000)
        elif kind == "tree":
            s = rng.randrange(5, 66)
            c.update(R=_log(rng, 1, 64), w_lo=s, w_hi=s, tree=True)
            hi = _log(rng, 16, 20000)
        else:
            w = _log(rng, 18, 8192)
            c.update(R=_log(rng, 1, 8), w_lo=max(1, w // rng.choice([1, 2, 20])), w_hi=w)
            hi = rng.choice([0, _log(rng, 16, 30000)])
        c.update(c_lo=hi // rng.choice([1, 3, 30]), c_hi=hi)
        if c["op"] == "attend" and rng.random() < 0.35:
            c.update(window=_log(rng, 16, 4096), sinks=rng.choice([0, 1, 4, 33]))
        if c["op"] == "cache":
            c["read"] = rng.choice(["new", "all"])
            c["tree"] = False
        w, ctx = lengths(c)
        longest = max(a + b for a, b in zip(w, ctx))
        n = work(c)
        plain = c["R"] * longest * G * D * 8 + (c["R"] * max(w) * H * longest * 8 if c["op"] == "attend" else 0)
        if max(n["bytes"], n["flops"] / 300) < cap and plain < 3e10:
            return c
    raise RuntimeError("no case drawn")


def lengths(case):
    """Each request's window and context: windows uniform, contexts spread over their logarithm, by `mix` alone."""
    rng = random.Random(case["mix"])
    w = [rng.randint(case["w_lo"], case["w_hi"]) for _ in range(case["R"])]
    lo, hi = case["c_lo"], case["c_hi"]
    ctx = [min(hi, max(lo, int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** rng.random())) - 1)) for _ in range(case["R"])]
    return w, ctx


def work(case):
    """Keys, values and scales that some row sees, queries and outputs, once each; two products per visible pair."""
    w, ctx = lengths(case)
    H, G, D = case["H"], case["G"], case["D"]
    per = (D if case["cache"] == "e4m3" else 2 * D) + (1 if case["cache"] == "e4m3" else 0)
    per *= 2 * G                                                # one token's key and value rows of every kv head
    new = sum(w)
    if case["op"] == "cache":
        back = new + (sum(ctx) if case["read"] == "all" else 0)
        return {"bytes": new * (4 * G * D + per) + back * (per + 4 * G * D), "flops": 0}
    if case["op"] == "commit":
        depth = min(16, case["w_hi"] - 1)                       # an accepted path is at most this long
        moved = case["R"] * max(1, depth // 2)
        back = case["R"] * (depth + 1) if case["cache"] == "e4m3" else 0
        return {"bytes": new * (4 * G * D + per) + 2 * moved * per + back * (per + 4 * G * D), "flops": 0}
    win = case["window"] if case["window"] > 0 else 1 << 60
    keys = pairs = 0
    for n, c in zip(w, ctx):
        first = max(0, c - win + 1)                             # the first key inside the first row's window
        keys += c + n - first + min(case["sinks"], first)
        if case["tree"]:
            pairs += n * (min(c, win) + min(case["sinks"], first) + 8)
        else:
            full = max(0, min(n, win - c))                      # rows that see every key up to their own
            pairs += full * c + full * (full + 1) // 2
            rest = n - full
            pairs += rest * win
            lo = c + full - win + 1                             # the first of the rest sees keys from here on
            if rest > 0:
                s = case["sinks"]
                ramp = max(0, min(rest, s - lo))                # rows whose window still covers some of the sinks
                pairs += ramp * lo + ramp * (ramp - 1) // 2 + (rest - ramp) * s
    return {"bytes": keys * per + new * H * D * 4 + new * H * 4, "flops": 4.0 * pairs * H * D}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _pow2(e):
    """2^e in 32 bits, exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    """Rows of the last axis as e4m3 codes and their scales' exponents (elementary operations in 32 bits)."""
    x = x.float()
    mant, power = torch.frexp(x.abs().amax(-1))
    e = torch.where(mant <= 0.875, power - 9, power - 8)        # the least e with max |x| <= 448 2^e
    e = e.clamp(EXP_LO, EXP_HI)
    y = (x * _pow2(-e)[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
    return y.to(torch.float8_e4m3fn), e


def _trees(case, seed, n_depth):
    """Random draft trees in rank order: tokens (distinct in a tree), parents, ancestor bits, a path that is accepted."""
    R, S = case["R"], case["w_hi"]
    rng = np.random.RandomState((seed * 7919 + case["mix"]) % (1 << 31))
    parent, depth = np.full((R, S), -1, np.int32), np.zeros((R, S), np.int32)
    anc = np.zeros((R, S, S), bool)
    anc[:, 0, 0] = True
    row = np.arange(R)
    for c in range(1, S):
        p = (c * rng.random_sample(R) ** 1.5).astype(np.int64)  # rather a young node than an old one
        p = np.where(depth[row, p] >= n_depth, 0, p)
        parent[:, c], depth[:, c] = p, depth[row, p] + 1
        anc[:, c] = anc[row, p]
        anc[:, c, c] = True
    tok = np.stack([rng.permutation(VOCAB)[:S] for _ in range(R)]).astype(np.int32)
    words = (S + 31) // 32
    bits = np.zeros((R, S, words * 32), np.uint64)
    bits[:, :, :S] = anc
    mask = (bits.reshape(R, S, words, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32).view(np.int32)
    end = rng.randint(0, S, R)                                  # the accepted path ends at this node
    accept = depth[row, end].astype(np.int32)
    out_tok = np.full((R, n_depth + 1), -1, np.int32)
    for i in range(R):
        at = end[i]
        while at > 0:
            out_tok[i, depth[i, at] - 1] = tok[i, at]
            at = parent[i, at]
        out_tok[i, accept[i]] = VOCAB + 7                       # the bonus token: no node's
    return dict(tok=tok, parent=parent, mask=mask, accept=accept, out_tok=out_tok,
                n_nodes=np.full((R,), S, np.int32))


def prepare(case, seed):
    """Pools of pages in use, the page table, packed rows as a fused projection leaves them, lengths; for the
    framework's own calls also the cache's handle, the outputs' buffers and the workspace."""
    w, ctx = lengths(case)
    R, H, G, D, page = case["R"], case["H"], case["G"], case["D"], case["page"]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + case["mix"])
    per_req = [(a + b + page - 1) // page for a, b in zip(w, ctx)]
    n_pages, most = sum(per_req) + 3, max(per_req)
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    start = torch.tensor([sum(per_req[:i]) for i in range(R)], device="cuda")
    used = torch.tensor(per_req, device="cuda")
    at = torch.arange(most, device="cuda")
    table = torch.where(at[None] < used[:, None], order[(start[:, None] + at[None]).clamp(max=n_pages - 1)], 0)
    s = dict(case=case, table=table.to(torch.int32).contiguous(), max_w=max(w), rows=sum(w),
             ctx=torch.tensor(ctx, dtype=torch.int32, device="cuda"),
             cu=torch.tensor([sum(w[:i]) for i in range(R + 1)], dtype=torch.int32, device="cuda"),
             req=torch.repeat_interleave(torch.arange(R, device="cuda"), torch.tensor(w, device="cuda")),
             most_len=max(a + b for a, b in zip(w, ctx)))
    s["pos"] = torch.arange(s["rows"], device="cuda") - s["cu"].long()[s["req"]]
    shape = (n_pages, G, page, D)
    for name in ("k", "v"):
        pool = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
        # tokens differ in size, as activations do
        pool *= torch.exp2(torch.randint(-1, 2, shape[:3], generator=gen, device="cuda").to(torch.bfloat16))[..., None]
        if case["cache"] == "e4m3":
            code, e = _quantise(pool)
            s[name], s[name + "_exp"] = code, (e + 127).to(torch.uint8)
        else:
            s[name], s[name + "_exp"] = pool, None
    # queries, keys and values of the new tokens: slices of one projection's output
    qkv = torch.randn((s["rows"], H + 2 * G, D), generator=gen, device="cuda", dtype=torch.bfloat16)
    s["q"], s["new_k"], s["new_v"] = qkv[:, :H], qkv[:, H:H + G], qkv[:, H + G:]
    s["scale"] = 1.0 / math.sqrt(D)
    if case["tree"]:
        t = _trees(case, seed, min(16, case["w_hi"] - 1))
        s.update({k: torch.as_tensor(v).cuda() for k, v in t.items()})
    # which tokens a pass reads back: `first` and how many of each request
    whole = case["read"] == "all"
    first = [0 if whole else c for c in ctx]
    count = [a + b for a, b in zip(w, ctx)] if whole else w
    s["first"] = torch.tensor(first, dtype=torch.int32, device="cuda")
    s["back_cu"] = torch.tensor([sum(count[:i]) for i in range(R + 1)], dtype=torch.int32, device="cuda")
    s["back_rows"] = sum(count)
    s["back_req"] = torch.repeat_interleave(torch.arange(R, device="cuda"), torch.tensor(count, device="cuda"))
    s["back_pos"] = (torch.arange(s["back_rows"], device="cuda") - s["back_cu"].long()[s["back_req"]]
                     + s["first"].long()[s["back_req"]])
    if own:
        from speculative_decoding_markov_gb300 import binding as sdm
        s["handle"] = sdm.PagedCache(s["k"], s["v"], s["table"], s["k_exp"], s["v_exp"])
        s["status"] = sdm.new_status()
        if case["op"] == "attend":
            s["out"] = dict(out=torch.empty((s["rows"], H, D), dtype=torch.bfloat16, device="cuda"),
                            lse=torch.empty((s["rows"], H), dtype=torch.float32, device="cuda"))
            s["ws"] = sdm.attend_workspace(s["handle"], s["rows"], s["max_w"], H)
        elif case["op"] == "cache" or case["cache"] == "e4m3":
            s["out"] = dict(k=torch.empty((s["back_rows"], G, D), dtype=torch.bfloat16, device="cuda"),
                            v=torch.empty((s["back_rows"], G, D), dtype=torch.bfloat16, device="cuda"))
        if case["op"] == "commit":
            s["done"] = dict(path=torch.empty_like(s["out_tok"]), length=torch.empty_like(s["ctx"]))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _place(s, req, pos):
    """Page and slot of tokens `pos` of requests `req`."""
    page = s["case"]["page"]
    return s["table"].long()[req, pos // page], pos % page


def _tokens(s, name, req, pos):
    """Rows [..., kv heads, head dim] of the cache in 32 bits."""
    page, slot = _place(s, req, pos)
    x = s[name].view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn) if s["case"]["cache"] == "e4m3" \
        else s[name][page, :, slot]
    x = x.float()
    if s[name + "_exp"] is not None:
        x = x * _pow2(s[name + "_exp"][page, :, slot].int() - 127)[..., None]
    return x


def _write(s):
    page, slot = _place(s, s["req"], s["ctx"].long()[s["req"]] + s["pos"])
    for name in ("k", "v"):
        x = s["new_" + name]
        if s["case"]["cache"] == "e4m3":
            code, e = _quantise(x)
            s[name].view(torch.uint8)[page, :, slot] = code.view(torch.uint8)
            s[name + "_exp"][page, :, slot] = (e + 127).to(torch.uint8)
        else:
            s[name][page, :, slot] = x


def _read(s):
    return {n: _tokens(s, n, s["back_req"], s["back_pos"]).to(torch.bfloat16) for n in ("k", "v")}


def _visible(s, L):
    """[R, rows of a window, L]: whether a row of the window sees the token at a position."""
    c = s["case"]
    key = torch.arange(L, device="cuda")[None, None]
    ctx = s["ctx"].long()[:, None, None]
    row = torch.arange(s["max_w"], device="cuda")[None, :, None]
    if c["tree"]:
        S, words = s["mask"].shape[1:]
        bits = (s["mask"][..., None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        bits = bits.reshape(c["R"], S, words * 32)
        depth = (bits.sum(-1, keepdim=True) - 1).clamp(min=0)
        at = (key - ctx).expand(c["R"], 1, L)
        inside = (at >= 0) & (at < words * 32)
        node = torch.gather(bits, 2, at.clamp(0, words * 32 - 1).expand(c["R"], S, L)) == 1
        pos, seen = ctx + depth, torch.where(inside, node, at < 0)
        old = at < 0
    else:
        pos = ctx + row
        seen, old = key <= pos, True
    if c["window"] > 0:
        near = (pos - key < c["window"]) | (key < c["sinks"])
        seen = seen & (near | ~old if c["tree"] else near)
    return seen


def _attend(s):
    c = s["case"]
    R, H, G, D, W = c["R"], c["H"], c["G"], c["D"], s["max_w"]
    L, group = s["most_len"], H // G
    key = torch.arange(L, device="cuda")
    last = (s["ctx"].long() + (s["cu"][1:] - s["cu"][:-1]).long() - 1)[:, None]
    k, v = (_tokens(s, n, torch.arange(R, device="cuda")[:, None], torch.minimum(key[None], last)) for n in "kv")
    q = torch.zeros((R, W, H, D), device="cuda")
    q[s["req"], s["pos"]] = s["q"].float()
    q = q.view(R, W, G, group, D).permute(0, 2, 1, 3, 4).reshape(R, G, W * group, D)
    x = (q @ k.permute(0, 2, 3, 1)).mul_(s["scale"]).view(R, G, W, group, L)
    x.masked_fill_(~_visible(s, L)[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    lse = torch.log(total) + top
    out = (x.view(R, G, W * group, L) @ v.permute(0, 2, 1, 3)).view(R, G, W, group, D)
    out = torch.where(total > 0, out / total, 0.0)
    back = lambda t: t.permute(0, 2, 1, 3, 4).reshape(R, W, H, -1)[s["req"], s["pos"]]  # noqa: E731
    return {"out": back(out).to(torch.bfloat16), "lse": back(lse)[..., 0]}


def _commit(s):
    """The accepted path: the nodes all of whose ancestors (and themselves) carry the committed tokens in turn."""
    R, S = s["tok"].shape
    words = s["mask"].shape[2]
    bits = ((s["mask"][..., None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1).reshape(R, S, words * 32)
    bits = bits[..., :S].bool()
    depth = bits.sum(-1) - 1
    said = torch.gather(s["out_tok"], 1, (depth - 1).clamp(min=0))
    fits = ((s["tok"] == said) & (depth <= s["accept"][:, None])) | (depth == 0)
    on = (~bits | fits[:, None]).all(-1)
    n = s["out_tok"].shape[1]
    node = torch.where(on, torch.arange(S, device="cuda")[None], S).to(torch.int32).sort(-1)[0]
    path = torch.full((R, n), -1, dtype=torch.int32, device="cuda")
    path[:, :min(n, S)] = node[:, :n]
    step = torch.arange(n, device="cuda")[None]
    path = torch.where(step <= s["accept"][:, None], path, -1)
    req, j = torch.nonzero(path >= 0, as_tuple=True)
    src = _place(s, req, s["ctx"].long()[req] + path[req, j])
    dst = _place(s, req, s["ctx"].long()[req] + j)
    for name in ("k", "v", "k_exp", "v_exp"):
        if s[name] is not None:
            x = s[name].view(torch.uint8) if s[name].dtype == torch.float8_e4m3fn else s[name]
            x[dst[0], :, dst[1]] = x[src[0], :, src[1]]
    return path, s["ctx"] + s["accept"] + 1


def run(state):
    s, case = state, state["case"]
    if own:
        from speculative_decoding_markov_gb300 import binding as sdm
        if case["op"] == "attend":
            return sdm.attend(s["handle"], s["q"], s["cu"], s["ctx"], s["max_w"], scale=s["scale"],
                              window=case["window"], sinks=case["sinks"], tree_mask=s.get("mask"), out=s["out"],
                              ws=s["ws"], dev_status=s["status"], lse=True)
        sdm.cache_write(s["handle"], s["new_k"], s["new_v"], s["cu"], s["ctx"], dev_status=s["status"])
        if case["op"] == "cache":
            got = sdm.cache_read(s["handle"], s["back_cu"], s["back_rows"], first=s["first"], out=s["out"],
                                 dev_status=s["status"])
            return [got] + ([s["k"], s["v"]] if case["cache"] == "bf16" else [])
        done = sdm.cache_commit(s["handle"], s["tok"], s["parent"], s["n_nodes"], s["out_tok"], s["accept"],
                                s["ctx"], out=s["done"], dev_status=s["status"])
        got = [done["path"], done["length"]]
        if case["cache"] == "bf16":
            return got + [s["k"], s["v"]]
        return got + [sdm.cache_read(s["handle"], s["back_cu"], s["back_rows"], first=s["first"], out=s["out"],
                                     dev_status=s["status"])]
    if case["op"] == "attend":
        return _attend(s)
    _write(s)
    if case["op"] == "cache":
        return [_read(s)] + ([s["k"], s["v"]] if case["cache"] == "bf16" else [])
    got = list(_commit(s))
    return got + ([s["k"], s["v"]] if case["cache"] == "bf16" else [_read(s)])


# ---------------------------------------------------------------------------
# the definitions in 64 bits, request by request
# ---------------------------------------------------------------------------
def _two64(e):
    """2^e in 64 bits, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _held64(x, kind):
    """What the cache holds for rows x: themselves, or the nearest multiples on the 8-bit grid."""
    x = x.double()
    if kind == "bf16":
        return x
    top = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / E4M3_MAX))
    e = torch.where(top > E4M3_MAX * _two64(e), e + 1, torch.where(top <= E4M3_MAX * _two64(e - 1), e - 1, e))
    e = torch.where(top > 0, e, 0.0).clamp(EXP_LO, EXP_HI)
    y = (x * _two64(-e)).clamp(-E4M3_MAX, E4M3_MAX)
    step = _two64(torch.floor(torch.log2(torch.where(y != 0, y.abs(), 1.0))).clamp(min=-6) - 3)
    return torch.round(y / step) * step * _two64(e)


def _pool64(s, name):
    x = s[name].double()
    if s[name + "_exp"] is not None:
        x = x * _two64(s[name + "_exp"].long() - 127)[..., None]
    return x


def exact(case, seed):
    s = prepare(case, seed)
    w, ctx = lengths(case)
    G, D, page, group = case["G"], case["D"], case["page"], case["H"] // case["G"]
    table = s["table"].long()
    if case["op"] == "attend":
        outs, lses, row = [], [], 0
        for i in range(case["R"]):
            n = w[i] + ctx[i]
            ids = table[i, :(n + page - 1) // page]
            kv = {}
            for name in "kv":
                x = s[name][ids].double()
                if s[name + "_exp"] is not None:
                    x = x * _two64(s[name + "_exp"][ids].long() - 127)[..., None]
                kv[name] = x.permute(1, 0, 2, 3).reshape(G, -1, D)[:, :n]
            q = s["q"][row:row + w[i]].double().view(w[i], G, group, D)
            key = torch.arange(n, device="cuda")
            if case["tree"]:
                bits = s["mask"][i, :w[i]].long() & 0xFFFFFFFF
                c = torch.arange(w[i], device="cuda")
                node = (bits[:, c // 32] >> (c % 32)) & 1
                where_ = ctx[i] + node.sum(1) - 1
                see = torch.cat([torch.ones(w[i], ctx[i], device="cuda", dtype=torch.bool), node.bool()], 1)
                if case["window"]:
                    far = (key[None, :ctx[i]] <= where_[:, None] - case["window"]) & (key[:ctx[i]] >= case["sinks"])
                    see[:, :ctx[i]] &= ~far
            else:
                where_ = ctx[i] + torch.arange(w[i], device="cuda")
                see = key[None] <= where_[:, None]
                if case["window"]:
                    see &= (key[None] > where_[:, None] - case["window"]) | (key < case["sinks"])
            o = torch.empty((w[i], G, group, D), dtype=torch.float64, device="cuda")
            z = torch.empty((w[i], G, group), dtype=torch.float64, device="cuda")
            for h in range(G):
                for part in range(0, w[i], 1024):
                    x = torch.einsum("wgd,nd->wgn", q[part:part + 1024, h], kv["k"][h]) * s["scale"]
                    x = x.masked_fill(~see[part:part + 1024, None], -math.inf)
                    z[part:part + 1024, h] = torch.logsumexp(x, -1)
                    o[part:part + 1024, h] = torch.softmax(x, -1) @ kv["v"][h]
            outs.append(o.reshape(w[i], -1, D))
            lses.append(z.reshape(w[i], -1))
            row += w[i]
        return {"out": torch.cat(outs), "lse": torch.cat(lses)}
    pools = {name: _pool64(s, name) for name in "kv"}
    row, paths = 0, []
    for i in range(case["R"]):
        p = torch.arange(ctx[i], ctx[i] + w[i], device="cuda")
        for name in "kv":
            pools[name][table[i, p // page], :, p % page] = _held64(s["new_" + name][row:row + w[i]], case["cache"])
        row += w[i]
        if case["op"] == "commit":
            par, tok = s["parent"][i].tolist(), s["tok"][i].tolist()
            path = [0]
            for t in s["out_tok"][i].tolist()[:int(s["accept"][i])]:
                path.append(next(c for c in range(w[i]) if par[c] == path[-1] and tok[c] == t))
            paths.append(path)
            src, dst = ctx[i] + torch.tensor(path, device="cuda"), ctx[i] + torch.arange(len(path), device="cuda")
            for name in "kv":
                moved = pools[name][table[i, src // page], :, src % page]
                pools[name][table[i, dst // page], :, dst % page] = moved
    back = {}
    for name in "kv":
        back[name] = torch.cat([pools[name][table[i, p // page], :, p % page] for i in range(case["R"])
                                for p in [torch.arange(0 if case["read"] == "all" else ctx[i], ctx[i] + w[i],
                                                       device="cuda")]])
    if case["op"] == "cache":
        return [back] + ([pools["k"], pools["v"]] if case["cache"] == "bf16" else [])
    n = s["out_tok"].shape[1]
    path = torch.tensor([p + [-1] * (n - len(p)) for p in paths], dtype=torch.int32, device="cuda")
    got = [path, s["ctx"] + torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda")]
    return got + ([pools["k"], pools["v"]] if case["cache"] == "bf16" else [back])

"""Operators around the paged cache and the verification: what is timed, on which inputs, and what they compute.

  rotate    queries and keys of a window normalised per head (RMS, with a weight) and rotated by their positions, the
            keys and values written into the cache (bf16, or e4m3 with a power-of-two scale per token and head)
  logprobs  of the committed tokens: log probability, rank, the distribution's entropy, the most probable tokens
  weight    the attention weight that each cached token got from the committed rows, added to what it had
  evict     a cache cut to `keep` tokens per request and kv head: the first and the last positions, then those of
            largest weight; kept tokens behind slot `keep` move into the slots that become free

A case fixes every length (`mix` seeds their spread); a seed fixes the values, the page order and the paths.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
EXP_LO, EXP_HI = -110, 119      # the scale exponents that a cache row may have
EPS = 1e-6


def listed():
    base = dict(norm=True, rot=128, inter=False, path=False, window=0, sinks=0, mix=1)
    return [
        # decoding one token of one short conversation: nothing but latency
        dict(base, name="rotate_one_token", op="rotate", R=1, w_lo=1, w_hi=1, c_lo=500, c_hi=500, H=32, G=8, D=128,
             page=16, cache="bf16"),
        # the mixed traffic's step: 256 requests, a root and up to 8 drafts, an 8-bit cache, half of each head rotated
        dict(base, name="rotate_verify_256_e4m3", op="rotate", R=256, w_lo=1, w_hi=9, c_lo=200, c_hi=1000, H=28, G=4,
             D=128, page=32, cache="e4m3", norm=False, rot=64, inter=True),
        # a whole prompt of 8192 tokens
        dict(base, name="rotate_prompt_8192", op="rotate", R=1, w_lo=8192, w_hi=8192, c_lo=0, c_hi=0, H=32, G=8, D=128,
             page=128, cache="bf16"),
        # one committed token of one request with five alternatives
        dict(base, name="logprobs_one", op="logprobs", R=1, w_lo=1, w_hi=1, V=151936, top=5, temp=1.0, dt="bf16"),
        # what the headline cycle commits: 64 requests, 1 to 8 tokens each, with twenty alternatives
        dict(base, name="logprobs_step_64", op="logprobs", R=64, w_lo=1, w_hi=8, V=151936, top=20, temp=1.0, dt="bf16"),
        # a prompt of 1000 tokens scored, logits in 32 bits
        dict(base, name="logprobs_prompt_1000", op="logprobs", R=1, w_lo=1000, w_hi=1000, V=129280, top=1, temp=1.0,
             dt="fp32"),
        # one token over a short context
        dict(base, name="weight_one_token", op="weight", R=1, w_lo=1, w_hi=1, c_lo=500, c_hi=500, H=32, G=8, D=128,
             page=16, cache="bf16"),
        # the headline cycle's committed rows over uneven contexts
        dict(base, name="weight_verify_64", op="weight", R=64, w_lo=1, w_hi=8, c_lo=300, c_hi=8000, H=32, G=8, D=128,
             page=64, cache="bf16"),
        # one token each of two long documents, an 8-bit cache: few rows, a long axis
        dict(base, name="weight_long_e4m3", op="weight", R=2, w_lo=1, w_hi=1, c_lo=150001, c_hi=199999, H=28, G=4,
             D=128, page=128, cache="e4m3"),
        # a whole prompt of 8192 tokens at once: the largest product
        dict(base, name="weight_prompt_8192", op="weight", R=1, w_lo=8192, w_hi=8192, c_lo=0, c_hi=0, H=32, G=8, D=128,
             page=128, cache="bf16"),
        # after a decode cycle over full caches of 2048 tokens: what the cycle added has to go again
        dict(base, name="evict_step_64", op="evict", R=64, w_lo=1, w_hi=8, c_lo=2048, c_hi=2048, H=32, G=8, D=128,
             page=64, cache="bf16", keep=2048, first=4, recent=64),
        # five prompts read, each cut to 4096 tokens, an 8-bit cache
        dict(base, name="evict_prompts_e4m3", op="evict", R=5, w_lo=5000, w_hi=30000, c_lo=0, c_hi=0, H=28, G=4, D=128,
             page=32, cache="e4m3", keep=4096, first=4, recent=256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the same ranges: single tokens, verify windows, accepted paths of trees, chunks of prompts."""
    cap = 0.55e9                                                # the largest listed case's cost in bytes, or less
    for _ in range(1000):
        H, G, D = rng.choice([(32, 8, 128), (28, 4, 128), (16, 16, 64), (64, 8, 64), (12, 2, 64), (8, 1, 128),
                              (40, 8, 128), (4, 4, 128)])
        c = dict(op=rng.choice(["rotate", "logprobs", "weight", "weight", "evict"]), mix=rng.randrange(1, 1 << 20), H=H,
                 G=G, D=D, page=rng.choice([16, 32, 64, 128]), cache=rng.choice(["bf16", "e4m3"]), norm=True, rot=D,
                 inter=False, path=False, window=0, sinks=0)
        kind = rng.choice(["one", "verify", "path", "chunk"])
        if kind == "one":
            c.update(R=_log(rng, 1, 256), w_lo=1, w_hi=1)
            hi = _log(rng, 16, 200000)
        elif kind == "verify":
            c.update(R=_log(rng, 1, 256), w_lo=1, w_hi=rng.randrange(2, 18))
            hi = _log(rng, 16, 60000)
        elif kind == "path":
            c.update(R=_log(rng, 1, 64), w_lo=1, w_hi=rng.randrange(2, 18), path=True)
            hi = _log(rng, 16, 20000)
        else:
            w = _log(rng, 18, 8192)
            c.update(R=_log(rng, 1, 8), w_lo=max(1, w // rng.choice([1, 2, 20])), w_hi=w)
            hi = rng.choice([0, _log(rng, 16, 30000)])
        c.update(c_lo=hi // rng.choice([1, 3, 30]), c_hi=hi)
        if c["op"] == "rotate":
            c.update(path=False, norm=rng.random() < 0.6, rot=rng.choice([D, D, D // 2, 24]), inter=rng.random() < 0.4)
        if c["op"] == "logprobs":
            c.update(V=8 * _log(rng, 4, 32768), top=rng.choice([0, 1, 5, 20, 32]), temp=rng.choice([1.0, 0.7, 1.3]),
                     dt=rng.choice(["bf16", "fp32"]))
        if c["op"] == "weight" and rng.random() < 0.35:
            c.update(window=_log(rng, 16, 4096), sinks=rng.choice([0, 1, 4, 33]))
        if c["op"] == "evict":
            keep = max(2, _log(rng, 16, max(17, c["c_hi"] + c["w_hi"])))
            c.update(path=False, keep=keep, first=min(keep // 4, rng.choice([0, 1, 4])),
                     recent=min(keep // 4, rng.choice([0, 1, 16, 256])))
        w, ctx = lengths(c)
        longest = max(a + b for a, b in zip(w, ctx))
        n = work(c)
        plain = 0
        if c["op"] == "logprobs":
            plain = (sum(w) + c["R"] * c["w_hi"] * 3) * c["V"] * 16
        elif c["op"] == "weight":
            plain = c["R"] * longest * G * D * 8 + c["R"] * max(w) * H * longest * 8
        elif c["op"] == "evict":
            plain = c["R"] * G * longest * (D * 4 + 64)
        else:
            plain = c["R"] * longest * G * D * 4
        if max(n["bytes"], n["flops"] / 300) < cap and plain < 3e10:
            return c
    raise RuntimeError("no case drawn")


def lengths(case):
    """Each request's committed rows and context: rows uniform, contexts spread over their logarithm, by `mix` alone."""
    rng = random.Random(case["mix"])
    w = [rng.randint(case["w_lo"], case["w_hi"]) for _ in range(case["R"])]
    if case["op"] == "logprobs":
        return w, [0] * case["R"]
    lo, hi = case["c_lo"], case["c_hi"]
    ctx = [min(hi, max(lo, int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** rng.random())) - 1)) for _ in range(case["R"])]
    return w, ctx


def work(case):
    """Inputs once, outputs once; for `weight` one product per visible pair, for `evict` the rows that have to move."""
    w, ctx = lengths(case)
    new = sum(w)
    if case["op"] == "logprobs":
        out = 12 + 8 * case["top"]
        return {"bytes": new * case["V"] * (2 if case["dt"] == "bf16" else 4) + new * (4 + out),
                "flops": 5.0 * new * case["V"]}
    H, G, D = case["H"], case["G"], case["D"]
    per = D + 1 if case["cache"] == "e4m3" else 2 * D           # one key or value row in the cache
    if case["op"] == "rotate":
        back = new * 2 * G * (per + 2 * D) if case["cache"] == "e4m3" else 0
        return {"bytes": new * ((H + 2 * G) * D * 2 + H * D * 2 + 2 * G * per) + back, "flops": 10.0 * new * (H + G) * D}
    if case["op"] == "evict":
        keep, cost = case["keep"], 0.0
        for a, c in zip(w, ctx):
            n = a + c
            kept = min(n, keep)
            moved = (n - kept) * kept / n                       # of the evicted, those in front of slot `keep`
            cost += n * 8 + kept * 8 + 2 * moved * 2 * per
        return {"bytes": G * cost, "flops": 0}
    win = case["window"] if case["window"] > 0 else 1 << 60
    keys = pairs = slots = 0
    for n, c in zip(w, ctx):
        first = max(0, c - win + 1)                             # the first key inside the first row's window
        keys += c + n - first + min(case["sinks"], first)
        slots += 2 * c + n
        full = max(0, min(n, win - c))                          # rows that see every key up to their own
        pairs += full * c + full * (full + 1) // 2
        if n > full:
            pairs += (n - full) * win + sum(min(case["sinks"], t - win + 1) for t in range(c + full, c + n))
    return {"bytes": keys * G * per + new * H * (D * 2 + 4) + slots * G * 4, "flops": 2.0 * pairs * H * D}


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


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _starts(n):
    return [sum(n[:i]) for i in range(len(n) + 1)]


def _logits(case, s, gen, w):
    """Rows as a verification leaves them: [rows, V], windows longer than what is committed, or trees and a path."""
    R, V = case["R"], case["V"]
    most = max(w)
    # a window has up to three rows more than it commits; a tree three slots for each node of its path
    wide = [3 * n if case["path"] else n + (n * 7 + i) % 4 for i, n in enumerate(w)]
    rows = sum(wide)
    dtype = torch.bfloat16 if case["dt"] == "bf16" else torch.float32
    z = torch.randn((rows, V), generator=gen, device=DEV, dtype=dtype)
    # peaked rows and flat ones, as a language model's are
    z *= torch.exp2(torch.rand((rows, 1), generator=gen, device=DEV) * 3 - 1).to(dtype)
    s["target"], s["cu"] = z, _i32(_starts(wide))
    s["tok"] = torch.full((R, most), -1, dtype=torch.int32, device=DEV)
    s["n"] = _i32(w)
    s["path"] = None
    row = s["cu"].long()[s["req"]] + s["pos"]
    if case["path"]:
        s["path"] = torch.full((R, most), -1, dtype=torch.int32, device=DEV)
        s["path"][s["req"], s["pos"]] = (3 * s["pos"] - (s["pos"] > 0).long()
                                         + (torch.rand(row.shape, generator=gen, device=DEV) < 0.5) * (s["pos"] > 0)).int()
        row = s["cu"].long()[s["req"]] + s["path"][s["req"], s["pos"]]
    s["row"] = row
    # a committed token is often the most probable one
    best = z[row].float().argmax(-1)
    other = torch.randint(0, V, row.shape, generator=gen, device=DEV)
    s["tok"][s["req"], s["pos"]] = torch.where(torch.rand(row.shape, generator=gen, device=DEV) < 0.7, best, other).int()
    n, k = (R, most), (R, most, case["top"])
    s["out"] = dict(logp=torch.zeros(n, device=DEV), entropy=torch.zeros(n, device=DEV),
                    rank=torch.zeros(n, dtype=torch.int32, device=DEV))
    if case["top"]:
        s["out"].update(top_tok=torch.zeros(k, dtype=torch.int32, device=DEV), top_logp=torch.zeros(k, device=DEV))


def prepare(case, seed):
    """Pools of pages in use, the page table, packed rows as a fused projection leaves them, lengths, positions and
    the weights so far; for the framework's own calls also the cache's handle, the outputs' buffers and a workspace."""
    w, ctx = lengths(case)
    R = case["R"]
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 1000003 + case["mix"])
    s = dict(case=case, max_w=max(w), rows=sum(w))
    s["req"] = torch.repeat_interleave(torch.arange(R, device=DEV), torch.tensor(w, device=DEV))
    s["pos"] = torch.arange(s["rows"], device=DEV) - torch.tensor(_starts(w), device=DEV)[s["req"]]
    if case["op"] == "logprobs":
        _logits(case, s, gen, w)
    else:
        _paged(case, s, gen, w, ctx)
    if own:
        _handles(case, s)
    return s


def _paged(case, s, gen, w, ctx):
    R, H, G, D, page = case["R"], case["H"], case["G"], case["D"], case["page"]
    op = case["op"]
    per_req = [(a + b + page - 1) // page for a, b in zip(w, ctx)]
    n_pages, most = sum(per_req) + 3, max(per_req)
    order = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    start = torch.tensor(_starts(per_req)[:-1], device=DEV)
    used = torch.tensor(per_req, device=DEV)
    at = torch.arange(most, device=DEV)
    table = torch.where(at[None] < used[:, None], order[(start[:, None] + at[None]).clamp(max=n_pages - 1)], 0)
    s.update(table=table.to(torch.int32).contiguous(), ctx=_i32(ctx), n=_i32(w),
             len=max(a + b for a, b in zip(w, ctx)))
    shape = (n_pages, G, page, D)
    for name in ("k", "v"):
        pool = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)
        # tokens differ in size, as activations do
        pool *= torch.exp2(torch.randint(-1, 2, shape[:3], generator=gen, device=DEV).to(torch.bfloat16))[..., None]
        if case["cache"] == "e4m3":
            code, e = _quantise(pool)
            s[name], s[name + "_exp"] = code, (e + 127).to(torch.uint8)
        else:
            s[name], s[name + "_exp"] = pool, None
    # a cache that has lost tokens before: more positions have been than it holds
    s["start"] = s["ctx"] + (s["ctx"] // 2 if op == "evict" else 0)
    if op == "evict":
        n = (R, G, s["len"])
        s["mass"] = torch.exp(2 * torch.randn(n, generator=gen, device=DEV) - 3)
        s["mass"] *= torch.rand(n, generator=gen, device=DEV) > 0.1        # some were never looked at
        seen = int(s["start"].max())
        u = torch.rand((R, G, max(seen, 1)), generator=gen, device=DEV)
        u = torch.where(torch.arange(u.shape[2], device=DEV)[None, None] < s["start"][:, None, None], u, 2.0)
        s["where"] = torch.full(n, -1, dtype=torch.int32, device=DEV)
        s["where"][:, :, :min(seen, s["len"])] = u.argsort(-1)[:, :, :s["len"]].int()
        s["out"] = dict(mass=torch.zeros(n, device=DEV), pos=torch.zeros(n, dtype=torch.int32, device=DEV),
                        length=torch.zeros((R,), dtype=torch.int32, device=DEV))
        return
    # queries, keys and values of the new tokens: slices of one projection's output
    wide, s["path"] = w, None
    if case["path"]:                                            # trees of three slots for each node of the path
        wide = [3 * n for n in w]
        s["path"] = torch.full((R, s["max_w"]), -1, dtype=torch.int32, device=DEV)
        s["path"][s["req"], s["pos"]] = (3 * s["pos"] - (s["pos"] > 0).long() + (
            torch.rand(s["pos"].shape, generator=gen, device=DEV) < 0.5) * (s["pos"] > 0)).int()
    s["cu"], s["packed"] = _i32(_starts(wide)), sum(wide)
    s["row"] = s["cu"].long()[s["req"]] + (s["path"][s["req"], s["pos"]] if case["path"] else s["pos"])
    qkv = torch.randn((s["packed"], H + 2 * G, D), generator=gen, device=DEV, dtype=torch.bfloat16)
    s["q"], s["new_k"], s["new_v"] = qkv[:, :H], qkv[:, H:H + G], qkv[:, H + G:]
    if op == "rotate":
        s["freq"] = 10000.0 ** (-torch.arange(case["rot"] // 2, device=DEV, dtype=torch.float64) * 2 / case["rot"])
        s["wq"], s["wk"] = ((1 + 0.2 * torch.randn((D,), generator=gen, device=DEV)) if case["norm"] else None
                            for _ in range(2))
        s["q_out"] = torch.zeros((s["rows"], H, D), dtype=torch.bfloat16, device=DEV)
        s["back_pos"] = s["ctx"].long()[s["req"]] + s["pos"]
        return
    s["scale"] = 1.0 / math.sqrt(D)
    s["mass"] = torch.rand((R, G, s["len"]), generator=gen, device=DEV) * 4
    s["out"] = dict(mass=torch.zeros((R, G, s["len"]), device=DEV))
    # what the attention left: the log-sum-exp of each row's scores
    s["lse"] = torch.ones((s["packed"], H), device=DEV)
    for h in range(G):
        x = _scores(s, h)
        top = x.amax(-1, keepdim=True)
        z = (torch.log((x - top).exp_().sum(-1, keepdim=True)) + top)[:, 0, :, :, 0]
        s["lse"][s["row"], h * (H // G):(h + 1) * (H // G)] = z[s["req"], s["pos"]]


def _handles(case, s):
    from speculative_decoding_markov_gb300 import binding as sdm
    s["status"] = sdm.new_status()
    if case["op"] == "logprobs":
        return
    s["handle"] = sdm.PagedCache(s["k"], s["v"], s["table"], s["k_exp"], s["v_exp"])
    if case["op"] == "rotate":
        s["out"] = dict(q=s["q_out"])
        if case["cache"] == "e4m3":
            shape = (s["rows"], case["G"], case["D"])
            s["back"] = {n: torch.empty(shape, dtype=torch.bfloat16, device=DEV) for n in "kv"}
    elif case["op"] == "weight":
        s["ws"] = sdm.attend_weight_workspace(s["handle"], s["max_w"], case["H"])
    else:
        s["ws"] = sdm.cache_evict_workspace(s["handle"], s["len"], case["keep"])


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _place(s, req, pos):
    """Page and slot of tokens `pos` of requests `req`."""
    page = s["case"]["page"]
    return s["table"].long()[req, pos // page], pos % page


def _tokens(s, name, req, pos, heads=slice(None)):
    """Rows [..., kv heads, head dim] of the cache in 32 bits."""
    page, slot = _place(s, req, pos)
    pool = s[name].view(torch.uint8) if s["case"]["cache"] == "e4m3" else s[name]
    x = pool[:, heads][page, :, slot]
    x = x.view(torch.float8_e4m3fn).float() if s["case"]["cache"] == "e4m3" else x.float()
    if s[name + "_exp"] is not None:
        x = x * _pow2(s[name + "_exp"][:, heads][page, :, slot].int() - 127)[..., None]
    return x


def _rotated(s, x, weight):
    """Rows [rows, heads, D] normalised and rotated in 32 bits; the angles in 64."""
    c = s["case"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    angle = (s["start"].long()[s["req"]] + s["pos"]).double()[:, None] * s["freq"][None]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    half = c["rot"] // 2
    turn = x[..., :c["rot"]]
    a, b = (turn[..., 0::2], turn[..., 1::2]) if c["inter"] else (turn[..., :half], turn[..., half:])
    a, b = a * cos - b * sin, a * sin + b * cos
    turn = torch.stack([a, b], -1).flatten(-2) if c["inter"] else torch.cat([a, b], -1)
    return torch.cat([turn, x[..., c["rot"]:]], -1).to(torch.bfloat16)


def _rotate(s):
    s["q_out"].copy_(_rotated(s, s["q"], s["wq"]))
    page, slot = _place(s, s["req"], s["back_pos"])
    for name, x in (("k", _rotated(s, s["new_k"], s["wk"])), ("v", s["new_v"])):
        if s["case"]["cache"] == "e4m3":
            code, e = _quantise(x)
            s[name].view(torch.uint8)[page, :, slot] = code.view(torch.uint8)
            s[name + "_exp"][page, :, slot] = (e + 127).to(torch.uint8)
        else:
            s[name][page, :, slot] = x
    if s["case"]["cache"] == "bf16":
        return [s["q_out"], s["k"], s["v"]]
    return [s["q_out"]] + [_tokens(s, n, s["req"], s["back_pos"]).to(torch.bfloat16) for n in "kv"]


def _logprobs(s):
    c, o = s["case"], s["out"]
    z = s["target"][s["row"]].float() + 0.0                     # -0 is +0
    tok = s["tok"][s["req"], s["pos"]].long()[:, None]
    x = z / c["temp"]
    top = x.amax(-1, keepdim=True)
    d = x - top
    e = torch.exp(d)
    total = e.sum(-1, keepdim=True)
    lse = torch.log(total) + top
    said = torch.gather(z, 1, tok)
    ids = torch.arange(c["V"], device=DEV)[None]
    o["logp"][s["req"], s["pos"]] = (torch.gather(x, 1, tok) - lse)[:, 0]
    o["entropy"][s["req"], s["pos"]] = (torch.log(total) - (e * d).sum(-1, keepdim=True) / total)[:, 0]
    o["rank"][s["req"], s["pos"]] = ((z > said) | ((z == said) & (ids < tok))).sum(-1).int()
    if c["top"]:
        bits = z.view(torch.int32).long()                       # in order: sign and magnitude turned, ties by the id
        key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits) * (1 << 32) + (c["V"] - 1 - ids)
        best = c["V"] - 1 - (torch.topk(key, c["top"], -1)[0] & 0xFFFFFFFF)
        o["top_tok"][s["req"], s["pos"]] = best.int()
        o["top_logp"][s["req"], s["pos"]] = torch.gather(x, 1, best) - lse
    return o


def _scores(s, h=None):
    """[R, kv heads, rows, heads a kv head, tokens] in 32 bits, -inf where a row does not see a token."""
    c = s["case"]
    R, G, D, W, L = c["R"], c["G"], c["D"], s["max_w"], s["len"]
    group, G = c["H"] // G, G if h is None else 1
    heads = slice(None) if h is None else slice(h, h + 1)
    key = torch.arange(L, device=DEV)
    last = (s["ctx"] + s["n"]).long()[:, None] - 1
    k = _tokens(s, "k", torch.arange(R, device=DEV)[:, None], torch.minimum(key[None], last), heads)
    q = torch.zeros((R, W, G * group, D), device=DEV)
    q[s["req"], s["pos"]] = s["q"][s["row"]][:, heads.start * group if h is not None else 0:
                                             (heads.stop * group) if h is not None else c["H"]].float()
    q = q.view(R, W, G, group, D).permute(0, 2, 1, 3, 4).reshape(R, G, W * group, D)
    x = (q @ k.permute(0, 2, 3, 1)).mul_(s["scale"]).view(R, G, W, group, L)
    row = s["ctx"].long()[:, None, None] + torch.arange(W, device=DEV)[None, :, None]
    seen = key[None, None] <= row
    if c["window"] > 0:
        seen = seen & ((row - key < c["window"]) | (key < c["sinks"]))
    return x.masked_fill_(~seen[:, None, :, None], -math.inf)


def _weight(s):
    c = s["case"]
    R, H, G, W, L = c["R"], c["H"], c["G"], s["max_w"], s["len"]
    lse = torch.full((R, W, H), math.inf, device=DEV)           # rows past the counted ones weigh nothing
    lse[s["req"], s["pos"]] = s["lse"][s["row"]]
    lse = lse.view(R, W, G, H // G).permute(0, 2, 1, 3)[..., None]
    got = _scores(s).sub_(lse).exp_().sum((2, 3))
    key = torch.arange(L, device=DEV)[None, None]
    ctx, n = s["ctx"].long()[:, None, None], s["n"].long()[:, None, None]
    new = torch.where(key < ctx, s["mass"], 0.0) + got
    s["out"]["mass"].copy_(torch.where(key < ctx + n, new, s["out"]["mass"]))
    return s["out"]


def _evict(s):
    c, o = s["case"], s["out"]
    slot = torch.arange(s["len"], device=DEV)[None, None]
    ctx, start, n = (s[x].long()[:, None, None] for x in ("ctx", "start", "n"))
    held, end = ctx + n, start + n
    pos = torch.where(slot < ctx, s["where"].long(), start + slot - ctx)
    key = torch.where((pos < c["first"]) | (pos >= end - c["recent"]), math.inf, s["mass"])
    key = torch.where(slot < held, key, -math.inf)
    best = torch.sort(key, dim=-1, descending=True, stable=True)[1][:, :, :c["keep"]]
    kept = torch.zeros_like(key, dtype=torch.bool).scatter_(2, best, True) & (slot < held)
    hole = torch.nonzero(~kept & (slot < c["keep"]) & (slot < held), as_tuple=True)
    late = torch.nonzero(kept & (slot >= c["keep"]), as_tuple=True)
    mass, pos = s["mass"].clone(), pos.int()
    mass[hole], pos[hole] = mass[late], pos[late]
    dst, src = _place(s, hole[0], hole[2]), _place(s, late[0], late[2])
    for name in ("k", "v", "k_exp", "v_exp"):
        if s[name] is not None:
            x = s[name].view(torch.uint8) if s[name].dtype == torch.float8_e4m3fn else s[name]
            x[dst[0], hole[1], dst[1]] = x[src[0], late[1], src[1]]
    length = held.clamp(max=c["keep"])
    o["mass"].copy_(torch.where(slot < length, mass, o["mass"]))
    o["pos"].copy_(torch.where(slot < length, pos, o["pos"]))
    o["length"].copy_(length[:, 0, 0])
    return [o["mass"], o["pos"], o["length"]] + _pools(s)


def _pools(s):
    """What the cache holds: bf16 rows, or 8-bit ones and their scales (a moved row keeps both)."""
    return [s[n] for n in ("k", "v", "k_exp", "v_exp") if s[n] is not None]


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        from speculative_decoding_markov_gb300 import binding as sdm
        if op == "rotate":
            sdm.qk_rotate(s["q"], s["new_k"], s["cu"], s["ctx"], s["freq"], v=s["new_v"], cache=s["handle"],
                          start=s["start"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS, interleaved=case["inter"],
                          out=s["out"], dev_status=s["status"])
            if case["cache"] == "bf16":
                return [s["q_out"], s["k"], s["v"]]
            sdm.cache_read(s["handle"], s["cu"], s["rows"], first=s["ctx"], out=s["back"], dev_status=s["status"])
            return [s["q_out"], s["back"]["k"], s["back"]["v"]]
        if op == "logprobs":
            return sdm.token_logprobs(s["target"], s["cu"], s["tok"], n=s["n"], path=s["path"],
                                      temperature=case["temp"], top=case["top"], out=s["out"], dev_status=s["status"])
        if op == "weight":
            return sdm.attend_weight(s["handle"], s["q"], s["lse"], s["cu"], s["ctx"], s["max_w"], mass=s["mass"],
                                     count=s["n"], path=s["path"], scale=s["scale"], window=case["window"],
                                     sinks=case["sinks"], out=s["out"], ws=s["ws"], dev_status=s["status"])
        o = sdm.cache_evict(s["handle"], s["mass"], s["where"], s["ctx"], s["start"], case["keep"], count=s["n"],
                            sinks=case["first"], recent=case["recent"], out=s["out"], ws=s["ws"],
                            dev_status=s["status"])
        return [o["mass"], o["pos"], o["length"]] + _pools(s)
    return {"rotate": _rotate, "logprobs": _logprobs, "weight": _weight, "evict": _evict}[op](s)


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


def _exact_rotate(case, s, w, ctx):
    D, rot = case["D"], case["rot"]

    def turned(x, weight):
        x = x.double()
        if weight is not None:
            x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / D + EPS) * weight.double()
        y = x.clone()
        at = torch.cat([s["start"][i].double() + torch.arange(w[i], device=DEV) for i in range(case["R"])])
        for j in range(rot // 2):
            a, b = (2 * j, 2 * j + 1) if case["inter"] else (j, j + rot // 2)
            cos, sin = torch.cos(at * s["freq"][j])[:, None], torch.sin(at * s["freq"][j])[:, None]
            y[..., a] = cos * x[..., a] - sin * x[..., b]
            y[..., b] = sin * x[..., a] + cos * x[..., b]
        return y

    q, k = turned(s["q"], s["wq"]), turned(s["new_k"], s["wk"])
    if case["cache"] == "e4m3":      # the cache takes bf16 rows
        return [q, _held64(k.to(torch.bfloat16), "e4m3"), _held64(s["new_v"], "e4m3")]
    pools, row = {n: s[n].double() for n in "kv"}, 0
    for i in range(case["R"]):
        p = torch.arange(ctx[i], ctx[i] + w[i], device=DEV)
        where = s["table"][i].long()[p // case["page"]], p % case["page"]
        for name, x in (("k", k), ("v", s["new_v"].double())):
            pools[name][where[0], :, where[1]] = x[row:row + w[i]]
        row += w[i]
    return [q, pools["k"], pools["v"]]


def _exact_logprobs(case, s, w):
    o = {n: s["out"][n].double() if s["out"][n].is_floating_point() else s["out"][n].clone() for n in s["out"]}
    cu = s["cu"].tolist()
    for i in range(case["R"]):
        for p0 in range(0, w[i], 64):
            p = torch.arange(p0, min(w[i], p0 + 64), device=DEV)
            z = s["target"][cu[i] + (s["path"][i, p].long() if case["path"] else p)].double()
            x, t = z / case["temp"], s["tok"][i, p].long()
            logp = x - torch.logsumexp(x, -1, keepdim=True)
            o["logp"][i, p] = logp.gather(1, t[:, None])[:, 0]
            o["entropy"][i, p] = -(logp.exp() * logp).sum(-1)
            order = torch.sort(z, dim=-1, descending=True, stable=True)[1]
            o["rank"][i, p] = (order == t[:, None]).int().argmax(-1).int()
            if case["top"]:
                best = order[:, :case["top"]]
                o["top_tok"][i, p] = best.int()
                o["top_logp"][i, p] = logp.gather(1, best)
    return o


def _exact_weight(case, s, w, ctx):
    G, D, page, group = case["G"], case["D"], case["page"], case["H"] // case["G"]
    out, cu = s["out"]["mass"].double(), s["cu"].tolist()
    for i in range(case["R"]):
        n = w[i] + ctx[i]
        ids = s["table"].long()[i, :(n + page - 1) // page]
        k = s["k"][ids].double()
        if s["k_exp"] is not None:
            k = k * _two64(s["k_exp"][ids].long() - 127)[..., None]
        k = k.permute(1, 0, 2, 3).reshape(G, -1, D)[:, :n]
        p = torch.arange(w[i], device=DEV)
        row = cu[i] + (s["path"][i, p].long() if case["path"] else p)
        q, lse = s["q"][row].double().view(w[i], G, group, D), s["lse"][row].double().view(w[i], G, group)
        key = torch.arange(n, device=DEV)
        out[i, :, :ctx[i]] = s["mass"][i, :, :ctx[i]].double()
        out[i, :, ctx[i]:n] = 0
        for part in range(0, w[i], 512):
            at = ctx[i] + p[part:part + 512, None]
            see = key[None] <= at
            if case["window"]:
                see &= (key[None] > at - case["window"]) | (key[None] < case["sinks"])
            for h in range(G):
                x = torch.einsum("wgd,nd->wgn", q[part:part + 512, h], k[h]) * s["scale"]
                x = torch.exp(x - lse[part:part + 512, h, :, None])
                out[i, h, :n] += torch.where(see[:, None], x, 0.0).sum((0, 1))
    return dict(mass=out)


def _exact_evict(case, s, w, ctx):
    mass, pos = s["out"]["mass"].double(), s["out"]["pos"].clone()
    length, keep = s["out"]["length"].clone(), case["keep"]
    pools = [x.double() if x.is_floating_point() else x.clone() for x in _pools(s)]
    for i in range(case["R"]):
        n, start = w[i] + ctx[i], int(s["start"][i])
        slot = torch.arange(n, device=DEV)
        length[i] = min(n, keep)
        for h in range(case["G"]):
            at = torch.where(slot < ctx[i], s["where"][i, h, :n], start + slot - ctx[i]).long()
            m = s["mass"][i, h, :n].double()
            always = (at < case["first"]) | (at >= start + w[i] - case["recent"])
            order = torch.sort(torch.where(always, math.inf, m), descending=True, stable=True)[1]
            kept = order[:keep].sort()[0]
            free = torch.ones(n, dtype=torch.bool, device=DEV)
            free[kept] = False
            to, frm = torch.nonzero(free[:keep])[:, 0], kept[kept >= keep]
            m[to], at[to] = m[frm], at[frm]
            mass[i, h, :min(n, keep)], pos[i, h, :min(n, keep)] = m[:keep], at[:keep].int()
            table = s["table"].long()[i]
            for x in pools:
                x[table[to // case["page"]], h, to % case["page"]] = x[table[frm // case["page"]], h, frm % case["page"]]
    return [mass, pos, length] + pools


def exact(case, seed):
    s = prepare(case, seed)
    w, ctx = lengths(case)
    if case["op"] == "logprobs":
        return _exact_logprobs(case, s, w)
    return {"rotate": _exact_rotate, "weight": _exact_weight, "evict": _exact_evict}[case["op"]](case, s, w, ctx)

"""Decoding over caches of bounded size, as a serving loop runs it: queries and
keys rotated into the cache, attention, log probabilities of what is committed,
the tokens' weight, and the cut of every cache; against a plain simulation in 64
bits that keeps its own list of tokens per request and head."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from speculative_decoding_markov_gb300 import binding as sdm
from tests import paged_reference as ref
from tests.test_gpu_logprobs import check_rows
from tests.test_gpu_rotate import close, formula, freqs
from tests.test_gpu_weight_evict import plain_evict, weights

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Loop:
    """The buffers of a serving loop: lengths and positions have two sets, for a
    cut reads one while it writes the other."""

    def __init__(self, R, H, G, D, page, keep, most, e4m3, seed):
        self.R, self.H, self.G, self.D, self.keep, self.e4m3 = R, H, G, D, keep, e4m3
        self.gen = torch.Generator().manual_seed(seed)
        self.tokens = keep + most
        cols = -(-self.tokens // page)
        table = torch.randperm(R * cols, generator=self.gen).to(torch.int32).view(R, cols).cuda()
        self.cache = sdm.PagedCache.empty(R * cols, G, page, D, table, torch.float8_e4m3fn if e4m3 else torch.bfloat16)
        self.mass = torch.zeros((R, G, self.tokens), device="cuda")
        self.pos = torch.zeros((R, G, self.tokens), dtype=torch.int32, device="cuda")
        self.ctx, self.start = [i32([0] * R), i32([0] * R)], [i32([0] * R), i32([0] * R)]
        self.freq, self.kw = freqs(D).cuda(), (1 + torch.rand((D,), generator=self.gen)).cuda()
        self.status = sdm.new_status()
        # the simulation: per request and head the keys, values and positions of its slots
        self.held = [[dict(k=np.zeros((0, D)), v=np.zeros((0, D)), pos=np.zeros(0, np.int64)) for _ in range(G)]
                     for _ in range(R)]
        self.seen = [0] * R

    def rows(self, n, heads):
        return torch.randn((n, heads, self.D), generator=self.gen).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("R,H,G,D,page,keep,most,cycles", [(3, 4, 2, 64, 16, 24, 5, 9), (5, 6, 1, 128, 64, 70, 9, 12),
                                                           (2, 8, 2, 128, 32, 300, 200, 4)])
def test_cycles(gpu_lib, e4m3, R, H, G, D, page, keep, most, cycles):
    s = Loop(R, H, G, D, page, keep, most, e4m3, seed=R)
    rng = np.random.default_rng(R)
    V, sinks, recent, scale = 1000, 2, 6, D ** -0.5
    for cycle in range(cycles):
        w = rng.integers(1, most + 1, R).tolist()
        n = [int(rng.integers(1, x + 1)) for x in w]               # what verification commits of each window
        cu = i32(np.concatenate([[0], np.cumsum(w)]).tolist())
        ctx, start = s.ctx[cycle & 1], s.start[cycle & 1]
        q, k, v = s.rows(sum(w), H), s.rows(sum(w), G), s.rows(sum(w), G)
        rot = sdm.qk_rotate(q, k, cu, ctx, s.freq, v=v, cache=s.cache, start=start, k_weight=s.kw, dev_status=s.status)
        att = sdm.attend(s.cache, rot["q"], cu, ctx, most, lse=True, dev_status=s.status)
        target = torch.randn((sum(w), V), generator=s.gen).to(torch.bfloat16).cuda()
        tok = torch.randint(0, V, (R, most), generator=s.gen, dtype=torch.int32).cuda()
        lp = sdm.token_logprobs(target, cu, tok, n=i32(n), top=3, dev_status=s.status)
        before = s.mass.clone()
        sdm.attend_weight(s.cache, rot["q"], att["lse"], cu, ctx, most, mass=s.mass, count=i32(n), out=dict(mass=s.mass),
                          dev_status=s.status)
        grown, pos0 = s.mass.clone(), s.pos.clone()
        out = dict(mass=s.mass, pos=s.pos, length=s.ctx[1 - (cycle & 1)], next=s.start[1 - (cycle & 1)])
        sdm.cache_evict(s.cache, s.mass, s.pos, ctx, start, keep, count=i32(n), sinks=sinks, recent=recent, out=out,
                        dev_status=s.status)
        assert s.status.item() == 0

        check_rows(lp, target, [(i, p, int(cu[i]) + p) for i in range(R) for p in range(n[i])],
                   [int(tok[i, p]) for i in range(R) for p in range(n[i])], 1.0, 3)
        at = torch.cat([torch.arange(a, a + b) for a, b in zip(s.seen, w)])
        close(rot["q"], *formula(q, at, freqs(D), None, 0, False))
        keys, _ = formula(k, at, freqs(D), s.kw, 1e-6, False)
        lengths = out["length"].tolist()
        back = sdm.cache_read(s.cache, i32(np.concatenate([[0], np.cumsum(lengths)]).tolist()), sum(lengths))
        row = off = 0
        for i in range(R):
            ctx_i = s.held[i][0]["pos"].size
            see = ref.visible(w[i], ctx_i)
            for g in range(G):
                h = s.held[i][g]
                heads = slice(g * (H // G), (g + 1) * (H // G))
                # what the cache holds of the new rows is compared as it is read back, below
                new_k = keys[row:row + w[i], g].numpy()
                held_k = ref.held(torch.tensor(new_k).to(torch.bfloat16), e4m3).numpy()
                held_v = ref.held(v[row:row + w[i], g].cpu(), e4m3).numpy()
                kk, vv = np.concatenate([h["k"], held_k]), np.concatenate([h["v"], held_v])
                qq = rot["q"][row:row + w[i], heads]
                o, z, size = ref.attend(qq, torch.tensor(kk)[:, None], torch.tensor(vv)[:, None], see, scale)
                # a key that was rounded the other way (its fp32 value beside a rounding's
                # border) differs by a step: 2^-7 of itself, 2^-3 in 8 bits
                step = 2.0 ** -3 if e4m3 else 2.0 ** -7
                loose = step * scale * (qq.double().abs().cpu().numpy()[:, :, None] * np.abs(kk)[None, None]).max(-1).max()
                got_lse = att["lse"][row:row + w[i], heads].double().cpu().numpy()
                assert (np.abs(got_lse - z) <= 1e-5 + loose).all()
                m = before[i, g, :ctx_i + n[i]].double().cpu().numpy()
                m[ctx_i:] = 0
                want, tol = weights(qq[:n[i]], torch.tensor(got_lse[:n[i]]), torch.tensor(kk[:ctx_i + n[i], None]),
                                    see[:n[i], :ctx_i + n[i]], scale, H // G)
                err = np.abs(grown[i, g, :ctx_i + n[i]].double().cpu().numpy() - m - want[0])
                assert (err <= tol[0] + 2.0 ** -23 * (m + want[0]) + 2 * loose * want[0]).all(), (cycle, i, g, err.max())
                # the cut, by the weights that the library found
                mm = grown[i, g].cpu().numpy()
                src, wm, wp = plain_evict(mm, pos0[i, g].cpu().numpy(), ctx_i, n[i], s.seen[i], keep, sinks, recent)
                assert np.array_equal(s.mass[i, g, :lengths[i]].cpu().numpy(), wm)
                assert np.array_equal(s.pos[i, g, :lengths[i]].cpu().numpy(), wp)
                for name, x in (("k", kk), ("v", vv)):
                    got = back[name][off:off + lengths[i], g].double().cpu().numpy()
                    assert (np.abs(got - x[src]) <= step * np.abs(x[src]) + 1e-30).all()
                    assert (got == x[src]).mean() > 0.99
                    h[name] = got                                   # what is held, to the bit, from here on
                h["pos"] = wp
            row += w[i]
            off += lengths[i]
            s.seen[i] += n[i]
        assert out["next"].tolist() == s.seen


def test_a_captured_cycle(gpu_lib):
    """Two cycles (one for each set of lengths) captured and replayed: the same
    cache, weights and positions as the calls by themselves."""
    R, H, G, D, keep, w = 4, 8, 2, 128, 64, 5

    def make():
        s = Loop(R, H, G, D, 16, keep, w, False, seed=11)
        s.q, s.k, s.v = (torch.randn((R * w, h, D), generator=s.gen).to(torch.bfloat16).cuda() for h in (H, G, G))
        s.cu, s.n = i32([w * i for i in range(R + 1)]), i32([5, 1, 3, 2])
        s.qo = torch.empty_like(s.q)
        s.att = dict(out=torch.empty_like(s.q), lse=torch.empty((R * w, H), device="cuda"))
        s.ws = [sdm.attend_workspace(s.cache, R * w, w, H), sdm.attend_weight_workspace(s.cache, w, H),
                sdm.cache_evict_workspace(s.cache, s.tokens, keep)]
        return s

    def cycle(s, a):
        ctx, start = s.ctx[a], s.start[a]
        sdm.qk_rotate(s.q, s.k, s.cu, ctx, s.freq, v=s.v, cache=s.cache, start=start, out=dict(q=s.qo), dev_status=s.status)
        sdm.attend(s.cache, s.qo, s.cu, ctx, w, lse=True, out=s.att, ws=s.ws[0], dev_status=s.status)
        sdm.attend_weight(s.cache, s.qo, s.att["lse"], s.cu, ctx, w, mass=s.mass, count=s.n, out=dict(mass=s.mass),
                          ws=s.ws[1], dev_status=s.status)
        sdm.cache_evict(s.cache, s.mass, s.pos, ctx, start, keep, count=s.n, sinks=1, recent=8, ws=s.ws[2],
                        out=dict(mass=s.mass, pos=s.pos, length=s.ctx[1 - a], next=s.start[1 - a]), dev_status=s.status)

    one, two = make(), make()
    for k in range(24):
        cycle(one, k & 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cycle(two, 0)
        cycle(two, 1)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cycle(two, 0)
        cycle(two, 1)
    for _ in range(11):
        graph.replay()
    torch.cuda.synchronize()
    assert one.status.item() == 0 and two.status.item() == 0
    assert one.ctx[0].tolist() == two.ctx[0].tolist() == [min(keep, 24 * x) for x in (5, 1, 3, 2)]
    assert one.start[0].tolist() == two.start[0].tolist()
    for i, n in enumerate(one.ctx[0].tolist()):
        assert torch.equal(one.mass[i, :, :n], two.mass[i, :, :n]) and torch.equal(one.pos[i, :, :n], two.pos[i, :, :n])
    cu = i32(np.concatenate([[0], np.cumsum(one.ctx[0].tolist())]).tolist())
    a, b = (sdm.cache_read(s.cache, cu, int(cu[-1])) for s in (one, two))
    assert torch.equal(a["k"], b["k"]) and torch.equal(a["v"], b["v"])


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_tree_verified_and_committed(gpu_lib, e4m3):
    """A drafted tree's cycle: depths as positions, attention under the mask, the
    committed path's log probabilities and weight, the cut."""
    R, H, G, D, page, S, B, V = 3, 4, 2, 64, 16, 9, 8, 512
    rng = np.random.default_rng(2)
    tree = ref.random_trees(R, S, 6, rng, vocab=V)
    s = ref.Setup([S] * R, [20, 0, 33], G, D, page, e4m3, seed=2, fill=0.0)
    s.write_all()                                                  # contexts, and the tree's rows (rotated anew below)
    bits = (tree["mask"][:, :, :, None].astype(np.int64) >> np.arange(32)) & 1
    depth = np.maximum(bits.reshape(R, S, -1).sum(-1) - 1, 0).astype(np.int32)
    q = torch.randn((R * S, H, D), generator=s.gen).to(torch.bfloat16).cuda()
    freq = freqs(D).cuda()
    start = s.ctx + 100
    qr = sdm.qk_rotate(q, s.packed("k"), s.cu, s.ctx, freq, v=s.packed("v"), cache=s.cache, start=start,
                       row_pos=i32(depth.reshape(-1).tolist()), dev_status=s.status)["q"]
    mask = i32(tree["mask"].tolist())
    att = sdm.attend(s.cache, qr, s.cu, s.ctx, S, tree_mask=mask, lse=True, dev_status=s.status)
    target = torch.randn((R, S, V), generator=s.gen)
    for i in range(R):                                             # the target walks to the deepest node
        at = int(depth[i].argmax())
        while at > 0:
            up = int(tree["parent"][i, at])
            target[i, up, int(tree["tok"][i, at])] = 50.0
            at = up
    target = target.to(torch.bfloat16).cuda()
    tok, parent, nodes = (i32(tree[x].tolist()) for x in ("tok", "parent", "n_nodes"))
    ver = sdm.verify_tree(target, tok, parent, nodes, B)
    com = sdm.cache_commit(s.cache, tok, parent, nodes, ver["out_tok"], ver["accept"], s.ctx, dev_status=s.status)
    lp = sdm.token_logprobs(target, i32([S * i for i in range(R + 1)]), ver["out_tok"], n=ver["n_out"], path=com["path"],
                            top=2, dev_status=s.status)
    T = 33 + S
    mass = dict(mass=torch.zeros((R, G, T), device="cuda"))
    sdm.attend_weight(s.cache, qr, att["lse"], s.cu, s.ctx, B + 1, count=ver["n_out"], path=com["path"], out=mass,
                      dev_status=s.status)
    assert s.status.item() == 0
    n = ver["n_out"].tolist()
    assert n == [int(depth[i].max()) + 1 for i in range(R)]
    rows, toks = [], []
    for i in range(R):
        for p in range(n[i]):
            rows.append((i, p, S * i + int(com["path"][i, p])))
            toks.append(int(ver["out_tok"][i, p]))
    check_rows(lp, target, rows, toks, 1.0, 2)
    assert com["length"].tolist() == [a + b for a, b in zip([20, 0, 33], n)]
    cu = i32(np.concatenate([[0], np.cumsum(com["length"].tolist())]).tolist())
    back = sdm.cache_read(s.cache, cu, int(cu[-1]))
    for i in range(R):
        path = [int(x) for x in com["path"][i, :n[i]]]
        k = back["k"][int(cu[i]):int(cu[i + 1])]
        r = [S * i + x for x in path]
        want, tol = weights(qr[r], att["lse"][r], k, ref.visible(n[i], [20, 0, 33][i]), D ** -0.5, H // G)
        got = mass["mass"][i, :, :k.shape[0]].double().cpu().numpy()
        assert (np.abs(got - want) <= tol).all()
        # every counted row's weights are a softmax: they add up to one
        assert np.allclose(got.sum(-1), n[i] * (H // G), rtol=1e-4)
    keep = 12
    pos = torch.arange(T, dtype=torch.int32, device="cuda").repeat(R, G, 1)
    ev = dict(mass=mass["mass"], pos=pos, length=i32([0] * R), next=i32([0] * R))
    sdm.cache_evict(s.cache, mass["mass"], pos, s.ctx, start, keep, count=ver["n_out"], sinks=1, recent=4, out=ev,
                    dev_status=s.status)
    assert s.status.item() == 0 and ev["length"].tolist() == [min(keep, x) for x in com["length"].tolist()]

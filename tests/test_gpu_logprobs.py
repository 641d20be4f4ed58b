"""Log probabilities of committed tokens, entropies, ranks and the most
probable tokens against 64-bit forms."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from speculative_decoding_markov_gb300 import binding as sdm

pytestmark = pytest.mark.gpu
INF = float("inf")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check_rows(out, target, rows, toks, T, top):
    """rows: (i, p, target row).  Roundings: a thread adds up to `n` terms whose
    2^x is off by 2^-22, a shift of the exponent by 2^-24 of itself; the
    entropy's two parts are at most itself and the reference's lag (10)."""
    V = target.shape[-1]
    n = 8 * -(-V // 4096) + 64
    z = target.reshape(-1, V).double().cpu().numpy()
    for (i, p, r), y in zip(rows, toks):
        x = z[r] / T
        m = x.max()
        lp = (x - m) - np.log(np.exp(x - m).sum())                 # in this order: m may be 10^38
        unit = 2.0 ** -24 * (n + 16)
        span = 2.0 ** -22 * (np.abs(x[np.isfinite(x)] - m).max() if np.isfinite(m) else 0)
        got = out["logp"][i, p].item()
        order = np.argsort(-z[r], kind="stable")
        if 0 <= y < V:
            if np.isfinite(lp[y]):
                assert abs(got - lp[y]) <= unit + 2.0 ** -22 * (m - x[y]) + 2.0 ** -22 * abs(lp[y]), (i, p, got, lp[y])
            else:
                assert got == -INF
            if "rank" in out:
                assert out["rank"][i, p].item() == int(np.nonzero(order == y)[0][0])
        if "entropy" in out:
            pr = np.exp(lp)
            H = -(pr[pr > 0] * lp[pr > 0]).sum()
            assert abs(out["entropy"][i, p].item() - H) <= (unit + 2.0 ** -21) * (H + 10), (i, p)
        if top:
            ids = out["top_tok"][i, p].cpu().numpy()
            assert (ids == order[:top]).all(), (i, p, ids, order[:top])
            tl = out["top_logp"][i, p].double().cpu().numpy()
            want = lp[order[:top]]
            fin = np.isfinite(want)
            assert (np.isneginf(tl) == ~fin).all()
            assert (np.abs(tl[fin] - want[fin]) <= unit + span + 2.0 ** -22 * np.abs(want[fin])).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [8, 24, 200, 2048, 4096, 4104, 33000, 151936])
@pytest.mark.parametrize("top,T", [(0, 1.0), (1, 0.7), (5, 1.0), (20, 1.3), (32, 1.0)])
def test_ragged_windows(gpu_lib, dt, V, top, T):
    top = min(top, V)
    w, n = [5, 1, 0, 7], [3, 1, 0, 7]
    R, W = 4, 7
    gen = torch.Generator().manual_seed(V + top)
    cu = np.concatenate([[0], np.cumsum(w)])
    target = (3 * torch.randn((int(cu[-1]) + 2, V), generator=gen)).to(dt).cuda()
    tok = torch.randint(0, V, (R, W), generator=gen, dtype=torch.int32)
    for i in range(R):                                             # every other one is the most probable
        for p in range(0, n[i], 2):
            tok[i, p] = int(target[cu[i] + p].float().argmax())
    out = sdm.token_logprobs(target, i32(cu.tolist()), tok.cuda(), n=i32(n), temperature=T, top=top)
    assert out["dev_status"].item() == 0
    rows = [(i, p, int(cu[i]) + p) for i in range(R) for p in range(n[i])]
    check_rows(out, target, rows, [int(tok[i, p]) for i, p, _ in rows], T, top)
    for i in range(R):                                             # the others keep what they held
        assert (out["rank"][i, n[i]:] == -1).all() and (out["logp"][i, n[i]:] == 0).all()
    if n == [3, 1, 0, 7]:
        whole = sdm.token_logprobs(target, i32(cu.tolist()), tok.cuda(), temperature=T, top=top)
        rows = [(i, p, int(cu[i]) + p) for i in range(R) for p in range(w[i])]
        check_rows(whole, target, rows, [int(tok[i, p]) for i, p, _ in rows], T, top)


@pytest.mark.parametrize("R", [1, 20, 300])
def test_a_trees_path(gpu_lib, R):
    S, V, W = 9, 4096, 5
    gen = torch.Generator().manual_seed(R)
    target = torch.randn((R, S, V), generator=gen).to(torch.bfloat16).cuda()
    path = torch.full((R, W), -1, dtype=torch.int32)
    n = torch.randint(1, W + 1, (R,), generator=gen)
    tok = torch.full((R, W), -1, dtype=torch.int32)
    for i in range(R):
        path[i, :n[i]] = torch.cat([torch.zeros(1), torch.randperm(S - 1, generator=gen)[:n[i] - 1].sort()[0] + 1]).int()
        tok[i, :n[i]] = torch.randint(0, V, (int(n[i]),), generator=gen).int()
    out = sdm.token_logprobs(target, i32([S * i for i in range(R + 1)]), tok.cuda(), n=n.int().cuda(),
                             path=path.cuda(), top=3)
    rows = [(i, p, S * i + int(path[i, p])) for i in range(R) for p in range(int(n[i]))]
    check_rows(out, target, rows, [int(tok[i, p]) for i, p, _ in rows], 1.0, 3)
    assert out["dev_status"].item() == 0


def special(V, dt):
    """Rows that masks and overflows leave."""
    low = torch.finfo(dt).min
    a = torch.linspace(-3, 3, V)
    rows = [torch.where(torch.arange(V) % 97 == 5, a, -INF),       # a few allowed tokens
            torch.where(torch.arange(V) == V - 3, 1.0, -INF),      # one
            torch.full((V,), 0.25), torch.full((V,), low),         # every token alike
            torch.where(torch.arange(V) < 3, 2.0, low), torch.where(torch.arange(V) % 2 == 0, -1e38, a),
            torch.arange(V).float() / V * 80 - 40, -torch.arange(V).float() / V * 80, a * 1e30, a * 1e37,
            torch.where(torch.arange(V) == 7, 3e38, a), torch.round(a), torch.round(a * 40) / 8]
    return torch.stack(rows).to(dt)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [64, 5000, 40008])
def test_masked_flat_and_huge_rows(gpu_lib, dt, V):
    target = special(V, dt).cuda()
    n = target.shape[0]
    for top in (4, min(32, V)):
        tok = i32([[(11 * r) % V for r in range(n)]])
        out = sdm.token_logprobs(target, i32([0, n]), tok, top=top)
        assert out["dev_status"].item() == 0
        check_rows(out, target, [(0, r, r) for r in range(n)], tok[0].tolist(), 1.0, top)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_more_equal_values_than_a_list_holds_above_the_bound(gpu_lib, dt):
    """The largest elements all in the places of one thread."""
    V = 65536
    z = torch.zeros(V)
    z[torch.arange(0, V, 4096)] = 5.0                              # one thread's in a row by itself
    z[torch.arange(3, V, 7)] += 1.0
    target = torch.stack([z, torch.arange(V) % 256 * 0.125]).to(dt).cuda().repeat(200, 1)
    tok = i32([[5] * 400])
    out = sdm.token_logprobs(target, i32([0, 400]), tok, top=32)
    check_rows(out, target, [(0, r, r) for r in (0, 1, 398, 399)], [5] * 4, 1.0, 32)


def test_infinite_and_nan_rows(gpu_lib):
    V = 1000
    t = torch.zeros((4, V))
    t[0] = -INF
    t[1, 3] = INF
    t[2, 700] = float("nan")
    for dt in (torch.bfloat16, torch.float32):
        out = sdm.token_logprobs(t.to(dt).cuda(), i32([0, 4]), i32([[0, 5, 5, 5]]), top=6)
        logp, H = out["logp"][0].tolist(), out["entropy"][0].tolist()
        assert np.isnan(logp[0]) and logp[1] == -INF and np.isnan(logp[2])
        assert all(np.isnan(h) for h in H[:3]) and abs(logp[3] + np.log(V)) < 1e-4
        ids = out["top_tok"][0].cpu()
        assert ids[0].tolist() == list(range(6)) and ids[1].tolist() == [3, 0, 1, 2, 4, 5]
        assert all(len(set(r.tolist())) == 6 and (r >= 0).all() and (r < V).all() for r in ids)


def test_the_same_bits_again_and_beside_other_rows(gpu_lib):
    gen = torch.Generator().manual_seed(1)
    target = torch.randn((600, 20000), generator=gen).to(torch.bfloat16).cuda()
    tok = torch.randint(0, 20000, (1, 600), generator=gen, dtype=torch.int32).cuda()
    a, b = (sdm.token_logprobs(target, i32([0, 600]), tok, top=9) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_what_the_device_finds_wrong(gpu_lib):
    V = 4096
    gen = torch.Generator().manual_seed(2)
    target = torch.randn((6, V), generator=gen).cuda()

    def call(cu, tok, n, path=None):
        out = sdm.token_logprobs(target, i32(cu), i32(tok), n=i32(n), path=None if path is None else i32(path), top=2)
        return out["dev_status"].item(), out

    st, out = call([0, 3, 6], [[1, V, -1], [2, 3, 4]], [3, 3])
    assert st == sdm.DEV_BAD_TOKEN and out["logp"][0, 1].item() == -INF and out["rank"][0, 2].item() == V
    check_rows(out, target, [(0, 0, 0), (1, 2, 5)], [1, 4], 1.0, 2)
    assert call([0, 3, 6], [[1, 1, 1], [2, 3, 4]], [4, -1])[0] == sdm.DEV_BAD_WINDOW
    assert call([0, 2, 6], [[1, 1, 1], [2, 3, 4]], [3, 3])[0] == sdm.DEV_BAD_WINDOW      # past its window
    assert call([0, 3, 9], [[1, 1, 1, 1], [2, 3, 4, 5]], [3, 4])[0] == sdm.DEV_CAPACITY
    assert call([-2, 3, 6], [[1, 1, 1], [2, 3, 4]], [3, 3])[0] == sdm.DEV_BAD_WINDOW
    assert call([0, 3, 6], [[1, 1, 1], [2, 3, 4]], [3, 3], [[0, 1, 3], [0, 1, 2]])[0] == sdm.DEV_BAD_WINDOW
    assert call([0, 3, 6], [[1, 1, 1], [2, 3, 4]], [3, 3], [[0, 2, 1], [0, 1, 2]])[0] == 0


def test_a_captured_call_and_another_stream(gpu_lib):
    gen = torch.Generator().manual_seed(3)
    target = torch.randn((8, 30000), generator=gen).to(torch.bfloat16).cuda()
    tok = torch.randint(0, 30000, (2, 4), generator=gen, dtype=torch.int32).cuda()
    cu, st = i32([0, 4, 8]), sdm.new_status()
    out = sdm.token_logprobs(target, cu, tok, top=5, dev_status=st)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        sdm.token_logprobs(target, cu, tok, top=5, out=out, dev_status=st)
    target.neg_()
    graph.replay()
    check_rows(out, target, [(i, p, 4 * i + p) for i in range(2) for p in range(4)], tok.flatten().tolist(), 1.0, 5)
    assert st.item() == 0


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [256, 264, 832, 1200, 1792, 2040])
@pytest.mark.parametrize("top,T", [(13, 1.0), (20, 0.7), (32, 1.3)])
def test_long_lists_of_short_rows(gpu_lib, dt, V, top, T):
    test_ragged_windows(gpu_lib, dt, V, top, T)

"""Attention weight and eviction at their limits: infinite keys beside columns
that no row fills, the longest caches."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from speculative_decoding_markov_gb300 import binding as sdm
from tests import paged_reference as ref
from tests.test_gpu_weight_evict import i32, weights

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group,w", [(7, 18), (3, 42), (5, 25), (6, 21), (65, 1), (100, 1), (7, 40), (3, 130), (12, 60),
                                     (33, 9), (100, 5), (8, 16), (8, 50)])
def test_keys_of_minus_infinity_against_every_row(gpu_lib, D, group, w):
    """Every score of such a key is -inf and its weight nothing, also where the
    rows' tiles have columns without a row: 0 times infinity is in no sum."""
    s = ref.Setup([w], [400], 1, D, 16, False, seed=group)
    for j in (0, 130, 257, 399, 400):
        s.kv[0]["k"][j, 0, j % D] = -INF
    s.write_all()
    q = torch.rand((w, group, D), generator=s.gen).add(0.25).to(torch.bfloat16).cuda()
    lse = (3 + torch.rand((w, group), generator=s.gen)).cuda()
    T = 400 + w
    mass = torch.rand((1, 1, T), generator=s.gen).cuda()
    out = dict(mass=torch.zeros_like(mass))
    sdm.attend_weight(s.cache, q, lse, s.cu, s.ctx, w, mass=mass, out=out, dev_status=s.status)
    assert s.status.item() == 0
    want, tol = weights(q, lse, s.held(0, "k"), ref.visible(w, 400), D ** -0.5, group)
    old = mass[0].double().cpu().numpy()
    old[:, 400:] = 0
    got = out["mass"][0].double().cpu().numpy()
    assert (np.abs(got - want - old) <= tol + 2.0 ** -24 * (want + old)).all()
    assert (got[0, [0, 130, 257, 399, 400]] == old[0, [0, 130, 257, 399, 400]]).all()
    again = dict(mass=torch.zeros_like(mass))                      # the rows gathered along a path
    sdm.attend_weight(s.cache, q, lse, s.cu, s.ctx, w, mass=mass, path=i32([list(range(w))]), out=again, dev_status=s.status)
    assert torch.equal(again["mass"], out["mass"]) and s.status.item() == 0


def test_eviction_from_the_longest_cache(gpu_lib):
    """2^31 - 256 tokens, the most that a call takes: 20 of 29 unseen ones go."""
    n, page = 2 ** 31 - 256, 128
    keep = n - 20
    table = torch.zeros((1, 2 ** 31 // page), dtype=torch.int32, device="cuda")    # one page of zeros for all
    cache = sdm.PagedCache.empty(1, 1, page, 64, table)
    mass = torch.ones((1, 1, n), device="cuda")
    unseen = list(range(5, n, n // 23))[:24] + [n - 1, n - 3, n - 19, n - 20, n - 21, n - 22]
    mass[0, 0, unseen] = 0.0
    pos = torch.zeros((1, 1, n), dtype=torch.int32, device="cuda")
    out = dict(mass=mass, pos=pos, length=i32([0]), next=i32([0]))
    status = sdm.new_status()
    sdm.cache_evict(cache, mass, pos, i32([0]), None, keep, count=i32([n]), out=out, dev_status=status)
    assert status.item() == 0 and out["length"].item() == keep and out["next"].item() == n
    gone = sorted(unseen)[-(n - keep):]                            # of equals the lowest stay
    holes, late = [s for s in gone if s < keep], [s for s in range(keep, n) if s not in gone]
    assert pos[0, 0, holes].tolist() == late and (mass[0, 0, holes] == 1).all()
    assert sum(int((mass[0, 0, a:min(a + 2 ** 28, keep)] == 0).sum()) for a in range(0, keep, 2 ** 28)) == 9
    moved = 0
    for a in range(0, keep, 2 ** 28):
        b = min(a + 2 ** 28, keep)
        moved += int((pos[0, 0, a:b] != torch.arange(a, b, dtype=torch.int32, device="cuda")).sum())
    assert moved == len(holes)


@pytest.mark.parametrize("w", [1, 200])
def test_weights_of_the_longest_cache(gpu_lib, w):
    """2^31 - 256 tokens, of which a window sees the last: the others' weights
    pass through, and nothing behind them is written."""
    n, page, window = 2 ** 31 - 256, 128, 10
    table = torch.zeros((1, 2 ** 31 // page), dtype=torch.int32, device="cuda")    # one page of zeros for all
    cache = sdm.PagedCache.empty(1, 1, page, 64, table)
    mass = torch.arange(1, 2 ** 16 + 1, dtype=torch.float32, device="cuda").repeat(2 ** 15)[:2 ** 31 - 1].view(1, 1, -1)
    out = dict(mass=torch.full_like(mass, -7.0))
    q, lse = torch.ones((w, 1, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((w, 1), device="cuda")
    status = sdm.new_status()
    sdm.attend_weight(cache, q, lse, i32([0, w]), i32([n - w]), w, mass=mass, window=window, out=out, dev_status=status)
    assert status.item() == 0
    got, first = out["mass"][0, 0], n - w - window + 1             # a score of 0 beside an lse of 0: a weight of 1 a row
    assert all(torch.equal(got[a:min(a + 2 ** 28, first)], mass[0, 0, a:min(a + 2 ** 28, first)])
               for a in range(0, first, 2 ** 28))
    t = torch.arange(first, n, device="cuda")
    want = sum(((t <= n - w + p) & (t > n - w + p - window)).float() for p in range(w))
    assert torch.equal(got[first:n], want + torch.where(t < n - w, mass[0, 0, first:n], 0.0))
    assert (got[n:] == -7).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("w,window", [(3, 0), (3, 40), (200, 0), (200, 40)])
def test_rows_of_the_lowest_lse(gpu_lib, e4m3, w, window):
    """A row whose lse is the type's lowest value gives what it sees infinite
    weights, and nothing to what it does not see."""
    s = ref.Setup([w], [300], 1, 64, 16, e4m3, seed=w)
    s.write_all()
    q = torch.randn((w, 2, 64), generator=s.gen).to(torch.bfloat16).cuda()
    lse = (2 + torch.rand((w, 2), generator=s.gen)).cuda()
    lse[1], lse[2, 1] = torch.finfo(torch.float32).min, -3e38
    out = dict(mass=torch.zeros((1, 1, 300 + w), device="cuda"))
    sdm.attend_weight(s.cache, q, lse, s.cu, s.ctx, w, window=window, sinks=2, out=out, dev_status=s.status)
    want, tol = weights(q, lse, s.held(0, "k"), ref.visible(w, 300, window, 2), 0.125, 2)
    got, fine = out["mass"][0].double().cpu().numpy(), np.isfinite(want)
    assert s.status.item() == 0 and not fine.all() and (w == 3 or fine.sum() > 150)
    assert np.isposinf(got[~fine]).all() and (np.abs(got - want)[fine] <= tol[fine]).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("power", [-115, -60, 100, 113, 116, 118, 124])
@pytest.mark.parametrize("w", [1, 5, 60])
def test_queries_of_any_size_over_an_e4m3_cache(gpu_lib, D, power, w):
    """Queries near the type's ends beside keys of the other end: scores of
    ordinary size."""
    s = ref.Setup([w], [300], 1, D, 16, True, seed=w)
    s.kv[0]["k"] *= 2.0 ** (-112 if power > 0 else 40)
    s.write_all()
    q = (torch.randn((w, 4, D), generator=s.gen) * 2.0 ** power).to(torch.bfloat16).cuda()
    lse = (2 + torch.rand((w, 4), generator=s.gen)).cuda()
    scale = 2.0 ** ((112 if power > 0 else -40) - power - 3)
    out = dict(mass=torch.zeros((1, 1, 300 + w), device="cuda"))
    sdm.attend_weight(s.cache, q, lse, s.cu, s.ctx, w, scale=scale, out=out, dev_status=s.status)
    want, tol = weights(q, lse, s.held(0, "k"), ref.visible(w, 300), scale, 4)
    assert s.status.item() == 0 and np.isfinite(want).all() and want.std() > 0.02
    assert (np.abs(out["mass"][0].double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group,w", [(7, 18), (7, 11), (1, 3), (16, 8)])
def test_huge_and_small_queries_of_one_tile(gpu_lib, D, group, w):
    """Rows of all sizes side by side, a window, rows that add nothing."""
    s = ref.Setup([w, 1, w], [300, 40, 700], 2, D, 32, True, seed=group)
    for kv in s.kv:
        kv["k"] *= 2.0 ** -100
    s.write_all()
    rows, H = s.rows, 2 * group
    size = 2.0 ** torch.randint(60, 120, (rows, H, 1), generator=s.gen).double()
    size[rows // 2:] = 2.0 ** 96                                   # the last request has no huge row
    q = (torch.randn((rows, H, D), generator=s.gen).double() * size).to(torch.bfloat16).cuda()
    scale = 2.0
    top = (q.double().abs().amax(-1) * 2.0 ** -98 * D ** 0.5).cpu()  # some way above a row's scores
    lse = (top * scale).clamp(min=1.0).float().cuda()
    lse[1, 0], lse[rows - 1] = -INF, INF
    for window, sinks in ((0, 0), (50, 3)):
        out = dict(mass=torch.zeros((3, 2, 700 + w), device="cuda"))
        sdm.attend_weight(s.cache, q, lse, s.cu, s.ctx, w, scale=scale, window=window, sinks=sinks, out=out,
                          dev_status=s.status)
        assert s.status.item() == 0
        cu = s.cu.tolist()
        for i in range(3):
            a, b, n = cu[i], cu[i + 1], s.ctx_list[i] + cu[i + 1] - cu[i]
            want, tol = weights(q[a:b], lse[a:b], s.held(i, "k"), ref.visible(b - a, s.ctx_list[i], window, sinks), scale, group)
            got = out["mass"][i, :, :n].double().cpu().numpy()
            assert np.isfinite(want).all() and (np.abs(got - want) <= tol).all(), (window, i)


@pytest.mark.parametrize("e4m3", [False, True])
def test_infinite_weights_of_long_windows(gpu_lib, e4m3):
    """An infinite weight among the sums of many tiles of rows stays infinite."""
    s = ref.Setup([1000], [3000], 2, 64, 64, e4m3, seed=21)
    s.write_all()
    q = torch.randn((1000, 16, 64), generator=s.gen).to(torch.bfloat16).cuda()
    lse = (5 + torch.rand((1000, 16), generator=s.gen)).cuda()
    lse[3, 2], lse[400, 9] = torch.finfo(torch.float32).min, -1e30
    out = dict(mass=torch.zeros((1, 2, 4000), device="cuda"))
    sdm.attend_weight(s.cache, q, lse, s.cu, s.ctx, 1000, out=out, dev_status=s.status)
    want, tol = weights(q, lse, s.held(0, "k"), ref.visible(1000, 3000), 0.125, 8)
    got, fine = out["mass"][0].double().cpu().numpy(), np.isfinite(want)
    assert s.status.item() == 0 and (~fine).sum() == 3004 + 3401
    assert np.isposinf(got[~fine]).all() and (np.abs(got - want)[fine] <= tol[fine]).all()

"""The attention weight of cached tokens and the eviction by it, against plain
forms in 64 bits."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from speculative_decoding_markov_gb300 import binding as sdm
from tests import paged_reference as ref

pytestmark = pytest.mark.gpu
INF = float("inf")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def weights(q, lse, k, see, scale, group):
    """[G, n]: what the rows q [w, H, D] give the tokens k [n, G, D], and a
    bound on its error: the score's 2 D fp32 roundings, those of score and lse,
    2^x's, and the sum's."""
    w, H, D = q.shape
    n, G = k.shape[:2]
    out, tol = np.zeros((G, n)), np.zeros((G, n))
    q, k, lse = q.double().cpu().numpy(), k.double().cpu().numpy(), lse.double().cpu().numpy()
    for h in range(H):
        g = h // group
        with np.errstate(invalid="ignore", over="ignore"):
            s = scale * q[:, h] @ k[:, g].T
            size = scale * np.abs(q[:, h]) @ np.abs(k[:, g]).T
            x = np.where(see & ~np.isneginf(lse[:, h, None]), np.exp(s - lse[:, h, None]), 0.0)
            off = 2.0 ** -23 * (D * size + 4 * np.abs(s) + 4 * np.abs(lse[:, h, None])) + 2.0 ** -21
        out[g] += x.sum(0)
        tol[g] += np.where(x > 0, x * off, 0.0).sum(0)
    return out, tol + 2.0 ** -23 * (w * group + 4) * out + 1e-37


def check(s, H, window=0, sinks=0, count=None, path=None, seed=0, scale=None, own_lse=True):
    """attend's lse, then attend_weight twice (apart and in place)."""
    G, D, R = s.G, s.D, len(s.w)
    q = torch.randn((s.rows, H, D), generator=s.gen).to(torch.bfloat16).cuda()
    scale = D ** -0.5 if scale is None else scale
    count_list = s.w if count is None else count
    top = max(list(count_list) + [1])
    if own_lse:
        got = sdm.attend(s.cache, q, s.cu, s.ctx, max(max(s.w), 1), scale=scale, window=window, sinks=sinks, lse=True,
                         dev_status=s.status)
        lse = got["lse"]
    else:
        lse = (3 * torch.randn((s.rows, H), generator=s.gen)).cuda() + 2
    T = max(a + b for a, b in zip(s.w, s.ctx_list)) + 5
    before = torch.rand((R, G, T), generator=s.gen).cuda()
    kw = dict(count=None if count is None else i32(count), path=None if path is None else i32(path), scale=scale,
              window=window, sinks=sinks, dev_status=s.status)
    out = dict(mass=torch.full((R, G, T), -7.0, device="cuda"))
    sdm.attend_weight(s.cache, q, lse, s.cu, s.ctx, top, mass=before, out=out, **kw)
    again = dict(mass=before.clone())
    sdm.attend_weight(s.cache, q, lse, s.cu, s.ctx, top, mass=again["mass"], out=again, **kw)
    fresh = dict(mass=torch.full((R, G, T), -7.0, device="cuda"))
    sdm.attend_weight(s.cache, q, lse, s.cu, s.ctx, top, out=fresh, **kw)
    cu = s.cu.tolist()
    for i in range(R):
        n, ctx = count_list[i], s.ctx_list[i]
        off = list(range(n)) if path is None else path[i][:n]
        rows = [cu[i] + o for o in off]
        k = s.held(i, "k")[:ctx + n]
        see = ref.visible(n, ctx, window, sinks)
        want, tol = weights(q[rows], lse[rows], k, see, scale, H // G)
        old = before[i].double().cpu().numpy()[:, :ctx + n].copy()
        old[:, ctx:] = 0
        err = np.abs(out["mass"][i, :, :ctx + n].double().cpu().numpy() - want - old)
        assert (err <= tol + 2.0 ** -24 * (want + old)).all(), (i, err.max())
        err = np.abs(fresh["mass"][i, :, :ctx + n].double().cpu().numpy() - want)
        assert (err <= tol).all(), (i, err.max())
        assert torch.equal(out["mass"][i, :, :ctx + n], again["mass"][i, :, :ctx + n])
        assert (out["mass"][i, :, ctx + n:] == -7).all()
        assert torch.equal(again["mass"][i, :, ctx + n:], before[i, :, ctx + n:])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("G,group,D,page", [(2, 4, 128, 16), (1, 7, 128, 64), (3, 1, 64, 32), (2, 16, 64, 128)])
@pytest.mark.parametrize("w,ctx", [([1], [0]), ([1], [500]), ([1, 3, 0, 8], [127, 128, 40, 1000]), ([5, 300], [3000, 17])])
def test_windows(gpu_lib, e4m3, G, group, D, page, w, ctx):
    s = ref.Setup(w, ctx, G, D, page, e4m3, seed=G)
    s.write_all()
    check(s, G * group)
    assert s.status.item() == 0


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("window,sinks", [(1, 0), (20, 3), (128, 4), (130, 200), (700, 0), (10 ** 6, 5)])
def test_sliding_windows(gpu_lib, e4m3, window, sinks):
    s = ref.Setup([1, 6, 200], [900, 333, 150], 2, 64, 16, e4m3, seed=3)
    s.write_all()
    check(s, 6, window=window, sinks=sinks)
    assert s.status.item() == 0


@pytest.mark.parametrize("e4m3", [False, True])
def test_some_of_the_rows_and_paths(gpu_lib, e4m3):
    s = ref.Setup([8, 8, 3], [200, 0, 511], 2, 128, 16, e4m3, seed=4)
    s.write_all()
    check(s, 8, count=[3, 8, 1], own_lse=False)
    check(s, 8, count=[4, 2, 0], path=[[0, 2, 3, 7, -1], [0, 7, -1, -1, -1], [0, 1, 2, -1, -1]], own_lse=False)
    assert s.status.item() == 0


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("w,group", [(65, 4), (64, 4), (130, 2), (33, 128), (2, 128), (700, 5), (129, 7)])
def test_many_rows_a_head(gpu_lib, e4m3, w, group):
    s = ref.Setup([w], [260], 1, 64, 16, e4m3, seed=w)
    s.write_all()
    check(s, group)
    s = ref.Setup([w, 3], [5, 700], 2, 128, 64, e4m3, seed=w)
    s.write_all()
    check(s, 2 * group)
    assert s.status.item() == 0


@pytest.mark.parametrize("e4m3", [False, True])
def test_long_paths_and_parts_of_long_windows(gpu_lib, e4m3):
    s = ref.Setup([100, 300], [260, 5], 2, 64, 16, e4m3, seed=12)
    s.write_all()
    check(s, 8, count=[70, 41], own_lse=False)
    path = [sorted(np.random.default_rng(i).permutation(n)[:70].tolist()) for i, n in enumerate((100, 300))]
    check(s, 8, count=[70, 69], path=path, own_lse=False)
    check(s, 8, count=[70, 69], path=path, own_lse=False, window=50, sinks=7)
    assert s.status.item() == 0


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_every_number_of_rows_over_short_contexts(gpu_lib, e4m3, D):
    """Heads of 4 to 128 rows, a unit or two of keys each: the next head's rows
    are made ready while this one's are multiplied."""
    w = list(range(1, 33))
    s = ref.Setup(w, [(37 * k) % 400 for k in w], 2, D, 32, e4m3, seed=17)
    s.write_all()
    check(s, 8)
    check(s, 8, window=90, sinks=2, own_lse=False)
    assert s.status.item() == 0


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_long_windows_whose_units_have_one_tile_or_two(gpu_lib, e4m3, D):
    """An odd and an even number of tiles of rows a unit, units of one tile of
    keys between units of two, heads that follow one another."""
    s = ref.Setup([100, 513, 65, 290], [20, 0, 300, 100], 3, D, 64, e4m3, seed=18)
    s.write_all()
    for _ in range(2):
        check(s, 12)
    check(s, 12, window=77, sinks=5, own_lse=False)
    assert s.status.item() == 0


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("G,window,sinks,count", [(1, 100, 3, None), (8, 700, 300, None), (2, 1, 0, [1, 0, 2, 0])])
def test_long_contexts_of_which_little_is_seen(gpu_lib, e4m3, G, window, sinks, count):
    """Weights that only pass through, many units at a time."""
    s = ref.Setup([1, 4, 2, 1], [60001, 20011, 257, 40448], G, 64, 64, e4m3, seed=19)
    s.write_all()
    check(s, 2 * G, window=window, sinks=sinks, count=count, own_lse=False)
    assert s.status.item() == 0


@pytest.mark.parametrize("keep", [300, 70000])
@pytest.mark.parametrize("G", [2, 160])
def test_runs_of_slots_that_a_block_cannot_hold(gpu_lib, keep, G):
    """More slots than one block's shared memory has keys for, with few heads
    and with more than fill the SMs; weights that are often equal."""
    n = 100003
    gen = torch.Generator().manual_seed(G + keep)
    table = torch.zeros((1, -(-n // 128)), dtype=torch.int32, device="cuda")
    table[0] = torch.arange(table.shape[1], dtype=torch.int32, device="cuda")
    cache = sdm.PagedCache.empty(table.shape[1], G, 128, 64, table)
    cache.k.view(torch.int16).copy_(torch.arange(n // 128 + 1, device="cuda")[:, None, None, None] * 128 % 32003 +
                                    torch.arange(128, device="cuda")[None, None, :, None])
    before = cache.k.view(torch.int16).permute(1, 0, 2, 3).reshape(G, -1, 64)[:, :, 0].clone()
    mass = torch.randint(0, 5000, (1, G, n), generator=gen).float().cuda()
    pos = torch.arange(n, dtype=torch.int32, device="cuda").expand(1, G, n).contiguous()
    out = dict(mass=torch.zeros_like(mass), pos=torch.zeros_like(pos),
               length=torch.zeros((1,), dtype=torch.int32, device="cuda"))
    status = sdm.new_status()
    sdm.cache_evict(cache, mass, pos, i32([n]), i32([n]), keep, sinks=4, recent=9, out=out, dev_status=status)
    assert status.item() == 0 and out["length"].item() == keep
    key = mass[0].clone()
    key[:, :4] = key[:, n - 9:] = 1e30
    order = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :keep]
    want = torch.sort(order, dim=1).values
    got = out["pos"][0, :, :keep].long()
    assert torch.equal(torch.sort(got, dim=1).values, want)
    assert torch.equal(out["mass"][0, :, :keep], mass[0].gather(1, got))
    after = cache.k.view(torch.int16).permute(1, 0, 2, 3).reshape(G, -1, 64)[:, :keep]
    assert torch.equal(after[:, :, 0], before.gather(1, got)) and torch.equal(after[:, :, 63], after[:, :, 0])


@pytest.mark.parametrize("e4m3", [False, True])
def test_heads_that_end_in_a_single_tile_of_keys(gpu_lib, e4m3):
    """Units of one tile of keys, which only one half of the threads multiplies,
    between units of two: each half waits for its own products all the same."""
    rng = np.random.default_rng(15)
    ctx = [int(rng.choice([3, 60, 100, 300, 250, 500, 20, 513])) for _ in range(60)]
    s = ref.Setup([2] * 60, ctx, 4, 64, 16, e4m3, seed=15)         # a head's rows in one tile
    s.write_all()
    for _ in range(3):
        check(s, 8)
    s = ref.Setup([1300, 1100, 1420], [0, 10, 0], 8, 64, 32, e4m3, seed=16)   # many rows, few of which see a key
    s.write_all()
    for window, sinks in ((23, 0), (61, 1), (5, 0)):
        check(s, 16, window=window, sinks=sinks, own_lse=False)
    assert s.status.item() == 0


def test_many_requests_with_many_rows(gpu_lib):
    rng = np.random.default_rng(13)
    w, ctx = rng.integers(0, 60, 50).tolist(), rng.integers(0, 900, 50).tolist()
    s = ref.Setup(w, ctx, 1, 128, 32, False, seed=13)
    s.write_all()
    check(s, 4)
    assert s.status.item() == 0


@pytest.mark.parametrize("rows", [0, 3])
def test_weights_of_no_rows(gpu_lib, rows):
    """Without counted rows the old weights stay, and no other entry changes."""
    s = ref.Setup([rows], [200], 2, 64, 16, False, seed=14)
    s.write_all()
    q, lse = torch.ones((rows, 4, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((rows, 4), device="cuda")
    mass = torch.rand((1, 2, 220), generator=s.gen).cuda()
    out = dict(mass=torch.full_like(mass, -7))
    sdm.attend_weight(s.cache, q, lse, s.cu, s.ctx, 3, mass=mass, count=i32([0]), out=out, dev_status=s.status)
    assert torch.equal(out["mass"][:, :, :200], mass[:, :, :200]) and (out["mass"][:, :, 200:] == -7).all()
    assert s.status.item() == 0


def test_many_requests_of_all_lengths(gpu_lib):
    rng = np.random.default_rng(5)
    w, ctx = rng.integers(0, 9, 70).tolist(), rng.integers(0, 700, 70).tolist()
    s = ref.Setup(w, ctx, 2, 64, 16, False, seed=5)
    s.write_all()
    check(s, 4)
    assert s.status.item() == 0


@pytest.mark.parametrize("e4m3", [False, True])
def test_odd_values_reach_only_their_token(gpu_lib, e4m3):
    """NaN and infinite keys, rows that saw nothing, rows of infinite lse."""
    s = ref.Setup([3], [300], 1, 128, 16, e4m3, seed=6)
    s.kv[0]["k"][17, 0, 3] = float("nan")
    s.kv[0]["k"][140, 0, 9] = INF
    s.write_all()
    q = torch.randn((3, 2, 128), generator=s.gen).to(torch.bfloat16).cuda()
    lse = torch.tensor([[1.0, 2.0], [-INF, INF], [0.5, 0.0]], device="cuda")
    out = dict(mass=torch.zeros((1, 1, 320), device="cuda"))
    sdm.attend_weight(s.cache, q, lse, s.cu, s.ctx, 3, out=out, dev_status=s.status)
    k = s.held(0, "k")
    want, tol = weights(q, lse, k, ref.visible(3, 300), 128 ** -0.5, 2)
    got = out["mass"][0, :, :303].double().cpu().numpy()
    fine = np.isfinite(want) & np.isfinite(tol)
    assert np.isnan(got[0, 17]) and fine.sum() >= 301
    assert (np.abs(got - want)[fine] <= tol[fine]).all()
    assert s.status.item() == 0


def test_weights_what_the_device_finds_wrong(gpu_lib):
    s = ref.Setup([4, 4], [100, 50], 1, 64, 16, False, seed=7)
    s.write_all()
    q = torch.randn((8, 2, 64), generator=s.gen).to(torch.bfloat16).cuda()
    lse = torch.zeros((8, 2), device="cuda")

    def call(mc=4, stride=200, cu=s.cu, ctx=s.ctx, **kw):
        st = sdm.new_status()
        out = dict(mass=torch.full((2, 1, stride), -7.0, device="cuda"))
        sdm.attend_weight(s.cache, q, lse, cu, ctx, mc, out=out, dev_status=st, **kw)
        return st.item(), out["mass"]

    assert call()[0] == 0
    st, m = call(mc=2)                                             # windows longer than max_count
    assert st == sdm.DEV_BAD_WINDOW and (m[0, 0, 102:] == -7).all() and (m[0, 0, :102] >= 0).all()
    assert call(count=i32([5, 0]), mc=8)[0] == sdm.DEV_BAD_WINDOW
    assert call(count=i32([-1, 0]))[0] == sdm.DEV_BAD_WINDOW
    assert call(ctx=i32([-3, 5]))[0] == sdm.DEV_BAD_WINDOW
    assert call(cu=i32([0, 9, 8]))[0] == sdm.DEV_BAD_WINDOW
    assert call(count=i32([2, 2]), path=i32([[0, 4], [0, 1]]), mc=2)[0] == sdm.DEV_BAD_WINDOW
    st, m = call(stride=101)
    assert st == sdm.DEV_BAD_PAGE and (m[0] >= 0).all()
    s.cache.table[1, 2] = -5
    assert call()[0] == sdm.DEV_BAD_PAGE


def test_the_same_weights_on_every_run(gpu_lib):
    s = ref.Setup([300, 1, 9], [5000, 9000, 100], 2, 128, 64, False, seed=8)
    s.write_all()
    q = torch.randn((s.rows, 8, 128), generator=s.gen).to(torch.bfloat16).cuda()
    lse = sdm.attend(s.cache, q, s.cu, s.ctx, 300, lse=True)["lse"]
    got = []
    for _ in range(3):
        out = dict(mass=torch.zeros((3, 2, 9100), device="cuda"))
        sdm.attend_weight(s.cache, q, lse, s.cu, s.ctx, 300, out=out, dev_status=s.status)
        got.append(out["mass"])
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2]) and s.status.item() == 0


# ---------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------
def plain_evict(mass, pos, ctx, count, start, keep, sinks, recent):
    """One head: the slots' sources after the cut, their weights and positions."""
    n = ctx + count
    at = np.array(list(pos[:ctx]) + [start + j for j in range(count)], dtype=np.int64)
    order = sorted(range(n), key=lambda s: (0 if at[s] < sinks or at[s] >= start + count - recent else 1,
                                            0.0 if at[s] < sinks or at[s] >= start + count - recent
                                            else INF if np.isnan(mass[s]) else -mass[s], s))
    kept = sorted(order[:keep])
    src = np.arange(min(n, keep))
    holes = [s for s in range(min(n, keep)) if s not in set(kept)]
    late = [s for s in kept if s >= keep]
    assert len(holes) == len(late)
    src[holes] = late
    return src, mass[src], at[src]


def random_positions(R, G, ctx, start, stride, rng):
    pos = np.full((R, G, stride), -9, np.int32)
    for i in range(R):
        for g in range(G):
            pos[i, g, :ctx[i]] = rng.permutation(start[i])[:ctx[i]]
    return pos


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("e4m3,D,page", [(False, 128, 16), (True, 128, 64), (True, 64, 32), (False, 64, 128)])
@pytest.mark.parametrize("ctx,count,keep,sinks,recent", [
    ([1], [0], 1, 0, 0), ([0], [1], 1, 1, 0), ([10, 40, 3], [2, 0, 5], 9, 2, 3), ([64, 64, 60], [8, 1, 4], 64, 4, 16),
    ([0, 0], [700, 5], 33, 4, 29), ([500], [8], 8, 0, 8), ([300, 299], [0, 1], 299, 0, 0), ([90], [4], 500, 4, 4)])
def test_cuts(gpu_lib, in_place, e4m3, D, page, ctx, count, keep, sinks, recent):
    R, G, rng = len(ctx), 2, np.random.default_rng(sum(ctx) + keep)
    s = ref.Setup(count, ctx, G, D, page, e4m3, seed=keep)
    s.write_all()
    start = [c + 37 * (c > 0) for c in ctx]
    stride = max(a + b for a, b in zip(ctx, count)) + 3
    mass = np.exp(2 * rng.standard_normal((R, G, stride))).astype(np.float32)
    mass[rng.random(mass.shape) < 0.3] = 0.0                       # ties
    pos = random_positions(R, G, ctx, start, stride, rng)
    m, p = torch.tensor(mass).cuda(), torch.tensor(pos).cuda()
    out = dict(length=i32([0] * R), next=i32([0] * R))
    if in_place:
        out.update(mass=m, pos=p)
    else:
        out.update(mass=torch.full_like(m, -7), pos=torch.full_like(p, -7))
    sdm.cache_evict(s.cache, m, p, s.ctx, i32(start), keep, count=i32(count), sinks=sinks, recent=recent, out=out,
                    dev_status=s.status)
    assert s.status.item() == 0
    assert out["length"].tolist() == [min(a + b, keep) for a, b in zip(ctx, count)]
    assert out["next"].tolist() == [a + b for a, b in zip(start, count)]
    n = out["length"].tolist()
    back = sdm.cache_read(s.cache, i32(np.concatenate([[0], np.cumsum(n)]).tolist()), sum(n))
    row = 0
    for i in range(R):
        for g in range(G):
            src, wm, wp = plain_evict(mass[i, g], pos[i, g], ctx[i], count[i], start[i], keep, sinks, recent)
            assert np.array_equal(out["mass"][i, g, :n[i]].cpu().numpy(), wm)
            assert np.array_equal(out["pos"][i, g, :n[i]].cpu().numpy(), wp)
            for name in "kv":
                held = s.held(i, name)[src, g]
                assert torch.equal(back[name][row:row + n[i], g].double().cpu(), held), (i, g, name)
        if not in_place:
            assert (out["mass"][i, :, n[i]:] == -7).all() and (out["pos"][i, :, n[i]:] == -7).all()
        row += n[i]


@pytest.mark.parametrize("R,n,keep", [(1, 70000, 30000), (1, 20001, 20000), (3, 9000, 100), (40, 3000, 2992),
                                      (80, 6000, 700), (40, 3000, 2983), (40, 3000, 2984), (1, 450000, 449000)])
def test_long_caches(gpu_lib, R, n, keep):
    """Several CTAs a head, against a sort."""
    G, D, page = 2, 64, 64
    gen = torch.Generator().manual_seed(n)
    pages = -(-n // page)
    table = torch.randperm(R * pages, generator=gen).to(torch.int32).view(R, pages).cuda()
    cache = sdm.PagedCache.empty(R * pages, G, page, D, table)
    for x in (cache.k, cache.v):
        x.copy_(torch.randn(x.shape, generator=gen).to(torch.bfloat16))
    mass = torch.rand((R, G, n), generator=gen).mul(500).round().div(16).cuda()       # many ties
    mass[:, :, 1000:1300] = torch.randn((R, G, 300), generator=gen).cuda()            # negative ones
    pos = torch.zeros((R, G, n), dtype=torch.int32, device="cuda")
    before = {x: cache_rows(cache, x, n) for x in "kv"}
    st = sdm.new_status()
    out = dict(mass=torch.zeros_like(mass), pos=torch.zeros_like(pos), length=i32([0] * R))
    sdm.cache_evict(cache, mass, pos, i32([0] * R), None, keep, count=i32([n] * R), sinks=4, recent=50, out=out,
                    dev_status=st)
    assert st.item() == 0 and out["length"].tolist() == [keep] * R
    key = mass.clone()
    key[:, :, :4] = key[:, :, n - 50:] = INF
    order = torch.sort(key, dim=-1, descending=True, stable=True)[1][:, :, :keep]
    kept = torch.zeros_like(key, dtype=torch.bool).scatter_(2, order, True)
    src = torch.arange(keep, device="cuda").repeat(R, G, 1)
    src[~kept[:, :, :keep]] = torch.nonzero(kept[:, :, keep:], as_tuple=True)[2] + keep
    assert torch.equal(out["pos"][:, :, :keep].long(), src)
    assert torch.equal(out["mass"][:, :, :keep], mass.gather(2, src))
    for x in "kv":
        after = cache_rows(cache, x, keep)
        assert torch.equal(after, before[x].gather(2, src[..., None].expand(-1, -1, -1, D)))


def cache_rows(cache, name, n):
    """[R, G, n, D] of a bf16 cache."""
    x = getattr(cache, name)[cache.table.long()]
    return x.permute(0, 2, 1, 3, 4).reshape(x.shape[0], x.shape[2], -1, x.shape[4])[:, :, :n].clone()


def test_weights_that_are_no_numbers(gpu_lib):
    s = ref.Setup([0], [6], 1, 64, 16, False, seed=9)
    s.write_all()
    mass = torch.tensor([[[1.0, float("nan"), INF, -INF, -0.0, 0.0]]], device="cuda")
    pos = torch.arange(6, dtype=torch.int32, device="cuda").view(1, 1, 6)
    for keep, want in ((1, [2]), (2, [0, 2]), (3, [0, 4, 2]), (4, [0, 5, 2, 4]), (5, [0, 4, 2, 3, 5])):
        out = dict(mass=torch.zeros_like(mass), pos=torch.zeros_like(pos), length=i32([0]))
        sdm.cache_evict(s.cache, mass, pos, s.ctx, None, keep, out=out, dev_status=s.status)
        assert sorted(out["pos"][0, 0, :keep].tolist()) == sorted(want), keep
    assert s.status.item() == 0


def test_evictions_what_the_device_finds_wrong(gpu_lib):
    s = ref.Setup([0, 0], [40, 40], 1, 64, 16, False, seed=10)
    s.write_all()
    mass = torch.rand((2, 1, 50), generator=s.gen).cuda()
    pos = torch.arange(50, dtype=torch.int32, device="cuda").repeat(2, 1, 1)

    def call(ctx, count, keep=10, stride=50):
        st = sdm.new_status()
        out = dict(mass=torch.zeros_like(mass), pos=torch.zeros_like(pos), length=i32([0, 0]))
        sdm.cache_evict(s.cache, mass, pos, i32(ctx), None, keep, count=i32(count), out=out, dev_status=st)
        return st.item(), out["length"].tolist()

    assert call([40, 40], [0, 0]) == (0, [10, 10])
    assert call([-1, 40], [3, -2]) == (sdm.DEV_BAD_WINDOW, [3, 10])
    assert call([40, 40], [11, 0], keep=60) == (sdm.DEV_BAD_PAGE, [50, 40])
    s.cache.table[0, 0] = 999
    assert call([40, 40], [0, 0])[0] == sdm.DEV_BAD_PAGE

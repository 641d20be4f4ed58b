"""Rotation in place beside windows that are not sound."""
from __future__ import annotations

import pytest
import torch

from speculative_decoding_markov_gb300 import binding as sdm
from tests import paged_reference as ref
from tests.test_gpu_rotate import freqs, i32, rows_of

pytestmark = pytest.mark.gpu


def alone(q, k, row, pos, **kw):
    """One row's queries and keys by a call of its own."""
    got = sdm.qk_rotate(q[row:row + 1], k[row:row + 1], i32([0, 1]), None, freqs(q.shape[2]).cuda(), start=i32([pos]), **kw)
    return got["q"][0], got["k"][0]


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("H", [4, 40])
@pytest.mark.parametrize("cu,ctx", [
    ([0, 3, 3, 9], [5, -1, 70]), ([0, 0, 3000], [-7, 12]), ([0, 3, 1, 9], [0, 14, 5]), ([0, 5, 3, 9, 9], [9, 1, 400, -2]),
    ([0, 1500, 9, 2900, -1, 40], [3, 1, 60, 0, 7]), ([4, 2, 3000, 2990, 3000], [8, 11, 2, 30])])
def test_in_place_every_row_is_turned_once(gpu_lib, norm, H, cu, ctx):
    """A window that counts as empty leaves the others' rows as they are without
    it; where offsets make two windows hold a row, it is one of theirs."""
    G, D, gen = 2, 64, torch.Generator().manual_seed(len(cu) + H)
    rows = max(cu)
    q, k = rows_of(rows, H, D, gen), rows_of(rows, G, D, gen)
    w = dict(q_weight=(1 + torch.rand((D,), generator=gen)).cuda(), k_weight=torch.ones(D).cuda()) if norm else {}
    sound = [i for i in range(len(ctx)) if 0 <= cu[i] <= cu[i + 1] <= rows]
    holders = [[i for i in sound if cu[i] <= r < cu[i + 1]] for r in range(rows)]
    assert any(holders) and rows < 4000
    by = {i: sdm.qk_rotate(q, k, i32([0, rows]), None, freqs(D).cuda(), start=i32([max(ctx[i], 0) - cu[i]]), **w) for i in sound}
    one = alone(q, k, cu[sound[-1]], max(ctx[sound[-1]], 0), **w) if cu[sound[-1]] < rows else None
    if one:                                                        # the comparison itself, for one row
        assert torch.equal(one[0], by[sound[-1]]["q"][cu[sound[-1]]])
    for _ in range(5):
        x, y, st = q.clone(), k.clone(), sdm.new_status()
        sdm.qk_rotate(x, y, i32(cu), i32(ctx), freqs(D).cuda(), out=dict(q=x, k=y), dev_status=st, **w)
        assert st.item() == sdm.DEV_BAD_WINDOW
        fits_q, fits_k = (torch.zeros(rows, dtype=torch.bool, device="cuda") for _ in range(2))
        for i in sound:
            a, b = cu[i], cu[i + 1]
            fits_q[a:b] |= (x[a:b] == by[i]["q"][a:b]).flatten(1).all(1)
            fits_k[a:b] |= (y[a:b] == by[i]["k"][a:b]).flatten(1).all(1)
        free = torch.tensor([not h for h in holders], device="cuda")
        assert (fits_q | free).all() and (fits_k | free).all()
        assert torch.equal(x[free], q[free]) and torch.equal(y[free], k[free])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("H", [2, 40])
def test_in_place_into_a_cache_beside_unsound_windows(gpu_lib, e4m3, H):
    """The queries once, every sound window's keys and values in its slots."""
    G, D, gen = 2, 64, torch.Generator().manual_seed(H)
    q, k, v = (rows_of(20, h, D, gen) for h in (H, G, G))
    cu, ctx = [0, 9, 4, 20, 20], [3, 5, 30, -1]
    a, b = (ref.Setup([9, 0, 16, 0], [3, 5, 30, 0], G, D, 16, e4m3, fill=0.0) for _ in range(2))
    x, st = q.clone(), sdm.new_status()
    sdm.qk_rotate(x, k, i32(cu), i32(ctx), freqs(D).cuda(), v=v, cache=a.cache, out=dict(q=x), dev_status=st)
    assert st.item() == sdm.DEV_BAD_WINDOW
    by = []
    for i, (lo, hi) in ((0, (0, 9)), (2, (4, 20))):                # the two sound windows, each by itself
        n = hi - lo
        one = sdm.PagedCache(b.cache.k, b.cache.v, b.cache.table[i:i + 1].contiguous(), b.cache.k_exp, b.cache.v_exp)
        by.append(sdm.qk_rotate(q[lo:hi], k[lo:hi], i32([0, n]), i32([ctx[i]]), freqs(D).cuda(), v=v[lo:hi], cache=one)["q"])
    same0, same2 = (x[:9] == by[0]).flatten(1).all(1), (x[4:] == by[1]).flatten(1).all(1)
    assert same0[:4].all() and same2[5:].all() and (same0[4:] | same2[:5]).all()
    for n in ("k", "v", "k_exp", "v_exp"):
        p, r = getattr(a.cache, n), getattr(b.cache, n)
        if p is not None:
            assert torch.equal(p.view(torch.uint8), r.view(torch.uint8)), n


@pytest.mark.parametrize("first", [0, 100000, 2 ** 24, -3000])
@pytest.mark.parametrize("inter", [False, True])
def test_the_angle_keeps_what_32_bits_of_turns_lose(gpu_lib, first, inter):
    """The turned unit vectors' sines and cosines below 1/4: the 32-bit functions'
    last bit and a product's rounding are 2.3e-8 of them, so that whoever is 3e-8
    from a border of bf16's rounding is on its side.  (An angle cut to 24 bits of
    turns is off by up to 9e-8.)"""
    n, D = 16384, 128
    q = torch.zeros((n, 1, D), dtype=torch.bfloat16, device="cuda")
    q[..., (slice(0, D, 2) if inter else slice(0, D // 2))] = 1.0
    freq = freqs(D).cuda()
    got = sdm.qk_rotate(q, q.clone(), i32([0, n]), None, freq, start=i32([first]), interleaved=inter)["q"][:, 0]
    t = (first + torch.arange(n, device="cuda", dtype=torch.float64))[:, None] * freq
    parts = [(torch.cos(t), got[:, 0::2] if inter else got[:, :D // 2]), (torch.sin(t), got[:, 1::2] if inter else got[:, D // 2:])]
    for y, x in parts:
        step = 2.0 ** (torch.floor(torch.log2(y.abs().clamp(min=1e-30))) - 7)
        off = ((y.abs() / step) % 1.0 - 0.5).abs() * step
        sure = (off > 3e-8) & (y.abs() < 0.25)
        assert sure.sum() > 10000 and torch.equal(x[sure], y.to(torch.bfloat16)[sure])

"""Norm and rotation of queries and keys, with and without the cache, against
the formula in 64 bits and against cache_write."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from speculative_decoding_markov_gb300 import binding as sdm
from tests import paged_reference as ref

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def freqs(rot, base=10000.0):
    return base ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)


def formula(x, pos, freq, weight, eps, inter):
    """Rows [n, heads, D] in 64 bits, and each element's pair's size."""
    x = x.double().cpu()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double().cpu()
    y, size = x.clone(), x.abs()
    half = freq.numel()
    for j in range(half):
        a, b = (2 * j, 2 * j + 1) if inter else (j, j + half)
        t = pos.double() * freq[j]
        c, s = torch.cos(t)[:, None], torch.sin(t)[:, None]
        y[..., a], y[..., b] = c * x[..., a] - s * x[..., b], c * x[..., b] + s * x[..., a]
        size[..., a] = size[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, size


def close(got, want, size):
    """Half a bf16 step of the result; before it some 16 fp32 roundings of the
    norm, the angle's (half a turn has 2^-24 pi) and the rotation's."""
    err = (got.double().cpu() - want).abs()
    assert (err <= 2.0 ** -8 * want.abs() + 2.0 ** -19 * size).all(), (err - 2.0 ** -8 * want.abs()).max()


def rows_of(n, heads, D, gen, wide=0):
    """A slice of a wider projection's output."""
    x = torch.randn((n, heads * D + wide), generator=gen).to(torch.bfloat16).cuda()
    return x[:, :heads * D].view(n, heads, D) if wide == 0 else x.as_strided((n, heads, D), (heads * D + wide, D, 1))


@pytest.mark.parametrize("D,rot,inter,norm", [(128, 128, False, True), (128, 64, False, False), (128, 128, True, True),
                                              (64, 64, False, True), (64, 24, True, False), (128, 24, False, True),
                                              (64, 0, False, True), (128, 8, True, True), (64, 0, False, False)])
@pytest.mark.parametrize("w,start", [([1], [0]), ([3, 0, 1, 9], [7, 5, 120000, 0]), ([700], [2 ** 20])])
def test_rows_against_the_formula(gpu_lib, D, rot, inter, norm, w, start):
    H, G, gen = 6, 2, torch.Generator().manual_seed(D + rot + len(w))
    n = sum(w)
    q, k = rows_of(n, H, D, gen, 40), rows_of(n, G, D, gen, 8)
    wq, wk = ((1 + 0.5 * torch.randn((D,), generator=gen)).cuda() if norm else None for _ in range(2))
    freq = freqs(rot)
    cu = i32(np.concatenate([[0], np.cumsum(w)]).tolist())
    got = sdm.qk_rotate(q, k, cu, None, freq.cuda() if rot else None, start=i32(start), q_weight=wq, k_weight=wk,
                        interleaved=inter)
    assert got["dev_status"].item() == 0
    pos = torch.cat([torch.arange(a, a + b) for a, b in zip(start, w)])
    close(got["q"], *formula(q, pos, freq, wq, 1e-6, inter))
    close(got["k"], *formula(k, pos, freq, wk, 1e-6, inter))


@pytest.mark.parametrize("weights", [(True, False), (False, True)])
def test_one_of_the_two_normalised(gpu_lib, weights):
    gen = torch.Generator().manual_seed(3)
    q, k = rows_of(5, 3, 128, gen), rows_of(5, 1, 128, gen)
    wt = [(1 + torch.rand((128,), generator=gen)).cuda() if x else None for x in weights]
    got = sdm.qk_rotate(q, k, i32([0, 5]), i32([9]), freqs(128).cuda(), q_weight=wt[0], k_weight=wt[1], eps=0.1)
    pos = torch.arange(9, 14)
    close(got["q"], *formula(q, pos, freqs(128), wt[0], 0.1, False))
    close(got["k"], *formula(k, pos, freqs(128), wt[1], 0.1, False))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D,page,G,inter,w,ctx", [(128, 16, 2, False, [1], [500]), (64, 32, 3, True, [5, 0, 17], [3, 40, 31]),
                                                  (128, 64, 1, False, [300, 2], [0, 63]), (128, 128, 5, True, [9] * 40, [100] * 40)])
def test_into_the_cache_like_rotating_and_writing(gpu_lib, e4m3, D, page, G, inter, w, ctx):
    """The same bits in the cache, and only there where rows were written."""
    H, gen = 2 * G, torch.Generator().manual_seed(G)
    a, b = (ref.Setup(w, ctx, G, D, page, e4m3, seed=1, fill=0.0) for _ in range(2))
    q, k, v = rows_of(a.rows, H, D, gen, 16), rows_of(a.rows, G, D, gen, 16), rows_of(a.rows, G, D, gen, 24)
    wk = (1 + torch.rand((D,), generator=gen)).cuda()
    freq, start = freqs(D).cuda(), a.ctx + 1000
    kw = dict(start=start, k_weight=wk, interleaved=inter)
    one = sdm.qk_rotate(q, k, a.cu, a.ctx, freq, v=v, cache=a.cache, dev_status=a.status, **kw)
    two = sdm.qk_rotate(q, k, a.cu, a.ctx, freq, dev_status=b.status, **kw)
    sdm.cache_write(b.cache, two["k"], v, b.cu, b.ctx, dev_status=b.status)
    assert torch.equal(one["q"], two["q"])
    for n in ("k", "v", "k_exp", "v_exp"):
        x, y = getattr(a.cache, n), getattr(b.cache, n)
        if x is not None:
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), n
    assert a.status.item() == 0 and b.status.item() == 0


def test_a_trees_depths_as_positions(gpu_lib):
    gen = torch.Generator().manual_seed(5)
    q, k = rows_of(6, 4, 64, gen), rows_of(6, 4, 64, gen)
    depth = [0, 1, 1, 2, 0, 3]
    got = sdm.qk_rotate(q, k, i32([0, 4, 6]), i32([10, 20]), freqs(64).cuda(), row_pos=i32(depth))
    pos = torch.tensor([10, 11, 11, 12, 20, 23])
    close(got["q"], *formula(q, pos, freqs(64), None, 0, False))
    close(got["k"], *formula(k, pos, freqs(64), None, 0, False))


@pytest.mark.parametrize("rows", [3, 3000])
def test_in_place_and_rows_that_no_window_holds(gpu_lib, rows):
    gen = torch.Generator().manual_seed(6)
    qkv = torch.randn((rows, 12, 128), generator=gen).to(torch.bfloat16).cuda()
    before = qkv.clone()
    q, k = qkv[:, :8], qkv[:, 8:10]
    cu = i32([0, 1, rows - 1])
    sdm.qk_rotate(q, k, cu, i32([5, 6]), freqs(128).cuda(), out=dict(q=q, k=k), dev_status=sdm.new_status())
    apart = sdm.qk_rotate(before[:, :8], before[:, 8:10], cu, i32([5, 6]), freqs(128).cuda())
    assert torch.equal(q[:rows - 1], apart["q"][:rows - 1]) and torch.equal(k[:rows - 1], apart["k"][:rows - 1])
    assert torch.equal(qkv[rows - 1], before[rows - 1]) and torch.equal(qkv[:, 10:], before[:, 10:])


def test_unsound_windows_and_pages(gpu_lib):
    """A window that is not monotone counts as empty, the others are done; a
    token whose page is bad is not written, its query is rotated."""
    gen = torch.Generator().manual_seed(7)
    q, k, v = (rows_of(9, 2, 64, gen) for _ in range(3))
    s = ref.Setup([3, 3, 3], [0, 14, 5], 2, 64, 16, False, fill=0.0)
    s.cache.table[1, 1] = 1000                                     # tokens 16 on of the second request
    out = dict(q=torch.zeros_like(q))
    sdm.qk_rotate(q, k, s.cu, s.ctx, freqs(64).cuda(), v=v, cache=s.cache, out=out, dev_status=s.status)
    assert s.status.item() == sdm.DEV_BAD_PAGE
    pos = torch.tensor([0, 1, 2, 14, 15, 16, 5, 6, 7])
    close(out["q"], *formula(q, pos, freqs(64), None, 0, False))
    st = sdm.new_status()
    out = dict(q=torch.zeros_like(q), k=torch.zeros_like(k))
    sdm.qk_rotate(q, k, i32([0, 3, 1, 9]), i32([0, 14, 5]), freqs(64).cuda(), out=out, dev_status=st)
    assert st.item() == sdm.DEV_BAD_WINDOW
    want, size = formula(q[1:], torch.arange(5, 13), freqs(64), None, 0, False)
    close(out["q"][3:], want[2:], size[2:])


def test_infinities_and_nan_stay_in_their_head(gpu_lib):
    gen = torch.Generator().manual_seed(8)
    q, k = rows_of(4, 3, 128, gen), rows_of(4, 1, 128, gen)
    q[1, 1, 5], q[2, 0, 100] = float("nan"), float("inf")
    w = torch.ones(128, device="cuda")
    got = sdm.qk_rotate(q, k, i32([0, 4]), i32([3]), freqs(128).cuda(), q_weight=w)["q"]
    odd = ~torch.isfinite(got.float()).all(-1)
    assert odd.nonzero().tolist() == [[1, 1], [2, 0]]


def test_a_captured_call_follows_its_inputs(gpu_lib):
    gen = torch.Generator().manual_seed(9)
    s = ref.Setup([4, 4], [16, 16], 2, 128, 16, True, fill=0.0)
    q, k, v = (rows_of(8, h, 128, gen) for h in (4, 2, 2))
    freq, out = freqs(128).cuda(), dict(q=torch.zeros((8, 4, 128), dtype=torch.bfloat16, device="cuda"))
    call = lambda: sdm.qk_rotate(q, k, s.cu, s.ctx, freq, v=v, cache=s.cache, out=out, dev_status=s.status)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    q.mul_(-2)
    s.ctx.add_(3)
    graph.replay()
    got = out["q"].clone()
    call()
    assert torch.equal(got, out["q"]) and s.status.item() == 0
    close(got, *formula(q, torch.cat([torch.arange(19, 23)] * 2), freqs(128), None, 0, False))

"""Attention over the paged cache on the GPU against the plain 64-bit form.

Tolerance of out, elementwise: the weights enter the second product as bf16
(relative error at most 2^-9 each, so at most 2^-9 sum_j p_j |v_j|), and the
result is rounded to bf16 (2^-9 |out|, |out| <= sum_j p_j |v_j|); fp32 sums,
scores and exponentials stay below 2^-14 of that sum at these sizes.  So
(2^-8 + 2^-14) sum_j p_j |v_j|, and 2^-133 for results below bf16's range.
lse: fp32 scores of size |s| <= 100 carry at most D 2^-24 |s| from the dot
product (exact bf16 products) and the exponentials 2^-21: 2e-4 + 1e-6 |lse|
at the largest, 3e-5 where scores are of order 10."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from speculative_decoding_markov_gb300 import binding as sdm
from tests import paged_reference as ref

pytestmark = pytest.mark.gpu


def check(s, H, window=0, sinks=0, mask=None, scale=None, q=None, size=1.0, max_window=None, lse_tol=3e-5, rows=None):
    """Runs the kernel on setup s and compares every row; returns its outputs."""
    D = s.D
    scale = D ** -0.5 if scale is None else scale
    rows = s.rows if rows is None else rows
    if q is None:
        q = (torch.randn((rows, H, D), generator=s.gen) * size).to(torch.bfloat16).cuda()
    m = None if mask is None else torch.as_tensor(mask).cuda()
    got = sdm.attend(s.cache, q, s.cu, s.ctx, max_window or max(s.w), scale=scale, window=window, sinks=sinks,
                     tree_mask=m, lse=True, dev_status=s.status)
    out, lse = got["out"].double().cpu().numpy(), got["lse"].double().cpu().numpy()
    at = 0
    for i, (w, c) in enumerate(zip(s.w, s.ctx_list)):
        if w == 0:
            continue
        see = ref.visible(w, c, window, sinks, None if mask is None else np.asarray(mask)[i])
        o, z, big = ref.attend(q[at:at + w], s.held(i, "k"), s.held(i, "v"), see, scale)
        mine, zm = out[at:at + w], lse[at:at + w]
        assert np.array_equal(np.isnan(mine), np.isnan(o)), (i, np.argwhere(np.isnan(mine) != np.isnan(o))[:4])
        fine = np.isfinite(o)
        err = np.abs(mine - o)[fine] - ((2.0 ** -8 + 2.0 ** -14) * big[fine] + 2.0 ** -133)
        assert err.size == 0 or err.max() <= 0, (i, err.max())
        assert np.array_equal(np.isneginf(zm), np.isneginf(z)), i
        fine = np.isfinite(z)
        assert np.all(np.abs(zm - z)[fine] <= lse_tol + 1e-6 * np.abs(z[fine])), np.abs(zm - z)[fine].max()
        at += w
    return got


HEADS = [(32, 8, 128), (28, 4, 128), (4, 4, 64), (16, 2, 64), (5, 5, 128), (12, 1, 64), (48, 1, 128)]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("H,G,D", HEADS)
@pytest.mark.parametrize("page", [16, 128])
def test_verify_windows(gpu_lib, e4m3, H, G, D, page):
    """Ragged windows, contexts around the tiles' and pages' ends, length one."""
    w = [1, 8, 3, 0, 5, 1, 2, 7]
    ctx = [0, 0, 1, 9, 127, 128, 255, 300]
    s = ref.Setup(w, ctx, G, D, page, e4m3, seed=H + page)
    s.write_all()
    check(s, H)
    assert s.status.item() == 0


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("H,G,D", [(32, 8, 128), (7, 1, 128), (8, 4, 64)])
@pytest.mark.parametrize("w,ctx", [([1], [5000]), ([1, 1, 1], [2047, 2048, 12001]), ([9], [3333])])
def test_long_contexts(gpu_lib, e4m3, H, G, D, w, ctx):
    s = ref.Setup(w, ctx, G, D, 32, e4m3, seed=sum(ctx))
    s.write_all()
    check(s, H)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("H,G,D", [(8, 2, 128), (7, 1, 128), (4, 4, 64), (16, 2, 64)])
@pytest.mark.parametrize("w,ctx", [([300], [0]), ([129, 1, 64, 33], [77, 500, 0, 128]), ([513], [257])])
def test_chunks(gpu_lib, e4m3, H, G, D, w, ctx):
    s = ref.Setup(w, ctx, G, D, 64, e4m3, seed=sum(w))
    s.write_all()
    check(s, H)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 0), (64, 4), (127, 1), (128, 0), (129, 130), (200, 300),
                                          (100000, 3)])
@pytest.mark.parametrize("w,ctx", [([1, 8, 1], [700, 511, 0]), ([260, 40], [333, 1000])])
def test_windows_and_sinks(gpu_lib, e4m3, window, sinks, w, ctx):
    s = ref.Setup(w, ctx, 2, 64, 16, e4m3, seed=window + sinks)
    s.write_all()
    check(s, 8, window=window, sinks=sinks)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("H,G,D", [(32, 8, 128), (14, 2, 64)])
@pytest.mark.parametrize("S,depth", [(5, 4), (17, 6), (33, 5), (65, 16), (200, 30)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 2)])
def test_trees(gpu_lib, e4m3, H, G, D, S, depth, window, sinks):
    rng = np.random.default_rng(S)
    t = ref.random_trees(3, S, depth, rng)
    s = ref.Setup([S, max(1, S - 3), S], [0, 100, 333], G, D, 32, e4m3, seed=S)
    s.write_all()
    check(s, H, mask=t["mask"], window=window, sinks=sinks, max_window=S)


def test_tree_rows_that_see_nothing(gpu_lib):
    """Rows without any bit: with a context they see it, without one nothing."""
    t = ref.random_trees(2, 40, 8, np.random.default_rng(1))
    t["mask"][:, [0, 7, 39]] = 0
    s = ref.Setup([40, 40], [0, 60], 2, 128, 16, False)
    s.write_all()
    got = check(s, 8, mask=t["mask"])
    for r in (0, 7, 39):
        assert not got["out"][r].any() and torch.isneginf(got["lse"][r]).all()
    assert torch.isfinite(got["lse"][40:]).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("w,ctx", [([6], [140]), ([6, 1], [3, 1]), ([200], [100])])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("which", ["k", "v"])
def test_unseen_tokens_do_not_touch_a_row(gpu_lib, e4m3, w, ctx, bad, which):
    """A NaN or infinity in a token reaches the rows that see it and no other:
    the rows before it, and those whose window has passed it."""
    s = ref.Setup(w, ctx, 2, 128, 16, e4m3, seed=3)
    for at in (ctx[0] + 3, ctx[0] // 2):
        s.kv[0][which][at, 1, 5] = bad
        if e4m3 or which == "v":
            s.kv[0][which][at, 0, 17] = -bad
    s.write_all()
    with np.errstate(invalid="ignore"):
        if which == "k" and bad == float("inf") and not e4m3:
            return     # scores of either sign: covered by the NaN case
        if which == "v" and bad == float("inf") and not e4m3:
            check_inf(s, 8)
        else:
            check(s, 8, window=20, sinks=1)


def check_inf(s, H):
    """Infinite values: a row that sees one gives that infinity there."""
    q = torch.randn((s.rows, H, s.D), generator=s.gen).to(torch.bfloat16).cuda()
    got = sdm.attend(s.cache, q, s.cu, s.ctx, max(s.w), lse=True, dev_status=s.status)["out"].double().cpu().numpy()
    at = 0
    for i, (w, c) in enumerate(zip(s.w, s.ctx_list)):
        o, _, big = ref.attend(q[at:at + w], s.held(i, "k"), s.held(i, "v"), ref.visible(w, c), s.D ** -0.5)
        mine = got[at:at + w]
        assert np.array_equal(np.isposinf(mine), np.isposinf(o)) and np.array_equal(np.isneginf(mine), np.isneginf(o))
        fine = np.isfinite(o)
        assert np.all(np.abs(mine - o)[fine] <= (2.0 ** -8 + 2.0 ** -14) * big[fine])
        at += w


def test_sizes_of_scores(gpu_lib):
    """Peaked softmax (large scores of both signs) and a nearly flat one."""
    s = ref.Setup([5, 130], [400, 64], 2, 128, 64, False)
    s.write_all()
    check(s, 8, size=8.0, lse_tol=2e-4)
    check(s, 8, size=1e-3)
    check(s, 8, scale=1.0, lse_tol=2e-4)


def test_rising_and_falling_scores(gpu_lib):
    """Keys ordered so that the running maximum grows with every tile (each
    needs the sums rescaled), and the reverse."""
    for sign in (1.0, -1.0):
        s = ref.Setup([2, 140], [1500, 900], 1, 64, 32, False)
        for kv in s.kv:
            n = kv["k"].shape[0]
            ramp = torch.linspace(-4, 4, n) * sign
            kv["k"][:] = (kv["k"] * 0.25 + ramp[:, None, None]).to(torch.bfloat16)
        s.write_all()
        q = (torch.rand((s.rows, 4, 64), generator=s.gen) + 0.5).to(torch.bfloat16).cuda()
        check(s, 4, q=q, scale=1.0, lse_tol=2e-3)


def test_query_slices_padding_rows_and_streams(gpu_lib):
    """q as a slice of a wider projection, rows past the last window left
    alone, work on a side stream, and the same bits on every run."""
    s = ref.Setup([3, 1, 4], [100, 0, 513], 2, 128, 16, True)
    s.write_all()
    rows, H = s.rows + 9, 14
    wide = torch.randn((rows, H + 4, 128)).to(torch.bfloat16).cuda()
    check(s, H, q=wide[:, :H], rows=rows)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    outs = []
    with torch.cuda.stream(st):
        for _ in range(2):
            out = dict(out=torch.full((rows, H, 128), 3.0, dtype=torch.bfloat16, device="cuda"),
                       lse=torch.full((rows, H), 3.0, device="cuda"))
            outs.append(sdm.attend(s.cache, wide[:, :H], s.cu, s.ctx, 4, lse=True, out=out, dev_status=s.status))
    st.synchronize()
    assert torch.equal(outs[0]["out"], outs[1]["out"]) and torch.equal(outs[0]["lse"], outs[1]["lse"])
    assert (outs[0]["out"][s.rows:] == 3.0).all() and (outs[0]["lse"][s.rows:] == 3.0).all()


def test_many_requests(gpu_lib):
    """More requests than threads in a block, most of them short, some empty."""
    rng = np.random.default_rng(0)
    w = [int(x) for x in rng.integers(0, 4, 700)]
    ctx = [int(x) for x in rng.integers(0, 40, 700)]
    s = ref.Setup(w, ctx, 1, 64, 16, False)
    s.write_all()
    check(s, 4, max_window=3)


def test_in_a_graph(gpu_lib):
    """Captured once, replayed on new lengths and values."""
    s = ref.Setup([2, 6], [300, 20], 2, 128, 32, False)
    s.write_all()
    q = torch.randn((s.rows, 8, 128), generator=s.gen).to(torch.bfloat16).cuda()
    out = dict(out=torch.zeros_like(q), lse=torch.zeros((s.rows, 8), device="cuda"))
    ws = sdm.attend_workspace(s.cache, s.rows, 6, 8)
    sdm.attend(s.cache, q, s.cu, s.ctx, 6, lse=True, out=out, ws=ws, dev_status=s.status)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sdm.attend(s.cache, q, s.cu, s.ctx, 6, lse=True, out=out, ws=ws, dev_status=s.status)
    s.ctx.copy_(torch.tensor([123, 5], dtype=torch.int32))
    g.replay()
    want = sdm.attend(s.cache, q, s.cu, s.ctx, 6, lse=True, dev_status=s.status)
    assert torch.equal(out["out"], want["out"]) and torch.equal(out["lse"], want["lse"])


def test_pool_past_32_bits(gpu_lib):
    page, G, D = 128, 4, 128
    n = 2 ** 32 // (page * G * D) + 8
    k, v = (torch.empty((n, G, page, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    s = ref.Setup([3], [200], G, D, page, False)
    table = torch.tensor([[n - 1, n - 3]], dtype=torch.int32).cuda()
    s.cache = sdm.PagedCache(k, v, table)
    s.write_all()
    check(s, 8)


def test_device_checks(gpu_lib):
    """Bad lengths and pages are flagged, cut, and read nothing out of range."""
    s = ref.Setup([3, 4], [50, 20], 2, 64, 16, False, fill=0.0)
    s.write_all()
    q = torch.randn((s.rows, 4, 64)).to(torch.bfloat16).cuda()

    def run(cu=None, ctx=None, max_window=4):
        s.status.zero_()
        sdm.attend(s.cache, q, s.cu if cu is None else torch.tensor(cu, dtype=torch.int32).cuda(),
                   s.ctx if ctx is None else torch.tensor(ctx, dtype=torch.int32).cuda(), max_window,
                   dev_status=s.status)
        return s.status.item()

    assert run() == 0
    assert run(max_window=3) == sdm.DEV_BAD_WINDOW
    assert run(cu=[0, 5, 3]) & sdm.DEV_BAD_WINDOW
    assert run(cu=[-2, 3, 7]) & sdm.DEV_BAD_WINDOW
    assert run(cu=[0, 3, 99]) & sdm.DEV_BAD_WINDOW
    assert run(ctx=[-1, 20]) & sdm.DEV_BAD_WINDOW
    assert run(ctx=[2 ** 31 - 1, 20]) & sdm.DEV_BAD_PAGE
    s.cache.table[1, 0] = -7
    assert run() == sdm.DEV_BAD_PAGE


def test_outputs_on_a_16_byte_boundary(gpu_lib):
    """out 16 but not 32 bytes aligned: the narrower stores, the same bits."""
    s = ref.Setup([3, 130], [70, 0], 2, 64, 16, False)
    s.write_all()
    q = torch.randn((s.rows, 8, 64), generator=s.gen).to(torch.bfloat16).cuda()
    want = sdm.attend(s.cache, q, s.cu, s.ctx, 130, dev_status=s.status)["out"]
    room = torch.zeros(q.numel() + 8, dtype=torch.bfloat16, device="cuda")
    out = room[8:].view(q.shape)
    assert out.data_ptr() % 32 == 16
    sdm.attend(s.cache, q, s.cu, s.ctx, 130, out=dict(out=out), dev_status=s.status)
    assert torch.equal(out, want) and not room[:8].any()


@pytest.mark.parametrize("e4m3", [False, True])
def test_many_long_windows(gpu_lib, e4m3):
    """More requests than a warp plans, windows of several blocks, the most
    query heads per kv head, empty requests between."""
    rng = np.random.default_rng(2)
    w = [int(x) for x in rng.integers(0, 30, 40)]
    ctx = [int(x) for x in rng.integers(0, 300, 40)]
    s = ref.Setup(w, ctx, 1, 64, 32, e4m3, seed=9)
    s.write_all()
    check(s, 128, max_window=29)
    check(s, 33, max_window=29)
    s = ref.Setup([40, 0, 700, 3], [500, 3, 0, 90], 2, 128, 64, e4m3, seed=10)
    s.write_all()
    check(s, 14)


def test_splits_of_every_length(gpu_lib):
    """One request at lengths that cut its tiles between CTAs in every way."""
    for n in (1, 2, 127, 129, 255, 385, 1000, 2600, 4999):
        for w in (1, 20, 70):
            s = ref.Setup([w], [max(0, n - w)], 2, 64, 64, n % 2 == 0, seed=n + w)
            s.write_all()
            check(s, 8)

"""Attention over the paged cache where it went wrong, or could have: one
group of tests for each such case, against plain 64-bit forms."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from speculative_decoding_markov_gb300 import binding as sdm
from tests import paged_reference as ref
from tests.test_gpu_attend import check

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# A tile has 128 rows; those that its block does not fill take no part in
# anything the others do, whatever an earlier call left in their place.
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("w,before,G", [(5, 8, 1), (200, 200, 2)])
def test_the_same_bits_whatever_ran_before(gpu_lib, e4m3, w, before, G):
    """7 heads a kv head after a call with 8, whose queries fill the rows that
    7 leave free: once with zeros, once with queries whose scores rise by more
    from tile to tile than the running maximum follows without moving."""
    R, n = 40 if w < 10 else 6, 3000
    s = ref.Setup([w] * R, [n - w] * R, G, 128, 16, e4m3, seed=w)
    for kv in s.kv:
        kv["k"][:, :, 0] = (torch.arange(n) // 128).to(torch.bfloat16)[:, None]
    s.write_all()
    q = torch.randn((s.rows, 7 * G, 128), generator=s.gen).to(torch.bfloat16)
    q[:, :, 0] = 0
    q = q.cuda()
    got = []
    for size in (0.0, 200.0):
        first = torch.zeros((R * before, 8 * G, 128), dtype=torch.bfloat16, device="cuda")
        first[:, :, 0] = size
        cu = torch.arange(R + 1, dtype=torch.int32, device="cuda") * before
        sdm.attend(s.cache, first, cu, i32([n - before] * R), before, dev_status=s.status)
        got.append(sdm.attend(s.cache, q, s.cu, s.ctx, w, lse=True, dev_status=s.status))
    assert torch.equal(got[0]["lse"], got[1]["lse"]) and torch.equal(got[0]["out"], got[1]["out"])
    assert s.status.item() == 0


@pytest.mark.parametrize("sinks", [2 ** 31 - 1, 2 ** 31 - 128, 2 ** 31 - 129, 10 ** 6])
@pytest.mark.parametrize("e4m3,w,ctx,tree", [(False, [3, 1], [700, 2500], False), (True, [3, 1], [700, 2500], False),
                                             (False, [150, 20], [333, 900], False), (False, [33], [600], True)])
def test_all_tokens_as_sinks(gpu_lib, sinks, e4m3, w, ctx, tree):
    """The largest numbers of first tokens that stay visible: every one does."""
    mask = ref.random_trees(1, w[0], 6, np.random.default_rng(4))["mask"] if tree else None
    s = ref.Setup(w, ctx, 2, 64, 32, e4m3, seed=7)
    s.write_all()
    check(s, 8, window=20, sinks=sinks, mask=mask)
    assert s.status.item() == 0


@pytest.mark.parametrize("e4m3", [False, True])
def test_the_last_positions_of_32_bits(gpu_lib, e4m3):
    """A page table of 2^31 tokens over four pages in turn: windows that end at
    the last position in use, 2^31 - 257, and one that runs past it."""
    page, G, H, D, w, last = 128, 2, 8, 64, 5, 2 ** 31 - 256
    s = ref.Setup([4 * page], [0], G, D, page, e4m3, seed=11, spare=0)
    s.write_all()
    order = s.cache.table[0, :4]
    table = order.repeat(2 ** 31 // page // 4)[None].contiguous()
    cache = sdm.PagedCache(s.cache.k, s.cache.v, table, s.cache.k_exp, s.cache.v_exp)
    q = torch.randn((w, H, D), generator=s.gen).to(torch.bfloat16).cuda()
    k, v = s.held(0, "k"), s.held(0, "v")
    for ctx, rows, status in ((last - w, w, 0), (last - 3, 3, sdm.DEV_BAD_PAGE)):
        for window in (1, 64, 300):
            flag = sdm.new_status()
            got = sdm.attend(cache, q, i32([0, w]), i32([ctx]), w, window=window, dev_status=flag)["out"]
            at = torch.arange(ctx - 300, last) % (4 * page)                    # the tokens' places in the four pages
            see = ref.visible(rows, 300, window)
            o, _, big = ref.attend(q[:rows], k[at], v[at], see, D ** -0.5)
            err = np.abs(got[:rows].double().cpu().numpy() - o)
            assert (err <= (2.0 ** -7 + 2.0 ** -12) * big).all(), err.max()
            assert flag.item() == status
    flag = sdm.cache_write(cache, s.packed("k")[:w], s.packed("v")[:w], i32([0, w]), i32([last - 3]))
    assert flag.item() == sdm.DEV_BAD_PAGE


# The scales of an e4m3 cache: every reader takes a byte for the same factor.
BYTES = [0, 1, 2, 16, 17, 126, 127, 200, 246, 247, 253, 254, 255]


def test_every_exponent_byte_reads_alike(gpu_lib):
    """A row that sees its own token alone gives that token's values, as
    cache_read has them: infinities where code and scale leave bf16's range,
    NaN codes, and zeros under any scale."""
    n, D = len(BYTES), 64
    s = ref.Setup([1] * n, [0] * n, 1, D, 16, True, seed=1, fill=0.0)
    codes = torch.arange(256, dtype=torch.uint8)[torch.randperm(256, generator=s.gen)][:D]
    codes[:6] = torch.tensor([0, 0x80, 0x7f, 0x7e, 0x38, 0xb8])             # zeros, NaN, 448, 1, -1
    for i, byte in enumerate(BYTES):
        page = s.table_cpu[i, 0].item()
        s.cache.v.view(torch.uint8)[page, 0, 0] = codes.cuda()
        s.cache.v_exp[page, 0, 0] = byte
        s.cache.k.view(torch.uint8)[page, 0, 0] = 0                          # scores of zero: NaN if a scale is infinite
        s.cache.k_exp[page, 0, 0] = byte
    held = sdm.cache_read(s.cache, s.cu, n, dev_status=s.status)["v"].double().cpu().numpy()[:, 0]
    value = codes.view(torch.float8_e4m3fn).double().numpy()
    for i, byte in enumerate(BYTES):                                         # cache_read: the definition
        want = torch.from_numpy(value * 2.0 ** (min(max(byte, 1), 254) - 127)).to(torch.bfloat16).double().numpy()
        assert np.array_equal(held[i], want, equal_nan=True), byte
    q = torch.randn((n, 4, D), generator=s.gen).to(torch.bfloat16).cuda()
    got = sdm.attend(s.cache, q, s.cu, s.ctx, 1, lse=True, dev_status=s.status)
    out = got["out"].double().cpu().numpy()
    assert (got["lse"] == 0).all()
    for i, byte in enumerate(BYTES):
        for h in range(4):
            assert np.array_equal(np.isnan(out[i, h]), np.isnan(held[i])), byte
            assert np.array_equal(np.isinf(out[i, h]), np.isinf(held[i])), byte
            fine = np.isfinite(held[i])
            # products of subnormal numbers may count as zero
            assert (np.abs(out[i, h] - held[i])[fine] <= 2.0 ** -126).all(), byte
            assert np.array_equal(np.sign(out[i, h])[np.isinf(held[i])], np.sign(held[i])[np.isinf(held[i])])
    assert s.status.item() == 0


def by_scores(q, k, v, see, scale):
    """ref.attend by the definition where keys hold infinities: lse is NaN if a
    score is, else +inf if one is; out is NaN in both cases; a row with scores
    of -inf alone is one that sees nothing."""
    out, lse, size = ref.attend(q, k, v, see, scale)
    rep = q.shape[1] // k.shape[1]
    q, k = q.double().cpu().numpy(), k.double().numpy()
    for p in range(q.shape[0]):
        at = np.nonzero(see[p])[0]
        for h in range(q.shape[1]):
            with np.errstate(invalid="ignore"):
                s = scale * (k[at, h // rep] @ q[p, h]) if at.size else np.array([-np.inf])
            if np.isnan(s).any() or np.isposinf(s).any():
                out[p, h], lse[p, h] = np.nan, np.nan if np.isnan(s).any() else np.inf
            elif np.isneginf(s).all():
                out[p, h], lse[p, h] = 0.0, -np.inf
    return out, lse, size


@pytest.mark.parametrize("w,ctx", [([6], [140]), ([6, 1], [3, 1]), ([200], [100]), ([5], [6000]), ([300], [2000])])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 1)])
def test_infinite_keys(gpu_lib, w, ctx, window, sinks):
    """Scores of +inf, -inf and (two of either sign together) NaN, for the rows
    that see them and no other."""
    s = ref.Setup(w, ctx, 2, 128, 16, False, seed=3)
    k = s.kv[0]["k"]
    k[ctx[0] + 3, 1, 5] = float("inf")
    k[ctx[0] // 2, 0, 17] = -float("inf")
    k[ctx[0] + 2, 0, 17] = k[ctx[0] + 2, 0, 18] = float("inf")
    s.write_all()
    q = torch.randn((s.rows, 8, 128), generator=s.gen).to(torch.bfloat16).cuda()
    got = sdm.attend(s.cache, q, s.cu, s.ctx, max(w), window=window, sinks=sinks, lse=True, dev_status=s.status)
    out, lse = got["out"].double().cpu().numpy(), got["lse"].double().cpu().numpy()
    at, kinds = 0, set()
    for i, (a, c) in enumerate(zip(w, ctx)):
        with np.errstate(invalid="ignore"):
            o, z, big = by_scores(q[at:at + a], s.held(i, "k"), s.held(i, "v"), ref.visible(a, c, window, sinks),
                                  128 ** -0.5)
        mine, zm = out[at:at + a], lse[at:at + a]
        at += a
        assert np.array_equal(np.isnan(mine), np.isnan(o)) and np.array_equal(np.isnan(zm), np.isnan(z))
        assert np.array_equal(np.isposinf(zm), np.isposinf(z)) and np.array_equal(np.isneginf(zm), np.isneginf(z))
        fine = np.isfinite(o)
        assert (np.abs(mine - o)[fine] <= (2.0 ** -7 + 2.0 ** -12) * big[fine]).all()
        fine = np.isfinite(z)
        assert (np.abs(zm - z)[fine] <= 3e-5).all()
        kinds |= {"nan"} if np.isnan(z).any() else set()
        kinds |= {"inf"} if np.isposinf(z).any() else set()
        kinds |= {"fine"} if fine.any() else set()
    assert kinds == {"nan", "inf", "fine"} and s.status.item() == 0


def test_rows_of_scores_of_minus_infinity(gpu_lib):
    s = ref.Setup([2, 1], [3, 400], 1, 64, 16, False, seed=5)
    for kv in s.kv:
        kv["k"][:, 0, 7] = -float("inf")
    s.write_all()
    q = torch.rand((3, 4, 64), generator=s.gen).add(0.5).to(torch.bfloat16).cuda()
    got = sdm.attend(s.cache, q, s.cu, s.ctx, 2, lse=True, dev_status=s.status)
    assert not got["out"].any() and torch.isneginf(got["lse"]).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("w,ctx", [([5, 3], [384, 300]), ([40], [513])])
def test_bits_past_the_window(gpu_lib, e4m3, w, ctx):
    """Mask rows with more bits than the window has tokens: they count as
    depth, and so move the sliding window, and show no token."""
    t = ref.random_trees(len(w), 70, 9, np.random.default_rng(3))["mask"]
    t[:, 1::2, 1:] = -1
    t[:, 2::3] = -1
    s = ref.Setup(w, ctx, 2, 64, 32, e4m3, seed=12)
    s.write_all()
    for window, sinks in ((140, 0), (140, 3), (70, 0), (300, 200)):
        check(s, 8, mask=t, window=window, sinks=sinks, max_window=max(w))


def test_the_largest_scale(gpu_lib):
    """Scores of zero stay zero."""
    s = ref.Setup([2], [200], 2, 64, 16, False, seed=4)
    s.write_all()
    check(s, 8, scale=1.99e38, q=torch.zeros((2, 8, 64), dtype=torch.bfloat16, device="cuda"))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("w,ctx,tree", [(1100, 0, False), (130, 300, False), (65, 500, True)])
def test_values_that_are_all_infinite_or_nan(gpu_lib, e4m3, w, ctx, tree):
    """They come out as they are, and in a time that is no threat to the waits
    of the rows beside them (2 s): 1100 tokens, 32 heads, took 115 ms."""
    mask = ref.random_trees(1, w, 8, np.random.default_rng(5))["mask"] if tree else None
    s = ref.Setup([w], [ctx], 8, 128, 64, e4m3, seed=13)
    for kv in s.kv:
        kv["v"][:] = float("inf")
        kv["v"][:, :, 1::2] = float("nan")
    s.write_all()
    q = torch.randn((w, 32, 128), generator=s.gen).to(torch.bfloat16).cuda()
    m = None if mask is None else torch.as_tensor(mask).cuda()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for _ in range(2):
        start.record()
        out = sdm.attend(s.cache, q, s.cu, s.ctx, w, tree_mask=m, dev_status=s.status)["out"]
        end.record()
    torch.cuda.synchronize()
    assert torch.isnan(out[:, :, 1::2]).all() and s.status.item() == 0
    assert (torch.isnan(out) if e4m3 else torch.isposinf(out))[:, :, ::2].all()
    print(f"{start.elapsed_time(end):.2f} ms")
    assert start.elapsed_time(end) < 40.0

"""The paged cache's write, read and commit where they went wrong, or could
have, against the plain forms."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from speculative_decoding_markov_gb300 import binding as sdm
from tests import paged_reference as ref

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("e4m3", [False, True])
def test_batches_without_rows(gpu_lib, e4m3):
    """A cycle in which no request has a row changes nothing and is no error."""
    s = ref.Setup([0, 0], [5, 20], 2, 64, 16, e4m3, fill=1.0)
    before = s.cache.k.clone()
    kv = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    assert kv.data_ptr() == 0
    sdm.cache_write(s.cache, kv, kv, s.cu, s.ctx, dev_status=s.status)
    got = sdm.cache_read(s.cache, s.cu, 0, dev_status=s.status)
    assert got["k"].shape == got["v"].shape == (0, 2, 64)
    q = torch.empty((0, 8, 64), dtype=torch.bfloat16, device="cuda")
    for longest in (0, 3):
        got = sdm.attend(s.cache, q, s.cu, s.ctx, longest, lse=True, dev_status=s.status)
        assert got["out"].shape == (0, 8, 64) and got["lse"].shape == (0, 8)
    assert s.status.item() == 0 and torch.equal(before.view(torch.uint8), s.cache.k.view(torch.uint8))


def test_a_single_row_of_an_odd_projection(gpu_lib):
    """One token's query, key and value as slices of a row of an odd width."""
    s = ref.Setup([1], [40], 2, 64, 16, False, seed=2)
    s.write_all()
    wide = torch.zeros((1, 8 * 64 + 2 * 128 + 1), dtype=torch.bfloat16, device="cuda")
    q, k, v = (wide.as_strided((1, n, 64), (769, 64, 1), at) for n, at in ((8, 0), (2, 512), (2, 640)))
    q.copy_(torch.randn((1, 8, 64), generator=s.gen))
    k.copy_(s.packed("k"))
    v.copy_(s.packed("v"))
    assert q.stride(0) % 8
    sdm.cache_write(s.cache, k, v, s.cu, s.ctx, dev_status=s.status)
    got = sdm.attend(s.cache, q, s.cu, s.ctx, 1, dev_status=s.status)["out"]
    want = sdm.attend(s.cache, q.contiguous(), s.cu, s.ctx, 1, dev_status=s.status)["out"]
    assert torch.equal(got, want) and s.status.item() == 0


# Offsets that are not sound: what is wrong is flagged, whether or not a row
# leads to it, and windows that are valid by themselves are done all the same.
def slots(s, name, i, first, n):
    """Tokens first .. first + n - 1 of request i as the pool holds them [n, G, D]."""
    page = s.page
    pool = s.cache.k if name == "k" else s.cache.v
    return torch.stack([pool[s.table_cpu[i, t // page].item(), :, t % page] for t in range(first, first + n)])


@pytest.mark.parametrize("cu,valid", [([0, 5, 3], {0: (0, 5)}), ([0, 3, -1], {0: (0, 3)}), ([0, -1, 4], {}),
                                      ([2, 2, 7], {1: (2, 5)}), ([0, 5, 3, 7], {0: (0, 5), 2: (3, 4)}),
                                      ([0, 9, 4, 7], {2: (4, 3)}), ([0, 2 ** 31 - 1, 7], {}), ([-1, 2, 4], {1: (2, 2)})])
@pytest.mark.parametrize("G", [2, 40])
def test_windows_that_are_not_sound(gpu_lib, cu, valid, G):
    R, rows = len(cu) - 1, 7
    sound = all(0 <= a <= b <= rows for a, b in zip(cu, cu[1:]))
    s = ref.Setup([7] * R, [10 + i for i in range(R)], G, 64, 16, False, seed=R, fill=7.0)
    x = torch.randn((rows, G, 64), generator=s.gen).to(torch.bfloat16).cuda()
    want = [p.clone() for p in (s.cache.k, s.cache.v)]
    for i, (at, n) in valid.items():
        for t in range(n):
            pos = s.ctx_list[i] + t
            page, slot = s.table_cpu[i, pos // 16].item(), pos % 16
            want[0][page, :, slot], want[1][page, :, slot] = x[at + t], -x[at + t]
    flag = sdm.cache_write(s.cache, x, -x, i32(cu), s.ctx)
    assert torch.equal(s.cache.k, want[0]) and torch.equal(s.cache.v, want[1])
    assert flag.item() == (0 if sound else sdm.DEV_BAD_WINDOW)
    out = {n: torch.full((rows, G, 64), 3.0, dtype=torch.bfloat16, device="cuda") for n in "kv"}
    back = sdm.new_status()
    sdm.cache_read(s.cache, i32(cu), rows, first=s.ctx, out=out, dev_status=back)
    want = torch.full_like(x, 3.0)
    for at, n in valid.values():
        want[at:at + n] = x[at:at + n]
    assert torch.equal(out["k"], want) and back.item() == flag.item()


def test_windows_are_checked_without_rows_in_use(gpu_lib):
    """A negative length of an empty window, one past the table's end, and
    offsets that end below zero."""
    s = ref.Setup([0, 3], [5, 20], 2, 64, 16, False, fill=0.0)
    end = s.cache.table.shape[1] * 16
    k = s.packed("k")
    for cu, ctx, status in (([0, 0, 3], [-4, 20], sdm.DEV_BAD_WINDOW), ([0, 0, 3], [end + 1, 20], sdm.DEV_BAD_PAGE),
                            ([0, 0, 3], [end, 20], 0), ([0, -5, -5], [5, 20], sdm.DEV_BAD_WINDOW),
                            ([0, 0, 3], [0, 20], 0), ([0, 0, 0], [0, 20], 0)):
        assert sdm.cache_write(s.cache, k, k, i32(cu), i32(ctx)).item() == status, (cu, ctx)
    for cu, first, status in (([0, 0, 3], [-4, 20], sdm.DEV_BAD_WINDOW), ([0, -5, -5], [5, 20], sdm.DEV_BAD_WINDOW),
                              ([0, 0, 3], [4, 20], 0)):
        flag = sdm.new_status()
        sdm.cache_read(s.cache, i32(cu), 3, first=i32(first), dev_status=flag)
        assert flag.item() == status, (cu, first)


def test_the_checks_over_many_requests(gpu_lib):
    """The last of more windows than a block has threads is the wrong one."""
    R = 1500
    w = [i % 2 for i in range(R)]
    s = ref.Setup(w, [3] * R, 1, 64, 16, False, seed=6)
    s.write_all()
    assert s.status.item() == 0
    cu = s.cu.clone()
    cu[R] = s.rows + 1                                     # past the packed rows: its row is not written
    before = s.cache.k.clone()
    flag = sdm.cache_write(s.cache, -s.packed("k"), s.packed("v"), cu, s.ctx)
    assert flag.item() == sdm.DEV_BAD_WINDOW
    got, want = s.cache.k, before.clone()
    for i in range(1, R - 1, 2):
        want[s.table_cpu[i, 0].item(), :, 3] *= -1
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))    # bits: what no token holds is NaN


@pytest.mark.parametrize("S,B", [(6140, 7), (6139, 9), (6140, 6), (6000, 287), (6140, 8), (16384, 16384), (3, 2)])
def test_commits_of_large_trees(gpu_lib, S, B):
    """Sizes around what fits 48 KB of shared memory (the tree's two arrays and
    the path, beside the kernel's own few bytes), and the largest."""
    depth = 40
    t = ref.random_trees(1, 65, depth, np.random.default_rng(8), vocab=S + 70)
    if S > 65:                                                       # the rest of the slots: children of the root
        parent, tok = np.zeros((1, S), np.int32), np.arange(100000, 100000 + S, dtype=np.int32)[None]
        parent[:, :65], tok[:, :65] = t["parent"], t["tok"]
    else:
        parent, tok = t["parent"][:, :S].copy(), t["tok"][:, :S].copy()
    path, end = [], min(64, S - 1)
    while end > 0:
        path.insert(0, end)
        end = int(parent[0, end])
    path = path[:B]
    s = ref.Setup([65], [20], 1, 64, 16, False, seed=9)
    s.write_all()
    out_tok = np.full((1, B + 1), -1, np.int32)
    out_tok[0, :len(path)] = tok[0, path]
    got = sdm.cache_commit(s.cache, torch.as_tensor(tok).cuda(), torch.as_tensor(parent.copy()).cuda(), i32([S]),
                           torch.as_tensor(out_tok).cuda(), i32([len(path)]), s.ctx, dev_status=s.status)
    assert got["path"][0].tolist() == [0] + path + [-1] * (B - len(path))
    assert got["length"].tolist() == [21 + len(path)] and s.status.item() == 0
    assert torch.equal(slots(s, "k", 0, 20, 1 + len(path)).cpu(), s.kv[0]["k"][[20] + [20 + c for c in path]])

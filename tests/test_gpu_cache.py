"""The paged cache on the GPU: writes in bf16 and e4m3, reads, commits, and
what they refuse, against the plain 64-bit forms.  Everything here is exact:
the codes are a rounding that the definition fixes, the rest moves bytes."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from speculative_decoding_markov_gb300 import binding as sdm
from tests import paged_reference as ref

pytestmark = pytest.mark.gpu


def same(a, b):
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    return np.array_equal(a, b, equal_nan=True)


def read_back(s, count, first=None):
    cu = torch.tensor(np.concatenate([[0], np.cumsum(count)]), dtype=torch.int32, device="cuda")
    f = None if first is None else torch.tensor(first, dtype=torch.int32, device="cuda")
    got = sdm.cache_read(s.cache, cu, int(sum(count)), first=f, dev_status=s.status)
    return {n: got[n].double().cpu() for n in "kv"}, cu.cpu().numpy()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("G,D,page", [(1, 64, 16), (8, 128, 64), (3, 128, 128), (5, 64, 32)])
@pytest.mark.parametrize("w,ctx", [([1], [0]), ([1, 8, 3], [31, 0, 200]), ([0, 5, 0, 1, 0], [3, 15, 7, 127, 0]),
                                   ([130, 1], [63, 129])])
def test_write_then_read(gpu_lib, e4m3, G, D, page, w, ctx):
    s = ref.Setup(w, ctx, G, D, page, e4m3, seed=G * D + len(w))
    s.write_all()
    count = [a + b for a, b in zip(w, ctx)]
    if sum(count) == 0:
        return
    got, cu = read_back(s, count)
    for i in range(len(w)):
        for n in "kv":
            assert same(got[n][cu[i]:cu[i + 1]], s.held(i, n)), (i, n)
    assert s.status.item() == 0
    # a part of each request's tokens, from the middle
    first = [c // 2 for c in count]
    got, cu = read_back(s, [c - f for c, f in zip(count, first)], first)
    for i in range(len(w)):
        assert same(got["v"][cu[i]:cu[i + 1]], s.held(i, "v")[first[i]:])


def test_write_touches_only_its_slots(gpu_lib):
    s = ref.Setup([2, 1], [5, 40], 2, 64, 16, False, fill=7.0)
    before = s.cache.k.clone()
    sdm.cache_write(s.cache, s.packed("k"), s.packed("v"), s.cu, s.ctx, dev_status=s.status)
    changed = (s.cache.k != before).any(-1).any(1)              # [pages, slots]
    want = torch.zeros_like(changed)
    for i, (w, c) in enumerate(zip(s.w, s.ctx_list)):
        for t in range(c, c + w):
            want[s.table_cpu[i, t // 16].item(), t % 16] = True
    assert torch.equal(changed, want)


@pytest.mark.parametrize("D", [64, 128])
def test_e4m3_values_at_the_edges(gpu_lib, D):
    """Rows of one size and mixed sizes, zeros, the largest and smallest
    numbers, subnormals, ties, NaN and infinities."""
    rows = []
    g = torch.Generator().manual_seed(5)
    for k in list(range(-133, 128, 3)) + [127]:
        rows.append(torch.randn(D, generator=g) * 2.0 ** min(k, 125))
    rows.append(torch.zeros(D))
    rows.append(torch.linspace(-448, 448, D))
    rows.append(torch.arange(D).float() / 16 + 16)                        # exact ties of the grid
    rows.append(torch.cat([torch.full((1,), 448.0), torch.arange(D - 1) * 2.0 ** -10]))   # code subnormals
    rows.append(torch.cat([torch.full((1,), 449.0), torch.ones(D - 1)]))
    rows.append(torch.full((D,), torch.finfo(torch.bfloat16).max))
    rows.append(torch.full((D,), -2.0 ** -133))
    x = torch.randn(D, generator=g)
    x[3], x[7], x[D - 1] = float("nan"), float("inf"), float("-inf")
    rows.append(x)
    rows.append(torch.full((D,), float("nan")))
    x = torch.stack(rows).to(torch.bfloat16)[:, None]                     # [n, 1, D]
    n = x.shape[0]
    s = ref.Setup([n], [0], 1, D, 16, True)
    sdm.cache_write(s.cache, x.cuda(), -x.cuda(), s.cu, s.ctx, dev_status=s.status)
    got, _ = read_back(s, [n])
    assert same(got["k"], ref.held(x, True))
    assert same(got["v"], ref.held(-x, True))
    assert s.status.item() == 0


def test_write_takes_slices_and_streams(gpu_lib):
    """Rows inside a wider projection output, on a side stream."""
    s = ref.Setup([3, 9], [10, 0], 4, 128, 32, True)
    wide = torch.randn((12, 20, 128)).to(torch.bfloat16).cuda()
    wide[:, 8:12], wide[:, 12:16] = s.packed("k"), s.packed("v")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        sdm.cache_write(s.cache, wide[:, 8:12], wide[:, 12:16], s.cu, s.ctx, dev_status=s.status)
        got, cu = read_back(s, s.w, s.ctx_list)
    st.synchronize()
    for i in range(2):
        assert same(got["k"][cu[i]:cu[i + 1]], s.held(i, "k")[s.ctx_list[i]:])


def commit_reference(tok, parent, n, out_tok, accept):
    path = [0]
    for t in out_tok[:accept]:
        hit = [c for c in range(path[-1] + 1, n) if parent[c] == path[-1] and tok[c] == t]
        if not hit:
            break
        path.append(hit[0])
    return path


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("G,D,page,S,depth", [(2, 64, 16, 17, 6), (8, 128, 64, 65, 16), (1, 128, 32, 5, 4),
                                              (3, 64, 128, 200, 40)])
def test_commit_moves_the_accepted_path(gpu_lib, e4m3, G, D, page, S, depth):
    R = 6
    rng = np.random.default_rng(S)
    t = ref.random_trees(R, S, depth, rng)
    t["n_nodes"][1] = max(1, S // 2)
    ctx = [0, 15, 16, 100, 63, 1]
    s = ref.Setup([S] * R, ctx, G, D, page, e4m3, seed=S)
    s.write_all()
    out_tok, accept, paths = np.full((R, depth + 1), -1, np.int32), np.zeros(R, np.int32), []
    for i in range(R):
        end = [0, 0, S - 1, S // 2, S - 2, 1][i] % max(1, t["n_nodes"][i])
        chain = []
        while end > 0:
            chain.append(t["tok"][i, end])
            end = t["parent"][i, end]
        accept[i] = len(chain)
        out_tok[i, :len(chain)] = chain[::-1]
        out_tok[i, len(chain)] = 5000
        paths.append(commit_reference(t["tok"][i], t["parent"][i], t["n_nodes"][i], out_tok[i], accept[i]))
        assert len(paths[-1]) == accept[i] + 1
    d = {k: torch.as_tensor(v).cuda() for k, v in t.items()}
    got = sdm.cache_commit(s.cache, d["tok"], d["parent"], d["n_nodes"], torch.as_tensor(out_tok).cuda(),
                           torch.as_tensor(accept).cuda(), s.ctx, dev_status=s.status)
    assert got["length"].tolist() == [c + len(p) for c, p in zip(ctx, paths)]
    for i in range(R):
        assert got["path"][i].tolist() == paths[i] + [-1] * (depth + 1 - len(paths[i]))
    back, cu = read_back(s, [c + S for c in ctx])
    for i in range(R):
        for n in "kv":
            want = s.held(i, n)
            want[ctx[i]:ctx[i] + len(paths[i])] = want[[ctx[i] + c for c in paths[i]]]
            assert same(back[n][cu[i]:cu[i + 1]], want), (i, n)
    assert s.status.item() == 0


def test_commit_cuts_a_broken_path(gpu_lib):
    tok = torch.tensor([[9, 1, 2, 3]], dtype=torch.int32).cuda()
    parent = torch.tensor([[-1, 0, 1, 0]], dtype=torch.int32).cuda()
    s = ref.Setup([4], [3], 1, 64, 16, False)
    s.write_all()
    got = sdm.cache_commit(s.cache, tok, parent, torch.tensor([4], dtype=torch.int32).cuda(),
                           torch.tensor([[3, 77, 5]], dtype=torch.int32).cuda(),
                           torch.tensor([2], dtype=torch.int32).cuda(), s.ctx, dev_status=s.status)
    assert got["path"].tolist() == [[0, 3, -1]] and got["length"].tolist() == [5]
    assert s.status.item() == sdm.DEV_BAD_TOKEN


def test_pages_outside_the_pool_are_skipped(gpu_lib):
    s = ref.Setup([4], [14], 2, 64, 16, False, fill=0.0)
    s.cache.table[0, 1] = 10 ** 6
    keep = s.cache.k.clone()
    sdm.cache_write(s.cache, s.packed("k"), s.packed("v"), s.cu, s.ctx, dev_status=s.status)
    assert s.status.item() == sdm.DEV_BAD_PAGE
    page = s.table_cpu[0, 0].item()
    assert torch.equal(s.cache.k[page, :, 14:].cpu(), s.kv[0]["k"][14:16].permute(1, 0, 2))
    keep[page, :, 14:] = s.cache.k[page, :, 14:]
    assert torch.equal(s.cache.k, keep)                          # the two other tokens went nowhere
    s.status.zero_()
    got, _ = read_back(s, [4], [14])
    assert s.status.item() == sdm.DEV_BAD_PAGE
    assert same(got["k"][:2], s.kv[0]["k"][14:16].double()) and not got["k"][2:].any()


def test_lengths_outside_the_table_are_cut(gpu_lib):
    s = ref.Setup([4, 2], [10, 3], 1, 64, 16, False, fill=0.0)
    columns = s.cache.table.shape[1]
    for ctx, bit in ((16 * columns - 2, sdm.DEV_BAD_PAGE), (2 ** 31 - 2, sdm.DEV_BAD_PAGE),
                     (-5, sdm.DEV_BAD_WINDOW)):
        s.status.zero_()
        c = s.ctx.clone()
        c[0] = ctx
        sdm.cache_write(s.cache, s.packed("k"), s.packed("v"), s.cu, c, dev_status=s.status)
        assert s.status.item() & bit
    s.status.zero_()
    cu = torch.tensor([0, 5, 3], dtype=torch.int32).cuda()       # not monotone, and past the rows
    sdm.cache_write(s.cache, s.packed("k")[:4], s.packed("v")[:4], cu, s.ctx, dev_status=s.status)
    assert s.status.item() & sdm.DEV_BAD_WINDOW


def test_slots_past_32_bits(gpu_lib):
    """A pool whose last pages lie beyond 2^32 elements."""
    page, G, D = 128, 4, 128
    n = 2 ** 32 // (page * G * D) + 8
    k, v = (torch.empty((n, G, page, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.tensor([[n - 1, n - 3]], dtype=torch.int32).cuda()
    cache = sdm.PagedCache(k, v, table)
    cu, ctx = torch.tensor([0, 5], dtype=torch.int32).cuda(), torch.tensor([126], dtype=torch.int32).cuda()
    x = torch.randn((5, G, D)).to(torch.bfloat16).cuda()
    status = sdm.cache_write(cache, x, -x, cu, ctx)
    assert torch.equal(k[n - 1, :, 126:].permute(1, 0, 2), x[:2])
    assert torch.equal(v[n - 3, :, :3].permute(1, 0, 2), -x[2:])
    got = sdm.cache_read(cache, cu, 5, first=ctx, dev_status=status)
    assert torch.equal(got["k"], x) and torch.equal(got["v"], -x) and status.item() == 0

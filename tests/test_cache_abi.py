"""Host validation of the paged-cache entry points and the binding's checks
(no GPU: these paths return before any CUDA call)."""
from __future__ import annotations

import ctypes

import pytest
import torch

from speculative_decoding_markov_gb300 import binding, build

FAKE = 0x1000   # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def cache(**kw):
    a = dict(k=FAKE, v=FAKE, k_exp=None, v_exp=None, table=FAKE, dtype=0, n_pages=4, kv_heads=2, page=16,
             head_dim=128, max_pages=2)
    a.update(kw)
    return ctypes.byref(binding.SdmCache(*a.values()))


def write(lib, c=None, k=FAKE, v=FAKE, ks=256, vs=256, cu=FAKE, ctx=FAKE, R=1, rows=1):
    return lib.sdm_cache_write(c or cache(), k, v, ks, vs, cu, ctx, R, rows, None, None)


def attend(lib, c=None, q=FAKE, qs=1024, cu=FAKE, ctx=FAKE, R=1, rows=1, mw=1, H=8, scale=1.0, window=0, sinks=0,
           mask=None, nodes=0, out=FAKE, ws=FAKE, ws_bytes=1 << 30):
    return lib.sdm_attend(c or cache(), q, qs, cu, ctx, R, rows, mw, H, scale, window, sinks, mask, nodes, out, None,
                          ws, ws_bytes, None, None)


@pytest.mark.parametrize("bad,want", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(table=None), 1), (dict(dtype=1), 1), (dict(dtype=3), 1),
    (dict(dtype=2), 1), (dict(dtype=2, k_exp=FAKE), 1), (dict(n_pages=0), 1), (dict(kv_heads=0), 1),
    (dict(max_pages=0), 1), (dict(head_dim=96), 2), (dict(head_dim=256), 2), (dict(page=8), 2), (dict(page=48), 2),
    (dict(n_pages=1 << 30), 2), (dict(k=FAKE + 8), 2), (dict(dtype=2, k_exp=FAKE + 4, v_exp=FAKE), 2)])
def test_caches_that_are_refused(lib, bad, want):
    c = cache(**bad)
    assert write(lib, c) == want
    assert attend(lib, c) == want
    assert lib.sdm_cache_read(c, FAKE, None, 1, 1, FAKE, FAKE, None, None) == want
    assert lib.sdm_cache_commit(c, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1, 4, 4, FAKE, None, None, None) == want


@pytest.mark.parametrize("bad,want", [
    (dict(k=None), 1), (dict(cu=None), 1), (dict(ctx=None), 1), (dict(R=0), 1), (dict(rows=-1), 1),
    (dict(ks=255), 2), (dict(ks=128), 2), (dict(vs=260), 2), (dict(k=FAKE + 2), 2), (dict(rows=0), 0)])
def test_write_validation(lib, bad, want):
    assert write(lib, **bad) == want


def test_read_and_commit_validation(lib):
    read = lib.sdm_cache_read
    assert read(cache(), None, None, 1, 1, FAKE, FAKE, None, None) == 1
    assert read(cache(), FAKE, None, 1, 1, None, FAKE, None, None) == 1
    assert read(cache(), FAKE, None, 0, 1, FAKE, FAKE, None, None) == 1
    assert read(cache(), FAKE, None, 1, 1, FAKE + 2, FAKE, None, None) == 2
    assert read(cache(), FAKE, None, 1, 0, FAKE, FAKE, None, None) == 0
    commit = lib.sdm_cache_commit
    a = [cache(), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1, 4, 4, FAKE, None, None, None]
    for at, value, want in ((1, None, 1), (6, None, 1), (10, None, 1), (7, 0, 1), (8, -1, 1), (9, 0, 1),
                            (8, 16384, 2), (9, 20000, 2)):
        b = list(a)
        b[at] = value
        assert commit(*b) == want, (at, value)


@pytest.mark.parametrize("bad,want", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(cu=None), 1), (dict(ctx=None), 1), (dict(R=0), 1), (dict(mw=0), 1),
    (dict(H=0), 1), (dict(H=7), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(sinks=-1), 1), (dict(mask=FAKE, nodes=3, mw=4), 1), (dict(R=16385), 2),
    (dict(qs=1000), 2), (dict(qs=1020), 2), (dict(q=FAKE + 4), 2), (dict(out=FAKE + 4), 2), (dict(mw=1 << 29), 2),
    (dict(ws=None), 5), (dict(ws_bytes=0), 5), (dict(rows=0), 0)])
def test_attend_validation(lib, bad, want):
    assert attend(lib, **bad) == want


def test_the_binding_refuses_what_the_kernels_cannot_check():
    table = torch.zeros((1, 2), dtype=torch.int32)
    k = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        binding.PagedCache(k, k, table)                  # not on a GPU
    with pytest.raises(TypeError):
        binding._need_rows("q", torch.zeros((3, 4, 64)), 4, 64)
    with pytest.raises(ValueError):
        binding._need_i32("cu_seqlens", torch.zeros(4, dtype=torch.int32), 4)


def test_device_bit_of_a_bad_page(lib):
    assert lib.sdm_status_of_device(binding.DEV_BAD_PAGE) == 6
    assert lib.sdm_workspace_size(binding.OP_ATTEND, 64, 8, 32, 128, 512, 8, 0) > 0


def test_attend_refuses_more_heads_per_kv_head_than_a_tile_holds(lib):
    assert attend(lib, H=2 * 129, qs=2 * 129 * 128) == 2
    assert attend(lib, H=2 * 128, qs=2 * 128 * 128, ws_bytes=0) == 5      # accepted up to the workspace
    assert attend(lib, ws=FAKE + 16) == 5                                 # the workspace starts on 256 bytes

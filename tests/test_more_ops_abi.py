"""Host validation of the norm-and-rotation, log-probability, attention-weight
and eviction entry points and the binding's checks (no GPU: these paths return
before any CUDA call)."""
from __future__ import annotations

import weakref

import pytest
import torch

from speculative_decoding_markov_gb300 import binding, build
from tests.test_cache_abi import FAKE, cache
from tests.test_cache_binding import Library, Tensor


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def rotate(lib, c="none", q=FAKE, qs=1024, H=8, k=FAKE, ks=256, v=None, vs=256, G=2, D=128, wq=None, wk=None, eps=1e-6,
           freq=FAKE, rot=128, inter=0, cu=FAKE, ctx=FAKE, start=None, pos=None, R=1, rows=1, qo=FAKE, qos=1024, ko=FAKE,
           kos=256):
    return lib.sdm_qk_rotate(None if c == "none" else c, q, qs, H, k, ks, v, vs, G, D, wq, wk, eps, freq, rot, inter, cu,
                             ctx, start, pos, R, rows, qo, qos, ko, kos, None, None)


@pytest.mark.parametrize("bad,want", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(qo=None), 1), (dict(ko=None), 1), (dict(v=FAKE), 1), (dict(cu=None), 1),
    (dict(ctx=None), 1), (dict(R=0), 1), (dict(rows=-1), 1), (dict(H=0), 1), (dict(G=0), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(rot=-8), 1), (dict(rot=136), 1), (dict(freq=None), 1),
    (dict(D=96, rot=8), 2), (dict(rot=12), 2), (dict(qs=1000), 2), (dict(qs=1028), 2), (dict(ks=128), 2), (dict(qos=512), 2),
    (dict(kos=250), 2), (dict(q=FAKE + 8), 2), (dict(ko=FAKE + 4), 2), (dict(wq=FAKE + 4), 2), (dict(wk=FAKE + 8), 2),
    (dict(rows=1 << 28), 2), (dict(rows=0), 0), (dict(rows=0, q=None, ctx=None, start=FAKE), 0)])
def test_rotate_validation(lib, bad, want):
    assert rotate(lib, **bad) == want


@pytest.mark.parametrize("bad,want", [
    (dict(), 1), (dict(ko=None), 1), (dict(v=FAKE), 1), (dict(v=FAKE, ko=None, D=64, rot=64), 1),
    (dict(v=FAKE, ko=None, G=4), 1), (dict(v=FAKE, ko=None, ctx=None, start=FAKE), 1), (dict(v=FAKE, ko=None, vs=250), 2),
    (dict(v=FAKE + 2, ko=None), 2), (dict(v=FAKE, ko=None, rows=0), 0)])
def test_rotate_into_a_cache_validation(lib, bad, want):
    assert rotate(lib, c=cache(), **bad) == want


def test_rotate_takes_no_bad_cache(lib):
    assert rotate(lib, c=cache(page=48), v=FAKE, ko=None) == 2
    assert rotate(lib, c=cache(dtype=2), v=FAKE, ko=None) == 1


def logprobs(lib, z=FAKE, dt=0, rows=1, V=1024, cu=FAKE, path=None, tok=FAKE, n=None, R=1, W=1, T=1.0, top=0, logp=FAKE,
             tt=None, tl=None):
    return lib.sdm_token_logprobs(z, dt, rows, V, cu, path, tok, n, R, W, T, top, logp, None, None, tt, tl, None, None)


@pytest.mark.parametrize("bad,want", [
    (dict(z=None), 1), (dict(dt=2), 1), (dict(rows=-1), 1), (dict(V=0), 1), (dict(V=1020), 2), (dict(cu=None), 1),
    (dict(tok=None), 1), (dict(R=0), 1), (dict(W=0), 1), (dict(T=0.0), 1), (dict(T=-1.0), 1), (dict(T=float("nan")), 1),
    (dict(T=float("inf")), 1), (dict(T=1e-35), 1), (dict(T=1e35), 1), (dict(top=-1), 1), (dict(top=3), 1),
    (dict(top=3, tt=FAKE), 1), (dict(top=33, tt=FAKE, tl=FAKE), 2), (dict(V=8, top=9, tt=FAKE, tl=FAKE), 1),
    (dict(logp=None), 1), (dict(z=FAKE + 8), 2), (dict(R=1 << 20, W=1 << 8), 2), (dict(rows=0, z=None), 0)])
def test_logprobs_validation(lib, bad, want):
    assert logprobs(lib, **bad) == want


def weight(lib, c=None, q=FAKE, qs=1024, lse=FAKE, cu=FAKE, ctx=FAKE, count=None, path=None, ps=0, R=1, rows=1, mc=1, H=8,
           scale=1.0, window=0, sinks=0, mass=None, out=FAKE, stride=100, ws=FAKE, ws_bytes=1 << 40):
    return lib.sdm_attend_weight(c or cache(), q, qs, lse, cu, ctx, count, path, ps, R, rows, mc, H, scale, window, sinks,
                                 mass, out, stride, ws, ws_bytes, None, None)


@pytest.mark.parametrize("bad,want", [
    (dict(q=None), 1), (dict(lse=None), 1), (dict(cu=None), 1), (dict(ctx=None), 1), (dict(out=None), 1), (dict(R=0), 1),
    (dict(rows=-1), 1), (dict(mc=-1), 1), (dict(H=0), 1), (dict(H=7), 1), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(sinks=-1), 1), (dict(path=FAKE, ps=0), 1), (dict(stride=0), 1),
    (dict(stride=1 << 31), 2), (dict(R=16385), 2), (dict(qs=1000), 2), (dict(qs=1020), 2), (dict(q=FAKE + 4), 2),
    (dict(H=258, qs=1 << 20), 2), (dict(mc=1 << 29), 2)])
def test_weight_validation(lib, bad, want):
    assert weight(lib, **bad) == want
    assert weight(lib, c=cache(head_dim=96)) == 2


def evict(lib, c=None, mass=FAKE, pos=FAKE, stride=100, ctx=FAKE, count=None, start=None, R=1, keep=10, sinks=0, recent=0,
          mo=FAKE, po=FAKE, length=FAKE * 2, nxt=None, ws=FAKE, ws_bytes=1 << 40):
    return lib.sdm_cache_evict(c or cache(), mass, pos, stride, ctx, count, start, R, keep, sinks, recent, mo, po, length,
                               nxt, ws, ws_bytes, None, None)


@pytest.mark.parametrize("bad,want", [
    (dict(mass=None), 1), (dict(pos=None), 1), (dict(mo=None), 1), (dict(po=None), 1), (dict(ctx=None), 1),
    (dict(length=None), 1), (dict(R=0), 1), (dict(stride=0), 1), (dict(stride=1 << 31), 2), (dict(keep=0), 1),
    (dict(sinks=-1), 1), (dict(recent=-1), 1), (dict(sinks=5, recent=6), 1), (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), 1),
    (dict(length=FAKE), 1), (dict(nxt=FAKE), 1), (dict(start=FAKE * 3, nxt=FAKE * 3), 1), (dict(R=1 << 24), 2),
    (dict(ws=None), 5), (dict(ws=FAKE + 16), 5), (dict(ws_bytes=8), 5)])
def test_evict_validation(lib, bad, want):
    assert evict(lib, **bad) == want
    assert evict(lib, c=cache(page=7)) == 2


def test_workspaces(lib):
    size = lib.sdm_workspace_size
    assert size(binding.OP_CACHE_EVICT, 2, 3, 0, 0, 100, 0, 40) == 2 * 3 * 40 * 8
    assert size(binding.OP_CACHE_EVICT, 2, 3, 0, 0, 100, 0, 90) == 2 * 3 * 10 * 8
    assert size(binding.OP_CACHE_EVICT, 2, 3, 0, 0, 100, 0, 200) == 0


# ---------------------------------------------------------------------------
# the binding: stand-ins for tensors and the library
# ---------------------------------------------------------------------------
BF16, F32, F64, U8 = torch.bfloat16, torch.float32, torch.float64, torch.uint8


@pytest.fixture
def called(monkeypatch):
    stand_in = Library()
    stand_in.sdm_workspace_size = lambda *a: 0
    monkeypatch.setattr(binding, "lib", lambda: stand_in)
    monkeypatch.setattr(binding, "_this_device", lambda: 0)
    monkeypatch.setattr(binding, "_raw_stream", lambda d: 0)
    return stand_in.calls


def paged():
    c = binding.PagedCache.__new__(binding.PagedCache)
    c.requests, c.device, c.alone, c.kv_heads, c.head_dim, c.ref = 2, 0, True, 2, 128, None
    c.k = Tensor((4, 2, 16, 128), BF16)
    return c


def rotate_args(**kw):
    a = dict(q=Tensor((3, 8, 128), BF16), k=Tensor((3, 2, 128), BF16), cu_seqlens=Tensor((3,)), ctx_len=Tensor((2,)),
             freq=Tensor((64,), F64), v=Tensor((3, 2, 128), BF16), cache=paged(), out=dict(q=Tensor((3, 8, 128), BF16)),
             dev_status=Tensor((1,)))
    a.update(kw)
    return a


@pytest.mark.parametrize("bad", [
    dict(v=None), dict(cache=None), dict(k=Tensor((3, 4, 128), BF16)), dict(q=Tensor((3, 8, 128), F32)),
    dict(q=Tensor((4, 8, 128), BF16)), dict(v=Tensor((2, 2, 128), BF16)), dict(q=Tensor((3, 8, 128), BF16, device=-1)),
    dict(freq=Tensor((64,), F32)), dict(freq=Tensor((64,), F64, device=1)), dict(q_weight=Tensor((64,), F32)),
    dict(k_weight=Tensor((128,), BF16)), dict(cu_seqlens=Tensor((2,))), dict(ctx_len=Tensor((1,))),
    dict(start=Tensor((2,), torch.int64)), dict(row_pos=Tensor((2,))), dict(out=dict(q=Tensor((2, 8, 128), BF16))),
    dict(out=dict(q=Tensor((3, 8, 128), BF16, device=1))), dict(dev_status=Tensor((1,), device=1))])
def test_rotate_binding(called, bad):
    with pytest.raises((ValueError, TypeError)):
        binding.qk_rotate(**rotate_args(**bad))
    assert not called
    binding.qk_rotate(**rotate_args())
    assert len(called) == 1


def weight_args(**kw):
    a = dict(cache=paged(), q=Tensor((3, 8, 128), BF16), lse=Tensor((3, 8), F32), cu_seqlens=Tensor((3,)),
             ctx_len=Tensor((2,)), max_count=2, mass=Tensor((2, 2, 50), F32), out=dict(mass=Tensor((2, 2, 50), F32)),
             ws=Tensor((256,), U8), dev_status=Tensor((1,)))
    a.update(kw)
    return a


@pytest.mark.parametrize("bad", [
    dict(q=Tensor((3, 7, 128), BF16)), dict(lse=Tensor((3, 7), F32)), dict(lse=Tensor((3, 8), BF16)),
    dict(mass=Tensor((2, 2, 49), F32)), dict(out=dict(mass=Tensor((2, 3, 50), F32))), dict(mass=None, out=None),
    dict(out=dict(mass=Tensor((2, 2, 50), F32, device=1))), dict(path=Tensor((2, 1))), dict(path=Tensor((3, 2))),
    dict(count=Tensor((1,))), dict(ws=Tensor((256,), F32)), dict(dev_status=Tensor((1,), device=-1))])
def test_weight_binding(called, bad):
    with pytest.raises((ValueError, TypeError)):
        binding.attend_weight(**weight_args(**bad))
    assert not called
    binding.attend_weight(**weight_args(path=Tensor((2, 5)), count=Tensor((2,))))
    assert len(called) == 1


def evict_args(**kw):
    a = dict(cache=paged(), mass=Tensor((2, 2, 50), F32), pos=Tensor((2, 2, 50)), ctx_len=Tensor((2,)), start=Tensor((2,)),
             keep=10, ws=Tensor((256,), U8), dev_status=Tensor((1,)),
             out=dict(mass=Tensor((2, 2, 50), F32), pos=Tensor((2, 2, 50)), length=Tensor((2,))))
    a.update(kw)
    return a


@pytest.mark.parametrize("bad", [
    dict(mass=Tensor((2, 2), F32)), dict(mass=Tensor((2, 3, 50), F32)), dict(mass=Tensor((2, 2, 50), BF16)),
    dict(pos=Tensor((2, 2, 49))), dict(pos=Tensor((2, 2, 50), torch.int64)), dict(start=Tensor((1,))),
    dict(out=dict(mass=Tensor((2, 2, 50), F32), pos=Tensor((2, 2, 50)), length=Tensor((1,)))),
    dict(count=Tensor((2,), F32)), dict(ws=Tensor((256,), U8, device=1))])
def test_evict_binding(called, bad):
    with pytest.raises((ValueError, TypeError)):
        binding.cache_evict(**evict_args(**bad))
    assert not called
    binding.cache_evict(**evict_args())
    assert len(called) == 1


def logprob_args(**kw):
    a = dict(target=Tensor((5, 64), BF16), cu_seqlens=Tensor((3,)), tok=Tensor((2, 4)), top=2, dev_status=Tensor((1,)),
             out=dict(logp=Tensor((2, 4), F32), top_tok=Tensor((2, 4, 2)), top_logp=Tensor((2, 4, 2), F32)))
    a.update(kw)
    return a


@pytest.mark.parametrize("bad", [
    dict(target=Tensor((5, 64), torch.float16)), dict(target=Tensor((5, 64), BF16, device=-1)),
    dict(target=Tensor((5, 64), BF16, device=1)), dict(target=Tensor((5, 64), BF16, stride=(128, 1))),
    dict(cu_seqlens=Tensor((2,))), dict(tok=Tensor((2, 4), torch.int64)), dict(n=Tensor((1,))), dict(path=Tensor((2, 3))),
    dict(out=dict(logp=Tensor((2, 4), F32), top_tok=Tensor((2, 4, 1)), top_logp=Tensor((2, 4, 2), F32))),
    dict(out=dict(logp=Tensor((2, 4), F64), top_tok=Tensor((2, 4, 2)), top_logp=Tensor((2, 4, 2), F32)))])
def test_logprobs_binding(called, bad):
    with pytest.raises((ValueError, TypeError)):
        binding.token_logprobs(**logprob_args(**bad))
    assert not called
    binding.token_logprobs(**logprob_args())
    assert len(called) == 1


def test_tensors_live_until_the_library_is_called(called, monkeypatch):
    """A tensor made in the call itself is not freed before the launch: the
    workspace would be allocated where it was."""
    refs = []

    def made(*a):
        refs.append(weakref.ref(x := Tensor(*a)))
        return x

    def alive(*a):
        assert all(r() is not None for r in refs)
        return Tensor((256,), U8)

    for name in ("workspace", "attend_weight_workspace", "cache_evict_workspace", "attend_workspace"):
        monkeypatch.setattr(binding, name, lambda *a, **k: alive())
    monkeypatch.setattr(binding, "new_status", lambda d: alive() and Tensor((1,)))
    binding.attend_weight(paged(), made((3, 8, 128), BF16), made((3, 8), F32), made((3,)), made((2,)), 2,
                          mass=made((2, 2, 50), F32), count=made((2,)), path=made((2, 5)),
                          out=dict(mass=made((2, 2, 50), F32)))
    assert len(called) == 1 and len(refs) == 8
    refs.clear()
    binding.cache_evict(paged(), made((2, 2, 50), F32), made((2, 2, 50)), made((2,)), made((2,)), 10, count=made((2,)),
                        out=dict(mass=made((2, 2, 50), F32), pos=made((2, 2, 50)), length=made((2,))))
    refs.clear()
    binding.qk_rotate(made((3, 8, 128), BF16), made((3, 2, 128), BF16), made((3,)), made((2,)), made((64,), F64),
                      v=made((3, 2, 128), BF16), cache=paged(), start=made((2,)), row_pos=made((3,)),
                      q_weight=made((128,), F32), k_weight=made((128,), F32), out=dict(q=made((3, 8, 128), BF16)))
    refs.clear()
    binding.token_logprobs(made((5, 64), BF16), made((3,)), made((2, 4)), n=made((2,)), path=made((2, 4)),
                           out=dict(logp=made((2, 4), F32)))
    refs.clear()
    binding.attend(paged(), made((3, 8, 128), BF16), made((3,)), made((2,)), 2, lse=True, tree_mask=made((2, 5, 1)),
                   out=dict(out=made((3, 8, 128), BF16), lse=made((3, 8), F32)))
    assert len(called) == 5


@pytest.mark.parametrize("path,fits", [((2, 4), True), ((8,), True), ((2, 5), False), ((2, 9), False), ((4, 4), True),
                                       ((1, 8), False), ((2, 4, 1), False), ((9,), True)])
def test_logprobs_path_has_rows_as_long_as_the_tokens(called, path, fits):
    """Rows of another length would be read as if they had the tokens'."""
    if fits:
        binding.token_logprobs(**logprob_args(path=Tensor(path)))
    else:
        with pytest.raises(ValueError):
            binding.token_logprobs(**logprob_args(path=Tensor(path)))
    assert len(called) == fits

"""What the paged cache's binding checks before the library is called: types,
shapes, layouts and devices.  No GPU: stand-ins describe tensors, and a
stand-in of the library records the calls that come through."""
from __future__ import annotations

import ctypes

import pytest
import torch

from speculative_decoding_markov_gb300 import binding, build

DEV = 0


class Tensor:
    """As much of a CUDA tensor as the binding looks at."""

    def __init__(self, shape, dtype=torch.int32, device=DEV, stride=None, at=0x10000):
        self.shape, self.dtype, self.index, self.at = torch.Size(shape), dtype, device, at
        packed = [1]
        for n in reversed(shape[1:]):
            packed.insert(0, packed[0] * n)
        self.packed, self.st = tuple(packed), tuple(stride or packed)
        self.is_cuda = device >= 0
        self.device = torch.device("cuda", device) if device >= 0 else torch.device("cpu")

    def stride(self):
        return self.st

    def is_contiguous(self):
        return self.st == self.packed

    def get_device(self):
        return self.index

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return self.at if self.numel() else 0


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def called(monkeypatch):
    """The library's stand-in; the current device is DEV."""
    lib = Library()
    monkeypatch.setattr(binding, "lib", lambda: lib)
    monkeypatch.setattr(binding, "_this_device", lambda: DEV)
    monkeypatch.setattr(binding, "_raw_stream", lambda index: 7000 + index)
    return lib


def a_cache(R=2, G=2, D=64):
    c = object.__new__(binding.PagedCache)
    c.k = Tensor((8, G, 16, D), torch.bfloat16)
    c.requests, c.kv_heads, c.page, c.head_dim, c.device = R, G, 16, D, DEV
    c.c = binding.SdmCache()
    c.ref = ctypes.byref(c.c)
    return c


bf = dict(dtype=torch.bfloat16)


def attend_args(**kw):
    a = dict(cache=a_cache(), q=Tensor((6, 4, 64), **bf), cu_seqlens=Tensor((3,)), ctx_len=Tensor((2,)), max_window=4,
             out=dict(out=Tensor((6, 4, 64), **bf)), ws=Tensor((4096,), torch.uint8), dev_status=Tensor((1,)))
    a.update(kw)
    return a


def write_args(**kw):
    a = dict(cache=a_cache(), k=Tensor((6, 2, 64), **bf), v=Tensor((6, 2, 64), **bf), cu_seqlens=Tensor((3,)),
             ctx_len=Tensor((2,)), dev_status=Tensor((1,)))
    a.update(kw)
    return a


def read_args(**kw):
    a = dict(cache=a_cache(), cu_rows=Tensor((3,)), rows=6, dev_status=Tensor((1,)),
             out=dict(k=Tensor((6, 2, 64), **bf), v=Tensor((6, 2, 64), **bf)))
    a.update(kw)
    return a


def commit_args(**kw):
    a = dict(cache=a_cache(), tok=Tensor((2, 5)), parent=Tensor((2, 5)), n_nodes=Tensor((2,)), out_tok=Tensor((2, 4)),
             accept=Tensor((2,)), ctx_len=Tensor((2,)), dev_status=Tensor((1,)),
             out=dict(path=Tensor((2, 4)), length=Tensor((2,))))
    a.update(kw)
    return a


CALLS = dict(attend=(binding.attend, attend_args), write=(binding.cache_write, write_args),
             read=(binding.cache_read, read_args), commit=(binding.cache_commit, commit_args))


@pytest.mark.parametrize("which", CALLS)
def test_calls_that_are_right_reach_the_library(called, which):
    call, args = CALLS[which]
    call(**args())
    assert len(called.calls) == 1 and called.calls[0][1][-1] == 7000 + DEV     # on the device's current stream


@pytest.mark.parametrize("where", [-1, DEV + 1])
@pytest.mark.parametrize("which,bad", [
    ("attend", dict(q=((6, 4, 64), torch.bfloat16))), ("attend", dict(cu_seqlens=((3,),))),
    ("attend", dict(ctx_len=((2,),))), ("attend", dict(ws=((4096,), torch.uint8))),
    ("attend", dict(dev_status=((1,),))), ("attend", dict(tree_mask=((2, 9, 1),))),
    ("attend", dict(out=dict(out=((6, 4, 64), torch.bfloat16)))),
    ("attend", dict(out=dict(out=None, lse=((6, 4), torch.float32)))),
    ("write", dict(k=((6, 2, 64), torch.bfloat16))), ("write", dict(v=((6, 2, 64), torch.bfloat16))),
    ("write", dict(cu_seqlens=((3,),))), ("write", dict(ctx_len=((2,),))), ("write", dict(dev_status=((1,),))),
    ("read", dict(cu_rows=((3,),))), ("read", dict(first=((2,),))), ("read", dict(dev_status=((1,),))),
    ("read", dict(out=dict(k=((6, 2, 64), torch.bfloat16), v=None))),
    ("read", dict(out=dict(k=None, v=((6, 2, 64), torch.bfloat16)))),
    ("commit", dict(tok=((2, 5),))), ("commit", dict(parent=((2, 5),))), ("commit", dict(out_tok=((2, 4),))),
    ("commit", dict(accept=((2,),))), ("commit", dict(ctx_len=((2,),))), ("commit", dict(dev_status=((1,),))),
    ("commit", dict(out=dict(path=((2, 4),), length=None))), ("commit", dict(out=dict(path=None, length=((2,),))))])
def test_tensors_elsewhere_are_refused(called, which, bad, where):
    """Host memory and other devices, for inputs, outputs and scratch alike."""
    call, args = CALLS[which]
    a = args()
    for name, what in bad.items():
        if isinstance(what, dict):
            a[name] = {n: a[name][n] if t is None else Tensor(*t, device=where) for n, t in what.items()}
        else:
            a[name] = Tensor(*what, device=where)
    with pytest.raises((ValueError, TypeError)):
        call(**a)
    assert not called.calls


@pytest.mark.parametrize("which,bad", [
    ("attend", dict(ws=Tensor((4096,), torch.float32))), ("attend", dict(dev_status=Tensor((1,), torch.int64))),
    ("attend", dict(dev_status=Tensor((0,)))), ("attend", dict(out=dict(out=Tensor((6, 4, 64), torch.float32)))),
    ("attend", dict(out=dict(out=Tensor((5, 4, 64), **bf)))),
    ("attend", dict(out=dict(out=Tensor((6, 4, 64), torch.bfloat16, stride=(512, 64, 1))))),
    ("read", dict(out=dict(k=Tensor((6, 2, 64), **bf), v=Tensor((5, 2, 64), **bf)))),
    ("read", dict(out=dict(k=Tensor((6, 2, 64), torch.float16), v=Tensor((6, 2, 64), **bf))))])
def test_buffers_of_another_kind_are_refused(called, which, bad):
    call, args = CALLS[which]
    with pytest.raises((ValueError, TypeError)):
        call(**args(**bad))
    assert not called.calls


@pytest.mark.parametrize("which", CALLS)
def test_a_cache_off_the_current_device_is_refused(called, which, monkeypatch):
    """Its default stream's handle would be the current device's."""
    monkeypatch.setattr(binding, "_this_device", lambda: DEV + 1)
    call, args = CALLS[which]
    with pytest.raises(ValueError):
        call(**args())
    assert not called.calls


def test_a_cache_on_two_devices_is_refused():
    k = Tensor((8, 2, 16, 64), **bf)
    with pytest.raises(ValueError):
        binding.PagedCache(k, Tensor((8, 2, 16, 64), torch.bfloat16, device=DEV + 1), Tensor((2, 4)))
    with pytest.raises(ValueError):
        binding.PagedCache(k, k, Tensor((2, 4), device=DEV + 1))
    assert binding.PagedCache(k, k, Tensor((2, 4))).device == DEV


def test_an_lse_without_a_place_is_refused(called):
    with pytest.raises(ValueError):
        binding.attend(**attend_args(lse=True))
    assert not called.calls
    binding.attend(**attend_args(lse=True, out=dict(out=Tensor((6, 4, 64), **bf), lse=Tensor((6, 4), torch.float32))))
    assert len(called.calls) == 1


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def test_batches_without_rows(lib):
    """Tensors without rows have no address: nothing to do, nothing refused."""
    FAKE = 0x1000
    c = ctypes.byref(binding.SdmCache(FAKE, FAKE, None, None, FAKE, 0, 4, 2, 16, 64, 2))
    assert lib.sdm_cache_write(c, None, None, 128, 128, FAKE, FAKE, 1, 0, None, None) == 0
    assert lib.sdm_cache_read(c, FAKE, None, 1, 0, None, None, None, None) == 0
    for longest in (0, 4):
        assert lib.sdm_attend(c, None, 512, FAKE, FAKE, 1, 0, longest, 8, 1.0, 0, 0, None, 0, None, None, None, 0,
                              None, None) == 0
    # the rest is still looked at
    assert lib.sdm_cache_write(c, None, None, 128, 128, None, FAKE, 1, 0, None, None) == 1
    assert lib.sdm_cache_write(c, None, None, 128, 128, FAKE, FAKE, 1, 1, None, None) == 1
    assert lib.sdm_cache_read(c, FAKE, None, 0, 0, None, None, None, None) == 1
    assert lib.sdm_attend(c, None, 512, FAKE, FAKE, 1, 0, 4, 7, 1.0, 0, 0, None, 0, None, None, None, 0, None,
                          None) == 1
    assert lib.sdm_attend(c, FAKE, 512, FAKE, FAKE, 1, 1, 0, 8, 1.0, 0, 0, None, 0, FAKE, None, FAKE, 1 << 30, None,
                          None) == 1


def test_calls_without_rows_pass_the_binding(called):
    none = Tensor((0, 4, 64), **bf)
    binding.attend(**attend_args(q=none, out=dict(out=Tensor((0, 4, 64), **bf)), max_window=0))
    binding.cache_write(**write_args(k=Tensor((0, 2, 64), **bf), v=Tensor((0, 2, 64), **bf)))
    assert len(called.calls) == 2 and called.calls[0][1][1] == 0


def test_the_stride_of_a_single_row(called):
    """It leads nowhere: any value will do."""
    for stride in (1, 7, 128, 1001):
        assert binding._need_rows("k", Tensor((1, 2, 64), torch.bfloat16, stride=(stride, 64, 1)), 2, 64, DEV) == (1, 128)
    assert binding._need_rows("k", Tensor((2, 2, 64), torch.bfloat16, stride=(1000, 64, 1)), 2, 64, DEV) == (2, 1000)


def test_scales_whose_product_with_log2_e_is_infinite(lib):
    FAKE = 0x1000
    c = ctypes.byref(binding.SdmCache(FAKE, FAKE, None, None, FAKE, 0, 4, 2, 16, 64, 2))

    def attend(scale):
        return lib.sdm_attend(c, FAKE, 512, FAKE, FAKE, 1, 1, 4, 8, scale, 0, 0, None, 0, FAKE, None, None, 0, None, None)

    assert attend(2.5e38) == attend(2.9e38) == 1
    assert attend(1.9e38) == attend(1e-38) == 5                # accepted up to the workspace


@pytest.mark.parametrize("which", CALLS)
def test_a_status_of_the_calls_own_comes_back(called, which, monkeypatch):
    """What the device finds wrong is not lost when no dev_status is given."""
    made = Tensor((1,), at=0x7700)
    monkeypatch.setattr(binding, "new_status", lambda device: made)
    call, args = CALLS[which]
    got = call(**args(dev_status=None))
    assert (got if which == "write" else got["dev_status"]) is made
    assert 0x7700 in called.calls[0][1]
    if which != "write":
        assert "dev_status" not in call(**args())                    # a caller's own stays the caller's


@pytest.mark.parametrize("R,rows", [(2 ** 31 - 1, 1), (1, 2 ** 31 - 1), (2 ** 31 - 2 ** 16 + 1, 1)])
def test_counts_that_the_grids_strides_would_pass(lib, R, rows):
    FAKE = 0x1000
    c = ctypes.byref(binding.SdmCache(FAKE, FAKE, None, None, FAKE, 0, 4, 2, 16, 64, 2))
    assert lib.sdm_cache_write(c, FAKE, FAKE, 128, 128, FAKE, FAKE, R, rows, None, None) == 2
    assert lib.sdm_cache_read(c, FAKE, None, R, rows, FAKE, FAKE, None, None) == 2

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

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

"""Attention weight at its limits: infinite keys beside columns that no row
fills."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from speculative_decoding_markov_gb300 import binding as sdm
from tests import paged_reference as ref
from tests.test_gpu_weight_evict import i32, weights

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group,w", [(7, 18), (3, 42), (5, 25), (6, 21), (65, 1), (100, 1), (7, 40), (3, 130), (12, 60),
                                     (33, 9), (100, 5), (8, 16), (8, 50)])
def test_keys_of_minus_infinity_against_every_row(gpu_lib, D, group, w):
    """Every score of such a key is -inf and its weight nothing, also where the
    rows' tiles have columns without a row: 0 times infinity is in no sum."""
    s = ref.Setup([w], [400], 1, D, 16, False, seed=group)
    for j in (0, 130, 257, 399, 400):
        s.kv[0]["k"][j, 0, j % D] = -INF
    s.write_all()
    q = torch.rand((w, group, D), generator=s.gen).add(0.25).to(torch.bfloat16).cuda()
    lse = (3 + torch.rand((w, group), generator=s.gen)).cuda()
    T = 400 + w
    mass = torch.rand((1, 1, T), generator=s.gen).cuda()
    out = dict(mass=torch.zeros_like(mass))
    sdm.attend_weight(s.cache, q, lse, s.cu, s.ctx, w, mass=mass, out=out, dev_status=s.status)
    assert s.status.item() == 0
    want, tol = weights(q, lse, s.held(0, "k"), ref.visible(w, 400), D ** -0.5, group)
    old = mass[0].double().cpu().numpy()
    old[:, 400:] = 0
    got = out["mass"][0].double().cpu().numpy()
    assert (np.abs(got - want - old) <= tol + 2.0 ** -24 * (want + old)).all()
    assert (got[0, [0, 130, 257, 399, 400]] == old[0, [0, 130, 257, 399, 400]]).all()
    again = dict(mass=torch.zeros_like(mass))                      # the rows gathered along a path
    sdm.attend_weight(s.cache, q, lse, s.cu, s.ctx, w, mass=mass, path=i32([list(range(w))]), out=again, dev_status=s.status)
    assert torch.equal(again["mass"], out["mass"]) and s.status.item() == 0

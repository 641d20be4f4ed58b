"""How far the attention's result may be from the 64-bit form, per form of the
weights, on rows where few of the keys count.

The result is rounded to bf16, 8 significant bits: at most 2^-8 |out|.  The
weights enter the second product as bf16, an error of at most 2^-8 of each and
so of 2^-8 size in the sum, size = sum_j p_j |v_j|.  Where their remainders
are multiplied too, what is left of a weight is the remainder's own rounding,
2^-16.  The scores' error: the products of bf16 are exact, a row's 128 are
added in fp32 with at most 2^-22 of their sum of magnitudes (below 60 here) in
each of 8 steps, 2^-13.1 in all, twice that in a quotient of exponentials; the
exponentials and the sums of weights stay below 2^-20.  Together below

    with remainders     2^-8 |out| + 2^-11 size
    without             2^-8 |out| + (2^-8 + 2^-11) size
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import paged_reference as ref

EXACT, PLAIN = 2.0 ** -11, 2.0 ** -8 + 2.0 ** -11
gpu = pytest.mark.gpu


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).double().numpy()


def over(got, out, size, part):
    """By how much the error is past the bound, as a part of it (below 0: within)."""
    return ((np.abs(got - out) - 2.0 ** -133) / (2.0 ** -8 * np.abs(out) + part * size) - 1.0).max()


def queries(kind, shape, gen):
    """Peaked rows: scores with a deviation of 8 to 11, so that a handful of keys hold the weight."""
    q = torch.randn(shape, generator=gen)
    return (q * 8.0 if kind == "large" else q).to(torch.bfloat16), shape[-1] ** -0.5 if kind == "large" else 1.0


def with_weights(q, k, v, see, scale, remainders):
    """The kernel's arithmetic in 64 bits with bf16 weights, with or without their remainders."""
    q, k, v = (t.double().numpy() for t in (q, k, v))
    out = np.zeros(q.shape)
    rep = q.shape[1] // k.shape[1]
    for p in range(q.shape[0]):
        at = np.nonzero(see[p])[0]
        for h in range(q.shape[1]):
            s = scale * (k[at, h // rep] @ q[p, h])
            e = np.exp(s - s.max())
            w = bf16(e)
            if remainders:
                w = w + bf16(e - w)
            out[p, h] = w @ v[at, h // rep] / e.sum()
    return bf16(out)


@pytest.mark.parametrize("kind", ["large", "unscaled"])
def test_the_bounds_tell_the_forms_apart(kind):
    """Weights without their remainders break the tighter bound and keep the
    wider one; with them they keep both."""
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn((2048, 1, 128), generator=g).to(torch.bfloat16) for _ in range(2))
    q, scale = queries(kind, (4, 8, 128), g)
    see = ref.visible(4, 2044)
    out, _, size = ref.attend(q, k, v, see, scale)
    plain, full = (with_weights(q, k, v, see, scale, r) for r in (False, True))
    assert over(plain, out, size, EXACT) > 0.2
    assert over(plain, out, size, PLAIN) < 0 and over(full, out, size, EXACT) < 0


@gpu
@pytest.mark.parametrize("kind", ["large", "unscaled"])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("w,total,H,G,D,part", [
    (8, 2048, 8, 1, 128, EXACT),        # 64 rows of 16 tiles: remainders as more rows
    (1, 2048, 8, 1, 64, EXACT), (3, 300, 28, 4, 128, EXACT),
    (20, 1152, 4, 1, 128, EXACT),       # 80 rows of 9 tiles, then 520 rows: remainders in a second product
    (130, 1152, 8, 2, 128, EXACT), (130, 700, 8, 2, 64, EXACT),
    (8, 2049, 8, 1, 128, PLAIN), (130, 1153, 8, 2, 128, PLAIN),
    (4, 2500, 8, 2, 128, PLAIN), (4, 8000, 8, 2, 64, PLAIN), (1, 40000, 8, 2, 128, PLAIN),
    (70, 5000, 8, 2, 128, PLAIN)])
def test_rows_where_few_keys_count(gpu_lib, kind, e4m3, w, total, H, G, D, part):
    from speculative_decoding_markov_gb300 import binding as sdm
    s = ref.Setup([w], [total - w], G, D, 64, e4m3, seed=total + w)
    s.write_all()
    q, scale = queries(kind, (w, H, D), s.gen)
    got = sdm.attend(s.cache, q.cuda(), s.cu, s.ctx, w, scale=scale, dev_status=s.status)["out"].double().cpu().numpy()
    out, _, size = ref.attend(q, s.held(0, "k"), s.held(0, "v"), ref.visible(w, total - w), scale)
    past = over(got, out, size, part)
    print(f"past the bound by {past:+.2f}; error {np.max(np.abs(got - out) / size) * 256:.2f} x 2^-8 size")
    assert past < 0

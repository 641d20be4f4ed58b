"""The decoding example: one token at a time, by chains and by trees over the
paged cache, to the same text."""
from __future__ import annotations

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_three_ways_to_the_same_text(gpu_lib, cache):
    spec = importlib.util.spec_from_file_location("decode_with_cache",
                                                  os.path.join(ROOT, "examples", "decode_with_cache.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    texts, steps = m.main(tokens=40, cache=cache, seed=3)
    for way in ("chain", "tree"):
        for a, b in zip(texts[way], texts["one"]):
            n = min(len(a), len(b))
            assert n > 20 and a[:n] == b[:n]
        assert steps[way] < steps["one"]       # drafts were accepted

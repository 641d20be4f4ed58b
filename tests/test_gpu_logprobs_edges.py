"""Log probabilities where they went wrong once: masked tokens of rows that
several blocks share, rows of NaN, lists of rows just too long for a rule."""
from __future__ import annotations

import pytest
import torch

from speculative_decoding_markov_gb300 import binding as sdm
from tests.test_gpu_logprobs import test_ragged_windows as ragged_windows

pytestmark = pytest.mark.gpu
INF = float("inf")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [40008, 151936])
@pytest.mark.parametrize("items", [1, 13, 150, 300, 600, 700])
def test_ranks_of_masked_tokens_in_every_share(gpu_lib, dt, V, items):
    """Tokens of -inf, which only those of -inf in front of them and the allowed
    ones come before, in each of the 8, 4 or 2 shares of a row, and in one."""
    gen = torch.Generator().manual_seed(items)
    z = torch.full((items, V), -INF)
    z[:, 5::1013] = torch.randn((items, -(-(V - 5) // 1013)), generator=gen)
    z[1::5] = -INF                                                 # rows without an allowed token
    z[2::5, V - 2] = 1.0                                           # and with one of the last
    tok = torch.randint(0, V, (1, items), generator=gen, dtype=torch.int32)
    ends = [V - 1, V - 7, V - 9, V - V // 8, V // 8 * 3 - 1, V // 2 + 8, V // 2 - 1, 0]
    for k in range(items):
        if k % 3 != 2:
            tok[0, k] = ends[k // 3 % len(ends) if items > 1 else 0]
    z, tok = z.to(dt).cuda(), tok.cuda()
    out = sdm.token_logprobs(z, i32([0, items]), tok, top=3)
    assert out["dev_status"].item() == 0
    y = tok[0].long()[:, None]
    said, ids = z.gather(1, y), torch.arange(V, device="cuda")
    rank = ((z > said) | ((z == said) & (ids < y))).sum(1).int()
    assert torch.equal(out["rank"][0], rank)
    some = (z > -INF).any(1)
    assert (out["logp"][0][some & (said[:, 0] == -INF)] == -INF).all()
    key = torch.where(z > -INF, z.float(), -1e30)
    assert torch.equal(out["top_tok"][0].long(), torch.sort(key, dim=1, descending=True, stable=True)[1][:, :3])


@pytest.mark.parametrize("dt,bits", [(torch.bfloat16, 0x7fc0), (torch.bfloat16, 0xffc0), (torch.bfloat16, 0xffff),
                                     (torch.float32, 0x7fffffff), (torch.float32, 0xffc00000), (torch.float32, 0xffffffff)])
@pytest.mark.parametrize("V", [8, 64, 1000, 5000, 40008, 151936])
def test_lists_of_rows_of_nan(gpu_lib, dt, bits, V):
    """Different tokens of the row, NaN last of all whatever their sign and payload."""
    whole, size = (torch.int16, 16) if dt is torch.bfloat16 else (torch.int32, 32)
    nan = torch.tensor([bits - (1 << size if bits >> (size - 1) else 0)]).to(whole).view(dt)
    at, gen = torch.arange(V), torch.Generator().manual_seed(V)
    a = torch.randn((V,), generator=gen).to(dt)
    rows = [torch.where(at < 0, a, nan), torch.where(at % 101 == 3, a, nan), torch.where(at == V - 1, a, nan),
            torch.where(at % 2 == 0, a, nan), torch.where(at % 3 == 0, torch.tensor(-INF, dtype=dt), nan),
            torch.where(at == V // 2, nan, a), torch.where(at < V // 2, nan, a)]
    target = torch.stack(rows).cuda()
    n = target.shape[0]
    for items in (n, 700):                                         # rows of several blocks, and of one
        z = target.repeat(-(-items // n), 1)[:items].contiguous()
        for top in (1, 6, 32):
            top = min(top, V)
            out = sdm.token_logprobs(z, i32([0, items]), i32([[0] * items]), top=top)
            assert out["dev_status"].item() == 0
            assert out["logp"].isnan().all() and out["entropy"].isnan().all()
            ids = out["top_tok"][0].cpu()
            assert (ids >= 0).all() and (ids < V).all()
            assert out["top_logp"].isnan().all()
            key = torch.where(target.isnan(), -INF, target.float())
            want = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :top].cpu()
            assert torch.equal(ids, want.repeat(-(-items // n), 1)[:items].int())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V,top", [(1800, 32), (1808, 32), (1816, 32), (1800, 30), (1032, 20), (1040, 20), (1048, 20)])
def test_lists_of_rows_whose_last_warp_has_few_elements(gpu_lib, dt, V, top):
    """As many warps have elements as the list takes, but not as many threads of
    them: the same tokens, and not many times as long as a few elements less."""
    ragged_windows(gpu_lib, dt, V, top, 1.0)

    def time(V):
        gen = torch.Generator().manual_seed(V)
        z = torch.randn((4000, V), generator=gen).to(dt).cuda()
        args = z, i32([0, 4000]), i32([[3] * 4000])
        out, st = sdm.token_logprobs(*args, top=top), sdm.new_status()
        best = INF
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            sdm.token_logprobs(*args, top=top, out=out, dev_status=st)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    # a list of every element, ranked by all pairs, takes 13 times as long
    assert time(V) < 4 * time(V // 256 * 256)

"""The weights of the paged latent attention add up to one.

The probabilities are rounded to bf16 for the product with the values, by up
to 2^-8 each.  Divided by the sum of the rounded ones, an average of equal
values is that value again: the products are exact in fp32, and the sums'
truncations (one per 16 tokens, 2^-23 each, over at most 20000 tokens) stay
below 2^-12 of it, far from the 2^-9 that would reach the next bf16.  Divided
by the sum of the unrounded ones it is off by up to 2^-8, a whole step."""

import math

import pytest
import torch

import gemm_dsnq_dual_gb300 as dsnq

pytestmark = pytest.mark.gpu
DEV = "cuda"
DK, DV, PAGE = 576, 512, 64


def equal_values(lens, H, weight, seed):
    """A cache whose rows share the value columns 1.. (bf16 numbers of either
    sign) and whose column 0, the only one that the queries see, makes
    probabilities 1 and `weight`: below 1, the first token of every 64 has
    probability 1 (in every tile, whichever way the requests are cut); above 1,
    the request's first 64 tokens (so that a row's maximum is the lower one
    when the others come)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    held = [-(-n // PAGE) for n in lens]
    cache = torch.empty(sum(held) + 2, PAGE, DK, dtype=torch.bfloat16, device=DEV)
    row = torch.randn(DK, generator=g, device=DEV) + 1.9
    cache[:] = row.to(torch.bfloat16)
    cache[:, :, 0] = -1 if weight < 1 else 1
    if weight < 1:
        cache[:, 0, 0] = 0
    table = torch.full((len(lens), max(held) + 1), -1, dtype=torch.int32, device=DEV)
    ids = torch.randperm(sum(held) + 2, generator=g, device=DEV).to(torch.int32)
    at = 0
    for b, k in enumerate(held):
        table[b, :k] = ids[at:at + k]
        if weight > 1 and k:
            cache[ids[at].long(), :, 0] = 0
        at += k
    q = torch.zeros(len(lens), H, DK, dtype=torch.bfloat16, device=DEV)
    q[:, :, 0] = 1
    lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out, lse = dsnq.paged_latent_attention(q, cache, table, lens, DV, abs(math.log(weight)))
    assert dsnq.debug_status() == 0
    return out, lse, cache[0, 0, 1:DV]


# 0.5019 and 0.2509 lie almost half a step above bf16 numbers, 129.4 (a row's
# maximum may grow by 2^8 before it is raised) likewise.
WEIGHTS = [0.5019, 0.2509, 129.4]
BATCHES = [[101], [64], [40, 700, 0, 130], [20000], [3000, 65], [500] * 70, [900, 30, 2000] * 14, [260] * 200]


@pytest.mark.parametrize("weight", WEIGHTS)
@pytest.mark.parametrize("H", [3, 16, 64, 128])
@pytest.mark.parametrize("lens", BATCHES, ids=lambda v: f"{len(v)}x{max(v)}")
def test_equal_values_come_out_as_they_are(lens, H, weight):
    out, lse, value = equal_values(lens, H, weight, seed=len(lens) + H)
    for b, n in enumerate(lens):
        if n == 0:
            assert bool((out[b] == 0).all())
            continue
        assert torch.equal(out[b, :, 1:], value.expand(H, DV - 1)), (b, n)
        # lse is of the unrounded probabilities: 2^-18 for sums and exponentials.
        ones = -(-n // 64) if weight < 1 else min(n, 64)
        want = math.log(ones + (n - ones) * weight)
        assert float((lse[b] - want).abs().max()) <= 2.0**-18 + 2.0**-21 * abs(want), (b, n)

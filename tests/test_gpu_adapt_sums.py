"""How exact the sums of gdn_in_proj_adapted are, at any length.

The tensor core cuts each sum off instead of rounding it: by half a unit of 2^-23 of it on the average.
For products of random sign and size the sum after s of S steps (K = 16) is sqrt(s / S) of the whole, so
a chain of S steps in one accumulator is off by about
    2^-24 sum_s sqrt(s / S) = 2^-24 (2/3 S + 1/2)
of what it adds up to, and so is what is joined from several such chains.  Each joining rounds once.

A float32 y: chains of 60 steps (K = 960) at most, joined in float32.

A bf16 y of up to 96 tokens: four chains.  Against the rounded exact result: a value with an error of e and a
rounding step of u falls on the neighbour with a probability of |e| / u, and is off by u then, so that the
squares add up to E[|e| u].  Normally distributed results of RMS 1 have E[u] = sum_k P(2^k <= |y| <
2^(k+1)) 2^(k-7) = 4.5e-3."""
import math

import numpy as np
import pytest
import torch

from gated_deltanet_recurrent_gb300 import abi
from oracle.adapt_oracle import adapted

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pool():
    p = abi.Pool(1, 1, 1, 1, 16, 16, 48, 4, host_checks=False)
    yield p
    p.close()


def cut_off(steps):
    return 2.0 ** -24 * (2 / 3 * steps + 0.5)


def inputs(tokens, hidden, n_out, rank, n, ids):
    gen = torch.Generator(device="cuda").manual_seed(hidden + tokens)

    def normal(*shape, by=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * by).bfloat16()
    x, w = normal(tokens, hidden), normal(n_out, hidden, by=hidden ** -0.5)
    a, b = normal(n, rank, hidden, by=hidden ** -0.5), normal(n, n_out, rank, by=0.3 * rank ** -0.5)
    want = x.double() @ w.double().T
    for i in range(n):
        rows = (ids == i).nonzero()[:, 0]
        want[rows] += (x[rows].double() @ a[i].double().T) @ b[i].double().T
    return x, w, abi.Adapters(a, b), want


def off(y, want):
    return float((y.double() - want).norm() / want.norm())


# one tile for a block, a tile shared by several, wider tiles, and pairs of blocks
CALLS = [(1, 5120), (64, 12352), (64, 2048), (256, 5120), (96, 12352), (2049, 1024)]


@pytest.mark.parametrize("tokens,n_out", CALLS)
@pytest.mark.parametrize("hidden", [512, 960, 2048, 8192, 16384, 32768])
@pytest.mark.parametrize("pattern", ["none", "one", "three", "own"])
def test_float32_sums_of_any_length(pool, tokens, n_out, hidden, pattern):
    if pattern in ("three", "own") and hidden not in (2048, 16384, 32768):
        return
    n = 12
    t = torch.arange(tokens, device="cuda", dtype=torch.int32)
    ids = {"none": t * 0 - 1, "one": t * 0 + 5, "three": t % 4 - 1, "own": t % n}[pattern]
    x, w, ad, want = inputs(tokens, hidden, n_out, 40, n, ids)
    y = torch.empty(tokens, n_out, device="cuda")
    abi.gdn_in_proj_adapted(pool, ad, x, w, ids, y)
    # (the low side: a sum over hidden as well, mma.sync's in eight chains, of 0.3 of the whole)
    low = 0 if pattern == "none" else 0.3 * (cut_off(hidden / 16 / 8) + 10 * 2.0 ** -24)
    assert off(y, want) <= cut_off(60) + (hidden / 960 + 10) * 2.0 ** -24 + low
    assert abi.gdn_pool_get_error(pool) == 0


@pytest.mark.parametrize("tokens,n_out", [(1, 12352), (64, 12352), (64, 2048), (256, 5120), (96, 12352)])
def test_bf16_roundings_of_few_tokens_are_those_of_the_exact_sum(pool, tokens, n_out):
    hidden = 2048
    ids = torch.full((tokens,), -1, dtype=torch.int32, device="cuda")
    x, w, ad, want = inputs(tokens, hidden, n_out, 16, 2, ids)
    y = torch.empty(tokens, n_out, device="cuda", dtype=torch.bfloat16)
    abi.gdn_in_proj_adapted(pool, ad, x, w, ids, y)
    assert off(y, want.bfloat16().double()) <= math.sqrt(4.5e-3 * cut_off(hidden / 16 / 4))


@pytest.mark.parametrize("tokens", [3, 64, 200, 2100])
@pytest.mark.parametrize("pattern", ["one", "two", "own"])
def test_the_low_side_of_a_float32_result_keeps_24_bits(pool, tokens, pattern):
    """Sums A x of up to 2^22 whole numbers, of which two bf16 parts hold 16 or 17 bits; everything is
    exact: |w| <= 1 and x <= 32 over 2048 are 2^16 at most, and 3 B (A x) of 2^22 stay below 2^24."""
    hidden, n_out, rank, n = 2048, 264, 3, 20
    rng = np.random.default_rng(tokens)
    x = rng.integers(0, 33, (tokens, hidden)).astype(np.float64)
    a = rng.integers(0, 65, (n, rank, hidden)).astype(np.float64)
    w = rng.integers(-1, 2, (n_out, hidden)).astype(np.float64)
    b = rng.integers(-1, 2, (n, n_out, rank)).astype(np.float64)
    ids = {"one": [4] * tokens, "two": [t % 2 for t in range(tokens)],
           "own": [t % n for t in range(tokens)]}[pattern]
    bf = lambda v: torch.from_numpy(v).float().cuda().bfloat16()
    want, _, _ = adapted(x, w, a, b, np.ones(n), ids)
    h = torch.from_numpy((x[0] @ a[ids[0]].T)).float()
    rest = h - h.bfloat16().float()
    assert (rest - rest.bfloat16().float()).abs().max() >= 1, "no third part"
    assert np.abs(want).max() < 2 ** 24 and h.max() <= 2 ** 22
    wide = torch.zeros(n, n_out, 8, device="cuda", dtype=torch.bfloat16)
    wide[:, :, :rank] = bf(b)
    y = torch.empty(tokens, n_out, device="cuda")
    abi.gdn_in_proj_adapted(pool, abi.Adapters(bf(a), wide[:, :, :rank]), bf(x), bf(w),
                            torch.tensor(ids, dtype=torch.int32, device="cuda"), y)
    assert np.array_equal(y.double().cpu().numpy(), want)

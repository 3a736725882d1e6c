"""An adapter that is NaN all over, in calls of many tokens: it spoils its own tokens only, and does not stop
the others' either.

Small whole numbers (|x|, |w|, |a| <= 2, |b| <= 3): every sum is exact, and the result is the oracle's bit
for bit."""
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


def bf(x):
    return torch.from_numpy(np.asarray(x, np.float32)).cuda().bfloat16()


def whole(rng, most, *shape):
    return rng.integers(-most, most + 1, shape).astype(np.float64)


def i32(x):
    return torch.tensor([int(v) for v in x], dtype=torch.int32, device="cuda")


def padded(x):
    """Rows with a stride of a multiple of 8 elements, and NaN behind each."""
    t = torch.full((*x.shape[:-1], -(-x.shape[-1] // 8) * 8 + 8), math.nan, device="cuda")
    t[..., :x.shape[-1]] = torch.from_numpy(np.asarray(x, np.float32))
    return t.bfloat16()[..., :x.shape[-1]]


def microseconds(call):
    call()
    best = math.inf
    for _ in range(4):
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        call()
        end.record()
        torch.cuda.synchronize()
        best = min(best, begin.elapsed_time(end) * 1e3)
    return best


@pytest.mark.parametrize("tokens,hidden,n_out,rank", [
    (5000, 256, 1296, 32), (2100, 2048, 1024, 16), (2049, 2048, 648, 128), (2300, 1000, 1032, 24),
    (2055, 100, 200, 5), (2049, 8, 264, 1), (600, 4096, 25600, 64)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pattern", ["own", "runs", "two"])
def test_one_adapter_that_is_nan_all_over(pool, tokens, hidden, n_out, rank, dtype, pattern):
    if tokens == 600 and pattern != "own":
        return
    rng = np.random.default_rng(tokens + hidden)
    n, bad = 8, 3
    w, x = whole(rng, 2, n_out, hidden), whole(rng, 2, tokens, hidden)
    a, b = whole(rng, 2, n, rank, hidden), whole(rng, 3, n, n_out, rank)
    scale = np.ones(n)
    t = np.arange(tokens)
    ids = {"own": t % (n + 1) - 1, "runs": t // 50 % n, "two": np.where(t % 7 == 0, bad, -1)}[pattern]
    want, _, _ = adapted(x, w, a, b, scale, np.where(ids == bad, -1, ids))
    nan = b.copy()
    nan[bad] = math.nan
    gx, gw, gids = padded(x), padded(w), i32(ids)
    y = torch.full((tokens, -(-n_out // 8) * 8), 77.0, dtype=dtype, device="cuda")[:, :n_out]
    times = []
    for high in (b, nan):
        ad = abi.Adapters(padded(a), padded(high))
        times.append(microseconds(lambda: abi.gdn_in_proj_adapted(pool, ad, gx, gw, gids, y)))
    assert abi.gdn_pool_get_error(pool) == 0
    good = ids != bad
    got = y.double().cpu().numpy()
    assert np.array_equal(got[good], torch.from_numpy(want[good]).to(dtype).double().numpy())
    assert np.isnan(got[~good]).all()
    # with all results of a tile computed again, the tile takes some ten times as long
    assert times[1] <= 25 * times[0] + 100, times


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_one_element_that_is_infinite(pool, dtype):
    """One output row of one adapter: every token's result in that row is computed again, with real
    numbers, and is as exact as it was."""
    tokens, hidden, n_out, rank, n = 2200, 2048, 520, 40, 5
    gen = torch.Generator(device="cuda").manual_seed(1)
    real = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()
    x, w, a, b = real(tokens, hidden), real(n_out, hidden), real(n, rank, hidden) / 8, real(n, n_out, rank)
    ids = i32(np.arange(tokens) % n)
    y, z = (torch.empty(tokens, n_out, dtype=dtype, device="cuda") for _ in range(2))
    abi.gdn_in_proj_adapted(pool, abi.Adapters(a, b), x, w, ids, y)
    b[2, 333, 39] = math.inf
    abi.gdn_in_proj_adapted(pool, abi.Adapters(a, b), x, w, ids, z)
    own = ids == 2
    assert not torch.isfinite(z[own, 333]).any()
    z[own, 333] = y[own, 333]
    same = torch.ones(n_out, dtype=torch.bool, device="cuda")
    same[333] = False
    assert torch.equal(y[:, same], z[:, same])
    # two float32 sums of 2048 products and 2 * 40 of the low side in short chains: 2^-23 of the
    # magnitudes a step of 16, in any order, each; and the bf16 rounding
    size = x.double().abs() @ w[333].double().abs() + 1
    for i in range(n):
        low = (x[ids == i].double().abs() @ a[i].double().abs().T) @ b[i, 333].double().abs().nan_to_num(posinf=0)
        size[ids == i] += 2 * low
    off = 2 * (2048 + 160) / 16 * 2.0 ** -23 * size
    if dtype == torch.bfloat16:
        off += 2.0 ** -7 * y[:, 333].double().abs()
    assert ((y[:, 333].double() - z[:, 333].double()).abs() <= off).all()
    assert abi.gdn_pool_get_error(pool) == 0

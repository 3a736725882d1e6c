"""The input projection with a low-rank adapter per token (gdn_in_proj_adapted).

Most tests use small whole numbers, for which every sum is exact in float32 and the low side fits
its bf16 parts: |x|, |w|, |a| <= 2 and |b| <= 3, so that |a x| <= 4 hidden < 2^16 and all sums stay
below 2^24 (in halves, where a scale is 1/2).  The result is then the oracle's, bit for bit, and in
bf16 its rounding.

With real numbers, a float32 sum of n products in any order is off by at most n 2^-24 of the
sum of magnitudes (a tensor core that cuts terms off instead of rounding them: twice that); the low
side is rounded to 2^-16 of itself (bf16 y) or 2^-24 (float32 y)."""
import math
import random

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


def whole(rng, most, *shape):
    return rng.integers(-most, most + 1, shape).astype(np.float64)


def bf(x):
    return torch.from_numpy(np.asarray(x, np.float32)).cuda().to(torch.bfloat16)


def i32(x):
    return torch.tensor([int(v) for v in x], dtype=torch.int32, device="cuda")


def make(rng, hidden, n_out, rank, n):
    w, a, b = whole(rng, 2, n_out, hidden), whole(rng, 2, n, rank, hidden), whole(
        rng, 3, n, n_out, rank)
    scale = rng.choice([0.5, 1.0, 2.0, -1.0], n)
    return w, a, b, scale


def device_rows(x):
    """bf16 rows with a stride of a multiple of 8 elements, and NaN behind each row."""
    x = np.asarray(x, np.float32)
    width = x.shape[-1]
    ld = -(-width // 8) * 8 + 8
    t = torch.full((*x.shape[:-1], ld), math.nan, dtype=torch.bfloat16, device="cuda")
    t[..., :width] = bf(x)
    return t[..., :width]


def same(y, want):
    if y.dtype == torch.bfloat16:
        want = torch.from_numpy(want).to(torch.bfloat16).double().numpy()
    assert np.array_equal(y.double().cpu().numpy(), want)


def patterns(tokens, n, seed=0):
    """Ways in which a batch's tokens may have adapters."""
    rnd = random.Random(seed + tokens)
    runs = []
    while len(runs) < tokens:
        runs += [rnd.randrange(-1, n)] * rnd.randint(1, max(1, tokens // 3))
    return {"none": [-1] * tokens, "one": [n - 1] * tokens,
            "own": [t % n for t in range(tokens)],
            "some": [rnd.randrange(-1, n) for _ in range(tokens)], "runs": runs[:tokens]}


SHAPES = [(256, 384, 16), (64, 128, 8), (2048, 2048, 64), (512, 1040, 32), (72, 40, 24),
          (1000, 136, 128), (8, 8, 1), (200, 264, 40), (100, 24, 5), (128, 130, 72)]


@pytest.mark.parametrize("hidden,n_out,rank", SHAPES)
@pytest.mark.parametrize("tokens", [1, 2, 3, 4, 5, 17, 64, 100, 129, 300])
def test_whole_numbers(pool, hidden, n_out, rank, tokens):
    rng = np.random.default_rng(hidden + rank + tokens)
    n = 5 if tokens < 100 else 37
    w, a, b, scale = make(rng, hidden, n_out, rank, n)
    x = whole(rng, 2, tokens, hidden)
    ad = abi.Adapters(device_rows(a), device_rows(b),
                      torch.tensor(scale, dtype=torch.float32, device="cuda"))
    gx, gw = device_rows(x), device_rows(w)
    for name, ids in patterns(tokens, n).items():
        want, _, _ = adapted(x, w, a, b, scale, ids)
        for dtype in (torch.float32, torch.bfloat16):
            ld = -(-n_out // 8) * 8 + 8
            store = torch.full((tokens + 1, ld), 77.0, dtype=dtype, device="cuda")
            abi.gdn_in_proj_adapted(pool, ad, gx, gw, i32(ids), store[:tokens, :n_out])
            same(store[:tokens, :n_out], want)
            assert (store[tokens] == 77).all() and (store[:, n_out:] == 77).all(), name
    assert abi.gdn_pool_get_error(pool) == 0


@pytest.mark.parametrize("hidden,n_out,rank", [
    (2048, 12352, 16), (512, 10000, 64), (512, 10000, 128), (192, 24576, 32), (256, 130, 48)])
@pytest.mark.parametrize("tokens", [65, 96, 97, 192, 260, 2048, 2049])
def test_tiles_that_fill_the_device_more_than_once(pool, tokens, hidden, n_out, rank):
    """Where wider tiles of tokens, and then pairs of blocks, take over."""
    rng = np.random.default_rng(tokens + n_out)
    n = 70
    w, a, b, scale = make(rng, hidden, n_out, rank, n)
    x = whole(rng, 2, tokens, hidden)
    ad = abi.Adapters(bf(a), bf(b), torch.tensor(scale, dtype=torch.float32, device="cuda"))
    gx, gw = bf(x), bf(w)
    for name, ids in patterns(tokens, n).items():
        if tokens * n_out > 4e6 and name not in ("some", "runs"):
            continue
        want, _, _ = adapted(x, w, a, b, scale, ids)
        for dtype in (torch.float32, torch.bfloat16):
            y = torch.full((tokens + 1, -(-n_out // 8) * 8), 77.0, dtype=dtype, device="cuda")
            abi.gdn_in_proj_adapted(pool, ad, gx, gw, i32(ids), y[:tokens, :n_out])
            same(y[:tokens, :n_out], want)
            assert (y[tokens] == 77).all(), name
    assert abi.gdn_pool_get_error(pool) == 0


@pytest.mark.parametrize("tokens,hidden,n_out,rank,n", [
    (1500, 512, 1040, 64, 200), (4097, 256, 640, 16, 9), (777, 2048, 5120, 32, 24),
    (2500, 192, 12352, 128, 3), (16384, 128, 2560, 24, 40)])
def test_whole_numbers_of_many_tokens(pool, tokens, hidden, n_out, rank, n):
    rng = np.random.default_rng(tokens)
    w, a, b, scale = make(rng, hidden, n_out, rank, n)
    x = whole(rng, 2, tokens, hidden)
    ad = abi.Adapters(bf(a), bf(b), torch.tensor(scale, dtype=torch.float32, device="cuda"))
    for name, ids in patterns(tokens, n).items():
        want, _, _ = adapted(x, w, a, b, scale, ids)
        for dtype in (torch.float32, torch.bfloat16):
            y = torch.full((tokens, n_out), 77.0, dtype=dtype, device="cuda")
            abi.gdn_in_proj_adapted(pool, ad, bf(x), bf(w), i32(ids), y)
            same(y, want)
    assert abi.gdn_pool_get_error(pool) == 0


@pytest.mark.parametrize("n_out", [5120, 6400, 2600, 1000])
@pytest.mark.parametrize("tokens", [1, 33, 64])
def test_tiles_that_several_blocks_share(pool, tokens, n_out):
    """Long sums and few outputs: a tile is split over 3 or 4 blocks."""
    hidden, rank, n = 2048, 64, 12
    rng = np.random.default_rng(n_out + tokens)
    w, a, b, scale = make(rng, hidden, n_out, rank, n)
    x = whole(rng, 2, tokens, hidden)
    ad = abi.Adapters(bf(a), bf(b), torch.tensor(scale, dtype=torch.float32, device="cuda"))
    gx, gw = bf(x), bf(w)
    for name, ids in patterns(tokens, n).items():
        want, _, _ = adapted(x, w, a, b, scale, ids)
        for dtype in (torch.float32, torch.bfloat16):
            y = torch.full((tokens, n_out), 77.0, dtype=dtype, device="cuda")
            abi.gdn_in_proj_adapted(pool, ad, gx, gw, i32(ids), y)
            same(y, want)
    assert abi.gdn_pool_get_error(pool) == 0


def test_the_most_tokens(pool):
    """2^18 tokens with runs, mixed tiles and scattered adapters among them."""
    tokens, hidden, n_out, rank, n = 1 << 18, 64, 72, 16, 300
    rng = np.random.default_rng(11)
    w, a, b, scale = make(rng, hidden, n_out, rank, n)
    x = whole(rng, 2, tokens, hidden)
    ids = np.arange(tokens) // 700 % n
    ids[5000:6000] = rng.integers(-1, n, 1000)
    ids[-3:] = [7, -1, 299]
    ad = abi.Adapters(bf(a), bf(b), torch.tensor(scale, dtype=torch.float32, device="cuda"))
    want, _, _ = adapted(x, w, a, b, scale, ids)
    for dtype in (torch.float32, torch.bfloat16):
        y = torch.full((tokens, n_out), 77.0, dtype=dtype, device="cuda")
        abi.gdn_in_proj_adapted(pool, ad, bf(x), bf(w), i32(ids), y)
        same(y, want)
    assert abi.gdn_pool_get_error(pool) == 0
    with pytest.raises(abi.GDNError) as e:
        abi.gdn_in_proj_adapted(pool, ad, torch.empty(tokens + 1, 64, device="cuda").bfloat16(), bf(w),
                                i32([-1] * (tokens + 1)))
    assert e.value.name == "GDN_ERR_SIZE"


@pytest.mark.parametrize("tokens", [1, 40, 600, 4000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_real_numbers(pool, tokens, dtype):
    hidden, n_out, rank, n = 1024, 768, 48, 11
    rng = np.random.default_rng(tokens)
    real = lambda *s: bf(rng.standard_normal(s))
    x, w, a, b = real(tokens, hidden), real(n_out, hidden), real(n, rank, hidden), real(n, n_out, rank)
    scale = torch.rand(n, device="cuda") + 0.1
    host = lambda t: t.double().cpu().numpy()
    ad = abi.Adapters(a, b, scale)
    for ids in patterns(tokens, n).values():
        want, size, low = adapted(host(x), host(w), host(a), host(b), host(scale), ids)
        y = torch.empty(tokens, n_out, dtype=dtype, device="cuda")
        abi.gdn_in_proj_adapted(pool, ad, x, w, i32(ids), y)
        # one sum of hidden + 3 rank terms; the low side's own sum of hidden, its scale, its parts
        step = 2.0 ** -23
        off = (hidden + 3 * rank) * step * (size + low) + (hidden + 1) * step * low
        off = off + (2.0 ** -16 if dtype == torch.bfloat16 else 2.0 ** -24) * low
        if dtype == torch.bfloat16:
            off = off + 2.0 ** -8 * np.abs(want)
        assert (np.abs(host(y) - want) <= off).all()
        # and on the whole: the roundings of random sign of these sums are far below their bound
        rel = np.sqrt(np.mean((host(y) - want) ** 2) / np.mean(want ** 2))
        assert rel <= (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -18)


@pytest.mark.parametrize("tokens,n", [(1, 8), (3, 8), (4, 8), (5, 8), (64, 8), (200, 8), (5000, 8), (600, 8), (600, 40)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_adapters_that_are_not_finite_spoil_their_own_tokens_only(pool, tokens, n, dtype):
    hidden, n_out, rank = 256, 1300 // 8 * 8, 32
    rng = np.random.default_rng(3)
    w, a, b, scale = make(rng, hidden, n_out, rank, n)
    x = whole(rng, 2, tokens, hidden)
    x[-1, 5] = math.inf
    a[1, 3, 7], a[2, 0, 0] = math.nan, math.inf
    b[3, 9, 31], b[4, :, 2], b[5, n_out - 1, 0] = math.inf, math.nan, -math.inf
    scale[6] = math.inf
    for ids in patterns(tokens, n).values():
        ids = list(ids)
        ids[0] = 3
        with np.errstate(invalid="ignore"):
            want, _, _ = adapted(x, w, a, b, scale, ids)
        y = torch.empty(tokens, n_out, dtype=dtype, device="cuda")
        ad = abi.Adapters(bf(a), bf(b), torch.tensor(scale, dtype=torch.float32, device="cuda"))
        abi.gdn_in_proj_adapted(pool, ad, bf(x), bf(w), i32(ids), y)
        y = y.double().cpu().numpy()
        good = np.isfinite(want)
        assert good[:-1].any() or tokens == 1
        want = torch.from_numpy(want).to(dtype).double().numpy()
        assert np.array_equal(y[good], want[good])
        assert not np.isfinite(y[~good]).any()


def test_ids_out_of_range_get_no_adapter(pool):
    rng = np.random.default_rng(4)
    w, a, b, scale = make(rng, 128, 256, 16, 3)
    x = whole(rng, 2, 70, 128)
    ids = [3, -2, 2 ** 31 - 1, -2 ** 31] + [0, 1, -1, 2] * 16 + [2, 7]
    ad = abi.Adapters(bf(a), bf(b), torch.tensor(scale, dtype=torch.float32, device="cuda"))
    y = abi.gdn_in_proj_adapted(pool, ad, bf(x), bf(w), i32(ids))
    same(y, adapted(x, w, a, b, scale, ids)[0])
    assert abi.gdn_pool_get_error(pool) == abi.DEVERR_ADAPTER
    strict = abi.Adapters(ad.a, ad.b, ad.scale, host_checks=True)
    with pytest.raises(abi.GDNError) as e:
        abi.gdn_in_proj_adapted(pool, strict, bf(x), bf(w), i32(ids))
    assert e.value.name == "GDN_ERR_SIZE"


def test_without_adapters_it_is_the_projection(pool):
    """Tokens without an adapter: what gdn_in_proj gives, up to the order of the sum."""
    x, w = torch.randn(90, 512, device="cuda").bfloat16(), torch.randn(300, 512, device="cuda")
    w = (w / 512 ** 0.5).bfloat16()[:296]
    ad = abi.Adapters(torch.zeros(1, 8, 512, device="cuda").bfloat16(),
                      torch.zeros(1, 296, 8, device="cuda").bfloat16())
    got = abi.gdn_in_proj_adapted(pool, ad, x, w, i32([-1] * 90))
    want = abi.gdn_in_proj(pool, x, w)
    size = x.double().abs() @ w.double().abs().T
    assert ((got - want).abs().double() <= 512 * 2.0 ** -22 * size).all()


def test_empty_calls(pool):
    ad = abi.Adapters(bf(np.zeros((2, 8, 64))), bf(np.zeros((2, 128, 8))))
    y = abi.gdn_in_proj_adapted(pool, ad, bf(np.zeros((0, 64))), bf(np.zeros((128, 64))), i32([]))
    assert y.shape == (0, 128)


@pytest.mark.parametrize("tokens", [5, 900])
def test_two_captured_graphs_and_an_eager_call_at_once(pool, tokens):
    """Workspaces are not shared between graphs, streams and eager calls."""
    rng = np.random.default_rng(tokens)
    w, a, b, scale = make(rng, 256, 512, 16, 6)
    ad = abi.Adapters(bf(a), bf(b), torch.tensor(scale, dtype=torch.float32, device="cuda"))
    gw = bf(w)
    runs = []
    for i in range(3):
        x, ids = whole(rng, 2, tokens, 256), [rng.integers(-1, 6) for _ in range(tokens)]
        runs.append((bf(x), i32(ids), torch.empty(tokens, 512, device="cuda"),
                     adapted(x, w, a, b, scale, ids)[0], torch.cuda.Stream()))
    abi.gdn_in_proj_adapted(pool, ad, runs[0][0], gw, runs[0][1], runs[0][2])
    graphs = []
    for x, ids, y, _, s in runs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            abi.gdn_in_proj_adapted(pool, ad, x, gw, ids, y)
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(5):
        for r in runs:
            r[2].zero_()
        torch.cuda.synchronize()
        for g, r in zip(graphs, runs):
            with torch.cuda.stream(r[4]):
                g.replay()
        x, ids, y, _, s = runs[2]
        abi.gdn_in_proj_adapted(pool, ad, x, gw, ids, y, stream=s)
        torch.cuda.synchronize()
        for r in runs:
            same(r[2], r[3])


def test_rewritten_adapters_are_seen(pool):
    rng = np.random.default_rng(8)
    w, a, b, scale = make(rng, 128, 256, 16, 2)
    x, ids = whole(rng, 2, 20, 128), [t % 2 for t in range(20)]
    ad = abi.Adapters(bf(a), bf(b), torch.tensor(scale, dtype=torch.float32, device="cuda"))
    same(abi.gdn_in_proj_adapted(pool, ad, bf(x), bf(w), i32(ids)),
         adapted(x, w, a, b, scale, ids)[0])
    a2, b2 = whole(rng, 2, *a.shape), whole(rng, 3, *b.shape)
    ad.a.copy_(bf(a2)), ad.b.copy_(bf(b2))
    same(abi.gdn_in_proj_adapted(pool, ad, bf(x), bf(w), i32(ids)),
         adapted(x, w, a2, b2, scale, ids)[0])

"""The bounded waits of gdn_in_proj_adapted, made to run out without a fault: two test hooks give a CTA of every
other tile (or pair of CTAs) a barrier that waits for more than it gets.  Those tiles of y keep what they
held, GDN_DEVERR_TIMEOUT says so, all others are right, and with the hook cleared the same call on
the same handle is right again.  Whole numbers: every result is the oracle's, bit for bit."""
import numpy as np
import pytest
import torch

from gated_deltanet_recurrent_gb300 import abi
from oracle.adapt_oracle import adapted

pytestmark = pytest.mark.gpu
KEPT = 77.0


def whole(rng, most, *shape):
    return rng.integers(-most, most + 1, shape).astype(np.float64)


def bf(x):
    return torch.from_numpy(np.asarray(x, np.float32)).cuda().bfloat16()


def run(tokens, hidden, n_out, rank, pattern, flag, dtype, lost):
    """lost [tokens, n_out]: what the hook's CTAs would have written."""
    rng = np.random.default_rng(tokens + hidden)
    n = 6
    w, x = whole(rng, 1, n_out, hidden), whole(rng, 1, tokens, hidden)
    a, b = whole(rng, 1, n, rank, hidden), whole(rng, 1, n, n_out, rank)
    ids = np.arange(tokens) % n if pattern == "own" else np.full(tokens, 2 if pattern == "one" else -1)
    want, _, _ = adapted(x, w, a, b, np.ones(n), ids)
    want = torch.from_numpy(want).to(dtype).double()
    pool = abi.Pool(1, 1, 1, 1, 16, 16, 48, 4, host_checks=False)
    ad = abi.Adapters(bf(a), bf(b))
    gx, gw, gids = bf(x), bf(w), torch.tensor(ids, dtype=torch.int32, device="cuda")

    def call():
        y = torch.full((tokens, n_out), KEPT + 0.5, dtype=dtype, device="cuda")
        abi.gdn_in_proj_adapted(pool, ad, gx, gw, gids, y)
        return y.double().cpu(), abi.gdn_pool_get_error(pool)
    kept = torch.full_like(want, KEPT + 0.5).to(dtype).double()
    abi.gdn_pool_set_test_flags(pool, flag)
    y, err = call()
    assert err == abi.DEVERR_TIMEOUT
    lost = torch.from_numpy(lost)
    assert torch.equal(y[lost], kept[lost])
    assert torch.equal(y[~lost], want[~lost])
    abi.gdn_pool_set_test_flags(pool, 0)
    for _ in range(2):
        y, err = call()
        assert err == 0 and torch.equal(y, want)
    ad.close()
    pool.close()


def tiles(tokens, n_out, bt, bn):
    """Numbers of the tiles, of tokens and of outputs, that each result is in."""
    return np.arange(tokens)[:, None] // bt, np.arange(n_out)[None] // bn


@pytest.mark.parametrize("tokens,bt,hidden,n_out,rank", [
    (5, 16, 2048, 640, 16), (64, 64, 2048, 1040, 64),          # tiles that several CTAs share
    (5, 16, 192, 640, 16), (60, 64, 128, 1040, 128), (130, 64, 64, 264, 24),
    (96, 96, 256, 12352, 32), (64, 64, 8256, 10000, 16)])        # (the last: several rounds of sums)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pattern,flag", [
    ("none", abi.TEST_ADAPT_WAIT_TIMEOUT), ("one", abi.TEST_ADAPT_WAIT_TIMEOUT),
    ("own", abi.TEST_ADAPT_WAIT_TIMEOUT), ("own", abi.TEST_ADAPT_SIDE_TIMEOUT)])
def test_few_tokens(tokens, bt, hidden, n_out, rank, dtype, pattern, flag):
    t, n = tiles(tokens, n_out, bt, 128)
    run(tokens, hidden, n_out, rank, pattern, flag, dtype, (t + n) % 2 == 1)


@pytest.mark.parametrize("tokens,hidden,n_out,rank", [
    (2049, 256, 1040, 16), (2100, 64, 264, 40), (5000, 512, 2048, 128), (2300, 4096, 520, 8)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pattern", ["none", "one", "own"])
@pytest.mark.parametrize("flag", [abi.TEST_ADAPT_WAIT_TIMEOUT, abi.TEST_ADAPT_SIDE_TIMEOUT])
def test_many_tokens(tokens, hidden, n_out, rank, dtype, pattern, flag):
    bt = 128 if dtype == torch.float32 else 256
    t, n = tiles(tokens, n_out, bt, 256)
    n_tiles, t_tiles = -(-n_out // 256), -(-tokens // bt)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    pairs = min(n_tiles * t_tiles, sms // 2)
    run(tokens, hidden, n_out, rank, pattern, flag, dtype, (t * n_tiles + n) % pairs % 2 == 1)


def test_other_flags_are_refused():
    pool = abi.Pool(1, 1, 1, 1, 16, 16, 48, 4, host_checks=False)
    for flags in (16, 2 | abi.TEST_ADAPT_WAIT_TIMEOUT):
        with pytest.raises(abi.GDNError) as e:
            abi.gdn_pool_set_test_flags(pool, flags)
        assert e.value.name == "GDN_ERR_ARG"
    pool.close()

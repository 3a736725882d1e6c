"""What the 8 bits cost against the values that were appended: the bounds that
include/gdn.h states, on the oracle (which append equals bit for bit)."""
import numpy as np
import pytest

from oracle.kv_oracle import KVOracle, attend_values


def cache(code, page, d, length, x, v, pieces):
    o = KVOracle(1, length // page, x.shape[1], page, d, code, np.arange(length // page)[None])
    for p in range(0, length, pieces):
        o.append(0, [0], [p], [pieces], x[p:p + pieces], v[p:p + pieces])
    return o


@pytest.mark.parametrize("page,pieces", [(16, 128), (16, 1), (128, 128), (128, 1), (32, 8)])
@pytest.mark.parametrize("code", ["i8", "e4m3"])
def test_values_are_within_the_stated_bounds(code, page, pieces):
    """At once: half a scale (int8), 2^-4 of the value or 2^-10 scales (e4m3).
    A page that grows: each larger scale rounds again, which at most doubles the
    bound (a halving series)."""
    rng = np.random.default_rng(page + pieces)
    length, d = 256, 64
    gain = np.ones(d)
    gain[::29] = 6.0
    x = rng.standard_normal((length, 2, d)) * gain * np.exp2(rng.uniform(-3, 3, (length, 1, 1)))
    o = cache(code, page, d, length, x, x, pieces)
    err = np.abs(o.values(0, 0, "k", 0, length) - x)
    pages = np.arange(length) // page
    s = o.scale["k"][0, pages][:, :, None]
    amax = np.abs(x).reshape(-1, page, 2, d).max((1, 3))[pages][:, :, None]
    assert (s <= 2 * amax / (127 if code == "i8" else 448)).all()
    twice = 1 if pieces >= page else 2
    bound = s / 2 if code == "i8" else np.maximum(np.abs(x) * 2.0 ** -4, s * 2.0 ** -10)
    assert (err <= twice * bound).all()


def test_which_code_for_which_keys():
    """Without channels that are much larger than the others int8 is the closer
    one; with them its step is theirs, and e4m3 keeps its precision."""
    rng = np.random.default_rng(0)
    length, d = 512, 128
    got = {}
    for outlier in (1, 6):
        gain = np.ones(d)
        gain[::29] = outlier
        k = rng.standard_normal((length, 2, d)) * gain
        v = rng.standard_normal((length, 2, d)) * 0.5
        q = rng.standard_normal((32, 8, d)) * 1.5 / gain
        want, _ = attend_values(q, k, v, d ** -0.5)
        for code in ("i8", "e4m3"):
            o = cache(code, 16, d, length, k, v, length)
            x, _ = o.attend(0, [0], [length], [32], q, d ** -0.5)
            got[outlier, code] = np.linalg.norm(x - want) / np.linalg.norm(want)
    assert got[1, "i8"] < got[1, "e4m3"] < got[6, "i8"]
    assert abs(got[6, "e4m3"] - got[1, "e4m3"]) < 0.2 * got[1, "e4m3"]

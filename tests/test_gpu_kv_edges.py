"""gdn_kv_attend at the edges of its range: value scales far apart, queries of
the largest magnitudes.  Tolerances are those of test_gpu_kv_attend.py."""
import numpy as np
import pytest
import torch

from gated_deltanet_recurrent_gb300 import abi, synth
from tests.gpu_util import dev, dev_i32, host, tdtype
from tests.test_gpu_kv_attend import assert_close, queries, run
from tests.test_gpu_kv_cache import append, cum, make, rows

pytestmark = pytest.mark.gpu

# (h_q, h_kv, d, query tokens a slot): what chooses each form of the tensor-core kernel, given
# calls of that many tokens and a long enough context
FORMS = [(16, 2, 256, 40), (16, 2, 256, 9), (32, 8, 128, 80), (32, 8, 128, 40), (32, 8, 128, 20),
         (12, 4, 64, 80), (12, 4, 64, 20)]
SPLIT = [(16, 2, 256, 1), (32, 8, 128, 1), (12, 4, 64, 1), (40, 1, 64, 1), (16, 2, 256, 2)]


def padded(kv, slots, kv_lens, lens, q, o_dtype, scale, hint):
    """The call with rows after the last sequence's, so that a bound of `hint` tokens holds a
    bound that large; those rows keep what they held."""
    n = len(q)
    wide = torch.zeros(max(n, hint), *q.shape[1:], device="cuda", dtype=torch.bfloat16)
    wide[:n] = dev(q, "bf16")
    o = torch.full(wide.shape, 7.0, device="cuda", dtype=tdtype(o_dtype))
    abi.gdn_kv_attend(kv, 0, dev_i32(slots), dev_i32(kv_lens), wide, o, cu_seqlens=cum(lens),
                      max_seqlen=hint, max_kv_len=200000, scale=scale)
    assert (o[n:] == 7).all()
    return o[:n]


def call(kv, slots, kv_lens, lens, q, q_dtype, scale, tensor_core):
    if tensor_core:
        return padded(kv, slots, kv_lens, lens, q, "f32", scale, max(lens))
    return run(kv, 0, slots, kv_lens, lens, q, q_dtype, "f32", scale)


SIDES = [(s, "bf16", False) for s in SPLIT] + [(s, "f32", False) for s in SPLIT] + \
    [((16, 2, 256, 40), "f32", False), ((12, 4, 64, 40), "f32", False)] + \
    [(s, "bf16", True) for s in FORMS]


@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("shape,q_dtype,tensor_core", SIDES)
def test_value_pages_of_zeros_beside_values_of_any_size(code, shape, q_dtype, tensor_core):
    """All-zero value pages count in the denominator whatever the other pages
    hold.  Equal scores: the output is the plain mean of the values."""
    h_q, h_kv, d, n = shape
    rng = np.random.default_rng(d + n)
    q = queries(rng, n, h_q, d, q_dtype)
    for length in (32, 96, 1500):
        for big in (30, 40, 64, 110):
            for first in (True, False):
                kv, ref = make(code, 16, h_kv, d, 1, -(-length // 16), h_q=h_q, seed=big)
                k = np.zeros((length, h_kv, d), dtype=np.float32)
                v = rows(rng, length, h_kv, d, "bf16", 0)
                v *= np.float32(2.0) ** big
                half = length // 32 * 16
                v[:half] *= not first
                v[half:] *= first
                append(kv, ref, 0, [0], [0], [length], k, v, "bf16")
                want, mag = ref.attend(0, [0], [length], [n], q, 0.25)
                got = call(kv, [0], [length], [n], q, q_dtype, 0.25, tensor_core)
                assert_close(got, want, mag, q_dtype, "f32", (length, big, first))


@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("shape,q_dtype,tensor_core", SIDES)
def test_value_scales_of_the_whole_range(code, shape, q_dtype, tensor_core):
    """Pages of tiny values beside pages of huge ones, in any order, at equal
    scores and with the tiny ones' scores far above; and nothing but tiny ones."""
    h_q, h_kv, d, n = shape
    rng = np.random.default_rng(d * n + 1)
    q = queries(rng, n, h_q, d, q_dtype)
    for exps, peak in (((-80, 60, -80, 60), 0), ((60, -80, -60, 70), 0), ((-40, 100, -30, 90), 0),
                       ((-95, -95, 0, 0), 0), ((-95,) * 4, 0), ((-90, -90, 40, 40), 1),
                       ((0, 100, 0, 0), 1)):
        length = 16 * 10 * len(exps)
        kv, ref = make(code, 16, h_kv, d, 1, -(-length // 16), h_q=h_q, seed=3)
        k = np.zeros((length, h_kv, d), dtype=np.float32)
        v = rows(rng, length, h_kv, d, "bf16", 0)
        v *= np.exp2(np.repeat(np.array(exps, dtype=np.float32), 160))[:, None, None]
        if peak:    # every query head's score is q.q / 4 or so of one of the first tokens
            for g in range(h_q // h_kv):
                k[g % 16] = synth.cast(q[-1].reshape(h_kv, -1, d)[:, g], "bf16")
        append(kv, ref, 0, [0], [0], [length], k, v, "bf16")
        scale = (90.0 if q_dtype == "bf16" else 30.0) / d if peak else 0.25
        want, mag = ref.attend(0, [0], [length], [n], q, scale)
        got = call(kv, [0], [length], [n], q, q_dtype, scale, tensor_core)
        # (peaked rows: see test_weights_far_below_the_largest for the second term)
        keys = np.repeat(ref.values(0, 0, "k", 0, length), h_q // h_kv, 1)
        s = np.einsum("thd,jhd->thj", q.astype(np.float64), keys) * scale
        late = np.arange(length)[None, None] > np.arange(length - n, length)[:, None, None]
        s[np.broadcast_to(late, s.shape)] = -np.inf
        w = np.exp(s - s.max(-1, keepdims=True))
        w /= w.sum(-1, keepdims=True)
        pages = ref.table[0, np.arange(length) // 16]
        vs = np.repeat(np.maximum(ref.scale["v"][0, pages], 2.0 ** -84), h_q // h_kv, 1)
        top = 127 if code == "i8" else 448
        peak_y = (w * vs.T[None]).max(-1)[..., None]
        err = np.abs(host(got) - want)
        tol = 2e-5 if q_dtype == "f32" else 5.5e-4
        lim = tol * mag + length * 2.0 ** -32 * top * peak_y + 1e-37
        if not peak:
            lim = tol * mag + 1e-37
        assert (err <= lim).all(), (exps, peak, float((err / lim).max()), int((err > lim).sum()))


@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("tensor_core", [False, True])
def test_many_value_tokens_of_zero(code, tensor_core):
    """Thousands of zero values with scores just above the first tile's, before
    a page that has some: the sum of their weights does not overflow."""
    n_seqs, n = (80, 20) if tensor_core else (700, 1)
    length, d, h_q = 16384 + 64, 64, 4
    kv, ref = make(code, 16, 1, d, 1, length // 16, h_q=h_q, seed=2)
    k = np.full((length, 1, d), 6.8 / (1.4427 * d), dtype=np.float32)
    k[:128] = 0
    v = np.zeros((length, 1, d), dtype=np.float32)
    v[-64:-32] = rows(np.random.default_rng(1), 32, 1, d, "bf16", 0)
    k, v = synth.cast(k, "bf16"), synth.cast(v, "bf16")
    append(kv, ref, 0, [0], [0], [length], k, v, "bf16")
    q = np.ones((n_seqs * n, h_q, d), dtype=np.float32)
    want, mag = ref.attend(0, [0], [length], [n], q[:n], 1.0)
    assert np.abs(want).max() > 1e-4
    got = run(kv, 0, [0] * n_seqs, [length] * n_seqs, [n] * n_seqs, q, "bf16", "f32", 1.0,
              max_seqlen=n, max_kv_len=length)
    for i in (0, 1, n_seqs // 2, n_seqs - 1):
        assert_close(got[i * n:(i + 1) * n], want, mag, "bf16", "f32", i)


@pytest.mark.parametrize("shape,q_dtype,tensor_core", SIDES)
def test_queries_of_the_largest_magnitudes(shape, q_dtype, tensor_core):
    """Finite queries up to the largest float, whose scores are ordinary."""
    h_q, h_kv, d, n = shape
    rng = np.random.default_rng(d + 3)
    kv, ref = make("i8", 16, h_kv, d, 1, 8, h_q=h_q)
    k = synth.cast(rows(rng, 100, h_kv, d, "bf16", 0) * np.float32(2.0 ** -90), "bf16")
    v = rows(rng, 100, h_kv, d, "bf16", 0)
    append(kv, ref, 0, [0], [0], [100], k, v, "bf16")
    for e in (115, 125, 126, 127):
        q = rng.uniform(-1.98, 1.98, (n, h_q, d)) * 2.0 ** e
        q[:, :, 0] = 1.98 * 2.0 ** e
        q = synth.cast(q, q_dtype)
        assert np.isfinite(q).all()
        scale = 2.0 ** (90 - e) / d ** 0.5
        want, mag = ref.attend(0, [0], [100], [n], q, scale)
        got = call(kv, [0], [100], [n], q, q_dtype, scale, tensor_core)
        assert_close(got, want, mag, q_dtype, "f32", e)

"""gdn_kv_attend at the edges of its range: value scales far apart, queries of
the largest magnitudes, loose bounds, every form of the tensor-core kernel over
long contexts, the unequal cut of large decode batches, and more streams than a
handle keeps workspaces for.  Tolerances are those of test_gpu_kv_attend.py."""
import numpy as np
import pytest
import torch

from gated_deltanet_recurrent_gb300 import abi, synth
from oracle.kv_oracle import KVOracle, attend_values
from tests.gpu_util import dev, dev_i32, host, tdtype
from tests.test_gpu_kv_attend import assert_close, filled, queries, run
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


@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("h_q,h_kv,d,hint", [(16, 2, 256, 40), (32, 8, 128, 80), (8, 2, 128, 130)])
def test_pairs_of_ctas_at_their_edges(code, h_q, h_kv, d, hint):
    """The bound of the query tokens makes pairs of CTAs take a few rows: an
    invalid page, queries that are not finite, more queries than positions."""
    rng = np.random.default_rng(hint + 1)
    kv, ref = filled(rng, code, 16, h_q, h_kv, d, [200, 2, 333])
    n = 9
    q = queries(rng, n, h_q, d, "bf16")
    o = padded(kv, [1], [2], [n], q, "f32", 0.1, hint)
    assert (host(o)[:n - 2] == 0).all()
    want, mag = attend_values(q[n - 2:].astype(np.float64),
                              *(ref.values(0, 1, s, 0, 2) for s in "kv"), 0.1)
    assert_close(o[n - 2:], want, mag, "bf16", "f32")
    bad = q.copy()
    bad[0, 1, 5], bad[n - 1, h_q - 1, 0] = np.nan, np.inf
    hit = np.zeros((n, h_q), dtype=bool)
    hit[0, 1] = hit[n - 1, h_q - 1] = True
    want, mag = ref.attend(0, [2], [333], [n], q, 0.1)
    o = padded(kv, [2], [333], [n], bad, "f32", 0.1, hint)
    assert np.isnan(host(o)[hit]).all()
    assert_close(o[torch.from_numpy(~hit).cuda()], want[~hit], mag[~hit], "bf16", "f32")
    assert abi.gdn_kv_get_error(kv) == 0
    kv.page_table[0, 4] = -1
    want, mag = attend_values(q.astype(np.float64), *(ref.values(0, 0, s, 0, 200) for s in "kv"),
                              0.1, np.arange(200) // 16 == 4)
    assert_close(padded(kv, [0], [200], [n], q, "f32", 0.1, hint), want, mag, "bf16", "f32")
    assert abi.gdn_kv_get_error(kv) == abi.DEVERR_PAGE


@pytest.mark.parametrize("h_q,h,d,page,n_pages,hint", [(32, 4, 256, 128, 18000, 40),
                                                       (32, 8, 128, 64, 36000, 80)])
def test_pairs_of_ctas_and_offsets_past_32_bits(h_q, h, d, page, n_pages, hint):
    rng = np.random.default_rng(22)
    kv = abi.KVCache.empty(2, 1, n_pages, 5, page, h_q, h, d, torch.int8, host_checks=False)
    assert kv.k.numel() > 1 << 32
    table = np.array([[n_pages - 1, n_pages - 7, 11, n_pages - 2, 12]])
    kv.page_table.copy_(torch.from_numpy(table.astype(np.int32)))
    k, v = rows(rng, 300, h, d, "bf16"), rows(rng, 300, h, d, "bf16")
    abi.gdn_kv_append(kv, 1, dev_i32([0]), dev_i32([0]), dev(k, "bf16"), dev(v, "bf16"),
                      cu_seqlens=cum([300]))
    ref = KVOracle(1, 5, h, page, d, "i8", np.arange(5)[None])
    ref.append(0, [0], [0], [300], k, v)
    q = queries(rng, hint, h_q, d, "bf16")
    want, mag = ref.attend(0, [0], [300], [hint], q, 1 / 16)
    o = run(kv, 1, [0], [300], [hint], q, "bf16", "f32", 1 / 16, max_seqlen=hint,
            max_kv_len=200000)
    assert_close(o, want, mag, "bf16", "f32")


def test_bounds_far_beyond_the_call():
    """Every bound is correct, also the largest there is."""
    rng = np.random.default_rng(23)
    kv, ref = filled(rng, "i8", 16, 8, 2, 128, [100, 40])
    huge = 2 ** 31 - 1
    for lens in ([3, 2], [40, 25]):
        q = queries(rng, sum(lens), 8, 128, "bf16")
        want, mag = ref.attend(0, [0, 1], [100, 40], lens, q, 0.1)
        got = run(kv, 0, [0, 1], [100, 40], lens, q, "bf16", "f32", 0.1, max_seqlen=huge,
                  max_kv_len=huge)
        assert_close(got, want, mag, "bf16", "f32")
    back = torch.empty(90, 2, 128, device="cuda")
    abi.gdn_kv_read(kv, 0, dev_i32([0, 1]), dev_i32([10, 40]), back, None, cu_seqlens=cum([90, 0]),
                    max_seqlen=huge)
    assert np.array_equal(host(back), ref.values(0, 0, "k", 10, 100))
    assert abi.gdn_kv_get_error(kv) == 0


@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("h_q,h_kv,d,n", FORMS)
def test_tensor_core_kernel_over_long_contexts(code, h_q, h_kv, d, n):
    """Enough sequences that no context is cut, of some 20 tiles each."""
    rng = np.random.default_rng(n + d)
    lens = [2500, 2311, 1100]
    kv, ref = filled(rng, code, 64 if d == 64 else 128, h_q, h_kv, d, lens)
    n_seqs = 160 // h_kv + 1
    slots = [i % 3 for i in range(n_seqs)]
    kv_lens = [int(rng.integers(max(n, lens[s] - 300), lens[s] + 1)) for s in slots]
    q = queries(rng, n * n_seqs, h_q, d, "bf16")
    o = run(kv, 0, slots, kv_lens, [n] * n_seqs, q, "bf16", "bf16", d ** -0.5, max_seqlen=n,
            max_kv_len=2500)
    for i in (0, 1, 2, n_seqs - 1):
        part = q[i * n:(i + 1) * n]
        want, mag = ref.attend(0, [slots[i]], [kv_lens[i]], [n], part, d ** -0.5)
        assert_close(o[i * n:(i + 1) * n], want, mag, "bf16", "bf16", i)
    # one of them alone: its context is cut into several CTAs' pieces
    o = run(kv, 0, [0], [2500], [n], q[:n], "bf16", "f32", d ** -0.5, max_seqlen=n,
            max_kv_len=5000)
    want, mag = ref.attend(0, [0], [2500], [n], q[:n], d ** -0.5)
    assert_close(o, want, mag, "bf16", "f32")
    assert abi.gdn_kv_get_error(kv) == 0


@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("q_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("h_q,n_seqs", [(16, 45), (16, 64), (6, 200)])
def test_decode_batches_in_unequal_pieces(code, q_dtype, h_q, n_seqs):
    """d = 256, up to eight query heads per KV head, and more than four tiles
    a CTA of a full grid: the pieces of the line of tiles differ in length by
    the CTA's order on its SM, and units are cut where the orders meet.  Up to
    8 tiles a CTA the line has no places for the units' starts, above it has."""
    rng = np.random.default_rng(n_seqs)
    lens = [2500, 2311, 2400, 2100, 2048, 2499, 1900, 2450]
    kv, ref = filled(rng, code, 64, h_q, 2, 256, lens)
    slots = [i % 8 for i in range(n_seqs)]
    kv_lens = [int(rng.integers(1 if i % 9 == 7 else lens[s] * 3 // 4, lens[s] + 1))
               for i, s in enumerate(slots)]
    kv_lens[0] = 2500
    ctas = 3 * torch.cuda.get_device_properties(0).multi_processor_count
    assert 2 * sum(-(-x // 64) for x in kv_lens) >= 4 * ctas
    assert (n_seqs * 2 * (2500 // 64 + 1) >= 8 * ctas) == (n_seqs > 45)
    q = queries(rng, n_seqs, h_q, 256, q_dtype)
    got = run(kv, 0, slots, kv_lens, [1] * n_seqs, q, q_dtype, "f32", 1 / 16, max_kv_len=2500)
    want, mag = ref.attend(0, slots, kv_lens, [1] * n_seqs, q, 1 / 16)
    assert_close(got, want, mag, q_dtype, "f32")
    assert abi.gdn_kv_get_error(kv) == 0


def test_more_streams_than_kept_workspaces():
    """A handle keeps workspaces for 16 streams; calls on others are as right."""
    rng = np.random.default_rng(30)
    kv, ref = filled(rng, "i8", 64, 8, 2, 128, [3000, 700])
    for n in (1, 24):
        q = queries(rng, 2 * n, 8, 128, "bf16")
        want, mag = ref.attend(0, [0, 1], [3000, 700], [n, n], q, 0.1)
        qd, slots, kv_lens, cu = dev(q, "bf16"), dev_i32([0, 1]), dev_i32([3000, 700]), cum([n, n])
        streams, outs = [torch.cuda.Stream() for _ in range(20)], []
        torch.cuda.synchronize()
        for rep in range(3):
            for s in streams:
                with torch.cuda.stream(s):
                    outs.append(abi.gdn_kv_attend(kv, 0, slots, kv_lens, qd, cu_seqlens=cu,
                                                  max_seqlen=n, max_kv_len=3000, scale=0.1))
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o, outs[0])
        assert_close(outs[0], want, mag, "bf16", "bf16")

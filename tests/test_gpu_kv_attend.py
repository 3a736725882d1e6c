"""gdn_kv_attend (causal grouped-query attention over the 8-bit paged cache)
against the float64 oracle, through the C ABI.

Tolerances, with mag = sum_j w_j |v_j| of the same output element and all
inputs held as the oracle holds them (the codes are exact on both sides):
  float32 q: a score carries the query's two binary16 parts (2^-22 of it) and
    float32 sums, a weight the same and one exponential; for |score| < 40 that
    is under 40 * 2^-21 = 2e-5 relative on each weight:   err <= 2e-5 mag
  bf16 q: the weights are rounded to binary16 (2^-11):    err <= 5.5e-4 mag
  bf16 o: one more rounding of the output (2^-8):         + 2^-8 |ref|"""
import numpy as np
import pytest
import torch

from gated_deltanet_recurrent_gb300 import abi, synth
from oracle.kv_oracle import attend_values
from tests.gpu_util import dev, dev_i32, host, tdtype
from tests.test_gpu_kv_cache import append, cum, make, rows

pytestmark = pytest.mark.gpu


def assert_close(got, ref, mag, q_dtype, o_dtype, what=""):
    got = host(got)
    lim = (2e-5 if q_dtype == "f32" else 5.5e-4) * mag + 1e-30
    if o_dtype == "bf16":
        lim = lim + 2.0 ** -8 * np.abs(ref)
    err = np.abs(got - ref)
    assert (err <= lim).all(), (what, float((err / lim).max()), int((err > lim).sum()), err.size)


def run(kv, layer, slots, kv_lens, lens, q, q_dtype, o_dtype, scale, **kw):
    o = torch.full(q.shape, 7.0, device="cuda", dtype=tdtype(o_dtype))
    cu = None if all(n == 1 for n in lens) and kw.pop("no_cu", True) else cum(lens)
    abi.gdn_kv_attend(kv, layer, dev_i32(slots), dev_i32(kv_lens), dev(q, q_dtype), o,
                      cu_seqlens=cu, scale=scale, **kw)
    return o


def filled(rng, code, page, h_q, h_kv, d, lens, dtype="bf16", spread=1.0, n_layers=1, layer=0):
    """A cache holding lens[i] tokens in slot i (shuffled pages, stale bytes elsewhere)."""
    max_pages = max(1, -(-max(lens) // page)) + 1
    kv, ref = make(code, page, h_kv, d, len(lens), max_pages, h_q=h_q, n_layers=n_layers,
                   seed=int(rng.integers(1 << 30)))
    k, v = (rows(rng, sum(lens), h_kv, d, dtype, spread) for _ in range(2))
    append(kv, ref, layer, list(range(len(lens))), [0] * len(lens), lens, k, v, dtype)
    return kv, ref


def queries(rng, n, h_q, d, dtype):
    return synth.cast(rng.standard_normal((n, h_q, d)), dtype)


SHAPES = [(16, 2, 256), (32, 8, 128), (28, 4, 128), (3, 3, 128), (12, 4, 64), (40, 1, 64),
          (20, 1, 256), (6, 2, 256)]


@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("q_dtype,o_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"),
                                             ("f32", "bf16")])
@pytest.mark.parametrize("h_q,h_kv,d", SHAPES)
def test_single_tokens(code, q_dtype, o_dtype, h_q, h_kv, d):
    """Decode: one token a slot, contexts from one token past several pages."""
    rng = np.random.default_rng(h_q * d)
    page = {64: 16, 128: 32, 256: 128}[d] if code == "i8" else 64
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 777]
    kv, ref = filled(rng, code, page, h_q, h_kv, d, lens)
    slots = rng.permutation(len(lens))
    kv_lens = [lens[s] for s in slots]
    q = queries(rng, len(lens), h_q, d, q_dtype)
    want, mag = ref.attend(0, slots, kv_lens, [1] * len(lens), q, d ** -0.5)
    for hint in (777, 1, 1 << 20):
        got = run(kv, 0, slots, kv_lens, [1] * len(lens), q, q_dtype, o_dtype, d ** -0.5,
                  max_kv_len=hint)
        assert_close(got, want, mag, q_dtype, o_dtype, hint)
    assert abi.gdn_kv_get_error(kv) == 0


@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("h_q,h_kv,d", SHAPES)
@pytest.mark.parametrize("lens,kv_lens", [
    ([4, 1, 0, 3, 2], [70, 1, 9, 3, 130]),                # drafts
    ([17, 40, 1, 0, 128], [33, 40, 200, 0, 129]),         # pieces of prompts
    ([300], [300]),                                       # a whole prompt
    ([129, 257], [500, 260]),
])
def test_many_tokens(code, dtype, h_q, h_kv, d, lens, kv_lens):
    rng = np.random.default_rng(sum(lens) + h_q)
    page = 16 if code == "i8" else {64: 128, 128: 32, 256: 64}[d]
    kv, ref = filled(rng, code, page, h_q, h_kv, d, kv_lens)
    q = queries(rng, sum(lens), h_q, d, dtype)
    slots = list(range(len(lens)))
    want, mag = ref.attend(0, slots, kv_lens, lens, q, d ** -0.5)
    for hint in (max(lens), 1, 100000):
        got = run(kv, 0, slots, kv_lens, lens, q, dtype, dtype, d ** -0.5, max_seqlen=hint,
                  max_kv_len=max(kv_lens))
        assert_close(got, want, mag, dtype, dtype, hint)
    assert abi.gdn_kv_get_error(kv) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [3, 40])
def test_queries_with_nothing_to_attend_get_zeros(dtype, n):
    """More query tokens than cached ones: the first have no position; an
    empty slot's queries have none at all."""
    rng = np.random.default_rng(n)
    kv, ref = filled(rng, "e4m3", 16, 8, 2, 128, [2, 1, 50])
    q = queries(rng, 3 * n, 8, 128, dtype)
    o = run(kv, 0, [0, 1, 2], [2, 0, 50], [n, n, n], q, dtype, "f32", 0.1)
    got = host(o)
    assert (got[:n - 2] == 0).all() and (got[n:2 * n] == 0).all()
    for slot, lo, length, m in ((0, n - 2, 2, 2), (2, 2 * n, 50, n)):
        k, v = (ref.values(0, slot, s, 0, length) for s in "kv")
        want, mag = attend_values(q[lo:lo + m].astype(np.float64), k, v, 0.1)
        assert_close(o[lo:lo + m], want, mag, dtype, "f32")


@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("n", [1, 33])
def test_value_scales_far_apart(code, n):
    """A dominant token whose values are 2^-30 of the others' (and pages of
    zeros): its contribution keeps its precision."""
    rng = np.random.default_rng(7)
    h, d, length = 2, 128, 400
    kv, ref = make(code, 16, h, d, 1, 26, h_q=8, seed=3)
    k, v = rows(rng, length, h, d, "bf16", 0), rows(rng, length, h, d, "bf16", 0)
    q = queries(rng, n, 8, d, "bf16")
    k[:16] = 0
    k[5] = q[-1].reshape(h, 4, d)[:, 0] * 4        # a peak for one query head of each group
    v[:16] *= 2.0 ** -30
    v[64:128] = 0
    append(kv, ref, 0, [0], [0], [length], k, v, "bf16")
    want, mag = ref.attend(0, [0], [length], [n], q, 1.0)
    got = run(kv, 0, [0], [length], [n], q, "bf16", "f32", 1.0)
    assert_close(got, want, mag, "bf16", "f32")


@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-6, 3.0])
@pytest.mark.parametrize("n", [1, 40])
def test_scales_of_any_sign(scale, n):
    rng = np.random.default_rng(8)
    kv, ref = filled(rng, "i8", 32, 8, 2, 64, [150], spread=0)
    q = queries(rng, n, 8, 64, "bf16") * np.float32(0.25)
    want, mag = ref.attend(0, [0], [150], [n], q, scale)
    assert_close(run(kv, 0, [0], [150], [n], q, "bf16", "f32", scale), want, mag, "bf16", "f32")


@pytest.mark.parametrize("n", [1, 40])
def test_a_query_that_is_not_finite_stays_alone(n):
    rng = np.random.default_rng(10)
    kv, ref = filled(rng, "e4m3", 64, 8, 2, 128, [100, 90])
    q = queries(rng, 2 * n, 8, 128, "bf16")
    want, mag = ref.attend(0, [0, 1], [100, 90], [n, n], q, 0.1)
    q[0, 3, 5], q[n, 7, 0], q[n, 1] = np.nan, np.inf, 0.0
    want[n, 1], mag[n, 1] = (x[0, 0] for x in attend_values(
        np.zeros((1, 8, 128)), *(ref.values(0, 1, s, 0, 90 - n + 1) for s in "kv"), 0.1))
    got = run(kv, 0, [0, 1], [100, 90], [n, n], q, "bf16", "f32", 0.1)
    hit = np.zeros(q.shape[:2], dtype=bool)
    hit[0, 3] = hit[n, 7] = True
    assert np.isnan(host(got)[hit]).all()
    keep = torch.from_numpy(~hit)
    assert_close(got[keep.cuda()], want[~hit], mag[~hit], "bf16", "f32")


def test_keys_and_queries_of_any_magnitude():
    """Queries of 1e30 against keys of 1e-30, and the other way round."""
    rng = np.random.default_rng(12)
    for a in (1e30, 1e-30):
        for n in (1, 40):
            kv, ref = make("i8", 16, 1, 64, 1, 8, h_q=4)
            k, v = rows(rng, 100, 1, 64, "bf16", 0), rows(rng, 100, 1, 64, "bf16", 0)
            append(kv, ref, 0, [0], [0], [100], synth.cast(k / a, "bf16"), v, "bf16")
            q = synth.cast(queries(rng, n, 4, 64, "bf16") * a, "bf16")
            want, mag = ref.attend(0, [0], [100], [n], q, 0.125)
            got = run(kv, 0, [0], [100], [n], q, "bf16", "f32", 0.125)
            assert_close(got, want, mag, "bf16", "f32")


@pytest.mark.parametrize("n", [1, 5, 60])
@pytest.mark.parametrize("bad", [-1, 1 << 20])
def test_tokens_of_an_invalid_page_are_masked_and_reported(n, bad):
    rng = np.random.default_rng(13)
    kv, ref = filled(rng, "i8", 16, 8, 2, 128, [200, 16])
    q = queries(rng, n, 8, 128, "bf16")
    k, v = (ref.values(0, 0, s, 0, 200) for s in "kv")
    kv.page_table[0, 3] = bad
    skip = (np.arange(200) // 16) == 3
    want, mag = attend_values(q.astype(np.float64), k, v, 0.1, skip)
    got = run(kv, 0, [0], [200], [n], q, "bf16", "f32", 0.1)
    assert_close(got, want, mag, "bf16", "f32")
    assert abi.gdn_kv_get_error(kv) == abi.DEVERR_PAGE
    kv.page_table[1, 0] = bad          # nothing left: zeros
    got = run(kv, 0, [1], [min(16, n + 3)], [n], q, "bf16", "f32", 0.1)
    assert (host(got) == 0).all()
    assert abi.gdn_kv_get_error(kv) == abi.DEVERR_PAGE


def test_bad_entries_are_skipped_and_reported():
    rng = np.random.default_rng(14)
    kv, ref = filled(rng, "i8", 16, 4, 2, 64, [20, 30, 20])
    for n in (1, 50):
        q = queries(rng, 3 * n, 4, 64, "bf16")
        o = run(kv, 0, [0, 3, 2], [20, 5, 49], [n] * 3, q, "bf16", "f32", 0.1)
        assert abi.gdn_kv_get_error(kv) == abi.DEVERR_SLOT | abi.DEVERR_SEQ
        assert (host(o)[n:] == 7).all()
        m = min(n, 20)
        want, mag = attend_values(q[n - m:n].astype(np.float64),
                                  *(ref.values(0, 0, s, 0, 20) for s in "kv"), 0.1)
        assert_close(o[n - m:n], want, mag, "bf16", "f32")
    o = torch.full((4, 4, 64), 7.0, device="cuda")
    abi.gdn_kv_attend(kv, 0, dev_i32([0, 1, 2]), dev_i32([20, 30, -1]), torch.zeros_like(o), o,
                      cu_seqlens=dev_i32([-1, 5, 2, 3]))
    assert abi.gdn_kv_get_error(kv) == abi.DEVERR_SEQ
    assert (o == 7).all()


def test_strided_queries_on_a_side_stream_and_in_a_graph():
    """q as columns of wider rows, o into wider rows; the call is captured and
    replayed on new inputs and a longer context."""
    rng = np.random.default_rng(15)
    for n in (1, 24):
        kv, ref = filled(rng, "e4m3", 64, 16, 2, 128, [400, 500, 80])
        wide = torch.zeros(3 * n, 20, 128, device="cuda", dtype=torch.bfloat16)
        out = torch.full((3 * n, 18, 128), 7.0, device="cuda", dtype=torch.bfloat16)
        slots, kv_lens, cu = dev_i32([1, 0, 2]), dev_i32([60, 60, 60]), cum([n] * 3)
        side = torch.cuda.Stream()
        call = lambda: abi.gdn_kv_attend(kv, 0, slots, kv_lens, wide[:, 2:18], out[:, 1:17],
                                         cu_seqlens=cu, max_seqlen=n, max_kv_len=500)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            call()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call()
        for lens in ([500, 400, 80], [70, 333, 24]):
            q = queries(rng, 3 * n, 16, 128, "bf16")
            wide[:, 2:18] = dev(q, "bf16")
            kv_lens.copy_(dev_i32(lens))
            g.replay()
            torch.cuda.synchronize()
            want, mag = ref.attend(0, [1, 0, 2], lens, [n] * 3, q, 128 ** -0.5)
            assert_close(out[:, 1:17], want, mag, "bf16", "bf16")
            assert (out[:, 0] == 7).all() and (out[:, 17] == 7).all()


def test_two_streams_at_once():
    """Calls on one handle overlap on two streams without disturbing each other."""
    rng = np.random.default_rng(16)
    kv, ref = filled(rng, "i8", 64, 16, 2, 256, [3000, 2500])
    q = queries(rng, 2, 16, 256, "bf16")
    want, mag = ref.attend(0, [0, 1], [3000, 2500], [1, 1], q, 1 / 16)
    streams = [torch.cuda.Stream() for _ in range(2)]
    qs, os_ = [dev(q[i:i + 1], "bf16") for i in range(2)], []
    ids, lens = [dev_i32([i]) for i in range(2)], [dev_i32([n]) for n in (3000, 2500)]
    torch.cuda.synchronize()
    for rep in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                os_.append((i, abi.gdn_kv_attend(kv, 0, ids[i], lens[i], qs[i], max_kv_len=3000)))
    torch.cuda.synchronize()
    for i, o in os_:
        assert_close(o, want[i:i + 1], mag[i:i + 1], "bf16", "bf16")


@pytest.mark.parametrize("n", [1, 40])
def test_offsets_past_32_bits(n):
    """Codes of more than 4 GiB a side: pages at the far end, in the last layer."""
    rng = np.random.default_rng(17)
    h, d, page, n_pages = 4, 256, 128, 18000
    kv = abi.KVCache.empty(2, 1, n_pages, 3, page, 8, h, d, torch.int8, host_checks=False)
    assert kv.k.numel() > 1 << 32
    table = np.array([[n_pages - 1, n_pages - 7, 11]])
    kv.page_table.copy_(torch.from_numpy(table.astype(np.int32)))
    k, v = rows(rng, 300, h, d, "bf16"), rows(rng, 300, h, d, "bf16")
    abi.gdn_kv_append(kv, 1, dev_i32([0]), dev_i32([0]), dev(k, "bf16"), dev(v, "bf16"),
                      cu_seqlens=cum([300]))
    from oracle.kv_oracle import KVOracle
    ref = KVOracle(1, 3, h, page, d, "i8", np.array([[0, 1, 2]]))
    ref.append(0, [0], [0], [300], k, v)
    back = torch.empty(300, h, d, device="cuda")
    abi.gdn_kv_read(kv, 1, dev_i32([0]), dev_i32([0]), back, None, cu_seqlens=cum([300]))
    assert np.array_equal(host(back), ref.values(0, 0, "k", 0, 300))
    q = queries(rng, n, 8, d, "bf16")
    want, mag = ref.attend(0, [0], [300], [n], q, 1 / 16)
    o = run(kv, 1, [0], [300], [n], q, "bf16", "f32", 1 / 16)
    assert_close(o, want, mag, "bf16", "f32")
    assert not kv.k[0].any()


def test_long_context_and_many_slots():
    """One context split over the whole GPU; then many slots of mixed lengths."""
    rng = np.random.default_rng(18)
    kv, ref = filled(rng, "e4m3", 128, 8, 2, 128, [20011], spread=0)
    q = queries(rng, 1, 8, 128, "f32")
    want, mag = ref.attend(0, [0], [20011], [1], q, 128 ** -0.5)
    assert_close(run(kv, 0, [0], [20011], [1], q, "f32", "f32", 128 ** -0.5), want, mag, "f32",
                 "f32")
    lens = [int(x) for x in rng.integers(1, 120, 300)]
    kv, ref = filled(rng, "i8", 16, 4, 1, 64, lens, spread=0)
    slots = rng.permutation(300)
    q = queries(rng, 300, 4, 64, "bf16")
    want, mag = ref.attend(0, slots, [lens[s] for s in slots], [1] * 300, q, 0.125)
    got = run(kv, 0, slots, [lens[s] for s in slots], [1] * 300, q, "bf16", "bf16", 0.125,
              max_kv_len=120)
    assert_close(got, want, mag, "bf16", "bf16")


@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("h_q,h_kv,d", [(16, 2, 256), (8, 2, 128), (28, 4, 128), (12, 4, 64)])
def test_weights_far_below_the_largest(code, h_q, h_kv, d):
    """The tensor-core kernel (the length hints choose it) on scores up to 100
    apart and V scales 2^-30 apart.  Weights are rounded to 2^-11, or to a step
    of 2^-24 under a largest weight of at least 2^7: the contribution of a
    position is off by at most 2^-32 of the largest y = weight * V scale of its
    row, times its code, of at most top.  So, beside the usual relative part,
    err <= positions * 2^-32 * max_j(w_j s_j) * top."""
    rng = np.random.default_rng(20)
    length, n, page, top = 300, 40, 16, 127 if code == "i8" else 448
    kv, ref = make(code, page, h_kv, d, 1, 20, h_q=h_q, seed=4)
    k, v = rows(rng, length, h_kv, d, "bf16", 0), rows(rng, length, h_kv, d, "bf16", 0)
    q = queries(rng, n, h_q, d, "bf16")
    k[:16] = 0
    k[5] = q[-1].reshape(h_kv, -1, d)[:, 0] * 2
    v[:16] *= 2.0 ** -30
    v[64:128] = 0
    append(kv, ref, 0, [0], [0], [length], k, v, "bf16")
    scale = 100.0 / (2 * d)
    want, mag = ref.attend(0, [0], [length], [n], q, scale)
    got = run(kv, 0, [0], [length], [n], q, "bf16", "f32", scale, max_seqlen=2000,
              max_kv_len=40000)
    group = h_q // h_kv
    keys = np.repeat(ref.values(0, 0, "k", 0, length), group, 1)
    s = np.einsum("thd,jhd->thj", q.astype(np.float64), keys) * scale
    s[np.arange(length)[None, None] > np.arange(length - n, length)[:, None, None] + 0 * s] = -np.inf
    w = np.exp(s - s.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    pages = ref.table[0, np.arange(length) // page]
    v_scale = np.repeat(ref.scale["v"][0, pages], group, 1)            # [length, h_q]
    peak = (w * v_scale.T[None]).max(-1)
    lim = 5.5e-4 * mag + length * 2.0 ** -32 * top * peak[..., None]
    err = np.abs(host(got) - want)
    assert (err <= lim).all(), (float((err / lim).max()), int((err > lim).sum()))


@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("h_q,h_kv,d,hint", [(16, 2, 256, 5), (16, 2, 256, 40), (32, 8, 128, 20),
                                             (32, 8, 128, 40), (8, 2, 128, 80), (12, 4, 64, 40),
                                             (12, 4, 64, 60)])
def test_more_rows_than_the_hint_says(code, h_q, h_kv, d, hint):
    """The hints choose the tensor-core kernel in each of its forms, for fewer
    query tokens than there are: its CTAs take several units one after another."""
    rng = np.random.default_rng(hint + d)
    lens, kv_lens = [300, 0, 129, 1, 37], [301, 5, 700, 64, 37]
    kv, ref = filled(rng, code, 32, h_q, h_kv, d, kv_lens)
    q = queries(rng, sum(lens), h_q, d, "bf16")
    slots = list(range(5))
    want, mag = ref.attend(0, slots, kv_lens, lens, q, d ** -0.5)
    for kv_hint in (40000, 700):
        got = run(kv, 0, slots, kv_lens, lens, q, "bf16", "bf16", d ** -0.5, max_seqlen=hint,
                  max_kv_len=kv_hint)
        assert_close(got, want, mag, "bf16", "bf16", kv_hint)
    assert abi.gdn_kv_get_error(kv) == 0


# hints that choose the tensor-core kernel whatever the call's size; a call of 200 tokens a slot
# takes pairs of CTAs (d = 128, 256), one of 40 tokens or fewer a CTA alone
FORMS = [(16, 2, 256, 200), (16, 2, 256, 9), (32, 8, 128, 200), (32, 8, 128, 40), (32, 8, 128, 20),
         (12, 4, 64, 200), (12, 4, 64, 20)]


@pytest.mark.parametrize("h_q,h_kv,d,hint", FORMS)
def test_tensor_core_kernel_at_its_edges(h_q, h_kv, d, hint):
    """Queries without positions, an invalid page, queries that are not finite,
    scales of any sign, strided rows: each for the other kernel too, above."""
    rng = np.random.default_rng(d + hint)
    force = dict(max_seqlen=hint, max_kv_len=200000)
    n = min(hint, 50)
    kv, ref = filled(rng, "e4m3", 16, h_q, h_kv, d, [2, 0, 200, 333])
    lens, kv_lens, slots = [n, n, n, n], [2, 0, 200, 333], [0, 1, 2, 3]
    q = queries(rng, 4 * n, h_q, d, "bf16")
    for scale in (d ** -0.5, -0.1, 0.0):
        o = run(kv, 0, slots, kv_lens, lens, q, "bf16", "f32", scale, **force)
        assert (host(o)[:n - 2] == 0).all() and (host(o)[n:2 * n] == 0).all()
        for slot, lo, m in ((0, n - 2, 2), (2, 2 * n, n), (3, 3 * n, n)):
            k, v = (ref.values(0, slot, s, 0, kv_lens[slot]) for s in "kv")
            want, mag = attend_values(q[lo:lo + m].astype(np.float64), k, v, scale)
            assert_close(o[lo:lo + m], want, mag, "bf16", "f32", (slot, scale))
    assert abi.gdn_kv_get_error(kv) == 0
    # a page in the middle that is none
    kv.page_table[2, 4] = kv.desc.n_pages
    k, v = (ref.values(0, 2, s, 0, 200) for s in "kv")
    want, mag = attend_values(q[:n].astype(np.float64), k, v, 0.1, np.arange(200) // 16 == 4)
    assert_close(run(kv, 0, [2], [200], [n], q[:n], "bf16", "f32", 0.1, **force), want, mag,
                 "bf16", "f32")
    assert abi.gdn_kv_get_error(kv) == abi.DEVERR_PAGE
    # queries that are not finite, in rows of their own
    bad = q[:n].copy()
    bad[0, 1, 5], bad[n - 1, h_q - 1, 0] = np.nan, np.inf
    k, v = (ref.values(0, 3, s, 0, 333) for s in "kv")
    want, mag = attend_values(q[:n].astype(np.float64), k, v, 0.1)
    wide = torch.zeros(n, h_q + 3, d, device="cuda", dtype=torch.bfloat16)
    out = torch.full((n, h_q + 2, d), 7.0, device="cuda")
    wide[:, 1:h_q + 1] = dev(bad, "bf16")
    abi.gdn_kv_attend(kv, 0, dev_i32([3]), dev_i32([333]), wide[:, 1:h_q + 1], out[:, 2:],
                      cu_seqlens=cum([n]), scale=0.1, **force)
    hit = np.zeros((n, h_q), dtype=bool)
    hit[0, 1] = hit[n - 1, h_q - 1] = True
    got = out[:, 2:]
    assert np.isnan(host(got)[hit]).all() and (out[:, :2] == 7).all()
    keep = torch.from_numpy(~hit).cuda()
    assert_close(got[keep], want[~hit], mag[~hit], "bf16", "f32")


@pytest.mark.parametrize("hint", [9, 200])
def test_tensor_core_kernel_offsets_past_32_bits(hint):
    rng = np.random.default_rng(21)
    h, d, page, n_pages, n = 4, 256, 128, 18000, 9
    kv = abi.KVCache.empty(2, 1, n_pages, 3, page, 32, h, d, torch.int8, host_checks=False)
    table = np.array([[n_pages - 1, n_pages - 7, 11]])
    kv.page_table.copy_(torch.from_numpy(table.astype(np.int32)))
    k, v = rows(rng, 300, h, d, "bf16"), rows(rng, 300, h, d, "bf16")
    abi.gdn_kv_append(kv, 1, dev_i32([0]), dev_i32([0]), dev(k, "bf16"), dev(v, "bf16"),
                      cu_seqlens=cum([300]))
    from oracle.kv_oracle import KVOracle
    ref = KVOracle(1, 3, h, page, d, "i8", np.array([[0, 1, 2]]))
    ref.append(0, [0], [0], [300], k, v)
    q = queries(rng, n, 32, d, "bf16")
    want, mag = ref.attend(0, [0], [300], [n], q, 1 / 16)
    o = run(kv, 1, [0], [300], [n], q, "bf16", "f32", 1 / 16, max_seqlen=hint, max_kv_len=200000)
    assert_close(o, want, mag, "bf16", "f32")


def test_zero_tokens_and_the_same_answer_twice():
    rng = np.random.default_rng(19)
    kv, _ = filled(rng, "i8", 16, 4, 2, 64, [500, 3])
    empty = torch.zeros(0, 4, 64, device="cuda", dtype=torch.bfloat16)
    abi.gdn_kv_attend(kv, 0, dev_i32([]), dev_i32([]), empty)
    abi.gdn_kv_attend(kv, 0, dev_i32([0, 1]), dev_i32([5, 3]), empty, cu_seqlens=cum([0, 0]))
    for n in (1, 30):
        q = queries(rng, n, 4, 64, "bf16")
        a, b = (run(kv, 0, [0], [500], [n], q, "bf16", "f32", 0.1) for _ in range(2))
        assert torch.equal(a, b)

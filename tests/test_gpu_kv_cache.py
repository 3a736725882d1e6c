"""The 8-bit paged KV cache: gdn_kv_append and gdn_kv_read against the float64
oracle, through the C ABI.

Scales are powers of two, so value / scale, a change of scale and code * scale
are exact in float32 and every code is one rounding to nearest even: codes,
scales and values have to equal the oracle's exactly, in any order of work."""
import numpy as np
import pytest
import torch

from gated_deltanet_recurrent_gb300 import abi, synth
from oracle.kv_oracle import KVOracle
from tests.gpu_util import dev, dev_i32, tdtype

pytestmark = pytest.mark.gpu

CODES = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn}


def make(code, page, h_kv, d, n_slots, max_pages, h_q=None, n_layers=1, spare=3, checks=False,
         seed=0):
    """A cache whose slots own every page of a shuffled list, with stale bytes
    and scales in its memory, and its oracle."""
    rng = np.random.default_rng(seed)
    n_pages = n_slots * max_pages + spare
    kv = abi.KVCache.empty(n_layers, n_slots, n_pages, max_pages, page, h_q or h_kv, h_kv, d,
                           CODES[code], host_checks=checks)
    kv.k.view(torch.uint8).fill_(0xff)
    kv.v.view(torch.uint8).fill_(0x7f)
    kv.k_scale.fill_(float("nan"))
    kv.v_scale.fill_(float("inf"))
    table = rng.permutation(n_pages)[:n_slots * max_pages].reshape(n_slots, max_pages)
    kv.page_table.copy_(torch.from_numpy(table.astype(np.int32)))
    return kv, KVOracle(n_layers, n_pages, h_kv, page, d, code, table)


def cum(lens):
    return dev_i32(np.concatenate([[0], np.cumsum(lens)]))


def rows(rng, n, h, d, dtype, spread=2.0):
    x = rng.standard_normal((n, h, d)) * np.exp2(rng.uniform(-spread, spread, (n, 1, 1)))
    return synth.cast(x, dtype)


def append(kv, ref, layer, slots, pos, lens, k, v, dtype, **kw):
    abi.gdn_kv_append(kv, layer, dev_i32(slots), dev_i32(pos), dev(k, dtype), dev(v, dtype),
                      cu_seqlens=cum(lens), **kw)
    ref.append(layer, slots, pos, lens, k, v)


def check(kv, ref, layer, slot, length, dtype="f32"):
    d = kv.desc
    k = torch.full((length, d.h_kv, d.d), 7.0, device="cuda", dtype=tdtype(dtype))
    v = torch.full_like(k, 9.0)
    abi.gdn_kv_read(kv, layer, dev_i32([slot]), dev_i32([0]), k, v, cu_seqlens=cum([length]))
    assert np.array_equal(k.double().cpu().numpy(), ref.values(layer, slot, "k", 0, length))
    assert np.array_equal(v.double().cpu().numpy(), ref.values(layer, slot, "v", 0, length))
    pages = ref.table[slot, :-(-length // ref.page)]
    for side, s in (("k", kv.k_scale), ("v", kv.v_scale)):
        assert np.array_equal(s[layer].double().cpu().numpy()[pages], ref.scale[side][layer, pages])


@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("page,h,d", [(16, 3, 64), (32, 2, 128), (64, 1, 256), (128, 2, 256),
                                      (128, 5, 64)])
def test_pieces_of_prompts_match_the_oracle(code, dtype, page, h, d):
    """Prompts of mixed lengths (none, one, page - 1, page + 1, ...) fed in
    pieces that end inside pages, then single tokens."""
    rng = np.random.default_rng(page + d)
    max_pages = 5
    kv, ref = make(code, page, h, d, 6, max_pages, seed=page)
    slots = np.array([4, 0, 5, 2, 1])
    total = np.zeros(5, dtype=int)
    for lens in ([0, 1, page - 1, page + 1, 2 * page + 3], [page, 1, 1, page, 9],
                 [1, 1, 1, 1, 1], [1, 0, 3, 8, 2]):
        k, v = (rows(rng, sum(lens), h, d, dtype) for _ in range(2))
        append(kv, ref, 0, slots, total, lens, k, v, dtype, max_seqlen=max(lens))
        total = total + np.array(lens)
    for s, n in zip(slots, total):
        check(kv, ref, 0, s, int(n), dtype)
    assert abi.gdn_kv_get_error(kv) == 0


@pytest.mark.parametrize("code", ["i8", "e4m3"])
def test_a_growing_page_rescales_what_it_keeps(code):
    """Single tokens whose magnitude grows and shrinks: kept codes are rounded
    again at each larger scale, and the scale never shrinks within a page."""
    rng = np.random.default_rng(5)
    kv, ref = make(code, 32, 2, 64, 1, 3)
    for p in range(70):
        x = rng.standard_normal((2, 1, 2, 64)) * 2.0 ** (rng.integers(-6, 7) + p / 16)
        k, v = synth.cast(x[0], "bf16"), synth.cast(x[1], "bf16")
        append(kv, ref, 0, [0], [p], [1], k, v, "bf16")
        check(kv, ref, 0, 0, p + 1)


def test_rejected_drafts_are_overwritten():
    rng = np.random.default_rng(6)
    kv, ref = make("i8", 16, 2, 128, 2, 3)
    k, v = rows(rng, 30, 2, 128, "bf16"), rows(rng, 30, 2, 128, "bf16")
    append(kv, ref, 0, [1], [0], [13], k[:13], v[:13], "bf16")
    append(kv, ref, 0, [1], [13], [6], k[13:19] * 8, v[13:19] * 8, "bf16")   # crosses a page
    append(kv, ref, 0, [1], [14], [4], k[19:23], v[19:23], "bf16")
    check(kv, ref, 0, 1, 18)
    append(kv, ref, 0, [1], [16], [2], k[23:25], v[23:25], "bf16")           # a page starts anew
    check(kv, ref, 0, 1, 18)


@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("hint", [8, 100])
def test_zeros_tiny_huge_and_non_finite_values(code, hint):
    """Zeros, subnormals and values beyond the largest scale, then infinities
    and NaN (reported): the finite values of a block decide its scale."""
    n = 40
    kv, ref = make(code, 16, 2, 64, 1, 4)
    x = np.zeros((n, 2, 64), dtype=np.float32)
    x[0, 0, :4] = [1e-38, -3e-39, 2.0 ** -100, 1e-30]
    x[1, 1, :4] = [3e38, -3e38, 1.0, -1e30]
    append(kv, ref, 0, [0], [0], [n], x, -x, "f32", max_seqlen=hint)
    check(kv, ref, 0, 0, n)
    assert abi.gdn_kv_get_error(kv) == 0
    y = np.random.default_rng(1).standard_normal((n, 2, 64)).astype(np.float32)
    y[0, 0, 0], y[1, 0, 1], y[n - 1, 1, 63] = np.nan, np.inf, -np.inf
    append(kv, ref, 0, [0], [16], [n], y, y[::-1].copy(), "f32", max_seqlen=hint)
    check(kv, ref, 0, 0, 16 + n)
    assert abi.gdn_kv_get_error(kv) == abi.DEVERR_VALUE
    assert abi.gdn_kv_get_error(kv) == 0


def test_rounding_ties_and_scale_limits():
    """Exact halves round to even; a block whose largest value is exactly
    top * 2^e takes that e, and the next float above takes the next."""
    for code, top in (("i8", 127.0), ("e4m3", 448.0)):
        kv, ref = make(code, 16, 1, 64, 4, 1)
        x = np.zeros((4, 1, 64), dtype=np.float32)
        x[0, 0] = np.arange(64) / 2 - 16
        x[0, 0, 0] = top
        x[1, 0, 0] = np.nextafter(np.float32(top), np.float32(1e9))
        x[1, 0, 1:] = np.arange(63) + 0.5
        x[2, 0, 0] = top / 8
        x[3, 0, :] = np.linspace(-17, 17, 64, dtype=np.float32)
        append(kv, ref, 0, [0, 1, 2, 3], [0] * 4, [1] * 4, x, x, "f32")
        for s in range(4):
            check(kv, ref, 0, s, 1)
        assert ref.scale["k"][0, ref.table[0, 0], 0] == 1.0
        assert ref.scale["k"][0, ref.table[1, 0], 0] == 2.0


@pytest.mark.parametrize("hint", [1, 8, 9, 100000])
def test_any_length_hint_is_correct(hint):
    rng = np.random.default_rng(hint)
    kv, ref = make("e4m3", 32, 2, 128, 3, 4, n_layers=2)
    lens = [100, 0, 1]
    k, v = rows(rng, 101, 2, 128, "bf16"), rows(rng, 101, 2, 128, "bf16")
    append(kv, ref, 1, [2, 1, 0], [7, 0, 31], lens, k, v, "bf16", max_seqlen=hint)
    got_k = torch.empty(101, 2, 128, device="cuda")
    got_v = torch.empty_like(got_k)
    abi.gdn_kv_read(kv, 1, dev_i32([2, 1, 0]), dev_i32([7, 0, 31]), got_k, got_v,
                    cu_seqlens=cum(lens), max_seqlen=hint)
    want = np.concatenate([ref.values(1, 2, "k", 7, 107), ref.values(1, 0, "k", 31, 32)])
    assert np.array_equal(got_k.double().cpu().numpy(), want)
    want = np.concatenate([ref.values(1, 2, "v", 7, 107), ref.values(1, 0, "v", 31, 32)])
    assert np.array_equal(got_v.double().cpu().numpy(), want)


def test_strided_rows_other_streams_and_one_side():
    """Keys and values as columns of one projection's rows, on a side stream;
    read-back of one side into strided rows leaves the rest alone."""
    rng = np.random.default_rng(9)
    kv, ref = make("i8", 64, 2, 64, 2, 2)
    x = rows(rng, 70, 6, 64, "bf16")
    wide = dev(x, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    slots, pos, cu = dev_i32([1]), dev_i32([5]), cum([70])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        abi.gdn_kv_append(kv, 0, slots, pos, wide[:, 2:4], wide[:, 4:6], cu_seqlens=cu)
        out = torch.full((70, 6, 64), 5.0, device="cuda", dtype=torch.bfloat16)
        abi.gdn_kv_read(kv, 0, slots, pos, None, out[:, 2:4], cu_seqlens=cu)
    side.synchronize()
    ref.append(0, [1], [5], [70], x[:, 2:4], x[:, 4:6])
    got = out.double().cpu().numpy()
    assert np.array_equal(got[:, 2:4], ref.values(0, 1, "v", 5, 75))
    assert (got[:, :2] == 5).all() and (got[:, 4:] == 5).all()


def test_bad_entries_are_skipped_and_reported():
    """Without host checks a bad slot, range or page skips its entry (or page)
    and sets a bit; the other entries are written."""
    rng = np.random.default_rng(11)
    kv, ref = make("i8", 16, 1, 64, 3, 2)
    before = kv.k.clone()
    k, v = rows(rng, 3, 1, 64, "f32"), rows(rng, 3, 1, 64, "f32")
    abi.gdn_kv_append(kv, 0, dev_i32([3, -1, 1]), dev_i32([0, 0, 32]), dev(k), dev(v))
    assert abi.gdn_kv_get_error(kv) == abi.DEVERR_SLOT | abi.DEVERR_SEQ
    abi.gdn_kv_append(kv, 0, dev_i32([0, 1, 2]), dev_i32([-1, 31, 2 ** 31 - 1]), dev(k), dev(v))
    assert abi.gdn_kv_get_error(kv) == abi.DEVERR_SEQ
    changed = (kv.k[0].view(torch.uint8) != before[0].view(torch.uint8)).flatten(1).any(1)
    assert changed.nonzero().flatten().tolist() == [int(ref.table[1, 1])]
    for bad in (-1, int(kv.desc.n_pages)):
        kv.page_table[0, 0] = bad
        x = rows(rng, 20, 1, 64, "f32")
        for hint in (1, 20):
            abi.gdn_kv_append(kv, 0, dev_i32([0]), dev_i32([0]), dev(x), dev(x),
                              cu_seqlens=cum([20]), max_seqlen=hint)
            assert abi.gdn_kv_get_error(kv) == abi.DEVERR_PAGE
        ref2 = KVOracle(1, kv.desc.n_pages, 1, 16, 64, "i8", ref.table)
        ref2.append(0, [0], [16], [4], x[16:], x[16:])
        out = torch.full((20, 1, 64), 3.0, device="cuda")
        abi.gdn_kv_read(kv, 0, dev_i32([0]), dev_i32([0]), out, None, cu_seqlens=cum([20]))
        assert abi.gdn_kv_get_error(kv) == abi.DEVERR_PAGE
        got = out.double().cpu().numpy()
        assert (got[:16] == 3).all()
        assert np.array_equal(got[16:], ref2.values(0, 0, "k", 16, 20))
    abi.gdn_kv_append(kv, 0, dev_i32([0, 1]), dev_i32([0, 0]), dev(k), dev(v),
                      cu_seqlens=dev_i32([2, 1, 9]))
    assert abi.gdn_kv_get_error(kv) == abi.DEVERR_SEQ


def test_refusals_with_host_checks():
    kv, _ = make("i8", 16, 2, 64, 4, 2, h_q=4, checks=True)
    k = torch.zeros(2, 2, 64, device="cuda")
    q = torch.zeros(2, 4, 64, device="cuda")

    def refused(name, call, *args, **kw):
        with pytest.raises(abi.GDNError) as e:
            call(kv, 0, *args, **kw)
        assert e.value.name == name, e.value

    a, r, t = abi.gdn_kv_append, abi.gdn_kv_read, abi.gdn_kv_attend
    refused("GDN_ERR_SLOT", a, dev_i32([0, 4]), dev_i32([0, 0]), k, k)
    refused("GDN_ERR_DUP_SLOT", a, dev_i32([1, 1]), dev_i32([0, 0]), k, k)
    refused("GDN_ERR_SIZE", a, dev_i32([0, 1]), dev_i32([0, 32]), k, k)
    refused("GDN_ERR_SIZE", a, dev_i32([0, 1]), dev_i32([0, -1]), k, k)
    refused("GDN_ERR_SIZE", r, dev_i32([0]), dev_i32([31]), k, k, cu_seqlens=dev_i32([0, 2]))
    refused("GDN_ERR_SIZE", a, dev_i32([0]), dev_i32([0]), k, k, cu_seqlens=dev_i32([0, 1]))
    refused("GDN_ERR_SIZE", a, dev_i32([0]), dev_i32([0]), k, k)
    refused("GDN_ERR_SIZE", t, dev_i32([0, 1]), dev_i32([1, 33]), q)
    refused("GDN_ERR_SIZE", t, dev_i32([0, 1]), dev_i32([1, -1]), q)
    refused("GDN_ERR_ARG", t, dev_i32([0, 1]), dev_i32([1, 1]), q, scale=float("nan"))
    refused("GDN_ERR_SIZE", t, dev_i32([0, 1]), dev_i32([1, 1]), q[:, :2])
    refused("GDN_ERR_DTYPE", t, dev_i32([0, 1]), dev_i32([1, 1]), q.half())
    refused("GDN_ERR_ARG", a, dev_i32([0, 1]), dev_i32([0, 0]), k.transpose(1, 2).contiguous()
            .transpose(1, 2), k)
    refused("GDN_ERR_ARG", a, dev_i32([0, 1]).long(), dev_i32([0, 0]), k, k)
    odd = torch.zeros(2 * 129 + 1, device="cuda")[1:].as_strided((2, 2, 64), (129, 64, 1))
    refused("GDN_ERR_ARG", a, dev_i32([0, 1]), dev_i32([0, 0]), odd, k)
    kv.page_table[2, 1] = -1
    refused("GDN_ERR_SIZE", a, dev_i32([2]), dev_i32([15]), k, k, cu_seqlens=dev_i32([0, 2]))
    refused("GDN_ERR_SIZE", t, dev_i32([2, 1]), dev_i32([17, 1]), q)
    abi.gdn_kv_append(kv, 0, dev_i32([2, 3]), dev_i32([15, 31]), k, k)
    # two entries may read one slot
    abi.gdn_kv_attend(kv, 0, dev_i32([2, 2]), dev_i32([16, 15]), q)
    empty = torch.zeros(0, 2, 64, device="cuda")
    abi.gdn_kv_append(kv, 0, dev_i32([]), dev_i32([]), empty, empty)
    assert abi.gdn_kv_get_error(kv) == 0
    other = torch.zeros(1, 5, 2, 24, 64, dtype=torch.int8, device="cuda")
    s = torch.zeros(1, 5, 2, device="cuda")
    with pytest.raises(abi.GDNError) as e:
        abi.KVCache(other, other.clone(), s, s.clone(), kv.page_table, 4)
    assert e.value.name == "GDN_ERR_UNSUPPORTED"

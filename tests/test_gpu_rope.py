"""Rotary positions (gdn_rope) against a 64-bit form on the CPU.

Tolerance.  Sine and cosine come from a reduced angle that is right to |p| 2^-52 of a turn (2 pi
of that in radians; the 64-bit form itself errs as much); sincospi is within 2 units of 2^-24,
the correction, the scale and the two products and their sum round once each: 7 roundings of
2^-24 relative to s (|a| + |b|).  A bf16 result is rounded once more, half a step: 2^-8 of itself
(and half a step at the smallest normal number)."""
import math

import numpy as np
import pytest
import torch

from gated_deltanet_recurrent_gb300 import abi

pytestmark = pytest.mark.gpu


def theta(rot, base=10000.0, factor=1.0, original_len=0, low_turns=1.0, high_turns=32.0, **_):
    out = []
    for j in range(rot // 2):
        f = math.exp(-2 * j / rot * math.log(base))
        if original_len:
            n = f * original_len / (2 * math.pi)
            m = min(1.0, max(0.0, (n - low_turns) / (high_turns - low_turns)))
            f = f * m + f / factor * (1 - m)
        else:
            f = f / factor
        out.append(f)
    return np.array(out)


def rotated(x, positions, rot, layout, out_scale=1.0, **rule):
    """x [tokens, heads, d] in 64 bits, and what its elements may be off by in float32."""
    x = x.double().cpu().numpy()
    angle = np.asarray(positions, np.float64)[:, None, None] * theta(rot, **rule)
    c, s = np.cos(angle) * out_scale, np.sin(angle) * out_scale
    at = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else \
        (slice(0, rot, 2), slice(1, rot, 2))
    a, b = x[..., at[0]], x[..., at[1]]
    y, off = x.copy(), np.zeros_like(x)
    y[..., at[0]], y[..., at[1]] = a * c - b * s, b * c + a * s
    far = np.abs(np.asarray(positions, np.float64))[:, None, None] * 2.0 ** -51 * 2 * math.pi
    size = (np.abs(a) + np.abs(b)) * abs(out_scale) * (7 * 2.0 ** -24 + far)
    off[..., at[0]], off[..., at[1]] = size, size
    return y, off


def check(got, want, off):
    if got.dtype == torch.bfloat16:
        off = off + 2.0 ** -8 * np.abs(want) * (off > 0) + 2.0 ** -134
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= off).all(), float((err - off).max())


def positions_of(n, most, seed=0):
    p = np.random.default_rng(seed).integers(-most, most + 1, n)
    p[-1] = most
    p[0] = 0
    return p


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


SHAPES = [(256, 64), (128, 128), (64, 24), (96, 10), (6, 2), (128, 126), (512, 512), (100, 52)]


@pytest.mark.parametrize("d,rot", SHAPES)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,h_q,h_k", [(1, 16, 2), (7, 3, 1), (333, 1, 1)])
def test_columns_of_a_projection(d, rot, layout, dtype, tokens, h_q, h_k):
    gen = torch.Generator(device="cuda").manual_seed(d + rot)
    rows = torch.randn(tokens, (h_q + 2 * h_k) * d, generator=gen, device="cuda").to(dtype)
    q = rows[:, :h_q * d].unflatten(1, (h_q, d))
    k = rows[:, h_q * d:(h_q + h_k) * d].unflatten(1, (h_k, d))
    p = positions_of(tokens, 40000)
    rope = abi.Rope(d, rot, layout)
    q_out, k_out = torch.empty(tokens, h_q, d, dtype=dtype, device="cuda"), torch.empty(
        tokens, h_k, d, dtype=dtype, device="cuda")
    before = rows.clone()
    abi.gdn_rope(rope, i32(p), q, k, q_out, k_out)
    assert torch.equal(rows, before)
    want = [rotated(x, p, rot, layout) for x in (q, k)]
    check(q_out, *want[0])
    check(k_out, *want[1])
    # in place: the same bits, and nothing else of the rows
    abi.gdn_rope(rope, i32(p), q, k)
    assert torch.equal(q, q_out) and torch.equal(k, k_out)
    assert torch.equal(rows[:, (h_q + h_k) * d:], before[:, (h_q + h_k) * d:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_tokens(layout, dtype):
    """Several tokens per block, the last block not full."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(5003, 5, 64, generator=gen, device="cuda").to(dtype)
    p = positions_of(5003, 1 << 20)
    rope = abi.Rope(64, 32, layout)
    out, none = abi.gdn_rope(rope, i32(p), q, q_out=torch.empty_like(q))
    assert none is None
    check(out, *rotated(q, p, 32, layout))


@pytest.mark.parametrize("d,rot,start", [(4096, 64, 0), (4096, 512, 0), (2048, 510, 0), (1024, 512, 1)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens", [3, 4100])
def test_heads_with_more_places_than_a_block_has_threads(d, rot, start, layout, dtype, tokens):
    x = torch.randn(tokens * d + 8, device="cuda").to(dtype)[start:start + tokens * d]
    x = x.view(tokens, 1, d)
    p = positions_of(tokens, 9000)
    out, _ = abi.gdn_rope(abi.Rope(d, rot, layout), i32(p), x, q_out=torch.empty_like(x))
    check(out, *rotated(x, p, rot, layout))


@pytest.mark.parametrize("shift", [1, 2, 3, 4])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_any_alignment(shift, layout, dtype):
    """Rows whose start and stride are multiples of a few elements only."""
    store = torch.randn(40 * 540, device="cuda").to(dtype)
    x = store[shift:].as_strided((40, 4, 128), (528 + shift, 128, 1))
    y = torch.zeros(40 * 540, device="cuda", dtype=dtype)[:40 * (513 + shift)].view(40, -1)[:, :512]
    y = y.unflatten(1, (4, 128))
    p = positions_of(40, 5000)
    want = rotated(x, p, 64, layout)
    abi.gdn_rope(abi.Rope(128, 64, layout), i32(p), None, x, None, y)
    check(y, *want)


RULES = [dict(factor=4.0), dict(base=500000.0), dict(base=1e6, factor=0.5),
         dict(factor=8.0, original_len=8192, low_turns=1.0, high_turns=32.0,
              out_scale=0.1 * math.log(8) + 1),
         dict(base=500000.0, factor=32.0, original_len=4096, low_turns=0.0, high_turns=4.0),
         dict(out_scale=-0.5), dict(base=0.5)]


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_scaled_for_long_contexts(rule, layout):
    x = torch.randn(50, 2, 128, device="cuda")
    p = positions_of(50, 1 << 20)
    got, _ = abi.gdn_rope(abi.Rope(128, 96, layout, **rule), i32(p), x, q_out=torch.empty_like(x))
    check(got, *rotated(x, p, 96, layout, **rule))


def test_the_ends_of_int32():
    x = torch.randn(4, 1, 64, device="cuda")
    p = np.array([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, -1])
    got, _ = abi.gdn_rope(abi.Rope(64), i32(p), x, q_out=torch.empty_like(x))
    check(got, *rotated(x, p, 64, "half"))


def test_whole_turns_are_nothing():
    """base 1, one turn a position: theta_j = 2 pi cannot be set, but 2 pi / 8 of it can by factor;
    eight positions on is where it began, a million positions on too."""
    x = torch.randn(3, 2, 8, device="cuda")
    rope = abi.Rope(8, base=1.0, factor=8 / (2 * math.pi))
    p = np.array([3, 3 + 8, 3 + 8 * 131072])
    x[1:] = x[0]
    got, _ = abi.gdn_rope(rope, i32(p), x, q_out=torch.empty_like(x))
    assert (got[1:] - got[0]).abs().max() <= 4 * 2.0 ** -24 * x.abs().max()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_the_gradient_is_the_rotation_back(layout):
    """<R x, y> = <x, R(-p) y> in both, and differences of the loss say the same."""
    x, y = torch.randn(2, 9, 3, 32, device="cuda")
    p = positions_of(9, 300)
    rope = abi.Rope(32, 20, layout)
    fwd = lambda z: abi.gdn_rope(rope, i32(p), z, q_out=torch.empty_like(z))[0]
    grad, _ = abi.gdn_rope(rope, i32(-p), y, q_out=torch.empty_like(y))
    want, off = rotated(y, -p, 20, layout)
    check(grad, want, off)
    loss = lambda z: float((fwd(z).double() * y.double()).sum())
    for t, h, j in ((0, 0, 0), (4, 1, 7), (8, 2, 19), (3, 0, 25)):
        e = torch.zeros_like(x)
        e[t, h, j] = 1.0
        # the loss is linear: a difference of any step is exact but for rounding, which for the
        # token's 32 values of 7 roundings is at most
        size = 2 * 7 * 2.0 ** -24 * float(((x[t, h].abs() + 1).sum() * y[t, h].abs().max()) * 2)
        assert abs(loss(x + e) - loss(x) - float(grad[t, h, j])) <= size + 1e-6


def test_infinities_stay_in_their_pairs():
    x = torch.randn(2, 2, 64, device="cuda")
    x[0, 0, 3], x[1, 1, 40] = math.inf, math.nan
    got, _ = abi.gdn_rope(abi.Rope(64, 32), i32([5, 6]), x, q_out=torch.empty_like(x))
    bad = ~torch.isfinite(got)
    want = torch.zeros_like(bad)
    want[0, 0, 3] = want[0, 0, 19] = want[1, 1, 40] = True
    assert torch.equal(bad, want)


def test_empty_calls_and_single_sides():
    rope = abi.Rope(64)
    none = torch.empty(0, 4, 64, device="cuda")
    abi.gdn_rope(rope, i32([]), none, none)
    k = torch.randn(3, 2, 64, device="cuda")
    got = abi.gdn_rope(rope, i32([1, 2, 3]), None, k, None, torch.empty_like(k))[1]
    both = abi.gdn_rope(rope, i32([1, 2, 3]), k, k, torch.empty_like(k), torch.empty_like(k))
    assert torch.equal(got, both[0]) and torch.equal(got, both[1])


def test_captured_and_replayed_with_other_positions():
    x = torch.randn(6, 4, 64, device="cuda")
    p, out = i32(range(6)), torch.empty_like(x)
    rope = abi.Rope(64)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        abi.gdn_rope(rope, p, x, q_out=out)
    for start in (7, 100000):
        p.copy_(i32(np.arange(6) + start))
        graph.replay()
        torch.cuda.synchronize()
        check(out, *rotated(x, np.arange(6) + start, 64, "half"))


def test_another_stream():
    x = torch.randn(300, 4, 64, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out, _ = abi.gdn_rope(abi.Rope(64), i32(range(300)), x, q_out=torch.empty_like(x), stream=s)
    s.synchronize()
    check(out, *rotated(x, np.arange(300), 64, "half"))

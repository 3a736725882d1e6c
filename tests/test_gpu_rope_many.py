"""As many tokens as an int32 counts, in place."""
import pytest
import torch

from gated_deltanet_recurrent_gb300 import abi

pytestmark = pytest.mark.gpu


def test_the_most_tokens():
    n = 2 ** 31 - 1
    q = torch.empty(n, 1, 2, dtype=torch.bfloat16, device="cuda")
    q[..., 0], q[..., 1] = 1, 0
    at = torch.arange(n, dtype=torch.int32, device="cuda")
    abi.gdn_rope(abi.Rope(2), at, q)
    # |p| 2^-52 of a turn, 7 roundings of 2^-24 and one of bf16, of sines and cosines
    for rows in (slice(0, 5000), slice(2 ** 30 - 2000, 2 ** 30 + 3000), slice(n - 5000, n)):
        p = at[rows].double()
        want = torch.stack([p.cos(), p.sin()], 1)
        off = 2 * 3.15 * 2.0 ** -52 * p[:, None] * 2 + 7 * 2.0 ** -24 + 2.0 ** -8 * want.abs()
        assert ((q[rows, 0].double() - want).abs() <= off).all()

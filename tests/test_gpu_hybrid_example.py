"""The hybrid example: recurrent layers and attention over the 8-bit cache on
one set of slots.  Feeding a prompt at once, and feeding its first part and
then the rest token by token, have to lead to the same hidden states.

Tolerance: both ways round activations to bf16 (2^-8) at each of three layers'
inputs and outputs, and a page that grows token by token has codes that were
rounded once more than those of a page written at once (int8: half a step of
2^-7 of the page's largest magnitude, at most).  3 layers x (3 roundings x 2^-8 +
2^-8) = 0.047 of the largest magnitude bounds them together."""
import pytest
import torch

from examples.hybrid_decode import HIDDEN, Hybrid
from gated_deltanet_recurrent_gb300 import abi

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("code", [torch.int8, torch.float8_e4m3fn])
def test_a_prompt_at_once_and_token_by_token_agree(code):
    gen = torch.Generator(device="cuda").manual_seed(3)
    lens, tail = [75, 23], 6
    x = [torch.randn(n, HIDDEN, generator=gen, device="cuda").to(torch.bfloat16) for n in lens]
    whole = Hybrid(code=code)
    slots = i32([1, 3])
    abi.gdn_pool_reset(whole.pool, slots)
    cu = i32([0, lens[0], sum(lens)])
    at_once = whole.forward(torch.cat(x), slots, i32([0, 0]), cu, longest=max(lens))
    parts = Hybrid(code=code)
    abi.gdn_pool_reset(parts.pool, slots)
    head = [n - tail for n in lens]
    parts.forward(torch.cat([v[:n] for v, n in zip(x, head)]), slots, i32([0, 0]),
                  i32([0, head[0], sum(head)]), longest=max(head))
    for t in range(tail):
        step = torch.stack([v[n + t] for v, n in zip(x, head)])
        out = parts.forward(step, slots, i32([n + t for n in head]))
        want = at_once[torch.tensor([head[0] + t, lens[0] + head[1] + t], device="cuda")]
        err = (out.float() - want.float()).abs().max()
        assert err <= 0.047 * want.float().abs().max(), (t, float(err))
    assert whole.errors() == 0 and parts.errors() == 0


def test_the_example_runs(capsys):
    from examples import hybrid_decode
    hybrid_decode.main()
    out = capsys.readouterr().out
    assert "lengths [108, 25, 72]" in out and "errors 0" in out and "nan" not in out

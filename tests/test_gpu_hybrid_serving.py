"""Pages handed out on the GPU, rotary positions and adapters per request, together in the hybrid
example: project, rotate, grow the cache, append, attend.

Tolerance, as for the example without them: activations are rounded to bf16 (2^-8) at each of three
layers' inputs and outputs, once more where positions are rotated, and the codes of a page that grows
token by token are rounded once more (int8: 2^-8 of its largest magnitude): (3 x 4 + 1) x 2^-8 = 0.051
of the largest magnitude bounds them together."""
import pytest
import torch

from examples.hybrid_decode import ATTN, HIDDEN, PAGE, Hybrid
from gated_deltanet_recurrent_gb300 import abi

pytestmark = pytest.mark.gpu
TOL = 0.051


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def tokens(n, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, HIDDEN, generator=gen, device="cuda").to(torch.bfloat16)


def per_token(ids, lens):
    return i32([a for a, n in zip(ids, lens) for _ in range(n)])


def near(got, want):
    err = (got.float() - want.float()).abs().max()
    assert err <= TOL * want.float().abs().max(), float(err)


def test_a_prompt_at_once_and_token_by_token_agree():
    lens, tail, ids = [75, 23], 6, [1, 0]
    x = [tokens(n, i) for i, n in enumerate(lens)]
    make = lambda: Hybrid(rope=True, n_pages=12, adapters=2)
    whole, parts, slots = make(), make(), i32([1, 3])
    abi.gdn_pool_reset(whole.pool, slots)
    abi.gdn_pool_reset(parts.pool, slots)
    at_once = whole.forward(torch.cat(x), slots, i32([0, 0]), i32([0, 75, 98]), longest=75,
                            ids=per_token(ids, lens))
    head = [n - tail for n in lens]
    parts.forward(torch.cat([v[:n] for v, n in zip(x, head)]), slots, i32([0, 0]),
                  i32([0, head[0], sum(head)]), longest=max(head), ids=per_token(ids, head))
    for t in range(tail):
        out = parts.forward(torch.stack([v[n + t] for v, n in zip(x, head)]), slots,
                            i32([n + t for n in head]), ids=i32(ids))
        near(out, at_once[torch.tensor([head[0] + t, lens[0] + head[1] + t], device="cuda")])
    assert parts.pages.held.tolist() == whole.pages.held.tolist() == [0, 5, 0, 2]
    assert whole.errors() == 0 and parts.errors() == 0


def test_a_request_is_what_it_is_alone():
    """Other requests' adapters, pages and positions change nothing of one's own."""
    lens, ids = [40, 33, 50, 17], [2, -1, 0, 2]
    x = [tokens(n, 10 + i) for i, n in enumerate(lens)]
    both = Hybrid(rope=True, n_pages=16, adapters=3)
    slots = i32([2, 0, 3, 1])
    abi.gdn_pool_reset(both.pool, slots)
    cu = [0, 40, 73, 123, 140]
    out = both.forward(torch.cat(x), slots, i32([0] * 4), i32(cu), longest=50,
                       ids=per_token(ids, lens))
    for i, n in enumerate(lens):
        alone = Hybrid(rope=True, n_pages=16, adapters=3)
        abi.gdn_pool_reset(alone.pool, i32([0]))
        near(out[cu[i]:cu[i + 1]], alone.forward(x[i], i32([0]), i32([0]), i32([0, n]), longest=n,
                                                 ids=per_token(ids[i:i + 1], [n])))
    assert both.errors() == 0


def test_adapters_and_positions_matter():
    x, slots, cu = tokens(30, 5), i32([0]), i32([0, 30])
    def run(ids, **kw):
        m = Hybrid(n_pages=8, adapters=2, **kw)
        abi.gdn_pool_reset(m.pool, slots)
        return m.forward(x, slots, i32([0]), cu, longest=30, ids=per_token(ids, [30])).float()
    base = run([-1], rope=True)
    for other in (run([0], rope=True), run([1], rope=True), run([-1])):
        assert (other - base).abs().max() > TOL * base.abs().max()


def test_rejected_drafts_and_finished_requests_give_pages_back():
    m = Hybrid(rope=True, n_pages=9, adapters=1)
    slots = i32([3, 1])
    abi.gdn_pool_reset(m.pool, slots)
    m.forward(tokens(60, 1), slots, i32([0, 0]), i32([0, 30, 60]), longest=30, ids=i32([0] * 60))
    assert m.pages.held.tolist() == [0, 2, 0, 2]
    m.forward(tokens(10, 2), slots, i32([30, 30]), i32([0, 5, 10]), longest=5, ids=i32([0] * 10))
    assert m.pages.held.tolist() == [0, 3, 0, 3] and m.pages.n_free.item() == 3
    m.release(slots, i32([31, 33]))                      # one of five drafts accepted, and three
    assert m.pages.held.tolist() == [0, 3, 0, 2] and m.pages.n_free.item() == 4
    m.release(slots, i32([0, 0]))
    assert m.pages.n_free.item() == 9 and (m.kv.page_table == -1).all()
    assert m.errors() == 0


def test_the_attention_layers_input_against_64_bits():
    """One attention layer: what reaches the cache is the adapted projection, rotated.  The values in
    the cache are off by half an int8 step of their page (2^-7 of its largest magnitude: the scale is
    a power of two) after the projection's and the rotation's bf16 roundings (2^-8 each)."""
    m = Hybrid(layers="a", rope=True, n_pages=16, adapters=2)
    a, p = ATTN, m.params[0]
    lens, ids = [20, 45], [1, 0]
    x = tokens(65, 9)
    slots, cu = i32([2, 0]), i32([0, 20, 65])
    m.forward(x, slots, i32([0, 0]), cu, longest=45, ids=per_token(ids, lens))
    ad = p["adapters"]
    y = x.double() @ p["in"].double().T
    for t, i in enumerate(per_token(ids, lens).tolist()):
        y[t] += 0.5 * (ad.b[i].double() @ (ad.a[i].double() @ x[t].double()))
    k = y[:, a["h_q"] * a["d"]:(a["h_q"] + a["h_kv"]) * a["d"]].unflatten(1, (a["h_kv"], a["d"]))
    rot = a["d"] // 4
    at = torch.cat([torch.arange(n, device="cuda") for n in lens]).double()
    angle = at[:, None, None] * 10000.0 ** (-2 * torch.arange(rot // 2, device="cuda").double() / rot)
    lo, hi = k[..., :rot // 2].clone(), k[..., rot // 2:rot].clone()
    k[..., :rot // 2] = lo * angle.cos() - hi * angle.sin()
    k[..., rot // 2:rot] = hi * angle.cos() + lo * angle.sin()
    back = torch.empty(65, a["h_kv"], a["d"], device="cuda")
    abi.gdn_kv_read(m.kv, 0, slots, i32([0, 0]), back, None, cu_seqlens=cu)
    for first, n in ((0, 20), (20, 45)):
        for page in range(0, n, PAGE):
            rows = slice(first + page, first + min(n, page + PAGE))
            top = k[rows].abs().amax((0, 2), keepdim=True)
            err = (back[rows].double() - k[rows]).abs()
            assert (err <= (2.0 ** -7 + 4 * 2.0 ** -8) * top).all(), float((err / top).max())
    assert m.errors() == 0


def test_the_whole_run_in_a_graph():
    """A decode step captured once and replayed: the pages grow on the GPU as it goes."""
    eager, graphed = (Hybrid(rope=True, n_pages=16, adapters=2, host_checks=False)
                      for _ in range(2))
    slots, ids = i32([0, 2]), i32([1, -1])
    x = tokens(24, 3)
    for m in (eager, graphed):
        abi.gdn_pool_reset(m.pool, slots)
        m.forward(x, slots, i32([0, 0]), i32([0, 15, 24]), longest=15, ids=per_token([1, -1], [15, 9]))
    pos, step = i32([15, 9]), tokens(2, 4)
    static_x, static_pos = step.clone(), pos.clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = graphed.forward(static_x, slots, static_pos, ids=ids, longest_context=256)
    for t in range(20):
        step = tokens(2, 100 + t)
        static_x.copy_(step), static_pos.copy_(pos)
        graph.replay()
        want = eager.forward(step, slots, pos, ids=ids, longest_context=256)
        assert torch.equal(out, want), t
        pos = pos + 1
    assert graphed.pages.held.tolist() == eager.pages.held.tolist() == [3, 0, 2, 0]
    assert graphed.errors() == 0 and eager.errors() == 0

"""The operators around an attention layer's cache, as cases that can be timed and compared.

  pages    pages of the KV cache for the tokens that a step adds, taken from a list of free pages
           in device memory, with each token's position and cache row; and given back
  rope     rotary positions on the query and key heads of packed tokens
  adapted  the shared input projection with a low-rank adapter per token:
           y[t] = W x[t] + c[a] B[a] (A[a] x[t]),  a = ids[t], or W x[t] alone where ids[t] = -1

With `own` false, run() computes them with elementary torch operations in 32
bits (angles in 64); with `own` true it calls the library's entry points on the
same data.
"""
import math
import random

import torch

own = False

#: heads: query heads, KV heads, head dimension
HEADS = {
    "16x2x256": (16, 2, 256),
    "32x8x128": (32, 8, 128),
    "28x4x128": (28, 4, 128),
    "12x4x64": (12, 4, 64),
}
#: projections: hidden size, outputs
PROJ = {
    "2048-12352": (2048, 12352),  # a recurrent layer's: q | k | v, gate, decay and beta logits
    "2048-5120": (2048, 5120),    # an attention layer's: 16 query and 2 + 2 KV heads of 256
    "2048-2048": (2048, 2048),    # a square one
    "512-1040": (512, 1040),      # a small layer's, outputs that fill no tile
}


def _named(name, c):
    return {"name": name, **c} if name else c


def _pages(name, n, new, ctx, page, short=False):
    """n sequences of up to `new` new tokens, up to `ctx` tokens each with them; short: there are
    fewer free pages than they need."""
    return _named(name, {"op": "pages", "n": n, "new": new, "ctx": ctx, "page": page,
                         "short": short})


def _rope(name, tokens, heads, rot, layout, dtype, far, scaled):
    """positions below `far`; scaled: "no", "even" or "turns" (see _frequencies)."""
    return _named(name, {"op": "rope", "tokens": tokens, "heads": heads, "rot": rot,
                         "layout": layout, "dtype": dtype, "far": far, "scaled": scaled})


def _adapted(name, tokens, proj, rank, adapters, run, out):
    """`run`: the longest run of tokens with one adapter (1: every token draws its own)."""
    return _named(name, {"op": "adapted", "tokens": tokens, "proj": proj, "rank": rank,
                         "adapters": adapters, "run": run, "out": out})


def listed():
    return [
        # one request's next token needs a page: nothing but latency
        _pages("pages-one", 1, 1, 1025, 64),
        # a decode step of a usual batch: most tokens fit the page that is open
        _pages("pages-step", 256, 1, 8192, 64),
        # a batch of whole prompts comes in, small pages
        _pages("pages-prompts", 64, 8192, 8192, 16),
        # many long prompts of which the last find no page any more
        _pages("pages-short", 301, 1777, 32768, 32, True),
        # one request's next token, a quarter of each head rotated
        _rope("rope-one", 1, "16x2x256", 64, "half", "bf16", 8192, "no"),
        # a full decode batch, whole heads, neighbouring pairs
        _rope("rope-step", 256, "32x8x128", 128, "interleaved", "bf16", 32768, "even"),
        # pieces of prompts
        _rope("rope-prompts", 16384, "16x2x256", 64, "half", "bf16", 8192, "no"),
        # a model run in float32 over far positions, frequencies mixed by turns
        _rope("rope-far", 5003, "28x4x128", 128, "half", "f32", 1000000, "turns"),
        # one request's next token
        _adapted("adapted-one", 1, "2048-5120", 16, 8, 1, "bf16"),
        # a decode batch in which nearly every request brings its own adapter
        _adapted("adapted-step", 64, "2048-12352", 16, 64, 1, "bf16"),
        # decode tokens, drafts and short prompts of a float32 layer, packed
        _adapted("adapted-mixed", 777, "2048-5120", 32, 24, 100, "f32"),
        # pieces of prompts
        _adapted("adapted-prompts", 16384, "2048-12352", 64, 16, 2048, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(("pages-step", "pages-prompts", "rope", "rope", "adapted-step",
                       "adapted-prompts"))
    page = rng.choice((16, 32, 64, 128))
    if kind == "pages-step":
        new = _log_int(rng, 1, 8)
        return _pages("", _log_int(rng, 1, 512), new, _log_int(rng, 16, 32768), page,
                      rng.random() < 0.3)
    if kind == "pages-prompts":
        new = _log_int(rng, 9, 8192)
        n = _log_int(rng, 1, min(512, 64 * 8192 // new))
        return _pages("", n, new, _log_int(rng, new, 32768), page, rng.random() < 0.3)
    if kind == "rope":
        heads = rng.choice(sorted(HEADS))
        d = HEADS[heads][2]
        rot = rng.choice((d, d, d // 2, d // 4, 2 * rng.randint(1, d // 2)))
        return _rope("", _log_int(rng, 1, 16384), heads, rot,
                     rng.choice(("half", "interleaved")), rng.choice(("bf16", "bf16", "f32")),
                     _log_int(rng, 64, 1 << 20), rng.choice(("no", "even", "turns")))
    proj, rank = rng.choice(sorted(PROJ)), rng.choice((8, 16, 24, 32, 64, 128))
    out = rng.choice(("bf16", "bf16", "f32"))
    if kind == "adapted-step":
        return _adapted("", _log_int(rng, 1, 512), proj, min(rank, 64), _log_int(rng, 1, 64), 1,
                        out)
    tokens = _log_int(rng, 64, 8192)
    return _adapted("", tokens, proj, rank, _log_int(rng, 1, 32), _log_int(rng, 16, 4096), out)


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


# ------------------------------------------------------------- what a case holds

def _lens(case):
    """Per sequence: tokens held before, and new ones."""
    n, new, ctx = case["n"], case["new"], max(case["ctx"], case["new"])
    rnd = random.Random("%d/%d/%d" % (n, new, ctx))
    news = [rnd.randint(max(1, new // 4), new) for _ in range(n)]
    news[0] = new
    if n >= 4 and new > 1:
        news[-1] = 0  # a slot of the batch without new tokens in this step
    alls = [ctx] + [rnd.randint(max(x, ctx // 16), ctx) for x in news[1:]]
    return [a - x for a, x in zip(alls, news)], news


def _grants(case):
    """Per sequence: pages held before, pages it needs, and whether it gets them."""
    page = case["page"]
    before, news = _lens(case)
    held = [-(-p // page) for p in before]
    need = [-(-(p + x) // page) - h for p, x, h in zip(before, news, held)]
    n_free = sum(need) * 3 // 4 if case["short"] else sum(need) + 7
    got, total = [], 0
    for x in need:
        total += x
        got.append(x == 0 or total <= n_free)
    return held, need, got, n_free


def _ids(case):
    """Each token's adapter, or -1."""
    rnd = random.Random("%d/%d/%d" % (case["tokens"], case["adapters"], case["run"]))
    ids = []
    while len(ids) < case["tokens"]:
        a = rnd.randrange(case["adapters"]) if rnd.random() < 0.9 else -1
        run = 1 if case["run"] == 1 else rnd.randint(1, case["run"])
        ids += [a] * min(run, case["tokens"] - len(ids))
    return ids


def work(case):
    if case["op"] == "pages":
        before, news = _lens(case)
        _, need, got, _ = _grants(case)
        moved = sum(x for x, g in zip(need, got) if g)
        # a page moved: its free entry and its table entry, read and written once each way;
        # a token: its position and its row; a sequence: slot, position, offset, held, granted
        return {"bytes": 16 * moved + 12 * sum(news) + 36 * len(news), "flops": 0}
    if case["op"] == "rope":
        h_q, h_kv, d = HEADS[case["heads"]]
        size = 2 if case["dtype"] == "bf16" else 4
        heads = case["tokens"] * (h_q + h_kv)
        return {"bytes": 2 * heads * d * size + 4 * case["tokens"], "flops": 3 * heads * case["rot"]}
    hidden, n_out = PROJ[case["proj"]]
    ids = _ids(case)
    used, some = len(set(ids) - {-1}), sum(a >= 0 for a in ids)
    t, r = len(ids), case["rank"]
    size = 2 if case["out"] == "bf16" else 4
    return {"bytes": 2 * t * hidden + 2 * n_out * hidden + 2 * used * r * (hidden + n_out) +
            size * t * n_out + 4 * t,
            "flops": 2 * t * hidden * n_out + 2 * some * r * (hidden + n_out)}


# ------------------------------------------------------------------ inputs

def _pages_inputs(case, seed):
    """The state between two rounds: the slots hold their tokens and the new ones' pages."""
    dev, rnd = "cuda", random.Random(seed)
    i32 = dict(dtype=torch.int32, device=dev)
    page = case["page"]
    before, news = _lens(case)
    held, need, got, n_free = _grants(case)
    n = len(news)
    n_slots, max_pages = n + 3, max(-(-(p + x) // page) for p, x in zip(before, news)) + 1
    now = [h + (x if g else 0) for h, x, g in zip(held, need, got)]
    taken = sum(x for x, g in zip(need, got) if g)
    n_pages = sum(held) + n_free + 5
    gen = torch.Generator(device=dev).manual_seed(seed)
    order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    slots = rnd.sample(range(n_slots), n)
    rows = torch.repeat_interleave(torch.tensor(slots, device=dev), torch.tensor(now, device=dev))
    cols = torch.cat([torch.arange(c) for c in now]).to(dev)
    table = torch.full((n_slots, max_pages), -1, **i32)
    table[rows, cols] = order[:rows.numel()]
    held_t = torch.zeros(n_slots, **i32)
    held_t[torch.tensor(slots, device=dev)] = torch.tensor(now, **i32)
    free = torch.full((n_pages,), -1, **i32)
    left = n_free - taken
    free[:left] = order[rows.numel():rows.numel() + left]
    cum = [0]
    for x in news:
        cum.append(cum[-1] + x)
    total = cum[-1]
    single = total == n and max(news) == 1
    return {"case": dict(case), "page": page, "total": total, "moved": taken, "table": table,
            "held": held_t, "free": free, "n_free": torch.tensor([left], **i32),
            "slots": torch.tensor(slots, **i32), "pos": torch.tensor(before, **i32),
            "cu": None if single else torch.tensor(cum, **i32), "new": torch.tensor(news, **i32),
            "positions": torch.empty(total, **i32), "granted": torch.empty(n, **i32),
            "rows": torch.empty(total, dtype=torch.int64, device=dev)}


def _rope_inputs(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    h_q, h_kv, d = HEADS[case["heads"]]
    t, dtype = case["tokens"], _dtype(case["dtype"])
    # queries and keys are columns of one projection's rows, values after them
    rows = torch.randn(t, (h_q + 2 * h_kv) * d, generator=gen, device=dev).to(dtype)
    # runs of neighbouring positions from several starts, and the last position there is
    runs = max(1, t // 256)
    start = torch.randint(0, max(1, case["far"] - -(-t // runs)), (runs,), generator=gen,
                          device=dev)
    at = torch.arange(t, device=dev)
    positions = (start[at * runs // t] + at % 256).clamp(max=case["far"] - 1)
    positions[-1] = case["far"] - 1
    s = {"case": dict(case), "q": rows[:, :h_q * d].unflatten(1, (h_q, d)),
         "k": rows[:, h_q * d:(h_q + h_kv) * d].unflatten(1, (h_kv, d)),
         "positions": positions.to(torch.int32), "rule": _rule(case)}
    s["q_out"] = torch.empty(t, h_q, d, dtype=dtype, device=dev)
    s["k_out"] = torch.empty(t, h_kv, d, dtype=dtype, device=dev)
    return s


def _adapted_inputs(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    hidden, n_out = PROJ[case["proj"]]
    t, r, n = case["tokens"], case["rank"], case["adapters"]
    ids = _ids(case)

    def normal(*shape, by=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * by).to(torch.bfloat16)

    # the runs of tokens that share an adapter, which a program that packs its requests knows
    runs, first = [], 0
    for i in range(1, t + 1):
        if i == t or ids[i] != ids[first]:
            if ids[first] >= 0:
                runs.append((ids[first], first, i))
            first = i
    return {"case": dict(case), "x": normal(t, hidden), "w": normal(n_out, hidden, by=hidden ** -0.5),
            "a": normal(n, r, hidden, by=hidden ** -0.5), "b": normal(n, n_out, r, by=0.3 * r ** -0.5),
            "scale": 0.5 + torch.rand(n, generator=gen, device=dev),
            "ids": torch.tensor(ids, dtype=torch.int32, device=dev), "runs": runs,
            "y": torch.empty(t, n_out, dtype=_dtype(case["out"]), device=dev)}


_INPUTS = {"pages": _pages_inputs, "rope": _rope_inputs, "adapted": _adapted_inputs}


def prepare(case, seed):
    s = _INPUTS[case["op"]](case, seed)
    if not own:
        return s
    from gated_deltanet_recurrent_gb300 import abi
    s["abi"] = abi
    if case["op"] == "pages":  # the handles that a program keeps, on the same memory
        shape = (1, s["free"].numel(), 1, case["page"], 64)
        codes = [torch.zeros(shape, dtype=torch.int8, device="cuda") for _ in range(2)]
        scales = [torch.zeros(shape[:3], device="cuda") for _ in range(2)]
        s["cache"] = abi.KVCache(*codes, *scales, s["table"], h_q=1, host_checks=False)
        s["book"] = abi.KVPages(s["cache"], held=s["held"], free_pages=s["free"],
                                n_free=s["n_free"])
    elif case["op"] == "rope":
        rule = s["rule"]
        s["rope"] = abi.Rope(HEADS[case["heads"]][2], rot=case["rot"], layout=case["layout"],
                             base=rule["base"], factor=rule["factor"],
                             original_len=rule["original_len"], low_turns=rule["low_turns"],
                             high_turns=rule["high_turns"], out_scale=rule["out_scale"])
    else:
        s["pool"] = abi.Pool(1, 1, 1, 1, 16, 16, 48, 4, host_checks=False)
        s["adapters"] = abi.Adapters(s["a"], s["b"], s["scale"])
    return s


# -------------------------------------------------------------- plain forms

def _spread(count, total):
    """For each of `total` items, count[i] of them for i: its i, and its place among them."""
    i = torch.repeat_interleave(torch.arange(count.numel(), device="cuda"), count,
                                output_size=total)
    first = torch.cumsum(count, 0) - count
    return i, torch.arange(total, device="cuda") - first[i]


def _plain_pages(s):
    page, table, held, free = s["page"], s["table"], s["held"], s["free"]
    slots, pos, new = s["slots"].long(), s["pos"].long(), s["new"].long()
    # back to the tokens that were there before this round
    kept = (pos + page - 1) // page
    drop = (held[slots] - kept).clamp(min=0)
    i, j = _spread(drop, s["moved"])
    top = s["n_free"].long() + s["moved"]
    at = top - 1 - torch.arange(s["moved"], device="cuda")
    free[at] = table[slots[i], kept[i] + j]
    table[slots[i], kept[i] + j] = -1
    held[slots] = torch.minimum(held[slots], kept.to(torch.int32))
    # and pages for the new ones
    have = held[slots].long()
    need = ((pos + new + page - 1) // page - have).clamp(min=0)
    granted = (need == 0) | (torch.cumsum(need, 0) <= top)
    need = torch.where(granted, need, 0)
    i, j = _spread(need, s["moved"])
    table[slots[i], have[i] + j] = free[at]
    held[slots] = (have + need).to(torch.int32)
    s["n_free"].copy_(top - s["moved"])
    i, j = _spread(new, s["total"])
    p = pos[i] + j
    rows = table[slots[i], p // page].long() * page + p % page
    s["positions"].copy_(p)
    s["rows"].copy_(torch.where(granted[i], rows, -1))
    s["granted"].copy_(granted)
    return _pages_out(s)


def _pages_out(s):
    return {x: s[x] for x in ("positions", "rows", "granted", "table", "held", "free", "n_free")}


def _rule(case):
    """How a case's frequencies are scaled for long contexts."""
    rule = {"base": 10000.0, "factor": 1.0, "original_len": 0, "low_turns": 0.0,
            "high_turns": 0.0, "out_scale": 1.0}
    if case["scaled"] == "even":
        rule |= {"factor": 4.0, "base": 500000.0}
    if case["scaled"] == "turns":
        rule |= {"factor": 8.0, "original_len": 8192, "low_turns": 1.0, "high_turns": 32.0,
                 "out_scale": 0.1 * math.log(8.0) + 1.0}
    return rule


def _frequencies(rot, rule):
    """base^(-2j/rot); divided by the factor, or, with an original length, only as far as a pair
    makes few turns in it: wholly below low_turns, not at all above high_turns, linearly between."""
    j = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    theta = rule["base"] ** (-2 * j / rot)
    if not rule["original_len"]:
        return theta / rule["factor"]
    turns = theta * rule["original_len"] / (2 * math.pi)
    keep = ((turns - rule["low_turns"]) / (rule["high_turns"] - rule["low_turns"])).clamp(0, 1)
    return theta * (keep + (1 - keep) / rule["factor"])


def _plain_rope(s):
    rot, rule = s["case"]["rot"], s["rule"]
    angle = s["positions"].double()[:, None] * _frequencies(rot, rule)
    cos = (torch.cos(angle) * rule["out_scale"]).float()[:, None]
    sin = (torch.sin(angle) * rule["out_scale"]).float()[:, None]
    for x, out in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        if s["case"]["layout"] == "half":
            a, b = x[..., :rot // 2].float(), x[..., rot // 2:rot].float()
            out[..., :rot // 2] = a * cos - b * sin
            out[..., rot // 2:rot] = b * cos + a * sin
        else:
            a, b = x[..., 0:rot:2].float(), x[..., 1:rot:2].float()
            out[..., 0:rot:2] = a * cos - b * sin
            out[..., 1:rot:2] = b * cos + a * sin
        out[..., rot:] = x[..., rot:]
    return {"q": s["q_out"], "k": s["k_out"]}


def _plain_adapted(s):
    x, t = s["x"].float(), s["case"]["tokens"]
    y = x @ s["w"].float().T
    if s["case"]["run"] == 1:  # every token's own adapter, gathered
        for lo in range(0, t, 64):
            ids = s["ids"][lo:lo + 64].long()
            pick = ids.clamp(min=0)
            h = (s["a"][pick].float() @ x[lo:lo + 64, :, None]) * s["scale"][pick][:, None, None]
            delta = (s["b"][pick].float() @ h)[..., 0]
            y[lo:lo + 64] += torch.where(ids[:, None] >= 0, delta, 0.0)
    else:
        for a, lo, hi in s["runs"]:
            h = (x[lo:hi] @ s["a"][a].float().T) * s["scale"][a]
            y[lo:hi] += h @ s["b"][a].float().T
    s["y"].copy_(y)
    return {"y": s["y"]}


_PLAIN = {"pages": _plain_pages, "rope": _plain_rope, "adapted": _plain_adapted}


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return _PLAIN[op](s)
    abi = s["abi"]
    if op == "pages":
        abi.gdn_kv_pages_trim(s["cache"], s["book"], s["slots"], s["pos"])
        abi.gdn_kv_pages_grow(s["cache"], s["book"], s["slots"], s["pos"], cu_seqlens=s["cu"],
                              positions=s["positions"], rows=s["rows"], granted=s["granted"])
        return _pages_out(s)
    if op == "rope":
        abi.gdn_rope(s["rope"], s["positions"], s["q"], s["k"], s["q_out"], s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    abi.gdn_in_proj_adapted(s["pool"], s["adapters"], s["x"], s["w"], s["ids"], s["y"])
    return {"y": s["y"]}


# ------------------------------------------------- the definition, in 64 bits

def _exact_pages(s):
    page = s["page"]
    table, held = s["table"].tolist(), s["held"].tolist()
    free, n_free = s["free"].tolist(), int(s["n_free"])
    slots, pos, new = s["slots"].tolist(), s["pos"].tolist(), s["new"].tolist()
    back = []
    for slot, p in zip(slots, pos):
        keep = math.ceil(p / page)
        back += table[slot][keep:held[slot]]
        for c in range(keep, held[slot]):
            table[slot][c] = -1
        held[slot] = min(held[slot], keep)
    for x in reversed(back):
        free[n_free] = x
        n_free += 1
    asked, limit = 0, n_free
    out = {"positions": [], "rows": [], "granted": []}
    for slot, p, t in zip(slots, pos, new):
        last = math.ceil((p + t) / page)
        need = max(0, last - held[slot])
        asked += need
        ok = need == 0 or asked <= limit
        while ok and held[slot] < last:
            n_free -= 1
            table[slot][held[slot]] = free[n_free]
            held[slot] += 1
        out["granted"].append(int(ok))
        for u in range(p, p + t):
            out["positions"].append(u)
            out["rows"].append(table[slot][u // page] * page + u % page if ok else -1)
    out |= {"table": table, "held": held, "free": free, "n_free": [n_free]}
    return {x: torch.tensor(y, device="cuda", dtype=s[x].dtype) for x, y in out.items()}


def _exact_rope(s):
    case, rule = s["case"], s["rule"]
    rot = case["rot"]
    theta = []
    for j in range(rot // 2):
        f = math.exp(-2 * j / rot * math.log(rule["base"]))
        if rule["original_len"]:
            wave = 2 * math.pi / f
            turns = rule["original_len"] / wave
            keep = (turns - rule["low_turns"]) / (rule["high_turns"] - rule["low_turns"])
            keep = min(1.0, max(0.0, keep))
            f = keep * f + (1 - keep) * f / rule["factor"]
        else:
            f = f / rule["factor"]
        theta.append(f)
    angle = torch.outer(s["positions"].double(), torch.tensor(theta, dtype=torch.float64,
                                                              device="cuda"))
    turn = torch.polar(torch.full_like(angle, rule["out_scale"]), angle)[:, None]
    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        y = x.clone()
        if case["layout"] == "half":
            z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous())
            z = z * turn
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        else:
            z = torch.view_as_complex(x[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * turn
            y[..., :rot] = torch.view_as_real(z).flatten(-2)
        out[name] = y
    return out


def _exact_adapted(s):
    x, w = s["x"].double(), s["w"].double()
    y = torch.empty(x.shape[0], w.shape[0], dtype=torch.float64, device="cuda")
    for lo in range(0, x.shape[0], 4096):
        torch.mm(x[lo:lo + 4096], w.T, out=y[lo:lo + 4096])
    for a in range(s["a"].shape[0]):
        rows = (s["ids"] == a).nonzero()[:, 0]
        if rows.numel():
            low = torch.einsum("tk,rk->tr", x[rows], s["a"][a].double())
            y[rows] += torch.einsum("tr,nr->tn", low, s["b"][a].double()) * s["scale"][a].double()
    return {"y": y}


def exact(case, seed):
    if case["op"] == "pages" and sum(_lens(case)[1]) > 2000000:
        return None
    return {"pages": _exact_pages, "rope": _exact_rope, "adapted": _exact_adapted}[case["op"]](
        _INPUTS[case["op"]](case, seed))

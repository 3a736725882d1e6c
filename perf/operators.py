"""The 8-bit KV cache operators, as cases that can be timed and compared.

A cache of keys and values is held in pages of `page` tokens.  Each page, KV
head and side (K or V) has one power-of-two scale, and holds its elements as
8-bit codes (int8, or e4m3 floats): value = code * scale.  Two operators:

  write   new tokens' keys and values are quantised into their slots' pages,
          and the pages that they touch are read back as values
  attend  causal grouped-query attention of packed query tokens (one a slot,
          a few drafts, or pieces of prompts) over the slots' cached tokens

With `own` false, run() computes them with elementary torch operations in 32
bits; with `own` true it calls the library's entry points on the same data.
"""
import math
import random

import torch

own = False

#: heads: query heads, KV heads, head dimension
HEADS = {
    "16x2x256": (16, 2, 256),   # wide heads, eight query heads to a KV head
    "32x8x128": (32, 8, 128),   # four query heads to a KV head
    "28x4x128": (28, 4, 128),   # seven: a group that is no power of two
    "16x16x128": (16, 16, 128),  # every query head has its own KV head
    "12x4x64": (12, 4, 64),     # narrow heads, groups of three
}


def _case(name, op, n, new, ctx, heads, code, page, dtype="bf16", ragged=True):
    """n sequences of up to `new` new tokens, up to `ctx` tokens each with them."""
    c = {"op": op, "n": n, "new": new, "ctx": ctx, "heads": heads, "code": code, "page": page,
         "dtype": dtype, "ragged": ragged}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one request's next token: nothing but latency
        _case("write-one", "write", 1, 1, 1000, "16x2x256", "i8", 64, ragged=False),
        # a full batch's next tokens, small pages
        _case("write-step", "write", 512, 1, 4096, "32x8x128", "e4m3", 16),
        # a batch of prompt pieces that start and end inside pages
        _case("write-prompts", "write", 8, 2048, 8192, "16x2x256", "i8", 64),
        # one long prompt of a model run in float32
        _case("write-f32", "write", 1, 8192, 8192, "32x8x128", "e4m3", 128, "f32", False),
        # one request with a short context
        _case("decode-one", "attend", 1, 1, 777, "16x2x256", "i8", 64, ragged=False),
        # a usual decode batch, contexts of mixed lengths
        _case("decode-64", "attend", 64, 1, 8192, "16x2x256", "i8", 64),
        # a full decode batch, small pages
        _case("decode-256", "attend", 256, 1, 8192, "32x8x128", "e4m3", 16),
        # one request with a very long context
        _case("decode-long", "attend", 1, 1, 131072, "32x8x128", "e4m3", 128, ragged=False),
        # speculative verify: four drafts a slot
        _case("drafts-128", "attend", 128, 4, 4096, "16x2x256", "i8", 64, ragged=True),
        # pieces of prompts over what is already in the cache
        _case("prompt-pieces", "attend", 8, 2048, 8192, "16x2x256", "i8", 64),
        # a whole prompt at once
        _case("prompt-8192", "attend", 1, 8192, 8192, "32x8x128", "e4m3", 64, ragged=False),
        # short odd sequences of a model run in float32
        _case("drafts-f32", "attend", 5, 17, 1003, "12x4x64", "i8", 16, "f32"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    heads = rng.choice(sorted(HEADS))
    h_q, h_kv, d = HEADS[heads]
    code, page = rng.choice(("i8", "e4m3")), rng.choice((16, 32, 64, 128))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    kind = rng.choice(("write-step", "write-prompts", "decode", "decode", "drafts", "prompts"))
    if kind == "write-step":
        return _case("", "write", _log_int(rng, 1, 512), _log_int(rng, 1, 8),
                     _log_int(rng, 16, 4096), heads, code, page, dtype)
    if kind == "write-prompts":
        new = _log_int(rng, 32, 8192)
        n = _log_int(rng, 1, max(1, min(16, 16384 * 512 // (new * h_kv * d))))
        return _case("", "write", n, new, _log_int(rng, new, 8192), heads, code, page, dtype)
    if kind == "decode":
        n = _log_int(rng, 1, 256)
        most = min(131072, 256 * 8192 * 8 * 128 // (2 * n * h_kv * d))
        return _case("", "attend", n, 1, _log_int(rng, 1, most), heads, code, page, dtype)
    if kind == "drafts":
        n = _log_int(rng, 1, 128)
        return _case("", "attend", n, rng.randint(2, 17), _log_int(rng, 17, 4096), heads, code,
                     page, dtype)
    new = _log_int(rng, 18, 4096)
    n = _log_int(rng, 1, max(1, min(8, 8192 // new)))
    return _case("", "attend", n, new, _log_int(rng, new, 8192), heads, code, page, "bf16")


def _lens(case):
    """Per sequence: new tokens, and tokens in all with them.  The longest are as the case says."""
    n, new, ctx = case["n"], case["new"], case["ctx"]
    ctx = max(ctx, new)
    if not case["ragged"]:
        return [new] * n, [ctx] * n
    rnd = random.Random("%d/%d/%d" % (n, new, ctx))
    news = [rnd.randint(max(1, new // 4), new) for _ in range(n)]
    news[0] = new
    if n >= 4 and new > 1:
        news[-1] = 0  # a slot of the batch without new tokens in this step
    return news, [ctx] + [rnd.randint(max(x, ctx // 16), ctx) for x in news[1:]]


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def work(case):
    h_q, h_kv, d = HEADS[case["heads"]]
    news, alls = _lens(case)
    size = 2 if case["dtype"] == "bf16" else 4
    pages = sum(-(-x // case["page"]) for x in alls)
    if case["op"] == "write":
        new = sum(news)
        back = sum(x - (x - y) // case["page"] * case["page"] for x, y in zip(alls, news) if y)
        elems = 2 * h_kv * d
        return {"bytes": elems * (new * (size + 1) + back * (1 + size)), "flops": 3 * elems * new}
    pairs = sum(y * (x - y) + y * (y + 1) // 2 for x, y in zip(alls, news))
    live = sum(x for x, y in zip(alls, news) if y)
    return {"bytes": 2 * live * h_kv * d + 8 * pages * h_kv + 2 * sum(news) * h_q * d * size,
            "flops": 4 * d * h_q * pairs}


# ------------------------------------------------------------------ inputs

def _exponent(amax, code):
    """The least e with amax <= top * 2^e, top the largest code; -100 for nothing but zeros."""
    m, x = torch.frexp(amax)
    if code == "i8":
        e = (x - 7 + (m > 127 / 128)).clamp(-100, 120)
    else:
        e = (x - 9 + (m > 0.875)).clamp(-100, 118)
    return torch.where(amax == 0, torch.full_like(e, -100), e)


def _pow2(e):
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _to_codes(x, code):
    if code == "i8":
        return x.round().clamp(-127, 127).to(torch.int8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _pick(codes, at):
    """codes[at]: 8-bit floats are indexed as bytes."""
    return codes.view(torch.uint8)[at].view(codes.dtype)


def _put(codes, at, x):
    codes.view(torch.uint8)[at] = x.view(torch.uint8)


def _filled(shape, code, gain, gen):
    """Pages of quantised normal values: codes, and a scale for each page and head."""
    x = torch.empty(shape, dtype=torch.float16, device="cuda").normal_(generator=gen).mul_(gain)
    scale = _pow2(_exponent(x.abs().amax((-2, -1)).float(), code))
    codes = _to_codes(x.mul_((1 / scale).half()[..., None, None]), code)
    return codes[None], scale[None].contiguous()


def _inputs(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    rnd = random.Random(seed)
    h_q, h_kv, d = HEADS[case["heads"]]
    page, code, dtype = case["page"], case["code"], _dtype(case)
    news, alls = _lens(case)
    n, total = len(news), sum(news)
    n_slots = n + 3
    slots = rnd.sample(range(n_slots), n)
    counts = [-(-x // page) for x in alls]
    n_pages, max_pages = sum(counts) + 5, max(counts) + 1
    order = torch.randperm(n_pages, generator=gen, device=dev)
    table = torch.full((n_slots, max_pages), -1, dtype=torch.int64, device=dev)
    i32 = dict(dtype=torch.int32, device=dev)
    row = torch.repeat_interleave(torch.tensor(slots, device=dev),
                                  torch.tensor(counts, device=dev))
    col = torch.cat([torch.arange(c) for c in counts]).to(dev)
    table[row, col] = order[:row.numel()]
    # keys have a few channels that are much larger than the others
    gain = torch.ones(d, device=dev).half()
    gain[::29] = 6.0
    k, k_scale = _filled((n_pages, h_kv, page, d), code, gain, gen)
    v, v_scale = _filled((n_pages, h_kv, page, d), code, gain * 0 + 0.5, gen)
    cum = [0]
    for x in news:
        cum.append(cum[-1] + x)
    s = {"k": k, "v": v, "k_scale": k_scale, "v_scale": v_scale, "table": table.to(torch.int32),
         "slots": torch.tensor(slots, **i32), "case": dict(case), "total": total,
         "max_new": max(news), "max_all": max(alls), "code": code, "page": page,
         "cu": None if total == n and max(news) == 1 else torch.tensor(cum, **i32),
         "new": torch.tensor(news, **i32), "all": torch.tensor(alls, **i32),
         "pos": torch.tensor([x - y for x, y in zip(alls, news)], **i32)}
    if case["op"] == "write":
        # keys and values are columns of one projection's rows, queries before them
        rows = torch.randn(total, (h_q + 2 * h_kv) * d, generator=gen, device=dev)
        rows[:, h_q * d:(h_q + h_kv) * d] *= gain.float().repeat(h_kv)
        rows = rows.to(dtype)
        s["new_k"] = rows[:, h_q * d:(h_q + h_kv) * d].unflatten(1, (h_kv, d))
        s["new_v"] = rows[:, (h_q + h_kv) * d:].unflatten(1, (h_kv, d))
        # read back from the start of the first page that each sequence touches
        from_ = [(x - y) // page * page if y else x for x, y in zip(alls, news)]
        back = [x - f for x, f in zip(alls, from_)]
        cum = [0]
        for x in back:
            cum.append(cum[-1] + x)
        s |= {"back_pos": torch.tensor(from_, **i32), "back": torch.tensor(back, **i32),
              "back_cu": torch.tensor(cum, **i32), "max_back": max(back), "back_total": cum[-1],
              "out_k": torch.empty(cum[-1], h_kv, d, dtype=dtype, device=dev),
              "out_v": torch.empty(cum[-1], h_kv, d, dtype=dtype, device=dev)}
    else:
        q = torch.randn(total, h_q, d, generator=gen, device=dev)
        s["q"] = (q * 1.5 / gain.float()).to(dtype)
        s["scale"] = 1 / math.sqrt(d)
        s["o"] = torch.empty_like(s["q"])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:  # the handle that a program keeps, on the same memory
        from gated_deltanet_recurrent_gb300 import abi
        s["abi"] = abi
        s["cache"] = abi.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"],
                                 h_q=HEADS[case["heads"]][0], host_checks=False)
    return s


# -------------------------------------------------------------- plain forms

def _token_places(s, count, total, start):
    """For each of the packed tokens: its sequence, its position, its page and its place there."""
    seq = torch.repeat_interleave(torch.arange(count.numel(), device="cuda"), count.long(),
                                  output_size=total)
    first = torch.cumsum(count.long(), 0) - count.long()
    pos = torch.arange(total, device="cuda") - first[seq] + start.long()[seq]
    page = s["table"].long()[s["slots"].long()[seq], pos // s["page"]]
    return seq, pos, page, pos % s["page"]


def _write_side(s, x, codes, scale, page, off, opened, kept):
    """Quantise x [tokens][heads][d] into its pages; `opened`: the page that each sequence's first
    token goes to, `kept`: whether it holds earlier tokens."""
    x = x.float()
    amax = torch.zeros_like(scale).scatter_reduce_(
        0, page[:, None].expand(-1, scale.shape[1]), x.abs().amax(-1), "amax")
    fresh = _pow2(_exponent(amax, s["code"]))
    old = scale[opened]
    grown = torch.where(kept[:, None], torch.maximum(old, fresh[opened]), fresh[opened])
    held = _pick(codes, opened).float()
    rescaled = torch.where(kept[:, None, None, None], held * (old / grown)[..., None, None], held)
    _put(codes, opened, _to_codes(rescaled, s["code"]))
    scale[page] = fresh[page]
    scale[opened] = grown
    _put(codes, (page, slice(None), off), _to_codes(x / scale[page][..., None], s["code"]))


def _plain_write(s):
    _, _, page, off = _token_places(s, s["new"], s["total"], s["pos"])
    # a sequence without new tokens opens no page: it takes the place of the first that has some
    has = (s["new"] > 0).long()
    who = torch.where(has > 0, torch.arange(has.numel(), device="cuda"), has.argmax())
    pos = s["pos"].long()[who]
    opened, kept = s["table"].long()[s["slots"].long()[who], pos // s["page"]], pos % s["page"] > 0
    _write_side(s, s["new_k"], s["k"][0], s["k_scale"][0], page, off, opened, kept)
    _write_side(s, s["new_v"], s["v"][0], s["v_scale"][0], page, off, opened, kept)
    _, _, page, off = _token_places(s, s["back"], s["back_total"], s["back_pos"])
    dtype = s["out_k"].dtype
    at = (page, slice(None), off)
    return {"k": (_pick(s["k"][0], at).float() * s["k_scale"][0][page][..., None]).to(dtype),
            "v": (_pick(s["v"][0], at).float() * s["v_scale"][0][page][..., None]).to(dtype),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _plain_attend(s):
    q = s["q"]
    n, t_max = s["new"].numel(), s["max_new"]
    pages = -(-s["max_all"] // s["page"])
    h_kv, d = s["k"].shape[2], s["k"].shape[4]
    ids = s["table"].long()[s["slots"].long(), :pages].clamp(min=0)

    def cached(codes, scale):
        x = _pick(codes[0], ids).float().mul_(scale[0][ids][..., None, None])
        return x.transpose(1, 2).reshape(n, h_kv, pages * s["page"], d)

    seq, pos, _, _ = _token_places(s, s["new"], s["total"], s["pos"])
    t = pos - s["pos"].long()[seq]
    rows = torch.zeros(n, t_max, *q.shape[1:], device="cuda")
    rows[seq, t] = q.float()
    rows = rows.view(n, t_max, h_kv, -1, d).permute(0, 2, 3, 1, 4).reshape(n, h_kv, -1, d)
    score = torch.matmul(rows, cached(s["k"], s["k_scale"]).transpose(2, 3)).mul_(s["scale"])
    score = score.view(n, h_kv, -1, t_max, score.shape[-1])
    at = s["pos"].long()[:, None] + torch.arange(t_max, device="cuda")
    hidden = torch.arange(score.shape[-1], device="cuda") > at[..., None]
    score.masked_fill_(hidden[:, None, None], -math.inf)
    score.sub_(score.amax(-1, keepdim=True)).exp_()
    score.div_(score.sum(-1, keepdim=True))
    o = torch.matmul(score.view(n, h_kv, -1, score.shape[-1]), cached(s["v"], s["v_scale"]))
    o = o.view(n, h_kv, -1, t_max, d).permute(0, 3, 1, 2, 4).reshape(n, t_max, -1, d)
    return {"o": o[seq, t].to(q.dtype)}


def run(state):
    s = state
    if not own:
        return _plain_write(s) if s["case"]["op"] == "write" else _plain_attend(s)
    abi, kv = s["abi"], s["cache"]
    if s["case"]["op"] == "write":
        abi.gdn_kv_append(kv, 0, s["slots"], s["pos"], s["new_k"], s["new_v"],
                          cu_seqlens=s["cu"], max_seqlen=s["max_new"])
        abi.gdn_kv_read(kv, 0, s["slots"], s["back_pos"], s["out_k"], s["out_v"],
                        cu_seqlens=s["back_cu"], max_seqlen=s["max_back"])
        return {"k": s["out_k"], "v": s["out_v"], "k_scale": s["k_scale"],
                "v_scale": s["v_scale"]}
    abi.gdn_kv_attend(kv, 0, s["slots"], s["all"], s["q"], s["o"], cu_seqlens=s["cu"],
                      max_seqlen=s["max_new"], max_kv_len=s["max_all"], scale=s["scale"])
    return {"o": s["o"]}


# ------------------------------------------------- the definition, in 64 bits

def _nearest(y, code):
    """y rounded to the nearest code, ties to even."""
    if code == "i8":
        return torch.round(y).clamp(-127, 127)
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -60))).clamp(min=-6)
    return (torch.round(y / 2.0 ** (e - 3)) * 2.0 ** (e - 3)).clamp(-448, 448)


def _exact_page(held, old, x, code):
    """One page of one head: `held` earlier codes [a][d] under scale `old`, then x [b][d]."""
    top, hi = (127.0, 120) if code == "i8" else (448.0, 118)
    amax = float(x.abs().max())
    e = -100
    if amax > 0:
        e = max(-100, min(hi, math.ceil(math.log2(amax / top))))
        while e > -100 and amax <= top * 2.0 ** (e - 1):
            e -= 1
        while e < hi and amax > top * 2.0 ** e:
            e += 1
    scale = 2.0 ** e
    if held.shape[0]:
        scale = max(scale, old)
    return torch.cat([_nearest(held * old / scale, code), _nearest(x / scale, code)]), scale


def _exact_write(s):
    news, page = s["new"].tolist(), s["page"]
    table, first = s["table"].tolist(), 0
    out = {"k": [], "v": [], "k_scale": s["k_scale"].double(), "v_scale": s["v_scale"].double()}
    amount = sum(-(-x // page) + 1 for x in news) * s["k"].shape[2]
    if amount > 12000:
        return None
    for slot, t, pos in zip(s["slots"].tolist(), news, s["pos"].tolist()):
        done = 0
        while done < t:
            off = (pos + done) % page
            take, pid = min(t - done, page - off), table[slot][(pos + done) // page]
            for side in ("k", "v"):
                x = s["new_" + side][first + done:first + done + take].double().cpu()
                held = s[side][0, pid, :, :off].float().double().cpu()
                old = s[side + "_scale"][0, pid].tolist()
                got = [_exact_page(held[h], old[h], x[:, h], s["code"]) for h in range(len(old))]
                out[side].append(torch.stack([c * f for c, f in got], 1))
                out[side + "_scale"][0, pid] = torch.tensor([f for _, f in got]).to("cuda")
            done += take
        first += t
    return {x: torch.cat(y).to("cuda") if isinstance(y, list) else y for x, y in out.items()}


def _exact_attend(s):
    q = s["q"].double()
    o = torch.zeros_like(q)
    h_kv, d, page = s["k"].shape[2], s["k"].shape[4], s["page"]
    group, first = q.shape[1] // h_kv, 0
    for slot, t, length in zip(s["slots"].tolist(), s["new"].tolist(), s["all"].tolist()):
        ids = s["table"][slot, :-(-length // page)].long()
        for h in range(h_kv if t else 0):
            key = s["k"][0, :, h].view(torch.uint8)[ids].view(s["k"].dtype).double()
            val = s["v"][0, :, h].view(torch.uint8)[ids].view(s["v"].dtype).double()
            key = key * s["k_scale"][0, ids, h, None, None].double()
            val = val * s["v_scale"][0, ids, h, None, None].double()
            key, val = key.reshape(-1, d)[:length], val.reshape(-1, d)[:length]
            for g in range(h * group, (h + 1) * group):
                a = q[first:first + t, g] @ key.T * s["scale"]
                late = torch.ones(t, length, dtype=torch.bool, device="cuda").triu(length - t + 1)
                o[first:first + t, g] = torch.softmax(a.masked_fill_(late, -math.inf), -1) @ val
        first += t
    return {"o": o}


def exact(case, seed):
    s = _inputs(case, seed)
    return _exact_write(s) if case["op"] == "write" else _exact_attend(s)

"""A small hybrid model on the library: recurrent (Gated DeltaNet) layers with
an attention layer between them, serving several requests from one set of
slots.

    python examples/hybrid_decode.py

Each request owns a slot: its recurrent states and conv windows live in the
pool, its keys and values in pages of the 8-bit KV cache.  Prompts of mixed
lengths are fed in one packed call per layer, then tokens are decoded one per
slot and step.  Weights are random; the model is as small as the library's
shapes allow and shows how the calls fit together.

Three things are optional: rotary positions in the attention layer, pages that
are handed out on the GPU as requests grow (and taken back), and low-rank adapters
on every input projection, one per request."""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from gated_deltanet_recurrent_gb300 import abi  # noqa: E402

HIDDEN = 512
GDN = dict(h_v=8, h_k=4, dk=64, dv=64, conv_k=4)
ATTN = dict(h_q=8, h_kv=2, d=64)
PAGE = 16


class Hybrid:
    """Layers "g" (recurrent) and "a" (attention) over `n_slots` slots of up to
    max_len tokens each.  rope: rotate queries and keys to their positions; n_pages: the
    cache's pages are handed out on the GPU, from so many; adapters: so many low-rank
    adapters of rank 16 beside each input projection."""

    def __init__(self, layers="gag", n_slots=4, max_len=256, code=torch.int8, seed=0,
                 device="cuda", host_checks=True, rope=False, n_pages=None, adapters=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.layers = layers
        g, a = GDN, ATTN
        self.conv_ch = 2 * g["h_k"] * g["dk"] + g["h_v"] * g["dv"]
        self.pool = abi.Pool(max(1, layers.count("g")), n_slots, g["h_v"], g["h_k"], g["dk"],
                             g["dv"], self.conv_ch, g["conv_k"], host_checks=host_checks,
                             device=device)
        max_pages = -(-max_len // PAGE)
        self.kv = abi.KVCache.empty(max(1, layers.count("a")), n_slots,
                                    n_pages or n_slots * max_pages, max_pages, PAGE, a["h_q"],
                                    a["h_kv"], a["d"], code=code, host_checks=host_checks,
                                    device=device)
        self.pages = abi.KVPages(self.kv) if n_pages else None
        if self.pages is None:  # every slot owns its pages
            self.kv.page_table.copy_(torch.arange(n_slots * max_pages, dtype=torch.int32,
                                                  device=device).view(n_slots, max_pages))
        # a quarter of each head is rotated, as in models that have both kinds of layers
        self.rope = abi.Rope(a["d"], rot=a["d"] // 4, host_checks=host_checks) if rope else None
        self.device = device

        def weight(rows, cols):
            w = torch.randn(rows, cols, generator=gen, device=device) / cols ** 0.5
            return w.to(torch.bfloat16)

        self.params = []
        for kind in layers:
            if kind == "g":
                heads = g["h_v"] * g["dv"]
                self.params.append({
                    "in": weight(self.conv_ch + heads + 2 * g["h_v"], HIDDEN),
                    "conv": torch.randn(self.conv_ch, g["conv_k"], generator=gen,
                                        device=device) * 0.5,
                    "norm": torch.ones(g["dv"], device=device), "out": weight(HIDDEN, heads)})
            else:
                self.params.append({
                    "in": weight((a["h_q"] + 2 * a["h_kv"]) * a["d"], HIDDEN),
                    "out": weight(HIDDEN, a["h_q"] * a["d"])})
        for p in self.params if adapters else ():
            low = torch.stack([weight(16, HIDDEN) for _ in range(adapters)])
            high = torch.stack([weight(p["in"].shape[0], 16) for _ in range(adapters)])
            p["adapters"] = abi.Adapters(low, high, torch.full((adapters,), 0.5, device=device),
                                         host_checks=host_checks)

    def _project(self, x, p, ids):
        y = torch.empty(x.shape[0], p["in"].shape[0], dtype=torch.bfloat16, device=x.device)
        if ids is None:
            return abi.gdn_in_proj(self.pool, x, p["in"], y)
        return abi.gdn_in_proj_adapted(self.pool, p["adapters"], x, p["in"], ids, y)

    def _recurrent(self, layer, p, x, slots, cu, longest, ids):
        g, n = GDN, x.shape[0]
        y = self._project(x, p, ids)
        conv = torch.empty(n, self.conv_ch, dtype=torch.bfloat16, device=x.device)
        abi.gdn_conv_silu(self.pool, layer, slots, y[:, :self.conv_ch], p["conv"], conv,
                          cu_seqlens=cu, max_seqlen=longest)
        nk = g["h_k"] * g["dk"]
        q = conv[:, :nk].unflatten(1, (g["h_k"], g["dk"]))
        k = conv[:, nk:2 * nk].unflatten(1, (g["h_k"], g["dk"]))
        v = conv[:, 2 * nk:].unflatten(1, (g["h_v"], g["dv"]))
        heads = g["h_v"] * g["dv"]
        gate, logits = y[:, self.conv_ch:self.conv_ch + heads], y[:, self.conv_ch + heads:].float()
        decay = -torch.nn.functional.softplus(logits[:, :g["h_v"]])
        beta = torch.sigmoid(logits[:, g["h_v"]:])
        decay, beta = (t.to(torch.bfloat16).contiguous() for t in (decay, beta))
        o = torch.empty(n, g["h_v"], g["dv"], device=x.device)
        if cu is None:
            abi.gdn_decode_step(self.pool, layer, slots, q, k, v, decay, beta, o)
        else:
            abi.gdn_prefill_chunked(self.pool, layer, slots, cu, q, k, v, decay, beta, o,
                                    max_seqlen=longest)
        z = gate.reshape(n, g["h_v"], g["dv"]).contiguous()
        o = abi.gdn_gated_rmsnorm(o, z, p["norm"], torch.empty_like(z))
        return o.view(n, heads) @ p["out"].T

    def _attention(self, layer, p, x, slots, cu, pos, lens, longest, longest_context, ids,
                   positions):
        a, n = ATTN, x.shape[0]
        y = self._project(x, p, ids)
        nq, nk = a["h_q"] * a["d"], a["h_kv"] * a["d"]
        q = y[:, :nq].unflatten(1, (a["h_q"], a["d"]))
        k = y[:, nq:nq + nk].unflatten(1, (a["h_kv"], a["d"]))
        v = y[:, nq + nk:].unflatten(1, (a["h_kv"], a["d"]))
        if self.rope is not None:
            abi.gdn_rope(self.rope, positions, q, k)
        # the new tokens first: a query attends its own position too
        abi.gdn_kv_append(self.kv, layer, slots, pos, k, v, cu_seqlens=cu, max_seqlen=longest)
        o = torch.empty(n, a["h_q"], a["d"], dtype=torch.bfloat16, device=x.device)
        abi.gdn_kv_attend(self.kv, layer, slots, lens, q, o, cu_seqlens=cu, max_seqlen=longest,
                          max_kv_len=longest_context)
        return o.view(n, nq) @ p["out"].T

    def reserve(self, slots, pos, new):
        """Pages for new[i] more tokens of slots[i], which holds pos[i]: True where there were
        enough.  Where there were not, the request must not go into forward(): it would attend to
        less than it was given.  It waits until others end, or ends itself."""
        if self.pages is None:
            return [True] * len(new)
        cu = torch.tensor([0] + new, dtype=torch.int32).cumsum(0, dtype=torch.int32)
        granted = torch.empty(len(new), dtype=torch.int32, device=self.device)
        abi.gdn_kv_pages_grow(self.kv, self.pages, slots, pos, cu.to(self.device), sum(new),
                              granted=granted)
        return [bool(x) for x in granted.tolist()]

    def _positions(self, n, slots, pos, cu):
        """Each new token's position; with pages of its own, the cache gets those the tokens need
        (reserve() has done that already where they may not suffice)."""
        if self.pages is not None:
            at = torch.empty(n, dtype=torch.int32, device=self.device)
            abi.gdn_kv_pages_grow(self.kv, self.pages, slots, pos, cu, positions=at)
            return at
        if self.rope is None or cu is None:
            return pos
        new = (cu[1:] - cu[:-1]).long()
        first = torch.repeat_interleave(pos - cu[:-1], new, output_size=n)
        return first + torch.arange(n, dtype=torch.int32, device=self.device)

    def forward(self, x, slots, pos, cu=None, longest=1, longest_context=0, ids=None):
        """Hidden states x [tokens, HIDDEN] bf16 of the new tokens of `slots` (packed by cu, or
        one each), which hold pos[i] tokens so far; ids: each token's adapter, -1 for none.
        Returns the hidden states after the last layer; the slots then hold the new tokens too."""
        new = 1 if cu is None else cu[1:] - cu[:-1]
        lens = pos + new
        positions = self._positions(x.shape[0], slots, pos, cu)
        seen = {"g": 0, "a": 0}
        for kind, p in zip(self.layers, self.params):
            if kind == "g":
                x = x + self._recurrent(seen["g"], p, x, slots, cu, longest, ids)
            else:
                x = x + self._attention(seen["a"], p, x, slots, cu, pos, lens, longest,
                                        longest_context, ids, positions)
            seen[kind] += 1
        return x

    def release(self, slots, lens):
        """Give back the pages that the first lens[i] tokens of slots[i] do not use."""
        if self.pages is not None:
            abi.gdn_kv_pages_trim(self.kv, self.pages, slots, lens)

    def errors(self):
        return abi.gdn_pool_get_error(self.pool) | abi.gdn_kv_get_error(self.kv)


def serve(model, adapters=None, prompts=(100, 17, 64), steps=8):
    """Three prompts, and `steps` more tokens of each; adapters: the one of each request.  Returns the
    lengths that were reached, and prints them."""
    torch.manual_seed(0)
    x = torch.randn(sum(prompts), HIDDEN, device="cuda").to(torch.bfloat16).split(list(prompts))
    slots, adapters = [2, 0, 3], adapters or [None] * 3
    lens, norms, waiting = [0] * 3, [0.0] * 3, [0, 1, 2]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    while waiting:
        # the first of the waiting requests for which there are pages; the others come when these have ended
        here = i32([slots[i] for i in waiting])
        fits = model.reserve(here, torch.zeros_like(here), [prompts[i] for i in waiting])
        batch = [i for i, ok in zip(waiting, fits) if ok]
        if not batch:
            raise RuntimeError("a prompt needs more pages than there are")
        waiting = [i for i in waiting if i not in batch]
        new = [prompts[i] for i in batch]
        here, pos, ids, packed = i32([slots[i] for i in batch]), i32([0] * len(batch)), None, None
        abi.gdn_pool_reset(model.pool, here)
        cu = i32([sum(new[:k]) for k in range(len(new) + 1)])
        if adapters[0] is not None:
            ids = i32([adapters[i] for i in batch])
            packed = torch.repeat_interleave(ids, i32(new))
        h = model.forward(torch.cat([x[i] for i in batch]), here, pos, cu, longest=max(new),
                          longest_context=max(new), ids=packed)
        h, pos = h[cu[1:].long() - 1], i32(new)
        for step in range(steps + 1):
            fits = [False] * len(batch) if step == steps else model.reserve(here, pos, [1] * len(batch))
            ended = [k for k, ok in enumerate(fits) if not ok]
            if ended:  # at their full length, or because there is no page left
                for k in ended:
                    lens[batch[k]], norms[batch[k]] = int(pos[k]), float(h[k].float().norm())
                model.release(here[ended], torch.zeros_like(pos[ended]))
                rest = [k for k, ok in enumerate(fits) if ok]
                batch, here, pos, h = [batch[k] for k in rest], here[rest], pos[rest], h[rest]
                ids = None if ids is None else ids[rest]
            if not batch:
                break
            # a model would sample a token and embed it; here the state itself is fed back
            h = torch.nn.functional.normalize(h.float(), dim=-1).mul(HIDDEN ** 0.5).to(torch.bfloat16)
            h = model.forward(h, here, pos, longest_context=max(prompts) + step + 1, ids=ids)
            pos = pos + 1
    print("lengths", lens, "norms", [round(v, 3) for v in norms], "errors", model.errors())
    return lens


def main():
    serve(Hybrid(n_slots=4, max_len=256))
    # the same requests with positions, an adapter for two of them, and half as many pages
    serve(Hybrid(n_slots=4, max_len=256, rope=True, n_pages=32, adapters=3), adapters=[2, -1, 0])


if __name__ == "__main__":
    main()

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

    def _positions(self, n, slots, pos, cu):
        """Each new token's position; with pages of its own, the cache gets those the tokens need."""
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


def serve(model, adapters=None):
    """Three prompts and eight steps; adapters: the one of each request."""
    torch.manual_seed(0)
    prompts = [100, 17, 64]
    slots = torch.tensor([2, 0, 3], dtype=torch.int32, device="cuda")
    abi.gdn_pool_reset(model.pool, slots)
    cu = torch.tensor([0, 100, 117, 181], dtype=torch.int32, device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    x = torch.randn(sum(prompts), HIDDEN, device="cuda").to(torch.bfloat16)
    ids = packed = None
    if adapters is not None:
        ids = torch.tensor(adapters, dtype=torch.int32, device="cuda")
        packed = torch.repeat_interleave(ids, torch.tensor(prompts, device="cuda"))
    h = model.forward(x, slots, pos, cu, longest=max(prompts), longest_context=max(prompts),
                      ids=packed)
    h = h[cu[1:].long() - 1]
    pos = pos + torch.tensor(prompts, dtype=torch.int32, device="cuda")
    for step in range(8):
        # a model would sample a token and embed it; here the state itself is fed back
        h = torch.nn.functional.normalize(h.float(), dim=-1).mul(HIDDEN ** 0.5).to(torch.bfloat16)
        h = model.forward(h, slots, pos, longest_context=max(prompts) + step + 1, ids=ids)
        pos = pos + 1
    model.release(slots, torch.zeros_like(pos))
    torch.cuda.synchronize()
    print("lengths", pos.tolist(), "norms", [round(float(v), 3) for v in h.float().norm(dim=-1)],
          "errors", model.errors())


def main():
    serve(Hybrid(n_slots=4, max_len=256))
    # the same requests with positions, an adapter for two of them, and half as many pages
    serve(Hybrid(n_slots=4, max_len=256, rope=True, n_pages=32, adapters=3), adapters=[2, -1, 0])


if __name__ == "__main__":
    main()

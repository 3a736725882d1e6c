"""A small hybrid model on the library: recurrent (Gated DeltaNet) layers with
an attention layer between them, serving several requests from one set of
slots.

    python examples/hybrid_decode.py

Each request owns a slot: its recurrent states and conv windows live in the
pool, its keys and values in pages of the 8-bit KV cache.  Prompts of mixed
lengths are fed in one packed call per layer, then tokens are decoded one per
slot and step.  Weights are random; the model is as small as the library's
shapes allow and shows how the calls fit together."""
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
    max_len tokens each."""

    def __init__(self, layers="gag", n_slots=4, max_len=256, code=torch.int8, seed=0,
                 device="cuda", host_checks=True):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.layers = layers
        g, a = GDN, ATTN
        self.conv_ch = 2 * g["h_k"] * g["dk"] + g["h_v"] * g["dv"]
        self.pool = abi.Pool(max(1, layers.count("g")), n_slots, g["h_v"], g["h_k"], g["dk"],
                             g["dv"], self.conv_ch, g["conv_k"], host_checks=host_checks,
                             device=device)
        max_pages = -(-max_len // PAGE)
        self.kv = abi.KVCache.empty(max(1, layers.count("a")), n_slots, n_slots * max_pages,
                                    max_pages, PAGE, a["h_q"], a["h_kv"], a["d"], code=code,
                                    host_checks=host_checks, device=device)
        # every slot owns its pages here; a server hands them out as requests grow
        self.kv.page_table.copy_(torch.arange(n_slots * max_pages, dtype=torch.int32,
                                              device=device).view(n_slots, max_pages))
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

    def _project(self, x, w):
        y = torch.empty(x.shape[0], w.shape[0], dtype=torch.bfloat16, device=x.device)
        return abi.gdn_in_proj(self.pool, x, w, y)

    def _recurrent(self, layer, p, x, slots, cu, longest):
        g, n = GDN, x.shape[0]
        y = self._project(x, p["in"])
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

    def _attention(self, layer, p, x, slots, cu, pos, lens, longest, longest_context):
        a, n = ATTN, x.shape[0]
        y = self._project(x, p["in"])
        nq, nk = a["h_q"] * a["d"], a["h_kv"] * a["d"]
        q = y[:, :nq].unflatten(1, (a["h_q"], a["d"]))
        k = y[:, nq:nq + nk].unflatten(1, (a["h_kv"], a["d"]))
        v = y[:, nq + nk:].unflatten(1, (a["h_kv"], a["d"]))
        # the new tokens first: a query attends its own position too
        abi.gdn_kv_append(self.kv, layer, slots, pos, k, v, cu_seqlens=cu, max_seqlen=longest)
        o = torch.empty(n, a["h_q"], a["d"], dtype=torch.bfloat16, device=x.device)
        abi.gdn_kv_attend(self.kv, layer, slots, lens, q, o, cu_seqlens=cu, max_seqlen=longest,
                          max_kv_len=longest_context)
        return o.view(n, nq) @ p["out"].T

    def forward(self, x, slots, pos, cu=None, longest=1, longest_context=0):
        """Hidden states x [tokens, HIDDEN] bf16 of the new tokens of `slots` (packed by cu, or
        one each), which hold pos[i] tokens so far.  Returns the hidden states after the
        last layer; the slots then hold the new tokens too."""
        new = 1 if cu is None else cu[1:] - cu[:-1]
        lens = pos + new
        seen = {"g": 0, "a": 0}
        for kind, p in zip(self.layers, self.params):
            if kind == "g":
                x = x + self._recurrent(seen["g"], p, x, slots, cu, longest)
            else:
                x = x + self._attention(seen["a"], p, x, slots, cu, pos, lens, longest,
                                        longest_context)
            seen[kind] += 1
        return x

    def errors(self):
        return abi.gdn_pool_get_error(self.pool) | abi.gdn_kv_get_error(self.kv)


def main():
    torch.manual_seed(0)
    model = Hybrid(n_slots=4, max_len=256)
    prompts = [100, 17, 64]
    slots = torch.tensor([2, 0, 3], dtype=torch.int32, device="cuda")
    abi.gdn_pool_reset(model.pool, slots)
    cu = torch.tensor([0, 100, 117, 181], dtype=torch.int32, device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    x = torch.randn(sum(prompts), HIDDEN, device="cuda").to(torch.bfloat16)
    h = model.forward(x, slots, pos, cu, longest=max(prompts), longest_context=max(prompts))
    h = h[cu[1:].long() - 1]
    pos = pos + torch.tensor(prompts, dtype=torch.int32, device="cuda")
    for step in range(8):
        # a model would sample a token and embed it; here the state itself is fed back
        h = torch.nn.functional.normalize(h.float(), dim=-1).mul(HIDDEN ** 0.5).to(torch.bfloat16)
        h = model.forward(h, slots, pos, longest_context=max(prompts) + step + 1)
        pos = pos + 1
    torch.cuda.synchronize()
    print("lengths", pos.tolist(), "norms", [round(float(v), 3) for v in h.float().norm(dim=-1)],
          "errors", model.errors())


if __name__ == "__main__":
    main()

"""Float64 oracle of the 8-bit paged KV cache: quantised writes, values read
back, and causal grouped-query attention, straight from the definitions in
include/gdn.h.  numpy only; shares nothing with the CUDA code."""
import math

import numpy as np

TOP = {"i8": 127.0, "e4m3": 448.0}
MAX_EXP = {"i8": 120, "e4m3": 118}


def block_exponent(amax, code):
    """The least e with amax <= top * 2^e, within [-100, MAX_EXP]."""
    if amax == 0:
        return -100
    e = math.ceil(math.log2(amax / TOP[code]))
    while amax <= TOP[code] * 2.0 ** (e - 1):
        e -= 1
    while amax > TOP[code] * 2.0 ** e:
        e += 1
    return max(-100, min(MAX_EXP[code], e))


def to_code(y, code):
    """Nearest code of each y (ties to even); infinities saturate, NaN is zero."""
    y = np.where(np.isnan(y), 0.0, y)
    y = np.clip(y, -TOP[code], TOP[code])
    if code == "i8":
        return np.rint(y)
    mag = np.maximum(np.abs(y), 2.0 ** -60)
    step = 2.0 ** (np.maximum(np.floor(np.log2(mag)), -6) - 3)
    return np.clip(np.rint(y / step) * step, -TOP[code], TOP[code])


class KVOracle:
    """Codes (as float64 values) [n_layers, n_pages, h_kv, page, d] and scales,
    updated by append() as the library's pages are."""

    def __init__(self, n_layers, n_pages, h_kv, page, d, code, table):
        self.page, self.code = page, code
        self.table = np.asarray(table)
        shape = (n_layers, n_pages, h_kv, page, d)
        self.codes = {"k": np.zeros(shape), "v": np.zeros(shape)}
        self.scale = {"k": np.zeros(shape[:3]), "v": np.zeros(shape[:3])}

    def append(self, layer, slots, pos, lens, k, v):
        lo = 0
        for slot, p0, n in zip(slots, pos, lens):
            for side, x in (("k", k), ("v", v)):
                self._append_one(layer, slot, p0, np.asarray(x[lo:lo + n], np.float64), side)
            lo += n

    def _append_one(self, layer, slot, p0, x, side):
        done = 0
        while done < len(x):
            off = (p0 + done) % self.page
            take = min(len(x) - done, self.page - off)
            pid = self.table[slot, (p0 + done) // self.page]
            for h in range(x.shape[1]):
                new = x[done:done + take, h]
                fin = np.abs(new[np.isfinite(new)])
                e = block_exponent(fin.max() if fin.size else 0.0, self.code)
                block = self.codes[side][layer, pid, h]
                s = 2.0 ** e
                if off:
                    old = self.scale[side][layer, pid, h]
                    s = max(s, old)
                    block[:off] = to_code(block[:off] * old / s, self.code)
                block[off:off + take] = to_code(new / s, self.code)
                self.scale[side][layer, pid, h] = s
            done += take

    def values(self, layer, slot, side, a, b):
        """Values of positions [a, b) of a slot: [b - a, h_kv, d]."""
        p = np.arange(a, b)
        pid = self.table[slot, p // self.page]
        return self.codes[side][layer, pid, :, p % self.page] * \
            self.scale[side][layer, pid][:, :, None]

    def attend(self, layer, slots, kv_lens, lens, q, scale):
        """o [tokens, h_q, d], and sum_j w_j |v_j| of the same shape (what errors scale with)."""
        q = np.asarray(q, np.float64)
        o, mag = np.zeros_like(q), np.zeros_like(q)
        lo = 0
        for slot, kv_len, n in zip(slots, kv_lens, lens):
            if n and kv_len:
                k = self.values(layer, slot, "k", 0, kv_len)
                v = self.values(layer, slot, "v", 0, kv_len)
                o[lo:lo + n], mag[lo:lo + n] = attend_values(q[lo:lo + n], k, v, scale)
            lo += n
        return o, mag


def attend_values(q, k, v, scale, skip=None):
    """Causal attention of q [n, h_q, d], the last n of len(k) positions, over k, v
    [len, h_kv, d]; positions in `skip` are left out."""
    n, h_q, _ = q.shape
    length, h_kv, _ = k.shape
    group = h_q // h_kv
    s = np.einsum("thgd,jhd->thgj", q.reshape(n, h_kv, group, -1), k) * scale
    at = np.arange(length - n, length)
    hidden = np.arange(length)[None] > at[:, None]
    if skip is not None:
        hidden = hidden | np.asarray(skip)[None]
    s = np.where(hidden[:, None, None], -np.inf, s)
    m = s.max(-1, keepdims=True)
    w = np.exp(s - np.where(np.isfinite(m), m, 0.0))
    total = w.sum(-1, keepdims=True)
    w = w / np.where(total > 0, total, 1.0)
    o = np.einsum("thgj,jhd->thgd", w, v)
    mag = np.einsum("thgj,jhd->thgd", w, np.abs(v))
    return o.reshape(q.shape), mag.reshape(q.shape)

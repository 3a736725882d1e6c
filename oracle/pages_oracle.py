"""Plain Python pages of a KV cache: what the GPU calls have to do, entry by entry."""
import numpy as np

SLOT, SEQ, PAGE = 1, 2, 16


class PagesOracle:
    def __init__(self, table, held, free_pages, n_free, page_tokens):
        self.table = np.array(table, dtype=np.int64)
        self.held = [int(x) for x in held]
        self.free = [int(x) for x in free_pages]
        self.n_free = int(n_free)
        self.page = page_tokens
        self.err = 0

    def _slot(self, slot_ids, i):
        slot = int(slot_ids[i])
        if not 0 <= slot < len(self.held) or list(slot_ids).count(slot) > 1:
            self.err |= SLOT
            return None
        return slot

    def _page(self, page):
        if not 0 <= page < len(self.free):
            self.err |= PAGE

    def grow(self, slot_ids, pos, cu, total, positions, rows):
        """positions, rows: arrays that are changed where a token belongs to a sequence.  Returns
        granted."""
        n_pages, max_pages = len(self.free), self.table.shape[1]
        top, asked, granted = self.n_free, 0, []
        if not 0 <= top <= n_pages:
            self.err |= PAGE
            top = 0
        left = top
        for i in range(len(slot_ids)):
            t0, t1 = (i, i + 1) if cu is None else (int(cu[i]), int(cu[i + 1]))
            p, slot = int(pos[i]), self._slot(slot_ids, i)
            if 0 <= t0 <= t1 <= total:
                positions[t0:t1], rows[t0:t1] = -1, -1
            if slot is None:
                granted.append(0)
                continue
            if t0 < 0 or t1 < t0 or t1 > total or p < 0 or p + t1 - t0 > max_pages * self.page:
                self.err |= SEQ
                granted.append(0)
                continue
            if not 0 <= self.held[slot] <= max_pages:
                self.err |= PAGE
                granted.append(0)
                continue
            need = 0
            if t1 > t0:
                need = max(0, -(-(p + t1 - t0) // self.page) - self.held[slot])
            asked += need
            ok = need == 0 or asked <= top
            granted.append(int(ok))
            for _ in range(need if ok else 0):
                left -= 1
                self._page(self.free[left])
                self.table[slot, self.held[slot]] = self.free[left]
                self.held[slot] += 1
            for t in range(t0, t1):
                positions[t] = p + t - t0
                if ok:
                    at = self.table[slot, (p + t - t0) // self.page]
                    if 0 <= at < n_pages:
                        rows[t] = at * self.page + (p + t - t0) % self.page
                    else:
                        self.err |= PAGE
        if left < top:
            self.n_free = left
        return granted

    def trim(self, slot_ids, lens):
        n_pages, max_pages = len(self.free), self.table.shape[1]
        drops, back = [], 0
        for i in range(len(slot_ids)):
            slot = self._slot(slot_ids, i)
            if slot is None:
                continue
            if lens[i] < 0:
                self.err |= SEQ
                continue
            if not 0 <= self.held[slot] <= max_pages:
                self.err |= PAGE
                continue
            keep = -(-int(lens[i]) // self.page)
            if self.held[slot] > keep:
                drops.append((slot, keep))
                back += self.held[slot] - keep
        if not 0 <= self.n_free <= n_pages or self.n_free + back > n_pages:
            self.err |= PAGE
            return
        self.n_free += back
        at = self.n_free
        for slot, keep in drops:
            for col in range(keep, self.held[slot]):
                at -= 1
                self._page(self.table[slot, col])
                self.free[at] = int(self.table[slot, col])
                self.table[slot, col] = -1
            self.held[slot] = keep

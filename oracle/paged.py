"""fp64 definitions of the paged-cache operators: attention whose keys lie in
pages, its latent form, and the upkeep of a page table.  numpy and Python
lists only; one sequence, one list entry at a time."""

import numpy as np


def gather(pages, row, n):
    """The first n keys that a table row names: pages [P, ..., page, d] (keys
    on the last axis but one) -> [..., n, d]."""
    size = pages.shape[-2]
    keys = [pages[row[j // size]][..., j % size, :] for j in range(n)]
    if not keys:
        return np.zeros(pages.shape[1:-2] + (0, pages.shape[-1]))
    return np.stack(keys, axis=-2)


def _rows(q, k, v, n, n_q, t, scale, causal):
    end = n if not causal else min(n, max(0, n - n_q + t + 1))
    if end == 0:
        return np.zeros(v.shape[-1]), -np.inf, np.zeros(v.shape[-1])
    s = float(np.float32(scale)) * (k[:end] @ q)
    m = s.max()
    lse = m + np.log(np.exp(s - m).sum())
    p = np.exp(s - lse)
    return p @ v[:end], lse, p @ np.abs(v[:end])


def paged_decode(q, k_pages, v_pages, table, lens, scale, causal=True):
    """q [B, H, n_q, d], pages [P, H_kv, page, d].  Returns O, L and
    A = sum_j P_j |V_j|, the magnitude that rounding P acts on."""
    B, H, n_q, _ = q.shape
    H_kv, d_v = k_pages.shape[1], v_pages.shape[-1]
    O = np.zeros((B, H, n_q, d_v))
    A = np.zeros_like(O)
    L = np.zeros((B, H, n_q))
    for b in range(B):
        n = int(lens[b])
        k, v = gather(k_pages, table[b], n), gather(v_pages, table[b], n)
        for h in range(H):
            for t in range(n_q):
                O[b, h, t], L[b, h, t], A[b, h, t] = _rows(
                    q[b, h, t], k[h // (H // H_kv)], v[h // (H // H_kv)], n, n_q, t, scale, causal)
    return O, L, A


def latent_decode(q, c_pages, table, lens, scale, d_v, causal=True):
    """q [B, H, n_q, D], c_pages [P, page, D]: the vectors are keys, their
    first d_v columns values, of all heads."""
    c = c_pages[:, None]
    return paged_decode(q, c, c[..., :d_v], table, lens, scale, causal)


class PageTable:
    """A page table as plain lists; each method does what the device call of
    its name documents and returns what it returns."""

    def __init__(self, table, lens, refs, page_size):
        self.table = [list(map(int, r)) for r in table]
        self.lens = list(map(int, lens))
        self.refs = list(map(int, refs))
        self.size = page_size

    def held(self, n):
        return -(-n // self.size)

    def free_pages(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def extend(self, seqs, new_lens):
        free, seen, full = self.free_pages(), set(), False
        cap = len(self.table[0]) * self.size
        for s, n in zip(seqs, new_lens):
            if not 0 <= s < len(self.table) or s in seen:
                continue
            seen.add(s)
            if n < self.lens[s] or n > cap:
                continue
            need = self.held(n) - self.held(self.lens[s])
            if need and (full or need > len(free)):
                full = True
                continue
            for j in range(self.held(self.lens[s]), self.held(n)):
                self.table[s][j] = free.pop(0)
                self.refs[self.table[s][j]] = 1
            self.lens[s] = n

    def fork(self, parents, children, pools=()):
        free, seen, new = self.free_pages(), set(), []
        lens, refs = list(self.lens), list(self.refs)
        for p, c in zip(parents, children):
            rows = range(len(self.table))
            if c not in rows or c in seen:
                new.append(-2)
                continue
            seen.add(c)
            if p not in rows or lens[c] != 0:
                new.append(-2)
                continue
            full, rest = divmod(lens[p], self.size)
            held = self.table[p][:self.held(lens[p])]
            if (lens[p] < 0 or lens[p] > len(self.table[p]) * self.size
                    or not all(0 <= g < len(refs) and refs[g] > 0 for g in held)):
                new.append(-2)
                continue
            if rest and not free:
                new.append(-2)
                continue
            for j in range(full):
                self.table[c][j] = self.table[p][j]
                self.refs[self.table[p][j]] += 1
            new.append(free.pop(0) if rest else -1)
            if rest:
                self.table[c][full] = new[-1]
                self.refs[new[-1]] = 1
                for pool in pools:
                    pool[new[-1]] = pool[self.table[p][full]]
            self.lens[c] = lens[p]
        return new

    def free(self, seqs):
        for s in seqs:
            if not 0 <= s < len(self.table):
                continue
            for j in range(self.held(self.lens[s])):
                self.refs[self.table[s][j]] -= 1
                self.table[s][j] = -1
            self.lens[s] = 0

    def compact(self, pools=()):
        used = [p for p, r in enumerate(self.refs) if r]
        holes = [p for p in range(len(used)) if self.refs[p] == 0]
        moved = [p if r else -1 for p, r in enumerate(self.refs)]
        for src, dst in zip([p for p in used if p >= len(used)], holes):
            moved[src] = dst
            self.refs[dst], self.refs[src] = self.refs[src], 0
            for pool in pools:
                pool[dst] = pool[src]
        for row, n in zip(self.table, self.lens):
            for j in range(self.held(n)):
                row[j] = moved[row[j]]
        return moved

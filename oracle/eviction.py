"""fp64 definitions of the attention weight of cached keys and of eviction by it.
numpy and Python lists; one sequence, one head at a time."""

import numpy as np

from .paged import gather


def key_weights(q, k_pages, table, lens, lse, scale, causal=True):
    """W [B][H_kv, n]: what the rows of q [B, H, n_q, d] with logsumexps lse [B, H, n_q]
    give each cached key; and T, the largest scale * sum |q_c k_c| of all."""
    B, H, n_q, _ = q.shape
    H_kv = k_pages.shape[1]
    W, T = [], 0.0
    for b in range(B):
        n = int(lens[b])
        k = gather(k_pages, table[b], n)
        w = np.zeros((H_kv, n))
        for h in range(H):
            for t in range(n_q):
                end = n if not causal else min(n, max(0, n - n_q + t + 1))
                if end == 0 or np.isneginf(lse[b, h, t]):
                    continue
                g = h // (H // H_kv)
                c = float(np.float32(scale))
                w[g, :end] += np.exp(c * (k[g, :end] @ q[b, h, t]) - lse[b, h, t])
                T = max(T, c * (np.abs(k[g, :end]) @ np.abs(q[b, h, t])).max())
        W.append(w)
    return W, T


def kept(weights, n, new_len, recent):
    """The slots, ascending, that a head with these weights keeps of its n keys."""
    r = min(recent, new_len)
    w = np.where(np.isnan(weights[:n - r]), np.inf, weights[:n - r])
    # (a NaN above an infinity)
    order = np.lexsort((np.arange(n - r), -np.isnan(weights[:n - r]).astype(int), -w))
    return np.concatenate([np.sort(order[:new_len - r]), np.arange(n - r, n)]).astype(int)


def evict(twin, pools, weights, seqs, new_lens, recent):
    """pages_evict on a paged.PageTable and numpy arrays: pools [P, H, page, ...],
    weights [rows, H, width].  Returns slots [n, H, width]."""
    H, width = weights.shape[1:]
    slots = np.full((len(seqs), H, width), -1, dtype=np.int32)
    size, seen = twin.size, set()
    refs, before = list(twin.refs), [list(r) for r in twin.table]
    lens = list(twin.lens)
    for i, (s, new) in enumerate(zip(seqs, new_lens)):
        first = s not in seen
        seen.add(s)
        ok = first and 0 <= s < len(lens) and new >= 0 and 0 <= lens[s] <= len(before[s]) * size
        if ok:
            held = before[s][:twin.held(lens[s])]
            stay = twin.held(new) if new < lens[s] else 0
            ok = all(0 <= g < len(refs) and (refs[g] == 1 if j < stay else refs[g] > 0)
                     for j, g in enumerate(held))
        if not ok:
            slots[i] = -2
            continue
        old = lens[s]
        if new >= old:
            slots[i, :, :old] = np.arange(old)
            continue
        for h in range(H):
            src = kept(weights[s, h], old, new, recent)
            slots[i, h, :new] = src
            weights[s, h, :old] = np.concatenate([weights[s, h, src], np.zeros(old - new)])
            page = np.array(before[s])
            at, to = np.arange(new), src
            for x in pools:
                x[page[at // size], h, at % size] = x[page[to // size], h, to % size].copy()
        for j in range(twin.held(new), twin.held(old)):
            twin.refs[before[s][j]] -= 1
            twin.table[s][j] = -1
        twin.lens[s] = new
    return slots

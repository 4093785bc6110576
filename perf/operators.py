"""What the serving operators over a paged key/value cache are measured on.

Five paths: the decode step against a paged cache, the same step for a batch
whose sequences share a long prefix, the decode step against a paged cache of
latent vectors, forking sequences of a paged cache, and freeing sequences and
compacting what is left.  `run` computes each in its plain form (elementary
torch operations in 32 bits) or, with `own`, through the package.
"""

import math

import numpy as np
import torch

own = False

ROPE = 64   # columns of a latent vector beside the d_v that are also the values


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one chat turn: a single sequence, one new token, a short cache of small pages
        dict(name="paged-single", op="paged", B=1, H=32, H_kv=8, d=128, n_q=1, page=16, lo=517,
             hi=517, causal=True),
        # an ordinary serving batch: the decode-gqa-8k workload's heads and lengths, in pages
        dict(name="paged-batch", op="paged", B=16, H=32, H_kv=8, d=128, n_q=1, page=64, lo=4096,
             hi=8192, causal=True),
        # verifying four drafted tokens for many sequences of very different lengths
        dict(name="paged-drafts", op="paged", B=64, H=64, H_kv=8, d=128, n_q=4, page=128, lo=0,
             hi=16384, causal=True),
        # a few samples of one short prompt
        dict(name="shared-small", op="shared", B=4, H=16, H_kv=4, d=64, n_q=1, page=16,
             shared=1024, lo=1, hi=65, causal=True),
        # many requests about one long document
        dict(name="shared-document", op="shared", B=128, H=32, H_kv=8, d=128, n_q=1, page=64,
             shared=16384, lo=64, hi=1024, causal=True),
        # one sequence against a short cache of latent vectors
        dict(name="latent-single", op="latent", B=1, H=16, d_v=512, n_q=1, page=64, lo=700,
             hi=700, causal=True),
        # a serving batch whose heads are divided over several devices
        dict(name="latent-batch", op="latent", B=32, H=16, d_v=512, n_q=1, page=64, lo=0,
             hi=8192, causal=True),
        # a serving batch with all heads on one device
        dict(name="latent-wide", op="latent", B=64, H=128, d_v=512, n_q=1, page=64, lo=4096,
             hi=8192, causal=True),
        # four samples branch off one short prompt
        dict(name="fork-prompt", op="fork", parents=1, branch=4, H_kv=8, d=128, page=16, lo=333,
             hi=333),
        # a search step: every sequence of a batch branches eight ways
        dict(name="fork-search", op="fork", parents=64, branch=8, H_kv=8, d=128, page=64, lo=1024,
             hi=4096),
        # a small cache of short sequences, a quarter of which have ended
        dict(name="compact-small", op="compact", S=16, drop=4, H_kv=8, d=128, page=16, lo=0,
             hi=300),
        # every other sequence of a large cache has ended: free its pages, close the gaps
        dict(name="compact-cache", op="compact", S=128, drop=64, H_kv=8, d=128, page=64, lo=1024,
             hi=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["paged", "paged", "shared", "latent", "latent", "fork", "compact"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op in ("paged", "shared"):
        H_kv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 3, 4, 5, 8])
        n_q = rng.choice([1, 1, 1, 2, 3, 5])
        c = dict(op=op, B=_log(rng, 1, 96), H=H_kv * group, H_kv=H_kv, d=rng.choice([64, 128]),
                 n_q=n_q, page=page, causal=rng.random() < 0.8)
        if op == "shared":
            c["shared"] = page * max(1, _log(rng, 64, 12000) // page)
            c["lo"] = rng.choice([n_q, 33])
            c["hi"] = c["lo"] + _log(rng, 1, 900)
        else:
            c["hi"] = _log(rng, 1, 12000)
            c["lo"] = rng.choice([0, 1, c["hi"] // 3, c["hi"]])
        return c
    if op == "latent":
        hi = _log(rng, 1, 8000)
        return dict(op=op, B=_log(rng, 1, 56), H=rng.choice([8, 16, 20, 32, 64, 128]),
                    d_v=rng.choice([256, 512, 512]), n_q=rng.choice([1, 1, 1, 2, 3]) if hi < 4000 else 1,
                    page=page, lo=rng.choice([0, 1, hi // 2]), hi=hi, causal=rng.random() < 0.8)
    hi = _log(rng, 1, 4000)
    c = dict(op=op, H_kv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128]), page=page,
             lo=rng.choice([0, 1, hi // 2]), hi=hi)
    if op == "fork":
        c.update(parents=_log(rng, 1, 48), branch=rng.randint(1, 8))
    else:
        c["S"] = _log(rng, 2, 120)
        c["drop"] = max(1, int(c["S"] * rng.uniform(0.1, 0.9)))
    return c


# ------------------------------------------------------------------ inputs --

def _lens(case, seed, n):
    r = np.random.RandomState(seed % (1 << 31))
    return torch.from_numpy(r.randint(case["lo"], case["hi"] + 1, n).astype(np.int32))


def _normal(shape, g, std=1.0):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    return x if std == 1.0 else x * std


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, page = case["op"], case["page"]
    s = dict(case=case)
    if op in ("paged", "shared", "latent"):
        B, H, n_q, shared = case["B"], case["H"], case["n_q"], case.get("shared", 0)
        lens = _lens(case, seed, B)
        own_pages = -(-case["hi"] // page) if case["hi"] else 1
        pre = shared // page
        P = B * own_pages + pre + 3
        perm = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
        table = torch.empty(B, pre + own_pages, dtype=torch.int32, device="cuda")
        table[:, :pre] = perm[:pre]
        table[:, pre:] = perm[pre:pre + B * own_pages].view(B, own_pages)
        s.update(table=table, lens=lens.cuda() + shared, shared=shared, causal=case["causal"])
        if op == "latent":
            D = case["d_v"] + ROPE
            s.update(c_pages=_normal((P, page, D), g), q=_normal((B, H, n_q, D), g, 0.5),
                     d_v=case["d_v"], scale=(128 + ROPE) ** -0.5 / 2)
        else:
            shape = (P, case["H_kv"], page, case["d"])
            s.update(k_pages=_normal(shape, g), v_pages=_normal(shape, g),
                     q=_normal((B, H, n_q, case["d"]), g), scale=case["d"] ** -0.5)
        return s
    # fork, compact: a cache of sequences with their page tables and reference counts, all three
    # in one buffer that a pass starts from anew
    rows = case["parents"] * (1 + case["branch"]) if op == "fork" else case["S"]
    filled = case["parents"] if op == "fork" else case["S"]
    most = max(1, -(-case["hi"] // page))
    lens = torch.zeros(rows, dtype=torch.int32)
    lens[:filled] = _lens(case, seed, filled)
    count = (lens + page - 1) // page
    P = filled * most + (rows - filled) + 2
    perm = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    table = torch.full((rows, most), -1, dtype=torch.int32, device="cuda")
    used = torch.arange(most) < count[:, None]
    n = int(count.sum())
    table[used.cuda()] = perm[:n]
    refs = torch.zeros(P, dtype=torch.int32, device="cuda")
    refs[perm[:n].long()] = 1
    start = torch.cat([table.reshape(-1), lens.cuda(), refs])
    meta = start.clone()
    a, b = rows * most, rows * most + rows
    shape = (P, case["H_kv"], page, case["d"])
    s.update(start=start, meta=meta, table=meta[:a].view(rows, most), lens=meta[a:b],
             refs=meta[b:], k_pages=_normal(shape, g), v_pages=_normal(shape, g), page=page)
    if op == "fork":
        s["parents"] = torch.arange(filled, dtype=torch.int32, device="cuda").repeat_interleave(
            case["branch"])
        s["children"] = torch.arange(filled, rows, dtype=torch.int32, device="cuda")
    else:
        r = np.random.RandomState((seed + 1) % (1 << 31))
        s["ended"] = torch.from_numpy(r.permutation(rows)[:case["drop"]].astype(np.int32)).cuda()
    return s


# -------------------------------------------------------------- plain forms --

def _allowed(lens, n_q, first, n, causal):
    """bool [B, n_q, n]: which of the keys first .. first + n - 1 each query row attends."""
    j = torch.arange(first, first + n, device=lens.device)
    last = lens[:, None].expand(-1, n_q)
    if causal:
        last = torch.minimum(last, lens[:, None] - n_q + 1 + torch.arange(n_q, device=lens.device))
    return j < last[:, :, None]


def _softmax(scores, allowed):
    """Probabilities and logsumexp over the last axis; a row with nothing allowed: 0 and -inf."""
    scores = torch.where(allowed, scores, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    base = torch.where(torch.isinf(top), 0.0, top)
    e = torch.exp(scores - base)
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, 1.0, total), (base + torch.log(total)).squeeze(-1)


def _gather(pages, table):
    """[P, H_kv, page, d] by a table [B, n] -> [B, H_kv, n * page, d], 32 bits."""
    x = pages[table.long()].transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[4]).float()


def _plain_decode(s):
    q, lens, shared, scale = s["q"], s["lens"], s["shared"], s["scale"]
    B, H, n_q, d = q.shape
    H_kv, page = s["k_pages"].shape[1:3]
    qg = q.float().reshape(B, H_kv, -1, d)
    pre = shared // page
    k, v = (_gather(s[x], s["table"][:, pre:]) for x in ("k_pages", "v_pages"))
    scores = torch.matmul(qg, k.transpose(2, 3))
    if shared:   # the prefix once, for the rows of all sequences together
        kp, vp = (_gather(s[x], s["table"][:1, :pre])[0] for x in ("k_pages", "v_pages"))
        rows = qg.transpose(0, 1).reshape(H_kv, -1, d)
        before = torch.matmul(rows, kp.transpose(1, 2)).reshape(H_kv, B, -1, shared).transpose(0, 1)
        scores = torch.cat([before, scores], -1)
    scores = scores.reshape(B, H, n_q, -1) * scale
    p, lse = _softmax(scores, _allowed(lens, n_q, 0, scores.shape[-1], s["causal"])[:, None])
    p = p.reshape(B, H_kv, -1, p.shape[-1])
    o = torch.matmul(p[..., shared:], v)
    if shared:
        rows = p[..., :shared].transpose(0, 1).reshape(H_kv, -1, shared)
        o = o + torch.matmul(rows, vp).reshape(H_kv, B, -1, d).transpose(0, 1)
    return o.reshape(B, H, n_q, d).to(q.dtype), lse


def _plain_latent(s):
    q, d_v = s["q"], s["d_v"]
    B, H, n_q, D = q.shape
    c = s["c_pages"][s["table"].long()].reshape(B, -1, D).float()
    scores = torch.matmul(q.float().reshape(B, H * n_q, D), c.transpose(1, 2)) * s["scale"]
    p, lse = _softmax(scores.reshape(B, H, n_q, -1),
                      _allowed(s["lens"], n_q, 0, c.shape[1], s["causal"])[:, None])
    o = torch.matmul(p.reshape(B, H * n_q, -1), c[..., :d_v])
    return o.reshape(B, H, n_q, d_v).to(q.dtype), lse


def _plain_fork(s):
    table, lens, refs, page = s["table"], s["lens"], s["refs"], s["page"]
    par, child = s["parents"].long(), s["children"].long()
    n = lens[par]
    part = (n % page) != 0
    held = torch.arange(table.shape[1], device=table.device) < ((n + page - 1) // page)[:, None]
    last = torch.arange(table.shape[1], device=table.device) == (n // page)[:, None]
    last = last & part[:, None]
    rows = table[par]
    # new pages for the part-filled last ones: the lowest free pages in the forks' order
    free = torch.argsort((refs != 0).to(torch.int32), stable=True).to(torch.int32)
    new = torch.where(part, free[torch.cumsum(part, 0) - part.long()], -1)
    src = torch.where(last, rows, 0).sum(1)[part]
    for_rows = torch.where(last, new[:, None], rows)
    refs.index_add_(0, for_rows.clamp(min=0).reshape(-1).long(),
                    held.reshape(-1).to(torch.int32))
    table[child] = torch.where(held, for_rows, table[child]).to(torch.int32)
    lens[child] = n
    dst = new[part].long()
    s["k_pages"][dst] = s["k_pages"][src]
    s["v_pages"][dst] = s["v_pages"][src]
    return new.to(torch.int32)


def _plain_free_compact(s):
    table, lens, refs, page = s["table"], s["lens"], s["refs"], s["page"]
    width = torch.arange(table.shape[1], device=table.device)
    ended = s["ended"].long()
    rows, held = table[ended], width < ((lens[ended] + page - 1) // page)[:, None]
    refs.index_add_(0, rows.clamp(min=0).reshape(-1).long(), -held.reshape(-1).to(torch.int32))
    table[ended] = torch.where(held, -1, rows)
    lens[ended] = 0
    # the used pages behind the first n_used places move, in order, to the free ones before it
    P = refs.shape[0]
    used = refs != 0
    at = torch.arange(P, device=refs.device)
    before = at < used.sum()
    src, dst = (used & ~before).nonzero()[:, 0], (~used & before).nonzero()[:, 0]
    moved = torch.where(used, at, -1).to(torch.int32)
    moved[src] = dst.to(torch.int32)
    s["k_pages"][dst] = s["k_pages"][src]
    s["v_pages"][dst] = s["v_pages"][src]
    refs[dst] = refs[src]
    refs[src] = 0
    held = width < ((lens + page - 1) // page)[:, None]
    table.copy_(torch.where(held, moved[table.clamp(min=0).long()], table))
    return moved


# --------------------------------------------------------------------- run --

def run(s):
    op = s["case"]["op"]
    if op in ("paged", "shared"):
        if not own:
            return _plain_decode(s)
        import exact_attention_12_gb300 as ea
        return ea.attention_decode_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                                         scale=s["scale"], causal=s["causal"],
                                         shared_len=s["shared"])
    if op == "latent":
        if not own:
            return _plain_latent(s)
        import exact_attention_12_gb300 as ea
        return ea.attention_decode_latent(s["q"], s["c_pages"], s["table"], s["lens"],
                                          scale=s["scale"], d_v=s["d_v"], causal=s["causal"])
    s["meta"].copy_(s["start"])
    if op == "fork":
        if own:
            import exact_attention_12_gb300 as ea
            new = ea.pages_fork((s["k_pages"], s["v_pages"]), s["table"], s["lens"], s["refs"],
                                s["parents"], s["children"], page_size=s["page"])
        else:
            new = _plain_fork(s)
    elif own:
        import exact_attention_12_gb300 as ea
        ea.pages_free(s["table"], s["lens"], s["refs"], s["ended"], page_size=s["page"])
        new = ea.pages_compact((s["k_pages"], s["v_pages"]), s["table"], s["lens"], s["refs"],
                               page_size=s["page"])
    else:
        new = _plain_free_compact(s)
    return new, s["table"], s["lens"], s["refs"], s["k_pages"], s["v_pages"]


def work(case):
    op, page = case["op"], case["page"]
    mean = (case["lo"] + case["hi"]) / 2
    if op in ("paged", "shared"):
        rows, d = case["B"] * case["H"] * case["n_q"], case["d"]
        keys = case["B"] * mean + case.get("shared", 0)
        bytes_ = keys * case["H_kv"] * d * 4 + rows * (4 * d + 4) + case["B"] * (mean / page + 1) * 4
        return dict(bytes=bytes_, flops=4.0 * d * rows * (mean + case.get("shared", 0)))
    if op == "latent":
        rows, D = case["B"] * case["H"] * case["n_q"], case["d_v"] + ROPE
        bytes_ = case["B"] * mean * D * 2 + rows * (2 * D + 2 * case["d_v"] + 4) \
            + case["B"] * (mean / page + 1) * 4
        return dict(bytes=bytes_, flops=2.0 * rows * mean * (D + case["d_v"]))
    page_bytes = 2 * case["H_kv"] * page * case["d"] * 2   # keys and values
    if op == "fork":
        n = case["parents"] * case["branch"]
        partial = 1 - 1 / page if case["hi"] > case["lo"] else float(case["lo"] % page != 0)
        P = case["parents"] * max(1, case["hi"] / page)
        return dict(bytes=n * partial * page_bytes * 2 + n * mean / page * 8 + 12 * P, flops=0)
    S, stay = case["S"], case["S"] - case["drop"]
    P = S * max(1, -(-case["hi"] // page)) + 2
    n_used = stay * (mean / page + 0.5)
    moves = n_used * (1 - n_used / P)
    return dict(bytes=moves * page_bytes * 2 + 8 * P + 8 * n_used, flops=0)


# ------------------------------------------------------- 64-bit definitions --

def _exact_attention(q, keys, values, scale, causal):
    """q [H, n_q, d], keys [G, n, d], values [G, n, d_v] in 64 bits, H a multiple of G."""
    H, n_q, _ = q.shape
    G, n, d_v = values.shape
    o = torch.zeros(H, n_q, d_v, dtype=torch.float64, device=q.device)
    lse = torch.full((H, n_q), float("-inf"), dtype=torch.float64, device=q.device)
    for t in range(n_q):
        end = min(n, n - n_q + t + 1) if causal else n
        if end <= 0:
            continue
        x = torch.einsum("ghd,gnd->ghn", q[:, t].reshape(G, H // G, -1), keys[:, :end]) * scale
        z = torch.logsumexp(x, -1)
        o[:, t] = torch.einsum("ghn,gnd->ghd", torch.exp(x - z[..., None]),
                               values[:, :end]).reshape(H, d_v)
        lse[:, t] = z.reshape(H)
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    op, page = case["op"], case["page"]
    if op in ("paged", "shared", "latent"):
        got = []
        for b, n in enumerate(s["lens"].tolist()):
            at = s["table"][b, :-(-n // page)].long()
            if op == "latent":
                keys = s["c_pages"][at].double().reshape(1, -1, s["q"].shape[3])[:, :n]
                values = keys[..., :s["d_v"]]
            else:
                keys, values = (s[x][at].double().permute(1, 0, 2, 3).reshape(
                    case["H_kv"], -1, case["d"])[:, :n] for x in ("k_pages", "v_pages"))
            got.append(_exact_attention(s["q"][b].double(), keys, values, s["scale"],
                                        s["causal"]))
        return torch.stack([o for o, _ in got]), torch.stack([z for _, z in got])
    table, lens, refs = (s[x].tolist() for x in ("table", "lens", "refs"))
    k, v = s["k_pages"].double(), s["v_pages"].double()
    if op == "fork":
        new = []
        free = iter([p for p, r in enumerate(refs) if r == 0])
        pairs = list(zip(s["parents"].tolist(), s["children"].tolist()))
        for p, c in pairs:
            full, rest = divmod(lens[p], page)
            lens[c] = lens[p]
            for i in range(full):
                table[c][i] = table[p][i]
                refs[table[p][i]] += 1
            new.append(next(free) if rest else -1)
            if rest:
                table[c][full] = new[-1]
                refs[new[-1]] = 1
                k[new[-1]] = k[table[p][full]]
                v[new[-1]] = v[table[p][full]]
    else:
        for e in s["ended"].tolist():
            for i in range(-(-lens[e] // page)):
                refs[table[e][i]] -= 1
                table[e][i] = -1
            lens[e] = 0
        n_used = sum(r != 0 for r in refs)
        holes = [p for p in range(n_used) if refs[p] == 0]
        new = [p if r else -1 for p, r in enumerate(refs)]
        for src in range(n_used, len(refs)):
            if refs[src]:
                dst = holes.pop(0)
                new[src] = dst
                k[dst], v[dst] = k[src], v[src]
                refs[dst], refs[src] = refs[src], 0
        for row, n in zip(table, lens):
            for i in range(-(-n // page)):
                row[i] = new[row[i]]
    return tuple(torch.tensor(x, dtype=torch.int32) for x in (new, table, lens, refs)) + (k, v)

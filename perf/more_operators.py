"""What the operators of compact key/value caches are measured on.

A paged cache held in 4 bits (E2M1 codes, an E4M3 scale per 16 columns, one factor per tensor):
storing new keys and values, the decode step that reads them.  And the eviction of keys by the
attention weight that they have gathered: adding up the weights, keeping the heaviest keys.  `run`
computes each in its plain form (elementary torch operations in 32 bits) or, with `own`, through the
package.
"""

import math

import numpy as np
import torch

own = False

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)   # of a code's low three bits; bit 3 is the sign
BLOCK = 16                                           # columns that share a scale


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one chat turn: a single sequence, one new token, a short cache of small pages
        dict(name="decode-single", op="decode", B=1, H=32, H_kv=8, d=128, n_q=1, page=16, lo=517,
             hi=517, causal=True),
        # an ordinary serving batch
        dict(name="decode-batch", op="decode", B=16, H=32, H_kv=8, d=128, n_q=1, page=64, lo=4096,
             hi=8192, causal=True),
        # verifying four drafted tokens for many sequences of very different lengths
        dict(name="decode-drafts", op="decode", B=64, H=64, H_kv=8, d=128, n_q=4, page=128, lo=0,
             hi=16384, causal=True),
        # two very long sequences, narrow heads
        dict(name="decode-long", op="decode", B=2, H=16, H_kv=2, d=64, n_q=1, page=256, lo=100000,
             hi=131072, causal=True),
        # every sequence of a batch stores its newest token
        dict(name="store-step", op="store", B=64, H_kv=8, d=128, n=1, page=64, lo=1, hi=4096),
        # prompts of different lengths are stored whole
        dict(name="store-prompt", op="store", B=8, H_kv=8, d=128, n=8192, page=64, lo=1000,
             hi=8192),
        # the weights that one step's queries give, added to what the keys have gathered
        dict(name="weights-step", op="weights", B=16, H=32, H_kv=8, d=128, n_q=1, page=64, lo=2048,
             hi=8192, causal=True, bits=16, add=True),
        # a prompt's keys judged by its last 32 queries
        dict(name="weights-window", op="weights", B=2, H=32, H_kv=8, d=128, n_q=32, page=64,
             lo=16384, hi=16384, causal=True, bits=16, add=False),
        # the same step on a short cache in 4 bits
        dict(name="weights-step-4bit", op="weights", B=4, H=16, H_kv=4, d=64, n_q=1, page=16,
             lo=300, hi=1500, causal=True, bits=4, add=True),
        # one sequence has outgrown its budget by a few pages
        dict(name="evict-small", op="evict", S=1, H_kv=8, d=128, page=16, lo=333, hi=333, keep=256,
             recent=32, bits=16),
        # a serving batch is brought back to its budget
        dict(name="evict-batch", op="evict", S=32, H_kv=8, d=128, page=64, lo=2048, hi=8192,
             keep=4096, recent=256, bits=16),
        # long sequences in 4 bits lose three quarters of their keys
        dict(name="evict-long-4bit", op="evict", S=4, H_kv=8, d=128, page=128, lo=90000, hi=100000,
             keep=24000, recent=1024, bits=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "store", "weights", "weights", "evict", "evict"])
    c = dict(op=op, H_kv=rng.choice([1, 2, 3, 4, 8]), d=rng.choice([64, 128]),
             page=rng.choice([16, 32, 64, 128, 256]))
    if op == "store":
        hi = _log(rng, 1, 6000)
        c.update(B=_log(rng, 1, 64 if hi < 600 else 8), hi=hi, lo=rng.choice([0, 1, hi // 2, hi]),
                 n=rng.choice([1, 1, max(1, hi // 3), hi]))
        return c
    hi = _log(rng, 1, 14000)
    c.update(hi=hi, lo=rng.choice([0, 1, hi // 3, hi]))
    if op == "evict":
        hi = c["hi"] = min(hi, 8000)
        c["lo"] = min(c["lo"], hi)
        c.update(S=_log(rng, 1, 16), bits=rng.choice([16, 4]), keep=_log(rng, 1, hi),
                 recent=rng.choice([0, 1, _log(rng, 1, 400)]))
        return c
    n_q = rng.choice([1, 1, 1, 2, 3, 5])
    c.update(B=_log(rng, 1, 48), causal=rng.random() < 0.8, n_q=n_q,
             H=c["H_kv"] * rng.choice([1, 2, 3, 4, 5, 8]))
    if op == "weights":
        c.update(bits=rng.choice([16, 4]), add=rng.random() < 0.5)
        if rng.random() < 0.25:
            c.update(n_q=_log(rng, 8, 40), B=min(c["B"], 4))
    return c


# ------------------------------------------------------------------ inputs --

def _lens(case, seed, n):
    r = np.random.RandomState(seed % (1 << 31))
    return torch.from_numpy(r.randint(case["lo"], case["hi"] + 1, n).astype(np.int32))


def _normal(shape, g, std=1.0):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    return x if std == 1.0 else x * std


# the code that stands for the i-th 256-quantile of a normal distribution whose blocks of 16 have
# their largest values at 6 (about 2 standard deviations)
_EDGES = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]) / 2.9


def _code_table():
    x = torch.special.ndtri((torch.arange(256) + 0.5) / 256)
    return (torch.bucketize(x.abs(), _EDGES) + 8 * (x < 0)).to(torch.uint8)


def _packed(shape, g):
    """Codes [..., d / 2] of normal values, and their scales [..., d / 16]."""
    table = _code_table().cuda()
    one = shape[:-1] + (shape[-1] // 2,)
    lo, hi = (table[torch.randint(0, 256, one, generator=g, device="cuda",
                                  dtype=torch.uint8).int()] for _ in range(2))
    scales = torch.rand(shape[:-1] + (shape[-1] // BLOCK,), generator=g, device="cuda")
    # of values of deviation 1 with a factor that takes their largest to the largest scale's
    return lo | hi << 4, (100.0 + 160.0 * scales).to(torch.float8_e4m3fn)


def _table(rows, most, spare, g):
    P = rows * most + spare
    perm = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    return perm[:rows * most].view(rows, most).contiguous(), P


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, page, H_kv, d = case["op"], case["page"], case["H_kv"], case["d"]
    most = max(1, -(-case["hi"] // page))
    s = dict(case=case, page=page)
    if op == "evict":
        S = case["S"]
        lens = _lens(case, seed, S)
        table, P = _table(S, most, 3, g)
        held = torch.arange(most) < ((lens + page - 1) // page)[:, None]
        table[~held.cuda()] = -1
        refs = torch.zeros(P, dtype=torch.int32, device="cuda")
        refs[table[held.cuda()].long()] = 1
        start = torch.cat([table.reshape(-1), lens.cuda(), refs])
        meta = start.clone()
        a, b = S * most, S * most + S
        s.update(start=start, meta=meta, table=meta[:a].view(S, most), lens=meta[a:b],
                 refs=meta[b:], seqs=torch.arange(S, dtype=torch.int32, device="cuda"),
                 new_lens=torch.full((S,), case["keep"], dtype=torch.int32, device="cuda"),
                 recent=case["recent"])
        # gathered weights: a few keys have most, many about the same little
        w = torch.randn(S, H_kv, most * page, generator=g, device="cuda").mul(2.0).exp()
        w = torch.where(w < 0.2, (w * 64).round() / 64, w)
        s.update(weights0=w, weights=w.clone())
        if case["bits"] == 16:
            s["pools"] = tuple(_normal((P, H_kv, page, d), g) for _ in range(2))
        else:
            s["pools"] = tuple(x for _ in range(2) for x in _packed((P, H_kv, page, d), g))
        return s
    B = case["B"]
    lens = _lens(case, seed, B)
    table, P = _table(B, most, 3, g)
    s.update(table=table, lens=lens.cuda())
    if op == "store":
        n = case["n"]
        counts = torch.minimum(lens, torch.tensor(n, dtype=torch.int32))
        # keys and values come with a few large columns, as projections give them
        wide = torch.ones(d, device="cuda", dtype=torch.bfloat16)
        wide[torch.randperm(d, generator=g, device="cuda")[:d // 16]] = 6.0
        k, v = (_normal((B, H_kv, n, d), g) * wide for _ in range(2))
        shape = (P, H_kv, page, d)
        # a program's calibration: the largest value over the largest that the format holds
        s.update(k=k, v=v, n=n, counts=counts.cuda(), k_descale=float(np.float32(24.0 / 2688)),
                 v_descale=float(np.float32(17.0 / 2688)))
        for x in ("k", "v"):
            s[x + "_codes"] = torch.zeros(shape[:3] + (d // 2,), dtype=torch.uint8, device="cuda")
            s[x + "_scales"] = torch.zeros(shape[:3] + (d // BLOCK,), dtype=torch.float8_e4m3fn,
                                           device="cuda")
        return s
    H, n_q = case["H"], case["n_q"]
    shape = (P, H_kv, page, d)
    s.update(q=_normal((B, H, n_q, d), g), scale=d ** -0.5, causal=case["causal"])
    if op == "decode" or case["bits"] == 4:
        s["k_codes"], s["k_scales"] = _packed(shape, g)
        s["k_descale"] = float(np.float32(1 / (2.9 * 180)))
    else:
        s["k_pages"] = _normal(shape, g)
    if op == "decode":
        s["v_codes"], s["v_scales"] = _packed(shape, g)
        s["v_descale"] = float(np.float32(1 / (2.9 * 170)))
    else:
        # the logsumexps are the decode step's, in 32 bits; the weights what earlier steps gave
        rows = [_scores(s, b) for b in range(B)]
        s["lse"] = torch.stack([torch.logsumexp(x, -1) for x in rows])
        w = torch.rand(B, H_kv, most * page, generator=g, device="cuda")
        s.update(weights0=w, weights=w.clone(), add=case["add"])
    return s


# -------------------------------------------------------------- plain forms --

def _decoded(codes, scales, descale):
    """The values that codes [..., d / 2] and scales [..., d / 16] stand for, 32 bits."""
    level = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=codes.device)
    byte = torch.arange(256, device=codes.device)
    pairs = torch.stack([level[byte & 15], level[byte >> 4]], -1)
    x = pairs[codes.int()].reshape(scales.shape + (BLOCK,))
    return (x * (scales.float()[..., None] * descale)).reshape(codes.shape[:-1] + (-1,))


def _allowed(lens, n_q, n, causal):
    """bool [B, n_q, n]: which keys each query row attends."""
    j = torch.arange(n, device=lens.device)
    last = lens[:, None].expand(-1, n_q)
    if causal:
        last = torch.minimum(last, lens[:, None] - n_q + 1 + torch.arange(n_q, device=lens.device))
    return j < last[:, :, None]


def _keys(s, at):
    """The keys of the pages `at` [..., n]: [..., H_kv, n * page, d], 32 bits."""
    x = _decoded(s["k_codes"][at], s["k_scales"][at], s["k_descale"]) if "k_codes" in s \
        else s["k_pages"][at].float()
    x = x.transpose(-4, -3)
    return x.reshape(x.shape[:-3] + (-1, x.shape[-1]))


def _scores(s, b):
    """Masked scores of sequence b, [H, n_q, n], 32 bits."""
    q = s["q"][b]
    H, n_q, d = q.shape
    k = _keys(s, s["table"][b].long())
    x = torch.matmul(q.float().reshape(k.shape[0], -1, d), k.transpose(1, 2)) * s["scale"]
    ok = _allowed(s["lens"][b:b + 1], n_q, k.shape[1], s["causal"])[0]
    return torch.where(ok, x.reshape(H, n_q, -1), float("-inf"))


def _plain_decode(s):
    q, at = s["q"], s["table"].long()
    B, H, n_q, d = q.shape
    k = _keys(s, at)
    H_kv = k.shape[1]
    x = torch.matmul(q.float().reshape(B, H_kv, -1, d), k.transpose(2, 3)) * s["scale"]
    ok = _allowed(s["lens"], n_q, k.shape[2], s["causal"])[:, None]
    x = torch.where(ok, x.reshape(B, H, n_q, -1), float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total == 0, 1.0, total)
    v = _decoded(s["v_codes"][at], s["v_scales"][at], s["v_descale"]).transpose(1, 2)
    o = torch.matmul(p.reshape(B, H_kv, -1, p.shape[-1]), v.reshape(B, H_kv, -1, d))
    return o.reshape(B, H, n_q, d).to(q.dtype), (top + torch.log(total)).squeeze(-1)


def _plain_weights(s):
    q, lse = s["q"], s["lse"]
    B, H, n_q, d = q.shape
    k = _keys(s, s["table"].long())
    H_kv = k.shape[1]
    x = torch.matmul(q.float().reshape(B, H_kv, -1, d), k.transpose(2, 3)) * s["scale"]
    ok = _allowed(s["lens"], n_q, k.shape[2], s["causal"])[:, None]
    z = torch.where(torch.isinf(lse), 0.0, lse)[..., None]
    p = torch.where(ok, torch.exp(x.reshape(B, H, n_q, -1) - z), 0.0)
    got = p.reshape(B, H_kv, -1, p.shape[-1]).sum(2)
    there = torch.arange(got.shape[2], device=q.device) < s["lens"][:, None, None]
    base = s["weights"] if s["add"] else 0.0
    s["weights"].copy_(torch.where(there, base + got, s["weights"]))
    return s["weights"]


def _nearest(x, steps):
    """Index of the nearest of the ascending `steps`, ties to the even index (64 bits: the values
    lie on the borders often)."""
    middle = (steps[1:] + steps[:-1]) / 2
    up, down = torch.bucketize(x, middle, right=True), torch.bucketize(x, middle)
    return torch.where(up % 2 == 0, up, down)


def _plain_store(s):
    B, H_kv, n, d = s["k"].shape
    page = s["page"]
    t = torch.arange(n, device="cuda")
    live = t < s["counts"][:, None]
    at = torch.where(live, (s["lens"] - s["counts"])[:, None] + t, 0).long()
    pages = torch.gather(s["table"].long(), 1, at // page)
    b, t = live.nonzero(as_tuple=True)
    to, row = pages[b, t], (at % page)[b, t]
    e4m3 = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    levels = torch.tensor(LEVELS, dtype=torch.float64, device="cuda")
    got = []
    for name in ("k", "v"):
        x, descale = s[name].transpose(1, 2)[b, t], s[name + "_descale"]
        x = x.reshape(x.shape[:-1] + (-1, BLOCK)).double() / descale
        scale = _nearest(x.abs().amax(-1) / 6, e4m3)
        unit = e4m3[scale][..., None]
        code = _nearest(x.abs() / torch.where(unit == 0, 1.0, unit), levels)
        code = (torch.where(unit == 0, 0, code) + 8 * (x < 0)).to(torch.uint8).flatten(-2)
        s[name + "_codes"][to, :, row] = code[..., ::2] | code[..., 1::2] << 4
        s[name + "_scales"].view(torch.uint8)[to, :, row] = scale.to(torch.uint8)
        # and back
        x = _decoded(s[name + "_codes"][to, :, row], s[name + "_scales"].view(torch.uint8)[
            to, :, row].view(torch.float8_e4m3fn), descale).to(torch.bfloat16)
        y = torch.zeros(B, n, H_kv, d, dtype=torch.bfloat16, device="cuda")
        y[b, t] = x
        got.append(y.transpose(1, 2).contiguous())
    return tuple(got)


def _plain_evict(s):
    table, lens, refs, page, w = s["table"], s["lens"], s["refs"], s["page"], s["weights"]
    S, H, W = w.shape
    j = torch.arange(W, device=w.device)
    old = lens[s["seqs"].long()].long()
    new = torch.minimum(s["new_lens"].long(), old)
    recent = torch.minimum(new, torch.tensor(s["recent"], device=w.device))
    # keys in the order of their claim: the recent ones, then by weight, the lower slot first
    rank = torch.where(j < old[:, None, None], w, -1.0)
    rank = torch.where((j >= (old - recent)[:, None, None]) & (j < old[:, None, None]),
                       float("inf"), rank)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    mine = torch.arange(W, device=w.device) < new[:, None, None]
    kept = torch.zeros_like(w, dtype=torch.bool).scatter_(2, order, mine.expand_as(order))
    slots = torch.sort(torch.where(kept, j, W), dim=-1).values
    slots = torch.where(slots == W, -1, slots)
    i, h, to = (slots >= 0).nonzero(as_tuple=True)
    src = slots[i, h, to]
    gone = (j >= new[:, None, None]) & (j < old[:, None, None])
    moved = torch.where(slots >= 0, torch.gather(w, 2, slots.clamp(min=0)), w)
    w.copy_(torch.where(gone, 0.0, moved))
    # rows that stay where they are need no move
    away = src != to
    i, h, to, src = i[away], h[away], to[away], src[away]
    pages = table.long()
    for pool in s["pools"]:
        x = pool.view(torch.uint8) if pool.element_size() == 1 else pool
        x[pages[i, to // page], h, to % page] = x[pages[i, src // page], h, src % page]
    held = torch.arange(table.shape[1], device=w.device) < ((old + page - 1) // page)[:, None]
    stay = torch.arange(table.shape[1], device=w.device) < ((new + page - 1) // page)[:, None]
    back = held & ~stay
    refs.index_add_(0, table.clamp(min=0).reshape(-1).long(), -back.reshape(-1).to(torch.int32))
    table.copy_(torch.where(back, -1, table))
    lens.copy_(new)
    return slots.to(torch.int32)


# --------------------------------------------------------------------- run --

def run(s):
    op = s["case"]["op"]
    if own:
        import exact_attention_12_gb300 as ea
    if op == "decode":
        if not own:
            return _plain_decode(s)
        return ea.attention_decode_fp4(s["q"], s["k_codes"], s["k_scales"], s["v_codes"],
                                       s["v_scales"], s["table"], s["lens"], scale=s["scale"],
                                       causal=s["causal"], k_descale=s["k_descale"],
                                       v_descale=s["v_descale"])
    if op == "store":
        if not own:
            return _plain_store(s)
        cache = (s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["table"], s["lens"])
        factors = dict(k_descale=s["k_descale"], v_descale=s["v_descale"], counts=s["counts"])
        ea.pages_store_fp4(s["k"], s["v"], *cache, **factors)
        return ea.pages_load_fp4(*cache, s["n"], **factors)
    if op == "weights":
        if s["add"]:
            s["weights"].copy_(s["weights0"])
        if not own:
            return _plain_weights(s)
        packed = dict(k_scales=s["k_scales"], k_descale=s["k_descale"]) if "k_codes" in s else {}
        return ea.attention_key_weights(s["q"], s["k_codes"] if packed else s["k_pages"],
                                        s["table"], s["lens"], s["lse"], s["weights"],
                                        scale=s["scale"], causal=s["causal"], add=s["add"],
                                        **packed)
    s["meta"].copy_(s["start"])
    s["weights"].copy_(s["weights0"])
    if own:
        slots = ea.pages_evict(s["pools"], s["table"], s["lens"], s["refs"], s["weights"],
                               s["seqs"], s["new_lens"], recent=s["recent"], page_size=s["page"])
    else:
        slots = _plain_evict(s)
    return (slots, s["table"], s["lens"], s["refs"], s["weights"]) + tuple(
        x.view(torch.uint8) if x.element_size() == 1 else x for x in s["pools"])


def work(case):
    op, page, H_kv, d = case["op"], case["page"], case["H_kv"], case["d"]
    mean = (case["lo"] + case["hi"]) / 2
    packed = 9 * d / 16   # bytes of a key in 4 bits
    if op == "store":
        n = min(mean, case["n"])
        return dict(bytes=case["B"] * n * H_kv * 2 * (4 * d + packed), flops=0)
    if op == "evict":
        moves = case["S"] * min(case["keep"], mean) * (case["keep"] < case["hi"])
        row = 4 * d if case["bits"] == 16 else 2 * packed
        W = max(1, -(-case["hi"] // page)) * page
        return dict(bytes=H_kv * (moves * 2 * row + case["S"] * (mean * 4 + 4 * W)), flops=0)
    rows, B = case["B"] * case["H"] * case["n_q"], case["B"]
    table = B * (mean / page + 1) * 4
    if op == "decode":
        return dict(bytes=B * mean * H_kv * 2 * packed + rows * (4 * d + 4) + table,
                    flops=4.0 * d * rows * mean)
    key = packed if case["bits"] == 4 else 2 * d
    return dict(bytes=B * mean * H_kv * (key + (8 if case["add"] else 4)) + rows * (2 * d + 4)
                + table, flops=2.0 * d * rows * mean)


# ------------------------------------------------------- 64-bit definitions --

def _exact_values(codes, scales, descale):
    """What packed codes stand for, in 64 bits, from the formats' definitions."""
    def e2m1(c):
        sign, e, m = 1.0 - 2.0 * (c >> 3), (c >> 1) & 3, (c & 1).double()
        return sign * torch.where(e == 0, 0.5 * m, torch.exp2(e.double() - 1) * (1 + 0.5 * m))
    c, u = codes.long(), scales.view(torch.uint8).long()
    e, m = u >> 3 & 15, (u & 7).double()
    unit = torch.where(e == 0, m * 2.0 ** -9, torch.exp2(e.double() - 7) * (1 + m / 8))
    x = torch.stack([e2m1(c & 15), e2m1(c >> 4)], -1).flatten(-2)
    return x * unit.repeat_interleave(BLOCK, -1) * descale


def _exact_keys(s, b, n, name):
    at = s["table"][b, :-(-n // s["page"])].long()
    if name + "_codes" in s:
        x = _exact_values(s[name + "_codes"][at], s[name + "_scales"][at], s[name + "_descale"])
    else:
        x = s[name + "_pages"][at].double()
    return x.permute(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3])[:, :n]


def _exact_attention(s):
    B, H, n_q, d = s["q"].shape
    o = torch.zeros(B, H, n_q, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, n_q), float("-inf"), dtype=torch.float64, device="cuda")
    w = s["weights"].double() if "weights" in s else None
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        keys = _exact_keys(s, b, n, "k")
        G = keys.shape[0]
        values = _exact_keys(s, b, n, "v") if w is None else None
        if w is not None and not s["add"]:
            w[b, :, :n] = 0
        for t in range(n_q):
            end = min(n, n - n_q + t + 1) if s["causal"] else n
            if end <= 0:
                continue
            x = torch.einsum("ghd,gnd->ghn", s["q"][b, :, t].double().reshape(G, H // G, -1),
                             keys[:, :end]) * s["scale"]
            if w is not None:
                z = s["lse"][b, :, t].double().reshape(G, -1, 1)
                w[b, :, :end] += torch.exp(x - z).sum(1)
                continue
            z = torch.logsumexp(x, -1)
            o[b, :, t] = torch.einsum("ghn,gnd->ghd", torch.exp(x - z[..., None]),
                                      values[:, :end]).reshape(H, d)
            lse[b, :, t] = z.reshape(H)
    return (o, lse) if w is None else w


def _round_to(x, bits, low, top):
    """Nearest value with `bits` significant bits and steps of at least 2^low, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x.clamp(min=1e-300))).clamp(min=low + bits - 1)
                      - (bits - 1))
    return (torch.round(x / step) * step).clamp(max=top)


def _exact_store(x, counts, descale):
    B, H, n, d = x.shape
    y = x.double().reshape(B, H, n, d // BLOCK, BLOCK) / descale
    unit = _round_to(y.abs().amax(-1, keepdim=True) / 6, 4, -9, 448.0)
    code = _round_to(y.abs() / torch.where(unit == 0, 1.0, unit), 2, -1, 6.0)
    y = (torch.sign(y) * code * unit * descale).reshape(B, H, n, d)
    live = torch.arange(n, device="cuda") < counts[:, None]
    return torch.where(live[:, None, :, None], y, 0.0)


def _exact_evict(s):
    table, lens, refs = (s[x].tolist() for x in ("table", "lens", "refs"))
    page, w = s["page"], s["weights0"].double().cpu().numpy().copy()
    pools = [x.view(torch.uint8).clone() if x.element_size() == 1 else x.double()
             for x in s["pools"]]
    S, H, W = w.shape
    slots = np.full((S, H, W), -1, dtype=np.int32)
    for i in range(S):
        old, new = lens[i], min(lens[i], int(s["new_lens"][i]))
        r = min(s["recent"], new)
        pages = torch.tensor(table[i], device="cuda")
        for h in range(H):
            order = np.lexsort((np.arange(old - r), -w[i, h, :old - r]))[:new - r]
            src = np.concatenate([np.sort(order), np.arange(old - r, old)])
            slots[i, h, :new] = src
            w[i, h, :new], w[i, h, new:old] = w[i, h, src], 0
            a, b = torch.from_numpy(src).cuda(), torch.arange(new, device="cuda")
            for x in pools:
                x[pages[b // page].long(), h, b % page] = x[pages[a // page].long(), h, a % page]
        for j in range(-(-new // page), -(-old // page)):
            refs[table[i][j]] -= 1
            table[i][j] = -1
        lens[i] = new
    ints = tuple(torch.tensor(x, dtype=torch.int32) for x in (table, lens, refs))
    return (torch.from_numpy(slots),) + ints + (torch.from_numpy(w),) + tuple(pools)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "store":
        return tuple(_exact_store(s[x], s["counts"], s[x + "_descale"]) for x in ("k", "v"))
    if case["op"] == "evict":
        return _exact_evict(s)
    return _exact_attention(s)

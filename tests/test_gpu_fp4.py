"""Caches in 4 bits (pages_store_fp4, pages_load_fp4, attention_decode_fp4) against
their definitions in 64 bits.

Tolerances.  Codes and scales are whole numbers, equal.  A loaded value is a
product of exact numbers rounded in fp32 twice (2^-24 each) and to bf16: its 8
significant bits put neighbours 2^-7 of the power of two below apart, half a step is
2^-8: 2^-8 + 2^-22 relative.  L: the bar of every L here (L_MAX_ABS).
O: P is rounded to fp16, a relative 2^-11 of each term, below 2^-14 an absolute
2^-25 of the largest P's scale; scores and L off by L_MAX_ABS each; O rounded to
bf16: |O - O*| <= (2^-11 + 2 L_MAX_ABS) sum_j P_j |V_j| + 2^-25 sum_j |V_j| + 2^-8 |O|,
with a hundredth on top for the products of these.
"""

import ctypes

import numpy as np
import pytest
import torch

from oracle import fp4, paged as oracle
from tests.helpers import L_MAX_ABS, max_abs, np64
from tests.test_gpu_paged import WIDE, _table, ea  # noqa: F401

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def _i(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def _layout(x, layout):
    """The tensor on the GPU, its pages and heads laid out as asked."""
    x = x.cuda()
    if layout == "nhd":      # heads' blocks of a page apart by more than a block
        big = torch.full((x.shape[0], 2 * x.shape[1] + 1) + x.shape[2:], 0x7f, dtype=torch.uint8,
                         device="cuda")
        x8 = x.view(torch.uint8)
        view = big[:, 1::2]
        view.copy_(x8)
        return view.view(x.dtype)
    if layout == "apart":    # pages apart, heads' blocks next to one another
        big = torch.full((x.shape[0], x.shape[1] + 3) + x.shape[2:], 0x7f, dtype=torch.uint8,
                         device="cuda")
        view = big[:, :x.shape[1]]
        view.copy_(x.view(torch.uint8))
        return view.view(x.dtype)
    return x


def _cache(rng, table, lens, P, H_kv, page, d, poison=True):
    """Random codes and scales (uint8, on the CPU); rows that no sequence holds have
    NaN scales."""
    codes = rng.integers(0, 256, (P, H_kv, page, d // 2), dtype=np.uint8)
    scales = rng.integers(0x20, 0x58, (P, H_kv, page, d // 16), dtype=np.uint8)
    scales[rng.random(scales.shape) < 0.02] = 0
    if poison:
        keep = np.zeros((P, page), dtype=bool)
        for b, n in enumerate(lens):
            for j in range(-(-n // page)):
                keep[table[b, j], :min(page, n - j * page)] = True
        scales[np.broadcast_to(~keep[:, None, :, None], scales.shape)] = 0x7f
    return codes, scales


def _on_gpu(codes, scales, layout="hnd"):
    return _layout(torch.from_numpy(codes), layout), \
        _layout(torch.from_numpy(scales).view(E4M3), layout)


def _hold(o, lse, want, total, what=""):
    O, L, A = want
    got = np64(o.cpu())
    bound = 1.01 * ((2.0 ** -11 + 2 * L_MAX_ABS) * A + 2.0 ** -25 * total + 2.0 ** -8 * np.abs(O)) + 1e-30
    assert np.isfinite(got).all(), what
    worst = np.max(np.abs(got - O) / bound) if O.size else 0.0
    assert worst <= 1.0, (what, worst)
    assert max_abs(lse.cpu().numpy(), L) <= L_MAX_ABS, what


def _decode(ea, lens, H, H_kv, n_q, d, page, causal=True, seed=0, layout="hnd", scale=None, room=0,
            q_scale=1.0, k_descale=2.0 ** -7, v_descale=0.011):
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    table, P = _table(rng, lens, page, room=room)
    k, v = (_cache(rng, table, lens, P, H_kv, page, d) for _ in range(2))
    q = (torch.randn(len(lens), H, n_q, d, generator=g) * q_scale).to(torch.bfloat16)
    # scores of a few units whatever q's and the keys' magnitudes
    scale = 0.3 * d ** -0.5 / q_scale / (k_descale * 2 ** 7) if scale is None else scale
    o, lse = ea.attention_decode_fp4(
        q.cuda(), *_on_gpu(*k, layout), *_on_gpu(*v, layout), torch.from_numpy(table).cuda(),
        _i(lens), scale=scale, causal=causal, k_descale=k_descale, v_descale=v_descale)
    torch.cuda.synchronize()
    ea.check()
    kd, vd = fp4.decode(*k, k_descale), fp4.decode(*v, v_descale)
    want = oracle.paged_decode(np64(q), kd, vd, table, lens, scale, causal)
    total = np.zeros((len(lens), H, 1, 1))
    for b, n in enumerate(lens):
        x = np.abs(oracle.gather(vd, table[b], n)).sum(1).max(-1) if n else np.zeros(H_kv)
        total[b, :, 0, 0] = np.repeat(x, H // H_kv)
    _hold(o, lse, want, total)
    return o, lse


# ------------------------------------------------------------------ decode --

# rows per key/value head: 1, 8, 9, 16, 17, 32, 33, 64, 65, 130: every width, one
# more, and blocks
@pytest.mark.parametrize("H,H_kv,n_q", [(2, 2, 1), (16, 2, 1), (18, 2, 1), (8, 1, 2), (17, 1, 1),
                                         (8, 1, 4), (33, 1, 1), (32, 1, 2), (65, 1, 1), (26, 1, 5)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("room", [0, WIDE])
def test_rows_and_widths(ea, H, H_kv, n_q, d, room):  # noqa: F811
    _decode(ea, [300, 1, 33, 0, 129], H, H_kv, n_q, d, 16, seed=H + d, room=room)


@pytest.mark.parametrize("page", [16, 32, 64, 512])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("room", [0, WIDE])
def test_page_sizes(ea, page, causal, room):  # noqa: F811
    _decode(ea, [0, 1, 15, 16, 17, 31, 32, 33, 512, 513, 700], 4, 2, 3, 64, page, causal, seed=page,
            room=room)


# many segments: a warp each (short), a CTA each (longer), the balanced split
@pytest.mark.parametrize("most,H_kv,n_q", [(200, 8, 1), (200, 4, 5), (900, 8, 1), (200, 8, 9)])
def test_many_sequences(ea, most, H_kv, n_q):  # noqa: F811
    rng = np.random.default_rng(most)
    B = 90 if most > 500 else 170
    lens = [int(x) for x in rng.integers(0, most, B)]
    lens[1], lens[-1] = 0, most
    _decode(ea, lens, 2 * H_kv, H_kv, n_q, 64, 16, seed=most)


@pytest.mark.parametrize("lens,H,H_kv,n_q,d", [([20000], 2, 1, 1, 64), ([6001, 5999], 64, 1, 1, 128),
                                               ([9000, 40], 4, 1, 3, 64), ([3000, 10, 700], 32, 2, 1, 128)])
@pytest.mark.parametrize("room", [0, WIDE])
def test_long_sequences(ea, lens, H, H_kv, n_q, d, room):  # noqa: F811
    _decode(ea, lens, H, H_kv, n_q, d, 64, seed=9, room=room)


@pytest.mark.parametrize("layout", ["nhd", "apart"])
@pytest.mark.parametrize("d", [64, 128])
def test_layouts(ea, layout, d):  # noqa: F811
    _decode(ea, [200, 77], 8, 4, 1, d, 32, layout=layout, seed=3)


def test_query_strides(ea):  # noqa: F811
    q = torch.randn(2, 6, 8, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    q = q.transpose(1, 2)[:, :, :3]     # [B, H = 8, n_q = 3, d]
    rng = np.random.default_rng(1)
    table, P = _table(rng, [70, 40], 16)
    cache = [*_on_gpu(*_cache(rng, table, [70, 40], P, 2, 16, 128)),
             *_on_gpu(*_cache(rng, table, [70, 40], P, 2, 16, 128))]
    args = (torch.from_numpy(table).cuda(), _i([70, 40]))
    out = torch.empty_strided(q.shape, q.stride(), dtype=q.dtype, device="cuda")
    o, lse = ea.attention_decode_fp4(q, *cache, *args, scale=1e-3, out=out)
    o2, lse2 = ea.attention_decode_fp4(q.contiguous(), *cache, *args, scale=1e-3)
    assert o is out and torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("q_scale", [2.0 ** -60, 2.0 ** 70, 3e4])
@pytest.mark.parametrize("rows", [1, 9, 20])
def test_magnitudes_of_q(ea, q_scale, rows):  # noqa: F811
    # far outside fp16: every row is scaled by its own power of two
    _decode(ea, [150, 33], rows, 1, 1, 64, 16, q_scale=q_scale, seed=rows)


@pytest.mark.parametrize("k_descale,v_descale", [(2.0 ** -90, 2.0 ** 60), (3e20, 2.0 ** -99), (0.37, 1.0)])
def test_factors(ea, k_descale, v_descale):  # noqa: F811
    _decode(ea, [150, 33], 4, 2, 1, 128, 16, k_descale=k_descale, v_descale=v_descale, seed=2)


def test_large_scores(ea):  # noqa: F811
    # scores to +-100: the lazily followed maximum has to hold
    _decode(ea, [500, 64], 4, 2, 2, 64, 32, scale=4.0 * 0.25, seed=11)


def test_a_row_of_zeros_and_rows_that_are_no_numbers(ea):  # noqa: F811
    rng = np.random.default_rng(5)
    lens = [70, 40]
    table, P = _table(rng, lens, 16)
    k, v = (_cache(rng, table, lens, P, 1, 16, 64) for _ in range(2))
    q = torch.randn(2, 4, 1, 64, generator=torch.Generator().manual_seed(1))
    q[0, 1] = 0
    q[0, 2, 0, 5] = float("nan")
    q[1, 3, 0, 9] = float("inf")
    q = q.to(torch.bfloat16)
    o, lse = ea.attention_decode_fp4(q.cuda(), *_on_gpu(*k), *_on_gpu(*v),
                                     torch.from_numpy(table).cuda(), _i(lens), scale=0.01)
    for b, h in ((0, 2), (1, 3)):
        assert torch.isnan(o[b, h]).all() and torch.isnan(lse[b, h]).all()
    vd = fp4.decode(*v, 1.0)
    mean = oracle.gather(vd, table[0], 70).mean(1)[0]
    bound = (2.0 ** -8 + 2e-3) * np.abs(oracle.gather(vd, table[0], 70)).mean(1)[0]
    assert np.all(np.abs(np64(o)[0, 1, 0] - mean) <= bound)
    assert abs(lse[0, 1, 0].item() - np.log(70)) <= L_MAX_ABS
    keep = torch.ones(2, 4, dtype=torch.bool)
    keep[0, 2] = keep[1, 3] = False
    assert torch.isfinite(o.cpu()[keep].float()).all() and torch.isfinite(lse.cpu()[keep]).all()


@pytest.mark.parametrize("room", [0, WIDE])
def test_a_page_outside_the_cache_reads_as_zeros(ea, room):  # noqa: F811
    from exact_attention_12_gb300 import AttnError
    rng = np.random.default_rng(6)
    lens = [100, 40]
    table, P = _table(rng, lens, 16, room=room)
    k, v = (_cache(rng, table, lens, P, 2, 16, 64) for _ in range(2))
    bad = table.copy()
    bad[0, 2], bad[1, 1] = P, -5
    q = torch.randn(2, 4, 1, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    o, lse = ea.attention_decode_fp4(q.cuda(), *_on_gpu(*k), *_on_gpu(*v),
                                     torch.from_numpy(bad).cuda(), _i(lens), scale=0.01)
    with pytest.raises(AttnError) as e:
        ea.check()
    assert e.value.status == 6
    ea.check()
    zero = [np.concatenate([x, np.zeros_like(x[:1])]) for x in (*k, *v)]
    t = np.where((bad < 0) | (bad >= P), P, bad)
    want = oracle.paged_decode(np64(q), fp4.decode(zero[0], zero[1], 1.0),
                               fp4.decode(zero[2], zero[3], 1.0), t, lens, 0.01)
    _hold(o, lse, want, 1e4)


# ----------------------------------- decode: many rows, long tables, d = 128 --

@pytest.mark.parametrize("page", [16, 32, 64, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_page_sizes_of_many_rows(ea, page, causal):  # noqa: F811
    # (causal: rows that attend nothing where n_q exceeds the sequence)
    _decode(ea, [0, 1, 15, 16, 33, 127, 128, 129, 700, 2000], 24, 2, 4, 128, page, causal, seed=page,
            room=WIDE)


# 33 to 64 rows: both halves full, one of them part full; 72 in two blocks of 36
@pytest.mark.parametrize("H,n_q", [(33, 1), (12, 4), (49, 1), (1, 64), (72, 1), (3, 24)])
@pytest.mark.parametrize("layout", ["hnd", "nhd", "apart"])
def test_many_rows_of_long_sequences(ea, H, n_q, layout):  # noqa: F811
    _decode(ea, [30000, 5], H, 1, n_q, 128, 64, seed=H, layout=layout)


def test_many_rows_of_many_sequences(ea):  # noqa: F811
    # more segments than CTAs, pieces that end and begin inside a CTA, empty ones
    rng = np.random.default_rng(12)
    lens = [int(x) for x in rng.integers(0, 700, 170)]
    lens[3] = lens[4] = lens[-1] = 0
    lens[5] = 4100
    _decode(ea, lens, 40, 1, 1, 128, 16, seed=12)


@pytest.mark.parametrize("q_scale", [2.0 ** -60, 2.0 ** 70])
def test_magnitudes_of_many_rows(ea, q_scale):  # noqa: F811
    _decode(ea, [150, 33], 40, 1, 1, 128, 16, q_scale=q_scale, seed=4, room=WIDE)
    _decode(ea, [150, 33], 40, 1, 1, 128, 16, k_descale=3e20, v_descale=2.0 ** -99, seed=4, room=WIDE)


def test_large_scores_of_many_rows(ea):  # noqa: F811
    # scores to +-100, over many tiles: maxima rise late, and O is scaled in place
    _decode(ea, [2500, 64], 48, 1, 1, 128, 32, scale=3.0 * 0.25, seed=11, room=WIDE)


def test_many_rows_some_of_them_no_numbers(ea):  # noqa: F811
    rng = np.random.default_rng(5)
    lens = [700, 40]
    table, P = _table(rng, lens, 16, room=WIDE)
    k, v = (_cache(rng, table, lens, P, 1, 16, 128) for _ in range(2))
    q = torch.randn(2, 40, 1, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    args = (*_on_gpu(*k), *_on_gpu(*v), torch.from_numpy(table).cuda(), _i(lens))
    want, want_l = ea.attention_decode_fp4(q.cuda(), *args, scale=0.01)
    odd = q.clone()
    odd[0, 2, 0, 5], odd[0, 33, 0, 7] = float("nan"), float("nan")
    odd[1, 3, 0, 9], odd[1, 39, 0, 100] = float("inf"), -float("inf")
    o, lse = ea.attention_decode_fp4(odd.cuda(), *args, scale=0.01)
    ea.check()
    for b, h in ((0, 2), (0, 33), (1, 3), (1, 39)):
        assert torch.isnan(o[b, h]).all() and torch.isnan(lse[b, h]).all()
    keep = torch.ones(2, 40, dtype=torch.bool)
    keep[0, 2] = keep[0, 33] = keep[1, 3] = keep[1, 39] = False
    assert torch.equal(o.cpu()[keep], want.cpu()[keep])
    assert torch.equal(lse.cpu()[keep], want_l.cpu()[keep])


@pytest.mark.parametrize("page", [16, 64])
def test_a_page_outside_the_cache_under_many_rows(ea, page):  # noqa: F811
    from exact_attention_12_gb300 import AttnError
    rng = np.random.default_rng(6)
    lens = [700, 140]
    table, P = _table(rng, lens, page, room=WIDE)
    k, v = (_cache(rng, table, lens, P, 1, page, 128) for _ in range(2))
    bad = table.copy()
    bad[0, 2], bad[0, 7], bad[1, 1] = P, -5, 2 ** 31 - 1
    q = torch.randn(2, 40, 1, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    o, lse = ea.attention_decode_fp4(q.cuda(), *_on_gpu(*k), *_on_gpu(*v),
                                     torch.from_numpy(bad).cuda(), _i(lens), scale=0.01)
    with pytest.raises(AttnError) as e:
        ea.check()
    assert e.value.status == 6
    zero = [np.concatenate([x, np.zeros_like(x[:1])]) for x in (*k, *v)]
    t = np.where((bad < 0) | (bad >= P), P, bad)
    want = oracle.paged_decode(np64(q), fp4.decode(zero[0], zero[1], 1.0),
                               fp4.decode(zero[2], zero[3], 1.0), t, lens, 0.01)
    _hold(o, lse, want, 1e5)


def test_a_stalled_step_of_many_rows_ends_and_reports(ea):  # noqa: F811
    from exact_attention_12_gb300 import _abi
    lib = _abi.lib()
    z = dict(device="cuda")
    P = 640
    codes = torch.full((P, 1, 128, 64), 0x22, dtype=torch.uint8, **z)       # ones
    scales = torch.full((P, 1, 128, 8), 0x38, dtype=torch.uint8, **z).view(E4M3)
    t, n = torch.arange(P, dtype=torch.int32, **z).view(1, P), _i([P * 128])
    q = torch.zeros(1, 40, 1, 128, dtype=torch.bfloat16, **z)
    ws = torch.zeros(1 << 24, dtype=torch.uint8, **z)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert lib.attn_debug_stall(_abi.ATTN_STALL_FP4_VALUES, 20_000_000) == _abi.ATTN_OK
    ea.attention_decode_fp4(q, codes, scales, codes, scales, t, n, ws=ws)
    assert lib.attn_check(ws.data_ptr(), stream) == _abi.ATTN_ERR_TIMEOUT
    assert int(lib.attn_last_error().decode().rsplit("wait site", 1)[1]) in range(90, 98)
    for _ in range(2):
        o, lse = ea.attention_decode_fp4(q, codes, scales, codes, scales, t, n, ws=ws)
        assert lib.attn_check(ws.data_ptr(), stream) == _abi.ATTN_OK
        assert torch.all(o == 1) and torch.all((lse - float(np.log(P * 128))).abs() <= L_MAX_ABS)


def test_nothing_to_do(ea):  # noqa: F811
    z = dict(device="cuda")
    codes, scales = torch.zeros(3, 2, 16, 32, dtype=torch.uint8, **z), torch.zeros(3, 2, 16, 4, **z).to(E4M3)
    t, n = torch.zeros(0, 4, dtype=torch.int32, **z), torch.zeros(0, dtype=torch.int32, **z)
    q = torch.zeros(0, 4, 1, 64, dtype=torch.bfloat16, **z)
    o, lse = ea.attention_decode_fp4(q, codes, scales, codes, scales, t, n)
    assert o.shape == (0, 4, 1, 64) and lse.shape == (0, 4, 1)
    # no pages, no heads, empty sequences
    t, n = _i([[7, 7]]), _i([0])
    q = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16, **z)
    o, lse = ea.attention_decode_fp4(q, codes[:0], scales[:0], codes[:0], scales[:0], t, n)
    assert torch.all(o == 0) and torch.all(torch.isneginf(lse))
    o, lse = ea.attention_decode_fp4(q[:, :0], codes[:, :0], scales[:, :0], codes[:, :0],
                                     scales[:, :0], t, n)
    assert o.shape == (1, 0, 1, 64)
    ea.check()


# ---------------------------------------------------------- store and load --

def _values(rng, shape):
    """bf16 values of all kinds: ordinary ones, wide blocks, exact ties, zeros,
    infinities, NaN, tiny and huge ones."""
    x = rng.normal(size=shape).astype(np.float32)
    x = x * np.exp2(rng.integers(-6, 7, shape[:-1] + (shape[-1] // 16, 1))).repeat(16, -1).reshape(shape)
    blocks = x.reshape(-1, 16)
    kind = rng.integers(0, 16, len(blocks))
    ties = np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -5, -2.5, 0, -0.0, 4])
    blocks[kind == 0] = ties * np.exp2(rng.integers(-3, 4, ((kind == 0).sum(), 1)))
    blocks[kind == 1] = 0
    blocks[kind == 2, 3] = np.inf
    blocks[kind == 3, 7] = -np.inf
    blocks[kind == 4, 0] = np.nan
    blocks[kind == 5] *= 1e-6
    blocks[kind == 6] *= 1e30
    blocks[kind == 7] = 1e-38
    return torch.from_numpy(blocks.reshape(shape)).to(torch.bfloat16)


def _store(ea, lens, counts, n, H, d, page, descales, layout="hnd", seed=0, kv="plain"):
    rng = np.random.default_rng(seed)
    table, P = _table(rng, lens, page)
    B = len(lens)
    k, v = (_values(rng, (B, H, n, d)) for _ in range(2))
    pad = torch.full((P, H, page, d // 2), 0xa5, dtype=torch.uint8)
    spad = torch.full((P, H, page, d // 16), 0x11, dtype=torch.uint8)
    cache = [_layout(pad, layout), _layout(spad.view(E4M3), layout), _layout(pad, layout),
             _layout(spad.view(E4M3), layout)]
    dk, dv = k.cuda(), v.cuda()
    if kv == "tokens first":
        dk, dv = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (dk, dv))
    t, ln = torch.from_numpy(table).cuda(), _i(lens)
    kw = dict(k_descale=descales[0], v_descale=descales[1],
              counts=None if counts is None else _i(counts))
    ea.pages_store_fp4(dk, dv, *cache, t, ln, **kw)
    back = ea.pages_load_fp4(*cache, t, ln, n, **kw)
    torch.cuda.synchronize()
    ea.check()
    for x, (c, s), y, D in ((k, cache[:2], back[0], descales[0]), (v, cache[2:], back[1], descales[1])):
        want_c, want_s = pad.numpy().copy(), spad.numpy().copy()
        codes, scales = fp4.encode(np64(x), D)
        want = np.zeros(x.shape)
        for b in range(B):
            m = n if counts is None else min(max(counts[b], 0), n)
            for j in range(m):
                pos = lens[b] - m + j
                if pos < 0:
                    continue
                at = table[b, pos // page], slice(None), pos % page
                want_c[at], want_s[at] = codes[b, :, j], scales[b, :, j]
                want[b, :, j] = fp4.decode(codes[b, :, j], scales[b, :, j], D)
        assert np.array_equal(s.view(torch.uint8).cpu().numpy(), want_s)
        got_c = c.cpu().numpy()
        differ = (got_c != want_c).sum()
        assert differ == 0, differ
        got = np64(y)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        want = np.where(np.isnan(want), 0, want)
        got = np.where(np.isnan(got), 0, got)
        big = np.abs(want) > 3.38e38    # beyond bf16
        far = ~big & (np.abs(got - want) > np.abs(want) * (2.0 ** -8 + 2.0 ** -22) + 2.0 ** -134)
        assert far.sum() == 0, far.sum()


@pytest.mark.parametrize("H,d,page", [(1, 64, 16), (2, 128, 32), (3, 64, 64), (8, 128, 16), (5, 128, 128)])
@pytest.mark.parametrize("n", [1, 2, 13, 70])
def test_stored_codes_are_the_definitions(ea, H, d, page, n):  # noqa: F811
    rng = np.random.default_rng(n)
    lens = [int(x) for x in rng.integers(0, 150, 6)] + [n, 0]
    counts = [min(x, int(rng.integers(0, n + 1))) for x in lens]
    _store(ea, lens, counts, n, H, d, page, (24.0 / 2688, 1.0), seed=n)


# factors whose borders fall next to (and on) bf16 values, and extreme ones
@pytest.mark.parametrize("descales", [(1.0, 2.0 ** -9), (24.0 / 2688, 17.0 / 2688), (0.3, 7.0 / 3),
                                      (2.0 ** -100, 2.0 ** 100), (1e-7, 1e7)])
def test_factors_of_a_store(ea, descales):  # noqa: F811
    _store(ea, [300, 250], None, 200, 4, 128, 32, descales, seed=3)


@pytest.mark.parametrize("layout", ["nhd", "apart"])
@pytest.mark.parametrize("kv", ["plain", "tokens first"])
def test_layouts_of_a_store(ea, layout, kv):  # noqa: F811
    _store(ea, [50, 7], [33, 5], 40, 3, 64, 16, (0.01, 0.02), layout, 5, kv)


def test_tokens_before_the_sequence_are_left_out(ea):  # noqa: F811
    # (counts above the length, negative, above n)
    _store(ea, [5, 20, 9], [9, -3, 100], 9, 2, 64, 16, (0.01, 0.02), seed=6)


def test_many_sequences_and_heads_of_a_store(ea):  # noqa: F811
    _store(ea, [3] * 200, None, 1, 9, 64, 16, (0.01, 0.02), seed=7)


def test_a_bad_page_of_a_store_is_left_out(ea):  # noqa: F811
    from exact_attention_12_gb300 import AttnError
    g = torch.Generator().manual_seed(1)
    k = torch.randn(1, 2, 40, 64, generator=g).to(torch.bfloat16).cuda()
    codes = torch.full((3, 2, 16, 32), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.ones(3, 2, 16, 4, device="cuda").to(E4M3)
    t, n = _i([[2, 3, 0]]), _i([40])
    ea.pages_store_fp4(k, k, codes, scales, codes, scales, t, n, k_descale=0.01, v_descale=0.01)
    with pytest.raises(AttnError) as e:
        ea.check()
    assert e.value.status == 6
    assert torch.all(codes[1] == 0x55) and not torch.all(codes[2] == 0x55)
    x, _ = ea.pages_load_fp4(codes, scales, codes, scales, t, n, 40, k_descale=0.01, v_descale=0.01)
    assert torch.all(x[:, :, 16:32] == 0) and not torch.all(x[:, :, :16] == 0)
    with pytest.raises(AttnError):
        ea.check()


# --------------------------------------------------------------- a whole run --

def test_streams_and_graphs(ea):  # noqa: F811
    # two steps at once on two streams, each with its own workspace; then one captured
    # with the store before it, and replayed with other tokens
    rng = np.random.default_rng(8)
    lens = [700, 90, 333]
    table, P = _table(rng, lens, 16, room=WIDE)
    k, v = (_cache(rng, table, lens, P, 2, 16, 64) for _ in range(2))
    cache = [*_on_gpu(*k), *_on_gpu(*v)]
    t, ln = torch.from_numpy(table).cuda(), _i(lens)
    q = [torch.randn(3, 8, 1, 64, device="cuda").to(torch.bfloat16) for _ in range(2)]
    kw = dict(scale=0.02, k_descale=0.01, v_descale=0.01)
    want = [ea.attention_decode_fp4(x, *cache, t, ln, **kw) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in q]
    spaces = [torch.zeros(1 << 23, dtype=torch.uint8, device="cuda") for _ in q]
    torch.cuda.synchronize()
    got = []
    for s, w, x in zip(streams, spaces, q):
        with torch.cuda.stream(s):
            got.append([ea.attention_decode_fp4(x, *cache, t, ln, ws=w, **kw) for _ in range(5)])
    torch.cuda.synchronize()
    for runs, (o, lse) in zip(got, want):
        for a, b in runs:
            assert torch.equal(a, o) and torch.equal(b, lse)
    new = torch.randn(3, 2, 1, 64, device="cuda").to(torch.bfloat16)

    def step():
        ea.pages_store_fp4(new, new, *cache, t, ln, k_descale=0.01, v_descale=0.01, ws=spaces[0])
        return ea.attention_decode_fp4(q[0], *cache, t, ln, ws=spaces[0], **kw)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step()
    for i in range(2):
        new.copy_(torch.randn(3, 2, 1, 64, device="cuda"))
        graph.replay()
        o1, lse1 = o.clone(), lse.clone()
        o2, lse2 = step()
        assert torch.equal(o1, o2) and torch.equal(lse1, lse2)
    ea.check()
    ea.check(ws=spaces[0])

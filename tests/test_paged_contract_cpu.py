"""What the paged-cache calls promise beyond their results, as far as it shows
without a GPU: the sources, the argument checks, the binding."""

import ctypes
import glob
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_attention_12_gb300", "csrc")


def _code(path):
    """A source file without its comments."""
    text = open(path, encoding="utf-8").read()
    return re.sub(r"/\*.*?\*/|//[^\n]*", "", text, flags=re.S)


def test_no_copy_or_commit_reaches_another_cta():
    # the library is loaded by every replica of a multi-GPU job, and a cache may be
    # any device pointer: a TMA copy goes to the CTA that issues it only
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        assert "multicast" not in _code(path), path


def test_every_note_is_checked_before_it_is_followed():
    # a wait that has run out leaves notes unwritten: whatever the workspace holds in
    # their place must not be used as an index
    text = _code(os.path.join(CSRC, "attn_paged.cu"))
    kernels = [k for k in re.split(r"__global__", text) if "const MergeNote note{raw" in k]
    assert len(kernels) == 2
    for k in kernels:
        body = k[k.index("const MergeNote note{raw"):]
        check = re.search(r"if \([^\n]*!note_holds\(a, note\)\) return;", body)
        assert check and not re.search(r"note\.(b|h|slot)", body[:check.start()])


def test_the_paged_kernels_can_be_stalled():
    from exact_attention_12_gb300 import _abi
    lib = _abi.lib()
    for which in (_abi.ATTN_STALL_PAGED_TILE, _abi.ATTN_STALL_PREFIX_SOFTMAX,
                  _abi.ATTN_STALL_LATENT_SOFTMAX, _abi.ATTN_STALL_NONE):
        assert lib.attn_debug_stall(which, 1) == _abi.ATTN_OK
    for which in (-1, 6):
        assert lib.attn_debug_stall(which, 1) == _abi.ATTN_ERR_INVALID_ARG


def test_thread_indices_are_compared_as_what_they_are():
    # threadIdx.x is unsigned: against a signed count that may be negative the comparison
    # holds for every thread.  Constants (kItems, 32) are never negative.
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        for other in re.findall(r"threadIdx\.x\s*(?:<|>=|<=|>)\s*([\w:]+)", _code(path)):
            assert re.fullmatch(r"(C::)?k[A-Z]\w*|\d+", other), (path, other)


@pytest.mark.parametrize("H_kv", [0, 2])
@pytest.mark.parametrize("n_q", [1, 3])
def test_no_heads_reach_the_library_with_strides_it_takes(monkeypatch, H_kv, n_q):
    from exact_attention_12_gb300 import _abi, paged
    seen = []

    def call(fn, size_fn, size_args, args, device, ws, what):
        p, q, g = size_args
        seen.append(size_fn(p, q, g))

    monkeypatch.setattr(paged, "_call", call)
    bf = torch.bfloat16
    t, n = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    k = torch.zeros(5, H_kv, 16, 64, dtype=bf)
    paged.attention_decode_paged(torch.zeros(3, 0, n_q, 64, dtype=bf), k, k, t, n)
    paged.attention_decode_latent(torch.zeros(3, 0, n_q, 320, dtype=bf),
                                  torch.zeros(5, 16, 320, dtype=bf), t, n, scale=0.1, d_v=256)
    assert min(seen) >= 256, _abi.lib().attn_last_error()


def test_check_reads_every_workspace_of_the_device(monkeypatch):
    from exact_attention_12_gb300 import _abi, api

    class Lib:
        def attn_check(self, ptr, stream):
            seen.append(ptr)
            return bad.pop(ptr, _abi.ATTN_OK)   # read and cleared

        def attn_last_error(self):
            return b""

    monkeypatch.setattr(api, "lib", Lib)
    monkeypatch.setattr(_abi, "lib", Lib)
    monkeypatch.setattr(api, "_stream", lambda dev: None)
    monkeypatch.setattr(api, "_workspaces", {})
    monkeypatch.setattr(api, "_retired", {})
    spaces = [api.workspace("cpu", 256 << i) for i in range(3)]
    for w in spaces:
        seen, bad = [], {w.data_ptr(): _abi.ATTN_ERR_PAGE}
        with pytest.raises(_abi.AttnError) as e:
            api.check(device="cpu")
        assert e.value.status == _abi.ATTN_ERR_PAGE
        assert sorted(seen) == sorted(x.data_ptr() for x in spaces)
        api.check(device="cpu")
    seen = []
    api.check(ws=spaces[1], device="cpu")   # the caller's own: that one alone
    assert seen == [spaces[1].data_ptr()]


def _step(latent, **kw):
    """The workspace size of a decode step with these sizes; 0: refused."""
    from exact_attention_12_gb300 import _abi
    d = 256 if latent else 64
    cols = d + 64 if latent else d
    p, g = _abi.AttnParams(), _abi.AttnPages()
    p.B, p.H, p.H_kv, p.d, p.scale = 1, 4, 1, d, 1.0
    p.stride_b, p.stride_h, p.stride_n = 1 << 30, 1 << 20, cols
    p.kv_stride_b, p.kv_stride_h, p.kv_stride_n = 1 << 30, 1 << 20, cols
    p.key_lens = g.table = 0x1000
    g.max_pages, g.page_size, g.num_pages = 1, 16, 1
    n_q = kw.pop("n_q", 1)
    for k, v in kw.items():
        setattr(g if hasattr(g, k) else p, k, v)
    g.table_stride, p.N = g.max_pages, g.max_pages * g.page_size
    f = _abi.lib().attn_decode_latent_workspace_size if latent \
        else _abi.lib().attn_decode_paged_workspace_size
    size = f(ctypes.byref(p), n_q, ctypes.byref(g))
    assert size or b"2^3" in _abi.lib().attn_last_error()
    return size


@pytest.mark.parametrize("latent", [False, True])
@pytest.mark.parametrize("most,more", [
    (dict(H=32768), dict(H=32769)), (dict(H=8, n_q=4096), dict(H=8, n_q=4097)),
    (dict(H=1 << 10, B=1 << 20), dict(H=1 << 10, B=(1 << 20) + 1)),
    (dict(max_pages=1 << 15, page_size=32768), dict(max_pages=(1 << 15) + 1, page_size=32768))])
def test_the_documented_limits(latent, most, more):
    assert _step(latent, **most) > 0 and _step(latent, **more) == 0


def test_the_documented_limit_of_all_work_together():
    # B * H_kv * ceil(rows / 64) * (N / 32 + 9) < 2^31, latent B * (N / 64 + 9)
    units = (1 << 15) // 32 + 9
    b = ((1 << 31) - 1) // (2 * units)
    wide = dict(H=65, H_kv=1, max_pages=1 << 11)
    assert b * 65 <= 1 << 30
    assert _step(False, B=b, **wide) > 0 and _step(False, B=b + 1, **wide) == 0
    units = (1 << 22) // 64 + 9
    b = ((1 << 31) - 1) // units
    wide = dict(max_pages=1 << 18)
    assert _step(True, B=b, **wide) > 0 and _step(True, B=b + 1, **wide) == 0


def test_kernels_wait_before_they_let_the_next_one_start():
    # a kernel behind a shared prefix's relies on it: all work before the prefix kernel is
    # complete once that has let it start
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        for kernel in re.split(r"__global__", _code(path))[1:]:
            launch = kernel.find("grid_dep_launch();")
            if launch >= 0:
                assert 0 <= kernel.find("grid_dep_wait();") < launch, path

"""Refusals of the grouped products with 16-bit weights before any launch (no GPU needed)."""
import ctypes

import pytest

import grouped_expert_gemm_amd as geg

P = 0x10000


def L():
    return geg.lib()


def _call(name, p=P, sizes=P, q=P, out=2 * P, dtype=0, out_dtype=0, M=16, N=64, K=64, E=4, ws=P, nbytes=256, opts=None):
    o = ctypes.byref(opts) if opts else None
    if name == "geg_grouped_wgrad":
        return L().geg_grouped_wgrad(p, q, sizes, out, dtype, out_dtype, M, N, K, E, ws, nbytes, o, None)
    return getattr(L(), name)(p, sizes, q, out, dtype, M, N, K, E, 0, ws, nbytes, o, None)


NAMES = ("geg_grouped_gemm", "geg_grouped_dgrad", "geg_grouped_wgrad")


@pytest.mark.parametrize("name", NAMES)
def test_refusals(name):
    c = lambda **k: _call(name, **k)
    passes = (0, 1, 2, 3, 5, 8)
    assert c() not in passes                                     # stops at the device check
    assert c(dtype=2) == 8 and c(dtype=-1) == 8
    assert c(M=-1) == 2 and c(N=0) == 2 and c(K=0) == 2 and c(E=0) == 2 and c(E=1025) == 2 and c(M=1 << 31) == 2
    assert c(K=60) == 2 and c(K=1 << 23) == 2 and c(N=1 << 23) == 2 and c(N=1 << 62) == 2 and c(K=1 << 62) == 2
    assert c(N=63) == (2 if name != NAMES[0] else c())
    for p in ("p", "sizes", "q", "out"):
        assert c(**{p: None}) == 1, p
    for p in ("p", "q", "out"):
        assert c(**{p: P + 8}) == 3, p
    assert c(sizes=P + 2) == 3
    assert c(out=P) == 8 and c(q=2 * P) == 8
    assert c(ws=None) == 5 and c(ws=P + 16) == 5 and c(nbytes=255) == 5
    assert c(opts=geg.Opts(1, 0)) == 8 and c(opts=geg.Opts(3, 0)) == 8 and c(opts=geg.Opts(0, 0, None, -1)) == 8
    assert c(opts=geg.Opts(4, 0)) == (8 if name != NAMES[0] else c())
    assert c(opts=geg.Opts(2, 0)) not in passes
    # an expert's weights may pass one buffer window
    assert c(N=65536, K=65536) not in passes


def test_workspace_bytes():
    need = L().geg_grouped_workspace_bytes
    assert need(0, 8192, 2048, 4096, 8) == 256 and need(2, 100, 64, 64, 4) == 256
    # 3 tiles at most, the contraction in 8 pieces
    assert need(0, 100, 128, 4096, 2) == 256 + 3 * 8 * 65536 and need(1, 100, 4096, 128, 2) == 256 + 3 * 8 * 65536
    assert need(2, 2100, 128, 256, 1) == 256 + 2 * 4 * 65536
    assert need(3, 1, 1, 8, 1) == 0 and need(-1, 1, 1, 8, 1) == 0 and need(0, -1, 8, 8, 1) == 0 and need(0, 1, 8, 8, 0) == 0
    assert need(0, 1 << 31, 8, 8, 1) == 0 and need(0, 1, 1 << 40, 8, 1) == 0 and need(0, 0, 8, 4096, 1) == 256


def test_empty_batches():
    for name in NAMES[:2]:
        assert _call(name, M=0, p=None, q=None, sizes=None, out=None, ws=None) == 0
    # the weights' gradient of an empty batch is written all the same
    assert _call(NAMES[2], M=0, p=None, q=None, out=None) == 1
    assert _call(NAMES[2], M=0, p=None, q=None) not in (0, 1, 2, 3, 5, 8)


def test_types_of_the_weights_gradient():
    assert _call(NAMES[2], dtype=0, out_dtype=1) == 8 and _call(NAMES[2], dtype=1, out_dtype=0) == 8
    assert _call(NAMES[2], dtype=1, out_dtype=2) not in (0, 8)


def test_python_refusals():
    torch = pytest.importorskip("torch")
    bf = torch.bfloat16
    a, dy, w, sz = torch.zeros(8, 64, dtype=bf), torch.zeros(8, 32, dtype=bf), torch.zeros(2, 32, 64, dtype=bf), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: geg.grouped_gemm(a.float(), sz, w.float()), lambda: geg.grouped_gemm(a, sz, w.half()),
                 lambda: geg.grouped_gemm(a, sz, w[:, :, :56]), lambda: geg.grouped_gemm(a, sz.long(), w),
                 lambda: geg.grouped_gemm(a, sz[:1], w), lambda: geg.grouped_gemm(a.t(), sz, w), lambda: geg.grouped_gemm(a, sz, w[0]),
                 lambda: geg.grouped_gemm(a, sz, w, out=dy[:4]), lambda: geg.grouped_dgrad(a, sz, w),
                 lambda: geg.grouped_dgrad(dy, sz, w, dx=dy), lambda: geg.grouped_wgrad(dy, a[:4], sz),
                 lambda: geg.grouped_wgrad(dy, a.half(), sz), lambda: geg.grouped_wgrad(dy, a, sz, dtype=torch.float16),
                 lambda: geg.grouped_wgrad(dy, a, sz, dw=torch.zeros(2, 32, 56, dtype=bf)), lambda: geg.grouped_wgrad(dy[0], a, sz)):
        with pytest.raises(geg.GegError, match="GEG_ERR_BAD_SHAPE"):
            call()
    for call in (lambda: geg.grouped_gemm(a, sz, w), lambda: geg.grouped_dgrad(dy, sz, w), lambda: geg.grouped_wgrad(dy, a, sz),
                 lambda: geg.grouped_matmul(a, sz, w)):
        with pytest.raises(geg.GegError, match="GPU"):
            call()

"""Refusals of the MXFP4 packer, the gate, the combine's gradient and the few-token layer
before any launch (no GPU needed)."""
import pytest

import grouped_expert_gemm_amd as geg

P = 0x10000


def L():
    return geg.lib()


def _quant(x=P, dtype=0, rows=4, K=64, ld=64, blocks=P, scales=P, values=None):
    return L().gmxfp4_quantize(x, dtype, rows, K, ld, blocks, scales, values, None)


def test_quantize_refusals():
    assert _quant(dtype=3) == 8 and _quant(dtype=-1) == 8
    assert _quant(K=48) == 2 and _quant(K=0) == 2 and _quant(rows=-1) == 2
    assert _quant(ld=32) == 2
    assert b"pitch" in L().geg_last_error()
    assert _quant(rows=1 << 40, K=64) == 2 and _quant(K=1 << 41) == 2
    assert _quant(rows=(1 << 29) + 1) == 2 and _quant(rows=1 << 29) not in (0, 1, 2, 3)
    assert _quant(rows=0, x=None, blocks=None, scales=None) == 0
    assert _quant(x=None) == 1 and _quant(scales=None) == 1
    assert _quant(x=P + 8) == 3 and _quant(values=P + 8) == 3 and _quant(blocks=P + 2) == 3
    assert _quant(ld=68) == 3                     # rows of bf16 136 bytes apart
    assert _quant(rows=1, ld=68) not in (0, 2, 3)   # one row has no pitch: stops at the device check
    assert _quant(dtype=2, ld=68) not in (0, 2, 3)  # 272 bytes
    assert _quant() not in (0, 1, 2, 3, 8)


def _topk(logits=P, dtype=2, T=4, E=8, k=2, w=P, ids=P, err=None):
    return L().geg_route_topk(logits, dtype, T, E, k, 1, w, ids, err, None)


def _topk_grad(dw=P, logits=P, dtype=2, ids=P, w=P, T=4, E=8, k=2, dl=2 * P):
    return L().geg_route_topk_grad(dw, logits, dtype, ids, w, T, E, k, 1, dl, None)


def test_gate_refusals():
    for call in (_topk, _topk_grad):
        assert call(dtype=7) == 8
        assert call(T=-1) == 2 and call(E=0) == 2 and call(k=0) == 2 and call(k=9) == 2
        assert call(E=1025, k=2) == 2
        assert call(E=128, k=65) == 2
        assert call(T=1 << 31) == 2 and call(T=1 << 62) == 2 and call(T=1 << 30, k=4) == 2
        assert call(T=0, logits=None) == 0
        assert call(logits=None) == 1 and call(ids=None) == 1 and call(w=None) == 1
        assert call(logits=P + 2) == 3 and call(logits=P + 2, dtype=0) not in (0, 3)
        assert call() not in (0, 1, 2, 3, 8)
        assert call(T=(1 << 25) + 1) == 2 and call(T=1 << 25) not in (0, 1, 2, 3)
    assert _topk(err=P + 2) == 3
    assert _topk_grad(dl=P) == 8


def _combine_grad(dout=P, y=P, row=P, src=None, w=P, T=4, k=2, N=64, dy=2 * P, dw=P):
    return L().geg_route_combine_grad(dout, y, row, src, w, T, k, N, dy, dw, None)


def test_combine_gradient_refusals():
    assert _combine_grad(N=60) == 2 and _combine_grad(T=-1) == 2 and _combine_grad(k=0) == 2
    assert _combine_grad(T=1 << 62) == 2
    # a launch of one wavefront per entry holds fewer than 2^32 threads
    assert _combine_grad(T=(1 << 24) + 1, k=2) == 2 and _combine_grad(T=1 << 24, k=2) not in (0, 1, 2, 3)
    assert _combine_grad(T=0, dout=None) == 0
    assert _combine_grad(dout=None) == 1 and _combine_grad(y=None) == 1 and _combine_grad(dy=None) == 1
    assert _combine_grad(y=None, dw=None) not in (0, 1)
    assert _combine_grad(dy=P) == 8
    assert _combine_grad(y=P + 8) == 3


def _layer(name="gnf4_moe_layer", x=P, ids=P, w=P, w13=P, s13=P, w2=P, s2=P, out=P, T=4, k=2, H=128, I=64, E=8, ws=P,
           nbytes=1 << 20, opts=None):
    return getattr(L(), name)(x, ids, w, w13, s13, w2, s2, out, T, k, H, I, E, ws, nbytes, opts, None)


def test_layer_refusals():
    for name, m in (("gnf4_moe_layer", 64), ("gmxfp4_moe_layer", 32)):
        assert _layer(name, H=128 + m // 2) == 2 and _layer(name, I=64 + m // 2) == 2
        assert _layer(name, T=17) == 2
        assert b"geg_route_combine" in L().geg_last_error()
        assert _layer(name, T=16, k=17) == 2 and _layer(name, T=-1) == 2 and _layer(name, k=0) == 2
        assert _layer(name, E=0) == 2 and _layer(name, E=1025) == 2
        assert _layer(name, H=65536, I=65536) == 2       # an expert's weights past one buffer window
        assert _layer(name, I=1 << 62) == 2
        assert _layer(name, T=0, x=None, ws=None) == 0
        for p in ("x", "ids", "w", "w13", "s13", "w2", "s2", "out"):
            assert _layer(name, **{p: None}) == 1, p
        for p in ("x", "w13", "w2", "out"):
            assert _layer(name, **{p: P + 8}) == 3, p
        assert _layer(name, ws=None) == 5 and _layer(name, ws=P + 16) == 5
        need = L().geg_moe_layer_workspace_bytes(4, 2, 64)
        assert need == 256 + 3328 + 8 * 64 * 2 + 256   # act fp16 and its scales
        assert _layer(name, nbytes=need - 1) == 5
        assert _layer(name, nbytes=need) not in (0, 1, 2, 3, 5, 8)
    assert _layer(s13=P + 2) == 3 and _layer("gmxfp4_moe_layer", s13=P + 1) not in (0, 3)
    assert L().geg_moe_layer_workspace_bytes(17, 1, 64) == 0


def _w4a4(a=P, sizes=P, w=P, s=P, out=P, M=16, N=64, K=128, E=4, ws=P, nbytes=1 << 20, opts=None):
    import ctypes
    return L().gmxfp4_w4a4_grouped_gemm(a, sizes, w, s, out, M, N, K, E, ws, nbytes,
                                        ctypes.byref(opts) if opts else None, None)


def test_w4a4_refusals():
    assert _w4a4(K=48) == 2 and _w4a4(M=-1) == 2 and _w4a4(N=0) == 2 and _w4a4(E=1025) == 2
    assert _w4a4(N=65536, K=65536) == 2
    assert _w4a4(M=0, a=None, ws=None) == 0
    for p in ("a", "sizes", "w", "s", "out"):
        assert _w4a4(**{p: None}) == 1, p
    assert _w4a4(a=P + 8) == 3 and _w4a4(w=P + 4) == 3 and _w4a4(out=P + 2) == 3
    assert _w4a4(ws=None) == 5 and _w4a4(ws=P + 16) == 5
    assert _w4a4(opts=geg.Opts(1, 0)) == 8 and _w4a4(opts=geg.Opts(3, 0)) == 8 and _w4a4(opts=geg.Opts(0, 0, None, -1)) == 8
    assert _w4a4(opts=geg.Opts(4, 0), K=65536, N=64) == 8      # the narrow kernel's rows past LDS
    assert _w4a4() not in (0, 1, 2, 3, 5, 8)
    # header only up to one row per expert; else codes [ceil(K/128)][M][64] and scales [ceil(K/512)][M][16]
    op = geg.GEG_OP_MXFP4_W4A4
    assert geg.geg_workspace_bytes(op, 4, 64, 128, 4) == 256
    assert geg.geg_workspace_bytes(op, 5, 64, 128, 4) == 256 + 512 + 256
    assert geg.geg_workspace_bytes(op, 8192, 5760, 2880, 32) == 256 + 23 * 8192 * 64 + 6 * 8192 * 16
    assert geg.geg_workspace_bytes(op, 64, 64, 512, 4, geg.Opts(2, 0)) == 256 + 64 * 256 + 64 * 16
    need = geg.geg_workspace_bytes(op, 8192, 64, 128, 4)
    assert _w4a4(M=8192, nbytes=need - 1) == 5 and _w4a4(M=8192, nbytes=need) not in (0, 1, 2, 3, 5, 8)


def test_python_refusals():
    torch = pytest.importorskip("torch")
    bf, i32, f32, u8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8
    x, l = torch.zeros(4, 64, dtype=bf), torch.zeros(4, 8)
    ids, w = torch.zeros(4, 2, dtype=i32), torch.zeros(4, 2)
    y, row = torch.zeros(8, 64, dtype=bf), torch.zeros(8, dtype=i32)
    w13, s13 = torch.zeros(3, 128, 32, dtype=u8), torch.zeros(3, 128, 1)
    w2, s2 = torch.zeros(3, 64, 32, dtype=u8), torch.zeros(3, 64, 1)
    m13, m2 = torch.zeros(3, 128, 2, dtype=u8), torch.zeros(3, 64, 2, dtype=u8)
    for call in (lambda: geg.gmxfp4_quantize(x.double()), lambda: geg.gmxfp4_quantize(x[:, :48]),
                 lambda: geg.gmxfp4_quantize(x.t()), lambda: geg.gmxfp4_quantize(x.reshape(2, 2, 64).transpose(0, 1)),
                 lambda: geg.gmxfp4_quantize(torch.zeros((), dtype=bf)),
                 lambda: geg.route_topk(l.long(), 2), lambda: geg.route_topk(l[0], 2),
                 lambda: geg.route_topk(l, 2, error_word=torch.zeros(2, dtype=i32)),
                 lambda: geg.route_topk_grad(w, l, ids.long(), w), lambda: geg.route_topk_grad(w[:3], l, ids, w),
                 lambda: geg.route_combine_grad(x, y[:7], row, w), lambda: geg.route_combine_grad(x, y, row, w, row[:3]),
                 lambda: geg.gmxfp4_w4a4_grouped_gemm(x.float(), torch.zeros(3, dtype=i32), w2, m2),
                 lambda: geg.gmxfp4_w4a4_grouped_gemm(x, torch.zeros(3, dtype=i32), w2, s2),
                 lambda: geg.gmxfp4_w4a4_grouped_gemm(x, torch.zeros(2, dtype=i32), w2, m2),
                 lambda: geg.gnf4_moe_layer(x, ids, w, w13, m13, w2, s2),
                 lambda: geg.gmxfp4_moe_layer(x, ids, w, w13, s13, w2, m2),
                 lambda: geg.gnf4_moe_layer(x, ids.long(), w, w13, s13, w2, s2),
                 lambda: geg.gnf4_moe_layer(x, ids, w.double(), w13, s13, w2, s2),
                 lambda: geg.gnf4_moe_layer(x, ids[:3], w, w13, s13, w2, s2),
                 lambda: geg.gnf4_moe_layer(x, ids, w, w13, s13, w2[:2], s2)):
        with pytest.raises(geg.GegError, match="GEG_ERR_BAD_SHAPE"):
            call()
    for call in (lambda: geg.gmxfp4_quantize(x), lambda: geg.route_topk(l, 2),
                 lambda: geg.route_topk_grad(w, l, ids, w), lambda: geg.route_combine_grad(x, y, row, w),
                 lambda: geg.gmxfp4_w4a4_grouped_gemm(x, torch.zeros(3, dtype=i32), w2, m2),
                 lambda: geg.gnf4_moe_layer(x, ids, w, w13, s13, w2, s2),
                 lambda: geg.gmxfp4_moe_layer(x, ids, w, w13, m13, w2, m2)):
        with pytest.raises(geg.GegError, match="GPU"):
            call()


def test_the_packages_paths_stay_paths():
    import os
    assert os.path.isdir(geg._HERE) and os.path.dirname(geg.LIB_PATH) == geg._HERE

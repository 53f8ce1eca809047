"""Dropout from a counter-based generator (philox_dropout, dropout) and of an adapter's input
(grouped_linear_lora's dropout) against the oracle's mask.

Tolerance of plain dropout: the scale is an fp32 value (2^-24 off), the product and the sum with
the residual round once each in fp32, the result once to its type: finfo.eps / 2 of it, or half
a subnormal step."""
import numpy as np
import pytest

import oracle
from gpu_util import assert_close, bf16_to_f64, log, up, up_u16_as_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def geg():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_expert_gemm_amd as g
    g.lib()
    return g


def _type(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def _keep(shape, p, seed, offset):
    import torch
    return torch.from_numpy(oracle.dropout_keep(tuple(shape), p, seed, offset)).cuda()


def _check(got, x, keep, p, residual, what):
    import torch
    v = torch.where(keep, x.double() * oracle.dropout_scale(p), 0.0)
    ref = v if residual is None else v + residual.double()
    info = torch.finfo(x.dtype)
    step = 0.0 if x.dtype == torch.float32 else info.eps / 2
    tol = step * ref.abs() + 3 * 2.0 ** -24 * (v.abs() + ref.abs()) + info.smallest_normal * info.eps / 2
    assert ((got.double() - ref).abs() <= tol).all(), what
    if residual is None:
        assert ((got == 0) | keep).all() and torch.equal(got != 0, keep & (x != 0)) or p == 1.0, what


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shape,p", [((1,), 0.5), ((7,), 0.3), ((8,), 0.5), ((3, 5), 0.1), ((65, 33), 0.0), ((1000, 129), 0.25),
                                     ((64, 2048), 0.05), ((3, 5, 77), 0.9), ((4097, 641), 0.4), ((16, 16), 1.0)])
def test_values_and_mask(geg, dtype, shape, p):
    import torch
    log(f"case: dropout {dtype} {shape} p={p}")
    g = torch.Generator(device="cuda").manual_seed(len(shape) + shape[0])
    x, res = (torch.randn(*shape, generator=g, device="cuda").to(_type(dtype)) for _ in range(2))
    for seed, offset in ((0, 0), (0x123456789ABCDEF0, 0xFEDCBA9876543210), ((1 << 64) - 1, 5)):
        keep = _keep(shape, p, seed, offset)
        _check(geg.philox_dropout(x, p, seed, offset), x, keep, p, None, "plain")
        _check(geg.philox_dropout(x, p, seed, offset, residual=res), x, keep, p, res, "with a residual")
    # words on the device: seed instead of the given one, offset added to it
    rng = torch.tensor([77, (1 << 62) + 3], dtype=torch.int64, device="cuda")
    assert torch.equal(geg.philox_dropout(x, p, rng, 9), geg.philox_dropout(x, p, 77, (1 << 62) + 12))


def test_in_place_and_unaligned(geg):
    import torch
    log("case: dropout in place and at odd addresses")
    for dtype in ("bf16", "fp32"):
        x, res = torch.randn(5001, device="cuda").to(_type(dtype)), torch.randn(5001, device="cuda").to(_type(dtype))
        want, wres = geg.philox_dropout(x, 0.3, 1, 2), geg.philox_dropout(x, 0.3, 1, 2, residual=res)
        y = x.clone()
        assert geg.philox_dropout(y, 0.3, 1, 2, out=y) is y and torch.equal(y, want)
        z = res.clone()
        geg.philox_dropout(x, 0.3, 1, 2, residual=z, out=z)
        assert torch.equal(z, wres)
        buf = torch.full((5010,), 9.0, dtype=x.dtype, device="cuda")
        buf[3:5004] = x
        got = torch.full((5010,), 4.0, dtype=x.dtype, device="cuda")
        geg.philox_dropout(buf[3:5004], 0.3, 1, 2, out=got[1:5002])
        assert torch.equal(got[1:5002], want) and got[0] == 4 and (got[5002:] == 4).all()


def test_dropped_infinities_leave_nothing(geg):
    import torch
    x = torch.full((4096,), float("inf"), dtype=torch.bfloat16, device="cuda")
    x[::2] = float("nan")
    out, keep = geg.philox_dropout(x, 0.5, 3), _keep((4096,), 0.5, 3, 0)
    assert (out[~keep] == 0).all() and not out[keep].isfinite().any()


def test_past_2_31_elements(geg):
    import torch
    log("case: dropout of more than 2^31 elements")
    n = (1 << 31) + 24
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    out = geg.philox_dropout(x, 0.5, 11, 4, out=x)
    for first in (0, (1 << 31) - 32):
        m = min(64, n - first)
        keep = torch.from_numpy(oracle.dropout_bits(m, 11, 4, first) >= 32768).cuda()
        assert torch.equal(out[first:first + m] == 2, keep) and torch.equal(out[first:first + m] == 0, ~keep)


def test_autograd_op(geg):
    import torch
    log("case: dropout as an autograd op")
    x = torch.randn(33, 70, device="cuda", dtype=torch.float32, requires_grad=True)
    res = torch.randn(33, 70, device="cuda", requires_grad=True)
    dout = torch.randn(33, 70, device="cuda")
    for seed in (5, torch.tensor([5, 0], dtype=torch.int64, device="cuda")):
        x.grad = res.grad = None
        out = geg.dropout(x, 0.2, seed, 3, residual=res)
        out.backward(dout)
        keep = _keep((33, 70), 0.2, 5, 3)
        _check(x.grad, dout, keep, 0.2, None, "dx")
        assert torch.equal(res.grad, dout)
    # the op is linear in x: a difference along a direction equals the gradient's product with it
    v = torch.randn(33, 70, device="cuda")
    with torch.no_grad():
        diff = ((geg.dropout(x + v, 0.2, 5, 3) - geg.dropout(x - v, 0.2, 5, 3)).double() / 2 * dout.double()).sum()
    slope = (x.grad.double() * v.double()).sum()
    bound = 2.0 ** -22 * ((x.abs() + v.abs()).double() * 2 * dout.abs().double()).sum()
    assert (diff - slope).abs() <= bound
    # a seed tensor changed before the backward pass is refused
    words = torch.tensor([5, 0], dtype=torch.int64, device="cuda")
    out = geg.dropout(x, 0.2, words)
    words.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.backward(dout)


def test_captured_masks_change_with_their_words(geg):
    import torch
    log("case: dropout captured")
    x = torch.randn(300, 41, device="cuda").to(torch.bfloat16)
    words = torch.tensor([9, 0], dtype=torch.int64, device="cuda")
    geg.philox_dropout(x, 0.5, words)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = geg.philox_dropout(x, 0.5, words, 1)
        dx = geg.philox_dropout(out, 0.5, words, 1)
        words[1].add_(1)
    words.copy_(torch.tensor([9, 0]))
    for step in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert int(words[1]) == step + 1
        want = geg.philox_dropout(x, 0.5, 9, 1 + step)
        assert torch.equal(out, want) and torch.equal(dx, geg.philox_dropout(want, 0.5, 9, 1 + step))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = geg.philox_dropout(x, 0.5, 9, 4, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)


@pytest.mark.parametrize("fmt,r,K,N,sizes,p", [("nf4", 16, 256, 200, [0, 5, 40, 0, 130, 1], 0.1),
                                               ("nf4", 40, 320, 136, [33, 2], 0.5), ("mxfp4", 64, 288, 136, [9, 0, 70], 0.25),
                                               ("mxfp4", 8, 1056, 96, [17, 300], 0.9), ("nf4", 8, 64, 64, [20], 1.0)])
def test_adapter_dropout(geg, fmt, r, K, N, sizes, p):
    """The adapter's path with a mask: forward and backward against the same oracle as without
    one, its adapter part on the masked activations; the tolerance is that of the path."""
    import torch
    from oracle import lora as L
    from test_gpu_lora import _case
    log(f"case: adapter dropout {fmt} r={r} K={K} N={N} sizes={sizes} p={p}")
    x, dy, A, B, sz, W, codes, scales = _case(fmt, len(sizes), K, N, r, sizes, seed=K + N + r)
    s, seed, offset = 0.5, 0x1234567812345678, 40
    keep = oracle.dropout_keep(x.shape, p, seed, offset)
    xm = np.where(keep, L._f64(x), 0.0)
    s2 = s * oracle.dropout_scale(p)
    a = up_u16_as_bf16(x).requires_grad_(True)
    At, Bt = up(A).requires_grad_(True), up(B).requires_grad_(True)
    szt, wt, st = up(sz), up(codes), up(scales)
    zero = lambda e: np.zeros((N, K))
    fwd_ref = oracle.grouped_ref(x, sz, W, N) + L.lora_delta_ref(xm, sz, A, B, s2)[0]
    dx_w = oracle.dgrad_ref(dy, sz, W, K)
    dx_a, dA_ref, dB_ref = L.lora_backward_ref(xm, dy, sz, zero, A, B, s2, K)
    words = torch.tensor([seed, 30], dtype=torch.int64, device="cuda")
    for which, off in ((seed, offset), (words, 10)):
        a.grad = At.grad = Bt.grad = None
        out = geg.grouped_linear_lora(a, szt, wt, st, At, Bt, s, fmt, True, dropout=p, seed=which, offset=off)
        out.backward(up_u16_as_bf16(dy))
        assert_close(bf16_to_f64(out), fwd_ref, "forward")
        assert_close(bf16_to_f64(a.grad), dx_w + np.where(keep, dx_a, 0.0), "dx")
        assert_close(At.grad.cpu().numpy().astype(np.float64), dA_ref, "dA")
        assert_close(Bt.grad.cpu().numpy().astype(np.float64), dB_ref, "dB")


def test_adapter_dropout_leaves_the_projection_and_p_0(geg):
    import torch
    from test_gpu_lora import _case
    log("case: adapter dropout of nothing, and of an adapter that is zero")
    x, dy, A, B, sz, W, codes, scales = _case("nf4", 3, 256, 136, 16, [5, 40, 300], seed=3)
    a, szt, wt, st = up_u16_as_bf16(x), up(sz), up(codes), up(scales)
    At, Bt = up(A), up(B)
    plain = geg.grouped_linear_lora(a, szt, wt, st, At, Bt, 0.5)
    assert torch.equal(geg.grouped_linear_lora(a, szt, wt, st, At, Bt, 0.5, dropout=0.0), plain)
    tiny = geg.grouped_linear_lora(a, szt, wt, st, At, Bt, 0.5, dropout=1e-9, seed=1)   # rounds to no drop at all
    assert torch.equal(tiny, plain)
    zero = torch.zeros_like(Bt)
    base = geg.grouped_linear_lora(a, szt, wt, st, At, zero, 0.5)
    assert torch.equal(geg.grouped_linear_lora(a, szt, wt, st, At, zero, 0.5, dropout=0.5, seed=1), base)
    with pytest.raises(geg.GegError, match="seed"):
        geg.grouped_linear_lora(a, szt, wt, st, At, Bt, 0.5, dropout=0.1)


def test_captured_adapter_step(geg):
    """Forward and backward of the adapter's path captured: the words of the seed and the inputs
    change between replays, each as the eager step."""
    import torch
    from test_gpu_lora import _case
    log("case: adapter dropout, a captured training step")
    x, dy, A, B, sz, W, codes, scales = _case("nf4", 3, 256, 136, 16, [5, 40, 300], seed=4)
    a, A, B = up_u16_as_bf16(x).requires_grad_(True), up(A).requires_grad_(True), up(B).requires_grad_(True)
    szt, wt, st, d = up(sz), up(codes), up(scales), up_u16_as_bf16(dy)
    words = torch.tensor([3, 0], dtype=torch.int64, device="cuda")

    def step():
        out = geg.grouped_linear_lora(a, szt, wt, st, A, B, 0.5, dropout=0.3, seed=words)
        return (out.detach(), *torch.autograd.grad(out, (a, A, B), d))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    before = None
    for i in range(4):
        words.copy_(torch.tensor([3, 7 + i]))
        with torch.no_grad():
            a.mul_(0.5)
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w)
        assert before is None or not torch.equal(before, want[0])
        before = want[0]

"""Grouped products with 16-bit weights (grouped_gemm, grouped_dgrad, grouped_wgrad, grouped_matmul)
against a per-expert loop in fp64.

Tolerance per element: the products of 16-bit values are exact in fp32; a sum of C of them takes
at most 32 additions inside a matrix instruction and C / 32 between them, each off by at most one
fp32 step (2^-23) of the sum of magnitudes S = sum |p q|; the result is rounded once, by at most
finfo.eps / 2 of its value, or half a subnormal step."""
import pytest

from gpu_util import log

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def geg():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_expert_gemm_amd as g
    g.lib()
    return g


def _types():
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16}


def _case(dtype, sizes, N, K, seed, extra=0):
    import torch
    t = _types()[dtype]
    g = torch.Generator(device="cuda").manual_seed(seed)
    M, E = sum(sizes) + extra, len(sizes)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(t)
    return rand(M, K), rand(M, N), rand(E, N, K), torch.tensor(sizes, dtype=torch.int32, device="cuda")


def _groups(sizes):
    r = 0
    for e, n in enumerate(sizes):
        yield e, slice(r, r + n)
        r += n


def _ref(p, q, sizes, kind):
    """The product in fp64 and the sums of magnitudes: forward (p = a, q = w), dgrad (p = dy,
    q = w), wgrad (p = dy, q = a)."""
    import torch
    out = []
    for f in (lambda x: x.double(), lambda x: x.double().abs()):
        if kind == "wgrad":
            r = torch.zeros(len(sizes), p.shape[1], q.shape[1], dtype=torch.float64, device="cuda")
            for e, rows in _groups(sizes):
                r[e] = f(p[rows]).t().contiguous() @ f(q[rows])
        else:
            width = q.shape[1] if kind == "forward" else q.shape[2]
            r = torch.zeros(sum(sizes), width, dtype=torch.float64, device="cuda")
            for e, rows in _groups(sizes):
                r[rows] = f(p[rows]) @ (f(q[e]).t().contiguous() if kind == "forward" else f(q[e]))
        out.append(r)
    return out


def _check(got, ref, mag, C, what):
    import torch
    info = torch.finfo(got.dtype)
    step = 0.0 if got.dtype == torch.float32 else info.eps / 2
    tol = step * ref.abs() + (C / 32 + 32) * 2.0 ** -23 * mag + info.smallest_normal * info.eps / 2
    over = ((got.double() - ref).abs() / tol).max().item() if ref.numel() else 0.0
    log(f"  {what}: largest error {over:.3f} of its bound")
    assert got.isfinite().all() and over <= 1.0, what


SHAPES = [
    # sizes, N, K: experts without rows, one row, borders of the tiles in rows, columns and contraction
    ([0, 1, 5, 0, 40, 17], 40, 64),
    ([3], 8, 8),
    ([1, 0, 0, 1], 264, 72),
    ([255, 256, 257, 0], 256, 64),
    ([64, 65, 127, 128, 129, 191], 248, 200),
    ([700, 2, 0, 31], 520, 328),
    ([63, 1000], 72, 1096),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("sizes,N,K", SHAPES)
def test_each_direction(geg, dtype, sizes, N, K):
    import torch
    log(f"case: 16-bit products {dtype} sizes={sizes} N={N} K={K}")
    a, dy, w, sz = _case(dtype, sizes, N, K, seed=N + K)
    ref, mag = _ref(a, w, sizes, "forward")
    for path in (0, 2, 4, 5):
        _check(geg.grouped_gemm(a, sz, w, opts=geg.Opts(path, 0), check_errors=True), ref, mag, K, f"forward path {path}")
    ref, mag = _ref(dy, w, sizes, "dgrad")
    for path in (0, 2, 5):
        _check(geg.grouped_dgrad(dy, sz, w, opts=geg.Opts(path, 0), check_errors=True), ref, mag, N, f"dgrad path {path}")
    ref, mag = _ref(dy, a, sizes, "wgrad")
    for path in (0, 2, 5):
        for out in (None, torch.float32):
            dw = geg.grouped_wgrad(dy, a, sz, dtype=out, opts=geg.Opts(path, 0), check_errors=True)
            assert dw.dtype == (out or a.dtype)
            _check(dw, ref, mag, max(sizes), f"wgrad {dw.dtype} path {path}")
        assert (dw[sz == 0] == 0).all()


@pytest.mark.parametrize("N", [1, 7, 257, 1023])
def test_forward_odd_widths(geg, N):
    log(f"case: 16-bit forward N={N}")
    sizes = [3, 0, 290]
    a, _, w, sz = _case("bf16", sizes, N, 136, seed=N)
    ref, mag = _ref(a, w, sizes, "forward")
    for path in (2, 4, 5):
        _check(geg.grouped_gemm(a, sz, w, opts=geg.Opts(path, 0)), ref, mag, 136, f"path {path}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_contraction_in_pieces(geg, dtype):
    import torch
    log(f"case: 16-bit products {dtype}, few tiles and a long contraction")
    o, few = geg.Opts(5, 0), geg.Opts(5, 0, None, 8)
    for sizes, N, K in (([100, 0, 130], 200, 4104), ([1, 2], 257, 8200), ([5, 300, 0, 1], 72, 2104), ([140], 8, 2048)):
        a, _, w, sz = _case(dtype, sizes, N, K, seed=N + K, extra=3)
        assert geg.lib().geg_grouped_workspace_bytes(0, sum(sizes) + 3, N, K, len(sizes)) > 256
        a[sum(sizes):] = float("nan")
        got = geg.grouped_gemm(a, sz, w, opts=o, zero_rest=True, check_errors=True)
        assert (got[sum(sizes):] == 0).all()
        _check(got[:sum(sizes)], *_ref(a[:sum(sizes)], w, sizes, "forward"), K, f"forward {sizes}")
        assert torch.equal(geg.grouped_gemm(a, sz, w, opts=few, zero_rest=True), got)
    for sizes, N, K in (([100, 0, 130], 4104, 200), ([1, 2], 8200, 264), ([5, 300, 0, 1], 2104, 72)):
        _, dy, w, sz = _case(dtype, sizes, N, K, seed=N + K)
        assert geg.lib().geg_grouped_workspace_bytes(1, sum(sizes), N, K, len(sizes)) > 256
        got = geg.grouped_dgrad(dy, sz, w, opts=o)
        _check(got, *_ref(dy, w, sizes, "dgrad"), N, f"dgrad {sizes}")
        assert torch.equal(geg.grouped_dgrad(dy, sz, w, opts=few), got)
    for sizes, N, K in (([6100, 0, 300], 264, 136), ([2030, 2200], 8, 520), ([5001], 128, 256)):
        a, dy, _, sz = _case(dtype, sizes, N, K, seed=N + K)
        assert geg.lib().geg_grouped_workspace_bytes(2, sum(sizes), N, K, len(sizes)) > 256
        for out in (None, torch.float32):
            got = geg.grouped_wgrad(dy, a, sz, dtype=out, opts=o)
            _check(got, *_ref(dy, a, sizes, "wgrad"), max(sizes), f"wgrad {sizes}")
            assert torch.equal(geg.grouped_wgrad(dy, a, sz, dtype=out, opts=few), got)


def test_many_rounds_per_workgroup(geg):
    import torch
    log("case: 16-bit products on 8 compute units")
    sizes, N, K = [300, 0, 77, 513, 1, 256, 90], 776, 584
    a, dy, w, sz = _case("bf16", sizes, N, K, seed=3)
    for limit in (1, 3, 8):
        for path in (2, 4, 5):
            o = geg.Opts(path, 0, None, limit)
            assert torch.equal(geg.grouped_gemm(a, sz, w, opts=o), geg.grouped_gemm(a, sz, w, opts=geg.Opts(path, 0)))
        for path in (2, 5):
            o, free = geg.Opts(path, 0, None, limit), geg.Opts(path, 0)
            assert torch.equal(geg.grouped_dgrad(dy, sz, w, opts=o), geg.grouped_dgrad(dy, sz, w, opts=free))
            assert torch.equal(geg.grouped_wgrad(dy, a, sz, opts=o), geg.grouped_wgrad(dy, a, sz, opts=free))


def test_1024_experts(geg):
    log("case: 16-bit products, 1024 experts")
    sizes = [(7 * e) % 5 if e % 3 else 0 for e in range(1024)]
    a, dy, w, sz = _case("fp16", sizes, 48, 40, seed=4)
    ref, mag = _ref(a, w, sizes, "forward")
    for path in (2, 4, 5):
        _check(geg.grouped_gemm(a, sz, w, opts=geg.Opts(path, 0)), ref, mag, 40, f"path {path}")
    for path in (2, 5):
        o = geg.Opts(path, 0)
        _check(geg.grouped_dgrad(dy, sz, w, opts=o), *_ref(dy, w, sizes, "dgrad"), 48, f"dgrad path {path}")
        _check(geg.grouped_wgrad(dy, a, sz, opts=o), *_ref(dy, a, sizes, "wgrad"), max(sizes), f"wgrad path {path}")


@pytest.mark.parametrize("path", [2, 4, 5])
def test_rows_past_the_experts(geg, path):
    import torch
    log(f"case: 16-bit products, rows past the experts, path {path}")
    sizes, N, K = [20, 0, 9], 41, 64
    a, dy, w, sz = _case("bf16", sizes, N, K, seed=5, extra=300)
    o = geg.Opts(path, 0)
    a[29:] = float("nan")
    out = torch.full((329, N), 7.0, dtype=a.dtype, device="cuda")
    geg.grouped_gemm(a, sz, w, out=out, opts=o)
    assert (out[29:] == 7).all() and out[:29].isfinite().all()
    out = geg.grouped_gemm(a, sz, w, out=out, opts=o, zero_rest=True)
    assert (out[29:] == 0).all()
    if path != 4:
        dy, w = dy[:, :40].contiguous(), w[:, :40].contiguous()
        dy[29:] = float("nan")
        dx = torch.full((329, K), 7.0, dtype=a.dtype, device="cuda")
        geg.grouped_dgrad(dy, sz, w, dx=dx, opts=o)
        assert (dx[29:] == 7).all() and dx[:29].isfinite().all()
        assert (geg.grouped_dgrad(dy, sz, w, dx=dx, zero_rest=True, opts=o)[29:] == 0).all()
        dw = geg.grouped_wgrad(dy, a, sz, opts=o)
        assert dw.isfinite().all() and (dw[1] == 0).all()


def test_flagged_sizes(geg):
    import torch
    log("case: 16-bit products, sizes past M and negative ones")
    a, dy, w, _ = _case("bf16", [10, 10], 64, 64, seed=6)
    for sizes, bit in (([15, 9], geg.DEVERR_SIZES_EXCEED_M), ([-3, 20], geg.DEVERR_NEGATIVE_SIZE)):
        sz = torch.tensor(sizes, dtype=torch.int32, device="cuda")
        for call in (lambda: geg.grouped_gemm(a, sz, w, check_errors=True),
                     lambda: geg.grouped_gemm(a, sz, w, check_errors=True, opts=geg.Opts(2, 0)),
                     lambda: geg.grouped_dgrad(dy, sz, w, check_errors=True),
                     lambda: geg.grouped_wgrad(dy, a, sz, check_errors=True)):
            with pytest.raises(geg.GegDeviceError) as e:
                call()
            assert e.value.bits == bit


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_value_stays_in_its_row(geg, bad):
    import torch
    log(f"case: 16-bit products with {bad}")
    sizes, N, K = [30, 5, 40], 72, 72   # contraction tails of 8 past a whole stage
    a, dy, w, sz = _case("bf16", sizes, N, K, seed=7)
    plain = [geg.grouped_gemm(a, sz, w, opts=geg.Opts(p, 0)) for p in (2, 4, 5)] + [geg.grouped_dgrad(dy, sz, w, opts=geg.Opts(p, 0)) for p in (2, 5)]
    row = 31
    a2, dy2 = a.clone(), dy.clone()
    a2[row], dy2[row] = bad, bad
    got = [geg.grouped_gemm(a2, sz, w, opts=geg.Opts(p, 0)) for p in (2, 4, 5)] + [geg.grouped_dgrad(dy2, sz, w, opts=geg.Opts(p, 0)) for p in (2, 5)]
    for p, q in zip(plain, got):
        assert not q[row].isfinite().any()
        q[row] = p[row]
        assert torch.equal(p, q)
    # a column of dy reaches its row of dW alone, a column of a its column, in their expert
    for path in (2, 5):
        o = geg.Opts(path, 0)
        dw = geg.grouped_wgrad(dy, a, sz, opts=o)
        dy2 = dy.clone()
        dy2[row, 70] = bad
        got = geg.grouped_wgrad(dy2, a, sz, opts=o)
        assert not got[1, 70].isfinite().any()
        got[1, 70] = dw[1, 70]
        assert torch.equal(got, dw)
        a2 = a.clone()
        a2[row, 3] = bad
        got = geg.grouped_wgrad(dy, a2, sz, opts=o)
        assert not got[1, :, 3].isfinite().any()
        got[1, :, 3] = dw[1, :, 3]
        assert torch.equal(got, dw)


def test_overflow_to_inf_in_fp16(geg):
    import torch
    log("case: fp16 results past 65504")
    sz = torch.tensor([4], dtype=torch.int32, device="cuda")
    a, w = torch.full((4, 64), 200.0, dtype=torch.float16, device="cuda"), torch.full((1, 8, 64), 100.0, dtype=torch.float16, device="cuda")
    for p in (2, 4, 5):
        assert (geg.grouped_gemm(a, sz, w, opts=geg.Opts(p, 0)) == float("inf")).all()
    assert (geg.grouped_wgrad(a, a, sz) == float("inf")).all()
    assert (geg.grouped_wgrad(a, a, sz, dtype=torch.float32) == 160000.0).all()


def test_empty_batch(geg):
    import torch
    log("case: 16-bit products, M = 0")
    a, dy, w, sz = _case("bf16", [0, 0, 0], 64, 32, seed=8)
    assert geg.grouped_gemm(a, sz, w).shape == (0, 64) and geg.grouped_dgrad(dy, sz, w).shape == (0, 32)
    dw = torch.full((3, 64, 32), 5.0, dtype=torch.bfloat16, device="cuda")
    assert (geg.grouped_wgrad(dy, a, sz, dw=dw) == 0).all()


def test_offsets_past_2_31(geg):
    import torch
    log("case: 16-bit products with more than 2^31 elements")
    t = torch.bfloat16
    K, N = 8, 32768
    M = (1 << 31) // N + 300
    sizes = [M - 200, 0, 200]
    a, sz = torch.randn(M, K, device="cuda").to(t), torch.tensor(sizes, dtype=torch.int32, device="cuda")
    w = torch.randn(3, N, K, device="cuda").to(t)
    out = geg.grouped_gemm(a, sz, w)
    rows = torch.tensor([0, 5, M - 201, M - 200, M - 1], device="cuda")
    for r in rows.tolist():
        ref = w[0 if r < M - 200 else 2].double() @ a[r].double()
        assert ((out[r].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-4).all(), r
    dx = geg.grouped_dgrad(out, sz, w)
    dw = geg.grouped_wgrad(out, a, sz)
    r = M - 1
    ref, mag = out[r].double() @ w[2].double(), out[r].double().abs() @ w[2].double().abs()
    _check(dx[r:], ref[None], mag[None], N, "dgrad of the last row")
    rows = slice(M - 200, M)
    o, x = out[rows].double(), a[rows].double()
    _check(dw[2], o.t().contiguous() @ x, o.abs().t().contiguous() @ x.abs(), 200, "wgrad of the last expert")
    del out, dx, dw
    E, N, K = 9, 16384, 16384   # weights of 2.4 10^9 elements
    w = torch.zeros(E, N, K, dtype=t, device="cuda")
    w[E - 1].fill_diagonal_(2.0)
    sz = torch.tensor([0] * (E - 1) + [40], dtype=torch.int32, device="cuda")
    a = torch.randn(40, K, device="cuda").to(t)
    for p in (2, 4, 5):
        assert torch.equal(geg.grouped_gemm(a, sz, w, opts=geg.Opts(p, 0)), 2 * a)
    for p in (2, 5):
        assert torch.equal(geg.grouped_dgrad(a, sz, w, opts=geg.Opts(p, 0)), 2 * a)


def test_autograd_op_and_differences(geg):
    import torch
    log("case: grouped_matmul")
    sizes, N, K = [20, 0, 31, 3], 40, 56
    a, dy, w, sz = _case("bf16", sizes, N, K, seed=9, extra=10)
    a[54:], dy[54:] = float("nan"), float("nan")   # padding
    a.requires_grad_(True), w.requires_grad_(True)
    out = geg.grouped_matmul(a, sz, w)
    assert (out[54:] == 0).all()
    out.backward(dy)
    assert (a.grad[54:] == 0).all()
    ad, wd, gd = a.detach(), w.detach(), dy
    _check(out[:54].detach(), *_ref(ad, wd, sizes, "forward"), K, "forward")
    _check(a.grad[:54], *_ref(gd, wd, sizes, "dgrad"), N, "da")
    _check(w.grad, *_ref(gd, ad, sizes, "wgrad"), max(sizes), "dw")
    # a step along a direction against the gradients: the product is bilinear, so central
    # differences in fp64 are exact up to rounding
    g = torch.Generator(device="cuda").manual_seed(1)
    va = torch.randn(54, K, generator=g, device="cuda", dtype=torch.float64)
    vw = torch.randn(4, N, K, generator=g, device="cuda", dtype=torch.float64)

    def value(a, w):
        return sum(((a[r] @ w[e].t().contiguous()) * gd[r].double()).sum() for e, r in _groups(sizes))
    x, y = ad[:54].double(), wd.double()
    diff = (value(x + va, y + vw) - value(x - va, y - vw)) / 2
    slope = (a.grad[:54].double() * va).sum() + (w.grad.double() * vw).sum()
    # each gradient entry is off by at most 2^-8 of itself
    bound = 2.0 ** -8 * ((a.grad[:54].double() * va).abs().sum() + (w.grad.double() * vw).abs().sum())
    assert (diff - slope).abs() <= bound


def test_captured_training_step(geg):
    """Two products with dropout between them and on the way into the residual, forward and both
    backward passes in one graph; inputs, sizes and the dropout's words change between replays."""
    import torch
    log("case: captured training step")
    E, K, I, M = 4, 64, 136, 300
    g = torch.Generator(device="cuda").manual_seed(13)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    x, w1, w2, dout = draw(M, K).requires_grad_(True), draw(E, I, K).requires_grad_(True), draw(E, K, I).requires_grad_(True), draw(M, K)
    sz = torch.tensor([100, 0, 190, 7], dtype=torch.int32, device="cuda")
    words = torch.tensor([5, 0], device="cuda")

    def step():
        h = geg.dropout(geg.grouped_matmul(x, sz, w1), 0.25, words, 0)
        out = geg.dropout(geg.grouped_matmul(h, sz, w2), 0.25, words, 1, residual=x)
        return (out, *torch.autograd.grad(out, (x, w1, w2), dout))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [t.detach() for t in step()]
    seen = []
    for n in range(3):
        with torch.no_grad():
            x.copy_(draw(M, K)), w1.copy_(draw(E, I, K)), w2.copy_(draw(E, K, I))
        words[1] += 2
        sz.copy_(torch.tensor([100 - n, n, 190, 7], dtype=torch.int32))
        want = [t.detach().clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        seen.append((got[0] == x.detach()).float().mean().item())
    # values whose delta was dropped: 0.25 of all, 4 standard deviations of a binomial of 300 * 64
    assert all(abs(v - 0.25) < 4 * (0.25 * 0.75 / (M * K)) ** 0.5 + 3 / M for v in seen), seen


def test_only_one_gradient(geg):
    import torch
    a, dy, w, sz = _case("fp16", [4, 9], 16, 24, seed=10)
    a.requires_grad_(True)
    geg.grouped_matmul(a, sz, w).backward(dy)
    assert a.grad is not None and w.grad is None
    a2, w2 = a.detach(), w.requires_grad_(True)
    geg.grouped_matmul(a2, sz, w2).backward(dy)
    assert a2.grad is None and w2.grad is not None


def test_captured_and_on_streams(geg):
    import torch
    log("case: 16-bit products captured and on another stream")
    sizes, N, K = [40, 0, 300, 7], 264, 136
    a, dy, w, sz = _case("bf16", sizes, N, K, seed=11)

    def step():
        return (geg.grouped_gemm(a, sz, w), geg.grouped_gemm(a, sz, w, opts=geg.Opts(4, 0)), geg.grouped_dgrad(dy, sz, w),
                geg.grouped_wgrad(dy, a, sz))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in range(3):
        na, ndy, nw, _ = _case("bf16", sizes, N, K, seed=20 + seed)
        a.copy_(na), dy.copy_(ndy), w.copy_(nw)
        sz.copy_(torch.tensor([40, 0, 300 - seed, 7 + seed], dtype=torch.int32))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [geg.grouped_gemm(a, sz, w, stream=s), geg.grouped_dgrad(dy, sz, w, stream=s), geg.grouped_wgrad(dy, a, sz, stream=s)]
    torch.cuda.current_stream().wait_stream(s)
    for x, y in zip(outs, (want[0], want[2], want[3])):
        assert torch.equal(x, y)


def test_training_layer(geg):
    """Router, dispatch, two products with a gated unit between them, combine: a whole layer of
    experts that are not quantised, against fp64 autograd on the CPU. Tolerance: every stored
    16-bit intermediate is off by 2^-8 of itself at most; along the longest chain (rows, gate/up,
    unit, down, combine; and back) twelve such roundings meet, taken against the largest value."""
    import torch
    log("case: training layer of 16-bit experts")
    T, E, k, H, I = 96, 6, 2, 64, 40
    g = torch.Generator().manual_seed(12)
    x0 = torch.randn(T, H, generator=g).bfloat16()
    logits0 = torch.randn(T, E, generator=g)
    w13_0 = (torch.randn(E, 2 * I, H, generator=g) * H ** -0.5).bfloat16()
    w2_0 = (torch.randn(E, H, I, generator=g) * I ** -0.5).bfloat16()
    dout = torch.randn(T, H, generator=g).bfloat16()

    x, logits, w13, w2 = (v.cuda().requires_grad_(True) for v in (x0, logits0, w13_0, w2_0))
    weights, ids = geg.router_gate(logits, k)
    xs, sizes, row_of, src_of = geg.dispatch_rows(x, ids, E)
    h = geg.grouped_matmul(xs, sizes, w13).float()
    act = (torch.nn.functional.silu(h[:, 0::2]) * h[:, 1::2]).bfloat16()
    out = geg.combine_rows(geg.grouped_matmul(act, sizes, w2), weights, row_of, src_of)
    out.backward(dout.cuda())

    xr, lr, w13r, w2r = (v.double().requires_grad_(True) for v in (x0, logits0, w13_0, w2_0))
    wr = torch.softmax(lr.gather(1, ids.cpu().long()), 1)
    ref = 0
    for s in range(k):
        e = ids.cpu()[:, s].long()
        hr = (w13r[e] @ xr.unsqueeze(-1)).squeeze(-1)
        ar = torch.nn.functional.silu(hr[:, 0::2]) * hr[:, 1::2]
        ref = ref + wr[:, s:s + 1] * (w2r[e] @ ar.unsqueeze(-1)).squeeze(-1)
    ref.backward(dout.double())
    for got, want, what in ((out, ref, "out"), (x.grad, xr.grad, "dx"), (logits.grad, lr.grad, "dlogits"),
                            (w13.grad, w13r.grad, "dw13"), (w2.grad, w2r.grad, "dw2")):
        off = ((got.detach().double().cpu() - want.detach()).abs().max() / want.detach().abs().max()).item()
        log(f"  {what}: {off:.2e} of the largest value")
        assert off <= 12 * 2.0 ** -8, what


def test_an_expert_of_nearly_2_31_rows(geg):
    """Rows past 2^31 - 256 in one expert, where a count of its tiles no longer fits the sum of the rows
    and a tile less one."""
    import torch
    log("case: 16-bit products with one expert of 2^31 - 100 rows")
    t, M = torch.bfloat16, (1 << 31) - 100
    rows = torch.cat([torch.arange(0, 50), torch.arange(1 << 30, (1 << 30) + 50), torch.arange(M - 300, M)]).cuda()
    a = torch.zeros(M, 8, dtype=t, device="cuda")
    a[rows] = torch.randn(len(rows), 8, device="cuda").to(t)
    w, sz = torch.randn(2, 8, 8, device="cuda").to(t), torch.tensor([0, M], dtype=torch.int32, device="cuda")
    x = a[rows]
    out = torch.empty(M, 8, dtype=t, device="cuda")
    n = len(rows)
    ref, mag = _ref(x, w, [0, n], "forward")
    for path in (0, 4, 5):
        out.fill_(float("nan"))
        geg.grouped_gemm(a, sz, w, out=out, opts=geg.Opts(path, 0), check_errors=True)
        _check(out[rows], ref, mag, 8, f"forward path {path}")
    ref, mag = _ref(x, w, [0, n], "dgrad")
    for path in (0, 5):
        out.fill_(float("nan"))
        geg.grouped_dgrad(a, sz, w, dx=out, opts=geg.Opts(path, 0), check_errors=True)
        _check(out[rows], ref, mag, 8, f"dgrad path {path}")
    # the zeros between are exact; the three blocks of rows pass at most 20 instructions and 8 pieces
    _check(geg.grouped_wgrad(a, out, sz, dtype=torch.float32, check_errors=True), *_ref(x, out[rows], [0, n], "wgrad"), 28 * 32,
           "wgrad")


def _pieces(seed):
    """One expert, few tiles and a contraction of 8192."""
    return _case("bf16", [64], 256, 8192, seed=seed)


def test_pieces_are_chosen_by_the_sizes(geg):
    log("case: 16-bit products, which kernels the sizes choose")
    # tiles in eight and in four pieces, two launches; where two is the most, few rows go to the narrow kernel
    for M, N, path, launches in ((3, 256, 0, 2), (64, 256, 0, 2), (3, 4096, 0, 2), (3, 8192, 0, 1), (64, 256, 4, 1)):
        a, _, w, sz = _case("bf16", [M], N, 8192, seed=M)
        geg.grouped_gemm(a, sz, w)   # (a workspace that grows is a launch)
        before = geg.geg_launch_count()
        got = geg.grouped_gemm(a, sz, w, opts=geg.Opts(path, 0))
        assert geg.geg_launch_count() - before == launches
        _check(got, *_ref(a, w, [M], "forward"), 8192, f"{M} rows, {N} columns, path {path}")


def test_pieces_without_room_for_them(geg):
    """A workspace of the error word alone: whole tiles, as documented."""
    import ctypes
    import torch
    log("case: 16-bit products, a workspace too small for the pieces")
    a, dy, w, sz = _pieces(3)
    need = geg.lib().geg_grouped_workspace_bytes(0, 64, 256, 8192, 1)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    ref = _ref(a, w, [64], "forward")
    for nbytes in (256, need - 1, need):
        ws = torch.zeros(max(nbytes, 512) + 256, dtype=torch.uint8, device="cuda")
        ws[nbytes:] = 7
        out = torch.empty(64, 256, dtype=a.dtype, device="cuda")
        before = geg.geg_launch_count()
        assert geg.lib().geg_grouped_gemm(a.data_ptr(), sz.data_ptr(), w.data_ptr(), out.data_ptr(), 0, 64, 256, 8192, 1, 0,
                                          ws.data_ptr(), nbytes, None, stream) == 0
        assert geg.geg_launch_count() - before == (2 if nbytes == need else 1)
        _check(out, *ref, 8192, f"{nbytes} bytes")
        assert (ws[nbytes:] == 7).all()


def test_pieces_captured_and_on_streams_at_once(geg):
    """The sums of the pieces stand in a workspace between two launches."""
    import torch
    log("case: 16-bit products in pieces, captured and on two streams")
    a, _, w, sz = _pieces(1)
    ga, dy, gw, gsz = _case("bf16", [5000], 128, 136, seed=2)      # the weights' gradient in pieces
    _, da, dw, dsz = _case("bf16", [60], 4096, 136, seed=3)        # the activations' gradient in pieces

    def step():
        return geg.grouped_gemm(a, sz, w), geg.grouped_wgrad(dy, ga, gsz), geg.grouped_dgrad(da, dsz, dw)
    step()
    before = geg.geg_launch_count()
    step()
    assert geg.geg_launch_count() - before == 6
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in range(3):
        a.copy_(_pieces(10 + seed)[0])
        ga.copy_(_case("bf16", [5000], 128, 136, seed=20 + seed)[0])
        da.copy_(_case("bf16", [60], 4096, 136, seed=30 + seed)[1])
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
    others = [_pieces(40 + i)[0] for i in range(2)]
    want = [geg.grouped_gemm(o, sz, w) for o in others]
    streams = [torch.cuda.Stream() for _ in others]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(geg.grouped_gemm(others[i], sz, w))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])

"""The router's gate, its gradient and the combine's gradient against fp64 references
and against differences."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}


def _reference(logits, k, renorm):
    """(weights, ids, p over all experts) of fp64 logits, ties to the lower index."""
    l = np.where(np.isnan(logits), -np.inf, logits)
    ids = np.argsort(-l, axis=1, kind="stable")[:, :k]
    m = l.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.where(m == -np.inf, 0.0, np.where(l == m, 1.0, np.exp(l - m)))
    p = e / np.maximum(e.sum(1, keepdims=True), 1e-300)
    w = np.take_along_axis(p, ids, 1)
    if renorm:
        w = w / np.maximum(w.sum(1, keepdims=True), 1e-300)
    return w, ids, p


def _logits(T, E, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + 7 * T + E)
    return (torch.randn(T, E, generator=g) * 2).to(TYPES[dtype])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (5, 8, 8), (64, 128, 8), (33, 63, 4), (7, 65, 1), (130, 200, 6),
                                   (9, 512, 10), (3, 1000, 64), (2, 1024, 16), (1, 1, 1)])
def test_top_k_and_weights(T, E, k, renorm, dtype):
    import grouped_expert_gemm_amd as geg
    l = _logits(T, E, dtype)
    w, ids = geg.route_topk(l.cuda(), k, renormalize=renorm)
    rw, rids, _ = _reference(l.double().numpy(), k, renorm)
    assert np.array_equal(ids.cpu().numpy(), rids)
    # fp32: the exponent's argument (2^-24 of |l - m| <= 32), expf and the quotient (a few
    # 2^-24 each) and the sum of E terms
    tol = (32 + E + 8) * 2.0 ** -24
    assert np.all(np.abs(w.double().cpu().numpy() - rw) <= tol * rw + 1e-38)


@pytest.mark.parametrize("renorm", [True, False])
def test_ties_infinities_and_nan(renorm):
    import grouped_expert_gemm_amd as geg
    inf, nan = float("inf"), float("nan")
    low = torch.finfo(torch.float32).min
    rows = [[1.0] * 8, [0.0, -0.0, 0.0, -0.0, -1, -1, -1, -1], [-inf] * 8, [-inf, 2.0, -inf, -inf, -inf, 1.0, -inf, -inf],
            [low] * 8, [low, 0.0, low, low, low, low, low, low], [nan, 3.0, nan, 1.0, 2.0, 0.0, -1.0, nan],
            [inf, 0.0, inf, 1.0, 0.0, 0.0, 0.0, 0.0], [nan] * 8]
    l = torch.tensor(rows)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    w, ids = geg.route_topk(l.cuda(), 4, renormalize=renorm, error_word=err)
    rw, rids, _ = _reference(l.double().numpy(), 4, renorm)
    assert np.array_equal(ids.cpu().numpy(), rids)
    assert np.allclose(w.double().cpu().numpy(), rw, rtol=64 * 2.0 ** -24, atol=0)
    assert int(err.item()) == geg.DEVERR_NON_FINITE
    err.zero_()
    geg.route_topk(l[:6].cuda(), 4, renormalize=renorm, error_word=err)   # -inf alone is no error
    assert int(err.item()) == 0


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (64, 128, 8), (5, 300, 7), (3, 1024, 16), (4, 5, 1)])
def test_gate_gradient(T, E, k, renorm, dtype):
    import grouped_expert_gemm_amd as geg
    l = _logits(T, E, dtype)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(1))
    w, ids = geg.route_topk(l.cuda(), k, renormalize=renorm)
    got = geg.route_topk_grad(dw.cuda(), l.cuda(), ids, w, renormalize=renorm)
    assert got.dtype == l.dtype and got.shape == l.shape
    rw, rids, p = _reference(l.double().numpy(), k, renorm)
    d = dw.double().numpy()
    S = (rw * d).sum(1, keepdims=True)
    ref = np.zeros((T, E)) if renorm else -p * S
    mag = np.zeros((T, E)) if renorm else p * (rw * np.abs(d)).sum(1, keepdims=True)
    own = rw * (d - S) if renorm else rw * d
    for s in range(k):
        ref[np.arange(T), rids[:, s]] += own[:, s]
        mag[np.arange(T), rids[:, s]] += rw[:, s] * (np.abs(d[:, s]) + (rw * np.abs(d)).sum(1))
    # the result's rounding, and the fp32 weights' error (test above) on every term
    tol = HALF_STEP[dtype] * np.abs(ref) + (32 + E + 2 * k + 16) * 2.0 ** -24 * mag
    # results below fp16's normal range lie on its 2^-24 grid
    tol = tol + (2.0 ** -25 if dtype == "fp16" else 1e-38)
    assert np.all(np.abs(got.double().cpu().numpy() - ref) <= tol)


@pytest.mark.parametrize("renorm", [True, False])
def test_gate_gradient_against_differences(renorm):
    import grouped_expert_gemm_amd as geg
    T, E, k = 3, 12, 4
    l = _logits(T, E, "fp32", 5).double().numpy()
    c = np.random.default_rng(0).standard_normal((T, k))
    _, ids, _ = _reference(l, k, renorm)

    def loss(v):   # the chosen experts stay the chosen ones for small steps
        e = np.exp(v - v.max(1, keepdims=True))
        w = np.take_along_axis(e, ids, 1) / e.sum(1, keepdims=True)
        return float((c * (w / w.sum(1, keepdims=True) if renorm else w)).sum())

    ref = np.zeros_like(l)
    for i in range(T):
        for j in range(E):
            h = np.zeros_like(l)
            h[i, j] = 1e-6
            ref[i, j] = (loss(l + h) - loss(l - h)) / 2e-6
    lt = torch.tensor(l, dtype=torch.float32, device="cuda", requires_grad=True)
    w, got_ids = geg.router_gate(lt, k, renorm)
    assert np.array_equal(got_ids.cpu().numpy(), ids)
    (w * torch.tensor(c, dtype=torch.float32, device="cuda")).sum().backward()
    # central differences of step 1e-6 in fp64: 1e-9; fp32 logits and arithmetic: 1e-6
    assert np.allclose(lt.grad.double().cpu().numpy(), ref, atol=4e-6)


@pytest.mark.parametrize("T,k,N,E", [(1, 1, 8, 4), (3, 2, 24, 4), (17, 8, 2048, 16), (5, 4, 2880, 8), (64, 6, 520, 128)])
def test_combine_gradient(T, k, N, E):
    import grouped_expert_gemm_amd as geg
    g = torch.Generator().manual_seed(T * N)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    _, row_of, src_of, _ = geg.route_sort(ids.cuda(), E)
    y = torch.randn(T * k, N, generator=g).to(torch.bfloat16)
    dout = torch.randn(T, N, generator=g).to(torch.bfloat16)
    w = torch.rand(T, k, generator=g)
    dy, dw = geg.route_combine_grad(dout.cuda(), y.cuda(), row_of, w.cuda(), src_of)
    r = row_of.cpu().long().reshape(T, k)
    yd, dd = y.double()[r], dout.double()[:, None, :]
    ref_dw, mag = (yd * dd).sum(-1), (yd * dd).abs().sum(-1)
    assert bool(((dw.double().cpu() - ref_dw).abs() <= (N / 64 + 8) * 2.0 ** -24 * mag).all())
    ref_dy = torch.empty(T * k, N, dtype=torch.float64)
    ref_dy[r.flatten()] = (w.double()[..., None] * dd).reshape(T * k, N)
    # one fp32 product, then bf16: half a step of each
    assert bool(((dy.double().cpu() - ref_dy).abs() <= (2.0 ** -8 + 2.0 ** -23) * ref_dy.abs() + 1e-38).all())


def test_dropped_entries_and_untouched_rows():
    import grouped_expert_gemm_amd as geg
    ids = torch.tensor([[0, 9], [1, -1], [2, 3]], dtype=torch.int32, device="cuda")
    _, row_of, src_of, _ = geg.route_sort(ids, 4, workspace=geg.Workspace())
    y = torch.randn(6, 64, device="cuda").to(torch.bfloat16)
    dout = torch.randn(3, 64, device="cuda").to(torch.bfloat16)
    w = torch.rand(3, 2, device="cuda")
    dy, dw = geg.route_combine_grad(dout, y, row_of, w, src_of)
    assert bool((dy[4:] == 0).all()) and dw[0, 1] == 0 and dw[1, 1] == 0
    assert bool((dw[0, 0] != 0)) and bool((dy[:4] != 0).any(1).all())
    # without src_of the rows that no entry lands on are left as they were
    L = geg.lib()
    dy2 = torch.full((6, 64), 7.0, device="cuda").to(torch.bfloat16)
    s = torch.cuda.current_stream().cuda_stream
    assert L.geg_route_combine_grad(dout.data_ptr(), None, row_of.data_ptr(), None, w.data_ptr(), 3, 2, 64,
                                    dy2.data_ptr(), None, s) == 0
    assert torch.equal(dy2[:4], dy[:4]) and bool((dy2[4:] == 7).all())


def test_an_expert_named_twice_gets_both_gradients():
    import grouped_expert_gemm_amd as geg
    l = torch.randn(2, 8, device="cuda")
    ids = torch.tensor([[3, 3], [1, 9]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 0.25], [0.5, 0.5]], device="cuda")
    dw = torch.tensor([[1.0, 2.0], [1.0, 5.0]], device="cuda")
    g = geg.route_topk_grad(dw, l, ids, w).cpu()
    # S = 0.5 + 0.5 = 1: 0.5 (1 - 1) + 0.25 (2 - 1); the id outside [0, 8) adds nothing: S = 0.5
    assert g[0].tolist() == [0, 0, 0, 0.25, 0, 0, 0, 0] and g[1].tolist() == [0, 0.25, 0, 0, 0, 0, 0, 0]


@pytest.mark.parametrize("fmt", ["nf4", "mxfp4"])
def test_a_differentiable_layer_from_logits_to_loss(fmt):
    """gate -> dispatch -> grouped gate/up -> SwiGLU -> grouped down -> combine, with the
    gradients of the tokens and of the router's logits against autograd in fp64."""
    import grouped_expert_gemm_amd as geg
    from oracle import pack as P
    T, E, k, H, I = 24, 6, 3, 128, 64
    g = torch.Generator().manual_seed(11)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    logits = torch.randn(T, E, generator=g)
    w13, w2 = torch.randn(E, 2 * I, H, generator=g) * 0.1, torch.randn(E, H, I, generator=g) * 0.1
    if fmt == "nf4":
        q13, q2 = geg.gnf4_quantize(w13.cuda()), geg.gnf4_quantize(w2.cuda())
        d13, d2 = (torch.tensor(P.dequant_nf4(c.cpu().numpy(), s.cpu().numpy())) for c, s in (q13, q2))
    else:
        q13, q2 = geg.gmxfp4_quantize(w13.cuda()), geg.gmxfp4_quantize(w2.cuda())
        d13, d2 = (torch.tensor(P.dequant_mxfp4(c.cpu().numpy(), s.cpu().numpy())) for c, s in (q13, q2))
    dout = torch.randn(T, H, generator=g).to(torch.bfloat16)

    xg, lg = x.cuda().requires_grad_(), logits.cuda().requires_grad_()
    weights, ids = geg.router_gate(lg, k)
    xs, sizes, row_of, src_of = geg.dispatch_rows(xg, ids, E)
    h = geg.grouped_linear(xs, sizes, *q13, fmt=fmt).float()
    act = (torch.nn.functional.silu(h[:, 0::2]) * h[:, 1::2]).to(torch.bfloat16)
    out = geg.combine_rows(geg.grouped_linear(act, sizes, *q2, fmt=fmt), weights, row_of, src_of)
    out.backward(dout.cuda())

    xd, ld = x.double().requires_grad_(), logits.double().requires_grad_()
    top = ids.cpu().long()
    p = torch.softmax(ld.gather(1, top), 1)
    h = torch.einsum("tknh,th->tkn", d13[top], xd)
    act = torch.nn.functional.silu(h[..., 0::2]) * h[..., 1::2]
    ref = (p[..., None] * torch.einsum("tkhi,tki->tkh", d2[top], act)).sum(1)
    ref.backward(dout.double())
    # chains of bf16 roundings: h, act and y forward, dy, dact, dh and dx backward; each at
    # most 2^-8 of its term, seven on the longest chain, in the norm over all elements
    for got, want, n in ((out, ref, 4), (xg.grad, xd.grad, 7), (lg.grad, ld.grad, 5)):
        got = got.detach().double().cpu()
        assert float((got - want).norm() / want.norm()) <= n * 2.0 ** -8


def _pipeline(geg, ops, dout):
    """Forward and backward of the routing around experts that pass their rows on."""
    logits, x = ops
    w, ids = geg.route_topk(logits, 4)
    xs, sizes, row_of, src_of = geg.dispatch_rows(x, ids, logits.shape[1])
    out = geg.route_combine(xs, row_of, w, 4)
    dy, dw = geg.route_combine_grad(dout, xs, row_of, w, src_of)
    return out, sizes, dy, geg.route_topk_grad(dw, logits, ids, w)


def _routing_case(seed, T=300, E=40, H=256):
    g = torch.Generator().manual_seed(seed)
    return ((torch.randn(T, E, generator=g).cuda(), torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()),
            torch.randn(T, H, generator=g).to(torch.bfloat16).cuda())


def test_routing_in_two_captured_graphs():
    import grouped_expert_gemm_amd as geg
    cases = [_routing_case(s) for s in range(4)]
    want = [[t.clone() for t in _pipeline(geg, *c)] for c in cases]
    held = [(tuple(t.clone() for t in c[0]), c[1].clone()) for c in cases[:2]]
    graphs, outs = [], []
    for h in held:
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(_pipeline(geg, *h))
        graphs.append(gr)
    for turn in range(4):
        for i in range(2):
            c = cases[(turn + 2 * i) % 4]
            for dst, src in zip((*held[i][0], held[i][1]), (*c[0], c[1])):
                dst.copy_(src)
            graphs[i].replay()
        _pipeline(geg, *cases[turn])   # eager work between the replays
        torch.cuda.synchronize()
        for i in range(2):
            for got, w in zip(outs[i], want[(turn + 2 * i) % 4]):
                assert torch.equal(got, w), (turn, i)


def test_routing_on_two_streams():
    import grouped_expert_gemm_amd as geg
    cases = [_routing_case(s) for s in (5, 6)]
    want = [[t.clone() for t in _pipeline(geg, *c)] for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(_pipeline(geg, *c))
    torch.cuda.synchronize()
    for i, outs in enumerate(got):
        assert all(torch.equal(g, w) for g, w in zip(outs, want[i % 2])), i
    # a stream given by hand: allocated there, usable here after a wait
    logits, s = cases[0][0][0], streams[0]
    s.wait_stream(torch.cuda.current_stream())
    w, ids = geg.route_topk(logits, 4, stream=s)
    dl = geg.route_topk_grad(torch.ones_like(w), logits, ids, w, stream=s.cuda_stream)
    torch.cuda.current_stream().wait_stream(s)
    ref, ref_ids = geg.route_topk(logits, 4)
    assert torch.equal(w, ref) and torch.equal(ids, ref_ids)
    # dw = 1 for all: w (1 - sum w) = w (1 - 1 up to four roundings of the sum and the division)
    assert float(dl.abs().max()) <= 8 * 2.0 ** -24


def test_no_second_derivative():
    import grouped_expert_gemm_amd as geg
    l = torch.randn(6, 8, device="cuda", requires_grad=True)
    w, _ = geg.router_gate(l, 2)
    g, = torch.autograd.grad((w * w).sum(), l, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.sum(), l)

"""Adapters of many requests (request_lora) against fp64.

Tolerance per element, with U = sum |x| |A| of the first product: u is summed over K (at most
32 additions inside a matrix instruction, K / 32 between them, and 40 across wavefronts and
ranges), each off by at most 2^-23 of U; it enters the second product with 16 significant bits
at least (2^-17 of |u|, or 2^-34 of its row's largest); that one's r products again (r / 8 + 32
additions of both parts); the result is rounded once, finfo.eps / 2 of its value or half a
subnormal step."""
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


def _case(dtype, M, K, N, L, r, seed, mixed=True):
    import torch
    t = _types()[dtype]
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, y = rand(M, K).to(t), rand(M, N).to(t)
    A, B = (rand(L, r, K) * K ** -0.5).to(t), rand(L, N, r).to(t)
    scales = torch.rand(L, generator=g, device="cuda") + 0.5
    ids = torch.randint(-1, L, (M,), generator=g, device="cuda").to(torch.int32)
    return y, x, ids if mixed else torch.sort(ids).values, A, B, scales


def _ref(y, x, ids, A, B, scales):
    """(result, tolerance) in fp64."""
    import torch
    K, r = x.shape[1], A.shape[1]
    out = torch.zeros(x.shape[0], B.shape[1], dtype=torch.float64, device="cuda") if y is None else y.double()
    tol = 2.0 ** -23 * out.abs()
    for i in sorted(set(ids.tolist())):
        if i < 0 or i >= A.shape[0]:
            continue
        rows = torch.nonzero(ids == i).flatten()
        s = 1.0 if scales is None else scales[i].double()
        X, At, Bt = x[rows].double(), A[i].double().t().contiguous(), B[i].double().t().contiguous()
        u, U = X @ At, X.abs() @ At.abs()
        du = (K / 32 + 72) * 2.0 ** -23 * U + 2.0 ** -17 * u.abs() + 2.0 ** -34 * u.abs().amax(1, keepdim=True)
        out[rows] += s * (u @ Bt)
        tol[rows] += s * (du @ Bt.abs() + (r / 8 + 34) * 2.0 ** -23 * (u.abs() @ Bt.abs()))
    info = torch.finfo(x.dtype)
    return out, tol + info.eps / 2 * (out.abs() + tol) + info.smallest_normal * info.eps / 2


def _check(got, ref, tol, what):
    over = ((got.double() - ref).abs() / tol).max().item() if ref.numel() else 0.0
    log(f"  {what}: largest error {over:.3f} of its bound")
    assert got.isfinite().all() and over <= 1.0, what


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,K,N,L,r,mixed", [
    (1, 8, 8, 1, 8, True), (1, 2048, 1024, 8, 16, True), (5, 264, 72, 3, 24, True), (17, 4096, 200, 40, 64, True),
    (96, 1000, 520, 32, 128, True), (300, 512, 64, 7, 40, False), (513, 136, 264, 5, 16, False), (700, 72, 136, 300, 32, True),
    (1025, 320, 328, 6, 104, False), (640, 256, 96, 4, 72, True),
    # both sides of the rule by which the units are listed; runs of work that pass from unit to
    # unit; counters of every adapter past 48 KB
    (128, 128, 776, 40, 16, True), (129, 264, 4104, 5, 64, True), (256, 72, 520, 9, 40, True), (257, 72, 520, 9, 40, True),
    (100, 64, 16392, 5, 32, True), (200, 64, 16392, 70, 128, True), (1500, 64, 2056, 3, 128, False),
    (900, 40, 16392, 2, 24, False), (20000, 8, 8, 32768, 8, True)])
def test_shapes(geg, dtype, M, K, N, L, r, mixed):
    log(f"case: request adapters {dtype} M={M} K={K} N={N} L={L} r={r} mixed={mixed}")
    args = _case(dtype, M, K, N, L, r, seed=M + K + N, mixed=mixed)
    _check(geg.request_lora(*args, check_errors=True), *_ref(*args), "out")
    y, x, ids, A, B, _ = args
    _check(geg.request_lora(None, x, ids, A, B), *_ref(None, x, ids, A, B, None), "without y and scales")


def test_rows_without_an_adapter_and_in_place(geg):
    import torch
    log("case: request adapters, rows without one")
    for M in (40, 600):
        y, x, ids, A, B, scales = _case("bf16", M, 128, 264, 4, 16, seed=1)
        y[ids < 0] = float("nan")
        bits = y[ids < 0].view(torch.int16).clone()
        out = geg.request_lora(y, x, ids, A, B, scales)
        assert torch.equal(out[ids < 0].view(torch.int16), bits)
        z = y.clone()
        assert geg.request_lora(z, x, ids, A, B, scales, out=z) is z
        assert torch.equal(z.view(torch.int16), out.view(torch.int16))
        none = torch.full_like(ids, -5)
        assert torch.equal(geg.request_lora(z, x, none, A, B, scales).view(torch.int16), z.view(torch.int16))
        assert (geg.request_lora(None, x, none, A, B, scales) == 0).all()


def test_one_adapter_and_all_different(geg):
    import torch
    log("case: request adapters, every row the same and every row another")
    for M in (128, 256, 1000):
        y, x, _, A, B, scales = _case("bf16", M, 64, 72, M, 8, seed=9)
        for ids in (torch.zeros(M), torch.arange(M), torch.arange(M).flip(0), torch.full((M,), M - 1)):
            ids = ids.to(torch.int32).cuda()
            _check(geg.request_lora(y, x, ids, A, B, scales, check_errors=True), *_ref(y, x, ids, A, B, scales), f"M={M}")


def test_ids_out_of_range(geg):
    import torch
    log("case: request adapters, ids past L")
    for M, row in ((33, 20), (128, 127), (256, 255), (300, 299)):
        y, x, ids, A, B, scales = _case("bf16", M, 64, 64, 3, 8, seed=2)
        ids[row] = 3
        with pytest.raises(geg.GegDeviceError) as e:
            geg.request_lora(y, x, ids, A, B, scales, check_errors=True)
        assert e.value.bits == geg.DEVERR_BAD_EXPERT_ID
        out = geg.request_lora(y, x, ids, A, B, scales)
        assert torch.equal(out[row], y[row])
        _check(out, *_ref(y, x, ids, A, B, scales), "the other rows")


def test_slices_of_wider_tensors(geg):
    import torch
    log("case: request adapters on slices of columns")
    for M in (1, 50, 700):
        y, x, ids, A, B, scales = _case("fp16", M, 72, 136, 6, 16, seed=3)
        wide_y, wide_x, wide_o = (torch.full((M, 400), 3.0, dtype=torch.float16, device="cuda") for _ in range(3))
        wide_y[:, 8:144], wide_x[:, 320:392] = y, x
        out = geg.request_lora(wide_y[:, 8:144], wide_x[:, 320:392], ids, A, B, scales, out=wide_o[:, 200:336])
        want = geg.request_lora(y, x, ids, A, B, scales)
        assert torch.equal(out, want)
        assert (wide_o[:, :200] == 3).all() and (wide_o[:, 336:] == 3).all()
        geg.request_lora(wide_y[:, 8:144], x, ids, A, B, scales, out=wide_y[:, 8:144])
        assert torch.equal(wide_y[:, 8:144], want) and (wide_y[:, :8] == 3).all() and (wide_y[:, 144:] == 3).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_values_stay_with_their_rows(geg, dtype):
    import torch
    log(f"case: request adapters {dtype} with infinities and NaN")
    for M in (30, 530):
        y, x, ids, A, B, scales = _case(dtype, M, 72, 72, 4, 8, seed=4)
        plain = geg.request_lora(y, x, ids, A, B, scales)
        x2 = x.clone()
        row = int(torch.nonzero(ids >= 0)[3])
        x2[row, 70] = float("nan")
        got = geg.request_lora(y, x2, ids, A, B, scales)
        assert got[row].isnan().all()
        got[row] = plain[row]
        assert torch.equal(got, plain)
        bad = int(ids[row])
        A2, B2 = A.clone(), B.clone()
        A2[bad, 7], B2[bad, 71] = float("inf"), float("nan")
        for a, b in ((A2, B), (A, B2)):
            got = geg.request_lora(y, x, ids, a, b, scales)
            assert not got[ids == bad][:, -1].isfinite().any()
            assert torch.equal(got[ids != bad], plain[ids != bad])


def test_scales_of_any_size_in_fp16(geg):
    """u far outside fp16's range, and far below it."""
    import torch
    log("case: request adapters, fp16 with large and small u")
    for factor, back in ((2.0 ** 9, 2.0 ** -14), (2.0 ** -11, 2.0 ** 10)):
        y, x, ids, A, B, scales = _case("fp16", 40, 512, 64, 3, 16, seed=5)
        x, A, B = x * factor, A * factor, B * back
        _check(geg.request_lora(y, x, ids, A, B, scales), *_ref(y, x, ids, A, B, scales), f"factor {factor}")


def test_offsets_past_2_31(geg):
    import torch
    log("case: request adapters with more than 2^31 elements of y and of the adapters")
    t = torch.bfloat16
    M, N, K = 70000, 32768, 64
    y = torch.zeros(M, N, dtype=t, device="cuda")
    x = torch.randn(M, K, device="cuda").to(t)
    A, B = torch.randn(2, 8, K, device="cuda").to(t), torch.randn(2, N, 8, device="cuda").to(t)
    ids = (torch.arange(M, device="cuda") >= M - 100).to(torch.int32)
    geg.request_lora(y, x, ids, A, B, out=y)
    at = torch.tensor([0, M - 101, M - 100, M - 1], device="cuda")
    ref, tol = _ref(None, x[at], ids[at], A, B, None)
    _check(y[at], ref, tol, "rows at both ends")
    del y
    L, r = 2100, 64
    A = torch.zeros(L, r, 16384, dtype=t, device="cuda")
    B = torch.zeros(L, 16384, r, dtype=t, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(6)
    A[L - 1] = torch.randn(r, 16384, generator=g, device="cuda") / 128
    B[L - 1] = torch.randn(16384, r, generator=g, device="cuda")
    x = torch.randn(3, 16384, generator=g, device="cuda").to(t)
    ids = torch.full((3,), L - 1, dtype=torch.int32, device="cuda")
    out = geg.request_lora(None, x, ids, A, B)
    _check(out, *_ref(None, x, torch.zeros_like(ids), A[L - 1:], B[L - 1:], None), "the last adapter")


def test_captured_and_on_streams(geg):
    import torch
    log("case: request adapters captured and on another stream")
    for M, L, r in ((24, 5, 16), (600, 5, 16), (300, 13000, 8)):
        args = _case("bf16", M, 256, 264, L, r, seed=7)
        geg.request_lora(*args)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = geg.request_lora(*args)
        for seed in range(3):
            for old, new in zip(args, _case("bf16", M, 256, 264, L, r, seed=10 + seed)):
                old.copy_(new)
            want = geg.request_lora(*args)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(got, want)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        out = geg.request_lora(*args, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(out, want)


def test_two_streams_at_once(geg):
    import torch
    log("case: request adapters on two streams at once")
    cases = [_case("bf16", 200, 2048, 512, 6, 32, seed=20 + i) for i in range(2)]
    want = [geg.request_lora(*c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(geg.request_lora(*cases[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])


def test_beside_quantised_experts(geg):
    """A decode batch through a quantised projection and through quantised experts, each request
    with its adapter, one per expert: the calls as a server makes them."""
    import torch
    log("case: request adapters beside quantised projections")
    T, k, E, H, N, P, r = 12, 2, 6, 128, 192, 3, 16
    g = torch.Generator(device="cuda").manual_seed(8)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x = rand(T, H).bfloat16()
    owner = torch.randint(-1, P, (T,), generator=g, device="cuda").to(torch.int32)
    # shared projection, E = 1
    w, am = geg.gnf4_quantize((rand(1, N, H) * 0.05))
    sizes1 = torch.tensor([T], dtype=torch.int32, device="cuda")
    A1, B1 = (rand(P, r, H) * H ** -0.5).bfloat16(), rand(P, N, r).bfloat16()
    y = geg.gnf4_grouped_gemm(x, sizes1, w, am)
    _check(geg.request_lora(y, x, owner, A1, B1), *_ref(y, x, owner, A1, B1, None), "shared projection")
    # routed experts: row r of the sorted rows belongs to token src_of[r] // k and its expert
    wE, amE = geg.gnf4_quantize((rand(E, N, H) * 0.05))
    weights, ids = geg.route_topk(rand(T, E), k)
    sizes, row_of, src_of, xs = geg.route_sort(ids, E, x)
    h = geg.gnf4_grouped_gemm(xs, sizes, wE, amE)
    expert = ids.flatten()[src_of.long()]
    own = owner[(src_of // k).long()]
    rows = torch.where(own < 0, -1, own * E + expert).to(torch.int32)
    AE, BE = (rand(P * E, r, H) * H ** -0.5).bfloat16(), rand(P * E, N, r).bfloat16()
    _check(geg.request_lora(h, xs, rows, AE, BE), *_ref(h, xs, rows, AE, BE, None), "routed experts")


def _by_element(y, x, ids, A, B):
    """The result in fp64, summed element by element: infinities and NaN go where the definition has them."""
    import torch
    out = y.double()
    for i in range(A.shape[0]):
        rows = torch.nonzero(ids == i).flatten()
        u = (x[rows].double()[:, None, :] * A[i].double()[None]).sum(-1)
        out[rows] += (u[:, None, :] * B[i].double()[None]).sum(-1)
    return out


def _same_places(got, ref, tol, what):
    """Infinities and NaN in the same places, the rest within the bound."""
    import torch
    got = got.double()
    big = ref.abs().isinf()
    log(f"  {what}: {int(big.sum())} infinities, {int(ref.isnan().sum())} NaN of {ref.numel()}")
    assert torch.equal(got.isnan(), ref.isnan()), what
    assert torch.equal(got[big], ref[big]), what
    rest = ref.isfinite()
    assert ((got - ref).abs() <= tol)[rest].all(), what


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("r", [8, 16, 24, 64, 128])
@pytest.mark.parametrize("M", [30, 530])
def test_an_infinity_in_an_adapter(geg, dtype, r, M):
    """u times an infinity is an infinity of u's sign, whatever u's low bits are; a row of u with an
    infinity keeps its other values."""
    import torch
    log(f"case: request adapters {dtype} rank {r}, {M} rows, infinities in an adapter")
    inf = float("inf")
    y, x, ids, A, B, _ = _case(dtype, M, 72, 136, 3, r, seed=r + M)
    ids = ids.clamp(min=0)
    exact = x.clone()
    exact[:, 1:] = 0      # u = x[:, 0] A[:, 0]: with A = 1 there, few bits and no second part
    exact[:, 0] = torch.where(exact[:, 0] == 0, 1, exact[:, 0])
    ones = A.clone()
    ones[:, :, 0] = 1
    for name, x1, A1 in (("u of few bits", exact, ones), ("u of many bits", x, A)):
        B1 = B.clone()
        B1[0, 5, 3], B1[0, 70, 0], B1[1, 135, r - 1] = inf, -inf, inf
        B1[2, 9, 1], B1[2, 9, 2], B1[2, 64, 4] = inf, -inf, float("nan")
        clean = torch.where(B1.isfinite(), B1, torch.zeros_like(B1))
        _, tol = _ref(y, x1, ids, A1, clean, None)
        _same_places(geg.request_lora(y, x1, ids, A1, B1), _by_element(y, x1, ids, A1, B1), tol, name)
    zero = exact.clone()
    zero[::2] = 0         # u = 0: times an infinity NaN
    ref = _by_element(y, zero, ids, ones, B1)
    assert ref[(ids == 0)][:, 5].isnan().any()
    _, tol = _ref(y, zero, ids, ones, clean, None)
    _same_places(geg.request_lora(y, zero, ids, ones, B1), ref, tol, "u of zeros")
    # u with an infinity and values past 65504 of either sign
    big, wide = A.clone(), x * 2.0 ** 6
    big[:, 1:] *= 2.0 ** 12
    big[1, 0, 3] = inf
    small = B * 2.0 ** -12
    ref = _by_element(y, wide, ids, big, small)
    assert ref[ids == 1].isinf().all()
    _, tol = _ref(y, wide, ids, torch.where(big.isfinite(), big, torch.zeros_like(big)), small, None)
    _same_places(geg.request_lora(y, wide, ids, big, small), ref, tol, "an infinity in u")


def test_captured_with_many_adapters(geg):
    """Counters of every adapter past the launch's usual LDS, in a captured call."""
    import torch
    log("case: request adapters, 20000 adapters captured")
    y, x, ids, A, B, scales = _case("bf16", 700, 40, 72, 20000, 8, seed=12)
    geg.request_lora(y, x, ids, A, B, scales)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = geg.request_lora(y, x, ids, A, B, scales)
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        ids.copy_(torch.randint(-1, 20000 >> (6 * seed), (700,), generator=g, device="cuda"))
        want = geg.request_lora(y, x, ids, A, B, scales)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        _check(got, *_ref(y, x, ids, A, B, scales), f"replay {seed}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("below", [0, 11, 25, 30])
def test_how_exactly_u_is_kept(geg, dtype, below):
    """One value of u 2^-below of its row's largest, whose column of B is zero: in bf16 within 2^-17 of
    itself, in fp16 within 2^-22 of itself or 2^-35 of the largest; the output's rounding comes on top."""
    import torch
    log(f"case: request adapters {dtype}, u at 2^-{below} of its row's largest")
    t, N, K = _types()[dtype], 72, 8
    for M in (20, 400):
        g = torch.Generator(device="cuda").manual_seed(below)
        x, A, B = torch.zeros(M, K, device="cuda"), torch.zeros(1, 8, K, device="cuda"), torch.zeros(1, N, 8, device="cuda")
        x[:, 0], x[:, 1] = torch.rand(M, generator=g, device="cuda") + 1, 1
        A[0, 0, 1], A[0, 3, 0] = 2.0 ** 14, 1.3125 * 2.0 ** (14 - below)
        B[0, :, 3] = (torch.rand(N, generator=g, device="cuda") + 1) * 2.0 ** (below - 16)   # below 2^15
        x, A, B = x.to(t), A.to(t), B.to(t)
        u = x[:, :1].double() * A[0, 3, 0].double()      # exact in fp32: two 16-bit values
        kept = 2.0 ** -17 * u if dtype == "bf16" else torch.maximum(2.0 ** -22 * u, torch.full_like(u, 2.0 ** -35 * 2.0 ** 14))
        ref = u * B[0, :, 3].double()
        tol = kept * B[0, :, 3].double() + 2.0 ** -23 * ref
        got = geg.request_lora(None, x, torch.zeros(M, dtype=torch.int32, device="cuda"), A, B)
        _check(got, ref, tol + torch.finfo(t).eps / 2 * (ref + tol), f"{M} rows")

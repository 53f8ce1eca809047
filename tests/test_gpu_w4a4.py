"""The W4A4 grouped GEMM against the fp64 product of the oracle's quantised operands."""
import numpy as np
import pytest

from oracle import pack as P

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TILES, NARROW = 2, 4


def _case(sizes, N, K, seed=0, extra=0):
    rng = np.random.default_rng([seed, N, K, len(sizes)])
    M, E = int(sum(sizes)) + extra, len(sizes)
    return {"a": torch.tensor(rng.standard_normal((M, K)), dtype=torch.float32).to(torch.bfloat16),
            "sizes": torch.tensor(sizes, dtype=torch.int32),
            "w": rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8),
            "s": rng.integers(116, 124, (E, N, K // 32), dtype=np.uint8)}


def _call(c, path=0, out=None, workspace=None, cu_limit=0, **kw):
    import grouped_expert_gemm_amd as geg
    return geg.gmxfp4_w4a4_grouped_gemm(c["a"].cuda(), c["sizes"].cuda(), torch.tensor(c["w"]).cuda(),
                                        torch.tensor(c["s"]).cuda(), out=out, workspace=workspace,
                                        opts=geg.Opts(force_path=path, cu_limit=cu_limit), **kw)


def _reference(c):
    """(out, allowed error) in fp64: bf16 result 2^-8; the instruction keeps about 12 bits below
    the largest product of its 128-wide sum, 2^-11 of the largest |a w| per step, and the fp32
    sums K 2^-24 of their magnitudes."""
    a = P.dequant_mxfp4(*P.quantize_pack_mxfp4(c["a"].float().numpy()))
    N, K = c["w"].shape[1], a.shape[1]
    out, tol, r = np.zeros((len(a), N)), np.zeros((len(a), N)), 0
    for e, n in enumerate(c["sizes"].tolist()):
        if n == 0:
            continue
        w = P.dequant_mxfp4(c["w"][e], c["s"][e])
        out[r:r + n] = a[r:r + n] @ w.T
        tol[r:r + n] = K * 2.0 ** -24 * (np.abs(a[r:r + n]) @ np.abs(w).T)
        for k in range(0, K, 128):
            big = np.abs(a[r:r + n, None, k:k + 128] * w[None, :, k:k + 128]).max(-1)
            tol[r:r + n] += 2.0 ** -11 * big
        r += n
    return out, tol + 2.0 ** -8 * np.abs(out), r


def _check(c, path, **kw):
    got = _call(c, path, **kw).double().cpu().numpy()
    ref, tol, r = _reference(c)
    worst = float(np.max(np.abs(got[:r] - ref[:r]) / np.maximum(tol[:r], 1e-300))) if r else 0.0
    print(f"  path {path} M={len(got)} N={got.shape[1]} K={c['a'].shape[1]}: {worst:.3f} of the allowed error", flush=True)
    assert np.all(np.isfinite(got[:r])) and worst <= 1.0
    return got


SHAPES = [([1], 16, 32), ([3, 0, 2], 48, 64), ([1, 1, 1, 1], 320, 2880), ([17, 5, 0, 33], 64, 160), ([16, 32, 1], 1, 96),
          ([2, 7], 23, 512), ([9, 40], 130, 544), ([70, 0, 3], 272, 1024), ([5], 36, 4320),
          ([1, 0, 0, 2, 0], 50, 96), ([0, 3, 0, 0], 33, 1056)]


@pytest.mark.parametrize("path", [0, TILES, NARROW])
@pytest.mark.parametrize("sizes,N,K", SHAPES)
def test_product_matches_fp64(sizes, N, K, path):
    _check(_case(sizes, N, K), path)


@pytest.mark.parametrize("K", list(range(32, 1216, 32)))
def test_every_contraction_tail_of_the_tiles(K):
    # steps of 128, pieces of 512, pairs of pieces, and every remainder of each
    _check(_case([5, 20], 40, K), TILES)


@pytest.mark.parametrize("K", list(range(32, 1216, 32)))
def test_every_contraction_tail_of_the_narrow_kernel(K):
    # rows quantised by the kernel itself (no more rows than experts), and before it
    _check(_case([2, 0, 0], 20, K), NARROW)
    _check(_case([5, 20], 40, K), NARROW)


@pytest.mark.parametrize("sizes,N,K", [([300, 129, 0, 256, 7, 257], 264, 352), ([513], 513, 640), ([128, 127], 255, 256)])
def test_tiles_past_one_block_of_rows_and_columns(sizes, N, K):
    c = _case(sizes, N, K)
    got = _check(c, TILES)
    # few workgroups: several tiles each, the same bits
    assert np.array_equal(_call(c, TILES, cu_limit=2).double().cpu().numpy(), got)
    narrow = _check(c, NARROW)
    assert np.array_equal(_call(c, NARROW, cu_limit=1).double().cpu().numpy(), narrow)


def test_exact_integers_bit_for_bit():
    # codes of small integers, scales 1: every sum is an integer below 2^8, exact in bf16
    rng = np.random.default_rng(3)
    vals = np.array([0, 0, 1, 2, -1, -2], dtype=np.float32)
    a = vals[rng.integers(0, 6, (40, 256))]
    a[:, ::32] = 4.0                                     # amax 4: scale 2^0
    w = vals[rng.integers(0, 6, (2, 64, 256))] * (rng.random((2, 64, 256)) < 0.1)
    w[:, :, 1::32] = 4.0
    wb, ws = P.quantize_pack_mxfp4(w)
    c = {"a": torch.tensor(a).to(torch.bfloat16), "sizes": torch.tensor([25, 15], dtype=torch.int32),
         "w": wb.reshape(2, 64, 128), "s": ws}
    ref = np.concatenate([a[:25] @ w[0].T, a[25:] @ w[1].T])
    ref = torch.tensor(ref, dtype=torch.float32).to(torch.bfloat16)
    for path in (TILES, NARROW):
        assert torch.equal(_call(c, path).cpu(), ref)


@pytest.mark.parametrize("path", [TILES, NARROW])
def test_rows_past_the_last_expert_and_neighbours_stay(path):
    c = _case([9, 0, 30], 72, 288, extra=4)
    M = c["a"].shape[0]
    buf = torch.full((M + 2, 72), 5.0, dtype=torch.bfloat16, device="cuda")
    _call(c, path, out=buf[1:M + 1])
    assert bool((buf[0] == 5).all()) and bool((buf[M - 3:] == 5).all())
    assert torch.equal(buf[1:M - 3], _call(c, path)[:M - 4])


@pytest.mark.parametrize("path", [TILES, NARROW])
def test_bad_sizes_are_clamped_and_flagged(path):
    import grouped_expert_gemm_amd as geg
    c = _case([4, 6], 32, 64)
    c["sizes"] = torch.tensor([-3, 40], dtype=torch.int32)
    ws = geg.Workspace()
    got = _call(c, path, workspace=ws)
    assert ws.read_error() == geg.DEVERR_NEGATIVE_SIZE | geg.DEVERR_SIZES_EXCEED_M
    c["sizes"] = torch.tensor([0, 10], dtype=torch.int32)
    assert torch.equal(got, _call(c, path))


@pytest.mark.parametrize("path", [TILES, NARROW])
def test_a_row_with_nan_is_nan_and_flagged_the_others_unchanged(path):
    import grouped_expert_gemm_amd as geg
    c = _case([20, 3], 40, 160)
    ref = _call(c, path)
    c["a"][7, 159], c["a"][21, 0] = float("nan"), float("inf")
    ws = geg.Workspace()
    got = _call(c, path, workspace=ws)
    assert ws.read_error() == geg.DEVERR_NON_FINITE
    bad = torch.zeros(23, dtype=torch.bool)
    bad[[7, 21]] = True
    few = _case([2, 0, 0], 40, 160)        # no more rows than experts
    few["a"][1, 33] = float("nan")
    ws.reset()
    one = _call(few, path, workspace=ws)
    assert ws.read_error() == geg.DEVERR_NON_FINITE and bool(one[1].isnan().all()) and not bool(one[0].isnan().any())
    assert bool(got[bad.cuda()].isnan().all()) and torch.equal(got[~bad.cuda()], ref[~bad.cuda()])


@pytest.mark.parametrize("path", [TILES, NARROW])
def test_a_nan_weight_scale_reaches_its_column_only(path):
    c = _case([20, 3], 40, 160)
    ref = _call(c, path)
    c["s"][0, 39, 4] = 255
    got = _call(c, path)
    assert bool(got[:20, 39].isnan().all()) and torch.equal(got[:20, :39], ref[:20, :39]) and torch.equal(got[20:], ref[20:])


@pytest.mark.parametrize("path", [TILES, NARROW])
def test_streams_and_captured_graphs(path):
    import grouped_expert_gemm_amd as geg
    c, c2 = _case([20, 3, 9], 136, 320), _case([5, 50], 64, 512, seed=1)
    o = geg.Opts(force_path=path)
    up = [[v.cuda() if torch.is_tensor(v) else torch.tensor(v).cuda() for v in (d["a"], d["sizes"], d["w"], d["s"])]
          for d in (c, c2)]
    f = geg.gmxfp4_w4a4_grouped_gemm
    r1, r2 = f(*up[0], opts=o), f(*up[1], opts=o)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [(f(*up[0], opts=o, stream=s1), f(*up[1], opts=o, stream=s2)) for _ in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, r1) and torch.equal(y, r2) for x, y in outs)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        o1 = f(*up[0], opts=o)
    with torch.cuda.graph(g2):
        o2 = f(*up[1], opts=o)
    for _ in range(4):
        up[0][0].copy_(torch.randn_like(up[0][0]))
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(o1, f(*up[0], opts=o)) and torch.equal(o2, r2)


def test_empty_batch_and_no_experts_with_rows():
    c = _case([0, 0], 32, 64)
    assert _call(c).shape == (0, 32)
    c = _case([0, 0], 32, 64, extra=3)
    buf = torch.full((3, 32), 2.0, dtype=torch.bfloat16, device="cuda")
    for path in (TILES, NARROW):
        _call(c, path, out=buf)
        assert bool((buf == 2).all())


def test_quantised_values_through_the_plain_mxfp4_gemm_agree():
    """The packer's values fed to the bf16 x MXFP4 GEMM give the W4A4 product."""
    import grouped_expert_gemm_amd as geg
    c = _case([60, 4, 0, 36], 96, 512)
    _, _, values = geg.gmxfp4_quantize(c["a"].cuda(), values=True)
    d = [c["sizes"].cuda(), torch.tensor(c["w"]).cuda(), torch.tensor(c["s"]).cuda()]
    ref = geg.gmxfp4_grouped_gemm(values, *d).double().cpu().numpy()
    _, tol, _ = _reference(c)
    for path in (0, TILES, NARROW):
        # two roundings to bf16 and the sums of both
        assert np.all(np.abs(_call(c, path).double().cpu().numpy() - ref) <= 2 * tol)


@pytest.mark.parametrize("N,K", [(64, 288), (71, 2080), (256, 512)])
@pytest.mark.parametrize("path", [TILES, NARROW])
def test_scales_at_any_byte_and_an_output_at_any_pair(path, N, K):
    import grouped_expert_gemm_amd as geg
    c = _case([4, 0, 21], N, K)
    want = _check(c, path)
    M, n = len(want), c["s"].size
    for shift in (1, 2, 3, 7):
        s = torch.zeros(n + shift, dtype=torch.uint8, device="cuda")[shift:].view(c["s"].shape)
        s.copy_(torch.tensor(c["s"]))
        buf = torch.full((M * N + 2 * shift + 2,), 5.0, dtype=torch.bfloat16, device="cuda")
        out = buf[2 * shift:2 * shift + M * N].view(M, N)
        geg.gmxfp4_w4a4_grouped_gemm(c["a"].cuda(), c["sizes"].cuda(), torch.tensor(c["w"]).cuda(), s, out=out,
                                     opts=geg.Opts(path, 0))
        assert np.array_equal(out.double().cpu().numpy(), want), shift
        assert bool((buf[:2 * shift] == 5).all()) and bool((buf[-2:] == 5).all())


@pytest.mark.parametrize("path", [TILES, NARROW])
def test_many_experts_few_of_them_with_rows(path):
    sizes = np.zeros(1024, int)
    sizes[[0, 3, 511, 1023]] = 2, 19, 1, 5
    c = _case(sizes.tolist(), 40, 320)
    got = _check(c, path)
    assert np.array_equal(_call(c, path, cu_limit=1).double().cpu().numpy(), got)


@pytest.mark.parametrize("path", [0, TILES, NARROW])
@pytest.mark.parametrize("sizes,extra", [([20, 3], 5), ([1, 0, 0, 0, 0, 0, 0, 0], 4), ([3, -2, 9], 40)])
def test_nan_rows_that_no_expert_owns_are_not_flagged(path, sizes, extra):
    import grouped_expert_gemm_amd as geg
    c = _case([max(n, 0) for n in sizes], 40, 160, extra=extra)
    c["sizes"] = torch.tensor(sizes, dtype=torch.int32)
    negative = geg.DEVERR_NEGATIVE_SIZE if min(sizes) < 0 else 0
    c["a"][-extra:] = float("nan")
    ws = geg.Workspace()
    got = _call(c, path, workspace=ws)
    rows = len(c["a"]) - extra
    assert ws.read_error() == negative and bool(got[:rows].isfinite().all())
    c["a"][rows - 1, 159] = float("inf")      # the last row that one owns
    got = _call(c, path, workspace=ws)
    assert ws.read_error() == negative | geg.DEVERR_NON_FINITE and bool(got[rows - 1].isnan().all())

"""MXFP4 quantisation on the GPU, bit for bit against the oracle's packer (fp64)."""
import numpy as np
import pytest

from oracle import pack as P

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _check(x, what):
    """codes, scales and values of the tensor x (any type) against the oracle."""
    import grouped_expert_gemm_amd as geg
    codes, scales, values = geg.gmxfp4_quantize(x.cuda(), values=True)
    plain = geg.gmxfp4_quantize(x.cuda())
    assert torch.equal(plain[0], codes) and torch.equal(plain[1], scales)
    assert values.dtype == x.dtype and values.shape == x.shape
    ref_b, ref_s = P.quantize_pack_mxfp4(x.float().numpy())
    assert np.array_equal(scales.cpu().numpy(), ref_s), f"{what}: scales"
    assert np.array_equal(codes.cpu().numpy().reshape(ref_b.shape), ref_b), f"{what}: codes"
    # the values the codes stand for are exact in every type
    ref_v = P.dequant_mxfp4(ref_b, ref_s)
    assert np.array_equal(values.double().cpu().numpy(), ref_v), f"{what}: values"


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (4, 2880), (257, 2048), (1, 14336), (2100, 2880)])
def test_codes_scales_and_values(dtype, rows, K):
    g = torch.Generator().manual_seed(rows * K)
    x = torch.randn(rows, K, generator=g) * torch.exp(torch.randn(K, generator=g))
    _check(x.to(TYPES[dtype]), f"{dtype} {rows}x{K}")


@pytest.mark.parametrize("dtype", list(TYPES))
def test_ties_saturation_zeros_and_signs(dtype):
    # every midpoint and its neighbours at several scales, blocks led by an amax just
    # below 8 (saturates), all zeros, negative values that round to -0
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    blocks = []
    for lead in (4.0, 6.0, 7.75, 7.0):
        v = [lead] + [s * m * f for m in mids for s in (1, -1) for f in (1.0, 1.015625)] + [-0.0, 0.1, -0.1]
        blocks.append((v + [0.0] * 32)[:32])
    b = torch.tensor(blocks)
    x = torch.cat([b * 2.0 ** e for e in (-10, 0, 3)] + [torch.zeros(2, 32), -torch.zeros(1, 32)])
    _check(x.to(TYPES[dtype]), f"ties {dtype}")


@pytest.mark.parametrize("dtype", list(TYPES))
def test_smallest_and_largest_magnitudes(dtype):
    # blocks whose amax runs over the type's whole range, subnormals included
    t = TYPES[dtype]
    g = torch.Generator().manual_seed(3)
    lo, hi = {"bf16": (-133, 127), "fp16": (-24, 15), "fp32": (-149, 127)}[dtype]
    e = torch.arange(lo, hi + 1).double()
    x = (torch.rand(len(e), 32, generator=g).double() * 2 - 1) * (2.0 ** e)[:, None]
    x[:, 0] = (2.0 ** e)
    _check(x.to(torch.float32).to(t), f"range {dtype}")


@pytest.mark.parametrize("dtype", list(TYPES))
def test_every_bf16_and_fp16_bit_pattern(dtype):
    # every finite 16-bit pattern as an element beside a fixed amax (fp32: bf16's)
    t = TYPES[dtype]
    if dtype == "fp16":
        v = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(torch.float16)
    else:
        v = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = v[torch.isfinite(v)].float()
    v = v[v.abs() <= 8.0]
    v = torch.cat([v, torch.zeros(-len(v) % 31)]).reshape(-1, 31)
    x = torch.cat([torch.full((len(v), 1), 7.0), v], 1)
    _check(x.to(t), f"patterns {dtype}")


def test_a_block_with_inf_or_nan_decodes_to_nan_and_leaves_its_neighbours():
    import grouped_expert_gemm_amd as geg
    for dtype, t in TYPES.items():
        x = torch.ones(2, 96, dtype=t)
        x[0, 40], x[1, 0] = float("inf"), float("nan")
        codes, scales, values = geg.gmxfp4_quantize(x.cuda(), values=True)
        bad = torch.tensor([[False, True, False], [True, False, False]])
        assert torch.equal((scales.cpu() == 255), bad)
        assert torch.equal(values.cpu().float().isnan().reshape(2, 3, 32).all(-1), bad)
        assert torch.equal(values.cpu().float().reshape(2, 3, 32)[~bad], torch.ones(4, 32))
        f32 = geg.gmxfp4_dequant(codes.reshape(1, 2, 48), scales.reshape(1, 2, 3))[0]
        assert torch.equal(f32.cpu()[0].isnan().reshape(2, 3, 32).all(-1), bad)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_row_pitch_and_leading_dimensions(dtype):
    import grouped_expert_gemm_amd as geg
    big = torch.randn(37, 256, generator=torch.Generator().manual_seed(1)).to(TYPES[dtype]).cuda()
    part = big[:, 64:160]
    for got, ref in zip(geg.gmxfp4_quantize(part, values=True), geg.gmxfp4_quantize(part.contiguous(), values=True)):
        assert torch.equal(got, ref)
    x3 = big.reshape(37, 4, 64)
    c, s = geg.gmxfp4_quantize(x3)
    assert c.shape == (37, 4, 32) and s.shape == (37, 4, 2)
    assert torch.equal(c.reshape(37, 128), geg.gmxfp4_quantize(big)[0])
    assert geg.gmxfp4_quantize(big[:0])[0].shape == (0, 128)


def test_quantised_weights_feed_the_grouped_gemm():
    # packer -> grouped GEMM -> the product of the decoded values
    import grouped_expert_gemm_amd as geg
    g = torch.Generator().manual_seed(5)
    E, N, K, M = 3, 64, 128, 40
    w = torch.randn(E, N, K, generator=g) * 0.05
    codes, scales, values = geg.gmxfp4_quantize(w.cuda(), values=True)
    a = torch.randn(M, K, generator=g).to(torch.bfloat16)
    sizes = torch.tensor([10, 0, 30], dtype=torch.int32)
    out = geg.gmxfp4_grouped_gemm(a.cuda(), sizes.cuda(), codes, scales).double().cpu()
    v = values.double().cpu()
    ref = torch.cat([a[:10].double() @ v[0].T, a[10:].double() @ v[2].T])
    # bf16 result (2^-8) and fp32 sums of K exact products (K 2^-24 of the sum of magnitudes)
    mag = torch.cat([a[:10].double().abs() @ v[0].abs().T, a[10:].double().abs() @ v[2].abs().T])
    assert bool(((out - ref).abs() <= 2 ** -8 * ref.abs() + K * 2.0 ** -24 * mag).all())


def test_another_stream_and_a_captured_graph():
    import grouped_expert_gemm_amd as geg
    x = torch.randn(64, 2880, device="cuda").to(torch.bfloat16)
    ref = geg.gmxfp4_quantize(x, values=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = geg.gmxfp4_quantize(x, values=True, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = geg.gmxfp4_quantize(x, values=True)
    for i in range(3):
        x.copy_(torch.randn(64, 2880, device="cuda") * (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, geg.gmxfp4_quantize(x, values=True)))

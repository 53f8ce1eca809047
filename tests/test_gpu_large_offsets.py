"""Operators on tensors of more than 2^31 elements: the rows past that border come out
bit for bit as the same rows do in a call of their own."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

K, ROWS, TAIL = 2048, (1 << 20) + 4099, 300   # 2^31 + 8.4e6 elements
assert ROWS * K > 1 << 31


def _rows(n):
    """[n, K] bf16 with values of several magnitudes, cheap to make."""
    base = torch.randn(4096, K, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    x = torch.empty(n, K, dtype=torch.bfloat16, device="cuda")
    for r in range(0, n, 4096):
        m = min(4096, n - r)
        torch.mul(base[:m], float(2.0 ** ((r >> 12) % 7 - 3)), out=x[r:r + m])
    return x


def test_quantize():
    import grouped_expert_gemm_amd as geg
    x = _rows(ROWS)
    got = geg.gmxfp4_quantize(x, values=True)
    for at in (0, (1 << 20) - TAIL // 2, ROWS - TAIL):   # the start, across the border, the end
        want = geg.gmxfp4_quantize(x[at:at + TAIL].clone(), values=True)
        for g, w in zip(got, want):
            assert torch.equal(g[at:at + TAIL], w), at


@pytest.mark.parametrize("first", [0, 1])
def test_w4a4_tiles(first):
    import grouped_expert_gemm_amd as geg
    g = torch.Generator().manual_seed(2)
    w = torch.randint(0, 256, (3, 64, K // 2), dtype=torch.uint8, generator=g).cuda()
    s = torch.randint(120, 128, (3, 64, K // 32), dtype=torch.uint8, generator=g).cuda()
    x = _rows(ROWS)
    sizes = [0, 0, TAIL]
    sizes[first] = ROWS - TAIL
    out = geg.gmxfp4_w4a4_grouped_gemm(x, torch.tensor(sizes, dtype=torch.int32, device="cuda"), w, s)
    # the last expert's rows, and the first expert's across the border
    for e, at in ((2, ROWS - TAIL), (first, (1 << 20) - TAIL // 2)):
        n = [0, 0, 0]
        n[e] = TAIL
        want = geg.gmxfp4_w4a4_grouped_gemm(x[at:at + TAIL].clone(), torch.tensor(n, dtype=torch.int32, device="cuda"),
                                            w, s, opts=geg.Opts(2, 0))
        assert torch.equal(out[at:at + TAIL], want), (e, at)


def test_combine_gradient():
    import grouped_expert_gemm_amd as geg
    k = 4
    T = ROWS // k
    y = _rows(T * k)
    dout = y[:T] * 0.5
    w = torch.rand(T, k, generator=torch.Generator().manual_seed(3)).cuda()
    row_of = torch.arange(T * k, dtype=torch.int32, device="cuda").flip(0)   # entry f's row is the f-th from the end
    dy, dw = geg.route_combine_grad(dout, y, row_of, w)
    n = 64
    for t0 in (0, T - n):
        rows = slice(T * k - (t0 + n) * k, T * k - t0 * k)   # of the tokens t0 .. t0 + n - 1
        local = torch.arange(n * k, dtype=torch.int32, device="cuda").flip(0)
        ry, rw = geg.route_combine_grad(dout[t0:t0 + n].clone(), y[rows].clone(), local, w[t0:t0 + n].clone())
        assert torch.equal(dy[rows], ry) and torch.equal(dw[t0:t0 + n], rw), t0

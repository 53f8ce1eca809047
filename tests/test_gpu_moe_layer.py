"""The few-token MoE layer against a plain fp64 computation, every element."""
import numpy as np
import pytest

from oracle import pack as P

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _weights(fmt, rng, E, N, K):
    """Packed weights (uint8 codes, scales) and their exact fp64 values [E, N, K]."""
    codes = rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
    if fmt == "nf4":
        scales = (0.02 + 0.03 * rng.random((E, N, K // 64))).astype(np.float32)
        return codes, scales, P.dequant_nf4(codes, scales)
    scales = rng.integers(118, 122, (E, N, K // 32), dtype=np.uint8)
    return codes, scales, P.dequant_mxfp4(codes, scales)


def _case(fmt, T, k, E, H, I, seed=0, ids=None):
    rng = np.random.default_rng([seed, T, k, E, H, I])
    c = {"fmt": fmt, "T": T, "k": k, "E": E, "H": H, "I": I}
    c["x"] = torch.tensor(rng.standard_normal((T, H)), dtype=torch.float32).to(torch.bfloat16)
    if ids is None:
        ids = np.argsort(rng.random((T, E)), axis=1)[:, :k]
    c["ids"] = torch.tensor(np.asarray(ids).reshape(T, k).copy(), dtype=torch.int32)
    c["w"] = torch.tensor(rng.random((T, k)), dtype=torch.float32)
    c["q13"], c["s13"], c["d13"] = _weights(fmt, rng, E, 2 * I, H)
    c["q2"], c["s2"], c["d2"] = _weights(fmt, rng, E, H, I)
    return c


def _reference(c):
    """(out, allowed error) in fp64.

    Allowed: the bf16 result (2^-8); fp32 sums of n products, n 2^-24 of their magnitudes;
    NF4's table as fp16, 2^-11 of every product; silu's slope is at most 1.1; the hardware
    exponential and reciprocal, 2^-20 of act; act as fp16 scaled per 32 values so that the
    largest lies in [2^14, 2^15): 2^-11 of each, or for those below fp16's normal range
    (2^-14) half its last step, 2^-25 against at least 2^14: 2^-39 of the block's largest."""
    x, w = c["x"].double().numpy(), c["w"].double().numpy()
    T, H, I = c["T"], c["H"], c["I"]
    table = 2.0 ** -11 if c["fmt"] == "nf4" else 0.0
    out, off = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for s, e in enumerate(c["ids"][t].tolist()):
            if not 0 <= e < c["E"]:
                continue
            h, mag = c["d13"][e] @ x[t], np.abs(c["d13"][e]) @ np.abs(x[t])
            dh = (table + H * 2.0 ** -24) * mag
            g, u, dg, du = h[0::2], h[1::2], dh[0::2], dh[1::2]
            silu = g / (1 + np.exp(-g))
            act = silu * u
            dact = 1.1 * dg * np.abs(u) + np.abs(silu) * du + 1.1 * dg * du + 2.0 ** -20 * np.abs(act)
            block = np.repeat(np.abs(act).reshape(-1, 32).max(1), 32)
            dact = dact * (1 + 2.0 ** -11) + 2.0 ** -11 * np.abs(act) + 2.0 ** -39 * block
            d2 = np.abs(c["d2"][e])
            out[t] += w[t, s] * (c["d2"][e] @ act)
            off[t] += w[t, s] * (d2 @ dact + (table + (I + 64) * 2.0 ** -24) * (d2 @ (np.abs(act) + dact)))
    return out, off + 2.0 ** -8 * (np.abs(out) + off)


def _call(c, **kw):
    import grouped_expert_gemm_amd as geg
    f = geg.gnf4_moe_layer if c["fmt"] == "nf4" else geg.gmxfp4_moe_layer
    d = [torch.tensor(np.ascontiguousarray(v)).cuda() if isinstance(v, np.ndarray) else v.cuda()
         for v in (c["x"], c["ids"], c["w"], c["q13"], c["s13"], c["q2"], c["s2"])]
    return f(*d, **kw)


def _check(c, **kw):
    got = _call(c, **kw).double().cpu().numpy()
    ref, tol = _reference(c)
    worst = float(np.max(np.abs(got - ref) / np.maximum(tol, 1e-300))) if got.size else 0.0
    print(f"  {c['fmt']} T={c['T']} k={c['k']} E={c['E']} H={c['H']} I={c['I']}: {worst:.3f} of the allowed error", flush=True)
    assert np.all(np.isfinite(got)) and worst <= 1.0


@pytest.mark.parametrize("fmt", ["nf4", "mxfp4"])
@pytest.mark.parametrize("T,k,E,H,I", [(1, 1, 1, 64, 64), (1, 8, 16, 256, 128), (1, 4, 8, 576, 1088), (2, 2, 4, 512, 512),
                                       (3, 5, 8, 1024, 320), (4, 2, 4, 2112, 128), (16, 8, 32, 256, 192),
                                       (16, 16, 16, 128, 64), (16, 1, 2, 1088, 576), (13, 3, 5, 4096, 64),
                                       (5, 4, 6, 64, 2240)])
def test_layer_matches_fp64(fmt, T, k, E, H, I):
    _check(_case(fmt, T, k, E, H, I))


@pytest.mark.parametrize("scale", [1e-12, 3e4])
@pytest.mark.parametrize("fmt", ["nf4", "mxfp4"])
def test_activations_of_any_scale(fmt, scale):
    # act runs as the square of the gate/up weights' scale: far outside fp16 without its own
    c = _case(fmt, 3, 2, 4, 256, 128)
    if fmt == "nf4":
        c["s13"] = (c["s13"] * scale).astype(np.float32)
        c["d13"] = P.dequant_nf4(c["q13"], c["s13"])
    else:
        shift = int(np.round(np.log2(scale)))
        c["s13"] = (c["s13"].astype(np.int32) + shift).astype(np.uint8)
        c["d13"] = P.dequant_mxfp4(c["q13"], c["s13"])
    _check(c)


@pytest.mark.parametrize("T,k,E,H,I", [(1, 2, 4, 32, 96), (3, 2, 4, 96, 32), (2, 4, 4, 2880, 160), (16, 4, 8, 160, 2880)])
def test_mxfp4_sizes_that_are_multiples_of_32_only(T, k, E, H, I):
    _check(_case("mxfp4", T, k, E, H, I))


@pytest.mark.parametrize("fmt", ["nf4", "mxfp4"])
def test_every_token_on_one_expert_and_an_expert_named_twice(fmt):
    _check(_case(fmt, 16, 2, 4, 256, 128, ids=[[3, 1]] * 16))
    _check(_case(fmt, 3, 4, 4, 256, 128, ids=[[2, 2, 0, 2]] * 3))
    _check(_case(fmt, 1, 6, 4, 256, 128, ids=[[2, 2, 0, 2, 2, 2]]))
    # more entries on one expert than one pass over its weights takes
    _check(_case(fmt, 16, 16, 4, 128, 64, ids=[[1] * 16] * 16))


@pytest.mark.parametrize("fmt", ["nf4", "mxfp4"])
def test_ids_outside_the_experts_are_dropped_and_flagged(fmt):
    import grouped_expert_gemm_amd as geg
    c = _case(fmt, 4, 2, 4, 256, 128, ids=[[0, -1], [-1, 7], [3, 2], [4, 1]])
    ws = geg.Workspace()
    got = _call(c, workspace=ws)
    assert ws.read_error() == geg.DEVERR_BAD_EXPERT_ID
    assert bool((got[1] == 0).all())       # a token without any valid entry
    ref, tol = _reference(c)
    assert np.all(np.abs(got.double().cpu().numpy() - ref) <= tol)
    with pytest.raises(geg.GegDeviceError):
        _call(c, check_errors=True)
    none = _case(fmt, 2, 2, 4, 256, 128, ids=[[-1, -1], [9, 9]])
    assert bool((_call(none) == 0).all())


@pytest.mark.parametrize("fmt", ["nf4", "mxfp4"])
@pytest.mark.parametrize("T,k,E,H,I", [(1, 64, 64, 64, 64), (1, 65, 80, 128, 64), (1, 256, 300, 64, 64),
                                       (1, 8, 1024, 64, 128), (16, 16, 1024, 64, 64), (1, 3, 4, 6208, 4160),
                                       (1, 1, 1, 71744, 64), (2, 2, 3, 35904, 64)])
def test_most_entries_experts_and_tokens_past_the_staging(fmt, T, k, E, H, I):
    _check(_case(fmt, T, k, E, H, I))


@pytest.mark.parametrize("k", [5, 70])
@pytest.mark.parametrize("fmt", ["nf4", "mxfp4"])
def test_one_token_with_dropped_ids(fmt, k):
    import grouped_expert_gemm_amd as geg
    rng = np.random.default_rng(k)
    c = _case(fmt, 1, k, 6, 256, 192, ids=[rng.integers(-2, 9, k)])
    c["ids"][0, :4] = torch.tensor([6, 0, -1, 1 << 30])
    ws = geg.Workspace(1 << 20)
    ws.buf[256:] = 255   # act that nobody writes would be NaN
    got = _call(c, workspace=ws)
    assert ws.read_error() == geg.DEVERR_BAD_EXPERT_ID
    ref, tol = _reference(c)
    assert np.all(np.abs(got.double().cpu().numpy() - ref) <= tol)
    none = _case(fmt, 1, k, 6, 256, 192, ids=[[-1] * k])
    assert bool((_call(none, workspace=ws) == 0).all())


def test_nf4_fp16_overflow_is_flagged():
    import grouped_expert_gemm_amd as geg
    for H in (256, 4096):                  # tokens staged in LDS, and read from memory
        c = _case("nf4", 16, 2, 4, H, 64)
        c["x"][15, H - 1] = 1e5
        ws = geg.Workspace()
        _call(c, workspace=ws)
        assert ws.read_error() == geg.DEVERR_FP16_RANGE


@pytest.mark.parametrize("fmt", ["nf4", "mxfp4"])
def test_a_bad_token_leaves_the_others_alone(fmt):
    c = _case(fmt, 4, 2, 4, 320, 192)
    ref = _call(c)
    c["x"][2, 5] = float("nan")
    got = _call(c)
    assert torch.equal(got[[0, 1, 3]], ref[[0, 1, 3]]) and bool(got[2].isnan().all())


@pytest.mark.parametrize("fmt", ["nf4", "mxfp4"])
def test_grids_smaller_than_the_work_give_the_same_bits(fmt):
    import grouped_expert_gemm_amd as geg
    c = _case(fmt, 5, 3, 8, 512, 320)
    ref = _call(c)
    assert torch.equal(_call(c, opts=geg.Opts(cu_limit=3)), ref)
    assert torch.equal(_call(c), ref)


def test_inputs_and_rows_outside_the_output_are_left_alone():
    import grouped_expert_gemm_amd as geg
    c = _case("nf4", 3, 2, 4, 256, 128)
    d = [torch.tensor(np.ascontiguousarray(v)).cuda() if isinstance(v, np.ndarray) else v.cuda()
         for v in (c["x"], c["ids"], c["w"], c["q13"], c["s13"], c["q2"], c["s2"])]
    before = [t.clone() for t in d]
    buf = torch.full((5, 256), 3.0, dtype=torch.bfloat16, device="cuda")
    need = geg.lib().geg_moe_layer_workspace_bytes(3, 2, 128)
    ws = geg.Workspace(need + 4096)
    ws.buf[need:] = 77
    geg.gnf4_moe_layer(*d, out=buf[1:4], workspace=ws)
    assert bool((buf[[0, 4]] == 3).all()) and bool((ws.buf[need:] == 77).all())
    assert all(torch.equal(a, b) for a, b in zip(d, before))


def test_empty_batch():
    c = _case("nf4", 1, 2, 4, 256, 128)
    c["x"], c["ids"], c["w"] = c["x"][:0], c["ids"][:0], c["w"][:0]
    assert _call(c).shape == (0, 256)


@pytest.mark.parametrize("fmt", ["nf4", "mxfp4"])
def test_captured_graph_and_calls_on_two_streams(fmt):
    c, c2 = _case(fmt, 4, 2, 8, 512, 256), _case(fmt, 7, 3, 8, 512, 256, seed=1)
    import grouped_expert_gemm_amd as geg
    f = geg.gnf4_moe_layer if fmt == "nf4" else geg.gmxfp4_moe_layer

    def up(c):
        return [torch.tensor(np.ascontiguousarray(v)).cuda() if isinstance(v, np.ndarray) else v.cuda()
                for v in (c["x"], c["ids"], c["w"], c["q13"], c["s13"], c["q2"], c["s2"])]
    a, b = up(c), up(c2)
    ra, rb = f(*a), f(*b)
    # two streams at once, each with the library's own workspace for it
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        outs.append((f(*a, stream=s1), f(*b, stream=s2)))
    torch.cuda.synchronize()
    assert all(torch.equal(x, ra) and torch.equal(y, rb) for x, y in outs)
    # two captured graphs replayed in turn with eager calls between
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        o1 = f(*a)
    with torch.cuda.graph(g2):
        o2 = f(*b)
    for i in range(4):
        a[0].copy_(torch.randn_like(a[0]))
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(o1, f(*a)) and torch.equal(o2, rb)


@pytest.mark.parametrize("fmt", ["nf4", "mxfp4"])
def test_gate_and_layer_agree_with_the_large_batch_path(fmt):
    """logits -> route_topk -> layer, against route_sort -> expert block -> combine."""
    import grouped_expert_gemm_amd as geg
    c = _case(fmt, 8, 4, 16, 512, 256)
    logits = torch.randn(8, 16, generator=torch.Generator().manual_seed(2)).cuda()
    weights, ids = geg.route_topk(logits, 4)
    c["ids"], c["w"] = ids.cpu(), weights.cpu()
    _check(c)
    got = _call(c).double()
    d = [torch.tensor(np.ascontiguousarray(v)).cuda() for v in (c["q13"], c["s13"], c["q2"], c["s2"])]
    sizes, row_of, _, xs = geg.route_sort(ids, 16, c["x"].cuda())
    block = geg.gnf4_expert_block if fmt == "nf4" else geg.gmxfp4_expert_block
    ref = geg.route_combine(block(xs, sizes, *d), row_of, weights, 4).double()
    # that path rounds act and each expert's output to bf16 as well
    assert float((got - ref).norm() / ref.norm()) <= 3 * 2.0 ** -8


@pytest.mark.parametrize("T", [1, 5])
def test_mxfp4_scales_at_any_byte(T):
    c = _case("mxfp4", T, 2, 4, 288, 96)
    want = _call(c)
    for shift in (1, 2, 3):
        d = dict(c)
        for name in ("s13", "s2"):
            s = torch.zeros(c[name].size + shift, dtype=torch.uint8, device="cuda")[shift:].view(c[name].shape)
            d[name] = s.copy_(torch.tensor(c[name]))
        assert torch.equal(_call(d), want), shift


@pytest.mark.parametrize("fmt", ["nf4", "mxfp4"])
@pytest.mark.parametrize("T,k,E,H,I", [(1, 2, 4, 256, 128), (3, 2, 4, 320, 128), (16, 2, 3, 2112, 64),
                                       (1, 2, 2, 32832, 64), (5, 8, 8, 64, 64)])
def test_tokens_of_any_scale(fmt, T, k, E, H, I):
    """Small and large tokens beside each other, staged (T H <= 32768) or not. What fp16 values
    under a common power of two lose, 2^-39 of the largest, vanishes in the table's 2^-11."""
    c = _case(fmt, T, k, E, H, I, seed=7)
    scale = torch.tensor([1e-8, 1e4, 1e-12, 1.0, 3e-5]).repeat(4)[:T]
    c["x"] = (c["x"].float() * scale[:, None]).to(torch.bfloat16)
    _check(c)


@pytest.mark.parametrize("fmt", ["nf4", "mxfp4"])
@pytest.mark.parametrize("T,H,I", [(1, 192, 192), (3, 192, 192), (1, 64, 64), (3, 32832, 64)])
def test_an_infinity_in_the_last_block_stays_one(fmt, T, H, I):
    # every weight is positive, so gate, up, act and the result of that token are +inf; lanes
    # that have no block of the row must not turn it into NaN
    c = _case(fmt, T, 2, 4, H, I)
    c["q13"][:] = c["q2"][:] = 0xFF if fmt == "nf4" else 0x22
    c["x"][T - 1, H - 1] = float("inf")
    got = _call(c)
    assert bool((got[T - 1] == float("inf")).all()) and bool(got[:T - 1].isfinite().all())

"""Cases of four operators beside the grouped 4-bit expert GEMM, as a program calls them.

* quantise: MXFP4 quantisation (e2m1 codes, one e8m0 scale per 32 values) of activations
  or of weights, with the values that the codes stand for.
* w4a4: the grouped expert GEMM with activations and weights both in MXFP4.
* layer: the routed experts of a whole MoE layer for a few tokens, from hidden states,
  expert ids and router weights to the layer's output.
* route: the router's top-k gate; in training also the gradients of the weighted
  combine and of the gate.

`own = False` computes them from elementary torch operations in fp32, `own = True` calls
grouped_expert_gemm_amd.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # activations of one decode step, four routed rows: latency
        {"name": "quantise_decode", "op": "quantise", "type": "bf16", "rows": 4, "K": 2880},
        # activations of a prefill of 2048 tokens with four experts each
        {"name": "quantise_prefill", "op": "quantise", "type": "bf16", "rows": 8192, "K": 2880},
        # eight experts' gate/up weights packed at load time
        {"name": "quantise_weights", "op": "quantise", "type": "fp32", "rows": 46080, "K": 2880},
        # one token through the gate/up projection of its four experts
        {"name": "w4a4_t1", "op": "w4a4", "E": 32, "K": 2880, "N": 5760, "T": 1, "k": 4},
        # a decode batch of 64 sequences through the down projection
        {"name": "w4a4_t64", "op": "w4a4", "E": 32, "K": 2880, "N": 2880, "T": 64, "k": 4},
        # prefill of 2048 tokens, gate/up
        {"name": "w4a4_t2048", "op": "w4a4", "E": 32, "K": 2880, "N": 5760, "T": 2048, "k": 4},
        # one token through many small NF4 experts
        {"name": "layer_nf4_t1", "op": "layer", "fmt": "nf4", "E": 128, "k": 8, "H": 2048, "I": 768, "T": 1},
        # one token through MXFP4 experts
        {"name": "layer_mxfp4_t1", "op": "layer", "fmt": "mxfp4", "E": 32, "k": 4, "H": 2880, "I": 2880, "T": 1},
        # a small decode batch over many small experts
        {"name": "layer_nf4_t16", "op": "layer", "fmt": "nf4", "E": 128, "k": 8, "H": 2048, "I": 768, "T": 16},
        # four tokens over a few large experts, several tokens sharing one
        {"name": "layer_nf4_large_t4", "op": "layer", "fmt": "nf4", "E": 8, "k": 2, "H": 4096, "I": 14336, "T": 4},
        # the gate of one decode batch: latency
        {"name": "route_decode", "op": "route", "type": "bf16", "T": 64, "E": 128, "k": 8, "N": 0, "renorm": True},
        # routing of a training step: gate, sort, gradients of the combine and of the gate
        {"name": "route_train", "op": "route", "type": "fp32", "T": 4096, "E": 128, "k": 8, "N": 2048, "renorm": True},
    ]


def draw(rng):
    def log_int(lo, hi):
        return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))

    op = rng.choice(("quantise", "w4a4", "layer", "route"))
    if op == "quantise":
        K = 32 * log_int(1, 448)
        return {"op": op, "type": rng.choice(tuple(TYPES)), "rows": log_int(1, min(65536, 132_000_000 // K)), "K": K}
    if op == "w4a4":
        E, K, N = log_int(1, 64), 32 * log_int(2, 128), log_int(16, 8192)
        k = rng.randint(1, min(E, 8))
        most = 8192 * 5760 * 2880 // (K * N) // k
        return {"op": op, "E": E, "K": K, "N": N, "T": log_int(1, max(1, min(8192 // k, most))), "k": k}
    if op == "layer":
        E, H, fmt = log_int(4, 128), 64 * log_int(4, 64), rng.choice(("nf4", "mxfp4"))
        T, k = rng.randint(1, 16), rng.randint(1, min(E, 8))
        # packed experts within 1.5 GB in all, the plain form's decoded ones within 16 GB
        most = min(1_000_000_000 // (E * H), 1_400_000_000 // (T * k * H), 14336)
        return {"op": op, "fmt": fmt, "E": E, "k": k, "H": H, "I": 64 * log_int(2, max(2, most // 64)), "T": T}
    E = log_int(4, 512)
    k = rng.randint(1, min(E, 8))
    N = rng.choice((0, 8 * log_int(8, 512)))
    T = log_int(1, 8192) if N == 0 else log_int(1, min(4096, 67_000_000 // (N * k)))
    return {"op": op, "type": rng.choice(tuple(TYPES)), "T": T, "E": E, "k": k, "N": N, "renorm": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs
def _routing(g, T, E, k):
    """Logits of a router whose experts differ in popularity, and their top-k."""
    rank = torch.randperm(E, generator=g, device="cuda") + 1
    logits = torch.randn(T, E, generator=g, device="cuda") - torch.log(rank)
    return logits, torch.topk(logits, k, dim=1)


def _packed(g, fmt, E, N, K):
    """4-bit codes of normally distributed weights of deviation about 0.02 and their block scales
    (NF4's codes are quantiles, MXFP4's drawn from scaled normal values, byte by byte)."""
    if fmt == "nf4":
        codes = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, generator=g, device="cuda")
        scales = 0.05 + 0.01 * torch.randn(E, N, K // 64, generator=g, device="cuda").abs()
        return codes, scales
    # bytes that pairs of e2m1 codes of normal values (largest of 32 near 4) take, by their share
    z = torch.randn(2, 1 << 16, generator=g, device="cuda") * 2.0
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    c = torch.bucketize(z.abs(), mids) + 8 * (z < 0)
    pairs = (c[0] + 16 * c[1]).to(torch.uint8)
    at = torch.randint(0, 1 << 16, (E, N, K // 2), dtype=torch.int32, generator=g, device="cuda")
    scales = torch.randint(119, 122, (E, N, K // 32), dtype=torch.uint8, generator=g, device="cuda")
    return pairs[at], scales


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    op = s["op"]
    if op == "quantise":
        x = torch.randn(s["rows"], s["K"], generator=g, device="cuda")
        # channels of uneven size and a few outliers, as activations and weights have
        x *= torch.exp(torch.randn(s["K"], generator=g, device="cuda") * 0.5)
        s["x"] = (x * 0.02 if s["type"] == "fp32" else x).to(TYPES[s["type"]])
    elif op == "w4a4":
        E, K, N, T, k = s["E"], s["K"], s["N"], s["T"], s["k"]
        ids = _routing(g, T, E, k)[1].indices
        order = torch.sort(ids.flatten(), stable=True).indices
        x = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
        s["a"] = x[order // k].contiguous()
        s["sizes"] = torch.bincount(ids.flatten(), minlength=E).to(torch.int32)
        s["w"], s["ws"] = _packed(g, "mxfp4", E, N, K)
        # the grouping as a host-side plan: experts with rows, their padded height, each row's padded place
        n = s["sizes"].tolist()
        used = [e for e in range(E) if n[e]]
        s["most"] = max(n)
        s["used"] = torch.tensor(used, device="cuda")
        s["place"] = torch.tensor([i * s["most"] + j for i, e in enumerate(used) for j in range(n[e])], device="cuda")
    elif op == "layer":
        E, H, I, T, k = s["E"], s["H"], s["I"], s["T"], s["k"]
        s["x"] = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
        values, ids = _routing(g, T, E, k)[1]
        s["ids"] = ids.to(torch.int32)
        s["weights"] = torch.softmax(values, dim=1)
        s["w13"], s["s13"] = _packed(g, s["fmt"], E, 2 * I, H)
        s["w2"], s["s2"] = _packed(g, s["fmt"], E, H, I)
    else:
        T, E, k, N = s["T"], s["E"], s["k"], s["N"]
        s["logits"] = _routing(g, T, E, k)[0].to(TYPES[s["type"]])
        if N:
            s["y"] = torch.randn(T * k, N, generator=g, device="cuda").to(torch.bfloat16)
            s["dout"] = (torch.randn(T, N, generator=g, device="cuda") * 1e-3).to(torch.bfloat16)
    return s


# ------------------------------------------------------------------ the plain forms
_NF4 = (-1.0, -0.6961928009986877, -0.5250730514526367, -0.39491748809814453, -0.28444138169288635, -0.18477343022823334,
        -0.09105003625154495, 0.0, 0.07958029955625534, 0.16093020141124725, 0.24611230194568634, 0.33791524171829224,
        0.44070982933044434, 0.5626170039176941, 0.7229568362236023, 1.0)
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
_tables = {}


def _byte_pairs(fmt, dtype):
    """The two values of each code byte: [256, 2] (NF4: high nibble first, MXFP4: low nibble first)."""
    if (fmt, dtype) not in _tables:
        t = torch.tensor(_NF4 if fmt == "nf4" else _E2M1, dtype=torch.float32, device="cuda").to(dtype)
        b = torch.arange(256, device="cuda")
        hi, lo = t[b >> 4], t[b & 15]
        _tables[fmt, dtype] = torch.stack((hi, lo) if fmt == "nf4" else (lo, hi), dim=1)
    return _tables[fmt, dtype]


def _decoded(fmt, codes, scales):
    """[.., K/2] codes and block scales -> fp32 values [.., K]."""
    v = _byte_pairs(fmt, torch.float32)[codes.to(torch.int32)]
    v = v.reshape(*scales.shape, 64 if fmt == "nf4" else 32)
    s = scales if fmt == "nf4" else torch.exp2(scales.to(torch.float32) - 127)
    return (v * s[..., None]).reshape(*codes.shape[:-1], -1)


def _mxfp4(x):
    """fp32 values of x after MXFP4 quantisation and the blocks' exponents: scale 2^(floor(log2 amax) - 2),
    nearest e2m1 value, ties to the even code, saturating at 6."""
    b = x.to(torch.float32).reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    X = torch.where(amax > 0, torch.frexp(amax).exponent - 3, 0).clamp(min=-127)
    t = torch.ldexp(b, -X)
    a = t.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp(max=6)
    return torch.ldexp(torch.copysign(q, t), X).reshape(x.shape), X.squeeze(-1)


def _plain_w4a4(s):
    a = _mxfp4(s["a"])[0]
    w = _decoded("mxfp4", s["w"][s["used"]], s["ws"][s["used"]])
    rows = a.new_zeros(w.shape[0] * s["most"], a.shape[1])
    rows[s["place"]] = a
    rows = rows.reshape(w.shape[0], s["most"], -1).transpose(1, 2).contiguous()
    out = torch.bmm(w, rows).transpose(1, 2).reshape(-1, s["N"])
    return out[s["place"]].to(torch.bfloat16)


def _plain_layer(s):
    T, k = s["ids"].shape
    e = s["ids"].flatten()
    x = s["x"].to(torch.float32).repeat_interleave(k, 0).unsqueeze(-1)
    h = torch.bmm(_decoded(s["fmt"], s["w13"][e], s["s13"][e]), x)
    gate, up = h[:, 0::2], h[:, 1::2]
    act = gate / (1 + torch.exp(-gate)) * up
    y = torch.bmm(_decoded(s["fmt"], s["w2"][e], s["s2"][e]), act).reshape(T, k, -1)
    return (s["weights"].unsqueeze(-1) * y).sum(1).to(torch.bfloat16)


def _plain_route(s):
    k, logits = s["k"], s["logits"]
    values = logits.to(torch.float32)
    ids = torch.sort(values, dim=1, descending=True, stable=True).indices[:, :k]
    p = torch.exp(values - values.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    w = p.gather(1, ids)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    if not s["N"]:
        return {"weights": w, "ids": ids.to(torch.int32)}
    order = torch.sort(ids.flatten(), stable=True).indices
    row = torch.empty_like(order).scatter_(0, order, torch.arange(order.numel(), device=order.device))
    dout = s["dout"].to(torch.float32).unsqueeze(1)
    dw = (s["y"][row].to(torch.float32).reshape(*ids.shape, -1) * dout).sum(-1)
    dy = torch.empty_like(s["y"])
    dy[row] = (w.unsqueeze(-1) * dout).reshape(s["y"].shape).to(torch.bfloat16)
    back = w * (dw - (w * dw).sum(1, keepdim=True))
    if s["renorm"]:
        dlogits = torch.zeros_like(values).scatter_(1, ids, back)
    else:  # w are the softmax's own values: the others fall as the chosen ones' weighted sum grows
        dlogits = (-p * (w * dw).sum(1, keepdim=True)).scatter_add_(1, ids, w * dw)
    return {"weights": w, "ids": ids.to(torch.int32), "dy": dy, "dlogits": dlogits.to(logits.dtype)}


def _plain(s):
    if s["op"] == "quantise":
        values, X = _mxfp4(s["x"])
        return {"values": values.to(s["x"].dtype), "exponents": (X + 127).to(torch.uint8)}
    return {"w4a4": _plain_w4a4, "layer": _plain_layer, "route": _plain_route}[s["op"]](s)


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    import grouped_expert_gemm_amd as geg

    op = s["op"]
    if op == "quantise":
        codes, scales, values = geg.gmxfp4_quantize(s["x"], values=True)
        return {"values": values, "exponents": scales}
    if op == "w4a4":
        return geg.gmxfp4_w4a4_grouped_gemm(s["a"], s["sizes"], s["w"], s["ws"])
    if op == "layer":
        layer = geg.gnf4_moe_layer if s["fmt"] == "nf4" else geg.gmxfp4_moe_layer
        return layer(s["x"], s["ids"], s["weights"], s["w13"], s["s13"], s["w2"], s["s2"])
    weights, ids = geg.route_topk(s["logits"], s["k"], renormalize=s["renorm"])
    if not s["N"]:
        return {"weights": weights, "ids": ids}
    sizes, row_of, src_of, _ = geg.route_sort(ids, s["E"])
    dy, dw = geg.route_combine_grad(s["dout"], s["y"], row_of, weights)
    dlogits = geg.route_topk_grad(dw, s["logits"], ids, weights, renormalize=s["renorm"])
    return {"weights": weights, "ids": ids, "dy": dy, "dlogits": dlogits}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def _experts_used(E, k, T):
    """Experts that T tokens of k distinct experts each reach, as if all were equally likely."""
    return E * (1 - (1 - k / E) ** T)


def work(case):
    op = case["op"]
    if op == "quantise":
        n = case["rows"] * case["K"]
        size = 4 if case["type"] == "fp32" else 2
        return {"bytes": n * (2 * size + 0.5 + 1 / 32), "flops": 4 * n}
    if op == "w4a4":
        E, K, N, M = case["E"], case["K"], case["N"], case["T"] * case["k"]
        w = _experts_used(E, case["k"], case["T"]) * N * (K // 2 + K // 32)
        return {"bytes": w + 2 * M * K + 2 * M * N + 4 * E, "flops": 2 * M * N * K}
    if op == "layer":
        E, k, H, I, T = case["E"], case["k"], case["H"], case["I"], case["T"]
        w = _experts_used(E, k, T) * 3 * H * I * (0.5 + (1 / 16 if case["fmt"] == "nf4" else 1 / 32))
        return {"bytes": w + 4 * T * H + 8 * T * k, "flops": 6 * T * k * H * I}
    T, E, k, N = case["T"], case["E"], case["k"], case["N"]
    size = 4 if case["type"] == "fp32" else 2
    gate = T * E * size + 8 * T * k
    if not N:
        return {"bytes": gate, "flops": 4 * T * E}
    return {"bytes": gate + T * E * size + 2 * T * N + 4 * T * k * N, "flops": 4 * T * E + 3 * T * k * N}


# ------------------------------------------------------------------ the definitions in 64 bits
def _weights64(fmt, codes, scales):
    """One expert's weights, code by code."""
    first, second = (codes >> 4, codes & 15) if fmt == "nf4" else (codes & 15, codes >> 4)
    c = torch.stack((first, second), dim=-1).flatten(-2).to(torch.int64)
    if fmt == "nf4":
        v = torch.tensor(_NF4, dtype=torch.float32, device=codes.device).to(torch.float64)[c]
        return v * scales.to(torch.float64).repeat_interleave(64, -1)
    sign = 1.0 - 2.0 * (c >> 3)
    e, m = (c >> 1) & 3, (c & 1).to(torch.float64)
    mag = torch.where(e == 0, 0.5 * m, 2.0 ** (e - 1).to(torch.float64) * (1 + 0.5 * m))
    return sign * mag * (2.0 ** (scales.to(torch.float64) - 127)).repeat_interleave(32, -1)


def _mxfp4_64(x):
    """Quantisation by search among the seven midpoints of neighbouring magnitudes."""
    mag = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)
    mid = (mag[1:] + mag[:-1]) / 2
    b = x.to(torch.float64).unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    X = torch.where(amax > 0, torch.floor(torch.log2(amax.clamp(min=1e-300))) - 2, 0.0).clamp(min=-127)
    t = b * (2.0 ** -X).unsqueeze(-1)
    below, upto = torch.bucketize(t.abs(), mid), torch.bucketize(t.abs(), mid, right=True)
    code = torch.where(below % 2 == 0, below, upto)
    return (torch.where(t < 0, -mag[code], mag[code]) * (2.0 ** X).unsqueeze(-1)).flatten(-2), X


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "quantise":
        values = [_mxfp4_64(x) for x in s["x"].split(8192)]
        return {"values": torch.cat([v for v, _ in values]), "exponents": (torch.cat([X for _, X in values]) + 127).to(torch.uint8)}
    if op == "w4a4":
        a, out, r0 = _mxfp4_64(s["a"])[0], [], 0
        for e, n in enumerate(s["sizes"].tolist()):
            if n:
                out.append(torch.mm(a[r0:r0 + n], _weights64("mxfp4", s["w"][e], s["ws"][e]).t().contiguous()))
                r0 += n
        return torch.cat(out)
    if op == "layer":
        x, weights = s["x"].to(torch.float64), s["weights"].to(torch.float64)
        out = torch.zeros_like(x)
        for e in sorted(set(s["ids"].flatten().tolist())):
            tok, slot = torch.nonzero(s["ids"] == e, as_tuple=True)
            h = torch.mm(_weights64(s["fmt"], s["w13"][e], s["s13"][e]), x[tok].t().contiguous())
            act = h[0::2] * torch.sigmoid(h[0::2]) * h[1::2]
            y = torch.mm(_weights64(s["fmt"], s["w2"][e], s["s2"][e]), act).t()
            out.index_add_(0, tok, weights[tok, slot].unsqueeze(1) * y)
        return out
    logits = s["logits"].to(torch.float64)
    T, E, k, N = s["T"], s["E"], s["k"], s["N"]
    # rank of an expert: those with larger logits, and equal ones before it
    left, ids = logits.clone(), []
    for _ in range(k):
        top = left.amax(1, keepdim=True)
        first = torch.where(left == top, torch.arange(E, device=left.device), E).amin(1)
        ids.append(first)
        left.scatter_(1, first.unsqueeze(1), -math.inf)
    ids = torch.stack(ids, 1)
    chosen = torch.zeros_like(logits).scatter_(1, ids, 1.0)
    masked = logits if not s["renorm"] else torch.where(chosen > 0, logits, -math.inf)
    p = torch.softmax(masked, 1)
    w = p.gather(1, ids)
    if not N:
        return {"weights": w, "ids": ids.to(torch.int32)}
    row = torch.argsort(torch.argsort(ids.flatten() * (T * k) + torch.arange(T * k, device=ids.device)))
    dout = s["dout"].to(torch.float64)
    y = s["y"].to(torch.float64)
    dp = torch.zeros_like(logits)
    dy = torch.zeros_like(y)
    for j in range(k):
        r = row[j::k]
        dp.scatter_(1, ids[:, j:j + 1], (y[r] * dout).sum(1, keepdim=True))
        dy[r] = w[:, j:j + 1] * dout
    dlogits = p * (dp - (p * dp).sum(1, keepdim=True))
    return {"weights": w, "ids": ids.to(torch.int32), "dy": dy, "dlogits": dlogits}

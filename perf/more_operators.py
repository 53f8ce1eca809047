"""Cases of three operators beside the grouped 4-bit expert GEMM, as a program calls them.

* experts: the grouped expert product with 16-bit weights: the forward pass, and the
  backward pass with the gradients of the activations and of the weights.
* adapters: low-rank adapters of many requests in one batch, added to what a shared
  projection gave: out = y + scale_i (x A_i^T) B_i^T with each row's own adapter i.
* dropout: dropout from a counter-based generator (Philox4x32-10, Salmon et al. 2011), in
  training with its gradient, optionally added to a residual.

`own = False` computes them from elementary torch operations in fp32, `own = True` calls
grouped_expert_gemm_amd.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token through the gate/up projection of its eight experts: latency
        {"name": "experts_decode_t1", "op": "experts", "pass": "forward", "type": "bf16", "E": 64, "K": 2048, "N": 2048, "T": 1, "k": 8},
        # a decode batch of 48 sequences over many small experts
        {"name": "experts_decode_t48", "op": "experts", "pass": "forward", "type": "fp16", "E": 128, "K": 2048, "N": 1536, "T": 48, "k": 8},
        # a prompt of odd length, gate/up
        {"name": "experts_ragged_t777", "op": "experts", "pass": "forward", "type": "fp16", "E": 32, "K": 2880, "N": 5760, "T": 777, "k": 4},
        # prefill of 4096 tokens through large experts
        {"name": "experts_prefill_t4096", "op": "experts", "pass": "forward", "type": "bf16", "E": 8, "K": 4096, "N": 28672, "T": 4096, "k": 2},
        # backward pass of a training step: both gradients in the weights' type
        {"name": "experts_backward_t2048", "op": "experts", "pass": "backward", "type": "bf16", "E": 64, "K": 2048, "N": 2048, "T": 2048, "k": 8, "grad": "bf16"},
        # backward pass of a small micro-batch, the weights' gradient kept in fp32 for accumulation
        {"name": "experts_backward_t300", "op": "experts", "pass": "backward", "type": "fp16", "E": 32, "K": 2880, "N": 2880, "T": 300, "k": 4, "grad": "fp32"},
        # one request with its adapter: latency
        {"name": "adapters_t1", "op": "adapters", "type": "bf16", "L": 8, "r": 16, "K": 2048, "N": 2048, "T": 1, "runs": False},
        # a decode batch, every row another request, some without an adapter
        {"name": "adapters_decode_t96", "op": "adapters", "type": "bf16", "L": 32, "r": 16, "K": 4096, "N": 4096, "T": 96, "runs": False},
        # prompts of several requests one after the other through a wide projection
        {"name": "adapters_prefill_t8000", "op": "adapters", "type": "fp16", "L": 16, "r": 64, "K": 4096, "N": 14336, "T": 8000, "runs": True},
        # the input of an adapter in a small step: latency
        {"name": "dropout_small", "op": "dropout", "type": "bf16", "rows": 64, "C": 2048, "p": 0.05, "residual": False},
        # a layer's output on its way into the residual stream of a training step
        {"name": "dropout_residual", "op": "dropout", "type": "bf16", "rows": 16384, "C": 4096, "p": 0.1, "residual": True},
        # an odd number of values in full precision
        {"name": "dropout_fp32_odd", "op": "dropout", "type": "fp32", "rows": 4097, "C": 2881, "p": 0.4, "residual": False},
    ]


def draw(rng):
    def log_int(lo, hi):
        return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))

    op = rng.choice(("experts", "experts", "adapters", "dropout"))
    if op == "experts":
        E, K = log_int(1, 128), 8 * log_int(8, 640)
        N = 8 * log_int(8, 1024)
        k = rng.randint(1, min(E, 8))
        # weights within 2.5 GB in fp32, rows within the plain form's padding
        E = max(1, min(E, 640_000_000 // (K * N)))
        k = min(k, E)
        T = log_int(1, min(4096, 30_000_000 // (k * max(K, N)) + 1))
        case = {"op": op, "pass": rng.choice(("forward", "backward")), "type": rng.choice(("bf16", "fp16")), "E": E, "K": K, "N": N, "T": T, "k": k}
        if case["pass"] == "backward":
            case["grad"] = rng.choice((case["type"], "fp32"))
        elif rng.random() < 0.3:
            case["N"] = N - rng.randint(1, 7)
        return case
    if op == "adapters":
        K, N = 8 * log_int(8, 1024), 8 * log_int(8, 1792)
        return {"op": op, "type": rng.choice(("bf16", "fp16")), "L": log_int(1, 64), "r": 8 * rng.randint(1, 16), "K": K, "N": N,
                "T": log_int(1, min(8192, 100_000_000 // max(K, N))), "runs": rng.random() < 0.5}
    C = log_int(1, 16384)
    return {"op": op, "type": rng.choice(tuple(TYPES)), "rows": log_int(1, min(16384, 60_000_000 // C)), "C": C,
            "p": round(rng.uniform(0.0, 0.9), 2), "residual": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs
def _grouping(ids, n):
    """A host-side plan of rows grouped by id: the ids with rows, the most rows of one, and
    the place of each row (in grouped order) in a padded [ids with rows, most] layout."""
    counts = torch.bincount(ids, minlength=n).tolist()
    used = [e for e in range(n) if counts[e]]
    most = max(counts)
    place = [i * most + j for i, e in enumerate(used) for j in range(counts[e])]
    return torch.tensor(used, device="cuda"), most, torch.tensor(place, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)

    def normal(*shape, scale=1.0):
        # drawn in the type itself: no fp32 copy of large weights
        return torch.randn(*shape, generator=g, device="cuda", dtype=TYPES[s["type"]]).mul_(scale)

    if s["op"] == "experts":
        E, K, N, T, k = s["E"], s["K"], s["N"], s["T"], s["k"]
        # a router trained for balance: experts differ somewhat in popularity
        logits = torch.randn(T, E, generator=g, device="cuda") + 0.3 * torch.randn(E, generator=g, device="cuda")
        ids = torch.topk(logits, k, dim=1).indices
        order = torch.sort(ids.flatten(), stable=True).indices
        s["a"] = normal(T, K)[order // k].contiguous()
        s["sizes"] = torch.bincount(ids.flatten(), minlength=E).to(torch.int32)
        s["w"] = normal(E, N, K, scale=0.02)
        if s["pass"] == "backward":
            s["dy"] = normal(T * k, N, scale=0.01)
        s["used"], s["most"], s["place"] = _grouping(ids.flatten(), E)
    elif s["op"] == "adapters":
        L, r, K, N, T = s["L"], s["r"], s["K"], s["N"], s["T"]
        s["x"], s["y"] = normal(T, K), normal(T, N)
        s["A"], s["B"] = normal(L, r, K, scale=K ** -0.5), normal(L, N, r, scale=0.02)
        s["scales"] = torch.rand(L, generator=g, device="cuda") + 0.5
        # requests with an adapter each, one in sixteen without
        requests = max(1, T // 500) if s["runs"] else T
        ids = torch.randint(0, L, (requests,), generator=g, device="cuda")
        ids[torch.rand(requests, generator=g, device="cuda") < (1 / 16 if requests > 1 else 0)] = -1
        if s["runs"]:   # the requests' rows stand together, in runs of uneven length
            ends = torch.sort(torch.randint(0, T + 1, (requests - 1,), generator=g, device="cuda")).values
            ids = ids[torch.bucketize(torch.arange(T, device="cuda"), ends, right=True)]
        s["ids"] = ids.to(torch.int32)
        with_one = torch.nonzero(ids >= 0).flatten()
        s["rows"] = with_one[torch.sort(ids[with_one], stable=True).indices]
        if with_one.numel():
            s["used"], s["most"], s["place"] = _grouping(ids[with_one], L)
    else:
        s["x"] = normal(s["rows"], s["C"])
        s["dy"] = normal(s["rows"], s["C"], scale=0.01)
        s["base"] = normal(s["rows"], s["C"]) if s["residual"] else None
        s["seed"] = int(torch.randint(0, 1 << 62, (1,), generator=g, device="cuda"))
        s["offset"] = int(torch.randint(0, 1 << 20, (1,), generator=g, device="cuda"))
    return s


# ------------------------------------------------------------------ the plain forms
def _padded(rows, s):
    """Grouped rows in fp32 [groups, most, width], zeros behind each group's last."""
    out = rows.new_zeros(s["used"].numel() * s["most"], rows.shape[1], dtype=torch.float32)
    out[s["place"]] = rows.to(torch.float32)
    return out.reshape(-1, s["most"], rows.shape[1])


def _plain_experts(s):
    dt = s["a"].dtype
    w = s["w"][s["used"]].to(torch.float32)
    if s["pass"] == "forward":
        a = _padded(s["a"], s).transpose(1, 2).contiguous()
        return torch.bmm(w, a).transpose(1, 2).reshape(-1, s["N"])[s["place"]].to(dt)
    dy, a = _padded(s["dy"], s), _padded(s["a"], s)
    dx = torch.bmm(dy, w).reshape(-1, s["K"])[s["place"]].to(dt)
    dw = torch.zeros(s["w"].shape, dtype=TYPES[s["grad"]], device=w.device)
    dw[s["used"]] = torch.bmm(dy.transpose(1, 2).contiguous(), a).to(dw.dtype)
    return {"dx": dx, "dw": dw}


def _plain_adapters(s):
    y = s["y"].to(torch.float32)
    if s["rows"].numel():
        x = _padded(s["x"][s["rows"]], s)
        u = torch.bmm(x, s["A"][s["used"]].to(torch.float32).transpose(1, 2).contiguous())
        d = torch.bmm(u, s["B"][s["used"]].to(torch.float32).transpose(1, 2).contiguous())
        d = d * s["scales"][s["used"]].reshape(-1, 1, 1)
        y[s["rows"]] += d.reshape(-1, s["N"])[s["place"]]
    return y.to(s["x"].dtype)


def _threshold(p):
    """A value is dropped where its 16 random bits are below this."""
    return round(p * 65536)


def _kept(shape, seed, offset, p):
    """Which values stay: value i takes half i % 8 (low halves first) of the four words that
    the generator gives for the counter (i // 8, offset), 64 bits each, and the key seed."""
    n = math.prod(shape)
    i = torch.arange((n + 7) // 8, device="cuda")
    c0, c1 = i & 0xFFFFFFFF, i >> 32
    c2 = torch.full_like(i, offset & 0xFFFFFFFF)
    c3 = torch.full_like(i, offset >> 32)
    k0, k1 = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF

    def product(m, c):
        """The high and low words of m * c: partial products of 16 bits of m fit 48 bits."""
        top, low = (m >> 16) * c, (m & 0xFFFF) * c
        return (top + (low >> 16)) >> 16, (((top & 0xFFFF) << 16) + low) & 0xFFFFFFFF

    for _ in range(10):
        h0, l0 = product(0xD2511F53, c0)
        h1, l1 = product(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    halves = torch.stack((c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16, c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16), 1)
    return (halves >= _threshold(p)).flatten()[:n].reshape(shape)


def _plain_dropout(s):
    x = s["x"]
    keep = _kept(x.shape, s["seed"], s["offset"], s["p"])
    scale = 65536 / (65536 - _threshold(s["p"]))
    out = torch.where(keep, x.to(torch.float32) * scale, 0.0)
    if s["residual"]:
        out = s["base"].to(torch.float32) + out
    dx = torch.where(keep, s["dy"].to(torch.float32) * scale, 0.0)
    return {"out": out.to(x.dtype), "dx": dx.to(x.dtype)}


def _plain(s):
    return {"experts": _plain_experts, "adapters": _plain_adapters, "dropout": _plain_dropout}[s["op"]](s)


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    import grouped_expert_gemm_amd as geg

    if s["op"] == "experts":
        if s["pass"] == "forward":
            return geg.grouped_gemm(s["a"], s["sizes"], s["w"])
        dx = geg.grouped_dgrad(s["dy"], s["sizes"], s["w"])
        dw = geg.grouped_wgrad(s["dy"], s["a"], s["sizes"], dtype=TYPES[s["grad"]])
        return {"dx": dx, "dw": dw}
    if s["op"] == "adapters":
        return geg.request_lora(s["y"], s["x"], s["ids"], s["A"], s["B"], s["scales"])
    out = geg.philox_dropout(s["x"], s["p"], s["seed"], s["offset"], residual=s["base"])
    return {"out": out, "dx": geg.philox_dropout(s["dy"], s["p"], s["seed"], s["offset"])}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def _expected_used(n, share, draws):
    """How many of n equally likely groups are met in `draws` draws of a share of 1/n each (or k distinct ones)."""
    return n * (1 - (1 - share) ** draws)


def work(case):
    op = case["op"]
    if op == "experts":
        E, K, N, T, k = case["E"], case["K"], case["N"], case["T"], case["k"]
        M, used = T * k, _expected_used(E, k / E, T)
        if case["pass"] == "forward":
            return {"bytes": 2 * (used * N * K + M * K + M * N) + 4 * E, "flops": 2 * M * N * K}
        size = 4 if case["grad"] == "fp32" else 2
        return {"bytes": 2 * (used * N * K + M * N + 2 * M * K) + size * E * N * K + 4 * E, "flops": 4 * M * N * K}
    if op == "adapters":
        L, r, K, N, T = case["L"], case["r"], case["K"], case["N"], case["T"]
        used = _expected_used(L, 1 / L, max(1, T // 500) if case["runs"] else T)
        return {"bytes": 2 * (T * K + 2 * T * N + used * r * (K + N)) + 4 * T, "flops": 2 * T * r * (K + N)}
    n = case["rows"] * case["C"]
    size = 4 if case["type"] == "fp32" else 2
    return {"bytes": n * size * (5 if case["residual"] else 4), "flops": 4 * n}


# ------------------------------------------------------------------ the definitions in 64 bits
def _kept64(n, seed, offset, p):
    """The kept values from the generator's definition, in unsigned 64-bit integers on the host."""
    low = np.uint64(0xFFFFFFFF)
    i = np.arange(-(-n // 8), dtype=np.uint64)
    words = [i & low, i >> np.uint64(32), np.full_like(i, offset & 0xFFFFFFFF), np.full_like(i, offset >> 32)]
    key = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for step in range(10):
        a = words[0] * np.uint64(0xD2511F53)
        b = words[2] * np.uint64(0xCD9E8D57)
        k0, k1 = ((key[0] + step * 0x9E3779B9) & 0xFFFFFFFF, (key[1] + step * 0xBB67AE85) & 0xFFFFFFFF)
        words = [(b >> np.uint64(32)) ^ words[1] ^ np.uint64(k0), b & low, (a >> np.uint64(32)) ^ words[3] ^ np.uint64(k1), a & low]
    bits = np.stack([w.astype(np.uint32) for w in words], 1).view("<u2").reshape(-1)[:n]
    return torch.from_numpy(bits.astype(np.int32) >= round(p * 65536)).to("cuda")


def exact(case, seed):
    s = prepare(case, seed)
    d = torch.float64
    if s["op"] == "experts":
        n, M = s["sizes"].tolist(), s["a"].shape[0]
        starts = np.concatenate(([0], np.cumsum(n))).tolist()
        groups = [(e, slice(starts[e], starts[e + 1])) for e in range(s["E"]) if n[e]]
        if s["pass"] == "forward":
            out = torch.empty(M, s["N"], dtype=d, device="cuda")
            for e, rows in groups:
                out[rows] = torch.mm(s["a"][rows].to(d), s["w"][e].to(d).t())
            return out
        dx = torch.empty(M, s["K"], dtype=d, device="cuda")
        dw = torch.zeros(s["w"].shape, dtype=d, device="cuda")
        for e, rows in groups:
            dx[rows] = torch.mm(s["dy"][rows].to(d), s["w"][e].to(d))
            dw[e] = torch.mm(s["dy"][rows].to(d).t(), s["a"][rows].to(d))
        return {"dx": dx, "dw": dw}
    if s["op"] == "adapters":
        out = s["y"].to(d)
        for i in sorted(set(s["ids"].tolist()) - {-1}):
            rows = torch.nonzero(s["ids"] == i).flatten()
            u = torch.mm(s["x"][rows].to(d), s["A"][i].to(d).t())
            out[rows] += s["scales"][i].to(d) * torch.mm(u, s["B"][i].to(d).t())
        return out
    x, dy = s["x"].to(d), s["dy"].to(d)
    keep = _kept64(x.numel(), s["seed"], s["offset"], s["p"]).reshape(x.shape)
    q = 1 - round(s["p"] * 65536) / 65536
    out = torch.where(keep, x / q, torch.zeros_like(x))
    if s["residual"]:
        out = out + s["base"].to(d)
    return {"out": out, "dx": torch.where(keep, dy / q, torch.zeros_like(dy))}

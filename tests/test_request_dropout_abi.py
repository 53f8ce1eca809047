"""Refusals of the request adapters and of dropout before any launch (no GPU needed)."""
import ctypes

import pytest

import grouped_expert_gemm_amd as geg

P = 0x10000


def L():
    return geg.lib()


def _req(y=P, ldy=64, x=2 * P, ldx=128, ids=P, a=P, b=P, scales=P, out=3 * P, ldo=64, dtype=0, M=4, N=64, K=128, L_=3, r=16,
         ws=P, nbytes=1 << 20):
    return L().geg_request_lora(y, ldy, x, ldx, ids, a, b, scales, out, ldo, dtype, M, N, K, L_, r, ws, nbytes, None)


def test_request_refusals():
    passes = (0, 1, 2, 3, 5, 8)
    assert _req() not in passes and _req(y=None, ldy=0) not in passes and _req(scales=None) not in passes
    assert _req(dtype=2) == 8 and _req(dtype=-1) == 8
    assert _req(M=-1) == 2 and _req(N=0) == 2 and _req(K=0) == 2 and _req(L_=0) == 2 and _req(M=1 << 31) == 2
    assert _req(N=60, ldy=64) == 2 and _req(K=100) == 2
    assert _req(r=0) == 2 and _req(r=12) == 2 and _req(r=136) == 2 and _req(r=128) not in passes
    assert _req(ldy=56) == 2 and _req(ldx=120) == 2 and _req(ldo=56) == 2
    assert _req(N=1 << 62, ldy=1 << 62, ldo=1 << 62) == 2 and _req(ldx=1 << 40) == 2
    assert _req(M=1 << 30) == 2 and _req(M=1 << 24, N=65536, ldy=65536, ldo=65536) == 2    # more workgroups than a launch holds
    assert _req(L_=32769) == 2 and _req(L_=32768) not in passes
    assert _req(M=0, x=None, ws=None) == 0
    for p in ("x", "ids", "a", "b", "out"):
        assert _req(**{p: None}) == 1, p
    for p in ("y", "x", "a", "b", "out"):
        assert _req(**{p: 5 * P + 8}) == 3, p
    assert _req(ldy=68) == 3 and _req(ldx=132) == 3 and _req(ldo=68) == 3
    assert _req(M=1, ldy=68, ldx=132, ldo=68) not in passes       # one row has no pitch
    assert _req(ids=P + 2) == 3 and _req(scales=P + 2) == 3
    assert _req(out=2 * P) == 8                                     # out is x
    assert _req(out=P, ldo=72) == 8 and _req(out=P) not in passes  # in place: one pitch
    assert _req(ws=None) == 5 and _req(ws=P + 16) == 5
    need = L().geg_request_lora_workspace_bytes(4, 128, 3, 16)
    # 5 units at most and their number, the rows in the units' order, one range of the contraction
    assert need == 256 + 256 + 256 + 256
    assert _req(nbytes=need - 1) == 5 and _req(nbytes=need) not in passes
    assert L().geg_request_lora_workspace_bytes(4, 128, 3, 136) == 0
    assert L().geg_request_lora_workspace_bytes(200, 128, 1, 16) == 256 + 256 + 1024 + 200 * 64


def _drop(x=P, res=None, out=P, dtype=0, n=100, p=0.5, seed=1, offset=0, rng=None):
    return L().geg_dropout(x, res, out, dtype, n, p, seed, offset, rng, None)


def test_dropout_refusals():
    passes = (0, 1, 2, 3, 5, 8)
    assert _drop() not in passes and _drop(res=P, rng=P) not in passes and _drop(seed=(1 << 64) - 1) not in passes
    assert _drop(dtype=3) == 8 and _drop(dtype=-1) == 8
    assert _drop(p=-0.1) == 8 and _drop(p=1.1) == 8 and _drop(p=float("nan")) == 8 and _drop(p=1.0) not in passes
    assert _drop(n=-1) == 2 and _drop(n=1 << 49) == 2
    assert _drop(n=0, x=None, out=None) == 0
    assert _drop(x=None) == 1 and _drop(out=None) == 1
    assert _drop(x=P + 1) == 3 and _drop(res=P + 1) == 3 and _drop(out=P + 2, dtype=2) == 3 and _drop(rng=P + 4) == 3
    assert _drop(x=P + 2, out=P + 6) not in passes


def test_adapter_dropout_refusals():
    for name, more in (("gnf4", 64), ("gmxfp4", 32)):
        f = getattr(L(), name + "_grouped_gemm_lora_dropout")
        call = lambda p=0.5, r=16, rng=None: f(P, P, P, P, P, P, 1.0, p, 1, 0, rng, P, P, 4, 64, 128, 2, r, P, 1 << 20, None, None)
        assert call(p=1.5) == 8 and call(rng=P + 4) == 3 and call(r=12) == 2
        b = getattr(L(), name + "_grouped_dgrad_lora_dropout")
        back = lambda p=0.5, N=64, nbytes=1 << 22: b(P, P, P, P, P, P, P, P, 1.0, p, 1, 0, None, P, P, P, 4, N, 128, 2, 16, P,
                                                     nbytes, None, None)
        assert back(p=-1.0) == 8 and back(N=60) == 2
    op = geg.GEG_OP_MXFP4_DGRAD
    plain, drop = L().geg_lora_workspace_bytes(op, 4, 64, 128, 2, 16), L().geg_lora_dropout_workspace_bytes(op, 4, 64, 128, 2, 16)
    assert drop == plain + 4 * 128 * 2 + 256   # the masked activations and their mask
    assert L().geg_lora_dropout_workspace_bytes(geg.GEG_OP_NF4_FWD, 4, 64, 128, 2, 16) == \
        L().geg_lora_workspace_bytes(geg.GEG_OP_NF4_FWD, 4, 64, 128, 2, 16)


def test_python_refusals():
    torch = pytest.importorskip("torch")
    bf, i32 = torch.bfloat16, torch.int32
    y, x, ids = torch.zeros(6, 64, dtype=bf), torch.zeros(6, 128, dtype=bf), torch.zeros(6, dtype=i32)
    A, B, s = torch.zeros(3, 16, 128, dtype=bf), torch.zeros(3, 64, 16, dtype=bf), torch.zeros(3)
    w, sc, sz = torch.zeros(2, 64, 64, dtype=torch.uint8), torch.zeros(2, 64, 2), torch.zeros(2, dtype=i32)
    la, lb = torch.zeros(2, 16, 128), torch.zeros(2, 64, 16)
    for call in (lambda: geg.request_lora(y, x.float(), ids, A, B, s), lambda: geg.request_lora(y.half(), x, ids, A, B, s),
                 lambda: geg.request_lora(y, x, ids.long(), A, B, s), lambda: geg.request_lora(y, x, ids[:5], A, B, s),
                 lambda: geg.request_lora(y, x, ids, A[:, :8], B, s), lambda: geg.request_lora(y, x, ids, A, B[:2], s),
                 lambda: geg.request_lora(y, x, ids, A, B, s.double()), lambda: geg.request_lora(y, x, ids, A, B, s[:2]),
                 lambda: geg.request_lora(y, x.t().contiguous().t(), ids, A, B, s),
                 lambda: geg.request_lora(y[:1].expand(6, 64), x, ids, A, B, s),
                 lambda: geg.request_lora(y, x, ids, A, B, s, out=y[:, :56]), lambda: geg.request_lora(y, x[0], ids, A, B, s),
                 lambda: geg.philox_dropout(x.double(), 0.1, 1), lambda: geg.philox_dropout(x.t(), 0.1, 1),
                 lambda: geg.philox_dropout(x, 0.1, 1, residual=y), lambda: geg.philox_dropout(x, 0.1, 1, residual=x.float()),
                 lambda: geg.philox_dropout(x, 0.1, torch.zeros(2)), lambda: geg.philox_dropout(x, 0.1, torch.zeros(3, dtype=torch.int64))):
        with pytest.raises(geg.GegError, match="GEG_ERR_BAD_SHAPE"):
            call()
    for call in (lambda: geg.request_lora(y, x, ids, A, B, s), lambda: geg.philox_dropout(x, 0.1, 1),
                 lambda: geg.dropout(x, 0.1, 1), lambda: geg.grouped_linear_lora(x, sz, w, sc, la, lb, 1.0, dropout=0.1, seed=1)):
        with pytest.raises(geg.GegError, match="GPU"):
            call()
    with pytest.raises(geg.GegError, match="seed"):
        geg.grouped_linear_lora(x, sz, w, sc, la, lb, 1.0, dropout=0.1)


def test_a_seed_on_another_device():
    """The words of a seed are read by the kernels: they have to be where the operands are."""
    torch = pytest.importorskip("torch")

    class On(torch.Tensor):
        """A tensor that says it is on a GPU."""
        __torch_function__ = torch._C._disabled_torch_function_impl
        index = 0
        device = property(lambda self: torch.device("cuda", self.index))

        def get_device(self):
            return self.index

    on = lambda t: t.as_subclass(On)
    x, sz = on(torch.zeros(6, 128, dtype=torch.bfloat16)), on(torch.zeros(2, dtype=torch.int32))
    w, sc = on(torch.zeros(2, 64, 64, dtype=torch.uint8)), on(torch.zeros(2, 64, 2))
    la, lb = on(torch.zeros(2, 16, 128)), on(torch.zeros(2, 64, 16))
    words = on(torch.zeros(2, dtype=torch.int64))
    words.index = 1
    with pytest.raises(geg.GegError, match="several devices"):
        geg.grouped_linear_lora(x, sz, w, sc, la, lb, 1.0, dropout=0.1, seed=words)
    with pytest.raises(geg.GegError, match="several devices"):
        geg.philox_dropout(x, 0.1, words)

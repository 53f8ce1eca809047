"""The routing sort over many chunks of entries, any number of experts, repeated
and invalid ids: index work, exact against a stable sort."""
import numpy as np
import pytest

from gpu_util import log, up

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def geg():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_expert_gemm_amd as g
    g.lib()
    return g


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (513, 1, 2), (70000, 1, 1), (9000, 4, 33), (5000, 8, 1000),
                                   (20000, 2, 1024), (131072, 2, 7)])
@pytest.mark.parametrize("invalid", [False, True])
def test_many_chunks(geg, T, k, E, invalid):
    log(f"case: route sort of {T} x {k} over {E} experts, invalid ids: {invalid}")
    rng = np.random.default_rng(T + k + E)
    # half of the entries go to a few experts
    ids = np.where(rng.random((T, k)) < 0.5, rng.integers(0, E, (T, k)), rng.integers(0, min(E, 3), (T, k)))
    if invalid:
        ids = np.where(rng.random((T, k)) < 0.1, rng.choice([-1, E, 1 << 30, -(1 << 31)], (T, k)), ids)
    ids = ids.astype(np.int32)
    ws = geg.Workspace(1 << 24)
    sizes, row_of, src_of, _ = geg.route_sort(up(ids), E, workspace=ws)
    flat = ids.ravel()
    good = np.flatnonzero((flat >= 0) & (flat < E))
    order = good[np.argsort(flat[good], kind="stable")]
    rows = np.full(T * k, -1, np.int32)
    rows[order] = np.arange(len(order), dtype=np.int32)
    back = np.full(T * k, -1, np.int32)
    back[:len(order)] = order
    np.testing.assert_array_equal(sizes.cpu().numpy(), np.bincount(flat[good], minlength=E))
    np.testing.assert_array_equal(row_of.cpu().numpy().ravel(), rows)
    np.testing.assert_array_equal(src_of.cpu().numpy().ravel(), back)
    assert bool(ws.read_error() & geg.DEVERR_BAD_EXPERT_ID) == (len(good) < T * k)

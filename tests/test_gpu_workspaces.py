"""Workspaces of calls that overlap: branches of one captured graph, streams, host threads."""
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _up(*arrays):
    return [torch.tensor(np.ascontiguousarray(v)).cuda() if isinstance(v, np.ndarray) else v.cuda() for v in arrays]


def _calls(name):
    """(function, two argument lists of different values and sizes) of an operator with scratch."""
    import grouped_expert_gemm_amd as geg
    import test_gpu_moe_layer as layer
    import test_gpu_w4a4 as w4a4
    if name in ("nf4", "mxfp4"):
        cases = [layer._case(name, T, k, 8, 512, 256, seed=i) for i, (T, k) in enumerate([(16, 4), (7, 3)])]
        return (geg.gnf4_moe_layer if name == "nf4" else geg.gmxfp4_moe_layer,
                [_up(c["x"], c["ids"], c["w"], c["q13"], c["s13"], c["q2"], c["s2"]) for c in cases])
    if name == "sort":
        rng = np.random.default_rng(3)
        return geg.route_sort, [(*_up(rng.integers(0, E, (T, k)).astype(np.int32)), E,
                                 torch.randn(T, 64, device="cuda").to(torch.bfloat16))
                                for T, k, E in ((6000, 8, 64), (300, 4, 40))]
    cases = [w4a4._case(sizes, 136, 320, seed=i) for i, sizes in enumerate([[20, 3, 9], [0, 41, 200]])]
    return geg.gmxfp4_w4a4_grouped_gemm, [_up(c["a"], c["sizes"], c["w"], c["s"]) for c in cases]


OPERATORS = ["nf4", "mxfp4", "w4a4", "sort"]


def _as_list(r):
    return [t for t in r if t is not None] if isinstance(r, tuple) else [r]


def _equal(got, want):
    return all(torch.equal(g, w) for g, w in zip(_as_list(got), _as_list(want)))


@pytest.mark.parametrize("name", OPERATORS)
def test_branches_of_one_graph_with_a_stream_given(name):
    """Two side streams forked into a capture, each with calls of its own, and allocations that
    the main branch fills meanwhile."""
    f, (a, b) = _calls(name)
    want = f(*a), f(*b)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    outs = []
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        s1.wait_stream(main)
        s2.wait_stream(main)
        for _ in range(3):
            outs.append((f(*a, stream=s1), f(*b, stream=s2)))
            for n in (1 << 10, 1 << 14, 1 << 18, 1 << 20):
                torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
        main.wait_stream(s1)
        main.wait_stream(s2)
    for turn in range(4):
        for pair in outs:
            for r in pair:
                for t in _as_list(r):
                    t.zero_()
        g.replay()
        f(*a)   # eager work between the replays
        torch.cuda.synchronize()
        assert all(_equal(x, want[0]) and _equal(y, want[1]) for x, y in outs), turn


@pytest.mark.parametrize("name", OPERATORS)
def test_a_call_onto_a_stream_that_is_captured(name):
    """Made while another stream is the current one; eager calls on the same stream follow."""
    f, (b, a) = _calls(name)
    want = f(*a), f(*b)
    s, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        with torch.cuda.stream(other):
            out = f(*a, stream=s)
    for turn in range(3):
        assert _equal(f(*b, stream=s), want[1])
        torch.empty(1 << 20, dtype=torch.uint8, device="cuda").fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert _equal(out, want[0]), turn


@pytest.mark.parametrize("name", OPERATORS)
def test_two_host_threads_on_one_stream(name):
    f, args = _calls(name)
    want = [f(*a) for a in args]
    torch.cuda.synchronize()
    start, outs, failed = threading.Barrier(2), [[], []], []

    def work(i):
        try:
            torch.cuda.set_device(0)
            start.wait(30)
            for _ in range(60):
                outs[i].append(f(*args[i]))
        except Exception as e:   # shown by the assertion below
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    torch.cuda.synchronize()
    assert not failed, failed
    for i in range(2):
        assert len(outs[i]) == 60 and all(_equal(o, want[i]) for o in outs[i])


def test_sorts_on_two_streams_at_once():
    f, args = _calls("sort")
    want = [f(*a) for a in args]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        for a, s in zip(args, streams):
            with torch.cuda.stream(s):
                outs.append(f(*a))
        outs += [f(*a, stream=s) for a, s in zip(args, streams)]
    torch.cuda.synchronize()
    assert all(_equal(o, want[i % 2]) for i, o in enumerate(outs))


def test_a_captured_sort_before_a_larger_one():
    """The larger one must not take away the memory that the graph writes."""
    f, (large, small) = _calls("sort")
    large = (large[0].repeat(40, 1), *large[1:2])
    want = f(*small), f(*large)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = f(*small)
    for turn in range(4):
        assert _equal(f(*large), want[1])
        torch.empty(1 << 24, dtype=torch.uint8, device="cuda").fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert _equal(out, want[0]), turn


def _busy(stream, seconds=0.02):
    """Work on `stream` that outlasts what the caller does next."""
    with torch.cuda.stream(stream):
        a = torch.randn(4096, 4096, device="cuda")
        for _ in range(max(1, int(seconds / 1.5e-3))):
            a = a @ a * 1e-3
    return a


@pytest.mark.parametrize("name", OPERATORS)
def test_a_workspace_that_grows_on_another_stream(name):
    """What growing replaces belongs to the stream that the workspace was made on, which goes on
    allocating while the earlier call still waits for its turn."""
    import grouped_expert_gemm_amd as geg
    f, args = _calls(name)
    args = sorted(args, key=lambda a: a[0].numel())
    want = [f(*a) for a in args]
    s = torch.cuda.Stream()
    for _ in range(3):
        ws = geg.Workspace(256)
        f(*args[0], workspace=ws)            # the small call's size
        torch.cuda.synchronize()
        n = ws.nbytes
        _busy(s)
        small = f(*args[0], workspace=ws, stream=s)
        large = f(*args[1], workspace=ws, stream=s)
        assert ws.nbytes > n
        junk = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255) for _ in range(8)]
        torch.cuda.synchronize()
        assert _equal(small, want[0]) and _equal(large, want[1])
        del junk


def test_the_first_call_on_another_stream_keeps_its_flags():
    import grouped_expert_gemm_amd as geg
    f, args = _calls("sort")
    ids = args[1][0].clone()
    ids[0, 0] = -1
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    _busy(torch.cuda.current_stream())
    ws = geg.Workspace(1 << 20)
    f(ids, 40, workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert ws.read_error() == geg.DEVERR_BAD_EXPERT_ID


@pytest.mark.parametrize("name", OPERATORS)
def test_a_captured_workspace_that_grows_later(name):
    import grouped_expert_gemm_amd as geg
    f, args = _calls(name)
    args = sorted(args, key=lambda a: a[0].numel())
    want = [f(*a) for a in args]
    ws = geg.Workspace(256)
    f(*args[0], workspace=ws)
    n = ws.nbytes
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = f(*args[0], workspace=ws)
    for turn in range(3):
        assert _equal(f(*args[1], workspace=ws), want[1])
        junk = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255) for _ in range(8)]
        g.replay()
        torch.cuda.synchronize()
        assert _equal(out, want[0]) and all(bool((j == 255).all()) for j in junk), turn
    assert ws.nbytes > n


def _gemm_calls(name):
    """(function, a large and a small argument list) of the grouped GEMM, its gradient and the block."""
    import grouped_expert_gemm_amd as geg
    g = torch.Generator(device="cuda").manual_seed(5)
    E, N, K = 4, 384, 1024

    def weights(n, k):
        return (torch.randint(0, 256, (E, n, k // 2), dtype=torch.uint8, generator=g, device="cuda"),
                0.02 + 0.03 * torch.rand(E, n, k // 64, generator=g, device="cuda"))

    def rows(sizes, k):
        return (torch.randn(sum(sizes), k, generator=g, device="cuda").to(torch.bfloat16),
                torch.tensor(sizes, dtype=torch.int32, device="cuda"))
    sizes = ([700, 300, 0, 500], [90, 70, 3, 200])
    if name == "gemm":
        w = weights(N, K)
        return geg.gnf4_grouped_gemm, [(*rows(n, K), *w) for n in sizes]
    if name == "dgrad":
        w = weights(N, K)
        return geg.gnf4_grouped_dgrad, [(*rows(n, N), *w) for n in sizes]
    w13, w2 = weights(512, K), weights(K, 256)
    return geg.gnf4_expert_block, [(*rows(n, K), *w13, *w2) for n in sizes]


@pytest.mark.parametrize("name", ["gemm", "dgrad", "block"])
def test_the_gemms_at_once_on_streams_and_threads(name):
    f, args = _gemm_calls(name)
    want = [f(*a) for a in args]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for a, s in zip(args, streams):
            with torch.cuda.stream(s):
                outs.append(f(*a))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i % 2]) for i, o in enumerate(outs))
    threaded = [[], []]

    def work(i):
        torch.cuda.set_device(0)
        for _ in range(30):
            threaded[i].append(f(*args[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    torch.cuda.synchronize()
    for i in range(2):
        assert len(threaded[i]) == 30 and all(torch.equal(o, want[i]) for o in threaded[i])


@pytest.mark.parametrize("name", ["gemm", "dgrad", "block"])
def test_a_captured_gemm_before_a_larger_one(name):
    f, (large, small) = _gemm_calls(name)
    large = (large[0].repeat(20, 1), large[1] * 20, *large[2:])
    want = f(*small), f(*large)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = f(*small)
    for turn in range(4):
        assert torch.equal(f(*large), want[1])
        torch.empty(1 << 26, dtype=torch.uint8, device="cuda").fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]), turn


def test_a_checked_call_does_not_raise_for_an_earlier_one():
    import grouped_expert_gemm_amd as geg
    f, args = _calls("sort")
    bad = args[1][0].clone()
    bad[0, 0] = -1
    f(bad, 40)                                    # flagged in the library's own workspace, unchecked
    assert _equal(f(*args[1], check_errors=True), f(*args[1]))
    gemm, calls = _gemm_calls("gemm")
    f(bad, 40)
    gemm(*calls[1], check_errors=True)
    with pytest.raises(geg.GegDeviceError):
        f(bad, 40, check_errors=True)


@pytest.mark.parametrize("name", ["nf4", "w4a4", "sort", "gemm"])
def test_streams_in_any_form(name):
    """A torch stream, its handle (0: the null stream) and any object that has one."""
    from types import SimpleNamespace
    f, args = _gemm_calls(name) if name == "gemm" else _calls(name)
    want = f(*args[0])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    here = torch.cuda.current_stream().cuda_stream
    outs = [f(*args[0], stream=form) for form in (s, s.cuda_stream, SimpleNamespace(cuda_stream=s.cuda_stream), 0,
                                                  torch.cuda.current_stream())]
    assert torch.cuda.current_stream().cuda_stream == here
    torch.cuda.synchronize()
    assert all(_equal(o, want) for o in outs)

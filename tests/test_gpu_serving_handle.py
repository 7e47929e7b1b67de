"""What the serving calls share in a handle, under capture and beside work on other streams."""
import pytest

from approximate_long_context_b200 import binding

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def busy(stream, ms=300):
    """Keeps a stream busy for about so long; the event behind it."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(int(ms * 1.9e6))
        return stream.record_event()


def rows(n=40):
    q = torch.randn(n, 2, 64, device="cuda").to(torch.bfloat16)
    return q, torch.empty_like(q)


def test_status_waits_for_the_handles_stream_alone():
    """A handle that only serves asks for its status without waiting for the default stream."""
    side = torch.cuda.Stream()
    ha = binding.HyperAttention(0)
    ha.set_options(dtype="bf16", stream=side.cuda_stream)
    q, o = rows()
    cu, bad = ints([0, 40]), ints([0, 41])
    torch.cuda.synchronize()
    ha.prompt(q, q, q, o, cu)
    assert ha.status() == 0
    end = busy(torch.cuda.default_stream())
    assert ha.status() == 0
    ha.prompt(q, q, q, o, bad)
    assert ha.status() == binding.HA_ERR_INVALID_ARG and ha.status() == 0
    assert not end.query()
    torch.cuda.synchronize()
    ha.close()


def test_reports_of_a_graph_on_another_stream():
    """A graph that always reports runs on another stream while the status is asked for: every replay that had ended before the
    question is in the answer."""
    side, own = torch.cuda.Stream(), torch.cuda.Stream()
    ha = binding.HyperAttention(0)
    q, o = rows()
    bad = ints([0, 41])
    torch.cuda.synchronize()
    ha.set_options(dtype="bf16", stream=side.cuda_stream)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        ha.prompt(q, q, q, o, bad)
    ha.set_options(dtype="bf16", stream=own.cuda_stream)
    assert ha.status() == 0
    asked = 0
    for _ in range(300):
        with torch.cuda.stream(side):
            g.replay()
            done = side.record_event()
        while not done.query():
            asked += 1
            ha.status()
        with torch.cuda.stream(side):
            g.replay()
        side.synchronize()
        assert ha.status() == binding.HA_ERR_INVALID_ARG
    assert ha.status() == 0
    ha.close()


def test_report_of_a_call_right_behind_the_handles_creation():
    """The status word is cleared before hyper_attn_create returns, also when the default stream is busy."""
    side = torch.cuda.Stream()
    q, o = rows()
    bad = ints([0, 41])
    torch.cuda.synchronize()
    busy(torch.cuda.default_stream())
    ha = binding.HyperAttention(0)
    ha.set_options(dtype="bf16", stream=side.cuda_stream)
    ha.prompt(q, q, q, o, bad)
    side.synchronize()
    torch.cuda.synchronize()
    assert ha.status() == binding.HA_ERR_INVALID_ARG and ha.status() == 0
    ha.close()


def raw_capture(stream):
    """A capture begun and ended without torch's knowledge."""
    runtime = pytest.importorskip("cuda.bindings.runtime")

    class Capture:
        def __enter__(self):
            err, = runtime.cudaStreamBeginCapture(stream.cuda_stream, runtime.cudaStreamCaptureMode.cudaStreamCaptureModeGlobal)
            assert err == runtime.cudaError_t.cudaSuccess
            return self

        def __exit__(self, *_):
            err, graph = runtime.cudaStreamEndCapture(stream.cuda_stream)
            self.ok = err == runtime.cudaError_t.cudaSuccess
            if self.ok:
                runtime.cudaGraphDestroy(graph)

    return Capture()


def test_a_handle_made_while_a_stream_is_captured():
    """Making or closing a handle does not end a capture that is under way."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with raw_capture(side) as c:
        ha = binding.HyperAttention(0)
    assert c.ok
    ha.set_options(dtype="bf16", stream=side.cuda_stream)
    q, o = rows()
    torch.cuda.synchronize()
    ha.prompt(q, q, q, o, ints([0, 40]))
    assert ha.status() == 0
    with raw_capture(side) as c:
        binding.HyperAttention(0).close()
    assert c.ok
    ha.close()


def test_profile_of_eager_and_captured_calls():
    """A captured call has no time of its own: it is not recorded, and the calls around it are."""
    side = torch.cuda.Stream()
    ha = binding.HyperAttention(0)
    ha.set_options(dtype="bf16", stream=side.cuda_stream)
    q, o = rows()
    cu = ints([0, 40])
    torch.cuda.synchronize()
    ha.profile(True)
    ha.prompt(q, q, q, o, cu)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        ha.prompt(q, q, q, o, cu)
    ha.prompt(q, q, q, o, cu)
    with torch.cuda.stream(side):
        g.replay()
    ms, launches = ha.profile_read()["prompt"]
    assert launches == 2 and ms > 0
    assert ha.profile_read()["prompt"] == (0.0, 0)
    ha.profile(False)
    assert ha.status() == 0
    ha.close()


def decoding(ha):
    c = binding.PagedCache.empty(layers=1, pages=6, kv_heads=2, page=16, d=64, slots=1, max_pages=3)
    ha.cache_reserve(c, ints([0]), ints([20]))
    ha.cache_commit(c, ints([0]), ints([19]))
    q, o = rows(1)
    slots, at = ints([0]), ints([0, 1])
    ha.tree(q, c, o, slots, at, max_draft=1)       # eager once: the buffers' memory is there
    torch.cuda.synchronize()
    return lambda: ha.tree(q, c, o, slots, at, max_draft=1)


@pytest.mark.parametrize("current", [True, False])
def test_workspace_of_a_capture_that_torch_does_not_know_of(current):
    """Its buffer is kept for the graph's replays; memory that torch hands out afterwards is other memory."""
    side = torch.cuda.Stream()
    ha = binding.HyperAttention(0)
    ha.set_options(dtype="bf16", stream=side.cuda_stream)
    step = decoding(ha)
    nbytes = binding.lib().hyper_attn_tree_workspace(ha._h, 64)
    with torch.cuda.stream(side):
        spare = torch.empty(nbytes, dtype=torch.uint8, device="cuda")   # what the capture finds in torch's cache
    side.synchronize()
    del spare
    used = []
    real = ha._workspace
    ha._workspace = lambda n: used.append(real(n)) or used[-1]
    with torch.cuda.stream(side if current else torch.cuda.default_stream()):
        with raw_capture(side) as c:
            step()
            step()
    assert c.ok and len(used) == 2
    with torch.cuda.stream(side):
        later = [torch.empty(nbytes, dtype=torch.uint8, device="cuda") for _ in range(3)]
    for x in later:
        for p in used:
            assert x.data_ptr() + nbytes <= p or p + nbytes <= x.data_ptr()
    ha.close()


def test_workspaces_of_torch_graphs_are_the_graphs():
    """Torch's own captures have the buffers in the graph's pool: nothing is kept for them in the handle, and the calls of a
    graph, which run one after the other, have one buffer."""
    side = torch.cuda.Stream()
    ha = binding.HyperAttention(0)
    ha.set_options(dtype="bf16", stream=side.cuda_stream)
    step = decoding(ha)
    used = []
    real = ha._workspace
    ha._workspace = lambda n: used.append(real(n)) or used[-1]
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            for _ in range(3):
                step()
        graphs.append(g)
    assert not ha._captured
    assert len(set(used[:3])) == 1 and len(set(used[3:])) == 1 and used[0] != used[3]
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert ha.status() == 0
    ha.close()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("captured", [False, True])
def test_serving_calls_between_matrix_products(d, captured):
    """A step as a model makes it: products on the tensor cores before and behind every attention call, which start early on the
    stream. The results are those of each call on its own."""
    side = torch.cuda.Stream()
    ha = binding.HyperAttention(0)
    ha.set_options(dtype="bf16", stream=side.cuda_stream)
    g = torch.Generator(device="cuda").manual_seed(d)
    new = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    lens, hq, hk = [300, 41, 1, 700], 8, 2
    at = [0, 300, 341, 342, 1042]
    x, w, out = new(1042, 512), new(512, (hq + 2 * hk) * d) / 16, new(hq * d, 512) / 16
    c = binding.PagedCache.empty(layers=1, pages=40, kv_heads=hk, page=64, d=d, slots=4, max_pages=20)
    cu, slots, ones = ints(at), ints([0, 1, 2, 3]), ints([0, 1, 2, 3, 4])
    o, o1 = torch.empty(1042, hq, d, device="cuda", dtype=torch.bfloat16), torch.empty(4, hq, d, device="cuda", dtype=torch.bfloat16)
    last = torch.tensor(at[1:], device="cuda") - 1
    ints_lens, ints_one = ints(lens), ints([1] * 4)
    torch.cuda.synchronize()

    def heads(y):
        y = y.view(y.shape[0], hq + 2 * hk, d)
        return y[:, :hq], y[:, hq:hq + hk], y[:, hq + hk:]

    def step(wait):
        q, k, v = heads(x @ w)
        wait()
        ha.prompt(q, k, v, o, cu, max_len=700, scale=d ** -0.5)
        wait()
        y = o.view(1042, hq * d) @ out
        q1, k1, v1 = heads(y[last] @ w)
        wait()
        ha.cache_free(c, slots)
        ha.cache_reserve(c, slots, ints_lens)
        ha.cache_append(c, slots, cu, k[None], v[None])
        ha.cache_commit(c, slots, ints_lens)
        ha.cache_reserve(c, slots, ints_one)
        ha.cache_append(c, slots, ones, k1[None], v1[None])
        wait()
        ha.tree(q1, c, o1, slots, ones, max_draft=1, scale=d ** -0.5)
        wait()
        return y, o1.view(4, hq * d) @ out

    with torch.cuda.stream(side):
        want = [t.clone() for t in step(torch.cuda.synchronize)]
        torch.cuda.synchronize()
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                got = step(lambda: None)
            for _ in range(20):
                graph.replay()
        else:
            for _ in range(20):
                got = step(lambda: None)
        torch.cuda.synchronize()
    assert ha.status() == 0, ha.last_error()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    ha.close()

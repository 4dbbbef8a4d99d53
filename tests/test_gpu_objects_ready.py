"""Linear8 and AdamW on streams other than the one that they are made on, on a GB300: ready at once, and their memory theirs
until the last kernel that uses it has ended."""

import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
SLEEP = 20_000_000  # some ten milliseconds


@pytest.fixture(scope="module")
def P():
    from co_folding_pair_gb300 import train_ops
    return train_ops


def randn(*shape, seed=1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


def raw(t):
    return t.view(torch.uint8) if t.element_size() == 1 else t


def test_a_linear_layer_is_ready_for_any_stream(P):
    """The stream that it is made on is busy when its weight is laid out."""
    x, w, dy = randn(200, 64, seed=2).to(BF), randn(136, 64, seed=3), randn(200, 136, seed=4).to(BF)
    lin = P.Linear8(w)
    want = [lin(x), *(v for v in lin.backward(x, dy).values() if v is not None)]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    torch.cuda._sleep(SLEEP)
    lin = P.Linear8(w)
    lin.forward(x, stream=stream)
    got = [lin.forward(x, stream=stream), *(v for v in lin.backward(x, dy, stream=stream).values() if v is not None)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("states", ["float32", "8bit"])
def test_an_optimiser_is_ready_for_any_stream(P, states):
    """Its states are zeros, and the count, when the first step reads them."""
    sizes, g = [70000, 5, 1000], [randn(n, seed=n) for n in (70000, 5, 1000)]

    def after(busy):
        params = [torch.ones(n, device="cuda") for n in sizes]
        stream = torch.cuda.Stream()
        junk = torch.full((1 << 20,), 3.0, device="cuda")  # what the allocator gives out again is not zeros
        torch.cuda.synchronize()
        del junk
        if busy:
            torch.cuda._sleep(SLEEP)
        opt = P.AdamW(params, states=states, seed=3)
        opt.step(g, stream=stream)
        torch.cuda.synchronize()
        return [*params, *(raw(v).clone() for v in opt.state.values())]

    want = after(False)  # (a kernel's first launch may wait by itself)
    assert all(torch.equal(a, b) for a, b in zip(after(True), want))


def test_objects_may_be_made_in_a_capture(P):
    """Where waiting is not possible: the graph's order holds."""
    x, w = randn(64, 32, seed=5).to(BF), randn(40, 32, seed=6)
    p, g = torch.ones(300, device="cuda"), randn(300, seed=7)
    want = P.Linear8(w)(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lin, opt = P.Linear8(w), P.AdamW([p], lr=1e-2, weight_decay=0.0)
        y = lin(x)
        opt.step([g])
    for _ in range(2):
        y.zero_()
        graph.replay()
        assert torch.equal(y, want) and int(opt.state["count"]) == 1  # (the states are made anew in each replay)
    assert float((1 - p).abs().max()) < 0.03 and float((1 - p).abs().max()) > 0.01


@pytest.mark.parametrize("how", ["stream=", "current"])
def test_a_linear_layers_memory_outlives_its_last_call(P, how):
    """The object goes while another stream still has its call before it; the next tensor of its size is another's memory."""
    x, w, dy = randn(300, 256, seed=2).to(BF), randn(520, 256, seed=3), randn(300, 520, seed=4).to(BF)
    lin = P.Linear8(w)
    want = [lin(x), lin.backward(x, dy)["dx"]]
    stream = torch.cuda.Stream()
    y, dx = torch.empty_like(want[0]), torch.empty_like(want[1])
    torch.cuda.synchronize()
    lin, junk = P.Linear8(w), []
    with torch.cuda.stream(stream):
        torch.cuda._sleep(SLEEP)
        if how == "current":
            lin(x, out=y)
            lin.backward(x, dy, dx=dx, want=("dx",))
    if how == "stream=":
        lin(x, out=y, stream=stream)
        lin.backward(x, dy, dx=dx, want=("dx",), stream=stream)
    size = lin.packed.numel()
    del lin
    for _ in range(4):
        junk.append(torch.full((size,), 0x33, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(dx, want[1])


@pytest.mark.parametrize("states", ["float32", "8bit"])
def test_an_optimisers_memory_outlives_its_last_step(P, states):
    n = 300000
    g = randn(n, seed=1)

    def after(busy):
        p = torch.ones(n, device="cuda")
        stream = torch.cuda.Stream()
        opt = P.AdamW([p], states=states, seed=3)
        opt.step([g])
        torch.cuda.synchronize()
        if busy:
            with torch.cuda.stream(stream):
                torch.cuda._sleep(SLEEP)
        opt.step([g], stream=stream)
        sizes = [(v.numel(), v.dtype) for v in opt.state.values()]
        del opt
        junk = [torch.full((k,), 3, device="cuda").to(dt) for k, dt in sizes for _ in range(4)]
        torch.cuda.synchronize()
        del junk
        return p

    want = after(False)
    assert torch.equal(after(True), want)


def test_an_optimisers_dicts_go_by_name(P):
    """Gradients, copies and weight decays in another order than the parameters', of the same shape."""
    def after(flip):
        order = lambda d: dict(reversed(d.items())) if flip else d  # noqa: E731
        p = {"a": torch.ones(200, device="cuda"), "b": 2 * torch.ones(200, device="cuda")}
        copies = {k: torch.zeros(200, dtype=BF, device="cuda") for k in p}
        opt = P.AdamW(p, lr=0.1, weight_decay=order({"a": 0.0, "b": 0.5}), copies=order(copies))
        opt.step(order({"a": randn(200, seed=8), "b": randn(200, seed=9)}))
        return [*p.values(), *(copies[k] for k in p)]

    assert all(torch.equal(a, b) for a, b in zip(after(False), after(True)))


def test_a_refused_step_leaves_the_learning_rate(P):
    p, g = torch.ones(64, device="cuda"), randn(64, seed=8)
    opt = P.AdamW([p], lr=0.25)
    for bad in (float("nan"), torch.ones(2, device="cuda"), torch.ones(())):
        with pytest.raises(Exception, match="lr must be"):
            opt.step([g], lr=bad)
    with pytest.raises(Exception, match="its gradient has 8 elements"):
        opt.step([g[:8]], lr=1.0)
    assert opt.lr == 0.25 and int(opt.state["count"]) == 0
    opt.step([g], lr=0.5)
    assert opt.lr == 0.5 and int(opt.state["count"]) == 1


def test_objects_used_on_a_stream_that_is_gone(P):
    """A stream that torch does not own: the objects go after it, and their memory is given out again."""
    import ctypes
    x, w, g = randn(64, 32, seed=5).to(BF), randn(40, 32, seed=6), randn(300, seed=7)
    want = P.Linear8(w)(x)
    lin, opt = P.Linear8(w), P.AdamW([torch.ones(300, device="cuda")])
    cuda, handle = torch.cuda.cudart(), ctypes.c_uint64(0)
    assert int(cuda.cudaStreamCreate(ctypes.addressof(handle))) == 0
    stream = torch.cuda.ExternalStream(handle.value)
    y = torch.empty_like(want)
    torch.cuda.synchronize()
    lin(x, out=y, stream=stream)
    with torch.cuda.stream(stream):
        opt.step([g])
    stream.synchronize()
    assert torch.equal(y, want) and int(opt.state["count"]) == 1
    assert int(cuda.cudaStreamDestroy(handle.value)) == 0
    del lin, opt
    assert torch.equal(P.Linear8(w)(x), want)
    torch.cuda.synchronize()

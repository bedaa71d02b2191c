"""The norm's backward adds up the weight gradient in two launches that meet in a workspace: every call has its own,
whoever calls on whichever stream."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    import __graft_entry__
    __graft_entry__.build()
    from chunkwise_gated_linear_chunked_gb300 import binding
    return binding


def inputs(rows, D, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s, dy = (torch.randn(rows, D, device="cuda", generator=gen) for _ in range(2))
    return s, (s.square().mean(-1) + 1e-6).rsqrt(), dy


@pytest.mark.parametrize("checked", [True, False])
def test_two_threads_on_one_stream(B, monkeypatch, checked):
    """A call that another thread makes on the same stream while the first is inside the library (which it enters
    without the interpreter's lock) is given other memory for its partial sums."""
    side, w = torch.cuda.Stream(), torch.ones(256, device="cuda")
    a, b = inputs(4000, 256, 0), inputs(4000, 256, 1)
    torch.cuda.synchronize()
    seen, library, short = [], B._lib, B._calls

    def second():
        with torch.cuda.stream(side):
            B.norm_bwd(*b, weight=w, stream=side if checked else None)

    class Library:
        def __getattr__(self, name):
            return getattr(library, name)

        def gla_norm_bwd(self, *args):
            seen.append(args[11])
            if len(seen) == 1:
                other = threading.Thread(target=second)
                other.start()
                other.join()
            return library.gla_norm_bwd(*args)

    class Short:
        def __getattr__(self, name):
            return getattr(short, name)

        def norm_bwd(self, *args):
            if args[6] is not None:   # memory handed over by the binding
                seen.append(args[6].data_ptr())
            return short.norm_bwd(*args)

    monkeypatch.setattr(B, "_lib", Library())
    monkeypatch.setattr(B, "_calls", Short())
    dw = B.norm_bwd(*a, weight=w, stream=side)[2]
    torch.cuda.synchronize()
    assert len(seen) == len(set(seen)) and len(seen) >= (2 if checked else 1)
    ref = (a[2].double() * a[0].double() * a[1].double()[:, None]).sum(0)
    assert (dw - ref).norm() <= 1e-5 * ref.norm()


def test_two_streams_at_once(B):
    """Calls under way on two streams together, each with its own dy and several CTAs' partial sums: the bits of each
    alone."""
    w, sets = torch.ones(384, device="cuda"), [inputs(30000, 384, 2), inputs(30000, 384, 3)]
    alone = [B.norm_bwd(*x, weight=w) for x in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [B.norm_bwd(*x, weight=w, stream=s) for x, s in zip(sets, streams)]
        with torch.cuda.stream(streams[0]):
            got.append(B.norm_bwd(*sets[0], weight=w))   # and by the short way
        torch.cuda.synchronize()
        for a, b in zip(got, alone + alone[:1]):
            assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])


def test_replays_beside_calls(B):
    """A captured call and a plain one, replayed in turn on new inputs."""
    w, (s, rstd, dy) = torch.ones(512, device="cuda"), inputs(9000, 512, 4)
    B.norm_bwd(s, rstd, dy, weight=w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dx, _, dw = B.norm_bwd(s, rstd, dy, weight=w)
    for seed in (5, 6, 7):
        for t, new in zip((s, rstd, dy), inputs(9000, 512, seed)):
            t.copy_(new)
        graph.replay()
        other = B.norm_bwd(*inputs(9000, 512, 8), weight=w)[2]
        ref = B.norm_bwd(s, rstd, dy, weight=w)
        assert torch.equal(ref[0], dx) and torch.equal(ref[2], dw) and not torch.equal(other, dw)

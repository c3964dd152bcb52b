"""Calls on a given stream (``stream=``): what they allocate comes from that stream's memory.

Two hazards of a workspace or output taken from the caller's current stream, each made certain here by a stream
that is kept busy: the workspace, free again when the call returns, is the current stream's next allocation while
the kernels have yet to run; and a block that the current stream's earlier work still has to read becomes an
output that the kernels overwrite."""
import pytest
import torch

from gated_deltanet_linear_eqs_b200 import api
from gated_deltanet_linear_eqs_b200.inputs import cu_seqlens_from

pytestmark = pytest.mark.gpu

BUSY = 400_000_000  # cycles: a fifth of a second


def inputs(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x = {n: r(1, 4096, 4, 128).bfloat16() for n in ("q", "dy")}
    x.update({n: r(1, 4096, 2, 128).bfloat16() for n in "kv"})
    x.update(g=torch.log1p(-torch.exp2(-6.0 - torch.arange(4, device="cuda"))), cu=cu_seqlens_from([3000, 1096]).cuda(),
             s0=r(2, 4, 128, 128), alpha=torch.rand(1, 4096, 4, generator=g, device="cuda"),
             beta=torch.rand(1, 4096, 4, generator=g, device="cuda"), h=r(4096, 2048), w=r(2048), d_o=r(4096, 2048),
             pos=torch.arange(4096, device="cuda", dtype=torch.int32), f=api.gdn_rotary_inv_freq(128)[0].cuda())
    return x


CALLS = {
    "prompt": lambda x, **k: api.gdn_linear_attn(x["q"], x["k"], x["v"], x["g"], **k),
    "packed": lambda x, **k: api.gdn_linear_attn_varlen(x["q"], x["k"], x["v"], x["g"], x["cu"], s0=x["s0"], **k),
    "gradients": lambda x, **k: api.gdn_linear_attn_backward(x["q"], x["k"], x["v"], x["g"], x["dy"], **k),
    "packed gradients": lambda x, **k: api.gdn_linear_attn_backward_varlen(x["q"], x["k"], x["v"], x["g"], x["cu"],
                                                                           x["dy"], s0=x["s0"], **k),
    "norm gradients": lambda x, **k: api.gdn_add_rmsnorm_backward(x["h"], x["w"], x["d_o"], **k),
    "norm": lambda x, **k: api.gdn_add_rmsnorm(x["h"], x["d_o"], x["w"], **k),
    "norm to 8 bits": lambda x, **k: api.gdn_add_rmsnorm_fp8(x["h"], x["d_o"], x["w"], group=128, **k),
    "rotary": lambda x, **k: api.gdn_rotary(x["q"], x["k"], x["pos"][None], x["f"], **k),
    "delta rule": lambda x, **k: api.gdn_prefill(x["q"], x["q"], x["dy"], x["alpha"], x["beta"], **k),
}


def tensors(out):
    return [t for t in (out.values() if isinstance(out, dict) else out) if t is not None]


def same(a, b):
    return all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(tensors(a), tensors(b), strict=True))


@pytest.mark.parametrize("call", CALLS)
def test_allocations_are_the_given_streams(call):
    f, x = CALLS[call], inputs(1)
    want = f(x)
    torch.cuda.synchronize()
    sizes = {t.numel() * t.element_size() for t in tensors(want)}
    sizes |= {1 << n for n in range(16, 26)}
    side = torch.cuda.Stream()
    torch.cuda.empty_cache()
    # the workspace: nothing that the current stream allocates behind the call may be written by it
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    out = f(x, stream=side)
    mine = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sorted(sizes) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in mine)
    assert same(out, want)
    del out, mine
    # outputs: blocks that the current stream has freed but still reads must not become outputs
    torch.cuda.empty_cache()
    bufs = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sorted(sizes) for _ in range(3)]
    seen = [torch.empty_like(t) for t in bufs]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    for a, b in zip(seen, bufs):
        a.copy_(b)
    del bufs, a, b
    out = f(x, stream=side)
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in seen)
    assert same(out, want)


@pytest.mark.parametrize("call", ["prompt", "packed", "gradients", "packed gradients", "norm gradients", "delta rule"])
def test_two_streams_from_one(call):
    """Calls on two streams, issued in turn and without a workspace, against the same calls one by one; the outputs
    are used on the current stream afterwards and their memory is given back to their streams."""
    f, xs = CALLS[call], [inputs(s) for s in (1, 2)]
    want = [f(x) for x in xs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [f(x, stream=s) for x, s in zip(xs, streams)]
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        kept = [[t.clone() for t in tensors(g)] for g in got]
        del got
        assert all(same(k, w) for k, w in zip(kept, want))
    assert api.gdn_read_device_status() == 0


def test_a_foreign_stream_object():
    """An object that only carries a raw handle (another library's stream)."""
    side = torch.cuda.Stream()

    class Raw:
        cuda_stream = side.cuda_stream

    x = inputs(3)
    want = CALLS["packed"](x)
    torch.cuda.synchronize()
    got = CALLS["packed"](x, stream=Raw())
    torch.cuda.synchronize()
    assert same(got, want)


@pytest.mark.parametrize("call", ["packed", "packed gradients", "norm gradients", "rotary"])
def test_captured_on_a_forked_stream(call):
    """A graph whose capture forks to the given stream: workspace and outputs come from the graph's own memory."""
    f, x = CALLS[call], inputs(4)
    want = f(x)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        out = f(x, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    mine = [torch.full((1 << n,), 7, dtype=torch.uint8, device="cuda") for n in range(16, 26)]
    for _ in range(2):
        for t in tensors(out):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, want)
    assert all(bool((t == 7).all()) for t in mine)

"""GPU parity of the decayed linear attention (prompts, gradients, single tokens; through the C ABI)
against its fp64 oracle.

Tolerances, elementwise, from the roundings that a value passes through.  Let A be the same formula
with the absolute values of all inputs: every partial sum is at most A.
 * bf16 outputs: the scores (or the state) are rounded to bf16 once (half a step, 2^-8 of the value
   each at most, so 2^-8 A in the sum) and the output is rounded to bf16 (2^-8 |y|); fp32 sums add
   less than 2^-15 A.
 * fp32 outputs and states: products of at most 128 + 64 + 128 terms and up to 40 chunks, each step
   off by 2^-24 of a partial sum (the tensor cores' sums by 2^-23), decay factors by 2^-21: less than
   2^-15 A.
 * gradients of shared heads add the parts in fp32: within the same bounds."""
import numpy as np
import pytest
import torch

import oracle.linear_attn as oattn
from gated_deltanet_linear_eqs_b200 import _abi, api
from gated_deltanet_linear_eqs_b200.inputs import cu_seqlens_from

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def make(lens, H, Hk, d, dtype, seed=0, decay="mixed"):
    g = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    r = lambda *s: torch.randn(*s, generator=g)
    x = {n: r(T, h, d).to(DT[dtype]) for n, h in (("q", H), ("k", Hk), ("v", Hk), ("dy", H))}
    x["s0"], x["ds_final"] = 0.5 * r(N, H, d, d), 0.2 * r(N, H, d, d)
    ld = {"mixed": -torch.exp2(2.0 - 2.0 * torch.arange(H)), "none": torch.zeros(H),
          "slow": torch.log1p(-torch.exp2(-6.0 - torch.arange(H)))}[decay]
    if decay == "mixed":
        ld[-1] = 0.0
    x["log_decay"] = ld.float()
    x["cu_seqlens"] = cu_seqlens_from(lens)
    return x


def cuda(x):
    return {n: t.cuda() for n, t in x.items()}


def close(got, ref, mag, dtype, what):
    got = got.double().cpu().numpy()
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    tol = 2.0 ** -15 * mag + 1e-30
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * (mag + np.abs(ref)) * (1 + 2.0 ** -7)
    bad = np.abs(got - ref) > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.max(np.abs(got - ref) / tol):.3g} bounds"
    if dtype == "bf16" and ref.size >= 4096:
        # two independent roundings of at most half a step each, uniform in it: their root mean
        # square is at most sqrt(2) 2^-8 / sqrt(3) = 0.82 2^-8 of the values
        rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
        assert rel <= 2.0 ** -8, f"{what}: relative error {rel:.3g}"


def mags(x, scale):
    a = {n: (t.double().abs().numpy() if n != "log_decay" else t.double().numpy()) for n, t in x.items()}
    ya, sa = oattn.forward(a["q"], a["k"], a["v"], a["log_decay"], x["cu_seqlens"], s0=a["s0"], scale=scale)
    ga = oattn.backward(a["q"], a["k"], a["v"], a["log_decay"], x["cu_seqlens"], a["dy"], s0=a["s0"],
                        ds_final=a["ds_final"], scale=scale)
    return ya, sa, ga


LENS = [[1], [64], [65], [200], [1, 63, 0, 64, 2, 65, 0, 130], [0, 0, 3], [700, 0, 1, 640]]


@pytest.mark.parametrize("lens", LENS, ids=lambda l: "-".join(map(str, l)))
@pytest.mark.parametrize("H,Hk,d,dtype,decay", [
    (1, 1, 64, "fp32", "mixed"), (2, 2, 128, "fp32", "slow"), (4, 1, 64, "fp32", "none"),
    (1, 1, 64, "bf16", "slow"), (3, 3, 128, "bf16", "mixed"), (4, 2, 128, "bf16", "slow"),
    (6, 2, 64, "bf16", "none"), (1, 1, 128, "bf16", "none")])
def test_varlen_and_gradients(lens, H, Hk, d, dtype, decay):
    x = make(lens, H, Hk, d, dtype, seed=sum(lens) + H, decay=decay)
    scale = d ** -0.5
    c = cuda(x)
    y, sf = api.gdn_linear_attn_varlen(c["q"], c["k"], c["v"], c["log_decay"], c["cu_seqlens"], s0=c["s0"], scale=scale)
    out = api.gdn_linear_attn_backward_varlen(c["q"], c["k"], c["v"], c["log_decay"], c["cu_seqlens"], c["dy"],
                                              s0=c["s0"], ds_final=c["ds_final"], scale=scale)
    torch.cuda.synchronize()
    assert api.gdn_read_device_status() == 0
    ya, sa, ga = mags(x, scale)
    yr, sr = oattn.forward(x["q"], x["k"], x["v"], x["log_decay"], x["cu_seqlens"], s0=x["s0"], scale=scale)
    gr = oattn.backward(x["q"], x["k"], x["v"], x["log_decay"], x["cu_seqlens"], x["dy"], s0=x["s0"],
                        ds_final=x["ds_final"], scale=scale)
    close(y, yr, ya, dtype, "y")
    close(sf, sr, sa, "fp32", "s_final")
    for n in ("dq", "dk", "dv"):
        close(out[n], gr[n], ga[n], dtype, n)
    close(out["ds0"], gr["ds0"], ga["ds0"], "fp32", "ds0")


@pytest.mark.parametrize("B,T,H,Hk,d,dtype", [(2, 1, 2, 1, 64, "bf16"), (1, 1300, 1, 1, 128, "bf16"),
                                              (3, 129, 2, 2, 128, "bf16"), (2, 577, 4, 2, 64, "fp32")])
def test_dense_equals_packed(B, T, H, Hk, d, dtype):
    """Dense sequences against the oracle, without states as well."""
    x = make([T] * B, H, Hk, d, dtype, seed=T, decay="slow")
    c = cuda(x)
    b = lambda t: t.view(B, T, *t.shape[1:])
    scale = 0.3
    for states in (True, False):
        s0, dsf = (c["s0"], c["ds_final"]) if states else (None, None)
        y, sf = api.gdn_linear_attn(b(c["q"]), b(c["k"]), b(c["v"]), c["log_decay"], s0=s0, scale=scale,
                                    want_final=states)
        out = api.gdn_linear_attn_backward(b(c["q"]), b(c["k"]), b(c["v"]), c["log_decay"], b(c["dy"]), s0=s0,
                                           ds_final=dsf, scale=scale, want_ds0=states)
        torch.cuda.synchronize()
        assert api.gdn_read_device_status() == 0
        z = dict(x) if states else {**x, "s0": torch.zeros_like(x["s0"]), "ds_final": torch.zeros_like(x["ds_final"])}
        ya, sa, ga = mags(z, scale)
        yr, sr = oattn.forward(z["q"], z["k"], z["v"], z["log_decay"], z["cu_seqlens"], s0=z["s0"], scale=scale)
        gr = oattn.backward(z["q"], z["k"], z["v"], z["log_decay"], z["cu_seqlens"], z["dy"], s0=z["s0"],
                            ds_final=z["ds_final"], scale=scale)
        close(y.flatten(0, 1), yr, ya, dtype, "y")
        for n in ("dq", "dk", "dv"):
            close(out[n].flatten(0, 1), gr[n], ga[n], dtype, n)
        if states:
            close(sf, sr, sa, "fp32", "s_final")
            close(out["ds0"], gr["ds0"], ga["ds0"], "fp32", "ds0")
        else:
            assert sf is None and out["ds0"] is None


@pytest.mark.parametrize("what", ["cut", "cut evenly", "sorted", "as they come", "dense rounds"])
def test_many_chains(what):
    """More chains (documents times heads) than the GPU's 148 SMs, or a few that are cut into as many pieces."""
    rng = np.random.default_rng(len(what))
    H = {"cut": 1, "cut evenly": 4, "sorted": 4, "as they come": 1, "dense rounds": 1}[what]
    lens = {"cut": list(rng.integers(0, 9, 90)) + [1211, 0, 64, 777],  # pieces that hold many chains, and parts
            "cut evenly": [64 * 37, 64],
            "sorted": list(rng.integers(0, 140, 80)),
            "as they come": list(rng.integers(0, 90, 200)),
            "dense rounds": [66] * 300}[what]
    lens = [int(n) for n in lens]
    x = make(lens, H, 1, 64, "bf16", seed=3, decay="slow")
    c = cuda(x)
    b = lambda t: t.view(len(lens), lens[0], *t.shape[1:])
    if what == "dense rounds":
        y, sf = api.gdn_linear_attn(b(c["q"]), b(c["k"]), b(c["v"]), c["log_decay"], s0=c["s0"], scale=0.25)
        out = api.gdn_linear_attn_backward(b(c["q"]), b(c["k"]), b(c["v"]), c["log_decay"], b(c["dy"]), s0=c["s0"],
                                           ds_final=c["ds_final"], scale=0.25)
        y, out = y.flatten(0, 1), {n: t.flatten(0, 1) if n != "ds0" else t for n, t in out.items()}
    else:
        y, sf = api.gdn_linear_attn_varlen(c["q"], c["k"], c["v"], c["log_decay"], c["cu_seqlens"], s0=c["s0"],
                                           scale=0.25)
        out = api.gdn_linear_attn_backward_varlen(c["q"], c["k"], c["v"], c["log_decay"], c["cu_seqlens"], c["dy"],
                                                  s0=c["s0"], ds_final=c["ds_final"], scale=0.25)
    torch.cuda.synchronize()
    assert api.gdn_read_device_status() == 0
    ya, sa, ga = mags(x, 0.25)
    yr, sr = oattn.forward(x["q"], x["k"], x["v"], x["log_decay"], x["cu_seqlens"], s0=x["s0"], scale=0.25)
    gr = oattn.backward(x["q"], x["k"], x["v"], x["log_decay"], x["cu_seqlens"], x["dy"], s0=x["s0"],
                        ds_final=x["ds_final"], scale=0.25)
    close(y, yr, ya, "bf16", "y")
    close(sf, sr, sa, "fp32", "s_final")
    for n in ("dq", "dk", "dv"):
        close(out[n], gr[n], ga[n], "bf16", n)
    close(out["ds0"], gr["ds0"], ga["ds0"], "fp32", "ds0")


def test_gradients_against_differences():
    """fp32, the sum of y dy + s_final ds_final: a central difference along a random direction is exact for a
    function that is linear in each tensor, up to the fp32 rounding of the two losses."""
    x = make([70, 3], 2, 1, 64, "fp32", seed=5)
    c = cuda(x)
    g = api.gdn_linear_attn_backward_varlen(c["q"], c["k"], c["v"], c["log_decay"], c["cu_seqlens"], c["dy"],
                                            s0=c["s0"], ds_final=c["ds_final"], scale=0.2)

    def loss(a):
        y, s = api.gdn_linear_attn_varlen(a["q"], a["k"], a["v"], a["log_decay"], a["cu_seqlens"], s0=a["s0"], scale=0.2)
        return float((y.double() * a["dy"].double()).sum() + (s.double() * a["ds_final"].double()).sum())

    gen = torch.Generator(device="cuda").manual_seed(0)
    for n in ("q", "k", "v", "s0"):
        e = torch.randn(c[n].shape, generator=gen, device="cuda")
        num = (loss({**c, n: c[n] + e}) - loss({**c, n: c[n] - e})) / 2
        ref = float((g["d" + n].double() * e.double()).sum())
        terms = float((g["d" + n].double() * e.double()).square().sum().sqrt())
        # rounding of 10^5 outputs of size ~100 at 2^-18 each, adding at random: 2^-18 * 100 * 300
        assert abs(num - ref) <= 0.2 + 1e-4 * terms, (n, num, ref)


@pytest.mark.parametrize("N,H,Hk,d,dtype", [(1, 1, 1, 64, "bf16"), (5, 6, 2, 128, "bf16"), (3, 2, 2, 128, "fp32"),
                                            (33, 4, 1, 64, "fp32")])
def test_decode_steps(N, H, Hk, d, dtype):
    """Ten steps against the oracle's token loop (each step starts from the oracle's bounds of the last)."""
    steps = 10
    x = make([steps] * N, H, Hk, d, dtype, seed=N)
    c = cuda(x)
    b = lambda t: t.view(N, steps, *t.shape[1:])
    st = c["s0"].clone()
    ys = [api.gdn_linear_attn_decode_step(b(c["q"])[:, t].contiguous(), b(c["k"])[:, t].contiguous(),
                                          b(c["v"])[:, t].contiguous(), c["log_decay"], st, scale=0.25)
          for t in range(steps)]
    y = torch.stack(ys, 1).flatten(0, 1)
    yr, sr = oattn.forward(x["q"], x["k"], x["v"], x["log_decay"], x["cu_seqlens"], s0=x["s0"], scale=0.25)
    ya, sa, _ = mags(x, 0.25)
    close(st, sr, sa, "fp32", "state")
    close(y, yr, ya, dtype, "y")


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("fp32", 64)])
def test_resume_and_long_segments(dtype, d):
    """A prompt in two calls equals one; cut into many segments (one head, 5000 tokens) it equals the oracle."""
    x = make([5000], 1, 1, d, dtype, seed=9, decay="slow")
    c = cuda(x)
    a = (c["log_decay"],)
    y, sf = api.gdn_linear_attn(*(c[n][None] for n in "qkv"), *a, s0=c["s0"], scale=0.1)
    y1, s1 = api.gdn_linear_attn(*(c[n][None, :1999].contiguous() for n in "qkv"), *a, s0=c["s0"], scale=0.1)
    y2, s2 = api.gdn_linear_attn(*(c[n][None, 1999:].contiguous() for n in "qkv"), *a, s0=s1, scale=0.1)
    ya, sa, _ = mags(x, 0.1)
    yr, sr = oattn.forward(x["q"], x["k"], x["v"], x["log_decay"], x["cu_seqlens"], s0=x["s0"], scale=0.1)
    close(y[0], yr, ya, dtype, "y")
    close(torch.cat([y1, y2], 1)[0], yr, ya, dtype, "y in two calls")
    close(sf, sr, sa, "fp32", "s_final")
    close(s2, sr, sa, "fp32", "s_final in two calls")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_other_documents_and_heads_are_untouched(dtype):
    """NaN and infinities in one document (up to its last, partial chunk) reach no other document, no other
    head, and nothing before their 64-token chunk; rows behind the last document stay as they were."""
    lens, H, d = [70, 100, 40], 2, 128
    x = make(lens, H, H, d, dtype, seed=3, decay="slow")
    c = cuda(x)
    T = sum(lens)
    run = lambda c, y=None: api.gdn_linear_attn_varlen(c["q"], c["k"], c["v"], c["log_decay"], c["cu_seqlens"],
                                                       s0=c["s0"], y=y)
    back = lambda c: api.gdn_linear_attn_backward_varlen(c["q"], c["k"], c["v"], c["log_decay"], c["cu_seqlens"],
                                                         c["dy"], s0=c["s0"], ds_final=c["ds_final"])
    y0, s0 = run(c)
    b0 = back(c)
    z = {n: t.clone() for n, t in c.items()}
    for n in ("q", "k", "v", "dy"):
        z[n][170 - 30:170, 0] = float("nan")     # the second document's last 30 tokens, head 0
        z[n][170 - 20, 0, 5] = float("inf")
    buf = torch.full((T + 3, H, d), 7.0, dtype=DT[dtype], device="cuda")
    y1, s1 = run(z, y=buf[:T])
    b1 = back(z)
    torch.cuda.synchronize()
    assert torch.equal(y1[:134], y0[:134]) and torch.equal(y1[170:], y0[170:]) and torch.equal(y1[:, 1], y0[:, 1])
    assert torch.equal(s1[[0, 2]], s0[[0, 2]]) and torch.equal(s1[:, 1], s0[:, 1])
    assert bool((buf[T:] == 7.0).all())
    for n in ("dq", "dk", "dv"):
        assert torch.equal(b1[n][:70], b0[n][:70]) and torch.equal(b1[n][170:], b0[n][170:])
        assert torch.equal(b1[n][:, 1], b0[n][:, 1])
    assert torch.equal(b1["ds0"][[0, 2]], b0["ds0"][[0, 2]])


@pytest.mark.parametrize("lens,bad", [([1500, 90, 0, 65], (1400, 1405)), ([1500, 90, 0, 65], (1590, 1591)),
                                      ([1500, 90, 0, 65], (64, 65)), ([40, 3] * 40, (43 * 20, 43 * 20 + 40))])
def test_shared_walks_keep_chains_apart(lens, bad):
    """CTAs that walk several chains, or parts of them, one after the other (a cut, and 320 chains on 148 SMs): tokens
    that are not finite reach only their own document and head, forward from (backward: up to) their chunk; rows
    behind the last document and states of others stay."""
    H, d, N, T = 4, 64, len(lens), sum(lens)
    x = make(lens, H, 2, d, "bf16", seed=5, decay="slow")
    c = cuda(x)
    cu = [0] + list(np.cumsum(lens))
    n = next(i for i in range(N) if cu[i] <= bad[0] < cu[i + 1])
    first = cu[n] + (bad[0] - cu[n]) // 64 * 64
    z = {k: t.clone() for k, t in c.items()}
    for k in ("q", "dy"):
        z[k][bad[0]:bad[1], 2] = float("nan")
    pad = {k: torch.cat([t, torch.full_like(t[:70], float("nan"))]) if k in ("q", "k", "v", "dy") else t
           for k, t in z.items()}  # the stream is longer than its documents
    run = lambda a, y: api.gdn_linear_attn_varlen(a["q"], a["k"], a["v"], a["log_decay"], a["cu_seqlens"],
                                                  s0=a["s0"], y=y)
    back = lambda dy: api.gdn_linear_attn_backward_varlen(c["q"], c["k"], c["v"], c["log_decay"], c["cu_seqlens"], dy,
                                                          s0=c["s0"])
    buf = torch.full((T + 70, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    y0, s0 = run({k: torch.cat([t, torch.zeros_like(t[:70])]) if k in ("q", "k", "v", "dy") else t
                  for k, t in c.items()}, None)
    y1, s1 = run(pad, buf)
    b0, b1 = back(c["dy"]), back(z["dy"])
    torch.cuda.synchronize()
    assert api.gdn_read_device_status() == 0
    keep = torch.ones(T, H, dtype=torch.bool, device="cuda")
    keep[bad[0]:bad[1], 2] = False
    assert torch.equal(y1[:T][keep], y0[:T][keep]) and bool((buf[T:] == 7.0).all())  # q reaches its own row alone
    assert torch.equal(s1, s0)
    keep[bad[0]:bad[1]] = True
    keep[first:cu[n + 1], 2] = False  # dq: rows of the chunk on; dk, dv (heads 2, 3 share theirs): up to its end
    assert torch.equal(b1["dq"][keep], b0["dq"][keep])
    for k in ("dk", "dv"):
        keep = torch.ones(T, 2, dtype=torch.bool, device="cuda")
        keep[cu[n]:first + 64, 1] = False
        assert torch.equal(b1[k][keep], b0[k][keep])
    keep = torch.ones(N, H, dtype=torch.bool, device="cuda")
    keep[n, 2] = False
    assert torch.equal(b1["ds0"][keep], b0["ds0"][keep])


@pytest.mark.parametrize("d", [64, 128])
def test_one_long_chain(d):
    """One head's 20011 tokens over all SMs, with its gradients."""
    x = make([20011], 1, 1, d, "bf16", seed=d, decay="slow")
    c = cuda(x)
    y, sf = api.gdn_linear_attn_varlen(c["q"], c["k"], c["v"], c["log_decay"], c["cu_seqlens"], s0=c["s0"], scale=0.1)
    out = api.gdn_linear_attn_backward_varlen(c["q"], c["k"], c["v"], c["log_decay"], c["cu_seqlens"], c["dy"],
                                              s0=c["s0"], ds_final=c["ds_final"], scale=0.1)
    torch.cuda.synchronize()
    assert api.gdn_read_device_status() == 0
    ya, sa, ga = mags(x, 0.1)
    yr, sr = oattn.forward(x["q"], x["k"], x["v"], x["log_decay"], x["cu_seqlens"], s0=x["s0"], scale=0.1)
    gr = oattn.backward(x["q"], x["k"], x["v"], x["log_decay"], x["cu_seqlens"], x["dy"], s0=x["s0"],
                        ds_final=x["ds_final"], scale=0.1)
    close(y, yr, ya, "bf16", "y")
    close(sf, sr, sa, "fp32", "s_final")
    for n in ("dq", "dk", "dv"):
        close(out[n], gr[n], ga[n], "bf16", n)
    close(out["ds0"], gr["ds0"], ga["ds0"], "fp32", "ds0")


def test_same_result_every_time_and_captured():
    """Runs are bit-equal; a captured graph replays them on new inputs; two streams with a workspace each."""
    x = make([900, 70, 1], 2, 1, 128, "bf16", seed=1, decay="slow")
    z = make([900, 70, 1], 2, 1, 128, "bf16", seed=2, decay="slow")
    c, w = cuda(x), cuda(z)
    n = api.gdn_linear_attn_workspace_bytes(1, 971, 2, 1, 128, 128, 3, backward=True)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]

    def both(c, ws):
        y, s = api.gdn_linear_attn_varlen(c["q"], c["k"], c["v"], c["log_decay"], c["cu_seqlens"], s0=c["s0"], ws=ws)
        g = api.gdn_linear_attn_backward_varlen(c["q"], c["k"], c["v"], c["log_decay"], c["cu_seqlens"], c["dy"],
                                                s0=c["s0"], ds_final=c["ds_final"], ws=ws)
        return [y, s, g["dq"], g["dk"], g["dv"], g["ds0"]]

    ref, ref2 = both(c, ws[0]), both(w, ws[0])
    assert all(torch.equal(a, b) for a, b in zip(ref, both(c, ws[0])))
    static = {k: t.clone() for k, t in c.items()}
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = both(static, ws[0])
    for src, want in ((c, ref), (w, ref2), (c, ref)):
        for k, t in src.items():
            static[k].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        o1 = both(c, ws[0])
    with torch.cuda.stream(s2):
        o2 = both(w, ws[1])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(o1, ref)) and all(torch.equal(a, b) for a, b in zip(o2, ref2))
    assert api.gdn_read_device_status() == 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_falling_offsets_stay_inside(dtype):
    """Offsets that fall and rise again are not allowed (their results mean nothing) but lead nowhere outside the
    tensors: three documents, the first and the last over the whole stream, have more segments than the stream's
    length and the documents' number make room for.  The workspace is NaN where no pass has written it."""
    T, H, d = 512, 1, 64
    x = make([T], H, H, d, dtype, seed=11, decay="slow")
    c = cuda(x)
    cu = torch.tensor([0, T, 0, T], dtype=torch.int32, device="cuda")
    s0, dsf = c["s0"].repeat(3, 1, 1, 1), c["ds_final"].repeat(3, 1, 1, 1)
    n = api.gdn_linear_attn_workspace_bytes(1, T, H, H, d, d, 3, backward=True)
    ws = torch.full((n // 4,), float("nan"), device="cuda")
    y, sf = api.gdn_linear_attn_varlen(c["q"], c["k"], c["v"], c["log_decay"], cu, s0=s0, ws=ws)
    ws.fill_(float("nan"))
    g = api.gdn_linear_attn_backward_varlen(c["q"], c["k"], c["v"], c["log_decay"], cu, c["dy"], s0=s0, ds_final=dsf, ws=ws)
    torch.cuda.synchronize()
    assert api.gdn_read_device_status() == 0
    for t in (y, *g.values()):
        assert bool(torch.isfinite(t).all())


def far_decays(H):
    """Decays of about 2^-14 a token whose e^{64 g} lies nearly half a step from its nearest float: in one float they
    would be off by H 2^-25 and more after H chunks."""
    g = []
    for h in range(H):
        x = np.float32(-(2.0 ** -14) * (1 + h / 3))
        while True:
            e = np.exp(64.0 * np.float64(x))
            off = (e - np.float64(np.float32(e))) / np.spacing(np.float32(e))
            if abs(off) > 0.45 and (off > 0) == (h % 2 == 0):
                break
            x = np.nextafter(x, np.float32(-1))
        g.append(x)
    return torch.tensor(np.array(g))


def relative(got, ref):
    return float(np.linalg.norm(got.double().cpu().numpy() - ref) / np.linalg.norm(ref))


# What fp32 states and outputs may be off by, relative, as 2-norms.  In each of about 256 chunks that a state with this
# decay remembers one rounding of it, 2^-24 / sqrt(3) in the root mean square: sixteen of them, 2^-20.8, where all are of
# a value just above a power of two (2^-21.3 as they come); the chunk's own sums 2^-22 (products in parts, sums in the
# tensor cores that are cut off below 2^-23).  A decay in one float, off by 0.45 2^-24 a chunk, would be off by 100 and
# more chunks' worth: 2^-18.5.
STATE_TOL = 2.0 ** -20


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("fp32", 64)])
@pytest.mark.parametrize("walk", ["cut", "in turn"])
def test_states_keep_fp32_accuracy(dtype, d, walk):
    """Long chains with weak decays, the last chunk short: cut into pieces, and uncut (more chains than SMs, so that
    some start where their CTA has walked another one)."""
    H, T, B = 3, 16411, 1 if walk == "cut" else 50
    g = torch.Generator(device="cuda").manual_seed(d)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    q, k, v, dy = (r(B, T, H, d).to(DT[dtype]) for _ in range(4))
    s0, dsf, ld = 8 * r(B, H, d, d), 8 * r(B, H, d, d), far_decays(H)
    y, sf = api.gdn_linear_attn(q, k, v, ld.cuda(), s0=s0, scale=0.1)
    out = api.gdn_linear_attn_backward(q, k, v, ld.cuda(), dy, s0=s0, ds_final=dsf, scale=0.1)
    torch.cuda.synchronize()
    assert api.gdn_read_device_status() == 0
    for b in sorted({0, B // 2, B - 1}):
        x = [t[b].cpu() for t in (q, k, v)]
        yr, sr = oattn.forward(*x, ld, [0, T], s0=s0[b:b + 1].cpu(), scale=0.1)
        gr = oattn.backward(*x, ld, [0, T], dy[b].cpu(), s0=s0[b:b + 1].cpu(), ds_final=dsf[b:b + 1].cpu(), scale=0.1)
        err = {"s_final": relative(sf[b], sr[0]), "ds0": relative(out["ds0"][b], gr["ds0"][0])}
        if dtype == "fp32":
            err.update(y=relative(y[b], yr), **{n: relative(out[n][b], gr[n]) for n in ("dq", "dk", "dv")})
        print(walk, dtype, d, b, err)
        assert max(err.values()) <= STATE_TOL, err


def test_documents_do_not_depend_on_each_other():
    """bf16, uncut: a document gives the same bits alone and among 79 others, wherever its CTA stood before."""
    rng = np.random.default_rng(4)
    H, d = 4, 64
    lens = [int(n) for n in rng.integers(0, 1000, 80)]
    x = make(lens, H, 2, d, "bf16", seed=7, decay="slow")
    x["log_decay"] = far_decays(H) * 16
    c = cuda(x)
    y, sf = api.gdn_linear_attn_varlen(c["q"], c["k"], c["v"], c["log_decay"], c["cu_seqlens"], s0=c["s0"], scale=0.25)
    out = api.gdn_linear_attn_backward_varlen(c["q"], c["k"], c["v"], c["log_decay"], c["cu_seqlens"], c["dy"],
                                              s0=c["s0"], ds_final=c["ds_final"], scale=0.25)
    at = 0
    for i, n in enumerate(lens):
        if n == 0:
            continue
        one = {m: c[m][at:at + n].contiguous()[None] for m in ("q", "k", "v", "dy")}
        s0, dsf = c["s0"][i:i + 1], c["ds_final"][i:i + 1]
        y1, s1 = api.gdn_linear_attn(one["q"], one["k"], one["v"], c["log_decay"], s0=s0, scale=0.25)
        o1 = api.gdn_linear_attn_backward(one["q"], one["k"], one["v"], c["log_decay"], one["dy"], s0=s0, ds_final=dsf,
                                          scale=0.25)
        assert torch.equal(y1[0], y[at:at + n]) and torch.equal(s1[0], sf[i]), (i, n)
        assert all(torch.equal(o1[m][0], out[m][at:at + n]) for m in ("dq", "dk", "dv")), (i, n)
        assert torch.equal(o1["ds0"][0], out["ds0"][i]), (i, n)
        at += n
    assert api.gdn_read_device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("H,Hk", [(4, 1), (4, 2), (2, 2)])
@pytest.mark.parametrize("lens", [[70, 0, 100], [1500, 65]], ids=["short", "long"])
def test_rows_outside_the_documents_are_left(lens, H, Hk, dtype):
    """A stream that is longer than its documents (a padded batch, its rows NaN): outputs and gradients behind the last
    document keep what they held, shared heads or not, and the others are those of the stream without them."""
    d, T, more = 64, sum(lens), 77
    x = make(lens, H, Hk, d, dtype, seed=T + Hk, decay="slow")
    c = cuda(x)
    N = len(lens)
    want = [api.gdn_linear_attn_varlen(c["q"], c["k"], c["v"], c["log_decay"], c["cu_seqlens"], s0=c["s0"])[0]]
    g = api.gdn_linear_attn_backward_varlen(c["q"], c["k"], c["v"], c["log_decay"], c["cu_seqlens"], c["dy"], s0=c["s0"])
    want += [g["dq"], g["dk"], g["dv"]]
    p = {n: torch.cat([c[n], torch.full_like(c[n][:more], float("nan"))]) for n in ("q", "k", "v", "dy")}
    out = [torch.full((T + more, h, d), 7.0, dtype=DT[dtype], device="cuda") for h in (H, H, Hk, Hk)]
    ds0 = torch.empty_like(c["s0"])
    n = api.gdn_linear_attn_workspace_bytes(1, T + more, H, Hk, d, d, N, backward=True)
    ws = torch.full((n // 4 + 4,), float("nan"), device="cuda")
    api.gdn_linear_attn_varlen(p["q"], p["k"], p["v"], c["log_decay"], c["cu_seqlens"], s0=c["s0"], y=out[0], ws=ws)
    rc = _abi.load().gdn_linear_attn_backward_varlen(
        *(p[n].data_ptr() for n in "qkv"), c["log_decay"].data_ptr(), c["cu_seqlens"].data_ptr(), N, c["s0"].data_ptr(),
        p["dy"].data_ptr(), None, *(t.data_ptr() for t in out[1:]), ds0.data_ptr(), T + more, H, Hk, d, d,
        _abi.GDN_BF16 if dtype == "bf16" else _abi.GDN_FP32, 1.0, ws.data_ptr(), ws.numel() * 4,
        torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0 and api.gdn_read_device_status() == 0
    for a, b in zip(out, want):
        assert bool((a[T:] == 7.0).all())
        # the cuts may fall elsewhere: two results, each off by two bf16 roundings (2^-8.7 in the root mean square, most of
        # it alike), or by 2^-20
        rel = float((a[:T].double() - b.double()).norm() / b.double().norm())
        assert rel <= (2.0 ** -8 if dtype == "bf16" else 2.0 ** -19), rel
    assert bool(torch.isfinite(ds0).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_scaled_inputs_give_the_same_bits(dtype):
    """Powers of two are exact in every product, part and sum: k times 2^-100 with v times 2^100 is the same call."""
    x = make([200, 65], 2, 1, 128, dtype, seed=12, decay="slow")
    c = cuda(x)
    z = {**c, "k": c["k"] * 2.0 ** -100, "v": c["v"] * 2.0 ** 100}
    f = lambda a: api.gdn_linear_attn_varlen(a["q"], a["k"], a["v"], a["log_decay"], a["cu_seqlens"], s0=a["s0"], scale=0.1)
    g = lambda a: api.gdn_linear_attn_backward_varlen(a["q"], a["k"], a["v"], a["log_decay"], a["cu_seqlens"], a["dy"],
                                                      s0=a["s0"], scale=0.1)
    for a, b in zip(f(c), f(z)):
        assert torch.equal(a, b)
    a, b = g(c), g(z)
    assert torch.equal(a["dq"], b["dq"]) and torch.equal(a["ds0"], b["ds0"])
    assert torch.equal(a["dk"] * 2.0 ** 100, b["dk"]) and torch.equal(a["dv"] * 2.0 ** -100, b["dv"])

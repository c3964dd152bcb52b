"""The layer operators together, as a layer uses them: norm with the residual, projections (torch), rotary
positions, decayed linear attention, gated RMSNorm, output projection; a prompt, its gradients, and single
tokens that continue from its states.  Against the same layer in fp64 with torch's autograd, on the CPU.

Tolerances, of a tensor's relative error (2-norms):
 * fp32: eight operators in a row, each within 2^-15 of its outputs' norm: 2^-12.
 * bf16: an output has about sixteen roundings behind it (the norm's output; q, k and v and their
   turned values, each of the three with the norm's; scores or state; y; z; the gated norm; the
   output), independent and of a root mean square of at most 2^-8 / sqrt(3): together 4 / sqrt(3) 2^-8
   = 2^-6.8.  Sigmoid and norms do not enlarge a relative error: 2^-6."""
import pytest
import torch

from gated_deltanet_linear_eqs_b200 import api
from gated_deltanet_linear_eqs_b200.inputs import cu_seqlens_from

pytestmark = pytest.mark.gpu

C, H, HK, D, EPS, SCALE = 256, 4, 2, 64, 1e-6, 64 ** -0.5
TOL = {torch.float32: 2.0 ** -12, torch.bfloat16: 2.0 ** -6}
WIDTHS = (H * D, HK * D, HK * D, H * D)


def make(lens, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    T, N = sum(lens), len(lens)
    f, _ = api.gdn_rotary_inv_freq(D)
    x = {"x": r(T, C).to(dtype), "res": r(T, C).to(dtype), "d_out": r(T, C).to(dtype), "d_h": r(T, C).to(dtype),
         "proj": (r(C, sum(WIDTHS)) * C ** -0.5).to(dtype), "out": (r(H * D, C) * (H * D) ** -0.5).to(dtype),
         "w": 0.2 * r(C), "wg": 0.2 * r(D), "s0": 0.5 * r(N, H, D, D), "ds": 0.2 * r(N, H, D, D),
         "g": torch.log1p(-torch.exp2(-2.0 - torch.arange(H))), "f": f,
         "pos": torch.cat([torch.arange(n) + 1000 * i for i, n in enumerate(lens)]).int(),
         "cu": cu_seqlens_from(lens)}
    return x


def norm64(h, w):
    return (1 + w) * h / torch.sqrt(h.square().mean(-1, keepdim=True) + EPS)


def rotary64(x, pos, f):
    a = pos.double()[:, None, None] * f.double()
    u, v = x.chunk(2, -1)
    return torch.cat([u * a.cos() - v * a.sin(), v * a.cos() + u * a.sin()], -1)


def layer64(x, lens):
    """Everything in fp64; returns (out, h, states)."""
    h = x["x"] + x["res"]
    q, k, v, z = (norm64(h, x["w"]) @ x["proj"]).split(WIDTHS, -1)
    q, k, v, z = (t.unflatten(-1, (-1, D)) for t in (q, k, v, z))
    q, k = rotary64(q, x["pos"], x["f"]), rotary64(k, x["pos"], x["f"])
    k, v = (t.repeat_interleave(H // HK, 1) for t in (k, v))
    ys, states, at = [], [], 0
    for n, L in enumerate(lens):
        a = slice(at, at + L)
        at += L
        i = torch.arange(L)
        e = (i[:, None] - i[None, :]).clamp(min=0) * x["g"][:, None, None]
        P = torch.einsum("ihd,jhd->hij", q[a], k[a]) * torch.exp(e).tril()
        y = torch.einsum("hij,jhv->ihv", P, v[a])
        y = y + torch.exp((i[:, None] + 1) * x["g"])[..., None] * torch.einsum("ihk,hkv->ihv", q[a], x["s0"][n])
        ys.append(SCALE * y)
        wts = torch.exp((L - 1 - i)[:, None] * x["g"])
        states.append(torch.exp(L * x["g"])[:, None, None] * x["s0"][n]
                      + torch.einsum("jhk,jhv->hkv", k[a] * wts[..., None], v[a]))
    o = torch.sigmoid(z) * norm64(torch.cat(ys), x["wg"])
    return o.flatten(1) @ x["out"], h, torch.stack(states)


def layer(x, saved=None):
    """The framework's calls.  Returns (out, h, states)."""
    o, h = api.gdn_add_rmsnorm(x["x"], x["res"], x["w"], eps=EPS)
    q, k, v, z = (t.unflatten(-1, (-1, D)) for t in (o @ x["proj"]).split(WIDTHS, -1))
    v, z = v.contiguous(), z.contiguous()
    q, k = api.gdn_rotary(q, k, x["pos"], x["f"])  # views into the projection
    y, states = api.gdn_linear_attn_varlen(q, k, v, x["g"], x["cu"], s0=x["s0"], scale=SCALE)
    out = api.gdn_gated_rmsnorm(y, z, x["wg"], eps=EPS).flatten(1) @ x["out"]
    if saved is not None:
        saved.update(h=h, q=q, k=k, v=v, y=y, z=z)
    return out, h, states


def layer_backward(x, s):
    d_o = (x["d_out"] @ x["out"].t()).unflatten(-1, (H, D))
    g = api.gdn_gated_rmsnorm_backward(s["y"], s["z"], x["wg"], d_o, eps=EPS)
    a = api.gdn_linear_attn_backward_varlen(s["q"], s["k"], s["v"], x["g"], x["cu"], g["dy"], s0=x["s0"],
                                            ds_final=x["ds"], scale=SCALE)
    d = torch.empty(x["x"].shape[0], sum(WIDTHS), dtype=x["x"].dtype, device="cuda")
    dq, dk, dv, dz = (t.unflatten(-1, (-1, D)) for t in d.split(WIDTHS, -1))
    api.gdn_rotary(a["dq"], a["dk"], x["pos"], x["f"], inverse=True, q_out=dq, k_out=dk)
    dv.copy_(a["dv"])
    dz.copy_(g["dz"])
    n = api.gdn_add_rmsnorm_backward(s["h"], x["w"], d @ x["proj"].t(), d_h=x["d_h"], eps=EPS)
    return {"x": n["dx"], "w": n["dw"], "s0": a["ds0"]}


def check(got, ref, tol, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    e = float((got - ref).norm() / ref.norm())
    assert e <= tol, f"{what}: relative error {e:.3g} > {tol:.3g}"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("lens", [[70, 0, 1, 130], [300]], ids=["documents", "one"])
def test_layer_prompt_gradients_and_tokens(lens, dtype):
    x = make(lens, dtype, seed=sum(lens))
    leaves = ("x", "w", "s0")
    x64 = {n: t.double() if t.is_floating_point() else t for n, t in x.items()}
    for n in leaves:
        x64[n].requires_grad_()
    out64, h64, st64 = layer64(x64, lens)
    loss = (out64 * x64["d_out"]).sum() + (h64 * x64["d_h"]).sum() + (st64 * x64["ds"]).sum()
    grads = dict(zip(leaves, torch.autograd.grad(loss, [x64[n] for n in leaves])))
    c = {n: t.cuda() for n, t in x.items()}
    saved = {}
    out, h, states = layer(c, saved)
    got = layer_backward(c, saved)
    torch.cuda.synchronize()
    assert api.gdn_read_device_status() == 0
    check(out, out64.detach(), TOL[dtype], "out")
    check(h, h64.detach(), TOL[dtype], "h")
    check(states, st64.detach(), TOL[dtype], "states")
    for n in leaves:
        check(got[n], grads[n], TOL[dtype], "d" + n)

    # three single tokens of every document, behind the prompt
    steps, N = 3, len(lens)
    more = make([steps] * N, dtype, seed=99)
    full = dict(x64)
    for n in ("x", "res"):
        new = more[n].double().unflatten(0, (N, steps))
        full[n] = torch.cat([torch.cat([a, b]) for a, b in zip(x64[n].detach().split(lens), new)])
    first = torch.tensor([1000 * i + n for i, n in enumerate(lens)])
    full["pos"] = torch.cat([torch.arange(n + steps) + 1000 * i for i, n in enumerate(lens)])
    out64, _, st64 = layer64(full, [n + steps for n in lens])
    last = [t[-steps:] for t in out64.detach().split([n + steps for n in lens])]
    xt, rt = (more[n].cuda().unflatten(0, (N, steps)) for n in ("x", "res"))
    for j in range(steps):
        o, _ = api.gdn_add_rmsnorm(xt[:, j].contiguous(), rt[:, j].contiguous(), c["w"], eps=EPS)
        q, k, v, z = (t.unflatten(-1, (-1, D)) for t in (o @ c["proj"]).split(WIDTHS, -1))
        q, k = api.gdn_rotary(q, k, (first + j).int().cuda(), c["f"])
        y = api.gdn_linear_attn_decode_step(q, k, v.contiguous(), c["g"], states, scale=SCALE)
        out = api.gdn_gated_rmsnorm(y, z.contiguous(), c["wg"], eps=EPS).flatten(1) @ c["out"]
        check(out, torch.stack([t[j] for t in last]), TOL[dtype], f"token {j}")
    check(states, st64.detach(), TOL[dtype], "states behind the tokens")


def test_layer_captured_beside_an_eager_one():
    """Two captured layers (their workspaces come from the graphs' own pools) replayed at once on two streams, with an
    eager one between; new inputs are copied in before the replay."""
    lens = [500, 0, 65, 1700]  # long enough for a cut into pieces
    x = [{n: t.cuda() for n, t in make(lens, torch.bfloat16, seed=s).items()} for s in (1, 2)]
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for c, st in zip(x, streams):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            layer(c)
        st.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            saved = {}
            r = layer(c, saved)
            outs.append((*r, *layer_backward(c, saved).values()))
        graphs.append(gr)
    for seed, c in zip((3, 4), x):
        for n, t in make(lens, torch.bfloat16, seed=seed).items():
            c[n].copy_(t)
    torch.cuda.synchronize()
    eager = None
    for gr, st in zip(graphs, streams):
        with torch.cuda.stream(st):
            gr.replay()
        if eager is None:
            eager = layer(x[0])
    torch.cuda.synchronize()
    for a, b in zip(outs[0], eager):
        assert torch.equal(a, b)
    for c, got in zip(x, outs):
        saved = {}
        r = layer(c, saved)
        want = (*r, *layer_backward(c, saved).values())
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert api.gdn_read_device_status() == 0

"""GPU parity of the norm with the residual's addition (16- and 32-bit, 8-bit, backward) against the fp64
oracle.

Tolerances, elementwise.  h: its rounding alone.  o: the 32-bit sum and square sum (2^-24 a step; tree sums
of C / 32 terms a lane at most: (C / 256 + 16) 2^-24, halved by the root), then three products: bounded by
(C / 512 + 16) 2^-23 of |o|, plus 2^-8 |o| for bf16.  8-bit: scales as o; a value may fall to the other
neighbour where o / scale is within that error of the border between two, so each value is within one step
(2^-3 of it) and all but 2^-10 of them are equal.  dx: the two terms' magnitudes times the same bound.  dw:
sums over the rows, rows 2^-24 of the absolute sum at most."""
import numpy as np
import pytest
import torch

import oracle.add_norm as onorm
from gated_deltanet_linear_eqs_b200 import api

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


def np64(t):
    return t.double().cpu().numpy()


def make(rows, C, dtype, seed=0, std=3.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, std=1.0: (std * torch.randn(*s, generator=g))
    return dict(x=r(rows, C).to(DT[dtype]), residual=r(rows, C, std=std).to(DT[dtype]), w=r(C, std=0.2),
                d_o=r(rows, C).to(DT[dtype]), d_h=r(rows, C).to(DT[dtype]))


def tol_of(mag, C, dtype):
    t = (C / 512 + 16) * 2.0 ** -23 * mag + 1e-37
    return t + (2.0 ** -8 * mag if dtype == "bf16" else 0.0)


SIZES = [(1, 8), (3, 24), (5, 256), (2, 264), (7, 520), (33, 1000), (4, 2048), (9, 4104), (3, 5120), (2, 16384),
         (700, 128), (1300, 64)]


@pytest.mark.parametrize("rows,C", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_forward(rows, C, dtype):
    x = make(rows, C, dtype, seed=C)
    c = {n: t.cuda() for n, t in x.items()}
    o, h = api.gdn_add_rmsnorm(c["x"], c["residual"], c["w"], eps=EPS)
    torch.cuda.synchronize()
    orf, hr = onorm.forward(x["x"], x["residual"], x["w"], EPS)
    want = torch.from_numpy(hr).float().to(DT[dtype])  # the fp32 sum of two bf16 (or fp32) values, rounded
    assert torch.equal(h.cpu(), (x["x"].float() + x["residual"].float()).to(DT[dtype]))
    assert np.all(np.abs(np64(h) - hr) <= 2.0 ** (-8 if dtype == "bf16" else -24) * np.abs(hr)), want.shape
    assert np.all(np.abs(np64(o) - orf) <= tol_of(np.abs(orf), C, dtype))
    # without a residual; in place
    o1, h1 = api.gdn_add_rmsnorm(c["x"], None, c["w"], eps=EPS)
    orf, _ = onorm.forward(x["x"], None, x["w"], EPS)
    assert h1 is c["x"]
    assert np.all(np.abs(np64(o1) - orf) <= tol_of(np.abs(orf), C, dtype))
    res, xx = c["residual"].clone(), c["x"].clone()
    o2, h2 = api.gdn_add_rmsnorm(xx, res, c["w"], eps=EPS, h=res, o=xx)
    torch.cuda.synchronize()
    assert torch.equal(o2, o) and torch.equal(h2, h) and h2 is res and o2 is xx


@pytest.mark.parametrize("rows,C,group", [(1, 8, 0), (5, 256, 0), (3, 128, 128), (3, 128, 0), (33, 1000, 0), (17, 2048, 128),
                                          (4, 5120, 0), (4, 5120, 128), (2, 16384, 128), (2, 16384, 0), (600, 640, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_fp8(rows, C, group, dtype):
    x = make(rows, C, dtype, seed=C + group)
    x["w"][: min(C, 128)] = -1.0 if group == 128 and C > 128 else x["w"][: min(C, 128)]  # a group of zeros
    c = {n: t.cuda() for n, t in x.items()}
    o, s, h = api.gdn_add_rmsnorm_fp8(c["x"], c["residual"], c["w"], eps=EPS, group=group)
    torch.cuda.synchronize()
    orf, _ = onorm.forward(x["x"], x["residual"], x["w"], EPS)
    q, sr = onorm.quantise(orf, group or C)
    assert s.shape == sr.shape and o.dtype == torch.float8_e4m3fn
    assert torch.equal(h.cpu(), (x["x"].float() + x["residual"].float()).to(DT[dtype]))
    assert np.all(np.abs(np64(s) - sr) <= tol_of(sr, C, "fp32"))
    got = np64(o.float())
    assert np.all(np.abs(got - q) <= np.maximum(2.0 ** -3 * np.abs(q), 2.0 ** -9))
    assert np.mean(got != q) <= 2.0 ** -10 + 1.0 / got.size
    if group == 128 and C > 128:
        assert np.all(got[:, :128] == 0) and np.all(np64(s)[:, 0] == 0)


@pytest.mark.parametrize("rows,C", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_backward(rows, C, dtype):
    x = make(rows, C, dtype, seed=C + 1)
    c = {n: t.cuda() for n, t in x.items()}
    for d_h in (True, False):
        g = api.gdn_add_rmsnorm_backward(c["residual"], c["w"], c["d_o"], d_h=c["d_h"] if d_h else None, eps=EPS)
        torch.cuda.synchronize()
        ref = onorm.backward(x["residual"], x["w"], x["d_o"], x["d_h"] if d_h else None, EPS)
        h, do, w = np64(x["residual"]), np64(x["d_o"]), np64(x["w"])
        r = 1 / np.sqrt(np.mean(h * h, -1, keepdims=True) + EPS)
        n, dn = np.abs(h * r), np.abs(do * (1 + w))
        mag = r * (dn + n * np.mean(dn * n, -1, keepdims=True)) + (np.abs(np64(x["d_h"])) if d_h else 0)
        tol = tol_of(mag, C, "fp32") + (2.0 ** -8 * np.abs(ref["dx"]) if dtype == "bf16" else 0)
        assert np.all(np.abs(np64(g["dx"]) - ref["dx"]) <= tol)
        wmag = (np.abs(do) * n).sum(0)
        assert np.all(np.abs(np64(g["dw"]) - ref["dw"]) <= (rows + C / 512 + 16) * 2.0 ** -23 * wmag)
    again = api.gdn_add_rmsnorm_backward(c["residual"], c["w"], c["d_o"], eps=EPS)
    assert torch.equal(again["dw"], g["dw"]) and torch.equal(again["dx"], g["dx"])


def test_backward_against_differences():
    x = make(6, 64, "fp32", seed=4)
    c = {n: t.cuda() for n, t in x.items()}
    g = api.gdn_add_rmsnorm_backward(c["residual"], c["w"], c["d_o"], d_h=c["d_h"], eps=EPS)

    def loss(h, w):
        o, _ = api.gdn_add_rmsnorm(h, None, w, eps=EPS)
        return float((o.double() * c["d_o"].double()).sum() + (h.double() * c["d_h"].double()).sum())

    gen = torch.Generator(device="cuda").manual_seed(0)
    for n, t, grad in (("h", c["residual"], g["dx"]), ("w", c["w"], g["dw"])):
        e = torch.randn(t.shape, generator=gen, device="cuda")
        s = 2.0 ** -6
        up, dn = (t + s * e, t - s * e)
        num = (loss(up, c["w"]) - loss(dn, c["w"]) if n == "h" else loss(c["residual"], up) - loss(c["residual"], dn)) / (2 * s)
        ref = float((grad.double() * e.double()).sum())
        # 384 outputs of size 1 rounded at 2^-22 over 2 s = 2^-5, and s^2 / 6 times third derivatives (below 1 for
        # rows of root mean square 3) of the 384 terms adding at random
        assert abs(num - ref) <= 384 * 2.0 ** -17 + 2.0 ** -12 / 6 * 20 * 4, (n, num, ref)


def test_rows_that_are_not_finite_stay_alone():
    x = make(4, 256, "bf16", seed=8)
    c = {n: t.cuda() for n, t in x.items()}
    o0, h0 = api.gdn_add_rmsnorm(c["x"], c["residual"], c["w"])
    q0, s0, _ = api.gdn_add_rmsnorm_fp8(c["x"], c["residual"], c["w"], group=128)
    c["x"][1, 7] = float("nan")
    c["x"][2] = 0
    c["residual"][2] = 0
    o, h = api.gdn_add_rmsnorm(c["x"], c["residual"], c["w"])
    q, s, _ = api.gdn_add_rmsnorm_fp8(c["x"], c["residual"], c["w"], group=128)
    torch.cuda.synchronize()
    for r in (0, 3):
        assert torch.equal(o[r], o0[r]) and torch.equal(h[r], h0[r])
        assert torch.equal(q[r].view(torch.uint8), q0[r].view(torch.uint8)) and torch.equal(s[r], s0[r])
    assert bool(o[1].isnan().all()) and bool(s[1].isnan().all()) and bool(q[1].float().isnan().all())
    assert bool((o[2] == 0).all()) and bool((s[2] == 0).all()) and bool((q[2].float() == 0).all())


def test_no_rows_and_graph():
    w = torch.randn(64, device="cuda")
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    o, h = api.gdn_add_rmsnorm(e, e, w)
    assert o.shape == e.shape
    q, s, _ = api.gdn_add_rmsnorm_fp8(e, e, w)
    assert s.shape == (0, 1)
    g = api.gdn_add_rmsnorm_backward(e, w, e)
    torch.cuda.synchronize()
    assert bool((g["dw"] == 0).all())
    x = make(50, 512, "bf16")
    c = {n: t.cuda() for n, t in x.items()}
    want = api.gdn_add_rmsnorm_backward(c["x"], c["w"], c["d_o"])
    ws = torch.empty(api.gdn_workspace_bytes(api._abi.GDN_OP_ADD_RMSNORM_BACKWARD, 1, 50, 1, 512, 512), dtype=torch.uint8,
                     device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = api.gdn_add_rmsnorm_backward(c["x"], c["w"], c["d_o"], ws=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got["dx"], want["dx"]) and torch.equal(got["dw"], want["dw"])


def test_in_place_without_a_residual_keeps_no_h():
    """h = x is overwritten by o: the caller is not given o for it."""
    x = make(5, 256, "bf16", seed=2)["x"].cuda()
    w = torch.randn(256, device="cuda")
    want, h = api.gdn_add_rmsnorm(x, None, w)
    assert h is x
    kept = torch.empty_like(x)
    xx = x.clone()
    o, h = api.gdn_add_rmsnorm(xx, None, w, o=xx)
    assert o is xx and h is None and torch.equal(o, want)
    xx = x.clone()
    o, h = api.gdn_add_rmsnorm(xx, None, w, o=xx, h=kept)
    assert o is xx and h is kept and torch.equal(h, x) and torch.equal(o, want)
    with pytest.raises(api.GdnError):
        api.gdn_add_rmsnorm(x, x, w, o=x, h=x)
    e = torch.empty(0, 256, device="cuda")
    assert api.gdn_add_rmsnorm(e, None, w)[1] is e

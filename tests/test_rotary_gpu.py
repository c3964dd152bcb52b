"""GPU parity of the rotary positions against the fp64 oracle.

Tolerance, elementwise: cos and sin in fp32 (2 ulp) of an angle reduced in 64 bits and rounded to
fp32 (2^-25 of a turn at most, 2^-22 of the pair's norm), the products and their sum (2^-23): 2^-21 of the
pair's norm times the scale; bf16 outputs add their rounding, 2^-8 of the value."""
import numpy as np
import pytest
import torch

import oracle.rotary as orot
from gated_deltanet_linear_eqs_b200 import api

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def check(got, x, pos, f, dtype, interleaved, inverse, scale):
    ref = orot.rotate(x, pos, f, interleaved, inverse, scale)
    half = len(f)
    ia = np.arange(half) * 2 if interleaved else np.arange(half)
    ib = ia + 1 if interleaved else ia + half
    xd = x.double().cpu().numpy()
    norm = np.zeros_like(xd)
    norm[..., ia] = norm[..., ib] = np.hypot(xd[..., ia], xd[..., ib]) * scale
    tol = 2.0 ** -21 * norm + 1e-30
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * np.abs(ref)
    got = got.double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) / tol))
    np.testing.assert_array_equal(got[..., 2 * half:], xd[..., 2 * half:])


@pytest.mark.parametrize("T,Hq,Hk,d,r", [(1, 1, 1, 8, 2), (7, 3, 2, 64, 64), (33, 5, 1, 80, 20), (19, 2, 2, 96, 48),
                                         (700, 4, 1, 128, 128), (5, 2, 1, 1024, 1024), (64, 8, 8, 256, 64),
                                         (3, 1, 1, 40, 38), (5000, 1, 1, 64, 32)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rotary(T, Hq, Hk, d, r, interleaved, dtype):
    g = torch.Generator().manual_seed(T + d)
    W = (Hq + 2 * Hk) * d
    qkv = torch.randn(T, W, generator=g).to(DT[dtype])
    pos = torch.randint(0, 1 << 20, (T,), generator=g, dtype=torch.int32)
    f = (1e6 ** (-torch.arange(r // 2) / (r / 2))).float()
    scale = 1.25
    c = qkv.cuda()
    q, k = c[:, :Hq * d].view(T, Hq, d), c[:, Hq * d:(Hq + Hk) * d].view(T, Hk, d)
    qx, kx = qkv[:, :Hq * d].view(T, Hq, d), qkv[:, Hq * d:(Hq + Hk) * d].view(T, Hk, d)
    for inverse in (False, True):
        qo, ko = api.gdn_rotary(q, k, pos.cuda(), f.cuda(), interleaved=interleaved, inverse=inverse, scale=scale)
        torch.cuda.synchronize()
        check(qo, qx, pos, f, dtype, interleaved, inverse, scale)
        check(ko, kx, pos, f, dtype, interleaved, inverse, scale)
    # in place in the projection's output: v and the kept values stay as they were
    api.gdn_rotary(q, k, pos.cuda(), f.cuda(), interleaved=interleaved, scale=scale, q_out=q, k_out=k)
    torch.cuda.synchronize()
    check(q, qx, pos, f, dtype, interleaved, False, scale)
    check(k, kx, pos, f, dtype, interleaved, False, scale)
    assert torch.equal(c[:, (Hq + Hk) * d:].cpu(), qkv[:, (Hq + Hk) * d:])


def test_far_positions_and_batches():
    """Positions up to 2^31 - 1 and negative ones; [B, T, heads, d] tensors; q alone."""
    x = torch.randn(2, 3, 2, 64, generator=torch.Generator().manual_seed(0))
    pos = torch.tensor([0, 2 ** 31 - 1, 123456789, -1, -2 ** 31, 1000001], dtype=torch.int32)
    f, _ = api.gdn_rotary_inv_freq(64, base=1e7)
    y, none = api.gdn_rotary(x.cuda(), None, pos.cuda(), f.cuda())
    torch.cuda.synchronize()
    assert none is None and y.shape == x.shape
    check(y.flatten(0, 1), x.flatten(0, 1), pos, f, "fp32", False, False, 1.0)


def test_inverse_is_the_gradient():
    """<rotary(x), y> = <x, inverse(y)>: both sides in fp32, compared in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x, y = (torch.randn(50, 4, 96, generator=g, device="cuda") for _ in range(2))
    pos = torch.arange(50, device="cuda", dtype=torch.int32) * 991
    f = api.gdn_rotary_inv_freq(48)[0].cuda()
    for il in (False, True):
        a, _ = api.gdn_rotary(x, None, pos, f, interleaved=il, scale=1.1)
        b, _ = api.gdn_rotary(y, None, pos, f, interleaved=il, inverse=True, scale=1.1)
        lhs, rhs = (a.double() * y.double()).sum(), (x.double() * b.double()).sum()
        # 19200 products of size ~1, each off by 2^-21 at most
        assert abs(float(lhs - rhs)) <= 19200 * 2.0 ** -21 * 4


def test_no_tokens_and_graph():
    f = api.gdn_rotary_inv_freq(64)[0].cuda()
    e = torch.empty(0, 2, 64, device="cuda")
    p = torch.empty(0, dtype=torch.int32, device="cuda")
    q, k = api.gdn_rotary(e, e, p, f)
    assert q.shape == e.shape and k.shape == e.shape
    x = torch.randn(9, 2, 64, device="cuda")
    pos = torch.arange(9, device="cuda", dtype=torch.int32)
    want, _ = api.gdn_rotary(x, None, pos, f)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, _ = api.gdn_rotary(x, None, pos, f)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_token_counts_up_to_31_bits():
    """2^31 - 1 tokens, in place (a step of the grid past the last token does not fit 31 bits): every token is turned
    once, those of position 0 keep their values."""
    T = 2 ** 31 - 1
    f = api.gdn_rotary_inv_freq(8)[0]
    x = torch.ones(T, 1, 8, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    at = torch.tensor([0, 1, 17759, 17760, 2 ** 28, 2 ** 30 + 1, T - 17761, T - 17760, T - 4, T - 3, T - 2, T - 1])
    pos[at.cuda()] = torch.arange(1, len(at) + 1, dtype=torch.int32, device="cuda")
    api.gdn_rotary(x, None, pos, f.cuda(), q_out=x)
    torch.cuda.synchronize()
    check(x[at.cuda()], torch.ones(len(at), 1, 8, dtype=torch.bfloat16), torch.arange(1, len(at) + 1, dtype=torch.int32), f,
          "bf16", False, False, 1.0)
    x[at.cuda()] = 1
    for i in range(0, T, 2 ** 28):
        assert bool((x[i:i + 2 ** 28] == 1).all())
    del x, pos
    torch.cuda.empty_cache()

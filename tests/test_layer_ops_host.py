"""Host-side checks of the decayed linear attention's, the rotary positions' and the residual norm's calls:
refusals before any launch, workspace sizes, the rotary frequencies."""
import ctypes
import math

import numpy as np
import pytest
import torch

from gated_deltanet_linear_eqs_b200 import _abi, api
from gated_deltanet_linear_eqs_b200.build import build

A = 0x10000  # a 16-byte-aligned fake address: a rejected call touches nothing
BAD, SHAPE, WS = _abi.GDN_ERR_INVALID_ARG, _abi.GDN_ERR_UNSUPPORTED_SHAPE, _abi.GDN_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    build()
    return _abi.load()


def dense(lib, **kw):
    a = dict(q=A, k=A, v=A, g=A, s0=0, y=A, sf=0, B=1, T=4096, H=2, Hk=1, dk=128, dv=128, dt=0, scale=1.0, ws=A, wsb=1 << 40)
    a.update(kw)
    return lib.gdn_linear_attn(*a.values(), None)


def varlen(lib, **kw):
    a = dict(q=A, k=A, v=A, g=A, cu=A, n=2, s0=0, y=A, sf=0, T=4096, H=2, Hk=1, dk=64, dv=64, dt=1, scale=1.0, ws=A,
             wsb=1 << 40)
    a.update(kw)
    return lib.gdn_linear_attn_varlen(*a.values(), None)


def back(lib, **kw):
    a = dict(q=A, k=A, v=A, g=A, s0=0, dy=A, dsf=0, dq=A, dk_=A, dv_=A, ds0=0, B=1, T=4096, H=2, Hk=1, dk=128, dv=128, dt=0,
             scale=1.0, ws=A, wsb=1 << 40)
    a.update(kw)
    return lib.gdn_linear_attn_backward(*a.values(), None)


def back_varlen(lib, **kw):
    a = dict(q=A, k=A, v=A, g=A, cu=A, n=2, s0=0, dy=A, dsf=0, dq=A, dk_=A, dv_=A, ds0=0, T=4096, H=2, Hk=1, dk=128, dv=128,
             dt=0, scale=1.0, ws=A, wsb=1 << 40)
    a.update(kw)
    return lib.gdn_linear_attn_backward_varlen(*a.values(), None)


@pytest.mark.parametrize("call", [dense, varlen, back, back_varlen])
@pytest.mark.parametrize("kw,code", [
    (dict(q=0), BAD), (dict(k=A + 8), BAD), (dict(v=0), BAD), (dict(g=0), BAD), (dict(s0=A + 4), BAD), (dict(T=0), BAD),
    (dict(H=0), BAD), (dict(Hk=0), BAD), (dict(H=3, Hk=2), BAD), (dict(dt=2), BAD), (dict(dk=96, dv=96), SHAPE),
    (dict(dk=64, dv=128), SHAPE), (dict(ws=0), WS), (dict(wsb=4096), WS), (dict(ws=A + 8), WS),
    (dict(T=2 ** 31 - 1, H=1 << 10), BAD)])
def test_linear_attn_refusals(lib, call, kw, code):
    assert call(lib, **kw) == code


def test_linear_attn_more_refusals(lib):
    assert dense(lib, y=0) == BAD and dense(lib, sf=A + 4) == BAD and dense(lib, B=0) == BAD
    assert dense(lib, B=1 << 20, T=1 << 12) == BAD           # 2^32 tokens
    assert varlen(lib, cu=0) == BAD and varlen(lib, n=0) == BAD and varlen(lib, y=A + 2) == BAD
    for f in (back, back_varlen):
        for n in ("dy", "dq", "dk_", "dv_"):
            assert f(lib, **{n: 0}) == BAD
        assert f(lib, ds0=A + 4) == BAD and f(lib, dsf=A + 8) == BAD
    step = lambda **kw: lib.gdn_linear_attn_decode_step(*{**dict(q=A, k=A, v=A, g=A, s=A, y=A, N=4, H=4, Hk=2, dk=64, dv=64,
                                                                 dt=0, scale=1.0), **kw}.values(), None)
    assert step(q=0) == BAD and step(s=A + 4) == BAD and step(N=0) == BAD and step(Hk=3) == BAD and step(dt=9) == BAD
    assert step(dk=32, dv=32) == SHAPE and step(N=1 << 30) == BAD


def test_linear_attn_states_in_place_are_refused(lib):
    """A long sequence is cut: the CTA that writes its last state may run ahead of the one that reads its first."""
    for call in (dense, varlen):
        assert call(lib, s0=A, sf=A) == BAD
    for call in (back, back_varlen):
        assert call(lib, dsf=A, ds0=A) == BAD
        assert call(lib, s0=A, ds0=A) == BAD


def test_linear_attn_workspace(lib):
    n = ctypes.c_size_t(0)
    f = lambda *a: lib.gdn_linear_attn_workspace_bytes(*a, ctypes.byref(n))
    # enough sequences and heads for every SM: one segment each, no states in between
    assert f(0, 8, 4096, 32, 32, 128, 128, 0) == 0 and n.value == 0
    # one long sequence: a state for each segment and head
    assert f(0, 1, 32768, 16, 16, 128, 128, 0) == 0
    assert n.value > 0 and n.value % (16 * 128 * 128 * 4) == 0
    # shared heads' gradients: fp32 parts of dk and dv for every head
    assert f(1, 8, 4096, 32, 8, 128, 128, 0) == 0 and n.value == 2 * 8 * 4096 * 32 * 128 * 4
    for bad in ((0, 0, 1, 1, 1, 64, 64, 0), (0, 1, 0, 1, 1, 64, 64, 0), (0, 1, 1, 3, 2, 64, 64, 0), (0, 2, 5, 1, 1, 64, 64, 3),
                (0, 1, 5, 1, 1, 64, 64, -1)):
        assert f(*bad) == BAD
    assert f(0, 1, 5, 1, 1, 32, 32, 0) == SHAPE
    assert lib.gdn_linear_attn_workspace_bytes(0, 1, 5, 1, 1, 64, 64, 0, None) == BAD


def test_rotary_refusals(lib):
    def call(**kw):
        a = dict(q=A, k=A, qo=A, ko=A, p=A, f=A, T=10, Hq=4, Hk=2, d=64, r=32, lq=256, lk=128, lqo=256, lko=128, il=0, inv=0,
                 scale=1.0, dt=0)
        a.update(kw)
        return lib.gdn_rotary(*a.values(), None)
    assert call(q=0) == BAD and call(qo=A + 8) == BAD and call(k=0) == BAD and call(p=0) == BAD and call(p=A + 2) == BAD
    assert call(f=0) == BAD and call(T=-1) == BAD and call(Hq=0) == BAD and call(Hk=-1) == BAD and call(dt=3) == BAD
    assert call(lq=248) == BAD and call(lk=132) == BAD and call(lqo=264) == BAD  # below a row; not of 8; in place
    assert call(d=60) == SHAPE and call(d=2048, lq=8192, lk=4096) == SHAPE
    assert call(r=31) == SHAPE and call(r=66) == SHAPE and call(r=0) == SHAPE


def test_rotary_frequencies(lib):
    f, s = api.gdn_rotary_inv_freq(128, base=1e4)
    np.testing.assert_allclose(f.double().numpy(), 1e4 ** (-np.arange(64) / 64), rtol=2.0 ** -24)
    assert s == 1.0
    lin, _ = api.gdn_rotary_inv_freq(128, base=1e4, scaling="linear", factor=4)
    np.testing.assert_allclose(lin.double().numpy(), f.double().numpy() / 4, rtol=2.0 ** -23)
    ntk, _ = api.gdn_rotary_inv_freq(128, base=1e4, scaling="ntk", factor=4)
    np.testing.assert_allclose([float(ntk[0]), float(ntk[-1])], [1.0, float(f[-1]) / 4], rtol=2.0 ** -22)
    y, s = api.gdn_rotary_inv_freq(64, base=1e7, scaling="yarn", factor=4, original_context=262144)
    assert s == pytest.approx(0.1 * math.log(4) + 1, rel=1e-6)
    # 32 turns within 262144 positions fall to pair 14.2, one turn to pair 21.1: whole pairs 14 and 22
    base = 1e7 ** (-np.arange(32) / 32)
    slow = np.clip((np.arange(32) - 14) / 8, 0, 1)
    np.testing.assert_allclose(y.double().numpy(), base / 4 * slow + base * (1 - slow), rtol=2.0 ** -23)
    one, _ = api.gdn_rotary_inv_freq(2, base=1e4, scaling="ntk", factor=8)
    assert one.tolist() == [1.0]
    for kw in (dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=64, base=1.0), dict(rotary_dim=64, base=float("nan")),
               dict(rotary_dim=64, scaling="linear", factor=0.5), dict(rotary_dim=64, scaling="yarn", factor=2),
               dict(rotary_dim=64, scaling="yarn", factor=2, original_context=100, beta_fast=1, beta_slow=2)):
        with pytest.raises(api.GdnError):
            api.gdn_rotary_inv_freq(**kw)
    with pytest.raises(ValueError):
        api.gdn_rotary_inv_freq(64, scaling="other")


def test_add_norm_refusals(lib):
    fwd = lambda **kw: lib.gdn_add_rmsnorm(*{**dict(x=A, r=A, w=A, o=A, h=A, rows=10, C=256, dt=0, eps=1e-6), **kw}.values(),
                                           None)
    q = lambda **kw: lib.gdn_add_rmsnorm_fp8(*{**dict(x=A, r=A, w=A, o=A, s=A, h=A, rows=10, C=256, g=128, dt=0, eps=1e-6),
                                               **kw}.values(), None)
    b = lambda **kw: lib.gdn_add_rmsnorm_backward(*{**dict(h=A, w=A, do=A, dh=0, dx=A, dw=A, rows=10, C=256, dt=0, eps=1e-6,
                                                           ws=A, wsb=1 << 30), **kw}.values(), None)
    for f in (fwd, q, b):
        assert f(w=0) == BAD and f(rows=-1) == BAD and f(rows=1 << 31) == BAD and f(eps=-1.0) == BAD
        assert f(eps=float("nan")) == BAD and f(dt=4) == BAD
        assert f(C=4) == SHAPE and f(C=252) == SHAPE and f(C=16392) == SHAPE
    for f in (fwd, q):
        assert f(x=0) == BAD and f(o=A + 8) == BAD and f(r=A + 2) == BAD and f(h=A + 8) == BAD
    assert q(s=0) == BAD and q(g=64) == BAD and q(C=264, g=128) == SHAPE
    assert b(h=0) == BAD and b(do=0) == BAD and b(dx=0) == BAD and b(dw=0) == BAD and b(dh=A + 8) == BAD
    assert b(ws=0) == WS and b(wsb=100) == WS and b(ws=A + 8) == WS
    n = ctypes.c_size_t(0)
    w = lambda rows, C: lib.gdn_workspace_bytes(_abi.GDN_OP_ADD_RMSNORM_BACKWARD, 1, rows, 1, C, C, 0, ctypes.byref(n))
    assert w(3, 256) == 0 and n.value == 3 * 256 * 4
    assert w(10 ** 6, 4096) == 0 and n.value == 592 * 4096 * 4
    assert w(3, 12) == SHAPE


def test_bindings_refuse_host_tensors_and_shapes():
    t = torch.zeros(1, 8, 2, 64)
    g = torch.zeros(2)
    st = torch.zeros(1, 2, 64, 64)
    with pytest.raises(ValueError, match="CUDA"):
        api.gdn_linear_attn(t, t, t, g)
    with pytest.raises(ValueError, match="CUDA"):
        api.gdn_linear_attn_varlen(t[0], t[0], t[0], g, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        api.gdn_linear_attn_backward(t, t, t, g, t)
    with pytest.raises(ValueError, match="CUDA"):
        api.gdn_linear_attn_decode_step(t[:, 0], t[:, 0], t[:, 0], g, st)
    with pytest.raises(ValueError, match="shared"):
        api.gdn_linear_attn(t, t[:, :, :1].expand(1, 8, 3, 64), t, g)
    with pytest.raises(ValueError, match="bf16 or fp32"):
        api.gdn_linear_attn(t.half(), t.half(), t.half(), g)
    with pytest.raises(ValueError, match="CUDA"):
        api.gdn_rotary(t[0], None, torch.zeros(8, dtype=torch.int32), torch.zeros(32))
    with pytest.raises(ValueError, match="CUDA"):
        api.gdn_add_rmsnorm(t[0, :, 0], None, torch.zeros(64))
    with pytest.raises(ValueError, match="CUDA"):
        api.gdn_add_rmsnorm_backward(t[0, :, 0], torch.zeros(64), t[0, :, 0])


def test_rotary_rows_of_31_bits_are_refused(lib):
    """Places within a token's row are kept in 32 bits."""
    def call(Hq, Hk, d):
        lq, lk = Hq * d, max(Hk, 1) * d
        return lib.gdn_rotary(A, A, A, A, A, A, 1, Hq, Hk, d, 8, lq, lk, lq, lk, 0, 0, 1.0, 0, None)
    assert call(1 << 21, 0, 1024) == BAD and call(1, 1 << 28, 8) == BAD and call(1 << 28, 1 << 28, 8) == BAD


def test_bindings_refuse_sizes_past_31_bits():
    """The library takes them as ints, and ctypes hands over the low 32 bits without a word."""
    big = torch.zeros(1, dtype=torch.bfloat16).expand((1 << 32) + 8)
    pos, f, w = torch.zeros(8, dtype=torch.int32), torch.zeros(4), torch.zeros(8)
    with pytest.raises(ValueError, match="2\\^31"):
        api.gdn_rotary(big[:, None, None].expand(-1, 1, 8), None, pos, f)
    with pytest.raises(ValueError, match="2\\^31"):
        api.gdn_rotary(big[None, :, None].expand(1, -1, 8), None, pos, f)
    with pytest.raises(ValueError, match="2\\^31"):
        api.gdn_add_rmsnorm(big[None], None, w)
    with pytest.raises(ValueError, match="2\\^31"):
        api.gdn_add_rmsnorm_fp8(big[None], None, w)
    with pytest.raises(ValueError, match="2\\^31"):
        api.gdn_add_rmsnorm_backward(big[None], w, big[None])
    with pytest.raises(ValueError, match="2\\^31"):
        api._documents(1, torch.zeros(1, dtype=torch.int32).expand((1 << 32) + 2), 0)


def test_linear_attn_counts_up_to_31_bits(lib):
    """2^30 (document, head) pairs and more are refused (a CTA's next pair is counted in 32 bits); sizes right below
    the tokens' limit are formed without an overflow."""
    n = ctypes.c_size_t(0)
    f = lambda *a: lib.gdn_linear_attn_workspace_bytes(*a, ctypes.byref(n))
    for call in (varlen, back_varlen):
        assert call(lib, T=1, H=1 << 10, Hk=1, n=1 << 20) == BAD
    for call in (dense, back):
        assert call(lib, T=1, H=1 << 10, Hk=1, B=1 << 20) == BAD
    assert f(0, 1, 1, 1 << 10, 1, 64, 64, 1 << 20) == BAD and f(0, 1, 1, 1 << 10, 1, 64, 64, (1 << 20) - 1) == 0
    # one chain in as many pieces as the GPU has SMs
    assert f(0, 1, 2 ** 31 - 65, 1, 1, 64, 64, 0) == 0 and n.value == 148 * 64 * 64 * 4
    # 148 chains: none is cut
    assert f(0, 1, 2 ** 23, 148, 148, 64, 64, 0) == 0 and n.value == 0


def test_linear_attn_offsets_must_be_aligned(lib):
    for call in (varlen, back_varlen):
        assert call(lib, cu=A + 2) == BAD and call(lib, cu=A + 1) == BAD


def test_decay_factors_that_take_turns():
    """The bf16 kernel's factors of a state, restated: over any run of chunks their product is within one step of the
    exact power (2^-23, and the second order of many steps), where one float's drifts away."""
    rng = np.random.default_rng(0)
    g = np.concatenate([-np.exp2(rng.uniform(-22, -8, 200)), [-1e-9, -2.0 ** -30, 0.0, -0.5, -1.25]]).astype(np.float32)
    left = np.arange(2048, 0, -1)
    worst = drift = 0.0
    for x in g:
        e = np.exp(64.0 * np.float64(x))
        hi = np.float32(e)
        lo = np.float32(e - np.float64(hi))
        nxt = (hi.view(np.int32) + np.int32(-1 if lo < 0 else 1)).view(np.float32)
        rho = np.float32(lo / (nxt - hi)) * np.float32(-1 if lo < 0 else 1)
        steps = np.rint(left.astype(np.float32) * rho).astype(np.int32) - np.rint((left - 1).astype(np.float32) * rho).astype(
            np.int32)
        f = (hi.view(np.int32) + steps).view(np.float32).astype(np.float64)
        off = np.concatenate([[0.0], np.cumsum(np.log(f) - 64.0 * np.float64(x))])  # of the products, relative
        worst = max(worst, off.max() - off.min())
        drift = max(drift, 2048 * abs(np.log(np.float64(hi)) - 64.0 * np.float64(x)))
    assert worst <= 2.0 ** -23 * 1.01, worst
    assert drift >= 2.0 ** -15, drift


def test_add_norm_outputs_that_share_memory_are_refused(lib):
    """o and h in one buffer: one of them would be lost.  8-bit rows and scales lie elsewhere than the rows that other
    blocks still read."""
    fwd = lambda **kw: lib.gdn_add_rmsnorm(*{**dict(x=A, r=2 * A, w=3 * A, o=4 * A, h=5 * A, rows=10, C=256, dt=0, eps=1e-6),
                                             **kw}.values(), None)
    q = lambda **kw: lib.gdn_add_rmsnorm_fp8(*{**dict(x=A, r=2 * A, w=3 * A, o=4 * A, s=6 * A, h=5 * A, rows=10, C=256, g=128,
                                                      dt=0, eps=1e-6), **kw}.values(), None)
    assert fwd(o=A, h=A) == BAD and fwd(o=5 * A) == BAD and fwd(x=0, r=0, o=0, h=0, rows=0) not in (BAD, SHAPE)
    for same in (dict(o=A), dict(o=2 * A), dict(o=5 * A), dict(s=A), dict(s=2 * A), dict(s=5 * A), dict(s=4 * A)):
        assert q(**same) == BAD


def test_yarn_where_all_pairs_are_slow_or_fast(lib):
    """A context in which no pair makes beta_slow turns: all are divided by the factor, the first one,
    too; one in which all make more than beta_fast: none is."""
    plain = api.gdn_rotary_inv_freq(64, base=1e4)[0].double().numpy()
    for kw in (dict(original_context=4), dict(original_context=100, beta_fast=64.0, beta_slow=16.0)):
        y, _ = api.gdn_rotary_inv_freq(64, base=1e4, scaling="yarn", factor=8, **kw)
        np.testing.assert_allclose(y.double().numpy(), plain / 8, rtol=2.0 ** -23)
    y, _ = api.gdn_rotary_inv_freq(64, base=1e4, scaling="yarn", factor=8, original_context=10 ** 9)
    np.testing.assert_allclose(y.double().numpy(), plain, rtol=2.0 ** -23)


def test_rotary_outputs_in_the_others_place_are_refused(lib):
    def call(q=A, k=2 * A, qo=3 * A, ko=4 * A, Hk=2, T=10):
        return lib.gdn_rotary(q, k, qo, ko, A, A, T, 2, Hk, 64, 32, 128, 128, 128, 128, 0, 0, 1.0, 0, None)
    assert call(qo=4 * A) == BAD and call(qo=2 * A) == BAD and call(ko=A) == BAD and call(k=A, qo=A, ko=A) == BAD
    assert call(T=0) not in (BAD, SHAPE) and call(k=0, qo=A, ko=A, Hk=0, T=0) != BAD  # (no tokens: nothing is launched)
    assert call(q=0, k=0, qo=0, ko=0, T=0) != BAD and call(qo=4 * A, T=0) == BAD


def test_refusals_with_tensors_apart(lib):
    """Every refusal on its own, with a buffer for each tensor.  The calls that are not refused have no rows or tokens, so
    that none launches anything."""
    no = (BAD, SHAPE, WS)

    def rotary(**kw):
        a = dict(q=A, k=2 * A, qo=3 * A, ko=4 * A, p=5 * A, f=6 * A, T=10, Hq=4, Hk=2, d=64, r=32, lq=256, lk=128, lqo=256,
                 lko=128, il=0, inv=0, scale=1.0, dt=0)
        a.update(kw)
        return lib.gdn_rotary(*a.values(), None)
    assert rotary(T=0) not in no and rotary(qo=A, ko=2 * A, T=0) not in no and rotary(k=A, T=0) not in no
    for kw in (dict(q=0), dict(qo=3 * A + 8), dict(k=0), dict(ko=0), dict(p=0), dict(p=A + 2), dict(f=0), dict(T=-1), dict(Hq=0),
               dict(Hk=-1), dict(dt=3), dict(lq=248), dict(lk=132), dict(qo=A, lqo=264)):
        assert rotary(**kw) == BAD, kw

    def fwd(**kw):
        a = dict(x=A, r=2 * A, w=3 * A, o=4 * A, h=5 * A, rows=10, C=256, dt=0, eps=1e-6)
        a.update(kw)
        return lib.gdn_add_rmsnorm(*a.values(), None)

    def fp8(**kw):
        a = dict(x=A, r=2 * A, w=3 * A, o=4 * A, s=6 * A, h=5 * A, rows=10, C=256, g=128, dt=0, eps=1e-6)
        a.update(kw)
        return lib.gdn_add_rmsnorm_fp8(*a.values(), None)

    def back(**kw):
        a = dict(h=A, w=2 * A, do=3 * A, dh=0, dx=4 * A, dw=5 * A, rows=10, C=256, dt=0, eps=1e-6, ws=6 * A, wsb=1 << 30)
        a.update(kw)
        return lib.gdn_add_rmsnorm_backward(*a.values(), None)
    for kw in ({}, dict(o=A), dict(h=A), dict(h=2 * A), dict(r=0, h=0)):
        assert fwd(rows=0, **kw) not in no
    assert fp8(rows=0) == 0 and back(ws=0) == WS and back(ws=0, dx=3 * A) == WS
    for f in (fwd, fp8, back):
        for kw in (dict(w=0), dict(rows=-1), dict(rows=1 << 31), dict(eps=-1.0), dict(eps=float("nan")), dict(dt=4)):
            assert f(**kw) == BAD, kw
        for C in (4, 252, 16392):
            assert f(C=C) == SHAPE
    for f in (fwd, fp8):
        for kw in (dict(x=0), dict(o=4 * A + 8), dict(r=A + 2), dict(h=A + 8)):
            assert f(**kw) == BAD, kw
    assert fp8(s=0) == BAD and fp8(g=64) == BAD and fp8(C=264) == SHAPE

"""Parity of muir_rotary against the float64 oracle.

Tolerance per element, from the arithmetic: the angle is rounded to float32 after its
reduction to half turns in [-1, 1] (pi 2^-24 = 1.9e-7), sincospi is within 2 ulp, mscale
and the two products and their sum round once each (4 2^-24): 6e-7 m (|a| + |b|) in all,
and bfloat16 storage adds half a step, 2^-8 |y|."""
import numpy as np
import pytest
import torch

from oracle import attention as A

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import gated_delta_rule_115_b200 as m
    m.lib()
    return m


def close(y, x, pos, f, inter, mscale, inverse, dtype):
    want = A.rotary(x.double().cpu().numpy(), pos, f, inter, mscale, inverse)
    size = np.abs(x.double().cpu().numpy())
    half = len(f)
    i = np.arange(half)
    ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + half)
    tol = np.zeros_like(want)
    tol[..., ia] = tol[..., ib] = 6e-7 * mscale * (size[..., ia] + size[..., ib])
    if dtype == torch.bfloat16:
        tol += 2.0 ** -8 * np.abs(want)
    err = np.abs(y.double().cpu().numpy() - want)
    assert (err <= tol + 1e-30).all(), float((err - tol).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,T,Hq,Hk,d,rot,far", [
    (1, 1, 1, 0, 64, 16, 0), (3, 1, 16, 4, 128, 128, 2 ** 31 - 10), (2, 37, 3, 1, 128, 64, 1000000),
    (1, 700, 5, 5, 64, 64, 0), (2, 301, 2, 8, 128, 48, 10 ** 7), (1, 1500, 1, 1, 64, 32, 0)])
def test_parity(m, B, T, Hq, Hk, d, rot, far, inter, dtype):
    g = torch.Generator().manual_seed(B * T + rot)
    q = torch.randn(B, T, Hq, d, generator=g).to(dtype)
    k = torch.randn(B, T, Hk, d, generator=g).to(dtype) if Hk else None
    pos = (torch.randint(0, far + 1, (B, 1), generator=g) + torch.arange(T)).clamp(max=2 ** 31 - 1).to(torch.int32)
    f, _ = m.rotary_frequencies(rot)
    for inverse, mscale in ((False, 1.0), (True, 1.25)):
        r = m.rotary(q.cuda(), None if k is None else k.cuda(), positions=pos.cuda(), inv_freq=f,
                     interleaved=inter, mscale=mscale, inverse=inverse)
        fc = f.cpu().numpy()
        close(r if k is None else r[0], q, pos.numpy(), fc, inter, mscale, inverse, dtype)
        if k is not None:
            close(r[1], k, pos.numpy(), fc, inter, mscale, inverse, dtype)


def test_packed_projection_in_place_and_default_positions(m):
    """q and k as parts of one projection's rows, rotated where they lie; v untouched."""
    B, T, Hq, Hk, d = 2, 130, 4, 2, 64
    x = torch.randn(B, T, (Hq + 2 * Hk) * d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    f, s = m.rotary_frequencies(d, scaling="yarn", factor=4.0)
    old = x.clone()
    q = x[..., : Hq * d].unflatten(-1, (Hq, d))
    k = x[..., Hq * d: (Hq + Hk) * d].unflatten(-1, (Hk, d))
    pos = torch.arange(T, dtype=torch.int32).repeat(B, 1)
    rq, rk = m.rotary(q.contiguous(), k.contiguous(), positions=pos.cuda(), inv_freq=f, mscale=s)
    m.rotary(q, k, inv_freq=f, mscale=s, q_out=q, k_out=k)
    assert torch.equal(q, rq) and torch.equal(k, rk)
    assert torch.equal(x[..., (Hq + Hk) * d:], old[..., (Hq + Hk) * d:])
    close(rq, old[..., : Hq * d].unflatten(-1, (Hq, d)), pos.numpy(), f.cpu().numpy(), False, s, False, torch.bfloat16)


def test_special_values_stay_in_their_pair(m):
    x = torch.ones(1, 4, 1, 64)
    x[0, 1, 0, 3], x[0, 2, 0, 40] = float("nan"), float("inf")
    f, _ = m.rotary_frequencies(32)
    y = m.rotary(x.cuda(), inv_freq=f).cpu()
    bad = ~torch.isfinite(y)
    assert bad[0, 1, 0, 3] and bad[0, 1, 0, 19] and bad[0, 2, 0, 40] and int(bad.sum()) == 3


def test_gradient_by_differences(m):
    """<R x, g> moves with x as <x, R^T g>: the inverse call is the gradient."""
    g = torch.Generator().manual_seed(4)
    x, dy, dx = (torch.randn(1, 50, 2, 64, generator=g).cuda() for _ in range(3))
    f, _ = m.rotary_frequencies(64)
    fwd = lambda t: (m.rotary(t, inv_freq=f).double() * dy.double()).sum()  # noqa: E731
    slope = (fwd(x + dx) - fwd(x - dx)) / 2  # linear: exact up to rounding
    grad = (m.rotary(dy, inv_freq=f, inverse=True).double() * dx.double()).sum()
    # both sums round 6400 products' inputs: 6e-7 (|a| + |b|) each
    assert abs(slope - grad) <= 2 * 6e-7 * 2 * float((dx.abs() + x.abs()).sum() * dy.abs().max())


def test_empty_and_other_stream(m):
    f, _ = m.rotary_frequencies(64)
    assert m.rotary(torch.empty(1, 0, 2, 64, device="cuda"), inv_freq=f).numel() == 0
    x = torch.randn(1, 64, 2, 64, device="cuda")
    want = m.rotary(x, inv_freq=f)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = m.rotary(x, inv_freq=f)
    s.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("base", [0, 2 ** 20, 2 ** 30, -2 ** 31])
def test_angles_at_any_position(m, base):
    """Rows (1, 0) give cosine and sine themselves.  The reduced angle, in half turns within
    [-1, 1], is rounded to float32 once (2^-25 half turns: 9.4e-8), sincospi is within 2 ulp
    (2^-23: 1.2e-7), products with 1 and 0 are exact: 2.2e-7 at any position.  (An angle formed
    and reduced in float64 alone is off by up to 2^-22.9 half turns, 4e-7, from 2^30 on.)"""
    T = 4000
    pos = torch.randint(0, 2 ** 30 if base < 0 else max(base, 4096), (1, T), generator=torch.Generator().manual_seed(5)) + base
    f = torch.tensor([1.0, 0.8659643233600653, 0.99, 0.75, 0.5, 0.1, 1e-3, 0.95], dtype=torch.float64)
    x = torch.zeros(1, T, 1, 64)
    x[..., :8] = 1.0
    y = m.rotary(x.cuda(), positions=pos.to(torch.int32).cuda(), inv_freq=f.cuda()).double().cpu().numpy()
    t = A.angles(pos.numpy(), f.numpy())[:, :, None]
    assert np.abs(y[..., :8] - np.cos(t)).max() <= 2.2e-7
    assert np.abs(y[..., 8:16] - np.sin(t)).max() <= 2.2e-7

"""Pins of the softmax-attention oracle (CPU): closed forms, invariants, torch float64
autograd and central differences."""
import math

import numpy as np
import pytest
import torch

from oracle import attention as A


def rnd(*shape, seed=0):
    return np.random.default_rng(seed).standard_normal(shape)


@pytest.mark.parametrize("inter", [False, True])
def test_rotary_is_a_rotation_and_its_transpose(inter):
    x, y = rnd(2, 5, 3, 64, seed=1), rnd(2, 5, 3, 64, seed=2)
    pos = np.random.default_rng(3).integers(0, 1000, (2, 5))
    f = 10000.0 ** (-np.arange(16) / 16)
    rx = A.rotary(x, pos, f, inter)
    assert np.allclose(np.linalg.norm(rx, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-12)
    assert np.array_equal(rx[..., 32:], x[..., 32:])
    # <R x, y> = <x, R^T y>, and R^T R = m^2 on the rotated channels
    assert math.isclose((rx * y).sum(), (x * A.rotary(y, pos, f, inter, inverse=True)).sum(), rel_tol=1e-12)
    back = A.rotary(A.rotary(x, pos, f, inter, 1.5), pos, f, inter, 1.5, inverse=True)
    assert np.allclose(back[..., :32], 2.25 * x[..., :32])
    # the score of two rotated rows depends on their distance only
    a, b = x[:1, :1, :1], y[:1, :1, :1]
    s = [(A.rotary(a, [[p + 7]], f, inter) * A.rotary(b, [[p]], f, inter)).sum() for p in (0, 100, 12345)]
    assert np.allclose(s, s[0])


@pytest.mark.parametrize("Tq,Tk,causal,window", [(5, 5, True, 0), (4, 9, True, 3), (9, 4, True, 0),
                                                 (6, 6, False, 0), (7, 7, True, 1), (3, 5, False, 2)])
def test_attention_against_autograd(Tq, Tk, causal, window):
    q, k, v, do = rnd(Tq, 4, 8, seed=1), rnd(Tk, 2, 8, seed=2), rnd(Tk, 2, 8, seed=3), rnd(Tq, 4, 8, seed=4)
    r = A.attention(q, k, v, causal, window, do=do)
    tq, tk, tv = (torch.tensor(t, requires_grad=True) for t in (q, k, v))
    see = torch.tensor(A.visible(Tq, Tk, causal, window))
    s = torch.einsum("ihd,jhd->hij", tq, tk.repeat_interleave(2, 1)) / math.sqrt(8)
    some = see.any(1)
    p = torch.softmax(s.masked_fill(~see, -1e300), -1) * some[None, :, None]
    o = torch.einsum("hij,jhd->ihd", p, tv.repeat_interleave(2, 1))
    (o * torch.tensor(do)).sum().backward()
    assert np.allclose(r["o"], o.detach().numpy())
    for n, t in (("dq", tq), ("dk", tk), ("dv", tv)):
        assert np.allclose(r[n], t.grad.numpy()), n
    assert np.isneginf(r["lse"][:, ~some.numpy()]).all() and np.isfinite(r["lse"][:, some.numpy()]).all()


def test_attention_differences():
    q, k, v, do = rnd(6, 2, 8, seed=1), rnd(6, 1, 8, seed=2), rnd(6, 1, 8, seed=3), rnd(6, 2, 8, seed=4)
    r = A.attention(q, k, v, True, 4, do=do)
    args = dict(q=q, k=k, v=v)
    for name in args:
        x = args[name]
        step = rnd(*x.shape, seed=9)
        lo, hi = dict(args), dict(args)
        hi[name], lo[name] = x + 1e-6 * step, x - 1e-6 * step
        f = [(A.attention(**a, causal=True, window=4)["o"] * do).sum() for a in (hi, lo)]
        assert math.isclose((f[0] - f[1]) / 2e-6, (r["d" + name] * step).sum(), rel_tol=1e-6), name


def test_e4m3_matches_torch():
    codes = np.arange(256)
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(A.e4m3_decode(codes), t, equal_nan=True)
    x = np.concatenate([rnd(4000, seed=1) * 100, np.exp(rnd(4000, seed=2) * 4) * 1e-3,
                        (t[:126] + t[1:127]) / 2, t[:127], [0.0, 500.0, np.inf, np.nan]])
    x = np.concatenate([x, -x[:-1]])
    want = torch.tensor(x).float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = A.e4m3_encode(x.astype(np.float32))
    nan = np.isnan(x)
    assert np.array_equal(got[~nan], want[~nan]) and (got[nan] & 0x7f == 0x7f).all()


@pytest.mark.parametrize("amax", [0.0, 1e-40, 448.0, 448.1, 3.5, 7.0, 1e30, 2.0 ** -91 * 448, 0.875, 0.8750001])
def test_page_scale_is_the_smallest(amax):
    s = A.page_scale(amax)
    assert math.log2(s) == round(math.log2(s)) and amax <= 448 * s
    assert s == 2.0 ** -100 or amax > 448 * s / 2


def test_append_and_step_agree_with_plain_attention():
    """Tokens appended in pieces; values exactly representable: the step equals attention."""
    rng = np.random.default_rng(5)
    k, v = (rng.integers(-8, 9, (1, 40, 2, 8)).astype(float) for _ in range(2))
    pages = [np.full((5, 2, 16, 8), 0x7f, np.uint8) for _ in range(2)]
    scales = [np.full((5, 2), 3.0) for _ in range(2)]
    table = np.array([[4, 0, 2]])
    at = 0
    for n in (1, 17, 0, 22):
        for i, x in enumerate((k, v)):
            pages[i], scales[i] = A.kv_append(x[:, at: at + n], pages[i], scales[i], table, [at], [n])
        at += n
    q = rng.standard_normal((1, 4, 8))
    for window in (0, 7):
        o, _ = A.attn_step(q, *pages, *scales, table, [40], window=window)
        assert np.allclose(o, A.attention(q, k[0], v[0], True, window)["o"])


def test_angles_are_reduced_exactly():
    """Against rational arithmetic with more digits of pi, and plain float64 where that is exact
    enough."""
    from fractions import Fraction
    pi = Fraction(3141592653589793238462643383279502884197169399375105820974944592307816406286, 10 ** 75)
    f = [1.0, 0.8659643233600653, 1e-4, 3.0, 2.0 ** 60, 0.0]
    p = np.array([[0, 1, -7], [2 ** 31 - 1, 2097695146, 12345]])
    got = A.angles(p, f)
    for i, j in np.ndindex(p.shape):
        for n, x in enumerate(f):
            t = Fraction(int(p[i, j])) * Fraction(x) / (2 * pi)
            assert abs(got[i, j, n] - float((t - round(t)) * 2 * pi)) < 1e-15 * 4
    small = np.random.default_rng(1).integers(0, 1000, (4, 5))
    t = small[..., None] * np.array([1.0, 0.1])
    assert np.allclose(np.cos(A.angles(small, [1.0, 0.1])), np.cos(t), atol=1e-12)

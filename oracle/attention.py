"""float64 oracle of the softmax-attention layer (numpy, slow): rotary positions,
attention and its gradients, the paged 8-bit cache and single-token attention over it.

Every function follows the definition in ``include/muir.h`` and shares no code with
the kernels.  Each attention result comes with a bound on the error that rounding the
weights (and weight gradients) to a 16-bit type of half-step ``u`` can cause, as a sum
of absolute values, from which the tests derive their tolerances."""
import math

import numpy as np


_PI = 314159265358979323846264338327950288419716939937510  # 10^50 pi


def angles(positions, inv_freq):
    """[..., rot / 2]: position times frequency (the float64 value as it stands), reduced to
    [-pi, pi].  Product and reduction in whole numbers: in float64 they are off by 2^-53 of
    the angle, which at positions near 2^31 is more than the kernel's own rounding."""
    p, one = np.asarray(positions).astype(object), 1 << 200
    turn = one * 10 ** 50 // (2 * _PI)
    out = np.empty(p.shape + (len(inv_freq),))
    for i, f in enumerate(inv_freq):
        m, e = math.frexp(float(f))
        x = p * (int(m * 2.0 ** 53) * turn)
        x = x * 2 ** (e - 53) if e > 53 else x // 2 ** (53 - e)
        out[..., i] = ((x + one // 2) % one - one // 2) / one * (2 * math.pi)
    return out


def rotary(x, positions, inv_freq, interleaved=False, mscale=1.0, inverse=False):
    """x [B, T, H, d] -> rotated, float64."""
    x = np.asarray(x, np.float64)
    half = len(inv_freq)
    t = angles(positions, inv_freq)
    c, s = mscale * np.cos(t)[:, :, None], mscale * np.sin(t)[:, :, None]
    if inverse:
        s = -s
    i = np.arange(half)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y = x.copy()
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


def visible(lq, lk, causal, window):
    """[lq, lk]: keys a query sees; query i stands at position i + lk - lq of the keys."""
    at = np.arange(lq)[:, None] + lk - lq
    j = np.arange(lk)[None, :]
    see = np.ones((lq, lk), bool)
    if causal:
        see &= j <= at
    if window:
        see &= j > at - window
    return see


def attention(q, k, v, causal=True, window=0, scale=None, do=None):
    """One sequence: q [Tq, Hq, d], k, v [Tk, Hk, d].  Returns a dict with ``o``, ``lse``
    and, with ``do``, ``dq, dk, dv``; for each ``<name>_abs``, the sum of the absolute terms
    whose weights a kernel rounds; and what errors relative to sum |do||o|, to
    sum |do| (p |v|) and to sum |do||v| in the weights' gradients come to in dq and dk
    (``_dd``, ``_da``, ``_dp``)."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    Tq, Hq, d = q.shape
    Tk, Hk, _ = k.shape
    G = Hq // Hk
    scale = d ** -0.5 if scale is None else scale
    see = visible(Tq, Tk, causal, window)
    r = dict(o=np.zeros((Tq, Hq, d)), lse=np.full((Hq, Tq), -np.inf), o_abs=np.zeros((Tq, Hq, d)))
    if do is not None:
        do = np.asarray(do, np.float64)
        for n, like in (("dq", q), ("dk", k), ("dv", v)):
            r[n], r[n + "_abs"] = np.zeros_like(like), np.zeros_like(like)
        for n in ("_dd", "_da", "_dp"):
            r["dq" + n], r["dk" + n] = np.zeros_like(q), np.zeros_like(k)
    if Tq == 0 or Tk == 0:
        return r
    for h in range(Hq):
        s = np.where(see, scale * q[:, h] @ k[:, h // G].T, -np.inf)
        m = s.max(1, keepdims=True)
        m0 = np.where(np.isneginf(m), 0.0, m)
        e = np.exp(s - m0)
        tot = e.sum(1, keepdims=True)
        with np.errstate(divide="ignore"):
            r["lse"][h] = (m0 + np.log(tot))[:, 0]
        p = e / np.where(tot == 0, 1.0, tot)
        r["o"][:, h] = p @ v[:, h // G]
        r["o_abs"][:, h] = p @ np.abs(v[:, h // G])
        if do is not None:
            g = do[:, h]
            r["dv"][:, h // G] += p.T @ g
            r["dv_abs"][:, h // G] += p.T @ np.abs(g)
            dd = (g * r["o"][:, h]).sum(1, keepdims=True)
            ds = p * (g @ v[:, h // G].T - dd) * scale
            r["dq"][:, h] = ds @ k[:, h // G]
            r["dk"][:, h // G] += ds.T @ q[:, h]
            r["dq_abs"][:, h] = np.abs(ds) @ np.abs(k[:, h // G])
            r["dk_abs"][:, h // G] += np.abs(ds).T @ np.abs(q[:, h])
            for n, size in (("_dd", (np.abs(g) * np.abs(r["o"][:, h])).sum(1, keepdims=True)),
                            ("_da", (np.abs(g) * r["o_abs"][:, h]).sum(1, keepdims=True)),
                            ("_dp", np.abs(g) @ np.abs(v[:, h // G]).T)):
                w = p * scale * size
                r["dq" + n][:, h] = w @ np.abs(k[:, h // G])
                r["dk" + n][:, h // G] += w.T @ np.abs(q[:, h])
    return r


# ------------------------------------------------------------------ 8-bit cache


def e4m3_decode(code):
    code = np.asarray(code).astype(np.int64)
    sign = np.where(code & 0x80, -1.0, 1.0)
    e, m = (code >> 3) & 15, code & 7
    val = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    return np.where((code & 0x7f) == 0x7f, np.nan, sign * val)


_E4M3 = e4m3_decode(np.arange(127))  # 0 .. 448, ascending


def e4m3_encode(x):
    """Round to nearest, ties to the even code, saturating at 448; NaN keeps NaN."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=448.0, neginf=-448.0)), 448.0)
    lo = np.clip(np.searchsorted(_E4M3, a, side="right") - 1, 0, 125)
    dl, dh = a - _E4M3[lo], _E4M3[lo + 1] - a
    up = (dh < dl) | ((dh == dl) & (lo % 2 == 1))
    code = lo + up
    code = np.where(np.isnan(x), 0x7f, code)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def page_scale(amax):
    """Smallest 2^e >= 2^-100 with amax <= 448 2^e."""
    if amax == 0:
        return 2.0 ** -100
    e = math.ceil(math.log2(amax) - math.log2(448.0))
    while amax > 448.0 * 2.0 ** e:
        e += 1
    while e > -100 and amax <= 448.0 * 2.0 ** (e - 1):
        e -= 1
    return 2.0 ** max(e, -100)


def kv_append(x, pages, scale, table, start, count):
    """x [B, T, Hk, d] float64; pages uint8 [num, Hk, page, d]; scale [num, Hk]; both
    returned as new arrays."""
    pages, scale = pages.copy(), np.asarray(scale, np.float64).copy()
    num, Hk, page, d = pages.shape
    x = np.asarray(x, np.float64)
    for b in range(x.shape[0]):
        n = min(max(int(count[b]), 0), x.shape[1])
        if start[b] < 0:
            continue
        for slot in range(int(start[b]) // page, (int(start[b]) + n - 1) // page + 1 if n else 0):
            if slot >= table.shape[1] or not 0 <= table[b, slot] < num:
                continue
            i = table[b, slot]
            lo, hi = max(int(start[b]), slot * page), min(int(start[b]) + n, (slot + 1) * page)
            held = lo - slot * page
            for h in range(Hk):
                rows = x[b, lo - start[b]: hi - start[b], h]
                fin = np.abs(rows[np.isfinite(rows)])
                s = page_scale(fin.max() if fin.size else 0.0)
                if held:
                    s = max(s, scale[i, h])
                    if s != scale[i, h]:
                        pages[i, h, :held] = e4m3_encode(e4m3_decode(pages[i, h, :held]) * (scale[i, h] / s))
                pages[i, h, held: hi - slot * page] = e4m3_encode(rows / s)
                scale[i, h] = s
    return pages, scale


def attn_step(q, k_pages, v_pages, k_scale, v_scale, table, lens, scale=None, window=0):
    """q [B, Hq, d].  Returns (o, o_abs)."""
    q = np.asarray(q, np.float64)
    B, Hq, d = q.shape
    num, Hk, page, _ = k_pages.shape
    G = Hq // Hk
    scale = d ** -0.5 if scale is None else scale
    o, oa = np.zeros((B, Hq, d)), np.zeros((B, Hq, d))
    for b in range(B):
        n = min(max(int(lens[b]), 0), table.shape[1] * page)
        js = [j for j in range(max(0, n - window) if window else 0, n) if 0 <= table[b, j // page] < num]
        if not js:
            continue
        ids, rows = np.array([table[b, j // page] for j in js]), np.array([j % page for j in js])
        for h in range(Hk):
            kk = e4m3_decode(k_pages[ids, h, rows]) * np.asarray(k_scale, np.float64)[ids, h][:, None]
            vv = e4m3_decode(v_pages[ids, h, rows]) * np.asarray(v_scale, np.float64)[ids, h][:, None]
            s = scale * q[b, h * G: (h + 1) * G] @ kk.T
            e = np.exp(s - s.max(1, keepdims=True))
            p = e / e.sum(1, keepdims=True)
            o[b, h * G: (h + 1) * G] = p @ vv
            oa[b, h * G: (h + 1) * G] = p @ np.abs(vv)
    return o, oa

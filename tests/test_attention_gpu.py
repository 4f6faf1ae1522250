"""Parity of softmax attention and its gradients against the float64 oracle.

Tolerances per element, from the arithmetic.  u = 2^-8 is half a bfloat16 step.
  o   : output rounding u |o|, weights rounded as operands u sum p |v|, and 1e-4 of that
        sum for float32 scores (128 exact products each, sum |q k| scale below 64 in these
        inputs: 64 2^-21), exponentials (2^-21) and sums
  lse : 64 2^-21 = 3e-5
  dv  : the same with dO for v;  lse adds 3e-5 to a weight
  dq, dk : u |dq|; u sum |ds||k| for ds rounded as an operand, 2e-4 of it for p; D = dO.o
        from a bfloat16 o (rows of more than 8 keys; fewer take it in float32, which is
        smaller): u sum p (sum |dO||o|) scale |k|, with a kernel's own o another
        u sum p (sum |dO| sum p |v|) scale |k|; dO.v and D as float32 sums of 128 products:
        2^-17 of sum p (sum |dO||v|) scale |k|"""
import numpy as np
import pytest
import torch

from oracle import attention as A

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


@pytest.fixture(scope="module")
def m():
    import gated_delta_rule_115_b200 as m
    m.lib()
    return m


def rnd(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def within(got, want, tol, what):
    err = np.abs(got.double().cpu().numpy() - want)
    bad = ~(err <= tol + 1e-30)
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(err - tol)), np.argwhere(bad)[:3].tolist())


def check_fwd(o, lse, r):
    within(o, r["o"], U * np.abs(r["o"]) + (U + 1e-4) * r["o_abs"], "o")
    got = lse.double().cpu().numpy()
    none = np.isneginf(r["lse"])
    assert np.array_equal(np.isneginf(got), none)
    assert (np.abs(got[~none] - r["lse"][~none]) <= 3e-5).all()


def check_bwd(g, r, own_o=False):
    within(g["dv"], r["dv"], U * np.abs(r["dv"]) + (U + 1e-4) * r["dv_abs"], "dv")
    for n in ("dq", "dk"):
        tol = U * np.abs(r[n]) + (U + 2e-4) * r[n + "_abs"] + U * r[n + "_dd"] + 2.0 ** -17 * r[n + "_dp"]
        within(g[n], r[n], tol + (U * 1.01 * r[n + "_da"] if own_o else 0.0), n)


def oracle(q, k, v, do, seqs, **kw):
    """Results of every sequence (rows of q, rows of k)."""
    return [A.attention(q[a].double().numpy(), k[b].double().numpy(), v[b].double().numpy(),
                        do=None if do is None else do[a].double().numpy(), **kw) for a, b in seqs]


CASES = [
    # B, Tq, Tk, Hq, Hk, d, causal, window
    (1, 1, 1, 1, 1, 64, True, 0), (1, 128, 128, 1, 1, 128, False, 0), (2, 127, 127, 2, 1, 128, True, 0),
    (1, 129, 129, 3, 3, 64, True, 0), (2, 300, 300, 4, 2, 128, True, 0), (1, 513, 513, 2, 2, 64, False, 0),
    (1, 257, 700, 2, 1, 128, True, 0), (1, 700, 257, 2, 2, 128, True, 0), (1, 1, 400, 8, 2, 128, True, 0),
    (1, 640, 640, 2, 1, 64, True, 1), (1, 640, 640, 2, 1, 128, True, 128), (1, 700, 700, 2, 2, 64, True, 200),
    (2, 300, 500, 2, 1, 128, False, 150), (1, 1000, 1000, 6, 2, 128, True, 0), (1, 100, 1, 2, 2, 64, True, 0),
    (1, 385, 640, 1, 1, 128, False, 0), (3, 256, 256, 5, 1, 64, True, 77), (1, 2100, 2100, 1, 1, 128, True, 0),
    # enough blocks for two query tiles each: of one head, or two heads' of an even group; the
    # latter also has two heads to a block of dq at d = 64
    (1, 1400, 1400, 28, 28, 128, True, 0), (1, 1400, 1400, 28, 28, 64, True, 300), (2, 900, 1000, 32, 2, 128, True, 0),
    (1, 1201, 1201, 64, 2, 64, True, 0), (1, 1201, 700, 64, 2, 64, True, 111), (2, 640, 650, 64, 8, 64, False, 0),
]


@pytest.mark.parametrize("B,Tq,Tk,Hq,Hk,d,causal,window", CASES)
def test_forward(m, B, Tq, Tk, Hq, Hk, d, causal, window):
    q, k, v = rnd(B, Tq, Hq, d, seed=1), rnd(B, Tk, Hk, d, seed=2), rnd(B, Tk, Hk, d, seed=3)
    o, lse = m.attn_fwd(q.cuda(), k.cuda(), v.cuda(), causal=causal, window=window)
    m.device_wait_status()
    for b, r in enumerate(oracle(q, k, v, None, [(b, b) for b in range(B)], causal=causal, window=window)):
        check_fwd(o[b], lse[b], r)


@pytest.mark.parametrize("B,Tq,Tk,Hq,Hk,d,causal,window", CASES)
def test_backward(m, B, Tq, Tk, Hq, Hk, d, causal, window):
    q, k, v, do = (rnd(B, T, H, d, seed=s) for T, H, s in ((Tq, Hq, 1), (Tk, Hk, 2), (Tk, Hk, 3), (Tq, Hq, 4)))
    rs = oracle(q, k, v, do, [(b, b) for b in range(B)], causal=causal, window=window)
    o = torch.from_numpy(np.stack([r["o"] for r in rs])).to(torch.bfloat16).cuda()
    lse = torch.from_numpy(np.stack([r["lse"] for r in rs])).float().cuda()
    args = (q.cuda(), k.cuda(), v.cuda(), o, lse, do.cuda())
    g = m.attn_bwd(*args, causal=causal, window=window)
    m.device_wait_status()
    for b, r in enumerate(rs):
        check_bwd({n: t[b] for n, t in g.items()}, r)
    again = m.attn_bwd(*args, causal=causal, window=window)
    assert all(torch.equal(g[n], again[n]) for n in g)


PACKED = [([5, 0, 130, 1, 256, 77], None, 4, 2, 128, True, 0), ([300, 128, 0, 0, 1], None, 2, 2, 64, True, 50),
          ([10, 200, 3], [300, 50, 3], 2, 1, 128, True, 0), ([64, 0, 100], [0, 90, 129], 3, 3, 64, False, 0),
          ([0, 0], [3, 5], 2, 2, 64, True, 0)]


def spans(lens):
    at = np.concatenate([[0], np.cumsum(lens)]).tolist()
    return at, [(0, slice(a, b)) for a, b in zip(at, at[1:])]


@pytest.mark.parametrize("lens,lens_k,Hq,Hk,d,causal,window", PACKED)
def test_packed(m, lens, lens_k, Hq, Hk, d, causal, window):
    """Forward and, on the kernel's own o and lse, backward; NaN in one sequence stays there."""
    cu, sq = spans(lens)
    ck, sk = spans(lens_k or lens)
    q, k, v, do = (rnd(1, T, H, d, seed=s) for T, H, s in ((cu[-1], Hq, 1), (ck[-1], Hk, 2), (ck[-1], Hk, 3), (cu[-1], Hq, 4)))
    args = dict(cu_seqlens=cu, cu_seqlens_k=None if lens_k is None else torch.tensor(ck), causal=causal, window=window)
    dev = [t.cuda() for t in (q, k, v, do)]
    o, lse = m.attn_fwd_varlen(*dev[:3], **args)
    g = m.attn_bwd_varlen(*dev[:3], o, lse, dev[3], **args)
    m.device_wait_status()
    for (a, b), r in zip(zip(sq, sk), oracle(q, k, v, do, list(zip(sq, sk)), causal=causal, window=window)):
        check_fwd(o[a], lse[0, :, a[1]], r)
        check_bwd({"dq": g["dq"][a], "dk": g["dk"][b], "dv": g["dv"][b]}, r, own_o=True)
    big = max(range(len(lens)), key=lambda i: lens[i])
    if lens[big]:
        for t, s in zip(dev, (sq, sk, sk, sq)):
            t[s[big]] = float("nan")
        o2, lse2 = m.attn_fwd_varlen(*dev[:3], **args)
        g2 = m.attn_bwd_varlen(*dev[:3], o2, lse2, dev[3], **args)
        for i in range(len(lens)):
            if i != big:
                assert torch.equal(o2[sq[i]], o[sq[i]])
                for n, s in (("dq", sq), ("dk", sk), ("dv", sk)):
                    assert torch.equal(g2[n][s[i]], g[n][s[i]]), (n, i)
    m.device_wait_status()


def test_many_sequences(m):
    """More sequences than one launch holds, against the same ones as a dense batch."""
    n, T, H, d = 300, 9, 2, 64
    q, k, v, do = (rnd(n, T, H, d, seed=s).cuda() for s in (1, 2, 3, 4))
    o, lse = m.attn_fwd(q, k, v)
    g = m.attn_bwd(q, k, v, o, lse, do)
    flat = [t.reshape(1, n * T, H, d) for t in (q, k, v, do)]
    cu = list(range(0, n * T + 1, T))
    o2, lse2 = m.attn_fwd_varlen(*flat[:3], cu)
    assert torch.equal(o2.reshape(o.shape), o)
    assert torch.equal(lse2.reshape(H, n, T).transpose(0, 1), lse)
    g2 = m.attn_bwd_varlen(*flat[:3], o2, lse2, flat[3], cu)
    for x in g:
        assert torch.equal(g2[x].reshape(g[x].shape), g[x])
    r = A.attention(q[0].double().cpu().numpy(), k[0].double().cpu().numpy(), v[0].double().cpu().numpy(),
                    do=do[0].double().cpu().numpy())
    check_fwd(o[0], lse[0], r)
    check_bwd({x: t[0] for x, t in g.items()}, r, own_o=True)


def test_packed_projection_scale_and_large_scores(m):
    """q, k, v as parts of one projection's rows; a scale of its own; scores in the hundreds,
    where the running maximum moves."""
    B, T, Hq, Hk, d = 2, 333, 4, 2, 64
    x = rnd(B, T, (Hq + 2 * Hk) * d, seed=7).cuda()
    part = [x[..., a * d: b * d].unflatten(-1, (b - a, d)) for a, b in ((0, 4), (4, 6), (6, 8))]
    dense = [t.contiguous() for t in part]
    do = rnd(B, T, Hq, d, seed=8).cuda()
    for scale in (0.05, 8.0):
        o, lse = m.attn_fwd(*part, scale=scale)
        o1, lse1 = m.attn_fwd(*dense, scale=scale)
        assert torch.equal(o, o1) and torch.equal(lse, lse1)
        g, g1 = (m.attn_bwd(*t, o, lse, do, scale=scale) for t in (part, dense))
        assert all(torch.equal(g[n], g1[n]) for n in g)
        for b in range(B):
            q, k, v = (t[b].double().cpu().numpy() for t in dense)
            r = A.attention(q, k, v, scale=scale, do=do[b].double().cpu().numpy())
            # scores up to sum |q k| scale = 64 * 8 * 2: 2^-21 of it on lse and on a weight
            e = max(1e-4, 1024 * 2.0 ** -20)
            within(o[b], r["o"], U * np.abs(r["o"]) + (U + e) * r["o_abs"], "o")
            assert (np.abs(lse[b].double().cpu().numpy() - r["lse"]) <= e).all()
            if scale < 1:
                check_bwd({n: t[b] for n, t in g.items()}, r, own_o=True)


def test_infinite_and_nan_keys_behind_the_mask(m):
    """Keys that a causal query does not see: a NaN in them reaches no score."""
    T, d = 300, 128
    q, k, v = (rnd(1, T, 1, d, seed=s).cuda() for s in (1, 2, 3))
    o, lse = m.attn_fwd(q, k, v)
    k2 = k.clone()
    k2[0, 250, 0, 3], k2[0, 280, 0, 0] = float("nan"), float("inf")
    o2, lse2 = m.attn_fwd(q, k2, v)
    assert torch.equal(o2[:, :250], o[:, :250]) and torch.equal(lse2[..., :250], lse[..., :250])
    assert torch.isnan(o2[:, 250:]).all()


def test_autograd_graph_and_other_stream(m):
    """The wrapper's gradients, a captured and replayed pass, and a pass on another stream."""
    B, T, Hq, Hk, d = 1, 200, 4, 2, 128
    q, k, v, do = (rnd(B, T, H, d, seed=s).cuda() for H, s in ((Hq, 1), (Hk, 2), (Hk, 3), (Hq, 4)))
    o, lse = m.attn_fwd(q, k, v)
    g = m.attn_bwd(q, k, v, o, lse, do)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    out = m.MuirAttentionFunction.apply(*leaves)
    out.backward(do)
    assert torch.equal(out, o)
    for t, n in zip(leaves, ("dq", "dk", "dv")):
        assert torch.equal(t.grad, g[n])
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    m.MuirAttentionFunction.apply(*leaves, True, 0, None, [0, 50, 200]).backward(do)
    o3, lse3 = m.attn_fwd_varlen(q, k, v, [0, 50, 200])
    g3 = m.attn_bwd_varlen(q, k, v, o3, lse3, do, [0, 50, 200])
    for t, n in zip(leaves, ("dq", "dk", "dv")):
        assert torch.equal(t.grad, g3[n])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        m.attn_bwd(q, k, v, *m.attn_fwd(q, k, v), do)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        og, lg = m.attn_fwd(q, k, v)
        gg = m.attn_bwd(q, k, v, og, lg, do)
    for t in (q, k, v, do):
        t.copy_(t.roll(1, 1))
    graph.replay()
    o2, lse2 = m.attn_fwd(q, k, v)
    g2 = m.attn_bwd(q, k, v, o2, lse2, do)
    assert torch.equal(og, o2) and torch.equal(lg, lse2) and all(torch.equal(gg[n], g2[n]) for n in gg)
    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.current_stream())
        o4, _ = m.attn_fwd(q, k, v)
    s.synchronize()
    assert torch.equal(o4, o2)


def test_gradients_by_differences(m):
    """The analytic gradient against central differences of the kernel's own forward.  A step
    h along a direction: o is rounded to bfloat16, so the slope of sum(o dO) is uncertain by
    2 u sum(|o||dO| + |dO| sum p|v|) / (2 h), and h^2 / 6 times the third derivative; the
    bound below takes the first in full (worst case, so the comparison is of the whole
    gradient against its size, not of its digits)."""
    T, d, h = 64, 64, 0.25
    q, k, v, do = (rnd(1, T, 1, d, seed=s).float() for s in (1, 2, 3, 4))
    r = A.attention(*(t[0].double().numpy() for t in (q, k, v)), do=do[0].double().numpy())
    o, lse = m.attn_fwd(*(t.to(torch.bfloat16).cuda() for t in (q, k, v)))
    g = m.attn_bwd(*(t.to(torch.bfloat16).cuda() for t in (q, k, v)), o, lse, do.to(torch.bfloat16).cuda())
    # v enters linearly: the difference quotient has no truncation error.  Moving v along its
    # own gradient makes the slope as large as it gets: |dv|^2 / |dv|
    step = torch.from_numpy(r["dv"])[None].float()
    step = (step / step.abs().max()).to(torch.bfloat16).float()
    hi, lo = ((v + s * h * step).to(torch.bfloat16) for s in (1, -1))
    moved = (hi.double() - lo.double())
    f = [(m.attn_fwd(q.to(torch.bfloat16).cuda(), k.to(torch.bfloat16).cuda(), t.cuda())[0].double().cpu() * do.double()).sum()
         for t in (hi, lo)]
    slope = float((g["dv"].double().cpu() * moved).sum())
    size = 0.0
    for t in (hi, lo):
        rr = A.attention(q[0].double().numpy(), k[0].double().numpy(), t[0].double().numpy())
        size += U * float(((np.abs(rr["o"]) + 1.03 * rr["o_abs"]) * np.abs(do[0].double().numpy())).sum())
    tol = size + float(((U * np.abs(r["dv"]) + (U + 1e-4) * r["dv_abs"]) * moved[0].abs().numpy()).sum())
    assert abs(float(f[0] - f[1]) - slope) <= tol
    # and the bound means something: the slope itself is several times larger
    assert abs(slope) > 2 * tol


@pytest.mark.parametrize("d,Hq,Hk", [(64, 16, 4), (128, 8, 8)])
def test_many_launches(m, d, Hq, Hk):
    """Hundreds of launches in a row give one result, and no wait inside them runs out: the
    two halves of a block's columns may drift apart by more than a step."""
    q, do = (rnd(4, 640, Hq, d, seed=s).cuda() for s in (1, 4))
    k, v = (rnd(4, 640, Hk, d, seed=s).cuda() for s in (2, 3))
    o, lse = m.attn_fwd(q, k, v)
    g = m.attn_bwd(q, k, v, o, lse, do)
    for _ in range(600):
        o2, lse2 = m.attn_fwd(q, k, v)
        g2 = m.attn_bwd(q, k, v, o, lse, do)
    m.device_wait_status()
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and all(torch.equal(g[n], g2[n]) for n in g)


@pytest.mark.parametrize("d", [64, 128])
def test_one_visible_key_has_no_score_gradient(m, d):
    """A weight of 1 does not depend on its score: dq and what it adds to dk are exactly
    zero, and dv is dO's (rounded) sum."""
    for lens, causal, window in (([1, 1, 1], True, 0), ([1, 300, 1], True, 0), ([200, 130], True, 1), ([1], False, 0)):
        cu, _ = spans(lens)
        q, k, v, do = (rnd(1, cu[-1], H, d, seed=s).cuda() for s, H in ((1, 4), (2, 2), (3, 2), (4, 4)))
        o, lse = m.attn_fwd_varlen(q, k, v, cu, causal=causal, window=window)
        g = m.attn_bwd_varlen(q, k, v, o, lse, do, cu, causal=causal, window=window)
        for a, b in zip(cu, cu[1:]):
            rows = slice(a, b) if window == 1 or b - a == 1 else slice(a, a + 1)
            assert not g["dq"][0, rows].any() and torch.equal(o[0, rows], v[0, rows].repeat_interleave(2, 1))
            if window == 1 or b - a == 1:
                assert not g["dk"][0, rows].any()
                want = do[0, rows].double().unflatten(1, (2, 2)).sum(2)
                assert ((g["dv"][0, rows].double() - want).abs() <= U * want.abs() + 1e-6).all()
    # one key, many queries
    q, k, v, do = (rnd(1, T, H, d, seed=s).cuda() for s, T, H in ((1, 50, 4), (2, 1, 2), (3, 1, 2), (4, 50, 4)))
    o, lse = m.attn_fwd(q, k, v, causal=False)
    g = m.attn_bwd(q, k, v, o, lse, do, causal=False)
    assert not g["dq"].any() and not g["dk"].any()
    m.device_wait_status()


@pytest.mark.parametrize("T,window,Hq,Hk,d", [(2, 0, 4, 2, 64), (5, 0, 2, 2, 128), (8, 0, 6, 2, 64), (300, 2, 2, 1, 128),
                                              (300, 8, 3, 3, 64)])
def test_rows_of_few_keys(m, T, window, Hq, Hk, d):
    """Up to eight visible keys: D comes from the keys themselves, and a rounded o adds
    nothing to the gradients."""
    q, k, v, do = (rnd(3, T, H, d, seed=s) for s, H in ((1, Hq), (2, Hk), (3, Hk), (4, Hq)))
    dev = [t.cuda() for t in (q, k, v, do)]
    o, lse = m.attn_fwd(*dev[:3], window=window)
    g = m.attn_bwd(*dev[:3], o, lse, dev[3], window=window)
    wrong = m.attn_bwd(*dev[:3], torch.zeros_like(o), lse, dev[3], window=window)
    assert all(torch.equal(g[n], wrong[n]) for n in g)  # o is not read for these rows' D
    for b, r in enumerate(oracle(q, k, v, do, [(b, b) for b in range(3)], window=window)):
        for n in ("dq", "dk"):
            tol = U * np.abs(r[n]) + (U + 2e-4) * r[n + "_abs"] + 2.0 ** -17 * r[n + "_dp"]
            within(g[n][b], r[n], tol, n)
    m.device_wait_status()


@pytest.mark.parametrize("B,Tq,Tk,Hq,Hk,d,window", [
    (1, 300, 300, 2, 1, 64, 1), (2, 300, 333, 2, 2, 128, 1), (1, 333, 200, 4, 2, 64, 1), (1, 129, 2, 2, 1, 128, 1),
    (2, 200, 333, 4, 2, 64, 5), (1, 333, 200, 2, 1, 128, 8), (1, 140, 140, 8, 4, 64, 2)])
def test_windows_that_look_ahead(m, B, Tq, Tk, Hq, Hk, d, window):
    """Not causal, with a window: a query sees the last few keys up to its own and all
    that follow; with a window of 1 the last query alone sees one key."""
    q, k, v, do = (rnd(B, T, H, d, seed=s) for T, H, s in ((Tq, Hq, 1), (Tk, Hk, 2), (Tk, Hk, 3), (Tq, Hq, 4)))
    rs = oracle(q, k, v, do, [(b, b) for b in range(B)], causal=False, window=window)
    dev = [t.cuda() for t in (q, k, v, do)]
    o, lse = m.attn_fwd(*dev[:3], causal=False, window=window)
    g = m.attn_bwd(*dev[:3], o, lse, dev[3], causal=False, window=window)
    m.device_wait_status()
    for b, r in enumerate(rs):
        check_fwd(o[b], lse[b], r)
        check_bwd({n: t[b] for n, t in g.items()}, r, own_o=True)
    if window == 1:
        assert not g["dq"][:, -1].any()


@pytest.mark.parametrize("d,causal,window", [(64, True, 0), (128, True, 5), (64, False, 0), (128, True, 40)])
def test_ragged_sequences_of_several_launches(m, d, causal, window):
    """300 sequences of their own lengths, each against the oracle: what a later launch takes
    from its place in the list (offsets, order of blocks, rows of few keys) is its own."""
    r = np.random.default_rng(d + window)
    lens = r.integers(0, 40, 300)
    lens_k = np.where(r.random(300) < 0.5, lens, r.integers(0, 60, 300))
    for i, (a, b) in {0: (1, 1), 5: (300, 300), 127: (9, 9), 128: (140, 141), 255: (3, 7), 256: (1, 30), 299: (17, 17)}.items():
        lens[i], lens_k[i] = a, b
    cu, sq = spans(lens)
    ck, sk = spans(lens_k)
    q, k, v, do = (rnd(1, T, H, d, seed=s) for T, H, s in ((cu[-1], 4, 1), (ck[-1], 2, 2), (ck[-1], 2, 3), (cu[-1], 4, 4)))
    args = dict(cu_seqlens=cu, cu_seqlens_k=ck, causal=causal, window=window)
    dev = [t.cuda() for t in (q, k, v, do)]
    o, lse = m.attn_fwd_varlen(*dev[:3], **args)
    g = m.attn_bwd_varlen(*dev[:3], o, lse, dev[3], **args)
    m.device_wait_status()
    for a, b, res in zip(sq, sk, oracle(q, k, v, do, list(zip(sq, sk)), causal=causal, window=window)):
        check_fwd(o[a], lse[0, :, a[1]], res)
        check_bwd({"dq": g["dq"][a], "dk": g["dk"][b], "dv": g["dv"][b]}, res, own_o=True)


@pytest.mark.parametrize("d,Hq,Hk", [(64, 16, 4), (128, 8, 8)])
def test_every_one_of_many_launches(m, d, Hq, Hk):
    """Each of hundreds of results is compared, on the device, not the last one alone."""
    q, do = (rnd(3, 513, Hq, d, seed=s).cuda() for s in (1, 4))
    k, v = (rnd(3, 513, Hk, d, seed=s).cuda() for s in (2, 3))
    o, lse = m.attn_fwd(q, k, v)
    g = m.attn_bwd(q, k, v, o, lse, do)
    differ = torch.zeros(5, dtype=torch.int64, device="cuda")
    for _ in range(400):
        o2, lse2 = m.attn_fwd(q, k, v)
        g2 = m.attn_bwd(q, k, v, o, lse, do)
        pairs = [(o, o2), (lse, lse2)] + [(g[n], g2[n]) for n in ("dq", "dk", "dv")]
        differ += torch.stack([(a != b).any() for a, b in pairs])
    m.device_wait_status()
    assert not differ.any(), differ.tolist()

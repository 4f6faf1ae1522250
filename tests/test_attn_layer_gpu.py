"""The softmax-attention layer's operators together, as a stack that mixes it with the gated
delta rule runs them, and at the ends of their ranges: training, prefill and decoding from
one packed projection; two calls at once; tensors past 2^31 elements and caches past 2^32
bytes; views that must be refused."""
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


def test_training_layer(m):
    """One projection's rows -> rotary in place -> attention -> gradients -> rotary's transpose
    in place on the gradients, against the float64 chain.  Rotated q and k are rounded to
    bfloat16 in between: the oracle takes the rounded ones, so every stage keeps its bound;
    the last rounding of the rotated gradients adds u |y|, and the gradients' own errors pass
    the rotation as sqrt(2) of the pair's larger one."""
    T, Hq, Hk, d = 300, 4, 2, 64
    x = rnd(1, T, (Hq + 2 * Hk) * d, seed=1).cuda()
    do = rnd(1, T, Hq, d, seed=2)
    q, k, v = (x[..., a * d: b * d].unflatten(-1, (b - a, d)) for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)))
    f, s = m.rotary_frequencies(32, scaling="yarn", factor=4.0)
    raw = [t.double().cpu().numpy() for t in (q, k)]
    m.rotary(q, k, inv_freq=f, mscale=s, q_out=q, k_out=k)
    pos = np.arange(T)[None]
    for t, r in zip((q, k), raw):
        w = A.rotary(r, pos, f.cpu().numpy(), mscale=s)
        assert (np.abs(t.double().cpu().numpy() - w) <= U * np.abs(w) + 6e-7 * 2 * s * np.abs(r).max()).all()
    o, lse = m.attn_fwd(q, k, v)
    g = m.attn_bwd(q, k, v, o, lse, do.cuda())
    r = A.attention(*(t[0].double().cpu().numpy() for t in (q, k, v)), do=do[0].double().numpy())
    grads = {n: g[n].clone() for n in ("dq", "dk")}
    m.rotary(g["dq"], g["dk"], inv_freq=f, mscale=s, inverse=True, q_out=g["dq"], k_out=g["dk"])
    for n in ("dq", "dk"):
        tol = U * np.abs(r[n]) + (U + 2e-4) * r[n + "_abs"] + U * (r[n + "_dd"] + 1.01 * r[n + "_da"]) + 2.0 ** -17 * r[n + "_dp"]
        assert (np.abs(grads[n][0].double().cpu().numpy() - r[n]) <= tol).all(), n
        want = A.rotary(r[n][None], pos, f.cpu().numpy(), mscale=s, inverse=True)
        pair = tol.copy()
        pair[..., :16] = pair[..., 16:32] = np.sqrt(2) * s * np.maximum(tol[..., :16], tol[..., 16:32])
        err = np.abs(g[n].double().cpu().numpy() - want)
        assert (err <= pair + U * (np.abs(want) + pair) + 1e-6).all(), n
    m.device_wait_status()


def test_prefill_then_decode(m):
    """Prompts of different length go through attention and into the cache (right-padded
    batch), then five tokens each are decoded: rotary at the token's position, append, step.
    Each step is checked against float64 attention over the very codes in the cache."""
    B, Hq, Hk, d, page = 3, 8, 2, 128, 32
    lens = np.array([70, 1, 33])
    T = int(lens.max())
    f, _ = m.rotary_frequencies(d)
    q, k, v = rnd(B, T, Hq, d, seed=1).cuda(), rnd(B, T, Hk, d, seed=2).cuda(), rnd(B, T, Hk, d, seed=3).cuda()
    q, k = m.rotary(q, k, inv_freq=f)
    o, lse = m.attn_fwd(q, k, v)
    for b in range(B):  # causal: the padding behind a prompt does not reach its rows
        r = A.attention(*(t[b, : lens[b]].double().cpu().numpy() for t in (q, k, v)))
        err = np.abs(o[b, : lens[b]].double().cpu().numpy() - r["o"])
        assert (err <= U * np.abs(r["o"]) + (U + 1e-4) * r["o_abs"]).all()
    pages = -(-(T + 5) // page)
    table = np.random.default_rng(1).permutation(B * pages).reshape(B, pages).astype(np.int32)
    tb = torch.from_numpy(table).cuda()
    c = m.kv_cache(B * pages, Hk, page, d)
    n = torch.from_numpy(lens.astype(np.int32)).cuda()
    m.kv_append(k, v, *c, tb, torch.zeros_like(n), count=n)
    code = lambda t: t.view(torch.uint8).cpu().numpy()  # noqa: E731
    for i in range(5):
        qt, kt, vt = (rnd(B, 1, H, d, seed=10 * i + s).cuda() for H, s in ((Hq, 1), (Hk, 2), (Hk, 3)))
        qt, kt = m.rotary(qt, kt, positions=n[:, None], inv_freq=f)
        before = [code(t).copy() for t in c[:2]]
        m.kv_append(kt, vt, *c, tb, n)
        n += 1
        ot = m.attn_step(qt[:, 0], *c, tb, n)
        for b in range(B):  # pages that no token went to are as they were
            keep = [p for j, p in enumerate(table[b]) if j != (int(n[b]) - 1) // page]
            assert all(np.array_equal(code(t)[keep], w[keep]) for t, w in zip(c[:2], before))
        want, size = A.attn_step(qt[:, 0].double().cpu().numpy(), code(c[0]), code(c[1]), c[2].cpu().numpy(),
                                 c[3].cpu().numpy(), table, n.cpu().numpy())
        err = np.abs(ot.double().cpu().numpy() - want)
        assert (err <= U * np.abs(want) + (2.0 ** -11 + 7e-5) * size).all()
    m.device_wait_status()


def test_two_streams_at_once(m):
    """The same operators on two streams, with inputs of their own: results of each alone."""
    def inputs(seed):
        return [rnd(1, 700, H, 128, seed=seed + i).cuda() for i, H in enumerate((8, 4, 4, 8))]

    def run(x):
        o, lse = m.attn_fwd(*x[:3])
        g = m.attn_bwd(*x[:3], o, lse, x[3])
        return [o, lse, g["dq"], g["dk"], g["dv"]]

    sets = [inputs(1), inputs(50)]
    alone = [run(x) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = run(sets[i])
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_past_32_bit_offsets(m):
    """Queries past 2^31 elements: the last tokens of a long sequence under a window, forward
    and backward, against the oracle on those tokens alone."""
    T, H, d, w = 265000, 64, 128, 100
    assert T * H * d > 2 ** 31
    tail = 300
    torch.manual_seed(0)
    q = torch.randn(1, T, H, d, device="cuda", dtype=torch.bfloat16)
    do = torch.randn(1, T, H, d, device="cuda", dtype=torch.bfloat16)
    k, v = (torch.randn(1, T, 1, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    o, lse = m.attn_fwd(q, k, v, window=w)
    g = m.attn_bwd(q, k, v, o, lse, do, window=w)
    heads = [0, 63]
    qt, dt = (t[0, -tail:, heads].double().cpu().numpy() for t in (q, do))
    kt, vt = (t[0, -tail:].double().cpu().numpy() for t in (k, v))
    r = A.attention(qt, kt, vt, True, w, do=dt)
    whole = slice(w, tail)  # queries whose window lies inside the tail
    err = np.abs(o[0, -tail:, heads].double().cpu().numpy() - r["o"])[whole]
    assert (err <= (U * np.abs(r["o"]) + (U + 1e-4) * r["o_abs"])[whole]).all()
    assert (np.abs(lse[0, heads, -tail:].double().cpu().numpy() - r["lse"])[:, whole] <= 3e-5).all()
    tol = U * np.abs(r["dq"]) + (U + 2e-4) * r["dq_abs"] + U * (r["dq_dd"] + 1.01 * r["dq_da"]) + 2.0 ** -17 * r["dq_dp"]
    err = np.abs(g["dq"][0, -tail:, heads].double().cpu().numpy() - r["dq"])
    assert (err <= tol)[whole].all()
    m.device_wait_status()


def test_cache_past_32_bit_offsets(m):
    """Pages behind the first 2^32 bytes of a cache."""
    Hk, page, d, num = 4, 128, 128, 66000
    assert num * Hk * page * d > 2 ** 32
    c = [torch.empty(num, Hk, page, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    c += [torch.ones(num, Hk, device="cuda") for _ in range(2)]
    table = np.array([[num - 1, 5], [num - 2, 65999 - 40]], np.int32)
    tb = torch.from_numpy(table).cuda()
    k, v, q = rnd(2, 150, Hk, d, seed=1), rnd(2, 150, Hk, d, seed=2), rnd(2, 8, d, seed=3)
    m.kv_append(k.cuda(), v.cuda(), *c, tb, torch.zeros(2, dtype=torch.int32, device="cuda"))
    o = m.attn_step(q.cuda(), *c, tb, torch.tensor([150, 140], dtype=torch.int32, device="cuda"))
    ids = np.unique(table)
    small = np.searchsorted(ids, table).astype(np.int32)
    part = [t.view(torch.uint8)[torch.from_numpy(ids).long().cuda()].cpu().numpy() for t in c[:2]]
    sc = [t[torch.from_numpy(ids).long().cuda()].cpu().numpy() for t in c[2:]]
    z = [np.zeros_like(p) for p in part]
    for i, x in enumerate((k, v)):
        w, s = A.kv_append(x.double().numpy(), z[i], np.ones_like(sc[i]), small, [0, 0], [150, 150])
        assert np.array_equal(s, sc[i])
        for b in range(2):
            assert np.array_equal(part[i][small[b, 0]], w[small[b, 0]])
            assert np.array_equal(part[i][small[b, 1], :, :22], w[small[b, 1], :, :22])
    want, size = A.attn_step(q.double().numpy(), *part, *sc, small, [150, 140])
    err = np.abs(o.double().cpu().numpy() - want)
    assert (err <= U * np.abs(want) + (2.0 ** -11 + 7e-5) * size).all()


def test_views_that_are_refused(m):
    q, k, v = (rnd(2, 1, 4, 64, seed=s).cuda() for s in (1, 2, 3))
    f, _ = m.rotary_frequencies(64)
    with pytest.raises(ValueError):
        m.attn_fwd(q[:1].expand(2, 1, 4, 64), k, v)       # one token for both sequences
    with pytest.raises(ValueError):
        m.rotary(q.transpose(2, 3).contiguous().transpose(2, 3), inv_freq=f)  # channels apart
    with pytest.raises(ValueError):
        m.rotary(q[:, :, ::2], inv_freq=f)                # heads apart
    x = rnd(2, 8, 4, 64, seed=4).cuda()
    with pytest.raises(ValueError):
        m.attn_fwd(x[:, :6], x, x)                        # tokens not evenly spaced over the batch
    with pytest.raises(TypeError):
        m.attn_fwd(q.float(), k, v)
    with pytest.raises(ValueError):
        m.attn_fwd(q, k[:1], v[:1])
    with pytest.raises(m.MuirError):
        m.attn_fwd(q[:, :, :3], k[:, :, :2].contiguous(), v[:, :, :2].contiguous())  # 3 heads over 2
    # evenly spaced tokens of every second row are taken as they lie
    y = rnd(1, 64, 4, 64, seed=5).cuda()
    o, lse = m.attn_fwd(y[:, ::2], y[:, 1::2], y[:, ::2])
    o2, lse2 = m.attn_fwd(y[:, ::2].contiguous(), y[:, 1::2].contiguous(), y[:, ::2].contiguous())
    assert torch.equal(o, o2) and torch.equal(lse, lse2)

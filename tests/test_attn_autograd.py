"""The autograd side of the softmax-attention layer.  On the CPU the wrappers run over plain
float64 stand-ins of the kernels' entry points, which shows what they record and pass on; on
the GPU, gradients of a projection through rotation and attention equal the chain of single
calls bit for bit, and the float64 chain within the bounds of those calls."""
import numpy as np
import pytest
import torch

from oracle import attention as A

U = 2.0 ** -8


@pytest.fixture(scope="module")
def m():
    from gated_delta_rule_115_b200 import build
    build.build()
    import gated_delta_rule_115_b200 as m
    m.lib()
    return m


def plain_rotary(q, k=None, positions=None, inv_freq=None, interleaved=False, mscale=1.0, inverse=False,
                 q_out=None, k_out=None):
    def turn(x, out):
        at = torch.arange(x.shape[1])[None] if positions is None else positions
        t = at.double()[..., None] * inv_freq * (-1 if inverse else 1)
        c, s, h = mscale * t.cos()[:, :, None], mscale * t.sin()[:, :, None], len(inv_freq)
        a, b = (x[..., 0:2 * h:2], x[..., 1:2 * h:2]) if interleaved else (x[..., :h], x[..., h:2 * h])
        ya, yb = a * c - b * s, b * c + a * s
        y = torch.stack((ya, yb), -1).flatten(-2) if interleaved else torch.cat((ya, yb), -1)
        y = torch.cat((y, x[..., 2 * h:]), -1)
        return y if out is None else out.copy_(y)
    return turn(q, q_out) if k is None else (turn(q, q_out), turn(k, k_out))


def rnd(*shape, seed, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64).to(dtype)


# ------------------------------------------------------------------ rotary, on the CPU


def test_rotary_refuses_what_it_would_cut_from_the_graph(m):
    q, k = (torch.zeros(1, 4, 2, 64) for _ in range(2))
    f, _ = m.rotary_frequencies(64, device="cpu")
    for over in (dict(q=q.clone().requires_grad_()), dict(k=k.clone().requires_grad_()),
                 dict(q_out=q.clone().requires_grad_()), dict(k_out=k.clone().requires_grad_())):
        a = dict(q=q, k=k, inv_freq=f)
        a.update(over)
        with pytest.raises(ValueError, match="MuirRotaryFunction"):
            m.rotary(**a)
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):  # past that check
            m.rotary(**a)


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("inter", [False, True])
def test_rotary_gradient(m, monkeypatch, inter, inplace):
    """Against torch's own gradient of the formula, for both outputs and for each alone; and
    the gradient's gradient."""
    monkeypatch.setattr(m, "rotary", plain_rotary)
    f = torch.tensor([1.0, 0.3, 0.01], dtype=torch.float64)
    pos = torch.tensor([[5, 6, 7, 100], [0, 1, 2, 3]], dtype=torch.int32)
    x = [rnd(2, 4, H, 8, seed=H, dtype=torch.float64) for H in (3, 2)]
    w = [rnd(2, 4, H, 8, seed=10 + H, dtype=torch.float64) for H in (3, 2)]
    for use in ((0, 1), (0,), (1,)):
        got, want = ([t.clone().requires_grad_() for t in x] for _ in range(2))
        y = m.MuirRotaryFunction.apply(*(t * 1 for t in got), pos, f, inter, 1.25, False, inplace)
        r = plain_rotary(*want, pos, f, inter, 1.25)
        assert all(torch.equal(a, b) for a, b in zip(y, r))
        for out, leaves in ((y, got), (r, want)):
            g = torch.autograd.grad(sum((out[i] * w[i]).sin().sum() for i in use), leaves, create_graph=True,
                                    allow_unused=True)
            sum((t ** 2).sum() for t in g if t is not None).backward()
        for i in range(2):
            assert (got[i].grad is not None) == (i in use)
            if i in use:
                assert torch.allclose(got[i].grad, want[i].grad, rtol=1e-12)
    one = x[0].clone().requires_grad_()
    z = m.MuirRotaryFunction.apply(one * 1, None, pos, f, inter, 1.25, True, inplace)
    z.sum().backward()  # an expanded gradient
    assert torch.allclose(one.grad, plain_rotary(torch.ones_like(one), None, pos, f, inter, 1.25))


def test_rotary_in_place_on_parts_of_a_projection(m, monkeypatch):
    """A call for each part; what autograd cannot follow is refused before it is written."""
    monkeypatch.setattr(m, "rotary", plain_rotary)
    f = torch.tensor([1.0, 0.1], dtype=torch.float64)
    leaf = rnd(1, 5, 12, seed=1, dtype=torch.float64).requires_grad_()
    x = leaf * 1
    q, k = x[..., :8].unflatten(-1, (2, 4)), x[..., 8:].unflatten(-1, (1, 4))
    old = x.detach().clone()
    for bad in ((q, k), (leaf.unflatten(-1, (3, 4)).detach().requires_grad_(), None)):
        with pytest.raises(ValueError):
            m.MuirRotaryFunction.apply(*bad, None, f, False, 1.0, False, True)
    assert torch.equal(x.detach(), old)
    for part in (q, k):
        m.MuirRotaryFunction.apply(part, None, None, f, False, 1.0, False, True)
    (x ** 2 * torch.arange(12.0, dtype=torch.float64)).sum().backward()
    want = leaf.detach().clone().requires_grad_()
    y = torch.cat([plain_rotary(want[..., a:b].unflatten(-1, (-1, 4)), inv_freq=f).flatten(2) for a, b in ((0, 8), (8, 12))], -1)
    (y ** 2 * torch.arange(12.0, dtype=torch.float64)).sum().backward()
    assert torch.allclose(leaf.grad, want.grad, rtol=1e-12)


# ------------------------------------------------------------------ attention, on the CPU


def plain_attention(q, k, v, causal, window, scale, cu=None, cu_k=None):
    """Float64 attention of packed (or dense) sequences, in torch."""
    cu = [0, q.shape[1]] if cu is None else [int(x) for x in cu]
    cu_k = ([0, k.shape[1]] if cu == [0, q.shape[1]] else cu) if cu_k is None else [int(x) for x in cu_k]
    o = []
    for a, b, c, d in zip(cu, cu[1:], cu_k, cu_k[1:]):
        see = torch.tensor(A.visible(b - a, d - c, causal, window))
        kk, vv = (t[:, c:d].repeat_interleave(q.shape[2] // k.shape[2], 2) for t in (k, v))
        z = torch.einsum("bihd,bjhd->bhij", q[:, a:b], kk) * (q.shape[-1] ** -0.5 if scale is None else scale)
        p = torch.softmax(z.masked_fill(~see, -1e300), -1) * see.any(1)[:, None]
        o.append(torch.einsum("bhij,bjhd->bihd", p, vv))
    return torch.cat(o, 1)


@pytest.fixture
def plain(m, monkeypatch):
    """The module with its attention calls replaced by float64 formulas on the CPU."""
    def fwd(q, k, v, cu=None, cu_k=None, causal=True, window=0, scale=None):
        return plain_attention(q, k, v, causal, window, scale, cu, cu_k), torch.zeros(1)

    def bwd(q, k, v, o, lse, dO, cu=None, cu_k=None, causal=True, window=0, scale=None, ws=None):
        with torch.enable_grad():
            x = [t.detach().double().requires_grad_() for t in (q, k, v)]
            g = torch.autograd.grad(plain_attention(*x, causal, window, scale, cu, cu_k), x, dO.double())
        return dict(zip(("dq", "dk", "dv"), (t.detach() for t in g)))

    monkeypatch.setattr(m, "attn_fwd", lambda q, k, v, **kw: fwd(q, k, v, **kw))
    monkeypatch.setattr(m, "attn_bwd", lambda q, k, v, o, lse, dO, **kw: bwd(q, k, v, o, lse, dO, **kw))
    monkeypatch.setattr(m, "attn_fwd_varlen", lambda q, k, v, cu_seqlens, cu_seqlens_k=None, **kw:
                        fwd(q, k, v, cu_seqlens, cu_seqlens_k, **kw))
    monkeypatch.setattr(m, "attn_bwd_varlen", lambda q, k, v, o, lse, dO, cu_seqlens, cu_seqlens_k=None, **kw:
                        bwd(q, k, v, o, lse, dO, cu_seqlens, cu_seqlens_k, **kw))
    return m


@pytest.mark.parametrize("kind", [list, torch.tensor, np.array])
@pytest.mark.parametrize("apart", [False, True])
def test_offsets_refilled_before_the_backward_pass(plain, kind, apart):
    """The gradients belong to the sequences of the forward pass, whatever the caller's
    buffer of offsets holds by then.  (The wrapper rounds dO to bfloat16: ones are exact.)"""
    q, k, v = (rnd(1, 12, H, 8, seed=H, dtype=torch.float64) for H in (4, 2, 2))
    cu, ck = [0, 5, 12], [0, 9, 12]
    held, held_k = kind(cu), kind(ck)
    got, want = ([t.clone().requires_grad_() for t in (q, k, v)] for _ in range(2))
    o = plain.MuirAttentionFunction.apply(*got, True, 0, None, held, held_k if apart else None)
    held[1], held_k[1] = 7, 2
    o.sum().backward()
    plain_attention(*want, True, 0, None, cu, ck if apart else None).sum().backward()
    for a, b in zip(got, want):
        assert torch.allclose(a.grad, b.grad, rtol=1e-12, atol=1e-13)


def chunk_stand_in(m, monkeypatch):
    """MuirChunkFunction over a formula that is quadratic in q (its second gradient is not 0)."""
    def fwd(q, k, v, g, e, w, gamma, S0=None, **kw):
        return q * q * v, torch.zeros(1), None, None, None

    def bwd(q, k, v, g, e, w, gamma, S0, dO, dS, **kw):
        z = torch.zeros_like(q)
        return dict(dq=2 * q * v * dO, dk=z, dv=q * q * dO, dg=z, de=z, dw=z, dgamma=z, dS0=None)

    monkeypatch.setattr(m, "chunk_fwd", fwd)
    monkeypatch.setattr(m, "chunk_bwd", bwd)


@pytest.mark.parametrize("which", ["attention", "chunk"])
def test_gradients_of_gradients_are_refused(plain, monkeypatch, which):
    """The backward passes have no derivative of their own: a gradient penalty has to fail
    where it is taken, not vanish.  The first gradient with create_graph stays as it was."""
    x = [rnd(1, 6, 2, 8, seed=s, dtype=torch.float64).requires_grad_() for s in range(7)]
    if which == "attention":
        o = plain.MuirAttentionFunction.apply(*x[:3])
        want = torch.autograd.grad(plain_attention(*x[:3], True, 0, None).sum(), x[0])
    else:
        chunk_stand_in(plain, monkeypatch)
        o, _ = plain.MuirChunkFunction.apply(*x, None, 64)
        want = (2 * x[0] * x[2],)
    # the loss holds q by another path as well, which a silently dropped part would leave
    loss = o.sum() + (x[0] ** 2).sum()
    got = torch.autograd.grad(loss, x[0], create_graph=True)
    assert torch.allclose(got[0], want[0] + 2 * x[0], rtol=1e-12)
    with pytest.raises(RuntimeError, match="differentiated again"):
        (got[0] ** 2).sum().backward()


def test_key_offsets_alone_are_refused(m):
    """Packed rows must not run as one dense sequence."""
    q, lse = torch.zeros(1, 6, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 2, 6)
    ck = [0, 2, 6]
    for call in (lambda: m.attn_fwd_varlen(q, q, q, None), lambda: m.attn_fwd_varlen(q, q, q, None, ck),
                 lambda: m.attn_bwd_varlen(q, q, q, q, lse, q, None), lambda: m.attn_bwd_varlen(q, q, q, q, lse, q, None, ck),
                 lambda: m.MuirAttentionFunction.apply(q, q, q, True, 0, None, None, ck)):
        with pytest.raises(ValueError, match="cu_seqlens"):
            call()


# ------------------------------------------------------------------ on the GPU


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["new", "in place", "together in place"])
def test_projection_through_rotation_and_attention(m, how):
    """The gradient of a projection's rows through rotary and attention.  Bit for bit the
    chain of single calls; and against float64 as in that chain's own test: rotated q and k
    are rounded in between, so the oracle's attention takes the rounded ones; the attention's
    own bounds pass the transposed rotation as sqrt(2) mscale of the pair's larger one, and the
    rotated gradient is rounded once more, u |y|."""
    T, Hq, Hk, d = 300, 4, 2, 64
    x0, do = rnd(1, T, (Hq + 2 * Hk) * d, seed=1).cuda(), rnd(1, T, Hq, d, seed=2).cuda()
    f, s = m.rotary_frequencies(32, scaling="yarn", factor=4.0)

    def parts(x):
        return [x[..., a * d: b * d].unflatten(-1, (b - a, d)) for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk))]

    leaf = x0.clone().requires_grad_()
    q, k, v = parts(leaf * 1)
    if how == "new":
        qr, kr = m.MuirRotaryFunction.apply(q, k, None, f, False, s)
    elif how == "in place":
        qr, kr = (m.MuirRotaryFunction.apply(t, None, None, f, False, s, False, True) for t in (q, k))
        assert qr.data_ptr() == q.data_ptr()
    else:
        q, k = q.clone(memory_format=torch.contiguous_format), k.clone(memory_format=torch.contiguous_format)
        qr, kr = m.MuirRotaryFunction.apply(q, k, None, f, False, s, False, True)
        assert qr is q and kr is k
    m.MuirAttentionFunction.apply(qr, kr, v).backward(do)
    got = parts(leaf.grad)

    q0, k0, v0 = (t.contiguous() for t in parts(x0))
    qr0, kr0 = m.rotary(q0, k0, inv_freq=f, mscale=s)
    assert torch.equal(qr.detach(), qr0) and torch.equal(kr.detach(), kr0)
    g = m.attn_bwd(qr0, kr0, v0, *m.attn_fwd(qr0, kr0, v0), do)
    dq, dk = m.rotary(g["dq"], g["dk"], inv_freq=f, mscale=s, inverse=True)
    assert all(torch.equal(a, b) for a, b in zip(got, (dq, dk, g["dv"])))

    r = A.attention(*(t[0].double().cpu().numpy() for t in (qr0, kr0, v0)), do=do[0].double().cpu().numpy())
    for n, t in zip(("dq", "dk"), got):
        tol = U * np.abs(r[n]) + (U + 2e-4) * r[n + "_abs"] + U * (r[n + "_dd"] + 1.01 * r[n + "_da"]) + 2.0 ** -17 * r[n + "_dp"]
        want = A.rotary(r[n][None], np.arange(T)[None], f.cpu().numpy(), mscale=s, inverse=True)[0]
        tol[..., :16] = tol[..., 16:32] = np.sqrt(2) * s * np.maximum(tol[..., :16], tol[..., 16:32])
        err = np.abs(t[0].double().cpu().numpy() - want)
        assert (err <= tol + U * (np.abs(want) + tol) + 1e-6).all(), n
    m.device_wait_status()


@pytest.mark.gpu
def test_rotary_in_place_is_seen_by_saved_tensors(m):
    """A tensor that autograd saved and rotary then overwrites: backward says so."""
    f, _ = m.rotary_frequencies(64)
    w = torch.ones(1, 8, 2, 64, device="cuda", requires_grad=True)
    x = torch.randn(1, 8, 2, 64, device="cuda")
    y = (w * x).sum()
    m.rotary(x, inv_freq=f, q_out=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():  # tensors without a version are written all the same
        z = torch.randn(1, 8, 2, 64, device="cuda")
        want = m.rotary(z, inv_freq=f)
        m.rotary(z, inv_freq=f, q_out=z)
        assert torch.equal(z, want)


@pytest.mark.gpu
def test_offsets_refilled_before_the_backward_pass_of_the_kernels(m):
    q, k, v, do = (rnd(1, 400, H, 64, seed=s).cuda() for H, s in ((4, 1), (2, 2), (2, 3), (4, 4)))
    cu = torch.tensor([0, 130, 400])
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    o = m.MuirAttentionFunction.apply(*leaves, True, 0, None, cu)
    cu[1] = 255
    o.backward(do)
    g = m.attn_bwd_varlen(q, k, v, *m.attn_fwd_varlen(q, k, v, [0, 130, 400]), do, [0, 130, 400])
    assert all(torch.equal(t.grad, g[n]) for t, n in zip(leaves, ("dq", "dk", "dv")))
    m.device_wait_status()


@pytest.mark.gpu
def test_gradients_with_create_graph(m):
    """The same gradients as without, and no second ones."""
    q, k, v = (rnd(1, 130, H, 64, seed=s).cuda().requires_grad_() for H, s in ((4, 1), (2, 2), (2, 3)))
    first = torch.autograd.grad(m.MuirAttentionFunction.apply(q, k, v).float().sum(), (q, k, v))
    again = torch.autograd.grad(m.MuirAttentionFunction.apply(q, k, v).float().sum(), (q, k, v), create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    with pytest.raises(RuntimeError, match="differentiated again"):
        sum((t.float() ** 2).sum() for t in again).backward()


@pytest.mark.gpu
@pytest.mark.parametrize("state", [False, True])
def test_chunk_gradients_with_create_graph(m, state):
    from gated_delta_rule_115_b200.inputs import chunk_inputs
    x = chunk_inputs(0, B=1, H=2, T=150)
    x = [None if t is None else t.cuda() for t in (x[n] for n in ("q", "k", "v", "g", "e", "w", "gamma", "S0"))]
    x[7] = torch.randn(1, 2, *x[0].shape[-1:], x[2].shape[-1], device="cuda") if state else None
    leaves = [t.requires_grad_() for t in x if t is not None]
    got = [torch.autograd.grad(m.MuirChunkFunction.apply(*x, 64)[0].float().sum(), leaves, create_graph=c)
           for c in (False, True)]
    assert all(torch.equal(a, b) for a, b in zip(*got))
    with pytest.raises(RuntimeError, match="differentiated again"):
        sum((t.float() ** 2).sum() for t in got[1]).backward()
    m.device_wait_status()


@pytest.mark.gpu
def test_captured_training_pass(m):
    """Rotation, attention and both backward passes in one graph, replayed on new values."""
    T, Hq, Hk, d = 200, 4, 2, 64
    f, s = m.rotary_frequencies(d)
    x = rnd(1, T, (Hq + 2 * Hk) * d, seed=1).cuda().requires_grad_()
    do = rnd(1, T, Hq, d, seed=2).cuda()

    def one():
        p = x * 1
        q, k, v = (p[..., a * d: b * d].unflatten(-1, (b - a, d)) for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)))
        q, k = (m.MuirRotaryFunction.apply(t, None, None, f, False, s, False, True) for t in (q, k))
        return torch.autograd.grad(m.MuirAttentionFunction.apply(q, k, v, True, 70, None, [0, 77, T]), x, do)[0]

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        one()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = one()
    for seed in (3, 4):
        with torch.no_grad():
            x.copy_(rnd(*x.shape, seed=seed))
            do.copy_(rnd(*do.shape, seed=seed + 10))
        graph.replay()
        assert torch.equal(got, one())
    m.device_wait_status()


@pytest.mark.gpu
@pytest.mark.parametrize("B,Tq,Tk", [(0, 5, 5), (2, 0, 7), (2, 7, 0), (1, 0, 0), (3, 1, 1)])
def test_gradients_of_empty_calls(m, B, Tq, Tk):
    """No sequences, no queries, no keys: shapes kept, zeros where nothing is seen."""
    q, k, v = (rnd(B, T, H, 64, seed=T + H).cuda().requires_grad_() for T, H in ((Tq, 4), (Tk, 2), (Tk, 2)))
    f, _ = m.rotary_frequencies(64)
    qr, kr = m.MuirRotaryFunction.apply(q, None, None, f), m.MuirRotaryFunction.apply(k, None, None, f)
    o = m.MuirAttentionFunction.apply(qr, kr, v)
    o.sum().backward()
    assert [t.grad.shape for t in (q, k, v)] == [t.shape for t in (q, k, v)] and o.shape == q.shape
    if Tq != 1:
        assert not o.any() and not any(t.grad.any() for t in (q, k, v))
    else:
        assert torch.equal(o, v.repeat_interleave(2, 2)) and not q.grad.any() and not k.grad.any()
        assert (v.grad == 2).all()
    m.device_wait_status()

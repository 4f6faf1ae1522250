"""Host-side checks of the softmax-attention entry points (no GPU needed): documented
refusals before anything is enqueued, workspace sizes, the binding's own checks, the
frequency tables of the rotary positions."""
import ctypes
import math

import pytest
import torch

FAKE = 0x10000  # 16-byte aligned, never dereferenced: checks fail first
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def m():
    from gated_delta_rule_115_b200 import build
    build.build()
    import gated_delta_rule_115_b200 as m
    m.lib()
    return m


def rotary(m, **over):
    a = dict(B=1, T=4, Hq=2, Hk=2, d=64, rot=64, dtype=0, q=FAKE, q_ld=0, k=FAKE, k_ld=0, positions=FAKE,
             inv_freq=FAKE, mscale=1.0, inter=0, inverse=0, q_out=FAKE + 4096, qo_ld=0, k_out=FAKE + 8192,
             ko_ld=0, stream=None)
    a.update(over)
    return m.lib().muir_rotary(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(B=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hk=-1), INVALID), (dict(dtype=5), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(rot=8), UNSUPPORTED), (dict(rot=80), UNSUPPORTED),
    (dict(rot=40), UNSUPPORTED), (dict(B=1 << 20, T=1 << 20), UNSUPPORTED), (dict(q=None), INVALID),
    (dict(q=FAKE + 8), INVALID), (dict(k=None), INVALID), (dict(k_out=None), INVALID),
    (dict(Hk=0), INVALID), (dict(inv_freq=None), INVALID), (dict(inv_freq=FAKE + 4), INVALID),
    (dict(positions=FAKE + 2), INVALID), (dict(q_ld=64), INVALID), (dict(q_ld=132), INVALID),
    (dict(qo_ld=100), INVALID), (dict(mscale=math.inf), INVALID), (dict(mscale=math.nan), INVALID),
    (dict(q_out=FAKE, qo_ld=256), INVALID)])
def test_rotary_refusals(m, over, code):
    assert rotary(m, **over) == code


def test_rotary_of_nothing(m):
    assert rotary(m, T=0) == 0 and rotary(m, B=0, q=None, k=None) == 0


def cache(m, **over):
    a = dict(Hk=2, d=64, page=64, num_pages=8, max_pages=4, k_pages=FAKE, v_pages=FAKE, k_scale=FAKE,
             v_scale=FAKE, table=FAKE)
    a.update(over)
    return m.MuirKvCache(*a.values())


def append(m, c, **over):
    a = dict(B=2, T=3, dtype=0, k=FAKE, k_ld=0, v=FAKE, v_ld=0, c=c, start=FAKE, count=None, stream=None)
    a.update(over)
    a["c"] = None if a["c"] is None else ctypes.byref(a["c"])
    return m.lib().muir_kv_append(*a.values())


def step(m, c, **over):
    a = dict(B=2, Hq=4, c=c, q=FAKE, lens=FAKE, scale=0.125, window=0, o=FAKE, ws=FAKE, ws_bytes=1 << 30,
             stream=None)
    a.update(over)
    a["c"] = None if a["c"] is None else ctypes.byref(a["c"])
    return m.lib().muir_attn_step(*a.values())


BAD_CACHES = [(dict(Hk=0), INVALID), (dict(num_pages=0), INVALID), (dict(max_pages=0), INVALID),
              (dict(d=96), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(page=256), UNSUPPORTED),
              (dict(num_pages=1 << 30, Hk=4), UNSUPPORTED), (dict(max_pages=1 << 26), UNSUPPORTED),
              (dict(k_pages=None), INVALID), (dict(v_pages=FAKE + 8), INVALID), (dict(k_scale=None), INVALID),
              (dict(v_scale=FAKE + 2), INVALID), (dict(table=None), INVALID), (dict(table=FAKE + 1), INVALID)]


@pytest.mark.parametrize("over,code", BAD_CACHES)
def test_cache_refusals(m, over, code):
    assert append(m, cache(m, **over)) == code
    assert step(m, cache(m, **over)) == code
    assert m.lib().muir_attn_step_workspace(2, 4, ctypes.byref(cache(m, **over))) == 0


@pytest.mark.parametrize("over,code", [
    (dict(c=None), INVALID), (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(dtype=3), INVALID),
    (dict(k=None), INVALID), (dict(v=FAKE + 4), INVALID), (dict(start=None), INVALID),
    (dict(start=FAKE + 1), INVALID), (dict(count=FAKE + 2), INVALID), (dict(k_ld=64), INVALID),
    (dict(v_ld=129), INVALID), (dict(B=40000), UNSUPPORTED)])
def test_append_refusals(m, over, code):
    a = dict(over)
    c = a.pop("c", cache(m))
    assert append(m, c, **a) == code


@pytest.mark.parametrize("over,code", [
    (dict(c=None), INVALID), (dict(B=0), INVALID), (dict(Hq=3), INVALID), (dict(Hq=0), INVALID),
    (dict(q=None), INVALID), (dict(o=FAKE + 2), INVALID), (dict(lens=None), INVALID),
    (dict(scale=math.nan), INVALID), (dict(window=-1), INVALID), (dict(B=70000), UNSUPPORTED)])
def test_step_refusals(m, over, code):
    a = dict(over)
    c = a.pop("c", cache(m))
    assert step(m, c, **a) == code


def test_step_workspace(m):
    c = cache(m, max_pages=1024)
    need = m.lib().muir_attn_step_workspace(2, 4, ctypes.byref(c))
    assert need > 0
    assert step(m, c, ws_bytes=need - 1) == WORKSPACE and step(m, c, ws=None) == WORKSPACE
    # a cache of one split needs none
    assert m.lib().muir_attn_step_workspace(2, 4, ctypes.byref(cache(m, max_pages=1))) == 0


def test_append_of_nothing(m):
    assert append(m, cache(m), T=0, k=None, v=None) == 0 and append(m, cache(m), B=0) == 0


def test_binding_refuses_cpu_and_mismatched_tensors(m):
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    f, _ = m.rotary_frequencies(64, device="cpu")
    with pytest.raises(ValueError):
        m.rotary(q, inv_freq=f)
    with pytest.raises(ValueError):
        m.rotary(q)
    with pytest.raises(TypeError):
        m.rotary(q.half(), inv_freq=f)
    with pytest.raises(ValueError):
        m.rotary(q, q[:, :2], inv_freq=f)
    kp, vp, ks, vs = m.kv_cache(3, 2, 16, 64, device="cpu")
    assert kp.dtype == torch.float8_e4m3fn and tuple(vs.shape) == (3, 2)
    with pytest.raises(ValueError):
        m.attn_step(q[:, 0], kp, vp, ks, vs, torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


def test_frequencies(m):
    f, s = m.rotary_frequencies(64, device="cpu")
    assert s == 1.0 and f.dtype == torch.float64 and f[0] == 1.0
    assert math.isclose(f[16], 10000.0 ** -0.5, rel_tol=1e-15)
    lin, _ = m.rotary_frequencies(64, scaling="linear", factor=8.0, device="cpu")
    assert torch.allclose(lin * 8, f)
    ntk, _ = m.rotary_frequencies(64, scaling="ntk", factor=8.0, device="cpu")
    assert ntk[0] == 1.0 and math.isclose(ntk[-1] * 8, f[-1], rel_tol=1e-12)
    y, s = m.rotary_frequencies(64, scaling="yarn", factor=8.0, original_length=4096, device="cpu")
    assert math.isclose(s, 0.1 * math.log(8.0) + 1.0)
    assert torch.equal(y[:8], f[:8]) and torch.allclose(y[-4:] * 8, f[-4:])
    assert (y <= f).all() and (y * 8 >= f * (1 - 1e-12)).all()
    for bad in (dict(rot=63), dict(rot=64, scaling="x"), dict(rot=64, base=1.0), dict(rot=64, factor=0.0)):
        with pytest.raises(ValueError):
            m.rotary_frequencies(device="cpu", **bad)


def attn(m, backward=False, **over):
    s = dict(B=1, Tq=8, Tk=8, Hq=4, Hk=2, d=64, causal=1, window=0, scale=0.125, q_ld=0, k_ld=0, v_ld=0)
    a = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE)
    if backward:
        a.update(dO=FAKE, dq=FAKE, dk=FAKE, dv=FAKE, ws=FAKE, ws_bytes=1 << 30)
    for n, x in over.items():
        (s if n in s else a)[n] = x
    shape = m.MuirAttnShape(*s.values())
    fn = m.lib().muir_attn_bwd if backward else m.lib().muir_attn_fwd
    return fn(ctypes.byref(shape), *a.values(), None)


@pytest.mark.parametrize("over,code", [
    (dict(B=-1), INVALID), (dict(Tq=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hq=3), INVALID),
    (dict(window=-1), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(d=256), UNSUPPORTED), (dict(q_ld=64), INVALID), (dict(k_ld=132), INVALID), (dict(v_ld=-128), INVALID),
    (dict(B=1 << 16, Tq=1 << 16), UNSUPPORTED), (dict(Tk=1 << 30), UNSUPPORTED), (dict(B=1 << 20, Tq=1, Hq=1 << 16, Hk=1), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(k=FAKE + 8), INVALID), (dict(v=None), INVALID), (dict(o=None), INVALID),
    (dict(lse=None), INVALID), (dict(lse=FAKE + 2), INVALID)])
def test_attention_refusals(m, over, code):
    assert attn(m, **over) == code
    assert attn(m, True, **over) == code


@pytest.mark.parametrize("over,code", [
    (dict(dO=None), INVALID), (dict(dq=FAKE + 4), INVALID), (dict(dk=None), INVALID), (dict(dv=None), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=8 * 4 * 8 - 1), WORKSPACE)])
def test_attention_backward_refusals(m, over, code):
    assert attn(m, True, **over) == code


@pytest.mark.parametrize("cu,ck,over,code", [
    ([0, 8], None, dict(B=2), INVALID), ([1, 8], None, {}, INVALID), ([0, 7], None, {}, INVALID),
    ([0, 5, 4, 8], None, {}, INVALID), ([0, 4, 8], [0, 9, 8], {}, INVALID), ([0, 8], None, dict(Tk=9), INVALID),
    ([0, 8], [0, 8], dict(Tk=9), INVALID), (None, None, {}, INVALID), ([0], None, dict(n=0), INVALID)])
def test_attention_varlen_refusals(m, cu, ck, over, code):
    s = dict(B=1, Tq=8, Tk=8, Hq=4, Hk=2, d=64, causal=1, window=0, scale=0.125, q_ld=0, k_ld=0, v_ld=0)
    n = over.pop("n", len(cu or [0, 0]) - 1)
    s.update(over)
    shape = m.MuirAttnShape(*s.values())
    arr = lambda x: None if x is None else (ctypes.c_longlong * len(x))(*x)  # noqa: E731
    for fn, rest in ((m.lib().muir_attn_fwd_varlen, [FAKE] * 5 + [None]),
                     (m.lib().muir_attn_bwd_varlen, [FAKE] * 10 + [1 << 30, None])):
        assert fn(ctypes.byref(shape), n, arr(cu), arr(ck), *rest) == code


def test_attention_workspace(m):
    s = m.MuirAttnShape(2, 100, 50, 4, 2, 64, 1, 0, 0.125, 0, 0, 0)
    assert m.lib().muir_attn_bwd_workspace(ctypes.byref(s)) == 2 * 100 * 4 * 8
    s.d = 32
    assert m.lib().muir_attn_bwd_workspace(ctypes.byref(s)) == 0


def test_scales_that_leave_float32_in_base_two(m):
    """The kernels take scale log2(e): past 2.35e38 that is no float32 any more."""
    assert attn(m, scale=2.4e38) == attn(m, True, scale=2.4e38) == INVALID
    assert step(m, cache(m), scale=2.4e38) == step(m, cache(m), scale=-2.4e38) == INVALID


@pytest.mark.parametrize("d,Hq,Hk,resident", [(128, 16, 4, 296), (64, 16, 4, 296), (64, 16, 1, 296), (128, 16, 1, 148),
                                              (128, 64, 4, 148)])
@pytest.mark.parametrize("B", [1, 2, 8])
def test_step_splits_fill_one_round(m, B, d, Hq, Hk, resident):
    """Sequences are split into as many blocks as the kernel has resident on 148 SMs (two each;
    one with 16 heads of 128 channels a block), as long as that leaves 256 tokens or more."""
    tokens = 16384
    c = cache(m, Hk=Hk, d=d, page=64, max_pages=tokens // 64)
    splits = m.lib().muir_attn_step_workspace(B, Hq, ctypes.byref(c)) // (B * Hq * (d + 1) * 4)
    units = B * Hk * -(-Hq // Hk // 16)
    assert splits == max(tokens // 2048, min(resident // units, tokens // 256))

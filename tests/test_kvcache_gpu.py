"""The paged 8-bit cache on the GPU: appended codes and scales equal the oracle's bit for
bit; the single-token step matches float64 attention over the cached values.

Tolerance of the step, per element: the value codes' weights are rounded to fp16 (half a
step, 2^-11) and the output to bfloat16 (2^-8); scores are float32 sums of exact fp16
products, with |score terms| summing below 64 in these inputs: 64 2^-20 = 6e-5 on a
weight, and 1e-5 covers the exponentials: 2^-8 |o| + (2^-11 + 7e-5) sum_j p_j |v_j|."""
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


def table_for(B, pages, spare, seed):
    order = np.random.default_rng(seed).permutation(B * pages + spare)[: B * pages]
    return order.reshape(B, pages).astype(np.int32)


def codes(t):
    return t.view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page,d,Hk", [(16, 64, 1), (64, 128, 2), (32, 64, 3), (128, 128, 1)])
def test_append_in_pieces(m, page, d, Hk, dtype):
    """Prompts, single tokens, nothing, page borders inside and between calls; magnitudes
    that grow, shrink, vanish and end in infinities and NaN."""
    B, pages = 3, 5
    table = table_for(B, pages, 2, page)
    c = m.kv_cache(B * pages + 2, Hk, page, d)
    for t in c[:2]:
        t.view(torch.uint8).fill_(0x7f)  # stale slots: NaN codes
    for t in c[2:]:
        t.fill_(1e30)                    # stale scales
    want = [(codes(x).copy(), s.cpu().numpy().astype(np.float64)) for x, s in ((c[0], c[2]), (c[1], c[3]))]
    tb = torch.from_numpy(table).cuda()
    g = torch.Generator().manual_seed(page)
    start = np.array([0, page - 1, 2 * page + 3])
    for T, gain in ((1, 1.0), (page + 5, 30.0), (1, 1e-3), (3, 0.0), (1, 1e4), (2, 1e-30), (7, 1e20)):
        x = [(torch.randn(B, T, Hk, d, generator=g) * gain).to(dtype) for _ in range(2)]
        if gain == 1e4:
            x[0][0, 0, 0, :3] = torch.tensor([float("inf"), -float("inf"), float("nan")])
        count = np.array([T, max(T - 1, 0), T])
        m.kv_append(x[0].cuda(), x[1].cuda(), *c, tb, torch.from_numpy(start.astype(np.int32)).cuda(),
                    torch.from_numpy(count.astype(np.int32)).cuda())
        for i in range(2):
            want[i] = A.kv_append(x[i].double().numpy(), *want[i], table, start, count)
            assert np.array_equal(c[2 + i].cpu().numpy(), want[i][1]), (T, gain)
            got = codes(c[i])
            nan = (want[i][0] & 0x7f) == 0x7f
            assert np.array_equal(got[~nan], want[i][0][~nan]) and ((got[nan] & 0x7f) == 0x7f).all(), (T, gain)
        start = start + count


def test_append_strides_bounds_and_bad_pages(m):
    """Parts of a packed projection; a table too short for the tokens, page ids that name
    no page, a negative start and counts out of range: nothing is written for those."""
    B, T, Hk, d, page = 5, 40, 2, 64, 16
    x = torch.randn(B, T, 3 * Hk * d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    k = x[..., Hk * d: 2 * Hk * d].unflatten(-1, (Hk, d))
    v = x[..., 2 * Hk * d:].unflatten(-1, (Hk, d))
    xd = x.cuda()
    table = table_for(B, 3, 4, 2)
    table[1, 1], table[2, 0] = 99, -1
    start = np.array([20, 0, 0, -3, 1])
    count = np.array([40, 40, 40, 40, 1000])
    c = m.kv_cache(19, Hk, page, d)
    want = [(codes(t).copy(), s.cpu().numpy().astype(np.float64)) for t, s in ((c[0], c[2]), (c[1], c[3]))]
    m.kv_append(xd[..., Hk * d: 2 * Hk * d].unflatten(-1, (Hk, d)), xd[..., 2 * Hk * d:].unflatten(-1, (Hk, d)),
                *c, torch.from_numpy(table).cuda(), torch.from_numpy(start.astype(np.int32)).cuda(),
                torch.from_numpy(count.astype(np.int32)).cuda())
    for i, t in enumerate((k, v)):
        w = A.kv_append(t.double().numpy(), *want[i], table, start, count)
        assert np.array_equal(codes(c[i]), w[0]) and np.array_equal(c[2 + i].cpu().numpy(), w[1])


def filled(B, most, Hk, d, page, seed, wide=False, tail_nan=True):
    """A cache with random codes; slots behind each sequence hold NaN codes."""
    r = np.random.default_rng(seed)
    pages = max(1, -(-most // page))
    table = table_for(B, pages, 3, seed)
    num = B * pages + 3
    code = [A.e4m3_encode(r.standard_normal((num, Hk, page, d)) * 64) for _ in range(2)]
    low, high = (-30, 20) if wide else (-8, -4)
    ks = 2.0 ** r.integers(-8, -5, (num, Hk))
    vs = 2.0 ** r.integers(low, high, (num, Hk))
    lens = r.integers(0, most + 1, B)
    lens[0] = most
    if B > 2:
        lens[1], lens[2] = 0, 1
    if tail_nan:
        for b in range(B):
            for s in range(pages):
                keep = int(np.clip(lens[b] - s * page, 0, page))
                for x in code:
                    x[table[b, s], :, keep:] = 0x7f
    return code, (ks, vs), table, lens


def step(m, q, code, scales, table, lens, **kw):
    f8 = [torch.from_numpy(x).cuda().view(torch.float8_e4m3fn) for x in code]
    sc = [torch.from_numpy(s.astype(np.float32)).cuda() for s in scales]
    return m.attn_step(q.cuda(), *f8, *sc, torch.from_numpy(table).cuda(),
                       torch.from_numpy(lens.astype(np.int32)).cuda(), **kw)


def check(o, q, code, scales, table, lens, **kw):
    want, size = A.attn_step(q.double().numpy(), *code, *scales, table, lens, **kw)
    err = np.abs(o.double().cpu().numpy() - want)
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 7e-5) * size
    assert (err <= tol).all(), float((err - tol).max())


@pytest.mark.parametrize("B,most,Hq,Hk,d,page,window", [
    (1, 1, 1, 1, 64, 16, 0), (4, 15, 2, 2, 128, 16, 0), (4, 300, 4, 1, 128, 16, 0), (3, 700, 16, 4, 128, 64, 0),
    (4, 64, 8, 1, 64, 32, 0), (3, 1000, 6, 2, 64, 128, 37), (4, 500, 20, 1, 128, 64, 0), (2, 513, 33, 1, 64, 64, 1),
    (1, 9000, 2, 1, 128, 128, 0), (2, 5000, 4, 2, 64, 32, 3333), (5, 257, 3, 3, 128, 64, 64)])
def test_step_parity(m, B, most, Hq, Hk, d, page, window):
    code, scales, table, lens = filled(B, most, Hk, d, page, most + d)
    q = torch.randn(B, Hq, d, generator=torch.Generator().manual_seed(most)).to(torch.bfloat16)
    o = step(m, q, code, scales, table, lens, window=window)
    check(o, q, code, scales, table, lens, window=window)
    assert torch.equal(o, step(m, q, code, scales, table, lens, window=window))
    m.device_wait_status()


def test_step_wide_scales_and_small_weights(m):
    """Pages whose value scales differ by 2^50, and queries of very different size."""
    code, scales, table, lens = filled(3, 400, 2, 128, 16, 5, wide=True)
    q = torch.randn(3, 8, 128, generator=torch.Generator().manual_seed(3))
    q = (q * torch.tensor([1.0, 1e-30, 0.0, 3.0, 1e-3, 1.0, 1e-10, 2.0])[None, :, None]).to(torch.bfloat16)
    check(step(m, q, code, scales, table, lens), q, code, scales, table, lens)


def test_step_bad_pages_and_lengths(m):
    """Ids that name no page hide their tokens; lengths are clamped to the table."""
    code, scales, table, lens = filled(4, 200, 2, 64, 32, 9, tail_nan=False)
    table[0, 2], table[0, 6], table[3, :] = -1, 1 << 20, -7
    lens = np.array([200, 100000, -5, 50])
    q = torch.randn(4, 4, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    o = step(m, q, code, scales, table, lens)
    check(o, q, code, scales, table, lens)
    assert not o[2].any() and not o[3].any()


def test_step_nan_reaches_its_sequence_only(m):
    code, scales, table, lens = filled(3, 100, 1, 64, 16, 4)
    lens[:] = 90
    for x in code:
        x[x & 0x7f == 0x7f] = 0x30
    code[1][table[1, 2], 0, 3, 5] = 0x7f
    q = torch.randn(3, 2, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    o = step(m, q, code, scales, table, lens).float()
    assert torch.isnan(o[1, :, 5]).all() and int(torch.isnan(o).sum()) == 2


def test_step_in_a_graph_follows_lengths_and_cache(m):
    """One captured pass of append and step, replayed as the sequences grow."""
    B, Hk, Hq, d, page = 2, 2, 4, 128, 16
    table = table_for(B, 8, 0, 1)
    c = m.kv_cache(16, Hk, page, d)
    tb = torch.from_numpy(table).cuda()
    start, lens = (torch.tensor([14, 0], dtype=torch.int32, device="cuda") + i for i in (0, 1))
    g = torch.Generator().manual_seed(2)
    k0, v0 = (torch.randn(B, 14, Hk, d, generator=g).to(torch.bfloat16) for _ in range(2))
    first = [(codes(t).copy(), s.cpu().numpy().astype(np.float64)) for t, s in ((c[0], c[2]), (c[1], c[3]))]
    m.kv_append(k0.cuda(), v0.cuda(), *c, tb, torch.zeros(B, dtype=torch.int32, device="cuda"),
                torch.tensor([14, 0], dtype=torch.int32, device="cuda"))
    want = [A.kv_append(t.double().numpy(), *first[i], table, [0, 0], [14, 0]) for i, t in enumerate((k0, v0))]
    k, v = (torch.zeros(B, 1, Hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(B, Hq, d, dtype=torch.bfloat16, device="cuda")
    o = torch.empty_like(q)

    def one():
        m.kv_append(k, v, *c, tb, start)
        m.attn_step(q, *c, tb, lens, o=o)

    keep = [t.clone() for t in c]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        one()
    torch.cuda.current_stream().wait_stream(s)
    for t, w in zip(c, keep):
        t.view(torch.uint8).copy_(w.view(torch.uint8))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one()
    for i in range(5):
        nk, nv, nq = (torch.randn(B, 1, Hk, d, generator=g) * (i + 1), torch.randn(B, 1, Hk, d, generator=g),
                      torch.randn(B, Hq, d, generator=g))
        nk, nv, nq = (t.to(torch.bfloat16) for t in (nk, nv, nq))
        k.copy_(nk); v.copy_(nv); q.copy_(nq)
        graph.replay()
        at = np.array([14, 0]) + i
        for j, t in enumerate((nk, nv)):
            want[j] = A.kv_append(t.double().numpy(), *want[j], table, at, [1, 1])
            assert np.array_equal(codes(c[j]), want[j][0])
        check(o, nq, [w[0] for w in want], [w[1] for w in want], table, at + 1)
        start += 1
        lens += 1


def test_append_after_rows_of_scale_zero(m):
    """A page that another writer filled with codes under scale 0 holds zeros, and still does
    once new tokens give it a scale."""
    Hk, page, d = 2, 32, 64
    c = m.kv_cache(1, Hk, page, d)
    for t in c[:2]:
        t.view(torch.uint8).copy_(torch.arange(Hk * page * d, device="cuda").view(1, Hk, page, d) % 0x7f)
    for t in c[2:]:
        t.zero_()
    x = torch.randn(1, 3, Hk, d, generator=torch.Generator().manual_seed(3)).cuda()
    at = torch.tensor([5], dtype=torch.int32, device="cuda")
    m.kv_append(x, x, *c, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), at)
    for i in range(2):
        want, scale = A.kv_append(x.double().cpu().numpy(), np.zeros((1, Hk, page, d), np.uint8), np.zeros((1, Hk)),
                                  np.zeros((1, 1), np.int64), [5], [3])
        assert np.array_equal(c[2 + i].cpu().numpy(), scale)
        assert np.array_equal(A.e4m3_decode(codes(c[i])[:, :, :8]), A.e4m3_decode(want[:, :, :8]))


@pytest.mark.parametrize("lens", [[0, 0], [1, 0], [4096, 0], [4096, 4095]])
def test_step_captured_twice(m, lens):
    """Two graphs of the same step, each with its own output and parts, replayed in turn."""
    code, scales, table, _ = filled(2, 4096, 2, 64, 128, 21, tail_nan=False)
    g = torch.Generator().manual_seed(22)
    qs = [torch.randn(2, 8, 64, generator=g).to(torch.bfloat16) for _ in range(2)]
    ln = np.array(lens)
    args = [x.cuda() for x in (torch.from_numpy(code[0]).view(torch.float8_e4m3fn),
                               torch.from_numpy(code[1]).view(torch.float8_e4m3fn),
                               torch.from_numpy(scales[0]).float(), torch.from_numpy(scales[1]).float(),
                               torch.from_numpy(table), torch.from_numpy(ln.astype(np.int32)))]
    outs, graphs, dq = [], [], [q.cuda() for q in qs]
    m.attn_step(dq[0], *args)
    for q in dq:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(m.attn_step(q, *args))
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for o, q in zip(outs, qs):
        check(o, q, code, scales, table, ln)


@pytest.mark.parametrize("d,Hq", [(64, 2), (128, 16)])
def test_step_small_queries_over_large_keys(m, d, Hq):
    """Queries of subnormal size over pages near the largest scale: their scores are ordinary,
    and the factor between them and the products must not pass through a subnormal."""
    code, (ks, vs), table, lens = filled(3, 300, 1, d, 32, 31)
    r = np.random.default_rng(32)
    sign = r.choice([-1.0, 1.0], d)
    k = r.uniform(100, 448, code[0].shape) * np.where(r.random(code[0].shape) < r.random((*code[0].shape[:3], 1)), sign, -sign)
    code[0] = np.where(code[0] & 0x7f == 0x7f, code[0], A.e4m3_encode(k))
    scales = (np.full_like(ks, 2.0 ** 119), vs)
    q = torch.from_numpy(sign * r.integers(17, 32, (3, Hq, d)) * 2.0 ** -133).to(torch.bfloat16)
    top = np.abs(A.e4m3_decode(code[0][table[0, 0], 0, :16]) * 2.0 ** 119 @ q[0].double().numpy().T).max() * d ** -0.5
    assert 0.5 < top < 16
    check(step(m, q, code, scales, table, lens), q, code, scales, table, lens)


@pytest.mark.parametrize("B,most,Hq,Hk,d,page,wide", [(3, 700, 16, 4, 128, 64, 40000), (4, 300, 16, 1, 128, 16, 9000),
                                                     (2, 257, 24, 1, 64, 32, 300000), (8, 5000, 32, 2, 128, 64, 8192)])
def test_step_with_a_table_wider_than_the_sequences(m, B, most, Hq, Hk, d, page, wide):
    """As a server allocates it: room for a context limit that no sequence has reached; the
    entries behind a sequence name no page, or pages of others."""
    code, scales, table, lens = filled(B, most, Hk, d, page, 41)
    q = torch.randn(B, Hq, d, generator=torch.Generator().manual_seed(42)).to(torch.bfloat16)
    full = np.full((B, wide // page), -1, np.int32)
    full[:, : table.shape[1]] = table
    full[1, table.shape[1]:] = table[0, 0]
    for window in (0, 100):
        check(step(m, q, code, scales, full, lens, window=window), q, code, scales, full, lens, window=window)
    m.device_wait_status()

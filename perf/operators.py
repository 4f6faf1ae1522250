"""Cases of the softmax-attention layer that stands between gated-delta-rule layers.

Five operators, each in its plain form (elementary torch operations in 32 bits, one
rounding at the end) and through the framework's entry points:

  rotary   rotary positions of q and k, and the same map's transpose (its gradient)
  fwd      softmax attention over token-major q, k, v: dense batches or packed sequences
  train    the same with its gradients, which recompute the probabilities
  append   new keys and values written into a paged cache of 8-bit values, one power-of-two
           scale for each page and head
  step     one token of each sequence attending over that cache

Shapes follow the recurrence's own workloads (16 heads of 128 channels, 32768 tokens; 2 heads
of 64 and 256 tokens; batches of 2, 8 and 64 sequences), with 4 or all of the heads on the
key side.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
LOW_EXP = -100  # exponent of the smallest scale of a cache page


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one new token of 64 streams, at positions far into long contexts
        dict(name="rotary_token", op="rotary", B=64, T=1, Hq=16, Hk=4, d=128, rot=128, inter=False,
             inverse=False, dtype="bf16", yarn=False, far=1000000),
        # a whole training sequence of the long-context workload, frequencies stretched for it
        dict(name="rotary_sequence", op="rotary", B=1, T=32768, Hq=16, Hk=4, d=128, rot=128,
             inter=False, inverse=False, dtype="bf16", yarn=True, far=0),
        # the gradient, on half of each head, pairs interleaved, float32, an odd length
        dict(name="rotary_grad_half_head", op="rotary", B=2, T=8191, Hq=8, Hk=8, d=64, rot=32,
             inter=True, inverse=True, dtype="fp32", yarn=False, far=0),
        # a short prompt of a small layer: latency
        dict(name="fwd_short", op="fwd", lens="256", lens_k="256", Hq=2, Hk=2, d=64, causal=True,
             window=0, packed=False),
        # prefill of one long document
        dict(name="fwd_long", op="fwd", lens="16384", lens_k="16384", Hq=16, Hk=4, d=128,
             causal=True, window=0, packed=False),
        # prefill of documents of mixed length in one buffer
        dict(name="fwd_packed", op="fwd", lens="1 37 700 2049 300 0 1500 130 3331",
             lens_k="1 37 700 2049 300 0 1500 130 3331", Hq=16, Hk=4, d=128, causal=True,
             window=0, packed=True),
        # a training step of a dense batch
        dict(name="train_dense", op="train", lens="8192 8192", lens_k="8192 8192", Hq=8, Hk=8,
             d=128, causal=True, window=0, packed=False),
        # a training step over packed documents, small heads, a sliding window, shared key heads
        dict(name="train_packed_window", op="train", lens="600 2500 333 1 1111 700",
             lens_k="600 2500 333 1 1111 700", Hq=16, Hk=4, d=64, causal=True, window=513,
             packed=True),
        # decoding: the new token of each of 64 streams goes into the cache
        dict(name="append_token", op="append", B=64, T=1, Hk=4, d=128, page=64, most=4096,
             dtype="bf16"),
        # prompts of mixed length (right-padded batch) go into the cache
        dict(name="append_prompts", op="append", B=8, T=4096, Hk=4, d=128, page=64, most=8192,
             dtype="bf16"),
        # one stream decoding: latency, work split over its length
        dict(name="step_one", op="step", B=1, most=4097, Hq=16, Hk=4, d=128, page=64, window=0),
        # 64 streams of mixed length decoding
        dict(name="step_batch", op="step", B=64, most=16384, Hq=16, Hk=4, d=128, page=64, window=0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "fwd", "fwd", "train", "train", "append", "step", "step"])
    d = rng.choice([64, 128])
    Hk = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 1, 2, 3, 4, 8])
    Hq = Hk * group
    if op == "rotary":
        B = rng.choice([1, 2, 3, 8, 64])
        T = _log_int(rng, 1, max(1, 32768 * 20 // (B * (Hq + Hk))))
        return dict(op=op, B=B, T=min(T, 32768), Hq=Hq, Hk=Hk, d=d, rot=rng.choice([d, d, d // 2, d // 4]),
                    inter=rng.random() < 0.5, inverse=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), yarn=rng.random() < 0.3,
                    far=rng.choice([0, 0, 1000, 10000000]))
    if op in ("fwd", "train"):
        causal = rng.random() < 0.8
        window = rng.choice([0, 0, _log_int(rng, 1, 2000)]) if causal else 0
        packed = rng.random() < 0.5
        if packed:
            n = rng.randint(1, 8)
            lens = [rng.choice([0, 1, _log_int(rng, 1, 2000), _log_int(rng, 100, 2000)]) for _ in range(n)]
            if sum(lens) == 0:
                lens[0] = 77
            lens_k = list(lens)
        else:
            B = rng.choice([1, 2, 3])
            T = _log_int(rng, 1, 4096)
            lens = [T] * B
            # queries that follow a prefix already seen, or fewer keys than queries
            Tk = max(1, rng.choice([T, T, T + _log_int(rng, 1, 1000), T // 2]))
            lens_k = [Tk] * B
        while Hq * len(lens) * max(lens) * max(lens_k) > 8 * 2 * 8192 * 8192:
            Hq //= 2
            Hk = max(1, Hk // 2)
            Hq = max(Hq // Hk, 1) * Hk
        return dict(op=op, lens=" ".join(map(str, lens)), lens_k=" ".join(map(str, lens_k)), Hq=Hq,
                    Hk=Hk, d=d, causal=causal, window=window, packed=packed)
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        B = rng.choice([1, 2, 5, 8, 64])
        T = rng.choice([1, 1, _log_int(rng, 2, max(2, 32768 // B))])
        return dict(op=op, B=B, T=T, Hk=min(Hk, 4), d=d, page=page, most=T + _log_int(rng, 1, 2000),
                    dtype=rng.choice(["bf16", "bf16", "fp32"]))
    B = rng.choice([1, 2, 7, 16, 64])
    most = _log_int(rng, 1, min(65536, 64 * 16384 * 4 // (B * Hk)) // 2)
    return dict(op=op, B=B, most=most, Hq=Hq, Hk=Hk, d=d, page=page,
                window=rng.choice([0, 0, 0, _log_int(rng, 1, 2000)]))


# ------------------------------------------------------------------ inputs


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _lens(case):
    """Query and key lengths of the sequences."""
    return list(map(int, case["lens"].split())), list(map(int, case["lens_k"].split()))


def _frequencies(case):
    """Angles per position, in 64 bits, and the factor on the rotated values: base 10000; with
    "yarn" the published blend (arXiv 2309.00071) for 16 times the length of 2048."""
    r = case["rot"]
    f = 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)
    if not case["yarn"]:
        return f, 1.0
    factor, length = 16.0, 2048
    low = r * math.log(length / (32 * 2 * math.pi)) / (2 * math.log(10000.0))
    high = r * math.log(length / (2 * math.pi)) / (2 * math.log(10000.0))
    low, high = max(math.floor(low), 0), min(math.ceil(high), r - 1)
    ramp = ((torch.arange(r // 2, dtype=torch.float64) - low) / max(high - low, 0.001)).clamp(0, 1)
    return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0


def _lengths(gen, B, most):
    """Ragged lengths up to `most`, the first one at it."""
    n = (torch.rand(B, generator=gen) * most).long() + 1
    n[0] = most
    return n.clamp(max=most)


def _pages(case, gen, B, most):
    """A cache's page table (unused entries -1, pages in no order) and its number of pages."""
    per = -(-most // case["page"])
    order = torch.randperm(B * per + 3, generator=gen)[: B * per].reshape(B, per)
    return order.to(torch.int32), B * per + 3


def prepare(case, seed):
    cpu = torch.Generator().manual_seed(seed * 7919 + 17)
    gpu = torch.Generator("cuda").manual_seed(seed * 7919 + 17)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gpu, device="cuda").to(dtype)

    s = dict(case)
    op = case["op"]
    if op == "rotary":
        B, T, d = case["B"], case["T"], case["d"]
        s["q"] = normal(B, T, case["Hq"], d, dtype=_dtype(case["dtype"]))
        s["k"] = normal(B, T, case["Hk"], d, dtype=_dtype(case["dtype"]))
        start = torch.randint(0, case["far"] + 1, (B, 1), generator=cpu)
        s["positions"] = (start + torch.arange(T)).to(torch.int32).cuda()
        f, s["mscale"] = _frequencies(case)
        s["inv_freq"] = f.cuda()
    elif op in ("fwd", "train"):
        Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
        lens, lens_k = s["lens"], s["lens_k"] = _lens(case)
        lead = (1, sum(lens)) if case["packed"] else (len(lens), lens[0])
        lead_k = (1, sum(lens_k)) if case["packed"] else (len(lens), lens_k[0])
        s["q"], s["k"], s["v"] = normal(*lead, Hq, d), normal(*lead_k, Hk, d), normal(*lead_k, Hk, d)
        if op == "train":
            s["do"] = normal(*lead, Hq, d)
        s["cu"] = [0] + np.cumsum(lens).tolist()
    else:
        B, Hk, d, page, most = case["B"], case["Hk"], case["d"], case["page"], case["most"]
        table, num = _pages(case, cpu, B, most)
        s["k_pages"] = (normal(num, Hk, page, d) * 64).clamp(-448, 448).to(torch.float8_e4m3fn)
        s["v_pages"] = (normal(num, Hk, page, d) * 64).clamp(-448, 448).to(torch.float8_e4m3fn)
        for name in ("k_scale", "v_scale"):
            s[name] = torch.pow(2.0, torch.randint(-8, -4, (num, Hk), generator=cpu).float()).cuda()
        if op == "append":
            T = case["T"]
            room = torch.full((B,), most) - T
            s["start"] = (torch.rand(B, generator=cpu) * (room + 1)).long().to(torch.int32).cuda()
            count = _lengths(cpu, B, T)
            s["count"] = count.to(torch.int32).cuda()
            s["k"] = normal(B, T, Hk, d, dtype=_dtype(case["dtype"]))
            s["v"] = normal(B, T, Hk, d, dtype=_dtype(case["dtype"]))
            s["table"] = table.cuda()
        else:
            lens = _lengths(cpu, B, most)
            used = torch.arange(table.shape[1])[None] * page < lens[:, None]
            s["table"] = torch.where(used, table, torch.full_like(table, -1)).cuda()
            s["lens"] = lens.to(torch.int32).cuda()
            s["q"] = normal(B, case["Hq"], d)
    return s


# ------------------------------------------------------------------ plain forms


def _rotate(x, cos, sin, rot, inter):
    """Pairs (a, b) -> (a cos - b sin, b cos + a sin) of the first `rot` channels."""
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., : rot // 2], x[..., rot // 2: rot])
    ya, yb = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((ya, yb), -1).flatten(-2) if inter else torch.cat((ya, yb), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _plain_rotary(s):
    angle = s["positions"].double()[..., None] * s["inv_freq"]
    cos = (angle.cos() * s["mscale"]).float()[:, :, None]
    sin = (angle.sin() * s["mscale"]).float()[:, :, None]
    sin = -sin if s["inverse"] else sin
    return (_rotate(s["q"], cos, sin, s["rot"], s["inter"]).to(s["q"].dtype),
            _rotate(s["k"], cos, sin, s["rot"], s["inter"]).to(s["k"].dtype))


def _padded(x, lens):
    """[1, sum, H, d] or [n, L, H, d] -> float32 [n, H, L, d]; and which rows are tokens."""
    n, L = len(lens), max(lens)
    length = torch.tensor(lens, device=x.device)
    rows = torch.arange(L, device=x.device)
    valid = rows < length[:, None]
    if x.shape[0] == n and x.shape[1] == L:
        return x.float().transpose(1, 2), valid
    first = torch.cumsum(length, 0) - length
    at = (first[:, None] + rows).clamp(max=x.shape[1] - 1)
    return x[0][at].float().transpose(1, 2), valid


def _unpadded(x, valid, like):
    """The reverse of _padded, rounded to the type of `like`."""
    return x.transpose(1, 2)[valid].reshape(like.shape[:2] + x.shape[1:2] + x.shape[3:]).to(like.dtype)


def _visible(s, device):
    """[n, 1, Lq, Lk]: which keys a query sees; its own position is counted from the keys' end."""
    lq = torch.tensor(s["lens"], device=device)[:, None, None]
    lk = torch.tensor(s["lens_k"], device=device)[:, None, None]
    i = torch.arange(max(s["lens"]), device=device)[None, :, None]
    j = torch.arange(max(s["lens_k"]), device=device)[None, None, :]
    see = (i < lq) & (j < lk)
    if s["causal"]:
        see = see & (j <= i + lk - lq)
    if s["window"]:
        see = see & (j > i + lk - lq - s["window"])
    return see[:, None]


def _plain_attention(s):
    q, valid = _padded(s["q"], s["lens"])
    k, valid_k = _padded(s["k"], s["lens_k"])
    v, _ = _padded(s["v"], s["lens_k"])
    group, scale = s["Hq"] // s["Hk"], s["d"] ** -0.5
    kg, vg = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
    p = q @ kg.transpose(2, 3)
    p.mul_(scale).masked_fill_(~_visible(s, q.device), -math.inf)
    m = p.amax(-1, keepdim=True)
    p.sub_(m.masked_fill(m == -math.inf, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(total.masked_fill(total == 0, 1.0))
    lse = (m + total.log()).transpose(1, 2)[valid].reshape(s["q"].shape[:3]).transpose(1, 2)
    o = p @ vg
    if s["op"] == "fwd":
        return _unpadded(o, valid, s["q"]), lse.contiguous()
    do, _ = _padded(s["do"], s["lens"])
    do = do * valid[:, None, :, None]
    n, Hk, Lk, d = k.shape
    dv = (p.transpose(2, 3) @ do).reshape(n, Hk, group, Lk, d).sum(2)
    ds = do @ vg.transpose(2, 3)
    ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    dq = ds @ kg
    dk = (ds.transpose(2, 3) @ q).reshape(n, Hk, group, Lk, d).sum(2)
    return (_unpadded(o, valid, s["q"]), _unpadded(dq, valid, s["q"]),
            _unpadded(dk, valid_k, s["k"]), _unpadded(dv, valid_k, s["v"]))


def _plain_append_one(s, new, pages, scale):
    """The pages that the new rows touch: their scale grows to what the rows need, values held
    under a smaller scale are encoded again, the new rows are encoded."""
    B, T, Hk, d = new.shape
    page = s["page"]
    start, count = s["start"].long()[:, None, None], s["count"].long()[:, None, None]
    slot = start // page + torch.arange((T + page - 2) // page + 1, device=new.device)[None, :, None]
    t = slot * page + torch.arange(page, device=new.device) - start  # [B, slots, page]
    fresh, held = (t >= 0) & (t < count), t < 0
    touched = fresh.any(-1)
    x = new.float()[torch.arange(B, device=new.device)[:, None, None], t.clamp(0, T - 1)]
    size = torch.where(fresh[..., None, None] & x.isfinite(), x.abs(), 0.0).amax((2, 4))
    mantissa, exponent = torch.frexp(size)  # 448 = 0.875 * 2^9
    exponent = (exponent - torch.where(mantissa <= 0.875, 9, 8)).clamp(min=LOW_EXP)
    need = torch.ldexp(torch.ones_like(size), exponent)
    ids = s["table"].long().gather(1, slot[:, :, 0].clamp(max=s["table"].shape[1] - 1)).clamp(min=0)
    old = torch.where(held.any(-1)[..., None], scale[ids], 0.0)
    grown = torch.maximum(old, need)  # [B, slots, Hk]
    was = pages.view(torch.uint8)[ids].view(torch.float8_e4m3fn)  # [B, slots, Hk, page, d]
    again = (was.float() * (old / grown)[..., None, None]).to(torch.float8_e4m3fn)
    code = (x.permute(0, 1, 3, 2, 4) / grown[..., None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    out = torch.where(fresh[:, :, None, :, None], code.view(torch.uint8),
                      torch.where(held[:, :, None, :, None], again.view(torch.uint8), was.view(torch.uint8)))
    pages.view(torch.uint8)[ids[touched]] = out[touched]
    scale[ids[touched]] = grown[touched]


def _plain_append(s):
    _plain_append_one(s, s["k"], s["k_pages"], s["k_scale"])
    _plain_append_one(s, s["v"], s["v_pages"], s["v_scale"])
    return s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]


def _plain_step(s):
    ids = s["table"].long().clamp(min=0)
    B, P = ids.shape

    def rows(pages, scale):
        x = pages.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float() * scale[ids][..., None, None]
        return x.transpose(1, 2).reshape(B, s["Hk"], P * s["page"], s["d"])

    q = s["q"].float().reshape(B, s["Hk"], -1, s["d"])
    p = (q @ rows(s["k_pages"], s["k_scale"]).transpose(2, 3)) * s["d"] ** -0.5
    j, n = torch.arange(P * s["page"], device=q.device), s["lens"].long()[:, None]
    see = j < n
    if s["window"]:
        see = see & (j >= n - s["window"])
    p.masked_fill_(~see[:, None, None], -math.inf)
    p = (p - p.amax(-1, keepdim=True)).exp_()
    o = (p @ rows(s["v_pages"], s["v_scale"])) / p.sum(-1, keepdim=True)
    return o.reshape(s["q"].shape).to(s["q"].dtype)


# ------------------------------------------------------------------ one pass


def run(state):
    s = state
    if own:
        import gated_delta_rule_115_b200 as m
        if s["op"] == "rotary":
            return m.rotary(s["q"], s["k"], positions=s["positions"], inv_freq=s["inv_freq"],
                            interleaved=s["inter"], mscale=s["mscale"], inverse=s["inverse"])
        if s["op"] in ("fwd", "train"):
            if s["packed"]:
                o, lse = m.attn_fwd_varlen(s["q"], s["k"], s["v"], s["cu"], causal=s["causal"],
                                           window=s["window"])
            else:
                o, lse = m.attn_fwd(s["q"], s["k"], s["v"], causal=s["causal"], window=s["window"])
            if s["op"] == "fwd":
                return o, lse
            if s["packed"]:
                g = m.attn_bwd_varlen(s["q"], s["k"], s["v"], o, lse, s["do"], s["cu"],
                                      causal=s["causal"], window=s["window"])
            else:
                g = m.attn_bwd(s["q"], s["k"], s["v"], o, lse, s["do"], causal=s["causal"],
                               window=s["window"])
            return o, g["dq"], g["dk"], g["dv"]
        if s["op"] == "append":
            m.kv_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"],
                        s["table"], s["start"], count=s["count"])
            return s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]
        return m.attn_step(s["q"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"],
                           s["table"], s["lens"], window=s["window"])
    return dict(rotary=_plain_rotary, fwd=_plain_attention, train=_plain_attention,
                append=_plain_append, step=_plain_step)[s["op"]](s)


# ------------------------------------------------------------------ what a pass cannot do without


def _pairs(case):
    """Visible (query, key) pairs of one head, over all sequences."""
    total = 0
    for lq, lk in zip(*_lens(case)):
        last = np.arange(lq, dtype=np.int64) + lk - lq
        hi = np.minimum(last, lk - 1) if case["causal"] else np.full(lq, lk - 1)
        lo = np.maximum(last - case["window"] + 1, 0) if case["window"] else 0
        total += int(np.maximum(hi - lo + 1, 0).sum())
    return total


def work(case):
    op, d = case["op"], case["d"]
    if op == "rotary":
        n = case["B"] * case["T"] * (case["Hq"] + case["Hk"])
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * n * d * size + 4 * case["B"] * case["T"], "flops": 3 * n * case["rot"]}
    if op in ("fwd", "train"):
        lens, lens_k = _lens(case)
        q, k = sum(lens) * case["Hq"] * d, sum(lens_k) * case["Hk"] * d
        products = _pairs(case) * case["Hq"] * d * 2
        if op == "fwd":
            return {"bytes": 2 * (2 * q + 2 * k) + 4 * q // d, "flops": 2 * products}
        return {"bytes": 2 * (4 * q + 4 * k), "flops": 7 * products}
    Hk = case["Hk"]
    if op == "append":
        gen = torch.Generator().manual_seed(0)
        n = int(_lengths(gen, case["B"], case["T"]).sum()) * Hk * d * 2
        return {"bytes": n * (1 + (2 if case["dtype"] == "bf16" else 4)), "flops": n}
    gen = torch.Generator().manual_seed(0)
    n = _lengths(gen, case["B"], case["most"])
    n = int((n.clamp(max=case["window"]) if case["window"] else n).sum())
    return {"bytes": n * Hk * (2 * d + 8.0 / case["page"]) + 4 * case["B"] * case["Hq"] * d,
            "flops": 4 * n * case["Hq"] * d}


# ------------------------------------------------------------------ the definitions, in 64 bits


def _exact_rotary(s):
    half = s["rot"] // 2

    def turn(x):
        x = x.double()
        j = torch.arange(half, device=x.device)
        first, second = (2 * j, 2 * j + 1) if s["inter"] else (j, j + half)
        unit = torch.polar(torch.full_like(s["inv_freq"], s["mscale"])[None, None].expand(s["B"], s["T"], half).contiguous(),
                           (-1.0 if s["inverse"] else 1.0) * s["positions"].double()[..., None] * s["inv_freq"])
        z = torch.complex(x[..., first], x[..., second]) * unit[:, :, None]
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    return turn(s["q"]), turn(s["k"])


def _exact_attention(s):
    """Each sequence and head by itself."""
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    o, lse = torch.zeros_like(q), torch.zeros(q.shape[0], q.shape[2], q.shape[1], dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    group, at_q, at_k = s["Hq"] // s["Hk"], 0, 0
    for n, (lq, lk) in enumerate(zip(s["lens"], s["lens_k"])):
        b = 0 if s["packed"] else n
        rq = slice(at_q, at_q + lq) if s["packed"] else slice(0, lq)
        rk = slice(at_k, at_k + lk) if s["packed"] else slice(0, lk)
        at_q, at_k = at_q + lq, at_k + lk
        if lq == 0 or lk == 0:
            continue
        back = torch.arange(lq, device="cuda")[:, None] + (lk - lq) - torch.arange(lk, device="cuda")
        hidden = torch.zeros_like(back, dtype=torch.bool)
        if s["causal"]:
            hidden |= back < 0
        if s["window"]:
            hidden |= back >= s["window"]
        none = hidden.all(-1, keepdim=True)
        for h in range(s["Hq"]):
            a, kk, vv = q[b, rq, h], k[b, rk, h // group], v[b, rk, h // group]
            z = torch.where(hidden, -math.inf, a @ kk.T / math.sqrt(s["d"]))
            lse[b, h, rq] = torch.logsumexp(z, -1)
            w = torch.softmax(z.masked_fill(none, 0.0), -1) * ~none
            del z
            o[b, rq, h] = w @ vv
            if s["op"] == "train":
                g = s["do"][b, rq, h].double()
                dv[b, rk, h // group] += w.T @ g
                w *= g @ vv.T - (g * o[b, rq, h]).sum(-1, keepdim=True)
                dq[b, rq, h] = w @ kk / math.sqrt(s["d"])
                dk[b, rk, h // group] += w.T @ a / math.sqrt(s["d"])
            del w
    return (o, lse) if s["op"] == "fwd" else (o, dq, dk, dv)


def _exact_append(s):
    """Page by page; stored values as they would be without the rounding to 8 bits."""
    page = s["page"]
    out = []
    for new, pages, scale in ((s["k"], s["k_pages"], s["k_scale"]), (s["v"], s["v_pages"], s["v_scale"])):
        codes, scales = pages.double(), scale.double()
        start, count, table = s["start"].tolist(), s["count"].tolist(), s["table"].tolist()
        for b in range(s["B"]):
            for c in range(start[b] // page, (start[b] + count[b] - 1) // page + 1):
                lo, hi = max(start[b], c * page), min(start[b] + count[b], (c + 1) * page)
                x = new[b, lo - start[b]: hi - start[b]].double().transpose(0, 1)  # [Hk, rows, d]
                i = table[b][c]
                need = torch.exp2(torch.ceil(torch.log2(x.abs().amax((1, 2)) / E4M3_MAX)).clamp(min=LOW_EXP))
                old = scales[i].clone()
                now = torch.maximum(old, need) if lo > c * page else need
                codes[i, :, : lo - c * page] *= (old / now)[:, None, None]
                codes[i, :, lo - c * page: hi - c * page] = x / now[:, None, None]
                scales[i] = now
        out.append((codes, scales))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def _exact_step(s):
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        ids = s["table"][b, : -(-n // s["page"])].long()
        first = max(0, n - s["window"]) if s["window"] else 0

        def rows(pages, scale):
            x = pages.view(torch.uint8)[ids].view(torch.float8_e4m3fn).double() * scale.double()[ids][:, :, None, None]
            return x.transpose(0, 1).reshape(s["Hk"], -1, s["d"])[:, first:n]

        q = s["q"][b].double().reshape(s["Hk"], -1, s["d"])
        w = torch.softmax(q @ rows(s["k_pages"], s["k_scale"]).transpose(1, 2) / math.sqrt(s["d"]), -1)
        o[b] = (w @ rows(s["v_pages"], s["v_scale"])).reshape(-1, s["d"])
    return o


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append" and sum(-(-int(n) // case["page"]) + 1 for n in s["count"]) > 4000:
        return None
    return dict(rotary=_exact_rotary, fwd=_exact_attention, train=_exact_attention,
                append=_exact_append, step=_exact_step)[case["op"]](s)

"""What is measured of the 4-bit paged KV cache: filling it, attending over it, reading it back.

Three operators, in the order in which a decoder layer uses them after its QKV projection:

  append   rotates queries and keys by their positions, quantizes keys and values to 4 bits and
           writes them into the pages of their sequences;
  attend   attention of the newest tokens of each sequence over the cached ones, causal, with an
           optional sliding window and a few first positions that stay visible;
  values   the cached keys and values of given positions as 16-bit floats.

A page holds `page` positions of every kv head.  Of one head it holds, in 32-bit words,

  key codes     [page][D / 8]       code of channel 8 i + j in bits 4 j of word i
  value codes   [page / 4][D / 8][4]  the same words, four positions side by side
  key groups    [Gd][page]          one word for each position and group of channels
  value groups  [Gd][page]

with groups of min(D, 128) channels, Gd = max(1, D / 128).  A group's word holds its scale s
(binary32 with 7 significant bits: the upper half) and zero point z (the low 4 bits); code q
stands for (q - z) s.  Sequence b has its position p in page page_table[b][p / page]; its newest
tokens, rows offsets[b] .. offsets[b + 1] - 1 of a call, end at position lengths[b] - 1.

Heads, widths and lengths are those of the repository's cache and QKV workloads (32 heads of 128,
4096 positions, a fused projection of 12288) and common ones with shared kv heads.  `own` chooses
between the plain torch forms below and the framework's entry points.
"""
import math
import random

import torch

own = False

DEV = "cuda"
_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one decode step of sixteen requests: rotate, quantize and store one token each (latency)
        _append("append_step", B=16, n=1, ragged=False, ctx=4096, Hq=32, H=8, D=128, page=64, x="bf16"),
        # a prompt of 4096 tokens as it leaves the fused QKV projection: q, k and v are views of its output
        _append("append_prompt", B=1, n=4096, ragged=False, ctx=4096, Hq=32, H=32, D=128, page=64, x="f16"),
        # prompts of several lengths, wide heads, neighbouring channels rotated and only half of them
        _append("append_ragged", B=7, n=300, ragged=True, ctx=1000, Hq=8, H=2, D=256, page=16, x="f32", rot=128, pairs=True),
        # one request's next token, a kv head for each query head
        _attend("attend_step", B=1, n=1, ragged=False, ctx=4096, Hq=32, H=32, D=128, page=64, x="f16"),
        # continuous batching: 64 requests of very different lengths, long caches
        _attend("attend_batch", B=64, n=1, ragged=False, ctx=16384, Hq=32, H=8, D=128, page=64, x="bf16"),
        # the same with a sliding window and visible first tokens: most of the cache is out of sight
        _attend("attend_window", B=32, n=1, ragged=False, ctx=16384, Hq=32, H=8, D=128, page=128, x="bf16", window=1024, sinks=4),
        # checking five drafted tokens of each request in one step, narrow heads, small pages
        _attend("attend_draft", B=8, n=5, ragged=False, ctx=2047, Hq=16, H=2, D=64, page=16, x="f16"),
        # a whole prompt
        _attend("attend_prompt", B=1, n=4096, ragged=False, ctx=4096, Hq=32, H=32, D=128, page=64, x="bf16"),
        # the next chunks of three long prompts under a sliding window
        _attend("attend_chunk", B=3, n=1500, ragged=True, ctx=8192, Hq=16, H=4, D=128, page=64, x="f16", window=2048, sinks=16),
        # prompts and single tokens in one call, wide heads, one kv head
        _attend("attend_mixed", B=9, n=900, ragged=True, ctx=4001, Hq=8, H=1, D=256, page=32, x="bf16"),
        # a cached prefix read back, and the caches of eight requests
        _values("values_prefix", B=1, n=500, ragged=False, ctx=2048, H=8, D=128, page=64, out="bf16"),
        _values("values_all", B=8, n=8192, ragged=False, ctx=8192, H=8, D=128, page=64, out="f16"),
    ]


def _append(name=None, rot=None, pairs=False, **c):
    return _named(name, dict(op="append", rot=c["D"] if rot is None else rot, pairs=pairs, **c))


def _attend(name=None, window=0, sinks=0, **c):
    return _named(name, dict(op="attend", window=window, sinks=sinks, **c))


def _values(name=None, **c):
    return _named(name, dict(op="values", **c))


def _named(name, case):
    return case if name is None else {"name": name, **case}


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "attend", "values"])
    D = rng.choice([64, 128, 128, 256])
    H = rng.choice([1, 2, 4, 8, 32])
    Hq = H * rng.choice([g for g in (1, 2, 3, 4, 6, 8, 16) if g * H <= 64])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "append":
        T = _log(rng, 1, min(8192, (50 << 20) // (D * (Hq + 2 * H))))
        B = _log(rng, 1, min(T, 64))
        n = max(1, T // B)
        return _append(B=B, n=n, ragged=rng.random() < 0.5, ctx=n + rng.randint(0, 2000), Hq=Hq, H=H, D=D, page=page,
                       x=rng.choice(list(_DT)), rot=rng.choice([D, D, D // 2]), pairs=rng.random() < 0.3)
    if op == "values":
        T = _log(rng, 1, min(65536, (1 << 26) // (D * H)))
        B = _log(rng, 1, min(T, 32))
        n = max(1, T // B)
        return _values(B=B, n=n, ragged=rng.random() < 0.5, ctx=n + rng.randint(0, 500), H=H, D=D, page=page,
                       out=rng.choice(["f16", "bf16"]))
    more = dict(Hq=Hq, H=H, D=D, page=page, x=rng.choice(["f16", "bf16"]))
    if rng.random() < 0.4:
        more.update(window=_log(rng, 16, 4096), sinks=rng.choice([0, 1, 4, 64]))
    if rng.random() < 0.6:  # single tokens and drafts
        B = _log(rng, 1, 64)
        ctx = _log(rng, 1, min(65536, (9 << 26) // (B * H * D)))
        return _attend(B=B, n=min(ctx, rng.choice([1, 1, 1, 2, 5])), ragged=rng.random() < 0.2, ctx=ctx, **more)
    n = _log(rng, 2, min(4096, math.isqrt((1 << 35) // (D * Hq))))
    B = _log(rng, 1, max(1, min(8, 4096 // n, (1 << 35) // (D * Hq * n * n))))
    ctx = n + rng.randint(0, min(8192, (1 << 35) // (D * Hq * B * n) - n))
    return _attend(B=B, n=n, ragged=rng.random() < 0.5, ctx=ctx, **more)


# ---- inputs ------------------------------------------------------------------


def _plan(case):
    """Tokens of the call and cached positions of each sequence: a batch's lengths lie between a
    quarter of the longest and the longest; a ragged call has between one token and n of each."""
    B, n, ctx = case["B"], case["n"], case["ctx"]
    rng = random.Random("%d %d %d" % (B, n, ctx))
    new = [n] + [n if not case["ragged"] else rng.choice([1, rng.randint(1, n)]) for _ in range(B - 1)]
    length = [ctx] + [rng.randint(max(m, ctx // 4), ctx) for m in new[1:]]
    return new, length


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _magnitudes(g, H, D):
    """Channels differ in size, and two of each head are ten times the others."""
    m = torch.exp(torch.randn((H, D), generator=g, device=DEV) * 0.5)
    most = torch.rand((H, D), generator=g, device=DEV).argsort(1)[:, :2]
    return m.scatter(1, most, m.gather(1, most) * 10.0)


def _groups(D):
    return max(1, D // 128)


def _words(page, D):
    return page * (D // 4 + 2 * _groups(D))


def _cache(g, case, total):
    """Pages of quantized draws, a few at a time to bound the memory."""
    H, D, page = case["H"], case["D"], case["page"]
    pages = torch.empty((total, H, _words(page, D)), dtype=torch.int32, device=DEV)
    kmag, vmag = _magnitudes(g, H, D), _magnitudes(g, H, D) * 0.2
    some = max(1, (1 << 26) // (page * H * D))
    for at in range(0, total, some):
        here = min(some, total - at)
        kw, kp = _encode(torch.randn((here, page, H, D), generator=g, device=DEV) * kmag)
        vw, vp = _encode(torch.randn((here, page, H, D), generator=g, device=DEV) * vmag)
        pages[at:at + here] = torch.cat([
            kw.permute(0, 2, 1, 3).reshape(here, H, -1),
            vw.permute(0, 2, 1, 3).reshape(here, H, page // 4, 4, D // 8).transpose(3, 4).reshape(here, H, -1),
            kp.permute(0, 2, 3, 1).reshape(here, H, -1), vp.permute(0, 2, 3, 1).reshape(here, H, -1)], 2)
    return pages


def prepare(case, seed):
    g, s = _gen(seed), dict(case)
    B, D, H, page = case["B"], case["D"], case["H"], case["page"]
    new, length = _plan(case)
    T = sum(new)
    width = -(-case["ctx"] // page)
    used = [-(-l // page) for l in length]
    total = sum(used) + 3
    free = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b in range(B):
        table[b, : used[b]] = free[at: at + used[b]]
        at += used[b]
    s["table"] = table
    s["lengths"] = torch.tensor(length, dtype=torch.int32, device=DEV)
    s["offsets"] = None
    if case["ragged"]:
        s["offsets"] = torch.tensor([0] + new, device=DEV).cumsum(0).int()
    s["T"] = T
    if case["op"] == "append":
        s["pages"] = torch.zeros((total, H, _words(page, D)), dtype=torch.int32, device=DEV)
        x = torch.randn((T, case["Hq"] + 2 * H, D), generator=g, device=DEV)
        x[:, case["Hq"]:] *= torch.cat([_magnitudes(g, H, D), _magnitudes(g, H, D) * 0.2])
        x = x.to(_DT[case["x"]])
        s["q"], s["k"], s["v"] = x.split([case["Hq"], H, H], 1)  # views of the projection's rows
        turn = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device=DEV) / case["rot"])
        angle = torch.arange(case["ctx"], dtype=torch.float64, device=DEV)[:, None] * turn
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        return s
    s["pages"] = _cache(g, case, total)
    if case["op"] == "attend":
        s["q"] = torch.randn((T, case["Hq"], D), generator=g, device=DEV).to(_DT[case["x"]])
    return s


# ---- one pass ------------------------------------------------------------------


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import bit_quantized_gemm_int8_amd as qg
    op, where = s["op"], (s["pages"], s["table"], s["lengths"])
    if op == "append":
        q = qg.append_kv_u4_pages(s["k"], s["v"], *where, offsets=s["offsets"], q=s["q"], cos=s["cos"], sin=s["sin"],
                                  interleaved=s["pairs"])
        # the cache is the state's own; its new positions as the values they stand for
        return (q,) + tuple(qg.dequantize_kv_u4_pages(*where, s["T"], s["D"], offsets=s["offsets"], out_dtype=torch.float16))
    if op == "attend":
        return qg.attend_kv_u4_pages(s["q"], *where, offsets=s["offsets"], window=s["window"], sinks=s["sinks"])
    return qg.dequantize_kv_u4_pages(*where, s["T"], s["D"], offsets=s["offsets"], out_dtype=_DT[s["out"]])


def _encode(x):
    """[..., D] values -> code words [..., D / 8] and group words [..., Gd]; every step is one binary32 rounding."""
    D = x.shape[-1]
    x = x.unflatten(-1, (_groups(D), min(D, 128)))
    lo, hi = x.amin(-1).clamp_max(0.0), x.amax(-1).clamp_min(0.0)
    t = (hi - lo) / torch.full_like(lo, 15.0)
    s = ((t.view(torch.int32) + 0x1FFFF) & ~0x1FFFF).view(torch.float32)  # up to 7 significant bits
    full = s > 0
    d = torch.where(full, s, 1.0)
    z = torch.where(full, torch.round(-lo / d), 0.0).clamp(0, 15)
    q = torch.where(full[..., None], torch.round(x / d[..., None]) + z[..., None], 0.0).clamp(0, 15)
    q = q.to(torch.int32).flatten(-2).unflatten(-1, (D // 8, 8))
    shift = torch.arange(0, 32, 4, dtype=torch.int32, device=x.device)
    return (q << shift).sum(-1, dtype=torch.int32), s.view(torch.int32) | z.to(torch.int32)


def _decode(words, params):
    """Code words [..., D / 8] and group words [..., Gd] -> [..., D] values in binary32."""
    shift = torch.arange(0, 32, 4, dtype=torch.int32, device=words.device)
    q = ((words[..., None] >> shift) & 15).flatten(-2)
    s, z = (params & -0x10000).view(torch.float32), params & 15
    q = q.unflatten(-1, (params.shape[-1], -1))
    return ((q - z[..., None]).float() * s[..., None]).flatten(-2)


def _sections(page, D):
    """First word of the key codes, value codes, key groups, value groups of a head, and the end."""
    c, p = page * D // 8, page * _groups(D)
    return 0, c, 2 * c, 2 * c + p, 2 * (c + p)


def _cached(words, page, D):
    """[..., words] of pages -> keys and values [..., page, D]."""
    a, b, c, d, e = _sections(page, D)
    k = words[..., a:b].unflatten(-1, (page, D // 8))
    v = words[..., b:c].unflatten(-1, (page // 4, D // 8, 4)).transpose(-1, -2).flatten(-3, -2)
    kp = words[..., c:d].unflatten(-1, (_groups(D), page)).transpose(-1, -2)
    vp = words[..., d:e].unflatten(-1, (_groups(D), page)).transpose(-1, -2)
    return _decode(k, kp), _decode(v, vp)


def _rows(s):
    """(sequence, number in the sequence's tokens, position) of each row of the call."""
    T, B, length = s["T"], s["B"], s["lengths"].long()
    row = torch.arange(T, device=DEV)
    if s["offsets"] is None:
        off = torch.arange(B + 1, device=DEV) * (T // B)
    else:
        off = s["offsets"].long()
    b = torch.searchsorted(off, row, right=True) - 1
    i = row - off[b]
    return b, i, length[b] - (off[b + 1] - off[b]) + i, off


def _turned(x, c, n, rot, pairs):
    """The first `rot` channels turned by their angles, as neighbours or as halves."""
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., : rot // 2], x[..., rot // 2: rot])
    u, w = a * c - b * n, b * c + a * n
    both = torch.stack([u, w], -1).flatten(-2) if pairs else torch.cat([u, w], -1)
    return torch.cat([both, x[..., rot:]], -1)


def _plain(s):
    op, page, D, H = s["op"], s["page"], s["D"], s["H"]
    b, i, p, off = _rows(s)
    at = s["table"].long()[b, p // page]
    if op == "append":
        c, n = s["cos"][p][:, None], s["sin"][p][:, None]
        q = _turned(s["q"], c, n, s["rot"], s["pairs"]).to(s["q"].dtype)
        flat, (o0, o1, o2, o3, _) = s["pages"].view(-1), _sections(page, D)
        head = (at[:, None] * H + torch.arange(H, device=DEV)) * _words(page, D)
        slot, word = (p % page)[:, None, None], torch.arange(D // 8, device=DEV)
        group = torch.arange(_groups(D), device=DEV) * page
        kw, kp = _encode(_turned(s["k"], c, n, s["rot"], s["pairs"]))
        vw, vp = _encode(s["v"].float())
        flat[head[..., None] + o0 + slot * (D // 8) + word] = kw
        flat[head[..., None] + o1 + slot // 4 * (D // 2) + word * 4 + slot % 4] = vw
        flat[head[..., None] + o2 + group + slot] = kp
        flat[head[..., None] + o3 + group + slot] = vp
        return (q,) + _read(s, at, p, torch.float16)
    if op == "values":
        return _read(s, at, p, _DT[s["out"]])
    return _plain_attend(s, b, i, off)


def _read(s, at, p, dtype):
    page, D, H = s["page"], s["D"], s["H"]
    flat, (o0, o1, o2, o3, _) = s["pages"].view(-1), _sections(page, D)
    head = ((at[:, None] * H + torch.arange(H, device=DEV)) * _words(page, D))[..., None]
    slot, word = (p % page)[:, None, None], torch.arange(D // 8, device=DEV)
    group = torch.arange(_groups(D), device=DEV) * page
    k = _decode(flat[head + o0 + slot * (D // 8) + word], flat[head + o2 + group + slot])
    v = _decode(flat[head + o1 + slot // 4 * (D // 2) + word * 4 + slot % 4], flat[head + o3 + group + slot])
    return k.to(dtype), v.to(dtype)


def _plain_attend(s, b, i, off):
    B, H, D, n, page = s["B"], s["H"], s["D"], s["n"], s["page"]
    G = s["Hq"] // H
    k, v = _cached(s["pages"][s["table"].long().clamp_min(0)], page, D)  # [B, pages, H, page, D]
    L = k.shape[1] * page
    k, v = (x.transpose(1, 2).reshape(B * H, L, D) for x in (k, v))
    q = s["q"].new_zeros((B, n, s["Hq"], D), dtype=torch.float32)
    q[b, i] = s["q"].float()
    q = q.view(B, n, H, G, D).permute(0, 2, 3, 1, 4).reshape(B * H, G * n, D)
    x = torch.matmul(q, k.transpose(1, 2).contiguous()).view(B, H * G, n, L) / math.sqrt(D)
    new = off[1:] - off[:-1]
    p = (s["lengths"].long() - new)[:, None] + torch.arange(n, device=DEV)
    j = torch.arange(L, device=DEV)
    seen = j <= p[..., None]
    if s["window"]:
        seen &= (j > p[..., None] - s["window"]) | (j < s["sinks"])
    x = torch.where(seen[:, None], x, -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True).clamp_min(-3e38))
    o = torch.matmul(x.view(B * H, G * n, L), v).view(B, H * G, n, D) / x.sum(-1, keepdim=True).clamp_min(1e-30)
    return o.permute(0, 2, 1, 3)[b, i].to(s["q"].dtype)


# ---- what a pass cannot do without ------------------------------------------------


def _seen(case, new, length):
    """(visible cached positions, visible (query, position) pairs) of one sequence."""
    w, k = case["window"], case["sinks"]
    first = length - new
    if not w:
        return length, new * first + new * (new + 1) // 2
    pairs = 0
    for p in range(first, length):
        lo = max(0, p - w + 1)
        pairs += p + 1 - lo + min(k, lo)
    lo = max(0, first - w + 1)
    return length - lo + min(k, lo), pairs


def work(case):
    D, H = case["D"], case["H"]
    size = {"f32": 4, "f16": 2, "bf16": 2}
    new, length = _plan(case)
    T, held = sum(new), H * (D + 8 * _groups(D))  # bytes of one cached position
    if case["op"] == "append":
        inout = T * D * size[case["x"]] * (2 * case["Hq"] + 2 * H) + T * held
        read_back = T * held + T * H * D * 2 * 2
        return {"bytes": inout + 4 * T * case["rot"] + read_back, "flops": T * D * (6 * case["Hq"] + 14 * H)}
    if case["op"] == "values":
        return {"bytes": T * held + T * H * D * 2 * size[case["out"]], "flops": 4 * T * H * D}
    seen = [_seen(case, m, l) for m, l in zip(new, length)]
    return {"bytes": sum(x for x, _ in seen) * held + 2 * T * case["Hq"] * D * size[case["x"]],
            "flops": 4 * D * case["Hq"] * sum(x for _, x in seen)}


# ---- the definitions in 64 bits ----------------------------------------------------


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    page, D, H = case["page"], case["D"], case["H"]
    new, length = _plan(case)
    first, ks, vs, qs = 0, [], [], []
    for b in range(case["B"]):
        at = torch.arange(length[b] - new[b], length[b], device=DEV)
        rows = slice(first, first + new[b])
        first += new[b]
        if op == "append":
            qs.append(_exact_turn(s["q"][rows].double(), s["cos"][at].double(), s["sin"][at].double(), case))
            ks.append(_exact_quant(_exact_turn(s["k"][rows].double(), s["cos"][at].double(), s["sin"][at].double(), case)))
            vs.append(_exact_quant(s["v"][rows].double()))
            continue
        rows_of = torch.arange(length[b], device=DEV) if op == "attend" else at
        k, v = _exact_cached(s["pages"], s["table"][b], rows_of, page, D)
        if op == "values":
            ks.append(k)
            vs.append(v)
            continue
        q = s["q"][rows].double()
        o = torch.zeros_like(q)
        j, p = rows_of[None], at[:, None]
        hidden = j > p
        if case["window"]:
            hidden |= (j <= p - case["window"]) & (j >= case["sinks"])
        for h in range(case["Hq"]):
            kv = h // (case["Hq"] // H)
            x = q[:, h] @ k[:, kv].t().contiguous() * D ** -0.5
            o[:, h] = torch.softmax(x.masked_fill(hidden, -math.inf), -1) @ v[:, kv].contiguous()
        qs.append(o)
    if op == "attend":
        return torch.cat(qs)
    return ((torch.cat(qs),) if op == "append" else ()) + (torch.cat(ks), torch.cat(vs))


def _exact_turn(x, c, n, case):
    """Each pair of channels as a complex number times that of its angle."""
    rot, D = case["rot"], case["D"]
    first = torch.arange(0, rot, 2, device=DEV) if case["pairs"] else torch.arange(rot // 2, device=DEV)
    second = first + (1 if case["pairs"] else rot // 2)
    y = torch.complex(x[..., first], x[..., second]) * torch.complex(c, n)[:, None]
    x = x.clone()
    x[..., first], x[..., second] = y.real, y.imag
    return x


def _exact_quant(x):
    out = torch.empty_like(x)
    width = min(x.shape[-1], 128)
    for c in range(0, x.shape[-1], width):
        part = x[..., c: c + width]
        lo, hi = part.amin(-1, keepdim=True).clamp(max=0), part.amax(-1, keepdim=True).clamp(min=0)
        m, e = torch.frexp((hi - lo) / 15)
        scale = torch.ldexp(torch.ceil(m * 128) / 128, e).clamp_min(1e-300)
        zero = torch.round(-lo / scale)
        out[..., c: c + width] = ((torch.round(part / scale) + zero).clamp(0, 15) - zero) * scale
    return out


def _exact_cached(pages, table, at, page, D):
    """Keys and values [positions, H, D] of one sequence, a channel at a time."""
    H, gd, c8 = pages.shape[1], _groups(D), D // 8
    flat, slot = pages.view(-1), (at % page)[:, None]
    head = (table[at // page].long()[:, None] * H + torch.arange(H, device=DEV)) * pages.shape[2]
    out = []
    for keys in (True, False):
        x = torch.empty((len(at), H, D), dtype=torch.float64, device=DEV)
        for d in range(D):
            w = slot * c8 + d // 8 if keys else page * c8 + (slot // 4 * c8 + d // 8) * 4 + slot % 4
            g = 2 * page * c8 + (0 if keys else gd * page) + d // 128 * page + slot
            code, group = flat[head + w] >> (4 * (d % 8)) & 15, flat[head + g]
            scale = (group >> 16 << 16).view(torch.float32).double()
            x[:, :, d] = (code - (group & 15)).double() * scale
        out.append(x)
    return out

"""What is measured of the block-scaled 8-bit float linear layer and of its expert form.

Five operators, in the order in which a layer of experts uses them:

  route      scores, top-k choice and weights of the experts of each token, and the row plan
             (which rows of the experts' products belong to which token and expert);
  quantize   8-bit float codes (e4m3) with a binary32 scale for each 128 inputs of a token,
             or for each 128 x 128 block of a weight matrix;
  gemm       the product of the two, Y = X W;
  experts    the same product where each run of rows has its own expert's weights;
  combine    the weighted sum of a token's expert rows.

Layer widths are those of the repository's workloads (4096, 11008, 12288); an expert is 1376
= 11008 / 8 wide, so the inner width of its second product is no multiple of 128.
`own` chooses between the plain torch forms below and the framework's entry points.
"""
import math

import torch

own = False

BLOCK = 128
TOP = 448.0  # largest finite e4m3 value
DEV = "cuda"
_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # activations of eight requests entering a product, one decode step: latency
        {"name": "quantize_decode", "op": "quantize", "M": 8, "K": 4096, "x": "bf16"},
        # activations of a long prompt entering the down projection: bandwidth
        {"name": "quantize_prefill", "op": "quantize", "M": 4096, "K": 11008, "x": "bf16"},
        # one projection of a checkpoint prepared at load time
        {"name": "quantize_weight", "op": "weight", "E": 1, "K": 4096, "N": 11008, "x": "f32"},
        # one request's next token through the fused QKV projection
        {"name": "gemm_one_row", "op": "gemm", "M": 1, "K": 4096, "N": 12288, "out": "f16"},
        # a step of continuous batching: a ragged number of tokens, a partial last block of K and N
        {"name": "gemm_ragged", "op": "gemm", "M": 77, "K": 5520, "N": 4100, "out": "f32"},
        # a prompt of 4096 tokens through the up projection
        {"name": "gemm_prefill", "op": "gemm", "M": 4096, "K": 4096, "N": 11008, "out": "bf16"},
        # routing of one decode step: sigmoid scores, balance bias, groups of experts
        {"name": "route_decode", "op": "route", "T": 16, "E": 64, "k": 6, "score": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "renorm": True, "logits": "f32", "pad": 0},
        # routing of a long, padded prompt batch with softmax scores over many experts
        {"name": "route_prefill", "op": "route", "T": 16384, "E": 256, "k": 8, "score": "softmax", "bias": False,
         "groups": 1, "top_groups": 1, "renorm": True, "logits": "f32", "pad": 37},
        # the experts' gate and up product of a decode step: few rows for each expert, weights streamed
        {"name": "experts_decode", "op": "experts", "T": 16, "k": 6, "E": 64, "K": 4096, "N": 2752, "gather": True,
         "out": "bf16"},
        # the experts' down product of a prompt: hundreds of rows for each expert
        {"name": "experts_prefill", "op": "experts", "T": 4096, "k": 6, "E": 64, "K": 1376, "N": 4096,
         "gather": False, "out": "bf16"},
        # the joining of the experts' rows of a decode step and of a prompt
        {"name": "combine_decode", "op": "combine", "T": 16, "k": 6, "E": 64, "N": 4096, "rows": "bf16"},
        {"name": "combine_prefill", "op": "combine", "T": 4096, "k": 6, "E": 64, "N": 4096, "rows": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _width(rng, lo, hi):
    return min(hi, max(lo, 16 * round(_log(rng, lo, hi) / 16)))


def draw(rng):
    op = rng.choice(["quantize", "weight", "gemm", "gemm", "route", "experts", "experts", "combine"])
    if op == "quantize":
        K = _width(rng, 64, 16384)
        return {"op": op, "M": _log(rng, 1, min(8192, 45000000 // K)), "K": K, "x": rng.choice(list(_DT))}
    if op == "weight":
        E, K = rng.choice([1, 1, 4]), _width(rng, 64, 11008)
        return {"op": op, "E": E, "K": K, "N": _log(rng, 16, min(12288, 45000000 // (E * K))), "x": rng.choice(list(_DT))}
    if op == "gemm":
        K, N = _width(rng, 64, 11008), _log(rng, 64, 12288)
        return {"op": op, "M": _log(rng, 1, min(8192, 184000000000 // (K * N))), "K": K, "N": N, "out": rng.choice(list(_DT))}
    E = rng.choice([8, 16, 60, 64, 128, 256])
    k = rng.choice([x for x in (1, 2, 4, 6, 8) if x <= E // 2])
    if op == "route":
        groups = rng.choice([g for g in (1, 1, 4, 8) if E % g == 0 and E // g >= 4])
        top_groups = rng.randint(max(1, groups // 2), groups)
        score = rng.choice(["softmax", "sigmoid"])
        T = _log(rng, 1, 16384)
        return {"op": op, "T": T, "E": E, "k": min(k, top_groups * (E // groups)), "score": score,
                "bias": rng.random() < 0.5, "groups": groups, "top_groups": top_groups, "renorm": rng.random() < 0.7,
                "logits": rng.choice(list(_DT)), "pad": min(T - 1, rng.choice([0, 0, 1, 9]))}
    if op == "experts":
        K, N = _width(rng, 128, 4096), _width(rng, 64, 4096)
        E = min(E, max(8, 700000000 // (K * N)))
        k = min(k, E // 2)
        return {"op": op, "T": _log(rng, 1, min(4096, 130000000000 // (k * K * N))), "k": k, "E": E, "K": K, "N": N,
                "gather": rng.random() < 0.5, "out": rng.choice(list(_DT))}
    return {"op": op, "T": _log(rng, 1, 4096), "k": min(k, 6), "E": E, "N": _width(rng, 64, 4096), "rows": rng.choice(list(_DT))}


# ---- inputs ------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _acts(g, M, K):
    """Activations with a hundredth of the channels fifty times larger, as ahead of a projection."""
    x = torch.randn((M, K), generator=g, device=DEV)
    x[:, torch.randperm(K, generator=g, device=DEV)[: max(1, K // 100)]] *= 50.0
    return x


def _codes_of_rows(x):
    M, K = x.shape
    G = -(-K // BLOCK)
    b = torch.nn.functional.pad(x, (0, G * BLOCK - K)).view(M, G, BLOCK)
    s = b.abs().amax(-1) / TOP
    q = torch.where(s[..., None] > 0, b / s[..., None], 0.0).clamp(-TOP, TOP)
    return q.view(M, G * BLOCK)[:, :K].contiguous().to(torch.float8_e4m3fn), s


def _codes_of_weights(w):
    """[E][K][N] weights -> codes [E][N][K] and scales [E][ceil(N/128)][ceil(K/128)]."""
    E, K, N = w.shape
    G, B = -(-K // BLOCK), -(-N // BLOCK)
    b = torch.nn.functional.pad(w.transpose(1, 2), (0, G * BLOCK - K, 0, B * BLOCK - N)).reshape(E, B, BLOCK, G, BLOCK)
    s = b.abs().amax((2, 4)) / TOP
    t = s[:, :, None, :, None]
    q = torch.where(t > 0, b / t, 0.0).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
    return q.reshape(E, B * BLOCK, G * BLOCK)[:, :N, :K].contiguous(), s


def _weights_in_hand(g, E, K, N):
    """Prepared weights, made an expert at a time to bound the memory."""
    qs = [_codes_of_weights((torch.randn((1, K, N), generator=g, device=DEV) * 0.02)) for _ in range(E)]
    return torch.cat([q.view(torch.uint8) for q, _ in qs]).view(torch.float8_e4m3fn), torch.cat([s for _, s in qs])


def _choices(g, T, k, E):
    """k different experts of each token, all experts alike."""
    return torch.rand((T, E), generator=g, device=DEV).argsort(1)[:, :k].to(torch.int32).contiguous()


def _plan(expert, E):
    """(offsets [E+1], row_token [T k], slot [T, k]) of a choice: rows sorted by expert, tokens in order;
    an entry that is no expert has slot -1, rows behind the last expert's have token -1."""
    T, k = expert.shape
    flat = expert.reshape(-1).long()
    flat = torch.where((flat >= 0) & (flat < E), flat, E)
    counts = (flat[:, None] == torch.arange(E, device=flat.device)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    order = torch.argsort(flat, stable=True)
    at = torch.arange(T * k, device=flat.device)
    row_token = torch.where(at < offsets[-1], order // k, -1)
    slot = torch.empty_like(flat)
    slot[order] = at
    slot = torch.where(flat < E, slot, -1)
    return offsets.int(), row_token.int(), slot.view(T, k).int()


def prepare(case, seed):
    g, op, s = _gen(seed), case["op"], dict(case)
    if op == "quantize":
        s["data"] = _acts(g, case["M"], case["K"]).to(_DT[case["x"]])
    elif op == "weight":
        s["data"] = (torch.randn((case["E"], case["K"], case["N"]), generator=g, device=DEV) * 0.02).to(_DT[case["x"]])
    elif op == "gemm":
        s["xq"], s["xs"] = _codes_of_rows(_acts(g, case["M"], case["K"]))
        wq, ws = _weights_in_hand(g, 1, case["K"], case["N"])
        s["wq"], s["ws"] = wq[0], ws[0]
    elif op == "route":
        x = torch.randn((case["T"], case["E"]), generator=g, device=DEV) * 1.5
        if case["pad"]:
            x[-case["pad"]:] = -math.inf  # padding tokens choose no expert
        s["data"] = x.to(_DT[case["logits"]])
        s["b"] = torch.randn(case["E"], generator=g, device=DEV) * 0.05 if case["bias"] else None
    elif op == "experts":
        T, k, E = case["T"], case["k"], case["E"]
        s["offsets"], token, _ = _plan(_choices(g, T, k, E), E)
        s["xq"], s["xs"] = _codes_of_rows(_acts(g, T if case["gather"] else T * k, case["K"]))
        s["token"] = token if case["gather"] else None
        s["wq"], s["ws"] = _weights_in_hand(g, E, case["K"], case["N"])
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    else:
        T, k = case["T"], case["k"]
        s["slot"] = _plan(_choices(g, T, k, case["E"]), case["E"])[2]
        s["data"] = torch.randn((T * k, case["N"]), generator=g, device=DEV).to(_DT[case["rows"]])
        w = torch.rand((T, k), generator=g, device=DEV) + 0.05
        s["weight"] = w / w.sum(1, keepdim=True)
    return s


# ---- one pass ------------------------------------------------------------------


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import bit_quantized_gemm_int8_amd as qg
    op = s["op"]
    if op == "quantize":
        return qg.quantize_f8_g128(s["data"])
    if op == "weight":
        return qg.quantize_weight_f8_b128(s["data"])
    if op == "gemm":
        return qg.gemm_f8_b128(s["xq"], s["xs"], s["wq"], s["ws"], out_dtype=_DT[s["out"]])
    if op == "route":
        expert, weight = qg.route_experts(s["data"], s["k"], bias=s["b"], score=s["score"], groups=s["groups"],
                                          top_groups=s["top_groups"], renormalize=s["renorm"], scale=2.5)
        return (expert, weight) + tuple(qg.plan_experts(expert, s["E"]))
    if op == "experts":
        return qg.gemm_f8_b128_experts(s["xq"], s["xs"], s["wq"], s["ws"], s["offsets"], row_token=s["token"],
                                       out_dtype=_DT[s["out"]])
    return qg.combine_experts(s["data"], s["slot"], s["weight"])


def _values_of_rows(q, s):
    return q.float() * s.repeat_interleave(BLOCK, 1)[:, : q.shape[1]]


def _values_of_weights(q, s):
    return q.float() * s.repeat_interleave(BLOCK, -2)[..., : q.shape[-2], :].repeat_interleave(BLOCK, -1)[..., : q.shape[-1]]


def _plain(s):
    op = s["op"]
    if op == "quantize":
        return _codes_of_rows(s["data"].float())
    if op == "weight":
        return _codes_of_weights(s["data"].float())
    if op == "gemm":
        return (_values_of_rows(s["xq"], s["xs"]) @ _values_of_weights(s["wq"], s["ws"]).t()).to(_DT[s["out"]])
    if op == "route":
        expert, weight = _plain_route(s)
        return (expert, weight) + _plan(expert, s["E"])
    if op == "experts":
        x, off = _values_of_rows(s["xq"], s["xs"]), s["offsets"].long()
        if s["token"] is not None:
            x = x[s["token"].long()]
        row = torch.arange(x.shape[0], device=x.device)
        e = torch.searchsorted(off, row, right=True) - 1
        at = row - off[e]
        padded = x.new_zeros((s["E"], s["most"], s["K"]))
        padded[e, at] = x
        return torch.bmm(padded, _values_of_weights(s["wq"], s["ws"]).transpose(1, 2).contiguous())[e, at].to(_DT[s["out"]])
    rows = s["data"].float()[s["slot"].long()]  # every slot is a row here
    return (rows * s["weight"][..., None]).sum(1).to(s["data"].dtype)


def _plain_route(s):
    """Scores and the choice in 64 bits, since values next to a border decide: the largest of score + bias, ties to
    the lowest expert, within the groups whose two largest have the largest sum; a logit of -inf is no choice."""
    x = s["data"].double()
    E, groups, k = s["E"], s["groups"], s["k"]
    off = x == -math.inf
    if s["score"] == "softmax":
        p = torch.exp(x - x.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-x))
    p = torch.where(off, 0.0, p)
    c = p if s["b"] is None else p + s["b"].double()
    c = torch.where(off, -math.inf, c)
    if groups > 1:
        two = c.view(-1, groups, E // groups).sort(2, descending=True).values[..., :2]
        two = torch.where(two[..., 0] == -math.inf, -math.inf, two[..., 0] + torch.where(two[..., 1] == -math.inf, 0.0, two[..., 1]))
        rank = two.sort(dim=1, descending=True, stable=True).indices.argsort(1)
        c = torch.where((rank < s["top_groups"]).repeat_interleave(E // groups, 1), c, -math.inf)
    best = c.sort(dim=1, descending=True, stable=True)
    value, expert = best.values[:, :k], best.indices[:, :k]
    weight = torch.where(value == -math.inf, 0.0, p.gather(1, expert))
    if s["renorm"]:
        total = weight.sum(1, keepdim=True)
        weight = torch.where(total > 0, weight / total, 0.0)
    return torch.where(value == -math.inf, -1, expert).int(), (weight * 2.5).float()


# ---- what a pass cannot do without ------------------------------------------------


def work(case):
    op = case["op"]
    size = {"f32": 4, "f16": 2, "bf16": 2}
    if op == "quantize":
        n = case["M"] * case["K"]
        return {"bytes": n * (size[case["x"]] + 1) + 4 * case["M"] * -(-case["K"] // BLOCK), "flops": 3 * n}
    if op == "weight":
        n = case["E"] * case["K"] * case["N"]
        return {"bytes": n * (size[case["x"]] + 1) + 4 * case["E"] * -(-case["K"] // BLOCK) * -(-case["N"] // BLOCK), "flops": 3 * n}
    if op == "gemm":
        M, K, N = case["M"], case["K"], case["N"]
        G = -(-K // BLOCK)
        return {"bytes": M * K + 4 * M * G + N * K + 4 * G * -(-N // BLOCK) + M * N * size[case["out"]], "flops": 2 * M * N * K}
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * size[case["logits"]] + 16 * T * k + 4 * (E + 1) + 4 * E * case["bias"], "flops": T * E * (8 + k)}
    if op == "experts":
        T, k, E, K, N = (case[n] for n in ("T", "k", "E", "K", "N"))
        G, R = -(-K // BLOCK), T * k
        used = E * (1 - (1 - k / E) ** T)  # experts that some token chose
        rows = T if case["gather"] else R
        return {"bytes": int(rows * (K + 4 * G) + used * (N * K + 4 * G * -(-N // BLOCK)) + 4 * (E + 1 + R * case["gather"])
                             + R * N * size[case["out"]]), "flops": 2 * R * N * K}
    n = case["T"] * case["N"]
    return {"bytes": n * (case["k"] + 1) * size[case["rows"]] + 8 * case["T"] * case["k"], "flops": 2 * n * case["k"]}


# ---- the definitions in 64 bits ----------------------------------------------------


def _grid(q):
    """The nearest e4m3 value (3 bits behind the leading one, exponents from -6), halves to even."""
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -9))).clamp_min(-6.0) - 3.0)
    return (torch.round(q / step) * step).clamp(-TOP, TOP)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("quantize", "weight"):
        x = s["data"].double()
        t = x if op == "quantize" else x.transpose(1, 2).contiguous()
        K = t.shape[-1]
        tall = 1 if op == "quantize" else BLOCK
        t = t.view(1, -1, K) if op == "quantize" else t
        codes, scales = torch.zeros_like(t), []
        for k0 in range(0, K, BLOCK):
            part = t[:, :, k0:k0 + BLOCK]
            top = part.abs().amax(2)
            if tall > 1:
                top = torch.stack([c.amax(1) for c in top.split(tall, 1)], 1)
            scale = top / TOP
            each = scale.repeat_interleave(tall, 1)[:, : t.shape[1], None]
            codes[:, :, k0:k0 + BLOCK] = torch.where(each > 0, _grid(part / each.clamp_min(1e-300)), 0.0)
            scales.append(scale)
        scales = torch.stack(scales, 2)
        return (codes[0], scales[0]) if op == "quantize" else (codes, scales)
    if op == "gemm":
        return _sum_of_blocks(s["xq"], s["xs"], s["wq"], s["ws"])
    if op == "route":
        return _exact_route(s)
    if op == "experts":
        off = s["offsets"].tolist()
        parts = []
        for e in range(case["E"]):
            if off[e] == off[e + 1]:
                continue
            rows = torch.arange(off[e], off[e + 1], device=DEV)
            rows = rows if s["token"] is None else s["token"][rows].long()
            parts.append(_sum_of_blocks(s["xq"].view(torch.uint8)[rows].view(torch.float8_e4m3fn), s["xs"][rows], s["wq"][e], s["ws"][e]))
        return torch.cat(parts)
    rows, out = s["data"].double(), 0.0
    for j in range(case["k"]):
        out = out + rows.index_select(0, s["slot"][:, j].long()) * s["weight"][:, j, None].double()
    return out


def _sum_of_blocks(xq, xs, wq, ws):
    y = torch.zeros((xq.shape[0], wq.shape[0]), dtype=torch.float64, device=DEV)
    for g in range(xs.shape[1]):
        at = slice(g * BLOCK, min((g + 1) * BLOCK, xq.shape[1]))
        part = xq[:, at].double() @ wq[:, at].double().t().contiguous()
        y += part * xs[:, g, None].double() * ws[:, g].double().repeat_interleave(BLOCK)[: wq.shape[0]]
    return y


def _exact_route(s):
    """Choices one at a time: the first largest of what is left."""
    x = s["data"].double()
    T, E = x.shape
    open_ = torch.isfinite(x)
    p = torch.softmax(x.masked_fill(~open_, -1e4), 1) if s["score"] == "softmax" else torch.sigmoid(x)
    left = (p + (0.0 if s["b"] is None else s["b"].double())).masked_fill(~open_, -math.inf)
    if s["groups"] > 1:
        by = left.view(T, s["groups"], -1)
        value = by.topk(2, dim=2).values.clamp_min(-1e9).sum(2)
        keep = torch.zeros_like(value, dtype=torch.bool)
        for _ in range(s["top_groups"]):
            keep.scatter_(1, value.masked_fill(keep, -math.inf).argmax(1, keepdim=True), True)
        left = by.masked_fill(~keep[..., None], -math.inf).view(T, E).clone()
    chosen, weights = [], []
    for _ in range(s["k"]):
        best, at = left.max(1)
        none = best == -math.inf
        chosen.append(torch.where(none, -1, at))
        weights.append(torch.where(none, 0.0, p.gather(1, at[:, None])[:, 0]))
        left.scatter_(1, at[:, None], -math.inf)
    weight = torch.stack(weights, 1)
    if s["renorm"]:
        weight = weight / weight.sum(1, keepdim=True).clamp_min(1e-300)
    return torch.stack(chosen, 1).int(), weight * 2.5, None, None, None

"""Expert routing, row plans and the weighted sum against the oracle, and the
whole routed layer as a program runs it: eager, on another stream, and captured
and replayed."""
import numpy as np
import pytest
import torch

import bit_quantized_gemm_int8_amd as qg
from oracle import experts as oe
from oracle import f8
from tests.gpu_util import out_f64, to_dev

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def check_route(lg, k, **kw):
    """Experts equal; weights within 2^-20 relative: the GPU's binary64 scores
    round to binary32 once (2^-24), times a binary32 `scale`."""
    score = kw.pop("score", "softmax")
    bias = kw.pop("bias", None)
    e, w = qg.route_experts(lg, k, bias=None if bias is None else to_dev(bias), score=score, **kw)
    eo, wo = oe.route_experts(lg.float().cpu().numpy(), k, bias=bias, sigmoid=score == "sigmoid", **kw)
    assert np.array_equal(e.cpu().numpy(), eo)
    assert np.all(np.abs(out_f64(w) - wo) <= 2.0 ** -20 * np.abs(wo) + 2.0 ** -149)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,top", [
    (1, 1, 1, 1, 1), (3, 8, 2, 1, 1), (5, 60, 4, 4, 2), (33, 64, 6, 8, 3), (9, 65, 65 // 2, 1, 1), (17, 128, 8, 1, 1),
    (12, 256, 8, 8, 4), (4, 256, 64, 64, 32), (6, 300, 10, 3, 1), (5, 512, 16, 16, 5), (3, 1024, 64, 64, 64), (2, 1000, 7, 8, 8)])
def test_route(T, E, k, groups, top, score, dt):
    rng = np.random.default_rng(T * E + k)
    lg = torch.from_numpy((rng.standard_normal((T, E)) * 2).astype(np.float32)).to(DEV).to(DT[dt])
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    check_route(lg, k, score=score, groups=groups, top_groups=top, renormalize=False, scale=1.0)
    check_route(lg, k, score=score, groups=groups, top_groups=top, renormalize=True, scale=2.5, bias=bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top", [(16, 1, 1), (64, 8, 4), (200, 4, 3), (512, 8, 2)])
def test_route_masked_and_tied(E, groups, top, score):
    """Closed experts (-inf, NaN, a bias of -inf), rows with fewer open experts
    than choices or none, equal logits, the type's ends, far apart logits."""
    rng = np.random.default_rng(E)
    lg = np.round(rng.standard_normal((16, E)) * 2).astype(np.float32) / 2     # many ties
    lg[1] = -np.inf
    lg[2, 3:] = -np.inf
    lg[3] = np.nan
    lg[4, ::2] = np.nan
    lg[5] = 0
    lg[6] = -3.4028234663852886e38
    lg[7] = 3.4028234663852886e38
    lg[8, 5] = np.inf
    lg[9] = rng.standard_normal(E) * 1e4
    lg[10, : E // 2] = -np.inf
    lg[11] = rng.standard_normal(E) * 1e-6
    lg[12] = 60 + rng.standard_normal(E)                                        # sigmoid is 1 here
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    bias[0], bias[E - 1] = -np.inf, np.nan
    k = min(6, top * (E // groups))
    for b in (None, bias):
        for renorm in (False, True):
            check_route(to_dev(lg), k, score=score, groups=groups, top_groups=top, renormalize=renorm, scale=1.5, bias=b)


def near_ties(E, seed):
    """Scores + bias that differ by a binary32 rounding or less: the bias is
    the difference of two scores, rounded."""
    rng = np.random.default_rng(seed)
    lg = rng.standard_normal((64, E)).astype(np.float32)
    p = 1 / (1 + np.exp(-lg[0].astype(np.float64)))
    bias = (p.mean() - p).astype(np.float32)
    lg[1:] = lg[0]
    lg[32:] = np.nextafter(lg[0], np.float32(9))
    return lg, bias


@pytest.mark.parametrize("groups,top", [(1, 1), (8, 3)])
@pytest.mark.parametrize("E", [16, 64, 256])
def test_route_decides_near_ties_in_binary64(E, groups, top):
    lg, bias = near_ties(E, E)
    check_route(to_dev(lg), 4, score="sigmoid", groups=groups, top_groups=top, bias=bias)
    few = np.unique(lg[:, :1] + np.zeros((1, E), np.float32), axis=0)
    check_route(to_dev(np.ascontiguousarray(few)), 4, score="softmax", groups=groups, top_groups=top, bias=bias)


@pytest.mark.parametrize("T,k,E", [(0, 2, 4), (1, 1, 1), (1, 8, 8), (16, 6, 64), (37, 7, 33), (511, 8, 256), (512, 1, 1024),
                                   (3000, 8, 60), (70, 64, 500), (1025, 4, 1024), (513, 8, 7), (2049, 2, 1023),
                                   (20000, 7, 256), (16385, 9, 1024)])
def test_plan(T, k, E):
    rng = np.random.default_rng(T + k + E)
    for kind in range(3):
        e = rng.integers(-1 if kind else 0, E + (1 if kind else 0), (T, k)).astype(np.int32)
        if kind == 2:
            e[:] = E // 2                      # the same expert over and over
            e[::5] = -7
        off, tok, slot = qg.plan_experts(to_dev(e), E)
        oo, to, so = oe.plan_experts(e, E)
        assert np.array_equal(off.cpu().numpy(), oo)
        assert np.array_equal(tok.cpu().numpy(), to)
        assert np.array_equal(slot.cpu().numpy(), so)


def test_plan_of_a_slice():
    """Choices that start off a 16-byte boundary."""
    e = torch.randint(0, 9, (50, 3), dtype=torch.int32, device=DEV)
    part = e[3:]
    oo, to, so = oe.plan_experts(part.cpu().numpy(), 9)
    off, tok, slot = qg.plan_experts(part, 9)
    assert np.array_equal(off.cpu().numpy(), oo) and np.array_equal(tok.cpu().numpy(), to) and np.array_equal(slot.cpu().numpy(), so)


@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("T,k,R,N", [(1, 1, 1, 1), (5, 2, 9, 40), (7, 6, 42, 131), (3, 64, 20, 8), (40, 8, 320, 4096), (2, 3, 0, 16)])
def test_combine(T, k, R, N, dt, out):
    rng = np.random.default_rng(T + k + R + N)
    rows = torch.from_numpy(rng.standard_normal((R, N)).astype(np.float32)).to(DT[dt])
    slot = rng.integers(-1, R + 2, (T, k)).astype(np.int32)
    weight = rng.standard_normal((T, k)).astype(np.float32)
    y = qg.combine_experts(rows.to(DEV), to_dev(slot), to_dev(weight), out_dtype=DT[out])
    ye, B = oe.combine_experts(rows.float().numpy(), slot, weight)
    # k binary32 roundings of sums no larger than B, one of the output
    bound = HALF_STEP[out] * np.abs(ye) + k * 2.0 ** -24 * B * (1 + HALF_STEP[out]) + 2.0 ** -25
    assert np.all(np.abs(out_f64(y) - ye) <= bound)


def test_combine_of_slices():
    """Rows and outputs that start off a 16-byte boundary."""
    rows = torch.randn((9, 20), device=DEV).bfloat16()[1:]
    slot = torch.arange(8, dtype=torch.int32, device=DEV).view(4, 2)
    w = torch.ones((4, 2), device=DEV)
    out = torch.zeros((5, 20), dtype=torch.bfloat16, device=DEV)
    qg.combine_experts(rows, slot, w, out=out[1:])
    want = (rows.float()[0::2] + rows.float()[1::2]).bfloat16()
    assert torch.equal(out[1:], want) and not out[0].any()


# ---- the layer ------------------------------------------------------------------

class Layer:
    """A routed feed-forward layer as a program would hold it: router logits
    given, gate and up product, silu, down product, weighted sum."""

    def __init__(self, T, k, E, H, F, seed, groups=1, top=1):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.x = torch.randn((T, H), generator=g, device=DEV).bfloat16()
        self.logits = torch.randn((T, E), generator=g, device=DEV)
        self.logits[-1] = -float("inf")                                     # a padding token
        self.bias = torch.randn((E,), generator=g, device=DEV) * 0.05
        self.up = qg.quantize_weight_f8_b128(torch.randn((E, H, 2 * F), generator=g, device=DEV) * 0.05)
        self.down = qg.quantize_weight_f8_b128(torch.randn((E, F, H), generator=g, device=DEV) * 0.05)
        self.T, self.k, self.E, self.H, self.F, self.groups, self.top = T, k, E, H, F, groups, top
        # rows of no run stay as they are here: zeros, as the next step reads them
        self.h = torch.zeros((T * k, 2 * F), dtype=torch.bfloat16, device=DEV)
        self.y = torch.zeros((T * k, H), dtype=torch.bfloat16, device=DEV)
        self.out = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)

    def step(self):
        expert, weight = qg.route_experts(self.logits, self.k, bias=self.bias, score="sigmoid", groups=self.groups, top_groups=self.top)
        offsets, token, slot = qg.plan_experts(expert, self.E)
        xq, xs = qg.quantize_f8_g128(self.x)
        qg.gemm_f8_b128_experts(xq, xs, *self.up, offsets, row_token=token, out=self.h)
        gate, up = self.h.float().chunk(2, 1)
        a = (torch.nn.functional.silu(gate) * up).bfloat16()
        aq, as_ = qg.quantize_f8_g128(a)
        qg.gemm_f8_b128_experts(aq, as_, *self.down, offsets, out=self.y)
        qg.combine_experts(self.y, slot, weight, out=self.out)
        return expert, weight, offsets, token, slot, xq, xs, a, aq, as_

    def check(self, r):
        """Every stage against the oracle of its own inputs."""
        expert, weight, offsets, token, slot, xq, xs, a, aq, as_ = (v.cpu() for v in r)
        eo, wo = oe.route_experts(self.logits.cpu().numpy(), self.k, bias=self.bias.cpu().numpy(), sigmoid=True,
                                  groups=self.groups, top_groups=self.top)
        assert np.array_equal(expert.numpy(), eo) and np.allclose(weight.numpy(), wo, rtol=2.0 ** -20)
        oo, to, so = oe.plan_experts(eo, self.E)
        assert np.array_equal(offsets.numpy(), oo) and np.array_equal(token.numpy(), to) and np.array_equal(slot.numpy(), so)
        assert so[-1].tolist() == [-1] * self.k
        qo, sc = f8.quantize_f8_g128(self.x.float().cpu().numpy())
        assert np.array_equal(xq.view(torch.uint8).numpy(), qo) and np.array_equal(xs.numpy(), sc)
        for e in range(self.E):
            rows = np.arange(oo[e], oo[e + 1])
            for q, s, (wq, ws), y, t in ((qo, sc, self.up, self.h, to[rows]),
                                         (aq.view(torch.uint8).numpy(), as_.numpy(), self.down, self.y, rows)):
                ye, B, D = f8.gemm_f8_b128(q[t], s[t], wq[e].view(torch.uint8).cpu().numpy(), ws[e].cpu().numpy())
                G = s.shape[1]
                bound = 2.0 ** -8 * np.abs(ye) + (128 + 2 * G + 12) * 2.0 ** -23 * B + 7 * 2.0 ** -13 * D
                assert np.all(np.abs(out_f64(y)[rows] - ye) <= bound * (1 + 2.0 ** -8))
        ye, B = oe.combine_experts(self.y.float().cpu().numpy(), so, weight.numpy())
        assert np.all(np.abs(out_f64(self.out) - ye) <= 2.0 ** -8 * np.abs(ye) + (self.k + 1) * 2.0 ** -24 * B)


@pytest.mark.parametrize("T,k,E,H,F,groups,top", [(1, 2, 4, 144, 80, 1, 1), (9, 3, 16, 272, 144, 4, 2), (150, 4, 8, 144, 176, 1, 1)])
def test_layer(T, k, E, H, F, groups, top):
    layer = Layer(T, k, E, H, F, seed=T, groups=groups, top=top)
    layer.check(layer.step())


def test_layer_on_another_stream():
    layer = Layer(20, 2, 8, 272, 144, seed=1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        r = layer.step()
    s.synchronize()
    layer.check(r)


@pytest.mark.parametrize("T", [4, 300])
def test_layer_captured_and_replayed(T):
    """Replays with other eager work between them; new inputs in place reach
    the next replay."""
    layer = Layer(T, 2, 8, 272, 144, seed=2)
    layer.step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = layer.step()
    want = None
    for i in range(4):
        layer.h.zero_(), layer.y.zero_(), layer.out.zero_()
        g.replay()
        torch.cuda.synchronize()
        if i in (0, 2):
            layer.check(r)
        if i == 0:
            want = layer.out.clone()
        elif i == 1:
            assert torch.equal(layer.out, want)
            layer.x.copy_(layer.x.flip(0))
            layer.logits[:-1] = layer.logits[:-1].flip(0)
        torch.randn((256, 256), device=DEV) @ torch.randn((256, 256), device=DEV)
        torch.cuda.synchronize()


def test_two_graphs_share_the_weights():
    """Two captured layers on the same weights, replayed in turn."""
    a = Layer(4, 2, 8, 272, 144, seed=3)
    b = Layer(4, 2, 8, 272, 144, seed=4)
    b.up, b.down = a.up, a.down
    graphs = []
    for l in (a, b):
        l.step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = l.step()
        graphs.append((l, g, r))
    for _ in range(2):
        for l, g, r in graphs:
            g.replay()
        torch.cuda.synchronize()
    for l, g, r in graphs:
        l.check(r)


def test_refused_operands():
    lg = torch.zeros((4, 12), device=DEV)
    for kw in (dict(k=13), dict(k=0), dict(k=2, groups=5), dict(k=2, groups=4, top_groups=5), dict(k=4, groups=4, top_groups=1)):
        with pytest.raises(RuntimeError):
            qg.route_experts(lg, **kw)
    with pytest.raises(ValueError):
        qg.route_experts(lg, 2, score="linear")
    with pytest.raises(ValueError):
        qg.route_experts(lg, 2, bias=torch.zeros(11, device=DEV))
    with pytest.raises(RuntimeError):
        qg.route_experts(torch.zeros((1, 1025), device=DEV), 2)
    e = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    with pytest.raises(TypeError):
        qg.plan_experts(e.long(), 4)
    with pytest.raises(RuntimeError):
        qg.plan_experts(e, 1025)
    with pytest.raises(ValueError):
        qg.combine_experts(torch.zeros((8, 16), device=DEV), e, torch.zeros((4, 3), device=DEV))
    with pytest.raises(TypeError):
        qg.combine_experts(torch.zeros((8, 16), device=DEV), e, torch.zeros((4, 2), device=DEV), out_dtype=torch.int32)

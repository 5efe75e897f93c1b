"""Routing weights to the last bit: scores in binary64, one rounding."""
import numpy as np
import pytest
import torch

import bit_quantized_gemm_int8_amd as qg
from oracle import experts as oe
from tests.gpu_util import out_f64, to_dev

pytestmark = pytest.mark.gpu

# Half a step of binary32, and what two binary64 computations may differ by:
# exponentials and sums over up to 1024 experts, (1024 + 8) 2^-53 < 2^-42, for
# numerator and denominator.
BOUND = 2.0 ** -24 + 2.0 ** -41


@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,top", [(40, 8, 2, 1, 1), (64, 64, 6, 8, 3), (37, 100, 4, 1, 1), (64, 256, 8, 1, 1),
                                              (33, 256, 32, 32, 16), (9, 1000, 7, 8, 8), (5, 1024, 64, 1, 1)])
def test_weights_are_binary64_scores_rounded_once(T, E, k, groups, top, score, renormalize):
    """Tokens that the binary32 choice decides and tokens that it leaves to
    binary64 (equal logits but for one), the scores spread, close and far down."""
    rng = np.random.default_rng(T + E + k)
    lg = (rng.standard_normal((T, E)) * rng.choice([0.1, 2.0, 8.0], (T, 1))).astype(np.float32)
    lg[1] = np.float32(-9.3)
    lg[1, E // 3] = 0
    lg[2] += 70
    lg[3, ::2] = -np.inf
    for bias in (None, (rng.standard_normal(E) * 0.1).astype(np.float32)):
        kw = dict(groups=groups, top_groups=top, renormalize=renormalize, scale=2.5)
        e, w = qg.route_experts(to_dev(lg), k, bias=None if bias is None else to_dev(bias), score=score, **kw)
        eo, wo = oe.route_experts(lg, k, bias=bias, sigmoid=score == "sigmoid", **kw)
        assert np.array_equal(e.cpu().numpy(), eo)
        off = np.abs(out_f64(w) - wo)
        bad = off > BOUND * wo + 2.0 ** -150
        assert not bad.any(), (np.argwhere(bad)[:4].tolist(), off[bad][:4].tolist(), wo[bad][:4].tolist())

"""Row plans of millions of choices, against a stable sort."""
import pytest
import torch

import bit_quantized_gemm_int8_amd as qg

pytestmark = pytest.mark.gpu
DEV = "cuda"


def choices(T, k, E, seed, kind):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    e = torch.randint(-1, E + 1, (T, k), generator=g, device=DEV, dtype=torch.int32)
    if kind == "skewed":                    # four of five choices go to one expert
        e[torch.rand((T, k), generator=g, device=DEV) < 0.8] = E // 2
    elif kind == "runs":                    # an expert's choices all in one place
        e = (torch.arange(T * k, device=DEV) * (E + 1) // (T * k)).int().view(T, k).contiguous()
    return e


def check(e, E):
    T, k = e.shape
    offsets, token, slot = qg.plan_experts(e, E)
    flat = e.reshape(-1).long()
    flat = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(flat, stable=True)
    ends = torch.searchsorted(flat[order], torch.arange(E + 1, device=DEV), right=False)
    assert torch.equal(offsets.long(), ends)
    rows = int(ends[-1])
    assert torch.equal(token[:rows].long(), order[:rows] // k) and torch.all(token[rows:] == -1)
    want = torch.full_like(flat, -1)
    want[order[:rows]] = torch.arange(rows, device=DEV)
    assert torch.equal(slot.reshape(-1).long(), want)


# one and several runs of 16384 choices for a workgroup, the last of them short,
# or none left for the last workgroups
@pytest.mark.parametrize("kind", ["even", "skewed", "runs"])
@pytest.mark.parametrize("T,k,E", [(2 ** 19, 8, 256), (2 ** 22 + 1, 1, 1024), (1100003, 4, 7), (1700000, 5, 300), (2 ** 20 + 3, 9, 1)])
def test_plan_of_millions(T, k, E, kind):
    check(choices(T, k, E, T % 1000 + k, kind), E)


def test_time_grows_with_the_choices():
    """Eight times the choices: eight times the time, with room for noise, and
    far from the 64 times of a quadratic cost."""
    def ms(T):
        e = choices(T, 8, 256, 1, "even")
        out = qg.plan_experts(e, 256)
        best = float("inf")
        for _ in range(3):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            qg.plan_experts(e, 256, out=out)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best
    short, long = ms(2 ** 19), ms(2 ** 22)
    print(f"plan of 2^22 choices {short:.3f} ms, of 2^25 {long:.3f} ms")
    assert long < 20 * short

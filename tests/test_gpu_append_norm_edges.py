"""lowbit_kv_append_norm far from ordinary magnitudes, against the fp64 oracle.

Tolerance: that of test_gpu_append_norm.py, which is relative to the result, and half a step of bf16's subnormal
numbers.  These have bf16's 7 bits behind 2^-126, so their step is 2^-133 whatever the value, and a result under 2^-126
is off by up to 2^-134; fp32's own (steps of 2^-149) leave 2^-150 in each product, a part in 2^16 of that."""
import numpy as np
import pytest

from oracle import paged
from test_gpu_append_norm import i32, lb  # noqa: F401  (lb is a fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def run(lb, x, w, eps):  # noqa: F811
    """q of T rows of one head, without rotation, and k with the same elements: what is stored of both."""
    T, _, D = x.shape
    kc = torch.zeros((-(-T // 16), 16, 1, D), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(x)
    lb.lowbit_kv_append_norm(x, x, x, w, w, eps, None, i32([0, T]), i32([T]), i32([range(kc.shape[0])]),
                             lb.lowbit_paged_cache(kc, kc.clone()), out)
    k = kc.view(-1, 1, D)[:T]
    assert torch.equal(out.view(torch.int16), k.view(torch.int16))
    return out


def check(lb, x, w, eps):  # noqa: F811
    want = paged.normalise(x.double().cpu().numpy(), w.cpu().numpy(), eps)
    got = run(lb, x, w, eps).float().cpu().double().numpy()
    room = (2.0 ** -16 + 2.0 ** -8) * 1.001 * np.abs(want) + 2.0 ** -134 * 1.001
    bad = ~(np.abs(got - want) <= room)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4])


SIZES = [(5, 64), (300, 128), (3, 256), (600, 128), (1200, 64), (2000, 256)]   # eight warps a token, four, two, one


def heads(T, D, seed=0):
    g = np.random.default_rng(seed)
    x, w = g.standard_normal((T, 1, D)), 1 + 0.4 * g.standard_normal(D)
    return torch.from_numpy(x).to(torch.bfloat16).cuda(), torch.from_numpy(w).float().cuda()


@pytest.mark.parametrize("T,D", SIZES)
@pytest.mark.parametrize("x_scale,w_scale", [(50, -100), (50, -110), (-45, 100), (-40, 110), (60 - 4, 60)])
def test_weights_far_from_one(lb, x_scale, w_scale, T, D):  # noqa: F811
    """The reciprocal root and the weight are in range, and so is the result; their product is not."""
    x, w = heads(T, D)
    check(lb, x * 2.0 ** x_scale, w * 2.0 ** w_scale, 0.0)


@pytest.mark.parametrize("T,D", SIZES)
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -149, 1e-38, 2.0 ** -95, 2.0 ** -89])
@pytest.mark.parametrize("scale", [-41, -46, -60, -64, -75, -100, -126])
def test_heads_whose_squares_leave_fp32(lb, scale, eps, T, D):  # noqa: F811
    """Elements are exact in bf16 down to 2^-133: those of a scale below 2^-120 are rounded to it before the oracle sees them."""
    x, w = heads(T, D, 1)
    x = x.float() * 2.0 ** scale
    if T > 2:
        x[1] *= 2.0 ** 30                     # an ordinary head beside a small one
    x = x.to(torch.bfloat16)
    check(lb, x, w, eps)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("e", [-60, -63, -70, -73, -75, -90, -120, -133])
def test_a_head_with_one_small_element(lb, e, D):  # noqa: F811
    x = torch.zeros((4, 1, D), device="cuda")
    x[0, 0, 5] = x[2, 0, D - 1] = 2.0 ** e
    x[1] = 1.0
    x[3, 0, 7], x[3, 0, 8] = 2.0 ** e, 3.0
    check(lb, x.to(torch.bfloat16), torch.ones(D, device="cuda"), 0.0)

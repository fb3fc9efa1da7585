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

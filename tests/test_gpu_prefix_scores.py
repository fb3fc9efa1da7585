"""lowbit_prefix_attention with large scores, against the fp64 oracle.

Tolerance, beside test_gpu_paged.py's of weights and output: a score is a sum of D exact products in fp32, and each
addition is off by 2^-23 of the partial sum at most (a tensor core may cut off instead of rounding), whose magnitude stays
under A = scale * max_j sum_d |q_d k_jd|; scaling it for the exponential adds two roundings, the exponential 2^-22.  So a
score is off by delta = (D + 2) 2^-23 A + 2^-22, a softmax weight by a factor of e^(2 delta) (its own score, and the sum's),
the output by (e^(2 delta) - 1) sum_j p_j |v_j|, and lse by delta and its own rounding, 2^-23 of it."""
import numpy as np
import pytest

from oracle import paged
from test_gpu_paged import lb  # noqa: F401  (a fixture)
from test_gpu_prefix import SHAPES, Shared

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def check(pr, out, lse):
    scale = pr.D ** -0.5
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(pr.B):
        n, kv = pr.new[b], pr.kv[b]
        if not n:
            continue
        k, v = (paged.gather(x, pr.table[b], kv, pr.page) for x in pr.kv64)
        rows = slice(pr.cu[b], pr.cu[b + 1])
        see = paged.visible(n, kv, True, 0)
        want, norm, spread = paged.attention(pr.q64[rows], k, v, see, scale)
        size = np.stack([np.abs(pr.q64[rows][:, h]) @ np.abs(k[:, h // (pr.Hq // pr.Hk)]).T for h in range(pr.Hq)], 1) * scale
        delta = (pr.D + 2) * 2.0 ** -23 * np.where(see[:, None], size, 0).max(-1) + 2.0 ** -22
        flat = kv * 2.0 ** -25 * np.abs(v).max() if pr.fp8 else 0.0
        room = 1.05 * (((2.0 ** -11 if pr.fp8 else 2.0 ** -8) + np.expm1(2 * delta))[..., None] * spread + flat
                       + 2.0 ** -8 * np.abs(want))
        assert (np.abs(out[rows] - want) <= room).all(), (b, float((np.abs(out[rows] - want) - room).max()))
        assert (np.abs(lse[rows] - norm) <= 1.05 * (delta + 2.0 ** -23 * np.abs(norm))).all(), b


@pytest.mark.parametrize("room", [0, 2304])                # the plain call's kernels, and those of shared parts
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("qscale", [6.0, 40.0])            # scores of up to 30 and 200 among hundreds of keys
@pytest.mark.parametrize("i", [0, 2, 3, 5, 7, 9, 10])
def test_large_scores(lb, i, qscale, fp8, room):  # noqa: F811
    bounds, prefix, new, own, Hq, Hk, D, page = SHAPES[i]
    pr = Shared(70 + i, bounds, prefix, new, own, Hq, Hk, D, page, fp8, qscale=qscale, room=room)
    check(pr, *pr.shared(lb))
    assert lb.lowbit_device_error() == 0

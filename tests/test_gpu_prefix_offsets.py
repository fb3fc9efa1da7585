"""lowbit_prefix_attention where cu_groups or cu_q is out of order: rows are right or left alone, never wrong.

Rows that are written are compared with those of the call whose arrays are in order.  The work is cut elsewhere, so
weights and output are rounded twice each, 2^-8 of values up to 4: the tolerance of test_gpu_prefix.py's bad groups."""
import pytest

from test_gpu_paged import i32
from test_gpu_paged import lb  # noqa: F401  (a fixture)
from test_gpu_prefix import Shared

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

INVALID = 1


def rows_of(pr, requests):
    return [t for b in requests for t in range(int(pr.cu[b]), int(pr.cu[b + 1]))]


def check(out, good, right, either):
    """Rows `right` are good's, rows `either` are good's or untouched, all others untouched."""
    for t in range(out.shape[0]):
        untouched = bool((out[t] == 7.0).all())
        same = torch.allclose(out[t].float(), good[t].float(), rtol=2.0 ** -7, atol=2.0 ** -7 * 4)
        assert same if t in right else (same or untouched if t in either else untouched), (t, same, untouched)


# a bound past the requests, below zero, or before the one ahead of it, between groups that share unlike lengths
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("each", [1, 9])                   # up to 32 requests, and more
@pytest.mark.parametrize("bad,prefix,right,undefined", [
    ([0, 2, 9, 4, 6], [96, 64, 0, 160], [0, 1], []),
    ([0, 2, 9, 4, 6], [96, 160, 0, 64], [0, 1], []),
    ([0, 2, -1, 4, 6], [96, 160, 0, 64], [], []),
    ([0, 4, 2, 2, 6], [96, 64, 0, 160], [], [2, 3, 4, 5])])  # two groups claim two requests, the last one others' pages too
def test_groups_out_of_order(lb, bad, prefix, right, undefined, each, fp8):  # noqa: F811
    def spread(requests):
        return [b * each + i for b in requests for i in range(each)]
    n = 6 * each
    pr = Shared(21, [each * b for b in (0, 2, 4, 4, 6)], prefix, [1 + b % 2 for b in range(n)],
                [150 + b % 11 for b in range(n)], 4, 2, 64, 16, fp8)
    good = pr.shared(lb)[0].clone()
    assert lb.lowbit_device_error() == 0
    pr.bounds = [each * b for b in bad]
    out, _ = pr.shared(lb)
    assert lb.lowbit_device_error() == INVALID
    keep = torch.ones(pr.T, dtype=torch.bool)
    keep[rows_of(pr, spread(undefined))] = False
    keep = keep.nonzero()[:, 0].tolist()
    where = {t: i for i, t in enumerate(keep)}
    mine = [where[t] for t in rows_of(pr, spread(right))]
    check(out[keep], good[keep], mine, range(len(keep)))

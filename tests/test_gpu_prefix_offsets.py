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


# an offset below zero, past the rows, or before the one ahead of it: the requests on either side of it are inconsistent
@pytest.mark.parametrize("room", [0, 2304])                # the plain call's kernels, and those of shared parts
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [5, 45])                     # up to 32 requests, and more
@pytest.mark.parametrize("bad", [-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1])
def test_offsets_of_rows_out_of_order(lb, bad, n, fp8, room):  # noqa: F811
    pr = Shared(22, [0, n], [96], [2] * n, [30 + b % 40 for b in range(n)], 4, 2, 64, 16, fp8, room=room)
    args = pr.args(lb)
    lb.lowbit_prefix_attention(**args)
    good = pr.out[:pr.T].clone()
    assert lb.lowbit_device_error() == 0
    at = 3 * n // 5                                        # requests at - 1 and at have it as their end and start
    right = [b for b in range(n) if b not in (at - 1, at)]
    rows = rows_of(pr, right)
    cu = pr.cu.copy()
    cu[at] = bad
    args["cu_q"].copy_(i32(cu))
    for _ in range(2):                                     # with what either call leaves in the workspace
        pr.out[:] = 7.0
        lb.lowbit_prefix_attention(**args)
        check(pr.out[:pr.T], good, rows, [])
        assert lb.lowbit_device_error() == INVALID
    args["workspace"].fill_(0)                             # a request that zeros name
    pr.out[:] = 7.0
    lb.lowbit_prefix_attention(**args)
    check(pr.out[:pr.T], good, rows, [])
    assert lb.lowbit_device_error() == INVALID


def test_rows_left_out_after_a_call_that_had_them(lb):  # noqa: F811
    """The workspace names requests of an earlier call for rows that nobody has now."""
    pr = Shared(23, [0, 6], [96], [3, 1, 2, 0, 4, 2], [30, 2, 70, 5, 0, 9], 4, 2, 64, 16)
    args = pr.args(lb)
    lb.lowbit_prefix_attention(**args)
    good = pr.out[:pr.T].clone()
    for cu, kept in (([0, 3, 4, 6, 6, 6, 6], 6), ([0, 3, 3, 3, 3, 3, 3], 3), ([0, 0, 0, 0, 0, 0, 0], 0)):
        args["cu_q"].copy_(i32(cu))
        pr.out[:] = 7.0
        lb.lowbit_prefix_attention(**args)
        check(pr.out[:pr.T], good, range(kept), [])
    assert lb.lowbit_device_error() == 0

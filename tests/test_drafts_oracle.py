"""CPU pins of the oracle for verified drafts, and the host-side refusals of lowbit_verify_drafts."""
import struct

import numpy as np
import pytest

from oracle import drafts, sample
from test_paged_oracle import native  # noqa: F401  (a fixture)

ROW = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
PLAIN = (1.0, 0, 1.0, 0.0)


def test_by_hand():
    y = np.log(np.array([0.4, 0.2, 0.2, 0.2]))
    q = drafts.proposal(4, 0, y)
    assert np.allclose(q[0], [0.4, 0.2, 0.2, 0.2]) and np.isclose(q[1], 0.4)
    # p(0) / q(0) = 1/4; the rest after a rejection is (0, 0.2, 0, 0.1)
    for u, n in ((0.2499, 1), (0.2501, 0)):
        k, tokens, accept = drafts.verify([ROW, ROW], [0], [u], 0.51, PLAIN, [q])
        assert k == n and np.isclose(accept[0], 0.25)
        assert tokens == ([0, 2] if n else [1, -1])      # p: token 2 begins at 0.5; rest: 0.2 of 0.3 is token 1's
    assert drafts.verify([ROW, ROW], [0], [0.3], 0.67, PLAIN, [q])[1] == [3, -1]
    # more likely than the drafter thought: always taken
    k, tokens, accept = drafts.verify([ROW, ROW], [1], [0.999999], 0.05, PLAIN, [drafts.proposal(4, 1, y)])
    assert (k, tokens, accept) == (1, [1, 0], [1.0])


def test_proposed_with_certainty():
    q = drafts.proposal(4, 2)
    assert q[0].tolist() == [0, 0, 1, 0] and q[1] == 1.0
    assert drafts.verify([ROW, ROW], [2], [0.19], 0.0, PLAIN, [q])[0] == 1
    k, tokens, _ = drafts.verify([ROW, ROW], [2], [0.21], 0.6, PLAIN, [q])
    assert k == 0 and tokens == [1, -1]                  # the others: 0.1, 0.4, 0.3 of 0.8; 0.6 of it is 0.48
    assert drafts.verify([ROW, ROW], [2], [0.21], 0.63, PLAIN, [q])[1] == [3, -1]


def test_dropped_tokens_columns_and_outsiders():
    top2 = (1.0, 2, 1.0, 0.0)                            # tokens 1 and 3: 4/7 and 3/7
    assert drafts.verify([ROW, ROW], [0], [0.0], 0.0, top2, [drafts.proposal(4, 0)])[:2] == (0, [1, -1])
    q = drafts.proposal(4, 3, np.zeros(2), index=[0, -1, 1, -1])
    assert q[0].tolist() == [0.5, 0, 0.5, 0] and q[1] == 0.0
    assert drafts.verify([ROW, ROW], [3], [0.99], 0.0, PLAIN, [q])[2] == [1.0]       # q = 0 and p > 0
    assert drafts.proposal(4, 9, np.zeros(4))[1] == 0.0 and not drafts.proposal(4, -1)[0].any()
    assert drafts.verify([ROW, ROW], [9], [0.0], 0.0, PLAIN, [drafts.proposal(4, 9)])[0] == 0


def test_no_drafts_is_plain_sampling():
    for v in (0.0, 0.3, 0.77, 0.9999):
        assert drafts.verify([ROW], [], [], v, PLAIN, [])[1] == [sample.draw(np.exp(ROW), v)]


def test_equal_rows_accept_everything_and_empty_rows_nothing():
    q = drafts.proposal(4, 1, ROW)
    assert drafts.verify([ROW] * 3, [1, 1], [0.99, 0.99], 0.0, PLAIN, [q, q])[0] == 2
    none = np.full(4, -np.inf)
    assert drafts.verify([none, ROW], [1], [0.0], 0.5, PLAIN, [q])[:2] == (0, [-1, -1])


def test_the_outcome_is_distributed_as_the_target():
    """Over all drafts and a grid of numbers the first token's share is p."""
    g = np.random.default_rng(0)
    z, y = g.standard_normal(5) * 1.5, g.standard_normal(5) * 1.5
    p, q = drafts.shares(z, PLAIN), drafts.shares(y, PLAIN)
    got, grid = np.zeros(5), 200
    for d in range(5):
        pr = drafts.proposal(5, d, y)
        for u in (np.arange(grid) + 0.5) / grid:
            if u * pr[1] < p[d]:
                got[d] += q[d] / grid
            else:
                r = drafts.rest(p, pr[0])
                got += q[d] / grid * r / r.sum()
    assert np.abs(got - p).max() < 2 / grid


# ------------------------------------------------------------------ host-side refusals

INVALID, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 4
P = 0x10000      # never dereferenced


def rows(**kw):
    f = dict(logits=P, stride=100, dtype=0, rows=8, V=100, temperature=None, top_k=None, top_p=None, min_p=None) | kw
    return struct.pack("@Pqiii0qPPPP", f["logits"] or 0, f["stride"], f["dtype"], f["rows"], f["V"],
                       *(f[x] or 0 for x in ("temperature", "top_k", "top_p", "min_p")))


def call(n, target=None, draft=None, **kw):
    f = dict(B=2, N=6, cu=P, drafts=P, index=None, u=P, v=P, count=P, ids=P, accept=None, ws=P, bytes=1 << 20) | kw
    g = n.lib.lowbit_verify_drafts
    return g(target if target is not None else rows(), draft, f["B"], f["N"], f["cu"], f["drafts"], f["index"], f["u"], f["v"],
             f["count"], f["ids"], f["accept"], f["ws"], f["bytes"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(target=rows(logits=None)), INVALID), (dict(target=rows(dtype=2)), INVALID), (dict(cu=None), INVALID),
    (dict(drafts=None), INVALID), (dict(u=None), INVALID), (dict(v=None), INVALID), (dict(count=None), INVALID), (dict(ids=None), INVALID),
    (dict(index=P), INVALID), (dict(draft=rows(logits=None, rows=6)), INVALID), (dict(draft=rows(dtype=7, rows=6)), INVALID),
    (dict(B=0), SHAPE), (dict(B=(1 << 16) + 1), SHAPE), (dict(N=-1), SHAPE), (dict(target=rows(rows=0)), SHAPE),
    (dict(target=rows(V=0)), SHAPE), (dict(target=rows(V=(1 << 19) + 1, stride=1 << 20)), SHAPE), (dict(target=rows(stride=99)), SHAPE),
    (dict(draft=rows(rows=5)), SHAPE), (dict(draft=rows(rows=6, V=101)), SHAPE), (dict(draft=rows(rows=6, V=0)), SHAPE),
    (dict(target=rows(logits=P + 2)), ALIGN), (dict(target=rows(logits=P + 1, dtype=1)), ALIGN), (dict(ids=P + 2), ALIGN),
    (dict(draft=rows(rows=6, top_p=P + 1)), ALIGN), (dict(accept=P + 1), ALIGN), (dict(ws=P + 8), ALIGN), (dict(ws=None), WORKSPACE),
    (dict(bytes=8 * 2080 + 6 * 32 - 1), WORKSPACE)])
def test_refusals(native, kw, status):  # noqa: F811
    assert call(native, **kw) == status


# Arrays of two requests and six drafts, a megabyte apart, and what of them lies over another one's bytes.
APART = {x: P + (i << 20) for i, x in enumerate(("cu", "drafts", "index", "u", "v", "count", "ids", "accept", "ws"))}
Z, Y = P + (20 << 20), P + (30 << 20)


@pytest.mark.parametrize("written", ["count", "ids", "accept", "ws"])
def test_outputs_over_anything_else_are_refused(native, written):  # noqa: F811
    import torch
    if torch.cuda.is_available():
        pytest.skip("calls that are not refused would run on these addresses")
    bytes_of = dict(cu=12, drafts=24, index=400, u=24, v=8, count=8, ids=32, accept=24, ws=8 * 2080 + 6 * 32)
    temp = P + (40 << 20)

    def status(**kw):
        target, draft = rows(logits=Z, temperature=temp), rows(logits=Y, rows=6, min_p=temp + 4096)
        return call(native, target, draft, **(APART | kw))

    near = 16 if written == "ws" else 4
    for other, at in APART.items():
        if other == written:
            continue
        end = (bytes_of[other] + near - 1) // near * near
        assert status(**{written: at}) == status(**{written: at + end - near}) == INVALID, other
        assert status(**{written: at + end}) != INVALID, other      # a device is all that is missing
    for at in (Z, Z + 4 * 796, Y + 4 * 592, temp, temp + 4096):
        assert status(**{written: at}) == INVALID
    assert status(**{written: Y + 4 * 600}) != INVALID
    assert status(index=None) != INVALID


def test_no_rows_at_all(native):  # noqa: F811
    f = native.lib.lowbit_verify_drafts
    assert f(None, None, 1, 0, P, None, None, None, P, P, P, None, P, 100, None) == INVALID


def test_workspace_sizes(native):  # noqa: F811
    f = native.lowbit_verify_drafts_workspace_bytes
    assert f(8, 6) == 8 * 2080 + 6 * 32 and f(1, 0) == 2080
    assert f(0, 0) == f(4, -1) == f((1 << 24) + 1, 0) == 0


def test_the_binding_refuses_host_tensors(native):  # noqa: F811
    import torch
    import bit_weight_gemv_gb300 as lb
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError):
        lb.lowbit_verify_drafts(torch.zeros((1, 8)), i, i, torch.zeros(1), torch.zeros(1), i, i, torch.zeros(32, dtype=torch.uint8))

"""Host-side refusals of lowbit_kv_append that need no GPU: outputs that lie over what is still read."""
import pytest

from test_paged_oracle import append, batch, cache, native  # noqa: F401  (native is a fixture)

OK_BUT_NO_GPU = 6   # every argument is accepted; the device error word then has no device
INVALID = 1
AT = 1 << 20


def rows(native, T, **kw):
    """An append of T rows with q, k, v and q_out where `kw` puts them; 4 query and 2 key/value heads of 128."""
    place = dict(q=AT << 4, qs=512, k=AT << 1, ks=256, v=AT << 2, vs=256, q_out=AT << 3) | kw
    return append(native, batch(native, T=T), cache(native), **place)


# rows of 1,024 bytes (q) and 512 bytes (k, v); one product's output has rows of 2,048 bytes
@pytest.mark.parametrize("T,kw", [
    (2, dict(q=AT, qs=1024, q_out=AT)),                               # in place, but rows apart
    (5, dict(q=AT, qs=520, q_out=AT)),
    (2, dict(q=AT, qs=512, q_out=AT + 16)),                           # shifted
    (2, dict(q=AT, qs=512, q_out=AT - 1024)),
    (3, dict(q=AT, qs=1024, k=AT + 1024, ks=1024, v=AT + 1536, vs=1024, q_out=AT + 3 * 2048 - 528)),  # the last row of v
    (3, dict(q=AT, qs=1024, k=AT + 1024, ks=1024, v=AT + 1536, vs=1024, q_out=AT - 3 * 1024 + 16)),
    (1, dict(k=AT, q_out=AT)), (1, dict(v=AT, q_out=AT)), (1, dict(v=AT, q_out=AT + 496)), (1, dict(k=AT, q_out=AT - 1008)),
    (4, dict(k=AT, ks=1 << 40, q_out=AT + (3 << 41))),                # far apart: the fourth row
])
def test_outputs_over_inputs_are_refused(native, T, kw):  # noqa: F811
    assert rows(native, T, **kw) == INVALID


@pytest.mark.parametrize("T,kw", [
    (5, dict(q=AT, qs=512, q_out=AT)),                                # in place
    (1, dict(q=AT, qs=4096, q_out=AT)),                               # one row: dense whatever the stride
    (1, dict(q=AT, qs=1024, k=AT + 1024, ks=1024, v=AT + 1536, vs=1024, q_out=AT + 2048)),
    (3, dict(q=AT, qs=1024, k=AT + 1024, ks=1024, v=AT + 1536, vs=1024, q_out=AT + 3 * 2048)),
    (3, dict(q=AT, qs=1024, k=AT + 1024, ks=1024, v=AT + 1536, vs=1024, q_out=AT - 3 * 1024)),
    (2, dict(q=AT, qs=4096, q_out=AT + 1024)),                        # between two rows
    (4, dict(k=AT, ks=1 << 40, q_out=AT + (4 << 41))),
    (4, dict(k=AT, ks=(1 << 62) + 8, q_out=AT + 512)),
])
def test_outputs_beside_inputs_are_taken(native, T, kw):  # noqa: F811
    import torch
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only where no kernel can run")
    assert rows(native, T, **kw) == OK_BUT_NO_GPU

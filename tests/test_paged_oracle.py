"""CPU pins of the oracle for the paged-cache operators and sampling, the host-side refusals of
their entry points, and the binding's checks."""
import ctypes
import struct

import numpy as np
import pytest

from oracle import paged, sample


def test_positions_of_a_ragged_batch():
    req, pos = paged.positions([0, 2, 2, 5], [7, 9, 3])
    assert req.tolist() == [0, 0, 2, 2, 2]
    assert pos.tolist() == [5, 6, 0, 1, 2]


def test_rotation_by_hand():
    # a quarter turn takes (a, b) to (-b, a); pairs (0, 2), (1, 3) in halves, (0, 1), (2, 3) adjacent
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 9.0]]], dtype=np.float32)
    rows = np.array([[0.0, 0.0, 1.0, 1.0]], dtype=np.float32)
    assert paged.rotate(x, rows, False)[0, 0].tolist() == [-3.0, -4.0, 1.0, 2.0, 9.0]
    assert paged.rotate(x, rows, True)[0, 0].tolist() == [-2.0, 1.0, -4.0, 3.0, 9.0]


def test_rotation_keeps_relative_positions():
    g = np.random.default_rng(0)
    q, k = g.standard_normal((2, 1, 1, 8)).astype(np.float32)
    rate = 1.0 / 100.0 ** (np.arange(4) / 4)

    def at(x, p):
        a = p * rate
        return paged.rotate(x, np.concatenate([np.cos(a), np.sin(a)])[None].astype(np.float32), False)

    d = [float(np.sum(at(q, p + 5) * at(k, p))) for p in (0, 3, 40)]
    assert np.allclose(d, d[0], atol=1e-4)


def test_visible_by_hand():
    assert paged.visible(2, 4, True, 0).astype(int).tolist() == [[1, 1, 1, 0], [1, 1, 1, 1]]
    assert paged.visible(2, 4, True, 2).astype(int).tolist() == [[0, 1, 1, 0], [0, 0, 1, 1]]
    assert paged.visible(2, 4, False, 2).astype(int).tolist() == [[0, 1, 1, 1], [0, 0, 1, 1]]
    # more new tokens than keys: the first ones come before every key
    assert paged.visible(3, 1, True, 0).astype(int).tolist() == [[0], [0], [1]]


def test_attention_closed_forms():
    g = np.random.default_rng(1)
    q, k, v = g.standard_normal((3, 4, 8)), g.standard_normal((5, 2, 8)), g.standard_normal((5, 2, 8))
    see = paged.visible(3, 5, True, 0)
    out, lse, _ = paged.attention(np.zeros_like(q), k, v, see, 0.3)
    for i in range(3):                      # equal scores: the mean of the visible values
        n = see[i].sum()
        assert np.allclose(out[i, 3], v[:n, 1].mean(0)) and np.allclose(lse[i], np.log(n))
    k2 = k.copy()
    k2[1, 0] = 100 * q[2, 1]                # one key far ahead of the rest
    out, _, _ = paged.attention(q, k2, v, see, 1.0)
    assert np.allclose(out[2, 1], v[1, 0])
    out, lse, _ = paged.attention(q, k[:1], v[:1], paged.visible(3, 1, True, 0), 1.0)
    assert (out[0] == 0).all() and np.isneginf(lse[0]).all() and np.allclose(out[2, 0], v[0, 0])


def test_attention_joins_over_split_keys():
    g = np.random.default_rng(2)
    q, k, v = g.standard_normal((1, 2, 8)), g.standard_normal((9, 1, 8)), g.standard_normal((9, 1, 8))
    see = np.ones((1, 9), dtype=bool)
    out, lse, _ = paged.attention(q, k, v, see, 0.5)
    o1, l1, _ = paged.attention(q, k[:4], v[:4], see[:, :4], 0.5)
    o2, l2, _ = paged.attention(q, k[4:], v[4:], see[:, 4:], 0.5)
    assert np.allclose(np.logaddexp(l1, l2), lse)
    assert np.allclose(np.exp(l1 - lse)[..., None] * o1 + np.exp(l2 - lse)[..., None] * o2, out)


def test_sampling_by_hand():
    z = np.log(np.array([0.1, 0.4, 0.1, 0.4]))
    assert np.allclose(sample.distribution(z), [0.25, 1, 0.25, 1])
    assert np.flatnonzero(sample.distribution(z, top_k=1)).tolist() == [1]        # lowest of equals
    assert np.flatnonzero(sample.distribution(z, top_k=3)).tolist() == [0, 1, 3]
    assert np.flatnonzero(sample.distribution(z, top_p=0.39)).tolist() == [1]
    assert np.flatnonzero(sample.distribution(z, top_p=0.41)).tolist() == [1, 3]
    assert np.flatnonzero(sample.distribution(z, top_p=0.0)).tolist() == [1]
    assert np.flatnonzero(sample.distribution(z, min_p=0.5)).tolist() == [1, 3]
    assert np.flatnonzero(sample.distribution(z, temperature=0.0)).tolist() == [1]
    # top-p counts the mass that top-k left: 0.4 of 0.8 is one token
    assert np.flatnonzero(sample.distribution(z, top_k=2, top_p=0.5)).tolist() == [1]
    w = sample.distribution(z)
    assert [sample.draw(w, u) for u in (0.0, 0.0999, 0.11, 0.49, 0.51, 0.61, 0.9999)] == [0, 0, 1, 1, 2, 3, 3]


def test_sampling_edges():
    inf = float("inf")
    assert sample.distribution([-inf, -inf]) is None
    assert sample.distribution([float("nan"), -inf]) is None
    assert np.flatnonzero(sample.distribution([1.0, inf, 2.0])).tolist() == [1]
    assert np.flatnonzero(sample.distribution([-inf, 0.0, float("nan")])).tolist() == [1]
    assert sample.distribution([0.0, -28.5])[1] == 0.0 and sample.distribution([0.0, -28.0])[1] > 0.0


# ------------------------------------------------------------------ host-side refusals


@pytest.fixture(scope="module")
def native():
    from bit_weight_gemv_gb300 import build
    build.build()
    from bit_weight_gemv_gb300 import _native
    return _native


P = 0x10000      # never dereferenced: every call below is refused on the host


def batch(n, **kw):
    f = dict(cu_q=P, kv_lens=P, block_table=P, table_stride=8, B=2, T=4, width=8)
    f |= kw
    return struct.pack("@PPPqiii0q", *(f[x] or 0 for x in ("cu_q", "kv_lens", "block_table", "table_stride", "B", "T", "width")))


def cache(n, **kw):
    f = dict(k=P, v=P, page_stride=64 * 2 * 128, token_stride=2 * 128, head_stride=128, num_pages=9,
             page_size=64, heads=2, head_dim=128, dtype=0, k_scale=None, v_scale=None)
    return n._PagedCache(**(f | kw))


INVALID, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 4
BAD_BATCH = [(dict(cu_q=None), INVALID), (dict(kv_lens=None), INVALID), (dict(block_table=None), INVALID),
             (dict(B=0), SHAPE), (dict(T=-1), SHAPE), (dict(width=0), SHAPE), (dict(table_stride=7), SHAPE),
             (dict(cu_q=P + 2), ALIGN)]
BAD_CACHE = [(dict(k=None), INVALID), (dict(v=None), INVALID), (dict(dtype=2), INVALID),
             (dict(k_scale=P), INVALID), (dict(page_size=48), SHAPE), (dict(page_size=2048), SHAPE),
             (dict(num_pages=0), SHAPE), (dict(heads=0), SHAPE), (dict(head_dim=96), SHAPE),
             (dict(k=P + 8), ALIGN), (dict(token_stride=132), ALIGN), (dict(page_stride=0), ALIGN),
             (dict(dtype=1, head_stride=136), ALIGN)]


def append(n, b, c, **kw):
    f = dict(q=P, qs=4 * 128, k=P, ks=2 * 128, v=P, vs=2 * 128, Hq=4, rope=P, rows=100, rot=128, q_out=P)
    f |= kw
    return n.lib.lowbit_kv_append(f["q"], f["qs"], f["k"], f["ks"], f["v"], f["vs"], f["Hq"], f["rope"],
                                  f["rows"], f["rot"], 0, b, ctypes.byref(c), f["q_out"], None)


def attend(n, b, c, **kw):
    f = dict(q=P, qs=4 * 128, Hq=4, scale=0.1, window=0, out=P, lse=P, ws=P, bytes=1 << 40)
    f |= kw
    return n.lib.lowbit_paged_attention(f["q"], f["qs"], f["Hq"], b, ctypes.byref(c), f["scale"],
                                        1, f["window"], f["out"], f["lse"], f["ws"], f["bytes"], None)


def draw(n, **kw):
    f = dict(logits=P, dtype=0, stride=100, M=1, V=100, t=None, k=None, p=None, mp=None, u=P, map=None,
             ids=P, lp=None, kept=None)
    f |= kw
    return n.lib.lowbit_sample(f["logits"], f["dtype"], f["stride"], f["M"], f["V"], f["t"], f["k"], f["p"],
                               f["mp"], f["u"], f["map"], f["ids"], f["lp"], f["kept"], None)


@pytest.mark.parametrize("kw,status", BAD_BATCH)
def test_bad_batches_are_refused(native, kw, status):
    assert append(native, batch(native, **kw), cache(native)) == status
    assert attend(native, batch(native, **kw), cache(native)) == status


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_bad_caches_are_refused(native, kw, status):
    assert append(native, batch(native), cache(native, **kw)) == status
    assert attend(native, batch(native), cache(native, **kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(q_out=None), INVALID), (dict(q=None), INVALID),
    (dict(rope=None), INVALID), (dict(rot=0), INVALID), (dict(rows=0), INVALID), (dict(rot=24), SHAPE),
    (dict(rot=144), SHAPE), (dict(qs=4 * 128 - 8), SHAPE), (dict(ks=248), SHAPE), (dict(Hq=0), SHAPE),
    (dict(q=P + 8), ALIGN), (dict(vs=2 * 128 + 4), ALIGN), (dict(rope=P + 4), ALIGN)])
def test_append_refusals(native, kw, status):
    assert append(native, batch(native), cache(native), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(Hq=3), SHAPE), (dict(Hq=0), SHAPE), (dict(window=-1), SHAPE), (dict(qs=504), SHAPE),
    (dict(ws=None), WORKSPACE), (dict(bytes=100), WORKSPACE), (dict(out=P + 8), ALIGN), (dict(qs=516), ALIGN),
    (dict(lse=P + 2), ALIGN)])
def test_attention_refusals(native, kw, status):
    assert attend(native, batch(native), cache(native), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), INVALID), (dict(u=None), INVALID), (dict(ids=None), INVALID), (dict(dtype=2), INVALID),
    (dict(M=0), SHAPE), (dict(V=0), SHAPE), (dict(V=(1 << 19) + 1, stride=1 << 20), SHAPE), (dict(stride=99), SHAPE),
    (dict(logits=P + 2), ALIGN), (dict(dtype=1, logits=P + 1), ALIGN), (dict(ids=P + 2), ALIGN)])
def test_sample_refusals(native, kw, status):
    assert draw(native, **kw) == status


def test_nothing_to_do_is_no_error(native):
    assert append(native, batch(native, T=0), cache(native)) == 0
    assert attend(native, batch(native, T=0), cache(native)) == 0


def test_workspace_sizes(native):
    f = native.lowbit_paged_attention_workspace_bytes
    assert f(16, 1, 32, 8, 128) > 0 and f(0, 1, 32, 8, 64) > 0
    assert f(-1, 1, 32, 8, 128) == f(16, 0, 32, 8, 128) == f(16, 1, 30, 8, 128) == f(16, 1, 32, 8, 96) == 0


def test_binding_refuses_host_tensors(native):
    import torch
    import bit_weight_gemv_gb300 as lb
    t = torch.zeros((2, 16, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        lb.lowbit_paged_cache(t, t)
    with pytest.raises(TypeError):
        lb.lowbit_sample(torch.zeros((1, 8)), torch.zeros(1), torch.zeros(1, dtype=torch.int32))

"""Host-side refusals of lowbit_kv_append_norm and lowbit_prefix_attention, which need no GPU."""
import ctypes

import pytest

from test_paged_oracle import BAD_BATCH, BAD_CACHE, P, batch, cache, native  # noqa: F401  (native is a fixture)

INVALID, SHAPE, ALIGN, WORKSPACE, NO_GPU = 1, 2, 3, 4, 6


def append(n, b, c, **kw):
    f = dict(q=P, qs=4 * 128, k=P << 1, ks=2 * 128, v=P << 2, vs=2 * 128, Hq=4, qw=P, kw=P, eps=1e-6, rope=P, rows=100, rot=128,
             q_out=P << 3) | kw
    return n.lib.lowbit_kv_append_norm(f["q"], f["qs"], f["k"], f["ks"], f["v"], f["vs"], f["Hq"], f["qw"], f["kw"], f["eps"],
                                       f["rope"], f["rows"], f["rot"], 0, b, ctypes.byref(c), f["q_out"], None)


def attend(n, b, c, **kw):
    f = dict(q=P, qs=4 * 128, Hq=4, groups=P, lens=P, count=1, scale=0.1, out=P, lse=P, ws=P, bytes=1 << 40) | kw
    return n.lib.lowbit_prefix_attention(f["q"], f["qs"], f["Hq"], b, ctypes.byref(c), f["groups"], f["lens"], f["count"],
                                         f["scale"], 1, f["out"], f["lse"], f["ws"], f["bytes"], None)


@pytest.mark.parametrize("kw,status", BAD_BATCH)
def test_bad_batches(native, kw, status):  # noqa: F811
    assert append(native, batch(native, **kw), cache(native)) == status
    assert attend(native, batch(native, **kw), cache(native)) == status


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_bad_caches(native, kw, status):  # noqa: F811
    assert append(native, batch(native), cache(native, **kw)) == status
    assert attend(native, batch(native), cache(native, **kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(q_out=None), INVALID), (dict(q=None), INVALID),
    (dict(q=None, q_out=None), INVALID), (dict(rope=None), INVALID), (dict(rot=0), INVALID), (dict(rot=24), SHAPE),
    (dict(rot=144), SHAPE), (dict(qs=4 * 128 - 8), SHAPE), (dict(Hq=0), SHAPE), (dict(q=P + 8), ALIGN), (dict(qw=P + 4), ALIGN),
    (dict(kw=P + 8), ALIGN), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(q_out=P << 1), INVALID), (dict(qs=1024, q_out=P), INVALID)])
def test_append_norm(native, kw, status):  # noqa: F811
    assert append(native, batch(native), cache(native), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(scale=float("nan")), INVALID), (dict(groups=None), INVALID),
    (dict(lens=None), INVALID), (dict(count=0), SHAPE), (dict(count=-1), SHAPE), (dict(count=(1 << 16) + 1), SHAPE), (dict(Hq=3), SHAPE),
    (dict(qs=504), SHAPE), (dict(ws=None), WORKSPACE), (dict(bytes=100), WORKSPACE), (dict(ws=P + 8), ALIGN), (dict(out=P + 8), ALIGN),
    (dict(groups=P + 2), ALIGN), (dict(lens=P + 1), ALIGN), (dict(lse=P + 2), ALIGN)])
def test_prefix_attention(native, kw, status):  # noqa: F811
    assert attend(native, batch(native), cache(native), **kw) == status


def test_nothing_to_do_is_no_error(native):  # noqa: F811
    assert append(native, batch(native, T=0), cache(native)) == 0
    assert attend(native, batch(native, T=0), cache(native)) == 0


def test_workspace_sizes(native):  # noqa: F811
    f, plain = native.lowbit_prefix_attention_workspace_bytes, native.lowbit_paged_attention_workspace_bytes
    assert f(16, 2, 32, 8, 128) == 2 * plain(16, 2, 32, 8, 128) + 16 * 32 * (8 * 128 + 48)
    assert f(0, 2, 32, 8, 64) == 2 * plain(0, 2, 32, 8, 64)
    assert f(-1, 1, 32, 8, 128) == f(16, 0, 32, 8, 128) == f(16, 1, 30, 8, 128) == f(16, 1, 32, 8, 96) == 0

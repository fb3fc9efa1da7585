"""The example that runs the products, the append, the attention and the sampling as one serving
step: each stage against the oracle on what the stage before left behind."""
import os
import sys

import numpy as np
import pytest

from oracle import paged, sample

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import decode_block
    return decode_block


@pytest.mark.parametrize("fp8", [False, True])
def test_stages(ex, fp8):
    B, new = 3, 5
    d = ex.Decoder(B, 64, seed=1, fp8_cache=fp8)
    s = d.buffers(new)
    for _ in range(3):
        s["tokens"].random_(0, ex.VOCAB)
        s["u"].uniform_()
        d.step(s)
    torch.cuda.synchronize()
    assert d.kv_lens.tolist() == [3 * new] * B
    cache = [t.float().cpu().numpy().astype(np.float64) * (1 / 32 if fp8 else 1.0) for t in (d.cache.k, d.cache.v)]
    table = d.block_table.cpu().numpy()
    q, out = s["q"].double().cpu().numpy(), s["out"].double().cpu().numpy()
    see = paged.visible(new, 3 * new, True, 0)
    for b in range(B):
        k, v = (paged.gather(c, table[b], 3 * new, ex.PAGE) for c in cache)
        rows = slice(b * new, (b + 1) * new)
        want, _, spread = paged.attention(q[rows], k, v, see, ex.DIM ** -0.5)
        # weights and output rounded to bf16 (see test_gpu_paged), 15 keys of fp16 weights over e4m3
        assert (np.abs(out[rows] - want) <= 1.05 * (2.0 ** -8 * (spread + np.abs(want)) + 1e-4 * spread) + 1e-6).all()
    # the newest keys in the cache are the rotated products
    last = 3 * new - 1
    row = d.rope.cpu().numpy()[[last]]
    for b in range(B):
        raw = s["k"][(b + 1) * new - 1].float().cpu().numpy()[None]
        want = paged.rotate(raw, row, False)[0]
        got = cache[0][table[b, last // ex.PAGE], last % ex.PAGE]
        step = 2.0 ** -4 if fp8 else 2.0 ** -8      # half a unit of e4m3 (4 significant bits), of bf16
        assert (np.abs(got - want) <= step * np.abs(want) * 1.01 + (2.0 ** -10 / 32 if fp8 else 0)).all()
    for b in range(B):
        w = sample.distribution(s["logits"][b].float().cpu().numpy(), 0.8, 50, 0.95, 0.02)
        i, cum = int(s["ids"][b]), np.cumsum(w)
        assert w[i] > 0
        assert (cum[i] - w[i]) / cum[-1] - 1e-5 <= float(s["u"][b]) <= cum[i] / cum[-1] + 1e-5


def test_runs_as_a_program(ex):
    rows, lens = ex.main(batch=2, prompt=32, decode=4)
    assert lens == [36, 36] and all(len(r) == 4 and all(0 <= i < ex.VOCAB for i in r) for r in rows)

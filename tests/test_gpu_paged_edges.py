"""GPU checks of the paged calls at their edges: scores far beyond those of a model.

Row counts choose the kernels: tokens times grouped heads per request of up to 8, 16, 32, then 128
rows an item and, past 1,024, 256."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lb():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_weight_gemv_gb300 as lb
    lb.lowbit_device_error()
    yield lb


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def attend(lb, q, kc, vc, new, kv, table, causal=True, window=0, scale=1.0):
    """out and lse of a batch, from plain tensors."""
    T, Hq, D = q.shape
    out = torch.empty_like(q)
    lse = torch.empty((T, Hq), device="cuda")
    ws = torch.full((lb.lowbit_paged_attention_workspace_bytes(T, len(new), Hq, kc.shape[2], D),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    lb.lowbit_paged_attention(q, lb.lowbit_paged_cache(kc, vc), i32(np.concatenate([[0], np.cumsum(new)])), i32(kv),
                              i32(table), out, ws, scale=scale, causal=causal, window=window, lse=lse)
    torch.cuda.synchronize()
    return out, lse


ROWS = [(2, 64), (2, 128), (2, 256), (4, 128), (8, 64), (8, 128), (16, 256), (16, 128), (40, 64), (300, 128), (300, 64)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,D", ROWS)
@pytest.mark.parametrize("scale", [1e3, 3e4, 1e6, 4e7, 3e9])
def test_scores_past_whole_numbers(lb, new, D, scale, fp8):
    """Scores of 21 * scale for one key and 3 * scale for the others: its value is the output, however
    coarse fp32 is there, but for the rounding of its weight (to bf16 at worst) and of the output, 2^-8
    each, times 1.05.  The logarithm of the sum is the score, good to the few roundings of 2^-24 that
    take it to powers of two and back."""
    B, G, kv, page, lead = 3, 4, 700, 32, 333
    pages = -(-kv // page)
    g = torch.Generator(device="cuda").manual_seed(new + D)
    kc = torch.zeros((pages, page, 1, D), device="cuda")
    kc[..., 0] = 1.0
    kc[lead // page, lead % page, 0, 0] = 7.0
    vc = torch.randint(-8, 9, (pages, page, 1, D), device="cuda", generator=g).float()
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    q = torch.zeros((B * new, G, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 3.0
    out, lse = attend(lb, q, kc.to(dt), vc.to(dt), [new] * B, [kv] * B, [list(range(pages))] * B, causal=False, scale=scale)
    want = vc[lead // page, lead % page, 0].expand_as(out)
    assert bool(((out.float() - want).abs() <= 1.05 * 2.0 ** -7 * want.abs()).all())
    assert float((lse.double() / (21.0 * scale) - 1.0).abs().max()) <= 2.0 ** -21

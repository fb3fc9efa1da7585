"""GPU checks of the attention kernels' give-up path.

Under the library's test-only stall setting the first data of a CTA (its key tiles, or on tcgen05
its queries) never come, so the waits of every role run out (a second each), with no access out of
bounds.  Such a call
must record LOWBIT_ERR_TIMEOUT and write neither out nor lse, of whole items or of those that were
cut and are joined afterwards (the workspace holds NaN before it); the same call made normally
afterwards gives the bits that it gave before."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TIMEOUT = 5


@pytest.fixture(scope="module")
def lb():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_weight_gemv_gb300 as lb
    lb.lowbit_device_error()
    yield lb


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# rows per request and head: 2 (eight rows an item), 16, 32, 64 on the warp-level MMA, 64 (128 an item) and
# 1,200 (256 an item) on tcgen05; one long request that is cut many times and short ones that are not
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,D", [(1, 64), (1, 128), (1, 256), (8, 128), (16, 128), (32, 256), (32, 128), (32, 64), (600, 128),
                                   (600, 64)])
def test_stall_times_out_writes_nothing_then_recovers(lb, new, D, fp8):
    G, Hk, page, B = 2, 2, 32, 4
    kv = [5000, new, new + 40, new + 200]
    need = [-(-x // page) for x in kv]
    pages = sum(need)
    g = torch.Generator(device="cuda").manual_seed(new + D)
    kc, vc = (torch.randn((pages, page, Hk, D), device="cuda", generator=g).to(torch.float8_e4m3fn if fp8 else torch.bfloat16)
              for _ in range(2))
    table = np.zeros((B, max(need)), dtype=np.int32)
    for b in range(B):
        table[b, :need[b]] = np.arange(need[b]) + sum(need[:b])
    T = B * new
    q = torch.randn((T, G * Hk, D), device="cuda", generator=g).to(torch.bfloat16)
    cache = lb.lowbit_paged_cache(kc, vc)
    cu, lens, table = i32(np.arange(B + 1) * new), i32(kv), i32(table)

    def run():
        out = torch.full((T, G * Hk, D), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((T, G * Hk), 7.0, device="cuda")
        ws = torch.full((lb.lowbit_paged_attention_workspace_bytes(T, B, G * Hk, Hk, D),), 0xFF, dtype=torch.uint8, device="cuda")
        lb.lowbit_paged_attention(q, cache, cu, lens, table, out, ws, lse=lse)
        return out, lse

    want = run()
    assert lb.lowbit_device_error() == 0 and bool(torch.isfinite(want[1]).all())
    lb.lowbit_debug_inject_stall(True)
    try:
        out, lse = run()
    finally:
        lb.lowbit_debug_inject_stall(False)
    assert lb.lowbit_device_error() == TIMEOUT
    assert bool((out == 7.0).all()) and bool((lse == 7.0).all()), "a timed-out call wrote outputs"
    again = run()
    assert lb.lowbit_device_error() == 0
    assert torch.equal(again[0].view(torch.int16), want[0].view(torch.int16)) and torch.equal(again[1], want[1])

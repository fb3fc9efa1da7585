"""GPU checks of the paged calls at their edges: weights far below the largest one, scores far
beyond those of a model, descriptions of a batch that do not hold together.

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


@pytest.mark.parametrize("below", [25.4, 26.5, 28.0])
@pytest.mark.parametrize("new,D", ROWS)
def test_a_tail_of_tiny_weights_over_e4m3(lb, new, D, below):
    """One leading key whose value is 0, and 2,999 keys 2^below under it whose value is 1: the output is
    the tail's share.  Weights are fp16, good to 2^-11 of themselves or to half of fp16's smallest step,
    2^-25, with the largest at 2^15 (up to 32 rows, and heads of 256) or between 2^7 and 2^15; the output is
    rounded to bf16 (2^-8); scores of below * ln 2 in fp32 move a weight by less than 1e-4.  These times
    1.05.  So many requests that most are not cut: a piece of the keys without the leading one refers to
    its own largest."""
    B, G, kv, page = 300, 4, 3000, 64
    pages = -(-kv // page)
    kc = torch.zeros((pages, page, 1, D), device="cuda")
    vc = torch.ones((pages, page, 1, D), device="cuda")
    kc[0, 0, 0, 0] = 8.0
    vc[0, 0] = 0.0
    kc, vc = kc.to(torch.float8_e4m3fn), vc.to(torch.float8_e4m3fn)
    q = torch.zeros((B * new, G, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 2.0
    scale = float(np.float32(below * np.log(2.0) / 16.0))
    out, lse = attend(lb, q, kc, vc, [new] * B, [kv] * B, [list(range(pages))] * B, causal=False, scale=scale)
    tail = (kv - 1) * np.exp(-16.0 * scale)
    want = tail / (1.0 + tail)
    step = 2.0 ** (below - 25 - (15 if D == 256 or new * G <= 32 else 7))
    tol = 1.05 * (max(2.0 ** -11, step) + 2.0 ** -8 + 1e-4) * want
    assert float((out.double() - want).abs().max()) <= tol
    assert float((lse.double() - (16.0 * scale + np.log1p(tail))).abs().max()) <= 1e-4
    assert lb.lowbit_device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,D", ROWS)
@pytest.mark.parametrize("scale", [1e3, 3e4, 1e6, 4e7, 3e9, -1e6, -3e9])
def test_scores_past_whole_numbers(lb, new, D, scale, fp8):
    """Scores of 21 * |scale| for one key and 3 * |scale| for the others: its value is the output, however
    coarse fp32 is there, but for the rounding of its weight (to bf16 at worst) and of the output, 2^-8
    each, times 1.05.  The logarithm of the sum is the score, good to the few roundings of 2^-24 that
    take it to powers of two and back."""
    B, G, kv, page, lead = 3, 4, 700, 32, 333
    pages = -(-kv // page)
    g = torch.Generator(device="cuda").manual_seed(new + D)
    kc = torch.zeros((pages, page, 1, D), device="cuda")
    kc[..., 0] = 1.0
    kc[lead // page, lead % page, 0, 0] = 7.0
    kc *= 1 if scale > 0 else -1
    vc = torch.randint(-8, 9, (pages, page, 1, D), device="cuda", generator=g).float()
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    q = torch.zeros((B * new, G, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 3.0
    out, lse = attend(lb, q, kc.to(dt), vc.to(dt), [new] * B, [kv] * B, [list(range(pages))] * B, causal=False, scale=scale)
    want = vc[lead // page, lead % page, 0].expand_as(out)
    assert bool(((out.float() - want).abs() <= 1.05 * 2.0 ** -7 * want.abs()).all())
    assert float((lse.double() / (21.0 * abs(scale)) - 1.0).abs().max()) <= 2.0 ** -21


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,D", ROWS)
@pytest.mark.parametrize("scale", [1e3, -1e3, -2e5])
def test_scores_that_come_back_from_afar(lb, new, D, scale, fp8):
    """The first 300 keys score -1,344 |scale|, past whole numbers, and the others next to nothing: their
    weights are those of ordinary scores (weights and output rounded to 2^-8 each, 1e-4 for fp32 scores,
    times 1.05; over e4m3 the weights of a warp that comes back are taken as they come, still 2^-8)."""
    B, G, kv, page = 3, 4, 1000, 32
    pages = -(-kv // page)
    g = torch.Generator(device="cuda").manual_seed(new + D)
    near = torch.randint(-2, 3, (kv,), device="cuda", generator=g) * (2.0 ** -9 if abs(scale) < 1e4 else 2.0 ** -17)
    if fp8 and abs(scale) > 1e4:
        near = near * 0                                  # below e4m3's smallest
    near[:300] = -448.0
    near = near * (1 if scale > 0 else -1)
    kc = torch.zeros((pages * page, 1, D), device="cuda")
    kc[:kv, 0, 0] = near
    vc = torch.randn((pages * page, 1, D), device="cuda", generator=g)
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    kc, vc = (x.view(pages, page, 1, D).to(dt) for x in (kc, vc))
    q = torch.zeros((B * new, G, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 3.0
    out, lse = attend(lb, q, kc, vc, [new] * B, [kv] * B, [list(range(pages))] * B, causal=False, scale=scale)
    x = 3.0 * scale * near.double()
    p = torch.softmax(x, 0)
    v = vc.double().view(-1, D)[:kv]
    want, spread = p @ v, p @ v.abs()
    tol = 1.05 * ((2.0 ** -8 + 1e-4) * spread + 2.0 ** -8 * want.abs())
    assert bool(((out.double() - want).abs() <= tol).all())
    assert float((lse.double() - torch.logsumexp(x, 0)).abs().max()) <= 1e-4


# ------------------------------------------------------------------------------------ descriptions


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 50, 2 ** 30, 200])
@pytest.mark.parametrize("new,kv,G,D", [(100, 3, 1, 64), (100, 60, 4, 128), (6, 2, 4, 128), (2, 1, 4, 64), (9, 4, 4, 256),
                                        (400, 90, 4, 128)])
def test_windows_past_every_length(lb, window, new, kv, G, D):
    """A window that no key falls out of changes nothing, whatever its size, also for a request whose
    first tokens come before every key (more new tokens than keys: positions below zero)."""
    g = torch.Generator(device="cuda").manual_seed(window % 1000 + new)
    page = 16
    pages = -(-kv // page)
    kc, vc = (torch.randn((pages, page, 1, D), device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn((new, G, D), device="cuda", generator=g).to(torch.bfloat16)
    args = (lb, q, kc, vc, [new], [kv], [list(range(pages))])
    for causal in (True, False):
        want, norm = attend(*args, causal=causal, scale=D ** -0.5)
        out, lse = attend(*args, causal=causal, window=window, scale=D ** -0.5)
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, norm)
    assert lb.lowbit_device_error() == 0


def test_append_finds_requests_whatever_the_order_of_the_rows(lb):
    """Offsets that decrease somewhere are recorded; the requests that are consistent are appended (a row
    that two of them claim, for the earlier one)."""
    D = 64
    for cu, kv, want in (
            ([0, 5, 3, 8], [5, 9, 9], {0: [0, 1, 2, 3, 4], 2: [6, 7, 8]}),
            ([0, 3, 8, 6], [3, 5, 9], {0: [0, 1, 2], 1: [0, 1, 2, 3, 4]}),
            ([3, 1, 8], [4, 7], {1: list(range(7))}),
            ([0] * 40 + [3, 2, 6], [6] * 42, {39: [3, 4, 5], 41: [3, 4, 5]})):
        T, B = 8, len(kv)
        x = torch.arange(1, T + 1, device="cuda").to(torch.bfloat16).view(T, 1, 1).expand(T, 1, D).contiguous()
        kc = torch.zeros((B, 16, 1, D), dtype=torch.bfloat16, device="cuda")
        vc = kc.clone()
        q_out = torch.zeros_like(x)
        lb.lowbit_kv_append(x, x, x, None, i32(cu), i32(kv), i32([[b] for b in range(B)]), lb.lowbit_paged_cache(kc, vc), q_out)
        assert lb.lowbit_device_error() == 1
        ref = torch.zeros_like(kc)
        seen = torch.zeros(T, dtype=torch.bool)
        for b, places in want.items():
            for p in places:
                row = cu[b] + p - (kv[b] - (cu[b + 1] - cu[b]))
                ref[b, p] = x[row]
                seen[row] = True
        assert torch.equal(kc, ref) and torch.equal(vc, ref)
        assert torch.equal((q_out[:, 0, 0] != 0).cpu(), seen)

"""GPU parity of lowbit_kv_append and lowbit_paged_attention against the oracle.

Append: the stored bits equal the fp32 formula's, rounded once (exactly).
Attention tolerance, per element, with S = sum_j p_j |v_j| of the row (from the oracle):
  weights rounded to bf16 (8 significant bits: 2^-8 each at most) or, over an e4m3 cache, to fp16
  (11 bits: 2^-11 each, and 2^-25 flat for those below 2^-14: at most keys * 2^-25 * max|v| over a
  sum of at least 1); the output rounded to bf16 (2^-8 of it); scores in fp32: |s| 2^-23 sqrt(D) and the exponential's 2^-22,
  which for the |s| <= 40 of these inputs stay under 1e-4 of S.  The sum of the three, times 1.05.
lse: 1e-4 absolute, on the same scores."""
import numpy as np
import pytest

from oracle import paged

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


class Problem:
    """A ragged batch over a cache whose slots hold NaN except where a request's keys are."""

    def __init__(self, seed, new, kv, Hq, Hk, D, page, fp8=False, order="token", dead=None, qscale=1.0):
        g = np.random.default_rng(seed)
        self.new, self.kv, self.Hq, self.Hk, self.D, self.page, self.fp8 = new, kv, Hq, Hk, D, page, fp8
        B, T = len(new), int(sum(new))
        self.B, self.T = B, T
        need = [max(1, -(-x // page)) for x in kv]
        pages = sum(need) + 2
        ids = g.permutation(pages)
        width = max(need) + 2
        table = np.full((B, width), -7, dtype=np.int64)   # entries past a request's pages: never read
        at = 0
        for b in range(B):
            table[b, :need[b]] = ids[at:at + need[b]]
            at += need[b]
        self.table = table
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
        self.k_scale = self.v_scale = None
        shape = (pages, page, Hk, D)
        live = np.zeros((pages, page), dtype=bool)
        for b in range(B):
            j = np.arange(kv[b])
            live[table[b, j // page], j % page] = True
        if dead is not None:                              # slots before a window: freed, reused
            for b in range(B):
                j = np.arange(max(0, dead[b]))
                live[table[b, j // page], j % page] = False
        vals = []
        for _ in range(2):
            x = g.standard_normal(shape).astype(np.float32)
            t = torch.from_numpy(x * (16 if fp8 else 1)).to(torch.float8_e4m3fn if fp8 else torch.bfloat16)
            vals.append(t.float().numpy().astype(np.float64))
            raw = t.view(torch.uint8 if fp8 else torch.int16).clone()
            raw[torch.from_numpy(~live)] = 0x7F if fp8 else 0x7FC0
            t = raw.view(t.dtype).cuda()
            if order == "head":
                t = t.transpose(1, 2).contiguous().transpose(1, 2)
            setattr(self, "kc" if len(vals) == 1 else "vc", t)
        if fp8:
            self.k_scale = torch.linspace(0.05, 0.08, Hk, device="cuda")
            self.v_scale = torch.linspace(0.09, 0.04, Hk, device="cuda")
            vals[0] = vals[0] * self.k_scale.cpu().numpy()[:, None].astype(np.float64)
            vals[1] = vals[1] * self.v_scale.cpu().numpy()[:, None].astype(np.float64)
        self.kv64 = vals
        q = torch.from_numpy((g.standard_normal((max(T, 1), Hq, D)) * qscale).astype(np.float32)).to(torch.bfloat16)[:T]
        self.q64 = q.double().numpy()
        wide = torch.zeros((T, Hq * D + 72), dtype=torch.bfloat16)   # rows apart
        wide[:, 8:8 + Hq * D] = q.reshape(T, Hq * D)
        self.q = wide.cuda()[:, 8:8 + Hq * D].view(T, Hq, D)

    def run(self, lb, causal=True, window=0, scale=None, ctas_ws=None, stream=None, lse=True):
        c = lb.lowbit_paged_cache(self.kc, self.vc, self.k_scale, self.v_scale)
        out = torch.full((self.T + 2, self.Hq, self.D), 7.0, dtype=torch.bfloat16, device="cuda")
        ls = torch.full((self.T + 2, self.Hq), 7.0, device="cuda")
        ws = torch.full((lb.lowbit_paged_attention_workspace_bytes(self.T, self.B, self.Hq, self.Hk, self.D),),
                        0xFF, dtype=torch.uint8, device="cuda")
        lb.lowbit_paged_attention(self.q, c, i32(self.cu), i32(self.kv), i32(self.table), out[:self.T], ws,
                                  scale=scale, causal=causal, window=window, lse=ls[:self.T] if lse else None,
                                  stream=stream)
        torch.cuda.synchronize()
        assert (out[self.T:] == 7.0).all() and (ls[self.T:] == 7.0).all()
        return out[:self.T], ls[:self.T]

    def check(self, out, lse, causal=True, window=0, scale=None):
        scale = self.D ** -0.5 if scale is None else scale
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for b in range(self.B):
            n, kv = self.new[b], self.kv[b]
            if not n:
                continue
            k = paged.gather(self.kv64[0], self.table[b], kv, self.page)
            v = paged.gather(self.kv64[1], self.table[b], kv, self.page)
            see = paged.visible(n, kv, causal, window)
            rows = slice(self.cu[b], self.cu[b + 1])
            want, norm, spread = paged.attention(self.q64[rows], k, v, see, scale)
            top = np.abs(v[see.any(0)]).max() if see.any() else 0.0
            flat = kv * 2.0 ** -25 * top if self.fp8 else 0.0
            tol = 1.05 * ((2.0 ** -11 if self.fp8 else 2.0 ** -8) * spread + flat
                          + 2.0 ** -8 * np.abs(want) + 1e-4 * spread)
            err = np.abs(out[rows] - want)
            assert (err <= tol + 1e-30).all(), (b, float((err - tol).max()), np.argwhere(~(err <= tol))[:3])
            seen = np.isfinite(norm)
            assert (np.isneginf(lse[rows]) == ~seen).all()
            assert (np.abs(lse[rows][seen] - norm[seen]) <= 1e-4).all()
            assert (out[rows][~seen] == 0).all()


SHAPES = [  # new, kv, Hq, Hk, D, page
    ([1], [1], 4, 1, 64, 16),
    ([1], [777], 32, 8, 128, 16),
    ([1], [4097], 8, 8, 128, 64),
    ([16], [3001], 32, 8, 128, 64),
    ([1, 0, 1, 1], [5, 9, 64, 700], 10, 2, 128, 32),
    ([16, 3, 0, 31, 1], [16, 500, 77, 1030, 65], 16, 4, 64, 16),
    ([5, 7], [300, 129], 6, 2, 256, 8),
    ([1, 2], [130, 63], 8, 1, 256, 1),
    ([70, 1, 200], [70, 900, 333], 8, 2, 128, 128),
    ([129], [1500], 5, 1, 128, 1024),
    ([64, 65, 63, 1], [64, 65, 64, 128], 4, 4, 64, 64),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("order", ["token", "head"])
@pytest.mark.parametrize("shape", SHAPES)
def test_attention(lb, shape, fp8, order):
    pr = Problem(3, *shape, fp8=fp8, order=order)
    pr.check(*pr.run(lb))
    assert lb.lowbit_device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 1), (True, 100), (False, 100), (True, 65), (False, 64)])
@pytest.mark.parametrize("shape", [([16, 1, 40], [900, 513, 130], 16, 4, 64, 32),
                                   ([16, 200], [2000, 450], 8, 2, 128, 64),
                                   ([3, 20], [333, 140], 4, 2, 256, 16),
                                   ([1, 0, 2, 1], [700, 3, 130, 65], 16, 4, 128, 16),
                                   ([2, 1], [300, 80], 4, 1, 64, 64), ([1, 1], [129, 600], 8, 1, 256, 32)])
def test_masks(lb, shape, causal, window, fp8):
    new, kv = shape[:2]
    dead = [x - n - window + 1 if window else 0 for n, x in zip(new, kv)]
    pr = Problem(4, *shape, fp8=fp8, dead=dead)
    pr.check(*pr.run(lb, causal, window), causal, window)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,kv", [([4], [0]), ([4, 2], [2, 0]), ([100, 5], [3, 20]), ([0, 0], [5, 0])])
def test_rows_that_see_nothing(lb, new, kv, fp8):
    pr = Problem(5, new, kv, 8, 2, 128, 16, fp8=fp8)
    out, lse = pr.run(lb)
    pr.check(out, lse)
    pr.check(*pr.run(lb, False), False)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,kv,Hq,Hk,D", [([4, 2], [70, 33], 4, 2, 128), ([9], [200], 8, 4, 64), ([30], [500], 8, 2, 256),
                                            ([90], [300], 8, 2, 128), ([700], [900], 8, 2, 128), ([700], [700], 4, 1, 64)])
def test_hidden_keys_may_hold_anything(lb, new, kv, Hq, Hk, D, fp8):
    """A key that is NaN reaches the tokens that see it and no others (its value is finite)."""
    pr = Problem(14, new, kv, Hq, Hk, D, 16, fp8=fp8)
    bad = [n // 2 for n in new]                                   # the new token whose key is NaN
    for b, i in enumerate(bad):
        j = kv[b] - new[b] + i
        at = pr.kc[int(pr.table[b, j // 16]), j % 16]
        at.view(torch.uint8 if fp8 else torch.int16).fill_(0x7F if fp8 else 0x7FC0)
    out, lse = (x.double().cpu().numpy() for x in pr.run(lb))
    clean = Problem(14, new, kv, Hq, Hk, D, 16, fp8=fp8)
    out0, lse0 = (x.double().cpu().numpy() for x in clean.run(lb))
    for b, i in enumerate(bad):
        before, after = slice(pr.cu[b], pr.cu[b] + i), slice(pr.cu[b] + i, pr.cu[b + 1])
        assert np.array_equal(out[before], out0[before]) and np.array_equal(lse[before], lse0[before])
        assert np.isnan(out[after]).all()


def test_sharp_and_flat_scores(lb):
    """Scores far apart (one key takes all) and all equal; scale negative and zero."""
    for scale in (4.0, 0.0, -0.3):
        pr = Problem(6, [16], [1000], 8, 2, 128, 64, qscale=1.0)
        out, lse = pr.run(lb, scale=scale)
        want, norm, _ = paged.attention(pr.q64, paged.gather(pr.kv64[0], pr.table[0], 1000, 64),
                                        paged.gather(pr.kv64[1], pr.table[0], 1000, 64),
                                        paged.visible(16, 1000, True, 0), scale)
        # |s| up to 4 * 128: fp32 scores are good to 512 * 2^-23 * sqrt(128), which moves a weight
        # by that fraction of itself
        assert np.abs(out.double().cpu().numpy() - want).max() <= 2 * 2.0 ** -8 * 4.5 + 4.5e-3
        assert np.abs(lse.double().cpu().numpy() - norm).max() <= 1e-3


@pytest.mark.parametrize("fp8", [False, True])
def test_huge_and_tiny_queries(lb, fp8):
    """The power of two that takes queries into fp16 over an e4m3 cache changes nothing."""
    for f in (2.0 ** 40, 2.0 ** -40):
        pr = Problem(7, [3, 16], [200, 300], 8, 2, 128, 16, fp8=fp8)
        pr.q.mul_(f)
        pr.check(*pr.run(lb, scale=128 ** -0.5 / f))


def test_same_bits_every_time_and_on_another_stream(lb):
    pr = Problem(8, [16] * 9, [4000, 1, 17, 800, 2222, 64, 65, 3999, 16], 32, 8, 128, 64)
    a = pr.run(lb)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        b = pr.run(lb, stream=s)
        assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])
    c = pr.run(lb, lse=False)
    assert torch.equal(a[0].view(torch.int16), c[0].view(torch.int16))


def test_many_requests(lb):
    """More requests than a block has threads: the schedule's second pass."""
    g = np.random.default_rng(9)
    new = [int(x) for x in g.integers(0, 3, 700)]
    kv = [int(n + x) for n, x in zip(new, g.integers(0, 90, 700))]
    pr = Problem(9, new, kv, 4, 2, 64, 16)
    pr.check(*pr.run(lb))


def test_bad_batches_are_recorded_and_skipped(lb):
    pr = Problem(10, [2, 3], [40, 50], 4, 2, 64, 16)
    good, _ = pr.run(lb)
    bad = [("cu", np.array([0, -1, 5])), ("cu", np.array([0, 2, 9])), ("kv", [40, 10 ** 6]), ("kv", [40, -3])]
    for name, value in bad:
        keep = getattr(pr, name)
        setattr(pr, name, value)
        out, _ = pr.run(lb)
        assert lb.lowbit_device_error() == 1
        if name == "kv":
            assert torch.equal(out[:2], good[:2]) and (out[2:] == 7.0).all()
        setattr(pr, name, keep)
    for page in (-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31):
        keep = pr.table.copy()
        pr.table[1, 1] = page
        out, _ = pr.run(lb)
        assert lb.lowbit_device_error() == 1
        assert torch.equal(out[:2], good[:2])
        pr.table = keep


# ------------------------------------------------------------------------------------ append


def append_case(lb, seed, new, kv, Hq, Hk, D, page, rot, inter, fp8, order, apart=True, inplace=False):
    g = np.random.default_rng(seed)
    T, B = int(sum(new)), len(new)
    need = [max(1, -(-x // page)) for x in kv]
    pages = sum(need) + 1
    ids = g.permutation(pages)
    table = np.full((B, max(need)), -1, dtype=np.int64)
    at = 0
    for b in range(B):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
    cu = np.concatenate([[0], np.cumsum(new)])
    wide = torch.from_numpy(g.standard_normal((T, (Hq + 2 * Hk) * D + 8)).astype(np.float32)).to(torch.bfloat16).cuda()
    q = wide[:, :Hq * D].view(T, Hq, D)
    k = wide[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    v = wide[:, (Hq + Hk) * D:(Hq + 2 * Hk) * D].view(T, Hk, D)
    if not apart:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    host = [t.float().cpu().numpy() for t in (q, k, v)]
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    kc = torch.full((pages, page, Hk, D) if order == "token" else (pages, Hk, page, D), 3.0, device="cuda").to(dt)
    vc = torch.full_like(kc, 5.0) if not fp8 else torch.full(kc.shape, 5.0, device="cuda").to(dt)
    if order == "head":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    sc = [torch.rand(Hk, device="cuda") + 0.01 for _ in range(2)] if fp8 else [None, None]
    cache = lb.lowbit_paged_cache(kc, vc, *sc)
    rope = None
    if rot:
        a = np.arange(max(kv) + 1)[:, None] * (1.0 / 10000.0 ** (np.arange(0, rot, 2) / rot))[None]
        rope = torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).cuda()
    q_out = q if inplace else torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    lb.lowbit_kv_append(q, k, v, rope, i32(cu), i32(kv), i32(table), cache, q_out, interleaved=inter)
    torch.cuda.synchronize()
    req, pos = paged.positions(cu, kv)
    rows = rope.cpu().numpy()[pos] if rot else np.zeros((T, 0), dtype=np.float32)
    wq, wk = (paged.rotate(x, rows, inter) if rot else x for x in host[:2])
    assert torch.equal(q_out.cpu().view(torch.int16), torch.from_numpy(wq).to(torch.bfloat16).view(torch.int16))
    for got, want, s, fill in ((kc, wk, sc[0], 3.0), (vc, host[2], sc[1], 5.0)):
        ref = torch.full((pages, page, Hk, D), fill).to(dt)
        x = torch.from_numpy(want)
        if fp8:
            x = (x / s.cpu()[:, None]).clamp(-448, 448)
        ref.view(torch.uint8 if fp8 else torch.int16)[torch.from_numpy(table[req, pos // page]),
                                                      torch.from_numpy(pos % page)] = \
            x.to(dt).view(torch.uint8 if fp8 else torch.int16)
        bits = torch.uint8 if fp8 else torch.int16
        assert torch.equal(got.cpu().contiguous().view(bits), ref.view(bits))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("new,kv,Hq,Hk,D,page,rot,order", [
    ([1], [1], 4, 1, 64, 16, 64, "token"),
    ([1], [4000], 32, 8, 128, 64, 128, "head"),
    ([16, 0, 3, 1], [900, 5, 3, 129], 32, 8, 128, 16, 64, "head"),
    ([300, 41], [301, 1000], 8, 2, 128, 32, 128, "token"),
    ([5, 6], [5, 70], 6, 3, 256, 1, 256, "token"),
    ([9], [33], 5, 1, 256, 8, 16, "head"),
    ([7], [7], 3, 3, 64, 1024, 0, "token")])
def test_append(lb, new, kv, Hq, Hk, D, page, rot, order, inter, fp8):
    append_case(lb, 11, new, kv, Hq, Hk, D, page, rot, inter, fp8, order)


def test_append_many_requests_and_in_place(lb):
    g = np.random.default_rng(12)
    new = [int(x) for x in g.integers(0, 3, 600)]
    kv = [n + int(x) for n, x in zip(new, g.integers(0, 40, 600))]
    append_case(lb, 12, new, kv, 4, 2, 64, 8, 64, False, False, "token")
    append_case(lb, 13, [5, 3], [9, 20], 4, 2, 64, 8, 32, True, False, "token", apart=False, inplace=True)


def test_append_saturates_and_keeps_nan(lb):
    D = 64
    k = torch.zeros((1, 1, D), dtype=torch.bfloat16, device="cuda")
    k[0, 0, :4] = torch.tensor([1e6, -1e6, float("nan"), float("inf")])
    kc = torch.zeros((1, 4, 1, D), device="cuda").to(torch.float8_e4m3fn)
    vc = kc.clone()
    lb.lowbit_kv_append(None, k, k, None, i32([0, 1]), i32([2]), i32([[0]]), lb.lowbit_paged_cache(kc, vc), None)
    got = kc.float()[0, 1, 0, :4].cpu()
    assert got[0] == 448 and got[1] == -448 and torch.isnan(got[2]) and got[3] == 448
    assert (kc.float()[0, 0] == 0).all() and (kc.float()[0, 2:] == 0).all()


def test_append_bad_places_are_recorded_and_skipped(lb):
    D, T = 64, 3
    x = torch.ones((T, 1, D), dtype=torch.bfloat16, device="cuda")
    rope = torch.zeros((6, D), device="cuda")
    rope[:, :D // 2] = 1
    for cu, kv, table, rows, done in (
            ([0, 3], [3], [[5]], 6, 0),            # page outside the cache
            ([0, 3], [3], [[-1]], 6, 0),
            ([0, 3], [30], [[0]], 6, 0),           # more keys than the table's pages hold
            ([0, 3], [2], [[0]], 6, 2),            # position -1: the two others are appended
            ([0, 3], [8], [[0]], 6, 1),            # positions 6 and 7 are past the table of angles
            ([0, 4], [4], [[0]], 6, 0),            # rows past the arrays
            ([2, 1], [4], [[0]], 6, 0)):
        kc = torch.zeros((2, 8, 1, D), dtype=torch.bfloat16, device="cuda")
        c = lb.lowbit_paged_cache(kc, kc.clone())
        lb.lowbit_kv_append(None, x, x, rope, i32(cu), i32(kv), i32(table), c, None)
        err = lb.lowbit_device_error()
        assert err == 1 or cu[0] == 2      # rows that belong to nobody are no error
        assert int((kc[..., 0] != 0).sum()) == done


def test_rows_of_nobody_are_left_alone(lb):
    """T may be padded past cu_q[B], as captured graphs do."""
    D = 64
    x = torch.ones((5, 2, D), dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros((2, 8, 2, D), dtype=torch.bfloat16, device="cuda")
    c = lb.lowbit_paged_cache(kc, kc.clone())
    q_out = torch.full((5, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lb.lowbit_kv_append(x, x, x, None, i32([0, 2]), i32([3]), i32([[1]]), c, q_out)
    assert (q_out[:2] == 1).all() and (q_out[2:] == 7).all()
    assert int((kc[1, :, 0, 0] != 0).sum()) == 2 and not kc[0].any()
    out = torch.full((5, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(lb.lowbit_paged_attention_workspace_bytes(5, 1, 2, 2, D), dtype=torch.uint8, device="cuda")
    lb.lowbit_paged_attention(x, c, i32([0, 2]), i32([3]), i32([[1]]), out, ws)
    assert (out[2:] == 7).all() and torch.isfinite(out).all() and (out[:2] != 7).any()
    assert lb.lowbit_device_error() == 0


def test_far_offsets(lb):
    """Page offsets past 2^31 elements: a cache of 6 GB, of which the last pages are used."""
    D, Hk, page = 128, 8, 64
    pages = 2 ** 31 // (page * Hk * D) + 3000
    kc = torch.empty((pages, page, Hk, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    g = torch.Generator(device="cuda").manual_seed(1)
    kv = 150
    k, v = (torch.randn((kv, Hk, D), device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    table = [[pages - 1, 0, pages - 3]]
    cache = lb.lowbit_paged_cache(kc, vc)
    lb.lowbit_kv_append(None, k, v, None, i32([0, kv]), i32([kv]), i32(table), cache, None)
    assert torch.equal(kc[pages - 3, kv - 129], k[kv - 1])
    q = torch.randn((4, 32, D), device="cuda", generator=g).to(torch.bfloat16)
    out = torch.empty_like(q)
    ws = torch.empty(lb.lowbit_paged_attention_workspace_bytes(4, 1, 32, Hk, D), dtype=torch.uint8, device="cuda")
    lb.lowbit_paged_attention(q, cache, i32([0, 4]), i32([kv]), i32(table), out, ws)
    want, _, spread = paged.attention(q.double().cpu().numpy(), k.double().cpu().numpy(), v.double().cpu().numpy(),
                                      paged.visible(4, kv, True, 0), D ** -0.5)
    assert (np.abs(out.double().cpu().numpy() - want) <= 1.05 * (2.0 ** -8 * (spread + np.abs(want)) + 1e-4 * spread)).all()
    assert lb.lowbit_device_error() == 0

"""GPU parity of lowbit_kv_append_norm with the fp64 oracle.

Tolerance, per element y of a head of D, with size = |a cos| + |b sin| of its pair (|y| where nothing turns):
  the sum of D squares in fp32, D 2^-24 of it at most, of which the root halves the share: 2^-17 for D = 256;
  the reciprocal root 2 ulp, two products and the rotation's two products and sum: under 2^-20 in all;
  together under 2^-16 of size; then the stored rounding, half a step of the type: 2^-8 of the value for
  bf16, 2^-4 for e4m3, whose steps below 2^-6 are 2^-9 (half of one: 2^-10)."""
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
    assert lb.lowbit_device_error() == 0


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def within(got, want, size, fp8=False):
    """Element by element; got of the stored type."""
    got = got.float().cpu().double().numpy()
    step = 2.0 ** -4 if fp8 else 2.0 ** -8
    room = 2.0 ** -16 * size + step * np.abs(want) + (2.0 ** -10 if fp8 else 0.0)
    bad = ~(np.abs(got - want) <= room * 1.001)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(np.abs(got - want).max()))


class Case:
    def __init__(self, seed, new, kv, Hq, Hk, D, page, rot, inter=False, fp8=False, order="token", scale=2.0):
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
        self.T, self.D, self.fp8, self.inter = T, D, fp8, inter
        wide = g.standard_normal((T, (Hq + 2 * Hk) * D + 8)) * scale
        wide = torch.from_numpy(wide).to(torch.bfloat16).cuda()
        self.q = wide[:, :Hq * D].view(T, Hq, D) if Hq else None
        self.k = wide[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        self.v = wide[:, (Hq + Hk) * D:(Hq + 2 * Hk) * D].view(T, Hk, D)
        self.qw, self.kw = (torch.from_numpy(1 + 0.4 * g.standard_normal(D)).float().cuda() for _ in range(2))
        dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
        shape = (pages, page, Hk, D) if order == "token" else (pages, Hk, page, D)
        self.kc, self.vc = (torch.full(shape, x, device="cuda").to(dt) for x in (3.0, 5.0))
        if order == "head":
            self.kc, self.vc = self.kc.transpose(1, 2), self.vc.transpose(1, 2)
        self.sc = [torch.rand(Hk, device="cuda") * 0.1 + 0.02 for _ in range(2)] if fp8 else [None, None]
        self.cache = lambda lb: lb.lowbit_paged_cache(self.kc, self.vc, *self.sc)
        self.rope = None
        if rot:
            a = np.arange(max(kv) + 1)[:, None] * (1.0 / 10000.0 ** (np.arange(0, rot, 2) / rot))[None]
            self.rope = torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).cuda()
        self.cu, self.kv, self.table = i32(cu), i32(kv), i32(table)
        self.req, self.pos = paged.positions(cu, kv)
        self.page, self.host_table = page, table
        self.q_out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda") if Hq else None

    def run(self, lb, qw=True, kw=True, eps=1e-6, stream=None):
        lb.lowbit_kv_append_norm(self.q, self.k, self.v, self.qw if qw else None, self.kw if kw else None, eps, self.rope,
                                 self.cu, self.kv, self.table, self.cache(lb), self.q_out, interleaved=self.inter,
                                 stream=stream)

    def want(self, x, weight, eps):
        y = x.double().cpu().numpy()
        if weight is not None:
            y = paged.normalise(y, weight.cpu().numpy(), eps)
        rows = self.rope.cpu().numpy()[self.pos] if self.rope is not None else np.zeros((self.T, 0))
        return paged.rotate64(y, rows, self.inter)

    def stored(self, cache):
        return cache.float().cpu()[torch.from_numpy(self.host_table[self.req, self.pos // self.page]),
                                   torch.from_numpy(self.pos % self.page)]

    def check(self, lb, qw=True, kw=True, eps=1e-6):
        q, k = (None if self.q is None else self.q.clone()), self.k.clone()
        self.run(lb, qw, kw, eps)
        torch.cuda.synchronize()
        if q is not None:
            within(self.q_out, *self.want(q, self.qw if qw else None, eps))
        y, size = self.want(k, self.kw if kw else None, eps)
        got = self.stored(self.kc)
        if self.fp8:
            s = self.sc[0].cpu().double().numpy()[:, None]
            y, size = np.clip(y / s, -448, 448), size / s
        within(got, y, size, self.fp8)
        # values and every other slot: bits of the plain append
        v = self.v.float().cpu()
        if self.fp8:
            v = (v / self.sc[1].cpu()[:, None]).clamp(-448, 448)
        assert torch.equal(self.stored(self.vc), v.to(self.vc.dtype).float())
        for c, fill in ((self.kc, 3.0), (self.vc, 5.0)):
            rest = c.float().cpu().clone()
            rest[torch.from_numpy(self.host_table[self.req, self.pos // self.page]), torch.from_numpy(self.pos % self.page)] = fill
            assert (rest == fill).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("new,kv,Hq,Hk,D,page,rot,order", [
    ([1], [1], 4, 1, 64, 16, 64, "token"),
    ([1], [4000], 32, 8, 128, 64, 128, "head"),
    ([16, 0, 3, 1], [900, 5, 3, 129], 32, 8, 128, 16, 64, "head"),
    ([300, 41], [301, 1000], 9, 3, 128, 32, 128, "token"),
    ([5, 6], [5, 70], 6, 3, 256, 1, 256, "token"),
    ([9], [33], 5, 1, 256, 8, 16, "head"),
    ([7], [7], 3, 3, 64, 1024, 0, "token"),
    ([456, 1], [501, 9], 5, 1, 64, 64, 32, "token"),         # four warps a token, two, one
    ([911, 3], [1000, 3], 5, 3, 128, 64, 96, "head"),
    ([2001, 1], [2001, 9], 3, 1, 64, 64, 32, "token"),
    ([3, 2500], [77, 2600], 5, 2, 128, 16, 128, "head"),
    ([1030, 1031], [1030, 1100], 2, 1, 256, 32, 64, "head")])
def test_parity(lb, new, kv, Hq, Hk, D, page, rot, order, inter, fp8):
    Case(31, new, kv, Hq, Hk, D, page, rot, inter, fp8, order).check(lb)


@pytest.mark.parametrize("T", [3, 2100])
def test_one_side_alone(lb, T):
    Case(1, [T], [T + 5], 4, 2, 128, 32, 128).check(lb, qw=False)
    Case(2, [T], [T + 5], 4, 2, 128, 32, 128).check(lb, kw=False)
    Case(3, [T], [T + 5], 0, 2, 64, 32, 64).check(lb, qw=False)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [5, 2050])
def test_without_weights_the_bits_are_the_plain_append_s(lb, T, fp8):
    a, b = (Case(4, [T, 2], [T + 9, 40], 6, 3, 128, 16, 64, fp8=fp8, order="head") for _ in range(2))
    b.sc = a.sc
    a.run(lb, qw=False, kw=False)
    lb.lowbit_kv_append(b.q, b.k, b.v, b.rope, b.cu, b.kv, b.table, b.cache(lb), b.q_out)
    for x, y in ((a.q_out, b.q_out), (a.kc, b.kc), (a.vc, b.vc)):
        assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


def test_equal_calls_give_equal_bits_and_heads_do_not_mix(lb):
    """A row's result does not depend on the rows beside it, nor on how many warps a token has."""
    big = Case(5, [2300], [2300], 7, 2, 128, 64, 128)
    big.run(lb)
    few = Case(5, [2300], [2300], 7, 2, 128, 64, 128)
    few.T = 11
    few.q, few.k, few.v, few.q_out = few.q[100:111], few.k[100:111], few.v[100:111], few.q_out[100:111]
    few.cu, few.kv = i32([0, 11]), i32([111])
    few.run(lb)
    assert torch.equal(big.q_out[100:111].view(torch.int16), few.q_out.view(torch.int16))


def test_in_place(lb):
    c = Case(6, [40], [50], 4, 2, 128, 16, 128)
    q = c.q.contiguous()
    c.run(lb)
    lb.lowbit_kv_append_norm(q, c.k, c.v, c.qw, c.kw, 1e-6, c.rope, c.cu, c.kv, c.table, c.cache(lb), q)
    assert torch.equal(q.view(torch.int16), c.q_out.view(torch.int16))


def test_zero_heads_eps_and_values_that_are_not_finite(lb):
    D, T = 64, 6
    x = torch.randn((T, 1, D), device="cuda").to(torch.bfloat16)
    x[0] = 0
    x[1, 0, 3] = float("inf")
    x[2, 0, 5] = float("nan")
    x[3] = 2.0 ** 70                      # squares past fp32: zeros
    x[4] = 2.0 ** -60                     # far below eps: x / sqrt(eps)
    one = torch.ones(D, device="cuda")
    kc = torch.zeros((2, 8, 1, D), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(x)
    cache = lb.lowbit_paged_cache(kc, kc.clone())
    args = (None, i32([0, T]), i32([T]), i32([[1]]), cache, out)
    lb.lowbit_kv_append_norm(x, x, x, one, one, 1e-6, *args)
    y = out.float().cpu()[:, 0]
    assert (y[0] == 0).all()
    assert torch.isnan(y[1, 3]) and (y[1, :3] == 0).all() and torch.isnan(y[2]).all()
    assert (y[3] == 0).all()
    assert torch.allclose(y[4], torch.full((D,), 2.0 ** -60 * 1000), rtol=2.0 ** -8)
    assert torch.isfinite(y[5]).all()     # its neighbours are not reached
    lb.lowbit_kv_append_norm(x, x, x, one, one, 0.0, *args)
    assert torch.isnan(out[0]).all()


def test_bad_places_are_recorded_and_skipped(lb):
    D, T = 64, 3
    x = torch.ones((T, 1, D), dtype=torch.bfloat16, device="cuda")
    one = torch.ones(D, device="cuda")
    rope = torch.zeros((6, D), device="cuda")
    rope[:, :D // 2] = 1
    for cu, kv, table, done in (([0, 3], [3], [[5]], 0), ([0, 3], [3], [[-1]], 0), ([0, 3], [30], [[0]], 0),
                                ([0, 3], [2], [[0]], 2), ([0, 3], [8], [[0]], 1), ([0, 4], [4], [[0]], 0),
                                ([2, 1], [4], [[0]], 0), ([0, 2], [2], [[0]], 2)):
        kc = torch.zeros((2, 8, 1, D), dtype=torch.bfloat16, device="cuda")
        out = torch.full_like(x, 7.0)
        lb.lowbit_kv_append_norm(x, x, x, one, one, 0.0, rope, i32(cu), i32(kv), i32(table), lb.lowbit_paged_cache(kc, kc.clone()), out)
        err = lb.lowbit_device_error()
        assert err == 1 or cu[0] == 2 or cu[1] == 2
        assert int((kc[..., 0] != 0).sum()) == done and int((out[:, 0, 0] == 7).sum()) == T - done


def test_graph_and_other_stream(lb):
    c = Case(7, [9, 1], [30, 8], 8, 2, 128, 16, 128)
    c.run(lb)
    want = c.q_out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.q_out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    c.run(lb, stream=side)
    side.synchronize()
    assert torch.equal(c.q_out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(lb)
    for _ in range(2):
        c.q_out.zero_()
        graph.replay()
        assert torch.equal(c.q_out, want)


@pytest.mark.parametrize("change,kind", [
    (dict(q_weight=lambda t: t.bfloat16()), TypeError), (dict(q_weight=lambda t: t[:-1]), ValueError),
    (dict(k_weight=lambda t: t.cpu()), TypeError), (dict(k_weight=lambda t: torch.stack([t, t], 1)[:, 0]), TypeError),
    (dict(eps=lambda e: "x"), TypeError), (dict(eps=lambda e: -1e-6), 1), (dict(eps=lambda e: float("nan")), 1),
    (dict(eps=lambda e: float("inf")), 1), (dict(q=lambda t: None, q_out=lambda t: None), 1),
    (dict(q_weight=lambda t: torch.ones(129, device="cuda")[1:]), 3), (dict(q=lambda t: None), ValueError)])
def test_refusals(lb, change, kind):
    c = Case(8, [2], [9], 4, 2, 128, 16, 128)
    a = dict(q=c.q, k=c.k, v=c.v, q_weight=c.qw, k_weight=c.kw, eps=1e-6, rope=c.rope, cu_q=c.cu, kv_lens=c.kv,
             block_table=c.table, cache=c.cache(lb), q_out=c.q_out)
    for name, f in change.items():
        a[name] = f(a[name])
    if isinstance(kind, int):
        with pytest.raises(lb.LowbitError) as e:
            lb.lowbit_kv_append_norm(**a)
        assert e.value.status == kind
    else:
        with pytest.raises(kind):
            lb.lowbit_kv_append_norm(**a)

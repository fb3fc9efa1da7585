"""GPU checks of lowbit_verify_drafts.

As in lowbit_sample every sum is one of whole numbers, and every product and difference before it is
rounded by itself, so the outcome is a function of the fp32 weights alone: with torch's own exponential the counts
and tokens of `plain` below must be met exactly, the acceptance probabilities to one rounding (2^-24, of numbers
up to 1).  Against the fp64 oracle a weight is off by 2^-21 of itself at most, so a probability by 2^-20: a decision
may differ where u q and p are closer than 2^-19 of p, and a token where v of the mass falls within 1e-5 of
a boundary, once the rest after a rejection (a difference, of at least `least`) has been divided by."""
import numpy as np
import pytest

from oracle import drafts as od, sample as osample

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


def f32(x):
    return torch.tensor(x, dtype=torch.float32, device="cuda")


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


PLAIN = (1.0, 0, 1.0, 0.0)


def kept(z, settings):
    """(weights, masses) that the settings leave of one row, fp32 and whole numbers, zeros elsewhere."""
    temp, k, p, mp = settings
    z = torch.where(torch.isnan(z), -torch.inf, z.float()).clamp(max=torch.finfo(torch.float32).max)
    V = z.numel()
    if z.max() == -torch.inf:
        return torch.zeros_like(z), torch.zeros(V, dtype=torch.int64, device="cuda")
    greedy = not temp >= 1e-6
    w = torch.exp((z - z.max()) * (1.0 / f32(1.0 if greedy else min(temp, 1e6))))
    w = torch.where(z == -torch.inf, 0.0, w)
    mass = (w * 2.0 ** 40).round().long()
    order = torch.sort(z, descending=True, stable=True).indices
    order = order[:1 if greedy else (k if 0 < k <= V else V)]
    m = mass[order]
    if not p >= 1.0:
        limit = max(1, int((f32(p).double() * m.sum().double()).ceil()))
        order = order[m.cumsum(0) - m < limit]
    keep = torch.zeros_like(mass)
    keep[order] = mass[order]
    if mp > 0:
        keep[w < f32(min(mp, 1.0))] = 0
    return torch.where(keep > 0, w, 0.0), keep


def draw(mass, v):
    total = int(mass.sum())
    if not total:
        return -1
    v = 0.0 if np.isnan(v) else min(max(v, 0.0), 1.0)
    aim = min(int(np.floor(np.float64(np.float32(v)) * np.float64(total))), total - 1)
    return int((mass.cumsum(0) <= aim).sum())


def plain(c, b):
    """Request b in whole numbers: (accepted, tokens, acceptance probabilities)."""
    c0, c1 = int(c.cu[b]), int(c.cu[b + 1])
    n, V = c1 - c0, c.z.shape[1]
    accept, bad = [], n
    for i in range(n):
        d = int(c.drafts[c0 + i])
        _, m = kept(c.z[c0 + b + i], c.settings[b])
        share = float(m[d]) / float(max(1, int(m.sum()))) if 0 <= d < V else 0.0
        given = 1.0
        if c.y is not None:
            _, mq = kept(c.y[c0 + i], c.draft_settings[b])
            col = (int(c.index[d]) if c.index is not None else d) if 0 <= d < V else -1
            given = float(mq[col]) / float(max(1, int(mq.sum()))) if 0 <= col < mq.numel() else 0.0
        u = float(np.float32(c.u[c0 + i]))
        u = 0.0 if np.isnan(u) else min(max(u, 0.0), 1.0)
        accept.append(min(1.0, share / given) if given > 0 else float(share > 0))
        if bad == n and not u * given < share:
            bad = i
    w, mass = kept(c.z[c0 + b + bad], c.settings[b])
    if bad < n and int(mass.sum()):
        x = w * (2.0 ** 40 / mass.sum().double()).float()
        if c.y is None:
            d = int(c.drafts[c0 + bad])
            if 0 <= d < V:
                x[d] -= 1.0
        else:
            wq, mq = kept(c.y[c0 + bad], c.draft_settings[b])
            q = wq * (2.0 ** 40 / mq.sum().double()).float() if int(mq.sum()) else wq
            over = torch.zeros_like(x)
            if c.index is None:
                over[:min(V, q.numel())] = q[:V]
            else:
                has = (c.index >= 0) & (c.index < q.numel())
                over[has] = q[c.index[has].long()]
            x = x - over
        rest = (x.clamp(min=0) * 2.0 ** 40).round().long()
        if int(rest.sum()):
            mass = rest
    tokens = [int(x) for x in c.drafts[c0:c0 + bad]] + [draw(mass, c.v[b])]
    return bad, tokens + [-1] * (n + 1 - len(tokens)), accept


class Case:
    """Requests of `n` drafts each over random rows; drafts are drawn from the drafter, or its likeliest."""

    def __init__(self, seed, n, V, Vd=None, bf16=False, draft_bf16=None, settings=None, draft_settings=None, certain=False,
                 near=0.6, pad=3, index=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        B, N = len(n), int(sum(n))
        self.n, self.B, self.N, self.M = n, B, N, N + B
        self.cu = np.concatenate([[0], np.cumsum(n)])
        Vd = Vd or V
        dt, ddt = (torch.bfloat16 if x else torch.float32 for x in (bf16, bf16 if draft_bf16 is None else draft_bf16))
        z = 2.5 * torch.randn((self.M, V + pad), device="cuda", generator=g)      # rows apart
        hot = torch.randint(0, V, (self.M, 6), device="cuda", generator=g)
        z.scatter_(1, hot + pad // 2, 9 + torch.randn((self.M, 6), device="cuda", generator=g))
        self.z = z.to(dt)[:, pad // 2:V + pad // 2]
        self.index = None
        cols = torch.arange(V, device="cuda")
        if index or Vd < V:
            cols = torch.randperm(V, device="cuda", generator=g)[:Vd]
            self.index = torch.full((V,), -1, dtype=torch.int32, device="cuda")
            self.index[cols] = torch.arange(Vd, dtype=torch.int32, device="cuda")
        judge = torch.tensor([int(self.cu[b]) + b + i for b in range(B) for i in range(n[b])], device="cuda", dtype=torch.long)
        y = self.z[judge].float()[:, cols[:min(V, Vd)]]
        if Vd > V:
            y = torch.cat([y, torch.zeros((N, Vd - V), device="cuda")], 1)
        y = y + near * torch.randn(y.shape, device="cuda", generator=g)
        self.y = None if certain else y.to(ddt)
        self.settings = [PLAIN] * B if settings is None else [settings[b % len(settings)] for b in range(B)]
        self.draft_settings = [PLAIN] * B if draft_settings is None else [draft_settings[b % len(draft_settings)] for b in range(B)]
        if certain or not N:
            pick = y.argmax(1) if N else torch.zeros(0, dtype=torch.long, device="cuda")
        else:
            pick = torch.multinomial(torch.softmax(self.y.float(), 1), 1, generator=g)[:, 0]
        self.drafts = (cols[pick.clamp(max=cols.numel() - 1)] if Vd <= V else pick).to(torch.int32)
        self.u, self.v = (rng.random(x).astype(np.float32) for x in (N, B))

    def args(self, lb):
        def cols(s):
            return (f32([float(x[0]) for x in s]), i32([x[1] for x in s]), f32([x[2] for x in s]), f32([x[3] for x in s]))
        t, k, p, mp = cols(self.settings)
        self.n_accept = torch.full((self.B + 1,), -9, dtype=torch.int32, device="cuda")
        self.ids = torch.full((self.z.shape[0] + 1,), -9, dtype=torch.int32, device="cuda")
        self.accept = torch.full((self.drafts.numel() + 1,), 5.0, device="cuda")
        a = dict(logits=self.z, cu_drafts=i32(self.cu), drafts=self.drafts, u=f32(self.u), v=f32(self.v),
                 n_accept=self.n_accept[:-1], ids=self.ids[:-1], accept=self.accept[:-1], temperature=t, top_k=k, top_p=p, min_p=mp,
                 workspace=torch.full((lb.lowbit_verify_drafts_workspace_bytes(self.z.shape[0], self.drafts.numel()),), 0xFF,
                                      dtype=torch.uint8, device="cuda"))
        if self.y is not None:
            t, k, p, mp = cols(self.draft_settings)
            a |= dict(draft_logits=self.y, draft_index=self.index, draft_temperature=t, draft_top_k=k, draft_top_p=p, draft_min_p=mp)
        return a

    def run(self, lb, **kw):
        lb.lowbit_verify_drafts(**(self.args(lb) | kw))
        torch.cuda.synchronize()
        assert self.n_accept[-1] == -9 and self.ids[-1] == -9 and self.accept[-1] == 5.0
        return self.n_accept[:-1].tolist(), self.ids[:-1].tolist(), self.accept[:-1].tolist()

    def check(self, lb):
        got, ids, accept = self.run(lb)
        for b in range(self.B):
            c0, c1 = int(self.cu[b]), int(self.cu[b + 1])
            want = plain(self, b)
            assert (got[b], ids[c0 + b:c1 + b + 1]) == want[:2], (b, self.settings[b], got[b], want)
            assert np.abs(np.array(accept[c0:c1]) - np.array(want[2])).max(initial=0.0) <= 2.0 ** -24
        return got, ids, accept

    def check_oracle(self, lb):
        got, ids, accept = self.run(lb)
        sure = 0
        for b in range(self.B):
            c0, c1 = int(self.cu[b]), int(self.cu[b + 1])
            index = None if self.index is None else self.index.cpu().numpy()
            host = lambda t: t.float().cpu().numpy()  # noqa: E731
            rows = [host(self.z[c0 + b + i]) for i in range(c1 - c0 + 1)]
            given = [od.proposal(len(rows[0]), int(self.drafts[c0 + i]), None if self.y is None else host(self.y[c0 + i]),
                                 self.draft_settings[b], index) for i in range(c1 - c0)]
            n, tokens, prob = od.verify(rows, [int(x) for x in self.drafts[c0:c1]], self.u[c0:c1], self.v[b], self.settings[b], given)
            assert np.abs(np.array(accept[c0:c1]) - np.array(prob)).max(initial=0.0) <= 2.0 ** -19
            near = [abs(float(self.u[c0 + i]) * given[i][1] - od.ratio(od.shares(rows[i], self.settings[b]), given[i][1],
                                                                       int(self.drafts[c0 + i]))[0]) for i in range(c1 - c0)]
            if any(x < 2.0 ** -19 for x in near):
                continue
            assert got[b] == n
            p = od.shares(rows[n], self.settings[b])
            last = p if n == c1 - c0 else od.rest(p, given[n][0])
            cum = np.cumsum(last) / last.sum()
            if np.abs(cum - float(self.v[b])).min() * last.sum() < 1e-5:
                continue
            sure += 1
            assert ids[c0 + b:c1 + b + 1] == tokens
        return sure


SETTINGS = [PLAIN, (0.7, 20, 0.95, 0.0), (1.3, 0, 0.9, 0.0), (0.5, 300, 1.0, 0.0), (1.0, 0, 1.0, 0.05), (0.9, 50, 0.8, 0.02),
            (0.0, 40, 0.5, 0.1), (2.0, 1, 1.0, 0.0), (1.0, 10 ** 9, 0.999, 0.0), (1.0, -3, 0.0, 0.0), (50.0, 0, 0.5, 0.0),
            (1e9, 0, 1.0, 0.0), (float("nan"), 0, 1.0, 0.0), (1.0, 0, 1.0, 1.0), (1.0, 100000, 0.5, 0.0), (1.0, 3000, 1.0, 0.0)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("how", ["certain", "full", "index", "trimmed"])
@pytest.mark.parametrize("V", [2, 31, 1000, 4097, 32768, 70001])
def test_settings(lb, V, how, bf16):
    n = [3, 0, 1, 4, 2, 5, 1, 3, 2, 4, 1, 2, 3, 1, 2, 6]
    Case(V, n, V, Vd=max(1, V // 4) if how == "trimmed" else None, bf16=bf16, settings=SETTINGS, certain=how == "certain",
         index=how == "index").check(lb)


@pytest.mark.parametrize("bf16,draft_bf16", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("n,V,Vd", [([15], 248320, None), ([15, 7, 0], 248320, 32768), ([15] * 9, 248309, None),
                                    ([1] * 70, 131073, 5000), ([2] * 40, 33000, 33000)])
def test_sizes(lb, n, V, Vd, bf16, draft_bf16):
    """Every split of a row over CTAs, in both steps; rows that share no alignment."""
    Case(len(n) + V, n, V, Vd, bf16, draft_bf16, settings=SETTINGS, pad=0 if V % 8 == 0 else 3).check(lb)


@pytest.mark.parametrize("certain", [True, False])
def test_long_blocks(lb, certain):
    """More drafts than a CTA has threads, accepted to the last or rejected far in."""
    for n in (1022, 1023, 1024, 1500):
        c = Case(n, [n, 2], 40, certain=certain, near=0.1)
        c.u[:] = 0.0
        got, _, _ = c.check(lb)
        assert got == [n, 2]
        c.z[n - 3, int(c.drafts[n - 3])] = -torch.inf      # p = 0: never accepted
        assert c.check(lb)[0][0] == n - 3


@pytest.mark.parametrize("V", [1000, 70001])
def test_drafters_that_truncate(lb, V):
    c = Case(5, [4] * 16, V, settings=[PLAIN, (0.8, 40, 0.9, 0.0)], draft_settings=SETTINGS, near=1.5)
    c.check(lb)
    Case(6, [4] * 16, V, Vd=V // 3, settings=[(0.8, 40, 0.9, 0.0), PLAIN], draft_settings=SETTINGS, near=1.5).check(lb)


def test_ties_that_a_cut_goes_through(lb):
    """Equal logits at the cut: those of lower indices stay.  More of them than any list holds, over several CTAs."""
    for V, k, p in ((50000, 7000, 1.0), (50000, 49999, 1.0), (50000, 0, 0.37), (3000, 2500, 0.5), (50000, 20, 1.0)):
        c = Case(9, [2, 2, 2], V, certain=True, settings=[(1.0, k, p, 0.0)])
        c.z = c.z.clone()
        c.z[:] = 1.0
        c.z[:, 7::9] = 2.0
        edge = k - len(range(7, V, 9)) if k else 0
        c.drafts = i32([5, 8, V - 1, 0, max(0, edge), 3])
        c.u[:] = 0.0
        c.check(lb)
        c.u[:] = 1.0
        c.check(lb)


@pytest.mark.parametrize("how", ["certain", "full", "trimmed"])
def test_oracle(lb, how):
    sure = 0
    for seed in range(4):
        c = Case(40 + seed, [3, 0, 5, 1, 2, 4, 6, 2], 3001, Vd=900 if how == "trimmed" else None, certain=how == "certain",
                 settings=[PLAIN, (0.7, 20, 0.95, 0.0), (1.2, 0, 0.9, 0.0), (0.9, 0, 1.0, 0.01)])
        sure += c.check_oracle(lb)
    assert sure >= 28


def test_no_drafts_is_lowbit_sample(lb):
    c = Case(11, [0] * 16, 70001, settings=SETTINGS)
    got, ids, _ = c.run(lb, draft_logits=None, draft_index=None, draft_temperature=None, draft_top_k=None, draft_top_p=None,
                        draft_min_p=None)
    want = torch.empty(16, dtype=torch.int32, device="cuda")
    a = c.args(lb)
    lb.lowbit_sample(c.z, a["v"], want, a["temperature"], a["top_k"], a["top_p"], a["min_p"])
    assert got == [0] * 16 and ids == want.tolist()


def test_equal_distributions_accept_everything(lb):
    c = Case(12, [6, 6, 6], 20000, near=0.0, settings=[(0.8, 50, 0.9, 0.0)], draft_settings=[(0.8, 50, 0.9, 0.0)])
    c.drafts = c.z[[0, 1, 2, 3, 4, 5, 7, 8, 9, 10, 11, 12, 14, 15, 16, 17, 18, 19]].float().argmax(1).to(torch.int32)
    c.u[:] = np.float32(1 - 2.0 ** -24)
    got, _, accept = c.check(lb)
    assert got == [6, 6, 6] and accept == [1.0] * 18


def test_rows_without_finite_logits_and_odd_values(lb):
    c = Case(13, [2, 2, 2, 2, 1], 500)
    c.z = c.z.clone()
    c.y = c.y.clone()
    c.z[0] = -torch.inf                    # request 0: nothing to accept, and nothing to draw
    c.z[3 + 2] = torch.nan                 # request 1: its last row
    c.drafts[2:4] = c.z[3:5].float().argmax(1).to(torch.int32)
    c.u[2:4] = 0.0
    c.y[4] = -torch.inf                    # request 2: a drafter's row with nothing: q = 0, taken where p > 0
    c.z[6, int(c.drafts[4])] = -torch.inf  # ... and p = 0 there: rejected, the rest is p
    c.z[9, 3], c.z[9, 4] = torch.inf, torch.nan
    c.u[6], c.u[7], c.u[8] = np.nan, -1.0, 7.0
    c.v[3], c.v[4] = np.nan, 2.0
    got, ids, _ = c.check(lb)
    assert got[0] == 0 and ids[0] == -1 and got[1] == 2 and ids[5] == -1 and got[2] == 0 and ids[6] >= 0


@pytest.mark.parametrize("many", [3, 700])
@pytest.mark.parametrize("settings", [(1.0, 2, 1.0, 0.0), (0.7, 400, 1.0, 0.0), (1.0, 0, 0.6, 0.0), (0.0, 0, 1.0, 0.0)])
@pytest.mark.parametrize("bf16", [False, True])
def test_several_infinities_count_as_equal(lb, many, settings, bf16):
    """A cut through logits of +inf leaves the lower ones in, in the target's rows and the drafter's."""
    c = Case(23, [4, 4], 6000, settings=[settings, PLAIN], draft_settings=[PLAIN, settings], bf16=bf16)
    c.z, c.y = c.z.clone(), c.y.clone()
    at = torch.arange(many, device="cuda") * 8 + 5
    c.z[:5, at] = torch.inf
    c.y[4:, at] = torch.inf
    c.y[2, at] = torch.inf
    first, last = int(at[0]), int(at[-1])
    c.drafts = i32([first, first, first, last, last, first, last, first])
    c.u[:] = [0.0, 0.0, 1e-6, 0.5, 0.5, 0.5, 0.999, 1.0]
    c.check(lb)


def test_drafts_outside_the_vocabulary(lb):
    for certain in (True, False):
        c = Case(14, [2, 2, 2], 400, Vd=100, certain=certain)
        c.drafts = i32([-1, 5, 400, 2 ** 31 - 1, 3, -2 ** 31])
        c.u[:] = 0.0
        got, ids, accept = c.check(lb)
        assert got[0] == 0 and got[1] == 0 and accept[0] == accept[2] == accept[3] == accept[5] == 0.0


def test_columns_outside_the_drafter_are_none(lb):
    c = Case(15, [3, 3], 300, Vd=50)
    c.index[::7] = 50
    c.index[3::7] = -5
    c.index[5::7] = 2 ** 31 - 1
    c.check(lb)


def test_padded_arrays_and_requests_without_rows(lb):
    """Arrays longer than cu_drafts says, as captured graphs have them."""
    c = Case(16, [4, 0, 3, 5], 1000, settings=SETTINGS)
    want = [x[:] for x in c.run(lb)]
    keep = c.N, c.M
    c.z = torch.cat([c.z, torch.full((5, 1000), torch.nan, device="cuda")])
    c.y = torch.cat([c.y, torch.full((3, 1000), torch.nan, device="cuda")])
    c.drafts = torch.cat([c.drafts, i32([7, 7, 7])])
    c.u = np.concatenate([c.u, [0, 0, 0]]).astype(np.float32)
    got, ids, accept = c.run(lb)
    assert got == want[0] and ids[:keep[1]] == want[1] and accept[:keep[0]] == want[2]
    assert set(ids[keep[1]:]) == {-9} and set(accept[keep[0]:]) == {5.0}


def test_bad_offsets_are_recorded_and_left_out(lb):
    c = Case(17, [2, 3, 1], 600)
    want = [x[:] for x in c.run(lb)]
    for cu, bad in (([0, 2, 5, 7], [2]), ([0, -1, 5, 6], [0, 1]), ([-2, 2, 5, 6], [0]), ([0, 2, 1, 6], [1]), ([0, 9, 5, 6], [0, 1])):
        c.cu = np.array(cu)
        got, ids, _ = c.run(lb)
        assert lb.lowbit_device_error() == 1
        for b in range(3):
            c0, c1 = cu[b], cu[b + 1]
            if b in bad:
                assert got[b] == 0
            elif (c0, c1) == ([0, 2, 5][b], [2, 5, 6][b]):
                assert got[b] == want[0][b] and ids[c0 + b:c1 + b + 1] == want[1][c0 + b:c1 + b + 1]
    c = Case(17, [2, 3, 1], 600)
    c.z, c.M = c.z[:8], 8                      # a row short: the last request does not fit
    got, ids, _ = c.run(lb)
    assert lb.lowbit_device_error() == 1 and got == want[0][:2] + [0] and ids[:7] == want[1][:7]


def test_a_captured_step_serves_other_rows(lb):
    a, b = (Case(s, n, 5000, Vd=1000, settings=SETTINGS) for s, n in ((18, [3, 0, 4, 1]), (19, [1, 6, 0, 1])))
    args = a.args(lb)
    lb.lowbit_verify_drafts(**args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lb.lowbit_verify_drafts(**args)
    for c in (b, a):
        for name, x in c.args(lb).items():
            if name not in ("workspace", "n_accept", "ids", "accept"):
                args[name].copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        for r in range(4):
            c0, c1 = int(c.cu[r]), int(c.cu[r + 1])
            want = plain(c, r)
            assert (int(args["n_accept"][r]), args["ids"][c0 + r:c1 + r + 1].tolist()) == want[:2]


def test_same_result_again_on_another_stream_and_beside_another_call(lb):
    c = Case(20, [5, 3], 248320, Vd=32768, bf16=True, settings=[(0.8, 0, 0.97, 0.0), PLAIN])
    want = c.run(lb)
    assert c.run(lb) == want
    streams = [torch.cuda.Stream() for _ in range(2)]
    args = [c.args(lb) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, a in zip(streams, args):
            lb.lowbit_verify_drafts(**a, stream=s)
    torch.cuda.synchronize()
    for a in args:
        assert (a["n_accept"].tolist(), a["ids"].tolist(), a["accept"].tolist()) == want


def test_the_outcome_is_distributed_as_the_target(lb):
    """16,000 requests of one draft over the same rows: the first token's frequencies against p, five standard
    deviations of a binomial share, 5 sqrt(p (1 - p) / 16000)."""
    V, B = 7, 16000
    g = torch.Generator(device="cuda").manual_seed(21)
    z, y = (1.5 * torch.randn((1, V), device="cuda", generator=g) for _ in range(2))
    for settings, y_of in ((PLAIN, y), ((0.7, 4, 0.9, 0.0), y), (PLAIN, None)):
        q = torch.softmax(y, 1)[0] if y_of is not None else torch.nn.functional.one_hot(y.argmax(), V).float()
        drafts = torch.multinomial(q, B, replacement=True, generator=g).to(torch.int32)
        f = dict(device="cuda", generator=g)
        n_accept, ids = i32([0] * B), i32([0] * (2 * B))
        ws = torch.empty(lb.lowbit_verify_drafts_workspace_bytes(2 * B, B), dtype=torch.uint8, device="cuda")
        lb.lowbit_verify_drafts(z.expand(2 * B, V).contiguous(), i32(np.arange(B + 1)), drafts, torch.rand(B, **f), torch.rand(B, **f),
                                n_accept, ids, ws, draft_logits=None if y_of is None else y_of.expand(B, V).contiguous(),
                                temperature=f32([settings[0]] * B), top_k=i32([settings[1]] * B), top_p=f32([settings[2]] * B))
        p = od.shares(z[0].double().cpu().numpy(), settings)
        first = torch.bincount(ids[::2].long(), minlength=V).cpu().numpy() / B
        assert (np.abs(first - p) <= 5 * np.sqrt(p * (1 - p) / B) + 1e-6).all(), (first, p)
        second = ids[1::2]
        assert bool(((second >= 0) == (n_accept == 1)).all())


@pytest.mark.parametrize("name,change,kind", [
    ("logits", lambda t: t.half(), TypeError), ("logits", lambda t: t.cpu(), TypeError), ("logits", lambda t: t[0], TypeError),
    ("logits", lambda t: t.t().contiguous().t(), ValueError), ("cu_drafts", lambda t: t.long(), TypeError),
    ("cu_drafts", lambda t: t[:-1].contiguous(), ValueError), ("drafts", lambda t: t.long(), TypeError),
    ("drafts", lambda t: t[:-1].contiguous(), ValueError), ("u", lambda t: t[:-1].contiguous(), ValueError), ("u", lambda t: None, TypeError),
    ("v", lambda t: t.double(), TypeError), ("v", lambda t: t[:-1].contiguous(), ValueError), ("n_accept", lambda t: t.long(), TypeError),
    ("ids", lambda t: t[:-1], ValueError), ("workspace", lambda t: t.int(), TypeError), ("workspace", lambda t: t[:64], 4),
    ("draft_logits", lambda t: t[:-1], ValueError), ("draft_logits", lambda t: t.half(), TypeError), ("draft_logits", lambda t: None, ValueError),
    ("draft_index", lambda t: t[:-1], ValueError), ("draft_index", lambda t: t.long(), TypeError), ("temperature", lambda t: t[:1], ValueError),
    ("top_k", lambda t: t.float(), TypeError), ("draft_top_p", lambda t: 0.9, TypeError), ("draft_min_p", lambda t: t[:1], ValueError),
    ("accept", lambda t: t.half(), TypeError), ("accept", lambda t: t[:-1], ValueError), ("stream", lambda t: "x", Exception)])
def test_refusals(lb, name, change, kind):
    a = Case(22, [2, 1], 100, Vd=30).args(lb)
    a[name] = change(a.get(name))
    if isinstance(kind, int):
        with pytest.raises(lb.LowbitError) as e:
            lb.lowbit_verify_drafts(**a)
        assert e.value.status == kind
    else:
        with pytest.raises(kind):
            lb.lowbit_verify_drafts(**a)

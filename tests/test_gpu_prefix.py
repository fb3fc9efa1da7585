"""GPU parity of lowbit_prefix_attention with the fp64 oracle, which looks at every request's keys on their own.

Tolerance: that of test_gpu_paged.py.  A row's weights are rounded once each, in the part that they belong to,
and the parts are joined in fp32 (two products and a sum per element, and the factors' exponential: under
2^-20 of the spread, inside the 1e-4 of it that stands there for fp32)."""
import numpy as np
import pytest

from test_gpu_paged import Problem, i32
from test_gpu_paged import lb  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TIMEOUT = 5


class Shared(Problem):
    """Requests in groups; bounds [groups + 1], prefix [groups]; own: keys of a request that are neither new nor
    shared (None: an idle request whose table row is no page).  The table has room for `room` keys a request: under short
    ones the plain call's kernels do the work.  Slots that nobody uses hold NaN."""

    def __init__(self, seed, bounds, prefix, new, own, Hq, Hk, D, page, fp8=False, order="token", qscale=1.0, room=2304):
        g = np.random.default_rng(seed)
        B, T = len(new), int(sum(new))
        self.new, self.Hq, self.Hk, self.D, self.page, self.fp8, self.B, self.T = new, Hq, Hk, D, page, fp8, B, T
        self.bounds, self.prefix = bounds, prefix
        group = [max(i for i in range(len(prefix)) if bounds[i] <= b) for b in range(B)]
        self.kv = kv = [0 if own[b] is None else prefix[group[b]] + new[b] + own[b] for b in range(B)]
        whole = [p // page for p in prefix]
        need = [-(-x // page) for x in kv]
        pages = sum(whole) + sum(max(0, n - whole[c]) for n, c in zip(need, group)) + 2
        ids = g.permutation(pages)
        width = max(max(need) + 1, room // page)
        table = np.full((B, width), -7, dtype=np.int64)
        live = np.zeros((pages, page), dtype=bool)
        at, common = 0, []
        for n in whole:
            common.append(ids[at:at + n])
            live[common[-1]] = True
            at += n
        for b in range(B):
            if bounds[group[b]] == b:                     # the group's first request has the shared pages in any case
                table[b, :whole[group[b]]] = common[group[b]]
            if kv[b]:
                n = need[b] - whole[group[b]]
                table[b, :need[b]] = np.concatenate([common[group[b]], ids[at:at + n]])
                at += n
                j = np.arange(kv[b])
                live[table[b, j // page], j % page] = True
        self.table, self.cu = table, np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
        self.k_scale = self.v_scale = None
        vals = []
        for name in ("kc", "vc"):
            x = g.standard_normal((pages, page, Hk, D)).astype(np.float32)
            t = torch.from_numpy(x * (16 if fp8 else 1)).to(torch.float8_e4m3fn if fp8 else torch.bfloat16)
            vals.append(t.float().numpy().astype(np.float64))
            raw = t.view(torch.uint8 if fp8 else torch.int16).clone()
            raw[torch.from_numpy(~live)] = 0x7F if fp8 else 0x7FC0
            t = raw.view(t.dtype).cuda()
            setattr(self, name, t.transpose(1, 2).contiguous().transpose(1, 2) if order == "head" else t)
        if fp8:
            self.k_scale = torch.linspace(0.05, 0.08, Hk, device="cuda")
            self.v_scale = torch.linspace(0.09, 0.04, Hk, device="cuda")
            vals[0] = vals[0] * self.k_scale.cpu().numpy()[:, None].astype(np.float64)
            vals[1] = vals[1] * self.v_scale.cpu().numpy()[:, None].astype(np.float64)
        self.kv64 = vals
        q = torch.from_numpy((g.standard_normal((T, Hq, D)) * qscale).astype(np.float32)).to(torch.bfloat16)
        self.q64 = q.double().numpy()
        wide = torch.zeros((T, Hq * D + 72), dtype=torch.bfloat16)
        wide[:, 8:8 + Hq * D] = q.reshape(T, Hq * D)
        self.q = wide.cuda()[:, 8:8 + Hq * D].view(T, Hq, D)

    def args(self, lb):
        self.out = torch.full((self.T + 2, self.Hq, self.D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.ls = torch.full((self.T + 2, self.Hq), 7.0, device="cuda")
        ws = torch.full((lb.lowbit_prefix_attention_workspace_bytes(self.T, self.B, self.Hq, self.Hk, self.D),),
                        0xFF, dtype=torch.uint8, device="cuda")
        return dict(q=self.q, cache=lb.lowbit_paged_cache(self.kc, self.vc, self.k_scale, self.v_scale), cu_q=i32(self.cu),
                    kv_lens=i32(self.kv), block_table=i32(self.table), cu_groups=i32(self.bounds),
                    prefix_lens=i32(self.prefix), out=self.out[:self.T], workspace=ws, lse=self.ls[:self.T])

    def shared(self, lb, **kw):
        lb.lowbit_prefix_attention(**(self.args(lb) | kw))
        torch.cuda.synchronize()
        assert (self.out[self.T:] == 7.0).all() and (self.ls[self.T:] == 7.0).all()
        return self.out[:self.T], self.ls[:self.T]


SHAPES = [  # bounds, prefix, new, own, Hq, Hk, D, page
    # rows of the shared part: 8 or fewer, up to 16, 32, 64 (and tcgen05), and more than 1,024
    ([0, 2], [100], [1, 1], [3, 40], 8, 2, 64, 16),
    ([0, 1], [777], [1], [0], 32, 8, 128, 16),                       # a group of one, nothing of its own but its token
    ([0, 3], [500], [1, 1, 1], [0, 65, 7], 8, 2, 128, 64),
    ([0, 3], [321], [2, 0, 4], [9, 5, 77], 8, 2, 256, 8),
    ([0, 4], [1000], [4, 4, 4, 4], [0, 1, 2, 300], 8, 2, 128, 32),
    ([0, 9], [2049], [1] * 9, [0, 15, 16, 17, 100, 1, 2, 3, 700], 32, 8, 128, 64),
    ([0, 5], [300], [16, 16, 0, 16, 9], [1, 2, None, 200, 64], 16, 4, 64, 16),
    ([0, 2], [129], [200, 70], [40, 0], 16, 2, 128, 128),            # own rows on tcgen05 too
    ([0, 3], [400], [190, 333, 20], [40, 0, 5], 10, 2, 64, 32),
    ([0, 2], [640], [700, 650], [20, 333], 8, 4, 128, 64),           # more than 1,024 rows
    # several groups: unlike lengths, nothing shared, less than a page, empty, one whose requests are all idle
    ([0, 3, 5, 5, 8], [260, 0, 99, 31], [1, 2, 1, 3, 1, 1, 1, 1], [5, 9, 0, 70, 12, 0, 44, 3], 8, 2, 128, 32),
    ([0, 1, 4, 6, 7], [1030, 70, 200, 64], [5, 1, 0, 8, 0, 0, 16], [0, 40, 0, 3, None, None, 90], 8, 8, 64, 64),
    ([0, 2, 40], [512, 90], [1] * 40, [i % 50 for i in range(40)], 4, 1, 128, 16),   # more than 32 requests
    (list(range(0, 81, 2)), [17 * i for i in range(40)], [1, 2] * 40, [i % 9 for i in range(80)], 5, 1, 128, 16),
    ([0, 2], [40], [1, 3], [2, 9], 8, 1, 256, 1),                    # pages of one slot
]


@pytest.mark.parametrize("order", ["token", "head"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_parity(lb, i, fp8, causal, order):  # noqa: F811
    bounds, prefix, new, own, Hq, Hk, D, page = SHAPES[i]
    if fp8 and page * D < 128:
        pytest.skip("pages below 128 bytes are refused")
    pr = Shared(50 + i, bounds, prefix, new, own, Hq, Hk, D, page, fp8, order)
    pr.check(*pr.shared(lb, causal=causal), causal=causal)
    assert lb.lowbit_device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("i", range(len(SHAPES)))
@pytest.mark.parametrize("room", [0, 1024, 2048])
def test_short_tables(lb, i, fp8, room):  # noqa: F811
    bounds, prefix, new, own, Hq, Hk, D, page = SHAPES[i]
    if fp8 and page * D < 128:
        pytest.skip("pages below 128 bytes are refused")
    pr = Shared(50 + i, bounds, prefix, new, own, Hq, Hk, D, page, fp8, room=room)
    pr.check(*pr.shared(lb))
    assert lb.lowbit_device_error() == 0


@pytest.mark.parametrize("i", [0, 2, 5, 7, 9, 10])
def test_large_scores_and_far_ones(lb, i):  # noqa: F811
    """The parts' references far apart: either part may hold all of a row's weight."""
    bounds, prefix, new, own, Hq, Hk, D, page = SHAPES[i]
    for qscale in (6.0, 0.01):
        pr = Shared(90 + i, bounds, prefix, new, own, Hq, Hk, D, page, qscale=qscale)
        out, lse = pr.shared(lb)
        # |s| grows with qscale: fp32 scores are off by 2^-23 sqrt(D) |s|, up to 3e-4 for |s| of 250
        pr.check(out, lse) if qscale < 1 else self_consistent(lb, pr, out, lse)


def self_consistent(lb, pr, out, lse):  # noqa: F811
    """Against lowbit_paged_attention on the same inputs: two roundings of weights and two of the output apart
    (2^-8 each of values up to 5), scores alike to their last bits."""
    want, norm = Problem.run(pr, lb)
    assert ((out.float() - want.float()).abs() <= 4 * 2.0 ** -8 * 5).all()
    assert ((lse - norm).abs() <= 1e-3).all()


def test_one_part_holds_everything(lb):  # noqa: F811
    D, page = 64, 16
    for where in (0, 1):
        pr = Shared(3, [0, 3], [64], [1, 1, 1], [20, 3, 40], 4, 2, D, page)
        q = torch.ones_like(pr.q)
        kc, vc = torch.zeros_like(pr.kc), torch.zeros_like(pr.vc)
        first = [pr.table[0][0]] if where == 0 else [pr.table[b][4] for b in range(3)]
        for p_ in first:
            kc[p_, 2] = 30.0                       # a score of 30 * 64 / 8 = 240 above all others
            vc[p_, 2] = 3.0
        pr.q, pr.kc, pr.vc = q, kc, vc
        out, lse = pr.shared(lb)
        assert (out == 3.0).all() and torch.allclose(lse, torch.full_like(lse, 240.0))


def test_same_bits_again_and_on_another_stream(lb):  # noqa: F811
    pr = Shared(7, *SHAPES[10])
    a = [t.clone() for t in pr.shared(lb)]
    b = [t.clone() for t in pr.shared(lb)]
    side = torch.cuda.Stream()
    args = pr.args(lb)
    torch.cuda.synchronize()
    lb.lowbit_prefix_attention(**args, stream=side)
    side.synchronize()
    for x, y, z in zip(a, b, (pr.out[:pr.T], pr.ls[:pr.T])):
        assert torch.equal(x, y) and torch.equal(x, z)


# one launch for both parts; a launch each (tcgen05 and the warp-level MMA, of 128 rows and of 256); the plain kernels
@pytest.mark.parametrize("fp8,B,new", [(False, 5, 2), (True, 40, 1), (False, 520, 1), (True, 40, 16), (False, 5, 40)])
def test_a_captured_step_serves_other_lengths_and_groups(lb, fp8, B, new):  # noqa: F811
    pr = Shared(8, [0, 2, B], [200, 64], [new] * B, [(7 * b) % 71 for b in range(B)], 8, 2, 128, 16, fp8)
    args = pr.args(lb)
    lb.lowbit_prefix_attention(**args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lb.lowbit_prefix_attention(**args)
    for prefix, kv in (([200, 64], pr.kv), ([64, 16], [x - 3 for x in pr.kv]), ([7, 0], pr.kv)):
        pr.prefix, pr.kv = prefix, kv
        args["prefix_lens"].copy_(i32(prefix))
        args["kv_lens"].copy_(i32(kv))
        graph.replay()
        torch.cuda.synchronize()
        pr.check(pr.out[:pr.T], pr.ls[:pr.T])
    assert lb.lowbit_device_error() == 0


# a table with room for long requests takes taller items: in one launch with the own part, and in one of their own
TALL = [(False, 40, 16, 600), (True, 40, 16, 600), (True, 160, 1, 40), (False, 256, 1, 2100), (True, 80, 8, 600)]


def tall(seed, fp8, B, new, width, prefix):
    pr = Shared(seed, [0, B], [prefix], [new] * (B - 1) + [0], [(7 * b) % 71 for b in range(B)], 8, 2, 128, 16, fp8)
    pr.table = np.concatenate([pr.table, np.full((B, width), -7, dtype=np.int64)], 1)
    return pr


@pytest.mark.parametrize("fp8,B,new,width", TALL)
def test_tables_with_room_for_long_requests(lb, fp8, B, new, width):  # noqa: F811
    pr = tall(13, fp8, B, new, width, 1000)
    pr.check(*pr.shared(lb))
    args = pr.args(lb)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lb.lowbit_prefix_attention(**args)
    for prefix, kv in (([1000], pr.kv), ([90], [x - 3 for x in pr.kv])):
        pr.prefix, pr.kv = prefix, kv
        args["prefix_lens"].copy_(i32(prefix))
        args["kv_lens"].copy_(i32(kv))
        graph.replay()
        torch.cuda.synchronize()
        pr.check(pr.out[:pr.T], pr.ls[:pr.T])
    assert lb.lowbit_device_error() == 0


@pytest.mark.parametrize("fp8,B,new,width", TALL)
def test_stall_with_tall_items(lb, fp8, B, new, width):  # noqa: F811
    pr = tall(14, fp8, B, new, width, 300)
    want = [t.clone() for t in pr.shared(lb)]
    lb.lowbit_debug_inject_stall(True)
    try:
        out, lse = pr.shared(lb)
    finally:
        lb.lowbit_debug_inject_stall(False)
    assert lb.lowbit_device_error() == TIMEOUT
    assert bool((out == 7.0).all()) and bool((lse == 7.0).all()), "a timed-out call wrote outputs"
    assert all(torch.equal(x, y) for x, y in zip(pr.shared(lb), want)) and lb.lowbit_device_error() == 0


def test_calls_at_the_same_time(lb):  # noqa: F811
    """Two batches on two streams, a workspace each, over and over: the bits of either alone."""
    batches = [tall(15, False, 40, 16, 600, 700), tall(16, True, 160, 1, 40, 500)]
    want = [[t.clone() for t in pr.shared(lb)] for pr in batches]
    args, streams = [pr.args(lb) for pr in batches], [torch.cuda.Stream() for _ in batches]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for a, s in zip(args, streams):
            lb.lowbit_prefix_attention(**a, stream=s)
    torch.cuda.synchronize()
    for pr, w in zip(batches, want):
        assert torch.equal(pr.out[:pr.T], w[0]) and torch.equal(pr.ls[:pr.T], w[1])
    assert lb.lowbit_device_error() == 0


def test_rows_of_nobody_are_left_alone(lb):  # noqa: F811
    pr = Shared(9, [0, 2], [100], [2, 3], [4, 5], 4, 2, 64, 16)
    wide = torch.cat([pr.q, pr.q])            # rows past cu_q[B], as captured graphs have them
    out, lse = torch.full_like(wide, 7.0), torch.full((10, 4), 7.0, device="cuda")
    args = pr.args(lb)
    args |= dict(q=wide, out=out, lse=lse, workspace=torch.zeros(
        lb.lowbit_prefix_attention_workspace_bytes(10, 2, 4, 2, 64), dtype=torch.uint8, device="cuda"))
    lb.lowbit_prefix_attention(**args)
    pr.check(out[:5], lse[:5])                # twice the rows: another kernel, so not the bits of five rows
    assert (out[5:] == 7.0).all() and (lse[5:] == 7.0).all()


def test_bad_groups_are_recorded_and_left_out(lb):  # noqa: F811
    pr = Shared(10, [0, 2, 4], [96, 32], [1, 2, 1, 1], [5, 40, 8, 0], 4, 2, 64, 16)
    good = [t.clone() for t in pr.shared(lb)]
    keep = dict(bounds=pr.bounds, prefix=pr.prefix, kv=pr.kv)
    assert lb.lowbit_device_error() == 0
    whole = pr.table.shape[1] * 16
    for change, done in ((dict(bounds=[0, 2, 9]), [0, 1, 2]), (dict(bounds=[0, -1, 4]), []), (dict(bounds=[2, 2, 4]), [3, 4]),
                         (dict(bounds=[0, 2, 3]), [0, 1, 2, 3]), (dict(prefix=[96, -1]), [0, 1, 2]),
                         (dict(prefix=[whole + 16, 32]), [3, 4]),
                         (dict(prefix=[112, 32]), [1, 2, 3, 4]),        # request 0 has new tokens at position 101
                         (dict(kv=[40, keep["kv"][1]] + keep["kv"][2:]), [1, 2, 3, 4])):
        for name, x in (keep | change).items():
            setattr(pr, name, x)
        if "prefix" in change and change["prefix"][0] == 112:            # request 1's own pages behind 96 are not request 0's
            pr.table[0, 6] = pr.table[1, 6]
        out, lse = pr.shared(lb)
        assert lb.lowbit_device_error() == 1, change
        for t in range(5):  # cut elsewhere, the rows may differ by two roundings of the weights and of the output
            assert torch.equal(out[t], torch.full_like(out[t], 7.0)) if t not in done else \
                torch.allclose(out[t].float(), good[0][t].float(), rtol=2.0 ** -7, atol=2.0 ** -7 * 4), (change, t)
    for name, x in keep.items():
        setattr(pr, name, x)


def test_a_page_outside_the_cache_is_recorded(lb):  # noqa: F811
    for at, rows in (((0, 1), range(3)), ((1, 7), [1, 2])):
        pr = Shared(11, [0, 2], [96], [1, 2], [5, 40], 4, 2, 64, 16)
        good = pr.shared(lb)[0].clone()
        pr.table[at] = 10 ** 6
        out, _ = pr.shared(lb)
        assert lb.lowbit_device_error() == 1
        for t in range(3):
            assert t in rows or torch.equal(out[t], good[t])


# rows of the shared and of the own part: every kernel once in each
@pytest.mark.parametrize("new,B,D", [(1, 2, 128), (1, 6, 128), (2, 7, 64), (1, 40, 128), (16, 3, 128), (40, 30, 128), (600, 2, 64)])
def test_stall_times_out_writes_nothing_then_recovers(lb, new, B, D):  # noqa: F811
    pr = Shared(12, [0, B], [1000], [new] * B, [7 * b for b in range(B)], 4, 2, D, 32)
    want = [t.clone() for t in pr.shared(lb)]
    assert lb.lowbit_device_error() == 0 and bool(torch.isfinite(want[1]).all())
    lb.lowbit_debug_inject_stall(True)
    try:
        out, lse = pr.shared(lb)
    finally:
        lb.lowbit_debug_inject_stall(False)
    assert lb.lowbit_device_error() == TIMEOUT
    assert bool((out == 7.0).all()) and bool((lse == 7.0).all()), "a timed-out call wrote outputs"
    again = pr.shared(lb)
    assert lb.lowbit_device_error() == 0
    assert all(torch.equal(x, y) for x, y in zip(again, want))


@pytest.mark.parametrize("change,kind", [
    (dict(cu_groups=lambda t: t.long()), TypeError), (dict(cu_groups=lambda t: t[:-1].contiguous()), ValueError),
    (dict(prefix_lens=lambda t: t.float()), TypeError), (dict(prefix_lens=lambda t: None), TypeError),
    (dict(prefix_lens=lambda t: t.cpu()), TypeError), (dict(cu_groups=lambda t: None), TypeError),
    (dict(prefix_lens=lambda t: t[:0], cu_groups=lambda t: t[:1]), 1), (dict(q=lambda t: t.float()), TypeError),
    (dict(workspace=lambda t: t[:1 << 20]), 4), (dict(out=lambda t: t[:-1]), ValueError), (dict(lse=lambda t: t.half()), TypeError),
    (dict(scale=lambda t: float("nan")), 1), (dict(scale=lambda t: "x"), TypeError), (dict(causal=lambda t: []), None)])
def test_refusals(lb, change, kind):  # noqa: F811
    pr = Shared(13, [0, 1, 2], [32, 16], [1, 1], [3, 4], 4, 2, 64, 16)
    a = pr.args(lb) | dict(scale=0.1, causal=True)
    for name, f in change.items():
        a[name] = f(a[name])
    if kind is None:
        lb.lowbit_prefix_attention(**a)          # a truth value like any other
    elif isinstance(kind, int):
        with pytest.raises(lb.LowbitError) as e:
            lb.lowbit_prefix_attention(**a)
        assert e.value.status in (kind, 2)
    else:
        with pytest.raises(kind):
            lb.lowbit_prefix_attention(**a)
    torch.cuda.synchronize()
    assert lb.lowbit_device_error() == 0

"""GPU checks of lowbit_sample.

Sums are whole numbers, so the outcome is a function of the fp32 weights alone: with the weights
from torch's own exponential (elementwise fp32) the tokens, kept counts and log-probabilities of
`plain` below must be met exactly (log-probabilities to two roundings).  Against the oracle in 64
bits a token may differ only where u of the mass falls within 1e-5 of a boundary (2^-22 relative
per weight, and half a unit of 2^-40 for each of at most 2^19 tokens)."""
import numpy as np
import pytest

from oracle import sample as osample

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lb():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_weight_gemv_gb300 as lb
    return lb


def plain(z, temp, k, p, mp, u):
    """One row in whole numbers; tensors on the GPU, settings as Python numbers in fp32."""
    z = torch.where(torch.isnan(z), -torch.inf, z.float()).clamp(max=torch.finfo(torch.float32).max)
    V = z.numel()
    if z.max() == -torch.inf:
        return -1, 0, -np.inf
    f32 = lambda x: torch.tensor(x, dtype=torch.float32, device="cuda")  # noqa: E731
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
    total = int(keep.sum())
    aim = min(int(np.floor(np.float64(np.float32(u)) * np.float64(total))), total - 1)
    token = int((keep.cumsum(0) <= aim).sum())
    lp = torch.log((keep[token].double() / total).float())
    return token, int((keep > 0).sum()), float(lp)


def draw(lb, z, rows, id_map=None, stream=None):
    M = len(rows)
    cols = [[r[i] for r in rows] for i in range(5)]
    f = dict(dtype=torch.float32, device="cuda")
    ids = torch.full((M + 1,), -9, dtype=torch.int32, device="cuda")
    kept, lp = ids.clone(), torch.full((M + 1,), 5.0, **f)
    lb.lowbit_sample(z, torch.tensor(cols[4], **f), ids[:M], torch.tensor(cols[0], **f),
                     torch.tensor(cols[1], dtype=torch.int32, device="cuda"), torch.tensor(cols[2], **f),
                     torch.tensor(cols[3], **f), id_map, lp[:M], kept[:M], stream)
    torch.cuda.synchronize()
    assert ids[M] == -9 and kept[M] == -9 and lp[M] == 5.0
    return ids[:M].tolist(), kept[:M].tolist(), lp[:M].tolist()


def check(lb, z, rows):
    ids, kept, lp = draw(lb, z, rows)
    for m, r in enumerate(rows):
        want = plain(z[m], *r)
        assert (ids[m], kept[m]) == want[:2], (m, r, ids[m], kept[m], want)
        assert lp[m] == want[2] or abs(lp[m] - want[2]) <= 2.0 ** -22 * (1 + abs(want[2]))
    return ids


SETTINGS = [(1.0, 0, 1.0, 0.0), (0.7, 20, 0.95, 0.0), (1.3, 0, 0.9, 0.0), (0.5, 300, 1.0, 0.0),
            (1.0, 0, 1.0, 0.05), (0.9, 50, 0.8, 0.02), (0.0, 40, 0.5, 0.1), (2.0, 1, 1.0, 0.0),
            (1.0, 10 ** 9, 0.999, 0.0), (1.0, -3, 0.0, 0.0), (1e-3, 5, 0.99, 0.0), (50.0, 0, 0.5, 0.0),
            (1e9, 0, 1.0, 0.0), (float("nan"), 0, 1.0, 0.0), (1.0, 0, 1.0, 1.0), (1.0, 0, 1.0, 7.0),
            (1.0, 100000, 0.5, 0.0)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [1, 2, 31, 33, 1000, 4097, 16385, 32768, 70001, 248320])
def test_settings(lb, V, bf16):
    g = torch.Generator(device="cuda").manual_seed(V)
    rng = np.random.default_rng(V)
    rows = [s + (float(np.float32(rng.random())),) for s in SETTINGS]
    z = 3 * torch.randn((len(rows), V + 3), device="cuda", generator=g)   # rows apart
    z = z.to(torch.bfloat16) if bf16 else z
    check(lb, z[:, 1:V + 1], rows)


@pytest.mark.parametrize("M,V", [(1, 248320), (6, 100003), (40, 248320), (40, 248309), (40, 33000), (3, 5000), (17, 131073)])
@pytest.mark.parametrize("bf16", [False, True])
def test_prefix_lengths(lb, M, V, bf16):
    """Prefixes on both sides of what the first list, the candidates and a step can hold, over every
    split of a row, with ties, hot tokens and masked ones."""
    g = torch.Generator("cuda").manual_seed(M * 7 + V + bf16)
    z = 2.0 * torch.randn((M, V), device="cuda", generator=g)
    z[:, ::97] += 3.0
    z[0, :V // 2] = 4.0                                   # more equal logits than any list holds
    if M > 1:
        z[1, 200:] = -torch.inf                           # fewer tokens than the bound asks for
        z[2, ::3] = z[2, 5].item()
    z = z.to(torch.bfloat16) if bf16 else z
    wide = torch.full((M, -(-V // 8) * 8 + 8 * (M % 2)), 99.0, dtype=z.dtype, device="cuda")  # whole vectors, rows apart
    wide[:, :V] = z
    z = wide[:, :V]
    kinds = [(0.8, 0, 0.9, 0.0), (1.0, 0, 0.5, 0.0), (1.5, 0, 0.97, 0.0), (0.5, 0, 0.9999, 0.01), (1.0, 255, 1.0, 0.0),
             (1.0, 256, 0.9, 0.0), (1.2, 1024, 0.99, 0.0), (1.2, 1025, 0.99, 0.001), (0.7, 2048, 1.0, 0.0),
             (1.0, 2049, 0.8, 0.0), (1.0, V - 1, 1.0, 0.0), (1.0, 0, 0.02, 0.0), (1.0, 0, 1.0, 1e-3)]
    n = len(kinds) if M < 8 else 1
    for i in range(n):
        check(lb, z, [kinds[(i + m) % len(kinds)] + (((m * 37 + i * 11) % 101) / 101,) for m in range(M)])


@pytest.mark.parametrize("V", [7, 5000, 100003])
def test_edge_rows(lb, V):
    inf, nan = float("inf"), float("nan")
    g = torch.Generator(device="cuda").manual_seed(5)
    base = torch.randn(V, device="cuda", generator=g)
    kinds = [torch.full((V,), 1.5, device="cuda"), torch.full((V,), -inf, device="cuda"),
             torch.full((V,), nan, device="cuda"), base.clone(), base.clone(), base.clone(), base * 1e30,
             torch.zeros(V, device="cuda"), base.round(), base.clone()]
    kinds[3][V // 2] = inf
    kinds[4][::2] = -inf
    kinds[4][1] = nan
    kinds[5][: V - 1] = -inf
    kinds[7][1::2] = -0.0
    kinds[9][2] = kinds[9][5] = inf
    z = torch.stack(kinds)
    for s in SETTINGS:
        for u in (0.0, 0.37, 1.0 - 2.0 ** -24):
            check(lb, z, [s + (u,)] * len(kinds))


def test_u_out_of_range(lb):
    z = torch.zeros((4, 10), device="cuda")
    ids, _, _ = draw(lb, z, [(1.0, 0, 1.0, 0.0, u) for u in (-1.0, float("nan"), 1.0, 5.0)])
    assert ids == [0, 0, 9, 9]


def test_defaults_and_id_map(lb):
    V = 3000
    z = torch.randn((3, V), device="cuda")
    u = torch.rand(3, device="cuda")
    ids = torch.empty(3, dtype=torch.int32, device="cuda")
    lb.lowbit_sample(z, u, ids)
    torch.cuda.synchronize()
    for m in range(3):
        assert int(ids[m]) == plain(z[m], 1.0, 0, 1.0, 0.0, float(u[m]))[0]
    table = torch.arange(V, dtype=torch.int32, device="cuda") * 7 + 3
    mapped = torch.empty_like(ids)
    lb.lowbit_sample(z, u, mapped, id_map=table)
    assert torch.equal(mapped, ids * 7 + 3)


def test_against_the_oracle_in_64_bits(lb):
    V = 50000
    g = torch.Generator(device="cuda").manual_seed(3)
    rng = np.random.default_rng(3)
    rows = [s + (float(np.float32(rng.random())),) for s in SETTINGS[:9]] * 4
    z = 3 * torch.randn((len(rows), V), device="cuda", generator=g)
    ids, _, lp = draw(lb, z, rows)
    for m, r in enumerate(rows):
        w = osample.distribution(z[m].cpu().numpy(), *r[:4])
        cum = np.cumsum(w)
        lo, hi = (cum[ids[m]] - w[ids[m]]) / cum[-1], cum[ids[m]] / cum[-1]
        assert w[ids[m]] > 0 and lo - 1e-5 <= r[4] <= hi + 1e-5
        assert abs(lp[m] - np.log(w[ids[m]] / cum[-1])) <= 1e-5


def test_frequencies(lb):
    """Draws over a grid of u hit each token in proportion to its share."""
    w = np.array([1.0, 2.0, 0.0, 5.0, 2.0])
    n = 2000
    with np.errstate(divide="ignore"):
        z = torch.from_numpy(np.log(w).astype(np.float32)).cuda().expand(n, 5).contiguous()
    ids, _, _ = draw(lb, z, [(1.0, 0, 1.0, 0.0, (i + 0.5) / n) for i in range(n)])
    got = np.bincount(ids, minlength=5)
    assert np.abs(got / n - w / w.sum()).max() <= 2.0 / n


def test_same_every_time_on_another_stream(lb):
    g = torch.Generator(device="cuda").manual_seed(8)
    z = (3 * torch.randn((40, 100000), device="cuda", generator=g)).to(torch.bfloat16)
    rows = [SETTINGS[i % 6] + ((i + 0.5) / 40,) for i in range(40)]
    a = draw(lb, z, rows)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        assert draw(lb, z, rows, stream=s) == a

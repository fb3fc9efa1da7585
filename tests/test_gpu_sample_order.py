"""lowbit_sample with a small top-k on rows whose large tokens lie side by side, as in a vocabulary by frequency: every CTA's
list of them may be long, or not be made at all where another CTA's tokens are larger.  Compared in whole numbers, as
in test_gpu_sample.py."""
import numpy as np
import pytest

from test_gpu_sample import check, lb  # noqa: F401  (lb is a fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

KS = [1, 2, 5, 9, 16, 17, 20, 31, 32, 33]
# slices in shared memory (few rows, or short ones) and read again, by one CTA a row and up to 16
SHAPES = [(10, 5000), (10, 40000), (3, 131072), (5, 248320), (10, 524288), (10, 248320), (40, 131075), (70, 65536), (200, 65536)]


def rows_of(kind, M, V, g):
    z = 2.0 * torch.randn((M, V), device="cuda", generator=g)
    if kind == "descending":
        z = z.sort(1, descending=True).values
    elif kind == "ascending":
        z = z.sort(1).values
    elif kind == "block":                         # 300 large ones in the middle, none far apart from its neighbours
        z[:, V // 2:V // 2 + 300] = 12 + 0.01 * torch.randn((M, 300), device="cuda", generator=g)
    elif kind == "blocks":                        # as large ones at both ends, and one above them all
        for at in (0, V - 150):
            z[:, at:at + 150] = 12 + 0.2 * torch.randn((M, 150), device="cuda", generator=g)
        z[:, V // 3] = 14
    elif kind == "ties":                          # seven values: more equal tokens than any list holds
        z = (z / 2).clamp(-3, 3).round()
    elif kind == "few":                           # fewer tokens than k, in one slice; the other CTAs have none
        z[:, :] = -torch.inf
        z[:, V - 40:V - 30] = torch.randn((M, 10), device="cuda", generator=g)
    elif kind == "wide":                          # all but a few have no mass beside the largest, whose slice may have no other
        z[:, ::5] = torch.nan
        z[:, 7] = 60.0
        z[:, V - 1] = torch.inf if M % 2 else 59.0
    return z


@pytest.mark.parametrize("kind", ["descending", "ascending", "block", "blocks", "ties", "few", "wide"])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M,V", SHAPES)
def test_small_top_k(lb, M, V, bf16, kind):  # noqa: F811
    g = torch.Generator("cuda").manual_seed(M + V)
    rng = np.random.default_rng(M + V)
    z = rows_of(kind, M, V, g)
    z = z.to(torch.bfloat16) if bf16 else z
    rows = [(float(rng.choice([0.7, 1.0, 4.0, 30.0])), KS[m % len(KS)], float(rng.choice([0.9, 1.0])), 0.0,
             float(np.float32(rng.random()))) for m in range(M)]
    check(lb, z, rows)

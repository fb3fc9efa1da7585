"""GPU parity of lowbit_paged_attention on batches of unlike requests and on heads of 256 at a prompt's
size, against the oracle with the tolerances of test_gpu_paged."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_paged import Problem, lb  # noqa: E402,F401  (lb is a fixture)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", [
    # a prompt's chunk among decoding requests: short items and many tiles of one request
    ([1] * 30 + [500] + [1] * 29, [7 * i + 1 for i in range(30)] + [900] + [400 - 9 * i for i in range(29)], 8, 2, 128, 32),
    ([500] + [1] * 200, [600] + [3 * i + 1 for i in range(200)], 4, 1, 64, 16),
    # one block among idle slots, whose lengths still stand in the arrays
    ([0] * 7 + [16] + [0] * 8, [50] * 7 + [3000] + [0] * 8, 16, 4, 128, 64),
    ([0, 0, 40], [9, 0, 700], 4, 2, 256, 32),
    # heads of 256: a prompt's chunk, alone and beside a decoding request
    ([1200], [2500], 4, 1, 256, 64),
    ([300, 1], [301, 4000], 4, 2, 256, 128)])
def test_unlike_requests(lb, shape, fp8):  # noqa: F811
    pr = Problem(21, *shape, fp8=fp8)
    pr.check(*pr.run(lb))
    assert lb.lowbit_device_error() == 0


def test_windows_on_long_heads_of_256(lb):  # noqa: F811
    for causal, window in ((True, 700), (False, 90)):
        pr = Problem(22, [400, 3], [1500, 900], 4, 2, 256, 32)
        pr.check(*pr.run(lb, causal, window), causal, window)

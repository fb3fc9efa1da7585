"""GPU parity of long appends, eight tokens a block (bit-exact, as the short ones of test_gpu_paged): row
counts that end inside a block, blocks that several requests share, idle requests between."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_paged import append_case, lb  # noqa: E402,F401  (lb is a fixture)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("new,kv,Hq,Hk,D,page,rot,order", [
    ([1001], [1001], 1, 1, 64, 16, 64, "token"),
    ([1, 2, 3, 0, 5] * 150, [7, 2, 40, 9, 5] * 150, 4, 2, 64, 8, 32, "head"),
    ([4001, 0, 3], [4100, 8, 900], 5, 1, 128, 64, 128, "head"),
    ([2047, 2], [2050, 3], 2, 2, 128, 1, 64, "token"),
    ([4003], [4010], 4, 2, 256, 32, 64, "token")])
def test_append(lb, new, kv, Hq, Hk, D, page, rot, order, inter, fp8):  # noqa: F811
    append_case(lb, 31, new, kv, Hq, Hk, D, page, rot, inter, fp8, order)


def test_rows_of_nobody_in_a_long_call(lb):  # noqa: F811
    """T padded past the last request, inside and past a block of eight."""
    T, D = 1208, 64
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    x = torch.ones((T, 1, D), dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros((80, 16, 1, D), dtype=torch.bfloat16, device="cuda")
    q_out = torch.full((T, 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lb.lowbit_kv_append(x, x, x, None, i32([3, 1101, 1101, 1190]), i32([1098, 5, 89]),
                        i32([list(range(70)), [0] * 70, list(range(70, 80)) + [0] * 60]),
                        lb.lowbit_paged_cache(kc, kc.clone()), q_out)
    assert lb.lowbit_device_error() == 0
    done = torch.zeros(T, dtype=torch.bool, device="cuda")
    done[3:1190] = True
    assert bool((q_out[done] == 1).all()) and bool((q_out[~done] == 7).all())
    flat = kc.view(-1, D)
    assert bool((flat[:1098] == 1).all()) and not bool(flat[1098:1120].any())
    assert bool((flat[1120:1209] == 1).all()) and not bool(flat[1209:].any())

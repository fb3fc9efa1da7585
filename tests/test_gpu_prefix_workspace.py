"""lowbit_prefix_attention at the most rows a request for which it needs places for every row, and past that."""
import pytest

from test_gpu_paged import lb  # noqa: F401  (a fixture)
from test_gpu_prefix import Shared

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,new", [(128, 24), (128, 25), (64, 24), (256, 12), (256, 13), (128, 150)])
def test_nothing_behind_the_workspace_is_written(lb, D, new, fp8):  # noqa: F811
    pr = Shared(31, [0, 3], [200], [new] * 3, [40, 0, 77], 8, 2, D, 16, fp8)
    size = lb.lowbit_prefix_attention_workspace_bytes(pr.T, pr.B, pr.Hq, pr.Hk, pr.D)
    ws = torch.full((size + (1 << 24),), 0x5A, dtype=torch.uint8, device="cuda")
    pr.check(*pr.shared(lb, workspace=ws[:size]))
    assert bool((ws[size:] == 0x5A).all())
    assert lb.lowbit_device_error() == 0
    with pytest.raises(lb.LowbitError) as e:
        pr.shared(lb, workspace=ws[:size - 1])
    assert e.value.status == 4

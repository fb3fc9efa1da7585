"""lowbit_prefix_attention on both sides of the rules that choose its kernels: by rows a request (which bounds its workspace),
and by requests under short block tables."""
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


# Short tables, on either side of the rule that chooses the kernels: requests times heads over e4m3, heads of 256 in bf16,
# several groups of 16.
@pytest.mark.parametrize("B,groups,Hq,Hk,D,fp8,room", [
    (512, 1, 16, 8, 64, True, 512), (511, 3, 16, 8, 64, True, 512), (128, 1, 32, 8, 256, False, 1024), (127, 1, 32, 8, 256, False, 1024),
    (64, 4, 32, 8, 128, False, 2048), (64, 4, 8, 2, 128, False, 2048), (16, 1, 8, 2, 128, False, 2048), (17, 1, 8, 2, 128, False, 2048)])
def test_many_requests_under_short_tables(lb, B, groups, Hq, Hk, D, fp8, room):  # noqa: F811
    prefix = [64 + 32 * g for g in range(groups)]
    pr = Shared(41, [B * g // groups for g in range(groups + 1)], prefix, [int(b % 7 != 3) for b in range(B)],
                [(5 * b) % 37 for b in range(B)], Hq, Hk, D, 16, fp8, room=room)
    pr.check(*pr.shared(lb))
    assert lb.lowbit_device_error() == 0

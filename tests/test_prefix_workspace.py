"""Size of lowbit_prefix_attention's workspace: what the rows that the join can see need, and no more."""
import pytest

from test_paged_oracle import native  # noqa: F401  (a fixture)


@pytest.mark.parametrize("D,limit", [(64, 96), (128, 96), (256, 48)])
@pytest.mark.parametrize("B,Hq,Hk", [(1, 8, 8), (6, 32, 8), (64, 32, 4), (1000, 5, 1)])
def test_bytes(native, D, limit, B, Hq, Hk):  # noqa: F811
    f, plain = native.lowbit_prefix_attention_workspace_bytes, native.lowbit_paged_attention_workspace_bytes
    before = 0
    for T in (0, 1, B, limit * B * Hk // Hq, limit * B * Hk // Hq + 1, 20000, 1 << 20, 1 << 24):
        rows = min(T * Hq, limit * B * Hk)
        assert f(T, B, Hq, Hk, D) == 2 * plain(T, B, Hq, Hk, D) + rows * (8 * D + 48)
        if T > B:
            assert f(T, B, Hq, Hk, D) >= before    # one for the largest call serves the smaller ones
            before = f(T, B, Hq, Hk, D)
        assert f(T, B + 1, Hq, Hk, D) >= f(T, B, Hq, Hk, D)

"""Arrays of no elements lie over nothing: lowbit_verify_drafts without drafts, host side."""
import pytest

from test_drafts_oracle import APART, INVALID, Y, Z, call, rows
from test_paged_oracle import native  # noqa: F401  (a fixture)


@pytest.mark.parametrize("empty", ["drafts", "u", "accept", "logits"])
@pytest.mark.parametrize("over", ["count", "ids", "ws"])
def test_empty_arrays_over_outputs(native, empty, over):  # noqa: F811
    import torch
    if torch.cuda.is_available():
        pytest.skip("calls that are not refused would run on these addresses")
    at = APART[over] + (16 if over == "ws" else 4)      # inside it
    place = APART | ({empty: at} if empty != "logits" else {})
    draft = rows(logits=at if empty == "logits" else Y, rows=0)
    assert call(native, rows(logits=Z), draft, **(place | dict(N=0))) != INVALID
    if empty != "logits":                                # one element is refused
        assert call(native, rows(logits=Z), rows(logits=Y, rows=1), **(place | dict(N=1))) == INVALID

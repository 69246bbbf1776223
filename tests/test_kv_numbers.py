"""Numbers that the paged cache's Python calls refuse (before they look at the tensors)."""
import pytest
import torch

from barrier_free_message_gb300 import _build, sfar


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()


@pytest.mark.parametrize("max_q,window,what", [(-1, 0, "max_q"), (1, -1, "window"), (-(1 << 62), 5, "max_q"), (4, -(1 << 40), "window")])
def test_negative_numbers(max_q, window, what):
    i, bf = torch.zeros(4, dtype=torch.int32), torch.zeros(2, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match=f"{what}: must not be negative"):
        sfar._tensors().attention(None, 2, 2, 64, bf, bf, i.view(2, 2), i, i, max_q, 1.0, window, 0)


def test_numbers_beyond_64_bits():
    i, bf = torch.zeros(4, dtype=torch.int32), torch.zeros(2, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(OverflowError):
        sfar._tensors().attention(None, 2, 2, 64, bf, bf, i.view(2, 2), i, i, 1, 1.0, 1 << 64, 0)


def test_no_handle():
    assert sfar.lib().sfar_test_kv_record_failure(None) == sfar.SFAR_ERR_INVALID

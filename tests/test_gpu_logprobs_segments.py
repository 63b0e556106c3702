"""GPU parity of log probabilities on rows that fill their segments exactly,
nearly, and by a few values more, aligned and not."""
import pytest
import torch

from gpu_util import dev
from test_gpu_logprobs import F, _check, _logits  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,v", [(3, 8192), (1, 16384), (40, 16384), (3, 32768), (1, 65536), (3, 65536), (3, 131072)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_of_whole_segments(F, t, v, dtype):  # noqa: F811
    x = _logits(t, v + 8, dtype)
    for d in (-7, -1, 0, 1):
        _check(F, x[:, :v + d].contiguous(), 5)
        _check(F, x[:, 3:3 + v + d], 20)                    # rows 3 and more places past an aligned one
    _check(F, x[:, :v].contiguous(), 0)


@pytest.mark.parametrize("v", [16384, 65536])
@pytest.mark.parametrize("pad", [1, 2, 3, 4, 5, 6, 7])
def test_a_rows_last_values(F, v, pad):  # noqa: F811
    """The best, the target and the only live values are the row's last few,
    which lie past the last whole step of an unaligned row."""
    x = torch.full((2, v + pad), -30.0, dtype=torch.bfloat16, device=dev())
    x[0, -7:] = torch.arange(7, device=dev()).to(torch.bfloat16)
    x[1] = float("-inf")
    x[1, -3:] = torch.tensor([1.0, 3.0, 2.0], dtype=torch.bfloat16)
    r = _check(F, x[:, pad:], 7, targets=torch.tensor([v - 1, v - 2], dtype=torch.int32).numpy())
    assert r.top_ids[0].tolist() == list(range(v - 1, v - 8, -1))
    assert r.top_ids[1, :3].tolist() == [v - 2, v - 1, v - 3]

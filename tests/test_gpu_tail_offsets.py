"""Offsets of the tails' copies that decrease: reported, whichever sequences the tokens then fall to, with
the offsets in shared memory and (1,024 and more) where they stand; nothing outside is touched."""
import pytest
import torch

import linear_attention_recurrence_simple_gb300 as gla
from tests.prefix_helpers import DK, DV
from tests.test_gpu_prefix import i32

pytestmark = pytest.mark.gpu
SHAPE = -2


@pytest.mark.parametrize("n_seq, at", [(3, 2), (700, 699), (1500, 1), (1500, 1400)])
@pytest.mark.parametrize("fmt", [torch.bfloat16, torch.float8_e4m3fn])
def test_decreasing_offsets_are_reported(fmt, n_seq, at):
    H, T = 2, 3 * n_seq
    cu = [3 * i for i in range(n_seq + 1)]
    t = gla.gla_tail_alloc(n_seq, H, 16, fmt)
    k, v = (torch.randn(T, H, d, device="cuda").to(torch.bfloat16) for d in (DK, DV))
    pos = i32([0] * n_seq)
    gla.gla_tail_append(k, v, t, pos, i32(cu))
    gla.gla_tail_read(t, pos, i32(cu), T, dtype=torch.bfloat16)
    assert gla.gla_get_device_error() == 0
    cu[at] = cu[at - 1] - (1 if at > 1 else -7)  # the one before, or the one behind, now lies above it
    gla.gla_tail_append(k, v, t, pos, i32(cu))
    assert gla.gla_get_device_error() == SHAPE
    ko, vo = (torch.full((T + 9, H, d), 7.0, device="cuda", dtype=torch.bfloat16) for d in (DK, DV))
    gla.gla_tail_read(t, pos, i32(cu), T + 9, k=ko, v=vo)
    assert gla.gla_get_device_error() == SHAPE
    assert bool((ko[T:] == 7.0).all()) and bool((vo[T:] == 7.0).all())

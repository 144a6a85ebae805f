"""moe_token_logprobs on finite logits of large magnitude: masks such as -1e9
or -1e20 and rows far from zero, where neighbouring fp32 values are tens of
powers of two apart in probability and more.

Definition and tolerance are those of test_token_logprobs_gpu; rows of more
than four an SM go by test_token_logprobs_many_rows_gpu."""
import pytest
import torch

from test_token_logprobs_gpu import BF, DEV, F32, check, some_targets
from test_token_logprobs_many_rows_gpu import check as check_many

pytestmark = pytest.mark.gpu

STEP = 4096        # fp32 logits that a block of 256 threads visits at once


@pytest.mark.parametrize("m,scale", [(m, s) for m in (-2.0e9, -1.5e9, -1.0e9, -8.0e8, -5.5e8, -2.0e8, 1.0e9, 5.5e8)
                                     for s in (0.7, 0.9, 1.0, 1.25) if abs(m) * s * 1.4427 < 2.0 ** 31])
def test_next_value_above_a_large_reference(m, scale):
    """Every thread meets m first, then the next fp32 value above it.  u m below
    2^31, where the rounding of u m itself is at most 64 powers of two."""
    l = torch.full((2, 3 * STEP + 5), m, device=DEV)
    up = torch.nextafter(l[0, :1], torch.full((1,), float("inf"), device=DEV))
    l[:, STEP:] = up
    l[1, 2 * STEP:] = m
    check(l, some_targets(2, l.shape[1], 3), top_n=5, scale=scale)
    check_many(l, some_targets(2, l.shape[1], 1), scale=scale)

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


LARGE = [-1e9, -2e9, -1e10, -1e12, -1e18, -1e20, -3e38]


def masked(V, dtype, mask, seed=0):
    """Rows with half, a hundredth, one and none of their logits left, and one
    with them at the end of the row only."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    l = (torch.randn(5, V, generator=g, device=DEV) * 3).to(dtype)
    keep = torch.rand(5, V, generator=g, device=DEV)
    l[0, keep[0] > 0.5] = mask
    l[1, keep[1] > 0.01] = mask
    l[2, :] = mask
    l[2, V // 3] = 1.5
    l[3, :] = mask
    l[4, :V - 9] = mask
    return l


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("mask,scale", [(m, s) for m in LARGE for s in (0.7, 0.9, 1.0, 1.25) if abs(m) * s < 3.4e38])
def test_masks(mask, scale, dtype):
    for V in (300, 12003, 70001):       # 70001: rows in parts
        check(masked(V, dtype, mask), some_targets(5, V, 3), top_n=6, scale=scale)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("mask", LARGE)
def test_masks_in_many_rows(mask, dtype):
    for V in (5003, 14003, 60003):      # blocks of 128 threads, with copies through shared memory, of 256
        check_many(masked(V, dtype, mask), some_targets(5, V, 2), top_n=6, scale=0.9)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [0.9, 1.0])
@pytest.mark.parametrize("offset", [1e7, 2e8, -3e8, 6e8, 1e9, 2e9, 1e10, -1e12, 1e18, 1e20, 1e38])
def test_rows_far_from_zero(offset, scale, dtype):
    """Rows around a large value: a few neighbouring values, each many times."""
    for V in (300, 12003, 70001):
        g = torch.Generator(device=DEV).manual_seed(V)
        ulps = torch.randint(-2, 3, (3, V), generator=g, device=DEV)
        l = torch.full((3, V), offset, device=DEV).to(dtype)
        one = l[0, 0].abs().float() * (2.0 ** -7 if dtype == BF else 2.0 ** -23)
        l = (l.float() + ulps * one).to(dtype)
        l[1, 0] = 3.0
        check(l, some_targets(3, V, 2), top_n=4, scale=scale)


@pytest.mark.parametrize("scale", [2.0 ** -64, 1e-6, 1e6, 1e9, 1e15, 2.0 ** 64])
def test_extreme_scales(scale):
    """Temperatures that leave nothing but the largest logits, and nearly none."""
    for dtype in (BF, torch.float16, F32):
        g = torch.Generator(device=DEV).manual_seed(3)
        l = (torch.randn(3, 9001, generator=g, device=DEV) * 3).to(dtype)
        l[1] = (l[1] * 4).round() / 4   # ties at the top
        check(l, some_targets(3, 9001, 2), top_n=4, scale=scale)

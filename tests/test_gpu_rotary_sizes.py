"""Rotary positions and their gradient at sizes whose blocks walk heads several
at a time, more than one round of them, and (gradient with a norm) several items
each, q's and k's blocks in proportion to their work."""

import pytest

from tests.test_gpu_rotary import test_rotary as forward_case, test_rotary_gradient as gradient_case

pytestmark = pytest.mark.gpu

# B, Hq, Hk, grid, d, dims, dtype, pairing, spectrum, norm of (q, k), positions given
CASES = [
    (1, 24, 8, (4, 48, 49), 128, (44, 42, 42), "bf16", "interleaved", "axis", (True, True), False),
    (2, 13, 6, (1, 97, 83), 128, (32, 32, 32), "fp16", "halves", "shared", (True, False), True),
    (2, 13, 6, (1, 97, 83), 128, (32, 32, 32), "bf16", "halves", "shared", (False, True), True),
    (1, 9, 0, (1, 121, 127), 128, (22, 20, 20), "fp32", "halves", "axis", (True, False), False),
    (3, 5, 1, (7, 31, 53), 64, (6, 2, 10), "bf16", "halves", "axis", (True, True), False),
    (2, 11, 3, (5, 61, 67), 64, (16, 24, 24), "fp32", "interleaved", "axis", (True, True), True),
    (1, 6, 6, (9, 41, 43), 64, (16, 24, 24), "fp16", "interleaved", "shared", (False, False), False),
]
ids = lambda c: "-".join(str(x) for x in c).replace(" ", "")  # noqa: E731


def split(c):
    """Heads of q a block walks, and items of q and of k: what rotary.cu's plan makes of a case."""
    B, Hq, Hk, grid, d = c[:5]
    tiles = -(-grid[0] * grid[1] * grid[2] // (256 // (d // 8)))
    share = max(1, tiles * B * (Hq + Hk) // (148 * 3))
    items, per = [], []
    for H in (Hq, Hk):
        n = min(H, -(-share // 4) * 4)
        parts = -(-H // n) if n else 0
        per.append(-(-H // parts) if parts else 0)
        items.append(tiles * B * parts)
    return per, items


@pytest.mark.parametrize("c", CASES, ids=ids)
def test_rotary_large(c):
    per, items = split(c)
    assert per[0] > 4                               # more than one group of heads in flight
    forward_case(c)


@pytest.mark.parametrize("c", CASES, ids=ids)
def test_rotary_gradient_large(c):
    per, items = split(c)
    assert not any(c[9]) or sum(items) > 888        # more items than blocks
    gradient_case(c)

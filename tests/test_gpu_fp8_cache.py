"""Writing the 8-bit KV cache where slots are skipped."""
from __future__ import annotations

import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests import test_gpu_fp8 as base  # noqa: E402


# ------------------------------------------------------------------ skipped slots


def _holes(rng, P, page, block, T, share):
    """Runs of tokens, some of them masked, alone and in stretches of up to 700, before, inside and after the runs."""
    slots = []
    for b in rng.sample(range(P * page // block), P * page // block):
        a = rng.randrange(block)
        for r in range(a, rng.randint(a + 1, block)):
            slots.append(b * block + r)
            if rng.random() < share:
                slots += [rng.choice((-1, P * page, -(1 << 40)))] * rng.choice((1, 1, 1, 2, 31, 32, 33, 300, 700))
    return torch.tensor(slots[:T])


@pytest.mark.parametrize("Hk,D,page,block", [(2, 64, 16, 16), (8, 64, 64, 64), (3, 128, 256, 256), (1, 128, 64, 32)])
@pytest.mark.parametrize("share", [0.02, 0.3])
@pytest.mark.parametrize("T", [9, 300, 6000])
def test_append_around_skipped_slots(T, share, Hk, D, page, block):
    # tokens of a block with skipped ones between them: the tokens of the block that came in earlier
    # calls keep their values, but for a scale that grows
    rng = random.Random(T + block)
    P = max(3, T // page)
    slots = _holes(rng, P, page, block, T, share)
    slots = torch.cat((torch.full((rng.choice((0, 1, 40)),), -1), slots))
    x = [base._rand((slots.numel(), Hk, D), s) * 2 ** (6 * s) for s in (1, 2)]
    base._check_append(*x, slots, P, page, block)


def test_append_of_one_block_with_every_other_slot_skipped():
    P, page, block, Hk, D = 2, 256, 256, 4, 64
    slots = torch.arange(1, 513) // 2
    slots[::2] = -1
    x = [base._rand((512, Hk, D), s) for s in (1, 2)]
    base._check_append(*x, slots, P, page, block)
    base._check_append(x[0].repeat(20, 1, 1), x[1].repeat(20, 1, 1),
                       torch.cat((slots[:300], torch.full((20 * 512 - 512,), -1), slots[300:])), P, page, block)

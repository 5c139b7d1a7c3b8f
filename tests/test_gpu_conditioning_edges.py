"""Conditioning entry points where they can go wrong in ways that plain sizes and values do not show.

Tolerances and helpers are those of the parity tests of the same operators.
"""
import pytest
import torch

import sequence_parallelism_st_b200 as st
from test_gpu_conditioning import BF, check_attn, rand, run_cross, sets_of

pytestmark = pytest.mark.gpu

# rows and row tiles of a work item, keys per step and steps whose K and V stay in shared memory
TILES = {32: (3, 96), 64: (3, 96), 72: (3, 80), 80: (3, 80), 96: (3, 64), 128: (2, 128)}


def first_blocks(cols, q_blocks, ctas):
    """(head, row block) of each block's first item where the items are cut evenly: heads and units outside,
    row blocks inside, as the launch does when there are more heads and units than blocks."""
    assert cols > ctas
    n = cols * q_blocks
    share = -(-n // ctas)
    assert share >= q_blocks                           # one band
    return [divmod(n * c // ctas, q_blocks) for c in range(ctas)]


@pytest.mark.parametrize("last", [100, 200])
@pytest.mark.parametrize("D", sorted(TILES))
def test_kept_keys_of_heads_that_share_them(D, last):
    """A block starts on the last rows of a head, where some of its row tiles have none, and goes on with a head
    of the same K and V, where they all have: every tile waits for the stages, which held NaN before."""
    nt, bn = TILES[D]
    last = min(last, (nt - 1) * 128)
    H, Hkv, ctas, full = 4, 1, 3, 2
    S, L = full * nt * 128 + last, 2 * bn - 7
    heads = first_blocks(H, full + 1, ctas)
    assert any(qb == full and h + 1 < H for h, qb in heads), heads
    assert -(-last // 128) < nt
    q, k, v = rand(200, 1, 1, S, H, D), rand(201, 1, L, Hkv, D), rand(202, 1, L, Hkv, D)
    poison = torch.full((148, L, 1, D), float("nan"), dtype=BF, device="cuda")
    qp = rand(203, 148, 1, nt * 128, 1, D)
    for _ in range(5):
        run_cross(qp, poison, poison)                  # every SM's stages hold NaN
        st.st_set_sm_budget(ctas)
        try:
            o, lse, _ = run_cross(q, k, v)
        finally:
            st.st_set_sm_budget(0)
        check_attn(q, [sets_of(k, v)], o, lse, what=f"D{D}")

"""Limits of the drafter-training losses' sizes, at and past them (CPU: nothing is launched)."""

import pytest

from test_loss_abi import BF16, F32, INVALID, UNSUPPORTED, L, kd  # noqa: F401

MOST = 1 << 30  # rows of given logits


@pytest.mark.parametrize("bwd", [True, False])
@pytest.mark.parametrize("N", [MOST + 1, 2 ** 31 - 256, 2 ** 31 - 1])
def test_rows_past_the_counters(L, N, bwd):  # noqa: F811
    """A row loop in steps of 256 would pass 2^31 - 1 and start again."""
    assert kd(L, bwd=bwd, N=N, V=1, k=1, wsb=2 ** 63) == UNSUPPORTED
    assert kd(L, bwd=bwd, N=MOST, V=1, k=1, wsb=1 << 20) == INVALID  # only the workspace is too small
    assert L.spec_topk_distill_workspace_bytes(N, 1, 1) == 0 < L.spec_topk_distill_workspace_bytes(MOST, 1, 1)

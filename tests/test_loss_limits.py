"""Limits of the drafter-training losses' sizes, at and past them (CPU: nothing is launched)."""

import pytest

from test_loss_abi import BF16, F16, F32, INVALID, UNSUPPORTED, L, head, kd  # noqa: F401

MOST = 1 << 30  # rows of given logits


@pytest.mark.parametrize("bwd", [True, False])
@pytest.mark.parametrize("N", [MOST + 1, 2 ** 31 - 256, 2 ** 31 - 1])
def test_rows_past_the_counters(L, N, bwd):  # noqa: F811
    """A row loop in steps of 256 would pass 2^31 - 1 and start again."""
    assert kd(L, bwd=bwd, N=N, V=1, k=1, wsb=2 ** 63) == UNSUPPORTED
    assert kd(L, bwd=bwd, N=MOST, V=1, k=1, wsb=1 << 20) == INVALID  # only the workspace is too small
    assert L.spec_topk_distill_workspace_bytes(N, 1, 1) == 0 < L.spec_topk_distill_workspace_bytes(MOST, 1, 1)


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("N,V,H", [(300, 6100, 712), (1792, 151936, 2048), (4096, 129280, 4096), (65536, 151936, 4096)])
def test_the_workspace_can_be_bounded(L, N, V, H, dt):  # noqa: F811
    """The least workspace holds a piece of 2048 tokens of every row, not the vocabulary's."""
    for k, grads in ((1, (1, 1)), (64, (1, 0)), (64, (0, 1))):
        most, least = (f(dt, N, V, H, k, *grads) for f in (L.spec_linear_loss_workspace_bytes,
                                                          L.spec_linear_loss_workspace_least))
        fixed = L.spec_linear_loss_workspace_bytes(dt, N, V, H, k, 0, 0)
        partials = 2 * (N + 255) // 256 * 256 * H * 4 * grads[0]  # two splits of a piece at most
        copy = max(N, 65536 // H + 1) * (H + 63) * 2 + 4 * N
        assert fixed < least and (least < most if N < 8192 else least <= most)
        assert N * 4096 - 256 <= least - fixed <= N * 4096 + partials + copy + 8192
        if N * V * (2 if dt == BF16 else 6) < 4e9:
            assert most - fixed >= N * V * (2 if dt == BF16 else 6)
        what = "lce" if k == 1 else "lkd"
        o = {name: None for name, wanted in zip(("gx", "gw"), grads) if not wanted}
        assert head(L, what, dt=dt, gdt=dt, N=N, V=V, H=H, k=k, wsb=least // 2, **o) == INVALID
    for f in (L.spec_linear_loss_workspace_bytes, L.spec_linear_loss_workspace_least):  # without gradients
        assert f(dt, N, V, H, 1, 0, 0) == L.spec_linear_loss_workspace_bytes(dt, N, V, H, 1, 0, 0)


def test_least_sizes_refuse_what_the_calls_refuse(L):  # noqa: F811
    f = L.spec_linear_loss_workspace_least
    assert f(F32, 1, 10, 8, 1, 0, 0) == f(3, 1, 10, 8, 1, 0, 0) == f(BF16, 1, 10, 12, 1, 0, 0) == 0
    assert f(BF16, -1, 10, 8, 1, 0, 0) == f(BF16, 1, 10, 8, 257, 1, 1) == f(BF16, (1 << 20) + 1, 10, 8, 1, 1, 1) == 0
    assert f(BF16, 0, 10, 8, 1, 1, 1) == 256
    for V in (1, 255, 2048, 2049):  # a vocabulary of a piece or less has little to save
        for dt in (BF16, F16):
            assert f(dt, 5, V, 64, 1, 1, 1) <= L.spec_linear_loss_workspace_bytes(dt, 5, V, 64, 1, 1, 1)


@pytest.mark.parametrize("bwd", [True, False])
def test_longest_rows(L, bwd):  # noqa: F811
    """The header's limit, on both sides: a row of 16 times 208 KiB and one vector more."""
    for dt, V in ((BF16, 1703936), (F16, 1703936), (F32, 851968)):
        assert kd(L, bwd=bwd, dt=dt, gdt=dt, V=V, ws=None) == INVALID  # only the workspace is missing
        assert kd(L, bwd=bwd, dt=dt, gdt=dt, V=V + 8, ws=None) == UNSUPPORTED

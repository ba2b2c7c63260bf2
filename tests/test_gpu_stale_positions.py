"""What a workspace holds from an earlier call names no rows, also where an entry of reverse_indices is no slot and every row
counts as routed: the slot that no entry names is like a dropped one, and every other slot has its own result."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu


# rows of whole 16-byte pieces and others; more slots than a CTA looks through by itself
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,k,H", [(5000, 2, 64), (5000, 2, 33), (1500, 8, 264), (9001, 1, 8)])
def test_a_slot_without_an_entry_has_no_row(dtype, T, k, H):
    moe = need_gpu()
    S = T * k
    g = torch.Generator(device=DEV).manual_seed(H)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV).to(dtype)  # noqa: E731
    d_out, y, d_x, w = n(T, H), n(S, H), n(S, H), torch.rand(T, k, generator=g, device=DEV)
    reverse = np.random.default_rng(T).permutation(S).astype(np.int32)
    off = torch.tensor([0] + [S] * max(4, k), dtype=torch.int32, device=DEV)
    rev = torch.from_numpy(reverse).to(DEV)
    need = max(moe.moe_ep_combine_backward_workspace_size(T, k), moe.moe_gather_rows_backward_workspace_size(T, k))
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    want_y, want_w = moe.moe_ep_combine_backward(d_out, y, w, rev, off)
    want_h = moe.moe_gather_rows_backward(d_x, rev, off, k)
    broken = rev.clone()
    row = S // 3                              # its slot has no entry now
    broken[row] = -1
    slot = int(reverse[row])
    for stale in (row + 1, row, 0, S - 1):    # a row of another slot, and its own
        words = ws.view(torch.int32)

        def left():
            words.fill_(stale)
            return ws

        d_y = torch.full_like(y, 7.0)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        got_y, got_w = moe.moe_ep_combine_backward(d_out, y, w, broken, off, d_y=d_y, workspace=left(), status=status)
        assert int(status) == moe.MOE_STATUS_BAD_INDEX
        got_h = moe.moe_gather_rows_backward(d_x, broken, off, k, workspace=left())
        others = torch.ones(S, dtype=torch.bool, device=DEV)
        others[row] = False
        assert torch.equal(got_y[others], want_y[others]) and (got_y[row] == 7).all()
        others = torch.ones(S, dtype=torch.bool, device=DEV)
        others[slot] = False
        assert torch.equal(got_w.view(-1)[others], want_w.view(-1)[others]) and float(got_w.view(-1)[slot]) == 0
        tokens = torch.ones(T, dtype=torch.bool, device=DEV)
        tokens[slot // k] = False
        assert torch.equal(got_h[tokens], want_h[tokens])
        alone = moe.moe_gather_rows_backward(torch.where(torch.arange(S, device=DEV)[:, None] == row, 0, d_x), rev, off, k)
        assert torch.equal(got_h[slot // k], alone[slot // k])


@pytest.mark.parametrize("dtype,H", [(torch.float16, 64), (torch.bfloat16, 33)])
def test_the_sum_back_takes_no_row_of_another_slot(dtype, H):
    moe = need_gpu()
    T, k = 5000, 2
    S = T * k
    g = torch.Generator(device=DEV).manual_seed(H)
    y, w = torch.randn(S, H, generator=g, device=DEV).to(dtype), torch.rand(T, k, generator=g, device=DEV)
    reverse = np.random.default_rng(H).permutation(S).astype(np.int32)
    off = torch.tensor([0, 0, 0, 0, S], dtype=torch.int32, device=DEV)
    rev = torch.from_numpy(reverse).to(DEV)
    row = S // 2
    broken = rev.clone()
    broken[row] = S
    ws = torch.full((S,), row + 1, dtype=torch.int32, device=DEV)
    got = moe.moe_ep_combine(y, w, broken, off, workspace=ws)
    w.view(-1)[int(reverse[row])] = 0         # the same without that row
    assert torch.equal(got, moe.moe_ep_combine(y, w, rev, off))

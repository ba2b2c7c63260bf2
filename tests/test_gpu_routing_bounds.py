"""Routing words that name nothing (slots, tokens and counts outside the arrays) on the forward steps around the expert
products: what they concern is left out or zero, everything else is as without them, whichever kernel the row width takes."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, need_gpu
from oracle import sorted_rows

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
LOW, HIGH = -2 ** 31, 2 ** 31 - 1


def half(dtype):
    return torch.finfo(dtype).eps / 2


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)


# widths of whole 16-byte pieces (kernels of their own in float32 and bf16) and others
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,H", [(6, 2, 64), (6, 2, 33), (3000, 3, 72), (3000, 3, 41), (9, 2, 16400)])
def test_combine_leaves_out_what_is_no_slot(dtype, T, k, H):
    moe = need_gpu()
    dt, S = TYPES[dtype], T * k
    g = torch.Generator().manual_seed(H)
    y, w = torch.randn(S, H, generator=g).to(dt), torch.rand(T, k, generator=g)
    reverse = np.random.default_rng(T).permutation(S).astype(np.int32)
    off = np.array([0, 0, S // 2, S], np.int32)
    bad = {0: -1, 1: S, 3: LOW, S - 1: HIGH}
    broken = reverse.copy()
    for p, v in bad.items():
        broken[p] = v
    got = moe.moe_ep_combine(y.to(DEV), w.to(DEV), i32(broken), i32(off)).double().cpu().numpy()
    kept = np.array([p not in bad for p in range(S)])
    rows, names = y.double().numpy()[kept], reverse[kept]      # the rows that have a slot, and their slots
    want = sorted_rows.combine(rows, w.double().numpy(), names, len(names))
    mag = sorted_rows.combine(np.abs(rows), w.double().numpy(), names, len(names))
    # k products and sums in float32, one rounding to the type
    assert (np.abs(got - want) <= 2 * k * 2.0 ** -24 * mag + 1.01 * half(dt) * (np.abs(want) + 2 * k * 2.0 ** -24 * mag) + 2.0 ** -25).all()
    # counts outside [0, S] are cut to it
    whole = moe.moe_ep_combine(y.to(DEV), w.to(DEV), i32(reverse), i32(off))
    for last, want in ((S + 1, whole), (HIGH, whole), (-1, torch.zeros_like(whole)), (LOW, torch.zeros_like(whole))):
        o = off.copy()
        o[-1] = last
        assert torch.equal(moe.moe_ep_combine(y.to(DEV), w.to(DEV), i32(reverse), i32(o)), want)


# bulk copies, 16-byte vectors (rows over 16 KB) and windows, by the rows' bytes
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,H", [(6, 2, 64), (6, 2, 33), (700, 3, 4096), (700, 3, 1001), (40, 2, 8192), (9, 2, 16400), (9, 2, 16401)])
def test_gather_gives_zeros_for_what_is_no_token(dtype, T, k, H):
    moe = need_gpu()
    dt, S = TYPES[dtype], T * k
    hidden = torch.randn(T, H, generator=torch.Generator().manual_seed(H)).to(dt)
    ids = (np.random.default_rng(T).permutation(S) // k).astype(np.int32)
    n = S - 2                                # the rows behind are left as they are
    off = np.array([0, 1, n // 2, n], np.int32)
    for p, v in ((0, -1), (1, T), (2, LOW), (n // 2, HIGH), (n // 2 + 1, T + 7), (n - 1, -5)):
        ids[p] = v
    there = torch.from_numpy((ids >= 0) & (ids < T))
    want = torch.where(there[:, None], hidden[torch.from_numpy(ids).long().clamp(0, T - 1)], torch.zeros(1, dtype=dt))
    out = torch.full((S, H), 7.0, dtype=dt, device=DEV)
    moe.moe_gather_rows(hidden.to(DEV), i32(ids), i32(off), k, out=out)
    assert torch.equal(out[:n].cpu(), want[:n]) and (out[n:] == 7).all()
    for last, rows in ((S + 1, S), (HIGH, S), (-1, 0), (LOW, 0)):
        o = off.copy()
        o[-1] = last
        out.fill_(7)
        moe.moe_gather_rows(hidden.to(DEV), i32(ids), i32(o), k, out=out)
        assert torch.equal(out[:rows].cpu(), want[:rows]) and (out[rows:] == 7).all()

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

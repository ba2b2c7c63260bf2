"""float32 grouped products that are large enough for the tensor cores (three bf16 parts a value): as exact as float32
sums, over float32's whole range, and blind to rows that no expert owns. Every test first makes sure that its calls take
that path: their workspaces then hold three parts, six bytes, of every value.

Tolerances. A product of parts leaves out less than 2^-24 of a value. An accumulator holds 128 terms; 8 of the additions
to it have its full size and are off by at most 2^-23 of it, 2^-24 on average and of half the size where all terms have
one sign: 3e-7. 5 to 17 sums are then added with 2^-24 each, of either sign: 2e-7. So 1e-6 in the 2-norm; without the
products of a third part (2^-17 of a value at most, a third of it in the mean) more than 2e-6 would be missing.
"""
import numpy as np
import pytest
import torch

from gpu_util import DEV, need_gpu
from oracle import grouped

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    return need_gpu()


def takes_parts(moe, S, K, N, E):
    """Whether the product and the gradients take the tensor cores."""
    return (moe.moe_grouped_gemm_workspace_size(moe.MOE_F32, S, K, N, E) >= 6 * (S + E * N) * K
            and moe.moe_grouped_gemm_backward_workspace_size(moe.MOE_F32, S, K, N, E) >= 6 * ((S + E * N) * K + S * N))


def normal(shape, seed, scale=1.0):
    return torch.from_numpy((np.random.default_rng(seed).standard_normal(shape) * scale).astype(np.float32))


def offsets(counts, first=0):
    off = np.concatenate([[first], first + np.cumsum(counts)]).astype(np.int32)
    return off, torch.from_numpy(off).to(DEV)


def run(moe, x, w, o, g):
    return (moe.moe_grouped_gemm(x, w, o), *moe.moe_grouped_gemm_backward(x, w, o, g))


def to64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("positive", [False, True])
@pytest.mark.parametrize("counts,K,N", [([1100, 0, 900], 517, 1030), ([4000, 3, 3997], 1024, 640), ([700, 900], 2048, 1100)])
def test_close_as_float32_is(moe, counts, K, N, positive):
    off, o = offsets(counts)
    S, E = int(off[-1]), len(counts)
    assert takes_parts(moe, S, K, N, E)
    x, w, g = normal((S, K), 1), normal((E, N, K), 2), normal((S, N), 3)
    if positive:
        x, w, g = abs(x), abs(w), abs(g)
    got = run(moe, x.to(DEV), w.to(DEV), o, g.to(DEV))
    x, w, g = x.double().numpy(), w.double().numpy(), g.double().numpy()
    for name, a, b in zip(("y", "d_x", "d_w"), got, (grouped.grouped_gemm(x, w, off), *grouped.grouped_gemm_backward(x, w, off, g))):
        assert np.linalg.norm(to64(a) - b) <= 1e-6 * np.linalg.norm(b), name


@pytest.mark.parametrize("junk", [float("nan"), float("inf"), 3.0e38])
def test_rows_without_an_expert_change_nothing(moe, junk):
    """Rows before the first group and after the last one: whatever they hold, the same bits come out."""
    off, o = offsets([1100, 0, 900], first=2)
    S, K, N, E = 2005, 517, 1030, 3
    assert takes_parts(moe, S, K, N, E)
    x, w, g = normal((S, K), 1).to(DEV), normal((E, N, K), 2).to(DEV), normal((S, N), 3).to(DEV)
    none = torch.ones(S, dtype=torch.bool, device=DEV)
    none[2:2002] = False
    x[none], g[none] = 0.0, 0.0
    want = run(moe, x, w, o, g)
    x[none], g[none] = junk, junk
    got = run(moe, x, w, o, g)
    for name, a, b in zip(("y", "d_x", "d_w"), got, want):
        assert torch.equal(a, b), name
    assert not got[0][none].any() and not got[1][none].any()

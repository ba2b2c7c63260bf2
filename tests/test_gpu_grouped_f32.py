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

TERM = 8 * 2.0 ** -23      # a sum with one term: six products, added with truncation, and what is left out
GRID = 2.0 ** -149


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


@pytest.mark.parametrize("junk", [float("nan"), float("inf"), 3.0e38, 1e-40])
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


def few_terms(S, K, N, E, off, terms):
    """Operands whose sums are all the given numbers times 4, `terms` in places 16 apart: for the product, for d_x and
    for d_w (one output column of it), and the operand that holds a 4 everywhere."""
    at = 16 * torch.arange(len(terms))
    v = torch.tensor(terms)
    x, g = torch.zeros(S, K), torch.zeros(S, N)
    x[:, at], g[:, at] = v, v
    gw = torch.zeros(S, N)
    for e in range(E):
        if off[e + 1] - off[e] > int(at[-1]):
            gw[off[e] + at] = v[:, None].expand(-1, N)
    return x.to(DEV), g.to(DEV), gw.to(DEV)


def test_sums_that_pass_near_the_largest_float32(moe):
    """A first term just below the largest float32 and three negative ones whose leading parts are too large: the small
    products of parts, which are added first, then carry the first term over the edge. In order all sums are finite."""
    off, o = offsets([1100, 0, 900])
    S, K, N, E = 2000, 517, 1030, 3
    assert takes_parts(moe, S, K, N, E)
    # 255/256 has 8 bits; 1/2 + 3/512 + 2^-20 rounds up to 1/2 + 4/512 in 8 bits, by almost half a step of 2^-8
    terms = [255 / 256 * 2.0 ** 126] + 3 * [-(0.5 + 3 / 512 + 2.0 ** -20) * 2.0 ** 126]
    want = sum(4 * t for t in terms)
    tol = 8 * 2.0 ** -23 * sum(abs(4 * t) for t in terms)
    x, g, gw = few_terms(S, K, N, E, off, terms)
    w, four = torch.full((E, N, K), 4.0, device=DEV), torch.full((S, K), 4.0, device=DEV)
    y = moe.moe_grouped_gemm(x, w, o)
    d_x, _ = moe.moe_grouped_gemm_backward(four, w, o, g, want_d_w=False)
    _, d_w = moe.moe_grouped_gemm_backward(four, w, o, gw, want_d_x=False)
    for name, got in (("y", y), ("d_x", d_x), ("d_w", d_w[[0, 2]])):
        assert torch.isfinite(got).all() and ((got.double() - want).abs() <= tol).all(), name


def test_largest_values_in_parts(moe):
    """128 terms of values just below those that leave the parts: their sum passes through 2^127 on the way."""
    off, o = offsets([1100, 0, 900])
    S, K, N, E = 2000, 517, 1030, 3
    rng = np.random.default_rng(4)
    x, w = np.zeros((S, K), np.float32), (1.9 + 0.099 * rng.random((E, N, K))).astype(np.float32) * np.float32(2.0 ** 43)
    x[:, :128] = (1.9 + 0.099 * rng.random((S, 128))).astype(np.float32) * np.float32(2.0 ** 43)
    y = moe.moe_grouped_gemm(torch.from_numpy(x).to(DEV), torch.from_numpy(w).to(DEV), o)
    want = grouped.grouped_gemm(x, w, off)
    assert torch.isfinite(y).all() and np.linalg.norm(to64(y) - want) <= 1e-6 * np.linalg.norm(want)


def one_term(moe, a, b):
    """Products and gradients all of whose sums have one term, a value of `a` times one of `b` -> pairs (got, exact)."""
    off, o = offsets([1100, 0, 900])
    S, K, N, E = 2000, 517, 1030, 3
    assert takes_parts(moe, S, K, N, E)
    left = lambda i: torch.tensor(a, device=DEV)[i % len(a)]  # noqa: E731
    right = lambda *s: torch.tensor(b, device=DEV)[torch.arange(int(np.prod(s)), device=DEV) % len(b)].reshape(s)  # noqa: E731
    p = torch.arange(S, device=DEV)
    expert = torch.from_numpy(grouped.expert_of_rows(off, S)).to(DEV)
    x, w, g = torch.zeros(S, K, device=DEV), right(E, N, K), torch.zeros(S, N, device=DEV)
    x[p, p % K] = left(p)
    yield moe.moe_grouped_gemm(x, w, o), x[p, p % K].double()[:, None] * w[expert, :, p % K].double()
    g[p, p % N] = left(p)
    d_x, _ = moe.moe_grouped_gemm_backward(x, w, o, g, want_d_w=False)
    yield d_x, g[p, p % N].double()[:, None] * w[expert, p % N].double()
    x, g = right(S, K), torch.zeros(S, N, device=DEV)
    g[7], g[1500] = left(torch.arange(N, device=DEV)), left(torch.arange(N, device=DEV) + 1)
    _, d_w = moe.moe_grouped_gemm_backward(x, w, o, g, want_d_x=False)
    want = torch.zeros(E, N, K, dtype=torch.float64, device=DEV)
    want[0], want[2] = g[7].double()[:, None] * x[7].double(), g[1500].double()[:, None] * x[1500].double()
    yield d_w, want


@pytest.mark.parametrize("a,b", [([1.999 * 2.0 ** 126], [1.999, -1.5]), ([1.999 * 2.0 ** 63, -(2.0 ** 63)], [1.999 * 2.0 ** 63]),
                                 ([1.998 * 2.0 ** 20], [1.9985 * 2.0 ** 106, 3.0])])
def test_results_next_to_the_largest_float32(moe, a, b):
    """Values whose leading parts round up, with a product that then passes the largest float32 while theirs does not."""
    for got, want in one_term(moe, a, b):
        assert torch.isfinite(got).all() and ((got.double() - want).abs() <= TERM * want.abs()).all()


@pytest.mark.parametrize("top", [55, 40])
@pytest.mark.parametrize("exponent", [-104, -110, -126, -130, -140])
def test_small_values_keep_their_bits(moe, exponent, top):
    """Values next to float32's smallest, times large ones."""
    small = (1 + np.random.default_rng(1).random(61)) * 2.0 ** exponent * np.random.default_rng(2).choice([-1, 1], 61)
    large = (1 + np.random.default_rng(3).random(53)) * 2.0 ** top
    for a, b in ((small, large), (large, small)):
        for got, want in one_term(moe, a.astype(np.float32).tolist(), b.astype(np.float32).tolist()):
            assert ((got.double() - want).abs() <= TERM * want.abs()).all()


@pytest.mark.parametrize("ex,ew", [(-60, -55), (-70, -50), (-75, -60)])
def test_small_sums_of_values_of_either_size(moe, ex, ew):
    """Sums whose low parts, or all of them, lie below float32's smallest normal value: a step of 2^-149 at most for
    each of the additions, 49 for 128 terms."""
    off, o = offsets([1100, 0, 900])
    S, K, N, E = 2000, 517, 1030, 3
    assert takes_parts(moe, S, K, N, E)
    x, w, g = normal((S, K), 1, 2.0 ** ex), normal((E, N, K), 2, 2.0 ** ew), normal((S, N), 3, 2.0 ** ew)
    y, d_x, d_w = run(moe, x.to(DEV), w.to(DEV), o, (g * 2.0 ** (ex - ew)).to(DEV))
    d_w = moe.moe_grouped_gemm_backward(x.to(DEV), w.to(DEV), o, g.to(DEV), want_d_x=False)[1]
    x, w, g = x.double().numpy(), w.double().numpy(), g.double().numpy()
    d_x64, d_w64 = grouped.grouped_gemm_backward(x, w, off, g * 2.0 ** (ex - ew))[0], grouped.grouped_gemm_backward(x, w, off, g)[1]
    for name, got, want, R in (("y", y, grouped.grouped_gemm(x, w, off), K), ("d_x", d_x, d_x64, N), ("d_w", d_w, d_w64, 1100)):
        steps = 49 * (R // 128 + 1)
        assert np.linalg.norm(to64(got) - want) <= 1e-6 * np.linalg.norm(want) + steps * GRID * want.size ** 0.5, name

"""Grouped products, their gradients and the 4-bit microscaled calls against the float64 oracle.

Tolerances. An output is rounded once, by at most u = half a step (2^-8 bf16, 2^-11 float16,
2^-24 float32) of its value. Before that it is a float32 sum of R products in some order; a
float32 addition that truncates is off by at most 2^-23 of its result, so the sum by at most
R 2^-23 A, where A is the sum of the products' magnitudes. float16 outputs below 2^-14 have a
step of 2^-24. With the gate, silu(g) u inherits the errors dg, du of its arguments
(|silu'| <= 1.1, |silu(g)| <= |g|) and the float32 exponential and division add at most
(8 + |g|) 2^-22 of the value.
"""
import numpy as np
import pytest
import torch

from gpu_util import DEV, need_gpu
from oracle import grouped, mxfp4

pytestmark = pytest.mark.gpu

TYPES = {"f32": (torch.float32, 2.0 ** -24), "bf16": (torch.bfloat16, 2.0 ** -8), "f16": (torch.float16, 2.0 ** -11)}


@pytest.fixture(scope="module")
def moe():
    return need_gpu()


def draw(shape, dtype, seed, scale=1.0):
    """Values of the dtype on the device and the same values in float64."""
    t = torch.from_numpy((np.random.default_rng(seed).standard_normal(shape) * scale).astype(np.float32)).to(TYPES[dtype][0])
    return t.to(DEV), t.double().numpy()


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def to64(t):
    return t.double().cpu().numpy()


def check(got, want, magnitude, R, dtype, what):
    u = TYPES[dtype][1]
    tol = u * np.abs(want) + (1 + u) * R * 2.0 ** -23 * magnitude + (2.0 ** -25 if dtype == "f16" else 2.0 ** -134)
    got = to64(got)
    assert got.shape == want.shape, what
    assert np.isfinite(got).all(), what
    bad = np.abs(got - want) > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.max((np.abs(got - want) - tol)[bad])}, first at {np.argwhere(bad)[0]}"


SHAPES = [
    # counts, rows beyond the groups, K, N
    ([1], 0, 64, 64),
    ([0, 1, 0], 0, 128, 256),
    ([8, 0, 3, 1], 2, 8, 8),
    ([5, 0, 130, 64, 1], 0, 72, 136),
    ([257, 255, 0, 256, 1], 3, 192, 520),
    ([300, 20, 513], 0, 1000, 264),
    ([2, 2, 1, 0, 0, 3, 1, 1], 0, 2048, 384),
    ([33, 70], 1, 63, 65),
    ([7, 0, 140], 0, 201, 77),
    ([3, 2], 0, 1, 1),
    ([1] * 40 + [0] * 3 + [17], 0, 96, 40),
]


# float32: reductions cut into pieces; then products that go to the tensor cores in parts
SHAPES_F32 = [
    ([3, 0, 9, 1], 2, 4100, 130),
    ([20, 7], 0, 90, 3001),
    ([200, 90], 1, 2500, 70),
    ([257, 255, 0, 256, 1], 3, 520, 523),
    ([63, 65, 1, 0, 500], 0, 777, 333),
    ([700], 1, 129, 1100),
    ([128, 64, 0, 192, 320], 0, 512, 640),
    ([5, 900, 0, 33], 2, 64, 1700),
    ([900, 0, 700, 1], 3, 517, 1030),
    ([2000, 30], 0, 129, 1100),
    ([1100, 600, 0, 300], 2, 1030, 264),
]


def shape_id(s):
    return f"{len(s[0])}x{sum(s[0])}+{s[1]}_K{s[2]}_N{s[3]}"


CASES = [(s, d) for s in SHAPES for d in ("f32", "bf16", "f16")] + [(s, "f32") for s in SHAPES_F32]
IDS = [f"{shape_id(s)}-{d}" for s, d in CASES]


@pytest.mark.parametrize("shape,dtype", CASES, ids=IDS)
def test_grouped_gemm(moe, shape, dtype):
    counts, beyond, K, N = shape
    off = offsets_of(counts)
    S, E = int(off[-1]) + beyond, len(counts)
    x, x64 = draw((S, K), dtype, 1)
    w, w64 = draw((E, N, K), dtype, 2, K ** -0.5)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full((S, N), float("nan"), dtype=x.dtype, device=DEV)
    y = moe.moe_grouped_gemm(x, w, torch.from_numpy(off).to(DEV), out=out, status=status)
    check(y, grouped.grouped_gemm(x64, w64, off), grouped.grouped_gemm(abs(x64), abs(w64), off), K, dtype, "y")
    assert int(status.item()) == 0


@pytest.mark.parametrize("shape,dtype", CASES, ids=IDS)
def test_grouped_gemm_backward(moe, shape, dtype):
    counts, beyond, K, N = shape
    off = offsets_of(counts)
    S, E = int(off[-1]) + beyond, len(counts)
    x, x64 = draw((S, K), dtype, 3)
    w, w64 = draw((E, N, K), dtype, 4, K ** -0.5)
    g, g64 = draw((S, N), dtype, 5)
    if beyond:                       # rows without an expert take no part, whatever they hold
        x[-beyond:], g[-beyond:] = float("inf"), float("nan")
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    d_x, d_w = moe.moe_grouped_gemm_backward(x, w, torch.from_numpy(off).to(DEV), g,
                                             d_x=torch.full_like(x, float("nan")), d_w=torch.full_like(w, float("nan")), status=status)
    rx, rw = grouped.grouped_gemm_backward(x64, w64, off, g64)
    ax, aw = grouped.grouped_gemm_backward(abs(x64), abs(w64), off, abs(g64))
    check(d_x, rx, ax, N, dtype, "d_x")
    check(d_w, rw, aw, max(max(counts), 1), dtype, "d_w")
    assert int(status.item()) == 0
    again_x, again_w = moe.moe_grouped_gemm_backward(x, w, torch.from_numpy(off).to(DEV), g)
    assert torch.equal(again_x, d_x) and torch.equal(again_w, d_w)      # the same bits
    only_x, none = moe.moe_grouped_gemm_backward(x, w, torch.from_numpy(off).to(DEV), g, want_d_w=False)
    assert none is None and torch.equal(only_x, d_x)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient_against_differences(moe, dtype):
    """The product is linear in each operand: f(x + h) - f(x - h) is the gradient's scalar product
    with 2 h. Entries are small integers and h is 1, so every sum is exact in float32 and every
    output (below 256) exact in bf16."""
    off = offsets_of([3, 0, 6, 1])
    rng = np.random.default_rng(6)
    t = TYPES[dtype][0]
    mk = lambda *s: torch.from_numpy(rng.integers(-2, 3, s).astype(np.float32)).to(t).to(DEV)  # noqa: E731
    x, w, g, o = mk(10, 16), mk(4, 8, 16), mk(10, 8), torch.from_numpy(off).to(DEV)
    d_x, d_w = moe.moe_grouped_gemm_backward(x, w, o, g)
    f = lambda x, w: float((moe.moe_grouped_gemm(x, w, o).double() * g.double()).sum())  # noqa: E731
    for _ in range(6):
        hx, hw = mk(10, 16), mk(4, 8, 16)
        assert f(x + hx, w) - f(x - hx, w) == 2 * float((d_x.double() * hx.double()).sum())
        assert f(x, w + hw) - f(x, w - hw) == 2 * float((d_w.double() * hw.double()).sum())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_values_do_not_leak_between_groups(moe, dtype):
    """An expert whose rows and weights are NaN or infinite leaves its neighbours alone, in tiles
    that hold rows of several experts and in reductions that end inside a tile."""
    off = offsets_of([5, 9, 70, 3])
    S, K, N = 87, 72, 88
    x, x64 = draw((S, K), dtype, 7)
    w, w64 = draw((4, N, K), dtype, 8)
    g, g64 = draw((S, N), dtype, 9)
    for t in (x, g):
        t[5:14] = float("nan")
    w[1] = float("inf")
    for a in (x64, g64):
        a[5:14] = 0
    w64[1] = 0
    o = torch.from_numpy(off).to(DEV)
    keep = np.r_[0:5, 14:87]
    y = moe.moe_grouped_gemm(x, w, o)
    want, mag = grouped.grouped_gemm(x64, w64, off), grouped.grouped_gemm(abs(x64), abs(w64), off)
    check(y[keep], want[keep], mag[keep], K, dtype, "y")
    assert not torch.isfinite(y[5:14]).any()
    d_x, d_w = moe.moe_grouped_gemm_backward(x, w, o, g)
    rx, rw = grouped.grouped_gemm_backward(x64, w64, off, g64)
    ax, aw = grouped.grouped_gemm_backward(abs(x64), abs(w64), off, abs(g64))
    check(d_x[keep], rx[keep], ax[keep], N, dtype, "d_x")
    check(d_w[[0, 2, 3]], rw[[0, 2, 3]], aw[[0, 2, 3]], 70, dtype, "d_w")


def test_f32_in_parts_is_float32(moe):
    """Large float32 products: close to float64 as float32 sums are (2-norm), in both directions, also
    where all products have one sign, so that a bias of the sums would add up."""
    off = offsets_of([300, 0, 212])
    o = torch.from_numpy(off).to(DEV)
    for positive in (False, True):
        x, x64 = draw((512, 2048), "f32", 1)
        w, w64 = draw((3, 384, 2048), "f32", 2)
        g, g64 = draw((512, 384), "f32", 3)
        if positive:
            x, w, g, x64, w64, g64 = abs(x), abs(w), abs(g), abs(x64), abs(w64), abs(g64)
        y = moe.moe_grouped_gemm(x, w, o)
        d_x, d_w = moe.moe_grouped_gemm_backward(x, w, o, g)
        for got, want in zip((y, d_x, d_w), (grouped.grouped_gemm(x64, w64, off), *grouped.grouped_gemm_backward(x64, w64, off, g64))):
            # sums of n rounded additions: at most n 2^-24 of the magnitudes, and their square root in the mean;
            # 16 of them between two roundings to nearest, 6e-8 each, are 1e-6
            assert np.linalg.norm(to64(got) - want) <= 1e-6 * np.linalg.norm(want)


def test_f32_infinities_follow_float32(moe):
    """Infinities, NaN and values next to the largest float32 give what float32 arithmetic gives."""
    off = offsets_of([257, 255, 0, 256, 1])
    o = torch.from_numpy(off).to(DEV)
    x, _ = draw((769, 520), "f32", 1)
    w, _ = draw((5, 523, 520), "f32", 2)
    x[3, 5], x[300, 0], x[600, 519], x[601, 2] = float("inf"), float("nan"), -float("inf"), 3.0e38
    y = moe.moe_grouped_gemm(x, w, o).cpu()
    e = grouped.expert_of_rows(off, 769)
    for p in (3, 300, 600, 601, 0, 768):
        want = (x[p].double() * w[e[p]].double()).sum(1).float().cpu()
        assert torch.equal(torch.isnan(y[p]), torch.isnan(want)) and torch.equal(torch.isinf(y[p]), torch.isinf(want))
        fin = torch.isfinite(want)
        assert torch.equal(torch.sign(y[p][~torch.isnan(want)]), torch.sign(want[~torch.isnan(want)]))
        assert (y[p][fin] - want[fin]).abs().max() <= 1e-5 * max(1e-30, float(want[fin].abs().max())) if fin.any() else True


def test_f32_values_without_parts_in_a_large_product(moe):
    """Infinities, NaN and 3e38 among the rows of a product that is large enough for the tensor cores."""
    off = offsets_of([1100, 0, 900])
    o = torch.from_numpy(off).to(DEV)
    x, x64 = draw((2003, 517), "f32", 1)
    w, w64 = draw((3, 1030, 517), "f32", 2)
    plain = moe.moe_grouped_gemm(x, w, o)
    for value in (float("inf"), float("nan"), 3.0e38):
        y = x.clone()
        y[1500, 516] = value
        got = moe.moe_grouped_gemm(y, w, o)
        want = (y[1500].double() * w[2].double()).sum(1).float()
        assert torch.equal(torch.isnan(got[1500]), torch.isnan(want)) and torch.equal(torch.isinf(got[1500]), torch.isinf(want))
        ok = torch.isfinite(want)
        if ok.any():
            assert ((got[1500] - want)[ok].abs() <= 1e-5 * want[ok].abs().max()).all()
        rest = torch.arange(2003, device=DEV) != 1500
        # both float32: 517 rounded additions each, in the 2-norm far below 517 2^-24
        assert (got[rest] - plain[rest]).double().norm() <= 2 * 517 * 2.0 ** -24 * plain[rest].double().norm()
    assert not plain[2000:].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bad_offsets_are_reported(moe, dtype):
    x, _ = draw((40, 64), dtype, 1)
    w, _ = draw((3, 64, 64), dtype, 2)
    g, _ = draw((40, 64), dtype, 3)
    for off in ([0, 20, 10, 40], [-5, 3, 9, 40], [0, 3, 9, 41], [0, 1 << 30, 1 << 30, 40]):
        o = torch.tensor(off, dtype=torch.int32, device=DEV)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        moe.moe_grouped_gemm(x, w, o, status=status)
        assert int(status.item()) == moe.MOE_STATUS_BAD_INDEX
        status.zero_()
        moe.moe_grouped_gemm_backward(x, w, o, g, status=status)
        assert int(status.item()) == moe.MOE_STATUS_BAD_INDEX


def test_no_more_than_the_workspace_is_written(moe):
    """A workspace of just the size asked for, with guards on both sides."""
    off = torch.tensor([0, 200, 200, 600], dtype=torch.int32, device=DEV)
    for dtype, K, N in (("bf16", 129, 515), ("f32", 513, 515), ("f16", 257, 130)):
        t = TYPES[dtype][0]
        x, _ = draw((600, K), dtype, 1)
        w, _ = draw((3, N, K), dtype, 2)
        g, _ = draw((600, N), dtype, 3)
        code = {"f32": moe.MOE_F32, "bf16": moe.MOE_BF16, "f16": moe.MOE_F16}[dtype]
        n = moe.moe_grouped_gemm_workspace_size(code, 600, K, N, 3)
        m = moe.moe_grouped_gemm_backward_workspace_size(code, 600, K, N, 3)
        assert n > 0 and m > 0
        buf = torch.full((max(n, m) + 8192,), 77, dtype=torch.uint8, device=DEV)
        y = moe.moe_grouped_gemm(x, w, off, workspace=buf[4096:4096 + n])
        assert torch.equal(y, moe.moe_grouped_gemm(x, w, off))
        assert (buf[:4096] == 77).all() and (buf[4096 + n:] == 77).all()
        moe.moe_grouped_gemm_backward(x, w, off, g, workspace=buf[4096:4096 + m])
        assert (buf[:4096] == 77).all() and (buf[4096 + m:] == 77).all()
        with pytest.raises(moe.MoeError, match="too small"):
            moe.moe_grouped_gemm(x, w, off, workspace=buf[4096:4096 + n - 256])
    c, s = moe.moe_mxfp4_quantize(torch.randn(600, 288, device=DEV))
    wc, ws = moe.moe_mxfp4_quantize(torch.randn(3, 260, 288, device=DEV))
    for act in (None, "silu_and_mul"):
        n = moe.moe_mxfp4_grouped_gemm_workspace_size(600, 288, 260, 3, act)
        assert n > 0
        buf = torch.full((n + 8192,), 77, dtype=torch.uint8, device=DEV)
        y = moe.moe_mxfp4_grouped_gemm(c, s, wc, ws, off, activation=act, workspace=buf[4096:4096 + n])
        assert torch.equal(y, moe.moe_mxfp4_grouped_gemm(c, s, wc, ws, off, activation=act))
        assert (buf[:4096] == 77).all() and (buf[4096 + n:] == 77).all()


def test_binding_refusals(moe):
    x, _ = draw((10, 64), "bf16", 1)
    w, _ = draw((2, 32, 64), "bf16", 2)
    off = torch.tensor([0, 4, 10], dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_grouped_gemm(x.t().contiguous().t(), w, off)
    with pytest.raises(ValueError, match="w must be torch.bfloat16"):
        moe.moe_grouped_gemm(x, w.half(), off)
    with pytest.raises(ValueError, match="shapes"):
        moe.moe_grouped_gemm(x, w[:, :, :32].contiguous(), off)
    with pytest.raises(ValueError, match="shapes"):
        moe.moe_grouped_gemm(x, w, off[:2].contiguous())
    with pytest.raises(ValueError, match="int32"):
        moe.moe_grouped_gemm(x, w, off.long())
    with pytest.raises(ValueError, match="out must have shape"):
        moe.moe_grouped_gemm(x, w, off, out=torch.empty(10, 31, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError, match="unsupported dtype"):
        moe.moe_grouped_gemm(x.double(), w.double(), off)
    with pytest.raises(ValueError, match="status"):
        moe.moe_grouped_gemm(x, w, off, status=torch.zeros(1, device=DEV))
    with pytest.raises(moe.MoeError, match="aligned"):
        moe.moe_grouped_gemm(torch.zeros(10 * 64 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(10, 64), w, off)
    with pytest.raises(ValueError, match="multiple of 32"):
        moe.moe_mxfp4_quantize(torch.zeros(4, 48, device=DEV))
    with pytest.raises(ValueError, match="rows"):
        moe.moe_mxfp4_quantize(torch.zeros(4, 2, 64, device=DEV), rows=off)
    c, s = moe.moe_mxfp4_quantize(x)
    wc, ws = moe.moe_mxfp4_quantize(w)
    with pytest.raises(ValueError, match="activation"):
        moe.moe_mxfp4_grouped_gemm(c, s, wc, ws, off, activation="gelu")
    with pytest.raises(ValueError, match="scales"):
        moe.moe_mxfp4_grouped_gemm(c, s[:, :1].contiguous(), wc, ws, off)
    with pytest.raises(ValueError, match="even"):
        moe.moe_mxfp4_grouped_gemm(c, s, wc[:, :31].contiguous(), ws[:, :31].contiguous(), off, activation="silu_and_mul")
    with pytest.raises(ValueError, match="scales"):
        moe.moe_mxfp4_dequantize(c, s[:5])


def test_wait_limits_give_up(moe):
    """A limit too short for any wait: the kernels report it and the next call is right."""
    off = torch.tensor([0, 300, 1000], dtype=torch.int32, device=DEV)
    x, _ = draw((1000, 512), "bf16", 1)
    w, _ = draw((2, 512, 512), "bf16", 2)
    g, _ = draw((1000, 512), "bf16", 3)
    c, s = moe.moe_mxfp4_quantize(x)
    wc, ws = moe.moe_mxfp4_quantize(w)
    calls = [lambda st: moe.moe_grouped_gemm(x, w, off, status=st),
             lambda st: moe.moe_grouped_gemm(x.float(), w.float(), off, status=st),
             lambda st: moe.moe_grouped_gemm_backward(x, w, off, g, status=st)[1],
             lambda st: moe.moe_grouped_gemm(x[:20].contiguous(), w, off.clamp(max=20), status=st),
             lambda st: moe.moe_mxfp4_grouped_gemm(c, s, wc, ws, off, status=st),
             lambda st: moe.moe_mxfp4_grouped_gemm(c[:20].contiguous(), s[:20].contiguous(), wc, ws, off.clamp(max=20), activation="silu_and_mul", status=st)]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = [f(status).clone() for f in calls]
    assert int(status.item()) == 0
    for f, y in zip(calls, want):
        before = moe.set_wait_limit_ns(1)
        try:
            status.zero_()
            f(status)
            torch.cuda.synchronize()
            assert int(status.item()) == moe.MOE_STATUS_TIMEOUT
        finally:
            moe.set_wait_limit_ns(before)
        status.zero_()
        assert torch.equal(f(status), y) and int(status.item()) == 0


@pytest.mark.parametrize("S", [3000, 90000])
def test_most_experts(moe, S):
    """1024 experts, most with few rows, some with none, in every operator."""
    rng = np.random.default_rng(S)
    counts = rng.multinomial(S, rng.dirichlet(np.full(1024, 0.3)))
    off = offsets_of(counts)
    assert (counts == 0).any()
    o = torch.from_numpy(off).to(DEV)
    for dtype in ("f32", "bf16"):
        x, x64 = draw((S, 64), dtype, 1)
        w, w64 = draw((1024, 72, 64), dtype, 2)
        g, g64 = draw((S, 72), dtype, 3)
        check(moe.moe_grouped_gemm(x, w, o), grouped.grouped_gemm(x64, w64, off), grouped.grouped_gemm(abs(x64), abs(w64), off), 64, dtype, "y")
        d_x, d_w = moe.moe_grouped_gemm_backward(x, w, o, g)
        rx, rw = grouped.grouped_gemm_backward(x64, w64, off, g64)
        ax, aw = grouped.grouped_gemm_backward(abs(x64), abs(w64), off, abs(g64))
        check(d_x, rx, ax, 72, dtype, "d_x")
        check(d_w, rw, aw, int(counts.max()), dtype, "d_w")
    c, s = moe.moe_mxfp4_quantize(x)
    wc, ws = moe.moe_mxfp4_quantize(w)
    xv, wv = to64(moe.moe_mxfp4_dequantize(c, s)), to64(moe.moe_mxfp4_dequantize(wc, ws))
    check(moe.moe_mxfp4_grouped_gemm(c, s, wc, ws, o), grouped.grouped_gemm(xv, wv, off), grouped.grouped_gemm(abs(xv), abs(wv), off), 64, "bf16", "y4")


def test_more_than_2_31_elements(moe):
    """Rows whose element offsets pass 32 bits, in inputs and outputs: the last ones are those of a
    call on them alone."""
    S, n = 1100000, 777
    off = torch.tensor([0, 5, S - n, S], dtype=torch.int32, device=DEV)
    tail = torch.tensor([0, 0, 0, n], dtype=torch.int32, device=DEV)
    x = torch.empty(S, 2048, dtype=torch.bfloat16, device=DEV)
    x[:-n].fill_(1.0)
    x[-n:] = draw((n, 2048), "bf16", 1)[0]
    w, _ = draw((3, 64, 2048), "bf16", 2)
    y = moe.moe_grouped_gemm(x, w, off)
    assert torch.equal(y[-n:], moe.moe_grouped_gemm(x[-n:].contiguous(), w, tail))
    w2, _ = draw((3, 2048, 64), "bf16", 3)
    y2 = moe.moe_grouped_gemm(y, w2, off)                       # output past 2^31
    assert torch.equal(y2[-n:], moe.moe_grouped_gemm(y[-n:].contiguous(), w2, tail))
    d_x, _ = moe.moe_grouped_gemm_backward(x, w, off, y, d_x=y2, want_d_w=False)
    want, dw = moe.moe_grouped_gemm_backward(x[-n:].contiguous(), w, tail, y[-n:].contiguous())
    assert torch.equal(d_x[-n:], want)
    _, d_w = moe.moe_grouped_gemm_backward(x, w, off, y, want_d_x=False)
    assert torch.equal(d_w[2], dw[2])
    c, s = moe.moe_mxfp4_quantize(x)
    tc, ts = moe.moe_mxfp4_quantize(x[-n:].contiguous())
    assert torch.equal(c[-n:], tc) and torch.equal(s[-n:], ts)
    moe.moe_mxfp4_dequantize(c, s, out=y2)
    assert torch.equal(y2[-n:], moe.moe_mxfp4_dequantize(tc, ts))
    wc, ws = moe.moe_mxfp4_quantize(w)
    y4 = moe.moe_mxfp4_grouped_gemm(c, s, wc, ws, off, out=y)
    assert torch.equal(y4[-n:], moe.moe_mxfp4_grouped_gemm(tc, ts, wc, ws, tail))


def test_empty_sizes(moe):
    o = torch.zeros(3, dtype=torch.int32, device=DEV)
    for dtype in (torch.float32, torch.bfloat16):
        z = lambda *s: torch.zeros(s, dtype=dtype, device=DEV)  # noqa: E731
        assert moe.moe_grouped_gemm(z(0, 64), z(2, 64, 64), o).shape == (0, 64)
        assert moe.moe_grouped_gemm(z(3, 64), z(2, 0, 64), o).shape == (3, 0)
        y = moe.moe_grouped_gemm(z(3, 0), z(2, 64, 0), o, out=torch.ones(3, 64, dtype=dtype, device=DEV))
        assert not y.any()
        d_x, d_w = moe.moe_grouped_gemm_backward(z(0, 64), z(2, 64, 64), o, z(0, 64), d_w=torch.ones(2, 64, 64, dtype=dtype, device=DEV))
        assert d_x.shape == (0, 64) and not d_w.any()
        d_x, d_w = moe.moe_grouped_gemm_backward(z(3, 64), z(2, 0, 64), o, z(3, 0), d_x=torch.ones(3, 64, dtype=dtype, device=DEV))
        assert not d_x.any() and d_w.shape == (2, 0, 64)
    c, s = moe.moe_mxfp4_quantize(torch.zeros(0, 64, device=DEV))
    assert c.shape == (0, 32) and s.shape == (0, 2)
    assert moe.moe_mxfp4_dequantize(c, s).shape == (0, 64)


def test_other_stream_and_graph(moe):
    """On a stream of the caller's, and captured into a graph that is replayed on new inputs."""
    off = torch.tensor([0, 40, 100], dtype=torch.int32, device=DEV)
    x, _ = draw((100, 128), "bf16", 1)
    w, _ = draw((2, 192, 128), "bf16", 2)
    g, _ = draw((100, 192), "bf16", 3)
    want, (wx, ww) = moe.moe_grouped_gemm(x, w, off), moe.moe_grouped_gemm_backward(x, w, off, g)
    codes, scales = moe.moe_mxfp4_quantize(x)
    wc, ws = moe.moe_mxfp4_quantize(w)
    w4 = moe.moe_mxfp4_grouped_gemm(codes, scales, wc, ws, off)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = moe.moe_grouped_gemm(x, w, off)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    out, dx, dw, y4 = torch.empty_like(want), torch.empty_like(wx), torch.empty_like(ww), torch.empty_like(w4)
    xin = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_grouped_gemm(xin, w, off, out=out)
        moe.moe_grouped_gemm_backward(xin, w, off, g, d_x=dx, d_w=dw)
        c, sc = moe.moe_mxfp4_quantize(xin)
        moe.moe_mxfp4_grouped_gemm(c, sc, wc, ws, off, out=y4)
    xin.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(dx, wx) and torch.equal(dw, ww) and torch.equal(y4, w4)


def test_workspace_on_a_stream_of_the_callers(moe):
    """A call on another stream with a workspace of its own making: what the current stream allocates
    next must not be that workspace while the call may still run."""
    off = torch.tensor([0, 200, 600], dtype=torch.int32, device=DEV)
    x, _ = draw((600, 129), "bf16", 1)
    w, _ = draw((2, 515, 129), "bf16", 2)
    want = moe.moe_grouped_gemm(x, w, off)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        got = torch.zeros_like(want)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(2000000)
        moe.moe_grouped_gemm(x, w, off, out=got, stream=stream)
        junk = [torch.full((moe.moe_grouped_gemm_workspace_size(moe.MOE_BF16, 600, 129, 515, 2),), 255, dtype=torch.uint8, device=DEV) for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(got, want) and junk


def test_memory_of_a_call_on_another_stream(moe):
    """Outputs and workspaces made for a call on a stream of the caller's: what the current stream has given
    back, but not yet read, must not be among them; nor may an output that the current stream still reads be
    given out again on the other stream."""
    off = torch.tensor([0, 200, 600], dtype=torch.int32, device=DEV)
    x, _ = draw((600, 129), "bf16", 1)
    w, _ = draw((2, 515, 129), "bf16", 2)
    want = moe.moe_grouped_gemm(x, w, off)
    size = moe.moe_grouped_gemm_workspace_size(moe.MOE_BF16, 600, 129, 515, 2)
    assert size > 0
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        torch.cuda.synchronize()
        mine = [torch.full((n,), 7, dtype=torch.uint8, device=DEV) for n in (size, 600 * 515 * 2) for _ in range(2)]
        s.wait_stream(torch.cuda.current_stream())
        torch.cuda._sleep(2000000)
        copies = [m.clone() for m in mine]
        del mine
        got = moe.moe_grouped_gemm(x, w, off, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and all((c == 7).all() for c in copies)
        torch.cuda._sleep(2000000)
        kept = got.clone()
        del got
        with torch.cuda.stream(s):
            junk = [torch.full((600, 515), 3, dtype=want.dtype, device=DEV) for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(kept, want) and junk


# ---- 4-bit microscaled values ----------------------------------------------------------


def bytes_of(code):
    return torch.from_numpy(mxfp4.pack(code)).to(DEV)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,K", [(1, 32), (3, 64), (7, 2048), (129, 96), (1000, 1408), (5, 32 * 33)])
def test_quantize(moe, dtype, T, K):
    x, x64 = draw((T, K), dtype, T + K)
    x *= torch.exp(torch.from_numpy(np.random.default_rng(9).standard_normal((T, 1)).astype(np.float32))).to(x)
    x64 = to64(x)
    codes, scales = moe.moe_mxfp4_quantize(x)
    rc, rs = mxfp4.quantize(x64)
    assert torch.equal(scales.cpu(), torch.from_numpy(rs))
    assert torch.equal(codes.cpu(), torch.from_numpy(mxfp4.pack(rc)))
    for out, (t, _) in TYPES.items():
        v = moe.moe_mxfp4_dequantize(codes, scales, dtype=t)
        want = torch.from_numpy(mxfp4.dequantize(rc, rs)).to(t)
        assert torch.equal(v.cpu(), want)


def test_quantize_ties_extremes_and_nonfinite(moe):
    """Every tie of the grid at several scales, subnormal and largest values, infinities and NaN."""
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.5, 7.5, 4.0])
    rows = []
    for s in (-126, -100, -1, 0, 1, 60, 124):
        r = np.zeros(32)
        r[:10], r[10:20], r[31] = ties, -ties, 7.0
        rows.append(r * 2.0 ** s)
    for e in (-149, -140, -130, -127, -126, 127):
        r = np.zeros(32)
        r[7], r[8] = 2.0 ** e, -(2.0 ** e)
        rows.append(r)
    rows += [np.zeros(32), np.full(32, -0.0), np.full(32, 3.4028234663852886e38)]
    for v in (np.nan, np.inf, -np.inf, -np.nan):
        r = np.ones(32)
        r[13] = v
        rows.append(r)
    x = np.stack(rows).astype(np.float32)
    codes, scales = moe.moe_mxfp4_quantize(torch.from_numpy(x).to(DEV))
    rc, rs = mxfp4.quantize(x.astype(np.float64))
    assert torch.equal(scales.cpu(), torch.from_numpy(rs))
    assert torch.equal(codes.cpu(), torch.from_numpy(mxfp4.pack(rc)))
    v = moe.moe_mxfp4_dequantize(codes, scales, dtype=torch.float32).cpu().double().numpy()
    np.testing.assert_array_equal(v, mxfp4.dequantize(rc, rs))


def test_quantize_rows(moe):
    x, x64 = draw((50, 96), "bf16", 1)
    rows = torch.tensor([3, 3, 49, 0, 7, -1, 50, 1 << 30, 12], dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    codes, scales = moe.moe_mxfp4_quantize(x, rows=rows, status=status)
    assert int(status.item()) == moe.MOE_STATUS_BAD_INDEX
    all_c, all_s = moe.moe_mxfp4_quantize(x)
    for r, t in enumerate(rows.tolist()):
        if 0 <= t < 50:
            assert torch.equal(codes[r], all_c[t]) and torch.equal(scales[r], all_s[t])
        else:
            assert not codes[r].any() and not scales[r].any()
    status.zero_()
    moe.moe_mxfp4_quantize(x, rows=rows[:5].contiguous(), status=status)
    assert int(status.item()) == 0


@pytest.mark.parametrize("K", [2048, 1056, 1120])
def test_quantize_rows_many_times(moe, K):
    """Each row wanted several times: quantised once, then copied."""
    x, _ = draw((700, K), "bf16", 2)
    g = torch.Generator().manual_seed(3)
    rows = torch.randint(0, 700, (6000,), dtype=torch.int32, generator=g)
    rows[17], rows[5999] = -4, 700
    assert moe.moe_mxfp4_quantize_workspace_size(700, K, True, 6000) > 0
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    codes, scales = moe.moe_mxfp4_quantize(x, rows=rows.to(DEV), status=status)
    assert int(status.item()) == moe.MOE_STATUS_BAD_INDEX
    all_c, all_s = moe.moe_mxfp4_quantize(x)
    good = (rows >= 0) & (rows < 700)
    at = torch.where(good, rows, 0).long().to(DEV)
    keep = good.to(DEV)[:, None]
    assert torch.equal(codes, all_c[at] * keep) and torch.equal(scales, all_s[at] * keep)


SHAPES4 = [
    ([1], 0, 32, 16),
    ([0, 3, 0], 0, 64, 256),
    ([8, 0, 3, 1], 2, 96, 30),
    ([5, 0, 130, 64, 1], 0, 256, 258),
    ([257, 255, 0, 256, 1], 3, 160, 520),
    ([300, 20, 513], 1, 1408, 264),
    ([2, 2, 1, 0, 0, 3, 1, 1], 0, 2048, 384),
    ([1] * 40 + [0] * 3 + [17], 0, 512, 130),
    ([700], 0, 4096, 600),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("shape", SHAPES4, ids=shape_id)
def test_mxfp4_grouped_gemm(moe, shape, silu, dtype):
    counts, beyond, K, N = shape
    off = offsets_of(counts)
    S, E = int(off[-1]) + beyond, len(counts)
    rng = np.random.default_rng(K + N)
    xc, wc = rng.integers(0, 16, (S, K)).astype(np.uint8), rng.integers(0, 16, (E, N, K)).astype(np.uint8)
    # scales that differ from block to block and row to row, small enough for float16 outputs
    xs, ws = rng.integers(118, 126, (S, K // 32)).astype(np.uint8), rng.integers(119, 126, (E, N, K // 32)).astype(np.uint8)
    x64, w64 = mxfp4.dequantize(xc, xs), mxfp4.dequantize(wc, ws)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    t, u = TYPES[dtype]
    out = torch.full((S, N // 2 if silu else N), float("nan"), dtype=t, device=DEV)
    y = moe.moe_mxfp4_grouped_gemm(bytes_of(xc), torch.from_numpy(xs).to(DEV), bytes_of(wc), torch.from_numpy(ws).to(DEV),
                                   torch.from_numpy(off).to(DEV), activation="silu_and_mul" if silu else None,
                                   out_dtype=t, out=out, status=status)
    assert int(status.item()) == 0
    want, mag = grouped.grouped_gemm(x64, w64, off), grouped.grouped_gemm(abs(x64), abs(w64), off)
    if not silu:
        check(y, want, mag, K, dtype, "y")
        return
    h, err = N // 2, K * 2.0 ** -23 * mag
    g, v = want[:, :h], want[:, h:]
    ref = mxfp4.silu_and_mul(want)
    tol = 1.1 * err[:, :h] * (np.abs(v) + err[:, h:]) + np.abs(g) * err[:, h:] + (8 + np.abs(g)) * 2.0 ** -22 * np.abs(ref)
    tol = u * np.abs(ref) + (1 + u) * tol + (2.0 ** -25 if dtype == "f16" else 2.0 ** -134)
    bad = ~(np.abs(to64(y) - ref) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}"


def test_mxfp4_exact_sums(moe):
    """Unit scales and few terms: every sum is a multiple of 1/4 below 2^22, exact in float32."""
    rng = np.random.default_rng(3)
    off = offsets_of([130, 0, 77])
    xc, wc = rng.integers(0, 16, (207, 512)).astype(np.uint8), rng.integers(0, 16, (3, 144, 512)).astype(np.uint8)
    one = lambda *s: torch.full(s, 127, dtype=torch.uint8, device=DEV)  # noqa: E731
    y = moe.moe_mxfp4_grouped_gemm(bytes_of(xc), one(207, 16), bytes_of(wc), one(3, 144, 16), torch.from_numpy(off).to(DEV),
                                   out_dtype=torch.float32)
    unit = np.full(1, 127, np.uint8)
    dec = lambda c: mxfp4.dequantize(c, np.broadcast_to(unit, c.shape[:-1] + (16,)))  # noqa: E731
    np.testing.assert_array_equal(to64(y), grouped.grouped_gemm(dec(xc), dec(wc), off))


def test_mxfp4_nan_scales_stay_in_their_rows(moe):
    rng = np.random.default_rng(4)
    off = offsets_of([20, 150])
    xc, wc = rng.integers(0, 16, (170, 256)).astype(np.uint8), rng.integers(0, 16, (2, 64, 256)).astype(np.uint8)
    xs, ws = np.full((170, 8), 120, np.uint8), np.full((2, 64, 8), 121, np.uint8)
    clean = moe.moe_mxfp4_grouped_gemm(bytes_of(xc), torch.from_numpy(xs).to(DEV), bytes_of(wc), torch.from_numpy(ws).to(DEV),
                                       torch.from_numpy(off).to(DEV))
    xs[5, 3], xs[100, 7], ws[1, 9, 0] = 255, 255, 255
    y = moe.moe_mxfp4_grouped_gemm(bytes_of(xc), torch.from_numpy(xs).to(DEV), bytes_of(wc), torch.from_numpy(ws).to(DEV),
                                   torch.from_numpy(off).to(DEV))
    nan = torch.zeros_like(y, dtype=torch.bool)
    nan[5], nan[100], nan[20:, 9] = True, True, True
    assert torch.equal(torch.isnan(y), nan)
    assert torch.equal(y[~nan], clean[~nan])


def test_mxfp4_bad_offsets_are_reported(moe):
    x = torch.zeros(40, 32, dtype=torch.uint8, device=DEV)
    w = torch.zeros(3, 64, 32, dtype=torch.uint8, device=DEV)
    xs, ws = torch.zeros(40, 2, dtype=torch.uint8, device=DEV), torch.zeros(3, 64, 2, dtype=torch.uint8, device=DEV)
    for off in ([0, 20, 10, 40], [0, 3, 9, 41]):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        moe.moe_mxfp4_grouped_gemm(x, xs, w, ws, torch.tensor(off, dtype=torch.int32, device=DEV), status=status)
        assert int(status.item()) == moe.MOE_STATUS_BAD_INDEX

"""8-bit rows and weights on the GPU against the oracle: quantisation bit for bit, the norm, the copy into expert order, and
the grouped product."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, need_gpu
from oracle import fp8, grouped

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
F8 = torch.float8_e4m3fn


def half(dtype):
    return torch.finfo(dtype).eps / 2


def bits(t):
    return t.view(torch.uint8).cpu().numpy()


def rows_of(T, K, dtype, seed=0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, K, generator=g) * torch.exp(spread * torch.randn(T, 1, generator=g))).to(dtype)


def same(got, want):
    codes, scales = got
    np.testing.assert_array_equal(scales.cpu().numpy(), want[1])
    np.testing.assert_array_equal(bits(codes), want[0])


# ---- quantisation ------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K", [(1, 16), (1, 2048), (3, 128), (7, 144), (64, 1408), (5, 4096), (33, 400), (500, 272), (2, 16384)])
def test_rows(dtype, T, K):
    moe = need_gpu()
    x = rows_of(T, K, TYPES[dtype], seed=K)
    got = moe.moe_fp8_quantize(x.to(DEV))
    want = fp8.quantize(x.float().numpy())
    same(got, want)
    values = fp8.dequantize(*want)
    for out in TYPES.values():
        v = moe.moe_fp8_dequantize(*got, dtype=out).double().cpu().numpy()
        # the product in float32, then the type; float16 ends at 2^-24
        tol = (2.0 ** -24 + 1.01 * half(out)) * np.abs(values) + (2.0 ** -25 if out == torch.float16 else 2.0 ** -150)
        assert (np.abs(v - values) <= tol).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (2, 128, 128), (3, 130, 272), (1, 257, 1408), (5, 64, 64), (2, 300, 144)])
def test_blocks(dtype, M, N, K):
    moe = need_gpu()
    x = rows_of(M * N, K, TYPES[dtype], seed=N).reshape(M, N, K)
    got = moe.moe_fp8_quantize(x.to(DEV), block_rows=128)
    want = fp8.quantize(x.float().numpy(), 128)
    same(got, want)
    values = fp8.dequantize(*want, 128)
    v = moe.moe_fp8_dequantize(*got, dtype=torch.float32, block_rows=128).double().cpu().numpy()
    assert (np.abs(v - values) <= 2.0 ** -24 * np.abs(values) + 2.0 ** -150).all()


@pytest.mark.parametrize("block_rows", [1, 128])
def test_blocks_of_zeros_small_large_and_nonfinite_values(block_rows):
    moe = need_gpu()
    x = torch.zeros(3, 1024)
    x[0, 128], x[0, 256], x[0, 300], x[0, 390] = 1e-40, float("inf"), 1.0, float("nan")
    x[1, 512:640] = torch.linspace(-3.4e38, 3.4e38, 128)
    x[2, 640:768] = 2.0 ** -120 * torch.arange(128)
    x[2, 768:896] = -0.0
    x[0, 900] = float("-inf")
    same(moe.moe_fp8_quantize(x.to(DEV), block_rows=block_rows), fp8.quantize(x.numpy(), block_rows))
    codes, scales = moe.moe_fp8_quantize(x.to(DEV), block_rows=block_rows)
    v = moe.moe_fp8_dequantize(codes, scales, block_rows=block_rows)[0]
    assert torch.isnan(v[256:512]).all() and torch.isnan(v[896:]).all() and not torch.isnan(v[:256]).any()


def test_every_code_comes_back():
    moe = need_gpu()
    codes = torch.arange(256, dtype=torch.uint8).reshape(2, 128)
    scales = torch.tensor([[1.0], [2.0 ** -3]])
    v = moe.moe_fp8_dequantize(codes.to(DEV).view(F8), scales.to(DEV), dtype=torch.float32).cpu().numpy()
    np.testing.assert_array_equal(v, fp8.dequantize(codes.numpy(), scales.numpy()))


def test_ties_round_to_even():
    moe = need_gpu()
    grid = fp8.GRID
    x = np.zeros((1, 256), np.float32)
    x[0, :126] = (grid[:-1] + grid[1:]) / 2          # with 448 in the block the scale is 1
    x[0, 126], x[0, 128:254], x[0, 254] = 448, -(grid[:-1] + grid[1:]) / 2, -448
    same(moe.moe_fp8_quantize(torch.from_numpy(x).to(DEV)), fp8.quantize(x))


def test_empty():
    moe = need_gpu()
    for shape in ((0, 128), (4, 0), (0, 0)):
        codes, scales = moe.moe_fp8_quantize(torch.zeros(shape, device=DEV))
        assert codes.shape == shape and scales.shape == (shape[0], fp8.pieces(shape[1]))
        assert moe.moe_fp8_dequantize(codes, scales).shape == shape
    codes, scales = moe.moe_fp8_quantize(torch.zeros(0, 256, 128, device=DEV), block_rows=128)
    assert scales.shape == (0, 2, 1)


# ---- norm --------------------------------------------------------------------------------------

# relative error of a float32 norm: the sum of squares (positive terms) of at most 64 additions in a thread (32 at most
# in the widest rows here) and 13 between threads is off by 78 steps of 2^-24, its root's inverse by half of that, and
# root, division and two products add 5
NORM = 2.0 ** -18


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H", [(1, 16), (5, 128), (1, 4096), (9, 144), (33, 272), (70, 512), (11, 1040), (257, 2048), (3, 2064),
                                 (4, 4112), (2, 8192), (3, 8208)])
@pytest.mark.parametrize("residual", [True, False])
def test_norm(dtype, T, H, residual):
    moe = need_gpu()
    dt = TYPES[dtype]
    x, r, w = rows_of(T, H, dt, 1), rows_of(T, H, dt, 2), rows_of(1, H, dt, 3, 0.0)[0]
    got = moe.moe_rms_norm_fp8(x.to(DEV), w.to(DEV), residual=r.to(DEV) if residual else None, eps=1e-5, want_normed=True)
    codes, scales, total, normed = got
    h = x
    if residual:
        h = (x.float() + r.float()).to(dt)
        assert torch.equal(total.cpu(), h)
    else:
        assert total is None
    n = fp8.rms_norm(h.double().numpy(), w.double().numpy(), 1e-5)
    _, want_scales = fp8.quantize(n.astype(np.float32))
    s = scales.double().cpu().numpy()
    assert (np.abs(s - want_scales) <= (NORM + 2.0 ** -23) * want_scales).all()
    v = fp8.dequantize(bits(codes), scales.cpu().numpy())
    step = np.maximum(np.abs(n) / 16, np.repeat(s, 128, 1)[:, :H] * 2.0 ** -10)      # half a step of the 8-bit grid
    assert (np.abs(v - n) <= step * (1 + 2.0 ** -10) + NORM * np.abs(n)).all()
    tol = (half(dt) * 1.01 + NORM) * np.abs(n) + (2.0 ** -25 if dt == torch.float16 else 0)
    assert (np.abs(normed.double().cpu().numpy() - n) <= tol).all()
    # what is not wanted is not needed
    again = moe.moe_rms_norm_fp8(x.to(DEV), w.to(DEV), residual=r.to(DEV) if residual else None, eps=1e-5)
    assert torch.equal(bits_t(again[0]), bits_t(codes)) and torch.equal(again[1], scales) and again[3] is None


def bits_t(t):
    return t.view(torch.uint8)


@pytest.mark.parametrize("H", [256, 2048, 8208, 20000])
def test_norm_in_place(H):
    moe = need_gpu()
    x, r, w = (t.to(DEV) for t in (rows_of(6, H, torch.bfloat16, 1), rows_of(6, H, torch.bfloat16, 2), rows_of(1, H, torch.bfloat16, 3)[0]))
    want = moe.moe_rms_norm_fp8(x, w, residual=r, want_normed=True)
    r2, x2 = r.clone(), x.clone()
    got = moe.moe_rms_norm_fp8(x2, w, residual=r2, residual_out=r2, normed=x2)
    assert got[2] is r2 and torch.equal(r2, want[2]) and got[3] is x2 and torch.equal(x2, want[3])
    assert torch.equal(bits_t(got[0]), bits_t(want[0])) and torch.equal(got[1], want[1])
    x3 = x.clone()
    got = moe.moe_rms_norm_fp8(x3, w, residual=r, residual_out=x3)
    assert torch.equal(x3, want[2]) and torch.equal(bits_t(got[0]), bits_t(want[0]))


def test_norm_of_zeros_and_nonfinite_rows():
    moe = need_gpu()
    x = torch.ones(4, 256)
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, 200] = float("inf")
    w = torch.ones(256)
    codes, scales, _, normed = moe.moe_rms_norm_fp8(x.to(DEV), w.to(DEV), want_normed=True)
    codes, scales, normed = bits(codes), scales.cpu().numpy(), normed.cpu().numpy()
    assert not codes[0].any() and (scales[0] == np.float32(2.0 ** -126)).all() and not normed[0].any()
    assert np.isnan(scales[1]).all() and not codes[1].any()
    # the infinity makes its row's root infinite: 0 elsewhere, NaN at its own place
    assert scales[2, 0] == np.float32(2.0 ** -126) and np.isnan(scales[2, 1]) and np.isnan(normed[2, 200]) and not normed[2, :200].any()
    assert (codes[3] == 0x7E).all()


def test_norm_without_rows():
    moe = need_gpu()
    w = torch.ones(128, device=DEV)
    codes, scales, total, _ = moe.moe_rms_norm_fp8(torch.zeros(0, 128, device=DEV), w, residual=torch.zeros(0, 128, device=DEV))
    assert codes.shape == (0, 128) and scales.shape == (0, 1) and total.shape == (0, 128)


# ---- rows into expert order ------------------------------------------------------------------------

@pytest.mark.parametrize("T,k,H,dropped", [(1, 1, 16, 0), (5, 2, 144, 3), (40, 8, 2048, 0), (300, 4, 400, 77), (1000, 2, 4096, 0), (64, 8, 16, 511)])
def test_gather(T, k, H, dropped):
    moe = need_gpu()
    rng = np.random.default_rng(T)
    S, E = T * k, 4
    ids = torch.from_numpy((rng.permutation(S) // k).astype(np.int32)).to(DEV)
    n = S - dropped
    off = torch.tensor([0, n // 3, n // 3, n // 2, n], dtype=torch.int32, device=DEV)
    codes = torch.from_numpy(rng.integers(0, 256, (T, H)).astype(np.uint8)).to(DEV).view(F8)
    scales = torch.from_numpy(rng.standard_normal((T, fp8.pieces(H))).astype(np.float32)).to(DEV)
    out = torch.full((S, H), 7, dtype=torch.uint8, device=DEV).view(F8)
    out_scales = torch.full((S, fp8.pieces(H)), 7.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    moe.moe_fp8_gather_rows(codes, scales, ids, off, out=out, out_scales=out_scales, status=status)
    assert torch.equal(bits_t(out)[:n], bits_t(codes)[ids[:n].long()]) and torch.equal(out_scales[:n], scales[ids[:n].long()])
    assert (bits_t(out)[n:] == 7).all() and (out_scales[n:] == 7).all() and int(status) == 0


def test_gather_reports_bad_tokens_and_offsets():
    moe = need_gpu()
    codes, scales = moe.moe_fp8_quantize(torch.ones(4, 256, device=DEV))
    ids = torch.tensor([0, -1, 4, 3, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, out_scales = moe.moe_fp8_gather_rows(codes, scales, ids, torch.tensor([0, 5], dtype=torch.int32, device=DEV), status=status)
    assert int(status) == moe.MOE_STATUS_BAD_INDEX
    assert (bits(out)[[1, 2, 4]] == 0).all() and (out_scales.cpu()[[1, 2, 4]] == 0).all() and (bits(out)[[0, 3]] == 0x7E).all()
    for last in (6, -1, 2 ** 31 - 1):
        status.zero_()
        moe.moe_fp8_gather_rows(codes, scales, ids.clamp(0, 3), torch.tensor([0, last], dtype=torch.int32, device=DEV), status=status)
        assert int(status) == moe.MOE_STATUS_BAD_INDEX


# ---- product -----------------------------------------------------------------------------------------

def operands(counts, K, N, seed=0, lead=0, tail=0, wide=False):
    """Quantised operands with `lead` and `tail` rows that no expert owns."""
    g = torch.Generator().manual_seed(seed)
    S = lead + sum(counts) + tail
    x = torch.randn(S, K, generator=g) * torch.exp(torch.randn(S, 1, generator=g))
    w = torch.randn(len(counts), N, K, generator=g) * K ** -0.5
    if wide:      # blocks of very different size
        x *= torch.exp2(torch.randint(-12, 12, (S, fp8.pieces(K)), generator=g).float().repeat_interleave(128, 1)[:, :K])
    off = np.concatenate([[lead], lead + np.cumsum(counts)]).astype(np.int32)
    return fp8.quantize(x.numpy()), fp8.quantize(w.numpy(), 128), off


def to_gpu(q):
    return torch.from_numpy(q[0]).to(DEV).view(F8), torch.from_numpy(q[1]).to(DEV)


def check_product(moe, x, w, off, dtype, silu, **kw):
    """Within a block products are exact and the tensor cores' additions (at most 8 that cut below 2^-23 of the block's
    sum of magnitudes) truncate; a scale's product, a block's and its addition round to 2^-24. The gate's exponential is
    off by 2 + 1.2 |z| steps of 2^-23, the division by 2, the products by 1."""
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    dt = TYPES[dtype]
    got = moe.moe_fp8_grouped_gemm(*to_gpu(x), *to_gpu(w), torch.from_numpy(off).to(DEV), activation="silu_and_mul" if silu else None,
                                   out_dtype=dt, status=status, **kw)
    assert int(status) == 0
    v, wv = fp8.dequantize(*x), fp8.dequantize(*w, 128)
    y, a = grouped.grouped_gemm(v, wv, off), grouped.grouped_gemm(np.abs(v), np.abs(wv), off)
    err = (8 * 2.0 ** -23 + (x[1].shape[1] + 3) * 2.0 ** -24) * a
    if silu:
        I = y.shape[1] // 2
        g, u = y[:, :I], y[:, I:]
        s = g / (1 + np.exp(-g))
        err = 1.1 * err[:, :I] * (np.abs(u) + err[:, I:]) + np.abs(s) * err[:, I:] + (6 + 1.2 * np.abs(g)) * 2.0 ** -23 * np.abs(s * u)
        y = s * u
    got = got.double().cpu().numpy()
    tol = err * 1.01 + half(dt) * (np.abs(y) + err) + (2.0 ** -25 if dt == torch.float16 else 2.0 ** -134)
    bad = np.abs(got - y) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], (np.abs(got - y) / np.maximum(tol, 1e-300)).max())
    return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("counts,K,N", [
    ([1], 128, 16), ([1], 16, 1), ([0, 1, 0], 2048, 176), ([2, 0, 3, 1], 144, 130), ([8] * 4, 400, 1030), ([32, 1], 272, 64),
    ([20, 0, 40, 0], 1408, 300), ([17, 64, 0, 5, 33], 640, 96), ([0, 0], 128, 128), ([63, 2, 31, 0], 256, 257)])
def test_product_of_few_rows(dtype, counts, K, N):
    moe = need_gpu()
    check_product(moe, *operands(counts, K, N, seed=K + N), dtype, False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("counts,K,N", [
    ([300], 128, 256), ([1, 0, 250], 256, 384), ([700, 3], 144, 130), ([129, 128, 127, 1], 400, 1030), ([40, 50], 16, 17),
    ([513], 1408, 640), ([256, 0, 0, 255], 2048, 258), ([97, 161], 4096, 300)])
def test_product_of_many_rows(dtype, counts, K, N):
    moe = need_gpu()
    check_product(moe, *operands(counts, K, N, seed=K + N), dtype, False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("counts,K,N", [
    ([1], 128, 32), ([3, 0, 2], 2048, 352), ([8] * 4, 400, 1056), ([64, 1], 272, 256), ([30, 5, 0], 1408, 96),
    ([300, 3], 128, 256), ([129, 128, 0, 1], 144, 416), ([513], 640, 1408), ([70, 80], 256, 32), ([200, 90], 400, 2816)])
def test_product_with_the_gate(dtype, counts, K, N):
    moe = need_gpu()
    check_product(moe, *operands(counts, K, N, seed=K + N), dtype, True)


# more tiles than SMs
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("counts,K,N", [
    ([20] * 30, 400, 1030), ([129, 0, 257, 3] * 8, 144, 1056), ([300] * 8, 144, 1090), ([10] * 200, 272, 64), ([2000, 2300], 128, 1281)])
def test_product_of_many_tiles(dtype, silu, counts, K, N):
    moe = need_gpu()
    N -= N % 32 if silu else 0          # what the gate takes
    got = check_product(moe, *operands(counts, K, N, seed=K + N, lead=3, tail=4), dtype, silu)
    assert not got[:3].any() and not got[-4:].any()


# few rows an expert on average, many of one of them
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("counts,K,N", [
    ([0] * 15 + [128], 400, 352), ([0, 130, 1, 0] + [0] * 15, 2048, 96), ([70, 2] + [1] * 20 + [33], 640, 1030),
    ([3, 0, 17, 0, 0, 0, 49, 0, 0], 144, 160), ([63] + [0] * 6 + [1], 528, 258)])
def test_product_of_uneven_groups(dtype, silu, counts, K, N):
    moe = need_gpu()
    N -= N % 32 if silu else 0          # what the gate takes
    check_product(moe, *operands(counts, K, N, seed=K + N), dtype, silu)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("counts", [[5, 0, 7], [300, 0, 90]])
def test_rows_without_an_expert_are_zero(silu, counts):
    moe = need_gpu()
    x, w, off = operands(counts, 256, 160, lead=3, tail=4)
    x[0][:3], x[0][-4:], x[1][:3] = 0x7F, 0x7F, np.nan          # not looked at
    got = moe.moe_fp8_grouped_gemm(*to_gpu(x), *to_gpu(w), torch.from_numpy(off).to(DEV), activation="silu_and_mul" if silu else None)
    got = got.float().cpu().numpy()
    assert not got[:3].any() and not got[-4:].any() and np.isfinite(got).all() and got[3:-4].any(1).all()


@pytest.mark.parametrize("counts", [[5, 9], [300, 90]])
def test_blocks_of_different_size(counts):
    moe = need_gpu()
    check_product(moe, *operands(counts, 1024, 256, wide=True), "f32", False)


@pytest.mark.parametrize("counts", [[5, 9], [300, 90]])
def test_nan_scales_and_codes_reach_only_their_own_rows_and_columns(counts):
    moe = need_gpu()
    x, w, off = operands(counts, 384, 300)
    clean = moe.moe_fp8_grouped_gemm(*to_gpu(x), *to_gpu(w), torch.from_numpy(off).to(DEV)).float().cpu().numpy()
    x[1][2, 1] = np.nan
    x[0][4, 7] = 0x7F
    w[1][1, 1, 2] = np.nan
    got = moe.moe_fp8_grouped_gemm(*to_gpu(x), *to_gpu(w), torch.from_numpy(off).to(DEV)).float().cpu().numpy()
    bad = np.zeros(got.shape, bool)
    bad[[2, 4]] = True
    bad[off[1]:, 128:256] = True
    assert np.isnan(got[bad]).all() and np.array_equal(got[~bad], clean[~bad])


def test_every_k_and_n_around_a_block():
    moe = need_gpu()
    for K in (16, 112, 128, 144, 240, 256, 272):
        for N in (1, 127, 128, 129, 255, 256, 257):
            for counts in ([3, 1], [70, 65]):
                check_product(moe, *operands(counts, K, N, seed=N), "f32", False)


@pytest.mark.parametrize("counts", [[3, 2], [200, 100]])
def test_offsets_out_of_order_are_reported(counts):
    moe = need_gpu()
    x, w, off = operands(counts, 128, 64)
    S = int(off[-1])
    for bad in ([0, S + 1, S], [0, -1, S], [S, 0, 1], [5, 2, 2 ** 31 - 1], [-5, -3, -1]):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        moe.moe_fp8_grouped_gemm(*to_gpu(x), *to_gpu(w), torch.tensor(bad, dtype=torch.int32, device=DEV), status=status)
        assert int(status) == moe.MOE_STATUS_BAD_INDEX


def test_empty_products():
    moe = need_gpu()
    q = lambda *s, **k: moe.moe_fp8_quantize(torch.ones(s, device=DEV), **k)  # noqa: E731
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    assert moe.moe_fp8_grouped_gemm(*q(0, 128), *q(2, 64, 128, block_rows=128), off).shape == (0, 64)
    assert moe.moe_fp8_grouped_gemm(*q(4, 128), *q(2, 0, 128, block_rows=128), off).shape == (4, 0)
    y = moe.moe_fp8_grouped_gemm(*q(4, 0), *q(2, 64, 0, block_rows=128), off)
    assert y.shape == (4, 64) and not y.any()


def test_many_experts():
    moe = need_gpu()
    counts = [(7 * i) % 5 for i in range(1024)]
    check_product(moe, *operands(counts, 128, 48), "bf16", False)
    check_product(moe, *operands([64 if i % 16 == 0 else 32 for i in range(130)], 128, 32), "bf16", True)


@pytest.mark.parametrize("counts", [[3, 0, 6], [300, 0, 120], [20] * 60])
def test_a_call_in_a_graph_and_equal_bits(counts):
    moe = need_gpu()
    x, w, off = operands(counts, 512, 320)
    xg, wg, og = to_gpu(x), to_gpu(w), torch.from_numpy(off).to(DEV)
    want = moe.moe_fp8_grouped_gemm(*xg, *wg, og)
    xc, xs, out = torch.zeros_like(bits_t(xg[0])).view(F8), torch.zeros_like(xg[1]), torch.empty_like(want)
    offs = torch.zeros_like(og)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_fp8_grouped_gemm(xc, xs, *wg, offs, out=out)
    bits_t(xc).copy_(bits_t(xg[0]))
    xs.copy_(xg[1])
    offs.copy_(og)
    for _ in range(3):
        out.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("counts,K", [([5, 3], 4096), ([300, 90], 4096), ([20] * 40, 512)])
def test_a_wait_that_runs_out_is_reported(silu, counts, K):
    moe = need_gpu()
    x, w, off = operands(counts, K, 512)
    args = (*to_gpu(x), *to_gpu(w), torch.from_numpy(off).to(DEV))
    act = "silu_and_mul" if silu else None
    want = moe.moe_fp8_grouped_gemm(*args, activation=act)
    torch.cuda.synchronize()
    before = moe.set_wait_limit_ns(1)
    try:
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        moe.moe_fp8_grouped_gemm(*args, activation=act, status=status)
        torch.cuda.synchronize()
        assert int(status) & moe.MOE_STATUS_TIMEOUT
    finally:
        moe.set_wait_limit_ns(before)
    assert torch.equal(moe.moe_fp8_grouped_gemm(*args, activation=act), want)


def test_rows_past_2_to_the_31():
    """Codes, values, sorted rows and operands of more than 2^31 elements: the last rows as those of small calls."""
    moe = need_gpu()
    K, T = 2048, (1 << 20) + 5
    g = torch.Generator(device=DEV).manual_seed(0)
    x = torch.empty(T, K, dtype=torch.bfloat16, device=DEV)
    x[-300:] = torch.randn(300, K, generator=g, device=DEV)
    codes, scales = moe.moe_fp8_quantize(x)
    few = moe.moe_fp8_quantize(x[-300:].contiguous())
    assert torch.equal(bits_t(codes[-300:]), bits_t(few[0])) and torch.equal(scales[-300:], few[1])
    values = moe.moe_fp8_dequantize(codes, scales, out=x)
    assert torch.equal(values[-300:], moe.moe_fp8_dequantize(*few))
    w = moe.moe_fp8_quantize(torch.randn(2, 32, K, generator=g, device=DEV), block_rows=128)
    for split in (T - 3, T - 290):          # the last expert has 3 rows or 290
        off = torch.tensor([0, split, T], dtype=torch.int32, device=DEV)
        y = moe.moe_fp8_grouped_gemm(codes, scales, *w, off)
        n = T - split
        # the same kernel on the last rows alone: a first expert with enough rows
        head = 300 - n if n > 200 else 297
        small = torch.tensor([0, head, head + n], dtype=torch.int32, device=DEV)
        last = (codes[T - head - n:].contiguous(), scales[T - head - n:].contiguous())
        assert torch.equal(y[-n:], moe.moe_fp8_grouped_gemm(*last, *w, small)[-n:])
    ids = torch.arange(T, dtype=torch.int32, device=DEV).flip(0).contiguous()
    out, out_scales = moe.moe_fp8_gather_rows(codes, scales, ids, torch.tensor([0, T], dtype=torch.int32, device=DEV))
    assert torch.equal(bits_t(out[:300]), bits_t(codes[-300:].flip(0))) and torch.equal(out_scales[:300], scales[-300:].flip(0))
    assert torch.equal(bits_t(out[-300:]), bits_t(codes[:300].flip(0)))


def test_calls_on_two_streams_at_once():
    moe = need_gpu()
    cases = [(operands(c, 1024, 320, seed=s), act) for s, (c, act) in enumerate((([300, 0, 120], None), ([5, 3, 9], None),
                                                                              ([300, 90, 7], "silu_and_mul"), ([2, 8, 1], "silu_and_mul")))]
    args = [((*to_gpu(x), *to_gpu(w), torch.from_numpy(off).to(DEV)), act) for (x, w, off), act in cases]
    want = [moe.moe_fp8_grouped_gemm(*a, activation=act) for a, act in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    got = []
    for _ in range(5):
        for (a, act), s in zip(args, streams):
            got.append(moe.moe_fp8_grouped_gemm(*a, activation=act, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(got[i], want[i % 4]) for i in range(len(got)))

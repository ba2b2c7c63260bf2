"""The 8-bit grouped product in each of its three forms (few rows an expert; tiles of 128 rows of w where all find an SM; tiles
of 256), against products of the codes' values in float64. Shapes follow from the device's SM count and the rule by which a call
takes its form, so that each test runs the form it names."""
import pytest
import torch

from gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
F8 = torch.float8_e4m3fn
FORMS = ("few", "narrow", "wide")


def half(dtype):
    return torch.finfo(dtype).eps / 2


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def form(S, E, N, silu):
    """The form that a call of these sizes takes."""
    if S <= 8 * E:
        return "few"
    columns, width = (N // 2, 64) if silu else (N, 128)
    return "narrow" if max(min(S, E), S // 128 + E // 2) * -(-columns // width) <= sms() else "wide"


def counts_for(name):
    """Rows of the experts: some without any, some with more than one tile (few: more than 64) of them."""
    if name == "few":
        return [17, 64, 0, 5, 70] + [0] * 14 + [1]
    if name == "narrow":
        return [70, 0, 129, 3]
    return [(7 * i) % 29 for i in range(sms() + 40)] + [130, 0, 257]


def operands(counts, K, N, seed=0, lead=0, tail=0, uneven=False):
    """Codes and scales of rows and matrices, offsets; `lead` and `tail` rows that no expert owns."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    S, E, kb, nb = lead + sum(counts) + tail, len(counts), -(-K // 128), -(-N // 128)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, w = ((n(*s) * 64).clamp(-448, 448).to(F8) for s in ((S, K), (E, N, K)))
    xs, ws = torch.exp(n(S, kb)) / 64, torch.exp(n(E, nb, kb)) * K ** -0.5 / 64
    if uneven:
        xs *= torch.exp2(torch.randint(-12, 12, (S, kb), generator=g, device=DEV).float())
        ws *= torch.exp2(torch.randint(-12, 12, (E, nb, kb), generator=g, device=DEV).float())
    off = torch.tensor([lead] + [lead + sum(counts[:e + 1]) for e in range(E)], dtype=torch.int32, device=DEV)
    return x, xs, w, ws, off


def spread(scales, rows, columns, blocks):
    s = scales.double().repeat_interleave(128, -1)[..., :columns]
    return s.repeat_interleave(128, -2)[..., :rows, :] if blocks else s


def products(x, xs, w, ws, off, counts):
    """y and the sums of its terms' magnitudes, [S, N] in float64."""
    (S, K), (E, N, _), most = x.shape, w.shape, max(counts + [1])
    step = torch.arange(most, device=DEV)
    rows = (off[:-1].long()[:, None] + step).clamp(max=S - 1)
    mine = step < torch.tensor(counts, device=DEV)[:, None]
    xv, wv = x.double() * spread(xs, S, K, False), w.double() * spread(ws, N, K, True)
    y = []
    for f in (lambda t: t, torch.abs):
        out = torch.zeros(S, N, dtype=torch.float64, device=DEV)
        out[rows[mine]] = torch.bmm(f(xv)[rows], f(wv).transpose(1, 2))[mine]
        y.append(out)
    return y


def call(moe, x, xs, w, ws, off, silu, dtype=torch.bfloat16, **kw):
    return moe.moe_fp8_grouped_gemm(x, xs, w, ws, off, activation="silu_and_mul" if silu else None, out_dtype=dtype, **kw)


def check(moe, ops, counts, dtype, silu, expected):
    """Within a block products are exact and the tensor cores' additions (at most 8 that cut below 2^-23 of the block's sum of
    magnitudes) truncate; a scale's product, a block's and its addition round to 2^-24. The gate's exponential is off by
    2 + 1.2 |z| steps of 2^-23, the division by 2, the products by 1."""
    x, xs, w, ws, off = ops
    assert form(x.shape[0], w.shape[0], w.shape[1], silu) == expected
    dt = TYPES[dtype]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = call(moe, *ops, silu, dt, status=status)
    assert int(status) == 0 and got.dtype is dt
    y, mag = products(*ops, counts)
    err = (8 * 2.0 ** -23 + (xs.shape[1] + 3) * 2.0 ** -24) * mag
    if silu:
        I = y.shape[1] // 2
        g, u = y[:, :I], y[:, I:]
        s = g * torch.sigmoid(g)
        err = 1.1 * err[:, :I] * (u.abs() + err[:, I:]) + s.abs() * err[:, I:] + (6 + 1.2 * g.abs()) * 2.0 ** -23 * (s * u).abs()
        y = s * u
    tol = err * 1.01 + half(dt) * (y.abs() + err) + (2.0 ** -25 if dt == torch.float16 else 2.0 ** -134)
    bad = (got.double() - y).abs() > tol
    if dt == torch.float16:
        # its largest value is 65504 and the next step would be 65536: what is 65520 (half-way, to even) or more rounds to
        # infinity. So a result whose exact value is surely there has to be infinite, and one that may be there may be.
        infinite = torch.isinf(got) & (got.double() * y > 0)
        bad = torch.where(y.abs() - err >= 65520, ~infinite, bad & ~(infinite & (y.abs() + err >= 65520)))
    assert not bad.any(), (torch.nonzero(bad)[:5], ((got.double() - y).abs() / tol).max())
    return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("K", [1408, 2048, 4096])
def test_long_reductions_and_three_tiles_a_cta(dtype, silu, K):
    moe = need_gpu()
    counts = [700, 0, 1290, 65]
    mtiles = sum(-(-c // 128) for c in counts)
    tiles = -(-3 * sms() // mtiles)              # of columns
    N = 2 * (128 * tiles - 48) if silu else 256 * tiles - 37
    assert mtiles * tiles >= 3 * sms()
    check(moe, operands(counts, K, N, seed=K), counts, dtype, silu, "wide")


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("name", FORMS)
def test_every_k_and_n_around_a_block(name, silu):
    moe = need_gpu()
    counts = counts_for(name)
    for K in (16, 112, 128, 144, 240, 256, 272):
        for N in (32, 64, 96, 224, 256, 288, 512, 544) if silu else (1, 2, 127, 128, 129, 136, 255, 256, 257):
            check(moe, operands(counts, K, N, seed=K + N), counts, "f32", silu, name)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("name", FORMS)
def test_types_and_odd_sizes(name, silu, dtype):
    moe = need_gpu()
    counts = counts_for(name)
    for K, N in ((1408, 352), (400, 1056)) if silu else ((1408, 300), (400, 1030), (528, 257)):
        check(moe, operands(counts, K, N, seed=K + N), counts, dtype, silu, name)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("name", FORMS)
def test_blocks_of_different_size(name, silu):
    moe = need_gpu()
    counts = counts_for(name)
    ops = operands(counts, 1024, 256, uneven=True)
    if silu:                # the gate's exponential within its range
        ops[3].mul_(2.0 ** -12)
    check(moe, ops, counts, "f32", silu, name)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("name", FORMS)
def test_rows_without_an_expert_are_zero_and_not_looked_at(name, silu, dtype):
    moe = need_gpu()
    counts = counts_for(name)
    N = 288 if silu else 257
    ops = operands(counts, 400, N, lead=1, tail=2)
    clean = call(moe, *ops, silu, TYPES[dtype])
    for rows in (slice(0, 1), slice(-2, None)):
        ops[0].view(torch.uint8)[rows] = 0x7F
        ops[1][rows] = float("nan")
    assert form(ops[0].shape[0], len(counts), N, silu) == name
    got = call(moe, *ops, silu, TYPES[dtype], out=torch.full_like(clean, 7.0))
    assert torch.equal(got, clean) and not got[:1].any() and not got[-2:].any() and got[1:-2].any(1).all()


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("name", FORMS)
def test_nan_reaches_only_its_own_rows_and_columns(name, silu):
    moe = need_gpu()
    counts = counts_for(name)
    N = 608 if silu else 300
    x, xs, w, ws, off = operands(counts, 384, N)
    assert form(x.shape[0], len(counts), N, silu) == name
    clean = call(moe, x, xs, w, ws, off, silu)
    S, e = x.shape[0], max(range(len(counts)), key=lambda i: counts[i])      # an expert of several tiles
    lo, hi = int(off[e]), int(off[e + 1])
    xs[2, 1] = float("nan")
    x.view(torch.uint8)[S - 1, 383] = 0x7F
    ws[e, 1, 2] = float("nan")                      # rows 128 .. 255 of w
    w.view(torch.uint8)[e, N - 1, 5] = 0x7F         # the last one
    bad = torch.zeros(S, N, dtype=torch.bool, device=DEV)
    bad[[2, S - 1]] = True
    bad[lo:hi, 128:256] = True
    bad[lo:hi, N - 1] = True
    if silu:
        bad = bad[:, :N // 2] | bad[:, N // 2:]
    got = call(moe, x, xs, w, ws, off, silu)
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], clean[~bad])


@pytest.mark.parametrize("silu", [False, True])
def test_the_forms_at_once_and_in_a_graph(silu):
    """Each form on a stream of its own, all at the same time, and captured; equal bits every time."""
    moe = need_gpu()
    N = 608 if silu else 300
    ops = [operands(counts_for(name), 1024, N, seed=i) for i, name in enumerate(FORMS)]
    want = [call(moe, *o, silu) for o in ops]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ops]
    got = [call(moe, *o, silu, stream=s) for _ in range(5) for o, s in zip(ops, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 3]) for i, g in enumerate(got))
    outs = [torch.empty_like(w) for w in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for o, out in zip(ops, outs):
            call(moe, *o, silu, out=out)
    for _ in range(3):
        for out in outs:
            out.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("counts,K,N", [([20, 0, 40, 0, 0, 0, 0, 0], 1408, 300), ([17, 64, 0, 5, 33] + [0] * 10, 640, 96),
                                        ([63, 2, 31] + [0] * 9, 256, 257), ([32, 1, 0, 0, 0], 272, 64), ([8] * 9, 4096, 130)])
def test_few_rows_on_average(dtype, counts, K, N):
    moe = need_gpu()
    check(moe, operands(counts, K, N, seed=K), counts, dtype, False, "few")
    check(moe, operands(counts, K, N // 32 * 32, seed=N), counts, dtype, True, "few")

"""Rows into expert order and back with their weights, and both gradients, on the GPU against the oracle, in three types and
rows of any width."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, need_gpu
from oracle import sorted_rows

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def half(dtype):
    return torch.finfo(dtype).eps / 2


def least(dtype):
    """Half a step of the type's smallest values."""
    return {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}[dtype]


def routing(T, k, dropped, seed=0):
    """reverse [T k] in expert order (ascending slots within an expert), offsets of max(4, k) experts, routed rows."""
    rng = np.random.default_rng(seed)
    E = max(4, k)
    expert = rng.integers(0, E, T * k)
    expert[rng.permutation(T * k)[:dropped]] = E
    reverse = np.argsort(expert, kind="stable").astype(np.int32)
    off = np.concatenate([[0], np.cumsum(np.bincount(expert, minlength=E + 1)[:E])]).astype(np.int32)
    return reverse, off, int(off[-1])


def tensors(T, k, H, dt, seed=1):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return n(T, H).to(dt), n(T * k, H).to(dt), n(T * k, H).to(dt), torch.softmax(n(T, k), 1)


def f64(t):
    return t.double().cpu().numpy()


SIZES = [(1, 1, 8, 0), (1, 4, 1, 1), (3, 2, 64, 0), (77, 2, 1001, 9), (40, 4, 2048, 0), (300, 3, 136, 100), (9, 4, 4096, 0),
         (1100, 2, 24, 5), (600, 4, 33, 0), (2000, 4, 16, 7999), (513, 4, 8200, 3), (5, 4, 20000, 2), (700, 3, 7, 11),
         (2500, 4, 24, 5), (2500, 4, 33, 9999), (9000, 1, 40, 100), (2100, 1, 72, 0),
         (50, 5, 264, 3), (700, 8, 1032, 60), (1300, 8, 257, 0), (40, 11, 520, 7), (9, 32, 72, 0), (300, 32, 35, 900)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,H,dropped", SIZES)
def test_gradients(dtype, T, k, H, dropped):
    moe = need_gpu()
    dt = TYPES[dtype]
    reverse, off, n = routing(T, k, dropped, T)
    d_out, y, d_x, w = tensors(T, k, H, dt)
    y[n:] = float("nan")                      # rows behind the last expert's are not looked at
    d_x[n:] = float("nan")
    rg, og = torch.from_numpy(reverse).to(DEV), torch.from_numpy(off).to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    d_y = torch.full((T * k, H), 7.0, dtype=dt, device=DEV)
    got_y, got_w = moe.moe_ep_combine_backward(d_out.to(DEV), y.to(DEV), w.to(DEV), rg, og, d_y=d_y, status=status)
    got_h = moe.moe_gather_rows_backward(d_x.to(DEV), rg, og, k, status=status)
    assert int(status) == 0 and got_y is d_y and (d_y[n:] == 7).all()
    want_y, want_w = sorted_rows.combine_backward(d_out.double().numpy(), y.double().numpy(), w.double().numpy(), reverse, n)
    # a product in float32, then the type
    assert (np.abs(f64(got_y[:n]) - want_y) <= (2.0 ** -24 + 1.01 * half(dt)) * np.abs(want_y) + least(dt)).all()
    mag = sorted_rows.combine_backward(np.abs(d_out.double().numpy()), np.abs(y.double().numpy()), w.double().numpy(), reverse, n)[1]
    # every thread adds at most ceil(H / 32) values one after the other, then 13 sums of threads
    assert (np.abs(f64(got_w) - want_w) <= (-(-H // 32) + 14) * 2.0 ** -24 * mag + 2.0 ** -140).all()
    want_h = sorted_rows.gather_backward(d_x.double().numpy(), reverse, n, T, k)
    mag = sorted_rows.gather_backward(np.abs(d_x.double().numpy()), reverse, n, T, k)
    assert (np.abs(f64(got_h) - want_h) <= k * 2.0 ** -24 * mag + 1.01 * half(dt) * (np.abs(want_h) + k * 2.0 ** -24 * mag) + least(dt)).all()
    # either alone, with the same bits; and again
    only_y = moe.moe_ep_combine_backward(d_out.to(DEV), None, w.to(DEV), rg, og, d_y=torch.full_like(d_y, 7.0), want_d_weights=False)
    only_w = moe.moe_ep_combine_backward(d_out.to(DEV), y.to(DEV), w.to(DEV), rg, og, want_d_y=False)
    assert only_y[1] is None and only_w[0] is None and torch.equal(only_y[0], got_y) and torch.equal(only_w[1], got_w)
    assert torch.equal(moe.moe_gather_rows_backward(d_x.to(DEV), rg, og, k), got_h)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,H,dropped", SIZES)
def test_forward(dtype, T, k, H, dropped):
    moe = need_gpu()
    dt = TYPES[dtype]
    reverse, off, n = routing(T, k, dropped, T)
    hidden, y, _, w = tensors(T, k, H, dt)
    y[n:] = float("nan")
    rg, og = torch.from_numpy(reverse).to(DEV), torch.from_numpy(off).to(DEV)
    out = torch.full((T * k, H), 7.0, dtype=dt, device=DEV)
    moe.moe_gather_rows(hidden.to(DEV), rg // k, og, k, out=out)
    assert torch.equal(out[:n].cpu(), hidden[torch.from_numpy(reverse[:n]).long() // k]) and (out[n:] == 7).all()
    got = f64(moe.moe_ep_combine(y.to(DEV), w.to(DEV), rg, og))
    want = sorted_rows.combine(y.double().numpy(), w.double().numpy(), reverse, n)
    mag = sorted_rows.combine(np.abs(y.double().numpy()), w.double().numpy(), reverse, n)
    assert (np.abs(got - want) <= 2 * k * 2.0 ** -24 * mag + 1.01 * half(dt) * (np.abs(want) + mag * k * 2.0 ** -23) + least(dt)).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,H", [(5, 1, 1), (9, 3, 3), (40, 2, 7), (40, 4, 9), (3, 2, 1001), (300, 3, 130), (1500, 4, 31), (2100, 1, 4098), (7, 4, 2044)])
def test_rows_of_any_width_keep_to_themselves(dtype, T, k, H):
    """NaN in one row stays in what that row has a part in, wherever the rows lie against 16 bytes."""
    moe = need_gpu()
    dt = TYPES[dtype]
    reverse, off, n = routing(T, k, 0, T)
    d_out, y, d_x, w = (t.to(DEV) for t in tensors(T, k, H, dt))
    rg, og = torch.from_numpy(reverse).to(DEV), torch.from_numpy(off).to(DEV)
    pos = torch.empty(T * k, dtype=torch.long, device=DEV)
    pos[rg.long()] = torch.arange(T * k, device=DEV)
    run = lambda: (*moe.moe_ep_combine_backward(d_out, y, w, rg, og), moe.moe_gather_rows_backward(d_x, rg, og, k),  # noqa: E731
                   moe.moe_ep_combine(y, w, rg, og), moe.moe_gather_rows(d_out, rg // k, og, k))
    clean = run()
    for row in sorted({0, 1, n // 2, n - 2, n - 1} & set(range(n))):
        kept = y[row].clone(), d_x[row].clone()
        y[row], d_x[row] = float("nan"), float("inf")
        d_y, d_w, d_h, out, rows = run()
        slot = int(reverse[row])
        t = slot // k
        others = torch.arange(T, device=DEV) != t
        assert torch.equal(d_y, clean[0]) and torch.equal(rows, clean[4])
        assert torch.isnan(d_w.view(-1)[slot]) and int(torch.isnan(d_w).sum()) == 1
        assert torch.equal(d_w.view(-1)[torch.arange(T * k, device=DEV) != slot], clean[1].view(-1)[torch.arange(T * k, device=DEV) != slot])
        assert not torch.isfinite(d_h[t]).any() and torch.equal(d_h[others], clean[2][others])
        assert torch.isnan(out[t]).all() and torch.equal(out[others], clean[3][others])
        y[row], d_x[row] = kept
    for t in sorted({0, T // 2, T - 1}):
        kept = d_out[t].clone()
        d_out[t] = float("nan")
        d_y, d_w, d_h, out, rows = run()
        mine = pos[t * k:(t + 1) * k]
        others = torch.ones(T * k, dtype=torch.bool, device=DEV)
        others[mine] = False
        for got, was in ((d_y, clean[0]), (rows, clean[4])):
            assert torch.isnan(got[mine]).all() and torch.equal(got[others], was[others])
        assert int(torch.isnan(d_w).sum()) == k and torch.isnan(d_w[t]).all()
        assert torch.equal(d_h, clean[2]) and torch.equal(out, clean[3])
        d_out[t] = kept


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_are_the_transposes(dtype):
    """<combine(y), d> = <y, d_y> = <w, d_w> and <gather(x), d_x> = <x, d_hidden>, as the calls give them."""
    moe = need_gpu()
    dt = TYPES[dtype]
    T, k, H = 700, 4, 264
    reverse, off, n = routing(T, k, 30)
    x, y, d_x, w = (t.to(DEV) for t in tensors(T, k, H, dt))
    d = torch.randn(T, H, device=DEV).to(dt)
    rg, og = torch.from_numpy(reverse).to(DEV), torch.from_numpy(off).to(DEV)
    d_y, d_w = moe.moe_ep_combine_backward(d, y, w, rg, og)
    a = (moe.moe_ep_combine(y, w, rg, og).double() * d.double()).sum()
    xs = moe.moe_gather_rows(x, rg // k, og, k)
    b = (xs[:n].double() * d_x[:n].double()).sum()
    # sums of roundings of independent sign: the 2-norms of the terms times half a step
    norm = lambda p, q: float((p.double() * q.double()).norm()) * (8 * half(dt))  # noqa: E731
    assert abs(a - (y[:n].double() * d_y[:n].double()).sum()) <= norm(y[:n], d_y[:n]) + 1e-3
    assert abs(a - (w.double() * d_w.double()).sum()) <= norm(y[:n], d_y[:n]) + 1e-3
    assert abs(b - (x.double() * moe.moe_gather_rows_backward(d_x, rg, og, k).double()).sum()) <= norm(xs[:n], d_x[:n]) + 1e-3


def test_no_tokens_and_no_routed_rows():
    moe = need_gpu()
    off = torch.zeros(5, dtype=torch.int32, device=DEV)
    e = lambda *s, **k: torch.empty(*s, device=DEV, **k)  # noqa: E731
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    assert moe.moe_gather_rows_backward(e(0, 64), none, off, 2).shape == (0, 64)
    d_y, d_w = moe.moe_ep_combine_backward(e(0, 64), e(0, 64), e(0, 2), none, off)
    assert d_y.shape == (0, 64) and d_w.shape == (0, 2)
    for T in (3, 2000):
        rev = torch.arange(T * 2, dtype=torch.int32, device=DEV)
        nan = torch.full((T * 2, 64), float("nan"), device=DEV)
        d_y = nan.clone()
        _, d_w = moe.moe_ep_combine_backward(torch.ones(T, 64, device=DEV), nan, torch.ones(T, 2, device=DEV), rev, off, d_y=d_y)
        assert not d_w.any() and torch.isnan(d_y).all()
        assert not moe.moe_gather_rows_backward(nan, rev, off, 2).any()


@pytest.mark.parametrize("T", [5, 3000])
def test_bad_routing_is_reported_and_stays_in_bounds(T):
    """Entries that the kernels' own checks leave out: no row is read or written for them."""
    moe = need_gpu()
    k, H = 2, 64
    rev = torch.arange(T * k, dtype=torch.int32, device=DEV)
    off = torch.tensor([0, 0, 0, 0, T * k], dtype=torch.int32, device=DEV)
    w, d, y = torch.ones(T, k, device=DEV), torch.ones(T, H, device=DEV), torch.ones(T * k, H, device=DEV)
    for place, value in ((1, -1), (2, T * k), (3, 2 ** 31 - 1), (0, -2 ** 31)):
        r = rev.clone()
        r[place] = value
        for call in (lambda s: moe.moe_gather_rows_backward(y, r, off, k, status=s),
                     lambda s: moe.moe_ep_combine_backward(d, y, w, r, off, status=s)):
            status = torch.zeros(1, dtype=torch.int32, device=DEV)
            call(status)
            assert int(status) == moe.MOE_STATUS_BAD_INDEX
    for last in (T * k + 1, -1, 2 ** 31 - 1):
        o = off.clone()
        o[-1] = last
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        moe.moe_ep_combine_backward(d, y, w, rev, o, status=status)
        assert int(status) == moe.MOE_STATUS_BAD_INDEX


@pytest.mark.parametrize("T", [40, 1500, 2600])
def test_in_a_graph(T):
    moe = need_gpu()
    k, H = 4, 256
    reverse, off, n = routing(T, k, 17)
    d_out, y, d_x, w = (t.to(DEV) for t in tensors(T, k, H, torch.bfloat16))
    rg, og = torch.from_numpy(reverse).to(DEV), torch.from_numpy(off).to(DEV)
    start = torch.zeros(T * k, H, dtype=torch.bfloat16, device=DEV)
    want = (*moe.moe_ep_combine_backward(d_out, y, w, rg, og, d_y=start.clone()), moe.moe_gather_rows_backward(d_x, rg, og, k))
    r2, o2, d_y, d_w, d_h = torch.zeros_like(rg), torch.zeros_like(og), start.clone(), torch.empty_like(w), torch.empty_like(d_out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_ep_combine_backward(d_out, y, w, r2, o2, d_y=d_y, d_weights=d_w)
        moe.moe_gather_rows_backward(d_x, r2, o2, k, d_hidden=d_h)
    r2.copy_(rg)
    o2.copy_(og)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((d_y, d_w, d_h), want))


def test_a_workspace_that_holds_other_positions():
    """What an earlier call left in the workspace names no rows."""
    moe = need_gpu()
    T, k, H = 2600, 4, 64
    ws = torch.zeros(moe.moe_gather_rows_backward_workspace_size(T, k), dtype=torch.uint8, device=DEV)
    for seed, dropped in ((0, 0), (1, 3000), (2, 10399), (3, 0)):
        reverse, off, n = routing(T, k, dropped, seed)
        d_x = torch.randn(T * k, H, device=DEV)
        rg, og = torch.from_numpy(reverse).to(DEV), torch.from_numpy(off).to(DEV)
        got = moe.moe_gather_rows_backward(d_x, rg, og, k, workspace=ws)
        np.testing.assert_allclose(f64(got), sorted_rows.gather_backward(f64(d_x), reverse, n, T, k), rtol=0, atol=2.0 ** -18)
    ws.view(torch.int32).fill_(5)
    reverse, off, n = routing(T, k, 5000, 9)
    rg, og = torch.from_numpy(reverse).to(DEV), torch.from_numpy(off).to(DEV)
    _, d_w = moe.moe_ep_combine_backward(torch.ones(T, H, device=DEV), torch.ones(T * k, H, device=DEV), torch.ones(T, k, device=DEV), rg, og,
                                         workspace=ws)
    want = torch.zeros(T * k)
    want[torch.from_numpy(reverse[:n]).long()] = H
    assert torch.equal(d_w.cpu().reshape(-1), want)


@pytest.mark.parametrize("H", [2048, 2049])
def test_rows_past_2_to_the_31(H):
    moe = need_gpu()
    T, k = (1 << 19) + 3, 2
    S = T * k
    rev = torch.arange(S, dtype=torch.int32, device=DEV).flip(0).contiguous()
    off = torch.tensor([0, 5, S], dtype=torch.int32, device=DEV)
    y = torch.empty(S, H, dtype=torch.bfloat16, device=DEV)
    y[:200], y[-200:] = torch.randn(200, H, device=DEV), torch.randn(200, H, device=DEV)
    d_out = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    d_out[:100], d_out[-100:] = torch.randn(100, H, device=DEV), torch.randn(100, H, device=DEV)
    w = torch.rand(T, k, device=DEV)
    d_y, d_w = moe.moe_ep_combine_backward(d_out, y, w, rev, off)
    d_h = moe.moe_gather_rows_backward(y, rev, off, k)
    # slot s lies in row S - 1 - s: the last tokens in the first rows and the other way round
    for tokens, rows in ((slice(0, 100), slice(S - 200, S)), (slice(T - 100, T), slice(0, 200))):
        d, v, p = d_out[tokens].double(), y[rows].double().flip(0).reshape(100, k, H), w[tokens].double()
        got = d_y[rows].double().flip(0).reshape(100, k, H)
        want = p[:, :, None] * d[:, None]
        assert ((got - want).abs() <= (2.0 ** -24 + 1.01 * half(torch.bfloat16)) * want.abs() + least(torch.bfloat16)).all()
        mag = (d[:, None].abs() * v.abs()).sum(2)
        assert ((d_w[tokens].double() - (d[:, None] * v).sum(2)).abs() <= (H // 32 + 14) * 2.0 ** -24 * mag).all()
        total, mag = v.sum(1), v.abs().sum(1)
        assert ((d_h[tokens].double() - total).abs() <= k * 2.0 ** -24 * mag + 1.01 * half(torch.bfloat16) * mag).all()


def test_calls_on_two_streams_at_once():
    moe = need_gpu()
    cases = []
    for seed, (T, k, H) in enumerate(((40, 4, 256), (2600, 4, 256), (300, 2, 1001), (9000, 1, 64))):
        reverse, off, n = routing(T, k, 7, seed)
        d_out, y, d_x, w = (t.to(DEV) for t in tensors(T, k, H, torch.bfloat16, seed))
        cases.append((d_out, y, d_x, w, torch.from_numpy(reverse).to(DEV), torch.from_numpy(off).to(DEV), k))

    def run(d_out, y, d_x, w, rg, og, k, s):
        return (*moe.moe_ep_combine_backward(d_out, y, w, rg, og, d_y=torch.zeros_like(y) if s is None else None, stream=s),
                moe.moe_gather_rows_backward(d_x, rg, og, k, stream=s))

    want = [run(*c, None) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [run(*c, s) for _ in range(5) for c, s in zip(cases, streams)]
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        c, w = cases[i % 4], want[i % 4]
        n = int(c[5][-1])
        assert torch.equal(g[0][:n], w[0][:n]) and torch.equal(g[1], w[1]) and torch.equal(g[2], w[2])

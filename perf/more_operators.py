"""Cases of the 8-bit expert layer's operators and of the gradients of sorting rows by expert, with their plain forms.

Rows in 8 bits (e4m3) have one float32 scale for each 128 values, weights one for each block of 128 x 128:

  norm        h = x + residual, its root-mean-square norm as 8-bit rows, and the norm itself      (moe_rms_norm_fp8)
  quantise    rows or weights -> 8-bit codes and scales, and the values they stand for            (moe_fp8_quantize, moe_fp8_dequantize)
  product     y[p] = x[p] w[e]^T on such codes and scales for the rows p of expert e, as it is
              or followed by silu(first half) * second half                                       (moe_fp8_grouped_gemm)
  sort        each token's 8-bit row and scales to its k places in expert order                   (moe_fp8_gather_rows)
  gradient    of the weighted sum out[t] = sum_j w[t, j] y[pos(t, j)], d_y and d_w; and of the
              copy x[pos(t, j)] = hidden[t], d_hidden                          (moe_ep_combine_backward, moe_gather_rows_backward)
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}
BLOCK = 128
EPS = 1e-6
MOST_FLOPS = 1.6e12
MOST_F32_FLOPS = 4e10
MOST_BYTES = {"norm": 4e8, "quantise": 2.2e9, "product": 1.2e9, "sort": 3.2e8, "gradient": 1.1e9}


def listed():
    return [
        # one token's decode step: the norm in front of the experts, residual stream updated, normed row for the router
        dict(name="norm token bf16", op="norm", dtype="bf16", T=1, H=4096, residual=True, normed=True),
        # the same for a 16384-token prompt
        dict(name="norm prompt bf16", op="norm", dtype="bf16", T=16384, H=2048, residual=True, normed=True),
        # activations of a decode batch between the two projections
        dict(name="quantise batch f16", op="quantise", dtype="f16", T=512, K=1408, E=1, blocks=False),
        # the master weights of an expert layer, converted once for serving
        dict(name="quantise weights f32", op="quantise", dtype="f32", T=2048, K=1408, E=64, blocks=True),
        # one token's decode step through the first projection of a 64-expert layer, with the gate
        dict(name="product decode bf16", op="product", dtype="bf16", T=1, k=8, E=64, K=2048, N=2816, skew=0.0, empty=0, silu=True),
        # a decode batch of 64 tokens through its second projection
        dict(name="product batch f16", op="product", dtype="f16", T=64, k=8, E=64, K=1408, N=2048, skew=0.3, empty=0, silu=False),
        # a small layer with odd sizes, float32 results, an expert without rows
        dict(name="product odd f32", op="product", dtype="f32", T=1000, k=2, E=8, K=528, N=1030, skew=0.3, empty=1, silu=False),
        # a 16384-token prompt with the gate
        dict(name="product prompt bf16", op="product", dtype="bf16", T=16384, k=8, E=64, K=2048, N=2816, skew=0.3, empty=0, silu=True),
        # rows of a decode batch of a wide layer
        dict(name="sort batch", op="sort", T=64, k=2, E=8, H=4096, skew=0.3, dropped=0),
        # rows of a prompt
        dict(name="sort prompt", op="sort", T=16384, k=8, E=64, H=2048, skew=0.3, dropped=0),
        # a small training step with an odd width, some slots without an expert
        dict(name="gradient odd f16", op="gradient", dtype="f16", T=777, k=2, E=16, H=1001, skew=0.5, dropped=9),
        # a training step of a 64-expert layer
        dict(name="gradient step bf16", op="gradient", dtype="bf16", T=8192, k=8, E=64, H=2048, skew=0.3, dropped=0),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "quantise", "product", "product", "product", "sort", "gradient", "gradient"])
    c = dict(op=op)
    if op != "sort":
        c["dtype"] = rng.choice(["bf16", "f16", "bf16", "f32"])
    if op == "norm":
        c |= dict(T=spread(1, 16384), H=16 * spread(2, 512), residual=rng.random() < 0.7, normed=rng.random() < 0.6)
    elif op == "quantise":
        blocks = rng.random() < 0.5
        c |= dict(T=spread(16, 4096) if blocks else spread(1, 65536), K=16 * spread(2, 512), E=spread(1, 64) if blocks else 1, blocks=blocks)
    elif op == "product":
        E = spread(4, 128)
        c |= dict(T=spread(1, 16384), k=rng.randint(1, min(8, E)), E=E, K=16 * spread(4, 256), N=16 * spread(4, 512),
                  skew=round(rng.uniform(0.0, 0.5), 2), empty=rng.randint(0, E // 8), silu=rng.random() < 0.5)
        if rng.random() < 0.5:      # whole blocks along the reduction, as most layers have
            c["K"] = max(BLOCK, c["K"] // BLOCK * BLOCK)
        if c["silu"]:
            c["N"] = max(32, c["N"] // 32 * 32)
        elif rng.random() < 0.3:    # odd sizes
            c["N"] = max(1, c["N"] - rng.randint(1, 15))
        c["k"] = min(c["k"], E - c["empty"])
        while c["E"] * c["N"] * c["K"] > 1 << 29:
            c["N"] = max(32, c["N"] // 64 * 32)
    else:
        E = spread(4, 128)
        k = rng.randint(1, min(8, E))
        c |= dict(T=spread(1, 16384), k=k, E=E, H=16 * spread(2, 512), skew=round(rng.uniform(0.0, 0.5), 2), dropped=0)
        if op == "gradient" and rng.random() < 0.3:
            c["H"] = max(1, c["H"] - rng.randint(1, 15))
    dropped = rng.random() * 0.25 if rng.random() < 0.3 else 0.0
    flops = MOST_F32_FLOPS if c.get("dtype") == "f32" else MOST_FLOPS
    while (work(c)["flops"] > flops or work(c)["bytes"] > MOST_BYTES[op]) and c["T"] > 1:
        c["T"] = (c["T"] + 1) // 2
    if "dropped" in c:
        c["dropped"] = int(dropped * c["T"] * c["k"])
    return c


def pieces(n):
    return -(-n // BLOCK)


def work(case):
    op, b = case["op"], SIZES.get(case.get("dtype"), 1)
    T = case["T"]
    if op == "norm":
        H = case["H"]
        packed = T * (H + 4 * pieces(H))
        moved = T * H * b * (1 + 2 * case["residual"] + case["normed"]) + H * b
        # the 8-bit rows are written by the norm, read by the second call, which writes their values in 16 bits
        return {"bytes": moved + 2 * packed + 2 * T * H, "flops": 0}
    if op == "quantise":
        E, K = case["E"], case["K"]
        packed = E * (T * K + 4 * pieces(K) * (pieces(T) if case["blocks"] else T))
        return {"bytes": E * T * K * b + 2 * packed + 2 * E * T * K, "flops": 0}
    k, E = case["k"], case["E"]
    S = T * k - case.get("dropped", 0)
    if op == "sort":
        row = case["H"] + 4 * pieces(case["H"])
        return {"bytes": (T + S) * row + 4 * S, "flops": 0}
    if op == "gradient":
        return {"bytes": b * case["H"] * (2 * T + 3 * S) + 12 * S, "flops": 0}
    K, N = case["K"], case["N"]
    live = E - case["empty"]
    seen = live * (1 - (1 - min(1.0, k / live)) ** T)   # experts that some token reaches, on average
    weight = seen * (N * K + 4 * pieces(N) * pieces(K))
    out = N // 2 if case["silu"] else N
    return {"bytes": S * (K + 4 * pieces(K)) + weight + b * S * out + 4 * E, "flops": 2.0 * S * N * K}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op, T, dt = case["op"], case["T"], DTYPES.get(case.get("dtype"))
    st = dict(case=dict(case))

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, device=dev, generator=gen) * scale).to(dtype)

    if op == "norm":
        H = case["H"]
        # some channels of a residual stream are much larger than the others
        channel = torch.exp(normal(H))
        st["x"] = (normal(T, H) * channel).to(dt)
        st["residual"] = (normal(T, H, scale=4.0) * channel).to(dt) if case["residual"] else None
        st["weight"] = (1.0 + 0.1 * normal(H)).to(dt)
        st["codes"] = torch.empty(T, H, dtype=torch.float8_e4m3fn, device=dev)
        st["scales"] = torch.empty(T, pieces(H), device=dev)
        st["sum"] = torch.empty(T, H, dtype=dt, device=dev) if case["residual"] else None
        st["normed"] = torch.empty(T, H, dtype=dt, device=dev) if case["normed"] else None
        st["out"] = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
        return st
    if op == "quantise":
        E, K = case["E"], case["K"]
        # rows (or rows of weights) differ in size
        st["x"] = (normal(E, T, K) * torch.exp(normal(E, T, 1))).to(dt)
        if not case["blocks"]:
            st["x"] = st["x"][0]
        st["codes"] = torch.empty(st["x"].shape, dtype=torch.float8_e4m3fn, device=dev)
        st["scales"] = torch.empty(E, pieces(T), pieces(K), device=dev) if case["blocks"] else torch.empty(T, pieces(K), device=dev)
        st["out"] = torch.empty(st["x"].shape, dtype=torch.bfloat16, device=dev)
        return st
    # routing: each token takes its k best experts of perturbed popularities
    k, E = case["k"], case["E"]
    S = T * k
    popularity = case["skew"] * normal(E)
    if case.get("empty"):
        popularity[torch.randperm(E, device=dev, generator=gen)[: case["empty"]]] = -1e4
    gumbel = -torch.log(-torch.log(torch.rand(T, E, device=dev, generator=gen).clamp(1e-7, 1 - 1e-7)))
    chosen = (popularity + gumbel).topk(k, dim=1).indices.reshape(-1)
    if case.get("dropped"):     # slots that no expert takes
        chosen[torch.randperm(S, device=dev, generator=gen)[: case["dropped"]]] = E
    order = torch.sort(chosen, stable=True).indices
    counts = torch.bincount(chosen, minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=dev)
    offsets[1:] = counts.cumsum(0).to(torch.int32)
    st["offsets"] = offsets
    st["live"] = S - case.get("dropped", 0)
    if op in ("sort", "gradient"):
        H = case["H"]
        st["reverse"] = order.to(torch.int32)
        st["tokens"] = (order // k).to(torch.int32)
        if op == "sort":
            st["rows"], st["scales"] = encode(normal(T, H) * torch.exp(normal(T, 1)), False)
            # rows behind the last expert's stay as they are
            st["x"] = torch.zeros(S, H, dtype=torch.float8_e4m3fn, device=dev)
            st["x_scales"] = torch.zeros(S, pieces(H), device=dev)
            return st
        st["d_out"], st["y"], st["d_x"] = normal(T, H, dtype=dt), normal(S, H, dtype=dt), normal(S, H, dtype=dt)
        st["weights"] = torch.softmax(normal(T, k), dim=1)
        st["d_y"] = torch.zeros(S, H, dtype=dt, device=dev)
        st["d_weights"] = torch.empty(T, k, device=dev)
        st["d_hidden"] = torch.empty(T, H, dtype=dt, device=dev)
        return st
    K, N = case["K"], case["N"]
    # what the plain form's batched products index by: the experts that have rows, padded to one length
    alive = torch.nonzero(counts).reshape(-1)
    longest = int(counts.max())
    step = torch.arange(longest, device=dev)
    st["alive"] = alive
    st["member"] = step[None, :] < counts[alive][:, None]
    st["index"] = (offsets[alive].long()[:, None] + step[None, :]).clamp(max=S - 1)
    place = torch.zeros(E, dtype=torch.int64, device=dev)
    place[alive] = torch.arange(alive.numel(), device=dev) * longest
    expert = chosen[order]
    st["slot"] = place[expert] + torch.arange(S, device=dev) - offsets[expert].long()
    st["x"], st["x_scales"] = encode(normal(S, K) * torch.exp(0.5 * normal(S, 1)), False)
    w = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device=dev)
    w_scales = torch.empty(E, pieces(N), pieces(K), device=dev)
    for e in range(E):
        w[e], w_scales[e] = encode(normal(N, K, scale=K ** -0.5), True)
    st["w"], st["w_scales"] = w, w_scales
    st["out"] = torch.empty(S, N // 2 if case["silu"] else N, dtype=dt, device=dev)
    return st


def spans(scales, shape, blocks):
    """Scales as they apply to the single values of `shape`."""
    s = scales.repeat_interleave(BLOCK, dim=-1)[..., : shape[-1]]
    return s.repeat_interleave(BLOCK, dim=-2)[..., : shape[-2], :] if blocks else s


def encode(v, blocks):
    """8-bit codes and scales of v [..., K] in 32 bits; `blocks`: a scale for 128 x 128 values, else for 1 x 128."""
    rows, K = v.shape[-2], v.shape[-1]
    a = torch.nn.functional.pad(v.abs(), (0, pieces(K) * BLOCK - K, 0, pieces(rows) * BLOCK - rows if blocks else 0))
    most = a.unflatten(-1, (-1, BLOCK)).amax(-1)
    if blocks:
        most = most.unflatten(-2, (-1, BLOCK)).amax(-2)
    scales = (most / 448.0).clamp(min=2.0 ** -126)
    return (v * spans(1.0 / scales, v.shape, blocks)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scales


def batch(rows, st):
    """rows [S, C] as [experts with rows, longest, C], zero where an expert has no such row."""
    return rows[st["index"]] * st["member"][..., None]


def run(st):
    case = st["case"]
    op, dt = case["op"], DTYPES.get(case.get("dtype"))
    if own:
        import mixture_experts_routing_token_gb300 as moe
        if op == "norm":
            codes, scales, total, normed = moe.moe_rms_norm_fp8(st["x"], st["weight"], eps=EPS, residual=st["residual"], codes=st["codes"],
                                                                scales=st["scales"], residual_out=st["sum"], normed=st["normed"],
                                                                want_normed=case["normed"])
            return moe.moe_fp8_dequantize(codes, scales, out=st["out"]), scales, total, normed
        if op == "quantise":
            rows = BLOCK if case["blocks"] else 1
            codes, scales = moe.moe_fp8_quantize(st["x"], block_rows=rows, codes=st["codes"], scales=st["scales"])
            return moe.moe_fp8_dequantize(codes, scales, block_rows=rows, out=st["out"]), scales
        if op == "product":
            return moe.moe_fp8_grouped_gemm(st["x"], st["x_scales"], st["w"], st["w_scales"], st["offsets"],
                                            activation="silu_and_mul" if case["silu"] else None, out_dtype=dt, out=st["out"])
        if op == "sort":
            return moe.moe_fp8_gather_rows(st["rows"], st["scales"], st["tokens"], st["offsets"], out=st["x"], out_scales=st["x_scales"])
        d_y, d_weights = moe.moe_ep_combine_backward(st["d_out"], st["y"], st["weights"], st["reverse"], st["offsets"],
                                                     d_y=st["d_y"], d_weights=st["d_weights"])
        return d_y, d_weights, moe.moe_gather_rows_backward(st["d_x"], st["reverse"], st["offsets"], case["k"], d_hidden=st["d_hidden"])
    if op == "norm":
        h = st["x"].float()
        total = None
        if case["residual"]:
            total = (h + st["residual"].float()).to(dt)
            h = total.float()
        n = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * st["weight"].float()
        codes, scales = encode(n, False)
        return (codes.float() * spans(scales, n.shape, False)).to(torch.bfloat16), scales, total, n.to(dt) if case["normed"] else None
    if op == "quantise":
        codes, scales = encode(st["x"].float(), case["blocks"])
        return (codes.float() * spans(scales, codes.shape, case["blocks"])).to(torch.bfloat16), scales
    if op == "product":
        w = st["w"][st["alive"]].float() * spans(st["w_scales"][st["alive"]], st["w"].shape, True)
        x = batch(st["x"].float() * spans(st["x_scales"], st["x"].shape, False), st)
        y = torch.bmm(x, w.transpose(1, 2)).reshape(-1, case["N"])[st["slot"]]
        if case["silu"]:
            gate, up = y.chunk(2, dim=1)
            y = gate / (1.0 + torch.exp(-gate)) * up
        return y.to(dt)
    T, k, live = case["T"], case["k"], st["live"]
    if op == "sort":
        token = st["tokens"][:live].long()
        x, scales = torch.zeros_like(st["x"]), torch.zeros_like(st["x_scales"])
        x[:live] = st["rows"].view(torch.uint8)[token].view(torch.float8_e4m3fn)
        scales[:live] = st["scales"][token]
        return x, scales
    slot = st["reverse"][:live].long()
    token = slot // k
    d = st["d_out"][token].float()
    d_y = torch.zeros_like(st["y"])
    d_y[:live] = (d * st["weights"].reshape(-1)[slot][:, None]).to(dt)
    d_weights = torch.zeros(T * k, device=d.device)
    d_weights[slot] = (d * st["y"][:live].float()).sum(1)
    back = torch.zeros(T * k, case["H"], device=d.device)
    back[slot] = st["d_x"][:live].float()
    return d_y, d_weights.reshape(T, k), back.reshape(T, k, -1).sum(1).to(dt)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]

    def held(v, blocks):
        """The values that 8 bits hold for v, and the scales, 128 rows or the rows themselves at a time."""
        most = torch.zeros(*v.shape[:-2], pieces(v.shape[-2]) if blocks else v.shape[-2], pieces(v.shape[-1]), dtype=torch.float64, device=v.device)
        for b in range(most.shape[-1]):
            high = v[..., b * BLOCK:(b + 1) * BLOCK].abs().max(dim=-1).values
            if blocks:
                for r in range(most.shape[-2]):
                    most[..., r, b] = high[..., r * BLOCK:(r + 1) * BLOCK].max(dim=-1).values
            else:
                most[..., b] = high
        scale = torch.maximum(most / 448, torch.full_like(most, 2.0 ** -126))
        out = torch.empty(v.shape, dtype=torch.float64, device=v.device)
        for b in range(most.shape[-1]):
            cols = slice(b * BLOCK, (b + 1) * BLOCK)
            s = scale[..., b]
            s = (s.repeat_interleave(BLOCK, dim=-1)[..., : v.shape[-2]] if blocks else s)[..., None]
            a = v[..., cols] / s
            # spacing of the 8-bit values around a: 2^(e - 3) from 2^e on, 2^-9 below 2^-6; round() takes ties to even
            _, e = torch.frexp(a)
            gap = torch.ldexp(torch.ones_like(a), (e - 1).clamp(min=-6) - 3)
            out[..., cols] = (torch.round(a / gap) * gap).clamp(-448, 448) * s
        return out, scale

    if op == "norm":
        h = st["x"].double()
        total = None
        if case["residual"]:
            total = h + st["residual"].double()
            # the norm is of the sum as the stream holds it, in its own type; added in 32 bits first
            h = (st["x"].float() + st["residual"].float()).to(st["x"].dtype).double()
        n = st["weight"].double() * h / torch.sqrt(h.square().sum(-1, keepdim=True) / case["H"] + EPS)
        values, scale = held(n, False)
        return values, scale, total, n if case["normed"] else None
    if op == "quantise":
        if not case["blocks"]:
            parts = [held(p.double(), False) for p in st["x"].split(8192)]
        else:
            parts = [held(p[None].double(), True) for p in st["x"]]
        return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
    lo = st["offsets"].tolist()
    if op == "product":
        S, E, K, N = case["T"] * case["k"], case["E"], case["K"], case["N"]
        y = torch.zeros(S, N, dtype=torch.float64, device="cuda")
        for e in range(E):
            rows = slice(lo[e], lo[e + 1])
            if lo[e + 1] == lo[e]:
                continue
            w = st["w"][e].double()
            for r in range(pieces(N)):
                for b in range(pieces(K)):
                    w[r * BLOCK:(r + 1) * BLOCK, b * BLOCK:(b + 1) * BLOCK] *= st["w_scales"][e, r, b].double()
            x = st["x"][rows].double()
            for b in range(pieces(K)):
                x[:, b * BLOCK:(b + 1) * BLOCK] *= st["x_scales"][rows, b, None].double()
            y[rows] = x @ w.t()
        if case["silu"]:
            half = N // 2
            y = y[:, :half] * torch.sigmoid(y[:, :half]) * y[:, half:]
        return y
    T, k, live = case["T"], case["k"], st["live"]
    if op == "sort":
        token = st["tokens"].long()
        x, scales = st["rows"].double().index_select(0, token), st["scales"].double().index_select(0, token)
        x[live:], scales[live:] = 0, 0
        return x, scales
    place = torch.full((T * k,), -1, dtype=torch.int64, device="cuda")
    place[st["reverse"][:live].long()] = torch.arange(live, device="cuda")
    place = place.reshape(T, k)
    d_out = st["d_out"].double()
    d_y = torch.zeros(T * k, case["H"], dtype=torch.float64, device="cuda")
    d_weights = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    d_hidden = torch.zeros(T, case["H"], dtype=torch.float64, device="cuda")
    for j in range(k):
        t = torch.nonzero(place[:, j] >= 0).reshape(-1)
        p = place[t, j]
        d_y[p] = d_out[t] * st["weights"][t, j, None].double()
        d_weights[t, j] = torch.einsum("th,th->t", d_out[t], st["y"][p].double())
        d_hidden[t] += st["d_x"][p].double()
    return d_y, d_weights, d_hidden

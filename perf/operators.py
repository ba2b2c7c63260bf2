"""Cases of the grouped products and the 4-bit microscaled operators, with their plain forms.

Operators (x [S, K] are rows sorted by expert, expert e owns rows offsets[e]..offsets[e + 1] - 1):

  product     y[p] = x[p] w[e]^T                                     (moe_grouped_gemm)
  gradient    d_x[p] = d_y[p] w[e], d_w[e] = sum_p d_y[p]^T x[p]      (moe_grouped_gemm_backward)
  quantise    blocks of 32 values -> 4-bit codes and an 8-bit power-of-two scale, and the values
              they stand for                                         (moe_mxfp4_quantize, moe_mxfp4_dequantize)
  product4    y[p] = x[p] w[e]^T on such codes and scales, as it is or followed by
              silu(first half) * second half                         (moe_mxfp4_grouped_gemm)
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}
BLOCK = 32
MOST_FLOPS = {"product": 1.6e12, "gradient": 1.9e12, "product4": 1.6e12}
MOST_F32_FLOPS = 4e9
MOST_BYTES = 1.65e9


def listed():
    return [
        # one token's decode step through the first projection of a 64-expert layer
        dict(name="product decode bf16", op="product", dtype="bf16", T=1, k=8, E=64, K=2048, N=2816, skew=0.0, empty=0),
        # a decode batch of 64 tokens through its second projection
        dict(name="product batch f16", op="product", dtype="f16", T=64, k=8, E=64, K=1408, N=2048, skew=0.3, empty=0),
        # a small float32 layer with odd sizes, as in tests and fine-tuning of a head
        dict(name="product odd f32", op="product", dtype="f32", T=1000, k=2, E=8, K=517, N=1030, skew=0.3, empty=1),
        # a 16384-token prompt
        dict(name="product prompt bf16", op="product", dtype="bf16", T=16384, k=8, E=64, K=2048, N=2816, skew=0.3, empty=0),
        # a small training step with ragged groups, an expert without rows and an odd width
        dict(name="gradient odd f16", op="gradient", dtype="f16", T=777, k=2, E=16, K=1000, N=714, skew=0.5, empty=1),
        # a training step of an 8-expert layer with wide experts
        dict(name="gradient wide bf16", op="gradient", dtype="bf16", T=4096, k=2, E=8, K=4096, N=14336, skew=0.3, empty=0),
        # the rows of a decode batch, spread to their experts
        dict(name="quantise batch bf16", op="quantise", dtype="bf16", T=8, k=8, E=64, K=2048, skew=0.0, gather=True),
        # a prompt's rows, spread to their experts
        dict(name="quantise prompt bf16", op="quantise", dtype="bf16", T=16384, k=8, E=64, K=2048, skew=0.3, gather=True),
        # the master weights of an expert layer, converted once for serving
        dict(name="quantise weights f32", op="quantise", dtype="f32", T=131072, k=1, E=1, K=1408, skew=0.0, gather=False),
        # one token's decode step on 4-bit weights
        dict(name="product4 decode bf16", op="product4", dtype="bf16", T=1, k=8, E=64, K=2048, N=2816, skew=0.0, empty=0, silu=True),
        # a 16384-token prompt on 4-bit weights, with the gate
        dict(name="product4 prompt bf16", op="product4", dtype="bf16", T=16384, k=8, E=64, K=2048, N=2816, skew=0.3, empty=0, silu=True),
        # the second projection of a 128-expert layer under an uneven load, some experts without rows
        dict(name="product4 uneven f16", op="product4", dtype="f16", T=5000, k=8, E=128, K=1536, N=4096, skew=0.5, empty=9, silu=False),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["product", "product", "gradient", "quantise", "product4", "product4"])
    if op == "quantise":
        gather = rng.random() < 0.5
        E = spread(4, 128)
        c = dict(op=op, dtype=rng.choice(["bf16", "f16", "f32"]), T=spread(1, 16384 if gather else 131072),
                 k=rng.randint(1, min(8, E)) if gather else 1, E=E if gather else 1, K=BLOCK * spread(1, 64),
                 skew=round(rng.uniform(0.0, 0.5), 2) if gather else 0.0, gather=gather)
        while work(c)["bytes"] > MOST_BYTES:
            c["T"] = max(1, c["T"] // 2)
        return c
    E = spread(4, 128)
    dtype = rng.choice(["bf16", "f16", "bf16", "f32"]) if op != "product4" else rng.choice(["bf16", "f16"])
    c = dict(op=op, dtype=dtype, T=spread(1, 16384), k=rng.randint(1, min(8, E)), E=E, K=8 * spread(8, 512), N=8 * spread(4, 1024),
             skew=round(rng.uniform(0.0, 0.5), 2), empty=rng.randint(0, E // 8))
    if op == "product4":
        c["K"] = BLOCK * spread(2, 128)
        c["silu"] = rng.random() < 0.5
    elif rng.random() < 0.3:      # odd sizes
        c["K"] = max(1, c["K"] - rng.randint(1, 7))
        c["N"] = max(1, c["N"] - rng.randint(1, 7))
    most = MOST_F32_FLOPS if dtype == "f32" else MOST_FLOPS[op]
    c["k"] = min(c["k"], E - c["empty"])
    while c["E"] * c["N"] * c["K"] > (1 << 26 if dtype == "f32" else 1 << 29):
        c["N"] = max(8, c["N"] // 16 * 8)
    while (work(c)["flops"] > most or work(c)["bytes"] > MOST_BYTES) and c["T"] > 1:
        c["T"] = (c["T"] + 1) // 2
    return c


def work(case):
    T, k, E, K, b = case["T"], case["k"], case["E"], case["K"], SIZES[case["dtype"]]
    S = T * k
    if case["op"] == "quantise":
        packed = S * K * (0.5 + 1 / BLOCK)
        # the first call reads the rows and writes codes and scales, the second reads those and writes values
        return {"bytes": T * K * b + packed + packed + S * K * b + (4 * S if case["gather"] else 0), "flops": 0}
    N, live = case["N"], E - case["empty"]
    seen = live * (1 - (1 - min(1.0, k / live)) ** T)   # experts that some token reaches, on average
    weight = seen * N * K
    if case["op"] == "product":
        return {"bytes": b * (S * K + weight + S * N) + 4 * E, "flops": 2.0 * S * N * K}
    if case["op"] == "gradient":
        return {"bytes": b * (2 * S * K + S * N + weight + E * N * K) + 4 * E, "flops": 4.0 * S * N * K}
    out = N // 2 if case["silu"] else N
    return {"bytes": (0.5 + 1 / BLOCK) * (S * K + weight) + b * S * out + 4 * E, "flops": 2.0 * S * N * K}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    T, k, E, K, dt = case["T"], case["k"], case["E"], case["K"], DTYPES[case["dtype"]]
    S = T * k

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, device=dev, generator=gen) * scale).to(dtype)

    # routing: each token takes its k best experts of perturbed popularities
    popularity = case["skew"] * torch.randn(E, device=dev, generator=gen)
    if case.get("empty"):
        popularity[torch.randperm(E, device=dev, generator=gen)[: case["empty"]]] = -1e4
    gumbel = -torch.log(-torch.log(torch.rand(T, E, device=dev, generator=gen).clamp(1e-7, 1 - 1e-7)))
    chosen = (popularity + gumbel).topk(k, dim=1).indices.reshape(-1)
    order = torch.sort(chosen, stable=True).indices
    counts = torch.bincount(chosen, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=dev)
    offsets[1:] = counts.cumsum(0).to(torch.int32)
    st = dict(case=dict(case), offsets=offsets)
    if case["op"] == "quantise":
        # rows differ in size, and blocks within a row
        st["x"] = (normal(T, K, dtype=torch.float32) * torch.exp(normal(T, 1, dtype=torch.float32))).to(dt)
        st["rows"] = (order // k).to(torch.int32) if case["gather"] else None
        st["codes"] = torch.empty(S, K // 2, dtype=torch.uint8, device=dev)
        st["scales"] = torch.empty(S, K // BLOCK, dtype=torch.uint8, device=dev)
        st["out"] = torch.empty(S, K, dtype=dt, device=dev)
        return st
    N = case["N"]
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
    x, w = normal(S, K), normal(E, N, K, scale=K ** -0.5)
    if case["op"] == "product4":
        st["x"], st["x_scales"] = pack(x)
        st["w"], st["w_scales"] = pack(w)
        st["out"] = torch.empty(S, N // 2 if case["silu"] else N, dtype=dt, device=dev)
        return st
    st["x"], st["w"] = x, w
    if case["op"] == "product":
        st["out"] = torch.empty(S, N, dtype=dt, device=dev)
    else:
        st["d_y"] = normal(S, N)
        st["d_x"], st["d_w"] = torch.empty_like(x), torch.empty_like(w)
    return st


def encode(x):
    """4-bit magnitudes-and-signs (int32, one per value) and biased scale exponents of x [..., K]."""
    v = x.float().reshape(*x.shape[:-1], x.shape[-1] // BLOCK, BLOCK)
    most = v.abs().amax(-1)
    low = torch.frexp(most).exponent - 3               # floor(log2 of the largest) - 2
    low = torch.where(most > 0, low, -127).clamp(-127, 127)
    up = ((127 - low) << 23).to(torch.int32).view(torch.float32)   # 2^-low
    a = (v * up[..., None]).abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int() + (a >= 3.5).int() + (a > 5.0).int())
    code = code + 8 * torch.signbit(v).int()
    return code.reshape(x.shape), (low + 127).to(torch.uint8)


def pack(x):
    code, scale = encode(x)
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8), scale


def values(code, scale):
    """What codes (one per value) and scales stand for, in 32 bits."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=code.device)
    v = grid[(code & 7).long()] * (1.0 - 2.0 * (code >> 3).float())
    up = torch.where(scale > 0, scale.int() << 23, 1 << 22).to(torch.int32).view(torch.float32)   # 2^(scale - 127)
    return (v.reshape(*scale.shape, BLOCK) * up[..., None]).reshape(code.shape)


def unpack(packed, scale):
    code = torch.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], 2 * packed.shape[-1])
    return values(code, scale)


def batch(rows, st):
    """rows [S, C] as [experts with rows, longest, C] in 32 bits, zero where an expert has no such row."""
    return rows[st["index"]].float() * st["member"][..., None]


def run(st):
    case = st["case"]
    op, dt = case["op"], DTYPES[case["dtype"]]
    if own:
        import mixture_experts_routing_token_gb300 as moe
        if op == "product":
            return moe.moe_grouped_gemm(st["x"], st["w"], st["offsets"], out=st["out"])
        if op == "gradient":
            return moe.moe_grouped_gemm_backward(st["x"], st["w"], st["offsets"], st["d_y"], d_x=st["d_x"], d_w=st["d_w"])
        if op == "quantise":
            codes, scales = moe.moe_mxfp4_quantize(st["x"], rows=st["rows"], codes=st["codes"], scales=st["scales"])
            return moe.moe_mxfp4_dequantize(codes, scales, dtype=dt, out=st["out"]), scales
        return moe.moe_mxfp4_grouped_gemm(st["x"], st["x_scales"], st["w"], st["w_scales"], st["offsets"],
                                          activation="silu_and_mul" if case["silu"] else None, out_dtype=dt, out=st["out"])
    if op == "quantise":
        x = st["x"] if st["rows"] is None else st["x"][st["rows"].long()]
        code, scale = encode(x)
        return values(code, scale).to(dt), scale
    if op == "product4":
        x, w = batch(unpack(st["x"], st["x_scales"]), st), unpack(st["w"][st["alive"]], st["w_scales"][st["alive"]])
        y = torch.bmm(x, w.transpose(1, 2)).reshape(-1, case["N"])[st["slot"]]
        if case["silu"]:
            gate, up = y.chunk(2, dim=1)
            y = gate / (1.0 + torch.exp(-gate)) * up
        return y.to(dt)
    x, w = batch(st["x"], st), st["w"][st["alive"]].float()
    if op == "product":
        return torch.bmm(x, w.transpose(1, 2)).reshape(-1, case["N"])[st["slot"]].to(dt)
    d_y = batch(st["d_y"], st)
    d_x = torch.bmm(d_y, w).reshape(-1, case["K"])[st["slot"]].to(dt)
    d_w = torch.zeros_like(st["w"])
    d_w[st["alive"]] = torch.bmm(d_y.transpose(1, 2), x).to(dt)
    return d_x, d_w


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantise":
        power = torch.tensor([2.0 ** (i - 512) for i in range(1024)], dtype=torch.float64, device="cuda")
        x = st["x"] if st["rows"] is None else st["x"].index_select(0, st["rows"].long())
        out, scales = [], []
        for part in x.split(8192):
            v = part.double().unflatten(1, (-1, BLOCK))
            most = v.abs().max(dim=2).values
            low = torch.floor(torch.log2(most.clamp(min=2.0 ** -500)) + 0.5)
            low = low - (power[low.long() + 512] > most).double() - 2      # the logarithm's floor, exact at powers of two
            low = torch.where(most > 0, low, -200.0).clamp(-127, 127)
            up = power[low.long() + 512][..., None]
            a = v / up
            # spacing of the grid 0, 0.5, 1, 1.5, 2, 3, 4, 6 around a; round() takes ties to even
            gap = torch.where(a.abs() < 2, 0.5, torch.where(a.abs() < 4, 1.0, 2.0)).double()
            q = (torch.round(a / gap) * gap).clamp(-6, 6)
            out.append((q * up).flatten(1))
            scales.append((low + 127).to(torch.uint8))
        return torch.cat(out), torch.cat(scales)
    lo = st["offsets"].tolist()
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
    power = torch.tensor([2.0 ** (i - 127) for i in range(256)], dtype=torch.float64, device="cuda")

    def wide(name, at):
        t = st[name][at]
        if op != "product4":
            return t.double()
        nibbles = torch.empty(*t.shape[:-1], 2 * t.shape[-1], dtype=torch.int64, device=t.device)
        nibbles[..., 0::2], nibbles[..., 1::2] = (t % 16).long(), (t // 16).long()
        return table[nibbles] * power[st[name + "_scales"][at].long()].repeat_interleave(BLOCK, dim=-1)

    S, E, K, N = case["T"] * case["k"], case["E"], case["K"], case["N"]
    if op == "gradient":
        d_x = torch.zeros(S, K, dtype=torch.float64, device="cuda")
        d_w = torch.zeros(E, N, K, dtype=torch.float64, device="cuda")
        for e in range(E):
            rows = slice(lo[e], lo[e + 1])
            if lo[e + 1] > lo[e]:
                d_y = st["d_y"][rows].double()
                d_x[rows] = d_y @ st["w"][e].double()
                d_w[e] = d_y.t() @ st["x"][rows].double()
        return d_x, d_w
    y = torch.zeros(S, N, dtype=torch.float64, device="cuda")
    for e in range(E):
        rows = slice(lo[e], lo[e + 1])
        if lo[e + 1] > lo[e]:
            y[rows] = wide("x", rows) @ wide("w", e).t()
    if op == "product4" and case["silu"]:
        half = N // 2
        y = y[:, :half] * torch.sigmoid(y[:, :half]) * y[:, half:]
    return y

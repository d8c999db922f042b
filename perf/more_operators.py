"""Cases of the products in 8 bits and of the updates made of products, for timing and comparison.

Four operators: a matrix laid out in 8-bit floating point (e4m3) with a scale for each block of 128 (``quant``), the product
of two such matrices (``product``), the same for ragged groups of rows, each group with its own right operand (``grouped``),
and an update orthogonalised by Newton-Schulz products (``orthogonalise``).  ``run`` computes a case in plain torch
operations or, with ``own`` set, through the library's entry points.

A scale belongs to 128 columns of one row (block 1) or of 128 rows (block 128).  Scales are stored with the block of columns
outermost: the value at (i, k) is q[i, k] * s[k // 128, i // block].
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn

# coefficients of x -> a x + b x^3 + c x^5 for the singular values: five steps to somewhere near 1, or eight to 1
QUINTIC = {"fast": [(3.4445, -4.7750, 2.0315)] * 5, "tight": [(1.875, -1.25, 0.375)] * 8}


def listed():
    return [
        # one decode step's activations before a layer: latency counts
        {"name": "quant-decode", "op": "quant", "dtype": "bf16", "batch": 1, "M": 16, "K": 4096, "block": 1, "transpose": 0},
        # a prefill's or a training batch's activations
        {"name": "quant-rows", "op": "quant", "dtype": "bf16", "batch": 1, "M": 8192, "K": 4096, "block": 1, "transpose": 0},
        # a training batch's output gradients turned for the weight gradient, whose sum runs over the tokens
        {"name": "quant-turned", "op": "quant", "dtype": "f32", "batch": 1, "M": 4096, "K": 8192, "block": 1, "transpose": 1},
        # a decode step of 16 requests through one layer: the weights are read once
        {"name": "product-decode", "op": "product", "M": 16, "N": 4096, "K": 4096, "blockB": 128},
        # a prefill or a training batch, forward or input gradient
        {"name": "product-prefill", "op": "product", "M": 4096, "N": 4096, "K": 4096, "blockB": 128},
        # a weight gradient: both operands turned, scales by row in both, summed over 8192 tokens
        {"name": "product-wgrad", "op": "product", "M": 2048, "N": 4096, "K": 8192, "blockB": 1},
        # odd sizes
        {"name": "product-odd", "op": "product", "M": 1001, "N": 777, "K": 513, "blockB": 128},
        # a decode step's expert layer: 128 rows over 64 experts
        {"name": "grouped-decode", "op": "grouped", "G": 64, "R": 128, "T": 16, "N": 1024, "K": 2048, "skew": 1.0},
        # a prefill's expert layer: 4096 tokens, 8 experts each of 32
        {"name": "grouped-prefill", "op": "grouped", "G": 32, "R": 32768, "T": 4096, "N": 2048, "K": 2048, "skew": 1.0},
        # many small matrices (one per head), one call for all
        {"name": "orthogonalise-heads", "op": "orthogonalise", "dtype": "f32", "batch": 32, "M": 128, "N": 512, "steps": "fast",
         "rank": 16},
        # a layer's weights, odd and tall
        {"name": "orthogonalise-odd", "op": "orthogonalise", "dtype": "bf16", "batch": 1, "M": 1001, "N": 513, "steps": "tight",
         "rank": 64},
        # a large layer's weights
        {"name": "orthogonalise-large", "op": "orthogonalise", "dtype": "f32", "batch": 1, "M": 4096, "N": 4096, "steps": "fast",
         "rank": 256},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, evenly spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """Mostly multiples of 64, as models have them; one in five as it comes."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.2 else max(64, n // 64 * 64)


def draw(rng):
    op = rng.choice(["quant", "product", "product", "grouped", "orthogonalise"])
    if op == "quant":
        block, batch = rng.choice([1, 1, 128]), rng.choice([1, 1, 8])
        return {"op": op, "dtype": rng.choice(["f32", "f16", "bf16"]), "batch": batch, "M": _log(rng, 1, 8192 // batch),
                "K": _size(rng, 64, 4096), "block": block, "transpose": rng.choice([0, 1])}
    if op == "product":
        return {"op": op, "M": _log(rng, 1, 4096), "N": _size(rng, 64, 4096), "K": _size(rng, 64, 4096), "blockB": rng.choice([1, 128])}
    if op == "grouped":
        R = _log(rng, 1, 16384)
        return {"op": op, "G": _log(rng, 2, 64), "R": R, "T": rng.choice([0, max(1, R // 8)]), "N": _size(rng, 256, 2048),
                "K": _size(rng, 256, 2048), "skew": round(rng.uniform(0.5, 2.0), 2)}
    batch = rng.choice([1, 1, 4, 16])
    M, N = _size(rng, 32, 2048 // batch), _size(rng, 32, 2048 // batch)
    return {"op": op, "dtype": rng.choice(["f32", "bf16"]), "batch": batch, "M": M, "N": N, "steps": rng.choice(["fast", "tight"]),
            "rank": max(4, min(M, N) // 8)}


def _splits(rng, G, R, skew):
    """Row counts of G groups that sum to R, from popularities that differ by a factor of about e**skew; some are empty when R is small."""
    p = np.exp(skew * rng.standard_normal(G) / 2)
    return rng.multinomial(R, p / p.sum())


def _blocks(x, n, dim):
    """x with dimension `dim` filled up with zeros to whole blocks of n and split into (blocks, n)."""
    size = x.shape[dim]
    short = -size % n
    if short:
        shape = list(x.shape)
        shape[dim] = short
        x = torch.cat([x, x.new_zeros(shape)], dim)
    return x.unflatten(dim, ((size + short) // n, n))


def _quantised(y, block):
    """(values, scales) of y (batch, rows, k): the least power of two s with max|y| / s <= 448 in each block, 1 for zeros."""
    y = y.float()
    b, m, k = y.shape
    top = _blocks(y.abs(), 128, 2).amax(3)
    if block > 1:
        top = _blocks(top, block, 1).amax(2)
    bits = top.view(torch.int32)
    # the exponent of top / 1.75, rounded up, less the 8 of 448 = 1.75 * 2^8; as a normal number's bits
    s = ((((bits + 0x1FFFFF) >> 23) - 8).clamp_min(1) << 23).view(torch.float32)
    s = torch.where(top == 0, torch.ones_like(s), s)
    full = s.repeat_interleave(block, 1)[:, :m].repeat_interleave(128, 2)[:, :, :k]
    return (y / full).to(E4M3), s.transpose(1, 2).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case}

    def normal(*shape, std=1.0):
        return torch.empty(*shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen)

    def spread(*shape):
        """Rows of different size, as tokens and weights have them."""
        return normal(*shape) * torch.exp(normal(*shape[:-1], 1))

    def ints(a):
        return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()

    op = case["op"]
    if op == "quant":
        n, M, K = case["batch"], case["M"], case["K"]
        st["X"] = (spread(n, K, M) if case["transpose"] else spread(n, M, K)).to(DTYPES[case["dtype"]])
        st["Q"] = torch.zeros(n, M, K, device="cuda").to(E4M3)
        st["S"] = torch.zeros(n, -(-K // 128), -(-M // case["block"]), device="cuda")
    elif op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        qa, sa = _quantised(spread(1, M, K), 1)
        qb, sb = _quantised(spread(1, N, K) * K ** -0.5, case["blockB"])
        # scales as they come from elsewhere: any 32-bit values, not only powers of two
        st.update(A=qa[0], SA=sa[0] * (1 + torch.rand(sa[0].shape, generator=gen, device="cuda")), B=qb[0],
                  SB=sb[0] * (1 + torch.rand(sb[0].shape, generator=gen, device="cuda")), C=torch.zeros(M, N, device="cuda"))
    elif op == "grouped":
        G, R, T, N, K = case["G"], case["R"], case["T"], case["N"], case["K"]
        rng = np.random.default_rng(seed)
        counts = _splits(rng, G, R, case["skew"])
        st["longest"] = int(counts.max())
        st["offsets"] = ints(np.concatenate([[0], np.cumsum(counts)]))
        st["rows"] = ints(rng.integers(0, T, R)) if T else None
        qa, sa = _quantised(spread(1, T or R, K), 1)
        qb, sb = _quantised(normal(G, N, K, std=K ** -0.5), 128)
        st.update(A=qa[0], SA=sa[0], B=qb, SB=sb * (1 + torch.rand(sb.shape, generator=gen, device="cuda")),
                  C=torch.zeros(R, N, device="cuda"))
    else:
        # a gradient: some strong directions, and noise all over
        n, M, N, r = case["batch"], case["M"], case["N"], case["rank"]
        g = torch.bmm(normal(n, M, r) * torch.exp(normal(n, 1, r)), normal(n, r, N)) * r ** -0.5 + normal(n, M, N, std=0.2)
        st["G"] = (g * 1e-3).to(DTYPES[case["dtype"]])
        st["O"] = torch.zeros(n, M, N, dtype=torch.bfloat16, device="cuda")
    return st


# ------------------------------------------------------------------ the library's entry points
def _run_own(st):
    import dense_gemm_optimisation_f32_amd as dg

    c = st["case"]
    if c["op"] == "quant":
        n, M, K = c["batch"], c["M"], c["K"]
        fn = {"f32": dg.quant_e4m3_f32, "f16": dg.quant_e4m3_f16, "bf16": dg.quant_e4m3_bf16}[c["dtype"]]
        kb, rb = st["S"].shape[1:]
        fn(c["transpose"], c["block"], M, K, st["X"], M if c["transpose"] else K, M * K, st["Q"], K, M * K, st["S"], rb, kb * rb, n)
        return {"values": st["Q"], "scales": st["S"]}
    if c["op"] == "product":
        M, N, K = c["M"], c["N"], c["K"]
        dg.gemm_e4m3_f32acc(c["blockB"], M, N, K, 1.0, st["A"], K, st["SA"], M, st["B"], K, st["SB"], st["SB"].shape[1], 0.0, st["C"], N)
        return {"C": st["C"]}
    if c["op"] == "grouped":
        G, R, N, K = c["G"], c["R"], c["N"], c["K"]
        rows = c["T"] or R
        kb, nb = st["SB"].shape[1:]
        dg.gemm_grouped_e4m3_f32acc(128, G, R, N, K, 1.0, st["A"], rows, K, st["SA"], rows, st["rows"], st["B"], K, N * K, st["SB"], nb,
                                    kb * nb, st["offsets"], 0.0, st["C"], N)
        return {"C": st["C"]}
    n, M, N = c["batch"], c["M"], c["N"]
    fn = {"f32": dg.orthogonalise_f32, "bf16": dg.orthogonalise_bf16}[c["dtype"]]
    fn(M, N, QUINTIC[c["steps"]], 1.0, st["G"], N, M * N, st["O"], N, M * N, n)
    return {"O": st["O"]}


# ------------------------------------------------------------------ the plain forms
def _plain_quant(st):
    x = st["X"]
    q, s = _quantised(x.transpose(1, 2).contiguous() if st["case"]["transpose"] else x, st["case"]["block"])
    return {"values": q, "scales": s}


def _values(q, s, block):
    """The numbers that values q (rows, k) and scales s (blocks of k, blocks of rows) stand for, in 32 bits."""
    return q.float() * s.t().repeat_interleave(block, 0)[: q.shape[0]].repeat_interleave(128, 1)[:, : q.shape[1]]


def _plain_product(st):
    return {"C": _values(st["A"], st["SA"], 1) @ _values(st["B"], st["SB"], st["case"]["blockB"]).t()}


def _plain_grouped(st):
    c, at = st["case"], st["rows"]
    a = _values(st["A"], st["SA"], 1)
    # rows laid out as groups x longest, zero behind each group's end
    i = st["offsets"][:-1].long()[:, None] + torch.arange(st["longest"], device=a.device)
    held = i < st["offsets"][1:, None]
    i = torch.where(held, i, 0)
    a = torch.where(held[..., None], a[i if at is None else at.long()[i]], 0.0)
    s = st["SB"].transpose(1, 2).repeat_interleave(128, 1)[:, : c["N"]].repeat_interleave(128, 2)[:, :, : c["K"]]
    y = torch.bmm(a, (st["B"].float() * s).transpose(1, 2).contiguous())
    p = torch.arange(c["R"], device=a.device)
    g = (p[:, None] >= st["offsets"][1:]).sum(1)   # the group of row p: how many end at or before it
    return {"C": y[g, p - st["offsets"].long()[g]]}


def _plain_orthogonalise(st):
    x = st["G"].float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    x = x / x.square().sum((1, 2), keepdim=True).sqrt()
    for a, b, c in QUINTIC[st["case"]["steps"]]:
        s = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.bmm(b * s + c * torch.bmm(s, s), x)
    return {"O": (x.transpose(1, 2).contiguous() if tall else x).bfloat16()}


_PLAIN = {"quant": _plain_quant, "product": _plain_product, "grouped": _plain_grouped, "orthogonalise": _plain_orthogonalise}


def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state)


def work(case):
    """Bytes with each input read and each output written once, and the operations of the products."""
    op = case["op"]
    if op == "quant":
        n, M, K = case["batch"], case["M"], case["K"]
        each = 5 if case["dtype"] == "f32" else 3
        return {"bytes": n * (each * M * K + 4 * -(-M // case["block"]) * -(-K // 128)), "flops": 2 * n * M * K}
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + 4 * M * N + 4 * -(-K // 128) * (M + -(-N // case["blockB"])), "flops": 2 * M * N * K}
    if op == "grouped":
        G, R, T, N, K = case["G"], case["R"], case["T"], case["N"], case["K"]
        a_rows, hit = (min(T, R) if T else R), min(G, R)
        return {"bytes": a_rows * K + hit * N * K + 4 * (R * N + a_rows * -(-K // 128) + (R if T else 0) + G + 1), "flops": 2 * R * N * K}
    n, m, k = case["batch"], min(case["M"], case["N"]), max(case["M"], case["N"])
    # a step: X X^T and A A are symmetric (half of each), and B X
    return {"bytes": n * m * k * (6 if case["dtype"] == "f32" else 4), "flops": n * len(QUINTIC[case["steps"]]) * (m * m * k + m ** 3 + 2 * m * m * k)}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        x = st["X"].double()
        if case["transpose"]:
            x = x.transpose(1, 2)
        n, M, K, block = case["batch"], case["M"], case["K"], case["block"]
        q = torch.zeros(n, M, K, dtype=torch.float64, device="cuda")
        s = torch.ones(n, -(-K // 128), -(-M // block), dtype=torch.float64, device="cuda")
        for j in range(s.shape[1]):
            part = x[:, :, 128 * j: 128 * j + 128]
            top = part.abs().amax(2)
            if block > 1:
                top = torch.stack([t.amax(1) for t in top.split(block, 1)], 1)
            fraction, power = torch.frexp(top / 448)   # top / 448 = fraction * 2^power, 1/2 <= fraction < 1
            scale = torch.exp2((power - (fraction == 0.5).int()).double())
            scale = torch.where(top == 0, 1.0, scale.clamp_min(2.0 ** -126))
            s[:, j] = scale
            rows = torch.arange(M, device="cuda") // block
            v = part / scale[:, rows, None]
            # neighbours of v in e4m3 lie 2^(exponent - 3) apart, 2^-9 near zero
            step = torch.exp2((torch.frexp(v).exponent - 1).clamp_min(-6).double() - 3)
            q[:, :, 128 * j: 128 * j + 128] = torch.round(v / step) * step
        return {"values": q, "scales": s}
    if op in ("product", "grouped"):
        def row(q, s, block):
            at = torch.arange(q.shape[1], device="cuda") // 128
            r = torch.arange(q.shape[0], device="cuda") // block
            return q.double() * s.double()[at][:, r].t()

        a = row(st["A"], st["SA"], 1)
        if op == "product":
            return {"C": a @ row(st["B"], st["SB"], case["blockB"]).t()}
        out = torch.zeros(st["C"].shape, dtype=torch.float64, device="cuda")
        at = st["offsets"].tolist()
        for g in range(case["G"]):
            lo, hi = at[g], at[g + 1]
            if hi > lo:
                out[lo:hi] = (a[lo:hi] if st["rows"] is None else a[st["rows"][lo:hi].long()]) @ row(st["B"][g], st["SB"][g], 128).t()
        return {"C": out}
    # where it is quick, through the eigenvectors of the smaller G G^T and a polynomial of the singular values
    out = torch.zeros(st["O"].shape, dtype=torch.float64, device="cuda")
    for i in range(case["batch"]):
        g = st["G"][i].double()
        short = g if g.shape[0] <= g.shape[1] else g.t()
        norm = torch.linalg.norm(g)
        if short.shape[0] <= 640:
            value, vector = (t.cuda() for t in torch.linalg.eigh((short @ short.t()).cpu()))
            sigma = value.clamp_min(0).sqrt() / norm
            gain = torch.ones_like(sigma) / norm
            for a, b, c in QUINTIC[case["steps"]]:
                factor = a + b * sigma ** 2 + c * sigma ** 4
                sigma, gain = sigma * factor, gain * factor
            x = (vector * gain) @ (vector.t() @ short)
        else:
            x = short / norm
            for a, b, c in QUINTIC[case["steps"]]:
                y = x @ x.t()
                x = a * x + b * (y @ x) + c * (y @ (y @ x))
        out[i] = x if g.shape[0] <= g.shape[1] else x.t()
    return {"O": out}

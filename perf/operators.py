"""Cases of the products whose right operand is chosen per row, for timing and comparison.

Seven directions of four operators: routing to experts and its gradient (``route``, ``route_grad``), the experts' products and
their weight gradient (``experts``, ``wgrad``), the weighted sum back to tokens and its gradient (``combine``,
``combine_grad``), and low-rank adapters beside a shared projection (``lora``).  ``run`` computes a case in plain torch
operations or, with ``own`` set, through the library's entry points.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one decode step of 16 requests: many experts in groups, sigmoid scores with a balancing bias; latency counts
        {"name": "route-decode", "op": "route", "T": 16, "E": 256, "k": 8, "score": "sigmoid", "bias": True, "groups": 8,
         "group_k": 4, "group_top": 2, "renorm": True, "scale": 2.5},
        # a long prefill or a training batch over the same experts
        {"name": "route-prefill", "op": "route", "T": 32768, "E": 256, "k": 8, "score": "sigmoid", "bias": True, "groups": 8,
         "group_k": 4, "group_top": 2, "renorm": True, "scale": 2.5},
        # a training batch's gradient through softmax scores that are not renormalised
        {"name": "route-grad", "op": "route_grad", "T": 16384, "E": 128, "k": 8, "score": "softmax", "renorm": False, "scale": 1.0},
        # a decode step's expert layer: 128 rows over 64 experts, every hit expert's weights read once
        {"name": "experts-decode", "op": "experts", "dtype": "bf16", "G": 64, "R": 128, "T": 16, "K": 2048, "N": 1024, "transB": 1,
         "skew": 1.0},
        # a prefill's expert layer: 4096 tokens, 8 experts each of 32
        {"name": "experts-prefill", "op": "experts", "dtype": "bf16", "G": 32, "R": 32768, "T": 4096, "K": 2048, "N": 2048,
         "transB": 0, "skew": 1.0},
        # odd sizes, fp16, the input-gradient orientation, rows in place (not gathered)
        {"name": "experts-odd", "op": "experts", "dtype": "f16", "G": 5, "R": 1001, "T": 0, "K": 777, "N": 513, "transB": 1, "skew": 2.0},
        # weight gradients of an expert layer
        {"name": "wgrad", "op": "wgrad", "dtype": "bf16", "G": 32, "R": 16384, "T": 4096, "M": 2048, "N": 1024, "skew": 1.0},
        # a prefill's expert outputs back in token order
        {"name": "combine", "op": "combine", "T": 4096, "k": 8, "N": 2048},
        # its gradient in training
        {"name": "combine-grad", "op": "combine_grad", "dtype": "bf16", "T": 8192, "k": 4, "N": 1024},
        # one token of one request with an adapter
        {"name": "lora-token", "op": "lora", "dtype": "f16", "M": 1, "N": 4096, "K": 4096, "rank": 16, "adapters": 4, "transB": 0},
        # a decode step of 48 requests over 32 adapters
        {"name": "lora-decode", "op": "lora", "dtype": "bf16", "M": 48, "N": 4096, "K": 4096, "rank": 32, "adapters": 32, "transB": 1},
        # a prefill of requests with 8 adapters
        {"name": "lora-prefill", "op": "lora", "dtype": "bf16", "M": 4096, "N": 4096, "K": 4096, "rank": 16, "adapters": 8, "transB": 1},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, evenly spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """Mostly multiples of 64, as models have them; one in five as it comes."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.2 else max(64, n // 64 * 64)


def draw(rng):
    op = rng.choice(["route", "route_grad", "experts", "experts", "wgrad", "combine", "combine_grad", "lora", "lora"])
    dtype = rng.choice(["f16", "bf16"])
    skew = round(rng.uniform(0.5, 2.0), 2)
    if op in ("route", "route_grad"):
        E = rng.choice([8, 16, 32, 60, 64, 96, 128, 160, 256])
        k = rng.choice([k for k in (1, 2, 4, 6, 8) if 2 * k <= E])
        c = {"op": op, "T": _log(rng, 1, 32768), "E": E, "k": k, "score": rng.choice(["softmax", "sigmoid"]),
             "renorm": k > 1 and rng.random() < 0.5, "scale": rng.choice([1.0, 2.5])}
        if op == "route":
            groups = rng.choice([g for g in (1, 4, 8) if E % g == 0 and E // g >= max(2, k // 2)])
            c.update(bias=rng.random() < 0.5, groups=groups, group_k=max(1, groups // 2), group_top=rng.choice([1, 2]))
        return c
    if op == "experts":
        G, R = _log(rng, 2, 64), _log(rng, 1, 16384)
        T = rng.choice([0, max(1, R // 8)])
        return {"op": op, "dtype": dtype, "G": G, "R": R, "T": T, "K": _size(rng, 256, 2048), "N": _size(rng, 256, 2048),
                "transB": rng.choice([0, 1]), "skew": skew}
    if op == "wgrad":
        G, R = _log(rng, 2, 32), _log(rng, 64, 16384)
        T = rng.choice([0, max(1, R // 8)])
        return {"op": op, "dtype": dtype, "G": G, "R": R, "T": T, "M": _size(rng, 256, 2048), "N": _size(rng, 256, 2048), "skew": skew}
    if op in ("combine", "combine_grad"):
        c = {"op": op, "T": _log(rng, 1, 4096), "k": rng.choice([1, 2, 4, 6, 8]), "N": _size(rng, 256, 4096)}
        return dict(c, dtype=dtype) if op == "combine_grad" else c
    return {"op": op, "dtype": dtype, "M": _log(rng, 1, 4096), "N": _size(rng, 512, 4096), "K": _size(rng, 512, 4096),
            "rank": rng.choice([4, 8, 16, 32, 64]), "adapters": _log(rng, 1, 32), "transB": rng.choice([0, 1])}


def _splits(rng, G, R, skew):
    """Row counts of G groups that sum to R, from popularities that differ by a factor of about e**skew; some are empty when R is small."""
    p = np.exp(skew * rng.standard_normal(G) / 2)
    return rng.multinomial(R, p / p.sum())


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case}

    def normal(*shape, dtype=torch.float32, std=1.0):
        return torch.empty(*shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen).to(dtype)

    def ints(a):
        return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()

    def empty(*shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype, device="cuda")

    op = case["op"]
    if op in ("route", "route_grad"):
        T, E, k = case["T"], case["E"], case["k"]
        st["logits"] = normal(T, E, std=2.0)
        if op == "route":
            st["bias"] = normal(E, std=0.1) if case["bias"] else None
            st.update(ids=empty(T, k, dtype=torch.int32), weights=empty(T, k), offsets=empty(E + 1, dtype=torch.int32),
                      rows=empty(T * k, dtype=torch.int32), slots=empty(T, k, dtype=torch.int32))
        else:
            # k distinct experts of each token, as a router chose them
            st["ids"] = torch.argsort(normal(T, E), dim=1)[:, :k].to(torch.int32).contiguous()
            st["dweights"] = normal(T, k)
            st["dlogits"] = empty(T, E)
    elif op in ("experts", "wgrad"):
        G, R, T, dt = case["G"], case["R"], case["T"], DTYPES[case["dtype"]]
        counts = _splits(rng, G, R, case["skew"])
        st["longest"] = int(counts.max())
        st["offsets"] = ints(np.concatenate([[0], np.cumsum(counts)]))
        st["rows"] = ints(rng.integers(0, T, R)) if T else None
        if op == "experts":
            K, N = case["K"], case["N"]
            st["A"] = normal(T or R, K, dtype=dt)
            st["B"] = normal(*((G, N, K) if case["transB"] else (G, K, N)), dtype=dt, std=K ** -0.5)
            st["C"] = empty(R, N)
        else:
            st["A"] = normal(T or R, case["M"], dtype=dt)
            st["B"] = normal(R, case["N"], dtype=dt)
            st["C"] = empty(G, case["M"], case["N"])
    elif op in ("combine", "combine_grad"):
        T, k, N = case["T"], case["k"], case["N"]
        st["Y"] = normal(T * k, N)
        st["slots"] = torch.randperm(T * k, generator=gen, device="cuda").to(torch.int32).view(T, k)
        w = torch.rand(T, k, generator=gen, device="cuda")
        st["weights"] = w / w.sum(1, keepdim=True)
        if op == "combine":
            st["C"] = empty(T, N)
        else:
            st["dC"] = normal(T, N)
            st["dY"] = empty(T * k, N, dtype=DTYPES[case["dtype"]])
            st["dweights"] = empty(T, k)
    else:
        M, N, K, r, n, dt = case["M"], case["N"], case["K"], case["rank"], case["adapters"], DTYPES[case["dtype"]]
        st["A"] = normal(M, K, dtype=dt)
        st["B"] = normal(*((N, K) if case["transB"] else (K, N)), dtype=dt, std=K ** -0.5)
        st["LA"] = normal(n, r, K, dtype=dt, std=K ** -0.5)
        st["LB"] = normal(n, N, r, dtype=dt, std=0.5 * r ** -0.5)
        # requests are runs of rows: one row each in a decode step, up to some hundreds in a prefill; one in nine has no adapter
        run = 1 if M <= 64 else 192
        ids = np.repeat(rng.integers(0, n, M // run + 1), run)[:M]
        ids[np.repeat(rng.random(M // run + 1) < 1 / 9, run)[:M]] = -1
        if M < 4:
            ids[:] = rng.integers(0, n, M)
        st["ids"] = ints(ids)
        st["ranks"] = ints(rng.integers((r + 1) // 2, r + 1, n))
        st["scales"] = torch.rand(n, generator=gen, device="cuda") + 0.5
        st["C"] = empty(M, N)
    return st


# ------------------------------------------------------------------ the library's entry points
def _run_own(st):
    import dense_gemm_optimisation_f32_amd as dg

    c = st["case"]
    op = c["op"]
    if op == "route":
        dg.moe_route_f32(c["T"], c["E"], st["logits"], c["E"], st["bias"], int(c["score"] == "sigmoid"), c["groups"], c["group_k"],
                         c["group_top"], c["k"], int(c["renorm"]), c["scale"], st["ids"], st["weights"], st["offsets"], st["rows"],
                         st["slots"])
        return {n: st[n] for n in ("ids", "weights", "offsets", "rows", "slots")}
    if op == "route_grad":
        dg.moe_route_f32_grad(c["T"], c["E"], st["logits"], c["E"], int(c["score"] == "sigmoid"), c["k"], int(c["renorm"]), c["scale"],
                              st["ids"], st["dweights"], st["dlogits"], c["E"])
        return {"dlogits": st["dlogits"]}
    if op == "experts":
        G, R, N, K = c["G"], c["R"], c["N"], c["K"]
        fn = dg.gemm_grouped_f16_f32acc_ex if c["dtype"] == "f16" else dg.gemm_grouped_bf16_f32acc_ex
        fn(c["transB"], G, R, N, K, 1.0, st["A"], c["T"] or R, K, st["rows"], st["B"], K if c["transB"] else N, K * N, st["offsets"],
           0.0, st["C"], N)
        return {"C": st["C"]}
    if op == "wgrad":
        G, R, M, N = c["G"], c["R"], c["M"], c["N"]
        fn = dg.gemm_grouped_wgrad_f16_f32acc if c["dtype"] == "f16" else dg.gemm_grouped_wgrad_bf16_f32acc
        fn(G, R, M, N, 1.0, st["A"], c["T"] or R, M, st["rows"], st["B"], R, N, None, st["offsets"], 0.0, st["C"], N, M * N)
        return {"C": st["C"]}
    if op == "combine":
        dg.moe_combine_f32(c["T"], c["k"], c["N"], st["Y"], c["T"] * c["k"], c["N"], st["slots"], st["weights"], 0.0, st["C"], c["N"])
        return {"C": st["C"]}
    if op == "combine_grad":
        fn = dg.moe_combine_grad_f16 if c["dtype"] == "f16" else dg.moe_combine_grad_bf16
        fn(c["T"], c["k"], c["N"], st["dC"], c["N"], st["Y"], c["T"] * c["k"], c["N"], st["slots"], st["weights"], st["dY"], c["N"],
           st["dweights"])
        return {"dY": st["dY"], "dweights": st["dweights"]}
    M, N, K, r = c["M"], c["N"], c["K"], c["rank"]
    fn = dg.gemm_lora_f16_f32acc_ex if c["dtype"] == "f16" else dg.gemm_lora_bf16_f32acc_ex
    fn(c["transB"], M, N, K, r, c["adapters"], 1.0, st["A"], K, st["B"], K if c["transB"] else N, st["LA"], K, r * K, st["LB"], r, N * r,
       st["scales"], st["ranks"], st["ids"], 0.0, st["C"], N)
    return {"C": st["C"]}


# ------------------------------------------------------------------ the plain forms
def _plain_route(st):
    c = st["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    # the choice in 64 bits: scores next to one another decide which expert is taken
    x = st["logits"].double()
    s = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, 1)
    choice = s if st["bias"] is None else s + st["bias"].double()
    if G > 1:
        g = choice.view(T, G, E // G).sort(dim=2, descending=True, stable=True).values[:, :, : c["group_top"]].sum(2)
        best = g.sort(dim=1, descending=True, stable=True).indices[:, : c["group_k"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, best, True)
        choice = torch.where(keep.view(T, G, 1), choice.view(T, G, E // G), -math.inf).view(T, E)
    ids = choice.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(s, 1, ids)
    w = (w / w.sum(1, keepdim=True) if c["renorm"] else w) * c["scale"]
    flat = ids.reshape(-1)
    order = flat.sort(stable=True).indices
    counts = torch.zeros(E, dtype=torch.int64, device=x.device).scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat([torch.zeros_like(counts[:1]), counts.cumsum(0)])
    slots = torch.empty_like(order).scatter_(0, order, torch.arange(T * k, device=x.device))
    return {"ids": ids.int(), "weights": w.float(), "offsets": offsets.int(), "rows": (order // k).int(), "slots": slots.view(T, k).int()}


def _plain_route_grad(st):
    c = st["case"]
    ids = st["ids"].long()
    s = torch.sigmoid(st["logits"]) if c["score"] == "sigmoid" else torch.softmax(st["logits"], 1)
    chosen, dw = torch.gather(s, 1, ids), st["dweights"] * c["scale"]
    if c["renorm"]:
        total = chosen.sum(1, keepdim=True)
        dw = (dw - (dw * chosen / total).sum(1, keepdim=True)) / total
    ds = torch.zeros_like(s).scatter_(1, ids, dw)
    return {"dlogits": ds * s * (1 - s) if c["score"] == "sigmoid" else s * (ds - (ds * s).sum(1, keepdim=True))}


def _padded(st, x, at):
    """Rows `at` of x laid out as groups x longest, zero behind each group's end, and the places that hold rows."""
    i = st["offsets"][:-1].long()[:, None] + torch.arange(st["longest"], device=x.device)
    held = i < st["offsets"][1:, None]
    i = torch.where(held, i, 0)
    i = i if at is None else at.long()[i]
    return torch.where(held[..., None], x[i].float(), 0.0), held


def _plain_experts(st):
    a, held = _padded(st, st["A"], st["rows"])
    b = st["B"].float()
    y = torch.bmm(a, b.transpose(1, 2).contiguous() if st["case"]["transB"] else b)
    p = torch.arange(st["case"]["R"], device=a.device)
    g = (p[:, None] >= st["offsets"][1:]).sum(1)   # the group of row p: how many end at or before it
    return {"C": y[g, p - st["offsets"].long()[g]]}


def _plain_wgrad(st):
    a, _ = _padded(st, st["A"], st["rows"])
    b, _ = _padded(st, st["B"], None)
    return {"C": torch.bmm(a.transpose(1, 2).contiguous(), b)}


def _plain_combine(st):
    return {"C": (st["Y"][st["slots"].long()] * st["weights"][:, :, None]).sum(1)}


def _plain_combine_grad(st):
    slots = st["slots"].long()
    dy = st["weights"][:, :, None] * st["dC"][:, None, :]
    out = torch.empty_like(st["dY"]).index_copy_(0, slots.reshape(-1), dy.view(-1, dy.shape[2]).to(st["dY"].dtype))
    return {"dY": out, "dweights": (st["Y"][slots] * st["dC"][:, None, :]).sum(2)}


def _plain_lora(st):
    c = st["case"]
    M, N, K, r, n = c["M"], c["N"], c["K"], c["rank"], c["adapters"]
    a, b = st["A"].float(), st["B"].float()
    base = a @ (b.t() if c["transB"] else b)
    # every adapter's narrow product, of which a row keeps its own adapter's and that one's rank
    t = (a @ st["LA"].float().view(n * r, K).t()).view(M, n, r)
    mine = st["ids"][:, None] == torch.arange(n, device=a.device)
    within = torch.arange(r, device=a.device) < st["ranks"][:, None]
    t = torch.where(mine[:, :, None] & within, t * st["scales"][:, None], 0.0)
    lb = torch.where(within[:, None, :], st["LB"].float(), 0.0)
    return {"C": base + t.view(M, n * r) @ lb.permute(0, 2, 1).reshape(n * r, N)}


_PLAIN = {"route": _plain_route, "route_grad": _plain_route_grad, "experts": _plain_experts, "wgrad": _plain_wgrad,
          "combine": _plain_combine, "combine_grad": _plain_combine_grad, "lora": _plain_lora}


def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state)


def work(case):
    """Bytes with each input read and each output written once, and the operations of the products (of the scores and sums elsewhere)."""
    op = case["op"]
    if op in ("route", "route_grad"):
        T, E, k = case["T"], case["E"], case["k"]
        if op == "route":
            return {"bytes": 4 * (T * E + E * case["bias"] + 4 * T * k + E + 1), "flops": 8 * T * E}
        return {"bytes": 4 * (2 * T * E + 2 * T * k), "flops": 8 * T * E}
    if op in ("combine", "combine_grad"):
        T, k, N = case["T"], case["k"], case["N"]
        if op == "combine":
            return {"bytes": 4 * (T * k * N + T * N + 2 * T * k), "flops": 2 * T * k * N}
        return {"bytes": 4 * (T * k * N + T * N + 3 * T * k) + 2 * T * k * N, "flops": 3 * T * k * N}
    if op == "lora":
        M, N, K, r, n = case["M"], case["N"], case["K"], case["rank"], min(case["adapters"], case["M"])
        return {"bytes": 2 * (M * K + K * N + n * r * (K + N)) + 4 * (M * N + M + 2 * n), "flops": 2 * M * N * K + 2 * M * r * (K + N)}
    G, R, T = case["G"], case["R"], case["T"]
    a_rows = min(T, R) if T else R
    if op == "experts":
        K, N = case["K"], case["N"]
        return {"bytes": 2 * (a_rows * K + min(G, R) * K * N) + 4 * (R * N + (R if T else 0) + G + 1), "flops": 2 * R * K * N}
    M, N = case["M"], case["N"]
    return {"bytes": 2 * (a_rows * M + R * N) + 4 * (G * M * N + (R if T else 0) + G + 1), "flops": 2 * R * M * N}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        x = st["logits"].cpu().numpy().astype(np.float64)
        T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
        if case["score"] == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-x))
        else:
            e = np.exp(x - x.max(1, keepdims=True))
            s = e / e.sum(1, keepdims=True)
        choice = s + (0.0 if st["bias"] is None else st["bias"].cpu().numpy().astype(np.float64))
        if G > 1:
            size = E // G
            score = np.sort(choice.reshape(T, G, size), axis=2)[:, :, size - case["group_top"]:].sum(2)
            lost = np.argsort(-score, axis=1, kind="stable")[:, case["group_k"]:]
            dead = np.zeros((T, G), dtype=bool)
            np.put_along_axis(dead, lost, True, 1)
            choice = np.where(np.repeat(dead, size, axis=1), -np.inf, choice)
        ids = np.argsort(-choice, axis=1, kind="stable")[:, :k]
        w = np.take_along_axis(s, ids, 1)
        if case["renorm"]:
            w = w / w.sum(1, keepdims=True)
        # token t's choice j is row (how many choose a lower expert) + (how many before it choose the same)
        flat = ids.reshape(-1)
        order = np.lexsort((np.arange(T * k), flat))
        slots = np.empty(T * k, dtype=np.int64)
        slots[order] = np.arange(T * k)
        offsets = np.searchsorted(flat[order], np.arange(E + 1))
        out = {"ids": ids, "weights": w * case["scale"], "offsets": offsets, "rows": order // k, "slots": slots.reshape(T, k)}
        return {n: torch.from_numpy(v if n == "weights" else v.astype(np.int32)) for n, v in out.items()}
    if op == "route_grad":
        # differentiated by torch's own rules, in 64 bits
        x = st["logits"].double().requires_grad_(True)
        s = 1.0 / (1.0 + torch.exp(-x)) if case["score"] == "sigmoid" else torch.exp(x - torch.logsumexp(x, 1, keepdim=True))
        w = torch.gather(s, 1, st["ids"].long())
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        (w * case["scale"] * st["dweights"].double()).sum().backward()
        return {"dlogits": x.grad}
    if op in ("experts", "wgrad"):
        at, A, B = st["offsets"].tolist(), st["A"], st["B"]
        out = torch.zeros(st["C"].shape, dtype=torch.float64, device="cuda")
        for g in range(case["G"]):
            lo, hi = at[g], at[g + 1]
            if hi == lo:
                continue
            a = (A[st["rows"][lo:hi].long()] if st["rows"] is not None else A[lo:hi]).double()
            if op == "experts":
                b = B[g].double()
                out[lo:hi] = a @ (b.t() if case["transB"] else b)
            else:
                out[g] = a.t() @ B[lo:hi].double()
        return {"C": out}
    if op == "combine":
        out = torch.zeros(case["T"], case["N"], dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            out += st["weights"][:, j, None].double() * st["Y"][st["slots"][:, j].long()].double()
        return {"C": out}
    if op == "combine_grad":
        dY = torch.zeros(st["Y"].shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros(case["T"], case["k"], dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            at = st["slots"][:, j].long()
            dY[at] = st["weights"][:, j, None].double() * st["dC"].double()
            dw[:, j] = (st["dC"].double() * st["Y"][at].double()).sum(1)
        return {"dY": dY, "dweights": dw}
    a, b = st["A"].double(), st["B"].double()
    out = a @ (b.t() if case["transB"] else b)
    ids, ranks = st["ids"].tolist(), st["ranks"].tolist()
    for n in sorted(set(ids) - {-1}):
        at = torch.tensor([i for i, v in enumerate(ids) if v == n], device="cuda")
        la, lb = st["LA"][n, : ranks[n]].double(), st["LB"][n, :, : ranks[n]].double()
        out[at] += st["scales"][n].double() * ((a[at] @ la.t()) @ lb.t())
    return {"C": out}

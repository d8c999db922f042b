"""The calls whose right operand is chosen per row against their definitions in 64 bits (GPU).

Tolerances, u = 2^-24 (half a step of fp32, relative):
  * products: normalized error |C - ref| / (sum of the magnitudes of all terms) <= 1e-5, the library's own bound for
    fp32 accumulation; bit-exact where every entry is a small whole number.
  * routing: ids, offsets, rows and slots are equal.  A weight is a score made of exponentials of differences of logits:
    rounding the difference d costs |d| u, an exponential, the sum and the quotients a few u: (16 + range of the row) u.
  * its gradient: the same, on the sum of the magnitudes of its terms.
  * combining: k + 1 fused multiply-adds: (k + 2) u on the magnitudes; dY is one product (u) rounded once to 16 bits, half
    a step of that type (and half its smallest subnormal); dweights a sum of N terms, four columns per thread and
    1024 columns apart, then ten pairwise sums: (4 ceil(N / 1024) + 12) u.
"""
from __future__ import annotations

import math

import numpy as np
import pytest

import dense_gemm_optimisation_f32_amd as dg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TOL = 1e-5
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dg.load_library()
    yield
    torch.cuda.synchronize()


def rng_of(*key):
    return np.random.default_rng(list(str(key).encode()))


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def host(t):
    return t.detach().cpu().double().numpy() if t.is_floating_point() else t.cpu().numpy()


def done():
    torch.cuda.synchronize()


# ------------------------------------------------------------------ routing
def route_oracle(x, bias, score, groups, group_k, group_top, k, renorm, scale):
    """The definition, token by token."""
    x = x.astype(np.float64)
    T, E = x.shape
    b = np.zeros(E) if bias is None else bias.astype(np.float64)
    ids, w = np.full((T, k), -1), np.zeros((T, k))
    order = lambda v: np.lexsort((np.arange(len(v)), np.where(np.isnan(v), np.inf, -v), np.isnan(v)))  # noqa: E731
    for t in range(T):
        free = (x[t] != -np.inf) & (b != -np.inf)
        with np.errstate(all="ignore"):
            if score:
                s = 1.0 / (1.0 + np.exp(-x[t]))
            else:
                e = np.exp(x[t] - np.max(x[t])) if np.any(x[t] != -np.inf) else np.zeros(E)
                s = e / e.sum()
            c = s + b
            if bias is None and (groups == 1 or group_top == 1):   # the logits order the experts, also where 64 bits saturate
                c = np.where(np.isnan(s), np.nan, x[t])
            if groups > 1:
                size, best = E // groups, np.full(groups, -np.inf)
                some = np.zeros(groups, dtype=bool)
                for g in range(groups):
                    v = c[g * size : (g + 1) * size][free[g * size : (g + 1) * size]]
                    if len(v):
                        best[g], some[g] = v[order(v)[:group_top]].sum(), True
                rank = np.lexsort((np.arange(groups), np.where(np.isnan(best), np.inf, -best), np.isnan(best), ~some))
                keep = np.zeros(groups, dtype=bool)
                keep[rank[:group_k]] = True
                free = free & np.repeat(keep, size)
        at = np.flatnonzero(free)
        pick = at[order(c[at])][:k]
        ids[t, : len(pick)] = pick
        with np.errstate(all="ignore"):
            v = s[pick]
            if renorm and score == 0 and len(pick) and not np.isnan(v).any():
                v = np.exp(x[t, pick] - x[t, pick].max())   # the same quotient where every chosen score underflows
            if renorm and len(pick):
                v = v / v.sum() if v.sum() != 0 else v * 0
            w[t, : len(pick)] = scale * v
    flat = np.where(ids < 0, E, ids).reshape(-1)
    by = np.argsort(flat, kind="stable")
    offsets = np.searchsorted(flat[by], np.arange(E + 1))
    rows = np.where(flat[by] < E, by // k, -1)
    slots = np.empty(T * k, dtype=np.int64)
    slots[by] = np.arange(T * k)
    return ids, w, offsets, rows, np.where(flat < E, slots, -1).reshape(T, k)


def route_call(x, ldl, bias, score, groups, group_k, group_top, k, renorm, scale, T, E, layout=True, stream=None):
    n = T * k
    out = {"ids": torch.full((n,), 77, dtype=I32, device="cuda"), "weights": torch.full((n,), 7.0, device="cuda")}
    if layout:
        out.update(offsets=torch.full((E + 1,), 77, dtype=I32, device="cuda"), rows=torch.full((n,), 77, dtype=I32, device="cuda"),
                   slots=torch.full((n,), 77, dtype=I32, device="cuda"))
    dg.moe_route_f32(T, E, x, ldl, bias, score, groups, group_k, group_top, k, renorm, scale, out["ids"], out["weights"],
                     out.get("offsets"), out.get("rows"), out.get("slots"), stream=stream)
    return out


def route_check(x, bias, score, groups, group_k, group_top, k, renorm, scale, ldl=None):
    T, E = x.shape
    ldl = ldl or E
    buf = np.full((T, ldl), np.nan, dtype=np.float32)
    buf[:, :E] = x
    got = route_call(dev(buf), ldl, None if bias is None else dev(bias), score, groups, group_k, group_top, k, renorm, scale, T, E)
    done()
    ids, w, offsets, rows, slots = route_oracle(x, bias, score, groups, group_k, group_top, k, renorm, scale)
    assert np.array_equal(host(got["ids"]).reshape(T, k), ids)
    assert np.array_equal(host(got["offsets"]), offsets)
    assert np.array_equal(host(got["rows"]), rows)
    assert np.array_equal(host(got["slots"]).reshape(T, k), slots)
    fin = np.where(np.isfinite(x), x, 0.0)
    tol = (16 + fin.max(1, initial=0) - fin.min(1, initial=0))[:, None] * U
    g = host(got["weights"]).reshape(T, k)
    assert np.array_equal(np.isnan(g), np.isnan(w))
    ok = ~np.isnan(w)
    assert np.all((np.abs(g - w) <= tol * np.abs(w) + 1e-37)[ok]), np.nanmax(np.abs(g - w))
    return got


@pytest.mark.parametrize("T", [1, 3, 64, 65, 500])
@pytest.mark.parametrize("E,groups,group_k,k", [(1, 1, 1, 1), (5, 1, 1, 2), (8, 4, 2, 4), (60, 1, 1, 4), (64, 8, 3, 8), (100, 4, 2, 7),
                                                (160, 8, 3, 6), (256, 8, 4, 8), (512, 1, 1, 8), (1000, 50, 5, 32), (1024, 64, 64, 10)])
@pytest.mark.parametrize("score", [0, 1])
def test_route(T, E, groups, group_k, k, score):
    print(f"[route] T={T} E={E} groups={groups} k={k} score={score}", flush=True)
    rng = rng_of("route", T, E, groups, k, score)
    for bias, renorm, top in ((True, 1, min(2, E // groups)), (False, 0, 1)):
        x = (rng.standard_normal((T, E)) * 2).astype(np.float32)
        b = (rng.standard_normal(E) * 0.1).astype(np.float32) if bias else None
        route_check(x, b, score, groups, group_k, top, k, renorm, 2.5 if bias else 1.0, ldl=E + 3 if T < 64 else None)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("T", [7, 200])
def test_route_ties_and_unavailable(T, score):
    rng = rng_of("ties", T, score)
    x = rng.integers(-2, 3, (T, 96)).astype(np.float32)          # many equal scores: lowest index, lowest group
    route_check(x, None, score, 1, 1, 1, 8, 1, 1.0)
    route_check(x, None, score, 8, 3, 1, 8, 0, 1.0)
    x[rng.random((T, 96)) < 0.9] = -np.inf                        # fewer experts than choices
    x[::3] = -np.inf                                              # padded tokens
    route_check(x, None, score, 1, 1, 1, 12, 1, 1.0)
    route_check(x, None, score, 8, 2, 2, 6, 0, 1.0)
    b = np.zeros(96, dtype=np.float32)
    b[rng.random(96) < 0.5] = -np.inf                             # experts taken out for all tokens
    route_check(x, b, score, 4, 2, 2, 6, 1, 1.0)
    route_check(np.full((T, 96), -np.inf, dtype=np.float32), None, score, 1, 1, 1, 4, 1, 1.0)
    b[:] = -np.inf
    route_check(np.zeros((T, 96), dtype=np.float32), b, score, 1, 1, 1, 4, 1, 1.0)


@pytest.mark.parametrize("score", [0, 1])
def test_route_extreme_values(score):
    low = np.finfo(np.float32).min
    x = np.array([[low] * 8, [low, 0, low, 1, low, low, low, low], [80, -80, 0, 100, -100, 3, 2, 1], [0, 0, 0, 0, 0, 0, 0, 0],
                  [np.nan, 1, 2, 3, -np.inf, -1, 0, 5], [1, np.nan, np.nan, np.nan, np.nan, np.nan, np.nan, np.nan]], dtype=np.float32)
    for renorm in (0, 1):
        for k in (1, 3, 8):
            route_check(x, None, score, 1, 1, 1, k, renorm, 1.0)
            route_check(x, np.array([0, 0, 0, 0, 9, 9, 9, 9], dtype=np.float32), score, 1, 1, 1, k, renorm, 1.0)
    x = np.array([[np.inf, 1, 2, 3]], dtype=np.float32)
    route_check(x, None, score, 1, 1, 1, 2, 1, 1.0)
    route_check(x, None, score, 1, 1, 1, 2, 0, 1.0)


@pytest.mark.parametrize("E,k", [(8, 2), (64, 8), (256, 8), (1000, 32)])
@pytest.mark.parametrize("score,renorm", [(0, 0), (0, 1), (1, 0), (1, 1)])
@pytest.mark.parametrize("bias", [False, True])
def test_route_weights_of_far_logits(E, k, score, renorm, bias):
    """Weights keep their digits wherever the logits are: an exponential is off by 3 u, 1 + e and its reciprocal by 3, the
    k scores' sum by 6 and their own, the quotient by 4: 24 u.  A softmax that is not renormalised divides by a sum of E
    exponentials, each off by 3 u and its difference's rounding, which its share of the sum weighs (ln E at most), and
    21 additions: 48 u."""
    rng = rng_of("far", E, k, score, renorm, bias)
    T = 300
    x = (rng.standard_normal((T, E)) * 0.7).astype(np.float32)
    x += rng.choice([-57.0, -40.0, -20.0, -8.0, 0.0, 20.0], (T, 1)).astype(np.float32)      # all of a token's
    x[::2, : E // 2] -= rng.uniform(0, 55, (T // 2, 1)).astype(np.float32)                # half of its experts far below
    b = None
    if bias:      # the lower half is chosen too
        b = np.zeros(E, dtype=np.float32)
        b[: max(1, k // 2)] = 2
    got = route_call(dev(x), E, None if b is None else dev(b), score, 1, 1, 1, k, renorm, 1.0, T, E)
    done()
    ids, w = host(got["ids"]).reshape(T, k), host(got["weights"]).reshape(T, k)
    xd = x.astype(np.float64)
    v = np.take_along_axis(xd, ids, 1)
    if score:
        want = 1 / (1 + np.exp(-v))
    elif renorm:
        want = np.exp(v - v.max(1, keepdims=True))
    else:
        want = np.exp(v - xd.max(1, keepdims=True)) / np.exp(xd - xd.max(1, keepdims=True)).sum(1, keepdims=True)
    if renorm:
        want = want / want.sum(1, keepdims=True)
    # (a weight below 2^-126, e^-87.3, is below fp32's normal values and may be held as anything from 0 to that)
    off = (np.maximum(np.abs(w - want) - 2.0 ** -126, 0) / want).max() / U
    print(f"[far] {off:.1f} u", flush=True)
    assert off <= (24 if score or renorm else 48)


@pytest.mark.parametrize("score,seed", [(1, 88), (1, 89), (0, 3)])
def test_route_near_ties(score, seed):
    """Many tokens, so that some hold scores nearer to one another than 32 bits tell; and scores made so: experts in
    pairs whose biases differ by a few 2^-24."""
    T, E, k = 20000, 256, 8
    g = torch.Generator().manual_seed(seed)
    x, b = torch.randn(T, E, generator=g) * 2, torch.randn(E, generator=g) * 0.1
    x[:300, 1::2] = x[:300, ::2]
    b[1::2] = torch.where(torch.rand(E // 2, generator=g) < 0.5, b[::2] + 2.0 ** -23, b[1::2])
    s = torch.sigmoid(x.double()) if score else torch.softmax(x.double(), 1)
    c = s + b.double()
    for groups, group_k, top in ((1, 1, 1), (8, 4, 2)):
        d = c
        if groups > 1:
            best = c.view(T, groups, -1).sort(dim=2, descending=True).values[:, :, :top].sum(2)
            keep = best.sort(dim=1, descending=True, stable=True).indices[:, :group_k]
            d = torch.where(torch.zeros(T, groups, dtype=torch.bool).scatter_(1, keep, True)[:, :, None], c.view(T, groups, -1), -math.inf).view(T, E)
        want = d.sort(dim=1, descending=True, stable=True).indices[:, :k]
        got = route_call(x.cuda(), E, b.cuda(), score, groups, group_k, top, k, 1, 1.0, T, E)["ids"].view(T, k).cpu().long()
        done()
        assert torch.equal(got, want), (got != want).any(1).nonzero()[:5]


@pytest.mark.parametrize("E", [40, 100, 256, 500, 1000])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_scores_that_differ_in_their_last_bits(E, groups):
    """Choice scores 1 + m 2^-52, m = 1 .. 24 (sigmoid of a logit near -35 beside a bias of 1, in the middle of what rounds
    to m), of which equal ones go by index and all others by score; and 1 - m 2^-52 (logits near 35, no bias)."""
    T, k = 50, min(32, E // 2)
    rng = rng_of("last bits", E, groups)
    m = rng.integers(1, 25, (T, E))
    x = np.log(m * 2.0 ** -52)          # sigmoid(x) = m 2^-52 (1 - m 2^-52): rounded to 32 bits, within 2^-19 of it
    x = x.astype(np.float32)
    b = np.ones(E, dtype=np.float32)
    c = 1 / (1 + np.exp(-x.astype(np.float64))) + 1.0
    assert np.array_equal(c, 1 + m * 2.0 ** -52)
    route_check(x, b, 1, groups, max(1, groups // 2), min(2, E // groups), k, 0, 1.0)
    if groups > 1:                      # (without a bias and groups the logits themselves are compared)
        y = -np.log(m * 2.0 ** -52).astype(np.float32)
        c = 1 / (1 + np.exp(-y.astype(np.float64)))
        assert np.array_equal(c, 1 - m * 2.0 ** -52)
        route_check(y, None, 1, groups, 2, 2, k, 0, 1.0)


@pytest.mark.parametrize("T,E,k", [(20011, 100, 32), (70001, 40, 8), (9000, 1000, 32)])
def test_route_many_choices(T, E, k):
    """More runs of choices than one pass over their counts takes."""
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(T))
    x[::5] = -math.inf                                            # padded tokens
    got = {n: v.cpu().long() for n, v in route_call(x.cuda(), E, None, 0, 1, 1, 1, k, 1, 1.0, T, E).items()}
    ids = torch.where(x[:, :1] == -math.inf, -1, x.sort(dim=1, descending=True, stable=True).indices[:, :k]).reshape(-1)
    flat = torch.where(ids < 0, E, ids)
    by = flat.sort(stable=True).indices
    assert torch.equal(got["ids"], ids)
    assert torch.equal(got["offsets"], torch.searchsorted(flat[by], torch.arange(E + 1)))
    assert torch.equal(got["rows"], torch.where(flat[by] < E, by // k, -1))
    slots = torch.empty_like(by)
    slots[by] = torch.arange(T * k)
    assert torch.equal(got["slots"], torch.where(flat < E, slots, -1))


def test_route_without_layout_and_empty():
    x = dev(np.random.default_rng(5).standard_normal((300, 32)).astype(np.float32))
    a = route_call(x, 32, None, 0, 1, 1, 1, 4, 1, 1.0, 300, 32)
    b = route_call(x, 32, None, 0, 1, 1, 1, 4, 1, 1.0, 300, 32, layout=False)
    assert torch.equal(a["ids"], b["ids"]) and torch.equal(a["weights"], b["weights"])
    c = route_call(x, 32, None, 0, 1, 1, 1, 4, 1, 1.0, 0, 32)
    done()
    assert torch.equal(c["offsets"], torch.zeros(33, dtype=I32, device="cuda"))


def grad_forward(x, ids, score, renorm, scale):
    """fp64 weights of given ids, differentiable."""
    s = torch.sigmoid(x) if score else torch.softmax(x, 1)
    w = torch.gather(s, 1, ids.clamp(min=0)) * (ids >= 0)
    if renorm:
        w = w / w.sum(1, keepdim=True)
    return w * scale


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 5, 2), (9, 64, 8), (50, 100, 7), (130, 256, 8), (11, 1000, 32)])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [0, 1])
def test_route_grad(T, E, k, score, renorm):
    rng = rng_of("rgrad", T, E, k, score, renorm)
    x = torch.from_numpy((rng.standard_normal((T, E)) * 2).astype(np.float32))
    ids = torch.from_numpy(np.argsort(rng.random((T, E)), 1)[:, :k].astype(np.int32))
    if T > 8 and k > 1:
        ids[::4, k - 1] = -1                     # an unfilled choice
    dw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32))
    scale = 1.5
    out = torch.full((T, E + 2), math.nan, device="cuda")
    xin = torch.full((T, E + 1), math.nan)
    xin[:, :E] = x
    dg.moe_route_f32_grad(T, E, xin.cuda(), E + 1, score, k, renorm, scale, ids.cuda(), dw.cuda(), out, E + 2)
    done()
    xd = x.double().requires_grad_(True)
    loss = (grad_forward(xd, ids.long(), score, renorm, scale) * dw.double()).sum()
    loss.backward()
    got = out[:, :E].cpu().double()
    assert torch.isnan(out[:, E:]).all()
    # the magnitudes of the terms: p_j (|g_j| + sum p |g|), and s_e (|g_e| + sum s |g|) over all experts
    with torch.no_grad():
        s = torch.sigmoid(x.double()) if score else torch.softmax(x.double(), 1)
        p = grad_forward(x.double(), ids.long(), score, renorm, 1.0)
        g = scale * dw.double().abs()
        mag = torch.zeros(T, E, dtype=torch.float64)
        mag.scatter_add_(1, ids.long().clamp(min=0), p * (g + (p * g).sum(1, keepdim=True)) * (ids >= 0))
        if not renorm and not score:
            mag += s * (p * g).sum(1, keepdim=True)
        tol = (16 + x.max(1).values - x.min(1).values).double()[:, None] * U * mag + 1e-37
        # the definition's own rounding in 64 bits, where terms that cancel exactly leave it: a few 2^-53 of the
        # terms s_e / D * sum |g| (D the chosen scores' sum, or 1)
        d = (torch.gather(s, 1, ids.long().clamp(min=0)) * (ids >= 0)).sum(1, keepdim=True) if renorm else 1.0
        tol += 16 * 2.0 ** -53 * s / d * g.sum(1, keepdim=True)
    assert ((got - xd.grad).abs() <= tol).all(), ((got - xd.grad).abs() - tol).max()
    # differences of the definition: step h, error of the order h^2 and 2^-53 / h
    h = 1e-5
    for t in range(min(T, 2)):
        for e in list(range(min(E, 3))) + [int(i) for i in ids[t, :2] if i >= 0]:
            q = x.double().clone()
            q[t, e] += h
            r = x.double().clone()
            r[t, e] -= h
            d = ((grad_forward(q, ids.long(), score, renorm, scale) - grad_forward(r, ids.long(), score, renorm, scale)) * dw.double()).sum() / (2 * h)
            assert abs(float(d) - float(got[t, e])) <= 1e-6 * (1 + abs(float(loss.detach())) + scale * float(dw[t].abs().sum()))


def sure_grad(x, ids, dw, score, renorm, scale):
    """The gradient in 64 bits without a difference of near numbers, and the magnitude of its terms: for the chosen,
    s_e (sum_i s_i (g_e - g_i) + g_e u), u the scores of the others; renormalised p_e sum_i p_i (g_e - g_i), times s(-x)
    for sigmoid scores."""
    T, E = x.shape
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        at = ids[t]
        g = scale * dw[t]
        if renorm:
            p = np.exp(x[t, at] - x[t, at].max()) if score == 0 else 1 / (1 + np.exp(-x[t, at]))
            p = p / p.sum()
            d = g[:, None] - g[None, :]
            f = 1.0 if score == 0 else 1 / (1 + np.exp(x[t, at]))
            out[t, at], mag[t, at] = p * (d @ p) * f, p * (np.abs(d) @ p) * f
            continue
        e = np.exp(x[t] - x[t].max())
        others = np.ones(E, dtype=bool)
        others[at] = False
        u, s = e[others].sum() / e.sum(), e / e.sum()
        d = g[:, None] - g[None, :]
        out[t], mag[t] = -s * (g @ s[at]), s * (np.abs(g) @ s[at])
        out[t, at], mag[t, at] = s[at] * (d @ s[at] + g * u), s[at] * (np.abs(d) @ s[at] + np.abs(g) * u)
    return out, mag


@pytest.mark.parametrize("E,k", [(8, 1), (64, 2), (128, 1), (128, 8), (256, 8), (1000, 4)])
@pytest.mark.parametrize("gap", [12, 16, 20, 30, 60])
@pytest.mark.parametrize("score,renorm", [(0, 0), (0, 1), (1, 1)])
def test_route_grad_of_a_sure_router(E, k, gap, score, renorm):
    """One expert, or the k chosen ones, far above the rest.  Relative to the magnitude m of the gradient's own terms: a
    score is off by (range + 8) u (the difference of logits, an exponential, sum and quotient), its product and the sums
    by 8 u more, and differences from the gradient of the best expert, whose score is 1 / 2k or more of them, have terms
    |D_e| + sum_i s_i |D_i| of at most (2 + 4 k) m."""
    rng = rng_of("sure", E, k, gap, score, renorm)
    T = 12
    x = rng.standard_normal((T, E)).astype(np.float32)
    ids = np.argsort(rng.random((T, E)), 1)[:, :k].astype(np.int32)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    for t in range(T):
        if t % 3 == 2:
            x[t, ids[t]] += gap          # all of the chosen
        else:
            x[t, ids[t, 0]] += gap       # one of them
    dw[T // 2 :] = 1 + dw[T // 2 :] * np.float32(2.0 ** -20)   # nearly the same gradient for all
    out = torch.full((T, E), math.nan, device="cuda")
    dg.moe_route_f32_grad(T, E, dev(x), E, score, k, renorm, 2.5, dev(ids), dev(dw), out, E)
    done()
    want, mag = sure_grad(x.astype(np.float64), ids, dw.astype(np.float64), score, renorm, 2.5)
    # renormalised: everything is formed in 64 bits and rounded once
    tol = U * (2 if renorm else (16 + (x.max(1) - x.min(1))[:, None]) * (2 + 4 * k)) * mag + 1e-37
    off = np.abs(host(out) - want)
    worst = (off / np.maximum(mag, 1e-37)).max() / U
    print(f"[sure] {worst:.1f} u", flush=True)
    assert (off <= tol).all(), worst


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [0, 1])
def test_route_grad_of_ids_named_twice(score, renorm):
    """The definition's gradient also where two choices of a token are the same expert."""
    rng = rng_of("twice", score, renorm)
    T, E, k = 20, 40, 4
    x = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32))
    ids = torch.from_numpy(rng.integers(0, 3, (T, k)).astype(np.int32))
    dw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32))
    out = torch.full((T, E), math.nan, device="cuda")
    dg.moe_route_f32_grad(T, E, x.cuda(), E, score, k, renorm, 1.0, ids.cuda(), dw.cuda(), out, E)
    done()
    xd = x.double().requires_grad_(True)
    (grad_forward(xd, ids.long(), score, renorm, 1.0) * dw.double()).sum().backward()
    # each of the k terms, at most |dw| each with a score of at most 1, and their sum: (16 + range + 2 k) u of them
    tol = (16 + float(x.max() - x.min()) + 2 * k) * U * dw.double().abs().sum(1, keepdim=True) * 2
    assert ((out.cpu().double() - xd.grad).abs() <= tol).all()


def test_route_grad_of_padded_rows():
    x = torch.full((3, 8), -math.inf)
    x[1] = torch.arange(8.0)
    ids = torch.tensor([[-1, -1], [7, 6], [-1, -1]], dtype=I32)
    for score in (0, 1):
        for renorm in (0, 1):
            out = torch.full((3, 8), math.nan, device="cuda")
            dg.moe_route_f32_grad(3, 8, x.cuda(), 8, score, 2, renorm, 1.0, ids.cuda(), torch.ones(3, 2, device="cuda"), out, 8)
            done()
            assert (out[0] == 0).all() and (out[2] == 0).all() and torch.isfinite(out[1]).all()


# ------------------------------------------------------------------ grouped products
def counts_of(rng, G, R, how):
    if how == "even":
        c = np.full(G, R // G)
        c[: R - c.sum()] += 1
    elif how == "one":
        c = np.zeros(G, dtype=int)
        c[G // 2] = R
    else:
        c = rng.multinomial(R, rng.dirichlet(np.full(G, 0.3)))
    return np.concatenate([[0], np.cumsum(c)]).astype(np.int32)


def values(rng, shape, vals):
    return rng.integers(-4, 5, shape).astype(np.float32) if vals == "int4" else rng.uniform(-1, 1, shape).astype(np.float32)


def grouped_check(t, transB, G, R, N, K, *, M=None, how="skewed", gather=True, alpha=1.0, beta=0.0, vals="pm1", pads=(0, 0, 0),
                  offset=0, tail=0, bad_rows=False, shared=False):
    rng = rng_of("grouped", t, transB, G, R, N, K, how, gather, alpha, beta, vals, pads, offset, tail)
    print(f"[grouped] {t} transB={transB} G={G} R={R} N={N} K={K} how={how} gather={gather} beta={beta} {vals} pads={pads} off={offset}",
          flush=True)
    M = M or (max(1, R // 3) if gather else R + tail)
    lda, ldb, ldc = K + pads[0], (K if transB else N) + pads[1], N + pads[2]
    br = N if transB else K
    a = torch.from_numpy(values(rng, (M, lda), vals)).to(DT[t])
    b = torch.from_numpy(values(rng, (1 if shared else G, br, ldb), vals)).to(DT[t])
    c0 = torch.from_numpy(values(rng, (R + tail, ldc), vals))
    offs = counts_of(rng, G, R, how)
    rows = rng.integers(0, M, R + tail).astype(np.int32) if gather else None
    if bad_rows:
        rows[:: 3] = -1
        rows[1:: 3] = M
    a[:, K:] = math.nan                      # what lies between rows is never used
    b[:, :, (K if transB else N):] = math.nan
    put = lambda x: torch.cat([torch.zeros(offset, dtype=x.dtype), x.reshape(-1)]).cuda()[offset:]  # noqa: E731
    C = c0.clone() if beta != 0 else torch.full((R + tail, ldc), math.nan)
    mark = C.clone()
    dC = put(C)
    fn = dg.gemm_grouped_f16_f32acc_ex if t == "f16" else dg.gemm_grouped_bf16_f32acc_ex
    fn(transB, G, R + tail, N, K, alpha, put(a), M, lda, None if rows is None else dev(rows), put(b), ldb, 0 if shared else br * ldb,
       dev(offs), beta, dC, ldc)
    done()
    got = dC.cpu().view(R + tail, ldc)
    # rows of no group and the columns between rows stay as they were
    assert torch.equal(got[R:].view(torch.int32), mark[R:].view(torch.int32))
    assert torch.equal(got[:, N:].contiguous().view(torch.int32), mark[:, N:].contiguous().view(torch.int32))
    ad, bd = a[:, :K].double(), b.double()
    for g in range(G):
        lo, hi = int(offs[g]), int(offs[g + 1])
        if lo == hi:
            continue
        at = torch.from_numpy(rows[lo:hi]).long() if rows is not None else torch.arange(lo, hi)
        x = torch.where(((at >= 0) & (at < M))[:, None], ad[at.clamp(0, M - 1)], 0.0)
        w = bd[0 if shared else g]
        w = w[:, :K].t() if transB else w[:, :N]
        ref = alpha * (x @ w) + (beta * c0[lo:hi, :N].double() if beta else 0)
        mag = abs(alpha) * (x.abs() @ w.abs()) + (abs(beta) * c0[lo:hi, :N].double().abs() if beta else 0)
        out = got[lo:hi, :N].double()
        if vals == "int4":
            assert torch.equal(out, ref)
        assert ((out - ref).abs() <= TOL * mag).all(), float(((out - ref).abs() / mag.clamp(min=1e-30)).max())


SHAPES = [(1, 1, 1, 1), (3, 5, 7, 9), (2, 1, 64, 64), (4, 63, 65, 129), (5, 300, 130, 200), (8, 40, 256, 512), (3, 700, 264, 328),
          (16, 1000, 128, 256), (70, 500, 96, 96), (2, 1100, 520, 72), (130, 90, 72, 136)]


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("transB", [0, 1])
@pytest.mark.parametrize("G,R,N,K", SHAPES)
def test_grouped(t, transB, G, R, N, K):
    grouped_check(t, transB, G, R, N, K, vals="int4")
    grouped_check(t, transB, G, R, N, K, gather=False, how="even", alpha=1.5, beta=-0.5)


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("transB", [0, 1])
def test_grouped_layouts(t, transB):
    for how in ("one", "even"):
        grouped_check(t, transB, 6, 390, 192, 320, how=how, vals="int4")
    grouped_check(t, transB, 3, 200, 128, 256, pads=(2, 4, 1), vals="int4")             # dword-aligned rows
    grouped_check(t, transB, 3, 200, 127, 255, pads=(1, 2, 3), vals="int4")             # rows that start at odd halves
    grouped_check(t, transB, 3, 200, 128, 256, offset=1, vals="int4")                   # every base one element on
    grouped_check(t, transB, 3, 200, 128, 256, offset=2, pads=(8, 8, 4))
    grouped_check(t, transB, 4, 150, 128, 256, tail=41, vals="int4", beta=1.0)          # rows behind the last group
    grouped_check(t, transB, 4, 10, 128, 256, tail=300, gather=False, vals="int4")
    grouped_check(t, transB, 4, 150, 128, 256, bad_rows=True, vals="int4")
    grouped_check(t, transB, 4, 150, 128, 256, bad_rows=True, beta=0.5)
    grouped_check(t, transB, 9, 333, 128, 256, shared=True, vals="int4")                # strideB = 0
    grouped_check(t, transB, 2, 2000, 512, 1024, vals="int4")
    grouped_check(t, transB, 2, 2000, 520, 1032)
    grouped_check(t, transB, 3, 24, 1024, 2048)
    grouped_check(t, transB, 3, 24, 1032, 2056, beta=1.0)


@pytest.mark.parametrize("transB", [0, 1])
def test_grouped_no_product_and_bad_offsets(transB):
    c = torch.arange(48.0).view(8, 6)
    off = torch.tensor([0, 3, 5], dtype=I32, device="cuda")
    x = torch.full((64,), math.nan, dtype=torch.float16, device="cuda")
    for K, alpha in ((0, 1.0), (5, 0.0)):
        for beta in (0.0, 2.0):
            C = c.cuda()
            dg.gemm_grouped_f16_f32acc_ex(transB, 2, 8, 6, K, alpha, x, 8, max(K, 1), None, x, max(K, 6), 0, off, beta, C, 6)
            done()
            want = c.clone()
            want[:5] *= beta
            assert torch.equal(C.cpu(), want)
    # offsets below zero, past R and descending lead nowhere outside C
    ones = torch.ones(64, dtype=torch.float16, device="cuda")
    for o in ([-5, 3, 100], [2**31 - 1, -(2**31), 4], [7, 2, 2]):
        C = torch.full((10, 6), -1.0, device="cuda")
        dg.gemm_grouped_f16_f32acc_ex(transB, 2, 8, 6, 4, 1.0, ones, 8, 4, None, ones, 6, 0, torch.tensor(o, dtype=I32, device="cuda"), 0.0, C, 6)
        done()
        assert (C[8:] == -1).all()
        if o[0] == -5:
            assert (C[:8] == 4).all()


@pytest.mark.parametrize("G", [4, 40])
@pytest.mark.parametrize("N,K", [(64, 64), (65, 63), (256, 128)])
@pytest.mark.parametrize("transB", [0, 1])
def test_grouped_offsets_that_rise_again(transB, N, K, G):
    """Offsets 0, R, 0, R, ...: more row tiles than any ascending offsets hold.  What is written is written once more with
    the same values (one shared operand), and nothing outside C."""
    R = 200
    a = torch.ones(R, K, dtype=torch.float16, device="cuda")
    b = torch.ones(N * K, dtype=torch.float16, device="cuda")
    off = torch.tensor([0, R] * (G // 2) + [0], dtype=I32, device="cuda")
    buf = torch.full((R + 600, N), -1.0, device="cuda")
    dg.gemm_grouped_f16_f32acc_ex(transB, G, R, N, K, 1.0, a, R, K, None, b, K if transB else N, 0, off, 0.0, buf[300:], N)
    done()
    assert (buf[:300] == -1).all() and (buf[300 + R:] == -1).all()
    assert (buf[300 : 300 + R] == K).all()


def test_grouped_offsets_that_rise_again_past_32_bits():
    """The same with 32767 times 16384 row tiles of 16 columns of tiles each."""
    R, G, N, K = 16384 * 64, 65535, 1024, 3
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GiB of device memory")
    a = torch.ones(R, K, dtype=torch.float16, device="cuda")
    b = torch.ones(K * N, dtype=torch.float16, device="cuda")
    off = torch.tensor([0, R], dtype=I32).repeat((G + 1) // 2)
    off[-1] = R - 37 * 64
    buf = torch.full((R + 2048, N), -1.0, device="cuda")
    dg.gemm_grouped_f16_f32acc_ex(0, G, R, N, K, 1.0, a, R, K, None, b, N, 0, off.cuda(), 0.0, buf[1024:], N)
    done()
    assert (buf[:1024] == -1).all() and (buf[1024 + R:] == -1).all()
    assert (buf[1024 : 1024 + R] == K).all()


def test_grouped_no_product_reads_no_rows():
    # fewer row indices than rows of C: without a product none is read
    off = torch.tensor([0, 5000], dtype=I32, device="cuda")
    rows = torch.zeros(1, dtype=I32, device="cuda")
    x = torch.zeros(64, dtype=torch.float16, device="cuda")
    for K, M, alpha in ((0, 8, 1.0), (5, 8, 0.0), (5, 0, 1.0)):
        C = torch.ones(5000, 6, device="cuda")
        dg.gemm_grouped_f16_f32acc_ex(0, 1, 5000, 6, K, alpha, x, M, max(K, 1), rows, x, 6, 0, off, 3.0, C, 6)
        done()
        assert (C.cpu() == 3).all()


@pytest.mark.parametrize("R,K,N", [(20, 64, 64), (200, 64, 128), (600, 128, 256), (20, 63, 65), (200, 63, 65), (200, 64, 65)])
@pytest.mark.parametrize("transB", [0, 1])
def test_grouped_rows_outside_meet_infinite_weights(transB, R, K, N):
    rows = torch.arange(R, dtype=I32)
    rows[::3], rows[1::7] = -1, R
    b = torch.full((1, N, K) if transB else (1, K, N), math.inf, dtype=torch.float16)
    a = torch.ones(R, K, dtype=torch.float16)
    C = torch.full((R, N), math.nan, device="cuda")
    off = torch.tensor([0, R], dtype=I32, device="cuda")
    dg.gemm_grouped_f16_f32acc_ex(transB, 1, R, N, K, 1.0, a.cuda(), R, K, rows.cuda(), b.cuda(), K if transB else N, K * N, off, 0.0, C, N)
    done()
    out = ((rows < 0) | (rows >= R))
    assert (C.cpu()[out] == 0).all() and (C.cpu()[~out] == math.inf).all()
    C.fill_(math.nan)   # without indices: rows of C past A's last
    dg.gemm_grouped_f16_f32acc_ex(transB, 1, R, N, K, 1.0, a.cuda(), R - 7, K, None, b.cuda(), K if transB else N, K * N, off, 0.0, C, N)
    done()
    assert (C.cpu()[R - 7:] == 0).all() and (C.cpu()[:R - 7] == math.inf).all()


# ------------------------------------------------------------------ weight gradients
def wgrad_check(t, G, R, M, N, *, how="skewed", ga=True, gb=False, alpha=1.0, beta=0.0, vals="pm1", pads=(0, 0, 0), offset=0, bad=False):
    rng = rng_of("wgrad", t, G, R, M, N, how, ga, gb, alpha, beta, vals, pads, offset, bad)
    print(f"[wgrad] {t} G={G} R={R} M={M} N={N} how={how} ga={ga} gb={gb} beta={beta} {vals} pads={pads} off={offset}", flush=True)
    na, nb = (max(1, R // 2) if ga else R), (max(1, R // 2) if gb else R)
    lda, ldb, ldc = M + pads[0], N + pads[1], N + pads[2]
    a = torch.from_numpy(values(rng, (na, lda), vals)).to(DT[t])
    b = torch.from_numpy(values(rng, (nb, ldb), vals)).to(DT[t])
    a[:, M:] = math.nan
    b[:, N:] = math.nan
    c0 = torch.from_numpy(values(rng, (G, M, ldc), vals))
    offs = counts_of(rng, G, R, how)
    ra = rng.integers(0, na, R).astype(np.int32) if ga else None
    rb = rng.integers(0, nb, R).astype(np.int32) if gb else None
    if bad:
        ra[:: 3] = -1
        ra[1:: 3] = na
    put = lambda x: torch.cat([torch.zeros(offset, dtype=x.dtype), x.reshape(-1)]).cuda()[offset:]  # noqa: E731
    C = c0.clone() if beta != 0 else torch.full((G, M, ldc), math.nan)
    mark = C.clone()
    dC = put(C)
    fn = dg.gemm_grouped_wgrad_f16_f32acc if t == "f16" else dg.gemm_grouped_wgrad_bf16_f32acc
    fn(G, R, M, N, alpha, put(a), na, lda, None if ra is None else dev(ra), put(b), nb, ldb, None if rb is None else dev(rb), dev(offs),
       beta, dC, ldc, M * ldc)
    done()
    got = dC.cpu().view(G, M, ldc)
    assert torch.equal(got[:, :, N:].contiguous().view(torch.int32), mark[:, :, N:].contiguous().view(torch.int32))
    for g in range(G):
        lo, hi = int(offs[g]), int(offs[g + 1])
        at = torch.arange(lo, hi) if ra is None else torch.from_numpy(ra[lo:hi]).long()
        bt = torch.arange(lo, hi) if rb is None else torch.from_numpy(rb[lo:hi]).long()
        x = torch.where(((at >= 0) & (at < na))[:, None], a[at.clamp(0, na - 1), :M].double(), 0.0)
        y = b[bt, :N].double()
        ref = alpha * (x.t() @ y) + (beta * c0[g, :, :N].double() if beta else 0)
        mag = abs(alpha) * (x.abs().t() @ y.abs()) + (abs(beta) * c0[g, :, :N].double().abs() if beta else 0)
        out = got[g, :, :N].double()
        if vals == "int4":
            assert torch.equal(out, ref), (g, hi - lo)
        assert ((out - ref).abs() <= TOL * mag).all(), (g, hi - lo)


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("G,R,M,N", [(1, 1, 1, 1), (3, 5, 7, 9), (2, 64, 64, 64), (4, 129, 65, 72), (5, 300, 130, 200), (8, 40, 256, 128),
                                     (3, 700, 264, 328), (16, 1000, 128, 256), (70, 500, 32, 96), (2, 1100, 520, 512)])
def test_wgrad(t, G, R, M, N):
    wgrad_check(t, G, R, M, N, vals="int4")
    wgrad_check(t, G, R, M, N, ga=False, gb=True, how="even", alpha=1.5, beta=-0.5)


@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_wgrad_layouts(t):
    wgrad_check(t, 4, 390, 192, 320, how="one", vals="int4", beta=1.0)
    wgrad_check(t, 3, 200, 128, 256, pads=(2, 4, 1), vals="int4")
    wgrad_check(t, 3, 200, 127, 255, pads=(1, 2, 3), vals="int4")
    wgrad_check(t, 3, 200, 128, 256, offset=1, vals="int4")
    wgrad_check(t, 3, 200, 128, 256, offset=2, pads=(8, 8, 4))
    wgrad_check(t, 3, 200, 128, 256, bad=True, vals="int4")
    wgrad_check(t, 3, 200, 128, 256, ga=False, gb=False, vals="int4")
    wgrad_check(t, 2, 3000, 512, 768, gb=True)
    wgrad_check(t, 40, 900, 509, 515, gb=True, vals="int4")                             # odd sizes, many tiles
    wgrad_check(t, 40, 900, 509, 515, bad=True, beta=1.0)


def test_wgrad_without_rows():
    c = torch.randn(2, 5, 6)
    for beta in (0.0, 2.0):
        C = c.cuda()
        dg.gemm_grouped_wgrad_f16_f32acc(2, 0, 5, 6, 1.0, None, 0, 5, None, None, 0, 6, None, None, beta, C, 6, 30)
        done()
        assert torch.equal(C.cpu(), c * beta)


# ------------------------------------------------------------------ combining
@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (3, 2, 5), (17, 4, 128), (65, 8, 1030), (9, 32, 2048), (200, 6, 515)])
@pytest.mark.parametrize("beta", [0.0, -0.5])
def test_combine_and_grad(T, k, N, beta):
    rng = rng_of("combine", T, k, N, beta)
    R, ldy, ldc = T * k + 3, N + 1, N + 2
    Y = torch.from_numpy(rng.standard_normal((R, ldy)).astype(np.float32))
    Y[:, N:] = math.nan
    slots = torch.from_numpy(rng.permutation(R)[: T * k].astype(np.int32)).view(T, k)
    if T > 2:
        slots[1] = -1
        slots[2, 0] = R
    w = torch.from_numpy(rng.random((T, k)).astype(np.float32))
    w[slots < 0] = math.nan                     # the weight of a skipped slot is not used
    c0 = torch.from_numpy(rng.standard_normal((T, ldc)).astype(np.float32))
    ok = (slots >= 0) & (slots < R)
    y = torch.where(ok[:, :, None], Y[slots.long().clamp(0, R - 1), :N], torch.zeros(())).double()
    for weights in (w, None):
        C = c0.clone() if beta else torch.full((T, ldc), math.nan)
        mark, dC = C.clone(), C.cuda()
        dg.moe_combine_f32(T, k, N, Y.cuda(), R, ldy, slots.cuda(), None if weights is None else weights.cuda(), beta, dC, ldc)
        done()
        got = dC.cpu()
        wd = torch.where(ok, (torch.ones(T, k) if weights is None else weights).double(), 0.0)
        ref = (wd[:, :, None] * y).sum(1) + (beta * c0[:, :N].double() if beta else 0)
        mag = (wd[:, :, None] * y).abs().sum(1) + (abs(beta) * c0[:, :N].double().abs() if beta else 0)
        assert torch.equal(got[:, N:].contiguous().view(torch.int32), mark[:, N:].contiguous().view(torch.int32))
        assert ((got[:, :N].double() - ref).abs() <= (k + 2) * U * mag).all()
        if beta:
            continue
        for t, fn in (("f16", dg.moe_combine_grad_f16), ("bf16", dg.moe_combine_grad_bf16)):
            g = c0
            dY = torch.full((R, ldc), 9.0, dtype=DT[t], device="cuda")
            dw = torch.full((T, k), math.nan, device="cuda")
            fn(T, k, N, g.cuda(), ldc, Y.cuda(), R, ldy, slots.cuda(), None if weights is None else weights.cuda(), dY, ldc, dw)
            done()
            want = torch.full((R, ldc), 9.0, dtype=torch.float64)
            gd = g[:, :N].double()
            for i in range(T):
                for j in range(k):
                    if ok[i, j]:
                        want[slots[i, j].long(), :N] = wd[i, j] * gd[i]
            step = torch.finfo(DT[t]).eps / 2
            tiny = 2.0 ** -25 if t == "f16" else 2.0 ** -134
            assert ((dY.cpu().double() - want).abs() <= (step * (1 + U) + U) * want.abs() + tiny).all()
            terms = gd[:, None, :] * y
            assert ((dw.cpu().double() - terms.sum(2)).abs() <= (4 * math.ceil(N / 1024) + 12) * U * terms.abs().sum(2)).all()


# ------------------------------------------------------------------ adapters
def lora_check(t, transB, M, N, K, rank, n, *, alpha=1.0, beta=0.0, vals="pm1", ids=None, ranks=True, scales=True, pads=(0, 0, 0, 0, 0),
               offset=0, runs=1):
    rng = rng_of("lora", t, transB, M, N, K, rank, n, alpha, beta, vals, pads, offset, runs)
    print(f"[lora] {t} transB={transB} M={M} N={N} K={K} rank={rank} n={n} beta={beta} {vals} pads={pads} off={offset} runs={runs}", flush=True)
    lda, ldb, ldc, ldla, ldlb = K + pads[0], (K if transB else N) + pads[1], N + pads[2], K + pads[3], rank + pads[4]
    a = torch.from_numpy(values(rng, (M, lda), vals)).to(DT[t])
    b = torch.from_numpy(values(rng, (N if transB else K, ldb), vals)).to(DT[t])
    la = torch.from_numpy(values(rng, (n, rank, ldla), vals)).to(DT[t])
    lb = torch.from_numpy(values(rng, (n, N, ldlb), vals)).to(DT[t])
    if ids is None:
        ids = np.repeat(rng.integers(-1, n + 1, M // runs + 1), runs)[:M]
    ids = torch.from_numpy(np.asarray(ids, dtype=np.int32))
    rk = torch.from_numpy(rng.integers(0, rank + 1, n).astype(np.int32)) if ranks else torch.full((n,), rank, dtype=I32)
    if ranks and n > 2:
        rk[0], rk[1] = rank + 5, -3             # clamped
    r_in = rk.clone()
    rk = rk.clamp(0, rank)
    sc = torch.from_numpy((rng.integers(1, 4, n) if vals == "int4" else rng.random(n) + 0.5).astype(np.float32))
    a[:, K:] = math.nan
    b[:, (K if transB else N):] = math.nan
    la[:, :, K:] = math.nan
    lb[:, :, rank:] = math.nan
    for i in range(n):                          # what lies past an adapter's rank
        la[i, rk[i]:] = math.nan
        lb[i, :, rk[i]:] = math.inf
    c0 = torch.from_numpy(values(rng, (M, ldc), vals))
    put = lambda x: torch.cat([torch.zeros(offset, dtype=x.dtype), x.reshape(-1)]).cuda()[offset:]  # noqa: E731
    C = c0.clone() if beta != 0 else torch.full((M, ldc), math.nan)
    mark, dC = C.clone(), put(C)
    fn = dg.gemm_lora_f16_f32acc_ex if t == "f16" else dg.gemm_lora_bf16_f32acc_ex
    fn(transB, M, N, K, rank, n, alpha, put(a), lda, put(b), ldb, put(la), ldla, rank * ldla, put(lb), ldlb, N * ldlb,
       sc.cuda() if scales else None, r_in.cuda() if ranks else None, ids.cuda(), beta, dC, ldc)
    done()
    got = dC.cpu().view(M, ldc)
    assert torch.equal(got[:, N:].contiguous().view(torch.int32), mark[:, N:].contiguous().view(torch.int32))
    x = a[:, :K].double()
    w = b[:, :K].double().t() if transB else b[:, :N].double()
    ref, mag = x @ w, x.abs() @ w.abs()
    for i in range(n):
        at = (ids == i).nonzero()[:, 0]
        if len(at) == 0 or rk[i] == 0:
            continue
        s = float(sc[i]) if scales else 1.0
        p, q = la[i, : rk[i], :K].double(), lb[i, :, : rk[i]].double()
        ref[at] += s * ((x[at] @ p.t()) @ q.t())
        mag[at] += s * ((x[at].abs() @ p.abs().t()) @ q.abs().t())
    ref, mag = alpha * ref, abs(alpha) * mag
    if beta:
        ref, mag = ref + beta * c0[:, :N].double(), mag + abs(beta) * c0[:, :N].double().abs()
    out = got[:, :N].double()
    if vals == "int4":
        assert torch.equal(out, ref)
    assert ((out - ref).abs() <= TOL * mag).all(), float(((out - ref).abs() / mag.clamp(min=1e-30)).max())


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("transB", [0, 1])
@pytest.mark.parametrize("M,N,K,rank,n", [(1, 1, 1, 1, 1), (1, 256, 512, 16, 3), (3, 7, 9, 5, 2), (16, 128, 256, 8, 4), (17, 200, 328, 32, 9),
                                          (48, 264, 520, 64, 20), (64, 512, 1024, 16, 70), (65, 130, 72, 128, 3), (130, 256, 264, 24, 5),
                                          (300, 520, 520, 100, 4)])
def test_lora(t, transB, M, N, K, rank, n):
    lora_check(t, transB, M, N, K, rank, n)
    lora_check(t, transB, M, N, K, rank, n, alpha=1.5, beta=-0.5, ranks=False, scales=False)
    lora_check(t, transB, M, N, K, rank, n, vals="int4", runs=13)


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("transB", [0, 1])
@pytest.mark.parametrize("M", [5, 40, 200])
def test_lora_layouts(t, transB, M):
    lora_check(t, transB, M, 128, 256, 16, 4, ids=np.full(M, -1))                  # no row has an adapter
    lora_check(t, transB, M, 128, 256, 16, 4, ids=np.full(M, 2), vals="int4")      # all rows the same one
    lora_check(t, transB, M, 128, 256, 16, M, ids=np.arange(M)[::-1], vals="int4") # every row its own
    lora_check(t, transB, M, 128, 256, 16, 4, pads=(2, 4, 1, 2, 2), vals="int4")
    lora_check(t, transB, M, 127, 255, 15, 4, pads=(1, 2, 3, 1, 2), vals="int4")
    lora_check(t, transB, M, 128, 256, 16, 4, offset=1, vals="int4")
    lora_check(t, transB, M, 136, 264, 8, 4, offset=2, pads=(8, 8, 4, 8, 8), beta=1.0)
    lora_check(t, transB, M, 1024, 2048, 16, 4, runs=7)


@pytest.mark.parametrize("M,N,K", [(1, 64, 8192), (16, 64, 16384), (48, 100, 8200), (33, 512, 7936), (5, 63, 8191)])
def test_lora_few_columns_long_k(M, N, K):
    lora_check("f16", 1, M, N, K, 8, 3, beta=0.5)
    lora_check("bf16", 0, M, N, K, 8, 3, vals="int4")


@pytest.mark.parametrize("transB", [0, 1])
def test_lora_more_rows_than_a_grid_s_second_axis(transB):
    """More than 65535 rows where the narrow product is joined by a block a row."""
    lora_check("f16", transB, 70001, 9, 15, 3, 2, beta=0.5)
    lora_check("bf16", transB, 131200, 7, 9, 2, 5, vals="int4", runs=100)


@pytest.mark.parametrize("M", [2, 100])
def test_lora_narrow_product_outside_16_bits(M):
    """The narrow product reaches 2^20 and 2^-30, outside fp16; the result does not."""
    K, N, r = 64, 72, 4
    for e in (10, -15):
        a = torch.full((M, K), 2.0 ** e, dtype=torch.float16, device="cuda")
        la = torch.full((1, r, K), 2.0 ** e, dtype=torch.float16, device="cuda")
        lb = torch.full((1, N, r), 1.0 / 64, dtype=torch.float16, device="cuda")
        b = torch.zeros(N, K, dtype=torch.float16, device="cuda")
        C = torch.empty(M, N, device="cuda")
        dg.gemm_lora_f16_f32acc_ex(1, M, N, K, r, 1, 1.0, a, K, b, K, la, K, r * K, lb, r, N * r, None, None,
                                   torch.zeros(M, dtype=I32, device="cuda"), 0.0, C, N)
        done()
        assert torch.equal(C.cpu(), torch.full((M, N), K * 2.0 ** (2 * e) * r / 64))


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("M", [40, 100, 300])
@pytest.mark.parametrize("rank", [5, 16, 40])
def test_lora_narrow_product_keeps_its_bits(t, M, rank):
    """LB takes one column of the narrow product at a time, so that C shows each of its values as it is held.  They are
    sums of two products, x la below 2 and another 2^-2 (bf16: 2^-9) of such, with 24 bits in all, times 2^0 to 2^-26: the
    result is exact, for few rows and for many."""
    K, N = 128, 72
    rng = rng_of("bits", t, M, rank)
    bits, step = (10, 2.0 ** -2) if t == "f16" else (7, 2.0 ** -9)
    some = lambda *n: (1 + rng.integers(0, int(0.4 * 2 ** bits), n) / 2.0 ** bits).astype(np.float32)  # noqa: E731
    e = np.linspace(0, -26, rank).round().astype(int)
    down = np.maximum(e, -12)                               # LA's part of 2^e, A's is the rest: normal fp16 values both
    a, w = np.zeros((M, K), dtype=np.float32), np.zeros((1, rank, K), dtype=np.float32)
    for j in range(rank):
        up = np.float32(2.0 ** (e[j] - down[j]))
        a[:, j], a[:, rank + j] = some(M) * up, some(M) * up
        w[0, j, j], w[0, j, rank + j] = some(1)[0] * 2.0 ** down[j], some(1)[0] * 2.0 ** down[j] * step
    lb = np.zeros((1, N, rank), dtype=np.float32)
    lb[0, np.arange(rank), np.arange(rank)] = 1
    b = np.zeros((N, K), dtype=np.float32)
    mk = lambda v: torch.from_numpy(v).to(DT[t])  # noqa: E731
    for v in (a, w):
        assert torch.equal(mk(v).float(), torch.from_numpy(v))
    C = torch.full((M, N), math.nan, device="cuda")
    getattr(dg, f"gemm_lora_{t}_f32acc_ex")(1, M, N, K, rank, 1, 1.0, mk(a).cuda(), K, mk(b).cuda(), K, mk(w).cuda(), K, rank * K,
                                            mk(lb).cuda(), rank, N * rank, None, None, torch.zeros(M, dtype=I32, device="cuda"), 0.0, C, N)
    done()
    want = np.zeros((M, N))
    want[:, :rank] = a.astype(np.float64) @ w[0].astype(np.float64).T
    assert np.array_equal(want.astype(np.float32), want)
    assert np.array_equal(host(C), want), np.abs(host(C) / np.where(want == 0, 1, want) - (want != 0)).max()


@pytest.mark.parametrize("M", [3, 40, 200])
@pytest.mark.parametrize("K", [256, 255])
def test_lora_rows_keep_apart(M, K):
    """An adapter, or a row, that holds infinities and NaN reaches no other request's row."""
    N, r, n = 136, 16, 3
    g = torch.Generator().manual_seed(M)
    mk = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    a, b, la, lb = mk(M, K), mk(N, K), mk(n, r, K), mk(n, N, r)
    ids = (torch.arange(M) % n).to(I32).cuda()

    def run():
        C = torch.empty(M, N, device="cuda")
        dg.gemm_lora_bf16_f32acc_ex(1, M, N, K, r, n, 1.0, a, K, b, K, la, K, r * K, lb, r, N * r, None, None, ids, 0.0, C, N)
        done()
        return C

    want = run()
    lb[1] = math.inf
    la[1, 3:] = math.nan
    got = run()
    own = ids == 1
    assert torch.isnan(got[own]).all() and torch.equal(got[~own], want[~own])
    a[0] = math.nan
    again = run()
    assert torch.isnan(again[0]).all() and torch.equal(again[2::3], want[2::3]) and torch.equal(again[3::3], want[3::3])


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("M", [3, 40, 100])
@pytest.mark.parametrize("rank,used", [(16, 16), (16, 5), (40, 17)])
@pytest.mark.parametrize("K", [256, 255])
def test_lora_infinite_row_of_a(t, M, rank, used, K):
    """A row of A that holds an infinity: the product and the narrow product are infinite with the signs of the weights it
    meets, whatever lies past the adapter's rank, and a finite value of the narrow product stays finite."""
    N, n = 72, 2
    a = torch.ones(M, K, dtype=DT[t])
    a[1::3, 0] = math.inf
    b = torch.ones(N, K, dtype=DT[t])
    b[N // 2 :] = -1                                        # these columns of the product are -inf
    la = torch.zeros(n, rank, K, dtype=DT[t])
    la[:, 0, 0] = 2                                         # t_0 = inf, or 2
    la[:, 1, 0], la[:, 1, 1:] = 1, -1024
    lb = torch.zeros(n, N, rank, dtype=DT[t])
    lb[:, : N // 2, 0] = 1
    lb[:, N // 2 :, 0] = -1
    la[:, used:], lb[:, :, used:] = math.nan, math.inf
    la[:, 2:used] = 1
    lb[:, :, 2:used] = 0.5
    lb[:, N // 2 :, 2:used] = -0.5
    ids = (torch.arange(M) % n).to(I32)
    lb[:, : N // 2, 1], lb[:, N // 2 :, 1] = 1, -1          # (t is +inf throughout, LB has the product's signs)
    C = torch.full((M, N), math.nan, device="cuda")
    getattr(dg, f"gemm_lora_{t}_f32acc_ex")(1, M, N, K, rank, n, 1.0, a.cuda(), K, b.cuda(), K, la.cuda(), K, rank * K, lb.cuda(), rank,
                                            N * rank, None, torch.full((n,), used, dtype=I32, device="cuda"), ids.cuda(), 0.0, C, N)
    done()
    got = C.cpu()
    assert (got[1::3, : N // 2] == math.inf).all() and (got[1::3, N // 2 :] == -math.inf).all()
    rest = torch.ones(M, dtype=torch.bool)
    rest[1::3] = False
    assert torch.isfinite(got[rest]).all()


@pytest.mark.parametrize("M", [3, 40, 100])
def test_lora_infinity_beside_a_large_narrow_product(M):
    """A narrow product that is +inf in one column and, in another, finite, past fp16's largest and of the other sign."""
    N, K, rank = 72, 256, 16
    a = torch.ones(M, K, dtype=torch.float16)
    b = torch.zeros(N, K, dtype=torch.float16)
    la = torch.zeros(1, rank, K, dtype=torch.float16)
    la[:, 0, 0] = math.inf
    la[:, 1] = -1024                                        # t_1 = -2^18
    lb = torch.zeros(1, N, rank, dtype=torch.float16)
    lb[:, :, 0] = 1
    lb[:, :, 1] = 1
    C = torch.full((M, N), math.nan, device="cuda")
    dg.gemm_lora_f16_f32acc_ex(1, M, N, K, rank, 1, 1.0, a.cuda(), K, b.cuda(), K, la.cuda(), K, rank * K, lb.cuda(), rank, N * rank, None, None,
                               torch.zeros(M, dtype=I32, device="cuda"), 0.0, C, N)
    done()
    assert (C == math.inf).all()


@pytest.mark.parametrize("M", [5, 100])
def test_lora_without_adapters(M):
    a, b, C = torch.ones(M, 64, dtype=torch.float16, device="cuda"), torch.ones(72, 64, dtype=torch.float16, device="cuda"), torch.ones(M, 72, device="cuda")
    dg.gemm_lora_f16_f32acc_ex(1, M, 72, 64, 4, 0, 0.5, a, 64, b, 64, None, 64, 0, None, 4, 0, None, None, None, 2.0, C, 72)
    done()
    assert (C == 34).all()


def test_offsets_past_32_bits():
    """Rows a few MB apart, so that operands and results span more than 4 GiB each."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB of device memory")
    far, M, K, N, G = (1 << 20) + 8, 2200, 128, 64, 3
    g = torch.Generator().manual_seed(1)
    A = torch.empty(M * far, dtype=torch.bfloat16, device="cuda").view(M, far)
    A[:, :K] = torch.randint(-3, 4, (M, K), generator=g).to(torch.bfloat16)
    a = A[:, :K].double()
    off = torch.tensor([0, 700, 1500, M], dtype=I32, device="cuda")
    rows = torch.randperm(M, generator=g).to(I32).cuda()
    B = torch.empty(G << 30, dtype=torch.bfloat16, device="cuda")
    w = torch.randint(-3, 4, (G, K, N), generator=g).to(torch.bfloat16).cuda()
    for i in range(G):
        B[i << 30 : (i << 30) + K * N] = w[i].reshape(-1)
    C = torch.empty(M * far, device="cuda").view(M, far)
    dg.gemm_grouped_bf16_f32acc_ex(0, G, M, N, K, 1.0, A, M, far, rows, B, N, 1 << 30, off, 0.0, C, far)
    done()
    pick = a[rows.long()]
    want = torch.cat([pick[lo:hi] @ w[i].double() for i, (lo, hi) in enumerate(((0, 700), (700, 1500), (1500, M)))])
    assert torch.equal(C[:, :N].double(), want)
    # a group's few rows, streamed
    few = torch.tensor([0, 2, 2, 5], dtype=I32, device="cuda")
    C[:8, :N] = -1
    dg.gemm_grouped_bf16_f32acc_ex(0, G, 5, N, K, 1.0, A, M, far, rows, B, N, 1 << 30, few, 0.0, C, far)
    done()
    assert torch.equal(C[:5, :N].double(), torch.cat([pick[:2] @ w[0].double(), pick[2:5] @ w[2].double()]))
    D = torch.empty(G << 30, device="cuda")
    y = torch.randint(-3, 4, (M, N), generator=g).to(torch.bfloat16).cuda()
    dg.gemm_grouped_wgrad_bf16_f32acc(G, M, K, N, 1.0, A, M, far, rows, y, M, N, None, off, 0.0, D, N, 1 << 30)
    done()
    for i, (lo, hi) in enumerate(((0, 700), (700, 1500), (1500, M))):
        assert torch.equal(D[i << 30 : (i << 30) + K * N].view(K, N).double(), pick[lo:hi].t() @ y[lo:hi].double())
    del D, B
    slots = torch.randperm(M, generator=g)[: 1100 * 2].view(1100, 2).to(I32).cuda()
    out = torch.empty(1100, N, device="cuda")
    C[:, :N] = torch.randint(-3, 4, (M, N), generator=g).float()
    dg.moe_combine_f32(1100, 2, N, C, M, far, slots, None, 0.0, out, N)
    done()
    assert torch.equal(out, C[slots[:, 0].long(), :N] + C[slots[:, 1].long(), :N])


def test_results_larger_than_the_caches():
    """C of more than 192 MiB, whose whole tiles are stored past the caches: every element."""
    g = torch.Generator(device="cuda").manual_seed(5)
    ints = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").to(torch.float16)  # noqa: E731
    G, R, N, K = 3, 49300, 1032, 72
    a, b = ints(R, K), ints(G, K, N)
    off = torch.tensor([0, 20001, 20001, R], dtype=I32, device="cuda")
    C = torch.full((R, N), math.nan, device="cuda")
    dg.gemm_grouped_f16_f32acc_ex(0, G, R, N, K, 2.0, a, R, K, None, b, N, K * N, off, 0.0, C, N)
    done()
    assert torch.equal(C[:20001], 2 * (a[:20001].float() @ b[0].float()))
    assert torch.equal(C[20001:], 2 * (a[20001:].float() @ b[2].float()))
    del C
    G, R, M, N = 13, 300, 2048, 2040
    x, y = ints(R, M), ints(R, N)
    off = torch.linspace(0, R, G + 1).to(I32).cuda()
    D = torch.full((G, M, N), math.nan, device="cuda")
    dg.gemm_grouped_wgrad_f16_f32acc(G, R, M, N, 1.0, x, R, M, None, y, R, N, None, off, 0.0, D, N, M * N)
    done()
    at = off.tolist()
    for i in range(G):
        assert torch.equal(D[i], x[at[i] : at[i + 1]].float().t() @ y[at[i] : at[i + 1]].float())


@pytest.mark.parametrize("N,K", [(16392, 72), (16391, 71)])
def test_grouped_result_past_2_to_32_elements(N, K):
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB of device memory")
    g = torch.Generator(device="cuda").manual_seed(6)
    ints = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    G, R = 3, (1 << 18) + 77
    a, b = ints(R, K), ints(G, K, N)
    off = [0, 100001, 100001, R]
    C = torch.full((R, N), math.nan, device="cuda")
    dg.gemm_grouped_bf16_f32acc_ex(0, G, R, N, K, 1.0, a, R, K, None, b, N, K * N, torch.tensor(off, dtype=I32).cuda(), 0.0, C, N)
    done()
    for i in range(G):
        for lo in range(off[i], off[i + 1], 1 << 14):
            hi = min(lo + (1 << 14), off[i + 1])
            assert torch.equal(C[lo:hi], a[lo:hi].float() @ b[i].float())


@pytest.mark.parametrize("M,N,K,transB", [(16384, 131072, 64, 1), (16385, 131071, 63, 0)])
def test_lora_result_past_2_to_31_elements(M, N, K, transB):
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB of device memory")
    g = torch.Generator(device="cuda").manual_seed(7)
    ints = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").half()  # noqa: E731
    r, n = 4, 3
    a, b, la, lb = ints(M, K), ints(*((N, K) if transB else (K, N))), ints(n, r, K), ints(n, N, r)
    ids = (torch.arange(M, device="cuda") // 1000 % (n + 1)).to(I32)
    C = torch.full((M, N), math.nan, device="cuda")
    dg.gemm_lora_f16_f32acc_ex(transB, M, N, K, r, n, 1.0, a, K, b, K if transB else N, la, K, r * K, lb, r, N * r, None, None, ids, 0.0, C, N)
    done()
    w = (b.t() if transB else b).float()
    for lo in range(0, M, 1000):
        rows, i = a[lo : lo + 1000].float(), int(ids[lo])
        want = rows @ w
        if i < n:
            want += (rows @ la[i].float().t()) @ lb[i].float().t()
        assert torch.equal(C[lo : lo + 1000], want)


def test_lora_no_product():
    c = torch.randn(5, 6)
    nan = torch.full((64,), math.nan, dtype=torch.float16, device="cuda")
    ids = torch.zeros(5, dtype=I32, device="cuda")
    for K, alpha in ((0, 1.0), (5, 0.0)):
        for beta in (0.0, 2.0):
            C = c.cuda()
            dg.gemm_lora_f16_f32acc_ex(0, 5, 6, K, 2, 1, alpha, nan, max(K, 1), nan, 6, nan, max(K, 1), 10, nan, 2, 12, None, None, ids, beta, C, 6)
            done()
            assert torch.equal(C.cpu(), c * beta)


# ------------------------------------------------------------------ together
class Layer:
    """One expert layer, T tokens of width D through E experts of width F and back, forward and backward."""

    def __init__(self, T, D, F, E, k, t="bf16", seed=3):
        g = torch.Generator().manual_seed(seed)
        self.T, self.D, self.F, self.E, self.k, self.t = T, D, F, E, k, t
        n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.x, self.logits = n(T, D).to(DT[t]).cuda(), n(T, E).cuda()
        self.w1, self.w2 = (n(E, D, F) / D ** 0.5).to(DT[t]).cuda(), (n(E, F, D) / F ** 0.5).to(DT[t]).cuda()
        R = T * k
        e = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
        self.ids, self.w, self.off, self.rows, self.slots = e(T, k, dt=I32), e(T, k), e(E + 1, dt=I32), e(R, dt=I32), e(T, k, dt=I32)
        self.h, self.y, self.out = e(R, F), e(R, D), e(T, D)
        self.h16 = e(R, F, dt=DT[t])
        self.grouped = getattr(dg, f"gemm_grouped_{t}_f32acc_ex")
        self.wgrad = getattr(dg, f"gemm_grouped_wgrad_{t}_f32acc")

    def forward(self):
        T, D, F, E, k, R = self.T, self.D, self.F, self.E, self.k, self.T * self.k
        dg.moe_route_f32(T, E, self.logits, E, None, 0, 1, 1, 1, k, 1, 1.0, self.ids, self.w, self.off, self.rows, self.slots)
        self.grouped(0, E, R, F, D, 1.0, self.x, T, D, self.rows, self.w1, F, D * F, self.off, 0.0, self.h, F)
        self.h16.copy_(torch.relu(self.h))
        self.grouped(0, E, R, D, F, 1.0, self.h16, R, F, None, self.w2, D, D * F, self.off, 0.0, self.y, D)
        dg.moe_combine_f32(T, k, D, self.y, R, D, self.slots, self.w, 0.0, self.out, D)

    def backward(self, dout):
        T, D, F, E, k, R, dt = self.T, self.D, self.F, self.E, self.k, self.T * self.k, DT[self.t]
        e = lambda *s, d=torch.float32: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
        dy, dw, dl = e(R, D, d=dt), e(T, k), e(T, E)
        getattr(dg, f"moe_combine_grad_{self.t}")(T, k, D, dout, D, self.y, R, D, self.slots, self.w, dy, D, dw)
        dg.moe_route_f32_grad(T, E, self.logits, E, 0, k, 1, 1.0, self.ids, dw, dl, E)
        dw2, dw1, dh, dxr, dx = e(E, F, D), e(E, D, F), e(R, F), e(R, D), e(T, D)
        self.wgrad(E, R, F, D, 1.0, self.h16, R, F, None, dy, R, D, None, self.off, 0.0, dw2, D, F * D)
        self.grouped(1, E, R, F, D, 1.0, dy, R, D, None, self.w2, D, D * F, self.off, 0.0, dh, F)
        dh16 = torch.where(self.h > 0, dh, 0.0).to(dt)
        self.wgrad(E, R, D, F, 1.0, self.x, T, D, self.rows, dh16, R, F, None, self.off, 0.0, dw1, F, D * F)
        self.grouped(1, E, R, D, F, 1.0, dh16, R, F, None, self.w1, F, D * F, self.off, 0.0, dxr, D)
        dg.moe_combine_f32(T, k, D, dxr, R, D, self.slots, None, 0.0, dx, D)
        return dl, dw1, dw2, dx

    def dense(self, dout):
        """All of it in 64 bits by torch's own differentiation, for the ids chosen."""
        x, lg, w1, w2 = (v.cpu().double().requires_grad_(True) for v in (self.x, self.logits, self.w1, self.w2))
        ids = self.ids.cpu().long()
        assert torch.equal(ids, lg.detach().sort(dim=1, descending=True, stable=True).indices[:, : self.k])
        w = torch.softmax(torch.gather(lg, 1, ids), 1)
        out = torch.zeros(self.T, self.D, dtype=torch.float64)
        for e in range(self.E):
            at, j = (ids == e).nonzero(as_tuple=True)
            out = out.index_add(0, at, w[at, j][:, None] * (torch.relu(x[at] @ w1[e]) @ w2[e]))
        (out * dout.cpu().double()).sum().backward()
        return out.detach(), (lg.grad, w1.grad, w2.grad, x.grad)


@pytest.mark.parametrize("T,D,F,E,k,t", [(1, 64, 32, 4, 2, "bf16"), (37, 128, 200, 8, 3, "f16"), (300, 256, 136, 16, 4, "bf16")])
def test_expert_layer(T, D, F, E, k, t):
    layer = Layer(T, D, F, E, k, t)
    layer.forward()
    dout = torch.randn(T, D, generator=torch.Generator().manual_seed(9)).cuda()
    grads = layer.backward(dout)
    done()
    out, want = layer.dense(dout)
    # the activations and their gradients pass through 16 bits once each: half a step, of every term
    step = torch.finfo(DT[t]).eps / 2
    for got, ref in ((layer.out, out), *zip(grads, want)):
        # two such roundings in a row at most (dy, then dh), and a difference of two such values (the router's gradient)
        assert (got.cpu().double() - ref).norm() <= 4 * step * ref.norm() + 1e-30


def test_captured_layer_replays():
    layer = Layer(50, 128, 96, 8, 2)
    layer.forward()
    done()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward()
    for seed in range(4):
        g = torch.Generator().manual_seed(seed)
        layer.logits.copy_(torch.randn(50, 8, generator=g))
        layer.x.copy_(torch.randn(50, 128, generator=g).to(torch.bfloat16))
        layer.out.fill_(math.nan)
        graph.replay()
        done()
        got = layer.out.clone()
        layer.forward()
        done()
        assert torch.equal(got, layer.out), seed


@pytest.mark.parametrize("M", [7, 150])
def test_captured_lora_and_long_route_replay(M):
    K, N, r, n = 256, 320, 16, 5
    g = torch.Generator().manual_seed(1)
    mk = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    a, b, la, lb = mk(M, K), mk(N, K), mk(n, r, K), mk(n, N, r)
    ids = torch.randint(-1, n, (M,), generator=g).to(I32).cuda()
    x = torch.randn(700, 32, generator=g).cuda()
    C = torch.zeros(M, N, device="cuda")
    out = {}

    def work():
        dg.gemm_lora_bf16_f32acc_ex(1, M, N, K, r, n, 1.0, a, K, b, K, la, K, r * K, lb, r, N * r, None, None, ids, 0.0, C, N)
        out.update(route_call(x, 32, None, 1, 1, 1, 1, 4, 1, 1.0, 700, 32))

    work()
    done()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    held = dict(out)
    for seed in range(4):
        g = torch.Generator().manual_seed(seed)
        a.copy_(torch.randn(M, K, generator=g).to(torch.bfloat16))
        ids.copy_(torch.randint(-1, n, (M,), generator=g).to(I32))
        x.copy_(torch.randn(700, 32, generator=g))
        graph.replay()
        done()
        got, lay = C.clone(), {m: v.clone() for m, v in held.items()}
        work()
        done()
        assert torch.equal(got, C)
        assert all(torch.equal(lay[m], out[m]) for m in lay)


def test_other_streams_and_repeats():
    """Calls on two streams at once, each with its own workspace, give what one call gives."""
    x = torch.randn(3000, 64, generator=torch.Generator().manual_seed(2)).cuda()
    one = route_call(x, 64, None, 1, 1, 1, 1, 6, 1, 1.0, 3000, 64)
    M, K, N, r, n = 90, 512, 256, 8, 6
    mk = lambda *s: torch.randn(*s, generator=torch.Generator().manual_seed(4)).half().cuda()  # noqa: E731
    a, b, la, lb = mk(M, K), mk(N, K), mk(n, r, K), mk(n, N, r)
    ids = (torch.arange(M) % n).to(I32).cuda()
    Cs = [torch.zeros(M, N, device="cuda") for _ in range(5)]

    def lora(C, stream=None):
        dg.gemm_lora_f16_f32acc_ex(1, M, N, K, r, n, 1.0, a, K, b, K, la, K, r * K, lb, r, N * r, None, None, ids, 0.0, C, N, stream=stream)

    lora(Cs[0])
    done()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(4):
        s = streams[i % 2]
        got.append(route_call(x, 64, None, 1, 1, 1, 1, 6, 1, 1.0, 3000, 64, stream=s if i < 2 else s.cuda_stream))
        lora(Cs[1 + i], s)
    done()
    for o in got:
        assert all(torch.equal(o[m], one[m]) for m in one)
    for C in Cs[1:]:
        assert torch.equal(C, Cs[0])


def test_workspace_argument():
    x = torch.randn(200, 16).cuda()
    need = dg.moe_route_workspace(200, 16, 2)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    o = [torch.zeros(n, dtype=d, device="cuda") for n, d in ((400, I32), (400, torch.float32), (17, I32), (400, I32), (400, I32))]
    dg.moe_route_f32(200, 16, x, 16, None, 0, 1, 1, 1, 2, 1, 1.0, *o, workspace=ws)
    done()
    assert int(o[2][16]) == 400
    with pytest.raises(dg.GemmError) as e:
        dg.moe_route_f32(200, 16, x, 16, None, 0, 1, 1, 1, 2, 1, 1.0, *o, workspace=ws[: need - 4].clone())
    assert e.value.status == -7
    with pytest.raises(ValueError):   # the storage holds fewer elements than the call reads
        dg.moe_route_f32(201, 16, x, 16, None, 0, 1, 1, 1, 2, 1, 1.0, *o)
    with pytest.raises(ValueError):   # an index array with strides
        dg.moe_combine_f32(100, 2, 4, torch.zeros(400, 4, device="cuda"), 400, 4, o[4].view(200, 2)[:, :1], None, 0.0,
                           torch.zeros(100, 4, device="cuda"), 4)
    with pytest.raises(TypeError):
        dg.moe_combine_f32(100, 2, 4, torch.zeros(400, 4, device="cuda"), 400, 4, o[1], None, 0.0, torch.zeros(100, 4, device="cuda"), 4)

"""Orthogonalised updates held to the bounds that the header states, for gradients with few, unequal or nearly parallel rows (GPU).

The header's bounds on |X - ref| / |ref| (2-norm), before the result is rounded to bf16, do not come from the arithmetic of the
kernels: 5e-3 with five steps (3.4445, -4.7750, 2.0315) and 1e-3 with eight (1.875, -1.25, 0.375); 2e-2 and 2e-3 where
entries are equal.  Rounding a value to bf16 is off by at most half a step, 2^-8 of it: 2^-8 / sqrt(3) at random, whose square adds to that of
the error before it where there are some hundred entries; equal entries are rounded alike, and there 2^-8 adds to it.
"""
from __future__ import annotations

import numpy as np
import pytest

import dense_gemm_optimisation_f32_amd as dg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

STEPS = {"fast": [(3.4445, -4.7750, 2.0315)] * 5, "tight": [(1.875, -1.25, 0.375)] * 8}
BOUND = {"fast": 5e-3, "tight": 1e-3}
EQUAL = {"fast": 2e-2, "tight": 2e-3}
HALF = 2.0 ** -8   # of a bf16 value

# one workgroup a member; products in 32 x 32 tiles; in 64 x 64; in 128 x 128 and larger ones, up to 256 x 256
SIZES = [(4, 96), (16, 64), (64, 96), (64, 1024), (96, 300), (128, 512), (512, 128), (129, 127), (256, 512), (300, 500), (1001, 513),
         (1024, 1024), (1500, 2100), (4040, 4000)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dg.load_library()
    yield
    torch.cuda.synchronize()


def two_rows(rng, m, n):
    g = np.zeros((m, n))
    g[0] = rng.standard_normal(n)
    g[m // 2] = 0.7 * g[0]
    return g


def two_rows_and_noise(rng, m, n):
    return two_rows(rng, m, n) + 1e-3 * rng.standard_normal((m, n))


def weak_copy_of_a_row(rng, m, n):
    """Independent rows, and the first once more, of a twentieth of its size: hardly any off-diagonal beside a diagonal."""
    g = np.zeros((m, n))
    r = max(1, m // 4)
    g[:r] = rng.standard_normal((r, n))
    g[m - 1] = 0.05 * g[0]
    return g


def few_rows(rng, m, n):
    g = np.zeros((m, n))
    k = min(8, m)
    g[m - k:] = rng.standard_normal((k, (k + 1) // 2)) @ rng.standard_normal(((k + 1) // 2, n))
    return g


def unequal_rows(rng, m, n):
    return np.exp(2 * rng.standard_normal((m, 1))) * (rng.standard_normal((m, 2)) @ rng.standard_normal((2, n)))


def rank_one(rng, m, n):
    return np.exp(rng.standard_normal((m, 1))) * rng.standard_normal((m, 1)) * rng.standard_normal((1, n))


def unequal_everywhere(rng, m, n):
    return rank_one(rng, m, n) * np.exp(2 * rng.standard_normal((1, n)))


def one_direction_missing(rng, m, n):
    return rng.standard_normal((m, m - 1)) @ rng.standard_normal((m - 1, n))


def parallel_in_pairs(rng, m, n):
    return np.repeat(rng.standard_normal((m // 2, n)), 2, 0)[:m] * rng.uniform(0.5, 2, (2 * (m // 2), 1))[:m] if m > 1 else rng.standard_normal((m, n))


KINDS = [two_rows, two_rows_and_noise, weak_copy_of_a_row, few_rows, unequal_rows, rank_one, unequal_everywhere, one_direction_missing, parallel_in_pairs]


def gradient(kind, M, N):
    """With M <= N as its kind says, else the transpose of that."""
    rng = np.random.default_rng(list(f"{kind.__name__} {M} {N}".encode()))
    return kind(rng, M, N) if M <= N else np.ascontiguousarray(kind(rng, N, M).T)


def oracle(g, steps):
    x = g.double() if g.shape[0] <= g.shape[1] else g.double().t()
    x = x / torch.linalg.norm(x)
    for a, b, c in steps:
        s = x @ x.t()
        x = a * x + b * (s @ x) + c * (s @ (s @ x))
    return x if g.shape[0] <= g.shape[1] else x.t()


def off(G, steps, t="f32"):
    """How far each member's result is from the definition."""
    n, M, N = G.shape
    O = torch.empty(n, M, N, dtype=torch.bfloat16, device="cuda")
    getattr(dg, f"orthogonalise_{t}")(M, N, steps, 1.0, G, N, M * N, O, N, M * N, n)
    refs = [oracle(g, steps) for g in G]
    return [float(torch.linalg.norm(o.double() - r) / torch.linalg.norm(r)) for o, r in zip(O, refs)]


@pytest.mark.parametrize("steps", STEPS)
@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k.__name__)
@pytest.mark.parametrize("M,N", SIZES)
def test_rows_in_few_directions(M, N, kind, steps):
    """A rounding of X is noise in all directions: what of it is outside the gradient's must not be there for the steps to grow."""
    G = torch.from_numpy(gradient(kind, M, N)).cuda().float()[None]
    got = off(G, STEPS[steps])
    assert got[0] <= np.hypot(BOUND[steps], HALF / np.sqrt(3))


@pytest.mark.parametrize("kind", [two_rows, unequal_rows, parallel_in_pairs], ids=lambda k: k.__name__)
@pytest.mark.parametrize("M,N", [(128, 512), (300, 140), (1024, 1030)])
def test_rows_in_few_directions_bf16_members(M, N, kind):
    """The same of G in bf16, several members in one call, each of another kind."""
    kinds = [kind, rank_one, kind]
    G = torch.from_numpy(np.stack([gradient(k, M, N) for k in kinds])).cuda().bfloat16()
    for steps in STEPS:
        assert max(off(G, STEPS[steps], "bf16")) <= np.hypot(BOUND[steps], HALF / np.sqrt(3))


@pytest.mark.parametrize("steps", STEPS)
@pytest.mark.parametrize("M,N", [(1, 300), (300, 1), (4, 96), (43, 43), (64, 96), (128, 512), (129, 127), (300, 500), (1024, 1024)])
def test_equal_entries(M, N, steps):
    """The identity, ones and blocks of ones: all entries of a copy are off by the same."""
    m = min(M, N)
    blocks = np.kron(np.eye(max(1, m // 3)), np.ones((3 if m > 2 else 1, 3 if m > 2 else 1)))
    filled = np.zeros((M, N))
    filled[:blocks.shape[0], :blocks.shape[1]] = blocks
    G = torch.from_numpy(np.stack([np.eye(M, N), np.ones((M, N)), filled])).cuda().float()
    assert max(off(G, STEPS[steps])) <= EQUAL[steps] + HALF


@pytest.mark.parametrize("steps", STEPS)
@pytest.mark.parametrize("M,N", [(1, 300), (16, 400), (128, 512), (300, 500), (513, 1001), (1024, 1024), (1500, 1400), (4096, 4000)])
def test_full_rank(M, N, steps):
    """Gradients without structure, and rows that are orthogonal to one another."""
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    g = torch.randn(M, N, device="cuda", generator=gen)
    kinds = [g]
    if M * N <= 1 << 19:
        q = np.linalg.qr(g.double().cpu().numpy() if M > N else g.double().cpu().numpy().T)[0]
        kinds.append(torch.from_numpy(np.ascontiguousarray(q if M > N else q.T)).cuda().float())
    assert max(off(torch.stack(kinds), STEPS[steps])) <= np.hypot(BOUND[steps], HALF / np.sqrt(3))

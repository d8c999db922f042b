"""Updates orthogonalised by Newton-Schulz products, against the definition in 64 bits (GPU).

Tolerance on |O - ref| / |ref| (2-norm over the matrix).  The products take fp16 copies: of X, and of A and B without their
diagonals, each value off by half a step at most; everything else is fp32, 2^-13 of that.  How far the copies' errors carry depends on the
singular values' way through the steps (the polynomial's slope is between -1.6 and 1.7 where they end up), so it is computed: the definition in 64
bits with these copies rounded up or down at random (each value off by up to a whole step, at random 1.4 times what rounding
to the nearest does), the largest of three such runs.  The result's rounding to bf16 is off by half a step, 2^-8 of a value, at
most, 2^-8 / sqrt(3) at random where there are 256 entries or more.  The tolerance is twice the first beside the second (the root of their squares' sum; their
sum for fewer entries).
"""
from __future__ import annotations

import numpy as np
import pytest

import dense_gemm_optimisation_f32_amd as dg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

FAST = [(3.4445, -4.7750, 2.0315)] * 5
TIGHT = [(1.875, -1.25, 0.375)] * 8
MIXED = [(3.4445, -4.7750, 2.0315), (3.0, -3.2, 1.2), (2.2, -1.7, 0.5), (1.875, -1.25, 0.375)]
HALF = 2.0 ** -8   # of a bf16 value


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dg.load_library()
    yield
    torch.cuda.synchronize()


def rng_of(*key):
    return np.random.default_rng(list(str(key).encode()))


def oracle(g, steps, alpha=1.0):
    x = g.astype(np.float64)
    n = np.linalg.norm(x)
    x = x / n if n else x
    if x.shape[0] > x.shape[1]:
        return oracle(g.T, steps, alpha).T
    for a, b, c in steps:
        s = x @ x.T
        x = a * x + (b * s + c * s @ s) @ x
    return alpha * x


def either_way(rng, x):
    """x rounded to fp16, up or down at random."""
    h = x.astype(np.float16)
    low = np.where(h.astype(np.float64) <= x, h, np.nextafter(h, np.float16(-np.inf)))
    high = np.where(h.astype(np.float64) >= x, h, np.nextafter(h, np.float16(np.inf)))
    return np.where(rng.random(x.shape) < 0.5, low, high).astype(np.float64)


def tolerance(g, steps):
    ref = oracle(g, steps)
    if g.shape[0] > g.shape[1]:
        g, ref = g.T, ref.T
    worst = 0.0
    for k in range(3):
        rng = rng_of("rounding", k)
        size = np.sqrt(g.shape[1])                           # the copies are scaled to entries near 1
        x = g.astype(np.float64) / np.linalg.norm(g) * size
        for a, b, c in steps:
            copy = either_way(rng, x)
            s = copy @ copy.T / size ** 2
            d = np.diag(s)
            o = either_way(rng, (s - np.diag(d)) * 1024) / 1024
            sq = o @ o
            m = b * o + c * ((d[:, None] + d) * o + sq)
            diag = b * d + c * (d * d + np.diag(sq))
            m = either_way(rng, (m - np.diag(np.diag(m))) * 256) / 256
            x = (a + diag)[:, None] * x + m @ copy
        worst = max(worst, off(x / size, ref))
    return 2 * worst + HALF if g.size < 256 else np.hypot(2 * worst, HALF / np.sqrt(3))


def run(g, steps, alpha=1.0, t="f32", ldo=None, workspace=None):
    """O (members, M, ldo) in 64 bits for g (members, M, ldg) on the device."""
    n, M, N = g.shape
    ldo = ldo or N
    O = torch.full((n, M, ldo), 9.0, dtype=torch.bfloat16, device="cuda")
    getattr(dg, f"orthogonalise_{t}")(M, N, steps, alpha, g, g.shape[2], M * g.shape[2], O, ldo, M * ldo, n, workspace=workspace)
    torch.cuda.synchronize()
    return O.cpu().double().numpy()


def off(got, ref):
    return np.linalg.norm(got - ref) / np.linalg.norm(ref)


def gradient(rng, M, N, rank=None):
    r = rank or max(1, min(M, N) // 8)
    g = rng.standard_normal((M, r)) * np.exp(rng.standard_normal(r)) @ rng.standard_normal((r, N)) / np.sqrt(r)
    return g + (0 if rank else 0.2 * rng.standard_normal((M, N)))


TOLERANCES = {}


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("steps", [FAST, TIGHT, MIXED], ids=["fast", "tight", "mixed"])
@pytest.mark.parametrize("M,N", [(1, 1), (1, 300), (300, 1), (2, 2), (16, 16), (63, 65), (64, 64), (65, 64), (128, 128), (129, 127), (100, 1000),
                                 (1000, 100), (128, 512), (512, 128), (257, 513), (640, 640), (513, 1001)])
def test_against_the_definition(t, steps, M, N):
    g = gradient(rng_of(M, N), M, N) * 1e-3
    G = torch.from_numpy(g).cuda().to(torch.float32 if t == "f32" else torch.bfloat16)[None]
    got = run(G, steps, t=t)[0]
    if (M, N, steps[1]) not in TOLERANCES:
        TOLERANCES[M, N, steps[1]] = tolerance(g, steps)     # (that of the fp32 gradient for both types)
    assert off(got, oracle(G[0].cpu().double().numpy(), steps)) <= TOLERANCES[M, N, steps[1]]


@pytest.mark.parametrize("M,N,rank", [(300, 500, 16), (512, 256, 4), (200, 200, 2), (640, 1280, 1), (64, 96, 1)])
def test_low_rank(M, N, rank):
    """Directions that G does not have stay out of the result: rounding errors in them would grow by 3.4445 a step."""
    G = torch.from_numpy(gradient(rng_of(M, N, rank), M, N, rank)).cuda().float()[None]
    got = run(G, FAST)[0]
    g = G[0].cpu().double().numpy()
    assert off(got, oracle(g, FAST)) <= tolerance(g, FAST)


@pytest.mark.parametrize("M,N", [(40, 90), (130, 70), (128, 512)])
def test_members_strides_and_gaps(M, N):
    """Many members at once, rows apart in G and O: each as if alone, gaps left as they are, NaN between G's rows of no account."""
    rng = rng_of("members", M, N)
    n = 5
    g = np.stack([gradient(rng, M, N) for _ in range(n)])
    wide = np.full((n, M + 2, N + 3), np.nan)
    wide[:, :M, :N] = g
    G = torch.from_numpy(wide).cuda().float()
    O = torch.full((n, M + 1, N + 5), 9.0, dtype=torch.bfloat16, device="cuda")
    dg.orthogonalise_f32(M, N, FAST, 0.5, G, N + 3, (M + 2) * (N + 3), O, N + 5, (M + 1) * (N + 5), n)
    got = O.cpu().double().numpy()
    for i in range(n):
        x = G[i, :M, :N].contiguous()
        g = x.cpu().double().numpy()
        assert off(got[i, :M, :N], oracle(g, FAST, 0.5)) <= tolerance(g, FAST)
        assert np.array_equal(got[i, :M, :N], run(x[None], FAST, 0.5)[0])
    assert np.all(got[:, M:] == 9) and np.all(got[:, :, N:] == 9)


def test_sizes_of_numbers():
    """Neither large nor small entries leave the range; zeros give zeros; an infinity or NaN makes its member NaN, and that alone."""
    rng = rng_of("range")
    g = gradient(rng, 70, 90)
    ref, tol = oracle(g.astype(np.float32), FAST), tolerance(g, FAST)
    for scale in (1e-30, 1e-18, 1e18, 1e36):
        G = torch.from_numpy((g * scale)).cuda().float()[None]
        got = run(G, FAST)[0]
        assert off(got, oracle(G[0].cpu().double().numpy() / scale, FAST)) <= tol, scale
    G = torch.from_numpy(np.stack([g, g, g, g * 0, g])).cuda().float()
    G[1, 3, 5], G[2, 69, 89] = float("nan"), float("inf")
    got = run(G, FAST)
    assert np.all(np.isnan(got[1])) and np.all(np.isnan(got[2])) and np.all(got[3] == 0)
    assert off(got[0], ref) <= tol and np.array_equal(got[0], got[4])


@pytest.mark.parametrize("M,N", [(150, 200), (300, 140)])
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_sizes_of_numbers_in_larger_updates(t, M, N):
    """test_sizes_of_numbers where a member takes many workgroups, with a workspace full of NaN."""
    rng = rng_of("larger range", M)
    g = gradient(rng, M, N)
    tol = tolerance(g, FAST)
    dt = torch.float32 if t == "f32" else torch.bfloat16
    for scale in (1e-30, 1e36):
        G = torch.from_numpy(g * scale).cuda().to(dt)[None]
        got = run(G, FAST, t=t)[0]
        assert off(got, oracle(G[0].cpu().double().numpy() / scale, FAST)) <= tol, scale
    G = torch.from_numpy(np.stack([g, g, g, g * 0, g])).cuda().to(dt)
    G[1, 3, 5], G[2, M - 1, N - 1] = float("nan"), float("inf")
    O = torch.empty(5, M, N, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((dg.orthogonalise_workspace(M, N, 5),), 0xFF, dtype=torch.uint8, device="cuda")
    getattr(dg, f"orthogonalise_{t}")(M, N, FAST, 1.0, G, N, M * N, O, N, M * N, 5, workspace=ws)
    got = O.cpu().double().numpy()
    assert np.all(np.isnan(got[1])) and np.all(np.isnan(got[2])) and np.all(got[3] == 0)
    assert np.array_equal(got[0], got[4]) and np.array_equal(got[0], run(G[:1], FAST, t=t)[0])


def test_one_gradient_for_all_members():
    """Members a stride of 0 apart: the same G for each."""
    for M, N in ((40, 60), (140, 150)):
        G = torch.from_numpy(gradient(rng_of("shared", M), M, N)).cuda().float()
        O = torch.empty(3, M, N, dtype=torch.bfloat16, device="cuda")
        dg.orthogonalise_f32(M, N, FAST, 1.0, G, N, 0, O, N, M * N, 3)
        got = O.cpu().double().numpy()
        assert all(np.array_equal(got[i], run(G[None], FAST)[0]) for i in range(3))


def test_singular_values():
    """What it is for: singular values near 1, singular vectors kept, the sign of every direction too."""
    rng = rng_of("values")
    g = rng.standard_normal((96, 200))
    u, s, vt = np.linalg.svd(g, full_matrices=False)
    got = run(torch.from_numpy(g).cuda().float()[None], FAST)[0]
    d = np.diag(u.T @ got @ vt.T)
    assert np.all(d > 0.65) and np.all(d < 1.25)
    rest = u.T @ got @ vt.T - np.diag(d)
    assert np.linalg.norm(rest) <= tolerance(g, FAST) * np.linalg.norm(got)


def test_again_streams_workspaces_and_graphs():
    """The same bits from call to call, whatever the workspace held, on another stream, and replayed from a graph between eager calls."""
    rng = rng_of("again")
    M, N = 200, 333
    G = torch.from_numpy(gradient(rng, M, N)).cuda().float()
    need = dg.orthogonalise_workspace(M, N)
    outs = [torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    spaces = [torch.full((need,), f, dtype=torch.uint8, device="cuda") for f in (0x00, 0xFF, 0x7C)]

    def call(out, ws=None):
        dg.orthogonalise_f32(M, N, FAST, 1.0, G, N, 0, out, N, 0, workspace=ws)

    for o, w in zip(outs, spaces + [None]):
        call(o, w)
    torch.cuda.synchronize()
    assert all(torch.equal(outs[0], o) for o in outs[1:])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(outs[1])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(outs[2], spaces[1])
    for _ in range(3):
        G.add_(torch.randn_like(G) * 0.1)
        call(outs[0])
        outs[2].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[2])


def test_large():
    """A large layer's weights, tall, against 64 bits on the GPU."""
    # (2^-8 / sqrt(3), and twice what random roundings of the copies give at 1000 x 1400)
    tol = tolerance(rng_of("large").standard_normal((1000, 1400)), FAST)
    g = torch.randn(2100, 1500, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    O = torch.empty(2100, 1500, dtype=torch.bfloat16, device="cuda")
    dg.orthogonalise_f32(2100, 1500, FAST, 0.2, g, 1500, 0, O, 1500, 0)
    x = g.double().t()
    x = x / torch.linalg.norm(x)
    for a, b, c in FAST:
        s = x @ x.t()
        x = a * x + b * (s @ x) + c * (s @ (s @ x))
    ref = 0.2 * x.t()
    assert float(torch.linalg.norm(O.double() - ref) / torch.linalg.norm(ref)) <= tol


@pytest.mark.parametrize("M,N", [(4100, 4170), (4040, 4000)])
def test_largest_tiles(M, N):
    """Updates whose products are tiles of 192 x 192 and 256 x 256, cut off at their ends."""
    tol = tolerance(rng_of("large").standard_normal((1000, 1400)), FAST)     # (as in test_large)
    g = torch.randn(M, N, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    O = torch.full((M + 1, N + 2), 9.0, dtype=torch.bfloat16, device="cuda")
    dg.orthogonalise_f32(M, N, FAST, 1.0, g, N, 0, O, N + 2, 0)
    x = (g if M < N else g.t()).double()
    x = x / torch.linalg.norm(x)
    for a, b, c in FAST:
        s = x @ x.t()
        x = a * x + b * (s @ x) + c * (s @ (s @ x))
    ref = x if M < N else x.t()
    assert torch.all(O[M:] == 9) and torch.all(O[:, N:] == 9)
    assert float(torch.linalg.norm(O[:M, :N].double() - ref) / torch.linalg.norm(ref)) <= tol


@pytest.mark.parametrize("n,M,N", [(5, 500, 520), (5, 520, 500), (1, 1100, 1300), (3, 1020, 1030), (9, 260, 700), (1, 960, 990)])
def test_numbers_of_tiles(n, M, N):
    """Members whose products are some hundreds of tiles, of the sizes that the numbers choose."""
    tol = tolerance(rng_of("tiles").standard_normal((500, 520)), FAST)
    g = torch.randn(n, M, N, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7))
    O = torch.full((n, M, N + 3), 9.0, dtype=torch.bfloat16, device="cuda")
    dg.orthogonalise_f32(M, N, FAST, 1.0, g, N, M * N, O, N + 3, M * (N + 3), n)
    assert torch.all(O[:, :, N:] == 9)
    for i in range(n):
        x = (g[i] if M < N else g[i].t()).double()
        x = x / torch.linalg.norm(x)
        for a, b, c in FAST:
            s = x @ x.t()
            x = a * x + b * (s @ x) + c * (s @ (s @ x))
        ref = x if M < N else x.t()
        assert float(torch.linalg.norm(O[i, :, :N].double() - ref) / torch.linalg.norm(ref)) <= tol


def test_expert_gradients():
    """The weight gradients of an expert layer, as the grouped product leaves them (all experts, one call), orthogonalised in one call."""
    G, R, D, F = 4, 300, 128, 192
    rng = rng_of("experts")
    x = torch.from_numpy(rng.standard_normal((R, D))).cuda().bfloat16()
    h = torch.from_numpy(rng.standard_normal((R, F))).cuda().bfloat16()
    offsets = torch.tensor([0, 100, 100, 220, 300], dtype=torch.int32, device="cuda")
    W = torch.empty(G, D, F, device="cuda")
    dg.gemm_grouped_wgrad_bf16_f32acc(G, R, D, F, 1.0, x, R, D, None, h, R, F, None, offsets, 0.0, W, F, D * F)
    got = run(W, FAST)
    w = W.cpu().double().numpy()
    assert np.all(got[1] == 0)                       # an expert without rows: no gradient, no update
    for g in (0, 2, 3):
        assert off(got[g], oracle(w[g], FAST)) <= tolerance(w[g], FAST)

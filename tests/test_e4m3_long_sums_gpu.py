"""Products of 8-bit operands summed over long K where every term has the same sign (GPU): partial sums are then as large as the sum of
the terms' sizes, and roundings that all go one way add up.

Held to the library's bound, |C - ref| <= 1e-5 (|alpha| sum of |terms| + |beta c|), whatever K is.
"""
from __future__ import annotations

import numpy as np
import pytest

import dense_gemm_optimisation_f32_amd as dg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TOL = 1e-5
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dg.load_library()
    yield
    torch.cuda.synchronize()


def same(n, K, blocks, value, scale, gen):
    """(values, scales, numbers): n rows of one value each, near `value`, times one scale for each row or block, near `scale`."""
    v = (value * (1 + torch.rand(n, 1, device="cuda", generator=gen))).to(E4M3)
    A = v.view(torch.uint8).expand(n, K).contiguous().view(E4M3)
    s = scale * (1 + 0.5 * torch.rand(blocks, device="cuda", generator=gen))
    kb = -(-K // 128)
    each = s.double().repeat_interleave(-(-n // blocks))[:n] if blocks < n else s.double()
    return A, s.expand(kb, blocks).contiguous(), v[:, 0].double() * each


# rows up to 16: streamed; 64 x 64: streamed by 32 rows; 512 x 512: 64 x 64 tiles; 1024 x 2048: 64 x 128; 2048 x 2048: 128 x 128, in pieces of 32768 k up to sixteen;
# rows of 2^23 bytes: through registers
@pytest.mark.parametrize("M,N,K", [(1, 1, 262144), (16, 40, 1 << 20), (7, 33, 1000003), (64, 64, 262144), (60, 50, 300001), (512, 512, 262144),
                                   (500, 510, 262147), (1024, 2048, 131072), (1000, 2000, 131075), (2048, 2048, 131072), (2000, 2040, 131077), (2048, 2048, 655360),
                                   (2, 3, 8000000), (3, 2, 8388609)])
@pytest.mark.parametrize("blockB", [1, 128])
def test_equal_terms(M, N, K, blockB):
    """The same product in every k: each addition to the sum is rounded as the one before it."""
    gen = torch.Generator(device="cuda").manual_seed(M + N + K)
    A, SA, a = same(M, K, M, 1.0, 1.1, gen)
    B, SB, b = same(N, K, -(-N // blockB) if blockB > 1 else N, 1.0, 1.3, gen)
    if blockB > 1:
        b = B[:, 0].double() * SB[0].double().repeat_interleave(128)[:N]
    C = torch.empty(M, N, device="cuda")
    dg.gemm_e4m3_f32acc(blockB, M, N, K, 0.5, A, K, SA, M, B, K, SB, SB.shape[1], 0.0, C, N)
    ref = 0.5 * K * a[:, None] * b
    assert float(((C.double() - ref) / ref).abs().max()) <= TOL


@pytest.mark.parametrize("M,N,K", [(5, 3, 1 << 20), (3, 4, 3000017), (40, 50, 600000), (2, 3, 8400000)])
@pytest.mark.parametrize("blockB", [1, 128])
def test_positive_terms(M, N, K, blockB):
    """Random positive numbers and scales."""
    gen = torch.Generator(device="cuda").manual_seed(K)
    A, B = (torch.rand(n, K, device="cuda", generator=gen).add_(0.1).to(E4M3) for n in (M, N))
    kb, nb = -(-K // 128), -(-N // blockB)
    SA, SB = (torch.rand(kb, n, device="cuda", generator=gen) + 0.5 for n in (M, nb))
    old = torch.rand(M, N, device="cuda", generator=gen) * K
    C = old.clone()
    dg.gemm_e4m3_f32acc(blockB, M, N, K, 1.0, A, K, SA, M, B, K, SB, nb, 0.5, C, N)
    a = A.double() * SA.t().double().repeat_interleave(128, 1)[:, :K]
    b = B.double() * SB.t().double().repeat_interleave(blockB, 0)[:N].repeat_interleave(128, 1)[:, :K]
    ref = torch.stack([(a * row).sum(1) for row in b], 1) + 0.5 * old.double()
    assert float(((C.double() - ref) / ref).abs().max()) <= TOL


@pytest.mark.parametrize("counts,N,K", [([3, 0, 5, 1], 40, 262144), ([200, 30, 0, 282], 256, 262144), ([70, 58], 130, 262149)])
def test_groups(counts, N, K):
    """The same in groups of rows, looked up."""
    G, R, T = len(counts), sum(counts), 9
    gen = torch.Generator(device="cuda").manual_seed(R)
    A, SA, a = same(T, K, T, 1.0, 1.1, gen)
    B, SB, b = same(G * N, K, G * N, 1.0, 1.3, gen)
    rows = torch.randint(0, T, (R,), device="cuda", generator=gen, dtype=torch.int32)
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    C = torch.empty(R, N, device="cuda")
    dg.gemm_grouped_e4m3_f32acc(1, G, R, N, K, 1.0, A, T, K, SA, T, rows, B, K, N * K, SB, G * N, N, offsets, 0.0, C, N)
    group = torch.repeat_interleave(torch.arange(G, device="cuda"), torch.tensor(counts, device="cuda"))
    ref = K * a[rows.long()][:, None] * b.view(G, N)[group]
    assert float(((C.double() - ref) / ref).abs().max()) <= TOL


@pytest.mark.parametrize("K", [65536, 65541, 98304 + 200])
@pytest.mark.parametrize("beta", [0.0, 0.5])
def test_groups_in_pieces(K, beta):
    """128 x 128 tiles, whose K goes in pieces that add to C: beta counts once, rows without a group stay as they were, rows that A does
    not hold are zero, and a captured call gives the same when it is replayed."""
    G, R, N, T = 2, 2100, 2048, 50
    gen = torch.Generator(device="cuda").manual_seed(K)
    A, SA, a = same(T, K, T, 1.0, 1.1, gen)
    B, SB, b = same(G * N, K, G * N, 1.0, 1.3, gen)
    rows = torch.randint(0, T, (R,), device="cuda", generator=gen, dtype=torch.int32)
    rows[5], rows[1200] = T, -1
    offsets = torch.tensor([0, 1100, 2000], dtype=torch.int32, device="cuda")
    old = torch.rand(R, N, device="cuda", generator=gen) * K if beta else torch.full((R, N), float("nan"), device="cuda")
    C = old.clone()

    def call():
        dg.gemm_grouped_e4m3_f32acc(1, G, R, N, K, 1.0, A, T, K, SA, T, rows, B, K, N * K, SB, G * N, N, offsets, beta, C, N)

    call()
    group = torch.cat([torch.zeros(1100, dtype=torch.long), torch.ones(900, dtype=torch.long)]).cuda()
    held = ((rows >= 0) & (rows < T))[:2000, None]
    ref = torch.where(held, K * a[rows.long().clamp(0, T - 1)][:2000, None] * b.view(G, N)[group], 0)
    if beta:
        ref = ref + beta * old[:2000].double()
    assert torch.all((C[:2000].double() - ref).abs() <= TOL * ref)
    assert torch.equal(C[2000:].view(torch.int32), old[2000:].view(torch.int32))
    first = C.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        C.copy_(old)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(C.view(torch.int32), first.view(torch.int32))


@pytest.mark.parametrize("M,N,K", [(4, 5, 1 << 20), (64, 64, 262144), (512, 512, 262144), (2048, 2048, 65536), (2, 2, 8400000)])
def test_infinite_scales(M, N, K):
    """An infinite scale makes its row infinite, whatever stood in the sum before it; two of either sign NaN; other rows are not touched."""
    gen = torch.Generator(device="cuda").manual_seed(M)
    A, SA, a = same(M, K, M, 1.0, 1.1, gen)
    B, SB, b = same(N, K, N, 1.0, 1.3, gen)
    kb = SA.shape[0]
    SA[kb // 3, 0] = float("inf")
    SA[kb // 3, 1], SA[kb - 1, 1] = float("inf"), -float("inf")
    C = torch.empty(M, N, device="cuda")
    dg.gemm_e4m3_f32acc(1, M, N, K, 1.0, A, K, SA, M, B, K, SB, N, 0.0, C, N)
    assert torch.all(C[0] == float("inf")) and torch.all(torch.isnan(C[1]))
    if M > 2:
        ref = K * a[2:, None] * b
        assert float(((C[2:].double() - ref) / ref).abs().max()) <= TOL

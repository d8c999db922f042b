"""C-ABI checks of the calls whose right operand is chosen per row, without a GPU: bad
arguments get the documented status before any HIP call, empty problems are
no-ops, workspace sizes, and the binding's own refusals."""
from __future__ import annotations

import pytest

import dense_gemm_optimisation_f32_amd as dg

OK, ESIZE, ELD, ENULL, ELAUNCH, EALIGN, EOP, ESCRATCH = 0, -1, -2, -3, -4, -5, -6, -7
FAKE = 0x10000          # a non-NULL, 16-byte aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    return dg.load_library()


def changed(defaults: dict, **kw) -> list:
    assert set(kw) <= set(defaults), set(kw) - set(defaults)
    return list({**defaults, **kw}.values())


ROUTE = dict(T=100, E=8, logits=FAKE, ldl=8, bias=None, score=0, groups=1, group_k=1, group_top=1, k=2, renorm=1, scale=1.0,
             ids=FAKE, weights=FAKE, offsets=FAKE, rows=FAKE, slots=FAKE, ws=FAKE, ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(score=2), EOP), (dict(renorm=-1), EOP),
    (dict(T=-1), ESIZE), (dict(T=(1 << 23) + 1), ESIZE), (dict(E=0), ESIZE), (dict(E=1025, ldl=1025), ESIZE),
    (dict(k=0), ESIZE), (dict(k=9), ESIZE), (dict(E=64, ldl=64, k=33), ESIZE),
    (dict(groups=0), ESIZE), (dict(groups=3), ESIZE), (dict(groups=2, group_k=3), ESIZE), (dict(groups=2, group_k=0), ESIZE),
    (dict(E=130, ldl=130, groups=65), ESIZE), (dict(group_top=3), ESIZE), (dict(group_top=0), ESIZE),
    (dict(ldl=7), ELD),
    (dict(logits=None), ENULL), (dict(ids=None), ENULL), (dict(weights=None), ENULL),
    (dict(offsets=None), ENULL), (dict(rows=None), ENULL), (dict(slots=None), ENULL),
    (dict(ws=None), ENULL), (dict(ws_bytes=16), ESCRATCH), (dict(ws_bytes=-1), ESCRATCH),
    (dict(logits=FAKE + 2), EALIGN), (dict(ids=FAKE + 1), EALIGN), (dict(rows=FAKE + 2), EALIGN),
    (dict(T=0, logits=None, ids=None, weights=None, offsets=None, rows=None, slots=None, ws=None, ws_bytes=0), OK),
])
def test_route_arguments(lib, kw, want):
    assert lib.moe_route_f32(*changed(ROUTE, **kw)) == want


def test_route_workspace(lib):
    assert lib.moe_route_workspace(0, 8, 2) == 0
    assert lib.moe_route_workspace(64, 8, 2) == 0
    assert lib.moe_route_workspace(65, 8, 2) > 0
    assert lib.moe_route_workspace(100, 8, 9) == 0      # not a call that can be made
    # counts of chunks x (E + 1) experts, of chunks that hold all tokens
    for T, E, k in ((65, 8, 2), (32768, 256, 8), (1 << 20, 1024, 32)):
        b = lib.moe_route_workspace(T, E, k)
        assert b % (4 * (E + 1)) == 0 and 2 <= b // (4 * (E + 1)) <= T


GRAD = dict(T=4, E=8, logits=FAKE, ldl=8, score=0, k=2, renorm=0, scale=1.0, ids=FAKE, dweights=FAKE, dlogits=FAKE, lddl=8,
            stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(score=-1), EOP), (dict(renorm=2), EOP), (dict(T=-1), ESIZE), (dict(E=2000, ldl=2000, lddl=2000), ESIZE), (dict(k=9), ESIZE),
    (dict(ldl=7), ELD), (dict(lddl=7), ELD), (dict(logits=None), ENULL), (dict(ids=None), ENULL), (dict(dweights=None), ENULL),
    (dict(dlogits=None), ENULL), (dict(dlogits=FAKE + 2), EALIGN), (dict(T=0, logits=None), OK),
])
def test_route_grad_arguments(lib, kw, want):
    assert lib.moe_route_f32_grad(*changed(GRAD, **kw)) == want


GROUPED = dict(transB=0, groups=3, R=10, N=6, K=5, alpha=1.0, A=FAKE, M=10, lda=5, rows=None, B=FAKE, ldb=6, strideB=30, offsets=FAKE,
               beta=0.0, C=FAKE, ldc=6, stream=None)


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("kw,want", [
    (dict(transB=2), EOP), (dict(groups=-1), ESIZE), (dict(groups=65536), ESIZE), (dict(R=-1), ESIZE), (dict(N=-1), ESIZE),
    (dict(K=-1), ESIZE), (dict(K=(1 << 30) + 1, lda=2**31 - 1), ESIZE), (dict(M=-1), ESIZE), (dict(lda=4), ELD), (dict(ldb=5), ELD), (dict(transB=1, ldb=4), ELD),
    (dict(transB=1, ldb=5, N=0), OK), (dict(ldc=5), ELD), (dict(strideB=-1), ELD), (dict(strideB=1 << 62), ESIZE),
    (dict(A=None), ENULL), (dict(B=None), ENULL), (dict(C=None), ENULL), (dict(offsets=None), ENULL),
    (dict(A=FAKE + 1), EALIGN), (dict(B=FAKE + 1), EALIGN), (dict(C=FAKE + 2), EALIGN), (dict(offsets=FAKE + 2), EALIGN),
    (dict(rows=FAKE + 2), EALIGN), (dict(R=2**31 - 1, N=2**20, ldb=2**20, ldc=2**20), ESIZE),
    (dict(R=0, A=None, B=None, C=None, offsets=None), OK), (dict(groups=0, A=None, B=None, C=None, offsets=None), OK),
])
def test_grouped_arguments(lib, t, kw, want):
    assert getattr(lib, f"gemm_grouped_{t}_f32acc_ex")(*changed(GROUPED, **kw)) == want


WGRAD = dict(groups=3, R=10, M=5, N=6, alpha=1.0, A=FAKE, a_rows=10, lda=5, rowsA=None, B=FAKE, b_rows=10, ldb=6, rowsB=None,
             offsets=FAKE, beta=0.0, C=FAKE, ldc=6, strideC=30, stream=None)


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("kw,want", [
    (dict(groups=-1), ESIZE), (dict(groups=65536), ESIZE), (dict(R=-1), ESIZE), (dict(M=-1), ESIZE), (dict(N=-1), ESIZE),
    (dict(a_rows=-1), ESIZE), (dict(b_rows=-1), ESIZE), (dict(lda=4), ELD), (dict(ldb=5), ELD), (dict(ldc=5), ELD),
    (dict(R=(1 << 30) + 1), ESIZE), (dict(strideC=29), ELD), (dict(strideC=-1), ELD), (dict(strideC=1 << 62), ESIZE),
    (dict(A=None), ENULL), (dict(B=None), ENULL), (dict(C=None), ENULL), (dict(offsets=None), ENULL),
    (dict(A=FAKE + 1), EALIGN), (dict(B=FAKE + 1), EALIGN), (dict(C=FAKE + 2), EALIGN), (dict(rowsA=FAKE + 1), EALIGN),
    (dict(rowsB=FAKE + 2), EALIGN), (dict(groups=0, C=None), OK), (dict(M=0, C=None), OK),
])
def test_wgrad_arguments(lib, t, kw, want):
    assert getattr(lib, f"gemm_grouped_wgrad_{t}_f32acc")(*changed(WGRAD, **kw)) == want


COMBINE = dict(T=4, k=2, N=6, Y=FAKE, R=8, ldy=6, slots=FAKE, weights=FAKE, beta=0.0, C=FAKE, ldc=6, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), ESIZE), (dict(T=(1 << 23) + 1), ESIZE), (dict(k=0), ESIZE), (dict(k=33), ESIZE), (dict(N=-1), ESIZE),
    (dict(N=(1 << 25) + 1, ldy=1 << 26, ldc=1 << 26), ESIZE), (dict(R=-1), ESIZE), (dict(ldy=5), ELD), (dict(ldc=5), ELD),
    (dict(Y=None), ENULL), (dict(slots=None), ENULL), (dict(C=None), ENULL), (dict(Y=FAKE + 2), EALIGN),
    (dict(slots=FAKE + 1), EALIGN), (dict(T=0, Y=None, slots=None, C=None), OK), (dict(N=0, Y=None, slots=None, C=None), OK),
])
def test_combine_arguments(lib, kw, want):
    assert lib.moe_combine_f32(*changed(COMBINE, **kw)) == want


CGRAD = dict(T=4, k=2, N=6, dC=FAKE, lddc=6, Y=FAKE, R=8, ldy=6, slots=FAKE, weights=None, dY=FAKE, lddy=6, dweights=FAKE, stream=None)


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), ESIZE), (dict(k=33), ESIZE), (dict(N=-1), ESIZE), (dict(R=-1), ESIZE), (dict(lddc=5), ELD), (dict(ldy=5), ELD),
    (dict(lddy=5), ELD), (dict(dC=None), ENULL), (dict(Y=None), ENULL), (dict(slots=None), ENULL), (dict(dY=None), ENULL),
    (dict(dweights=None), ENULL), (dict(dY=FAKE + 1), EALIGN), (dict(dC=FAKE + 2), EALIGN), (dict(T=0, dC=None), OK),
])
def test_combine_grad_arguments(lib, t, kw, want):
    assert getattr(lib, f"moe_combine_grad_{t}")(*changed(CGRAD, **kw)) == want


LORA = dict(transB=0, M=4, N=6, K=5, rank=3, adapters=2, alpha=1.0, A=FAKE, lda=5, B=FAKE, ldb=6, LA=FAKE, ldla=5, strideLA=15, LB=FAKE,
            ldlb=3, strideLB=18, scales=None, ranks=None, ids=FAKE, beta=0.0, C=FAKE, ldc=6, ws=FAKE, ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("kw,want", [
    (dict(transB=-1), EOP), (dict(M=-1), ESIZE), (dict(M=(1 << 23) + 1), ESIZE), (dict(N=-1), ESIZE), (dict(K=-1), ESIZE),
    (dict(K=(1 << 30) + 1, lda=2**31 - 1, ldla=2**31 - 1), ESIZE), (dict(rank=0), ESIZE), (dict(rank=129, ldlb=129), ESIZE), (dict(adapters=-1), ESIZE),
    (dict(lda=4), ELD), (dict(ldb=5), ELD), (dict(transB=1, ldb=4), ELD), (dict(ldc=5), ELD), (dict(ldla=4), ELD), (dict(ldlb=2), ELD),
    (dict(strideLA=-1), ELD), (dict(strideLB=-1), ELD), (dict(strideLA=1 << 62), ESIZE),
    (dict(A=None), ENULL), (dict(B=None), ENULL), (dict(C=None), ENULL), (dict(LA=None), ENULL), (dict(LB=None), ENULL),
    (dict(ids=None), ENULL), (dict(ws=None), ENULL), (dict(ws_bytes=0), ESCRATCH), (dict(ws_bytes=-5), ESCRATCH),
    (dict(ws=FAKE + 4), EALIGN), (dict(A=FAKE + 1), EALIGN), (dict(LB=FAKE + 1), EALIGN), (dict(ids=FAKE + 2), EALIGN),
    (dict(C=FAKE + 2), EALIGN), (dict(M=0, A=None, C=None), OK), (dict(N=0, ldb=1, A=None, C=None), OK),
])
def test_lora_arguments(lib, t, kw, want):
    assert getattr(lib, f"gemm_lora_{t}_f32acc_ex")(*changed(LORA, **kw)) == want



@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_large_results_are_taken(lib, t):
    """C of 16 GiB to 512 GiB passes the size check (and stops at the next one); what no launch holds does not."""
    def grouped(R, N, groups=32, K=64, transB=0, A=FAKE):
        ld = max(N, K)
        return getattr(lib, f"gemm_grouped_{t}_f32acc_ex")(*changed(GROUPED, transB=transB, groups=groups, R=R, M=R, N=N, K=K, A=A, lda=ld,
                                                                    ldb=ld, strideB=0, ldc=N, C=None))
    assert grouped(1 << 18, 1 << 14) == ENULL
    assert grouped(1 << 18, (1 << 14) + 8, transB=1) == ENULL
    assert grouped(1 << 18, (1 << 14) + 1, K=63) == ENULL
    assert grouped(1 << 18, (1 << 14) + 1, K=63, transB=1) == ENULL
    assert grouped(1 << 22, 1 << 15) == ENULL                      # 16384 x 128 tiles of 256 x 256
    assert grouped(100, 1 << 20, groups=65535) == ENULL            # few rows a group, many columns
    assert grouped(33 * 65535, 8192, groups=65535) == ENULL        # 64-row tiles would be too many
    assert grouped(1 << 21, 1 << 15, K=63, transB=1) == ENULL      # 16384 x 256 tiles of 128 x 128
    assert grouped(1 << 22, 1 << 15, K=63) == ESIZE                # 65536 x 512 tiles of 64 x 64
    assert grouped(1 << 22, 1 << 15, A=FAKE + 2) == ESIZE
    assert grouped(1 << 25, 1 << 15) == ESIZE

    def wgrad(M, N, A=FAKE):
        return getattr(lib, f"gemm_grouped_wgrad_{t}_f32acc")(*changed(WGRAD, M=M, N=N, A=A, lda=M, ldb=N, ldc=N, strideC=M * N, C=None))
    assert wgrad(1 << 17, 1 << 17) == ENULL
    assert wgrad((1 << 17) - 3, (1 << 17) - 1) == ENULL
    assert wgrad(1 << 18, 1 << 18) == ENULL
    assert wgrad(1 << 18, 1 << 20) == ESIZE

    def lora(M, N, K=64, transB=0, adapters=2):
        ld = max(N, K)
        return getattr(lib, f"gemm_lora_{t}_f32acc_ex")(*changed(LORA, transB=transB, M=M, N=N, K=K, adapters=adapters, lda=K, ldb=ld, ldc=N,
                                                                 ldla=K, strideLA=0, strideLB=0, ws=None, ws_bytes=0))
    assert lora(1 << 14, 1 << 17) == ESCRATCH
    assert lora(1 << 17, 1 << 15, transB=1) == ESCRATCH
    assert lora((1 << 17) + 1, 1 << 15, K=63, transB=1) == ESCRATCH
    assert lora(1 << 17, 1 << 17, K=63) == ESCRATCH
    assert lora(64, 1 << 25, K=63) == ESCRATCH
    assert lora(1 << 23, 1 << 25) == ESIZE
    assert lora(1 << 18, 1 << 18, K=63) == ESIZE


def test_lora_workspace(lib):
    assert lib.gemm_lora_workspace(0, 6, 5, 3) == 0
    assert lib.gemm_lora_workspace(4, 6, 5, 0) == 0
    for M in (1, 17, 64, 65, 4096):   # at least the narrow product in 32 bits
        assert lib.gemm_lora_workspace(M, 4096, 4096, 16) >= 4 * 16 * M


@pytest.mark.parametrize("N", [1, 64, 128, 512, 4096])
@pytest.mark.parametrize("M", [1, 48, 64])
def test_lora_workspace_grows_with_k(lib, M, N):
    """At most 16 shares of K, for a wide or a narrow N: the narrow products of 16 and sums of 16."""
    sizes = [lib.gemm_lora_workspace(M, N, K, 16) for K in range(64, 70000, 64)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    assert sizes[-1] <= 4 * (16 * M * 16 + 16 * M * N)


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    f, i = torch.zeros(64), torch.zeros(64, dtype=torch.int32)
    with pytest.raises(ValueError):   # CPU tensors
        dg.moe_route_f32(4, 8, f, 8, None, 0, 1, 1, 1, 2, 1, 1.0, i, f, stream=0)
    with pytest.raises(ValueError):
        dg.moe_combine_f32(4, 2, 6, f, 8, 6, i, f, 0.0, f, 6, stream=0)
    with pytest.raises(ValueError):
        dg.gemm_lora_bf16_f32acc_ex(0, 4, 6, 5, 3, 2, 1.0, f, 5, f, 6, f, 5, 15, f, 3, 18, None, None, i, 0.0, f, 6, stream=0)
    with pytest.raises(TypeError):
        dg.moe_combine_f32(4, 2, 6, "Y", 8, 6, FAKE, FAKE, 0.0, FAKE, 6, stream=0)
    with pytest.raises(dg.GemmError) as e:
        dg.gemm_grouped_f16_f32acc_ex(3, 1, 4, 6, 5, 1.0, FAKE, 4, 5, None, FAKE, 6, 30, FAKE, 0.0, FAKE, 6, stream=0)
    assert e.value.status == EOP


def test_binding_stream_of_another_device(monkeypatch):
    """A call runs on the device of its stream, and is refused when its tensors are on another."""
    torch = pytest.importorskip("torch")
    current, seen = [0], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *a):
            current[0] = self.before

    class Stream:
        cuda_stream, device = 0, torch.device("cuda", 1)

    dg._load_torch()
    monkeypatch.setattr(dg, "_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    args = (3, 1, 4, 6, 5, 1.0, FAKE, 4, 5, None, FAKE, 6, 30, FAKE, 0.0, FAKE, 6)      # (transB = 3: refused before any launch)
    lib_fn = dg._function("gemm_grouped_f16_f32acc_ex")

    class Watch:
        __name__ = "gemm_grouped_f16_f32acc_ex"

        def __call__(self, *a):
            seen.append(current[0])
            return lib_fn(*a)

    monkeypatch.setattr(dg, "_function", lambda name: Watch())
    with pytest.raises(dg.GemmError):
        dg.gemm_grouped_f16_f32acc_ex(*args, stream=Stream())
    assert seen == [1] and current == [0]

    def on_device_0(x, name, dtype_name, need, packed=False):
        if current[0] != 0:
            raise dg._Elsewhere(0)
        return x

    monkeypatch.setattr(dg, "_strided", on_device_0)
    with pytest.raises(ValueError, match="more than one device"):
        dg.gemm_grouped_f16_f32acc_ex(*args, stream=Stream())
    assert seen == [1] and current == [0]

"""C-ABI checks of the 8-bit operators and the orthogonalised updates, without a GPU: bad arguments get the documented
status before any HIP call, empty problems are no-ops, workspace sizes, and the binding's own refusals."""
from __future__ import annotations

import ctypes

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


QUANT = dict(transpose=0, block=1, M=10, K=300, X=FAKE, ldx=300, strideX=3000, Q=FAKE, ldq=300, strideQ=3000, S=FAKE, lds=10, strideS=30,
             batch=2, stream=None)


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kw,want", [
    (dict(transpose=2), EOP), (dict(transpose=-1), EOP), (dict(block=0), ESIZE), (dict(block=64), ESIZE), (dict(M=-1), ESIZE),
    (dict(K=-1), ESIZE), (dict(batch=-1), ESIZE), (dict(ldx=299), ELD), (dict(transpose=1, ldx=9), ELD), (dict(ldq=299), ELD),
    (dict(lds=9), ELD), (dict(block=128, lds=0), ELD), (dict(strideX=-1), ELD), (dict(strideQ=2999), ELD), (dict(strideS=29), ELD),
    (dict(strideX=1 << 62), ESIZE), (dict(X=None), ENULL), (dict(Q=None), ENULL), (dict(S=None), ENULL), (dict(S=FAKE + 2), EALIGN),
    (dict(X=FAKE + 1), EALIGN), (dict(M=0, X=None), OK), (dict(K=0, X=None, S=None), OK), (dict(batch=0, Q=None), OK),
    (dict(M=2**30, K=2**20, ldx=2**20, ldq=2**20, lds=2**30, strideQ=2**51, strideS=2**44), ESIZE),     # more tiles than a launch holds
    (dict(batch=2**23), ESIZE), (dict(transpose=1, ldx=10, batch=2**23 // 3 + 1), ESIZE),
])
def test_quant_arguments(lib, t, kw, want):
    assert getattr(lib, f"quant_e4m3_{t}")(*changed(QUANT, **kw)) == want


def test_quant_alignment_is_the_elements(lib):
    assert lib.quant_e4m3_f32(*changed(QUANT, X=FAKE + 2)) == EALIGN


PRODUCT = dict(blockB=128, M=10, N=200, K=300, alpha=1.0, A=FAKE, lda=300, SA=FAKE, ldsa=10, B=FAKE, ldb=300, SB=FAKE, ldsb=2, beta=0.0,
               C=FAKE, ldc=200, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(blockB=2), ESIZE), (dict(blockB=0), ESIZE), (dict(M=-1), ESIZE), (dict(N=-1), ESIZE), (dict(K=-1), ESIZE),
    (dict(K=2**30 + 1, lda=2**31 - 1, ldb=2**31 - 1), ESIZE), (dict(lda=299), ELD), (dict(ldb=299), ELD), (dict(ldsa=9), ELD),
    (dict(ldsb=1), ELD), (dict(blockB=1, ldsb=199), ELD), (dict(ldc=199), ELD), (dict(A=None), ENULL), (dict(SA=None), ENULL),
    (dict(B=None), ENULL), (dict(SB=None), ENULL), (dict(C=None), ENULL), (dict(C=FAKE + 2), EALIGN), (dict(SA=FAKE + 2), EALIGN),
    (dict(SB=FAKE + 1), EALIGN), (dict(M=0, lda=300, A=None, C=None), OK), (dict(N=0, B=None, C=None), OK),
    (dict(M=2**31 - 1, N=2**31 - 1, ldsa=2**31 - 1, ldsb=2**24, ldc=2**31 - 1), ESIZE),
])
def test_product_arguments(lib, kw, want):
    assert lib.gemm_e4m3_f32acc(*changed(PRODUCT, **kw)) == want


GROUPED = dict(blockB=128, groups=3, R=10, N=200, K=300, alpha=1.0, A=FAKE, M=10, lda=300, SA=FAKE, ldsa=10, rows=None, B=FAKE, ldb=300,
               strideB=60000, SB=FAKE, ldsb=2, strideSB=6, offsets=FAKE, beta=0.0, C=FAKE, ldc=200, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(blockB=64), ESIZE), (dict(groups=-1), ESIZE), (dict(groups=65536), ESIZE), (dict(R=-1), ESIZE), (dict(N=-1), ESIZE),
    (dict(K=-1), ESIZE), (dict(M=-1), ESIZE), (dict(lda=299), ELD), (dict(ldb=299), ELD), (dict(ldsa=9), ELD), (dict(ldsb=1), ELD),
    (dict(ldc=199), ELD), (dict(strideB=-1), ELD), (dict(strideSB=-1), ELD), (dict(strideB=1 << 62), ESIZE), (dict(strideSB=1 << 62), ESIZE),
    (dict(A=None), ENULL), (dict(SA=None), ENULL), (dict(B=None), ENULL), (dict(SB=None), ENULL), (dict(C=None), ENULL),
    (dict(offsets=None), ENULL), (dict(offsets=FAKE + 2), EALIGN), (dict(rows=FAKE + 2), EALIGN), (dict(C=FAKE + 1), EALIGN),
    (dict(SB=FAKE + 2), EALIGN), (dict(groups=0, offsets=None, C=None), OK), (dict(R=0, C=None), OK),
    (dict(R=2**31 - 1, N=2**25, ldsb=2**18, ldc=2**25), ESIZE),
])
def test_grouped_arguments(lib, kw, want):
    assert lib.gemm_grouped_e4m3_f32acc(*changed(GROUPED, **kw)) == want


FIVE = (ctypes.c_float * 15)(*[3.4445, -4.775, 2.0315] * 5)
ORTHO = dict(M=200, N=300, steps=5, coefficients=ctypes.addressof(FIVE), alpha=1.0, G=FAKE, ldg=300, strideG=60000, O=FAKE, ldo=300, strideO=60000, batch=2,
             ws=FAKE, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), ESIZE), (dict(N=-1), ESIZE), (dict(M=65537), ESIZE), (dict(N=65537, ldg=65537, ldo=65537), ESIZE), (dict(steps=0), ESIZE),
    (dict(steps=101), ESIZE), (dict(batch=-1), ESIZE), (dict(batch=65536), ESIZE), (dict(M=65536, N=65536, ldg=65536, ldo=65536, batch=9), ESIZE),
    (dict(ldg=299), ELD), (dict(ldo=299), ELD), (dict(strideG=-1), ELD), (dict(strideO=59999), ELD), (dict(strideG=1 << 62), ESIZE),
    (dict(coefficients=None), ENULL), (dict(G=None), ENULL), (dict(O=None), ENULL), (dict(ws=None), ENULL), (dict(G=FAKE + 1), EALIGN),
    (dict(O=FAKE + 1), EALIGN), (dict(ws=FAKE + 8), EALIGN), (dict(ws_bytes=64), ESCRATCH), (dict(ws_bytes=-1), ESCRATCH),
    (dict(M=0, G=None, ws=None), OK), (dict(N=0, G=None, ws=None), OK), (dict(batch=0, G=None, ws=None), OK),
])
def test_orthogonalise_arguments(lib, t, kw, want):
    assert getattr(lib, f"orthogonalise_{t}")(*changed(ORTHO, **kw)) == want


def test_orthogonalise_workspace(lib):
    size = lib.orthogonalise_workspace
    assert size(0, 8, 1) == size(8, 0, 1) == size(8, 8, 0) == 0
    assert size(-1, 8, 1) == size(70000, 8, 1) == size(8, 8, 65536) == 0       # not calls that can be made
    for M, N in ((1, 1), (64, 1024), (512, 128), (129, 129), (513, 300), (4096, 4096)):
        one = size(M, N, 1)
        assert one % 16 == 0 and (one > 0) == (min(M, N) > 128) and size(M, N, 3) == 3 * one and size(N, M, 1) == one
        assert one <= 12 * (M + 127) * (N + 127) + 8 * (min(M, N) + 127) ** 2 + 16384


def test_binding_refuses(lib):
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 128)
    with pytest.raises(ValueError):
        dg.quant_e4m3_f32(0, 1, 4, 128, x, 128, 0, x, 128, 0, x, 4, 0)
    with pytest.raises(ValueError):
        dg.orthogonalise_f32(4, 128, [(1.0, 0.0, 0.0)], 1.0, x, 128, 0, x, 128, 0)
    with pytest.raises(ValueError):
        dg.orthogonalise_f32(4, 4, [(1.0, 0.0)], 1.0, None, 4, 0, None, 4, 0)
    with pytest.raises(dg.GemmError):
        dg.gemm_e4m3_f32acc(7, 4, 4, 4, 1.0, None, 4, None, 4, None, 4, None, 4, 0.0, None, 4, stream=0)
    with pytest.raises(dg.GemmError):
        dg.orthogonalise_bf16(4, 4, [], 1.0, FAKE, 4, 0, FAKE, 4, 0, workspace=FAKE, stream=0)


def test_quant_long_sides(lib):
    assert lib.quant_e4m3_bf16(*changed(QUANT, M=1, K=2**30 + 1, ldx=2**31 - 1, ldq=2**31 - 1, batch=1)) == ESIZE
    assert lib.quant_e4m3_bf16(*changed(QUANT, transpose=1, M=2**30 + 1, K=1, ldx=2**31 - 1, lds=2**31 - 1, batch=1)) == ESIZE


def test_coefficients_are_read_at_the_call(monkeypatch):
    """Coefficients that are tensors of one value, changed in place between calls."""
    torch = pytest.importorskip("torch")
    seen = []
    monkeypatch.setattr(dg, "_call", lambda fn, args, *rest: seen.append(list((ctypes.c_float * 3).from_address(args[3]))))
    steps = torch.tensor([[1.0, 2.0, 3.0]])
    kept = [list(step) for step in steps]
    for _ in range(2):
        dg.orthogonalise_f32(4, 4, kept, 1.0, FAKE, 4, 0, FAKE, 4, 0, workspace=FAKE, stream=0)
        steps.mul_(2)
    assert seen == [[1.0, 2.0, 3.0], [2.0, 4.0, 6.0]]


CALLS = {
    "quant_e4m3_bf16": (2, 1, 4, 6, FAKE, 6, 24, FAKE, 6, 24, FAKE, 4, 4),                    # (each refused before any launch)
    "gemm_e4m3_f32acc": (7, 4, 6, 5, 1.0, FAKE, 5, FAKE, 4, FAKE, 5, FAKE, 1, 0.0, FAKE, 6),
    "gemm_grouped_e4m3_f32acc": (7, 2, 4, 6, 5, 1.0, FAKE, 4, 5, FAKE, 4, None, FAKE, 5, 30, FAKE, 1, 1, FAKE, 0.0, FAKE, 6),
    "orthogonalise_f32": (4, 6, [], 1.0, FAKE, 6, 24, FAKE, 6, 24),
}


@pytest.mark.parametrize("name", CALLS)
def test_binding_devices(monkeypatch, name):
    """A call runs on the device of its stream, and is refused when an operand is on another."""
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
    lib_fn = dg._function(name)

    class Watch:
        __name__ = name

        def __call__(self, *a):
            seen.append(current[0])
            return lib_fn(*a)

    monkeypatch.setattr(dg, "_function", lambda name: Watch())
    kw = {"workspace": FAKE} if name.startswith("orthogonalise") else {}
    with pytest.raises(dg.GemmError):
        getattr(dg, name)(*CALLS[name], stream=Stream(), **kw)
    assert seen == [1] and current == [0]

    def on_device_0(x, name, dtype_name, need, packed=False):
        if current[0] != 0:
            raise dg._Elsewhere(0)
        return x

    monkeypatch.setattr(dg, "_strided", on_device_0)
    with pytest.raises(ValueError, match="more than one device"):
        getattr(dg, name)(*CALLS[name], stream=Stream(), **kw)
    assert seen == [1] and current == [0]

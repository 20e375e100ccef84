"""The operators around the products on the host (no GPU): argument checks and
workspace queries of the C ABI, and what the Python binding refuses.  No call
here launches a kernel."""
import ctypes

import pytest

import pipelined_warp_specialized_gb300 as pws
from pipelined_warp_specialized_gb300 import build as libbuild

BAD, ALIGN, OK = pws.GEMM_ERR_INVALID_ARG, pws.GEMM_ERR_ALIGNMENT, pws.GEMM_OK
H, B = pws.GEMM_TYPE_HALF, pws.GEMM_TYPE_BFLOAT
# fake, 256-byte aligned addresses far apart: never dereferenced on these paths
P = [(i + 1) << 40 for i in range(12)]


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return pws.load_library()


def swap(args, i, value):
    out = list(args)
    out[i] = value
    return out


# (entry, arguments that pass every check up to the device's, [(index, value, status), ...])
GATED = [4, 8, 16, P[0], P[1], P[2], P[3], P[4], P[5], H, 0, None, 0, None]
GATED_BWD = [4, 8, 16, P[0], P[1], P[2], P[3], P[4], P[5], P[6], P[7], P[8], B, 1, P[9], 1 << 30, None]
XENT = [4, 8, 16, P[0], P[1], P[2], -100, P[3], P[4], H, P[5], 1 << 30, None]
XENT_BWD = [4, 8, 16, P[0], P[1], P[2], -100, P[3], P[4], P[5], P[6], B, P[7], 1 << 30, None]
LINEAR = [4, 8, 16, P[0], P[1], P[2], P[3], P[4], H, P[5], 1 << 30, None]
REFUSALS = [
    ("gemm_gated_nt", GATED, [
        (0, -1, BAD), (1, -1, BAD), (2, -1, BAD), (0, 1 << 31, BAD), (1, 1 << 31, BAD), (2, 1 << 31, BAD),
        (3, 0, BAD), (4, 0, BAD), (5, 0, BAD), (6, 0, BAD),            # missing operands, missing h
        (7, 0, BAD), (8, 0, BAD),                                      # g without u, u without g
        (9, 2, BAD), (9, -1, BAD), (10, 2, BAD), (10, -1, BAD),        # unknown type, activation
        (3, P[0] + 1, ALIGN), (4, P[1] + 1, ALIGN), (6, P[3] + 1, ALIGN), (8, P[5] + 1, ALIGN),
        (6, P[0] + 2, BAD), (7, P[1], BAD), (7, P[3] + 8, BAD)]),      # overlaps: h and x, g and w_gate, g and h
    ("gemm_gated_nt_bwd", GATED_BWD, [
        (0, -1, BAD), (1, 1 << 31, BAD), (2, -5, BAD), (3, 0, BAD), (4, 0, BAD), (5, 0, BAD), (6, 0, BAD), (7, 0, BAD),
        (8, 0, BAD), (10, 0, BAD), (11, 0, BAD),                       # one weight gradient without the other
        (12, 7, BAD), (13, 7, BAD), (3, P[0] + 1, ALIGN), (11, P[8] + 1, ALIGN),
        (9, P[0], BAD), (10, P[8] + 16, BAD)]),
    ("gemm_xent_nt", XENT, [
        (0, -1, BAD), (1, 0, BAD), (1, -1, BAD), (2, -1, BAD), (1, 1 << 31, BAD), (3, 0, BAD), (4, 0, BAD), (5, 0, BAD),
        (7, 0, BAD), (8, 0, BAD), (9, 9, BAD), (3, P[0] + 1, ALIGN), (5, P[2] + 4, ALIGN), (7, P[3] + 2, ALIGN),
        (8, P[4] + 1, ALIGN), (7, P[0] + 4, BAD), (8, P[3] + 4, BAD)]),
    ("gemm_xent_nt_bwd", XENT_BWD, [
        (0, -1, BAD), (1, 0, BAD), (2, 1 << 31, BAD), (3, 0, BAD), (4, 0, BAD), (5, 0, BAD), (7, 0, BAD), (8, 0, BAD),
        (11, 3, BAD), (9, P[5] + 1, ALIGN), (10, P[6] + 1, ALIGN), (7, P[3] + 2, ALIGN), (8, P[4] + 3, ALIGN),
        (9, P[0] + 4, BAD), (10, P[5] + 4, BAD), (9, P[4], BAD)]),
    ("gemm_nt_bwd", LINEAR, [
        (0, -1, BAD), (1, -1, BAD), (2, 1 << 31, BAD), (3, 0, BAD), (4, 0, BAD), (5, 0, BAD), (8, 2, BAD),
        (3, P[0] + 1, ALIGN), (6, P[3] + 1, ALIGN), (7, P[4] + 1, ALIGN), (6, P[0], BAD), (7, P[3] + 8, BAD)]),
]


@pytest.mark.parametrize("name,args,cases", REFUSALS, ids=[r[0] for r in REFUSALS])
def test_refused_before_any_launch(lib, name, args, cases):
    fn = getattr(lib, name)
    for i, value, want in cases:
        assert fn(*swap(args, i, value)) == want, (i, value)
    # the arguments themselves pass: what is left to fail is the device
    import torch
    if not torch.cuda.is_available():
        assert fn(*args) not in (OK, BAD, ALIGN)


def test_empty_calls_are_no_ops(lib):
    assert lib.gemm_gated_nt(*swap(swap(GATED, 0, 0), 6, 0)) == OK
    assert lib.gemm_gated_nt(*swap(GATED, 1, 0)) == OK
    assert lib.gemm_gated_nt_bwd(*swap(GATED_BWD, 2, 0)) == OK
    assert lib.gemm_gated_nt_bwd(*swap(swap(swap(GATED_BWD, 9, 0), 10, 0), 11, 0)) == OK      # nothing wanted
    assert lib.gemm_xent_nt(*swap(XENT, 0, 0)) == OK
    assert lib.gemm_xent_nt_bwd(*swap(swap(XENT_BWD, 9, 0), 10, 0)) == OK
    assert lib.gemm_nt_bwd(*swap(LINEAR, 2, 0)) == OK
    assert lib.gemm_nt_bwd(*swap(swap(LINEAR, 6, 0), 7, 0)) == OK


def workspace(lib, name, *args):
    n = ctypes.c_int64(-1)
    assert getattr(lib, name + "_workspace")(*args, ctypes.byref(n)) == OK
    return n.value


def test_workspace_of_aligned_operands(lib):
    # the forward block needs none; the others hold what their formulas keep
    assert workspace(lib, "gemm_gated_nt", 300, 512, 256, P[0], P[1], P[2], H) == 0
    M, F, K = 300, 520, 256
    need = workspace(lib, "gemm_gated_nt_bwd", M, F, K, *P[:6], B)
    assert need >= 2 * M * 576 * 2                                      # dg, du in rows of 576
    M, V, K = 100, 1000, 64
    assert workspace(lib, "gemm_xent_nt", M, V, K, P[0], P[1], H) >= 8 * M + 4 * M
    assert workspace(lib, "gemm_xent_nt_bwd", M, V, K, P[0], P[1], H) >= 2 * M * V
    assert workspace(lib, "gemm_nt_bwd", 8192, 4096, 4096, P[0], P[1], P[2], H) == 0


def test_workspace_of_unaligned_operands(lib):
    # a copy of each operand that 16-byte copies cannot address, in rows of a
    # multiple of 64 elements; both weights share one form
    M, F, K = 300, 512, 256
    rows = 256 * 2
    assert workspace(lib, "gemm_gated_nt", M, F, K, P[0] + 2, P[1], P[2], H) == 300 * rows
    assert workspace(lib, "gemm_gated_nt", M, F, K, P[0], P[1] + 2, P[2], H) == 2 * 512 * rows
    assert workspace(lib, "gemm_gated_nt", M, F, 250, P[0], P[1], P[2], H) == (300 + 2 * 512) * rows
    base = workspace(lib, "gemm_nt_bwd", 8192, 4096, 4096, P[0], P[1], P[2], H)
    assert workspace(lib, "gemm_nt_bwd", 8192, 4096, 4096, P[0], P[1] + 2, P[2], H) == base + 8192 * 4096 * 2


def test_workspace_is_bounded_by_the_pieces(lib):
    # one piece of D, not the logits, for a large batch and vocabulary
    M, V, K = 65536, 131072, 4096
    need = workspace(lib, "gemm_xent_nt_bwd", M, V, K, P[0], P[1], B)
    assert need < 2 * M * V // 4
    assert need >= 2 * M * 8192


def test_workspace_refusals(lib):
    n = ctypes.c_int64()
    for name, args in (("gemm_gated_nt", (4, 8, 16, P[0], P[1], P[2], H)), ("gemm_gated_nt_bwd", (4, 8, 16, *P[:6], H)),
                       ("gemm_xent_nt", (4, 8, 16, P[0], P[1], H)), ("gemm_xent_nt_bwd", (4, 8, 16, P[0], P[1], H)),
                       ("gemm_nt_bwd", (4, 8, 16, P[0], P[1], P[2], H))):
        fn = getattr(lib, name + "_workspace")
        assert fn(*args, None) == BAD
        assert fn(-1, *args[1:], ctypes.byref(n)) == BAD
        assert fn(*args[:-1], 5, ctypes.byref(n)) == BAD
        assert fn(*args[:3], P[0] + 1, *args[4:], ctypes.byref(n)) == ALIGN


# ---------------------------------------------------------------- the binding

torch = pytest.importorskip("torch")
F16, BF16, F32, I64 = torch.float16, torch.bfloat16, torch.float32, torch.int64


class Stub:
    """A stand-in for a CUDA tensor: the binding must refuse before any launch."""

    def __init__(self, shape, dtype=F16, device="cuda:0", contiguous=True, cuda=True):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device(device)
        self._contiguous, self.is_cuda = contiguous, cuda

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return self._contiguous


M_, F_, V_, K_ = 4, 6, 9, 8
CALLS = {
    "gemm_gated_nt": lambda **o: (o.get("x", Stub((M_, K_))), o.get("w", Stub((F_, K_))), o.get("w2", Stub((F_, K_)))),
    "gemm_gated_nt_bwd": lambda **o: (o.get("dh", Stub((M_, F_))), o.get("g", Stub((M_, F_))), Stub((M_, F_)),
                                      o.get("x", Stub((M_, K_))), o.get("w", Stub((F_, K_))),
                                      o.get("w2", Stub((F_, K_)))),
    "gemm_xent_nt": lambda **o: (o.get("x", Stub((M_, K_))), o.get("w", Stub((V_, K_))),
                                 o.get("target", Stub((M_,), I64))),
    "gemm_xent_nt_bwd": lambda **o: (o.get("x", Stub((M_, K_))), o.get("w", Stub((V_, K_))),
                                     o.get("target", Stub((M_,), I64)), o.get("lse", Stub((M_,), F32)),
                                     o.get("dloss", Stub((M_,), F32))),
    "gemm_nt_bwd": lambda **o: (o.get("dy", Stub((M_, V_))), o.get("x", Stub((M_, K_))), o.get("w", Stub((V_, K_)))),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_binding_refusals(name):
    fn, args = getattr(pws, name), CALLS[name]
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        fn(*[Stub(t.shape, F32) if t.dtype == F16 else t for t in args()])
    with pytest.raises(TypeError, match="one type"):
        fn(*args(w=Stub(args()[-1].shape if name == "gemm_nt_bwd" else (F_ if "gated" in name else V_, K_), BF16)))
    with pytest.raises(ValueError, match="contiguous CUDA"):
        fn(*args(x=Stub((M_, K_), contiguous=False)))
    with pytest.raises(ValueError, match="contiguous CUDA"):
        fn(*args(x=Stub((M_, K_), cuda=False)))
    with pytest.raises(ValueError, match="one device"):
        fn(*args(x=Stub((M_, K_), device="cuda:1")))
    with pytest.raises(ValueError, match="matrices"):
        fn(*args(x=Stub((M_ * K_,))))
    with pytest.raises(ValueError, match="do not form"):
        fn(*args(w=Stub((F_ if "gated" in name else V_, K_ + 1))))


def test_binding_refuses_bad_vectors_and_activations():
    for name in ("gemm_xent_nt", "gemm_xent_nt_bwd"):
        fn, args = getattr(pws, name), CALLS[name]
        with pytest.raises(TypeError, match="target"):
            fn(*args(target=Stub((M_,), torch.int32)))
        with pytest.raises(ValueError, match="target"):
            fn(*args(target=Stub((M_ + 1,), I64)))
        with pytest.raises(ValueError, match="target"):
            fn(*args(target=Stub((M_,), I64, contiguous=False)))
        with pytest.raises(ValueError, match="one device"):
            fn(*args(target=Stub((M_,), I64, device="cuda:1")))
    bwd, args = pws.gemm_xent_nt_bwd, CALLS["gemm_xent_nt_bwd"]
    with pytest.raises(TypeError, match="dloss"):
        bwd(*args(dloss=Stub((M_,), F16)))
    with pytest.raises(ValueError, match="lse"):
        bwd(*args(lse=Stub((M_, 1), F32)))
    for name in ("gemm_gated_nt", "gemm_gated_nt_bwd"):
        with pytest.raises(ValueError, match="act"):
            getattr(pws, name)(*CALLS[name](), act="relu")
    with pytest.raises(ValueError, match="shape"):
        pws.gemm_gated_nt_bwd(*CALLS["gemm_gated_nt_bwd"](g=Stub((M_, F_ + 1))))


def test_half_unit_of_the_types():
    # the tolerances' rounding terms: half a unit is 2^-11 of a binary16 value
    # and 2^-8 of a bfloat16 one, and both are reached
    y = torch.rand(200000, dtype=torch.float64, generator=torch.Generator().manual_seed(1)) + 1.0
    for dtype, bound in ((F16, 2.0 ** -11), (BF16, 2.0 ** -8)):
        err = ((y.to(dtype).double() - y).abs() / y).max()
        assert bound * 0.95 < float(err) <= bound

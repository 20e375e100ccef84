"""The 8-bit operators and the mixture of experts on the host (no GPU):
argument checks and workspace queries of the C ABI, and what the Python binding
refuses.  No call here launches a kernel."""
import ctypes

import pytest

import pipelined_warp_specialized_gb300 as pws
from pipelined_warp_specialized_gb300 import build as libbuild

BAD, ALIGN, OK = pws.GEMM_ERR_INVALID_ARG, pws.GEMM_ERR_ALIGNMENT, pws.GEMM_OK
H, B, I8 = pws.GEMM_TYPE_HALF, pws.GEMM_TYPE_BFLOAT, pws.GEMM_TYPE_BYTE
# fake, 256-byte aligned addresses far apart: never dereferenced on these paths
P = [(i + 1) << 40 for i in range(14)]


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return pws.load_library()


def swap(args, *changes):
    out = list(args)
    for i, value in changes:
        out[i] = value
    return out


QUANTIZE = [4, 16, P[0], P[1], P[2], H, None]
PRODUCT = [4, 8, 16, P[0], P[1], P[2], P[3], P[4], B, P[5], 1 << 30, None]
# M, K, F, E, top_k, x, router, gate, up, down, three scales, y, experts, weights, type, weight type, act, normalize, ws, bytes, stream
MOE = [4, 16, 8, 6, 2, P[0], P[1], P[2], P[3], P[4], None, None, None, P[8], P[9], P[10], H, H, 0, 1, P[11], 1 << 30, None]
MOE8 = swap(MOE, (10, P[5]), (11, P[6]), (12, P[7]), (17, I8))
REFUSALS = [
    ("gemm_i8_quantize", QUANTIZE, [
        (0, -1, BAD), (1, -1, BAD), (0, 1 << 31, BAD), (1, 1 << 31, BAD), (2, 0, BAD), (3, 0, BAD), (4, 0, BAD),
        (5, I8, BAD), (5, -1, BAD), (2, P[0] + 1, ALIGN), (4, P[2] + 2, ALIGN), (3, P[0] + 3, BAD), (4, P[1] + 4, BAD)]),
    ("gemm_i8_nt", PRODUCT, [
        (0, -1, BAD), (1, -1, BAD), (2, -1, BAD), (0, 1 << 31, BAD), (1, 1 << 31, BAD), (2, 131072, BAD),
        (3, 0, BAD), (4, 0, BAD), (5, 0, BAD), (6, 0, BAD), (7, 0, BAD), (8, I8, BAD), (8, -1, BAD),
        (5, P[2] + 2, ALIGN), (6, P[3] + 1, ALIGN), (7, P[4] + 1, ALIGN),
        (7, P[0] + 2, BAD), (7, P[1] + 4, BAD), (7, P[2], BAD), (7, P[3] + 8, BAD)]),
    ("gemm_moe_nt", MOE, [
        (0, -1, BAD), (1, -1, BAD), (2, -1, BAD), (0, 1 << 31, BAD), (1, 1 << 31, BAD), (2, 1 << 31, BAD),
        (3, 0, BAD), (3, 1025, BAD), (4, 0, BAD), (4, 7, BAD), (4, -1, BAD),
        (5, 0, BAD), (6, 0, BAD), (7, 0, BAD), (8, 0, BAD), (9, 0, BAD), (10, P[5], BAD), (12, P[5], BAD),
        (13, 0, BAD), (14, 0, BAD), (15, 0, BAD), (16, I8, BAD), (16, B, BAD), (17, B, BAD), (17, I8, BAD), (17, 3, BAD),
        (18, 2, BAD), (19, 2, BAD), (19, -1, BAD),
        (5, P[0] + 1, ALIGN), (6, P[1] + 1, ALIGN), (7, P[2] + 1, ALIGN), (9, P[4] + 1, ALIGN), (13, P[8] + 1, ALIGN),
        (14, P[9] + 2, ALIGN), (15, P[10] + 2, ALIGN),
        (13, P[0], BAD), (13, P[4] + 2, BAD), (14, P[8] + 4, BAD), (15, P[9] + 4, BAD), (14, P[1], BAD),
        (20, 0, BAD), (20, P[11] + 64, BAD), (21, 16, BAD), (20, P[0], BAD), (20, P[8], BAD)]),
    ("gemm_moe_nt", MOE8, [
        (10, 0, BAD), (11, 0, BAD), (12, 0, BAD), (10, P[5] + 2, ALIGN), (12, P[7] + 1, ALIGN), (13, P[6], BAD), (17, H, BAD)]),
]


@pytest.mark.parametrize("name,args,cases", REFUSALS, ids=["quantize", "product", "moe", "moe8"])
def test_refused_before_any_launch(lib, name, args, cases):
    fn = getattr(lib, name)
    for i, value, want in cases:
        assert fn(*swap(args, (i, value))) == want, (i, value)
    # the arguments themselves pass: what is left to fail is the device
    import torch
    if not torch.cuda.is_available():
        assert fn(*args) not in (OK, BAD, ALIGN)


def test_accepted_where_only_the_device_is_missing(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch on fake addresses")
    for name, args in (("gemm_i8_nt", swap(PRODUCT, (2, 131071))), ("gemm_i8_nt", swap(PRODUCT, (3, P[0] + 1), (4, P[1] + 7))),
                       ("gemm_i8_quantize", swap(QUANTIZE, (3, P[1] + 1), (5, B))),
                       ("gemm_moe_nt", swap(MOE, (4, 6))), ("gemm_moe_nt", swap(MOE, (3, 1024), (4, 32), (0, 65))),
                       ("gemm_moe_nt", swap(MOE, (16, B), (17, B), (18, 1), (19, 0))),
                       ("gemm_moe_nt", swap(MOE8, (7, P[2] + 1), (8, P[3] + 3), (9, P[4] + 5), (16, B))),
                       ("gemm_moe_nt", swap(MOE, (2, 0), (7, 0), (8, 0), (9, 0)))):
        assert getattr(lib, name)(*args) not in (OK, BAD, ALIGN), (name, args)


def test_top_k_is_at_most_32(lib):
    assert lib.gemm_moe_nt(*swap(MOE, (3, 64), (4, 33))) == BAD


def test_width_is_at_most_2_to_the_22(lib):
    top, n = 1 << 22, ctypes.c_int64()
    for i in (1, 2):
        assert lib.gemm_moe_nt(*swap(MOE, (i, top + 1))) == BAD
        sizes = swap([64, 16, 8, 1024, 32, H, H], (i, top))
        assert lib.gemm_moe_nt_workspace(*sizes, ctypes.byref(n)) == OK and n.value > 0
        assert lib.gemm_moe_nt_workspace(*swap(sizes, (i, top + 1)), ctypes.byref(n)) == BAD


def test_empty_calls_are_no_ops(lib):
    assert lib.gemm_i8_quantize(*swap(QUANTIZE, (0, 0), (2, 0))) == OK
    assert lib.gemm_i8_nt(*swap(PRODUCT, (0, 0), (7, 0))) == OK
    assert lib.gemm_i8_nt(*swap(PRODUCT, (1, 0), (4, 0))) == OK
    assert lib.gemm_moe_nt(*swap(MOE, (0, 0), (5, 0), (13, 0), (20, 0))) == OK


def workspace(lib, name, *args):
    n = ctypes.c_int64(-1)
    assert getattr(lib, name + "_workspace")(*args, ctypes.byref(n)) == OK
    return n.value


def test_workspaces(lib):
    # the experts' activations of a pass, two 16-bit values each in rows of a multiple of 64, and partial sums
    for M, passes in ((1, 1), (64, 64), (1000, 64)):
        need = workspace(lib, "gemm_moe_nt", M, 512, 100, 8, 2, H, H)
        held = 2 * passes * 2 * 128 * 2 + passes * 512 * 2 + passes * 2 * 512 * 4
        assert held < need < held + 16384
    assert workspace(lib, "gemm_moe_nt", 1000, 512, 100, 8, 2, H, H) == workspace(lib, "gemm_moe_nt", 64, 512, 100, 8, 2, H, H)
    assert workspace(lib, "gemm_moe_nt", 0, 512, 100, 8, 2, H, H) == 0
    assert workspace(lib, "gemm_i8_nt", 0, 512, 100, P[0], P[1], H) == 0
    # no more than both operands in 16 bits, whatever their alignment
    for K in (64, 100, 4096):
        for off in (0, 1):
            need = workspace(lib, "gemm_i8_nt", 300, 512, K, P[0] + off, P[1], H)
            assert need <= 2 * (300 + 512) * ((K + 63) // 64 * 64) + 512


def test_ragged_weights_of_many_tiles_are_widened_in_memory(lib):
    # 128 x 128 tiles: 48 and 64 of them go past memory in any rows, 96 and 128 in rows of whole 16 bytes alone
    for M, N, K, tiles in ((768, 1024, 8200, 48), (512, 2048, 8200, 64), (768, 2048, 8200, 96), (512, 4096, 4104, 128)):
        ld = (K + 63) // 64 * 64
        tokens, both = 2 * M * ld, 2 * (M + N) * ld
        need = workspace(lib, "gemm_i8_nt", M, N, K, P[0], P[1], H)
        assert (both if tiles > 64 else tokens) <= need < (both if tiles > 64 else tokens) + 1024
        assert tokens <= workspace(lib, "gemm_i8_nt", M, N, ld, P[0], P[1], H) < tokens + 1024
        assert workspace(lib, "gemm_i8_nt", M, N, ld, P[0], P[1] + 1, H) == need


def test_workspace_refusals(lib):
    n = ctypes.c_int64()
    ref = ctypes.byref(n)
    assert lib.gemm_i8_nt_workspace(4, 8, 16, P[0], P[1], H, None) == BAD
    assert lib.gemm_i8_nt_workspace(4, 8, 131072, P[0], P[1], H, ref) == BAD
    assert lib.gemm_i8_nt_workspace(4, 8, 16, P[0], P[1], I8, ref) == BAD
    good = [4, 16, 8, 6, 2, H, I8]
    assert lib.gemm_moe_nt_workspace(*good, None) == BAD
    for i, value in ((0, -1), (1, -1), (2, -1), (3, 0), (4, 0), (4, 7), (5, I8), (6, B)):
        assert lib.gemm_moe_nt_workspace(*swap(good, (i, value)), ref) == BAD, (i, value)


# ---------------------------------------------------------------- the binding

torch = pytest.importorskip("torch")
F16, BF16, F32, S8 = torch.float16, torch.bfloat16, torch.float32, torch.int8


class Stub:
    """A stand-in for a CUDA tensor: the binding must refuse before any launch."""

    def __init__(self, shape, dtype=F16, device="cuda:0", contiguous=True, cuda=True):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device(device)
        self._contiguous, self.is_cuda = contiguous, cuda

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return self._contiguous


M_, N_, K_, F_, E_ = 4, 9, 8, 6, 5


def test_binding_refuses_quantize():
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        pws.gemm_i8_quantize(Stub((M_, K_), F32))
    for bad in (Stub((M_, K_), contiguous=False), Stub((M_, K_), cuda=False)):
        with pytest.raises(ValueError, match="contiguous CUDA"):
            pws.gemm_i8_quantize(bad)
    with pytest.raises(ValueError, match="matrices"):
        pws.gemm_i8_quantize(Stub((2, M_, K_)))


def i8_args(**o):
    return [o.get("a", Stub((M_, K_), S8)), o.get("b", Stub((N_, K_), S8)), o.get("sa", Stub((M_,), F32)),
            o.get("sb", Stub((N_,), F32))]


@pytest.mark.parametrize("change,kind,match", [
    (dict(a=Stub((M_, K_))), TypeError, "int8"), (dict(b=Stub((N_, K_), torch.uint8)), TypeError, "int8"),
    (dict(a=Stub((1, M_, K_), S8)), ValueError, "matrices"), (dict(b=Stub((N_, K_ + 1), S8)), ValueError, "do not form"),
    (dict(a=Stub((M_, K_), S8, contiguous=False)), ValueError, "contiguous CUDA"),
    (dict(b=Stub((N_, K_), S8, cuda=False)), ValueError, "contiguous CUDA"),
    (dict(b=Stub((N_, K_), S8, device="cuda:1")), ValueError, "one device"),
    (dict(sa=Stub((M_,), F16)), TypeError, "a_scale"), (dict(sb=Stub((N_ + 1,), F32)), ValueError, "b_scale"),
    (dict(sa=Stub((M_, 1), F32)), ValueError, "a_scale"), (dict(sb=Stub((N_,), F32, device="cuda:1")), ValueError, "one device"),
])
def test_binding_refuses_product(change, kind, match):
    with pytest.raises(kind, match=match):
        pws.gemm_i8_nt(*i8_args(**change))


def test_binding_refuses_product_type():
    with pytest.raises(TypeError, match="dtype"):
        pws.gemm_i8_nt(*i8_args(), dtype=F32)


def moe_args(kind=F16, **o):
    return [o.get("x", Stub((M_, K_))), o.get("wr", Stub((E_, K_))), o.get("wg", Stub((E_, F_, K_), kind)),
            o.get("wu", Stub((E_, F_, K_), kind)), o.get("wd", Stub((E_, K_, F_), kind)), 2]


SCALES = (Stub((E_, F_), F32), Stub((E_, F_), F32), Stub((E_, K_), F32))


@pytest.mark.parametrize("change,kind,match", [
    (dict(x=Stub((M_, K_), F32)), TypeError, "float16 or bfloat16"), (dict(wr=Stub((E_, K_), BF16)), TypeError, "one type"),
    (dict(x=Stub((M_, 1, K_))), ValueError, "matrices"), (dict(wr=Stub((E_, K_ + 1))), ValueError, "do not form"),
    (dict(wg=Stub((E_ * F_, K_))), ValueError, "do not form"), (dict(wg=Stub((E_, F_, K_), BF16)), TypeError, "w_gate"),
    (dict(wu=Stub((E_, F_ + 1, K_))), ValueError, "w_up"), (dict(wd=Stub((E_, F_, K_))), ValueError, "w_down"),
    (dict(wd=Stub((E_, K_, F_), S8)), TypeError, "w_down"), (dict(wg=Stub((E_, F_, K_), contiguous=False)), ValueError, "contiguous"),
    (dict(wu=Stub((E_, F_, K_), device="cuda:1")), ValueError, "one device"),
])
def test_binding_refuses_moe(change, kind, match):
    with pytest.raises(kind, match=match):
        pws.gemm_moe_nt(*moe_args(**change))


def test_binding_refuses_moe_scales_and_codes():
    with pytest.raises(TypeError, match="w_gate"):
        pws.gemm_moe_nt(*moe_args(), scales=SCALES)                        # scales, but 16-bit weights
    with pytest.raises(TypeError, match="w_gate"):
        pws.gemm_moe_nt(*moe_args(S8))                                     # 8-bit weights without scales
    with pytest.raises(ValueError, match="scales"):
        pws.gemm_moe_nt(*moe_args(S8), scales=SCALES[:2])
    with pytest.raises(TypeError, match="scales of w_down"):
        pws.gemm_moe_nt(*moe_args(S8), scales=SCALES[:2] + (Stub((E_, K_), F16),))
    with pytest.raises(ValueError, match="scales of w_up"):
        pws.gemm_moe_nt(*moe_args(S8), scales=(SCALES[0], Stub((E_, K_), F32), SCALES[2]))
    with pytest.raises(ValueError, match="act"):
        pws.gemm_moe_nt(*moe_args(), act="relu")

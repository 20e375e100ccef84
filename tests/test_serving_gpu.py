"""The 8-bit operators and the mixture of experts on the GPU, against their
formulas in 64 bits.

Every tolerance is an error bound of the computation, elementwise:

* 8-bit integers: the quantization is exact (whole numbers and a correctly
  rounded scale), and so is the product's sum; its fp32 value, two products with
  scales and the rounding to 16 bits are four roundings: 3 * 2^-24 relative and half
  a unit;
* a sum of K products on the tensor cores adds 16 of them at a time into an fp32
  accumulator.  Each of the K/16 additions loses at most one unit in the last place
  of a partial sum no larger than S = sum |a b|, and the sum inside a group of
  16 at most 8 more: (K/16 + 8) 2^-23 S; joining eight warps' sums stays below
  what their shorter sums save;
* h' as two 16-bit values: 2^-16 relative in bfloat16 (its remainder rounded to
  8 bits more), 2^-22 and 2^-25 absolute in binary16;
* exp2, the fast division and the routing weights are good to 2^-20 relative, for
  arguments below 32 in magnitude.
"""
import math

import pytest

torch = pytest.importorskip("torch")

import pipelined_warp_specialized_gb300 as pws  # noqa: E402

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
TYPES = [F16, BF16]


@pytest.fixture(autouse=True)
def _no_timeouts():
    yield
    assert pws.gemm_device_status() == pws.GEMM_OK


def half_unit(y, dtype):
    y = y.abs()
    return y * 2.0 ** -11 + 2.0 ** -25 if dtype == F16 else y * 2.0 ** -8 + 2.0 ** -134


def acc_error(K, s):
    return (K / 16 + 8) * 2.0 ** -23 * s


def rand(shape, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def rand_i8(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-128, 128, shape, generator=g, device="cuda", dtype=torch.int8)


def off_by_one(t):
    """The same values at an address one element past a 16-byte boundary."""
    flat = torch.empty(t.numel() + 16, dtype=t.dtype, device=t.device)
    out = flat[1:1 + t.numel()].view(t.shape)
    out.copy_(t)
    assert out.data_ptr() % 16 == t.element_size()
    return out


def same_bits(a, b):
    kind = {1: torch.int8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.view(kind), b.view(kind))


# ---------------------------------------------------------------- quantization


def quantized64(x):
    xd = x.double()
    top = xd.abs().amax(dim=1) if x.shape[1] else torch.zeros(x.shape[0], device=x.device, dtype=torch.float64)
    fine = torch.isfinite(top)
    q = torch.round(127 * xd / torch.where(top > 0, top, torch.ones_like(top))[:, None])
    q = torch.where(fine[:, None], q, torch.zeros_like(q)).to(torch.int8)
    # (a tensor over a number is a product with its reciprocal: over a tensor, and rounded once)
    scale = (top / torch.full_like(top, 127)).float()
    return q, torch.where(fine, scale, torch.full_like(scale, math.nan))


def same_scales(a, b):
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(), b.nan_to_num())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K", [(1, 1), (1, 7), (3, 8), (9, 64), (5, 257), (33, 1024), (7, 1025), (64, 4096), (2, 8191),
                                 (3, 8192), (2, 8200), (2, 32768), (2, 32777), (1, 70001), (4000, 2050), (1000, 96)])
def test_quantize(M, K, dtype):
    for x in (rand((M, K), dtype, M + K), rand((M, K), dtype, K) * torch.exp(3 * rand((M, 1), torch.float32, 1)).to(dtype)):
        for y in (x, off_by_one(x)):
            q, scale = pws.gemm_i8_quantize(y)
            want, want_scale = quantized64(x)
            assert torch.equal(q, want) and same_scales(scale, want_scale)


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_every_value(dtype):
    """Every finite value beside every tenth of a set of largest ones, at three magnitudes."""
    bits = torch.arange(0, 1 << 16, dtype=torch.int32, device="cuda").to(torch.int16).view(dtype)
    bits = bits[torch.isfinite(bits)]
    g = torch.Generator().manual_seed(5)
    for exponent in ((-20, 0, 15) if dtype == F16 else (-130, -70, 0, 70, 127)):
        tops = (1 + torch.randint(0, 1024, (40,), generator=g).double() / 1024) * 2.0 ** exponent
        for top in tops.to(dtype).unique():
            x = bits[bits.abs() <= top.to("cuda")]
            x = torch.cat([x, top.to("cuda").view(1)]).view(1, -1)
            q, scale = pws.gemm_i8_quantize(x)
            want, want_scale = quantized64(x)
            assert torch.equal(q, want) and same_scales(scale, want_scale), (exponent, top)


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_halves_go_to_even(dtype):
    # 127 x / top halfway between integers: top = 127 * 2^k and x = (n + 1/2) 2^k, and x = top / 2
    n = torch.arange(-127, 127, device="cuda").double() + 0.5
    for top in (127.0, 127 * 2.0 ** -12):
        x = torch.cat([n * top / 127, torch.tensor([top], device="cuda")]).to(dtype).view(1, -1)
        q, _ = pws.gemm_i8_quantize(x)
        assert torch.equal(q, torch.round(x.double() * 127 / top).to(torch.int8))
    x = rand((50, 64), dtype, 3)
    x[:, 1] = x.abs().amax(dim=1)
    x[:, 2] = x[:, 1] / 2
    q, _ = pws.gemm_i8_quantize(x)
    assert (q[:, 2] == 64).all()                    # 63.5


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_zero_and_nonfinite_rows(dtype):
    for K in (5, 64, 3000, 9000):
        x = rand((6, K), dtype, K)
        x[0] = 0
        x[1, K - 1] = math.inf
        x[2, 0] = -math.inf
        x[3, K // 2] = math.nan
        q, scale = pws.gemm_i8_quantize(x)
        assert not q[:4].any() and scale[0] == 0 and torch.isnan(scale[1:4]).all()
        want, want_scale = quantized64(x[4:])
        assert torch.equal(q[4:], want) and torch.equal(scale[4:], want_scale)


def test_quantize_empty():
    q, scale = pws.gemm_i8_quantize(torch.empty(3, 0, device="cuda", dtype=F16))
    assert q.shape == (3, 0) and torch.equal(scale, torch.zeros(3, device="cuda"))
    q, scale = pws.gemm_i8_quantize(torch.empty(0, 5, device="cuda", dtype=F16))
    assert q.shape == (0, 5) and scale.shape == (0,)


# ---------------------------------------------------------------- 8-bit product

I8 = [(1, 1, 1), (1, 16, 64), (1, 4096, 1000), (1, 333, 4096), (2, 100, 17), (3, 1000, 2048), (4, 129, 1023), (5, 40, 16),
      (7, 4096, 4096), (8, 500, 1030), (9, 64, 1024), (15, 77, 1025), (16, 2048, 512), (17, 256, 2050), (32, 1000, 8192),
      (33, 100, 96), (64, 300, 4100), (65, 3000, 640), (100, 128, 131071), (128, 129, 1040), (129, 640, 3000),
      (300, 2052, 2050), (1000, 1000, 1), (700, 5, 333), (2048, 1536, 768), (4000, 300, 2049)]


def i8_want(a, b, sa, sb):
    total = (a.double() @ b.double().t())
    assert total.abs().max() < 2 ** 53
    return total * sa.double()[:, None] * sb.double()


def i8_check(out, want, dtype):
    assert out.dtype == dtype and out.shape == want.shape
    tol = want.abs() * 3 * 2.0 ** -24
    err = (out.double() - want).abs()
    assert (err <= tol + half_unit(want.abs() + tol, dtype)).all(), float((err / want.abs()).max())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", I8)
def test_i8(M, N, K, dtype):
    a, b = rand_i8((M, K), 1), rand_i8((N, K), 2)
    # (binary16: the largest sum, K * 2^14, times the scales stays below 65504)
    sa, sb = rand((M,), torch.float32, 3).abs() * 0.02 + 0.001, rand((N,), torch.float32, 4).abs() * 0.02 + 0.001
    want = i8_want(a, b, sa, sb)
    out = pws.gemm_i8_nt(a, b, sa, sb, dtype=dtype)
    i8_check(out, want, dtype)
    for i in range(2):
        ops = [off_by_one(t) if i == j else t for j, t in enumerate((a, b))]
        assert same_bits(pws.gemm_i8_nt(*ops, sa, sb, dtype=dtype), out)


# a batch of tokens where its weights are large, small, split over a cluster and at the edges of tiles and chunks
@pytest.mark.parametrize("M", [17, 24, 32, 33, 63, 64, 65, 127, 128, 129])
@pytest.mark.parametrize("N,K", [(1000, 8400), (4100, 2056), (20000, 449), (77, 130), (129, 64), (128, 3136), (333, 8193), (3, 5)])
def test_i8_batches(M, N, K):
    a, b = rand_i8((M, K), M), rand_i8((N, K), N)
    sa, sb = rand((M,), torch.float32, 3).abs() * 0.02 + 0.001, rand((N,), torch.float32, 4).abs() * 0.02 + 0.001
    want = i8_want(a, b, sa, sb)
    out = pws.gemm_i8_nt(a, b, sa, sb, dtype=BF16)
    i8_check(out, want, BF16)
    assert same_bits(pws.gemm_i8_nt(a, off_by_one(b), sa, sb, dtype=BF16), out)
    # a token's row is its own: alone and in the batch the same bits
    assert same_bits(pws.gemm_i8_nt(a[M - 1:], b, sa[M - 1:], sb, dtype=BF16), out[M - 1:])


# several tiles of tokens, the last one a few, and a count of tiles that leaves the batch's kernel
@pytest.mark.parametrize("M,N,K", [(130, 20000, 100), (255, 129, 64), (256, 700, 8200), (257, 70, 2049), (513, 1030, 4100), (1000, 300, 2048),
                                   (5000, 40, 2050), (300, 8000, 2050), (700, 3000, 2304)])
def test_i8_token_tiles(M, N, K):
    a, b = rand_i8((M, K), M), rand_i8((N, K), N)
    sa, sb = rand((M,), torch.float32, 3).abs() * 0.02 + 0.001, rand((N,), torch.float32, 4).abs() * 0.02 + 0.001
    out = pws.gemm_i8_nt(a, b, sa, sb, dtype=BF16)
    i8_check(out, i8_want(a, b, sa, sb), BF16)
    assert same_bits(pws.gemm_i8_nt(off_by_one(a), off_by_one(b), sa, sb, dtype=BF16), out)


@pytest.mark.parametrize("M,N,K", [(5000, 40, 2050), (1000, 300, 4096), (128, 3000, 4096)])
def test_i8_repeats(M, N, K):
    """The same bits every time, whatever else keeps memory busy and the copies out of step."""
    a, b = rand_i8((M, K), 1), rand_i8((N, K), 2)
    ones = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    want = (a.double() @ b.double().t()).bfloat16()
    junk, side = torch.empty(1 << 26, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for i in range(100):
        if i % 4 == 0:
            with torch.cuda.stream(side):
                junk.mul_(1.0)
        outs.append(pws.gemm_i8_nt(a, b, *ones))
    torch.cuda.synchronize()
    assert all(same_bits(o, want) for o in outs)


@pytest.mark.parametrize("M,N,K", [(2100, 1100, 131071), (1, 40, 131071), (8, 33, 131071), (12, 33, 131071), (40, 24, 131071), (300, 300, 131071), (2, 64, 4096),
                                   (200, 64, 4096)])
def test_i8_sums_are_exact(M, N, K):
    """Sums near 2^31 that differ in their last bits: the difference of two of
    them is exact only if each is."""
    a = torch.full((M, K), -128, device="cuda", dtype=torch.int8)
    b = torch.full((N, K), -128, device="cuda", dtype=torch.int8)
    a[:, -1] = torch.arange(M, device="cuda").to(torch.int8) % 100
    b[:, K // 2] = torch.arange(N, device="cuda").to(torch.int8) % 100 - 50
    total = (a.double() @ b.double().t())
    # 2^-16 of the largest sum is 32768: in binary16 units of 16 or 32; so look at the sum in
    # pieces through the scale, whose fp32 product is exact for powers of two
    out = pws.gemm_i8_nt(a, b, torch.full((M,), 2.0 ** -16, device="cuda"), torch.ones(N, device="cuda"), dtype=F16)
    i8_check(out, total * 2.0 ** -16, F16)
    # one more column cancels all but the last bits: -128 * 128 each, with opposite sign
    half = K // 2
    c = a.clone()
    c[:, :half] = 127
    d = b.clone()
    d[:, :2 * half] = -128
    c[:, half:2 * half] = -127
    want = c.double() @ d.double().t()
    assert want.abs().max() < 2 ** 15
    ones = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    i8_check(pws.gemm_i8_nt(c, d, *ones, dtype=F16), want, F16)


@pytest.mark.parametrize("dtype", TYPES)
def test_i8_scales(dtype):
    """Zero, infinite and NaN scales act on their own row and column; scales whose
    product leaves fp32's range act one after the other."""
    for M, N, K in ((1, 64, 64), (20, 96, 256), (300, 260, 128)):
        a, b = rand_i8((M, K), 1), rand_i8((N, K), 2)
        a[:, 0] = b[:, 0] = 1
        sa, sb = torch.full((M,), 1e-3, device="cuda"), torch.full((N,), 1e-3, device="cuda")
        sb[3], sb[5], sb[7] = 0.0, math.nan, math.inf
        want = i8_want(a, b, sa, sb)
        out = pws.gemm_i8_nt(a, b, sa, sb, dtype=dtype)
        assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.equal(torch.isinf(out), torch.isinf(want))
        fine = torch.isfinite(want)
        assert ((out.double() - want).abs() <= want.abs() * 3 * 2.0 ** -24 + half_unit(want, dtype))[fine].all()
        tiny = pws.gemm_i8_nt(a, b, torch.full((M,), 1e-30, device="cuda"), torch.full((N,), 1e30, device="cuda"), dtype=dtype)
        total = a.double() @ b.double().t()
        err = (tiny.double() - total).abs()
        ok = total.abs() < 60000
        assert (err <= total.abs() * 2.0 ** -20 + half_unit(total, dtype))[ok].all()


def test_i8_empty():
    f = torch.zeros(0, device="cuda")
    e = lambda *s: torch.empty(*s, device="cuda", dtype=torch.int8)  # noqa: E731
    one = torch.ones(3, device="cuda")
    assert not pws.gemm_i8_nt(e(3, 0), e(4, 0), one, torch.ones(4, device="cuda")).any()
    assert pws.gemm_i8_nt(e(0, 8), e(3, 8), f, one).shape == (0, 3)
    assert pws.gemm_i8_nt(e(3, 8), e(0, 8), one, f).shape == (3, 0)


def test_i8_writes_its_rows_alone():
    for M, N, K in ((3, 70, 100), (20, 33, 64), (200, 65, 128)):
        a, b = rand_i8((M, K), 1), rand_i8((N, K), 2)
        ones = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
        want = pws.gemm_i8_nt(a, b, *ones, dtype=F16)
        room = torch.full((M * N + 64,), 7.0, device="cuda", dtype=F16)
        need = pws.ctypes.c_int64()
        lib = pws.load_library()
        assert lib.gemm_i8_nt_workspace(M, N, K, a.data_ptr(), b.data_ptr(), 0, pws.ctypes.byref(need)) == 0
        ws = torch.full((need.value + 256,), 0xFF, dtype=torch.uint8, device="cuda")
        rc = lib.gemm_i8_nt(M, N, K, a.data_ptr(), b.data_ptr(), ones[0].data_ptr(), ones[1].data_ptr(),
                            room[32:].data_ptr(), 0, ws.data_ptr() if need.value else None, need.value,
                            torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        assert same_bits(room[32:32 + M * N].view(M, N), want)
        assert (room[:32] == 7).all() and (room[32 + M * N:] == 7).all() and (ws[need.value:] == 0xFF).all()


# ---------------------------------------------------------------- mixture of experts


def act64(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))


def layer(M, K, F, E, dtype, i8, seed=0, logits=1.5):
    """x, router, the three weights as the call takes them, scales or None, and their values in 64 bits."""
    x = rand((M, K), dtype, seed + 1)
    wr = rand((E, K), dtype, seed + 2, logits * max(1, K) ** -0.5)
    ws, scales, values = [], [], []
    for i, shape in enumerate(((E, F, K), (E, F, K), (E, K, F))):
        w = rand(shape, dtype, seed + 3 + i, max(1, shape[2]) ** -0.5)
        if i8:
            q, s = pws.gemm_i8_quantize(w.view(-1, shape[2]))
            ws.append(q.view(shape))
            scales.append(s.view(shape[:2]))
            values.append(ws[-1].double() * scales[-1].double()[..., None])
        else:
            ws.append(w)
            values.append(w.double())
    return x, wr, ws, tuple(scales) if i8 else None, values


def moe_want(x, wr, values, top_k, act, normalize, dtype):
    """(y, experts, weights, bound on y's error before its rounding) in 64 bits."""
    xd = x.double()
    M, K = x.shape
    F = values[0].shape[1]
    z = xd @ wr.double().t()
    order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :top_k]
    chosen = z.gather(1, order)
    p = torch.exp(chosen - torch.logsumexp(chosen if normalize else z, dim=1, keepdim=True))
    y, bound = torch.zeros_like(xd), torch.zeros_like(xd)
    for m in range(M):
        for j in range(top_k):
            e = int(order[m, j])
            wg, wu, wd = (v[e] for v in values)
            g, u = wg @ xd[m], wu @ xd[m]
            eg, eu = acc_error(K, wg.abs() @ xd[m].abs()), acc_error(K, wu.abs() @ xd[m].abs())
            h = p[m, j] * act64(g, act) * u
            # |act'| <= 1.13; act, p and the scales to 2^-19 relative together
            eh = p[m, j] * (1.13 * eg * (u.abs() + eu) + act64(g, act).abs() * eu) + 2.0 ** -19 * h.abs()
            eh = eh + (2.0 ** -16 * h.abs() if dtype == BF16 else 2.0 ** -22 * h.abs() + 2.0 ** -25)
            y[m] += wd @ h
            bound[m] += wd.abs() @ eh + acc_error(F, wd.abs() @ h.abs()) * 2
    # (all experts' sums of a token are one more sum of top_k terms)
    return y, order.int(), p, bound + top_k * 2.0 ** -23 * y.abs()


MOE = [(1, 64, 64, 4, 2), (1, 1024, 512, 32, 4), (1, 1030, 333, 12, 3), (1, 8, 1, 1, 1), (2, 96, 40, 5, 5), (3, 257, 129, 64, 6),
       (5, 512, 768, 16, 1), (7, 1030, 731, 12, 3), (8, 640, 256, 128, 8), (9, 130, 66, 7, 2), (16, 1024, 320, 64, 8),
       (17, 72, 96, 3, 2), (31, 500, 100, 33, 4), (32, 256, 512, 8, 2), (64, 192, 80, 6, 3), (65, 128, 64, 4, 2),
       (130, 64, 48, 9, 4), (4, 16, 4100, 3, 2), (4, 4104, 16, 3, 2), (6, 48, 32, 1024, 32)]


@pytest.mark.parametrize("i8", [False, True], ids=["16bit", "8bit"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,F,E,top_k", MOE)
def test_moe(M, K, F, E, top_k, dtype, i8):
    act, normalize = ("gelu" if (M + F) % 2 else "silu"), bool((M + E) % 2)
    x, wr, ws, scales, values = layer(M, K, F, E, dtype, i8)
    y, experts, weights = pws.gemm_moe_nt(x, wr, *ws, top_k, scales=scales, act=act, normalize=normalize)
    want, order, p, bound = moe_want(x, wr, values, top_k, act, normalize, dtype)
    assert experts.dtype == torch.int32 and torch.equal(experts, order)
    assert weights.dtype == torch.float32 and ((weights.double() - p).abs() <= 2.0 ** -20 * p + 1e-30).all()
    assert y.dtype == dtype and y.shape == x.shape
    err = (y.double() - want).abs()
    ok = err <= bound + half_unit(want.abs() + bound, dtype)
    assert ok.all(), f"{int((~ok).sum())} off, worst {float((err / (bound + half_unit(want, dtype))).max()):.3f}"


@pytest.mark.parametrize("i8", [False, True], ids=["16bit", "8bit"])
def test_moe_any_alignment(i8):
    for M, K, F in ((3, 128, 64), (20, 64, 128)):
        x, wr, ws, scales, _ = layer(M, K, F, 6, BF16, i8)
        want = pws.gemm_moe_nt(x, wr, *ws, 2, scales=scales)
        for i in range(5):
            ops = [off_by_one(t) if i == j else t for j, t in enumerate((x, wr, *ws))]
            got = pws.gemm_moe_nt(*ops, 2, scales=scales)
            assert all(same_bits(a, b) for a, b in zip(got, want)), i


@pytest.mark.parametrize("dtype", TYPES)
def test_moe_ties_go_to_the_lower_index(dtype):
    M, K, F, E = 5, 96, 32, 24
    x, wr, ws, _, _ = layer(M, K, F, E, dtype, False)
    wr[7], wr[3], wr[20] = wr[11], wr[11], wr[11]
    _, experts, weights = pws.gemm_moe_nt(x, wr, *ws, E)
    for m in range(M):
        where = [experts[m].tolist().index(e) for e in (3, 7, 11, 20)]
        assert where == list(range(where[0], where[0] + 4))
        assert len(set(weights[m, where[0]:where[0] + 4].tolist())) == 1
    assert torch.equal(experts.sort(dim=1).values, torch.arange(E, device="cuda", dtype=torch.int32).expand(M, E))
    _, experts, weights = pws.gemm_moe_nt(x, torch.zeros_like(wr), *ws, 4)
    assert torch.equal(experts, torch.arange(4, device="cuda", dtype=torch.int32).expand(M, 4)) and (weights == 0.25).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_moe_near_logits_go_by_their_true_order(dtype):
    """Logits that differ by one part in 2^33 of the terms they are sums of."""
    K, E = 2048, 8
    x = rand((4, K), dtype, 1)
    x[:, -1] = 2.0 ** -11
    row = rand((1, K), dtype, 2)
    wr = row.repeat(E, 1)
    wr[:, -1] = torch.tensor([3.0, 1.0, 7.0, 0.0, 6.0, 2.0, 5.0, 4.0], device="cuda") * 2.0 ** -12
    _, _, ws, _, _ = layer(1, K, 8, E, dtype, False)
    _, experts, _ = pws.gemm_moe_nt(x, wr.to(dtype), *ws, E)
    assert experts.tolist() == [[2, 4, 6, 7, 0, 5, 1, 3]] * 4


@pytest.mark.parametrize("dtype", TYPES)
def test_moe_nonfinite_stays_in_its_row(dtype):
    M, K, F, E = 10, 64, 48, 8
    x, wr, ws, _, _ = layer(M, K, F, E, dtype, False)
    clean = pws.gemm_moe_nt(x, wr, *ws, 2)
    x[3, 5], x[7, 0] = math.nan, math.inf
    y, experts, weights = pws.gemm_moe_nt(x, wr, *ws, 2)
    good = [m for m in range(M) if m not in (3, 7)]
    for a, b in zip((y, experts, weights), clean):
        assert same_bits(a[good], b[good])
    assert torch.isnan(y[3]).all() and torch.isnan(weights[3]).all() and ((experts >= 0) & (experts < E)).all()
    assert all(len(set(r)) == 2 for r in experts.tolist())
    assert not torch.isfinite(y[7]).any()
    # experts that no token chose may hold anything
    x, wr, ws, _, _ = layer(1, 120, 100, E, dtype, False)
    want, experts, _ = pws.gemm_moe_nt(x, wr, *ws, 2)
    for e in set(range(E)) - set(experts[0].tolist()):
        for w in ws:
            w[e] = math.nan
    assert same_bits(pws.gemm_moe_nt(x, wr, *ws, 2)[0], want)


def test_moe_ragged_rows_do_not_meet_their_neighbours():
    """Odd rows followed by others' infinities: what lies behind a row's end never reaches its sum."""
    for K, F in ((33, 70), (70, 33), (1023, 15)):
        x, wr, ws, _, values = layer(2, K, F, 3, F16, False)
        want, experts, _ = pws.gemm_moe_nt(x[:1], wr, *ws, 1)
        keep = int(experts[0, 0])
        for w in ws:
            for e in range(3):
                if e != keep:
                    w[e] = math.inf
        both = torch.cat([x[:1], torch.full_like(x[:1], math.inf)])
        y, experts, _ = pws.gemm_moe_nt(both[:1].contiguous(), wr, *ws, 1)
        assert same_bits(y, want) and int(experts[0, 0]) == keep


def test_moe_large_values():
    """bfloat16 activations beyond binary16's range, and their 8-bit weights."""
    for i8 in (False, True):
        x, wr, ws, scales, values = layer(4, 128, 96, 6, BF16, i8)
        x = x * 256
        wr = wr / 256
        y, experts, _ = pws.gemm_moe_nt(x, wr, *ws, 2, scales=scales)
        want, order, _, bound = moe_want(x, wr, values, 2, "silu", True, BF16)
        assert torch.equal(experts, order) and want.abs().max() > 1e4
        assert ((y.double() - want).abs() <= bound + half_unit(want.abs() + bound, BF16)).all()


def test_moe_empty():
    x, wr, ws, _, _ = layer(3, 64, 0, 4, F16, False)
    y, experts, weights = pws.gemm_moe_nt(x, wr, *ws, 2)
    assert not y.any() and experts.shape == (3, 2) and ((weights.sum(1) - 1).abs() < 1e-6).all()
    x, wr, ws, _, _ = layer(3, 0, 8, 4, F16, False)
    y, experts, weights = pws.gemm_moe_nt(x, wr, *ws, 2)
    assert y.shape == (3, 0) and experts.tolist() == [[0, 1]] * 3 and (weights == 0.5).all()
    x, wr, ws, _, _ = layer(0, 16, 8, 4, F16, False)
    assert [t.shape[0] for t in pws.gemm_moe_nt(x, wr, *ws, 2)] == [0, 0, 0]


# ---------------------------------------------------------------- as they are used


def serve(x, p):
    """A block as it is served in 8 bits: a quantized projection, then the experts, then the head's projection."""
    q, s = pws.gemm_i8_quantize(x)
    a = pws.gemm_i8_nt(q, p["proj"][0], s, p["proj"][1], dtype=x.dtype)
    y, experts, weights = pws.gemm_moe_nt(a, p["router"], *p["w"], 2, scales=p["scales"])
    q, s = pws.gemm_i8_quantize(y)
    return pws.gemm_i8_nt(q, p["head"][0], s, p["head"][1], dtype=x.dtype), a, y, experts, weights


def block(K, F, E, dtype):
    _, wr, ws, scales, values = layer(1, K, F, E, dtype, True)
    return {"proj": pws.gemm_i8_quantize(rand((K, K), dtype, 50, K ** -0.5)), "router": wr, "w": ws, "scales": scales,
            "head": pws.gemm_i8_quantize(rand((777, K), dtype, 51, K ** -0.5)), "values": values}


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [1, 6, 40])
def test_run_together(M, dtype):
    K, F, E = 256, 192, 10
    p = block(K, F, E, dtype)
    x = rand((M, K), dtype, 60)
    out, a, y, experts, _ = serve(x, p)
    q, s = quantized64(x)
    i8_check(a, i8_want(q, p["proj"][0], s, p["proj"][1]), dtype)
    want, order, _, bound = moe_want(a, p["router"], p["values"], 2, "silu", True, dtype)
    assert torch.equal(experts, order)
    assert ((y.double() - want).abs() <= bound + half_unit(want.abs() + bound, dtype)).all()
    q, s = quantized64(y)
    i8_check(out, i8_want(q, p["head"][0], s, p["head"][1]), dtype)


def test_graph_replay_and_streams():
    """Captured and replayed on new inputs, on a stream of its own and while another stream runs the same layer:
    the same bits as one call after the other."""
    for M in (1, 12, 40):
        p = block(128, 96, 8, BF16)
        xs = [rand((M, 128), BF16, 70 + i) for i in range(3)]
        want = [[t.clone() for t in serve(x, p)] for x in xs]
        static = xs[0].clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            serve(static, p)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = serve(static, p)
        for x, w in zip(xs, want):
            static.copy_(x)
            graph.replay()
            assert all(same_bits(a, b) for a, b in zip(got, w))
        streams = [torch.cuda.Stream() for _ in range(3)]
        outs = []
        torch.cuda.synchronize()
        for _ in range(5):
            for s, x in zip(streams, xs):
                with torch.cuda.stream(s):
                    outs.append(serve(x, p))
        torch.cuda.synchronize()
        for i, o in enumerate(outs):
            assert all(same_bits(a, b) for a, b in zip(o, want[i % 3]))


def test_a_timed_out_wait_is_reported():
    # slots that never become empty: every wait runs out, the call returns, the status word says so, and the
    # next call is whole again
    for M, N, K in ((40, 500, 4096), (24, 20000, 512), (128, 300, 1000), (300, 500, 1024)):
        a, b = rand_i8((M, K), 1), rand_i8((N, K), 2)
        ones = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
        want = pws.gemm_i8_nt(a, b, *ones, dtype=BF16)
        torch.cuda.synchronize()
        pws.gemm_set_debug_flags(pws.GEMM_DEBUG_SKIP_EMPTY_SEED)
        pws.gemm_set_wait_timeout_ns(20_000_000)
        try:
            pws.gemm_i8_nt(a, b, *ones, dtype=BF16)
            assert pws.gemm_device_status() == pws.GEMM_ERR_TIMEOUT
        finally:
            pws.gemm_set_debug_flags(0)
            pws.gemm_set_wait_timeout_ns(0)
        assert same_bits(pws.gemm_i8_nt(a, b, *ones, dtype=BF16), want)
        assert pws.gemm_device_status() == pws.GEMM_OK


def test_operands_that_require_a_gradient():
    # the calls are not recorded: said once for each
    x, wr, ws, _, _ = layer(2, 64, 32, 4, F16, False)
    pws._warned.difference_update({"gemm_i8_quantize", "gemm_moe_nt"})
    x.requires_grad_(True)
    with pytest.warns(UserWarning, match="no backward pass"):
        assert not pws.gemm_i8_quantize(x)[1].requires_grad
    with pytest.warns(UserWarning, match="no backward pass"):
        assert not pws.gemm_moe_nt(x, wr, *ws, 2)[0].requires_grad


def test_more_tokens_than_a_pass_takes():
    # each token's row is its own, in whichever pass of 64 it lies
    x, wr, ws, scales, _ = layer(200, 136, 72, 5, BF16, True)
    y, experts, weights = pws.gemm_moe_nt(x, wr, *ws, 3, scales=scales)
    for rows in (slice(0, 64), slice(64, 128), slice(128, 192), slice(192, 200)):
        got = pws.gemm_moe_nt(x[rows], wr, *ws, 3, scales=scales)
        assert all(same_bits(a, b[rows]) for a, b in zip(got, (y, experts, weights)))


def test_the_same_matrix_as_both_operands():
    for M, K in ((7, 64), (40, 200), (200, 1030)):
        a = rand_i8((M, K), M)
        s = torch.rand(M, device="cuda") * 0.01
        i8_check(pws.gemm_i8_nt(a, a, s, s), i8_want(a, a, s, s), BF16)
    x, wr, ws, _, _ = layer(5, 96, 96, 4, F16, False)
    y = pws.gemm_moe_nt(x, wr, ws[0], ws[0], ws[0], 2)[0]
    assert same_bits(y, pws.gemm_moe_nt(x, wr, ws[0], ws[0].clone(), ws[0].clone(), 2)[0])


def test_outputs_at_any_element():
    # outputs one element past a 16-byte boundary: the same bits, and nothing beside them
    lib, stream = pws.load_library(), torch.cuda.current_stream().cuda_stream
    need = pws.ctypes.c_int64()
    for M, N, K in ((3, 71, 100), (40, 130, 4096), (40, 131, 200), (200, 131, 128), (300, 256, 256)):
        a, b = rand_i8((M, K), 1), rand_i8((N, K), 2)
        ones = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
        want = pws.gemm_i8_nt(a, b, *ones, dtype=BF16)
        room = torch.full((M * N + 2,), 7.0, device="cuda", dtype=BF16)
        assert lib.gemm_i8_nt_workspace(M, N, K, a.data_ptr(), b.data_ptr(), 1, pws.ctypes.byref(need)) == 0
        ws = torch.empty(max(need.value, 1), dtype=torch.uint8, device="cuda")
        assert lib.gemm_i8_nt(M, N, K, a.data_ptr(), b.data_ptr(), ones[0].data_ptr(), ones[1].data_ptr(), room[1:].data_ptr(), 1,
                              ws.data_ptr(), need.value, stream) == 0
        assert same_bits(room[1:-1].view(M, N), want) and room[0] == 7 and room[-1] == 7
    for M, K, F, E, top_k in ((2, 71, 40, 4, 2), (70, 136, 72, 5, 3)):
        x, wr, ws3, _, _ = layer(M, K, F, E, BF16, False)
        want = pws.gemm_moe_nt(x, wr, *ws3, top_k)
        y = torch.full((M * K + 2,), 7.0, device="cuda", dtype=BF16)
        e, p = torch.full((M * top_k + 2,), 7, device="cuda", dtype=torch.int32), torch.full((M * top_k + 2,), 7.0, device="cuda")
        assert lib.gemm_moe_nt_workspace(M, K, F, E, top_k, 1, 1, pws.ctypes.byref(need)) == 0
        ws = torch.full((need.value + 256,), 0xFF, dtype=torch.uint8, device="cuda")
        assert lib.gemm_moe_nt(M, K, F, E, top_k, x.data_ptr(), wr.data_ptr(), *(w.data_ptr() for w in ws3), None, None, None,
                               y[1:].data_ptr(), e[1:].data_ptr(), p[1:].data_ptr(), 1, 1, 0, 1, ws.data_ptr(), need.value, stream) == 0
        for got, t in zip((y, e, p), want):
            assert same_bits(got[1:-1].view(t.shape), t) and got[0] == 7 and got[-1] == 7
        assert (ws[need.value:] == 0xFF).all()


def test_weights_written_just_before_the_call():
    # the weights' last writer is the kernel before the call, on the call's stream, captured and not
    M, N, K = 24, 20000, 512
    sides = [(rand_i8((M, K), i), rand_i8((N, K), 10 + i)) for i in range(2)]
    ones = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    want = [pws.gemm_i8_nt(a, b, *ones) for a, b in sides]
    x, wr, ws3, _, _ = layer(5, 512, 256, 6, BF16, False)
    other = [w.flip(1).contiguous() for w in ws3]
    want_y = [pws.gemm_moe_nt(x, wr, *w, 2)[0] for w in (ws3, other)]
    a, b, held = sides[0][0].clone(), sides[0][1].clone(), [w.clone() for w in ws3]
    source = [[t.clone() for t in (*side, *w)] for side, w in zip(sides, (ws3, other))]

    def step(i):
        for to, t in zip((a, b, *held), source[i]):
            to.copy_(t)
        return pws.gemm_i8_nt(a, b, *ones), pws.gemm_moe_nt(x, wr, *held, 2)[0]

    graphs = []
    for i in range(2):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, step(i)))
    for turn in range(20):
        i = turn % 2
        got = step(i)
        assert same_bits(got[0], want[i]) and same_bits(got[1], want_y[i])
        graphs[i][0].replay()
        assert same_bits(graphs[i][1][0], want[i]) and same_bits(graphs[i][1][1], want_y[i])


def test_calls_from_several_threads():
    import threading
    sizes = [(1, 300, 512), (24, 20000, 512), (100, 260, 1030), (300, 512, 256)]
    p = block(128, 96, 8, F16)
    inputs = [(rand_i8((M, K), M), rand_i8((N, K), N), rand((3 + i, 128), F16, i)) for i, (M, N, K) in enumerate(sizes)]
    ones = torch.ones(20000, device="cuda")

    def step(a, b, x):
        return (pws.gemm_i8_nt(a, b, ones[:a.shape[0]], ones[:b.shape[0]]),) + serve(x, p)

    want = [step(*i) for i in inputs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    if not all(same_bits(g, w) for g, w in zip(step(*inputs[i]), want[i])):
                        wrong.append(i)
        except Exception as e:              # (a thread's exception is not the test's)
            wrong.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_stream_argument():
    s = torch.cuda.Stream()
    x, wr, ws, _, _ = layer(2, 64, 32, 4, F16, False)
    torch.cuda.synchronize()
    want = pws.gemm_moe_nt(x, wr, *ws, 2)
    got = pws.gemm_moe_nt(x, wr, *ws, 2, stream=s)
    q, sc = pws.gemm_i8_quantize(x, stream=s)
    out = pws.gemm_i8_nt(q, q, sc, sc, stream=s)
    s.synchronize()
    assert all(same_bits(a, b) for a, b in zip(got, want))
    assert same_bits(out, pws.gemm_i8_nt(q, q, sc, sc))
    assert pws.gemm_device_status(s) == pws.GEMM_OK


# ---------------------------------------------------------------- as a served layer runs


def moe_want_by_expert(x, wr, ws, scales, top_k, act, normalize, held):
    """moe_want with an expert's tokens at once; held(h): how far h' may be from its value as it is held."""
    xd = x.double()
    M, K = x.shape
    F = ws[0].shape[1]
    z = xd @ wr.double().t()
    order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :top_k]
    chosen = z.gather(1, order)
    p = torch.exp(chosen - torch.logsumexp(chosen if normalize else z, dim=1, keepdim=True))
    y, bound = torch.zeros_like(xd), torch.zeros_like(xd)
    for e in order.unique().tolist():
        token, slot = torch.nonzero(order == e, as_tuple=True)
        wg, wu, wd = (w[e].double() if scales is None else w[e].double() * s[e].double()[:, None] for w, s in zip(ws, scales or ws))
        xe, pe = xd[token], p[token, slot][:, None]
        g, u = xe @ wg.t(), xe @ wu.t()
        eg, eu = acc_error(K, xe.abs() @ wg.abs().t()), acc_error(K, xe.abs() @ wu.abs().t())
        a = act64(g, act)
        h = pe * a * u
        # |act'| <= 1.13; act, p and the scales to 2^-19 relative together
        eh = pe * (1.13 * eg * (u.abs() + eu) + a.abs() * eu) + 2.0 ** -19 * h.abs() + held(h)
        size = h.abs() @ wd.abs().t()
        y.index_add_(0, token, h @ wd.t())
        # (h is two or three 16-bit values, each with sums of its own)
        bound.index_add_(0, token, eh @ wd.abs().t() + acc_error(F, size) * 3)
    return y, order.int(), p, bound + top_k * 2.0 ** -23 * y.abs()


def held_in_two(dtype):
    """h' as two 16-bit values, as in moe_want."""
    return (lambda h: 2.0 ** -16 * h.abs()) if dtype == BF16 else (lambda h: 2.0 ** -22 * h.abs() + 2.0 ** -25)


# More units of work than blocks, claimed or in turn: rings that run on over units, row blocks whose last entry another block
# finished, 1 to 8 groups of rows a unit, one and two tiles of tokens, each in rows of whole 16 bytes and in ragged ones.
# (The groups of 32 rows of a gate and of a down unit, on 152 SMs; an expert's tokens.)
SERVED = [(1, 4096, 2048, 64, 6, False), (1, 4096, 2048, 64, 6, True),         # 1, 1; one
          (16, 4096, 1536, 64, 8, False), (16, 4098, 1531, 64, 8, False),      # 1, 4; two
          (16, 4096, 1536, 64, 8, True),                                       # 2, 8; two
          (32, 4096, 2048, 32, 4, True), (32, 4099, 2050, 32, 4, True),        # 2, 4; four
          (64, 4096, 128, 128, 8, False),                                      # 1, 8; four
          (48, 1024, 1056, 64, 4, False), (48, 1022, 1058, 64, 4, False),      # 4, 2; three
          (64, 2048, 4096, 8, 2, False), (64, 2050, 4100, 8, 2, False),        # 2, 1; sixteen, in tiles of two
          (64, 2048, 4096, 8, 2, True), (64, 2050, 4100, 8, 2, True),          # 2 or 4, 1; the same
          (64, 1000, 2049, 64, 8, True), (64, 4096, 512, 32, 8, False)]        # 8, 4 and 1, 4; eight and sixteen


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,F,E,top_k,i8", SERVED)
def test_moe_served(M, K, F, E, top_k, i8, dtype):
    act, normalize = ("gelu" if E % 64 else "silu"), bool(M % 32)
    x, wr, ws, scales = layer(M, K, F, E, dtype, i8)[:4]
    y, experts, weights = pws.gemm_moe_nt(x, wr, *ws, top_k, scales=scales, act=act, normalize=normalize)
    want, order, p, bound = moe_want_by_expert(x, wr, ws, scales, top_k, act, normalize, held_in_two(dtype))
    assert torch.equal(experts, order) and ((weights.double() - p).abs() <= 2.0 ** -20 * p + 1e-30).all()
    err = (y.double() - want).abs()
    ok = err <= bound + half_unit(want.abs() + bound, dtype)
    assert ok.all(), f"{int((~ok).sum())} off, worst {float((err / (bound + half_unit(want, dtype))).max()):.3f}"
    # units finished in another order give the same bits
    junk, side = torch.empty(1 << 26, device="cuda"), torch.cuda.Stream()
    for i in range(6):
        with torch.cuda.stream(side):
            junk.mul_(1.0)
        assert same_bits(pws.gemm_moe_nt(x, wr, *ws, top_k, scales=scales, act=act, normalize=normalize)[0], y)
    torch.cuda.synchronize()


def held_in_fp32(dtype, i8):
    """h in fp32, then as three bfloat16 values (all 24 bits), or as two binary16 ones of a multiple whose largest magnitude is
    2^14 or more: 11 bits, 11 bits of the rest, and half of binary16's smallest step, 2^-25."""
    if dtype == BF16 and not i8:
        return lambda h: 2.0 ** -24 * h.abs()
    return lambda h: (2.0 ** -24 + 2.0 ** -22) * h.abs() + 2.0 ** -39 * h.abs().amax(dim=1, keepdim=True)


def moe_in_range(x, wr, ws, scales, top_k, act, dtype):
    y, experts, weights = pws.gemm_moe_nt(x, wr, *ws, top_k, scales=scales, act=act, normalize=False)
    want, order, p, bound = moe_want_by_expert(x, wr, ws, scales, top_k, act, False, held_in_fp32(dtype, scales is not None))
    assert torch.equal(experts, order)
    assert torch.isfinite(want).all() and want.abs().max() < 60000 and want.abs().median() > (2.0 ** -13 if dtype == F16 else 0)
    err = (y.double() - want).abs()
    ok = err <= bound + half_unit(want.abs() + bound, dtype)
    assert ok.all(), f"{int((~ok).sum())} of {ok.numel()} off, worst {float((err / (bound + half_unit(want, dtype))).max()):.3f}"
    return want


# what x is multiplied by, and what the 8-bit gate's and up's scales are: h from 1e-20 to 1e20
@pytest.mark.parametrize("size,more", [(400.0, 1.0), (150.0, 1.0), (1e4, 1.0), (3e-3, 1.0), (1e-2, 1.0), (1e4, 1e6), (1e-2, 1e-8)])
@pytest.mark.parametrize("M,F", [(3, 160), (6, 1024), (40, 96)])
@pytest.mark.parametrize("dtype", TYPES)
def test_moe_activations_of_any_size(M, F, size, more, dtype):
    """y is off by its rounding and fp32's sums whatever the activations between the projections are: beyond binary16's largest
    value, and below its smallest."""
    K, E, top_k = 128, 6, 2
    for i8 in (False, True):
        if more != 1.0 and not i8:
            continue
        act = "gelu" if M % 2 else "silu"
        x, wr, ws, scales, _ = layer(M, K, F, E, dtype, i8, seed=M)
        x, wr = (x.float() * size).to(dtype), (wr.float() / size).to(dtype)
        # g and u are about size * more; an activation below 1 is about half of g
        h = (size * more) ** 2 * (1.0 if size * more > 1 else 0.5)
        back = (100.0 if dtype == F16 else 1.0) / h
        if i8:
            scales = (scales[0] * more, scales[1] * more, scales[2] * back)
        else:
            ws[2] = (ws[2].float() * min(back, 2000.0)).to(dtype)
        if not i8 and min(back, 2000.0) * h < 0.05:
            continue
        moe_in_range(x, wr, ws, scales, top_k, act, dtype)


@pytest.mark.parametrize("i8", [False, True], ids=["16bit", "8bit"])
def test_moe_activations_across_the_end_of_binary16(i8):
    """One token, one expert, one column: h a little below and above 65504, 65520 and 131008."""
    for h in (65000.0, 65504.0, 65519.0, 65520.0, 65536.0, 70000.0, 100000.0, 131000.0, 131008.0, 131072.0, 1e6, 2.6e8):       # (u itself is binary16: below 2^28)
        K = 16
        x = torch.zeros(1, K, device="cuda", dtype=F16)
        x[0, 0], x[0, 1] = 64.0, 1.0
        one = torch.zeros(1, 1, K, device="cuda", dtype=F16)
        one[0, 0, 0] = 1.0                                          # g = 64: silu(64) is 64 to 2^-90
        up = torch.zeros(1, 1, K, device="cuda", dtype=F16)
        up[0, 0, 0] = h / 64 / 64                                   # u = 64 up
        down = torch.full((1, K, 1), 2.0 ** -14, device="cuda", dtype=F16)
        ws, scales = [one, up, down], None
        if i8:
            q = [pws.gemm_i8_quantize(w.view(-1, w.shape[2])) for w in ws]
            ws, scales = [a.view(w.shape) for (a, _), w in zip(q, ws)], tuple(c.view(w.shape[:2]) for (_, c), w in zip(q, ws))
        want = moe_in_range(x, torch.zeros(1, K, device="cuda", dtype=F16), ws, scales, 1, "silu", F16)
        assert abs(float(want[0, 0]) / (h * 2.0 ** -14) - 1) < 0.01


@pytest.mark.parametrize("i8", [False, True], ids=["16bit", "8bit"])
@pytest.mark.parametrize("dtype", TYPES)
def test_moe_activations_of_different_tokens(dtype, i8):
    """Each token's activations are held by their own size: rows 2^30 apart in one call, each as when it is alone."""
    M, K, F, E = 31, 64, 200, 4
    x, wr, ws, scales, _ = layer(M, K, F, E, dtype, i8)
    x = (x.float() * torch.exp2(torch.arange(M, device="cuda") / 2.0 - 7.0)[:, None]).to(dtype)
    wr = (wr.float() / 16).to(dtype)
    ws[2], scales = (ws[2], scales[:2] + (scales[2] / 64,)) if i8 else ((ws[2].float() / 64).to(dtype), None)
    y, experts, _ = pws.gemm_moe_nt(x, wr, *ws, 2, scales=scales)
    want, order, _, bound = moe_want_by_expert(x, wr, ws, scales, 2, "silu", True, held_in_fp32(dtype, i8))
    assert torch.equal(experts, order)
    assert ((y.double() - want).abs() <= bound + half_unit(want.abs() + bound, dtype)).all()


@pytest.mark.parametrize("i8", [False, True], ids=["16bit", "8bit"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [1, 8, 40])
def test_moe_activations_that_cancel(M, dtype, i8):
    """h of two columns, a part in 2^12 apart, with weights of opposite sign: what is left shows to how many bits h is held."""
    K = 8
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.zeros(M, K, device="cuda")
    x[:, 0] = torch.randint(33, 65, (M,), generator=g, device="cuda")
    x[:, 1] = 1
    x[:, 2] = torch.rand(M, generator=g, device="cuda") * 4 + 0.5
    x = x.to(dtype)
    wg, wu, wd = torch.zeros(1, 2, K, device="cuda"), torch.zeros(1, 2, K, device="cuda"), torch.zeros(1, K, 2, device="cuda")
    wg[0, :, 2] = 1                                     # g = x_2
    wu[0, :, 0], wu[0, 1, 1] = 64, 1                    # u = 64 x_0 and 64 x_0 + 1, exactly
    wd[0, :, 0] = torch.arange(1, K + 1)
    wd[0, :, 1] = -wd[0, :, 0]
    kind = torch.int8 if i8 else dtype
    scales = (torch.ones(1, 2, device="cuda"), torch.ones(1, 2, device="cuda"), torch.ones(1, K, device="cuda")) if i8 else None
    y = pws.gemm_moe_nt(x, torch.zeros(1, K, device="cuda", dtype=dtype), *(w.to(kind) for w in (wg, wu, wd)), 1, scales=scales)[0]
    a, u = act64(x[:, 2:3].double(), "silu"), 64 * x[:, 0:1].double()
    want = -a * wd[0, :, 0].double()
    # a's error is the same in both columns; each h is rounded to fp32 and held; sums as in acc_error
    size = (a * (2 * u + 1)).abs()
    bound = 2.0 ** -19 * want.abs() + wd[0, :, 0].double() * (2.0 ** -24 + (2.0 ** -24 if dtype == BF16 and not i8 else 2.0 ** -22)) * size
    bound = bound + acc_error(2, wd[0, :, 0].double() * size) * 3
    err = (y.double() - want).abs()
    assert (err <= bound + half_unit(want.abs() + bound, dtype)).all(), float((err / (bound + half_unit(want, dtype))).max())


@pytest.mark.parametrize("dtype", TYPES)
def test_moe_infinite_activations(dtype):
    """h beyond fp32: its token's y is an infinity of the weight's sign, and NaN at a weight of zero, as products with it are; no other
    token's changes."""
    K, size = 16, 1e4
    x = torch.zeros(3, K, device="cuda", dtype=dtype)
    x[:, 0] = torch.tensor([1.0, size, 2.0], device="cuda")
    ones = [torch.zeros(1, 40, K, device="cuda", dtype=torch.int8) for _ in range(2)]
    for w in ones:
        w[0, :, 0] = 1
    down = torch.zeros(1, K, 40, device="cuda", dtype=torch.int8)
    down[0, 0], down[0, 1] = 3, -2
    s = torch.full((1, 40), 1e16, device="cuda")
    scales = (s, s, torch.full((1, K), 1e-33, device="cuda"))
    wr = torch.zeros(1, K, device="cuda", dtype=dtype)
    y = pws.gemm_moe_nt(x, wr, *ones, down, 1, scales=scales)[0]
    assert y[1, 0] == math.inf and y[1, 1] == -math.inf and torch.isnan(y[1, 2:]).all()
    for m in (0, 2):
        assert torch.isfinite(y[m]).all()
        assert same_bits(y[m:m + 1], pws.gemm_moe_nt(x[m:m + 1], wr, *ones, down, 1, scales=scales)[0])
    if dtype == BF16:
        x[1, 0] = 1e20
        w = [t.to(dtype) for t in (*ones, down)]
        y = pws.gemm_moe_nt(x, wr, *w, 1)[0]
        assert y[1, 0] == math.inf and y[1, 1] == -math.inf and torch.isnan(y[1, 2:]).all() and torch.isfinite(y[[0, 2]]).all()


def test_scales_that_require_a_gradient():
    # learned scales: the calls are not recorded for them either
    x, wr, ws, scales, _ = layer(2, 64, 32, 4, F16, True)
    q, s = pws.gemm_i8_quantize(x)
    for which in range(2):
        pws._warned.discard("gemm_i8_nt")
        pair = [s.clone().requires_grad_(which == i) for i in range(2)]
        with pytest.warns(UserWarning, match="no backward pass"):
            assert not pws.gemm_i8_nt(q, q, *pair).requires_grad
    for which in range(3):
        pws._warned.discard("gemm_moe_nt")
        three = tuple(c.clone().requires_grad_(which == i) for i, c in enumerate(scales))
        with pytest.warns(UserWarning, match="no backward pass"):
            assert not pws.gemm_moe_nt(x, wr, *ws, 2, scales=three)[0].requires_grad


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [(1, 64, 256), (20, 96, 256), (40, 130, 8200), (100, 96, 256), (300, 260, 256)])
def test_i8_scales_at_the_ends_of_their_range(M, N, K, dtype):
    """Either scale so large that it takes the sum out of fp32's range alone, or below its normal range: the other brings the element back."""
    a, b = rand_i8((M, K), 1), rand_i8((N, K), 2)
    a[0], b[0] = 127, 127                                   # (one sum of the largest)
    total = (a.double() @ b.double().t()).abs().max()
    assert total * 3e37 > 3.5e38
    for large, small in ((3e37, 2.0 ** -140), (3.4e38, 3 * 2.0 ** -148), (1e33, 1e-35), (2.0 ** 91, 2.0 ** -93), (2.0 ** 100, 2.0 ** -126)):
        for first in (large, small):
            sa = torch.full((M,), first, device="cuda")
            sb = torch.full((N,), small if first == large else large, device="cuda")
            # (to at most 30000 in binary16)
            if float(total) * large * small > 30000:
                (sa if first == small else sb).mul_(2.0 ** -math.ceil(math.log2(float(total) * large * small / 30000)))
            want = i8_want(a, b, sa, sb)
            assert 0 < want.abs().max() < 65504
            i8_check(pws.gemm_i8_nt(a, b, sa, sb, dtype=dtype), want, dtype)


def test_a_limit_shorter_than_a_copy():
    """Waits that give up while the tokens' copies are on their way: the call says so or is right, and so is the next one."""
    for M, N, K in ((40, 500, 4096), (24, 20000, 512), (100, 300, 256), (128, 300, 1030), (200, 500, 8200)):
        a, b = rand_i8((M, K), 1), rand_i8((N, K), 2)
        ones = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
        want = pws.gemm_i8_nt(a, b, *ones, dtype=BF16)
        torch.cuda.synchronize()
        for limit in (1, 1000, 4000):
            pws.gemm_set_wait_timeout_ns(limit)
            try:
                out = pws.gemm_i8_nt(a, b, *ones, dtype=BF16)
                status = pws.gemm_device_status()
                assert status == pws.GEMM_ERR_TIMEOUT or (status == pws.GEMM_OK and same_bits(out, want))
            finally:
                pws.gemm_set_wait_timeout_ns(0)
            assert same_bits(pws.gemm_i8_nt(a, b, *ones, dtype=BF16), want)
            assert pws.gemm_device_status() == pws.GEMM_OK


@pytest.mark.parametrize("M,N,K", [(600, 1100, 2050), (700, 1500, 2050), (700, 1500, 2064), (520, 2000, 4100)])
def test_i8_ragged_weights_on_both_sides_of_a_tile_count(M, N, K):
    a, b = rand_i8((M, K), M), rand_i8((N, K), N)
    sa, sb = rand((M,), torch.float32, 3).abs() * 0.02 + 0.001, rand((N,), torch.float32, 4).abs() * 0.02 + 0.001
    out = pws.gemm_i8_nt(a, b, sa, sb, dtype=BF16)
    i8_check(out, i8_want(a, b, sa, sb), BF16)
    for ops in ((off_by_one(a), b), (a, off_by_one(b))):
        assert same_bits(pws.gemm_i8_nt(*ops, sa, sb, dtype=BF16), out)


@pytest.mark.parametrize("i8", [False, True], ids=["16bit", "8bit"])
@pytest.mark.parametrize("M", [1, 7, 30, 70])
def test_moe_sizes_of_the_call_before_do_not_linger(M, i8):
    """Calls in turn on the same workspace, captured and not, whose activations are 2^40 apart: each as when it ran first."""
    x, wr, ws, scales, _ = layer(M, 128, 192, 6, F16, i8)
    ws[2], scales = (ws[2], scales[:2] + (scales[2] / 64,)) if i8 else ((ws[2].float() / 64).to(F16), scales)
    xs = [(x.float() * 2.0 ** k).to(F16) for k in (0, 10, -10, 10, 0, -10)]
    want = [pws.gemm_moe_nt(v, wr, *ws, 2, scales=scales)[0] for v in xs]
    torch.cuda.synchronize()
    lone = []
    for v in xs:
        # (another workspace, full of another call's remains)
        junk = torch.full((1 << 20,), 0x7E7E7E7E, dtype=torch.int32, device="cuda")
        del junk
        lone.append(pws.gemm_moe_nt(v, wr, *ws, 2, scales=scales)[0])
        torch.cuda.synchronize()
    static = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = pws.gemm_moe_nt(static, wr, *ws, 2, scales=scales)[0]
    for _ in range(10):
        for v, w, a in zip(xs, want, lone):
            static.copy_(v)
            graph.replay()
            assert torch.isfinite(w).all() and same_bits(got, w) and same_bits(a, w)


@pytest.mark.parametrize("i8", [False, True], ids=["16bit", "8bit"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,F,E", [(64, 203, 130, 40), (64, 208, 128, 1024), (70, 64, 77, 33), (64, 2050, 96, 36)])
def test_moe_as_many_choices_as_there_can_be(M, K, F, E, dtype, i8):
    x, wr, ws, scales, _ = layer(M, K, F, E, dtype, i8)
    y, experts, weights = pws.gemm_moe_nt(x, wr, *ws, 32, scales=scales, normalize=False)
    want, order, p, bound = moe_want_by_expert(x, wr, ws, scales, 32, "silu", False, held_in_fp32(dtype, i8))
    assert torch.equal(experts, order) and ((weights.double() - p).abs() <= 2.0 ** -20 * p + 1e-30).all()
    assert ((y.double() - want).abs() <= bound + half_unit(want.abs() + bound, dtype)).all()

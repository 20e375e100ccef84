"""The operators around the products on the GPU: the gated feed-forward block,
softmax cross entropy over a linear head and the linear layer's backward pass,
against their formulas in 64 bits.

Every tolerance is an error bound of the computation, elementwise:

* a sum of K products on the tensor cores adds 16 of them at a time into an
  fp32 accumulator.  Each of the K/16 additions loses at most one unit in the
  last place of a partial sum no larger than S = sum |a b|, and the sum inside
  a group of 16 at most 8 more: (K/16 + 8) 2^-23 S;
* rounding to 16 bits: half a unit, 2^-11 |y| in binary16 (11 significant bits;
  2^-25 below its normal range), 2^-8 |y| in bfloat16 (8 significant bits);
* exp2 and the fast division are good to 2^-20 relative with their arguments'
  rounding, for arguments below 32 in magnitude.
"""
import math

import pytest

torch = pytest.importorskip("torch")

import pipelined_warp_specialized_gb300 as pws  # noqa: E402

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
TYPES = [F16, BF16]
IGNORE = -100


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


def unaligned(t):
    """The same values at an address one element past a 16-byte boundary."""
    flat = torch.empty(t.numel() + 8, dtype=t.dtype, device=t.device)
    out = flat[1:1 + t.numel()].view(t.shape)
    out.copy_(t)
    assert out.data_ptr() % 16 == 2
    return out


def check(got, want, tol, dtype):
    assert got.dtype == dtype and got.shape == want.shape
    err = (got.double() - want).abs()
    bound = tol + half_unit(want.abs() + tol, dtype)
    bad = ~(err <= bound)
    assert not bad.any(), f"{int(bad.sum())} off, worst {float((err / bound).max()):.3f} of the bound"


def act64(g, act):
    """act(g) and act'(g) in float64."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


# ---------------------------------------------------------------- gated block

GATED = [(1, 64, 64), (1, 4096, 1024), (1, 333, 130), (2, 16, 8), (8, 100, 72), (31, 1000, 2048), (64, 257, 96),
         (65, 512, 512), (128, 2736, 1024), (129, 640, 200), (300, 3000, 2050), (1000, 128, 1), (5, 1, 7),
         (700, 2052, 640), (2048, 1536, 768)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,F,K", GATED)
def test_gated(M, F, K, dtype):
    act = "gelu" if (M + F) % 2 else "silu"
    x, wg, wu = rand((M, K), dtype, 1), rand((F, K), dtype, 2, K ** -0.5), rand((F, K), dtype, 3, K ** -0.5)
    h, g, u = pws.gemm_gated_nt(x, wg, wu, act=act, save=True)
    alone = pws.gemm_gated_nt(x, wg, wu, act=act)
    assert torch.equal(alone.view(torch.int16), h.view(torch.int16))
    xd, gd, ud = x.double(), wg.double(), wu.double()
    g64, u64 = xd @ gd.t(), xd @ ud.t()
    eg, eu = acc_error(K, xd.abs() @ gd.abs().t()), acc_error(K, xd.abs() @ ud.abs().t())
    check(g, g64, eg, dtype)
    check(u, u64, eu, dtype)
    a64, _ = act64(g64, act)
    # |act'| <= 1.13 for both; the activation itself to 2^-20 relative
    eh = 1.13 * eg * (u64.abs() + eu) + a64.abs() * eu + 2.0 ** -20 * (a64 * u64).abs()
    check(h, a64 * u64, eh, dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_gated_any_alignment(dtype):
    # every operand one element off a 16-byte boundary gives the same bits
    for M, F, K in [(33, 200, 64), (300, 520, 256)]:
        x, wg, wu = rand((M, K), dtype, 4), rand((F, K), dtype, 5, 0.1), rand((F, K), dtype, 6, 0.1)
        want = pws.gemm_gated_nt(x, wg, wu)
        for i in range(3):
            ops = [unaligned(t) if i == j else t for j, t in enumerate((x, wg, wu))]
            assert torch.equal(pws.gemm_gated_nt(*ops).view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("dtype", TYPES)
def test_gated_saturates(dtype):
    # gates far out on both sides, infinities and NaN in one row only
    K, F = 64, 96
    x = torch.zeros(6, K, device="cuda", dtype=dtype)
    for i, v in enumerate((60.0, -60.0, 3000.0, -3000.0, 0.0)):
        x[i, 0] = v
    x[5] = float("nan")
    wg, wu = torch.zeros(F, K, device="cuda", dtype=dtype), torch.zeros(F, K, device="cuda", dtype=dtype)
    wg[:, 0], wu[:, 0] = 1.0, 0.5
    for act in ("silu", "gelu"):
        h = pws.gemm_gated_nt(x, wg, wu, act=act).double()
        assert torch.isnan(h[5]).all()
        for i in range(5):
            v = float(x[i, 0])          # (as the type holds it)
            want = float(act64(torch.tensor(v, dtype=torch.float64), act)[0]) * 0.5 * v
            if dtype == F16 and want > 65504:
                assert torch.isinf(h[i]).all()
            else:
                # half a unit, and 2^-12 for exp's argument of up to 87 and more
                assert ((h[i] - want).abs() <= abs(want) * (2.0 ** -8 + 2.0 ** -12) + 2.0 ** -25).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,F,K", GATED)
def test_gated_bwd(M, F, K, dtype):
    act = "silu" if (M + F) % 2 else "gelu"
    x, wg, wu = rand((M, K), dtype, 11), rand((F, K), dtype, 12, K ** -0.5), rand((F, K), dtype, 13, K ** -0.5)
    g, u, dh = rand((M, F), dtype, 14), rand((M, F), dtype, 15), rand((M, F), dtype, 16, 0.02)
    dx, dwg, dwu = pws.gemm_gated_nt_bwd(dh, g, u, x, wg, wu, act=act)
    value, slope = act64(g.double(), act)
    dg, du = dh.double() * u.double() * slope, dh.double() * value
    # their fp32 computation, then their rounding to the type (twice over, the
    # remainder's, for up to 64 rows: no more than half a unit of half a unit)
    small = 2.0 ** -19 * (dh.double().abs() * (u.double().abs() + 1) * (1 + g.double().abs()))
    rounding = (lambda t: half_unit(t, dtype) * 2.0 ** -8 + 2.0 ** -25) if M <= 64 else (lambda t: half_unit(t, dtype))
    eg, eu = small + rounding(dg.abs() + small), small + rounding(du.abs() + small)
    wgd, wud, xd = wg.double(), wu.double(), x.double()
    # (with remainders every sum has twice the terms)
    check(dx, dg @ wgd + du @ wud,
          eg @ wgd.abs() + eu @ wud.abs() + acc_error(4 * F, dg.abs() @ wgd.abs() + du.abs() @ wud.abs()), dtype)
    check(dwg, dg.t() @ xd, eg.t() @ xd.abs() + acc_error(2 * M, dg.abs().t() @ xd.abs()), dtype)
    check(dwu, du.t() @ xd, eu.t() @ xd.abs() + acc_error(2 * M, du.abs().t() @ xd.abs()), dtype)
    # each side alone gives the same values to the bound of their two sums
    only_dx, none_g, none_u = pws.gemm_gated_nt_bwd(dh, g, u, x, wg, wu, act=act, need_dw=False)
    none_x, only_g, only_u = pws.gemm_gated_nt_bwd(dh, g, u, x, wg, wu, act=act, need_dx=False)
    assert none_g is None and none_u is None and none_x is None
    check(only_dx, dg @ wgd + du @ wud,
          eg @ wgd.abs() + eu @ wud.abs() + acc_error(4 * F, dg.abs() @ wgd.abs() + du.abs() @ wud.abs()), dtype)
    check(only_g, dg.t() @ xd, eg.t() @ xd.abs() + acc_error(2 * M, dg.abs().t() @ xd.abs()), dtype)
    check(only_u, du.t() @ xd, eu.t() @ xd.abs() + acc_error(2 * M, du.abs().t() @ xd.abs()), dtype)


def test_gated_bwd_overflow_is_infinite():
    # a dg past binary16's range is infinite, not NaN, with and without the
    # remainders that few rows carry
    for M in (2, 100):
        F = K = 64
        one = torch.ones(F, K, device="cuda", dtype=F16)
        g, u = torch.full((M, F), 10.0, device="cuda", dtype=F16), torch.full((M, F), 100.0, device="cuda", dtype=F16)
        dh = torch.full((M, F), 60000.0, device="cuda", dtype=F16)
        x = torch.ones(M, K, device="cuda", dtype=F16)
        for t in pws.gemm_gated_nt_bwd(dh, g, u, x, one, one):
            assert torch.isposinf(t).all()


def test_gated_gradient_against_differences():
    # the directional difference of sum(dh * h) in float64 against the gradients
    M, F, K, dtype = 24, 80, 48, F16
    for act in ("silu", "gelu"):
        x, wg, wu, dh = rand((M, K), dtype, 21), rand((F, K), dtype, 22, 0.15), rand((F, K), dtype, 23, 0.15), \
            rand((M, F), dtype, 24)
        _, g, u = pws.gemm_gated_nt(x, wg, wu, act=act, save=True)
        grads = pws.gemm_gated_nt_bwd(dh, g, u, x, wg, wu, act=act)
        at = [x.double(), wg.double(), wu.double()]

        def value(x, wg, wu):
            return (dh.double() * act64(x @ wg.t(), act)[0] * (x @ wu.t())).sum()

        for i in range(3):
            d = torch.sign(rand(at[i].shape, torch.float32, 30 + i)).double()
            e = 1e-5
            hi, lo = [list(at), list(at)]
            hi[i], lo[i] = at[i] + e * d, at[i] - e * d
            diff = (value(*hi) - value(*lo)) / (2 * e)
            # half a unit of each gradient, and g and u rounded to binary16
            # (2^-11 relative), whose effect on dg, du is below 2^-9 relative;
            # independent errors would be far below this sum
            bound = (grads[i].double().abs() * 2.0 ** -8 + 2.0 ** -8 * grads[i].double().abs().mean()).sum()
            assert abs(float(diff - (grads[i].double() * d).sum())) <= float(bound)


# ---------------------------------------------------------------- linear backward

LINEAR = [(1, 1, 1), (1, 40, 72), (64, 64, 64), (7, 9, 8200), (300, 1023, 513), (1024, 1024, 1024), (4096, 64, 128),
          (130, 4100, 264), (9000, 24, 40), (513, 2048, 1536), (2, 5000, 64)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear_bwd(M, N, K, dtype):
    dy, x, w = rand((M, N), dtype, 41), rand((M, K), dtype, 42), rand((N, K), dtype, 43, 0.1)
    dx, dw = pws.gemm_nt_bwd(dy, x, w)
    d, xd, wd = dy.double(), x.double(), w.double()
    for got, want, tol in ((dx, d @ wd, acc_error(N, d.abs() @ wd.abs())),
                           (dw, d.t() @ xd, acc_error(M, d.abs().t() @ xd.abs()))):
        check(got, want, tol, dtype)
    only_dx, none = pws.gemm_nt_bwd(dy, x, w, need_dw=False)
    assert none is None
    check(only_dx, d @ wd, acc_error(N, d.abs() @ wd.abs()), dtype)
    none, only_dw = pws.gemm_nt_bwd(dy, x, w, need_dx=False)
    assert none is None
    check(only_dw, d.t() @ xd, acc_error(M, d.abs().t() @ xd.abs()), dtype)


@pytest.mark.parametrize("M,N,K", [(8200, 8200, 520), (8200, 8200, 1030), (2050, 16400, 1032)])
def test_linear_bwd_long(M, N, K):
    # K loops of 129 blocks and more: the wide tile alone, for both products,
    # with stores TMA cannot make, and with a split
    dy, x, w = rand((M, N), BF16, 44), rand((M, K), BF16, 45), rand((N, K), BF16, 46, 0.1)
    d, xd, wd = dy.double(), x.double(), w.double()
    want = ((d @ wd, acc_error(N, d.abs() @ wd.abs())), (d.t() @ xd, acc_error(M, d.abs().t() @ xd.abs())))
    for needs in (dict(), dict(need_dw=False), dict(need_dx=False)):
        for got, (ref, tol) in zip(pws.gemm_nt_bwd(dy, x, w, **needs), want):
            if got is not None:
                check(got, ref, tol, BF16)


def test_linear_bwd_exact_on_small_integers():
    # sums that fp32 and binary16 hold exactly have one right answer, whatever
    # the tile, split or schedule
    for M, N, K in [(200, 300, 130), (1024, 64, 4096), (64, 2048, 64), (3000, 200, 520), (40, 33, 2000), (8200, 8256, 520)]:
        g = torch.Generator(device="cuda").manual_seed(M)
        dy, x, w = (torch.randint(-1, 2, s, generator=g, device="cuda").half() for s in ((M, N), (M, K), (N, K)))
        dx, dw = pws.gemm_nt_bwd(dy, x, w)
        assert torch.equal(dx.double(), dy.double() @ w.double())
        assert torch.equal(dw.double(), dy.double().t() @ x.double())


# ---------------------------------------------------------------- cross entropy

XENT = [(1, 1, 8), (1, 1000, 64), (1, 50001, 256), (3, 17, 40), (5, 4099, 130), (64, 3000, 512), (65, 2048, 100),
        (200, 257, 1024), (513, 8200, 333), (1030, 5000, 64), (2000, 20003, 128), (16, 130, 2500)]


def xent_case(M, V, K, dtype, seed=50, ignored=0.25):
    x, w = rand((M, K), dtype, seed), rand((V, K), dtype, seed + 1, 2.5 * K ** -0.5)
    g = torch.Generator(device="cuda").manual_seed(seed + 2)
    target = torch.randint(0, V, (M,), generator=g, device="cuda")
    target[torch.rand(M, generator=g, device="cuda") < ignored] = IGNORE
    dloss = torch.rand(M, generator=g, device="cuda") / max(1, M)
    return x, w, target, dloss


def xent64(x, w, target):
    z = x.double() @ w.double().t()
    lse = torch.logsumexp(z, 1)
    keep = target != IGNORE
    loss = torch.where(keep, lse - z.gather(1, target.clamp(min=0).unsqueeze(1)).squeeze(1), torch.zeros_like(lse))
    return z, lse, keep, loss


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,V,K", XENT)
def test_xent(M, V, K, dtype):
    x, w, target, _ = xent_case(M, V, K, dtype)
    loss, lse = pws.gemm_xent_nt(x, w, target)
    z, lse64, keep, loss64 = xent64(x, w, target)
    # the largest error of a row's logits, then exponentials to 2^-20 and the
    # logarithm's and the sums' last places
    ez = acc_error(K, x.double().abs() @ w.double().abs().t()).max(1).values
    tol = ez + 2.0 ** -19 + 2.0 ** -22 * lse64.abs()
    assert loss.dtype == lse.dtype == torch.float32
    assert ((lse.double() - lse64).abs() <= tol).all()
    assert ((loss.double() - loss64).abs() <= 2 * tol + 2.0 ** -22 * loss64.abs()).all()
    assert (loss[~keep] == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,V,K", XENT)
def test_xent_bwd(M, V, K, dtype):
    x, w, target, dloss = xent_case(M, V, K, dtype)
    _, lse = pws.gemm_xent_nt(x, w, target)
    dx, dw = pws.gemm_xent_nt_bwd(x, w, target, lse, dloss)
    z, lse64, keep, _ = xent64(x, w, target)
    p = torch.exp(z - lse64[:, None])
    hit = torch.zeros_like(p)
    rows = torch.nonzero(keep).squeeze(1)
    hit[rows, target[rows]] = 1.0
    c = (dloss.double() * keep)[:, None]
    d = c * (p - hit)
    xd, wd = x.double(), w.double()
    ez = acc_error(K, xd.abs() @ wd.abs().t())
    # p's relative error: both logits' and the exponential's; then D's rounding
    # at the scale that brings max |dloss| to 2^13
    ed = c * p * (ez + ez.max(1, keepdim=True).values + 2.0 ** -18 + 2.0 ** -22 * z.abs())
    top = float(c.max()) or 1.0
    unit = half_unit((d.abs() + ed) / top * 8192, dtype) * top / 8192
    ed = ed + (unit * 2.0 ** -8 + 2.0 ** -25 * top / 8192 if M <= 64 else unit)
    check(dx, d @ wd, ed @ wd.abs() + acc_error(2 * V, d.abs() @ wd.abs()) + 2.0 ** -20 * (d.abs() @ wd.abs()), dtype)
    check(dw, d.t() @ xd, ed.t() @ xd.abs() + acc_error(2 * M, d.abs().t() @ xd.abs()) +
          2.0 ** -20 * (d.abs().t() @ xd.abs()), dtype)
    only, none = pws.gemm_xent_nt_bwd(x, w, target, lse, dloss, need_dw=False)
    assert none is None
    check(only, d @ wd, ed @ wd.abs() + acc_error(2 * V, d.abs() @ wd.abs()) + 2.0 ** -20 * (d.abs() @ wd.abs()), dtype)


@pytest.mark.parametrize("M,V,K", [(20000, 9001, 64), (9000, 40001, 72)])
def test_xent_pieces(M, V, K):
    # more tokens than one piece's 256 MB of gradients hold at this vocabulary:
    # dx is summed over two pieces, and over three whose own sums are split
    x, w, target, dloss = xent_case(M, V, K, BF16, seed=60)
    loss, lse = pws.gemm_xent_nt(x, w, target)
    dx, dw = pws.gemm_xent_nt_bwd(x, w, target, lse, dloss)
    xf, wf = x.float().requires_grad_(), w.float().requires_grad_()
    ref = torch.nn.functional.cross_entropy(xf @ wf.t(), target, ignore_index=IGNORE, reduction="none")
    (ref * dloss).sum().backward()
    for got, want in ((dx, xf.grad), (dw, wf.grad)):
        # D's and the output's rounding, 2^-9 relative each and independent
        # over thousands of terms: twice that of the norm covers their sum
        assert float((got.float() - want).norm()) <= 2 * 2.0 ** -9 * float(want.norm())


def test_xent_gradient_against_differences():
    M, V, K = 20, 90, 32
    x, w, target, dloss = xent_case(M, V, K, F16, seed=70)
    dloss = dloss * M
    _, lse = pws.gemm_xent_nt(x, w, target)
    grads = pws.gemm_xent_nt_bwd(x, w, target, lse, dloss)
    at = [x.double(), w.double()]
    for i in range(2):
        d = torch.sign(rand(at[i].shape, torch.float32, 80 + i)).double()
        e = 1e-5
        hi, lo = [list(at), list(at)]
        hi[i], lo[i] = at[i] + e * d, at[i] - e * d
        diff = ((xent64(*hi, target)[3] - xent64(*lo, target)[3]) * dloss.double()).sum() / (2 * e)
        bound = (grads[i].double().abs() * 2.0 ** -9 + 2.0 ** -11 * grads[i].double().abs().mean()).sum()
        assert abs(float(diff - (grads[i].double() * d).sum())) <= float(bound)


@pytest.mark.parametrize("dtype", TYPES)
def test_xent_rows_that_do_not_count(dtype):
    M, V, K = 130, 1000, 72
    x, w, target, dloss = xent_case(M, V, K, dtype, ignored=0.5)
    target[:] = IGNORE
    loss, lse = pws.gemm_xent_nt(x, w, target)
    dx, dw = pws.gemm_xent_nt_bwd(x, w, target, lse, dloss)
    assert (loss == 0).all() and (dx == 0).all() and (dw == 0).all()
    # an ignored row's own gradient stays zero where its logits are not finite
    target[3] = 17
    x[5, :] = float("inf")
    loss, lse = pws.gemm_xent_nt(x, w, target)
    dx, _ = pws.gemm_xent_nt_bwd(x, w, target, lse, dloss, need_dw=False)
    assert loss[5] == 0 and (dx[5] == 0).all() and (dx[3] != 0).any()
    # another ignore_index, inside the vocabulary
    loss, lse = pws.gemm_xent_nt(x, w, target, ignore_index=17)
    assert loss[3] == 0


def test_xent_targets_outside_the_vocabulary_are_nan():
    M, V, K = 70, 300, 64
    for bad in (V, -1, 1 << 40, -(1 << 40)):
        x, w, target, dloss = xent_case(M, V, K, BF16, ignored=0.0)
        want, _ = pws.gemm_xent_nt(x, w, target)
        target[9] = bad
        loss, lse = pws.gemm_xent_nt(x, w, target)
        assert torch.isnan(loss[9]) and torch.isfinite(lse).all()
        assert torch.equal(loss[10:], want[10:])
        dx, dw = pws.gemm_xent_nt_bwd(x, w, target, lse, dloss)
        assert torch.isnan(dx[9]).all() and torch.isfinite(dx[:9]).all() and torch.isnan(dw).all()


def test_xent_extreme_logits():
    # logits of +-30000 and a row whose maximum is far above the rest
    V, K = 700, 64
    x = torch.zeros(4, K, device="cuda", dtype=BF16)
    x[0, 0], x[1, 0], x[2, 1] = 100.0, -100.0, 100.0
    w = torch.zeros(V, K, device="cuda", dtype=BF16)
    w[:, 0] = 300.0
    w[123, 1] = 300.0
    target = torch.tensor([5, 5, 123, 7], device="cuda")
    loss, lse = pws.gemm_xent_nt(x, w, target)
    want = torch.tensor([30000 + math.log(V), -30000 + math.log(V), 30000.0, math.log(V)], dtype=torch.float64)
    assert ((lse.cpu().double() - want).abs() <= 2.0 ** -22 * want.abs() + 2.0 ** -19).all()
    # a logit of 30000 held in fp32 has a unit of 2^-9
    want = torch.tensor([math.log(V), math.log(V), 0.0, math.log(V)], dtype=torch.float64)
    assert ((loss.cpu().double() - want).abs() <= 2.0 ** -8).all()
    dx, dw = pws.gemm_xent_nt_bwd(x, w, target, lse, torch.ones(4, device="cuda"))
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()


def test_xent_dloss_of_any_size():
    # the scale of D follows dloss: binary16 gradients of tiny and large loss
    # gradients are the plain ones' multiples
    M, V, K = 100, 3000, 64
    x, w, target, _ = xent_case(M, V, K, F16, ignored=0.1)
    _, lse = pws.gemm_xent_nt(x, w, target)
    base, _ = pws.gemm_xent_nt_bwd(x, w, target, lse, torch.ones(M, device="cuda"), need_dw=False)
    for s in (2.0 ** -6, 2.0 ** 6, -1.0):
        dx, _ = pws.gemm_xent_nt_bwd(x, w, target, lse, torch.full((M,), s, device="cuda"), need_dw=False)
        want = base.double() * s
        # (below binary16's normal range either one is rounded to 2^-25)
        assert ((dx.double() - want).abs() <= 2.0 ** -24 * max(1.0, abs(s)) + 2.0 ** -11 * want.abs()).all()
    zero, dw = pws.gemm_xent_nt_bwd(x, w, target, lse, torch.zeros(M, device="cuda"))
    assert (zero == 0).all() and (dw == 0).all()


# ---------------------------------------------------------------- all of them

def test_empty_sizes():
    e = lambda *s: torch.empty(s, device="cuda", dtype=F16)     # noqa: E731
    f = lambda n: torch.empty(n, device="cuda")                 # noqa: E731
    assert pws.gemm_gated_nt(e(0, 8), e(4, 8), e(4, 8)).shape == (0, 4)
    assert pws.gemm_gated_nt(e(3, 8), e(0, 8), e(0, 8)).shape == (3, 0)
    h, g, u = pws.gemm_gated_nt(e(3, 0), e(5, 0), e(5, 0), save=True)
    assert (h == 0).all() and (g == 0).all() and (u == 0).all()
    dx, dg, du = pws.gemm_gated_nt_bwd(e(0, 4), e(0, 4), e(0, 4), e(0, 8), e(4, 8), e(4, 8))
    assert dx.shape == (0, 8) and (dg == 0).all() and (du == 0).all()
    dx, dg, du = pws.gemm_gated_nt_bwd(e(3, 0), e(3, 0), e(3, 0), e(3, 8), e(0, 8), e(0, 8))
    assert (dx == 0).all() and dg.shape == (0, 8)
    dx, dw = pws.gemm_nt_bwd(e(0, 4), e(0, 8), e(4, 8))
    assert dx.shape == (0, 8) and (dw == 0).all()
    dx, dw = pws.gemm_nt_bwd(e(3, 0), e(3, 8), e(0, 8))
    assert (dx == 0).all() and dw.shape == (0, 8)
    none = torch.empty(0, device="cuda", dtype=torch.int64)
    loss, lse = pws.gemm_xent_nt(e(0, 8), e(9, 8), none)
    assert loss.shape == lse.shape == (0,)
    dx, dw = pws.gemm_xent_nt_bwd(e(0, 8), e(9, 8), none, f(0), f(0))
    assert dx.shape == (0, 8) and (dw == 0).all()
    loss, lse = pws.gemm_xent_nt(e(2, 0), e(9, 0), torch.tensor([1, IGNORE], device="cuda"))
    assert torch.allclose(lse, torch.full((2,), math.log(9), device="cuda")) and loss[1] == 0


def run_all(M, F, V, K, dtype, stream=None):
    """One training step's calls; every output."""
    x, wg, wu = rand((M, K), dtype, 91), rand((F, K), dtype, 92, 0.1), rand((F, K), dtype, 93, 0.1)
    head, dh = rand((V, K), dtype, 94, 0.1), rand((M, F), dtype, 95, 0.1)
    target = torch.arange(M, device="cuda") % V
    dloss = torch.full((M,), 1.0 / M, device="cuda")
    torch.cuda.synchronize()

    def step():
        h, g, u = pws.gemm_gated_nt(x, wg, wu, save=True, stream=stream)
        out = [h, g, u, *pws.gemm_gated_nt_bwd(dh, g, u, x, wg, wu, stream=stream)]
        loss, lse = pws.gemm_xent_nt(x, head, target, stream=stream)
        out += [loss, lse, *pws.gemm_xent_nt_bwd(x, head, target, lse, dloss, stream=stream)]
        return out + list(pws.gemm_nt_bwd(dh, x, wg, stream=stream))
    return step


def same(a, b):
    return all(torch.equal(p.view(torch.int16) if p.dtype != torch.float32 else p.view(torch.int32),
                           q.view(torch.int16) if q.dtype != torch.float32 else q.view(torch.int32))
               for p, q in zip(a, b))


@pytest.mark.parametrize("M,F,V,K", [(1, 256, 1000, 64), (50, 333, 777, 130), (600, 1024, 3000, 512)])
def test_same_bits_again_on_other_streams_and_from_a_graph(M, F, V, K):
    step = run_all(M, F, V, K, BF16)
    want = step()
    torch.cuda.synchronize()
    for _ in range(3):
        assert same(step(), want)
    # a stream of its own, passed as an argument: outputs and workspaces are
    # that stream's, while the current stream goes on allocating
    other = torch.cuda.Stream()
    on_other = run_all(M, F, V, K, BF16, stream=other)
    outs = [on_other() for _ in range(3)]
    junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert all(same(o, want) for o in outs)
    del junk
    # by its raw handle
    raw = run_all(M, F, V, K, BF16, stream=other.cuda_stream)()
    other.synchronize()
    assert same(raw, want)
    # a captured step, replayed
    with torch.cuda.stream(other):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=other):
            captured = step()
        for t in captured:
            t.fill_(1)
        graph.replay()
    other.synchronize()
    assert same(captured, want)


def test_a_timed_out_wait_is_reported():
    # ring slots that never become empty: every role's first wait runs out, the
    # call returns, the status word says so, and the next call is whole again
    x, wg, wu = rand((512, 4096), F16, 1), rand((4096, 4096), F16, 2, 0.02), rand((4096, 4096), F16, 3, 0.02)
    want = pws.gemm_gated_nt(x, wg, wu)
    torch.cuda.synchronize()
    pws.gemm_set_debug_flags(pws.GEMM_DEBUG_SKIP_EMPTY_SEED)
    pws.gemm_set_wait_timeout_ns(20_000_000)
    try:
        for rows in (512, 1):       # a CTA pair's tile, and a single CTA's
            pws.gemm_gated_nt(x[:rows], wg, wu)
            assert pws.gemm_device_status() == pws.GEMM_ERR_TIMEOUT
    finally:
        pws.gemm_set_debug_flags(0)
        pws.gemm_set_wait_timeout_ns(0)
    got = pws.gemm_gated_nt(x, wg, wu)
    assert pws.gemm_device_status() == pws.GEMM_OK
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_example_trains_and_scores():
    # the operators together, as a training step and as a token's score
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "language_model_block.py")
    spec = importlib.util.spec_from_file_location("language_model_block", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    x, target, masters = ex.make(300, 136, 328, 1003, seed=3)
    w = {k: v.half() for k, v in masters.items()}
    loss, grads = ex.forward_backward(x, target, w)
    want, want_grads = ex.autograd(x, target, w)
    # binary16 activations on the way: h, y, g and u are rounded to 2^-11, and a
    # logit is a sum of 136 such products of size one
    assert abs(float(loss) - float(want)) <= 2.0 ** -8
    for k, g in want_grads.items():
        # half a dozen roundings of 2^-11 each between the loss and a gradient
        assert float((grads[k].float() - g).norm()) <= 6 * 2.0 ** -11 * float(g.norm()), k
    losses = ex.train(x, target, masters, 6)
    assert all(b < a for a, b in zip(losses, losses[1:]))
    w = {k: v.half() for k, v in masters.items()}
    one = ex.score(x[7:8], target[7:8].clamp(min=0), w)
    many = ex.score(x, target.clamp(min=0), w)
    assert abs(float(one) - float(many[7])) <= 2.0 ** -8


def test_too_small_a_workspace_is_refused():
    lib = pws.load_library()
    held = [torch.zeros(1 << 16, device="cuda", dtype=F16) for _ in range(9)]
    p = [t.data_ptr() for t in held]
    bad, half = pws.GEMM_ERR_INVALID_ARG, pws.GEMM_TYPE_HALF
    # missing, misaligned, too small, on an input (p[0]), on an output (p[3], p[6])
    for ws, size in ((None, 1 << 30), (p[8] + 2, 1 << 30), (p[8], 16), (p[0], 1 << 30)):
        assert lib.gemm_gated_nt_bwd(4, 8, 16, *p[:6], p[6], None, None, half, 0, ws, size, None) == bad
        assert lib.gemm_xent_nt(4, 8, 16, p[0], p[1], p[2], -100, p[3], p[4], half, ws, size, None) == bad
        assert lib.gemm_xent_nt_bwd(4, 8, 16, p[0], p[1], p[2], -100, p[3], p[4], p[5], None, half, ws, size, None) == bad
        # 9 columns: rows that need a copy
        assert lib.gemm_gated_nt(4, 8, 9, *p[:3], p[3], None, None, half, 0, ws, size, None) == bad
        assert lib.gemm_nt_bwd(4, 9, 16, *p[:3], p[3], None, half, ws, size, None) == bad
    assert lib.gemm_gated_nt_bwd(4, 8, 16, *p[:6], p[6], None, None, half, 0, p[6], 1 << 30, None) == bad
    assert lib.gemm_nt_bwd(4, 9, 16, *p[:3], p[3], None, half, p[3], 1 << 30, None) == bad

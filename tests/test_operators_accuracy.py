"""Where the operators around the products could lose accuracy without the
bounds of their other tests showing it: gradients far below and above
binary16's range, confident targets over a long K, large logits, rows whose
loss gradient is zero; the wide tile's forms; gradients against differences
along themselves; sizes at the limit; tensors that require gradients.

Tolerances are derived beside each test, from the rounding of each type (half a
unit: 2^-11 relative in binary16, 2^-8 in bfloat16, 2^-24 in fp32).
"""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

import pipelined_warp_specialized_gb300 as pws  # noqa: E402
from test_operators_gpu import BF16, F16, IGNORE, TYPES, acc_error, act64, check, half_unit, rand, xent64  # noqa: E402


@pytest.fixture(autouse=True)
def _no_timeouts():
    yield
    if torch.cuda.is_available():
        assert pws.gemm_device_status() == pws.GEMM_OK


# ---------------------------------------------------------------- gated gradients of any size

def gated_grads64(dh, g, u, x, wg, wu, act):
    value, slope = act64(g.double(), act)
    dg, du = dh.double() * u.double() * slope, dh.double() * value
    return dg, du, (dg @ wg.double() + du @ wu.double(), dg.t() @ x.double(), du.t() @ x.double())


@pytest.mark.gpu
@pytest.mark.parametrize("std", [0.02, 1e-4, 1e-5, 1e-6])
@pytest.mark.parametrize("M", [1, 64, 65, 2048])
def test_gated_bwd_of_small_gradients(M, std):
    # Against the error of rounding the exact gradient once, in norm.  Above 64
    # rows the sums' terms are rounded to as many bits as their result: terms
    # of random sign, so both errors are the same part of the result's norm
    # and add as squares: sqrt(2).  Up to 64 rows the terms keep twice the bits.
    F, K = 1024, 512
    x, wg, wu = rand((M, K), F16, 1), rand((F, K), F16, 2, K ** -0.5), rand((F, K), F16, 3, K ** -0.5)
    g, u, dh = rand((M, F), F16, 4), rand((M, F), F16, 5), rand((M, F), torch.float32, 6, std).half()
    got = pws.gemm_gated_nt_bwd(dh, g, u, x, wg, wu)
    for have, want in zip(got, gated_grads64(dh, g, u, x, wg, wu, "silu")[2]):
        once = (want.half().double() - want).norm()
        assert float((have.double() - want).norm()) <= (1.5 if M > 64 else 1.1) * float(once)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [9, 100])
def test_gated_bwd_of_gradients_past_the_range(M):
    # one row's dg is past binary16's range, its products with the weights and
    # the tokens are within it; the other rows keep what 2^-39 of the largest
    # |dh| max(1.13 |u|, g, 0.28) leaves them (half of binary16's smallest step,
    # where that lies in [2^14, 2^15))
    F, K = 320, 136
    x, wg, wu = rand((M, K), F16, 11), rand((F, K), F16, 12, 0.004), rand((F, K), F16, 13, 0.004)
    g, u, dh = rand((M, F), F16, 14), rand((M, F), F16, 15), rand((M, F), F16, 16, 0.02)
    dh[3] = rand((F,), F16, 17, 1e4).clamp(-3e4, 3e4)
    u[3] = 20.0
    x[3] = 0.002
    for act in ("silu", "gelu"):
        got = pws.gemm_gated_nt_bwd(dh, g, u, x, wg, wu, act=act)
        dg, du, want = gated_grads64(dh, g, u, x, wg, wu, act)
        top = float((dh.double().abs() * torch.maximum(1.13 * u.double().abs(), g.double().clamp(min=0.28))).max())
        assert float(dg.abs().max()) > 65504 and all(float(t.abs().max()) < 60000 for t in want)
        # fp32's own error of dg and du, as for the other sizes
        small = 2.0 ** -19 * dh.double().abs() * (u.double().abs() + 1) * (1 + g.double().abs())
        bits = 2.0 ** -11 if M > 64 else 2.0 ** -22
        eg, eu = (small + t.abs() * bits + 2.0 ** -39 * top for t in (dg, du))
        wgd, wud, xd = wg.double().abs(), wu.double().abs(), x.double().abs()
        check(got[0], want[0], eg @ wgd + eu @ wud + acc_error(4 * F, dg.abs() @ wgd + du.abs() @ wud), F16)
        check(got[1], want[1], eg.t() @ xd + acc_error(2 * M, dg.abs().t() @ xd), F16)
        check(got[2], want[2], eu.t() @ xd + acc_error(2 * M, du.abs().t() @ xd), F16)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [3, 80])
def test_gated_bwd_of_zeros_and_of_what_is_not_finite(M, dtype):
    # zero gradients give zeros; an infinite or NaN dh stays in its row of dx and
    # leaves the other rows' bits alone
    F, K = 96, 72
    x, wg, wu = rand((M, K), dtype, 21), rand((F, K), dtype, 22, 0.1), rand((F, K), dtype, 23, 0.1)
    g, u, dh = rand((M, F), dtype, 24), rand((M, F), dtype, 25), rand((M, F), dtype, 26, 0.02)
    for t in pws.gemm_gated_nt_bwd(torch.zeros_like(dh), g, u, x, wg, wu):
        assert (t == 0).all()
    dh[0, 0], u[0, 0], g[0, 0] = 1.0, 3.0, 3.0          # (the largest dg and du, which set their scale)
    want = pws.gemm_gated_nt_bwd(dh, g, u, x, wg, wu)[0]
    others = torch.arange(M, device="cuda") != 2
    for bad in (float("inf"), float("nan")):
        broken = dh.clone()
        broken[2, 5] = bad
        dx, dwg, dwu = pws.gemm_gated_nt_bwd(broken, g, u, x, wg, wu)
        assert not torch.isfinite(dx[2]).any() and not torch.isfinite(dwg[5]).any()
        assert torch.isfinite(dwg[4]).all() and torch.isfinite(dwu[4]).all()
        assert torch.equal(dx[others].view(torch.int16), want[others].view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M", [8, 80])
def test_gated_bwd_of_an_infinite_up_projection(M, act):
    # where u is infinite dg is and du is not: du = 240000 is the largest finite
    # element, past binary16's range, and its products with the tokens are within
    F, K = 96, 72
    x, wg, wu = rand((M, K), F16, 27), rand((F, K), F16, 28, 0.1), rand((F, K), F16, 29, 0.1)
    g, u, dh = rand((M, F), F16, 30), rand((M, F), F16, 31), rand((M, F), F16, 32, 0.02)
    dh[4, 5], g[4, 5], u[4, 5] = 30000.0, 8.0, float("inf")
    x[4] = 0.01
    _, dwg, dwu = pws.gemm_gated_nt_bwd(dh, g, u, x, wg, wu, act=act)
    du = dh.double() * act64(g.double(), act)[0]
    xd, top = x.double(), 30000.0 * 8
    bits = 2.0 ** -11 if M > 64 else 2.0 ** -22
    eu = 2.0 ** -19 * dh.double().abs() * (1 + g.double().abs()) + du.abs() * bits + 2.0 ** -39 * top
    check(dwu, du.t() @ xd, eu.t() @ xd.abs() + acc_error(2 * M, du.abs().t() @ xd.abs()), F16)
    assert not torch.isfinite(dwg[5]).any() and torch.isfinite(dwg[6]).all()


# ---------------------------------------------------------------- cross entropy

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [1, 64, 65, 300])
def test_xent_bwd_of_confident_targets_over_a_long_k(M, dtype):
    # Two classes with logits 7 and 0: D's entries are -(1 - p) and 1 - p with
    # 1 - p = 9e-4, so their sum (read off a column that is 1 in every class and 0
    # in every token) shows any difference between the logits here and those in
    # lse.  What is left is lse's rounding (2^-22 for [4, 8)), that of the sum
    # of exponentials and of the exponential itself (2^-21 each), and D's own
    # rounding above 64 rows; an accumulator that loses half a unit at each of
    # the K / 16 additions is off by 512 of them.
    K = 8192
    gen = torch.Generator(device="cuda").manual_seed(M)
    x = (torch.rand((M, K), generator=gen, device="cuda") + 0.5).to(dtype)
    w = torch.zeros((2, K), device="cuda", dtype=dtype)
    w[1] = ((torch.rand(K, generator=gen, device="cuda") + 0.5) * (7.0 / K)).to(dtype)
    x[:, 5], w[:, 5] = 0.0, 1.0
    target = torch.ones(M, dtype=torch.int64, device="cuda")
    _, lse = pws.gemm_xent_nt(x, w, target)
    dx, _ = pws.gemm_xent_nt_bwd(x, w, target, lse, torch.ones(M, device="cuda"))
    z = x.double() @ w.double().t()
    assert (z[:, 0] == 0).all() and (z[:, 1] > 6).all() and (lse < 8).all()
    rest = torch.sigmoid(z[:, 0] - z[:, 1])
    bits = {F16: 2.0 ** -11, BF16: 2.0 ** -8}[dtype]
    tol = 2.0 ** -22 + 3 * 2.0 ** -21 + (2 * bits * rest if M > 64 else 0.0)
    assert (dx[:, 5].double().abs() <= tol * (1 + bits) + 2.0 ** -25).all(), float(dx[:, 5].abs().max())


@pytest.mark.gpu
@pytest.mark.parametrize("V", [200, 700, 20003])
def test_lse_of_large_logits(V):
    # z = t_i + s_i c_v, multiples of 2^-14 below 2^7 that every sum holds exactly:
    # what is off in lse is its own rounding (half a unit of [64, 128): 2^-18) and
    # the relative error of the sum of exponentials: 2^-22 each from the
    # exponential, its argument (z - max, exact, times log2 e, below 2^4) and the
    # maximum's rescaling, 2^-24 for each of some 20 levels of sums, and the
    # logarithm's last place: 2^-19 in all
    M, K = 300, 16
    gen = torch.Generator(device="cuda").manual_seed(V)
    x, w = torch.zeros((M, K), device="cuda", dtype=F16), torch.zeros((V, K), device="cuda", dtype=F16)
    x[:, 0] = torch.randint(70 * 16, 110 * 16, (M,), generator=gen, device="cuda") / 16
    w[:, 0] = 1.0
    x[:, 1] = torch.randint(32, 65, (M,), generator=gen, device="cuda") / 64
    w[:, 1] = torch.randint(-4 * 256, 4 * 256, (V,), generator=gen, device="cuda") / 256
    target = torch.randint(0, V, (M,), generator=gen, device="cuda")
    z, want, _, loss64 = xent64(x, w, target)
    assert float(want.max()) < 128
    for rows in (M, 7):
        loss, lse = pws.gemm_xent_nt(x[:rows].contiguous(), w, target[:rows])
        assert ((lse.double() - want[:rows]).abs() <= 2.0 ** -18 + 2.0 ** -19).all()
        # (the loss is exact in lse and a logit that fp32 holds)
        assert ((loss.double() - loss64[:rows]).abs() <= 2.0 ** -18 + 2.0 ** -19).all()


@pytest.mark.gpu
def test_xent_bwd_of_large_logits():
    # D of the target is exp(z - lse) - 1, here with lse = z + 2^-8 handed in:
    # z and lse are exact, so are their difference and D up to the exponential's
    # 2^-22 and the argument's rounding; read off columns of w that are one class each
    M, V = 64, 40
    K = 8 + V
    x, w = torch.zeros((M, K), device="cuda", dtype=F16), torch.zeros((V, K), device="cuda", dtype=F16)
    x[:, 0] = 70.0 + torch.arange(M, device="cuda") / 2
    w[:, 0] = 1.0
    w[torch.arange(V), 8 + torch.arange(V)] = 1.0
    target = torch.arange(M, device="cuda") % V
    lse = x[:, 0].float() + 2.0 ** -8
    dx, _ = pws.gemm_xent_nt_bwd(x, w, target, lse, torch.ones(M, device="cuda"))
    p = math.exp(-2.0 ** -8)
    want = torch.full((M, V), p, device="cuda", dtype=torch.float64)
    want[torch.arange(M), target] = math.expm1(-2.0 ** -8)
    err = (dx[:, 8:].double() - want).abs()
    assert (err <= half_unit(want, F16) + 2.0 ** -21).all(), float((err / half_unit(want, F16)).max())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [6, 130])
def test_xent_bwd_of_rows_with_no_loss_gradient(M, dtype):
    # dloss = 0 gives zero times D: 0 for finite logits, NaN where the row
    # counts and a logit is NaN or infinite, 0 where the row does not count
    V, K = 300, 72
    x, w = rand((M, K), dtype, 31), rand((V, K), dtype, 32, 0.2)
    target = torch.randint(0, V, (M,), generator=torch.Generator(device="cuda").manual_seed(33), device="cuda")
    dloss = torch.ones(M, device="cuda")
    dloss[1] = dloss[2] = dloss[3] = 0.0
    dloss[3] *= -1.0
    x[2, 7] = x[4, 7] = float("nan")
    target[4] = IGNORE
    _, lse = pws.gemm_xent_nt(x, w, target)
    assert torch.isnan(lse[2]) and torch.isnan(lse[4])
    dx, _ = pws.gemm_xent_nt_bwd(x, w, target, lse, dloss, need_dw=False)
    assert torch.isnan(dx[2]).all()
    assert (dx[1] == 0).all() and (dx[3] == 0).all() and (dx[4] == 0).all()
    assert torch.isfinite(dx[5:]).all() and (dx[5:] != 0).any(1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [40, 200])
def test_xent_bwd_of_loss_gradients_of_many_sizes(M, dtype):
    # dloss over 24 powers of two.  Binary16 holds an element of D to half a
    # unit of its own, or to half its smallest step at the scale that brings
    # the largest |dloss| to 2^13: 2^-38 of that; bfloat16 to half a unit.
    V, K = 1000, 72
    x, w = rand((M, K), dtype, 41), rand((V, K), dtype, 42, 0.5 * K ** -0.5)
    target = torch.randint(0, V, (M,), generator=torch.Generator(device="cuda").manual_seed(43), device="cuda")
    dloss = 1024.0 * 2.0 ** -(torch.arange(M, device="cuda") % 25).float()
    _, lse = pws.gemm_xent_nt(x, w, target)
    dx, dw = pws.gemm_xent_nt_bwd(x, w, target, lse, dloss)
    z, lse64, _, _ = xent64(x, w, target)
    p = torch.exp(z - lse64[:, None])
    hit = torch.zeros_like(p)
    hit[torch.arange(M), target] = 1.0
    c = dloss.double()[:, None]
    d = c * (p - hit)
    xd, wd = x.double(), w.double()
    ez = acc_error(K, xd.abs() @ wd.abs().t())
    ed = c * p * (ez + ez.max(1, keepdim=True).values + 2.0 ** -18)
    bits = {F16: 2.0 ** -11, BF16: 2.0 ** -8}[dtype]
    ed = ed + d.abs() * (bits if M > 64 else bits * bits) + (2.0 ** -38 * 1024 if dtype == F16 else 0.0)
    check(dx, d @ wd, ed @ wd.abs() + acc_error(2 * V, d.abs() @ wd.abs()) + 2.0 ** -20 * (d.abs() @ wd.abs()), dtype)
    check(dw, d.t() @ xd, ed.t() @ xd.abs() + acc_error(2 * M, d.abs().t() @ xd.abs()) +
          2.0 ** -20 * (d.abs().t() @ xd.abs()), dtype)


# ---------------------------------------------------------------- gradients against differences

def along(value, at, grads):
    """For each argument i: the central difference of value in float64 along
    grads[i] / |grads[i]|, and |grads[i]|.  For exact gradients they are equal;
    errors of root sum square e move their difference by no more than e."""
    out = []
    for i, grad in enumerate(grads):
        grad = grad.double()
        size = float(grad.norm())
        e = 1e-5
        hi, lo = list(at), list(at)
        hi[i], lo[i] = at[i] + e * grad / size, at[i] - e * grad / size
        out.append((float(value(*hi) - value(*lo)) / (2 * e), size))
    return out


def gated_value(dh, act):
    def value(x, wg, wu):
        return (dh.double() * act64(x @ wg.t(), act)[0] * (x @ wu.t())).sum()
    return value


# Each gradient is rounded once (2^-11 of itself) and comes from g and u rounded
# to binary16: relative errors of 2^-11 in u and, times |g act''| <= 1.2 |act'| in
# norm over N(0, 1) gates, in act'; independent, over sums of dozens of
# terms, so they stay at a few 2^-11 of the norm.
GATED_ALONG = 8 * 2.0 ** -11


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M", [24, 100])
def test_gated_gradient_along_itself(M, act):
    F, K = 80, 48
    x, wg, wu, dh = rand((M, K), F16, 51), rand((F, K), F16, 52, 0.15), rand((F, K), F16, 53, 0.15), rand((M, F), F16, 54)
    _, g, u = pws.gemm_gated_nt(x, wg, wu, act=act, save=True)
    grads = pws.gemm_gated_nt_bwd(dh, g, u, x, wg, wu, act=act)
    at = [x.double(), wg.double(), wu.double()]
    for diff, size in along(gated_value(dh, act), at, grads):
        assert abs(diff - size) <= GATED_ALONG * size


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_a_wrong_slope_shows_along_the_gradient(act):
    # the comparison itself, on the host: exact gradients pass by far; slopes
    # without their second term or of the other activation do not (dWg), nor does
    # the other activation's value (dWu)
    M, F, K = 24, 80, 48
    gen = torch.Generator().manual_seed(55)

    def normal(rows, cols, std=1.0):
        return torch.randn(rows, cols, generator=gen, dtype=torch.float64) * std

    x, wg, wu, dh = normal(M, K), normal(F, K, 0.15), normal(F, K, 0.15), normal(M, F)
    g, u = x @ wg.t(), x @ wu.t()
    value, slope = act64(g, act)
    sigma = torch.where(g == 0, torch.full_like(g, 0.5), value / g)     # act(g) = g sigma(s(g))
    other_value, other_slope = act64(g, "gelu" if act == "silu" else "silu")
    for v, s, wrong in ((value, slope, None), (value, sigma, 1), (value, other_slope, 1), (other_value, slope, 2)):
        dg, du = dh * u * s, dh * v
        off = [abs(d - n) / n for d, n in along(gated_value(dh, act), [x, wg, wu],
                                                (dg @ wg + du @ wu, dg.t() @ x, du.t() @ x))]
        assert max(off) <= 1e-6 if wrong is None else off[wrong] > 1.5 * GATED_ALONG, off


@pytest.mark.gpu
@pytest.mark.parametrize("M", [20, 90])
def test_xent_gradient_along_itself(M):
    # the gradients' own rounding (2^-11) and, above 64 rows, D's (2^-11): twice
    # 2^-11 of the norm if all of it lay along the gradient
    V, K = 90, 32
    x, w = rand((M, K), F16, 61), rand((V, K), F16, 62, 0.4)
    gen = torch.Generator(device="cuda").manual_seed(63)
    target = torch.randint(0, V, (M,), generator=gen, device="cuda")
    target[::5] = IGNORE
    dloss = torch.rand(M, generator=gen, device="cuda")
    _, lse = pws.gemm_xent_nt(x, w, target)
    grads = pws.gemm_xent_nt_bwd(x, w, target, lse, dloss)
    for diff, size in along(lambda a, b: (xent64(a, b, target)[3] * dloss.double()).sum(), [x.double(), w.double()], grads):
        assert abs(diff - size) <= 2 * 2.0 ** -11 * size


# ---------------------------------------------------------------- the wide tile's forms

@pytest.mark.gpu
def test_gated_bwd_on_the_wide_tile():
    # 129 K blocks and more in both products: dx accumulates over two segments,
    # both weights' gradients are one job, and the last tile is ragged
    M, F, K = 8200, 4168, 264
    x, wg, wu = rand((M, K), BF16, 71), rand((F, K), BF16, 72, 0.05), rand((F, K), BF16, 73, 0.05)
    g, u, dh = rand((M, F), BF16, 74), rand((M, F), BF16, 75), rand((M, F), BF16, 76, 0.02)
    dg, du, want = gated_grads64(dh, g, u, x, wg, wu, "gelu")
    small = 2.0 ** -19 * dh.double().abs() * (u.double().abs() + 1) * (1 + g.double().abs())
    eg, eu = small + half_unit(dg.abs() + small, BF16), small + half_unit(du.abs() + small, BF16)
    wgd, wud, xd = wg.double().abs(), wu.double().abs(), x.double().abs()
    tols = (eg @ wgd + eu @ wud + acc_error(2 * F, dg.abs() @ wgd + du.abs() @ wud),
            eg.t() @ xd + acc_error(M, dg.abs().t() @ xd), eu.t() @ xd + acc_error(M, du.abs().t() @ xd))
    for needs in (dict(), dict(need_dw=False), dict(need_dx=False)):
        for got, ref, tol in zip(pws.gemm_gated_nt_bwd(dh, g, u, x, wg, wu, act="gelu", **needs), want, tols):
            if got is not None:
                check(got, ref, tol, BF16)


@pytest.mark.gpu
def test_xent_bwd_on_the_wide_tile_over_pieces():
    # 8200 tokens over two pieces of the vocabulary of 129 K blocks and more: dx
    # is a running fp32 sum between them
    M, V, K = 8200, 20003, 264
    x, w = rand((M, K), BF16, 81), rand((V, K), BF16, 82, 2.0 * K ** -0.5)
    gen = torch.Generator(device="cuda").manual_seed(83)
    target = torch.randint(0, V, (M,), generator=gen, device="cuda")
    target[::7] = IGNORE
    dloss = torch.rand(M, generator=gen, device="cuda") / M
    _, lse = pws.gemm_xent_nt(x, w, target)
    dx, dw = pws.gemm_xent_nt_bwd(x, w, target, lse, dloss)
    z, lse64, keep, _ = xent64(x, w, target)
    d = torch.exp(z - lse64[:, None])
    del z
    rows = torch.nonzero(keep).squeeze(1)
    d[rows, target[rows]] -= 1.0
    d *= (dloss.double() * keep)[:, None]
    xd, wd = x.double(), w.double()
    # a logit's error is far below D's rounding to bfloat16, 2^-8 of each entry
    ed = d.abs() * (2.0 ** -8 + 2.0 ** -13) + 2.0 ** -20 * dloss.double()[:, None] / V
    check(dx, d @ wd, ed @ wd.abs() + acc_error(2 * V, d.abs() @ wd.abs()), BF16)
    check(dw, d.t() @ xd, ed.t() @ xd.abs() + acc_error(2 * M, d.abs().t() @ xd.abs()), BF16)


# ---------------------------------------------------------------- the largest sizes

# fake, 256-byte aligned addresses far apart: never read, the calls below are
# refused or only count a workspace
AT = [(i + 1) << 48 for i in range(12)]
LARGEST = 2 ** 31 - 1024


def test_sizes_whose_tiles_would_pass_32_bits_are_refused():
    # Columns are counted in 32 bits, and the last tile's end, up to 512 past the
    # last column, has to fit: above 2^31 - 1024 it wrapped, and the tile's
    # columns were not written (or, between widths, others were)
    from pipelined_warp_specialized_gb300 import build as libbuild
    libbuild.build()
    lib = pws.load_library()
    H, bad = pws.GEMM_TYPE_HALF, pws.GEMM_ERR_INVALID_ARG
    calls = {
        "gemm_gated_nt": lambda d: (*d, *AT[:4], None, None, H, 0, None, 0, None),
        "gemm_gated_nt_bwd": lambda d: (*d, *AT[:6], *AT[6:9], H, 0, AT[9], 1 << 47, None),
        "gemm_xent_nt": lambda d: (*d, *AT[:3], -100, *AT[3:5], H, AT[5], 1 << 47, None),
        "gemm_xent_nt_bwd": lambda d: (*d, *AT[:3], -100, *AT[3:7], H, AT[7], 1 << 47, None),
        "gemm_nt_bwd": lambda d: (*d, *AT[:5], H, AT[5], 1 << 47, None),
    }
    for name, args in calls.items():
        for i in range(3):
            for size in (LARGEST + 1, 2 ** 31 - 1):
                dims = [4, 8, 16]
                dims[i] = size
                assert getattr(lib, name)(*args(dims)) == bad, (name, dims)
    # the largest sizes themselves are taken
    pointers = {"gemm_gated_nt": 3, "gemm_gated_nt_bwd": 6, "gemm_xent_nt": 2, "gemm_xent_nt_bwd": 2, "gemm_nt_bwd": 3}
    for name, count in pointers.items():
        for i in range(3):
            dims = [4, 8, 16]
            dims[i] = LARGEST
            n = ctypes.c_int64()
            assert getattr(lib, name + "_workspace")(*dims, *AT[:count], H, ctypes.byref(n)) == pws.GEMM_OK, (name, dims)


# ---------------------------------------------------------------- tensors that require gradients

@pytest.fixture
def _warnings_again():
    before = set(pws._warned)
    pws._warned.clear()
    yield
    pws._warned.update(before)


def test_unrecorded_calls_say_so_once(_warnings_again, recwarn):
    plain, leaf = torch.zeros(2, 2), torch.zeros(2, 2, requires_grad=True)
    pws._not_recorded("gemm_gated_nt", "gemm_gated_nt_bwd", plain, plain)
    with torch.no_grad():
        pws._not_recorded("gemm_gated_nt", "gemm_gated_nt_bwd", plain, leaf)
    assert not recwarn.list
    with pytest.warns(UserWarning, match="gemm_gated_nt is not recorded by autograd.*gemm_gated_nt_bwd"):
        pws._not_recorded("gemm_gated_nt", "gemm_gated_nt_bwd", plain, leaf)
    pws._not_recorded("gemm_gated_nt", "gemm_gated_nt_bwd", plain, leaf)
    assert not recwarn.list


@pytest.mark.gpu
def test_forward_calls_warn_of_gradients_they_do_not_carry(_warnings_again):
    x, w = rand((4, 16), F16, 91), rand((8, 16), F16, 92)
    target = torch.zeros(4, dtype=torch.int64, device="cuda")
    calls = {"gemm_gated_nt": lambda w: pws.gemm_gated_nt(x, w, w), "gemm_f16_nt": lambda w: pws.gemm_f16_nt(x, w),
             "gemm_xent_nt": lambda w: pws.gemm_xent_nt(x, w, target)[0]}
    for name, call in calls.items():
        want = call(w)
        with pytest.warns(UserWarning, match=f"{name} is not recorded"):
            got = call(w.clone().requires_grad_())
        assert not got.requires_grad and torch.equal(got, want)

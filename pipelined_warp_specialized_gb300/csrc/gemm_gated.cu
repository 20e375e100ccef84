// gemm_gated.cu -- the gated feed-forward block h = act(x Wg^T) * (x Wu^T) and
// its backward pass.
//
// Forward: one product with the gate's and the up projection's rows side by
// side in every tile (the first and second half of the accumulator's
// columns), so x is read once and the activation and the product happen in
// the epilogue on fp32 sums: h is rounded once, and g, u are rounded only to
// be kept for the backward pass.
//
// Backward: dg = dh u act'(g) and du = dh act(g) elementwise, rounded to the
// inputs' type because the tensor cores multiply 16-bit operands (the rounding
// an unfused backward pass makes as well); then dx = dg Wg + du Wu as one
// accumulation over both weights, and dWg = dg^T x, dWu = du^T x as one launch.
//
// In binary16 dh is first multiplied by the power of two that brings a bound of
// the largest |dg| and |du| (gated_top_kernel) into [2^14, 2^15), undone in fp32
// when dx, dWg and dWu are rounded: gradients of 1e-5 would otherwise lie below
// its normal range and lose their bits (dx of 2048 tokens off by 2.2 times its
// own rounding), and large ones would pass 65504 where dx and dW do not.  An element is
// then held to half a unit, or to 2^-39 of that bound.  bfloat16 has fp32's range
// and no scale.
#include "product_host.cuh"

namespace pws {
namespace fused {
namespace {

// Eight consecutive elements of a row at any 2-byte alignment; `left` of them
// are in the row (the rest are returned as zeros).
__device__ __forceinline__ uint4 load8(const uint16_t* src, int64_t left) {
    if (left >= 8) return load_unaligned16(src);
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = (2 * i < left ? src[2 * i] : 0u) | ((2 * i + 1 < left ? src[2 * i + 1] : 0u) << 16);
    return make_uint4(v[0], v[1], v[2], v[3]);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Binary16: the largest finite 1.13 |dh u| or |dh| max(g, 0.28), one value a block
// (of kTopParts).  No |dg| or |du| is above it: |act'| < 1.13 and -0.28 < act(g) <=
// max(g, 0) for both activations, so the pass needs no exponential and is bound by
// its reads (the exact maximum, with one, took twice as long).  The matrices are
// dense, so rows do not matter; they are read from the end, so that
// gated_grad_kernel begins with what L2 still holds.  What the scale costs: the
// backward pass of 8192 x 8192 x 4096 1444 to 1500 us, of 1000 x 2731 x 1030 38.3
// to 43.8, of one token through 4096 x 1024 15.1 to 16.9.
constexpr int kTopParts = 152;
constexpr int kTopThreads = 1024;

// The larger of two values, `a` where b is not finite.
__device__ __forceinline__ float finite_max(float a, float b) { return b <= 3.0e38f ? fmaxf(a, b) : a; }
// dg's bound and du's apart: an infinite u leaves du finite.
__device__ __forceinline__ float grad_bound(float top, float dh, float g, float u) {
    return finite_max(finite_max(top, fabsf(1.13f * dh * u)), fabsf(dh) * fmaxf(g, 0.28f));
}

template <bool ALIGNED>
__global__ void __launch_bounds__(kTopThreads)
gated_top_kernel(const uint16_t* __restrict__ dh, const uint16_t* __restrict__ g, const uint16_t* __restrict__ u,
                 int64_t count, float* __restrict__ parts) {
    grid_dependency_wait();
    allow_dependent_launch();
    __shared__ float part[kTopThreads / 32];
    float top = 0.0f;
    const auto load = [](const uint16_t* src) {
        return ALIGNED ? __ldg(reinterpret_cast<const uint4*>(src)) : load_unaligned16(src);
    };
    const auto take = [&](const uint4& a, const uint4& b, const uint4& d) {
        const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w}, dv[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 h2 = unpack16(av[j], 0), g2 = unpack16(bv[j], 0), u2 = unpack16(dv[j], 0);
            top = grad_bound(grad_bound(top, h2.x, g2.x, u2.x), h2.y, g2.y, u2.y);
        }
    };
    // two chunks of eight elements a step: six loads in flight
    const int64_t chunks = count / 8, step = static_cast<int64_t>(kTopParts) * kTopThreads;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(kTopThreads) + threadIdx.x; i < chunks; i += 2 * step) {
        const int64_t at = (chunks - 1 - i) * 8, next = i + step < chunks ? at - step * 8 : at;
        const uint4 a0 = load(dh + at), b0 = load(g + at), d0 = load(u + at);
        const uint4 a1 = load(dh + next), b1 = load(g + next), d1 = load(u + next);
        take(a0, b0, d0);
        take(a1, b1, d1);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0 && count % 8)
        take(load8(dh + chunks * 8, count % 8), load8(g + chunks * 8, count % 8), load8(u + chunks * 8, count % 8));
    top = warp_max(top);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = top;
    __syncthreads();
    if (threadIdx.x < 32) {
        top = warp_max(part[threadIdx.x]);
        if (threadIdx.x == 0) parts[blockIdx.x] = top;
    }
}

// The power of two that brings the largest of the parts into [2^14, 2^15), and
// its inverse (both normal: the exponent is held at 15 or more).  A warp's work.
__device__ __forceinline__ float grad_scale(const float* parts, float& inverse) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < (kTopParts + 31) / 32; ++i) {
        const int at = i * 32 + static_cast<int>(threadIdx.x % 32);
        if (at < kTopParts) top = fmaxf(top, parts[at]);
    }
    top = warp_max(top);
    const int e = max(static_cast<int>(__float_as_uint(top) >> 23), 15);     // biased exponent
    inverse = __uint_as_float(static_cast<uint32_t>(e - 14) << 23);
    return __uint_as_float(static_cast<uint32_t>(254 + 14 - e) << 23);
}

// dg, du [M, F] with rows ldo apart (a multiple of 64) from dh, g, u [M, F]
// (dense), times a power of two (grad_scale) where `parts` is given; with lo_offset
// also what their rounding left, that many elements further.  Memory bound: reads three and writes two 16-bit matrices.  Eight
// elements a thread; a block takes one row's next 256 threads' worth, so
// nothing divides.  Rows that do not start on 16-byte boundaries (odd F) are
// shifted into place from aligned loads: an element a thread took 14 us
// instead of 10.6 at 1000 x 2731.
__global__ void __launch_bounds__(256)
gated_grad_kernel(const uint16_t* __restrict__ dh, const uint16_t* __restrict__ g, const uint16_t* __restrict__ u,
                  uint16_t* __restrict__ dg, uint16_t* __restrict__ du, int F, int64_t ldo, int64_t lo_offset, int act,
                  int bf16, const float* __restrict__ parts, float* __restrict__ inv_scale) {
    grid_dependency_wait();
    allow_dependent_launch();
    const int64_t row = blockIdx.x;
    float scale = 1.0f;
    if (parts) {
        float inverse;
        scale = grad_scale(parts, inverse);
        if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *inv_scale = inverse;
    }
    for (int64_t c = (blockIdx.y * static_cast<int64_t>(blockDim.x) + threadIdx.x) * 8; c < F;
         c += static_cast<int64_t>(gridDim.y) * blockDim.x * 8) {
        const int64_t at = row * F + c, to = row * ldo + c;
        const uint4 a = load8(dh + at, F - c), b = load8(g + at, F - c), d = load8(u + at, F - c);
        const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w}, dv[4] = {d.x, d.y, d.z, d.w};
        uint32_t og[4], ou[4], rg[4], ru[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 h2 = unpack16(av[j], bf16), g2 = unpack16(bv[j], bf16), u2 = unpack16(dv[j], bf16);
            float v0, s0, v1, s1;
            act_value_slope(g2.x, act, v0, s0);
            act_value_slope(g2.y, act, v1, s1);
            const float h0 = scale * h2.x, h1 = scale * h2.y;
            const float g0 = h0 * u2.x * s0, g1 = h1 * u2.y * s1, u0 = h0 * v0, u1 = h1 * v1;
            og[j] = pack16(g0, g1, bf16);
            ou[j] = pack16(u0, u1, bf16);
            const float2 cg = unpack16(og[j], bf16), cu = unpack16(ou[j], bf16);
            rg[j] = pack16(remainder16(g0, cg.x), remainder16(g1, cg.y), bf16);
            ru[j] = pack16(remainder16(u0, cu.x), remainder16(u1, cu.y), bf16);
        }
        // (a last chunk's zeros lie inside the padded row)
        *reinterpret_cast<uint4*>(dg + to) = make_uint4(og[0], og[1], og[2], og[3]);
        *reinterpret_cast<uint4*>(du + to) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
        if (lo_offset) {
            *reinterpret_cast<uint4*>(dg + to + lo_offset) = make_uint4(rg[0], rg[1], rg[2], rg[3]);
            *reinterpret_cast<uint4*>(du + to + lo_offset) = make_uint4(ru[0], ru[1], ru[2], ru[3]);
        }
    }
}

bool bad_codes(int type, int act) {
    return (type != GEMM_TYPE_HALF && type != GEMM_TYPE_BFLOAT) || (act != GEMM_ACT_SILU && act != GEMM_ACT_GELU);
}

int check_gated(int64_t M, int64_t F, int64_t K, const void* x, const void* wg, const void* wu, const void* h,
                const void* g, const void* u, int type, int act) {
    if (bad_size(M) || bad_size(F) || bad_size(K) || bad_codes(type, act)) return GEMM_ERR_INVALID_ARG;
    if (too_many_tiles(M, F)) return GEMM_ERR_INVALID_ARG;
    if ((g == nullptr) != (u == nullptr)) return GEMM_ERR_INVALID_ARG;
    if (odd_address(x) || odd_address(wg) || odd_address(wu) || odd_address(h) || odd_address(g) || odd_address(u))
        return GEMM_ERR_ALIGNMENT;
    if (M > 0 && F > 0 && K > 0 && (!x || !wg || !wu)) return GEMM_ERR_INVALID_ARG;
    const Range in[3] = {{x, bytes16(M, K)}, {wg, bytes16(F, K)}, {wu, bytes16(F, K)}};
    const Range out[3] = {{h, bytes16(M, F)}, {g, bytes16(M, F)}, {u, bytes16(M, F)}};
    return overlaps(in, out) ? GEMM_ERR_INVALID_ARG : GEMM_OK;
}

struct GatedPlan {
    Product pr;
    Layout l;
    Source x, wg, wu;
    size_t bytes = 0;
};

// num_sms 0: the workspace only.
GatedPlan plan_gated(int64_t M, int64_t F, int64_t K, const void* x, const void* wg, const void* wu, int num_sms,
                     void* ws) {
    GatedPlan pl;
    Carver c;
    c.base = static_cast<char*>(ws);
    pl.pr.M = M; pl.pr.N = F; pl.pr.K = K;
    pl.pr.gated = true;
    if (num_sms) pl.l = choose_layout(pl.pr, num_sms);
    pl.x = source_of(x, M, K, !tma_ok(x, K), &c);
    // both weights share one row stride
    const bool rw = !tma_ok(wg, K) || !tma_ok(wu, K);
    pl.wg = source_of(wg, F, K, rw, &c);
    pl.wu = source_of(wu, F, K, rw, &c);
    pl.bytes = c.used;
    return pl;
}

int check_gated_bwd(int64_t M, int64_t F, int64_t K, const void* dh, const void* g, const void* u, const void* x,
                    const void* wg, const void* wu, const void* dx, const void* dwg, const void* dwu, int type,
                    int act) {
    if (bad_size(M) || bad_size(F) || bad_size(K) || bad_codes(type, act)) return GEMM_ERR_INVALID_ARG;
    if (too_many_tiles(M, K) || too_many_tiles(2 * F, K)) return GEMM_ERR_INVALID_ARG;
    if ((dwg == nullptr) != (dwu == nullptr)) return GEMM_ERR_INVALID_ARG;
    const void* all[9] = {dh, g, u, x, wg, wu, dx, dwg, dwu};
    for (const void* q : all)
        if (odd_address(q)) return GEMM_ERR_ALIGNMENT;
    if (M > 0 && F > 0 && K > 0 && (!dh || !g || !u || (dwg && !x) || (dx && (!wg || !wu))))
        return GEMM_ERR_INVALID_ARG;
    const Range in[6] = {{dh, bytes16(M, F)}, {g, bytes16(M, F)},  {u, bytes16(M, F)},
                         {x, bytes16(M, K)},  {wg, bytes16(F, K)}, {wu, bytes16(F, K)}};
    const Range out[3] = {{dx, bytes16(M, K)}, {dwg, bytes16(F, K)}, {dwu, bytes16(F, K)}};
    return overlaps(in, out) ? GEMM_ERR_INVALID_ARG : GEMM_OK;
}

struct GatedBwdPlan {
    StoreProduct sp[2];             // dx and dW, those that are wanted
    int n = 0;
    Layout l;
    Source x, wg, wu;
    uint16_t* dg = nullptr;
    uint16_t* du = nullptr;
    float* top_parts = nullptr;     // binary16: kTopParts, and the scale's inverse
    float* inv_scale = nullptr;
    int64_t ldf = 0, lo_offset = 0;
    size_t bytes = 0;
};

GatedBwdPlan plan_gated_bwd(int64_t M, int64_t F, int64_t K, const void* x, const void* wg, const void* wu,
                            bool want_dx, bool want_dw, int type, int num_sms, void* ws) {
    GatedBwdPlan pl;
    Carver c;
    c.base = static_cast<char*>(ws);
    pl.ldf = round_up(F, 64);
    const int halves = M <= kFewRows ? 2 : 1;
    pl.lo_offset = halves == 2 ? M * pl.ldf : 0;
    pl.dg = c.take<uint16_t>(halves * M * pl.ldf);
    pl.du = c.take<uint16_t>(halves * M * pl.ldf);
    if (type == GEMM_TYPE_HALF) {
        pl.top_parts = c.take<float>(kTopParts);
        pl.inv_scale = c.take<float>(1);
    }
    Product pr[2];
    if (want_dx) {
        // the gate's F and the up projection's F are two segments of K; the
        // remainders are M more rows
        Product& d = pr[pl.n++];
        d.M = halves * M; d.N = K; d.K = F;
        d.halves = halves;
        d.segments = 2;
        d.bmn = true;
        d.may_split = true;
    }
    if (want_dw) {
        // the remainders are M more tokens
        Product& d = pr[pl.n++];
        d.M = F; d.N = K; d.K = M;
        d.problems = 2;
        d.segments = halves;
        d.amn = d.bmn = true;
        d.may_split = true;
    }
    pl.x = source_of(x, M, K, want_dw && !tma_ok(x, K), &c);
    const bool rw = want_dx && (!tma_ok(wg, K) || !tma_ok(wu, K));
    pl.wg = source_of(wg, F, K, rw, &c);
    pl.wu = source_of(wu, F, K, rw, &c);
    pl.l = choose_layout(pr, pl.n, num_sms);
    for (int i = 0; i < pl.n; ++i) {
        pl.sp[i].pr = pr[i];
        pl.sp[i].partial = c.take<float>(split_floats(pr[i], pl.l.part[i]));
    }
    pl.bytes = c.used;
    return pl;
}

int zero16(void* p, int64_t rows, int64_t cols, cudaStream_t stream) {
    if (!p || rows == 0 || cols == 0) return GEMM_OK;
    return cudaMemsetAsync(p, 0, bytes16(rows, cols), stream) == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // namespace
}  // namespace fused
}  // namespace pws

extern "C" int gemm_gated_nt_workspace(int64_t M, int64_t F, int64_t K, const void* x, const void* w_gate,
                                       const void* w_up, int type, int64_t* bytes) {
    using namespace pws::fused;
    const int rc = check_gated(M, F, K, x, w_gate, w_up, nullptr, nullptr, nullptr, type, GEMM_ACT_SILU);
    if (rc != GEMM_OK) return rc;
    if (!bytes) return GEMM_ERR_INVALID_ARG;
    *bytes = M && F && K ? static_cast<int64_t>(plan_gated(M, F, K, x, w_gate, w_up, 0, nullptr).bytes) : 0;
    return GEMM_OK;
}

extern "C" int gemm_gated_nt(int64_t M, int64_t F, int64_t K, const void* x, const void* w_gate, const void* w_up,
                             void* h, void* g, void* u, int type, int act, void* workspace, int64_t workspace_bytes,
                             cudaStream_t stream) {
    using namespace pws;
    using namespace pws::fused;
    int rc = check_gated(M, F, K, x, w_gate, w_up, h, g, u, type, act);
    if (rc != GEMM_OK) return rc;
    if (M == 0 || F == 0) return GEMM_OK;
    if (!h) return GEMM_ERR_INVALID_ARG;
    DeviceInfo info;
    rc = current_device(&info);
    if (rc != GEMM_OK) return rc;
    if (K == 0) {
        // g = u = 0, so h = act(0) * 0 = 0
        if ((rc = zero16(h, M, F, stream)) != GEMM_OK) return rc;
        if ((rc = zero16(g, M, F, stream)) != GEMM_OK) return rc;
        return zero16(u, M, F, stream);
    }
    GatedPlan pl = plan_gated(M, F, K, x, w_gate, w_up, info.num_sms, workspace);
    const Range in[3] = {{x, bytes16(M, K)}, {w_gate, bytes16(F, K)}, {w_up, bytes16(F, K)}};
    const Range out[3] = {{h, bytes16(M, F)}, {g, bytes16(M, F)}, {u, bytes16(M, F)}};
    if (!workspace_ok(workspace, workspace_bytes, pl.bytes, in, out)) return GEMM_ERR_INVALID_ARG;
    if ((rc = fill_sources({{&pl.x, M}, {&pl.wg, F}, {&pl.wu, F}}, K, stream)) != GEMM_OK) return rc;
    Maps maps;
    memset(&maps, 0, sizeof(maps));
    Params p = base_params(pl.l, type, info, stream);
    Operands op;
    op.a[0] = pl.x.ptr;
    op.lda = pl.x.ld;
    op.b[0] = pl.wg.ptr;
    op.b[1] = pl.wu.ptr;
    op.ldb = pl.wg.ld;
    if (!set_job(&p, &maps, 0, pl.pr, pl.l, pl.l.part[0], op)) return GEMM_ERR_LAUNCH;
    p.act = act;
    Job& j = p.job[0];
    j.ld16 = F;
    j.out16[0] = static_cast<uint16_t*>(h);
    p.g_out = static_cast<uint16_t*>(g);
    p.u_out = static_cast<uint16_t*>(u);
    j.tma_store = output_map(&maps.c[0], pl.l, h, M, F, F) &&
                  (!g || (output_map(&maps.c[1], pl.l, g, M, F, F) && output_map(&maps.c[2], pl.l, u, M, F, F)));
    return launch_product<kEpiGated>(pl.l, maps, p, info, stream);
}

extern "C" int gemm_gated_nt_bwd_workspace(int64_t M, int64_t F, int64_t K, const void* dh, const void* g,
                                           const void* u, const void* x, const void* w_gate, const void* w_up,
                                           int type, int64_t* bytes) {
    using namespace pws::fused;
    const int rc = check_gated_bwd(M, F, K, dh, g, u, x, w_gate, w_up, nullptr, nullptr, nullptr, type, GEMM_ACT_SILU);
    if (rc != GEMM_OK) return rc;
    if (!bytes) return GEMM_ERR_INVALID_ARG;
    *bytes = 0;
    if (M && F && K) {
        // one side's gradients alone may be split further than all together
        const int sms = pws::sm_count_or_default();
        for (int want = 1; want <= 3; ++want) {
            const int64_t b = static_cast<int64_t>(
                plan_gated_bwd(M, F, K, x, w_gate, w_up, want & 1, want & 2, type, sms, nullptr).bytes);
            if (b > *bytes) *bytes = b;
        }
    }
    return GEMM_OK;
}

extern "C" int gemm_gated_nt_bwd(int64_t M, int64_t F, int64_t K, const void* dh, const void* g, const void* u,
                                 const void* x, const void* w_gate, const void* w_up, void* dx, void* dw_gate,
                                 void* dw_up, int type, int act, void* workspace, int64_t workspace_bytes,
                                 cudaStream_t stream) {
    using namespace pws;
    using namespace pws::fused;
    int rc = check_gated_bwd(M, F, K, dh, g, u, x, w_gate, w_up, dx, dw_gate, dw_up, type, act);
    if (rc != GEMM_OK) return rc;
    if (K == 0 || (M == 0 && F == 0) || (!dx && !dw_gate)) return GEMM_OK;
    DeviceInfo info;
    rc = current_device(&info);
    if (rc != GEMM_OK) return rc;
    if (M == 0 || F == 0) {
        if ((rc = zero16(dx, M, K, stream)) != GEMM_OK) return rc;
        if ((rc = zero16(dw_gate, F, K, stream)) != GEMM_OK) return rc;
        return zero16(dw_up, F, K, stream);
    }
    GatedBwdPlan pl = plan_gated_bwd(M, F, K, x, w_gate, w_up, dx != nullptr, dw_gate != nullptr, type,
                                     info.num_sms, workspace);
    const Range in[6] = {{dh, bytes16(M, F)}, {g, bytes16(M, F)},      {u, bytes16(M, F)},
                         {x, bytes16(M, K)},  {w_gate, bytes16(F, K)}, {w_up, bytes16(F, K)}};
    const Range out[3] = {{dx, bytes16(M, K)}, {dw_gate, bytes16(F, K)}, {dw_up, bytes16(F, K)}};
    if (!workspace_ok(workspace, workspace_bytes, pl.bytes, in, out)) return GEMM_ERR_INVALID_ARG;
    if ((rc = fill_sources({{&pl.x, M}, {&pl.wg, F}, {&pl.wu, F}}, K, stream)) != GEMM_OK) return rc;
    if (pl.top_parts) {
        const auto kern = tma_ok(dh, 0) && tma_ok(g, 0) && tma_ok(u, 0) ? gated_top_kernel<true> : gated_top_kernel<false>;
        if (launch_pdl(kern, dim3(kTopParts), dim3(kTopThreads), 0, stream, static_cast<const uint16_t*>(dh),
                       static_cast<const uint16_t*>(g), static_cast<const uint16_t*>(u), M * F, pl.top_parts) !=
            cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_LAUNCH;
        }
    }
    {
        int64_t across = cdiv(F, 8 * 256);
        if (across > 65535) across = 65535;
        if (launch_pdl(gated_grad_kernel, dim3(static_cast<unsigned>(M), static_cast<unsigned>(across)), dim3(256), 0, stream,
                       static_cast<const uint16_t*>(dh), static_cast<const uint16_t*>(g),
                       static_cast<const uint16_t*>(u), pl.dg, pl.du, static_cast<int>(F), pl.ldf,
                       pl.lo_offset, act, type == GEMM_TYPE_BFLOAT ? 1 : 0,
                       static_cast<const float*>(pl.top_parts), pl.inv_scale) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_LAUNCH;
        }
    }
    for (int i = 0; i < pl.n; ++i) {
        StoreProduct& q = pl.sp[i];
        q.scale = pl.inv_scale;
        q.op.lda = pl.ldf;
        if (q.pr.amn) {
            q.op.a[0] = pl.dg;
            q.op.a[1] = pl.dg + pl.lo_offset;
            q.op.a[2] = pl.du;
            q.op.a[3] = pl.du + pl.lo_offset;
            q.op.b[0] = pl.x.ptr;
            q.op.ldb = pl.x.ld;
            q.out16[0] = dw_gate;
            q.out16[1] = dw_up;
        } else {
            q.op.a[0] = pl.dg;
            q.op.a[1] = pl.du;
            q.op.b[0] = pl.wg.ptr;
            q.op.b[1] = pl.wu.ptr;
            q.op.ldb = pl.wg.ld;
            q.out16[0] = dx;
        }
    }
    return run_store_products(pl.sp, pl.n, pl.l, type, info, stream);
}

// gemm_xent.cu -- softmax cross entropy over a linear head, without keeping
// the logits z = x W^T.
//
// Forward: the product's epilogue reduces each tile's columns of a row to
// their maximum and sum of exponentials (fp32, from the fp32 accumulator), and
// keeps the target's logit; a second kernel joins the tiles' pairs in a fixed
// order:  lse = m + log sum_t s_t exp(m_t - m),  loss = lse - z_target.
//
// Backward: the vocabulary is taken in pieces.  For each piece the logits are
// computed again, summed over K in the forward pass's chunks (in one run, a
// confident target's 1 - p of 9e-4 was off by 3.5e-4 over K = 8192), the epilogue turns them into D = dloss (exp(z - lse) -
// onehot) in 16 bits, and the piece's two products follow: dx += D W (fp32
// between pieces) and the piece's rows of dW = D^T x.  The largest buffer is
// one piece of D.
//
// D is rounded to the inputs' type because the tensor cores multiply 16-bit
// operands of one type.  It is scaled so that the largest |dloss| becomes 2^13,
// undone in fp32 when dx and dW are rounded: without it binary16 would lose
// the probabilities below 6e-8 / dloss, and with it the usual uniform dloss
// adds no rounding of its own (2^13 (p - 1) rounds as p - 1 does).  One scale serves
// all rows, since dW sums over them: an element keeps half a unit or 2^-38 of the
// largest |dloss|.  With few rows D keeps its rounding remainder too (kFewRows).
#include "product_host.cuh"

namespace pws {
namespace fused {
namespace {

// One block: the largest finite |dloss| of a row that counts, brought to 2^13;
// per row the scaled loss gradient, 0 for an ignored row, NaN for a target
// outside the vocabulary.
__global__ void __launch_bounds__(1024)
xent_rows_kernel(const int64_t* __restrict__ target, const float* __restrict__ dloss, int M, int64_t V,
                 int64_t ignore_index, float* __restrict__ coef, float* __restrict__ inv_scale) {
    grid_dependency_wait();
    allow_dependent_launch();
    __shared__ float part[32];
    float top = 0.0f;
#pragma unroll 8
    for (int i = threadIdx.x; i < M; i += blockDim.x) {
        const float d = fabsf(dloss[i]);
        if (target[i] != ignore_index && d <= 3.0e38f) top = fmaxf(top, d);     // (finite ones)
    }
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = top;
    __syncthreads();
    top = part[threadIdx.x % 32];
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    top = fmaxf(top, 1e-30f);
    if (threadIdx.x == 0) *inv_scale = top * (1.0f / 8192.0f);
#pragma unroll 8
    for (int i = threadIdx.x; i < M; i += blockDim.x) {
        const int64_t t = target[i];
        float c = 0.0f;
        if (t != ignore_index) c = t >= 0 && t < V ? dloss[i] / top * 8192.0f : __int_as_float(0x7fffffff);
        coef[i] = c;
    }
}

// One block per row joins its half tiles' (maximum, sum) pairs, in an order
// that depends on their number alone.  tiles == 0: K == 0, every logit is 0.
__global__ void __launch_bounds__(128)
xent_join_kernel(const float2* __restrict__ stats, const float* __restrict__ z_target,
                 const int64_t* __restrict__ target, int tiles, int64_t V, int64_t ignore_index,
                 float* __restrict__ loss, float* __restrict__ lse) {
    grid_dependency_wait();
    allow_dependent_launch();
    __shared__ float2 part[4];
    const int64_t row = blockIdx.x;
    const float inf = __int_as_float(0x7f800000);
    const auto join = [&](float2 a, float2 b) {
        const float top = fmaxf(a.x, b.x);
        const float ref = top == -inf ? 0.0f : top;
        return make_float2(top, a.y * expf(a.x - ref) + b.y * expf(b.x - ref));
    };
    float2 v = make_float2(-inf, 0.0f);
    const float2* mine = stats + row * tiles;
    for (int t0 = threadIdx.x; t0 < tiles; t0 += 4 * 128) {
        float2 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = t0 + i * 128 < tiles ? mine[t0 + i * 128] : make_float2(-inf, 0.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i) v = join(v, w[i]);
    }
    for (int o = 16; o > 0; o >>= 1)
        v = join(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        v = join(join(part[0], part[1]), join(part[2], part[3]));
        const float total = tiles ? v.x + logf(v.y) : logf(static_cast<float>(V));
        const int64_t t = target[row];
        float l = 0.0f;
        if (t != ignore_index) l = t >= 0 && t < V ? total - (tiles ? z_target[row] : 0.0f) : __int_as_float(0x7fffffff);
        lse[row] = total;
        loss[row] = l;
    }
}

int check_xent(int64_t M, int64_t V, int64_t K, const void* x, const void* w, const int64_t* target, int type) {
    if (bad_size(M) || bad_size(V) || bad_size(K) || V == 0) return GEMM_ERR_INVALID_ARG;
    if (type != GEMM_TYPE_HALF && type != GEMM_TYPE_BFLOAT) return GEMM_ERR_INVALID_ARG;
    if (too_many_tiles(M, V)) return GEMM_ERR_INVALID_ARG;
    if (odd_address(x) || odd_address(w) || reinterpret_cast<uintptr_t>(target) % 8 != 0) return GEMM_ERR_ALIGNMENT;
    if (M > 0 && (!target || (K > 0 && (!x || !w)))) return GEMM_ERR_INVALID_ARG;
    return GEMM_OK;
}

bool odd_float(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 != 0; }

struct XentPlan {
    Product pr;
    Layout l;
    Source x, w;
    float2* stats = nullptr;
    float* z_target = nullptr;
    size_t bytes = 0;
};

// The logits of `v` columns.  Their chunk goes by the rows alone, so that the
// forward and the backward pass, whose tiles differ, sum a logit alike.
Product logits_of(int64_t M, int64_t v, int64_t K) {
    Product p;
    p.M = M; p.N = v; p.K = K;
    p.chunk = M > BM_CTA ? kLogitsChunk : kLogitsChunkFew;
    return p;
}

XentPlan plan_xent(int64_t M, int64_t V, int64_t K, const void* x, const void* w, int num_sms, void* ws) {
    XentPlan pl;
    Carver c;
    c.base = static_cast<char*>(ws);
    pl.pr = logits_of(M, V, K);
    pl.l = choose_layout(pl.pr, num_sms);
    pl.x = source_of(x, M, K, !tma_ok(x, K), &c);
    pl.w = source_of(w, V, K, !tma_ok(w, K), &c);
    pl.stats = c.take<float2>(2ll * pl.l.part[0].tiles_n * M);
    pl.z_target = c.take<float>(M);
    pl.bytes = c.used;
    return pl;
}

// Bytes of D a piece may take; at least kMinPiece columns.
constexpr int64_t kPieceBytes = 256ll << 20;
constexpr int64_t kMinPiece = 8192;

struct XentBwdPlan {
    int64_t piece = 0, ldd = 0, lo_offset = 0;
    int halves = 1;
    int pieces = 0;
    Source x, w;
    float* coef = nullptr;
    float* inv_scale = nullptr;
    uint16_t* d = nullptr;
    float* acc = nullptr;
    float* partial[2] = {nullptr, nullptr};
    size_t bytes = 0;
};

// The gradients' products of a piece of `v` columns: dx and dW, those that are
// wanted.
int grads_of(int64_t M, int64_t v, int64_t K, int halves, bool want_dx, bool want_dw, Product (&pr)[2]) {
    int n = 0;
    if (want_dx) {
        Product& d = pr[n++];
        d.M = halves * M; d.N = K; d.K = v;
        d.halves = halves;          // the remainders are M more rows
        d.bmn = true;
        d.may_split = true;
    }
    if (want_dw) {
        Product& d = pr[n++];
        d.M = v; d.N = K; d.K = M;
        d.segments = halves;        // the remainders are M more tokens
        d.amn = d.bmn = true;
        d.may_split = true;
    }
    return n;
}

XentBwdPlan plan_xent_bwd(int64_t M, int64_t V, int64_t K, const void* x, const void* w, bool want_dx, bool want_dw,
                          int num_sms, void* ws) {
    XentBwdPlan pl;
    Carver c;
    c.base = static_cast<char*>(ws);
    int64_t cols = kPieceBytes / (2 * M);
    if (cols < kMinPiece) cols = kMinPiece;
    pl.pieces = static_cast<int>(cdiv(V, cols));
    pl.piece = round_up(cdiv(V, pl.pieces), 256);
    pl.pieces = static_cast<int>(cdiv(V, pl.piece));
    pl.ldd = pl.pieces > 1 ? pl.piece : round_up(V, 64);
    pl.halves = M <= kFewRows ? 2 : 1;
    pl.lo_offset = pl.halves == 2 ? M * pl.ldd : 0;
    pl.x = source_of(x, M, K, !tma_ok(x, K), &c);
    pl.w = source_of(w, V, K, !tma_ok(w, K), &c);
    pl.coef = c.take<float>(M);
    pl.inv_scale = c.take<float>(1);
    pl.d = c.take<uint16_t>(pl.halves * M * pl.ldd);
    if (want_dx && pl.pieces > 1) pl.acc = c.take<float>(M * ld32_of(K));
    // the pieces share the space for partial sums; the last one's width differs
    int64_t most[2] = {0, 0};
    for (int i = 0; i < (pl.pieces > 1 ? 2 : 1); ++i) {
        const int64_t v = i || pl.pieces == 1 ? V - (pl.pieces - 1) * pl.piece : pl.piece;
        Product pr[2];
        const int n = grads_of(M, v, K, pl.halves, want_dx, want_dw, pr);
        const Layout l = choose_layout(pr, n, num_sms);
        for (int k = 0; k < n; ++k) {
            const int64_t f = split_floats(pr[k], l.part[k]);
            if (f > most[k]) most[k] = f;
        }
    }
    for (int k = 0; k < 2; ++k) pl.partial[k] = c.take<float>(most[k]);
    pl.bytes = c.used;
    return pl;
}

}  // namespace
}  // namespace fused
}  // namespace pws

extern "C" int gemm_xent_nt_workspace(int64_t M, int64_t V, int64_t K, const void* x, const void* w, int type,
                                      int64_t* bytes) {
    using namespace pws::fused;
    const int64_t* any = reinterpret_cast<const int64_t*>(static_cast<uintptr_t>(8));       // (not read)
    const int rc = check_xent(M, V, K, x, w, any, type);
    if (rc != GEMM_OK) return rc;
    if (!bytes) return GEMM_ERR_INVALID_ARG;
    *bytes = M && K ? static_cast<int64_t>(plan_xent(M, V, K, x, w, pws::sm_count_or_default(), nullptr).bytes) : 0;
    return GEMM_OK;
}

extern "C" int gemm_xent_nt(int64_t M, int64_t V, int64_t K, const void* x, const void* w, const int64_t* target,
                            int64_t ignore_index, float* loss, float* lse, int type, void* workspace,
                            int64_t workspace_bytes, cudaStream_t stream) {
    using namespace pws;
    using namespace pws::fused;
    int rc = check_xent(M, V, K, x, w, target, type);
    if (rc != GEMM_OK) return rc;
    if (M == 0) return GEMM_OK;
    if (!loss || !lse) return GEMM_ERR_INVALID_ARG;
    if (odd_float(loss) || odd_float(lse)) return GEMM_ERR_ALIGNMENT;
    const uint64_t row_bytes = static_cast<uint64_t>(M) * 4;
    const Range in[3] = {{x, bytes16(M, K)}, {w, bytes16(V, K)}, {target, 2 * row_bytes}};
    const Range out[2] = {{loss, row_bytes}, {lse, row_bytes}};
    if (overlaps(in, out)) return GEMM_ERR_INVALID_ARG;
    DeviceInfo info;
    rc = current_device(&info);
    if (rc != GEMM_OK) return rc;
    XentPlan pl;
    if (K > 0) {
        pl = plan_xent(M, V, K, x, w, info.num_sms, workspace);
        if (!workspace_ok(workspace, workspace_bytes, pl.bytes, in, out)) return GEMM_ERR_INVALID_ARG;
        if ((rc = fill_sources({{&pl.x, M}, {&pl.w, V}, {}}, K, stream)) != GEMM_OK) return rc;
        Maps maps;
        memset(&maps, 0, sizeof(maps));
        Params p = base_params(pl.l, type, info, stream);
        Operands op;
        op.a[0] = pl.x.ptr;
        op.lda = pl.x.ld;
        op.b[0] = pl.w.ptr;
        op.ldb = pl.w.ld;
        if (!set_job(&p, &maps, 0, pl.pr, pl.l, pl.l.part[0], op)) return GEMM_ERR_LAUNCH;
        p.target = target;
        p.stats = pl.stats;
        p.z_target = pl.z_target;
        rc = launch_product<kEpiXentStats>(pl.l, maps, p, info, stream);
        if (rc != GEMM_OK) return rc;
    }
    if (launch_pdl(xent_join_kernel, dim3(static_cast<unsigned>(M)), dim3(128), 0, stream,
                   static_cast<const float2*>(pl.stats), static_cast<const float*>(pl.z_target), target,
                   K > 0 ? 2 * pl.l.part[0].tiles_n : 0, V, ignore_index, loss, lse) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

extern "C" int gemm_xent_nt_bwd_workspace(int64_t M, int64_t V, int64_t K, const void* x, const void* w, int type,
                                          int64_t* bytes) {
    using namespace pws::fused;
    const int64_t* any = reinterpret_cast<const int64_t*>(static_cast<uintptr_t>(8));       // (not read)
    const int rc = check_xent(M, V, K, x, w, any, type);
    if (rc != GEMM_OK) return rc;
    if (too_many_tiles(M, K) || too_many_tiles(V, K)) return GEMM_ERR_INVALID_ARG;
    if (!bytes) return GEMM_ERR_INVALID_ARG;
    *bytes = 0;
    if (M && K) {
        // one gradient alone may be split further than the two together
        const int sms = pws::sm_count_or_default();
        for (int want = 1; want <= 3; ++want) {
            const int64_t b =
                static_cast<int64_t>(plan_xent_bwd(M, V, K, x, w, want & 1, want & 2, sms, nullptr).bytes);
            if (b > *bytes) *bytes = b;
        }
    }
    return GEMM_OK;
}

extern "C" int gemm_xent_nt_bwd(int64_t M, int64_t V, int64_t K, const void* x, const void* w, const int64_t* target,
                                int64_t ignore_index, const float* lse, const float* dloss, void* dx, void* dw,
                                int type, void* workspace, int64_t workspace_bytes, cudaStream_t stream) {
    using namespace pws;
    using namespace pws::fused;
    int rc = check_xent(M, V, K, x, w, target, type);
    if (rc != GEMM_OK) return rc;
    if (too_many_tiles(M, K) || too_many_tiles(V, K)) return GEMM_ERR_INVALID_ARG;
    if (odd_address(dx) || odd_address(dw) || odd_float(lse) || odd_float(dloss)) return GEMM_ERR_ALIGNMENT;
    if (M > 0 && (!lse || !dloss)) return GEMM_ERR_INVALID_ARG;
    const uint64_t row_bytes = static_cast<uint64_t>(M) * 4;
    const Range in[5] = {{x, bytes16(M, K)}, {w, bytes16(V, K)}, {target, 2 * row_bytes}, {lse, row_bytes},
                         {dloss, row_bytes}};
    const Range out[2] = {{dx, bytes16(M, K)}, {dw, bytes16(V, K)}};
    if (overlaps(in, out)) return GEMM_ERR_INVALID_ARG;
    if (K == 0 || (!dx && !dw)) return GEMM_OK;
    DeviceInfo info;
    rc = current_device(&info);
    if (rc != GEMM_OK) return rc;
    if (M == 0)
        return !dw || cudaMemsetAsync(dw, 0, bytes16(V, K), stream) == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
    XentBwdPlan pl = plan_xent_bwd(M, V, K, x, w, dx != nullptr, dw != nullptr, info.num_sms, workspace);
    if (!workspace_ok(workspace, workspace_bytes, pl.bytes, in, out)) return GEMM_ERR_INVALID_ARG;
    if ((rc = fill_sources({{&pl.x, M}, {&pl.w, V}, {}}, K, stream)) != GEMM_OK) return rc;
    if (launch_pdl(xent_rows_kernel, dim3(1), dim3(1024), 0, stream, target, dloss, static_cast<int>(M), V,
                   ignore_index, pl.coef, pl.inv_scale) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    for (int i = 0; i < pl.pieces; ++i) {
        const int64_t v0 = i * pl.piece, v = V - v0 < pl.piece ? V - v0 : pl.piece;
        const uint16_t* w_piece = static_cast<const uint16_t*>(pl.w.ptr) + v0 * pl.w.ld;
        {
            const Product pr = logits_of(M, v, K);
            const Layout l = choose_layout(pr, info.num_sms);
            Maps maps;
            memset(&maps, 0, sizeof(maps));
            Params p = base_params(l, type, info, stream);
            Operands op;
            op.a[0] = pl.x.ptr;
            op.lda = pl.x.ld;
            op.b[0] = w_piece;
            op.ldb = pl.w.ld;
            if (!set_job(&p, &maps, 0, pr, l, l.part[0], op)) return GEMM_ERR_LAUNCH;
            p.target = target;
            p.lse = lse;
            p.coef = pl.coef;
            p.ignore_index = ignore_index;
            p.col0 = v0;
            p.lo_offset = pl.lo_offset;
            Job& j = p.job[0];
            j.out16[0] = pl.d;
            j.ld16 = pl.ldd;
            j.tma_store = output_map(&maps.c[0], l, pl.d, M, v, pl.ldd) &&
                          (!pl.lo_offset || output_map(&maps.c[1], l, pl.d + pl.lo_offset, M, v, pl.ldd));
            if ((rc = launch_product<kEpiXentGrad>(l, maps, p, info, stream)) != GEMM_OK) return rc;
        }
        Product pr[2];
        StoreProduct sp[2];
        const int n = grads_of(M, v, K, pl.halves, dx != nullptr, dw != nullptr, pr);
        for (int k = 0; k < n; ++k) {
            StoreProduct& q = sp[k];
            q.pr = pr[k];
            q.partial = pl.partial[k];
            q.scale = pl.inv_scale;
            q.op.a[0] = pl.d;
            q.op.lda = pl.ldd;
            if (q.pr.amn) {
                q.op.a[1] = pl.d + pl.lo_offset;
                q.op.b[0] = pl.x.ptr;
                q.op.ldb = pl.x.ld;
                q.out16[0] = static_cast<uint16_t*>(dw) + v0 * K;
            } else {
                q.op.b[0] = w_piece;
                q.op.ldb = pl.w.ld;
                // dx is summed over the pieces in fp32 and rounded by the last one
                q.acc_in = i ? pl.acc : nullptr;
                if (i + 1 < pl.pieces) q.acc_out = pl.acc;
                else q.out16[0] = dx;
            }
        }
        rc = run_store_products(sp, n, choose_layout(pr, n, info.num_sms), type, info, stream);
        if (rc != GEMM_OK) return rc;
    }
    return GEMM_OK;
}

// gemm_bwd.cu -- the backward pass of y = x W^T:  dx = dy W  and  dW = dy^T x,
// and the plain-store products the other operators' backward passes share.
//
// Both read the forward pass's matrices as they lie.  dx contracts over dy's
// columns: dy's rows are K-major, and W [N, K] has the contraction along its
// rows, the MN-major form.  dW contracts over the tokens: both operands are
// MN-major.  Sums are fp32 in tensor memory and are rounded once.
#include "product_host.cuh"

namespace pws {
namespace fused {

namespace {

// Rows of `cols` 16-bit elements at any 2-byte alignment, copied to rows ld
// apart (ld a multiple of 64), up to three matrices in one launch.  A thread
// writes one 16-byte chunk; a row's last, ragged chunk is read element by
// element and padded with zeros.  The chunks of all rows are numbered
// through, so a row of 129 chunks wastes no threads.
struct Rows {
    const uint16_t* src[3];
    uint16_t* dst[3];
    uint32_t first[4];              // first chunk of each matrix, and the total
};

__global__ void __launch_bounds__(256)
align_rows_kernel(const __grid_constant__ Rows r, uint32_t chunks, int64_t cols, int64_t ld) {
    grid_dependency_wait();
    allow_dependent_launch();
    const uint32_t id = blockIdx.x * 256u + threadIdx.x;
    if (id >= r.first[3]) return;
    const int m = id >= r.first[2] ? 2 : (id >= r.first[1] ? 1 : 0);
    const uint32_t in = id - r.first[m], row = in / chunks, j = in - row * chunks;
    const uint16_t* src = r.src[m] + row * cols + 8 * static_cast<int64_t>(j);
    uint4 o;
    if (8 * static_cast<int64_t>(j) + 8 <= cols) {
        o = load_unaligned16(src);
    } else {
        uint32_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t c = 8 * static_cast<int64_t>(j) + 2 * i;
            const uint32_t lo = c < cols ? src[2 * i] : 0u, hi = c + 1 < cols ? src[2 * i + 1] : 0u;
            v[i] = lo | (hi << 16);
        }
        o = make_uint4(v[0], v[1], v[2], v[3]);
    }
    *reinterpret_cast<uint4*>(r.dst[m] + row * ld + 8 * static_cast<int64_t>(j)) = o;
}

}  // namespace

int fill_sources(const Fill (&f)[3], int64_t cols, cudaStream_t stream) {
    const int64_t chunks = cdiv(cols, 8), ld = round_up(cols, 64);
    // as many rows a launch as its 32-bit chunk numbers hold (one launch but
    // for operands of 32 GB)
    const int64_t most = 0xF0000000ll / chunks;
    int64_t done[3] = {0, 0, 0};
    for (;;) {
        Rows r = {};
        int64_t rows = 0;
        for (int i = 0; i < 3; ++i) {
            r.first[i] = static_cast<uint32_t>(rows * chunks);
            if (!f[i].s || !f[i].s->repack) continue;
            int64_t n = f[i].rows - done[i];
            if (n > most - rows) n = most - rows;
            r.src[i] = static_cast<const uint16_t*>(f[i].s->ptr) + done[i] * cols;
            r.dst[i] = f[i].s->copy + done[i] * ld;
            done[i] += n;
            rows += n;
        }
        if (rows == 0) break;
        r.first[3] = static_cast<uint32_t>(rows * chunks);
        if (launch_pdl(align_rows_kernel, dim3(static_cast<unsigned>(cdiv(rows * chunks, 256))), dim3(256), 0, stream, r,
                       static_cast<uint32_t>(chunks), cols, ld) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_LAUNCH;
        }
    }
    for (const Fill& x : f)
        if (x.s && x.s->repack) x.s->ptr = x.s->copy;
    return GEMM_OK;
}

namespace {

// The partial sums of one split product.
struct Join {
    const float* partial;
    int64_t stride;                 // from one split's to the next
    int splits;
    int N;
    int64_t rows;                   // of all problems
    int64_t rows_per_problem;
    int64_t ld;
    const float* acc_in;            // (may be acc_out)
    float* acc_out;
    uint16_t* out16[2];
    const float* scale;
};

// Joins the partial sums of one or two split products, in split order:
// sum = acc_in + p[0] + p[1] + ..., to fp32 (acc_out) or scaled to 16 bits.
// Memory bound: reads splits * 4 bytes per output.  One thread sums four
// columns; a block takes one row's next 512.
__global__ void __launch_bounds__(128)
join_splits_kernel(const __grid_constant__ Join first, const __grid_constant__ Join second, int bf16) {
    grid_dependency_wait();
    allow_dependent_launch();
    const bool other = blockIdx.x >= first.rows;
    const Join& j = other ? second : first;
    const int64_t row = other ? blockIdx.x - first.rows : blockIdx.x;
    const float f = j.scale ? *j.scale : 1.0f;
    const int problem = row >= j.rows_per_problem ? 1 : 0;
    uint16_t* out = j.out16[problem] + (row - problem * j.rows_per_problem) * j.N;
    for (int64_t c = 4ll * (blockIdx.y * blockDim.x + threadIdx.x); c < j.ld; c += 4ll * gridDim.y * blockDim.x) {
        const int64_t at = row * j.ld + c;
        float4 v = j.acc_in ? *reinterpret_cast<const float4*>(j.acc_in + at) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int s = 0; s < j.splits; ++s) {
            const float4 w = *reinterpret_cast<const float4*>(j.partial + s * j.stride + at);
            v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w;
        }
        if (j.acc_out) {
            *reinterpret_cast<float4*>(j.acc_out + at) = v;
            continue;
        }
        uint16_t* dst = out + c;
        const uint32_t lo = pack16(f * v.x, f * v.y, bf16), hi = pack16(f * v.z, f * v.w, bf16);
        if (c + 4 <= j.N && (reinterpret_cast<uintptr_t>(dst) & 7u) == 0) {
            *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
        } else {
            dst[0] = static_cast<uint16_t>(lo & 0xFFFFu);
            if (c + 1 < j.N) dst[1] = static_cast<uint16_t>(lo >> 16);
            if (c + 2 < j.N) dst[2] = static_cast<uint16_t>(hi & 0xFFFFu);
            if (c + 3 < j.N) dst[3] = static_cast<uint16_t>(hi >> 16);
        }
    }
}

}  // namespace

int run_store_products(const StoreProduct* sp, int n, const Layout& l, int type, const DeviceInfo& info,
                       cudaStream_t stream) {
    Maps maps;
    memset(&maps, 0, sizeof(maps));
    Params p = base_params(l, type, info, stream);
    Join join[2] = {};
    int joins = 0;
    for (int at = 0; at < n; ++at) {
        const int which = n == 2 ? (at ? 1 - l.first : l.first) : 0;
        const StoreProduct& s = sp[which];
        const Layout::Part& part = l.part[which];
        if (!set_job(&p, &maps, at, s.pr, l, part, s.op)) return GEMM_ERR_LAUNCH;
        Job& j = p.job[at];
        j.ld32 = ld32_of(s.pr.N);
        if (part.splits > 1 || s.pr.halves > 1) {
            j.out32 = s.partial;
            j.problem_stride = s.pr.M * j.ld32;
            j.split_stride = j.problem_stride * s.pr.problems;
            // (halves: the partial sums of a split's two halves lie one after the other)
            Join& q = join[joins++];
            q.partial = s.partial;
            q.stride = j.split_stride / s.pr.halves;
            q.splits = part.splits * s.pr.halves;
            q.N = j.N;
            q.rows_per_problem = s.pr.M / s.pr.halves;
            q.rows = q.rows_per_problem * s.pr.problems;
            q.ld = j.ld32;
            q.acc_in = s.acc_in;
            q.acc_out = s.acc_out;
            for (int i = 0; i < 2; ++i) q.out16[i] = static_cast<uint16_t*>(s.out16[i]);
            q.scale = s.scale;
            continue;
        }
        j.out32 = s.acc_out;
        j.acc_in = s.acc_in;
        j.scale = s.scale;
        j.ld16 = s.pr.N;
        j.tma_store = s.out16[0] != nullptr;
        for (int i = 0; i < s.pr.problems; ++i) {
            j.out16[i] = static_cast<uint16_t*>(s.out16[i]);
            if (j.tma_store && !output_map(&maps.c[j.c_map + i], l, s.out16[i], s.pr.M, s.pr.N, s.pr.N)) j.tma_store = 0;
        }
    }
    const int rc = launch_product<kEpiStore>(l, maps, p, info, stream);
    if (rc != GEMM_OK || joins == 0) return rc;
    const int64_t ld = join[1].ld > join[0].ld ? join[1].ld : join[0].ld;
    int64_t across = cdiv(ld, 4 * 128);
    if (across > 65535) across = 65535;
    if (launch_pdl(join_splits_kernel, dim3(static_cast<unsigned>(join[0].rows + join[1].rows),
                                            static_cast<unsigned>(across)),
                   dim3(128), 0, stream, join[0], join[1], p.bf16) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

namespace {

struct BwdPlan {
    StoreProduct sp[2];             // dx and dW, those that are wanted
    int n = 0;
    Layout l;
    Source dy, x, w;
    size_t bytes = 0;
};

BwdPlan plan_bwd(int64_t M, int64_t N, int64_t K, const void* dy, const void* x, const void* w, bool want_dx,
                 bool want_dw, int num_sms, void* ws) {
    BwdPlan pl;
    Carver c;
    c.base = static_cast<char*>(ws);
    Product pr[2];
    if (want_dx) {
        Product& d = pr[pl.n++];
        d.M = M; d.N = K; d.K = N;
        d.bmn = true;
        d.may_split = true;
    }
    if (want_dw) {
        Product& d = pr[pl.n++];
        d.M = N; d.N = K; d.K = M;
        d.amn = d.bmn = true;
        d.may_split = true;
    }
    pl.dy = source_of(dy, M, N, !tma_ok(dy, N), &c);
    pl.x = source_of(x, M, K, want_dw && !tma_ok(x, K), &c);
    pl.w = source_of(w, N, K, want_dx && !tma_ok(w, K), &c);
    pl.l = choose_layout(pr, pl.n, num_sms);
    for (int i = 0; i < pl.n; ++i) {
        pl.sp[i].pr = pr[i];
        pl.sp[i].partial = c.take<float>(split_floats(pr[i], pl.l.part[i]));
    }
    pl.bytes = c.used;
    return pl;
}

int check_bwd(int64_t M, int64_t N, int64_t K, const void* dy, const void* x, const void* w, const void* dx,
              const void* dw, int type) {
    if (bad_size(M) || bad_size(N) || bad_size(K)) return GEMM_ERR_INVALID_ARG;
    if (type != GEMM_TYPE_HALF && type != GEMM_TYPE_BFLOAT) return GEMM_ERR_INVALID_ARG;
    if (too_many_tiles(M, K) || too_many_tiles(N, K)) return GEMM_ERR_INVALID_ARG;
    if (odd_address(dy) || odd_address(x) || odd_address(w) || odd_address(dx) || odd_address(dw))
        return GEMM_ERR_ALIGNMENT;
    if (K > 0 && M > 0 && N > 0 && (!dy || (dw && !x) || (dx && !w))) return GEMM_ERR_INVALID_ARG;
    const Range in[3] = {{dy, bytes16(M, N)}, {x, bytes16(M, K)}, {w, bytes16(N, K)}};
    const Range out[2] = {{dx, bytes16(M, K)}, {dw, bytes16(N, K)}};
    return overlaps(in, out) ? GEMM_ERR_INVALID_ARG : GEMM_OK;
}

}  // namespace
}  // namespace fused
}  // namespace pws

extern "C" int gemm_nt_bwd_workspace(int64_t M, int64_t N, int64_t K, const void* dy, const void* x, const void* w,
                                     int type, int64_t* bytes) {
    using namespace pws::fused;
    const int rc = check_bwd(M, N, K, dy, x, w, nullptr, nullptr, type);
    if (rc != GEMM_OK) return rc;
    if (!bytes) return GEMM_ERR_INVALID_ARG;
    *bytes = 0;
    if (M && N && K) {
        // one gradient alone may be split further than the two together
        const int sms = pws::sm_count_or_default();
        for (int want = 1; want <= 3; ++want) {
            const int64_t b =
                static_cast<int64_t>(plan_bwd(M, N, K, dy, x, w, want & 1, want & 2, sms, nullptr).bytes);
            if (b > *bytes) *bytes = b;
        }
    }
    return GEMM_OK;
}

extern "C" int gemm_nt_bwd(int64_t M, int64_t N, int64_t K, const void* dy, const void* x, const void* w, void* dx,
                           void* dw, int type, void* workspace, int64_t workspace_bytes, cudaStream_t stream) {
    using namespace pws;
    using namespace pws::fused;
    int rc = check_bwd(M, N, K, dy, x, w, dx, dw, type);
    if (rc != GEMM_OK) return rc;
    if (K == 0 || (M == 0 && N == 0) || (!dx && !dw)) return GEMM_OK;
    DeviceInfo info;
    rc = current_device(&info);
    if (rc != GEMM_OK) return rc;
    if (M == 0 || N == 0) {
        // an empty sum: dx [M, K] = 0 where N == 0, dw [N, K] = 0 where M == 0
        if (M && dx && cudaMemsetAsync(dx, 0, bytes16(M, K), stream) != cudaSuccess) return GEMM_ERR_LAUNCH;
        if (N && dw && cudaMemsetAsync(dw, 0, bytes16(N, K), stream) != cudaSuccess) return GEMM_ERR_LAUNCH;
        return GEMM_OK;
    }
    BwdPlan pl = plan_bwd(M, N, K, dy, x, w, dx != nullptr, dw != nullptr, info.num_sms, workspace);
    const Range in[3] = {{dy, bytes16(M, N)}, {x, bytes16(M, K)}, {w, bytes16(N, K)}};
    const Range out[2] = {{dx, bytes16(M, K)}, {dw, bytes16(N, K)}};
    if (!workspace_ok(workspace, workspace_bytes, pl.bytes, in, out)) return GEMM_ERR_INVALID_ARG;
    if ((rc = fill_sources({{&pl.dy, M}, {}, {}}, N, stream)) != GEMM_OK) return rc;
    if ((rc = fill_sources({{&pl.x, M}, {&pl.w, N}, {}}, K, stream)) != GEMM_OK) return rc;
    for (int i = 0; i < pl.n; ++i) {
        StoreProduct& s = pl.sp[i];
        const Source& b = s.pr.amn ? pl.x : pl.w;
        s.op.a[0] = pl.dy.ptr;
        s.op.lda = pl.dy.ld;
        s.op.b[0] = b.ptr;
        s.op.ldb = b.ld;
        s.out16[0] = s.pr.amn ? dw : dx;
    }
    return run_store_products(pl.sp, pl.n, pl.l, type, info, stream);
}

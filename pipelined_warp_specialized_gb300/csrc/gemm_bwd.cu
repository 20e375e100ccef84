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
// writes one 16-byte chunk: it reads the one or two aligned 16-byte blocks
// that hold it (each holds at least a byte of the row, so no load leaves the
// operand's pages) and shifts; a row's last, ragged chunk is read element by
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
        const uintptr_t at = reinterpret_cast<uintptr_t>(src);
        const uint32_t sh = static_cast<uint32_t>(at & 15u);
        const uint4* blk = reinterpret_cast<const uint4*>(at - sh);
        o = __ldg(blk);
        if (sh) {
            const uint4 hi = __ldg(blk + 1);
            const uint32_t w[8] = {o.x, o.y, o.z, o.w, hi.x, hi.y, hi.z, hi.w};
            const uint32_t q = sh >> 2, bits = (sh & 3u) * 8u;
            uint32_t v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t lo = q == 0 ? w[i] : q == 1 ? w[i + 1] : q == 2 ? w[i + 2] : w[i + 3];
                const uint32_t up = q == 0 ? w[i + 1] : q == 1 ? w[i + 2] : q == 2 ? w[i + 3] : w[i + 4];
                v[i] = __funnelshift_r(lo, up, bits);
            }
            o = make_uint4(v[0], v[1], v[2], v[3]);
        }
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

// Joins the partial sums of a split product, in split order:
// sum = acc_in + p[0] + p[1] + ..., to fp32 (acc_out) or scaled to 16 bits.
// Reads splits * 4 bytes per output; one thread sums four columns, a block
// takes one row's next 512.  acc_in and acc_out may be the same buffer.
__global__ void __launch_bounds__(128)
join_splits_kernel(const float* __restrict__ partial, int splits, int64_t split_stride, int64_t rows_per_problem,
                   int N, int64_t ld, const float* acc_in, float* acc_out,
                   uint16_t* __restrict__ out0, uint16_t* __restrict__ out1, const float* __restrict__ scale, int bf16) {
    grid_dependency_wait();
    allow_dependent_launch();
    const float f = scale ? *scale : 1.0f;
    const int64_t row = blockIdx.x;
    for (int64_t c = 4ll * (blockIdx.y * blockDim.x + threadIdx.x); c < ld; c += 4ll * gridDim.y * blockDim.x) {
        const int64_t at = row * ld + c;
        float4 v = acc_in ? *reinterpret_cast<const float4*>(acc_in + at) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int s = 0; s < splits; ++s) {
            const float4 w = *reinterpret_cast<const float4*>(partial + s * split_stride + at);
            v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w;
        }
        if (acc_out) {
            *reinterpret_cast<float4*>(acc_out + at) = v;
            continue;
        }
        const bool second = row >= rows_per_problem;
        uint16_t* dst = (second ? out1 + (row - rows_per_problem) * N : out0 + row * N) + c;
        const uint32_t lo = pack16(f * v.x, f * v.y, bf16), hi = pack16(f * v.z, f * v.w, bf16);
        if (c + 4 <= N && (reinterpret_cast<uintptr_t>(dst) & 7u) == 0) {
            *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
        } else {
            dst[0] = static_cast<uint16_t>(lo & 0xFFFFu);
            if (c + 1 < N) dst[1] = static_cast<uint16_t>(lo >> 16);
            if (c + 2 < N) dst[2] = static_cast<uint16_t>(hi & 0xFFFFu);
            if (c + 3 < N) dst[3] = static_cast<uint16_t>(hi >> 16);
        }
    }
}

}  // namespace

int run_store_product(const Product& pr, const Layout& l, const void* const a[4], int64_t lda, const void* const b[2],
                      int64_t ldb, const StoreTarget& to, float* partial, int type, const DeviceInfo& info,
                      cudaStream_t stream) {
    Maps maps;
    if (!encode_operands(&maps, pr, l, a, lda, b, ldb)) return GEMM_ERR_LAUNCH;
    Params p = base_params(pr, l, type, info, stream);
    p.ld32 = ld32_of(pr.N);
    const bool split = l.splits > 1 || pr.halves > 1;
    if (split) {
        p.out32 = partial;
        p.problem_stride = pr.M * p.ld32;
        p.split_stride = p.problem_stride * pr.problems;
    } else {
        p.out32 = to.acc_out;
        p.acc_in = to.acc_in;
        p.scale = to.scale;
        p.ld16 = pr.N;
        p.tma_store = to.out16[0] != nullptr;
        for (int i = 0; i < pr.problems; ++i) {
            p.out16[i] = static_cast<uint16_t*>(to.out16[i]);
            if (p.tma_store && !output_map(&maps.c[i], l, to.out16[i], pr.M, pr.N, pr.N)) p.tma_store = 0;
        }
    }
    int rc;
    if (pr.amn && pr.bmn) rc = launch_product<kEpiStore, true, true>(l, maps, p, info, stream);
    else if (!pr.amn && pr.bmn) rc = launch_product<kEpiStore, false, true>(l, maps, p, info, stream);
    else return GEMM_ERR_INVALID_ARG;
    if (rc != GEMM_OK || !split) return rc;
    // (halves: the partial sums of the two halves of a split lie one after the other)
    const int64_t rows = pr.M / pr.halves * pr.problems;
    int64_t across = cdiv(p.ld32, 4 * 128);
    if (across > 65535) across = 65535;
    if (launch_pdl(join_splits_kernel, dim3(static_cast<unsigned>(rows), static_cast<unsigned>(across)), dim3(128), 0, stream,
                   static_cast<const float*>(partial), l.splits * pr.halves, p.split_stride / pr.halves, pr.M,
                   static_cast<int>(pr.N), p.ld32, to.acc_in, to.acc_out, static_cast<uint16_t*>(to.out16[0]),
                   static_cast<uint16_t*>(to.out16[1]), to.scale, p.bf16) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

namespace {

struct BwdPlan {
    Product dx, dw;
    Layout ldx, ldw;
    Source dy, x, w;
    float* partial = nullptr;
    size_t bytes = 0;
};

BwdPlan plan_bwd(int64_t M, int64_t N, int64_t K, const void* dy, const void* x, const void* w, bool want_dx,
                 bool want_dw, int num_sms, void* ws) {
    BwdPlan pl;
    Carver c;
    c.base = static_cast<char*>(ws);
    pl.dx.M = M; pl.dx.N = K; pl.dx.K = N;
    pl.dx.bmn = true;
    pl.dx.may_split = true;
    pl.dw.M = N; pl.dw.N = K; pl.dw.K = M;
    pl.dw.amn = pl.dw.bmn = true;
    pl.dw.may_split = true;
    pl.dy = source_of(dy, M, N, !tma_ok(dy, N), &c);
    pl.x = source_of(x, M, K, want_dw && !tma_ok(x, K), &c);
    pl.w = source_of(w, N, K, want_dx && !tma_ok(w, K), &c);
    pl.ldx = choose_layout(pl.dx, num_sms);
    pl.ldw = choose_layout(pl.dw, num_sms);
    const int64_t fx = want_dx ? split_floats(pl.dx, pl.ldx) : 0, fw = want_dw ? split_floats(pl.dw, pl.ldw) : 0;
    pl.partial = c.take<float>(fx > fw ? fx : fw);
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
    *bytes = M && N && K
                 ? static_cast<int64_t>(
                       plan_bwd(M, N, K, dy, x, w, true, true, pws::sm_count_or_default(), nullptr).bytes)
                 : 0;
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
    if (pl.bytes && (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 != 0 ||
                     workspace_bytes < static_cast<int64_t>(pl.bytes)))
        return GEMM_ERR_INVALID_ARG;
    if ((rc = fill_sources({{&pl.dy, M}, {}, {}}, N, stream)) != GEMM_OK) return rc;
    if ((rc = fill_sources({{&pl.x, M}, {&pl.w, N}, {}}, K, stream)) != GEMM_OK) return rc;
    if (dx) {
        const void* a[4] = {pl.dy.ptr};
        const void* b[2] = {pl.w.ptr, nullptr};
        StoreTarget to;
        to.out16[0] = dx;
        rc = run_store_product(pl.dx, pl.ldx, a, pl.dy.ld, b, pl.w.ld, to, pl.partial, type, info, stream);
        if (rc != GEMM_OK) return rc;
    }
    if (dw) {
        const void* a[4] = {pl.dy.ptr};
        const void* b[2] = {pl.x.ptr, nullptr};
        StoreTarget to;
        to.out16[0] = dw;
        rc = run_store_product(pl.dw, pl.ldw, a, pl.dy.ld, b, pl.x.ld, to, pl.partial, type, info, stream);
    }
    return rc;
}

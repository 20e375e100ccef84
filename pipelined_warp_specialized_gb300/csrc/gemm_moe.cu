// gemm_moe.cu -- a mixture-of-experts feed-forward layer for a few tokens.
//
//   z = x Wr^T;  a token's experts e_1..e_k are those of its top_k largest logits;
//   p_j = softmax(z)[e_j];  y = sum_j p_j Wd[e_j] (act(Wg[e_j] x) * (Wu[e_j] x))
//
// Three kernels in a row on the stream, each launched as a programmatic
// dependent of the one before: the router (moe_route_kernel), gate and up
// projections with the activation (moe_gate_kernel), down projections with the
// weighted sum (moe_down_kernel).  With few tokens the layer is bound by the
// bytes of the chosen experts' weights, each read once (few.cuh).
//
// Rounding.  Sums are fp32.  The router's logits decide between experts, so
// they are summed to twice fp32's precision: two experts whose logits differ by
// fp32's own error would else be taken in an order that no definition gives.
// h' = p act(g) u is held as two 16-bit values, its rounding and what that left
// (the tensor cores multiply 16-bit values): 16 bits alone would add an error as
// large as the output's own rounding.
#include "few.cuh"
#include "product_host.cuh"

namespace pws {
namespace moe {

using namespace few;

constexpr int kTokens = 64;             // tokens a pass: more are taken 64 at a time
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;
constexpr int kRouteCtas = 8;           // CTAs of a cluster that share a token's experts
constexpr int kRouteTokens = 4;         // tokens a cluster
constexpr int kWarps = 8;

// ---------------------------------------------------------------- router

// s + p exactly, as s and an error added to c.
__device__ __forceinline__ void two_sum(float& s, float& c, float p) {
    const float t = __fadd_rn(s, p), b = __fsub_rn(t, s);
    c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(p, b)));
    s = t;
}

// Doubles in an order of unsigned integers: larger values first, NaN before all,
// both zeros alike, never 0.
__device__ __forceinline__ unsigned long long key_of(double z) {
    if (z != z) return ~0ull;
    const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(z + 0.0));
    return b >> 63 ? ~b : b | (1ull << 63);
}
__device__ __forceinline__ double value_of(unsigned long long key) {
    if (key == ~0ull) return __longlong_as_double(0x7ff8000000000000ll);
    return __longlong_as_double(static_cast<long long>(key >> 63 ? key & ~(1ull << 63) : ~key));
}

// The logits of up to kRouteTokens tokens by a cluster of kRouteCtas CTAs, a warp
// an expert; the first CTA then chooses.  A product of two 16-bit values is exact
// in fp32, and the sum is carried with its error, so logits are good to about
// 2^-45 of sum |x w| and only a true tie is one (it goes to the lower index).
// 7 additions and multiplications a product: 64 tokens x 128 experts x 4096 take
// about 9 us of the GPU, where their experts' weights take hundreds.
template <bool BF16, bool ALIGNED>
__global__ void __cluster_dims__(kRouteCtas, 1, 1) __launch_bounds__(256)
moe_route_kernel(const uint8_t* __restrict__ x, const uint8_t* __restrict__ w, int M, int64_t K, int E, int top_k,
                 int normalize, int* __restrict__ experts, float* __restrict__ weights, int per_cluster) {
    extern __shared__ unsigned long long keys[];        // [per_cluster][E], the first CTA's
    grid_dependency_wait();
    allow_dependent_launch();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_ctarank();
    const int token0 = static_cast<int>(blockIdx.x / kRouteCtas) * per_cluster;
    const int count = min(per_cluster, M - token0);
    const uint32_t keys0 = mapa_shared(smem_u32(keys), 0);
    for (int e = static_cast<int>(rank) * kWarps + warp; e < E; e += kRouteCtas * kWarps) {
        float s[kRouteTokens][2], c[kRouteTokens][2];
#pragma unroll
        for (int t = 0; t < kRouteTokens; ++t) s[t][0] = s[t][1] = c[t][0] = c[t][1] = 0.0f;
        const uint8_t* wr = w + static_cast<int64_t>(e) * K * 2;
        for (int64_t k = lane * 8; k < K; k += 256) {
            const uint4 wv = load_row<ALIGNED, false>(wr + 2 * k, 2 * (K - k));
            const uint32_t wp[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
            for (int t = 0; t < kRouteTokens; ++t) {
                if (t >= count) break;
                const uint4 xv = load_row<ALIGNED, false>(x + (static_cast<int64_t>(token0 + t) * K + k) * 2, 2 * (K - k));
                const uint32_t xp[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 a = fused::unpack16(wp[i], BF16), b = fused::unpack16(xp[i], BF16);
                    two_sum(s[t][0], c[t][0], __fmul_rn(a.x, b.x));
                    two_sum(s[t][1], c[t][1], __fmul_rn(a.y, b.y));
                }
            }
        }
#pragma unroll
        for (int t = 0; t < kRouteTokens; ++t) {
            if (t >= count) break;
            const float top = __fadd_rn(s[t][0], s[t][1]);
            // (an infinite sum's error terms are NaN)
            double z = fabsf(top) <= 3.4e38f
                           ? (static_cast<double>(s[t][0]) + c[t][0]) + (static_cast<double>(s[t][1]) + c[t][1])
                           : static_cast<double>(top);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
            if (lane == 0) {
                const unsigned long long key = key_of(z);
                asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(keys0 + 8u * static_cast<uint32_t>(t * E + e)), "l"(key)
                             : "memory");
            }
        }
    }
    cluster_sync();
    if (rank != 0) return;
    for (int t = warp; t < count; t += kWarps) {
        unsigned long long* row = keys + t * E;
        double z_top = 0.0;
        float mine = 0.0f, total = 0.0f;        // lane j's chosen expert's exponential
        int my_expert = 0;
        for (int j = 0; j < top_k; ++j) {
            unsigned long long best = 0;
            int at = 0;
            for (int e = lane; e < E; e += 32)
                if (row[e] > best) { best = row[e]; at = e; }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const unsigned long long other = __shfl_xor_sync(0xffffffffu, best, o);
                const int where = __shfl_xor_sync(0xffffffffu, at, o);
                if (other > best || (other == best && where < at)) { best = other; at = where; }
            }
            if (j == 0) z_top = value_of(best);
            if (lane == j) {
                my_expert = at;
                mine = expf(static_cast<float>(value_of(best) - z_top));
            }
            __syncwarp();
            if (lane == 0) row[at] = 0ull;
            __syncwarp();
        }
        if (lane < top_k) total = mine;
        if (!normalize)
            for (int e = lane; e < E; e += 32)
                if (row[e]) total += expf(static_cast<float>(value_of(row[e]) - z_top));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        if (lane < top_k) {
            const int64_t to = static_cast<int64_t>(token0 + t) * top_k + lane;
            experts[to] = my_expert;
            weights[to] = mine / total;
        }
    }
}

// ---------------------------------------------------------------- experts

struct Params {
    const uint8_t* x;                   // [M, K]
    const uint8_t* w_gate;              // [E, F, K]
    const uint8_t* w_up;
    const uint8_t* w_down;              // [E, K, F]
    const float* s_gate;                // [E, F], [E, F], [E, K]: 8-bit weights' scales
    const float* s_up;
    const float* s_down;
    const int* experts;                 // [M, top_k]
    const float* weights;
    uint16_t* h;                        // [2][M top_k][ldh]: h' rounded, and what that left
    uint16_t* y;                        // [M, K]
    int64_t K, F, ldh, lo_offset;
    int M, E, top_k, act;
};

// The distinct experts of M * top_k choices, as a bit mask (a warp's lane holds a
// word of it).  Every thread of the block.
__device__ __forceinline__ void mark_experts(uint32_t* mask, const int* experts, int choices) {
    if (threadIdx.x < 32) mask[threadIdx.x] = 0u;
    __syncthreads();
    for (int i = threadIdx.x; i < choices; i += blockDim.x) {
        const int e = experts[i];
        atomicOr(&mask[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
}

// The n-th marked expert, and how many there are; a whole warp.
__device__ __forceinline__ int nth_expert(const uint32_t* mask, int n, int& total) {
    const int lane = threadIdx.x % 32;
    const uint32_t word = mask[lane];
    int before = __popc(word);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
    }
    total = __shfl_sync(0xffffffffu, before, 31);
    before -= __popc(word);
    int at = -1;
    if (n >= before && n < before + __popc(word)) {
        uint32_t rest = word;
        for (int i = before; i < n; ++i) rest &= rest - 1;
        at = lane * 32 + __ffs(static_cast<int>(rest)) - 1;
    }
    const uint32_t has = __ballot_sync(0xffffffffu, at >= 0);
    return has ? __shfl_sync(0xffffffffu, at, __ffs(static_cast<int>(has)) - 1) : -1;
}

// h' = p act(Wg x) (Wu x) of one expert's tokens, 16 rows of F a block: eight
// warps take the steps of K in turn and their sums are joined in warp order.
// Block (b, a): rows 16 b .., the a-th distinct expert.
template <int FORM, bool ALIGNED, int NT>
__global__ void __launch_bounds__(kWarps * 32)
moe_gate_kernel(const __grid_constant__ Params p) {
    constexpr int STEP = step_k(FORM), WB = weight_bytes(FORM), NP = pairs_of(FORM);
    constexpr int UNROLL = NT <= 2 ? 4 : 2;
    __shared__ uint32_t mask[32];
    __shared__ int list[kTokens];
    __shared__ int shared_expert, shared_count;
    __shared__ float part[kWarps][2][16][8];
    grid_dependency_wait();
    allow_dependent_launch();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int choices = p.M * p.top_k;
    mark_experts(mask, p.experts, choices);
    if (warp == 0) {
        int total;
        const int e = nth_expert(mask, static_cast<int>(blockIdx.y), total);
        int n = 0;
        if (e >= 0)
            for (int i0 = 0; i0 < choices; i0 += 32) {
                const bool match = i0 + lane < choices && p.experts[i0 + lane] == e;
                const uint32_t b = __ballot_sync(0xffffffffu, match);
                if (match) list[n + __popc(b & ((1u << lane) - 1u))] = i0 + lane;
                n += __popc(b);
            }
        if (lane == 0) {
            shared_expert = e;
            shared_count = n;
        }
    }
    __syncthreads();
    const int expert = shared_expert, count = shared_count;
    if (expert < 0) return;
    const int row0 = static_cast<int>(blockIdx.x) * 16;
    const int tiles = (count + 7) / 8;
    float acc[NT][2][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][0][j] = acc[i][1][j] = 0.0f;

    const int64_t F = p.F, K = p.K;
    if (row0 < F) {
        // (a row past F reads the last one; its results are dropped)
        const int64_t r0 = min(static_cast<int64_t>(row0 + g), F - 1), r1 = min(static_cast<int64_t>(row0 + g + 8), F - 1);
        const int64_t first = static_cast<int64_t>(expert) * F;
        const uint8_t* wp[4] = {p.w_gate + (first + r0) * K * WB, p.w_gate + (first + r1) * K * WB,
                                p.w_up + (first + r0) * K * WB, p.w_up + (first + r1) * K * WB};
        const uint8_t* xp[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int at = 8 * i + g;
            xp[i] = at < count ? p.x + static_cast<int64_t>(list[at] / p.top_k) * K * 2 : nullptr;
        }
        constexpr int LANE = 16 / WB;                   // k of a lane's 16 bytes
        for (int64_t k0 = static_cast<int64_t>(warp) * STEP; k0 < K; k0 += static_cast<int64_t>(kWarps) * STEP * UNROLL) {
            uint4 w[UNROLL][4];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int64_t k = k0 + static_cast<int64_t>(u) * kWarps * STEP + t * LANE;
#pragma unroll
                for (int i = 0; i < 4; ++i) w[u][i] = load_row<ALIGNED, true>(wp[i] + k * WB, (K - k) * WB);
            }
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int64_t k = k0 + static_cast<int64_t>(u) * kWarps * STEP + t * LANE;
                uint32_t v[4][NP];
#pragma unroll
                for (int i = 0; i < 4; ++i) widen<FORM>(w[u][i], v[i]);
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    if (i >= tiles) break;
                    uint32_t xv[NP];
#pragma unroll
                    for (int j = 0; j < NP; j += 4) {
                        const int64_t kj = k + 2 * j;
                        const uint4 a = xp[i] ? load_row<ALIGNED, false>(xp[i] + 2 * kj, 2 * (K - kj)) : make_uint4(0u, 0u, 0u, 0u);
                        xv[j] = a.x; xv[j + 1] = a.y; xv[j + 2] = a.z; xv[j + 3] = a.w;
                    }
                    mma_step<FORM>(acc[i][0], v[0], v[1], xv);
                    mma_step<FORM>(acc[i][1], v[2], v[3], xv);
                }
            }
        }
    }
    // join the warps' sums tile by tile; thread (row, token) finishes h'
    const int r = threadIdx.x / 8 % 16, n = threadIdx.x % 8;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        if (i >= tiles) break;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            *reinterpret_cast<float2*>(&part[warp][m][g][2 * t]) = make_float2(acc[i][m][0], acc[i][m][1]);
            *reinterpret_cast<float2*>(&part[warp][m][g + 8][2 * t]) = make_float2(acc[i][m][2], acc[i][m][3]);
        }
        __syncthreads();
        if (threadIdx.x < 128 && 8 * i + n < count) {
            float gate = 0.0f, up = 0.0f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                gate += part[k][0][r][n];
                up += part[k][1][r][n];
            }
            const int choice = list[8 * i + n], row = row0 + r;
            float h = 0.0f;
            if (row < F) {
                if constexpr (is_i8(FORM)) {
                    gate *= p.s_gate[static_cast<int64_t>(expert) * F + row];
                    up *= p.s_up[static_cast<int64_t>(expert) * F + row];
                }
                h = p.weights[choice] * (fused::act_value(gate, p.act) * up);
            }
            // (columns from F to the padded row's end are zeros)
            const uint32_t hi = fused::pack16(h, 0.0f, is_bf16(FORM));
            const float kept = fused::unpack16(hi, is_bf16(FORM)).x;
            uint16_t* out = p.h + static_cast<int64_t>(choice) * p.ldh + row;
            out[0] = static_cast<uint16_t>(hi);
            out[p.lo_offset] = static_cast<uint16_t>(fused::pack16(fused::remainder16(h, kept), 0.0f, is_bf16(FORM)));
        }
        __syncthreads();
    }
}

// y = sum over the experts of Wd h', 16 rows of K a block.  The steps of all
// experts are one long axis, cut into a contiguous part for each warp; tokens
// keep their own accumulator columns, so one sum runs over all of a warp's experts.
template <int FORM, bool ALIGNED, int NT>
__global__ void __launch_bounds__(kWarps * 32)
moe_down_kernel(const __grid_constant__ Params p) {
    constexpr int STEP = step_k(FORM), WB = weight_bytes(FORM), NP = pairs_of(FORM);
    constexpr int UNROLL = NT <= 2 ? 4 : 2;
    __shared__ uint32_t mask[32];
    extern __shared__ int choice_experts[];             // [M top_k], then the warps' sums
    __shared__ float part[kWarps][16][8];
    grid_dependency_wait();
    allow_dependent_launch();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int choices = p.M * p.top_k;
    for (int i = threadIdx.x; i < choices; i += blockDim.x) choice_experts[i] = p.experts[i];
    mark_experts(mask, p.experts, choices);
    const int row0 = static_cast<int>(blockIdx.x) * 16;
    const int64_t F = p.F, K = p.K;
    float acc[NT][4], sum[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = sum[i][j] = 0.0f;
    int total;
    nth_expert(mask, 0, total);
    const int steps = static_cast<int>((F + STEP - 1) / STEP);
    const int64_t all = static_cast<int64_t>(total) * steps;
    int64_t s = all * warp / kWarps;
    const int64_t end = all * (warp + 1) / kWarps;
    const int64_t r0 = min(static_cast<int64_t>(row0 + g), K - 1), r1 = min(static_cast<int64_t>(row0 + g + 8), K - 1);
    constexpr int LANE = 16 / WB;
    while (s < end) {
        const int a = static_cast<int>(s / steps);
        int dummy;
        const int expert = nth_expert(mask, a, dummy);
        const int from = static_cast<int>(s - static_cast<int64_t>(a) * steps);
        const int to = static_cast<int>(min(static_cast<int64_t>(steps), end - static_cast<int64_t>(a) * steps));
        s += to - from;
        const uint8_t* wp[2] = {p.w_down + (static_cast<int64_t>(expert) * K + r0) * F * WB,
                                p.w_down + (static_cast<int64_t>(expert) * K + r1) * F * WB};
        // each tile's row of h' of this expert, where token g of the tile chose it
        const uint8_t* hp[NT];
        uint32_t live = 0;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int token = 8 * i + g;
            hp[i] = nullptr;
            if (token < p.M)
                for (int j = 0; j < p.top_k; ++j)
                    if (choice_experts[token * p.top_k + j] == expert)
                        hp[i] = reinterpret_cast<const uint8_t*>(p.h + static_cast<int64_t>(token * p.top_k + j) * p.ldh);
            if (__any_sync(0xffffffffu, hp[i] != nullptr)) live |= 1u << i;
        }
        for (int k0 = from; k0 < to; k0 += UNROLL) {
            uint4 w[UNROLL][2];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int64_t k = static_cast<int64_t>(k0 + u) * STEP + t * LANE;
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    w[u][i] = load_row<ALIGNED, true>(wp[i] + k * WB, k0 + u < to ? (F - k) * WB : 0);
            }
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                if (k0 + u >= to) break;
                const int64_t k = static_cast<int64_t>(k0 + u) * STEP + t * LANE;
                uint32_t v[2][NP];
                widen<FORM>(w[u][0], v[0]);
                widen<FORM>(w[u][1], v[1]);
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    if (!(live >> i & 1u)) continue;
                    uint32_t hi[NP], lo[NP];
#pragma unroll
                    for (int j = 0; j < NP; j += 4) {
                        uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
                        if (hp[i]) {
                            a = __ldcg(reinterpret_cast<const uint4*>(hp[i] + 2 * (k + 2 * j)));
                            b = __ldcg(reinterpret_cast<const uint4*>(hp[i] + 2 * (p.lo_offset + k + 2 * j)));
                        }
                        hi[j] = a.x; hi[j + 1] = a.y; hi[j + 2] = a.z; hi[j + 3] = a.w;
                        lo[j] = b.x; lo[j + 1] = b.y; lo[j + 2] = b.z; lo[j + 3] = b.w;
                    }
                    mma_step<FORM>(acc[i], v[0], v[1], hi);
                    mma_step<FORM>(acc[i], v[0], v[1], lo);
                }
            }
        }
        if constexpr (is_i8(FORM)) {
            const float s0 = p.s_down[static_cast<int64_t>(expert) * K + r0], s1 = p.s_down[static_cast<int64_t>(expert) * K + r1];
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                if (!(live >> i & 1u)) continue;
                // (a token that did not choose the expert adds nothing, whatever the scale is)
                const uint32_t mine = __ballot_sync(0xffffffffu, hp[i] != nullptr);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int column = 2 * t + (j & 1);
                    if (mine >> (4 * column) & 1u) sum[i][j] += (j < 2 ? s0 : s1) * acc[i][j];
                    acc[i][j] = 0.0f;
                }
            }
        }
    }
    const int r = threadIdx.x / 8 % 16, n = threadIdx.x % 8;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        if (8 * i >= p.M) break;
        const float(&v)[4] = is_i8(FORM) ? sum[i] : acc[i];
        *reinterpret_cast<float2*>(&part[warp][g][2 * t]) = make_float2(v[0], v[1]);
        *reinterpret_cast<float2*>(&part[warp][g + 8][2 * t]) = make_float2(v[2], v[3]);
        __syncthreads();
        if (threadIdx.x < 128 && 8 * i + n < p.M && row0 + r < K) {
            float total_y = 0.0f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) total_y += part[k][r][n];
            p.y[static_cast<int64_t>(8 * i + n) * K + row0 + r] =
                static_cast<uint16_t>(fused::pack16(total_y, 0.0f, is_bf16(FORM)));
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- host

using fused::bad_size;
using fused::cdiv;
using fused::odd_address;
using fused::Range;
using fused::round_up;

struct Call {
    int64_t M, K, F, E, top_k;
    const void *x, *w_router, *w_gate, *w_up, *w_down;
    const float *s_gate, *s_up, *s_down;
    void* y;
    int* experts;
    float* weights;
    int type, weight_type, act, normalize;
};

bool odd_word(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 != 0; }

// What a call refuses before it looks at the device.
int check(const Call& c) {
    if (bad_size(c.M) || bad_size(c.K) || bad_size(c.F)) return GEMM_ERR_INVALID_ARG;
    if (c.E < 1 || c.E > kMaxExperts || c.top_k < 1 || c.top_k > kMaxTopK || c.top_k > c.E) return GEMM_ERR_INVALID_ARG;
    if (c.type != GEMM_TYPE_HALF && c.type != GEMM_TYPE_BFLOAT) return GEMM_ERR_INVALID_ARG;
    if (c.weight_type != c.type && c.weight_type != GEMM_TYPE_BYTE) return GEMM_ERR_INVALID_ARG;
    if (c.act != GEMM_ACT_SILU && c.act != GEMM_ACT_GELU) return GEMM_ERR_INVALID_ARG;
    if (c.normalize != 0 && c.normalize != 1) return GEMM_ERR_INVALID_ARG;
    // (a row block of 16 to a block of the grid; bytes of all experts in 63 bits)
    if (c.F && c.K > ((1ll << 48) / c.F)) return GEMM_ERR_INVALID_ARG;
    const bool i8 = c.weight_type == GEMM_TYPE_BYTE;
    if (odd_address(c.x) || odd_address(c.w_router) || odd_address(c.y)) return GEMM_ERR_ALIGNMENT;
    if (!i8 && (odd_address(c.w_gate) || odd_address(c.w_up) || odd_address(c.w_down))) return GEMM_ERR_ALIGNMENT;
    if (odd_word(c.s_gate) || odd_word(c.s_up) || odd_word(c.s_down) || odd_word(c.experts) || odd_word(c.weights))
        return GEMM_ERR_ALIGNMENT;
    if (i8 != (c.s_gate != nullptr) || i8 != (c.s_up != nullptr) || i8 != (c.s_down != nullptr)) return GEMM_ERR_INVALID_ARG;
    if (c.M > 0) {
        if (c.K > 0 && (!c.x || !c.w_router || (c.F > 0 && (!c.w_gate || !c.w_up || !c.w_down)))) return GEMM_ERR_INVALID_ARG;
    }
    return GEMM_OK;
}

uint64_t weight_matrix_bytes(const Call& c) {
    return static_cast<uint64_t>(c.E) * c.F * c.K * (c.weight_type == GEMM_TYPE_BYTE ? 1u : 2u);
}

int64_t pass_tokens(int64_t M) { return M < kTokens ? M : kTokens; }
int64_t ldh_of(int64_t F) { return round_up(F, 64); }
int64_t workspace_bytes_of(const Call& c) {
    if (c.M == 0 || c.K == 0 || c.F == 0) return 0;
    return round_up(2 * pass_tokens(c.M) * c.top_k * ldh_of(c.F) * 2, 256);
}

bool rows16(const void* p, int64_t row_bytes) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && row_bytes % 16 == 0; }

int launched(cudaError_t e) {
    if (e == cudaSuccess) return GEMM_OK;
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
}

template <bool BF16, bool ALIGNED>
int launch_route(const Call& c, const uint8_t* x, int M, int* experts, float* weights, cudaStream_t stream) {
    // few tokens: a cluster each
    const int per = M <= 16 ? 1 : kRouteTokens;
    return launched(launch_pdl(moe_route_kernel<BF16, ALIGNED>, dim3(static_cast<unsigned>(cdiv(M, per) * kRouteCtas)), dim3(256),
                               static_cast<size_t>(per) * c.E * 8, stream, x, static_cast<const uint8_t*>(c.w_router), M, c.K,
                               static_cast<int>(c.E), static_cast<int>(c.top_k), c.normalize, experts, weights, per));
}

template <int FORM, bool ALIGNED, int NT>
int launch_experts(const Params& p, bool down, cudaStream_t stream) {
    const int choices = p.M * p.top_k;
    if (!down) {
        const dim3 grid(static_cast<unsigned>(cdiv(p.ldh, 16)), static_cast<unsigned>(choices < p.E ? choices : p.E));
        return launched(launch_pdl(moe_gate_kernel<FORM, ALIGNED, NT>, grid, dim3(kWarps * 32), 0, stream, p));
    }
    return launched(launch_pdl(moe_down_kernel<FORM, ALIGNED, NT>, dim3(static_cast<unsigned>(cdiv(p.K, 16))), dim3(kWarps * 32),
                               static_cast<size_t>(choices) * 4, stream, p));
}

template <int FORM, bool ALIGNED>
int launch_tiles(const Params& p, bool down, cudaStream_t stream) {
    if (p.M <= 8) return launch_experts<FORM, ALIGNED, 1>(p, down, stream);
    if (p.M <= 16) return launch_experts<FORM, ALIGNED, 2>(p, down, stream);
    return launch_experts<FORM, ALIGNED, 8>(p, down, stream);
}

template <int FORM>
int launch_form(const Params& p, bool down, bool aligned, cudaStream_t stream) {
    return aligned ? launch_tiles<FORM, true>(p, down, stream) : launch_tiles<FORM, false>(p, down, stream);
}

int launch_kernel(const Params& p, int form, bool down, bool aligned, cudaStream_t stream) {
    switch (form) {
        case kHalf: return launch_form<kHalf>(p, down, aligned, stream);
        case kBfloat: return launch_form<kBfloat>(p, down, aligned, stream);
        case kI8Half: return launch_form<kI8Half>(p, down, aligned, stream);
        default: return launch_form<kI8Bfloat>(p, down, aligned, stream);
    }
}

int run(const Call& c, void* workspace, int64_t workspace_bytes, cudaStream_t stream) {
    int rc = check(c);
    if (rc != GEMM_OK) return rc;
    if (c.M == 0) return GEMM_OK;
    if (!c.experts || !c.weights || (c.K > 0 && !c.y)) return GEMM_ERR_INVALID_ARG;
    const uint64_t wb = weight_matrix_bytes(c), xb = fused::bytes16(c.M, c.K), fb = 4ull * c.E * c.F;
    const uint64_t cb = 4ull * c.M * c.top_k;
    const Range in[8] = {{c.x, xb},      {c.w_router, fused::bytes16(c.E, c.K)}, {c.w_gate, wb}, {c.w_up, wb}, {c.w_down, wb},
                         {c.s_gate, fb}, {c.s_up, fb},                           {c.s_down, 4ull * c.E * c.K}};
    const Range out[3] = {{c.y, xb}, {c.experts, cb}, {c.weights, cb}};
    if (fused::overlaps(in, out)) return GEMM_ERR_INVALID_ARG;
    if (!fused::workspace_ok(workspace, workspace_bytes, workspace_bytes_of(c), in, out)) return GEMM_ERR_INVALID_ARG;
    DeviceInfo info;
    rc = current_device(&info);
    if (rc != GEMM_OK) return rc;

    const bool i8 = c.weight_type == GEMM_TYPE_BYTE, bf16 = c.type == GEMM_TYPE_BFLOAT;
    const int form = (i8 ? 2 : 0) + (bf16 ? 1 : 0), wbytes = i8 ? 1 : 2;
    const bool route_aligned = rows16(c.x, 2 * c.K) && rows16(c.w_router, 2 * c.K);
    const bool gate_aligned = rows16(c.x, 2 * c.K) && rows16(c.w_gate, wbytes * c.K) && rows16(c.w_up, wbytes * c.K);
    const bool down_aligned = rows16(c.w_down, wbytes * c.F);
    Params p = {};
    p.w_gate = static_cast<const uint8_t*>(c.w_gate);
    p.w_up = static_cast<const uint8_t*>(c.w_up);
    p.w_down = static_cast<const uint8_t*>(c.w_down);
    p.s_gate = c.s_gate;
    p.s_up = c.s_up;
    p.s_down = c.s_down;
    p.h = static_cast<uint16_t*>(workspace);
    p.K = c.K;
    p.F = c.F;
    p.ldh = ldh_of(c.F);
    p.E = static_cast<int>(c.E);
    p.top_k = static_cast<int>(c.top_k);
    p.act = c.act;
    for (int64_t m = 0; m < c.M; m += kTokens) {
        p.M = static_cast<int>(c.M - m < kTokens ? c.M - m : kTokens);
        p.lo_offset = static_cast<int64_t>(p.M) * c.top_k * p.ldh;
        p.x = static_cast<const uint8_t*>(c.x) + m * c.K * 2;
        p.y = static_cast<uint16_t*>(c.y) + m * c.K;
        p.experts = c.experts + m * c.top_k;
        p.weights = c.weights + m * c.top_k;
        int* experts = c.experts + m * c.top_k;
        float* weights = c.weights + m * c.top_k;
        if (bf16)
            rc = route_aligned ? launch_route<true, true>(c, p.x, p.M, experts, weights, stream)
                               : launch_route<true, false>(c, p.x, p.M, experts, weights, stream);
        else
            rc = route_aligned ? launch_route<false, true>(c, p.x, p.M, experts, weights, stream)
                               : launch_route<false, false>(c, p.x, p.M, experts, weights, stream);
        if (rc != GEMM_OK) return rc;
        if (c.K == 0) continue;
        if (c.F > 0 && (rc = launch_kernel(p, form, false, gate_aligned, stream)) != GEMM_OK) return rc;
        if ((rc = launch_kernel(p, form, true, down_aligned, stream)) != GEMM_OK) return rc;
    }
    return GEMM_OK;
}

}  // namespace moe
}  // namespace pws

extern "C" int gemm_moe_nt_workspace(int64_t M, int64_t K, int64_t F, int64_t E, int64_t top_k, int type, int weight_type,
                                     int64_t* bytes) {
    using namespace pws::moe;
    // (scales where the weights have them; pointers are not looked at otherwise)
    const float* s = weight_type == GEMM_TYPE_BYTE ? reinterpret_cast<const float*>(16) : nullptr;
    const void* any = reinterpret_cast<const void*>(16);
    const Call c = {M, K, F, E, top_k, any, any, any, any, any, s, s, s, nullptr, nullptr, nullptr, type, weight_type,
                    GEMM_ACT_SILU, 0};
    const int rc = check(c);
    if (rc != GEMM_OK) return rc;
    if (!bytes) return GEMM_ERR_INVALID_ARG;
    *bytes = workspace_bytes_of(c);
    return GEMM_OK;
}

extern "C" int gemm_moe_nt(int64_t M, int64_t K, int64_t F, int64_t E, int64_t top_k, const void* x, const void* w_router,
                           const void* w_gate, const void* w_up, const void* w_down, const float* s_gate, const float* s_up,
                           const float* s_down, void* y, int32_t* experts, float* weights, int type, int weight_type, int act,
                           int normalize, void* workspace, int64_t workspace_bytes, cudaStream_t stream) {
    using namespace pws::moe;
    const Call c = {M,      K,      F, E,       top_k,   x,    w_router,    w_gate, w_up,     w_down,
                    s_gate, s_up,   s_down, y,  experts, weights, type, weight_type, act,    normalize};
    return run(c, workspace, workspace_bytes, stream);
}

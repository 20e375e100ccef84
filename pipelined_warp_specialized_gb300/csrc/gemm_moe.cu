// gemm_moe.cu -- a mixture-of-experts feed-forward layer for a few tokens.
//
//   z = x Wr^T;  a token's experts e_1..e_k are those of its top_k largest logits;
//   p_j = softmax(z)[e_j];  y = sum_j p_j Wd[e_j] (act(Wg[e_j] x) * (Wu[e_j] x))
//
// Three kernels in a row on the stream, each launched as a programmatic
// dependent of the one before: the router (moe_route_kernel), gate and up
// projections with the activation, down projections with the weighted sum (both
// moe_experts_kernel).  With few tokens the layer is bound by the
// bytes of the chosen experts' weights (few.cuh), which is what one token or a few over
// many experts come near (a token's six of 64 experts of 2048 x 4096 take 76 us in
// all, their 302 MB alone 45; 16 tokens over 56 of 1536 x 4096 375 us, 2.1 GB alone 318).
//
// Rounding.  Sums are fp32.  The router's logits decide between experts, so
// they are summed to twice fp32's precision: two experts whose logits differ by
// fp32's own error would else be taken in an order that no definition gives.
// h = act(g) u is held in fp32.  The tensor cores multiply 16-bit values, so the down
// projections take it apart as they read it: for bfloat16 weights into three bfloat16
// values, which are all of its 24 bits; for binary16 and 8-bit weights (8-bit integers
// are binary16 values, whatever the tokens' type) into two binary16 values of
// h times a power of two that brings the token's largest |h| to 2^14 .. 2^15: 22 bits, and
// 2^-39 of that largest one, whatever the magnitudes.  The power and p are taken into
// account in fp32 when sums are joined.  Two 16-bit values of the tokens' type, written by gate and
// multiplied as they are, took 2 to 4 % less (one token's six experts 73.5 us, 76 so; 32 tokens in 8
// bits 189 and 196), but are infinite in binary16 from 65520 on, and 16 bits in bfloat16.
#include <type_traits>

#include "few.cuh"
#include "product_host.cuh"

namespace pws {
namespace moe {

using namespace few;

constexpr int kTokens = 64;             // tokens a pass: more are taken 64 at a time
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;
constexpr int64_t kMaxWidth = 1 << 22;  // of K and F
constexpr int kRouteCtas = 8;           // CTAs of a cluster that share a token's experts
constexpr int kRouteTokens = 4;         // tokens a cluster, where there are many
constexpr int route_threads(int tokens) { return tokens == 1 ? 1024 : 512; }
constexpr int kWarps = 8;

// ---------------------------------------------------------------- router

// s + p exactly, as s and an error added to c (Knuth's sum of two numbers and its error, The Art of Computer
// Programming, volume 2, 4.2.2).
__device__ __forceinline__ void two_sum(float& s, float& c, float p) {
    const float t = __fadd_rn(s, p), b = __fsub_rn(t, s);
    c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(p, b)));
    s = t;
}

// A sum and its error as one value and what it lacks: hi = fl(s + c), lo the rest.
// (FP64 has few units here: a row's last sums in doubles took as long as the row.)
__device__ __forceinline__ float2 settled(float s, float c) {
    const float hi = __fadd_rn(s, c);
    // (an infinite or NaN sum's error terms mean nothing)
    return fabsf(s) <= 3.4e38f ? make_float2(hi, __fadd_rn(__fsub_rn(s, hi), c)) : make_float2(s, 0.0f);
}

// Floats in the order of unsigned integers: larger values first, NaN before all,
// both zeros alike, never 0.
__device__ __forceinline__ uint32_t key32(float v) {
    if (v != v) return 0xFFFFFFFFu;
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value32(uint32_t key) {
    return key == 0xFFFFFFFFu ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float(key >> 31 ? key & 0x7FFFFFFFu : ~key);
}
__device__ __forceinline__ unsigned long long key_of(float2 z) {
    return static_cast<unsigned long long>(key32(z.x)) << 32 | key32(z.y);
}
__device__ __forceinline__ float2 value_of(unsigned long long key) {
    return make_float2(value32(static_cast<uint32_t>(key >> 32)), value32(static_cast<uint32_t>(key)));
}
__device__ __forceinline__ float exp_difference(float2 z, float2 top) { return expf((z.x - top.x) + (z.y - top.y)); }

// What the router hands to the experts' kernels besides the choice.
struct Handover {
    int* counters;
    uint16_t* x;
    int64_t num_counters, ldx;
};

// The logits of TOKENS tokens by a cluster of kRouteCtas CTAs, a warp a part of
// an expert's row; the first CTA then adds the parts and chooses.  A product of two
// 16-bit values is exact in fp32, and the sum is carried with its error, so logits are good to about
// 2^-44 of sum |x w| and only a true tie is one (it goes to the lower index).
// Seven additions and multiplications a product, latency for few tokens: every
// lane has eight or more loads in flight.
template <bool BF16, bool ALIGNED, int TOKENS>
__global__ void __cluster_dims__(kRouteCtas, 1, 1) __launch_bounds__(route_threads(TOKENS))
moe_route_kernel(const uint8_t* __restrict__ x, const uint8_t* __restrict__ w, int M, int64_t K, int E, int parts, int top_k,
                 int normalize, int* __restrict__ experts, float* __restrict__ weights, const __grid_constant__ Handover out) {
    constexpr int UNROLL = TOKENS == 1 ? 4 : 2, THREADS = route_threads(TOKENS);
    extern __shared__ unsigned long long sums[];        // [TOKENS][E][parts] pairs, then keys; the first CTA's
    grid_dependency_wait();
    allow_dependent_launch();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_ctarank();
    cluster_arrive_release();           // (no store to a CTA that has not begun)
    const int token0 = static_cast<int>(blockIdx.x / kRouteCtas) * TOKENS;
    const int count = min(TOKENS, M - token0);
    const uint32_t sums0 = mapa_shared(smem_u32(sums), 0);
    bool begun = false;
    const int64_t span = ((K + parts - 1) / parts + 255) / 256 * 256;
    for (int task = static_cast<int>(rank) * (THREADS / 32) + warp; task < E * parts; task += kRouteCtas * (THREADS / 32)) {
        const int e = task / parts, part = task - e * parts;
        float s[TOKENS][2], c[TOKENS][2];
#pragma unroll
        for (int t = 0; t < TOKENS; ++t) s[t][0] = s[t][1] = c[t][0] = c[t][1] = 0.0f;
        const uint8_t* wr = w + static_cast<int64_t>(e) * K * 2;
        const uint8_t* xr = x + static_cast<int64_t>(token0) * K * 2;
        const int64_t end = min(K, (part + 1) * span);
        for (int64_t k0 = part * span + lane * 8; k0 < end; k0 += 256 * UNROLL) {
            uint4 wv[UNROLL], xv[TOKENS][UNROLL];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int64_t k = k0 + 256 * u, left = k < end ? 2 * (K - k) : 0;
                wv[u] = load_row<ALIGNED, false>(wr + 2 * k, left);
#pragma unroll
                for (int t = 0; t < TOKENS; ++t)
                    xv[t][u] = load_row<ALIGNED, false>(xr + (t * K + k) * 2, t < count ? left : 0);
            }
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const uint32_t wp[4] = {wv[u].x, wv[u].y, wv[u].z, wv[u].w};
#pragma unroll
                for (int t = 0; t < TOKENS; ++t) {
                    const uint32_t xp[4] = {xv[t][u].x, xv[t][u].y, xv[t][u].z, xv[t][u].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 a = fused::unpack16(wp[i], BF16), b = fused::unpack16(xp[i], BF16);
                        two_sum(s[t][0], c[t][0], __fmul_rn(a.x, b.x));
                        two_sum(s[t][1], c[t][1], __fmul_rn(a.y, b.y));
                    }
                }
            }
        }
        if (!begun) cluster_wait_acquire();
        begun = true;
#pragma unroll
        for (int t = 0; t < TOKENS; ++t) {
            // (both pairs, then all lanes', with every error kept)
            float sum = s[t][0], err = __fadd_rn(c[t][0], c[t][1]);
            two_sum(sum, err, s[t][1]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const float other = __shfl_xor_sync(0xffffffffu, sum, o), more = __shfl_xor_sync(0xffffffffu, err, o);
                err = __fadd_rn(err, more);
                two_sum(sum, err, other);
            }
            if (lane == 0 && t < count)
                asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(sums0 + 8u * static_cast<uint32_t>((t * E + e) * parts + part)),
                             "f"(sum), "f"(err)
                             : "memory");
        }
    }
    if (!begun) cluster_wait_acquire();
    __syncthreads();            // (the cluster barrier wants whole warps, and the loops above part them)
    cluster_sync();
    if (rank != 0) {
        // what the experts' kernels start from: counters at zero, and the tokens in rows of a
        // multiple of 64, padded with zeros, whatever x's alignment is
        const int64_t others = kRouteCtas - 1, clusters = gridDim.x / kRouteCtas;
        const int64_t thread = (blockIdx.x / kRouteCtas * others + rank - 1) * THREADS + threadIdx.x, threads = clusters * others * THREADS;
        for (int64_t i = thread; i < out.num_counters; i += threads) out.counters[i] = 0;
        for (int64_t i = thread; i < M * (out.ldx / 8); i += threads) {
            const int64_t m = i / (out.ldx / 8), k = (i - m * (out.ldx / 8)) * 8;
            *reinterpret_cast<uint4*>(out.x + m * out.ldx + k) = load_row<ALIGNED, false>(x + (m * K + k) * 2, 2 * (K - k));
        }
        return;
    }
    if (warp >= count) return;
    // a warp a token: keys in place of the first parts
    unsigned long long* row = sums + warp * E * parts;
    const auto key_at = [&](int e) { return row + e * parts; };
    for (int e = lane; e < E; e += 32) {
        const float2* part = reinterpret_cast<const float2*>(row + e * parts);
        float sum = part[0].x, err = part[0].y;
        for (int i = 1; i < parts; ++i) {
            err = __fadd_rn(err, part[i].y);
            two_sum(sum, err, part[i].x);
        }
        *key_at(e) = key_of(settled(sum, err));
    }
    float2 z_top = make_float2(0.0f, 0.0f);
    float mine = 0.0f, total = 0.0f;            // lane j's chosen expert's exponential
    int my_expert = 0;
    // each lane's largest key; the one that is taken looks for its next
    unsigned long long best = 0;
    int at = 0;
    const auto look = [&]() {
        best = 0;
        for (int e = lane; e < E; e += 32)
            if (*key_at(e) > best) { best = *key_at(e); at = e; }
    };
    look();
    for (int j = 0; j < top_k; ++j) {
        // the largest: its high word, then its low word, then its lowest index
        const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(best >> 32));
        const uint32_t lo = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(best >> 32) == hi ? static_cast<uint32_t>(best) : 0u);
        const unsigned long long top = static_cast<unsigned long long>(hi) << 32 | lo;
        const int chosen = static_cast<int>(__reduce_min_sync(0xffffffffu, best == top ? static_cast<uint32_t>(at) : 0xffffffffu));
        if (j == 0) z_top = value_of(top);
        if (lane == j) {
            my_expert = chosen;
            mine = exp_difference(value_of(top), z_top);
        }
        if (chosen % 32 == lane) {
            *key_at(chosen) = 0ull;
            look();
        }
        __syncwarp();
    }
    if (lane < top_k) total = mine;
    if (!normalize)
        for (int e = lane; e < E; e += 32)
            if (*key_at(e)) total += exp_difference(value_of(*key_at(e)), z_top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane < top_k) {
        const int64_t to = static_cast<int64_t>(token0 + warp) * top_k + lane;
        experts[to] = my_expert;
        weights[to] = mine / total;
    }
}

// ---------------------------------------------------------------- experts

struct Params {
    const uint16_t* x;                  // [M][ldx], padded with zeros
    const uint8_t* w_gate;              // [E, F, K]
    const uint8_t* w_up;
    const uint8_t* w_down;              // [E, K, F]
    const float* s_gate;                // [E, F], [E, F], [E, K]: 8-bit weights' scales
    const float* s_up;
    const float* s_down;
    const int* experts;                 // [M, top_k]
    const float* weights;
    float* h;                           // [M top_k][ldh], each step's in the order of h_place
    uint16_t* y;                        // [M, K]
    int64_t K, F, ldx, ldh;
    int M, E, top_k, act, bf16;         // bf16: the type of y
    int groups;                         // 32 rows a unit takes: 1, 2, 4 or 8
    int* counters;                      // claims of gate and of down units, then each row block's arrivals; zero at first
    uint32_t* tops;                     // [M top_k], the bits of each choice's largest |h|; zero at first
    float* partial;                     // [M top_k][K]: each choice's part of y
};

// Shared memory of a block beside its rings and the routing's arrays.
constexpr int kBeside = 11264;

// What a block of the experts' kernels knows of the routing.  A kernel's entries
// hold up to 8 NT tokens of an expert (NT tiles): an expert with more is taken once for
// each 8 NT of them, its weights coming from L2 again, and the accumulators stay few.
struct alignas(16) Routing {
    uint16_t* experts;                          // each choice's
    uint16_t* active;                           // an entry's expert, in ascending order (no more entries than choices)
    int entries;
    uint8_t tokens[kMaxExperts];                // of each expert
    uint16_t list[kWarps][2][16];               // choices of the entry a warp copies, and of the one it multiplies
};
constexpr int routing_bytes(int choices) { return (4 * choices + 15) / 16 * 16; }

// Every thread of the block.
template <int SIZE>
__device__ __forceinline__ void read_routing(Routing& r, uint16_t* room, const int* experts, int choices, int num_experts) {
    const int lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        r.experts = room;
        r.active = room + choices;
    }
    for (int i = threadIdx.x; i < (num_experts + 3) / 4; i += blockDim.x) reinterpret_cast<uint32_t*>(r.tokens)[i] = 0u;
    __syncthreads();
    for (int i = threadIdx.x; i < choices; i += blockDim.x) {
        const int e = __ldcg(experts + i);
        room[i] = static_cast<uint16_t>(e);
        // (a byte holds an expert's tokens: each of 64 at most once)
        atomicAdd(reinterpret_cast<uint32_t*>(r.tokens) + e / 4, 1u << (8 * (e % 4)));
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        int before = 0;
        for (int e0 = 0; e0 < num_experts; e0 += 32) {
            const int e = e0 + lane, passes = e < num_experts ? (r.tokens[e] + SIZE - 1) / SIZE : 0;
            int at = passes;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, at, o);
                if (lane >= o) at += v;
            }
            const int total = __shfl_sync(0xffffffffu, at, 31);
            at += before - passes;
            for (int i = 0; i < passes; ++i) room[choices + at + i] = static_cast<uint16_t>(e);
            before += total;
        }
        if (lane == 0) r.entries = before;
    }
    __syncthreads();
}

// The choices of one entry in ascending order, to a warp's list; their number.
template <int SIZE>
__device__ __forceinline__ int list_tokens(const Routing& r, uint16_t* list, int entry, int choices) {
    const int lane = threadIdx.x % 32, expert = r.active[entry];
    // (an expert's entries follow one another)
    int n = 0;
    for (int i = entry; i > 0 && r.active[i - 1] == expert; --i) n -= SIZE;
    __syncwarp();
    for (int i = lane; i - lane < choices && n < SIZE; i += 32) {
        const bool match = i < choices && r.experts[i] == expert;
        const uint32_t b = __ballot_sync(0xffffffffu, match);
        const int at = n + __popc(b & ((1u << lane) - 1u));
        if (match && at >= 0 && at < SIZE) list[at] = static_cast<uint16_t>(i);
        n += __popc(b);
    }
    __syncwarp();
    return min(n, SIZE);
}

// h in shared memory and on its way there.  A lane multiplies 8 consecutive elements of a token (few.cuh), which
// are two 16-byte pieces of fp32; each piece of the four lanes of a token lies side by side, so that a copy's and a
// read's 16 bytes a lane are 64 in a row.  Element k of a row:
template <bool I8>
__device__ __forceinline__ int64_t h_place(int64_t k) {
    constexpr int LANE = I8 ? 16 : 8;
    const int in = static_cast<int>(k) & (4 * LANE - 1);
    return k - in + in % LANE / 4 * 16 + in / LANE * 4 + in % 4;
}

// The exponent field of the power of two that brings `top` (the bits of the largest |h|) to 2^14 .. 2^15.  A largest
// one that is infinite or NaN gives kNoScale, 2^-114: what is finite beside it stays so, and the products are what
// the infinity or NaN makes of them.
constexpr uint32_t kNoScale = 268u - 255u;
__device__ __forceinline__ uint32_t scale_bits(uint32_t top) { return min(268u - (top >> 23), 253u); }
__device__ __forceinline__ float scale_of(uint32_t bits) { return __uint_as_float(bits << 23); }
__device__ __forceinline__ float unscale_of(uint32_t bits) { return __uint_as_float((254u - bits) << 23); }

// Eight elements of h as the pairs of 16-bit values the multiply takes, the largest parts first.
constexpr int h_parts(bool bf16) { return bf16 ? 3 : 2; }
template <bool BF16>
__device__ __forceinline__ void take_apart(const uint32_t (&a)[4], const uint32_t (&b)[4], uint32_t scale, uint32_t (&v)[h_parts(BF16)][4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float f0 = __uint_as_float(j < 2 ? a[2 * j] : b[2 * j - 4]), f1 = __uint_as_float(j < 2 ? a[2 * j + 1] : b[2 * j - 3]);
        if constexpr (BF16) {
            // 8 bits, 8 more, and the 8 that are left: every difference is exact
            const auto high = [](float f) { return __uint_as_float(__float_as_uint(f) & 0xFFFF0000u); };
            const auto pair = [](float x, float y) { return __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632); };
            const float m0 = __fsub_rn(f0, high(f0)), m1 = __fsub_rn(f1, high(f1));
            const float l0 = __fsub_rn(m0, high(m0)), l1 = __fsub_rn(m1, high(m1));
            // (an infinity has no rest: inf - inf would make it NaN)
            const bool finite = scale != kNoScale;
            v[0][j] = pair(f0, f1);
            v[1][j] = finite ? pair(m0, m1) : 0u;
            v[2][j] = finite ? pair(l0, l1) : 0u;
        } else {
            const float s = scale_of(scale), g0 = f0 * s, g1 = f1 * s;
            v[0][j] = fused::pack16(g0, g1, false);
            const float2 kept = fused::unpack16(v[0][j], false);
            v[1][j] = scale != kNoScale ? fused::pack16(__fsub_rn(g0, kept.x), __fsub_rn(g1, kept.y), false) : 0u;
        }
    }
}

__device__ __forceinline__ void prefetch_l1(const void* p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }

// One pass over the chosen experts' weights, 32 rows of an entry's at a time (a
// unit): eight warps take the steps of the rows' length in turn, their sums are
// joined in warp order, and a thread finishes a row of a token.
//
// Gate and up (DOWN false): 16 rows of F of each;  h = act(Wg x) (Wu x), and each choice's largest |h|.
// Down (DOWN true): 32 rows of K;  p Wd h of each choice, in fp32 to `partial`.  The
// block that finishes the last of a row block's entries adds up every token's
// choices in their order: y, whatever order the units were finished in.  The
// arrival's number is looked at one unit later, so that nobody waits for it.
//
// A unit is p.groups such 32 rows, each 8 / p.groups of the warps': short rows in
// 8 bits are a few steps, and a join for each 64 KB took as long as reading them
// (down of 32 tokens, 32 experts of 2048 x 4096 in 8 bits, 138 us).
template <int FORM, bool ALIGNED, int NT, bool DOWN>
__global__ void __launch_bounds__(kWarps * 32, 2)
moe_experts_kernel(const __grid_constant__ Params p) {
    constexpr int STEP = step_k(FORM), WB = weight_bytes(FORM), LANE = 16 / WB, HALVES = halves_of(FORM);
    // (16-byte pieces of tokens: 8 elements of x are one, of h two)
    constexpr int XB = NT * HALVES, PIECES = DOWN ? 2 * XB : XB, ROWS = DOWN ? 32 : 16;
    using ExpertsRing = Ring<ALIGNED, PIECES, kBeside>;
    constexpr bool BF16 = is_bf16(FORM);
    extern __shared__ uint4 ring_smem[];
    __shared__ Routing routing;
    __shared__ __align__(16) int queue[Claims::QUEUE];
    __shared__ __align__(16) float part[kWarps][2][16][8];      // (read and written in pairs)
    __shared__ int finished;
    __shared__ uint32_t tile_tops[8];                           // gate and up: of a unit's tile, each token's largest |h|
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    // Down reads the routing while gate and up still run: they let it start after their own wait for
    // the router, so its results are there, in L2, where they are read (ptx.cuh; one token's layer 20.6 to 17.4 us, with the second unit's claim
    // under way while the ring fills).  h is read, and units are claimed, behind the wait alone.
    if (!DOWN) {
        // (in this order: down's early read rests on it)
        grid_dependency_wait();
        allow_dependent_launch();
    }
    const int choices = p.M * p.top_k;
    // the routing's arrays lie behind the rings
    read_routing<8 * NT>(routing, reinterpret_cast<uint16_t*>(reinterpret_cast<char*>(ring_smem) + kWarps * ExpertsRing::WARP_BYTES),
                         p.experts, choices, p.E);
    const int64_t F = p.F, K = p.K, length = DOWN ? F : K, height = DOWN ? K : F;
    // this warp's 32 rows of a unit, and its number among those that share them
    const int split = kWarps / p.groups, group = warp / split, part_of = warp % split, unit_rows = ROWS * p.groups;
    const int blocks = static_cast<int>(((DOWN ? K : p.ldh) + unit_rows - 1) / unit_rows), units = routing.entries * blocks;
    const int steps = static_cast<int>((length + STEP - 1) / STEP), stride = split * STEP;
    const int mine = (steps - part_of + split - 1) / split;     // of a unit; may be none
    const Claims claims{queue, p.counters + (DOWN ? 1 : 0), Claims::too_short(steps / split, ExpertsRing::STAGES)};
    if (!DOWN && threadIdx.x < 8) tile_tops[threadIdx.x] = 0u;
    if (threadIdx.x == 0) claims.start();
    __syncthreads();

    // this lane's 16 bytes of rows g and g + 8 of gate and up, or g, g + 8, g + 16 and g + 24, and what
    // the rows have left from there on (a row past the last reads that one; its results are dropped)
    struct Rows {
        const uint8_t* at[kLoads];
        int left;
    };
    const int row_bytes = static_cast<int>(length) * WB, offset = (part_of * STEP + t * LANE) * WB;
    const auto rows_of = [&](int u) {
        const int a = u / blocks;
        const int64_t row0 = static_cast<int64_t>(u - a * blocks) * unit_rows + group * ROWS, first = routing.active[a] * height;
        Rows r;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int64_t at = (first + min(row0 + g + 8 * (DOWN ? i : i % 2), height - 1)) * row_bytes + offset;
            r.at[i] = (DOWN ? p.w_down : i < 2 ? p.w_gate : p.w_up) + at;
        }
        r.left = row_bytes - offset;
        return r;
    };
    ExpertsRing ring(smem_u32(ring_smem), warp);
    int next_i = 0, next_j = 0, next_entry = -1, next_count = 0;
    Rows next = {{p.w_down, p.w_down, p.w_down, p.w_down}, 0};
    using Token = typename std::conditional<DOWN, float, uint16_t>::type;
    const Token* xp[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) xp[i] = nullptr;
    bool more = mine > 0;
    const auto enter = [&](int u) {
        more = more && u < units;
        if (!more) return;
        next = rows_of(u);
        const int a = u / blocks;
        if (a != next_entry) {
            next_entry = a;
            next_count = list_tokens<8 * NT>(routing, routing.list[warp][0], a, choices);
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            // (columns past the entry's tokens are the first one's once more, and not looked at)
            const int choice = routing.list[warp][0][8 * i + g < next_count ? 8 * i + g : 0];
            if constexpr (DOWN)
                xp[i] = p.h + choice * p.ldh + part_of * STEP + t * 4;
            else
                xp[i] = p.x + choice / p.top_k * p.ldx + part_of * STEP + t * LANE;
        }
    };
    enter(claims.unit(0));
    const auto fill = [&]() {
        if (more) {
            ring.copy(next.at, next.left);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                if (8 * i >= next_count) break;
#pragma unroll
                for (int half = 0; half < HALVES; ++half) {
                    const int piece = i * HALVES + half;
                    if constexpr (DOWN) {
                        ring.copy_token(2 * piece, xp[i] + 32 * half);
                        ring.copy_token(2 * piece + 1, xp[i] + 32 * half + 16);
                    } else {
                        ring.copy_token(piece, xp[i] + 8 * half);
                    }
                }
                xp[i] += stride;
            }
            if (++next_j == mine) {
                next_j = 0;
                enter(claims.unit(++next_i));
            } else {
#pragma unroll
                for (int i = 0; i < kLoads; ++i) next.at[i] += stride * WB;
                next.left -= stride * WB;
            }
        }
        ring.commit();
    };
    if (DOWN) {
        grid_dependency_wait();
        allow_dependent_launch();
        if (static_cast<int>(threadIdx.x) * 32 < choices) {
            // what the units and their joins ask for of each choice, into L1
            prefetch_l1(p.tops + threadIdx.x * 32);
            prefetch_l1(p.weights + threadIdx.x * 32);
        }
    }
    const int second = threadIdx.x == 0 ? claims.claim() : 0;
#pragma unroll
    for (int i = 0; i < ExpertsRing::STAGES - 1; ++i) fill();
    if (threadIdx.x == 0) claims.second(second);
    __syncthreads();            // (if units are claimed, the first one fills the ring)

    // Down: the unit before's row block and the number of its arrival (thread 0's)
    int before = -1, arrival = 0;
    // Thread 0, before a barrier: that row block if its last arrival was this block's, or -1.  The fence between the
    // counter and the barrier orders the other blocks' stores, each fenced ahead of its own arrival, before
    // all of this block's loads behind the barrier.
    const auto last_there = [&]() {
        if (before < 0 || arrival != routing.entries - 1) return -1;
        __threadfence();
        return before;
    };
    const auto add_choices = [&](int done) {
        if (done < 0) return;
        const int64_t row0 = static_cast<int64_t>(done) * unit_rows;
        for (int i = threadIdx.x; i < p.M * unit_rows; i += kWarps * 32) {
            const int m = i / unit_rows;
            const int64_t row = row0 + i % unit_rows;
            if (row >= K) continue;
            const float* from = p.partial + static_cast<int64_t>(m) * p.top_k * K + row;
            float sum = 0.0f;
            for (int j = 0; j < p.top_k; ++j) sum += __ldcg(from + j * K);
            p.y[m * K + row] = static_cast<uint16_t>(fused::pack16(sum, 0.0f, p.bf16));
        }
    };

    int entry = -1, count = 0, tiles = 0;
    uint16_t* const list = routing.list[warp][1];
    uint32_t scale[NT];                 // down: of the token this lane multiplies, of each tile
#pragma unroll
    for (int i = 0; i < NT; ++i) scale[i] = 0u;
    for (int i_unit = 0;; ++i_unit) {
        const int u = claims.unit(i_unit);
        if (u >= units) break;
        const int claimed = threadIdx.x == 0 ? claims.claim() : 0;
        const int a = u / blocks, block = u - a * blocks, expert = routing.active[a];
        const int64_t row0 = static_cast<int64_t>(block) * unit_rows;
        if (a != entry) {
            entry = a;
            count = list_tokens<8 * NT>(routing, list, a, choices);
            tiles = (count + 7) / 8;
            if (DOWN) {
#pragma unroll
                for (int i = 0; i < NT; ++i) scale[i] = scale_bits(p.tops[list[8 * i + g < count ? 8 * i + g : 0]]);
            }
        }
        if constexpr (is_i8(FORM)) {
            // the join's scales, into L1 ahead of it
            const int64_t row = row0 + threadIdx.x;
            if (static_cast<int>(threadIdx.x) < unit_rows && row < height) {
                const int64_t at = expert * height + row;
                prefetch_l1((DOWN ? p.s_down : p.s_gate) + at);
                if (!DOWN) prefetch_l1(p.s_up + at);
            }
        }
        Rows rows = rows_of(u);
        float acc[NT][2][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][0][j] = acc[i][1][j] = 0.0f;
        for (int j = 0; j < mine; ++j) {
            ring.wait();
            uint4 w[kLoads];
            uint32_t xv[PIECES][4];
#pragma unroll
            for (int i = 0; i < kLoads; ++i) w[i] = ring.get(i, rows.at[i], rows.left);
            rows.left -= stride * WB;
#pragma unroll
            for (int i = 0; i < PIECES; ++i)
                if (i / (PIECES / NT) < tiles) ring.get_token(i, xv[i]);
            ring.pop();
            fill();
#pragma unroll
            for (int half = 0; half < HALVES; ++half) {
                uint32_t v[kLoads][4];
#pragma unroll
                for (int i = 0; i < kLoads; ++i) widen<FORM>(w[i], half, v[i]);
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    if (i >= tiles) break;
                    const int piece = i * HALVES + half;
                    if constexpr (DOWN) {
                        uint32_t h[h_parts(BF16)][4];
                        take_apart<BF16>(xv[2 * piece], xv[2 * piece + 1], scale[i], h);
#pragma unroll
                        for (int k = 0; k < h_parts(BF16); ++k) {
                            mma_step<BF16>(acc[i][0], v[0], v[1], h[k]);
                            mma_step<BF16>(acc[i][1], v[2], v[3], h[k]);
                        }
                    } else {
                        mma_step<BF16>(acc[i][0], v[0], v[1], xv[piece]);
                        mma_step<BF16>(acc[i][1], v[2], v[3], xv[piece]);
                    }
                }
            }
        }
        if (threadIdx.x == 0) {
            claims.put(i_unit, claimed);
            finished = last_there();
        }
        // join the warps' sums tile by tile; a thread finishes row r of token n, of group m (gate
        // and up) or of each group's half m (down)
        const int r = threadIdx.x / 8 % 16, n = threadIdx.x % 8, m = threadIdx.x / 128;
        int done = -1;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            if (i >= tiles) break;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                *reinterpret_cast<float2*>(&part[warp][k][g][2 * t]) = make_float2(acc[i][k][0], acc[i][k][1]);
                *reinterpret_cast<float2*>(&part[warp][k][g + 8][2 * t]) = make_float2(acc[i][k][2], acc[i][k][3]);
            }
            __syncthreads();
            done = finished;            // (written before this barrier, and not again before the next)
            uint32_t top = 0u;          // bits of the largest |h| (magnitudes are ordered as their bits are, NaN above infinity)
            for (int of = DOWN ? 0 : m; 8 * i + n < count && of < p.groups; of += DOWN ? 1 : 2) {
                const int choice = list[8 * i + n];
                const int64_t row = row0 + of * ROWS + (DOWN ? 16 * m : 0) + r;
                float sum = 0.0f, up = 0.0f;
                for (int k = of * split; k < (of + 1) * split; ++k) {
                    sum += part[k][DOWN ? m : 0][r][n];
                    if (!DOWN) up += part[k][1][r][n];
                }
                if constexpr (DOWN) {
                    if (row < K) {
                        // (binary16: out of the scale's units, by the weights' scale first so that neither leaves fp32's range alone)
                        float back = BF16 ? 1.0f : unscale_of(scale_bits(p.tops[choice]));
                        if constexpr (is_i8(FORM)) back *= p.s_down[expert * K + row];
                        p.partial[choice * K + row] = sum * p.weights[choice] * back;
                    }
                } else if (row < p.ldh) {
                    float h = 0.0f;
                    if (row < F) {
                        if constexpr (is_i8(FORM)) {
                            sum *= p.s_gate[expert * F + row];
                            up *= p.s_up[expert * F + row];
                        }
                        h = fused::act_value(sum, p.act) * up;
                    }
                    // (columns from F to the padded row's end are zeros)
                    p.h[choice * p.ldh + h_place<is_i8(FORM)>(row)] = h;
                    top = max(top, __float_as_uint(h) & 0x7FFFFFFFu);
                }
            }
            if (!DOWN) {
                // this warp's rows of each token
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 8));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 16));
                if (lane < 8 && top != 0u) atomicMax(tile_tops + lane, top);
            }
            __syncthreads();
            if (!DOWN && threadIdx.x < 8 && 8 * i + n < count) {
                // the unit's, once for each token (an atomic of every warp made 64 tokens over 8 experts 4 us longer)
                if (const uint32_t all = tile_tops[n]) atomicMax(p.tops + list[8 * i + n], all);
                tile_tops[n] = 0u;
            }
        }
        if (DOWN) {
            // (the barrier ordered the block's stores before this thread's fence)
            if (threadIdx.x == 0) {
                __threadfence();
                arrival = atomicAdd(p.counters + 2 + block, 1);
            }
            before = block;
            add_choices(done);
        }
    }
    cp_async_wait_group<0>();
    if (DOWN) {
        if (threadIdx.x == 0) finished = last_there();
        __syncthreads();
        add_choices(finished);
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
    // (a row's bytes and the units of work are counted in an int)
    if (bad_size(c.M) || c.K < 0 || c.K > kMaxWidth || c.F < 0 || c.F > kMaxWidth) return GEMM_ERR_INVALID_ARG;
    if (c.E < 1 || c.E > kMaxExperts || c.top_k < 1 || c.top_k > kMaxTopK || c.top_k > c.E) return GEMM_ERR_INVALID_ARG;
    if (c.type != GEMM_TYPE_HALF && c.type != GEMM_TYPE_BFLOAT) return GEMM_ERR_INVALID_ARG;
    if (c.weight_type != c.type && c.weight_type != GEMM_TYPE_BYTE) return GEMM_ERR_INVALID_ARG;
    if (c.act != GEMM_ACT_SILU && c.act != GEMM_ACT_GELU) return GEMM_ERR_INVALID_ARG;
    if (c.normalize != 0 && c.normalize != 1) return GEMM_ERR_INVALID_ARG;
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
struct Workspace {
    uint16_t* x = nullptr;
    float* h = nullptr;
    int* counters = nullptr;
    float* partial = nullptr;
    size_t bytes = 0;
};
// the kernels' counters, and the choices' largest |h| behind them
int64_t num_counters(int64_t K) { return 2 + cdiv(K, 32); }
Workspace workspace_of(const Call& c, void* base) {
    Workspace w;
    if (c.M == 0 || c.K == 0) return w;
    fused::Carver carver;
    carver.base = static_cast<char*>(base);
    const int64_t tokens = pass_tokens(c.M);
    w.x = carver.take<uint16_t>(tokens * ldh_of(c.K));
    w.h = carver.take<float>(tokens * c.top_k * ldh_of(c.F));
    w.counters = carver.take<int>(num_counters(c.K) + tokens * c.top_k);
    w.partial = carver.take<float>(tokens * c.top_k * c.K);
    w.bytes = carver.used;
    return w;
}

bool rows16(const void* p, int64_t row_bytes) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && row_bytes % 16 == 0; }

int launched(cudaError_t e) {
    if (e == cudaSuccess) return GEMM_OK;
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
}

// Parts of K a row of the router is cut into: all of a cluster's warps have one.
int route_parts(int64_t E, int64_t K, int warps) {
    int parts = 1;
    while (parts < 8 && 2 * E * parts <= warps && K > 512 * parts) parts *= 2;
    return parts;
}

template <bool BF16, bool ALIGNED, int TOKENS>
int launch_route(const Call& c, const uint8_t* x, int M, int* experts, float* weights, const Workspace& ws, cudaStream_t stream) {
    constexpr int threads = route_threads(TOKENS);
    const int parts = route_parts(c.E, c.K, kRouteCtas * threads / 32);
    Handover out = {ws.counters, ws.x, num_counters(c.K) + M * c.top_k, ldh_of(c.K)};
    if (!ws.counters) out.num_counters = 0;
    return launched(launch_pdl(moe_route_kernel<BF16, ALIGNED, TOKENS>, dim3(static_cast<unsigned>(cdiv(M, TOKENS) * kRouteCtas)),
                               dim3(threads), static_cast<size_t>(TOKENS) * c.E * parts * 8, stream, x,
                               static_cast<const uint8_t*>(c.w_router), M, c.K, static_cast<int>(c.E), parts,
                               static_cast<int>(c.top_k), c.normalize, experts, weights, out));
}

// 16 tokens, a cluster each, still fit the GPU at once.
template <bool BF16, bool ALIGNED>
int launch_route_tokens(const Call& c, const uint8_t* x, int M, int* experts, float* weights, const Workspace& ws, cudaStream_t stream) {
    return M <= 16 ? launch_route<BF16, ALIGNED, 1>(c, x, M, experts, weights, ws, stream)
                   : launch_route<BF16, ALIGNED, kRouteTokens>(c, x, M, experts, weights, ws, stream);
}

// How many blocks of a kernel fit the GPU at once, with `smem` bytes of the `most` it
// may have; set up on the first call on a device.
struct Fit {
    std::atomic<int> blocks[64] = {};
};
template <typename Kernel>
int blocks_at_once(Fit& fit, Kernel kern, int smem, int most, const DeviceInfo& info) {
    if (info.device < 0 || info.device >= 64) return 0;
    int n = fit.blocks[info.device].load(std::memory_order_relaxed);
    if (n == 0) {
        // concurrent first calls compute and store the same value
        int per_sm = 0;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kWarps * 32, smem) != cudaSuccess || per_sm <= 0) {
            cudaGetLastError();
            return 0;
        }
        n = per_sm * info.num_sms;
        fit.blocks[info.device].store(n, std::memory_order_relaxed);
    }
    return n;
}

template <int FORM, bool ALIGNED, int NT, bool DOWN>
int launch_experts(Params p, const DeviceInfo& info, cudaStream_t stream) {
    constexpr int ring = kWarps * Ring<ALIGNED, (DOWN ? 2 : 1) * NT * halves_of(FORM), kBeside>::WARP_BYTES;
    const auto kern = moe_experts_kernel<FORM, ALIGNED, NT, DOWN>;
    const int64_t choices = static_cast<int64_t>(p.M) * p.top_k;
    static Fit fit;
    const int64_t fits = blocks_at_once(fit, kern, ring + routing_bytes(256), ring + routing_bytes(kTokens * kMaxTopK), info);
    if (fits == 0) return GEMM_ERR_LAUNCH;
    // the most entries that the routing can give
    const int64_t entries = (choices < p.E ? choices : p.E) + choices / (8 * NT);
    const int64_t rows = DOWN ? p.K : p.ldh, steps = cdiv(DOWN ? p.F : p.K, step_k(FORM));
    // units of 16 steps a warp, as long as every block has four of them (8 and 32 steps: 209 and 197
    // against 196 us for 32 tokens over 32 experts of 2048 x 4096 in 8 bits, 394 and 410 against 392
    // for 16 tokens over 56 of 1536 x 4096 in 16)
    p.groups = 1;
    while (p.groups < kWarps && steps * p.groups < 16 * kWarps && entries * cdiv(rows, 2 * p.groups * (DOWN ? 32 : 16)) >= 4 * fits) p.groups *= 2;
    const int64_t units = entries * cdiv(rows, p.groups * (DOWN ? 32 : 16));
    return launched(launch_pdl(kern, dim3(static_cast<unsigned>(units < fits ? units : fits)), dim3(kWarps * 32),
                               ring + routing_bytes(static_cast<int>(choices)), stream, p));
}

// Two tiles where an expert has more than four tokens on average: one tile's ring
// leaves room for more blocks, two read a crowded expert's weights half as often.
template <int FORM, bool ALIGNED, bool DOWN>
int launch_tiles(const Params& p, const DeviceInfo& info, cudaStream_t stream) {
    if (p.M <= 8 || p.M * p.top_k <= 4 * p.E) return launch_experts<FORM, ALIGNED, 1, DOWN>(p, info, stream);
    return launch_experts<FORM, ALIGNED, 2, DOWN>(p, info, stream);
}

template <int FORM, bool DOWN>
int launch_form(const Params& p, bool aligned, const DeviceInfo& info, cudaStream_t stream) {
    return aligned ? launch_tiles<FORM, true, DOWN>(p, info, stream) : launch_tiles<FORM, false, DOWN>(p, info, stream);
}

template <bool DOWN>
int launch_kernel(const Params& p, int form, bool aligned, const DeviceInfo& info, cudaStream_t stream) {
    switch (form) {
        case kHalf: return launch_form<kHalf, DOWN>(p, aligned, info, stream);
        case kBfloat: return launch_form<kBfloat, DOWN>(p, aligned, info, stream);
        case kI8Half: return launch_form<kI8Half, DOWN>(p, aligned, info, stream);
        // (down's h is binary16 values beside 8-bit weights, whatever the tokens are)
        default: return launch_form<DOWN ? kI8Half : kI8Bfloat, DOWN>(p, aligned, info, stream);
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
    if (!fused::workspace_ok(workspace, workspace_bytes, workspace_of(c, nullptr).bytes, in, out)) return GEMM_ERR_INVALID_ARG;
    DeviceInfo info;
    rc = current_device(&info);
    if (rc != GEMM_OK) return rc;

    const bool i8 = c.weight_type == GEMM_TYPE_BYTE, bf16 = c.type == GEMM_TYPE_BFLOAT;
    const int form = (i8 ? 2 : 0) + (bf16 ? 1 : 0), wbytes = i8 ? 1 : 2;
    const bool route_aligned = rows16(c.x, 2 * c.K) && rows16(c.w_router, 2 * c.K);
    const bool gate_aligned = rows16(c.w_gate, wbytes * c.K) && rows16(c.w_up, wbytes * c.K);
    const bool down_aligned = rows16(c.w_down, wbytes * c.F);
    Params p = {};
    p.w_gate = static_cast<const uint8_t*>(c.w_gate);
    p.w_up = static_cast<const uint8_t*>(c.w_up);
    p.w_down = static_cast<const uint8_t*>(c.w_down);
    p.s_gate = c.s_gate;
    p.s_up = c.s_up;
    p.s_down = c.s_down;
    const Workspace ws = workspace_of(c, workspace);
    p.x = ws.x;
    p.ldx = ldh_of(c.K);
    p.h = ws.h;
    p.counters = ws.counters;
    p.tops = reinterpret_cast<uint32_t*>(ws.counters + num_counters(c.K));
    p.bf16 = bf16;
    p.partial = ws.partial;
    p.K = c.K;
    p.F = c.F;
    p.ldh = ldh_of(c.F);
    p.E = static_cast<int>(c.E);
    p.top_k = static_cast<int>(c.top_k);
    p.act = c.act;
    for (int64_t m = 0; m < c.M; m += kTokens) {
        p.M = static_cast<int>(c.M - m < kTokens ? c.M - m : kTokens);
        const uint8_t* x = static_cast<const uint8_t*>(c.x) + m * c.K * 2;
        p.y = static_cast<uint16_t*>(c.y) + m * c.K;
        p.experts = c.experts + m * c.top_k;
        p.weights = c.weights + m * c.top_k;
        int* experts = c.experts + m * c.top_k;
        float* weights = c.weights + m * c.top_k;
        if (bf16)
            rc = route_aligned ? launch_route_tokens<true, true>(c, x, p.M, experts, weights, ws, stream)
                               : launch_route_tokens<true, false>(c, x, p.M, experts, weights, ws, stream);
        else
            rc = route_aligned ? launch_route_tokens<false, true>(c, x, p.M, experts, weights, ws, stream)
                               : launch_route_tokens<false, false>(c, x, p.M, experts, weights, ws, stream);
        if (rc != GEMM_OK) return rc;
        if (c.K == 0) continue;
        if (c.F == 0) {
            if (cudaMemsetAsync(p.y, 0, fused::bytes16(p.M, c.K), stream) != cudaSuccess) return GEMM_ERR_LAUNCH;
            continue;
        }
        if ((rc = launch_kernel<false>(p, form, gate_aligned, info, stream)) != GEMM_OK) return rc;
        if ((rc = launch_kernel<true>(p, form, down_aligned, info, stream)) != GEMM_OK) return rc;
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
    *bytes = static_cast<int64_t>(workspace_of(c, nullptr).bytes);
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

// gemm_i8.cu -- products of 8-bit integer matrices with a scale for each row,
// and the quantization that makes such matrices.
//
// sm_103a's tensor cores multiply no 8-bit integers (tcgen05's kind::i8 does not
// exist there), but every 8-bit integer is a binary16 value, their products are
// exact in the fp32 accumulator, and so are sums of up to 1024 of them: 128 * 128 *
// 1024 = 2^24.  The product therefore runs at the 16-bit rate and is exact: the
// accumulator is handed over every 1024 of K and added up in integers.
#include "few.cuh"
#include "product_host.cuh"

namespace pws {
namespace i8 {

using namespace fused;

constexpr int64_t kMaxK = 131071;           // 128 * 128 * K < 2^31
constexpr int kChunk = 16;                  // K blocks of 64 whose sum fp32 holds exactly
static_assert(kChunk % kMaxBoxes == 0, "a chunk ends with a slot");

// ---------------------------------------------------------------- quantization

constexpr float kMagic = 12582912.0f;       // 1.5 * 2^23: a sum with it is rounded to a whole number, in its low bits

// rint(127 x / top) for eight values, in the low bytes of b, from x times inverse =
// fl(127 / top), which is off by less than 2^-16 where it is nearest to 127.  A quotient of
// two 16-bit values that is not halfway between two integers is at least 2^-19 of
// its power of two from there (the values have at most 11 significant bits), 16
// times what the product is off by: only near a half can it mislead.  There the sides
// of 127 |x| / top = m + 1/2 are compared without a division: 254 |x| and (2 m + 1) top have at
// most 19 bits and are exact.  Five operations an element and one branch for
// eight: with a conversion, a branch and a division for each the pass was bound
// by them (85 us for 16384 x 8192).
__device__ __forceinline__ void quantize8(const float (&x)[8], float top, float inverse, uint32_t (&b)[8]) {
    float off = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float t = __fmaf_rn(x[j], inverse, kMagic), n = __fsub_rn(t, kMagic);
        off = fmaxf(off, fabsf(__fmaf_rn(x[j], inverse, -n)));
        b[j] = __float_as_uint(t);
    }
    if (off > 0.49998f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float q = fabsf(x[j]) * inverse, m = floorf(q);
            if (fabsf(q - m - 0.5f) < 2e-5f) {
                const float left = 254.0f * fabsf(x[j]), right = (2.0f * m + 1.0f) * top;
                const uint32_t low = __float_as_uint(m + kMagic);
                const uint32_t n = low + (left > right || (left == right && (low & 1u)) ? 1u : 0u);
                b[j] = x[j] < 0.0f ? 0u - n : n;
            }
        }
    }
}

// A row of x by LANES threads (a warp, or the block): its largest magnitude, then
// its integers.  Each thread keeps its first four chunks of eight elements in
// registers, so rows up to 32 LANES are read once; longer ones again, from L2.
// Bound by memory: 2 bytes read and 1 written per element.
template <int LANES, bool BF16, bool ALIGNED>
__global__ void __launch_bounds__(LANES < 256 ? 256 : LANES)
quantize_kernel(const uint8_t* __restrict__ x, int8_t* __restrict__ q, float* __restrict__ scale, int64_t M, int64_t K) {
    grid_dependency_wait();
    allow_dependent_launch();
    constexpr int KEEP = 4;
    __shared__ uint32_t part[32];
    const int lane = threadIdx.x % LANES;
    const int64_t row = LANES < 256 ? blockIdx.x * static_cast<int64_t>(256 / LANES) + threadIdx.x / LANES : blockIdx.x;
    if (LANES < 256 && row >= M) return;
    const uint8_t* src = x + row * K * 2;
    const int64_t chunks = (K + 7) / 8;
    const auto load = [&](int64_t i) { return few::load_row<ALIGNED, true>(src + 16 * i, 2 * (K - 8 * i)); };
    uint4 kept[KEEP];
    // magnitudes are ordered as their bits are, NaN above infinity
    uint32_t top = 0u;
    const auto take = [&](const uint4& v) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) top = __vmaxu2(top, w[i] & 0x7FFF7FFFu);
    };
#pragma unroll
    for (int j = 0; j < KEEP; ++j) {
        const int64_t i = lane + static_cast<int64_t>(j) * LANES;
        kept[j] = i < chunks ? load(i) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int j = 0; j < KEEP; ++j) take(kept[j]);
    for (int64_t i = lane + static_cast<int64_t>(KEEP) * LANES; i < chunks; i += LANES) take(load(i));
    top = max(top & 0xFFFFu, top >> 16);
    top = __reduce_max_sync(0xffffffffu, top);
    if (LANES > 32) {
        if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = top;
        __syncthreads();
        top = threadIdx.x % 32 < LANES / 32 ? part[threadIdx.x % 32] : 0u;
        top = __reduce_max_sync(0xffffffffu, top);
    }
    float most = unpack16(top, BF16).x;
    const bool finite = most <= 3.4e38f;
    if (lane == 0) scale[row] = finite ? __fdiv_rn(most, 127.0f) : __int_as_float(0x7fffffff);
    // bfloat16's range: brought to where neither 127 x nor 127 / top leaves fp32's.  (What
    // becomes zero on the way is below 2^-60 of the largest.)
    float by = 1.0f;
    if (BF16) by = most > 0x1p64f ? 0x1p-64f : (most < 0x1p-64f ? 0x1p64f : 1.0f);
    most *= by;
    const float inverse = finite && most > 0.0f ? __fdiv_rn(127.0f, most) : 0.0f;
    int8_t* dst = q + row * K;
    const bool wide = (reinterpret_cast<uintptr_t>(dst) & 7u) == 0;
    const auto put = [&](int64_t i, const uint4& v) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        float f[8];
        uint32_t b[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 two = unpack16(w[j], BF16);
            f[2 * j] = two.x;
            f[2 * j + 1] = two.y;
        }
        if (BF16 && by != 1.0f) {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] *= by;
        }
        if (finite) {
            quantize8(f, most, inverse, b);
        } else {
            // (a row with an infinity or a NaN is zeros)
#pragma unroll
            for (int j = 0; j < 8; ++j) b[j] = 0u;
        }
        if (wide && 8 * i + 8 <= K) {
            const uint32_t lo = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
            const uint32_t hi = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
            *reinterpret_cast<uint2*>(dst + 8 * i) = make_uint2(lo, hi);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (8 * i + j < K) dst[8 * i + j] = static_cast<int8_t>(b[j]);
        }
    };
#pragma unroll
    for (int j = 0; j < KEEP; ++j) {
        const int64_t i = lane + static_cast<int64_t>(j) * LANES;
        if (i < chunks) put(i, kept[j]);
    }
    for (int64_t i = lane + static_cast<int64_t>(KEEP) * LANES; i < chunks; i += LANES) put(i, load(i));
}

template <int LANES, bool BF16>
int launch_quantize(int64_t M, int64_t K, const void* x, int8_t* q, float* scale, cudaStream_t stream) {
    const bool aligned = reinterpret_cast<uintptr_t>(x) % 16 == 0 && K % 8 == 0;
    const int64_t blocks = LANES < 256 ? cdiv(M, 256 / LANES) : M;
    const auto kern = aligned ? quantize_kernel<LANES, BF16, true> : quantize_kernel<LANES, BF16, false>;
    if (launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(LANES < 256 ? 256 : LANES), 0, stream,
                   static_cast<const uint8_t*>(x), q, scale, M, K) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

// ---------------------------------------------------------------- widening

// Rows of 8-bit integers at any address as binary16 rows ld apart (a multiple of
// 64, the rest of the last 16 elements zeros), two matrices in one launch.  16
// elements a thread: 16 bytes read, 32 written.
struct Widen {
    const uint8_t* src[2];
    uint16_t* dst[2];
    int64_t rows[2];
};

template <bool ALIGNED>
__global__ void __launch_bounds__(256)
widen_kernel(const __grid_constant__ Widen p, int64_t K, int64_t ld) {
    // (in this order: batch_kernel's early copies rest on it)
    grid_dependency_wait();
    allow_dependent_launch();
    const int64_t chunks = (K + 15) / 16, total = (p.rows[0] + p.rows[1]) * chunks;
    for (int64_t id = blockIdx.x * 256ll + threadIdx.x; id < total; id += gridDim.x * 256ll) {
        int64_t row = id / chunks;
        const int64_t c = (id - row * chunks) * 16;
        const int m = row >= p.rows[0] ? 1 : 0;
        row -= m * p.rows[0];
        const uint4 w = few::load_row<ALIGNED, true>(p.src[m] + row * K + c, K - c);
        uint4* to = reinterpret_cast<uint4*>(p.dst[m] + row * ld + c);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t v[4];
            few::widen<few::kI8Half>(w, half, v);
            to[half] = make_uint4(v[0], v[1], v[2], v[3]);
        }
    }
}

// ---------------------------------------------------------------- few tokens

// A few rows of `a` (few_tokens): 32 rows of b at a time by a cluster of `ctas` CTAs,
// whose warps take the steps of K in turn (few.cuh).  Bound by b's bytes.  A warp's fp32
// sums are whole numbers and exact over 16 steps (1024 of K); they are added up
// as integers in shared memory, whose order does not matter: the parts of a cluster
// and of its warps are joined exactly.
constexpr int kFewRows32 = 32;
constexpr int kFewWarps = 8;
constexpr int kExactSteps = 16;
// Up to 16 tokens (16384 x 4096, cold caches: 19.7 us, batch_kernel 22.0), and up to 32
// through matrices of up to 8 MB: with four token tiles a warp's loads no longer run
// ahead of its multiplies (32 tokens 35.5 us through 16384 x 4096 where batch_kernel
// takes 22.5, 15.3 and 11.6 through 4096 x 4096), but a small matrix ends before the
// other kernel's widened copy of the tokens, its barriers and its longer epilogue pay
// (1024 x 8192 8.4 and 11.1 us, 4096 x 1024 6.1 and 8.2).
constexpr int64_t kFewBytes = 8 << 20;
bool few_tokens(int64_t M, int64_t N, int64_t K) { return M <= 16 || (M <= 32 && N * K <= kFewBytes); }
// bytes of the warps' sums of NT tiles
constexpr int few_columns(int tiles) { return kFewWarps * kFewRows32 * 8 * tiles * 4; }

struct FewParams {
    const uint8_t* a;               // [M][lda], rows on 16-byte boundaries
    const uint8_t* b;               // [N, K]
    const float* a_scale;
    const float* b_scale;
    uint16_t* out;                  // [M, N]
    int64_t lda, N;
    int M, K, ctas, bf16;
};

template <bool ALIGNED, int NT>
__global__ void __launch_bounds__(kFewWarps * 32, NT <= 2 ? 2 : 1)
few_kernel(const __grid_constant__ FewParams p) {
    using few::kLoads;
    constexpr int STEP = 64, LDC = 8 * NT;
    using Ring = few::Ring<ALIGNED, NT, few_columns(NT)>;
    extern __shared__ uint4 ring_smem[];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const uint32_t rank = cluster_ctarank();
    // [kFewWarps][32][LDC]
    int* const columns = reinterpret_cast<int*>(reinterpret_cast<char*>(ring_smem) + kFewWarps * Ring::WARP_BYTES);
    int* const own = columns + warp * (kFewRows32 * LDC);
    for (int i = lane; i < kFewRows32 * LDC; i += 32) own[i] = 0;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x / static_cast<unsigned>(p.ctas)) * kFewRows32;
    const int workers = p.ctas * kFewWarps, worker = static_cast<int>(rank) * kFewWarps + warp;
    const int steps = (p.K + STEP - 1) / STEP, mine = steps > worker ? (steps - worker + workers - 1) / workers : 0;
    const int stride = workers * STEP;

    // this lane's 16 bytes of rows g, g + 8, g + 16 and g + 24 (a row past N reads the last one; its results are dropped)
    const uint8_t* at[kLoads];
    const uint8_t* xp[NT];
    int left = p.K - worker * STEP - t * 16;
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
        at[i] = p.b + min(row0 + g + 8 * i, p.N - 1) * p.K + worker * STEP + t * 16;
#pragma unroll
    for (int i = 0; i < NT; ++i) xp[i] = p.a + min(8 * i + g, p.M - 1) * p.lda + worker * STEP + t * 16;
    int read_left = left;
    const uint8_t* const row[kLoads] = {at[0], at[1], at[2], at[3]};
    Ring ring(smem_u32(ring_smem), warp);
    grid_dependency_wait();
    allow_dependent_launch();
    int filled = 0;
    const auto fill = [&]() {
        if (filled < mine) {
            ring.copy(at, left);
            // (behind the row's end b's zeros meet any bytes of a's rows)
#pragma unroll
            for (int i = 0; i < NT; ++i) ring.copy_token(i, left > 0 ? xp[i] : p.a);
#pragma unroll
            for (int i = 0; i < kLoads; ++i) at[i] += stride;
#pragma unroll
            for (int i = 0; i < NT; ++i) xp[i] += stride;
            left -= stride;
            ++filled;
        }
        ring.commit();
    };
#pragma unroll
    for (int i = 0; i < Ring::STAGES - 1; ++i) fill();

    float acc[NT][2][4];
    const auto clear = [&]() {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][0][j] = acc[i][1][j] = 0.0f;
    };
    const auto add_up = [&]() {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int r = 0; r < kLoads; ++r)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    own[(g + 8 * r) * LDC + 8 * i + 2 * t + j] += __float2int_rn(acc[i][r / 2][2 * (r & 1) + j]);
    };
    clear();
    __syncwarp();
    for (int j = 0; j < mine;) {
        for (const int end = min(mine, j + kExactSteps); j < end; ++j) {
            ring.wait();
            uint4 w[kLoads];
            uint32_t x[NT][4];
#pragma unroll
            for (int i = 0; i < kLoads; ++i) w[i] = ring.get(i, row[i], read_left);
#pragma unroll
            for (int i = 0; i < NT; ++i) ring.get_token(i, x[i]);
            read_left -= stride;
            ring.pop();
            fill();
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t v[kLoads][4];
#pragma unroll
                for (int i = 0; i < kLoads; ++i) few::widen<few::kI8Half>(w[i], half, v[i]);
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    uint32_t xv[4];
                    few::widen4<false>(x[i][2 * half], xv[0], xv[1]);
                    few::widen4<false>(x[i][2 * half + 1], xv[2], xv[3]);
                    few::mma_step<false>(acc[i][0], v[0], v[1], xv);
                    few::mma_step<false>(acc[i][1], v[2], v[3], xv);
                }
            }
        }
        add_up();
        clear();
    }
    cp_async_wait_group<0>();
    __syncthreads();
    for (int i = threadIdx.x; i < kFewRows32 * LDC; i += kFewWarps * 32) {
        int sum = columns[i];
#pragma unroll
        for (int k = 1; k < kFewWarps; ++k) sum += columns[k * (kFewRows32 * LDC) + i];
        columns[i] = sum;
    }
    __syncthreads();
    if (p.ctas > 1) cluster_sync();
    // 32 rows of a token in a row, the cluster's CTAs in turn
    for (int i = static_cast<int>(rank) * (kFewWarps * 32) + threadIdx.x; i < p.M * kFewRows32; i += p.ctas * (kFewWarps * 32)) {
        const int m = i / kFewRows32, r = i % kFewRows32;
        if (row0 + r >= p.N) continue;
        int sum = 0;
        const uint32_t from = smem_u32(columns + r * LDC + m);
        for (int q = 0; q < p.ctas; ++q) sum += static_cast<int>(ld_relaxed_cluster_u32(mapa_shared(from, q)));
        const float v = i8_value(sum, __ldg(p.a_scale + m), __ldg(p.b_scale + row0 + r));
        p.out[m * p.N + row0 + r] = static_cast<uint16_t>(pack16(v, 0.0f, p.bf16));
    }
    if (p.ctas > 1) {
        __syncthreads();
        cluster_sync();         // (no CTA leaves while another reads its sums)
    }
}

template <bool ALIGNED, int NT>
int launch_few(FewParams p, const DeviceInfo& info, cudaStream_t stream) {
    const auto kern = few_kernel<ALIGNED, NT>;
    constexpr int smem = kFewWarps * few::Ring<ALIGNED, NT, few_columns(NT)>::WARP_BYTES + few_columns(NT);
    static std::atomic<bool> ready[64] = {};
    if (info.device < 0 || info.device >= 64) return GEMM_ERR_LAUNCH;
    if (!ready[info.device].load(std::memory_order_relaxed)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_LAUNCH;
        }
        ready[info.device].store(true, std::memory_order_relaxed);
    }
    // few row blocks: K over the CTAs of a cluster, four steps a warp at least
    const int64_t blocks = cdiv(p.N, kFewRows32);
    int ctas = 1;
    while (ctas < 8 && 2 * ctas * blocks <= 2 * info.num_sms && p.K >= 2 * ctas * kFewWarps * 64 * 4) ctas *= 2;
    p.ctas = ctas;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1] = pdl_attribute();
    cfg.gridDim = dim3(static_cast<unsigned>(blocks * ctas));
    cfg.blockDim = dim3(kFewWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

template <bool ALIGNED>
int launch_few_tiles(const FewParams& p, const DeviceInfo& info, cudaStream_t stream) {
    if (p.M <= 8) return launch_few<ALIGNED, 1>(p, info, stream);
    return p.M <= 16 ? launch_few<ALIGNED, 2>(p, info, stream) : launch_few<ALIGNED, 4>(p, info, stream);
}

// Rows of bytes at any address in rows ld apart (a multiple of 64), padded with
// zeros: 16 bytes a thread.
__global__ void __launch_bounds__(256)
align_bytes_kernel(const uint8_t* __restrict__ src, uint8_t* __restrict__ dst, int64_t rows, int64_t K, int64_t ld) {
    grid_dependency_wait();
    allow_dependent_launch();
    const int64_t chunks = ld / 16, i = blockIdx.x * 256ll + threadIdx.x;
    if (i >= rows * chunks) return;
    const int64_t row = i / chunks, c = (i - row * chunks) * 16;
    *reinterpret_cast<uint4*>(dst + row * ld + c) = few::load_row<false, false>(src + row * K + c, K - c);
}

// ---------------------------------------------------------------- a batch of tokens

// More tokens than registers hold and fewer than pay for widening b in memory: 128
// rows of b are the tensor core's rows, up to NB tokens (binary16, widened before) its
// columns.  Two groups of eight warps take the stages (two K blocks) in turn: a warp
// copies 32 rows of one K block through a ring of its own, then a lane widens a row in
// registers and writes it into tensor memory, where the multiply takes its left operand.
// One thread copies the tokens, and one for each group multiplies into accumulators of the
// group's own; after 1024 of K all warps add their sums up in integers.  More than 128
// tokens are tiles of 128, each with CTAs of its own.  A cluster's CTAs take a part of K each where row tiles alone would not fill the GPU; integer sums
// are joined exactly.
//
// b's bytes bound it; it takes about twice as long (cold caches, through 16384 x 4096: 32
// tokens 22.3 us, 64 23.7, 128 29.5, where b alone is 10; widening b in memory first takes 58
// to 62).  8 us are the tokens' widening (a launch), the prologue and the joining of sums.  Of the rest the
// issue of multiplies and barriers is the most: a thread takes some 50 clocks a multiply and 100 or
// more for each wait or commit, 1300 a stage, so with one for both groups 32 tokens took 30.1 us
// wherever b was widened to (tensor or shared memory), with an arrival for each K block 33.
constexpr int kBatchWarps = 16;
constexpr int kBatchThreads = (kBatchWarps + 3) * 32;
constexpr int kBatchRows = 128;
constexpr int kStageChunk = kChunk / 2;                 // stages of a chunk, of one group's

template <bool ALIGNED, int NB>
struct Batch {
    static constexpr int PIECE = 32 * 64 + (ALIGNED ? 0 : 32 * 16);                 // a warp's of a stage (ragged: a row's last block)
    static constexpr int STAGES = (NB == 128 ? 2 : 4) + (ALIGNED ? 1 : 0);            // of each warp
    static constexpr int TILE_SLOTS = 4;                                            // b's operand tiles of a stage, in tensor memory
    static constexpr int TOKENS = 2 * NB * 128;                                     // the tokens' of a stage
    // (even numbers of slots: a group's thread then sees every phase of its slots' barriers; of one that the other
    // group fills in between it would take a phase long past for the one that it waits for)
    static constexpr int TOKEN_SLOTS = 4;
    static_assert(TILE_SLOTS % 2 == 0 && TOKEN_SLOTS % 2 == 0, "a slot is one group's");
    static constexpr int OFF_TOKENS = (kBatchWarps * STAGES * PIECE + 1023) / 1024 * 1024;
    static constexpr int OFF_BAR = OFF_TOKENS + TOKEN_SLOTS * TOKENS;
    static constexpr int SMEM = OFF_BAR + 256 + 1024;                               // + slack to align the base to 1024
    static_assert(SMEM <= SMEM_LIMIT, "shared memory");
    static_assert(kBatchRows * NB * 4 <= OFF_BAR, "the sums fit where the copies were");
    // tensor memory: each group's accumulators, one or two in 128 columns, then the tiles, 64 columns each
    static constexpr int BUFFERS = NB == 128 ? 1 : 2, TILES_AT = 256, TILE = 64;
    static constexpr int acc(int group, int buffer) { return 128 * group + 64 * buffer; }
    static_assert(TILES_AT + TILE_SLOTS * TILE <= 512 && NB * BUFFERS <= 128, "tensor memory");
};

struct BatchParams {
    const uint8_t* b;               // [N, K]
    const float* a_scale;
    const float* b_scale;
    uint16_t* out;                  // [M, N]
    int64_t N;
    int M, K, ctas, bf16, token_tiles;
    unsigned flags;
    unsigned long long timeout_ns;
    unsigned* status;
};

template <bool ALIGNED, int NB>
__global__ void __launch_bounds__(kBatchThreads, 1)
batch_kernel(const __grid_constant__ CUtensorMap tokens, const __grid_constant__ BatchParams p) {
    using L = Batch<ALIGNED, NB>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t* const gbase = smem_raw + (base - raw);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_ctarank();
    // b's tiles' and the tokens' full and empty barriers, the accumulators' (buffer b of group g: b 2 + g)
    const uint32_t bFULL = base + L::OFF_BAR, bEMPTY = bFULL + 8 * L::TILE_SLOTS;
    const uint32_t tFULL = bEMPTY + 8 * L::TILE_SLOTS, tEMPTY = tFULL + 8 * L::TOKEN_SLOTS;
    const uint32_t bTFULL = tEMPTY + 8 * L::TOKEN_SLOTS, bTEMPTY = bTFULL + 16 * L::BUFFERS;
    const uint32_t bDRAIN = bTEMPTY + 16 * L::BUFFERS, sTMEM = bDRAIN + 16, sABORT = sTMEM + 4;
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(gbase + (sABORT - base));

    if (threadIdx.x == 0) {
        for (int s = 0; s < L::TILE_SLOTS; ++s) {
            mbar_init(bFULL + 8 * s, kBatchWarps / 2);
            mbar_init(bEMPTY + 8 * s, 1);
        }
        for (int s = 0; s < L::TOKEN_SLOTS; ++s) {
            mbar_init(tFULL + 8 * s, 1);
            mbar_init(tEMPTY + 8 * s, 1);
        }
        for (int i = 0; i < 2 * L::BUFFERS; ++i) {
            mbar_init(bTFULL + 8 * i, 1);
            mbar_init(bTEMPTY + 8 * i, kBatchWarps);
        }
        for (int g = 0; g < 2; ++g) mbar_init(bDRAIN + 8 * g, 1);
        *abort_flag = 0u;
        fence_mbar_init();
        tma_prefetch_desc(&tokens);
    }
    if (warp == kBatchWarps + 1) {
        tmem_alloc<1>(sTMEM, 512);
        tmem_relinquish<1>();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *reinterpret_cast<uint32_t*>(gbase + (sTMEM - base));

    // this CTA's K blocks (an even number, but for the last part's) and stages of two
    const int nkb = (p.K + BK - 1) / BK, per = ((nkb + p.ctas - 1) / p.ctas + 1) / 2 * 2;
    const int kb0 = min(nkb, static_cast<int>(rank) * per), count = min(nkb - kb0, per);
    // (a row tile's token tiles lie side by side: its rows come from memory once)
    const unsigned tile = blockIdx.x / static_cast<unsigned>(p.ctas), tiles = static_cast<unsigned>(p.token_tiles);
    const int64_t row0 = static_cast<int64_t>(tile / tiles) * kBatchRows;
    const int token0 = static_cast<int>(tile % tiles) * NB;
    const int stages = (count + 1) / 2;
    const auto stages_of = [&](int group) { return (stages - group + 1) / 2; };         // group, group + 2, ..
    const auto chunks_of = [&](int group) { return (stages_of(group) + kStageChunk - 1) / kStageChunk; };
    int sums[NB / 4];
#pragma unroll
    for (int i = 0; i < NB / 4; ++i) sums[i] = 0;
    bool ok = true;

    if (warp < kBatchWarps) {
        // ======================================================== copies and widening of b, sums
        const Waiter W{p.timeout_ns, abort_flag, p.status, kStatusRoleProducer};
        // group warp / 8, K block warp / 4 % 2 of a stage, rows 32 (warp % 4) .. (the lanes this warp may write)
        const int group = warp / (kBatchWarps / 2), block = warp / 4 % 2, rows = warp % 4 * 32;
        // a lane copies 16 bytes at 16 c of rows r, r + 8, r + 16 and r + 24
        const int c = lane % 4, r = lane / 4;
        const int mine = stages_of(group);
        const uint32_t ring = base + warp * (L::STAGES * L::PIECE);
        const int k0 = (kb0 + 2 * group + block) * BK;          // of its first K block
        const uint8_t* at[4];
        int left = p.K - k0 - 16 * c;                           // of a row, from the lane's 16 bytes on
#pragma unroll
        for (int j = 0; j < 4; ++j) at[j] = p.b + min(row0 + rows + r + 8 * j, p.N - 1) * p.K + k0 + 16 * c;
        // (blocks trade places in a row so that 32 lanes' reads of a row each, and a copy's writes, share no banks)
        const auto place = [](int row, int block16) { return row * 64 + ((block16 ^ (row >> 1 & 3)) << 4); };
        int filled = 0, fill_stage = 0, read_stage = 0;
        const auto fill = [&]() {
            if (filled < mine) {
                const uint32_t to = ring + fill_stage * L::PIECE;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int off = ALIGNED ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(at[j]) & 15u);
                    // (few.cuh's ragged rows: blocks from the one below on, as far as they hold bytes of the row)
                    if (left > -off) cp_async<16>(to + place(r + 8 * j, c), at[j] - off, 16u);
                    if (!ALIGNED && c == 3 && left > 16 - off) cp_async<16>(to + 2048 + (r + 8 * j) * 16, at[j] - off + 16, 16u);
                    at[j] += 4 * BK;
                }
                left -= 4 * BK;
                ++filled;
            }
            cp_async_commit();
            if (++fill_stage == L::STAGES) fill_stage = 0;
        };
        // this lane's own row, as it is widened
        int row_left = p.K - k0;
        const uint32_t shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p.b + min(row0 + rows + lane, p.N - 1) * p.K + k0) & 15u);
#pragma unroll
        for (int i = 0; i < L::STAGES - 1; ++i) fill();

        // the sums of chunk i of both groups: lane quarter warp % 4, quarter warp / 4 of the columns
        const auto add_up = [&](int i) {
            const int b = i % L::BUFFERS;
            for (int g = 0; g < 2; ++g) {
                if (i >= chunks_of(g)) continue;
                bool got = lane == 0 ? W.wait(bTFULL + 8 * (2 * b + g), i / L::BUFFERS & 1) : true;
                got = __shfl_sync(0xffffffffu, got, 0);
                if (!got) return false;
                tc_fence_after_sync();
                const uint32_t from = tmem_base + (static_cast<uint32_t>(warp % 4 * 32) << 16) + L::acc(g, b) + warp / 4 * (NB / 4);
#pragma unroll
                for (int k = 0; k < NB / 4; k += 8) {
                    uint32_t v[8];
                    tmem_ld_32x32b_x8(from + k, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int x = 0; x < 8; ++x) sums[k + x] += __float2int_rn(__uint_as_float(v[x]));
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(bTEMPTY + 8 * (2 * b + g));
            }
            return true;
        };
        int added = 0;
        for (int i = 0; ok && i < mine; ++i) {
            const int st = 2 * i + group, slot = st % L::TILE_SLOTS;
            cp_async_wait_group<L::STAGES - 2>();
            bool got = lane == 0 ? W.wait(bEMPTY + 8 * slot, st / L::TILE_SLOTS & 1) : true;
            got = __shfl_sync(0xffffffffu, got, 0);
            __syncwarp();                                       // (every lane's copies have landed, and are seen)
            if (!got) { ok = false; break; }
            tc_fence_after_sync();
            const uint32_t stage = ring + read_stage * L::PIECE;
            uint32_t v[32];
            uint4 w[ALIGNED ? 4 : 5];
#pragma unroll
            for (int q = 0; q < 4; ++q) ld_shared_v4(stage + place(lane, q), w[q].x, w[q].y, w[q].z, w[q].w);
            if constexpr (!ALIGNED) ld_shared_v4(stage + 2048 + lane * 16, w[4].x, w[4].y, w[4].z, w[4].w);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint4 x = w[q];
                if constexpr (!ALIGNED) x = few::shifted(x, w[q + 1], shift);
                if (row_left < BK) x = few::cleared(x, row_left - 16 * q);      // (K's last block)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t pairs[4];
                    few::widen<few::kI8Half>(x, half, pairs);
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[8 * q + 4 * half + k] = pairs[k];
                }
            }
            row_left -= 4 * BK;
            tmem_st_32x32b_x32(tmem_base + (static_cast<uint32_t>(rows) << 16) + L::TILES_AT + slot * L::TILE + block * (L::TILE / 2), v);
            tmem_st_wait();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bFULL + 8 * slot);
            if (++read_stage == L::STAGES) read_stage = 0;
            fill();
            // a chunk widened: with two accumulators the one before it has been multiplied, or soon; with
            // one the next cannot begin before this one's sums are taken
            if ((i + 1) % kStageChunk == 0 && (i + 1) / kStageChunk >= L::BUFFERS) ok = add_up(added++);
        }
        cp_async_wait_group<0>();
        for (; ok && added < chunks_of(0); ++added) ok = add_up(added);
    } else if (warp == kBatchWarps) {
        // ======================================================== copies of the tokens
        // The kernel before widens them; this one starts once that one's own wait is over, so b is
        // there already, in L2, where its copies go (ptx.cuh), and only this warp waits.
        grid_dependency_wait();
        allow_dependent_launch();
        if (lane == 0) {
            const Waiter W{p.timeout_ns, abort_flag, p.status, kStatusRoleProducer};
            int armed = 0;
            for (; armed < stages; ++armed) {
                const int st = armed, slot = st % L::TOKEN_SLOTS, pair = min(2, count - 2 * st);
                if (!W.wait(tEMPTY + 8 * slot, st / L::TOKEN_SLOTS & 1)) break;
                mbar_arrive_expect_tx(tFULL + 8 * slot, pair * (L::TOKENS / 2));
                for (int k = 0; k < pair; ++k)
                    tma_load_2d(base + L::OFF_TOKENS + slot * L::TOKENS + k * (L::TOKENS / 2), &tokens, (kb0 + 2 * st + k) * BK, token0,
                                tFULL + 8 * slot);
            }
            // Copies in flight into this CTA land before it may end.  A slot that was armed last is not armed again, so its
            // phase is there to be seen, whichever role gave up and however short the limit is.
            volatile uint32_t no_abort = 0;
            const Waiter D{max(p.timeout_ns, kDrainNs), &no_abort, p.status, kStatusRoleProducer};
            for (int st = max(0, armed - L::TOKEN_SLOTS); st < armed; ++st)
                if (!D.wait(tFULL + 8 * (st % L::TOKEN_SLOTS), st / L::TOKEN_SLOTS & 1)) break;
        }
        __syncwarp();
    } else {
        // ======================================================== multiplies, a warp each group's stages
        const int group = warp - kBatchWarps - 1;
        if (lane == 0) {
            const Waiter W{p.timeout_ns, abort_flag, p.status, kStatusRoleMma};
            if (group == 0 && !(p.flags & GEMM_DEBUG_SKIP_EMPTY_SEED)) {
                // every slot starts empty
                for (int s = 0; s < L::TILE_SLOTS; ++s) mbar_arrive(bEMPTY + 8 * s);
                for (int s = 0; s < L::TOKEN_SLOTS; ++s) mbar_arrive(tEMPTY + 8 * s);
            }
            const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(NB >> 3) << 17) | (static_cast<uint32_t>(kBatchRows >> 4) << 24);
            const int mine = stages_of(group);
            bool issued = false;
            for (int i = 0; i < mine; ++i) {
                const int st = 2 * i + group, chunk = i / kStageChunk, b = chunk % L::BUFFERS, pair = min(2, count - 2 * st);
                const int slot = st % L::TILE_SLOTS, tslot = st % L::TOKEN_SLOTS;
                const bool first = i % kStageChunk == 0;
                // (the first chunks' accumulators are free)
                if (first && chunk >= L::BUFFERS && !W.wait(bTEMPTY + 8 * (2 * b + group), (chunk / L::BUFFERS - 1) & 1)) { ok = false; break; }
                if (!W.wait(tFULL + 8 * tslot, st / L::TOKEN_SLOTS & 1)) { ok = false; break; }
                if (!W.wait(bFULL + 8 * slot, st / L::TILE_SLOTS & 1)) { ok = false; break; }
                tc_fence_after_sync();
                for (int k = 0; k < pair; ++k) {
                    const uint32_t ad = tmem_base + L::TILES_AT + slot * L::TILE + k * (L::TILE / 2);
                    const uint64_t bd = operand_desc(base + L::OFF_TOKENS + tslot * L::TOKENS + k * (L::TOKENS / 2), false);
#pragma unroll
                    for (int x = 0; x < BK / UMMA_K; ++x)
                        tc_mma_f16_tmem_a(tmem_base + L::acc(group, b), ad + x * (UMMA_K / 2), bd + x * k_step(false), idesc,
                                          !first || k != 0 || x != 0);
                }
                issued = true;
                tc_commit_1(bEMPTY + 8 * slot);
                tc_commit_1(tEMPTY + 8 * tslot);
                if (i == mine - 1 || i % kStageChunk == kStageChunk - 1) tc_commit_1(bTFULL + 8 * (2 * b + group));
            }
            if (issued) {
                // all multiplies have finished before tensor memory is released
                tc_commit_1(bDRAIN + 8 * group);
                volatile uint32_t no_abort = 0;
                const Waiter D{max(p.timeout_ns, kDrainNs), &no_abort, p.status, kStatusRoleMma};
                D.wait(bDRAIN + 8 * group, 0);
            }
        }
        __syncwarp();
    }

    // the sums, [NB][128], where the copies were
    tc_fence_before_sync();
    __syncthreads();
    const bool alive = *abort_flag == 0u;
    int* const shared_sums = reinterpret_cast<int*>(gbase);
    if (warp < kBatchWarps) {
        const int n = warp % 4 * 32 + lane, first = warp / 4 * (NB / 4);
#pragma unroll
        for (int i = 0; i < NB / 4; ++i) shared_sums[(first + i) * kBatchRows + n] = sums[i];
    }
    __syncthreads();
    if (p.ctas > 1) cluster_sync();
    // CTA r of a cluster takes every ctas-th token; a thread two rows of b side by side
    const bool pairs = p.N % 2 == 0 && (reinterpret_cast<uintptr_t>(p.out) & 3u) == 0;
    for (int i = threadIdx.x; alive && i < NB / p.ctas * (kBatchRows / 2); i += kBatchThreads) {
        const int m = i / (kBatchRows / 2) * p.ctas + static_cast<int>(rank), n = i % (kBatchRows / 2) * 2;
        if (token0 + m >= p.M || row0 + n >= p.N) continue;
        const bool both = row0 + n + 1 < p.N;
        int s0 = 0, s1 = 0;
        const uint32_t from = smem_u32(shared_sums + m * kBatchRows + n);
        for (int q = 0; q < p.ctas; ++q) {
            const uint32_t remote = mapa_shared(from, q);
            s0 += static_cast<int>(ld_relaxed_cluster_u32(remote));
            s1 += static_cast<int>(ld_relaxed_cluster_u32(remote + 4));
        }
        const float sa = __ldg(p.a_scale + token0 + m), sb0 = __ldg(p.b_scale + row0 + n), sb1 = both ? __ldg(p.b_scale + row0 + n + 1) : 0.0f;
        const uint32_t v = pack16(i8_value(s0, sa, sb0), i8_value(s1, sa, sb1), p.bf16);
        uint16_t* to = p.out + (token0 + m) * p.N + row0 + n;
        if (pairs) {
            *reinterpret_cast<uint32_t*>(to) = v;
        } else {
            to[0] = static_cast<uint16_t>(v & 0xFFFFu);
            if (both) to[1] = static_cast<uint16_t>(v >> 16);
        }
    }
    __syncthreads();
    if (p.ctas > 1) cluster_sync();             // (no CTA leaves while another reads its sums)
    if (warp == kBatchWarps + 1) {
        tc_fence_after_sync();
        tmem_dealloc<1>(tmem_base, 512);
    }
}

template <bool ALIGNED, int NB>
int launch_batch(const CUtensorMap& tokens, BatchParams p, const DeviceInfo& info, cudaStream_t stream) {
    const auto kern = batch_kernel<ALIGNED, NB>;
    constexpr int smem = Batch<ALIGNED, NB>::SMEM;
    static std::atomic<bool> ready[64] = {};
    if (info.device < 0 || info.device >= 64) return GEMM_ERR_LAUNCH;
    if (!ready[info.device].load(std::memory_order_relaxed)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_LAUNCH;
        }
        ready[info.device].store(true, std::memory_order_relaxed);
    }
    p.token_tiles = static_cast<int>(cdiv(p.M, NB));
    const int64_t tiles = cdiv(p.N, kBatchRows) * p.token_tiles;
    int ctas = 1;
    // (clusters of four find places on 144 of 152 SMs, of eight on 120: with 16 of them a second round,
    // 128 tokens through 2048 x 8192 29.6 us)
    const auto places = [&](int n) { return n == 8 ? info.num_sms * 15 / 19 : n == 4 ? info.num_sms * 18 / 19 : info.num_sms; };
    while (ctas < 8 && 2 * ctas * tiles <= places(2 * ctas) && p.K >= 2 * ctas * 4 * BK) ctas *= 2;
    p.ctas = ctas;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1] = pdl_attribute();
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * ctas));
    cfg.blockDim = dim3(kBatchThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kern, tokens, p) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

// Up to 256 tokens (16384 x 4096 53.8 us, widened in memory 64.8; 4096 x 1024 13.2 and 15.0), and more while
// all tiles run at once and K is long enough for the widening to count (512 tokens through
// 4096 x 4096 28.5 and 30.6 us, through 2048 x 8192 29.1 and 44.3; 384 through 8192 x 8192, more tiles than
// SMs, 89.0 and 80.2; 512 through 4096 x 1024 15.0 and 14.2).  Ragged rows of b go through rings of two
// stages here, whose copies and widening do not overlap: half as many tiles (768 tokens through 1024 x 8200, 48
// tiles, 40.0 and 43.5 us, 512 through 2048 x 8200, 64, 40.1 and 47.4, 768, 96, 65.9 and 48.8; 512 through 4096 x 4104, 128,
// 39.8 and 33.7; up to 256 tokens 16384 x 4104 77.3 and 75.7, 4096 x 4104 26.6 and 32.3, 4096 x 1032 15.0 both).
bool batch_tokens(int64_t M, int64_t N, int64_t K, bool aligned) {
    return M <= 256 || (K >= 2048 && cdiv(N, kBatchRows) * cdiv(M, 128) <= (aligned ? 128 : 64));
}
int batch_columns(int64_t M) { return M <= 32 ? 32 : M <= 64 ? 64 : 128; }

template <bool ALIGNED>
int launch_batch_columns(const CUtensorMap& tokens, const BatchParams& p, const DeviceInfo& info, cudaStream_t stream) {
    switch (batch_columns(p.M)) {
        case 32: return launch_batch<ALIGNED, 32>(tokens, p, info, stream);
        case 64: return launch_batch<ALIGNED, 64>(tokens, p, info, stream);
        default: return launch_batch<ALIGNED, 128>(tokens, p, info, stream);
    }
}

// ---------------------------------------------------------------- product

int check(int64_t M, int64_t N, int64_t K, const void* a, const void* b, const float* sa, const float* sb,
          const void* out, int type) {
    if (bad_size(M) || bad_size(N) || K < 0 || K > kMaxK) return GEMM_ERR_INVALID_ARG;
    if (type != GEMM_TYPE_HALF && type != GEMM_TYPE_BFLOAT) return GEMM_ERR_INVALID_ARG;
    if (too_many_tiles(M, N)) return GEMM_ERR_INVALID_ARG;
    if (odd_address(out) || reinterpret_cast<uintptr_t>(sa) % 4 != 0 || reinterpret_cast<uintptr_t>(sb) % 4 != 0)
        return GEMM_ERR_ALIGNMENT;
    if (M > 0 && N > 0 && K > 0 && (!a || !b)) return GEMM_ERR_INVALID_ARG;
    return GEMM_OK;
}

// Whether rows of K bytes start on 16-byte boundaries.
bool rows16(const void* p, int64_t K) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && K % 16 == 0; }

struct Plan {
    bool few = false;               // a few tokens
    bool batch = false;             // a batch of them
    uint8_t* few_a = nullptr;       // their aligned copy, where they need one
    Product pr;
    Layout l;
    uint16_t *a = nullptr, *b = nullptr;
    int64_t ld = 0;
    size_t bytes = 0;
};

// num_sms 0: the workspace only.
Plan plan_of(int64_t M, int64_t N, int64_t K, const void* a, const void* b, int num_sms, void* ws) {
    Plan pl;
    Carver c;
    c.base = static_cast<char*>(ws);
    pl.ld = round_up(K, 64);
    pl.few = few_tokens(M, N, K);
    if (pl.few) {
        if (!rows16(a, K)) pl.few_a = c.take<uint8_t>(M * pl.ld);
        pl.bytes = c.used;
        return pl;
    }
    pl.a = c.take<uint16_t>(M * pl.ld);
    pl.batch = batch_tokens(M, N, K, rows16(b, K));
    if (pl.batch) {
        pl.bytes = c.used;
        return pl;
    }
    pl.pr.M = M; pl.pr.N = N; pl.pr.K = K;
    pl.pr.chunk = kChunk;
    if (num_sms) pl.l = choose_layout(pl.pr, num_sms);
    pl.b = c.take<uint16_t>(N * pl.ld);
    pl.bytes = c.used;
    return pl;
}

}  // namespace i8
}  // namespace pws

extern "C" int gemm_i8_quantize(int64_t M, int64_t K, const void* x, int8_t* q, float* scale, int type,
                                cudaStream_t stream) {
    using namespace pws;
    using namespace pws::i8;
    if (bad_size(M) || bad_size(K)) return GEMM_ERR_INVALID_ARG;
    if (type != GEMM_TYPE_HALF && type != GEMM_TYPE_BFLOAT) return GEMM_ERR_INVALID_ARG;
    if (odd_address(x) || reinterpret_cast<uintptr_t>(scale) % 4 != 0) return GEMM_ERR_ALIGNMENT;
    if (M == 0) return GEMM_OK;
    if (!scale || (K > 0 && (!x || !q))) return GEMM_ERR_INVALID_ARG;
    const Range in[1] = {{x, bytes16(M, K)}};
    const Range out[2] = {{q, static_cast<uint64_t>(M) * K}, {scale, 4ull * M}};
    if (overlaps(in, out)) return GEMM_ERR_INVALID_ARG;
    DeviceInfo info;
    const int rc = current_device(&info);
    if (rc != GEMM_OK) return rc;
    const bool bf16 = type == GEMM_TYPE_BFLOAT;
    if (K <= 1024)
        return bf16 ? launch_quantize<32, true>(M, K, x, q, scale, stream) : launch_quantize<32, false>(M, K, x, q, scale, stream);
    if (K <= 8192)
        return bf16 ? launch_quantize<256, true>(M, K, x, q, scale, stream) : launch_quantize<256, false>(M, K, x, q, scale, stream);
    return bf16 ? launch_quantize<1024, true>(M, K, x, q, scale, stream) : launch_quantize<1024, false>(M, K, x, q, scale, stream);
}

extern "C" int gemm_i8_nt_workspace(int64_t M, int64_t N, int64_t K, const int8_t* a, const int8_t* b, int type,
                                    int64_t* bytes) {
    using namespace pws::i8;
    const int rc = check(M, N, K, a, b, nullptr, nullptr, nullptr, type);
    if (rc != GEMM_OK) return rc;
    if (!bytes) return GEMM_ERR_INVALID_ARG;
    *bytes = M && N && K ? static_cast<int64_t>(plan_of(M, N, K, a, b, 0, nullptr).bytes) : 0;
    return GEMM_OK;
}

extern "C" int gemm_i8_nt(int64_t M, int64_t N, int64_t K, const int8_t* a, const int8_t* b, const float* a_scale,
                          const float* b_scale, void* out, int type, void* workspace, int64_t workspace_bytes,
                          cudaStream_t stream) {
    using namespace pws;
    using namespace pws::i8;
    int rc = check(M, N, K, a, b, a_scale, b_scale, out, type);
    if (rc != GEMM_OK) return rc;
    if (M == 0 || N == 0) return GEMM_OK;
    if (!out || !a_scale || !b_scale) return GEMM_ERR_INVALID_ARG;
    const Range in[4] = {{a, static_cast<uint64_t>(M) * K}, {b, static_cast<uint64_t>(N) * K}, {a_scale, 4ull * M}, {b_scale, 4ull * N}};
    const Range outs[1] = {{out, bytes16(M, N)}};
    if (overlaps(in, outs)) return GEMM_ERR_INVALID_ARG;
    DeviceInfo info;
    rc = current_device(&info);
    if (rc != GEMM_OK) return rc;
    if (K == 0) return cudaMemsetAsync(out, 0, bytes16(M, N), stream) == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
    Plan pl = plan_of(M, N, K, a, b, info.num_sms, workspace);
    if (!workspace_ok(workspace, workspace_bytes, pl.bytes, in, outs)) return GEMM_ERR_INVALID_ARG;
    if (pl.few) {
        FewParams p = {reinterpret_cast<const uint8_t*>(a), reinterpret_cast<const uint8_t*>(b), a_scale, b_scale,
                       static_cast<uint16_t*>(out), K, N, static_cast<int>(M), static_cast<int>(K), 1, type == GEMM_TYPE_BFLOAT};
        if (!rows16(a, K)) {
            if (launch_pdl(align_bytes_kernel, dim3(static_cast<unsigned>(cdiv(M * pl.ld / 16, 256))), dim3(256), 0, stream, p.a,
                           pl.few_a, M, K, pl.ld) != cudaSuccess) {
                cudaGetLastError();
                return GEMM_ERR_LAUNCH;
            }
            p.a = pl.few_a;
            p.lda = pl.ld;
        }
        return rows16(b, K) ? launch_few_tiles<true>(p, info, stream) : launch_few_tiles<false>(p, info, stream);
    }
    const bool aligned = rows16(a, K) && rows16(b, K);
    {
        // (a batch's b is widened on its way)
        const int64_t rows_b = pl.batch ? 0 : N;
        const Widen w = {{reinterpret_cast<const uint8_t*>(a), reinterpret_cast<const uint8_t*>(b)}, {pl.a, pl.b}, {M, rows_b}};
        int64_t blocks = cdiv((M + rows_b) * cdiv(K, 16), 256);
        if (blocks > (1 << 30)) blocks = 1 << 30;
        if (launch_pdl((pl.batch ? rows16(a, K) : aligned) ? widen_kernel<true> : widen_kernel<false>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
                       stream, w, K, pl.ld) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_LAUNCH;
        }
    }
    if (pl.batch) {
        CUtensorMap tokens;
        if (!encode_tmap_f16_2d(&tokens, pl.a, K, M, pl.ld * 2, BK, batch_columns(M))) return GEMM_ERR_LAUNCH;
        const BatchParams p = {reinterpret_cast<const uint8_t*>(b), a_scale, b_scale, static_cast<uint16_t*>(out), N, static_cast<int>(M),
                               static_cast<int>(K), 1, type == GEMM_TYPE_BFLOAT, 1, debug_flags(), wait_timeout_ns(), status_word(info, stream)};
        return rows16(b, K) ? launch_batch_columns<true>(tokens, p, info, stream) : launch_batch_columns<false>(tokens, p, info, stream);
    }
    Maps maps;
    memset(&maps, 0, sizeof(maps));
    Params p = base_params(pl.l, GEMM_TYPE_HALF, info, stream);
    Operands op;
    op.a[0] = pl.a;
    op.lda = pl.ld;
    op.b[0] = pl.b;
    op.ldb = pl.ld;
    if (!set_job(&p, &maps, 0, pl.pr, pl.l, pl.l.part[0], op)) return GEMM_ERR_LAUNCH;
    p.bf16 = type == GEMM_TYPE_BFLOAT;          // (the output's; the operands are binary16)
    p.a_scale = a_scale;
    p.b_scale = b_scale;
    Job& j = p.job[0];
    j.ld16 = N;
    j.out16[0] = static_cast<uint16_t*>(out);
    j.tma_store = output_map(&maps.c[0], pl.l, out, M, N, N);
    return launch_product<kEpiI8>(pl.l, maps, p, info, stream);
}

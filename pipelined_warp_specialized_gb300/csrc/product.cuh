// product.cuh -- the tensor-core product under the fused operators: a
// persistent, warp-specialized tcgen05 kernel whose operands may be stored
// with K or with rows/columns innermost, and whose epilogue is the model's
// next operation instead of a plain store.
//
//   D[m, n] = sum_k A[m, k] B[n, k]           fp32 in tensor memory
//
//   operands  "K-major" (rows of K elements, as lhs and rhs of gemm_f16_nt) or
//             "MN-major" (K rows of M or N elements): the backward products
//             dx = dy W and dW = dy^T x read the forward pass's matrices as
//             they lie, so nothing is ever transposed in memory.
//   segments  the K axis may run over two operand pairs, one after the other
//             (dx = dg Wg + du Wu is one accumulation).
//   problems  two products of one shape may be one job (dWg and dWu).
//   jobs      two products of different shapes may share a launch (dx and dW):
//             the groups of CTAs that the first job's last wave leaves idle
//             start on the second one's tiles.
//   chunks    the cross entropy's epilogues sum each logit over K in chunks of
//             4 or 8 blocks, each chunk's tensor-memory sum added in
//             registers (round to nearest): the tensor core's own accumulation
//             truncates, which over a long K shifts every logit the same way.
//             Forward and backward take the same chunks, so that z - lse holds
//             no difference between two sums of one logit.  The 8-bit product's
//             takes chunks of 16 blocks, whose sums of whole numbers are exact,
//             and adds them in integers.
//   splits    few output tiles with a long K are split over K; the fp32
//             partial sums are joined in a fixed order by a later kernel, so a
//             result never depends on the order in which CTAs finish.
//
// The pipeline is the one of gemm_f16_nt (TMA producer thread, ring of
// shared-memory slots with full/empty barriers, one MMA-issuing thread,
// double-buffered accumulator, four epilogue warps, bounded waits), with a
// tile width, box height and ring depth chosen at run time: one token's
// product wants slots of 1 KB + a few weight rows and 32 of them in flight, a
// training product wants 256 x 256 on a CTA pair.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"
#include "pwsgemm.h"
#include "waiter.cuh"

namespace pws {
namespace fused {

constexpr int BK = 64;                      // K per ring slot: one 128-byte swizzle row of 16-bit elements
constexpr int UMMA_K = 16;
constexpr int BM_CTA = 128;                 // accumulator rows per CTA (tensor-memory lanes)
constexpr int MAX_BN = 256;                 // accumulator columns per buffer
constexpr int MAX_STAGES = 32;
constexpr int EPI_COLS = 64;                // output columns per staged chunk: 128 bytes
constexpr int EPI_BUF = 32 * EPI_COLS * 2;  // one warp's 32 rows of a chunk
constexpr int EPI_BYTES = 8 * EPI_BUF;
constexpr int MN_BOX = 64 * BK * 2;         // one MN-major box: 64 K rows of 64 elements
constexpr int WIDE_B = 128 * BK * 2;        // the wide tile's B halves in a slot: one CTA's 128 rows each
constexpr int WIDE_STAGES = 4;
constexpr int kWideBlocks = 128;

// Shared memory: ring, epilogue staging, barriers.
constexpr int SMEM_LIMIT = 232448;
constexpr int BAR_BYTES = 1024;
constexpr int RING_BYTES = (SMEM_LIMIT - 1024 - EPI_BYTES - BAR_BYTES) / 1024 * 1024;
constexpr int OFF_EPI = RING_BYTES;
constexpr int OFF_BAR = OFF_EPI + EPI_BYTES;
constexpr int OFF_FULL = OFF_BAR;
constexpr int OFF_EMPTY = OFF_FULL + 8 * MAX_STAGES;
constexpr int OFF_TFULL = OFF_EMPTY + 8 * MAX_STAGES;
constexpr int OFF_TEMPTY = OFF_TFULL + 16;
constexpr int OFF_DRAIN = OFF_TEMPTY + 16;
constexpr int OFF_TMEM = OFF_DRAIN + 8;
constexpr int OFF_ABORT = OFF_TMEM + 4;
constexpr int OFF_PROGRESS = OFF_ABORT + 4;
static_assert(OFF_PROGRESS + 4 <= OFF_BAR + BAR_BYTES, "barriers");
constexpr int SMEM_BYTES = OFF_BAR + BAR_BYTES + 1024;      // + slack to align the base to 1024
static_assert(SMEM_BYTES <= SMEM_LIMIT, "shared memory");
static_assert(SMEM_BYTES > 120 * 1024, "one CTA per SM: each owns all of tensor memory");

// A wait for what is in flight before the CTA may exit outlasts any limit a
// caller sets: copies and multiplies already issued end in microseconds.
constexpr unsigned long long kDrainNs = 100000000ull;

enum Epilogue { kEpiStore = 0, kEpiGated = 1, kEpiXentStats = 2, kEpiXentGrad = 3, kEpiI8 = 4 };

// Epilogue warps: two per tensor-memory lane quarter, which take the tile's
// 64-column chunks (32-column groups for the statistics) in turn, so that the
// epilogue of a short K loop keeps up with the multiplies.
constexpr int EPI_WARPS = 8;
// Producer warps: A's copies and B's (an MN-major operand takes two copies a
// slot, and one thread issuing three or four of them fell behind the
// multiplies), then the MMA issuer.
constexpr int kMmaWarp = 2;
constexpr int THREADS = (kMmaWarp + 1 + EPI_WARPS) * 32;

// K blocks per chunk of the logits' sums, for more rows than a CTA's and for no
// more (whole slots: kMaxBoxes divides them).  For many rows 8 take no
// measurable time (loss of 4096 x 131072 x 4096: 2.53 ms with 8 or 64) and 4 take
// 4 %.  For few rows the product is bound by the weights' bytes, where 4 are
// free, and few losses average no error out.  In the backward pass they take 0
// to 2 % (64 tokens over 131072 x 4096 581 to 588 us).
constexpr int kLogitsChunk = 8;
constexpr int kLogitsChunkFew = 4;
constexpr int kMaxBoxes = 4;
static_assert(kLogitsChunk % kMaxBoxes == 0 && kLogitsChunkFew % kMaxBoxes == 0, "a chunk ends with a slot");

// One product of a launch.
struct Job {
    int M, N;                       // output rows and columns
    int nkb0, nkb;                  // K blocks of the first segment, of all segments
    int tiles_m, tiles_n, num_tiles;    // tiles of one problem; num_tiles counts all problems
    int kb_per_split;
    int units;                      // num_tiles * splits
    int amn;                        // A is MN-major
    int a_map, b_map, c_map;        // a_map + 2 * problem + segment, b_map + b_seg * segment, c_map + problem
    int b_seg;                      // 1: each K segment has its own B; 0: one for both
    int tma_store;
    uint32_t idesc;
    // out = scale * acc, to 16 bits (out16), or to fp32 (out32, partial sums:
    // split s of problem i at out32 + s * split_stride + i * problem_stride),
    // plus acc_in
    uint16_t* out16[2];
    int64_t ld16;
    float* out32;
    const float* acc_in;
    int64_t ld32, split_stride, problem_stride;
    const float* scale;             // device scalar, or null for 1
};

struct Params {
    Job job[2];                     // job[1].units == 0: one job
    int extra_rounds;               // schedule of the second job's units (Schedule)
    int chunk;                      // K blocks per accumulator hand-over
    int bn;                         // accumulator columns per tile (a multiple of 16)
    int tile_n;                     // output columns per tile (bn, or bn / 2 for the gated epilogue)
    int stages, boxes;              // ring slots, K blocks in each
    int a_bytes, box_bytes, slot_bytes;
    int tx_bytes;                   // bytes one CTA's copies bring per K block
    int bf16;                       // output type
    int act;
    unsigned flags;                 // GEMM_DEBUG_SKIP_EMPTY_SEED is honoured
    unsigned long long timeout_ns;
    unsigned* status;
    // kEpiGated: h = act(gate) * up to out16[0], and gate, up where g_out is not null
    uint16_t* g_out;
    uint16_t* u_out;
    // cross entropy
    const int64_t* target;
    float2* stats;                  // [M][2 tiles_n]: maximum and sum of exponentials of half a tile's columns
    float* z_target;                // [M]
    const float* lse;
    const float* coef;              // [M]: scaled loss gradient
    int64_t ignore_index;           // a target of a row that does not count: D is 0 there
    int64_t col0;                   // vocabulary index of column 0
    int64_t lo_offset;              // elements from D to its rounding remainder, 0 for none
    // kEpiI8: out16[0] = (whole-number sum) a_scale[row] b_scale[column]
    const float* a_scale;
    const float* b_scale;
};

struct Maps {
    CUtensorMap a[6], b[3], c[3];
};

// The units a group of CTAs (of `groups`) runs, in order.  The first job's are
// dealt round by round.  Its last round leaves groups rest .. groups - 1 with a
// unit less, so the second job's first extra_rounds rounds go to those alone,
// then its rounds go to all, those groups first.
struct Schedule {
    int group, groups, units0, units1, rest, extra;
    int i = 0, k = 0;
    __device__ __forceinline__ Schedule(const Params& p, int g, int n)
        : group(g), groups(n), units0(p.job[0].units), units1(p.job[1].units), rest(p.job[0].units % n),
          extra(p.extra_rounds) {}
    __device__ __forceinline__ bool next(int& job, int& unit) {
        job = 0;
        unit = i * groups + group;
        if (unit < units0) {
            ++i;
            return true;
        }
        job = 1;
        const int late = group >= rest ? group - rest : group + groups - rest;
        if (group >= rest && k < extra) unit = k * (groups - rest) + late;
        else unit = extra * (groups - rest) + (k - (group >= rest ? extra : 0)) * groups + late;
        ++k;
        return unit < units1;
    }
};

// K-major operand in the 128-byte swizzle: rows of 128 bytes, 8-row atoms
// 1024 bytes apart (stride offset).
// MN-major operand: a box is 64 K rows of 128 bytes (64 elements of M or N);
// 8 K rows form an atom, atoms 1024 bytes apart along K (stride offset), boxes
// 8192 bytes apart along M or N (leading offset).
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr, bool mn) {
    uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>((mn ? MN_BOX : 16) >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

// (address >> 4) step of one UMMA_K: 32 bytes inside the swizzle row, or 16 K rows.
__device__ __forceinline__ uint32_t k_step(bool mn) { return (mn ? UMMA_K * 128 : UMMA_K * 2) >> 4; }

struct Tile {
    int problem, tm, tn, kb0, kb1, split;
};

// The K blocks of unit u.
__device__ __forceinline__ void k_range(uint32_t u, const Job& job, Tile& t) {
    t.split = job.units == job.num_tiles ? 0 : u / static_cast<uint32_t>(job.num_tiles);
    t.kb0 = t.split * job.kb_per_split;
    t.kb1 = min(job.nkb, t.kb0 + job.kb_per_split);
}

template <uint32_t GROUP_M>
__device__ __forceinline__ Tile tile_of(uint32_t u, const Job& job) {
    Tile t;
    k_range(u, job, t);
    uint32_t r = u - t.split * static_cast<uint32_t>(job.num_tiles);
    const uint32_t tiles_n = job.tiles_n, tiles_m = job.tiles_m, per = tiles_m * tiles_n;
    t.problem = r >= per ? 1 : 0;
    r -= t.problem * per;
    // tile rows are walked GROUP_M at a time and odd groups right to left, so
    // the CTAs at work share A and B strips in L2
    const uint32_t group = GROUP_M * tiles_n;
    const uint32_t g = r / group;
    const uint32_t first = g * GROUP_M, v = r - g * group;
    const uint32_t rows = min(tiles_m - first, GROUP_M);
    const uint32_t col = rows == GROUP_M ? v / GROUP_M : v / rows;
    t.tm = static_cast<int>(first + v - col * rows);
    t.tn = static_cast<int>(g & 1 ? tiles_n - 1 - col : col);
    return t;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2e = 1.4426950408889634f;

// exp(x - ref).  The difference comes first: it is exact where x is near ref, which
// the fused x log2 e - round(ref log2 e) is not (at 100 it is off by 5e-6).
__device__ __forceinline__ float exp_from(float x, float ref) { return ex2((x - ref) * kLog2e); }

// Both activations are g * sigma(s(g)): silu with s = g, gelu (tanh form)
// with s = 2 sqrt(2/pi) (g + 0.044715 g^3), since (1 + tanh y) / 2 = sigma(2 y).
constexpr float kGeluC = 1.5957691216057308f;       // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

__device__ __forceinline__ float sigmoid(float s) { return __fdividef(1.0f, 1.0f + ex2(-kLog2e * s)); }

__device__ __forceinline__ float act_arg(float g, int act) {
    return act == GEMM_ACT_SILU ? g : kGeluC * g * (1.0f + kGeluA * g * g);
}

__device__ __forceinline__ float act_value(float g, int act) { return g * sigmoid(act_arg(g, act)); }

// act(g) and act'(g) = sigma + g sigma (1 - sigma) s'(g)
__device__ __forceinline__ void act_value_slope(float g, int act, float& value, float& slope) {
    const float s = sigmoid(act_arg(g, act));
    value = g * s;
    const float t = value * (1.0f - s);
    const float ds = act == GEMM_ACT_SILU ? 1.0f : kGeluC * (1.0f + 3.0f * kGeluA * g * g);
    slope = s + (t == 0.0f ? 0.0f : t * ds);        // (a saturated gate's s' may overflow)
}

// 16 bytes at any 2-byte alignment: the one or two aligned 16-byte blocks that
// hold them (each holds at least one of the bytes, so no load leaves their
// pages), shifted into place.
__device__ __forceinline__ uint4 load_unaligned16(const uint16_t* src) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(src);
    const uint32_t sh = static_cast<uint32_t>(at & 15u);
    const uint4* blk = reinterpret_cast<const uint4*>(at - sh);
    const uint4 lo = __ldg(blk);
    if (sh == 0) return lo;
    const uint4 hi = __ldg(blk + 1);
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    const uint32_t q = sh >> 2, bits = (sh & 3u) * 8u;
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = q == 0 ? w[i] : q == 1 ? w[i + 1] : q == 2 ? w[i + 2] : w[i + 3];
        const uint32_t b = q == 0 ? w[i + 1] : q == 1 ? w[i + 2] : q == 2 ? w[i + 3] : w[i + 4];
        v[i] = __funnelshift_r(a, b, bits);
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}

__device__ __forceinline__ uint32_t pack16(float lo, float hi, int bf16) {
    if (bf16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ float2 unpack16(uint32_t v, int bf16) {
    if (bf16) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// An element of the 8-bit product from its sum of whole numbers.  The scales one
// after the other: their product could leave fp32's range where the element does
// not.  A whole number times a scale loses nothing to underflow (it is a multiple of
// fp32's smallest value where it is below the normal range), and overflows with a scale
// of 2^97 or more: such a one comes last.
__device__ __forceinline__ float i8_value(int sum, float a_scale, float b_scale) {
    const bool b_first = fabsf(a_scale) > 0x1p90f;
    return static_cast<float>(sum) * (b_first ? b_scale : a_scale) * (b_first ? a_scale : b_scale);
}

// What rounding to 16 bits left of d, for a second 16-bit value beside it; 0
// where the rounded value is not finite (inf - inf would make it NaN).
__device__ __forceinline__ float remainder16(float d, float rounded) {
    return fabsf(rounded) <= 3.4e38f ? d - rounded : 0.0f;
}

// NW = 2, the wide tile (256 x 512, a CTA pair's): each slot carries two B
// halves, whose accumulators are the two buffers, so an A slot written once
// feeds twice the multiplies.  Shared memory bounds the 256 x 256 tile: a K
// block's multiplies read 12 KB per 128 clocks of it while 32 KB are written,
// 80 KB at 128 bytes a clock (648 clocks measured, its multiplies take 512).
// The buffers are then not free to overlap two units, so it is for backward
// products of at least kWideBlocks K blocks a unit.  Measured, wide against
// 256 x 256: gated backward 8192 x 8192 x 4096 (256 and 128 blocks) 1348
// against 1405 us; a product of 64 blocks 579 against 555; of 12, 43 against 36.

// kEpiStore serves the backward products, whose B is MN-major; the others are
// forward (NT) products.
template <int CG, int EPI, int NW>
__global__ void __launch_bounds__(THREADS, 1)
product_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
    static_assert(NW == 1 || (CG == 2 && EPI == kEpiStore), "the wide tile is a CTA pair's, for plain stores");
    constexpr bool BMN = EPI == kEpiStore;
    // Tile rows walked together, so that their A strips stay in L2 while B
    // streams by.  Forward products, whose B is the weights: with 16 the head's
    // 131072 rows are read once for 4096 tokens (2436 us; 2520 with 8, 2591 with
    // 4).  Backward products: 8 (8192 x 4096 x 8192 643 us; 651 with 16).
    constexpr uint32_t GROUP_M = EPI == kEpiStore ? 8 : 16;
    // slots of several K blocks, for the narrow tiles of few rows
    constexpr bool MULTI = CG == 1 && EPI != kEpiStore;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;       // swizzle atoms are 1024-byte aligned
    uint8_t* const gbase = smem_raw + (base - raw);
    const int warp = threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
    const int group_id = blockIdx.x / CG;
    const int num_groups = gridDim.x / CG;
    const uint32_t bFULL = base + OFF_FULL, bEMPTY = base + OFF_EMPTY;
    const uint32_t bTFULL = base + OFF_TFULL, bTEMPTY = base + OFF_TEMPTY, bDRAIN = base + OFF_DRAIN;
    const uint32_t sPROGRESS = base + OFF_PROGRESS;
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(gbase + OFF_ABORT);
    const uint32_t S = NW == 2 ? WIDE_STAGES : static_cast<uint32_t>(p.stages);

    // ------------------------------------------------------------ set-up
    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < S; ++s) {
            mbar_init(bFULL + 8 * s, 1);
            mbar_init(bEMPTY + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bTFULL + 8 * b, 1);
            mbar_init(bTEMPTY + 8 * b, EPI_WARPS * CG);
        }
        mbar_init(bDRAIN, 1);
        *abort_flag = 0u;
        *reinterpret_cast<volatile uint32_t*>(gbase + OFF_PROGRESS) = 0u;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&maps.a[0]);
        tma_prefetch_desc(&maps.b[0]);
    }
    if (warp == kMmaWarp) {
        tmem_alloc<CG>(base + OFF_TMEM, 512);
        tmem_relinquish<CG>();
    }
    tc_fence_before_sync();
    __syncthreads();
    if (CG == 2) cluster_sync();
    tc_fence_after_sync();
    const uint32_t tmem_base = *reinterpret_cast<uint32_t*>(gbase + OFF_TMEM);
    // everything above overlaps the previous grid's tail; global memory is
    // touched only once that grid has completed
    grid_dependency_wait();
    allow_dependent_launch();
    const bool leader = CG == 1 || rank == 0;

    if (warp < kMmaWarp) {
        // ======================================================== producers
        if (lane == 0) {
            const bool for_a = warp == 0;
            const Waiter W{p.timeout_ns, abort_flag, p.status, kStatusRoleProducer};
            const uint32_t full_leader = CG == 2 ? mapa_shared(bFULL, 0) : bFULL;
            const bool arm = for_a && leader;
            const uint32_t tx = static_cast<uint32_t>(CG * p.tx_bytes), slot = static_cast<uint32_t>(p.slot_bytes);
            const int boxes = MULTI ? p.boxes : 1;
            const uint32_t box = static_cast<uint32_t>(p.box_bytes);
            const uint32_t dst0 = base + (for_a ? 0u : static_cast<uint32_t>(p.a_bytes));
            uint32_t stage = 0, phase = 0, issued = 0, dst = dst0;
            bool ok = true;
            auto load = [&](uint32_t to, const CUtensorMap* map, int x, int y, uint32_t bar) {
                if constexpr (CG == 1) tma_load_2d(to, map, x, y, bar);
                else tma_load_2d_pair(to, map, x, y, bar);
            };
            // `count` K blocks from element k on, `boxes` of them to a slot:
            // copy(the block's operand in the slot, the slot's full barrier, k).
            auto stream = [&](int count, int k, auto copy) {
                while (count > 0) {
                    const int n = min(count, boxes);
                    count -= n;
                    if (!W.wait(bEMPTY + 8 * stage, phase)) return false;
                    if (arm) mbar_arrive_expect_tx(bFULL + 8 * stage, static_cast<uint32_t>(n) * tx);
                    uint32_t to = dst;
                    for (int i = 0; i < n; ++i, to += box, k += BK) copy(to, full_leader + 8 * stage, k);
                    ++issued;
                    if (for_a) st_volatile_shared_u32(sPROGRESS, issued);
                    dst += slot;
                    if (++stage == S) { stage = 0; phase ^= 1u; dst = dst0; }
                }
                return true;
            };
            Schedule sched(p, group_id, num_groups);
            for (int jn, u; ok && sched.next(jn, u);) {
                const Job& job = p.job[jn];
                const Tile t = tile_of<GROUP_M>(u, job);
                // the unit's blocks of the first K segment, then of the second
                const int nkb0 = job.nkb0;
                for (int seg = 0; ok && seg < 2; ++seg) {
                    const int first = seg ? max(t.kb0, nkb0) : t.kb0, last = seg ? t.kb1 : min(t.kb1, nkb0);
                    const int count = last - first, k0 = (first - (seg ? nkb0 : 0)) * BK;
                    if (count <= 0) continue;
                    if (for_a) {
                        const CUtensorMap* map = &maps.a[job.a_map + 2 * t.problem + seg];
                        const int m = t.tm * (BM_CTA * CG) + static_cast<int>(rank) * BM_CTA;
                        if (BMN && job.amn) {
                            ok = stream(count, k0, [&](uint32_t to, uint32_t bar, int k) {
                                load(to, map, m, k, bar);
                                load(to + MN_BOX, map, m + 64, k, bar);
                            });
                        } else {
                            ok = stream(count, k0, [&](uint32_t to, uint32_t bar, int k) { load(to, map, k, m, bar); });
                        }
                    } else if constexpr (EPI == kEpiGated) {
                        // gate rows are the first half of the tile's columns, up rows the second
                        const int n = t.tn * p.tile_n;
                        if constexpr (CG == 2) {
                            const CUtensorMap* map = &maps.b[rank];
                            ok = stream(count, k0, [&](uint32_t to, uint32_t bar, int k) { load(to, map, k, n, bar); });
                        } else {
                            const uint32_t half = static_cast<uint32_t>(p.tile_n) * 128;
                            ok = stream(count, k0, [&](uint32_t to, uint32_t bar, int k) {
                                load(to, &maps.b[0], k, n, bar);
                                load(to + half, &maps.b[1], k, n, bar);
                            });
                        }
                    } else {
                        const int b_rows = p.bn / CG;                    // B rows (accumulator columns) of this CTA
                        const int n = t.tn * NW * p.tile_n + static_cast<int>(rank) * b_rows, n2 = n + p.tile_n;
                        const CUtensorMap* map = &maps.b[job.b_map + job.b_seg * seg];
                        if (BMN && b_rows == 128) {
                            ok = stream(count, k0, [&](uint32_t to, uint32_t bar, int k) {
                                load(to, map, n, k, bar);
                                load(to + MN_BOX, map, n + 64, k, bar);
                                if (NW == 2) {
                                    load(to + WIDE_B, map, n2, k, bar);
                                    load(to + WIDE_B + MN_BOX, map, n2 + 64, k, bar);
                                }
                            });
                        } else if constexpr (BMN) {
                            ok = stream(count, k0, [&](uint32_t to, uint32_t bar, int k) {
                                for (int j = 0; j < b_rows; j += 64) load(to + j * (MN_BOX / 64), map, n + j, k, bar);
                            });
                        } else {
                            ok = stream(count, k0, [&](uint32_t to, uint32_t bar, int k) { load(to, map, k, n, bar); });
                        }
                    }
                }
            }
            if (!ok && leader && for_a) {
                // drain: wait (bounded) for the copies still in flight into this CTA
                volatile uint32_t no_abort = 0;
                const Waiter D{max(p.timeout_ns, kDrainNs), &no_abort, p.status, kStatusRoleProducer};
                const uint32_t first = issued > S ? issued - S : 0u;
                for (uint32_t it = first; it < issued; ++it)
                    if (!D.wait(bFULL + 8 * (it % S), (it / S) & 1u)) break;
            } else if (!ok && issued > 0) {
                // a pair's peer cannot wait on the leader's barriers, nor B's
                // producer on a slot that A's has not armed: copies land within
                // microseconds, so a bounded millisecond outlasts them
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
            }
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ======================================================== MMA issuer
        if (lane == 0 && !(p.flags & GEMM_DEBUG_SKIP_EMPTY_SEED))
            for (uint32_t s = 0; s < S; ++s) mbar_arrive(bEMPTY + 8 * s);      // every slot starts empty
        if (leader && lane == 0) {
            const Waiter W{p.timeout_ns, abort_flag, p.status, kStatusRoleMma};
            // Descriptors of slot s: slot 0's plus s slots.  Addresses lie below
            // 256 KB, so the 14-bit address field never carries and the sum is
            // taken in the low words alone.
            const uint32_t slot16 = static_cast<uint32_t>(p.slot_bytes) >> 4;
            const uint64_t bdesc0 = operand_desc(base + p.a_bytes, BMN);
            const uint32_t box16 = static_cast<uint32_t>(p.box_bytes) >> 4;
            const int chunk = p.chunk, boxes = MULTI ? p.boxes : 1;
            auto desc = [](uint32_t lo, uint64_t of) { return (of & 0xFFFFFFFF00000000ull) | lo; };
            uint32_t stage = 0, phase = 0, tcount = 0, off = 0;
            bool ok = true, issued_any = false;
            // One unit's multiplies.  The A operand's form is a compile-time
            // constant: the issuing thread's own instructions between
            // multiplies idle the tensor pipe (descriptor steps computed at
            // run time cost 14 % at 8192 x 4096 x 8192).
            auto unit = [&](const Tile& t, uint32_t idesc, auto a_mn) {
                constexpr bool AMN = decltype(a_mn)::value;
                const uint64_t adesc0 = operand_desc(base, AMN);
                if constexpr (NW == 2) {
                    // The K blocks of a group of J at both ends of a unit run
                    // half 0 and then half 1 on the same, still held, slots: the
                    // epilogue drains half 0 while the tensor pipe finishes
                    // half 1, and half 1 while half 0 of the next unit starts.
                    // Straight-line code: J and the slot size are constants.
                    constexpr uint32_t J = WIDE_STAGES - 1, SLOT = (BM_CTA * 128 + 2 * WIDE_B) >> 4;
                    const int nkb = t.kb1 - t.kb0;
                    const uint32_t aph = tcount & 1u;
                    ++tcount;
                    auto slot = [](uint32_t x) { return x < WIDE_STAGES ? x : x - WIDE_STAGES; };
                    auto mma_block = [&](uint32_t s, int h, bool first) {
                        const uint32_t alo = static_cast<uint32_t>(adesc0) + s * SLOT;
                        const uint32_t blo = static_cast<uint32_t>(bdesc0) + s * SLOT + h * (WIDE_B >> 4);
#pragma unroll
                        for (int k = 0; k < BK / UMMA_K; ++k)
                            tc_mma_f16<CG>(tmem_base + h * MAX_BN, desc(alo + k * k_step(AMN), adesc0),
                                           desc(blo + k * k_step(BMN), bdesc0), idesc, !(first && k == 0));
                    };
                    auto wait_full = [&]() {
                        if (!W.wait(bFULL + 8 * stage, phase)) return false;
                        if (++stage == WIDE_STAGES) { stage = 0; phase ^= 1u; }
                        return true;
                    };
                    auto wait_acc = [&](int h) {
                        if (!W.template wait<true>(bTEMPTY + 8 * h, aph)) return false;
                        tc_fence_after_sync();
                        return true;
                    };
                    if (nkb > static_cast<int>(2 * J)) {
                        const uint32_t h0 = stage;
#pragma unroll
                        for (uint32_t j = 0; j < J; ++j)
                            if (!wait_full()) return false;
                        tc_fence_after_sync();
                        if (!wait_acc(0)) return false;
                        issued_any = true;
#pragma unroll
                        for (uint32_t j = 0; j < J; ++j) mma_block(slot(h0 + j), 0, j == 0);
                        if (!wait_acc(1)) return false;
#pragma unroll
                        for (uint32_t j = 0; j < J; ++j) {
                            mma_block(slot(h0 + j), 1, j == 0);
                            tc_commit_2_mc(bEMPTY + 8 * slot(h0 + j), 0x3);
                        }
                        for (int kb = J; kb < nkb - static_cast<int>(J); ++kb) {
                            const uint32_t s0 = stage;
                            if (!wait_full()) return false;
                            tc_fence_after_sync();
                            mma_block(s0, 0, false);
                            mma_block(s0, 1, false);
                            tc_commit_2_mc(bEMPTY + 8 * s0, 0x3);
                        }
                        const uint32_t t0 = stage;
#pragma unroll
                        for (uint32_t j = 0; j < J; ++j)
                            if (!wait_full()) return false;
                        tc_fence_after_sync();
#pragma unroll
                        for (uint32_t j = 0; j < J; ++j) mma_block(slot(t0 + j), 0, false);
                        tc_commit_2_mc(bTFULL, 0x3);
#pragma unroll
                        for (uint32_t j = 0; j < J; ++j) {
                            mma_block(slot(t0 + j), 1, false);
                            tc_commit_2_mc(bEMPTY + 8 * slot(t0 + j), 0x3);
                        }
                        tc_commit_2_mc(bTFULL + 8, 0x3);
                    } else {
                        for (int kb = 0; kb < nkb; ++kb) {
                            const uint32_t s0 = stage;
                            if (!wait_full()) return false;
                            tc_fence_after_sync();
                            if (kb == 0 && (!wait_acc(0) || !wait_acc(1))) return false;
                            issued_any = true;
                            mma_block(s0, 0, kb == 0);
                            mma_block(s0, 1, kb == 0);
                            tc_commit_2_mc(bEMPTY + 8 * s0, 0x3);
                        }
                        tc_commit_2_mc(bTFULL, 0x3);
                        tc_commit_2_mc(bTFULL + 8, 0x3);
                    }
                    return true;
                }
                // (counted in what is left: a chunk may be "all")
                for (int left = t.kb1 - t.kb0; left > 0; ++tcount) {
                    const int count = min(left, chunk);
                    left -= count;
                    const uint32_t b = tcount & 1u, aph = (tcount >> 1) & 1u;
                    if (!W.template wait<CG == 2>(bTEMPTY + 8 * b, aph)) return false;
                    tc_fence_after_sync();
                    const uint32_t d_tmem = tmem_base + b * MAX_BN;
                    for (int i = 0; i < count;) {
                        if (!W.wait(bFULL + 8 * stage, phase)) return false;
                        tc_fence_after_sync();
                        uint32_t alo = static_cast<uint32_t>(adesc0) + off, blo = static_cast<uint32_t>(bdesc0) + off;
                        const int end = min(count, i + boxes);
                        do {
#pragma unroll
                            for (int k = 0; k < BK / UMMA_K; ++k)
                                tc_mma_f16<CG>(d_tmem, desc(alo + k * k_step(AMN), adesc0),
                                               desc(blo + k * k_step(BMN), bdesc0), idesc, i != 0 || k != 0);
                            alo += box16;
                            blo += box16;
                        } while (++i < end);
                        issued_any = true;
                        if constexpr (CG == 1) tc_commit_1(bEMPTY + 8 * stage);
                        else tc_commit_2_mc(bEMPTY + 8 * stage, 0x3);
                        off += slot16;
                        if (++stage == S) { stage = 0; phase ^= 1u; off = 0; }
                    }
                    if constexpr (CG == 1) tc_commit_1(bTFULL + 8 * b);
                    else tc_commit_2_mc(bTFULL + 8 * b, 0x3);
                }
                return true;
            };
            Schedule sched(p, group_id, num_groups);
            for (int jn, u; ok && sched.next(jn, u);) {
                const Job& job = p.job[jn];
                Tile t;
                k_range(u, job, t);
                if constexpr (BMN) {
                    ok = job.amn ? unit(t, job.idesc, std::true_type{}) : unit(t, job.idesc, std::false_type{});
                } else {
                    ok = unit(t, job.idesc, std::false_type{});
                }
            }
            if (issued_any) {
                // all multiplies have finished before tensor memory is released
                if constexpr (CG == 1) tc_commit_1(bDRAIN);
                else tc_commit_2_mc(bDRAIN, 0x1);
                volatile uint32_t no_abort = 0;
                const Waiter D{max(p.timeout_ns, kDrainNs), &no_abort, p.status, kStatusRoleMma};
                D.wait(bDRAIN, 0);
            }
        }
        __syncwarp();
    } else {
        // ======================================================== epilogue
        const int e = warp - kMmaWarp - 1;
        const int q = warp & 3;                  // tensor-memory lane quarter of this warp
        const Waiter W{p.timeout_ns, abort_flag, p.status, kStatusRoleEpilogue};
        const uint32_t tempty_leader = CG == 2 ? mapa_shared(bTEMPTY, 0) : bTEMPTY;
        if (lane == 0)
            for (int b = 0; b < 2; ++b) {
                if constexpr (CG == 1) mbar_arrive(bTEMPTY + 8 * b);
                else mbar_arrive_cluster(tempty_leader + 8 * b);
            }
        const uint32_t buf = base + OFF_EPI + static_cast<uint32_t>(e) * EPI_BUF;     // this warp's staging buffer
        // the chunks whose number is 1 mod 2 are the lane quarter's second warp's
        const int first_chunk = (e >> 2) * EPI_COLS;
        constexpr int CHUNK_STEP = 2 * EPI_COLS;
        int tile_end = 0;                        // the tile's last column + 1, past N or not
        // One 64-column chunk (this lane's row, 32 packed pairs) of a 16-bit
        // output: staged in the swizzle its tensor map uses and stored by TMA,
        // or, where TMA cannot address the output or the tile ends inside the
        // chunk, staged and stored by the warp.
        auto emit = [&](const uint32_t(&h)[32], const Job& job, const CUtensorMap* map, uint16_t* out, int row0,
                        int col0, int col_end) {
            const bool by_tma = job.tma_store && col0 + EPI_COLS <= tile_end;
            // the store issued from the buffer has finished reading it
            if (lane == 0) bulk_wait_group_read<0>();
            __syncwarp();
            const uint32_t row_addr = buf + static_cast<uint32_t>(lane) * 128;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t dst = row_addr + ((static_cast<uint32_t>(j) ^ static_cast<uint32_t>(lane & 7)) << 4);
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(h[4 * j]),
                             "r"(h[4 * j + 1]), "r"(h[4 * j + 2]), "r"(h[4 * j + 3])
                             : "memory");
            }
            if (by_tma) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (row0 < job.M && col0 < job.N) tma_store_2d(map, buf, col0, row0);
                    bulk_commit_group();
                }
                return;
            }
            // The warp writes row by row, consecutive lanes at consecutive
            // addresses: 16 bytes a lane and four rows at a time where rows
            // start on 16-byte boundaries, else a 4-byte pair (or two
            // elements) a lane.  Eight reads are in flight before the writes:
            // one at a time, the 32 round trips of a chunk took longer than
            // the multiplies of a K loop of 13 blocks.
            __syncwarp();
            const int64_t ld = job.ld16;
            if ((reinterpret_cast<uintptr_t>(out) & 15u) == 0 && (ld & 7) == 0 && (col_end & 7) == 0) {
                const int j = lane & 7, col = col0 + 8 * j;
#pragma unroll
                for (int r0 = 0; r0 < 32; r0 += 4) {
                    const int r = r0 + (lane >> 3);
                    uint32_t v[4];
                    ld_shared_v4(buf + static_cast<uint32_t>(r) * 128 + (static_cast<uint32_t>(j ^ (r & 7)) << 4), v[0],
                                 v[1], v[2], v[3]);
                    if (row0 + r < job.M && col < col_end)
                        *reinterpret_cast<uint4*>(out + static_cast<int64_t>(row0 + r) * ld + col) =
                            make_uint4(v[0], v[1], v[2], v[3]);
                }
            } else {
                const int col = col0 + 2 * lane;
                const bool pairs = (reinterpret_cast<uintptr_t>(out) & 3u) == 0 && (ld & 1) == 0;
                const uint32_t in_row = static_cast<uint32_t>(lane & 3) * 4;
                for (int r0 = 0; r0 < 32 && row0 + r0 < job.M; r0 += 8) {
                    uint32_t v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        v[i] = ld_shared_u32(buf + static_cast<uint32_t>(r0 + i) * 128 +
                                             (static_cast<uint32_t>((lane >> 2) ^ i) << 4) + in_row);
                    uint16_t* dst = out + static_cast<int64_t>(row0 + r0) * ld + col;
#pragma unroll
                    for (int i = 0; i < 8; ++i, dst += ld) {
                        if (row0 + r0 + i >= job.M) break;
                        if (pairs && col + 1 < col_end) {
                            *reinterpret_cast<uint32_t*>(dst) = v[i];
                        } else {
                            if (col < col_end) dst[0] = static_cast<uint16_t>(v[i] & 0xFFFFu);
                            if (col + 1 < col_end) dst[1] = static_cast<uint16_t>(v[i] >> 16);
                        }
                    }
                }
            }
        };
        uint32_t tcount = 0;
        // waits for the next accumulator hand-over; its tensor-memory address
        auto acquire = [&](uint32_t& tbase) {
            const uint32_t b = tcount & 1u;
            bool got = true;
            if (lane == 0) got = W.wait_progress(bTFULL + 8 * b, (tcount >> 1) & 1u, sPROGRESS, false);
            got = __shfl_sync(0xffffffffu, got, 0);
            tc_fence_after_sync();
            tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + b * MAX_BN;
            return got;
        };
        // This warp's reads of the accumulator are complete (tcgen05.wait::ld after
        // every load) and fenced: tensor memory is all that is handed over, so the
        // arrival at the leader's barrier is relaxed (ptx.cuh gives the rule; the
        // MMA thread's side is its wait and tc_fence_after_sync).  A releasing one waits for the warp's output
        // stores: 1800 to 3100 clocks a tile, of about 6600.
        auto release = [&]() {
            const uint32_t b = tcount & 1u;
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if constexpr (CG == 1) mbar_arrive(bTEMPTY + 8 * b);
                else mbar_arrive_cluster_relaxed(tempty_leader + 8 * b);
            }
            ++tcount;
        };
        Schedule sched(p, group_id, num_groups);
        for (int jn, u; sched.next(jn, u);) {
            const Job& job = p.job[jn];
            const Tile t = tile_of<GROUP_M>(u, job);
            const int row0 = t.tm * (BM_CTA * CG) + static_cast<int>(rank) * BM_CTA + q * 32;
            const int row = row0 + lane;
            // (the wide tile's halves, one accumulator buffer each, in turn)
            bool alive = true;
            for (int wide = 0; wide < NW; ++wide) {
                const int n0 = (t.tn * NW + wide) * p.tile_n;
                tile_end = n0 + p.tile_n;
                const int col_end = min(job.N, tile_end);
                uint32_t tbase;
                if constexpr (EPI == kEpiI8) {
                    // This warp's two 64-column chunks.  128 * 128 * 1024 = 2^24: a chunk's
                    // sum of products of 8-bit integers is a whole number that fp32 holds,
                    // as is every partial sum of it, and chunks are added as integers.
                    const bool rows_live = row0 < job.M;
                    int z[4][32];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int i = 0; i < 32; ++i) z[j][i] = 0;
                    bool got = true;
                    for (int c0 = t.kb0; c0 < t.kb1; c0 += p.chunk) {
                        if (!acquire(tbase)) { got = false; break; }
                        if (rows_live) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int c = first_chunk + CHUNK_STEP * (j >> 1) + 32 * (j & 1);
                                if (c < p.tile_n) {
#pragma unroll
                                    for (int h = 0; h < 32; h += 16) {
                                        uint32_t v[16];
                                        tmem_ld_32x32b_x16(tbase + static_cast<uint32_t>(c + h), v);
                                        tmem_ld_wait();
#pragma unroll
                                        for (int i = 0; i < 16; ++i) z[j][h + i] += __float2int_rn(__uint_as_float(v[i]));
                                    }
                                }
                            }
                        }
                        release();
                    }
                    if (!got) { alive = false; break; }
                    if (!rows_live) continue;
                    const float sa = row < job.M ? __ldg(p.a_scale + row) : 0.0f;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int c = n0 + first_chunk + CHUNK_STEP * k;
                        if (c >= col_end) continue;
                        uint32_t h[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const int col = c + 2 * i;
                            const float s0 = col < col_end ? __ldg(p.b_scale + col) : 0.0f;
                            const float s1 = col + 1 < col_end ? __ldg(p.b_scale + col + 1) : 0.0f;
                            const int(&v)[32] = z[2 * k + i / 16];
                            h[i] = pack16(i8_value(v[2 * i % 32], sa, s0), i8_value(v[2 * i % 32 + 1], sa, s1), p.bf16);
                        }
                        emit(h, job, &maps.c[0], job.out16[0], row0, c, col_end);
                    }
                    continue;
                }
                if constexpr (EPI == kEpiXentStats || EPI == kEpiXentGrad) {
                    // This warp's four 32-column groups: 2 j + half of the tile's, or
                    // for the gradient those of its 64-column chunks.  The logits
                    // are summed over K chunk by chunk first.
                    const int half = e >> 2;
                    const auto group = [&](int j) {
                        return EPI == kEpiXentStats ? 32 * (2 * j + half)
                                                    : first_chunk + CHUNK_STEP * (j >> 1) + 32 * (j & 1);
                    };
                    const bool rows_live = row0 < job.M;
                    float z[4][32];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int i = 0; i < 32; ++i) z[j][i] = 0.0f;
                    bool got = true;
                    for (int c0 = t.kb0; c0 < t.kb1; c0 += p.chunk) {
                        if (!acquire(tbase)) { got = false; break; }
                        if (rows_live) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int c = group(j);
                                if (c < p.tile_n) {
                                    // (16 columns at a time: 128 running sums leave
                                    // 40 registers of the 168 a thread can have)
#pragma unroll
                                    for (int h = 0; h < 32; h += 16) {
                                        uint32_t v[16];
                                        tmem_ld_32x32b_x16(tbase + static_cast<uint32_t>(c + h), v);
                                        tmem_ld_wait();
#pragma unroll
                                        for (int i = 0; i < 16; ++i) z[j][h + i] += __uint_as_float(v[i]);
                                    }
                                }
                            }
                        }
                        release();
                    }
                    if (!got) { alive = false; break; }
                    if (!rows_live) continue;
                    const int64_t tgt = row < job.M ? p.target[row] - p.col0 : -1;
                    if constexpr (EPI == kEpiXentGrad) {
                        // D = coef (exp(z - lse) - [column = target])
                        const float lse = row < job.M ? p.lse[row] : 0.0f;
                        const float coef = row < job.M ? p.coef[row] : 0.0f;
                        const bool counts = row < job.M && p.target[row] != p.ignore_index;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int c = n0 + first_chunk + CHUNK_STEP * k;
                            if (c >= col_end) continue;
                            uint32_t h[32], lo[32];
#pragma unroll
                            for (int s = 0; s < 2; ++s) {
                                float(&d)[32] = z[2 * k + s];
                                const int cc = c + 32 * s;
#pragma unroll
                                for (int i = 0; i < 32; ++i) d[i] = exp_from(d[i], lse);
                                if (__any_sync(0xffffffffu, tgt >= cc && tgt < cc + 32)) {
#pragma unroll
                                    for (int i = 0; i < 32; ++i)
                                        if (tgt == cc + i) d[i] -= 1.0f;
                                }
                                // a row that does not count is zero whatever its logits are
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    const float d0 = counts ? coef * d[2 * i] : 0.0f;
                                    const float d1 = counts ? coef * d[2 * i + 1] : 0.0f;
                                    const uint32_t hi = pack16(d0, d1, p.bf16);
                                    h[16 * s + i] = hi;
                                    if constexpr (CG == 1) {
                                        const float2 r = unpack16(hi, p.bf16);
                                        lo[16 * s + i] = pack16(remainder16(d0, r.x), remainder16(d1, r.y), p.bf16);
                                    }
                                }
                            }
                            emit(h, job, &maps.c[0], job.out16[0], row0, c, col_end);
                            // (remainders are few rows', which a single CTA holds)
                            if (CG == 1 && p.lo_offset)
                                emit(lo, job, &maps.c[1], job.out16[0] + p.lo_offset, row0, c, col_end);
                        }
                        continue;
                    }
                    // Statistics: the running maximum m and sum s = sum exp(z - m) of the row.
                    const float inf = __int_as_float(0x7f800000);
                    float m = -inf, s = 0.0f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int c = n0 + 32 * (2 * j + half);
                        if (c >= col_end) continue;
                        if (c + 32 > col_end) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (c + i >= col_end) z[j][i] = -inf;
                        }
                        const bool mine = tgt >= c && tgt < c + 32;
                        if (__any_sync(0xffffffffu, mine)) {
                            float zt = 0.0f;
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (tgt == c + i) zt = z[j][i];
                            if (mine && tgt < col_end) p.z_target[row] = zt;
                        }
                        float top = m;
#pragma unroll
                        for (int i = 0; i < 32; ++i) top = fmaxf(top, z[j][i]);
                        // a row of -inf so far: any finite reference gives exp(-inf) = 0
                        const float ref = top == -inf ? 0.0f : top;
                        s *= exp_from(m, ref);
                        float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            s0 += exp_from(z[j][i], ref);
                            s1 += exp_from(z[j][i + 1], ref);
                            s2 += exp_from(z[j][i + 2], ref);
                            s3 += exp_from(z[j][i + 3], ref);
                        }
                        s += (s0 + s1) + (s2 + s3);
                        m = top;
                    }
                    if (row < job.M) p.stats[static_cast<int64_t>(row) * (2 * job.tiles_n) + 2 * t.tn + half] = make_float2(m, s);
                    continue;
                }
                if (!acquire(tbase)) { alive = false; break; }
                if (row0 < job.M) {
                    if constexpr (EPI == kEpiStore) {
                        const float scale = job.scale ? *job.scale : 1.0f;
                        if (job.out32) {
                            // fp32 partial or running sums
                            float* out = job.out32 + t.split * job.split_stride + t.problem * job.problem_stride +
                                         static_cast<int64_t>(row) * job.ld32;
                            const float* in = job.acc_in ? job.acc_in + static_cast<int64_t>(row) * job.ld32 : nullptr;
                            for (int c = n0 + first_chunk / 2; c < col_end; c += CHUNK_STEP / 2) {
                                uint32_t v[32];
                                tmem_ld_32x32b_x32(tbase + static_cast<uint32_t>(c - n0), v);
                                tmem_ld_wait();
                                if (row < job.M) {
#pragma unroll
                                    for (int i = 0; i < 32; i += 4) {
                                        if (c + i < col_end) {          // rows are padded to a multiple of 4
                                            float4 o = make_float4(__uint_as_float(v[i]), __uint_as_float(v[i + 1]),
                                                                   __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
                                            if (in) {
                                                const float4 a = *reinterpret_cast<const float4*>(in + c + i);
                                                o.x += a.x; o.y += a.y; o.z += a.z; o.w += a.w;
                                            }
                                            *reinterpret_cast<float4*>(out + c + i) = o;
                                        }
                                    }
                                }
                            }
                        } else {
                            const float* in = job.acc_in ? job.acc_in + static_cast<int64_t>(row) * job.ld32 : nullptr;
                            for (int c = n0 + first_chunk; c < col_end; c += CHUNK_STEP) {
                                uint32_t h[32];
#pragma unroll
                                for (int half = 0; half < 2; ++half) {
                                    uint32_t v[32];
                                    tmem_ld_32x32b_x32(tbase + static_cast<uint32_t>(c - n0 + 32 * half), v);
                                    tmem_ld_wait();
                                    if (in && row < job.M) {
#pragma unroll
                                        for (int i = 0; i < 32; i += 4) {
                                            if (c + 32 * half + i < col_end) {
                                                const float4 a = *reinterpret_cast<const float4*>(in + c + 32 * half + i);
                                                v[i] = __float_as_uint(__uint_as_float(v[i]) + a.x);
                                                v[i + 1] = __float_as_uint(__uint_as_float(v[i + 1]) + a.y);
                                                v[i + 2] = __float_as_uint(__uint_as_float(v[i + 2]) + a.z);
                                                v[i + 3] = __float_as_uint(__uint_as_float(v[i + 3]) + a.w);
                                            }
                                        }
                                    }
#pragma unroll
                                    for (int i = 0; i < 16; ++i)
                                        h[16 * half + i] = pack16(scale * __uint_as_float(v[2 * i]),
                                                                  scale * __uint_as_float(v[2 * i + 1]), p.bf16);
                                }
                                emit(h, job, &maps.c[job.c_map + t.problem], job.out16[t.problem], row0, c, col_end);
                            }
                        }
                    } else if constexpr (EPI == kEpiGated) {
                        for (int c = n0 + first_chunk; c < col_end; c += CHUNK_STEP) {
                            const uint32_t at = tbase + static_cast<uint32_t>(c - n0);
                            uint32_t h[32];
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                uint32_t g[32], up[32];
                                if (c - n0 + 32 * half < p.tile_n) {
                                    tmem_ld_32x32b_x32(at + 32 * half, g);
                                    tmem_ld_32x32b_x32(at + p.tile_n + 32 * half, up);
                                    tmem_ld_wait();
                                } else {
#pragma unroll
                                    for (int i = 0; i < 32; ++i) g[i] = up[i] = 0u;
                                }
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    h[16 * half + i] =
                                        pack16(act_value(__uint_as_float(g[2 * i]), p.act) * __uint_as_float(up[2 * i]),
                                               act_value(__uint_as_float(g[2 * i + 1]), p.act) *
                                                   __uint_as_float(up[2 * i + 1]),
                                               p.bf16);
                            }
                            emit(h, job, &maps.c[0], job.out16[0], row0, c, col_end);
                            if (!p.g_out) continue;
                            // gate and up themselves, read from tensor memory again:
                            // kept from above they take more registers than eleven
                            // warps leave a thread
#pragma unroll 1
                            for (int which = 0; which < 2; ++which) {
#pragma unroll
                                for (int half = 0; half < 2; ++half) {
                                    uint32_t v[32];
                                    if (c - n0 + 32 * half < p.tile_n) {
                                        tmem_ld_32x32b_x32(at + which * p.tile_n + 32 * half, v);
                                        tmem_ld_wait();
                                    } else {
#pragma unroll
                                        for (int i = 0; i < 32; ++i) v[i] = 0u;
                                    }
#pragma unroll
                                    for (int i = 0; i < 16; ++i)
                                        h[16 * half + i] =
                                            pack16(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]), p.bf16);
                                }
                                emit(h, job, &maps.c[1 + which], which ? p.u_out : p.g_out, row0, c, col_end);
                            }
                        }
                    }
                }
                release();
            }
            if (!alive) break;
        }
        // the staging buffers must stay until the last stores have read them
        if (lane == 0) bulk_wait_group_read<0>();
        __syncwarp();
    }

    // ------------------------------------------------------------ tear-down
    tc_fence_before_sync();
    __syncthreads();
    if (CG == 2) cluster_sync();
    if (warp == kMmaWarp) {
        tc_fence_after_sync();
        tmem_dealloc<CG>(tmem_base, 512);
    }
}

}  // namespace fused
}  // namespace pws

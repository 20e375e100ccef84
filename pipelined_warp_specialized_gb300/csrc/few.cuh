// few.cuh -- products of a few tokens: weights stream through a ring of each warp's
// own into the registers that multiply them.
//
//   D[r, t] = sum_k W[r, k] X[t, k]        16 weight rows r, 8 tokens t a tile
//
// With few tokens a product is bound by the weights' bytes, so what counts is
// that every warp has many 16-byte copies in flight: they go asynchronously into
// shared memory (Ring, below), and each lane reads its own back.  The operand
// layout of mma.m16n8k16 needs no exchange between lanes on the way: the
// instruction's k index only has to mean the same for both
// operands, so lane (g, t) (g = lane / 4, t = lane % 4) takes 16 consecutive
// bytes of rows g and g + 8, at byte 16 t of a 64-byte step, and 8 or 16
// consecutive elements of token g at the same k.  A step is 32 k of 16-bit
// weights or 64 of 8-bit ones, which are converted in registers: every 8-bit
// integer is a binary16 and a bfloat16 value.  Shared memory, which weights and tokens both
// enter and leave, is the busiest unit of these kernels next to memory.
#pragma once

#include "product.cuh"

namespace pws {
namespace few {

// Weights' form, and the type of the tokens they are multiplied by.
enum Form { kHalf = 0, kBfloat = 1, kI8Half = 2, kI8Bfloat = 3 };

constexpr bool is_bf16(int form) { return form & 1; }
constexpr bool is_i8(int form) { return form >= kI8Half; }
// k of a step, bytes of a weight, and the halves of a step that 8-bit weights are widened in
constexpr int step_k(int form) { return is_i8(form) ? 64 : 32; }
constexpr int weight_bytes(int form) { return is_i8(form) ? 1 : 2; }
constexpr int halves_of(int form) { return is_i8(form) ? 2 : 1; }

template <bool BF16>
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 32 k of a 16-row weight tile (rows g and g + 8 of this lane) by one tile of
// eight tokens.
template <bool BF16>
__device__ __forceinline__ void mma_step(float (&d)[4], const uint32_t (&lo)[4], const uint32_t (&hi)[4], const uint32_t (&x)[4]) {
    mma_16x8x16<BF16>(d, lo[0], hi[0], lo[1], hi[1], x[0], x[1]);
    mma_16x8x16<BF16>(d, lo[2], hi[2], lo[3], hi[3], x[2], x[3]);
}

// Four 8-bit integers as two pairs of 16-bit values, exactly, by the common way without
// conversions: an integer below the bits of a power of two reads as their sum.
//   binary16: a byte b + 128 below the bits of 1024 reads 1152 + b; minus 1152.
//   bfloat16: below the bits of 128 (units of one) the low seven bits read 128 + (b & 127),
//             the sign bit alone 128 or 256; their difference is b.
template <bool BF16>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (BF16) {
        const uint32_t p = __byte_perm(w, 0x43434343u, 0x4140), q = __byte_perm(w, 0x43434343u, 0x4342);
        const auto diff = [](uint32_t v) {
            const uint32_t a = v & 0x437F437Fu, b = v & 0x43804380u;
            const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                             *reinterpret_cast<const __nv_bfloat162*>(&b));
            return *reinterpret_cast<const uint32_t*>(&d);
        };
        lo = diff(p);
        hi = diff(q);
    } else {
        const uint32_t u = w ^ 0x80808080u, c = 0x64806480u;
        const uint32_t p = __byte_perm(u, 0x64646464u, 0x4140), q = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 off = *reinterpret_cast<const __half2*>(&c);
        const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&p), off);
        const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&q), off);
        lo = *reinterpret_cast<const uint32_t*>(&a);
        hi = *reinterpret_cast<const uint32_t*>(&b);
    }
}

// A step's 16 bytes of a weight row (or half of them) as the pairs the multiply takes.
template <int FORM>
__device__ __forceinline__ void widen(const uint4& w, int half, uint32_t (&v)[4]) {
    if constexpr (is_i8(FORM)) {
        widen4<is_bf16(FORM)>(half ? w.z : w.x, v[0], v[1]);
        widen4<is_bf16(FORM)>(half ? w.w : w.y, v[2], v[3]);
    } else {
        v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
    }
}

// Bytes shift .. shift + 15 of two 16-byte blocks.  Selections, not branches: a warp's rows
// lie at four shifts or more, and with a branch for each of them this was most of a ragged
// row's time (7 tokens over 12 experts of 731 x 1030 60 us, and 43 so; 28 where rows are aligned).
__device__ __forceinline__ uint32_t chosen(uint32_t a, uint32_t b, uint32_t which) {
    uint32_t v;
    asm("{.reg .pred p; setp.ne.u32 p, %3, 0; selp.b32 %0, %2, %1, p;}" : "=r"(v) : "r"(a), "r"(b), "r"(which));
    return v;
}
__device__ __forceinline__ uint4 shifted(const uint4& lo, const uint4& hi, uint32_t shift) {
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    uint32_t two[6], one[5];
#pragma unroll
    for (int k = 0; k < 6; ++k) two[k] = chosen(w[k], w[k + 2], shift & 8u);
#pragma unroll
    for (int k = 0; k < 5; ++k) one[k] = chosen(two[k], two[k + 1], shift & 4u);
    const uint32_t bits = (shift & 3u) * 8u;
    return make_uint4(__funnelshift_r(one[0], one[1], bits), __funnelshift_r(one[1], one[2], bits),
                      __funnelshift_r(one[2], one[3], bits), __funnelshift_r(one[3], one[4], bits));
}

// The first `n` bytes of 16, and zeros.
__device__ __forceinline__ uint4 cleared(const uint4& b, int n) {
    if (n >= 16) return b;
    uint32_t v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = n >= 4 * i + 4 ? v[i] : n > 4 * i ? v[i] & ((1u << (8 * (n - 4 * i))) - 1u) : 0u;
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// 16 bytes read once: past L1.
__device__ __forceinline__ uint4 load_stream(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// 16 bytes of a row, `left` bytes before its end; what lies behind the end is
// zeros, whatever follows in memory (a neighbour's infinity times a zero would be
// NaN).  ALIGNED: rows start on 16-byte boundaries and are a multiple of 16
// bytes long.  Otherwise the one or two aligned blocks that hold bytes of the row
// are read and shifted together; a block that holds none is not touched.
template <bool ALIGNED, bool STREAM>
__device__ __forceinline__ uint4 load_row(const uint8_t* p, int64_t left) {
    const auto load = [](const void* q) { return STREAM ? load_stream(q) : __ldg(static_cast<const uint4*>(q)); };
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (ALIGNED) {
        if (left > 0) v = load(p);
    } else {
        const uint32_t shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15u);
        const uint8_t* block = p - shift;
        uint4 w = v;
        if (left > 0) v = load(block);
        if (shift != 0 && left > 16 - static_cast<int>(shift)) w = load(block + 16);
        v = shifted(v, w, shift);
        v = cleared(v, left < 16 ? static_cast<int>(left) : 16);
    }
    return v;
}

// The way of weights and tokens into registers: a ring of a few steps in shared
// memory for each warp alone, filled by 16-byte asynchronous copies.  A lane
// reads what it copied itself, so no other warp is waited for, and the
// ring runs on over the borders of row blocks and experts, so that memory is
// never idle while sums are joined.  The tokens come the same way: they are L2's, but
// behind the weights' traffic an L2 load takes as long as a whole step (loaded one step
// ahead into registers, 16 tokens over 56 experts of 1536 x 4096 read 4.9 TB/s; with
// no token loads at all 5.9).
//
// Rows that do not start on 16-byte boundaries: the two aligned blocks that
// hold the lane's 16 bytes, shifted together when they are read and cleared behind
// the row's end.  The second one is the next lane's first (the last of a row's four
// lanes copies its own).  A block that holds none of the row's bytes is not touched.
constexpr int kLoads = 4;               // weight rows a lane reads a step

__device__ __forceinline__ void cp_async_l1(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// TOKENS: 16-byte pieces of token rows a lane takes a step.
constexpr int ring_slot(bool aligned, int tokens) { return (kLoads + (aligned ? 0 : 1) + tokens) * 512; }
// As many stages, up to four, as leave room for two blocks of eight warps an SM,
// `beside` bytes of other shared memory in each; where that is less than three, for one.
constexpr int ring_stages(bool aligned, int tokens, int beside) {
    const int stage = 8 * ring_slot(aligned, tokens), two = (115200 - beside) / stage, one = (231424 - beside) / stage;
    return two >= 3 ? (two < 4 ? two : 4) : one < 4 ? one : 4;
}

template <bool ALIGNED, int TOKENS, int BESIDE>
struct Ring {
    static constexpr int STAGES = ring_stages(ALIGNED, TOKENS, BESIDE), WEIGHTS = kLoads + (ALIGNED ? 0 : 1);
    static constexpr uint32_t BLOCK = 512, SLOT = ring_slot(ALIGNED, TOKENS), WARP_BYTES = STAGES * SLOT;
    uint32_t first, fill, read;

    // base: of the block's rings, one after the other.
    __device__ __forceinline__ Ring(uint32_t base, int warp)
        : first(base + warp * WARP_BYTES + (threadIdx.x % 32) * 16), fill(first), read(first) {}
    __device__ __forceinline__ uint32_t after(uint32_t at) const { return at == first + (STAGES - 1) * SLOT ? first : at + SLOT; }

    // The block behind the last lane's of row i.
    __device__ __forceinline__ uint32_t after_row(uint32_t stage, int i) const {
        return stage - (threadIdx.x % 32) * 16 + kLoads * BLOCK + i * 128 + (threadIdx.x % 32) / 4 * 16;
    }
    // The lane's 16 bytes of each row into the next stage; `left` bytes of the
    // rows from there on (none or less: zeros).
    __device__ __forceinline__ void copy(const uint8_t* const (&at)[kLoads], int left) {
        if (ALIGNED && left <= 0) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(fill + i * BLOCK), "r"(0) : "memory");
            return;
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            if constexpr (ALIGNED) {
                cp_async<16>(fill + i * BLOCK, at[i], 16u);
            } else {
                const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(at[i]) & 15u);
                // (the lane before may want what its block holds of the row's end; what none wants is cleared)
                if (left > -shift) cp_async<16>(fill + i * BLOCK, at[i] - shift, 16u);
                if (threadIdx.x % 4 == 3 && left > 16 - shift) cp_async<16>(after_row(fill, i), at[i] - shift + 16, 16u);
            }
        }
    }
    // Piece i of the tokens: 16 bytes at `at`, through L1 (past it, every block of the GPU asks the
    // same few lines of L2: 78 us instead of 44 for one token's gate).
    __device__ __forceinline__ void copy_token(int i, const void* at) { cp_async_l1(fill + (WEIGHTS + i) * BLOCK, at); }
    // Ends a stage (an empty one too: stages are counted).
    __device__ __forceinline__ void commit() {
        cp_async_commit();
        fill = after(fill);
    }
    // The oldest stage has landed, of STAGES - 1 in flight.
    __device__ __forceinline__ void wait() {
        cp_async_wait_group<STAGES - 2>();
        __syncwarp();               // (ragged rows read each other's blocks)
    }
    // Row i's 16 bytes of the oldest stage.  `row`: any address of the row's that is a multiple of 16
    // bytes from its start; `left`: as it was copied.
    __device__ __forceinline__ uint4 get(int i, const uint8_t* row, int left) const {
        uint4 lo, hi;
        ld_shared_v4(read + i * BLOCK, lo.x, lo.y, lo.z, lo.w);
        if constexpr (ALIGNED) return lo;
        ld_shared_v4(threadIdx.x % 4 == 3 ? after_row(read, i) : read + i * BLOCK + 16, hi.x, hi.y, hi.z, hi.w);
        return cleared(shifted(lo, hi, static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) & 15u)), left);
    }
    __device__ __forceinline__ void get_token(int i, uint32_t (&v)[4]) const {
        ld_shared_v4(read + (WEIGHTS + i) * BLOCK, v[0], v[1], v[2], v[3]);
    }
    __device__ __forceinline__ void pop() { read = after(read); }
};

// Units of work handed out to the blocks of a grid as they get to them: memory's
// bandwidth is not shared evenly between SMs, and with equal parts the GPU waited
// for its slowest (SMs busy for 73 % of the kernel, 4.3 TB/s).  A block's first
// unit is its number; later ones come from a counter that starts at zero.
//
// Rings run on into the next unit, so a block knows one unit beyond the one at work:
// unit i + 2 is claimed at the start of unit i and put into the queue before a
// barrier of unit i.  A warp with n steps a unit looks at unit i + 2 when it copies the
// last step before it, which is in unit i + 1 or later if n >= the ring's stages.  Shorter
// units would have to be claimed several ahead, and the first blocks would leave
// none to the others (7 tokens over 12 experts of 736 x 1024 37 us): they go round
// the blocks in turn (27 us).
struct Claims {
    static constexpr int QUEUE = 4;
    int* queue;                 // [QUEUE], shared
    int* counter;
    bool in_turn;

    // steps: the fewest a warp that has any takes of a unit
    static __device__ __forceinline__ bool too_short(int64_t steps, int stages) { return steps < stages; }
    __device__ __forceinline__ int claim() const { return in_turn ? 0 : static_cast<int>(gridDim.x) + atomicAdd(counter, 1); }
    // One thread, before a barrier: the first unit, the second, unit i + 2.
    __device__ __forceinline__ void start() const { queue[0] = static_cast<int>(blockIdx.x); }
    __device__ __forceinline__ void second(int unit) const { queue[1] = unit; }
    __device__ __forceinline__ void put(int i, int unit) const { queue[(i + 2) % QUEUE] = unit; }
    __device__ __forceinline__ int unit(int i) const {
        return in_turn ? static_cast<int>(blockIdx.x) + i * static_cast<int>(gridDim.x) : queue[i % QUEUE];
    }
};

}  // namespace few
}  // namespace pws

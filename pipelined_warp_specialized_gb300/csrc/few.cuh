// few.cuh -- products of a few tokens: weights stream from memory into the
// registers of the warps that multiply them.
//
//   D[r, t] = sum_k W[r, k] X[t, k]        16 weight rows r, 8 tokens t a tile
//
// With few tokens a product is bound by the weights' bytes, so what counts is
// that every warp has many 16-byte loads in flight.  The operand layout of
// mma.m16n8k16 lets a weight go from memory to the tensor core without shared
// memory in between: the instruction's k index only has to mean the same for both
// operands, so lane (g, t) (g = lane / 4, t = lane % 4) takes 16 consecutive
// bytes of rows g and g + 8, at byte 16 t of a 64-byte step, and 8 or 16
// consecutive elements of token g at the same k.  A step is 32 k of 16-bit
// weights or 64 of 8-bit ones, which are converted in registers: every 8-bit
// integer is a binary16 and a bfloat16 value.
#pragma once

#include "product.cuh"

namespace pws {
namespace few {

// Weights' form, and the type of the tokens they are multiplied by.
enum Form { kHalf = 0, kBfloat = 1, kI8Half = 2, kI8Bfloat = 3 };

constexpr bool is_bf16(int form) { return form & 1; }
constexpr bool is_i8(int form) { return form >= kI8Half; }
// k of a step, bytes of a weight, 32-bit registers of 16-bit values a lane holds of a row
constexpr int step_k(int form) { return is_i8(form) ? 64 : 32; }
constexpr int weight_bytes(int form) { return is_i8(form) ? 1 : 2; }
constexpr int pairs_of(int form) { return is_i8(form) ? 8 : 4; }

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

// One step's multiplies of a 16-row weight tile (rows g and g + 8 of this
// lane) by one tile of eight tokens.
template <int FORM>
__device__ __forceinline__ void mma_step(float (&d)[4], const uint32_t (&lo)[pairs_of(FORM)],
                                         const uint32_t (&hi)[pairs_of(FORM)], const uint32_t (&x)[pairs_of(FORM)]) {
#pragma unroll
    for (int i = 0; i < pairs_of(FORM); i += 2)
        mma_16x8x16<is_bf16(FORM)>(d, lo[i], hi[i], lo[i + 1], hi[i + 1], x[i], x[i + 1]);
}

// Four 8-bit integers as two pairs of 16-bit values, exactly.
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

// A step's 16 bytes of a weight row as the pairs the multiply takes.
template <int FORM>
__device__ __forceinline__ void widen(const uint4& w, uint32_t (&v)[pairs_of(FORM)]) {
    if constexpr (is_i8(FORM)) {
        widen4<is_bf16(FORM)>(w.x, v[0], v[1]);
        widen4<is_bf16(FORM)>(w.y, v[2], v[3]);
        widen4<is_bf16(FORM)>(w.z, v[4], v[5]);
        widen4<is_bf16(FORM)>(w.w, v[6], v[7]);
    } else {
        v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
    }
}

// 16 bytes read once: past L1.
__device__ __forceinline__ uint4 load_stream(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// 16 bytes of a row at any alignment; `left` of them are the row's, the rest
// are zeros, whatever follows in memory (a neighbour's infinity times a zero
// would be NaN).
static __device__ __noinline__ uint4 load_ragged_end(const uint8_t* p, int left) {
    uint32_t v[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < left) v[i / 4] |= static_cast<uint32_t>(p[i]) << (8 * (i % 4));
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// 16 bytes of a row, `left` bytes before its end.  ALIGNED: rows start on
// 16-byte boundaries and are a multiple of 16 bytes long.
template <bool ALIGNED, bool STREAM>
__device__ __forceinline__ uint4 load_row(const uint8_t* p, int64_t left) {
    if constexpr (ALIGNED) {
        if (left <= 0) return make_uint4(0u, 0u, 0u, 0u);
        return STREAM ? load_stream(p) : __ldg(reinterpret_cast<const uint4*>(p));
    } else {
        if (left >= 16) return fused::load_unaligned16(reinterpret_cast<const uint16_t*>(p));
        return left <= 0 ? make_uint4(0u, 0u, 0u, 0u) : load_ragged_end(p, static_cast<int>(left));
    }
}

}  // namespace few
}  // namespace pws

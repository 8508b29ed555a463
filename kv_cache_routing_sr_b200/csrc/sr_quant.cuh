// The 8-bit row format of the quantised KV cache and its device arithmetic,
// shared by the bulk write and read kernels and the single-token append.
//
// A row of 128 bf16 values x with top = max(max_i |x_i|, 2^-100) is stored as
// 128 codes c_i and one fp32 scale s; it stands for c_i * s.
//   e4m3: s = the power of two with 224 < top / s <= 448, c_i = e4m3(x_i / s).
//         The division is exact, so a code is the one rounding of its value, and
//         c_i * s has 4 significant bits: reading it back into bf16 is exact.
//   int8: s = top / 127 (fp32, nearest), c_i = round(127 x_i / top) as the real
//         quotient rounds, nearest with ties to even.
// The floor on top keeps s and 1 / s far from the ends of fp32 and makes an
// all-zero row an ordinary one. A row with an infinity or a NaN is stored as
// codes 0 and scale NaN: it reads back as NaN, as the row itself would poison
// whatever attends to it.
#pragma once

#include <cstdint>

#include "sinkrouter.h"
#include "sr_ptx.cuh"

namespace sr {

constexpr uint32_t kTopFloor = 0x0d800000u; // 2^-100 as fp32 bits

// Largest |x| of packed bf16 pairs, both halves at once, as bf16 bits: sign-less
// bf16 bit patterns order like the values, with infinities and NaNs on top.
__device__ __forceinline__ uint32_t abs_max_bf16x2(uint32_t acc, uint32_t w)
{
    return __vmaxu2(acc, w & 0x7fff7fffu);
}

// What a row's codes are computed from.
struct RowQuant {
    float scale; // stored scale (NaN for a row with a non-finite value)
    float mul;   // e4m3: 1 / scale; int8: 127 / top; 0 for a non-finite row
    // int8, with top = f 2^E, f in [1, 2): 127 2^-E, f and 1 / f. Without the power
    // of two 127 x could pass fp32's end, and 1 / top be subnormal.
    float up, f, rcp;
};

// top_bits: bf16 bits of the row's largest magnitude.
template <int KV> __device__ __forceinline__ RowQuant row_quant(uint32_t top_bits)
{
    RowQuant r;
    if (top_bits >= 0x7f80u) {
        r.scale = __uint_as_float(0x7fc00000u);
        r.mul = r.up = r.f = r.rcp = 0.f;
        return r;
    }
    uint32_t t = top_bits << 16;
    t = t < kTopFloor ? kTopFloor : t;
    if constexpr (KV == SR_KV_E4M3) {
        // top = f 2^E with f in [1, 2); 448 = 1.75 2^8
        const uint32_t se = (t >> 23) - 8u + ((t & 0x7fffffu) > 0x600000u ? 1u : 0u);
        r.scale = __uint_as_float(se << 23);
        r.mul = __uint_as_float((254u - se) << 23);
        r.up = r.f = r.rcp = 0.f;
    } else {
        const float down2 = __uint_as_float((255u - (t >> 23)) << 23); // 2 2^-E, normal for every E
        // top / 127, corrected like a code below; nearest for all 128 significands of
        // a bf16 top (checked in exact arithmetic, as all codes of all pairs of them)
        const float top = __uint_as_float(t), s0 = top * (1.f / 127.f);
        r.scale = fmaf(fmaf(-s0, 127.f, top), 1.f / 127.f, s0);
        r.f = __uint_as_float((t & 0x7fffffu) | 0x3f800000u);
        r.rcp = __frcp_rn(r.f);
        r.mul = 63.5f * r.rcp * down2;
        r.up = 63.5f * down2;
    }
    return r;
}

// Codes of four values held as two bf16 pairs, in element order from the low byte.
template <int KV> __device__ __forceinline__ uint32_t quant4(uint32_t w0, uint32_t w1, const RowQuant &r)
{
    const float x[4] = {__uint_as_float(w0 << 16), __uint_as_float(w0 & 0xffff0000u), __uint_as_float(w1 << 16),
                        __uint_as_float(w1 & 0xffff0000u)};
    if (r.mul == 0.f)
        return 0u;
    if constexpr (KV == SR_KV_E4M3) {
        uint32_t d;
        asm("{\n\t.reg .b16 lo, hi;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
            "mov.b32 %0, {lo, hi};\n\t}"
            : "=r"(d)
            : "f"(x[0] * r.mul), "f"(x[1] * r.mul), "f"(x[2] * r.mul), "f"(x[3] * r.mul));
        return d;
    } else {
        // y = 127 x / top, corrected by its own residual (Markstein, IBM J. R&D
        // 34, 1990), both sides over 2^E: 127 x has 15 bits, so the residual is
        // exact, and a quotient that fp32 can hold -- every tie between two codes is one --
        // comes out exactly; any other quotient is at least 2^-16 of itself
        // away from a tie, since x and top have 8 bits each. Adding 1.5 2^23
        // rounds to an integer, ties to even, whose low byte is the code. Two
        // values an instruction.
        const uint64_t mul = pack2(r.mul, r.mul), up = pack2(r.up, r.up), nf = pack2(-r.f, -r.f),
                       rcp = pack2(r.rcp, r.rcp), magic = pack2(12582912.f, 12582912.f);
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; i += 2)
            asm("{\n\t.reg .b64 y, u, z;\n\t"
                "mul.rn.f32x2 y, %2, %3;\n\t"
                "mul.rn.f32x2 u, %2, %4;\n\t"
                "fma.rn.f32x2 u, y, %5, u;\n\t"
                "fma.rn.f32x2 y, u, %6, y;\n\t"
                "add.rn.f32x2 z, y, %7;\n\t"
                "mov.b64 {%0, %1}, z;\n\t}"
                : "=r"(c[i]), "=r"(c[i + 1])
                : "l"(pack2(x[i], x[i + 1])), "l"(mul), "l"(up), "l"(nf), "l"(rcp), "l"(magic));
        return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    }
}

// The four values of a code word, times scale, in fp32.
template <int KV> __device__ __forceinline__ float4 dequant4(uint32_t w, float scale)
{
    if constexpr (KV == SR_KV_E4M3) {
        uint32_t h0, h1;
        asm("{\n\t.reg .b16 lo, hi;\n\t"
            "mov.b32 {lo, hi}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
            : "=r"(h0), "=r"(h1)
            : "r"(w));
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&h0));
        const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&h1));
        return make_float4(a.x * scale, a.y * scale, b.x * scale, b.y * scale);
    } else {
        return make_float4((float)(int8_t)(w & 0xffu) * scale, (float)(int8_t)((w >> 8) & 0xffu) * scale,
                           (float)(int8_t)((w >> 16) & 0xffu) * scale, (float)(int8_t)(w >> 24) * scale);
    }
}

} // namespace sr

// cache4.cuh -- the cache in 4 bits: how 16 features of a key are held, and how
// they come back.
//
// A block of 16 features x is held as whole numbers c = rint(x / s), -8 to 7, and a
// scale s = max|x| / 7 rounded to a floating-point number of 5 exponent and 3
// mantissa bits without a sign: the byte's value is that of the f16 with the bits
// byte << 7. So its range (normal from 2^-14 on, steps of 2^-17 below) needs no
// second scale, and c * s has 7 significant bits: it is exact in f16 and in bf16.
// Scales end at 240: the constants that bring a value back (-264 s) stay within
// f16. A block that holds an infinity or a NaN has the byte 0xff, a NaN.
//
// Whole numbers of 4 bits next to the same bits as a floating-point number (e2m1)
// with a scale per 16: normal values come back 8.6 % off against 9.5 % (rms), and
// in 2.75 instructions a pair against 4.
//
// 16 keys of a head ("group") are 9 d bytes in one run: their codes in the order
// in which the lanes of a matrix instruction take them, then their scales.
//   K: lane (g, t) of S^T = K Q^T has the features [t d/4, (t + 1) d/4) of the keys
//      kappa(g) and kappa(g) + 2, kappa(g) = 4 (g / 2) + g % 2
//   V: lane (g, t) of O^T = V^T P^T has the features [g d/8, (g + 1) d/8) of the
//      keys 4t, 4t + 1 (first part) and 4t + 2, 4t + 3 (second)
// Two 16-bit halves of a 32-bit word are the two values of a register: K's the even
// and odd features of 8, V's two keys' values of the same 4 features. In a half
// the codes c + 8 lie at bits 6-9 and 2-5, and the other two there after a swap of
// its bytes, where an "or" with the bits of 16 and of 256 makes them the numbers
// 16 + c + 8 and 256 + c + 8.
#pragma once

#include "cache.cuh"
#include "ptx.cuh"

namespace swa {

constexpr float kMaxScale4 = 240.f;
constexpr uint32_t kNanScale4 = 0xffu;

template <int HD>
struct Group4 {
    static constexpr uint32_t kCodes = 8 * HD, kBytes = 9 * HD;
};

// Byte of a group at which K's word (8 features, from 8 * w8) of key x lies.
template <int HD>
__device__ __forceinline__ uint32_t k4_word(uint32_t x, uint32_t w8)
{
    const uint32_t g = 2 * (x >> 2) + (x & 1), h = (x >> 1) & 1;
    constexpr uint32_t W = HD / 32;                 // words of a lane and key
    const uint32_t t = w8 / W, w = w8 % W;
    return HD == 128 ? h * 512 + (g * 4 + t) * 16 + w * 4 : (g * 4 + t) * 16 + h * 8 + w * 4;
}

// Byte of K's scale of key x, block f16 (16 features).
template <int HD>
__device__ __forceinline__ uint32_t k4_scale(uint32_t x, uint32_t f16)
{
    const uint32_t g = 2 * (x >> 2) + (x & 1), h = (x >> 1) & 1;
    return Group4<HD>::kCodes + (HD == 128 ? (g * 4 + (f16 >> 1)) * 4 + h * 2 + (f16 & 1) : (g * 4 + f16) * 2 + h);
}

// Byte of V's half word of key x that has the 4 features from 4 * f4.
template <int HD>
__device__ __forceinline__ uint32_t v4_half(uint32_t x, uint32_t f4)
{
    constexpr uint32_t W = HD / 32;                 // words of a lane and part
    const uint32_t t = x >> 2, part = (x >> 1) & 1, g = f4 / W, w = f4 % W;
    return (HD == 128 ? part * 512 + (g * 4 + t) * 16 + w * 4 : (g * 4 + t) * 16 + part * 8 + w * 4) + (x & 1) * 2;
}

template <int HD>
__device__ __forceinline__ uint32_t v4_scale(uint32_t x, uint32_t f16)
{
    return Group4<HD>::kCodes + f16 * 16 + x;
}

__device__ __forceinline__ uint32_t h2fma(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

__device__ __forceinline__ uint32_t h2mul(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Two scales as f16 (both exact), and the offsets that go with them.
struct Scale4 {
    uint32_t s, n24, n264;
};

// SEL: byte_perm selector that puts the two scale bytes of w at bytes 1 and 3,
// zeros (byte 4) at 0 and 2.
template <uint32_t SEL>
__device__ __forceinline__ Scale4 scale4(uint32_t w)
{
    Scale4 r;
    r.s = __byte_perm(w, 0u, SEL) >> 1;
    r.n24 = h2mul(r.s, 0xce00ce00u);        // -24
    r.n264 = h2mul(r.s, 0xdc20dc20u);       // -264
    return r;
}

// (x & M) | C as one instruction: it takes one of the two constants as such, the other in a register.
template <uint32_t M, uint32_t C>
__device__ __forceinline__ uint32_t and_or(uint32_t x)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(x), "r"(M), "n"(C));
    return r;
}

// The 8 values of a word as 4 registers of two f16 (register j: code j of the low and of the high half).
__device__ __forceinline__ void values4(uint32_t w, const Scale4& s, uint32_t (&r)[4])
{
    const uint32_t b = __byte_perm(w, 0u, 0x2301);
    r[0] = h2fma(and_or<0x03c003c0u, 0x4c004c00u>(w), s.s, s.n24);
    r[1] = h2fma(and_or<0x003c003cu, 0x5c005c00u>(w), s.s, s.n264);
    r[2] = h2fma(and_or<0x03c003c0u, 0x4c004c00u>(b), s.s, s.n24);
    r[3] = h2fma(and_or<0x003c003cu, 0x5c005c00u>(b), s.s, s.n264);
}

// Lane (g, t)'s words of a group: K's of the keys kappa(g), kappa(g) + 2, or V's of the keys 4t, 4t + 1 and 4t + 2, 4t + 3.
template <int HD>
struct Words4 {
    uint32_t w[2][HD / 32];
};

template <int HD>
__device__ __forceinline__ Words4<HD> words4(const uint8_t* group, int lane)
{
    Words4<HD> r;
    const uint4 x = *reinterpret_cast<const uint4*>(group + lane * 16);
    if constexpr (HD == 128) {
        const uint4 y = *reinterpret_cast<const uint4*>(group + 512 + lane * 16);
        r.w[0][0] = x.x, r.w[0][1] = x.y, r.w[0][2] = x.z, r.w[0][3] = x.w;
        r.w[1][0] = y.x, r.w[1][1] = y.y, r.w[1][2] = y.z, r.w[1][3] = y.w;
    } else {
        r.w[0][0] = x.x, r.w[0][1] = x.y;
        r.w[1][0] = x.z, r.w[1][1] = x.w;
    }
    return r;
}

// The scale bytes that go with them: K's of key kappa(g), then kappa(g) + 2 (d = 128: two blocks each), V's of keys 4t to 4t + 3.
template <int HD>
__device__ __forceinline__ uint32_t k_scales4(const uint8_t* group, int lane)
{
    if constexpr (HD == 128) return *reinterpret_cast<const uint32_t*>(group + Group4<HD>::kCodes + lane * 4);
    else return *reinterpret_cast<const uint16_t*>(group + Group4<HD>::kCodes + lane * 2);
}

template <int HD>
__device__ __forceinline__ uint32_t v_scales4(const uint8_t* group, int lane)
{
    return *reinterpret_cast<const uint32_t*>(group + Group4<HD>::kCodes + (HD == 128 ? lane >> 2 : lane >> 3) * 16 + (lane & 3) * 4);
}

// Two 16-bit values of the I/O type as f16 (bf16: what f16 does not reach is taken as its largest number).
template <bool BF16>
__device__ __forceinline__ uint32_t to_f16x2(uint32_t x)
{
    if constexpr (!BF16) return x;
    uint32_t r;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(__uint_as_float(x & 0xffff0000u)), "f"(__uint_as_float(x << 16)));
    return r;
}

// The power of two that a bf16 row is multiplied by on its way to f16, and the
// one that brings its products back, from the bits of its largest magnitude: that comes to lie
// between 2^14 and 2^15.
struct QScale4 {
    float mul, back;
};

__device__ __forceinline__ QScale4 q_scale4(uint32_t most)
{
    const int e = min(max(static_cast<int>(most >> 7) - 14, 1), 253);
    return QScale4{__uint_as_float(static_cast<uint32_t>(254 - e) << 23), __uint_as_float(static_cast<uint32_t>(e) << 23)};
}

// The 8 values of a word as bf16 pairs, exactly: 16 + c + 8 in bf16 has the code at bits 3-6. s: the two scales in bf16.
__device__ __forceinline__ void values4_bf16(uint32_t w, uint32_t s, uint32_t n24, uint32_t (&r)[4])
{
    const uint32_t b = __byte_perm(w, 0u, 0x2301);
    auto fma = [&](uint32_t x) -> uint32_t {
        uint32_t y;
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(and_or<0x00780078u, 0x41804180u>(x)), "r"(s), "r"(n24));
        return y;
    };
    r[0] = fma(w >> 3);
    r[1] = fma(w << 1);
    r[2] = fma(b >> 3);
    r[3] = fma(b << 1);
}

// The scale byte of a block whose largest magnitude is `most` (the bits of an fp32; those of an infinity or a NaN are
// above every number's), and 1 / s to within 2^-22 (0 where the scale is 0 or NaN: every code is 0 or of no account).
// The border between two scales, 7 times a number of 5 bits, and the inputs' 11 bits are on one grid: most / 7 is at
// least 2^-11 of itself away from a border that it is not on, and the product with 1 / 7 within 2^-23 of it. So the
// product is first rounded to 2^-12 of its power of two, which puts what is on a border there, then to 2^-3 (ties to
// even). Rounding is done by adding a power of two whose unit in the last place is the grid's.
// `wide`: codes may pass 7: the scale ends at 240, and is coarse below 2^-14.
__device__ __forceinline__ uint32_t scale_byte4(uint32_t most, float& inv, bool& wide)
{
    const float v = fminf(__fmul_rn(__uint_as_float(most), 0.14285714924335479736f), kMaxScale4);
    const uint32_t e = max(__float_as_uint(v) >> 23, 113u);     // (below 2^-14: the step of 2^-14)
    const float fine = __uint_as_float((e + 11) << 23), coarse = __uint_as_float((e + 20) << 23);
    const float s = __fsub_rn(__fadd_rn(__fadd_rn(v, fine), __fsub_rn(coarse, fine)), coarse);
    wide = v >= kMaxScale4 || e == 113u;
    const bool bad = most >= 0x7f800000u;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    inv = s > 0.f && !bad ? r : 0.f;
    return bad ? kNanScale4 : static_cast<uint32_t>(__half_as_ushort(__float2half_rn(s))) >> 7;
}

// rint(x / s) + 8 in the low 4 bits of each of two numbers, -8 to 7 where it is in that range; the bits below 16 above
// them are 0. A border (k + 1/2) s, 8 bits, is on the grid of x: x / s is at least 2^-12 away from a border that it is not
// on, and x * inv within 2^-19 of itself; rounding the product to multiples of 2^-14 puts what is on a border there, and
// then ties go to even.
__device__ __forceinline__ uint64_t code4_2(uint64_t x, uint64_t inv)
{
    // 768: unit in the last place 2^-14; 2^23 + 2^22 + 8: units, the code in the lowest bits
    constexpr uint64_t kFine = 0x4440000044400000ull;
    constexpr uint32_t kOnes = 0x4b400000u + 8 - 768;           // bits of 12582920 - 768
    uint64_t y;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(x), "l"(inv));
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(y) : "l"(kFine));
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(y) : "l"((static_cast<uint64_t>(kOnes) << 32) | kOnes));
    return y;
}

// Four codes each (low 4 bits; the other bits below 16 are 0) as a word's low and high half.
__device__ __forceinline__ uint32_t pack_word4(const uint32_t (&lo)[4], const uint32_t (&hi)[4])
{
    const uint32_t a = __byte_perm(lo[0] * 16 + lo[1], hi[0] * 16 + hi[1], 0x5410) << 2;
    const uint32_t b = __byte_perm(lo[2] * 16 + lo[3], hi[2] * 16 + hi[3], 0x5410) << 2;
    return a | __byte_perm(b, 0u, 0x2301);
}

}  // namespace swa

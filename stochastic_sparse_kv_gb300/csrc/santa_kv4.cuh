// santa_kv4.cuh -- the 4-bit KV cache: its number format, and the kernels that write rows
// into it and read them back, sm_103a.
//
// A cache row of D values is D/16 groups of 16.  A group x has one scale and 16 codes:
//   s = the UE5M3 number nearest max|x| / 6 (ties to even), at most 10240
//   c = sign(x) and the index of the value of {0, .5, 1, 1.5, 2, 3, 4, 6} nearest |x| / s
//       (ties to the even index): the E2M1 code
// and stands for x^ = sign * grid[index] * s.  UE5M3 is an unsigned 8-bit float, 5 exponent
// bits (bias 15) and 3 mantissa bits: the top byte-and-a-half of a non-negative fp16, so a
// scale is decoded by one shift, and its range (2^-17 .. 10240) covers keys and values
// without a second scale per tensor.  A group that holds a NaN or an infinity gets the
// scale 0xff (a NaN): the whole group reads back as NaN.
//
// Exactness.  A code has at most 2 significant bits and a scale 4, so x^ has at most 6 and
// a magnitude in [2^-18, 61440]: fp16 and bf16 both hold it exactly, and reading rounds
// nothing.  When writing, max|x| / 6 and |x| / s are quotients of short integers (8 by 2 and
// 8 by 4 significant bits): a quotient is either a tie of the coarser format exactly or at
// least 2^-12 (relative) away from one, and the fp32 quotient (2^-24) decides as the real
// number would.
#pragma once

#include <cuda_fp16.h>

#include "santa_common.cuh"

namespace santa {

constexpr int KV_GROUP = 16;              // values per scale
constexpr int KV_NT = 256;                // threads per CTA of the write and read kernels
constexpr uint32_t UE5M3_MAX = 0xE2;      // 10240: 6 * 10240 still fits fp16
constexpr uint32_t UE5M3_NAN = 0xFF;

// The scale code of a group whose largest |x| has the bf16 bits amax (sign cleared).
__device__ __forceinline__ uint32_t ue5m3_scale(uint32_t amax)
{
    if (amax >= 0x7f80u) return UE5M3_NAN;
    const float want = __fdiv_rn(__uint_as_float(amax << 16), 6.f);
    if (want < 0x1p-14f) return (uint32_t)__float2int_rn(want * 0x1p17f);  // below the normal range
    const uint32_t u = __float_as_uint(want);
    const uint32_t r = (u + 0x7ffffu + ((u >> 20) & 1u)) >> 20;            // 8 exponent, 3 mantissa bits
    return min(r - ((127u - 15u) << 3), UE5M3_MAX);
}

// A scale as fp16 (exact): its bits are the fp16's bits 7-14.
__device__ __forceinline__ __half ue5m3_half(uint32_t code) { return __ushort_as_half((unsigned short)(code << 7)); }

// Eight E2M1 codes (value i in bits 4i..4i+3), each x rounded to the grid, ties to even.
__device__ __forceinline__ uint32_t e2m1_pack8(const float (&x)[8])
{
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

// The four bytes of w as fp16 pairs: h[i] = (low nibble, high nibble) of byte i, unscaled.
__device__ __forceinline__ void e2m1_unpack8(uint32_t w, uint32_t (&h)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

__device__ __forceinline__ uint32_t h2mul(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Rows moved between a 4-bit cache and bf16 rows.
struct Kv4Move {
    uint8_t *code[2], *scale[2];      // K, V: [B][H_kv][n_max][D/2], [B][H_kv][n_max][D/16]
    uint16_t *row[2];                 // bf16 rows; strides in elements
    long long sb[2], st[2], sh[2];    // batch, token, head
    const int32_t *pos, *counts;      // first cache row of each batch row; live tokens (NULL: T)
    int32_t *ctrl;                    // device error word (or NULL)
    int B, H_kv, D, n_max, T;
};

// One thread moves one group (32 bytes of bf16, 8 bytes of codes, 1 of scale); consecutive
// threads take the groups of a row, then the tokens of a head, so that a warp's cache side
// is contiguous.  Returns whether the thread has a live group.
__device__ __forceinline__ bool kv4_group(const Kv4Move &m, size_t &crow, int &grp, const uint16_t *&src)
{
    const int ng = m.D / KV_GROUP;
    const uint32_t idx = blockIdx.x * (uint32_t)KV_NT + threadIdx.x;
    const uint32_t row = idx / (uint32_t)ng;
    grp = (int)(idx % (uint32_t)ng);
    const uint32_t bh = row / (uint32_t)m.T;
    const int t = (int)(row % (uint32_t)m.T);
    const int b = (int)(bh / (uint32_t)m.H_kv), h = (int)(bh % (uint32_t)m.H_kv);
    if (b >= m.B) return false;
    const int which = blockIdx.y;
    const int first = m.pos[b], cnt = m.counts ? m.counts[b] : m.T;
    if (first < 0 || cnt < 0 || cnt > m.T || first > m.n_max - cnt) {
        if (m.ctrl && which == 0 && h == 0 && t == 0 && grp == 0) set_dev_error(m.ctrl, DEV_BAD_POSITION);
        return false;
    }
    if (t >= cnt) return false;
    crow = ((size_t)b * m.H_kv + h) * m.n_max + (size_t)(first + t);
    src = m.row[which] + (b * m.sb[which] + t * m.st[which] + h * m.sh[which] + grp * KV_GROUP);
    return true;
}

// New rows into the cache.
__global__ void __launch_bounds__(KV_NT) santa_kv4_append_kernel(const Kv4Move m)
{
    size_t crow;
    int grp;
    const uint16_t *src;
    if (!kv4_group(m, crow, grp, src)) return;
    const uint4 *s4 = reinterpret_cast<const uint4 *>(src);
    const uint4 a = s4[0], b = s4[1];
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max(amax, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
    const uint32_t sc = ue5m3_scale(amax);
    uint32_t c[2] = {0, 0};
    if (sc != 0 && sc != UE5M3_NAN) {
        const float s = __half2float(ue5m3_half(sc));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __fdiv_rn(bf16lo_to_f32(w[4 * j + i]), s);
                x[2 * i + 1] = __fdiv_rn(bf16hi_to_f32(w[4 * j + i]), s);
            }
            c[j] = e2m1_pack8(x);
        }
    }
    const int which = blockIdx.y;
    *reinterpret_cast<uint2 *>(m.code[which] + crow * (m.D / 2) + grp * 8) = make_uint2(c[0], c[1]);
    m.scale[which][crow * (m.D / KV_GROUP) + grp] = (uint8_t)sc;
}

// Cache rows back to bf16.
__global__ void __launch_bounds__(KV_NT) santa_kv4_read_kernel(const Kv4Move m)
{
    size_t crow;
    int grp;
    const uint16_t *src;
    if (!kv4_group(m, crow, grp, src)) return;
    const int which = blockIdx.y;
    const uint2 c = *reinterpret_cast<const uint2 *>(m.code[which] + crow * (m.D / 2) + grp * 8);
    const float s = __half2float(ue5m3_half(m.scale[which][crow * (m.D / KV_GROUP) + grp]));
    uint4 *dst = reinterpret_cast<uint4 *>(const_cast<uint16_t *>(src));
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t h[4], o[4];
        e2m1_unpack8(j ? c.y : c.x, h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
            const __nv_bfloat162 v = __floats2bfloat162_rn(f.x * s, f.y * s);
            o[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
        dst[j] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

}  // namespace santa

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
// Exactness.  A code has at most 2 significant bits and a scale 4, so x^ has at most 6 and a
// magnitude in [2^-18, 61440]: fp16 and bf16 both hold it exactly, and reading rounds nothing.
// Writing rounds the quotients max|x| / 6 and |x| / s as the real numbers: they are quotients of
// integers of 8 bits by 2 and by 4 bits, a border of the rounding (5 and 3 bits) times its
// divisor is an integer of the same grid as the dividend, so a quotient lies on a border exactly
// or at least 2^-8 of itself away.  An fp32 product with the reciprocal (off by less than 2^-21)
// rounded to 16 bits is on the border or on the same
// side of it.
//
// Both kernels move 2.56 bytes a value and are bound by that: one thread takes one group of K
// and of V, in one 32-byte access where the rows allow it.  4 rows of 32k tokens, 8 heads, d = 128:
// read back in 103-105 us, 6.6 TB/s, 0.98 of the measured copy rate (16-byte accesses and index
// divisions: 127 us).  8k tokens written and read back in 53-54 us, 51 at the copy rate (dividing
// exactly, 16 times a group: 85 us).
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
    const float sixth = __uint_as_float(amax << 16) * (1.f / 6.f);
    const uint32_t u = (__float_as_uint(sixth) + 0x80u) & ~0xffu;  // 16 bits
    const float want = __uint_as_float(u);
    if (want < 0x1p-14f) return (uint32_t)__float2int_rn(want * 0x1p17f);  // below the normal range
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

// Two fp32 operations in one instruction.
__device__ __forceinline__ void add2(float &a, float &b, float x, float y)
{
    asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
        "add.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(x), "f"(y));
}

// (a, b) * (x, y) + (u, v)
__device__ __forceinline__ float2 fma2(float a, float b, float x, float y, float u, float v)
{
    float2 r;
    asm("{\n\t.reg .b64 p, q, s;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tmov.b64 s, {%6, %7};\n\t"
        "fma.rn.f32x2 p, p, q, s;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a), "f"(b), "f"(x), "f"(y), "f"(u), "f"(v));
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
    int H_kv, n_max, T;
};

// A thread's group, of K and of V: blockIdx.y is a (batch row, head) pair; consecutive threads
// take the groups of a row, then the tokens, so that a warp's cache side is contiguous.
// Returns whether the thread has a live group; its place in the cache and its bf16 values.
template <int D>
__device__ __forceinline__ bool kv4_group(const Kv4Move &m, size_t &place, uint16_t *(&row)[2])
{
    constexpr int NG = D / KV_GROUP;
    const int idx = blockIdx.x * blockDim.x + threadIdx.x;
    const int t = idx / NG, grp = idx % NG;
    const int b = (int)(blockIdx.y / (unsigned)m.H_kv), h = (int)(blockIdx.y % (unsigned)m.H_kv);
    const int first = m.pos[b], cnt = m.counts ? m.counts[b] : m.T;
    if (first < 0 || cnt < 0 || cnt > m.T || first > m.n_max - cnt) {
        if (m.ctrl && idx == 0 && h == 0) set_dev_error(m.ctrl, DEV_BAD_POSITION);
        return false;
    }
    if (t >= cnt) return false;
    place = ((size_t)blockIdx.y * m.n_max + (size_t)(first + t)) * NG + grp;
#pragma unroll
    for (int i = 0; i < 2; ++i) row[i] = m.row[i] + (b * m.sb[i] + t * m.st[i] + h * m.sh[i] + grp * KV_GROUP);
    return true;
}

// Code and scale of one group: its bf16 bits in pairs.
__device__ __forceinline__ uint2 kv4_encode(const uint32_t (&w)[8], uint32_t &scale)
{
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = __vmaxu2(amax, w[i] & 0x7fff7fffu);
    amax = max(amax & 0xffffu, amax >> 16);
    scale = ue5m3_scale(amax);
    if (scale == 0 || scale == UE5M3_NAN) return make_uint2(0, 0);
    const float inv = __frcp_rn(__half2float(ue5m3_half(scale)));
    uint32_t c[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // t rounded to 16 bits: u - (u - t) with u = (2^8 + 1) t (Veltkamp's splitting)
            const float2 t = fma2(bf16lo_to_f32(w[4 * j + i]), bf16hi_to_f32(w[4 * j + i]), inv, inv, -0.f, -0.f);
            const float2 u = fma2(t.x, t.y, 257.f, 257.f, -0.f, -0.f);
            const float2 d = fma2(t.x, t.y, -1.f, -1.f, u.x, u.y);
            const float2 y = fma2(d.x, d.y, -1.f, -1.f, u.x, u.y);
            x[2 * i] = y.x;
            x[2 * i + 1] = y.y;
        }
        c[j] = e2m1_pack8(x);
    }
    return make_uint2(c[0], c[1]);
}

// New rows into the cache.  WIDE: the rows are 32-byte aligned.
template <int D, bool WIDE>
__global__ void __launch_bounds__(KV_NT) santa_kv4_append_kernel(const Kv4Move m)
{
    size_t place;
    uint16_t *row[2];
    if (!kv4_group<D>(m, place, row)) return;
    uint32_t w[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (WIDE) {
            asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3]), "=r"(w[i][4]), "=r"(w[i][5]), "=r"(w[i][6]),
                           "=r"(w[i][7])
                         : "l"(__cvta_generic_to_global(row[i])));
        } else {
            const uint4 a = reinterpret_cast<const uint4 *>(row[i])[0], b = reinterpret_cast<const uint4 *>(row[i])[1];
            w[i][0] = a.x, w[i][1] = a.y, w[i][2] = a.z, w[i][3] = a.w, w[i][4] = b.x, w[i][5] = b.y, w[i][6] = b.z, w[i][7] = b.w;
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t sc;
        reinterpret_cast<uint2 *>(m.code[i])[place] = kv4_encode(w[i], sc);
        m.scale[i][place] = (uint8_t)sc;
    }
}

// Cache rows back to bf16.
template <int D, bool WIDE>
__global__ void __launch_bounds__(KV_NT) santa_kv4_read_kernel(const Kv4Move m)
{
    size_t place;
    uint16_t *row[2];
    if (!kv4_group<D>(m, place, row)) return;
    uint2 c[2];
    float s[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        c[i] = reinterpret_cast<const uint2 *>(m.code[i])[place];
        s[i] = __half2float(ue5m3_half(m.scale[i][place]));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t h[4];
            e2m1_unpack8(j ? c[i].y : c[i].x, h);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[x]));
                const __nv_bfloat162 v = __floats2bfloat162_rn(f.x * s[i], f.y * s[i]);
                o[4 * j + x] = *reinterpret_cast<const uint32_t *>(&v);
            }
        }
        if (WIDE) {
            asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]),
                         "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7]), "l"(__cvta_generic_to_global(row[i]))
                         : "memory");
        } else {
            reinterpret_cast<uint4 *>(row[i])[0] = make_uint4(o[0], o[1], o[2], o[3]);
            reinterpret_cast<uint4 *>(row[i])[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
}

}  // namespace santa

// santa_window.cuh -- exact decode attention over the visible keys of a sequence, for a
// bf16 cache and for the 4-bit cache of santa_kv4.cuh, sm_103a.
//
//   o = sum_j p_j v_j,  p = softmax over visible j of scale q.k_j
//   visible(j):  j < n  and  (window == 0  or  j >= n - window  or  j < sinks)
//
// The decoding token is the sequence's last key.  A sequence without keys gives zeros.
#pragma once

#include "santa_kv4.cuh"

namespace santa {

struct WinParams {
    const uint16_t *q;            // bf16 [B][H_q][D]
    const uint8_t *k, *v;         // bf16 rows, or 4-bit codes
    const uint8_t *ks, *vs;       // scales of a 4-bit cache
    const int32_t *seq_lens;
    float *out;
    int32_t *ctrl;
    int B, H_q, H_kv, n_max, G;
    int window, sinks;
    int out_bf16;
    float k2;                     // scale * log2(e)
};

constexpr int WN_NT = 256;

template <int D, bool KV4>
__device__ __forceinline__ void load_row(const uint8_t *rows, const uint8_t *scales, size_t row, int lane, float (&x)[D / 32])
{
    constexpr int E = D / 32;
    if (KV4) {
        const float s = __half2float(ue5m3_half(scales[row * (D / KV_GROUP) + lane * E / KV_GROUP]));
        const uint8_t *c = rows + row * (D / 2) + lane * E / 2;
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            uint32_t h[4];
            e2m1_unpack8(c[i], h);
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[0]));
            x[2 * i] = f.x * s;
            x[2 * i + 1] = f.y * s;
        }
    } else {
        const uint32_t *r = reinterpret_cast<const uint32_t *>(rows + row * (D * 2)) + lane * E / 2;
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            x[2 * i] = bf16lo_to_f32(r[i]);
            x[2 * i + 1] = bf16hi_to_f32(r[i]);
        }
    }
}

// One CTA per (batch row, query head); its warps take alternate visible keys and join their
// (maximum, sum, output) through shared memory.
template <int D, bool KV4>
__global__ void __launch_bounds__(WN_NT) santa_window_kernel(const WinParams p)
{
    constexpr int E = D / 32, NW = WN_NT / 32;
    __shared__ float sm[NW], sl[NW], so[NW][D];
    const int b = blockIdx.x / p.H_q, h = blockIdx.x % p.H_q, g = h / p.G;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int n = p.seq_lens[b];
    if (n < 0 || n > p.n_max) {
        if (threadIdx.x == 0 && h == 0) set_dev_error(p.ctrl, DEV_BAD_SEQLEN);
        n = 0;
    }
    const int w0 = p.window > 0 ? max(0, n - p.window) : 0;
    const int se = min(p.sinks, w0);
    const int nv = se + n - w0;
    float q[E], o[E] = {};
    const uint16_t *qh = p.q + ((size_t)b * p.H_q + h) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) q[e] = __uint_as_float((uint32_t)qh[e] << 16);
    float m = __int_as_float(0xff800000), l = 0.f;
    for (int i = warp; i < nv; i += NW) {
        const size_t row = ((size_t)b * p.H_kv + g) * p.n_max + (size_t)(i < se ? i : w0 + i - se);
        float k[E], v[E];
        load_row<D, KV4>(p.k, p.ks, row, lane, k);
        load_row<D, KV4>(p.v, p.vs, row, lane, v);
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= p.k2;
        const float mn = fmaxf(m, s);
        const float f = m == mn ? 1.f : exp2f(m - mn), w = exp2f(s - mn);
        l = l * f + w;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(w, v[e], o[e] * f);
        m = mn;
    }
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
    __syncthreads();
    if (threadIdx.x < D) {
        float M = sm[0];
        for (int w = 1; w < NW; ++w) M = fmaxf(M, sm[w]);
        float L = 0.f, O = 0.f;
        for (int w = 0; w < NW; ++w) {
            const float f = sm[w] == M ? 1.f : exp2f(sm[w] - M);
            L = fmaf(f, sl[w], L);
            O = fmaf(f, so[w][threadIdx.x], O);
        }
        const float r = nv > 0 ? O / L : 0.f;
        const size_t i = ((size_t)b * p.H_q + h) * D + threadIdx.x;
        if (p.out_bf16)
            reinterpret_cast<__nv_bfloat16 *>(p.out)[i] = __float2bfloat16_rn(r);
        else
            p.out[i] = r;
    }
}

}  // namespace santa

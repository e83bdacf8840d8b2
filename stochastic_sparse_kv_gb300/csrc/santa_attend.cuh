// santa_attend.cuh -- exact causal attention of a chunk of new tokens over a paged cache, sm_103a.
//
//   o = sum_j p_j v_j,  p = softmax over visible j of scale q.k_j
//   visible(j):  j <= P  and  (window == 0  or  j > P - window  or  j < sinks)
//
// for the token at position P.
#pragma once

#include "santa_common.cuh"

namespace santa {

struct AttendParams {
    const uint16_t *q;
    long long q_sb, q_st, q_sh;   // elements, for (batch, token, head)
    const uint16_t *k, *v;
    const int32_t *table, *pos, *counts;
    uint16_t *out;
    int32_t *ctrl;
    int B, T, H_q, H_kv, G, n_max, cols, n_pages, page_shift;
    int window, sinks;
    float k2;                     // scale log2 e
    uint64_t wait_ns;
};

// One warp a (token, head): the plainest form.
template <int D>
__global__ void __launch_bounds__(128) santa_attend_kernel(const AttendParams p)
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (w >= (long long)p.T * p.H_q) return;
    const int b = blockIdx.y, t = (int)(w / p.H_q), h = (int)(w % p.H_q);
    const int first = p.pos[b], cnt = p.counts ? p.counts[b] : p.T;
    if (first < 0 || cnt < 0 || cnt > p.T || first > p.n_max - cnt) {
        if (w == 0 && lane == 0) set_dev_error(p.ctrl, DEV_BAD_POSITION);
        return;
    }
    if (t >= cnt) return;
    const int P = first + t;
    float q[E], o[E], m = __int_as_float(0xff800000), l = 0.f;
    for (int e = 0; e < E; ++e) {
        q[e] = bf16lo_to_f32(p.q[b * p.q_sb + t * p.q_st + h * p.q_sh + lane * E + e]);
        o[e] = 0.f;
    }
    const int lo = p.window > 0 ? max(0, P - p.window + 1) : 0;
    for (int j = p.sinks > 0 && lo > 0 ? 0 : lo; j <= P; ++j) {
        if (j >= p.sinks && j < lo) j = lo;
        const int page = p.table[(size_t)b * p.cols + (j >> p.page_shift)];
        const bool good = (unsigned)page < (unsigned)p.n_pages;
        if (!good && lane == 0) set_dev_error(p.ctrl, DEV_BAD_PAGE);
        const long long row = ((((long long)(good ? page : 0) * p.H_kv + h / p.G) << p.page_shift) + (j & ((1 << p.page_shift) - 1))) * D;
        float s = 0.f;
        for (int e = 0; e < E; ++e) s += q[e] * (good ? bf16lo_to_f32(p.k[row + lane * E + e]) : 0.f);
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        const float mn = fmaxf(m, s), ref = mn == __int_as_float(0xff800000) ? 0.f : mn;
        const float f = exp2f((m - ref) * p.k2), w1 = exp2f((s - ref) * p.k2);
        m = mn;
        l = l * f + w1;
        for (int e = 0; e < E; ++e) o[e] = o[e] * f + w1 * (good ? bf16lo_to_f32(p.v[row + lane * E + e]) : 0.f);
    }
    for (int e = 0; e < E; ++e)
        p.out[(((size_t)b * p.T + t) * p.H_q + h) * D + lane * E + e] = __bfloat16_as_ushort(__float2bfloat16_rn(o[e] / l));
}

}  // namespace santa

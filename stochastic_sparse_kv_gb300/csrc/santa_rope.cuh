// santa_rope.cuh -- rotary positions, and the rows of new tokens written into a paged cache,
// sm_103a.
//
//   (x, y) -> A (x cos a - y sin a, x sin a + y cos a),  a = p f_i
//
// for the pairs i of a head's first `rot` features at position p.  f_i is held as turns a position
// in units of 2^-64, so that p f_i modulo one turn is one 64-bit product modulo 2^64: exact, at any
// position, with no fp64 (slow on this part) and no reduction of a large angle.  Its signed value
// over 2^63 is the angle in half turns, in [-1, 1), rounded once to fp32.
//
// One kernel serves the rotation alone and a step's q, K and V together: the heads of a token are
// those of q, then K, then V.  A thread takes 16 features of up to RP_HEADS heads of a token, so that its
// eight angles serve them all (the sines of one head are as much work as moving it), and reads
// RP_AHEAD rows before it uses the first.
//
// Bound by bytes, 4 a value.  Rows of 4 x 8192 tokens, 32 heads, d = 128: 537 MB in 82 us, 6.5 TB/s, 0.98 of
// the measured copy rate (a head a thread: 141 us).  4 x 2048 tokens of 32 + 8 + 8 heads into pages of 16:
// 201 MB in 37 us, 0.81 (59 us).  With 4 CTAs an SM (64 registers): rows ahead and heads a
// thread 3 and 6 82 and 37 us, 2 and 4 84 and 37, 2 and 8 84 and 39, 4 and 8 91 and 44; 3 CTAs
// 4 and 4 86 and 37; 6 CTAs 2 and 4 92 and 41.
#pragma once

#include "santa_common.cuh"

namespace santa {

constexpr int RP_NT = 256;
constexpr int RP_VALUES = 16;             // features a thread moves of a row
constexpr int RP_AHEAD = 3;               // rows that a thread has in flight
constexpr int RP_HEADS = 6;               // rows a thread moves at the most (its angles serve them all)

// Rows of one kind; strides in elements for (batch, token, head).
struct RopeRows {
    const uint16_t *src;
    uint16_t *dst;
    long long sb, st, sh;                 // of src
    long long db, dt, dh;                 // of dst (rows; pages are addressed through the table)
};

struct RopeParams {
    RopeRows q, k, v;
    int H_q, H_kv;                        // heads of q, of K and of V (H_kv = 0: q alone)
    int T, B, rot;                        // rot = 0: nothing is rotated
    int clear;                            // rows of q that no live token writes become zeros
    int groups;                           // threads that share a token's heads: each takes every groups-th
    const uint64_t *turns;
    float amplitude;
    const int32_t *pos, *counts;          // counts NULL: T
    int last;                             // largest pos + counts
    const int32_t *table;                 // [B][cols]
    int cols, n_pages, page_shift;
    int32_t *ctrl;                        // device error word (or NULL)
};

// A thread's 16 features as two 16-byte accesses, and what it does with them.
template <int D, bool PAIRS>
__global__ void __launch_bounds__(RP_NT, 4) santa_rope_kernel(const RopeParams p)
{
    constexpr int NU = D / RP_VALUES;
    const int b = blockIdx.y;
    const int idx = blockIdx.x * blockDim.x + threadIdx.x;
    const int c = idx % NU, slot = idx / NU;
    const int g = slot % p.groups, t = slot / p.groups;
    const int first = p.pos[b], cnt = p.counts ? p.counts[b] : p.T;
    const bool skip = first < 0 || cnt < 0 || cnt > p.T || first > p.last - cnt;
    if (skip && p.ctrl && idx == 0) set_dev_error(p.ctrl, DEV_BAD_POSITION);
    if (skip || t >= cnt) {
        if (!p.clear || t >= p.T) return;
        for (int h = g; h < p.H_q; h += p.groups) {
            uint16_t *dst = p.q.dst + (b * p.q.db + t * p.q.dt + h * p.q.dh) + RP_VALUES * c;
            *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<uint4 *>(dst + 8) = make_uint4(0, 0, 0, 0);
        }
        return;
    }
    const int at = first + t;
    const bool turn = RP_VALUES * c < p.rot;
    // where the two halves of this thread's features begin
    const int f0 = PAIRS || !turn ? RP_VALUES * c : 8 * c;
    const int f1 = PAIRS || !turn ? f0 + 8 : p.rot / 2 + 8 * c;
    float cs[8], sn[8];
    if (turn) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint64_t a = (uint64_t)(uint32_t)at * p.turns[8 * c + i];
            sincospif(__ll2float_rn((long long)a) * 0x1p-63f, &sn[i], &cs[i]);
            cs[i] *= p.amplitude;
            sn[i] *= p.amplitude;
        }
    }
    // this token's row 0 of its page (head 0)
    long long place = -1;
    if (p.H_kv > 0) {
        const int entry = p.table[(size_t)b * p.cols + (at >> p.page_shift)];
        if ((unsigned)entry < (unsigned)p.n_pages)
            place = (((long long)entry * p.H_kv << p.page_shift) + (at & ((1 << p.page_shift) - 1))) * D;
        else if (p.ctrl && g == 0 && c == 0)
            set_dev_error(p.ctrl, DEV_BAD_PAGE);
    }
    const int heads = p.H_q + 2 * p.H_kv;
    // RP_AHEAD rows are read before the first of them is used
    for (int h0 = g; h0 < heads; h0 += RP_AHEAD * p.groups) {
        uint4 u[RP_AHEAD], w[RP_AHEAD];
        uint16_t *dst[RP_AHEAD];
        bool rotate[RP_AHEAD];
#pragma unroll
        for (int x = 0; x < RP_AHEAD; ++x) {
            const int h = h0 + x * p.groups;
            const uint16_t *src;
            dst[x] = nullptr;
            if (h >= heads || (h >= p.H_q && place < 0)) continue;
            if (h < p.H_q) {
                src = p.q.src + (b * p.q.sb + t * p.q.st + h * p.q.sh);
                dst[x] = p.q.dst + (b * p.q.db + t * p.q.dt + h * p.q.dh);
                rotate[x] = turn;
            } else {
                const bool value = h - p.H_q >= p.H_kv;
                const int hk = h - p.H_q - (value ? p.H_kv : 0);
                src = value ? p.v.src + (b * p.v.sb + t * p.v.st + hk * p.v.sh) : p.k.src + (b * p.k.sb + t * p.k.st + hk * p.k.sh);
                dst[x] = (value ? p.v.dst : p.k.dst) + (place + ((long long)hk << p.page_shift) * D);
                rotate[x] = turn && !value;
            }
            // (a row of V is copied in the same two pieces)
            u[x] = *reinterpret_cast<const uint4 *>(src + f0);
            w[x] = *reinterpret_cast<const uint4 *>(src + f1);
        }
#pragma unroll
        for (int x = 0; x < RP_AHEAD; ++x) {
            if (!dst[x]) continue;
            if (rotate[x]) {
                uint32_t a[4] = {u[x].x, u[x].y, u[x].z, u[x].w}, e[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (PAIRS) {
                        // words 0-3 hold pairs 0-3 of this thread, words 4-7 pairs 4-7
                        const float x0 = bf16lo_to_f32(a[i]), y0 = bf16hi_to_f32(a[i]);
                        const float x1 = bf16lo_to_f32(e[i]), y1 = bf16hi_to_f32(e[i]);
                        a[i] = bf16x2(x0 * cs[i] - y0 * sn[i], x0 * sn[i] + y0 * cs[i]);
                        e[i] = bf16x2(x1 * cs[4 + i] - y1 * sn[4 + i], x1 * sn[4 + i] + y1 * cs[4 + i]);
                    } else {
                        const float x0 = bf16lo_to_f32(a[i]), x1 = bf16hi_to_f32(a[i]);
                        const float y0 = bf16lo_to_f32(e[i]), y1 = bf16hi_to_f32(e[i]);
                        a[i] = bf16x2(x0 * cs[2 * i] - y0 * sn[2 * i], x1 * cs[2 * i + 1] - y1 * sn[2 * i + 1]);
                        e[i] = bf16x2(x0 * sn[2 * i] + y0 * cs[2 * i], x1 * sn[2 * i + 1] + y1 * cs[2 * i + 1]);
                    }
                }
                u[x] = make_uint4(a[0], a[1], a[2], a[3]);
                w[x] = make_uint4(e[0], e[1], e[2], e[3]);
            }
            *reinterpret_cast<uint4 *>(dst[x] + f0) = u[x];
            *reinterpret_cast<uint4 *>(dst[x] + f1) = w[x];
        }
    }
}

}  // namespace santa

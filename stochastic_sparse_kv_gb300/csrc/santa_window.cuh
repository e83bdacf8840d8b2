// santa_window.cuh -- exact decode attention over the visible keys of a sequence, for a
// bf16 cache and for the 4-bit cache of santa_kv4.cuh, sm_103a.
//
//   o = sum_j p_j v_j,  p = softmax over visible j of scale q.k_j
//   visible(j):  j < n  and  (window == 0  or  j >= n - window  or  j < sinks)
//
// The decoding token is the sequence's last key.  A sequence without keys gives zeros.
//
// One launch.  The work is the list of all tiles of TK keys that hold a visible key, over
// all (batch row, KV head) groups; every CTA takes one contiguous share of the list and
// every warp of it a contiguous share of that, so any mix of lengths and windows is spread
// evenly without a queue.  A warp streams its tiles through a ring of its own in shared
// memory, with no barrier between warps, and keeps the group's running sums in registers:
//
//  * scores: mma.sync m16n8k16, A = 16 keys, B = the group's query heads as the 8 columns.
//    The product is 8 columns wide at most, and the 4-bit cache has to pass through
//    registers to become fp16 anyway: a tcgen05 tile (M = 128 from shared memory or TMEM)
//    would add a store and a load of every converted value to save the MMA issue slots,
//    16 of about 280 per 16 keys.
//  * p = 2^(k2 (s - m) + 9), m a score so far, with which the largest p so far lies in [2^9, 2^15]:
//    m moves only when p would exceed that, so most tiles rescale nothing.  The difference of
//    two scores is taken before it is scaled: k2 s - k2 m, each rounded at the size of the
//    score, left the range of p at scores of 1e8 and more.  k2 = |scale| log2 e is one fp32
//    number: its rounding moves p by 2^-25 x ln 2 of p, x = log2(2^9 / p), at most 2^-25 of the
//    leading weight (a second term would turn a score of minus infinity into a NaN).
//  * output: A = V^T (16 of the d dimensions by 16 keys), B = p.  movmatrix turns the score
//    accumulators into that operand in registers.
//
// Precision.  The result is fp32, and the tensor cores round operands to 11 (fp16) or 8
// (bf16) bits and truncate their sums, so: 4-bit values are exact in fp16, q is bf16 times a
// power of two, products are exact; p is split into two fp16 or three bf16 terms (22 or 24
// bits; groups of at most 4 heads put the first two terms side by side in the 8 columns).  The
// second fp16 term is held times 2^11: fp16 ends at 2^-24, and without the factor a p below
// 2^-25 left the numerator and stayed in the denominator.  Few MMA steps are chained before
// their sum is added in fp32 with rounding: two in a score and, in V^T p, two for 4 bits and for
// bf16 at d = 128 with up to 4 heads a group, three with 8 heads, four and six at d = 64.
// (A factor of q below 2^-31 of its head's largest is rounded to a step of 2^-38 of that.)
// Error against 64 bits, over 4 x 32k and 64 x 4k keys, 1 to 8 heads a group and both d, relative
// to the largest output: 4 bits 2.1e-7 to 6.9e-7, bf16 3.7e-7 to 1.1e-6, root mean square
// 1.8e-7 to 3.5e-7 and 3.6e-7 to 5.3e-7 (fp32 products and sums of a library: 3.3e-7 to
// 1.3e-6); one serial fp32 sum over 32k keys had 4e-6.
//
// Groups that one warp holds whole are finished by it.  Pieces of others meet in shared
// memory (their CTA joins them) and, where a group spans CTAs, in the workspace: the last
// CTA to arrive (a counter per group, left at zero) joins the pieces in the order of the
// list, so results do not depend on timing.
//
// What bounds it.  bf16: the cache's bytes.  16 rows, window 8192 + 16 sinks of 32k keys,
// d = 128, 8 KV heads: 538 MB in 81-83 us, 6.5-6.7 TB/s, 0.97-0.99 of the measured copy rate.
// 4-bit: 16 rows of 32k keys, 604 MB, take 107-108 us, 5.6 TB/s, 0.84 of the copy rate (8 heads a
// group 122 us; d = 64, half the bytes, 72 us, 8 heads a group 77).  No unit
// is full (half that batch: 636 warp instructions per 32 keys of a KV head, 0.62 of the issue
// slots, 0.47 of the ALU pipe, which the 128 conversions among them take at half rate, 0.25 of
// the tensor pipe); with four warps to a scheduler neither copies nor arithmetic hide the
// other wholly.  An earlier state's copies took 94-96 us without the arithmetic.  What it
// took from 162 us: chains that begin at zero in the MMA, two fp32 operations an instruction,
// copies by the lanes that use them (bulk copies of a tile by one lane: 126 us against 113; by
// warps of their own: 139-143 against 127), 16 warps (12 of 168 registers: 119 against 110; the
// 128 registers of 16 spill at d = 128: 8 bytes, with 8 heads a group 32 stored and 76 loaded),
// seldom used state in shared memory, joins side by side.
// Small calls: a group of 32 keys 3.8-7.0 us in one CTA; one that spans CTAs 9 us (bf16) or
// 11 us (4 bits) and more.
#pragma once

#include "santa_kv4.cuh"
#include "santa_sample.cuh"
#include "santa_tcgen05.cuh"

namespace santa {

constexpr int WN_MAX_CTAS = 512;          // partial slots in the workspace
constexpr int WN_MAX_WARPS = 16;
constexpr int WN_RED = 4 * 32 * WN_MAX_WARPS;  // floats of a join's partial sums: 4 x max(G D / 4, threads)
constexpr float WN_TOP = 9.f;             // log2 of p where a new maximum puts it
constexpr float WN_SLACK = 6.f;           // and how far above that later ones may be
constexpr float WN_LOW = 2048.f;          // 4-bit: the factor of the second term of p, whose steps are those of 2^-35
// Tiles a warp up to which a group stays in one CTA.  One sequence of 8 KV heads, 4 heads a group,
// alone against split, at 2 tiles and at 4: 4-bit d = 128 1024 keys 11.2 and 12.4 us, 2048 keys
// 14.7 and 12.5; d = 64 8.7 and 11.0, 10.7 and 11.0; bf16 d = 128 256 keys 8.1 and 9.2, 512 keys
// 10.4 and 9.2; d = 64 512 keys 7.3 and 9.1, 1024 keys 8.8 and 9.1.  (d = 64 could go to 4, for
// 0.3 us; with 8 sequences 1.2.)
constexpr int WN_ALONE = 2;
constexpr int WN_SETUP = 2;               // tiles that beginning a group costs about as much as

// One CTA to an SM.  4-bit: 16 warps, each copying its own tiles; bf16: the 8 whose rings fit,
// and one that issues all of their copies.
__host__ __device__ constexpr int win_warps(bool kv4) { return kv4 ? 16 : 8; }
__host__ __device__ constexpr int win_threads(bool kv4) { return 32 * (kv4 ? win_warps(true) : win_warps(false) + 1); }
// Keys of a tile, which is a ring stage, and the stages of a warp's ring (what 227 KB hold).
__host__ __device__ constexpr int win_tile(int D, bool kv4) { return kv4 || D == 64 ? 32 : 16; }
__host__ __device__ constexpr int win_stage(int D, bool kv4)
{
    return kv4 ? win_tile(D, true) * (D + D / 8) : win_tile(D, false) * D * 4;
}
__host__ __device__ constexpr int win_stages(int D, bool kv4) { return !kv4 ? 3 : D == 128 ? 3 : 5; }
// A piece of a group's sums: fp32 o[G][D + 4] (the heads' rows in different banks), m[8], l[8].
__host__ __device__ constexpr int win_piece(int G, int D) { return G * (D + 4) + 16; }

struct WinParams {
    const uint16_t *q;            // bf16 [B][H_q][D]
    const uint8_t *k, *v;         // 4-bit codes (a bf16 cache is read through tensor maps)
    const uint8_t *ks, *vs;       // scales of a 4-bit cache
    const int32_t *seq_lens;
    float *out;
    int32_t *ctrl;
    float *first;                 // [CTAs][warps] pieces: a warp's first group, begun before its share
    float *part;                  // [CTAs][2] pieces: a group begun before the CTA's share, one not ended in it
    int B, H_q, H_kv, n_max, G;
    int window, sinks;
    int out_bf16;
    float k2;                     // |scale| * log2(e)
    float qsign;                  // the sign of scale
    uint64_t wait_ns;             // bf16: limit of a stage's wait
};

struct WinSmem {
    int ring, bar, seg, stop, flag, list, group, nb, prefix, total;
};

__host__ __device__ inline WinSmem win_smem(int D, bool kv4, int B)
{
    const int W = win_warps(kv4), ns = win_stages(D, kv4);
    WinSmem s{};
    int off = 0;
    s.ring = off; off += W * ns * win_stage(D, kv4);
    s.bar = off; off += W * ns * 16;             // a full and an empty barrier for each stage
    s.seg = off; off += 2 * W * 4;               // group index of each warp's two pieces, or -1
    s.stop = off; off += (int)align_up((size_t)W * 4, 16);  // set by a warp that gave up
    s.flag = off; off += 16;
    s.list = off; off += 32 * W;
    s.group = off; off += 2 * W * 32;            // each warp's groups: of the tile at hand, of the next to fetch
    s.nb = off; off += (int)align_up((size_t)B * 4, 16);
    s.prefix = off; off += (int)align_up((size_t)(B + 1) * 4, 16);
    s.total = off + (kv4 ? 0 : 1024);            // (swizzled tiles begin at multiples of 1024)
    return s;
}

// ------------------------------------------------------------------ tensor-core pieces

// D = A B (+ D): 16 x 16 by 16 x 8, fp32 sums.  BF16: the operands' type, else fp16.
template <bool BF16>
__device__ __forceinline__ void mma_add(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    if (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <bool BF16>
__device__ __forceinline__ void mma_set(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    if (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Transpose of an 8x8 matrix of 16-bit elements held one row of two per lane.
__device__ __forceinline__ uint32_t movmatrix(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// A barrier of N threads (1: all that work; 2, 3: its halves).
template <int N>
__device__ __forceinline__ void bar_sync(int id = 1)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(N) : "memory");
}

__device__ __forceinline__ float2 unpack_f16(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2 *>(&h)); }

// Whether the phase of that parity has ended (no waiting).
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Wait for the phase with the given parity; give up after limit_ns.  (A limit below a
// microsecond, a diagnostic, polls: a suspended wait may outlast it.)
__device__ __forceinline__ bool win_wait(uint64_t *bar, uint32_t parity, uint64_t limit_ns)
{
    if (mbar_test(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        if (limit_ns >= 1000 ? mbar_try_wait(bar, parity) : mbar_test(bar, parity)) return true;
        if (globaltimer_ns() - t0 > limit_ns) return false;
    }
}

// 16 bytes, global to shared memory, past the L1 cache; groups of them are waited for in order.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(__cvta_generic_to_global(src)) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ------------------------------------------------------------------ the list of tiles
//
// Positions of the list: every group with keys has WN_SETUP positions without work, then one
// for each of its tiles.  Shares are even in positions, so that a run of short groups
// (each costs a load of its queries and a result) is not taken for a few tiles.

// A sequence of n keys: tiles [0, ns) cover the sinks, then tiles tw.. up to the last key.
struct WinTiles {
    int w0, ns, tw, cnt;
};

template <int TK>
__device__ __forceinline__ WinTiles win_tiles(int n, int window, int sinks)
{
    WinTiles t;
    t.w0 = window > 0 ? max(0, n - window) : 0;
    t.tw = t.w0 / TK;
    t.ns = min((min(sinks, t.w0) + TK - 1) / TK, t.tw);
    t.cnt = n > 0 ? t.ns + (n + TK - 1) / TK - t.tw : 0;
    return t;
}

// Positions of a group with cnt tiles.
__device__ __forceinline__ int win_span(int cnt) { return cnt > 0 ? cnt + WN_SETUP : 0; }

// A group of the list: batch row, KV head, its tiles and the position of the first tile.
template <int TK>
struct WinGroup {
    int b, g, n, start;
    WinTiles t;

    // the group of a position
    __device__ __forceinline__ void seek(int pos, const int *prefix, const int *nb, const WinParams &p)
    {
        int lo = 0, hi = p.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (prefix[mid] <= pos) lo = mid; else hi = mid - 1;
        }
        b = lo;
        n = nb[lo];
        t = win_tiles<TK>(n, p.window, p.sinks);
        g = (pos - prefix[lo]) / win_span(t.cnt);
        start = prefix[lo] + g * win_span(t.cnt) + WN_SETUP;
    }
    __device__ __forceinline__ int end() const { return start + t.cnt; }
    __device__ __forceinline__ int index(const WinParams &p) const { return b * p.H_kv + g; }
    __device__ __forceinline__ int key0(int pos) const
    {
        const int i = pos - start;
        return (i < t.ns ? i : t.tw + i - t.ns) * TK;
    }
    // tiles whose keys are all seen, but for those of the sinks: first keys lo .. lo + span
    __device__ __forceinline__ void whole(int &lo, unsigned &span) const
    {
        lo = (t.w0 + TK - 1) / TK * TK;
        const int last = n / TK * TK - TK;
        span = (unsigned)(last - lo);
        if (last < lo) {  // none: no tile begins there
            lo = 1 << 30;
            span = 0;
        }
    }
    // the keys of the tile from k0 that may be visible, in whole 16s
    __device__ __forceinline__ int2 rows(int k0, int sinks) const
    {
        const int lo = k0 < sinks ? k0 : max(k0, t.w0 & ~15);
        const int hi = min(k0 + TK, k0 < t.tw * TK ? (sinks + 15) & ~15 : (n + 15) & ~15);
        return make_int2(lo, hi);
    }
    // the group after this one (there is one)
    __device__ __forceinline__ void next(const int *nb, const WinParams &p)
    {
        start += win_span(t.cnt);
        if (++g == p.H_kv) {
            g = 0;
            do n = nb[++b]; while (n == 0);
            t = win_tiles<TK>(n, p.window, p.sinks);
        }
    }
};

// The list's T positions in n shares, the first T % n of them one longer: the first position
// of share i, and the share that holds a position.
struct WinShares {
    int q, rem;

    __device__ __forceinline__ WinShares(int T, int n) : q(T / n), rem(T % n) {}
    __device__ __forceinline__ int first(int i) const { return i * q + min(i, rem); }
    __device__ __forceinline__ int owner(int pos) const
    {
        const int wide = rem * (q + 1);
        return pos < wide ? pos / (q + 1) : rem + (pos - wide) / q;
    }
};

// Orders this thread's accesses, and those of others that it has seen, for the whole GPU.
__device__ __forceinline__ void fence_acq_rel() { asm volatile("fence.acq_rel.gpu;" ::: "memory"); }

__device__ __forceinline__ void win_store(const WinParams &p, size_t i, float v)
{
    if (p.out_bf16)
        reinterpret_cast<__nv_bfloat16 *>(p.out)[i] = __float2bfloat16_rn(v);
    else
        p.out[i] = v;
}

// Where the pieces of a group lie: those of a CTA's warps (list[j]: piece 2 w + 1 of warp w in its
// ring, 2 w in the workspace) or, list null, those of CTAs (the first one's second, then firsts).
struct WinPieces {
    const uint8_t *list;
    const float *ring, *near;
    int ring_step, step;

    __device__ __forceinline__ const float *at(int j) const
    {
        if (!list) return near + (size_t)(2 * j + (j == 0)) * step;
        const int x = list[j];
        return (x & 1) ? ring + (x >> 1) * ring_step : near + (size_t)(x >> 1) * step;
    }
};

// NT threads (tid of them, barrier bar): the n pieces of group gi joined into `part` (a piece) or,
// when that is null, into the output.  red: WN_RED floats; scratch: 16 n + 16; factor: of
// the pieces' m.  Begins and
// ends with both free.  FAR: the pieces were written by other CTAs too and are read past the
// L1 cache.
template <int D, int NT, bool FAR>
__device__ __forceinline__ void win_join(const WinParams &p, float factor, int tid, int bar, int n, const WinPieces pieces, float *red,
                                         float *scratch, int gi, float *part)
{
    constexpr unsigned FULL = 0xffffffffu;
    constexpr int AHEAD = 8, HS = D + 4;
    const float NEG_INF = __int_as_float(0xff800000);
    const int lane = tid & 31, GS = p.G * HS;
    float *tot = scratch, *wt = scratch + 16, *lt = wt + 8 * n;
    auto load = [](const float *a) { return FAR ? __ldcg(a) : *a; };
    auto load4 = [](const float *a) {
        return FAR ? __ldcg(reinterpret_cast<const float4 *>(a)) : *reinterpret_cast<const float4 *>(a);
    };
    // four outputs a thread; with few outputs, ns slices of the pieces.  The first pieces are on
    // their way while the weights are worked out (indexes past the last are those of the last:
    // a load under a condition would be waited for before the next)
    const int nv = p.G * (D / 4), cols = min(nv, NT), ns = NT / cols, sl = tid / cols;
    int v = tid % cols, h = v / (D / 4), at = h * HS + 4 * (v % (D / 4));
    float4 ahead[AHEAD];
    auto fetch = [&]() {
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) ahead[k] = load4(pieces.at(min(sl + k * ns, n - 1)) + at);
    };
    fetch();
    // a warp a head: the largest of the pieces' m, their weights, the sum
    for (int hd = tid >> 5; hd < p.G; hd += NT / 32) {
        float M = NEG_INF;
        for (int j = lane; j < n; j += 32) {
            const float *pc = pieces.at(j) + GS + hd;
            const float m = load(pc), l = load(pc + 8);
            wt[8 * j + hd] = m;
            lt[8 * j + hd] = l;
            M = fmaxf(M, m);
        }
#pragma unroll
        for (int m = 16; m; m >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL, M, m));
        float L = 0.f;
        for (int j = lane; j < n; j += 32) {
            const float w = M == NEG_INF ? 1.f : ex2((wt[8 * j + hd] - M) * factor);  // (all empty: empty)
            wt[8 * j + hd] = w;
            L = fmaf(w, lt[8 * j + hd], L);
        }
#pragma unroll
        for (int m = 16; m; m >>= 1) L += __shfl_xor_sync(FULL, L, m);
        if (lane == 0) {
            tot[hd] = M;
            tot[8 + hd] = L;
        }
    }
    bar_sync<NT>(bar);
    auto add = [](float4 &o, const float4 &x, float w) {
        o.x = fmaf(w, x.x, o.x);
        o.y = fmaf(w, x.y, o.y);
        o.z = fmaf(w, x.z, o.z);
        o.w = fmaf(w, x.w, o.w);
    };
    for (;;) {
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (sl + k * ns < n) add(o, ahead[k], wt[8 * (sl + k * ns) + h]);
        for (int j = sl + AHEAD * ns; j < n; j += 4 * ns) {
#pragma unroll
            for (int k = 0; k < 4; ++k) ahead[k] = load4(pieces.at(min(j + k * ns, n - 1)) + at);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (j + k * ns < n) add(o, ahead[k], wt[8 * (j + k * ns) + h]);
        }
        if (ns > 1) {
            reinterpret_cast<float4 *>(red)[tid] = o;
            bar_sync<NT>(bar);
            if (sl == 0)
                for (int s = 1; s < ns; ++s) add(o, reinterpret_cast<const float4 *>(red)[s * cols + tid], 1.f);
        }
        if (sl == 0) {
            if (part) {
                *reinterpret_cast<float4 *>(part + at) = o;
                if (v % (D / 4) == 0) {
                    part[GS + h] = tot[h];
                    part[GS + 8 + h] = tot[8 + h];
                }
            } else {
                const float r = 1.f / tot[8 + h];
                const size_t to = ((size_t)(gi / p.H_kv) * p.H_q + (size_t)(gi % p.H_kv) * p.G) * D + 4 * (size_t)v;
                o = make_float4(o.x * r, o.y * r, o.z * r, o.w * r);
                if (p.out_bf16)
                    *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(p.out) + to) = make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
                else
                    *reinterpret_cast<float4 *>(p.out + to) = o;
            }
        }
        v += NT;  // (more outputs than threads: ns = 1)
        if (v >= nv) break;
        h = v / (D / 4);
        at = h * HS + 4 * (v % (D / 4));
        fetch();
    }
    bar_sync<NT>(bar);
}

// ------------------------------------------------------------------ the kernel

// WIDE: groups of 5 to 8 heads (a column each); else up to 4 heads, columns 4-7 repeat 0-3.
template <int D, bool KV4, bool WIDE>
__device__ __forceinline__ void window_body(const WinParams &p, const CUtensorMap *tm_k, const CUtensorMap *tm_v)
{
    constexpr int W = win_warps(KV4), NT = 32 * W;  // warps and threads that work
    constexpr int TK = win_tile(D, KV4), SUB = TK / 16, STAGE = win_stage(D, KV4), NS = win_stages(D, KV4);
    constexpr int MT = D / 16;   // 16-row pieces of the output, and MMA steps of a score
    constexpr int NB = KV4 ? (WIDE ? 2 : 1) : (WIDE ? 3 : 2);  // MMAs that the terms of p take (4-bit: two, bf16: three)
    constexpr unsigned FULL = 0xffffffffu;
    const float NEG_INF = __int_as_float(0xff800000);
    extern __shared__ __align__(16) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *smem = KV4 ? smem_raw : smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const WinSmem lay = win_smem(D, KV4, p.B);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
    // (the copying warp: lane w works for warp w)
    const int owner = warp < W ? warp : min(lane, W - 1);
    uint8_t *ring = smem + lay.ring + owner * NS * STAGE;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + lay.bar) + owner * 2 * NS, *empty = full + NS;
    volatile int *stop = reinterpret_cast<volatile int *>(smem + lay.stop);
    int *seg = reinterpret_cast<int *>(smem + lay.seg);
    int *flag = reinterpret_cast<int *>(smem + lay.flag);
    int *nb = reinterpret_cast<int *>(smem + lay.nb);
    int *prefix = reinterpret_cast<int *>(smem + lay.prefix);
    const int PIECE = win_piece(p.G, D);

    // ---- setup: checked lengths and the list's prefix, barriers
    if (warp == 0) {
        int run = 0, longest = 0;
        bool bad = false;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const int b = b0 + lane;
            int n = b < p.B ? p.seq_lens[b] : 0;
            if (n < 0 || n > p.n_max) {
                bad = true;
                n = 0;
            }
            const int tiles = win_tiles<TK>(n, p.window, p.sinks).cnt, cnt = p.H_kv * win_span(tiles);
            longest = max(longest, tiles);
            int x = cnt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(FULL, x, o);
                if (lane >= o) x += y;
            }
            if (b < p.B) {
                nb[b] = n;
                prefix[b] = run + x - cnt;
            }
            run += __shfl_sync(FULL, x, 31);
        }
        longest = __reduce_max_sync(FULL, longest);
        if (lane == 0) {
            prefix[p.B] = run;
            flag[0] = longest;
        }
        if (bad && blockIdx.x == 0) set_dev_error(p.ctrl, DEV_BAD_SEQLEN);
    }
    if (!KV4 && warp == W && lane < W) {
        for (int s = 0; s < 2 * NS; ++s) mbar_init(&full[s], 1);
        mbar_fence_init();
        stop[lane] = 0;
    }
    if (tid < 2 * W) seg[tid] = -1;
    __syncthreads();

    const int T = prefix[p.B];
    for (int b = blockIdx.x; b < p.B; b += gridDim.x)  // sequences without keys
        if (nb[b] == 0)
            for (int i = tid; i < p.H_q * D; i += blockDim.x) win_store(p, (size_t)b * p.H_q * D + i, 0.f);
    // Few short groups: a CTA for each.  Else even shares of the list, which split groups between
    // CTAs and join them through the workspace: fence, arrival and join make a group of 128 keys
    // 2.3-3.6 us (bf16) or 5.5-6 us (4 bits) longer than one CTA would be.
    const bool alone = p.B * p.H_kv <= (int)gridDim.x && flag[0] <= WN_ALONE * W;
    const int NC = alone ? p.B * p.H_kv : min((int)gridDim.x, (T + W - 1) / W);  // CTAs with a share
    if ((int)blockIdx.x >= NC) return;
    const WinShares ctas(T, NC);
    int t0 = ctas.first(blockIdx.x), t1 = ctas.first(blockIdx.x + 1);
    if (alone) {
        const int b = blockIdx.x / p.H_kv, span = win_span(win_tiles<TK>(nb[b], p.window, p.sinks).cnt);
        t0 = prefix[b] + blockIdx.x % p.H_kv * span;
        t1 = t0 + span;
    }
    const WinShares warps(t1 - t0, W);
    const int ta = t0 + warps.first(owner), tb = t0 + warps.first(owner + 1);

    WinGroup<TK> head;  // the group of the share's first tile, whose position is t
    int t = ta;
    if (ta < tb) {
        head.seek(ta, prefix, nb, p);
        t = max(ta, head.start);
    }
    if (warp == W) {  // (bf16)
        // ---- the copies: one lane a ring; `t` is the next tile to fetch, of group `head`
        const uint64_t policy = l2_policy_evict_first();
        bool live = lane < W && t < tb;
        int filled = 0, is = 0;                       // stages filled, the next one to fill
        uint32_t phase = 1;                           // a fresh barrier lets this parity pass
        int jump = 0, k0 = 0;                         // where the rows break off; the tile's first key
        auto follow = [&]() {
            jump = t < head.start + head.t.ns ? head.start + head.t.ns : head.end();
            k0 = head.key0(t);
        };
        if (live) follow();
        uint64_t since = globaltimer_ns();
        while (__any_sync(FULL, live)) {
            const bool go = live && mbar_test(&empty[is], phase);
            if (go) {
                uint8_t *st = ring + is * STAGE;
                // whole boxes: rows past the group's last key are other keys or zeros, never used
                const int row = head.index(p) * p.n_max + k0;
                mbar_arrive_tx(&full[is], (uint32_t)STAGE);
#pragma unroll
                for (int hf = 0; hf < D / 64; ++hf) {
                    tma_load_2d(st + hf * TK * 128, tm_k, hf * 64, row, &full[is], policy);
                    tma_load_2d(st + TK * D * 2 + hf * TK * 128, tm_v, hf * 64, row, &full[is], policy);
                }
                ++filled;
                if (++is == NS) {
                    is = 0;
                    phase ^= 1u;
                }
                ++t;
                k0 += TK;
                if (t == jump) {  // the sinks end, or the group
                    if (t == head.end()) {
                        t += WN_SETUP;
                        if (t < tb) {
                            head.next(nb, p);
                            const uint16_t *q0 = p.q + ((size_t)head.b * p.H_q + head.g * p.G) * D;  // its queries, into L2
                            for (int i = 0; i < p.G * D; i += 64) prefetch_l2(q0 + i);
                        }
                    }
                    if (t < tb) follow();
                }
                live = t < tb;
            } else if (live && stop[lane]) {
                live = false;
            }
            // (warps that work are never this slow; those that gave up have set `stop`)
            if (__any_sync(FULL, go)) since = globaltimer_ns();
            else if (globaltimer_ns() - since > p.wait_ns + DRAIN_NS) {
                if (live) set_dev_error(p.ctrl, DEV_TIMEOUT);
                live = false;
            }
        }
        // every copy has landed before the CTA ends
        if (lane < W)
            for (int x = max(0, filled - NS); x < filled; ++x) mbar_wait_bounded(&full[x % NS], (uint32_t)(x / NS) & 1u, DRAIN_NS);
        return;
    }
    if (t < tb) {
        // the groups of the tile at hand and (4-bit) of the next to fetch: seldom needed, so kept
        // in shared memory; lane 0 writes
        WinGroup<TK> *groups = reinterpret_cast<WinGroup<TK> *>(smem + lay.group) + 2 * warp;
        WinGroup<TK> &cg = groups[0], &ig = groups[1];
        static_assert(sizeof(WinGroup<TK>) == 32, "the layout of shared memory");
        auto advance = [&](WinGroup<TK> &g) {
            __syncwarp();
            if (lane == 0) g.next(nb, p);
            __syncwarp();
        };
        if (lane == 0) cg = ig = head;
        __syncwarp();
        // ---- a group's queries: head column r (zero in columns without a head).  4-bit: lane c
        // takes dimensions D/4 c .., four to an MMA step; bf16: 16 c .. of each 64
        uint4 qraw[MT / 2];
        auto load_q = [&]() {
            const int h = WIDE ? r : (r & 3);
            const uint16_t *qh = p.q + ((size_t)cg.b * p.H_q + cg.g * p.G + h) * D;
#pragma unroll
            for (int i = 0; i < MT / 2; ++i)
                qraw[i] = h >= p.G ? make_uint4(0, 0, 0, 0)
                          : KV4    ? reinterpret_cast<const uint4 *>(qh + (D / 4) * c)[i]
                                   : reinterpret_cast<const uint4 *>(qh + (i / 2) * 64 + 16 * c)[i & 1];
        };
        load_q();
        int cs = 0;            // the stage to use next
        uint32_t cphase = 0;

        // ---- 4-bit: the copies, by all lanes.  `ig` is the group of the next tile to fetch, `it`
        // its position, fk its first key, frow its cache row; the rows break off at `fjump`.
        // Every call makes one group of copies
        int it = t, fjump = 0, fk = 0, flo = 0;
        unsigned fspan = 0;
        uint32_t frow = 0;
        auto follow = [&]() {
            fjump = it < ig.start + ig.t.ns ? ig.start + ig.t.ns : ig.end();
            fk = ig.key0(it);
            frow = (uint32_t)ig.index(p) * (uint32_t)p.n_max + (uint32_t)fk;
            ig.whole(flo, fspan);
        };
        auto fetch = [&](int stage) {
            if (it < tb) {
                constexpr int RB = D / 2, NC16 = TK * RB / 512, NS16 = TK * (D / 16) / 16;  // copies a lane; lanes for scales
                const uint32_t dst = smem_u32(ring) + stage * STAGE + 16 * lane;
                const uint8_t *gk = p.k + (size_t)frow * RB + 16 * lane, *gv = p.v + (size_t)frow * RB + 16 * lane;
                const uint8_t *gks = p.ks + (size_t)frow * (D / 16) + 16 * lane, *gvs = p.vs + (size_t)frow * (D / 16) + 16 * lane;
                if ((unsigned)(fk - flo) <= fspan) {
#pragma unroll
                    for (int i = 0; i < NC16; ++i) copy16(dst + 512 * i, gk + 512 * i);
#pragma unroll
                    for (int i = 0; i < NC16; ++i) copy16(dst + TK * RB + 512 * i, gv + 512 * i);
                    if (lane < NS16) {
                        copy16(dst + TK * D, gks);
                        copy16(dst + TK * (D + D / 16), gvs);
                    }
                } else {
                    const int2 rw = ig.rows(fk, p.sinks);  // multiples of 16, as n_max is
                    const int lo = rw.x - fk, hi = rw.y - fk;
#pragma unroll 1
                    for (int i = 0; i < NC16; ++i) {
                        const int row = (512 * i + 16 * lane) / RB;
                        if (row >= lo && row < hi) {
                            copy16(dst + 512 * i, gk + 512 * i);
                            copy16(dst + TK * RB + 512 * i, gv + 512 * i);
                        }
                    }
                    const int row = 16 * lane / (D / 16);
                    if (row >= lo && row < hi) {
                        copy16(dst + TK * D, gks);
                        copy16(dst + TK * (D + D / 16), gvs);
                    }
                }
                ++it;
                fk += TK;
                frow += TK;
                if (it == fjump) {  // the sinks end, or the group
                    if (it == ig.end()) {
                        it += WN_SETUP;
                        if (it < tb) {
                            advance(ig);
                            const uint16_t *q0 = p.q + ((size_t)ig.b * p.H_q + ig.g * p.G) * D;  // its queries, into L2
                            if (lane * 64 < p.G * D) prefetch_l2(q0 + lane * 64);
                        }
                    }
                    if (it < tb) follow();
                }
            }
            copy_commit();
        };
        if (KV4) {
            follow();
#pragma unroll 1
            for (int i = 0; i < NS; ++i) fetch(i);
        }

        // ---- the sums
        uint32_t qf[MT][2];                  // B operand of the scores
        float o[MT][4];                      // columns 2c, 2c+1 of output rows r, r+8 of each piece
        float l0 = 0.f, l1 = 0.f, m0 = 0.f, m1 = 0.f, thr0 = NEG_INF, thr1 = NEG_INF;
        float ka0 = p.k2, ka1 = p.k2;
        const float second = c < 2 ? 0.f : -1.f, low = c < 2 ? 1.f : WN_LOW;
        // ---- one tile: the keys from k0, whose rows and scales the pointers are at
        // (whole: every one is seen, no masks)
        auto pass = [&](const uint8_t *kc, const uint8_t *vc, const uint8_t *ks, const uint8_t *vs, int k0, bool whole) {
            auto seen = [&](int j) { return j < cg.n && (j >= cg.t.w0 || j < p.sinks); };

            // ---- scores of keys r, r+8 of each 16, columns 2c, 2c+1
            float s[SUB][4];
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                float acc[MT / 2][4];  // chains of two steps
                if (KV4) {
                    uint32_t w[2][D / 32], sc[2][2];  // rows r, r+8: codes, scales (twice, as fp16)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int kr = 16 * u + r + 8 * y;
                        if (D == 128) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(kc + kr * 64 + c * 16);
                            w[y][0] = x.x, w[y][1] = x.y, w[y][D / 32 - 2] = x.z, w[y][D / 32 - 1] = x.w;
                            sc[y][0] = (uint32_t)ks[kr * 8 + 2 * c] * 0x00800080u;
                            sc[y][1] = (uint32_t)ks[kr * 8 + 2 * c + 1] * 0x00800080u;
                        } else {
                            const uint2 x = *reinterpret_cast<const uint2 *>(kc + kr * 32 + c * 8);
                            w[y][0] = x.x, w[y][1] = x.y;
                            sc[y][0] = sc[y][1] = (uint32_t)ks[kr * 4 + c] * 0x00800080u;
                        }
                    }
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) {  // a word: two steps
                        uint32_t a[2][4];
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            e2m1_unpack8(w[y][j], a[y]);
#pragma unroll
                            for (int i = 0; i < 4; ++i) a[y][i] = h2mul(a[y][i], sc[y][j / 2]);
                        }
                        mma_set<false>(acc[j], a[0][0], a[1][0], a[0][1], a[1][1], qf[2 * j][0], qf[2 * j][1]);
                        mma_add<false>(acc[j], a[0][2], a[1][2], a[0][3], a[1][3], qf[2 * j + 1][0], qf[2 * j + 1][1]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < MT / 2; ++i) {  // piece i & 1 of the lane's 16 dimensions of half i / 2
                        const uint8_t *kt = kc + (i / 2) * TK * 128;
                        const int pc = 2 * c + (i & 1), kr = 16 * u + r;
                        const uint4 x = *reinterpret_cast<const uint4 *>(kt + kr * 128 + ((pc ^ r) << 4));
                        const uint4 y = *reinterpret_cast<const uint4 *>(kt + (kr + 8) * 128 + ((pc ^ r) << 4));
                        mma_set<true>(acc[i], x.x, y.x, x.y, y.y, qf[2 * i][0], qf[2 * i][1]);
                        mma_add<true>(acc[i], x.z, y.z, x.w, y.w, qf[2 * i + 1][0], qf[2 * i + 1][1]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    add2(acc[0][e], acc[0][e + 1], acc[1][e], acc[1][e + 1]);
                    if (MT == 8) {
                        add2(acc[MT / 2 - 2][e], acc[MT / 2 - 2][e + 1], acc[MT / 2 - 1][e], acc[MT / 2 - 1][e + 1]);
                        add2(acc[0][e], acc[0][e + 1], acc[MT / 2 - 2][e], acc[MT / 2 - 2][e + 1]);
                    }
                    s[u][e] = acc[0][e];
                    s[u][e + 1] = acc[0][e + 1];
                }
            }
            if (!whole)
#pragma unroll
                for (int u = 0; u < SUB; ++u) {
                    const int ja = k0 + 16 * u + r;
                    if (!seen(ja)) s[u][0] = s[u][1] = NEG_INF;
                    if (!seen(ja + 8)) s[u][2] = s[u][3] = NEG_INF;
                }

            // ---- a new maximum, when it is far above m
            float x0 = NEG_INF, x1 = NEG_INF;
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                x0 = fmaxf(x0, fmaxf(s[u][0], s[u][2]));
                x1 = fmaxf(x1, fmaxf(s[u][1], s[u][3]));
            }
            if (__any_sync(FULL, x0 > thr0 || x1 > thr1)) {
#pragma unroll
                for (int m = 4; m <= 16; m <<= 1) {
                    x0 = fmaxf(x0, __shfl_xor_sync(FULL, x0, m));
                    x1 = fmaxf(x1, __shfl_xor_sync(FULL, x1, m));
                }
                float f0 = 1.f, f1 = 1.f;
                if (x0 > thr0) {
                    f0 = ex2(fminf((m0 - x0) * ka0, 0.f));  // (of empty sums m is not yet set)
                    m0 = x0;
                    thr0 = __fadd_rd(x0, WN_SLACK / ka0);  // (rounded up, it could pass the range of p)
                }
                if (x1 > thr1) {
                    f1 = ex2(fminf((m1 - x1) * ka1, 0.f));
                    m1 = x1;
                    thr1 = __fadd_rd(x1, WN_SLACK / ka1);
                }
                l0 *= f0;
                l1 *= f1;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    o[i][0] *= f0;
                    o[i][1] *= f1;
                    o[i][2] *= f0;
                    o[i][3] *= f1;
                }
            }

            // ---- p, its sum, and its terms as the B operand of V^T p
            uint32_t pb[SUB][NB][2];
#pragma unroll
            for (int u = 0; u < SUB; ++u)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    add2(s[u][2 * y], s[u][2 * y + 1], -m0, -m1);
                    const float2 x = fma2(s[u][2 * y], s[u][2 * y + 1], ka0, ka1, WN_TOP, WN_TOP);
                    s[u][2 * y] = ex2(x.x);
                    s[u][2 * y + 1] = ex2(x.y);
                }
            if (!whole)
#pragma unroll
                for (int u = 0; u < SUB; ++u)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        if (!seen(k0 + 16 * u + r + 8 * y)) s[u][2 * y] = s[u][2 * y + 1] = 0.f;
#pragma unroll
            for (int u = 0; u < SUB; ++u)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    float a = s[u][2 * y], b = s[u][2 * y + 1];
                    add2(l0, l1, a, b);
                    if (KV4) {
                        // what the first term leaves, times WN_LOW, is the second.  Up to 4 heads: columns
                        // 0-3 hold the first, 4-7 the second (second = 0 or -1)
                        const uint32_t t = pack_f16(a, b);
                        const float2 f = unpack_f16(t);
                        const float take = WIDE ? -1.f : second, by = WIDE ? WN_LOW : low;
                        float2 g = fma2(f.x, f.y, take, take, a, b);
                        g = fma2(g.x, g.y, by, by, -0.f, -0.f);
                        pb[u][NB - 1][y] = movmatrix(pack_f16(g.x, g.y));
                        if (WIDE) pb[u][0][y] = movmatrix(t);
                    } else {
                        uint32_t term[3];
#pragma unroll
                        for (int i = 0; i < 3; ++i) {
                            term[i] = pack_bf16(a, b);
                            a -= bf16lo_to_f32(term[i]);
                            b -= bf16hi_to_f32(term[i]);
                        }
                        if (WIDE) {
#pragma unroll
                            for (int i = 0; i < 3; ++i) pb[u][i % NB][y] = movmatrix(term[i]);
                        } else {
                            pb[u][0][y] = movmatrix(c < 2 ? term[0] : term[1]);
                            pb[u][NB - 1][y] = movmatrix(c < 2 ? term[2] : 0u);
                        }
                    }
                }

            // ---- o += V^T p, the tile's keys in one chain per piece
            if (KV4) {
                constexpr int RB = D / 2, W = D / 64;  // bytes of a row; words of a lane's D/8 dimensions
                uint32_t sp[SUB][2];
#pragma unroll
                for (int u = 0; u < SUB; ++u) {
                    uint32_t sb[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int kk = 16 * u + 2 * c + (i & 1) + 8 * (i >> 1);
                        sb[i] = vs[kk * (D / 16) + (D == 128 ? r : r >> 1)];
                    }
                    sp[u][0] = sb[1] * 0x800000u + sb[0] * 0x80u;  // the key pair's scales as fp16
                    sp[u][1] = sb[3] * 0x800000u + sb[2] * 0x80u;
                }
                if (!whole)  // what is not seen may be a NaN
#pragma unroll
                    for (int u = 0; u < SUB; ++u)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int j = k0 + 16 * u + 2 * c + 8 * y;
                            sp[u][y] &= (seen(j) ? 0xffffu : 0u) | (seen(j + 1) ? 0xffff0000u : 0u);
                        }
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    // (wide groups: each term in sums of its own, two of a word's four bytes at a time)
                    constexpr int NI = WIDE ? 2 : 4;
#pragma unroll
                    for (int i0 = 0; i0 < 4; i0 += NI) {
                        float acc[NB][NI][4];
#pragma unroll
                        for (int u = 0; u < SUB; ++u) {
                            uint32_t a[2][2][4];  // key pair, even or odd dimension, byte
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const uint8_t *v0 = vc + (16 * u + 2 * c + 8 * y) * RB + r * 4 * W + 4 * w;
                                const uint32_t x0w = *reinterpret_cast<const uint32_t *>(v0);
                                const uint32_t x1w = *reinterpret_cast<const uint32_t *>(v0 + RB);
                                e2m1_unpack8((x0w & 0x0f0f0f0fu) | ((x1w << 4) & 0xf0f0f0f0u), a[y][0]);
                                e2m1_unpack8(((x0w >> 4) & 0x0f0f0f0fu) | (x1w & 0xf0f0f0f0u), a[y][1]);
#pragma unroll
                                for (int i = i0; i < i0 + NI; ++i) {
                                    a[y][0][i] = h2mul(a[y][0][i], sp[u][y]);
                                    a[y][1][i] = h2mul(a[y][1][i], sp[u][y]);
                                }
                            }
#pragma unroll
                            for (int i = 0; i < NI; ++i)
#pragma unroll
                                for (int n = 0; n < NB; ++n) {
                                    const int j = i0 + i;
                                    if (u == 0)
                                        mma_set<false>(acc[n][i], a[0][0][j], a[0][1][j], a[1][0][j], a[1][1][j], pb[u][n][0], pb[u][n][1]);
                                    else
                                        mma_add<false>(acc[n][i], a[0][0][j], a[0][1][j], a[1][0][j], a[1][1][j], pb[u][n][0], pb[u][n][1]);
                                }
                        }
#pragma unroll
                        for (int i = 0; i < NI; ++i)
#pragma unroll
                            for (int e = 0; e < 4; e += 2) {
                                float *to = &o[4 * w + i0 + i][e];
                                if (WIDE) {
                                    const float2 t = fma2(acc[NB - 1][i][e], acc[NB - 1][i][e + 1], 1.f / WN_LOW, 1.f / WN_LOW, to[0], to[1]);
                                    to[0] = t.x, to[1] = t.y;
                                }
                                add2(to[0], to[1], acc[0][i][e], acc[0][i][e + 1]);
                            }
                    }
                }
            } else {
                const uint32_t vt = smem_u32(vc);
                uint32_t mk[SUB][2];
#pragma unroll
                for (int u = 0; u < SUB; ++u) mk[u][0] = mk[u][1] = 0xffffffffu;
                if (!whole)  // what is not seen may be a NaN
#pragma unroll
                    for (int u = 0; u < SUB; ++u)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int j = k0 + 16 * u + 2 * c + 8 * y;
                            mk[u][y] = (seen(j) ? 0xffffu : 0u) | (seen(j + 1) ? 0xffff0000u : 0u);
                        }
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    float acc[4];
#pragma unroll
                    for (int u = 0; u < SUB; ++u) {
                        // matrices: keys 0-7 and 8-15 by dimensions 0-7 and 8-15 of piece i
                        const int kk = 16 * u + (lane & 7) + ((lane >> 4) << 3);
                        const int pc = 2 * (i & 3) + ((lane >> 3) & 1);
                        uint32_t a[4];
                        ldmatrix_x4_trans(a, vt + (uint32_t)((i / 4) * TK * 128 + kk * 128 + ((pc ^ (kk & 7)) << 4)));
#pragma unroll
                        for (int n = 0; n < NB; ++n) {
                            if (u == 0 && n == 0)
                                mma_set<true>(acc, a[0] & mk[u][0], a[1] & mk[u][0], a[2] & mk[u][1], a[3] & mk[u][1], pb[u][n][0], pb[u][n][1]);
                            else
                                mma_add<true>(acc, a[0] & mk[u][0], a[1] & mk[u][0], a[2] & mk[u][1], a[3] & mk[u][1], pb[u][n][0], pb[u][n][1]);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; e += 2) add2(o[i][e], o[i][e + 1], acc[e], acc[e + 1]);
                }
            }
        };

        bool dead = false;
        for (;;) {  // groups
            int k0 = cg.key0(t);  // the tile's first key; where the keys break off; whole tiles
            int tend = min(t < cg.start + cg.t.ns ? cg.start + cg.t.ns : cg.end(), tb), wlo;
            unsigned wspan;
            cg.whole(wlo, wspan);
            if (KV4) {
                // scaled by the power of two that puts the head's largest value near 2^14
                uint32_t big = 0;  // its bf16 bits without the sign
#pragma unroll
                for (int i = 0; i < MT / 2; ++i) {
                    const uint32_t u[4] = {qraw[i].x, qraw[i].y, qraw[i].z, qraw[i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) big = max(big, max(u[j] & 0x7fffu, (u[j] >> 16) & 0x7fffu));
                }
                big = max(big, __shfl_xor_sync(FULL, big, 1));
                big = max(big, __shfl_xor_sync(FULL, big, 2));
                const int e = max(-100, min(127, (int)(big >> 7) - 127)) - 14;
                const float up = p.qsign * exp2i(-e);
#pragma unroll
                for (int i = 0; i < MT / 2; ++i) {
                    qf[2 * i][0] = pack_f16(bf16lo_to_f32(qraw[i].x) * up, bf16hi_to_f32(qraw[i].x) * up);
                    qf[2 * i][1] = pack_f16(bf16lo_to_f32(qraw[i].y) * up, bf16hi_to_f32(qraw[i].y) * up);
                    qf[2 * i + 1][0] = pack_f16(bf16lo_to_f32(qraw[i].z) * up, bf16hi_to_f32(qraw[i].z) * up);
                    qf[2 * i + 1][1] = pack_f16(bf16lo_to_f32(qraw[i].w) * up, bf16hi_to_f32(qraw[i].w) * up);
                }
                const int h0 = WIDE ? 2 * c : (2 * c) & 3;  // heads of this lane's columns
                const float d0 = exp2i(__shfl_sync(FULL, e, h0 * 4)), d1 = exp2i(__shfl_sync(FULL, e, h0 * 4 + 4));
                ka0 = p.k2 * d0;
                ka1 = p.k2 * d1;
            } else {
                const uint32_t flip = p.qsign < 0.f ? 0x80008000u : 0u;
#pragma unroll
                for (int i = 0; i < MT / 2; ++i) {
                    qf[2 * i][0] = qraw[i].x ^ flip;
                    qf[2 * i][1] = qraw[i].y ^ flip;
                    qf[2 * i + 1][0] = qraw[i].z ^ flip;
                    qf[2 * i + 1][1] = qraw[i].w ^ flip;
                }
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
            l0 = l1 = m0 = m1 = 0.f;
            thr0 = thr1 = NEG_INF;
            for (;;) {  // tiles
                if (KV4) {
                    copy_wait<NS - 1>();
                    __syncwarp();
                } else if (!dead && !__all_sync(FULL, win_wait(&full[cs], cphase, p.wait_ns))) {
                    dead = true;  // no more copies, no more sums (the pieces still meet)
                    if (lane == 0) {
                        set_dev_error(p.ctrl, DEV_TIMEOUT);
                        stop[warp] = 1;
                    }
                }
                if (!dead) {
                    const bool whole = (unsigned)(k0 - wlo) <= wspan;
                    const uint8_t *st = ring + cs * STAGE;
                    if (KV4)
                        pass(st, st + TK * (D / 2), st + TK * D, st + TK * (D + D / 16), k0, whole);
                    else
                        pass(st, st + TK * D * 2, nullptr, nullptr, k0, whole);
                }
                __syncwarp();
                if (KV4) fetch(cs);
                else if (!dead && lane == 0) mbar_arrive(&empty[cs]);
                cs = cs + 1 == NS ? 0 : cs + 1;
                if (cs == 0) cphase ^= 1u;
                ++t;
                k0 += TK;
                if (t != tend) continue;
                if (t == tb || t == cg.end()) break;
                tend = min(cg.end(), tb);  // the sinks end
                k0 = cg.key0(t);
            }

            // ---- the group's last tile here: its result, or a piece of it
            const bool ended = t == cg.end(), all = ta <= cg.start && ended;
            if (ended) t += WN_SETUP;
            // sums that no score has set m for are empty (or NaN): they weigh nothing
            if (thr0 == NEG_INF) m0 = NEG_INF;
            if (thr1 == NEG_INF) m1 = NEG_INF;
            if (KV4 && !all) {
                // m of all pieces of a head in one unit: times the power of two that ka holds (from the
                // difference of the exponents), and 2^-24, so that it cannot overflow
                m0 *= __int_as_float(__float_as_int(ka0) - __float_as_int(p.k2) + 0x3f800000) * 0x1p-24f;
                m1 *= __int_as_float(__float_as_int(ka1) - __float_as_int(p.k2) + 0x3f800000) * 0x1p-24f;
            }
#pragma unroll
            for (int m = 4; m <= 16; m <<= 1) {
                l0 += __shfl_xor_sync(FULL, l0, m);
                l1 += __shfl_xor_sync(FULL, l1, m);
            }
            // a piece lies in the warp's ring if it is the warp's last, else in the workspace
            const int slot = t < tb ? 0 : 1;
            float *piece = slot ? reinterpret_cast<float *>(ring) : p.first + (size_t)(blockIdx.x * W + warp) * PIECE;
            const size_t orow = (size_t)cg.b * p.H_q + cg.g * p.G;
            // heads of the lane's values: x of column 2c (and z of 2c+1 in wide groups)
            const int hx = WIDE ? 2 * c : 2 * (c & 1) + (c >> 1);
            const float lx = WIDE || c < 2 ? l0 : l1, mx = WIDE || c < 2 ? m0 : m1;
            const float ix = all ? 1.f / lx : 1.f, iz = all ? 1.f / l1 : 1.f;
            if (!WIDE)  // columns j and j + 4 hold terms of the same head: lanes c, c ^ 2
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        if (KV4 && c >= 2) {
                            o[i][e] *= 1.f / WN_LOW;
                            o[i][e + 1] *= 1.f / WN_LOW;
                        }
                        const float got = __shfl_xor_sync(FULL, c < 2 ? o[i][e + 1] : o[i][e], 2);
                        o[i][e] = (c < 2 ? o[i][e] : o[i][e + 1]) + got;
                    }
#pragma unroll
            for (int x = 0; x < (WIDE ? 2 : 1); ++x) {
                const int h = hx + x;
                const float inv = x ? iz : ix;
                if (h >= p.G) continue;
                if (KV4) {
                    // D/8 dimensions in a row, from D/8 r
                    const size_t at = (orow + h) * D + (D / 8) * r;
                    float *dst = all ? p.out + at : piece + h * (D + 4) + (D / 8) * r;
                    if (all && p.out_bf16) {
#pragma unroll
                        for (int i = 0; i < MT; i += 4)
                            *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(p.out) + at + 2 * i) =
                                make_uint4(pack_bf16(o[i][x] * inv, o[i][x + 2] * inv), pack_bf16(o[i + 1][x] * inv, o[i + 1][x + 2] * inv),
                                           pack_bf16(o[i + 2][x] * inv, o[i + 2][x + 2] * inv),
                                           pack_bf16(o[i + 3][x] * inv, o[i + 3][x + 2] * inv));
                    } else {
#pragma unroll
                        for (int i = 0; i < MT; i += 2)
                            *reinterpret_cast<float4 *>(dst + 2 * i) =
                                make_float4(o[i][x] * inv, o[i][x + 2] * inv, o[i + 1][x] * inv, o[i + 1][x + 2] * inv);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int dim = 16 * i + 8 * y + r;
                            if (all) win_store(p, (orow + h) * D + dim, o[i][x + 2 * y] * inv);
                            else piece[h * (D + 4) + dim] = o[i][x + 2 * y];
                        }
                }
                if (!all && r == 0) {
                    piece[p.G * (D + 4) + h] = x ? m1 : mx;
                    piece[p.G * (D + 4) + 8 + h] = x ? l1 : lx;
                }
            }
            if (!all && lane == 0) seg[2 * warp + slot] = cg.index(p);
            if (t >= tb) break;
            advance(cg);
            load_q();
        }
    }
    bar_sync<NT>();  // (also makes the pieces in the workspace visible to the CTA)

    // ---- join the CTA's pieces group by group, in the order of the list, two groups at a time by
    // half of the threads each (two are usual, where a share ends one and begins the next).
    // Scratch: behind the pieces, which are the first stage of each warp's ring
    const int half = warp >= W / 2;
    const float factor = KV4 ? p.k2 * 0x1p24f : p.k2;
    float *scratch = reinterpret_cast<float *>(smem + lay.ring + 2 * half * NS * STAGE + STAGE);
    float *red = scratch + NS * STAGE / 4;
    uint8_t *list = reinterpret_cast<uint8_t *>(smem + lay.list) + 32 * warp;
    const int mine = lane < 2 * W ? seg[lane] : -1;
    const unsigned same = __match_any_sync(FULL, mine);
    unsigned leaders = __ballot_sync(FULL, mine >= 0 && lane == __ffs((int)same) - 1);
    int open0 = -1, open1 = -1;  // the CTA's groups that other CTAs share: begun before it, begun here
    while (leaders) {
        int gi = -1;
        unsigned set = 0;
        float *part = nullptr;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (!leaders) continue;
            const int i = __ffs((int)leaders) - 1;
            leaders &= leaders - 1;
            const int g = __shfl_sync(FULL, mine, i);
            const unsigned who = __shfl_sync(FULL, same, i);
            const int b = g / p.H_kv;
            const int cnt = win_tiles<TK>(nb[b], p.window, p.sinks).cnt;
            const int start = prefix[b] + g % p.H_kv * win_span(cnt) + WN_SETUP;
            const int slot = t0 <= start ? 1 : 0;  // begun here, or before
            const bool all = slot && start + cnt <= t1;
            if (!all) (slot ? open1 : open0) = g;
            if (k == half) {
                gi = g;
                set = who;
                part = all ? nullptr : p.part + (size_t)(2 * blockIdx.x + slot) * PIECE;
            }
        }
        if (gi >= 0) {
            // list[j]: which is the j-th of the group's pieces, a copy for each warp
            if (set >> lane & 1) list[__popc(set & ((1u << lane) - 1))] = (uint8_t)lane;
            __syncwarp();
            const WinPieces pieces{list, reinterpret_cast<const float *>(smem + lay.ring), p.first + (size_t)blockIdx.x * W * PIECE,
                                   NS * STAGE / 4, PIECE};
            win_join<D, NT / 2, false>(p, factor, tid - half * (NT / 2), 2 + half, __popc(set), pieces, red, scratch, gi, part);
        }
    }
    if (open0 < 0 && open1 < 0) return;

    // ---- groups that span CTAs: the last to arrive joins
    bar_sync<NT>();
    if (warp == 0) {
        // lanes 0 and 1 arrive for the two at once: one fence for what the CTA wrote, one round
        // trip (the lanes one after the other, each with its fences, took 2.5 us more)
        const int gi = lane == 0 ? open0 : lane == 1 ? open1 : -1;
        int ca = 0, n = 0, old = -1;
        if (gi >= 0) {
            const int b = gi / p.H_kv;
            const int cnt = win_tiles<TK>(nb[b], p.window, p.sinks).cnt;
            const int start = prefix[b] + gi % p.H_kv * win_span(cnt) + WN_SETUP;
            ca = ctas.owner(start);
            n = ctas.owner(start + cnt - 1) - ca + 1;
        }
        __syncwarp();
        fence_acq_rel();
        if (gi >= 0) old = atomicAdd(p.ctrl + CTRL_GROUPS + gi, 1);
        const bool last = gi >= 0 && old == n - 1;
        if (last) p.ctrl[CTRL_GROUPS + gi] = 0;
        if (__any_sync(FULL, last)) fence_acq_rel();
        if (lane < 2) {
            flag[lane] = last ? n : 0;
            flag[2 + lane] = ca;
        }
    }
    bar_sync<NT>();
    // half of the threads for each of the two (one after the other took 2.3 us more)
    const int n = flag[half], ca = flag[2 + half];
    if (n > 0) {
        // (the rings are free: n <= WN_MAX_CTAS pieces take 41 KB of them)
        float *far = reinterpret_cast<float *>(smem + lay.ring) + half * (WN_RED + 16 * WN_MAX_CTAS + 16);
        const WinPieces pieces{nullptr, nullptr, p.part + (size_t)2 * ca * PIECE, 0, PIECE};
        win_join<D, NT / 2, true>(p, factor, tid - half * (NT / 2), 2 + half, n, pieces, far, far + WN_RED, half ? open1 : open0, nullptr);
    }
}

template <int D, bool WIDE>
__global__ void __launch_bounds__(win_threads(true), 1) santa_window_kv4_kernel(const __grid_constant__ WinParams p)
{
    window_body<D, true, WIDE>(p, nullptr, nullptr);
}

template <int D, bool WIDE>
__global__ void __launch_bounds__(win_threads(false), 1)
    santa_window_bf16_kernel(const __grid_constant__ WinParams p, const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v)
{
    window_body<D, false, WIDE>(p, &tm_k, &tm_v);
}

}  // namespace santa

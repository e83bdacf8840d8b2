// santa_attend.cuh -- exact causal attention of a chunk of new tokens over a paged cache, sm_103a.
//
//   o = sum_j p_j v_j,  p = softmax over visible j of scale q.k_j
//   visible(j):  j <= P  and  (window == 0  or  j > P - window  or  j < sinks)
//
// for the token at position P.
//
// Rows and items.  The G query heads of a KV head and consecutive tokens share K and V: they are
// the rows of one product, token by token, 128 to a tile (a row of the MMA, a lane of TMEM).  An
// item is NQ tiles of one sequence and KV head with the tiles of 128 keys that any of its tokens sees.
// NQ = 1 where the whole chunk is one tile (decode steps, drafted tokens): HBM bounds it, and all
// other shared memory is ring.  NQ = 2 else: K and V in shared memory serve 256 rows.
//
// Shares.  The list of all items' key tiles, over sequences, row tiles and KV heads, is cut into
// equal contiguous shares, one a CTA, one CTA an SM: any mix of prompts, decode steps, lengths and
// windows fills the GPU, without a queue.  An item counts AT_SETUP tiles more than it has, for its ends.  One that spans CTAs leaves pieces (the reference
// and the sum of the weights, and the sum over V, of each row) in the workspace; the last CTA to arrive
// joins them in the order of the list, so results do not depend on timing.
//
// Warps of a CTA:
//  * a producer: the item's q rows by one tiled TMA copy a column block (strides of any projection's
//    slice), then K and V of each tile, page by page, a lane a page, into a ring of 32 KB stages (five,
//    or six with one row tile; d = 64: eight of 16 KB);
//  * an MMA warp a row tile, an elected lane of which issues S = Q K^T (both from shared memory) and
//    O += P V, P read from TMEM, V from shared memory as it lies (keys as rows: MN-major);
//  * four softmax warps a row tile, a thread a row: the scores' maximum; p = 2^(k2 s - r), rounded to bf16
//    and written to TMEM over the scores, in two halves, so that P V begins with the first; the sum of the
//    rounded values, so that a rounding moves numerator and denominator alike.  r belongs to a score
//    so far and moves only when one exceeds it by 2^AT_SLACK, so that O in TMEM is seldom
//    rescaled.
// TMEM has room for one score buffer a row tile beside two outputs of 128 columns, so the chain scores,
// softmax, product, scores of a row tile cannot overlap itself.  The two row tiles overlap one
// another: their MMA warps take turns, and while one row tile is in the tensor cores the other is in
// its softmax (without turns both come to do the same at the same time: 2048 tokens on 30k keys 850 us
// against 772, d = 64 631 against 595).  One row tile has two score buffers.
//
// Masks.  A tile that all the item's tokens see whole takes no mask.  In the others the scores of
// hidden keys become minus infinity.  p is 0 there, but 0 times a NaN or an infinity in V is not:
// in those tiles such values of hidden keys are set to zero in shared memory, and when one belongs to a key
// that some token sees, the rows that see it get it added at the end.  That also covers what a page
// holds behind the last key.
//
// Precision.  Scores, references, sums of weights and outputs are fp32.  A score is a chain of d / 16 MMA
// steps, an output one of a step for every 16 keys of AT_CHAIN tiles at most.  A step cuts off what is below 2^-25 of the
// sum's power of 2 in each product and below 2^-23 in the sum (measured), 2.5 2^-23 on average: where all values have
// one sign, 3e-4 of a chain of 2048 steps (measured 2.3e-4), but 2.1e-3 of 300000 keys in one chain.  So a longer
// share's chains are added up in fp32, rounded to the nearest, in the CTA's piece.  P is bf16, as V is: one rounding of each
// weight, 2^-8 at most, of which the common part cancels.  Error against 64 bits (root mean square, relative) 1.8e-3 (a
// few keys lead) to 2.4e-3 (scores nearly alike); the rounding of the result alone is 1.7e-3.  With two terms a weight
// that is all that is left, but with one row tile, whose four warps have no time to spare, one token on 16 x 32k keys
// takes 368 us instead of 317 and 32 ragged sequences of 5 tokens 136 instead of 103, and with two the tensor cores
// would have half as much again to do.  Decode steps in fp32: santa_decode_window, over a contiguous cache.
//
// What bounds it.  Long chunks: the chain of a row tile, about 3500 clocks a tile of 128 keys, of which
// 2 x 1024 are MMAs (the tensor pipe is active 60% of the time, issue slots 48%, the exponential
// unit 30%).  2048 tokens on 30k keys, 32 heads: 1.07 TFLOP in 772 to 805 us (machines differ), 0.69 to 0.72 of the
// measured dense rate; 2 prompts of 8192 tokens 795 to 848 us, 0.67 to 0.72; at d = 64 595 and 671 us, 0.46 and 0.44, as
// the softmax is as long as at d = 128 and an MMA of 64 columns takes as long as one of 128.  Of an item's ends, the
// tiles with masks take 5000 clocks and the results 2500.  One token on 16 sequences of 32k keys: 312 to 318 us, 6.8 TB/s,
// above the measured copy rate; on one sequence of 32k keys 34.5 us, of which 6 are the first copies' way and 6
// the joins.  (MMAs whose lane is picked by its number have their operands moved to uniform registers one at a time:
// 95 clocks an MMA instead of 64.)
#pragma once

#include "santa_tcgen05.cuh"

namespace santa {

constexpr int AT_ROWS = 128;              // rows of a tile: (token, head) pairs
constexpr int AT_KEYS = 128;              // keys of a tile
constexpr int AT_SUB = 64;                // keys of one of its halves
constexpr int AT_MAX_CTAS = 160;          // shares that the workspace has pieces for
// What an item costs beside its tiles, in tiles.  2, 3, 4, 6 and 8: prompts of 2 x 8k tokens 879, 798, 795, 815 and 818 us,
// d = 64 692, 664, 671, 691 and 703; 64 prompts of 200 tokens 129, 135, 129, 131 and 130, d = 64 108, 111, 112, 109 and 109;
// the mixed ragged batch 243, 244, 242, 244 and 243; 32 ragged sequences of 5 tokens 104, 103, 101, 104 and 106.
constexpr int AT_SETUP = 4;
// A share's least size, in tiles.  1, 2, 4 and 8: one token on 777 keys, 4 KV heads, d = 64 11.9, 12.4, 14.5 and 20.6 us, d = 128
// 14.1, 14.4, 16.5 and 22.5; four sequences, d = 64 14.4, 14.4, 14.4 and 18.3; eight, d = 128 16.5, 16.5, 17.0 and 20.6.
constexpr int AT_MIN_SHARE = 2;
constexpr int AT_CHAIN = 256;             // tiles that the tensor cores add up (a power of 2)
constexpr float AT_SLACK = 24.f;          // log2 of the largest p (sums of values below 2^80 stay in range)
constexpr int AT_SMEM = 232448;           // shared memory a CTA may have
constexpr int AT_MISC = 2048;             // of it for barriers and the like
constexpr int AT_STAGES_MAX = 8;

// four softmax warps and an MMA warp a row tile, and the producer
__host__ __device__ constexpr int at_threads(int NQ) { return NQ * 160 + 32; }
__host__ __device__ constexpr int at_qbytes(int D, int NQ) { return NQ * AT_ROWS * D * 2; }
__host__ __device__ constexpr int at_stage_bytes(int D) { return AT_KEYS * D * 2; }
__host__ __device__ constexpr int at_stages(int D, int NQ)
{
    const int n = (AT_SMEM - AT_MISC - at_qbytes(D, NQ)) / at_stage_bytes(D);
    return n < AT_STAGES_MAX ? n : AT_STAGES_MAX;
}
__host__ __device__ constexpr int at_smem(int D, int NQ)
{
    return at_qbytes(D, NQ) + at_stages(D, NQ) * at_stage_bytes(D) + AT_MISC;
}

// Row tiles of an item, and rows that a piece holds, by the rows T * G of a sequence and KV head.  One tile
// against two: 2048 tokens on 30k keys (8192 rows) 1016 and 771 us, d = 64 877 and 596, the mixed batch of up to 2040
// rows 303 and 243, 16 x 64 tokens on 4k (256 rows) 100 and 77, 16 x 40 (160 rows) 99 and 72; 16 x 32 (128 rows) 63 and 67,
// 16 x 5 (20 rows) 58 and 60, one token (4 rows) on 32k keys 34.5 and 36.9, on 16 x 32k 316 and 321, on 777 keys, d = 64 12.5
// and 14.4.
__host__ __device__ constexpr int at_nq(long long rows) { return rows > AT_ROWS ? 2 : 1; }
__host__ __device__ constexpr int at_piece_rows(long long rows) { return rows > AT_ROWS ? 2 * AT_ROWS : (int)rows; }

struct AttendParams {
    const uint16_t *v;            // the pool (the slow path of values that are not finite)
    const int32_t *table, *pos, *counts;
    uint16_t *out;
    int32_t *ctrl;
    float *part;                  // [cta][2][piece rows][D] sums over V
    float *part_ml;               // [cta][2][piece rows][2] maximum, sum
    int B, T, H_q, H_kv, lg_g, n_max, cols, n_pages, page_shift;
    int window, sinks, piece_rows;
    float k2;                     // scale log2 e
    uint64_t wait_ns;
    int tries;                    // of a wait between two looks at the clock
    uint32_t nap;                 // ns that one may sleep
    int wide;                     // out begins at a multiple of 32 bytes
    int clear;                    // rows of out that no live token writes become zeros
};

// A batch row's tokens; none where pos and counts leave the cache.
__device__ __forceinline__ void at_row(const AttendParams &p, int b, int &first, int &cnt)
{
    first = p.pos[b];
    cnt = p.counts ? p.counts[b] : p.T;
    if (first < 0 || cnt < 0 || cnt > p.T || first > p.n_max - cnt) {
        if (blockIdx.x == 0) set_dev_error(p.ctrl, DEV_BAD_POSITION);
        cnt = 0;
    }
}

// The key tiles of row tile group qt of a batch row.
struct AtItem {
    int first, t0, t1;            // position of token 0; first and last live token
    int lo;                       // least key in the window of any of the tokens
    int nsink, tlo, L;            // tile i is i below nsink, else tlo + i - nsink
    __device__ __forceinline__ int key(int i) const { return (i < nsink ? i : tlo + i - nsink) * AT_KEYS; }
};

template <int NQ>
__device__ __forceinline__ int at_item(const AttendParams &p, int first, int cnt, int qt, AtItem &it)
{
    const int tpi = (NQ * AT_ROWS) >> p.lg_g;
    it.L = 0;
    it.first = first;
    it.t0 = qt * tpi;
    if (it.t0 >= cnt) return 0;
    it.t1 = min(it.t0 + tpi, cnt) - 1;
    const int kmax = first + it.t1;
    it.lo = p.window > 0 ? max(0, first + it.t0 - p.window + 1) : 0;
    it.tlo = it.lo / AT_KEYS;
    it.nsink = (min(p.sinks, kmax + 1) + AT_KEYS - 1) / AT_KEYS;  // (p.sinks is 0 without a window)
    if (it.nsink > 0 && it.nsink >= it.tlo) it.tlo = it.nsink = 0;
    it.L = it.nsink + kmax / AT_KEYS - it.tlo + 1;
    return it.L;
}

// The items of the share [f0, f1) of the list, one after another.
template <int NQ>
struct AtWalk {
    long long base;
    int b, qt, h, qts, first, cnt;
    AtItem it;
    int i0, i1;                   // this share's tiles of the item

    __device__ __forceinline__ void begin(const AttendParams &p, long long f0, long long base_, int pair)
    {
        qts = (p.T + ((NQ * AT_ROWS) >> p.lg_g) - 1) / ((NQ * AT_ROWS) >> p.lg_g);
        b = pair / qts, qt = pair % qts;
        at_row(p, b, first, cnt);
        const int cost = AT_SETUP + at_item<NQ>(p, first, cnt, qt, it);
        h = (int)((f0 - base_) / cost);
        base = base_ + (long long)h * cost;
    }
    __device__ __forceinline__ void step(const AttendParams &p)
    {
        base += AT_SETUP + it.L;
        if (++h < p.H_kv) return;
        h = 0;
        do {
            if (++qt >= qts || qt * ((NQ * AT_ROWS) >> p.lg_g) >= cnt) {
                qt = 0;
                if (++b >= p.B) return;
                at_row(p, b, first, cnt);
            }
        } while (at_item<NQ>(p, first, cnt, qt, it) == 0);
    }
    // Moves to the first item at or after this one of which the share holds a tile.
    __device__ __forceinline__ bool seek(const AttendParams &p, long long f0, long long f1)
    {
        for (;; step(p)) {
            if (base >= f1 || b >= p.B) return false;
            const long long a = f0 - base - AT_SETUP, e = f1 - base - AT_SETUP;
            i0 = (int)max(0ll, min(a, (long long)it.L));
            i1 = (int)max(0ll, min(e, (long long)it.L));
            if (i0 < i1) return true;
        }
    }
    __device__ __forceinline__ bool whole() const { return i0 == 0 && i1 == it.L; }
    __device__ __forceinline__ int live_rows(const AttendParams &p) const { return (it.t1 - it.t0 + 1) << p.lg_g; }
    // whether all tokens of the item see key j; all keys of the tile at `key`
    __device__ __forceinline__ bool all_see(const AttendParams &p, int j) const
    {
        return j <= it.first + it.t0 && (p.window == 0 || j > it.first + it.t1 - p.window || j < p.sinks);
    }
    __device__ __forceinline__ bool open(const AttendParams &p, int key) const
    {
        return key + AT_KEYS - 1 <= it.first + it.t0 &&
               (p.window == 0 || key > it.first + it.t1 - p.window || key + AT_KEYS <= p.sinks);
    }
};

// mbar_wait_bounded for warps that wait long and often beside warps that work: the clock is looked at
// after `tries` tries only, each of which may sleep `nap` ns in the hardware (a line more in this loop, which
// every wait has, cost 3 to 6% of a long chunk's time).  No tries: the wait is given up.
__device__ __forceinline__ bool at_wait(uint64_t *bar, uint32_t parity, uint64_t limit_ns, int tries, uint32_t nap)
{
    uint64_t t0 = 0;
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < tries; ++i) {
            uint32_t ok;
            asm volatile(
                "{\n\t.reg .pred p;\n\t"
                "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(ok)
                : "r"(smem_u32(bar)), "r"(parity), "r"(nap)
                : "memory");
            if (ok) return true;
        }
        const uint64_t t = globaltimer_ns();
        if (t0 == 0) t0 = t;
        if (t - t0 > limit_ns) return false;
    }
}

constexpr int AT_WALK = 96;
static_assert(sizeof(AtWalk<1>) <= AT_WALK && sizeof(AtWalk<2>) <= AT_WALK, "room for a walk");
struct AtSmem {
    uint64_t full[AT_STAGES_MAX], empty[AT_STAGES_MAX];
    uint64_t qfull, qempty;
    uint64_t sfull[2], phalf[2], pfull[2];   // of a score buffer (NQ = 2: one a row tile)
    uint64_t ofull[2][2];         // [row tile][tile % 2]
    uint64_t oempty[2], wg[2], drain[2];
    uint64_t turn[2];             // NQ = 2, items with two row tiles: whose products come next
    long long sums[16];
    long long start_base;
    int start_pair;
    uint32_t tmem;
    int bad_v;                    // a value that is not finite was set to zero
    int timeout;
    int fills, fills_used[2];     // stages filled, and their fills seen by the MMA warps
    int qfills, qfills_used[2];
    int is_last[2];
    int arrived[2][2];            // [slot][row tile]: arrivals of this CTA's pieces
    alignas(16) uint8_t walk[8][AT_WALK];   // the softmax warps' walks: not in their registers
};
static_assert(sizeof(AtSmem) <= AT_MISC, "barriers and the like");

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Weights are 2^(k2 s - r), r = k2 m rounded to fp32: its rounding moves all weights of a row alike.  Where
// that could be by more than 2^0.5 (scores of a size that no model has), they are 2^(k2 (s - m))
// instead, r = k2 m exactly.
constexpr float AT_FAR = 0x1p24f;
__device__ __forceinline__ bool at_far(float m, float k2) { return fabsf(m * k2) >= AT_FAR; }

// 2^(r of m - r of n): what sums of weights taken with m are multiplied with to be sums taken with n.
__device__ __forceinline__ float at_ratio(float m, float n, float k2)
{
    const float rm = m * k2, rn = n * k2;
    const float x = at_far(m, k2) ? (at_far(n, k2) ? (m - n) * k2 : fmaf(m, k2, -rn))
                                  : (at_far(n, k2) ? fmaf(-n, k2, rm) : rm - rn);
    return ex2(x);
}

// Pairs of fp32 numbers in 64 bits, so that one that is used often is packed once.
__device__ __forceinline__ uint64_t pack2(float x, float y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 fma2_packed(float a, float b, uint64_t m, uint64_t c)
{
    float2 r;
    asm("{\n\t.reg .b64 p;\n\tmov.b64 p, {%2, %3};\n\tfma.rn.f32x2 p, p, %4, %5;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a), "f"(b), "l"(m), "l"(c));
    return r;
}
// a += the low half of w, b += the high half, in fp32
__device__ __forceinline__ void add_bf16x2(float &a, float &b, uint32_t w)
{
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tadd.rn.f32.bf16 %0, x, %0;\n\tadd.rn.f32.bf16 %1, y, %1;\n\t}"
        : "+f"(a), "+f"(b)
        : "r"(w));
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// A store to shared memory that whoever reads it finds this thread's earlier ones behind.
__device__ __forceinline__ void st_release(uint32_t *at, uint32_t x)
{
    asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(smem_u32(at)), "r"(x) : "memory");
}

// Whether one of the bf16 halves of w is not finite; bit 15 and bit 31 say which.
__device__ __forceinline__ uint32_t at_not_finite(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

// bits 0 .. x-1
__device__ __forceinline__ uint32_t at_low_bits(int x) { return x <= 0 ? 0u : x >= 32 ? ~0u : (1u << x) - 1u; }

__device__ __forceinline__ uint32_t at_scaled(uint32_t a, uint32_t b, float f)
{
    return bf16x2(__uint_as_float(a) * f, __uint_as_float(b) * f);
}

// Element of `out` where row R (token by token, head by head) of an item begins.
template <int D>
__device__ __forceinline__ size_t out_at(const AttendParams &p, int b, int t0, int h, int R)
{
    return (((size_t)b * p.T + t0 + (R >> p.lg_g)) * p.H_q + (h << p.lg_g) + (R & ((1 << p.lg_g) - 1))) * D;
}

// Float of a piece where columns 4 c .. 4 c + 3 of row r are: row by row where rows are few and the threads
// of a join take columns, else the rows of a column group side by side (a warp's accesses are 512 bytes), a
// thread a row.  The first way against the second: 4 rows and 20 pieces 34.5 and 52.1 us (one token on 32k keys), 2 rows
// and few pieces 12.4 and 14.5 (777 keys), 20 rows 59.6 and 57.3 (16 x 5 tokens on 4k keys) and 104 and 101 (32 ragged
// sequences of 5), 40 rows 65.9 and 58.0, 128 rows 95.8 and 62.4.
constexpr int AT_FEW = 16;
constexpr int AT_BATCH = 10;
template <int D>
__device__ __forceinline__ size_t at_piece(int rows, int r, int c)
{
    return rows > AT_FEW ? ((size_t)c * rows + r) * 4 : (size_t)r * D + 4 * c;
}

// Rows of `out` behind the live tokens of every batch row, all of them where the row is skipped, become
// zeros: equal shares of each to the CTAs of the grid, of a few rows to other CTAs for every batch row.  One warp of a
// CTA calls it, the producer behind its last copy.  Half of 134 MB (32 x 255 tokens of 64 heads, d = 128): 16 us more
// for the call; by all warps before their work 14, but then a call with nothing to clear took 2 more; a fill of the whole
// before the call 40.
template <int D>
__device__ __noinline__ void at_clear(const AttendParams &p)
{
    const int lane = threadIdx.x & 31;
    const long long row = (long long)p.H_q * (D / 8);   // of a token, in 16 bytes
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int mine = b0 + lane;
        int first, cnt = p.T;
        if (mine < p.B) at_row(p, mine, first, cnt);
        for (uint32_t some = __ballot_sync(0xffffffffu, cnt < p.T); some; some &= some - 1) {
            const int at = __ffs(some) - 1, b = b0 + at, live = __shfl_sync(0xffffffffu, cnt, at);
            uint4 *out = reinterpret_cast<uint4 *>(p.out) + ((long long)b * p.T + live) * row;
            const long long n = (p.T - live) * row, step = (long long)gridDim.x * 32;
            const unsigned cta = n < step ? (blockIdx.x + b) % gridDim.x : blockIdx.x;
#pragma unroll 8
            for (long long i = (long long)cta * 32 + lane; i < n; i += step)
                out[i] = make_uint4(0, 0, 0, 0);
        }
    }
}

// CHAINS: a share may have more than AT_CHAIN tiles of an item.  Against the kernel without chains: one token on 16 x
// 64k keys 625 and 620 us, d = 64 on 32 x 128k 1807 and 1780, 2048 tokens on 64k 1493 and 1449, d = 64 1327 and 1367.
template <int D, int NQ, bool CHAINS>
__global__ void __launch_bounds__(at_threads(NQ), 1)
    santa_attend_kernel(const AttendParams p, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v)
{
    constexpr int NT_ = at_threads(NQ);
    constexpr int NW = NT_ / 32;
    constexpr int NS = at_stages(D, NQ);
    constexpr int SB = at_stage_bytes(D);
    constexpr int PANELS = D / 64;
    constexpr int PANEL = AT_KEYS * 128;       // bytes of 64 columns of a tile
    constexpr int W_MMA = NQ * 4, W_PROD = W_MMA + NQ;   // warps: softmax, MMA (one a row tile), producer
    constexpr uint32_t ID_S = idesc_bf16_f32(AT_ROWS, AT_KEYS), ID_O = idesc_bf16_f32(AT_ROWS, D) | IDESC_B_MN;
    constexpr uint32_t O_COL = 256;            // score buffers in columns 0-255, outputs behind them
    constexpr uint32_t P_COL = 64;             // weights over the upper half of their scores
    constexpr unsigned FULL = 0xffffffffu;
    static_assert(NS >= 4, "ring");
    const float NEG_INF = __int_as_float(0xff800000);

    extern __shared__ __align__(1024) uint8_t at_shared[];
    uint8_t *qs = at_shared;
    uint8_t *ring = at_shared + at_qbytes(D, NQ);
    AtSmem &sh = *reinterpret_cast<AtSmem *>(ring + NS * SB);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(FULL, tid >> 5, 0);

    // ---- the list's size, and where this CTA's share begins
    const int tpi = (NQ * AT_ROWS) >> p.lg_g;
    const int qts = (p.T + tpi - 1) / tpi;
    const long long pairs = (long long)p.B * qts;
    const long long per = (pairs + NT_ - 1) / NT_;
    const long long x0 = min(pairs, per * tid), x1 = min(pairs, x0 + per);
    long long mine = 0;
    bool dead = false;   // some token is not live
    {
        int b_at = -1, first = 0, cnt = 0;
        for (long long x = x0; x < x1; ++x) {
            const int b = (int)(x / qts), qt = (int)(x % qts);
            if (b != b_at) at_row(p, b_at = b, first, cnt);
            dead |= cnt < p.T;
            AtItem it;
            const int L = at_item<NQ>(p, first, cnt, qt, it);
            if (L) mine += (long long)p.H_kv * (AT_SETUP + L);
        }
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(FULL, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) sh.sums[warp] = incl;
    const bool clear = __syncthreads_or(p.clear && dead);
    long long total = 0, before = incl - mine;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const long long s = sh.sums[w];
        if (w < warp) before += s;
        total += s;
    }
    const long long ctas = max(1ll, min((long long)gridDim.x, total / AT_MIN_SHARE));
    const long long cta = blockIdx.x;
    if (total == 0 || cta >= ctas) {
        if (clear && warp == 0) at_clear<D>(p);
        return;
    }
    const long long f0 = total * cta / ctas, f1 = total * (cta + 1) / ctas;
    if (before <= f0 && f0 < before + mine) {
        int b_at = -1, first = 0, cnt = 0;
        for (long long x = x0; x < x1; ++x) {
            const int b = (int)(x / qts), qt = (int)(x % qts);
            if (b != b_at) at_row(p, b_at = b, first, cnt);
            AtItem it;
            const int L = at_item<NQ>(p, first, cnt, qt, it);
            const long long cost = L ? (long long)p.H_kv * (AT_SETUP + L) : 0;
            if (f0 < before + cost) {
                sh.start_pair = (int)x;
                sh.start_base = before;
                break;
            }
            before += cost;
        }
    }
    // the CTA whose share holds unit x of the list
    auto owner = [&](long long x) { return (int)(((x + 1) * ctas - 1) / total); };

    // ---- setup: TMEM, barriers
    if (warp == W_MMA) {
        tmem_alloc(&sh.tmem, 512);
        tmem_relinquish();
    }
    if (warp == W_PROD && lane == 0) {
        tma_prefetch_map(&tm_q);
        tma_prefetch_map(&tm_k);
        tma_prefetch_map(&tm_v);
        for (int s = 0; s < NS; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], NQ);
        }
        mbar_init(&sh.qfull, 1);
        mbar_init(&sh.qempty, NQ);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.sfull[i], 1);
            mbar_init(&sh.phalf[i], 4);
            mbar_init(&sh.pfull[i], 4);
            sh.arrived[i][0] = sh.arrived[i][1] = 0;
            mbar_init(&sh.ofull[i][0], 1);
            mbar_init(&sh.ofull[i][1], 1);
            mbar_init(&sh.turn[i], 1);
            mbar_init(&sh.oempty[i], 4);
            mbar_init(&sh.wg[i], 4);
            mbar_init(&sh.drain[i], 1);
            sh.fills_used[i] = sh.qfills_used[i] = 0;
        }
        mbar_fence_init();
        sh.bad_v = sh.timeout = 0;
        sh.fills = sh.qfills = 0;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = sh.tmem;
    auto failed = [&]() {
        set_dev_error(p.ctrl, DEV_TIMEOUT);
        sh.timeout = 1;
    };

    if (warp == W_PROD) {
        // ================= producer
        const int page = 1 << p.page_shift, box = min(page, AT_KEYS);
        const int rows_all = (p.n_pages * p.H_kv) << p.page_shift;   // (below 2^31) beyond the pool: zeros
        AtWalk<NQ> w;
        w.begin(p, f0, sh.start_base, sh.start_pair);
        int n = 0, items = 0, stage = 0, phase = 1;
        bool ok = true;
        for (; ok && w.seek(p, f0, f1); w.step(p), ++items) {
            const int nq = NQ == 2 && w.live_rows(p) > AT_ROWS ? 2 : 1;
            if (items > 0 && !__all_sync(FULL, at_wait(&sh.qempty, (items - 1) & 1, p.wait_ns, p.tries, p.nap))) {
                ok = false;
                break;
            }
            if (lane == 0) {
                mbar_arrive_tx(&sh.qfull, (uint32_t)(nq * AT_ROWS * D * 2));
                for (int i = 0; i < nq; ++i)
                    for (int c = 0; c < PANELS; ++c)
                        tma_load_4d(qs + (i * PANELS + c) * (AT_ROWS * 128), &tm_q, c * 64, w.h << p.lg_g,
                                    w.it.t0 + i * (AT_ROWS >> p.lg_g), w.b, &sh.qfull);
                sh.qfills = items + 1;
            }
            const int kmax = w.it.first + w.it.t1;
            for (int i = w.i0; ok && i < w.i1; ++i, ++n) {
                const int key = w.it.key(i);
                const int boxes = (min(AT_KEYS, kmax + 1 - key) + box - 1) / box;
                // a lane a (page, panel) box
                const int bi = lane / PANELS, c = lane % PANELS;
                int row = 0;
                if (bi < boxes) {
                    const int j = key + bi * box;
                    const int entry = p.table[(size_t)w.b * p.cols + (j >> p.page_shift)];
                    if ((unsigned)entry < (unsigned)p.n_pages) {
                        row = ((entry * p.H_kv + w.h) << p.page_shift) + (j & (page - 1));
                    } else {
                        row = rows_all;
                        if (j + box > w.it.lo || j < p.sinks) set_dev_error(p.ctrl, DEV_BAD_PAGE);   // (else no token sees it)
                    }
                }
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    if (!__all_sync(FULL, at_wait(&sh.empty[stage], phase, p.wait_ns, p.tries, p.nap))) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) {
                        mbar_arrive_tx(&sh.full[stage], (uint32_t)(boxes * box * D * 2));
                        sh.fills = 2 * n + kv + 1;
                    }
                    __syncwarp();
                    if (bi < boxes)
                        tma_load_2d_plain(ring + stage * SB + c * PANEL + bi * box * 128, kv ? &tm_v : &tm_k, c * 64, row,
                                          &sh.full[stage]);
                    if (++stage == NS) stage = 0, phase ^= 1;
                }
            }
        }
        if (!ok && lane == 0) failed();
        __syncwarp();
        if (clear) at_clear<D>(p);
    } else if (warp >= W_MMA) {
        // ================= MMA issuer of row tile q: the whole warp waits, one lane issues
        const int q = warp - W_MMA;
        AtWalk<NQ> w;
        w.begin(p, f0, sh.start_base, sh.start_pair);
        int items = 0;
        int n = 0, no = 0;                    // tiles and chains of this row tile so far
        int turns = 0;                        // turns taken
        bool first_two = true;
        int stage = 0, phase = 0, used = 0;   // of the next fill to wait for
        const uint32_t qaddr = smem_u32(qs) + q * AT_ROWS * D * 2, raddr = smem_u32(ring);
        const uint32_t t_o = tbase + O_COL + q * D;
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (ok) ok = __all_sync(FULL, at_wait(bar, parity, p.wait_ns, p.tries, p.nap));
            return ok;
        };
        // the next fill of the ring (K of a tile, then its V) has landed; its stage
        auto landed = [&]() {
            const int at = stage;
            if (wait(&sh.full[stage], phase)) {
                if (lane == 0) sh.fills_used[q] = ++used;
                if (++stage == NS) stage = 0, phase ^= 1;
            }
            return at;
        };
        // S = Q K^T
        auto scores = [&](int at, int buf) {
            if (elect_one()) {
                const uint64_t k = umma_desc_sw128(raddr + at * SB), a = umma_desc_sw128(qaddr);
#pragma unroll
                for (int x = 0; x < D / 16; ++x)
                    tc_mma_bf16(tbase + buf * AT_KEYS, a + ((x / 4) * (AT_ROWS * 128) + (x % 4) * 32) / 16,
                                k + ((x / 4) * PANEL + (x % 4) * 32) / 16, ID_S, x != 0);
                tc_commit(&sh.sfull[buf]);
                tc_commit(&sh.empty[at]);
            }
            __syncwarp();
        };
        // O += P V over the upper (part 0) or the lower half of the keys
        auto values = [&](int at, int buf, int part, bool first) {
            if (elect_one()) {
                const uint64_t v = umma_desc_sw128_mn(raddr + at * SB, PANEL);
#pragma unroll
                for (int y = 0; y < AT_SUB / 16; ++y) {
                    const int x = y + (part ? 0 : AT_SUB / 16);
                    tc_mma_bf16_ta(t_o, tbase + buf * AT_KEYS + P_COL + x * 8, v + x * (2048 / 16), ID_O, !first || part != 0 || y != 0);
                }
                if (part) {
                    tc_commit(&sh.ofull[q][n & 1]);
                    tc_commit(&sh.empty[at]);
                }
            }
            __syncwarp();
        };
        auto commit = [&](uint64_t *bar) {
            if (elect_one()) tc_commit(bar);
            __syncwarp();
        };
        for (; ok && w.seek(p, f0, f1); w.step(p), ++items) {
            const int L = w.i1 - w.i0;
            if (!wait(&sh.qfull, items & 1)) break;
            if (lane == 0) sh.qfills_used[q] = items + 1;
            if (NQ == 2 && w.live_rows(p) <= q * AT_ROWS) {
                // no row of this tile lives: its stages are given back as they come
                if (lane == 0) mbar_arrive(&sh.qempty);
                for (int f = 0; ok && f < 2 * L; ++f) {
                    const int at = landed();
                    if (ok && lane == 0) mbar_arrive(&sh.empty[at]);
                }
                continue;
            }
            int k_at = landed();
            // two row tiles take turns in the tensor cores, so that one is in its softmax meanwhile: side by
            // side, both would be in the tensor cores and then both in their softmax
            const bool two = NQ == 2 && w.live_rows(p) > AT_ROWS;
            auto my_turn = [&]() {
                if (two) wait(&sh.turn[q], turns++ & 1);
            };
            auto your_turn = [&]() {
                if (two && lane == 0) mbar_arrive(&sh.turn[q ^ 1]);
            };
            if (q == 1 || !first_two) my_turn();
            if (two) first_two = false;
            if (!ok) break;
            tc_fence_after();
            scores(k_at, NQ == 2 ? q : n & 1);
            your_turn();
            if (L == 1) commit(&sh.qempty);
            for (int j = 0; ok && j < L; ++j, ++n) {
                const bool more = j + 1 < L;
                const int buf = NQ == 2 ? q : n & 1;
                const uint32_t parity = (NQ == 2 ? n : n >> 1) & 1;
                const int v_at = landed();
                if (more) k_at = landed();   // (here by the time that the weights are)
                if (!ok) break;
                if (NQ == 1 && more) {       // two buffers: the next scores are under way before
                    tc_fence_after();
                    scores(k_at, (n + 1) & 1);
                    if (j + 2 == L) commit(&sh.qempty);
                }
                wait(&sh.phalf[buf], parity);
                my_turn();
                const bool fresh = CHAINS ? j % AT_CHAIN == 0 : j == 0;
                if (fresh && no++ > 0) wait(&sh.oempty[q], no & 1);
                if (!ok) break;
                tc_fence_after();
                values(v_at, buf, 0, fresh);
                if (!wait(&sh.pfull[buf], parity)) break;
                tc_fence_after();
                values(v_at, buf, 1, fresh);
                if (NQ == 2 && more) {
                    scores(k_at, buf);
                    if (j + 2 == L) commit(&sh.qempty);
                }
                your_turn();
            }
        }
        if (!ok && lane == 0) failed();
        commit(&sh.drain[q]);
        if (lane == 0) mbar_wait_bounded(&sh.drain[q], 0u, DRAIN_NS);
        __syncwarp();
    } else {
        // ================= softmax of row tile q: a thread a row, which is a lane of TMEM
        const int q = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t t_o = tbase + lanes + O_COL + q * D;
        AtWalk<NQ> &w = *reinterpret_cast<AtWalk<NQ> *>(sh.walk[warp]);   // (lane 0 moves it)
        int n = 0, n0 = 0;            // tiles of this row tile so far; tiles of the CTA before the item
        uint32_t wg_phase = 0;
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (ok) ok = __all_sync(FULL, at_wait(bar, parity, p.wait_ns, p.tries, p.nap));
            return ok;
        };
        // rendezvous of the row tile's warps (a bounded wait, unlike bar.sync)
        auto wg_sync = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.wg[q]);
            wait(&sh.wg[q], wg_phase);
            wg_phase ^= 1u;
            return ok;
        };
        int more = 0;
        if (lane == 0) {
            w.begin(p, f0, sh.start_base, sh.start_pair);
            more = w.seek(p, f0, f1);
        }
        auto next = [&]() {
            __syncwarp();
            if (lane == 0) {
                w.step(p);
                more = w.seek(p, f0, f1);
            }
        };
        for (; ok && __shfl_sync(FULL, more, 0); next()) {
            __syncwarp();
            const int live = w.live_rows(p) - q * AT_ROWS;   // of this row tile
            const int tiles = w.i1 - w.i0;
            if (live <= 0) {
                n0 += tiles;
                continue;
            }
            const bool warp_live = 32 * (warp & 3) < live;
            const int P = w.it.first + w.it.t0 + ((q * AT_ROWS + row) >> p.lg_g);
            const int seen_lo = p.window > 0 ? P - p.window + 1 : 0;
            // a tile that begins before the one and after the other all tokens see whole
            const int open_hi = w.it.first + w.it.t0 - AT_KEYS + 2, open_lo = p.window > 0 ? w.it.first + w.it.t1 - p.window : -1;
            int key = w.it.key(w.i0), left = w.it.nsink - w.i0;
            // m: the reference of the row's weights (a score so far); off, sub: how they are taken with it
            float m = NEG_INF, l = 0.f, off = 0.f, sub = 0.f;
            bool any_far = false;
            // The output of a chain of AT_CHAIN tiles is added to that of the chains before it, which is kept in this
            // CTA's piece; `last`: the other way round, for the item's end.  `i` tiles are done.
            auto chain = [&](int i, bool last) {
                const int R = q * AT_ROWS + row;
                const bool mine_live = row < live, some = last || i > AT_CHAIN;
                const size_t at = (size_t)(blockIdx.x * 2 + (w.i0 > 0 ? 0 : 1)) * p.piece_rows;
                float f = 0.f;
                if (some && mine_live) {
                    const float was = __ldcg(p.part_ml + (at + R) * 2);
                    f = was == NEG_INF ? 0.f : at_ratio(was, m, p.k2);
                }
#pragma unroll 1
                for (int c = 0; c < D; c += 8) {
                    uint32_t o[8];
                    __syncwarp();
                    tmem_ld32<8>(t_o + c, o);
                    if (mine_live) {
#pragma unroll
                        for (int e = 0; e < 8; e += 4) {
                            float4 *sum = reinterpret_cast<float4 *>(p.part + at * D + at_piece<D>(p.piece_rows, R, (c + e) / 4));
                            const float4 x = some ? __ldcg(sum) : make_float4(0.f, 0.f, 0.f, 0.f);
                            o[e] = __float_as_uint(fmaf(f, x.x, __uint_as_float(o[e])));
                            o[e + 1] = __float_as_uint(fmaf(f, x.y, __uint_as_float(o[e + 1])));
                            o[e + 2] = __float_as_uint(fmaf(f, x.z, __uint_as_float(o[e + 2])));
                            o[e + 3] = __float_as_uint(fmaf(f, x.w, __uint_as_float(o[e + 3])));
                            if (!last) __stcg(reinterpret_cast<uint4 *>(sum), make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]));
                        }
                    }
                    __syncwarp();
                    if (last) tmem_st8(t_o + c, o);
                }
                if (last)
                    tmem_st_wait();
                else if (mine_live)
                    __stcg(p.part_ml + (at + R) * 2, m);
            };
            for (int i = 0; i < tiles; ++i, ++n) {
                if (CHAINS && i > 0 && i % AT_CHAIN == 0) {
                    if (!wait(&sh.ofull[q][(n - 1) & 1], ((n - 1) >> 1) & 1)) break;
                    tc_fence_after();
                    if (warp_live) chain(i, false);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.oempty[q]);
                }
                const int buf = NQ == 2 ? q : n & 1;
                const uint32_t t_s = tbase + lanes + buf * AT_KEYS;
                const bool open = key < open_hi && (key > open_lo || key + AT_KEYS <= p.sinks);
                if (!wait(&sh.sfull[buf], (NQ == 2 ? n : n >> 1) & 1)) break;
                if (!open) {
                    // values of V that are not finite become zeros (both row tiles' warps look at all of
                    // them: what the other has set to zero is zero, or becomes it twice)
                    const int f = 2 * (n0 + i) + 1;
                    if (!wait(&sh.full[f % NS], (f / NS) & 1)) break;
                    uint8_t *v = ring + (f % NS) * SB;
                    auto clear = [&](int r0, int r1) {   // in rows r0 .. r1 - 1
                        uint32_t bad = 0;
#pragma unroll
                        for (int h = 0; h < PANELS; ++h)
#pragma unroll 8
                            for (int c = 8 * r0 + row; c < 8 * r1; c += 128) {
                                const uint4 x = *reinterpret_cast<const uint4 *>(v + h * PANEL + c * 16);
                                bad |= at_not_finite(x.x) | at_not_finite(x.y) | at_not_finite(x.z) | at_not_finite(x.w);
                            }
                        if (bad == 0) return;   // (nearly always)
                        for (int h = 0; h < PANELS; ++h)
                            for (int c = 8 * r0 + row; c < 8 * r1; c += 128) {
                                uint4 &at = *reinterpret_cast<uint4 *>(v + h * PANEL + c * 16);
                                const uint4 x = at;
                                const uint4 y = make_uint4(x.x & ~((at_not_finite(x.x) >> 15) * 0xffffu), x.y & ~((at_not_finite(x.y) >> 15) * 0xffffu),
                                                           x.z & ~((at_not_finite(x.z) >> 15) * 0xffffu), x.w & ~((at_not_finite(x.w) >> 15) * 0xffffu));
                                if (x.x == y.x && x.y == y.y && x.z == y.z && x.w == y.w) continue;
                                const int j = key + c / 8;
                                if (j <= w.it.first + w.it.t1 && (j >= w.it.lo || j < p.sinks)) *(volatile int *)&sh.bad_v = 1;
                                st_release(&at.x, y.x);   // (who finds zeros finds the flag)
                                st_release(&at.y, y.y);
                                st_release(&at.z, y.z);
                                st_release(&at.w, y.w);
                            }
                    };
                    // keys beyond the first token, and keys before the last one's window
                    const int beyond = min(AT_KEYS, max(0, w.it.first + w.it.t0 + 1 - key));
                    clear(beyond, AT_KEYS);
                    if (p.window > 0) clear(max(0, p.sinks - key), min(beyond, w.it.first + w.it.t1 - p.window + 1 - key));
                    fence_proxy_async_smem();
                }
                if (warp_live) {
                    tc_fence_after();
                    // the upper half of the scores stays in registers, the lower half is read again (all kept,
                    // or both halves read again: 2 to 3% more of a long chunk's time)
                    uint32_t lower[AT_SUB], upper[AT_SUB];
                    auto hide = [&](uint32_t (&s)[AT_SUB], int at) {
#pragma unroll
                        for (int c = 0; c < AT_SUB; c += 32) {
                            const int k0 = key + at + c;
                            const uint32_t seen = at_low_bits(P + 1 - k0) & (~at_low_bits(seen_lo - k0) | at_low_bits(p.sinks - k0));
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!((seen >> e) & 1u)) s[c + e] = 0xff800000u;
                        }
                    };
                    float mx[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
                    auto most = [&](const uint32_t (&s)[AT_SUB]) {
#pragma unroll
                        for (int e = 0; e < AT_SUB; e += 8)
#pragma unroll
                            for (int c = 0; c < 4; ++c) mx[c] = max3(mx[c], __uint_as_float(s[e + 2 * c]), __uint_as_float(s[e + 2 * c + 1]));
                    };
                    tmem_ld32_two(t_s, lower, t_s + AT_SUB, upper);
                    if (!open) {
                        hide(lower, 0);
                        hide(upper, AT_SUB);
#pragma unroll
                        for (int c = 0; c < AT_SUB; c += 8) tmem_st8(t_s + c, lower + c);   // (as it is read again)
                    }
                    most(lower);
                    most(upper);
                    const float top = max3(mx[0], mx[1], fmaxf(mx[2], mx[3]));
                    const bool grow = (top - m) * p.k2 > AT_SLACK;   // (a first one: infinity)
                    if (__any_sync(FULL, grow)) {
                        const float f = grow ? (m == NEG_INF ? 0.f : at_ratio(m, top, p.k2)) : 1.f;
                        if (grow) m = top;
                        l *= f;
                        const bool far = at_far(m == NEG_INF ? 0.f : m, p.k2);
                        sub = far ? m : 0.f;
                        off = far || m == NEG_INF ? 0.f : -(m * p.k2);
                        any_far = __any_sync(FULL, far);
                        if (i > 0) {
                            if (!wait(&sh.ofull[q][(n - 1) & 1], ((n - 1) >> 1) & 1)) break;
                            tc_fence_after();
#pragma unroll 1
                            for (uint32_t at = t_o; at < t_o + D; at += 16) {
                                uint32_t o[16];
                                tmem_ld32<16>(at, o);
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tmem_st8(at, o);
                                tmem_st8(at + 8, o + 8);
                            }
                        }
                    }
                    const uint64_t k2k2 = pack2(p.k2, p.k2), offoff = pack2(off, off);
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
                    auto weigh = [&](uint32_t (&x)[AT_SUB], int at) {
                        if (any_far) {
#pragma unroll
                            for (int e = 0; e < AT_SUB; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) - sub);
                        }
#pragma unroll
                        for (int c = 0; c < AT_SUB; c += 16) {
                            uint32_t pk[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float2 y = fma2_packed(__uint_as_float(x[c + 2 * e]), __uint_as_float(x[c + 2 * e + 1]), k2k2, offoff);
                                pk[e] = bf16x2(ex2(y.x), ex2(y.y));
                                add_bf16x2(sum[2 * (e & 1)], sum[2 * (e & 1) + 1], pk[e]);
                            }
                            tmem_st8(t_s + P_COL + (at + c) / 2, pk);
                        }
                    };
                    auto told = [&](uint64_t *bar) {
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar);
                    };
                    weigh(upper, AT_SUB);
                    told(&sh.phalf[buf]);
                    tmem_ld32<AT_SUB>(t_s, lower);
                    weigh(lower, 0);
                    told(&sh.pfull[buf]);
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                } else {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sh.phalf[buf]);
                        mbar_arrive(&sh.pfull[buf]);
                    }
                }
                key += AT_KEYS;
                if (--left == 0) key = w.it.tlo * AT_KEYS;
            }
            n0 += tiles;
            if (!ok) break;
            // (a parity tells only a phase from the next.  When scores are here, the product of two tiles before
            // is done and that of the tile before may be: one barrier would be one or two phases on)
            if (!wait(&sh.ofull[q][(n - 1) & 1], ((n - 1) >> 1) & 1)) break;
            tc_fence_after();

            if (CHAINS && tiles > AT_CHAIN && warp_live) chain(tiles, true);

            // ---- the item's (or the piece's) sums
            const bool whole = w.whole(), mine_live = row < live;
            const bool fix = *reinterpret_cast<volatile int *>(&sh.bad_v) != 0;
            const int slot = w.i0 > 0 ? 0 : 1;
            const int R = q * AT_ROWS + row;
            if (warp_live) {
                const float inv = whole ? 1.f / l : 1.f;
                const size_t slot_at = (size_t)(blockIdx.x * 2 + slot) * p.piece_rows;
#pragma unroll 1
                for (int c = 0; c < D; c += 64) {
                    uint32_t o[64];
                    tmem_ld32<64>(t_o + c, o);
                    if (fix && mine_live) {
                        // values that are not finite, of the keys that this row sees
                        for (int x = w.i0; x < w.i1; ++x) {
                            const int first = w.it.key(x);
                            if (w.open(p, first)) continue;
                            for (int j = first; j < first + AT_KEYS && j <= P; ++j) {
                                if (w.all_see(p, j) || (p.window > 0 && j <= P - p.window && j >= p.sinks)) continue;
                                const int entry = p.table[(size_t)w.b * p.cols + (j >> p.page_shift)];
                                if ((unsigned)entry >= (unsigned)p.n_pages) continue;
                                const uint32_t *v = reinterpret_cast<const uint32_t *>(
                                    p.v + ((((long long)entry * p.H_kv + w.h) << p.page_shift) + (j & ((1 << p.page_shift) - 1))) * D + c);
#pragma unroll
                                for (int e = 0; e < 32; ++e) {
                                    const uint32_t u = v[e], bad = at_not_finite(u);
                                    if (bad & 0x8000u) o[2 * e] = __float_as_uint(__uint_as_float(o[2 * e]) + bf16lo_to_f32(u));
                                    if (bad >> 31) o[2 * e + 1] = __float_as_uint(__uint_as_float(o[2 * e + 1]) + bf16hi_to_f32(u));
                                }
                            }
                        }
                    }
                    if (!mine_live) continue;
                    if (whole) {
                        uint16_t *out = p.out + out_at<D>(p, w.b, w.it.t0, w.h, R) + c;
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = at_scaled(o[2 * e], o[2 * e + 1], inv);
                        if (p.wide) {
#pragma unroll
                            for (int e = 0; e < 32; e += 8)
                                asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(o[e]), "r"(o[e + 1]),
                                             "r"(o[e + 2]), "r"(o[e + 3]), "r"(o[e + 4]), "r"(o[e + 5]), "r"(o[e + 6]), "r"(o[e + 7]),
                                             "l"(__cvta_generic_to_global(out + 2 * e))
                                             : "memory");
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; e += 4)
                                *reinterpret_cast<uint4 *>(out + 2 * e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                        }
                    } else {
                        float *piece = p.part + slot_at * D;
#pragma unroll
                        for (int e = 0; e < 64; e += 4)
                            __stcg(reinterpret_cast<uint4 *>(piece + at_piece<D>(p.piece_rows, R, (c + e) / 4)),
                                   make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]));
                    }
                }
                if (!whole && mine_live) __stcg(reinterpret_cast<float2 *>(p.part_ml + (slot_at + R) * 2), make_float2(m, l));
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.oempty[q]);

            // ---- a piece: the last CTA of the item to arrive joins them all
            if (!whole) {
                const int c0 = owner(w.base + AT_SETUP), c1 = owner(w.base + AT_SETUP + w.it.L - 1);
                __threadfence();
                if (wg_sync() && row == 0) {
                    int32_t *arrivals = p.ctrl + CTRL_GROUPS + 2 * c0 + q;
                    sh.arrived[slot][q] = 1;
                    const bool last = atomicAdd(arrivals, 1) == c1 - c0;
                    if (last) *arrivals = 0;
                    sh.is_last[q] = last;
                    __threadfence();
                }
                if (wg_sync() && sh.is_last[q]) {
                    __threadfence();
                    const int rows_live = min(live, AT_ROWS);
                    auto at = [&](int c) { return (size_t)(c * 2 + (c == c0 ? 1 : 0)) * p.piece_rows; };
                    if (p.piece_rows > AT_FEW) {
                        // a thread a row, 64 columns at a time: a row's pieces lie side by side for the lanes
                        if (mine_live) {
                            float M = NEG_INF, sl = 0.f;
#pragma unroll 4
                            for (int c = c0; c <= c1; ++c) M = fmaxf(M, __ldcg(p.part_ml + (at(c) + R) * 2));
#pragma unroll 1
                            for (int x = 0; x < D / 4; x += 16) {
                                float4 o[16];
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                                sl = 0.f;
#pragma unroll 1
                                for (int c = c0; c <= c1; ++c) {
                                    const float2 ml = __ldcg(reinterpret_cast<const float2 *>(p.part_ml + (at(c) + R) * 2));
                                    float4 v[16];
#pragma unroll
                                    for (int e = 0; e < 16; ++e)
                                        v[e] = __ldcg(reinterpret_cast<const float4 *>(p.part + at(c) * D + at_piece<D>(p.piece_rows, R, x + e)));
                                    const float f = ml.x == NEG_INF ? 0.f : at_ratio(ml.x, M, p.k2);
                                    sl = fmaf(f, ml.y, sl);
#pragma unroll
                                    for (int e = 0; e < 16; ++e) {
                                        o[e].x = fmaf(f, v[e].x, o[e].x), o[e].y = fmaf(f, v[e].y, o[e].y);
                                        o[e].z = fmaf(f, v[e].z, o[e].z), o[e].w = fmaf(f, v[e].w, o[e].w);
                                    }
                                }
                                const float inv = 1.f / sl;
                                uint16_t *out = p.out + out_at<D>(p, w.b, w.it.t0, w.h, R) + 4 * x;
#pragma unroll
                                for (int e = 0; e < 16; e += 2)
                                    *reinterpret_cast<uint4 *>(out + 4 * e) =
                                        make_uint4(bf16x2(o[e].x * inv, o[e].y * inv), bf16x2(o[e].z * inv, o[e].w * inv),
                                                   bf16x2(o[e + 1].x * inv, o[e + 1].y * inv), bf16x2(o[e + 1].z * inv, o[e + 1].w * inv));
                            }
                        }
                    } else {
                        // few rows, many pieces: a thread four columns of a row
                        for (int x = row; x < rows_live * (D / 4); x += 128) {
                            const int r = x / (D / 4), e = x % (D / 4);
                            // AT_BATCH pieces are on their way at a time
                            float M = NEG_INF, sl = 0.f, o0 = 0.f, o1 = 0.f, o2 = 0.f, o3 = 0.f;
                            for (int c = c0; c <= c1; c += AT_BATCH) {
                                float2 ml[AT_BATCH];
                                float4 o[AT_BATCH];
#pragma unroll
                                for (int y = 0; y < AT_BATCH; ++y) {
                                    ml[y] = make_float2(NEG_INF, 0.f);
                                    o[y] = make_float4(0.f, 0.f, 0.f, 0.f);
                                    if (c + y <= c1) {
                                        ml[y] = __ldcg(reinterpret_cast<const float2 *>(p.part_ml + (at(c + y) + r) * 2));
                                        o[y] = __ldcg(reinterpret_cast<const float4 *>(p.part + at(c + y) * D + at_piece<D>(p.piece_rows, r, e)));
                                    }
                                }
                                float N = M;
#pragma unroll
                                for (int y = 0; y < AT_BATCH; ++y) N = fmaxf(N, ml[y].x);
                                const float g = M == NEG_INF ? 0.f : at_ratio(M, N, p.k2);
                                M = N;
                                sl *= g, o0 *= g, o1 *= g, o2 *= g, o3 *= g;
#pragma unroll
                                for (int y = 0; y < AT_BATCH; ++y) {
                                    const float f = ml[y].x == NEG_INF ? 0.f : at_ratio(ml[y].x, M, p.k2);
                                    sl = fmaf(f, ml[y].y, sl);
                                    o0 = fmaf(f, o[y].x, o0), o1 = fmaf(f, o[y].y, o1), o2 = fmaf(f, o[y].z, o2), o3 = fmaf(f, o[y].w, o3);
                                }
                            }
                            const float inv = 1.f / sl;
                            *reinterpret_cast<uint2 *>(p.out + out_at<D>(p, w.b, w.it.t0, w.h, r) + 4 * e) =
                                make_uint2(bf16x2(o0 * inv, o1 * inv), bf16x2(o2 * inv, o3 * inv));
                        }
                    }
                }
            }
        }
        if (!ok && lane == 0) failed();
        __syncwarp();
        tmem_st_wait();   // (after a wait that ran out, stores to TMEM may be under way)
    }

    // ---- teardown: every MMA and every store to TMEM has completed (waited for above); release TMEM.  After a timeout, copies
    // that were not waited for get a bounded wait to land, and pieces that did not arrive do, so that
    // the counters are zero again after the last CTA.
    tc_fence_before();
    __syncthreads();
    if (warp == W_MMA) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
    if (warp == W_PROD && lane == 0 && sh.timeout) {
        for (int f = NQ == 2 ? min(sh.fills_used[0], sh.fills_used[1]) : sh.fills_used[0]; f < sh.fills; ++f)
            if (!mbar_wait_bounded(&sh.full[f % NS], (f / NS) & 1, DRAIN_NS)) break;
        if (sh.qfills_used[0] < sh.qfills || (NQ == 2 && sh.qfills_used[1] < sh.qfills))
            mbar_wait_bounded(&sh.qfull, (sh.qfills - 1) & 1, DRAIN_NS);
        AtWalk<NQ> a;
        a.begin(p, f0, sh.start_base, sh.start_pair);
        for (; a.seek(p, f0, f1); a.step(p)) {
            if (a.whole()) continue;
            const int c0 = owner(a.base + AT_SETUP), c1 = owner(a.base + AT_SETUP + a.it.L - 1);
            for (int q = 0; q < NQ && a.live_rows(p) > q * AT_ROWS; ++q) {
                int32_t *arrivals = p.ctrl + CTRL_GROUPS + 2 * c0 + q;
                if (!sh.arrived[a.i0 > 0 ? 0 : 1][q] && atomicAdd(arrivals, 1) == c1 - c0) *arrivals = 0;
            }
        }
    }
}

}  // namespace santa

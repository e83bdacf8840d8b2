// santa_paged_api.cu -- the entry points of rotary positions, of the paged cache and of attention
// over it (declared in include/santa.h): argument checks and launches.
#include <algorithm>
#include <cmath>
#include <utility>

#include "../../include/santa.h"
#include "santa_attend.cuh"
#include "santa_host.h"
#include "santa_rope.cuh"

using namespace santa;

namespace {

// Strides of rows [B, T, H, d] that are read, or (`distinct`) written: no two rows written may
// share memory.  In order of size each stride has to step over all that the smaller ones span.
int check_strides(const int64_t *st, long long B, long long T, long long H, int d, bool distinct)
{
    const long long dims[3] = {B, T, H};
    int order[3] = {0, 1, 2};
    for (int i = 0; i < 3; ++i) {
        if (dims[i] <= 1) continue;  // this stride is never used
        if (st[i] < 0 || st[i] > (1ll << 40)) return SANTA_ERR_INVALID_ARG;
        if (st[i] % 8 != 0) return SANTA_ERR_MISALIGNED;
    }
    if (!distinct) return SANTA_OK;
    for (int i = 1; i < 3; ++i)
        for (int j = i; j > 0 && st[order[j]] < st[order[j - 1]]; --j) std::swap(order[j], order[j - 1]);
    long long extent = d;
    for (int i = 0; i < 3; ++i) {
        const int x = order[i];
        if (dims[x] <= 1) continue;
        if (st[x] < extent || dims[x] - 1 > ((1ll << 60) - extent) / st[x]) return SANTA_ERR_INVALID_ARG;
        extent += st[x] * (dims[x] - 1);
    }
    return SANTA_OK;
}

int check_rotation(const santa_rotation *r, int d)
{
    if (!r->turns || (r->layout != SANTA_ROPE_HALVES && r->layout != SANTA_ROPE_PAIRS) || !std::isfinite(r->amplitude))
        return SANTA_ERR_INVALID_ARG;
    if (!aligned(r->turns, 8)) return SANTA_ERR_MISALIGNED;
    return r->rot >= 16 && r->rot <= d && r->rot % 16 == 0 ? SANTA_OK : SANTA_ERR_UNSUPPORTED;
}

// Shape and pool of a paged cache (its limits on n_max hold for one sequence, not for the batch).
int check_paged(const santa_shape *sh, const santa_paged *c)
{
    if (!sh) return SANTA_ERR_INVALID_ARG;
    santa_shape one = *sh;
    one.B = std::min(one.B, 1);
    int rc = check_shape(&one);
    if (rc) return rc;
    if (sh->B > BMAX) return SANTA_ERR_UNSUPPORTED;
    if (!c || !c->k || !c->v || !c->table || c->n_pages < 1) return SANTA_ERR_INVALID_ARG;
    if (c->page < 16 || c->page > 256 || (c->page & (c->page - 1)) || sh->n_max % c->page != 0 ||
        (long long)c->n_pages * sh->H_kv * c->page >= (1ll << 31))
        return SANTA_ERR_UNSUPPORTED;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->table, 4)) return SANTA_ERR_MISALIGNED;
    return SANTA_OK;
}

// T of a call is the number of tokens and a flag.
bool take_clear(int32_t &T)
{
    const bool clear = T > 0 && (T & SANTA_CLEAR_REST);
    if (clear) T &= ~SANTA_CLEAR_REST;
    return clear;
}

template <int D>
const void *attend_kernel(int NQ, bool chains)
{
    if (NQ == 2) return chains ? (const void *)santa_attend_kernel<D, 2, true> : (const void *)santa_attend_kernel<D, 2, false>;
    return chains ? (const void *)santa_attend_kernel<D, 1, true> : (const void *)santa_attend_kernel<D, 1, false>;
}

int log2_of(int x)
{
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

RopeRows rope_rows(const void *src, const int64_t *ss, void *dst, const int64_t *ds)
{
    RopeRows r{};
    r.src = static_cast<const uint16_t *>(src);
    r.dst = static_cast<uint16_t *>(dst);
    r.sb = ss[0], r.st = ss[1], r.sh = ss[2];
    if (ds) r.db = ds[0], r.dt = ds[1], r.dh = ds[2];
    return r;
}

int launch_rope(RopeParams &p, int d, const santa_rotation *rotation, void *stream)
{
    const long long heads = p.H_q + 2ll * p.H_kv;
    if (p.T > 0 && heads * p.B * (d / RP_VALUES) > ((1ll << 31) - 1) / p.T) return SANTA_ERR_UNSUPPORTED;
    if (p.T == 0) return SANTA_OK;
    if (rotation) {
        p.rot = rotation->rot;
        p.turns = rotation->turns;
        p.amplitude = rotation->amplitude;
    }
    int dev, sms, optin, rc;
    if ((rc = device_info(&dev, &sms, &optin))) return rc;
    // as many rows to a thread as leave every SM its threads twice over
    const long long all = heads * p.B * p.T * (d / RP_VALUES);
    const long long each = std::min<long long>(RP_HEADS, std::max<long long>(1, all / (2ll * 2048 * sms)));
    p.groups = (int)((heads + each - 1) / each);
    const bool pairs = rotation && rotation->layout == SANTA_ROPE_PAIRS;
    const void *fn = d == 128 ? (pairs ? (const void *)santa_rope_kernel<128, true> : (const void *)santa_rope_kernel<128, false>)
                              : (pairs ? (const void *)santa_rope_kernel<64, true> : (const void *)santa_rope_kernel<64, false>);
    const long long threads = (long long)p.T * p.groups * (d / RP_VALUES);
    const dim3 grid((unsigned)((threads + RP_NT - 1) / RP_NT), (unsigned)p.B);
    void *args[] = {&p};
    return cudaLaunchKernel(fn, grid, dim3(RP_NT), args, 0, (cudaStream_t)stream) == cudaSuccess ? SANTA_OK : SANTA_ERR_CUDA;
}

}  // namespace

extern "C" {

int santa_rope_turns(const santa_rope_spec *s, int32_t rot, uint64_t *turns, float *amplitude)
{
    if (!s || !turns || !amplitude || rot < 2 || rot % 2 != 0 || rot > 65536) return SANTA_ERR_INVALID_ARG;
    if (!(s->base > 1.0) || !std::isfinite(s->base)) return SANTA_ERR_INVALID_ARG;
    const int how = s->scaling;
    if (how < SANTA_ROPE_SCALE_NONE || how > SANTA_ROPE_SCALE_RAMP) return SANTA_ERR_INVALID_ARG;
    if (how != SANTA_ROPE_SCALE_NONE && (!(s->factor >= 1.0) || !std::isfinite(s->factor))) return SANTA_ERR_INVALID_ARG;
    if (how >= SANTA_ROPE_SCALE_BANDS && (!(s->low > 0.0) || !(s->high > s->low) || !std::isfinite(s->high) || s->original < 1))
        return SANTA_ERR_INVALID_ARG;
    if (how == SANTA_ROPE_SCALE_BASE && rot < 4) return SANTA_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925286766559;
    const double base = how == SANTA_ROPE_SCALE_BASE ? s->base * std::pow(s->factor, (double)rot / (rot - 2)) : s->base;
    if (!std::isfinite(base)) return SANTA_ERR_INVALID_ARG;
    double first = 0.0, last = 0.0;  // RAMP: the pairs between which the blend runs
    if (how == SANTA_ROPE_SCALE_RAMP) {
        auto index = [&](double n) { return rot * std::log(s->original / (two_pi * n)) / (2.0 * std::log(base)); };
        first = std::max(std::floor(index(s->high)), 0.0);
        last = std::max(std::min(std::ceil(index(s->low)), rot - 1.0), first + 0.001);
    }
    for (int i = 0; i < rot / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot);
        double keep = 1.0;  // how much of f is not divided
        if (how == SANTA_ROPE_SCALE_LINEAR)
            keep = 0.0;
        else if (how == SANTA_ROPE_SCALE_BANDS)
            keep = std::min(std::max((s->original * f / two_pi - s->low) / (s->high - s->low), 0.0), 1.0);
        else if (how == SANTA_ROPE_SCALE_RAMP)
            keep = 1.0 - std::min(std::max((i - first) / (last - first), 0.0), 1.0);
        if (keep < 1.0) f = keep * f + (1.0 - keep) * f / s->factor;
        turns[i] = (uint64_t)(f / two_pi * 18446744073709551616.0);  // f <= 1: below 2^62
    }
    *amplitude = how == SANTA_ROPE_SCALE_RAMP ? (float)(0.1 * std::log(s->factor) + 1.0) : 1.f;
    return SANTA_OK;
}

int santa_rope(int32_t B, int32_t T, int32_t H, int32_t d, const void *x, const int64_t x_stride[3], void *out,
               const int64_t out_stride[3], const santa_rotation *rotation, const int32_t *pos, const int32_t *counts,
               void *workspace, void *stream)
{
    const bool clear = take_clear(T);
    if (B < 1 || T < 0 || H < 1 || d < 1 || !x || !x_stride || !out || !out_stride || !rotation || !pos)
        return SANTA_ERR_INVALID_ARG;
    if (B > BMAX || H > 1024 || (d != 64 && d != 128)) return SANTA_ERR_UNSUPPORTED;
    if (!aligned(x, 16) || !aligned(out, 16) || !aligned(pos, 4) || (counts && !aligned(counts, 4)) ||
        (workspace && !aligned(workspace, 256)))
        return SANTA_ERR_MISALIGNED;
    int rc;
    if ((rc = check_rotation(rotation, d)) || (rc = check_strides(x_stride, B, T, H, d, false)) ||
        (rc = check_strides(out_stride, B, T, H, d, true)))
        return rc;
    RopeParams p{};
    p.q = rope_rows(x, x_stride, out, out_stride);
    p.B = B, p.T = T, p.H_q = H;
    p.clear = clear;
    p.pos = pos, p.counts = counts;
    p.last = 0x7fffffff;
    p.ctrl = static_cast<int32_t *>(workspace);
    return launch_rope(p, d, rotation, stream);
}

int santa_paged_append(const santa_shape *shape, const santa_paged *cache, const santa_rows *rows, int32_t T,
                       const int32_t *pos, const int32_t *counts, const santa_rotation *rotation, const void *q,
                       const int64_t q_stride[3], void *q_out, const int64_t q_out_stride[3], void *workspace,
                       void *stream)
{
    const bool clear = take_clear(T);
    int rc = check_paged(shape, cache);
    if (rc) return rc;
    if (!rows || !rows->k || !rows->v || !pos || T < 0 || !q != !q_out) return SANTA_ERR_INVALID_ARG;
    if (cache->k == cache->v) return SANTA_ERR_INVALID_ARG;  // (K and V would be written to the same rows)
    if (q && (!q_stride || !q_out_stride || !rotation)) return SANTA_ERR_INVALID_ARG;
    if (!aligned(rows->k, 16) || !aligned(rows->v, 16) || !aligned(pos, 4) || (counts && !aligned(counts, 4)) ||
        (q && (!aligned(q, 16) || !aligned(q_out, 16))) || (workspace && !aligned(workspace, 256)))
        return SANTA_ERR_MISALIGNED;
    const int B = shape->B, d = shape->d;
    if ((rotation && (rc = check_rotation(rotation, d))) || (rc = check_strides(rows->k_stride, B, T, shape->H_kv, d, false)) ||
        (rc = check_strides(rows->v_stride, B, T, shape->H_kv, d, false)))
        return rc;
    if (q && ((rc = check_strides(q_stride, B, T, shape->H_q, d, false)) ||
              (rc = check_strides(q_out_stride, B, T, shape->H_q, d, true))))
        return rc;
    RopeParams p{};
    if (q) p.q = rope_rows(q, q_stride, q_out, q_out_stride);
    p.k = rope_rows(rows->k, rows->k_stride, cache->k, nullptr);
    p.v = rope_rows(rows->v, rows->v_stride, cache->v, nullptr);
    p.B = B, p.T = T;
    p.clear = clear;
    p.H_q = q ? shape->H_q : 0;
    p.H_kv = shape->H_kv;
    p.pos = pos, p.counts = counts;
    p.last = shape->n_max;
    p.table = cache->table;
    p.cols = shape->n_max / cache->page;
    p.n_pages = cache->n_pages;
    p.page_shift = log2_of(cache->page);
    p.ctrl = static_cast<int32_t *>(workspace);
    return launch_rope(p, d, rotation, stream);
}

int santa_attend_workspace_size(const santa_shape *shape, int32_t T, size_t *bytes)
{
    if (!shape) return SANTA_ERR_INVALID_ARG;
    santa_shape one = *shape;
    one.B = std::min(one.B, 1);
    one.n_max = 1;
    const int rc = check_shape(&one);
    if (rc) return rc;
    if (!bytes || T < 0) return SANTA_ERR_INVALID_ARG;
    if (shape->B > BMAX || T > NMAX_LIMIT) return SANTA_ERR_UNSUPPORTED;
    const size_t rows = (size_t)at_piece_rows((long long)T * (shape->H_q / shape->H_kv));
    *bytes = align_up(CTRL_BYTES + (size_t)AT_MAX_CTAS * 2 * rows * (shape->d + 2) * sizeof(float), 256);
    return SANTA_OK;
}

int santa_attend_paged(const santa_shape *shape, const void *q, const int64_t q_stride[3], const santa_paged *cache,
                       int32_t T, const int32_t *pos, const int32_t *counts, int32_t window, int32_t sinks, void *out,
                       void *workspace, size_t workspace_bytes, void *stream)
{
    const bool clear = take_clear(T);
    int rc = check_paged(shape, cache);
    if (rc) return rc;
    if (!q || !q_stride || !pos || !out || T < 0 || window < 0 || sinks < 0 || shape->scale < 0.f) return SANTA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(pos, 4) || (counts && !aligned(counts, 4)))
        return SANTA_ERR_MISALIGNED;
    size_t need = 0;
    if ((rc = santa_attend_workspace_size(shape, T, &need)) || (rc = check_strides(q_stride, shape->B, T, shape->H_q, shape->d, false)))
        return rc;
    // (a tensor copy's strides are below 2^40 bytes)
    const long long dims[3] = {shape->B, T, shape->H_q};
    for (int i = 0; i < 3; ++i)
        if (dims[i] > 1 && q_stride[i] >= (1ll << 39)) return SANTA_ERR_INVALID_ARG;
    const double k2 = (shape->scale != 0.f ? (double)shape->scale : 1.0 / std::sqrt((double)shape->d)) * 1.4426950408889634;
    if (!std::isfinite((float)k2)) return SANTA_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < need) return SANTA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return SANTA_ERR_MISALIGNED;
    if (T == 0) return SANTA_OK;
    AttendParams p{};
    p.v = static_cast<const uint16_t *>(cache->v);
    p.table = cache->table;
    p.pos = pos, p.counts = counts;
    p.out = static_cast<uint16_t *>(out);
    const int D = shape->d, G = shape->H_q / shape->H_kv, NQ = at_nq((long long)T * G);
    p.B = shape->B, p.T = T, p.H_q = shape->H_q, p.H_kv = shape->H_kv, p.lg_g = log2_of(G);
    p.n_max = shape->n_max;
    p.cols = shape->n_max / cache->page;
    p.n_pages = cache->n_pages;
    p.page_shift = log2_of(cache->page);
    p.window = std::min(window, shape->n_max);  // (larger ones see no more; no sum below overflows)
    p.sinks = p.window > 0 ? std::min(sinks, shape->n_max) : 0;
    p.piece_rows = at_piece_rows((long long)T * G);
    p.k2 = (float)k2;
    p.wait_ns = wait_limit_ns();
    p.wide = aligned(out, 32);
    p.clear = clear;
    // (a try that may sleep would outlast a limit below a millisecond; one that may not still takes some
    // microseconds, so with limits below a microsecond, which only make the waits run out, none is tried)
    p.tries = p.wait_ns < 1000 ? 0 : p.wait_ns < 1000000 ? 1 : 64;
    p.nap = p.wait_ns < 1000000 ? 0 : 10000000;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.ctrl = reinterpret_cast<int32_t *>(ws);
    p.part = reinterpret_cast<float *>(ws + CTRL_BYTES);
    p.part_ml = p.part + (size_t)AT_MAX_CTAS * 2 * p.piece_rows * D;

    int dev, sms, optin, occ = 0;
    if ((rc = device_info(&dev, &sms, &optin))) return rc;
    // no more shares than the longest sequences would give
    const long long qts = ((long long)T * G + NQ * AT_ROWS - 1) / (NQ * AT_ROWS);
    const long long most = p.window > 0 ? std::min<long long>(p.n_max, (long long)p.window + p.sinks + (NQ * AT_ROWS) / G) : p.n_max;
    const long long units = (most + AT_KEYS - 1) / AT_KEYS + 2 + AT_SETUP;
    const long long all = units * shape->B * shape->H_kv * qts;
    const long long grid = std::min<long long>(std::min(sms, AT_MAX_CTAS), (all + AT_MIN_SHARE - 1) / AT_MIN_SHARE);
    // tiles of an item in a share, at the most (a window may begin and end inside one)
    const long long tiles = (most + AT_KEYS - 1) / AT_KEYS + (p.window > 0 ? 2 : 0);
    const bool chains = std::min(tiles, all / grid + 1) > AT_CHAIN;
    const void *fn = D == 128 ? attend_kernel<128>(NQ, chains) : attend_kernel<64>(NQ, chains);
    const int smem = at_smem(D, NQ);
    if (smem > optin) return SANTA_ERR_UNSUPPORTED;
    if ((rc = prepare_fn(fn, dev, smem, at_threads(NQ), &occ))) return rc;
    CUtensorMap tm_q, tm_k, tm_v;
    const long long rows = (long long)cache->n_pages * shape->H_kv * cache->page;
    const int box = std::min<int>(cache->page, AT_KEYS);
    if ((rc = make_map_rows(&tm_q, q, D, shape->H_q, T, shape->B, q_stride, G, AT_ROWS / G)) ||
        (rc = make_map_bf16(&tm_k, cache->k, D, rows, box)) || (rc = make_map_bf16(&tm_v, cache->v, D, rows, box)))
        return rc;
    void *args[] = {&p, &tm_q, &tm_k, &tm_v};
    return cudaLaunchKernel(fn, dim3((unsigned)grid), dim3((unsigned)at_threads(NQ)), args, (size_t)smem, (cudaStream_t)stream) ==
                   cudaSuccess
               ? SANTA_OK
               : SANTA_ERR_CUDA;
}

}  // extern "C"

// santa_window_api.cu -- the entry points of the 4-bit KV cache and of windowed decode
// attention (declared in include/santa.h): argument checks and launches.
#include <algorithm>
#include <cmath>
#include <utility>

#include "../../include/santa.h"
#include "santa_host.h"
#include "santa_window.cuh"

using namespace santa;

namespace {

int check_cache(const santa_shape *sh, const santa_kv4 *c)
{
    const int rc = check_shape(sh);
    if (rc) return rc;
    if (!c || !c->k || !c->k_scale || !c->v || !c->v_scale) return SANTA_ERR_INVALID_ARG;
    if (sh->n_max % KV_GROUP != 0) return SANTA_ERR_UNSUPPORTED;
    if (!aligned(c->k, 16) || !aligned(c->k_scale, 16) || !aligned(c->v, 16) || !aligned(c->v_scale, 16))
        return SANTA_ERR_MISALIGNED;
    return SANTA_OK;
}

const void *move_kernel(int D, bool read, bool wide)
{
    switch ((D == 128) * 4 + read * 2 + wide) {
    case 0: return (const void *)santa_kv4_append_kernel<64, false>;
    case 1: return (const void *)santa_kv4_append_kernel<64, true>;
    case 2: return (const void *)santa_kv4_read_kernel<64, false>;
    case 3: return (const void *)santa_kv4_read_kernel<64, true>;
    case 4: return (const void *)santa_kv4_append_kernel<128, false>;
    case 5: return (const void *)santa_kv4_append_kernel<128, true>;
    case 6: return (const void *)santa_kv4_read_kernel<128, false>;
    default: return (const void *)santa_kv4_read_kernel<128, true>;
    }
}

// The checks and the launch shared by append and read.  `distinct`: the rows are written, so
// no two may share memory.
int move_rows(const santa_shape *sh, const santa_kv4 *c, const santa_rows *r, int32_t T, const int32_t *pos,
              const int32_t *counts, void *workspace, void *stream, bool distinct)
{
    int rc = check_cache(sh, c);
    if (rc || (rc = check_groups(sh))) return rc;
    if (!r || !r->k || !r->v || !pos || T < 0) return SANTA_ERR_INVALID_ARG;
    if (!aligned(r->k, 16) || !aligned(r->v, 16) || !aligned(pos, 4) || (counts && !aligned(counts, 4)) ||
        (workspace && !aligned(workspace, 256)))
        return SANTA_ERR_MISALIGNED;
    const long long groups = (long long)sh->B * sh->H_kv * (sh->d / KV_GROUP);
    if (T > 0 && groups > ((1ll << 31) - 1) / T) return SANTA_ERR_UNSUPPORTED;
    const long long dims[3] = {sh->B, T, sh->H_kv};
    for (int w = 0; w < 2; ++w) {
        const int64_t *st = w ? r->v_stride : r->k_stride;
        int order[3] = {0, 1, 2};
        for (int i = 0; i < 3; ++i) {
            if (dims[i] <= 1) continue;  // this stride is never used
            if (st[i] < 0 || st[i] > (1ll << 40)) return SANTA_ERR_INVALID_ARG;
            if (st[i] % 8 != 0) return SANTA_ERR_MISALIGNED;
        }
        if (!distinct) continue;
        // from the innermost dimension out, each step clears everything inside it
        for (int i = 1; i < 3; ++i)
            for (int j = i; j > 0 && st[order[j]] < st[order[j - 1]]; --j) std::swap(order[j], order[j - 1]);
        long long extent = sh->d;
        for (int i = 0; i < 3; ++i) {
            const int x = order[i];
            if (dims[x] <= 1) continue;
            if (st[x] < extent) return SANTA_ERR_INVALID_ARG;
            if (dims[x] - 1 > ((1ll << 60) - extent) / st[x]) return SANTA_ERR_INVALID_ARG;  // no memory is that large
            extent += st[x] * (dims[x] - 1);
        }
    }
    if (T == 0) return SANTA_OK;
    Kv4Move m{};
    m.code[0] = static_cast<uint8_t *>(c->k);
    m.code[1] = static_cast<uint8_t *>(c->v);
    m.scale[0] = static_cast<uint8_t *>(c->k_scale);
    m.scale[1] = static_cast<uint8_t *>(c->v_scale);
    m.row[0] = static_cast<uint16_t *>(r->k);
    m.row[1] = static_cast<uint16_t *>(r->v);
    for (int w = 0; w < 2; ++w) {
        const int64_t *s = w ? r->v_stride : r->k_stride;
        m.sb[w] = s[0];
        m.st[w] = s[1];
        m.sh[w] = s[2];
    }
    m.pos = pos;
    m.counts = counts;
    m.ctrl = static_cast<int32_t *>(workspace);
    m.H_kv = sh->H_kv;
    m.n_max = sh->n_max;
    m.T = T;
    // 32-byte accesses where every row begins at one
    bool wide = aligned(r->k, 32) && aligned(r->v, 32);
    for (int i = 0; i < 3; ++i)
        if (dims[i] > 1) wide = wide && r->k_stride[i] % 16 == 0 && r->v_stride[i] % 16 == 0;
    const long long row_groups = (long long)T * (sh->d / KV_GROUP);
    const long long threads = std::min<long long>(KV_NT, (row_groups + 31) / 32 * 32);
    const dim3 grid((unsigned)((row_groups + threads - 1) / threads), (unsigned)(sh->B * sh->H_kv));
    void *args[] = {&m};
    const void *fn = move_kernel(sh->d, distinct, wide);
    return cudaLaunchKernel(fn, grid, dim3((unsigned)threads), args, 0, (cudaStream_t)stream) == cudaSuccess ? SANTA_OK : SANTA_ERR_CUDA;
}

int check_window(const santa_shape *sh, const void *q, const int32_t *seq_lens, int32_t window, int32_t sinks,
                 int32_t flags, const float *out, const void *workspace, size_t workspace_bytes)
{
    if (!q || !seq_lens || !out || window < 0 || sinks < 0 || (flags & ~SANTA_OUT_BF16)) return SANTA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(seq_lens, 4)) return SANTA_ERR_MISALIGNED;
    size_t need = 0;
    const int rc = santa_window_workspace_size(sh, &need);
    if (rc) return rc;
    if (!workspace || workspace_bytes < need) return SANTA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return SANTA_ERR_MISALIGNED;
    return SANTA_OK;
}

// CTAs that can hold a share of the shape's list of tiles (of either cache): the workspace
// has pieces for as many.
long long window_ctas(const santa_shape *sh)
{
    const long long spans = (long long)sh->B * sh->H_kv * ((sh->n_max + 15) / 16 + WN_SETUP);
    const int w = std::min(win_warps(false), win_warps(true));
    return std::min<long long>(WN_MAX_CTAS, std::max<long long>((spans + w - 1) / w, (long long)sh->B * sh->H_kv));
}

const void *window_kernel(int D, bool kv4, bool wide)
{
    switch ((D == 128) * 4 + kv4 * 2 + wide) {
    case 0: return (const void *)santa_window_bf16_kernel<64, false>;
    case 1: return (const void *)santa_window_bf16_kernel<64, true>;
    case 2: return (const void *)santa_window_kv4_kernel<64, false>;
    case 3: return (const void *)santa_window_kv4_kernel<64, true>;
    case 4: return (const void *)santa_window_bf16_kernel<128, false>;
    case 5: return (const void *)santa_window_bf16_kernel<128, true>;
    case 6: return (const void *)santa_window_kv4_kernel<128, false>;
    default: return (const void *)santa_window_kv4_kernel<128, true>;
    }
}

// bf16: k and v are the caches.  4-bit: p.k, p.ks, p.v and p.vs are set.
int launch_window(const santa_shape *sh, WinParams &p, const void *k, const void *v, int32_t flags, void *workspace,
                  void *stream)
{
    const bool kv4 = k == nullptr;
    const int D = sh->d, G = sh->H_q / sh->H_kv;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const long long cap = window_ctas(sh);
    p.ctrl = reinterpret_cast<int32_t *>(ws);
    p.first = reinterpret_cast<float *>(ws + CTRL_BYTES);
    p.part = p.first + (size_t)cap * win_warps(kv4) * win_piece(G, D);
    p.B = sh->B;
    p.H_q = sh->H_q;
    p.H_kv = sh->H_kv;
    p.n_max = sh->n_max;
    p.G = G;
    p.window = std::min(p.window, sh->n_max);  // (larger ones see no more; no sum below overflows)
    p.sinks = std::min(p.sinks, sh->n_max);
    p.out_bf16 = (flags & SANTA_OUT_BF16) ? 1 : 0;
    const float scale = sh->scale != 0.f ? sh->scale : (float)(1.0 / std::sqrt((double)D));
    p.k2 = (float)(std::fabs((double)scale) * 1.4426950408889634);
    p.qsign = scale < 0.f ? -1.f : 1.f;
    p.wait_ns = wait_limit_ns();

    int dev, sms, optin, rc;
    if ((rc = device_info(&dev, &sms, &optin))) return rc;
    const int smem = win_smem(D, kv4, sh->B).total;
    if (smem > optin) return SANTA_ERR_UNSUPPORTED;
    const void *fn = window_kernel(D, kv4, G > 4);
    int occ = 0;
    if ((rc = prepare_fn(fn, dev, smem, win_threads(kv4), &occ))) return rc;
    const int tile = win_tile(D, kv4);
    const int most = p.window > 0 ? (int)std::min<long long>(sh->n_max, (long long)p.window + p.sinks) : sh->n_max;
    // a group's visible keys touch at most two tiles more than they would fill
    const long long spans = (long long)sh->B * sh->H_kv * ((most + tile - 1) / tile + 2 + WN_SETUP);
    const long long want = std::max((spans + win_warps(kv4) - 1) / win_warps(kv4), (long long)sh->B * sh->H_kv);
    const long long grid = std::min(std::min<long long>(cap, (long long)sms * occ), want);
    CUtensorMap tm_k, tm_v;
    if (!kv4) {
        const long long rows = (long long)sh->B * sh->H_kv * sh->n_max;
        if ((rc = make_map_bf16(&tm_k, k, D, rows, tile))) return rc;
        if ((rc = make_map_bf16(&tm_v, v, D, rows, tile))) return rc;
    }
    void *args[] = {&p, &tm_k, &tm_v};
    if (cudaLaunchKernel(fn, dim3((unsigned)grid), dim3(win_threads(kv4)), args, (size_t)smem, (cudaStream_t)stream) != cudaSuccess)
        return SANTA_ERR_CUDA;
    return SANTA_OK;
}

}  // namespace

extern "C" {

int santa_kv4_append(const santa_shape *shape, const santa_kv4 *cache, const santa_rows *rows, int32_t T,
                     const int32_t *pos, const int32_t *counts, void *workspace, void *stream)
{
    return move_rows(shape, cache, rows, T, pos, counts, workspace, stream, false);
}

int santa_kv4_read(const santa_shape *shape, const santa_kv4 *cache, const santa_rows *rows, int32_t T,
                   const int32_t *pos, const int32_t *counts, void *workspace, void *stream)
{
    return move_rows(shape, cache, rows, T, pos, counts, workspace, stream, true);
}

int santa_window_workspace_size(const santa_shape *shape, size_t *bytes)
{
    int rc = check_shape(shape);
    if (rc || (rc = check_groups(shape))) return rc;
    if (!bytes) return SANTA_ERR_INVALID_ARG;
    const size_t piece = (size_t)win_piece(shape->H_q / shape->H_kv, shape->d) * sizeof(float);
    *bytes = align_up(CTRL_BYTES + (size_t)window_ctas(shape) * (WN_MAX_WARPS + 2) * piece, 256);
    return SANTA_OK;
}

int santa_decode_window(const santa_shape *shape, const void *q, const void *k_cache, const void *v_cache,
                        const int32_t *seq_lens, int32_t window, int32_t sinks, int32_t flags, float *out,
                        void *workspace, size_t workspace_bytes, void *stream)
{
    int rc = check_shape(shape);
    if (rc) return rc;
    if (!k_cache || !v_cache) return SANTA_ERR_INVALID_ARG;
    if ((rc = check_window(shape, q, seq_lens, window, sinks, flags, out, workspace, workspace_bytes))) return rc;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return SANTA_ERR_MISALIGNED;
    WinParams p{};
    p.q = static_cast<const uint16_t *>(q);
    p.seq_lens = seq_lens;
    p.window = window;
    p.sinks = sinks;
    p.out = out;
    return launch_window(shape, p, k_cache, v_cache, flags, workspace, stream);
}

int santa_decode_kv4(const santa_shape *shape, const void *q, const santa_kv4 *cache, const int32_t *seq_lens,
                     int32_t window, int32_t sinks, int32_t flags, float *out, void *workspace,
                     size_t workspace_bytes, void *stream)
{
    int rc = check_cache(shape, cache);
    if (rc) return rc;
    if ((rc = check_window(shape, q, seq_lens, window, sinks, flags, out, workspace, workspace_bytes))) return rc;
    WinParams p{};
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint8_t *>(cache->k);
    p.v = static_cast<const uint8_t *>(cache->v);
    p.ks = static_cast<const uint8_t *>(cache->k_scale);
    p.vs = static_cast<const uint8_t *>(cache->v_scale);
    p.seq_lens = seq_lens;
    p.window = window;
    p.sinks = sinks;
    p.out = out;
    return launch_window(shape, p, nullptr, nullptr, flags, workspace, stream);
}

}  // extern "C"

// santa_host.h -- internal: host helpers of santa_api.cu that the other entry points use.
#pragma once

#include <cuda.h>  // CUtensorMap

#include <cstddef>
#include <cstdint>

#include "../../include/santa.h"

namespace santa {

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// The current device, its SM count and its shared-memory limit per block.
int device_info(int *dev, int *sms, int *optin);

// Raise the kernel's dynamic shared-memory limit if needed; CTAs per SM in *occ.
int prepare_fn(const void *fn, int dev, int smem, int threads, int *occ);

// Limits on the shape, and on the number of (batch row, KV head) groups.
int check_shape(const santa_shape *sh);
int check_groups(const santa_shape *sh);

// The limit of the kernels' pipeline waits (santa_set_wait_limit).
uint64_t wait_limit_ns();

// Row-major bf16 matrix [rows][D] as a 2-D tensor map: boxes of 64 columns x box_rows rows.
int make_map_bf16(CUtensorMap *map, const void *base, int D, long long rows, int box_rows);

// bf16 rows [B][T][H][D] with strides in elements for (batch, token, head) as a 4-D tensor map:
// boxes of 64 columns x heads x tokens of one batch row.
int make_map_rows(CUtensorMap *map, const void *base, int D, int H, int T, int B, const int64_t stride[3], int heads, int tokens);

}  // namespace santa

// The sums of rows of shares, for kernels of 256 threads.
#pragma once

#include "elem.h"
#include "neural.h"

namespace gsmi {

// The sums of shares that workgroups left behind, a few thousand rows at most, in one launch: eight columns per
// workgroup and 128 rows at a time, so that a thread's loads (16 for 2048 rows) are in flight together.  The last
// four columns may be summed twice, in the same order, for a whole load.
constexpr int kShareCols = 8;
__device__ __forceinline__ void sum_shares(const ShareSum& s, int32_t block, f32x4* lds) {
    const int x = threadIdx.x & 1, y = threadIdx.x >> 1;
    const int32_t c0 = block * kShareCols + x * 4, c = c0 + 4 <= s.cols || s.cols < 4 ? c0 : s.cols - 4;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c + 4 <= s.cols) {
#pragma unroll 16
        for (int64_t r = y; r < s.rows; r += 128) v += load_elem4(s.in, GS_TYPE_F32, r * s.cols + c);
    } else {
        for (int64_t r = y; r < s.rows; r += 128)
            for (int k = 0; k < 4; k++)
                if (c + k < s.cols) v[k] += s.in[r * s.cols + c + k];
    }
#pragma unroll
    for (int m = 2; m < 64; m <<= 1)
#pragma unroll
        for (int k = 0; k < 4; k++) v[k] += __shfl_xor(v[k], m);
    if ((threadIdx.x & 63) < 2) lds[(threadIdx.x >> 6) * 2 + x] = v;
    __syncthreads();
    if (threadIdx.x >= 2) return;
    v = (lds[x] + lds[2 + x]) + (lds[4 + x] + lds[6 + x]);
    for (int k = 0; k < 4; k++)
        if (c + k < s.cols) s.out[c + k] = v[k];
}

}  // namespace gsmi

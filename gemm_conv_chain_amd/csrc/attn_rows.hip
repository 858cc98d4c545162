// attn_rows.hip -- instantiations of k_attn_rows (attn_rows.h) for new tokens in
// causal order or all seen, and the join of split results, k_attn_join, which
// every form of attention shares.
#include "attn_rows.h"

namespace fc {

// Joins the splits of a row by weights 2^(m - max m): WPR waves a row, a lane D /
// 64 of its elements, a wave every WPR-th split.  A split that saw no key has l =
// 0 and has written no o: what its place holds is loaded but not used.
template <class T, int WPR>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a, long rows)
{
    __shared__ float part[WPR > 1 ? WPR - 1 : 1][6][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, w = wave % WPR, D = a.s.d;
    for (long row0 = (long)blockIdx.x * (4 / WPR); row0 < rows; row0 += (long)gridDim.x * (4 / WPR)) {
        const bool live = row0 + wave / WPR < rows;
        const long row = live ? row0 + wave / WPR : rows - 1;
        const floatx4* ml = a.part_ml + row * a.nsplit;
        float m = kNegInf;
        for (int k = lane; k < a.nsplit; k += 64) m = fmaxf(m, ml[k][0]);
#pragma unroll
        for (int s = 32; s; s >>= 1) m = fmaxf(m, __shfl_xor(m, s));
        const float ms = m == kNegInf ? 0.0f : m;
        float l = 0.0f, le = 0.0f, o[4] = {0, 0, 0, 0};
        const float* p = a.part_o + row * a.nsplit * D + lane;
#pragma unroll 4
        for (int k = w; k < a.nsplit; k += WPR) {
            const floatx4 v = ml[k];
            const float f = __builtin_amdgcn_exp2f(v[0] - ms);
            const bool some = v[1] != 0.0f;
            l += some ? v[1] * f : 0.0f;
            le += some ? v[2] * f : 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i * 64 < D) {
                    const float y = p[(long)k * D + i * 64] * f;
                    o[i] += some ? y : 0.0f;
                }
        }
        if (WPR > 1) {   // in the waves' order, whatever their timing
            if (w > 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) part[w - 1][i][lane] = o[i];
                part[w - 1][4][lane] = l;
                part[w - 1][5][lane] = le;
            }
            __syncthreads();
            if (w == 0) {
#pragma unroll
                for (int j = 0; j < WPR - 1; ++j) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] += part[j][i][lane];
                    l += part[j][4][lane];
                    le += part[j][5][lane];
                }
            }
            __syncthreads();   // the shared memory is free again
        }
        if (!live || w > 0) continue;
        const float inv = l != 0.0f ? 1.0f / l : 0.0f;
        T* out = (T*)a.out + row * D;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i * 64 < D) out[i * 64 + lane] = (T)(o[i] * inv);
        if (a.lse && lane == 0) a.lse[row] = (m + __builtin_amdgcn_logf(le)) * (1.0f / kLog2e);
    }
}

hipError_t run_attn_rows(int dtype, const AttnArgs& a, hipStream_t st)
{
    return dtype == DT_F16 ? rows_by_d<half_t, false>(a, st) : rows_by_d<bf16_t, false>(a, st);
}

// Many splits come with few rows: the waves of a block share a row then.
template <class T>
static hipError_t launch_join(const AttnArgs& a, hipStream_t st)
{
    const long rows = a.s.tokens * a.s.hq;
    const long blocks = a.nsplit > 8 ? rows : (rows + 3) / 4;
    const dim3 grid((unsigned)(blocks < (1L << 20) ? blocks : 1L << 20));
    if (a.nsplit > 8) k_attn_join<T, 4><<<grid, dim3(256), 0, st>>>(a, rows);
    else k_attn_join<T, 1><<<grid, dim3(256), 0, st>>>(a, rows);
    return hipGetLastError();
}

hipError_t run_attn_join(int dtype, const AttnArgs& a, hipStream_t st)
{
    return dtype == DT_F16 ? launch_join<half_t>(a, st) : launch_join<bf16_t>(a, st);
}

}  // namespace fc

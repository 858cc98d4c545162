// rope.hip -- rotary positions on [tokens, heads, d], any strides.
//
// Pair i of the first rot elements turns by position * f_i: (a, b) -> mscale *
// (a cos - b sin, a sin + b cos); the inverse turns the other way, which for
// mscale = 1 undoes it and always is the gradient (a rotation's transpose).
//
// Bound by memory: 4 bytes an element move, against about 12 operations.  A
// thread holds one unit of 16 elements (two 16-byte vectors) of HPT heads of a
// token, so that the unit's 8 sines and cosines are computed once for HPT heads
// and 2 * HPT loads are in flight; it writes what it alone has read, so x and y
// may be the same.
#include "fc_launch.h"
#include "kv_common.h"

namespace fc {

template <class T, int HPT>
__global__ __launch_bounds__(256) void k_rope(const T* x, T* y, long xt, long xh, long yt,
                                              long yh, const int* __restrict__ positions, RopeArgs r, int heads,
                                              FastDiv units, FastDiv hblocks, float sign, unsigned total)
{
    const unsigned i = blockIdx.x * 256u + threadIdx.x;
    if (i >= total) return;
    const unsigned rest = units.div(i), u = i - rest * units.d;
    const unsigned t = hblocks.div(rest), hb = rest - t * hblocks.d;
    const Unit at = unit_of(u, r.rot, r.interleaved);
    const int h0 = hb * HPT;
    const T* px = x + (long)t * xt + (long)h0 * xh;
    T* py = y + (long)t * yt + (long)h0 * yh;
    turn_heads<T, HPT>(px, py, xh, yh, at, r, u, at.turned ? positions[t] : 0, sign, heads - h0);
}

template <class T, int HPT>
static hipError_t launch_rope(const void* x, void* y, long xt, long xh, long yt, long yh, const int* positions,
                              const RopeArgs& r, float sign, long tokens, int heads, int d, hipStream_t st)
{
    const int units = d / 16, hb = (heads + HPT - 1) / HPT;
    // tokens a launch: thread indices stay below 2^31
    const long step = 0x7fffff00L / ((long)units * hb);
    for (long t = 0; t < tokens; t += step) {
        const long n = tokens - t < step ? tokens - t : step;
        const unsigned total = (unsigned)(n * units * hb);
        k_rope<T, HPT><<<dim3((total + 255) / 256), dim3(256), 0, st>>>(
            (const T*)x + t * xt, (T*)y + t * yt, xt, xh, yt, yh, positions + t, r, heads, FastDiv::make(units),
            FastDiv::make(hb), sign, total);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t run_rope(int dtype, const void* x, void* y, long xt, long xh, long yt, long yh, const int* positions,
                    const RopeArgs& r, bool inverse, long tokens, int heads, int d, hipStream_t st)
{
    if (tokens == 0 || heads == 0) return hipSuccess;
    const float sign = inverse ? -1.0f : 1.0f;
    const bool four = heads >= 4 && tokens * heads * (d / 16) >= 4L * 256 * device_cu_count();
    if (dtype == DT_F16)
        return four ? launch_rope<half_t, 4>(x, y, xt, xh, yt, yh, positions, r, sign, tokens, heads, d, st)
                    : launch_rope<half_t, 1>(x, y, xt, xh, yt, yh, positions, r, sign, tokens, heads, d, st);
    return four ? launch_rope<bf16_t, 4>(x, y, xt, xh, yt, yh, positions, r, sign, tokens, heads, d, st)
                : launch_rope<bf16_t, 1>(x, y, xt, xh, yt, yh, positions, r, sign, tokens, heads, d, st);
}

}  // namespace fc

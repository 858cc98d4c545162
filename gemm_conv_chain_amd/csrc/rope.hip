// rope.hip -- rotary positions on [tokens, heads, d], any strides.
//
// Pair i of the first rot elements turns by position * f_i: (a, b) -> mscale *
// (a cos - b sin, a sin + b cos); the inverse turns the other way, which for
// mscale = 1 undoes it and always is the gradient (a rotation's transpose).
//
// Bound by memory: 4 bytes an element move, against about 12 operations.  A
// thread holds one unit of 16 elements (two 16-byte vectors, eight pairs) of a
// head and writes what it alone has read, so x and y may be the same.  Measured:
// 16385 x 40 x 128 in 58 us (5.8 TB/s read and written; a copy of as many bytes takes
// 61 to 63, both also with eight sets of buffers in turn); with four heads a thread,
// which share their angles, 63 us, and small calls 2.6 us against 3.3.
#include "fc_launch.h"
#include "kv_common.h"

namespace fc {

template <class T>
__global__ __launch_bounds__(256) void k_rope(const T* x, T* y, long xt, long xh, long yt, long yh,
                                              const int* __restrict__ positions, RopeArgs r, FastDiv units, FastDiv heads,
                                              float sign, unsigned total)
{
    const unsigned i = blockIdx.x * 256u + threadIdx.x;
    if (i >= total) return;
    const unsigned rest = units.div(i), u = i - rest * units.d;
    const unsigned t = heads.div(rest), h = rest - t * heads.d;
    const Unit at = unit_of(u, r.rot, r.interleaved);
    turn_heads<T, 1>(x + (long)t * xt + (long)h * xh, y + (long)t * yt + (long)h * yh, 0, 0, at, r, u,
                     at.turned ? positions[t] : 0, sign, 1);
}

template <class T>
static hipError_t launch_rope(const void* x, void* y, long xt, long xh, long yt, long yh, const int* positions,
                              const RopeArgs& r, float sign, long tokens, int heads, int d, hipStream_t st)
{
    const int units = d / 16;
    // tokens a launch: thread indices stay below 2^31
    const long step = 0x7fffff00L / ((long)units * heads);
    for (long t = 0; t < tokens; t += step) {
        const long n = tokens - t < step ? tokens - t : step;
        const unsigned total = (unsigned)(n * units * heads);
        k_rope<T><<<dim3((total + 255) / 256), dim3(256), 0, st>>>((const T*)x + t * xt, (T*)y + t * yt, xt, xh, yt, yh,
                                                                   positions + t, r, FastDiv::make(units),
                                                                   FastDiv::make(heads), sign, total);
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
    return dtype == DT_F16 ? launch_rope<half_t>(x, y, xt, xh, yt, yh, positions, r, sign, tokens, heads, d, st)
                           : launch_rope<bf16_t>(x, y, xt, xh, yt, yh, positions, r, sign, tokens, heads, d, st);
}

}  // namespace fc

// kv_append.hip -- appends keys and values to the paged 8-bit cache, the keys
// (and, in the same launch, the queries) rotated by their positions on the way.
//
// For each (page, kv head, side) that gets new tokens: the largest finite
// magnitude of the new values, in 32 bits after the rotation, gives the least
// power of two 2^e with amax <= 448 * 2^e; a page that keeps earlier tokens
// takes the larger of that and what it has, and where its scale grows its
// earlier codes are rounded again (by a power of two: exact but for the
// subnormal codes).  A code is the value over the scale, saturated to +-448 and
// rounded to nearest even: 4 bits of significand are the cache's choice.
//
// One block owns one (page, head), both sides, so that nothing is shared
// between blocks: no atomics, and results do not depend on any order.  Waves
// 0 .. WPS - 1 take K, the next WPS take V.
#include "fc_launch.h"
#include "kv_common.h"

namespace fc {

__device__ __forceinline__ float finite_abs(float x)
{
    const float a = fabsf(x);
    return a < __builtin_inff() ? a : 0.0f;   // false for NaN too
}

// amax <= 448 * 2^e, 448 = 1.75 * 2^8: from the exponent and whether the
// significand is over 1.75.
template <class T>
__device__ __forceinline__ int scale_exponent(float amax)
{
    const unsigned b = __builtin_bit_cast(unsigned, amax);
    const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e < Tr<T>::elo ? Tr<T>::elo : (e > Tr<T>::ehi ? Tr<T>::ehi : e);
}

__device__ __forceinline__ float pow2(int e) { return __builtin_bit_cast(float, (unsigned)(e + 127) << 23); }

__device__ __forceinline__ float sat(float x) { return fminf(fmaxf(x, -448.0f), 448.0f); }

// K: a NaN stays one.  V: a NaN becomes 0 (its token's key is marked instead).
template <bool KEY>
__device__ __forceinline__ float coded(float x, float inv)
{
    const float y = sat(x * inv);
    return x != x ? (KEY ? x : 0.0f) : y;
}

__device__ __forceinline__ unsigned pk4(float a, float b, float c, float d)
{
    return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false), true);
}

__device__ __forceinline__ unsigned recode4(unsigned w, float ratio)
{
    const floatx2 a = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
    return pk4(a[0] * ratio, a[1] * ratio, b[0] * ratio, b[1] * ratio);
}

struct AppendArgs {
    const void *k, *v, *q;
    void* q_out;
    long k_ts, k_hs, v_ts, v_hs, q_ts, q_hs;
    uint8_t* codes;
    float* scales;
    const int *table, *cu_q, *kv_lens, *positions;
    KvShape s;
    RopeArgs r;
    int nslots;       // blocks along x that append; those after them rotate q
    FastDiv units, qh;
};

template <class T, int WPS>
__device__ void append_page(const AppendArgs& a, int b, int h, int slot0, long tok0, int n, int start, int id)
{
    constexpr int NT = WPS * 64;
    const KvShape& s = a.s;
    const int side = threadIdx.x >= NT, tid = threadIdx.x - side * NT;
    // new tokens of this page: slots [lo, hi) of it
    const int lo = start > slot0 ? start - slot0 : 0;
    const int hi = start + n - slot0 < s.page ? start + n - slot0 : s.page;
    const int nt = hi - lo, units = s.d / 16;
    const long row0 = tok0 + (slot0 + lo - start);
    uint8_t* base = a.codes + side_base(id, h, side, s);
    float* scale = a.scales + ((size_t)id * s.hkv + h) * 2 + side;
    const T* kp = (const T*)a.k + (long)h * a.k_hs;
    const T* vp = (const T*)a.v + (long)h * a.v_hs;

    __shared__ float red[2][WPS];
    __shared__ unsigned bad[8];   // tokens whose value holds a NaN, a bit each
    if (threadIdx.x < 8) bad[threadIdx.x] = 0;
    __syncthreads();

    auto key_unit = [&](int i, float (&x0)[8], float (&x1)[8], Unit& at, int& t) {
        t = a.units.div(i);
        const int u = i - t * units;
        at = unit_of(u, a.r.rot, a.r.interleaved);
        const T* p = kp + (row0 + t) * a.k_ts;
        load8(p + at.e0, x0);
        load8(p + at.e1, x1);
        if (at.turned) {
            float cs[8], sn[8];
            const int pos = a.positions ? a.positions[row0 + t] : slot0 + lo + t;
            unit_angles(a.r.turns, u, pos, a.r.mscale, 1.0f, cs, sn);
            rotate_unit(x0, x1, cs, sn, a.r.interleaved);
        }
    };

    float amax = 0.0f;
    if (side == 0) {
        for (int i = tid; i < nt * units; i += NT) {
            float x0[8], x1[8];
            Unit at;
            int t;
            key_unit(i, x0, x1, at, t);
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fmaxf(finite_abs(x0[j]), finite_abs(x1[j])));
        }
    } else {
        for (int i = tid; i < nt * units; i += NT) {
            const int t = a.units.div(i), u = i - t * units;
            float x0[8], x1[8];
            const T* p = vp + (row0 + t) * a.v_ts + u * 16;
            load8(p, x0);
            load8(p + 8, x1);
            bool nan = false;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                amax = fmaxf(amax, fmaxf(finite_abs(x0[j]), finite_abs(x1[j])));
                nan |= x0[j] != x0[j] || x1[j] != x1[j];
            }
            if (nan) atomicOr(&bad[(lo + t) >> 5], 1u << ((lo + t) & 31));
        }
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
    if ((tid & 63) == 0) red[side][tid >> 6] = amax;
    const float held = lo > 0 ? *scale : 0.0f;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WPS; ++w) amax = fmaxf(amax, red[side][w]);
    int e = scale_exponent<T>(amax);
    if (lo > 0) {
        // the held scale is a power of two; anything else (a pool never written)
        // is taken by its exponent, inside the type's range
        int eh = (int)((__builtin_bit_cast(unsigned, held) >> 23) & 255) - 127;
        eh = eh < Tr<T>::elo ? Tr<T>::elo : (eh > Tr<T>::ehi ? Tr<T>::ehi : eh);
        if (eh < e) {   // earlier codes: 16 bytes at a time
            const float ratio = pow2(eh - e < -126 ? -126 : eh - e);
            if (side == 0) {
                for (int i = tid; i < lo * units; i += NT) {
                    const int t = a.units.div(i), u = i - t * units;
                    u32x4* p = reinterpret_cast<u32x4*>(base + (t >> 4) * 16 * s.d + u * 256 + (t & 15) * 16);
                    u32x4 w = *p;
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = recode4(w[j], ratio);
                    *p = w;
                }
            } else {
                const int nb = (lo + 15) >> 4;
                for (int i = tid; i < nb * s.d; i += NT) {
                    const int blk = i / s.d;
                    const int keep = lo - blk * 16;   // tokens of the block that stay
                    u32x4* p = reinterpret_cast<u32x4*>(base + (size_t)i * 16);
                    u32x4 w = *p;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int k = keep - 4 * j;
                        const unsigned m = k >= 4 ? ~0u : (k <= 0 ? 0u : (1u << (8 * k)) - 1u);
                        w[j] = (recode4(w[j], ratio) & m) | (w[j] & ~m);
                    }
                    *p = w;
                }
            }
        }
        e = eh > e ? eh : e;
    }
    __syncthreads();   // the earlier codes' vectors are written before the new tokens' bytes in them
    const float inv = pow2(-e);
    if (tid == 0) *scale = pow2(e);
    if (side == 0) {
        for (int i = tid; i < nt * units; i += NT) {
            float x0[8], x1[8];
            Unit at;
            int t;
            key_unit(i, x0, x1, at, t);
            t += lo;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x0[j] = coded<true>(x0[j], inv);
                x1[j] = coded<true>(x1[j], inv);
            }
            if (at.e0 == 0 && (bad[t >> 5] >> (t & 31) & 1)) x0[0] = __builtin_nanf("");
            uint8_t* p = base + (t >> 4) * 16 * s.d + (t & 15) * 16;
            u32x2 w;
            w[0] = pk4(x0[0], x0[1], x0[2], x0[3]);
            w[1] = pk4(x0[4], x0[5], x0[6], x0[7]);
            *reinterpret_cast<u32x2*>(p + (at.e0 >> 4) * 256 + (at.e0 & 15)) = w;
            w[0] = pk4(x1[0], x1[1], x1[2], x1[3]);
            w[1] = pk4(x1[4], x1[5], x1[6], x1[7]);
            *reinterpret_cast<u32x2*>(p + (at.e1 >> 4) * 256 + (at.e1 & 15)) = w;
        }
    } else {
        // whole blocks of 16 tokens: 8 dims a thread, transposed in registers
        const int d8 = s.d / 8, b0 = (lo + 15) >> 4, b1 = hi >> 4;
        for (int i = tid; i < (b1 - b0) * d8; i += NT) {
            const int blk = b0 + i / d8, g = i % d8;
            const T* p = vp + (row0 + blk * 16 - lo) * a.v_ts + g * 8;
            u32x4 w[8];
#pragma unroll
            for (int t4 = 0; t4 < 4; ++t4) {
                float x[4][8];
#pragma unroll
                for (int k = 0; k < 4; ++k) load8(p + (t4 * 4 + k) * a.v_ts, x[k]);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    w[j][t4] = pk4(coded<false>(x[0][j], inv), coded<false>(x[1][j], inv), coded<false>(x[2][j], inv),
                                   coded<false>(x[3][j], inv));
            }
            u32x4* o = reinterpret_cast<u32x4*>(base + (size_t)(blk * s.d + g * 8) * 16);
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = w[j];
        }
        // tokens of blocks at the ends: single bytes
        for (int i = tid; i < nt * d8; i += NT) {
            const int t = lo + i / d8, g = i % d8;
            if ((t >> 4) >= b0 && (t >> 4) < b1) continue;
            float x[8];
            load8(vp + (row0 + t - lo) * a.v_ts + g * 8, x);
            uint8_t* o = base + (size_t)((t >> 4) * s.d + g * 8) * 16 + (t & 15);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float c = coded<false>(x[j], inv);
                o[j * 16] = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, c, 0, false);
            }
        }
    }
}

// grid (nslots + blocks of q, hkv, min(batch, 65535)).
template <class T, int WPS>
__global__ __launch_bounds__(128 * WPS) void k_kv_append(AppendArgs a)
{
    for (int b = blockIdx.z; b < a.s.batch; b += gridDim.z) {
        long tok0;
        int n;
        seq_range(a.cu_q, a.s, b, &tok0, &n);
        if (n == 0) continue;
        const int kv_len = a.kv_lens[b], start = kv_len - n;
        if ((int)blockIdx.x < a.nslots) {
            if (kv_len <= 0) continue;
            const int p0 = (start > 0 ? start : 0) / a.s.page;
            int p1 = (kv_len - 1) / a.s.page;
            p1 = p1 < a.s.table_stride ? p1 : a.s.table_stride - 1;
            for (int p = p0 + blockIdx.x; p <= p1; p += a.nslots) {
                const int id = page_id(a.table, a.s, b, p);
                if (id < 0) continue;
                __syncthreads();   // the block's shared memory is free again
                append_page<T, WPS>(a, b, blockIdx.y, p * a.s.page, tok0, n, start, id);
            }
        } else {
            const long nq = (long)(gridDim.x - a.nslots) * gridDim.y * 128 * WPS;
            const int units = a.s.d / 16;
            const long total = (long)n * a.s.hq * units;
            for (long i = ((long)(blockIdx.x - a.nslots) * gridDim.y + blockIdx.y) * 128 * WPS + threadIdx.x; i < total;
                 i += nq) {
                const long rest = i / units;
                const int u = (int)(i - rest * units);
                const long t = rest / a.s.hq;
                const int h = (int)(rest - t * a.s.hq);
                const Unit at = unit_of(u, a.r.rot, a.r.interleaved);
                const T* p = (const T*)a.q + (tok0 + t) * a.q_ts + (long)h * a.q_hs;
                float x0[8], x1[8];
                load8(p + at.e0, x0);
                load8(p + at.e1, x1);
                if (at.turned) {
                    float cs[8], sn[8];
                    const int pos = a.positions ? a.positions[tok0 + t] : start + (int)t;
                    unit_angles(a.r.turns, u, pos, a.r.mscale, 1.0f, cs, sn);
                    rotate_unit(x0, x1, cs, sn, a.r.interleaved);
                }
                T* o = (T*)a.q_out + ((tok0 + t) * a.s.hq + h) * (long)a.s.d;
                *reinterpret_cast<u32x4*>(o + at.e0) = pack8<T>(x0);
                *reinterpret_cast<u32x4*>(o + at.e1) = pack8<T>(x1);
            }
        }
    }
}

template <class T>
static hipError_t launch_append(AppendArgs a, hipStream_t st)
{
    const int mq = a.s.max_q > 0 ? a.s.max_q : 1;
    const bool shortq = mq <= 16;
    const int wps = shortq ? 1 : 2;
    a.nslots = mq == 1 ? 1 : (mq + a.s.page - 2) / a.s.page + 1;
    long qblocks = 0;
    if (a.q) {
        const long per = 128L * wps * a.s.hkv;
        qblocks = ((long)mq * a.s.hq * (a.s.d / 16) + per - 1) / per;
        if (qblocks > 65535) qblocks = 65535;
    }
    const dim3 grid((unsigned)(a.nslots + qblocks), a.s.hkv, a.s.batch < 65535 ? a.s.batch : 65535);
    if (shortq) k_kv_append<T, 1><<<grid, dim3(128), 0, st>>>(a);
    else k_kv_append<T, 2><<<grid, dim3(256), 0, st>>>(a);
    return hipGetLastError();
}

hipError_t run_kv_append(int dtype, const void* k, const void* v, const void* q, void* q_out, const long* strides,
                         uint8_t* codes, float* scales, const int* table, const int* cu_q, const int* kv_lens,
                         const int* positions, const KvShape& s, const RopeArgs& r, hipStream_t st)
{
    if (s.batch == 0 || s.tokens == 0) return hipSuccess;
    AppendArgs a{k,       v,       q,        q_out,    strides[0], strides[1], strides[2],
                 strides[3], strides[4], strides[5], codes,    scales,     table,      cu_q,
                 kv_lens, positions, s,        r,        0,          FastDiv::make(s.d / 16), FastDiv::make(s.hq)};
    return dtype == DT_F16 ? launch_append<half_t>(a, st) : launch_append<bf16_t>(a, st);
}

}  // namespace fc

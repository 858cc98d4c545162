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
// between blocks, and results do not depend on any order (the only atomics set
// bits of a mask in LDS).  Waves 0 .. WPS - 1 take K, the next WPS take V.
//
// Bound by memory for prompts: six of them, 20 k tokens, 32 query heads, 8 kv
// heads of 128: 499 MB in 112 us (4.4 TB/s; a copy of as many bytes takes 94).  A
// step's token is a chain of loads (lengths, page, values, scale): 8 us for 128
// sequences.
#include "fc_launch.h"
#include "kv_common.h"

namespace fc {

__device__ __forceinline__ float finite_abs(float x)
{
    const float a = fabsf(x);
    return a < __builtin_inff() ? a : 0.0f;   // false for NaN too
}

// Magnitudes of 16-bit values compare as integers: the larger of each half of m
// and of w, sign aside.
typedef unsigned short ushort2v __attribute__((ext_vector_type(2)));
__device__ __forceinline__ unsigned max_abs16(unsigned m, unsigned w)
{
    return __builtin_bit_cast(unsigned, __builtin_elementwise_max(__builtin_bit_cast(ushort2v, m),
                                                                  __builtin_bit_cast(ushort2v, w & 0x7fff7fffu)));
}
__device__ __forceinline__ unsigned max_half(unsigned m) { return (m & 0xffffu) > (m >> 16) ? m & 0xffffu : m >> 16; }

// Bits from which on a value is infinite or NaN.
template <class T> struct Odd {
    static constexpr unsigned value = Tr<T>::elo == Tr<half_t>::elo ? 0x7c00u : 0x7f80u;
};
template <class T> __device__ __forceinline__ float value16(unsigned bits)
{
    const unsigned short b = (unsigned short)bits;
    return (float)__builtin_bit_cast(T, b);
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
// plain: the caller has seen that there is none.
template <bool KEY>
__device__ __forceinline__ float coded(float x, float inv, bool plain)
{
    if (plain) return __builtin_amdgcn_fmed3f(x * inv, -448.0f, 448.0f);
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

// Maximum over a wave, in every lane: quads, eights and rows by DPP, rows by
// register swaps (no LDS).
__device__ __forceinline__ float wave_max(float v)
{
    auto dpp = [](float x, auto ctl) {
        return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), decltype(ctl)::value, 0xF, 0xF, true));
    };
    v = fmaxf(v, dpp(v, IntC<0xB1>{}));    // quad_perm [1,0,3,2]
    v = fmaxf(v, dpp(v, IntC<0x4E>{}));    // quad_perm [2,3,0,1]
    v = fmaxf(v, dpp(v, IntC<0x141>{}));   // row_half_mirror
    v = fmaxf(v, dpp(v, IntC<0x140>{}));   // row_mirror
    return max_x32(max_x16(v));
}

// In every quad: a[r] at quad lane j -> a[j] at quad lane r.
__device__ __forceinline__ void quad_transpose_dw(unsigned (&a)[4], int lane)
{
    const bool b1 = (lane >> 1) & 1, b0 = lane & 1;
    unsigned y[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const unsigned other = dpp_quad_xor2(a[r ^ 2]);
        y[r] = b1 == (bool)((r >> 1) & 1) ? a[r] : other;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const unsigned other = dpp_quad_xor1(y[r ^ 1]);
        a[r] = b0 == (bool)(r & 1) ? y[r] : other;
    }
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
    int nslots, qblocks;   // blocks along x that append, and after them that turn q
    int lds_floats;        // of the block's LDS for turned keys
    FastDiv units, d8, dpair, qwork;   // d / 16, d / 8, d / 2; threads a token of q takes
};

// Values are looked at twice, for the amax and for the codes.  The turned keys
// wait in LDS in between (each thread's own, 16 floats a unit; a page of more
// than 15360 values is turned twice), the values are read again, from the caches.
// Holding both in registers took 300 a thread and, for six prompts, 303 us.
//
// The first look takes the amax of 16-bit values as integers and tells whether
// any is infinite or NaN; only a page that has one takes the careful forms.
template <class T, int WPS>
__device__ __forceinline__ void append_page(const AppendArgs& a, int b, int h, int slot0, long tok0, int n, int start)
{
    constexpr int NT = WPS * 64;
    const KvShape& s = a.s;
    const int side = threadIdx.x >= NT, tid = threadIdx.x - side * NT;
    // new tokens of this page: slots [lo, hi) of it
    const int lo = start > slot0 ? start - slot0 : 0;
    const int hi = start + n - slot0 < s.page ? start + n - slot0 : s.page;
    const int nt = hi - lo, units = s.d / 16, d8 = s.d / 8;
    const long row0 = tok0 + (slot0 + lo - start);
    const int id = page_id(a.table, s, b, slot0 / s.page);   // (not waited for before the values are here)
    const T* kp = (const T*)a.k + (long)h * a.k_hs;
    const T* vp = (const T*)a.v + (long)h * a.v_hs;

    extern __shared__ __align__(16) float turned[];
    __shared__ float red[2][WPS];
    __shared__ int rares[2][WPS];
    __shared__ unsigned bad[8];   // tokens whose value holds a NaN, a bit each
    if (threadIdx.x < 8) bad[threadIdx.x] = 0;

    // K, unit i: 16 elements (unit_of) of token t
    auto key_unit = [&](int i, float (&x)[16], unsigned& top) {
        const int t = a.units.div(i), u = i - t * units;
        const Unit at = unit_of(u, a.r.rot, a.r.interleaved);
        const T* p = kp + (row0 + t) * a.k_ts;
        const u32x4 w0 = *reinterpret_cast<const u32x4*>(p + at.e0), w1 = *reinterpret_cast<const u32x4*>(p + at.e1);
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max_abs16(max_abs16(top, w0[j]), w1[j]);
        float x0[8], x1[8];
        unpack8<T>(w0, x0);
        unpack8<T>(w1, x1);
        if (at.turned) {
            float cs[8], sn[8];
            const int pos = a.positions ? a.positions[row0 + t] : slot0 + lo + t;
            unit_angles(a.r.turns, u, pos, a.r.mscale, 1.0f, cs, sn);
            rotate_unit(x0, x1, cs, sn, a.r.interleaved);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = x0[j];
            x[8 + j] = x1[j];
        }
    };
    // V, task i of whole blocks b0 .. b1 - 1: 4 tokens (quad lane) of 8 dims
    const int b0 = (lo + 15) >> 4, b1 = hi >> 4;
    const int nwhole = b1 > b0 ? (b1 - b0) * 4 * d8 : 0;
    auto value_task = [&](int i, u32x4 (&w)[4], int& blk, int& g) {
        blk = b0 + a.d8.div(i >> 2);
        g = (i >> 2) - (blk - b0) * d8;
        const T* p = vp + (row0 + blk * 16 + (i & 3) * 4 - lo) * a.v_ts + g * 8;
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = *reinterpret_cast<const u32x4*>(p + k * a.v_ts);
    };
    // tokens of blocks at the ends: two dims a task
    const int head = nwhole ? b0 * 16 - lo : nt, ends = nwhole ? nt - (b1 - b0) * 16 : nt, dp = s.d / 2;
    auto end_task = [&](int i, int& t, int& d) {
        const int k = a.dpair.div(i);
        d = 2 * (i - k * dp);
        t = k < head ? k : k - head + (b1 * 16 - lo);
        const unsigned w = *reinterpret_cast<const unsigned*>(vp + (row0 + t) * a.v_ts + d);
        return w;
    };
    auto pair_of = [&](unsigned w, float& x, float& y) {
        if (sizeof(T) == 2 && Tr<T>::elo == Tr<half_t>::elo) {
            const half2v v = __builtin_bit_cast(half2v, w);
            x = (float)v[0];
            y = (float)v[1];
        } else {
            const bf2 v = __builtin_bit_cast(bf2, w);
            x = (float)v[0];
            y = (float)v[1];
        }
    };

    u32x4 v0[4] = {};   // the thread's first task of V
    const int nu = nt * units;
    const bool kept = nu * 16 <= a.lds_floats;
    float amax = 0.0f;
    bool rare = false;
    if (side == 0) {
        unsigned top = 0;
        for (int i = tid; i < nu; i += NT) {
            float y[16];
            key_unit(i, y, top);
#pragma unroll
            for (int j = 0; j < 16; ++j) amax = fmaxf(amax, fabsf(y[j]));
            if (kept) {
#pragma unroll
                for (int j = 0; j < 16; j += 4)
                    *reinterpret_cast<FC_LDS floatx4*>((FC_LDS float*)turned + (j * nu + i * 4)) =
                        floatx4{y[j], y[j + 1], y[j + 2], y[j + 3]};
            }
        }
        // (finite keys may leave 32 bits as they turn: one of the pair is infinite then, the other may be
        // NaN, which amax passes over)
        rare = max_half(top) >= Odd<T>::value || !(amax < __builtin_inff());
    } else {
        unsigned all = 0;
        for (int i = tid; i < nwhole; i += NT) {
            u32x4 w[4];
            int blk, g;
            value_task(i, w, blk, g);
            if (i == tid) {
#pragma unroll
                for (int k = 0; k < 4; ++k) v0[k] = w[k];
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                unsigned top = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) top = max_abs16(top, w[k][j]);
                all = max_abs16(all, top);
            }
        }
        for (int i = tid; i < ends * dp; i += NT) {
            int t, d;
            const unsigned top = end_task(i, t, d) & 0x7fff7fffu;
            all = max_abs16(all, top);
        }
        rare = max_half(all) >= Odd<T>::value;
        amax = rare ? 0.0f : value16<T>(max_half(all));
    }
    amax = wave_max(amax);
    const int any_rare = __any(rare);
    if ((tid & 63) == 0) {
        red[side][tid >> 6] = amax;
        rares[side][tid >> 6] = any_rare;
    }
    __syncthreads();
    int odd = 0;
#pragma unroll
    for (int w = 0; w < WPS; ++w) odd |= rares[0][w] | rares[1][w];
    if (id < 0) return;   // a page outside the pool: its tokens are not written
    uint8_t* base = a.codes + side_base(id, h, side, s);
    float* scale = a.scales + ((size_t)id * s.hkv + h) * 2 + side;
    const float held = lo > 0 ? *scale : 0.0f;
    if (odd) {   // the amax is over finite values; tokens whose value holds a NaN are noted
        amax = 0.0f;
        if (side == 0) {
            for (int i = tid; i < nu; i += NT) {
                float y[16];
                unsigned top = 0;
                key_unit(i, y, top);
#pragma unroll
                for (int j = 0; j < 16; ++j) amax = fmaxf(amax, finite_abs(y[j]));
            }
        } else {
            for (int i = tid; i < nt * d8; i += NT) {
                const int t = a.d8.div(i);
                float y[8];
                load8(vp + (row0 + t) * a.v_ts + (i - t * d8) * 8, y);
                bool nan = false;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    amax = fmaxf(amax, finite_abs(y[j]));
                    nan |= y[j] != y[j];
                }
                if (nan) atomicOr(&bad[(lo + t) >> 5], 1u << ((lo + t) & 31));
            }
        }
        amax = wave_max(amax);
        if ((tid & 63) == 0) red[side][tid >> 6] = amax;
        __syncthreads();
    }
    const bool plain = odd == 0;
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
                    const int blk = a.d8.div(i >> 3);
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
        __syncthreads();   // the earlier codes' vectors are written before the new tokens' bytes in them
    }
    const float inv = pow2(-e);
    if (tid == 0) *scale = pow2(e);
    if (side == 0) {
        for (int i = tid; i < nu; i += NT) {
            const int u0 = a.units.div(i);
            const Unit at = unit_of(i - u0 * units, a.r.rot, a.r.interleaved);
            const int t = u0 + lo;
            float y[16], z[16];
            if (kept) {
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const floatx4 v = *reinterpret_cast<const FC_LDS floatx4*>((FC_LDS float*)turned + (j * nu + i * 4));
#pragma unroll
                    for (int k = 0; k < 4; ++k) y[j + k] = v[k];
                }
            } else {
                unsigned top = 0;
                key_unit(i, y, top);
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) z[j] = coded<true>(y[j], inv, plain);
            if (!plain && at.e0 == 0 && (bad[t >> 5] >> (t & 31) & 1)) z[0] = __builtin_nanf("");
            uint8_t* p = base + (t >> 4) * 16 * s.d + (t & 15) * 16;
            u32x2 w;
            w[0] = pk4(z[0], z[1], z[2], z[3]);
            w[1] = pk4(z[4], z[5], z[6], z[7]);
            *reinterpret_cast<u32x2*>(p + (at.e0 >> 4) * 256 + (at.e0 & 15)) = w;
            w[0] = pk4(z[8], z[9], z[10], z[11]);
            w[1] = pk4(z[12], z[13], z[14], z[15]);
            *reinterpret_cast<u32x2*>(p + (at.e1 >> 4) * 256 + (at.e1 & 15)) = w;
        }
    } else {
        // a quad has a block's 16 tokens of 8 dims: transposed among its lanes to 16 bytes of a dim
        for (int i = tid; i < nwhole; i += NT) {   // (nwhole is a multiple of 4: whole quads)
            u32x4 v[4];
            int blk, g;
            if (i == tid) {
                const int r = a.d8.div(i >> 2);
                blk = b0 + r;
                g = (i >> 2) - r * d8;
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = v0[k];
            } else {
                value_task(i, v, blk, g);
            }
            float y[4][8];
#pragma unroll
            for (int k = 0; k < 4; ++k) unpack8<T>(v[k], y[k]);
#pragma unroll
            for (int j4 = 0; j4 < 8; j4 += 4) {
                unsigned w[4];
#pragma unroll
                for (int j = j4; j < j4 + 4; ++j)
                    w[j - j4] = pk4(coded<false>(y[0][j], inv, plain), coded<false>(y[1][j], inv, plain),
                                    coded<false>(y[2][j], inv, plain), coded<false>(y[3][j], inv, plain));
                quad_transpose_dw(w, i & 3);
                *reinterpret_cast<u32x4*>(base + (size_t)(blk * s.d + g * 8 + j4 + (i & 3)) * 16) =
                    u32x4{w[0], w[1], w[2], w[3]};
            }
        }
        for (int i = tid; i < ends * dp; i += NT) {
            int t, d;
            float y0, y1;
            pair_of(end_task(i, t, d), y0, y1);
            t += lo;
            const unsigned c = __builtin_amdgcn_cvt_pk_fp8_f32(coded<false>(y0, inv, plain), coded<false>(y1, inv, plain), 0, false);
            uint8_t* o = base + (size_t)((t >> 4) * s.d + d) * 16 + (t & 15);
            o[0] = (uint8_t)c;
            o[16] = (uint8_t)(c >> 8);
        }
    }
}

// Block i of `blocks` turns its share of sequence b's queries.  A thread holds
// one unit of HPT heads of a token, which share its angles.
template <class T, int HPT>
__device__ __forceinline__ void turn_queries(const AppendArgs& a, long tok0, int n, int start, unsigned i, unsigned blocks,
                                             unsigned threads)
{
    const unsigned per = a.qwork.d, id = i * threads + threadIdx.x;
    const int units = a.s.d / 16, step = blocks * threads / per;
    const int t0 = a.qwork.div(id), w = id - t0 * per;
    const int hb = a.units.div(w), u = w - hb * units, h0 = hb * HPT;
    if (t0 >= step) return;
    const Unit at = unit_of(u, a.r.rot, a.r.interleaved);
#pragma unroll 1
    for (int t = t0; t < n; t += step) {
        const T* p = (const T*)a.q + (tok0 + t) * a.q_ts + (long)h0 * a.q_hs;
        T* o = (T*)a.q_out + ((tok0 + t) * a.s.hq + h0) * (long)a.s.d;
        turn_heads<T, HPT>(p, o, a.q_hs, a.s.d, at, a.r, u, at.turned ? (a.positions ? a.positions[tok0 + t] : start + t) : 0,
                           1.0f, a.s.hq - h0);
    }
}

// grid (nslots + qblocks, hkv, min(batch, 65535)).
template <class T, int WPS, int HPT>
__global__ __launch_bounds__(128 * WPS) void k_kv_append(AppendArgs a)
{
    bool used = false;   // the block's shared memory
    for (int b = blockIdx.z; b < a.s.batch; b += gridDim.z) {
        long tok0;
        int n;
        const int kv_len = a.kv_lens[b];
        seq_range(a.cu_q, a.s, b, &tok0, &n);
        if (n == 0) continue;
        const int start = kv_len - n;
        if ((int)blockIdx.x < a.nslots) {
            if (kv_len <= 0) continue;
            const int p0 = (start > 0 ? start : 0) / a.s.page;
            int p1 = (kv_len - 1) / a.s.page;
            p1 = p1 < a.s.table_stride ? p1 : a.s.table_stride - 1;
            for (int p = p0 + (int)blockIdx.x; p <= p1; p += a.nslots) {
                if (used) __syncthreads();
                used = true;
                append_page<T, WPS>(a, b, blockIdx.y, p * a.s.page, tok0, n, start);
            }
        } else {
            turn_queries<T, HPT>(a, tok0, n, start, (blockIdx.x - a.nslots) * gridDim.y + blockIdx.y, a.qblocks * gridDim.y,
                               128 * WPS);
        }
    }
}

// Blocks of `threads` that turn mq tokens of a sequence, HPT heads a thread: at
// least one token's threads, and (they loop) at most what 32-bit numbers hold.
static long query_blocks(AppendArgs& a, int hpt, long mq, long threads)
{
    const long work = (long)((a.s.hq + hpt - 1) / hpt) * (a.s.d / 16);
    a.qwork = FastDiv::make((unsigned)work);
    const long least = (work + threads - 1) / threads, all = (mq * work + 4 * threads - 1) / (4 * threads);
    const long most = 65536;
    return all > most ? (least > most ? least : most) : (all < least ? least : all);
}

// One launch: the blocks that append and those that turn queries are independent,
// and the ones wait on chains of loads while the others stream (six prompts, four
// heads a thread: 119 us; as two launches, 70 + 66).
template <class T, int WPS, int HPT>
static hipError_t launch_append(AppendArgs a, hipStream_t st)
{
    const long mq = a.s.max_q > 0 ? a.s.max_q : 1;
    const long kept = (mq < a.s.page ? mq : a.s.page) * (long)a.s.d;   // keys a block turns at most
    a.lds_floats = kept <= 15360 ? (int)kept : 0;
    const long slots = mq == 1 ? 1 : (mq + a.s.page - 2) / a.s.page + 1;
    a.nslots = (int)(slots < 65536 ? slots : 65536);   // (blocks loop)
    a.qblocks = a.q ? (int)((query_blocks(a, HPT, mq, 128L * WPS) + a.s.hkv - 1) / a.s.hkv) : 0;
    const dim3 grid((unsigned)(a.nslots + a.qblocks), a.s.hkv, a.s.batch < 65535 ? a.s.batch : 65535);
    k_kv_append<T, WPS, HPT><<<grid, dim3(128 * WPS), a.lds_floats * 4, st>>>(a);
    return hipGetLastError();
}

// Waves a side by the page's values, and heads a thread that turns queries.
// Measured for prompts of 5000 (us): pages of 16 x 64 values 88 with one wave a
// side, 110 with two; 64 x 128 139 with two, 158 with four; 256 x 256 157 with
// four, 190 with two.  Six prompts with pages of 32 x 128: 132, 112 and 118 with
// one, two and four heads a thread; steps of few tokens want many threads.
template <class T>
static hipError_t pick_append(const AppendArgs& a, hipStream_t st)
{
    if (a.s.max_q <= 16) return launch_append<T, 1, 1>(a, st);
    const int values = a.s.page * a.s.d;
    if (values <= 2048) return launch_append<T, 1, 2>(a, st);
    return values <= 8192 ? launch_append<T, 2, 2>(a, st) : launch_append<T, 4, 2>(a, st);
}

hipError_t run_kv_append(int dtype, const void* k, const void* v, const void* q, void* q_out, const long* strides,
                         uint8_t* codes, float* scales, const int* table, const int* cu_q, const int* kv_lens,
                         const int* positions, const KvShape& s, const RopeArgs& r, hipStream_t st)
{
    if (s.batch == 0 || s.tokens == 0) return hipSuccess;
    AppendArgs a{};
    a.k = k;
    a.v = v;
    a.q = q;
    a.q_out = q_out;
    a.k_ts = strides[0];
    a.k_hs = strides[1];
    a.v_ts = strides[2];
    a.v_hs = strides[3];
    a.q_ts = strides[4];
    a.q_hs = strides[5];
    a.codes = codes;
    a.scales = scales;
    a.table = table;
    a.cu_q = cu_q;
    a.kv_lens = kv_lens;
    a.positions = positions;
    a.s = s;
    a.r = r;
    a.units = FastDiv::make(s.d / 16);
    a.d8 = FastDiv::make(s.d / 8);
    a.dpair = FastDiv::make(s.d / 2);
    return dtype == DT_F16 ? pick_append<half_t>(a, st) : pick_append<bf16_t>(a, st);
}

}  // namespace fc

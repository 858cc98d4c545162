// kv_common.h -- what the attention-serving kernels (rope.hip, kv_append.hip,
// attn_rows.hip, attn_tile.hip) share: the activations' types, the cache's
// layout, the lookup of a page and the angle of a position.
//
// Layout of the cache.  codes [pages][kv heads][2 (K, V)][page / 16][16 * d],
// OCP e4m3 bytes, in blocks of 16 tokens that are the matrix instructions' own
// operand order, so that a fragment is loaded by 16 bytes a lane from
// consecutive addresses, with no transposition on the way:
//     K block  [d / 16][16 tokens][16 dims]     (operand A of K q: rows = keys)
//     V block  [d][16 tokens]                   (operand A of V^T p: rows = dims)
// scales [pages][kv heads][2]: a power of two for each page, head and side.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "fc_device.h"

namespace fc {

typedef __bf16 bf16_t;
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float floatx2 __attribute__((ext_vector_type(2)));

enum { DT_F16 = 0, DT_BF16 = 1 };

// Strides in elements; see fc_kv_shape.
struct KvShape {
    int batch, hq, hkv, d, page, pages, table_stride;
    long tokens;
    int max_q, max_kv;
};

struct RopeArgs {
    const unsigned long long* turns;   // [rot / 2], fractions of a turn a position, 2^64 = one turn
    int rot, interleaved;
    float mscale;
};

// Type traits: vectors of 8, conversions, the two matrix instructions.
template <class T> struct Tr;
template <> struct Tr<half_t> {
    typedef half8 v8;
    static constexpr int elo = -15, ehi = 7;    // scale exponents: code * scale is exactly an fp16 value
    static constexpr int up = 15;               // 2^up is a value of the type: see the weights below
    __device__ static __forceinline__ unsigned from_fp8(unsigned w, float s, bool hi)
    {
        return hi ? __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, s, true))
                  : __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, s, false));
    }
    __device__ static __forceinline__ unsigned pk(float a, float b)
    {
        half2v h;
        h[0] = (half_t)a;
        h[1] = (half_t)b;
        return __builtin_bit_cast(unsigned, h);
    }
    // s + the two values of w, in 32 bits
    __device__ static __forceinline__ float add2(unsigned w, float s)
    {
        half2v one;
        one[0] = one[1] = (half_t)1.0f;
        return __builtin_amdgcn_fdot2(__builtin_bit_cast(half2v, w), one, s, false);
    }
    __device__ static __forceinline__ floatx4 mfma16(v8 a, v8 b, floatx4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    __device__ static __forceinline__ floatx16 mfma32(v8 a, v8 b, floatx16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
};
template <> struct Tr<bf16_t> {
    typedef bf8 v8;
    static constexpr int elo = -100, ehi = 119;
    static constexpr int up = 0;                // (the type has the range of 32 bits)
    __device__ static __forceinline__ unsigned from_fp8(unsigned w, float s, bool hi)
    {
        return hi ? __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true))
                  : __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false));
    }
    __device__ static __forceinline__ unsigned pk(float a, float b)
    {
        bf2 h;
        h[0] = (bf16_t)a;
        h[1] = (bf16_t)b;
        return __builtin_bit_cast(unsigned, h);
    }
    __device__ static __forceinline__ float add2(unsigned w, float s)
    {
        bf2 one;
        one[0] = one[1] = (bf16_t)1.0f;
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf2, w), one, s, false);
    }
    __device__ static __forceinline__ floatx4 mfma16(v8 a, v8 b, floatx4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    __device__ static __forceinline__ floatx16 mfma32(v8 a, v8 b, floatx16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};

// 8 codes (two dwords) to a matrix operand of 8 values, times the power of two s.
template <class T>
__device__ __forceinline__ typename Tr<T>::v8 frag8(unsigned w0, unsigned w1, float s)
{
    u32x4 r;
    r[0] = Tr<T>::from_fp8(w0, s, false);
    r[1] = Tr<T>::from_fp8(w0, s, true);
    r[2] = Tr<T>::from_fp8(w1, s, false);
    r[3] = Tr<T>::from_fp8(w1, s, true);
    return __builtin_bit_cast(typename Tr<T>::v8, r);
}

template <class T>
__device__ __forceinline__ void unpack8(u32x4 w, float (&x)[8])
{
    const typename Tr<T>::v8 v = __builtin_bit_cast(typename Tr<T>::v8, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)v[i];
}

template <class T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8])
{
    const typename Tr<T>::v8 v = *reinterpret_cast<const typename Tr<T>::v8*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)v[i];
}

template <class T>
__device__ __forceinline__ u32x4 pack8(const float (&x)[8])
{
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = Tr<T>::pk(x[2 * i], x[2 * i + 1]);
    return r;
}

// The byte of the pool at which (page id, head, side) begins.
__device__ __forceinline__ size_t side_base(int id, int h, int side, const KvShape& s)
{
    return ((size_t)((size_t)id * s.hkv + h) * 2 + side) * ((size_t)s.page * s.d);
}

// The id of page `pidx` of sequence b, or -1 where the table has none: an index
// past the table's row or an id outside the pool.  Every kernel goes through
// this, so that no table can make it read or write outside the pool.
__device__ __forceinline__ int page_id(const int* table, const KvShape& s, int b, int pidx)
{
    if ((unsigned)pidx >= (unsigned)s.table_stride) return -1;
    const int id = table[(size_t)b * s.table_stride + pidx];
    return (unsigned)id < (unsigned)s.pages ? id : -1;
}

// Sequence b's first token and its number of new tokens, inside [0, tokens).
__device__ __forceinline__ void seq_range(const int* cu_q, const KvShape& s, int b, long* first, int* n)
{
    long a = cu_q[b], z = cu_q[b + 1];
    a = a < 0 ? 0 : (a > s.tokens ? s.tokens : a);
    z = z < a ? a : (z > s.tokens ? s.tokens : z);
    *first = a;
    *n = (int)(z - a);
}

// Sequence b's number of keys.  A length that its row of the table cannot hold
// counts as none, and *over makes the caller's results NaN: a broken length
// neither reads past the table nor keeps a kernel busy.
__device__ __forceinline__ int seq_keys(const int* kv_lens, const KvShape& s, int b, bool* over)
{
    const int n = kv_lens[b];
    *over = n > s.page * s.table_stride;
    return n < 0 || *over ? 0 : n;
}

// sin and cos of position p times the frequency f (a 64-bit fraction of a
// turn).  The product's low 64 bits are the turn's fraction, exact for every
// 32-bit position (the far ones too, where a 32-bit float angle is off by
// whole radians); its upper 32 bits go to the hardware's sine and cosine,
// which take turns.  Measured against 64 bits over the turn: 1.25e-7 absolute.
__device__ __forceinline__ void turn_sincos(int p, unsigned long long f, float& sn, float& cs)
{
    const unsigned lo = (unsigned)f, hi = (unsigned)(f >> 32), u = (unsigned)p;
    unsigned frac = __umulhi(u, lo) + u * hi;
    if (p < 0) frac -= lo;   // u = p + 2^32
    const float t = (float)(int)frac * 0x1p-32f;
    sn = __builtin_amdgcn_sinf(t);
    cs = __builtin_amdgcn_cosf(t);
}

// One unit of 16 elements of a head: 8 rotated pairs, or 16 elements that pass.
// Unit u < rot / 16 holds the pairs 8u .. 8u + 7; the elements sit at e0 .. e0
// + 7 and e1 .. e1 + 7.
struct Unit {
    int e0, e1;
    bool turned;
};
__device__ __forceinline__ Unit unit_of(int u, int rot, int interleaved)
{
    Unit r;
    r.turned = u * 16 < rot;
    const bool half = r.turned && !interleaved;
    r.e0 = half ? u * 8 : u * 16;
    r.e1 = half ? rot / 2 + u * 8 : u * 16 + 8;
    return r;
}

// x0, x1: the elements at e0.. and e1..; cs, sn: the 8 pairs' cosines and sines.
__device__ __forceinline__ void rotate_unit(float (&x0)[8], float (&x1)[8], const float (&cs)[8], const float (&sn)[8],
                                            int interleaved)
{
    if (!interleaved) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float a = x0[j], b = x1[j];
            x0[j] = a * cs[j] - b * sn[j];
            x1[j] = a * sn[j] + b * cs[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float a = x0[2 * j], b = x0[2 * j + 1], c = x1[2 * j], d = x1[2 * j + 1];
            x0[2 * j] = a * cs[j] - b * sn[j];
            x0[2 * j + 1] = a * sn[j] + b * cs[j];
            x1[2 * j] = c * cs[4 + j] - d * sn[4 + j];
            x1[2 * j + 1] = c * sn[4 + j] + d * cs[4 + j];
        }
    }
}

__device__ __forceinline__ void unit_angles(const unsigned long long* turns, int u, int p, float mscale, float sign,
                                            float (&cs)[8], float (&sn)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        turn_sincos(p, turns[u * 8 + j], sn[j], cs[j]);
        cs[j] *= mscale;
        sn[j] *= mscale * sign;
    }
}

// One unit of up to HPT heads, whose angles are computed once: p + k * ph to o +
// k * oh.  The loads go out together and stay packed until their head's turn, so
// that registers leave room for waves (p and o may be the same).
template <class T, int HPT>
__device__ __forceinline__ void turn_heads(const T* p, T* o, long ph, long oh, const Unit& at, const RopeArgs& r, int u, int pos,
                                           float sign, int heads)
{
    u32x4 w[HPT][2];
#pragma unroll
    for (int k = 0; k < HPT; ++k) {
        if (HPT > 1 && k >= heads) break;
        w[k][0] = *reinterpret_cast<const u32x4*>(p + k * ph + at.e0);
        w[k][1] = *reinterpret_cast<const u32x4*>(p + k * ph + at.e1);
    }
    float cs[8], sn[8];
    if (at.turned) unit_angles(r.turns, u, pos, r.mscale, sign, cs, sn);
#pragma unroll
    for (int k = 0; k < HPT; ++k) {
        if (HPT > 1 && k >= heads) break;
        if (at.turned) {
            float x0[8], x1[8];
            unpack8<T>(w[k][0], x0);
            unpack8<T>(w[k][1], x1);
            rotate_unit(x0, x1, cs, sn, r.interleaved);
            w[k][0] = pack8<T>(x0);
            w[k][1] = pack8<T>(x1);
        }
        *reinterpret_cast<u32x4*>(o + k * oh + at.e0) = w[k][0];
        *reinterpret_cast<u32x4*>(o + k * oh + at.e1) = w[k][1];
    }
}

// Maximum over the lanes l, l ^ 32 (and l ^ 16): a register swap with itself
// puts the two halves (rows of 16) side by side.
__device__ __forceinline__ float max_x32(float v)
{
    const unsigned u = __builtin_bit_cast(unsigned, v);
    const auto p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return fmaxf(__builtin_bit_cast(float, (unsigned)p[0]), __builtin_bit_cast(float, (unsigned)p[1]));
}
__device__ __forceinline__ float max_x16(float v)
{
    const unsigned u = __builtin_bit_cast(unsigned, v);
    const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return fmaxf(__builtin_bit_cast(float, (unsigned)p[0]), __builtin_bit_cast(float, (unsigned)p[1]));
}
__device__ __forceinline__ float sum_x32(float v)
{
    const unsigned u = __builtin_bit_cast(unsigned, v);
    const auto p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __builtin_bit_cast(float, (unsigned)p[0]) + __builtin_bit_cast(float, (unsigned)p[1]);
}
__device__ __forceinline__ float sum_x16(float v)
{
    const unsigned u = __builtin_bit_cast(unsigned, v);
    const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return __builtin_bit_cast(float, (unsigned)p[0]) + __builtin_bit_cast(float, (unsigned)p[1]);
}

// The attention kernels' arguments.  A "row" is one query of one head; rows of
// the heads that share a kv head are adjacent: row r of (sequence, kv head) is
// query r / G, head h * G + r % G.
struct AttnArgs {
    const void* q;
    long q_ts, q_hs;
    const uint8_t* codes;
    const float* scales;
    const int *table, *cu_q, *kv_lens;
    const float* slopes;   // [hq] or NULL
    void* out;             // [tokens, hq, d]
    float* lse;            // [tokens, hq] or NULL
    float* part_o;         // workspace of nsplit > 1: [tokens, hq, nsplit, d] and
    floatx4* part_ml;      // [tokens, hq, nsplit] of {maximum (log 2), sum of weights, exact sum (for lse), -}
    KvShape s;
    int G, causal, window, nsplit, chunk;   // chunk: blocks of 16 keys a split
    int pg_shift;                            // a page holds 2^pg_shift blocks of 16
    float scale, cap;
    FastDiv by_g;
    // A tree of new tokens instead of causal order: which of its sequence's new tokens each sees, a
    // bit each [tokens, tree_words], and their positions [tokens].
    const unsigned long long* tree_bits;
    const int* tree_pos;
    int tree_words;
    // The tile form shares trees' work evenly (even != 0): the stages of all sequences' keys, one after
    // the other, go in equal parts to `even` blocks for each head and tile of rows. The results of a
    // sequence that several blocks have go to slot (block + sequence) of the head's and tile's `slots`,
    // each of the form's rows: part_o [hkv, row tiles, slots, rows, d], part_ml [hkv, row tiles, slots,
    // rows]; ends [batch][2]: the sequence's first and last block.
    int even, slots;
    int* ends;
};

// The bits of the 64 nodes from `node` on (which may lie before the tree or past it).
__device__ __forceinline__ unsigned long long tree_window(const unsigned long long* row, int words, int node)
{
    const int w = node >> 6, sh = node & 63;
    const unsigned long long lo = (unsigned)w < (unsigned)words ? row[w] : 0;
    const unsigned long long hi = (unsigned)(w + 1) < (unsigned)words ? row[w + 1] : 0;
    return sh ? lo >> sh | hi << (64 - sh) : lo;
}

// The position of new token `at`, kept where a tree of a sequence's nq tokens can reach.
__device__ __forceinline__ int tree_place(const AttnArgs& a, long at, int pos0, int kv_len)
{
    const int p = a.tree_pos[at];
    return p < pos0 ? pos0 : p < kv_len ? p : kv_len - 1;
}

// The first key that a query at `pos` sees (no difference of the two leaves 32 bits,
// whatever the window and for positions before 0 too).
__device__ __forceinline__ int first_seen(const AttnArgs& a, int pos)
{
    return a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
}

// The keys that rows r0 .. r1 - 1 (of q_len * G) may see, as blocks of 16
// [*g0, *g1), and the first query's position.
__device__ __forceinline__ void key_range(const AttnArgs& a, int kv_len, int pos0, int t0, int t1, int* g0, int* g1)
{
    const int lo = first_seen(a, pos0 + t0);
    int hi = a.causal ? pos0 + t1 + 1 : kv_len;   // t1: the last query
    hi = hi > kv_len ? kv_len : hi;
    *g0 = lo >> 4;
    *g1 = hi > lo ? (hi + 15) >> 4 : *g0;
}

// What a page outside the pool is read as: NaN keys, so that the rows that see
// them turn NaN and no others, and zero values.
struct NoPage {
    unsigned codes[2][1024];   // the 4 KiB of a block of 16 tokens, d = 256
    float scale[2];
};
__host__ __device__ constexpr NoPage make_no_page()
{
    NoPage p{};
    for (int i = 0; i < 1024; ++i) p.codes[0][i] = 0x7f7f7f7fu;
    p.scale[0] = p.scale[1] = 1.0f;
    return p;
}
static __device__ __align__(16) NoPage fc_no_page = make_no_page();

// Global memory by its address space: a pointer chosen between the pool and
// fc_no_page would otherwise be a generic one and its loads flat, and those are
// waited for with the LDS reads.
#define FC_GLOBAL __attribute__((address_space(1)))
typedef FC_GLOBAL const uint8_t global_u8;
__device__ __forceinline__ global_u8* global_at(const void* p) { return (global_u8*)p; }

// Kinds of scores: scale * q . k alone; with a bias by distance (causal); capped by
// at most NEAR_CAP; such a cap and a bias, or a bias to both sides; capped by more,
// with a bias or without.
enum { SC_PLAIN = 0, SC_BIAS = 1, SC_CAP = 2, SC_ANY = 3, SC_FAR = 4 };
constexpr float NEAR_CAP = 128.0f;
__host__ __device__ constexpr bool may_bias(int kind) { return kind == SC_BIAS || kind == SC_ANY || kind == SC_FAR; }
inline int score_kind(const AttnArgs& a)
{
    if (a.cap > NEAR_CAP) return SC_FAR;
    if (!a.slopes) return a.cap > 0.0f ? SC_CAP : SC_PLAIN;
    return a.cap > 0.0f || !a.causal ? SC_ANY : SC_BIAS;
}
// Calls f(IntC<kind>{}) for the call's kind.
template <class F> inline hipError_t by_kind(const AttnArgs& a, F&& f)
{
    switch (score_kind(a)) {
    case SC_PLAIN: return f(IntC<SC_PLAIN>{});
    case SC_BIAS: return f(IntC<SC_BIAS>{});
    case SC_CAP: return f(IntC<SC_CAP>{});
    case SC_FAR: return f(IntC<SC_FAR>{});
    default: return f(IntC<SC_ANY>{});
    }
}

// The same for a tree, whose keys are not in order of distance: a bias takes the general kind.
template <class F> inline hipError_t by_tree_kind(const AttnArgs& a, F&& f)
{
    switch (score_kind(a)) {
    case SC_PLAIN: return f(IntC<SC_PLAIN>{});
    case SC_CAP: return f(IntC<SC_CAP>{});
    case SC_FAR: return f(IntC<SC_FAR>{});
    default: return f(IntC<SC_ANY>{});
    }
}

// The weights are rounded to the activations' type before the second product.
// The sum that divides the result is of the rounded ones, so that it matches its
// numerator (a row of one dominant key comes out as that key's value); lse takes
// the sum of the unrounded ones.  fp16 weights are lifted by a power of two, which
// the division takes out again, to the top of the type's range: with the largest at
// 1, those under 2^-14 would lose bits and those under 2^-25 vanish, and a long flat
// tail under one dominant key with them (131071 keys 17.4 below it are 0.36 % of
// the result); lifted, a weight is rounded by 2^-32 of the largest at most.

// cap * tanh(t) - from, for s * c0 = 2 log2(e) t: cap (1 - 2 / (1 + e^2t)), which
// saturates at both ends.  Its error is absolute, up to 3e-7 cap however small the
// score: for caps to NEAR_CAP 4e-5, a tenth of a weight's rounding to fp16.
__device__ __forceinline__ float capped(float s, float c0, float cap, float from)
{
    return __builtin_fmaf(__builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(s * c0)), -2.0f * cap, cap - from);
}

// The same for any cap, to 2^-19 of the result: where |t| < 1/4 by the odd series t
// (1 - t^2 / 3 + 2 t^4 / 15 - 17 t^6 / 315 + 62 t^8 / 2835) (the next term is 2^-26
// of it), so that a cap far above the scores is none.  Seven more operations a score
// (two prompts of 4096 with 32 heads of 128: 464 us, against 366).
__device__ __forceinline__ float capped_far(float s, float c0, float cap, float from)
{
    constexpr float k2 = 0.12011325f;   // (t / z)^2, z = 2 log2(e) t
    const float z = s * c0, w = z * z * k2;
    float p = 62.0f / 2835.0f;
    p = __builtin_fmaf(p, w, -17.0f / 315.0f);
    p = __builtin_fmaf(p, w, 2.0f / 15.0f);
    p = __builtin_fmaf(p, w, -1.0f / 3.0f);
    p = __builtin_fmaf(p, w, 1.0f);
    const float small = __builtin_fmaf(z * (0.34657359f * cap), p, -from);   // z / (2 log2(e)) = t
    return fabsf(z) < 0.7213475f ? small : capped(s, c0, cap, from);
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_inff();

}  // namespace fc

// attn_rows.hip -- attention over the paged 8-bit cache for few rows (the
// queries of one step): k_attn_rows, and the join of split results,
// k_attn_join.
//
// A chain of two products whose intermediate stays in registers: a wave takes
// 64 keys (four cache blocks of 16) at a time, S^T = K q^T (rows = keys,
// columns = query rows, MFMA 16x16x32), the softmax of a column lives in the
// four lanes that hold it (the running maximum and sum in 32 bits), and the
// weights, rounded once to the activations' type, become the second product's
// operand B: O^T += V^T p^T.  Tile t is block t, so that a load of K is 1 KiB of
// consecutive bytes; the accumulators then hold keys 4g .. 4g + 3 of block t in
// lane group g and register t, and V's operand, 16 bytes a lane, wants block g
// in lane group g: a transposition of 4 x 4 by eight register swaps.
//
// Bound by the cache's bytes: every code is read once, by one wave, with the
// non-temporal hint (a plain gather of the same 16 KiB pieces: 6.1 TB/s without
// and 7.0 with it).  K of the next keys is requested when this one's products
// are done, V when its own are, so that a wave always has 8 to 16 KiB on the
// way.  The keys are split over a block's waves, and over blocks where
// sequences x heads alone do not fill the machine; the waves' results are
// joined through LDS and the blocks' by k_attn_join, both in a fixed order.
// Measured: 64 sequences x 8 kv heads of 128, to 8192 keys, 756 MB in 127 to 133 us
// (5.7 to 5.9 TB/s); 2 x 4, 131071 keys, 269 MB in 53 us with the join; 24 x 16 heads
// of 256, three tokens, a window of 4096, 786 MB in 135 to 141 us (5.6 to 5.8 TB/s).
// 17 to 32 rows with heads of 256 are far from that: two column tiles beside 64 keys
// of K and V take all 512 registers, 65 to 73 are spilled, and 24 sequences of up to
// 9000 keys x 8 heads, 24 rows each, take 216 us for 594 MB (2.7 TB/s).
#include "fc_launch.h"
#include "kv_common.h"

namespace fc {

constexpr int AR_WAVES = 4;

__device__ __forceinline__ u32x4 load_nt(global_u8* p)
{
    return __builtin_nontemporal_load((FC_GLOBAL const u32x4*)p);
}

template <class T, int D, int NT, int MODE>
__global__ __launch_bounds__(64 * AR_WAVES, NT == 1 && D <= 128 ? 2 : 1) void k_attn_rows(AttnArgs a, int row_blocks)
{
    typedef typename Tr<T>::v8 v8;
    constexpr int R = 16 * NT;       // rows a block
    constexpr int NJ = D / 64;       // 16-byte loads of K a lane and tile
    constexpr int ND = D / 16;       // tiles of V^T
    constexpr int UP = Tr<T>::up;    // weights, at most 1, times 2^UP
    // (the largest score's argument is exactly 0, whatever its size, so that 2^UP is not passed)
    auto weight = [](float x) { return __builtin_amdgcn_exp2f(UP ? x + (float)UP : x); };
    const KvShape& s = a.s;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int h = blockIdx.y / row_blocks, rb0 = blockIdx.y % row_blocks, split = blockIdx.z;

    extern __shared__ __align__(16) float lds[];   // [wave][NT][ND][lane] of four, then [wave][NT][16] of four
    FC_LDS floatx4* const lds_o = (FC_LDS floatx4*)(FC_LDS float*)lds;
    FC_LDS floatx4* const lds_ml = lds_o + AR_WAVES * NT * ND * 64;
    if constexpr (kPoison) {
        lds_poison((FC_LDS float*)lds, AR_WAVES * NT * (ND * 64 + 16) * 16, threadIdx.x, 64 * AR_WAVES);
        __syncthreads();
    }
    global_u8* no_page = global_at(&fc_no_page);
    asm("" : "+s"(no_page));   // the address is taken once, not by a load in every step

    {
        const int b = blockIdx.x;
        // The id of the first page that a lane group looks up, if the keys begin at 0: requested
        // with the lengths rather than after them, one memory latency less before the first codes.
        const int* const row_of = a.table + (size_t)b * s.table_stride;
        const int first = split * a.chunk + 4 * wave + g, first_pg = first >> a.pg_shift;
        const int raw0 = row_of[first_pg < s.table_stride ? first_pg : 0];
        long tok0;
        int nq;
        seq_range(a.cu_q, s, b, &tok0, &nq);
        const int rows = nq * a.G;
        bool over;
        const int kv_len = seq_keys(a.kv_lens, s, b, &over), pos0 = kv_len - nq;
        global_u8* const head = global_at(a.codes) + side_base(0, h, 0, s);
        const size_t page_bytes = (size_t)s.hkv * 2 * s.page * D;
        const int side_bytes = s.page * D;
        for (int r0 = rb0 * R; r0 < rows; r0 += row_blocks * R) {
            const int r1 = r0 + R < rows ? r0 + R : rows;
            const int t_first = a.by_g.div(r0), t_last = a.by_g.div(r1 - 1);
            int g_lo, g_hi;
            key_range(a, kv_len, pos0, t_first, t_last, &g_lo, &g_hi);

            if (a.nsplit > 1 && g_lo + split * a.chunk >= g_hi && !over) {   // no keys for this split
                for (int r = r0 + threadIdx.x; r < r1; r += 64 * AR_WAVES) {
                    const int t = a.by_g.div(r), hq = h * a.G + (r - t * a.G);
                    a.part_ml[((tok0 + t) * s.hq + hq) * a.nsplit + split] = floatx4{kNegInf, 0.0f, 0.0f, 0.0f};
                }
                continue;
            }
            // this lane's rows: position, bias, query
            int pos[NT];
            float slope[NT];
            v8 qf[NT][2 * NJ];
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                const int r = r0 + 16 * c + n, rr = r < rows ? r : rows - 1;
                const int t = a.by_g.div(rr), hq = h * a.G + (rr - t * a.G);
                pos[c] = pos0 + t;
                slope[c] = may_bias(MODE) && a.slopes ? a.slopes[hq] * kLog2e : 0.0f;
                const T* q = (const T*)a.q + (tok0 + t) * a.q_ts + (long)hq * a.q_hs;
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        qf[c][2 * j + e] = *reinterpret_cast<const v8*>(q + 16 * (4 * j + g) + 8 * e);
            }
            // keys that every row of the tile sees need no mask
            const int all_lo = first_seen(a, pos0 + t_last);
            const int all_hi = a.causal ? (pos0 + t_first + 1 < kv_len ? pos0 + t_first + 1 : kv_len) : kv_len;

            // scores in units of log 2 are q . k on the codes, times the page's scale, times this
            const bool cap = MODE == SC_CAP || MODE == SC_FAR || (MODE == SC_ANY && a.cap > 0.0f);
            const float factor = cap ? 2.0f * kLog2e * a.scale / a.cap : a.scale * kLog2e;
            floatx4 o[NT][ND];
            float m[NT], l[NT], le[NT];   // maximum; sums of rounded and (for lse) of exact weights
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                m[c] = kNegInf;
                l[c] = le[c] = 0.0f;
#pragma unroll
                for (int d = 0; d < ND; ++d) o[c][d] = floatx4{0, 0, 0, 0};
            }

            for (int c0 = g_lo + split * a.chunk; c0 < g_hi; c0 += a.nsplit * a.chunk) {
                const int c1 = c0 + a.chunk < g_hi ? c0 + a.chunk : g_hi;
                // Lane group g looks up block k0 + g: its page's id (two steps ahead), scales.
                auto block_of = [&](int k0) { return k0 + g < c1 ? k0 + g : c1 - 1; };
                auto load_id = [&](int k0) {
                    const int pg = block_of(k0) >> a.pg_shift;
                    const int id = row_of[pg < s.table_stride ? pg : 0];
                    return id;
                };
                u32x4 kr[4][NJ], vr[ND];
                floatx2 sc;
                int id;      // of this lane group's block, or -1
                auto settle_id = [&](int raw, int k0) {
                    id = (unsigned)raw < (unsigned)s.pages && (block_of(k0) >> a.pg_shift) < s.table_stride ? raw : -1;
                };
                auto load_k = [&](int k0) {
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const int it = __builtin_amdgcn_readlane(id, 16 * t);
                        const int kb = k0 + t < c1 ? k0 + t : c1 - 1;
                        global_u8* src = it < 0 ? no_page : head + it * page_bytes + (kb & ((1 << a.pg_shift) - 1)) * (16 * D);
#pragma unroll
                        for (int j = 0; j < NJ; ++j) kr[t][j] = load_nt(src + j * 1024 + lane * 16);
                    }
                };
                auto load_v = [&](int k0) {
                    global_u8* src = id < 0 ? no_page + 4096
                                            : head + side_bytes + id * page_bytes +
                                                  (block_of(k0) & ((1 << a.pg_shift) - 1)) * (16 * D);
                    global_u8* scale = id < 0 ? no_page + offsetof(NoPage, scale)
                                              : global_at(a.scales) + ((size_t)id * s.hkv + h) * 8;
                    sc = *(FC_GLOBAL const floatx2*)scale;
#pragma unroll
                    for (int d = 0; d < ND; ++d) vr[d] = load_nt(src + d * 256 + n * 16);
                };
                constexpr int STEP = 4 * AR_WAVES;
                int k0 = c0 + 4 * wave;
                if (k0 >= c1) continue;
                // (raw0 is block k0 + g's unless that lies past the end, where its page may differ)
                int raw = c0 == split * a.chunk && k0 + g < c1 ? raw0 : load_id(k0);
                settle_id(raw, k0);
                load_k(k0);
                load_v(k0);
                raw = load_id(k0 + STEP);
                for (; k0 < c1; k0 += STEP) {
                    floatx4 st[NT][4];
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
#pragma unroll
                        for (int c = 0; c < NT; ++c) st[c][t] = floatx4{0, 0, 0, 0};
#pragma unroll
                        for (int j = 0; j < NJ; ++j)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const v8 kf = frag8<T>(kr[t][j][2 * e], kr[t][j][2 * e + 1], 1.0f);
#pragma unroll
                                for (int c = 0; c < NT; ++c) st[c][t] = Tr<T>::mfma16(kf, qf[c][2 * j + e], st[c][t]);
                            }
                    }
                    const float vs = sc[1];
                    const float f = sc[0] * factor;
                    float ft[4];   // the factor of tile t's scores
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        ft[t] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, f), 16 * t));
                    __builtin_amdgcn_sched_barrier(0);
                    settle_id(raw, k0 + STEP);
                    load_k(k0 + STEP);   // past the end: the last block again, unused
                    __builtin_amdgcn_sched_barrier(0);

                    const int key0 = k0 * 16 + 4 * g;
                    const bool masked = k0 * 16 < all_lo || (k0 + 4) * 16 > all_hi || k0 + 4 > c1;
                    v8 pf[NT][2];
#pragma unroll
                    for (int c = 0; c < NT; ++c) {
                        float x[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float y = st[c][i >> 2][i & 3];
                            x[i] = MODE == SC_FAR ? capped_far(y, ft[i >> 2], a.cap * kLog2e, 0.0f)
                                   : cap          ? capped(y, ft[i >> 2], a.cap * kLog2e, 0.0f)
                                                  : y * ft[i >> 2];
                        }
                        if (may_bias(MODE)) {
                            const float gap = (float)(pos[c] - key0);
#pragma unroll
                            for (int i = 0; i < 16; ++i) x[i] -= slope[c] * fabsf(gap - (float)((i >> 2) * 16 + (i & 3)));
                        }
                        if (masked) {
                            int top = a.causal && pos[c] + 1 < kv_len ? pos[c] + 1 : kv_len;
                            top = (top < c1 * 16 ? top : c1 * 16) - key0;
                            const int low = first_seen(a, pos[c]) - key0;
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const int k = (i >> 2) * 16 + (i & 3);
                                x[i] = k < top && k >= low ? x[i] : kNegInf;
                            }
                        }
                        float mx = x[0];
#pragma unroll
                        for (int i = 1; i < 16; ++i) mx = fmaxf(mx, x[i]);
                        mx = max_x32(max_x16(mx));
                        const float mn = fmaxf(m[c], mx);
                        const float ms = mn == kNegInf ? 0.0f : mn;   // nothing seen yet: all weights are 0
                        if (__any(mx > m[c])) {
                            const float alpha = __builtin_amdgcn_exp2f(m[c] - ms);
                            m[c] = mn;
                            l[c] *= alpha;
                            le[c] *= alpha;
#pragma unroll
                            for (int d = 0; d < ND; ++d) o[c][d] *= alpha;
                        }
                        float sum = 0.0f, exact = 0.0f;
                        unsigned w[4][2];
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const float p0 = weight(x[i] - ms), p1 = weight(x[i + 1] - ms);
                            w[i >> 2][(i >> 1) & 1] = Tr<T>::pk(p0, p1);
                            sum = Tr<T>::add2(w[i >> 2][(i >> 1) & 1], sum);
                            exact += p0 + p1;
                        }
                        l[c] += sum;
                        le[c] += exact;
                        // [register t][lane group g] -> [g][t]
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
#pragma unroll
                            for (int t = 0; t < 2; ++t) {
                                const auto y = __builtin_amdgcn_permlane32_swap(w[t][e], w[t + 2][e], false, false);
                                w[t][e] = y[0];
                                w[t + 2][e] = y[1];
                            }
#pragma unroll
                            for (int t = 0; t < 4; t += 2) {
                                const auto y = __builtin_amdgcn_permlane16_swap(w[t][e], w[t + 1][e], false, false);
                                w[t][e] = y[0];
                                w[t + 1][e] = y[1];
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            pf[c][e] = __builtin_bit_cast(v8, u32x4{w[2 * e][0], w[2 * e][1], w[2 * e + 1][0], w[2 * e + 1][1]});
                    }
                    // tokens past the end hold whatever the page held: their weight is 0, and
                    // 0 times a NaN code is NaN, so their codes are cleared
                    if ((k0 + 4) * 16 > kv_len) {
                        const int keep = kv_len - (k0 + g) * 16;
                        u32x4 mk;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int k = keep - 4 * j;
                            mk[j] = k >= 4 ? ~0u : (k <= 0 ? 0u : (1u << (8 * k)) - 1u);
                        }
#pragma unroll
                        for (int d = 0; d < ND; ++d) vr[d] &= mk;
                    }
#pragma unroll
                    for (int d = 0; d < ND; ++d)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const v8 vf = frag8<T>(vr[d][2 * e], vr[d][2 * e + 1], vs);
#pragma unroll
                            for (int c = 0; c < NT; ++c) o[c][d] = Tr<T>::mfma16(vf, pf[c][e], o[c][d]);
                        }
                    __builtin_amdgcn_sched_barrier(0);
                    load_v(k0 + STEP);
                    raw = load_id(k0 + 2 * STEP);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            // Join the waves: each brings its result to the common maximum and leaves it in LDS,
            // and adds up, in the waves' order, a quarter of the dims.
            __syncthreads();   // LDS is free
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                l[c] = sum_x32(sum_x16(l[c]));
                le[c] = sum_x32(sum_x16(le[c])) * (1.0f / (1 << UP));
                if (g == 0) lds_ml[(wave * NT + c) * 16 + n] = floatx4{m[c], l[c], le[c], 0.0f};
            }
            __syncthreads();
            float inv[NT];
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                floatx4 ml[AR_WAVES];
                float top = kNegInf;
#pragma unroll
                for (int w = 0; w < AR_WAVES; ++w) {
                    ml[w] = lds_ml[(w * NT + c) * 16 + n];
                    top = fmaxf(top, ml[w][0]);
                }
                const float ms = top == kNegInf ? 0.0f : top;
                l[c] = le[c] = 0.0f;
#pragma unroll
                for (int w = 0; w < AR_WAVES; ++w) {
                    const float f = __builtin_amdgcn_exp2f(ml[w][0] - ms);
                    l[c] += ml[w][1] * f;
                    le[c] += ml[w][2] * f;
                }
                if (over) l[c] = le[c] = __builtin_nanf("");
                const float f = __builtin_amdgcn_exp2f(m[c] - ms);
                m[c] = top;
                inv[c] = a.nsplit > 1 ? 1.0f : l[c] != 0.0f ? 1.0f / l[c] : 0.0f;   // no key seen: 0
#pragma unroll
                for (int d = 0; d < ND; ++d) lds_o[((wave * NT + c) * ND + d) * 64 + lane] = o[c][d] * f;
            }
            __syncthreads();
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                const int r = r0 + 16 * c + n;
                if (r >= rows) continue;
                const int t = a.by_g.div(r), hq = h * a.G + (r - t * a.G);
                const long row = (tok0 + t) * s.hq + hq, at = row * a.nsplit + split;
#pragma unroll
                for (int dd = 0; dd < ND / AR_WAVES; ++dd) {
                    const int d = wave * (ND / AR_WAVES) + dd;
                    floatx4 y = lds_o[(c * ND + d) * 64 + lane];
#pragma unroll
                    for (int w = 1; w < AR_WAVES; ++w) y += lds_o[((w * NT + c) * ND + d) * 64 + lane];
                    if (over) y = floatx4{l[c], l[c], l[c], l[c]};
                    if (a.nsplit == 1) {
                        u32x2 w;
                        w[0] = Tr<T>::pk(y[0] * inv[c], y[1] * inv[c]);
                        w[1] = Tr<T>::pk(y[2] * inv[c], y[3] * inv[c]);
                        *reinterpret_cast<u32x2*>((T*)a.out + row * D + 16 * d + 4 * g) = w;
                    } else if (l[c] != 0.0f) {
                        *reinterpret_cast<floatx4*>(a.part_o + at * D + 16 * d + 4 * g) = y;
                    }
                }
                if (wave == 0 && g == 0) {
                    if (a.nsplit > 1) a.part_ml[at] = floatx4{m[c], l[c], le[c], 0.0f};
                    else if (a.lse) a.lse[row] = (m[c] + __builtin_amdgcn_logf(le[c])) * (1.0f / kLog2e);
                }
            }
        }
    }
}

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

template <class T, int D, int NT, int MODE>
static hipError_t launch_rows(const AttnArgs& a, hipStream_t st)
{
    static std::atomic<unsigned long long> done{0};
    const int lds = AR_WAVES * NT * (D / 16 * 64 + 16) * 16;
    hipError_t e = allow_full_lds((const void*)k_attn_rows<T, D, NT, MODE>, &done);
    if (e != hipSuccess) return e;
    const long rows = (long)(a.s.max_q > 0 ? a.s.max_q : 1) * a.G;
    long rb = (rows + 16 * NT - 1) / (16 * NT);
    if (rb * a.s.hkv > 65535) rb = 65535 / a.s.hkv;
    // Sequences fastest, splits slowest: workgroups go round-robin over the 8 XCDs, and with the
    // splits fastest a power of two of them put the later ones, which only long sequences have,
    // on the same XCDs (256 sequences of 170 - 500 keys, 8 splits: 121 us, against 52 with 6).
    const dim3 grid(a.s.batch, (unsigned)(rb * a.s.hkv), a.nsplit);
    k_attn_rows<T, D, NT, MODE><<<grid, dim3(64 * AR_WAVES), lds, st>>>(a, (int)rb);
    return hipGetLastError();
}

template <class T, int D, int MODE>
static hipError_t rows_tiles(const AttnArgs& a, hipStream_t st)
{
    return (long)a.s.max_q * a.G > 16 ? launch_rows<T, D, 2, MODE>(a, st) : launch_rows<T, D, 1, MODE>(a, st);
}

template <class T, int D>
static hipError_t pick_rows(const AttnArgs& a, hipStream_t st)
{
    return by_kind(a, [&](auto k) { return rows_tiles<T, D, decltype(k)::value>(a, st); });
}

template <class T>
static hipError_t rows_by_d(const AttnArgs& a, hipStream_t st)
{
    switch (a.s.d) {
    case 64: return pick_rows<T, 64>(a, st);
    case 128: return pick_rows<T, 128>(a, st);
    case 192: return pick_rows<T, 192>(a, st);
    default: return pick_rows<T, 256>(a, st);
    }
}

hipError_t run_attn_rows(int dtype, const AttnArgs& a, hipStream_t st)
{
    return dtype == DT_F16 ? rows_by_d<half_t>(a, st) : rows_by_d<bf16_t>(a, st);
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

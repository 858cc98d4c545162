// attn_rows.hip -- attention over the paged 8-bit cache for few rows (the
// queries of one step): k_attn_rows, and the join of split results,
// k_attn_join.
//
// A chain of two products whose intermediate stays in registers: a wave takes
// 64 keys at a time, S^T = K q^T (rows = keys, columns = query rows, MFMA
// 16x16x32), the softmax of a column lives in the four lanes that hold it (the
// running maximum and sum in 32 bits), and the weights, rounded once to the
// activations' type, are the second product's operand B in the lanes that
// already hold them: O^T += V^T p^T.  For that the 16 keys of accumulator rows
// 4g .. 4g + 3 of the four tiles are the 16 tokens of one cache block: tile t,
// row 4g + i <-> key 16g + 4t + i.
//
// Bound by the cache's bytes: every code is read once, 16 bytes a lane, by one
// wave.  The keys are split over a block's waves, and over blocks where
// sequences x heads alone do not fill the machine; the waves' results are
// joined through LDS and the blocks' by k_attn_join, both in a fixed order.
#include "fc_launch.h"
#include "kv_common.h"

namespace fc {

constexpr int AR_WAVES = 4;

template <class T, int D, int NT, bool CAP>
__global__ __launch_bounds__(64 * AR_WAVES) void k_attn_rows(AttnArgs a, int row_blocks)
{
    typedef typename Tr<T>::v8 v8;
    constexpr int R = 16 * NT;       // rows a block
    constexpr int NJ = D / 64;       // 16-byte loads of K a lane and tile
    constexpr int ND = D / 16;       // tiles of V^T
    const KvShape& s = a.s;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = lane & 15, g = lane >> 4;
    const int h = blockIdx.y / row_blocks, rb0 = blockIdx.y % row_blocks, split = blockIdx.x;

    extern __shared__ __align__(16) float lds[];
    if constexpr (kPoison) {
        lds_poison((FC_LDS float*)lds, 2 * NT * (D / 4 + 2) * 64 * 4, threadIdx.x, 64 * AR_WAVES);
        __syncthreads();
    }

    for (int b = blockIdx.z; b < s.batch; b += gridDim.z) {
        long tok0;
        int nq;
        seq_range(a.cu_q, s, b, &tok0, &nq);
        const int rows = nq * a.G;
        bool over;
        const int kv_len = seq_keys(a.kv_lens, s, b, &over), pos0 = kv_len - nq;
        for (int r0 = rb0 * R; r0 < rows; r0 += row_blocks * R) {
            const int r1 = r0 + R < rows ? r0 + R : rows;
            const int t_first = a.by_g.div(r0), t_last = a.by_g.div(r1 - 1);
            int g_lo, g_hi;
            key_range(a, kv_len, pos0, t_first, t_last, &g_lo, &g_hi);

            // this lane's rows: query, position, keys [lo, hi) that it sees
            int hi[NT], lo[NT];
            float slope[NT], posf[NT];
            v8 qf[NT][2 * NJ];
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                const int r = r0 + 16 * c + n, rr = r < rows ? r : rows - 1;
                const int t = a.by_g.div(rr), hq = h * a.G + (rr - t * a.G), pos = pos0 + t;
                hi[c] = a.causal ? (pos + 1 < kv_len ? pos + 1 : kv_len) : kv_len;
                lo[c] = a.window > 0 ? pos - a.window + 1 : 0;
                slope[c] = a.slopes ? a.slopes[hq] * kLog2e : 0.0f;
                posf[c] = (float)pos;
                const T* q = (const T*)a.q + (tok0 + t) * a.q_ts + (long)hq * a.q_hs;
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        qf[c][2 * j + e] = *reinterpret_cast<const v8*>(q + 16 * (4 * j + g) + 8 * e);
            }
            // keys that every row of the tile sees need no mask
            const int all_lo = a.window > 0 ? pos0 + t_last - a.window + 1 : 0;
            const int all_hi = a.causal ? (pos0 + t_first + 1 < kv_len ? pos0 + t_first + 1 : kv_len) : kv_len;

            floatx4 o[NT][ND];
            float m[NT], l[NT];
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                m[c] = kNegInf;
                l[c] = 0.0f;
#pragma unroll
                for (int d = 0; d < ND; ++d) o[c][d] = floatx4{0, 0, 0, 0};
            }

            for (int c0 = g_lo + split * a.chunk; c0 < g_hi; c0 += a.nsplit * a.chunk) {
                const int c1 = c0 + a.chunk < g_hi ? c0 + a.chunk : g_hi;
                for (int k0 = c0 + 4 * wave; k0 < c1; k0 += 4 * AR_WAVES) {
                    // the blocks of this lane: K rows of block n >> 2, scores and V of block g
                    const int gk = k0 + (n >> 2) < c1 ? k0 + (n >> 2) : c1 - 1;
                    const int gv = k0 + g < c1 ? k0 + g : c1 - 1;
                    const int pk = gk >> a.pg_shift, pv = gv >> a.pg_shift;
                    const int idk = page_id(a.table, s, b, pk), idv = page_id(a.table, s, b, pv);
                    const uint8_t* kb = a.codes + side_base(idk < 0 ? 0 : idk, h, 0, s) + (gk - (pk << a.pg_shift)) * (16 * D) +
                                        g * 256 + (n & 3) * 16;
                    const uint8_t* vb = a.codes + side_base(idv < 0 ? 0 : idv, h, 1, s) + (gv - (pv << a.pg_shift)) * (16 * D) +
                                        n * 16;
                    u32x4 kr[4][NJ], vr[ND];
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int j = 0; j < NJ; ++j) kr[t][j] = *reinterpret_cast<const u32x4*>(kb + j * 1024 + t * 64);
#pragma unroll
                    for (int d = 0; d < ND; ++d) vr[d] = *reinterpret_cast<const u32x4*>(vb + d * 256);
                    const float* sc = a.scales + ((size_t)(idv < 0 ? 0 : idv) * s.hkv + h) * 2;
                    float ks = sc[0], vs = sc[1];
                    if (idv < 0) {   // a page outside the pool: every row that sees its keys turns NaN
                        ks = __builtin_nanf("");
                        vs = 1.0f;
                    }

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
                    const float c0s = CAP ? 2.0f * kLog2e * ks * a.scale / a.cap : ks * a.scale * kLog2e;
                    const float c1s = a.cap * kLog2e;
                    const int key0 = (k0 + g) * 16;
                    const bool masked = k0 * 16 < all_lo || (k0 + 4) * 16 > all_hi || k0 + 4 > c1;
                    v8 pf[NT][2];
#pragma unroll
                    for (int c = 0; c < NT; ++c) {
                        float x[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] = score<CAP>(st[c][i >> 2][i & 3], c0s, c1s);
                        if (a.slopes) {
                            const float gap = posf[c] - (float)key0;
#pragma unroll
                            for (int i = 0; i < 16; ++i) x[i] -= slope[c] * fabsf(gap - (float)i);
                        }
                        if (masked) {
                            const int top = hi[c] < c1 * 16 ? hi[c] : c1 * 16;
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                x[i] = key0 + i < top && key0 + i >= lo[c] ? x[i] : kNegInf;
                        }
                        float mx = x[0];
#pragma unroll
                        for (int i = 1; i < 16; ++i) mx = fmaxf(mx, x[i]);
                        mx = max_x32(max_x16(mx));
                        const float mn = fmaxf(m[c], mx);
                        const float ms = mn == kNegInf ? 0.0f : mn;   // nothing seen yet: all weights are 0
                        const float alpha = __builtin_amdgcn_exp2f(m[c] - ms);
                        m[c] = mn;
                        float sum = 0.0f;
                        u32x4 w[2];
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const float p0 = __builtin_amdgcn_exp2f(x[i] - ms), p1 = __builtin_amdgcn_exp2f(x[i + 1] - ms);
                            sum += p0 + p1;
                            w[i >> 3][(i >> 1) & 3] = Tr<T>::pk(p0, p1);
                        }
                        l[c] = l[c] * alpha + sum;
#pragma unroll
                        for (int d = 0; d < ND; ++d) o[c][d] *= alpha;
                        pf[c][0] = __builtin_bit_cast(v8, w[0]);
                        pf[c][1] = __builtin_bit_cast(v8, w[1]);
                    }
                    // tokens past the end hold whatever the page held: their weight is 0, and
                    // 0 times a NaN code is NaN, so their codes are cleared
                    if ((k0 + 4) * 16 > kv_len || __any(idv < 0)) {
                        const int keep = idv < 0 ? 0 : kv_len - key0;
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
                }
            }
#pragma unroll
            for (int c = 0; c < NT; ++c) l[c] = over ? __builtin_nanf("") : sum_x32(sum_x16(l[c]));

            // join the waves: waves 2, 3 hand theirs to 0, 1, then 1 to 0
            constexpr int PW = NT * (ND * 4 + 2) * 64;   // floats a wave hands over
#pragma unroll
            for (int half = AR_WAVES / 2; half; half >>= 1) {
                __syncthreads();
                if (wave >= half && wave < 2 * half) {
                    float* w = lds + (wave - half) * PW + lane;
#pragma unroll
                    for (int c = 0; c < NT; ++c) {
                        w[(c * 2) * 64] = m[c];
                        w[(c * 2 + 1) * 64] = l[c];
#pragma unroll
                        for (int d = 0; d < ND; ++d)
#pragma unroll
                            for (int i = 0; i < 4; ++i) w[(NT * 2 + (c * ND + d) * 4 + i) * 64] = o[c][d][i];
                    }
                }
                __syncthreads();
                if (wave < half) {
                    const float* w = lds + wave * PW + lane;
#pragma unroll
                    for (int c = 0; c < NT; ++c) {
                        const float m2 = w[(c * 2) * 64], l2 = w[(c * 2 + 1) * 64];
                        const float mn = fmaxf(m[c], m2), ms = mn == kNegInf ? 0.0f : mn;
                        const float f1 = __builtin_amdgcn_exp2f(m[c] - ms), f2 = __builtin_amdgcn_exp2f(m2 - ms);
                        m[c] = mn;
                        l[c] = l[c] * f1 + l2 * f2;
#pragma unroll
                        for (int d = 0; d < ND; ++d)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                o[c][d][i] = o[c][d][i] * f1 + w[(NT * 2 + (c * ND + d) * 4 + i) * 64] * f2;
                    }
                }
            }
            if (wave == 0) {
#pragma unroll
                for (int c = 0; c < NT; ++c) {
                    const int r = r0 + 16 * c + n;
                    if (r >= rows) continue;
                    const int t = a.by_g.div(r), hq = h * a.G + (r - t * a.G);
                    const long row = (tok0 + t) * s.hq + hq;
                    if (a.nsplit == 1) {
                        const float inv = l[c] != 0.0f ? 1.0f / l[c] : 0.0f;   // no key seen: 0
                        T* out = (T*)a.out + row * D;
#pragma unroll
                        for (int d = 0; d < ND; ++d) {
                            u32x2 w;
                            w[0] = Tr<T>::pk(o[c][d][0] * inv, o[c][d][1] * inv);
                            w[1] = Tr<T>::pk(o[c][d][2] * inv, o[c][d][3] * inv);
                            *reinterpret_cast<u32x2*>(out + 16 * d + 4 * g) = w;
                        }
                        if (a.lse && g == 0) a.lse[row] = (m[c] + __builtin_amdgcn_logf(l[c])) * (1.0f / kLog2e);
                    } else {
                        const long at = row * a.nsplit + split;
                        if (l[c] != 0.0f) {
#pragma unroll
                            for (int d = 0; d < ND; ++d)
                                *reinterpret_cast<floatx4*>(a.part_o + at * D + 16 * d + 4 * g) = o[c][d];
                        }
                        if (g == 0) {
                            a.part_ml[at * 2] = m[c];
                            a.part_ml[at * 2 + 1] = l[c];
                        }
                    }
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
    __shared__ float part[WPR > 1 ? WPR - 1 : 1][5][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, w = wave % WPR, D = a.s.d;
    const long row = (long)blockIdx.x * (4 / WPR) + wave / WPR;
    const bool live = row < rows;
    const floatx2* ml = reinterpret_cast<const floatx2*>(a.part_ml) + (live ? row : 0) * a.nsplit;
    float m = kNegInf;
    for (int k = lane; k < a.nsplit; k += 64) m = fmaxf(m, ml[k][0]);
#pragma unroll
    for (int s = 32; s; s >>= 1) m = fmaxf(m, __shfl_xor(m, s));
    const float ms = m == kNegInf ? 0.0f : m;
    float l = 0.0f, o[4] = {0, 0, 0, 0};
    const float* p = a.part_o + (live ? row : 0) * a.nsplit * D + lane;
#pragma unroll 4
    for (int k = w; k < a.nsplit; k += WPR) {
        const floatx2 v = ml[k];
        const float f = __builtin_amdgcn_exp2f(v[0] - ms);
        const bool some = v[1] != 0.0f;
        l += some ? v[1] * f : 0.0f;
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
        }
        __syncthreads();
        if (w > 0) return;
#pragma unroll
        for (int j = 0; j < WPR - 1; ++j) {
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] += part[j][i][lane];
            l += part[j][4][lane];
        }
    }
    if (!live) return;
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
    T* out = (T*)a.out + row * D;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i * 64 < D) out[i * 64 + lane] = (T)(o[i] * inv);
    if (a.lse && lane == 0) a.lse[row] = (m + __builtin_amdgcn_logf(l)) * (1.0f / kLog2e);
}

template <class T, int D, int NT, bool CAP>
static hipError_t launch_rows(const AttnArgs& a, hipStream_t st)
{
    static std::atomic<unsigned long long> done{0};
    const int lds = 2 * NT * (D / 4 + 2) * 64 * 4;
    hipError_t e = allow_full_lds((const void*)k_attn_rows<T, D, NT, CAP>, &done);
    if (e != hipSuccess) return e;
    const long rows = (long)(a.s.max_q > 0 ? a.s.max_q : 1) * a.G;
    long rb = (rows + 16 * NT - 1) / (16 * NT);
    if (rb * a.s.hkv > 65535) rb = 65535 / a.s.hkv;
    const dim3 grid(a.nsplit, (unsigned)(rb * a.s.hkv), a.s.batch < 65535 ? a.s.batch : 65535);
    k_attn_rows<T, D, NT, CAP><<<grid, dim3(64 * AR_WAVES), lds, st>>>(a, (int)rb);
    return hipGetLastError();
}

template <class T, int D>
static hipError_t pick_rows(const AttnArgs& a, hipStream_t st)
{
    const bool two = (long)a.s.max_q * a.G > 16;
    if (a.cap > 0.0f) return two ? launch_rows<T, D, 2, true>(a, st) : launch_rows<T, D, 1, true>(a, st);
    return two ? launch_rows<T, D, 2, false>(a, st) : launch_rows<T, D, 1, false>(a, st);
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
    if (a.nsplit > 8) k_attn_join<T, 4><<<dim3((unsigned)rows), dim3(256), 0, st>>>(a, rows);
    else k_attn_join<T, 1><<<dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, st>>>(a, rows);
    return hipGetLastError();
}

hipError_t run_attn_join(int dtype, const AttnArgs& a, hipStream_t st)
{
    return dtype == DT_F16 ? launch_join<half_t>(a, st) : launch_join<bf16_t>(a, st);
}

}  // namespace fc

// attn_tile.hip -- attention over the paged 8-bit cache for many rows (prompts
// and chunks of them): k_attn_tile.
//
// The same chain as k_attn_rows with 32x32x16 matrix instructions.  A block
// owns 32 * NW rows (queries x the heads that share a kv head), a wave 32 of
// them, a lane one column: S^T = K q^T, the softmax of a row in one lane and
// its partner l ^ 32 (running maximum and sum in 32 bits), and p, rounded once
// to the activations' type, straight from the accumulators into operand B of
// O^T += V^T p^T.  Accumulator row 8b + 4h + i of lane half h is key 16h + 4b
// + i of a 32-key subtile, so that a half's 16 keys are one cache block and
// its V operand is 16 consecutive bytes.
//
// Codes go to LDS as they are (8 bits), 64 keys a stage by LDS-DMA, the next
// stage in flight during a stage's products; a wave widens them in registers
// as operands.  The blocks of 16 keys sit 16 * D + 128 bytes apart, so that the
// 16 lanes of a fragment read that straddle two blocks meet all 64 banks.
#include "fc_dma.h"
#include "fc_launch.h"
#include "kv_common.h"

namespace fc {

typedef FC_LDS uint8_t lds_u8;
typedef __attribute__((address_space(4))) const int const_int;
typedef __attribute__((address_space(4))) const float const_float;

template <class T, int D, int NW, bool CAP>
__global__ __launch_bounds__(64 * NW, D <= 128 ? 2 : 1) void k_attn_tile(AttnArgs a, int row_tiles)
{
    typedef typename Tr<T>::v8 v8;
    constexpr int GB = 16 * D + 128;       // bytes from block to block of 16 keys in LDS
    constexpr int STAGE = 8 * GB;          // 4 blocks of K, 4 of V
    constexpr int NJ = D / 32, ND = D / 32, NP = D / 64;
    static_assert(NW == 4 || NW == 8, "a wave fetches a whole block of 16 keys or one side of it");
    const KvShape& s = a.s;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 31, hf = lane >> 5;
    const int h = blockIdx.y, split = blockIdx.x % a.nsplit;
    const int rt0 = row_tiles - 1 - (int)(blockIdx.x / a.nsplit);   // long rows (causal) first

    __shared__ __align__(16) uint8_t buf[2 * STAGE];
    __shared__ float sc_lds[2][4][2];
    lds_u8* const lb = (lds_u8*)buf;
    if constexpr (kPoison) {
        lds_poison(lb, 2 * STAGE, threadIdx.x, 64 * NW);
        __syncthreads();
    }

    for (int b = blockIdx.z; b < s.batch; b += gridDim.z) {
        long tok0;
        int nq;
        seq_range(a.cu_q, s, b, &tok0, &nq);
        const int rows = nq * a.G;
        bool over;
        const int kv_len = seq_keys(a.kv_lens, s, b, &over), pos0 = kv_len - nq;
        for (int r0 = rt0 * 32 * NW; r0 < rows; r0 += row_tiles * 32 * NW) {
            const int r1 = r0 + 32 * NW < rows ? r0 + 32 * NW : rows;
            int g_lo, g_hi;
            key_range(a, kv_len, pos0, a.by_g.div(r0), a.by_g.div(r1 - 1), &g_lo, &g_hi);
            // this wave's rows
            const int w0 = r0 + 32 * wave, w1 = w0 + 32 < rows ? w0 + 32 : rows;
            const bool live = w0 < rows;
            const int t_first = a.by_g.div(live ? w0 : r0), t_last = a.by_g.div(live ? w1 - 1 : r0);
            int wg_lo, wg_hi;
            key_range(a, kv_len, pos0, t_first, t_last, &wg_lo, &wg_hi);
            const int all_lo = a.window > 0 ? pos0 + t_last - a.window + 1 : 0;
            const int all_hi = a.causal ? (pos0 + t_first + 1 < kv_len ? pos0 + t_first + 1 : kv_len) : kv_len;
            // this lane's row
            const int r = w0 + n, rr = r < rows ? r : rows - 1;
            const int t = a.by_g.div(rr), hq = h * a.G + (rr - t * a.G), pos = pos0 + t;
            const int hi = a.causal ? (pos + 1 < kv_len ? pos + 1 : kv_len) : kv_len;
            const int lo = a.window > 0 ? pos - a.window + 1 : 0;
            const float slope = a.slopes ? a.slopes[hq] * kLog2e : 0.0f, posf = (float)pos;
            v8 qf[2 * NJ];
            {
                const T* q = (const T*)a.q + (tok0 + t) * a.q_ts + (long)hq * a.q_hs;
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) qf[2 * j + e] = *reinterpret_cast<const v8*>(q + 16 * (2 * j + hf) + 8 * e);
            }
            floatx16 o[ND];
#pragma unroll
            for (int d = 0; d < ND; ++d) o[d] = zero16();
            float m = kNegInf, l = 0.0f;

            const int per_page = s.page >> 4;
            for (int c0 = g_lo + split * a.chunk; c0 < g_hi; c0 += a.nsplit * a.chunk) {
                const int c1 = c0 + a.chunk < g_hi ? c0 + a.chunk : g_hi;
                // requests of this wave for the stage that begins at block k0
                auto fetch = [&](int k0, int stage) {
                    const int gi = NW == 4 ? wave : wave >> 1;
                    const int gk = k0 + gi < c1 ? k0 + gi : c1 - 1;
                    const int pg = gk / per_page;
                    int id = -1;
                    if ((unsigned)pg < (unsigned)s.table_stride) id = ((const_int*)a.table)[(size_t)b * s.table_stride + pg];
                    const bool ok = (unsigned)id < (unsigned)s.pages;
                    id = ok ? id : 0;
                    const int inpage = (gk - pg * per_page) * (16 * D);
#pragma unroll
                    for (int sd = 0; sd < 2; ++sd) {
                        if (NW == 8 && sd != (wave & 1)) continue;
                        const i32x4 rs = buf_rsrc(a.codes + side_base(id, h, sd, s) + inpage, ok ? 16 * D : 0);   // none: zeros
                        lds_u8* dst = lb + stage * STAGE + (sd * 4 + gi) * GB;
#pragma unroll
                        for (int p = 0; p < NP; ++p) {
                            if (kPoison) dma16(buf_rsrc(&fc_poison_line, 1024), lane * 16, (const lds_half*)(dst + p * 1024));
                            dma16(rs, p * 1024 + lane * 16, (const lds_half*)(dst + p * 1024));
                        }
                        const float v = ((const_float*)a.scales)[((size_t)id * s.hkv + h) * 2 + sd];
                        // a page outside the pool: every row that sees its keys turns NaN
                        if (lane == 0) sc_lds[stage][gi][sd] = ok ? v : (sd ? 1.0f : __builtin_nanf(""));
                    }
                };
                __syncthreads();   // the buffers are free
                fetch(c0, 0);
                for (int k0 = c0, stage = 0; k0 < c1; k0 += 4, stage ^= 1) {
                    vm_wait<0>();
                    __syncthreads();   // this stage has arrived, and every wave is done with the other one
                    if (k0 + 4 < c1) fetch(k0 + 4, stage ^ 1);
                    if (!live || k0 >= wg_hi || k0 + 4 <= wg_lo) continue;
                    const lds_u8* kb = lb + stage * STAGE + ((n >> 2) & 1) * GB + (4 * (n >> 3) + (n & 3)) * 16 + hf * 256;
                    const lds_u8* vb = lb + stage * STAGE + (4 + hf) * GB + n * 16;
                    float x[32];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        floatx16 acc = zero16();
#pragma unroll
                        for (int j = 0; j < NJ; ++j) {
                            const u32x4 w = *reinterpret_cast<const FC_LDS u32x4*>(kb + 2 * u * GB + j * 512);
                            acc = Tr<T>::mfma32(frag8<T>(w[0], w[1], 1.0f), qf[2 * j], acc);
                            acc = Tr<T>::mfma32(frag8<T>(w[2], w[3], 1.0f), qf[2 * j + 1], acc);
                        }
                        const float ks = sc_lds[stage][2 * u + hf][0];
                        const float c0s = CAP ? 2.0f * kLog2e * ks * a.scale / a.cap : ks * a.scale * kLog2e;
                        const float c1s = a.cap * kLog2e;
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[16 * u + i] = score<CAP>(acc[i], c0s, c1s);
                    }
                    const int key0 = k0 * 16 + 16 * hf;
                    if (a.slopes) {
                        const float gap = posf - (float)key0;
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] -= slope * fabsf(gap - (float)((i >> 4) * 32 + (i & 15)));
                    }
                    if (k0 * 16 < all_lo || (k0 + 4) * 16 > all_hi || k0 + 4 > c1) {
                        const int top = hi < c1 * 16 ? hi : c1 * 16;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const int key = key0 + (i >> 4) * 32 + (i & 15);
                            x[i] = key < top && key >= lo ? x[i] : kNegInf;
                        }
                    }
                    float mx = x[0];
#pragma unroll
                    for (int i = 1; i < 32; ++i) mx = fmaxf(mx, x[i]);
                    mx = max_x32(mx);
                    const float mn = fmaxf(m, mx), ms = mn == kNegInf ? 0.0f : mn;
                    const float alpha = __builtin_amdgcn_exp2f(m - ms);
                    m = mn;
                    float sum = 0.0f;
                    u32x4 w[4];
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float p0 = __builtin_amdgcn_exp2f(x[i] - ms), p1 = __builtin_amdgcn_exp2f(x[i + 1] - ms);
                        sum += p0 + p1;
                        w[i >> 3][(i >> 1) & 3] = Tr<T>::pk(p0, p1);
                    }
                    l = l * alpha + sum;
#pragma unroll
                    for (int d = 0; d < ND; ++d) o[d] *= alpha;
                    const bool tail = (k0 + 4) * 16 > kv_len;
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const float vs = sc_lds[stage][2 * u + hf][1];
                        u32x4 mk = {~0u, ~0u, ~0u, ~0u};
                        if (tail) {   // tokens past the end: weight 0, but their codes may be NaN
                            const int keep = kv_len - key0 - 32 * u;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int k = keep - 4 * j;
                                mk[j] = k >= 4 ? ~0u : (k <= 0 ? 0u : (1u << (8 * k)) - 1u);
                            }
                        }
#pragma unroll
                        for (int d = 0; d < ND; ++d) {
                            u32x4 c = *reinterpret_cast<const FC_LDS u32x4*>(vb + 2 * u * GB + d * 512);
                            if (tail) c &= mk;
                            o[d] = Tr<T>::mfma32(frag8<T>(c[0], c[1], vs), __builtin_bit_cast(v8, w[2 * u]), o[d]);
                            o[d] = Tr<T>::mfma32(frag8<T>(c[2], c[3], vs), __builtin_bit_cast(v8, w[2 * u + 1]), o[d]);
                        }
                    }
                }
            }
            l = over ? __builtin_nanf("") : sum_x32(l);
            if (r < rows) {
                const long row = (tok0 + t) * s.hq + hq;
                if (a.nsplit == 1) {
                    const float inv = l != 0.0f ? 1.0f / l : 0.0f;   // no key seen: 0
                    T* out = (T*)a.out + row * D + 4 * hf;
#pragma unroll
                    for (int d = 0; d < ND; ++d)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            u32x2 w;
                            w[0] = Tr<T>::pk(o[d][4 * k] * inv, o[d][4 * k + 1] * inv);
                            w[1] = Tr<T>::pk(o[d][4 * k + 2] * inv, o[d][4 * k + 3] * inv);
                            *reinterpret_cast<u32x2*>(out + 32 * d + 8 * k) = w;
                        }
                    if (a.lse && hf == 0) a.lse[row] = (m + __builtin_amdgcn_logf(l)) * (1.0f / kLog2e);
                } else {
                    const long at = row * a.nsplit + split;
                    if (l != 0.0f) {
                        float* out = a.part_o + at * D + 4 * hf;
#pragma unroll
                        for (int d = 0; d < ND; ++d)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                *reinterpret_cast<floatx4*>(out + 32 * d + 8 * k) =
                                    floatx4{o[d][4 * k], o[d][4 * k + 1], o[d][4 * k + 2], o[d][4 * k + 3]};
                    }
                    if (hf == 0) {
                        a.part_ml[at * 2] = m;
                        a.part_ml[at * 2 + 1] = l;
                    }
                }
            }
        }
    }
}

template <class T, int D, bool CAP>
static hipError_t launch_tile(const AttnArgs& a, hipStream_t st)
{
    constexpr int NW = 4;
    const long rows = (long)(a.s.max_q > 0 ? a.s.max_q : 1) * a.G;
    long rt = (rows + 32 * NW - 1) / (32 * NW);
    if (rt * a.nsplit > 0x7fffffffL) rt = 0x7fffffffL / a.nsplit;
    const dim3 grid((unsigned)(rt * a.nsplit), a.s.hkv, a.s.batch < 65535 ? a.s.batch : 65535);
    k_attn_tile<T, D, NW, CAP><<<grid, dim3(64 * NW), 0, st>>>(a, (int)rt);
    return hipGetLastError();
}

template <class T>
static hipError_t tile_by_d(const AttnArgs& a, hipStream_t st)
{
    const bool cap = a.cap > 0.0f;
    switch (a.s.d) {
    case 64: return cap ? launch_tile<T, 64, true>(a, st) : launch_tile<T, 64, false>(a, st);
    case 128: return cap ? launch_tile<T, 128, true>(a, st) : launch_tile<T, 128, false>(a, st);
    case 192: return cap ? launch_tile<T, 192, true>(a, st) : launch_tile<T, 192, false>(a, st);
    default: return cap ? launch_tile<T, 256, true>(a, st) : launch_tile<T, 256, false>(a, st);
    }
}

hipError_t run_attn_tile(int dtype, const AttnArgs& a, hipStream_t st)
{
    return dtype == DT_F16 ? tile_by_d<half_t>(a, st) : tile_by_d<bf16_t>(a, st);
}

}  // namespace fc

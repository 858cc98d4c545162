// attn_tile.hip -- attention over the paged 8-bit cache for many rows (prompts
// and chunks of them): k_attn_tile.
//
// The same chain as k_attn_rows with 32x32x16 matrix instructions.  A block
// owns 32 * NW rows (queries x the heads that share a kv head), a wave 32 of
// them, a lane one column: S^T = K q^T, the softmax of a row in one lane and
// its partner l ^ 32 (running maximum and sum in 32 bits), and p, rounded once
// to the activations' type, straight from the accumulators into operand B of
// O^T += V^T p^T.  Accumulator row 8b + 4h + i of lane half h is key 16h + 4b
// + i of a 32-key subtile, so that a half's 16 keys are one cache block.
//
// Keys pass through LDS 64 a stage, widened once for the whole block: a wave
// loads its share of the codes two stages ahead, widens it (times the page's
// scale, which is exact) and writes it in operand order while the block
// computes the stage before.  Every wave widening its own operands from 8-bit
// codes in LDS, as this kernel first did, cost 128 of ~430 vector instructions
// a wave and stage.
//
// Bound by the two pipes of a SIMD together: a wave and stage of d = 128 is 1024
// cycles of matrix instructions and about 800 of vector ones (32 exponentials, at
// 8 cycles, are a third of these), two waves a SIMD fill each other's gaps, and
// the clock sinks under the load.  Measured for two prompts of 4096 with 32 query
// heads of 128: 271 to 304 us by card (906 to 1015 TFLOP/s; a library product of
// 8192^3 reaches 1170 to 1300); without the exponentials, the widening and the
// maximum the same loop still takes 227.  Two prompts of 4096 with other heads: 32
// of 64, where the vector pipe is the longer one, 188 to 198 us; with a cap 253 to
// 276 (three slow operations a score for one), with a bias 214 to 229 (172 registers
// leave a SIMD two waves, plain and capped scores three); 16 of 192 217 to 226; 16 of
// 256 318 to 347 (queries and accumulators are 192 of 256 registers, 25 to 40 are
// spilled); 32 of 128 with a cap 351 to 367.  lse takes every exponential twice: 352
// us against 293 (d = 128), 152 against 120 for chunks with a bias.
#include "fc_launch.h"
#include "kv_common.h"

namespace fc {

typedef FC_LDS uint8_t lds_u8;

// Waves a block and blocks of 16 keys a stage.  Heads of 192 and 256 leave a SIMD
// room for two waves only if a block of eight shares the widening (d = 192: 220
// us, against 401 with four waves of 512 registers, for two prompts of 4096 and
// 16 heads), and of 256 only with stages of 32 keys (355 us against 518 with 64,
// whose scores spill).
__host__ __device__ constexpr int tile_waves(int d) { return d <= 128 ? 4 : 8; }
__host__ __device__ constexpr int tile_blocks(int d) { return d <= 192 ? 4 : 2; }

template <class T, int D, int NW, int MODE>
__global__ __launch_bounds__(64 * NW, 2) void k_attn_tile(AttnArgs a, int row_tiles)
{
    typedef typename Tr<T>::v8 v8;
    constexpr int BR = 32 * NW;              // rows a block
    constexpr int KB = tile_blocks(D), U = KB / 2;   // blocks of 16 keys a stage, subtiles of 32
    constexpr int SIDE = 16 * KB * D * 2;    // bytes of a stage's keys (or values), 16 bits each
    constexpr int STAGE = 2 * SIDE;
    constexpr int NK = D / 16, ND = D / 32, NP = D / 64;
    constexpr int PW = 2 * KB * NP / NW;     // pieces of 1 KiB of codes a wave and stage
    static_assert(2 * KB * NP % NW == 0 && 2 * NP % PW == 0, "a wave's pieces are of one block");
    constexpr int AH = D == 64 ? 4 : 2;   // operands read ahead (d = 64 with a bias: 126 us, with two 152)
    constexpr int LAG = 8, UP = Tr<T>::up > LAG ? Tr<T>::up - LAG : 0;   // weights are at most 2^(LAG + UP)
    const KvShape& s = a.s;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 31, hf = lane >> 5;
    const int h = blockIdx.x, split = blockIdx.y / row_tiles;
    const int rt0 = row_tiles - 1 - (int)(blockIdx.y % row_tiles);   // long rows (causal) first

    extern __shared__ __align__(16) uint8_t buf[];
    lds_u8* const lb = (lds_u8*)buf;
    if constexpr (kPoison) {
        lds_poison(lb, 2 * STAGE, threadIdx.x, 64 * NW);
        __syncthreads();
    }
    global_u8* no_page = global_at(&fc_no_page);
    asm("" : "+s"(no_page));   // the address is taken once, not by a load in every stage
    // This wave's share of a stage: PW pieces of one of its blocks.  A
    // K row of 16 dims of a token goes to row m of the operand; the swap of
    // fours in every other row lets a write meet all the banks.
    const int blk = wave * PW / (2 * NP), piece0 = wave * PW % (2 * NP);   // piece: side * NP + p
    const int tok = lane & 15;
    const int k_to = (blk >> 1) * (SIDE / U) + (lane >> 4) * 1024 +
                     ((8 * (tok >> 2) + 4 * (blk & 1) + (tok & 3)) ^ (4 * ((lane >> 4) & 1))) * 16;
    const int v_to = SIDE + ((blk >> 1) * 4 + (blk & 1)) * (16 * D) + lane * 16;
    const int k_at = hf * 1024 + (n ^ (4 * hf)) * 16, v_at = SIDE + hf * (16 * D) + n * 16;

    for (int b = blockIdx.z; b < s.batch; b += gridDim.z) {
        long tok0;
        int nq;
        seq_range(a.cu_q, s, b, &tok0, &nq);
        const int rows = nq * a.G;
        bool over;
        const int kv_len = seq_keys(a.kv_lens, s, b, &over), pos0 = kv_len - nq;
        const int* const row_of = a.table + (size_t)b * s.table_stride;
        const uint8_t* const head = a.codes + side_base(0, h, 0, s);
        const size_t page_bytes = (size_t)s.hkv * 2 * s.page * D;
        for (int r0 = rt0 * BR; r0 < rows; r0 += row_tiles * BR) {
            const int r1 = r0 + BR < rows ? r0 + BR : rows;
            int g_lo, g_hi;
            key_range(a, kv_len, pos0, a.by_g.div(r0), a.by_g.div(r1 - 1), &g_lo, &g_hi);
            // this wave's rows
            const int w0 = r0 + 32 * wave, w1 = w0 + 32 < rows ? w0 + 32 : rows;
            const bool live = w0 < rows;
            const int t_first = a.by_g.div(live ? w0 : r0), t_last = a.by_g.div(live ? w1 - 1 : r0);
            int wg_lo, wg_hi;
            key_range(a, kv_len, pos0, t_first, t_last, &wg_lo, &wg_hi);
            const int all_lo = first_seen(a, pos0 + t_last);
            const int all_hi = a.causal ? (pos0 + t_first + 1 < kv_len ? pos0 + t_first + 1 : kv_len) : kv_len;
            // this lane's row
            const int r = w0 + n, rr = r < rows ? r : rows - 1;
            const int t = a.by_g.div(rr), hq = h * a.G + (rr - t * a.G), pos = pos0 + t;
            const float slope = may_bias(MODE) && a.slopes ? a.slopes[hq] * (MODE == SC_BIAS ? 1.0f / a.scale : kLog2e) : 0.0f;
            v8 qf[NK];
            {
                const T* q = (const T*)a.q + (tok0 + t) * a.q_ts + (long)hq * a.q_hs;
#pragma unroll
                for (int j = 0; j < NK; ++j) qf[j] = *reinterpret_cast<const v8*>(q + 16 * (2 * (j >> 1) + hf) + 8 * (j & 1));
            }
            // x * unit: the exponent of 2; of the capped and general kinds x is that already
            const float unit = MODE != SC_PLAIN && MODE != SC_BIAS ? 1.0f : a.scale * kLog2e, top_x = (LAG + UP) / unit;
            const float cap0 = 2.0f * kLog2e * a.scale / (a.cap > 0.0f ? a.cap : 1.0f);
            floatx16 o[ND];
#pragma unroll
            for (int d = 0; d < ND; ++d) o[d] = zero16();
            float m = kNegInf, mb = 0.0f;   // what weights refer to, a maximum less UP; with 0 for -inf
            float l = 0.0f, le = 0.0f;      // sums of rounded and (for lse) of exact weights

            for (int c0 = g_lo + split * a.chunk; c0 < g_hi; c0 += a.nsplit * a.chunk) {
                const int c1 = c0 + a.chunk < g_hi ? c0 + a.chunk : g_hi;
                // Loads of this wave's share of the stage at block k0, the page's id already here.
                auto block_of = [&](int k0) { return k0 + blk < c1 ? k0 + blk : c1 - 1; };
                auto load_id = [&](int k0) {
                    const int pg = block_of(k0) >> a.pg_shift;
                    return row_of[pg < s.table_stride ? pg : 0];
                };
                u32x4 raw[PW];
                float sc[PW];
                auto load = [&](int k0, int idv) {
                    const int gk = block_of(k0), pg = gk >> a.pg_shift;
                    int id = __builtin_amdgcn_readfirstlane(idv);
                    const bool ok = (unsigned)id < (unsigned)s.pages && pg < s.table_stride;
                    id = ok ? id : 0;
                    global_u8* src = global_at(head) + id * page_bytes + (gk - (pg << a.pg_shift)) * (16 * D);
                    global_u8* scale = global_at(a.scales) + ((size_t)id * s.hkv + h) * 8;
                    // (the choice is on the addresses: one on the values would wait for the loads)
                    scale = ok ? scale : no_page + offsetof(NoPage, scale);
#pragma unroll
                    for (int i = 0; i < PW; ++i) {
                        const int side = (piece0 + i) / NP, p = (piece0 + i) % NP;
                        sc[i] = *(FC_GLOBAL const float*)(scale + 4 * side);
                        global_u8* from = ok ? src + side * (s.page * D) : no_page + side * 4096;
                        raw[i] = *(FC_GLOBAL const u32x4*)(from + p * 1024 + lane * 16);
                    }
                };
                // weight 0 times a NaN code past the end would be NaN: those codes are cleared
                auto clear_tail = [&](int k0) {
                    const int keep = kv_len - (k0 + blk) * 16;   // tokens of the block that there are
                    if (keep >= 16) return;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int k = keep - 4 * j;
                        const unsigned mk = k >= 4 ? ~0u : (k <= 0 ? 0u : (1u << (8 * k)) - 1u);
#pragma unroll
                        for (int i = 0; i < PW; ++i) raw[i][j] &= piece0 + i < NP ? ~0u : mk;
                    }
                };
                // half i & 1 of piece i >> 1: eight codes a lane
                auto widen = [&](int stage, int i) {
                    const int pc = piece0 + (i >> 1), p = pc % NP, e = i & 1;
                    FC_LDS u32x4* d = (FC_LDS u32x4*)(lb + stage * STAGE + (pc >= NP ? v_to + p * 1024 + e * (32 * D)
                                                                                     : k_to + p * 4096 + e * 512));
                    if (kPoison) *d = u32x4{kPoisonWord, kPoisonWord, kPoisonWord, kPoisonWord};
                    *d = __builtin_bit_cast(u32x4, frag8<T>(raw[i >> 1][2 * e], raw[i >> 1][2 * e + 1], sc[i >> 1]));
                };
                constexpr int PARTS = 2 * PW;
                int id = load_id(c0);
                load(c0, id);
                id = load_id(c0 + KB);
                __syncthreads();   // the buffers are free
                clear_tail(c0);
#pragma unroll
                for (int i = 0; i < PARTS; ++i) widen(0, i);
                load(c0 + KB, id);
                id = load_id(c0 + 2 * KB);
                for (int k0 = c0, stage = 0; k0 < c1; k0 += KB, stage ^= 1) {
                    __syncthreads();   // this stage is here, and every wave is done with the other one
                    // the next stage's share is widened between this one's products (after the
                    // last stage to no purpose)
                    clear_tail(k0 + KB);
                    if (!live || k0 >= wg_hi || k0 + KB <= wg_lo) {
#pragma unroll
                        for (int i = 0; i < PARTS; ++i) widen(stage ^ 1, i);
                        load(k0 + 2 * KB, id);
                        id = load_id(k0 + 3 * KB);
                        continue;
                    }
                    const lds_u8* const kb = lb + stage * STAGE + k_at;
                    const lds_u8* const vb = lb + stage * STAGE + v_at;
                    const int key0 = k0 * 16 + 16 * hf;
                    // The accumulators begin at minus the reference maximum (and the bias), so that
                    // the products come out as the exponent's argument, up to its factor.
                    floatx16 x[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const float base = MODE == SC_BIAS ? slope * (float)(key0 + 32 * u - pos) - mb
                                           : MODE == SC_PLAIN ? -mb : 0.0f;
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[u][i] = MODE == SC_BIAS ? __builtin_fmaf(slope, (float)i, base) : base;
                    }
                    // Operands are read AH products ahead, the first of V before the softmax; the
                    // barriers keep the compiler from sinking each read to its use.
                    constexpr int NF = U * NK, NV = KB * ND;
                    auto k_read = [&](int i) {   // subtile i % U, dims of step i / U
                        const int j = i / U;
                        return *reinterpret_cast<const FC_LDS v8*>(kb + i % U * (SIDE / U) + (j >> 1) * 2048 + (j & 1) * 512);
                    };
                    auto v_read = [&](int i) {   // keys of step i / ND, dims of tile i % ND
                        return *reinterpret_cast<const FC_LDS v8*>(vb + (i / ND) * (32 * D) + (i % ND) * 512);
                    };
                    v8 kf[NF], vf[NV];
#pragma unroll
                    for (int i = 0; i < AH; ++i) kf[i] = k_read(i);
#pragma unroll
                    for (int g = 0; g < NF; g += AH) {
#pragma unroll
                        for (int i = g; i < g + AH; ++i) {
                            if (i + AH < NF) kf[i + AH] = k_read(i + AH);
                            else vf[i + AH - NF] = v_read(i + AH - NF);
                        }
                        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                        for (int i = g; i < g + AH; ++i) {
                            x[i % U] = Tr<T>::mfma32(kf[i], qf[i / U], x[i % U]);
                            if (i * PARTS / NF != (i + 1) * PARTS / NF) widen(stage ^ 1, i * PARTS / NF);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    load(k0 + 2 * KB, id);
                    id = load_id(k0 + 3 * KB);
                    if (MODE != SC_PLAIN && MODE != SC_BIAS) {
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            const float gap = (float)(pos - key0 - 32 * u);
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float bias = may_bias(MODE) ? __builtin_fmaf(slope, fabsf(gap - (float)i), mb) : mb;
                                x[u][i] = MODE == SC_FAR                   ? capped_far(x[u][i], cap0, a.cap * kLog2e, bias)
                                          : MODE == SC_CAP || a.cap > 0.0f ? capped(x[u][i], cap0, a.cap * kLog2e, bias)
                                                                           : x[u][i] * (a.scale * kLog2e) - bias;
                            }
                        }
                    }
                    if (k0 * 16 < all_lo || (k0 + KB) * 16 > all_hi || k0 + KB > c1) {
                        int top = a.causal && pos + 1 < kv_len ? pos + 1 : kv_len;
                        top = (top < c1 * 16 ? top : c1 * 16) - key0;
                        const int low = first_seen(a, pos) - key0;
#pragma unroll
                        for (int u = 0; u < U; ++u)
#pragma unroll
                            for (int i = 0; i < 16; ++i) x[u][i] = 32 * u + i < top && 32 * u + i >= low ? x[u][i] : kNegInf;
                    }
                    // From here on this wave goes first: the SIMD's other waves have their first product
                    // to fill the gaps with, which needs the vector unit least (314 -> 295 us for two
                    // prompts of 4096, 133 -> 115 for chunks with a bias).
                    __builtin_amdgcn_s_setprio(3);
                    float mx = x[0][0];
#pragma unroll
                    for (int i = 1; i < 16 * U; ++i) mx = fmaxf(mx, x[i >> 4][i & 15]);
                    mx = max_x32(mx);
                    // Weights refer to a maximum that may lag by a factor of 2^LAG, so that most stages do
                    // not touch the accumulators: a weight is as exact as if it were at most 1.
                    if (__any(mx > (m == kNegInf ? kNegInf : top_x))) {
                        const float below = UP ? top_x * (UP / (float)(LAG + UP)) : 0.0f;
                        const float mn = fmaxf(m, mx + mb - below), to = mn == kNegInf ? 0.0f : mn;
                        const float by = to - mb;
                        const float alpha = __builtin_amdgcn_exp2f((m - to) * unit);
                        m = mn;
                        mb = to;
                        l *= alpha;
                        le *= alpha;
#pragma unroll
                        for (int d = 0; d < ND; ++d) o[d] *= alpha;
#pragma unroll
                        for (int i = 0; i < 16 * U; ++i) x[i >> 4][i & 15] -= by;
                        // where a step of 32-bit scores is not small, the reference is off by as much
                        if (UP && __any(fabsf(to) * unit > 0x1p20f)) {
#pragma unroll
                            for (int i = 0; i < 16 * U; ++i) x[i >> 4][i & 15] = x[i >> 4][i & 15] > top_x ? top_x : x[i >> 4][i & 15];
                        }
                    }
                    if (a.lse) {   // (their weights once more, rather than a sum that other calls pay for)
                        float exact = 0.0f;
#pragma unroll
                        for (int i = 0; i < 16 * U; ++i) {
                            float y = x[i >> 4][i & 15];
                            asm("" : "+v"(y));   // (or all calls' exponentials are computed here)
                            exact += __builtin_amdgcn_exp2f(y * unit);
                        }
                        le += exact;
                    }
                    // weights and second product by turns: the products with 8 keys' weights, and
                    // between them the weights of the next 8
                    float sum = 0.0f;
                    u32x4 w[KB];
                    auto weigh = [&](int i) {
                        const float p0 = __builtin_amdgcn_exp2f(x[i >> 3][2 * (i & 7)] * unit);
                        const float p1 = __builtin_amdgcn_exp2f(x[i >> 3][2 * (i & 7) + 1] * unit);
                        w[i >> 2][i & 3] = Tr<T>::pk(p0, p1);
                        sum = Tr<T>::add2(w[i >> 2][i & 3], sum);
                    };
#pragma unroll
                    for (int i = 0; i < 4; ++i) weigh(i);
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        if (i + AH < NV) vf[i + AH] = v_read(i + AH);
                        o[i % ND] = Tr<T>::mfma32(vf[i], __builtin_bit_cast(v8, w[i / ND]), o[i % ND]);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (i / ND < KB - 1 && k * ND / 4 == i % ND) weigh(4 * (i / ND + 1) + k);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    __builtin_amdgcn_s_setprio(0);
                    l += sum;
                }
            }
            l = over ? __builtin_nanf("") : sum_x32(l);
            le = over ? l : sum_x32(le);
            if (r < rows) {
                const long row = (tok0 + t) * s.hq + hq;
                if (a.nsplit == 1) {
                    const float inv = l != 0.0f ? 1.0f / l : 0.0f;   // no key seen: 0
                    T* out = (T*)a.out + row * D + 4 * hf;
#pragma unroll
                    for (int d = 0; d < ND; ++d)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            u32x2 v;
                            v[0] = Tr<T>::pk(o[d][4 * k] * inv, o[d][4 * k + 1] * inv);
                            v[1] = Tr<T>::pk(o[d][4 * k + 2] * inv, o[d][4 * k + 3] * inv);
                            *reinterpret_cast<u32x2*>(out + 32 * d + 8 * k) = v;
                        }
                    if (a.lse && hf == 0) a.lse[row] = (m * unit + __builtin_amdgcn_logf(le)) * (1.0f / kLog2e);
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
                    if (hf == 0) a.part_ml[at] = floatx4{m * unit, l, le, 0.0f};
                }
            }
        }
    }
}

template <class T, int D, int MODE>
static hipError_t launch_tile(const AttnArgs& a, hipStream_t st)
{
    constexpr int NW = tile_waves(D);
    static std::atomic<unsigned long long> done{0};
    hipError_t e = allow_full_lds((const void*)k_attn_tile<T, D, NW, MODE>, &done);
    if (e != hipSuccess) return e;
    const long rows = (long)(a.s.max_q > 0 ? a.s.max_q : 1) * a.G;
    long rt = (rows + 32 * NW - 1) / (32 * NW);
    if (rt * a.nsplit > 65535) rt = 65535 / a.nsplit;
    // heads fastest: workgroups go round-robin over the 8 XCDs, so that the row
    // tiles of a head, which read the same codes, meet in one L2 (hkv % 8 == 0)
    const dim3 grid(a.s.hkv, (unsigned)(rt * a.nsplit), a.s.batch < 65535 ? a.s.batch : 65535);
    k_attn_tile<T, D, NW, MODE><<<grid, dim3(64 * NW), 2 * 2 * 16 * tile_blocks(D) * D * 2, st>>>(a, (int)rt);
    return hipGetLastError();
}

template <class T, int D>
static hipError_t tile_mode(const AttnArgs& a, hipStream_t st)
{
    return by_kind(a, [&](auto k) { return launch_tile<T, D, decltype(k)::value>(a, st); });
}

template <class T>
static hipError_t tile_by_d(const AttnArgs& a, hipStream_t st)
{
    switch (a.s.d) {
    case 64: return tile_mode<T, 64>(a, st);
    case 128: return tile_mode<T, 128>(a, st);
    case 192: return tile_mode<T, 192>(a, st);
    default: return tile_mode<T, 256>(a, st);
    }
}

hipError_t run_attn_tile(int dtype, const AttnArgs& a, hipStream_t st)
{
    return dtype == DT_F16 ? tile_by_d<half_t>(a, st) : tile_by_d<bf16_t>(a, st);
}

}  // namespace fc

// kv_move.hip -- moves tokens and pages of the paged 8-bit cache: the accepted
// tokens of a draft into consecutive slots (k_kv_keep), whole pages to others
// (k_kv_copy).
//
// Keeping is bound by its chain of dependent loads (lengths -> list -> page ids ->
// scales -> codes) and the launch: one sequence, two heads, 4.9 us; 32 sequences x
// 8 heads x 8 layers, a block each, 12.2 (with no token to move 3.6; page after page, every
// lookup by every thread again, 15.5).  Copying is bound by memory: 401 pages of
// 128 KiB in 8 layers, 842 MB in 166 us, 5.1 TB/s read and written, a plain copy's
// rate.
#include "fc_launch.h"
#include "kv_common.h"

namespace fc {

__device__ __forceinline__ unsigned recode_codes(unsigned w, float ratio)
{
    const floatx2 a = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
    return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(
        b[0] * ratio, b[1] * ratio, __builtin_amdgcn_cvt_pk_fp8_f32(a[0] * ratio, a[1] * ratio, 0, false), true);
}

struct KeepArgs {
    uint8_t* codes;
    float* scales;
    const int *table, *cu_q, *kv_lens, *keep, *kept;
    int max_keep;
    int staged;                         // tokens that a block holds at a time
    size_t layer_codes, layer_scales;   // bytes and scales of a layer
    KvShape s;
    FastDiv units, by_d;                // d / 16, d
};

constexpr int KEEP_PAGES = 4;   // that a block writes at a time

// A token's source: page (or -1), place in it, scales; and which of the pages it goes to.
struct alignas(16) Source {
    int page;
    short at, to;
    float scale[2];
};
struct alignas(16) KeepShared {
    unsigned now[KEEP_PAGES][2];   // bits of the pages' new scales
    float held[KEEP_PAGES][2];
    int id[KEEP_PAGES];
    unsigned bad, moves;
};

// One block a (sequence, kv head, layer).  Tokens only ever move to lower slots, a page's
// tokens come from it and from later ones: as many pages as there is room for are taken at a
// time, in order, their tokens gathered into LDS before any byte of them changes.
// A scale is a power of two, so that the codes of a page whose scale grows, and those that
// come from a smaller one, are rounded once more only where they become subnormal.
__global__ __launch_bounds__(256) void k_kv_keep(KeepArgs a)
{
    const KvShape& s = a.s;
    const int b = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, D = s.d, units = D / 16;
    uint8_t* const codes = a.codes + blockIdx.z * a.layer_codes;
    float* const scales = a.scales + blockIdx.z * a.layer_scales;
    long tok0;
    int n;
    seq_range(a.cu_q, s, b, &tok0, &n);
    const int kv_len = a.kv_lens[b], m = a.kept[b], start = kv_len - n;
    if (m <= 0 || m > n || m > a.max_keep || kv_len < n || kv_len > s.page * s.table_stride) return;
    const int* const list = a.keep + (size_t)b * a.max_keep;
    extern __shared__ __align__(16) uint8_t lds[];      // KeepShared, the sources, then [side][token][d]
    KeepShared& sh = *reinterpret_cast<KeepShared*>(lds);
    Source* const sources = reinterpret_cast<Source*>(lds + sizeof(KeepShared));
    uint8_t* const sk = lds + sizeof(KeepShared) + sizeof(Source) * a.staged;
    uint8_t* const sv = sk + a.staged * D;
    const auto poison = [&](void* from) {   // (poison build) all from there on
        if constexpr (kPoison) {
            lds_poison(from, (int)(sv + a.staged * D - (uint8_t*)from), tid, 256);
            __syncthreads();
        }
    };
    poison(lds);
    if (tid == 0) sh.bad = sh.moves = 0;
    __syncthreads();
    bool bad = false, moves = false;
    for (int i = tid; i < m; i += 256) {
        const int k = list[i], before = i ? list[i - 1] : -1;
        bad |= k <= before || k >= n;
        moves |= k != i;
    }
    if (bad) sh.bad = 1;
    if (moves) sh.moves = 1;
    __syncthreads();
    if (sh.bad || !sh.moves) return;

    const auto scale_at = [&](int page, int side) { return scales + ((size_t)page * s.hkv + h) * 2 + side; };
    const auto k_at = [&](int page, int at, int u) {
        return codes + side_base(page, h, 0, s) + (at >> 4) * 16 * D + u * 256 + (at & 15) * 16;
    };
    const auto v_at = [&](int page, int at, int dim) {
        return codes + side_base(page, h, 1, s) + (size_t)((at >> 4) * D + dim) * 16 + (at & 15);
    };
    const int last = (start + m - 1) / s.page;
    for (int p = start / s.page, i0 = 0; p <= last;) {
        // pages p .. p + pages - 1, tokens i0 .. i0 + cnt - 1
        const auto upto = [&](int q) { return min(m, (q + 1) * s.page - start); };
        int pages = 1;
        while (pages < KEEP_PAGES && p + pages <= last && upto(p + pages) - i0 <= a.staged) ++pages;
        const int cnt = upto(p + pages - 1) - i0;
        Source src{-1, 0, 0, {0.0f, 0.0f}};
        if (tid < cnt) {   // (at most a.staged, and that at most 256)
            const int slot = start + list[i0 + tid];
            src.page = page_id(a.table, s, b, slot / s.page);
            src.at = (short)(slot % s.page);
            src.to = (short)((start + i0 + tid) / s.page - p);
            if (src.page >= 0) {
                src.scale[0] = *scale_at(src.page, 0);
                src.scale[1] = *scale_at(src.page, 1);
            }
            sources[tid] = src;
        }
        if (tid < 2 * pages) {
            const int q = tid >> 1, side = tid & 1, id = page_id(a.table, s, b, p + q);
            const float held = id >= 0 ? *scale_at(id, side) : 0.0f;
            sh.id[q] = id;
            sh.held[q][side] = held;
            sh.now[q][side] = __builtin_bit_cast(unsigned, held);
        }
        __syncthreads();
        if (src.page >= 0)
#pragma unroll
            for (int side = 0; side < 2; ++side)   // (positive: they order as integers)
                atomicMax(&sh.now[src.to][side], __builtin_bit_cast(unsigned, src.scale[side]));
        __syncthreads();
        const auto now = [&](int q, int side) { return __builtin_bit_cast(float, sh.now[q][side]); };
        for (int e = tid; e < cnt * units; e += 256) {
            const int t = a.units.div(e), u = e - t * units;
            const Source from = sources[t];
            u32x4 w = {0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu};
            if (from.page >= 0) {
                w = *reinterpret_cast<const u32x4*>(k_at(from.page, from.at, u));
                const float ratio = from.scale[0] / now(from.to, 0);
                if (ratio != 1.0f) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = recode_codes(w[j], ratio);
                }
            }
            *reinterpret_cast<u32x4*>(sk + t * D + u * 16) = w;
        }
        for (int e0 = tid; e0 < cnt * D; e0 += 4 * 256) {   // four bytes on the way at a time
            unsigned w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int e = e0 + 256 * j, t = a.by_d.div(e);
                w[j] = e < cnt * D && sources[t].page >= 0 ? *v_at(sources[t].page, sources[t].at, e - t * D) : 0;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int e = e0 + 256 * j, t = a.by_d.div(e);
                if (e >= cnt * D) continue;
                const float ratio = sources[t].page >= 0 ? sources[t].scale[1] / now(sources[t].to, 1) : 1.0f;
                sv[e] = (uint8_t)(ratio != 1.0f ? recode_codes(w[j], ratio) : w[j]);
            }
        }
        __syncthreads();
        // earlier tokens of the first page, where its scale grows
        const int lo = start - p * s.page, id0 = sh.id[0];
        if (lo > 0 && id0 >= 0) {
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                const float held = sh.held[0][side];
                if (!(now(0, side) > held)) continue;
                const float ratio = held / now(0, side);
                uint8_t* const base = codes + side_base(id0, h, side, s);
                if (side == 0) {
                    for (int e = tid; e < lo * units; e += 256) {
                        const int t = a.units.div(e), u = e - t * units;
                        u32x4* q = reinterpret_cast<u32x4*>(base + (t >> 4) * 16 * D + u * 256 + (t & 15) * 16);
                        u32x4 w = *q;
#pragma unroll
                        for (int j = 0; j < 4; ++j) w[j] = recode_codes(w[j], ratio);
                        *q = w;
                    }
                } else {
                    for (int e = tid; e < ((lo + 15) >> 4) * D; e += 256) {
                        const int left = lo - a.by_d.div(e) * 16;   // tokens of the block that were there
                        u32x4* q = reinterpret_cast<u32x4*>(base + (size_t)e * 16);
                        u32x4 w = *q;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int k = left - 4 * j;
                            const unsigned mk = k >= 4 ? ~0u : (k <= 0 ? 0u : (1u << (8 * k)) - 1u);
                            w[j] = (recode_codes(w[j], ratio) & mk) | (w[j] & ~mk);
                        }
                        *q = w;
                    }
                }
            }
            __syncthreads();   // the vectors are written before single bytes of them
        }
        for (int e = tid; e < cnt * units; e += 256) {
            const int t = a.units.div(e), u = e - t * units, q = sources[t].to, at = start + i0 + t - (p + q) * s.page;
            if (sh.id[q] >= 0) *reinterpret_cast<u32x4*>(k_at(sh.id[q], at, u)) = *reinterpret_cast<const u32x4*>(sk + t * D + u * 16);
        }
        for (int e = tid; e < cnt * D; e += 256) {
            const int t = a.by_d.div(e), q = sources[t].to, at = start + i0 + t - (p + q) * s.page;
            if (sh.id[q] >= 0) *v_at(sh.id[q], at, e - t * D) = sv[e];
        }
        if (tid < 2 * pages && sh.id[tid >> 1] >= 0) *scale_at(sh.id[tid >> 1], tid & 1) = now(tid >> 1, tid & 1);
        __syncthreads();   // LDS is free again
        poison(lds);
        p += pages;
        i0 += cnt;
    }
}

// The pairs travel with the launch (4 KiB of arguments), so that the host's list needs no copy on the device.
constexpr int COPY_PAIRS = 448;
struct CopyArgs {
    uint8_t* codes;
    float* scales;
    size_t page_bytes, layer_codes, layer_scales;
    int per_page;   // scales of a page
    int pair[COPY_PAIRS][2];
};

__global__ __launch_bounds__(256) void k_kv_copy(CopyArgs a)
{
    const int from = a.pair[blockIdx.y][0], to = a.pair[blockIdx.y][1];
    uint8_t* const codes = a.codes + blockIdx.z * a.layer_codes;
    const u32x4* src = reinterpret_cast<const u32x4*>(codes + (size_t)from * a.page_bytes);
    u32x4* dst = reinterpret_cast<u32x4*>(codes + (size_t)to * a.page_bytes);
    const int n = (int)(a.page_bytes / 16);
    for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) dst[i] = src[i];
    if (blockIdx.x == 0) {
        float* const scales = a.scales + blockIdx.z * a.layer_scales;
        for (int i = threadIdx.x; i < a.per_page; i += 256)
            scales[(size_t)to * a.per_page + i] = scales[(size_t)from * a.per_page + i];
    }
}

hipError_t run_kv_keep(uint8_t* codes, float* scales, int layers, const int* table, const int* cu_q, const int* kv_lens,
                       const int* keep, const int* kept, int max_keep, const KvShape& s, hipStream_t st)
{
    static std::atomic<unsigned long long> done{0};
    hipError_t e = allow_full_lds((const void*)k_kv_keep, &done);
    if (e != hipSuccess) return e;
    KeepArgs a{};
    a.codes = codes;
    a.scales = scales;
    a.table = table;
    a.cu_q = cu_q;
    a.kv_lens = kv_lens;
    a.keep = keep;
    a.kept = kept;
    a.max_keep = max_keep;
    a.layer_scales = (size_t)s.pages * s.hkv * 2;
    a.layer_codes = a.layer_scales * s.page * s.d;
    a.s = s;
    a.units = FastDiv::make(s.d / 16);
    a.by_d = FastDiv::make(s.d);
    // a page's worth, or a few small pages'
    const int room = s.page < 32 ? 32 : s.page;
    a.staged = max_keep < room ? max_keep : room;
    const int lds = (int)sizeof(KeepShared) + (2 * s.d + (int)sizeof(Source)) * a.staged;
    k_kv_keep<<<dim3(s.batch, s.hkv, layers), dim3(256), lds, st>>>(a);
    return hipGetLastError();
}

hipError_t run_kv_copy(uint8_t* codes, float* scales, int layers, int pages, int hkv, int page, int d, const int* pairs, long n,
                       hipStream_t st)
{
    CopyArgs a;
    a.codes = codes;
    a.scales = scales;
    a.per_page = hkv * 2;
    a.page_bytes = (size_t)a.per_page * page * d;
    a.layer_codes = (size_t)pages * a.page_bytes;
    a.layer_scales = (size_t)pages * a.per_page;
    const size_t blocks = (a.page_bytes + 16383) / 16384;
    for (long i = 0; i < n; i += COPY_PAIRS) {
        const int m = (int)(n - i < COPY_PAIRS ? n - i : COPY_PAIRS);
        for (int k = 0; k < m; ++k) {
            a.pair[k][0] = pairs[2 * (i + k)];
            a.pair[k][1] = pairs[2 * (i + k) + 1];
        }
        k_kv_copy<<<dim3((unsigned)(blocks < 4096 ? blocks : 4096), m, layers), dim3(256), 0, st>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace fc

// kv_move.hip -- moves tokens and pages of the paged 8-bit cache: the accepted
// tokens of a draft into consecutive slots (k_kv_keep), whole pages to others
// (k_kv_copy).
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
    size_t layer_codes, layer_scales;   // bytes and scales of a layer
    KvShape s;
    FastDiv units, by_d;                // d / 16, d
};

// One block a (sequence, kv head, layer).  Tokens only ever move to lower slots, a page's
// tokens come from it and from later ones: the pages are taken in order, each one's tokens
// gathered into LDS before any byte of it changes.
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
    extern __shared__ __align__(16) uint8_t lds[];      // two scales, two flags, then [side][token][d]
    unsigned* const top = reinterpret_cast<unsigned*>(lds);
    uint8_t* const staged = lds + 16;
    if (tid < 2) top[2 + tid] = 0;
    __syncthreads();
    bool bad = false, moves = false;
    for (int i = tid; i < m; i += 256) {
        const int k = list[i], before = i ? list[i - 1] : -1;
        bad |= k <= before || k >= n;
        moves |= k != i;
    }
    if (bad) top[2] = 1;
    if (moves) top[3] = 1;
    __syncthreads();
    if (top[2] || !top[3]) return;

    for (int p = start / s.page; p <= (start + m - 1) / s.page; ++p) {
        const int slot0 = p * s.page;
        const int i0 = slot0 > start ? slot0 - start : 0, i1 = slot0 + s.page - start < m ? slot0 + s.page - start : m;
        const int cnt = i1 - i0, id = page_id(a.table, s, b, p);
        if (id < 0) continue;
        float* const scale = scales + ((size_t)id * s.hkv + h) * 2;
        const float held[2] = {scale[0], scale[1]};
        if (tid < 2) top[tid] = 0;
        __syncthreads();
        for (int i = tid; i < cnt; i += 256) {
            const int from = page_id(a.table, s, b, (start + list[i0 + i]) / s.page);
            if (from < 0) continue;
#pragma unroll
            for (int side = 0; side < 2; ++side)   // (positive: they order as integers)
                atomicMax(&top[side], __builtin_bit_cast(unsigned, scales[((size_t)from * s.hkv + h) * 2 + side]));
        }
        __syncthreads();
        float now[2];
#pragma unroll
        for (int side = 0; side < 2; ++side) now[side] = fmaxf(held[side], __builtin_bit_cast(float, top[side]));
        uint8_t* const sk = staged;
        uint8_t* const sv = staged + (size_t)cnt * D;
        for (int e = tid; e < cnt * units; e += 256) {
            const int t = a.units.div(e), u = e - t * units, slot = start + list[i0 + t], at = slot % s.page;
            const int from = page_id(a.table, s, b, slot / s.page);
            u32x4 w = {0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu};
            if (from >= 0) {
                w = *reinterpret_cast<const u32x4*>(codes + side_base(from, h, 0, s) + (at >> 4) * 16 * D + u * 256 + (at & 15) * 16);
                const float ratio = scales[((size_t)from * s.hkv + h) * 2] / now[0];
                if (ratio != 1.0f) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = recode_codes(w[j], ratio);
                }
            }
            *reinterpret_cast<u32x4*>(sk + t * D + u * 16) = w;
        }
        for (int e = tid; e < cnt * D; e += 256) {
            const int t = a.by_d.div(e), dim = e - t * D, slot = start + list[i0 + t], at = slot % s.page;
            const int from = page_id(a.table, s, b, slot / s.page);
            unsigned w = 0;
            if (from >= 0) {
                w = codes[side_base(from, h, 1, s) + (size_t)((at >> 4) * D + dim) * 16 + (at & 15)];
                const float ratio = scales[((size_t)from * s.hkv + h) * 2 + 1] / now[1];
                if (ratio != 1.0f) w = recode_codes(w, ratio);
            }
            sv[t * D + dim] = (uint8_t)w;
        }
        __syncthreads();
        // earlier tokens of the page, where its scale grows
        const int lo = start > slot0 ? start - slot0 : 0;
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            if (lo == 0 || !(now[side] > held[side])) continue;
            const float ratio = held[side] / now[side];
            uint8_t* const base = codes + side_base(id, h, side, s);
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
        for (int e = tid; e < cnt * units; e += 256) {
            const int t = a.units.div(e), u = e - t * units, at = start + i0 + t - slot0;
            *reinterpret_cast<u32x4*>(codes + side_base(id, h, 0, s) + (at >> 4) * 16 * D + u * 256 + (at & 15) * 16) =
                *reinterpret_cast<const u32x4*>(sk + t * D + u * 16);
        }
        for (int e = tid; e < cnt * D; e += 256) {
            const int t = a.by_d.div(e), dim = e - t * D, at = start + i0 + t - slot0;
            codes[side_base(id, h, 1, s) + (size_t)((at >> 4) * D + dim) * 16 + (at & 15)] = sv[t * D + dim];
        }
        if (tid < 2) scale[tid] = now[tid];
        __syncthreads();   // LDS is free again
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
    const int lds = 16 + 2 * s.d * (max_keep < s.page ? max_keep : s.page);
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

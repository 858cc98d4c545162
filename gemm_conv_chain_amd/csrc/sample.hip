// sample.hip -- draws a token from each row of logits: temperature, the top_k
// largest, the least set that holds top_p of the mass, min_p, and one random
// number (k_sample_row).
//
// What stays is a prefix of the row in falling order, so that it is described by
// its last element: a value and, among equal ones, an index (Cut).  No row is
// sorted: a histogram over log2 of the weights, with a count and a mass a bin,
// finds the bin in which the top_k-th element or the mass top_p lies, and only
// that bin's elements are looked at one by one.  The token is the first one in
// order of index at which the running sum passes u times the whole: sums of
// sixteenths of the row, then of sixteenths of the one it lies in, and so on.
//
// Weights are 64-bit exponentials, rounded once to integers in units of 2^-42:
// integer sums do not depend on their order, and with it the token.  32-bit
// weights would be off by 1e-7 of the mass, a token in as many million rows.
#include "fc_launch.h"
#include "kv_common.h"

namespace fc {

typedef unsigned long long u64;

constexpr int SR_WAVES = 16, SR_THREADS = 64 * SR_WAVES;
constexpr int SR_BINS = 4096;      // of 1/128 of an octave; the last holds all weights under 2^-32
constexpr int SR_SUB = 1024;       // of a bin's own values, where it holds more than SR_LIST
constexpr int SR_LIST = 256;
constexpr double SR_ONE = 0x1p42;  // a weight of 1

struct SampleArgs {
    const void* logits;
    long stride;
    const float* u;
    const float* temperatures;
    const int* top_ks;
    const float* top_ps;
    const float* min_ps;
    float temperature, top_p, min_p;
    int top_k, vocab;
    long rows;
    int* out;
};

// An element stays if it is larger than the cut, or equal and not behind it.
struct Cut {
    float x;
    int index;
};

struct RowShared {
    u64 mass[SR_BINS];
    unsigned count[SR_BINS];
    u64 sub_mass[SR_SUB];
    unsigned sub_count[SR_SUB];
    u64 list_w[SR_LIST];
    float list_x[SR_LIST];
    int list_i[SR_LIST];
    u64 wave_mass[SR_WAVES];
    unsigned wave_count[SR_WAVES];
    float wave_x[SR_WAVES];
    int wave_i[SR_WAVES];
    unsigned n_list, key_lo, key_hi;
    int border;
    unsigned border_count;
    u64 border_mass;
    Cut cut;
    u64 cut_mass;
};

// Eight logits from i on, -inf past the row's end; -0 becomes 0, which it equals.
template <class L>
__device__ __forceinline__ void load_logits(const L* row, int i, int vocab, float (&x)[8])
{
    struct __attribute__((packed, aligned(sizeof(L)))) Eight { L v[8]; };
    if (i + 8 <= vocab) {
        const Eight e = *reinterpret_cast<const Eight*>(row + i);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = (float)e.v[j] + 0.0f;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = i + j < vocab ? (float)row[i + j] + 0.0f : kNegInf;
    }
}

// Unsigned integers in the order of the floats (no NaN).
__device__ __forceinline__ unsigned order_key(float x)
{
    const unsigned b = __builtin_bit_cast(unsigned, x);
    return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_key(unsigned k)
{
    return __builtin_bit_cast(float, k >> 31 ? k & 0x7fffffffu : ~k);
}

// 2^z for z <= 0 in units of 2^-42, rounded; z = (x - max) log2(e) / temperature.
// 2^f for |f| <= 1/2 by its Taylor series, whose next term is 7e-15.
__device__ __forceinline__ u64 weight_of(float x, double max, double slope)
{
    const double z = ((double)x - max) * slope;
    if (!(z > -64.0)) return 0;                        // (also -inf times a slope of 0)
    constexpr double shift = 0x1.8p52;
    const double zi = z + shift;
    const int n = (int)__builtin_bit_cast(u64, zi);    // nearest integer
    const double f = z - (zi - shift);
    constexpr double l = 0.693147180559945309417;
    constexpr double c2 = l * l / 2, c3 = c2 * l / 3, c4 = c3 * l / 4, c5 = c4 * l / 5, c6 = c5 * l / 6, c7 = c6 * l / 7,
                     c8 = c7 * l / 8, c9 = c8 * l / 9, c10 = c9 * l / 10, c11 = c10 * l / 11;
    double p = c11;
    p = __builtin_fma(p, f, c10);
    p = __builtin_fma(p, f, c9);
    p = __builtin_fma(p, f, c8);
    p = __builtin_fma(p, f, c7);
    p = __builtin_fma(p, f, c6);
    p = __builtin_fma(p, f, c5);
    p = __builtin_fma(p, f, c4);
    p = __builtin_fma(p, f, c3);
    p = __builtin_fma(p, f, c2);
    p = __builtin_fma(p, f, l);
    p = __builtin_fma(p, f, 1.0);
    p = __builtin_bit_cast(double, __builtin_bit_cast(u64, p) + ((u64)(long long)n << 52));
    // 1024 + w: the unit of its last bit is 2^-42
    return __builtin_bit_cast(u64, p + 1024.0) - __builtin_bit_cast(u64, 1024.0);
}

__device__ __forceinline__ u64 shfl64(u64 v, int lane) { return __shfl(v, lane); }
template <class V> __device__ __forceinline__ V wave_sum(V v)
{
#pragma unroll
    for (int s = 32; s; s >>= 1) v += __shfl_xor(v, s);
    return v;
}
// Sum of the lanes up to this one.
template <class V> __device__ __forceinline__ V wave_scan(V v, int lane)
{
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
        const V o = __shfl_up(v, s);
        if (lane >= s) v += o;
    }
    return v;
}

template <class L> struct Sampler {
    const SampleArgs& a;
    RowShared& s;
    const L* row;
    const int lane, wave, tid;
    double max, slope;
    float max_x, bins;      // bins of the histogram a unit of x

    __device__ __forceinline__ u64 weight(float x) const { return weight_of(x, max, slope); }
    __device__ __forceinline__ int bin(float x) const { return (int)fminf((max_x - x) * bins, (float)(SR_BINS - 1)); }

    // f(index, logits) for every eight of the row, in the whole block's lanes.
    template <class F> __device__ __forceinline__ void each(F&& f) const
    {
        for (int i = tid * 8; i < a.vocab; i += SR_THREADS * 8) {
            float x[8];
            load_logits(row, i, a.vocab, x);
            f(i, x);
        }
    }

    // The first index at which the running sum of w(index, x) passes `goal`, or with `draw` u
    // times the whole sum.
    template <class W> __device__ int locate(u64 goal, bool draw, float u, W&& w)
    {
        int lo = 0, hi = a.vocab;
        while (hi - lo > 512 || draw) {
            const int per = ((hi - lo + SR_WAVES - 1) / SR_WAVES + 511) / 512 * 512;
            const int z = lo + (wave + 1) * per < hi ? lo + (wave + 1) * per : hi;
            u64 sum = 0;
            for (int i = lo + wave * per + lane * 8; i < z; i += 512) {
                float x[8];
                load_logits(row, i, a.vocab, x);
#pragma unroll
                for (int j = 0; j < 8; ++j) sum += w(i + j, x[j]);
            }
            sum = wave_sum(sum);
            if (lane == 0) s.wave_mass[wave] = sum;
            __syncthreads();
            u64 part[SR_WAVES];
#pragma unroll
            for (int k = 0; k < SR_WAVES; ++k) part[k] = s.wave_mass[k];
            if (draw) {
                u64 all = 0;
#pragma unroll
                for (int k = 0; k < SR_WAVES; ++k) all += part[k];
                goal = (u64)((double)u * (double)all);
                goal = goal < all ? goal : all - 1;
                draw = false;
            }
            int at = 0;
#pragma unroll
            for (int k = 0; k < SR_WAVES - 1; ++k)
                if (at == k && goal >= part[k]) {
                    goal -= part[k];
                    ++at;
                }
            lo += at * per;
            hi = lo + per < hi ? lo + per : hi;
            __syncthreads();   // wave_mass is free
        }
        const int i = lo + lane * 8;
        float x[8];
        u64 own[8], sum = 0;
        if (i < a.vocab) load_logits(row, i, a.vocab, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            own[j] = i + j < hi ? w(i + j, x[j]) : 0;
            sum += own[j];
        }
        const u64 upto = wave_scan(sum, lane);
        const u64 past = __ballot(upto > goal);
        const int at = past ? __builtin_ctzll(past) : 63;
        u64 run = upto - sum;
        int found = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            run += own[j];
            found += run <= goal;
        }
        return __builtin_amdgcn_readlane(i + found, at);
    }

    // Scans n bins (thread t has n / SR_THREADS of them) and leaves in s.border the one in which
    // the count reaches k (mass == false) or the mass goal, with what lies before it.
    __device__ void find_border(const u64* mass, const unsigned* count, int n, bool by_mass, unsigned k, u64 goal)
    {
        const int per = n / SR_THREADS;
        u64 m = 0;
        unsigned c = 0;
        for (int j = 0; j < per; ++j) {
            m += mass[tid * per + j];
            c += count[tid * per + j];
        }
        u64 ms = wave_scan(m, lane);
        unsigned cs = wave_scan(c, lane);
        if (lane == 63) {
            s.wave_mass[wave] = ms;
            s.wave_count[wave] = cs;
        }
        __syncthreads();
        ms -= m;
        cs -= c;
        for (int w = 0; w < wave; ++w) {
            ms += s.wave_mass[w];
            cs += s.wave_count[w];
        }
        for (int j = 0; j < per; ++j) {
            const u64 bm = mass[tid * per + j];
            const unsigned bc = count[tid * per + j];
            if (by_mass ? ms < goal && ms + bm >= goal : cs < k && cs + bc >= k) {
                s.border = tid * per + j;
                s.border_mass = ms;
                s.border_count = cs;
            }
            ms += bm;
            cs += bc;
        }
        __syncthreads();
    }

    // The last element that stays, in s.cut, and the mass up to it, in s.cut_mass.
    __device__ void cut_row(bool by_mass, unsigned k, u64 goal)
    {
        find_border(s.mass, s.count, SR_BINS, by_mass, k, goal);
        const int b = s.border;
        k -= s.border_count;
        goal -= s.border_mass;
        u64 ahead = s.border_mass;
        unsigned lo = 0, hi = ~0u;   // keys of the bin's elements that are still in question
        for (;;) {
            if (tid == 0) {
                s.n_list = 0;
                s.key_lo = ~0u;
                s.key_hi = 0;
            }
            __syncthreads();
            each([&](int i, const float(&x)[8]) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (x[j] == kNegInf || bin(x[j]) != b) continue;
                    const unsigned key = order_key(x[j]);
                    if (key < lo || key > hi) continue;
                    const unsigned at = atomicAdd(&s.n_list, 1u);
                    atomicMin(&s.key_lo, key);
                    atomicMax(&s.key_hi, key);
                    if (at < SR_LIST) {
                        s.list_x[at] = x[j];
                        s.list_i[at] = i + j;
                        s.list_w[at] = weight(x[j]);
                    }
                }
            });
            __syncthreads();
            const unsigned n = s.n_list;
            if (n <= SR_LIST) {   // one by one: what lies before each
                if (tid < (int)n) {
                    const float x = s.list_x[tid];
                    const int index = s.list_i[tid];
                    const u64 w = s.list_w[tid];
                    u64 m = 0;
                    unsigned c = 0;
                    for (unsigned j = 0; j < n; ++j) {
                        const float y = s.list_x[j];
                        const bool first = y > x || (y == x && s.list_i[j] < index);
                        m += first ? s.list_w[j] : 0;
                        c += first;
                    }
                    if (by_mass ? m < goal && m + w >= goal : c == k - 1) {
                        s.cut = Cut{x, index};
                        s.cut_mass = ahead + m + w;
                    }
                }
                __syncthreads();
                return;
            }
            lo = s.key_lo;
            hi = s.key_hi;
            if (lo == hi) {       // all equal: the first few by index
                const float x = from_key(lo);
                const u64 w = weight(x);
                const u64 many = by_mass ? (goal + w - 1) / w : k;
                const int index = locate(many - 1, false, 0.0f, [&](int, float y) { return y == x ? 1ull : 0ull; });
                if (tid == 0) {
                    s.cut = Cut{x, index};
                    s.cut_mass = ahead + many * w;
                }
                __syncthreads();
                return;
            }
            int shift = 0;
            while ((hi - lo) >> shift >= SR_SUB) ++shift;
            for (int j = tid; j < SR_SUB; j += SR_THREADS) {
                s.sub_mass[j] = 0;
                s.sub_count[j] = 0;
            }
            __syncthreads();
            each([&](int, const float(&x)[8]) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (x[j] == kNegInf || bin(x[j]) != b) continue;
                    const unsigned key = order_key(x[j]);
                    if (key < lo || key > hi) continue;
                    atomicAdd(&s.sub_mass[(hi - key) >> shift], weight(x[j]));
                    atomicAdd(&s.sub_count[(hi - key) >> shift], 1u);
                }
            });
            __syncthreads();
            find_border(s.sub_mass, s.sub_count, SR_SUB, by_mass, k, goal);
            k -= s.border_count;
            goal -= s.border_mass;
            ahead += s.border_mass;
            const unsigned top = hi - ((unsigned)s.border << shift);   // the largest key of the sub-bin
            const unsigned span = (1u << shift) - 1;
            lo = top - lo > span ? top - span : lo;
            hi = top;
            __syncthreads();   // s.border is free
        }
    }

    __device__ int draw(long r)
    {
        // the largest, the first of them, and whether the row is a distribution
        float best = kNegInf;
        int first = 0x7fffffff;
        bool bad = false;
        each([&](int i, const float(&x)[8]) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                bad |= !(x[j] < __builtin_inff());
                if (x[j] > best) {
                    best = x[j];
                    first = i + j;
                }
            }
        });
#pragma unroll
        for (int k = 32; k; k >>= 1) {
            const float x = __shfl_xor(best, k);
            const int i = __shfl_xor(first, k);
            if (x > best || (x == best && i < first)) {
                best = x;
                first = i;
            }
        }
        if (lane == 0) {
            s.wave_x[wave] = best;
            s.wave_i[wave] = first;
        }
        const bool any_bad = __any(bad);
        if (lane == 0) s.wave_count[wave] = any_bad;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < SR_WAVES; ++k) {
            const float x = s.wave_x[k];
            const int i = s.wave_i[k];
            bad |= s.wave_count[k] != 0;
            if (x > best || (x == best && i < first)) {
                best = x;
                first = i;
            }
        }
        const float u = a.u[r];
        if (bad || best == kNegInf || u != u) return -1;
        const float t = a.temperatures ? a.temperatures[r] : a.temperature;
        const int k = a.top_ks ? a.top_ks[r] : a.top_k;
        const float p = a.top_ps ? a.top_ps[r] : a.top_p;
        float mp = a.min_ps ? a.min_ps[r] : a.min_p;
        if (!(t > 0.0f) || k == 1 || p <= 0.0f) return first;
        mp = mp > 0.0f ? fminf(mp, 1.0f) : 0.0f;
        max = best;
        max_x = best;
        slope = 1.4426950408889634074 / (double)t;
        bins = (float)fmin(slope * 128.0, 3e38);
        const u64 least = (u64)__builtin_ceil((double)mp * SR_ONE);
        Cut cut{kNegInf, 0x7fffffff};
        if (k > 0 || p < 1.0f) {
            for (int j = tid; j < SR_BINS; j += SR_THREADS) {
                s.mass[j] = 0;
                s.count[j] = 0;
            }
            __syncthreads();
            each([&](int, const float(&x)[8]) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (x[j] == kNegInf) continue;
                    const int at = bin(x[j]);
                    atomicAdd(&s.mass[at], weight(x[j]));
                    atomicAdd(&s.count[at], 1u);
                }
            });
            __syncthreads();
            u64 all = 0;
            unsigned many = 0;
            for (int j = tid; j < SR_BINS; j += SR_THREADS) {
                all += s.mass[j];
                many += s.count[j];
            }
            all = wave_sum(all);
            many = wave_sum(many);
            if (lane == 0) {
                s.wave_mass[wave] = all;
                s.wave_count[wave] = many;
            }
            __syncthreads();
            all = 0;
            many = 0;
#pragma unroll
            for (int w = 0; w < SR_WAVES; ++w) {
                all += s.wave_mass[w];
                many += s.wave_count[w];
            }
            __syncthreads();
            if (k > 0 && (unsigned)k < many) {
                cut_row(false, k, 0);
                cut = s.cut;
                all = s.cut_mass;
                __syncthreads();
            }
            if (p < 1.0f) {
                cut_row(true, 0, (u64)__builtin_ceil((double)p * (double)all));
                cut = s.cut;
                __syncthreads();
            }
        }
        return locate(0, true, fmaxf(u, 0.0f), [&](int i, float x) -> u64 {
            if (x < cut.x || (x == cut.x && i > cut.index)) return 0;
            const u64 w = weight(x);
            return w >= least ? w : 0;
        });
    }
};

template <class L>
__global__ __launch_bounds__(SR_THREADS) void k_sample_row(SampleArgs a)
{
    extern __shared__ __align__(16) uint8_t raw[];
    RowShared& s = *reinterpret_cast<RowShared*>(raw);
    for (long r = blockIdx.x; r < a.rows; r += gridDim.x) {
        Sampler<L> w{a, s, (const L*)a.logits + r * a.stride, (int)threadIdx.x & 63,
                     (int)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6), (int)threadIdx.x, 0.0, 0.0, 0.0f, 0.0f};
        const int token = w.draw(r);
        if (threadIdx.x == 0) a.out[r] = token;
        __syncthreads();
    }
}

template <class L>
static hipError_t launch_sample(const SampleArgs& a, hipStream_t st)
{
    static std::atomic<unsigned long long> done{0};
    hipError_t e = allow_full_lds((const void*)k_sample_row<L>, &done);
    if (e != hipSuccess) return e;
    k_sample_row<L><<<dim3((unsigned)(a.rows < (1L << 20) ? a.rows : 1L << 20)), dim3(SR_THREADS), sizeof(RowShared), st>>>(a);
    return hipGetLastError();
}

hipError_t run_sample(int dtype, const void* logits, long rows, int vocab, long stride, const float* u, const float* temperatures,
                      const int* top_ks, const float* top_ps, const float* min_ps, float temperature, int top_k, float top_p,
                      float min_p, int* out, hipStream_t st)
{
    SampleArgs a{logits, stride, u, temperatures, top_ks, top_ps, min_ps, temperature, top_p, min_p, top_k, vocab, rows, out};
    if (dtype == DT_F16) return launch_sample<half_t>(a, st);
    return dtype == DT_BF16 ? launch_sample<bf16_t>(a, st) : launch_sample<float>(a, st);
}

}  // namespace fc

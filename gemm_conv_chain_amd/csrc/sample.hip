// sample.hip -- draws a token from each row of logits: temperature, the top_k
// largest, the least set that holds top_p of the mass, min_p, and one random
// number.
//
// One pass over the logits: a wave takes a batch of 2048, of which it keeps the
// largest, the sum of weights (relative to the batch's largest) where the row
// needs the whole mass, and the largest of each group of 8 or 32 logits where the
// row is cut.  The rest looks at little of the row again (k_sample's second
// part, or k_sample_pick):
//   whole distribution: the sums pick the batch, the batch's logits the token;
//   cut: a histogram of the groups' largest says below which bin of log2 of the
//     weights the wanted ones lie, only groups that reach it are read again, and
//     of what they hold (at most 512) each looks at all the others for its rank and the mass
//     ahead of it, in falling order and then in order of index;
//   cut, and more than 512 stay or might (flat distributions, many ties): the
//     whole row by histograms, to the bin, to the value and to the tie.
// What stays is a prefix of the row in falling order, so that its last element
// describes it: a value and, among equal ones, an index (Cut).  Nothing is sorted.
//
// Weights are 64-bit exponentials, rounded once to integers in units of 2^-42:
// integer sums do not depend on their order, and with it the token.  32-bit
// weights would be off by 1e-7 of the mass, a token in as many million rows.
// A batch's sum, whose unit its own largest is, is brought to the row's by one
// product in 64 bits, rounded down; the row's mass is the sum of these in every
// kernel, so that a row's token does not depend on which of them draw it.
//
// Bound by the vector unit where many rows need their sums (some 25
// instructions of 64 bits a logit; 128 x 131072 in bf16: 17 us for the pass,
// 33.5 MB at 1.9 TB/s, and 8 for the rest), by memory where logits are 32 bits (832 x
// 100003: 63 us, 333 MB at 5.3 TB/s), and for few rows by the chain of
// dependent steps of one block (1 x 32000, top_p 0.95: 21 us in all, 14 of them
// this).  Of 832
// rows with settings of their own, 42 us go to rows drawn from their largest
// and 60 to the flat ones, a CU each: its exponentials twice and the
// histograms.  Sorting a row would be 17 passes of a merge.
#include "fc_launch.h"
#include "kv_common.h"

namespace fc {

typedef unsigned long long u64;

constexpr int SR_BATCH = 2048;     // logits a wave takes at a time, 32 a lane
constexpr int SR_SHORT = 8;        // waves of a block that draws from a row's largest,
constexpr int SR_LONG = 16;        // and from all of a row
constexpr int SR_LIST = 64 * SR_SHORT;   // elements in question that a row's largest may be
constexpr int SR_NUCLEUS = 256;    // logits that a cut by mass alone looks at first
constexpr double SR_ONE = 0x1p42;  // a weight of 1
// In out: the row is k_sample_long's. Such a mark also says how large the row's mass is by its batches'
// sums, which a share of the mass (top_p) is taken of whichever kernels draw the row: SR_NOT_YET less
// that mass's low 30 bits. k_sample_long sums the weights in the row's units, and the two differ by far
// less than 2^29: by half a unit or less a weight on either side (2^20 in all), a unit a batch, and the
// 64-bit rounding of exponentials and products, under 2^-44 of at most 2^62.
constexpr int SR_NOT_YET = -2;
constexpr unsigned SR_MARK = (1u << 30) - 1;
__device__ __forceinline__ int not_yet(u64 mass) { return SR_NOT_YET - (int)((unsigned)mass & SR_MARK); }
__device__ __forceinline__ u64 marked_mass(int mark, u64 near)
{
    const unsigned low = (unsigned)(SR_NOT_YET - mark);
    return near + (long long)((int)((low - (unsigned)near) << 2) >> 2);
}

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
    int batches;            // of a row
    void* info;             // workspace: BatchInfo [rows][batches]
    float* groups;          // and the groups' largest [rows][batches][64]
};

// A batch's info: the bits of its largest, whether it holds a NaN or +inf, and the sum of its
// weights (two halves), its own largest being 1.  One 16-byte access, like an Entry.
typedef u32x4 BatchInfo;
__device__ __forceinline__ float info_max(BatchInfo b) { return __builtin_bit_cast(float, (unsigned)b[0]); }
__device__ __forceinline__ u64 high_pair(u32x4 b) { return (u64)b[3] << 32 | b[2]; }

// A row's settings, as the kernels use them.
struct RowSet {
    double slope, far;      // 32 log2(e) / temperature; the distance at which weights are 0
    float p;
    int k;                  // 0: off
    u64 least;              // the least weight that stays
    bool greedy, cut, sums; // cut: something may go; sums: the whole mass is needed
};

__device__ __forceinline__ RowSet row_set(const SampleArgs& a, long r)
{
    const float t = a.temperatures ? a.temperatures[r] : a.temperature;
    RowSet s;
    s.k = a.top_ks ? a.top_ks[r] : a.top_k;
    s.p = a.top_ps ? a.top_ps[r] : a.top_p;
    const float mp = a.min_ps ? a.min_ps[r] : a.min_p;
    s.greedy = !(t > 0.0f) || s.k == 1 || s.p <= 0.0f;
    if (s.k < 0 || s.k >= a.vocab) s.k = 0;
    s.slope = 32 * 1.4426950408889634074 / (double)fminf(t, 1e30f);
    s.far = -64 * 32 / s.slope;
    s.least = mp > 0.0f ? (u64)__builtin_ceil((double)fminf(mp, 1.0f) * SR_ONE) : 0;
    s.cut = !s.greedy && (s.k > 0 || s.p < 1.0f || s.least > 0);
    s.sums = !s.greedy && s.k == 0 && (s.p < 1.0f || s.least == 0);
    return s;
}

// An element in question: the bits of its logit, its index, its weight (two halves).
typedef u32x4 Entry;
__device__ __forceinline__ Entry entry(float x, int index, u64 w)
{
    return Entry{__builtin_bit_cast(unsigned, x), (unsigned)index, (unsigned)w, (unsigned)(w >> 32)};
}
// Whether a comes before b, in falling order and of equal ones by index.
__device__ __forceinline__ bool before(Entry a, Entry b)
{
    const float x = __builtin_bit_cast(float, (unsigned)a[0]), y = __builtin_bit_cast(float, (unsigned)b[0]);
    return x > y || (x == y && a[1] < b[1]);
}

__device__ __forceinline__ unsigned lds_add(FC_LDS unsigned* p, unsigned v)
{
    return __hip_atomic_fetch_add(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}
__device__ __forceinline__ void lds_add(FC_LDS u64* p, u64 v)
{
    __hip_atomic_fetch_add(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}
__device__ __forceinline__ void lds_min(FC_LDS unsigned* p, unsigned v)
{
    __hip_atomic_fetch_min(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}
__device__ __forceinline__ void lds_max(FC_LDS unsigned* p, unsigned v)
{
    __hip_atomic_fetch_max(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}

// A histogram has a bin a thread, which cover 32 octaves of weights (the last one what is less, too);
// of all of a row each wave keeps its own of the part it has.
template <int WAVES, bool ROW> struct Shared {
    double table[32];
    u64 bins[ROW ? WAVES : 1][64 * WAVES];
    static constexpr int FEW = ROW ? 512 : 128;   // elements of a bin that are looked at one by one
    u32x4 few[FEW];
    u64 extra[WAVES];
    u32x4 list[ROW ? 1 : SR_LIST];
    int chosen[ROW ? 1 : SR_LIST];    // groups
    u64 wave_mass[WAVES];
    float wave_x[WAVES];
    unsigned wave_bad[WAVES];
    unsigned n_list, n_chosen, n_few, key_lo, key_hi;
    int border, token;
    u64 border_before;
    // The cut: an element stays if it is larger, or equal and not behind it.
    float cut_x;
    int cut_i;
    float cut_top;
};

// Eight logits as they lie in memory, at any element; and as floats.
template <class L> struct __attribute__((packed, aligned(sizeof(L)))) Eight {
    L v[8];
};
template <class L> __device__ __forceinline__ void to_floats(const Eight<L>& e, float (&x)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = (float)e.v[j];
}

// The eight that a lane with logits i .. i + 7 loads: the row's last eight where it ends among them
// (rows have eight at least). unpack gives -inf for those that are other lanes', and the first one's
// index. `whole`: no lane of the wave or block is at the row's end.
template <class L> __device__ __forceinline__ Eight<L> fetch(const L* row, int i, int vocab)
{
    const unsigned at = i < vocab - 8 ? i : vocab - 8;
    return *reinterpret_cast<const Eight<L>*>(reinterpret_cast<const char*>(row) + at * (unsigned)sizeof(L));
}
template <class L>
__device__ __forceinline__ int unpack(const Eight<L>& e, int i, int vocab, bool whole, float (&x)[8])
{
    to_floats(e, x);
    if (whole) return i;
    const int at = i < vocab - 8 ? i : vocab - 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = at + j >= i ? x[j] : kNegInf;
    return at;
}

// Unsigned integers in the order of the floats (no NaN; -0 is 0, which it equals).
__device__ __forceinline__ unsigned order_key(float x)
{
    const unsigned b = __builtin_bit_cast(unsigned, x + 0.0f);
    return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_key(unsigned k)
{
    return __builtin_bit_cast(float, k >> 31 ? k & 0x7fffffffu : ~k);
}

// 2^(slope d / 32) + plus for slope d > -32000: a table of 2^(i / 32) (each entry has its own two of
// LDS's 64 banks) times 2^(r / 32), |r| <= 1/2, by its Taylor series, whose next term is 2e-15.
typedef FC_LDS double lds_double;
// a * b + c to a register of its own (the compiler adds in place, after a copy of each constant).
__device__ __forceinline__ double fma_to(double a, double b, double c)
{
    double d;
    asm("v_fma_f64 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "v"(c));
    return d;
}
__device__ __forceinline__ double exp2_down(double d, double slope, double plus, const lds_double* table)
{
    constexpr double shift = 0x1.8p52;
    const double zi = __builtin_fma(d, slope, shift);
    const int n = (int)__builtin_bit_cast(u64, zi);    // nearest integer
    const double r = __builtin_fma(d, slope, shift - zi);
    constexpr double l = 0.693147180559945309417 / 32;
    constexpr double c2 = l * l / 2, c3 = c2 * l / 3, c4 = c3 * l / 4, c5 = c4 * l / 5;
    double p = fma_to(c5, r, c4);
    p = fma_to(p, r, c3);
    p = fma_to(p, r, c2);
    p = fma_to(p, r, l);
    p = fma_to(p, r, 1.0);
    const u64 t = __builtin_bit_cast(u64, table[n & 31]) + ((u64)(unsigned)((n >> 5) << 20) << 32);
    return __builtin_fma(p, __builtin_bit_cast(double, t), plus);
}
// The table, by the first 32 threads: 2^(t / 32) by the series, to its last bits.  A barrier has to follow.
__device__ __forceinline__ void fill_table(lds_double* table, int tid)
{
    if (tid < 32) {
        const double x = 0.693147180559945309417 / 32 * tid;
        double p = 1.0;
#pragma unroll
        for (int k = 17; k > 0; --k) p = __builtin_fma(p, x * (1.0 / k), 1.0);
        table[tid] = p;   // (exactly 1 at 0: a batch that holds the row's largest is not scaled)
    }
}

// The weight of x in units of 2^-42, rounded: 2^((x - max) slope / 32). far: a distance, -64 octaves,
// from which on weights are 0 (that of -inf, too).
__device__ __forceinline__ u64 weight_of(float x, double max, double slope, double far, const lds_double* table)
{
    // 1024 + w: the unit of its last bit is 2^-42
    return __builtin_bit_cast(u64, exp2_down(__builtin_fmax((double)x - max, far), slope, 1024.0, table)) -
           __builtin_bit_cast(u64, 1024.0);
}

// Sum of the lanes up to this one, and of all, in the data path of the lanes' registers.
template <int CTRL, int ROWS> __device__ __forceinline__ u64 moved(u64 v)
{
    const unsigned lo = __builtin_amdgcn_update_dpp(0, (int)(unsigned)v, CTRL, ROWS, 0xf, false);
    const unsigned hi = __builtin_amdgcn_update_dpp(0, (int)(v >> 32), CTRL, ROWS, 0xf, false);
    return (u64)hi << 32 | lo;
}
__device__ __forceinline__ u64 wave_scan(u64 v)
{
    v += moved<0x111, 0xf>(v);   // row_shr 1, 2, 4, 8
    v += moved<0x112, 0xf>(v);
    v += moved<0x114, 0xf>(v);
    v += moved<0x118, 0xf>(v);
    v += moved<0x142, 0xa>(v);   // row_bcast 15, 31
    v += moved<0x143, 0xc>(v);
    return v;
}
__device__ __forceinline__ u64 lane_of(u64 v, int lane)
{
    return (u64)(unsigned)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 | (unsigned)__builtin_amdgcn_readlane((int)(unsigned)v, lane);
}
__device__ __forceinline__ u64 wave_sum(u64 v) { return lane_of(wave_scan(v), 63); }
template <int CTRL, int ROWS> __device__ __forceinline__ float top_moved(float v)
{
    const int i = __builtin_bit_cast(int, v);
    return fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(i, i, CTRL, ROWS, 0xf, false)));
}
__device__ __forceinline__ float wave_top(float v)
{
    v = top_moved<0x111, 0xf>(v);
    v = top_moved<0x112, 0xf>(v);
    v = top_moved<0x114, 0xf>(v);
    v = top_moved<0x118, 0xf>(v);
    v = top_moved<0x142, 0xa>(v);
    v = top_moved<0x143, 0xc>(v);
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// A batch, by one wave: lane l has logits base + 512 v + 8 l + j of it.  Its info, and the largest
// of each lane's 32 logits (SEGS = 4) or of each 8 (SEGS = 1).
template <int SEGS, class L, class G>
__device__ __forceinline__ BatchInfo scan_batch(const L* row, int base, int vocab, int lane, const RowSet& set, G groups,
                                                const lds_double* table)
{
    const bool whole = base + SR_BATCH <= vocab;
    const int i = base + 8 * lane;
    Eight<L> e[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) e[v] = fetch(row, i + 512 * v, vocab);
    float top[4];
    bool bad = false;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        float x[8];
        unpack(e[v], i + 512 * v, vocab, whole, x);
        top[v] = x[0];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            bad |= !(x[j] < __builtin_inff());
            top[v] = fmaxf(top[v], x[j]);
        }
    }
    const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    if (set.cut) {
        if (SEGS == 4) groups[lane] = most;
        else
#pragma unroll
            for (int v = 0; v < 4; ++v) groups[64 * v + lane] = top[v];
    }
    const float all = wave_top(most);
    u64 sum = 0;
    if (set.sums) {
        const double max = all;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            u32x4* w = reinterpret_cast<u32x4*>(&e[v]);   // (converted again: the floats of all four are 32 registers)
#pragma unroll
            for (int k = 0; k < (int)sizeof(e[v]) / 16; ++k) asm volatile("" : "+v"(w[k]));
            float x[8];
            unpack(e[v], i + 512 * v, vocab, whole, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sum += weight_of(x[j], max, set.slope, set.far, table);
                if (j % 4 == 3) {   // four exponentials at a time: all 32 take 200 registers
                    asm volatile("" : "+v"(sum));
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        sum = wave_sum(sum);
    }
    return BatchInfo{__builtin_bit_cast(unsigned, all), __any(bad) ? 1u : 0u, (unsigned)sum, (unsigned)(sum >> 32)};
}

// What a block does with a row: ROW by all of its logits, else by its largest (of the infos and groups
// of its batches).
template <class L, int WAVES, bool ROW> struct Sampler {
    static constexpr int THREADS = 64 * WAVES, BINS = THREADS, FEW = Shared<WAVES, ROW>::FEW;
    static constexpr int LOOK = sizeof(L) == 2 ? 3 : 2;   // loads on the way where little is done with them
    const SampleArgs& a;
    FC_LDS Shared<WAVES, ROW>& s;
    const L* row;
    const int lane, wave, tid;
    RowSet set;
    double max;
    float max_x, unit;      // bins of the histogram a unit of x
    int mark;               // (ROW: what out held)

    __device__ __forceinline__ u64 weight(float x) const { return weight_of(x, max, set.slope, set.far, s.table); }
    __device__ __forceinline__ int bin(float x) const { return (int)fminf((max_x - x) * unit, (float)(BINS - 1)); }
    // The least key of a logit in bin b or one before it: from an estimate, by steps that double and then halve.
    __device__ __forceinline__ unsigned edge(int b) const
    {
        const unsigned least = order_key(-3.402823466e38f), most = order_key(max_x);
        if (b >= BINS - 1) return least;
        if (b < 0) return most + 1;
        unsigned k = order_key(max_x - (float)(b + 1) / unit);
        k = k < least ? least : k > most ? most : k;
        auto in = [&](unsigned key) { return bin(from_key(key)) <= b; };
        unsigned no, yes, step = 1;   // `no` is below, `yes` at or above
        if (in(k)) {
            yes = k;
            for (no = k; no > least && in(no); step *= 2) {
                yes = no;
                no = no - least > step ? no - step : least;
            }
            if (in(no)) return no;
        } else {
            no = k;
            for (yes = k; !in(yes); step *= 2) {
                no = yes;
                yes = most - yes > step ? yes + step : most;
            }
        }
        while (yes - no > 1) {
            const unsigned mid = no + (yes - no) / 2;
            if (in(mid)) yes = mid;
            else no = mid;
        }
        return yes;
    }
    __device__ __forceinline__ float unit_of() const { return (float)fmin(set.slope * (BINS / 1024.0), 3e38); }   // (slope: 32 an octave)
    __device__ __forceinline__ bool stays(float x, int i, float cut_x, int cut_i) const
    {
        return x > cut_x || (x == cut_x && i <= cut_i);
    }

    // f(index, logit, weight()) for lo .. hi - 1, by one wave: lo and, but for the row's end, hi are
    // multiples of 512. -inf for what is past the row's end. Four logits' work together: more take more
    // registers than there are.
    // U: loads of this step, and as many of the next on the way.
    template <int U, class F> __device__ __forceinline__ void each(int lo, int hi, F&& f) const
    {
        Eight<L> next[U];
#pragma unroll
        for (int k = 0; k < U; ++k) next[k] = fetch(row, lo + lane * 8 + k * 512, a.vocab);
#pragma unroll 1
        for (int base = lo; base < hi; base += 512 * U) {
            Eight<L> e[U];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                e[k] = next[k];
                next[k] = fetch(row, base + 512 * (U + k) + lane * 8, a.vocab);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int b = base + k * 512;
                if (b >= hi) break;
                float x[8];
                const int at = unpack(e[k], b + lane * 8, a.vocab, b + 512 <= a.vocab, x);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float y = x[j];
                    f(at + j, y, [&] { return weight(y); });
                    if (j % 4 == 3) __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
    }

    // The same as sources of elements: all of the row (a wave has a sixteenth of it), n elements of
    // s.list, n groups' largest (as weights 1).
    __device__ __forceinline__ int part() const { return ((a.vocab + WAVES - 1) / WAVES + 511) / 512 * 512; }
    template <int U> struct Whole {
        const Sampler& p;
        template <class F> __device__ __forceinline__ void operator()(F&& f) const
        {
            const int per = p.part(), lo = p.wave * per, hi = lo + per < p.a.vocab ? lo + per : p.a.vocab;
            p.template each<U>(lo, hi, f);
        }
    };
    struct Listed {
        const Sampler& p;
        int n;
        template <class F> __device__ __forceinline__ void operator()(F&& f) const
        {
            if (p.tid < n) {
                const Entry e = p.s.list[p.tid];
                f((int)e[1], __builtin_bit_cast(float, (unsigned)e[0]), [&] { return high_pair(e); });
            }
        }
    };
    template <class G> struct Tops {
        const Sampler& p;
        G groups;
        int n;
        template <class F> __device__ __forceinline__ void operator()(F&& f) const
        {
            for (int g = p.tid; g < n; g += THREADS) f(g, groups[g], [] { return (u64)1; });
        }
    };

    __device__ __forceinline__ u64 block_sum(u64 v)
    {
        v = wave_sum(v);
        if (lane == 0) s.wave_mass[wave] = v;
        __syncthreads();
        u64 all = 0;
#pragma unroll
        for (int k = 0; k < WAVES; ++k) all += s.wave_mass[k];
        __syncthreads();
        return all;
    }

    // u times the whole, less than it.
    __device__ __forceinline__ u64 goal_of(float u, u64 all) const
    {
        const u64 g = (u64)((double)fmaxf(u, 0.0f) * (double)all);
        return u < 1.0f && g < all ? g : all - 1;
    }

    template <bool ALL = true> __device__ __forceinline__ void clear_bins()   // (ALL false: one copy)
    {
        if (ROW && ALL) {
            FC_LDS u32x4* const p = (FC_LDS u32x4*)s.bins;
#pragma unroll
            for (int k = 0; k < WAVES / 2; ++k) p[k * THREADS + tid] = u32x4{0, 0, 0, 0};
        } else {
            s.bins[0][tid] = 0;
        }
        if (tid == 0) s.border = -1;
        __syncthreads();
    }
    __device__ __forceinline__ void add_bin(int b, u64 v) { lds_add(&s.bins[ROW ? wave : 0][b], v); }
    // The bin at which the running sum reaches goal, -1 where none does; *before: the sum ahead of it.
    template <bool ALL = true> __device__ __forceinline__ int find_bin(u64 goal, u64* before)
    {
        __syncthreads();
        if constexpr (kPoison) lds_poison(s.few, sizeof(s.few), tid, THREADS);   // free from here on
        if (tid == 0) {
            s.n_few = 0;
            s.key_lo = ~0u;
            s.key_hi = 0;
        }
        if (tid < WAVES) s.extra[tid] = 0;
        u64 v = s.bins[0][tid];
        if (ROW && ALL)
#pragma unroll
            for (int k = 1; k < WAVES; ++k) v += s.bins[ROW ? k : 0][tid];
        u64 upto = wave_scan(v);
        if (lane == 63) s.wave_mass[wave] = upto;
        __syncthreads();
        for (int w = 0; w < wave; ++w) upto += s.wave_mass[w];
        if (upto >= goal && upto - v < goal) {
            s.border = tid;
            s.border_before = upto - v;
        }
        __syncthreads();
        *before = s.border_before;
        return s.border;
    }

    // Of the steps of 512 logits from lo on, the first before hi at which the running sum of w(index,
    // x) passes goal; for the first wave (16 that do the same take each other's time).
    template <int STEPS, class W> __device__ __forceinline__ int locate_here(int lo, int hi, u64 goal, W&& w)
    {
        if (wave > 0) return 0;
        Eight<L> e[STEPS];
#pragma unroll
        for (int v = 0; v < STEPS; ++v) e[v] = fetch(row, lo + v * 512 + lane * 8, a.vocab);
#pragma unroll
        for (int v = 0; v < STEPS; ++v) {
            float x[8];
            const int i = unpack(e[v], lo + v * 512 + lane * 8, a.vocab, false, x);
            u64 own[8], sum = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                own[j] = x[j] > kNegInf && i + j < hi ? w(i + j, x[j]) : 0;
                sum += own[j];
            }
            __builtin_amdgcn_sched_barrier(0);
            const u64 upto = wave_scan(sum);
            const u64 past = __ballot(upto > goal);
            if (past || v == STEPS - 1) {
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
            goal -= lane_of(upto, 63);
        }
        return 0;
    }

    // The first index of the row at which the running sum of w(index, x, weight()) passes goal, or
    // with `draw` u times the whole sum; for the first wave. known: this wave's part of the row has
    // the sum `mine`.
    template <class W> __device__ __forceinline__ int locate(u64 goal, bool draw, float u, bool known, u64 mine, W&& w)
    {
        int lo = 0, hi = a.vocab;
        while (hi - lo > 512 || draw) {
            const int per = ((hi - lo + WAVES - 1) / WAVES + 511) / 512 * 512;
            const int z = lo + (wave + 1) * per < hi ? lo + (wave + 1) * per : hi;
            u64 sum = 0;
            if (!known) each<2>(lo + wave * per, z, [&](int i, float x, auto&& weight) { sum += w(i, x, weight); });
            sum = known ? mine : wave_sum(sum);
            known = false;
            if (lane == 0) s.wave_mass[wave] = sum;
            __syncthreads();
            if (draw) {
                u64 all = 0;
#pragma unroll
                for (int k = 0; k < WAVES; ++k) all += s.wave_mass[k];
                goal = goal_of(u, all);
                draw = false;
            }
            int at = 0;
            for (; at < WAVES - 1 && goal >= s.wave_mass[at]; ++at) goal -= s.wave_mass[at];
            lo += at * per;
            hi = lo + per < hi ? lo + per : hi;
            __syncthreads();   // wave_mass is free
        }
        return locate_here<1>(lo, hi, goal, [&](int i, float x) { return w(i, x, [&] { return weight(x); }); });
    }

    // A histogram of which(x) over the source's elements, of their weights or (MASS false) number.
    // The last bin's, which may be most of them (-inf among them, as nothing), are added up in registers.
    template <bool MASS, class S, class B> __device__ __forceinline__ void fill_bins(const S& source, B&& which)
    {
        clear_bins();
        u64 rest = 0;
        source([&](int, float x, auto&& weight) {
            const int b = which(x);
            if (b < 0) return;
            u64 v = x > kNegInf;
            if constexpr (MASS) v = weight();
            if (b == BINS - 1) rest += v;
            else add_bin(b, v);
        });
        rest = wave_sum(rest);
        if (lane == 0 && rest) add_bin(BINS - 1, rest);
    }

    // Of n elements, a thread each (`live`), with keys lo .. hi, the one at which the running sum of their
    // weights in falling order reaches goal, to s.cut_x and s.cut_i: by histograms until at most 64
    // are left, or equal ones, and of these each looks at all.
    __device__ __forceinline__ void pick_few(Entry e, bool live, int n, u64 goal, unsigned lo, unsigned hi)
    {
        const unsigned key = order_key(__builtin_bit_cast(float, (unsigned)e[0]));
        const u64 w = high_pair(e);
        while (n > 64 && lo < hi) {
            int shift = 0;
            while ((hi - lo) >> shift >= BINS) ++shift;
            __syncthreads();   // everyone has read what the counts are reset of
            clear_bins<false>();
            if (live) lds_add(&s.bins[0][(hi - key) >> shift], w);
            u64 ahead;
            const int b = find_bin<false>(goal, &ahead);
            goal -= ahead;
            live = live && (int)((hi - key) >> shift) == b;
            if (live) {
                s.few[lds_add(&s.n_few, 1u)] = e;
                lds_min(&s.key_lo, key);
                lds_max(&s.key_hi, key);
            }
            __syncthreads();
            n = s.n_few;
            lo = s.key_lo;
            hi = s.key_hi;
        }
        if (live) {
            u64 m = 0;
#pragma unroll 4
            for (int j = 0; j < n; ++j) {
                const Entry y = s.few[j];
                m += before(y, e) ? high_pair(y) : 0;
            }
            if (m < goal && m + w >= goal) {
                s.cut_x = __builtin_bit_cast(float, (unsigned)e[0]);
                s.cut_i = e[1];
            }
        }
        __syncthreads();
    }

    // The last element that stays, in s.cut_x and s.cut_i: the goal-th in falling order, or (MASS)
    // that at which the mass reaches goal; `share` > 0: that share of the marked mass.  False where there are not so many.  `tie(many, x)`: the
    // index of the many-th element that is x.  Of a row, *mine: the sum of this wave's part in the bins
    // before the cut's, whose largest value may be s.cut_top; or (cut_top -inf) with what stays of that.
    // `look`: the source, for passes that do little.
    template <bool MASS, class S, class Q, class T>
    __device__ __forceinline__ bool cut_at(const S& source, const Q& look, u64 goal, float share, T&& tie, u64* mine)
    {
        fill_bins<MASS>(source, [&](float x) { return bin(x); });
        if (ROW && share > 0.0f) {
            __syncthreads();
            u64 v = 0;
#pragma unroll
            for (int k = 0; k < WAVES; ++k) v += s.bins[ROW ? k : 0][tid];
            goal = (u64)__builtin_ceil((double)share * (double)marked_mass(mark, block_sum(v)));
        }
        u64 ahead;
        const int b = find_bin(goal, &ahead);
        if (b < 0) return false;
        if (ROW) {
            u64 sum = 0;
            for (int k = lane; k < b; k += 64) sum += s.bins[ROW ? wave : 0][k];
            *mine = wave_sum(sum);
            if (tid == 0) s.cut_top = from_key(edge(b - 1) - 1);
        }
        goal -= ahead;
        unsigned lo = edge(b), hi = edge(b - 1) - 1;   // keys of the elements in question, the bin's at first
        for (bool all = true;; all = false) {   // all: of the bin's elements
            const float xa = from_key(lo), xb = from_key(hi);
            unsigned least = ~0u, most = 0;
            look([&](int i, float x, auto&& weight) {
                if (!(x >= xa && x <= xb)) return;
                const unsigned key = order_key(x);
                least = key < least ? key : least;
                most = key > most ? key : most;
                const u64 here = __ballot(true);
                const int first = __builtin_ctzll(here);
                unsigned at = 0;
                if (lane == first) at = lds_add(&s.n_few, (unsigned)__builtin_popcountll(here));
                at = __builtin_amdgcn_readlane(at, first) + __builtin_popcountll(here & ((1ull << lane) - 1));
                if (at < FEW) {
                    u64 w = 1;
                    if constexpr (MASS) w = weight();
                    s.few[at] = entry(x, i, w);
                }
            });
            if (most) {
                lds_min(&s.key_lo, least);
                lds_max(&s.key_hi, most);
            }
            __syncthreads();
            const int few = s.n_few;
            if (few <= FEW) {
                const bool mine_too = tid < few;
                const Entry e = mine_too ? s.few[tid] : Entry{0, 0, 0, 0};
                pick_few(e, mine_too, few, goal, s.key_lo, s.key_hi);
                if (ROW && MASS && all) {   // those that stay, to their parts' sums
                    if (mine_too) {
                        const int i = e[1];
                        if (stays(__builtin_bit_cast(float, (unsigned)e[0]), i, s.cut_x, s.cut_i)) lds_add(&s.extra[i / part()], high_pair(e));
                    }
                    if (tid == 0) s.cut_top = kNegInf;
                    __syncthreads();
                    *mine += s.extra[wave];
                }
                return true;
            }
            lo = s.key_lo;
            hi = s.key_hi;
            if (lo == hi) {       // all equal: the first few by index
                const float x = from_key(lo);
                const u64 w = MASS ? weight(x) : 1;
                const int index = tie((goal + w - 1) / w, x);
                if (tid == 0) {
                    s.cut_x = x;
                    s.cut_i = index;
                }
                __syncthreads();
                return true;
            }
            int shift = 0;
            while ((hi - lo) >> shift >= BINS) ++shift;
            const float ya = from_key(lo), yb = from_key(hi);
            fill_bins<MASS>(source, [&](float x) { return x >= ya && x <= yb ? (int)((hi - order_key(x)) >> shift) : -1; });
            const int sub = find_bin(goal, &ahead);
            goal -= ahead;
            const unsigned top = hi - ((unsigned)sub << shift);   // the largest key of the sub-bin
            const unsigned span = (1u << shift) - 1;
            lo = top - lo > span ? top - span : lo;
            hi = top;
        }
    }

    // Of the list, the first in order of index at which the running sum of w(index, x, weight) passes goal.
    template <class W> __device__ __forceinline__ int index_at(u64 goal, int n, W&& w)
    {
        int shift = 0;
        while ((a.vocab - 1) >> shift >= BINS) ++shift;
        clear_bins();
        const Entry e = tid < n ? s.list[tid] : Entry{0, 0, 0, 0};
        const u64 own = tid < n ? w((int)e[1], __builtin_bit_cast(float, (unsigned)e[0]), high_pair(e)) : 0;
        if (own) add_bin(e[1] >> shift, own);
        u64 ahead;
        const int b = find_bin(goal + 1, &ahead);
        goal -= ahead;
        // (a bin has 2^shift indices: up to FEW of the list here, else they are searched in the list)
        const bool mine = own && (int)(e[1] >> shift) == b;
        unsigned at = 0;
        if (mine) {
            at = lds_add(&s.n_few, 1u);
            if (at < FEW) s.few[at] = entry(0.0f, e[1], own);
        }
        __syncthreads();
        const int few = s.n_few;
        if (mine) {
            u64 m = 0;
            if (few <= FEW) {
                for (int j = 0; j < few; ++j) {
                    const Entry y = s.few[j];
                    m += y[1] < e[1] ? high_pair(y) : 0;
                }
            } else {
                for (int j = 0; j < n; ++j) {
                    const Entry y = s.list[j];
                    if ((int)(y[1] >> shift) == b && y[1] < e[1])
                        m += w((int)y[1], __builtin_bit_cast(float, (unsigned)y[0]), high_pair(y));
                }
            }
            if (m <= goal && goal < m + own) s.token = e[1];
        }
        __syncthreads();
        return s.token;
    }

    // A cut row, from all of it.
    __device__ __forceinline__ int draw_long(float u)
    {
        float cut_x = kNegInf;
        int cut_i = 0x7fffffff;
        const Whole<2> source{*this};
        const Whole<LOOK> look{*this};
        u64 mine = 0;
        const auto tie = [&](u64 many, float x) {
            return locate(many - 1, false, 0.0f, false, 0, [&](int, float y, auto&&) { return y == x ? 1ull : 0ull; });
        };
        if (set.k > 0) {
            if (cut_at<false>(look, look, set.k, 0.0f, tie, &mine)) {
                cut_x = s.cut_x;
                cut_i = s.cut_i;
            }
            __syncthreads();
        }
        if (set.p < 1.0f) {
            u64 left = 0;   // of what top_k left, or of the whole
            if (set.k > 0) {
                source([&](int i, float x, auto&& weight) { left += stays(x, i, cut_x, cut_i) ? weight() : 0; });
                left = (u64)__builtin_ceil((double)set.p * (double)block_sum(left));
            }
            if (cut_at<true>(source, look, left, set.k > 0 ? 0.0f : set.p, tie, &mine)) {
                cut_x = s.cut_x;
                cut_i = s.cut_i;
            }
            __syncthreads();
        }
        // Cut by mass alone: the parts' sums before the cut's bin are there, that bin's are added.
        const bool known = set.k == 0 && set.least == 0 && cut_x > kNegInf;
        const float top = s.cut_top;
        if (known && top > kNegInf) {
            u64 sum = 0;
            look([&](int i, float x, auto&& weight) {
                if (x <= top && stays(x, i, cut_x, cut_i)) sum += weight();
            });
            mine += wave_sum(sum);
        }
        return locate(0, true, u, known, mine, [&](int i, float x, auto&& weight) -> u64 {
            if (!stays(x, i, cut_x, cut_i)) return 0;
            const u64 w = weight();
            return w >= set.least ? w : 0;
        });
    }

    // The same from the n elements of s.list. not_yet: their mass is too little (floored: what they
    // lack would not stay).
    __device__ __forceinline__ int draw_short(int n, bool floored, u64 all, float u)
    {
        float cut_x = kNegInf;
        int cut_i = 0x7fffffff;
        const Listed source{*this, n};
        const Entry e = tid < n ? s.list[tid] : Entry{0, 0, 0, 0};
        const float x = __builtin_bit_cast(float, (unsigned)e[0]);
        u64 w = tid < n ? high_pair(e) : 0;
        const auto tie = [&](u64 many, float y) {
            return index_at(many - 1, n, [&](int, float z, u64) { return z == y ? 1ull : 0ull; });
        };
        if (set.k > 0) {
            if (cut_at<false>(source, source, set.k, 0.0f, tie, nullptr)) {
                cut_x = s.cut_x;
                cut_i = s.cut_i;
            }
            __syncthreads();
        }
        if (set.p < 1.0f) {
            if (set.k > 0) all = block_sum(stays(x, e[1], cut_x, cut_i) ? w : 0);
            if (cut_at<true>(source, source, (u64)__builtin_ceil((double)set.p * (double)all), 0.0f, tie, nullptr)) {
                cut_x = s.cut_x;
                cut_i = s.cut_i;
            } else if (!floored) {
                return not_yet(all);
            }
            __syncthreads();
        }
        const auto left = [&](int i, float x, u64 w) { return stays(x, i, cut_x, cut_i) && w >= set.least ? w : 0; };
        w = w ? left((int)e[1], x, w) : 0;
        return index_at(goal_of(u, block_sum(w)), n, left);
    }

    // Logits of a cut row that are wanted at least, as far as top_k or top_p says.
    __device__ __forceinline__ int wanted() const { return set.k > 0 ? set.k : set.p < 1.0f ? SR_NUCLEUS : 0x7fffffff; }

    // The elements in question of a cut row, if there are at most SR_LIST: into s.list; their number,
    // or -1.  *floored: those of less than the least weight are not among them.
    template <int SEGS, class G> __device__ __forceinline__ int gather(G groups, int ngroups, bool again, bool* floored)
    {
        *floored = false;
        if (set.k > SR_LIST) return -1;
        if constexpr (kPoison) {   // all of a call before is done with these
            lds_poison(s.list, sizeof(s.list), tid, THREADS);
            lds_poison(s.chosen, sizeof(s.chosen), tid, THREADS);
            if (tid == 0) s.n_list = s.n_chosen = kPoisonWord;
            __syncthreads();
        }
        const int first = wanted();
        // The least logit in question: so many groups hold one each down to a bin, or (the second time)
        // down to a value.
        float floor = kNegInf;
        if (first <= ngroups) {
            const Tops<G> source{*this, groups, ngroups};
            if (again) {
                if (cut_at<false>(source, source, first, 0.0f, [](u64, float) { return 0; }, nullptr)) floor = s.cut_x;
            } else {
                fill_bins<false>(source, [&](float x) { return bin(x); });
                u64 ahead;
                const int b = find_bin(first, &ahead);
                if (b >= 0) floor = from_key(edge(b));
            }
        }
        if (set.least > 0 && !(set.k > 0 && set.p < 1.0f)) {   // nor are the lesser weights counted in p
            // (the logarithm is good to 1e-6, the products to 2^-23)
            const float z = -__builtin_amdgcn_logf((float)set.least * (float)(1.0 / SR_ONE)) * 1.00001f + 0.001f;
            const float x = max_x - (float)((double)z * 32 / set.slope);
            const float lower = x - fabsf(x) * 1e-6f;
            *floored = lower > floor;
            floor = fmaxf(floor, lower);
        }
        if (tid == 0) s.n_list = s.n_chosen = 0;
        __syncthreads();
        for (int g = tid; g < ngroups; g += THREADS) {
            const float x = groups[g];
            if (x > kNegInf && x >= floor) {
                const unsigned at = lds_add(&s.n_chosen, 1u);
                if (at < SR_LIST) s.chosen[at] = g;
            }
        }
        __syncthreads();
        const int nc = s.n_chosen;
        if (nc > SR_LIST) {            // (each holds one at least)
            __syncthreads();           // every wave has read the count, which a second call resets
            return -1;
        }
        for (int e = tid; e < nc * SEGS; e += THREADS) {
            const int g = s.chosen[e / SEGS];
            // group g of 32: lane g % 64 of batch g / 64; of 8: lane g % 64 of a batch's quarter g / 64
            const int i = SEGS == 4 ? (g >> 6) * SR_BATCH + (e % SEGS) * 512 + (g & 63) * 8 : (g >> 6) * 512 + (g & 63) * 8;
            if (i >= a.vocab) continue;
            float x[8];
            const int at = unpack(fetch(row, i, a.vocab), i, a.vocab, false, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (!(x[j] > kNegInf && x[j] >= floor)) continue;
                const unsigned to = lds_add(&s.n_list, 1u);
                if (to < SR_LIST) s.list[to] = entry(x[j], at + j, 0);
            }
        }
        __syncthreads();
        const int n = s.n_list;
        if (n > SR_LIST) {
            __syncthreads();           // (as above)
            return -1;
        }
        if (tid < n) {
            const Entry e = s.list[tid];
            s.list[tid] = entry(__builtin_bit_cast(float, (unsigned)e[0]), e[1], weight(__builtin_bit_cast(float, (unsigned)e[0])));
        }
        __syncthreads();
        return n;
    }

    // The row's token from its batches' infos and groups.
    template <int SEGS, class I, class G> __device__ __forceinline__ int draw(long r, I infos, G groups)
    {
        float top = kNegInf;
        unsigned bad = 0;
        for (int b = tid; b < a.batches; b += THREADS) {
            const BatchInfo i = infos[b];
            top = fmaxf(top, info_max(i));
            bad |= i[1];
        }
        top = wave_top(top);
        bad = __any(bad != 0);
        if (lane == 0) {
            s.wave_x[wave] = top;
            s.wave_bad[wave] = bad;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < WAVES; ++k) {
            top = fmaxf(top, s.wave_x[k]);
            bad |= s.wave_bad[k];
        }
        const float u = a.u[r];
        if (bad || top == kNegInf || u != u) return -1;
        max = max_x = top;
        unit = unit_of();
        if (set.greedy) {   // the first batch that has it, and its place there
            if (tid == 0) s.key_lo = ~0u;
            __syncthreads();
            for (int b = tid; b < a.batches; b += THREADS)
                if (info_max(infos[b]) == top) lds_min(&s.key_lo, (unsigned)b);
            __syncthreads();
            const int lo = s.key_lo * SR_BATCH, hi = lo + SR_BATCH < a.vocab ? lo + SR_BATCH : a.vocab;
            return locate_here<4>(lo, hi, 0, [&](int, float x) { return x == top ? 1ull : 0ull; });
        }
        if (set.cut) {
            u64 all = 0;
            if (set.sums) {
                for (int b = tid; b < a.batches; b += THREADS) all += joined(infos[b]);
                all = block_sum(all);
            }
            bool floored;
            const int ngroups = a.batches * (SEGS == 4 ? 64 : 256);
            const int times = wanted() <= ngroups ? 2 : 1;   // (where the groups say nothing, a second look finds the same)
            int n = -1;
#pragma unroll 1
            for (int again = 0; again < times && n < 0; ++again) n = gather<SEGS>(groups, ngroups, again, &floored);
            return n < 0 ? not_yet(all) : draw_short(n, floored, all, u);
        }
        // the batch that u lies in: thread t has `per` batches
        const int per = (a.batches + THREADS - 1) / THREADS;
        u64 sum = 0;
        for (int b = tid * per; b < (tid + 1) * per && b < a.batches; ++b) sum += joined(infos[b]);
        u64 upto = wave_scan(sum), all = 0;
        if (lane == 63) s.wave_mass[wave] = upto;
        __syncthreads();
        upto -= sum;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            upto += w < wave ? s.wave_mass[w] : 0;
            all += s.wave_mass[w];
        }
        u64 goal = goal_of(u, all);
        for (int b = tid * per; b < (tid + 1) * per && b < a.batches; ++b) {
            const u64 w = joined(infos[b]);
            if (upto <= goal && goal < upto + w) {
                s.border = b;
                s.border_before = upto;
            }
            upto += w;
        }
        __syncthreads();
        const int b = s.border, lo = b * SR_BATCH, hi = lo + SR_BATCH < a.vocab ? lo + SR_BATCH : a.vocab;
        const BatchInfo info = infos[b];
        // in the batch's own units
        goal = (u64)((double)(goal - s.border_before) / scale_of(info));
        goal = goal < high_pair(info) ? goal : high_pair(info) - 1;
        const double m = info_max(info);
        return locate_here<4>(lo, hi, goal, [&](int, float x) { return weight_of(x, m, set.slope, set.far, s.table); });
    }

    // What brings a batch's weights to the row's.
    __device__ __forceinline__ double scale_of(BatchInfo b) const
    {
        return exp2_down(__builtin_fmax((double)info_max(b) - max, 14 * set.far), set.slope, 0.0, s.table);
    }
    __device__ __forceinline__ u64 joined(BatchInfo b) const { return (u64)((double)high_pair(b) * scale_of(b)); }
};

// Poison build: all that the block has, and `more` bytes behind it.
template <int WAVES, bool ROW>
__device__ __forceinline__ void poison_shared(FC_LDS Shared<WAVES, ROW>& s, int more, int tid)
{
    if constexpr (kPoison) {
        lds_poison(&s, sizeof s + more, tid, 64 * WAVES);
        __syncthreads();
    }
}

// One block a row: the infos and groups stay in LDS (vocabularies to 32768).
template <class L>
__global__ __launch_bounds__(64 * SR_SHORT) void k_sample(SampleArgs a)
{
    extern __shared__ __align__(16) uint8_t raw[];
    FC_LDS Shared<SR_SHORT, false>& s = *(FC_LDS Shared<SR_SHORT, false>*)raw;
    FC_LDS BatchInfo* const infos = (FC_LDS BatchInfo*)(&s + 1);
    FC_LDS float* const groups = (FC_LDS float*)(infos + a.batches);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    poison_shared(s, a.batches * (sizeof(BatchInfo) + 1024), threadIdx.x);
    fill_table(s.table, threadIdx.x);
    __syncthreads();
    for (long r = blockIdx.x; r < a.rows; r += gridDim.x) {
        Sampler<L, SR_SHORT, false> w{a, s, (const L*)a.logits + r * a.stride, lane, wave, (int)threadIdx.x, row_set(a, r), 0.0, 0.0f, 0.0f, 0};
        for (int b = wave; b < a.batches; b += SR_SHORT) {
            const BatchInfo info = scan_batch<1>(w.row, b * SR_BATCH, a.vocab, lane, w.set, groups + b * 256, s.table);
            if (lane == 0) infos[b] = info;
        }
        __syncthreads();
        const int token = w.template draw<1>(r, infos, groups);
        if (threadIdx.x == 0) a.out[r] = token;
        __syncthreads();
    }
}

// Others: the pass over the logits by as many blocks as there is work for,
constexpr int SR_SCAN = 4;   // waves a block
template <class L>
__global__ __launch_bounds__(64 * SR_SCAN, sizeof(L) == 2 ? 5 : 4) void k_sample_scan(SampleArgs a)
{
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int b = blockIdx.x * SR_SCAN + wave;
    __shared__ double table[32];
    fill_table((lds_double*)table, threadIdx.x);
    __syncthreads();
    if (b >= a.batches) return;
    for (long r = blockIdx.y; r < a.rows; r += gridDim.y) {
        const RowSet set = row_set(a, r);
        const long at = r * a.batches + b;
        const BatchInfo info = scan_batch<4>((const L*)a.logits + r * a.stride, b * SR_BATCH, a.vocab, lane, set, a.groups + at * 64, (lds_double*)table);
        if (lane == 0) ((BatchInfo*)a.info)[at] = info;
    }
}

// and one block a row for the rest.
template <class L>
__global__ __launch_bounds__(64 * SR_SHORT) void k_sample_pick(SampleArgs a)
{
    extern __shared__ __align__(16) uint8_t raw[];
    FC_LDS Shared<SR_SHORT, false>& s = *(FC_LDS Shared<SR_SHORT, false>*)raw;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    poison_shared(s, 0, threadIdx.x);
    fill_table(s.table, threadIdx.x);
    __syncthreads();
    for (long r = blockIdx.x; r < a.rows; r += gridDim.x) {
        Sampler<L, SR_SHORT, false> w{a, s, (const L*)a.logits + r * a.stride, lane, wave, (int)threadIdx.x, row_set(a, r), 0.0, 0.0f, 0.0f, 0};
        const int token = w.template draw<4>(r, (const BatchInfo*)a.info + r * a.batches, (const float*)a.groups + r * a.batches * 64);
        if (threadIdx.x == 0) a.out[r] = token;
        __syncthreads();
    }
}

// Cut rows that have no token yet: one block each.
template <class L>
__global__ __launch_bounds__(64 * SR_LONG) void k_sample_long(SampleArgs a)
{
    extern __shared__ __align__(16) uint8_t raw[];
    FC_LDS Shared<SR_LONG, true>& s = *(FC_LDS Shared<SR_LONG, true>*)raw;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    bool filled = false;
    poison_shared(s, 0, threadIdx.x);
    for (long r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int mark = __builtin_amdgcn_readfirstlane(a.out[r]);
        if (mark > SR_NOT_YET) continue;
        if (!filled) fill_table(s.table, threadIdx.x);
        filled = true;
        Sampler<L, SR_LONG, true> w{a, s, (const L*)a.logits + r * a.stride, lane, wave, (int)threadIdx.x, row_set(a, r), 0.0, 0.0f, 0.0f, mark};
        float top = kNegInf;
        if (a.info) {
            const BatchInfo* const infos = (const BatchInfo*)a.info + r * a.batches;
            for (int b = threadIdx.x; b < a.batches; b += 64 * SR_LONG) top = fmaxf(top, info_max(infos[b]));
        } else {
            typename Sampler<L, SR_LONG, true>::template Whole<2>{w}([&](int, float x, auto&&) { top = fmaxf(top, x); });
        }
        top = wave_top(top);
        if (lane == 0) s.wave_x[wave] = top;
        __syncthreads();
        for (int k = 0; k < SR_LONG; ++k) top = fmaxf(top, s.wave_x[k]);
        w.max = w.max_x = top;
        w.unit = w.unit_of();
        const int token = w.draw_long(a.u[r]);
        __syncthreads();   // (every wave has read out[r])
        if (threadIdx.x == 0) a.out[r] = token;
    }
}

// Rows of fewer than eight logits, which the loads above cannot take: a thread each.
template <class L>
__global__ __launch_bounds__(64) void k_sample_tiny(SampleArgs a)
{
    __shared__ double table[32];
    fill_table((lds_double*)table, threadIdx.x);
    __syncthreads();
    const long r = (long)blockIdx.x * 64 + threadIdx.x;
    if (r >= a.rows) return;
    const L* const row = (const L*)a.logits + r * a.stride;
    const RowSet set = row_set(a, r);
    const int n = a.vocab;
    float x[7];
    float top = kNegInf;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 7; ++i) {
        x[i] = i < n ? (float)row[i] : kNegInf;
        bad |= !(x[i] < __builtin_inff());
        top = fmaxf(top, x[i]);
    }
    const float u = a.u[r];
    int token = -1;
    if (!bad && top > kNegInf && u == u) {
        u64 w[7], all = 0;
        int rank[7];
#pragma unroll
        for (int i = 0; i < 7; ++i) {
            rank[i] = 0;
#pragma unroll
            for (int j = 0; j < 7; ++j) rank[i] += x[j] > x[i] || (x[j] == x[i] && j < i);
            w[i] = set.greedy ? 0 : weight_of(x[i], top, set.slope, set.far, (lds_double*)table);
            if (set.greedy ? rank[i] > 0 : set.k > 0 && rank[i] >= set.k) w[i] = 0;
            else if (set.greedy) w[i] = 1;
            all += w[i];
        }
        const u64 goal = set.greedy || !(set.p < 1.0f) ? ~0ull : (u64)__builtin_ceil((double)set.p * (double)all);
        u64 v[7];
        all = 0;
#pragma unroll
        for (int i = 0; i < 7; ++i) {
            u64 ahead = 0;
#pragma unroll
            for (int j = 0; j < 7; ++j) ahead += rank[j] < rank[i] ? w[j] : 0;
            v[i] = ahead < goal && (set.greedy || w[i] >= set.least) ? w[i] : 0;
            all += v[i];
        }
        u64 pick = (u64)((double)fmaxf(u, 0.0f) * (double)all);
        pick = u < 1.0f && pick < all ? pick : all - 1;
#pragma unroll
        for (int i = 0; i < 7; ++i) {
            if (token < 0 && pick < v[i]) token = i;
            pick -= v[i];
        }
    }
    a.out[r] = token;
}

// Whether one block takes in a row at once, rather than the pass over the logits by many and the
// rest by one.  One launch less, but a row's exponentials all on one CU, and rows past two a CU
// wait for a second round of the whole.  Measured, at once against apart (us; the whole distribution,
// top_k 50, top_p 0.95 with some flat rows; the rule is off by 2 us for the 128 x 17000 below, the most
// that it was seen to lose without flat rows):
//      1 x 9000   10.3 14 18  against 11 16 20        1 x 32000   14.3 17 23  against 12.4 18 21
//   128 x 17000   12.8 17 57  against 14.7 19 55    128 x 32000   15.5 18 71  against 15.2 20 58
//   600 x 9000    29   49 79  against 25   43 100   600 x 32000   41.5 63 115 against 36   48 92
//   256 x 32000   16.2 19     against 19.1 22       600 x 6000    25   39 45  against 22   32 67
static bool at_once(long rows, int vocab)
{
    const long cus = device_cu_count();
    if (vocab <= 4 * SR_BATCH) return true;
    if (vocab > 16 * SR_BATCH || rows > 2 * cus) return false;
    return vocab <= 8 * SR_BATCH || rows > cus / 2;
}

template <class L>
static hipError_t launch_sample(const SampleArgs& a, hipStream_t st)
{
    static std::atomic<unsigned long long> done{0};
    hipError_t e = allow_full_lds((const void*)k_sample_long<L>, &done);
    if (e != hipSuccess) return e;
    if (a.vocab < 8) {
        k_sample_tiny<L><<<dim3((unsigned)((a.rows + 63) / 64)), dim3(64), 0, st>>>(a);
        return hipGetLastError();
    }
    const dim3 rows((unsigned)(a.rows < (1L << 20) ? a.rows : 1L << 20));
    constexpr size_t lds = sizeof(Shared<SR_SHORT, false>);
    if (at_once(a.rows, a.vocab)) {
        k_sample<L><<<rows, dim3(64 * SR_SHORT), lds + a.batches * (sizeof(BatchInfo) + 1024), st>>>(a);
    } else {
        const dim3 grid((a.batches + SR_SCAN - 1) / SR_SCAN, (unsigned)(a.rows < 65535 ? a.rows : 65535));
        k_sample_scan<L><<<grid, dim3(64 * SR_SCAN), 0, st>>>(a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        k_sample_pick<L><<<rows, dim3(64 * SR_SHORT), lds, st>>>(a);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
    // a row that may be cut may need all of its logits
    const bool cut = a.top_ks || a.top_ps || a.min_ps || (a.top_k > 1 && a.top_k < a.vocab) || (a.top_p > 0.0f && a.top_p < 1.0f) || a.min_p > 0.0f;
    if (!cut || (!a.temperatures && !(a.temperature > 0.0f))) return hipSuccess;
    k_sample_long<L><<<rows, dim3(64 * SR_LONG), sizeof(Shared<SR_LONG, true>), st>>>(a);
    return hipGetLastError();
}

long sample_space(long rows, int vocab)
{
    const long batches = (vocab + SR_BATCH - 1) / SR_BATCH;
    return at_once(rows, vocab) ? 0 : rows * batches * (long)(sizeof(BatchInfo) + 256);
}

hipError_t run_sample(int dtype, const void* logits, long rows, int vocab, long stride, const float* u, const float* temperatures,
                      const int* top_ks, const float* top_ps, const float* min_ps, float temperature, int top_k, float top_p,
                      float min_p, int* out, void* workspace, hipStream_t st)
{
    SampleArgs a{logits, stride, u, temperatures, top_ks, top_ps, min_ps, temperature, top_p, min_p, top_k, vocab, rows, out,
                 (vocab + SR_BATCH - 1) / SR_BATCH, workspace, nullptr};
    if (at_once(rows, vocab)) a.info = nullptr;   // (a workspace that is not needed may be given)
    a.groups = reinterpret_cast<float*>((BatchInfo*)workspace + rows * a.batches);
    if (dtype == DT_F16) return launch_sample<half_t>(a, st);
    return dtype == DT_BF16 ? launch_sample<bf16_t>(a, st) : launch_sample<float>(a, st);
}

}  // namespace fc

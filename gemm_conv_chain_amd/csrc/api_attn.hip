// api_attn.hip -- the C ABI of the attention-serving operators: validation on
// the host before any HIP call, the choice of kernel form and split, launch.
#include <stdarg.h>
#include <stdio.h>

#include <new>
#include <vector>

#include "../../include/fusedchain.h"
#include "fc_launch.h"
#include "kv_common.h"

namespace fc {
hipError_t run_rope(int dtype, const void* x, void* y, long xt, long xh, long yt, long yh, const int* positions,
                    const RopeArgs& r, bool inverse, long tokens, int heads, int d, hipStream_t st);
hipError_t run_kv_append(int dtype, const void* k, const void* v, const void* q, void* q_out, const long* strides,
                         uint8_t* codes, float* scales, const int* table, const int* cu_q, const int* kv_lens,
                         const int* positions, const KvShape& s, const RopeArgs& r, hipStream_t st);
hipError_t run_attn_rows(int dtype, const AttnArgs& a, hipStream_t st);
hipError_t run_attn_tile(int dtype, const AttnArgs& a, hipStream_t st);
hipError_t run_attn_join(int dtype, const AttnArgs& a, hipStream_t st);
}  // namespace fc

namespace {

fc_status fail(fc_status s, const char* fmt, ...)
{
    char msg[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    return (fc_status)fc::api_fail(s, msg);
}

fc_status done(hipError_t e, const char* what)
{
    if (e != hipSuccess) return fail(FC_E_HIP, "%s: %s", what, hipGetErrorString(e));
    return (fc_status)fc::api_fail(FC_OK, "");
}

bool aligned(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

fc_status check_strides(const int64_t* strides, int n)
{
    if (!strides) return fail(FC_E_NULL, "strides are required");
    for (int i = 0; i < n; ++i)
        if (strides[i] % 8) return fail(FC_E_ALIGN, "stride %d (%lld) is not a multiple of 8 elements", i, (long long)strides[i]);
    return FC_OK;
}

fc_status check_rope(const fc_rope* r, int d)
{
    if (r->rot < 0 || r->rot > d || r->rot % 16)
        return fail(FC_E_SHAPE, "rot=%d must be a multiple of 16, at most d=%d", r->rot, d);
    if (r->rot > 0 && !r->turns) return fail(FC_E_NULL, "rope turns are required");
    if (!aligned(r->turns, 8)) return fail(FC_E_ALIGN, "rope turns must be 8-byte aligned");
    if (!(r->mscale - r->mscale == 0.0f)) return fail(FC_E_ARG, "mscale must be a finite number");
    return FC_OK;
}

fc::RopeArgs rope_args(const fc_rope* r)
{
    if (!r) return fc::RopeArgs{nullptr, 0, 0, 1.0f};
    return fc::RopeArgs{(const unsigned long long*)r->turns, r->rot, r->interleaved != 0, r->mscale};
}

fc_status check_shape(const fc_kv_shape* s)
{
    if (!s) return fail(FC_E_NULL, "shape is NULL");
    if (s->dtype != FC_F16 && s->dtype != FC_BF16) return fail(FC_E_ARG, "dtype %d out of range", s->dtype);
    if (s->batch < 0 || s->tokens < 0 || s->hq <= 0 || s->hkv <= 0 || s->d <= 0 || s->pages < 0 ||
        s->table_stride < 0 || s->max_q < 0 || s->max_kv < 0)
        return fail(FC_E_SHAPE, "negative or zero size");
    if (s->hq % s->hkv) return fail(FC_E_SHAPE, "hq=%d is not a multiple of hkv=%d", s->hq, s->hkv);
    if (s->d != 64 && s->d != 128 && s->d != 192 && s->d != 256)
        return fail(FC_E_UNSUPPORTED, "d=%d: 64, 128, 192 and 256 are implemented", s->d);
    if (s->page < 16 || s->page > 256 || (s->page & (s->page - 1)))
        return fail(FC_E_UNSUPPORTED, "page=%d: 16, 32, 64, 128 and 256 are implemented", s->page);
    // grid sizes, rows of a sequence and key positions are 32-bit
    if (s->batch > (1 << 20)) return fail(FC_E_UNSUPPORTED, "batch=%d exceeds 2^20", s->batch);
    if (s->hq > 65535) return fail(FC_E_UNSUPPORTED, "hq=%d exceeds 65535", s->hq);
    if (s->tokens > 0x3fffffffL / s->hq) return fail(FC_E_UNSUPPORTED, "tokens*hq exceeds 2^30 - 1");
    if ((int64_t)s->page * s->table_stride > 0x7fff0000L)
        return fail(FC_E_UNSUPPORTED, "page*table_stride exceeds the 32-bit positions");
    return FC_OK;
}

bool nothing(const fc_kv_shape* s) { return s->tokens == 0 || s->batch == 0; }

fc_status check_cache(const fc_kv_shape* s, const uint8_t* codes, const float* scales, const int32_t* table,
                      const int32_t* cu_q, const int32_t* kv_lens)
{
    if (s->pages == 0 || s->table_stride == 0) return fail(FC_E_SHAPE, "tokens need a pool with pages and a table");
    if (!codes || !scales || !table || !cu_q || !kv_lens)
        return fail(FC_E_NULL, "codes, scales, table, cu_q and kv_lens are required");
    if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(table, 4) || !aligned(cu_q, 4) || !aligned(kv_lens, 4))
        return fail(FC_E_ALIGN, "codes and scales must be 16-byte, indices 4-byte aligned");
    return FC_OK;
}

fc::KvShape kv(const fc_kv_shape* s)
{
    return fc::KvShape{s->batch, s->hq, s->hkv, s->d, s->page, s->pages, s->table_stride, (long)s->tokens, s->max_q, s->max_kv};
}

fc_status check_params(const fc_kv_shape* s, const fc_attn_params* p)
{
    if (!p) return fail(FC_E_NULL, "params is NULL");
    // (the kernels divide by either, and one by the other, in 32 bits)
    if (!(p->scale >= 1e-18f && p->scale <= 1e18f)) return fail(FC_E_ARG, "scale must be positive, 1e-18 to 1e18");
    if (p->softcap != 0.0f && !(p->softcap >= 1e-18f && p->softcap <= 1e18f))
        return fail(FC_E_ARG, "softcap must be 0 or 1e-18 to 1e18");
    if (p->window < 0) return fail(FC_E_ARG, "window %d is negative", p->window);
    if (p->window > 0 && !p->causal) return fail(FC_E_UNSUPPORTED, "a window needs causal scores");
    if (p->variant < 0 || p->variant > 2) return fail(FC_E_ARG, "variant %d out of range", p->variant);
    if (p->splits < 0 || p->splits > 1024) return fail(FC_E_ARG, "splits %d out of range", p->splits);
    return FC_OK;
}

// Blocks of 16 keys that a block of `rows` rows can see.
int64_t key_blocks(const fc_kv_shape* s, const fc_attn_params* p, int64_t rows)
{
    int64_t keys = s->max_kv > 0 ? s->max_kv : 1;
    const int64_t cap = (int64_t)s->page * s->table_stride;
    if (keys > cap && cap > 0) keys = cap;
    // the window and what the block's queries span
    int64_t span = rows / (s->hq / s->hkv) + 1;
    if (span > s->max_q) span = s->max_q;
    if (p->window > 0 && p->window + span < keys) keys = p->window + span;
    return (keys + 15) / 16 + 1;
}

// Splits of the tile form: the least of
//   max(1, (n * tiles / CUs + 1/2) / k) * (chunk + 5) * (d + 40) / 168       the products
//   + 20 + 2 n * tokens * hq * d / 10^6, if n > 1                           partial results and join
// where chunk is in blocks of 16 keys, tiles are those that `tokens` fill (fewer
// than max_q allows if the batch is ragged), and a CU does the work of k = 1.5 (d =
// 64), 2 (d = 128) or 1.5 tiles in the time of one.  More splits have to gain 4 %.  The
// numbers are fits to 80 drawn calls (d = 64 to 256, 1 to 16 sequences, to 32768 keys,
// most of them ragged) timed with 1 to 16 splits: the choice is 4 % from the best on
// average and 1.5 times it at worst; filling the machine once, by max_q, was 14 % and
// 2.1 times.  (us, by splits, the choice marked:)
//   d = 64, 138 tiles of 8000 keys, ragged      1: 122   2: 86   4: 70    6*: 59   8: 70
//   d = 64, 584 tiles of 12001 keys             1: 511   2*: 420  4: 386   8: 434
//   d = 128, 346 tiles of 4000 keys, ragged     1*: 110   2: 147   4: 141
//   d = 64, 62 tiles of 16000 keys, ragged      1: 238   4: 75   8: 55   10: 68   (9 taken)
//   d = 256, 8 tiles of 14400 keys              1: 890   4: 246   16: 87          (29 taken)
// One k serves all kinds of scores, though at d = 64 a CU holds three tiles of plain or
// capped ones and two with a bias (below, 496 blocks with keys at three splits: one
// round of either; four splits are one round of plain ones, and two with a bias):
//   4 chunks of 515 queries, 12001 keys, ragged 1: 198   2: 125   3*: 120  4: 102  6: 118
//   with a bias                                 1: 242   2: 149   3*: 113  4: 153  6: 122
int64_t tile_splits(const fc_kv_shape* s, int64_t per, int64_t base, int64_t blocks)
{
    const double rows = (double)s->tokens * (s->hq / s->hkv);
    double tiles = s->hkv * (rows / per + 0.5 * s->batch);
    if (tiles > base) tiles = (double)base;
    if (tiles < s->hkv) tiles = s->hkv;
    const double k = s->d == 128 ? 2.0 : 1.5, cus = fc::device_cu_count();
    int64_t best = 1;
    double least = 0.0;
    for (int64_t n = 1; n <= 64 && (n - 1) * 8 < blocks; ++n) {
        const int64_t chunk = ((blocks + n - 1) / n + 3) / 4 * 4;
        if ((blocks + chunk - 1) / chunk < n) continue;   // fewer splits have this chunk
        const double full = (n * tiles / cus + 0.5) / k;
        double t = (full > 1.0 ? full : 1.0) * (chunk + 5) * (s->d + 40) / 168.0;
        if (n > 1) t += 20.0 + 2e-6 * n * s->tokens * s->hq * s->d;
        if (n == 1 || t < 0.96 * least) {
            least = t;
            best = n;
        }
    }
    return best;
}

// Form and split of a call.  Few rows take the form whose waves split the keys,
// more the one that stages them for a tile of rows; where they meet depends on
// whether sequences x kv heads alone fill the machine (us, rows form / tile form):
//   32 x 4, 8000 keys    d = 64    16 rows 36 / 37     32 rows 46 / 38
//                        d = 128   32 rows 57 / 65     64 rows 91 / 83
//                        d = 256   64 rows 187 / 304   128 rows 338 / 340
//   8 x 4, 4000 keys     d = 64    64 rows 19 / 21     128 rows 26 / 24
//                        d = 128   64 rows 24 / 29     96 rows 38 / 31
//                        d = 256   64 rows 49 / 60     96 rows 77 / 63
// The rows form splits keys over blocks where rows and heads alone leave CUs
// without one (us, by splits):
//   rows, 2 sequences x 4 heads, 131071 keys    8: 126   16: 71   32: 52   64: 59
//   rows, 64 x 8, to 8192 keys                  1: 127    2: 133   4: 141
//   rows, 1 x 2, 513 keys                       1: 7.6    3: 8.5 (the join's launch)
void plan_attn(const fc_kv_shape* s, const fc_attn_params* p, fc_attn_plan* out)
{
    const int64_t rows = (int64_t)(s->max_q > 0 ? s->max_q : 1) * (s->hq / s->hkv);
    int v = p->variant;
    const int64_t cus = fc::device_cu_count();
    if (v == FC_ATTN_AUTO) {
        const bool full = (int64_t)s->batch * s->hkv * 2 >= cus;
        const int64_t few = !full || s->d > 128 ? 64 : s->d > 64 ? 32 : 16;
        v = rows <= few ? FC_ATTN_ROWS : FC_ATTN_TILE;
    }
    const bool tile = v == FC_ATTN_TILE;
    const int64_t per = tile ? (s->d <= 128 ? 128 : 256) : (rows > 16 ? 32 : 16);   // rows a block
    const int64_t base = (int64_t)(s->batch > 0 ? s->batch : 1) * s->hkv * ((rows + per - 1) / per);
    const int64_t blocks = key_blocks(s, p, per);
    int64_t n = p->splits;
    if (n == 0 && tile) n = tile_splits(s, per, base, blocks);
    else if (n == 0) {
        n = base < cus ? (cus + base - 1) / base : 1;   // one block a CU
        const int64_t most = blocks < 64 ? 1 : (blocks + 15) / 16;
        n = n > most ? most : n;
        n = n > 256 ? 256 : n;
    }
    n = n < 1 ? 1 : n;
    const int64_t unit = tile ? 4 : 16;
    const int64_t chunk = ((blocks + n - 1) / n + unit - 1) / unit * unit;
    if (p->splits == 0) n = (blocks + chunk - 1) / chunk;
    out->variant = v;
    out->splits = (int32_t)n;
    out->chunk = (int32_t)(chunk * 16);
    out->workspace = n > 1 ? s->tokens * s->hq * n * (s->d + 4) * 4 : 0;
}

}  // namespace

extern "C" {

fc_status rope_apply(const void* x, void* y, const int64_t* strides, const int32_t* positions, const fc_rope* rope,
                     int32_t inverse, fc_dtype dtype, int64_t tokens, int32_t heads, int32_t d, void* stream)
{
    if ((int)dtype != FC_F16 && (int)dtype != FC_BF16) return fail(FC_E_ARG, "dtype %d out of range", (int)dtype);
    if (tokens < 0 || heads < 0 || d <= 0 || d % 16) return fail(FC_E_SHAPE, "tokens, heads >= 0 and d a multiple of 16 required");
    if (d > 1024 || heads > 65535) return fail(FC_E_UNSUPPORTED, "d=%d exceeds 1024 or heads=%d 65535", d, heads);
    if (!rope) return fail(FC_E_NULL, "rope is NULL");
    fc_status s = check_rope(rope, d);
    if (s != FC_OK) return s;
    s = check_strides(strides, 4);
    if (s != FC_OK) return s;
    if (tokens == 0 || heads == 0) return done(hipSuccess, "");
    if (!x || !y || (rope->rot > 0 && !positions)) return fail(FC_E_NULL, "x, y and positions are required");
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(positions, 4))
        return fail(FC_E_ALIGN, "x and y must be 16-byte, positions 4-byte aligned");
    return done(fc::run_rope(dtype, x, y, strides[0], strides[1], strides[2], strides[3], positions, rope_args(rope),
                             inverse != 0, tokens, heads, d, (hipStream_t)stream),
                "rope_apply");
}

fc_status kv_append(const void* k, const void* v, const void* q, void* q_out, const int64_t* strides, uint8_t* codes,
                    float* scales, const int32_t* table, const int32_t* cu_q, const int32_t* kv_lens,
                    const int32_t* positions, const fc_rope* rope, const fc_kv_shape* shape, void* stream)
{
    fc_status s = check_shape(shape);
    if (s != FC_OK) return s;
    if (rope && (s = check_rope(rope, shape->d)) != FC_OK) return s;
    if ((s = check_strides(strides, 6)) != FC_OK) return s;
    if ((q == nullptr) != (q_out == nullptr) && !nothing(shape)) return fail(FC_E_NULL, "q and q_out go together");
    if (nothing(shape)) return done(hipSuccess, "");
    if (!k || !v) return fail(FC_E_NULL, "k and v are required");
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) || !aligned(q_out, 16) || !aligned(positions, 4))
        return fail(FC_E_ALIGN, "k, v, q and q_out must be 16-byte, positions 4-byte aligned");
    if ((s = check_cache(shape, codes, scales, table, cu_q, kv_lens)) != FC_OK) return s;
    long st[6];
    for (int i = 0; i < 6; ++i) st[i] = (long)strides[i];
    return done(fc::run_kv_append(shape->dtype, k, v, q, q_out, st, codes, scales, table, cu_q, kv_lens, positions,
                                  kv(shape), rope_args(rope), (hipStream_t)stream),
                "kv_append");
}

fc_status chain_attn_plan(const fc_kv_shape* shape, const fc_attn_params* params, fc_attn_plan* plan)
{
    fc_status s = check_shape(shape);
    if (s != FC_OK) return s;
    if ((s = check_params(shape, params)) != FC_OK) return s;
    if (!plan) return fail(FC_E_NULL, "plan is NULL");
    plan_attn(shape, params, plan);
    return done(hipSuccess, "");
}

fc_status chain_attn(const void* q, const int64_t* strides, const uint8_t* codes, const float* scales,
                     const int32_t* table, const int32_t* cu_q, const int32_t* kv_lens, const float* slopes,
                     const fc_attn_params* params, void* out, float* lse, const fc_kv_shape* shape, void* workspace,
                     int64_t workspace_bytes, void* stream)
{
    fc_status s = check_shape(shape);
    if (s != FC_OK) return s;
    if ((s = check_params(shape, params)) != FC_OK) return s;
    if ((s = check_strides(strides, 2)) != FC_OK) return s;
    if (nothing(shape)) return done(hipSuccess, "");
    if (!q || !out) return fail(FC_E_NULL, "q and out are required");
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(slopes, 4) || !aligned(workspace, 16))
        return fail(FC_E_ALIGN, "q, out and workspace must be 16-byte, lse and slopes 4-byte aligned");
    if ((s = check_cache(shape, codes, scales, table, cu_q, kv_lens)) != FC_OK) return s;
    fc_attn_plan p;
    plan_attn(shape, params, &p);
    if (p.workspace > 0 && (!workspace || workspace_bytes < p.workspace))
        return fail(workspace ? FC_E_SHAPE : FC_E_NULL, "a workspace of %lld bytes is required, got %lld",
                    (long long)p.workspace, (long long)workspace_bytes);
    fc::AttnArgs a;
    a.q = q;
    a.q_ts = strides[0];
    a.q_hs = strides[1];
    a.codes = codes;
    a.scales = scales;
    a.table = table;
    a.cu_q = cu_q;
    a.kv_lens = kv_lens;
    a.slopes = slopes;
    a.out = out;
    a.lse = lse;
    a.part_o = (float*)workspace;
    a.part_ml = p.splits > 1 ? (fc::floatx4*)(a.part_o + shape->tokens * shape->hq * p.splits * shape->d) : nullptr;
    a.s = kv(shape);
    a.G = shape->hq / shape->hkv;
    a.causal = params->causal != 0;
    a.window = params->window;
    a.nsplit = p.splits;
    a.chunk = p.chunk / 16;
    a.pg_shift = __builtin_ctz((unsigned)shape->page) - 4;
    a.scale = params->scale;
    a.cap = params->softcap;
    a.by_g = fc::FastDiv::make(a.G);
    hipError_t e = p.variant == FC_ATTN_TILE ? fc::run_attn_tile(shape->dtype, a, (hipStream_t)stream)
                                             : fc::run_attn_rows(shape->dtype, a, (hipStream_t)stream);
    if (e == hipSuccess && p.splits > 1) e = fc::run_attn_join(shape->dtype, a, (hipStream_t)stream);
    return done(e, "chain_attn");
}

fc_status kv_check(const int32_t* table, const int32_t* cu_q, const int32_t* kv_lens, const fc_kv_shape* shape,
                   int32_t writes)
{
    fc_status s = check_shape(shape);
    if (s != FC_OK) return s;
    if (shape->batch == 0) return done(hipSuccess, "");
    if (!table || !cu_q || !kv_lens) return fail(FC_E_NULL, "table, cu_q and kv_lens are required");
    if (cu_q[0] != 0) return fail(FC_E_SHAPE, "cu_q[0] = %d is not 0", cu_q[0]);
    std::vector<int32_t> owner;   // of each page: the sequences that name it, -2 for several
    if (writes) {
        try {
            owner.assign(shape->pages, -1);
        } catch (const std::bad_alloc&) {
            return fail(FC_E_SHAPE, "no memory to check %d pages", shape->pages);
        }
    }
    for (int b = 0; b < shape->batch; ++b) {
        const int64_t n = (int64_t)cu_q[b + 1] - cu_q[b];
        if (n < 0 || cu_q[b + 1] > shape->tokens)
            return fail(FC_E_SHAPE, "cu_q[%d] = %d falls or exceeds the %lld tokens", b + 1, cu_q[b + 1], (long long)shape->tokens);
        if (kv_lens[b] < n) return fail(FC_E_SHAPE, "kv_lens[%d] = %d is under its %lld new tokens", b, kv_lens[b], (long long)n);
        const int64_t used = ((int64_t)kv_lens[b] + shape->page - 1) / shape->page;
        if (used > shape->table_stride)
            return fail(FC_E_SHAPE, "kv_lens[%d] = %d needs %lld pages, the table's row has %d", b, kv_lens[b],
                        (long long)used, shape->table_stride);
        for (int64_t p = 0; p < used; ++p) {
            const int id = table[(int64_t)b * shape->table_stride + p];
            if (id < 0 || id >= shape->pages)
                return fail(FC_E_SHAPE, "table[%d][%lld] = %d is outside the pool of %d pages", b, (long long)p, id, shape->pages);
            if (writes) owner[id] = owner[id] == -1 ? b : -2;
        }
    }
    for (int b = 0; writes && b < shape->batch; ++b) {
        const int64_t n = (int64_t)cu_q[b + 1] - cu_q[b];
        if (n == 0) continue;
        for (int64_t p = (kv_lens[b] - n) / shape->page; p <= ((int64_t)kv_lens[b] - 1) / shape->page; ++p) {
            const int id = table[(int64_t)b * shape->table_stride + p];
            if (owner[id] == -2) return fail(FC_E_SHAPE, "page %d gets new tokens of sequence %d and is named twice", id, b);
        }
    }
    return done(hipSuccess, "");
}

}  // extern "C"

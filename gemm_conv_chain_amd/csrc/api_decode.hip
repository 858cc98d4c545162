// api_decode.hip -- the C ABI of the operators around a decoding step: trees of
// drafted tokens, drawing tokens, copying pages.  Validation on the host before
// any HIP call.
#include <new>
#include <vector>

#include "api_checks.h"

namespace fc {
hipError_t run_tree_plan(const int* parents, const int* cu_q, const int* kv_lens, int batch, long tokens, int words,
                         unsigned long long* bits, int* positions, hipStream_t st);
hipError_t run_tree_accept(const int* parents, const int* drafted, const int* targets, const int* cu_q, const int* kv_lens,
                           int batch, long tokens, int max_keep, int* keep, int* kept, int* next, int* lens, hipStream_t st);
hipError_t run_kv_copy(uint8_t* codes, float* scales, int layers, int pages, int hkv, int page, int d, const int* pairs, long n,
                       hipStream_t st);
hipError_t run_sample(int dtype, const void* logits, long rows, int vocab, long stride, const float* u, const float* temperatures,
                      const int* top_ks, const float* top_ps, const float* min_ps, float temperature, int top_k, float top_p,
                      float min_p, int* out, void* workspace, hipStream_t st);
long sample_space(long rows, int vocab);
}  // namespace fc

namespace {

using fc::aligned;
using fc::done;
using fc::fail;

fc_status check_batch(int32_t batch, int64_t tokens)
{
    if (batch < 0 || tokens < 0) return fail(FC_E_SHAPE, "negative batch or tokens");
    if (batch > (1 << 20)) return fail(FC_E_UNSUPPORTED, "batch=%d exceeds 2^20", batch);
    if (tokens > 0x3fffffffL) return fail(FC_E_UNSUPPORTED, "tokens exceeds 2^30 - 1");
    return FC_OK;
}

fc_status check_logits(int32_t dtype, int64_t rows, int32_t vocab)
{
    if (dtype != FC_F16 && dtype != FC_BF16 && dtype != FC_F32) return fail(FC_E_ARG, "dtype %d out of range", dtype);
    if (rows < 0 || vocab < 1) return fail(FC_E_SHAPE, "rows >= 0 and vocab >= 1 required");
    if (vocab > (1 << 20)) return fail(FC_E_UNSUPPORTED, "vocab=%d exceeds 2^20", vocab);
    if (rows > 0x7fffffffL) return fail(FC_E_UNSUPPORTED, "rows exceeds 2^31 - 1");
    return FC_OK;
}

}  // namespace

extern "C" {

fc_status tree_plan(const int32_t* parents, const int32_t* cu_q, const int32_t* kv_lens, int32_t batch, int64_t tokens,
                    int32_t words, uint64_t* bits, int32_t* positions, void* stream)
{
    fc_status s = check_batch(batch, tokens);
    if (s != FC_OK) return s;
    if (words < 1 || words > FC_TREE_WORDS)
        return fail(FC_E_UNSUPPORTED, "words=%d: 1 to %d are implemented", words, FC_TREE_WORDS);
    if (batch == 0 || tokens == 0) return done(hipSuccess, "");
    if (!parents || !cu_q || !kv_lens || !bits || !positions)
        return fail(FC_E_NULL, "parents, cu_q, kv_lens, bits and positions are required");
    if (!aligned(parents, 4) || !aligned(cu_q, 4) || !aligned(kv_lens, 4) || !aligned(bits, 8) || !aligned(positions, 4))
        return fail(FC_E_ALIGN, "bits must be 8-byte, indices 4-byte aligned");
    return done(fc::run_tree_plan(parents, cu_q, kv_lens, batch, tokens, words, (unsigned long long*)bits, positions,
                                  (hipStream_t)stream),
                "tree_plan");
}

fc_status tree_accept(const int32_t* parents, const int32_t* drafted, const int32_t* targets, const int32_t* cu_q,
                      const int32_t* kv_lens, int32_t batch, int64_t tokens, int32_t max_keep, int32_t* keep, int32_t* kept,
                      int32_t* next, int32_t* lens, void* stream)
{
    fc_status s = check_batch(batch, tokens);
    if (s != FC_OK) return s;
    if (max_keep < 1 || max_keep > 64 * FC_TREE_WORDS)
        return fail(FC_E_UNSUPPORTED, "max_keep=%d: 1 to %d are implemented", max_keep, 64 * FC_TREE_WORDS);
    if (batch == 0) return done(hipSuccess, "");
    if (!cu_q || !kv_lens || !keep || !kept || !next || !lens)
        return fail(FC_E_NULL, "cu_q, kv_lens, keep, kept, next and lens are required");
    if (tokens > 0 && (!parents || !drafted || !targets))
        return fail(FC_E_NULL, "parents, drafted and targets are required");
    const void* all[] = {parents, drafted, targets, cu_q, kv_lens, keep, kept, next, lens};
    for (const void* p : all)
        if (!aligned(p, 4)) return fail(FC_E_ALIGN, "indices must be 4-byte aligned");
    return done(fc::run_tree_accept(parents, drafted, targets, cu_q, kv_lens, batch, tokens, max_keep, keep, kept, next, lens,
                                    (hipStream_t)stream),
                "tree_accept");
}

fc_status kv_copy(uint8_t* codes, float* scales, int32_t layers, int32_t pages, int32_t hkv, int32_t page, int32_t d,
                  const int32_t* pairs, int64_t n, void* stream)
{
    if (layers < 0 || pages < 0 || hkv <= 0 || d <= 0 || n < 0) return fail(FC_E_SHAPE, "negative or zero size");
    if (layers > 65535) return fail(FC_E_UNSUPPORTED, "layers=%d exceeds 65535", layers);
    if (hkv > 65535) return fail(FC_E_UNSUPPORTED, "hkv=%d exceeds 65535", hkv);
    if (d != 64 && d != 128 && d != 192 && d != 256)
        return fail(FC_E_UNSUPPORTED, "d=%d: 64, 128, 192 and 256 are implemented", d);
    if (page < 16 || page > 256 || (page & (page - 1)))
        return fail(FC_E_UNSUPPORTED, "page=%d: 16, 32, 64, 128 and 256 are implemented", page);
    if (n == 0) return done(hipSuccess, "");
    if (!pairs) return fail(FC_E_NULL, "pairs are required");
    if (n > pages) return fail(FC_E_SHAPE, "%lld pairs cannot have destinations of their own in a pool of %d pages", (long long)n, pages);
    try {
        std::vector<uint8_t> is(pages, 0);   // bit 0: a source, bit 1: a destination
        for (int64_t i = 0; i < 2 * n; ++i) {
            const int32_t id = pairs[i];
            if (id < 0 || id >= pages)
                return fail(FC_E_SHAPE, "pair %lld names page %d, outside the pool of %d pages", (long long)(i / 2), id, pages);
            if (i & 1) {
                if (is[id] & 2) return fail(FC_E_SHAPE, "page %d is the destination of two pairs", id);
                is[id] |= 2;
            } else {
                is[id] |= 1;
            }
            if (is[id] == 3) return fail(FC_E_SHAPE, "page %d is a source and a destination", id);
        }
    } catch (const std::bad_alloc&) {
        return fail(FC_E_SHAPE, "no memory to check %d pages", pages);
    }
    if (layers == 0) return done(hipSuccess, "");
    if (!codes || !scales) return fail(FC_E_NULL, "codes and scales are required");
    if (!aligned(codes, 16) || !aligned(scales, 16)) return fail(FC_E_ALIGN, "codes and scales must be 16-byte aligned");
    return done(fc::run_kv_copy(codes, scales, layers, pages, hkv, page, d, pairs, n, (hipStream_t)stream), "kv_copy");
}

fc_status sample_workspace(int32_t dtype, int64_t rows, int32_t vocab, int64_t* bytes)
{
    fc_status s = check_logits(dtype, rows, vocab);
    if (s != FC_OK) return s;
    if (!bytes) return fail(FC_E_NULL, "bytes is NULL");
    *bytes = fc::sample_space(rows, vocab);
    return done(hipSuccess, "");
}

fc_status sample_tokens(const void* logits, int32_t dtype, int64_t rows, int32_t vocab, int64_t stride, const float* u,
                        const fc_sampling* sampling, int32_t* out, void* workspace, int64_t workspace_bytes, void* stream)
{
    fc_status s = check_logits(dtype, rows, vocab);
    if (s != FC_OK) return s;
    if (!sampling) return fail(FC_E_NULL, "sampling is NULL");
    if (stride < 0) return fail(FC_E_SHAPE, "a row stride of %lld is negative", (long long)stride);
    const fc_sampling& g = *sampling;
    if (!g.temperatures && !(g.temperature >= 0.0f && g.temperature - g.temperature == 0.0f))
        return fail(FC_E_ARG, "temperature must be a finite number, 0 or more");
    if (!g.top_ks && g.top_k < 0) return fail(FC_E_ARG, "top_k %d is negative", g.top_k);
    if (!g.top_ps && !(g.top_p >= 0.0f && g.top_p <= 1.0f)) return fail(FC_E_ARG, "top_p must be in 0 .. 1");
    if (!g.min_ps && !(g.min_p >= 0.0f && g.min_p <= 1.0f)) return fail(FC_E_ARG, "min_p must be in 0 .. 1");
    if (rows == 0) return done(hipSuccess, "");
    if (!logits || !u || !out) return fail(FC_E_NULL, "logits, u and out are required");
    if (!aligned(logits, dtype == FC_F32 ? 4 : 2)) return fail(FC_E_ALIGN, "logits must be aligned to their type");
    if (!aligned(u, 4) || !aligned(out, 4) || !aligned(g.temperatures, 4) || !aligned(g.top_ks, 4) || !aligned(g.top_ps, 4) ||
        !aligned(g.min_ps, 4))
        return fail(FC_E_ALIGN, "u, out and the settings' arrays must be 4-byte aligned");
    // (a token, or the mark of a row that is not done, would be read as a setting)
    const auto meets_out = [&](const void* p) {
        const uintptr_t x = (uintptr_t)p, y = (uintptr_t)out, bytes = (uintptr_t)rows * 4;
        return p && x < y + bytes && y < x + bytes;
    };
    if (meets_out(u) || meets_out(g.temperatures) || meets_out(g.top_ks) || meets_out(g.top_ps) || meets_out(g.min_ps))
        return fail(FC_E_ARG, "out overlaps u or a setting's array");
    const int64_t need = fc::sample_space(rows, vocab);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(workspace ? FC_E_SHAPE : FC_E_NULL, "a workspace of %lld bytes is required, got %lld", (long long)need,
                    (long long)workspace_bytes);
    if (!aligned(workspace, 16)) return fail(FC_E_ALIGN, "workspace must be 16-byte aligned");
    return done(fc::run_sample(dtype, logits, rows, vocab, stride, u, g.temperatures, g.top_ks, g.top_ps, g.min_ps,
                               g.temperature, g.top_k, g.top_p, g.min_p, out, workspace, (hipStream_t)stream),
                "sample_tokens");
}

}  // extern "C"

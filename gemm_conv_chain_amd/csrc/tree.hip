// tree.hip -- the bookkeeping of a tree of drafted tokens: from each node's
// parent to the bits and positions that attention reads (k_tree_plan), and from
// the model's tokens to the path that is accepted (k_tree_accept).
//
// Both are a few dependent reads a sequence and bound by the launch and these (a tree of 8
// nodes: 1.9 and 2.3 us; 512 sequences of up to 64: 3.6 and 4.7; one chain of 4096: 148 and 16).
#include "fc_launch.h"
#include "kv_common.h"

namespace fc {

constexpr int TREE_NODES = 64 * 64;   // 64 * FC_TREE_WORDS

// One block a sequence, a wave 64 nodes at a time, whose ancestors among each other are one word
// of bits: found in at most six rounds, in each of which a node takes over the bits of
// the ancestor that it has got to, and that one's next.  The lowest bit is the ancestor whose
// parent lies before the 64 nodes, and from there a row goes on by whole words: a
// chain of 4096 nodes takes 64 steps a node, not 4096.
__global__ __launch_bounds__(256) void k_tree_plan(const int* parents, const int* cu_q, const int* kv_lens, KvShape s, int words,
                                                   unsigned long long* bits, int* positions)
{
    __shared__ unsigned long long among[TREE_NODES];   // a node's ancestors and itself, of its 64
    __shared__ int out[TREE_NODES];                    // the first ancestor before them, or -1
    const int lane = threadIdx.x & 63;
    for (int b = blockIdx.x; b < s.batch; b += gridDim.x) {
        if constexpr (kPoison) {
            lds_poison(among, sizeof among, threadIdx.x, blockDim.x);
            lds_poison(out, sizeof out, threadIdx.x, blockDim.x);
            __syncthreads();
        }
        long tok0;
        int n;
        seq_range(cu_q, s, b, &tok0, &n);
        const int start = (int)((unsigned)kv_lens[b] - (unsigned)n);
        if (n > 64 * words) {
            for (int i = threadIdx.x; i < n; i += blockDim.x) {
                for (int w = 0; w < words; ++w) bits[(tok0 + i) * words + w] = 0;
                positions[tok0 + i] = start;
            }
            continue;
        }
        for (int i = threadIdx.x; i - lane < n; i += blockDim.x) {
            const int p = i < n ? parents[tok0 + i] : -1, up = p >= 0 && p < i ? p : -1;
            unsigned long long seen = 1ull << lane;
            int at = up >= i - lane ? up - (i - lane) : -1;   // (the lane of) the ancestor that comes next
            while (__any(at >= 0)) {
                const unsigned long long its = __shfl(seen, at < 0 ? lane : at);
                const int next = __shfl(at, at < 0 ? lane : at);
                seen |= its;
                at = at < 0 ? -1 : next;
            }
            const int before = __shfl(up, __builtin_ctzll(seen));
            if (i >= n) continue;
            if (words == 1) {
                bits[tok0 + i] = seen;
                positions[tok0 + i] = (int)((unsigned)start + (unsigned)__popcll(seen) - 1);
            } else {
                among[i] = seen;
                out[i] = before;
            }
        }
        if (words == 1) continue;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += blockDim.x) {
            unsigned long long* row = bits + (tok0 + i) * words;
            int a = i, depth = -1;
            for (int w = words - 1; w >= 0; --w) {
                unsigned long long m = 0;
                if (a >= 0 && a >> 6 == w) {
                    m = among[a];
                    a = out[a];
                }
                row[w] = m;
                depth += __popcll(m);
            }
            positions[tok0 + i] = (int)((unsigned)start + (unsigned)depth);
        }
        __syncthreads();   // LDS is free again
    }
}

// One wave a sequence.  A child comes after its parent, so that one pass over the nodes, 64
// at a time in registers, meets the whole path.  A target under 0 is no token (what sample_tokens
// gives for a row that is no distribution): no draft is it, and the path ends there.
__global__ __launch_bounds__(256) void k_tree_accept(const int* parents, const int* drafted, const int* targets, const int* cu_q,
                                                     const int* kv_lens, KvShape s, int max_keep, int* keep, int* kept, int* next,
                                                     int* lens)
{
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (long b = (long)blockIdx.x * 4 + wave; b < s.batch; b += (long)gridDim.x * 4) {
        long tok0;
        int n;
        seq_range(cu_q, s, (int)b, &tok0, &n);
        int* const list = keep + b * max_keep;
        int cur = 0, want = -1, count = 0;
        for (int base = 0; base < n && count < max_keep; base += 64) {
            const int j = base + lane;
            const bool live = j < n;
            const int par = live ? parents[tok0 + j] : -1;
            const int tok = live ? drafted[tok0 + j] : 0;
            const int tgt = live ? targets[tok0 + j] : 0;
            if (base == 0) {
                if (lane == 0) list[0] = 0;
                count = 1;
                want = __builtin_amdgcn_readfirstlane(tgt);
            }
            while (count < max_keep && want >= 0) {
                const unsigned long long m = __ballot(live && par == cur && j > cur && tok == want);
                if (!m) break;
                const int at = __builtin_ctzll(m);
                cur = base + at;
                want = __builtin_amdgcn_readlane(tgt, at);
                if (lane == 0) list[count] = cur;
                ++count;
            }
        }
        for (int i = count + lane; i < max_keep; i += 64) list[i] = -1;
        if (lane == 0) {
            const int len = kv_lens[b];
            kept[b] = count;
            next[b] = want;
            lens[b] = (int)((unsigned)len - (unsigned)n + (unsigned)count);
        }
    }
}

hipError_t run_tree_plan(const int* parents, const int* cu_q, const int* kv_lens, int batch, long tokens, int words,
                         unsigned long long* bits, int* positions, hipStream_t st)
{
    KvShape s{};
    s.batch = batch;
    s.tokens = tokens;
    const unsigned grid = batch < 65536 ? batch : 65536;
    k_tree_plan<<<dim3(grid), dim3(words == 1 ? 64 : 256), 0, st>>>(parents, cu_q, kv_lens, s, words, bits, positions);
    return hipGetLastError();
}

hipError_t run_tree_accept(const int* parents, const int* drafted, const int* targets, const int* cu_q, const int* kv_lens,
                           int batch, long tokens, int max_keep, int* keep, int* kept, int* next, int* lens, hipStream_t st)
{
    KvShape s{};
    s.batch = batch;
    s.tokens = tokens;
    const unsigned grid = (batch + 3) / 4 < 65536 ? (batch + 3) / 4 : 65536;
    k_tree_accept<<<dim3(grid), dim3(256), 0, st>>>(parents, drafted, targets, cu_q, kv_lens, s, max_keep, keep, kept, next, lens);
    return hipGetLastError();
}

}  // namespace fc

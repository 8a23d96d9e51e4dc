// Device helpers shared by the block-scaled paged cache's kernels (block_append.cu,
// block_attn.cu, block_select.cu): a batch's lengths, the block table, and the choice of the
// smallest keys of a list in (key, index) order.
#pragma once

#include <stdint.h>

#include "common.cuh"
#include "kernels.h"

namespace mtp {

// Sequence b's positions (>= 0) and its token count in this step (in [0, T]).
struct SeqStep {
    int len, q;
};
__device__ __forceinline__ SeqStep seq_step(const BlockBatch& t, int b) {
    SeqStep s;
    s.len = max(__ldg(t.seq_lens + b), 0);
    s.q = t.q_lens ? (int)min((int64_t)max(__ldg(t.q_lens + b), 0), t.T) : (int)t.T;
    return s;
}

// ceil(positions / bs) for positions >= 0, at most n_table
__device__ __forceinline__ int blocks_of(int positions, int bs, int64_t n_table) {
    const int nb = positions > 0 ? (positions - 1) / bs + 1 : 0;
    return (int)min((int64_t)nb, n_table);
}

// Physical block of logical block j of sequence b, or -1 (missing or out of range).
__device__ __forceinline__ int table_block(const BlockBatch& t, int64_t num_blocks, int b, int64_t j) {
    if (j >= t.n_table) return -1;
    const int n = __ldg(t.table + (int64_t)b * t.n_table + j);
    return n >= 0 && n < num_blocks ? n : -1;
}

// A float's bits as an unsigned key of the same order; NaN lowest, -0 as +0.
__device__ __forceinline__ uint32_t order_key(float f) {
    if (f != f) return 0u;
    const uint32_t u = __float_as_uint(f + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// 1 / 127 rounded to fp32: the step of 8-bit integers is the largest magnitude times this.
constexpr float kInv127 = 1.f / 127.f;

constexpr int kPickThreads = 1024;

struct PickSmem {
    uint32_t hist[256];
    uint32_t warp_sum[32];
    uint32_t digit, before;
};

// The `want` (1 <= want <= n) smallest of key(0) .. key(n - 1) in (key, index) order: every
// key < thr, and the first `need` of those equal to thr. Four passes over 8-bit digits from
// the top, each a histogram of the keys that share the digits found so far. All of the
// block's kPickThreads threads call it; integer counts, so the result is exact.
template <class Key>
__device__ void pick_threshold(const Key& key, int n, int want, PickSmem& sm, uint32_t* thr, int* need) {
    uint32_t prefix = 0, mask = 0;
    const int tid = threadIdx.x;
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) sm.hist[tid] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kPickThreads) {
            const uint32_t k = key(i);
            if ((k & mask) == prefix) atomicAdd(&sm.hist[(k >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (tid < 32) {  // the first digit at which the running count reaches `want`
            uint32_t c[8], sum = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += c[j] = sm.hist[8 * tid + j];
            uint32_t inc = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
                if (tid >= o) inc += u;
            }
            uint32_t run = inc - sum;  // keys in the digits before this lane's
            const bool here = run < (uint32_t)want && inc >= (uint32_t)want;
            if (here) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (run < (uint32_t)want && run + c[j] >= (uint32_t)want) {
                        sm.digit = 8 * tid + j;
                        sm.before = run;
                    }
                    run += c[j];
                }
            }
        }
        __syncthreads();
        prefix |= sm.digit << shift;
        mask |= 255u << shift;
        want -= (int)sm.before;
    }
    *thr = prefix;
    *need = want;
}

// Exclusive prefix sum of v (its sum over the block below 2^32) over the block's threads;
// *total gets the sum.
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, PickSmem& sm, uint32_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    __syncthreads();  // the previous use of warp_sum is over
    if (lane == 31) sm.warp_sum[warp] = inc;
    __syncthreads();
    uint32_t w = sm.warp_sum[lane], winc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, winc, o);
        if (lane >= o) winc += u;
    }
    *total = __shfl_sync(0xffffffffu, winc, 31);
    return inc - v + (warp ? __shfl_sync(0xffffffffu, winc, warp - 1) : 0u);
}

// Calls emit(i, taken, before) for every i < n in chunks of the block's threads, in order of
// i: whether i is among the picked, and how many picked ones come before it. Between a
// chunk's read(i) and its emit there is a block barrier, so emit may overwrite places that
// this or earlier chunks' reads used. read returns what emit gets as its last argument.
template <class Key, class Read, class Emit>
__device__ void pick_in_order(const Key& key, int n, uint32_t thr, int need, PickSmem& sm, const Read& read,
                              const Emit& emit) {
    uint32_t below = 0, equal = 0;  // picked for sure, and equal to thr, before this chunk
    for (int base = 0; base < n; base += kPickThreads) {
        const int i = base + (int)threadIdx.x;
        const uint32_t k = i < n ? key(i) : 0xffffffffu;
        const bool lt = i < n && k < thr, eq = i < n && k == thr;
        const auto val = read(i < n ? i : n - 1);
        uint32_t total;
        const uint32_t at = block_exclusive((lt ? 1u : 0u) | (eq ? 0x10000u : 0u), sm, &total);
        const uint32_t b_lt = below + (at & 0xffffu), b_eq = equal + (at >> 16);
        if (i < n) emit(i, lt || (eq && b_eq < (uint32_t)need), b_lt + min(b_eq, (uint32_t)need), val);
        below += total & 0xffffu;
        equal += total >> 16;
    }
}

// Launches `kern` so that it may start while the kernel before it in the stream ends (each of
// ours waits for that before it touches memory).
template <class K, class... A>
cudaError_t launch_after(K kern, dim3 grid, int threads, size_t smem, cudaStream_t s, const A&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace mtp

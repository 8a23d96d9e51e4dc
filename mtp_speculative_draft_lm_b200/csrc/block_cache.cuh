// Device helpers shared by the block-scaled paged cache's kernels (block_append.cu,
// block_attn.cu, block_select.cu): a batch's lengths, the block table, and the choice of the
// smallest keys of a list in (key, index) order.
#pragma once

#include <stdint.h>

#include <atomic>

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

// The `want` smallest of a list of keys in (key, index) order, by one CTA of THREADS threads that
// hold KEYS keys each, key u of thread t being entry u THREADS + t (whole rows of loads and
// stores). Digits are counted from the top among the keys that share the digits found so far
// until a count ends exactly at `want`: of 8 bits for 256 threads, of 11 for more (2.7 and 3.4
// thousand cycles for 512 and 2,048 spread floats, 6.3 for 8,192; most of it barriers). Integer
// counts: the choice is exact.
template <int THREADS>
struct PickSmem {
    static constexpr int kBits = THREADS <= 256 ? 8 : 11, kBins = 1 << kBits, kWarps = THREADS / 32;
    uint32_t hist[kBins];
    uint32_t tot[256];  // taken in each warp's row of 32 entries, then before it
    uint32_t warp_sum[32];
    uint32_t digit, before, in_digit;
};

__device__ __forceinline__ uint32_t warp_inclusive(uint32_t v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
        if ((int)(threadIdx.x & 31) >= o) v += u;
    }
    return v;
}

// Keys below *thr are picked, and the first *need of those equal to it (1 <= want <= the number
// of keys). each(f) calls f(key) for every key that this thread holds.
template <int THREADS, class Each>
__device__ __forceinline__ void pick_threshold(const Each& each, uint32_t want, PickSmem<THREADS>& sm, uint32_t* thr, uint32_t* need) {
    using S = PickSmem<THREADS>;
    constexpr int PER = S::kBins / THREADS;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t prefix = 0, mask = 0;
#pragma unroll 1
    for (int shift = 32 - S::kBits;;) {
#pragma unroll
        for (int j = 0; j < PER; ++j) sm.hist[j * THREADS + tid] = 0;
        __syncthreads();
        each([&](uint32_t k) {
            if ((k & mask) == prefix) atomicAdd(&sm.hist[(k >> shift) & (S::kBins - 1)], 1u);
        });
        __syncthreads();
        // the warp, then the lane, then the counter at which the running count reaches `want`
        uint32_t c[PER], sum = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) sum += c[j] = sm.hist[PER * tid + j];
        const uint32_t wsum = __reduce_add_sync(0xffffffffu, sum);
        if (lane == 0) sm.warp_sum[warp] = wsum;
        __syncthreads();
        const uint32_t w = lane < S::kWarps ? sm.warp_sum[lane] : 0u, winc = warp_inclusive(w);
        const int src = __ffs(__ballot_sync(0xffffffffu, winc >= want)) - 1;
        uint32_t run = __shfl_sync(0xffffffffu, winc - w, src);
        if (warp == src) {
            const uint32_t inc = run + warp_inclusive(sum);
            if (lane == __ffs(__ballot_sync(0xffffffffu, inc >= want)) - 1) {
                run = inc - sum;
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    if (run < want && run + c[j] >= want) {
                        sm.digit = PER * tid + j;
                        sm.before = run;
                        sm.in_digit = c[j];
                    }
                    run += c[j];
                }
            }
        }
        __syncthreads();
        const uint32_t digit = sm.digit;
        prefix |= digit << shift;
        mask |= (uint32_t)(S::kBins - 1) << shift;
        want -= sm.before;
        const uint32_t next = prefix + (1u << shift);
        if (shift && sm.in_digit == want && next) {  // all of this digit's keys
            *thr = next;
            *need = 0;
            return;
        }
        if (shift == 0) break;
        // (the last digit may overlap the one before: those bits are the prefix's already)
        shift = shift >= S::kBits ? shift - S::kBits : 0;
    }
    *thr = prefix;
    *need = want;
}

// Where each key stands: *taken bit u says whether key u is picked, before[u] how many picked
// ones come before it in index order. All threads call it; block barriers lie between what they
// read before the call and what they write after it.
template <int THREADS, int KEYS>
__device__ __forceinline__ void pick_places(const uint32_t (&k)[KEYS], int n, uint32_t thr, uint32_t need, PickSmem<THREADS>& sm,
                                            uint32_t* taken, uint32_t (&before)[KEYS]) {
    constexpr int W = THREADS / 32, N = KEYS * W;  // rows of 32 entries, in index order
    static_assert(N <= 256, "sm.tot");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t below = (1u << lane) - 1u;
#pragma unroll
    for (int u = 0; u < KEYS; ++u) {
        const bool in = u * THREADS + tid < n;
        const uint32_t lt = __ballot_sync(0xffffffffu, in && k[u] < thr), eq = __ballot_sync(0xffffffffu, in && k[u] == thr);
        before[u] = (uint32_t)__popc(lt & below) | (uint32_t)__popc(eq & below) << 16;  // in the row
        if (lane == 0) sm.tot[u * W + warp] = (uint32_t)__popc(lt) | (uint32_t)__popc(eq) << 16;
    }
    __syncthreads();
    if (warp == 0) {
        constexpr int PER = (N + 31) / 32;
        uint32_t c[PER], sum = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) sum += c[j] = PER * lane + j < N ? sm.tot[PER * lane + j] : 0u;
        uint32_t run = warp_inclusive(sum) - sum;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            if (PER * lane + j < N) sm.tot[PER * lane + j] = run;
            run += c[j];
        }
    }
    __syncthreads();
    *taken = 0;
#pragma unroll
    for (int u = 0; u < KEYS; ++u) {
        const uint32_t at = before[u] + sm.tot[u * W + warp], eq = at >> 16;
        const bool in = u * THREADS + tid < n;
        if (in && (k[u] < thr || (k[u] == thr && eq < need))) *taken |= 1u << u;
        before[u] = (at & 0xffffu) + min(eq, need);
    }
}

// SMs of the current device.
inline cudaError_t sm_count(int* sms) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    return e != cudaSuccess ? e : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

// Lets `kern` use `bytes` of shared memory, asked for once per device.
template <class K>
cudaError_t allow_smem(K kern, size_t bytes, std::atomic<uint64_t>& devices) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (devices.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) devices.fetch_or(bit, std::memory_order_release);
    return e;
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

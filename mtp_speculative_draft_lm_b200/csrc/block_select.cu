// Block selection (mtp_block_select) and eviction (mtp_block_evict) of the block-scaled cache.
//
// Selection: a block's score for a token and kv head is the largest, over the group's query
// heads, of an 8-bit dot product with the block's mean key. The dot is a whole number (127 127
// 256 < 2^24) and each fp32 step is rounded to nearest, so the scores, and with them the chosen
// blocks, are the same bits everywhere; ties go to the lowest index. The scores are bound by
// reading the means (hd + 4 bytes per block and head); the choice is four histogram passes
// over the scores by one CTA for each token and head, then one ordered pass that writes the
// list ascending.
//
// Eviction: the same choice of the smallest accumulated weights by one CTA per sequence, and
// one ordered pass that moves the table and the weights up in place.
#include <cuda_runtime.h>
#include <stdint.h>

#include "block_cache.cuh"
#include "common.cuh"
#include "kernels.h"

namespace mtp {
namespace {

constexpr int kScThreads = 256;
constexpr int kMaxGroup = 16;

struct SelectParams {
    BlockCache c;
    BlockBatch t;
    const uint16_t* q;
    int64_t q_stride;
    int group;
    int n_sel, n_first, n_last;
    int32_t* sel;
    float* score;  // [B, T, nkv, n_table]
};

// Grid (rows = B T nkv, chunks of kScThreads blocks): one block's score per thread.
template <int HD>
__global__ void __launch_bounds__(kScThreads) block_score_kernel(const __grid_constant__ SelectParams p) {
    __shared__ __align__(16) int8_t q8[kMaxGroup][HD];
    __shared__ float sq[kMaxGroup];
    const int64_t row = blockIdx.x;
    const int g = (int)(row % p.c.nkv);
    const int64_t bt = row / p.c.nkv;
    const int b = (int)(bt / p.t.T), tok = (int)(bt % p.t.T);
    const SeqStep s = seq_step(p.t, b);
    if (tok >= s.q) return;
    const int nb = blocks_of(s.len - s.q + tok + 1, p.c.bs, p.t.n_table);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int j0 = blockIdx.y * kScThreads; j0 < nb; j0 += gridDim.y * kScThreads) {
        if (j0 == (int)(blockIdx.y * kScThreads)) {
            for (int h = warp; h < p.group; h += kScThreads / 32) {
                const uint16_t* src = p.q + bt * p.q_stride + ((int64_t)g * p.group + h) * HD;
                float v[HD / 32], mx = 0.f;
                bool odd = false;  // an infinity or NaN
#pragma unroll
                for (int i = 0; i < HD / 32; ++i) {
                    v[i] = bf16_to_f32(src[lane + 32 * i]);
                    mx = fmaxf(mx, fabsf(v[i]));
                    odd = odd || !(fabsf(v[i]) < INFINITY);
                }
#pragma unroll
                for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                odd = __any_sync(0xffffffffu, odd);
                const float sc = __fmul_rn(mx, kInv127);
#pragma unroll
                for (int i = 0; i < HD / 32; ++i)
                    q8[h][lane + 32 * i] = odd || sc == 0.f ? 0 : (int8_t)__float2int_rn(__fdiv_rn(v[i], sc));
                if (lane == 0) sq[h] = odd ? -1.f : sc;
            }
            __syncthreads();
        }
        const int j = j0 + threadIdx.x;
        if (j < nb) {
            const int phys = table_block(p.t, p.c.num_blocks, b, j);
            float best = -INFINITY;
            if (phys >= 0) {
                const int64_t at = (int64_t)phys * p.c.nkv + g;
                const int4* m = reinterpret_cast<const int4*>(p.c.k_mean + at * HD);
                const float sk = p.c.k_mean_scale[at];
                int dot[kMaxGroup];
#pragma unroll
                for (int h = 0; h < kMaxGroup; ++h) dot[h] = 0;
                for (int i = 0; i < HD / 16; ++i) {
                    const int4 mv = m[i];
#pragma unroll
                    for (int h = 0; h < kMaxGroup; ++h)
                        if (h < p.group) {
                            const int4 qv = *reinterpret_cast<const int4*>(&q8[h][16 * i]);
                            dot[h] = __dp4a(mv.x, qv.x, dot[h]);
                            dot[h] = __dp4a(mv.y, qv.y, dot[h]);
                            dot[h] = __dp4a(mv.z, qv.z, dot[h]);
                            dot[h] = __dp4a(mv.w, qv.w, dot[h]);
                        }
                }
                bool nan = false;
#pragma unroll
                for (int h = 0; h < kMaxGroup; ++h)
                    if (h < p.group && sq[h] >= 0.f) {
                        const float f = __fmul_rn((float)dot[h], __fmul_rn(sq[h], sk));
                        nan = nan || f != f;
                        best = fmaxf(best, f);
                    }
                if (nan) best = __uint_as_float(0x7fc00000u);
            } else {
                raise_flag(p.t.dev_err, DEVFLAG_BAD_SLOT);
            }
            p.score[row * p.t.n_table + j] = best;
        }
    }
}

// One CTA per (sequence, token, kv head).
__global__ void __launch_bounds__(kPickThreads) block_choose_kernel(const __grid_constant__ SelectParams p) {
    __shared__ PickSmem sm;
    const int64_t row = blockIdx.x;
    const int64_t bt = row / p.c.nkv;
    const int b = (int)(bt / p.t.T), tok = (int)(bt % p.t.T);
    const SeqStep s = seq_step(p.t, b);
    if (tok >= s.q) return;
    const int lim = s.len - s.q + tok + 1;
    const int nb = blocks_of(lim, p.c.bs, p.t.n_table);
    if (threadIdx.x == 0 && lim > 0 && (lim - 1) / p.c.bs >= p.t.n_table) raise_flag(p.t.dev_err, DEVFLAG_BAD_SLOT);
    int32_t* out = p.sel + row * p.n_sel;
    for (int i = threadIdx.x; i < p.n_sel; i += kPickThreads)
        if (i >= nb) out[i] = -1;
    if (nb <= p.n_sel) {
        for (int i = threadIdx.x; i < nb; i += kPickThreads) out[i] = i;
        return;
    }
    const float* score = p.score + row * p.t.n_table;
    auto key = [&](int i) -> uint32_t {  // smaller is better; the forced blocks before all others
        return i < p.n_first || i >= nb - p.n_last ? 0u : ~order_key(__ldcg(score + i));
    };
    uint32_t thr;
    int need;
    pick_threshold(key, nb, p.n_sel, sm, &thr, &need);
    pick_in_order(key, nb, thr, need, sm, [](int) { return 0; },
                  [&](int i, bool taken, uint32_t before, int) {
                      if (taken) out[before] = i;
                  });
}

struct EvictParams {
    const int32_t* table;
    int64_t n_table;
    const int32_t* lens;
    const float* mass;
    int bs, keep, n_first, n_last;
    int32_t* out_table;
    int32_t* out_lens;
    float* out_mass;
    int32_t* freed;
    int32_t* n_freed;
};

// One CTA per sequence.
__global__ void __launch_bounds__(kPickThreads) block_evict_kernel(const __grid_constant__ EvictParams p) {
    __shared__ PickSmem sm;
    const int b = blockIdx.x, tid = threadIdx.x;
    const int n = (int)p.n_table;
    const int len = max(p.lens[b], 0);
    __syncthreads();  // (out_lens may be lens)
    const int nb = blocks_of(len, p.bs, n);
    const int go = max(nb - p.keep, 0);
    const int64_t base = (int64_t)b * p.n_table;
    const int32_t* table = p.table + base;
    const float* mass = p.mass + base;
    int32_t* out_table = p.out_table + base;
    float* out_mass = p.out_mass + base;
    int32_t* freed = p.freed + base;
    struct Entry {
        int32_t block;
        float mass;
    };
    if (go > 0) {
        auto key = [&](int i) -> uint32_t {  // smallest mass first; protected blocks last of all
            return i < p.n_first || i >= nb - p.n_last ? 0xffffffffu : order_key(mass[i]);
        };
        uint32_t thr;
        int need;
        pick_threshold(key, nb, go, sm, &thr, &need);
        pick_in_order(key, nb, thr, need, sm, [&](int i) { return Entry{table[i], mass[i]}; },
                      [&](int i, bool taken, uint32_t before, Entry e) {
                          if (taken) {
                              freed[before] = e.block;
                          } else {
                              out_table[i - (int)before] = e.block;
                              out_mass[i - (int)before] = e.mass;
                          }
                      });
    } else {
        for (int i = tid; i < nb; i += kPickThreads) {
            out_table[i] = table[i];
            out_mass[i] = mass[i];
        }
    }
    for (int i = nb - go + tid; i < n; i += kPickThreads) {
        out_table[i] = -1;
        out_mass[i] = 0.f;
    }
    for (int i = go + tid; i < n; i += kPickThreads) freed[i] = -1;
    if (tid == 0) {
        p.out_lens[b] = len - go * p.bs;
        p.n_freed[b] = go;
    }
}

}  // namespace

size_t block_select_ws_bytes(const BlockCache& c, int B, int T, int64_t n_table) {
    return (((size_t)B * T * c.nkv * n_table * sizeof(float)) + 15) & ~(size_t)15;
}

cudaError_t block_select_launch(const BlockCache& c, const BlockBatch& t, const uint16_t* q,
                                int64_t q_stride, int nq, int n_sel, int n_first, int n_last,
                                int32_t* sel, void* ws, cudaStream_t s) {
    SelectParams p{c, t, q, q_stride, nq / c.nkv, n_sel, n_first, n_last, sel, static_cast<float*>(ws)};
    const int64_t rows = (int64_t)t.B * t.T * c.nkv;
    if (rows > INT32_MAX) return cudaErrorInvalidValue;
    int64_t chunks = (t.n_table + kScThreads - 1) / kScThreads;
    if (chunks > 1024) chunks = 1024;
    const dim3 grid((unsigned)rows, (unsigned)chunks);
    if (c.hd == 64) block_score_kernel<64><<<grid, kScThreads, 0, s>>>(p);
    else if (c.hd == 128) block_score_kernel<128><<<grid, kScThreads, 0, s>>>(p);
    else block_score_kernel<256><<<grid, kScThreads, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    block_choose_kernel<<<(unsigned)rows, kPickThreads, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t block_evict_launch(int B, const int32_t* table, int64_t n_table, const int32_t* seq_lens,
                               const float* mass, int bs, int keep, int n_first, int n_last,
                               int32_t* out_table, int32_t* out_lens, float* out_mass, int32_t* freed,
                               int32_t* n_freed, cudaStream_t s) {
    EvictParams p{table, n_table, seq_lens, mass, bs, keep, n_first, n_last, out_table, out_lens,
                  out_mass, freed, n_freed};
    block_evict_kernel<<<(unsigned)B, kPickThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace mtp

// Block selection (mtp_block_select) and eviction (mtp_block_evict) of the block-scaled cache.
//
// Selection: a block's score for a token and kv head is the largest, over the group's query
// heads, of an 8-bit dot product with the block's mean key. The dot is a whole number (127 127
// 256 < 2^24, as fp32 exact) and each fp32 step is rounded to nearest, so the scores, and with
// them the chosen blocks, are the same bits everywhere; ties go to the lowest index. The
// scores are bound by reading the means (hd + 4 bytes per block and head): a warp takes 32
// blocks of a head at a time, whose bytes are the A operand of mma.sync m16n8k32 as they come
// (a lane's 16-byte loads, the K dimension permuted alike in q), for all of the step's tokens.
// (On f16 instructions, bytes made f16 by permutes, the same call issued an eighth more
// instructions.) 16 sequences of up to 131,072 positions and two tokens take 27 us, 2.6 TB/s: the
// loads' latency with 16 warps per SM. Bulk copies of a block's heads at once took 32 (a warp's
// lanes issue theirs one after the other), a ring of 16-byte copies 48.
// The choice is one CTA for each token and head, its keys in registers (tables of more than 8,192
// blocks: read again for each digit and for the places): a search for the last
// chosen key, then one prefix sum that gives every chosen block its place in the ascending list;
// 256 lists of 256 from up to 8,192 blocks take 10 us, most of it the search's barriers.
//
// Eviction: the same choice of the smallest accumulated weights by one CTA per sequence, whose
// prefix sum moves the table and the weights up, in place where asked (256 sequences of up to
// 8,192 blocks: 20 us). The forms of 1,024 threads are held to 32 registers and spill 28 bytes (all
// keys in registers) and 100 (keys read again); one CTA per SM with 64 took 21.5 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "block_cache.cuh"
#include "common.cuh"
#include "kernels.h"

namespace mtp {
namespace {

constexpr int kScThreads = 256;
constexpr int kPartBlocks = kScThreads / 32 * 32;  // blocks that a CTA's warps score at a time
constexpr int kMostRounds = 4;
constexpr int kScRows = 64;  // query rows in 8 bits (padded groups) at a time

// Sum over the block's threads, in every one of them.
template <int THREADS>
__device__ __forceinline__ int block_sum(int v, PickSmem<THREADS>& sm) {
    v = __reduce_add_sync(0xffffffffu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sm.warp_sum[threadIdx.x >> 5] = (uint32_t)v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return __reduce_add_sync(0xffffffffu, lane < THREADS / 32 ? (int)sm.warp_sum[lane] : 0);
}

struct SelectParams {
    BlockCache c;
    BlockBatch t;
    const uint16_t* q;
    int64_t q_stride;
    int group;
    int n_sel, n_first, n_last;
    int32_t* sel;
    uint32_t* keys;  // [B, T, nkv, n_table]: the score's order, smallest best
    int part;        // blocks of a CTA (the score's): a multiple of kPartBlocks
};

// D[16 x 8] += A[16 x 32] B[32 x 8], 8-bit integers.
__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float reciprocal(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Bytes between the 8-bit query rows in shared memory: two rows' 64-byte pieces in other banks.
template <int HD>
__host__ __device__ constexpr int q8_pitch() { return HD == 64 ? 64 : HD + 64; }
// (A token takes 8 or 16 rows there: its group, padded to the matrix unit's columns.)

// Grid (kv heads, parts of the blocks, sequences). The query rows are quantized to shared
// memory up to kScRows at a time; a warp has the next tile's blocks looked up while it waits for
// this tile's means.
template <int HD>
__global__ void __launch_bounds__(kScThreads) block_score_kernel(const __grid_constant__ SelectParams p) {
    constexpr int C = HD / 64;  // 16-byte chunks of a lane, 64 bytes apart
    __shared__ __align__(16) uint8_t q8[kScRows * q8_pitch<HD>()];
    __shared__ __align__(16) float2 sq[kScRows];  // scale; 0, or -infinity where the row does not count
    const int g = blockIdx.x, b = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch_dependents();
    const SeqStep s = seq_step(p.t, b);
    const int nb = blocks_of(s.len, p.c.bs, p.t.n_table);
    const int part0 = (int)blockIdx.y * p.part;
    if (s.q == 0 || part0 >= nb) return;
    const int gr_log = p.group > 8 ? 4 : 3, gr = 1 << gr_log, chunk = kScRows >> gr_log;  // a token's rows; tokens at a time
    const int gid = lane >> 2, tig = lane & 3;
    const int j_first = part0 + warp * 32, j_end = min(nb, part0 + p.part);
    uint32_t* const keys = p.keys + ((int64_t)b * p.t.T * p.c.nkv + g) * p.t.n_table;
    const int64_t key_step = (int64_t)p.c.nkv * p.t.n_table;
    const int8_t* const means = p.c.k_mean + (int64_t)g * HD + 16 * tig;
    const float* const scales = p.c.k_mean_scale + g;
    const int32_t* table = p.t.table + (int64_t)b * p.t.n_table;
    const uint32_t blocks = (uint32_t)p.c.num_blocks;
    auto look_up = [&](int j, int (&n)[4]) {  // blocks j + gid + 8 h (-1: none)
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            n[h] = j + gid + 8 * h < nb ? __ldg(table + j + gid + 8 * h) : -1;
            if ((uint32_t)n[h] >= blocks) {
                if (j + gid + 8 * h < nb && tig == 0) raise_flag(p.t.dev_err, DEVFLAG_BAD_SLOT);
                n[h] = -1;
            }
        }
    };
    for (int t0 = 0; t0 < s.q; t0 += chunk) {
        const int t1 = min(s.q, t0 + chunk), rows = (t1 - t0) * gr;
        int next[4];
        look_up(j_first, next);
        // two tiles of 16 blocks; rows gid and gid + 8 of tile u: blocks j0 + gid + 8 (2 u + {0, 1})
        uint4 m[4][C];
        float sk[4];
        uint32_t has = 0;
        auto fetch = [&](int j0) {  // the blocks looked up last; those after them are looked up
            has = 0;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                sk[h] = 0.f;
#pragma unroll
                for (int c = 0; c < C; ++c) m[h][c] = make_uint4(0, 0, 0, 0);
                if (next[h] >= 0) {
                    has |= 1u << h;
                    const int64_t at = (int64_t)next[h] * p.c.nkv;
                    sk[h] = scales[at];
#pragma unroll
                    for (int c = 0; c < C; ++c) m[h][c] = ldg_stream(means + at * HD + 64 * c);
                }
            }
            if (j0 + kPartBlocks < j_end) look_up(j0 + kPartBlocks, next);
        };
        fetch(j_first);  // (they arrive while the query rows are quantized)
        if (t0) __syncthreads();  // the earlier rows have been used
        // HD / 8 lanes per row, 8 values each: one load and one pass for 16 rows of 128
        constexpr int LPR = HD / 8, RPW = 32 / LPR;
        for (int r = warp * RPW + lane / LPR; r < rows; r += kScThreads / 32 * RPW) {  // (whole warps: rows is a multiple of 8)
            const int tok = t0 + (r >> gr_log), i = r & (gr - 1), l = lane % LPR;
            const bool has = i < p.group;
            uint4 x = make_uint4(0, 0, 0, 0);
            if (has) x = *reinterpret_cast<const uint4*>(p.q + ((int64_t)b * p.t.T + tok) * p.q_stride + ((int64_t)g * p.group + i) * HD + 8 * l);
            const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
            uint32_t top = 0;  // the largest magnitude's bits: infinities and NaN above all others
#pragma unroll
            for (int k = 0; k < 4; ++k) top = __vmaxu2(top, xw[k] & 0x7fff7fffu);
            top = max(top & 0xffffu, top >> 16);
#pragma unroll
            for (int o = LPR / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            const bool odd = !has || top >= 0x7f80u;  // no head, or one with an infinity or NaN
            const float sc = odd ? 0.f : __fmul_rn(bf16_to_f32((uint16_t)top), kInv127);
            // rint(v / sc), as the units of a float 1.5 2^23 above: by the reciprocal, and by the
            // division itself where one of the values is within 10^-4 of a half (the product's
            // error is below 5 10^-5) or the scale is tiny
            const bool tiny = sc < 1e-30f;
            const float inv = tiny ? 0.f : reciprocal(sc);
            float d[8], far = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float v = k & 1 ? bf16_hi(xw[k >> 1]) : bf16_lo(xw[k >> 1]);
                d[k] = odd ? 12582912.f : fmaf(v, inv, 12582912.f);
                far = fmaxf(far, fabsf(fmaf(v, inv, 12582912.f - d[k])));
            }
            if (sc > 0.f && (tiny || far > 0.4999f))
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    d[k] = rintf(__fdiv_rn(k & 1 ? bf16_hi(xw[k >> 1]) : bf16_lo(xw[k >> 1]), sc)) + 12582912.f;
            uint32_t w[2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
                w[k] = __byte_perm(__byte_perm(__float_as_uint(d[4 * k]), __float_as_uint(d[4 * k + 1]), 0x0040),
                                   __byte_perm(__float_as_uint(d[4 * k + 2]), __float_as_uint(d[4 * k + 3]), 0x0040), 0x5410);
            *reinterpret_cast<uint2*>(q8 + r * q8_pitch<HD>() + 8 * l) = make_uint2(w[0], w[1]);
            if (l == 0) sq[r] = odd ? make_float2(0.f, -INFINITY) : make_float2(sc, 0.f);
        }
        __syncthreads();
        for (int j0 = j_first; j0 < j_end; j0 += kPartBlocks) {
            if (j0 > j_first) fetch(j0);
            // lane tig of a row's four writes block j0 + gid + 8 tig
            const int j = j0 + gid + 8 * tig;
            uint32_t* out = keys + t0 * key_step + j;
            const bool there = (has >> tig) & 1u;
            for (int r1 = 0; r1 < rows; r1 += gr) {
                float best[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                uint32_t nan = 0;  // rows (bit h) with a NaN
                for (int r0 = r1; r0 < r1 + gr; r0 += 8) {
                    // sums onto 1.5 2^23 as fp32 bits: below 2^22, they are that float's units
                    int d[2][4];
#pragma unroll
                    for (int k = 0; k < 8; ++k) d[k >> 2][k & 3] = 0x4B400000;
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        const uint4 q = *reinterpret_cast<const uint4*>(q8 + (r0 + gid) * q8_pitch<HD>() + 64 * c + 16 * tig);
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            mma_s8(d[u], m[2 * u][c].x, m[2 * u + 1][c].x, m[2 * u][c].y, m[2 * u + 1][c].y, q.x, q.y);
                            mma_s8(d[u], m[2 * u][c].z, m[2 * u + 1][c].z, m[2 * u][c].w, m[2 * u + 1][c].w, q.z, q.w);
                        }
                    }
                    const float4 sc = *reinterpret_cast<const float4*>(&sq[r0 + 2 * tig]);  // rows 2 tig, 2 tig + 1
                    float f[4][2], any = 0.f;
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        f[h][0] = __fmul_rn(__int_as_float(d[h >> 1][2 * (h & 1)]) - 12582912.f, __fmul_rn(sc.x, sk[h]));
                        f[h][1] = __fmul_rn(__int_as_float(d[h >> 1][2 * (h & 1) + 1]) - 12582912.f, __fmul_rn(sc.z, sk[h]));
                        best[h] = fmaxf(best[h], fmaxf(f[h][0] + sc.y, f[h][1] + sc.w));
                        any += f[h][0] + f[h][1];
                    }
                    // a NaN (of a mean's scale, or 0 times an overflown product): which rows have one
                    if (__any_sync(0xffffffffu, any != any))
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            const bool mine = (sc.y == 0.f && f[h][0] != f[h][0]) || (sc.w == 0.f && f[h][1] != f[h][1]);
                            if ((__ballot_sync(0xffffffffu, mine) >> (4 * gid)) & 15u) nan |= 1u << h;
                        }
                }
                // the largest over a row's four lanes, lane tig going on with row h = tig
                const bool h2 = tig & 2, h1 = tig & 1;
                const float a0 = fmaxf(h2 ? best[2] : best[0], __shfl_xor_sync(0xffffffffu, h2 ? best[0] : best[2], 2));
                const float a1 = fmaxf(h2 ? best[3] : best[1], __shfl_xor_sync(0xffffffffu, h2 ? best[1] : best[3], 2));
                float v = fmaxf(h1 ? a1 : a0, __shfl_xor_sync(0xffffffffu, h1 ? a0 : a1, 1));
                if ((nan >> tig) & 1u) v = __uint_as_float(0x7fc00000u);
                if (j < j_end) *out = ~order_key(there ? v : -INFINITY);
                out += key_step;
            }
        }
    }
}

// One CTA per (sequence, token, kv head). ALL: the CTA holds every key (n_table <= THREADS KEYS);
// else they are read again (from L2) for each digit and then in order, THREADS KEYS at a time.
template <int THREADS, int KEYS, bool ALL>
__global__ void __launch_bounds__(THREADS, KEYS == 16 ? 2 : 2048 / THREADS) block_choose_kernel(const __grid_constant__ SelectParams p) {
    __shared__ PickSmem<THREADS> sm;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const int64_t bt = row / p.c.nkv;
    const int b = (int)(bt / p.t.T), tok = (int)(bt % p.t.T);
    const SeqStep s = seq_step(p.t, b);  // (written before the kernel that lets this one start)
    pdl_wait();
    if (tok >= s.q) return;
    const int lim = s.len - s.q + tok + 1;
    const int nb = blocks_of(lim, p.c.bs, p.t.n_table);
    if (tid == 0 && lim > 0 && (lim - 1) / p.c.bs >= p.t.n_table) raise_flag(p.t.dev_err, DEVFLAG_BAD_SLOT);
    int32_t* out = p.sel + row * p.n_sel;
    for (int i = tid; i < p.n_sel; i += THREADS)
        if (i >= nb) out[i] = -1;
    if (nb <= p.n_sel) {
        for (int i = tid; i < nb; i += THREADS) out[i] = i;
        return;
    }
    const uint32_t* keys = p.keys + row * p.t.n_table;
    auto load = [&](int base, uint32_t (&k)[KEYS]) {  // the forced blocks before all others
#pragma unroll
        for (int u = 0; u < KEYS; ++u) {
            const int i = base + u * THREADS + tid;
            k[u] = i < p.n_first || i >= nb - p.n_last ? 0u : keys[i];
        }
    };
    uint32_t k[KEYS], thr, need, before[KEYS], taken;
    if (ALL) load(0, k);
    pick_threshold<THREADS>([&](auto f) {
        for (int base = 0; base < nb; base += THREADS * KEYS) {
            if (!ALL) load(base, k);
#pragma unroll
            for (int u = 0; u < KEYS; ++u)
                if (base + u * THREADS + tid < nb) f(k[u]);
            if (ALL) break;
        }
    }, (uint32_t)p.n_sel, sm, &thr, &need);
    int done = 0;  // picked so far, the last `need` of them among the keys equal to thr
    for (int base = 0; base < nb && done < p.n_sel; base += THREADS * KEYS) {
        if (!ALL) load(base, k);
        pick_places<THREADS, KEYS>(k, nb - base, thr, need, sm, &taken, before);
#pragma unroll
        for (int u = 0; u < KEYS; ++u)
            if ((taken >> u) & 1u) out[done + (int)before[u]] = base + u * THREADS + tid;
        if (ALL) break;
        // what this part took, and how many of the equal keys are left for the next
        int lt = 0, eq = 0;
#pragma unroll
        for (int u = 0; u < KEYS; ++u)
            if ((taken >> u) & 1u) k[u] == thr ? ++eq : ++lt;
        done += block_sum<THREADS>(lt + eq, sm);
        need -= (uint32_t)block_sum<THREADS>(eq, sm);
    }
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

// One CTA per sequence, THREADS KEYS entries at a time (ALL: there are no more). A part's entries
// are read before any of it is written, and no part writes past itself, so that the outputs may
// be the inputs.
template <int THREADS, int KEYS, bool ALL>
__global__ void __launch_bounds__(THREADS, 2048 / THREADS) block_evict_kernel(const __grid_constant__ EvictParams p) {
    __shared__ PickSmem<THREADS> sm;
    const int b = blockIdx.x, tid = threadIdx.x;
    const int n = (int)p.n_table;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t base_at = (int64_t)b * p.n_table;
    const int32_t* table = p.table + base_at;
    const float* mass = p.mass + base_at;
    // A short table is read whole while the length is on its way and stays in registers (8
    // sequences of 500 blocks: 3.6 us, 3.9 with reads after the length and after the choice)
    constexpr bool EARLY = ALL && KEYS <= 2;
    int32_t blk0[EARLY ? KEYS : 1];
    float m0[EARLY ? KEYS : 1];
    if (EARLY)
#pragma unroll
        for (int u = 0; u < KEYS; ++u) {
            const int i = u * THREADS + tid;
            blk0[EARLY ? u : 0] = i < n ? table[i] : 0;
            m0[EARLY ? u : 0] = i < n ? mass[i] : 0.f;
        }
    const int len = max(p.lens[b], 0);
    const int nb = blocks_of(len, p.bs, n);
    const int go = max(nb - p.keep, 0);
    int32_t* out_table = p.out_table + base_at;
    float* out_mass = p.out_mass + base_at;
    int32_t* freed = p.freed + base_at;
    auto load = [&](int base, uint32_t (&k)[KEYS]) {  // smallest mass first; protected blocks last of all
#pragma unroll
        for (int u = 0; u < KEYS; ++u) {
            const int i = base + u * THREADS + tid;
            k[u] = i < p.n_first || i >= nb - p.n_last ? 0xffffffffu : order_key(EARLY ? m0[EARLY ? u : 0] : mass[i]);
        }
    };
    uint32_t k[KEYS], thr = 0, need = 0, before[KEYS] = {}, taken = 0;
    if (ALL && go > 0) load(0, k);
    __syncthreads();  // (out_lens may be lens)
    if (go > 0)
        pick_threshold<THREADS>([&](auto f) {
            for (int base = 0; base < nb; base += THREADS * KEYS) {
                if (!ALL) load(base, k);
#pragma unroll
                for (int u = 0; u < KEYS; ++u)
                    if (base + u * THREADS + tid < nb) f(k[u]);
                if (ALL) break;
            }
        }, (uint32_t)go, sm, &thr, &need);
    int done = 0;
    for (int base = 0; base < nb; base += THREADS * KEYS) {
        if (go > 0) {
            if (!ALL) load(base, k);
            pick_places<THREADS, KEYS>(k, nb - base, thr, need, sm, &taken, before);
        }
        constexpr int G = KEYS < 4 ? KEYS : 4;  // entries in registers at a time
#pragma unroll
        for (int u0 = 0; u0 < KEYS; u0 += G) {
            int32_t blk[G];
            float m[G];
#pragma unroll
            for (int u = 0; u < G; ++u) {
                const int i = base + (u0 + u) * THREADS + tid;
                blk[u] = EARLY ? blk0[EARLY ? u0 + u : 0] : i < nb ? table[i] : 0;
                m[u] = EARLY ? m0[EARLY ? u0 + u : 0] : i < nb ? mass[i] : 0.f;
            }
            if (!EARLY) __syncthreads();
#pragma unroll
            for (int u = 0; u < G; ++u) {
                const int i = base + (u0 + u) * THREADS + tid, gone = done + (int)before[u0 + u];
                if (i >= nb) continue;
                if ((taken >> (u0 + u)) & 1u) {
                    freed[gone] = blk[u];
                } else {
                    out_table[i - gone] = blk[u];
                    out_mass[i - gone] = m[u];
                }
            }
        }
        if (ALL || go == 0) {
            if (ALL) break;
            continue;
        }
        int lt = 0, eq = 0;
#pragma unroll
        for (int u = 0; u < KEYS; ++u)
            if ((taken >> u) & 1u) k[u] == thr ? ++eq : ++lt;
        done += block_sum<THREADS>(lt + eq, sm);
        need -= (uint32_t)block_sum<THREADS>(eq, sm);
    }
    for (int i = nb - go + tid; i < n; i += THREADS) {
        out_table[i] = -1;
        out_mass[i] = 0.f;
    }
    for (int i = go + tid; i < n; i += THREADS) freed[i] = -1;
    if (tid == 0) {
        p.out_lens[b] = len - go * p.bs;
        p.n_freed[b] = go;
    }
}

}  // namespace

bool block_select_fits(const BlockCache& c, int B, int T) { return (int64_t)B * T * c.nkv <= INT32_MAX; }

size_t block_select_ws_bytes(const BlockCache& c, int B, int T, int64_t n_table) {
    return (((size_t)B * T * c.nkv * n_table * sizeof(uint32_t)) + 15) & ~(size_t)15;
}

cudaError_t block_select_launch(const BlockCache& c, const BlockBatch& t, const uint16_t* q,
                                int64_t q_stride, int nq, int n_sel, int n_first, int n_last,
                                int32_t* sel, void* ws, cudaStream_t s) {
    SelectParams p{c, t, q, q_stride, nq / c.nkv, n_sel, n_first, n_last, sel, static_cast<uint32_t*>(ws), 0};
    const int64_t rows = (int64_t)t.B * t.T * c.nkv;
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    // a CTA's blocks: as many as leave about four CTAs per SM, at most kMostRounds rounds of its warps
    // (more only where the grid has no room for that many parts)
    const int64_t rounds = t.n_table * t.B * c.nkv / ((int64_t)kPartBlocks * sms * 4);
    const int64_t least = (t.n_table + (int64_t)kPartBlocks * 65535 - 1) / ((int64_t)kPartBlocks * 65535);
    p.part = kPartBlocks * (int)std::max(std::min(std::max<int64_t>(rounds, 1), (int64_t)kMostRounds), least);
    const int64_t parts = (t.n_table + p.part - 1) / p.part;
    const dim3 grid((unsigned)c.nkv, (unsigned)parts, (unsigned)t.B);
    e = c.hd == 64 ? launch_after(block_score_kernel<64>, grid, kScThreads, 0, s, p)
        : c.hd == 128 ? launch_after(block_score_kernel<128>, grid, kScThreads, 0, s, p)
                      : launch_after(block_score_kernel<256>, grid, kScThreads, 0, s, p);
    if (e != cudaSuccess) return e;
    const dim3 g2((unsigned)rows);
    // The fewest threads and keys that hold the table. A barrier of 512 threads costs less than one
    // of 1,024 where several CTAs share an SM (us for scores and choice: 256 rows of up to 8,192
    // blocks 36.6, and 38.1 with 1,024 threads; 512 rows of 2,048 27.1 and 29.5), and a CTA alone
    // on its SM is faster with more threads (128 rows of 2,048 16.2 and 15.5).
    if (t.n_table <= 512) return launch_after(block_choose_kernel<256, 2, true>, g2, 256, 0, s, p);
    if (t.n_table <= 2048 && rows <= 2 * sms) return launch_after(block_choose_kernel<1024, 2, true>, g2, 1024, 0, s, p);
    if (t.n_table <= 2048) return launch_after(block_choose_kernel<512, 4, true>, g2, 512, 0, s, p);
    if (t.n_table <= 8192) return launch_after(block_choose_kernel<512, 16, true>, g2, 512, 0, s, p);
    return launch_after(block_choose_kernel<1024, 8, false>, g2, 1024, 0, s, p);
}

cudaError_t block_evict_launch(int B, const int32_t* table, int64_t n_table, const int32_t* seq_lens,
                               const float* mass, int bs, int keep, int n_first, int n_last,
                               int32_t* out_table, int32_t* out_lens, float* out_mass, int32_t* freed,
                               int32_t* n_freed, cudaStream_t s) {
    EvictParams p{table, n_table, seq_lens, mass, bs, keep, n_first, n_last, out_table, out_lens,
                  out_mass, freed, n_freed};
    const dim3 grid((unsigned)B);
    if (n_table <= 512) return launch_after(block_evict_kernel<256, 2, true>, grid, 256, 0, s, p);
    if (n_table <= 2048) return launch_after(block_evict_kernel<1024, 2, true>, grid, 1024, 0, s, p);
    if (n_table <= 8192) return launch_after(block_evict_kernel<1024, 8, true>, grid, 1024, 0, s, p);
    return launch_after(block_evict_kernel<1024, 8, false>, grid, 1024, 0, s, p);
}

}  // namespace mtp

// Append to the block-scaled paged cache (mtp_block_append): new bf16 K and V rows become E4M3
// codes under one scale for each block and head.
//
// Mathematics: a block's scale is a power of two, s = 2^ceil(log2(a / 448)), a its largest
// finite |x|. E4M3 is a floating format: its relative step does not depend on the scale, so a
// power of two loses nothing against a / 448 but at the subnormal end, and gains that a scale
// which grows (a later row of the block is larger) moves the earlier rows' codes by whole
// binades: they keep their bits unless they become subnormal. a = m 2^E with m in [1, 2):
// 448 = 1.75 2^8, so s = 2^(E - 8) where m <= 1.75 and 2^(E - 7) otherwise: bits, no logarithm.
// The mean key is the exact sum of the code values (multiples of 2^-9 below 2^15: 24 bits, so
// fp32 sums are exact in any order) quantized to 8-bit integers under its own scale.
//
// Bound by HBM for prompts (6 bytes per element of K and V: 4 read in bf16, 2 written... per
// K and V pair) and by launch and load latency for single tokens. A warp takes 16 rows of one
// (sequence, block, head, K or V): its lanes hold 16 bytes of a row each, every row's load is
// in flight before the first is used, and nothing is read twice.
#include <cuda_runtime.h>
#include <stdint.h>

#include "block_cache.cuh"
#include "common.cuh"
#include "kernels.h"

namespace mtp {
namespace {

constexpr int kAppThreads = 128;

struct AppendParams {
    BlockCache c;
    BlockBatch t;
    const uint16_t* k;
    const uint16_t* v;
    int64_t kv_stride;
    int64_t jobs;  // (sequence, touched block, K or V, head)
    int touch;     // blocks that T tokens can touch
};

// Largest finite magnitude of 2 bf16 (as integer bits, each half separately) joined to acc.
__device__ __forceinline__ uint32_t finite_max2(uint32_t acc, uint32_t v) {
    const uint32_t m = v & 0x7fff7fffu;
    return __vmaxu2(acc, m & ~__vcmpgeu2(m, 0x7f807f80u));
}

// The least power of two >= a / 448 within [2^-110, 2^120]; a = bf16 magnitude bits; 0 for 0.
__device__ __forceinline__ float pow2_scale(uint32_t a) {
    if (a == 0) return 0.f;
    int e = (int)(a >> 7) - 8 + ((a & 0x7fu) > 0x60u ? 1 : 0);  // biased; subnormal a clamps below
    e = min(max(e, 127 - 110), 127 + 120);
    return __uint_as_float((uint32_t)e << 23);
}

template <int HD, int BS>
__global__ void __launch_bounds__(kAppThreads) block_append_kernel(const __grid_constant__ AppendParams p) {
    constexpr int WPJ = BS / 16;                // warps per job
    constexpr int JPC = kAppThreads / 32 / WPJ;  // jobs per CTA at a time
    constexpr int LPR = HD / 8;                 // lanes per row (8 values each)
    constexpr int RPI = 32 / LPR;               // rows per load instruction
    constexpr int NI = 16 / RPI;
    __shared__ uint32_t amax_sh[4];
    __shared__ float sum_sh[4][HD];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wj = warp % WPJ;
    const int sub = lane / LPR, chunk = lane % LPR;
    const int64_t step = (int64_t)gridDim.x * JPC;
    for (int64_t job0 = (int64_t)blockIdx.x * JPC; job0 < p.jobs; job0 += step) {
        const int64_t job = job0 + warp / WPJ;
        bool work = job < p.jobs;
        int b = 0, j = 0, g = 0, is_v = 0;
        if (work) {
            g = (int)(job % p.c.nkv);
            const int64_t r = job / p.c.nkv;
            is_v = (int)(r & 1);
            j = (int)((r >> 1) % p.touch);
            b = (int)((r >> 1) / p.touch);
        }
        const SeqStep s = seq_step(p.t, b);
        const int beg = s.len - s.q;          // position of token 0 (below 0: tokens before the sequence)
        const int first = max(beg, 0) / BS;   // the first touched block
        const int64_t lb = (int64_t)first + j;
        work = work && s.q > 0 && lb * BS < s.len;
        int phys = -1;
        if (work) {
            phys = table_block(p.t, p.c.num_blocks, b, lb);
            if (lane == 0 && (phys < 0 || (beg < 0 && j == 0))) raise_flag(p.t.dev_err, DEVFLAG_BAD_SLOT);
            work = phys >= 0;
        }
        const int pos0 = (int)(lb * BS) + 16 * wj;  // this warp's rows: pos0 + [0, 16)
        const bool has_old = beg > lb * BS;
        uint8_t* codes = (is_v ? p.c.v : p.c.k) + (int64_t)max(phys, 0) * p.c.block_stride + (int64_t)g * p.c.head_stride;
        float* scale_at = (is_v ? p.c.v_scale : p.c.k_scale) + (int64_t)max(phys, 0) * p.c.nkv + g;
        const uint16_t* x = (is_v ? p.v : p.k) + (int64_t)b * p.t.T * p.kv_stride + (int64_t)g * HD + 8 * chunk;

        uint4 in[NI];
        uint2 was[NI];
        float s_old = 0.f;
        uint32_t am = 0;
        if (work) {
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int pos = pos0 + i * RPI + sub;
                in[i] = make_uint4(0, 0, 0, 0);
                was[i] = make_uint2(0, 0);
                if (pos >= beg && pos < s.len)
                    in[i] = *reinterpret_cast<const uint4*>(x + (int64_t)(pos - beg) * p.kv_stride);
                else if (pos < beg)
                    was[i] = *reinterpret_cast<const uint2*>(codes + (int64_t)(16 * wj + i * RPI + sub) * p.c.row_stride + 8 * chunk);
            }
            if (has_old) s_old = *scale_at;
#pragma unroll
            for (int i = 0; i < NI; ++i)
                am = finite_max2(finite_max2(finite_max2(finite_max2(am, in[i].x), in[i].y), in[i].z), in[i].w);
            am = max(am & 0xffffu, am >> 16);
            am = __reduce_max_sync(0xffffffffu, am);
        }
        if (WPJ > 1) {  // every warp of the block's job
            if (lane == 0) amax_sh[warp] = am;
            __syncthreads();
            am = 0;
#pragma unroll
            for (int w = 0; w < WPJ; ++w) am = max(am, amax_sh[warp - wj + w]);
        } else {
            __syncwarp();
        }
        float sc = 0.f;
        float sum[8];
#pragma unroll
        for (int d = 0; d < 8; ++d) sum[d] = 0.f;
        if (work) {
            sc = fmaxf(s_old, pow2_scale(am));
            // a power of two's reciprocal is exact, and so is the product's rounding the quotient's
            const bool pow2 = (__float_as_uint(sc) & 0x7fffffu) == 0 && sc >= 1.17549435e-38f && sc <= 8.5e37f;
            const float inv = pow2 ? __fdiv_rn(1.f, sc) : 0.f;
            const bool grow = has_old && sc != s_old;
            const float ratio = grow ? __fdiv_rn(s_old, sc) : 1.f;
            const bool mean = !is_v && p.c.k_mean;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int pos = pos0 + i * RPI + sub;
                const bool isnew = pos >= beg && pos < s.len, isold = pos < beg;
                uint2 o = was[i];
                if (isnew) {
                    const uint32_t w[4] = {in[i].x, in[i].y, in[i].z, in[i].w};
                    uint16_t q[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const float lo = bf16_lo(w[u]), hi = bf16_hi(w[u]);
                        if (pow2) q[u] = f32x2_to_e4m3x2(lo * inv, hi * inv);
                        else if (sc > 0.f) q[u] = f32x2_to_e4m3x2(__fdiv_rn(lo, sc), __fdiv_rn(hi, sc));
                        else q[u] = f32x2_to_e4m3x2(lo, hi);  // zeros (or not finite)
                    }
                    o = make_uint2(q[0] | (uint32_t)q[1] << 16, q[2] | (uint32_t)q[3] << 16);
                } else if (isold && grow) {
                    const uint32_t w[2] = {o.x, o.y};
                    uint16_t q[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const float2 f = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(w[u >> 1] >> (16 * (u & 1)))));
                        q[u] = f32x2_to_e4m3x2(f.x * ratio, f.y * ratio);
                    }
                    o = make_uint2(q[0] | (uint32_t)q[1] << 16, q[2] | (uint32_t)q[3] << 16);
                }
                if (isnew || (isold && grow))
                    *reinterpret_cast<uint2*>(codes + (int64_t)(16 * wj + i * RPI + sub) * p.c.row_stride + 8 * chunk) = o;
                if (mean && (isnew || isold)) {
                    const uint32_t w[2] = {o.x, o.y};
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const float2 f = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(w[u >> 1] >> (16 * (u & 1)))));
                        sum[2 * u] += f.x;
                        sum[2 * u + 1] += f.y;
                    }
                }
            }
        }
        const bool mean = work && !is_v && p.c.k_mean;
        if (mean) {
#pragma unroll
            for (int d = 0; d < 8; ++d)
#pragma unroll
                for (int o = LPR; o < 32; o <<= 1) sum[d] += __shfl_xor_sync(0xffffffffu, sum[d], o);
            if (WPJ > 1 && sub == 0)
#pragma unroll
                for (int d = 0; d < 8; ++d) sum_sh[warp][8 * chunk + d] = sum[d];
        }
        __syncthreads();  // (also: everyone has read amax_sh and the block's scale)
        if (work && wj == 0) {
            if (lane == 0) *scale_at = sc;
            if (mean) {
                float A = 0.f;
#pragma unroll
                for (int d = 0; d < 8; ++d) {
                    if (WPJ > 1) {
                        sum[d] = sum_sh[warp][8 * chunk + d];
#pragma unroll
                        for (int w = 1; w < WPJ; ++w) sum[d] += sum_sh[warp + w][8 * chunk + d];
                    }
                    if (sum[d] != sum[d]) sum[d] = 0.f;
                    A = fmaxf(A, fabsf(sum[d]));
                }
#pragma unroll
                for (int o = 16; o; o >>= 1) A = fmaxf(A, __shfl_xor_sync(0xffffffffu, A, o));
                const float ms = __fmul_rn(A, kInv127);
                uint32_t q[2] = {0, 0};
                if (ms > 0.f)
#pragma unroll
                    for (int d = 0; d < 8; ++d)
                        q[d >> 2] |= ((uint32_t)__float2int_rn(__fdiv_rn(sum[d], ms)) & 255u) << (8 * (d & 3));
                const int64_t row = (int64_t)phys * p.c.nkv + g;
                if (sub == 0)
                    *reinterpret_cast<uint2*>(p.c.k_mean + row * HD + 8 * chunk) = make_uint2(q[0], q[1]);
                const int rows = min(s.len - (int)(lb * BS), BS);
                if (lane == 0) p.c.k_mean_scale[row] = __fdiv_rn(__fmul_rn(ms, sc), (float)rows);
            }
        }
        if (WPJ > 1) __syncthreads();  // sum_sh is read before the next job writes it
    }
}

template <int HD>
cudaError_t launch_append(const AppendParams& p, cudaStream_t s) {
    const int jpc = kAppThreads / 32 / (p.c.bs / 16);
    const int64_t want = (p.jobs + jpc - 1) / jpc;
    const unsigned grid = (unsigned)(want < (1 << 20) ? want : 1 << 20);
    if (p.c.bs == 16) block_append_kernel<HD, 16><<<grid, kAppThreads, 0, s>>>(p);
    else if (p.c.bs == 32) block_append_kernel<HD, 32><<<grid, kAppThreads, 0, s>>>(p);
    else block_append_kernel<HD, 64><<<grid, kAppThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t block_append_launch(const BlockCache& c, const BlockBatch& t, const uint16_t* k,
                                const uint16_t* v, int64_t kv_stride, cudaStream_t s) {
    AppendParams p{c, t, k, v, kv_stride, 0, 0};
    p.touch = (int)((t.T + c.bs - 2) / c.bs + 1);
    if (p.touch > t.n_table) p.touch = (int)t.n_table + 1;  // one more, whose tokens are flagged
    p.jobs = (int64_t)t.B * p.touch * 2 * c.nkv;
    return c.hd == 64 ? launch_append<64>(p, s) : c.hd == 128 ? launch_append<128>(p, s) : launch_append<256>(p, s);
}

}  // namespace mtp

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
// Bound by HBM for prompts (per element of K and V 2 bytes read and 1 written) and by three
// dependent loads (length, block, rows) for single tokens. A warp takes 16 rows of one
// (sequence, block, head, K or V): its lanes hold 16 bytes of a row each, every row's load is
// in flight before the first is used, and nothing is read twice. The heads of K and V are the
// fastest grid dimension, so that a row's bytes are read at about the same time. A prompt of
// 32,768 tokens of 8 heads of 128 takes 41 us (4.9 TB/s; 60% of the issue slots: converting and
// adding up each code), 24 single tokens 3.5 us, 256 of them 7.4 (13.2 with a CTA to a head, three
// of its four warps idle).
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
    int touch;   // blocks that T tokens can touch
    int jt_log;  // log2(blocks of one head that a CTA takes at a time)
};

// Largest magnitude of 2 bf16 each half separately (as integer bits), joined to acc.
__device__ __forceinline__ uint32_t max_bits2(uint32_t acc, uint32_t v) { return __vmaxu2(acc, v & 0x7fff7fffu); }
// The same over finite values alone.
__device__ __forceinline__ uint32_t finite_bits2(uint32_t acc, uint32_t v) {
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

// c0, c1 += the two f16 halves of h, in fp32.
__device__ __forceinline__ void add_halves(float& c0, float& c1, uint32_t h) {
    asm("{\n\t.reg .f16 l, u;\n\tmov.b32 {l, u}, %2;\n\tadd.rn.f32.f16 %0, l, %0;\n\tadd.rn.f32.f16 %1, u, %1;\n\t}"
        : "+f"(c0), "+f"(c1) : "r"(h));
}

// 8 bf16 -> 8 codes of x * inv (inv: a power of two, so that the product is the quotient).
__device__ __forceinline__ uint2 encode8(const uint4& x, float inv) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t q[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) q[u] = f32x2_to_e4m3x2(bf16_lo(w[u]) * inv, bf16_hi(w[u]) * inv);
    return make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
}

// sum[0 .. 8) += the values of 8 codes.
__device__ __forceinline__ void add_codes(float (&sum)[8], const uint2& o) {
    const uint32_t w[2] = {o.x, o.y};
#pragma unroll
    for (int u = 0; u < 4; ++u)
        add_halves(sum[2 * u], sum[2 * u + 1], e4m3x2_to_f16x2((uint16_t)(w[u >> 1] >> (16 * (u & 1)))));
}

// Grid (K or V of each head or of several, groups of touched blocks, sequences). OLD: the earlier
// rows' codes of a block that already has some are asked for together with the new rows, else
// only once they are needed (and the registers hold more rows in flight instead).
template <int HD, int BS, bool OLD>
__global__ void __launch_bounds__(kAppThreads) block_append_kernel(const __grid_constant__ AppendParams p) {
    constexpr int WPJ = BS / 16;                // warps per block
    constexpr int JPC = kAppThreads / 32 / WPJ;  // blocks per CTA at a time
    constexpr int LPR = HD / 8;                 // lanes per row (8 values each)
    constexpr int RPI = 32 / LPR;               // rows per load instruction
    constexpr int NI = 16 / RPI;
    constexpr int DPL = 8 / RPI;                // mean dims that a lane quantizes
    __shared__ uint32_t amax_sh[4];
    __shared__ float sum_sh[4][HD];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wj = warp % WPJ;
    const int sub = lane / LPR, chunk = lane % LPR;
    const int slot = warp / WPJ, jt = 1 << p.jt_log;  // (of JPC) block slots; those of one head
    const int item = (int)blockIdx.x * (JPC >> p.jt_log) + (slot >> p.jt_log);
    const int is_v = item & 1, g = item >> 1, b = blockIdx.z;
    pdl_wait();
    pdl_launch_dependents();
    const SeqStep s = seq_step(p.t, b);
    const int beg = s.len - s.q;         // position of token 0 (below 0: tokens before the sequence)
    const int first = max(beg, 0) / BS;  // the first touched block
    const uint16_t* x = (is_v ? p.v : p.k) + (int64_t)b * p.t.T * p.kv_stride + (int64_t)g * HD + 8 * chunk;
    const bool mean = !is_v && p.c.k_mean;
    for (int j0 = (int)blockIdx.y * jt; j0 < p.touch; j0 += (int)gridDim.y * jt) {
        const int j = j0 + (slot & (jt - 1));
        const int64_t lb = (int64_t)first + j;
        if ((int64_t)(first + j0) * BS >= s.len || s.q == 0) break;  // (the whole CTA's)
        bool work = g < p.c.nkv && j < p.touch && lb * BS < s.len;
        int phys = -1;
        if (work) {
            phys = table_block(p.t, p.c.num_blocks, b, lb);
            if (lane == 0 && (phys < 0 || (beg < 0 && j == 0))) raise_flag(p.t.dev_err, DEVFLAG_BAD_SLOT);
            work = phys >= 0;
        }
        const int pos0 = (int)(lb * BS) + 16 * wj;  // this warp's rows: pos0 + [0, 16)
        const bool has_old = beg > lb * BS;         // rows of the sequence before the new ones
        uint8_t* codes = (is_v ? p.c.v : p.c.k) + (int64_t)max(phys, 0) * p.c.block_stride +
                         (int64_t)g * p.c.head_stride + (int64_t)(16 * wj + sub) * p.c.row_stride + 8 * chunk;
        float* scale_at = (is_v ? p.c.v_scale : p.c.k_scale) + (int64_t)max(phys, 0) * p.c.nkv + g;

        uint4 in[NI];
        uint2 was[OLD ? NI : 1];
        float s_old = 0.f;
        uint32_t am = 0;
        // this lane's rows are pos0 + sub + RPI i: new ones for i in [i0, i1)
        const int i0 = beg > pos0 + sub ? min((beg - pos0 - sub + RPI - 1) / RPI, NI) : 0;
        const int i1 = s.len > pos0 + sub ? min((s.len - pos0 - sub + RPI - 1) / RPI, NI) : 0;
        const int64_t code_step = RPI * p.c.row_stride;
        if (work) {
            const uint16_t* row = x + (int64_t)(pos0 + sub - beg) * p.kv_stride;
            const int64_t step = RPI * p.kv_stride;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                in[i] = make_uint4(0, 0, 0, 0);
                if (i >= i0 && i < i1) in[i] = ldg_stream(row);
                row += step;
            }
            if (has_old) {
                s_old = *scale_at;
                if (OLD)
#pragma unroll
                    for (int i = 0; i < NI; ++i) {
                        was[OLD ? i : 0] = make_uint2(0, 0);
                        if (i < i0) was[OLD ? i : 0] = *reinterpret_cast<const uint2*>(codes + i * code_step);
                    }
            }
#pragma unroll
            for (int i = 0; i < NI; ++i) am = max_bits2(max_bits2(max_bits2(max_bits2(am, in[i].x), in[i].y), in[i].z), in[i].w);
            if (__any_sync(0xffffffffu, __vcmpgeu2(am, 0x7f807f80u))) {  // an infinity or NaN
                am = 0;
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    am = finite_bits2(finite_bits2(finite_bits2(finite_bits2(am, in[i].x), in[i].y), in[i].z), in[i].w);
            }
            am = __reduce_max_sync(0xffffffffu, max(am & 0xffffu, am >> 16));
        }
        if (WPJ > 1) {  // every warp of the block
            if (lane == 0) amax_sh[warp] = am;
            __syncthreads();
            am = 0;
#pragma unroll
            for (int w = 0; w < WPJ; ++w) am = max(am, amax_sh[warp - wj + w]);
        }
        float sc = 0.f;
        float sum[8];
#pragma unroll
        for (int d = 0; d < 8; ++d) sum[d] = 0.f;
        if (work) {
            sc = fmaxf(s_old, pow2_scale(am));
            // a power of two's reciprocal is exact, and so is the product's rounding the quotient's
            const bool pow2 = (__float_as_uint(sc) & 0x7fffffu) == 0 && sc >= 1.17549435e-38f && sc <= 8.5e37f;
            const float by = sc > 0.f ? sc : 1.f;  // (x itself where everything is zero or not finite)
            if ((pow2 || sc == 0.f) && !has_old) {
                // (rows behind the sequence are zeros, and count as such in the mean)
                const float inv = pow2 ? __uint_as_float((254u << 23) - __float_as_uint(sc)) : 1.f;
                uint8_t* out = codes;
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const uint2 o = encode8(in[i], inv);
                    if (i < i1) *reinterpret_cast<uint2*>(out) = o;
                    out += code_step;
                    if (mean) add_codes(sum, o);
                }
            } else {
                const bool grow = has_old && sc != s_old;
                const float ratio = grow ? __fdiv_rn(s_old, sc) : 1.f;
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    uint2 o = make_uint2(0, 0);
                    uint8_t* out = codes + i * code_step;
                    if (i < i0) {
                        o = OLD ? was[OLD ? i : 0] : *reinterpret_cast<const uint2*>(out);
                        if (grow) {
                            const uint32_t w[2] = {o.x, o.y};
                            uint32_t q[4];
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const float2 f = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(w[u >> 1] >> (16 * (u & 1)))));
                                q[u] = f32x2_to_e4m3x2(f.x * ratio, f.y * ratio);
                            }
                            o = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
                            *reinterpret_cast<uint2*>(out) = o;
                        }
                    } else if (i < i1) {
                        if (pow2) {
                            o = encode8(in[i], __uint_as_float((254u << 23) - __float_as_uint(sc)));
                        } else {  // a scale that an append did not write
                            const uint32_t w[4] = {in[i].x, in[i].y, in[i].z, in[i].w};
                            uint32_t q[4];
#pragma unroll
                            for (int u = 0; u < 4; ++u) q[u] = f32x2_to_e4m3x2(__fdiv_rn(bf16_lo(w[u]), by), __fdiv_rn(bf16_hi(w[u]), by));
                            o = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
                        }
                        *reinterpret_cast<uint2*>(out) = o;
                    }
                    if (mean) add_codes(sum, o);
                }
            }
        }
        if (work && mean) {
#pragma unroll
            for (int d = 0; d < 8; ++d)
#pragma unroll
                for (int o = LPR; o < 32; o <<= 1) sum[d] += __shfl_xor_sync(0xffffffffu, sum[d], o);
            if (WPJ > 1 && sub == 0)
#pragma unroll
                for (int d = 0; d < 8; ++d) sum_sh[warp][8 * chunk + d] = sum[d];
        }
        if (WPJ > 1) __syncthreads();
        else __syncwarp();  // (everyone has read the block's scale)
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
                A = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(A)));  // (not negative)
                const float ms = __fmul_rn(A, kInv127);
                // lane (sub, chunk) quantizes dims 8 chunk + DPL sub on
                uint32_t q[2] = {0, 0};
                if (ms > 0.f)
#pragma unroll
                    for (int d = 0; d < DPL; ++d) {
                        float v = sum[d];
#pragma unroll
                        for (int u = 1; u < RPI; ++u) v = sub == u ? sum[u * DPL + d] : v;
                        q[d >> 2] |= ((uint32_t)__float2int_rn(__fdiv_rn(v, ms)) & 255u) << (8 * (d & 3));
                    }
                const int64_t row = (int64_t)phys * p.c.nkv + g;
                int8_t* out = p.c.k_mean + row * HD + 8 * chunk + DPL * sub;
                if (DPL == 8) *reinterpret_cast<uint2*>(out) = make_uint2(q[0], q[1]);
                else if (DPL == 4) *reinterpret_cast<uint32_t*>(out) = q[0];
                else *reinterpret_cast<uint16_t*>(out) = (uint16_t)q[0];
                const int rows = min(s.len - (int)(lb * BS), BS);
                if (lane == 0) p.c.k_mean_scale[row] = __fdiv_rn(__fmul_rn(ms, sc), (float)rows);
            }
        }
        if (WPJ > 1) __syncthreads();  // sum_sh and amax_sh are read before the next blocks write them
    }
}

template <int HD, int BS>
cudaError_t launch_bs(const AppendParams& p, dim3 grid, bool old, cudaStream_t s) {
    return old ? launch_after(block_append_kernel<HD, BS, true>, grid, kAppThreads, 0, s, p)
               : launch_after(block_append_kernel<HD, BS, false>, grid, kAppThreads, 0, s, p);
}

template <int HD>
cudaError_t launch_append(AppendParams p, cudaStream_t s) {
    // a CTA's block slots: for one head as far as a step touches that many blocks, else for several heads
    // (single tokens of 8 heads of 128 with four heads to a CTA, and with one: 24 sequences 3.5 and 3.7
    // us, 40 of them 3.5 and 5.2, 24 of 256-wide heads 5.1 and 8.1)
    const int jpc = kAppThreads / 32 / (p.c.bs / 16);
    while ((1 << p.jt_log) < jpc && (1 << p.jt_log) < p.touch) ++p.jt_log;
    const int jt = 1 << p.jt_log, items = jpc >> p.jt_log;
    const int groups = (p.touch + jt - 1) / jt;
    const dim3 grid((unsigned)((2 * p.c.nkv + items - 1) / items), (unsigned)(groups < 65535 ? groups : 65535), (unsigned)p.t.B);
    // OLD while latency counts, which is while the CTAs fit the SMs at once (us with, without:
    // 24 single tokens of 8 heads 3.5, 4.1; 256 of them 7.4, 7.7, 512 13.3, 11.9; 64 steps of 16
    // tokens 4.4, 5.1, of 64 10.1, 9.3) and most of a step's blocks have earlier rows (16 steps of
    // 64 tokens 4.5, 5.0, of 128 6.1, 5.5; a prompt of 32,768 45.8, 41.4)
    const bool old = p.t.T <= 64 && (int64_t)grid.x * grid.y * grid.z <= 1024;
    return p.c.bs == 16 ? launch_bs<HD, 16>(p, grid, old, s) : p.c.bs == 32 ? launch_bs<HD, 32>(p, grid, old, s)
                                                                            : launch_bs<HD, 64>(p, grid, old, s);
}

}  // namespace

cudaError_t block_append_launch(const BlockCache& c, const BlockBatch& t, const uint16_t* k,
                                const uint16_t* v, int64_t kv_stride, cudaStream_t s) {
    AppendParams p{c, t, k, v, kv_stride, 0, 0};
    p.touch = (int)((t.T + c.bs - 2) / c.bs + 1);
    if (p.touch > t.n_table) p.touch = (int)t.n_table + 1;  // one more, whose tokens are flagged
    return c.hd == 64 ? launch_append<64>(p, s) : c.hd == 128 ? launch_append<128>(p, s) : launch_append<256>(p, s);
}

}  // namespace mtp

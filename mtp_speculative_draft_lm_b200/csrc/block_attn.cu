// Attention over the block-scaled paged cache (mtp_block_attn, mtp_block_sparse_attn).
//
// One warp per query head of a token: an online softmax over the positions it sees, the head's
// dimensions spread over the lanes.
#include <cuda_runtime.h>
#include <stdint.h>

#include "block_cache.cuh"
#include "common.cuh"
#include "kernels.h"

namespace mtp {
namespace {

constexpr int kMaxGroup = 16;
constexpr int kMaxT = 64;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnParams {
    BlockCache c;
    BlockBatch t;
    BlockAttnArgs a;
    int group;
    int tiles;        // 16-position tiles of n_table blocks
    float* row_lse;   // [B, T, nq] base-2 log-sum-exp (with mass)
    float* tile_lse;  // [B, T, nq, tiles] (with mass)
};

template <int HD>
__global__ void __launch_bounds__(128) block_attn_simple_kernel(const __grid_constant__ AttnParams p) {
    constexpr int VEC = HD / 32;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int64_t bt = w / p.a.nq;
    const int i = (int)(w % p.a.nq);
    const int b = (int)(bt / p.t.T), tok = (int)(bt % p.t.T);
    if (b >= p.t.B) return;
    const SeqStep s = seq_step(p.t, b);
    if (tok >= s.q) return;
    const int lim = s.len - s.q + tok + 1;
    const int g = i / p.group, bs = p.c.bs;
    float q[VEC], acc[VEC], m = -INFINITY, l = 0.f;
    for (int d = 0; d < VEC; ++d) {
        q[d] = bf16_to_f32(p.a.q[bt * p.a.q_stride + (int64_t)i * HD + lane * VEC + d]);
        acc[d] = 0.f;
    }
    const int entries = p.a.sel ? p.a.n_sel : blocks_of(lim, bs, p.t.n_table);
    if (!p.a.sel && lim > 0 && (lim - 1) / bs >= p.t.n_table) raise_flag(p.t.dev_err, DEVFLAG_BAD_SLOT);
    for (int e = 0; e < entries; ++e) {
        const int lb = p.a.sel ? p.a.sel[(bt * p.c.nkv + g) * p.a.n_sel + e] : e;
        if (lb < 0) continue;
        const int64_t pos0 = (int64_t)lb * bs;
        const int n = table_block(p.t, p.c.num_blocks, b, lb);
        if (pos0 < lim && n < 0) raise_flag(p.t.dev_err, DEVFLAG_BAD_SLOT);
        const int rows = n < 0 ? 0 : (int)max((int64_t)0, min((int64_t)bs, lim - pos0));
        for (int t0 = 0; t0 < bs; t0 += 16) {
            float tm = -INFINITY, tl = 0.f;
            for (int r = t0; r < min(rows, t0 + 16); ++r) {
                const float ks = p.c.k_scale[(int64_t)n * p.c.nkv + g], vs = p.c.v_scale[(int64_t)n * p.c.nkv + g];
                const int64_t at = (int64_t)n * p.c.block_stride + (int64_t)g * p.c.head_stride + (int64_t)r * p.c.row_stride + lane * VEC;
                float d = 0.f;
                for (int u = 0; u < VEC; ++u) d = fmaf(q[u], e4m3_to_f32(p.c.k[at + u]), d);
                for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
                const float sc = d * (p.a.scale * ks) * kLog2e;
                const float mn = fmaxf(m, sc);
                const float al = m == -INFINITY ? 0.f : exp2f(m - mn), wt = exp2f(sc - mn);
                l = l * al + wt;
                for (int u = 0; u < VEC; ++u) acc[u] = acc[u] * al + wt * vs * e4m3_to_f32(p.c.v[at + u]);
                m = mn;
                const float tn = fmaxf(tm, sc);
                tl = (tm == -INFINITY ? 0.f : tl * exp2f(tm - tn)) + exp2f(sc - tn);
                tm = tn;
            }
            if (p.a.out_mass && lane == 0)
                p.tile_lse[(bt * p.a.nq + i) * p.tiles + (pos0 + t0) / 16] = tl > 0.f ? tm + log2f(tl) : -INFINITY;
        }
    }
    for (int u = 0; u < VEC; ++u)
        p.a.out[(bt * p.a.nq + i) * HD + lane * VEC + u] = f32_to_bf16(l > 0.f || l != l ? acc[u] / l : 0.f);
    if (lane == 0) {
        const float lse2 = l > 0.f || l != l ? m + log2f(l) : -INFINITY;
        if (p.a.out_lse) p.a.out_lse[bt * p.a.nq + i] = lse2 * kLn2;
        if (p.a.out_mass) p.row_lse[bt * p.a.nq + i] = lse2;
    }
}

// out_mass[b, j]: one thread per logical block, the tokens and heads summed in order.
__global__ void __launch_bounds__(128) block_mass_kernel(const __grid_constant__ AttnParams p) {
    const int b = blockIdx.y;
    const int64_t j = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (j >= p.t.n_table) return;
    const SeqStep s = seq_step(p.t, b);
    const int tpb = p.c.bs / 16;
    const int64_t at = (int64_t)b * p.t.n_table + j;
    float sum = 0.f;
    for (int tok = 0; tok < s.q; ++tok) {
        if (j >= blocks_of(s.len - s.q + tok + 1, p.c.bs, p.t.n_table)) continue;
        for (int i = 0; i < p.a.nq; ++i) {
            const int64_t row = ((int64_t)b * p.t.T + tok) * p.a.nq + i;
            const float L = p.row_lse[row];
            for (int u = 0; u < tpb; ++u) {
                const float x = p.tile_lse[row * p.tiles + j * tpb + u];
                if (x != -INFINITY) sum += exp2f(x - L);
            }
        }
    }
    p.a.out_mass[at] = (p.a.mass ? p.a.mass[at] : 0.f) + sum;
}

size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

}  // namespace

int block_attn_max_group() { return kMaxGroup; }
int block_attn_max_t() { return kMaxT; }

size_t block_attn_ws_bytes(const BlockCache& c, int B, int T, int nq, int64_t n_table, int n_sel,
                           bool sparse, bool mass) {
    (void)n_sel;
    (void)sparse;
    const size_t rows = (size_t)B * T * nq;
    return 16 + (mass ? up16(rows * 4) + up16(rows * 4 * (size_t)(n_table * c.bs / 16)) : 0);
}

cudaError_t block_attn_launch(const BlockCache& c, const BlockBatch& t, const BlockAttnArgs& a,
                              cudaStream_t s) {
    const int64_t rows = (int64_t)t.B * t.T * a.nq;
    if (rows / 4 >= INT32_MAX) return cudaErrorInvalidValue;
    AttnParams p{c, t, a, a.nq / c.nkv, (int)(t.n_table * c.bs / 16), nullptr, nullptr};
    p.row_lse = static_cast<float*>(a.ws);
    p.tile_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + up16((size_t)rows * 4));
    const unsigned grid = (unsigned)((rows + 3) / 4);
    if (c.hd == 64) block_attn_simple_kernel<64><<<grid, 128, 0, s>>>(p);
    else if (c.hd == 128) block_attn_simple_kernel<128><<<grid, 128, 0, s>>>(p);
    else block_attn_simple_kernel<256><<<grid, 128, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.out_mass) return e;
    block_mass_kernel<<<dim3((unsigned)((t.n_table + 127) / 128), (unsigned)t.B), 128, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace mtp

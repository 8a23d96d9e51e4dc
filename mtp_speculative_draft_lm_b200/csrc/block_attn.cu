// Attention over the block-scaled paged cache (mtp_block_attn, mtp_block_sparse_attn).
//
// Mathematics, per query row r (a token's query head) and kv head g, in base 2:
//   s_p = (scale log2(e)) k_scale[block] sum_d q[r, d] e4m3(K[p, d]);  w_p = 2^(s_p - m)
//   out = sum_p w_p v_scale[block] e4m3(V[p]) / sum_p w_p,  lse = (m + log2(sum_p w_p)) ln 2
// with any reference m: a running one, raised only when a score exceeds it by more than 8
// binades (weights stay below 2^8, inside f16), so that most tiles need no maximum, no shuffle
// and no rescaling, just one vote. A block's v_scale is not folded into the weights (they would
// lose f16 bits where scales lie far apart): the accumulators are held in a unit near the v_scales,
// weights are multiplied by v_scale / unit before they are rounded to f16, and the unit moves when
// that leaves [2^2, 2^7]: weights of at most 2^15 fit f16, and a rounding to f16's smallest steps
// takes 2^-27 of the row's largest weight at most (a row's largest is 1 or more before it is
// multiplied), counted in the block's own v_scale. The unit follows the smaller scales, so that
// a block of small values behind one of large values keeps its part: with v_scale / unit down
// to 2^-10 the tail behind a position that has most of the weight was rounded away (67 times the
// error that the test allows). Scales within a factor of 32 of each other move the unit a few
// times at most.
//
// Work: the cache is read in tiles of 16 positions, each inside one block. A unit is a kv head
// of a sequence with up to 8 NT of its T (nq / nkv) query rows (for listed blocks: of a
// token). All units form one line, each as long as its steps and kUnitCost more, and each CTA
// takes an equal stretch of it, however ragged the batch. A unit that lies in one CTA is finished
// there; the others' partial sums go to the workspace and a second kernel joins them in order of
// the CTAs (fixed order: the same bits every time).
//
// Bound by HBM: every code is read once per row tile. Each of a CTA's four warps owns a ring of
// stages: it takes every fourth step (one or two tiles of K and V) of the stretch and issues
// their tensor copies into the stage it has just used, across units, so the warps meet only at
// a unit's end. The blocks and scales of up to 32 tiles ahead are looked up by the warp's lanes
// at once. The two tiles of a step keep two chains of dependent products going. Both
// contractions run on mma.sync m16n8k16 in f16 with fp32 sums: a tile has at most 40 query
// rows, far from where tcgen05's 128-row tiles would pay, and E4M3 decodes to f16 exactly (q is
// scaled per row by a power of two).
// Measured (64 query and 8 kv heads of 128): one sequence of 1,000 positions 7.5 us, of 32,768
// 20 us; 32 of up to 32,768 with block weights 196 us, 5.7 TB/s; listed blocks (24 x 4 tokens, 256
// each) 112 us, 5.9 TB/s. 31 x 5 tokens over up to 8,191 positions of 4 heads of 64 (five row
// tiles) take 54 us, bound by the latency of the decoding, exponentials and products at two
// warps per scheduler.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "block_cache.cuh"
#include "common.cuh"
#include "kernels.h"

namespace mtp {
namespace {

constexpr int kMaxGroup = 16;
constexpr int kMaxT = 64;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxGrid = 640;                  // CTAs (workspace slots are sized for it)
// Steps of the line before each unit's first: what its rows, joins and barriers cost (3 us against
// half a microsecond a step). With none the CTAs that have the short sequences are the last by far.
// us with 0, 8, 12, 16, 32: 31 x 5 tokens of 32 heads of 64 over up to 8,191 positions 75, 53.7,
// 54.0, 54.0, 58.5, over up to 2,000 38.9, 27.0, 26.3, 28.1, 30.7, over up to 400 29, 13.9, 14.4,
// 15.7, 16.4; 64 tokens of 32 heads of 128 over up to 4,096 74, 54.6, 55.1, 55.7, 58.8.
constexpr int kUnitCost = 12;
constexpr float kRaise = 8.f;                  // binades a score may exceed the reference by
constexpr float kLeastLift = 4.f, kMostLift = 128.f;  // v_scale over the accumulators' unit (kRaise and 7 binades: f16)

struct AttnParams {
    BlockCache c;
    BlockBatch t;
    BlockAttnArgs a;
    int grid;            // CTAs of block_attn_kernel
    int group;
    int row_tiles;       // dense: row tiles of 8 NT rows that T tokens have at most
    int64_t tiles;       // 16-position tiles of n_table blocks (tile_lse's pitch)
    int32_t* per;        // [1] steps per CTA
    int32_t* unit_base;  // [units] where each unit starts on the line
    int tile_shift;      // log2(16-position tiles per block)
    uint32_t group_inv;  // ceil(2^20 / group): r / group = r group_inv >> 20 for r <= 1024
    float* parts;        // [2 kMaxGrid][8 NT (hd + 4)] partial sums of a CTA's first and last unit
    float* row_lse;      // [B, nkv, T group] base-2 log-sum-exp (with mass)
    float* tile_lse;     // [B, nkv, tiles, T group] of each tile's positions (with mass)
};

// A sequence's units, outer * inner of them (dense: kv heads, each with its row tiles, the later
// ones of which find their codes in L2; listed blocks: tokens, each with its kv heads), and the
// tiles and steps of `P` tiles that each has.
struct SeqWork {
    int len, q, outer, inner, tiles, steps;
    __device__ __forceinline__ int line() const { return steps ? outer * inner * (steps + kUnitCost) : 0; }
};
template <int NT, bool SPARSE, int P>
__device__ __forceinline__ SeqWork seq_work(const AttnParams& p, int b) {
    const SeqStep s = seq_step(p.t, b);
    SeqWork w;
    w.len = s.len;
    w.q = s.q;
    if (SPARSE) {
        w.outer = s.q;
        w.inner = p.c.nkv;
        w.tiles = s.len > 0 ? p.a.n_sel << p.tile_shift : 0;
    } else {
        w.outer = p.c.nkv;
        w.inner = (s.q * p.group + 8 * NT - 1) / (8 * NT);
        w.tiles = (int)min((int64_t)(s.len >> 4) + ((s.len & 15) != 0), p.tiles);
    }
    w.steps = (w.tiles + P - 1) / P;
    return w;
}

// What each of `grid` CTAs takes of a line of this length.
__device__ __forceinline__ int stretch_of(int total, int grid) {
    return (total / grid + (total % grid != 0) + kWarps - 1) / kWarps * kWarps;
}

// The unit's index in unit_base: unit u of sequence b.
template <bool SPARSE>
__device__ __forceinline__ int64_t unit_index(const AttnParams& p, int b, int g, int part) {
    return SPARSE ? ((int64_t)b * p.t.T + part) * p.c.nkv + g : ((int64_t)b * p.c.nkv + g) * p.row_tiles + part;
}

template <int HD, int NT>
struct Shape {
    static constexpr int kTile = 16 * HD;                        // bytes of K (or V) of a tile
    static constexpr int P = HD == 256 ? 1 : 2;                  // tiles per step
    // of them worked on together, and CTAs per SM: as the accumulators leave registers. (Three of
    // 64-wide heads spill 40 bytes at two row tiles and 32 at three, and gain all the same: 32 x 1
    // token over up to 32,768 positions at 16 rows 70 us, 82 with two CTAs, 32 x 3 at 24 rows 83 and
    // 98. The 32 rows of 128-wide heads spill 224 bytes.)
    static constexpr int kJoint = HD < 256 && NT <= 2 ? P : 1;
    static constexpr int kPerSm = HD == 64 ? (NT <= 3 ? 3 : 2) : HD == 128 ? (NT <= 1 ? 3 : 2) : 2;
    static constexpr int kQPitch = HD + 8;                       // f16 elements
    static constexpr int kRows = 8 * NT;
    static constexpr size_t kFixed = (size_t)HD * NT * 64           // two warps' accumulators
                                     + (size_t)kRows * kQPitch * 2  // q
                                     + (size_t)kRows * 8            // score factors, limits
                                     + (size_t)2 * kWarps * kRows * 4 + 16;
    static constexpr size_t kStage = (size_t)kWarps * (P * (2 * kTile + 16) + 8);  // tiles, info, barrier
    // (1 KB of each CTA's share of the SM's 228 KB is the system's)
    static constexpr int kStages = (int)(((size_t)(228 * 1024) / kPerSm - 1024 - kFixed) / kStage);
    static constexpr size_t kSmem = kStages * kStage + kFixed;
    static_assert(kStages >= 2, "two stages at least");
};

constexpr int kNowhere = 1 << 30;  // a position behind every limit (limits are clamped to it)

struct TileInfo {
    int pos0;  // first position, or kNowhere: nothing was read
    float ks, vs;
    int pad;
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float lg2(float x) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
// Transpose of an 8 x 8 matrix of 16-bit values in the mma fragment layout.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ void copy4_async(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// Arrive on `bar` (one of its expected arrivals) when this thread's earlier cp.async are done.
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// mma_f16_16816 onto zeros.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void load_tile(void* dst, const CUtensorMap* map, int x, int row, int head, int block,
                                          uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(row), "r"(head), "r"(block), "r"(smem_u32(bar))
        : "memory");
}

// How a warp reads a stage's tile (rows of 128 bytes whose 16-byte chunks are swizzled by
// chunk ^ (row & 7); hd = 64: rows of 64 bytes, chunk ^ ((row / 2) & 3); hd = 256: two halves
// of 128 columns). Lane 4 gid + tig reads 16 bytes at a time, without bank conflicts because
// the tile's positions and columns are permuted, which no sum notices: MMA row m is position
// pos_of(m), and lane column group gid holds the columns col_of(gid) on.
template <int HD>
__device__ __forceinline__ constexpr int pos_of(int m) {  // m < 8; rows 8 .. 15: 8 more
    return HD == 64 ? m ^ ((m >> 1) & 1) : (m & 1) * 4 + (m >> 1);
}
template <int HD>
__device__ __forceinline__ constexpr int col_of(int gid) {
    return HD == 64 ? 8 * gid : 16 * ((gid >> 1) + 4 * (gid & 1));
}
template <int HD>
__device__ __forceinline__ uint32_t swizzled(int row, int byte) {  // row < 16, byte < min(HD, 128)
    return HD == 64 ? row * 64 + (byte ^ (((row >> 1) & 3) << 4)) : row * 128 + (byte ^ ((row & 7) << 4));
}
// Offset of what lane column group gid reads of MMA row m of V (its first half of 256 columns).
template <int HD>
__device__ __forceinline__ uint32_t v_offset(int m, int gid) {
    return HD == 64 ? swizzled<HD>(pos_of<HD>(m), col_of<HD>(gid) & ~15) + (col_of<HD>(gid) & 15)
                    : swizzled<HD>(pos_of<HD>(m), col_of<HD>(gid));
}
__device__ __forceinline__ uint4 lds4(uint32_t a) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
    return r;
}
__device__ __forceinline__ uint2 lds2(uint32_t a) {
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
    return r;
}

// The slow part of a wait, kept out of the tile loop's code.
__device__ __noinline__ void wait_long(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* dev_err) {
    if (!mbar_wait_bounded(bar, parity, abort)) raise_flag(dev_err, DEVFLAG_TIMEOUT);
}

template <int HD, int NT, bool SPARSE>
__global__ void __launch_bounds__(kThreads, Shape<HD, NT>::kPerSm)
    block_attn_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap) {
    using S = Shape<HD, NT>;
    constexpr int ST = S::kStages, P = S::P, HJ = S::kJoint, KC = HD / 16, DT = HD / 16, R = S::kRows, QP = S::kQPitch;
    constexpr uint32_t kStageBytes = P * 2 * S::kTile;                                    // of one warp
    extern __shared__ __align__(1024) uint8_t ring[];                                     // [warp][stage][tile][K, V][16 rows]
    float4* xacc = reinterpret_cast<float4*>(ring + (size_t)kWarps * ST * kStageBytes);   // [2][DT NT][32]
    TileInfo* info = reinterpret_cast<TileInfo*>(xacc + 2 * DT * NT * 32);                // [warp][stage][tile]
    uint64_t* full = reinterpret_cast<uint64_t*>(info + kWarps * ST * P);                 // [warp][stage]
    uint16_t* qh = reinterpret_cast<uint16_t*>(full + kWarps * ST);                       // [R][QP] f16
    float* hfac = reinterpret_cast<float*>(qh + R * QP);                                  // [R]
    int* lims = reinterpret_cast<int*>(hfac + R);                                         // [R]
    float* redm = reinterpret_cast<float*>(lims + R);                                     // [warp][R]
    float* redl = redm + kWarps * R;
    volatile int* abort = reinterpret_cast<volatile int*>(redl + kWarps * R);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t ring_at = smem_u32(ring);
    if (ring_at & 1023u) {  // (the swizzled copies need it; dynamic shared memory starts there)
        if (tid == 0) raise_flag(p.t.dev_err, DEVFLAG_TIMEOUT);
        return;
    }
    // arrivals: lane 0 with the tiles' bytes, and one per tile for its scales
    if (tid < kWarps * ST) mbar_init(&full[tid], 1 + P);
    if (tid == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&vmap) : "memory");
    }
    if (tid == 0) *abort = 0;
    mbar_fence_init();
    __syncthreads();
    pdl_wait();  // everything below reads or writes memory that earlier kernels may still use
    pdl_launch_dependents();  // (the next kernel may read what was there before this one)

    // this CTA's stretch of the line: `stretch` from `beg` on, and the sequence and unit it
    // starts with (every warp for itself, 32 sequences at a time)
    const int B = p.t.B;
    SeqWork w0 = seq_work<NT, SPARSE, P>(p, min(lane, B - 1));
    int n0 = lane < B ? w0.line() : 0, total = n0;
    for (int b = 32 + lane; b < B; b += 32) {
        total += seq_work<NT, SPARSE, P>(p, b).line();
    }
    total = __reduce_add_sync(0xffffffffu, total);
    const int per = stretch_of(total, p.grid);
    if (blockIdx.x == 0 && tid == 0) *p.per = per;
    if ((int64_t)blockIdx.x * per >= total) return;
    const int beg = (int)blockIdx.x * per;
    const int stretch = min(total - beg, per);

    // A place on the line: a unit, where in it the stretch enters, and the steps [t0, t1) of it
    // that belong to this CTA.
    struct Place {
        SeqWork sw;
        int b, outer, inner, off, t0, t1;
        int left;  // of the stretch, from there on
    };
    Place pl;
    for (int b0 = 0, before = 0;; b0 += 32) {
        if (b0) {
            w0 = seq_work<NT, SPARSE, P>(p, min(b0 + lane, B - 1));
            n0 = b0 + lane < B ? w0.line() : 0;
        }
        int inc = n0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, before + inc > beg);
        if (past) {  // (some chunk has it: beg < total)
            const int src = __ffs(past) - 1;
            const int off = beg - (before + __shfl_sync(0xffffffffu, inc - n0, src));
            pl.sw.len = __shfl_sync(0xffffffffu, w0.len, src);
            pl.sw.q = __shfl_sync(0xffffffffu, w0.q, src);
            pl.sw.outer = __shfl_sync(0xffffffffu, w0.outer, src);
            pl.sw.inner = __shfl_sync(0xffffffffu, w0.inner, src);
            pl.sw.tiles = __shfl_sync(0xffffffffu, w0.tiles, src);
            pl.sw.steps = __shfl_sync(0xffffffffu, w0.steps, src);
            pl.b = b0 + src;
            const int u = off / (pl.sw.steps + kUnitCost);
            pl.off = off - u * (pl.sw.steps + kUnitCost);
            pl.outer = u / pl.sw.inner;
            pl.inner = u - pl.outer * pl.sw.inner;
            break;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
    }
    auto settle = [&](Place& c) {
        c.t0 = max(c.off - kUnitCost, 0);
        c.t1 = min(max(c.off + c.left - kUnitCost, 0), c.sw.steps);
    };
    auto next_unit = [&](Place& c) -> bool {  // the next one with a step; false at the stretch's end
        do {
            c.left -= c.sw.steps + kUnitCost - c.off;
            if (c.left <= 0) return false;
            c.off = 0;
            if (++c.inner == c.sw.inner) {
                c.inner = 0;
                if (++c.outer == c.sw.outer) {
                    c.outer = 0;
                    do c.sw = seq_work<NT, SPARSE, P>(p, ++c.b);
                    while (c.sw.line() == 0 && c.b + 1 < B);
                }
            }
            settle(c);
        } while (c.t0 == c.t1);
        return true;
    };
    pl.left = stretch;
    settle(pl);
    if (pl.t0 == pl.t1 && !next_unit(pl)) return;

    // The copies' side of this warp, ST steps ahead. Lane l looks up tile l % P of the warp's
    // step l / P from ah_step on; ah_n counts the steps of those that have been issued.
    Place ah = pl;
    int ah_step = ah.t0 + warp, ah_n = 0, ah_cnt = 0, ah_blk = -1, ah_pos = kNowhere;
    uint32_t ah_read = 0;
    bool ah_more = true;
    int ist = 0;  // the stage the next copies go to
    auto look_up = [&]() {
        while (ah_step >= ah.t1) {  // past its unit: on to the next ones
            if (!next_unit(ah)) {
                ah_more = false;
                return;
            }
            ah_step = ah.t0 + warp;
        }
        ah_n = 0;
        ah_cnt = min(32 / P, (ah.t1 - ah_step + kWarps - 1) / kWarps);
        const int tile = (ah_step + lane / P * kWarps) * P + lane % P;
        const bool mine = lane / P < ah_cnt && tile < ah.sw.tiles;
        const int g = SPARSE ? ah.inner : ah.outer;
        int lb = tile >> p.tile_shift, lim = ah.sw.len;
        if (SPARSE) {
            lim += ah.outer + 1 - ah.sw.q;
            lb = mine ? __ldg(p.a.sel + (((int64_t)ah.b * p.t.T + ah.outer) * p.c.nkv + g) * p.a.n_sel + lb) : -1;
        }
        const int64_t pos = ((int64_t)lb << (4 + p.tile_shift)) + 16 * (tile & ((1 << p.tile_shift) - 1));
        const bool seen = mine && lb >= 0 && pos < lim;
        ah_blk = seen ? table_block(p.t, p.c.num_blocks, ah.b, lb) : -1;
        if (seen && ah_blk < 0) raise_flag(p.t.dev_err, DEVFLAG_BAD_SLOT);
        ah_pos = ah_blk >= 0 ? (int)pos : kNowhere;
        ah_read = __ballot_sync(0xffffffffu, ah_blk >= 0);
    };
    auto issue = [&]() {
        if (!ah_more) return;
        if (*abort) {  // a wait ran out: no more copies
            ah_more = false;
            return;
        }
        const int at = warp * ST + ist;
        if (lane == 0) mbar_arrive_expect_tx(&full[at], (uint32_t)__popc((ah_read >> (ah_n * P)) & ((1u << P) - 1u)) * 2u * S::kTile);
        __syncwarp();
        if (lane / P == ah_n) {
            TileInfo* ti = &info[at * P + lane % P];
            ti->pos0 = ah_pos;
            if (ah_blk >= 0) {
                uint8_t* kd = ring + (size_t)at * kStageBytes + (lane % P) * 2 * S::kTile;
                const int row = ah_pos & ((16 << p.tile_shift) - 1);
                const int g = SPARSE ? ah.inner : ah.outer;
#pragma unroll
                for (int x = 0; x < HD; x += 128) {
                    load_tile(kd + x * 16, &kmap, x, row, g, ah_blk, &full[at]);
                    load_tile(kd + S::kTile + x * 16, &vmap, x, row, g, ah_blk, &full[at]);
                }
                const int64_t sc = (int64_t)ah_blk * p.c.nkv + g;
                copy4_async(&ti->ks, p.c.k_scale + sc);
                copy4_async(&ti->vs, p.c.v_scale + sc);
                copies_arrive(&full[at]);
            } else {
                ti->ks = ti->vs = 0.f;
                mbar_arrive(&full[at]);
            }
        }
        if (++ist == ST) ist = 0;
        if (++ah_n == ah_cnt) {
            ah_step += ah_cnt * kWarps;
            look_up();
        }
    };
    // The query rows of a unit, 16 bytes per lane and row: the first unit's are asked for before
    // its tiles, which keep the memory busy for microseconds.
    constexpr int LH = HD / 8, HPL = 32 / LH, NQ = (R + kWarps * HPL - 1) / (kWarps * HPL);  // lanes per row, rows per warp
    uint4 qv[NQ];
    auto load_q = [&]() {
        const int row0 = SPARSE ? pl.outer * p.group : pl.inner * R, g = SPARSE ? pl.inner : pl.outer;
        const int nrows = SPARSE ? p.group : min(R, pl.sw.q * p.group - row0);
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const int r = (n * kWarps + warp) * HPL + lane / LH;
            const int tok = (int)(((uint32_t)(row0 + r) * p.group_inv) >> 20), i = (row0 + r) - tok * p.group;
            qv[n] = make_uint4(0, 0, 0, 0);
            if (r < nrows)
                qv[n] = *reinterpret_cast<const uint4*>(p.a.q + ((int64_t)pl.b * p.t.T + tok) * p.a.q_stride +
                                                        ((int64_t)g * p.group + i) * HD + 8 * (lane % LH));
        }
    };
    load_q();
    look_up();
#pragma unroll 1
    for (int i = 0; i < ST; ++i) issue();

    const int gid = lane >> 2, tig = lane & 3;
    constexpr int kPitch = HD == 64 ? 64 : 128, kWords = HD == 64 ? 2 : 4;  // of a (half) tile; words a lane holds of a V row
    const uint32_t koff = swizzled<HD>(pos_of<HD>(gid), 16 * tig);
    const uint32_t voff0 = v_offset<HD>(2 * tig, gid), voff1 = v_offset<HD>(2 * tig + 1, gid);
    int st = 0;
    uint32_t ph = 0;
    bool first = true;  // this CTA's first unit
    do {
        const SeqWork& sw = pl.sw;
        const int b = pl.b, g = SPARSE ? pl.inner : pl.outer, part = SPARSE ? pl.outer : pl.inner, t0 = pl.t0, t1 = pl.t1;
        // rows of this unit: row r is token tok, head i of the group, row0 + r = tok group + i
        const int row0 = SPARSE ? part * p.group : part * R;
        const int nrows = SPARSE ? p.group : min(R, sw.q * p.group - row0);
        auto token_of = [&](int r) { return (int)(((uint32_t)(row0 + r) * p.group_inv) >> 20); };
        const int lim0 = min(sw.len - sw.q + token_of(0) + 1, kNowhere);  // the fewest positions a row sees
        const int vlim = SPARSE ? lim0 : sw.len;                          // rows from here on hold nothing
        const int mass_pitch = (int)p.t.T * p.group;                      // rows of a kv head
        float* mass_at = nullptr;
        if (!SPARSE && p.a.out_mass) mass_at = p.tile_lse + ((int64_t)b * p.c.nkv + g) * p.tiles * mass_pitch + row0;
        if (tid == 0) {
            if (!SPARSE && t1 == sw.steps && (sw.len - 1) / p.c.bs >= p.t.n_table)
                raise_flag(p.t.dev_err, DEVFLAG_BAD_SLOT);  // positions past the table
            if (t0 == 0) p.unit_base[unit_index<SPARSE>(p, b, g, part)] = beg + (stretch - pl.left) - pl.off;
        }

        __syncthreads();  // the previous unit's rows and sums are no longer needed
        {
            // q rows in f16, each scaled by 2^e so that its largest |q| lies in [2^14, 2^15)
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                const int r = (n * kWarps + warp) * HPL + lane / LH;
                const bool has = r < nrows;
                const int tok = token_of(r);
                const uint4 v = qv[n];
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                float mx = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(w[k])), fabsf(bf16_hi(w[k]))));
#pragma unroll
                for (int o = LH / 2; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                // e within [-113, 126], so that 2^e and 2^-e are normal (an all but zero row keeps
                // a smaller largest value)
                const bool fin = mx < INFINITY;
                const int e = fin ? min(141 - (int)(__float_as_uint(mx) >> 23), 126) : 0;
                const float up = __uint_as_float((uint32_t)(127 + e) << 23), down = __uint_as_float((uint32_t)(127 - e) << 23);
                uint32_t o4[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) o4[k] = pack_f16x2(bf16_lo(w[k]) * up, bf16_hi(w[k]) * up);
                if (r < R) *reinterpret_cast<uint4*>(qh + r * QP + 8 * (lane % LH)) = make_uint4(o4[0], o4[1], o4[2], o4[3]);
                if (r < R && lane % LH == 0) {
                    hfac[r] = !has ? 0.f : fin ? p.a.scale * kLog2e * down : __uint_as_float(0x7fc00000u);
                    lims[r] = has ? min(sw.len - sw.q + tok + 1, kNowhere) : kNowhere;
                }
            }
        }
        __syncthreads();
        // B fragments of the scores: k-step 4 h + s of the matrix product is, in lane tig, dims
        // 64 h + 16 tig + 4 s .. + 3 (as the K bytes of a 16-byte load come)
        uint4 qf[NT == 1 ? KC / 2 : 1];
        if (NT == 1)
#pragma unroll
            for (int c = 0; c < KC / 2; ++c)
                qf[c] = *reinterpret_cast<const uint4*>(qh + gid * QP + 64 * (c >> 1) + 16 * tig + 8 * (c & 1));
        float2 hf[NT <= 2 ? NT : 1], nm[NT], l[NT];  // rows 8 j + 2 tig, + 1: score factor, minus reference, sum
        uint32_t fresh = (1u << (2 * NT)) - 1u;  // rows without a reference yet (nm 0): bits 2 j, 2 j + 1
        float acc[DT][NT][4];
        float vcur = 0.f, vinv = 0.f, vmax = 0.f;  // the accumulators' unit, 1 over it, the largest v_scale so far
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if (NT <= 2) hf[j] = *reinterpret_cast<const float2*>(hfac + 8 * j + 2 * tig);
            nm[j] = make_float2(0.f, 0.f);
            l[j] = make_float2(0.f, 0.f);
#pragma unroll
            for (int dt = 0; dt < DT; ++dt)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[dt][j][k] = 0.f;
        }

#pragma unroll 1
        for (int step = t0 + warp; step < t1; step += kWarps) {
            const int at = warp * ST + st;
            if (!mbar_try_wait(&full[at], ph)) wait_long(&full[at], ph, abort, p.t.dev_err);
#pragma unroll
            for (int h0 = 0; h0 < P; h0 += HJ) {
                int pos0[HJ];
                float ks[HJ], vs[HJ], x[HJ][NT][4];
                bool masked = false;  // a limit per row matters
#pragma unroll
                for (int z = 0; z < HJ; ++z) {
                    const TileInfo ti = info[at * P + h0 + z];
                    pos0[z] = ti.pos0;
                    ks[z] = ti.ks;
                    vs[z] = ti.vs;
                    masked = masked || ti.pos0 + 16 > lim0;
                }
                const uint32_t stage = ring_at + (uint32_t)at * kStageBytes + h0 * 2 * S::kTile;
                // scores of 16 positions (rows) and the unit's query rows (columns)
#pragma unroll
                for (int h = 0; h < HD / 64; ++h) {  // 64 dims at a time
                    uint32_t w0[HJ][4], w1[HJ][4];
#pragma unroll
                    for (int z = 0; z < HJ; ++z) {
                        const uint32_t ka = (stage + z * 2 * S::kTile + (h >> 1) * 2048 + koff) ^ ((h & 1) << 6);
                        const uint4 k0 = lds4(ka), k1 = lds4(ka + 8 * kPitch);
                        w0[z][0] = k0.x, w0[z][1] = k0.y, w0[z][2] = k0.z, w0[z][3] = k0.w;
                        w1[z][0] = k1.x, w1[z][1] = k1.y, w1[z][2] = k1.z, w1[z][3] = k1.w;
                    }
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        uint32_t a[HJ][2][4];
#pragma unroll
                        for (int z = 0; z < HJ; ++z)
#pragma unroll
                            for (int v = 0; v < 2; ++v) {
                                a[z][v][0] = e4m3x2_to_f16x2((uint16_t)(w0[z][2 * t + v] & 0xFFFFu));
                                a[z][v][1] = e4m3x2_to_f16x2((uint16_t)(w1[z][2 * t + v] & 0xFFFFu));
                                a[z][v][2] = e4m3x2_to_f16x2((uint16_t)(w0[z][2 * t + v] >> 16));
                                a[z][v][3] = e4m3x2_to_f16x2((uint16_t)(w1[z][2 * t + v] >> 16));
                            }
                        uint4 q4[NT];
#pragma unroll
                        for (int j = 0; j < NT; ++j)
                            q4[j] = NT == 1 ? qf[2 * h + t] : *reinterpret_cast<const uint4*>(qh + (8 * j + gid) * QP + 64 * h + 16 * tig + 8 * t);
                        // (products onto one sum as far apart as they can be)
#pragma unroll
                        for (int v = 0; v < 2; ++v)
#pragma unroll
                            for (int z = 0; z < HJ; ++z)
#pragma unroll
                                for (int j = 0; j < NT; ++j) {
                                    if (h == 0 && t == 0 && v == 0) mma_f16_first(x[z][j], a[z][v][0], a[z][v][1], a[z][v][2], a[z][v][3], q4[j].x, q4[j].y);
                                    else mma_f16_16816(x[z][j], a[z][v][0], a[z][v][1], a[z][v][2], a[z][v][3], v ? q4[j].z : q4[j].x, v ? q4[j].w : q4[j].y);
                                }
                    }
                }
                // s - m, (row 2 tig, row 2 tig + 1) of positions gid and gid + 8; masked ones -inf
#pragma unroll
                for (int z = 0; z < HJ; ++z)
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const float2 hfj = NT <= 2 ? hf[NT <= 2 ? j : 0] : *reinterpret_cast<const float2*>(hfac + 8 * j + 2 * tig);
                        const float2 f = mul2(hfj, make_float2(ks[z], ks[z]));
                        const float2 x0 = fma2(make_float2(x[z][j][0], x[z][j][1]), f, nm[j]);
                        const float2 x1 = fma2(make_float2(x[z][j][2], x[z][j][3]), f, nm[j]);
                        x[z][j][0] = x0.x, x[z][j][1] = x0.y, x[z][j][2] = x1.x, x[z][j][3] = x1.y;
                    }
                if (masked)
#pragma unroll
                    for (int z = 0; z < HJ; ++z)
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int lim = lims[8 * j + 2 * tig + e];
                                if (pos0[z] + pos_of<HD>(gid) >= lim) x[z][j][e] = -INFINITY;
                                if (pos0[z] + pos_of<HD>(gid) + 8 >= lim) x[z][j][2 + e] = -INFINITY;
                            }
                float top = -INFINITY;
#pragma unroll
                for (int z = 0; z < HJ; ++z)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        top = fmaxf(top, fmaxf(fmaxf(x[z][j][0], x[z][j][1]), fmaxf(x[z][j][2], x[z][j][3])));
                if (__any_sync(0xffffffffu, top > kRaise || fresh)) {
                    // the references move by d: up to the largest score, or to a row's first one
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        float d[2], al[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float m = -INFINITY;
#pragma unroll
                            for (int z = 0; z < HJ; ++z) m = fmaxf(m, fmaxf(x[z][j][e], x[z][j][2 + e]));
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                            const bool isnew = (fresh >> (2 * j + e)) & 1u;
                            d[e] = isnew ? (m == -INFINITY ? 0.f : m) : fmaxf(m, 0.f);
                            al[e] = isnew ? 0.f : ex2(-d[e]);
                            if (isnew && m != -INFINITY) fresh &= ~(1u << (2 * j + e));
#pragma unroll
                            for (int z = 0; z < HJ; ++z) {
                                x[z][j][e] -= d[e];
                                x[z][j][2 + e] -= d[e];
                            }
#pragma unroll
                            for (int dt = 0; dt < DT; ++dt) {
                                acc[dt][j][e] *= al[e];
                                acc[dt][j][2 + e] *= al[e];
                            }
                        }
                        nm[j] = make_float2(nm[j].x - d[0], nm[j].y - d[1]);
                        l[j] = mul2(l[j], make_float2(al[0], al[1]));
                    }
                }
#pragma unroll
                for (int z = 0; z < HJ; ++z) {
                    // the block's v_scale over the accumulators' unit
                    float wmul = vs[z] * vinv;
                    if (!(wmul >= kLeastLift && wmul <= kMostLift) && pos0[z] != kNowhere) {
                        // a new unit: as far below the block's v_scale as the side it left by asks for, but
                        // a normal number, and never more than 2^92 below the largest v_scale so far (the
                        // sums would overflow); a zero scale weighs nothing
                        if (vs[z] == 0.f) {
                            wmul = 0.f;
                        } else {
                            vmax = fmaxf(vmax, vs[z]);
                            const float unit = fmaxf(fmaxf(vs[z] * (wmul > kMostLift ? 1.f / kMostLift : 1.f / kLeastLift), vmax * 2.0194839173657902e-28f),
                                                     1.17549435e-38f);
                            wmul = vs[z] / unit;
                            const float ratio = vcur / unit;
                            vcur = unit;
                            vinv = 1.f / unit;
#pragma unroll
                            for (int dt = 0; dt < DT; ++dt)
#pragma unroll
                                for (int j = 0; j < NT; ++j)
#pragma unroll
                                    for (int k = 0; k < 4; ++k) acc[dt][j][k] *= ratio;
                        }
                    }
                    vmax = fmaxf(vmax, vs[z]);
                    // weights: summed in fp32, rounded to f16 for the product and transposed into
                    // its B fragments (rows to columns)
                    uint32_t bp[NT][2];
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const float2 w0 = make_float2(ex2(x[z][j][0]), ex2(x[z][j][1])), w1 = make_float2(ex2(x[z][j][2]), ex2(x[z][j][3]));
                        const float2 ws = add2(w0, w1);
                        x[z][j][0] = ws.x, x[z][j][1] = ws.y;
                        l[j] = add2(l[j], ws);
                        const float2 wm = make_float2(wmul, wmul), u0 = mul2(w0, wm), u1 = mul2(w1, wm);
                        bp[j][0] = transpose8(pack_f16x2(u0.x, u0.y));
                        bp[j][1] = transpose8(pack_f16x2(u1.x, u1.y));
                    }
                    const int tile = step * P + h0 + z;
                    if (!SPARSE && p.a.out_mass && (P == 1 || tile < sw.tiles)) {
                        // the tile's sum of weights per row: 2 NT values (padded to VP) summed over
                        // the 8 lanes of a column; each step halves what a lane carries
                        constexpr int VP = NT <= 1 ? 2 : NT <= 2 ? 4 : NT <= 4 ? 8 : 16;
                        float v[VP], m[VP];
#pragma unroll
                        for (int k = 0; k < VP; ++k) {
                            v[k] = k < 2 * NT ? x[z][k >> 1][k & 1] : 0.f;
                            m[k] = k >= 2 * NT ? 0.f : k & 1 ? nm[k >> 1].y : nm[k >> 1].x;
                        }
                        int k0 = 0;  // the value in v[0]
#pragma unroll
                        for (int o = 16, n = VP; o >= 4; o >>= 1) {
                            const bool hi = lane & o;
                            n >>= 1;
                            if (n) {
                                if (hi) k0 += n;
#pragma unroll
                                for (int k = 0; k < n; ++k) {
                                    const float give = hi ? v[k] : v[k + n];
                                    v[k] = (hi ? v[k + n] : v[k]) + __shfl_xor_sync(0xffffffffu, give, o);
                                    m[k] = hi ? m[k + n] : m[k];
                                }
                            } else {
                                v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
                            }
                        }
#pragma unroll
                        for (int k = 0; k < (VP > 8 ? VP / 8 : 1); ++k) {
                            const int r = 8 * ((k0 + k) >> 1) + 2 * tig + ((k0 + k) & 1);
                            if (r < nrows)  // (several lanes may hold the same value)
                                mass_at[(int64_t)tile * mass_pitch + r] = v[k] > 0.f ? lg2(v[k]) - m[k] : v[k] != v[k] ? v[k] : -INFINITY;
                        }
                    }
                    if (pos0[z] == kNowhere) continue;  // nothing was read (the stage holds other bytes)
                    // V^T (A) . W^T (B) over 16 positions: a lane holds kWords words of columns from
                    // col_of(gid) on of four positions; tile dt has column 2 dt of them in row gid,
                    // 2 dt + 1 in row gid + 8
#pragma unroll
                    for (int h = 0; h < (HD + 127) / 128; ++h) {
                        uint32_t y[4][kWords];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t va = stage + z * 2 * S::kTile + S::kTile + h * 2048 + (k & 1 ? voff1 : voff0) + (k >> 1) * 8 * kPitch;
                            if constexpr (HD == 64) {
                                const uint2 v = lds2(va);
                                y[k][0] = v.x, y[k][1] = v.y;
                            } else {
                                const uint4 v = lds4(va);
                                y[k][0] = v.x, y[k][1] = v.y, y[k][2] = v.z, y[k][3] = v.w;
                            }
                        }
                        // In a masked tile rows past the end are zeroed (0 * NaN is NaN), and NaN
                        // codes are taken out and given back to the rows that see them: the first
                        // position that has one, per column
                        bool nan_any = false;
                        if (masked) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
#pragma unroll
                                for (int w = 0; w < kWords; ++w) {
                                    if (pos0[z] + pos_of<HD>(2 * tig + (k & 1)) + 8 * (k >> 1) >= vlim) y[k][w] = 0;
                                    nan_any = nan_any || __vcmpeq4(y[k][w] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                                }
                            nan_any = __any_sync(0xffffffffu, nan_any);
                            if (nan_any) {
#pragma unroll
                                for (int w = 0; w < kWords; ++w) {
                                    uint32_t isn[4];
#pragma unroll
                                    for (int k = 0; k < 4; ++k) {
                                        isn[k] = __vcmpeq4(y[k][w] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                                        y[k][w] &= ~isn[k];
                                    }
#pragma unroll
                                    for (int d = 0; d < 4; ++d) {
                                        int first_at = 0x7fffffff;
#pragma unroll
                                        for (int k = 0; k < 4; ++k)
                                            if ((isn[k] >> (8 * d)) & 1u)
                                                first_at = min(first_at, pos0[z] + pos_of<HD>(2 * tig + (k & 1)) + 8 * (k >> 1));
                                        first_at = min(first_at, __shfl_xor_sync(0xffffffffu, first_at, 1));
                                        first_at = min(first_at, __shfl_xor_sync(0xffffffffu, first_at, 2));
#pragma unroll
                                        for (int j = 0; j < NT; ++j)
#pragma unroll
                                            for (int e = 0; e < 2; ++e)
                                                if (first_at < lims[8 * j + 2 * tig + e])
                                                    acc[8 * h + 2 * w + d / 2][j][2 * (d & 1) + e] = __uint_as_float(0x7fc00000u);
                                    }
                                }
                            }
                        }
#pragma unroll
                        for (int w = 0; w < kWords; ++w)
#pragma unroll
                            for (int u2 = 0; u2 < 2; ++u2) {
                                const uint32_t lo = __byte_perm(y[0][w], y[1][w], u2 ? 0x7362 : 0x5140);
                                const uint32_t hi = __byte_perm(y[2][w], y[3][w], u2 ? 0x7362 : 0x5140);
                                const uint32_t a0 = e4m3x2_to_f16x2((uint16_t)(lo & 0xFFFFu)), a1 = e4m3x2_to_f16x2((uint16_t)(lo >> 16));
                                const uint32_t a2 = e4m3x2_to_f16x2((uint16_t)(hi & 0xFFFFu)), a3 = e4m3x2_to_f16x2((uint16_t)(hi >> 16));
#pragma unroll
                                for (int j = 0; j < NT; ++j) mma_f16_16816(acc[8 * h + 2 * w + u2][j], a0, a1, a2, a3, bp[j][0], bp[j][1]);
                            }
                    }
                }
            }
            __syncwarp();  // everyone is done with the stage
            issue();
            if (++st == ST) {
                st = 0;
                ph ^= 1;
            }
        }

        const bool whole = t0 == 0 && t1 == sw.steps;
        const bool more = next_unit(pl);  // (sw is the next unit's from here on)
        if (more) load_q();               // (its rows arrive while this unit is joined)

        // join the four warps (fixed order): the largest reference M, everything times 2^(m - M)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                l[j].x += __shfl_xor_sync(0xffffffffu, l[j].x, o);
                l[j].y += __shfl_xor_sync(0xffffffffu, l[j].y, o);
            }
            if (gid == 0) {
                const int r = warp * R + 8 * j + 2 * tig;
                *reinterpret_cast<float2*>(redm + r) = make_float2((fresh >> (2 * j)) & 1u ? -INFINITY : -nm[j].x,
                                                                  (fresh >> (2 * j + 1)) & 1u ? -INFINITY : -nm[j].y);
                *reinterpret_cast<float2*>(redl + r) = l[j];
            }
        }
        __syncthreads();
        float* slot = p.parts + ((int64_t)blockIdx.x * 2 + (first ? 0 : 1)) * (R * (HD + 4));
        if (tid < R) {  // a thread per row: the warps' factors, the sum, and what does not need the accumulators
            const int r = tid, tok = token_of(r), i = (row0 + r) - tok * p.group;
            const int row = (b * (int)p.t.T + tok) * p.a.nq + g * p.group + i;
            float m[kWarps], M = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, m[w] = redm[w * R + r]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = m[w] == -INFINITY ? 0.f : ex2(m[w] - M);
                L += f * redl[w * R + r];
                redm[w * R + r] = f;
            }
            const bool some = !(L <= 0.f);
            redl[r] = whole ? (some ? 1.f / L : 0.f) : 1.f;
            redl[R + r] = __int_as_float(row);
            if (r < nrows) {
                if (whole) {
                    const float lse2 = some ? M + log2f(L) : -INFINITY;
                    if (p.a.out_lse) p.a.out_lse[row] = lse2 * kLn2;
                    if (!SPARSE && p.a.out_mass) p.row_lse[((int64_t)b * p.c.nkv + g) * mass_pitch + row0 + r] = lse2;
                } else {
                    slot[r] = M;
                    slot[R + r] = L;
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const float2 f = *reinterpret_cast<const float2*>(redm + warp * R + 8 * j + 2 * tig);
            const float f0 = f.x * vcur, f1 = f.y * vcur;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) {
                acc[dt][j][0] *= f0;
                acc[dt][j][1] *= f1;
                acc[dt][j][2] *= f0;
                acc[dt][j][3] *= f1;
            }
        }
        // each warp ends with a quarter of the columns: first halves are swapped between warps w and
        // w ^ 2, then quarters between w and w ^ 1 (through the half that w has just read)
        constexpr int H = DT / 2, Q = DT / 4;
        float4* mine = xacc + (size_t)warp * H * NT * 32;
        float4* other = xacc + (size_t)(warp ^ 2) * H * NT * 32;
        float red[H][NT][4], fin[Q][NT][4];
#pragma unroll
        for (int dt = 0; dt < H; ++dt)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float give[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    give[k] = warp & 2 ? acc[dt][j][k] : acc[H + dt][j][k];
                    red[dt][j][k] = warp & 2 ? acc[H + dt][j][k] : acc[dt][j][k];
                }
                mine[(dt * NT + j) * 32 + lane] = make_float4(give[0], give[1], give[2], give[3]);
            }
        __syncthreads();
#pragma unroll
        for (int dt = 0; dt < H; ++dt)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const float4 v = other[(dt * NT + j) * 32 + lane];
                red[dt][j][0] += v.x, red[dt][j][1] += v.y, red[dt][j][2] += v.z, red[dt][j][3] += v.w;
            }
#pragma unroll
        for (int dt = 0; dt < Q; ++dt)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float give[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    give[k] = warp & 1 ? red[dt][j][k] : red[Q + dt][j][k];
                    fin[dt][j][k] = warp & 1 ? red[Q + dt][j][k] : red[dt][j][k];
                }
                other[(dt * NT + j) * 32 + lane] = make_float4(give[0], give[1], give[2], give[3]);
            }
        __syncthreads();
        const float4* last = xacc + (size_t)(warp ^ 3) * H * NT * 32;
        const int dt0 = warp * Q;  // (a half's quarters in order of the warps: 0, 1, then 2, 3)
        const int col = (dt0 >> 3) * 128 + col_of<HD>(gid) + 2 * (dt0 & 7);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int dt = 0; dt < Q; ++dt) {
                const float4 v = last[(dt * NT + j) * 32 + lane];
                fin[dt][j][0] += v.x, fin[dt][j][1] += v.y, fin[dt][j][2] += v.z, fin[dt][j][3] += v.w;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * j + 2 * tig + e;
                if (r >= nrows) continue;
                if (whole) {
                    const float inv = redl[r];
                    uint32_t o[Q];
#pragma unroll
                    for (int dt = 0; dt < Q; ++dt)  // (a row without any weight has sums of 0, times 0)
                        o[dt] = f32x2_to_bf16x2(fin[dt][j][e] * inv, fin[dt][j][2 + e] * inv);
                    uint16_t* to = p.a.out + (int64_t)__float_as_int(redl[R + r]) * HD + col;
                    if constexpr (Q == 1) *reinterpret_cast<uint32_t*>(to) = o[0];
                    else if constexpr (Q == 2) *reinterpret_cast<uint2*>(to) = make_uint2(o[0], o[1]);
                    else *reinterpret_cast<uint4*>(to) = make_uint4(o[0], o[1], o[2], o[3]);
                } else {
                    float* to = slot + R * 4 + r * HD + col;
#pragma unroll
                    for (int dt = 0; dt < Q; dt += 2) {
                        if constexpr (Q == 1) *reinterpret_cast<float2*>(to) = make_float2(fin[0][j][e], fin[0][j][2 + e]);
                        else *reinterpret_cast<float4*>(to + 2 * dt) = make_float4(fin[dt][j][e], fin[dt][j][2 + e], fin[dt + 1][j][e], fin[dt + 1][j][2 + e]);
                    }
                }
            }
        }
        first = false;
        if (!more) break;
    } while (true);
    // after a timeout: wait (again with a limit) for the copies that are still in flight
    if (*abort && lane == 0)
        for (int s = 0; s < ST; ++s) mbar_wait_bounded(&full[warp * ST + s], ph ^ (s < st ? 1u : 0u), nullptr, kWaitLimitCycles / 8);
}

// Joins the partial sums of the units that several CTAs share, and writes the rows that see
// nothing. WPR warps per query row split the parts, each with all its loads in flight at once.
template <int HD, int NT, bool SPARSE, int WPR>
__global__ void __launch_bounds__(32 * (WPR > 4 ? WPR : 4)) block_attn_join_kernel(const __grid_constant__ AttnParams p) {
    constexpr int R = 8 * NT, V = HD / 32, P = Shape<HD, NT>::P, NW = WPR > 4 ? WPR : 4, K = 8;
    __shared__ __align__(16) float sums[WPR > 1 ? WPR : 1][HD];
    __shared__ float ms[WPR], ls[WPR];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * (NW / WPR) + warp / WPR;
    const int wr = warp % WPR;
    const int64_t bt = row / p.a.nq;
    const int b = (int)(bt / p.t.T), tok = (int)(bt % p.t.T), head = (int)(row % p.a.nq);
    if (b >= p.t.B) {
        pdl_wait();
        return;
    }
    // (the lengths were written before the kernel that lets this one start)
    const SeqWork sw = seq_work<NT, SPARSE, P>(p, b);
    const int g = head / p.group;
    const int r_abs = SPARSE ? head - g * p.group : tok * p.group + head - g * p.group;
    const int part = SPARSE ? tok : r_abs / R, r = SPARSE ? r_abs : r_abs - part * R;
    int per = 0, base = 0;  // the CTAs' stretch, and where the row's unit starts on the line
    if (p.t.B <= 32) {      // found while the parts are still being summed
        const int n = lane < p.t.B ? seq_work<NT, SPARSE, P>(p, min(lane, p.t.B - 1)).line() : 0;
        per = stretch_of(__reduce_add_sync(0xffffffffu, n), p.grid);
        base = __reduce_add_sync(0xffffffffu, lane < b ? n : 0) + (SPARSE ? part * p.c.nkv + g : g * sw.inner + part) * (sw.steps + kUnitCost);
    }
    pdl_wait();
    if (tok >= sw.q) return;
    float M = -INFINITY, L = 0.f, a[V];
#pragma unroll
    for (int v = 0; v < V; ++v) a[v] = 0.f;
    if (sw.steps > 0) {
        if (p.t.B > 32) {
            per = *p.per;
            base = p.unit_base[unit_index<SPARSE>(p, b, g, part)];
        }
        const int c0 = (base + kUnitCost) / per, c1 = (base + kUnitCost + sw.steps - 1) / per;  // of its first and last step
        if (c0 == c1) return;  // finished by one CTA
        // in CTA c0 the unit is the last (slot 1) unless it is also the first; in later ones the first
        auto slot = [&](int c) {
            return p.parts + (int64_t)(c * 2 + (c == c0 && c0 * per < base ? 1 : 0)) * (R * (HD + 4));
        };
        for (int k0 = c0 + wr; k0 <= c1; k0 += K * WPR) {
            float m[K], l[K], x[K][V];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = k0 + k * WPR;
                m[k] = -INFINITY;
                l[k] = 0.f;
#pragma unroll
                for (int v = 0; v < V; ++v) x[k][v] = 0.f;
                if (c <= c1) {
                    const float* s = slot(c);
                    m[k] = s[r];
                    l[k] = s[R + r];
                    const float* y = s + R * 4 + r * HD + lane * V;
                    if constexpr (V == 2) {
                        const float2 t = *reinterpret_cast<const float2*>(y);
                        x[k][0] = t.x, x[k][1] = t.y;
                    } else {
#pragma unroll
                        for (int v = 0; v < V; v += 4) {
                            const float4 t = *reinterpret_cast<const float4*>(y + v);
                            x[k][v] = t.x, x[k][v + 1] = t.y, x[k][v + 2] = t.z, x[k][v + 3] = t.w;
                        }
                    }
                }
            }
            float mn = M;
#pragma unroll
            for (int k = 0; k < K; ++k) mn = fmaxf(mn, m[k]);
            const float al = M == -INFINITY ? 0.f : ex2(M - mn);
            L *= al;
#pragma unroll
            for (int v = 0; v < V; ++v) a[v] *= al;
            M = mn;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const float f = m[k] == -INFINITY ? 0.f : ex2(m[k] - mn);
                L += f * l[k];
#pragma unroll
                for (int v = 0; v < V; ++v) a[v] = fmaf(f, x[k][v], a[v]);
            }
        }
        if constexpr (WPR > 1) {
#pragma unroll
            for (int v = 0; v < V; ++v) sums[wr][lane * V + v] = a[v];
            if (lane == 0) ms[wr] = M, ls[wr] = L;
            __syncthreads();  // (every warp of the CTA has the same row)
            if (wr) return;
            M = -INFINITY;
#pragma unroll
            for (int w = 0; w < WPR; ++w) M = fmaxf(M, ms[w]);
            L = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) a[v] = 0.f;
#pragma unroll
            for (int w = 0; w < WPR; ++w) {
                const float f = ms[w] == -INFINITY ? 0.f : ex2(ms[w] - M);
                L += f * ls[w];
#pragma unroll
                for (int v = 0; v < V; ++v) a[v] = fmaf(f, sums[w][lane * V + v], a[v]);
            }
        }
    } else if (wr) {
        return;
    }
    const bool some = !(L <= 0.f);
    const float inv = some ? 1.f / L : 0.f;
    uint16_t* out = p.a.out + row * HD + lane * V;
#pragma unroll
    for (int v = 0; v < V; v += 2)
        *reinterpret_cast<uint32_t*>(out + v) = some ? f32x2_to_bf16x2(a[v] * inv, a[v + 1] * inv) : 0u;
    if (lane == 0) {
        const float lse2 = some ? M + log2f(L) : -INFINITY;
        if (p.a.out_lse) p.a.out_lse[row] = lse2 * kLn2;
        if (!SPARSE && p.a.out_mass) p.row_lse[((int64_t)b * p.c.nkv + g) * p.t.T * p.group + r_abs] = lse2;
    }
}

// out_mass[b, j] over a CTA's 32 tiles: a thread sums one tile's rows of every eighth kv head in
// order (they are neighbours: four at a time where T group allows), then the eight sums and the
// block's tiles are added in order. (Lanes across the rows, one load in flight each, took 13
// us where this takes 8.)
__global__ void __launch_bounds__(256) block_mass_kernel(const __grid_constant__ AttnParams p) {
    __shared__ float sums[8][32];
    const int b = blockIdx.y, t = threadIdx.x & 31, gs = threadIdx.x >> 5;
    const int tile = (int)blockIdx.x * 32 + t;
    const SeqWork w = seq_work<1, false, 1>(p, b);  // (written before the kernels that let this one start)
    const int pitch = (int)p.t.T * p.group, rows = w.q * p.group, rows4 = pitch % 4 ? 0 : rows & ~3;
    pdl_wait();
    float sum = 0.f;
    if (tile < w.tiles)
        for (int g = gs; g < p.c.nkv; g += 8) {
            const int64_t head = (int64_t)b * p.c.nkv + g;
            const float* x = p.tile_lse + (head * p.tiles + tile) * pitch;
            const float* L = p.row_lse + head * pitch;
            auto add = [&](float v, float l) { sum += v == -INFINITY ? 0.f : ex2(v - l); };
#pragma unroll 4
            for (int r = 0; r < rows4; r += 4) {
                const float4 v = *reinterpret_cast<const float4*>(x + r), l = *reinterpret_cast<const float4*>(L + r);
                add(v.x, l.x), add(v.y, l.y), add(v.z, l.z), add(v.w, l.w);
            }
#pragma unroll 4
            for (int r = rows4; r < rows; ++r) add(x[r], L[r]);
        }
    sums[gs][t] = sum;
    __syncthreads();
    const int per = 1 << p.tile_shift;  // tiles per block
    const int64_t j = ((int64_t)blockIdx.x * 32 >> p.tile_shift) + threadIdx.x;
    if (threadIdx.x >= 32 >> p.tile_shift || j >= p.t.n_table) return;
    sum = 0.f;
    for (int u = 0; u < per; ++u)
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += sums[k][threadIdx.x * per + u];
    const int64_t at = (int64_t)b * p.t.n_table + j;
    p.a.out_mass[at] = (p.a.mass ? p.a.mass[at] : 0.f) + sum;
}

size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

// Query rows per unit, as 8 NT: a head's rows in as few row tiles as the accumulators allow
// (40 rows of 64 dims, 32 of 128, 16 of 256), each with an equal share of them.
int pick_nt(int hd, int64_t rows) {
    const int most = hd == 64 ? 5 : hd == 128 ? 4 : 2;
    const int64_t tiles = (rows + 8 * most - 1) / (8 * most);
    return (int)((rows + 8 * tiles - 1) / (8 * tiles));
}

struct Layout {
    int nt, row_tiles;
    int64_t units, tiles;
    size_t base, parts, row_lse, tile_lse, bytes;  // offsets
};
Layout layout_of(const BlockCache& c, int B, int64_t T, int nq, int64_t n_table, bool sparse, bool mass) {
    Layout l{};
    const int64_t rows = (sparse ? 1 : T) * (nq / c.nkv);
    l.nt = pick_nt(c.hd, rows);
    l.row_tiles = (int)((rows + 8 * l.nt - 1) / (8 * l.nt));
    l.units = (int64_t)B * c.nkv * (sparse ? T : l.row_tiles);
    l.tiles = n_table * (c.bs / 16);
    l.base = 16;
    l.parts = l.base + up16((size_t)l.units * 4);
    l.row_lse = l.parts + (size_t)2 * kMaxGrid * 8 * l.nt * (c.hd + 4) * 4;
    const size_t q_rows = (size_t)B * T * nq;
    l.tile_lse = l.row_lse + (mass ? up16(q_rows * 4) : 0);
    l.bytes = l.tile_lse + (mass ? up16(q_rows * 4 * (size_t)l.tiles) : 0);
    return l;
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static EncodeFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeFn>(f);
    });
    return fn;
}

// The cache's codes as a 4-D tensor (byte of the row, row of the block, head, block), in boxes
// of 16 rows of at most 128 bytes.
bool cache_map(CUtensorMap* m, const BlockCache& c, const uint8_t* base) {
    EncodeFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[4] = {(cuuint64_t)c.hd, (cuuint64_t)c.bs, (cuuint64_t)c.nkv, (cuuint64_t)c.num_blocks};
    cuuint64_t strides[3] = {(cuuint64_t)c.row_stride, (cuuint64_t)c.head_stride, (cuuint64_t)c.block_stride};
    cuuint32_t box[4] = {(cuuint32_t)(c.hd < 128 ? c.hd : 128), 16, 1, 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, c.hd == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HD, int NT, bool SPARSE>
cudaError_t launch_attn(AttnParams p, const CUtensorMap& km, const CUtensorMap& vm, int sms, cudaStream_t s) {
    using Sh = Shape<HD, NT>;
    auto kern = block_attn_kernel<HD, NT, SPARSE>;
    static std::atomic<uint64_t> devices{0};
    cudaError_t e = allow_smem(kern, Sh::kSmem, devices);
    if (e != cudaSuccess) return e;
    int grid = sms * Sh::kPerSm;
    if (grid > kMaxGrid) grid = kMaxGrid;
    p.grid = grid;
    if ((e = launch_after(kern, dim3((unsigned)grid), kThreads, Sh::kSmem, s, p, km, vm)) != cudaSuccess) return e;
    // eight warps per row while the rows are few (many parts each), one when they fill the GPU
    const int64_t rows = (int64_t)p.t.B * p.t.T * p.a.nq;
    if (rows <= 1024) return launch_after(block_attn_join_kernel<HD, NT, SPARSE, 8>, dim3((unsigned)rows), 256, 0, s, p);
    return launch_after(block_attn_join_kernel<HD, NT, SPARSE, 1>, dim3((unsigned)((rows + 3) / 4)), 128, 0, s, p);
}

template <int HD, bool SPARSE>
cudaError_t launch_attn_nt(int nt, const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm, int sms, cudaStream_t s) {
    if (nt == 1) return launch_attn<HD, 1, SPARSE>(p, km, vm, sms, s);
    if constexpr (!SPARSE && HD <= 128) {
        if (nt == 3) return launch_attn<HD, 3, SPARSE>(p, km, vm, sms, s);
        if (nt == 4) return launch_attn<HD, 4, SPARSE>(p, km, vm, sms, s);
    }
    if constexpr (!SPARSE && HD == 64)
        if (nt == 5) return launch_attn<HD, 5, SPARSE>(p, km, vm, sms, s);
    return launch_attn<HD, 2, SPARSE>(p, km, vm, sms, s);
}

template <int HD>
cudaError_t launch_attn_hd(int nt, const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm, int sms, cudaStream_t s) {
    return p.a.sel ? launch_attn_nt<HD, true>(nt, p, km, vm, sms, s) : launch_attn_nt<HD, false>(nt, p, km, vm, sms, s);
}

}  // namespace

int block_attn_max_group() { return kMaxGroup; }
int block_attn_max_t() { return kMaxT; }

bool block_attn_fits(const BlockCache& c, int B, int T, int nq, int64_t n_table, bool sparse, int n_sel) {
    const Layout l = layout_of(c, B, T, nq, n_table, sparse, false);
    const int64_t tiles = sparse ? (int64_t)n_sel * (c.bs / 16) : l.tiles;  // (at most 2^26, and units below 2^35)
    return (int64_t)B * T * nq <= INT32_MAX && l.units * (tiles + kUnitCost) <= INT32_MAX;
}

size_t block_attn_ws_bytes(const BlockCache& c, int B, int T, int nq, int64_t n_table, bool sparse, bool mass) {
    return layout_of(c, B, T, nq, n_table, sparse, mass).bytes;
}

cudaError_t block_attn_launch(const BlockCache& c, const BlockBatch& t, const BlockAttnArgs& a,
                              cudaStream_t s) {
    const bool sparse = a.sel != nullptr;
    const Layout l = layout_of(c, t.B, t.T, a.nq, t.n_table, sparse, a.out_mass != nullptr);
    uint8_t* ws = static_cast<uint8_t*>(a.ws);
    AttnParams p{c, t, a, 0, a.nq / c.nkv, l.row_tiles, l.tiles, reinterpret_cast<int32_t*>(ws),
                 reinterpret_cast<int32_t*>(ws + l.base), c.bs == 16 ? 0 : c.bs == 32 ? 1 : 2,
                 ((1u << 20) + (uint32_t)(a.nq / c.nkv) - 1u) / (uint32_t)(a.nq / c.nkv), reinterpret_cast<float*>(ws + l.parts),
                 reinterpret_cast<float*>(ws + l.row_lse), reinterpret_cast<float*>(ws + l.tile_lse)};
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    CUtensorMap km{}, vm{};
    if (!cache_map(&km, c, c.k) || !cache_map(&vm, c, c.v)) return cudaErrorInvalidValue;
    e = c.hd == 64 ? launch_attn_hd<64>(l.nt, p, km, vm, sms, s)
                   : c.hd == 128 ? launch_attn_hd<128>(l.nt, p, km, vm, sms, s) : launch_attn_hd<256>(l.nt, p, km, vm, sms, s);
    if (e != cudaSuccess || !a.out_mass) return e;
    return launch_after(block_mass_kernel, dim3((unsigned)((l.tiles + 31) / 32), (unsigned)t.B), 256, 0, s, p);
}

}  // namespace mtp

// tc_cache_attend: one new token's attention over a paged cache, fused with
// the memory's read and with the accumulation of each pair's weight.
//
//   y_h = sum_j p_j v_j + sigmoid(g_h) q_h A,  p = softmax_j(<q_h,k_j>/sqrt(d))
//
// Bound by memory: every key and value is read once per group of query heads.
// The work, tiles of 64 pairs of one (row, key/value head, group of query
// heads), is laid end to end and cut into equal parts, one per block, wherever
// the rows begin and end: rows of any lengths keep every SM equally busy.  A
// block walks its part with a running maximum and sum; at the end of a row's
// stretch it stores the partial (m, l, O).  The join kernel adds the partials
// of each row's stretches, the memory's read, and (from the scores the first
// kernel left in the workspace) the weights.
//
// bf16: each of the four warps takes 16 pairs of a tile, on its own: its own
// ring of TMA loads (16 x d boxes, swizzled; a page holds a multiple of 16
// pairs), its own running statistics; no barrier between warps until a row's
// stretch ends.  Products run as S^T = K Q^T (16 pairs x 8 heads) and
// O^T = V^T P^T with m16n8k16: with the pairs as M, eight heads fill a product
// that would be half empty with the heads as M, and the same lanes hold a
// head's scores and its outputs, so rescaling needs no exchange.  P enters as a
// bf16 pair hi + lo, so the outputs keep float32's precision up to their one
// rounding.  The tensor pipe is nowhere near busy (16 d multiply-adds a pair
// against 4 d bytes), so what matters is the loads in flight.
//
// float32: the same walk with float32 multiply-adds, d/4 lanes per pair.

#include <cuda.h>

#include <cfloat>

#include "paged_cache.cuh"
#include "sm100_ptx.cuh"

namespace tc {
namespace {

using namespace sm100;

constexpr int kTile = 64;        // pairs per tile
constexpr int kThreads = 128;    // first kernel
constexpr int kWarps = 4;
constexpr int kWarpPairs = 16;   // pairs of a tile one warp takes
constexpr int kJoinThreads = 256;

__device__ __forceinline__ int64_t row_pairs(const AttendParams &p, int b) {
    const int64_t n = p.row_len[b];
    return n < 0 || n > p.c.capacity() ? 0 : n;
}
__device__ __forceinline__ int row_tiles(const AttendParams &p, int b) {
    return (int)((row_pairs(p, b) + kTile - 1) / kTile);
}

// Position in the laid-out work: unit u is tile `tile` of item `item` of row b.
struct Cursor {
    int64_t left;  // units until the end of the part, this one included
    int b, item, tile, tiles;
    int64_t n;     // pairs of row b

    __device__ __forceinline__ void enter_row(const AttendParams &p) {
        n = row_pairs(p, b);
        tiles = (int)((n + kTile - 1) / kTile);
    }
    // `per_row`: items a row has
    __device__ __forceinline__ void next(const AttendParams &p, int per_row) {
        if (--left == 0) return;
        if (++tile < tiles) return;
        tile = 0;
        if (++item < per_row) return;
        item = 0;
        do {
            ++b;
            enter_row(p);
        } while (tiles == 0);  // left > 0: a row with tiles follows
    }
};

// This block's part of total = per_row * (tiles of all rows) units, cut evenly
// over min(gridDim.x, total) blocks.  Every block adds up the rows' tiles by
// itself; block 0 of the first kernel also stores them (prefix) for the join.
// Returns false when there is nothing to do.  Block-wide.
__device__ bool find_part(const AttendParams &p, int per_row, Cursor &cur) {
    __shared__ int64_t s_sum[kWarps];
    __shared__ int64_t s_off;
    __shared__ int s_row;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = p.c.B;
    const int per = (B + kThreads - 1) / kThreads;
    const int b0 = tid * per, b1 = min(B, b0 + per);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += row_tiles(p, b);
    int64_t v = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    if (lane == 31) s_sum[warp] = v;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_sum[w];
        all += s_sum[w];
    }
    before += v - mine;
    if (blockIdx.x == 0) {
        int64_t x = before;
        for (int b = b0; b < b1; ++b) {
            p.prefix[b] = x;
            x += row_tiles(p, b);
        }
        if (tid == 0) p.prefix[B] = all;
    }
    const int64_t total = all * per_row, G = total < gridDim.x ? total : gridDim.x;
    if (blockIdx.x >= G) return false;
    const int64_t u0 = blockIdx.x * total / G, u1 = (blockIdx.x + 1) * total / G;
    if (u0 >= before * per_row && u0 < (before + mine) * per_row) {
        int64_t x = before;
        int b = b0;
        for (;; ++b) {
            const int t = row_tiles(p, b);
            if (u0 < (x + t) * per_row) break;
            x += t;
        }
        s_row = b;
        s_off = u0 - x * per_row;
    }
    __syncthreads();
    cur.b = s_row;
    cur.enter_row(p);
    cur.item = (int)(s_off / cur.tiles);
    cur.tile = (int)(s_off % cur.tiles);
    cur.left = u1 - u0;
    return true;
}

// Partial results: the slot of (block, item) is block + item's number, which
// grows by at least one along the work, so no two share one.
__host__ __device__ inline int64_t part_floats(int heads, int d) { return (int64_t)heads * (d + 2); }

// ---- bf16 -----------------------------------------------------------------------

// Byte offset of 16-byte chunk c of row r in a 16-row tile of d bf16, as TMA
// writes it with the widest swizzle a row allows (boxes of at most 64 columns).
template <int D>
__device__ __forceinline__ uint32_t tile_offset(int r, int c) {
    constexpr int RB = D >= 64 ? 128 : D * 2;  // bytes of a box row
    constexpr int CPR = RB / 16;
    const int box = c / CPR, cc = c % CPR;
    const int x = RB == 128 ? (r & 7) : RB == 64 ? ((r >> 1) & 3) : ((r >> 2) & 1);
    return box * (16 * RB) + r * RB + ((cc ^ x) << 4);
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y)
        : "memory");
}

template <int D, int NT>
struct Bf16Shape {
    static constexpr int STAGES = D == 128 ? (NT == 1 ? 3 : 2) : 4;
    static constexpr int STAGE_BYTES = 16 * D * 2 * 2;  // one warp's keys and values
    static constexpr int HEADS = 8 * NT;
    static constexpr int OS = D + 4;                    // floats between heads of a warp's outputs
    static constexpr int RING = kWarps * STAGES * STAGE_BYTES;
    static constexpr int SMEM = 1024 + RING + 2 * HEADS * OS * 4;
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads) attend_bf16_kernel(const __grid_constant__ CUtensorMap map_k,
                                                               const __grid_constant__ CUtensorMap map_v,
                                                               const __grid_constant__ AttendParams p) {
    using S = Bf16Shape<D, NT>;
    constexpr int KS = D / 16;      // k-steps of a score, 16-wide blocks of the output
    constexpr int BOX = D >= 64 ? 64 : D;
    extern __shared__ unsigned char dyn[];
    __shared__ __align__(8) uint64_t s_bar[kWarps][S::STAGES];
    __shared__ float s_m[kWarps][S::HEADS], s_l[kWarps][S::HEADS];
    __shared__ int s_abort;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (lane == 0)
        for (int s = 0; s < S::STAGES; ++s) mbar_init(&s_bar[warp][s], 1);
    if (tid == 0) s_abort = 0;
    fence_mbar_init();
    griddep_wait();
    griddep_launch_dependents();
    const int per_row = p.c.H * p.items;
    Cursor cur;
    const bool any = find_part(p, per_row, cur);  // its barrier also publishes the mbarriers
    if (!any) return;
    __syncthreads();

    const uint32_t dyn0 = (smem_u32(dyn) + 1023u) & ~1023u;
    const uint32_t ring = dyn0 + warp * S::STAGES * S::STAGE_BYTES;
    float *s_o = reinterpret_cast<float *>(dyn + (dyn0 - smem_u32(dyn)) + S::RING);  // [2][HEADS][OS]

    Cursor ahead = cur;
    int ahead_page = -1;  // table entry of the next load, fetched one step early
    auto fetch_page = [&]() {
        const int64_t j0 = (int64_t)ahead.tile * kTile + warp * kWarpPairs;
        if (ahead.left > 0 && j0 < ahead.n) ahead_page = p.c.table[(int64_t)ahead.b * p.c.max_pages + j0 / p.c.page];
    };
    fetch_page();
    uint32_t valid = 0;   // pairs in each stage, 8 bits each
    // loads the next tile's 16 pairs into a stage, and moves on
    auto issue = [&](int st) {
        valid &= ~(0xffu << (8 * st));
        if (ahead.left <= 0) return;
        const int64_t j0 = (int64_t)ahead.tile * kTile + warp * kWarpPairs;
        if (j0 < ahead.n) {
            if (page_ok(p.c, ahead_page)) {
                valid |= (uint32_t)min((int64_t)kWarpPairs, ahead.n - j0) << (8 * st);
                if (lane == 0) {
                    const int row = (int)pool_row(p.c, ahead_page, ahead.item / p.items, (int)(j0 % p.c.page));
                    uint64_t *bar = &s_bar[warp][st];
                    const uint32_t dst = ring + st * S::STAGE_BYTES;
                    mbar_expect_tx(bar, S::STAGE_BYTES);
#pragma unroll
                    for (int x = 0; x < D; x += BOX) {
                        tma_load_2d(dst + x * 32, &map_k, bar, x, row);
                        tma_load_2d(dst + 32 * D + x * 32, &map_v, bar, x, row);
                    }
                }
            } else if (lane == 0) {
                report(p.c.status, TC_ERR_DEVICE_BOUNDS);
            }
        }
        ahead.next(p, per_row);
        fetch_page();
    };
#pragma unroll
    for (int s = 0; s < S::STAGES; ++s) issue(s);

    const float scale = rsqrtf((float)D) * 1.4426950408889634f;  // log2(e)/sqrt(d)
    uint32_t phase = 0;  // parity of each stage's next completion
    bool dead = false;
    int st = 0;
    while (cur.left > 0) {
        // ---- one stretch: tiles of one (row, head, group of query heads) -----------
        const int b = cur.b, h = cur.item / p.items, grp = cur.item % p.items;
        const int h0 = h * p.G + grp * S::HEADS;  // first query head
        const int heads = min(S::HEADS, p.G - grp * S::HEADS);
        const int64_t item = (int64_t)b * per_row + cur.item;
        uint32_t qf[NT][KS][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int hh = t * 8 + lane / 4;
            const uint32_t *qp = reinterpret_cast<const uint32_t *>(p.q) +
                                 (((int64_t)b * p.Hq + h0 + hh) * D + (lane % 4) * 2) / 2;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                qf[t][k][0] = hh < heads ? qp[k * 8] : 0u;
                qf[t][k][1] = hh < heads ? qp[k * 8 + 4] : 0u;
            }
        }
        float m[NT][2], l[NT][2], o[NT][KS][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            m[t][0] = m[t][1] = -INFINITY;
            l[t][0] = l[t][1] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][k][e] = 0.f;
        }
        bool more = true;
        while (more) {
            const int64_t j0 = (int64_t)cur.tile * kTile + warp * kWarpPairs;
            const int nv = (valid >> (8 * st)) & 0xff;
            if (nv && !dead) {
                if (!mbar_wait(&s_bar[warp][st], (phase >> st) & 1u, &s_abort, p.c.status, p.wait_ns)) dead = true;
            }
            if (nv && !dead) {
                phase ^= 1u << st;
                const uint32_t ks = ring + st * S::STAGE_BYTES, vs = ks + 32 * D;
                // S^T = K Q^T, in two chains of products
                float sc[NT][2][4];
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[t][0][e] = sc[t][1][e] = 0.f;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t a[4];
                    ldsm_x4(ks + tile_offset<D>((lane & 7) + ((lane >> 3) & 1) * 8, 2 * k + (lane >> 4)), a);
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma16816(sc[t][k & 1], a, qf[t][k][0], qf[t][k][1]);
                }
                uint32_t ph[NT][2], pl[NT][2];
                const int r0 = lane / 4, r1 = r0 + 8;  // this lane's pairs
                bool grew = false;
                float corr[NT][2];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    float z[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[e] = (sc[t][0][e] + sc[t][1][e]) * scale;
                    if (p.z) {
                        // the group's scores of a pair lie side by side
                        const int pg = p.c.table[(int64_t)b * p.c.max_pages + j0 / p.c.page];
                        float *zr = p.z + pool_row(p.c, pg, h, (int)(j0 % p.c.page)) * p.G + grp * S::HEADS;
                        const int c0 = t * 8 + (lane % 4) * 2;
                        if (r0 < nv) {
                            if (c0 < heads) zr[(int64_t)r0 * p.G + c0] = z[0];
                            if (c0 + 1 < heads) zr[(int64_t)r0 * p.G + c0 + 1] = z[1];
                        }
                        if (r1 < nv) {
                            if (c0 < heads) zr[(int64_t)r1 * p.G + c0] = z[2];
                            if (c0 + 1 < heads) zr[(int64_t)r1 * p.G + c0 + 1] = z[3];
                        }
                    }
                    if (r0 >= nv) z[0] = z[1] = -INFINITY;
                    if (r1 >= nv) z[2] = z[3] = -INFINITY;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = fmaxf(z[e], z[e + 2]);
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                        const float mn = fmaxf(m[t][e], x);
                        const float ref = mn == -INFINITY ? 0.f : mn;  // every score -inf so far
                        corr[t][e] = ex2(m[t][e] - ref);
                        grew |= mn > m[t][e];
                        m[t][e] = mn;
                        z[e] = ex2(z[e] - ref);
                        z[e + 2] = ex2(z[e + 2] - ref);
                        l[t][e] = fmaf(l[t][e], corr[t][e], z[e] + z[e + 2]);
                    }
                    // P^T as a bf16 pair: hi rounded, lo the rest
                    const uint32_t h01 = pack_bf16(z[0], z[1]), h23 = pack_bf16(z[2], z[3]);
                    const uint32_t l01 = pack_bf16(z[0] - __uint_as_float(h01 << 16), z[1] - __uint_as_float(h01 & 0xffff0000u));
                    const uint32_t l23 = pack_bf16(z[2] - __uint_as_float(h23 << 16), z[3] - __uint_as_float(h23 & 0xffff0000u));
                    ph[t][0] = transpose8x8(h01);
                    ph[t][1] = transpose8x8(h23);
                    pl[t][0] = transpose8x8(l01);
                    pl[t][1] = transpose8x8(l23);
                }
                if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int k = 0; k < KS; ++k)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[t][k][e] *= corr[t][e & 1];
                }
                // values of slots behind the row's pairs may hold anything: 0 * NaN
                const int c0 = (lane % 4) * 2;
                const uint32_t keep0 = (c0 < nv ? 0xffffu : 0u) | (c0 + 1 < nv ? 0xffff0000u : 0u);
                const uint32_t keep1 = (c0 + 8 < nv ? 0xffffu : 0u) | (c0 + 9 < nv ? 0xffff0000u : 0u);
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t a[4];
                    ldsm_x4_t(vs + tile_offset<D>((lane & 7) + (lane >> 4) * 8, 2 * k + ((lane >> 3) & 1)), a);
                    if (nv < kWarpPairs) {
                        a[0] &= keep0;
                        a[1] &= keep0;
                        a[2] &= keep1;
                        a[3] &= keep1;
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        mma16816(o[t][k], a, ph[t][0], ph[t][1]);
                        mma16816(o[t][k], a, pl[t][0], pl[t][1]);
                    }
                }
            }
            __syncwarp();
            if (!dead) issue(st);
            st = st + 1 == S::STAGES ? 0 : st + 1;
            const int item0 = cur.item, row0 = cur.b;
            cur.next(p, per_row);
            more = cur.left > 0 && cur.item == item0 && cur.b == row0;
        }
        // ---- the warps' results, joined ----------------------------------------------
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = l[t][e];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                if (lane < 4) {
                    s_m[warp][t * 8 + lane * 2 + e] = m[t][e];
                    s_l[warp][t * 8 + lane * 2 + e] = x;
                }
            }
        __syncthreads();
        // each warp scales its outputs to the common maximum; pairs of warps add
        float f[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int hh = t * 8 + (lane % 4) * 2 + e;
                float mx = fmaxf(fmaxf(s_m[0][hh], s_m[1][hh]), fmaxf(s_m[2][hh], s_m[3][hh]));
                if (mx == -INFINITY) mx = 0.f;
                f[t][e] = ex2(m[t][e] - mx);
            }
        float *so = s_o + (warp & 1) * S::HEADS * S::OS;
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
            if ((warp >> 1) == pass) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k = 0; k < KS; ++k)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float *x = so + (t * 8 + (lane % 4) * 2 + (e & 1)) * S::OS + k * 16 + lane / 4 + (e >> 1) * 8;
                            const float val = o[t][k][e] * f[t][e & 1];
                            *x = pass == 0 ? val : *x + val;
                        }
            }
            __syncthreads();
        }
        float *part = p.part + (blockIdx.x + item) * part_floats(S::HEADS, D);
        for (int x = tid; x < heads * D; x += kThreads) {
            const int hh = x / D, dd = x % D;
            part[x] = s_o[hh * S::OS + dd] + s_o[(S::HEADS + hh) * S::OS + dd];
        }
        if (tid < heads) {
            const float mx = fmaxf(fmaxf(s_m[0][tid], s_m[1][tid]), fmaxf(s_m[2][tid], s_m[3][tid]));
            float ls = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) ls += s_l[w][tid] * ex2(s_m[w][tid] - (mx == -INFINITY ? 0.f : mx));
            part[S::HEADS * D + 2 * tid] = mx;
            part[S::HEADS * D + 2 * tid + 1] = ls;
        }
        __syncthreads();
    }
    // after a wait that ran out: no copy may land once the block is gone
    if (dead)
        for (int s = 0; s < S::STAGES; ++s)
            if ((valid >> (8 * s)) & 0xff) mbar_wait_drain(&s_bar[warp][s], (phase >> s) & 1u);
}

// ---- float32 ----------------------------------------------------------------------

template <int D, int GT>
__global__ void __launch_bounds__(kThreads) attend_f32_kernel(const __grid_constant__ AttendParams p) {
    constexpr int LPK = D / 4;                 // lanes per pair
    constexpr int KPW = 32 / LPK;              // pairs a warp loads at once
    constexpr int NG = kWarps * KPW;           // groups of lanes with statistics of their own
    constexpr int BATCH = 4;                   // loads of keys in flight per lane (and of values)
    __shared__ float s_m[NG][GT], s_l[NG][GT];
    __shared__ __align__(16) float s_o[NG][GT][D];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int sub = lane / LPK, li = lane % LPK, grp_id = warp * KPW + sub;
    griddep_wait();
    griddep_launch_dependents();
    const int per_row = p.c.H * p.items;
    Cursor cur;
    if (!find_part(p, per_row, cur)) return;
    const float scale = rsqrtf((float)D) * 1.4426950408889634f;
    const float *kpool = reinterpret_cast<const float *>(p.c.k), *vpool = reinterpret_cast<const float *>(p.c.v);
    while (cur.left > 0) {
        const int b = cur.b, h = cur.item / p.items, grp = cur.item % p.items;
        const int h0 = h * p.G + grp * GT, heads = min(GT, p.G - grp * GT);
        const int64_t n = cur.n, item = (int64_t)b * per_row + cur.item;
        float4 q[GT], o[GT];
        float m[GT], l[GT];
#pragma unroll
        for (int g = 0; g < GT; ++g) {
            q[g] = g < heads ? reinterpret_cast<const float4 *>(p.q)[((int64_t)b * p.Hq + h0 + g) * LPK + li]
                             : make_float4(0.f, 0.f, 0.f, 0.f);
            o[g] = make_float4(0.f, 0.f, 0.f, 0.f);
            m[g] = -INFINITY;
            l[g] = 0.f;
        }
        bool more = true;
        while (more) {
            const int64_t j0 = (int64_t)cur.tile * kTile + warp * kWarpPairs;
            int nv = (int)max((int64_t)0, min((int64_t)kWarpPairs, n - j0));
            int64_t row = 0;
            if (nv) {
                const int pg = p.c.table[(int64_t)b * p.c.max_pages + j0 / p.c.page];
                if (page_ok(p.c, pg)) {
                    row = pool_row(p.c, pg, h, (int)(j0 % p.c.page));
                } else {
                    nv = 0;
                    if (lane == 0) report(p.c.status, TC_ERR_DEVICE_BOUNDS);
                }
            }
#pragma unroll
            for (int u = 0; u < kWarpPairs / KPW; u += BATCH) {
                if (u * KPW >= nv) break;
                float4 k4[BATCH], v4[BATCH];
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int j = (u + i) * KPW + sub;
                    k4[i] = v4[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (u + i < kWarpPairs / KPW && j < nv) {
                        k4[i] = reinterpret_cast<const float4 *>(kpool)[(row + j) * LPK + li];
                        v4[i] = reinterpret_cast<const float4 *>(vpool)[(row + j) * LPK + li];
                    }
                }
#pragma unroll
                for (int g = 0; g < GT; ++g) {
                    float z[BATCH], mx = m[g];
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        float x = q[g].x * k4[i].x;
                        x = fmaf(q[g].y, k4[i].y, x);
                        x = fmaf(q[g].z, k4[i].z, x);
                        x = fmaf(q[g].w, k4[i].w, x);
#pragma unroll
                        for (int off = LPK / 2; off >= 1; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
                        const int j = (u + i) * KPW + sub;
                        const bool in = u + i < kWarpPairs / KPW && j < nv;
                        z[i] = x * scale;
                        if (p.z && in && li == 0 && g < heads) p.z[(row + j) * p.G + grp * GT + g] = z[i];
                        if (!in) z[i] = -INFINITY;
                        mx = fmaxf(mx, z[i]);
                    }
                    const float ref = mx == -INFINITY ? 0.f : mx, corr = ex2(m[g] - ref);
                    m[g] = mx;
                    l[g] *= corr;
                    o[g].x *= corr;
                    o[g].y *= corr;
                    o[g].z *= corr;
                    o[g].w *= corr;
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        const float w = ex2(z[i] - ref);
                        l[g] += w;
                        o[g].x = fmaf(w, v4[i].x, o[g].x);
                        o[g].y = fmaf(w, v4[i].y, o[g].y);
                        o[g].z = fmaf(w, v4[i].z, o[g].z);
                        o[g].w = fmaf(w, v4[i].w, o[g].w);
                    }
                }
            }
            const int item0 = cur.item, row0 = cur.b;
            cur.next(p, per_row);
            more = cur.left > 0 && cur.item == item0 && cur.b == row0;
        }
#pragma unroll
        for (int g = 0; g < GT; ++g) {
            if (li == 0) {
                s_m[grp_id][g] = m[g];
                s_l[grp_id][g] = l[g];
            }
            reinterpret_cast<float4 *>(&s_o[grp_id][g][0])[li] = o[g];
        }
        __syncthreads();
        float *part = p.part + (blockIdx.x + item) * part_floats(GT, D);
        for (int x = tid; x < heads * D; x += kThreads) {
            const int g = x / D, dd = x % D;
            float mx = -INFINITY, sum = 0.f;
#pragma unroll
            for (int i = 0; i < NG; ++i) mx = fmaxf(mx, s_m[i][g]);
            if (mx == -INFINITY) mx = 0.f;
#pragma unroll
            for (int i = 0; i < NG; ++i) sum = fmaf(ex2(s_m[i][g] - mx), s_o[i][g][dd], sum);
            part[x] = sum;
        }
        if (tid < heads) {
            float mx = -INFINITY, sum = 0.f;
#pragma unroll
            for (int i = 0; i < NG; ++i) mx = fmaxf(mx, s_m[i][tid]);
#pragma unroll
            for (int i = 0; i < NG; ++i) sum = fmaf(ex2(s_m[i][tid] - (mx == -INFINITY ? 0.f : mx)), s_l[i][tid], sum);
            part[GT * D + 2 * tid] = mx;
            part[GT * D + 2 * tid + 1] = sum;
        }
        __syncthreads();
    }
}

// ---- the join ---------------------------------------------------------------------

struct JoinShape {
    int y_blocks, unit_heads, units_per_bh;  // outputs: blocks, query heads a unit covers
    int mass_blocks;                         // weights: blocks (0: none)
    int split_grid;                          // blocks of the first kernel
};

// The blocks of the first kernel that met units u0 .. u1-1 (u1 > u0).
struct Parts {
    int64_t first, last;
    __device__ __forceinline__ Parts(int64_t u0, int64_t u1, int64_t total, int64_t G)
        : first(((u0 + 1) * G - 1) / total), last((u1 * G - 1) / total) {}
};

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(const __grid_constant__ AttendParams p,
                                                                   const __grid_constant__ JoinShape js) {
    constexpr int HB = 4;                    // query heads per pass over A
    constexpr int CG = D / 4, RG = kJoinThreads / CG;
    constexpr int DG = kJoinThreads / D;     // groups of threads over the partials
    __shared__ __align__(16) float s_red[RG][HB][D];
    __shared__ float s_q[HB][D];
    __shared__ float s_w[128], s_x[128];
    __shared__ int s_row;
    float *red = &s_red[0][0][0];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const CacheParams &c = p.c;
    const int per_row = c.H * p.items;
    const int64_t pf = part_floats(p.heads, D);

    if ((int)blockIdx.x < js.y_blocks) {
        // ---- outputs: a unit is some query heads of one (row, key/value head) --------
        const int64_t units = (int64_t)c.B * c.H * js.units_per_bh;
        bool waited = false;
        for (int64_t u = blockIdx.x; u < units; u += js.y_blocks) {
            const int64_t bh = u / js.units_per_bh;
            const int b = (int)(bh / c.H), h = (int)(bh % c.H);
            const int g_begin = (int)(u % js.units_per_bh) * js.unit_heads;
            const int g_end = min(p.G, g_begin + js.unit_heads);
            const int64_t held = p.row_len[b];
            const bool live = held >= 0 && held <= c.capacity();
            if (held > c.capacity() && tid == 0) report(c.status, TC_ERR_DEVICE_BOUNDS);
            for (int g0 = g_begin; g0 < g_end && live; g0 += HB) {
                const int ng = min(HB, g_end - g0);
                const int64_t qh = (int64_t)b * p.Hq + h * p.G + g0;
                float mem[HB * D / kJoinThreads > 0 ? HB * D / kJoinThreads : 1];  // q A of this thread's outputs
#pragma unroll
                for (int x = 0; x < (int)(sizeof(mem) / 4); ++x) mem[x] = 0.f;
                if (p.g && !p.memo) {
                    __syncthreads();
                    for (int x = tid; x < ng * D; x += kJoinThreads)
                        s_q[x / D][x % D] = to_f32(reinterpret_cast<const T *>(p.q)[qh * D + x]);
                    __syncthreads();
                    const float4 *A4 = reinterpret_cast<const float4 *>(c.A + bh * D * D);
                    const int cg = tid % CG, rg = tid / CG;
                    float4 acc[HB];
#pragma unroll
                    for (int g = 0; g < HB; ++g) acc[g] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                    for (int r = rg; r < D; r += RG) {
                        const float4 a = A4[r * CG + cg];
#pragma unroll
                        for (int g = 0; g < HB; ++g) {
                            const float w = g < ng ? s_q[g][r] : 0.f;
                            acc[g].x = fmaf(w, a.x, acc[g].x);
                            acc[g].y = fmaf(w, a.y, acc[g].y);
                            acc[g].z = fmaf(w, a.z, acc[g].z);
                            acc[g].w = fmaf(w, a.w, acc[g].w);
                        }
                    }
#pragma unroll
                    for (int g = 0; g < HB; ++g) reinterpret_cast<float4 *>(&s_red[rg][g][0])[cg] = acc[g];
                    __syncthreads();
#pragma unroll
                    for (int x = 0; x < (int)(sizeof(mem) / 4); ++x) {
                        const int i = tid + x * kJoinThreads;
                        if (i < ng * D)
                            for (int r = 0; r < RG; ++r) mem[x] += s_red[r][i / D][i % D];
                    }
                }
                if (!waited) {
                    griddep_wait();
                    waited = true;
                }
                if (p.memo) {
#pragma unroll
                    for (int x = 0; x < (int)(sizeof(mem) / 4); ++x) {
                        const int i = tid + x * kJoinThreads;
                        if (i < ng * D)
                            for (int r = 0; r < p.slices; ++r)
                                mem[x] += p.memo[((bh * p.slices + r) * p.G + g0) * D + i];
                    }
                }
                const int64_t tiles = (held + kTile - 1) / kTile;
                const int64_t total = p.prefix[c.B] * per_row;
                const int64_t G = total < js.split_grid ? total : js.split_grid;
                for (int g = 0; g < ng; ++g) {
                    const int grp = (g0 + g) / p.heads, hh = (g0 + g) % p.heads;
                    const int64_t item = (int64_t)b * per_row + h * p.items + grp;
                    float sum = 0.f, L = 0.f;
                    const int d = tid % D, dg = tid / D;
                    if (tiles > 0) {
                        const int64_t u0 = p.prefix[b] * per_row + ((int64_t)h * p.items + grp) * tiles;
                        const Parts ps(u0, u0 + tiles, total, G);
                        const int64_t np = ps.last - ps.first + 1;
                        float M = -INFINITY;
                        for (int64_t i = 0; i < np; ++i) M = fmaxf(M, p.part[(ps.first + i + item) * pf + p.heads * D + 2 * hh]);
                        if (M == -INFINITY) M = 0.f;
                        for (int64_t i = dg; i < np; i += DG) {
                            const float *part = p.part + (ps.first + i + item) * pf;
                            const float w = ex2(part[p.heads * D + 2 * hh] - M);
                            sum = fmaf(w, part[hh * D + d], sum);
                            L = fmaf(w, part[p.heads * D + 2 * hh + 1], L);
                        }
                    }
                    __syncthreads();
                    red[tid] = sum;  // [DG][D]
                    if (d == 0) s_w[dg] = L;
                    __syncthreads();
                    // outputs of head g belong to threads of index i = g D + d
#pragma unroll
                    for (int x = 0; x < (int)(sizeof(mem) / 4); ++x) {
                        const int i = tid + x * kJoinThreads;
                        if (i / D == g) {
                            float num = 0.f, den = 0.f;
                            for (int r = 0; r < DG; ++r) {
                                num += red[r * D + i % D];
                                den += s_w[r];
                            }
                            float y = den == 0.f ? 0.f : num / den;  // no pair, or none that counts
                            if (p.g) y = fmaf(sigmoidf_acc(p.g[h * p.G + g0 + g]), mem[x], y);
                            reinterpret_cast<T *>(p.y)[qh * D + i] = from_f32<T>(y);
                        }
                    }
                }
                __syncthreads();
            }
        }
        if (!waited) griddep_wait();
        if (p.step && blockIdx.x == 0) {
            // the step's rows, once every kernel that reads them by the old
            // values is done: len is no longer read (row_len stands for it)
            for (int b = tid; b < c.B; b += kJoinThreads)
                if (p.row_len[b] >= 0) {
                    c.len[b] = p.row_len[b];
                    c.clock[b] += 1;
                }
        }
        return;
    }

    // ---- weights: this block's share of the tiles of every (row, key/value head) -----
    griddep_wait();
    const int64_t mb = blockIdx.x - js.y_blocks, all = p.prefix[c.B] * c.H;
    const int64_t total = p.prefix[c.B] * per_row;
    const int64_t G = total < js.split_grid ? total : js.split_grid;
    int64_t u = mb * all / js.mass_blocks;
    const int64_t u_end = (mb + 1) * all / js.mass_blocks;
    if (u >= u_end) return;
    if (tid == 0) {
        int lo = 0, hi = c.B - 1;  // the last row that begins at or before u
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (p.prefix[mid] * c.H <= u) lo = mid;
            else hi = mid - 1;
        }
        s_row = lo;
    }
    __syncthreads();
    int b = s_row;
    while (u < u_end) {
        while (p.prefix[b + 1] * c.H <= u) ++b;
        const int64_t tiles = p.prefix[b + 1] - p.prefix[b], off = u - p.prefix[b] * c.H;
        const int h = (int)(off / tiles);
        const int64_t tile = off % tiles, stop = min(tiles, tile + (u_end - u));
        const int64_t held = row_pairs(p, b);
        // the softmax's maximum and sum of every head of the group, joined
        __syncthreads();
        for (int g = warp; g < p.G; g += kJoinThreads / 32) {
            const int grp = g / p.heads, hh = g % p.heads;
            const int64_t item = (int64_t)b * per_row + h * p.items + grp;
            const int64_t u0 = p.prefix[b] * per_row + ((int64_t)h * p.items + grp) * tiles;
            const Parts ps(u0, u0 + tiles, total, G);
            float M = -INFINITY, L = 0.f;
            for (int64_t i = ps.first + lane; i <= ps.last; i += 32) M = fmaxf(M, p.part[(i + item) * pf + p.heads * D + 2 * hh]);
#pragma unroll
            for (int o = 16; o > 0; o /= 2) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
            if (M == -INFINITY) M = 0.f;
            for (int64_t i = ps.first + lane; i <= ps.last; i += 32) {
                const float *ml = p.part + (i + item) * pf + p.heads * D + 2 * hh;
                L = fmaf(ex2(ml[0] - M), ml[1], L);
            }
#pragma unroll
            for (int o = 16; o > 0; o /= 2) L += __shfl_xor_sync(0xffffffffu, L, o);
            if (lane == 0) {
                s_w[g] = M;
                s_x[g] = L == 0.f ? 0.f : 1.f / L;
            }
        }
        __syncthreads();
        const int64_t j_end = min(held, stop * kTile);
        for (int64_t j = tile * kTile + tid; j < j_end; j += kJoinThreads) {
            const int pg = c.table[(int64_t)b * c.max_pages + j / c.page];
            if (!page_ok(c, pg)) continue;
            const int64_t row = pool_row(c, pg, h, (int)(j % c.page));
            float w = 0.f;
            for (int g = 0; g < p.G; ++g) w = fmaf(ex2(p.z[row * p.G + g] - s_w[g]), s_x[g], w);
            c.mass[row] += w;
        }
        u += stop - tile;
    }
}

// ---- host -------------------------------------------------------------------------

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The pool as rows of d bf16; boxes of 16 rows, at most 64 columns.
bool make_pool_map(CUtensorMap *m, const void *base, int64_t rows, int d) {
    EncodeTiled fn = reinterpret_cast<EncodeTiled>(tensor_map_encoder());
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)d * 2};
    const cuuint32_t box[2] = {(cuuint32_t)(d < 64 ? d : 64), (cuuint32_t)kWarpPairs};
    const cuuint32_t es[2] = {1, 1};
    const CUtensorMapSwizzle sw = d >= 64 ? CU_TENSOR_MAP_SWIZZLE_128B : d == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B;
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Resident blocks of a kernel over the device, at most attend_grid's bound.
template <typename K>
cudaError_t fill_grid(K kernel, int smem, int num_sms, int *grid) {
    cudaError_t e = smem > 0 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) : cudaSuccess;
    if (e != cudaSuccess) return e;
    int per_sm = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, smem);
    if (e != cudaSuccess) return e;
    const int most = attend_grid(num_sms);
    *grid = per_sm * num_sms < most ? per_sm * num_sms : most;
    return *grid > 0 ? cudaSuccess : cudaErrorInvalidConfiguration;
}

cudaLaunchConfig_t early_launch(cudaLaunchAttribute *attr, int grid, int threads, int smem, cudaStream_t s, bool early) {
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = early ? 1 : 0;
    return cfg;
}

template <int D, int NT>
cudaError_t split_bf16(const AttendParams &p, int num_sms, int *grid, cudaStream_t s) {
    CUtensorMap mk, mv;
    const int64_t rows = (int64_t)p.c.n_pages * p.c.H * p.c.page;
    if (!make_pool_map(&mk, p.c.k, rows, D) || !make_pool_map(&mv, p.c.v, rows, D)) return cudaErrorInvalidValue;
    cudaError_t e = fill_grid(attend_bf16_kernel<D, NT>, Bf16Shape<D, NT>::SMEM, num_sms, grid);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = early_launch(&attr, *grid, kThreads, Bf16Shape<D, NT>::SMEM, s, p.step);
    return cudaLaunchKernelEx(&cfg, attend_bf16_kernel<D, NT>, mk, mv, p);
}

template <int D, int GT>
cudaError_t split_f32(const AttendParams &p, int num_sms, int *grid, cudaStream_t s) {
    cudaError_t e = fill_grid(attend_f32_kernel<D, GT>, 0, num_sms, grid);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = early_launch(&attr, *grid, kThreads, 0, s, p.step);
    return cudaLaunchKernelEx(&cfg, attend_f32_kernel<D, GT>, p);
}

template <int D>
cudaError_t launch_attend_d(const AttendParams &p, tc_dtype dtype, int num_sms, cudaStream_t s) {
    int grid = 0;
    cudaError_t e = cudaErrorInvalidValue;
    if (dtype == TC_BF16) {
        e = p.heads == 8 ? split_bf16<D, 1>(p, num_sms, &grid, s) : split_bf16<D, 2>(p, num_sms, &grid, s);
    } else {
        switch (p.heads) {
            case 1: e = split_f32<D, 1>(p, num_sms, &grid, s); break;
            case 2: e = split_f32<D, 2>(p, num_sms, &grid, s); break;
            case 4: e = split_f32<D, 4>(p, num_sms, &grid, s); break;
            case 8: e = split_f32<D, 8>(p, num_sms, &grid, s); break;
        }
    }
    if (e != cudaSuccess) return e;
    JoinShape js;
    js.split_grid = grid;
    // few (row, head) units: one query head each; else the whole group, so that
    // A is read once
    const int64_t BH = (int64_t)p.c.B * p.c.H;
    js.unit_heads = BH * 2 <= num_sms ? 1 : p.G;
    js.units_per_bh = (p.G + js.unit_heads - 1) / js.unit_heads;
    const int64_t units = BH * js.units_per_bh;
    js.y_blocks = (int)(units < 8 * num_sms ? units : 8 * num_sms);
    js.mass_blocks = p.z ? 2 * num_sms : 0;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = early_launch(&attr, js.y_blocks + js.mass_blocks, kJoinThreads, 0, s, true);
    return dtype == TC_BF16 ? cudaLaunchKernelEx(&cfg, attend_join_kernel<__nv_bfloat16, D>, p, js)
                            : cudaLaunchKernelEx(&cfg, attend_join_kernel<float, D>, p, js);
}

}  // namespace

// bf16: 8 heads fill a product; 16 share a pass over K and V when there are
// more than 8.  float32: a power of two up to 8, in registers.
int attend_heads_per_item(int G, tc_dtype dtype) {
    if (dtype == TC_BF16) return G <= 8 ? 8 : 16;
    return G <= 1 ? 1 : G <= 2 ? 2 : G <= 4 ? 4 : 8;
}

int attend_grid(int num_sms) { return 4 * num_sms; }

size_t attend_part_bytes(int64_t BH, int G, int d, tc_dtype dtype, int num_sms) {
    const int heads = attend_heads_per_item(G, dtype);
    const int64_t items = BH * ((G + heads - 1) / heads);
    return (size_t)(attend_grid(num_sms) + items) * (size_t)part_floats(heads, d) * sizeof(float);
}

bool attend_supported(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

cudaError_t launch_cache_attend(const AttendParams &p, tc_dtype dtype, int num_sms, cudaStream_t s) {
    switch (p.d) {
        case 16: return launch_attend_d<16>(p, dtype, num_sms, s);
        case 32: return launch_attend_d<32>(p, dtype, num_sms, s);
        case 64: return launch_attend_d<64>(p, dtype, num_sms, s);
        case 128: return launch_attend_d<128>(p, dtype, num_sms, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace tc

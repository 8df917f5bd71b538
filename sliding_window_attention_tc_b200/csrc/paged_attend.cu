// tc_cache_attend: one new token's attention over a paged cache, fused with
// the memory's read and with the accumulation of each pair's weight.
//
//   y_h = sum_j p_j v_j + sigmoid(g_h) q_h A,  p = softmax_j(<q_h,k_j>/sqrt(d))
//
// Bound by memory: every key and value is read once per group of query heads.
// The work, tiles of 128 pairs of one (row, key/value head, group of query
// heads), is laid end to end and cut into equal parts, one per block, wherever
// the rows begin and end: rows of any lengths keep every SM equally busy.  A
// block walks its part with a running maximum and sum; at the end of a row's
// stretch it stores the partial (m, l, O).  The join kernel adds the partials
// of each row's stretches, the memory's read, and (from the scores the first
// kernel left in the workspace) the weights.  Both kernels, 32 query heads over 8,
// d = 128, bf16: 64 rows of 2048 pairs 88 us, 6.1 TB/s; with the memory and the
// weights 104 us.
//
// bf16: a tile comes in by TMA (boxes of as many rows as always share a page;
// swizzled; one lane of a ninth warp a box) and each of eight warps takes 16 of
// its pairs, with running statistics of its own: no barrier between warps until
// a row's stretch ends.  Products run as S^T = K Q^T (16 pairs x 8 heads) and
// O^T = V^T P^T with m16n8k16: with the pairs as M, eight heads fill a product
// that would be half empty with the heads as M, and the same lanes hold a
// head's scores and its outputs, so rescaling needs no exchange.  P enters as a
// bf16 pair hi + lo (off by 2^-17 of a weight; a bf16 result is rounded by 2^-8).
// The tensor pipe is nowhere near busy (16 d multiply-adds a pair against 4 d
// bytes); a warp's chain score -> maximum -> weight -> output is what has to be
// hidden, by the other warps and the loads in flight.  (Four warps of 32 pairs
// each took 2090 cycles a tile with the data at hand, where memory brings one in
// 2670.)
//
// float32: the same walk with float32 multiply-adds, d/4 lanes per pair.

#include <cuda.h>

#include <atomic>

#include "paged_cache.cuh"
#include "sm100_ptx.cuh"

namespace tc {
namespace {

using namespace sm100;

constexpr int kTile = 128;       // pairs per tile
constexpr int kRun = 16;         // pairs that always share a page
constexpr int kRuns = kTile / kRun;
constexpr int kExtra = 1;        // tiles' worth of work that a row's item costs besides its tiles
constexpr int kJoinThreads = 256;

__device__ __forceinline__ int64_t row_pairs(const AttendParams &p, int b) {
    const int64_t n = p.row_len[b];
    return n < 0 || n > p.c.capacity() ? 0 : n;
}
// Units of work of one item of row b: its tiles and, where it has any, kExtra
// that stand for what a stretch costs by itself (its queries, its partials).
__device__ __forceinline__ int row_units(const AttendParams &p, int b) {
    const int tiles = (int)((row_pairs(p, b) + kTile - 1) / kTile);
    return tiles ? tiles + kExtra : 0;
}

// A place in the laid-out work, and the stretch of tiles from there on that
// belongs to one (row, item): tiles tile .. tile + count - 1 of it are this
// block's (none when only the units that stand for no tile are).
struct Cursor {
    int left;      // units until the end of the part, from the stretch's first
    int b, item;   // row, item of it
    int tile, tiles;  // first tile, tiles an item of the row has
    int units;     // of the stretch
    int count;     // tiles of it
    int n;         // pairs of row b

    __device__ __forceinline__ void enter_row(const AttendParams &p) {
        n = (int)row_pairs(p, b);
        tiles = (n + kTile - 1) / kTile;
    }
    __device__ __forceinline__ void measure() {
        units = min(tiles + kExtra - tile, left);
        count = max(0, min(tiles - tile, left));
    }
    // on to the next stretch; false at the part's end
    __device__ __forceinline__ bool next(const AttendParams &p, int per_row) {
        left -= units;
        if (left == 0) return false;
        tile = 0;
        if (++item == per_row) {
            item = 0;
            do {
                ++b;
                enter_row(p);
            } while (tiles == 0);  // left > 0: a row with tiles follows
        }
        measure();
        return true;
    }
    // to the first stretch that has tiles; false when the part has none
    __device__ __forceinline__ bool settle(const AttendParams &p, int per_row) {
        while (count == 0)
            if (!next(p, per_row)) return false;
        return true;
    }
};

// total units cut over G = min(grid, total) blocks: the first `more` of them
// have per + 1, the others per.  (Units fit 31 bits: checked on the host.)
struct Cut {
    uint32_t G, per, more;
    __device__ __forceinline__ Cut(uint32_t total, uint32_t grid) {
        G = total < grid ? total : grid;
        per = G ? total / G : 0;
        more = total - per * G;
    }
    __device__ __forceinline__ uint32_t begin(uint32_t block) const { return block * per + min(block, more); }
    // the block that has unit u
    __device__ __forceinline__ uint32_t block_of(uint32_t u) const {
        const uint32_t x = more * (per + 1);
        return u < x ? u / (per + 1) : more + (u - x) / per;
    }
};

// This block's part of the per_row * (units of all rows) units.  Every block
// adds up the rows' units by itself; block 0 also stores them (prefix) for the
// join.  Returns false when there is nothing to do.  Block-wide; WARPS warps.
template <int WARPS>
__device__ __forceinline__ bool find_part(const AttendParams &p, int per_row, Cursor &cur) {
    __shared__ int s_sum[WARPS];
    __shared__ int s_off, s_row;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = p.c.B;
    const int per = (B + WARPS * 32 - 1) / (WARPS * 32);
    const int b0 = tid * per, b1 = min(B, b0 + per);
    int mine = 0;
    for (int b = b0; b < b1; ++b) mine += row_units(p, b);
    int v = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    if (lane == 31) s_sum[warp] = v;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += s_sum[w];
        all += s_sum[w];
    }
    before += v - mine;
    if (blockIdx.x == 0) {
        int x = before;
        for (int b = b0; b < b1; ++b) {
            p.prefix[b] = x;
            x += row_units(p, b);
        }
        if (tid == 0) p.prefix[B] = all;
    }
    const Cut cut((uint32_t)all * per_row, gridDim.x);
    if (blockIdx.x >= cut.G) return false;
    const int u0 = (int)cut.begin(blockIdx.x), u1 = (int)cut.begin(blockIdx.x + 1);
    if (u0 >= before * per_row && u0 < (before + mine) * per_row) {
        int x = before, b = b0;
        for (;; ++b) {
            const int t = row_units(p, b);
            if (u0 < (x + t) * per_row) break;
            x += t;
        }
        s_row = b;
        s_off = u0 - x * per_row;
    }
    __syncthreads();
    cur.b = s_row;
    cur.enter_row(p);
    cur.item = s_off / (cur.tiles + kExtra);
    cur.tile = s_off - cur.item * (cur.tiles + kExtra);
    cur.left = u1 - u0;
    cur.measure();
    return cur.settle(p, per_row);
}

// Partial results: the slot of (block, item) is block + item's number, which
// grows by at least one along the work, so no two share one.  O [heads][d],
// then (m, l) per head, in whole 16-byte vectors.
__host__ __device__ inline int64_t part_floats(int heads, int d) { return ((int64_t)heads * (d + 2) + 3) / 4 * 4; }

// ---- bf16 -----------------------------------------------------------------------

constexpr int kBWarps = kRuns;               // warps that compute: one run of a tile each
constexpr int kBThreads = kBWarps * 32;

// A tile of d bf16 in shared memory: boxes of at most 64 columns, in each the
// rows one after the other, swizzled as TMA does it with the widest pattern a
// row allows.  lane_offset is the place of (row r, 16-byte chunk hi); k-step k
// (chunk 2k + hi) lies at that place with k's low bits flipped in, because the
// swizzle is an exclusive or.
template <int D>
struct TileLayout {
    static constexpr int RB = D >= 64 ? 128 : D * 2;   // bytes of a box row
    static constexpr int BOX = kTile * RB;             // bytes of a box
    static constexpr int KPB = RB / 32;                // k-steps of a box
    __device__ __forceinline__ static uint32_t lane_offset(int r, int hi) {
        const int x = RB == 128 ? (r & 7) : RB == 64 ? ((r >> 1) & 3) : ((r >> 2) & 1);
        return r * RB + ((hi ^ x) << 4);
    }
    __device__ __forceinline__ static uint32_t at(uint32_t lane, int k) {
        return (lane ^ ((k % KPB) << 5)) + (k / KPB) * BOX;
    }
};

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
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int x, int y, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, %4}], [%2], "
        "%5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "l"(policy)
        : "memory");
}

template <int D, int NT>
struct Bf16Shape {
    static constexpr int STAGES = D >= 64 ? 3 : 4;
    static constexpr int STAGE_BYTES = kTile * D * 2 * 2;  // a tile's keys and values
    static constexpr int HEADS = 8 * NT;
    static constexpr int OS = D + 4;                       // floats between heads of a warp's outputs
    static constexpr int SUMS = NT == 1 ? 4 : 2;           // buffers the warps' outputs are added in
    static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + SUMS * HEADS * OS * 4;
};

// What a stage holds of a run: its pool row and its pairs (0: not loaded).
struct RunNote {
    int row, pairs;
};

template <int D, int NT>
__global__ void __launch_bounds__(kBThreads + 32) attend_bf16_kernel(const __grid_constant__ CUtensorMap map_k,
                                                                     const __grid_constant__ CUtensorMap map_v,
                                                                     const __grid_constant__ AttendParams p, int box_rows) {
    using S = Bf16Shape<D, NT>;
    using L = TileLayout<D>;
    constexpr int KS = D / 16;      // k-steps of a score, 16-wide blocks of the output
    extern __shared__ unsigned char dyn[];
    __shared__ __align__(8) uint64_t s_full[S::STAGES], s_free[S::STAGES];
    __shared__ RunNote s_note[S::STAGES][kRuns];
    __shared__ float s_m[kBWarps][S::HEADS], s_l[kBWarps][S::HEADS];
    __shared__ int s_abort;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int boxes = kTile / box_rows;  // of rows; one lane brings in each
    if (tid == 0) {
        for (int s = 0; s < S::STAGES; ++s) {
            mbar_init(&s_full[s], boxes);
            mbar_init(&s_free[s], kBWarps);
        }
        s_abort = 0;
        fence_mbar_init();
    }
    if (tid == kBThreads) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_k) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_v) : "memory");
    }
    griddep_wait();
    griddep_launch_dependents();
    const int per_row = p.c.H * p.items;
    Cursor cur;
    if (!find_part<kBWarps + 1>(p, per_row, cur)) return;  // its barriers also publish the mbarriers

    const uint32_t ring = (smem_u32(dyn) + 1023u) & ~1023u;
    if (warp == kBWarps) {
        // ---- loads: a lane per box of rows ------------------------------------------------
        if (lane >= boxes) return;
        const int runs = box_rows / kRun, row0 = lane * box_rows;
        int page = -1;  // table entry, fetched a tile early
        int j = cur.tile * kTile + row0, left = cur.count;
        const int32_t *table = p.c.table + (int64_t)cur.b * p.c.max_pages;
        int head = (cur.item / p.items) * p.c.page;
        const int step = p.c.H * p.c.page;
        if (j < cur.n) page = table[p.c.page_of(j)];
        // keys and values are read once: they are the first to leave L2, so that
        // the scores stay for the join
        uint64_t policy;
        asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
        int st = 0;
        uint32_t round = 0;  // times the ring went around
        for (bool more = true; more;) {
            if (round > 0 && !mbar_wait(&s_free[st], (round - 1) & 1u, &s_abort, p.c.status, p.wait_ns)) break;
            int n = max(0, min(box_rows, cur.n - j));
            if (n && !page_ok(p.c, page)) {
                report(p.c.status, TC_ERR_DEVICE_BOUNDS);
                n = 0;
            }
            const int row = page * step + head + j - p.c.page_of(j) * p.c.page;
            for (int i = 0; i < runs; ++i)
                s_note[st][lane * runs + i] = RunNote{row + i * kRun, max(0, min(kRun, n - i * kRun))};
            uint64_t *bar = &s_full[st];
            if (n) {
                mbar_expect_tx(bar, (uint32_t)box_rows * D * 4);
                const uint32_t dst = ring + st * S::STAGE_BYTES + row0 * L::RB;
#pragma unroll
                for (int x = 0; x * L::RB < D * 2; ++x) {
                    tma_load_2d(dst + x * L::BOX, &map_k, bar, x * 64, row, policy);
                    tma_load_2d(dst + S::STAGE_BYTES / 2 + x * L::BOX, &map_v, bar, x * 64, row, policy);
                }
            } else {
                mbar_arrive(bar);
            }
            j += kTile;
            if (--left == 0) {
                more = cur.next(p, per_row) && cur.settle(p, per_row);
                j = cur.tile * kTile + row0;
                left = cur.count;
                table = p.c.table + (int64_t)cur.b * p.c.max_pages;
                head = (cur.item / p.items) * p.c.page;
            }
            if (more && j < cur.n) page = table[p.c.page_of(j)];
            if (++st == S::STAGES) {
                st = 0;
                ++round;
            }
        }
        // No copy may land once the block is gone, and whether a computing warp gave
        // up on one is not known here: the lanes stay until all have landed.  A lane
        // whose wait ran out is at most one use of a stage behind the others (the
        // next use waits for the computing warps, and they for this lane); it
        // arrives for that one, so that the phase the others wait for ends.  The
        // computing warps look at s_abort behind every wait and do not take the
        // stage for a loaded one.
        const uint32_t lanes = (1u << boxes) - 1u;
        __syncwarp(lanes);
        for (int s = 0; s < S::STAGES; ++s) {
            const uint32_t uses = round + (s < st ? 1 : 0), most = __reduce_max_sync(lanes, uses);
            if (uses < most) mbar_arrive(&s_full[s]);
            if (most) mbar_wait_drain(&s_full[s], (most - 1) & 1u);
        }
        return;
    }

    float *s_o = reinterpret_cast<float *>(dyn + (ring - smem_u32(dyn)) + S::STAGES * S::STAGE_BYTES);  // [SUMS][HEADS][OS]
    auto warps_sync = []() { asm volatile("bar.sync 1, %0;" ::"n"(kBThreads) : "memory"); };
    const float scale = rsqrtf((float)D) * 1.4426950408889634f;  // log2(e)/sqrt(d)
    const uint32_t k_lane = L::lane_offset(warp * kRun + (lane & 7) + ((lane >> 3) & 1) * 8, lane >> 4);
    const uint32_t v_lane = L::lane_offset(warp * kRun + (lane & 7) + (lane >> 4) * 8, (lane >> 3) & 1) + S::STAGE_BYTES / 2;
    const int c0 = (lane % 4) * 2, r0 = lane / 4;  // this lane's columns (heads) and first row (pair)
    uint32_t qf[NT][KS][2];
    auto load_q = [&]() {  // the queries of the cursor's stretch
        const int h = cur.item / p.items, grp = cur.item - h * p.items;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int hh = grp * S::HEADS + t * 8 + r0;
            const uint32_t *qp = reinterpret_cast<const uint32_t *>(p.q) + (((int64_t)cur.b * p.Hq + h * p.G + hh) * D + c0) / 2;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                qf[t][k][0] = hh < p.G ? qp[k * 8] : 0u;
                qf[t][k][1] = hh < p.G ? qp[k * 8 + 4] : 0u;
            }
        }
    };
    load_q();
    uint32_t parity = 0;  // of the ring's round
    bool dead = false;
    int st = 0;
    for (bool more = true; more;) {
        // ---- one stretch: tiles of one (row, head, group of query heads) -----------
        const int grp = cur.item - cur.item / p.items * p.items;
        const int heads = min(S::HEADS, p.G - grp * S::HEADS);
        const int64_t item = (int64_t)cur.b * per_row + cur.item;
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
        for (int i = 0; i < cur.count; ++i) {
            RunNote note{};
            if (!dead) {
                dead = !mbar_wait(&s_full[st], parity, &s_abort, p.c.status, p.wait_ns);
                note = s_note[st][warp];
                if (*const_cast<volatile int *>(&s_abort)) dead = true;  // a loading lane arrived without its rows
            }
            if (dead) break;
            if (note.pairs) {
                const uint32_t base = ring + st * S::STAGE_BYTES;
                // S^T = K Q^T, in two chains of products
                float sc[NT][2][4];
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[t][0][e] = sc[t][1][e] = 0.f;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t a[4];
                    ldsm_x4(base + L::at(k_lane, k), a);
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma16816(sc[t][k & 1], a, qf[t][k][0], qf[t][k][1]);
                }
                if (note.pairs < kRun) {
                    // values of slots behind the row's pairs may hold anything, and
                    // 0 * NaN is no 0: they are cleared
                    constexpr int VPR = D / 8;  // 16-byte vectors of a row
                    for (int x = lane; x < (kRun - note.pairs) * VPR; x += 32) {
                        const int r = note.pairs + x / VPR, v = x % VPR;
                        const uint32_t at = base + S::STAGE_BYTES / 2 + (v * 16 / L::RB) * L::BOX + (warp * kRun + r) * L::RB + v * 16 % L::RB;
                        asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(at), "r"(0) : "memory");
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                }
                uint32_t ph[NT][2], pl[NT][2];
                bool grew = false;
                float corr[NT][2];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    float z[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[e] = (sc[t][0][e] + sc[t][1][e]) * scale;
                    if (p.z) {
                        // the group's scores of a pair lie side by side
                        float *zr = p.z + ((int64_t)note.row + r0) * p.G + grp * S::HEADS + t * 8 + c0;
                        if (p.G % 2 == 0) {
                            if (t * 8 + c0 < heads) {
                                if (r0 < note.pairs) *reinterpret_cast<float2 *>(zr) = make_float2(z[0], z[1]);
                                if (r0 + 8 < note.pairs) *reinterpret_cast<float2 *>(zr + 8 * p.G) = make_float2(z[2], z[3]);
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (t * 8 + c0 + (e & 1) < heads && r0 + (e >> 1) * 8 < note.pairs)
                                    zr[(e & 1) + (e >> 1) * 8 * p.G] = z[e];
                        }
                    }
                    if (r0 >= note.pairs) z[0] = z[1] = -INFINITY;
                    if (r0 + 8 >= note.pairs) z[2] = z[3] = -INFINITY;
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
                    // P^T as a bf16 pair: hi cut off, lo the rest, so that both have the
                    // weight's sign.  A weight above zero has no lo of zero (the least
                    // bf16 instead, 2^-126): an infinite value then stays infinite in
                    // both products, where 0 * inf would make it NaN.
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        constexpr float least = 1.17549435e-38f;
                        const float x = z[2 * e], y = z[2 * e + 1];
                        const uint32_t hx = __float_as_uint(x) & 0xffff0000u, hy = __float_as_uint(y) & 0xffff0000u;
                        const float lx = fmaxf(x - __uint_as_float(hx), fminf(x, least));
                        const float ly = fmaxf(y - __uint_as_float(hy), fminf(y, least));
                        ph[t][e] = transpose8x8(__byte_perm(hx, hy, 0x7632));
                        pl[t][e] = transpose8x8(pack_bf16(lx, ly));
                    }
                }
                if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int k = 0; k < KS; ++k)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[t][k][e] *= corr[t][e & 1];
                }
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t a[4];
                    ldsm_x4_t(base + L::at(v_lane, k), a);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        mma16816(o[t][k], a, ph[t][0], ph[t][1]);
                        mma16816(o[t][k], a, pl[t][0], pl[t][1]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_free[st]);
            if (++st == S::STAGES) {
                st = 0;
                parity ^= 1u;
            }
        }
        // the next stretch's queries come in while this one's results are joined
        const int block = (int)blockIdx.x;
        more = cur.next(p, per_row) && cur.settle(p, per_row);
        if (more) load_q();
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
        warps_sync();
        // each warp scales its outputs to the common maximum; SUMS warps at a time add
        auto top = [&](int hh) {
            float mx = s_m[0][hh];
#pragma unroll
            for (int w = 1; w < kBWarps; ++w) mx = fmaxf(mx, s_m[w][hh]);
            return mx;
        };
        float f[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float mx = top(t * 8 + c0 + e);
                f[t][e] = ex2(m[t][e] - (mx == -INFINITY ? 0.f : mx));
            }
        float *so = s_o + (warp % S::SUMS) * S::HEADS * S::OS;
#pragma unroll
        for (int pass = 0; pass < kBWarps / S::SUMS; ++pass) {
            if (warp / S::SUMS == pass) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k = 0; k < KS; ++k)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float *x = so + (t * 8 + c0 + (e & 1)) * S::OS + k * 16 + r0 + (e >> 1) * 8;
                            const float val = o[t][k][e] * f[t][e & 1];
                            *x = pass == 0 ? val : *x + val;
                        }
            }
            warps_sync();
        }
        float *part = p.part + (block + item) * part_floats(S::HEADS, D);
        for (int x = tid; x < heads * D; x += kBThreads) {
            const int hh = x / D, dd = x % D;
            float sum = 0.f;
#pragma unroll
            for (int s = 0; s < S::SUMS; ++s) sum += s_o[(s * S::HEADS + hh) * S::OS + dd];
            part[x] = sum;
        }
        if (tid < heads) {
            const float mx = top(tid);
            float ls = 0.f;
#pragma unroll
            for (int w = 0; w < kBWarps; ++w) ls += s_l[w][tid] * ex2(s_m[w][tid] - (mx == -INFINITY ? 0.f : mx));
            part[S::HEADS * D + 2 * tid] = mx;
            // after a wait that ran out the stretch may lack pairs: no sum is negative
            part[S::HEADS * D + 2 * tid + 1] = *const_cast<volatile int *>(&s_abort) ? -1.f : ls;
        }
        warps_sync();
    }
}

// ---- float32 ----------------------------------------------------------------------

constexpr int kFWarps = 4;
constexpr int kFThreads = kFWarps * 32;
constexpr int kFPairs = kTile / kFWarps;  // pairs of a tile one warp takes

template <int D, int GT>
__global__ void __launch_bounds__(kFThreads) attend_f32_kernel(const __grid_constant__ AttendParams p) {
    constexpr int LPK = D / 4;                 // lanes per pair
    constexpr int KPW = 32 / LPK;              // pairs a warp loads at once
    constexpr int NG = kFWarps * KPW;           // groups of lanes with statistics of their own
    constexpr int BATCH = GT <= 2 ? 8 : 4;     // loads of keys in flight per lane (and of values)
    __shared__ float s_m[NG][GT], s_l[NG][GT];
    __shared__ __align__(16) float s_o[NG][GT][D];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int sub = lane / LPK, li = lane % LPK, grp_id = warp * KPW + sub;
    griddep_wait();
    griddep_launch_dependents();
    const int per_row = p.c.H * p.items;
    Cursor cur;
    if (!find_part<kFWarps>(p, per_row, cur)) return;
    const float scale = rsqrtf((float)D) * 1.4426950408889634f;
    const float *kpool = reinterpret_cast<const float *>(p.c.k), *vpool = reinterpret_cast<const float *>(p.c.v);
    bool more = true;
    while (more) {
        const int b = cur.b, h = cur.item / p.items, grp = cur.item - h * p.items;
        const int h0 = h * p.G + grp * GT, heads = min(GT, p.G - grp * GT);
        const int64_t item = (int64_t)b * per_row + cur.item;
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
        // the warp's 32 pairs of each tile, as two runs of 16 within a page
        for (int i2 = 0; i2 < 2 * cur.count; ++i2) {
            const int j0 = (cur.tile + i2 / 2) * kTile + warp * kFPairs + (i2 & 1) * kRun;
            int nv = max(0, min(kRun, cur.n - j0));
            int64_t row = 0;
            if (nv) {
                const int pi = p.c.page_of(j0), pg = p.c.table[(int64_t)b * p.c.max_pages + pi];
                if (page_ok(p.c, pg)) {
                    row = pool_row(p.c, pg, h, j0 - pi * p.c.page);
                } else {
                    nv = 0;
                    if (lane == 0) report(p.c.status, TC_ERR_DEVICE_BOUNDS);
                }
            }
#pragma unroll
            for (int u = 0; u < kRun / KPW; u += BATCH) {
                if (u * KPW >= nv) break;
                float4 k4[BATCH], v4[BATCH];
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int j = (u + i) * KPW + sub;
                    k4[i] = v4[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (u + i < kRun / KPW && j < nv) {
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
                        const bool in = u + i < kRun / KPW && j < nv;
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
        for (int x = tid; x < heads * D; x += kFThreads) {
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
        more = cur.next(p, per_row) && cur.settle(p, per_row);
    }
}

// ---- the join ---------------------------------------------------------------------

constexpr int kMassTiles = 16;    // tiles of a chunk of the weights
constexpr int kMassStats = 512;   // (tile, query head) statistics of a chunk

struct JoinShape {
    int y_blocks, unit_heads, units_per_bh;  // outputs: blocks, query heads a unit covers
    int mass_blocks;                         // weights: blocks (0: none)
    int split_grid;                          // blocks of the first kernel
};

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads, 4) attend_join_kernel(const __grid_constant__ AttendParams p,
                                                                   const __grid_constant__ JoinShape js) {
    constexpr int HB = 4;                     // query heads of a batch
    constexpr int CG = D / 4, RG = kJoinThreads / CG;
    constexpr int OUT = (HB * D + kJoinThreads - 1) / kJoinThreads;  // outputs per thread
    __shared__ __align__(16) float s_red[RG][HB][D];
    constexpr int WU = kTile / 32;            // pairs per lane in flight (weights)
    __shared__ float s_q[HB][D];
    __shared__ __align__(16) float s_m[kMassStats], s_l[kMassStats];
    __shared__ int s_b[kMassTiles], s_h[kMassTiles], s_t[kMassTiles], s_lost[kMassTiles];
    __shared__ int s_row[kMassTiles * (kTile / kRun)], s_nv[kMassTiles * (kTile / kRun)];
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
                float mem[OUT];  // q A of this thread's outputs, tid + x kJoinThreads
#pragma unroll
                for (int x = 0; x < OUT; ++x) mem[x] = 0.f;
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
                    for (int x = 0; x < OUT; ++x) {
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
                    for (int x = 0; x < OUT; ++x) {
                        const int i = tid + x * kJoinThreads;
                        if (i < ng * D)
                            for (int r = 0; r < p.slices; ++r) mem[x] += p.memo[((bh * p.slices + r) * p.G + g0) * D + i];
                    }
                }
                const int tiles = (int)((held + kTile - 1) / kTile);
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                float M = -INFINITY, L = 0.f;
                // every thread one float4 of one head, as many partials side by side as fit
                const int width = ng * CG, groups = kJoinThreads / width;
                const int e = tid % width, eg = e / CG, pg = tid / width;
                if (tiles > 0) {
                    const Cut cut((uint32_t)p.prefix[c.B] * per_row, js.split_grid);
                    const int grp = g0 / p.heads, hh = g0 % p.heads;  // a batch never crosses a group
                    const uint32_t u0 = (uint32_t)p.prefix[b] * per_row + (h * p.items + grp) * (tiles + kExtra);
                    const int p0 = (int)cut.block_of(u0), np = (int)cut.block_of(u0 + tiles - 1) - p0 + 1;
                    const float *part = p.part + (p0 + (int64_t)b * per_row + h * p.items + grp) * pf;
                    const float *ml = part + p.heads * D + 2 * (hh + eg);
                    const float *out = part + hh * D + 4 * e;
                    constexpr int U = 4;  // partials in flight per thread, their statistics with them
                    if (pg < groups)
                        for (int i0 = pg; i0 < np; i0 += U * groups) {
                            float2 v[U];
                            float4 o[U];
#pragma unroll
                            for (int k = 0; k < U; ++k) {
                                const int i = i0 + k * groups;
                                v[k] = make_float2(-INFINITY, 0.f);
                                o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                                if (i < np) {
                                    v[k] = *reinterpret_cast<const float2 *>(ml + i * pf);
                                    o[k] = *reinterpret_cast<const float4 *>(out + i * pf);
                                }
                            }
                            float mx = M;
#pragma unroll
                            for (int k = 0; k < U; ++k) mx = fmaxf(mx, v[k].x);
                            const float ref = mx == -INFINITY ? 0.f : mx, c0 = ex2(M - ref);
                            M = mx;
                            L *= c0;
                            acc.x *= c0;
                            acc.y *= c0;
                            acc.z *= c0;
                            acc.w *= c0;
#pragma unroll
                            for (int k = 0; k < U; ++k) {
                                const float f = ex2(v[k].x - ref);
                                L = fmaf(f, v[k].y, L);
                                acc.x = fmaf(f, o[k].x, acc.x);
                                acc.y = fmaf(f, o[k].y, acc.y);
                                acc.z = fmaf(f, o[k].z, acc.z);
                                acc.w = fmaf(f, o[k].w, acc.w);
                            }
                        }
                }
                __syncthreads();
                float *red = &s_red[0][0][0];  // [groups][ng D]
                if (pg < groups) {
                    reinterpret_cast<float4 *>(red)[tid] = acc;
                    if (e % CG == 0) {
                        s_m[pg * ng + eg] = M;
                        s_l[pg * ng + eg] = L;
                    }
                }
                __syncthreads();
#pragma unroll
                for (int x = 0; x < OUT; ++x) {
                    const int i = tid + x * kJoinThreads;
                    if (i < ng * D) {
                        const int g = i / D;
                        float top = -INFINITY, weight = 0.f, y = 0.f;
                        for (int r = 0; r < groups; ++r) top = fmaxf(top, s_m[r * ng + g]);
                        if (top == -INFINITY) top = 0.f;
                        for (int r = 0; r < groups; ++r) {
                            const float f = ex2(s_m[r * ng + g] - top);
                            weight = fmaf(f, s_l[r * ng + g], weight);
                            y = fmaf(f, red[r * ng * D + i], y);
                        }
                        y = weight == 0.f ? 0.f : y / weight;  // no pair that counts: the memory alone
                        if (p.g) y = fmaf(sigmoidf_acc(p.g[h * p.G + g0 + i / D]), mem[x], y);
                        reinterpret_cast<T *>(p.y)[qh * D + i] = from_f32<T>(y);
                    }
                }
                __syncthreads();
            }
        }
        if (!waited) griddep_wait();
        if (p.step && blockIdx.x == 0) {
            // the step's rows: lengths and clocks, which the step's first kernel
            // read and nothing after it does (row_len stands for them)
            for (int b = tid; b < c.B; b += kJoinThreads)
                if (p.row_len[b] >= 0) {
                    c.len[b] = p.row_len[b];
                    c.clock[b] += 1;
                }
        }
        return;
    }

    // ---- weights: this block's share of the tiles of every (row, key/value head) -----
    // A chunk of tiles at a time: which (row, head) each belongs to, the
    // joined maximum and sum of every query head of each, then the pairs.
    griddep_wait();
    int *s_pre = reinterpret_cast<int *>(&s_red[0][0][0]);  // rows' prefix, where it fits
    const uint32_t all = (uint32_t)p.prefix[c.B];
    const Cut cut(all * per_row, js.split_grid), mine(all * c.H, js.mass_blocks);
    const uint32_t mb = blockIdx.x - js.y_blocks;
    if (mb >= mine.G) return;
    int u = (int)mine.begin(mb);
    const int u_end = (int)mine.begin(mb + 1);
    const bool fits = c.B < (int)(sizeof(s_red) / 4);
    if (fits)
        for (int b = tid; b <= c.B; b += kJoinThreads) s_pre[b] = p.prefix[b];
    const int *pre = fits ? s_pre : p.prefix;
    const int most = min(kMassTiles, kMassStats / p.G);  // tiles of a chunk: each may be another (row, head)
    while (u < u_end) {
        const int nt = min(most, u_end - u);
        __syncthreads();
        if (tid < nt) {
            const int x = u + tid;
            int lo = 0, hi = c.B - 1;  // the last row that begins at or before x
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (pre[mid] * c.H <= x) lo = mid;
                else hi = mid - 1;
            }
            const int units = pre[lo + 1] - pre[lo], off = x - pre[lo] * c.H;
            s_b[tid] = lo;
            s_h[tid] = off / units;
            s_t[tid] = off - s_h[tid] * units;  // the last kExtra hold no pairs
            s_lost[tid] = 0;
        }
        __syncthreads();
        // pool row and pairs of every run of 16 (by the upper warps first: the lower
        // ones have the first statistics to fetch), its weights asked into L2
        for (int x = tid ^ (kJoinThreads / 2); x < nt * (kTile / kRun); x += kJoinThreads) {
            const int i = x / (kTile / kRun), b = s_b[i], j = s_t[i] * kTile + x % (kTile / kRun) * kRun;
            int nv = max(0, min(kRun, (int)row_pairs(p, b) - j)), row = 0;
            if (nv) {
                const int pi = c.page_of(j), pg = c.table[(int64_t)b * c.max_pages + pi];
                if (page_ok(c, pg)) {
                    row = (pg * c.H + s_h[i]) * c.page + j - pi * c.page;
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(c.mass + row));
                } else {
                    nv = 0;
                }
            }
            s_row[x] = row;
            s_nv[x] = nv;
        }
        // eight lanes per (tile, query head); tiles of one (row, head) share their first tile's
        for (int x0 = 0; x0 < nt * p.G; x0 += kJoinThreads / 8) {
            const int x = x0 + tid / 8, l8 = tid % 8;
            const int i = x < nt * p.G ? x / p.G : 0, g = x - i * p.G, b = s_b[i], h = s_h[i];
            const bool lead = x < nt * p.G && (i == 0 || s_t[i] == 0);
            float M = -INFINITY, L = 0.f;
            bool lost = false;  // a stretch of the row that a wait cut short
            if (lead) {
                const int units = pre[b + 1] - pre[b], tiles = units - kExtra, grp = g / p.heads, hh = g - grp * p.heads;
                const uint32_t u0 = (uint32_t)pre[b] * per_row + (h * p.items + grp) * units;
                const int p0 = (int)cut.block_of(u0), np = (int)cut.block_of(u0 + tiles - 1) - p0 + 1;
                const float *ml = p.part + (p0 + (int64_t)b * per_row + h * p.items + grp) * pf + p.heads * D + 2 * hh;
#pragma unroll 4
                for (int k = l8; k < np; k += 8) {
                    const float2 v = *reinterpret_cast<const float2 *>(ml + k * pf);
                    lost |= v.y < 0.f;
                    const float mx = fmaxf(M, v.x), ref = mx == -INFINITY ? 0.f : mx;
                    L = fmaf(L, ex2(M - ref), v.y * ex2(v.x - ref));
                    M = mx;
                }
            }
#pragma unroll
            for (int o = 4; o > 0; o /= 2) {
                const float m2 = __shfl_xor_sync(0xffffffffu, M, o), l2 = __shfl_xor_sync(0xffffffffu, L, o);
                const float mx = fmaxf(M, m2), ref = mx == -INFINITY ? 0.f : mx;
                L = L * ex2(M - ref) + l2 * ex2(m2 - ref);
                M = mx;
            }
            if (lost) s_lost[i] = 1;
            if (lead && l8 == 0) {
                s_m[x] = M == -INFINITY ? 0.f : M;
                s_l[x] = L == 0.f ? 0.f : 1.f / L;
            }
        }
        __syncthreads();
        // a warp per tile, WU pairs a lane: the statistics are the warp's
        for (int i = warp; i < nt; i += kJoinThreads / 32) {
            const int first = i - min(i, s_t[i]), stat = first * p.G;  // the (row, head)'s first tile of the chunk
            if (s_lost[first]) continue;  // not all of its scores are there: its weights stay as they are
            int row[WU];
            float w[WU], old[WU];
#pragma unroll
            for (int k = 0; k < WU; ++k) {
                const int x = k * 32 + lane, q = i * kRuns + x / kRun;
                row[k] = x % kRun < s_nv[q] ? s_row[q] + x % kRun : -1;
                w[k] = 0.f;
                if (row[k] >= 0) old[k] = c.mass[row[k]];
            }
            if (p.G % 4 == 0) {
                for (int g = 0; g < p.G; g += 4) {
                    float4 z[WU];
#pragma unroll
                    for (int k = 0; k < WU; ++k)
                        if (row[k] >= 0) z[k] = *reinterpret_cast<const float4 *>(p.z + (int64_t)row[k] * p.G + g);
                    const float4 m4 = *reinterpret_cast<const float4 *>(&s_m[stat + g]), l4 = *reinterpret_cast<const float4 *>(&s_l[stat + g]);
#pragma unroll
                    for (int k = 0; k < WU; ++k) {
                        w[k] = fmaf(ex2(z[k].x - m4.x), l4.x, w[k]);
                        w[k] = fmaf(ex2(z[k].y - m4.y), l4.y, w[k]);
                        w[k] = fmaf(ex2(z[k].z - m4.z), l4.z, w[k]);
                        w[k] = fmaf(ex2(z[k].w - m4.w), l4.w, w[k]);
                    }
                }
            } else {
                for (int g = 0; g < p.G; ++g) {
                    float z[WU];
#pragma unroll
                    for (int k = 0; k < WU; ++k)
                        if (row[k] >= 0) z[k] = p.z[(int64_t)row[k] * p.G + g];
                    const float m1 = s_m[stat + g], l1 = s_l[stat + g];
#pragma unroll
                    for (int k = 0; k < WU; ++k) w[k] = fmaf(ex2(z[k] - m1), l1, w[k]);
                }
            }
#pragma unroll
            for (int k = 0; k < WU; ++k)
                if (row[k] >= 0) c.mass[row[k]] = old[k] + w[k];
        }
        u += nt;
    }
}

// ---- host -------------------------------------------------------------------------

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The pool as rows of d bf16; boxes of at most 64 columns.
bool make_pool_map(CUtensorMap *m, const void *base, int64_t rows, int d, int box_rows) {
    EncodeTiled fn = reinterpret_cast<EncodeTiled>(tensor_map_encoder());
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)d * 2};
    const cuuint32_t box[2] = {(cuuint32_t)(d < 64 ? d : 64), (cuuint32_t)box_rows};
    const cuuint32_t es[2] = {1, 1};
    const CUtensorMapSwizzle sw = d >= 64 ? CU_TENSOR_MAP_SWIZZLE_128B : d == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B;
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Resident blocks of a kernel over the current device, at most attend_grid's
// bound.  Asked of the driver (and the shared memory granted) once per kernel
// and device: it takes longer than the launch.
struct ResidentGrid {
    static constexpr int kDevices = 64;
    std::atomic<int> per_sm[kDevices];
    template <typename K>
    cudaError_t get(K kernel, int threads, int smem, int num_sms, int *grid) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        int n = dev < kDevices ? per_sm[dev].load(std::memory_order_acquire) : 0;
        if (n == 0) {
            e = allow_smem(kernel, (size_t)smem);
            if (e != cudaSuccess) return e;
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, (size_t)smem);
            if (e != cudaSuccess) return e;
            if (n < 1) return cudaErrorInvalidConfiguration;
            if (dev < kDevices) per_sm[dev].store(n, std::memory_order_release);
        }
        const int most = attend_grid(num_sms);
        *grid = n * num_sms < most ? n * num_sms : most;
        return cudaSuccess;
    }
};

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
    // rows that always share a page: the fewer loads, the larger they are (16 rows of
    // 8000 pairs, 8 heads, d = 128, pages of 128: 86 us, in boxes of 16 rows 90)
    int box_rows = kRun;
    while (box_rows < kTile && p.c.page % (2 * box_rows) == 0) box_rows *= 2;
    if (!make_pool_map(&mk, p.c.k, rows, D, box_rows) || !make_pool_map(&mv, p.c.v, rows, D, box_rows))
        return cudaErrorInvalidValue;
    static ResidentGrid resident;
    cudaError_t e = resident.get(attend_bf16_kernel<D, NT>, kBThreads + 32, Bf16Shape<D, NT>::SMEM, num_sms, grid);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = early_launch(&attr, *grid, kBThreads + 32, Bf16Shape<D, NT>::SMEM, s, p.step);
    return cudaLaunchKernelEx(&cfg, attend_bf16_kernel<D, NT>, mk, mv, p, box_rows);
}

template <int D, int GT>
cudaError_t split_f32(const AttendParams &p, int num_sms, int *grid, cudaStream_t s) {
    static ResidentGrid resident;
    cudaError_t e = resident.get(attend_f32_kernel<D, GT>, kFThreads, 0, num_sms, grid);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = early_launch(&attr, *grid, kFThreads, 0, s, p.step);
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
    // A is read once (4 heads for 32 query heads, d = 128, one row of 131001 pairs:
    // the call takes 48 us, with whole groups 63; 64 rows of 2000, 8 heads for 64
    // query heads: 96 us, with single query heads 130)
    const int64_t BH = (int64_t)p.c.B * p.c.H;
    js.unit_heads = BH * 2 <= num_sms ? 1 : p.G;
    js.units_per_bh = (p.G + js.unit_heads - 1) / js.unit_heads;
    const int64_t units = BH * js.units_per_bh;
    js.y_blocks = (int)(units < 8 * num_sms ? units : 8 * num_sms);
    js.mass_blocks = p.z ? 4 * num_sms : 0;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = early_launch(&attr, js.y_blocks + js.mass_blocks, kJoinThreads, 0, s, true);
    return dtype == TC_BF16 ? cudaLaunchKernelEx(&cfg, attend_join_kernel<__nv_bfloat16, D>, p, js)
                            : cudaLaunchKernelEx(&cfg, attend_join_kernel<float, D>, p, js);
}

}  // namespace

// bf16: 8 heads fill a product; 16 share a pass over K and V when there are
// more than 8 (16 rows of 8000 pairs, 4 heads for 64, d = 128: 53 us, in two groups
// of 8 78).  float32: a power of two up to 8, in registers.
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

double attend_units(double items, int64_t capacity) { return items * (double)((capacity + kTile - 1) / kTile + kExtra); }

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

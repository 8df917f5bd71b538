// Insertion into, and eviction from, the paged cache.
//
// Insertion (tc_cache_append): new tokens' keys are rotated by their positions
// and stored with their values; queries are rotated beside them.  Bound by
// memory; one block owns some tokens of one row and walks the heads, so the
// angles are formed once per token.
//
// Eviction (tc_cache_evict, and the first kernel of tc_cache_step): with n
// pairs held and m = n - budget over, the m smallest by (protected, mass, pos)
// leave in that order, and
//   A <- lambda^m A + eta sum_i lambda^(m-1-i) k_i v_i^T.
// One cluster owns one (row, head); each of its blocks finds the same pairs on
// its own (no exchange) and writes its own slice of A's rows.  Rows of which
// one pair leaves (the steady state: an arg-min over the weights beside one
// pass over A, 8 d^2 bytes of A and 8 n of weights and positions) are the first
// kernel's; the second takes the rest (a sort, and products on the tensor
// cores) and stores the new lengths, which the first has to leave for its other
// blocks to read.

#include "paged_cache.cuh"
#include "sm100_ptx.cuh"

namespace tc {
namespace {

// ---- insertion ------------------------------------------------------------------

constexpr int kAppThreads = 256;

// Tokens row b appends, or -1 when the row is to be skipped (and not because
// it is empty: *bad says that an error has to be reported).  Block-wide.
__device__ __forceinline__ int64_t append_count(const AppendParams &p, int b, int64_t &len, int64_t &clock, bool &bad) {
    len = p.c.len[b];
    clock = p.c.clock[b];
    bad = false;
    if (len < 0) return -1;
    const int64_t n = p.counts ? p.counts[b] : p.T;
    bad = n < 0 || n > p.T || len + n > p.c.capacity() || len > p.c.capacity() || clock < 0 ||
          clock + n > (int64_t(1) << 31);
    if (!bad) bad = !block_pages_ok(p.c, b, len, len + n - 1);
    return bad ? -1 : n;
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kAppThreads) append_kernel(const __grid_constant__ AppendParams p, int chunks,
                                                             int tokens, int tiles, bool advance) {
    const int b = blockIdx.x / tiles;
    const int64_t t0 = (int64_t)(blockIdx.x % tiles) * tokens;
    int64_t len, clock;
    bool bad;
    const int64_t n = append_count(p, b, len, clock, bad);
    if (bad && threadIdx.x == 0) report(p.c.status, TC_ERR_DEVICE_BOUNDS);
    if (n < 0) return;
    const int H = p.c.H, d = p.d;
    const int chunk = threadIdx.x % chunks, r = threadIdx.x / chunks;
    const int hg = r / tokens, HG = kAppThreads / chunks / tokens;
    const int64_t t = t0 + r % tokens;
    if (t < n && hg < HG) {
        const int64_t slot = len + t, position = clock + t;
        const int pg = p.c.table[(int64_t)b * p.c.max_pages + slot / p.c.page];
        const int in_page = (int)(slot % p.c.page);
        RotChunk<VEC> rc;
        rc.place(p.table, chunk, d);
        rc.angles(p.table, chunk, position, false);
        // rows: the queries' heads, the keys', the values' (copied)
        const int rows = (p.q ? p.Hq : 0) + 2 * H, q_rows = p.q ? p.Hq : 0;
        for (int x = hg; x < rows; x += HG) {
            const T *src;
            T *dst;
            bool turn = true;
            if (x < q_rows) {
                src = reinterpret_cast<const T *>(p.q) + b * p.qs[0] + x * p.qs[1] + t * p.qs[2];
                dst = reinterpret_cast<T *>(p.q_out) + (((int64_t)b * p.Hq + x) * p.T + t) * d;
            } else {
                const bool value = x - q_rows >= H;
                const int h = x - q_rows - (value ? H : 0);
                const int64_t row = pool_row(p.c, pg, h, in_page);
                if (value) {
                    src = reinterpret_cast<const T *>(p.v) + b * p.vs[0] + h * p.vs[1] + t * p.vs[2];
                    dst = reinterpret_cast<T *>(p.c.v) + row * d;
                    turn = false;
                } else {
                    src = reinterpret_cast<const T *>(p.k) + b * p.ks[0] + h * p.ks[1] + t * p.ks[2];
                    dst = reinterpret_cast<T *>(p.c.k) + row * d;
                    if (chunk == 0) {
                        if (p.c.mass) p.c.mass[row] = p.mass_in ? p.mass_in[((int64_t)b * H + h) * p.T + t] : 0.f;
                        if (p.c.pos) p.c.pos[row] = (int32_t)position;
                    }
                }
            }
            float u[VEC], w[VEC];
            Row<T, VEC>::load(src + rc.a, u);
            if (rc.b >= 0) Row<T, VEC>::load(src + rc.b, w);
            if (turn) rc.turn(u, w);
            Row<T, VEC>::store(dst + rc.a, u);
            if (rc.b >= 0) Row<T, VEC>::store(dst + rc.b, w);
        }
    }
    if (advance) {  // this block is the row's only one
        __syncthreads();
        if (threadIdx.x == 0) {
            p.c.len[b] = len + n;
            p.c.clock[b] = clock + n;
        }
    }
}

__global__ void append_advance_kernel(const __grid_constant__ AppendParams p) {
    int64_t len, clock;
    bool bad;
    const int64_t n = append_count(p, blockIdx.x, len, clock, bad);
    __syncthreads();
    if (n > 0 && threadIdx.x == 0) {
        p.c.len[blockIdx.x] = len + n;
        p.c.clock[blockIdx.x] = clock + n;
    }
}

template <typename T, int VEC>
cudaError_t launch_append_vec(const AppendParams &p, cudaStream_t s) {
    const int chunks = (p.d + 2 * VEC - 1) / (2 * VEC);  // at most 64
    int tokens = 1;
    while (tokens < 8 && tokens < p.T && chunks * tokens * 2 <= kAppThreads) tokens *= 2;
    const int64_t tiles = (p.T + tokens - 1) / tokens;
    if ((int64_t)p.c.B * tiles > 0x7fffffffll) return cudaErrorInvalidValue;
    // a row that one block covers advances its own clock; else a second kernel
    // does, after every block has read it
    append_kernel<T, VEC><<<(unsigned)(p.c.B * tiles), kAppThreads, 0, s>>>(p, chunks, tokens, (int)tiles, tiles == 1);
    if (tiles > 1) append_advance_kernel<<<p.c.B, 128, 0, s>>>(p);
    return cudaGetLastError();
}

// ---- eviction -------------------------------------------------------------------

// The order in which pairs leave, as one number: unprotected first, then by
// weight (NaN last, -0 as 0), then by position.
__device__ __forceinline__ uint64_t leave_key(float mass, int32_t pos, int64_t protect_from) {
    uint32_t u = __float_as_uint(mass + 0.f);
    u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    if (mass != mass) u = 0xffffffffu;
    return ((uint64_t)(pos >= protect_from) << 63) | ((uint64_t)u << 31) | (uint32_t)(pos & 0x7fffffff);
}
__device__ __forceinline__ bool less_pair(uint64_t ka, uint32_t sa, uint64_t kb, uint32_t sb) {
    return ka < kb || (ka == kb && sa < sb);
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The row's pairs before the call's eviction (a step's new pair among them), or
// -1 for a row that is skipped (*bad: and reported).  Block-wide.
__device__ __forceinline__ int64_t evict_pairs(const EvictParams &p, bool step, int b, int64_t clock, bool &bad) {
    const int64_t held = p.c.len[b], n = held + (step ? 1 : 0);
    bad = false;
    if (held < 0) return -1;
    bad = held > p.c.capacity() || n > p.c.capacity() || (step && (clock < 0 || clock >= (int64_t(1) << 31)));
    if (!bad) bad = !block_pages_ok(p.c, b, 0, n - 1);
    return bad ? -1 : n;
}

// ---- at most one pair leaves (the steady state; the step's first kernel) ----------
//
// The slice of A comes in by one bulk copy while the weights are looked
// through, so it holds no registers; with d^2 / slices floats a block (32 KB at
// most) several blocks share an SM and cover one another's latencies, of which
// the chain length -> table -> weights -> pair -> A has many.
constexpr int kOneThreads = 256;
constexpr int kOneWarps = kOneThreads / 32;
constexpr int kQBatch = 4;    // query heads per pass over A
constexpr int kScanBatch = 4; // weights in flight per thread

template <typename T, int D, bool STEP>
__global__ void __launch_bounds__(kOneThreads) evict_one_kernel(const __grid_constant__ EvictParams p, int slices) {
    constexpr int CG = D / 4;              // float4 columns of A
    constexpr int RG = kOneThreads / CG;   // rows of A side by side
    extern __shared__ __align__(128) unsigned char dyn[];
    __shared__ __align__(16) float s_k[D], s_v[D];
    __shared__ float s_cos[D / 2 + 1], s_sin[D / 2 + 1];
    __shared__ uint64_t s_key[kOneWarps];
    __shared__ uint32_t s_slot[kOneWarps];
    __shared__ float s_q[kQBatch][D];
    __shared__ __align__(16) float s_mp[RG][kQBatch][D];
    __shared__ __align__(8) uint64_t s_bar;
    __shared__ int s_abort;

    const CacheParams &c = p.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = blockIdx.x % slices;
    const int64_t bh = blockIdx.x / slices;
    const int b = (int)(bh / c.H), h = (int)(bh % c.H);
    const int64_t clock0 = c.clock[b];
    const bool first = h == 0 && rank == 0 && tid == 0;
    const int rows = D / slices, row0 = rank * rows;
    const bool read = STEP && p.memo != nullptr;
    float4 *A4 = c.A ? reinterpret_cast<float4 *>(c.A + (bh * D + row0) * D) : nullptr;
    float4 *sA = reinterpret_cast<float4 *>(dyn);
    const int64_t expect = c.len[b] + (STEP ? 1 : 0);
    const bool copy = A4 && expect >= 0 && (read || expect > p.budget) && (STEP || expect - p.budget == 1);
    if (tid == 0) {
        s_abort = 0;
        sm100::mbar_init(&s_bar, 1);
        sm100::fence_mbar_init();
        if (copy) {
            sm100::mbar_expect_tx(&s_bar, (uint32_t)(rows * D * 4));
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                             sm100::smem_u32(dyn)),
                         "l"(A4), "r"(rows * D * 4), "r"(sm100::smem_u32(&s_bar))
                         : "memory");
        }
    }
    bool bad;
    const int64_t n64 = evict_pairs(p, STEP, b, clock0, bad);  // its barrier also publishes s_bar
    // a step lets one pair leave at most: a row above its budget stays above
    const int64_t over = n64 - p.budget;
    const int m = over <= 0 ? 0 : STEP ? 1 : over == 1 ? 1 : 0;
    const int n = (int)n64, keep = n - m;
    if (first) {
        if (bad) report(c.status, TC_ERR_DEVICE_BOUNDS);
        p.row_len[b] = n64 < 0 ? -1 : STEP ? keep : n64;
    }
    if (n64 < 0 || (m == 0 && !STEP)) {
        if (copy && tid == 0) sm100::mbar_wait_drain(&s_bar, 0);
        return;  // the whole cluster
    }
    const int32_t *table = c.table + (int64_t)b * c.max_pages;
    auto row_of = [&](int slot) {
        const int pg = c.page_of(slot);
        return pool_row(c, table[pg], h, slot - pg * c.page);
    };
    T *kp = reinterpret_cast<T *>(c.k), *vp = reinterpret_cast<T *>(c.v);
    const int G = STEP ? p.Hq / c.H : 0;

    if (STEP) {
        // the new pair enters slot n - 1 (every block of the cluster writes the
        // same values), the queries are rotated
        const RotaryTable &rt = p.table;
        for (int i = tid; i < rt.rot / 2; i += kOneThreads) rotary_angle(clock0, rt.inc[i], rt.gain, s_cos[i], s_sin[i]);
        __syncthreads();
        const int64_t row = row_of(n - 1);
        for (int x = tid; x < (G + 2) * D; x += kOneThreads) {
            const int which = x / D, i = x % D;
            if (which == G + 1) {
                vp[row * D + i] = reinterpret_cast<const T *>(p.v_new)[b * p.vs[0] + h * p.vs[1] + i];
                continue;
            }
            const T *src = which == G ? reinterpret_cast<const T *>(p.k_new) + b * p.ks[0] + h * p.ks[1]
                                      : reinterpret_cast<const T *>(p.q) + b * p.qs[0] + (h * G + which) * p.qs[1];
            float f = to_f32(src[i]);
            if (i < rt.rot) {
                const int half = rt.rot / 2;
                const int pair = rt.interleaved ? i / 2 : i < half ? i : i - half;
                const bool second = rt.interleaved ? (i & 1) : i >= half;
                const int other = rt.interleaved ? i ^ 1 : (second ? i - half : i + half);
                const float g = to_f32(src[other]);
                f = second ? g * s_sin[pair] + f * s_cos[pair] : f * s_cos[pair] - g * s_sin[pair];
            }
            if (which == G) kp[row * D + i] = from_f32<T>(f);
            else reinterpret_cast<T *>(p.q_rot)[(bh * G + which) * D + i] = from_f32<T>(f);
        }
        if (tid == 0) {
            c.mass[row] = 0.f;
            c.pos[row] = (int32_t)clock0;
        }
        __syncthreads();
    }

    int gone = 0;  // the slot that leaves
    if (m == 1) {
        const int64_t protect_from = clock0 + (STEP ? 1 : 0) - p.recent;
        uint64_t best = ~0ull;
        uint32_t slot = 0xffffffffu;
        for (int s0 = tid; s0 < n; s0 += kScanBatch * kOneThreads) {
            float w[kScanBatch];
            int32_t z[kScanBatch];
#pragma unroll
            for (int i = 0; i < kScanBatch; ++i) {
                const int s = s0 + i * kOneThreads;
                if (s < n) {
                    const int64_t row = row_of(s);
                    w[i] = c.mass[row];
                    z[i] = c.pos[row];
                }
            }
#pragma unroll
            for (int i = 0; i < kScanBatch; ++i) {
                const int s = s0 + i * kOneThreads;
                if (s < n) {
                    const uint64_t key = leave_key(w[i], z[i], protect_from);
                    if (less_pair(key, (uint32_t)s, best, slot)) {
                        best = key;
                        slot = (uint32_t)s;
                    }
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o /= 2) {
            const uint64_t k2 = __shfl_xor_sync(0xffffffffu, best, o);
            const uint32_t s2 = __shfl_xor_sync(0xffffffffu, slot, o);
            if (less_pair(k2, s2, best, slot)) {
                best = k2;
                slot = s2;
            }
        }
        if (lane == 0) {
            s_key[warp] = best;
            s_slot[warp] = slot;
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kOneWarps; ++w)
            if (w == 0 || less_pair(s_key[w], s_slot[w], best, slot)) {
                best = s_key[w];
                slot = s_slot[w];
            }
        gone = (int)slot;
    }

    if (copy) {
        const int cg = tid % CG, rg = tid / CG;
        const float lam = c.lam[h], eta = c.eta[h];
        if (m == 1) {
            const int64_t row = row_of(gone);
            for (int i = tid; i < 2 * D; i += kOneThreads) {
                if (i < D) s_k[i] = to_f32(kp[row * D + i]);
                else s_v[i - D] = to_f32(vp[row * D + i - D]);
            }
        }
        if (!sm100::mbar_wait(&s_bar, 0, &s_abort, c.status, p.wait_ns)) sm100::mbar_wait_drain(&s_bar, 0);
        __syncthreads();
        const float4 v4 = m == 1 ? reinterpret_cast<const float4 *>(s_v)[cg] : make_float4(0.f, 0.f, 0.f, 0.f);
        for (int g0 = 0; g0 == 0 || g0 < G; g0 += kQBatch) {
            const int ng = read ? min(kQBatch, G - g0) : 0;
            if (read) {
                for (int x = tid; x < kQBatch * rows; x += kOneThreads) {
                    const int g = x / rows, r = x - g * rows;
                    s_q[g][r] = g < ng ? to_f32(reinterpret_cast<const T *>(p.q_rot)[(bh * G + g0 + g) * D + row0 + r]) : 0.f;
                }
                __syncthreads();
            }
            float4 mp[kQBatch];
#pragma unroll
            for (int g = 0; g < kQBatch; ++g) mp[g] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int r = rg; r < rows; r += RG) {
                float4 a = sA[r * CG + cg];
                if (g0 == 0 && m == 1) {
                    const float ek = eta * s_k[row0 + r];
                    a.x = fmaf(lam, a.x, ek * v4.x);
                    a.y = fmaf(lam, a.y, ek * v4.y);
                    a.z = fmaf(lam, a.z, ek * v4.z);
                    a.w = fmaf(lam, a.w, ek * v4.w);
                    A4[r * CG + cg] = a;
                    if (G > kQBatch) sA[r * CG + cg] = a;
                }
                if (read) {
#pragma unroll
                    for (int g = 0; g < kQBatch; ++g) {
                        const float w = s_q[g][r];
                        mp[g].x = fmaf(w, a.x, mp[g].x);
                        mp[g].y = fmaf(w, a.y, mp[g].y);
                        mp[g].z = fmaf(w, a.z, mp[g].z);
                        mp[g].w = fmaf(w, a.w, mp[g].w);
                    }
                }
            }
            if (read) {
#pragma unroll
                for (int g = 0; g < kQBatch; ++g) reinterpret_cast<float4 *>(&s_mp[rg][g][0])[cg] = mp[g];
                __syncthreads();
                for (int x = tid; x < ng * D; x += kOneThreads) {
                    float sum = 0.f;
#pragma unroll
                    for (int r = 0; r < RG; ++r) sum += s_mp[r][x / D][x % D];
                    p.memo[((bh * slices + rank) * G + g0) * D + x] = sum;
                }
                __syncthreads();
            }
        }
    }
    if (m == 0) return;  // the whole cluster

    // the last pair moves to the freed slot, once every block of the cluster has
    // read what that overwrites
    if (slices > 1) cluster_sync();
    else __syncthreads();
    constexpr int LPR = D * (int)sizeof(T) / 16;  // 16-byte vectors of a row
    if (rank == 0 && gone < keep && tid < 2 * LPR) {
        const int64_t from = row_of(keep), to = row_of(gone);
        T *pool = tid < LPR ? kp : vp;
        const int i = tid < LPR ? tid : tid - LPR;
        reinterpret_cast<uint4 *>(pool + to * D)[i] = reinterpret_cast<const uint4 *>(pool + from * D)[i];
        if (tid == 0) {
            c.mass[to] = c.mass[from];
            c.pos[to] = c.pos[from];
        }
    }
}

// ---- several pairs leave ------------------------------------------------------------
//
// The slots are sorted by (protected, mass, pos) with a stable radix sort of 8
// bits a pass, in shared memory up to kSortMax pairs; passes whose digit is the
// same for every pair (most of the positions' and the protection's) are skipped.
// (A bitonic sort of 4096 keys with their slots took 139,000 cycles.)  The
// weighted sum runs on the tensor cores: tiles of TP pairs come in by
// asynchronous 16-byte copies, several in flight; the weighted keys
// lambda^(m-1-i) k_i are split into three bf16 parts (24 bits together; a
// float32 cache's values too), and the products' sums over one tile are added
// to float32 sums with the ordinary rounding, because the tensor cores' own
// accumulation truncates and would drift over thousands of pairs.  The blocks
// of a cluster take every SL-th tile and add their sums through one another's
// shared memory.
constexpr int kBulkThreads = 512;
constexpr int kBulkWarps = kBulkThreads / 32;
constexpr int kSortMax = 8192;   // pairs sorted in shared memory (16 bytes each)

// lambda^j for j >= 0 to float32's precision: the exponent in 64 bits, its
// fraction to exp2f.
struct Decay {
    double l2;
    bool negative, zero;
    __device__ __forceinline__ explicit Decay(float lam)
        : l2(lam == 0.f ? 0.0 : log2(fabs((double)lam))), negative(lam < 0.f), zero(lam == 0.f) {}
    __device__ __forceinline__ float pow(int64_t j) const {
        if (j == 0) return 1.f;
        if (zero) return 0.f;
        const double x = (double)j * l2, whole = rint(x);
        const int e = (int)fmax(-300.0, fmin(300.0, whole));
        const float r = ldexpf(exp2f((float)(x - whole)), e);
        return negative && (j & 1) ? -r : r;
    }
};

// Exclusive prefix of one count per thread over the block; *total the sum.
__device__ __forceinline__ int block_scan(int x, int *warp_sums, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int v = x;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kBulkWarps; ++w) {
        if (w < warp) before += warp_sums[w];
        all += warp_sums[w];
    }
    *total = all;
    return before + v - x;
}

// One stable pass of 8 bits: order b of n slots from order a by (key[slot] >>
// shift) & 255.  Each warp counts the digits of its share, the counts' prefix
// over (digit, warp) gives every element its place.  False (and b untouched)
// when all digits are the same.
__device__ bool radix_pass(const uint32_t *key, const uint32_t *a, uint32_t *b, int n, int shift, uint32_t *counts, int *scan) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int share = (n + kBulkWarps * 32 - 1) / (kBulkWarps * 32) * 32, i0 = warp * share, i1 = min(n, i0 + share);
    uint32_t *mine = counts + warp * 256;
    __syncthreads();
    for (int x = tid; x < kBulkWarps * 256; x += kBulkThreads) counts[x] = 0;
    __syncthreads();
    for (int i = i0 + lane; i < i0 + share; i += 32) {
        const uint32_t d = i < i1 ? (key[a[i]] >> shift) & 255u : 256u;
        const uint32_t same = __match_any_sync(0xffffffffu, d);
        if (d < 256u && (same & ((1u << lane) - 1u)) == 0) mine[d] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    int sum = 0, total;
    if (tid < 256) {
#pragma unroll
        for (int w = 0; w < kBulkWarps; ++w) sum += counts[w * 256 + tid];
    }
    if (__syncthreads_or(sum == n)) return false;
    int at = block_scan(sum, scan, &total);
    if (tid < 256) {
#pragma unroll
        for (int w = 0; w < kBulkWarps; ++w) {
            const int c = (int)counts[w * 256 + tid];
            counts[w * 256 + tid] = (uint32_t)at;
            at += c;
        }
    }
    __syncthreads();
    for (int i = i0 + lane; i < i0 + share; i += 32) {
        const uint32_t s = i < i1 ? a[i] : 0u;
        const uint32_t d = i < i1 ? (key[s] >> shift) & 255u : 256u;
        const uint32_t same = __match_any_sync(0xffffffffu, d);
        const uint32_t before = __popc(same & ((1u << lane) - 1u));
        const uint32_t base = d < 256u ? mine[d] : 0u;
        __syncwarp();
        if (d < 256u) {
            b[base + before] = s;
            if (before == 0) mine[d] = base + __popc(same);
        }
        __syncwarp();
    }
    __syncthreads();
    return true;
}

__device__ __forceinline__ void ldsm_t4(const void *p, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(sm100::smem_u32(p))
                 : "memory");
}
__device__ __forceinline__ void ldsm_t2(const void *p, uint32_t (&r)[2]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];"
                 : "=r"(r[0]), "=r"(r[1])
                 : "r"(sm100::smem_u32(p))
                 : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ void copy16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sm100::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void zero16(void *dst) { *reinterpret_cast<uint4 *>(dst) = make_uint4(0, 0, 0, 0); }

// x, y as three bf16 pairs whose sum is exact to 24 bits.
__device__ __forceinline__ void split3(float x, float y, uint32_t (&o)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        o[i] = pack_bf16_rn(x, y);
        const float hx = __uint_as_float(o[i] << 16), hy = __uint_as_float(o[i] & 0xffff0000u);
        x = isinf(hx) ? 0.f : x - hx;  // an infinity has no rest
        y = isinf(hy) ? 0.f : y - hy;
    }
}

// Shared memory of one block: the order of the pairs, then, one after the
// other in the same room, what sorting needs (keys, positions, a second order,
// counts), what the sum needs (raw tiles, parts; its result), and the lists of
// moves.
template <typename T, int D>
struct BulkShape {
    static constexpr int TP = sizeof(T) == 2 ? 64 : 32;     // pairs per tile
    static constexpr int STAGES = 3;
    static constexpr int VPARTS = sizeof(T) == 2 ? 0 : 3;   // bf16 values go in as they are
    static constexpr int KRAW = D * (int)sizeof(T);         // bytes of a raw row
    static constexpr int VRAW = D * (int)sizeof(T) + 16;    // padded: conflict-free reads by ldmatrix
    static constexpr int PS = D * 2 + 16;                   // bytes of a row of a part
    static constexpr int RAW = TP * (KRAW + VRAW);
    static constexpr int PARTS = TP * (3 + VPARTS) * PS;
    static constexpr int SUM = STAGES * RAW + PARTS;        // at least the result's 4 D^2
    // output tiles of 16 x 8: warps along the rows first
    static constexpr int TM = D / 16, TN = D / 8, NWN = kBulkWarps / TM;
    static constexpr int NT = TN / NWN > 0 ? TN / NWN : 1;  // tiles a warp holds
    static_assert(SUM >= 4 * D * D, "the block's sum has to fit");
};

// Bytes of sorting room for up to n pairs (a multiple of 32): keys, positions,
// second order; with the counts, and the first order, which stays.
__host__ __device__ constexpr size_t sort_room(size_t n) { return 12 * n + kBulkWarps * 256 * 4; }
__host__ __device__ constexpr size_t order_room(size_t n) { return (4 * n + n / 8 + 127) / 128 * 128; }  // and a bit per slot

template <typename T, int D, int SL>
__global__ void __launch_bounds__(kBulkThreads) evict_bulk_kernel(const __grid_constant__ EvictParams p, int n_cap) {
    using S = BulkShape<T, D>;
    extern __shared__ __align__(128) unsigned char dyn[];
    __shared__ int s_scan[kBulkWarps];
    __shared__ int s_row[S::STAGES + 1][S::TP];
    __shared__ float s_w[S::STAGES + 1][S::TP];

    const CacheParams &c = p.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = blockIdx.x % SL;
    const int64_t bh = blockIdx.x / SL;
    const int b = (int)(bh / c.H), h = (int)(bh % c.H);
    sm100::griddep_wait();
    const int64_t n64 = p.row_len[b];
    if (n64 <= p.budget) return;  // empty, skipped, or nothing to do: the whole cluster
    const int n = (int)n64, keep = (int)p.budget, m = n - keep;
    if (h == 0 && rank == 0 && tid == 0) c.len[b] = keep;  // read by no block of this kernel
    if (m == 1) return;
    const int32_t *table = c.table + (int64_t)b * c.max_pages;
    auto row_of = [&](int slot) {
        const int pg = c.page_of(slot);
        return (int)pool_row(c, table[pg], h, slot - pg * c.page);
    };
    T *kp = reinterpret_cast<T *>(c.k), *vp = reinterpret_cast<T *>(c.v);

    // ---- the order of leaving -----------------------------------------------------
    const bool inside = n <= n_cap;
    const size_t room = inside ? n_cap : n2_cap_global(c.capacity());
    unsigned char *kept = inside ? dyn : p.sort_ws + (bh * SL + rank) * (order_room(room) + sort_room(room));
    unsigned char *scratch = kept + order_room(room);     // sorting and lists
    unsigned char *tiles_mem = dyn + order_room(n_cap);   // the sum
    uint32_t *order = reinterpret_cast<uint32_t *>(kept), *bits = order + room;
    uint32_t *weight = reinterpret_cast<uint32_t *>(scratch), *place = weight + room, *other = place + room;
    uint32_t *counts = other + room;
    const int words = (n + 31) / 32;
    {
        const int64_t protect_from = c.clock[b] - p.recent;
        bool sorted = true;  // by position already, as tokens are appended
        uint32_t prot_any = 0, prot_all = 1;
        constexpr int U = 4;
        for (int s0 = tid; s0 < n; s0 += U * kBulkThreads) {
            float w[U];
            int32_t z[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int s = s0 + i * kBulkThreads;
                if (s < n) {
                    const int row = row_of(s);
                    w[i] = c.mass[row];
                    z[i] = c.pos[row];
                }
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int s = s0 + i * kBulkThreads;
                if (s < n) {
                    const uint64_t key = leave_key(w[i], z[i], protect_from);
                    weight[s] = (uint32_t)(key >> 31);
                    // the position, and above it the protection
                    place[s] = (uint32_t)(key & 0x7fffffffu) | (uint32_t)(key >> 63) << 31;
                    order[s] = s;
                    prot_any |= (uint32_t)(key >> 63);
                    prot_all &= (uint32_t)(key >> 63);
                }
            }
        }
        for (int s = tid; s < words; s += kBulkThreads) bits[s] = 0;
        __syncthreads();
        for (int s = tid; s + 1 < n; s += kBulkThreads)
            sorted = sorted && (place[s] & 0x7fffffffu) <= (place[s + 1] & 0x7fffffffu);
        const bool by_place = !__syncthreads_and(sorted);
        const bool split = __syncthreads_or(prot_any) && !__syncthreads_and(prot_all);
        uint32_t *from = order, *to = other;
        auto pass = [&](const uint32_t *key, int shift) {
            if (radix_pass(key, from, to, n, shift, counts, s_scan)) {
                uint32_t *x = from;
                from = to;
                to = x;
            }
        };
        // least significant first.  (The protection rides in the positions' top
        // digit, which changes nothing: it is the last criterion again.)
        if (by_place)
            for (int shift = 0; shift < 32; shift += 8) pass(place, shift);
        for (int shift = 0; shift < 32; shift += 8) pass(weight, shift);
        if (split) pass(place, 31);
        __syncthreads();
        if (from != order)
            for (int i = tid; i < n; i += kBulkThreads) order[i] = from[i];
        __syncthreads();
    }

    // ---- A: lambda^m A + eta sum of lambda^(m-1-i) k_i v_i^T -------------------------
    if (c.A) {
        const Decay decay(c.lam[h]);
        unsigned char *parts = tiles_mem + S::STAGES * S::RAW;
        const int wm = warp % S::TM, wn = (warp / S::TM) * S::NT;
        const bool works = wn < S::TN;
        float sum[S::NT][4];
#pragma unroll
        for (int t = 0; t < S::NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[t][e] = 0.f;
        const int all = (m + S::TP - 1) / S::TP, tiles = (all - rank + SL - 1) / SL;  // every SL-th is this block's
        // pool rows and weights of a tile's pairs
        auto plan = [&](int tile) {
            if (tid < S::TP && tile < tiles) {
                const int i = (tile * SL + rank) * S::TP + tid;
                s_row[tile % (S::STAGES + 1)][tid] = i < m ? row_of((int)order[i]) : -1;
                s_w[tile % (S::STAGES + 1)][tid] = i < m ? decay.pow(m - 1 - i) : 0.f;
            }
        };
        auto fetch = [&](int tile) {
            if (tile < tiles) {
                unsigned char *raw = tiles_mem + (tile % S::STAGES) * S::RAW;
                constexpr int RC = D * (int)sizeof(T) / 16, EL = 16 / (int)sizeof(T);  // chunks of a row, elements of one
                for (int x = tid; x < S::TP * 2 * RC; x += kBulkThreads) {
                    const int pr = x / (2 * RC), ch = x % (2 * RC);
                    const int64_t row = s_row[tile % (S::STAGES + 1)][pr];
                    unsigned char *dst = ch < RC ? raw + pr * S::KRAW + ch * 16 : raw + S::TP * S::KRAW + pr * S::VRAW + (ch - RC) * 16;
                    const T *src = ch < RC ? kp + row * D + ch * EL : vp + row * D + (ch - RC) * EL;
                    if (row >= 0) copy16(dst, src);
                    else zero16(dst);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");  // an empty group past the last tile
        };
        for (int i = 0; i < S::STAGES; ++i) plan(i);
        __syncthreads();
        for (int i = 0; i < S::STAGES - 1; ++i) fetch(i);
        for (int tile = 0; tile < tiles; ++tile) {
            asm volatile("cp.async.wait_group %0;" ::"n"(S::STAGES - 2) : "memory");
            __syncthreads();  // the tile is there; the parts and the last tile's buffer are free
            fetch(tile + S::STAGES - 1);
            plan(tile + S::STAGES);
            const unsigned char *raw = tiles_mem + (tile % S::STAGES) * S::RAW;
            for (int x = tid; x < S::TP * D / 2; x += kBulkThreads) {
                const int pr = x / (D / 2), e = x % (D / 2);
                const T *src = reinterpret_cast<const T *>(raw + pr * S::KRAW) + 2 * e;
                const float w = s_w[tile % (S::STAGES + 1)][pr];
                uint32_t o[3];
                split3(w * to_f32(src[0]), w * to_f32(src[1]), o);
#pragma unroll
                for (int i = 0; i < 3; ++i) *reinterpret_cast<uint32_t *>(parts + (i * S::TP + pr) * S::PS + e * 4) = o[i];
                if (S::VPARTS) {
                    const T *val = reinterpret_cast<const T *>(raw + S::TP * S::KRAW + pr * S::VRAW) + 2 * e;
                    split3(to_f32(val[0]), to_f32(val[1]), o);
#pragma unroll
                    for (int i = 0; i < 3; ++i) *reinterpret_cast<uint32_t *>(parts + ((3 + i) * S::TP + pr) * S::PS + e * 4) = o[i];
                }
            }
            __syncthreads();
            if (works) {
                const unsigned char *vbase = S::VPARTS ? parts + 3 * S::TP * S::PS : raw + S::TP * S::KRAW;
                constexpr int VROW = S::VPARTS ? S::PS : S::VRAW;
                float acc[S::NT][4];
#pragma unroll
                for (int t = 0; t < S::NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[t][e] = 0.f;
#pragma unroll
                for (int k = 0; k < S::TP / 16; ++k) {
                    // keys [pair][row]: as the transposed operand, pairs along k
                    uint32_t a[3][4];
#pragma unroll
                    for (int i = 0; i < 3; ++i)
                        ldsm_t4(parts + (i * S::TP + k * 16 + (lane & 7) + (lane >> 4) * 8) * S::PS + (wm * 16 + ((lane >> 3) & 1) * 8) * 2, a[i]);
#pragma unroll
                    for (int t = 0; t < S::NT; ++t) {
#pragma unroll
                        for (int j = 0; j < (S::VPARTS ? 3 : 1); ++j) {
                            uint32_t v[2];
                            ldsm_t2(vbase + (j * S::TP + k * 16 + (lane & 15)) * VROW + (wn + t) * 16, v);
#pragma unroll
                            for (int i = 2 - j; i >= 0; --i) mma_bf16(acc[t], a[i], v);
                        }
                    }
                }
#pragma unroll
                for (int t = 0; t < S::NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[t][e] += acc[t][e];
            }
        }
        const float lm = decay.pow(m), eta = c.eta[h];
        const int row = wm * 16 + lane / 4, col = (lane % 4) * 2;
        if constexpr (SL == 1) {
            if (works) {
#pragma unroll
                for (int t = 0; t < S::NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        float2 *x = reinterpret_cast<float2 *>(c.A + (bh * D + row + e * 4) * D + (wn + t) * 8 + col);
                        float2 o = *x;
                        o.x = fmaf(lm, o.x, eta * sum[t][e]);
                        o.y = fmaf(lm, o.y, eta * sum[t][e + 1]);
                        *x = o;
                    }
            }
        } else {
            float *mine = reinterpret_cast<float *>(tiles_mem);  // [D][D]
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();
            if (works) {
#pragma unroll
                for (int t = 0; t < S::NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; e += 2)
                        *reinterpret_cast<float2 *>(mine + (row + e * 4) * D + (wn + t) * 8 + col) = make_float2(sum[t][e], sum[t][e + 1]);
            }
            cluster_sync();
            // this block's rows of A, from every block's sum
            constexpr int R = D / SL;
            for (int x = tid; x < R * D / 4; x += kBulkThreads) {
                const int at = rank * R * D / 4 + x;
                float4 add = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int r = 0; r < SL; ++r) {
                    uint32_t there;
                    float4 y;
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(sm100::smem_u32(mine + at * 4)), "r"(r));
                    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(y.x), "=f"(y.y), "=f"(y.z), "=f"(y.w) : "r"(there) : "memory");
                    add.x += y.x;
                    add.y += y.y;
                    add.z += y.z;
                    add.w += y.w;
                }
                float4 *dst = reinterpret_cast<float4 *>(c.A + bh * D * D) + at;
                float4 o = *dst;
                o.x = fmaf(lm, o.x, eta * add.x);
                o.y = fmaf(lm, o.y, eta * add.y);
                o.z = fmaf(lm, o.z, eta * add.z);
                o.w = fmaf(lm, o.w, eta * add.w);
                *dst = o;
            }
            cluster_sync();  // the sums have been read: their room is free
        }
    }

    // ---- freed slots below keep, and the pairs behind it that stay ------------------
    for (int i = tid; i < m; i += kBulkThreads) atomicOr(&bits[order[i] / 32], 1u << (order[i] % 32));
    __syncthreads();
    int *hole = reinterpret_cast<int *>(scratch), *fill = hole + room;
    const int per = (words + kBulkThreads - 1) / kBulkThreads;
    auto freed = [&](int w) {  // slots of word w that leave and are below keep
        const int below = keep - w * 32;
        return below <= 0 ? 0u : bits[w] & (below >= 32 ? ~0u : (1u << below) - 1u);
    };
    auto stays = [&](int w) {  // slots of word w at or behind keep, held, that stay
        const int below = keep - w * 32, end = n - w * 32;
        uint32_t x = ~bits[w];
        if (below >= 32) return 0u;
        if (below > 0) x &= ~((1u << below) - 1u);
        if (end < 32) x &= (1u << end) - 1u;
        return x;
    };
    int nh = 0, nf = 0, moves, total;
    for (int w = tid * per; w < min(words, (tid + 1) * per); ++w) {
        nh += __popc(freed(w));
        nf += __popc(stays(w));
    }
    int ih = block_scan(nh, s_scan, &moves);
    int jf = block_scan(nf, s_scan, &total);
    for (int w = tid * per; w < min(words, (tid + 1) * per); ++w) {
        for (uint32_t x = freed(w); x; x &= x - 1) hole[ih++] = w * 32 + __ffs(x) - 1;
        for (uint32_t x = stays(w); x; x &= x - 1) fill[jf++] = w * 32 + __ffs(x) - 1;
    }
    __syncthreads();
    for (int x = tid; x < 2 * moves; x += kBulkThreads) {  // slots to pool rows
        int *at = x < moves ? hole + x : fill + (x - moves);
        *at = row_of(*at);
    }

    // ---- moves, once every block of the cluster has read what they overwrite --------
    if (SL > 1) cluster_sync();
    else __syncthreads();
    constexpr int LPR = D * (int)sizeof(T) / 16;  // 16-byte vectors of a row
    constexpr int UN = 4;                         // vectors in flight per thread
    const int64_t vectors = (int64_t)moves * 2 * LPR;
    for (int64_t x0 = (int64_t)rank * kBulkThreads + tid; x0 < vectors; x0 += (int64_t)UN * SL * kBulkThreads) {
        uint4 val[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int64_t x = x0 + (int64_t)u * SL * kBulkThreads;
            if (x < vectors) {
                const int mv = (int)(x / (2 * LPR)), i = (int)(x % (2 * LPR));
                const T *pool = i < LPR ? kp : vp;
                val[u] = reinterpret_cast<const uint4 *>(pool + (int64_t)fill[mv] * D)[i < LPR ? i : i - LPR];
            }
        }
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int64_t x = x0 + (int64_t)u * SL * kBulkThreads;
            if (x < vectors) {
                const int mv = (int)(x / (2 * LPR)), i = (int)(x % (2 * LPR));
                T *pool = i < LPR ? kp : vp;
                reinterpret_cast<uint4 *>(pool + (int64_t)hole[mv] * D)[i < LPR ? i : i - LPR] = val[u];
            }
        }
    }
    for (int x = rank * kBulkThreads + tid; x < moves; x += SL * kBulkThreads) {
        c.mass[hole[x]] = c.mass[fill[x]];
        c.pos[hole[x]] = c.pos[fill[x]];
    }
}

cudaLaunchConfig_t cluster_launch(cudaLaunchAttribute *attr, int64_t grid, int threads, size_t smem, int slices, bool early, cudaStream_t s) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)slices;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = early ? 2 : 1;
    return cfg;
}

template <typename T, int D, bool STEP>
cudaError_t launch_one(const EvictParams &p, int slices, cudaStream_t s) {
    const size_t smem = p.c.A ? (size_t)D * D / slices * sizeof(float) : 0;
    cudaError_t e = allow_smem(evict_one_kernel<T, D, STEP>, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = cluster_launch(attr, (int64_t)p.c.B * p.c.H * slices, kOneThreads, smem, slices, false, s);
    return cudaLaunchKernelEx(&cfg, evict_one_kernel<T, D, STEP>, p, slices);
}

template <typename T, int D, int SL>
cudaError_t launch_bulk(const EvictParams &p, cudaStream_t s) {
    const int64_t cap = n2_cap_global(p.c.capacity());
    const int n2 = (int)(cap < kSortMax ? cap : kSortMax);
    const size_t sum = BulkShape<T, D>::SUM, sort = sort_room(n2);
    const size_t smem = order_room(n2) + (sum > sort ? sum : sort);
    cudaError_t e = allow_smem(evict_bulk_kernel<T, D, SL>, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = cluster_launch(attr, (int64_t)p.c.B * p.c.H * SL, kBulkThreads, smem, SL, true, s);
    return cudaLaunchKernelEx(&cfg, evict_bulk_kernel<T, D, SL>, p, n2);
}

template <typename T, int D>
cudaError_t launch_bulk_sl(const EvictParams &p, int slices, cudaStream_t s) {
    if constexpr (D >= 64)
        if (slices == 4) return launch_bulk<T, D, 4>(p, s);
    if constexpr (D >= 32)
        if (slices == 2) return launch_bulk<T, D, 2>(p, s);
    return launch_bulk<T, D, 1>(p, s);
}

template <typename T>
cudaError_t launch_bulk_d(const EvictParams &p, int d, int slices, cudaStream_t s) {
    switch (d) {
        case 16: return launch_bulk_sl<T, 16>(p, slices, s);
        case 32: return launch_bulk_sl<T, 32>(p, slices, s);
        case 64: return launch_bulk_sl<T, 64>(p, slices, s);
        case 128: return launch_bulk_sl<T, 128>(p, slices, s);
    }
    return cudaErrorInvalidValue;
}

template <typename T, bool STEP>
cudaError_t launch_one_d(const EvictParams &p, int d, int slices, cudaStream_t s) {
    switch (d) {
        case 16: return launch_one<T, 16, STEP>(p, slices, s);
        case 32: return launch_one<T, 32, STEP>(p, slices, s);
        case 64: return launch_one<T, 64, STEP>(p, slices, s);
        case 128: return launch_one<T, 128, STEP>(p, slices, s);
    }
    return cudaErrorInvalidValue;
}

// Slices a head's A is cut into, one block of a cluster each, of 16 rows at
// least: more while the device has room for them, `least` at any rate.
int slices_for(int64_t BH, int d, int least, int most, int num_sms) {
    int slices = least;
    while (slices * 2 <= d / 16 && slices < most && BH * slices * 2 <= 2 * num_sms) slices *= 2;
    return slices;
}

}  // namespace

cudaError_t launch_cache_append(const AppendParams &p, tc_dtype dtype, cudaStream_t s) {
    if (p.T == 0) return cudaSuccess;
    const int64_t es = dtype == TC_BF16 ? 2 : 4;
    const int vec = (int)(16 / es);
    const int64_t qn[3] = {p.c.B, p.Hq, p.T}, kn[3] = {p.c.B, p.c.H, p.T};
    const bool wide = p.table.rot % (2 * vec) == 0 && rows_aligned16(p.k, p.ks, kn, es) &&
                      rows_aligned16(p.v, p.vs, kn, es) && (!p.q || rows_aligned16(p.q, p.qs, qn, es));
    if (dtype == TC_BF16)
        return wide ? launch_append_vec<__nv_bfloat16, 8>(p, s) : launch_append_vec<__nv_bfloat16, 1>(p, s);
    return wide ? launch_append_vec<float, 4>(p, s) : launch_append_vec<float, 1>(p, s);
}

// 32 KB of A a block at most, so that several share an SM.
int evict_slices(int64_t BH, int d, int num_sms) { return slices_for(BH, d, d == 128 ? 2 : 1, 4, num_sms); }

namespace {
int bulk_slices(int64_t BH, int d, int num_sms) { return slices_for(BH, d, 1, 4, num_sms); }
}  // namespace

size_t evict_sort_bytes(int64_t BH, int d, int64_t capacity, int num_sms) {
    const int64_t n2 = n2_cap_global(capacity);
    return n2 <= kSortMax ? 0 : (size_t)BH * (size_t)bulk_slices(BH, d, num_sms) * (order_room(n2) + sort_room(n2));
}

cudaError_t launch_cache_step_insert(const EvictParams &p, tc_dtype dtype, int d, int slices, cudaStream_t s) {
    return dtype == TC_BF16 ? launch_one_d<__nv_bfloat16, true>(p, d, slices, s) : launch_one_d<float, true>(p, d, slices, s);
}

cudaError_t launch_cache_evict(const EvictParams &p, tc_dtype dtype, int d, int num_sms, cudaStream_t s) {
    const int64_t BH = (int64_t)p.c.B * p.c.H;
    const int one = evict_slices(BH, d, num_sms), bulk = bulk_slices(BH, d, num_sms);
    const cudaError_t e = dtype == TC_BF16 ? launch_one_d<__nv_bfloat16, false>(p, d, one, s) : launch_one_d<float, false>(p, d, one, s);
    if (e != cudaSuccess) return e;
    return dtype == TC_BF16 ? launch_bulk_d<__nv_bfloat16>(p, d, bulk, s) : launch_bulk_d<float>(p, d, bulk, s);
}

}  // namespace tc

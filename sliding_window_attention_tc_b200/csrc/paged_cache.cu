// Insertion into, and eviction from, the paged cache.
//
// Insertion (tc_cache_append): new tokens' keys are rotated by their positions
// and stored with their values; queries are rotated beside them.  Bound by
// memory; one block owns up to 8 tokens of one row (a longer stretch leaves too
// few blocks, a shorter one writes too little at a place) and walks the heads.
// What it waits for is a chain (count, length, page, then its loads and stores),
// so small blocks, eight to an SM, whose chains overlap: 2500 tokens each for 4
// padded rows, 12 heads of d = 64, float32, 116 MB: 24.3 us, 4.8 TB/s (four of
// twice the threads: 25.7; 16 tokens a block: 32).
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

#include <atomic>
#include <type_traits>

#include "paged_cache.cuh"
#include "sm100_ptx.cuh"

namespace tc {
namespace {

// ---- insertion ------------------------------------------------------------------

constexpr int kAppThreads = 128;
constexpr int kAppUnroll = 3;

// Tokens row b appends, or -1 when the row is to be skipped (and not because
// it is empty: *bad says that an error has to be reported).  Block-wide.
__device__ __forceinline__ int64_t append_count(const AppendParams &p, int b, int64_t &len, int64_t &clock, bool &bad) {
    len = p.c.len[b];
    clock = p.c.clock[b];
    bad = false;
    if (len < 0) return -1;
    const int64_t n = p.counts ? p.counts[b] : p.T;
    bad = n < 0 || n > p.T || len + n > p.c.capacity() || len > p.c.capacity() || clock < 0 ||
          clock > (int64_t(1) << 31) - n;
    if (!bad) bad = !block_pages_ok(p.c, b, len, len + n - 1);
    return bad ? -1 : n;
}

template <typename T, int VEC, bool INTER>
__global__ void __launch_bounds__(kAppThreads, 8) append_kernel(const __grid_constant__ AppendParams p, int chunks,
                                                                int tokens, int tiles, bool advance) {
    const int b = blockIdx.x / tiles;
    const int64_t t0 = (int64_t)(blockIdx.x % tiles) * tokens;
    const int H = p.c.H, d = p.d;
    const int chunk = threadIdx.x % chunks, r = threadIdx.x / chunks;
    const int hg = r / tokens, HG = kAppThreads / chunks / tokens;
    const int64_t t = t0 + r % tokens;
    RotChunk<T, VEC, INTER> rc;
    rc.place(p.table, chunk, d);
    // rows: the queries' heads, the keys', the values' (copied); kAppUnroll in
    // flight, the first of them while the row's length and pages are looked up
    // a padded batch: nothing is read past a row's tokens (its first block reports bad counts)
    const int64_t known = p.counts && !advance ? min(p.counts[b], p.T) : p.T;
    if (t0 >= known && t0 > 0) return;
    const int q_rows = p.q ? p.Hq : 0, rows = t < known && hg < HG ? q_rows + 2 * H : 0;
    typename RotChunk<T, VEC, INTER>::Raw u[kAppUnroll], w[kAppUnroll];
    auto load = [&](int x0) {
#pragma unroll
        for (int i = 0; i < kAppUnroll; ++i) {
            const int x = x0 + i * HG;
            if (x < rows) {
                const T *src = x < q_rows       ? reinterpret_cast<const T *>(p.q) + b * p.qs[0] + x * p.qs[1] + t * p.qs[2]
                               : x < q_rows + H ? reinterpret_cast<const T *>(p.k) + b * p.ks[0] + (x - q_rows) * p.ks[1] + t * p.ks[2]
                                                : reinterpret_cast<const T *>(p.v) + b * p.vs[0] + (x - q_rows - H) * p.vs[1] + t * p.vs[2];
                rc.load(src, u[i], w[i]);
            }
        }
    };
    load(hg);
    sm100::griddep_launch_dependents();  // the clocks' kernel waits for this one's end by itself
    int64_t len, clock;
    bool bad;
    const int64_t n = append_count(p, b, len, clock, bad);
    if (bad && threadIdx.x == 0) report(p.c.status, TC_ERR_DEVICE_BOUNDS);
    if (n < 0) return;
    if (t < n && hg < HG) {
        const int slot = (int)(len + t), page = p.c.page_of(slot), in_page = slot - page * p.c.page;
        const int64_t position = clock + t;
        const int pg = p.c.table[(int64_t)b * p.c.max_pages + page];
        rc.angles(p.table, chunk, position, false);
        for (int x0 = hg;;) {
#pragma unroll
            for (int i = 0; i < kAppUnroll; ++i) {
                const int x = x0 + i * HG;
                if (x < rows) {
                    T *dst;
                    if (x < q_rows) {
                        dst = reinterpret_cast<T *>(p.q_out) + (((int64_t)b * p.Hq + x) * p.T + t) * d;
                    } else if (x < q_rows + H) {
                        const int h = x - q_rows;
                        const int64_t row = pool_row(p.c, pg, h, in_page);
                        dst = reinterpret_cast<T *>(p.c.k) + row * d;
                        if (chunk == 0) {
                            if (p.c.mass) p.c.mass[row] = p.mass_in ? p.mass_in[((int64_t)b * H + h) * p.T + t] : 0.f;
                            if (p.c.pos) p.c.pos[row] = (int32_t)position;
                        }
                    } else {
                        dst = reinterpret_cast<T *>(p.c.v) + pool_row(p.c, pg, x - q_rows - H, in_page) * d;
                    }
                    rc.store(dst, u[i], w[i], x < q_rows + H);
                }
            }
            x0 += kAppUnroll * HG;
            if (x0 >= rows) break;
            load(x0);
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
    sm100::griddep_wait();
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
    const unsigned grid = (unsigned)(p.c.B * tiles);
    if (p.table.interleaved) append_kernel<T, VEC, true><<<grid, kAppThreads, 0, s>>>(p, chunks, tokens, (int)tiles, tiles == 1);
    else append_kernel<T, VEC, false><<<grid, kAppThreads, 0, s>>>(p, chunks, tokens, (int)tiles, tiles == 1);
    if (tiles > 1) {
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)p.c.B);
        cfg.blockDim = dim3(128);
        cfg.stream = s;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, append_advance_kernel, p);
        if (e != cudaSuccess) return e;
    }
    return cudaGetLastError();
}

// ---- eviction -------------------------------------------------------------------

// The order in which pairs leave, as one number: unprotected first, then by
// weight (NaN last, -0 as 0), then by position.  No number is free to stand for
// "no pair" (a protected NaN at position 2^31 - 1 has them all set), so pairs are
// compared with their slots: no pair is (~0, ~0), behind every slot there is.
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

// ---- at most one pair leaves (the steady state; the step's first kernel) ----------
//
// What it waits for is the chain length -> table -> weights -> pair -> A: A is
// asked into L2 at the start, and the blocks are small enough (64 registers, 20
// KB) that four share an SM: 512 (row, head) of a serving step run at once.
// (With A staged in shared memory two shared an SM, in two waves: 26 us; half of
// A a block, twice the blocks: 30 us.)
constexpr int kOneThreads = 256;
constexpr int kOneWarps = kOneThreads / 32;
constexpr int kQBatch = 4;    // query heads per pass over A
constexpr int kScanBatch = 4; // weights in flight per thread

template <typename T, int D, bool STEP>
__global__ void __launch_bounds__(kOneThreads, 4) evict_one_kernel(const __grid_constant__ EvictParams p, int slices) {
    constexpr int CG = D / 4;              // float4 columns of A
    constexpr int RG = kOneThreads / CG;   // rows of A side by side
    constexpr int AU = 4;                  // float4 of A in flight per thread
    __shared__ __align__(16) float s_k[D], s_v[D];            // the pair that leaves
    __shared__ __align__(16) T s_new[2][D];                   // the new pair
    __shared__ float s_cos[D / 2 + 1], s_sin[D / 2 + 1];
    __shared__ uint64_t s_key[kOneWarps];
    __shared__ uint32_t s_slot[kOneWarps];
    __shared__ float s_q[kQBatch][D];
    __shared__ __align__(16) float s_mp[RG][kQBatch][D];

    const CacheParams &c = p.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = blockIdx.x % slices;
    const int64_t bh = blockIdx.x / slices;
    const int b = (int)(bh / c.H), h = (int)(bh % c.H);
    sm100::griddep_launch_dependents();  // the next kernel waits for this one's end by itself
    const int64_t held = c.len[b], clock0 = c.clock[b];
    const int G = STEP ? p.Hq / c.H : 0;
    const bool first = h == 0 && rank == 0 && tid == 0;
    const int rows = D / slices, row0 = rank * rows;
    const bool read = STEP && p.memo != nullptr;
    float4 *A4 = c.A ? reinterpret_cast<float4 *>(c.A + (bh * D + row0) * D) : nullptr;

    // the new token's rows do not wait for the length
    constexpr int NEW = (2 * D + kOneThreads - 1) / kOneThreads;
    float fresh[NEW];
    if (STEP) {
#pragma unroll
        for (int i = 0; i < NEW; ++i) {
            const int x = tid + i * kOneThreads;
            if (x < 2 * D)
                fresh[i] = to_f32(x < D ? reinterpret_cast<const T *>(p.k_new)[b * p.ks[0] + h * p.ks[1] + x]
                                        : reinterpret_cast<const T *>(p.v_new)[b * p.vs[0] + h * p.vs[1] + x - D]);
        }
        for (int i = tid; i < p.table.rot / 2; i += kOneThreads)
            rotary_angle(clock0, p.table.inc[i], p.table.gain, s_cos[i], s_sin[i]);
    }
    const int64_t n64 = held < 0 ? -1 : held + (STEP ? 1 : 0);
    // a step lets one pair leave at most: a row above its budget stays above
    const int64_t over = n64 - p.budget;
    const int m = over <= 0 ? 0 : STEP ? 1 : over == 1 ? 1 : 0;
    bool ok = held >= 0 && n64 <= c.capacity() && held <= c.capacity() && (!STEP || (clock0 >= 0 && clock0 < (int64_t(1) << 31)));
    const bool use_A = A4 && ok && (read || m == 1);
    if (use_A && tid == 0)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(A4), "r"(rows * D * 4) : "memory");
    if (ok) ok = block_pages_ok(c, b, 0, n64 - 1);  // its barrier also publishes s_cos, s_sin
    if (first) {
        if (held >= 0 && !ok) report(c.status, TC_ERR_DEVICE_BOUNDS);
        p.row_len[b] = !ok ? -1 : STEP ? n64 - m : n64;
    }
    if (!ok || (m == 0 && !STEP)) return;  // the whole cluster
    const int n = (int)n64, keep = n - m;
    const int32_t *table = c.table + (int64_t)b * c.max_pages;
    auto row_of = [&](int slot) {  // below 2^31
        const int pg = c.page_of(slot);
        return (table[pg] * c.H + h) * c.page + slot - pg * c.page;
    };
    T *kp = reinterpret_cast<T *>(c.k), *vp = reinterpret_cast<T *>(c.v);

    // weights and positions of the pairs held before: under way while the new pair enters
    const int seen = STEP ? n - 1 : n;
    float w[kScanBatch];
    int32_t z[kScanBatch];
    auto look = [&](int s0) {
#pragma unroll
        for (int i = 0; i < kScanBatch; ++i) {
            const int s = s0 + i * kOneThreads;
            if (s < seen) {
                const int row = row_of(s);
                w[i] = c.mass[row];
                z[i] = c.pos[row];
            }
        }
    };
    if (m == 1) look(tid);

    if (STEP) {
        // the new pair enters slot n - 1 (every block of the cluster writes the
        // same values), the queries are rotated
        const RotaryTable &rt = p.table;
        const int half = rt.rot / 2;
        auto turned = [&](float f, float g, int i) {  // element i, its pair's other element g
            const int pair = rt.interleaved ? i / 2 : i < half ? i : i - half;
            const bool second = rt.interleaved ? (i & 1) : i >= half;
            return rotated(f, g, s_cos[pair], second ? s_sin[pair] : -s_sin[pair]);
        };
        auto other = [&](int i) { return rt.interleaved ? i ^ 1 : i < half ? i + half : i - half; };
        const int64_t row = row_of(n - 1);
#pragma unroll
        for (int i = 0; i < NEW; ++i) {
            const int x = tid + i * kOneThreads;
            if (x < D) s_k[x] = fresh[i];
            else if (x < 2 * D) s_new[1][x - D] = from_f32<T>(fresh[i]);
        }
        __syncthreads();
        for (int x = tid; x < D; x += kOneThreads)
            s_new[0][x] = from_f32<T>(x < rt.rot ? turned(s_k[x], s_k[other(x)], x) : s_k[x]);
        for (int x = tid; x < G * D; x += kOneThreads) {
            const int g = x / D, i = x % D;
            const T *src = reinterpret_cast<const T *>(p.q) + b * p.qs[0] + (h * G + g) * p.qs[1];
            float f = to_f32(src[i]);
            if (i < rt.rot) f = turned(f, to_f32(src[other(i)]), i);
            const T r = from_f32<T>(f);
            if (rank == 0) reinterpret_cast<T *>(p.q_rot)[(bh * G + g) * D + i] = r;
            if (g < kQBatch) s_q[g][i] = to_f32(r);  // the first batch's; later ones are rotated again
        }
        __syncthreads();
        constexpr int LPR = D * (int)sizeof(T) / 16;  // 16-byte vectors of a row
        if (tid < 2 * LPR) {
            const int i = tid < LPR ? tid : tid - LPR;
            reinterpret_cast<uint4 *>((tid < LPR ? kp : vp) + row * D)[i] = reinterpret_cast<const uint4 *>(s_new[tid < LPR ? 0 : 1])[i];
        }
        if (tid == 0) {
            c.mass[row] = 0.f;
            c.pos[row] = (int32_t)clock0;
        }
    }

    int gone = 0;  // the slot that leaves
    if (m == 1) {
        const int64_t protect_from = clock0 + (STEP ? 1 : 0) - p.recent;
        uint64_t best = ~0ull;
        uint32_t slot = tid < seen ? (uint32_t)tid : 0xffffffffu;  // its own pairs may all be the last there is
        for (int s0 = tid;;) {
#pragma unroll
            for (int i = 0; i < kScanBatch; ++i) {
                const int s = s0 + i * kOneThreads;
                if (s < seen) {
                    const uint64_t key = leave_key(w[i], z[i], protect_from);
                    if (key < best) {  // equal pairs: the earlier slot, seen first
                        best = key;
                        slot = (uint32_t)s;
                    }
                }
            }
            s0 += kScanBatch * kOneThreads;
            if (s0 >= seen) break;
            look(s0);
        }
        if (STEP && tid == 0) {
            const uint64_t key = leave_key(0.f, (int32_t)clock0, protect_from);
            if (less_pair(key, (uint32_t)(n - 1), best, slot)) {
                best = key;
                slot = (uint32_t)(n - 1);
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
        for (int x = 0; x < kOneWarps; ++x)
            if (x == 0 || less_pair(s_key[x], s_slot[x], best, slot)) {
                best = s_key[x];
                slot = s_slot[x];
            }
        gone = (int)slot;
    }

    if (use_A) {
        if (m == 1) {
            const bool is_new = STEP && gone == n - 1;
            const int64_t row = is_new ? 0 : row_of(gone);
            for (int i = tid; i < 2 * D; i += kOneThreads) {
                const bool value = i >= D;
                const int e = value ? i - D : i;
                const T x = is_new ? s_new[value][e] : (value ? vp : kp)[row * D + e];
                if (value) s_v[e] = to_f32(x);
                else s_k[e] = to_f32(x);
            }
        }
        __syncthreads();
    }
    // every block of the cluster that gets here has read the pair that leaves:
    // the barrier is waited for where its slot is written
    if (m == 1 && slices > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (use_A) {
        const int cg = tid % CG, rg = tid / CG;
        const float lam = c.lam[h], eta = c.eta[h];
        const float4 v4 = m == 1 ? reinterpret_cast<const float4 *>(s_v)[cg] : make_float4(0.f, 0.f, 0.f, 0.f);
        for (int g0 = 0; g0 == 0 || (read && g0 < G); g0 += kQBatch) {
            const int ng = read ? min(kQBatch, G - g0) : 0;
            if (g0 > 0) {  // (read) later batches: the queries again
                for (int x = tid; x < ng * D; x += kOneThreads) {
                    const int g = x / D, i = x % D;
                    const T *src = reinterpret_cast<const T *>(p.q) + b * p.qs[0] + (h * G + g0 + g) * p.qs[1];
                    float f = to_f32(src[i]);
                    const int half = p.table.rot / 2;
                    if (i < p.table.rot) {
                        const int pair = p.table.interleaved ? i / 2 : i < half ? i : i - half;
                        const bool second = p.table.interleaved ? (i & 1) : i >= half;
                        const float y = to_f32(src[p.table.interleaved ? i ^ 1 : i < half ? i + half : i - half]);
                        f = rotated(f, y, s_cos[pair], second ? s_sin[pair] : -s_sin[pair]);
                    }
                    s_q[g][i] = to_f32(from_f32<T>(f));
                }
                __syncthreads();
            }
            float4 mp[kQBatch];
#pragma unroll
            for (int g = 0; g < kQBatch; ++g) mp[g] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int r0 = rg; r0 < rows; r0 += AU * RG) {
                float4 a[AU];
#pragma unroll
                for (int i = 0; i < AU; ++i)
                    if (r0 + i * RG < rows) a[i] = A4[(r0 + i * RG) * CG + cg];
#pragma unroll
                for (int i = 0; i < AU; ++i) {
                    const int r = r0 + i * RG;
                    if (r >= rows) break;
                    if (g0 == 0 && m == 1) {
                        const float ek = eta * s_k[row0 + r];
                        a[i].x = fmaf(lam, a[i].x, ek * v4.x);
                        a[i].y = fmaf(lam, a[i].y, ek * v4.y);
                        a[i].z = fmaf(lam, a[i].z, ek * v4.z);
                        a[i].w = fmaf(lam, a[i].w, ek * v4.w);
                        A4[r * CG + cg] = a[i];  // (later batches read it back)
                    }
                    if (read) {
#pragma unroll
                        for (int g = 0; g < kQBatch; ++g) {
                            const float x = s_q[g][row0 + r];  // heads past the last: never stored
                            mp[g].x = fmaf(x, a[i].x, mp[g].x);
                            mp[g].y = fmaf(x, a[i].y, mp[g].y);
                            mp[g].z = fmaf(x, a[i].z, mp[g].z);
                            mp[g].w = fmaf(x, a[i].w, mp[g].w);
                        }
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

    // the last pair moves to the freed slot (a step's: the new one, from here)
    if (slices > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    else __syncthreads();
    constexpr int LPR = D * (int)sizeof(T) / 16;
    if (rank == 0 && gone < keep && tid < 2 * LPR) {
        const int64_t from = row_of(keep), to = row_of(gone);
        T *pool = tid < LPR ? kp : vp;
        const int i = tid < LPR ? tid : tid - LPR;
        reinterpret_cast<uint4 *>(pool + to * D)[i] = STEP ? reinterpret_cast<const uint4 *>(s_new[tid < LPR ? 0 : 1])[i]
                                                           : reinterpret_cast<const uint4 *>(pool + from * D)[i];
        if (tid == 0) {
            c.mass[to] = STEP ? 0.f : c.mass[from];
            c.pos[to] = STEP ? (int32_t)clock0 : c.pos[from];
        }
    }
}

// ---- several pairs leave ------------------------------------------------------------
//
// The slots are sorted by (protected, mass, pos) with a stable radix sort, in
// shared memory up to kSortMax pairs, over the bits in which pairs differ; or,
// where the weights spread, by counting them into buckets first.  (2559 pairs: a
// bitonic sort of the keys took 139,000 cycles, a radix sort of 8 bits a pass with a
// warp's lanes matched against one another 82,000, the one below 41,000.)  The
// weighted sum runs on the tensor cores: tiles of TP pairs come in by
// asynchronous 16-byte copies, several in flight; a warp takes 16 pairs and 16 of
// A's rows, makes the weighted keys lambda^(m-1-i) k_i in registers, in three bf16
// parts (24 bits together; a float32 cache's values too), and the products' sums
// over one tile are added to float32 sums with the ordinary rounding, because the
// tensor cores' own accumulation truncates and would drift over thousands of
// pairs.  The blocks of a cluster take every SL-th tile and add their sums through
// one another's shared memory.
constexpr int kBulkThreads = 512;
constexpr int kBulkWarps = kBulkThreads / 32;
constexpr int kSortMax = 8192;   // pairs sorted in shared memory (16 bytes each)
// Pairs picked one after the other instead (rows of up to 32 * 512): of 96 heads
// of 512 pairs and more, 8 leave in 24.3 us picked and in 27.0 sorted, 32 in 34.0
// and 27.8; of 8 heads of 8000, 2 in 24.4 and 28.6, 32 in 43.9 and 32.8.
constexpr int kPickMax = 10;

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

// One stable pass over a digit: order b of n slots from order a by the bits of
// key[slot] from `shift` on.  A thread takes ITEMS consecutive places (an odd
// number, so that the lanes' reads fall into different banks) and counts its
// digits in counters of its own, [digit][thread]; a warp per row of counters
// makes their prefix; the counters then give every element its place.  Counters
// of 16 bits, two digits a row, make 5 bits a pass; ITEMS 0 (any number of
// pairs, each read twice) needs 32 and takes 4.  The counters are the thread's
// own, so the atomic additions meet nobody: they are used because they do not
// wait for one another as loads and stores would.
template <int ITEMS>
struct RadixDigit {
    static constexpr int BITS = ITEMS ? 5 : 4;
    static constexpr uint32_t MASK = (1u << BITS) - 1u;
    __device__ __forceinline__ static uint32_t row(uint32_t d) { return ITEMS ? d >> 1 : d; }
    __device__ __forceinline__ static uint32_t one(uint32_t d) { return ITEMS ? 1u << ((d & 1u) * 16) : 1u; }
    __device__ __forceinline__ static uint32_t count(uint32_t word, uint32_t d) { return ITEMS ? (word >> ((d & 1u) * 16)) & 0xffffu : word; }
};

template <int ITEMS>
__device__ __forceinline__ void radix_pass(const uint32_t *key, const uint32_t *a, uint32_t *b, int n, int shift, uint32_t *counts,
                                           uint32_t *total, uint32_t (*base)[32]) {
    using R = RadixDigit<ITEMS>;
    static_assert(kBulkWarps == 16, "a warp per row of counters");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = ITEMS ? ITEMS : ((n + kBulkThreads - 1) / kBulkThreads) | 1, i0 = min(n, tid * per), i1 = min(n, i0 + per);
    uint32_t *mine = counts + tid;
#pragma unroll
    for (int d = 0; d < 16; ++d) mine[d * kBulkThreads] = 0;
    uint32_t s[ITEMS ? ITEMS : 1], digit[ITEMS ? ITEMS : 1];
    if (ITEMS) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) s[i] = i0 + i < i1 ? a[i0 + i] : 0u;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) digit[i] = (key[s[i]] >> shift) & R::MASK;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
            if (i0 + i < i1) mine[R::row(digit[i]) * kBulkThreads] += R::one(digit[i]);
    } else {
        for (int i = i0; i < i1; ++i) atomicAdd(mine + ((key[a[i]] >> shift) & R::MASK) * kBulkThreads, 1u);
    }
    __syncthreads();
    uint4 *row = reinterpret_cast<uint4 *>(counts + warp * kBulkThreads);
    uint4 c[kBulkThreads / 128];
    uint32_t v[kBulkThreads / 128];
#pragma unroll
    for (int x = 0; x < kBulkThreads / 128; ++x) {
        c[x] = row[x * 32 + lane];
        v[x] = c[x].x + c[x].y + c[x].z + c[x].w;
    }
#pragma unroll
    for (int o = 1; o < 32; o *= 2)
#pragma unroll
        for (int x = 0; x < kBulkThreads / 128; ++x) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, v[x], o);
            if (lane >= o) v[x] += y;
        }
    uint32_t before = 0;
#pragma unroll
    for (int x = 0; x < kBulkThreads / 128; ++x) {
        const uint32_t p = before + v[x] - (c[x].x + c[x].y + c[x].z + c[x].w);
        row[x * 32 + lane] = make_uint4(p, p + c[x].x, p + c[x].x + c[x].y, p + c[x].x + c[x].y + c[x].z);
        before += __shfl_sync(0xffffffffu, v[x], 31);
    }
    if (lane == 0) {
        if (ITEMS) {
            total[2 * warp] = before & 0xffffu;
            total[2 * warp + 1] = before >> 16;
        } else {
            total[warp] = before;
        }
    }
    __syncthreads();
    {  // where each digit begins, a copy per warp
        const uint32_t x = lane <= (int)R::MASK ? total[lane] : 0u;
        uint32_t sum = x;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        base[warp][lane] = sum - x;
        __syncwarp();
    }
    if (ITEMS) {
        uint32_t to[ITEMS ? ITEMS : 1];
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
            if (i0 + i < i1) {
                uint32_t &word = mine[R::row(digit[i]) * kBulkThreads];
                const uint32_t old = word;
                word = old + R::one(digit[i]);
                to[i] = R::count(old, digit[i]);
            }
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
            if (i0 + i < i1) b[to[i] + base[warp][digit[i]]] = s[i];
    } else {
        for (int i = i0; i < i1; ++i) {
            const uint32_t x = a[i], d = (key[x] >> shift) & R::MASK;
            b[atomicAdd(mine + d * kBulkThreads, 1u) + base[warp][d]] = x;
        }
    }
    __syncthreads();
}

// Sorts the slots 0 .. n-1 by (place, then weight, then place's bit 31), least
// significant first; only the digits in which pairs differ take a pass.  The
// protection (bit 31) rides along in the position's last pass and changes
// nothing there: it is the last criterion again.  Returns where the order is.
template <int ITEMS>
__device__ __forceinline__ uint32_t *sort_slots(uint32_t *order, uint32_t *other, const uint32_t *weight, uint32_t *place, int n,
                                                bool by_place, uint32_t w_differ, uint32_t z_differ, uint32_t *counts,
                                                uint32_t *total, uint32_t (*base)[32]) {
    using R = RadixDigit<ITEMS>;
    bool swapped = false;
    auto pass = [&](const uint32_t *key, int shift) {
        radix_pass<ITEMS>(key, swapped ? other : order, swapped ? order : other, n, shift, counts, total, base);
        swapped = !swapped;
    };
    // digits begin at the lowest bit in which pairs differ
    for (int part = by_place ? 0 : 1; part < 2; ++part) {
        uint32_t left = part ? w_differ : z_differ;
        while (left) {
            const int shift = __ffs(left) - 1;
            pass(part ? weight : place, shift);
            left = shift + R::BITS < 32 ? left >> (shift + R::BITS) << (shift + R::BITS) : 0u;
        }
    }
    if (z_differ >> 31) {
        for (int s = threadIdx.x; s < n; s += kBulkThreads) place[s] >>= 31;
        __syncthreads();
        pass(place, 0);
    }
    return swapped ? other : order;
}

// The same order (of its first m places: the others are not defined), for weights
// that differ: the slots are counted into buckets by weight (the bits of a float
// are its logarithm, so even steps of the bits spread weights of any scale; zeros
// have a bucket of their own; protected pairs theirs behind the others), and each
// finds its place among its bucket's few by comparing.  Buckets of more than
// kCompareMost (tokens that nothing has attended to yet, for one) are cut into
// buckets again, by position where all their weights are equal.  (2559 pairs, the
// kernel over 96 heads of d = 64: 62 us; with 2047 zeros among them 65 us, 88 sorted
// by digits; with a quarter of them equal 67 us, 83.)  False, and nothing done, where
// pairs are alike in both or too many buckets are large.  lo, hi: the least weight
// above zero and the greatest, as ordered bits; none below zero.
constexpr int kBuckets = 4096;     // plain and protected; 16-bit counters, two to a word
constexpr int kCompareMost = 64;
constexpr int kMostLarge = 8;

// The counters of a thread (8, in 4 words), and as the places where their buckets begin.
__device__ __forceinline__ void bucket_begins(uint32_t *words, int *scan, uint32_t (&c)[kBuckets / kBulkThreads],
                                              uint32_t (&at)[kBuckets / kBulkThreads]) {
    constexpr int N = kBuckets / kBulkThreads;
    static_assert(N == 8, "one vector of words");
    uint4 *mine = reinterpret_cast<uint4 *>(words) + threadIdx.x;
    const uint4 w = *mine;
    const uint32_t x[N] = {w.x & 0xffffu, w.x >> 16, w.y & 0xffffu, w.y >> 16, w.z & 0xffffu, w.z >> 16, w.w & 0xffffu, w.w >> 16};
    int sum = 0, total;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        c[i] = x[i];
        sum += (int)x[i];
    }
    uint32_t begin = (uint32_t)block_scan(sum, scan, &total);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        at[i] = begin;
        begin += x[i];
    }
    *mine = make_uint4(at[0] | at[1] << 16, at[2] | at[3] << 16, at[4] | at[5] << 16, at[6] | at[7] << 16);
}
__device__ __forceinline__ uint32_t half_word(const uint32_t *words, uint32_t i) { return words[i / 2] >> (i % 2 * 16) & 0xffffu; }

// words: 2 x kBuckets / 2 counters and 32 more.
__device__ bool bucket_sort(uint32_t *order, uint32_t *other, const uint32_t *weight, const uint32_t *place, int n, int m, uint32_t lo,
                            uint32_t hi, uint32_t *words, int *scan) {
    constexpr int N = kBuckets / kBulkThreads;
    const int tid = threadIdx.x;
    uint32_t *sub = words + kBuckets / 2, *large = sub + kBuckets / 2, *ends = large + 16;
    const int shift = max(0, 32 - __clz(hi - lo) - 11);  // (hi - lo) >> shift below 2048
    auto bucket = [&](uint32_t s) {
        const uint32_t v = weight[s];
        return (place[s] >> 31) * (kBuckets / 2) + (v == 0x80000000u ? 0u : min(1u + ((v - lo) >> shift), (uint32_t)kBuckets / 2 - 1));
    };
    auto next_place = [](uint32_t *table, uint32_t b) { return atomicAdd(table + b / 2, 1u << (b % 2 * 16)) >> (b % 2 * 16) & 0xffffu; };
    // how many of list[0 .. count) come before slot s
    auto rank = [&](const uint32_t *list, uint32_t count, uint32_t s) {
        const uint32_t v = weight[s], z = place[s];
        uint32_t r = 0;
#pragma unroll 4
        for (uint32_t j = 0; j < count; ++j) {
            const uint32_t x = list[j], vx = weight[x], zx = place[x];  // (within a bucket z's top bits agree)
            r += vx < v || (vx == v && (zx < z || (zx == z && x < s)));
        }
        return r;
    };
    for (int x = tid; x < kBuckets / 2; x += kBulkThreads) words[x] = 0;
    if (tid == 0) large[0] = 0;
    __syncthreads();
    for (int s = tid; s < n; s += kBulkThreads) next_place(words, bucket(s));
    __syncthreads();
    uint32_t c[N], at[N];
    bucket_begins(words, scan, c, at);
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (c[i] > kCompareMost && (int)at[i] < m) {
            const uint32_t x = atomicAdd(large, 1u);
            if (x < kMostLarge) large[1 + x] = at[i] | (at[i] + c[i]) << 16;
        }
    __syncthreads();
    if (large[0] > kMostLarge) return false;
    for (int s = tid; s < n; s += kBulkThreads) other[next_place(words, bucket(s))] = s;
    __syncthreads();
    // the counters are the buckets' ends now
    for (int i = tid; i < n; i += kBulkThreads) {
        const uint32_t s = other[i], b = bucket(s), begin = b ? half_word(words, b - 1) : 0u, end = half_word(words, b);
        if ((int)begin < m && end - begin <= kCompareMost) order[begin + rank(other + begin, end - begin, s)] = s;
    }
    for (uint32_t l = 0; l < large[0]; ++l) {
        const uint32_t begin = large[1 + l] & 0xffffu, end = large[1 + l] >> 16;
        for (int x = tid; x < kBuckets / 2; x += kBulkThreads) sub[x] = 0;
        if (tid < 4) ends[tid] = tid % 2 ? 0u : ~0u;  // weights' least and greatest, positions'
        __syncthreads();
        uint32_t e[4] = {~0u, 0u, ~0u, 0u};
        for (uint32_t i = begin + tid; i < end; i += kBulkThreads) {
            const uint32_t s = other[i];
            e[0] = min(e[0], weight[s]);
            e[1] = max(e[1], weight[s]);
            e[2] = min(e[2], place[s]);
            e[3] = max(e[3], place[s]);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            e[x] = x % 2 ? __reduce_max_sync(0xffffffffu, e[x]) : __reduce_min_sync(0xffffffffu, e[x]);
            if (tid % 32 == 0) x % 2 ? atomicMax(ends + x, e[x]) : atomicMin(ends + x, e[x]);
        }
        __syncthreads();
        const bool equal = ends[0] == ends[1];
        const uint32_t *key = equal ? place : weight, least = equal ? ends[2] : ends[0], range = (equal ? ends[3] : ends[1]) - least;
        const int cut = max(0, 32 - __clz(range) - 12);  // range >> cut below 4096
        for (uint32_t i = begin + tid; i < end; i += kBulkThreads) next_place(sub, (key[other[i]] - least) >> cut);
        __syncthreads();
        bucket_begins(sub, scan, c, at);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (c[i] > kCompareMost && (int)(begin + at[i]) < m) {  // again; not where all are alike
                const uint32_t x = range ? atomicAdd(large, 1u) : kMostLarge;
                if (x < kMostLarge) large[1 + x] = (begin + at[i]) | (begin + at[i] + c[i]) << 16;
                else large[0] = kMostLarge + 1;
            }
        __syncthreads();
        if (large[0] > kMostLarge) {
            for (int s = tid; s < n; s += kBulkThreads) order[s] = s;
            __syncthreads();
            return false;
        }
        for (uint32_t i = begin + tid; i < end; i += kBulkThreads) {
            const uint32_t s = other[i];
            order[begin + next_place(sub, (key[s] - least) >> cut)] = s;
        }
        __syncthreads();
        for (uint32_t i = begin + tid; i < end; i += kBulkThreads) {
            const uint32_t s = order[i], x = (key[s] - least) >> cut, first = begin + (x ? half_word(sub, x - 1) : 0u),
                           count = begin + half_word(sub, x) - first;
            other[count > kCompareMost ? i : first + rank(order + first, count, s)] = s;
        }
        __syncthreads();
        for (uint32_t i = begin + tid; i < end; i += kBulkThreads) order[i] = other[i];
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

// x, y as three bf16 pairs whose sum is x, y: eight leading bits at a time, cut
// off and not rounded, so that 24 bits take three and nothing overflows.
__device__ __forceinline__ void split3(float x, float y, uint32_t (&o)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const uint32_t hx = __float_as_uint(x) & 0xffff0000u, hy = __float_as_uint(y) & 0xffff0000u;
        o[i] = __byte_perm(hx, hy, 0x7632);
        x -= __uint_as_float(hx);
        y -= __uint_as_float(hy);
        if (i == 0) {  // an infinity (or NaN) has no rest
            x = x == x ? x : 0.f;
            y = y == y ? y : 0.f;
        }
    }
}

// The same sum for four neighbours of one row of A, pair after pair in float32: for
// what is not finite.  It ends once all four are NaN, which no pair changes.
template <typename T, int D>
__device__ __noinline__ float4 sum_of_products(const T *kp, const T *vp, const uint32_t *order, const float *factor, int m, int r, int col) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < m; ++i) {
        const T *v = vp + (int64_t)order[i] * D + col;
        const float wk = factor[i] * to_f32(kp[(int64_t)order[i] * D + r]);
        a.x = fmaf(wk, to_f32(v[0]), a.x);
        a.y = fmaf(wk, to_f32(v[1]), a.y);
        a.z = fmaf(wk, to_f32(v[2]), a.z);
        a.w = fmaf(wk, to_f32(v[3]), a.w);
        if (a.x != a.x && a.y != a.y && a.z != a.z && a.w != a.w) break;
    }
    return a;
}

// Shared memory of one block: the order of the pairs, then, one after the
// other in the same room, what sorting needs (keys, positions, a second order,
// counts), what the sum needs (raw tiles, parts; its result), and the lists of
// moves.
template <typename T, int D>
struct BulkShape {
    static constexpr bool F32 = sizeof(T) == 4;
    static constexpr int TP = F32 ? 32 : 64;                // pairs per tile
    static constexpr int STAGES = 4;
    static constexpr int ROW = D * (int)sizeof(T) + 16;     // bytes of a row, padded: no bank conflicts
    static constexpr int RAW = TP * 2 * ROW;                // keys, then values
    static constexpr int SUM = STAGES * RAW;                // at least the result's 4 D^2
    // A's tiles of 16 x 8: a warp takes one row of tiles (or half of one, at
    // most 8), and one of KG parts of the pairs
    static constexpr int TM = D / 16, TN = D / 8, NW = TN > 8 ? TN / 8 : 1, NT = TN / NW;
    static constexpr int KS = TP / 16;                      // steps of 16 pairs in a tile
    static constexpr int KG = kBulkWarps / (TM * NW) < KS ? kBulkWarps / (TM * NW) : KS;
    static_assert(kSortMax <= 17 * kBulkThreads, "sorted in registers");
    static_assert(SUM >= 4 * D * D && KS % KG == 0, "the block's sum has to fit");
};

// Bytes of sorting room for up to n pairs (a multiple of 32): keys, positions,
// second order; and the counts.
__host__ __device__ constexpr size_t sort_room(size_t n) { return 12 * n + 16 * kBulkThreads * 4; }
// What stays through all of it: the order (later the pairs' pool rows), the
// weights in the sum, a bit per slot.
__host__ __device__ constexpr size_t order_room(size_t n) { return (8 * n + n / 8 + 127) / 128 * 128; }

template <typename T, int D, int SL>
__global__ void __launch_bounds__(kBulkThreads, D <= 64 ? 2 : 1) evict_bulk_kernel(const __grid_constant__ EvictParams p, int n_cap) {
    using S = BulkShape<T, D>;
    extern __shared__ __align__(128) unsigned char dyn[];
    __shared__ int s_scan[kBulkWarps];
    __shared__ uint32_t s_total[32], s_base[kBulkWarps][32], s_bits[7][kBulkWarps];
    __shared__ uint64_t s_pick[2][kBulkWarps];
    __shared__ float s_pow[64 + kSortMax / 64];
    __shared__ uint32_t s_pick_slot[2][kBulkWarps];

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
    const size_t room = inside ? n_cap : pairs_room(c.capacity());
    unsigned char *kept = inside ? dyn : p.sort_ws + (bh * SL + rank) * (order_room(room) + sort_room(room));
    unsigned char *scratch = kept + order_room(room);     // sorting and lists
    unsigned char *tiles_mem = dyn + order_room(n_cap);   // the sum
    uint32_t *order = reinterpret_cast<uint32_t *>(kept), *bits = order + 2 * room;
    float *factor = reinterpret_cast<float *>(order + room);
    uint32_t *weight = reinterpret_cast<uint32_t *>(scratch), *place = weight + room, *other = place + room;
    uint32_t *counts = other + room;
    const int words = (n + 31) / 32;
    {
        const int64_t protect_from = c.clock[b] - p.recent;
        bool sorted = true;  // by position already, as tokens are appended
        uint32_t w_or = 0, w_and = ~0u, z_or = 0, z_and = ~0u;  // bits that differ between pairs
        uint32_t w_lo = ~0u, w_hi = 0, w_min = ~0u;             // least above zero, greatest, least
        constexpr int U = 8;
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
                    w_or |= weight[s];
                    w_and &= weight[s];
                    z_or |= place[s];
                    z_and &= place[s];
                    w_min = min(w_min, weight[s]);
                    w_hi = max(w_hi, weight[s]);
                    if (weight[s] != 0x80000000u) w_lo = min(w_lo, weight[s]);
                }
            }
        }
        for (int s = tid; s < words; s += kBulkThreads) bits[s] = 0;
        __syncthreads();
        for (int s = tid; s + 1 < n; s += kBulkThreads)
            sorted = sorted && (place[s] & 0x7fffffffu) <= (place[s + 1] & 0x7fffffffu);
        const bool by_place = !__syncthreads_and(sorted);
        w_or = __reduce_or_sync(0xffffffffu, w_or);
        w_and = __reduce_and_sync(0xffffffffu, w_and);
        z_or = __reduce_or_sync(0xffffffffu, z_or);
        z_and = __reduce_and_sync(0xffffffffu, z_and);
        w_lo = __reduce_min_sync(0xffffffffu, w_lo);
        w_min = __reduce_min_sync(0xffffffffu, w_min);
        w_hi = __reduce_max_sync(0xffffffffu, w_hi);
        if (lane == 0) {
            s_bits[0][warp] = w_or;
            s_bits[1][warp] = ~w_and;
            s_bits[2][warp] = z_or;
            s_bits[3][warp] = ~z_and;
            s_bits[4][warp] = ~w_lo;
            s_bits[5][warp] = ~w_min;
            s_bits[6][warp] = w_hi;
        }
        __syncthreads();
        uint32_t differ[4] = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kBulkWarps; ++w)
#pragma unroll
            for (int i = 0; i < 4; ++i) differ[i] |= s_bits[i][w];
        const uint32_t mine = lane < kBulkWarps ? s_bits[4][lane] : 0u, low = lane < kBulkWarps ? s_bits[5][lane] : 0u;
        w_lo = ~__reduce_max_sync(0xffffffffu, mine);
        w_min = ~__reduce_max_sync(0xffffffffu, low);
        w_hi = __reduce_max_sync(0xffffffffu, lane < kBulkWarps ? s_bits[6][lane] : 0u);
        const uint32_t w_differ = differ[0] & differ[1], z_differ = differ[2] & differ[3];
        const uint32_t *from = order;
        if (m <= kPickMax && n <= 32 * kBulkThreads) {
            // few leave: the first of what is left, m times; each thread knows the
            // first of its own slots
            uint32_t gone = 0, slot;
            uint64_t first;
            auto look = [&]() {
                first = ~0ull;
                slot = 0xffffffffu;
                for (int s = tid, j = 0; s < n; s += kBulkThreads, ++j) {
                    const uint64_t key = (uint64_t)(place[s] >> 31) << 63 | (uint64_t)weight[s] << 31 | (place[s] & 0x7fffffffu);
                    if (!(gone >> (j & 31) & 1u) && less_pair(key, (uint32_t)s, first, slot)) {
                        first = key;
                        slot = (uint32_t)s;
                    }
                }
            };
            // the least (key, slot) of the lanes
            auto least = [&](uint64_t &k, uint32_t &s) {
                const uint32_t hi = __reduce_min_sync(0xffffffffu, (uint32_t)(k >> 32));
                const uint32_t lo = __reduce_min_sync(0xffffffffu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0xffffffffu);
                s = __reduce_min_sync(0xffffffffu, (uint32_t)(k >> 32) == hi && (uint32_t)k == lo ? s : 0xffffffffu);
                k = (uint64_t)hi << 32 | lo;
            };
            look();
            for (int i = 0; i < m; ++i) {
                uint64_t k = first;
                uint32_t s = slot;
                least(k, s);
                if (lane == 0) {
                    s_pick[i & 1][warp] = k;
                    s_pick_slot[i & 1][warp] = s;
                }
                __syncthreads();
                k = lane < kBulkWarps ? s_pick[i & 1][lane] : ~0ull;
                s = lane < kBulkWarps ? s_pick_slot[i & 1][lane] : 0xffffffffu;
                least(k, s);
                if ((int)(s % kBulkThreads) == tid) {
                    other[i] = s;
                    gone |= 1u << (s / kBulkThreads);
                    look();
                }
            }
            __syncthreads();
            from = other;
        } else if (inside) {
            // the same addresses, from the block's own shared memory, so that they
            // are accessed as such
            uint32_t *o = reinterpret_cast<uint32_t *>(dyn), *w = reinterpret_cast<uint32_t *>(dyn + order_room(n_cap));
            const bool spread = w_min >= 0x80000000u && w_differ;  // no weight below zero, two values
            auto sort = [&](auto items) {
                return sort_slots<decltype(items)::value>(o, w + 2 * n_cap, w, w + n_cap, n, by_place, w_differ, z_differ, w + 3 * n_cap, s_total, s_base);
            };
            from = spread && bucket_sort(o, w + 2 * n_cap, w, w + n_cap, n, m, w_lo, w_hi, w + 3 * n_cap, s_scan) ? o
                   : n <= kBulkThreads     ? sort(std::integral_constant<int, 1>())
                   : n <= 3 * kBulkThreads ? sort(std::integral_constant<int, 3>())
                   : n <= 5 * kBulkThreads ? sort(std::integral_constant<int, 5>())
                   : n <= 9 * kBulkThreads ? sort(std::integral_constant<int, 9>())
                                           : sort(std::integral_constant<int, 17>());
        } else {
            from = sort_slots<0>(order, other, weight, place, n, by_place, w_differ, z_differ, counts, s_total, s_base);
        }
        // the pairs that leave: marked, and from here on named by their pool rows
        // (rows sorted in shared memory: lambda^(m-1-i) from its powers below 64 and of 64)
        const Decay decay(c.A ? c.lam[h] : 1.f);
        if (inside)
            for (int x = tid; x < 64 + kSortMax / 64; x += kBulkThreads) s_pow[x] = decay.pow(x < 64 ? x : (int64_t)(x - 64) * 64);
        __syncthreads();
        for (int i = tid; i < m; i += kBulkThreads) {
            const uint32_t s = from[i];
            const int e = m - 1 - i;
            atomicOr(&bits[s / 32], 1u << (s % 32));
            factor[i] = inside ? s_pow[e & 63] * s_pow[64 + (e >> 6)] : decay.pow(e);
            order[i] = (uint32_t)row_of((int)s);
        }
        __syncthreads();
    }

    // ---- A: lambda^m A + eta sum of lambda^(m-1-i) k_i v_i^T -------------------------
    if (c.A) {
        const int wm = warp % S::TM, wn = warp / S::TM % S::NW * S::NT, kg = warp / (S::TM * S::NW);
        float sum[S::NT][4];
#pragma unroll
        for (int t = 0; t < S::NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[t][e] = 0.f;
        const int all = (m + S::TP - 1) / S::TP, tiles = (all - rank + SL - 1) / SL;  // every SL-th is this block's
        auto fetch = [&](int tile) {
            if (tile < tiles) {
                unsigned char *raw = tiles_mem + (tile % S::STAGES) * S::RAW;
                constexpr int RC = D * (int)sizeof(T) / 16, EL = 16 / (int)sizeof(T);  // chunks of a row, elements of one
#pragma unroll
                for (int x0 = 0; x0 < S::TP * 2 * RC; x0 += kBulkThreads) {
                    const int x = x0 + tid, pr = x / (2 * RC), ch = x % (2 * RC);
                    if (S::TP * 2 * RC % kBulkThreads != 0 && pr >= S::TP) break;
                    const int i = (tile * SL + rank) * S::TP + pr;
                    unsigned char *dst = raw + ((ch < RC ? 0 : S::TP) + pr) * S::ROW + ch % RC * 16;
                    if (i < m) copy16(dst, (ch < RC ? kp : vp) + (int64_t)order[i] * D + ch % RC * EL);
                    else zero16(dst);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");  // an empty group past the last tile
        };
        for (int i = 0; i < S::STAGES - 1; ++i) fetch(i);
        for (int tile = 0; tile < tiles; ++tile) {
            asm volatile("cp.async.wait_group %0;" ::"n"(S::STAGES - 2) : "memory");
            __syncthreads();  // the tile is there; the last tile's buffer is free
            fetch(tile + S::STAGES - 1);
            const unsigned char *keys = tiles_mem + (tile % S::STAGES) * S::RAW, *values = keys + S::TP * S::ROW;
            if (kg < S::KG) {
                float acc[S::NT][4];
#pragma unroll
                for (int t = 0; t < S::NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[t][e] = 0.f;
#pragma unroll
                for (int kk = 0; kk < S::KS / S::KG; ++kk) {
                    const int k0 = (kg * (S::KS / S::KG) + kk) * 16, p0 = k0 + lane % 4 * 2;  // this lane's pairs: p0, +1, +8, +9
                    float w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = (tile * SL + rank) * S::TP + p0 + (e & 1) + (e >> 1) * 8;
                        w[e] = i < m ? factor[i] : 0.f;
                    }
                    // the weighted keys, transposed (rows of A by pairs), in three parts
                    uint32_t a[3][4];
                    uint32_t raw[4];
                    if (!S::F32) ldsm_t4(keys + (k0 + (lane & 7) + (lane >> 4) * 8) * S::ROW + (wm * 16 + ((lane >> 3) & 1) * 8) * 2, raw);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        float x, y;  // row lane / 4 (+ 8), pairs p0, p0 + 1 (+ 8)
                        if (S::F32) {
                            const unsigned char *at = keys + (p0 + (r >> 1) * 8) * S::ROW + (wm * 16 + lane / 4 + (r & 1) * 8) * 4;
                            x = *reinterpret_cast<const float *>(at);
                            y = *reinterpret_cast<const float *>(at + S::ROW);
                        } else {
                            x = __uint_as_float(raw[r] << 16);
                            y = __uint_as_float(raw[r] & 0xffff0000u);
                        }
                        uint32_t o[3];
                        split3(w[(r >> 1) * 2] * x, w[(r >> 1) * 2 + 1] * y, o);
                        a[0][r] = o[0];
                        a[1][r] = o[1];
                        a[2][r] = o[2];
                    }
                    if (S::F32) {
#pragma unroll
                        for (int t = 0; t < S::NT; ++t) {
                            const unsigned char *at = values + p0 * S::ROW + ((wn + t) * 8 + lane / 4) * 4;
                            uint32_t v[3][2];
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                uint32_t o[3];
                                split3(*reinterpret_cast<const float *>(at + r * 8 * S::ROW), *reinterpret_cast<const float *>(at + (r * 8 + 1) * S::ROW), o);
                                v[0][r] = o[0];
                                v[1][r] = o[1];
                                v[2][r] = o[2];
                            }
#pragma unroll
                            for (int j = 2; j >= 0; --j)
#pragma unroll
                                for (int i = 2 - j; i >= 0; --i) mma_bf16(acc[t], a[i], v[j]);
                        }
                    } else {
#pragma unroll
                        for (int t = 0; t < S::NT; t += 2) {
                            uint32_t v[4];  // two tiles' values
                            ldsm_t4(values + (k0 + (lane & 7) + ((lane >> 3) & 1) * 8) * S::ROW + ((wn + t) * 8 + (lane >> 4) * 8) * 2, v);
                            const uint32_t v0[2] = {v[0], v[1]}, v1[2] = {v[2], v[3]};
#pragma unroll
                            for (int i = 2; i >= 0; --i) {
                                mma_bf16(acc[t], a[i], v0);
                                mma_bf16(acc[t + 1], a[i], v1);
                            }
                        }
                    }
                }
#pragma unroll
                for (int t = 0; t < S::NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[t][e] += acc[t][e];
            }
        }
        // the parts of the pairs, added; then the blocks' sums
        float *mine = reinterpret_cast<float *>(tiles_mem);  // [D][D]
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        for (int g = 0; g < S::KG; ++g) {
            __syncthreads();
            if (kg == g) {
#pragma unroll
                for (int t = 0; t < S::NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        float2 *x = reinterpret_cast<float2 *>(mine + (wm * 16 + lane / 4 + e * 4) * D + (wn + t) * 8 + lane % 4 * 2);
                        const float2 o = g ? *x : make_float2(0.f, 0.f);
                        *x = make_float2(o.x + sum[t][e], o.y + sum[t][e + 1]);
                    }
            }
        }
        if (SL > 1) cluster_sync();
        else __syncthreads();
        const float lm = Decay(c.lam[h]).pow(m), eta = c.eta[h];
        for (int at = rank * kBulkThreads + tid; at < D * D / 4; at += SL * kBulkThreads) {  // this block's share of A
            float4 add = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int r = 0; r < SL; ++r) {
                float4 y;
                if (SL > 1) {
                    uint32_t there;
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(sm100::smem_u32(mine + at * 4)), "r"(r));
                    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(y.x), "=f"(y.y), "=f"(y.z), "=f"(y.w) : "r"(there) : "memory");
                } else {
                    y = reinterpret_cast<const float4 *>(mine)[at];
                }
                add.x += y.x;
                add.y += y.y;
                add.z += y.z;
                add.w += y.w;
            }
            // a key's or value's second and third parts may be 0, and 0 * inf is NaN
            // where the pair's own product is infinite: what came out as NaN is summed
            // again from whole values
            if (add.x != add.x || add.y != add.y || add.z != add.z || add.w != add.w)
                add = sum_of_products<T, D>(kp, vp, order, factor, m, at / (D / 4), at % (D / 4) * 4);
            float4 *dst = reinterpret_cast<float4 *>(c.A + bh * D * D) + at;
            float4 o = *dst;
            o.x = fmaf(lm, o.x, eta * add.x);
            o.y = fmaf(lm, o.y, eta * add.y);
            o.z = fmaf(lm, o.z, eta * add.z);
            o.w = fmaf(lm, o.w, eta * add.w);
            *dst = o;
        }
        if (SL > 1) cluster_sync();  // the sums have been read: their room is free
    }

    // ---- freed slots below keep, and the pairs behind it that stay ------------------
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
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = cluster_launch(attr, (int64_t)p.c.B * p.c.H * slices, kOneThreads, 0, slices, false, s);
    return cudaLaunchKernelEx(&cfg, evict_one_kernel<T, D, STEP>, p, slices);
}

// Shared memory of a bulk eviction of rows of up to n2 pairs.
template <typename T, int D>
constexpr size_t bulk_smem(int n2) {
    const size_t sum = BulkShape<T, D>::SUM, sort = sort_room(n2);
    return order_room(n2) + (sum > sort ? sum : sort);
}

// The kernel's leave to use that much is state of the process: it is granted for
// the longest rows, and once per device, so that no call lowers what another
// thread's is about to use.  Before a call's first kernel, so that a refusal leaves
// the cache as it was.
template <typename T, int D, int SL>
cudaError_t grant_bulk() {
    static std::atomic<uint64_t> granted{0};  // a bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (granted.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = allow_smem(evict_bulk_kernel<T, D, SL>, bulk_smem<T, D>(kSortMax));
    if (e == cudaSuccess) granted.fetch_or(bit, std::memory_order_release);
    return e;
}

template <typename T, int D, int SL>
cudaError_t launch_bulk(const EvictParams *launch, cudaStream_t s) {
    if (!launch) return grant_bulk<T, D, SL>();
    const EvictParams &p = *launch;
    const int64_t cap = pairs_room(p.c.capacity());
    const int n2 = (int)(cap < kSortMax ? cap : kSortMax);  // pairs sorted in shared memory
    const size_t smem = bulk_smem<T, D>(n2);
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = cluster_launch(attr, (int64_t)p.c.B * p.c.H * SL, kBulkThreads, smem, SL, true, s);
    return cudaLaunchKernelEx(&cfg, evict_bulk_kernel<T, D, SL>, p, n2);
}

// (p null: the grant alone)
template <typename T, int D>
cudaError_t launch_bulk_sl(const EvictParams *p, int slices, cudaStream_t s) {
    if constexpr (D >= 64)
        if (slices == 4) return launch_bulk<T, D, 4>(p, s);
    if constexpr (D >= 32)
        if (slices == 2) return launch_bulk<T, D, 2>(p, s);
    return launch_bulk<T, D, 1>(p, s);
}

template <typename T>
cudaError_t launch_bulk_d(const EvictParams *p, int d, int slices, cudaStream_t s) {
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

}  // namespace

cudaError_t launch_cache_append(const AppendParams &p, tc_dtype dtype, cudaStream_t s) {
    if (p.T == 0) return cudaSuccess;
    const int64_t es = dtype == TC_BF16 ? 2 : 4;
    const int vec = (int)(16 / es);
    const int64_t qn[3] = {p.c.B, p.Hq, p.T}, kn[3] = {p.c.B, p.c.H, p.T};
    // 16-byte vectors where addresses and strides allow (2047 tokens for 8 rows, 12
    // heads of d = 64, bf16: 23 us; element by element 62)
    const bool wide = p.table.rot % (2 * vec) == 0 && rows_aligned16(p.k, p.ks, kn, es) &&
                      rows_aligned16(p.v, p.vs, kn, es) && (!p.q || rows_aligned16(p.q, p.qs, qn, es));
    if (dtype == TC_BF16)
        return wide ? launch_append_vec<__nv_bfloat16, 8>(p, s) : launch_append_vec<__nv_bfloat16, 1>(p, s);
    return wide ? launch_append_vec<float, 4>(p, s) : launch_append_vec<float, 1>(p, s);
}

// Slices a head's A is cut into, one block of a cluster each: where A is large,
// 2 or 4 while the device has room for them.  (A step of one row of 2048 pairs, 8
// heads for 64, d = 128: 21.2 us with 4 slices, 23.3 with one; an eviction from 12
// heads of d = 64: 8.2 us with 4 slices, 7.6 with one.)
int evict_slices(int64_t BH, int d, int num_sms) {
    return d < 128 ? 1 : BH * 4 <= 2 * num_sms ? 4 : BH * 2 <= 2 * num_sms ? 2 : 1;
}

namespace {
// Blocks that share a head's pairs: 1, 2 or 4 (2 for the narrow heads, whose sums
// are short), while all still run at once: two on an SM up to d = 64, one at 128.
// 2047 of 2559 pairs: 12 heads of d = 64 with 4 blocks 37 us, with one 60; 8 of d =
// 128 with 4 blocks 54 us, with one 124; 96 of d = 64 with 2 blocks 65 us, with one
// 93, with 4 (in two waves) 83.
int bulk_slices(int64_t BH, int d, int num_sms) {
    const int64_t room = (int64_t)(d <= 64 ? 2 : 1) * num_sms;
    return BH * 4 <= room && d >= 64 ? 4 : BH * 2 <= room && d >= 32 ? 2 : 1;
}
}  // namespace

size_t evict_sort_bytes(int64_t BH, int d, int64_t capacity, int num_sms) {
    const int64_t n2 = pairs_room(capacity);
    return n2 <= kSortMax ? 0 : (size_t)BH * (size_t)bulk_slices(BH, d, num_sms) * (order_room(n2) + sort_room(n2));
}

cudaError_t launch_cache_step_insert(const EvictParams &p, tc_dtype dtype, int d, int slices, cudaStream_t s) {
    return dtype == TC_BF16 ? launch_one_d<__nv_bfloat16, true>(p, d, slices, s) : launch_one_d<float, true>(p, d, slices, s);
}

cudaError_t launch_cache_evict(const EvictParams &p, tc_dtype dtype, int d, int num_sms, cudaStream_t s) {
    const int64_t BH = (int64_t)p.c.B * p.c.H;
    const int one = evict_slices(BH, d, num_sms), bulk = bulk_slices(BH, d, num_sms);
    auto bulk_call = [&](const EvictParams *launch) {
        return dtype == TC_BF16 ? launch_bulk_d<__nv_bfloat16>(launch, d, bulk, s) : launch_bulk_d<float>(launch, d, bulk, s);
    };
    cudaError_t e = bulk_call(nullptr);
    if (e != cudaSuccess) return e;
    e = dtype == TC_BF16 ? launch_one_d<__nv_bfloat16, false>(p, d, one, s) : launch_one_d<float, false>(p, d, one, s);
    return e != cudaSuccess ? e : bulk_call(&p);
}

}  // namespace tc

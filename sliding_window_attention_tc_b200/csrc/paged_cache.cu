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
// its own (no exchange) and writes its own slice of A's rows.  m = 1, the
// steady state, is an arg-min over the weights beside one pass over A, which is
// what bounds it: 8 d^2 bytes of A, plus 8 n of weights and positions.  m > 1
// sorts the weights in shared memory and forms the sum tile by tile.

#include <cooperative_groups.h>

#include "paged_cache.cuh"

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

constexpr int kEvThreads = 256;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kSortMax = 8192;   // pairs sorted in shared memory (12 bytes each)
constexpr int kPairTile = 32;    // pairs per step of the weighted sum
constexpr int kQBatch = 4;       // query heads per pass over A's registers

// The order in which pairs leave, as one number: unprotected first, then by
// weight (NaN last, -0 as 0), then by position.
__device__ __forceinline__ uint64_t leave_key(float mass, int32_t pos, int64_t protect_from) {
    uint32_t u = __float_as_uint(mass + 0.f);
    u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    if (mass != mass) u = 0xffffffffu;
    return ((uint64_t)(pos >= protect_from) << 63) | ((uint64_t)u << 31) | (uint32_t)(pos & 0x7fffffff);
}

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

__device__ __forceinline__ bool less_pair(uint64_t ka, uint32_t sa, uint64_t kb, uint32_t sb) {
    return ka < kb || (ka == kb && sa < sb);
}

// Bitonic sort of n2 (a power of two) keys with their slots, ascending.
__device__ void block_sort(uint64_t *key, uint32_t *slot, int n2) {
    for (int size = 2; size <= n2; size *= 2) {
        for (int stride = size / 2; stride > 0; stride /= 2) {
            __syncthreads();
            for (int i = threadIdx.x; i < n2 / 2; i += kEvThreads) {
                const int lo = 2 * i - (i & (stride - 1)), hi = lo + stride;
                const bool up = (lo & size) == 0;
                const uint64_t ka = key[lo], kb = key[hi];
                const uint32_t sa = slot[lo], sb = slot[hi];
                if (less_pair(kb, sb, ka, sa) == up) {
                    key[lo] = kb;
                    key[hi] = ka;
                    slot[lo] = sb;
                    slot[hi] = sa;
                }
            }
        }
    }
    __syncthreads();
}

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
    for (int w = 0; w < kEvWarps; ++w) {
        if (w < warp) before += warp_sums[w];
        all += warp_sums[w];
    }
    *total = all;
    return before + v - x;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <typename T, int D, bool STEP>
__global__ void __launch_bounds__(kEvThreads) evict_kernel(const __grid_constant__ EvictParams p, int slices, int n2_cap) {
    constexpr int CG = D / 4;                 // float4 columns of A
    constexpr int RG = kEvThreads / CG;       // rows of A the block holds side by side
    constexpr int RPT = (D + RG - 1) / RG;    // rows per thread of a whole A
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ float s_k[D], s_v[D], s_cos[D / 2 + 1], s_sin[D / 2 + 1];
    __shared__ uint64_t s_key[kEvWarps];
    __shared__ uint32_t s_slot[kEvWarps];
    __shared__ int s_scan[kEvWarps];
    __shared__ float s_q[kQBatch][D];
    __shared__ __align__(16) float s_mp[RG][kQBatch][D];

    const CacheParams &c = p.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = blockIdx.x % slices;
    const int64_t bh = blockIdx.x / slices;
    const int b = (int)(bh / c.H), h = (int)(bh % c.H);
    const int64_t held = c.len[b], clock0 = c.clock[b];
    const bool first = h == 0 && rank == 0 && tid == 0;
    if (held < 0) {
        if (first) p.row_len[b] = -1;
        return;
    }
    const int64_t n64 = held + (STEP ? 1 : 0);
    bool ok = held <= c.capacity() && n64 <= c.capacity() &&
              (!STEP || (clock0 >= 0 && clock0 < (int64_t(1) << 31)));
    if (ok) ok = block_pages_ok(c, b, 0, n64 - 1);
    if (!ok) {
        if (first) {
            p.row_len[b] = -1;
            report(c.status, TC_ERR_DEVICE_BOUNDS);
        }
        return;
    }
    const int n = (int)n64;
    const int m = n64 > p.budget ? (int)(n64 - p.budget) : 0;
    const int keep = n - m;
    const int64_t clock = clock0 + (STEP ? 1 : 0);
    if (first) p.row_len[b] = keep;
    const int32_t *table = c.table + (int64_t)b * c.max_pages;
    auto row_of = [&](int slot) { return pool_row(c, table[slot / c.page], h, slot % c.page); };
    T *kp = reinterpret_cast<T *>(c.k), *vp = reinterpret_cast<T *>(c.v);

    // this block's slice of A's rows, read while the weights are looked through
    const int rows = D / slices, row0 = rank * rows;
    const bool read = STEP && p.memo != nullptr;
    const bool simple = m <= 1;
    const int cg = tid % CG, rg = tid / CG;
    float4 *A4 = c.A ? reinterpret_cast<float4 *>(c.A + (bh * D + row0) * D) : nullptr;
    float4 a[RPT];
    if (A4 && simple && (m == 1 || read)) {
#pragma unroll
        for (int i = 0; i < RPT; ++i)
            if (rg + i * RG < rows) a[i] = A4[(rg + i * RG) * CG + cg];
    }

    if (STEP) {
        // the new pair enters slot n - 1 (every block of the cluster writes the
        // same values), the queries are rotated
        const RotaryTable &rt = p.table;
        for (int i = tid; i < rt.rot / 2; i += kEvThreads) rotary_angle(clock0, rt.inc[i], rt.gain, s_cos[i], s_sin[i]);
        __syncthreads();
        const int64_t row = row_of(n - 1);
        const int G = p.Hq / c.H;
        for (int x = tid; x < (G + 2) * D; x += kEvThreads) {
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
                const int pair = rt.interleaved ? i / 2 : i % half;
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
    if (m == 0 && !read) return;  // the whole cluster

    const int64_t protect_from = clock - p.recent;
    const float lam = c.A ? c.lam[h] : 0.f, eta = c.A ? c.eta[h] : 0.f;
    // lists for m > 1: the pairs that leave, in order, and the moves
    int moves = 0;
    int *hole = nullptr, *fill = nullptr;
    int gone = 0;  // m == 1: the slot that leaves

    if (m == 1) {
        uint64_t best = ~0ull;
        uint32_t slot = 0xffffffffu;
        for (int s = tid; s < n; s += kEvThreads) {
            const int64_t row = row_of(s);
            const uint64_t key = leave_key(c.mass[row], c.pos[row], protect_from);
            if (less_pair(key, (uint32_t)s, best, slot)) {
                best = key;
                slot = (uint32_t)s;
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
        for (int w = 0; w < kEvWarps; ++w)
            if (w == 0 || less_pair(s_key[w], s_slot[w], best, slot)) {
                best = s_key[w];
                slot = s_slot[w];
            }
        gone = (int)slot;
        if (A4) {
            const int64_t row = row_of(gone);
            for (int i = tid; i < D; i += kEvThreads) {
                s_k[i] = to_f32(kp[row * D + i]);
                s_v[i] = to_f32(vp[row * D + i]);
            }
            __syncthreads();
            const float4 v4 = reinterpret_cast<const float4 *>(s_v)[cg];
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const int r = rg + i * RG;
                if (r < rows) {
                    const float ek = eta * s_k[row0 + r];
                    a[i].x = fmaf(lam, a[i].x, ek * v4.x);
                    a[i].y = fmaf(lam, a[i].y, ek * v4.y);
                    a[i].z = fmaf(lam, a[i].z, ek * v4.z);
                    a[i].w = fmaf(lam, a[i].w, ek * v4.w);
                    A4[r * CG + cg] = a[i];
                }
            }
        }
    } else if (m > 1) {
        // ---- the order of leaving ------------------------------------------------
        int n2 = 1;
        while (n2 < n) n2 *= 2;
        unsigned char *ws = n2 <= n2_cap ? dyn : p.sort_ws + bh * ((size_t)n2_cap_global(c.capacity()) * 13);
        const int n2_room = n2 <= n2_cap ? n2_cap : n2_cap_global(c.capacity());
        uint64_t *key = reinterpret_cast<uint64_t *>(ws);
        uint32_t *slot = reinterpret_cast<uint32_t *>(ws + (size_t)n2_room * 8);
        uint32_t *bits = reinterpret_cast<uint32_t *>(ws + (size_t)n2_room * 12);
        const int words = (n + 31) / 32;
        for (int s = tid; s < n2; s += kEvThreads) {
            uint64_t x = ~0ull;
            if (s < n) {
                const int64_t row = row_of(s);
                x = leave_key(c.mass[row], c.pos[row], protect_from);
            }
            key[s] = x;
            slot[s] = s < n ? (uint32_t)s : 0xffffffffu;
        }
        for (int s = tid; s < words; s += kEvThreads) bits[s] = 0;
        block_sort(key, slot, n2);

        // ---- A's slice: lambda^m A + eta sum of lambda^(m-1-i) k_i v_i^T ----------
        if (A4) {
            const Decay decay(lam);
            float *tk = reinterpret_cast<float *>(dyn + (size_t)n2_cap * 13);  // [kPairTile][rows] weighted keys
            float *tv = tk + kPairTile * rows;                                 // [kPairTile][D]
            float4 acc[RPT];
#pragma unroll
            for (int i = 0; i < RPT; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int i0 = 0; i0 < m; i0 += kPairTile) {
                const int np = min(kPairTile, m - i0);
                __syncthreads();
                for (int x = tid; x < np * (rows + D); x += kEvThreads) {
                    const int pr = x / (rows + D), e = x % (rows + D);
                    const int64_t row = row_of((int)slot[i0 + pr]);
                    if (e < rows)
                        tk[pr * rows + e] = eta * decay.pow(m - 1 - (i0 + pr)) * to_f32(kp[row * D + row0 + e]);
                    else
                        tv[pr * D + e - rows] = to_f32(vp[row * D + e - rows]);
                }
                __syncthreads();
                for (int pr = 0; pr < np; ++pr) {
                    const float4 v4 = reinterpret_cast<const float4 *>(tv + pr * D)[cg];
#pragma unroll
                    for (int i = 0; i < RPT; ++i) {
                        const int r = rg + i * RG;
                        if (r < rows) {
                            const float w = tk[pr * rows + r];
                            acc[i].x = fmaf(w, v4.x, acc[i].x);
                            acc[i].y = fmaf(w, v4.y, acc[i].y);
                            acc[i].z = fmaf(w, v4.z, acc[i].z);
                            acc[i].w = fmaf(w, v4.w, acc[i].w);
                        }
                    }
                }
            }
            const float lm = decay.pow(m);
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const int r = rg + i * RG;
                if (r < rows) {
                    const float4 o = A4[r * CG + cg];
                    a[i].x = fmaf(lm, o.x, acc[i].x);
                    a[i].y = fmaf(lm, o.y, acc[i].y);
                    a[i].z = fmaf(lm, o.z, acc[i].z);
                    a[i].w = fmaf(lm, o.w, acc[i].w);
                    A4[r * CG + cg] = a[i];
                }
            }
        }

        // ---- freed slots below keep, and the pairs behind it that stay ------------
        for (int i = tid; i < m; i += kEvThreads) atomicOr(&bits[slot[i] / 32], 1u << (slot[i] % 32));
        __syncthreads();  // the keys are done with: their room takes the two lists
        hole = reinterpret_cast<int *>(key);
        fill = hole + n2_room;
        const int per = (words + kEvThreads - 1) / kEvThreads;
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
        int nh = 0, nf = 0, total;
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
    }

    // ---- q A for the step's queries, from the slice of A just written -------------
    if (read) {
        const int G = p.Hq / c.H;
        for (int g0 = 0; g0 < G; g0 += kQBatch) {
            const int ng = min(kQBatch, G - g0);
            __syncthreads();
            for (int x = tid; x < ng * rows; x += kEvThreads)
                s_q[x / rows][x % rows] = to_f32(reinterpret_cast<const T *>(p.q_rot)[(bh * G + g0 + x / rows) * D + row0 + x % rows]);
            __syncthreads();
#pragma unroll
            for (int g = 0; g < kQBatch; ++g) {
                float4 mp = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    const int r = rg + i * RG;
                    if (r < rows) {
                        const float w = g < ng ? s_q[g][r] : 0.f;
                        mp.x = fmaf(w, a[i].x, mp.x);
                        mp.y = fmaf(w, a[i].y, mp.y);
                        mp.z = fmaf(w, a[i].z, mp.z);
                        mp.w = fmaf(w, a[i].w, mp.w);
                    }
                }
                reinterpret_cast<float4 *>(&s_mp[rg][g][0])[cg] = mp;
            }
            __syncthreads();
            for (int x = tid; x < ng * D; x += kEvThreads) {
                float sum = 0.f;
#pragma unroll
                for (int r = 0; r < RG; ++r) sum += s_mp[r][x / D][x % D];
                p.memo[((bh * slices + rank) * G + g0) * D + x] = sum;
            }
        }
    }
    if (m == 0) return;  // the whole cluster

    // ---- moves, once every block of the cluster has read what they overwrite ------
    if (slices > 1) cluster_sync();
    else __syncthreads();
    if (m == 1) moves = gone < keep ? 1 : 0;
    constexpr int LPR = D * (int)sizeof(T) / 16;  // 16-byte vectors of a row
    for (int x = rank * kEvWarps + warp; x < moves; x += slices * kEvWarps) {
        const int64_t from = row_of(m == 1 ? keep : fill[x]), to = row_of(m == 1 ? gone : hole[x]);
        const uint4 *ks = reinterpret_cast<const uint4 *>(kp + from * D), *vs = reinterpret_cast<const uint4 *>(vp + from * D);
        uint4 *kd = reinterpret_cast<uint4 *>(kp + to * D), *vd = reinterpret_cast<uint4 *>(vp + to * D);
        for (int i = lane; i < 2 * LPR; i += 32) {
            if (i < LPR) kd[i] = ks[i];
            else vd[i - LPR] = vs[i - LPR];
        }
        if (lane == 0) {
            c.mass[to] = c.mass[from];
            c.pos[to] = c.pos[from];
        }
    }
}

__global__ void evict_finish_kernel(int64_t *len, const int64_t *row_len, int B) {
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b < B && row_len[b] >= 0) len[b] = row_len[b];
}

size_t evict_smem(int n2, int d, int slices) {
    return (size_t)n2 * 13 + (size_t)kPairTile * (d / slices + d) * sizeof(float);
}

template <typename T, int D, bool STEP>
cudaError_t launch_evict_t(const EvictParams &p, int slices, cudaStream_t s) {
    const int64_t cap = n2_cap_global(p.c.capacity());
    const int n2 = (int)(cap < kSortMax ? cap : kSortMax);
    const size_t smem = evict_smem(n2, D, slices);
    cudaError_t e = cudaFuncSetAttribute(evict_kernel<T, D, STEP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)slices;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)p.c.B * p.c.H * slices));
    cfg.blockDim = dim3(kEvThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_kernel<T, D, STEP>, p, slices, n2);
}

template <typename T, bool STEP>
cudaError_t launch_evict_d(const EvictParams &p, int d, int slices, cudaStream_t s) {
    switch (d) {
        case 16: return launch_evict_t<T, 16, STEP>(p, slices, s);
        case 32: return launch_evict_t<T, 32, STEP>(p, slices, s);
        case 64: return launch_evict_t<T, 64, STEP>(p, slices, s);
        case 128: return launch_evict_t<T, 128, STEP>(p, slices, s);
    }
    return cudaErrorInvalidValue;
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

// A slice has at least 16 rows of A; rows that sort in global memory stay whole
// (their workspace is per head).
int evict_slices(int64_t BH, int d, int64_t capacity, int num_sms) {
    int slices = 1;
    if (n2_cap_global(capacity) > kSortMax) return 1;
    while (slices * 2 <= d / 16 && slices < 8 && BH * slices * 2 <= 2 * num_sms) slices *= 2;
    return slices;
}

size_t evict_sort_bytes(int64_t BH, int64_t capacity) {
    const int64_t n2 = n2_cap_global(capacity);
    return n2 <= kSortMax ? 0 : (size_t)BH * (size_t)n2 * 13;
}

cudaError_t launch_cache_evict(const EvictParams &p, tc_dtype dtype, int d, bool step, int slices, cudaStream_t s) {
    if (dtype == TC_BF16)
        return step ? launch_evict_d<__nv_bfloat16, true>(p, d, slices, s) : launch_evict_d<__nv_bfloat16, false>(p, d, slices, s);
    return step ? launch_evict_d<float, true>(p, d, slices, s) : launch_evict_d<float, false>(p, d, slices, s);
}

cudaError_t launch_cache_evict_finish(const EvictParams &p, cudaStream_t s) {
    evict_finish_kernel<<<(p.c.B + 255) / 256, 256, 0, s>>>(p.c.len, p.row_len, p.c.B);
    return cudaGetLastError();
}

}  // namespace tc

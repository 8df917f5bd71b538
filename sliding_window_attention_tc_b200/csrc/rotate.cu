// tc_rotate: rotary positions of q and k, and their gradients.
//
// Pair i of a token at position p is turned by the angle p f'_i and scaled
// by gain; the backward is the transposed rotation.  Every element is read and
// written once: bound by memory.  One thread owns one chunk of 2 VEC elements
// (two 16-byte vectors) of one token and walks the heads, so the angles are
// formed once per token and some heads; what is under way is held as it came
// from memory (unpacked floats took the registers that more threads need: 53 us
// instead of 33 for the LM shape's q and k, 201 MB, bf16, 6.1 TB/s).

#include <cmath>

#include "rotary.cuh"

namespace tc {
namespace {

constexpr int kRotThreads = 128;
constexpr int kRotUnroll = 4;  // heads in flight per thread

template <typename T, int VEC, bool INTER>
__global__ void __launch_bounds__(kRotThreads, 5) rotate_kernel(const __grid_constant__ RotateParams p, int chunks,
                                                                      int heads_per_block) {
    const int64_t u = (int64_t)blockIdx.x * kRotThreads + threadIdx.x;
    if (u >= p.B * p.T * chunks) return;
    const int chunk = (int)(u % chunks);
    const int64_t bt = u / chunks, b = bt / p.T, t = bt - b * p.T;
    RotChunk<T, VEC, INTER> r;
    r.place(p.table, chunk, p.d);
    const int h0 = blockIdx.y * heads_per_block;
    const int h1 = min(h0 + heads_per_block, p.Hq + p.H);
    const T *q = reinterpret_cast<const T *>(p.q) + b * p.qs[0] + t * p.qs[2];
    const T *k = reinterpret_cast<const T *>(p.k) + b * p.ks[0] + t * p.ks[2];
    T *qo = reinterpret_cast<T *>(p.q_out) + b * p.qos[0] + t * p.qos[2];
    T *ko = reinterpret_cast<T *>(p.k_out) + b * p.kos[0] + t * p.kos[2];
    typename RotChunk<T, VEC, INTER>::Raw x[kRotUnroll], z[kRotUnroll];
    auto load = [&](int h) {
#pragma unroll
        for (int i = 0; i < kRotUnroll; ++i) {
            if (h + i < h1) {
                const T *src = h + i < p.Hq ? q + (h + i) * p.qs[1] : k + (h + i - p.Hq) * p.ks[1];
                r.load(src, x[i], z[i]);
            }
        }
    };
    load(h0);  // under way while the angles are formed
    r.angles(p.table, chunk, p.positions ? p.positions[bt] : p.t0 + t, p.backward);
    for (int h = h0;;) {
#pragma unroll
        for (int i = 0; i < kRotUnroll; ++i) {
            if (h + i < h1) {
                T *dst = h + i < p.Hq ? qo + (h + i) * p.qos[1] : ko + (h + i - p.Hq) * p.kos[1];
                r.store(dst, x[i], z[i], true);
            }
        }
        h += kRotUnroll;
        if (h >= h1) break;
        load(h);
    }
}

template <typename T, int VEC>
cudaError_t launch_vec(const RotateParams &p, int num_sms, cudaStream_t s) {
    const int chunks = (p.d + 2 * VEC - 1) / (2 * VEC), heads = p.Hq + p.H;
    const int64_t units = p.B * p.T * chunks;
    if (units == 0) return cudaSuccess;
    // few tokens: the heads are split too, at the price of forming the angles
    // again, until every SM has a full set of threads (32 + 8 heads of d = 128, 512
    // tokens: 4.3 us, unsplit 10.0; 12 + 12 heads of d = 64, 32768 tokens: 33.1 us
    // unsplit, as the rule has it, 34.5 split as far as it goes)
    const int64_t want = ((int64_t)num_sms * 2048 + units - 1) / units;
    const int most = (heads + kRotUnroll - 1) / kRotUnroll;
    const int split = (int)(want < most ? want : most);
    const int per = (heads + split - 1) / split;
    const dim3 grid((unsigned)((units + kRotThreads - 1) / kRotThreads), (unsigned)((heads + per - 1) / per));
    if (p.table.interleaved) rotate_kernel<T, VEC, true><<<grid, kRotThreads, 0, s>>>(p, chunks, per);
    else rotate_kernel<T, VEC, false><<<grid, kRotThreads, 0, s>>>(p, chunks, per);
    return cudaGetLastError();
}

}  // namespace

bool make_rotary_table(const tc_rotary *r, int64_t d, RotaryTable *out) {
    *out = RotaryTable{};
    if (!r) return true;
    if (r->rot < 0 || r->rot > d || r->rot % 2 || (r->interleaved != 0 && r->interleaved != 1)) return false;
    if (!(r->base > 1.0) || !(r->factor >= 1.0) || !(r->train_len >= 0.0)) return false;
    if (!std::isfinite(r->base) || !std::isfinite(r->factor) || !std::isfinite(r->train_len) ||
        !std::isfinite((float)r->gain) || !std::isfinite(r->low) || !std::isfinite(r->high))
        return false;
    out->rot = (int)r->rot;
    out->interleaved = (int)r->interleaved;
    out->gain = (float)r->gain;
    const long double to_turns = 1.0L / 6.283185307179586476925286766559L;
    const long double slow = 1.0L / (long double)r->factor;
    const bool ramp = r->high > r->low;
    const long double width = ramp ? 1.0L / ((long double)r->high - r->low) : 0.0L;
    // f_i by repeated products (63 at most, each off by 2^-64): a powl per
    // pair would cost more than the launch
    const long double ratio = out->rot ? powl((long double)r->base, -2.0L / (long double)r->rot) : 0.0L;
    long double f = 1.0L;
    for (int i = 0; i < out->rot / 2; ++i, f *= ratio) {
        long double keep = 0.0L;
        if (ramp) {
            keep = ((long double)r->train_len * f * to_turns - r->low) * width;
            keep = keep < 0.0L ? 0.0L : keep > 1.0L ? 1.0L : keep;
        }
        const long double turns = f * (keep + (1.0L - keep) * slow) * to_turns;  // at most 1/(2 pi)
        out->inc[i] = (uint64_t)(turns * 18446744073709551616.0L + 0.5L);
    }
    return true;
}

cudaError_t launch_rotate(const RotateParams &p, tc_dtype dtype, int num_sms, cudaStream_t s) {
    const int64_t es = dtype == TC_BF16 ? 2 : 4;
    const int vec = (int)(16 / es);
    const int64_t qn[3] = {p.B, p.Hq, p.T}, kn[3] = {p.B, p.H, p.T};
    // 16-byte vectors where sizes, addresses and strides allow (the LM shape's q and
    // k: 33 us; element by element 66; in float32, half the tokens, 33 and 42)
    bool wide = p.d % vec == 0 && p.table.rot % (2 * vec) == 0 && rows_aligned16(p.q, p.qs, qn, es) &&
                rows_aligned16(p.q_out, p.qos, qn, es);
    if (p.H) wide = wide && rows_aligned16(p.k, p.ks, kn, es) && rows_aligned16(p.k_out, p.kos, kn, es);
    if (dtype == TC_BF16)
        return wide ? launch_vec<__nv_bfloat16, 8>(p, num_sms, s) : launch_vec<__nv_bfloat16, 1>(p, num_sms, s);
    return wide ? launch_vec<float, 4>(p, num_sms, s) : launch_vec<float, 1>(p, num_sms, s);
}

}  // namespace tc

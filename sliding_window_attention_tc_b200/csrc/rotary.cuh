// Rotary positions: the per-frequency table and the rotation of one token's
// rows, shared by tc_rotate and the paged cache's insertions.
#pragma once

#include "tc_internal.cuh"

namespace tc {

// Turns per position of every pair, as 64-bit fractions of a turn: the angle
// of position p is p * inc[i] mod 2^64, exact in the position, so a far
// position costs no precision (a float32 product would have none left past
// 2^24, and a 64-bit one needs a range reduction).  Filled on the host.
struct RotaryTable {
    uint64_t inc[64];
    float gain;
    int rot;
    int interleaved;
};

// cos and sin (times gain) of position p at frequency inc.  The nearest
// quarter turn is taken off in integers; the rest, at most an eighth of a turn,
// is exact to 2^-32 turns.  There the Taylor series of sin and cos need five and
// six terms: the next ones are below 2^-29 at pi/4.  t is off by three roundings,
// 3 2^-24 t, which makes 2^-23.2 of a sine or cosine at most; with the sums' own
// roundings (2^-25 for the last, 2^-26 for the others) and the remainder both are
// off by less than 2^-22.  A rotated element adds gain, its product with cos or
// sin, a product and a sum, 2^-24 each: 2^-21 of gain (|x| + |z|) in all.  (CUDA's
// sincospif, which reduces its argument again, made the LM shape's rotation a
// fifth slower.)
__device__ __forceinline__ void rotary_angle(int64_t p, uint64_t inc, float gain, float &c, float &s) {
    const uint32_t u = (uint32_t)(((uint64_t)p * inc) >> 32);
    const uint32_t quarter = (u + 0x20000000u) >> 30;
    const int32_t rest = (int32_t)(u - (quarter << 30));
    const float t = (float)rest * (6.283185307179586f / 4294967296.0f), t2 = t * t;
    float sn = fmaf(t2, 1.0f / 362880.0f, -1.0f / 5040.0f);
    sn = fmaf(t2, sn, 1.0f / 120.0f);
    sn = fmaf(t2, sn, -1.0f / 6.0f);
    sn = fmaf(t * t2, sn, t);
    float cs = fmaf(t2, -1.0f / 3628800.0f, 1.0f / 40320.0f);
    cs = fmaf(t2, cs, -1.0f / 720.0f);
    cs = fmaf(t2, cs, 1.0f / 24.0f);
    cs = fmaf(t2, cs, -0.5f);
    cs = fmaf(t2, cs, 1.0f);
    const float a = (quarter & 1) ? sn : cs, b = (quarter & 1) ? cs : sn;
    c = gain * ((quarter == 1 || quarter == 2) ? -a : a);
    s = gain * ((quarter & 2) ? -b : b);
}

// One element of a rotated pair: itself, the other, cos, and sin (of the second
// element) or -sin (of the first).  Every kernel rounds in this order, so that a
// key has the same bits whichever call rotated it.
__device__ __forceinline__ float rotated(float self, float other, float c, float signed_s) {
    return fmaf(self, c, __fmul_rn(other, signed_s));
}

// Two-wide float32 arithmetic on register pairs.
__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair2(uint64_t x, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// VEC consecutive elements: as they are in memory (Raw, what is held while loads
// are under way) and as floats.
template <typename T, int VEC> struct Row {
    typedef T Raw;
    __device__ __forceinline__ static void unpack(const Raw &r, float *f) { f[0] = to_f32(r); }
    __device__ __forceinline__ static Raw pack(const float *f) { return from_f32<T>(f[0]); }
};
template <> struct Row<float, 4> {
    typedef uint4 Raw;
    __device__ __forceinline__ static void unpack(const Raw &r, float *f) { Vec16<float>::unpack(r, f); }
    __device__ __forceinline__ static Raw pack(const float *f) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};
template <> struct Row<__nv_bfloat16, 8> {
    typedef uint4 Raw;
    __device__ __forceinline__ static void unpack(const Raw &r, float *f) { Vec16<__nv_bfloat16>::unpack(r, f); }
    __device__ __forceinline__ static Raw pack(const float *f) {
        return make_uint4(pack_bf16_rn(f[0], f[1]), pack_bf16_rn(f[2], f[3]), pack_bf16_rn(f[4], f[5]), pack_bf16_rn(f[6], f[7]));
    }
};

// A head is cut into chunks of 2 VEC elements, one thread each: for the
// leading rot / (2 VEC) chunks the VEC pairs c VEC .. of frequencies of the
// same numbers (two vectors a head apart by rot/2, or adjacent when
// interleaved), behind them plain copies.  rot must be a multiple of 2 VEC
// (VEC = 1: even), d of VEC.
template <typename T, int VEC, bool INTER>
struct RotChunk {
    typedef typename Row<T, VEC>::Raw Raw;
    static constexpr int P = VEC > 1 ? VEC / 2 : 1;
    // VEC > 1: cos, sin and -sin of two pairs side by side (interleaved: of one
    // pair, as (cos, cos) and (-sin, sin)); VEC = 1: cos and sin
    uint64_t c2[VEC > 1 ? (INTER ? VEC : P) : 1], s2[VEC > 1 ? VEC : 1];
    int a, b;     // element offsets of the two vectors; b < 0: only a
    bool turned;

    __device__ __forceinline__ void place(const RotaryTable &r, int chunk, int d) {
        turned = chunk * 2 * VEC < r.rot;
        a = turned && !INTER ? chunk * VEC : chunk * 2 * VEC;
        b = turned && !INTER ? a + r.rot / 2 : a + VEC;
        if (b >= d) b = -1;
    }
    __device__ __forceinline__ void angles(const RotaryTable &r, int chunk, int64_t p, bool backward) {
        if (!turned) return;
        float c[VEC], s[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            rotary_angle(p, r.inc[chunk * VEC + e], r.gain, c[e], s[e]);
            if (backward) s[e] = -s[e];
        }
        if constexpr (VEC == 1) {
            c2[0] = pair2(c[0], s[0]);
        } else if constexpr (INTER) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                c2[e] = pair2(c[e], c[e]);
                s2[e] = pair2(-s[e], s[e]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < P; ++e) {
                c2[e] = pair2(c[2 * e], c[(2 * e + 1) % VEC]);
                s2[e] = pair2(s[2 * e], s[(2 * e + 1) % VEC]);
                s2[P + e] = pair2(-s[2 * e], -s[(2 * e + 1) % VEC]);
            }
        }
    }
    // the chunk's 2 VEC values, x the vector at a, z the one at b
    __device__ __forceinline__ void turn(float *x, float *z) const {
        if constexpr (VEC == 1) {
            float c, s;
            unpair2(c2[0], c, s);
            const float u = x[0], w = z[0];
            x[0] = rotated(u, w, c, -s);
            z[0] = rotated(w, u, c, s);
        } else if constexpr (INTER) {
#pragma unroll
            for (int e = 0; e < P; ++e) {
                unpair2(fma2(pair2(x[2 * e], x[2 * e + 1]), c2[e], mul2(pair2(x[2 * e + 1], x[2 * e]), s2[e])), x[2 * e], x[2 * e + 1]);
                unpair2(fma2(pair2(z[2 * e], z[2 * e + 1]), c2[P + e], mul2(pair2(z[2 * e + 1], z[2 * e]), s2[P + e])), z[2 * e], z[2 * e + 1]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const uint64_t u = pair2(x[2 * e], x[2 * e + 1]), w = pair2(z[2 * e], z[2 * e + 1]);
                unpair2(fma2(u, c2[e], mul2(w, s2[P + e])), x[2 * e], x[2 * e + 1]);
                unpair2(fma2(w, c2[e], mul2(u, s2[e])), z[2 * e], z[2 * e + 1]);
            }
        }
    }
    __device__ __forceinline__ void load(const T *row, Raw &x, Raw &z) const {
        x = *reinterpret_cast<const Raw *>(row + a);
        if (b >= 0) z = *reinterpret_cast<const Raw *>(row + b);
    }
    // turns (or, with turn_it false, copies) what load brought, into a row
    __device__ __forceinline__ void store(T *row, const Raw &x, const Raw &z, bool turn_it) const {
        if (turned && turn_it) {
            float f[VEC], g[VEC];
            Row<T, VEC>::unpack(x, f);
            Row<T, VEC>::unpack(z, g);
            turn(f, g);
            *reinterpret_cast<Raw *>(row + a) = Row<T, VEC>::pack(f);
            *reinterpret_cast<Raw *>(row + b) = Row<T, VEC>::pack(g);
        } else {
            *reinterpret_cast<Raw *>(row + a) = x;
            if (b >= 0) *reinterpret_cast<Raw *>(row + b) = z;
        }
    }
};

// Host side (rotate.cu): checks a tc_rotary for head dimension d and fills
// the table; rotary NULL gives rot = 0.
bool make_rotary_table(const tc_rotary *rotary, int64_t d, RotaryTable *out);

struct RotateParams {
    const void *q, *k;
    void *q_out, *k_out;
    const int64_t *positions;
    int64_t t0, B, T;
    int Hq, H, d;
    int64_t qs[3], ks[3], qos[3], kos[3];
    bool backward;
    RotaryTable table;
};
cudaError_t launch_rotate(const RotateParams &p, tc_dtype dtype, int num_sms, cudaStream_t s);

// Whether a set of rows can be moved in 16-byte vectors: address and strides
// (in elements of es bytes) of dimensions longer than one.
inline bool rows_aligned16(const void *p, const int64_t *stride, const int64_t *size, int64_t es) {
    if (reinterpret_cast<uintptr_t>(p) & 15u) return false;
    for (int i = 0; i < 3; ++i)
        if (size[i] > 1 && (stride[i] * es) % 16 != 0) return false;
    return true;
}

}  // namespace tc

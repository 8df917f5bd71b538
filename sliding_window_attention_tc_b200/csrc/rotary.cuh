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
// quarter turn is taken off in integers; the rest, at most an eighth of a turn, is exact
// to 2^-32 turns and goes to sincospif.
__device__ __forceinline__ void rotary_angle(int64_t p, uint64_t inc, float gain, float &c, float &s) {
    const uint32_t u = (uint32_t)(((uint64_t)p * inc) >> 32);
    const uint32_t quarter = (u + 0x20000000u) >> 30;
    const int32_t rest = (int32_t)(u - (quarter << 30));
    float sn, cs;
    sincospif((float)rest * (1.0f / 2147483648.0f), &sn, &cs);  // rest / 2^32 turns = rest / 2^31 * pi
    const float a = (quarter & 1) ? sn : cs, b = (quarter & 1) ? cs : sn;
    c = gain * ((quarter == 1 || quarter == 2) ? -a : a);
    s = gain * ((quarter & 2) ? -b : b);
}

// VEC consecutive elements held as floats.
template <typename T, int VEC> struct Row {
    __device__ __forceinline__ static void load(const T *p, float *f) { f[0] = to_f32(*p); }
    __device__ __forceinline__ static void store(T *p, const float *f) { *p = from_f32<T>(f[0]); }
};
template <> struct Row<float, 4> {
    __device__ __forceinline__ static void load(const float *p, float *f) {
        Vec16<float>::unpack(*reinterpret_cast<const uint4 *>(p), f);
    }
    __device__ __forceinline__ static void store(float *p, const float *f) {
        *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
    }
};
template <> struct Row<__nv_bfloat16, 8> {
    __device__ __forceinline__ static void load(const __nv_bfloat16 *p, float *f) {
        Vec16<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4 *>(p), f);
    }
    __device__ __forceinline__ static void store(__nv_bfloat16 *p, const float *f) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16_rn(f[0], f[1]), pack_bf16_rn(f[2], f[3]),
                                                   pack_bf16_rn(f[4], f[5]), pack_bf16_rn(f[6], f[7]));
    }
};

// A head is cut into chunks of 2 VEC elements, one thread each: for the
// leading rot / (2 VEC) chunks the VEC pairs c VEC .. of frequencies of the
// same numbers (two vectors a head apart by rot/2, or adjacent when
// interleaved), behind them plain copies.  rot must be a multiple of 2 VEC
// (VEC = 1: even), d of VEC.
template <int VEC>
struct RotChunk {
    float c[VEC], s[VEC];
    int a, b;     // element offsets of the two vectors; b < 0: only a
    bool turned;
    bool inter;

    __device__ __forceinline__ void place(const RotaryTable &r, int chunk, int d) {
        turned = chunk * 2 * VEC < r.rot;
        inter = r.interleaved != 0;
        a = turned && !inter ? chunk * VEC : chunk * 2 * VEC;
        b = turned && !inter ? a + r.rot / 2 : a + VEC;
        if (b >= d) b = -1;
    }
    __device__ __forceinline__ void angles(const RotaryTable &r, int chunk, int64_t p, bool backward) {
        if (!turned) return;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            rotary_angle(p, r.inc[chunk * VEC + e], r.gain, c[e], s[e]);
            if (backward) s[e] = -s[e];
        }
    }
    // the chunk's 2 VEC values, x the vector at a, z the one at b
    __device__ __forceinline__ void turn(float *x, float *z) const {
        if (!turned) return;
        if (!inter || VEC == 1) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float u = x[e], w = z[e];
                x[e] = u * c[e] - w * s[e];
                z[e] = u * s[e] + w * c[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < VEC / 2; ++e) {
                float u = x[2 * e], w = x[2 * e + 1];
                x[2 * e] = u * c[e] - w * s[e];
                x[2 * e + 1] = u * s[e] + w * c[e];
                u = z[2 * e];
                w = z[2 * e + 1];
                z[2 * e] = u * c[VEC / 2 + e] - w * s[VEC / 2 + e];
                z[2 * e + 1] = u * s[VEC / 2 + e] + w * c[VEC / 2 + e];
            }
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

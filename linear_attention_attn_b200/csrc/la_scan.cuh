// la_scan.cuh -- layout shared by the forward, step and backward kernels of the selective scan.
//
// A channel's N states are spread over LN lanes of a warp, kNS = 4 each (N is padded to 4 LN with
// rates and projections of zero, which contribute nothing, see Existing), so sums over n are log2(LN) shuffles and
// a warp works on S = 32 / LN channels.  Lane l has states 4 (l / S) on of channel l % S: lanes that
// read the same B and C are neighbours, and a 16-byte read of shared memory whose neighbours agree
// takes 2 passes instead of 4 (measured; 8 bytes: 1 instead of 2), while the reads that differ from
// channel to channel are single floats, which take 1 whatever they differ by.
#pragma once

#include "la_mixer.cuh"

namespace la {
namespace scan {

constexpr int kNS = 4;             // states a lane holds
constexpr int kTile = 16;          // tokens staged in shared memory at a time

// e^-|r| (0 from 128 on) with the argument's rounding repaired: r log2(e) as a product and its
// remainder, and the part of log2(e) that one float leaves out.  (One value at a time: a packed
// operation takes no constant operand, and keeping all of these in register pairs costs more.)
__device__ __forceinline__ float exp_neg_abs(float r) {
    constexpr float rest = (float)(1.44269504088896340736 - (double)kLog2e);
    const float m = fmaxf(-fabsf(r), -128.f), v = m * kLog2e;
    const float lo = fmaf(m, rest, fmaf(m, kLog2e, -v)), e = ex2(v);
    return fmaf(e, lo * 0.69314718055994531f, e);
}
// log(1 + e^r) = max(r, 0) + log1p(e), e = e^-|r| in (0, 1]: log1p(e) = 2 atanh(s), s = e / (2 + e) <= 1/3,
// with atanh(s) / s a polynomial in s^2, fitted through the Chebyshev points of [0, 1/9] (its error is
// below 2^-25).  A NaN stays one.
__device__ __forceinline__ float softplus_from(float r, float e) {
    const float s = e * rcp(2.f + e), q = s * s;
    float p = fmaf(q, 0.1342574900842183f, 0.1411830990323794f), top;
    p = fmaf(q, p, 0.200037803224282f);
    p = fmaf(q, p, 0.3333332016834966f);
    p = fmaf(q, p, 1.f);
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(top) : "f"(r));
    return fmaf(s + s, p, top);
}
__device__ __forceinline__ float softplus_f(float r) { return softplus_from(r, exp_neg_abs(r)); }
__device__ __forceinline__ f2 softplus2(f2 r) {
    float a, b;
    unpack2(r, a, b);
    return pack2(softplus_f(a), softplus_f(b));
}

__device__ __forceinline__ int seq_end(const int *lengths, int b, int T) {
    return lengths ? min(max(lengths[b], 0), T) : T;
}

// exp of a pair's steps times rates (A2 = A log2 e).  The exponential unit cuts its result off, which a state
// with a memory of many tokens would gather up; 3e-8 on the argument, in the product's own rounding, brings
// the average over rates within 1.2e-8 of 0.  Measured relative averages without and with it: |d A| in
// (0.025, 0.35) -1.65e-8 and 0.45e-8, (0.012, 0.17) -0.83e-8 and 0.17e-8, (0.0016, 0.016) -0.32e-8 and -0.06e-8,
// below that under 0.1e-8 both; only in (0.05, 0.69), a memory of a few tokens, nothing is gained (-1.7e-8 and
// 1.6e-8).  A step of 0 still gives exactly 1.
constexpr float kNudge = 3e-8f;
__device__ __forceinline__ f2 decay2(f2 d, f2 A2) { return ex2_2(fma2(d, A2, both(kNudge))); }

// The quarter (of 4 states) that this thread has, and its channel in the block's tile.
template <int LN> __device__ __forceinline__ int lane_states() { return (threadIdx.x & 31) / (32 / LN); }
template <int LN> __device__ __forceinline__ int lane_channel() {
    return (threadIdx.x >> 5) * (32 / LN) + (threadIdx.x & 31) % (32 / LN);
}

// Keeps the states that exist of a lane's four and makes the others 0.  Padded states have rates and
// projections of 0, but with an infinite step or input 0 times infinity would come to be among them, and
// the channel's sum NaN.  Only kernels for an N that does not fill its lanes (PAD) have to.
template <bool PAD> struct Existing {
    f2 mask[2];
    __device__ __forceinline__ Existing(int n0, int N) {
        if (PAD)
#pragma unroll
            for (int k = 0; k < 2; ++k)
                mask[k] = (n0 + 2 * k < N ? 0xffffffffull : 0) | (n0 + 2 * k + 1 < N ? 0xffffffffull << 32 : 0);
    }
    __device__ __forceinline__ f2 operator()(f2 v, int k) const { return PAD ? v & mask[k] : v; }
};

// Sums v[0..3] (four tokens) over the LN lanes of a channel.  Each step hands half of the values
// to the partner lane: afterwards lane nl holds the sums of tokens first_token(nl) ..
// first_token(nl) + kept - 1 in v[0..kept-1]; for LN > 4 only the lanes nl < 4 are to be used.
template <int LN> struct Kept { static constexpr int value = LN >= 4 ? 1 : 4 / LN; };
template <int LN>
__device__ __forceinline__ int first_token(int nl) {
    return LN == 1 ? 0 : LN == 2 ? 2 * nl : 2 * (nl & 1) + ((nl >> 1) & 1);
}
template <int LN>
__device__ __forceinline__ void reduce4(float (&v)[4], int nl) {
    constexpr int S = 32 / LN;
    if (LN >= 2) {
        const bool hi = nl & 1;
        const float s0 = hi ? v[0] : v[2], s1 = hi ? v[1] : v[3];
        v[0] = (hi ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, s0, S);
        v[1] = (hi ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, s1, S);
    }
    if (LN >= 4) {
        const bool hi = nl & 2;
        const float s = hi ? v[0] : v[1];
        v[0] = (hi ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, s, 2 * S);
    }
    if (LN >= 8) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 4 * S);
    if (LN >= 16) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 8 * S);
}

// Where a block works: batch entry, segment of the sequence, and a tile of channels of one group.
struct Place {
    int b, seg, g, c0, nc;           // first channel, channels of this tile
};
__device__ __forceinline__ Place place(long long block, int G, int cpg, int tiles, int segs, int width) {
    Place p;
    int tile;
    block = split(block, tiles, tile);
    block = split(block, G, p.g);
    p.b = (int)split(block, segs, p.seg);
    p.c0 = p.g * cpg + tile * width;
    p.nc = min(width, cpg - tile * width);
    return p;
}

__device__ __forceinline__ void load_states(const float *p, int n0, int N, float (&h)[kNS]) {
    // 16-byte accesses where rows are whole multiples of them
    if ((N & 3) == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        if (n0 < N) {
            const float4 v = *reinterpret_cast<const float4 *>(p + n0);
            h[0] = v.x; h[1] = v.y; h[2] = v.z; h[3] = v.w;
        } else {
            h[0] = h[1] = h[2] = h[3] = 0.f;
        }
    } else {
#pragma unroll
        for (int k = 0; k < kNS; ++k) h[k] = n0 + k < N ? p[n0 + k] : 0.f;
    }
}
__device__ __forceinline__ void store_states(float *p, int n0, int N, const float (&h)[kNS]) {
    if ((N & 3) == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        if (n0 < N) *reinterpret_cast<float4 *>(p + n0) = make_float4(h[0], h[1], h[2], h[3]);
    } else {
#pragma unroll
        for (int k = 0; k < kNS; ++k)
            if (n0 + k < N) p[n0 + k] = h[k];
    }
}

// Four neighbouring elements of a row as they lie in memory, of which the first `have` exist (the
// others 0).  vec: all or none do, and the address allows one access.  Kept as words, so that a load
// is not waited for before its values are used.
template <typename T, int SIZE = sizeof(T)> struct Quad;
template <typename T> struct Quad<T, 2> {
    uint2 w;
    __device__ __forceinline__ void load(const T *p, int have, bool vec) {
        w = make_uint2(0u, 0u);
        if (vec) {
            if (have >= 4) w = *reinterpret_cast<const uint2 *>(p);
        } else {
            const unsigned short *s = reinterpret_cast<const unsigned short *>(p);
            if (have > 0) w.x = s[0];
            if (have > 1) w.x |= (unsigned)s[1] << 16;
            if (have > 2) w.y = s[2];
            if (have > 3) w.y |= (unsigned)s[3] << 16;
        }
    }
    __device__ __forceinline__ void values(f2 (&v)[2]) const {
        const float2 a = Pair16<T>::widen(w.x), b = Pair16<T>::widen(w.y);
        v[0] = pack2(a.x, a.y);
        v[1] = pack2(b.x, b.y);
    }
};
template <typename T> struct Quad<T, 4> {
    float4 w;
    __device__ __forceinline__ void load(const T *p, int have, bool vec) {
        w = make_float4(0.f, 0.f, 0.f, 0.f);
        if (vec) {
            if (have >= 4) w = *reinterpret_cast<const float4 *>(p);
        } else {
            if (have > 0) w.x = p[0];
            if (have > 1) w.y = p[1];
            if (have > 2) w.z = p[2];
            if (have > 3) w.w = p[3];
        }
    }
    __device__ __forceinline__ void values(f2 (&v)[2]) const {
        v[0] = pack2(w.x, w.y);
        v[1] = pack2(w.z, w.w);
    }
};
template <typename T>
__device__ __forceinline__ void store4(T *p, const float (&v)[4], int have, bool vec) {
    if (vec && have >= 4) {
        stv<4>(p, v);
    } else if (!vec) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < have) p[i] = from_f<T>(v[i]);
    }
}

// Whether rows whose offsets are all multiples of `unit` elements allow accesses of 4 elements.
template <typename T, typename... P>
inline int quad_rows(int unit, P... p) {
    const uintptr_t bits = (0 | ... | (uintptr_t)p);
    return unit % 4 == 0 && (bits & (4 * sizeof(T) - 1)) == 0;
}

inline int lanes_for(int N) {
    int ln = 1;
    while (ln * kNS < N) ln *= 2;
    return ln;
}

}  // namespace scan
}  // namespace la

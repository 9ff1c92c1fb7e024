// la_scan.cuh -- layout shared by the forward, step and backward kernels of the selective scan.
//
// A channel's N states are spread over LN neighbouring lanes of a warp, kNS = 4 each (N is padded
// to 4 LN with rates and projections of zero, which contribute nothing), so sums over n are
// log2(LN) shuffles and a warp works on 32 / LN channels.
#pragma once

#include "la_mixer.cuh"

namespace la {
namespace scan {

constexpr int kNS = 4;             // states a lane holds
constexpr int kTile = 16;          // tokens staged in shared memory at a time
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float softplus_f(float r) { return fmaxf(r, 0.f) + log1pf(expf(-fabsf(r))); }

__device__ __forceinline__ int seq_end(const int *lengths, int b, int T) {
    return lengths ? min(max(lengths[b], 0), T) : T;
}

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
    if (LN >= 2) {
        const bool hi = nl & 1;
        const float s0 = hi ? v[0] : v[2], s1 = hi ? v[1] : v[3];
        v[0] = (hi ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, s0, 1);
        v[1] = (hi ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, s1, 1);
    }
    if (LN >= 4) {
        const bool hi = nl & 2;
        const float s = hi ? v[0] : v[1];
        v[0] = (hi ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, s, 2);
    }
    if (LN >= 8) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 4);
    if (LN >= 16) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 8);
}

// Where a block works: batch entry, segment of the sequence, and a tile of channels of one group.
struct Place {
    int b, seg, g, c0, nc;           // first channel, channels of this tile
};
__device__ __forceinline__ Place place(long long block, int G, int cpg, int tiles, int segs, int width) {
    Place p;
    const int tile = (int)(block % tiles);
    block /= tiles;
    p.g = (int)(block % G);
    block /= G;
    p.seg = (int)(block % segs);
    p.b = (int)(block / segs);
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

inline int lanes_for(int N) {
    int ln = 1;
    while (ln * kNS < N) ln *= 2;
    return ln;
}

}  // namespace scan
}  // namespace la

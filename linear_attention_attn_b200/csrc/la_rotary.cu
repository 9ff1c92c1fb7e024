// la_rotary.cu -- rotary positions on queries and keys, and the inverse rotation (its gradient).
//
// Pair i of a head's first R entries, at position p, turns by the angle p f_i.  The turns
// p f_i / (2 pi) are formed as a sum of two doubles, with the products' remainders and the part of
// 1 / (2 pi) that one double leaves out (one double alone is off by 7e-6 of a radian at positions of
// 2^35, and says nothing at 2^53), reduced to [-1/2, 1/2], and only then given to sincospi in fp32.
//
// Bound by HBM: every element is read and written once.  A thread owns V elements of one token's
// row (V of each half in the half layout, V / 2 neighbouring pairs interleaved) and walks over the
// heads, which share the angle: its sines and cosines stay in registers and are paid for once per
// head range.  The heads of q and k form one list, cut into as many ranges as fill the GPU, so a
// single new token spreads over the heads and a long prompt over tokens.
// B4 H32 + 8 T8192 D128 bf16 (671 MB in and out): 106 us, 6.3 TB/s, 97 % of the measured copy.
#include "la_mixer.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;          // heads whose elements a thread has on their way at a time

// The turns of frequency f at position p (a whole number of at most 53 bits), in [-1/2, 1/2].
__device__ __forceinline__ float turns_of(double p, float f) {
    constexpr double c = 0.15915494309189535, c_rest = -9.839338337591243e-18;     // 1 / (2 pi)
    const double t = p * (double)f, t_rest = ::fma(p, (double)f, -t);
    const double hi = t * c, lo = ::fma(t, c, -hi) + ::fma(t, c_rest, t_rest * c);
    const double r = (hi - rint(hi)) + lo;             // lo: up to 1 where hi has no bits behind the point
    return (float)(r - rint(r));
}

// V: elements an access; an interleaved item is at least a pair, of two accesses where V = 1
// (tensors aligned to one element only).
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kThreads)
rotary_kernel(RotaryArgs a, int items, int heads_per) {
    const long long idx = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long rows = (long long)a.B * a.T;
    if (idx >= rows * items) return;
    int item, t;
    const long long row = split(idx, items, item);
    const int b = (int)split(row, a.T, t);
    const int half = a.R / 2;
    constexpr int W = INTER && V == 1 ? 2 : V;         // elements of an item
    constexpr int P = INTER ? W / 2 : V;               // pairs of an item
    const int nrot = INTER ? a.R / W : half / W;       // items that rotate; the rest copy
    const bool rot = item < nrot;
    const int c0 = rot ? item * W : a.R + (item - nrot) * W;
    float cs[P], sn[P];
    if (rot) {
        const long long pos = a.positions ? a.positions[a.per_batch ? row : t] : a.start + t;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float f = a.freqs[INTER ? item * P + i : c0 + i];
            float s, c;
            sincospif(2.f * turns_of((double)pos, f), &s, &c);
            cs[i] = c * a.magnitude;
            sn[i] = s * a.sign * a.magnitude;
        }
    }
    const int h0 = blockIdx.y * heads_per, h1 = min(h0 + heads_per, a.H + a.Hk);
    const long long stride = (long long)a.T * a.D, at = (long long)t * a.D + c0;
    constexpr int N = W / V;                           // accesses of an item (of either half)
    auto heads = [&](const T *src, T *dst, int count) {
        for (int h = 0; h < count; h += kHeads) {
            // all loads before the first store, which the compiler may not pass (the output may be the input)
            Raw<T, V> x[kHeads][N], y[kHeads];
#pragma unroll
            for (int u = 0; u < kHeads; ++u) {
                const bool there = h + u < count;
#pragma unroll
                for (int j = 0; j < N; ++j) x[u][j].load(src + u * stride + j * V, there && (rot || c0 + j * V < a.D));
                if (!INTER) y[u].load(src + u * stride + half, there && rot);
            }
#pragma unroll
            for (int u = 0; u < kHeads; ++u) {
                if (h + u >= count) break;
                T *out = dst + u * stride;
                if (!rot) {
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        if (c0 + j * V < a.D) x[u][j].store(out + j * V);
                } else if constexpr (INTER) {
                    float v[W], w[W];
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        float e[V];
                        x[u][j].lanes().get(e);
#pragma unroll
                        for (int i = 0; i < V; ++i) v[j * V + i] = e[i];
                    }
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        w[2 * i] = fmaf(v[2 * i], cs[i], -v[2 * i + 1] * sn[i]);
                        w[2 * i + 1] = fmaf(v[2 * i], sn[i], v[2 * i + 1] * cs[i]);
                    }
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        float e[V];
#pragma unroll
                        for (int i = 0; i < V; ++i) e[i] = w[j * V + i];
                        stv<V>(out + j * V, e);
                    }
                } else {
                    float v[V], w[V], lo[V], hi[V];
                    x[u][0].lanes().get(v);
                    y[u].lanes().get(w);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        lo[i] = fmaf(v[i], cs[i], -w[i] * sn[i]);
                        hi[i] = fmaf(v[i], sn[i], w[i] * cs[i]);
                    }
                    stv<V>(out, lo);
                    stv<V>(out + half, hi);
                }
            }
            src += kHeads * stride;
            dst += kHeads * stride;
        }
    };
    const int q0 = min(h0, a.H), q1 = min(h1, a.H), k0 = max(h0, a.H) - a.H, k1 = max(h1, a.H) - a.H;
    const long long qo = ((long long)b * a.H + q0) * stride + at, ko = ((long long)b * a.Hk + k0) * stride + at;
    heads((const T *)a.q + qo, (T *)a.oq + qo, q1 - q0);
    heads((const T *)a.k + ko, (T *)a.ok + ko, k1 - k0);
}

template <typename T, int V, bool INTER>
la_status rotary_v(const RotaryArgs &a, cudaStream_t st) {
    constexpr int W = INTER && V == 1 ? 2 : V;
    const int items = (INTER ? a.R / W : a.R / 2 / W) + (a.D - a.R + W - 1) / W;
    const long long threads = (long long)a.B * a.T * items;
    const long long blocks = (threads + kThreads - 1) / kThreads;
    const int heads = a.H + a.Hk;
    // Head ranges: about one wave of 148 x 8 blocks, at most one range a head.  More ranges pay for the
    // angles again (the same inputs from call to call, so from L2; 4 waves: B8 H32 T1023 D64 f16 18.5 us instead of 12.3, B6 H40 T254 D80 R54 16.4
    // instead of 10.3; the other way only where they are few: B28 H64 T721 D36 R18 41 instead of 47).
    long long want = (148 * 8 + blocks - 1) / blocks;
    if (want > heads) want = heads;
    const int per = (int)((heads + want - 1) / want);
    const dim3 grid((unsigned)blocks, (unsigned)((heads + per - 1) / per));
    return launch(a.sign > 0 ? "rotary_fwd" : "rotary_bwd", rotary_kernel<T, V, INTER>, grid, dim3(kThreads), 0, st,
                  a, items, per);
}

template <typename T>
la_status rotary_t(const RotaryArgs &a, cudaStream_t st) {
    const uintptr_t bits = (uintptr_t)a.q | (uintptr_t)a.k | (uintptr_t)a.oq | (uintptr_t)a.ok;
    // every offset of an access is a multiple of D, R (the copied part) and, in the half layout, R / 2
    const long long unit = a.interleaved ? (a.D | a.R) : (a.D | (a.R / 2));
    const int v = vec_width(sizeof(T), unit, bits);
    if (a.interleaved) {
        switch (v) {
        case 8: return rotary_v<T, 16 / sizeof(T), true>(a, st);
        case 4: return rotary_v<T, 4, true>(a, st);
        case 2: return rotary_v<T, 2, true>(a, st);
        default: return rotary_v<T, 1, true>(a, st);
        }
    }
    switch (v) {
    case 8: return rotary_v<T, 16 / sizeof(T), false>(a, st);
    case 4: return rotary_v<T, 4, false>(a, st);
    case 2: return rotary_v<T, 2, false>(a, st);
    default: return rotary_v<T, 1, false>(a, st);
    }
}

}  // namespace

la_status rotary(const RotaryArgs &a, cudaStream_t st) {
    switch (a.dt) {
    case LA_F32: return rotary_t<float>(a, st);
    case LA_F16: return rotary_t<__half>(a, st);
    default: return rotary_t<__nv_bfloat16>(a, st);
    }
}

}  // namespace la

// la_rotary.cu -- rotary positions on queries and keys, and the inverse rotation (its gradient).
//
// Pair i of a head's first R entries, at position p, turns by the angle p f_i.  The turns
// p f_i / (2 pi) are formed in double (a position of 2^31 still leaves 2^-21 of a turn's last
// bit), reduced to [-1/2, 1/2], and only then given to sincospi in fp32.
//
// Bound by HBM: every element is read and written once.  A thread owns V elements of one token's
// row (V of each half in the half layout, V / 2 neighbouring pairs interleaved) and walks over the
// heads, which share the angle: its sines and cosines stay in registers and are paid for once per
// head range.  The heads of q and k form one list, cut into as many ranges as give the GPU about
// four waves of threads, so a single new token spreads over the heads and a long prompt over
// tokens.
#include "la_mixer.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;

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
            const double turns = (double)pos * ((double)f * 0.15915494309189533577);
            float s, c;
            sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
            cs[i] = c * a.magnitude;
            sn[i] = s * a.sign * a.magnitude;
        }
    }
    const int h0 = blockIdx.y * heads_per, h1 = min(h0 + heads_per, a.H + a.Hk);
#pragma unroll 4
    for (int h = h0; h < h1; ++h) {
        const bool isq = h < a.H;
        const long long off =
            (isq ? ((long long)b * a.H + h) : ((long long)b * a.Hk + (h - a.H))) * a.T * a.D + (long long)t * a.D + c0;
        const T *src = (const T *)(isq ? a.q : a.k) + off;
        T *dst = (T *)(isq ? a.oq : a.ok) + off;
        if (!rot) {
#pragma unroll
            for (int j = 0; j < W; j += V)
                if (c0 + j < a.D) *reinterpret_cast<Pack<T, V> *>(dst + j) = *reinterpret_cast<const Pack<T, V> *>(src + j);
        } else if constexpr (INTER) {
            float x[W], y[W];
            if constexpr (V == 1) {
                x[0] = to_f(src[0]);
                x[1] = to_f(src[1]);
            } else {
                ldv<V>(src, x);
            }
#pragma unroll
            for (int i = 0; i < P; ++i) {
                y[2 * i] = fmaf(x[2 * i], cs[i], -x[2 * i + 1] * sn[i]);
                y[2 * i + 1] = fmaf(x[2 * i], sn[i], x[2 * i + 1] * cs[i]);
            }
            if constexpr (V == 1) {
                dst[0] = from_f<T>(y[0]);
                dst[1] = from_f<T>(y[1]);
            } else {
                stv<V>(dst, y);
            }
        } else {
            float x[V], y[V], u[V], v[V];
            ldv<V>(src, x);
            ldv<V>(src + half, y);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                u[i] = fmaf(x[i], cs[i], -y[i] * sn[i]);
                v[i] = fmaf(x[i], sn[i], y[i] * cs[i]);
            }
            stv<V>(dst, u);
            stv<V>(dst + half, v);
        }
    }
}

template <typename T, int V, bool INTER>
la_status rotary_v(const RotaryArgs &a, cudaStream_t st) {
    constexpr int W = INTER && V == 1 ? 2 : V;
    const int items = (INTER ? a.R / W : a.R / 2 / W) + (a.D - a.R + W - 1) / W;
    const long long threads = (long long)a.B * a.T * items;
    const long long blocks = (threads + kThreads - 1) / kThreads;
    const int heads = a.H + a.Hk;
    // head ranges: about 4 waves of 148 x 8 blocks, at most one range per head
    long long want = (4 * 148 * 8 + blocks - 1) / blocks;
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

// la_conv.cu -- short causal depthwise convolution, channels last, with SiLU, and its gradients.
//
//   s[t] = bias + sum_{j<W} w[j] x[t-W+1+j],  y[t] = act(s[t]);  rows before the first token come
//   from the state (zeros without one), rows behind a sequence's end count as absent.
//   g[t] = dy[t] act'(s[t]);  dx[u] = sum_{k<W} w[W-1-k] g[u+k];  dw[j] = sum_t g[t] x[t-W+1+j].
//
// Bound by HBM: the forward reads and writes every element once, the backward reads x and dy and
// writes dx.  A thread owns V neighbouring channels and walks along a segment of kSeg tokens with
// the last W - 1 inputs in registers, so a segment re-reads only its W - 1 rows of overlap (from
// L2, where the neighbour just read them); threads of a warp lie along the channels, so every row
// is read in whole sectors.  The backward keeps a window of g as well, re-forms W - 1 rows of g to
// its right, and sums dw, dbias in registers over its segment, over the block's segments in shared
// memory, and over blocks in a second launch, each in a fixed order.
#include "la_mixer.cuh"

namespace la {
namespace {

constexpr int kSeg = 16;           // tokens a thread of the forward walks over
constexpr int kThreads = 128;

__device__ __forceinline__ int seq_end(const int *lengths, int b, int T) {
    return lengths ? min(max(lengths[b], 0), T) : T;
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads)
conv_fwd_kernel(ConvArgs a, int cvecs, int segs) {
    const long long idx = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (idx >= (long long)a.B * segs * cvecs) return;
    const long long bs = idx / cvecs;
    const int c = (int)(idx - bs * cvecs) * V;
    const int b = (int)(bs / segs), seg = (int)(bs - (long long)b * segs);
    const int n = seq_end(a.lengths, b, a.T);
    const int t0 = seg * kSeg, t1 = min(t0 + kSeg, a.T);
    const long long C = a.C;
    const T *x = (const T *)a.x + (long long)b * a.T * C + c;
    T *y = (T *)a.y + (long long)b * a.T * C + c;
    const T *first = a.state_in ? (const T *)a.state_in + (long long)b * (W - 1) * C + c : nullptr;

    float w[W][V], bias[V], win[W - 1][V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        bias[i] = a.bias ? a.bias[c + i] : 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = a.w[(long long)(c + i) * W + j];
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int u = t0 - (W - 1) + j;
#pragma unroll
        for (int i = 0; i < V; ++i) win[j][i] = 0.f;
        if (u >= 0) {
            if (u < n) ldv<V>(x + u * C, win[j]);
        } else if (first) {
            ldv<V>(first + (u + W - 1) * C, win[j]);
        }
    }
    // The state after n tokens: rows n .. n + W - 2 of the sequence extended by the entering state.  It
    // leaves through the only thread that reads the entering one, so the two may be one buffer.
    if (seg == 0 && a.state_out) {
        Pack<T, V> keep[W - 1];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int r = n + j;
            if (r >= W - 1) {
                keep[j] = *reinterpret_cast<const Pack<T, V> *>(x + (r - (W - 1)) * C);
            } else if (first) {
                keep[j] = *reinterpret_cast<const Pack<T, V> *>(first + r * C);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) keep[j].v[i] = from_f<T>(0.f);
            }
        }
        T *so = (T *)a.state_out + (long long)b * (W - 1) * C + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) *reinterpret_cast<Pack<T, V> *>(so + j * C) = keep[j];
    }
#pragma unroll 4
    for (int t = t0; t < t1; ++t) {
        float cur[V], o[V];
        if (t < n) {
            ldv<V>(x + t * C, cur);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float s = bias[i];
#pragma unroll
                for (int j = 0; j < W - 1; ++j) s = fmaf(w[j][i], win[j][i], s);
                s = fmaf(w[W - 1][i], cur[i], s);
                o[i] = a.silu ? s * sigmoid_f(s) : s;
            }
#pragma unroll
            for (int j = 0; j + 1 < W - 1; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) win[j][i] = win[j + 1][i];
#pragma unroll
            for (int i = 0; i < V; ++i) win[W - 2][i] = cur[i];
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = 0.f;
        }
        stv<V>(y + t * C, o);
    }
}

// Backward.  Block: 32 channel vectors x kBwdSegs segments of `seg` tokens of one batch entry.
constexpr int kBwdSegs = 8;

template <typename T, int V, int W>
__global__ void __launch_bounds__(32 * kBwdSegs)
conv_bwd_kernel(ConvArgs a, int seg, int blocks_t, int blocks_c, float *part) {
    __shared__ float red[kBwdSegs][32 * V * (W + 1) + 1];
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
    const int p = blockIdx.x / blocks_c, bc = blockIdx.x - p * blocks_c;   // token block, channel block
    const int c = (bc * 32 + lane) * V;
    const int b = p / blocks_t, bt = p - b * blocks_t;
    const long long C = a.C;
    const bool live = c < a.C;
    float dw[W][V], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        db[i] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][i] = 0.f;
    }
    const long long t0l = ((long long)bt * kBwdSegs + row) * seg;
    if (live && t0l < a.T) {
        const int t0 = (int)t0l, t1 = (int)min((long long)a.T, t0l + seg);
        const int n = seq_end(a.lengths, b, a.T);
        const T *x = (const T *)a.x + (long long)b * a.T * C + c;
        const T *dy = (const T *)a.dy + (long long)b * a.T * C + c;
        T *dx = (T *)a.dx + (long long)b * a.T * C + c;
        const T *first = a.state_in ? (const T *)a.state_in + (long long)b * (W - 1) * C + c : nullptr;
        const T *ds = a.dstate_in ? (const T *)a.dstate_in + (long long)b * (W - 1) * C + c : nullptr;
        T *dfirst = a.dstate_out ? (T *)a.dstate_out + (long long)b * (W - 1) * C + c : nullptr;
        float w[W][V], bias[V], win[W - 1][V], gw[W - 1][V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            bias[i] = a.bias ? a.bias[c + i] : 0.f;
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][i] = a.w[(long long)(c + i) * W + j];
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int u = t0 - (W - 1) + j;
#pragma unroll
            for (int i = 0; i < V; ++i) { win[j][i] = 0.f; gw[j][i] = 0.f; }
            if (u >= 0) {
                if (u < n) ldv<V>(x + u * C, win[j]);
            } else if (first) {
                ldv<V>(first + (u + W - 1) * C, win[j]);
            }
        }
        // at step t: g[t] is formed, and dx[u] with u = t - (W - 1) is complete
#pragma unroll 2
        for (int t = t0; t < t1 + W - 1; ++t) {
            float cur[V], g[V];
#pragma unroll
            for (int i = 0; i < V; ++i) { cur[i] = 0.f; g[i] = 0.f; }
            if (t < n) {
                ldv<V>(x + t * C, cur);
                ldv<V>(dy + t * C, g);
                if (a.silu) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        float s = bias[i];
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) s = fmaf(w[j][i], win[j][i], s);
                        s = fmaf(w[W - 1][i], cur[i], s);
                        const float sg = sigmoid_f(s);
                        g[i] *= sg * fmaf(s, 1.f - sg, 1.f);
                    }
                }
                if (t < t1) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        db[i] += g[i];
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) dw[j][i] = fmaf(g[i], win[j][i], dw[j][i]);
                        dw[W - 1][i] = fmaf(g[i], cur[i], dw[W - 1][i]);
                    }
                }
            }
            const int u = t - (W - 1);
            if (u >= t0 || (t0 == 0 && dfirst)) {
                // dx[u] = sum_k w[W-1-k] g[u+k]: g[u] is the oldest in the window
                float d[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    d[i] = w[0][i] * g[i];
#pragma unroll
                    for (int k = 0; k < W - 1; ++k) d[i] = fmaf(w[W - 1 - k][i], gw[k][i], d[i]);
                }
                const int j = u + (W - 1) - n;          // u's row of the leaving state
                if (ds && u < n && j >= 0) {
                    float e[V];
                    ldv<V>(ds + j * C, e);
#pragma unroll
                    for (int i = 0; i < V; ++i) d[i] += e[i];
                }
                stv<V>(u >= 0 ? dx + u * C : dfirst + (u + W - 1) * C, d);
            }
#pragma unroll
            for (int j = 0; j + 1 < W - 1; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    win[j][i] = win[j + 1][i];
                    gw[j][i] = gw[j + 1][i];
                }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                win[W - 2][i] = cur[i];
                gw[W - 2][i] = g[i];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) red[row][(lane * V + i) * (W + 1) + j] = dw[j][i];
        red[row][(lane * V + i) * (W + 1) + W] = db[i];
    }
    __syncthreads();
    const int n_out = min(32 * V, a.C - bc * 32 * V) * (W + 1);
    for (int e = threadIdx.x; e < n_out; e += 32 * kBwdSegs) {
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < kBwdSegs; ++r) s += red[r][e];
        part[((long long)p * a.C + bc * 32 * V) * (W + 1) + e] = s;
    }
}

// dw, dbias from the blocks' parts: block (32 outputs) x 8 rows of parts, fixed order.
__global__ void __launch_bounds__(256) conv_bwd_reduce(const float *part, int parts, int C, int W, float *dw,
                                                       float *dbias) {
    __shared__ float red[8][33];
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
    const int e = blockIdx.x * 32 + lane, n = C * (W + 1);
    float s = 0.f;
    if (e < n)
        for (int p = row; p < parts; p += 8) s += part[(long long)p * n + e];
    red[row][lane] = s;
    __syncthreads();
    if (row == 0 && e < n) {
        float r = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) r += red[k][lane];
        const int c = e / (W + 1), j = e - c * (W + 1);
        if (j < W) dw[c * W + j] = r;
        else if (dbias) dbias[c] = r;
    }
}

// Tokens a thread of the backward walks over, from the sizes alone: 64 (3 rows of overlap on
// either side), halved while the launch would not give every SM two blocks.
int bwd_seg(int B, int T, int C) {
    int seg = 64;
    while (seg > 8 && (long long)B * ((T + seg * kBwdSegs - 1) / (seg * kBwdSegs)) * ((C + 127) / 128) < 296) seg >>= 1;
    return seg;
}

int bwd_blocks_t(int B, int T, int C) {
    const int rows = bwd_seg(B, T, C) * kBwdSegs;
    return (int)(((long long)T + rows - 1) / rows);
}

uintptr_t address_bits(const ConvArgs &a) {
    return (uintptr_t)a.x | (uintptr_t)a.y | (uintptr_t)a.state_in | (uintptr_t)a.state_out | (uintptr_t)a.dy |
           (uintptr_t)a.dx | (uintptr_t)a.dstate_in | (uintptr_t)a.dstate_out;
}

template <typename T, int V, int W>
la_status fwd_v(const ConvArgs &a, cudaStream_t st) {
    const int cvecs = a.C / V, segs = (a.T + kSeg - 1) / kSeg;
    const long long n = (long long)a.B * segs * cvecs;
    return launch("short_conv_fwd", conv_fwd_kernel<T, V, W>, dim3((unsigned)((n + kThreads - 1) / kThreads)),
                  dim3(kThreads), 0, st, a, cvecs, segs);
}

template <typename T, int V, int W>
la_status bwd_v(const ConvArgs &a, cudaStream_t st) {
    const int seg = bwd_seg(a.B, a.T, a.C), bt = bwd_blocks_t(a.B, a.T, a.C);
    const int bc = (a.C + 32 * V - 1) / (32 * V);
    la_status rc = launch("short_conv_bwd", conv_bwd_kernel<T, V, W>, dim3((unsigned)a.B * bt * bc),
                          dim3(32 * kBwdSegs), 0, st, a, seg, bt, bc, (float *)a.ws);
    if (rc != LA_OK) return rc;
    return launch("short_conv_bwd_reduce", conv_bwd_reduce, dim3((unsigned)((a.C * (W + 1) + 31) / 32)), dim3(256), 0,
                  st, (const float *)a.ws, a.B * bt, a.C, W, a.dw, a.dbias);
}

// The forward takes the widest access; the backward at most 4 elements (8 would hold
// 8 x (3 W + 3) floats a thread in registers).
template <typename T, int W>
la_status conv_w(bool bwd, const ConvArgs &a, cudaStream_t st) {
    int v = vec_width(sizeof(T), a.C, address_bits(a));
    if (bwd) {
        if (v >= 4) return bwd_v<T, 4, W>(a, st);
        return v == 2 ? bwd_v<T, 2, W>(a, st) : bwd_v<T, 1, W>(a, st);
    }
    switch (v) {
    case 8: return fwd_v<T, 16 / sizeof(T), W>(a, st);
    case 4: return fwd_v<T, 4, W>(a, st);
    case 2: return fwd_v<T, 2, W>(a, st);
    default: return fwd_v<T, 1, W>(a, st);
    }
}

template <typename T>
la_status conv_t(bool bwd, const ConvArgs &a, cudaStream_t st) {
    switch (a.W) {
    case 2: return conv_w<T, 2>(bwd, a, st);
    case 3: return conv_w<T, 3>(bwd, a, st);
    case 4: return conv_w<T, 4>(bwd, a, st);
    case 5: return conv_w<T, 5>(bwd, a, st);
    case 6: return conv_w<T, 6>(bwd, a, st);
    case 7: return conv_w<T, 7>(bwd, a, st);
    default: return conv_w<T, 8>(bwd, a, st);
    }
}

la_status conv_d(bool bwd, const ConvArgs &a, cudaStream_t st) {
    switch (a.dt) {
    case LA_F32: return conv_t<float>(bwd, a, st);
    case LA_F16: return conv_t<__half>(bwd, a, st);
    default: return conv_t<__nv_bfloat16>(bwd, a, st);
    }
}

}  // namespace

size_t conv_bwd_workspace(int B, int T, int C, int W, la_dtype) {
    if (T == 0) return 0;
    return up256((size_t)B * bwd_blocks_t(B, T, C) * C * (W + 1) * sizeof(float));
}

la_status conv_fwd(const ConvArgs &a, cudaStream_t st) { return conv_d(false, a, st); }
la_status conv_bwd(const ConvArgs &a, cudaStream_t st) { return conv_d(true, a, st); }

}  // namespace la

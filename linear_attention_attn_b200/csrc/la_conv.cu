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
// B8 T4096 C2048 W4 bf16 gradient (403 MB): 98 us, 4.1 TB/s, 63 % of the measured copy; 26 instructions
// an element (SiLU's exponential and reciprocal among them) keep the issue slots 51 % busy, the
// memory 46 %.
#include "la_mixer.cuh"

namespace la {
namespace {

constexpr int kSeg = 16;           // tokens a thread of the forward walks over
constexpr int kThreads = 128;

__device__ __forceinline__ int seq_end(const int *lengths, int b, int T) {
    return lengths ? min(max(lengths[b], 0), T) : T;
}

// The taps of V channels, w[c .. c + V)[W]: V W neighbouring floats, read 16 bytes at a time where
// the array is aligned to them; and their biases.
template <int V, int W>
__device__ __forceinline__ void load_taps(const ConvArgs &a, int c, Lanes<V> (&w)[W], Lanes<V> &bias) {
    const float *p = a.w + (long long)c * W;
    float f[V * W], v[V];
    if ((V * W) % 4 == 0 && ((uintptr_t)a.w & 15) == 0) {
#pragma unroll
        for (int i = 0; i < V * W / 4; ++i) {
            const float4 q = reinterpret_cast<const float4 *>(p)[i];
            f[4 * i] = q.x; f[4 * i + 1] = q.y; f[4 * i + 2] = q.z; f[4 * i + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V * W; ++i) f[i] = p[i];
    }
#pragma unroll
    for (int j = 0; j < W; ++j) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = f[i * W + j];
        w[j].set(v);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = a.bias ? a.bias[c + i] : 0.f;
    bias.set(v);
}

// The W - 1 inputs before token t0: from x, from the entering state, or zeros.
template <typename T, int V, int W>
__device__ __forceinline__ void load_window(const T *x, const T *first, int t0, int n, long long C,
                                            Lanes<V> (&win)[W - 1]) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int u = t0 - (W - 1) + j;
        Raw<T, V> r;
        r.load(u >= 0 ? x + u * C : first + (u + W - 1) * C, u >= 0 ? u < n : first != nullptr);
        win[j] = r.lanes();
    }
}

// s = bias + sum_j w[j] x[t-W+1+j], the window's inputs and the current one.
template <int V, int W>
__device__ __forceinline__ Lanes<V> convolve(const Lanes<V> (&w)[W], const Lanes<V> &bias, const Lanes<V> (&win)[W - 1],
                                             const Lanes<V> &cur) {
    Lanes<V> s = bias;
#pragma unroll
    for (int i = 0; i < Lanes<V>::n; ++i) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) s.e[i] = fma(w[j].e[i], win[j].e[i], s.e[i]);
        s.e[i] = fma(w[W - 1].e[i], cur.e[i], s.e[i]);
    }
    return s;
}

template <int V, int N>
__device__ __forceinline__ void shift(Lanes<V> (&win)[N], const Lanes<V> &cur) {
#pragma unroll
    for (int j = 0; j + 1 < N; ++j) win[j] = win[j + 1];
    win[N - 1] = cur;
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads)
conv_fwd_kernel(ConvArgs a, int cvecs, int segs) {
    typedef Lanes<V> L;
    constexpr int U = 4;                       // rows in flight
    const long long idx = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (idx >= (long long)a.B * segs * cvecs) return;
    int c, seg;
    const long long bs = split(idx, cvecs, c);
    c *= V;
    const int b = (int)split(bs, segs, seg);
    const int n = seq_end(a.lengths, b, a.T);
    const int t0 = seg * kSeg, t1 = min(t0 + kSeg, a.T);
    const long long C = a.C;
    const T *__restrict__ x = (const T *)a.x + (long long)b * a.T * C + c;
    T *__restrict__ y = (T *)a.y + (long long)b * a.T * C + c;
    const T *first = a.state_in ? (const T *)a.state_in + (long long)b * (W - 1) * C + c : nullptr;

    const int Ci = a.C, live = min(n, t1) - t0;        // rows of the segment that exist
    const T *__restrict__ px = x + t0 * C;
    T *__restrict__ py = y + t0 * C;
    if (live <= 0 && seg > 0) {
        Lanes<V> zero;
#pragma unroll
        for (int i = 0; i < L::n; ++i) zero.e[i] = L::splat(0.f);
        for (int u = 0; u < t1 - t0; ++u) store_lanes<V>(py + (long long)u * Ci, zero);
        return;
    }
    Raw<T, V> row[U];
#pragma unroll
    for (int u = 0; u < U; ++u) row[u].load(px + (long long)u * Ci, u < live);
    L w[W], bias, win[W - 1];
    load_taps<V, W>(a, c, w, bias);
    load_window<T, V, W>(x, first, t0, n, C, win);
    // The state after n tokens: rows n .. n + W - 2 of the sequence extended by the entering state.  It
    // leaves through the only thread that reads the entering one, so the two may be one buffer.
    if (seg == 0 && a.state_out) {
        Raw<T, V> keep[W - 1];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int r = n + j;
            keep[j].load(r >= W - 1 ? x + (r - (W - 1)) * C : first + r * C, r >= W - 1 || first);
        }
        T *so = (T *)a.state_out + (long long)b * (W - 1) * C + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) keep[j].store(so + j * C);
    }
#pragma unroll
    for (int h = 0; h < kSeg; h += U) {
        if (t0 + h >= t1) break;
        Raw<T, V> next[U];
        if (h + U < kSeg)
#pragma unroll
            for (int u = 0; u < U; ++u) next[u].load(px + (long long)(h + U + u) * Ci, h + U + u < live);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const L cur = row[u].lanes();
            L o = convolve<V, W>(w, bias, win, cur);
#pragma unroll
            for (int i = 0; i < L::n; ++i) {
                if (a.silu) o.e[i] = mul(o.e[i], sigmoid(o.e[i]));
                if (h + u >= live) o.e[i] = L::splat(0.f);
            }
            if (h + u < t1 - t0) store_lanes<V>(py + (long long)(h + u) * Ci, o);
            shift<V, W - 1>(win, cur);
        }
        if (h + U < kSeg)
#pragma unroll
            for (int u = 0; u < U; ++u) row[u] = next[u];
    }
}

// Backward.  Block: 32 channel vectors x kBwdSegs segments of `seg` tokens of one batch entry.
constexpr int kBwdSegs = 8;
constexpr int kBwdRows = 4;        // rows taken at a time

// U tokens from tb on.  Inner: all of them lie in the segment and the sequence, and so do the
// W - 1 tokens before them.
template <typename T, int V, int W, int U, bool INNER>
__device__ __forceinline__ void bwd_tokens(const ConvArgs &a, const Raw<T, V> (&rx)[U], const Raw<T, V> (&rg)[U],
                                           const Lanes<V> (&w)[W], const Lanes<V> &bias, Lanes<V> (&win)[W - 1],
                                           Lanes<V> (&gw)[W - 1], Lanes<V> (&dw)[W], Lanes<V> &db, int tb, int t0,
                                           int t1, int n, T *__restrict__ dx, T *dfirst, const T *ds) {
    typedef Lanes<V> L;
    const long long C = a.C;
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int t = tb + k;
        const L cur = rx[k].lanes();
        L g = rg[k].lanes();
        if (a.silu) {
            const L s = convolve<V, W>(w, bias, win, cur);
#pragma unroll
            for (int i = 0; i < L::n; ++i) {
                // sg (1 + s (1 - sg))
                const auto sg = sigmoid(s.e[i]), r = fma(sg, L::splat(-1.f), L::splat(1.f));
                g.e[i] = mul(mul(g.e[i], sg), fma(s.e[i], r, L::splat(1.f)));
            }
        }
#pragma unroll
        for (int i = 0; i < L::n; ++i) {
            if (!INNER && t >= n) g.e[i] = L::splat(0.f);
            if (INNER || (t < t1 && t < n)) {
                db.e[i] = add(db.e[i], g.e[i]);
#pragma unroll
                for (int j = 0; j < W - 1; ++j) dw[j].e[i] = fma(g.e[i], win[j].e[i], dw[j].e[i]);
                dw[W - 1].e[i] = fma(g.e[i], cur.e[i], dw[W - 1].e[i]);
            }
        }
        const int u = t - (W - 1);
        if (INNER || (u < t1 && (u >= t0 || (t0 == 0 && dfirst)))) {
            // dx[u] = sum_k w[W-1-k] g[u+k]: g[u] is the oldest in the window.  Only tokens that exist take
            // part (a tap may be infinite, and its product with a zero no zero).
            L d;
#pragma unroll
            for (int i = 0; i < L::n; ++i) {
                d.e[i] = INNER || t < n ? mul(w[0].e[i], g.e[i]) : L::splat(0.f);
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
                    if (INNER || (u + j >= 0 && u + j < n)) d.e[i] = fma(w[W - 1 - j].e[i], gw[j].e[i], d.e[i]);
            }
            if (INNER) {
                store_lanes<V>(dx + u * C, d);
            } else {
                const int j = u + (W - 1) - n;          // u's row of the leaving state
                if (ds && u < n && j >= 0) {
                    Raw<T, V> e;
                    e.load(ds + j * C);
                    const L el = e.lanes();
#pragma unroll
                    for (int i = 0; i < L::n; ++i) d.e[i] = add(d.e[i], el.e[i]);
                }
                store_lanes<V>(u >= 0 ? dx + u * C : dfirst + (u + W - 1) * C, d);
            }
        }
        shift<V, W - 1>(win, cur);
        shift<V, W - 1>(gw, g);
    }
}

// Rows of x and dy on their way to a thread, U at a time.  Where an access has at least 4 bytes they
// come through the thread's own places in shared memory by asynchronous copies, 2 to 4 groups ahead,
// so that no registers hold them; 2-byte accesses go to registers, one group ahead.
template <typename T, int V, int U, bool ASYNC = (sizeof(T) * V >= 4)> struct Feed;
template <typename T, int V, int U> struct Feed<T, V, U, true> {
    typedef typename WordsOf<sizeof(T) * V>::W Word;
    static constexpr int kAhead = sizeof(Word) == 16 ? 2 : 4;          // at most 64 KB a block: three blocks an SM
    static constexpr size_t bytes = sizeof(Word) * kAhead * U * 2 * 32 * kBwdSegs;
    Word *s;
    const T *x, *g;
    int t, have, slot;
    long long C;
    __device__ __forceinline__ Feed(void *smem, const T *x_, const T *g_, int t0, int have_, long long C_)
        : s((Word *)smem + threadIdx.x), x(x_ + t0 * C_), g(g_ + t0 * C_), t(t0), have(have_), slot(0), C(C_) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) put(i);
    }
    __device__ __forceinline__ Word *at(int place, int k, int which) {
        return s + ((place * U + k) * 2 + which) * (32 * kBwdSegs);
    }
    __device__ __forceinline__ void put(int place) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            copy_async<sizeof(Word)>(at(place, k, 0), x + k * C, t + k < have);
            copy_async<sizeof(Word)>(at(place, k, 1), g + k * C, t + k < have);
        }
        copy_commit();
        x += U * C;
        g += U * C;
        t += U;
    }
    __device__ __forceinline__ void take(Raw<T, V> (&rx)[U], Raw<T, V> (&rg)[U]) {
        copy_wait<kAhead - 1>();
#pragma unroll
        for (int k = 0; k < U; ++k) {
            rx[k].w = *at(slot, k, 0);
            rg[k].w = *at(slot, k, 1);
        }
        put(slot);
        slot = slot + 1 == kAhead ? 0 : slot + 1;
    }
};
template <typename T, int V, int U> struct Feed<T, V, U, false> {
    static constexpr size_t bytes = 0;
    Raw<T, V> nx[U], ng[U];
    const T *x, *g;
    int t, have;
    long long C;
    __device__ __forceinline__ Feed(void *, const T *x_, const T *g_, int t0, int have_, long long C_)
        : x(x_ + t0 * C_), g(g_ + t0 * C_), t(t0), have(have_), C(C_) { put(); }
    __device__ __forceinline__ void put() {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            nx[k].load(x + k * C, t + k < have);
            ng[k].load(g + k * C, t + k < have);
        }
        x += U * C;
        g += U * C;
        t += U;
    }
    __device__ __forceinline__ void take(Raw<T, V> (&rx)[U], Raw<T, V> (&rg)[U]) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            rx[k] = nx[k];
            rg[k] = ng[k];
        }
        put();
    }
};

template <typename T, int V, int W>
__global__ void __launch_bounds__(32 * kBwdSegs, W <= 4 ? 2 : 1)
conv_bwd_kernel(ConvArgs a, int seg, int blocks_t, int blocks_c, float *part) {
    typedef Lanes<V> L;
    // the rows on their way, and after them the segments' sums [kBwdSegs][kRed]
    extern __shared__ uint4 s_feed[];
    constexpr int kRed = 32 * V * (W + 1) + 1;
    float *red = reinterpret_cast<float *>(s_feed);
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
    const int p = blockIdx.x / blocks_c, bc = blockIdx.x - p * blocks_c;   // token block, channel block
    const int c = (bc * 32 + lane) * V;
    const int b = p / blocks_t, bt = p - b * blocks_t;
    const long long C = a.C;
    const bool live = c < a.C;
    L dw[W], db;
#pragma unroll
    for (int i = 0; i < L::n; ++i) {
        db.e[i] = L::splat(0.f);
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j].e[i] = L::splat(0.f);
    }
    const long long t0l = ((long long)bt * kBwdSegs + row) * seg;
    if (live && t0l < a.T) {
        constexpr int U = kBwdRows;
        const int t0 = (int)t0l, t1 = (int)min((long long)a.T, t0l + seg);
        const int n = seq_end(a.lengths, b, a.T), end = t1 + W - 1, have = min(n, end);
        const T *__restrict__ x = (const T *)a.x + (long long)b * a.T * C + c;
        const T *__restrict__ dy = (const T *)a.dy + (long long)b * a.T * C + c;
        T *__restrict__ dx = (T *)a.dx + (long long)b * a.T * C + c;
        const T *first = a.state_in ? (const T *)a.state_in + (long long)b * (W - 1) * C + c : nullptr;
        const T *ds = a.dstate_in ? (const T *)a.dstate_in + (long long)b * (W - 1) * C + c : nullptr;
        T *dfirst = a.dstate_out ? (T *)a.dstate_out + (long long)b * (W - 1) * C + c : nullptr;
        Feed<T, V, U> feed(s_feed, x, dy, t0, have, C);
        L w[W], bias, win[W - 1], gw[W - 1];
        load_taps<V, W>(a, c, w, bias);
        load_window<T, V, W>(x, first, t0, n, C, win);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int i = 0; i < L::n; ++i) gw[j].e[i] = L::splat(0.f);
        // at step t: g[t] is formed, and dx[u] with u = t - (W - 1) is complete
        for (int tb = t0; tb < end; tb += U) {
            Raw<T, V> rx[U], rg[U];
            feed.take(rx, rg);
            if (tb - (W - 1) >= t0 && tb + U <= min(t1, n))
                bwd_tokens<T, V, W, U, true>(a, rx, rg, w, bias, win, gw, dw, db, tb, t0, t1, n, dx, dfirst, ds);
            else
                bwd_tokens<T, V, W, U, false>(a, rx, rg, w, bias, win, gw, dw, db, tb, t0, t1, n, dx, dfirst, ds);
        }
        copy_wait<0>();
    }
    __syncthreads();
    {
        float v[V];
#pragma unroll
        for (int j = 0; j <= W; ++j) {
            (j < W ? dw[j] : db).get(v);
#pragma unroll
            for (int i = 0; i < V; ++i) red[row * kRed + (lane * V + i) * (W + 1) + j] = v[i];
        }
    }
    __syncthreads();
    const int n_out = min(32 * V, a.C - bc * 32 * V) * (W + 1);
    for (int e = threadIdx.x; e < n_out; e += 32 * kBwdSegs) {
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < kBwdSegs; ++r) s += red[r * kRed + e];
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
    wait_for_stream();
    if (e < n)
#pragma unroll 8
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
    const size_t sums = sizeof(float) * kBwdSegs * (32 * V * (W + 1) + 1), feed = Feed<T, V, kBwdRows>::bytes;
    la_status rc = launch("short_conv_bwd", conv_bwd_kernel<T, V, W>, dim3((unsigned)a.B * bt * bc),
                          dim3(32 * kBwdSegs), feed > sums ? feed : sums, st, a, seg, bt, bc, (float *)a.ws);
    if (rc != LA_OK) return rc;
    return launch_pdl("short_conv_bwd_reduce", conv_bwd_reduce, dim3((unsigned)((a.C * (W + 1) + 31) / 32)), dim3(256), 0,
                  st, (const float *)a.ws, a.B * bt, a.C, W, a.dw, a.dbias);
}

// At most 4 elements an access: 8 of 16 bits hold twice the taps and windows in registers and leave
// half the warps (B8 T4096 C2048 W4 bf16 forward 73 us at 8, 66 at 4).
template <typename T, int W>
la_status conv_w(bool bwd, const ConvArgs &a, cudaStream_t st) {
    int v = vec_width(sizeof(T), a.C, address_bits(a));
    if (bwd) {
        if (v >= 4) return bwd_v<T, 4, W>(a, st);
        return v == 2 ? bwd_v<T, 2, W>(a, st) : bwd_v<T, 1, W>(a, st);
    }
    if (v >= 4) return fwd_v<T, 4, W>(a, st);
    return v == 2 ? fwd_v<T, 2, W>(a, st) : fwd_v<T, 1, W>(a, st);
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

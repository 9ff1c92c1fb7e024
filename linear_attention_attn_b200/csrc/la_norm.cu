// la_norm.cu -- group normalisation with an activation, channels last, and its gradient.
//
//   xh = (x - mean) rstd over a group's channels and all positions of a batch entry,
//   a = gamma xh + beta,  y = act(a);
//   g = dy act'(a):  dbeta = sum g,  dgamma = sum g xh,
//   dx = rstd (gamma g - m0 - xh m1),  m0 = mean(gamma g),  m1 = mean(gamma g xh) over the group.
//
// Bound by HBM.  A group that fits a block's registers is read once (small kernels: a part of a
// warp, a warp, or a block a group; mean first, then the squares about it).  A larger one takes two
// launches over the same tiles of tokens, whole rows at a time: sums, then the result, the second
// walking every tile backwards so that it begins with what the first left in L2 last.  Against forwards,
// C640 G32 with SiLU: fp32 55 instead of 59 us at 84 MB, 100 instead of 104 at 168 (gradient 88 and 91, 157 and
// 162); f16 68 and 67, 110 and 108 us (gradient 96 and 93, 170 and 162), where the loads are the smaller part.
// Means and squares never meet as large sums: a thread sums about its own first value, then about the
// mean of its first 8, 16, 32, ... values (the first may lie far from the rest), and threads and tiles are
// joined through their means, sum M2_i + n_i (mean_i - mean)^2, so a mean far above the spread costs no
// precision.  Every sum runs in a fixed order.  An infinity (which is no pivot) makes its group's mean
// infinite, and like a NaN the variance and the whole group NaN, as the formula does.
// B2 T65536 C640 G32 f16 with SiLU (168 MB in, 168 out): 109 us, where two reads and a write at the
// measured copy bandwidth would take 77; the second launch's special-function units are 62 % busy
// (an exponential and a reciprocal an element), the memory 50 %.  B3 T4087 C330 G30 fp32 gradient:
// 25 us for 81 MB in five passes over tensors of 16 MB (two reads of x and dy, dx), mostly the two launches'
// start and joins.
#include "la_mixer.cuh"

namespace la {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

__device__ __forceinline__ float splat_like(float, float x) { return x; }
__device__ __forceinline__ f2 splat_like(f2, float x) { return both(x); }
// act(a), and g act'(a), of a float or a pair.
template <typename E>
__device__ __forceinline__ E act_of(E a, int silu) { return silu ? mul(a, sigmoid(a)) : a; }
template <typename E>
__device__ __forceinline__ E through_act(E g, E a, int silu) {
    if (!silu) return g;
    const E one = splat_like(a, 1.f), s = sigmoid(a), r = fma(s, splat_like(a, -1.f), one);
    return mul(mul(g, s), fma(a, r, one));
}

// ------------------------------------------------------- groups in registers --
// L lanes a group (a power of two up to 32, or the whole block of kSmallBlock), each with up to K
// vectors of V elements.
constexpr int kSmallBlock = 256;

// Sum over a group's L lanes; red has kSmallBlock / 32 floats and is free on return.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], int L, float (*red)[N]) {
    for (int m = L > 32 ? 16 : L / 2; m > 0; m >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], m);
    if (L <= 32) return;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) red[threadIdx.x >> 5][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = 0.f;
#pragma unroll
        for (int w = 0; w < kSmallBlock / 32; ++w) v[i] += red[w][i];
    }
    __syncthreads();
}

template <typename T, int V, int K>
__global__ void __launch_bounds__(kSmallBlock) norm_small_fwd(NormArgs a, int L, int nvec) {
    __shared__ float red[kSmallBlock / 32][1];
    const int cg = a.C / a.G, gl = cg / V, lane = threadIdx.x % L;
    const long long group = (long long)blockIdx.x * (kSmallBlock / L) + threadIdx.x / L;
    const bool live = group < (long long)a.B * a.G;
    const int b = live ? (int)(group / a.G) : 0, g = live ? (int)(group - (long long)b * a.G) : 0;
    const long long base = (long long)b * a.T * a.C + (long long)g * cg;
    const T *x = (const T *)a.x + base;
    float v[K][V], s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int e = lane + k * L, t = e / gl, c = (e - t * gl) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) v[k][i] = 0.f;
        if (live && e < nvec) {
            ldv<V>(x + (long long)t * a.C + c, v[k]);
#pragma unroll
            for (int i = 0; i < V; ++i) s[0] += v[k][i];
        }
    }
    group_sum<1>(s, L, red);
    const float count = (float)nvec * V, mean = s[0] / count;
    s[0] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (live && lane + k * L < nvec)
#pragma unroll
            for (int i = 0; i < V; ++i) s[0] = fmaf(v[k][i] - mean, v[k][i] - mean, s[0]);
    group_sum<1>(s, L, red);
    const float rstd = 1.f / sqrtf(s[0] / count + a.eps);
    if (!live) return;
    if (lane == 0) {
        if (a.mean) a.mean[group] = mean;
        if (a.rstd) a.rstd[group] = rstd;
    }
    T *y = (T *)a.y + base;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int e = lane + k * L, t = e / gl, c = (e - t * gl) * V;
        if (e < nvec) {
            float o[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int ch = g * cg + c + i;
                const float ga = a.gamma ? a.gamma[ch] : 1.f, be = a.beta ? a.beta[ch] : 0.f;
                o[i] = act_of(fmaf((v[k][i] - mean) * rstd, ga, be), a.silu);
            }
            stv<V>(y + (long long)t * a.C + c, o);
        }
    }
}

// T = 1: a group's lanes keep their channels and walk over the batch rows b0 .. b1, so dgamma and
// dbeta gather in registers; part [splits][C] takes them.
template <typename T, int V, int K>
__global__ void __launch_bounds__(kSmallBlock) norm_small_bwd(NormArgs a, int L, int nvec, int rows_per, float2 *part) {
    __shared__ float red[kSmallBlock / 32][2];
    const int cg = a.C / a.G, lane = threadIdx.x % L;
    const int g = blockIdx.x * (kSmallBlock / L) + threadIdx.x / L;
    const bool live = g < a.G;
    const int b0 = blockIdx.y * rows_per, b1 = min(a.B, b0 + rows_per);
    float ga[K][V], be[K][V], dga[K][V], dbe[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + k * L, ch = g * cg + e * V + i;
            const bool in = live && e < nvec;
            ga[k][i] = in && a.gamma ? a.gamma[ch] : 1.f;
            be[k][i] = in && a.beta ? a.beta[ch] : 0.f;
            dga[k][i] = dbe[k][i] = 0.f;
        }
    const float inv = 1.f / ((float)nvec * V);
    // the next row's values come while this one's are worked on
    Raw<T, V> rx[K], rg[K];
    float mean = 0.f, rstd = 0.f;
    auto load = [&](int b) {
        const long long base = (long long)b * a.C + (long long)g * cg;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int e = lane + k * L;
            rx[k].load((const T *)a.x + base + e * V, live && b < b1 && e < nvec);
            rg[k].load((const T *)a.dy + base + e * V, live && b < b1 && e < nvec);
        }
        mean = live && b < b1 ? a.mean_in[(long long)b * a.G + g] : 0.f;
        rstd = live && b < b1 ? a.rstd_in[(long long)b * a.G + g] : 0.f;
    };
    load(b0);
    for (int b = b0; b < b1; ++b) {
        const long long base = (long long)b * a.C + (long long)g * cg;
        const float mu = mean, rs = rstd;
        float xh[K][V], gr[K][V], s[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            rx[k].lanes().get(xh[k]);
            rg[k].lanes().get(gr[k]);
        }
        load(b + 1);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int e = lane + k * L;
            if (live && e < nvec) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    xh[k][i] = (xh[k][i] - mu) * rs;
                    gr[k][i] = through_act(gr[k][i], fmaf(xh[k][i], ga[k][i], be[k][i]), a.silu);
                    dbe[k][i] += gr[k][i];
                    dga[k][i] = fmaf(gr[k][i], xh[k][i], dga[k][i]);
                    gr[k][i] *= ga[k][i];
                    s[0] += gr[k][i];
                    s[1] = fmaf(gr[k][i], xh[k][i], s[1]);
                }
            }
        }
        group_sum<2>(s, L, red);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int e = lane + k * L;
            if (live && e < nvec) {
                float o[V];
#pragma unroll
                for (int i = 0; i < V; ++i) o[i] = rs * (gr[k][i] - s[0] * inv - xh[k][i] * (s[1] * inv));
                stv<V>((T *)a.dx + base + e * V, o);
            }
        }
    }
    if (!live || !part) return;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int e = lane + k * L;
        if (e < nvec)
#pragma unroll
            for (int i = 0; i < V; ++i)
                part[(long long)blockIdx.y * a.C + g * cg + e * V + i] = make_float2(dga[k][i], dbe[k][i]);
    }
}

// dgamma, dbeta from `parts` rows of [C] pairs: 32 channels a block, the warps over the rows.
__device__ __forceinline__ void join_channels(const float2 *part, int parts, int C, int block, float *dgamma,
                                              float *dbeta) {
    __shared__ float2 red[16][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int c = block * 32 + lane;
    float2 s = make_float2(0.f, 0.f);
    if (c < C)
#pragma unroll 8
        for (int p = warp; p < parts; p += warps) {
            const float2 v = part[(long long)p * C + c];
            s.x += v.x;
            s.y += v.y;
        }
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < C) {
        for (int w = 1; w < warps; ++w) {
            s.x += red[w][lane].x;
            s.y += red[w][lane].y;
        }
        if (dgamma) dgamma[c] = s.x;
        if (dbeta) dbeta[c] = s.y;
    }
}

__global__ void __launch_bounds__(512) norm_join(const float2 *part, int parts, int C, float *dgamma, float *dbeta) {
    wait_for_stream();
    join_channels(part, parts, C, blockIdx.x, dgamma, dbeta);
}

// --------------------------------------------------------------- tiled groups --
// A block: one batch entry, one tile of tokens, one chunk of whole groups.  Its threads lie along
// the chunk's `w` vectors of V channels, in `rows` rows of tokens; vectors may lie across group
// borders (every channel looks up its own group), so V need not divide a group.  A single group
// wider than the block is walked in strides (rows = 1).
constexpr int kTiledBlock = 512;
constexpr int kRows = 8;                   // rows that a thread has on their way at a time

// Calls f(first row, full) for batches of U rows; full says that all rows of the batch exist, so that
// its loads and stores need no tests.
struct Yes { static constexpr bool value = true; };
struct No { static constexpr bool value = false; };
template <int U, typename F>
__device__ __forceinline__ void batches(int rows, F f) {
    int k = 0;
    for (; k + U <= rows; k += U) f(k, Yes());
    if (k < rows) f(k, No());
}

struct Tiling {
    int gpc, chunks, w, rows, threads, tiles, len;
    __host__ __device__ bool strided() const { return w > threads; }
};

// What a block of a tiled launch works on.
struct Where {
    int chunk, tile, b, cg, g0, ng, w, r, v0, t0, t1;
    long long base;                        // offset of the chunk's first channel at token 0
    __device__ __forceinline__ Where(const NormArgs &a, const Tiling &q, int V) {
        long long block = blockIdx.x;
        block = split(block, q.chunks, chunk);
        b = (int)split(block, q.tiles, tile);
        cg = a.C / a.G;
        g0 = chunk * q.gpc;
        ng = min(q.gpc, a.G - g0);
        w = ng * cg / V;
        r = threadIdx.x / q.w;
        v0 = threadIdx.x - r * q.w;
        t0 = tile * q.len;
        t1 = min(a.T, t0 + q.len);
        base = (long long)b * a.T * a.C + (long long)g0 * cg;
    }
    // tokens of row r of the tile
    __device__ __forceinline__ int tokens(const Tiling &q, int row) const {
        return row < q.rows && t0 + row < t1 ? (t1 - t0 - row + q.rows - 1) / q.rows : 0;
    }
};

// Moves the (negated) pivot of n values per channel, whose distances from it sum up to s and whose
// squares to sq, by their mean distance d: s - n d and sq - d (s + (s - n d)).
template <int V>
__device__ __forceinline__ void recentre(Lanes<V> &pivot, Lanes<V> &s, Lanes<V> &sq, float n) {
    float vp[V], vs[V], vq[V];
    pivot.get(vp);
    s.get(vs);
    sq.get(vq);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float to = vp[i] - vs[i] / n, d = vp[i] - to;        // the step as it was rounded
        if (finite(d)) {
            const float left = fmaf(-n, d, vs[i]);
            vq[i] = fmaf(-d, vs[i] + left, vq[i]);
            vs[i] = left;
            vp[i] = to;
        }
    }
    pivot.set(vp);
    s.set(vs);
    sq.set(vq);
}

// part [B tiles][G]: a tile's mean and sum of squares about it.
template <typename T, int V>
__global__ void __launch_bounds__(kTiledBlock, 2) norm_stats(NormArgs a, Tiling q, float2 *part) {
    typedef Lanes<V> L;
    extern __shared__ float2 s_sum[];      // (mean, M2) of [rows][w V] channels, or of the threads where strided
    __shared__ int s_n[kTiledBlock];       // strided: values of a thread
    const Where at(a, q, V);
    const int rows = at.tokens(q, at.r);
    const long long step = (long long)q.rows * a.C;
    float n = 0.f, mean = 0.f, m2 = 0.f;
    if (rows > 0)
        for (int v = at.v0; v < at.w; v += q.threads) {
            const T *p = (const T *)a.x + at.base + (long long)(at.t0 + at.r) * a.C + v * V;
            L pivot, s, sq;                // pivot: negated
            {
                float first[V];
                ldv<V>(p, first);
#pragma unroll
                for (int i = 0; i < V; ++i) first[i] = finite(first[i]) ? -first[i] : 0.f;
                pivot.set(first);
            }
#pragma unroll
            for (int i = 0; i < L::n; ++i) s.e[i] = sq.e[i] = L::splat(0.f);
            batches<kRows>(rows, [&](int k, auto full) {
                constexpr bool FULL = decltype(full)::value;
                Raw<T, V> row[kRows];
#pragma unroll
                for (int u = 0; u < kRows; ++u) row[u].load(p + u * step, FULL || k + u < rows);
#pragma unroll
                for (int u = 0; u < kRows; ++u)
                    if (FULL || k + u < rows) {
                        const L e = row[u].lanes();
#pragma unroll
                        for (int i = 0; i < L::n; ++i) {
                            const auto d = add(e.e[i], pivot.e[i]);
                            s.e[i] = add(s.e[i], d);
                            sq.e[i] = fma(d, d, sq.e[i]);
                        }
                    }
                p += kRows * step;
                // The pivot moves to the mean of the rows so far when their number doubles (8, 16, 32, ...):
                // about it, sq is at most twice the squares about the mean, however far away the first row lay.
                const int done = k + kRows;
                if (FULL && done < rows && (done & (done - 1)) == 0) recentre<V>(pivot, s, sq, (float)done);
            });
            float vp[V], vs[V], vq[V];
            pivot.get(vp);
            s.get(vs);
            sq.get(vq);
            const float inv = 1.f / rows;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float m = vs[i] * inv, c_mean = m - vp[i], c_m2 = vq[i] - vs[i] * m;
                if (!q.strided()) {
                    s_sum[(at.r * q.w + v) * V + i] = make_float2(c_mean, c_m2);
                } else {
                    const float d = c_mean - mean, all = n + rows;
                    mean += finite(d) ? d * (rows / all) : c_mean;
                    m2 += c_m2 + d * d * (n * rows / all);
                    n = all;
                }
            }
        }
    if (q.strided()) {
        s_n[threadIdx.x] = (int)n;
        s_sum[threadIdx.x] = make_float2(mean, m2);
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, members = q.strided() ? q.threads : q.rows * at.cg;
    for (int j = threadIdx.x >> 5; j < at.ng; j += q.threads >> 5) {
        auto member = [&](int e, float &cnt) {
            if (q.strided()) {
                cnt = (float)s_n[e];
                return s_sum[e];
            }
            const int row = e / at.cg;
            cnt = (float)at.tokens(q, row);
            return cnt > 0.f ? s_sum[row * q.w * V + j * at.cg + (e - row * at.cg)] : make_float2(0.f, 0.f);
        };
        float all = 0.f, sm = 0.f, sq = 0.f, cnt;
        for (int e = lane; e < members; e += 32) {
            const float2 m = member(e, cnt);
            all += cnt;
            sm = fmaf(cnt, m.x, sm);
        }
        all = warp_sum(all);
        const float mu = warp_sum(sm) / all;
        for (int e = lane; e < members; e += 32) {
            const float2 m = member(e, cnt);
            const float d = m.x - mu;
            sq += fmaf(cnt * d, d, m.y);
        }
        sq = warp_sum(sq);
        if (lane == 0) part[((long long)at.b * q.tiles + at.tile) * a.G + at.g0 + j] = make_float2(mu, sq);
    }
}

// gamma and beta of V channels from c on.
template <int V>
__device__ __forceinline__ void load_affine(const NormArgs &a, int c, Lanes<V> &ga, Lanes<V> &be) {
    float g[V], b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        g[i] = a.gamma ? a.gamma[c + i] : 1.f;
        b[i] = a.beta ? a.beta[c + i] : 0.f;
    }
    ga.set(g);
    be.set(b);
}

// factor * p[group] of the V channels of vector v, p indexed by the chunk's groups.
template <int V>
__device__ __forceinline__ Lanes<V> by_group(const float *p, int v, int cg, float factor) {
    float x[V];
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = factor * p[(v * V + i) / cg];
    Lanes<V> r;
    r.set(x);
    return r;
}

// A lane's part of a group's sums over the tiles, all loads at once (zeros behind the last tile).
constexpr int kTileTarget = 2 * 148;       // blocks of a tiled launch: two of 512 threads an SM
constexpr int kTileLoads = (kTileTarget + 31) / 32;
__device__ __forceinline__ void load_tiles(const float2 *p, int tiles, int G, int lane, float2 (&v)[kTileLoads]) {
#pragma unroll
    for (int i = 0; i < kTileLoads; ++i)
        v[i] = i * 32 + lane < tiles ? p[(long long)(i * 32 + lane) * G] : make_float2(0.f, 0.f);
}

template <typename T, int V>
__global__ void __launch_bounds__(kTiledBlock, 2) norm_apply(NormArgs a, Tiling q, const float2 *part) {
    typedef Lanes<V> L;
    extern __shared__ float s_group[];     // mean, rstd [2][gpc]
    float *s_mean = s_group, *s_rstd = s_group + q.gpc;
    const Where at(a, q, V);
    wait_for_stream();
    const int lane = threadIdx.x & 31;
    const float total = (float)a.T * at.cg;
    for (int j = threadIdx.x >> 5; j < at.ng; j += q.threads >> 5) {
        float2 v[kTileLoads];
        load_tiles(part + (long long)at.b * q.tiles * a.G + at.g0 + j, q.tiles, a.G, lane, v);
        float sm = 0.f, sq = 0.f;
#pragma unroll
        for (int i = 0; i < kTileLoads; ++i) {
            const int tile = i * 32 + lane;
            if (tile < q.tiles) sm = fmaf((float)min(q.len, a.T - tile * q.len) * at.cg, v[i].x, sm);
        }
        const float mean = warp_sum(sm) / total;
#pragma unroll
        for (int i = 0; i < kTileLoads; ++i) {
            const int tile = i * 32 + lane;
            const float d = v[i].x - mean;
            if (tile < q.tiles) sq += fmaf((float)min(q.len, a.T - tile * q.len) * at.cg * d, d, v[i].y);
        }
        sq = warp_sum(sq);
        const float rstd = 1.f / sqrtf((sq < 0.f ? 0.f : sq) / total + a.eps);      // a NaN stays one
        if (lane == 0) {
            s_mean[j] = mean;
            s_rstd[j] = rstd;
            if (at.tile == 0) {
                if (a.mean) a.mean[(long long)at.b * a.G + at.g0 + j] = mean;
                if (a.rstd) a.rstd[(long long)at.b * a.G + at.g0 + j] = rstd;
            }
        }
    }
    __syncthreads();
    const int rows = at.tokens(q, at.r);
    if (rows == 0) return;
    const long long step = -(long long)q.rows * a.C;
    for (int v = at.v0; v < at.w; v += q.threads) {
        const L minus = by_group<V>(s_mean, v, at.cg, -1.f), rstd = by_group<V>(s_rstd, v, at.cg, 1.f);
        L ga, be;
        load_affine<V>(a, at.g0 * at.cg + v * V, ga, be);
#pragma unroll
        for (int i = 0; i < L::n; ++i) ga.e[i] = mul(ga.e[i], rstd.e[i]);
        long long o = at.base + v * V + (long long)(at.t0 + at.r) * a.C - (rows - 1) * step;      // the last row
        batches<kRows>(rows, [&](int k, auto full) {
            constexpr bool FULL = decltype(full)::value;
            // all loads before the first store, which the compiler may not pass (y may be x)
            Raw<T, V> row[kRows];
#pragma unroll
            for (int u = 0; u < kRows; ++u) row[u].load((const T *)a.x + o + u * step, FULL || k + u < rows);
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                L e = row[u].lanes();
#pragma unroll
                for (int i = 0; i < L::n; ++i) e.e[i] = act_of(fma(add(e.e[i], minus.e[i]), ga.e[i], be.e[i]), a.silu);
                if (FULL || k + u < rows) store_lanes<V>((T *)a.y + o + u * step, e);
            }
            o += kRows * step;
        });
    }
}

// Sums of a tile: chan [B tiles][C] (sum g xh, sum g), part [B tiles][G] (sum gamma g, sum gamma g xh).
template <typename T, int V>
__global__ void __launch_bounds__(kTiledBlock, 2) norm_bwd_sums(NormArgs a, Tiling q, float2 *part, float2 *chan) {
    typedef Lanes<V> L;
    extern __shared__ float2 s_sum[];      // channels' sums [rows][w V], or the threads' of the group where strided
    const Where at(a, q, V);
    const int rows = at.tokens(q, at.r), width = at.w * V;
    const long long step = (long long)q.rows * a.C;
    const float *mean = a.mean_in + (long long)at.b * a.G + at.g0, *rstd = a.rstd_in + (long long)at.b * a.G + at.g0;
    float2 *out = chan + ((long long)at.b * q.tiles + at.tile) * a.C + (long long)at.g0 * at.cg;
    float2 grp = make_float2(0.f, 0.f);
    if (at.r < q.rows)
        for (int v = at.v0; v < at.w; v += q.threads) {
            const L minus = by_group<V>(mean, v, at.cg, -1.f), scale = by_group<V>(rstd, v, at.cg, 1.f);
            L ga, be, dg, db;
            load_affine<V>(a, at.g0 * at.cg + v * V, ga, be);
#pragma unroll
            for (int i = 0; i < L::n; ++i) dg.e[i] = db.e[i] = L::splat(0.f);
            const T *x = (const T *)a.x + at.base + (long long)(at.t0 + at.r) * a.C + v * V;
            const T *dy = (const T *)a.dy + at.base + (long long)(at.t0 + at.r) * a.C + v * V;
            constexpr int U = kRows / 2;
            batches<U>(rows, [&](int k, auto full) {
                constexpr bool FULL = decltype(full)::value;
                Raw<T, V> rx[U], rg[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    rx[u].load(x + u * step, FULL || k + u < rows);
                    rg[u].load(dy + u * step, FULL || k + u < rows);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const L e = rx[u].lanes(), d = rg[u].lanes();
#pragma unroll
                    for (int i = 0; i < L::n; ++i) {
                        const auto xh = mul(add(e.e[i], minus.e[i]), scale.e[i]);
                        auto g = through_act(d.e[i], fma(xh, ga.e[i], be.e[i]), a.silu);
                        if (!FULL && k + u >= rows) g = L::splat(0.f);
                        db.e[i] = add(db.e[i], g);
                        dg.e[i] = fma(g, xh, dg.e[i]);
                    }
                }
                x += U * step;
                dy += U * step;
            });
            float vga[V], vdg[V], vdb[V];
            ga.get(vga);
            dg.get(vdg);
            db.get(vdb);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (!q.strided()) {
                    s_sum[(at.r * q.w + v) * V + i] = make_float2(vdg[i], vdb[i]);
                } else {
                    out[v * V + i] = make_float2(vdg[i], vdb[i]);
                    grp.x = fmaf(vga[i], vdb[i], grp.x);
                    grp.y = fmaf(vga[i], vdg[i], grp.y);
                }
            }
        }
    if (q.strided()) s_sum[threadIdx.x] = grp;
    __syncthreads();
    if (!q.strided()) {
        for (int e = threadIdx.x; e < width; e += q.threads) {
            float2 s = s_sum[e];
            for (int k = 1; k < q.rows; ++k) {
                const float2 u = s_sum[k * q.w * V + e];
                s.x += u.x;
                s.y += u.y;
            }
            out[e] = s;
            const float ga = a.gamma ? a.gamma[at.g0 * at.cg + e] : 1.f;
            s_sum[e] = make_float2(ga * s.y, ga * s.x);          // what the group sums up
        }
        __syncthreads();
    }
    const int lane = threadIdx.x & 31, members = q.strided() ? q.threads : at.cg;
    for (int j = threadIdx.x >> 5; j < at.ng; j += q.threads >> 5) {
        float s0 = 0.f, s1 = 0.f;
        for (int e = lane; e < members; e += 32) {
            const float2 u = s_sum[j * at.cg + e];               // strided: a single group, j = 0
            s0 += u.x;
            s1 += u.y;
        }
        s0 = warp_sum(s0);
        s1 = warp_sum(s1);
        if (lane == 0) part[((long long)at.b * q.tiles + at.tile) * a.G + at.g0 + j] = make_float2(s0, s1);
    }
}

// dx; the blocks from `main_blocks` on join dgamma and dbeta instead.
template <typename T, int V>
__global__ void __launch_bounds__(kTiledBlock, 2)
norm_bwd_apply(NormArgs a, Tiling q, const float2 *part, const float2 *chan, unsigned main_blocks) {
    typedef Lanes<V> L;
    extern __shared__ float s_group[];     // mean(gamma g), mean(gamma g xh) [2][gpc]
    float *s_m0 = s_group, *s_m1 = s_group + q.gpc;
    wait_for_stream();
    if (blockIdx.x >= main_blocks) {
        join_channels(chan, a.B * q.tiles, a.C, blockIdx.x - main_blocks, a.dgamma, a.dbeta);
        return;
    }
    const Where at(a, q, V);
    const int lane = threadIdx.x & 31;
    const float inv = 1.f / ((float)a.T * at.cg);
    for (int j = threadIdx.x >> 5; j < at.ng; j += q.threads >> 5) {
        float2 v[kTileLoads];
        load_tiles(part + (long long)at.b * q.tiles * a.G + at.g0 + j, q.tiles, a.G, lane, v);
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int i = 0; i < kTileLoads; ++i) {
            s0 += v[i].x;
            s1 += v[i].y;
        }
        s0 = warp_sum(s0);
        s1 = warp_sum(s1);
        if (lane == 0) {
            s_m0[j] = s0 * inv;
            s_m1[j] = s1 * inv;
        }
    }
    __syncthreads();
    const int rows = at.tokens(q, at.r);
    if (rows == 0) return;
    const long long step = -(long long)q.rows * a.C;
    const float *mean = a.mean_in + (long long)at.b * a.G + at.g0, *rstd = a.rstd_in + (long long)at.b * a.G + at.g0;
    for (int v = at.v0; v < at.w; v += q.threads) {
        const L minus = by_group<V>(mean, v, at.cg, -1.f), scale = by_group<V>(rstd, v, at.cg, 1.f);
        const L m0 = by_group<V>(s_m0, v, at.cg, -1.f), m1 = by_group<V>(s_m1, v, at.cg, -1.f);
        L ga, be;
        load_affine<V>(a, at.g0 * at.cg + v * V, ga, be);
        long long o = at.base + v * V + (long long)(at.t0 + at.r) * a.C - (rows - 1) * step;      // the last row
        constexpr int U = kRows / 2;
        batches<U>(rows, [&](int k, auto full) {
            constexpr bool FULL = decltype(full)::value;
            // all loads before the first store, which the compiler may not pass (dx may be dy)
            Raw<T, V> rx[U], rg[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                rx[u].load((const T *)a.x + o + u * step, FULL || k + u < rows);
                rg[u].load((const T *)a.dy + o + u * step, FULL || k + u < rows);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const L e = rx[u].lanes();
                L d = rg[u].lanes();
#pragma unroll
                for (int i = 0; i < L::n; ++i) {
                    const auto xh = mul(add(e.e[i], minus.e[i]), scale.e[i]);
                    const auto g = through_act(d.e[i], fma(xh, ga.e[i], be.e[i]), a.silu);
                    d.e[i] = mul(scale.e[i], fma(xh, m1.e[i], fma(g, ga.e[i], m0.e[i])));
                }
                if (FULL || k + u < rows) store_lanes<V>((T *)a.dx + o + u * step, d);
            }
            o += U * step;
        });
    }
}

// -------------------------------------------------------------------- choices --

int pow2_at_least(long long n) {
    int p = 1;
    while (p < n) p *= 2;
    return p;
}

// Most tiles of a batch entry, whatever the access width.
int most_tiles(int B, int T) {
    const long long n = (kTileTarget + B - 1) / B;
    return (int)(n < T ? n : T);
}

// Groups of a chunk for vectors of V channels: as many as fill a block's threads, in whole vectors
// (0: none).
int chunk_groups(const NormArgs &a, int V) {
    const long long cg = a.C / a.G;
    if (a.C <= (long long)kTiledBlock * V) return a.G;
    for (long long g = kTiledBlock * (long long)V / cg; g > 1; --g)
        if (g * cg % V == 0) return (int)g;
    return cg % V == 0 ? 1 : 0;
}

// Widest vector that the addresses allow, divides the rows and leaves whole chunks; at most `most`.
int tiled_width(const NormArgs &a, int most) {
    const uintptr_t bits = (uintptr_t)a.x | (uintptr_t)a.y | (uintptr_t)a.dy | (uintptr_t)a.dx;
    int v = vec_width(elem_bytes(a.dt), a.C, bits);
    if (v > most) v = most;
    while (chunk_groups(a, v) == 0) v >>= 1;        // 1 always serves
    return v;
}

Tiling tiling(const NormArgs &a, int V) {
    Tiling q;
    q.gpc = chunk_groups(a, V);
    q.chunks = (a.G + q.gpc - 1) / q.gpc;
    q.w = q.gpc * (a.C / a.G) / V;
    q.rows = q.w >= kTiledBlock ? 1 : kTiledBlock / q.w;
    if (q.rows > a.T) q.rows = a.T;
    const int need = q.rows * q.w;
    q.threads = need >= kTiledBlock ? kTiledBlock : (need + 31) / 32 * 32;
    // rounded down: a few blocks more than fit at once would take a second turn of the whole GPU
    long long want = kTileTarget / ((long long)a.B * q.chunks);
    if (want < 1) want = 1;
    const long long most = (a.T + 4 * q.rows - 1) / (4 * q.rows);          // at least 4 tokens a thread
    if (want > most) want = most;
    q.len = (int)((a.T + want - 1) / want);
    q.tiles = (a.T + q.len - 1) / q.len;
    return q;
}

// Shared memory of the sums: a pair a channel and row, or a thread.
size_t sums_smem(const Tiling &q, int V) {
    const size_t n = q.strided() ? q.threads : (size_t)q.rows * q.w * V;
    return sizeof(float2) * n;
}

// The register kernels' vectors lie within a group.
int width_for(const NormArgs &a) {
    const uintptr_t bits = (uintptr_t)a.x | (uintptr_t)a.y | (uintptr_t)a.dy | (uintptr_t)a.dx;
    return vec_width(elem_bytes(a.dt), (long long)(a.C / a.G), bits);
}

// A group of at most 2048 vectors fits a block's registers.  It is taken from there where its rows
// are at least 64 bytes (T = 1 always: neighbouring groups share the sectors of one row) or the
// whole tensor is small; else narrow rows would be fetched in part-used sectors.
bool small_fwd(const NormArgs &a, int V) {
    const long long nvec = (long long)a.T * (a.C / a.G) / V;
    const size_t row = (size_t)(a.C / a.G) * elem_bytes(a.dt), all = (size_t)a.B * a.T * a.C * elem_bytes(a.dt);
    return nvec <= 8 * kSmallBlock && (a.T == 1 || row >= 64 || all <= ((size_t)4 << 20));
}

void small_lanes(long long nvec, int *L, int *K) {
    if (nvec <= 128) {
        *L = nvec >= 32 ? 32 : pow2_at_least(nvec);
        *K = pow2_at_least((nvec + *L - 1) / *L);
    } else {
        *L = kSmallBlock;
        *K = pow2_at_least((nvec + kSmallBlock - 1) / kSmallBlock);
    }
}

template <typename T, int V>
la_status small_fwd_v(const NormArgs &a, cudaStream_t st) {
    const int nvec = a.T * (a.C / a.G) / V;
    int L, K;
    small_lanes(nvec, &L, &K);
    const long long per = kSmallBlock / L;
    const dim3 grid((unsigned)(((long long)a.B * a.G + per - 1) / per)), block(kSmallBlock);
    switch (K) {
    case 1: return launch("group_norm_fwd", norm_small_fwd<T, V, 1>, grid, block, 0, st, a, L, nvec);
    case 2: return launch("group_norm_fwd", norm_small_fwd<T, V, 2>, grid, block, 0, st, a, L, nvec);
    case 4: return launch("group_norm_fwd", norm_small_fwd<T, V, 4>, grid, block, 0, st, a, L, nvec);
    default: return launch("group_norm_fwd", norm_small_fwd<T, V, 8>, grid, block, 0, st, a, L, nvec);
    }
}

template <typename T, int V>
la_status tiled_fwd_v(const NormArgs &a, cudaStream_t st) {
    const Tiling q = tiling(a, V);
    const dim3 grid((unsigned)((long long)a.B * q.tiles * q.chunks)), block(q.threads);
    la_status rc = launch("group_norm_stats", norm_stats<T, V>, grid, block, sums_smem(q, V), st, a, q, (float2 *)a.ws);
    if (rc != LA_OK) return rc;
    return launch_pdl("group_norm_fwd", norm_apply<T, V>, grid, block, sizeof(float) * 2 * q.gpc, st, a, q,
                  (const float2 *)a.ws);
}

// Lanes of a group in the T = 1 backward.
int bwd_lanes(int nvec) { return nvec > 64 ? kSmallBlock : nvec >= 32 ? 32 : pow2_at_least(nvec); }

// Batch rows a block of the T = 1 backward walks over: about eight blocks an SM, at most 512 parts (as
// for aligned tensors: the workspace's size does not go by addresses).
int rows_per_block(int B, int G, int cg, la_dtype dt) {
    const int per = kSmallBlock / bwd_lanes(cg / vec_width(elem_bytes(dt), cg, 0));
    long long splits = 8 * 148LL / ((G + per - 1) / per) + 1;
    if (splits > 512) splits = 512;
    if (splits > B) splits = B;
    return (int)((B + splits - 1) / splits);
}

// T = 1 with at most 16 channels a thread of a block (kept twice as sums, twice as values).
bool small_bwd(int T, long long cg) { return T == 1 && cg <= 16 * kSmallBlock; }

template <typename T, int V, int K>
la_status small_bwd_k(const NormArgs &a, int L, int nvec, int per, float2 *part, cudaStream_t st) {
    if constexpr (K * V <= 16) {
        const dim3 grid((a.G + kSmallBlock / L - 1) / (kSmallBlock / L), (a.B + per - 1) / per);
        return launch("group_norm_bwd", norm_small_bwd<T, V, K>, grid, dim3(kSmallBlock), 0, st, a, L, nvec, per, part);
    } else {
        return LA_ERR_UNSUPPORTED;       // K V <= 16 for every size that small_bwd admits
    }
}

template <typename T, int V>
la_status small_bwd_v(const NormArgs &a, cudaStream_t st) {
    const bool join = a.dgamma || a.dbeta;
    const int nvec = a.C / a.G / V;
    const int L = bwd_lanes(nvec);
    const int per = rows_per_block(a.B, a.G, a.C / a.G, a.dt), splits = (a.B + per - 1) / per;
    float2 *part = join ? (float2 *)a.ws : nullptr;
    la_status rc;
    switch (pow2_at_least((nvec + L - 1) / L)) {
    case 1: rc = small_bwd_k<T, V, 1>(a, L, nvec, per, part, st); break;
    case 2: rc = small_bwd_k<T, V, 2>(a, L, nvec, per, part, st); break;
    case 4: rc = small_bwd_k<T, V, 4>(a, L, nvec, per, part, st); break;
    case 8: rc = small_bwd_k<T, V, 8>(a, L, nvec, per, part, st); break;
    default: rc = small_bwd_k<T, V, 16>(a, L, nvec, per, part, st); break;
    }
    if (rc != LA_OK || !join) return rc;
    return launch_pdl("group_norm_bwd_join", norm_join, dim3((a.C + 31) / 32), dim3(512), 0, st, (const float2 *)part,
                  splits, a.C, a.dgamma, a.dbeta);
}

template <typename T, int V>
la_status tiled_bwd_v(const NormArgs &a, cudaStream_t st) {
    const bool join = a.dgamma || a.dbeta;
    const Tiling q = tiling(a, V);
    float2 *part = (float2 *)a.ws, *chan = (float2 *)((char *)a.ws + up256(sizeof(float2) * a.B * q.tiles * a.G));
    const unsigned blocks = (unsigned)((long long)a.B * q.tiles * q.chunks);
    la_status rc = launch("group_norm_bwd_sums", norm_bwd_sums<T, V>, dim3(blocks), dim3(q.threads), sums_smem(q, V),
                          st, a, q, part, chan);
    if (rc != LA_OK) return rc;
    return launch_pdl("group_norm_bwd", norm_bwd_apply<T, V>, dim3(blocks + (join ? (a.C + 31) / 32 : 0)),
                  dim3(q.threads), sizeof(float) * 2 * q.gpc, st, a, q, (const float2 *)part, (const float2 *)chan,
                  blocks);
}

// The tiled kernels take at most 4 channels a vector: 8 of 16 bits leave no registers for as many rows
// on their way (B2 T65536 C640 f16 sums: 63 us at 8, 46 us at 4).
template <typename T>
la_status norm_t(bool bwd, const NormArgs &a, cudaStream_t st) {
    const int v = width_for(a);
    if (bwd && small_bwd(a.T, a.C / a.G)) {
        switch (v) {
        case 8: return small_bwd_v<T, 16 / sizeof(T)>(a, st);
        case 4: return small_bwd_v<T, 4>(a, st);
        case 2: return small_bwd_v<T, 2>(a, st);
        default: return small_bwd_v<T, 1>(a, st);
        }
    }
    if (bwd) {
        switch (tiled_width(a, 4)) {
        case 4: return tiled_bwd_v<T, 4>(a, st);
        case 2: return tiled_bwd_v<T, 2>(a, st);
        default: return tiled_bwd_v<T, 1>(a, st);
        }
    }
    if (small_fwd(a, v)) {
        switch (v) {
        case 8: return small_fwd_v<T, 16 / sizeof(T)>(a, st);
        case 4: return small_fwd_v<T, 4>(a, st);
        case 2: return small_fwd_v<T, 2>(a, st);
        default: return small_fwd_v<T, 1>(a, st);
        }
    }
    switch (tiled_width(a, 4)) {
    case 4: return tiled_fwd_v<T, 4>(a, st);
    case 2: return tiled_fwd_v<T, 2>(a, st);
    default: return tiled_fwd_v<T, 1>(a, st);
    }
}

la_status norm_d(bool bwd, const NormArgs &a, cudaStream_t st) {
    switch (a.dt) {
    case LA_F32: return norm_t<float>(bwd, a, st);
    case LA_F16: return norm_t<__half>(bwd, a, st);
    default: return norm_t<__nv_bfloat16>(bwd, a, st);
    }
}

}  // namespace

size_t norm_fwd_workspace(int B, int T, int C, int G, la_dtype) {
    if (T == 0 || (T == 1 && C / G <= 8 * kSmallBlock)) return 0;      // in registers at any access width
    return up256(sizeof(float2) * B * most_tiles(B, T) * G);
}

size_t norm_bwd_workspace(int B, int T, int C, int G, la_dtype dt) {
    if (T == 0) return 0;
    if (small_bwd(T, C / G)) {
        const int per = rows_per_block(B, G, C / G, dt), splits = (B + per - 1) / per;
        return up256(sizeof(float2) * splits * C);
    }
    return up256(sizeof(float2) * B * most_tiles(B, T) * G) + up256(sizeof(float2) * B * most_tiles(B, T) * C);
}

la_status norm_fwd(const NormArgs &a, cudaStream_t st) { return norm_d(false, a, st); }
la_status norm_bwd(const NormArgs &a, cudaStream_t st) { return norm_d(true, a, st); }

}  // namespace la

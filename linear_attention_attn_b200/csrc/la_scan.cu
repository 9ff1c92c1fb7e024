// la_scan.cu -- selective state space scan, forward: whole sequences and single tokens.
//
//   h_t[n] = exp(d_t A[n]) h_{t-1}[n] + d_t x_t B_t[n],   y_t = (sum_n C_t[n] h_t[n] + D x_t) silu(z_t)
// per channel, with d_t = softplus(dt_t + bias).
//
// What bounds it: one exponential for every (token, channel, state).  At N = 16 a channel's token
// moves 8 bytes of x, dt, z and y and costs 16 exponentials and 4 special functions more (softplus, gate);
// an SM makes 16 a cycle in its special-function units, so they take 3.5 times as long as the traffic.
//
// A block owns 64 / LN channels of one batch entry and walks over its tokens in tiles of 16.  The
// rows of x, dt, z, B and C come in four elements an access, two tiles ahead, in registers; each
// d_t, d_t x_t is formed once and left in shared memory for the LN lanes that share it; states live in
// registers, in packed arithmetic.  Every fourth token the lanes of a channel exchange halves of
// their four partial sums, so a sum over n costs 3 shuffles for 4 tokens.
// Measured at B8 T4096 C2048 N16 bf16: 557 us, where the special functions alone would take 288 and the
// traffic 83; special-function units 53 %, issue slots 56 % busy, 3.5 warps a scheduler.  Blocks of two
// warps (not four or one tile of 32 tokens: 560, 702 us) spread most evenly over 148 SMs.
//
// Where the batch and channels alone give too few blocks, the sequence is cut into segments: the
// first launch runs segment 0 in full and the others for their end state from zero and their sum
// of d (a segment's decay is exp(A sum d), so no product is kept); the second starts every later
// segment from the states before it, joined in order.
#include "la_scan.cuh"

namespace la {
namespace {

using namespace scan;

constexpr int kThreads = 64;

template <int LN> struct Cfg {
    static constexpr int width = kThreads / LN;             // channels a block
    static constexpr int pairs = kTile * width;             // (token, channel)
    static constexpr int quads = pairs / 4;                 // 4 channels of a token, staged by one thread
    static constexpr int per = (quads + kThreads - 1) / kThreads;
    static constexpr int bquads = kTile * LN;               // 4 states of a token's B (or C)
    static constexpr int bper = (bquads + kThreads - 1) / kThreads;
    // Blocks an SM that the kernels for padded states are held to.  They keep more in registers; without a
    // bound N = 6 bf16 came to 138 and 225 us (B8 T2048 C1024; 168 with no state kept at 0), held to 128
    // registers 179 us.  One and four lanes (N < 4, 9 .. 16) take what they like: N = 12 bf16 186 us, 234 held.
    template <typename T> static constexpr int fit() {
        return LN == 1 || LN == 4 ? 1 : sizeof(T) == 4 ? (LN == 8 ? 8 : 6) : (LN == 8 ? 10 : 8);
    }
    static constexpr size_t smem = sizeof(float) * (6 * pairs + 2 * 2 * kTile * kNS * LN);
};

struct Seg {
    int segs, len;                 // segments of a sequence, tokens in each but the last (a multiple of kTile)
    float *S, *sum;                // [B, segs, C, N] end states, [B, segs, C] sums of d
    int vec, bvec;                 // rows of x, dt, z, y (of Bm, Cm) allow accesses of 4 elements
};

// Tokens [t0, t1) of the block's channels from state h.  FULL: with outputs; else only h and sum of d.
template <typename T, int LN, bool FULL, bool PAD>
__device__ __forceinline__ void walk(const ScanArgs &a, const Seg &sg, const Place &p, int t0, int t1,
                                     const f2 (&A2)[2], f2 (&h)[2], float &sum, float *smem) {
    using K = Cfg<LN>;
    float *s_d = smem;                                                // [2][kTile][width]
    float *s_u = s_d + 2 * K::pairs;                                  // [2][kTile][width]: d x
    float *s_B = s_u + 2 * K::pairs;                                  // [2][kTile][4 LN]
    float *s_C = s_B + 2 * kTile * kNS * LN;
    float *s_y = s_C + 2 * kTile * kNS * LN;                          // [2][kTile][width]
    const int tid = threadIdx.x, nl = lane_states<LN>(), ch = lane_channel<LN>();
    const int n = min(seq_end(a.lengths, p.b, a.T), t1);              // tokens that exist
    const int tiles = n > t0 ? (n - t0 + kTile - 1) / kTile : 0;
    const long long row0 = (long long)p.b * a.T + t0;
    const bool vec = sg.vec, bvec = sg.bvec;
    // a thread's quads are all of the same channels, in rows t_first, t_first + t_step, ...
    constexpr int row = K::width / 4, t_step = kThreads / row, b_step = kThreads / LN;
    static_assert(kThreads % row == 0, "");
    const int c = tid % row * 4, have = p.nc - c, t_first = tid / row;
    const Existing<PAD && FULL> real(nl * kNS, a.N);          // (without sums padded states meet no others)
    const int m = tid % LN * 4, b_have = a.N - m, b_first = tid / LN;
    const long long x0 = (row0 + t_first) * a.C + p.c0 + c, xs = (long long)t_step * a.C;
    const long long b0 = ((row0 + b_first) * a.G + p.g) * a.N + m, bs = (long long)b_step * a.G * a.N;
    f2 bias[2], Dc[2];
    {
        float v[4], w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = a.dt_bias && j < have ? a.dt_bias[p.c0 + c + j] : 0.f;
            w[j] = FULL && a.D && j < have ? a.D[p.c0 + c + j] : 0.f;
        }
        bias[0] = pack2(v[0], v[1]);
        bias[1] = pack2(v[2], v[3]);
        Dc[0] = pack2(w[0], w[1]);
        Dc[1] = pack2(w[2], w[3]);
    }
    // Two tiles are on their way at a time, in two sets of registers that take turns (a tile's work
    // alone is about as long as a loaded memory's latency).
    struct Rows {
        Quad<T> x[K::per], d[K::per], z[K::per], B[K::bper], C[K::bper];
    };
    auto load = [&](int tile, Rows &r) {
        const long long xo = x0 + (long long)tile * kTile * a.C, bo = b0 + (long long)tile * kTile * a.G * a.N;
        const int left = n - t0 - tile * kTile;                       // tokens from the tile's first on
#pragma unroll
        for (int i = 0; i < K::per; ++i)
            if (K::quads % kThreads == 0 || tid + i * kThreads < K::quads) {
                const int live = t_first + i * t_step < left ? have : 0;
                r.x[i].load((const T *)a.x + xo + i * xs, live, vec);
                r.d[i].load((const T *)a.dt_in + xo + i * xs, live, vec);
                if (FULL && a.z) r.z[i].load((const T *)a.z + xo + i * xs, live, vec);
            }
#pragma unroll
        for (int i = 0; i < K::bper; ++i)
            if (K::bquads % kThreads == 0 || tid + i * kThreads < K::bquads) {
                const int live = b_first + i * b_step < left ? b_have : 0;
                r.B[i].load((const T *)a.Bm + bo + i * bs, live, bvec);
                if (FULL) r.C[i].load((const T *)a.Cm + bo + i * bs, live, bvec);
            }
    };
    auto stage = [&](int tile, const Rows &r) {
        const int buf = tile & 1, left = n - t0 - tile * kTile;
#pragma unroll
        for (int i = 0; i < K::per; ++i)
            if (K::quads % kThreads == 0 || tid + i * kThreads < K::quads) {
                f2 d[2], x[2];
                r.d[i].values(d);
                r.x[i].values(x);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    d[j] = add2(d[j], bias[j]);
                    if (a.softplus) d[j] = softplus2(d[j]);
                    if (t_first + i * t_step >= left) d[j] = 0;       // behind the end: the state stays
                }
                const int at = buf * K::quads + tid + i * kThreads;
                reinterpret_cast<ulonglong2 *>(s_d)[at] = make_ulonglong2(d[0], d[1]);
                reinterpret_cast<ulonglong2 *>(s_u)[at] = make_ulonglong2(mul2(d[0], x[0]), mul2(d[1], x[1]));
            }
#pragma unroll
        for (int i = 0; i < K::bper; ++i)
            if (K::bquads % kThreads == 0 || tid + i * kThreads < K::bquads) {
                f2 v[2];
                const int at = buf * K::bquads + tid + i * kThreads;
                r.B[i].values(v);
                reinterpret_cast<ulonglong2 *>(s_B)[at] = make_ulonglong2(v[0], v[1]);
                if (FULL) {
                    r.C[i].values(v);
                    reinterpret_cast<ulonglong2 *>(s_C)[at] = make_ulonglong2(v[0], v[1]);
                }
            }
    };
    // `mine` holds this tile's rows and takes those of the one after next, `next` holds the next one's
    auto work = [&](int tile, Rows &mine, Rows &next) {
        const int buf = tile & 1;
        Quad<T> kx[K::per], kz[K::per];                       // for this tile's outputs
#pragma unroll
        for (int i = 0; i < K::per; ++i) {
            kx[i] = mine.x[i];
            kz[i] = mine.z[i];
        }
        if (tile + 2 < tiles) load(tile + 2, mine);
        const float *pd = s_d + buf * K::pairs + ch, *pu = s_u + buf * K::pairs + ch;
        const ulonglong2 *pB = reinterpret_cast<const ulonglong2 *>(s_B) + buf * K::bquads + nl;
        const ulonglong2 *pC = reinterpret_cast<const ulonglong2 *>(s_C) + buf * K::bquads + nl;
        // the sums stay in registers until the tile is done: a store to shared memory in between would
        // keep the next tokens' loads from moving up
        float ys[kTile / 4][4];
#pragma unroll
        for (int q = 0; q < kTile; q += 4) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float d1 = pd[(q + j) * K::width];
                const f2 d = both(d1), u = both(pu[(q + j) * K::width]);
                const ulonglong2 B = pB[(q + j) * LN];
                h[0] = real(fma2(decay2(d, A2[0]), h[0], mul2(u, B.x)), 0);
                h[1] = real(fma2(decay2(d, A2[1]), h[1], mul2(u, B.y)), 1);
                if (FULL) {
                    const ulonglong2 C = pC[(q + j) * LN];
                    float y0, y1;
                    unpack2(fma2(C.x, h[0], mul2(C.y, h[1])), y0, y1);
                    ys[q / 4][j] = y0 + y1;
                } else {
                    sum += d1;
                }
            }
            if (FULL) reduce4<LN>(ys[q / 4], nl);
        }
        if (FULL && (LN <= 4 || nl < 4)) {
            float *sy = s_y + buf * K::pairs + ch + first_token<LN>(nl) * K::width;
#pragma unroll
            for (int q = 0; q < kTile; q += 4)
#pragma unroll
                for (int j = 0; j < Kept<LN>::value; ++j) sy[(q + j) * K::width] = ys[q / 4][j];
        }
        if (tile + 1 < tiles) stage(tile + 1, next);
        __syncthreads();
        if (FULL) {
            const int left = n - t0 - tile * kTile, rows = t1 - t0 - tile * kTile;
            T *y = (T *)a.y + x0 + (long long)tile * kTile * a.C;
#pragma unroll
            for (int i = 0; i < K::per; ++i) {
                if ((K::quads % kThreads == 0 || tid + i * kThreads < K::quads) && t_first + i * t_step < rows) {
                    const ulonglong2 y2 = reinterpret_cast<const ulonglong2 *>(s_y + buf * K::pairs)[tid + i * kThreads];
                    f2 o[2] = {y2.x, y2.y}, x[2], z[2];
                    float v[4];
                    kx[i].values(x);
                    kz[i].values(z);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (a.D) o[j] = fma2(Dc[j], x[j], o[j]);
                        if (a.z) o[j] = mul2(o[j], mul2(z[j], sigmoid2(z[j])));
                        if (t_first + i * t_step >= left) o[j] = 0;
                        unpack2(o[j], v[2 * j], v[2 * j + 1]);
                    }
                    store4(y + i * xs, v, have, vec);
                }
            }
        }
    };
    Rows even, odd;
    if (tiles > 0) {
        load(0, even);
        if (tiles > 1) load(1, odd);
        stage(0, even);
    }
    __syncthreads();
    for (int tile = 0; tile < tiles; tile += 2) {
        work(tile, even, odd);
        if (tile + 1 < tiles) work(tile + 1, odd, even);
    }
    if (FULL)
        for (long long e = (long long)tiles * K::pairs + tid; e < (long long)(t1 - t0) * K::width; e += kThreads) {
            const int t = (int)(e / K::width), cc = (int)(e % K::width);
            if (cc < p.nc) ((T *)a.y)[(row0 + t) * a.C + p.c0 + cc] = from_f<T>(0.f);
        }
}

// PAD: N does not fill its lanes (see Existing).  Against padded states left to themselves, at B8 T2048 C1024 and
// N = 1, 6, 12, 30, 50: bf16 171, 179, 186, 453, 1321 us instead of 179, 167, 205, 445, 1280; f32 169, 214, 188, 335,
// 952 instead of 173, 192, 191, 311, 846.
// PASS 0: whole sequences.  PASS 1: segment 0 in full, segments 1 .. segs - 2 for (S, sum).
// PASS 2: segments 1 .. segs - 1 in full.
template <typename T, int LN, int PASS, bool PAD>
__global__ void __launch_bounds__(kThreads, PAD ? Cfg<LN>::template fit<T>() : 0)
scan_fwd_kernel(ScanArgs a, Seg sg, int tiles) {
    using K = Cfg<LN>;
    extern __shared__ float4 smem4[];
    float *smem = reinterpret_cast<float *>(smem4);
    Place p = place(blockIdx.x, a.G, a.C / a.G, tiles, PASS == 0 ? 1 : sg.segs - 1, K::width);
    if (PASS == 2) p.seg += 1;
    const int nl = lane_states<LN>(), ch = lane_channel<LN>(), n0 = nl * kNS;
    const bool live = ch < p.nc;
    const long long c = p.c0 + ch;
    float A4[kNS] = {}, h4[kNS] = {};
    if (PASS == 2) wait_for_stream();
    if (live) {
        load_states(a.A + c * a.N, n0, a.N, A4);
#pragma unroll
        for (int k = 0; k < kNS; ++k) A4[k] *= kLog2e;
    }
    const long long seg0 = ((long long)p.b * sg.segs) * a.C + c, seg_c = (long long)a.C;
    if (live) {
        if (PASS == 2) {
            // the state before this segment: segment 0's end, through the segments in between
            load_states(sg.S + seg0 * a.N, n0, a.N, h4);
#pragma unroll 4
            for (int s = 1; s < p.seg; ++s) {
                float S[kNS];
                load_states(sg.S + (seg0 + s * seg_c) * a.N, n0, a.N, S);
                const float d = sg.sum[seg0 + s * seg_c];
#pragma unroll
                for (int k = 0; k < kNS; ++k) h4[k] = fmaf(ex2(d * A4[k]), h4[k], S[k]);
            }
        } else if (p.seg == 0 && a.state_in) {
            load_states(a.state_in + ((long long)p.b * a.C + c) * a.N, n0, a.N, h4);
        }
    }
    const int t0 = PASS == 0 ? 0 : p.seg * sg.len, t1 = PASS == 0 ? a.T : min(a.T, t0 + sg.len);
    float sum = 0.f;
    const f2 A2[2] = {pack2(A4[0], A4[1]), pack2(A4[2], A4[3])};
    f2 h[2] = {pack2(h4[0], h4[1]), pack2(h4[2], h4[3])};
    if (PASS != 1 || p.seg == 0)
        walk<T, LN, true, PAD>(a, sg, p, t0, t1, A2, h, sum, smem);
    else
        walk<T, LN, false, PAD>(a, sg, p, t0, t1, A2, h, sum, smem);
    if (!live) return;
    unpack2(h[0], h4[0], h4[1]);
    unpack2(h[1], h4[2], h4[3]);
    if (PASS == 1) {
        store_states(sg.S + (seg0 + p.seg * seg_c) * a.N, n0, a.N, h4);
        if (nl == 0) sg.sum[seg0 + p.seg * seg_c] = sum;
    } else if (a.state_out && (PASS == 0 || p.seg == sg.segs - 1)) {
        store_states(a.state_out + ((long long)p.b * a.C + c) * a.N, n0, a.N, h4);
    }
}

constexpr int kStepThreads = 128;

// One token of four batch entries for every thread: the lanes of a channel as in the walk, so a warp's
// states are one run of memory.  All loads are under way before the first is used.  Each of four lanes
// forms the step of one entry and hands it to the others; the sums over n come back to it the same way.
// Bound by the fp32 state, read and written once; the rates are read once for the four entries.
template <typename T, int LN>
__global__ void __launch_bounds__(kStepThreads)
scan_step_kernel(ScanArgs a, int vec, int bvec) {
    constexpr int S = 32 / LN, own = Kept<LN>::value;
    const int lane = threadIdx.x & 31, nl = lane_states<LN>(), n0 = nl * kNS, r0 = first_token<LN>(nl);
    const int c = blockIdx.x * (kStepThreads / LN) + lane_channel<LN>(), b0 = blockIdx.y * 4;
    const Existing<true> real(n0, a.N);
    const bool live = c < a.C;
    const int rows = live ? min(4, a.B - b0) : 0;
    const int g = a.G == 1 || !live ? 0 : c / (a.C / a.G);
    const long long bc = (long long)b0 * a.C + c, bg = ((long long)b0 * a.G + g) * a.N + n0;
    float4 h[4];
    Quad<T> Bq[4], Cq[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const float *p = a.state_in + (bc + (long long)r * a.C) * a.N;
        h[r] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows) {
            if (vec) {
                if (n0 < a.N) h[r] = *reinterpret_cast<const float4 *>(p + n0);
            } else {
                float v[kNS];
                load_states(p, n0, a.N, v);
                h[r] = make_float4(v[0], v[1], v[2], v[3]);
            }
        }
        const int have = r < rows ? a.N - n0 : 0;
        Bq[r].load((const T *)a.Bm + bg + (long long)r * a.G * a.N, have, bvec);
        Cq[r].load((const T *)a.Cm + bg + (long long)r * a.G * a.N, have, bvec);
    }
    float A[kNS] = {}, d_own[own], u_own[own], x_own[own], z_own[own];
    if (live) load_states(a.A + (long long)c * a.N, n0, a.N, A);
    const float bias = live && a.dt_bias ? a.dt_bias[c] : 0.f, D = live && a.D ? a.D[c] : 0.f;
#pragma unroll
    for (int j = 0; j < own; ++j) {
        const long long at = bc + (long long)(r0 + j) * a.C;
        float d = 0.f;
        x_own[j] = z_own[j] = 0.f;
        if (r0 + j < rows) {
            x_own[j] = to_f(((const T *)a.x)[at]);
            d = to_f(((const T *)a.dt_in)[at]) + bias;
            if (a.z) z_own[j] = to_f(((const T *)a.z)[at]);
        }
        if (a.softplus) d = softplus_f(d);
        d_own[j] = d;
        u_own[j] = d * x_own[j];
    }
    const f2 A2[2] = {mul2(pack2(A[0], A[1]), both(kLog2e)), mul2(pack2(A[2], A[3]), both(kLog2e))};
    float sum[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        // the lane that formed this entry's step
        const int from = (LN == 1 ? 0 : LN == 2 ? r >> 1 : (r >> 1) | (r & 1) << 1) * S + lane % S;
        const float d = __shfl_sync(0xffffffffu, d_own[r % own], from), u = __shfl_sync(0xffffffffu, u_own[r % own], from);
        f2 B[2], C[2], s[2] = {pack2(h[r].x, h[r].y), pack2(h[r].z, h[r].w)};
        Bq[r].values(B);
        Cq[r].values(C);
#pragma unroll
        for (int k = 0; k < 2; ++k) s[k] = real(fma2(decay2(both(d), A2[k]), s[k], mul2(both(u), B[k])), k);
        float y0, y1;
        unpack2(fma2(C[0], s[0], mul2(C[1], s[1])), y0, y1);
        sum[r] = y0 + y1;
        unpack2(s[0], h[r].x, h[r].y);
        unpack2(s[1], h[r].z, h[r].w);
        float *p = a.state_out + (bc + (long long)r * a.C) * a.N;
        if (r < rows) {
            if (vec) {
                if (n0 < a.N) *reinterpret_cast<float4 *>(p + n0) = h[r];
            } else {
                const float v[kNS] = {h[r].x, h[r].y, h[r].z, h[r].w};
                store_states(p, n0, a.N, v);
            }
        }
    }
    reduce4<LN>(sum, nl);
    if (LN <= 4 || nl < 4)
#pragma unroll
        for (int j = 0; j < own; ++j)
            if (r0 + j < rows) {
                float y = sum[j];
                if (a.D) y = fmaf(D, x_own[j], y);
                if (a.z) y *= z_own[j] * sigmoid_f(z_own[j]);
                ((T *)a.y)[bc + (long long)(r0 + j) * a.C] = from_f<T>(y);
            }
}

// Segments of the forward, from the sizes alone: one where the (batch, channel) blocks are at least
// four an SM; else enough for about eight an SM, each of at least 32 tokens.  Both passes run all
// segments but one at once; fewer than 4 segments are not taken, although 2 or 3 gain something at 395 to
// 591 blocks (T4096 N16 bf16, one segment against them: B1 C6400 389 and 302 us, B1 C7168 391 and 347, B2 C4096
// 393 and 357, B1 C9216 393 and 362; fewer blocks take 4 or more).
void fwd_segments(int B, int T, int C, int G, int N, int *segs, int *len) {
    const int width = kThreads / lanes_for(N);
    const long long blocks = (long long)B * G * ((C / G + width - 1) / width);
    long long want = blocks >= 4 * 148 ? 1 : (8 * 148 + blocks - 1) / blocks;
    if (want > T / 32) want = T / 32;
    if (want < 4) {
        *segs = 1;
        *len = T;
        return;
    }
    *len = (int)(((T + want - 1) / want + kTile - 1) / kTile * kTile);
    *segs = (T + *len - 1) / *len;
}

template <typename T, int LN, bool PAD>
la_status fwd_pad(const ScanArgs &a, cudaStream_t st) {
    using K = Cfg<LN>;
    Seg sg;
    fwd_segments(a.B, a.T, a.C, a.G, a.N, &sg.segs, &sg.len);
    sg.S = (float *)a.ws;
    sg.sum = sg.S + (size_t)a.B * sg.segs * a.C * a.N;
    sg.vec = quad_rows<T>(a.C / a.G, a.x, a.dt_in, a.z, a.y);
    sg.bvec = quad_rows<T>(a.N, a.Bm, a.Cm);
    const int tiles = (a.C / a.G + K::width - 1) / K::width;
    const unsigned blocks = (unsigned)((long long)a.B * a.G * tiles);
    if (sg.segs == 1)
        return launch("selective_scan_fwd", scan_fwd_kernel<T, LN, 0, PAD>, dim3(blocks), dim3(kThreads), K::smem, st,
                      a, sg, tiles);
    const dim3 grid(blocks * (sg.segs - 1));
    la_status rc = launch("selective_scan_fwd_ends", scan_fwd_kernel<T, LN, 1, PAD>, grid, dim3(kThreads), K::smem, st,
                          a, sg, tiles);
    if (rc != LA_OK) return rc;
    return launch_pdl("selective_scan_fwd", scan_fwd_kernel<T, LN, 2, PAD>, grid, dim3(kThreads), K::smem, st, a, sg,
                      tiles);
}

template <typename T, int LN>
la_status fwd_ln(const ScanArgs &a, cudaStream_t st) {
    return a.N == kNS * LN ? fwd_pad<T, LN, false>(a, st) : fwd_pad<T, LN, true>(a, st);
}

template <typename T>
la_status fwd_t(const ScanArgs &a, cudaStream_t st) {
    switch (lanes_for(a.N)) {
    case 1: return fwd_ln<T, 1>(a, st);
    case 2: return fwd_ln<T, 2>(a, st);
    case 4: return fwd_ln<T, 4>(a, st);
    case 8: return fwd_ln<T, 8>(a, st);
    default: return fwd_ln<T, 16>(a, st);
    }
}

template <typename T, int LN>
la_status step_ln(const ScanArgs &a, cudaStream_t st) {
    constexpr int width = kStepThreads / LN;
    const dim3 grid((unsigned)((a.C + width - 1) / width), (unsigned)((a.B + 3) / 4));
    return launch("selective_scan_step", scan_step_kernel<T, LN>, grid, dim3(kStepThreads), 0, st, a,
                  quad_rows<float>(a.N, a.state_in, a.state_out), quad_rows<T>(a.N, a.Bm, a.Cm));
}

template <typename T>
la_status step_t(const ScanArgs &a, cudaStream_t st) {
    switch (lanes_for(a.N)) {
    case 1: return step_ln<T, 1>(a, st);
    case 2: return step_ln<T, 2>(a, st);
    case 4: return step_ln<T, 4>(a, st);
    case 8: return step_ln<T, 8>(a, st);
    default: return step_ln<T, 16>(a, st);
    }
}

}  // namespace

size_t scan_fwd_workspace(int B, int T, int C, int G, int N) {
    int segs, len;
    fwd_segments(B, T, C, G, N, &segs, &len);
    return segs == 1 ? 0 : up256((size_t)B * segs * C * (N + 1) * sizeof(float));
}

la_status scan_fwd(const ScanArgs &a, cudaStream_t st) {
    switch (a.dt) {
    case LA_F32: return fwd_t<float>(a, st);
    case LA_F16: return fwd_t<__half>(a, st);
    default: return fwd_t<__nv_bfloat16>(a, st);
    }
}

la_status scan_step(const ScanArgs &a, cudaStream_t st) {
    switch (a.dt) {
    case LA_F32: return step_t<float>(a, st);
    case LA_F16: return step_t<__half>(a, st);
    default: return step_t<__nv_bfloat16>(a, st);
    }
}

}  // namespace la

// la_scan.cu -- selective state space scan, forward: whole sequences and single tokens.
//
//   h_t[n] = exp(d_t A[n]) h_{t-1}[n] + d_t x_t B_t[n],   y_t = (sum_n C_t[n] h_t[n] + D x_t) silu(z_t)
// per channel, with d_t = softplus(dt_t + bias).
//
// What bounds it: one exponential for every (token, channel, state).  At N = 16 a channel's token
// moves 8 bytes of x, dt, z and y and costs 16 exponentials; an SM makes 16 a cycle in its
// special-function units, so they take 3 times as long as the traffic.
//
// A block owns 128 / LN channels of one batch entry and walks over its tokens in tiles of 16.  The
// tile's x, dt, z, B and C come in by coalesced loads a tile ahead (in registers while the previous
// tile is worked on), each d_t, d_t x_t is formed once and left in shared memory for the LN lanes
// that share it; states live in registers.  Every fourth token the lanes of a channel exchange
// halves of their four partial sums, so a sum over n costs 3 shuffles for 4 tokens.
//
// Where the batch and channels alone give too few blocks, the sequence is cut into segments: the
// first launch runs segment 0 in full and the others for their end state from zero and their sum
// of d (a segment's decay is exp(A sum d), so no product is kept); the second starts every later
// segment from the states before it, joined in order.
#include "la_scan.cuh"

namespace la {
namespace {

using namespace scan;

constexpr int kThreads = 128;

template <int LN> struct Cfg {
    static constexpr int width = kThreads / LN;             // channels a block
    static constexpr int NP = kNS * LN;                     // padded states
    static constexpr int per = kTile * width / kThreads;    // (token, channel) pairs a thread stages
    static constexpr int bc_per = (kTile * NP + kThreads - 1) / kThreads;
    static constexpr size_t smem = sizeof(float) * (2 * kTile * width * 2 + 2 * 2 * kTile * NP + 2 * kTile * width);
};

struct Seg {
    int segs, len;                 // segments of a sequence, tokens in each but the last (a multiple of kTile)
    float *S, *sum;                // [B, segs, C, N] end states, [B, segs, C] sums of d
};

// Tokens [t0, t1) of the block's channels from state h.  FULL: with outputs; else only h and sum of d.
template <typename T, int LN, bool FULL>
__device__ __forceinline__ void walk(const ScanArgs &a, const Place &p, int t0, int t1, const float (&A2)[kNS],
                                     float (&h)[kNS], float &sum, float *smem) {
    using K = Cfg<LN>;
    float2 *s_in = reinterpret_cast<float2 *>(smem);                  // [2][kTile][width]
    float *s_B = smem + 2 * kTile * K::width * 2;                     // [2][kTile][NP]
    float *s_C = s_B + 2 * kTile * K::NP;
    float *s_y = s_C + 2 * kTile * K::NP;                             // [2][kTile][width]
    const int tid = threadIdx.x, nl = tid % LN, ch = tid / LN;
    const int n = min(seq_end(a.lengths, p.b, a.T), t1);              // tokens that exist
    const int tiles = n > t0 ? (n - t0 + kTile - 1) / kTile : 0;
    const long long row0 = (long long)p.b * a.T;
    const T *x = (const T *)a.x, *dt = (const T *)a.dt_in, *z = (const T *)a.z;
    const T *Bm = (const T *)a.Bm, *Cm = (const T *)a.Cm;

    T rx[K::per], rd[K::per], rz[K::per], rB[K::bc_per], rC[K::bc_per];
    auto load = [&](int tile) {
        const int tb = t0 + tile * kTile;
#pragma unroll
        for (int i = 0; i < K::per; ++i) {
            const int e = tid + i * kThreads, t = tb + e / K::width, c = e % K::width;
            rx[i] = rd[i] = rz[i] = from_f<T>(0.f);
            if (t < n && c < p.nc) {
                const long long o = (row0 + t) * a.C + p.c0 + c;
                rx[i] = x[o];
                rd[i] = dt[o];
                if (FULL && z) rz[i] = z[o];
            }
        }
#pragma unroll
        for (int i = 0; i < K::bc_per; ++i) {
            const int e = tid + i * kThreads, t = tb + e / K::NP, m = e % K::NP;
            rB[i] = rC[i] = from_f<T>(0.f);
            if (e < kTile * K::NP && t < n && m < a.N) {
                const long long o = ((row0 + t) * a.G + p.g) * a.N + m;
                rB[i] = Bm[o];
                if (FULL) rC[i] = Cm[o];
            }
        }
    };
    float skip[K::per], gate[K::per], skip2[K::per], gate2[K::per];   // of the tile at work, of the next
    auto stage = [&](int tile) {
        const int buf = tile & 1, tb = t0 + tile * kTile;
#pragma unroll
        for (int i = 0; i < K::per; ++i) {
            const int e = tid + i * kThreads, t = tb + e / K::width, c = e % K::width;
            float2 in = make_float2(0.f, 0.f);
            skip2[i] = 0.f;
            gate2[i] = 1.f;
            if (t < n && c < p.nc) {
                const float xv = to_f(rx[i]);
                float d = to_f(rd[i]) + (a.dt_bias ? a.dt_bias[p.c0 + c] : 0.f);
                if (a.softplus) d = softplus_f(d);
                in = make_float2(d, d * xv);
                if (FULL) {
                    if (a.D) skip2[i] = a.D[p.c0 + c] * xv;
                    if (z) {
                        const float zv = to_f(rz[i]);
                        gate2[i] = zv * sigmoid_f(zv);
                    }
                }
            }
            s_in[buf * kTile * K::width + e] = in;
        }
#pragma unroll
        for (int i = 0; i < K::bc_per; ++i) {
            const int e = tid + i * kThreads;
            if (e < kTile * K::NP) {
                s_B[buf * kTile * K::NP + e] = to_f(rB[i]);
                if (FULL) s_C[buf * kTile * K::NP + e] = to_f(rC[i]);
            }
        }
    };
    if (tiles > 0) {
        load(0);
        stage(0);
    }
    for (int tile = 0; tile < tiles; ++tile) {
        __syncthreads();
        const int buf = tile & 1;
#pragma unroll
        for (int i = 0; i < K::per; ++i) {
            skip[i] = skip2[i];
            gate[i] = gate2[i];
        }
        if (tile + 1 < tiles) load(tile + 1);
        const float2 *in = s_in + buf * kTile * K::width + ch;
        const float *sB = s_B + buf * kTile * K::NP + nl * kNS, *sC = s_C + buf * kTile * K::NP + nl * kNS;
        float *sy = s_y + buf * kTile * K::width + ch;
#pragma unroll
        for (int q = 0; q < kTile; q += 4) {
            float ys[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 v = in[(q + j) * K::width];
                const float4 Bv = *reinterpret_cast<const float4 *>(sB + (q + j) * K::NP);
                const float Bk[4] = {Bv.x, Bv.y, Bv.z, Bv.w};
                if (!FULL) sum += v.x;
#pragma unroll
                for (int k = 0; k < kNS; ++k) h[k] = fmaf(ex2(v.x * A2[k]), h[k], v.y * Bk[k]);
                if (FULL) {
                    const float4 Cv = *reinterpret_cast<const float4 *>(sC + (q + j) * K::NP);
                    ys[j] = fmaf(Cv.x, h[0], fmaf(Cv.y, h[1], fmaf(Cv.z, h[2], Cv.w * h[3])));
                }
            }
            if (FULL) {
                reduce4<LN>(ys, nl);
                if (LN <= 4 || nl < 4) {
#pragma unroll
                    for (int j = 0; j < Kept<LN>::value; ++j) sy[(q + first_token<LN>(nl) + j) * K::width] = ys[j];
                }
            }
        }
        if (tile + 1 < tiles) stage(tile + 1);
        if (FULL) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < K::per; ++i) {
                const int e = tid + i * kThreads, t = t0 + tile * kTile + e / K::width, c = e % K::width;
                if (t < t1 && c < p.nc)
                    ((T *)a.y)[(row0 + t) * a.C + p.c0 + c] =
                        from_f<T>(t < n ? (s_y[buf * kTile * K::width + e] + skip[i]) * gate[i] : 0.f);
            }
        }
    }
    if (FULL)
        for (long long e = (long long)tiles * kTile * K::width + tid; e < (long long)(t1 - t0) * K::width; e += kThreads) {
            const int t = t0 + (int)(e / K::width), c = (int)(e % K::width);
            if (c < p.nc) ((T *)a.y)[(row0 + t) * a.C + p.c0 + c] = from_f<T>(0.f);
        }
}

// PASS 0: whole sequences.  PASS 1: segment 0 in full, segments 1 .. segs - 2 for (S, sum).
// PASS 2: segments 1 .. segs - 1 in full.
template <typename T, int LN, int PASS>
__global__ void __launch_bounds__(kThreads)
scan_fwd_kernel(ScanArgs a, Seg sg, int tiles) {
    using K = Cfg<LN>;
    extern __shared__ float4 smem4[];
    float *smem = reinterpret_cast<float *>(smem4);
    Place p = place(blockIdx.x, a.G, a.C / a.G, tiles, PASS == 0 ? 1 : sg.segs - 1, K::width);
    if (PASS == 2) p.seg += 1;
    const int nl = threadIdx.x % LN, ch = threadIdx.x / LN, n0 = nl * kNS;
    const bool live = ch < p.nc;
    const long long c = p.c0 + ch;
    float A2[kNS] = {}, h[kNS] = {};
    if (live) {
        load_states(a.A + c * a.N, n0, a.N, A2);
#pragma unroll
        for (int k = 0; k < kNS; ++k) A2[k] *= kLog2e;
    }
    const long long seg0 = ((long long)p.b * sg.segs) * a.C + c, seg_c = (long long)a.C;
    if (live) {
        if (PASS == 2) {
            // the state before this segment: segment 0's end, through the segments in between
            load_states(sg.S + seg0 * a.N, n0, a.N, h);
            for (int s = 1; s < p.seg; ++s) {
                float S[kNS];
                load_states(sg.S + (seg0 + s * seg_c) * a.N, n0, a.N, S);
                const float d = sg.sum[seg0 + s * seg_c];
#pragma unroll
                for (int k = 0; k < kNS; ++k) h[k] = fmaf(ex2(d * A2[k]), h[k], S[k]);
            }
        } else if (p.seg == 0 && a.state_in) {
            load_states(a.state_in + ((long long)p.b * a.C + c) * a.N, n0, a.N, h);
        }
    }
    const int t0 = PASS == 0 ? 0 : p.seg * sg.len, t1 = PASS == 0 ? a.T : min(a.T, t0 + sg.len);
    float sum = 0.f;
    if (PASS != 1 || p.seg == 0)
        walk<T, LN, true>(a, p, t0, t1, A2, h, sum, smem);
    else
        walk<T, LN, false>(a, p, t0, t1, A2, h, sum, smem);
    if (!live) return;
    if (PASS == 1) {
        store_states(sg.S + (seg0 + p.seg * seg_c) * a.N, n0, a.N, h);
        if (nl == 0) sg.sum[seg0 + p.seg * seg_c] = sum;
    } else if (a.state_out && (PASS == 0 || p.seg == sg.segs - 1)) {
        store_states(a.state_out + ((long long)p.b * a.C + c) * a.N, n0, a.N, h);
    }
}

// One token: LN lanes a channel; bound by the fp32 state, read and written once.
template <typename T, int LN>
__global__ void __launch_bounds__(kThreads)
scan_step_kernel(ScanArgs a) {
    const long long idx = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long bc = idx / LN;
    const int nl = (int)(idx % LN), n0 = nl * kNS;
    const bool live = bc < (long long)a.B * a.C;
    float acc = 0.f, xv = 0.f;
    int c = 0;
    if (live) {
        const int b = (int)(bc / a.C);
        c = (int)(bc - (long long)b * a.C);
        const long long bg = ((long long)b * a.G + c / (a.C / a.G)) * a.N;
        float A[kNS], h[kNS] = {};
        load_states(a.state_in + bc * a.N, n0, a.N, h);
        load_states(a.A + (long long)c * a.N, n0, a.N, A);
        xv = to_f(((const T *)a.x)[bc]);
        float d = to_f(((const T *)a.dt_in)[bc]) + (a.dt_bias ? a.dt_bias[c] : 0.f);
        if (a.softplus) d = softplus_f(d);
#pragma unroll
        for (int k = 0; k < kNS; ++k) {
            float Bk = 0.f, Ck = 0.f;
            if (n0 + k < a.N) {
                Bk = to_f(((const T *)a.Bm)[bg + n0 + k]);
                Ck = to_f(((const T *)a.Cm)[bg + n0 + k]);
            }
            h[k] = fmaf(ex2(d * (A[k] * kLog2e)), h[k], d * xv * Bk);
            acc = fmaf(Ck, h[k], acc);
        }
        store_states(a.state_out + bc * a.N, n0, a.N, h);
    }
#pragma unroll
    for (int m = 1; m < LN; m <<= 1) acc += __shfl_xor_sync(0xffffffffu, acc, m);
    if (live && nl == 0) {
        if (a.D) acc = fmaf(a.D[c], xv, acc);
        if (a.z) {
            const float zv = to_f(((const T *)a.z)[bc]);
            acc *= zv * sigmoid_f(zv);
        }
        ((T *)a.y)[bc] = from_f<T>(acc);
    }
}

// Segments of the forward, from the sizes alone: one where the (batch, channel) blocks are at least
// two an SM; else enough for about four an SM, each of at least 64 tokens.  Both passes run all
// segments but one at once, so fewer than 4 segments gain nothing.
void fwd_segments(int B, int T, int C, int G, int N, int *segs, int *len) {
    const int width = kThreads / lanes_for(N);
    const long long blocks = (long long)B * G * ((C / G + width - 1) / width);
    long long want = blocks >= 2 * 148 ? 1 : (4 * 148 + blocks - 1) / blocks;
    if (want > T / 64) want = T / 64;
    if (want < 4) {
        *segs = 1;
        *len = T;
        return;
    }
    *len = (int)(((T + want - 1) / want + kTile - 1) / kTile * kTile);
    *segs = (T + *len - 1) / *len;
}

template <typename T, int LN>
la_status fwd_ln(const ScanArgs &a, cudaStream_t st) {
    using K = Cfg<LN>;
    Seg sg;
    fwd_segments(a.B, a.T, a.C, a.G, a.N, &sg.segs, &sg.len);
    sg.S = (float *)a.ws;
    sg.sum = sg.S + (size_t)a.B * sg.segs * a.C * a.N;
    const int tiles = (a.C / a.G + K::width - 1) / K::width;
    const unsigned blocks = (unsigned)((long long)a.B * a.G * tiles);
    if (sg.segs == 1)
        return launch("selective_scan_fwd", scan_fwd_kernel<T, LN, 0>, dim3(blocks), dim3(kThreads), K::smem, st, a,
                      sg, tiles);
    const dim3 grid(blocks * (sg.segs - 1));
    la_status rc = launch("selective_scan_fwd_ends", scan_fwd_kernel<T, LN, 1>, grid, dim3(kThreads), K::smem, st, a,
                          sg, tiles);
    if (rc != LA_OK) return rc;
    return launch("selective_scan_fwd", scan_fwd_kernel<T, LN, 2>, grid, dim3(kThreads), K::smem, st, a, sg, tiles);
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
    const long long n = (long long)a.B * a.C * LN;
    return launch("selective_scan_step", scan_step_kernel<T, LN>, dim3((unsigned)((n + kThreads - 1) / kThreads)),
                  dim3(kThreads), 0, st, a);
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

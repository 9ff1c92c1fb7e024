// la_scan_bwd.cu -- gradients of the selective state space scan.
//
// With a_t = exp(d_t A), u_t = d_t x_t, e_t = dy_t silu(z_t) and lam_t the gradient of the state
// after token t,
//   lam_t = e_t C_t + w_{t+1},  w_t = a_t lam_t           (w past the end: the incoming gradient)
//   dC_t = sum_c e_t h_t,   dB_t = sum_c u_t lam_t         (sums over the group's channels)
//   q_t = sum_n lam_t B_t,  p_t = w_t h_{t-1}  (per state)
//   dx_t = d_t q_t + D e_t, dd_t = x_t q_t + sum_n A p_t,  ddt_t = dd_t sigma(dt_t + bias)
//   dA = sum_t d_t p_t,  dD = sum_t e_t x_t,  dbias = sum_t ddt_t
//   dz_t = dy_t silu'(z_t) (sum_n C_t h_t + D x_t).
//
// Nothing is kept from the forward.  A block owns a tile of channels (as in the forward, LN lanes a
// channel) and a segment of the sequence; it walks forwards once, leaving the state before every
// tile of kTile tokens in the workspace, then backwards tile by tile: the tile's states and decays
// are formed again in registers (one exponential each) and used in reverse order.  So a state costs
// two exponentials and about 12 multiply-adds, and 8 / kTile bytes of workspace traffic each way:
// the kernel is bound by instruction issue, not by HBM.  The sums over channels of dB and dC are
// butterflies over the lanes of a warp (each step hands half of the values to the partner), then
// over the block's warps in shared memory, then over the channel tiles in a last launch, always in
// the same order; that launch also joins the batch entries' parts of dA, dD and dbias.
//
// Few channels and a long sequence: segments as in the forward.  A first launch gives every
// segment's end state from zero, S, its sum of d, and the gradient that it hands to the state
// before it, R = sum_t (prod_{s<=t} a_s) e_t C_t, from the same exponentials in one sweep.
#include "la_scan.cuh"

namespace la {
namespace {

using namespace scan;

template <int LN> struct Cfg {
    static constexpr int threads = LN == 1 ? 128 : 256;
    static constexpr int warps = threads / 32;
    static constexpr int width = threads / LN;
    static constexpr int NP = kNS * LN;
    static constexpr int per = kTile * width / threads;
    static constexpr int bc_per = (kTile * NP + threads - 1) / threads;
    // floats of shared memory: per pair (d, u, e, x) and (sigma', dy silu') twice, B and C twice,
    // three sums per pair, the warps' sums of dC and dB
    static constexpr int pairs = kTile * width;
    static constexpr size_t smem =
        sizeof(float) * (2 * pairs * 6 + 2 * 2 * kTile * NP + 3 * pairs + warps * kTile * 2 * NP);
};

struct Seg {
    int segs, len;
    float *S, *R, *sum;            // [B, segs, C, N] twice, [B, segs, C]
    float *ckpt;                   // [B, ceil(T / kTile), C, N]
    float *bc;                     // [tiles][2][B T G N]: the channel tiles' parts of dC and dB
    float *pA, *pD, *pbias;        // [B segs][C N], [B segs][C] twice
};

template <int LN>
struct Smem {
    using K = Cfg<LN>;
    float4 *in;                    // [2][kTile][width]: d, u, e, x
    float2 *ex;                    // [2][kTile][width]: sigma(dt + bias) (1 without softplus), dy silu'(z)
    float *B, *C;                  // [2][kTile][NP]
    float *o;                      // [3][kTile][width]: sum_n C h, q, sum_n A p (in units of 1 / log2 e)
    float *red;                    // [warps][kTile][2][NP]
    __device__ explicit Smem(float *p) {
        in = reinterpret_cast<float4 *>(p);
        ex = reinterpret_cast<float2 *>(p + 2 * K::pairs * 4);
        B = p + 2 * K::pairs * 6;
        C = B + 2 * kTile * K::NP;
        o = C + 2 * kTile * K::NP;
        red = o + 3 * K::pairs;
    }
};

// Stages tiles of kTile tokens: load() fetches one into registers, store() converts it into shared
// memory.  BACK: with dy, z and C; else x, dt and B only.
template <typename T, int LN, bool BACK>
struct Stager {
    using K = Cfg<LN>;
    T rx[K::per], rd[K::per], rz[K::per], rg[K::per], rB[K::bc_per], rC[K::bc_per];
    __device__ __forceinline__ void load(const ScanArgs &a, const Place &p, int tb, int n) {
        const int tid = threadIdx.x;
        const long long row0 = (long long)p.b * a.T;
#pragma unroll
        for (int i = 0; i < K::per; ++i) {
            const int e = tid + i * K::threads, t = tb + e / K::width, c = e % K::width;
            rx[i] = rd[i] = rz[i] = rg[i] = from_f<T>(0.f);
            if (t < n && c < p.nc) {
                const long long o = (row0 + t) * a.C + p.c0 + c;
                rx[i] = ((const T *)a.x)[o];
                rd[i] = ((const T *)a.dt_in)[o];
                if (BACK) {
                    rg[i] = ((const T *)a.dy)[o];
                    if (a.z) rz[i] = ((const T *)a.z)[o];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < K::bc_per; ++i) {
            const int e = tid + i * K::threads, t = tb + e / K::NP, m = e % K::NP;
            rB[i] = rC[i] = from_f<T>(0.f);
            if (e < kTile * K::NP && t < n && m < a.N) {
                const long long o = ((row0 + t) * a.G + p.g) * a.N + m;
                rB[i] = ((const T *)a.Bm)[o];
                if (BACK) rC[i] = ((const T *)a.Cm)[o];
            }
        }
    }
    __device__ __forceinline__ void store(const ScanArgs &a, const Place &p, int tb, int n, Smem<LN> &s, int buf) {
        const int tid = threadIdx.x;
#pragma unroll
        for (int i = 0; i < K::per; ++i) {
            const int e = tid + i * K::threads, t = tb + e / K::width, c = e % K::width;
            float4 in = make_float4(0.f, 0.f, 0.f, 0.f);
            float2 ex = make_float2(1.f, 0.f);
            if (t < n && c < p.nc) {
                const float x = to_f(rx[i]);
                float d = to_f(rd[i]) + (a.dt_bias ? a.dt_bias[p.c0 + c] : 0.f);
                if (a.softplus) {
                    if (BACK) ex.x = sigmoid_f(d);
                    d = softplus_f(d);
                }
                in = make_float4(d, d * x, 0.f, x);
                if (BACK) {
                    in.z = to_f(rg[i]);
                    if (a.z) {
                        const float z = to_f(rz[i]), sg = sigmoid_f(z);
                        ex.y = in.z * sg * fmaf(z, 1.f - sg, 1.f);
                        in.z *= z * sg;
                    }
                }
            }
            s.in[buf * K::pairs + e] = in;
            if (BACK) s.ex[buf * K::pairs + e] = ex;
        }
#pragma unroll
        for (int i = 0; i < K::bc_per; ++i) {
            const int e = tid + i * K::threads;
            if (e < kTile * K::NP) {
                s.B[buf * kTile * K::NP + e] = to_f(rB[i]);
                if (BACK) s.C[buf * kTile * K::NP + e] = to_f(rC[i]);
            }
        }
    }
};

// Sums v[0..7] over the 32 / LN channels of a warp (lanes of equal nl) and leaves each sum in `out`
// at [quantity][state], quantity 0 from v[0..3] and 1 from v[4..7].
template <int LN>
__device__ __forceinline__ void reduce_channels(float (&v)[8], int lane, int nl, float *out) {
    constexpr int NP = kNS * LN;
    int base = 0;
    {
        const bool hi = lane & LN;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float s = hi ? v[i] : v[i + 4];
            v[i] = (hi ? v[i + 4] : v[i]) + __shfl_xor_sync(0xffffffffu, s, LN);
        }
        base = hi ? NP : 0;
    }
    if (LN <= 8) {
        const bool hi = lane & (2 * LN);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float s = hi ? v[i] : v[i + 2];
            v[i] = (hi ? v[i + 2] : v[i]) + __shfl_xor_sync(0xffffffffu, s, 2 * LN);
        }
        base += hi ? 2 : 0;
    }
    if (LN <= 4) {
        const bool hi = lane & (4 * LN);
        const float s = hi ? v[0] : v[1];
        v[0] = (hi ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, s, 4 * LN);
        base += hi ? 1 : 0;
    }
    if (LN <= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 8 * LN);
    if (LN <= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 16 * LN);
    constexpr int kept = LN >= 16 ? 4 : LN == 8 ? 2 : 1;
    if (LN <= 2 && lane >= 8 * LN) return;
#pragma unroll
    for (int i = 0; i < kept; ++i) out[base + nl * kNS + i] = v[i];
}

// First launch of the segmented form: (S, R, sum of d) of every segment.
template <typename T, int LN>
__global__ void __launch_bounds__(Cfg<LN>::threads)
scan_bwd_ends(ScanArgs a, Seg sg, int tiles) {
    using K = Cfg<LN>;
    extern __shared__ float4 smem4[];
    Smem<LN> s(reinterpret_cast<float *>(smem4));
    const Place p = place(blockIdx.x, a.G, a.C / a.G, tiles, sg.segs, K::width);
    const int nl = threadIdx.x % LN, ch = threadIdx.x / LN, n0 = nl * kNS;
    const bool live = ch < p.nc;
    const long long c = p.c0 + ch;
    float A2[kNS] = {}, h[kNS] = {}, P[kNS], R[kNS] = {}, sum = 0.f;
    if (live) load_states(a.A + c * a.N, n0, a.N, A2);
#pragma unroll
    for (int k = 0; k < kNS; ++k) {
        A2[k] *= kLog2e;
        P[k] = 1.f;
    }
    const int t0 = p.seg * sg.len, n = min(seq_end(a.lengths, p.b, a.T), min(a.T, t0 + sg.len));
    const int count = n > t0 ? (n - t0 + kTile - 1) / kTile : 0;
    Stager<T, LN, true> stg;
    if (count > 0) {
        stg.load(a, p, t0, n);
        stg.store(a, p, t0, n, s, 0);
    }
    for (int tile = 0; tile < count; ++tile) {
        __syncthreads();
        const int buf = tile & 1;
        if (tile + 1 < count) stg.load(a, p, t0 + (tile + 1) * kTile, n);
        const float4 *in = s.in + buf * K::pairs + ch;
        const float *sB = s.B + buf * kTile * K::NP + n0, *sC = s.C + buf * kTile * K::NP + n0;
#pragma unroll 4
        for (int j = 0; j < kTile; ++j) {
            const float4 v = in[j * K::width];
            sum += v.x;
#pragma unroll
            for (int k = 0; k < kNS; ++k) {
                const float e = ex2(v.x * A2[k]);
                h[k] = fmaf(e, h[k], v.y * sB[j * K::NP + k]);
                P[k] *= e;
                R[k] = fmaf(P[k], v.z * sC[j * K::NP + k], R[k]);
            }
        }
        if (tile + 1 < count) stg.store(a, p, t0 + (tile + 1) * kTile, n, s, buf ^ 1);
    }
    if (!live) return;
    const long long at = ((long long)p.b * sg.segs + p.seg) * a.C + c;
    store_states(sg.S + at * a.N, n0, a.N, h);
    store_states(sg.R + at * a.N, n0, a.N, R);
    if (nl == 0) sg.sum[at] = sum;
}

template <typename T, int LN>
__global__ void __launch_bounds__(Cfg<LN>::threads)
scan_bwd_kernel(ScanArgs a, Seg sg, int tiles) {
    using K = Cfg<LN>;
    extern __shared__ float4 smem4[];
    Smem<LN> s(reinterpret_cast<float *>(smem4));
    const Place p = place(blockIdx.x, a.G, a.C / a.G, tiles, sg.segs, K::width);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nl = tid % LN, ch = tid / LN, n0 = nl * kNS;
    const bool live = ch < p.nc;
    const long long c = p.c0 + ch;
    float A2[kNS] = {}, h[kNS] = {}, w[kNS] = {};
    if (live) {
        load_states(a.A + c * a.N, n0, a.N, A2);
#pragma unroll
        for (int k = 0; k < kNS; ++k) A2[k] *= kLog2e;
        // the state before this segment and the gradient of the state after it
        const long long bc = ((long long)p.b * a.C + c) * a.N;
        if (a.state_in) load_states(a.state_in + bc, n0, a.N, h);
        if (a.dstate_in) load_states(a.dstate_in + bc, n0, a.N, w);
        const long long at = (long long)p.b * sg.segs * a.C + c;
        for (int i = 0; i < p.seg; ++i) {
            const long long q = at + (long long)i * a.C;
            const float d = sg.sum[q];
            float S[kNS];
            load_states(sg.S + q * a.N, n0, a.N, S);
#pragma unroll
            for (int k = 0; k < kNS; ++k) h[k] = fmaf(ex2(d * A2[k]), h[k], S[k]);
        }
        for (int i = sg.segs - 1; i > p.seg; --i) {
            const long long q = at + (long long)i * a.C;
            const float d = sg.sum[q];
            float R[kNS];
            load_states(sg.R + q * a.N, n0, a.N, R);
#pragma unroll
            for (int k = 0; k < kNS; ++k) w[k] = fmaf(ex2(d * A2[k]), w[k], R[k]);
        }
    }
    const int t0 = p.seg * sg.len, t1 = min(a.T, t0 + sg.len), n = min(seq_end(a.lengths, p.b, a.T), t1);
    const int count = n > t0 ? (n - t0 + kTile - 1) / kTile : 0;
    const long long tiles_t = (a.T + kTile - 1) / kTile;
    // this lane's states before tile i of the segment
    float *ck = sg.ckpt + (((long long)p.b * tiles_t + t0 / kTile) * a.C + c) * a.N;
    const long long ck_step = (long long)a.C * a.N;

    // ---- forwards: the state before every tile
    {
        Stager<T, LN, false> stg;
        if (count > 1) {
            stg.load(a, p, t0, n);
            stg.store(a, p, t0, n, s, 0);
        }
        for (int tile = 0; tile < count; ++tile) {
            if (live) store_states(ck + tile * ck_step, n0, a.N, h);
            if (tile + 1 == count) break;
            __syncthreads();
            const int buf = tile & 1;
            if (tile + 2 < count) stg.load(a, p, t0 + (tile + 1) * kTile, n);
            const float4 *in = s.in + buf * K::pairs + ch;
            const float *sB = s.B + buf * kTile * K::NP + n0;
#pragma unroll
            for (int j = 0; j < kTile; ++j) {
                const float2 v = *reinterpret_cast<const float2 *>(in + j * K::width);
                const float4 B4 = *reinterpret_cast<const float4 *>(sB + j * K::NP);
                const float Bk[4] = {B4.x, B4.y, B4.z, B4.w};
#pragma unroll
                for (int k = 0; k < kNS; ++k) h[k] = fmaf(ex2(v.x * A2[k]), h[k], v.y * Bk[k]);
            }
            if (tile + 2 < count) stg.store(a, p, t0 + (tile + 1) * kTile, n, s, buf ^ 1);
        }
        __syncthreads();
    }

    // ---- backwards
    float dA[kNS] = {}, dD = 0.f, dbias = 0.f;
    const long long row0 = (long long)p.b * a.T;
    Stager<T, LN, true> stg;
    if (count > 0) {
        stg.load(a, p, t0 + (count - 1) * kTile, n);
        stg.store(a, p, t0 + (count - 1) * kTile, n, s, (count - 1) & 1);
    }
    __syncthreads();
    for (int tile = count - 1; tile >= 0; --tile) {
        const int buf = tile & 1, tb = t0 + tile * kTile;
        if (tile > 0) stg.load(a, p, tb - kTile, n);
        const float4 *in = s.in + buf * K::pairs + ch;
        const float *sB = s.B + buf * kTile * K::NP + n0, *sC = s.C + buf * kTile * K::NP + n0;
        float hs[kNS] = {};
        if (live) load_states(ck + tile * ck_step, n0, a.N, hs);
        float H[kTile][kNS], E[kTile][kNS];
#pragma unroll
        for (int q = 0; q < kTile; q += 4) {
            float ys[4];
#pragma unroll
            for (int j = q; j < q + 4; ++j) {
                const float2 v = *reinterpret_cast<const float2 *>(in + j * K::width);
                const float4 B4 = *reinterpret_cast<const float4 *>(sB + j * K::NP);
                const float4 C4 = *reinterpret_cast<const float4 *>(sC + j * K::NP);
                const float Bk[4] = {B4.x, B4.y, B4.z, B4.w};
#pragma unroll
                for (int k = 0; k < kNS; ++k) {
                    E[j][k] = ex2(v.x * A2[k]);
                    H[j][k] = fmaf(E[j][k], j ? H[j - 1][k] : hs[k], v.y * Bk[k]);
                }
                ys[j - q] = fmaf(C4.x, H[j][0], fmaf(C4.y, H[j][1], fmaf(C4.z, H[j][2], C4.w * H[j][3])));
            }
            if (a.z) {
                reduce4<LN>(ys, nl);
                if (LN <= 4 || nl < 4) {
#pragma unroll
                    for (int j = 0; j < Kept<LN>::value; ++j)
                        s.o[(q + first_token<LN>(nl) + j) * K::width + ch] = ys[j];
                }
            }
        }
#pragma unroll
        for (int q = kTile - 4; q >= 0; q -= 4) {
            float lb[4], dd[4];
#pragma unroll
            for (int j = q + 3; j >= q; --j) {
                const float4 v = in[j * K::width];
                const float4 B4 = *reinterpret_cast<const float4 *>(sB + j * K::NP);
                const float4 C4 = *reinterpret_cast<const float4 *>(sC + j * K::NP);
                const float Bk[4] = {B4.x, B4.y, B4.z, B4.w}, Ck[4] = {C4.x, C4.y, C4.z, C4.w};
                float red[8];
                lb[j - q] = dd[j - q] = 0.f;
#pragma unroll
                for (int k = 0; k < kNS; ++k) {
                    const float lam = fmaf(v.z, Ck[k], w[k]);
                    red[k] = v.z * H[j][k];
                    red[4 + k] = v.y * lam;
                    lb[j - q] = fmaf(lam, Bk[k], lb[j - q]);
                    w[k] = E[j][k] * lam;
                    const float pr = w[k] * (j ? H[j - 1][k] : hs[k]);
                    dd[j - q] = fmaf(A2[k], pr, dd[j - q]);
                    dA[k] = fmaf(v.x, pr, dA[k]);
                }
                reduce_channels<LN>(red, lane, nl, s.red + (warp * kTile + j) * 2 * K::NP);
            }
            reduce4<LN>(lb, nl);
            reduce4<LN>(dd, nl);
            if (LN <= 4 || nl < 4) {
#pragma unroll
                for (int j = 0; j < Kept<LN>::value; ++j) {
                    const int at = (q + first_token<LN>(nl) + j) * K::width + ch;
                    s.o[K::pairs + at] = lb[j];
                    s.o[2 * K::pairs + at] = dd[j];
                }
            }
        }
        if (tile > 0) stg.store(a, p, tb - kTile, n, s, buf ^ 1);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < K::per; ++i) {
            const int e = tid + i * K::threads, t = tb + e / K::width, cc = e % K::width;
            if (t < t1 && cc < p.nc) {
                const long long o = (row0 + t) * a.C + p.c0 + cc;
                const float4 v = s.in[buf * K::pairs + e];
                const float2 x2 = s.ex[buf * K::pairs + e];
                const float q = s.o[K::pairs + e], Dc = a.D ? a.D[p.c0 + cc] : 0.f;
                const float ddt = (fmaf(v.w, q, s.o[2 * K::pairs + e] * (1.f / kLog2e))) * x2.x;
                const bool in_seq = t < n;
                ((T *)a.dx)[o] = from_f<T>(in_seq ? fmaf(v.x, q, Dc * v.z) : 0.f);
                ((T *)a.ddt)[o] = from_f<T>(in_seq ? ddt : 0.f);
                if (a.z) ((T *)a.dz)[o] = from_f<T>(in_seq ? x2.y * fmaf(Dc, v.w, s.o[e]) : 0.f);
                if (in_seq) {
                    dD = fmaf(v.z, v.w, dD);
                    dbias += ddt;
                }
            }
        }
        for (int e = tid; e < kTile * 2 * K::NP; e += K::threads) {
            const int j = e / (2 * K::NP), m = e % (2 * K::NP), t = tb + j, st = m % K::NP;
            if (t < n && st < a.N) {
                float r = 0.f;
#pragma unroll
                for (int u = 0; u < K::warps; ++u) r += s.red[(u * kTile + j) * 2 * K::NP + m];
                const long long plane = (long long)a.B * a.T * a.G * a.N;
                const int ct = (p.c0 - p.g * (a.C / a.G)) / K::width;
                sg.bc[(2 * (long long)ct + m / K::NP) * plane + ((row0 + t) * a.G + p.g) * a.N + st] = r;
            }
        }
        __syncthreads();
    }
    // rows behind the sequence's end
    for (long long e = (long long)count * kTile * K::width + tid; e < (long long)(t1 - t0) * K::width; e += K::threads) {
        const int t = t0 + (int)(e / K::width), cc = (int)(e % K::width);
        if (cc < p.nc) {
            const long long o = (row0 + t) * a.C + p.c0 + cc;
            ((T *)a.dx)[o] = ((T *)a.ddt)[o] = from_f<T>(0.f);
            if (a.z) ((T *)a.dz)[o] = from_f<T>(0.f);
        }
    }
    // this block's parts of the sums over tokens
    const long long part = (long long)p.b * sg.segs + p.seg;
    if (live) {
        store_states(sg.pA + (part * a.C + c) * a.N, n0, a.N, dA);
        if (p.seg == 0 && a.dstate_out) store_states(a.dstate_out + ((long long)p.b * a.C + c) * a.N, n0, a.N, w);
    }
    // every thread's pairs were all of channel tid % width
    s.o[tid] = dD;
    s.o[K::threads + tid] = dbias;
    __syncthreads();
    if (tid < p.nc) {
        float r0 = 0.f, r1 = 0.f;
#pragma unroll
        for (int i = 0; i < LN; ++i) {
            r0 += s.o[i * K::width + tid];
            r1 += s.o[K::threads + i * K::width + tid];
        }
        sg.pD[part * a.C + p.c0 + tid] = r0;
        sg.pbias[part * a.C + p.c0 + tid] = r1;
    }
}

// Joins the parts: the first blocks dC and dB over the channel tiles, the others dA, dD and dbias
// over batch entries and segments.
constexpr int kJoin = 256;

template <typename T>
__global__ void __launch_bounds__(kJoin) scan_bwd_join(ScanArgs a, Seg sg, int tiles, int bc_blocks) {
    if ((int)blockIdx.x < bc_blocks) {
        const long long plane = (long long)a.B * a.T * a.G * a.N;
        const long long e = (long long)blockIdx.x * kJoin + threadIdx.x;
        if (e >= plane) return;
        const long long row = e / ((long long)a.G * a.N);
        const int b = (int)(row / a.T), t = (int)(row - (long long)b * a.T);
        float r0 = 0.f, r1 = 0.f;
        if (t < seq_end(a.lengths, b, a.T)) {
#pragma unroll 4
            for (int i = 0; i < tiles; ++i) {
                r0 += sg.bc[2 * i * plane + e];
                r1 += sg.bc[(2 * i + 1) * plane + e];
            }
        }
        ((T *)a.dCm)[e] = from_f<T>(r0);
        ((T *)a.dBm)[e] = from_f<T>(r1);
        return;
    }
    const long long e = (long long)(blockIdx.x - bc_blocks) * kJoin + threadIdx.x;
    const long long cn = (long long)a.C * a.N, all = cn + 2 * (long long)a.C;
    if (e >= all) return;
    const float *p = e < cn ? sg.pA + e : e < cn + a.C ? sg.pD + (e - cn) : sg.pbias + (e - cn - a.C);
    float *out = e < cn ? a.dA + e : e < cn + a.C ? (a.dD ? a.dD + (e - cn) : nullptr)
                                                  : (a.ddt_bias ? a.ddt_bias + (e - cn - a.C) : nullptr);
    if (!out) return;
    const long long step = e < cn ? cn : a.C;
    float r = 0.f;
    for (int i = 0; i < a.B * sg.segs; ++i) r += p[i * step];
    *out = r;
}

int block_threads(int N) { return lanes_for(N) == 1 ? 128 : 256; }

// Segments of the backward, from the sizes alone: one where the blocks fill two thirds of the SMs,
// else enough for two blocks an SM, each of at least 128 tokens.
void bwd_segments(int B, int T, int C, int G, int N, int *segs, int *len) {
    const int width = block_threads(N) / lanes_for(N);
    const long long blocks = (long long)B * G * ((C / G + width - 1) / width);
    long long want = blocks >= 100 ? 1 : (2 * 148 + blocks - 1) / blocks;
    if (want > T / 128) want = T / 128;
    if (want < 1) want = 1;
    *len = (int)(((T + want - 1) / want + kTile - 1) / kTile * kTile);
    *segs = (T + *len - 1) / *len;
}

// Cuts the workspace into its parts; returns its size.
size_t layout(int B, int T, int C, int G, int N, void *ws, Seg *sg) {
    bwd_segments(B, T, C, G, N, &sg->segs, &sg->len);
    const int width = block_threads(N) / lanes_for(N);
    const size_t tiles = (C / G + width - 1) / width, parts = (size_t)B * sg->segs, cn = (size_t)C * N;
    char *p = (char *)ws;
    auto take = [&](size_t floats) {
        float *r = (float *)p;
        p += up256(floats * sizeof(float));
        return r;
    };
    const bool split = sg->segs > 1;
    sg->S = take(split ? parts * cn : 0);
    sg->R = take(split ? parts * cn : 0);
    sg->sum = take(split ? parts * C : 0);
    sg->ckpt = take((size_t)B * ((T + kTile - 1) / kTile) * cn);
    sg->bc = take(tiles * 2 * B * T * G * N);
    sg->pA = take(parts * cn);
    sg->pD = take(parts * C);
    sg->pbias = take(parts * C);
    return (size_t)(p - (char *)ws);
}

template <typename T, int LN>
la_status bwd_ln(const ScanArgs &a, cudaStream_t st) {
    using K = Cfg<LN>;
    Seg sg;
    layout(a.B, a.T, a.C, a.G, a.N, a.ws, &sg);
    const int tiles = (a.C / a.G + K::width - 1) / K::width;
    const dim3 grid((unsigned)((long long)a.B * sg.segs * a.G * tiles)), block(K::threads);
    la_status rc = LA_OK;
    if (sg.segs > 1) {
        rc = launch("selective_scan_bwd_ends", scan_bwd_ends<T, LN>, grid, block, K::smem, st, a, sg, tiles);
        if (rc != LA_OK) return rc;
    }
    rc = launch("selective_scan_bwd", scan_bwd_kernel<T, LN>, grid, block, K::smem, st, a, sg, tiles);
    if (rc != LA_OK) return rc;
    const long long plane = (long long)a.B * a.T * a.G * a.N, rest = (long long)a.C * (a.N + 2);
    const int bc_blocks = (int)((plane + kJoin - 1) / kJoin);
    return launch("selective_scan_bwd_join", scan_bwd_join<T>, dim3((unsigned)(bc_blocks + (rest + kJoin - 1) / kJoin)),
                  dim3(kJoin), 0, st, a, sg, tiles, bc_blocks);
}

template <typename T>
la_status bwd_t(const ScanArgs &a, cudaStream_t st) {
    switch (lanes_for(a.N)) {
    case 1: return bwd_ln<T, 1>(a, st);
    case 2: return bwd_ln<T, 2>(a, st);
    case 4: return bwd_ln<T, 4>(a, st);
    case 8: return bwd_ln<T, 8>(a, st);
    default: return bwd_ln<T, 16>(a, st);
    }
}

}  // namespace

size_t scan_bwd_workspace(int B, int T, int C, int G, int N) {
    Seg sg;
    return layout(B, T, C, G, N, nullptr, &sg);
}

la_status scan_bwd(const ScanArgs &a, cudaStream_t st) {
    switch (a.dt) {
    case LA_F32: return bwd_t<float>(a, st);
    case LA_F16: return bwd_t<__half>(a, st);
    default: return bwd_t<__nv_bfloat16>(a, st);
    }
}

}  // namespace la

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
// kSub tokens in the workspace, then backwards, kSub tokens at a time: their states and decays are
// formed again in registers (one exponential each) and used in reverse order.  So a state costs two
// exponentials and about 12 multiply-adds, and 4 / kSub bytes of workspace traffic each way: the
// kernel is bound by instructions and their latency, not by HBM.  The sums over channels of dB and dC
// go through shared memory, first over a warp's lanes, then over the block's warps, then over the
// channel tiles in a last launch, always in the same order; that launch also joins the batch entries'
// parts of dA, dD and dbias.
// Measured at B4 T2048 C2048 N16 bf16: 620 us, where the traffic would take 36 and the special functions
// (32 exponentials and 7 more a token and channel) 141; issue slots 39 % busy, shared memory 52 %: 256 blocks
// of four warps and 254 registers are 1.7 warps a scheduler.  More warps by fewer registers or segments cost
// more than they give (kSub = 4 with 168 registers 747 us, with 128 and two segments 767; two channels a lane
// 980; two states a lane 806).
//
// Few channels and a long sequence: segments as in the forward.  A first launch gives every
// segment's end state from zero, S, its sum of d, and the gradient that it hands to the state
// before it, R = sum_t (prod_{s<=t} a_s) e_t C_t, from the same exponentials in one sweep.
#include "la_scan.cuh"

namespace la {
namespace {

using namespace scan;

constexpr int kSub = 8;            // tokens whose states and decays are in registers at a time

template <int LN> struct Cfg {
    static constexpr int threads = LN == 1 ? 64 : 128;
    static constexpr int warps = threads / 32;
    static constexpr int width = threads / LN;
    static constexpr int NP = kNS * LN;
    static constexpr int pairs = kTile * width;             // (token, channel)
    static constexpr int quads = pairs / 4;
    static constexpr int per = (quads + threads - 1) / threads;
    static constexpr int bquads = kTile * LN;
    static constexpr int bper = (bquads + threads - 1) / threads;
    static constexpr int subs = kTile / kSub;
    // d, u, e, sigma, dz (twice), B and C (twice), the three sums over states, the warps' sums of dC
    // and dB, and their places for forming them; the lanes' states before sub-tiles (twice)
    static constexpr size_t smem = sizeof(float) * (10 * pairs + 4 * kTile * NP + 3 * pairs + warps * kTile * 2 * NP) +
                                   warps * kSub * 2 * (512 + 16 * LN) + 2 * subs * threads * 16;
    static_assert(smem <= 227 * 1024, "shared memory of a block");
};

struct Seg {
    int segs, len;
    float *S, *R, *sum;            // [B, segs, C, N] twice, [B, segs, C]
    float *ckpt;                   // [B, ceil(T / kSub), C, 4 LN]
    float *bc;                     // [tiles][2][B T G N]: the channel tiles' parts of dC and dB
    float *pA, *pD, *pbias;        // [B segs][C N], [B segs][C] twice
    int vec, bvec;                 // rows of the [B,T,C] tensors (of Bm, Cm) allow accesses of 4 elements
};

// The sums over a warp's 32 / LN channels of what its lanes hold for dC and dB of kSub tokens, four
// states each: every lane leaves them in the warp's part of shared memory, then adds up whole columns.
// (Exchanging halves by shuffles takes 28 instructions a token for these sums; this takes 9.)
// A quarter's lanes are followed by 16 bytes of room, so that reads of different quarters and rows
// meet different banks.
template <int LN> struct Columns {
    static constexpr int quarter = 512 / LN + 16;                  // bytes from one quarter's lanes to the next
    static constexpr int stride = LN * quarter;                    // bytes from one (token, quantity) to the next
    static constexpr int bytes = kSub * 2 * stride;                // a warp
    static constexpr int items = kSub * 2 * LN;                    // columns of four states
};
template <int LN>
struct Smem {
    using K = Cfg<LN>;
    float *d, *u, *e;              // [2][kTile][width]
    float *sig, *dz;               // [2][kTile][width]: sigma(dt + bias) (1 without softplus), dy silu'(z)
    float *B, *C;                  // [2][kTile][NP]
    float *o;                      // [3][kTile][width]: sum_n C h, q, sum_n A p (in units of 1 / log2 e)
    float *red;                    // [warps][kTile][2][NP]
    char *columns;                 // [warps], see sum_channels
    float4 *before;                // [2][kTile / kSub][threads]
    __device__ explicit Smem(float *p) {
        d = p;
        u = d + 2 * K::pairs;
        e = u + 2 * K::pairs;
        sig = e + 2 * K::pairs;
        dz = sig + 2 * K::pairs;
        B = dz + 2 * K::pairs;
        C = B + 2 * kTile * K::NP;
        o = C + 2 * kTile * K::NP;
        red = o + 3 * K::pairs;
        columns = reinterpret_cast<char *>(red + K::warps * kTile * 2 * K::NP);
        before = reinterpret_cast<float4 *>(columns + K::warps * Columns<LN>::bytes);
    }
};

// Stages tiles of kTile tokens: load() fetches one into registers, store() converts it into shared
// memory.  BACK: with dy, z and C; else x, dt and B only.  A thread's quads are all of the same four
// channels.
template <typename T, int LN, bool BACK>
struct Stager {
    using K = Cfg<LN>;
    static constexpr int row = K::width / 4, t_step = K::threads / row, b_step = K::threads / LN;
    Quad<T> rx[K::per], rd[K::per], rz[K::per], rg[K::per], rB[K::bper], rC[K::bper];
    const ScanArgs &a;
    const Seg &sg;
    int c, have, t_first, b_first, b_have, n;
    long long x0, xs, b0, bs;      // element offsets of the thread's first quad at token 0, steps between quads
    f2 bias[2];

    __device__ __forceinline__ Stager(const ScanArgs &a_, const Seg &sg_, const Place &p, int n_) : a(a_), sg(sg_), n(n_) {
        const int tid = threadIdx.x, m = tid % LN * 4;
        const long long row0 = (long long)p.b * a.T;
        c = tid % row * 4;
        have = p.nc - c;
        t_first = tid / row;
        b_first = tid / LN;
        b_have = a.N - m;
        x0 = (row0 + t_first) * a.C + p.c0 + c;
        xs = (long long)t_step * a.C;
        b0 = ((row0 + b_first) * a.G + p.g) * a.N + m;
        bs = (long long)b_step * a.G * a.N;
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = a.dt_bias && j < have ? a.dt_bias[p.c0 + c + j] : 0.f;
        bias[0] = pack2(v[0], v[1]);
        bias[1] = pack2(v[2], v[3]);
    }
    static __device__ __forceinline__ bool mine(int i) { return K::quads % K::threads == 0 || (int)threadIdx.x + i * K::threads < K::quads; }
    static __device__ __forceinline__ bool mine_b(int i) { return K::bquads % K::threads == 0 || (int)threadIdx.x + i * K::threads < K::bquads; }

    __device__ __forceinline__ void load(int tb) {
        const long long xo = x0 + (long long)tb * a.C, bo = b0 + (long long)tb * a.G * a.N;
#pragma unroll
        for (int i = 0; i < K::per; ++i)
            if (mine(i)) {
                const int live = tb + t_first + i * t_step < n ? have : 0;
                rx[i].load((const T *)a.x + xo + i * xs, live, sg.vec);
                rd[i].load((const T *)a.dt_in + xo + i * xs, live, sg.vec);
                if (BACK) {
                    rg[i].load((const T *)a.dy + xo + i * xs, live, sg.vec);
                    if (a.z) rz[i].load((const T *)a.z + xo + i * xs, live, sg.vec);
                }
            }
#pragma unroll
        for (int i = 0; i < K::bper; ++i)
            if (mine_b(i)) {
                const int live = tb + b_first + i * b_step < n ? b_have : 0;
                rB[i].load((const T *)a.Bm + bo + i * bs, live, sg.bvec);
                if (BACK) rC[i].load((const T *)a.Cm + bo + i * bs, live, sg.bvec);
            }
    }
    static __device__ __forceinline__ void put(float *plane, int at, const f2 (&v)[2]) {
        reinterpret_cast<ulonglong2 *>(plane)[at] = make_ulonglong2(v[0], v[1]);
    }
    __device__ __forceinline__ void store(int tb, Smem<LN> &s, int buf) {
#pragma unroll
        for (int i = 0; i < K::per; ++i)
            if (mine(i)) {
                const int at = buf * K::quads + threadIdx.x + i * K::threads;
                const bool gone = tb + t_first + i * t_step >= n;         // behind the end: the state stays
                f2 d[2], x[2], u[2], sig[2] = {both(1.f), both(1.f)};
                rd[i].values(d);
                rx[i].values(x);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    d[j] = add2(d[j], bias[j]);
                    if (a.softplus) {
                        float r0, r1;
                        unpack2(d[j], r0, r1);
                        const float e0 = exp_neg_abs(r0), e1 = exp_neg_abs(r1);
                        // sigma(r): 1 / (1 + e) for r >= 0, e / (1 + e) below
                        if (BACK) sig[j] = pack2((r0 < 0.f ? e0 : 1.f) * rcp(1.f + e0), (r1 < 0.f ? e1 : 1.f) * rcp(1.f + e1));
                        d[j] = pack2(softplus_from(r0, e0), softplus_from(r1, e1));
                    }
                    if (gone) d[j] = 0;
                    u[j] = mul2(d[j], x[j]);
                }
                put(s.d, at, d);
                put(s.u, at, u);
                if (BACK) {
                    f2 g[2], z[2], dz[2] = {0, 0};
                    rg[i].values(g);
                    if (a.z) {
                        rz[i].values(z);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            // silu'(z) = sg (1 + z (1 - sg))
                            const f2 sg_ = sigmoid2(z[j]), gs = mul2(g[j], sg_);
                            dz[j] = mul2(gs, fma2(z[j], fma2(sg_, both(-1.f), both(1.f)), both(1.f)));
                            g[j] = mul2(gs, z[j]);
                        }
                    }
                    put(s.e, at, g);
                    put(s.sig, at, sig);
                    put(s.dz, at, dz);
                }
            }
#pragma unroll
        for (int i = 0; i < K::bper; ++i)
            if (mine_b(i)) {
                f2 v[2];
                const int at = buf * K::bquads + threadIdx.x + i * K::threads;
                rB[i].values(v);
                put(s.B, at, v);
                if (BACK) {
                    rC[i].values(v);
                    put(s.C, at, v);
                }
            }
    }
};

template <int LN>
__device__ __forceinline__ void sum_channels(const f2 (&rc)[kSub][2], const f2 (&rb)[kSub][2], char *mine, int lane,
                                             float *out) {
    typedef Columns<LN> Q;
    constexpr int NP = kNS * LN;
#pragma unroll
    for (int j = 0; j < kSub; ++j) {
        char *p = mine + 2 * j * Q::stride + lane / (32 / LN) * Q::quarter + lane % (32 / LN) * 16;
        *reinterpret_cast<ulonglong2 *>(p) = make_ulonglong2(rc[j][0], rc[j][1]);
        *reinterpret_cast<ulonglong2 *>(p + Q::stride) = make_ulonglong2(rb[j][0], rb[j][1]);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < Q::items; i += 32) {
        const int it = i + lane, row = it / LN, nl = it % LN;
        if (Q::items % 32 == 0 || it < Q::items) {
            f2 s0 = 0, s1 = 0;
#pragma unroll
            for (int ch = 0; ch < 32 / LN; ++ch) {
                const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(mine + row * Q::stride + nl * Q::quarter + ch * 16);
                s0 = ch ? add2(s0, v.x) : v.x;
                s1 = ch ? add2(s1, v.y) : v.y;
            }
            // row = 2 token + quantity: out is [token][quantity][NP]
            *reinterpret_cast<ulonglong2 *>(out + row * NP + nl * kNS) = make_ulonglong2(s0, s1);
        }
    }
    __syncwarp();
}

// Four states' B or C of a token.
struct Four {
    f2 v[2];
    __device__ __forceinline__ explicit Four(const float *p) {
        const ulonglong2 q = *reinterpret_cast<const ulonglong2 *>(p);
        v[0] = q.x;
        v[1] = q.y;
    }
};

// dA's sum over the `count` tokens of a tile that exist, one by one: hs is the state before them, w the
// gradient that the tokens behind them hand over.
__device__ __forceinline__ void last_tokens(int count, const float *d, const float *u, const float *e, int width,
                                            const float *B, const float *C, int NP, const f2 (&A2)[2],
                                            const f2 (&hs)[2], f2 w0, f2 w1, float (&dA)[kNS]) {
    f2 w[2] = {w0, w1}, sum[2] = {0, 0};
#pragma unroll 1
    for (int j = count - 1; j >= 0; --j) {
        f2 h[2] = {hs[0], hs[1]};
#pragma unroll 1
        for (int i = 0; i < j; ++i) {
            const f2 di = both(d[i * width]), ui = both(u[i * width]);
            const Four Bi(B + i * NP);
            h[0] = fma2(decay2(di, A2[0]), h[0], mul2(ui, Bi.v[0]));
            h[1] = fma2(decay2(di, A2[1]), h[1], mul2(ui, Bi.v[1]));
        }
        const f2 dj = both(d[j * width]), ej = both(e[j * width]);
        const Four Cj(C + j * NP);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            w[k] = mul2(decay2(dj, A2[k]), fma2(ej, Cj.v[k], w[k]));
            sum[k] = fma2(dj, mul2(w[k], h[k]), sum[k]);
        }
    }
    unpack2(sum[0], dA[0], dA[1]);
    unpack2(sum[1], dA[2], dA[3]);
}

// First launch of the segmented form: (S, R, sum of d) of every segment.
template <typename T, int LN>
__global__ void __launch_bounds__(Cfg<LN>::threads)
scan_bwd_ends(ScanArgs a, Seg sg, int tiles) {
    using K = Cfg<LN>;
    extern __shared__ float4 smem4[];
    Smem<LN> s(reinterpret_cast<float *>(smem4));
    const Place p = place(blockIdx.x, a.G, a.C / a.G, tiles, sg.segs, K::width);
    const int nl = lane_states<LN>(), ch = lane_channel<LN>(), n0 = nl * kNS;
    const bool live = ch < p.nc;
    const long long c = p.c0 + ch;
    float A4[kNS] = {}, sum = 0.f;
    if (live) load_states(a.A + c * a.N, n0, a.N, A4);
    const f2 A2[2] = {mul2(pack2(A4[0], A4[1]), both(kLog2e)), mul2(pack2(A4[2], A4[3]), both(kLog2e))};
    f2 h[2] = {0, 0}, P[2] = {both(1.f), both(1.f)}, R[2] = {0, 0};
    const int t0 = p.seg * sg.len, n = min(seq_end(a.lengths, p.b, a.T), min(a.T, t0 + sg.len));
    const int count = n > t0 ? (n - t0 + kTile - 1) / kTile : 0;
    Stager<T, LN, true> stg(a, sg, p, n);
    if (count > 0) {
        stg.load(t0);
        stg.store(t0, s, 0);
    }
    for (int tile = 0; tile < count; ++tile) {
        __syncthreads();
        const int buf = tile & 1;
        if (tile + 1 < count) stg.load(t0 + (tile + 1) * kTile);
        const int at = buf * K::pairs + ch, bt = buf * kTile * K::NP + n0;
#pragma unroll
        for (int j = 0; j < kTile; ++j) {
            const float d1 = s.d[at + j * K::width];
            const f2 d = both(d1), u = both(s.u[at + j * K::width]), e = both(s.e[at + j * K::width]);
            const Four B(s.B + bt + j * K::NP), C(s.C + bt + j * K::NP);
            sum += d1;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const f2 E = decay2(d, A2[k]);
                h[k] = fma2(E, h[k], mul2(u, B.v[k]));
                P[k] = mul2(P[k], E);
                R[k] = fma2(P[k], mul2(e, C.v[k]), R[k]);
            }
        }
        if (tile + 1 < count) stg.store(t0 + (tile + 1) * kTile, s, buf ^ 1);
    }
    if (!live) return;
    const long long at = ((long long)p.b * sg.segs + p.seg) * a.C + c;
    float v[4];
    unpack2(h[0], v[0], v[1]);
    unpack2(h[1], v[2], v[3]);
    store_states(sg.S + at * a.N, n0, a.N, v);
    unpack2(R[0], v[0], v[1]);
    unpack2(R[1], v[2], v[3]);
    store_states(sg.R + at * a.N, n0, a.N, v);
    if (nl == 0) sg.sum[at] = sum;
}

template <typename T, int LN, bool PAD>
__global__ void __launch_bounds__(Cfg<LN>::threads)
scan_bwd_kernel(ScanArgs a, Seg sg, int tiles) {
    using K = Cfg<LN>;
    extern __shared__ float4 smem4[];
    Smem<LN> s(reinterpret_cast<float *>(smem4));
    const Place p = place(blockIdx.x, a.G, a.C / a.G, tiles, sg.segs, K::width);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nl = lane_states<LN>(), ch = lane_channel<LN>(), n0 = nl * kNS;
    const bool live = ch < p.nc;
    const long long c = p.c0 + ch;
    f2 A2[2], h[2], w[2];
    wait_for_stream();
    {
        float A4[kNS] = {}, h4[kNS] = {}, w4[kNS] = {};
        if (live) {
            load_states(a.A + c * a.N, n0, a.N, A4);
#pragma unroll
            for (int k = 0; k < kNS; ++k) A4[k] *= kLog2e;
            // the state before this segment and the gradient of the state after it
            const long long bc = ((long long)p.b * a.C + c) * a.N;
            if (a.state_in) load_states(a.state_in + bc, n0, a.N, h4);
            if (a.dstate_in) load_states(a.dstate_in + bc, n0, a.N, w4);
            const long long at = (long long)p.b * sg.segs * a.C + c;
#pragma unroll 4
            for (int i = 0; i < p.seg; ++i) {
                const long long q = at + (long long)i * a.C;
                const float d = sg.sum[q];
                float S[kNS];
                load_states(sg.S + q * a.N, n0, a.N, S);
#pragma unroll
                for (int k = 0; k < kNS; ++k) h4[k] = fmaf(ex2(d * A4[k]), h4[k], S[k]);
            }
#pragma unroll 4
            for (int i = sg.segs - 1; i > p.seg; --i) {
                const long long q = at + (long long)i * a.C;
                const float d = sg.sum[q];
                float R[kNS];
                load_states(sg.R + q * a.N, n0, a.N, R);
#pragma unroll
                for (int k = 0; k < kNS; ++k) w4[k] = fmaf(ex2(d * A4[k]), w4[k], R[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            A2[k] = pack2(A4[2 * k], A4[2 * k + 1]);
            h[k] = pack2(h4[2 * k], h4[2 * k + 1]);
            w[k] = pack2(w4[2 * k], w4[2 * k + 1]);
        }
    }
    const int t0 = p.seg * sg.len, t1 = min(a.T, t0 + sg.len), n = min(seq_end(a.lengths, p.b, a.T), t1);
    const int count = n > t0 ? (n - t0 + kTile - 1) / kTile : 0;
    const long long subs_t = (a.T + kSub - 1) / kSub;
    // this lane's states before sub-tile i of the segment
    float *ck = sg.ckpt + (((long long)p.b * subs_t + t0 / kSub) * a.C + c) * K::NP + n0;
    const long long ck_step = (long long)a.C * K::NP;
    const int subs = count > 0 ? (n - t0 + kSub - 1) / kSub : 0;

    // ---- forwards: the state before every sub-tile
    {
        Stager<T, LN, false> stg(a, sg, p, n);
        if (count > 0) {
            stg.load(t0);
            stg.store(t0, s, 0);
        }
        for (int tile = 0; tile < count; ++tile) {
            __syncthreads();
            const int buf = tile & 1;
            if (tile + 1 < count) stg.load(t0 + (tile + 1) * kTile);
            const int at = buf * K::pairs + ch, bt = buf * kTile * K::NP + n0;
            f2 mid[kTile / kSub][2];
#pragma unroll
            for (int j = 0; j < kTile; ++j) {
                const f2 d = both(s.d[at + j * K::width]), u = both(s.u[at + j * K::width]);
                const Four B(s.B + bt + j * K::NP);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (j % kSub == 0) mid[j / kSub][k] = h[k];
                    h[k] = fma2(decay2(d, A2[k]), h[k], mul2(u, B.v[k]));
                }
            }
#pragma unroll
            for (int i = 0; i < kTile / kSub; ++i)
                if (live && tile * K::subs + i < subs)
                    *reinterpret_cast<ulonglong2 *>(ck + (tile * K::subs + i) * ck_step) =
                        make_ulonglong2(mid[i][0], mid[i][1]);
            if (tile + 1 < count) stg.store(t0 + (tile + 1) * kTile, s, buf ^ 1);
        }
        __syncthreads();
    }

    // ---- backwards
    const bool gated = a.z != nullptr;
    const Existing<PAD> real(n0, a.N);
    f2 dA[2] = {0, 0}, dD[2] = {0, 0}, dbias[2] = {0, 0}, Dc[2];
    Stager<T, LN, true> stg(a, sg, p, n);
    {
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = a.D && j < stg.have ? a.D[p.c0 + stg.c + j] : 0.f;
        Dc[0] = pack2(v[0], v[1]);
        Dc[1] = pack2(v[2], v[3]);
    }
    // the states before a tile's sub-tiles come a tile ahead, each lane's into its own place
    auto fetch = [&](int tile) {
#pragma unroll
        for (int i = 0; i < K::subs; ++i)
            copy_async<16>(s.before + ((tile & 1) * K::subs + i) * K::threads + tid,
                           ck + (long long)(tile * K::subs + i) * ck_step, live && tile * K::subs + i < subs);
        copy_commit();
    };
    if (count > 0) {
        fetch(count - 1);
        stg.load(t0 + (count - 1) * kTile);
        stg.store(t0 + (count - 1) * kTile, s, (count - 1) & 1);
    }
    __syncthreads();
    // Where the sequence ends within a sub-tile, the tile's sum for dA takes the tokens that exist one by one and
    // waits in the workspace (kept in registers over the loop, or as a test for each token, it spills and costs
    // up to 10 % at N = 5 .. 8 and N > 32): behind them d is 0, but the state may be infinite.
    if (count > 0 && (n - t0) % kSub != 0) {
        const int buf = (count - 1) & 1, at = buf * K::pairs + ch, bt = buf * kTile * K::NP + n0;
        copy_wait<0>();
        const ulonglong2 hs = *reinterpret_cast<const ulonglong2 *>(s.before + buf * K::subs * K::threads + tid);
        float v[kNS];
        last_tokens((n - t0 - 1) % kTile + 1, s.d + at, s.u + at, s.e + at, K::width, s.B + bt, s.C + bt, K::NP, A2,
                    {hs.x, hs.y}, w[0], w[1], v);
        if (live) store_states(sg.pA + (((long long)p.b * sg.segs + p.seg) * a.C + c) * a.N, n0, a.N, v);
    }
    for (int tile = count - 1; tile >= 0; --tile) {
        const int buf = tile & 1, tb = t0 + tile * kTile;
        copy_wait<0>();
        if (tile > 0) fetch(tile - 1);
        Quad<T> kx[K::per];                                   // this tile's x, for its outputs
#pragma unroll
        for (int i = 0; i < K::per; ++i) kx[i] = stg.rx[i];
        if (tile > 0) stg.load(tb - kTile);
#pragma unroll
        for (int sub = kTile / kSub - 1; sub >= 0; --sub) {
            const int at = buf * K::pairs + sub * kSub * K::width + ch, bt = (buf * kTile + sub * kSub) * K::NP + n0;
            const ulonglong2 before =
                *reinterpret_cast<const ulonglong2 *>(s.before + (buf * K::subs + sub) * K::threads + tid);
            const f2 hs[2] = {real(before.x, 0), real(before.y, 1)};
            f2 H[kSub][2], E[kSub][2];
            float ys[kSub / 4][4], lb[kSub / 4][4], dd[kSub / 4][4];
            f2 rc[kSub][2], rb[kSub][2];
#pragma unroll
            for (int j = 0; j < kSub; ++j) {
                const f2 d = both(s.d[at + j * K::width]), u = both(s.u[at + j * K::width]);
                const Four B(s.B + bt + j * K::NP);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    E[j][k] = real(decay2(d, A2[k]), k);
                    H[j][k] = real(fma2(E[j][k], j ? H[j - 1][k] : hs[k], mul2(u, B.v[k])), k);
                }
                if (gated) {
                    const Four C(s.C + bt + j * K::NP);
                    float y0, y1;
                    unpack2(fma2(C.v[0], H[j][0], mul2(C.v[1], H[j][1])), y0, y1);
                    ys[j / 4][j % 4] = y0 + y1;
                }
            }
            if (gated)
#pragma unroll
                for (int q = 0; q < kSub / 4; ++q) reduce4<LN>(ys[q], nl);
            f2 dAs[2] = {0, 0};
#pragma unroll
            for (int j = kSub - 1; j >= 0; --j) {
                const f2 d = both(s.d[at + j * K::width]), u = both(s.u[at + j * K::width]),
                         e = both(s.e[at + j * K::width]);
                const Four B(s.B + bt + j * K::NP), C(s.C + bt + j * K::NP);
                f2 ql[2], qa[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const f2 lam = real(fma2(e, C.v[k], w[k]), k);
                    rc[j][k] = mul2(e, H[j][k]);
                    rb[j][k] = mul2(u, lam);
                    ql[k] = mul2(lam, B.v[k]);
                    w[k] = mul2(E[j][k], lam);
                    const f2 pr = mul2(w[k], j ? H[j - 1][k] : hs[k]);
                    qa[k] = mul2(A2[k], pr);
                    dAs[k] = fma2(d, pr, dAs[k]);
                }
                float v0, v1;
                unpack2(add2(ql[0], ql[1]), v0, v1);
                lb[j / 4][j % 4] = v0 + v1;
                unpack2(add2(qa[0], qa[1]), v0, v1);
                dd[j / 4][j % 4] = v0 + v1;
            }
            dA[0] = add2(dA[0], dAs[0]);
            dA[1] = add2(dA[1], dAs[1]);
#pragma unroll
            for (int q = 0; q < kSub / 4; ++q) {
                reduce4<LN>(lb[q], nl);
                reduce4<LN>(dd[q], nl);
            }
            if (LN <= 4 || nl < 4) {
                float *o = s.o + (sub * kSub + first_token<LN>(nl)) * K::width + ch;
#pragma unroll
                for (int q = 0; q < kSub / 4; ++q)
#pragma unroll
                    for (int j = 0; j < Kept<LN>::value; ++j) {
                        if (gated) o[(4 * q + j) * K::width] = ys[q][j];
                        o[K::pairs + (4 * q + j) * K::width] = lb[q][j];
                        o[2 * K::pairs + (4 * q + j) * K::width] = dd[q][j];
                    }
            }
            sum_channels<LN>(rc, rb, s.columns + warp * Columns<LN>::bytes, lane,
                             s.red + (warp * kTile + sub * kSub) * 2 * K::NP);
        }
        if (n - tb <= kTile && (n & (kSub - 1))) dA[0] = dA[1] = 0;              // waits in the workspace
        if (tile > 0) stg.store(tb - kTile, s, buf ^ 1);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < K::per; ++i) {
            const int t = tb + stg.t_first + i * Stager<T, LN, true>::t_step;
            if (Stager<T, LN, true>::mine(i) && t < t1) {
                const int e4 = tid + i * K::threads;
                auto get = [&](const float *plane, int i4) { return reinterpret_cast<const ulonglong2 *>(plane)[i4]; };
                const int b4 = buf * K::quads + e4;
                const ulonglong2 sig = get(s.sig, b4), dz = get(s.dz, b4), d = get(s.d, b4), g = get(s.e, b4);
                const ulonglong2 y = get(s.o, e4), q = get(s.o, K::quads + e4), ap = get(s.o, 2 * K::quads + e4);
                const f2 sg2[2] = {sig.x, sig.y}, dz2[2] = {dz.x, dz.y}, d2[2] = {d.x, d.y}, g2[2] = {g.x, g.y};
                const f2 y2[2] = {y.x, y.y}, q2[2] = {q.x, q.y}, ap2[2] = {ap.x, ap.y};
                f2 x2[2];
                kx[i].values(x2);
                float ox[4], od[4], oz[4];
                const bool in_seq = t < n;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    // without D no product with a zero: x or dy may be infinite
                    f2 dx = a.D ? fma2(d2[j], q2[j], mul2(Dc[j], g2[j])) : mul2(d2[j], q2[j]);
                    f2 dt = mul2(fma2(x2[j], q2[j], mul2(ap2[j], both(1.f / kLog2e))), sg2[j]);
                    f2 gz = mul2(dz2[j], a.D ? fma2(Dc[j], x2[j], y2[j]) : y2[j]);
                    if (!in_seq) dx = dt = gz = 0;
                    dD[j] = fma2(g2[j], x2[j], dD[j]);                    // 0 behind the end: g and x are
                    dbias[j] = add2(dbias[j], dt);
                    unpack2(dx, ox[2 * j], ox[2 * j + 1]);
                    unpack2(dt, od[2 * j], od[2 * j + 1]);
                    unpack2(gz, oz[2 * j], oz[2 * j + 1]);
                }
                const long long at = stg.x0 + (long long)tb * a.C + i * stg.xs;
                store4((T *)a.dx + at, ox, stg.have, sg.vec);
                store4((T *)a.ddt + at, od, stg.have, sg.vec);
                if (gated) store4((T *)a.dz + at, oz, stg.have, sg.vec);
            }
        }
        for (int e = tid; e < kTile * 2 * LN; e += K::threads) {
            const int j = e / (2 * LN), q = e / LN % 2, st = e % LN * kNS, t = tb + j;
            if (t < n && st < a.N) {
                f2 r0 = 0, r1 = 0;
#pragma unroll
                for (int u = 0; u < K::warps; ++u) {
                    const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(s.red + u * kTile * 2 * K::NP + e * kNS);
                    r0 = u ? add2(r0, v.x) : v.x;
                    r1 = u ? add2(r1, v.y) : v.y;
                }
                const long long plane = (long long)a.B * a.T * a.G * a.N;
                const int ct = (p.c0 - p.g * (a.C / a.G)) / K::width;
                float v[4];
                unpack2(r0, v[0], v[1]);
                unpack2(r1, v[2], v[3]);
                store_states(sg.bc + (2 * (long long)ct + q) * plane + (((long long)p.b * a.T + t) * a.G + p.g) * a.N, st,
                             a.N, v);
            }
        }
        __syncthreads();
    }
    // rows behind the sequence's end
    const long long row0 = (long long)p.b * a.T;
    for (long long e = (long long)count * K::pairs + tid; e < (long long)(t1 - t0) * K::width; e += K::threads) {
        const int t = t0 + (int)(e / K::width), cc = (int)(e % K::width);
        if (cc < p.nc) {
            const long long o = (row0 + t) * a.C + p.c0 + cc;
            ((T *)a.dx)[o] = ((T *)a.ddt)[o] = from_f<T>(0.f);
            if (gated) ((T *)a.dz)[o] = from_f<T>(0.f);
        }
    }
    // this block's parts of the sums over tokens
    const long long part = (long long)p.b * sg.segs + p.seg;
    if (live) {
        float v[4];
        unpack2(dA[0], v[0], v[1]);
        unpack2(dA[1], v[2], v[3]);
        if (count > 0 && (n - t0) % kSub != 0) {
            float last[kNS];
            load_states(sg.pA + (part * a.C + c) * a.N, n0, a.N, last);
#pragma unroll
            for (int k = 0; k < kNS; ++k) v[k] += last[k];
        }
        store_states(sg.pA + (part * a.C + c) * a.N, n0, a.N, v);
        unpack2(w[0], v[0], v[1]);
        unpack2(w[1], v[2], v[3]);
        if (p.seg == 0 && a.dstate_out) store_states(a.dstate_out + ((long long)p.b * a.C + c) * a.N, n0, a.N, v);
    }
    // the threads' four channels, thread tid those from 4 (tid % row) on
    float4 *end = reinterpret_cast<float4 *>(smem4);
    reinterpret_cast<ulonglong2 *>(end)[tid] = make_ulonglong2(dD[0], dD[1]);
    reinterpret_cast<ulonglong2 *>(end)[K::threads + tid] = make_ulonglong2(dbias[0], dbias[1]);
    __syncthreads();
    if (tid < p.nc) {
        float r0 = 0.f, r1 = 0.f;
        const float *f = reinterpret_cast<const float *>(end);
#pragma unroll
        for (int i = 0; i < K::threads / (K::width / 4); ++i) {
            r0 += f[i * K::width + tid];
            r1 += f[4 * K::threads + i * K::width + tid];
        }
        sg.pD[part * a.C + p.c0 + tid] = r0;
        sg.pbias[part * a.C + p.c0 + tid] = r1;
    }
}

// Joins the parts: the first blocks dC and dB over the channel tiles, 32 elements each with the
// block's 8 warps over the tiles; the others dA, dD and dbias over batch entries and segments.
constexpr int kJoin = 256;

template <typename T>
__global__ void __launch_bounds__(kJoin) scan_bwd_join(ScanArgs a, Seg sg, int tiles, int bc_blocks) {
    wait_for_stream();
    if ((int)blockIdx.x < bc_blocks) {
        __shared__ float red[2][kJoin / 32][32];
        const long long plane = (long long)a.B * a.T * a.G * a.N;
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const long long e = (long long)blockIdx.x * 32 + lane;
        int t, in_row;
        const int b = (int)split(split(e, a.G * a.N, in_row), a.T, t);
        float r0 = 0.f, r1 = 0.f;
        if (e < plane && t < seq_end(a.lengths, b, a.T)) {
#pragma unroll 4
            for (int i = warp; i < tiles; i += kJoin / 32) {
                r0 += sg.bc[2 * i * plane + e];
                r1 += sg.bc[(2 * i + 1) * plane + e];
            }
        }
        red[0][warp][lane] = r0;
        red[1][warp][lane] = r1;
        __syncthreads();
        if (warp < 2 && e < plane) {
            float r = 0.f;
#pragma unroll
            for (int w = 0; w < kJoin / 32; ++w) r += red[warp][w][lane];
            (warp == 0 ? (T *)a.dCm : (T *)a.dBm)[e] = from_f<T>(r);
        }
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
#pragma unroll 8
    for (int i = 0; i < a.B * sg.segs; ++i) r += p[i * step];
    *out = r;
}

int block_threads(int N) { return lanes_for(N) == 1 ? 64 : 128; }

// Segments of the backward, from the sizes alone: as many as keep all blocks on the GPU at once (two
// an SM), each of at least 32 tokens.
void bwd_segments(int B, int T, int C, int G, int N, int *segs, int *len) {
    const int width = block_threads(N) / lanes_for(N);
    const long long blocks = (long long)B * G * ((C / G + width - 1) / width);
    long long want = 2 * 148 / blocks;
    if (want > T / 32) want = T / 32;
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
    sg->ckpt = take((size_t)B * ((T + kSub - 1) / kSub) * C * kNS * lanes_for(N));
    sg->bc = take(tiles * 2 * B * T * G * N);
    sg->pA = take(parts * cn);
    sg->pD = take(parts * C);
    sg->pbias = take(parts * C);
    return (size_t)(p - (char *)ws);
}

template <typename T, int LN, bool PAD>
la_status bwd_pad(const ScanArgs &a, cudaStream_t st) {
    using K = Cfg<LN>;
    Seg sg;
    layout(a.B, a.T, a.C, a.G, a.N, a.ws, &sg);
    sg.vec = quad_rows<T>(a.C / a.G, a.x, a.dt_in, a.z, a.dy, a.dx, a.ddt, a.dz);
    sg.bvec = quad_rows<T>(a.N, a.Bm, a.Cm);
    const int tiles = (a.C / a.G + K::width - 1) / K::width;
    const dim3 grid((unsigned)((long long)a.B * sg.segs * a.G * tiles)), block(K::threads);
    la_status rc = LA_OK;
    if (sg.segs > 1) {
        rc = launch("selective_scan_bwd_ends", scan_bwd_ends<T, LN>, grid, block, K::smem, st, a, sg, tiles);
        if (rc != LA_OK) return rc;
    }
    rc = launch_pdl("selective_scan_bwd", scan_bwd_kernel<T, LN, PAD>, grid, block, K::smem, st, a, sg, tiles);
    if (rc != LA_OK) return rc;
    const long long plane = (long long)a.B * a.T * a.G * a.N, rest = (long long)a.C * (a.N + 2);
    const int bc_blocks = (int)((plane + 31) / 32);
    return launch_pdl("selective_scan_bwd_join", scan_bwd_join<T>, dim3((unsigned)(bc_blocks + (rest + kJoin - 1) / kJoin)),
                  dim3(kJoin), 0, st, a, sg, tiles, bc_blocks);
}

template <typename T, int LN>
la_status bwd_ln(const ScanArgs &a, cudaStream_t st) {
    return a.N == kNS * LN ? bwd_pad<T, LN, false>(a, st) : bwd_pad<T, LN, true>(a, st);
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

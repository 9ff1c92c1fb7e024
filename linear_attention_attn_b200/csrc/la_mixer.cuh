// la_mixer.cuh -- shared pieces of the operators around the recurrent token mixers (rotary
// positions, short causal convolution, selective scan, group normalisation): vector element I/O,
// activations, and the internal entry points that la_mixer_api.cu calls after its checks.
#pragma once

#include "la_internal.cuh"

namespace la {

// ------------------------------------------------------------ vector I/O --
// V neighbouring elements as one access of V * sizeof(T) bytes (the caller picks a V
// that the pointer's alignment and every stride allow, see vec_width).
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
    T v[V];
};
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Two 16-bit elements as they lie in a word, and back (one rounding each, to nearest even).
template <typename T> struct Pair16;
template <> struct Pair16<__half> {
    static __device__ __forceinline__ float2 widen(unsigned w) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    }
    static __device__ __forceinline__ unsigned narrow(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const unsigned *>(&h);
    }
};
template <> struct Pair16<__nv_bfloat16> {
    static __device__ __forceinline__ float2 widen(unsigned w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    static __device__ __forceinline__ unsigned narrow(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const unsigned *>(&h);
    }
};

template <int V, typename T>
__device__ __forceinline__ void stv(T *p, const float (&x)[V]) {
    if constexpr (sizeof(T) == 2 && V >= 2) {
        Pack<unsigned, V / 2> k;
#pragma unroll
        for (int i = 0; i < V / 2; ++i) k.v[i] = Pair16<T>::narrow(x[2 * i], x[2 * i + 1]);
        *reinterpret_cast<Pack<unsigned, V / 2> *>(p) = k;
    } else {
        Pack<T, V> k;
#pragma unroll
        for (int i = 0; i < V; ++i) k.v[i] = from_f<T>(x[i]);
        *reinterpret_cast<Pack<T, V> *>(p) = k;
    }
}
// The elements of a word, or of several.
template <int V, typename T, typename W>
__device__ __forceinline__ void widen(const W &words, float (&x)[V]) {
    if constexpr (sizeof(T) == 2 && V >= 2) {
        Pack<unsigned, V / 2> k;
        *reinterpret_cast<W *>(&k) = words;
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 f = Pair16<T>::widen(k.v[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    } else {
        Pack<T, V> k;
        *reinterpret_cast<W *>(&k) = words;
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = to_f(k.v[i]);
    }
}

// Widest access in elements, a power of two of at most 16 bytes, that divides `unit` (every
// offset is a multiple of it) and that all the given addresses are aligned to.
inline int vec_width(size_t elem, long long unit, uintptr_t address_bits) {
    int v = (int)(16 / elem);
    while (v > 1 && (unit % v != 0 || (address_bits & (v * elem - 1)) != 0)) v >>= 1;
    return v;
}

inline size_t elem_bytes(la_dtype dt) { return dt == LA_F32 ? 4 : 2; }
inline size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// ------------------------------------------------------- index arithmetic --
// idx / n and the remainder, in 32 bits where idx fits them (a 64-bit division is some 100
// instructions, more than many of these kernels spend on an element).
__device__ __forceinline__ long long split(long long idx, int n, int &rest) {
    if ((idx >> 32) == 0) {
        const unsigned q = (unsigned)idx / (unsigned)n;
        rest = (int)((unsigned)idx - q * (unsigned)n);
        return q;
    }
    const long long q = idx / n;
    rest = (int)(idx - q * n);
    return q;
}

// ------------------------------------------------------ dependent launches --
// A kernel launched by launch_pdl waits here for everything before it in the stream.
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// -------------------------------------------------- packed fp32 arithmetic --
// Two fp32 operations at once on a register pair.  Kernels that work on V neighbouring channels
// hold them as Lanes<V>: V / 2 pairs, or one float.
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 operations at once on a register pair.
typedef unsigned long long f2;
__device__ __forceinline__ f2 pack2(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(f2 v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 ex2_2(f2 v) {
    float a, b;
    unpack2(v, a, b);
    return pack2(ex2(a), ex2(b));
}

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ f2 both(float x) { return pack2(x, x); }

// The same operations by element type, float or pair.
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ f2 mul(f2 a, f2 b) { return mul2(a, b); }
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ f2 add(f2 a, f2 b) { return add2(a, b); }
__device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ f2 fma(f2 a, f2 b, f2 c) { return fma2(a, b, c); }

// ----------------------------------------------------------- activations --
// 1 / (1 + e^-x).  Relative error 2.4e-7 down to x = -3, 1e-6 at -20, 3.8e-6 at -85 (the argument's rounding
// grows with it, next to a result of e^x); below -87.3 the reciprocal is 0.  x sigma(x) is off by
// less than 1e-7 for every x below 0.
__device__ __forceinline__ float sigmoid_f(float x) { return rcp(1.f + ex2(x * -kLog2e)); }
__device__ __forceinline__ f2 sigmoid2(f2 x) {
    float a, b;
    unpack2(x, a, b);
    return pack2(sigmoid_f(a), sigmoid_f(b));
}
__device__ __forceinline__ float sigmoid(float x) { return sigmoid_f(x); }
__device__ __forceinline__ f2 sigmoid(f2 x) { return sigmoid2(x); }

template <int V> struct Lanes {
    typedef f2 E;
    static constexpr int n = V / 2;
    E e[n];
    static __device__ __forceinline__ E splat(float x) { return both(x); }
    __device__ __forceinline__ void set(const float (&v)[V]) {
#pragma unroll
        for (int i = 0; i < n; ++i) e[i] = pack2(v[2 * i], v[2 * i + 1]);
    }
    __device__ __forceinline__ void get(float (&v)[V]) const {
#pragma unroll
        for (int i = 0; i < n; ++i) unpack2(e[i], v[2 * i], v[2 * i + 1]);
    }
};
template <> struct Lanes<1> {
    typedef float E;
    static constexpr int n = 1;
    E e[1];
    static __device__ __forceinline__ E splat(float x) { return x; }
    __device__ __forceinline__ void set(const float (&v)[1]) { e[0] = v[0]; }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = e[0]; }
};

// V elements as they lie in memory, in whole words: a load that may be left out (zeros then) is not
// waited for before its values are used, as it would be if its elements were taken apart at once.
template <int BYTES> struct WordsOf;
template <> struct WordsOf<2> { typedef unsigned short W; static __device__ __forceinline__ W zero() { return 0; } };
template <> struct WordsOf<4> { typedef unsigned W; static __device__ __forceinline__ W zero() { return 0; } };
template <> struct WordsOf<8> { typedef uint2 W; static __device__ __forceinline__ W zero() { return make_uint2(0, 0); } };
template <> struct WordsOf<16> { typedef uint4 W; static __device__ __forceinline__ W zero() { return make_uint4(0, 0, 0, 0); } };
template <typename T, int V> struct Raw {
    typedef WordsOf<sizeof(T) * V> O;
    typename O::W w;
    __device__ __forceinline__ void load(const T *p, bool there = true) {
        w = O::zero();
        if (there) w = *reinterpret_cast<const typename O::W *>(p);
    }
    __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<typename O::W *>(p) = w; }
    __device__ __forceinline__ Lanes<V> lanes() const {
        float v[V];
        widen<V, T>(w, v);
        Lanes<V> r;
        r.set(v);
        return r;
    }
};
// An asynchronous copy of BYTES (4, 8 or 16) into the thread's own place in shared memory, zeros
// where `there` is false (nothing is read then), and the waits on the groups of them.
template <int BYTES>
__device__ __forceinline__ void copy_async(void *smem, const void *p, bool there) {
    const unsigned d = (unsigned)__cvta_generic_to_shared(smem);
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(d), "l"(p), "n"(BYTES), "r"(there ? BYTES : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT> __device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

template <int V, typename T>
__device__ __forceinline__ void ldv(const T *p, float (&x)[V]) {
    Raw<T, V> r;
    r.load(p);
    widen<V, T>(r.w, x);
}
template <int V, typename T>
__device__ __forceinline__ void store_lanes(T *p, const Lanes<V> &x) {
    float v[V];
    x.get(v);
    stv<V>(p, v);
}

// --------------------------------------------------- internal entry points --
struct RotaryArgs {
    const void *q, *k;               // k and ok null: the queries only
    void *oq, *ok;
    const float *freqs;              // [R / 2]
    const long long *positions;      // null: start + t
    long long start;
    int per_batch;                   // positions is [B, T] rather than [T]
    int B, H, Hk, T, D, R, interleaved;
    float magnitude, sign;           // sign -1: the inverse rotation
    la_dtype dt;
};
la_status rotary(const RotaryArgs &a, cudaStream_t st);

struct ConvArgs {
    const void *x, *dy, *state_in, *dstate_in;
    const float *w, *bias;
    const int *lengths;
    void *y, *state_out, *dx, *dstate_out;
    float *dw, *dbias;
    int B, T, C, W, silu;
    la_dtype dt;
    void *ws;
};
size_t conv_bwd_workspace(int B, int T, int C, int W, la_dtype dt);
la_status conv_fwd(const ConvArgs &a, cudaStream_t st);
la_status conv_bwd(const ConvArgs &a, cudaStream_t st);

struct ScanArgs {
    const void *x, *dt_in, *Bm, *Cm, *z, *dy;
    const float *A, *D, *dt_bias, *state_in, *dstate_in;
    const int *lengths;
    void *y, *dx, *ddt, *dBm, *dCm, *dz;
    float *state_out, *dstate_out, *dA, *dD, *ddt_bias;
    int B, T, C, G, N, softplus;
    la_dtype dt;
    void *ws;
};
size_t scan_fwd_workspace(int B, int T, int C, int G, int N);
size_t scan_bwd_workspace(int B, int T, int C, int G, int N);
la_status scan_fwd(const ScanArgs &a, cudaStream_t st);
la_status scan_bwd(const ScanArgs &a, cudaStream_t st);
la_status scan_step(const ScanArgs &a, cudaStream_t st);

struct NormArgs {
    const void *x, *dy;
    const float *gamma, *beta, *mean_in, *rstd_in;
    void *y, *dx;
    float *mean, *rstd, *dgamma, *dbeta;
    int B, T, C, G, silu;
    float eps;
    la_dtype dt;
    void *ws;
};
size_t norm_fwd_workspace(int B, int T, int C, int G, la_dtype dt);
size_t norm_bwd_workspace(int B, int T, int C, int G, la_dtype dt);
la_status norm_fwd(const NormArgs &a, cudaStream_t st);
la_status norm_bwd(const NormArgs &a, cudaStream_t st);

}  // namespace la

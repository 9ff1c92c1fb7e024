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

template <int V, typename T>
__device__ __forceinline__ void ldv(const T *p, float (&x)[V]) {
    const Pack<T, V> k = *reinterpret_cast<const Pack<T, V> *>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = to_f(k.v[i]);
}
template <int V, typename T>
__device__ __forceinline__ void stv(T *p, const float (&x)[V]) {
    Pack<T, V> k;
#pragma unroll
    for (int i = 0; i < V; ++i) k.v[i] = from_f<T>(x[i]);
    *reinterpret_cast<Pack<T, V> *>(p) = k;
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

// ----------------------------------------------------------- activations --
// 1 / (1 + e^-x).  For x below about -88 the exponential overflows to infinity and the result
// is 0; the relative error is that of the fast exponential, a few 2^-22 where |x| is a few units.
__device__ __forceinline__ float sigmoid_f(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

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

// Shared by the layer operators (conv.cu, norm.cu, scan_*.cu): strided token
// arrays, vector accesses, activations, packed-sequence lookup, column sums.
#pragma once

#include "../../include/gdn_layers.h"
#include "common.cuh"

namespace gdn {
namespace lay {

// A strided token array as the kernels take it (element strides).
template <class T>
struct View {
    T *p;
    long long b, h, t;
    __device__ __forceinline__ T *at(int bi, int hi, long long ti) const { return p + bi * b + hi * h + ti * t; }
};

template <class T>
inline View<T> view_of(const dn_view *v)
{
    View<T> r{nullptr, 0, 0, 0};
    if (v && v->data) {
        r.p = (T *)v->data;
        r.b = v->batch; r.h = v->head; r.t = v->time;
    }
    return r;
}

// Whether rows of a view can be moved `bytes` at a time (absent views can).
inline bool can_vector(const dn_view *v, int elem, int bytes)
{
    if (!v || !v->data) return true;
    const long long m = bytes / elem;
    return ((uintptr_t)v->data % bytes) == 0 && v->batch % m == 0 && v->head % m == 0 && v->time % m == 0;
}

template <int BYTES> struct RawOf;
template <> struct RawOf<2> { using type = unsigned short; };
template <> struct RawOf<4> { using type = unsigned int; };
template <> struct RawOf<8> { using type = uint2; };
template <> struct RawOf<16> { using type = uint4; };

// V consecutive elements, held as loaded (conversion to float when used).
template <class T, int V>
struct Vec {
    typename RawOf<sizeof(T) * V>::type raw;
    __device__ __forceinline__ void load(const T *p) { raw = *reinterpret_cast<const decltype(raw) *>(p); }
    __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<decltype(raw) *>(p) = raw; }
    __device__ __forceinline__ void zero() { raw = {}; }
    __device__ __forceinline__ void get(float (&f)[V]) const
    {
        T e[V];
        memcpy(e, &raw, sizeof(e));
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = ld_in(&e[i]);
    }
    __device__ __forceinline__ void set(const float (&f)[V])
    {
        T e[V];
#pragma unroll
        for (int i = 0; i < V; ++i) st_out(&e[i], f[i]);
        memcpy(&raw, e, sizeof(e));
    }
};

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + ex2(-kLog2e * x)); }

// d/dx of x sigmoid(x)
__device__ __forceinline__ float dsilu(float x, float s) { return s * fmaf(x, 1.f - s, 1.f); }

// softplus(x) = max(x, 0) + log1p(e), e = exp(-|x|) in (0, 1], and its derivative
// sigmoid(x).  log1p(e) = 2 atanh(s), s = e / (2 + e) <= 1/3, by the series
// 2 (s + s^3/3 + s^5/5 + ...): lg2(1 + e) would lose the small e of small steps
// (delta ~ 1e-3) to the rounding of 1 + e.  Terms to s^15: the first one left out
// is below 2 (1/3)^17 / 17 = 1e-9 absolute, 1.3e-9 of log1p(1).
__device__ __forceinline__ void softplus(float x, float &val, float &der)
{
    const float e = ex2(-kLog2e * fabsf(x));
    const float s = __fdividef(e, 2.f + e), q = s * s;
    float p = fmaf(q, 1.f / 15.f, 1.f / 13.f);
    p = fmaf(q, p, 1.f / 11.f);
    p = fmaf(q, p, 1.f / 9.f);
    p = fmaf(q, p, 1.f / 7.f);
    p = fmaf(q, p, 1.f / 5.f);
    p = fmaf(q, p, 1.f / 3.f);
    p = fmaf(q, p, 1.f);
    val = fmaf(2.f * s, p, fmaxf(x, 0.f));
    const float r = __fdividef(1.f, 1.f + e);
    der = x >= 0.f ? r : e * r;
    if (x != x) val = x;   // fmaxf drops a NaN
}

// The sequence that holds token t: the last s with cu[s] <= t (an empty sequence
// shares its offset with the next one and is passed over).  N where t is behind
// the last sequence.
__device__ __forceinline__ int seq_at(const int32_t *cu, int N, int t)
{
    if (N == 0 || t >= cu[N]) return N;
    int lo = 0, hi = N;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid;
    }
    return lo;
}

// Checked copy of the packed offsets into the workspace: all zero, and the status
// word flagged, unless cu[0] = 0, cu[N] = T and cu never falls.
cudaError_t check_offsets(const int32_t *cu, int N, int T, int32_t *out, uint32_t *status, cudaStream_t st);

// out[map(col)] = sum over p < P of part[p * n + col], col < n, in a fixed order.
// Columns are split into `kinds` runs of n / kinds: run k of width C goes to
// dst[k] with element stride step[k].
struct ColSum {
    int kinds;
    long long C;
    float *dst[6];
    int step[6];
};
cudaError_t col_sum(const float *part, long long P, const ColSum &c, cudaStream_t st);

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
int sm_count();

}  // namespace lay
}  // namespace gdn

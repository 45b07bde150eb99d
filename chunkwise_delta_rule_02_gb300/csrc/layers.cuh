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
        if constexpr (sizeof(T) == 2 && V % 2 == 0) {   // two conversions an instruction
            __nv_bfloat162 e[V / 2];
#pragma unroll
            for (int i = 0; i < V / 2; ++i) e[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            memcpy(&raw, e, sizeof(e));
        } else {
            T e[V];
#pragma unroll
            for (int i = 0; i < V; ++i) st_out(&e[i], f[i]);
            memcpy(&raw, e, sizeof(e));
        }
    }
};

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / x for x >= 1 (the plain division's care for denormal divisors is several instructions)
__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The argument of the exponential is rounded after the scaling, so that e^-x, and with it a sigmoid far below 0
// (and softplus), is off by up to about |x| 2^-24 of itself: 1.0e-6 measured for x sigmoid(x) at -20 and 3.8e-6 at -80,
// where the plain float32 form keeps 2e-7.  Of the gate's range that is the part where it is e^x small; a second
// multiply-add a value would take it away.
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + ex2(-kLog2e * x)); }

// d/dx of x sigmoid(x)
__device__ __forceinline__ float dsilu(float x, float s) { return s * fmaf(x, 1.f - s, 1.f); }

// Pairs of float32 in one instruction: these kernels run out of issue slots before
// they run out of the float32 pipe.
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<unsigned long long &>(r))
        : "l"(reinterpret_cast<unsigned long long &>(a)), "l"(reinterpret_cast<unsigned long long &>(b)));
    return r;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(reinterpret_cast<unsigned long long &>(r))
        : "l"(reinterpret_cast<unsigned long long &>(a)), "l"(reinterpret_cast<unsigned long long &>(b)),
          "l"(reinterpret_cast<unsigned long long &>(c)));
    return r;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<unsigned long long &>(r))
        : "l"(reinterpret_cast<unsigned long long &>(a)), "l"(reinterpret_cast<unsigned long long &>(b)));
    return r;
}

__device__ __forceinline__ float2 two(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2 ex2_2(float2 a) { return make_float2(ex2(a.x), ex2(a.y)); }

// softplus(x) = max(x, 0) + log1p(e), e = exp(-|x|) in (0, 1], and its derivative
// sigmoid(x).  log1p(e) = 2 atanh(s) = 2 s f(s^2), s = e / (2 + e) <= 1/3: lg2(1 + e)
// would lose the small e of small steps (delta ~ 1e-3) to the rounding of 1 + e.
// f(q) = atanh(sqrt q) / sqrt q = 1 + q/3 + q^2/5 + ... on [0, 1/9] by the polynomial of
// degree 4 that is least off relative to f (fitted by reweighted least squares): 8e-9.
// e is NaN where x is, so a NaN stays one although max drops it.
__device__ __forceinline__ void softplus(float2 x, float2 &val, float2 &der)
{
    const float2 e = ex2_2(mul2(make_float2(fabsf(x.x), fabsf(x.y)), two(-kLog2e)));
    const float2 u = add2(e, two(2.f));
    const float2 s = mul2(e, make_float2(rcp(u.x), rcp(u.y))), q = mul2(s, s);
    float2 p = fma2(q, two(0.14089517295360565f), two(0.13980233669281006f));
    p = fma2(q, p, two(0.200124591588974f));
    p = fma2(q, p, two(0.3333315849304199f));
    p = fma2(q, p, two(1.f));
    val = fma2(add2(s, s), p, make_float2(fmaxf(x.x, 0.f), fmaxf(x.y, 0.f)));
    const float2 r = make_float2(rcp(1.f + e.x), rcp(1.f + e.y));
    der = make_float2(x.x >= 0.f ? r.x : e.x * r.x, x.y >= 0.f ? r.y : e.y * r.y);
}

__device__ __forceinline__ float2 sigmoid2(float2 x)
{
    const float2 e = add2(ex2_2(mul2(x, two(-kLog2e))), two(1.f));
    return make_float2(rcp(e.x), rcp(e.y));
}

// N floats as pairs (a single one is paired with itself)
template <int N>
__device__ __forceinline__ float2 pair_at(const float (&v)[N], int i)
{
    return N == 1 ? two(v[0]) : make_float2(v[i], v[N == 1 ? 0 : i + 1]);
}

template <int N>
__device__ __forceinline__ void put_pair(float (&v)[N], int i, float2 a)
{
    v[i] = a.x;
    if (N > 1) v[N == 1 ? 0 : i + 1] = a.y;
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

// Checked copy of the packed offsets into the workspace, and the call's status word:
// all zero and flagged unless cu[0] = 0, cu[N] = T and cu never falls.
cudaError_t check_offsets(const int32_t *cu, int N, int T, int32_t *out, uint32_t *status, cudaStream_t st);

// Sums of partial results in a fixed order: out[map(col)] = sum over p < P of part[p * n + col],
// col < n.  Columns are split into `kinds` runs of n / kinds: run k of width C goes to dst[k]
// (null: nowhere) with element stride step[k].  Two such sums go in one launch.
struct ColSum {
    const float *part;
    long long P, C;
    int kinds;
    float *dst[5];
    int step[5];
};
cudaError_t col_sum(const ColSum &a, const ColSum *b, cudaStream_t st);

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
int sm_count();

}  // namespace lay
}  // namespace gdn

// Shared by the selective state space scan's kernels (scan_fwd.cu, scan_bwd.cu):
// geometry, the lane layout, packed float pairs, the sums over lanes.
//
// Per channel c (of D) with N states, delta = softplus(dt + dt_bias):
//     h_t[n] = exp(delta A[n]) h_{t-1}[n] + delta x B_t[n],  o_t = sum_n C_t[n] h_t[n] + D x
//
// Lane layout.  L lanes share a channel, S states each (L S = Np >= N, padded states
// have A = B = C = 0 and stay 0); 256 threads hold CH = 256 / L channels.  Splitting a
// channel's states over lanes gives L times the threads of one thread a channel, which
// a few thousand channels need to fill the SMs, and keeps 16-byte reads of B_t and C_t;
// the price, sums over the L lanes, is paid once for L tokens: the L partial sums of a
// lane are exchanged in a halving butterfly (L - 1 shuffles) that leaves token l's sum
// in lane l, instead of log2 L shuffles a token.
#pragma once

#include "layers.h"

namespace gdn {
namespace lay {

constexpr int kScanThreads = 256;
constexpr int kScanKeep = 16;      // tokens between kept states

struct ScanDims {
    int B, T, D, N, G, Dg;         // Dg = D / G channels a group
    int tiles;                     // channel tiles of a group
    int softplus;
    int K, seg;                    // time segments of a row and their length
    int Nseq;
    const int32_t *cu;             // checked offsets, or null
    const float *A, *Dskip, *bias, *h0;
};

template <class T>
struct ScanIo {
    View<const T> x, dt, b, c, z;
    View<T> y;
    float *hT, *keep;              // keep: state entering every 16th token, [B][ceil(T/16)][D][Np], or null
    float *segP, *segH;            // per segment: product of the decays, end state from zero [B][K][D][Np]
};

// ---- packed pairs: two float32 operations an instruction (issue slots, not the
// arithmetic pipe, are what the scan runs out of first)
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

__device__ __forceinline__ float2 two(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2 ex2_2(float2 a) { return make_float2(ex2(a.x), ex2(a.y)); }

// S consecutive floats (16-byte aligned) as pairs
template <int S>
__device__ __forceinline__ void load_pairs(float2 (&v)[S / 2], const float *p)
{
#pragma unroll
    for (int i = 0; i < S / 4; ++i) {
        const float4 q = reinterpret_cast<const float4 *>(p)[i];
        v[2 * i] = make_float2(q.x, q.y);
        v[2 * i + 1] = make_float2(q.z, q.w);
    }
}

template <int S>
__device__ __forceinline__ void store_pairs(float *p, const float2 (&v)[S / 2])
{
#pragma unroll
    for (int i = 0; i < S / 4; ++i)
        reinterpret_cast<float4 *>(p)[i] = make_float4(v[2 * i].x, v[2 * i].y, v[2 * i + 1].x, v[2 * i + 1].y);
}

// A lane's states of [..][D][N] arrays (N need not be a multiple of anything)
template <int S>
__device__ __forceinline__ void load_states(float2 (&v)[S / 2], const float *p, int n0, int N, bool live)
{
#pragma unroll
    for (int i = 0; i < S / 2; ++i) {
        v[i].x = live && n0 + 2 * i < N ? p[n0 + 2 * i] : 0.f;
        v[i].y = live && n0 + 2 * i + 1 < N ? p[n0 + 2 * i + 1] : 0.f;
    }
}

template <int S>
__device__ __forceinline__ void store_states(float *p, const float2 (&v)[S / 2], int n0, int N, bool live)
{
#pragma unroll
    for (int i = 0; i < S / 2; ++i) {
        if (live && n0 + 2 * i < N) p[n0 + 2 * i] = v[i].x;
        if (live && n0 + 2 * i + 1 < N) p[n0 + 2 * i + 1] = v[i].y;
    }
}

// v[0 .. L-1] of each of L neighbouring lanes -> the sum over the lanes of v[l] in lane l
template <int L>
__device__ __forceinline__ float lane_sum(float (&v)[L], int lane)
{
#pragma unroll
    for (int m = L / 2; m > 0; m >>= 1) {
        const bool up = lane & m;
#pragma unroll
        for (int k = 0; k < m; ++k) {
            const float send = up ? v[k] : v[k + m], mine = up ? v[k + m] : v[k];
            v[k] = mine + __shfl_xor_sync(0xffffffffu, send, m);
        }
    }
    return v[0];
}

// L and S by N; tokens of a tile; elements of a tile a thread moves
template <int L_, int S_>
struct ScanCfg {
    static constexpr int L = L_, S = S_, Np = L_ * S_, CH = kScanThreads / L_;
};

// Sequence starts and ends among the tile's tokens t0 .. t0+n-1 (n <= 32): bit masks,
// and for each such token its sequence.  Called by one whole warp.
__device__ __forceinline__ void tile_edges(const ScanDims &g, int b, int t0, int n, int *seq, uint32_t *masks)
{
    const int lane = threadIdx.x & 31, t = t0 + lane;
    bool st = false, en = false;
    if (lane < n && t < g.T) {
        int s = b;
        if (g.cu) {
            s = seq_at(g.cu, g.Nseq, t);
            if (s < g.Nseq) {
                st = g.cu[s] == t;
                en = g.cu[s + 1] == t + 1;
            }
        } else {
            st = t == 0;
            en = t == g.T - 1;
        }
        seq[lane] = s;
    }
    const uint32_t ms = __ballot_sync(0xffffffffu, st), me = __ballot_sync(0xffffffffu, en);
    if (lane == 0) {
        masks[0] = ms;
        masks[1] = me;
    }
}

// The state entering segment k: the segments before it, composed in order.  A product
// of 0 is a sequence start inside the segment: nothing from before it, not even an
// infinity, goes on.
template <int S>
__device__ __forceinline__ void carry_in(float2 (&h)[S / 2], const ScanDims &g, const float *segP, const float *segH, int b,
                                         int k, long long c, int n0, int Np)
{
    for (int j = 0; j < k; ++j) {
        const size_t at = (((size_t)b * g.K + j) * g.D + c) * Np + n0;
        float2 p[S / 2], e[S / 2];
        load_pairs<S>(p, segP + at);
        load_pairs<S>(e, segH + at);
#pragma unroll
        for (int i = 0; i < S / 2; ++i) {
            h[i].x = p[i].x == 0.f ? e[i].x : fmaf(p[i].x, h[i].x, e[i].x);
            h[i].y = p[i].y == 0.f ? e[i].y : fmaf(p[i].y, h[i].y, e[i].y);
        }
    }
}

struct ScanCall {
    const dn_scan_shape *s;
    const dn_scan_io *io;
    const dn_scan_grads *gr;
    int Nseq;
    const int32_t *cu;
    float *keep;
    char *ws;                      // behind the status word and the offsets
};

int scan_padded(int N);            // Np
size_t scan_fwd_bytes(const dn_scan_shape *s);
size_t scan_bwd_bytes(const dn_scan_shape *s);
cudaError_t scan_fwd(const ScanCall &c, cudaStream_t st);
cudaError_t scan_bwd(const ScanCall &c, cudaStream_t st);
cudaError_t scan_step(const ScanCall &c, cudaStream_t st);

ScanDims scan_dims(const ScanCall &c);

// Calls f(ScanCfg<L, S>{}) for the layout of N states.
template <class F>
cudaError_t scan_layout(int N, F f)
{
    if (N <= 4) return f(ScanCfg<1, 4>{});
    if (N <= 8) return f(ScanCfg<2, 4>{});
    if (N <= 16) return f(ScanCfg<4, 4>{});
    if (N <= 32) return f(ScanCfg<8, 4>{});
    if (N <= 64) return f(ScanCfg<16, 4>{});
    return f(ScanCfg<16, 8>{});
}

}  // namespace lay
}  // namespace gdn

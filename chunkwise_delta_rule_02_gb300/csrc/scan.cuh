// Shared by the selective state space scan's kernels (scan_fwd.cu, scan_bwd.cu):
// geometry, the lane layout, packed float pairs, the sums over lanes.
//
// Per channel c (of D) with N states, delta = softplus(dt + dt_bias):
//     h_t[n] = exp(delta A[n]) h_{t-1}[n] + delta x B_t[n],  o_t = sum_n C_t[n] h_t[n] + D x
//
// Lane layout.  L lanes share a channel, S states each (L S = Np >= N, padded states
// have A = B = C = 0 and stay 0), and a lane holds CT neighbouring channels; a block of NT
// threads holds CH = NT CT / L channels (NT 128: 554 us at 4 x 8192 tokens of 2048 channels, 256
// 582 us, 64 561 us, 32 629 us).  Splitting a channel's states over lanes gives the
// threads that a few thousand channels need to fill the SMs; the price, sums over the L
// lanes, is paid once for L tokens: the L partial sums of a lane are exchanged in a
// halving butterfly (L - 1 shuffles) that leaves token l's sum in lane l, instead of
// log2 L shuffles a token.
//
// What CT is for: B_t and C_t come from shared memory at 8 bytes a state, 2 cycles of the
// SM's read port for 16 bytes a lane (measured: 2.1 where neighbouring lanes read the same
// address, 4.0 where they do not, which is why a channel's lanes are 32 / L apart).  With one
// channel a lane that port, at 1 cycle a state and warp for B and C alone, is what binds: the
// exponentials and the multiply-adds take 1 cycle each.  Two channels halve it.
#pragma once

#include "layers.h"

namespace gdn {
namespace lay {

// Tokens between the states that the forward pass keeps for the backward, by the padded
// number of states (the backward's tiles are whole spans of it).
__host__ __device__ constexpr int keep_of(int Np) { return Np <= 32 ? 8 : 16; }

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
    float *hT, *keep;              // keep: state entering every keep_of(Np)-th token, [B][ceil(T / that)][D][Np] with keep_place's order in [D][Np], or null
    float *segP, *segH;            // per segment: product of the decays (kCut: a sequence starts in it), end state from zero [B][K][D][Np]
};

// exp(delta A) of two states, a2 = A log2 e.  ex2.approx rounds towards zero rather than to the
// nearest: its results lie 0.1 .. 0.4 of 2^-24 low for arguments in [-0.125, 0] (0.85 below -0.25),
// the same way for every token, which a state that remembers a thousand tokens adds up.  A shift of
// the argument that raises results by 0.25 of 2^-24, in the multiplication that is there anyway,
// centres them: dA of 8 x 4096 tokens is then off by 1.4e-6 instead of 2.4e-6, of 3001 tokens in
// float32 by 0.6e-6 instead of 1.4e-6.
constexpr float kDecayUp = 0.25f / 16777216.f * kLog2e;
__device__ __forceinline__ float2 decay2(float delta, float2 a2) { return ex2_2(fma2(two(delta), a2, two(kDecayUp))); }

// S consecutive floats (aligned to them) as pairs
template <int S>
__device__ __forceinline__ void load_pairs(float2 (&v)[S / 2], const float *p)
{
    if constexpr (S == 2) {
        v[0] = *reinterpret_cast<const float2 *>(p);
    } else {
#pragma unroll
        for (int i = 0; i < S / 4; ++i) {
            const float4 q = reinterpret_cast<const float4 *>(p)[i];
            v[2 * i] = make_float2(q.x, q.y);
            v[2 * i + 1] = make_float2(q.z, q.w);
        }
    }
}

template <int S>
__device__ __forceinline__ void store_pairs(float *p, const float2 (&v)[S / 2])
{
    if constexpr (S == 2) {
        *reinterpret_cast<float2 *>(p) = v[0];
    } else {
#pragma unroll
        for (int i = 0; i < S / 4; ++i)
            reinterpret_cast<float4 *>(p)[i] = make_float4(v[2 * i].x, v[2 * i].y, v[2 * i + 1].x, v[2 * i + 1].y);
    }
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

// v[0 .. L-1] of each of a channel's L lanes (32 / L apart) -> the sum over them of v[l] in lane l
template <int L>
__device__ __forceinline__ float lane_sum(float (&v)[L], int lane)
{
    constexpr int M = 32 / L;
#pragma unroll
    for (int m = L / 2; m > 0; m >>= 1) {
        const bool up = lane & (m * M);
#pragma unroll
        for (int k = 0; k < m; ++k) {
            const float send = up ? v[k] : v[k + m], mine = up ? v[k + m] : v[k];
            v[k] = mine + __shfl_xor_sync(0xffffffffu, send, m * M);
        }
    }
    return v[0];
}

// TT: tokens of a tile; NT: threads of a block
template <int L_, int S_, int CT_, int TT_ = 16, int NT_ = 256>
struct ScanCfg {
    static constexpr int L = L_, S = S_, CT = CT_, TT = TT_, NT = NT_, M = 32 / L_, Np = L_ * S_;
    static constexpr int CH = NT / L_ * CT_;                             // channels of a block
    static constexpr int EPT = TT * CH / NT;                             // a tile's elements a thread moves
    static constexpr int VEC = EPT < 4 ? EPT : 4;
    static constexpr int NBC = (TT * Np + NT - 1) / NT;                  // elements of B (and of C) a thread moves
    static constexpr int RS = CH + M * CT_;   // row of a padded [token][channel] array: L rows of M CT channels, no bank twice
};

// Where a lane's S states of channel cg of a group lie among a token's kept states: the channels that
// one warp holds two a lane in the order of its lanes, so that a warp's access is one run of memory
// (in [channel][state] order 8 neighbouring lanes' 16 bytes touch 8 lines: the forward pass of 4 x 4096
// tokens of 2048 channels took 219 us instead of 187, the backward of 8 x 4096 1632 us instead of 1553).
// Channels behind the last such set keep the plain order.
template <class Cfg>
__device__ __forceinline__ unsigned keep_place(const ScanDims &g, int grp, int cg, int l)
{
    constexpr int L = Cfg::L, S = Cfg::S, M = Cfg::M, Np = Cfg::Np;
    const int first = cg & ~(2 * M - 1), e = cg & 1, m = (cg - first) >> 1;
    const int in = first + 2 * M <= g.Dg ? first * Np + ((e * L + l) * M + m) * S : cg * Np + l * S;
    return (unsigned)grp * g.Dg * Np + in;
}

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

// Time segments of a pass whose blocks are `tiles` a segment: the K that leaves the busiest SM
// the least to do.  An SM runs R blocks at once at full speed and n < R of them at
// 0.6 + 0.4 n / R of it; the first pass (all but one segment, R1 at once) does w1 of the main
// pass's work a token; a block's start costs as much as 8 tokens.  K = 1 has no first pass.
// At 4 x 8192 tokens of 2048 channels (128 tiles) this says 11714, 12850, 12039, 11283, 11500, 11289,
// 11426, 11514 (in tokens) for K = 1, 4, 7, 8, 9, 14, 19, 28, and the forward pass took 681, 644, 595, 560, 564,
// 553, 553, 552 us: ratios within 8 % from 3 segments on (12, 16 and 24 are the worst), the uncut pass 15 % too cheap.
inline int plan_segments(long long tiles, int T, int R, int R1, double w1)
{
    if (T <= 0) return 1;   // no tokens: nothing to cut (and no length to divide by)
    const int sms = sm_count();
    auto busiest = [&](long long blocks, int r) {   // rounds of the SM with the most blocks, in blocks at full speed
        const long long m = (blocks + sms - 1) / sms, full = m / r * r, n = m - full;
        return (double)full + (n ? (double)n / (0.6 + 0.4 * (double)n / r) : 0.0);
    };
    int best = 1;
    double least = 0.0;
    for (int k = 1; k <= 64 && (k == 1 || T / k >= 64); ++k) {
        const int len = ((T + k - 1) / k + 15) / 16 * 16, used = (T + len - 1) / len;
        const double cost = (len + 8) * (busiest(tiles * used, R) + (used > 1 ? w1 * busiest(tiles * (used - 1), R1) : 0.0));
        if (k == 1 || cost < 0.98 * least) {
            best = k;
            least = cost;
        }
    }
    return best;
}

// In the place of a segment's decay product: a sequence starts in the segment.  A product is never
// negative, and is 0 wherever it underflows, which a few tokens of a fast decay are enough for.
constexpr float kCut = -1.f;

// Composes the K segments of every (row, channel, state) in place: segH[k] becomes what
// enters segment k, from the segments before it (FWD) or behind it.  Nothing from before a
// sequence start, not even an infinity or NaN, goes on; through any other segment these
// do, as they do in the recurrence, whose decays of single tokens are not 0 where their product is.
// Segment k of the last one in that order is never read.
template <bool FWD>
__global__ void __launch_bounds__(128) k_scan_carry(const float *__restrict__ segP, float *segH, int K, long long per, long long all)
{
    const long long i = blockIdx.x * 128ll + threadIdx.x;   // (row, channel, state), per = channels x states of a row
    if (i >= all) return;
    const size_t at = (size_t)(i / per) * K * per + i % per;
    float h = 0.f;
    constexpr int U = 8;
    for (int k0 = 0; k0 < K; k0 += U) {
        float p[U], e[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = FWD ? k0 + u : K - 1 - k0 - u;
            if (k0 + u < K - 1) {
                p[u] = segP[at + k * per];
                e[u] = segH[at + k * per];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = FWD ? k0 + u : K - 1 - k0 - u;
            if (k0 + u < K) {
                segH[at + k * per] = h;
                if (k0 + u < K - 1) h = p[u] == kCut ? e[u] : p[u] == 0.f ? (isfinite(h) ? 0.f : h) + e[u] : fmaf(p[u], h, e[u]);
            }
        }
    }
}

template <bool FWD>
inline void scan_carry(const ScanDims &g, const float *segP, float *segH, int Np, cudaStream_t st)
{
    const long long per = (long long)g.D * Np, all = g.B * per;
    k_scan_carry<FWD><<<(unsigned)((all + 127) / 128), 128, 0, st>>>(segP, segH, g.K, per, all);
}

// (delta, delta x) of CT neighbouring channels
template <int CT>
__device__ __forceinline__ void load_steps(float (&dl)[CT], float (&dx)[CT], const float2 *p)
{
    if constexpr (CT == 1) {
        dl[0] = p->x;
        dx[0] = p->y;
    } else {
#pragma unroll
        for (int i = 0; i < CT / 2; ++i) {
            const float4 q = reinterpret_cast<const float4 *>(p)[i];
            dl[2 * i] = q.x; dx[2 * i] = q.y; dl[2 * i + 1] = q.z; dx[2 * i + 1] = q.w;
        }
    }
}

// CT neighbouring floats
template <int CT>
__device__ __forceinline__ void load_ct(float (&v)[CT], const float *p)
{
    Vec<float, CT> q;
    q.load(p);
    q.get(v);
}

template <int CT>
__device__ __forceinline__ void store_ct(float *p, const float (&v)[CT])
{
    Vec<float, CT> q;
    q.set(v);
    q.store(p);
}

// N neighbouring floats, 16 bytes at a time where N allows
template <int N>
__device__ __forceinline__ void load_wide(float (&v)[N], const float *p)
{
    constexpr int Q = N < 4 ? N : 4;
#pragma unroll
    for (int i = 0; i < N; i += Q) {
        float q[Q];
        load_ct<Q>(q, p + i);
#pragma unroll
        for (int u = 0; u < Q; ++u) v[i + u] = q[u];
    }
}

template <int N>
__device__ __forceinline__ void store_wide(float *p, const float (&v)[N])
{
    constexpr int Q = N < 4 ? N : 4;
#pragma unroll
    for (int i = 0; i < N; i += Q) {
        float q[Q];
#pragma unroll
        for (int u = 0; u < Q; ++u) q[u] = v[i + u];
        store_ct<Q>(p + i, q);
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

// Calls f(ScanCfg<...>{}) for the layout of N states: the forward pass's, and the backward
// pass's (the same Np).
template <class F>
cudaError_t fwd_layout(int N, F f)
{
    if (N <= 8) return f(ScanCfg<4, 2, 2, 16, 128>{});
    if (N <= 16) return f(ScanCfg<4, 4, 2, 16, 128>{});
    if (N <= 32) return f(ScanCfg<8, 4, 2, 16, 128>{});
    if (N <= 64) return f(ScanCfg<16, 4, 1, 16, 128>{});
    return f(ScanCfg<16, 8, 1, 16, 128>{});
}

template <class F>
cudaError_t bwd_layout(int N, F f)
{
    if (N <= 8) return f(ScanCfg<4, 2, 2, 16, 128>{});
    if (N <= 16) return f(ScanCfg<4, 4, 2, 16, 128>{});
    if (N <= 32) return f(ScanCfg<8, 4, 2, 16, 128>{});
    if (N <= 64) return f(ScanCfg<16, 4, 1, 16, 128>{});
    return f(ScanCfg<16, 8, 1, 16, 128>{});
}

}  // namespace lay
}  // namespace gdn

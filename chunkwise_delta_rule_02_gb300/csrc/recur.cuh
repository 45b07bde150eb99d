// Shared by the gated linear recurrence's kernels (recur_fwd.cu, recur_bwd.cu):
// geometry, the gates, the pieces of the recurrence and their exchange.
//
//     m = c softplus(lam) sigmoid(rg + rg_bias),  a = exp(-m),  s = sqrt(1 - a^2)
//     h_t = a_t h_{t-1} + s_t u_t,  u = sigmoid(ig + ig_bias) x,  y = z ? h silu(z) : h
//
// Layout.  A lane holds two neighbouring channels of a run of kRun tokens; a warp holds Q runs one after
// another of 64 / Q channels (Q = 2 or 4 where wider tiles would leave SMs idle), a block W warps, a
// cluster up to 8 blocks.  A run is a linear map h -> A h + H of what enters it; the runs of a warp exchange
// their maps by shuffles, a block's warps through shared memory, the cluster's blocks through each
// other's shared memory, and every thread then steps through its run.  So each input is read once whatever
// the number of rows: splitting the time axis over blocks costs a barrier a step, and no second pass
// over the inputs.
//
// The inputs of two steps lie in shared memory, filled by TMA (a box of 64 / Q channels and the block's tokens an
// array): a step's are in registers when its maps are exchanged, and the barrier there frees their place for the
// step after the next.  Of arrays that a tensor map cannot describe (rows that do not start at 16 bytes) every aligned 16 bytes that
// hold an element of a row are copied asynchronously, and read from where the row begins in them (by single words and elements before:
// 8 x 4096 tokens of 2047 channels, bf16 forward 591 us, backward 765, now 241 and 418; float32 527 and 839, now 271 and 469).
#pragma once

#include <stdlib.h>

#include <type_traits>

#include "layers.h"
#include "sm100.cuh"

namespace gdn {
namespace lay {

constexpr int kRun = 8;                       // tokens of a lane and step (and between kept states)
constexpr int kMaxCluster = 8;
constexpr float kNan = __builtin_nanf("");
constexpr long long kRecurBudget = 4000000000LL;   // clock cycles (about 2 s) for any one wait
constexpr long long kHookBudget = 2000000LL;       // the same (about 1 ms) with a test hook set (recur_dims)

enum { kTma, kChunks };                       // how inputs get to shared memory: boxes, or 16 bytes a lane

// Warps of a block by the type's bytes, blocks that an SM holds.  bf16 forward: 12 warps twice, what 80 registers allow (4 x 8192
// tokens of 2048 channels with the output gate, measured side by side: 148 us; 8 warps three times 157, 16 warps 186).  Backward: 6
// warps twice at 160 registers (training step of 8 x 4096 tokens, likewise: 437 us; 4 warps three times 459; runs of 4 tokens,
// 8 warps twice: 436, with twice the kept states).  float32 backward: 4 warps twice, at 160 registers where rows come by boxes (4 x 4096 tokens
// of 1000 channels 114 us, 5 warps 139) and 250 where they come in pieces.  Rows that come in whole 16 bytes (kChunks) leave room for fewer of them (bf16 forward, 2 x 4096 tokens of 1001
// channels: 8 warps 54 us, 9, which is one block an SM, 72).
__host__ __device__ constexpr int fwd_warps(int bytes, int Q, int mode)
{
    return mode == kTma ? (bytes == 2 ? 12 : 6) : bytes == 2 ? (Q == 4 ? 8 : 10) : Q == 4 ? 5 : 6;
}
__host__ __device__ constexpr int bwd_warps(int bytes) { return bytes == 2 ? 6 : 4; }
// Bytes of an array's place: W warps' runs
__host__ __device__ constexpr int place_bytes(int W, int Q, int mode, int bytes) { return W * kRun * (64 * bytes + (mode == kChunks ? 16 * Q : 0)); }
constexpr int kFwdResident = 2, kBwdResident = 2;


struct RecurDims {
    int B, T, D, Nseq, tiles, CL, Q;   // tiles: channel tiles of a row; CL: blocks that share a row's tokens
    float c;
    const int32_t *cu;             // checked offsets, or null
    const float *lam, *rbias, *ibias, *h0;
    uint32_t *status;
    long long budget;              // of a wait
    int short_in, short_map;       // test hooks: steps from which on 16 bytes too many are waited for, of inputs, of maps
};

enum { kX, kRg, kIg, kZ, kDy, kArrays };

template <class T>
struct RecurIo {
    View<const T> in[kArrays];     // x, rg, ig, z or null, dy
    View<T> out[4];                // forward: y at kX; backward: dx, drg, dig, dz
    float *hT, *keep;              // keep: state entering every kRun-th token, [B][ceil(T / kRun)][D], or null
    const float *dhT;
    float *dh0, *part;             // part: [B][CL][3][D] sums of dlam, drg_bias, dig_bias
};

struct RecurMaps {
    CUtensorMap in[kArrays], kept;   // kept: the kept states, backward
};

struct RecurCall {
    const dn_recur_shape *s;
    const dn_recur_io *io;
    const dn_recur_grads *gr;
    int Nseq;
    const int32_t *cu;
    uint32_t *status;
    float *keep, *part;
};

struct RecurPlan {
    int Q, CL;
};
RecurPlan recur_plan(const dn_recur_shape *s, bool bwd);
cudaError_t recur_fwd(const RecurCall &c, cudaStream_t st);
cudaError_t recur_bwd(const RecurCall &c, cudaStream_t st);
cudaError_t recur_step(const RecurCall &c, cudaStream_t st);

inline RecurDims recur_dims(const RecurCall &c, bool bwd)
{
    RecurDims g;
    g.B = c.s->B; g.T = c.s->T; g.D = c.s->D; g.c = c.s->c; g.Nseq = c.Nseq;
    const RecurPlan p = recur_plan(c.s, bwd);
    g.Q = p.Q;
    g.CL = p.CL;
    g.tiles = (g.D + 64 / p.Q - 1) / (64 / p.Q);
    g.cu = c.cu;
    g.lam = c.io->lam; g.rbias = c.io->rg_bias; g.ibias = c.io->ig_bias; g.h0 = c.io->h0;
    g.status = c.status;
    // Test hooks (failure detection): with GDN_DEBUG_WITHHOLD_INPUTS=n, GDN_DEBUG_WITHHOLD_MAP=n a block waits from step n on for 16 bytes
    // of inputs (where they come by TMA), of its cluster's maps, that nobody sends; the wait runs out after about 1 ms.
    auto hook = [](const char *name) {
        const char *v = getenv(name);
        return v && v[0] ? atoi(v) : 0x7fffffff;
    };
    g.short_in = hook("GDN_DEBUG_WITHHOLD_INPUTS");
    g.short_map = hook("GDN_DEBUG_WITHHOLD_MAP");
    g.budget = g.short_in != 0x7fffffff || g.short_map != 0x7fffffff ? kHookBudget : kRecurBudget;
    return g;
}

__device__ __forceinline__ float rsq(float x)
{
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float2 sub2(float2 a, float2 b)
{
    float2 r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<unsigned long long &>(r))
        : "l"(reinterpret_cast<unsigned long long &>(a)), "l"(reinterpret_cast<unsigned long long &>(b)));
    return r;
}

// sigmoid(x + bias), bias given as -bias log2 e
__device__ __forceinline__ float2 gate(float2 x, float2 nb)
{
    const float2 e = add2(ex2_2(fma2(x, two(-kLog2e), nb)), two(1.f));
    return make_float2(rcp(e.x), rcp(e.y));
}

// Two channels' parameters: km = c softplus(lam), biases times -log2 e; dk = sigmoid(lam) / softplus(lam), the factor from
// sum q to dlam (1, its limit, where softplus underflows).
struct RecurParams {
    float2 km, rb, ib;
    __device__ __forceinline__ void load(const RecurDims &g, int c, bool in0, bool in1, float2 *dk = nullptr)
    {
        const float2 lam = make_float2(in0 ? g.lam[c] : 0.f, in1 ? g.lam[c + 1] : 0.f);
        float2 sp, der;
        softplus(lam, sp, der);
        km = mul2(sp, two(g.c));
        rb = make_float2(in0 && g.rbias ? -kLog2e * g.rbias[c] : 0.f, in1 && g.rbias ? -kLog2e * g.rbias[c + 1] : 0.f);
        ib = make_float2(in0 && g.ibias ? -kLog2e * g.ibias[c] : 0.f, in1 && g.ibias ? -kLog2e * g.ibias[c + 1] : 0.f);
        if (dk) *dk = make_float2(sp.x == 0.f ? 1.f : der.x / sp.x, sp.y == 0.f ? 1.f : der.y / sp.y);
    }
    // Whether a decay of a warp's channels can be further from 1 than the series below serves (m <= km)
    __device__ __forceinline__ bool far() const;
};

// a = exp(-m), y = 1 - a^2 and rs = 1 / sqrt(y).  A decay close to 1, the usual one, leaves nothing of 1 - a^2 in
// float32 when a is rounded first, and a bias of ex2.approx adds up over the thousand tokens that such a state remembers:
// below kSmall both come from e = 1 - exp(-m) by its power series to m^7 (next term: 2e-8 of e at 0.35), a = 1 - e rounded
// once, y = e (1 + a).  m = 0 gives a = 1, y = 0 and a finite rs, so that m rs = 0, its limit.  FAR: an m may not be below it,
// which c softplus(lam), its bound, says for a warp's channels once.
constexpr float kSmall = 0.35f;
__device__ __forceinline__ bool RecurParams::far() const { return __any_sync(0xffffffffu, !(km.x < kSmall && km.y < kSmall)); }

template <bool FAR>
__device__ __forceinline__ void decay_of(float2 m, float2 &a, float2 &y, float2 &rs)
{
    float2 p = fma2(m, two(1.f / 5040.f), two(-1.f / 720.f));
    p = fma2(m, p, two(1.f / 120.f));
    p = fma2(m, p, two(-1.f / 24.f));
    p = fma2(m, p, two(1.f / 6.f));
    p = fma2(m, p, two(-0.5f));
    float2 e = fma2(mul2(m, m), p, m);
    a = sub2(two(1.f), e);
    if constexpr (FAR) {
        const float2 far = ex2_2(mul2(m, two(-kLog2e)));
        if (!(m.x < kSmall)) {
            a.x = far.x;
            e.x = 1.f - far.x;
        }
        if (!(m.y < kSmall)) {
            a.y = far.y;
            e.y = 1.f - far.y;
        }
    }
    y = fma2(e, a, e);
    rs = make_float2(rsq(fmaxf(y.x, 1e-37f)), rsq(fmaxf(y.y, 1e-37f)));
}

// The map of a stretch of tokens, h -> A h + H.  CUT: sequences may start (end) in it, and one that does lets nothing
// through: A is negative, which products of decays are not.  Products are held at the smallest normal number: no finite state
// notices (1e-38 of it goes through where less would), and an infinity or a NaN, which the recurrence's single decays let
// through, is not multiplied with 0.
constexpr float kLeast = 1.17549435e-38f;

template <bool CUT>
__device__ __forceinline__ float2 pass(float2 A, float2 H, float2 h)
{
    const float2 v = fma2(A, h, H);
    return CUT ? make_float2(A.x < 0.f ? H.x : v.x, A.y < 0.f ? H.y : v.y) : v;
}
// first (A, H), then (A2, H2)
template <bool CUT>
__device__ __forceinline__ void then(float2 &A, float2 &H, float2 A2, float2 H2)
{
    H = pass<CUT>(A2, H2, H);
    const float2 v = mul2(A, A2);
    auto one = [](float a, float a2, float v) { return CUT && (a < 0.f || a2 < 0.f) ? -1.f : fmaxf(v, kLeast); };
    A = make_float2(one(A.x, A2.x, v.x), one(A.y, A2.y, v.y));
}

__device__ __forceinline__ float2 load2(const float *p, bool in0, bool in1) { return make_float2(in0 ? p[0] : 0.f, in1 ? p[1] : 0.f); }
__device__ __forceinline__ void store2(float *p, float2 v, bool in0, bool in1)
{
    if (in0) p[0] = v.x;
    if (in1) p[1] = v.y;
}

__device__ __forceinline__ int cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return (int)r;
}

// The end of a cluster's block: it leaves when all of them have stopped storing.  Whoever has all maps knows that nothing is on its way
// to it; one that gave up waiting for them (`lost`) leaves a store in flight a thousand times the time that it takes.
__device__ __forceinline__ void leave_cluster(bool lost)
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (lost)
        for (const long long t0 = clock64(); clock64() - t0 < 1000000;) {}
}

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// 16 bytes into the shared memory of the cluster's block `rank`, at this block's address `dst`, counted by its barrier `bar`
__device__ __forceinline__ void remote_store(const float4 *dst, const uint64_t *bar, int rank, float4 v)
{
    asm volatile(
        "{\n\t.reg .b32 a, b;\n\tmapa.shared::cluster.u32 a, %0, %2;\n\tmapa.shared::cluster.u32 b, %1, %2;\n\t"
        "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [a], {%3, %4, %5, %6}, [b];\n\t}" ::"r"(sm100::smem_u32(dst)),
        "r"(sm100::smem_u32(bar)), "r"(rank), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
        : "memory");
}

// Bounded wait as sm100::mbar_wait, acquiring what the cluster's blocks stored
__device__ __forceinline__ bool cluster_wait(uint64_t *bar, uint32_t parity, long long budget)
{
    long long t0 = 0;
    for (int i = 0;; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(sm100::smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        if (i == 0) t0 = clock64();
        else if (clock64() - t0 > budget) return false;
    }
}

__device__ __forceinline__ void box_load(void *dst, const CUtensorMap *map, uint64_t *bar, int c, int t, int b)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            sm100::smem_u32(dst)),
        "l"((uint64_t)map), "r"(sm100::smem_u32(bar)), "r"(c), "r"(t), "r"(b)
        : "memory");
}

__host__ __device__ constexpr int recur_block_bytes(int CL, int Q) { return CL > 1 ? 2 * CL * (32 / Q) * 16 : 0; }

template <int W, int Q>
struct RecurShared {
    float4 warp[2][W][32 / Q];
    float2 carry[2][32 / Q];
    uint64_t bar[4];               // the inputs of a step are there; behind those: the cluster's maps are
};

// The maps of the runs of step `st`, exchanged: (A, H) of this thread's run in, what enters it out (the state before it in the
// order of the pass, BACK: from the last run to the first).  What entered the step is `carry` in a cluster, and becomes what leaves
// it; a block alone has it in shared memory, where the step's last run leaves it (leave()).  `rank` is the block's place in the
// cluster.  Maps of two steps have places of their own, so that one barrier a step suffices: a block stores its map into the others
// behind it, and they their next ones only when they have all of this step's, so that nobody overwrites what is still read.
// `block`: [2][CL][32 / Q] of the cluster's blocks.  `freed` is called behind the barrier.
// lost: the wait for the maps ran out, now or before.  The barrier that counts them is in the middle of its phase then, and neither
// it nor another block's is touched again; what enters the run and leaves the step is NaN.
template <int W, int Q, bool CUT, bool BACK, class F>
__device__ __forceinline__ float2 exchange(RecurShared<W, Q> &sm, float4 *block, int st, int CL, int rank, float2 A, float2 H, float2 &carry,
                                           bool &lost, const RecurDims &g, F freed)
{
    const int par = st & 1;
    constexpr int L = 32 / Q;
    const int lane = threadIdx.x & 31, l = lane % L, warp = threadIdx.x >> 5;
    const int mine = BACK ? W - 1 - warp : warp, at = BACK ? CL - 1 - rank : rank, q = BACK ? Q - 1 - lane / L : lane / L;
    float2 pA = two(1.f), pH = two(0.f);   // of what lies before this run in its warp
    if constexpr (Q > 1) {
        auto before = [&](float2 v, int d) {
            return BACK ? make_float2(__shfl_down_sync(0xffffffffu, v.x, d * L), __shfl_down_sync(0xffffffffu, v.y, d * L))
                        : make_float2(__shfl_up_sync(0xffffffffu, v.x, d * L), __shfl_up_sync(0xffffffffu, v.y, d * L));
        };
#pragma unroll
        for (int d = 1; d < Q; d *= 2) {
            float2 eA = before(A, d), eH = before(H, d);
            if (q >= d) {
                then<CUT>(eA, eH, A, H);
                A = eA;
                H = eH;
            }
        }
        const float2 eA = before(A, 1), eH = before(H, 1);
        if (q > 0) {
            pA = eA;
            pH = eH;
        }
    }
    if (q == Q - 1) sm.warp[par][mine][l] = make_float4(A.x, A.y, H.x, H.y);
    __syncthreads();
    freed();
    float2 h;
    if (Q < 4 || CL == 1) {   // wider tiles are never shared (recur_plan)
        h = sm.carry[par][l];
#pragma unroll 4
        for (int w = 0; w < mine; ++w) {
            const float4 m = sm.warp[par][w][l];
            h = pass<CUT>(make_float2(m.x, m.y), make_float2(m.z, m.w), h);
        }
    } else {
        if (threadIdx.x == 0 && !lost) sm100::mbar_expect_tx(&sm.bar[2 + par], (CL * L + (st >= g.short_map)) * 16);
        float2 wA = two(1.f), wH = two(0.f);   // of the warps before this one
#pragma unroll 4
        for (int w = 0; w < mine; ++w) {
            const float4 m = sm.warp[par][w][l];
            then<CUT>(wA, wH, make_float2(m.x, m.y), make_float2(m.z, m.w));
        }
        if (mine == W - 1) {   // the last one tells all blocks the whole
            const float4 m = sm.warp[par][W - 1][l];
            float2 oA = wA, oH = wH;
            then<CUT>(oA, oH, make_float2(m.x, m.y), make_float2(m.z, m.w));
            if (lane < L && !lost)
                for (int k = 0; k < CL; ++k) remote_store(block + (par * CL + at) * L + l, &sm.bar[2 + par], k, make_float4(oA.x, oA.y, oH.x, oH.y));
            __syncwarp();
        }
        if (lost || !cluster_wait(&sm.bar[2 + par], (uint32_t)(st >> 1) & 1u, g.budget)) {
            if (!lost) raise_status(g.status, kStatusTimeout);
            lost = true;
        }
        h = carry;
        for (int k = 0; k < CL; ++k) {
            if (k == at) h = carry;
            const float4 m = block[(par * CL + k) * L + l];
            carry = pass<CUT>(make_float2(m.x, m.y), make_float2(m.z, m.w), carry);
        }
        h = pass<CUT>(wA, wH, h);
        if (lost) h = carry = two(kNan);
    }
    return Q > 1 ? pass<CUT>(pA, pH, h) : h;
}

// What leaves the step's last run, for the next step
template <int W, int Q, bool BACK>
__device__ __forceinline__ void leave(RecurShared<W, Q> &sm, int par, float2 h)
{
    constexpr int L = 32 / Q;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x >> 5 == (BACK ? 0 : W - 1) && lane / L == (BACK ? 0 : Q - 1)) sm.carry[par ^ 1][lane % L] = h;
}

// Which of this lane's run's tokens t .. t+n-1 (n <= kRun) start and which end a sequence, as bit masks; the warp's tokens are
// w .. w+nw-1.  The lanes hold 32 sequences around them in registers (looked up in memory step by step, three loads a token one
// after the other, 8 sequences of 9001 tokens of 501 channels took 56 us forward and 89 backward, now 50 and 81).
struct Edges {
    int base, lo, hi;              // first of the 32 sequences; where this lane's begins and ends
    int first, last;               // the run's first and last token's
    __device__ __forceinline__ void init()
    {
        base = first = last = 0;
        lo = hi = 0x7fffffff;
    }
    __device__ __forceinline__ void find(const RecurDims &g, int w, int nw, int t, int n, uint32_t &starts, uint32_t &ends)
    {
        constexpr uint32_t kAll = 0xffffffffu;
        starts = ends = 0;
        if (nw <= 0) return;
        auto covered = [&] { return __shfl_sync(kAll, lo, 0) <= w && (base + 32 >= g.Nseq || __shfl_sync(kAll, hi, 31) >= w + nw); };
        if (!covered()) {
            base = g.Nseq <= 32 ? 0 : max(0, seq_at(g.cu, g.Nseq, w) - 12);
            const int s = min(base + (int)(threadIdx.x & 31), g.Nseq);
            lo = g.cu[s];
            hi = g.cu[min(s + 1, g.Nseq)];
            if (!covered()) {   // more than 19 sequences in a warp's tokens
                if (n <= 0) return;
                first = last = up(g.cu, seq_at(g.cu, g.Nseq, w), t);
#pragma unroll 1
                for (int k = 0; k < n; ++k) {
                    last = up(g.cu, last, t + k);
                    starts |= (g.cu[last] == t + k ? 1u : 0u) << k;
                    ends |= (g.cu[last + 1] == t + k + 1 ? 1u : 0u) << k;
                }
                return;
            }
        }
        for (uint32_t some = __ballot_sync(kAll, lo < w + nw && hi > w && hi > lo); some; some &= some - 1) {
            const int i = __ffs(some) - 1, from = __shfl_sync(kAll, lo, i), to = __shfl_sync(kAll, hi, i);
            if (from <= t) first = base + i;
            if (from < t + n) last = base + i;
            if (from >= t && from < t + n) starts |= 1u << (from - t);
            if (to > t && to <= t + n) ends |= 1u << (to - 1 - t);
        }
    }
    // The sequence of a token from that of an earlier (later) one
    __device__ __forceinline__ static int up(const int32_t *cu, int s, int t)
    {
        while (cu[s + 1] <= t) ++s;
        return s;
    }
    __device__ __forceinline__ static int down(const int32_t *cu, int s, int t)
    {
        while (cu[s] > t) --s;
        return s;
    }
};

// Final states (initial states' gradients) of empty sequences: the initial ones (the final states' gradients).  A warp looks at 32
// sequences at a time; a lane's channels are c and c + 1.
template <int W, int L>
__device__ __forceinline__ void pass_empty(const RecurDims &g, int rank, int CL, int c, bool in0, bool in1, const float *from, float *to)
{
    const int lane = threadIdx.x & 31;
    if (!to) return;
    for (int s0 = (rank * W + (threadIdx.x >> 5)) * 32; s0 < g.Nseq; s0 += CL * W * 32) {
        const int s = s0 + lane;
        for (uint32_t left = __ballot_sync(0xffffffffu, s < g.Nseq && g.cu[s] == g.cu[s + 1]); left; left &= left - 1) {
            const size_t at = (size_t)(s0 + __ffs(left) - 1) * g.D + c;
            if (lane < L) store2(to + at, from ? load2(from + at, in0, in1) : two(0.f), in0, in1);
        }
    }
}

// Tokens of a box: 256 at most
template <int W>
__host__ __device__ constexpr int box_rows(int Q)
{
    return W * kRun * Q / ((W * kRun * Q + 255) / 256);
}

// The inputs of a block's two steps.  `sets`: bit mask of the arrays that a call has; their places follow each other, and behind
// them, KEPT, the states that the block's runs start from.
template <class T, int W, int Q, int MODE, bool KEPT>
struct Inputs {
    static constexpr int C = 64 / Q, R = kRun * Q, kPlace = place_bytes(W, Q, MODE, sizeof(T));   // channels, tokens of a warp, bytes of an array's place
    static constexpr int kPer = 16 / (int)sizeof(T), kPitch = MODE == kChunks ? C + kPer : C;          // elements of 16 bytes; of a row
    struct Cells {
        const T *p;
        unsigned u, step;          // kChunks: where a row begins in its first 16 bytes, from token to token
    };
    static constexpr int kRows = box_rows<W>(Q), kBoxes = W * R / kRows;                         // of an array
    static_assert(MODE != kTma || kRows * kBoxes == W * R, "boxes share the rows evenly");
    static constexpr int kKept = KEPT ? W * 64 * 4 : 0;
    char *base;
    uint64_t *bar;
    const RecurIo<T> *io;
    const RecurMaps *maps;
    int sets, count, b, c0, D;     // arrays and their number; row; first channel
    int top;                       // steps asked for, of the thread that asks
    bool failed;                   // a wait ran out: nothing is asked for any more, what the places hold is not used

    __device__ __forceinline__ int place(int array) const { return __popc(sets & ((1 << array) - 1)); }
    __device__ __forceinline__ char *slot(int st, int array) const { return base + (st & 1) * (count * kPlace + kKept) + place(array) * kPlace; }
    __device__ __forceinline__ char *kept(int st) const { return base + (st & 1) * (count * kPlace + kKept) + count * kPlace; }
    // of a lane's two channels of its run, whose first token is t
    __device__ __forceinline__ Cells cells(int st, int array, int t) const
    {
        const int lane = threadIdx.x & 31, l = lane % (32 / Q), q = lane / (32 / Q);
        Cells r = {(const T *)slot(st, array) + (((threadIdx.x >> 5) * Q + q) * kRun) * kPitch + 2 * l, 0, 0};
        if (MODE == kChunks) {
            const View<const T> &v = io->in[array];
            r.u = (unsigned)((uintptr_t)v.p / sizeof(T)) + (unsigned)b * (unsigned)v.b + (unsigned)t * (unsigned)v.t + c0;
            r.step = (unsigned)v.t;
        }
        return r;
    }
    __device__ __forceinline__ static Vec<T, 2> raw(const Cells &cells, int k)
    {
        Vec<T, 2> v;
        if constexpr (MODE == kChunks) {
            const T *p = cells.p + k * kPitch + (cells.u + k * cells.step) % kPer;
            const T e[2] = {p[0], p[1]};
            memcpy(&v.raw, e, sizeof(e));
        } else {
            v.load(cells.p + k * kPitch);
        }
        return v;
    }
    __device__ __forceinline__ static float2 at(const Cells &cells, int k)
    {
        float f[2];
        raw(cells, k).get(f);
        return make_float2(f[0], f[1]);
    }

    // Before a block's first barrier
    __device__ __forceinline__ void init(char *sm, uint64_t *bars, const RecurIo<T> *io_, const RecurMaps *maps_, int sets_, int b_, int c0_, int D_)
    {
        base = sm;
        bar = bars;
        io = io_;
        maps = maps_;
        sets = sets_;
        count = __popc(sets);
        b = b_; c0 = c0_; D = D_;
        failed = false;
        top = 0;
        if (threadIdx.x == 0) {   // the cluster's two as well
            for (int i = 0; i < 4; ++i) sm100::mbar_init(&bar[i], 1);
            sm100::fence_barrier_init();
        }
    }
    // Asks for step `st`, the block's tokens t0 .. te - 1 at most; nobody reads what it overwrites any more.
    __device__ __forceinline__ void ask(int st, int t0, int te, int short_in)
    {
        if (MODE == kTma) {
            if (threadIdx.x == 0 && !failed) {
                top = st + 1;
                uint64_t *full = &bar[st & 1];
                sm100::mbar_expect_tx(full, count * kPlace + kKept + (st >= short_in ? 16 : 0));
                if (KEPT) box_load(kept(st), &maps->kept, full, c0, t0 / kRun, b);
#pragma unroll
                for (int a = 0; a < kArrays; ++a)
                    if (sets >> a & 1)
#pragma unroll
                        for (int i = 0; i < kBoxes; ++i) box_load(slot(st, a) + i * (kPlace / kBoxes), &maps->in[a], full, c0, t0 + i * kRows, b);
            }
        } else {
            // every 16 bytes of memory that hold an element of a row, so that nothing outside of the pages of the array is touched; what else
            // they hold is in channels that do not exist, or before the row
            constexpr int N = C / kPer + 1;
            const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = t0 + warp * R, n = te - t, live = min(C, D - c0);
#pragma unroll
            for (int a = 0; a < kArrays; ++a) {
                if (!(sets >> a & 1)) continue;
                const View<const T> v = io->in[a];
                const T *from = v.at(b, 0, t) + c0;
                const uint32_t to = sm100::smem_u32(slot(st, a)) + warp * (kPlace / W);
#pragma unroll
                for (int i = lane; i < R * N; i += 32) {
                    const int k = i / N, j = i % N;
                    const uintptr_t row = (uintptr_t)(from + k * v.t);
                    const int ahead = (int)(row % 16) / (int)sizeof(T);
                    const bool some = k < n && j * kPer < ahead + live;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + (k * kPitch * (int)sizeof(T) + 16 * j)),
                                 "l"((some ? row + 16 * j : (uintptr_t)v.p) & ~(uintptr_t)15), "r"(some ? 16 : 0)
                                 : "memory");
                }
            }
        }
    }
    // Every step asks or not, and closes what it asked for
    __device__ __forceinline__ void asked() const
    {
        if (MODE == kChunks) asm volatile("cp.async.commit_group;" ::: "memory");
    }
    __device__ __forceinline__ bool arrived(int st, long long budget) const
    {
        return sm100::mbar_wait(&bar[st & 1], (uint32_t)(st >> 1) & 1u, budget, nullptr);
    }
    // Waits for step st.  Where that runs out, the thread's results from there on are NaN, and by the maps those behind it: forward by
    // the decays' parameter, backward by its x and dy (the one costs the backward 2 of 395 us for 8 x 4096 tokens of 2048 channels, the
    // other the forward 3 of 141 for 4 x 8192).
    __device__ __forceinline__ void get(int st, const RecurDims &g, RecurParams &par)
    {
        if (MODE == kTma) {
            if constexpr (!KEPT) {
                if (!failed && !arrived(st, g.budget)) {
                    failed = true;
                    par.km = two(kNan);
                    raise_status(g.status, kStatusTimeout);
                }
            } else if (failed || !arrived(st, g.budget)) {
                if (!failed) raise_status(g.status, kStatusTimeout);
                failed = true;
#pragma unroll 1
                for (int a = kX; a <= kDy; a += kDy - kX) {
                    Vec<T, 2> v;
                    const float none[2] = {kNan, kNan};
                    v.set(none);
                    T *p = const_cast<T *>(cells(st, a, 0).p);
#pragma unroll 1
                    for (int k = 0; k < kRun; ++k, p += kPitch) v.store(p);
                }
            }
        } else {
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncwarp();
        }
    }
    // At a block's end: what was asked for before a wait ran out, of two steps at most, lands before the shared memory goes away.
    __device__ __forceinline__ void drain(long long budget) const
    {
        if (MODE == kTma && failed && threadIdx.x == 0) {
            for (int st = max(0, top - 2); st < top; ++st) arrived(st, budget);
        }
    }
};

// Two channels of a token of a result.  Where the inputs come by TMA both exist (D is even) and lie in one word (of two).  (Otherwise
// one store where they do, two where not, costs more instructions to fetch than it saves: 8 x 4096 tokens of 2047 channels, bf16
// backward 417 -> 478 us.)
template <int MODE, class T>
__device__ __forceinline__ void put_two(T *p, float2 f, bool in0, bool in1)
{
    if constexpr (MODE == kTma) {
        Vec<T, 2> v;
        const float e[2] = {f.x, f.y};
        v.set(e);
        if (in0) v.store(p);
    } else {
        if (in0) st_out(p, f.x);
        if (in1) st_out(p + 1, f.y);
    }
}

// How a call's inputs get to shared memory; TMA: their maps, in boxes of `rows` tokens (not without `maps`).  `in`: bit mask
// of the arrays there.
template <class T>
int recur_mode(RecurMaps &m, const RecurIo<T> &io, int in, int rows, const RecurDims &g, bool maps = true)
{
    bool tma = maps && g.T > 0 && g.D % 2 == 0;
    for (int a = 0; a < kArrays; ++a) {
        const View<const T> &i = io.in[a];
        if (in >> a & 1) {
            tma = tma && tensor_map(&m.in[a], sizeof(T) == 4, i.p, g.D, g.T, g.B, i.t, i.b, 64 / g.Q, rows, 0);
        }
        if (a < 4 && io.out[a].p) {
            const View<T> &o = io.out[a];
            tma = tma && (uintptr_t)o.p % (2 * sizeof(T)) == 0 && o.t % 2 == 0 && o.b % 2 == 0;
        }
    }
    return tma ? kTma : kChunks;
}

// Calls f(Q, mode, packed) with a call's variant as types.
template <class F>
cudaError_t recur_variant(const RecurDims &g, int mode, F f)
{
    auto with = [&](auto q) {
        auto how = [&](auto m) { return g.cu ? f(q, m, std::true_type{}) : f(q, m, std::false_type{}); };
        return mode == kTma ? how(std::integral_constant<int, kTma>{}) : how(std::integral_constant<int, kChunks>{});
    };
    return g.Q == 4 ? with(std::integral_constant<int, 4>{}) : g.Q == 2 ? with(std::integral_constant<int, 2>{}) : with(std::integral_constant<int, 1>{});
}

// One launch over channel tiles x rows, CL blocks of a cluster each.
template <class K, class... A>
cudaError_t recur_launch(K kernel, const RecurDims &g, int threads, int smem, cudaStream_t st, const A &...args)
{
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)g.tiles * g.B * g.CL));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    cfg.attrs = at;
    if (g.CL > 1) {
        at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        at[cfg.numAttrs].val.clusterDim.x = (unsigned)g.CL;
        at[cfg.numAttrs].val.clusterDim.y = at[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    if (g.cu) {   // behind the check of the offsets
        at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
        ++cfg.numAttrs;
    }
    e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e != cudaSuccess ? e : cudaPeekAtLastError();
}

}  // namespace lay
}  // namespace gdn

// Shared by the gated linear recurrence's kernels (recur_fwd.cu, recur_bwd.cu):
// geometry, the gates, the composition of pieces of the recurrence.
//
//     m = c softplus(lam) sigmoid(rg + rg_bias),  a = exp(-m),  s = sqrt(1 - a^2)
//     h_t = a_t h_{t-1} + s_t u_t,  u = sigmoid(ig + ig_bias) x,  y = z ? h silu(z) : h
//
// Layout.  A lane holds two neighbouring channels, a warp 64 of them and kRun tokens,
// a block kWarps runs of tokens one after another, a cluster up to 8 such blocks: kSpan
// tokens a block and step.  A run is a linear map h -> A h + H of what enters it; a
// block's warps exchange their maps through shared memory, the cluster's blocks theirs
// through each other's shared memory, and every thread then steps through its run with
// the values it has in registers.  So each input is read once whatever the number of
// rows: splitting the time axis over blocks costs a barrier a step, and no second
// pass over the inputs.
#pragma once

#include "layers.h"

namespace gdn {
namespace lay {

constexpr int kRun = 8;                       // tokens of a lane and step (and between kept states)
constexpr int kWarps = 8, kRecurThreads = 32 * kWarps;
constexpr int kSpan = kRun * kWarps;          // tokens of a block and step
constexpr int kChans = 64;                    // channels of a block
constexpr int kMaxCluster = 8;

struct RecurDims {
    int B, T, D, Nseq, tiles, CL;  // tiles: channel tiles of a row; CL: blocks that share a row's tokens
    float c;
    const int32_t *cu;             // checked offsets, or null
    const float *lam, *rbias, *ibias, *h0;
};

template <class T>
struct RecurIo {
    View<const T> x, rg, ig, z, dy;
    View<T> y, dx, drg, dig, dz;
    float *hT, *keep;              // keep: state entering every kRun-th token, [B][ceil(T / kRun)][D], or null
    const float *dhT;
    float *dh0, *part;             // part: [B][CL][3][D] sums of dlam, drg_bias, dig_bias
};

struct RecurCall {
    const dn_recur_shape *s;
    const dn_recur_io *io;
    const dn_recur_grads *gr;
    int Nseq;
    const int32_t *cu;
    float *keep, *part;
};

int recur_cluster(const dn_recur_shape *s, bool bwd);
cudaError_t recur_fwd(const RecurCall &c, cudaStream_t st);
cudaError_t recur_bwd(const RecurCall &c, cudaStream_t st);
cudaError_t recur_step(const RecurCall &c, cudaStream_t st);

inline RecurDims recur_dims(const RecurCall &c, bool bwd)
{
    RecurDims g;
    g.B = c.s->B; g.T = c.s->T; g.D = c.s->D; g.c = c.s->c; g.Nseq = c.Nseq;
    g.tiles = (g.D + kChans - 1) / kChans;
    g.CL = recur_cluster(c.s, bwd);
    g.cu = c.cu;
    g.lam = c.io->lam; g.rbias = c.io->rg_bias; g.ibias = c.io->ig_bias; g.h0 = c.io->h0;
    return g;
}

__device__ __forceinline__ float rsq(float x)
{
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two channels' parameters: km = c softplus(lam), biases; dk = sigmoid(lam) / softplus(lam), the factor from
// sum q to dlam (1, its limit, where softplus underflows).
struct RecurParams {
    float2 km, rb, ib;
    __device__ __forceinline__ void load(const RecurDims &g, int c, bool in0, bool in1, float2 *dk = nullptr)
    {
        const float2 lam = make_float2(in0 ? g.lam[c] : 0.f, in1 ? g.lam[c + 1] : 0.f);
        float2 sp, der;
        softplus(lam, sp, der);
        km = mul2(sp, two(g.c));
        rb = make_float2(in0 && g.rbias ? g.rbias[c] : 0.f, in1 && g.rbias ? g.rbias[c + 1] : 0.f);
        ib = make_float2(in0 && g.ibias ? g.ibias[c] : 0.f, in1 && g.ibias ? g.ibias[c + 1] : 0.f);
        if (dk) *dk = make_float2(sp.x == 0.f ? 1.f : der.x / sp.x, sp.y == 0.f ? 1.f : der.y / sp.y);
    }
};

// a = exp(-m) and rs = 1 / sqrt(1 - a^2), y = 1 - a^2.  A decay close to 1, the usual one, leaves nothing of 1 - a^2 in
// float32 when a is rounded first, and a bias of ex2.approx adds up over the thousand tokens that such a state remembers:
// below kSmall both come from e = 1 - exp(-m) by its power series to m^7 (next term: 2e-8 of e at 0.35), a = 1 - e rounded
// once, y = e (1 + a).  m = 0 gives a = 1, y = 0 and a finite rs, so that m rs = 0, its limit.
constexpr float kSmall = 0.35f;
__device__ __forceinline__ void decay_of(float2 m, float2 &a, float2 &y, float2 &rs)
{
    float2 p = fma2(m, two(1.f / 5040.f), two(-1.f / 720.f));
    p = fma2(m, p, two(1.f / 120.f));
    p = fma2(m, p, two(-1.f / 24.f));
    p = fma2(m, p, two(1.f / 6.f));
    p = fma2(m, p, two(-0.5f));
    const float2 e = fma2(mul2(m, m), p, m);
    const float2 far = ex2_2(mul2(m, two(-kLog2e)));
    const bool sx = m.x < kSmall, sy = m.y < kSmall;
    a = make_float2(sx ? 1.f - e.x : far.x, sy ? 1.f - e.y : far.y);
    const float2 one = make_float2(sx ? e.x : 1.f - far.x, sy ? e.y : 1.f - far.y);
    y = fma2(one, a, one);
    rs = make_float2(rsq(fmaxf(y.x, 1e-37f)), rsq(fmaxf(y.y, 1e-37f)));
}

// The map of a stretch of tokens, h -> A h + H.  A stretch in which a sequence starts lets nothing through: A has its
// sign bit set (a product of decays never has).  A product that underflowed lets no finite state through, but an infinity or
// a NaN goes through the recurrence's single decays, which are not 0.
__device__ __forceinline__ float pass1(float A, float H, float h)
{
    return signbit(A) ? H : A == 0.f && !isfinite(h) ? h + H : fmaf(A, h, H);
}
__device__ __forceinline__ float2 pass(float2 A, float2 H, float2 h) { return make_float2(pass1(A.x, H.x, h.x), pass1(A.y, H.y, h.y)); }
// first (A, H), then (A2, H2)
__device__ __forceinline__ void then(float2 &A, float2 &H, float2 A2, float2 H2)
{
    H = pass(A2, H2, H);
    A = make_float2(signbit(A2.x) ? A2.x : A.x * A2.x, signbit(A2.y) ? A2.y : A.y * A2.y);
}

// Two neighbouring channels of a token, WIDE: one access, both channels exist.
template <class T, bool WIDE>
struct Two {
    Vec<T, 2> v;
    __device__ __forceinline__ void load(const T *p, bool in0, bool in1)
    {
        if constexpr (WIDE) {
            v.zero();
            if (in0) v.load(p);
        } else {
            T e[2];
            st_out(&e[0], 0.f);
            st_out(&e[1], 0.f);
            if (in0) e[0] = p[0];
            if (in1) e[1] = p[1];
            memcpy(&v, e, sizeof(e));
        }
    }
    __device__ __forceinline__ float2 get() const
    {
        float f[2];
        v.get(f);
        return make_float2(f[0], f[1]);
    }
};

template <class T, bool WIDE>
__device__ __forceinline__ void put_two(T *p, float2 f, bool in0, bool in1)
{
    if constexpr (WIDE) {
        Vec<T, 2> v;
        const float e[2] = {f.x, f.y};
        v.set(e);
        if (in0) v.store(p);
    } else {
        if (in0) st_out(p, f.x);
        if (in1) st_out(p + 1, f.y);
    }
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

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// 16 bytes into the shared memory of the cluster's block `rank`, at this block's address `dst`
__device__ __forceinline__ void remote_store(const float4 *dst, int rank, float4 v)
{
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
        "st.shared::cluster.v4.f32 [a], {%2, %3, %4, %5};\n\t}" ::"r"((uint32_t)__cvta_generic_to_shared(dst)),
        "r"(rank), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
        : "memory");
}

// The maps of a step's runs, exchanged: (A, H) of this thread's run in, what enters it out (the state before it in the order
// of the pass); `carry`, what entered the step, becomes what leaves it.  `mine` is this warp's place in the block and `at`
// the block's in the cluster, in that order.  Maps of a step lie in buffer `par`, so that one barrier a level suffices.
struct RecurShared {
    float4 warp[2][kWarps][32];
    float4 block[2][kMaxCluster][32];
};

__device__ __forceinline__ float2 exchange(RecurShared &sm, int par, int CL, int at, int mine, float2 A, float2 H, float2 &carry)
{
    const int lane = threadIdx.x & 31;
    sm.warp[par][mine][lane] = make_float4(A.x, A.y, H.x, H.y);
    __syncthreads();
    float2 pA = two(1.f), pH = two(0.f), oA = pA, oH = pH;   // of the warps before this one; of all
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w == mine) {
            pA = oA;
            pH = oH;
        }
        const float4 q = sm.warp[par][w][lane];
        then(oA, oH, make_float2(q.x, q.y), make_float2(q.z, q.w));
    }
    float2 h = carry;
    if (CL > 1) {
        if (mine < CL) remote_store(&sm.block[par][at][lane], mine, make_float4(oA.x, oA.y, oH.x, oH.y));   // each warp tells one block
        cluster_barrier();
        for (int k = 0; k < CL; ++k) {
            if (k == at) h = carry;
            const float4 q = sm.block[par][k][lane];
            carry = pass(make_float2(q.x, q.y), make_float2(q.z, q.w), carry);
        }
    } else {
        carry = pass(oA, oH, carry);
    }
    return pass(pA, pH, h);
}

// Of a run's tokens t .. t+n-1 (n <= kRun): which start and which end a sequence, as bit masks; lane k has token t + k's sequence.
__device__ __forceinline__ void run_edges(const RecurDims &g, int t, int n, uint32_t &starts, uint32_t &ends, int &seq)
{
    const int lane = threadIdx.x & 31;
    bool st = false, en = false;
    seq = 0;
    if (lane < n) {
        const int s = seq_at(g.cu, g.Nseq, t + lane);
        seq = s;
        st = g.cu[s] == t + lane;
        en = g.cu[s + 1] == t + lane + 1;
    }
    starts = __ballot_sync(0xffffffffu, st);
    ends = __ballot_sync(0xffffffffu, en);
}

// One launch over channel tiles x rows, CL blocks of a cluster each.
template <class K, class... A>
cudaError_t recur_launch(K kernel, const RecurDims &g, cudaStream_t st, const A &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)g.tiles * g.B * g.CL));
    cfg.blockDim = dim3(kRecurThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)g.CL;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = g.CL > 1 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, g, args...);
    return e != cudaSuccess ? e : cudaPeekAtLastError();
}

}  // namespace lay
}  // namespace gdn

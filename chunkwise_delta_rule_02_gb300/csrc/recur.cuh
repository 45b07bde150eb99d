// Shared by the gated linear recurrence's kernels (recur_fwd.cu, recur_bwd.cu):
// geometry, the gates, the pieces of the recurrence and their exchange.
//
//     m = c softplus(lam) sigmoid(rg + rg_bias),  a = exp(-m),  s = sqrt(1 - a^2)
//     h_t = a_t h_{t-1} + s_t u_t,  u = sigmoid(ig + ig_bias) x,  y = z ? h silu(z) : h
//
// Layout.  A lane holds two neighbouring channels of a run of kRun tokens; a warp holds Q runs one after
// another of 64 / Q channels (Q = 4 where 64-channel tiles would leave most SMs idle), a block W warps, a
// cluster up to 8 blocks.  A run is a linear map h -> A h + H of what enters it; the runs of a warp exchange
// their maps by shuffles, a block's warps through shared memory, the cluster's blocks through each
// other's shared memory, and every thread then steps through its run.  So each input is read once whatever
// the number of rows: splitting the time axis over blocks costs a barrier a step, and no second pass
// over the inputs.
//
// Every warp has a ring of stages of its inputs in shared memory, filled by TMA ahead of their use (a box of
// 64 / Q channels x kRun Q tokens an array) and emptied the same way: a result takes the place of the input it
// belongs to.  Arrays that a tensor map cannot describe (rows that do not start at 16 bytes) go through the same
// ring in words of 4 bytes, or, bf16 that do not start at those, element by element in the step that needs them.
#pragma once

#include <type_traits>

#include "layers.h"
#include "sm100.cuh"

namespace gdn {
namespace lay {

constexpr int kRun = 8;                       // tokens of a lane and step (and between kept states)
constexpr int kMaxCluster = 8;
constexpr long long kRecurBudget = 4000000000LL;   // clock cycles (about 2 s) for any one wait

// Warps of a block, stages of the ring, blocks an SM holds, by the type's bytes
__host__ __device__ constexpr int fwd_warps(int bytes) { return bytes == 2 ? 8 : 4; }
__host__ __device__ constexpr int bwd_warps(int bytes) { return bytes == 2 ? 6 : 4; }
__host__ __device__ constexpr int fwd_stages(int) { return 3; }
__host__ __device__ constexpr int bwd_stages(int bytes) { return bytes == 2 ? 3 : 2; }
constexpr int kResident = 2;

enum { kElements, kWords, kTma };             // how a ring is filled

struct RecurDims {
    int B, T, D, Nseq, tiles, CL, Q;   // tiles: channel tiles of a row; CL: blocks that share a row's tokens
    float c;
    const int32_t *cu;             // checked offsets, or null
    const float *lam, *rbias, *ibias, *h0;
    uint32_t *status;
};

// Arrays: inputs first; a result lies in its input's place
enum { kX, kRg, kIg, kZ, kDy, kArrays };

template <class T>
struct RecurIo {
    View<const T> in[kArrays];     // x, rg, ig, z or null, dy
    View<T> out[kArrays];          // forward: y at kX; backward: dx, drg, dig, dz
    float *hT, *keep;              // keep: state entering every kRun-th token, [B][ceil(T / kRun)][D], or null
    const float *dhT;
    float *dh0, *part;             // part: [B][CL][3][D] sums of dlam, drg_bias, dig_bias
};

struct RecurMaps {
    CUtensorMap in[kArrays], out[kArrays];
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

__device__ __forceinline__ void box_load(void *dst, const CUtensorMap *map, uint64_t *bar, int c, int t, int b)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            sm100::smem_u32(dst)),
        "l"((uint64_t)map), "r"(sm100::smem_u32(bar)), "r"(c), "r"(t), "r"(b)
        : "memory");
}

__device__ __forceinline__ void box_store(const CUtensorMap *map, const void *src, int c, int t, int b)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"((uint64_t)map),
                 "r"(sm100::smem_u32(src)), "r"(c), "r"(t), "r"(b)
                 : "memory");
}

template <int W, int Q>
struct RecurShared {
    float4 warp[2][W][32 / Q];
    float4 block[2][kMaxCluster][32 / Q];
    uint64_t bar[W][3];
};

// The maps of a step's runs, exchanged: (A, H) of this thread's run in, what enters it out (the state before it in the order
// of the pass, BACK: from the last run to the first); `carry`, what entered the step, becomes what leaves it.  `rank` is the block's
// place in the cluster.  Maps of a step lie in buffer `par`, so that one barrier a level suffices.
template <int W, int Q, bool CUT, bool BACK>
__device__ __forceinline__ float2 exchange(RecurShared<W, Q> &sm, int par, int CL, int rank, float2 A, float2 H, float2 &carry)
{
    constexpr int L = 32 / Q;
    const int lane = threadIdx.x & 31, l = lane % L, warp = threadIdx.x >> 5;
    const int mine = BACK ? W - 1 - warp : warp, at = BACK ? CL - 1 - rank : rank, q = BACK ? Q - 1 - lane / L : lane / L;
    float2 pA = two(1.f), pH = two(0.f);   // of what lies before this run: in the warp, then in the block
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
    float2 h = carry;
    if (CL == 1) {
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w == mine) h = carry;
            const float4 m = sm.warp[par][w][l];
            carry = pass<CUT>(make_float2(m.x, m.y), make_float2(m.z, m.w), carry);
        }
    } else {
        float2 wA = two(1.f), wH = two(0.f), oA = wA, oH = wH;   // of the warps before this one; of all
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w == mine) {
                wA = oA;
                wH = oH;
            }
            const float4 m = sm.warp[par][w][l];
            then<CUT>(oA, oH, make_float2(m.x, m.y), make_float2(m.z, m.w));
        }
        // each warp tells some blocks
        if (lane < L)
            for (int k = warp; k < CL; k += W) remote_store(&sm.block[par][at][l], k, make_float4(oA.x, oA.y, oH.x, oH.y));
        __syncwarp();
        cluster_barrier();
        for (int k = 0; k < CL; ++k) {
            if (k == at) h = carry;
            const float4 m = sm.block[par][k][l];
            carry = pass<CUT>(make_float2(m.x, m.y), make_float2(m.z, m.w), carry);
        }
        h = pass<CUT>(wA, wH, h);
    }
    return Q > 1 ? pass<CUT>(pA, pH, h) : h;
}

// Which of this lane's run's tokens t .. t+n-1 (n <= kRun) start and which end a sequence, as bit masks, and the sequence of the
// first of them; the warp's tokens are w .. w+nw-1.  Tokens inside the sequence that the warp looked up last have neither.
struct Edges {
    int lo, hi;                    // that sequence
    __device__ __forceinline__ void find(const RecurDims &g, int w, int nw, int t, int n, uint32_t &starts, uint32_t &ends)
    {
        starts = ends = 0;
        if (nw <= 0 || (lo < w && w + nw < hi)) return;
        const int s = seq_at(g.cu, g.Nseq, w);
        lo = g.cu[s];
        hi = g.cu[s + 1];
        if (lo < w && w + nw < hi) return;
        for (int k = 0; k < n; ++k) {
            const int q = seq_at(g.cu, g.Nseq, t + k);
            starts |= (g.cu[q] == t + k ? 1u : 0u) << k;
            ends |= (g.cu[q + 1] == t + k + 1 ? 1u : 0u) << k;
        }
    }
};

// A warp's ring.  `sets`: bit mask of the input arrays that a call has; their places follow each other.
template <class T, int W, int Q, int S, int MODE>
struct Ring {
    static constexpr int kSlot = kRun * 64 * (int)sizeof(T), C = 64 / Q, R = kRun * Q;   // bytes, channels, tokens of an array's place
    char *base;                    // of this warp's first place
    uint64_t *bar;
    const RecurIo<T> *io;
    const RecurMaps *maps;
    int sets, count, b, c0, D;     // arrays and their number; row; first channel
    bool failed;

    __device__ __forceinline__ int place(int array) const { return __popc(sets & ((1 << array) - 1)); }
    __device__ __forceinline__ char *slot(int st, int array) const { return base + ((size_t)(st % S) * count + place(array)) * W * kSlot; }
    // of a lane's two channels of its run's token k
    __device__ __forceinline__ T *cell(int st, int array, int k) const
    {
        const int lane = threadIdx.x & 31, l = lane % (32 / Q), q = lane / (32 / Q);
        return (T *)slot(st, array) + (q * kRun + k) * C + 2 * l;
    }

    __device__ __forceinline__ void init(char *sm, uint64_t *bars, const RecurIo<T> *io_, const RecurMaps *maps_, int sets_, int b_, int c0_, int D_)
    {
        base = sm + (threadIdx.x >> 5) * kSlot;
        bar = bars;
        io = io_;
        maps = maps_;
        sets = sets_;
        count = __popc(sets);
        b = b_; c0 = c0_; D = D_;
        failed = false;
        if (MODE == kTma) {
            if ((threadIdx.x & 31) == 0) {
                for (int i = 0; i < S; ++i) sm100::mbar_init(&bar[i], 1);
                sm100::fence_barrier_init();
            }
            __syncwarp();
        }
    }
    // Asks for step `st`, the warp's tokens t .. t + n - 1; what it overwrites has been stored.
    __device__ __forceinline__ void ask(int st, int t, int n) const
    {
        if (MODE == kTma) {
            if ((threadIdx.x & 31) == 0) {
                uint64_t *full = &bar[st % S];
                sm100::bulk_wait_read();
                sm100::mbar_expect_tx(full, count * kSlot);
#pragma unroll
                for (int a = 0; a < kArrays; ++a)
                    if (sets >> a & 1) box_load(slot(st, a), &maps->in[a], full, c0, t, b);
            }
        } else if (MODE == kWords) {
            constexpr int P = 4 / sizeof(T), N = R * C / P / 32;   // elements of a word; words of a lane
            for (int a = 0; a < kArrays; ++a) {
                if (!(sets >> a & 1)) continue;
                const View<const T> v = io->in[a];
                const uint32_t to = sm100::smem_u32(slot(st, a));
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int w = j * 32 + (threadIdx.x & 31), k = w / (C / P), c = w % (C / P) * P;
                    const int bytes = k < n ? max(0, min(4, (D - c0 - c) * (int)sizeof(T))) : 0;
                    const T *from = v.at(b, 0, bytes ? t + k : 0) + (bytes ? c0 + c : 0);
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to + 4 * w), "l"(from), "r"(bytes) : "memory");
                }
            }
        }
    }
    // Every step asks or not, and closes what it asked for
    __device__ __forceinline__ void asked() const
    {
        if (MODE == kWords) asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // Waits for step st (or, elements, loads it)
    __device__ __forceinline__ void get(int st, int t, int n, uint32_t *status)
    {
        if (MODE == kTma) {
            if (!sm100::mbar_wait(&bar[st % S], (uint32_t)(st / S) & 1u, failed ? 1000 : kRecurBudget, nullptr)) {
                failed = true;
                raise_status(status, kStatusTimeout);
            }
        } else if (MODE == kWords) {
            asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
            __syncwarp();
        } else {
            const int lane = threadIdx.x & 31;
            T v[kArrays][2 * kRun];
#pragma unroll
            for (int a = 0; a < kArrays; ++a) {
                if (!(sets >> a & 1)) continue;
#pragma unroll
                for (int j = 0; j < 2 * kRun; ++j) {
                    const int i = j * 32 + lane, k = i / C, c = i % C;
                    st_out(&v[a][j], 0.f);
                    if (k < n && c0 + c < D) v[a][j] = io->in[a].at(b, 0, t + k)[c0 + c];
                }
            }
            __syncwarp();
#pragma unroll
            for (int a = 0; a < kArrays; ++a) {
                if (!(sets >> a & 1)) continue;
#pragma unroll
                for (int j = 0; j < 2 * kRun; ++j) ((T *)slot(st, a))[j * 32 + lane] = v[a][j];
            }
            __syncwarp();
        }
    }
    __device__ __forceinline__ float2 at(int st, int array, int k) const
    {
        Vec<T, 2> v;
        float f[2];
        v.load(cell(st, array, k));
        v.get(f);
        return make_float2(f[0], f[1]);
    }
    __device__ __forceinline__ void put(int st, int array, int k, float2 x) const
    {
        Vec<T, 2> v;
        const float f[2] = {x.x, x.y};
        v.set(f);
        v.store(cell(st, array, k));
    }
    // Stores the results that were put in the places of `arrays`
    __device__ __forceinline__ void flush(int st, int arrays, int t, int n) const
    {
        const int lane = threadIdx.x & 31;
        if (MODE == kTma) {
            sm100::fence_async_smem();
            __syncwarp();
            if (lane == 0 && n > 0) {
#pragma unroll
                for (int a = 0; a < kArrays; ++a)
                    if (arrays >> a & 1) box_store(&maps->out[a], slot(st, a), c0, t, b);
                sm100::bulk_commit();
            }
        } else {
            __syncwarp();
            for (int a = 0; a < kArrays; ++a) {
                if (!(arrays >> a & 1)) continue;
                const T *from = (const T *)slot(st, a);
#pragma unroll
                for (int j = 0; j < 2 * kRun; ++j) {
                    const int i = j * 32 + lane, k = i / C, c = i % C;
                    if (k < n && c0 + c < D) io->out[a].at(b, 0, t + k)[c0 + c] = from[i];
                }
            }
        }
    }
    __device__ __forceinline__ void end() const
    {
        if (MODE == kTma && (threadIdx.x & 31) == 0) sm100::bulk_wait_all();
    }
};

// How a call's arrays are moved; TMA: their maps.  `in`, `out`: bit masks of the arrays there.
template <class T>
int recur_mode(RecurMaps &m, const RecurIo<T> &io, int in, int out, const RecurDims &g)
{
    bool tma = g.T > 0, words = true;
    for (int a = 0; a < kArrays; ++a) {
        const View<const T> &i = io.in[a];
        const View<T> &o = io.out[a];
        const int c = 64 / g.Q, r = kRun * g.Q;
        if (in >> a & 1) {
            tma = tma && tensor_map(&m.in[a], sizeof(T) == 4, i.p, g.D, g.T, g.B, i.t, i.b, c, r, false);
            words = words && (uintptr_t)i.p % 4 == 0 && (sizeof(T) == 4 || (i.t % 2 == 0 && i.b % 2 == 0));
        }
        if (out >> a & 1) tma = tma && tensor_map(&m.out[a], sizeof(T) == 4, o.p, g.D, g.T, g.B, o.t, o.b, c, r, false);
    }
    return tma ? kTma : words ? kWords : kElements;
}

// Calls f(Q, mode, packed) with a call's variant as types; float32 that words serve always has no elements.
template <class T, class F>
cudaError_t recur_variant(const RecurDims &g, int mode, F f)
{
    auto with = [&](auto q) {
        auto how = [&](auto m) { return g.cu ? f(q, m, std::true_type{}) : f(q, m, std::false_type{}); };
        if (mode == kTma) return how(std::integral_constant<int, kTma>{});
        if (mode == kWords || sizeof(T) == 4) return how(std::integral_constant<int, kWords>{});
        return how(std::integral_constant<int, sizeof(T) == 4 ? kWords : kElements>{});
    };
    return g.Q == 4 ? with(std::integral_constant<int, 4>{}) : with(std::integral_constant<int, 1>{});
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
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)g.CL;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = g.CL > 1 ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e != cudaSuccess ? e : cudaPeekAtLastError();
}

}  // namespace lay
}  // namespace gdn

// Dropout from a counter-based generator, with the residual's addition; the backward pass is the same kernel
// without a residual.
//
//     y = residual + (word(i) >= threshold ? x scale : 0),  scale = 1 / (1 - p),  threshold = round(p 2^32)
//
// word(i), i the element's index in the [B][H][T][d] order whatever the strides, is word i mod 4 of
// Philox 4x32 with 10 rounds (Salmon, Moraes, Dror, Shaw: Parallel random numbers: as easy as 1, 2, 3; 2011) of the counter
// (i / 4, call number) under the key `seed`: no mask is stored, and none depends on how the work is split.
//
// With a residual bound by HBM (67 M bf16: 65 us, 93 % of a copy's rate), without one by the generator: 18 wide
// multiplications and 20 logic operations for 4 elements (57 us; multiplications of the halves by two instructions: 69).
#include <type_traits>

#include "layers.h"

namespace gdn {
namespace lay {

namespace {

// Threads of a block, blocks an SM, vectors a thread has in flight (67 M elements with the residual and without: 64.8 and 57.3 us;
// 512 x 4 x 2: 65.2, 64.1; 512 x 8 x 1: 64.8, 57.4; 256 x 16 x 1: 67.7, 58.6).
constexpr int kDropThreads = 256, kDropBlocks = 8, U = 2;

struct DropDims {
    int H, T;
    long long d, n;                // features of a row, elements
    int flat;                      // all arrays are dense: one row of n elements
    uint32_t threshold;
    float scale;
    const int64_t *rng;            // seed, call number
};

// The keys of the ten rounds are the same for all elements: a thread makes them once (added up in every round they were a
// third of the instructions: 8 x 4096 x 2048 elements took 70 us).
struct Philox {
    uint32_t k0[10], k1[10], c2, c3;
    __device__ __forceinline__ void load(const int64_t *rng)
    {
        const uint64_t seed = (uint64_t)rng[0], call = (uint64_t)rng[1];
        c2 = (uint32_t)call;
        c3 = (uint32_t)(call >> 32);
#pragma unroll
        for (int r = 0; r < 10; ++r) {
            k0[r] = (uint32_t)seed + r * 0x9E3779B9u;
            k1[r] = (uint32_t)(seed >> 32) + r * 0xBB67AE85u;
        }
    }
    // BIG: counters may pass 32 bits.  Where they do not, one product of the first round and one of the second are the same for
    // all elements, and are made once a thread.
    template <bool BIG>
    __device__ __forceinline__ void words(uint64_t group, uint32_t (&w)[4]) const
    {
        uint32_t a = (uint32_t)group, b = BIG ? (uint32_t)(group >> 32) : 0u, c = c2, d = c3;
#pragma unroll
        for (int r = 0; r < 10; ++r) {
            const uint64_t u = (uint64_t)a * 0xD2511F53u, v = (uint64_t)c * 0xCD9E8D57u;
            a = (uint32_t)(v >> 32) ^ b ^ k0[r];
            b = (uint32_t)v;
            c = (uint32_t)(u >> 32) ^ d ^ k1[r];
            d = (uint32_t)u;
        }
        w[0] = a; w[1] = b; w[2] = c; w[3] = d;
    }
};

// A thread takes V elements of a row at a time (V a multiple of 4: whole counters; what a flat row has beyond its vectors goes
// one by one), or, V = 1, the up to 4 elements of one counter, each with a row of its own.  NONE: the threshold is 2^32, above every
// word (a kernel of its own: as a second condition in the comparison it cost 3 of 57 us).
template <class T, int V, bool RES, bool BIG, bool NONE = false>
__global__ void __launch_bounds__(kDropThreads) k_dropout(DropDims g, View<const T> x, View<const T> res, View<T> y)
{
    Philox gen;
    gen.load(g.rng);
    auto place = [&](long long i, int &b, int &h, int &t) -> long long {   // of element i: its row; the feature
        b = h = t = 0;
        if (g.flat) return i;
        if (g.n < 1ll << 32) {   // divisions of 32 bits are a fifth of the others
            const unsigned row = (unsigned)i / (unsigned)g.d, bh = row / (unsigned)g.T;
            t = (int)(row - bh * (unsigned)g.T);
            b = (int)(bh / (unsigned)g.H);
            h = (int)(bh - (unsigned)b * (unsigned)g.H);
            return (unsigned)i - row * (unsigned)g.d;
        }
        const long long row = i / g.d, bh = row / g.T;
        t = (int)(row - bh * g.T);
        b = (int)(bh / g.H);
        h = (int)(bh - (long long)b * g.H);
        return i - row * g.d;
    };
    auto single = [&](long long i, uint32_t w) {
        int b, h, t;
        const long long j = place(i, b, h, t);
        float f = !NONE && w >= g.threshold ? ld_in(x.at(b, h, t) + j) * g.scale : 0.f;
        if (RES) f += ld_in(res.at(b, h, t) + j);
        st_out(y.at(b, h, t) + j, f);
    };
    const long long first = blockIdx.x * (long long)kDropThreads + threadIdx.x, step = (long long)gridDim.x * kDropThreads;
    if constexpr (V == 1) {
        for (long long q = first; q * 4 < g.n; q += step) {
            uint32_t w[4];
            gen.words<BIG>((uint64_t)q, w);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (q * 4 + e < g.n) single(q * 4 + e, w[e]);
        }
    } else {
        const long long all = g.n / V;
        auto some = [&](long long q0, auto whole) {   // U vectors, `step` apart
            Vec<T, V> vx[U], vr[U];
            T *to[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const long long q = q0 + u * step;
                if (decltype(whole)::value || q < all) {
                    int b, h, t;
                    const long long j = place(q * V, b, h, t);
                    vx[u].load(x.at(b, h, t) + j);
                    if (RES) vr[u].load(res.at(b, h, t) + j);
                    to[u] = y.at(b, h, t) + j;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const long long q = q0 + u * step;
                if (!decltype(whole)::value && q >= all) break;
                float f[V], r[V];
                vx[u].get(f);
                if (RES) vr[u].get(r);
#pragma unroll
                for (int e = 0; e < V; e += 4) {
                    uint32_t w[4];
                    gen.words<BIG>((uint64_t)(q * (V / 4) + e / 4), w);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        f[e + i] = w[i] >= g.threshold ? f[e + i] * g.scale : 0.f;
                        if (RES) f[e + i] += r[e + i];
                    }
                }
                vx[u].set(f);
                vx[u].store(to[u]);
            }
        };
        long long q = first;
        for (; q + (U - 1) * step < all; q += U * step) some(q, std::true_type{});
        if (q < all) some(q, std::false_type{});
        if (all * V + first < g.n) {   // at most V - 1, of the first threads
            const long long i = all * V + first;
            uint32_t w[4];
            gen.words<BIG>((uint64_t)i / 4, w);
            single(i, i % 4 == 0 ? w[0] : i % 4 == 1 ? w[1] : i % 4 == 2 ? w[2] : w[3]);
        }
    }
}

// Whether a view's elements lie one after another
bool dense(const dn_dropout_shape *s, const dn_view *v)
{
    if (!v || !v->data) return true;
    return (s->T == 1 || v->time == s->d) && (s->H == 1 || v->head == (long long)s->T * s->d) &&
           (s->B == 1 || v->batch == (long long)s->H * s->T * s->d);
}

template <class T>
cudaError_t run(const DropCall &c, cudaStream_t st)
{
    constexpr int V = 16 / sizeof(T);
    const dn_dropout_shape *s = c.s;
    DropDims g;
    g.H = s->H; g.T = s->T; g.d = s->d;
    g.n = (long long)s->B * s->H * s->T * s->d;
    g.rng = c.rng;
    const double th = s->p * 4294967296.0 + 0.5;
    const bool none = th >= 4294967296.0;
    g.threshold = none ? 0u : (uint32_t)th;
    g.scale = (float)(1.0 / (1.0 - s->p));
    if (g.n == 0) return cudaSuccess;
    dn_view at[3] = {};
    const dn_view *views[3] = {c.x, c.residual, c.y};
    g.flat = dense(s, c.x) && dense(s, c.residual) && dense(s, c.y);
    if (g.flat) {
        for (int i = 0; i < 3; ++i) {
            if (views[i]) at[i].data = views[i]->data;
            views[i] = &at[i];
        }
    }
    const bool wide = !none && (g.flat || s->d % V == 0) && can_vector(views[0], sizeof(T), 16) && can_vector(views[1], sizeof(T), 16) &&
                      can_vector(views[2], sizeof(T), 16);
    const View<const T> x = view_of<const T>(views[0]), r = view_of<const T>(views[1]);
    const View<T> y = view_of<T>(views[2]);
    const long long per = wide ? V : 4, need = ((g.n + per - 1) / per + kDropThreads - 1) / kDropThreads;
    const unsigned blocks = (unsigned)(need < (long long)kDropBlocks * sm_count() ? need : (long long)kDropBlocks * sm_count());
    auto go = [&](auto kernel) { kernel<<<blocks, kDropThreads, 0, st>>>(g, x, r, y); };
    if (none) {
        r.p ? go(k_dropout<T, 1, true, true, true>) : go(k_dropout<T, 1, false, true, true>);
    } else if (g.n > 1ll << 34) {
        if (wide) r.p ? go(k_dropout<T, V, true, true>) : go(k_dropout<T, V, false, true>);
        else r.p ? go(k_dropout<T, 1, true, true>) : go(k_dropout<T, 1, false, true>);
    } else {
        if (wide) r.p ? go(k_dropout<T, V, true, false>) : go(k_dropout<T, V, false, false>);
        else r.p ? go(k_dropout<T, 1, true, false>) : go(k_dropout<T, 1, false, false>);
    }
    return cudaPeekAtLastError();
}

}  // namespace

cudaError_t dropout(const DropCall &c, cudaStream_t st) { return c.s->dtype == DN_F32 ? run<float>(c, st) : run<__nv_bfloat16>(c, st); }

}  // namespace lay
}  // namespace gdn

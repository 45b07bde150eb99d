// Short causal convolution, depthwise, 2..4 taps: forward, backward, one token.
//
//     pre[t][c] = bias[c] + sum_k w[c][k] x[t-(W-1)+k][c],   y = silu(pre) or pre
//     dpre = dy silu'(pre),  dx[t] = sum_k w[k] dpre[t+(W-1)-k],
//     dw[c][k] = sum_t dpre[t] x[t-(W-1)+k],  dbias = sum_t dpre[t]
//
// Bound by HBM: x read, y written (backward: x, dy read, dx written).  A thread
// owns V consecutive channels (8 bytes where strides and alignment allow, else
// one element) and walks a run of tokens with the last W inputs in registers, so
// that an input is read once plus W - 1 halo tokens a run; a warp covers 32
// neighbouring vectors of one token.  Measured: forward 4.9 TB/s (72 % of a copy),
// backward 4.05 TB/s (60 %).  What stands against more is latency: a thread loads 8 tokens,
// then computes them with nothing in flight, and registers allow three blocks (backward
// two) an SM.  Issue slots are 43 % (42 %) used, by 11 (20) instructions an element, the
// DRAM 57 % (54 %), and a warp waits for its loads most of the time.
#include "layers.h"

namespace gdn {
namespace lay {

namespace {

constexpr int kTX = 32, kTY = 8;     // threads: channel vectors x runs

// Vectors of 8 bytes, and 8 tokens' loads in flight, measured at 4 x 8192 (forward) and
// 8 x 4096 tokens (backward) of 2048 bf16 channels: forward 59 us then, 55 now (16-byte vectors: 63 us with
// twice the registers, 4 tokens in flight 69 us), backward 99 us (16 bytes: 190 us; 4 tokens 119 us).
constexpr int kBytes = 8, kInFlight = 8;

struct ConvDims {
    int H, T, d, C, N, silu, run, runs, blocks_x;   // blocks_x: channel-vector blocks
    long long rows;                                  // (batch, group of kTY runs) pairs
    const int32_t *cu;
};

// The run of this thread: false when it has none.
template <int V>
__device__ __forceinline__ bool my_run(const ConvDims &g, int &cv, int &b, int &t0, long long &row)
{
    const int bx = blockIdx.x % g.blocks_x;
    row = blockIdx.x / g.blocks_x;
    cv = bx * kTX + threadIdx.x;
    const int per = (g.runs + kTY - 1) / kTY;
    b = (int)(row / per);
    const long long r = (row - (long long)b * per) * kTY + threadIdx.y;
    t0 = (int)min(r * g.run, (long long)g.T);
    return cv < g.C / V && r < g.runs;
}

// Channels go in pairs (two float32 operations an instruction); a single one is paired
// with a channel of zeros.
template <int V>
constexpr int kPairs = V == 1 ? 1 : V / 2;

template <class T, int V>
__device__ __forceinline__ void get_pairs(float2 (&f)[kPairs<V>], const Vec<T, V> &q)
{
    float e[V];
    q.get(e);
#pragma unroll
    for (int i = 0; i < kPairs<V>; ++i) f[i] = V == 1 ? make_float2(e[0], 0.f) : make_float2(e[2 * i], e[V == 1 ? 0 : 2 * i + 1]);
}

template <class T, int V>
__device__ __forceinline__ void set_pairs(Vec<T, V> &q, const float2 (&f)[kPairs<V>])
{
    float e[V];
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = i & 1 ? f[i / 2].y : f[i / 2].x;
    q.set(e);
}

template <int W, int V>
__device__ __forceinline__ void load_taps(const float *w, const float *bias, int c0, float2 (&wt)[W][kPairs<V>],
                                          float2 (&bs)[kPairs<V>])
{
    float tmp[V * W];
    if constexpr (V * W % 4 == 0 && V > 1) {
        const float4 *p = reinterpret_cast<const float4 *>(w + (size_t)c0 * W);
#pragma unroll
        for (int i = 0; i < V * W / 4; ++i) {
            const float4 q = p[i];
            tmp[4 * i] = q.x; tmp[4 * i + 1] = q.y; tmp[4 * i + 2] = q.z; tmp[4 * i + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V * W; ++i) tmp[i] = w[(size_t)c0 * W + i];
    }
#pragma unroll
    for (int i = 0; i < kPairs<V>; ++i) {
#pragma unroll
        for (int k = 0; k < W; ++k) wt[k][i] = V == 1 ? make_float2(tmp[k], 0.f) : make_float2(tmp[2 * i * W + k], tmp[V == 1 ? 0 : (2 * i + 1) * W + k]);
        bs[i] = !bias ? two(0.f) : V == 1 ? make_float2(bias[c0], 0.f) : make_float2(bias[c0 + 2 * i], bias[c0 + (V == 1 ? 0 : 2 * i + 1)]);
    }
}

// Window of the last W values of a thread's channels, as a ring with static places: before
// token u of an unrolled run (u counted from a multiple of W) place (u + 1 + k) % W holds the
// value k - (W - 1) tokens away, and place u % W takes the new one.
template <int W, int V>
using Ring = float2[W][kPairs<V>];

template <int W, int V>
__device__ __forceinline__ void rotate(Ring<W, V> &r)   // one token on, back to u = 0
{
#pragma unroll
    for (int i = 0; i < kPairs<V>; ++i) {
        const float2 newest = r[0][i];
#pragma unroll
        for (int k = 0; k + 1 < W; ++k) r[k][i] = r[k + 1][i];
        r[W - 1][i] = newest;
    }
}

// The W - 1 inputs before token t of a sequence [lo, ...): from x, or from the
// sequence's initial taps, or zero.
template <class T, int W, int V>
__device__ __forceinline__ void load_hist(Ring<W, V> &h, const T *xr, long long xt, int t, int lo, const T *s0, int C)
{
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        const int tt = t - (W - 1) + k;
        Vec<T, V> q;
        q.zero();
        if (tt >= lo) q.load(xr + tt * xt);
        else if (s0) q.load(s0 + (size_t)(W - 1 + tt - lo) * C);
        get_pairs<T, V>(h[k + 1], q);
    }
}

// pre-activation of ring place u's token
template <int W, int V>
__device__ __forceinline__ void taps_at(float2 (&p)[kPairs<V>], const Ring<W, V> &x, const float2 (&wt)[W][kPairs<V>],
                                        const float2 (&bs)[kPairs<V>], int u)
{
#pragma unroll
    for (int i = 0; i < kPairs<V>; ++i) {
        p[i] = bs[i];
#pragma unroll
        for (int k = 0; k < W; ++k) p[i] = fma2(wt[k][i], x[(u + 1 + k) % W][i], p[i]);
    }
}

// tokens whose loads are in flight together, a multiple of W
template <int W>
constexpr int kUnroll = (kInFlight + W - 1) / W * W;

template <class T, int W, int V>
__global__ void __launch_bounds__(kTX *kTY, 2) k_conv_fwd(ConvDims g, View<const T> x, View<T> y, const float *__restrict__ w,
                                                       const float *__restrict__ bias, const T *s0, T *sT)
{
    constexpr int U = kUnroll<W>, P = kPairs<V>;
    int cv, b, t0;
    long long row;
    if (!my_run<V>(g, cv, b, t0, row)) return;
    const int c0 = cv * V, hd = c0 / g.d, j = c0 - hd * g.d;
    const T *xr = x.at(b, hd, 0) + j;
    T *yr = y.at(b, hd, 0) + j;
    float2 wt[W][P], bs[P];
    Ring<W, V> h;
    load_taps<W, V>(w, bias, c0, wt, bs);
    int t = t0;
    const int t1 = min(t0 + g.run, g.T);
    int s = g.cu ? seq_at(g.cu, g.N, t0) : b;
    while (t < t1) {
        if (g.cu && s >= g.N) return;
        const int lo = g.cu ? g.cu[s] : 0, hi = g.cu ? g.cu[s + 1] : g.T;
        const int end = min(t1, hi);
        if (end > t) load_hist<T, W, V>(h, xr, x.t, t, lo, s0 ? s0 + (size_t)s * (W - 1) * g.C + c0 : nullptr, g.C);
        const T *px = xr + t * x.t;
        T *py = yr + t * y.t;
        auto token = [&](const Vec<T, V> &in, int u) {
            float2 p[P];
            get_pairs<T, V>(h[u % W], in);
            taps_at<W, V>(p, h, wt, bs, u);
            if (g.silu) {
#pragma unroll
                for (int i = 0; i < P; ++i) p[i] = mul2(p[i], sigmoid2(p[i]));
            }
            Vec<T, V> out;
            set_pairs<T, V>(out, p);
            out.store(py);
            py += y.t;
        };
        for (; t + U <= end; t += U) {
            Vec<T, V> in[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                in[u].load(px);
                px += x.t;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) token(in[u], u);
        }
        for (; t < end; ++t) {
            Vec<T, V> in;
            in.load(px);
            px += x.t;
            token(in, 0);
            rotate<W, V>(h);
        }
        if (sT && t == hi && hi > lo) {   // the ring holds the sequence's last inputs, initial taps included
#pragma unroll
            for (int k = 0; k < W - 1; ++k) {
                Vec<T, V> out;
                set_pairs<T, V>(out, h[k + 1]);
                out.store(sT + ((size_t)s * (W - 1) + k) * g.C + c0);
            }
        }
        ++s;
    }
}

// Final taps of empty sequences: their initial ones.
template <class T>
__global__ void k_conv_empty(ConvDims g, int taps, const T *s0, T *sT)
{
    const long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x;
    if (i >= (long long)g.N * g.C) return;
    const int s = (int)(i / g.C), c = (int)(i - (long long)s * g.C);
    if (g.cu ? g.cu[s + 1] > g.cu[s] : g.T > 0) return;
    for (int k = 0; k < taps; ++k) {
        const size_t at = ((size_t)s * taps + k) * g.C + c;
        if (s0) sT[at] = s0[at];
        else st_out(sT + at, 0.f);
    }
}

// Backward.  For the run's tokens t0 .. t1-1 and the W - 1 behind them (of the same
// sequence) the thread computes dpre once, keeps the last W of them, and writes
// dx of the token W - 1 back, whose sum is then complete.  dw and dbias sum over
// the run in registers, over the block's kTY runs in shared memory, and over
// blocks in col_sum: no atomics, one fixed order.
template <class T, int W, int V>
__global__ void __launch_bounds__(kTX *kTY, 2) k_conv_bwd(ConvDims g, View<const T> x, View<const T> dy, View<T> dx,
                                                       const float *__restrict__ w, const float *__restrict__ bias,
                                                       const T *__restrict__ s0, const T *__restrict__ dsT,
                                                       float *__restrict__ part)
{
    constexpr int U = kUnroll<W>, P = kPairs<V>;
    __shared__ float red[kTY][kTX * V];
    int cv, b, t0;
    long long row;
    const bool live = my_run<V>(g, cv, b, t0, row);
    float2 acc[W + 1][P];
#pragma unroll
    for (int k = 0; k <= W; ++k)
#pragma unroll
        for (int i = 0; i < P; ++i) acc[k][i] = two(0.f);
    if (live) {
        const int c0 = cv * V, hd = c0 / g.d, j = c0 - hd * g.d;
        const T *xr = x.at(b, hd, 0) + j, *gr = dy.at(b, hd, 0) + j;
        T *dr = dx.at(b, hd, 0) + j;
        float2 wt[W][P], bs[P];
        Ring<W, V> h, dp;   // inputs and dpre of the last W tokens
        load_taps<W, V>(w, bias, c0, wt, bs);
        int t = t0;
        const int t1 = min(t0 + g.run, g.T);
        int s = g.cu ? seq_at(g.cu, g.N, t0) : b;
        while (t < t1 && !(g.cu && s >= g.N)) {
            const int lo = g.cu ? g.cu[s] : 0, hi = g.cu ? g.cu[s + 1] : g.T;
            const int a = t, end = min(t1, hi);
            if (end > a) {
                load_hist<T, W, V>(h, xr, x.t, a, lo, s0 ? s0 + (size_t)s * (W - 1) * g.C + c0 : nullptr, g.C);
#pragma unroll
                for (int k = 0; k < W; ++k)
#pragma unroll
                    for (int i = 0; i < P; ++i) dp[k][i] = two(0.f);
                const int stop = min(hi, end + W - 1);
                const T *px = xr + a * x.t, *pg = gr + a * dy.t;
                T *pd = dr + (long long)(a - (W - 1)) * dx.t;
                // one token: its dpre into ring place u, and dx W - 1 tokens back into o
                auto token = [&](const Vec<T, V> &in, const Vec<T, V> &gi, int u, bool sums, float2 (&o)[P]) {
                    float2 p[P], q[P];
                    get_pairs<T, V>(h[u % W], in);
                    get_pairs<T, V>(q, gi);
                    taps_at<W, V>(p, h, wt, bs, u);
                    if (g.silu) {
#pragma unroll
                        for (int i = 0; i < P; ++i) {
                            // silu' = s (1 + p (1 - s))
                            const float2 sg = sigmoid2(p[i]);
                            q[i] = mul2(mul2(q[i], sg), fma2(p[i], fma2(sg, two(-1.f), two(1.f)), two(1.f)));
                        }
                    }
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        if (sums) {
#pragma unroll
                            for (int k = 0; k < W; ++k) acc[k][i] = fma2(q[i], h[(u + 1 + k) % W][i], acc[k][i]);
                            acc[W][i] = add2(acc[W][i], q[i]);
                        }
                        dp[u % W][i] = q[i];
                        o[i] = mul2(wt[W - 1][i], dp[(u + 1) % W][i]);
#pragma unroll
                        for (int k = 1; k < W; ++k) o[i] = fma2(wt[W - 1 - k][i], dp[(u + 1 + k) % W][i], o[i]);
                    }
                };
                int tt = a;
                for (; tt + U <= end; tt += U) {
                    Vec<T, V> in[U], gi[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        in[u].load(px);
                        gi[u].load(pg);
                        px += x.t;
                        pg += dy.t;
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        float2 o[P];
                        token(in[u], gi[u], u, true, o);
                        if (u >= W - 1 || tt > a) {   // the first W - 1 tokens complete nothing of this run
                            Vec<T, V> out;
                            set_pairs<T, V>(out, o);
                            out.store(pd);
                        }
                        pd += dx.t;
                    }
                }
#pragma unroll 1
                for (; tt < end + W - 1; ++tt) {
                    Vec<T, V> in, gi;
                    in.zero();
                    gi.zero();
                    if (tt < stop) {
                        in.load(px);
                        gi.load(pg);
                    }
                    px += x.t;
                    pg += dy.t;
                    float2 o[P];
                    token(in, gi, 0, tt < end, o);
                    rotate<W, V>(h);
                    rotate<W, V>(dp);
                    const int tau = tt - (W - 1);
                    if (tau >= a) {
                        if (dsT && tau >= hi - (W - 1)) {
                            Vec<T, V> e;
                            float2 ef[P];
                            e.load(dsT + ((size_t)s * (W - 1) + (tau - hi + W - 1)) * g.C + c0);
                            get_pairs<T, V>(ef, e);
#pragma unroll
                            for (int i = 0; i < P; ++i) o[i] = add2(o[i], ef[i]);
                        }
                        Vec<T, V> out;
                        set_pairs<T, V>(out, o);
                        out.store(pd);
                    }
                    pd += dx.t;
                }
            }
            t = max(t, end);
            ++s;
        }
    }
#pragma unroll
    for (int k = 0; k <= W; ++k) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) red[threadIdx.y][threadIdx.x * V + i] = i & 1 ? acc[k][i / 2].y : acc[k][i / 2].x;
        __syncthreads();
        for (int i = threadIdx.y * kTX + threadIdx.x; i < kTX * V; i += kTX * kTY) {
            const long long c = (long long)(blockIdx.x % g.blocks_x) * kTX * V + i;
            if (c < g.C) {
                float sum = 0.f;
#pragma unroll
                for (int r = 0; r < kTY; ++r) sum += red[r][i];
                part[(row * (W + 1) + k) * g.C + c] = sum;
            }
        }
    }
}

// Gradient of the initial taps: tap i reaches tokens 0 .. i of its sequence
// (weight w[i - t]), and is itself a final tap where the sequence is shorter.
template <class T, int W>
__global__ void k_conv_ds0(ConvDims g, View<const T> x, View<const T> dy, const float *w, const float *bias, const T *s0,
                           const T *dsT, T *ds0)
{
    const long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x;
    if (i >= (long long)g.N * g.C) return;
    const int s = (int)(i / g.C), c = (int)(i - (long long)s * g.C), hd = c / g.d, j = c - hd * g.d;
    const int lo = g.cu ? g.cu[s] : 0, len = g.cu ? g.cu[s + 1] - lo : g.T;
    const int b = g.cu ? 0 : s;
    float ext[2 * W - 2], dp[W - 1];   // initial taps, then the first W - 1 tokens
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        ext[k] = s0 ? ld_in(s0 + ((size_t)s * (W - 1) + k) * g.C + c) : 0.f;
        ext[W - 1 + k] = k < len ? ld_in(x.at(b, hd, lo + k) + j) : 0.f;
    }
#pragma unroll
    for (int t = 0; t < W - 1; ++t) {
        dp[t] = 0.f;
        if (t < len) {
            float p = bias ? bias[c] : 0.f;
#pragma unroll
            for (int k = 0; k < W; ++k) p = fmaf(w[(size_t)c * W + k], ext[t + k], p);
            dp[t] = ld_in(dy.at(b, hd, lo + t) + j);
            if (g.silu) dp[t] *= dsilu(p, sigmoid(p));
        }
    }
#pragma unroll
    for (int q = 0; q < W - 1; ++q) {
        float o = 0.f;
#pragma unroll
        for (int t = 0; t <= q; ++t) o = fmaf(w[(size_t)c * W + q - t], dp[t], o);
        if (dsT && q >= len) o += ld_in(dsT + ((size_t)s * (W - 1) + q - len) * g.C + c);
        st_out(ds0 + ((size_t)s * (W - 1) + q) * g.C + c, o);
    }
}

// One token: taps and input in, output and moved taps out (state_out may be state_in:
// a thread reads its taps before it writes them).
template <class T, int W, int V>
__global__ void __launch_bounds__(128) k_conv_step(int N, int C, int d, int silu, View<const T> x, View<T> y,
                                                   const float *__restrict__ w, const float *__restrict__ bias,
                                                   const T *state_in, T *state_out)
{
    const int CV = C / V;
    const long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x;
    if (i >= (long long)N * CV) return;
    const int n = (int)(i / CV), c0 = (int)(i - (long long)n * CV) * V, hd = c0 / d, j = c0 - hd * d;
    Vec<T, V> v[W];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        if (state_in) v[k].load(state_in + ((size_t)n * (W - 1) + k) * C + c0);
        else v[k].zero();
    }
    v[W - 1].load(x.at(n, hd, 0) + j);
    constexpr int P = kPairs<V>;
    float2 wt[W][P], o[P];
    load_taps<W, V>(w, bias, c0, wt, o);
#pragma unroll
    for (int k = 0; k < W; ++k) {
        float2 f[P];
        get_pairs<T, V>(f, v[k]);
#pragma unroll
        for (int i = 0; i < P; ++i) o[i] = fma2(wt[k][i], f[i], o[i]);
    }
    if (silu) {
#pragma unroll
        for (int i = 0; i < P; ++i) o[i] = mul2(o[i], sigmoid2(o[i]));
    }
    Vec<T, V> out;
    set_pairs<T, V>(out, o);
    out.store(y.at(n, hd, 0) + j);
    if (state_out) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) v[k + 1].store(state_out + ((size_t)n * (W - 1) + k) * C + c0);
    }
}

// Tokens of a run: the longest power of two (forward 16..64, backward 16..512) that leaves
// the SMs enough blocks, for 8-byte vectors.  A longer run reads its W - 1 halo tokens and, in
// the backward, writes its partial sums less often; 4 blocks an SM forward (three run at once),
// 3/2 backward (two run at once: 256 tokens at 8 x 4096 x 2048 99 us, 128 tokens 105 us, 64 tokens 108 us).
int run_of(const dn_conv_shape *s, bool bwd)
{
    const long long vec = kBytes / (s->dtype == DN_F32 ? 4 : 2), need = (bwd ? 3ll : 8ll) * sm_count() / 2;
    const long long cols = ((long long)s->H * s->d / vec + kTX - 1) / kTX;
    int run = bwd ? 512 : 64;
    while (run > 16 && s->B * ((s->T + (long long)run * kTY - 1) / ((long long)run * kTY)) * cols < need) run >>= 1;
    return run;
}

long long rows_of(const dn_conv_shape *s, bool bwd)
{
    const long long run = run_of(s, bwd), runs = (s->T + run - 1) / run;
    return (long long)s->B * ((runs + kTY - 1) / kTY);
}

ConvDims dims_of(const dn_conv_shape *s, int N, const int32_t *cu, int V, bool bwd)
{
    ConvDims g;
    g.H = s->H; g.T = s->T; g.d = s->d; g.C = s->H * s->d; g.N = N; g.silu = s->silu; g.cu = cu;
    g.run = run_of(s, bwd);
    g.runs = (s->T + g.run - 1) / g.run;
    g.blocks_x = (g.C / V + kTX - 1) / kTX;
    g.rows = rows_of(s, bwd);
    return g;
}

// Vectors of `bytes` need every view, the taps and the states aligned to them, and heads that
// are whole vectors; one element otherwise.
template <class T>
bool vectors(const ConvCall &c, int bytes)
{
    const int e = sizeof(T), V = bytes / e;
    auto al = [](const void *p, int n) { return ((uintptr_t)p % n) == 0; };
    return c.s->d % V == 0 && can_vector(c.x, e, bytes) && can_vector(c.y, e, bytes) && can_vector(c.dy, e, bytes) &&
           can_vector(c.dx, e, bytes) && al(c.w, 16) && al(c.s0, bytes) && al(c.sT, bytes) && al(c.dsT, bytes) && al(c.ds0, bytes);
}

template <class T, int W, int V>
cudaError_t fwd_t(const ConvCall &c, cudaStream_t st)
{
    const ConvDims g = dims_of(c.s, c.N, c.cu, V, false);
    const View<const T> x = view_of<const T>(c.x);
    if (g.T > 0) {
        const long long blocks = g.rows * g.blocks_x;
        if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
        k_conv_fwd<T, W, V><<<(unsigned)blocks, dim3(kTX, kTY), 0, st>>>(g, x, view_of<T>(c.y), c.w, c.bias, (const T *)c.s0, (T *)c.sT);
    }
    if (c.sT && c.N > 0 && (g.cu || g.T == 0)) {
        const long long n = (long long)c.N * g.C;
        k_conv_empty<T><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(g, W - 1, (const T *)c.s0, (T *)c.sT);
    }
    return cudaPeekAtLastError();
}

template <class T, int W, int V>
cudaError_t bwd_t(const ConvCall &c, cudaStream_t st)
{
    const ConvDims g = dims_of(c.s, c.N, c.cu, V, true);
    const View<const T> x = view_of<const T>(c.x), dy = view_of<const T>(c.dy);
    if (g.T > 0) {
        const long long blocks = g.rows * g.blocks_x;
        if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
        k_conv_bwd<T, W, V><<<(unsigned)blocks, dim3(kTX, kTY), 0, st>>>(g, x, dy, view_of<T>(c.dx), c.w, c.bias,
                                                                        (const T *)c.s0, (const T *)c.dsT, c.part);
    }
    ColSum r;
    r.part = c.part;
    r.P = g.T > 0 ? g.rows : 0;
    r.kinds = W + 1;
    r.C = g.C;
    for (int k = 0; k < W; ++k) {
        r.dst[k] = c.dw + k;
        r.step[k] = W;
    }
    r.dst[W] = c.dbias;
    r.step[W] = 1;
    cudaError_t e = col_sum(r, nullptr, st);
    if (e != cudaSuccess) return e;
    if (c.ds0 && c.N > 0) {
        const long long n = (long long)c.N * g.C;
        k_conv_ds0<T, W><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(g, x, dy, c.w, c.bias, (const T *)c.s0,
                                                                      (const T *)c.dsT, (T *)c.ds0);
    }
    return cudaPeekAtLastError();
}

template <class T, int W, int V>
cudaError_t step_t(const ConvCall &c, cudaStream_t st)
{
    const int C = c.s->H * c.s->d;
    const long long n = (long long)c.s->B * (C / V);
    if ((n + 127) / 128 > 0x7fffffffLL) return cudaErrorInvalidValue;
    k_conv_step<T, W, V><<<(unsigned)((n + 127) / 128), 128, 0, st>>>(c.s->B, C, c.s->d, c.s->silu, view_of<const T>(c.x),
                                                                    view_of<T>(c.y), c.w, c.bias, (const T *)c.s0, (T *)c.sT);
    return cudaPeekAtLastError();
}

enum Op { kFwd, kBwd, kStep };

// The step, whose few bytes are all latency, takes 16-byte vectors where it can.
template <class T, int W>
cudaError_t by_vector(Op op, const ConvCall &c, cudaStream_t st)
{
    const int bytes = op == kStep ? 16 : kBytes;
    const bool v = vectors<T>(c, bytes);
    if (op == kBwd) return v ? bwd_t<T, W, kBytes / sizeof(T)>(c, st) : bwd_t<T, W, 1>(c, st);
    if (op == kFwd) return v ? fwd_t<T, W, kBytes / sizeof(T)>(c, st) : fwd_t<T, W, 1>(c, st);
    return v ? step_t<T, W, 16 / sizeof(T)>(c, st) : step_t<T, W, 1>(c, st);
}

template <class T>
cudaError_t by_width(Op op, const ConvCall &c, cudaStream_t st)
{
    switch (c.s->width) {
    case 2: return by_vector<T, 2>(op, c, st);
    case 3: return by_vector<T, 3>(op, c, st);
    case 4: return by_vector<T, 4>(op, c, st);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t run(Op op, const ConvCall &c, cudaStream_t st)
{
    return c.s->dtype == DN_F32 ? by_width<float>(op, c, st) : by_width<__nv_bfloat16>(op, c, st);
}

}  // namespace

long long conv_part_rows(const dn_conv_shape *s) { return rows_of(s, true); }

cudaError_t conv_fwd(const ConvCall &c, cudaStream_t st) { return run(kFwd, c, st); }
cudaError_t conv_bwd(const ConvCall &c, cudaStream_t st) { return run(kBwd, c, st); }
cudaError_t conv_step(const ConvCall &c, cudaStream_t st) { return run(kStep, c, st); }

}  // namespace lay
}  // namespace gdn

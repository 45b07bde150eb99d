// Short causal convolution, depthwise, 2..4 taps: forward, backward, one token.
//
//     pre[t][c] = bias[c] + sum_k w[c][k] x[t-(W-1)+k][c],   y = silu(pre) or pre
//     dpre = dy silu'(pre),  dx[t] = sum_k w[k] dpre[t+(W-1)-k],
//     dw[c][k] = sum_t dpre[t] x[t-(W-1)+k],  dbias = sum_t dpre[t]
//
// Bound by HBM: x read, y written (backward: x, dy read, dx written).  A thread
// owns V consecutive channels (16 bytes where strides and alignment allow, else
// one element) and walks a run of tokens with the last W - 1 inputs in registers,
// so that an input is read once plus W - 1 halo tokens a run; a warp covers 32
// neighbouring vectors of one token.
#include "layers.h"

namespace gdn {
namespace lay {

namespace {

constexpr int kTX = 32, kTY = 8;     // threads: channel vectors x runs

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

template <int W, int V>
__device__ __forceinline__ void load_taps(const float *w, const float *bias, int c0, float (&wt)[V][W], float (&bs)[V])
{
    if constexpr (V * W % 4 == 0 && V > 1) {
        float tmp[V * W];
        const float4 *p = reinterpret_cast<const float4 *>(w + (size_t)c0 * W);
#pragma unroll
        for (int i = 0; i < V * W / 4; ++i) {
            const float4 q = p[i];
            tmp[4 * i] = q.x; tmp[4 * i + 1] = q.y; tmp[4 * i + 2] = q.z; tmp[4 * i + 3] = q.w;
        }
#pragma unroll
        for (int i = 0; i < V * W; ++i) wt[i / W][i % W] = tmp[i];
    } else {
#pragma unroll
        for (int i = 0; i < V * W; ++i) wt[i / W][i % W] = w[(size_t)c0 * W + i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) bs[i] = bias ? bias[c0 + i] : 0.f;
}

// The W - 1 inputs before token t of a sequence [lo, ...): from x, or from the
// sequence's initial taps, or zero.
template <class T, int W, int V>
__device__ __forceinline__ void load_hist(float (&h)[W - 1][V], const T *xr, long long xt, int t, int lo, const T *s0,
                                          int C)
{
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        const int tt = t - (W - 1) + k;
        Vec<T, V> q;
        q.zero();
        if (tt >= lo) q.load(xr + tt * xt);
        else if (s0) q.load(s0 + (size_t)(W - 1 + tt - lo) * C);
        q.get(h[k]);
    }
}

template <class T, int W, int V>
__global__ void __launch_bounds__(kTX *kTY) k_conv_fwd(ConvDims g, View<const T> x, View<T> y, const float *__restrict__ w,
                                                       const float *__restrict__ bias, const T *__restrict__ s0)
{
    constexpr int U = 4;   // tokens whose loads are in flight together
    int cv, b, t0;
    long long row;
    if (!my_run<V>(g, cv, b, t0, row)) return;
    const int c0 = cv * V, hd = c0 / g.d, j = c0 - hd * g.d;
    const T *xr = x.at(b, hd, 0) + j;
    T *yr = y.at(b, hd, 0) + j;
    float wt[V][W], bs[V], h[W - 1][V];
    load_taps<W, V>(w, bias, c0, wt, bs);
    int t = t0;
    const int t1 = min(t0 + g.run, g.T);
    int s = g.cu ? seq_at(g.cu, g.N, t0) : b;
    while (t < t1) {
        if (g.cu && s >= g.N) return;
        const int lo = g.cu ? g.cu[s] : 0, hi = g.cu ? g.cu[s + 1] : g.T;
        const int end = min(t1, hi);
        if (end > t) load_hist<T, W, V>(h, xr, x.t, t, lo, s0 ? s0 + (size_t)s * (W - 1) * g.C + c0 : nullptr, g.C);
        for (; t < end; t += U) {
            Vec<T, V> in[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (t + u < end) in[u].load(xr + (t + u) * x.t);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t + u < end) {
                    float f[V], o[V];
                    in[u].get(f);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        float a = bs[i];
#pragma unroll
                        for (int k = 0; k < W - 1; ++k) a = fmaf(wt[i][k], h[k][i], a);
                        a = fmaf(wt[i][W - 1], f[i], a);
                        o[i] = g.silu ? a * sigmoid(a) : a;
                    }
#pragma unroll
                    for (int i = 0; i < V; ++i) {
#pragma unroll
                        for (int k = 0; k + 1 < W - 1; ++k) h[k][i] = h[k + 1][i];
                        h[W - 2][i] = f[i];
                    }
                    Vec<T, V> out;
                    out.set(o);
                    out.store(yr + (t + u) * y.t);
                }
            }
        }
        t = end;
        ++s;
    }
}

// Final taps: the last W - 1 inputs of every sequence, its initial taps in front.
template <class T, int W>
__global__ void k_conv_state(ConvDims g, View<const T> x, const T *s0, T *sT)
{
    const long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x;
    if (i >= (long long)g.N * g.C) return;
    const int s = (int)(i / g.C), c = (int)(i - (long long)s * g.C), hd = c / g.d;
    const int lo = g.cu ? g.cu[s] : 0, len = g.cu ? g.cu[s + 1] - lo : g.T;
    const T *xr = x.at(g.cu ? 0 : s, hd, 0) + (c - hd * g.d);
    T v[W - 1];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        const int q = len + k - (W - 1);   // token of the sequence, negative: an initial tap
        if (q >= 0) v[k] = xr[(long long)(lo + q) * x.t];
        else if (s0) v[k] = s0[((size_t)s * (W - 1) + len + k) * g.C + c];
        else st_out(&v[k], 0.f);
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k) sT[((size_t)s * (W - 1) + k) * g.C + c] = v[k];
}

// Backward.  For the run's tokens t0 .. t1-1 and the W - 1 behind them (of the same
// sequence) the thread computes dpre once, keeps the last W of them, and writes
// dx of the token W - 1 back, whose sum is then complete.  dw and dbias sum over
// the run in registers, over the block's kTY runs in shared memory, and over
// blocks in col_sum: no atomics, one fixed order.
template <class T, int W, int V>
__global__ void __launch_bounds__(kTX *kTY) k_conv_bwd(ConvDims g, View<const T> x, View<const T> dy, View<T> dx,
                                                       const float *__restrict__ w, const float *__restrict__ bias,
                                                       const T *__restrict__ s0, const T *__restrict__ dsT,
                                                       float *__restrict__ part)
{
    constexpr int U = 4;
    __shared__ float red[kTY][kTX * V];
    int cv, b, t0;
    long long row;
    const bool live = my_run<V>(g, cv, b, t0, row);
    float acc[W + 1][V];
#pragma unroll
    for (int k = 0; k <= W; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[k][i] = 0.f;
    if (live) {
        const int c0 = cv * V, hd = c0 / g.d, j = c0 - hd * g.d;
        const T *xr = x.at(b, hd, 0) + j, *gr = dy.at(b, hd, 0) + j;
        T *dr = dx.at(b, hd, 0) + j;
        float wt[V][W], bs[V], h[W - 1][V], dp[W][V];
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
                    for (int i = 0; i < V; ++i) dp[k][i] = 0.f;
                const int stop = min(hi, end + W - 1);
                for (int tb = a; tb < end + W - 1; tb += U) {
                    Vec<T, V> in[U], gi[U];
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (tb + u < stop) {
                            in[u].load(xr + (tb + u) * x.t);
                            gi[u].load(gr + (tb + u) * dy.t);
                        }
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int tt = tb + u;
                        if (tt < end + W - 1) {
                            float f[V], q[V], o[V];
                            if (tt < stop) {
                                in[u].get(f);
                                gi[u].get(q);
                            } else {
#pragma unroll
                                for (int i = 0; i < V; ++i) f[i] = q[i] = 0.f;
                            }
#pragma unroll
                            for (int i = 0; i < V; ++i) {
                                float p = bs[i];
#pragma unroll
                                for (int k = 0; k < W - 1; ++k) p = fmaf(wt[i][k], h[k][i], p);
                                p = fmaf(wt[i][W - 1], f[i], p);
                                if (g.silu && tt < stop) q[i] *= dsilu(p, sigmoid(p));
                                if (tt < end) {
#pragma unroll
                                    for (int k = 0; k < W - 1; ++k) acc[k][i] = fmaf(q[i], h[k][i], acc[k][i]);
                                    acc[W - 1][i] = fmaf(q[i], f[i], acc[W - 1][i]);
                                    acc[W][i] += q[i];
                                }
#pragma unroll
                                for (int k = 0; k + 1 < W; ++k) dp[k][i] = dp[k + 1][i];
                                dp[W - 1][i] = q[i];
#pragma unroll
                                for (int k = 0; k + 1 < W - 1; ++k) h[k][i] = h[k + 1][i];
                                h[W - 2][i] = f[i];
                                o[i] = 0.f;
#pragma unroll
                                for (int k = 0; k < W; ++k) o[i] = fmaf(wt[i][W - 1 - k], dp[k][i], o[i]);
                            }
                            const int tau = tt - (W - 1);
                            if (tau >= a) {
                                if (dsT && tau >= hi - (W - 1)) {
                                    Vec<T, V> e;
                                    float ef[V];
                                    e.load(dsT + ((size_t)s * (W - 1) + (tau - hi + W - 1)) * g.C + c0);
                                    e.get(ef);
#pragma unroll
                                    for (int i = 0; i < V; ++i) o[i] += ef[i];
                                }
                                Vec<T, V> out;
                                out.set(o);
                                out.store(dr + tau * dx.t);
                            }
                        }
                    }
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
        for (int i = 0; i < V; ++i) red[threadIdx.y][threadIdx.x * V + i] = acc[k][i];
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
    float wt[V][W], o[V];
    load_taps<W, V>(w, bias, c0, wt, o);
#pragma unroll
    for (int k = 0; k < W; ++k) {
        float f[V];
        v[k].get(f);
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = fmaf(wt[e][k], f[e], o[e]);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = silu ? o[e] * sigmoid(o[e]) : o[e];
    Vec<T, V> out;
    out.set(o);
    out.store(y.at(n, hd, 0) + j);
    if (state_out) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) v[k + 1].store(state_out + ((size_t)n * (W - 1) + k) * C + c0);
    }
}

int run_of(const dn_conv_shape *s) { (void)s; return 64; }

ConvDims dims_of(const dn_conv_shape *s, int N, const int32_t *cu, int V)
{
    ConvDims g;
    g.H = s->H; g.T = s->T; g.d = s->d; g.C = s->H * s->d; g.N = N; g.silu = s->silu; g.cu = cu;
    g.run = run_of(s);
    g.runs = (s->T + g.run - 1) / g.run;
    g.blocks_x = (g.C / V + kTX - 1) / kTX;
    g.rows = conv_part_rows(s);
    return g;
}

// 16-byte vectors need every view, the taps and the states aligned to them, and heads
// that are whole vectors; one element otherwise.
template <class T>
bool vectors(const ConvCall &c)
{
    constexpr int V = 16 / sizeof(T);
    const int e = sizeof(T);
    auto al = [](const void *p) { return ((uintptr_t)p & 15u) == 0; };
    return c.s->d % V == 0 && can_vector(c.x, e, 16) && can_vector(c.y, e, 16) && can_vector(c.dy, e, 16) &&
           can_vector(c.dx, e, 16) && al(c.w) && al(c.s0) && al(c.sT) && al(c.dsT) && al(c.ds0);
}

template <class T, int W, int V>
cudaError_t fwd_t(const ConvCall &c, cudaStream_t st)
{
    const ConvDims g = dims_of(c.s, c.N, c.cu, V);
    const View<const T> x = view_of<const T>(c.x);
    if (g.T > 0) {
        const long long blocks = g.rows * g.blocks_x;
        if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
        k_conv_fwd<T, W, V><<<(unsigned)blocks, dim3(kTX, kTY), 0, st>>>(g, x, view_of<T>(c.y), c.w, c.bias, (const T *)c.s0);
    }
    if (c.sT && c.N > 0) {
        const long long n = (long long)c.N * g.C;
        k_conv_state<T, W><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(g, x, (const T *)c.s0, (T *)c.sT);
    }
    return cudaPeekAtLastError();
}

template <class T, int W, int V>
cudaError_t bwd_t(const ConvCall &c, cudaStream_t st)
{
    const ConvDims g = dims_of(c.s, c.N, c.cu, V);
    const View<const T> x = view_of<const T>(c.x), dy = view_of<const T>(c.dy);
    if (g.T > 0) {
        const long long blocks = g.rows * g.blocks_x;
        if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
        k_conv_bwd<T, W, V><<<(unsigned)blocks, dim3(kTX, kTY), 0, st>>>(g, x, dy, view_of<T>(c.dx), c.w, c.bias,
                                                                        (const T *)c.s0, (const T *)c.dsT, c.part);
    }
    ColSum r;
    r.kinds = W + 1;
    r.C = g.C;
    for (int k = 0; k < W; ++k) {
        r.dst[k] = c.dw + k;
        r.step[k] = W;
    }
    r.dst[W] = c.dbias;
    r.step[W] = 1;
    cudaError_t e = col_sum(c.part, g.T > 0 ? g.rows : 0, r, st);
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

template <class T, int W, int V>
cudaError_t op_t(Op op, const ConvCall &c, cudaStream_t st)
{
    return op == kFwd ? fwd_t<T, W, V>(c, st) : op == kBwd ? bwd_t<T, W, V>(c, st) : step_t<T, W, V>(c, st);
}

template <class T>
cudaError_t by_width(Op op, const ConvCall &c, cudaStream_t st)
{
    constexpr int V = 16 / sizeof(T);
    const bool v = vectors<T>(c);
    switch (c.s->width) {
    case 2: return v ? op_t<T, 2, V>(op, c, st) : op_t<T, 2, 1>(op, c, st);
    case 3: return v ? op_t<T, 3, V>(op, c, st) : op_t<T, 3, 1>(op, c, st);
    case 4: return v ? op_t<T, 4, V>(op, c, st) : op_t<T, 4, 1>(op, c, st);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t run(Op op, const ConvCall &c, cudaStream_t st)
{
    return c.s->dtype == DN_F32 ? by_width<float>(op, c, st) : by_width<__nv_bfloat16>(op, c, st);
}

}  // namespace

long long conv_part_rows(const dn_conv_shape *s)
{
    const long long runs = ((long long)s->T + run_of(s) - 1) / run_of(s);
    return (long long)s->B * ((runs + kTY - 1) / kTY);
}

cudaError_t conv_fwd(const ConvCall &c, cudaStream_t st) { return run(kFwd, c, st); }
cudaError_t conv_bwd(const ConvCall &c, cudaStream_t st) { return run(kBwd, c, st); }
cudaError_t conv_step(const ConvCall &c, cudaStream_t st) { return run(kStep, c, st); }

}  // namespace lay
}  // namespace gdn

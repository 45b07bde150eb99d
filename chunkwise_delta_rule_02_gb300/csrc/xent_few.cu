// Linear softmax cross entropy of few tokens, on the CUDA cores: up to 16 in float32, up to 4 in bf16 where the width is no multiple of 8
// (16 up to 512 features) or at most 512.
//
// Tiles of 256 tokens would be empty rows, and float32 operands three planes copied from a weight that is read once
// anyway.  Here a block has a contiguous share of the vocabulary and x in shared memory; a warp takes 4 or 8 entries at
// a time, lanes along the features, 32 or 64 sums a lane.  Backward, one pass over w: of every 64 entries first D (the logits
// again), then, a feature a thread, dw = sum_m D x and dx += sum_v D w, dx' sums in shared memory until the end, and of
// all blocks joined in a fixed order.  Everything is float32: D is not rounded.  w is read once from HBM (the second time, 64
// entries later, from a cache), dw written once.
//
// Bound by arithmetic and HBM about alike: 6 MT operations an element of w at 71 TFLOP/s against 8 bytes of float32.
#include "xent.cuh"

namespace gdn {
namespace xent {

namespace {

constexpr int kFewThreads = 256, kFewWarps = kFewThreads / 32, kFewRows = 64;
// threads of a backward block: 16 tokens leave room for one block an SM only
__host__ __device__ constexpr int bwd_threads(int MT) { return MT == 16 ? 512 : 256; }
// entries that a warp takes at a time, and steps along the features whose loads are in flight together
__host__ __device__ constexpr int at_once(int MT) { return MT == 16 ? 4 : 8; }
constexpr int kStepsAtOnce = 4;
constexpr int kFewShared = 200 << 10;   // bytes

struct Few {
    Gemm g;
    int M, K, V, share;             // share: entries of a block
    const void *x, *w;
    long long x_b, x_t, w_t;
    void *dw;
    float *dx;                      // [blocks][M][K]
};

// MASK: 0 for a token without a target, whose weight is 0 in dw whatever it holds
template <class T, int MT, bool MASK>
__device__ __forceinline__ void load_x(const Few &p, float *xs)
{
    for (int i = threadIdx.x; i < MT * p.K; i += blockDim.x) {
        const int m = i / p.K, k = i - m * p.K;
        xs[i] = m < p.M && (!MASK || target_of(p.g, m, false) >= 0) ? ld_in((const T *)p.x + (long long)(m / p.g.T) * p.x_b + (long long)(m % p.g.T) * p.x_t + k) : 0.f;
    }
}

// The logits of entries row .. row + at_once(MT) - 1 (those at or behind `end` are read as the one before it): value 32 g + lane, which is entry
// row + value / MT and token value % MT, in v[g].
template <class T, int MT>
__device__ __forceinline__ void logits(const Few &p, const float *xs, int row, int end, float (&v)[(at_once(MT) * MT + 31) / 32])
{
    constexpr int kAtOnce = at_once(MT), G = (kAtOnce * MT + 31) / 32;
    const int lane = threadIdx.x & 31;
    const T *w[kAtOnce];
#pragma unroll
    for (int r = 0; r < kAtOnce; ++r) w[r] = (const T *)p.w + (long long)min(row + r, end - 1) * p.w_t;
    float acc[G * 32] = {};
#pragma unroll kStepsAtOnce
    for (int k = lane; k < p.K; k += 32) {
        float f[kAtOnce];
#pragma unroll
        for (int r = 0; r < kAtOnce; ++r) f[r] = ld_in(w[r] + k);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const float x = xs[m * p.K + k];
#pragma unroll
            for (int r = 0; r < kAtOnce; ++r) acc[r * MT + m] = fmaf(f[r], x, acc[r * MT + m]);
        }
    }
    // sums over the lanes by halving: value i ends in lane i
#pragma unroll
    for (int g = 0; g < G; ++g) {
#pragma unroll
        for (int h = 16; h > 0; h >>= 1) {
            const bool up = lane & h;
#pragma unroll
            for (int i = 0; i < h; ++i) {
                const float send = up ? acc[32 * g + i] : acc[32 * g + i + h], keep = up ? acc[32 * g + i + h] : acc[32 * g + i];
                acc[32 * g + i] = keep + __shfl_xor_sync(0xffffffffu, send, h);
            }
        }
        v[g] = acc[32 * g];
    }
}

template <class T, int MT>
__global__ void __launch_bounds__(kFewThreads, 2) k_few_fwd(const __grid_constant__ Few p)
{
    extern __shared__ float xs[];
    __shared__ float2 sm[kFewWarps][MT];
    constexpr int kAtOnce = at_once(MT), N = kAtOnce * MT, G = (N + 31) / 32;
    let_next_start();
    wait_for_last();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, token = lane % MT;
    const int begin = blockIdx.x * p.share, end = min(p.V, begin + p.share);
    load_x<T, MT, false>(p, xs);
    const int target = token < p.M ? target_of(p.g, token, blockIdx.x == 0 && threadIdx.x < MT) : -1;
    __syncthreads();
    float mx = kNone, sum = 0.f;
    auto join = [&](float2 q) {
        const float top = fmaxf(mx, q.x);
        sum = sum * exp2f((mx - top) * kLog2e) + q.y * exp2f((q.x - top) * kLog2e);
        mx = top;
    };
    for (int row = begin + warp * kAtOnce; row < end; row += kFewWarps * kAtOnce) {
        float v[G];
        logits<T, MT>(p, xs, row, end, v);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int id = 32 * g + lane, r = row + id / MT;
            if (id < N && r < end) {
                if (r == target) p.g.row[token] = v[g];
                const float top = fmaxf(mx, v[g]);
                sum = fmaf(sum, ex2((mx - top) * kLog2e), ex2((v[g] - top) * kLog2e));
                mx = top;
            }
        }
    }
#pragma unroll
    for (int d = MT; d < 32; d *= 2) join(make_float2(__shfl_xor_sync(0xffffffffu, mx, d), __shfl_xor_sync(0xffffffffu, sum, d)));
    if (lane < MT) sm[warp][lane] = make_float2(mx, sum);
    __syncthreads();
    if (threadIdx.x < p.M) {
        mx = kNone;
        sum = 0.f;
        for (int w = 0; w < kFewWarps; ++w) join(sm[w][threadIdx.x]);
        p.g.part[(long long)blockIdx.x * p.M + threadIdx.x] = make_float2(mx, sum);
    }
}

template <class T, int MT>
__global__ void __launch_bounds__(bwd_threads(MT), MT == 16 ? 1 : 2) k_few_bwd(const __grid_constant__ Few p)
{
    extern __shared__ float xs[];   // x, then dx' sums, both [MT][K]
    __shared__ __align__(16) float D[kFewRows][MT];
    constexpr int kThreads = bwd_threads(MT), kWarps = kThreads / 32, kAtOnce = at_once(MT), N = kAtOnce * MT, G = (N + 31) / 32;
    let_next_start();
    wait_for_last();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, token = lane % MT;
    const int begin = blockIdx.x * p.share, end = min(p.V, begin + p.share);
    float *sums = xs + MT * p.K;
    load_x<T, MT, true>(p, xs);
    for (int i = threadIdx.x; i < MT * p.K; i += kThreads) sums[i] = 0.f;
    int target = -1;
    float lse = 0.f, dl = 0.f;
    if (token < p.M) {
        target = target_of(p.g, token, blockIdx.x == 0 && threadIdx.x < MT);
        lse = p.g.lse[token];
        if (target >= 0) dl = p.g.dloss[(long long)(token / p.g.T) * p.g.g_b + (long long)(token % p.g.T) * p.g.g_t];
    }
    __syncthreads();
    for (int row0 = begin; row0 < end; row0 += kFewRows) {
        const int n = min(kFewRows, end - row0);
        for (int row = row0 + warp * kAtOnce; row < row0 + kFewRows; row += kWarps * kAtOnce) {
            float v[G] = {};
            if (row < end) logits<T, MT>(p, xs, row, end, v);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int id = 32 * g + lane, r = row + id / MT;
                if (id < N) D[r - row0][token] = target >= 0 && r < end ? (ex2((v[g] - lse) * kLog2e) - (r == target ? 1.f : 0.f)) * dl : 0.f;
            }
        }
        __syncthreads();
        for (int k = threadIdx.x; k < p.K; k += kThreads) {
            float x[MT], dx[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                x[m] = xs[m * p.K + k];
                dx[m] = sums[m * p.K + k];
            }
            const T *w = (const T *)p.w + (long long)row0 * p.w_t + k;
            T *dw = (T *)p.dw + (long long)row0 * p.K + k;
#pragma unroll 8
            for (int r = 0; r < n; ++r) {
                const float f = ld_in(w + r * p.w_t);
                float s = 0.f;
#pragma unroll
                for (int m = 0; m < MT; m += 4) {
                    const float4 d = *reinterpret_cast<const float4 *>(&D[r][m]);
                    s = fmaf(d.x, x[m], fmaf(d.y, x[m + 1], fmaf(d.z, x[m + 2], fmaf(d.w, x[m + 3], s))));
                    dx[m] = fmaf(d.x, f, dx[m]);
                    dx[m + 1] = fmaf(d.y, f, dx[m + 1]);
                    dx[m + 2] = fmaf(d.z, f, dx[m + 2]);
                    dx[m + 3] = fmaf(d.w, f, dx[m + 3]);
                }
                st_out(dw + (long long)r * p.K, s);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) sums[m * p.K + k] = dx[m];
        }
        __syncthreads();
    }
    float *out = p.dx + (long long)blockIdx.x * p.M * p.K;
    for (int i = threadIdx.x; i < p.M * p.K; i += kThreads) out[i] = sums[i];
}

// dx from the blocks' sums: one block 32 elements, a warp every 8th of the blocks; then those 8 in a fixed order.
template <class T>
__global__ void __launch_bounds__(kFewThreads) k_few_dx(const __grid_constant__ Product o)
{
    __shared__ float sm[kFewWarps][32];
    let_next_start();
    wait_for_last();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, all = o.M * o.N, i = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (i < all) {
#pragma unroll 8
        for (int c = warp; c < o.cuts; c += kFewWarps) v += o.part[(long long)c * all + i];
    }
    sm[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && i < all) {
        for (int w = 1; w < kFewWarps; ++w) v += sm[w][lane];
        const int m = i / o.N;
        st_out((T *)o.out + (long long)(m / o.T) * o.out_b + (long long)(m % o.T) * o.out_t + (i - m * o.N), v);
    }
}

int padded(int M) { return M <= 4 ? 4 : M <= 8 ? 8 : 16; }
size_t shared_of(int M, int K, bool bwd) { return (size_t)padded(M) * K * sizeof(float) * (bwd ? 2 : 1); }

Few few_of(const Call &c, bool bwd)
{
    Few p;
    p.g = common(c);
    p.M = c.M; p.K = c.K; p.V = c.V;
    const int blocks = few_blocks(c.M, c.K, c.V, bwd);
    p.share = (c.V + blocks - 1) / blocks;
    p.x = c.x->data; p.x_b = c.x->batch; p.x_t = c.x->time;
    p.w = c.w->data; p.w_t = c.w->time;
    p.dw = c.dw;
    p.dx = c.cut;
    return p;
}

// Calls f with the kernel's types: the input's and the number of tokens
template <class F>
cudaError_t variant(const Call &c, F f)
{
    const int mt = padded(c.M);
    auto of = [&](auto *t) {
        return mt == 4 ? f(t, std::integral_constant<int, 4>{}) : mt == 8 ? f(t, std::integral_constant<int, 8>{}) : f(t, std::integral_constant<int, 16>{});
    };
    return c.s->dtype == DN_F32 ? of((float *)nullptr) : of((__nv_bfloat16 *)nullptr);
}

}  // namespace

// bf16, us forward and backward with the tensor cores and so, measured side by side:
//   widths that they read in place, 4 tokens of 131072 x 4096: 170, 686 and 356, 2129; 50000 x 1024: 28, 95 and 52, 116;
//     32000 x 512: 18, 45 and 18, 42; 1000 x 64: 17, 29 and 12, 14 (launches);
//   widths that they need copies for, 69380 x 1591: of 4 tokens 136, 342 and 94, 278, of 5 136, 342 and 140, 334, of 16 137, 348 and 183, 405;
//     5003 x 203: of 5 tokens 21, 33 and 14, 16, of 16 21, 35 and 16, 20.
// The same for both directions: a logit's sum is what the backward's has to repeat, and the tensor cores round otherwise.
bool few_tokens(int M, int K, bool f32)
{
    const int most = f32 ? 16 : K % 8 ? (K <= 512 ? 16 : 4) : K <= 512 ? 4 : 0;
    return M >= 1 && M <= most && shared_of(M, K, true) <= kFewShared;
}

int few_blocks(int M, int K, int V, bool bwd)
{
    const size_t room = shared_of(M, K, bwd) + 6144;
    const int resident = room > (110 << 10) || (bwd && padded(M) == 16) ? 1 : 2;
    const long long rows = bwd ? kFewRows : kFewWarps * at_once(padded(M)), need = (V + rows - 1) / rows, most = (long long)resident * lay::sm_count();
    const int blocks = (int)(need < most ? need : most), share = (V + blocks - 1) / blocks;
    return (V + share - 1) / share;
}

cudaError_t few_forward(const Call &c, cudaStream_t st)
{
    const Few p = few_of(c, false);
    const int blocks = few_blocks(c.M, c.K, c.V, false);
    const cudaError_t e = variant(c, [&](auto *t, auto mt) {
        auto kernel = k_few_fwd<std::remove_pointer_t<decltype(t)>, decltype(mt)::value>;
        const int smem = (int)shared_of(c.M, c.K, false);
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        return e != cudaSuccess ? e : start(kernel, blocks, kFewThreads, smem, st, p);
    });
    return e != cudaSuccess ? e : join_rows(p.g, c, blocks, st);
}

cudaError_t few_backward(const Call &c, cudaStream_t st)
{
    const Few p = few_of(c, true);
    const int blocks = few_blocks(c.M, c.K, c.V, true);
    const cudaError_t e = variant(c, [&](auto *t, auto mt) {
        auto kernel = k_few_bwd<std::remove_pointer_t<decltype(t)>, decltype(mt)::value>;
        const int smem = (int)shared_of(c.M, c.K, true);
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        return e != cudaSuccess ? e : start(kernel, blocks, bwd_threads(decltype(mt)::value), smem, st, p);
    });
    if (e != cudaSuccess) return e;
    Product o = {};
    o.M = c.M;
    o.N = c.K;
    o.cuts = blocks;
    o.part = c.cut;
    o.out = c.dx->data;
    o.out_b = c.dx->batch;
    o.out_t = c.dx->time;
    o.T = c.s->T;
    const int groups = (c.M * c.K + 31) / 32;
    return c.s->dtype == DN_F32 ? start(k_few_dx<float>, groups, kFewThreads, 0, st, o) : start(k_few_dx<__nv_bfloat16>, groups, kFewThreads, 0, st, o);
}

}  // namespace xent
}  // namespace gdn

// Linear softmax cross entropy without the logits: l = x w^T, lse = log sum_v exp l_v,
// loss = lse - l[target]; backward, by pieces of the vocabulary, D = (exp(l - lse) - onehot) dloss,
// dx = sum over pieces D w, dw = D^T x.
//
// k_gemm is the one matrix product: C = A B^T in tiles of 256 x 256 by a pair of CTAs (tcgen05.mma, cta_group::2), each holding 128
// of the tile's rows in TMEM and loading half of both operands by TMA into a ring of stages.  A and B are K-major or
// MN-major in memory, so that all four products run on x, w and D as they lie.  Warp 0 loads, warp 1 of the even CTA issues the
// MMAs, eight warps take the finished tile from TMEM while the next one is computed in the other half of it.  What they do with it:
//   STATS  maximum and sum of exponentials of a row over 128 columns, and the target's logit;
//   GRAD   D, rounded to the operand's type for the two products that read it;
//   OUT    the tile itself, added to what earlier pieces gave.
// D in bf16 (2^-9 of each value) is what a bf16 input's gradient is computed from: the sums over the vocabulary and over the tokens
// are float32.  float32 inputs are split into three bf16 planes, 8 bits each, and six of their nine products kept: what is
// left out is 2^-24 of the whole.
#include "pair.cuh"
#include "xent.h"

namespace gdn {
namespace xent {

namespace {

using namespace sm100;
using lay::ex2;
using lay::kLog2e;

constexpr int TILE = 256, HALF = 128, BK = 64, STAGES = 6, THREADS = 320, EPI_WARPS = 8;
constexpr int OPERAND = HALF * BK * 2, STAGE = 2 * OPERAND;          // bytes a CTA loads: of one operand, of both
constexpr int SMEM = STAGES * STAGE + 1024 + 256;
constexpr long long BUDGET = 4000000000LL;                           // clock cycles (about 2 s) for any one wait
constexpr int GROUP = 16;                                            // row tiles that share the column tiles of a wave
constexpr float kNone = -1e30f;                                      // maximum of no logits

// Steps after which float32 inputs' sums leave TMEM: the tensor core cuts what it adds off rather than rounding it, the same way each
// time, which a contraction of 70001 tokens added up to 8e-5 of dw; segments of 1024 are summed in registers, rounded.
constexpr int kSegment = 16;

enum { STATS, GRAD, OUT };

struct Gemm {
    int M, N;                       // rows and columns of C that exist
    int mt, nt, kb;                 // tiles; 64-wide steps of the contraction
    int b_row, b_k;                 // where B's rows and its contraction begin
    int seg;                        // steps of a segment: kb, or kSegment (SEG)
    int np;                         // plane products: nibbles of pa, pb
    uint32_t pa, pb;
    uint32_t *status;
    // STATS, GRAD
    const int32_t *tgt;
    const float *lse, *g;
    float *row;
    float2 *part;
    __nv_bfloat16 *d;
    long long d_pitch, d_plane;
    int v0, planes;
    // OUT
    const float *add;               // [M][N] or null
    float *sum;                     // [M][N], or null: out
    void *out;
    long long out_b, out_t;         // row (b, t) of out at b out_b + t out_t
    int T, f32;
};

enum { FULL = 0, EMPTY = STAGES, TFULL = 2 * STAGES, TEMPTY = TFULL + 2, DONE = TEMPTY + 2, NBAR = DONE + 1 };

template <bool A_MN, bool B_MN, int EPI, bool SEG>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    k_gemm(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb, const Gemm p)
{
    extern __shared__ char raw[];
    char *sm = (char *)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    uint64_t *bar = (uint64_t *)(sm + STAGES * STAGE);
    uint32_t *s_tmem = (uint32_t *)(bar + NBAR);
    volatile int *s_abort = (volatile int *)(s_tmem + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = pair_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1, tiles = p.mt * p.nt;

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&bar[FULL + i], 1);
            mbar_init(&bar[EMPTY + i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar[TFULL + i], 1);
            mbar_init(&bar[TEMPTY + i], 2 * EPI_WARPS);
        }
        mbar_init(&bar[DONE], 1);
        *s_abort = 0;
        fence_barrier_init();
        prefetch_tmap(&ta);
        prefetch_tmap(&tb);
    }
    if (warp == 1) {
        pair_tmem_alloc(s_tmem, 512);
        pair_tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    pair_sync();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    auto wait = [&](int b, uint32_t parity) -> bool {
        if (pair_wait(&bar[b], parity & 1u, BUDGET, s_abort)) return true;
        *s_abort = 1;
        raise_status(p.status, kStatusTimeout);
        return false;
    };
    auto place = [&](int tile, int &m, int &n) {
        const int per = GROUP * p.nt, grp = tile / per, r = tile - grp * per, gm = min(GROUP, p.mt - grp * GROUP);
        m = (grp * GROUP + r % gm) * TILE;
        n = r / gm * TILE;
    };
    const int segs = SEG ? (p.kb + p.seg - 1) / p.seg : 1;

    if (warp == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int tile = pair; ok && tile < tiles; tile += pairs) {
                int m, n;
                place(tile, m, n);
                m += rank * HALF;
                n += rank * HALF;
                for (int sq = 0; ok && sq < segs * p.np; ++sq) {
                    const int seg = sq / p.np, q = sq - seg * p.np;
                    const int a = p.pa >> 4 * q & 15, b = p.pb >> 4 * q & 15, end = min(p.kb, (seg + 1) * p.seg);
                    for (int k = seg * p.seg; k < end; ++k, ++it) {
                        const int s = it % STAGES;
                        if (!(ok = wait(EMPTY + s, it / STAGES + 1))) break;
                        const uint32_t full = peer_addr(&bar[FULL + s], 0);
                        char *sa = sm + s * STAGE, *sb = sa + OPERAND;
                        if (rank == 0) mbar_expect_tx(&bar[FULL + s], 2 * STAGE);
                        if (A_MN) {
                            pair_load_3d(sa, &ta, full, m, k * BK, a);
                            pair_load_3d(sa + OPERAND / 2, &ta, full, m + 64, k * BK, a);
                        } else {
                            pair_load_3d(sa, &ta, full, k * BK, m, a);
                        }
                        if (B_MN) {
                            pair_load_3d(sb, &tb, full, n, p.b_k + k * BK, b);
                            pair_load_3d(sb + OPERAND / 2, &tb, full, n + 64, p.b_k + k * BK, b);
                        } else {
                            pair_load_3d(sb, &tb, full, k * BK, p.b_row + n, b);
                        }
                    }
                }
            }
            // the last loads into each stage have landed, and been read, before shared memory goes away; where a wait
            // ran out nothing reads them any more, and they have the time that a load takes many times over
            volatile int never = 0;
            for (uint32_t j = it > STAGES ? it - STAGES : 0; j < it; ++j)
                pair_wait(&bar[EMPTY + j % STAGES], (j / STAGES) & 1u, ok ? BUDGET : BUDGET / 100, &never);
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            constexpr uint32_t id = idesc(1, TILE, TILE, A_MN, B_MN);
            constexpr uint32_t astep = A_MN ? 2048 : 32, bstep = B_MN ? 2048 : 32;
            uint32_t it = 0, n = 0;
            bool ok = true;
            for (int tile = pair; ok && tile < tiles; tile += pairs) {
                for (int seg = 0; ok && seg < segs; ++seg, ++n) {
                    const uint32_t acc = tmem + (n & 1) * TILE;
                    if (!(ok = wait(TEMPTY + (n & 1), (n >> 1) + 1))) break;
                    tc_fence_after();
                    const int steps = p.np * (min(p.kb, (seg + 1) * p.seg) - seg * p.seg);
                    for (int k = 0; k < steps; ++k, ++it) {
                        const int s = it % STAGES;
                        if (!(ok = wait(FULL + s, it / STAGES))) break;
                        tc_fence_after();
                        const uint32_t sa = smem_u32(sm + s * STAGE), sb = sa + OPERAND;
#pragma unroll
                        for (int j = 0; j < BK / 16; ++j)
                            pair_mma_bf16(acc, sdesc(sa + j * astep, A_MN ? OPERAND / 2 : 16, 1024),
                                          sdesc(sb + j * bstep, B_MN ? OPERAND / 2 : 16, 1024), id, k > 0 || j > 0);
                        pair_commit(&bar[EMPTY + s]);
                    }
                    if (ok) pair_commit(&bar[TFULL + (n & 1)]);
                }
            }
            // no MMA is in flight when TMEM is freed, also where a wait ran out
            volatile int never = 0;
            pair_commit(&bar[DONE]);
            pair_wait(&bar[DONE], 0, BUDGET, &never);
        }
    } else {
        const int e = warp - 2, quad = warp & 3, half = e >> 2;   // TMEM lanes of this warp: 32 quad ..; columns: 128 half ..
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        uint32_t n = 0;
        bool ok = true;
        for (int tile = pair; tile < tiles; tile += pairs) {
            int m0, n0;
            place(tile, m0, n0);
            const int row = m0 + rank * HALF + quad * 32 + lane, c0 = n0 + half * HALF;
            const bool in = row < p.M;
            [[maybe_unused]] int target = -1;
            [[maybe_unused]] float lse = 0.f, g = 0.f, mx = kNone, sum = 0.f;
            if (EPI != OUT && in) {
                target = p.tgt[row];
                if (EPI == GRAD) {
                    lse = p.lse[row];
                    g = p.g[row];
                }
            }
            auto finish = [&](int c, float (&v)[32]) {   // columns c0 + c .. + 31 of this thread's row
                const int col = c0 + c, live = p.N - col;   // columns of this chunk that exist
                if constexpr (EPI == STATS) {
                    if (live < 32) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = i < live ? v[i] : -INFINITY;
                    }
                    const int at = target - col;
                    if (at >= 0 && at < 32) {
                        float t = 0.f;
#pragma unroll
                        for (int i = 0; i < 32; ++i) t = i == at ? v[i] : t;
                        p.row[row] = t;
                    }
                    float top = mx;
#pragma unroll
                    for (int i = 0; i < 32; ++i) top = fmaxf(top, v[i]);
                    // the difference first: exact where the exponential counts, whatever the logits' size
                    float s0 = 0.f, s1 = 0.f;
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        s0 += ex2((v[i] - top) * kLog2e);
                        s1 += ex2((v[i + 1] - top) * kLog2e);
                    }
                    sum = fmaf(sum, ex2((mx - top) * kLog2e), s0 + s1);
                    mx = top;
                } else if constexpr (EPI == GRAD) {
                    // D: 0 behind the vocabulary's end, which the products read as well
                    const int at = p.v0 + col;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float prob = ex2((v[i] - lse) * kLog2e);
                        v[i] = (i < live ? prob - (at + i == target ? 1.f : 0.f) : 0.f) * g;
                    }
                    if (in && col < p.d_pitch) {
                        for (int pl = 0; pl < p.planes; ++pl) {
                            uint4 *dst = reinterpret_cast<uint4 *>(p.d + pl * p.d_plane + (long long)row * p.d_pitch + col);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                uint32_t w[4];
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    w[j] = pack_bf16(v[8 * i + 2 * j], v[8 * i + 2 * j + 1]);
                                    // what the next plane holds
                                    v[8 * i + 2 * j] -= __uint_as_float(w[j] << 16);
                                    v[8 * i + 2 * j + 1] -= __uint_as_float(w[j] & 0xFFFF0000u);
                                }
                                dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        }
                    }
                } else {
                    if (in) {
                        if (p.add) {
                            const float *a = p.add + (long long)row * p.N + col;
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (i < live) v[i] += a[i];
                        }
                        if (p.sum) {
                            float *o = p.sum + (long long)row * p.N + col;
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (i < live) o[i] = v[i];
                        } else {
                            const long long at = (long long)(row / p.T) * p.out_b + (long long)(row % p.T) * p.out_t + col;
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                if (i < live) {
                                    if (p.f32) ((float *)p.out)[at + i] = v[i];
                                    else st_out((__nv_bfloat16 *)p.out + at + i, v[i]);
                                }
                            }
                        }
                    }
                }
            };
            auto get = [&](int c, float (&v)[32]) {
                uint32_t r[32];
                tmem_ld32(tmem + (n & 1) * TILE + half * HALF + lanes + c, r);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
            };
            auto release = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) peer_arrive(peer_addr(&bar[TEMPTY + (n & 1)], 0));
                ++n;
            };
            if constexpr (SEG) {
                float all[HALF / 32][32] = {};
                for (int seg = 0; seg < segs; ++seg) {
                    if (!(ok = wait(TFULL + (n & 1), n >> 1))) break;
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < HALF / 32; ++c) {
                        float v[32];
                        get(32 * c, v);
#pragma unroll
                        for (int i = 0; i < 32; ++i) all[c][i] += v[i];
                    }
                    release();
                }
                if (!ok) break;
#pragma unroll
                for (int c = 0; c < HALF / 32; ++c) finish(32 * c, all[c]);
            } else {
                if (!(ok = wait(TFULL + (n & 1), n >> 1))) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < HALF; c += 32) {
                    float v[32];
                    get(c, v);
                    finish(c, v);
                }
                release();
            }
            if (EPI == STATS && in) p.part[(long long)(2 * (n0 / TILE) + half) * p.M + row] = make_float2(mx, sum);
        }
    }
    __syncwarp();
    __syncthreads();
    pair_sync();   // the other block's barriers are not touched any more
    tc_fence_after();
    if (warp == 1) pair_tmem_dealloc(tmem, 512);
}

// Targets as int32, -1 for none (ignored, or outside the vocabulary, which the status word says); backward: their dloss too.
__global__ void __launch_bounds__(256) k_targets(lay::View<const int64_t> t, lay::View<const float> dloss, int M, int T, int V, int64_t ignore,
                                                 int32_t *tgt, float *g, uint32_t *status)
{
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= M) return;
    const int64_t v = *t.at(i / T, 0, i % T);
    const bool in = v != ignore && v >= 0 && v < V;
    if (v != ignore && !in) raise_status(status, kStatusBadOffsets);
    tgt[i] = in ? (int32_t)v : -1;
    if (g) g[i] = in ? *dloss.at(i / T, 0, i % T) : 0.f;
}

// One block: 32 rows, a warp every 8th of a row's pieces; then the 8 in a fixed order.
__global__ void __launch_bounds__(256) k_lse(const float2 *part, int P, int M, const int32_t *tgt, const float *row, float *loss, float *lse)
{
    __shared__ float2 sm[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, r = blockIdx.x * 32 + lane;
    float mx = kNone, sum = 0.f;
    auto join = [&](float2 q) {
        const float top = fmaxf(mx, q.x);
        sum = sum * exp2f((mx - top) * kLog2e) + q.y * exp2f((q.x - top) * kLog2e);
        mx = top;
    };
    if (r < M) {
#pragma unroll 4
        for (int j = w; j < P; j += 8) join(part[(long long)j * M + r]);
    }
    sm[w][lane] = make_float2(mx, sum);
    __syncthreads();
    if (w == 0 && r < M) {
        for (int j = 1; j < 8; ++j) join(sm[j][lane]);
        const float l = mx + logf(sum);
        lse[r] = l;
        loss[r] = tgt[r] < 0 ? 0.f : l - row[r];
    }
}

// Rows into [planes][rows][pitch] bf16: as they are, or as three planes, the largest first.  pitch is a multiple of 8.
template <class T>
__global__ void __launch_bounds__(256) k_pack(lay::View<const T> v, int R, int T_, int K, __nv_bfloat16 *out, long long pitch, long long plane)
{
    const long long all = (long long)R * pitch, step = (long long)gridDim.x * 256;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < all; i += step) {
        const int r = (int)(i / pitch), k = (int)(i - r * pitch);
        const float f = k < K ? ld_in(v.at(r / T_, 0, r % T_) + k) : 0.f;
        const __nv_bfloat16 a = __float2bfloat16_rn(f);
        out[i] = a;
        if (sizeof(T) == 4) {
            const float g = f - __bfloat162float(a);
            const __nv_bfloat16 b = __float2bfloat16_rn(g);
            out[i + plane] = b;
            out[i + 2 * plane] = __float2bfloat16_rn(g - __bfloat162float(b));
        }
    }
}

// bf16 [planes][rows][cols], boxes of 64 columns x `high` rows
bool make_map(CUtensorMap *m, const Operand &o, long long cols, long long rows, int planes, int high)
{
    return lay::tensor_map(m, false, o.p, cols, rows, planes, o.pitch, o.plane, 64, high, true);
}

template <bool A_MN, bool B_MN, int EPI, bool SEG>
cudaError_t launch_as(const CUtensorMap &a, const CUtensorMap &b, Gemm &p, int contraction, cudaStream_t st)
{
    p.mt = tiles_of(p.M);
    p.nt = tiles_of(p.N);
    p.kb = (contraction + BK - 1) / BK;
    p.seg = SEG ? kSegment : p.kb;
    auto kernel = k_gemm<A_MN, B_MN, EPI, SEG>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    const long long tiles = (long long)p.mt * p.nt, pairs = lay::sm_count() / 2;
    kernel<<<(unsigned)(2 * (tiles < pairs ? tiles : pairs)), THREADS, SMEM, st>>>(a, b, p);
    return cudaPeekAtLastError();
}

template <bool A_MN, bool B_MN, int EPI>
cudaError_t launch(const CUtensorMap &a, const CUtensorMap &b, Gemm &p, int contraction, cudaStream_t st)
{
    return p.np > 1 ? launch_as<A_MN, B_MN, EPI, true>(a, b, p, contraction, st) : launch_as<A_MN, B_MN, EPI, false>(a, b, p, contraction, st);
}

Gemm common(const Call &c)
{
    Gemm p = {};
    p.status = c.status;
    p.planes = c.planes;
    // of three planes a side, the products from the smallest on
    p.np = c.planes == 1 ? 1 : 6;
    p.pa = c.planes == 1 ? 0 : 0x001102;
    p.pb = c.planes == 1 ? 0 : 0x010120;
    p.tgt = c.tgt;
    p.lse = c.lse;
    p.row = c.row;
    p.g = c.row;
    p.part = c.part;
    return p;
}

template <class T>
void pack(const dn_view *v, int rows, int per, int K, const Operand &o, cudaStream_t st)
{
    const long long n = ((long long)rows * o.pitch + 255) / 256, most = 32ll * lay::sm_count();
    k_pack<T><<<(unsigned)(n < most ? n : most), 256, 0, st>>>(lay::view_of<const T>(v), rows, per, K, (__nv_bfloat16 *)o.p, o.pitch, o.plane);
}

cudaError_t begin(const Call &c, bool bwd, cudaStream_t st)
{
    cudaError_t e = cudaMemsetAsync(c.status, 0, sizeof(uint32_t), st);
    if (e != cudaSuccess || c.M == 0) return e;
    const bool f32 = c.s->dtype == DN_F32;
    if (c.pack_x) f32 ? pack<float>(c.x, c.M, c.s->T, c.K, c.xo, st) : pack<__nv_bfloat16>(c.x, c.M, c.s->T, c.K, c.xo, st);
    if (c.pack_w) f32 ? pack<float>(c.w, c.V, c.V, c.K, c.wo, st) : pack<__nv_bfloat16>(c.w, c.V, c.V, c.K, c.wo, st);
    k_targets<<<(c.M + 255) / 256, 256, 0, st>>>(lay::view_of<const int64_t>(c.targets), lay::view_of<const float>(c.dloss), c.M, c.s->T, c.V,
                                                 c.s->ignore_index, c.tgt, bwd ? c.row : nullptr, c.status);
    return cudaPeekAtLastError();
}

}  // namespace

int tiles_of(int n) { return (int)(((long long)n + TILE - 1) / TILE); }

cudaError_t forward(const Call &c, cudaStream_t st)
{
    cudaError_t e = begin(c, false, st);
    if (e != cudaSuccess || c.M == 0) return e;
    CUtensorMap mx, mw;
    if (!make_map(&mx, c.xo, c.K, c.M, c.planes, HALF) || !make_map(&mw, c.wo, c.K, c.V, c.planes, HALF)) return cudaErrorInvalidValue;
    Gemm p = common(c);
    p.M = c.M;
    p.N = c.V;
    if ((e = launch<false, false, STATS>(mx, mw, p, c.K, st)) != cudaSuccess) return e;
    k_lse<<<(c.M + 31) / 32, 256, 0, st>>>(c.part, 2 * tiles_of(c.V), c.M, c.tgt, c.row, c.loss, c.lse);
    return cudaPeekAtLastError();
}

cudaError_t backward(const Call &c, cudaStream_t st)
{
    cudaError_t e = begin(c, true, st);
    if (e != cudaSuccess) return e;
    const bool f32 = c.s->dtype == DN_F32;
    if (c.M == 0) return cudaMemsetAsync(c.dw, 0, (size_t)c.V * c.K * (f32 ? 4 : 2), st);
    const Operand d = {c.d, c.piece, (long long)c.M * c.piece};
    CUtensorMap mx, mw, mxn, mwn;
    if (!make_map(&mx, c.xo, c.K, c.M, c.planes, HALF) || !make_map(&mw, c.wo, c.K, c.V, c.planes, HALF) ||
        !make_map(&mxn, c.xo, c.K, c.M, c.planes, BK) || !make_map(&mwn, c.wo, c.K, c.V, c.planes, BK))
        return cudaErrorInvalidValue;
    for (int v0 = 0; v0 < c.V; v0 += c.piece) {
        const int n = c.V - v0 < c.piece ? c.V - v0 : c.piece;
        const bool first = v0 == 0, last = v0 + n == c.V;
        // the maps end where this piece does: nothing behind it is read
        CUtensorMap md, mdn;
        if (!make_map(&md, d, n, c.M, c.planes, HALF) || !make_map(&mdn, d, n, c.M, c.planes, BK)) return cudaErrorInvalidValue;
        Gemm p = common(c);
        p.M = c.M;
        p.N = n;
        p.b_row = p.v0 = v0;
        p.d = (__nv_bfloat16 *)c.d;
        p.d_pitch = d.pitch;
        p.d_plane = d.plane;
        if ((e = launch<false, false, GRAD>(mx, mw, p, c.K, st)) != cudaSuccess) return e;
        p = common(c);
        p.M = c.M;
        p.N = c.K;
        p.b_k = v0;
        p.add = first ? nullptr : c.acc;
        p.sum = last ? nullptr : c.acc;
        p.out = c.dx->data;
        p.out_b = c.dx->batch;
        p.out_t = c.dx->time;
        p.T = c.s->T;
        p.f32 = f32;
        if ((e = launch<false, true, OUT>(md, mwn, p, n, st)) != cudaSuccess) return e;
        p = common(c);
        p.M = n;
        p.N = c.K;
        p.out = (char *)c.dw + (size_t)v0 * c.K * (f32 ? 4 : 2);
        p.out_t = c.K;
        p.T = n;
        p.f32 = f32;
        if ((e = launch<true, true, OUT>(mdn, mxn, p, c.M, st)) != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace xent
}  // namespace gdn

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
// time, which a contraction of 70001 tokens added up to 8e-5 of dw; segments of 256 are summed in registers, rounded.
constexpr int kSegment = 4;

enum { STATS, GRAD, OUT };

// One product C = A B^T and how its tiles are cut: units of a tile and a part of the contraction.
struct Product {
    int M, N;                       // rows and columns of C that exist
    int mt, nt, kb;                 // tiles; 64-wide steps of the contraction
    int cuts, len;                  // parts of the contraction and their steps
    int b_row, b_k;                 // where B's rows and its contraction begin
    // OUT: the sum, where cuts > 1 of one part, [cuts][M][N] in `part`
    const float *add;               // [M][N] or null
    float *sum;                     // [M][N], or null: out
    float *part;
    void *out;
    long long out_b, out_t;         // row (b, t) of out at b out_b + t out_t
    int T, f32, wide;               // wide: out's rows start at 16 bytes, and N is a multiple of 8
};

struct Gemm {
    Product of[2];                  // the second of OUT only
    int seg;                        // steps of a segment: all, or kSegment (SEG)
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
};

// Units of the two products for pair `p` of `n`: the first product's dealt in turn, the second's so that pairs with fewer of the
// first have the more of the second that its length makes up for.
struct Deal {
    int count[2], first[2], step[2];
    __host__ __device__ Deal(const Gemm &g, int p, int n)
    {
        const int n0 = g.of[0].mt * g.of[0].nt * g.of[0].cuts, n1 = g.of[1].mt * g.of[1].nt * g.of[1].cuts;
        const int r = n0 % n;   // pairs with one more of the first
        count[0] = n0 / n + (p < r ? 1 : 0);
        first[0] = p;
        step[0] = n;
        const int more = n1 > 0 ? (g.of[0].len + g.of[1].len / 2) / g.of[1].len : 0;
        int base = n1 - (n - r) * more, low = 0, high;   // units a pair with more, with fewer of the first
        if (r == 0) {
            low = high = n1 / n;
            base = n1 - n * low;
        } else if (base >= 0) {
            low = base / n;
            high = low + more;
            base -= n * low;
        } else {
            high = n1 / (n - r);
            base = n1 - (n - r) * high;   // over the pairs with fewer
        }
        // the rest, one each: from the last pair on
        const int rest = p >= n - base ? 1 : 0;
        count[1] = (p < r ? low : high) + rest;
        first[1] = (p < r ? p * low : r * low + (p - r) * high) + (rest ? p - (n - base) : 0);
        step[1] = 1;
    }
};

enum { FULL = 0, EMPTY = STAGES, TFULL = 2 * STAGES, TEMPTY = TFULL + 2, DONE = TEMPTY + 2, NBAR = DONE + 1 };

struct Maps {
    CUtensorMap a[2], b[2];
};

// OUT: two products, D w and D^T x: B is MN-major in both, A in the second.  Otherwise one, both operands K-major.
template <int EPI, bool SEG>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1) k_gemm(const __grid_constant__ Maps maps, const __grid_constant__ Gemm p)
{
    extern __shared__ char raw[];
    char *sm = (char *)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    uint64_t *bar = (uint64_t *)(sm + STAGES * STAGE);
    uint32_t *s_tmem = (uint32_t *)(bar + NBAR);
    volatile int *s_abort = (volatile int *)(s_tmem + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = pair_rank();
    const Deal deal(p, blockIdx.x >> 1, gridDim.x >> 1);

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
        prefetch_tmap(&maps.a[0]);
        prefetch_tmap(&maps.b[0]);
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
    // Unit u of product q: its tile and its steps of the contraction
    struct Unit {
        int m, n, k0, k1, cut;
    };
    auto unit = [&](const Product &o, int u) {
        Unit r;
        const int tiles = o.mt * o.nt;
        r.cut = u / tiles;
        const int tile = u - r.cut * tiles, per = GROUP * o.nt, grp = tile / per, in = tile - grp * per, gm = min(GROUP, o.mt - grp * GROUP);
        r.m = (grp * GROUP + in % gm) * TILE;
        r.n = in / gm * TILE;
        r.k0 = r.cut * o.len;
        r.k1 = min(o.kb, r.k0 + o.len);
        return r;
    };
    auto segments = [&](const Unit &u) { return SEG ? (u.k1 - u.k0 + p.seg - 1) / p.seg : 1; };
    constexpr int PRODUCTS = EPI == OUT ? 2 : 1;

    if (warp == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int o = 0; o < PRODUCTS; ++o) {
                const Product &pr = p.of[o];
                const CUtensorMap *ta = &maps.a[o], *tb = &maps.b[o];
                const bool a_mn = EPI == OUT && o == 1;
                constexpr bool B_MN = EPI == OUT;
                for (int i = 0; ok && i < deal.count[o]; ++i) {
                    const Unit u = unit(pr, deal.first[o] + i * deal.step[o]);
                    const int m = u.m + rank * HALF, n = u.n + rank * HALF, segs = segments(u);
                    for (int sq = 0; ok && sq < segs * p.np; ++sq) {
                        const int seg = sq / p.np, q = sq - seg * p.np;
                        const int a = p.pa >> 4 * q & 15, b = p.pb >> 4 * q & 15;
                        const int begin = SEG ? u.k0 + seg * p.seg : u.k0, end = SEG ? min(u.k1, begin + p.seg) : u.k1;
                        for (int k = begin; k < end; ++k, ++it) {
                            const int s = it % STAGES;
                            if (!(ok = wait(EMPTY + s, it / STAGES + 1))) break;
                            const uint32_t full = peer_addr(&bar[FULL + s], 0);
                            char *sa = sm + s * STAGE, *sb = sa + OPERAND;
                            if (rank == 0) mbar_expect_tx(&bar[FULL + s], 2 * STAGE);
                            if (a_mn) {
                                pair_load_3d(sa, ta, full, m, k * BK, a);
                                pair_load_3d(sa + OPERAND / 2, ta, full, m + 64, k * BK, a);
                            } else {
                                pair_load_3d(sa, ta, full, k * BK, m, a);
                            }
                            if (B_MN) {
                                pair_load_3d(sb, tb, full, n, pr.b_k + k * BK, b);
                                pair_load_3d(sb + OPERAND / 2, tb, full, n + 64, pr.b_k + k * BK, b);
                            } else {
                                pair_load_3d(sb, tb, full, k * BK, pr.b_row + n, b);
                            }
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
            constexpr bool B_MN = EPI == OUT;
            constexpr uint32_t bstep = B_MN ? 2048 : 32;
            uint32_t it = 0, n = 0;
            bool ok = true;
            for (int o = 0; o < PRODUCTS; ++o) {
                const bool a_mn = EPI == OUT && o == 1;
                const uint32_t id = a_mn ? idesc(1, TILE, TILE, true, B_MN) : idesc(1, TILE, TILE, false, B_MN);
                const uint32_t astep = a_mn ? 2048 : 32, alead = a_mn ? OPERAND / 2 : 16;
                for (int i = 0; ok && i < deal.count[o]; ++i) {
                    const Unit u = unit(p.of[o], deal.first[o] + i * deal.step[o]);
                    const int segs = segments(u);
                    for (int seg = 0; ok && seg < segs; ++seg, ++n) {
                        const uint32_t acc = tmem + (n & 1) * TILE;
                        if (!(ok = wait(TEMPTY + (n & 1), (n >> 1) + 1))) break;
                        tc_fence_after();
                        const int steps = p.np * (SEG ? min(p.seg, u.k1 - u.k0 - seg * p.seg) : u.k1 - u.k0);
                        for (int k = 0; k < steps; ++k, ++it) {
                            const int s = it % STAGES;
                            if (!(ok = wait(FULL + s, it / STAGES))) break;
                            tc_fence_after();
                            const uint32_t sa = smem_u32(sm + s * STAGE), sb = sa + OPERAND;
#pragma unroll
                            for (int j = 0; j < BK / 16; ++j)
                                pair_mma_bf16(acc, sdesc(sa + j * astep, alead, 1024), sdesc(sb + j * bstep, B_MN ? OPERAND / 2 : 16, 1024), id,
                                              k > 0 || j > 0);
                            pair_commit(&bar[EMPTY + s]);
                        }
                        if (ok) pair_commit(&bar[TFULL + (n & 1)]);
                    }
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
        for (int i = 0; i < deal.count[0] + (EPI == OUT ? deal.count[1] : 0); ++i) {
            const int o = EPI == OUT && i >= deal.count[0], j = o ? i - deal.count[0] : i;
            const Product &pr = p.of[o];
            const Unit u = unit(pr, deal.first[o] + j * deal.step[o]);
            const int row = u.m + rank * HALF + quad * 32 + lane, c0 = u.n + half * HALF;
            const bool in = row < pr.M;
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
                const int col = c0 + c, live = pr.N - col;   // columns of this chunk that exist
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
                } else if (in && live > 0) {
                    const bool whole = live >= 32 && pr.N % 4 == 0;   // columns and 16-byte rows of a float array
                    const long long at = (long long)row * pr.N + col;
                    if (pr.add && pr.cuts == 1) {
                        if (whole) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float4 f = reinterpret_cast<const float4 *>(pr.add + at)[i];
                                v[4 * i] += f.x;
                                v[4 * i + 1] += f.y;
                                v[4 * i + 2] += f.z;
                                v[4 * i + 3] += f.w;
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (i < live) v[i] += pr.add[at + i];
                        }
                    }
                    const bool partial = pr.cuts > 1, sums = partial || pr.sum != nullptr;
                    const long long place = sums ? at : (long long)(row / pr.T) * pr.out_b + (long long)(row % pr.T) * pr.out_t + col;
                    if (sums || pr.f32) {
                        float *to = (partial ? pr.part + (long long)u.cut * pr.M * pr.N : sums ? pr.sum : (float *)pr.out) + place;
                        if (whole && (sums || pr.wide)) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) reinterpret_cast<float4 *>(to)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (i < live) to[i] = v[i];
                        }
                    } else {
                        __nv_bfloat16 *to = (__nv_bfloat16 *)pr.out + place;
                        if (whole && pr.wide) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                reinterpret_cast<uint4 *>(to)[i] = make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                                                                              pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (i < live) st_out(to + i, v[i]);
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
                for (int seg = segments(u); seg > 0; --seg) {
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
            if (EPI == STATS && in) p.part[(long long)(2 * (u.n / TILE) + half) * pr.M + row] = make_float2(mx, sum);
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

// Sums of a product's parts in a fixed order, and what OUT does with a whole one.  A thread has 4 columns of a row where `wide`.
template <int V>
__global__ void __launch_bounds__(256) k_join(const __grid_constant__ Product o)
{
    const long long all = (long long)o.M * o.N, step = (long long)gridDim.x * 256 * V;
    for (long long i = (blockIdx.x * 256ll + threadIdx.x) * V; i < all; i += step) {
        float v[V] = {};
        for (int c = 0; c < o.cuts; ++c) {
            lay::Vec<float, V> q;
            float f[V];
            q.load(o.part + c * all + i);
            q.get(f);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] += f[e];
        }
        const int row = (int)(i / o.N), col = (int)(i - (long long)row * o.N);
        const long long place = o.sum ? i : (long long)(row / o.T) * o.out_b + (long long)(row % o.T) * o.out_t + col;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if (o.add) v[e] += o.add[i + e];
            if (o.sum) o.sum[place + e] = v[e];
            else if (o.f32) ((float *)o.out)[place + e] = v[e];
            else st_out((__nv_bfloat16 *)o.out + place + e, v[e]);
        }
    }
}

// bf16 [planes][rows][cols], boxes of 64 columns x `high` rows
bool make_map(CUtensorMap *m, const Operand &o, long long cols, long long rows, int planes, int high)
{
    return lay::tensor_map(m, false, o.p, cols, rows, planes, o.pitch, o.plane, 64, high, true);
}

void size(Product &o, int M, int N, int contraction)
{
    o.M = M;
    o.N = N;
    o.mt = tiles_of(M);
    o.nt = tiles_of(N);
    o.kb = o.len = (contraction + BK - 1) / BK;
    o.cuts = 1;
    o.T = 1;
}

int pairs_at_most() { return lay::sm_count() / 2; }

template <int EPI, bool SEG>
cudaError_t launch_as(const Maps &m, Gemm &p, cudaStream_t st)
{
    p.seg = kSegment;
    auto kernel = k_gemm<EPI, SEG>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    long long units = 0, pairs = pairs_at_most();
    for (const Product &o : p.of) units += (long long)o.mt * o.nt * o.cuts;
    kernel<<<(unsigned)(2 * (units < pairs ? units : pairs)), THREADS, SMEM, st>>>(m, p);
    return cudaPeekAtLastError();
}

template <int EPI>
cudaError_t launch(const Maps &m, Gemm &p, cudaStream_t st)
{
    return p.np > 1 ? launch_as<EPI, true>(m, p, st) : launch_as<EPI, false>(m, p, st);
}

cudaError_t join(const Product &o, cudaStream_t st)
{
    if (o.cuts == 1) return cudaSuccess;
    const bool four = o.N % 4 == 0;
    const long long n = ((long long)o.M * o.N / (four ? 4 : 1) + 255) / 256, most = 16ll * lay::sm_count();
    const unsigned blocks = (unsigned)(n < most ? n : most);
    if (four) k_join<4><<<blocks, 256, 0, st>>>(o);
    else k_join<1><<<blocks, 256, 0, st>>>(o);
    return cudaPeekAtLastError();
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

// How the contractions of a piece's two products are cut: not longer than a pair's share of all steps, so that a few long tiles
// do not keep the rest waiting, and 4 steps at least.
void cuts_of(int M, int K, int n, int planes, int &dx, int &dw)
{
    const long long nk = tiles_of(K), a = ((long long)n + BK - 1) / BK, b = ((long long)M + BK - 1) / BK;
    const long long all = nk * (tiles_of(M) * a + tiles_of(n) * b), least = planes == 1 ? 8 : 4;
    long long share = (all + pairs_at_most() - 1) / pairs_at_most();
    if (share < least) share = least;
    dx = (int)((a + share - 1) / share);
    dw = (int)((b + share - 1) / share);
}

cudaError_t forward(const Call &c, cudaStream_t st)
{
    cudaError_t e = begin(c, false, st);
    if (e != cudaSuccess || c.M == 0) return e;
    Maps m = {};
    if (!make_map(&m.a[0], c.xo, c.K, c.M, c.planes, HALF) || !make_map(&m.b[0], c.wo, c.K, c.V, c.planes, HALF)) return cudaErrorInvalidValue;
    Gemm p = common(c);
    size(p.of[0], c.M, c.V, c.K);
    if ((e = launch<STATS>(m, p, st)) != cudaSuccess) return e;
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
    Maps logits = {}, outs = {};
    if (!make_map(&logits.a[0], c.xo, c.K, c.M, c.planes, HALF) || !make_map(&logits.b[0], c.wo, c.K, c.V, c.planes, HALF) ||
        !make_map(&outs.b[1], c.xo, c.K, c.M, c.planes, BK) || !make_map(&outs.b[0], c.wo, c.K, c.V, c.planes, BK))
        return cudaErrorInvalidValue;
    const size_t el = f32 ? 4 : 2;
    for (int v0 = 0; v0 < c.V; v0 += c.piece) {
        const int n = c.V - v0 < c.piece ? c.V - v0 : c.piece;
        const bool first = v0 == 0, last = v0 + n == c.V;
        // the maps end where this piece does: nothing behind it is read
        if (!make_map(&outs.a[0], d, n, c.M, c.planes, HALF) || !make_map(&outs.a[1], d, n, c.M, c.planes, BK)) return cudaErrorInvalidValue;
        Gemm p = common(c);
        size(p.of[0], c.M, n, c.K);
        p.of[0].b_row = p.v0 = v0;
        p.d = (__nv_bfloat16 *)c.d;
        p.d_pitch = d.pitch;
        p.d_plane = d.plane;
        if ((e = launch<GRAD>(logits, p, st)) != cudaSuccess) return e;
        p = common(c);
        int dx_cuts, dw_cuts;
        cuts_of(c.M, c.K, n, c.planes, dx_cuts, dw_cuts);
        Product &dx = p.of[0], &dw = p.of[1];
        size(dx, c.M, c.K, n);
        size(dw, n, c.K, c.M);
        auto cut = [](Product &o, int cuts) {
            o.len = (o.kb + cuts - 1) / cuts;
            o.cuts = (o.kb + o.len - 1) / o.len;
        };
        cut(dx, dx_cuts);
        cut(dw, dw_cuts);
        dx.b_k = v0;
        dx.add = first ? nullptr : c.acc;
        dx.sum = last ? nullptr : c.acc;
        dx.part = c.cut;
        dx.out = c.dx->data;
        dx.out_b = c.dx->batch;
        dx.out_t = c.dx->time;
        dx.T = c.s->T;
        dw.part = c.cut + (dx.cuts > 1 ? (size_t)dx.cuts * c.M * c.K : 0);
        dw.out = (char *)c.dw + (size_t)v0 * c.K * el;
        dw.out_t = c.K;
        dw.T = n;
        for (Product *o : {&dx, &dw}) {
            o->f32 = f32;
            o->wide = c.K % 8 == 0 && (uintptr_t)o->out % 16 == 0 && o->out_b * el % 16 == 0 && o->out_t * el % 16 == 0;
        }
        if ((e = launch<OUT>(outs, p, st)) != cudaSuccess || (e = join(dx, st)) != cudaSuccess || (e = join(dw, st)) != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace xent
}  // namespace gdn

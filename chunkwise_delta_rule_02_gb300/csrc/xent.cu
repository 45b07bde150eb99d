// Linear softmax cross entropy without the logits: l = x w^T, lse = log sum_v exp l_v,
// loss = lse - l[target]; backward, by pieces of the vocabulary, D = (exp(l - lse) - onehot) dloss,
// dx = sum over pieces D w, dw = D^T x.
//
// k_gemm is the one matrix product: C = A B^T in tiles of 256 x 256 by a pair of CTAs (tcgen05.mma, cta_group::2), each holding 128
// of the tile's rows in TMEM and loading half of both operands by TMA into a ring of stages.  A and B are K-major or
// MN-major in memory, so that all four products run on x, w and D as they lie.  Warp 0 loads, warp 1 of the even CTA issues the
// MMAs, eight warps take the finished tile from TMEM while the next one is computed in the other half of it.  What they do with it:
//   STATS  maximum and sum of exponentials of a row over 128 columns, and the target's logit;
//   SCORE  the same of few tokens, which are the columns then: the weight's rows are read once, in equal shares;
//   GRAD   D, rounded to the operand's type for the two products that read it;
//   OUT    the tile itself, added to what earlier pieces gave.
// D in bf16 (2^-9 of each value) is what a bf16 input's gradient is computed from: the sums over the vocabulary and over the tokens
// are float32.  float32 inputs are split into three bf16 planes, 8 bits each, and six of their nine products kept: what is
// left out is 2^-24 of the whole.
//
// Bound by the tensor cores, and in a loop by the power limit.  8192 tokens, 2048 features, 32768 entries, bf16: logits with
// STATS 583 us alone (1.89 PFLOP/s, 83 % of the tensor cores' cycles; in a loop 655), both products of half the vocabulary 622 us
// (88 % of the cycles); the training step 2740 us, 1.6 PFLOP/s of the 8 M V K operations that it does.
#include "pair.cuh"
#include "xent.cuh"

namespace gdn {
namespace xent {

namespace {

using namespace sm100;
constexpr int TILE = 256, HALF = 128, BK = 64, STAGES = 6, THREADS = 320, EPI_WARPS = 8;
constexpr int OPERAND = HALF * BK * 2;                               // bytes of 128 rows of an operand
constexpr int BOX = 4096;                                            // bytes that an epilogue warp has for results on their way out
constexpr int SMEM = 2 * STAGES * OPERAND + EPI_WARPS * BOX + 1024 + 256;
constexpr long long BUDGET = 4000000000LL;                           // clock cycles (about 2 s) for any one wait
constexpr int GROUP = 16;                                            // row tiles that share the column tiles of a wave
constexpr int kScore = 128;                                          // tokens up to which they are the columns

// Steps after which float32 inputs' sums leave TMEM: the tensor core cuts what it adds off rather than rounding it, the same way each
// time, which a contraction of 70001 tokens added up to 8e-5 of dw; segments of 256 are summed in registers, rounded.
constexpr int kSegment = 4;
// The same for bf16 logits of more than kLong steps, which came out 3e-6 low with 3289 features: segments of 1024.  In both passes: what both lose
// cancels in a probability, and only that (300 tokens of 9001 features around 1: with segments in the forward alone dw was 7.8e-2 off).
constexpr int kLong = 32, kLongSegment = 16;
// bf16 contractions over the vocabulary or the tokens have no segments (the products of a training step would pay for them); they are cut
// into parts of 16384, whose sums are joined in float32 and rounded.  A part's sum comes out up to 6e-5 of its terms low (dx of 1024 tokens of
// 131072 x 1024, terms of one sign: 2.0e-4 in parts of 65536).
constexpr int kPart = 256;

enum { STATS, GRAD, OUT, SCORE };

// What a unit costs, in stages of the ring: those of its contraction, and its way out of TMEM, which is longer for float32 (2 tokens,
// 15733 entries of 474: 188 us for the product when only the contraction counted, and pairs without a unit of dx got a hundred
// short units of dw).  bf16, 8 tokens of 50000 x 1024, backward with 4, 8, 12, 24 for it: 103, 93, 96, 127 us; 29 of 69380 x 1592 246, 223, 225, 281;
// 1001 float32 of 5003 x 203 with 8, 12, 24: 131, 115, 115.
__host__ __device__ constexpr int way_out(int np) { return np > 1 ? 24 : 8; }
__host__ __device__ inline int cost_of(const Gemm &g, const Product &o) { return o.len * g.np + way_out(g.np); }

// Units of the two products for pair `p` of `n`: the first product's dealt in turn, the second's so that pairs with fewer of the
// first have the more of the second that its cost makes up for.
struct Deal {
    int count[2], first[2], step[2];
    __host__ __device__ Deal(const Gemm &g, int p, int n)
    {
        const int n0 = g.of[0].mt * g.of[0].nt * g.of[0].cuts, n1 = g.of[1].mt * g.of[1].nt * g.of[1].cuts;
        const int r = n0 % n;   // pairs with one more of the first
        count[0] = n0 / n + (p < r ? 1 : 0);
        first[0] = p;
        step[0] = n;
        const int cost = n1 > 0 ? cost_of(g, g.of[1]) : 1, more = n1 > 0 ? (cost_of(g, g.of[0]) + cost / 2) / cost : 0;
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

__device__ __forceinline__ void store_box(const CUtensorMap *map, const void *src, int c0, int c1, int c2)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"((uint64_t)map), "r"(smem_u32(src)),
                 "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}

__device__ __forceinline__ void add_box(const CUtensorMap *map, const void *src, int c0, int c1, int c2)
{
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"((uint64_t)map),
                 "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}

struct Maps {
    CUtensorMap a[2], b[2];
    CUtensorMap out[2], sum;        // boxes of 32 x 32: GRAD's D or OUT's results; OUT's sums of the first product
};

// OUT: two products, D w and D^T x: B is MN-major in both, A in the second.  Otherwise one, both operands K-major.
// NT: columns of a tile (SCORE: 32, 64 or 128 tokens).
template <int EPI, bool SEG, int NT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1) k_gemm(const __grid_constant__ Maps maps, const __grid_constant__ Gemm p)
{
    constexpr int STAGE = OPERAND + NT / 2 * BK * 2;   // bytes a CTA loads of both operands
    extern __shared__ char raw[];
    char *sm = (char *)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    char *boxes = sm + STAGES * STAGE;
    uint64_t *bar = (uint64_t *)(boxes + EPI_WARPS * BOX);
    uint32_t *s_tmem = (uint32_t *)(bar + NBAR);
    volatile int *s_abort = (volatile int *)(s_tmem + 1);
    let_next_start();
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
    wait_for_last();
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
        if (EPI == SCORE) return Unit{u * 2 * p.share, 0, 0, o.kb, 0};
        // divisions only where they are needed: in the one thread that loads or issues, a tile's four took as long as a stage
        const unsigned tiles = o.mt * o.nt, per = GROUP * o.nt;
        r.cut = o.cuts == 1 ? 0 : u / tiles;
        const unsigned tile = u - r.cut * tiles, grp = tile < per ? 0 : tile / per, in = tile - grp * per, gm = min(GROUP, o.mt - (int)grp * GROUP);
        const unsigned col = gm == GROUP ? in / GROUP : in / gm;
        r.m = (grp * GROUP + in - col * gm) * TILE;
        r.n = col * TILE;
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
                    const int m = u.m + rank * (EPI == SCORE ? p.share : HALF), n = u.n + rank * (NT / 2), segs = segments(u);
                    for (int sq = 0; ok && sq < segs * p.np; ++sq) {
                        const int seg = SEG ? sq / p.np : 0, q = sq - seg * p.np;
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
                const uint32_t id = a_mn ? idesc(1, TILE, NT, true, B_MN) : idesc(1, TILE, NT, false, B_MN);
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
    } else if constexpr (EPI == SCORE) {
        // Rows are entries of the vocabulary, columns tokens, 32 a chunk and in turn a lane each; a warp joins its units' statistics.
        const int quad = warp & 3, half = (warp - 2) >> 2;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        constexpr int CHUNKS = NT / 32, MINE = (CHUNKS + 1) / 2;   // of this warp: half, half + 2
        float mx[MINE], sum[MINE];
        int target[MINE];
#pragma unroll
        for (int i = 0; i < MINE; ++i) {
            const int token = 32 * (half + 2 * i) + lane;
            mx[i] = kNone;
            sum[i] = 0.f;
            target[i] = half + 2 * i < CHUNKS && token < p.of[0].N ? target_of(p, token, blockIdx.x == 0 && quad == 2) : -1;
        }
        uint32_t n = 0;
        bool ok = true;
        for (int i = 0; i < deal.count[0]; ++i) {
            const Unit u = unit(p.of[0], deal.first[0] + i * deal.step[0]);
            const int in_cta = quad * 32 + lane, row = u.m + rank * p.share + in_cta;
            const bool in = in_cta < p.share && row < p.of[0].M;
            float all[MINE][32];
#pragma unroll
            for (int c = 0; c < MINE; ++c)
#pragma unroll
                for (int k = 0; k < 32; ++k) all[c][k] = 0.f;
            for (int seg = segments(u); seg > 0; --seg) {
                if (!(ok = wait(TFULL + (n & 1), n >> 1))) break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < MINE; ++c) {
                    if (half + 2 * c < CHUNKS) {
                        uint32_t r[32];
                        tmem_ld32(tmem + (n & 1) * TILE + lanes + 32 * (half + 2 * c), r);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 32; ++k) all[c][k] += __uint_as_float(r[k]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) peer_arrive(peer_addr(&bar[TEMPTY + (n & 1)], 0));
                ++n;
            }
            if (!ok) break;
#pragma unroll
            for (int c = 0; c < MINE; ++c) {
                if (half + 2 * c >= CHUNKS) continue;
                float(&v)[32] = all[c];
                // targets among this warp's 32 entries
                const int at = target[c] - (row - lane);
                const bool mine = at >= 0 && at < 32 && quad * 32 + at < p.share;
                for (uint32_t left = __ballot_sync(0xffffffffu, mine); left; left &= left - 1) {
                    const int k = __ffs(left) - 1, who = __shfl_sync(0xffffffffu, at, k);
                    float t = 0.f;
#pragma unroll
                    for (int j = 0; j < 32; ++j) t = j == k ? v[j] : t;
                    if (lane == who) p.row[32 * (half + 2 * c) + k] = t;
                }
                // each column's maximum, in the lane of its token, by halving; then its sum
                float w[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) w[k] = v[k] = in ? v[k] : -INFINITY;
#pragma unroll
                for (int m = 16; m > 0; m >>= 1) {
                    const bool up = lane & m;
#pragma unroll
                    for (int k = 0; k < m; ++k) {
                        const float send = up ? w[k] : w[k + m], keep = up ? w[k + m] : w[k];
                        w[k] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, m));
                    }
                }
                const float top = fmaxf(mx[c], w[0]);
#pragma unroll
                for (int k = 0; k < 32; ++k) w[k] = ex2((v[k] - __shfl_sync(0xffffffffu, top, k)) * kLog2e);
#pragma unroll
                for (int m = 16; m > 0; m >>= 1) {
                    const bool up = lane & m;
#pragma unroll
                    for (int k = 0; k < m; ++k) {
                        const float send = up ? w[k] : w[k + m], keep = up ? w[k + m] : w[k];
                        w[k] = keep + __shfl_xor_sync(0xffffffffu, send, m);
                    }
                }
                sum[c] = fmaf(sum[c], ex2((mx[c] - top) * kLog2e), w[0]);
                mx[c] = top;
            }
        }
#pragma unroll
        for (int c = 0; c < MINE; ++c) {
            const int token = 32 * (half + 2 * c) + lane;
            if (half + 2 * c < CHUNKS && token < p.of[0].N) p.part[(long long)(blockIdx.x * 4 + quad) * p.of[0].N + token] = make_float2(mx[c], sum[c]);
        }
    } else {
        const int e = warp - 2, quad = warp & 3, half = e >> 2;   // TMEM lanes of this warp: 32 quad ..; columns: 128 half ..
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        uint32_t n = 0, flip = 0;
        bool ok = true, whole_box = false;
        [[maybe_unused]] const float scale = EPI == STATS ? 1.f : scale_of(p);
        // 32 columns of the warp's 32 rows to memory, through shared memory and a tensor map, which leaves out what lies behind the ends
        auto box_bf16 = [&](const CUtensorMap *map, const uint32_t (&w)[16], int col, int row0, int plane) {
            char *b = boxes + e * BOX + (flip ^= BOX / 2);
            if (lane == 0) {   // the box before the last is read; the last one too, where it was a float one of twice the size
                if (whole_box) bulk_wait_read();
                else asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
            }
            whole_box = false;
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint4 *>(b + lane * 64 + ((j ^ (lane >> 1 & 3)) << 4)) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                store_box(map, b, col, row0, plane);
                bulk_commit();
            }
        };
        auto box_f32 = [&](const CUtensorMap *map, const float (&v)[32], int col, int row0, bool add) {
            char *b = boxes + e * BOX;
            if (lane == 0) bulk_wait_read();
            whole_box = true;
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j)
                *reinterpret_cast<float4 *>(b + lane * 128 + ((j ^ (lane & 7)) << 4)) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (add) add_box(map, b, col, row0, 0);
                else store_box(map, b, col, row0, 0);
                bulk_commit();
            }
        };
        // What belongs to this thread's row of a unit is asked for a unit ahead: of few features a tile's 4 chunks take as long as
        // two or three trips to memory.
        struct Row {
            long long target;
            float lse, g;
        };
        auto ask = [&](int i) {
            Row r = {p.ignore, 0.f, 0.f};
            if ((EPI == STATS || EPI == GRAD) && i < deal.count[0]) {
                const int row = unit(p.of[0], deal.first[0] + i * deal.step[0]).m + rank * HALF + quad * 32 + lane;
                if (row < p.of[0].M) {
                    r.target = target_at(p, row);
                    if (EPI == GRAD) {
                        r.lse = p.lse[row];
                        r.g = p.dloss[(long long)(row / p.T) * p.g_b + (long long)(row % p.T) * p.g_t];
                    }
                }
            }
            return r;
        };
        Row next = ask(0);
        for (int i = 0; i < deal.count[0] + (EPI == OUT ? deal.count[1] : 0); ++i) {
            const int o = EPI == OUT && i >= deal.count[0], j = o ? i - deal.count[0] : i;
            const Product &pr = p.of[o];
            const Unit u = unit(pr, deal.first[o] + j * deal.step[o]);
            const int row = u.m + rank * HALF + quad * 32 + lane, c0 = u.n + half * HALF;
            const bool in = row < pr.M;
            [[maybe_unused]] int target = -1;
            [[maybe_unused]] float lse = 0.f, g = 0.f, mx = kNone, sum = 0.f;
            if constexpr (EPI == STATS || EPI == GRAD) {
                const Row r = next;
                next = ask(i + 1);
                target = target_from(p, r.target, p.v0 == 0 && u.n == 0 && half == 0);
                lse = r.lse;
                if (EPI == GRAD && target >= 0) g = r.g / scale;
            }
            auto finish = [&](int c, auto &v) {   // columns c0 + c .. of this thread's row, 32 or 64
                constexpr int W = sizeof(v) / sizeof(v[0]);
                const int col = c0 + c, live = pr.N - col;   // columns of this chunk that exist
                if constexpr (EPI == OUT) {
#pragma unroll
                    for (int i = 0; i < W; ++i) v[i] *= scale;
                }
                if constexpr (EPI == STATS) {
                    if (live < W) {
#pragma unroll
                        for (int i = 0; i < W; ++i) v[i] = i < live ? v[i] : -INFINITY;
                    }
                    const int at = target - col;
                    if (at >= 0 && at < W) {
                        float t = 0.f;
#pragma unroll
                        for (int i = 0; i < W; ++i) t = i == at ? v[i] : t;
                        p.row[row] = t;
                    }
                    float4 m = make_float4(mx, mx, mx, mx);
#pragma unroll
                    for (int i = 0; i < W; i += 4) {
                        m.x = fmaxf(m.x, v[i]);
                        m.y = fmaxf(m.y, v[i + 1]);
                        m.z = fmaxf(m.z, v[i + 2]);
                        m.w = fmaxf(m.w, v[i + 3]);
                    }
                    const float top = fmaxf(fmaxf(m.x, m.y), fmaxf(m.z, m.w));
                    // the difference first: exact where the exponential counts, whatever the logits' size
                    float2 s[2] = {};
#pragma unroll
                    for (int i = 0; i < W; i += 2)
                        s[i >> 1 & 1] = lay::add2(s[i >> 1 & 1], lay::ex2_2(lay::mul2(lay::add2(make_float2(v[i], v[i + 1]), lay::two(-top)), lay::two(kLog2e))));
                    s[0] = lay::add2(s[0], s[1]);
                    sum = fmaf(sum, ex2((mx - top) * kLog2e), s[0].x + s[0].y);
                    mx = top;
                } else if constexpr (EPI == GRAD) {
                    // two at a time: at 8 instructions an element a tile's way out took nearly as long as its products
                    const float2 neg = lay::two(-lse), gg = lay::two(g);
                    const int hit = target - p.v0 - col;   // this row's target among the columns
#pragma unroll
                    for (int i = 0; i < W; i += 2) {
                        const float2 q = lay::ex2_2(lay::mul2(lay::add2(make_float2(v[i], v[i + 1]), neg), lay::two(kLog2e)));
                        v[i] = q.x;
                        v[i + 1] = q.y;
                    }
                    if (__any_sync(0xffffffffu, hit >= 0 && hit < W)) {
#pragma unroll
                        for (int i = 0; i < W; ++i) v[i] -= i == hit ? 1.f : 0.f;
                    }
#pragma unroll
                    for (int i = 0; i < W; i += 2) {
                        const float2 q = lay::mul2(make_float2(v[i], v[i + 1]), gg);
                        v[i] = q.x;
                        v[i + 1] = q.y;
                    }
                    // Columns behind the vocabulary's end: a box is cut off at 16 bytes, so that up to seven get into D's padding, and exp(-lse)
                    // has no bound.  Rows without a target are 0 whatever they hold.
                    if (live < W) {
#pragma unroll
                        for (int i = 0; i < W; ++i) v[i] = i < live ? v[i] : 0.f;
                    }
                    const int row0 = row - lane;
                    if (row0 < pr.M) {
#pragma unroll
                        for (int h = 0; h < W; h += 32) {
                            if (live <= h) break;
                            for (int pl = 0; pl < p.planes; ++pl) {
                                uint32_t w[16];
#pragma unroll
                                for (int j = 0; j < 16; ++j) w[j] = target < 0 ? 0u : pack_bf16(v[h + 2 * j], v[h + 2 * j + 1]);
                                box_bf16(&maps.out[0], w, col + h, row0, pl);
                                if (pl + 1 < p.planes) {
#pragma unroll
                                    for (int j = 0; j < 16; ++j) {   // what the next plane holds
                                        v[h + 2 * j] -= __uint_as_float(w[j] << 16);
                                        v[h + 2 * j + 1] -= __uint_as_float(w[j] & 0xFFFF0000u);
                                    }
                                }
                            }
                        }
                    }
                } else if constexpr (W > 32) {
                    static_assert(EPI != OUT || W == 32, "OUT's boxes");
                } else if (live > 0 && row - lane < pr.M && pr.cuts == 1 && pr.sum && pr.sum_box) {
                    box_f32(&maps.sum, v, col, row - lane, pr.sum_box == 2);
                } else if (live > 0 && row - lane < pr.M) {
                    const bool partial = pr.cuts > 1, sums = partial || pr.sum != nullptr;
                    const long long at = (long long)row * pr.N + col;
                    const float *add = partial ? nullptr : pr.add;
                    const bool whole = live >= 32 && pr.N % 4 == 0;   // columns and 16-byte rows of a float array
                    const bool boxed = !sums && pr.out_box;
                    if (add && in && whole) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 f = reinterpret_cast<const float4 *>(add + at)[i];
                            v[4 * i] += f.x;
                            v[4 * i + 1] += f.y;
                            v[4 * i + 2] += f.z;
                            v[4 * i + 3] += f.w;
                        }
                    } else if (add && in && boxed) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i < live) v[i] += add[at + i];
                    }
                    if (boxed) {
                        uint32_t w[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) w[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
                        box_bf16(&maps.out[o], w, col, row - lane, 0);
                        return;
                    }
                    float *to = partial ? pr.part + (long long)u.cut * pr.M * pr.N : pr.sum;
                    if (whole && (sums || (pr.f32 && pr.wide))) {
                        if (!sums) to = (float *)pr.out + (long long)(row / pr.T) * pr.out_b + (long long)(row % pr.T) * pr.out_t + col;
                        else to += at;
                        if (in) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) reinterpret_cast<float4 *>(to)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                        }
                        return;
                    }
                    // Rows of no particular alignment: turned in shared memory, so that a warp writes a row's 32 columns at a time
                    float *turn = reinterpret_cast<float *>(boxes + e * BOX);
                    if (lane == 0) bulk_wait_read();
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 32; ++i) turn[lane * 32 + (i ^ lane)] = v[i];
                    __syncwarp();
                    const int rows = min(32, pr.M - (row - lane)), row0 = row - lane;
                    if (lane < live) {
                        // one column a lane: pointers to the first row's, and the distance of rows
                        const long long first = (long long)row0 * pr.N + col + lane, pitch = sums ? pr.N : pr.pitch;
                        const float *more = add && !whole ? add + first : nullptr;
                        auto put = [&](auto *dst) {
#pragma unroll 4
                            for (int r = 0; r < rows; ++r) {
                                float f = turn[r * 32 + (lane ^ r)];
                                if (more) f += more[r * (long long)pr.N];
                                if (pitch) st_out(dst + r * pitch, f);
                                else st_out(dst + (long long)((row0 + r) / pr.T) * pr.out_b + (long long)((row0 + r) % pr.T) * pr.out_t, f);
                            }
                        };
                        const long long begin = sums ? first : (pitch ? row0 * pitch : 0) + col + lane;
                        if (sums) put(to + begin);
                        else if (pr.f32) put((float *)pr.out + begin);
                        else put((__nv_bfloat16 *)pr.out + begin);
                    }
                    __syncwarp();
                }
            };
            auto get = [&](int c, auto &v) {
                constexpr int W = sizeof(v) / sizeof(v[0]);
                uint32_t r[W / 32][32];
#pragma unroll
                for (int h = 0; h < W / 32; ++h) tmem_ld32(tmem + (n & 1) * TILE + half * HALF + lanes + c + 32 * h, r[h]);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < W; ++i) v[i] = __uint_as_float(r[i / 32][i % 32]);
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
                // columns at a time: with 64, maxima and exponentials have chains enough to hide their latency; OUT has nothing to hide
                constexpr int WIDE = EPI == OUT ? 32 : 64;
#pragma unroll 1
                for (int c = 0; c < HALF; c += WIDE) {
                    float v[WIDE];
                    get(c, v);
                    finish(c, v);
                }
                release();
            }
            if (EPI == STATS && in) p.part[(long long)(2 * (u.n / TILE) + half) * pr.M + row] = make_float2(mx, sum);
        }
        if (lane == 0) bulk_wait_all();
    }
    __syncwarp();
    __syncthreads();
    // The last commit arrives on DONE of both blocks, and that the even one has seen its own says nothing about the other's: the odd
    // block stays until its own has come too (every tile is out, so it is on its way), or the arrival might find the barriers of the next kernel.
    if (warp == 1 && rank == 1) {
        volatile int never = 0;
        if (lane == 0) pair_wait(&bar[DONE], 0, BUDGET, &never);
        __syncwarp();
    }
    pair_sync();   // the other block's barriers are not touched any more
    tc_fence_after();
    if (warp == 1) pair_tmem_dealloc(tmem, 512);
}

// One block: R rows, each 256 / R threads that take every so manieth of the row's pieces; then those in a fixed order.
template <int R>
__global__ void __launch_bounds__(256) k_lse(const __grid_constant__ Gemm p, const float2 *part, int P, int M, float *loss, float *lse)
{
    constexpr int S = 256 / R;
    __shared__ float2 sm[S][R];
    let_next_start();
    wait_for_last();
    const int i = threadIdx.x % R, w = threadIdx.x / R, r = blockIdx.x * R + i;
    float mx = kNone, sum = 0.f;
    auto join = [&](float2 q) {
        const float top = fmaxf(mx, q.x);
        sum = sum * exp2f((mx - top) * kLog2e) + q.y * exp2f((q.x - top) * kLog2e);
        mx = top;
    };
    if (r < M) {
#pragma unroll 4
        for (int j = w; j < P; j += S) join(part[(long long)j * M + r]);
    }
    sm[w][i] = make_float2(mx, sum);
    for (int h = S / 2; h > 0; h >>= 1) {
        __syncthreads();
        if (w < h) {
            mx = sm[w][i].x;
            sum = sm[w][i].y;
            join(sm[w + h][i]);
            sm[w][i] = make_float2(mx, sum);
        }
    }
    if (w == 0 && r < M) {
        const float l = mx + logf(sum);
        lse[r] = l;
        loss[r] = target_of(p, r, false) < 0 ? 0.f : l - p.row[r];
    }
}

// The largest finite |dloss| of the tokens that have a target, into a word that begin() cleared: magnitudes are ordered as their bits.
__global__ void __launch_bounds__(256) k_scale(const __grid_constant__ Gemm p, int M, uint32_t *scale)
{
    let_next_start();
    wait_for_last();
    float top = 0.f;
    for (int i = blockIdx.x * 256 + threadIdx.x; i < M; i += gridDim.x * 256) {
        const float g = fabsf(p.dloss[(long long)(i / p.T) * p.g_b + (long long)(i % p.T) * p.g_t]);
        if (g > top && g <= 3.4e38f && target_of(p, i, false) >= 0) top = g;
    }
    const uint32_t v = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
    if ((threadIdx.x & 31) == 0 && v) atomicMax(scale, v);
}

// x and w into [planes][rows][pitch] bf16: as they are, or as three planes, the largest first.  A thread has 8 columns of a row,
// 2^shift threads a row at a time; the first blocks have x's rows.  Backward, rows of x without a target become 0: the products would
// take 0 times what is not finite for NaN in all of dw.
struct Packing {
    Gemm g;
    const void *from[2];
    long long b[2], t[2], pitch[2], plane[2];
    __nv_bfloat16 *to[2];
    int rows[2], T[2], blocks[2];
    int K, shift, mask;
    int whole[2];                   // rows of whole 16 bytes that start at 16 bytes (bf16)
};

template <class T>
__global__ void __launch_bounds__(256) k_pack(const __grid_constant__ Packing p)
{
    let_next_start();
    wait_for_last();
    const int o = blockIdx.x >= p.blocks[0], per = 256 >> p.shift;
    const int r = (blockIdx.x - (o ? p.blocks[0] : 0)) * per + (threadIdx.x >> p.shift);
    if (r >= p.rows[o]) return;
    const T *from = (const T *)p.from[o] + (long long)(r / p.T[o]) * p.b[o] + (long long)(r % p.T[o]) * p.t[o];
    __nv_bfloat16 *to = p.to[o] + r * p.pitch[o];
    const bool none = p.mask && o == 0 && target_of(p.g, r, false) < 0;
    for (int c = (threadIdx.x & ((1 << p.shift) - 1)) * 8; c < p.pitch[o]; c += 8 << p.shift) {
        if (sizeof(T) == 2 && (none || p.whole[o])) {
            // the copy's rows may be 8 columns longer than a row, and what lies behind the last one is not the caller's
            *reinterpret_cast<uint4 *>(to + c) = none || c >= p.K ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4 *>(from + c);
            continue;
        }
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = c + e < p.K && !none ? ld_in(from + c + e) : 0.f;
#pragma unroll
        for (int pl = 0; pl < (sizeof(T) == 4 ? 3 : 1); ++pl) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                w[e] = pack_bf16(f[2 * e], f[2 * e + 1]);
                f[2 * e] -= __uint_as_float(w[e] << 16);   // what the next plane holds
                f[2 * e + 1] -= __uint_as_float(w[e] & 0xFFFF0000u);
            }
            *reinterpret_cast<uint4 *>(to + pl * p.plane[o] + c) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// bf16 rows of 16 bytes' multiples into dense ones of any width: a thread writes 8 elements, which it shifts out of the 16 that they lie
// in, or, across rows, gathers.  (From the tiles such rows go 2 bytes a lane: 29 tokens, 69380 entries of 1591 features took 403 us for
// the product alone, now 216 and this.)
__global__ void __launch_bounds__(256) k_unpack(const __nv_bfloat16 *from, long long pitch, __nv_bfloat16 *to, int K, long long all)
{
    let_next_start();
    wait_for_last();
    const long long step = (long long)gridDim.x * 256 * 8;
    for (long long i = (blockIdx.x * 256ll + threadIdx.x) * 8; i < all; i += step) {
        const long long row = all < 1ll << 32 ? (unsigned)i / (unsigned)K : i / K;
        int col = (int)(i - row * K);
        const int n = (int)min(8ll, all - i);
        const __nv_bfloat16 *line = from + row * pitch;
        if (n == 8 && col + 8 <= K) {
            const uint4 *q = reinterpret_cast<const uint4 *>(line) + (col >> 3);
            const uint4 lo = q[0], hi = col & 7 ? q[1] : make_uint4(0, 0, 0, 0);
            uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int j = 0; j < 6; ++j) w[j] = col & 4 ? w[j + 2] : w[j];
#pragma unroll
            for (int j = 0; j < 5; ++j) w[j] = col & 2 ? w[j + 1] : w[j];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = col & 1 ? __funnelshift_r(w[j], w[j + 1], 16) : w[j];
            *reinterpret_cast<uint4 *>(to + i) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            for (int j = 0; j < n; ++j) {
                to[i + j] = line[col];
                if (++col == K) {
                    col = 0;
                    line += pitch;
                }
            }
        }
    }
}

// Sums of a product's parts in a fixed order, and what OUT does with a whole one.  A thread has 4 columns of a row where `wide`.
template <int V>
__global__ void __launch_bounds__(256) k_join(const __grid_constant__ Product o)
{
    let_next_start();
    wait_for_last();
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
    return lay::tensor_map(m, false, o.p, cols, rows, planes, o.pitch, o.plane, 64, high, 128);
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

template <int EPI, bool SEG, int NT = TILE>
cudaError_t launch_as(const Maps &m, Gemm &p, cudaStream_t st)
{
    p.seg = p.np > 1 ? kSegment : kLongSegment;
    auto kernel = k_gemm<EPI, SEG, NT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    long long units = 0, pairs = pairs_at_most();
    for (const Product &o : p.of) units += (long long)o.mt * o.nt * o.cuts;
    return start(kernel, 2 * (units < pairs ? units : pairs), THREADS, SMEM, st, m, p);
}

template <int EPI, int NT = TILE>
cudaError_t launch(const Maps &m, Gemm &p, cudaStream_t st)
{
    const bool seg = p.np > 1 || (EPI != OUT && p.of[0].kb > kLong);
    return seg ? launch_as<EPI, true, NT>(m, p, st) : launch_as<EPI, false, NT>(m, p, st);
}

// Clears the status word and the scale; copies what the tensor maps cannot read in place.
cudaError_t begin(const Call &c, bool bwd, cudaStream_t st)
{
    cudaError_t e = cudaMemsetAsync(c.status, 0, 2 * sizeof(uint32_t), st);   // and the scale behind it
    if (e != cudaSuccess || c.M == 0 || !(c.pack_x || c.pack_w)) return e;
    Packing p = {};
    const dn_view *views[2] = {c.x, c.w};
    const Operand *to[2] = {&c.xo, &c.wo};
    const int rows[2] = {c.M, c.V}, per[2] = {c.s->T, c.V};
    const bool packs[2] = {c.pack_x, c.pack_w};
    p.g = common(c);
    p.K = c.K;
    p.mask = bwd;
    while (p.shift < 8 && 8 << p.shift < c.K) ++p.shift;
    for (int o = 0; o < 2; ++o) {
        p.T[o] = per[o];
        if (!packs[o]) continue;
        p.from[o] = views[o]->data;
        p.b[o] = views[o]->batch;
        p.t[o] = views[o]->time;
        p.whole[o] = c.K % 8 == 0 && (uintptr_t)p.from[o] % 16 == 0 && p.b[o] % 8 == 0 && p.t[o] % 8 == 0;
        p.to[o] = (__nv_bfloat16 *)to[o]->p;
        p.pitch[o] = to[o]->pitch;
        p.plane[o] = to[o]->plane;
        p.rows[o] = rows[o];
        p.blocks[o] = (int)(((long long)rows[o] + (256 >> p.shift) - 1) / (256 >> p.shift));
    }
    const unsigned blocks = (unsigned)p.blocks[0] + (unsigned)p.blocks[1];
    return start(c.s->dtype == DN_F32 ? k_pack<float> : k_pack<__nv_bfloat16>, blocks, 256, 0, st, p);
}

// SCORE: pairs take equal shares of the vocabulary, in as few rounds as tiles of 256 rows need
int score_units(int V, int &share)
{
    const int pairs = pairs_at_most(), rounds = (tiles_of(V) + pairs - 1) / pairs;
    share = (int)(((long long)V + 2ll * pairs * rounds - 1) / (2ll * pairs * rounds));
    return (int)(((long long)V + 2 * share - 1) / (2 * share));
}

}  // namespace

cudaError_t join_rows(const Gemm &p, const Call &c, int P, cudaStream_t st)
{
    const float2 *part = c.part;
    return c.M > 2048 ? start(k_lse<32>, (c.M + 31) / 32, 256, 0, st, p, part, P, c.M, c.loss, c.lse)
                      : start(k_lse<4>, (c.M + 3) / 4, 256, 0, st, p, part, P, c.M, c.loss, c.lse);
}

// Where a product's bf16 rows cannot leave by boxes: has them left in `at` instead, and says so
static bool by_way_of(Product &o, CUtensorMap *map, void *at, int rows)
{
    const long long pitch = copy_pitch(o.N);
    if (!at || o.out_box || o.cuts > 1 || o.sum || o.f32 || o.pitch != o.N || (uintptr_t)o.out % 16 ||
        !lay::tensor_map(map, false, at, o.N, rows, 1, pitch, 0, 32, 32, 64))
        return false;
    o.out_box = 1;
    return true;
}

static cudaError_t unpack(const Product &o, const void *at, cudaStream_t st)
{
    const long long all = (long long)o.M * o.N, need = (all + 2047) / 2048, most = 16ll * lay::sm_count();
    return start(k_unpack, need < most ? need : most, 256, 0, st, (const __nv_bfloat16 *)at, copy_pitch(o.N), (__nv_bfloat16 *)o.out, o.N, all);
}

static cudaError_t join(const Product &o, cudaStream_t st)
{
    if (o.cuts == 1) return cudaSuccess;
    const bool four = o.N % 4 == 0;
    const long long n = ((long long)o.M * o.N / (four ? 4 : 1) + 255) / 256, most = 16ll * lay::sm_count();
    const unsigned blocks = (unsigned)(n < most ? n : most);
    return start(four ? k_join<4> : k_join<1>, blocks, 256, 0, st, o);
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
    p.tgt = (const int64_t *)c.targets->data;
    p.tgt_b = c.targets->batch;
    p.tgt_t = c.targets->time;
    p.ignore = c.s->ignore_index;
    p.T = c.s->T;
    p.V = c.V;
    if (c.dloss) {
        p.dloss = (const float *)c.dloss->data;
        p.g_b = c.dloss->batch;
        p.g_t = c.dloss->time;
    }
    p.scale = (const float *)(c.status + 1);
    p.lse = c.lse;
    p.row = c.row;
    p.part = c.part;
    return p;
}

int tiles_of(int n) { return (int)(((long long)n + TILE - 1) / TILE); }

// How the contractions of a piece's two products are cut: a unit not costlier than a pair's share of all, so that a few long
// tiles do not keep the rest waiting, and not below 8 stages' worth; bf16: nor above kPart.
void cuts_of(int M, int K, int n, int planes, int &dx, int &dw)
{
    const long long np = planes == 1 ? 1 : 6, a = ((long long)n + BK - 1) / BK, b = ((long long)M + BK - 1) / BK;
    const long long nx = (long long)tiles_of(K) * tiles_of(M), nw = (long long)tiles_of(K) * tiles_of(n), pairs = pairs_at_most();
    long long share = (nx * (a * np + way_out(np)) + nw * (b * np + way_out(np)) + pairs - 1) / pairs / np;
    if (share < 8) share = 8;
    if (planes == 1 && share > kPart) share = kPart;
    dx = (int)((a + share - 1) / share);
    dw = (int)((b + share - 1) / share);
}

// Pieces of a row that the forward pass leaves for k_lse
int parts_of(int M, int V)
{
    if (M > kScore) return 2 * tiles_of(V);
    int share;
    const int units = score_units(V, share), pairs = pairs_at_most();
    return 2 * 4 * (units < pairs ? units : pairs);
}

cudaError_t forward(const Call &c, cudaStream_t st)
{
    cudaError_t e = begin(c, false, st);
    if (e != cudaSuccess || c.M == 0) return e;
    if (c.few) return few_forward(c, st);
    Maps m = {};
    Gemm p = common(c);
    if (c.M > kScore) {
        if (!make_map(&m.a[0], c.xo, c.K, c.M, c.planes, HALF) || !make_map(&m.b[0], c.wo, c.K, c.V, c.planes, HALF)) return cudaErrorInvalidValue;
        size(p.of[0], c.M, c.V, c.K);
        e = launch<STATS>(m, p, st);
    } else {
        const int nt = c.M <= 32 ? 32 : c.M <= 64 ? 64 : 128;
        if (!make_map(&m.a[0], c.wo, c.K, c.V, c.planes, HALF) || !make_map(&m.b[0], c.xo, c.K, c.M, c.planes, nt / 2)) return cudaErrorInvalidValue;
        size(p.of[0], c.V, c.M, c.K);
        p.of[0].mt = score_units(c.V, p.share);
        p.of[0].nt = 1;
        // the planes change places
        const uint32_t pa = p.pa;
        p.pa = p.pb;
        p.pb = pa;
        e = nt == 32 ? launch<SCORE, 32>(m, p, st) : nt == 64 ? launch<SCORE, 64>(m, p, st) : launch<SCORE, 128>(m, p, st);
    }
    if (e != cudaSuccess) return e;
    return join_rows(p, c, parts_of(c.M, c.V), st);
}

cudaError_t backward(const Call &c, cudaStream_t st)
{
    cudaError_t e = begin(c, true, st);
    if (e != cudaSuccess) return e;
    const bool f32 = c.s->dtype == DN_F32;
    if (c.M == 0) return cudaMemsetAsync(c.dw, 0, (size_t)c.V * c.K * (f32 ? 4 : 2), st);
    if (c.few) return few_backward(c, st);
    const Operand d = {c.d, c.piece, (long long)c.M * c.piece};
    Maps logits = {}, outs = {};
    if (!make_map(&logits.a[0], c.xo, c.K, c.M, c.planes, HALF) || !make_map(&logits.b[0], c.wo, c.K, c.V, c.planes, HALF) ||
        !make_map(&outs.b[1], c.xo, c.K, c.M, c.planes, BK) || !make_map(&outs.b[0], c.wo, c.K, c.V, c.planes, BK))
        return cudaErrorInvalidValue;
    const size_t el = f32 ? 4 : 2;
    const int groups = (c.M + 255) / 256;
    if ((e = start(k_scale, groups < 128 ? groups : 128, 256, 0, st, common(c), c.M, c.status + 1)) != cudaSuccess) return e;
    for (int v0 = 0; v0 < c.V; v0 += c.piece) {
        const int n = c.V - v0 < c.piece ? c.V - v0 : c.piece;
        const bool first = v0 == 0, last = v0 + n == c.V;
        // the maps end where this piece does: nothing behind it is read
        if (!make_map(&outs.a[0], d, n, c.M, c.planes, HALF) || !make_map(&outs.a[1], d, n, c.M, c.planes, BK)) return cudaErrorInvalidValue;
        if (!lay::tensor_map(&logits.out[0], false, c.d, n, c.M, c.planes, d.pitch, d.plane, 32, 32, 64)) return cudaErrorInvalidValue;
        Gemm p = common(c);
        size(p.of[0], c.M, n, c.K);
        p.of[0].b_row = p.v0 = v0;
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
            o->wide = f32 && (uintptr_t)o->out % 16 == 0 && o->out_b % 4 == 0 && o->out_t % 4 == 0;
        }
        // results that tensor maps can describe: dx of rows at one distance, dw, the sums of dx over pieces.  A box is cut off at
        // 16 bytes, not at the element: a row has to end there.
        dx.pitch = c.s->B == 1 || dx.out_b == dx.out_t * dx.T ? dx.out_t : c.s->T == 1 ? dx.out_b : 0;
        dw.pitch = c.K;
        dx.out_box = !f32 && last && dx.cuts == 1 && dx.pitch > 0 && c.K % 8 == 0 && lay::tensor_map(&outs.out[0], false, dx.out, c.K, c.M, 1, dx.pitch, 0, 32, 32, 64);
        dw.out_box = !f32 && dw.cuts == 1 && lay::tensor_map(&outs.out[1], false, dw.out, c.K, n, 1, c.K, 0, 32, 32, 64);
        dx.sum_box = !last && lay::tensor_map(&outs.sum, true, c.acc, c.K, c.M, 1, c.K, 0, 32, 32, 128) ? first ? 1 : 2 : 0;
        const bool dx_later = last && by_way_of(dx, &outs.out[0], c.dx_rows, c.M), dw_later = by_way_of(dw, &outs.out[1], c.dw_rows, n);
        if ((e = launch<OUT>(outs, p, st)) != cudaSuccess || (e = join(dx, st)) != cudaSuccess || (e = join(dw, st)) != cudaSuccess) return e;
        if ((dx_later && (e = unpack(dx, c.dx_rows, st)) != cudaSuccess) || (dw_later && (e = unpack(dw, c.dw_rows, st)) != cudaSuccess)) return e;
    }
    return cudaSuccess;
}

}  // namespace xent
}  // namespace gdn

// Selective state space scan: backward.
//
// With g = dy silu(z), a_t = exp(delta_t A), and the lane layout of scan.cuh:
//     dh_t = C_t g_t + a_{t+1} dh_{t+1}      (from the last token back; dhT enters at a
//                                             sequence's last token)
//     e_t  = dh_t a_t h_{t-1},  p_t = sum_n dh_t B_t,  o_t = sum_n C_t h_t + D x_t
//     dx = delta p + D g,  ddt = (sum_n e A + x p) softplus'(dt),  dz = dy o silu'(z)
//     dA += delta e,  dB_t = sum_c delta x dh_t,  dC_t = sum_c g h_t,  dh0 = a_0 dh_0
//
// A block walks its channels' tokens backwards in tiles of 16.  From the kept state that enters
// it the tile is run forward once, the state before every token into shared memory, and then back.
// a_t is an exponential in both.  Tiles of 8 were 1553 us for the training step below instead of
// 1450: barriers, and the elementwise steps' latency, twice as often.  Both of a tile's kept
// states, as two recurrences at once, with asynchronous copies: no faster (2067 us the whole step
// against 2070).
// Tried with tiles of 8, the training step then at 2.3 ms: the tile's states in registers (16 tokens
// of them spill: 4.0 ms), groups of 4 tokens with states and decays in registers, run forward twice (2.7 ms),
// one channel a lane (2.8 ms: shared-memory reads double), dB and dC summed over channels on the
// tensor cores in tf32 (2.3 ms, no gain: the butterfly is not what it waits for).
//
// Bound by latency and issue: 203 instructions a token and 16 channels (a warp), 52 of them
// packed multiply-adds, 16 exponentials, 46 for the sums over lanes; two blocks of 4 warps fit an
// SM (registers, shared memory), and 8 x 4096 tokens of 2048 channels are 1.7 a SM: issue slots 51 %
// used, the shared-memory port 55 %, 1.45 ms.  The whole training step: 1.98 ms.
//
// Sums.  Over a channel's states (o, p, sum e A): the lanes' butterfly.  Over channels
// (dB, dC): a butterfly over the warp's channels that leaves a share of the 2 S values in
// each, the block's warps through shared memory, and the channel tiles by a second
// kernel from one partial result a tile.  Over tokens (dA, dD, ddt_bias): registers, then
// rows and segments by col_sum.  All in a fixed order, no atomics.
//
// Few rows: segments of the time axis, the entering dh composed from a first pass (SUM)
// over all but the first segment, as in the forward pass.
#include <type_traits>

#include "scan.cuh"

namespace gdn {
namespace lay {

namespace {

constexpr float kLn2 = 0.6931471805599453f;

template <class T>
struct BwdIo {
    View<const T> x, dt, b, c, z, dy;
    View<T> dx, ddt, dz;
    const float *keep, *dhT;
    float *dh0;
    float *segP, *segH;     // [B][K][D][Np]
    float *part_a;          // [B * K][D][N]
    float *part_d;          // [B * K][2][D]: dD, ddt_bias
    float *part_bc;         // [B][channel tiles][T][2 Np]
};

template <class Cfg>
struct BwdShared {
    static constexpr int WARPS = Cfg::NT / 32;
    float2 dd[Cfg::TT][Cfg::CH];                       // delta, delta x
    float g[Cfg::TT][Cfg::RS];
    float x[Cfg::TT][Cfg::RS], s[Cfg::TT][Cfg::RS], gz[Cfg::TT][Cfg::RS];   // x, softplus', dy silu'(z); then dx, ddt, dz
    __align__(16) float b[Cfg::TT][Cfg::Np];
    __align__(16) float c[Cfg::TT][Cfg::Np];
    __align__(16) float st[Cfg::TT][Cfg::CT][Cfg::NT][Cfg::S];              // the state before every token
    float bc[Cfg::TT][WARPS][2 * Cfg::Np];
    int seq[32];
    uint32_t edge[2];
};

// sum += v with the rounding error kept in rest and put into the next term (Kahan): the sums over
// a whole row of tokens whose terms largely cancel
__device__ __forceinline__ void add_kept(float &sum, float &rest, float v)
{
    const float y = v - rest, t = sum + y;
    rest = (t - sum) - y;
    sum = t;
}

template <class T, class Cfg, int VEC, bool SUM>
__global__ void __launch_bounds__(Cfg::NT, SUM ? 4 : 2) k_scan_bwd(ScanDims g, BwdIo<T> io)
{
    constexpr int L = Cfg::L, S = Cfg::S, CT = Cfg::CT, M = Cfg::M, Np = Cfg::Np, CH = Cfg::CH, P = S / 2, TT = Cfg::TT;
    constexpr int NV = Cfg::EPT / VEC, NBC = Cfg::NBC, KEEP = keep_of(Np);
    static_assert(TT % KEEP == 0, "a tile starts from a kept state");
    using Shared = BwdShared<Cfg>;
    extern __shared__ __align__(16) char smem_raw[];
    Shared &sm = *reinterpret_cast<Shared *>(smem_raw);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = lane / M, n0 = l * S;
    const int ch = (warp * M + lane % M) * CT;
    int id = blockIdx.x;
    const int tiles = g.G * g.tiles, tile = id % tiles;
    id /= tiles;
    const int nseg = SUM ? g.K - 1 : g.K, k = id % nseg + (SUM ? 1 : 0), b = id / nseg;
    const int grp = tile / g.tiles, cg0 = (tile - grp * g.tiles) * CH;
    const int c0 = grp * g.Dg + cg0;
    const long long c = c0 + ch;
    bool live[CT];
#pragma unroll
    for (int e = 0; e < CT; ++e) live[e] = cg0 + ch + e < g.Dg;
    const int ts = k * g.seg, te = min(ts + g.seg, g.T);
    const bool gated = io.z.p != nullptr;

    float2 a2[CT][P], dh[CT][P], dA[CT][P], open[CT];   // open: 1, 0 before a sequence start
    float Dc[CT], aD[CT], aBias[CT], rD[CT], rBias[CT], total[CT];
#pragma unroll
    for (int e = 0; e < CT; ++e) {
        load_states<S>(a2[e], g.A + (c + e) * g.N, n0, g.N, live[e]);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            a2[e][i] = mul2(a2[e][i], two(kLog2e));
            dh[e][i] = dA[e][i] = two(0.f);
        }
        open[e] = two(1.f);
        Dc[e] = !SUM && g.Dskip && live[e] ? g.Dskip[c + e] : 0.f;
        aD[e] = aBias[e] = rD[e] = rBias[e] = total[e] = 0.f;
        // what the segments behind this one send back
        if constexpr (!SUM) {
            if (k < g.K - 1 && live[e]) load_pairs<S>(dh[e], io.segH + (((size_t)b * g.K + k) * g.D + c + e) * Np + n0);
        }
    }

    // this thread's vectors of a tile: tokens vt, vt + ES, ..., channels vc .. vc + VEC - 1
    constexpr int RV = CH / VEC, ES = Cfg::NT / RV;
    const int vt = tid / RV, vc = tid % RV * VEC;
    const bool col = cg0 + vc < g.Dg;
    const int cv = c0 + (col ? vc : 0);
    Vec<T, VEC> xn[NV], dn[NV], zn[NV], gn[NV];
    T br[NBC], cr[NBC];
    float2 kn[CT][P];   // the state that enters the tile
    const float *kp = SUM ? nullptr : io.keep + ((size_t)b * ((g.T + KEEP - 1) / KEEP) + (te - 1) / TT * (TT / KEEP)) * g.D * Np;
    unsigned place[CT];
#pragma unroll
    for (int e = 0; e < CT; ++e) place[e] = keep_place<Cfg>(g, grp, cg0 + ch + e, l);
    float bias[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) bias[i] = col && g.bias ? g.bias[cv + i] : 0.f;
    auto fetch = [&](int t0) {
#pragma unroll
        for (int e = 0; e < NV; ++e) {
            const int t = t0 + vt + e * ES;
            xn[e].zero();
            dn[e].zero();
            zn[e].zero();
            gn[e].zero();
            if (col && t >= ts && t < te) {
                if (!SUM) xn[e].load(io.x.at(b, 0, t) + cv);
                dn[e].load(io.dt.at(b, 0, t) + cv);
                gn[e].load(io.dy.at(b, 0, t) + cv);
                if (gated) zn[e].load(io.z.at(b, 0, t) + cv);
            }
        }
#pragma unroll
        for (int e = 0; e < NBC; ++e) {
            const int i = tid + e * Cfg::NT, t = t0 + i / Np, n = i % Np;
            st_out(&br[e], 0.f);
            st_out(&cr[e], 0.f);
            if (i < TT * Np && t >= ts && t < te && n < g.N) {
                if (!SUM) br[e] = io.b.at(b, grp, t)[n];
                cr[e] = io.c.at(b, grp, t)[n];
            }
        }
        if constexpr (!SUM) {
#pragma unroll
            for (int e = 0; e < CT; ++e) {
#pragma unroll
                for (int i = 0; i < P; ++i) kn[e][i] = two(0.f);
                if (live[e] && t0 >= ts) load_pairs<S>(kn[e], kp + place[e]);
            }
            kp -= (size_t)g.D * Np * (TT / KEEP);   // read no further than the segment's first tile
        }
    };
    const int last = ts + (te - ts - 1) / TT * TT;
    fetch(last);

    for (int t0 = last; t0 >= ts; t0 -= TT) {
        // 1. the tile into shared memory
#pragma unroll
        for (int e = 0; e < NV; ++e) {
            float x[VEC], d[VEC], z[VEC], gy[VEC], sp[VEC], gz[VEC];
            xn[e].get(x);
            dn[e].get(d);
            zn[e].get(z);
            gn[e].get(gy);
            const int t = vt + e * ES;
            const bool in = col && t0 + t < te;
#pragma unroll
            for (int i = 0; i < VEC; i += 2) {
                float2 v = add2(pair_at(d, i), pair_at(bias, i)), der = two(1.f), w = two(0.f);
                if (g.softplus) softplus(v, v, der);
                if constexpr (!SUM) w = mul2(v, pair_at(x, i));
                if (!in) v = w = two(0.f);
                if constexpr (VEC > 1) *reinterpret_cast<float4 *>(&sm.dd[t][vc + i]) = make_float4(v.x, w.x, v.y, w.y);
                else sm.dd[t][vc] = make_float2(v.x, w.x);
                put_pair(sp, i, der);
                float2 gg = pair_at(gy, i);
                if (gated) {
                    const float2 zz = pair_at(z, i), sg = sigmoid2(zz);
                    if (!SUM) put_pair(gz, i, mul2(gg, make_float2(dsilu(zz.x, sg.x), dsilu(zz.y, sg.y))));
                    gg = mul2(gg, mul2(zz, sg));
                }
                put_pair(gy, i, gg);
            }
            store_wide<VEC>(&sm.g[t][vc], gy);
            if constexpr (!SUM) {
                store_wide<VEC>(&sm.x[t][vc], x);
                store_wide<VEC>(&sm.s[t][vc], sp);
                if (gated) store_wide<VEC>(&sm.gz[t][vc], gz);
            }
        }
#pragma unroll
        for (int e = 0; e < NBC; ++e) {
            const int i = tid + e * Cfg::NT;
            if (i < TT * Np) {
                if (!SUM) sm.b[i / Np][i % Np] = ld_in(&br[e]);
                sm.c[i / Np][i % Np] = ld_in(&cr[e]);
            }
        }
        if (tid < 32) tile_edges(g, b, t0, min(TT, te - t0), sm.seq, sm.edge);
        __syncthreads();
        float2 h[CT][P];   // forward: the state before the token at hand; back: the one behind it
        if constexpr (!SUM) {
#pragma unroll
            for (int e = 0; e < CT; ++e)
#pragma unroll
                for (int i = 0; i < P; ++i) h[e][i] = kn[e][i];
        }
        fetch(t0 - TT);
        const uint32_t starts = sm.edge[0], ends = sm.edge[1];
        // Sequence starts and ends: the states and gradients that come and go there.  Tiles without one,
        // nearly all, run a copy of the loops without this.
        auto end_of = [&](int t) {
            if ((ends >> t & 1) && io.dhT) {
#pragma unroll
                for (int e = 0; e < CT; ++e) {
                    float2 v[P];
                    load_states<S>(v, io.dhT + ((size_t)sm.seq[t] * g.D + c + e) * g.N, n0, g.N, live[e]);
#pragma unroll
                    for (int i = 0; i < P; ++i) dh[e][i] = add2(dh[e][i], v[i]);
                }
            }
        };
        auto initial = [&](float2 (&v)[P], int t, int e) {
            load_states<S>(v, g.h0 + ((size_t)sm.seq[t] * g.D + c + e) * g.N, n0, g.N, live[e] && g.h0);
        };

        if constexpr (SUM) {
            auto back = [&](int t, auto edges) {
                float dl[CT], dx[CT], gg[CT];
                load_steps<CT>(dl, dx, &sm.dd[t][ch]);
                load_ct<CT>(gg, &sm.g[t][ch]);
                float2 cc[P];
                load_pairs<S>(cc, &sm.c[t][n0]);
                if constexpr (decltype(edges)::value) end_of(t);
#pragma unroll
                for (int e = 0; e < CT; ++e) {
                    total[e] += dl[e];
#pragma unroll
                    for (int i = 0; i < P; ++i)
                        dh[e][i] = mul2(decay2(dl[e], a2[e][i]), fma2(two(gg[e]), cc[i], dh[e][i]));
                }
                if constexpr (decltype(edges)::value) {
                    if (starts >> t & 1) {
#pragma unroll
                        for (int e = 0; e < CT; ++e) {
                            open[e] = two(0.f);
                            total[e] = 0.f;
#pragma unroll
                            for (int i = 0; i < P; ++i) dh[e][i] = two(0.f);
                        }
                    }
                }
            };
            if ((starts | ends) == 0) {
#pragma unroll 4
                for (int t = TT - 1; t >= 0; --t) back(t, std::false_type());
            } else {
#pragma unroll 1
                for (int t = TT - 1; t >= 0; --t) back(t, std::true_type());
            }
            __syncthreads();
        } else {
            float2 tA[CT][P];
#pragma unroll
            for (int e = 0; e < CT; ++e)
#pragma unroll
                for (int i = 0; i < P; ++i) tA[e][i] = two(0.f);
            auto tile_back = [&](auto edges) {
                // 2. the tile's states, forward from the kept one
                auto forward = [&](int t) {
                    float dl[CT], dx[CT];
                    load_steps<CT>(dl, dx, &sm.dd[t][ch]);
                    float2 bb[P];
                    load_pairs<S>(bb, &sm.b[t][n0]);
#pragma unroll
                    for (int e = 0; e < CT; ++e) {
                        store_pairs<S>(sm.st[t][e][tid], h[e]);
                        if constexpr (decltype(edges)::value) {
                            if (starts >> t & 1) initial(h[e], t, e);
                        }
#pragma unroll
                        for (int i = 0; i < P; ++i) h[e][i] = fma2(decay2(dl[e], a2[e][i]), h[e][i], mul2(two(dx[e]), bb[i]));
                    }
                };
                if constexpr (decltype(edges)::value) {
#pragma unroll 1
                    for (int t = 0; t < TT; ++t) forward(t);
                } else {
#pragma unroll 4
                    for (int t = 0; t < TT; ++t) forward(t);
                }
                // 3. back through the tile
#pragma unroll 1
                for (int g0 = TT - L; g0 >= 0; g0 -= L) {
                    float po[CT][L], pp[CT][L], pe[CT][L];
#pragma unroll
                    for (int j = L - 1; j >= 0; --j) {
                        const int t = g0 + j;
                        float dl[CT], dx[CT], gg[CT];
                        load_steps<CT>(dl, dx, &sm.dd[t][ch]);
                        load_ct<CT>(gg, &sm.g[t][ch]);
                        float2 bb[P], cc[P], vb[P], vc2[P], before[CT][P];
                        load_pairs<S>(bb, &sm.b[t][n0]);
                        load_pairs<S>(cc, &sm.c[t][n0]);
#pragma unroll
                        for (int e = 0; e < CT; ++e) load_pairs<S>(before[e], sm.st[t][e][tid]);
                        if constexpr (decltype(edges)::value) end_of(t);
#pragma unroll
                        for (int e = 0; e < CT; ++e) {
                            float2 o, p, e2, hp[P];
#pragma unroll
                            for (int i = 0; i < P; ++i) hp[i] = before[e][i];
                            if constexpr (decltype(edges)::value) {
                                if (starts >> t & 1) initial(hp, t, e);
                            }
#pragma unroll
                            for (int i = 0; i < P; ++i) {
                                dh[e][i] = fma2(two(gg[e]), cc[i], dh[e][i]);
                                const float2 da = mul2(decay2(dl[e], a2[e][i]), dh[e][i]);   // what goes on to t - 1
                                const float2 q = mul2(da, hp[i]);
                                o = i == 0 ? mul2(cc[i], h[e][i]) : fma2(cc[i], h[e][i], o);
                                p = i == 0 ? mul2(dh[e][i], bb[i]) : fma2(dh[e][i], bb[i], p);
                                e2 = i == 0 ? mul2(q, a2[e][i]) : fma2(q, a2[e][i], e2);
                                tA[e][i] = fma2(two(dl[e]), q, tA[e][i]);
                                vb[i] = e == 0 ? mul2(two(dx[e]), dh[e][i]) : fma2(two(dx[e]), dh[e][i], vb[i]);
                                vc2[i] = e == 0 ? mul2(two(gg[e]), h[e][i]) : fma2(two(gg[e]), h[e][i], vc2[i]);
                                dh[e][i] = da;
                                h[e][i] = before[e][i];
                            }
                            po[e][j] = o.x + o.y;
                            pp[e][j] = p.x + p.y;
                            pe[e][j] = e2.x + e2.y;
                        }
                        if constexpr (decltype(edges)::value) {
                            if (starts >> t & 1) {
#pragma unroll
                                for (int e = 0; e < CT; ++e) {
                                    if (io.dh0) store_states<S>(io.dh0 + ((size_t)sm.seq[t] * g.D + c + e) * g.N, dh[e], n0, g.N, live[e]);
#pragma unroll
                                    for (int i = 0; i < P; ++i) dh[e][i] = two(0.f);
                                }
                            }
                        }
                        // dB, dC over the warp's channels
                        float v[2 * S];
#pragma unroll
                        for (int i = 0; i < P; ++i) {
                            v[2 * i] = vb[i].x;
                            v[2 * i + 1] = vb[i].y;
                            v[S + 2 * i] = vc2[i].x;
                            v[S + 2 * i + 1] = vc2[i].y;
                        }
                        constexpr int left = 2 * S > M ? 2 * S / M : 1;   // values a lane ends with
                        int off = 0, cur = 2 * S;
#pragma unroll
                        for (int bit = M / 2; bit > 0; bit >>= 1) {
                            const bool up = lane & bit;
                            if (cur > 1) {
                                cur >>= 1;
#pragma unroll
                                for (int i = 0; i < cur; ++i) {
                                    const float send = up ? v[i] : v[i + cur], mine = up ? v[i + cur] : v[i];
                                    v[i] = mine + __shfl_xor_sync(0xffffffffu, send, bit);
                                }
                                off += up ? cur : 0;
                            } else {
                                v[0] += __shfl_xor_sync(0xffffffffu, v[0], bit);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < left; ++i) {
                            const int w = off + i;
                            sm.bc[t][warp][(w >= S ? Np : 0) + n0 + (w & (S - 1))] = v[i];
                        }
                    }
                    const int t = g0 + l;
                    float dl[CT], dx[CT], x[CT], gg[CT], sp[CT], gz[CT];
                    load_steps<CT>(dl, dx, &sm.dd[t][ch]);
                    load_ct<CT>(x, &sm.x[t][ch]);
                    load_ct<CT>(gg, &sm.g[t][ch]);
                    load_ct<CT>(sp, &sm.s[t][ch]);
                    if (gated) load_ct<CT>(gz, &sm.gz[t][ch]);
#pragma unroll
                    for (int e = 0; e < CT; ++e) {
                        const float o = lane_sum<L>(po[e], lane), p = lane_sum<L>(pp[e], lane), q = lane_sum<L>(pe[e], lane) * kLn2;
                        const float ddt = fmaf(p, x[e], q) * sp[e];
                        add_kept(aD[e], rD[e], gg[e] * x[e]);
                        add_kept(aBias[e], rBias[e], ddt);
                        if (gated) gz[e] *= fmaf(Dc[e], x[e], o);
                        x[e] = fmaf(dl[e], p, Dc[e] * gg[e]);
                        sp[e] = ddt;
                    }
                    store_ct<CT>(&sm.x[t][ch], x);
                    store_ct<CT>(&sm.s[t][ch], sp);
                    if (gated) store_ct<CT>(&sm.gz[t][ch], gz);
                }
            };
            if ((starts | ends) == 0) tile_back(std::false_type());
            else tile_back(std::true_type());
            // a tile's sum first, then the total: fewer roundings on the long axis
#pragma unroll
            for (int e = 0; e < CT; ++e)
#pragma unroll
                for (int i = 0; i < P; ++i) dA[e][i] = add2(dA[e][i], tA[e][i]);
            __syncthreads();

            // 4. the tile's results
#pragma unroll
            for (int e = 0; e < NV; ++e) {
                const int t = vt + e * ES;
                if (col && t0 + t < te) {
                    Vec<T, VEC> out;
                    float f[VEC];
                    load_wide<VEC>(f, &sm.x[t][vc]);
                    out.set(f);
                    out.store(io.dx.at(b, 0, t0 + t) + cv);
                    load_wide<VEC>(f, &sm.s[t][vc]);
                    out.set(f);
                    out.store(io.ddt.at(b, 0, t0 + t) + cv);
                    if (gated) {
                        load_wide<VEC>(f, &sm.gz[t][vc]);
                        out.set(f);
                        out.store(io.dz.at(b, 0, t0 + t) + cv);
                    }
                }
            }
            float *pb = io.part_bc + (((size_t)b * tiles + tile) * g.T + t0) * (2 * Np);
            const int n = min(TT, te - t0) * 2 * Np;
            for (int i = tid; i < n; i += Cfg::NT) {
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < Shared::WARPS; ++w) s += sm.bc[i / (2 * Np)][w][i % (2 * Np)];
                pb[i] = s;
            }
            __syncthreads();
        }
    }
    if constexpr (SUM) {
#pragma unroll
        for (int e = 0; e < CT; ++e) {
            if (!live[e]) continue;
            const size_t at = (((size_t)b * g.K + k) * g.D + c + e) * Np + n0;
            float2 p[P];
#pragma unroll
            for (int i = 0; i < P; ++i) p[i] = open[e].x == 0.f ? two(kCut) : ex2_2(mul2(two(total[e]), a2[e][i]));
            store_pairs<S>(io.segP + at, p);
            store_pairs<S>(io.segH + at, dh[e]);
        }
    } else {
        const size_t row = (size_t)b * g.K + k;
#pragma unroll
        for (int e = 0; e < CT; ++e) {
            store_states<S>(io.part_a + (row * g.D + c + e) * g.N, dA[e], n0, g.N, live[e]);
#pragma unroll
            for (int o = M; o < 32; o <<= 1) {
                aD[e] += __shfl_xor_sync(0xffffffffu, aD[e], o);
                aBias[e] += __shfl_xor_sync(0xffffffffu, aBias[e], o);
            }
            if (live[e] && l == 0) {
                io.part_d[row * 2 * g.D + c + e] = aD[e];
                io.part_d[(row * 2 + 1) * g.D + c + e] = aBias[e];
            }
        }
    }
}

// dB, dC: the channel tiles' partial results of a group, in order.
template <class T>
__global__ void k_scan_bc(const float *__restrict__ part, View<T> db, View<T> dc, int B, int T_, int N, int Np, int G, int tiles)
{
    const long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x;
    const int w = 2 * Np;
    if (i >= (long long)B * G * T_ * w) return;
    const int j = (int)(i % w);
    const long long r = i / w;
    const int t = (int)(r % T_), bg = (int)(r / T_), grp = bg % G, b = bg / G;
    const int n = j < Np ? j : j - Np;
    if (n >= N) return;
    const float *p = part + (((size_t)b * G + grp) * tiles * T_ + t) * w + j;
    float s = 0.f;
#pragma unroll 4
    for (int q = 0; q < tiles; ++q) s += p[(size_t)q * T_ * w];
    st_out((j < Np ? db : dc).at(b, grp, t) + n, s);
}

// Gradient of the initial state of an empty sequence: that of its final state.
__global__ void k_scan_empty_grad(const float *dhT, float *dh0, const int32_t *cu, int Nseq, long long per)
{
    const int s = blockIdx.y;
    if (cu && cu[s + 1] > cu[s]) return;
    const long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x;
    if (i < per) dh0[s * per + i] = dhT ? dhT[s * per + i] : 0.f;
}

struct Plan {
    int K, seg, tiles;
    size_t segP, segH, part_a, part_d, part_bc, total;
};

Plan plan_of(const dn_scan_shape *s)
{
    Plan p;
    int CH = 0;
    bwd_layout(s->N, [&](auto cfg) { CH = decltype(cfg)::CH; return cudaSuccess; });
    const int Dg = s->D / s->G, Np = scan_padded(s->N);
    p.tiles = (Dg + CH - 1) / CH;
    // Counted as two blocks of the main pass an SM and four of the first, which does a fifth of the work.
    // That is what their registers allow; shared memory, of which the first pass is given as much as the
    // main one, allows three of either up to 8 states, two up to 64 and one above.  With these counts the same
    // model would take 19 segments instead of 38 for one row of 16384 tokens and 1024 channels of 16 states
    const int k = plan_segments((long long)s->B * s->G * p.tiles, s->T, 2, 4, 0.2);
    p.seg = (int)((((long long)s->T + k - 1) / k + 15) / 16 * 16);   // whole tiles, whole spans between kept states
    p.K = p.seg > 0 ? (s->T + p.seg - 1) / p.seg : 1;
    size_t off = 0;
    auto take = [&](size_t floats) { const size_t o = off; off += align256(floats * sizeof(float)); return o; };
    const size_t rows = (size_t)s->B * p.K;
    p.segP = take(p.K > 1 ? rows * s->D * Np : 0);
    p.segH = take(p.K > 1 ? rows * s->D * Np : 0);
    p.part_a = take(rows * s->D * s->N);
    p.part_d = take(rows * 2 * s->D);
    p.part_bc = take((size_t)s->B * s->G * p.tiles * s->T * 2 * Np);
    p.total = off;
    return p;
}

template <class T, class Cfg, int VEC>
cudaError_t launch(const ScanCall &c, cudaStream_t st)
{
    const Plan p = plan_of(c.s);
    const dn_scan_grads *gr = c.gr;
    ScanDims g = scan_dims(c);
    g.tiles = p.tiles;
    g.K = p.K;
    g.seg = p.seg;
    auto F = [&](size_t o) { return (float *)(c.ws + o); };
    BwdIo<T> io;
    io.x = view_of<const T>(&c.io->x); io.dt = view_of<const T>(&c.io->dt);
    io.b = view_of<const T>(&c.io->b); io.c = view_of<const T>(&c.io->c);
    io.z = view_of<const T>(&c.io->z); io.dy = view_of<const T>(&gr->dy);
    io.dx = view_of<T>(&gr->dx); io.ddt = view_of<T>(&gr->ddt); io.dz = view_of<T>(&gr->dz);
    io.keep = c.keep; io.dhT = gr->dhT; io.dh0 = gr->dh0;
    io.segP = F(p.segP); io.segH = F(p.segH);
    io.part_a = F(p.part_a); io.part_d = F(p.part_d); io.part_bc = F(p.part_bc);
    const long long per = (long long)g.B * g.G * g.tiles;
    if (per * g.K > 0x7fffffffLL) return cudaErrorInvalidValue;
    const size_t smem = sizeof(BwdShared<Cfg>);
    cudaError_t e;
    if (g.K > 1) {
        e = cudaFuncSetAttribute(k_scan_bwd<T, Cfg, VEC, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        k_scan_bwd<T, Cfg, VEC, true><<<(unsigned)(per * (g.K - 1)), Cfg::NT, smem, st>>>(g, io);
        scan_carry<false>(g, io.segP, io.segH, Cfg::Np, st);
    }
    e = cudaFuncSetAttribute(k_scan_bwd<T, Cfg, VEC, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    k_scan_bwd<T, Cfg, VEC, false><<<(unsigned)(per * g.K), Cfg::NT, smem, st>>>(g, io);
    const long long n = (long long)g.B * g.G * g.T * 2 * Cfg::Np;
    if ((n + 255) / 256 > 0x7fffffffLL) return cudaErrorInvalidValue;
    k_scan_bc<T><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(io.part_bc, view_of<T>(&gr->db), view_of<T>(&gr->dc), g.B, g.T, g.N,
                                                            Cfg::Np, g.G, g.tiles);
    return cudaPeekAtLastError();
}

template <class T>
cudaError_t bwd_t(const ScanCall &c, cudaStream_t st)
{
    const dn_scan_shape *s = c.s;
    const dn_scan_io *io = c.io;
    const dn_scan_grads *gr = c.gr;
    if (gr->dh0 && c.Nseq > 0 && (c.cu || s->T == 0)) {
        const long long per = (long long)s->D * s->N;
        for (int s0 = 0; s0 < c.Nseq; s0 += 65535) {
            const int n = c.Nseq - s0 < 65535 ? c.Nseq - s0 : 65535;
            k_scan_empty_grad<<<dim3((unsigned)((per + 255) / 256), n), 256, 0, st>>>(gr->dhT ? gr->dhT + s0 * per : nullptr, gr->dh0 + s0 * per,
                                                                                     c.cu ? c.cu + s0 : nullptr, n, per);
        }
    }
    const Plan p = plan_of(s);
    if (s->T > 0) {
        const cudaError_t e = bwd_layout(s->N, [&](auto cfg) {
            using Cfg = decltype(cfg);
            constexpr int VEC = Cfg::VEC;
            if constexpr (VEC > 1) {
                const dn_view *all[] = {&io->x, &io->dt, &io->z, &gr->dy, &gr->dx, &gr->ddt, &gr->dz};
                bool v = (s->D / s->G) % VEC == 0;
                for (const dn_view *q : all) v = v && can_vector(q, sizeof(T), VEC * sizeof(T));
                if (v) return launch<T, Cfg, VEC>(c, st);
            }
            return launch<T, Cfg, 1>(c, st);
        });
        if (e != cudaSuccess) return e;
    }
    const long long rows = s->T > 0 ? (long long)s->B * p.K : 0;
    ColSum ra, rd;
    ra.part = (float *)(c.ws + p.part_a);
    ra.P = rows;
    ra.C = (long long)s->D * s->N;
    ra.kinds = 1;
    ra.dst[0] = gr->dA;
    ra.step[0] = 1;
    rd.part = (float *)(c.ws + p.part_d);
    rd.P = rows;
    rd.C = s->D;
    rd.kinds = 2;
    rd.dst[0] = gr->dD;
    rd.dst[1] = gr->ddt_bias;
    rd.step[0] = rd.step[1] = 1;
    return col_sum(ra, gr->dD || gr->ddt_bias ? &rd : nullptr, st);
}

}  // namespace

size_t scan_bwd_bytes(const dn_scan_shape *s) { return plan_of(s).total; }

cudaError_t scan_bwd(const ScanCall &c, cudaStream_t st)
{
    return c.s->dtype == DN_F32 ? bwd_t<float>(c, st) : bwd_t<__nv_bfloat16>(c, st);
}

}  // namespace lay
}  // namespace gdn

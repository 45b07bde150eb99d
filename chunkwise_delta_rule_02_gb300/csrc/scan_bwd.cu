// Selective state space scan: backward.
//
// With g = dy silu(z), a_t = exp(delta_t A), and the lane layout of scan.cuh:
//     dh_t = C_t g_t + a_{t+1} dh_{t+1}      (from the last token back; dhT enters at a
//                                             sequence's last token)
//     e_t  = dh_t a_t h_{t-1},  p_t = sum_n dh_t B_t,  o_t = sum_n C_t h_t + D x_t
//     dx = delta p + D g,  ddt = (sum_n e A + x p) softplus'(dt),  dz = dy o silu'(z)
//     dA += delta e,  dB_t = sum_c delta x dh_t,  dC_t = sum_c g h_t,  dh0 = a_0 dh_0
//
// A block walks its channels' tokens backwards in tiles of 16.  The forward pass kept the
// state entering every tile, so a tile's states are computed forward from it into
// registers (S x 16 of them) and then used from the last one back; a_t is an exponential
// each time, which costs less than registers for it would.
//
// Sums.  Over a channel's states (o, p, sum e A): the lanes' butterfly.  Over channels
// (dB, dC): a butterfly over the warp's channels that leaves a share of the 2 S values in
// each, the block's warps through shared memory, and the channel tiles by a second
// kernel from one partial result a tile.  Over tokens (dA, dD, ddt_bias): registers, then
// rows and segments by col_sum.  All in a fixed order, no atomics.
//
// Few rows: segments of the time axis, the entering dh composed from a first pass (SUM)
// over all but the first segment, as in the forward pass.
#include "scan.cuh"

namespace gdn {
namespace lay {

namespace {

constexpr int kTile = kScanKeep;
constexpr int kWarps = kScanThreads / 32;
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
struct BwdTile {
    static constexpr int EPT = kTile * Cfg::CH / kScanThreads;
    static constexpr int NBC = (kTile * Cfg::Np + kScanThreads - 1) / kScanThreads;
    static constexpr int RS = Cfg::CH + Cfg::CH / 8;
    struct Shared {
        float2 dd[kTile][Cfg::CH];                      // delta, delta x
        float g[kTile][RS], x[kTile][RS], s[kTile][RS], gz[kTile][RS];   // the last three: results dx, ddt, dz
        __align__(16) float b[kTile][Cfg::Np];
        __align__(16) float c[kTile][Cfg::Np];
        float bc[kTile][kWarps][2 * Cfg::Np];
        int seq[32];
        uint32_t edge[2];
    };
};

template <class T, class Cfg, int VEC, bool SUM>
__global__ void __launch_bounds__(kScanThreads) k_scan_bwd(ScanDims g, BwdIo<T> io)
{
    constexpr int L = Cfg::L, S = Cfg::S, Np = Cfg::Np, CH = Cfg::CH, M = 32 / L;
    using Tile = BwdTile<Cfg>;
    constexpr int NV = Tile::EPT / VEC, NBC = Tile::NBC;
    extern __shared__ __align__(16) char smem_raw[];
    typename Tile::Shared &sm = *reinterpret_cast<typename Tile::Shared *>(smem_raw);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = tid & (L - 1), ch = tid / L, n0 = l * S;
    int id = blockIdx.x;
    const int tiles = g.G * g.tiles, tile = id % tiles;
    id /= tiles;
    const int nseg = SUM ? g.K - 1 : g.K, k = id % nseg + (SUM ? 1 : 0), b = id / nseg;
    const int grp = tile / g.tiles, cg0 = (tile - grp * g.tiles) * CH;
    const bool live = cg0 + ch < g.Dg;
    const int c0 = grp * g.Dg + cg0;
    const long long c = live ? c0 + ch : c0;
    const int ts = k * g.seg, te = min(ts + g.seg, g.T);
    const bool gated = io.z.p != nullptr;

    float2 a2[S / 2], dh[S / 2], dA[S / 2], prod[S / 2];
    load_states<S>(a2, g.A + c * g.N, n0, g.N, live);
#pragma unroll
    for (int i = 0; i < S / 2; ++i) {
        a2[i] = mul2(a2[i], two(kLog2e));
        dh[i] = dA[i] = two(0.f);
        prod[i] = two(1.f);
    }
    const float Dc = !SUM && g.Dskip && live ? g.Dskip[c] : 0.f;
    float aD = 0.f, aBias = 0.f;
    if constexpr (!SUM) {
        // the segments behind this one, composed from the last
        for (int j = g.K - 1; j > k; --j) {
            const size_t at = (((size_t)b * g.K + j) * g.D + c) * Np + n0;
            float2 p[S / 2], e[S / 2];
            load_pairs<S>(p, io.segP + at);
            load_pairs<S>(e, io.segH + at);
#pragma unroll
            for (int i = 0; i < S / 2; ++i) {
                dh[i].x = p[i].x == 0.f ? e[i].x : fmaf(p[i].x, dh[i].x, e[i].x);
                dh[i].y = p[i].y == 0.f ? e[i].y : fmaf(p[i].y, dh[i].y, e[i].y);
            }
        }
    }

    Vec<T, VEC> xn[NV], dn[NV], zn[NV], gn[NV];
    T br[NBC], cr[NBC];
    constexpr int RV = CH / VEC;
    auto vt = [&](int e) { return (tid + e * kScanThreads) / RV; };
    auto vc = [&](int e) { return (tid + e * kScanThreads) % RV * VEC; };
    auto fetch = [&](int t0) {
#pragma unroll
        for (int e = 0; e < NV; ++e) {
            const int t = t0 + vt(e), q = vc(e);
            xn[e].zero();
            dn[e].zero();
            zn[e].zero();
            gn[e].zero();
            if (t >= ts && t < te && cg0 + q < g.Dg) {
                if (!SUM) xn[e].load(io.x.at(b, 0, t) + c0 + q);
                dn[e].load(io.dt.at(b, 0, t) + c0 + q);
                gn[e].load(io.dy.at(b, 0, t) + c0 + q);
                if (gated) zn[e].load(io.z.at(b, 0, t) + c0 + q);
            }
        }
#pragma unroll
        for (int e = 0; e < NBC; ++e) {
            const int i = tid + e * kScanThreads, t = t0 + i / Np, n = i % Np;
            st_out(&br[e], 0.f);
            st_out(&cr[e], 0.f);
            if (i < kTile * Np && t >= ts && t < te && n < g.N) {
                if (!SUM) br[e] = io.b.at(b, grp, t)[n];
                cr[e] = io.c.at(b, grp, t)[n];
            }
        }
    };
    const int last = ts + (te - ts - 1) / kTile * kTile;
    fetch(last);

    for (int t0 = last; t0 >= ts; t0 -= kTile) {
        // 1. the tile into shared memory
#pragma unroll
        for (int e = 0; e < NV; ++e) {
            float x[VEC], d[VEC], z[VEC], gy[VEC];
            xn[e].get(x);
            dn[e].get(d);
            zn[e].get(z);
            gn[e].get(gy);
            const int t = vt(e), q = vc(e);
            const bool in = t0 + t < te && cg0 + q < g.Dg;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float v = d[i] + (in && g.bias ? g.bias[c0 + q + i] : 0.f), der = 1.f;
                if (g.softplus) softplus(v, v, der);
                sm.dd[t][q + i] = in ? make_float2(v, v * x[i]) : make_float2(0.f, 0.f);
                float gate = 1.f;
                if (gated) {
                    const float sg = sigmoid(z[i]);
                    gate = z[i] * sg;
                    if (!SUM) sm.gz[t][q + i] = gy[i] * dsilu(z[i], sg);
                }
                sm.g[t][q + i] = gy[i] * gate;
                if (!SUM) {
                    sm.x[t][q + i] = x[i];
                    sm.s[t][q + i] = der;
                }
            }
        }
#pragma unroll
        for (int e = 0; e < NBC; ++e) {
            const int i = tid + e * kScanThreads;
            if (i < kTile * Np) {
                if (!SUM) sm.b[i / Np][i % Np] = ld_in(&br[e]);
                sm.c[i / Np][i % Np] = ld_in(&cr[e]);
            }
        }
        if (tid < 32) tile_edges(g, b, t0, min(kTile, te - t0), sm.seq, sm.edge);
        __syncthreads();
        fetch(t0 - kTile);
        const uint32_t starts = sm.edge[0], ends = sm.edge[1];

        if constexpr (SUM) {
#pragma unroll
            for (int t = kTile - 1; t >= 0; --t) {
                const float dl = sm.dd[t][ch].x, gg = sm.g[t][ch];
                float2 cc[S / 2];
                load_pairs<S>(cc, &sm.c[t][n0]);
                if ((ends >> t & 1) && io.dhT) {
                    float2 v[S / 2];
                    load_states<S>(v, io.dhT + ((size_t)sm.seq[t] * g.D + c) * g.N, n0, g.N, live);
#pragma unroll
                    for (int i = 0; i < S / 2; ++i) dh[i].x += v[i].x, dh[i].y += v[i].y;
                }
#pragma unroll
                for (int i = 0; i < S / 2; ++i) {
                    const float2 a = ex2_2(mul2(two(dl), a2[i]));
                    dh[i] = mul2(a, fma2(two(gg), cc[i], dh[i]));
                    prod[i] = mul2(prod[i], a);
                }
                if (starts >> t & 1) {
#pragma unroll
                    for (int i = 0; i < S / 2; ++i) dh[i] = prod[i] = two(0.f);
                }
            }
            __syncthreads();
        } else {
            // 2. the tile's states, forward from the kept one: hist[t] enters token t
            float2 hist[kTile][S / 2], h[S / 2];
#pragma unroll
            for (int i = 0; i < S / 2; ++i) h[i] = two(0.f);
            if (live)
                load_pairs<S>(h, io.keep + (((size_t)b * ((g.T + kScanKeep - 1) / kScanKeep) + t0 / kScanKeep) * g.D + c) * Np + n0);
#pragma unroll
            for (int t = 0; t < kTile; ++t) {
                const float2 q = sm.dd[t][ch];
                float2 bb[S / 2];
                load_pairs<S>(bb, &sm.b[t][n0]);
                if (starts >> t & 1)
                    load_states<S>(h, g.h0 + ((size_t)sm.seq[t] * g.D + c) * g.N, n0, g.N, live && g.h0);
#pragma unroll
                for (int i = 0; i < S / 2; ++i) {
                    hist[t][i] = h[i];
                    h[i] = fma2(ex2_2(mul2(two(q.x), a2[i])), h[i], mul2(two(q.y), bb[i]));
                }
            }
            // 3. back through the tile
#pragma unroll
            for (int g0 = kTile - L; g0 >= 0; g0 -= L) {
                float po[L], pp[L], pe[L];
#pragma unroll
                for (int j = L - 1; j >= 0; --j) {
                    const int t = g0 + j;
                    const float2 q = sm.dd[t][ch];
                    const float gg = sm.g[t][ch];
                    float2 bb[S / 2], cc[S / 2];
                    load_pairs<S>(bb, &sm.b[t][n0]);
                    load_pairs<S>(cc, &sm.c[t][n0]);
                    if ((ends >> t & 1) && io.dhT) {
                        float2 v[S / 2];
                        load_states<S>(v, io.dhT + ((size_t)sm.seq[t] * g.D + c) * g.N, n0, g.N, live);
#pragma unroll
                        for (int i = 0; i < S / 2; ++i) dh[i].x += v[i].x, dh[i].y += v[i].y;
                    }
                    float2 o = two(0.f), p = two(0.f), e2 = two(0.f);
                    float v[2 * S];
#pragma unroll
                    for (int i = 0; i < S / 2; ++i) {
                        const float2 a = ex2_2(mul2(two(q.x), a2[i])), ah = mul2(a, hist[t][i]);
                        const float2 hn = fma2(two(q.y), bb[i], ah);
                        o = fma2(cc[i], hn, o);
                        dh[i] = fma2(two(gg), cc[i], dh[i]);
                        const float2 e = mul2(dh[i], ah);
                        p = fma2(dh[i], bb[i], p);
                        e2 = fma2(e, a2[i], e2);
                        dA[i] = fma2(two(q.x), e, dA[i]);
                        const float2 vb = mul2(two(q.y), dh[i]), vcc = mul2(two(gg), hn);
                        v[2 * i] = vb.x;
                        v[2 * i + 1] = vb.y;
                        v[S + 2 * i] = vcc.x;
                        v[S + 2 * i + 1] = vcc.y;
                        dh[i] = mul2(a, dh[i]);
                    }
                    po[j] = o.x + o.y;
                    pp[j] = p.x + p.y;
                    pe[j] = e2.x + e2.y;
                    if (starts >> t & 1) {
                        if (io.dh0) store_states<S>(io.dh0 + ((size_t)sm.seq[t] * g.D + c) * g.N, dh, n0, g.N, live);
#pragma unroll
                        for (int i = 0; i < S / 2; ++i) dh[i] = two(0.f);
                    }
                    // dB, dC over the warp's channels
                    constexpr int left = 2 * S > M ? 2 * S / M : 1;   // values a lane ends with
                    int off = 0;
                    int cur = 2 * S;
#pragma unroll
                    for (int bit = M / 2; bit > 0; bit >>= 1) {
                        const bool up = lane & (bit * L);
                        if (cur > 1) {
                            cur >>= 1;
#pragma unroll
                            for (int i = 0; i < cur; ++i) {
                                const float send = up ? v[i] : v[i + cur], mine = up ? v[i + cur] : v[i];
                                v[i] = mine + __shfl_xor_sync(0xffffffffu, send, bit * L);
                            }
                            off += up ? cur : 0;
                        } else {
                            v[0] += __shfl_xor_sync(0xffffffffu, v[0], bit * L);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < left; ++i) {
                        const int w = off + i;
                        sm.bc[t][warp][(w >= S ? Np : 0) + n0 + (w & (S - 1))] = v[i];
                    }
                }
                const float o = lane_sum<L>(po, lane), p = lane_sum<L>(pp, lane), e = lane_sum<L>(pe, lane) * kLn2;
                const int t = g0 + l;
                const float x = sm.x[t][ch], gg = sm.g[t][ch];
                const float ddt = fmaf(p, x, e) * sm.s[t][ch];
                aD = fmaf(gg, x, aD);
                aBias += ddt;
                sm.x[t][ch] = fmaf(sm.dd[t][ch].x, p, Dc * gg);
                sm.s[t][ch] = ddt;
                if (gated) sm.gz[t][ch] *= fmaf(Dc, x, o);
            }
            __syncthreads();

            // 4. the tile's results
#pragma unroll
            for (int e = 0; e < NV; ++e) {
                const int t = vt(e), q = vc(e);
                if (t0 + t < te && cg0 + q < g.Dg) {
                    Vec<T, VEC> out;
                    float f[VEC];
#pragma unroll
                    for (int i = 0; i < VEC; ++i) f[i] = sm.x[t][q + i];
                    out.set(f);
                    out.store(io.dx.at(b, 0, t0 + t) + c0 + q);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) f[i] = sm.s[t][q + i];
                    out.set(f);
                    out.store(io.ddt.at(b, 0, t0 + t) + c0 + q);
                    if (gated) {
#pragma unroll
                        for (int i = 0; i < VEC; ++i) f[i] = sm.gz[t][q + i];
                        out.set(f);
                        out.store(io.dz.at(b, 0, t0 + t) + c0 + q);
                    }
                }
            }
            float *pb = io.part_bc + (((size_t)b * tiles + tile) * g.T + t0) * (2 * Np);
            const int n = min(kTile, te - t0) * 2 * Np;
            for (int i = tid; i < n; i += kScanThreads) {
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) s += sm.bc[i / (2 * Np)][w][i % (2 * Np)];
                pb[i] = s;
            }
            __syncthreads();
        }
    }
    if constexpr (SUM) {
        if (live) {
            const size_t at = (((size_t)b * g.K + k) * g.D + c) * Np + n0;
            store_pairs<S>(io.segP + at, prod);
            store_pairs<S>(io.segH + at, dh);
        }
    } else {
        const size_t row = (size_t)b * g.K + k;
        store_states<S>(io.part_a + (row * g.D + c) * g.N, dA, n0, g.N, live);
#pragma unroll
        for (int o = L >> 1; o > 0; o >>= 1) {
            aD += __shfl_xor_sync(0xffffffffu, aD, o);
            aBias += __shfl_xor_sync(0xffffffffu, aBias, o);
        }
        if (live && l == 0) {
            io.part_d[row * 2 * g.D + c] = aD;
            io.part_d[(row * 2 + 1) * g.D + c] = aBias;
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
    scan_layout(s->N, [&](auto cfg) { CH = decltype(cfg)::CH; return cudaSuccess; });
    const int Dg = s->D / s->G, Np = scan_padded(s->N);
    p.tiles = (Dg + CH - 1) / CH;
    const long long blocks = (long long)s->B * s->G * p.tiles, want = 2 * sm_count();
    long long k = blocks >= want / 2 ? 1 : want / blocks;
    const long long most = (s->T + 127) / 128;
    if (k > most) k = most;
    if (k > 64) k = 64;
    if (k < 1) k = 1;
    p.seg = (int)((((long long)s->T + k - 1) / k + kTile - 1) / kTile * kTile);
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
    const size_t smem = sizeof(typename BwdTile<Cfg>::Shared);
    cudaError_t e;
    if (g.K > 1) {
        e = cudaFuncSetAttribute(k_scan_bwd<T, Cfg, VEC, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        k_scan_bwd<T, Cfg, VEC, true><<<(unsigned)(per * (g.K - 1)), kScanThreads, smem, st>>>(g, io);
    }
    e = cudaFuncSetAttribute(k_scan_bwd<T, Cfg, VEC, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    k_scan_bwd<T, Cfg, VEC, false><<<(unsigned)(per * g.K), kScanThreads, smem, st>>>(g, io);
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
        const cudaError_t e = scan_layout(s->N, [&](auto cfg) {
            using Cfg = decltype(cfg);
            constexpr int VEC = BwdTile<Cfg>::EPT < 4 ? BwdTile<Cfg>::EPT : 4;
            const dn_view *all[] = {&io->x, &io->dt, &io->z, &gr->dy, &gr->dx, &gr->ddt, &gr->dz};
            bool v = (s->D / s->G) % VEC == 0;
            for (const dn_view *q : all) v = v && can_vector(q, sizeof(T), VEC * sizeof(T));
            if constexpr (VEC > 1) {
                if (v) return launch<T, Cfg, VEC>(c, st);
            }
            return launch<T, Cfg, 1>(c, st);
        });
        if (e != cudaSuccess) return e;
    }
    const long long rows = s->T > 0 ? (long long)s->B * p.K : 0;
    ColSum r;
    r.kinds = 1;
    r.C = (long long)s->D * s->N;
    r.dst[0] = gr->dA;
    r.step[0] = 1;
    cudaError_t e = col_sum((float *)(c.ws + p.part_a), rows, r, st);
    if (e != cudaSuccess || (!gr->dD && !gr->ddt_bias)) return e;
    r.kinds = 2;
    r.C = s->D;
    r.dst[0] = gr->dD;
    r.dst[1] = gr->ddt_bias;
    r.step[1] = 1;
    return col_sum((float *)(c.ws + p.part_d), rows, r, st);
}

}  // namespace

size_t scan_bwd_bytes(const dn_scan_shape *s) { return plan_of(s).total; }

cudaError_t scan_bwd(const ScanCall &c, cudaStream_t st)
{
    return c.s->dtype == DN_F32 ? bwd_t<float>(c, st) : bwd_t<__nv_bfloat16>(c, st);
}

}  // namespace lay
}  // namespace gdn

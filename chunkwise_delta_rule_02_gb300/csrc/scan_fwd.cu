// Selective state space scan: forward over tokens, and the single-token step.
//
// k_scan_fwd.  A block owns CH channels of one group and walks a row's tokens (or one
// time segment of them) in tiles of 16:
//   1. every thread turns its part of the tile's x and dt into (delta, delta x), and
//      its part of B, C into float32, in shared memory;
//   2. the recurrence: per token a lane reads (delta, delta x) of its channels and S
//      values of B and C, and does S exponentials and 4 S multiply-adds for each channel;
//   3. y = (sum + D x) silu(z), stored with the tile's layout of x.
// The loads of the next tile are in flight during step 2, in registers (asynchronous copies
// to shared memory, with the 3 blocks an SM that the registers saved allow, were 5 % slower).
//
// Bound by instruction issue, not by HBM: per (token, channel) N exponentials at 32 lanes a
// cycle and SM and 4 N multiply-adds at 128 are N / 16 cycles, 0.12 ms for 67 M (token,
// channel) of 16 states; with the reads of B and C, the sums over lanes and the elementwise
// steps 1 and 3 it issues twice that.  Few rows: the time axis is cut into K segments.  A
// first pass (SUM) runs all but the last segment from a zero state and keeps its end state and
// its decay product, k_scan_carry composes them, and the second pass starts every segment from
// what enters it.  That costs the recurrence 1.6 times, so plan_segments weighs it against the
// SMs left idle.  4 x 8192 tokens of 2048 channels, 16 states, bf16 with gate: 553 us
// (197 us the first pass, 347 us the second); one row of 16384 tokens, 1024 channels: 160 us.
#include <algorithm>
#include <type_traits>

#include "scan.cuh"

namespace gdn {
namespace lay {

namespace {

template <class T, class Cfg, int VEC, bool SUM>
__global__ void __launch_bounds__(Cfg::NT) k_scan_fwd(ScanDims g, ScanIo<T> io)
{
    constexpr int L = Cfg::L, S = Cfg::S, CT = Cfg::CT, M = Cfg::M, Np = Cfg::Np, CH = Cfg::CH, P = S / 2;
    constexpr int TT = Cfg::TT, NV = Cfg::EPT / VEC, NBC = Cfg::NBC;
    __shared__ __align__(16) float2 dd[TT][CH];   // delta, delta x
    __shared__ __align__(16) float sb[TT][Np], sc[SUM ? 1 : TT][Np];
    __shared__ __align__(16) float sy[SUM ? 1 : TT][Cfg::RS];
    __shared__ int seq[32];
    __shared__ uint32_t edge[2];

    const int tid = threadIdx.x, lane = tid & 31, l = lane / M, n0 = l * S;
    const int ch = ((tid >> 5) * M + lane % M) * CT;   // first of this lane's channels in the block
    // block -> (channel tile, segment, row)
    int id = blockIdx.x;
    const int tile = id % (g.G * g.tiles);
    id /= g.G * g.tiles;
    const int nseg = SUM ? g.K - 1 : g.K, k = id % nseg, b = id / nseg;
    const int grp = tile / g.tiles, cg0 = (tile - grp * g.tiles) * CH;   // first channel within the group
    const int c0 = grp * g.Dg + cg0;
    const long long c = c0 + ch;
    bool live[CT];
#pragma unroll
    for (int e = 0; e < CT; ++e) live[e] = cg0 + ch + e < g.Dg;
    const int ts = k * g.seg, te = min(ts + g.seg, g.T);
    float total[CT];   // SUM: of delta since the last sequence start

    float2 a2[CT][P], h[CT][P], open[CT];   // open: 1, 0 after a sequence start
#pragma unroll
    for (int e = 0; e < CT; ++e) {
        load_states<S>(a2[e], g.A + (c + e) * g.N, n0, g.N, live[e]);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            a2[e][i] = mul2(a2[e][i], two(kLog2e));
            h[e][i] = two(0.f);
        }
        open[e] = two(1.f);
        total[e] = 0.f;
        if constexpr (!SUM) {
            if (k > 0 && live[e]) load_pairs<S>(h[e], io.segH + (((size_t)b * g.K + k) * g.D + c + e) * Np + n0);
        }
    }

    // where this lane's kept states go
    [[maybe_unused]] constexpr int KEEP = keep_of(Np);
    float *kp = nullptr;
    unsigned place[CT];
    if constexpr (!SUM) {
        if (io.keep) kp = io.keep + ((size_t)b * ((g.T + KEEP - 1) / KEEP) + ts / KEEP) * g.D * Np;
#pragma unroll
        for (int e = 0; e < CT; ++e) place[e] = keep_place<Cfg>(g, grp, cg0 + ch + e, l);
    }

    // This thread's vectors of a tile: tokens vt, vt + ES, ..., always channels vc .. vc + VEC - 1
    // (a token's vectors divide the threads).
    constexpr int RV = CH / VEC, ES = Cfg::NT / RV;
    const int vt = tid / RV, vc = tid % RV * VEC;
    const bool col = cg0 + vc < g.Dg, gated = !SUM && io.z.p != nullptr;
    const int cv = c0 + (col ? vc : 0);
    Vec<T, VEC> xr[NV], zr[NV], xn[NV], dn[NV], zn[NV];
    T br[NBC], cr[NBC];
    const T *px = io.x.at(b, 0, ts + vt) + cv, *pd = io.dt.at(b, 0, ts + vt) + cv;
    const T *pz = gated ? io.z.at(b, 0, ts + vt) + cv : nullptr;
    T *py = SUM ? nullptr : io.y.at(b, 0, ts + vt) + cv;
    float bias[VEC], skip[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        bias[i] = col && g.bias ? g.bias[cv + i] : 0.f;
        skip[i] = !SUM && col && g.Dskip ? g.Dskip[cv + i] : 0.f;
    }
    // this thread's elements of B and C: state bn of tokens bt, bt + BS, ...
    constexpr int BS = Cfg::NT / Np;
    const int bt = tid / Np, bn = tid % Np;
    const bool bc_in = bn < g.N && (NBC * Cfg::NT == TT * Np || tid < TT * Np);
    const T *pb = io.b.at(b, grp, ts + bt) + bn, *pc = SUM ? nullptr : io.c.at(b, grp, ts + bt) + bn;
    const bool whole = cg0 + CH <= g.Dg;   // no channel of the block is behind its group's end
    // whole tiles (the same for every thread) take the loads without their checks
    auto fetch = [&](int t0) {
        if (whole && t0 + TT <= te) {
#pragma unroll
            for (int e = 0; e < NV; ++e) {
                xn[e].load(px + e * ES * io.x.t);
                dn[e].load(pd + e * ES * io.dt.t);
                if (gated) zn[e].load(pz + e * ES * io.z.t);
            }
#pragma unroll
            for (int e = 0; e < NBC; ++e) {
                if (bc_in) {
                    br[e] = pb[e * BS * io.b.t];
                    if (!SUM) cr[e] = pc[e * BS * io.c.t];
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < NV; ++e) {
                xn[e].zero();
                dn[e].zero();
                if (!SUM) zn[e].zero();
                if (col && t0 + vt + e * ES < te) {
                    xn[e].load(px + e * ES * io.x.t);
                    dn[e].load(pd + e * ES * io.dt.t);
                    if (gated) zn[e].load(pz + e * ES * io.z.t);
                }
            }
#pragma unroll
            for (int e = 0; e < NBC; ++e) {
                st_out(&br[e], 0.f);
                st_out(&cr[e], 0.f);
                if (bc_in && t0 + bt + e * BS < te) {
                    br[e] = pb[e * BS * io.b.t];
                    if (!SUM) cr[e] = pc[e * BS * io.c.t];
                }
            }
        }
        px += TT * io.x.t;
        pd += TT * io.dt.t;
        if (gated) pz += TT * io.z.t;
        pb += TT * io.b.t;
        if (!SUM) pc += TT * io.c.t;
    };
#pragma unroll
    for (int e = 0; e < NBC; ++e) {   // padded states stay zero
        st_out(&br[e], 0.f);
        st_out(&cr[e], 0.f);
    }
    fetch(ts);

    for (int t0 = ts; t0 < te; t0 += TT) {
        const bool full = whole && t0 + TT <= te;
        // 1. the tile into shared memory
#pragma unroll
        for (int e = 0; e < NV; ++e) {
            float x[VEC], d[VEC];
            xr[e] = xn[e];
            if (!SUM) zr[e] = zn[e];
            xn[e].get(x);
            dn[e].get(d);
            // tokens behind the end (and channels behind the group's) change nothing: delta = 0
            const bool in = full || (col && t0 + vt + e * ES < te);
#pragma unroll
            for (int i = 0; i < VEC; i += 2) {
                float2 v = add2(pair_at(d, i), pair_at(bias, i)), der;
                if (g.softplus) softplus(v, v, der);
                float2 w = mul2(v, pair_at(x, i));
                if (!in) v = w = two(0.f);
                if constexpr (VEC > 1) *reinterpret_cast<float4 *>(&dd[vt + e * ES][vc + i]) = make_float4(v.x, w.x, v.y, w.y);
                else dd[vt + e * ES][vc] = make_float2(v.x, w.x);
            }
        }
#pragma unroll
        for (int e = 0; e < NBC; ++e) {
            if (NBC * Cfg::NT == TT * Np || tid < TT * Np) {
                sb[bt + e * BS][bn] = ld_in(&br[e]);
                if constexpr (!SUM) sc[bt + e * BS][bn] = ld_in(&cr[e]);
            }
        }
        if (tid < 32) tile_edges(g, b, t0, min(TT, te - t0), seq, edge);
        __syncthreads();
        fetch(t0 + TT);

        // 2. the recurrence
        const uint32_t starts = edge[0], ends = edge[1];
        // Tiles without a sequence start or end, nearly all, run a copy of the loop without what happens there.
        auto run = [&](auto edges) {
            constexpr bool EDGES = decltype(edges)::value;
#pragma unroll 1
            for (int g0 = 0; g0 < TT; g0 += L) {
                if constexpr (!SUM) {
                    if (kp && g0 % KEEP == 0 && t0 + g0 < te) {
#pragma unroll
                        for (int e = 0; e < CT; ++e)
                            if (live[e]) store_pairs<S>(kp + place[e], h[e]);
                        kp += (size_t)g.D * Np;
                    }
                }
                float yp[CT][L];
#pragma unroll
                for (int j = 0; j < L; ++j) {
                    const int t = g0 + j;
                    float dl[CT], dx[CT];
                    load_steps<CT>(dl, dx, &dd[t][ch]);
                    float2 bb[P];
                    [[maybe_unused]] float2 cc[P];
                    load_pairs<S>(bb, &sb[t][n0]);
                    if constexpr (!SUM) load_pairs<S>(cc, &sc[t][n0]);
#pragma unroll
                    for (int e = 0; e < CT; ++e) {
                        if constexpr (EDGES) {
                            if (starts >> t & 1) {
                                load_states<S>(h[e], g.h0 + ((size_t)seq[t] * g.D + c + e) * g.N, n0, g.N, live[e] && g.h0);
                                open[e] = two(0.f);
                                total[e] = 0.f;
                            }
                        }
                        if constexpr (SUM) total[e] += dl[e];
                        float2 yy = two(0.f);
#pragma unroll
                        for (int i = 0; i < P; ++i) {
                            const float2 a = decay2(dl[e], a2[e][i]);
                            h[e][i] = fma2(a, h[e][i], mul2(two(dx[e]), bb[i]));
                            if constexpr (!SUM) yy = i == 0 ? mul2(cc[i], h[e][i]) : fma2(cc[i], h[e][i], yy);
                        }
                        yp[e][j] = yy.x + yy.y;
                        if constexpr (!SUM && EDGES) {
                            if ((ends >> t & 1) && io.hT)
                                store_states<S>(io.hT + ((size_t)seq[t] * g.D + c + e) * g.N, h[e], n0, g.N, live[e]);
                        }
                    }
                }
                if constexpr (!SUM) {
                    float y[CT];
#pragma unroll
                    for (int e = 0; e < CT; ++e) y[e] = lane_sum<L>(yp[e], lane);
                    store_ct<CT>(&sy[g0 + l][ch], y);
                }
            }
        };
        if ((starts | ends) == 0) run(std::false_type());
        else run(std::true_type());
        __syncthreads();

        // 3. the results
        if constexpr (!SUM) {
#pragma unroll
            for (int e = 0; e < NV; ++e) {
                if (full || (col && t0 + vt + e * ES < te)) {
                    float x[VEC], z[VEC], o[VEC];
                    xr[e].get(x);
                    zr[e].get(z);
                    Vec<float, VEC> s4;
                    s4.load(&sy[vt + e * ES][vc]);
                    s4.get(o);
#pragma unroll
                    for (int i = 0; i < VEC; i += 2) {
                        float2 v = fma2(pair_at(skip, i), pair_at(x, i), pair_at(o, i));
                        if (gated) {
                            const float2 w = pair_at(z, i);
                            v = mul2(v, mul2(w, sigmoid2(w)));
                        }
                        put_pair(o, i, v);
                    }
                    Vec<T, VEC> out;
                    out.set(o);
                    out.store(py + e * ES * io.y.t);
                }
            }
            py += TT * io.y.t;
        }
    }
    if constexpr (SUM) {
#pragma unroll
        for (int e = 0; e < CT; ++e) {
            if (!live[e]) continue;
            const size_t at = (((size_t)b * g.K + k) * g.D + c + e) * Np + n0;
            // the product of the decays is one exponential of the steps' sum
            float2 p[P];
#pragma unroll
            for (int i = 0; i < P; ++i) p[i] = open[e].x == 0.f ? two(kCut) : ex2_2(mul2(two(total[e]), a2[e][i]));
            store_pairs<S>(io.segP + at, p);
            store_pairs<S>(io.segH + at, h[e]);
        }
    }
}

// Final states of empty sequences: their initial ones.
__global__ void k_scan_empty(const float *h0, float *hT, const int32_t *cu, int Nseq, long long per)
{
    const int s = blockIdx.y;
    if (cu && cu[s + 1] > cu[s]) return;
    const long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x;
    if (i < per) hT[s * per + i] = h0 ? h0[s * per + i] : 0.f;
}

// One token a sequence.  Lanes of a channel take V states at a time (16 bytes where N and the
// states' alignment allow), so that a warp moves whole rows of the states, which are what this is
// bound by (HBM: states read and written once), and U sequences each, whose states are in flight
// together and share A.
template <class T, int V, int U>
__global__ void __launch_bounds__(256, 4) k_scan_step(ScanDims g, ScanIo<T> io, int shift, bool wide, int first)
{
    // L = 2^shift lanes a channel; sequences from `first` on, so few that 32 bits count their channels
    const int L = 1 << shift, l = threadIdx.x & (L - 1);
    const unsigned i = blockIdx.x * (256u >> shift) + (threadIdx.x >> shift), q = i / (unsigned)g.D;
    const bool any = q * U + first < (unsigned)g.B;   // the whole warp takes part in the sums
    const int b0 = any ? (int)q * U + first : 0, c = any ? (int)(i - q * g.D) : 0, grp = g.G == 1 ? 0 : c / g.Dg;
    bool live[U];
    int b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        live[u] = any && b0 + u < g.B;
        b[u] = live[u] ? b0 + u : 0;
    }
    // the states' loads go out first: the step's arithmetic then runs under their latency
    Vec<float, V> hv[U], av;
    Vec<T, V> bv[U], cv[U];
    auto load = [&](int n) {
        av.load(g.A + (size_t)c * g.N + n);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            hv[u].zero();
            if (g.h0 && live[u]) hv[u].load(g.h0 + ((size_t)b[u] * g.D + c) * g.N + n);
            const T *pb = io.b.at(b[u], grp, 0) + n, *pc = io.c.at(b[u], grp, 0) + n;
            if (wide) {
                bv[u].load(pb);
                cv[u].load(pc);
            } else {
                T eb[V], ec[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    eb[e] = pb[e];
                    ec[e] = pc[e];
                }
                memcpy(&bv[u].raw, eb, sizeof(eb));
                memcpy(&cv[u].raw, ec, sizeof(ec));
            }
        }
    };
    int n = l * V;
    if (n < g.N) load(n);
    const float skip = g.Dskip ? g.Dskip[c] : 0.f, bias = g.bias ? g.bias[c] : 0.f;
    float x[U], d[U], z[U], y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        x[u] = ld_in(io.x.at(b[u], 0, 0) + c);
        d[u] = ld_in(io.dt.at(b[u], 0, 0) + c) + bias;
        z[u] = io.z.p ? ld_in(io.z.at(b[u], 0, 0) + c) : 0.f;
        y[u] = 0.f;
    }
    if (g.softplus) {
#pragma unroll
        for (int u = 0; u < U; u += 2) {
            float2 v, der;
            softplus(make_float2(d[u], d[U > 1 ? u + 1 : u]), v, der);
            d[u] = v.x;
            if (U > 1) d[U > 1 ? u + 1 : u] = v.y;
        }
    }
    while (n < g.N) {
        float a[V];
        av.get(a);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float h[V], bf[V], cf[V];
            hv[u].get(h);
            bv[u].get(bf);
            cv[u].get(cf);
            const float dx = d[u] * x[u];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                h[e] = fmaf(ex2(fmaf(d[u], a[e] * kLog2e, kDecayUp)), h[e], dx * bf[e]);
                y[u] = fmaf(cf[e], h[e], y[u]);
            }
            if (io.hT && live[u]) {
                hv[u].set(h);
                hv[u].store(io.hT + ((size_t)b[u] * g.D + c) * g.N + n);
            }
        }
        n += L * V;
        if (n < g.N) load(n);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        for (int o = L >> 1; o > 0; o >>= 1) y[u] += __shfl_xor_sync(0xffffffffu, y[u], o);
    // the results, a sequence a lane
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (live[u] && l == u % L) {
            float o = fmaf(skip, x[u], y[u]);
            if (io.z.p) o *= z[u] * sigmoid(z[u]);
            st_out(io.y.at(b0 + u, 0, 0) + c, o);
        }
    }
}

// Blocks of a segment.
long long tiles_of(const dn_scan_shape *s, int CH)
{
    const int Dg = s->D / s->G;
    return (long long)s->B * s->G * ((Dg + CH - 1) / CH);
}

// four blocks of the main pass fit an SM, six of the first, which does 0.6 of the work
int segments(const dn_scan_shape *s, int CH) { return plan_segments(tiles_of(s, CH), s->T, 4, 6, 0.6); }

int channels_of(int N)
{
    int ch = 0;
    fwd_layout(N, [&](auto cfg) { ch = decltype(cfg)::CH; return cudaSuccess; });
    return ch;
}

template <class T>
ScanIo<T> io_of(const ScanCall &c)
{
    ScanIo<T> io;
    io.x = view_of<const T>(&c.io->x); io.dt = view_of<const T>(&c.io->dt);
    io.b = view_of<const T>(&c.io->b); io.c = view_of<const T>(&c.io->c);
    io.z = view_of<const T>(&c.io->z); io.y = view_of<T>(&c.io->y);
    io.hT = c.io->hT; io.keep = c.keep;
    io.segP = io.segH = nullptr;
    return io;
}

// One segment, in a layout for few blocks.
template <class T, class Cfg, int VEC>
cudaError_t launch_few(const ScanCall &c, cudaStream_t st)
{
    ScanDims g = scan_dims(c);
    g.tiles = (g.Dg + Cfg::CH - 1) / Cfg::CH;
    g.K = 1;
    g.seg = (g.T + 15) / 16 * 16;
    const long long per = (long long)g.B * g.G * g.tiles;
    if (per > 0x7fffffffLL) return cudaErrorInvalidValue;
    k_scan_fwd<T, Cfg, VEC, false><<<(unsigned)per, Cfg::NT, 0, st>>>(g, io_of<T>(c));
    return cudaPeekAtLastError();
}

template <class T, class Cfg, int VEC>
cudaError_t launch(const ScanCall &c, cudaStream_t st)
{
    ScanDims g = scan_dims(c);
    g.tiles = (g.Dg + Cfg::CH - 1) / Cfg::CH;
    g.K = segments(c.s, Cfg::CH);
    // One segment, at most two blocks an SM of the four that fit, up to 16 states: what counts is
    // latency.  Up to 8 states, one channel a lane in twice the blocks hides more of it than two channels'
    // shared reads of B and C save (2048 channels of 8 states, 8 x 4096 tokens: 460 us against 612;
    // of 16 states 545 against 537).  With 9 to 16 states, tiles of 32 tokens halve the barriers and the
    // elementwise steps' waits (8 x 4096: 499 us against 536; where four blocks run on an SM, 4 x 8192, 563
    // against 554; 32 states, 4 x 4096, 455 against 450).
    if constexpr (Cfg::CT == 2 && Cfg::Np <= 16) {
        if (g.K == 1 && tiles_of(c.s, Cfg::CH) <= 2ll * sm_count()) {
            using Few = ScanCfg<Cfg::L, Cfg::S, Cfg::Np <= 8 ? 1 : 2, Cfg::Np <= 8 ? Cfg::TT : 32, Cfg::NT>;
            return launch_few<T, Few, (VEC < Few::VEC ? VEC : Few::VEC)>(c, st);
        }
    }
    g.seg = ((g.T + g.K - 1) / g.K + 15) / 16 * 16;   // whole tiles, whole spans between kept states
    g.K = (g.T + g.seg - 1) / g.seg;
    ScanIo<T> io = io_of<T>(c);
    const long long per = (long long)g.B * g.G * g.tiles;
    if (per * g.K > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (g.K > 1) {
        io.segP = (float *)c.ws;
        io.segH = io.segP + (size_t)g.B * g.K * g.D * Cfg::Np;
        k_scan_fwd<T, Cfg, VEC, true><<<(unsigned)(per * (g.K - 1)), Cfg::NT, 0, st>>>(g, io);
        scan_carry<true>(g, io.segP, io.segH, Cfg::Np, st);
    }
    k_scan_fwd<T, Cfg, VEC, false><<<(unsigned)(per * g.K), Cfg::NT, 0, st>>>(g, io);
    return cudaPeekAtLastError();
}

template <class T>
cudaError_t fwd_t(const ScanCall &c, cudaStream_t st)
{
    const dn_scan_shape *s = c.s;
    const dn_scan_io *io = c.io;
    if (io->hT && c.Nseq > 0 && (c.cu || s->T == 0)) {
        const long long per = (long long)s->D * s->N;
        for (int s0 = 0; s0 < c.Nseq; s0 += 65535) {   // grid.y
            const int n = c.Nseq - s0 < 65535 ? c.Nseq - s0 : 65535;
            k_scan_empty<<<dim3((unsigned)((per + 255) / 256), n), 256, 0, st>>>(io->h0 ? io->h0 + s0 * per : nullptr, io->hT + s0 * per,
                                                                                c.cu ? c.cu + s0 : nullptr, n, per);
        }
    }
    if (s->T == 0) return cudaPeekAtLastError();
    return fwd_layout(s->N, [&](auto cfg) {
        using Cfg = decltype(cfg);
        constexpr int VEC = Cfg::VEC;
        const int bytes = VEC * sizeof(T);
        const bool v = (s->D / s->G) % VEC == 0 && can_vector(&io->x, sizeof(T), bytes) && can_vector(&io->dt, sizeof(T), bytes) &&
                       can_vector(&io->z, sizeof(T), bytes) && can_vector(&io->y, sizeof(T), bytes);
        if constexpr (VEC > 1) {
            if (v) return launch<T, Cfg, VEC>(c, st);
        }
        return launch<T, Cfg, 1>(c, st);
    });
}

template <class T>
cudaError_t step_t(const ScanCall &c, cudaStream_t st)
{
    const ScanDims g = scan_dims(c);
    const ScanIo<T> io = io_of<T>(c);
    auto al = [](const void *p, int n) { return ((uintptr_t)p % n) == 0; };
    auto ok = [&](int V) { return g.N % V == 0 && al(g.A, 4 * V) && al(g.h0, 4 * V) && al(io.hT, 4 * V); };
    const int V = ok(4) ? 4 : 1;
    int shift = 0;
    while (shift < 5 && (V << shift) < g.N) ++shift;
    // two sequences a lane once that leaves the SMs four blocks each (256 sequences, 2048 channels, 16
    // states: 33 us with one, 23 us with two and with four).  The kernel's 64 registers let four blocks run on an
    // SM: 21.5 us, at 70 registers 24 us
    const int U = ((long long)g.B * g.D << shift) / 2 / 256 >= 4ll * sm_count() ? 2 : 1;
    const bool wide = can_vector(&c.io->b, sizeof(T), V * sizeof(T)) && can_vector(&c.io->c, sizeof(T), V * sizeof(T));
    const int most = (int)std::max(1ll, std::min<long long>(g.B, (1ll << 29) / g.D)) * U;   // sequences of a launch
    auto go = [&](auto v, auto u) {
        for (long long first = 0; first < g.B; first += most) {
            const int n = (int)std::min<long long>(g.B - first, most);
            const unsigned blocks = (unsigned)(((((long long)(n + U - 1) / U) * g.D << shift) + 255) / 256);
            ScanDims part = g;
            part.B = (int)first + n;
            k_scan_step<T, decltype(v)::value, decltype(u)::value><<<blocks, 256, 0, st>>>(part, io, shift, wide, (int)first);
        }
    };
    using one = std::integral_constant<int, 1>;
    using two_ = std::integral_constant<int, 2>;
    using four = std::integral_constant<int, 4>;
    if (V == 4) U == 2 ? go(four(), two_()) : go(four(), one());
    else U == 2 ? go(one(), two_()) : go(one(), one());
    return cudaPeekAtLastError();
}

}  // namespace

int scan_padded(int N)
{
    int np = 0;
    fwd_layout(N, [&](auto cfg) { np = decltype(cfg)::Np; return cudaSuccess; });
    return np;
}

ScanDims scan_dims(const ScanCall &c)
{
    ScanDims g;
    g.B = c.s->B; g.T = c.s->T; g.D = c.s->D; g.N = c.s->N; g.G = c.s->G; g.Dg = g.D / g.G;
    g.tiles = 0; g.softplus = c.s->dt_softplus; g.K = 1; g.seg = 0;
    g.Nseq = c.Nseq; g.cu = c.cu;
    g.A = c.io->A; g.Dskip = c.io->D; g.bias = c.io->dt_bias; g.h0 = c.io->h0;
    return g;
}

size_t scan_fwd_bytes(const dn_scan_shape *s)
{
    const int K = segments(s, channels_of(s->N));
    return K > 1 ? align256(2 * sizeof(float) * (size_t)s->B * K * s->D * scan_padded(s->N)) : 0;
}

cudaError_t scan_fwd(const ScanCall &c, cudaStream_t st)
{
    return c.s->dtype == DN_F32 ? fwd_t<float>(c, st) : fwd_t<__nv_bfloat16>(c, st);
}

cudaError_t scan_step(const ScanCall &c, cudaStream_t st)
{
    return c.s->dtype == DN_F32 ? step_t<float>(c, st) : step_t<__nv_bfloat16>(c, st);
}

}  // namespace lay
}  // namespace gdn

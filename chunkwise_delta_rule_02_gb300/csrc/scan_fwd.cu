// Selective state space scan: forward over tokens, and the single-token step.
//
// k_scan_fwd.  A block owns CH channels of one group and walks a row's tokens (or one
// time segment of them) in tiles:
//   1. every thread turns its part of the tile's x and dt into (delta, delta x), and
//      its part of B, C into float32, in shared memory;
//   2. the recurrence: per token a lane reads (delta, delta x) of its channel and S
//      values of B and C, and does S exponentials and 4 S multiply-adds;
//   3. y = (sum + D x) silu(z), stored with the tile's layout of x.
// The loads of the next tile are in flight during step 2.
//
// Bound by the exponentials and the float32 pipe, not by HBM: per (token, channel) N
// exponentials at 32 lanes a cycle and SM, and 4 N multiply-adds at 128: both N / 32
// cycles.  Few rows: the time axis is cut into K segments.  A first pass (SUM) runs all
// but the last segment from a zero state and keeps its end state and its decay product;
// the second pass composes what lies before its segment and runs it.  That costs the
// recurrence twice, so it is done only while the blocks do not fill the SMs.
#include "scan.cuh"

namespace gdn {
namespace lay {

namespace {

template <class Cfg>
struct FwdTile {
    static constexpr int TT = Cfg::L <= 2 ? 16 : 32;                 // tokens
    static constexpr int EPT = TT * Cfg::CH / kScanThreads;          // elements a thread
    static constexpr int NBC = (TT * Cfg::Np + kScanThreads - 1) / kScanThreads;   // elements of B (and of C) a thread
    static constexpr int YS = Cfg::CH + Cfg::CH / 8;                 // padded row of y: L rows x 32/L channels, no bank twice
};

template <class T, class Cfg, int VEC, bool SUM>
__global__ void __launch_bounds__(kScanThreads) k_scan_fwd(ScanDims g, ScanIo<T> io)
{
    constexpr int L = Cfg::L, S = Cfg::S, Np = Cfg::Np, CH = Cfg::CH;
    using F = FwdTile<Cfg>;
    constexpr int TT = F::TT, NV = F::EPT / VEC, NBC = F::NBC;
    __shared__ float2 dd[TT][CH];
    __shared__ __align__(16) float sb[TT][Np], sc[SUM ? 1 : TT][Np];
    __shared__ float sy[SUM ? 1 : TT][F::YS];
    __shared__ int seq[32];
    __shared__ uint32_t edge[2];

    const int tid = threadIdx.x, lane = tid & 31, l = tid & (L - 1), ch = tid / L, n0 = l * S;
    // block -> (channel tile, segment, row)
    int id = blockIdx.x;
    const int tile = id % (g.G * g.tiles);
    id /= g.G * g.tiles;
    const int nseg = SUM ? g.K - 1 : g.K, k = id % nseg, b = id / nseg;
    const int grp = tile / g.tiles, cg0 = (tile - grp * g.tiles) * CH;   // first channel within the group
    const bool live = cg0 + ch < g.Dg;
    const int c0 = grp * g.Dg + cg0;
    const long long c = live ? c0 + ch : c0;
    const int ts = k * g.seg, te = min(ts + g.seg, g.T);

    float2 a2[S / 2], h[S / 2], prod[S / 2];
    load_states<S>(a2, g.A + c * g.N, n0, g.N, live);
#pragma unroll
    for (int i = 0; i < S / 2; ++i) {
        a2[i] = mul2(a2[i], two(kLog2e));
        h[i] = two(0.f);
        prod[i] = two(1.f);
    }
    if constexpr (!SUM) {
        if (k > 0) carry_in<S>(h, g, io.segP, io.segH, b, k, c, n0, Np);
    }

    // this thread's vectors of a tile: token vt[e], channels vc[e] ..
    Vec<T, VEC> xr[NV], dr[NV], zr[NV], xn[NV], dn[NV], zn[NV];
    T br[NBC], cr[NBC];
    constexpr int RV = CH / VEC;   // vectors of a token
    auto vt = [&](int e) { return (tid + e * kScanThreads) / RV; };
    auto vc = [&](int e) { return (tid + e * kScanThreads) % RV * VEC; };
    const bool gated = !SUM && io.z.p != nullptr;
    auto fetch = [&](int t0) {
#pragma unroll
        for (int e = 0; e < NV; ++e) {
            const int t = t0 + vt(e), q = vc(e);
            xn[e].zero();
            dn[e].zero();
            zn[e].zero();
            if (t < te && cg0 + q < g.Dg) {
                xn[e].load(io.x.at(b, 0, t) + c0 + q);
                dn[e].load(io.dt.at(b, 0, t) + c0 + q);
                if (gated) zn[e].load(io.z.at(b, 0, t) + c0 + q);
            }
        }
#pragma unroll
        for (int e = 0; e < NBC; ++e) {
            const int i = tid + e * kScanThreads, t = t0 + i / Np, n = i % Np;
            st_out(&br[e], 0.f);
            st_out(&cr[e], 0.f);
            if (i < TT * Np && t < te && n < g.N) {
                br[e] = io.b.at(b, grp, t)[n];
                if (!SUM) cr[e] = io.c.at(b, grp, t)[n];
            }
        }
    };
    fetch(ts);

    for (int t0 = ts; t0 < te; t0 += TT) {
        // 1. the tile into shared memory
#pragma unroll
        for (int e = 0; e < NV; ++e) {
            float x[VEC], d[VEC];
            xr[e] = xn[e];
            dr[e] = dn[e];
            zr[e] = zn[e];
            xr[e].get(x);
            dr[e].get(d);
            const int t = vt(e), q = vc(e);
            const bool in = t0 + t < te && cg0 + q < g.Dg;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float v = d[i] + (in && g.bias ? g.bias[c0 + q + i] : 0.f), der;
                if (g.softplus) softplus(v, v, der);
                // tokens behind the end change nothing: delta = 0
                dd[t][q + i] = in ? make_float2(v, v * x[i]) : make_float2(0.f, 0.f);
            }
        }
#pragma unroll
        for (int e = 0; e < NBC; ++e) {
            const int i = tid + e * kScanThreads;
            if (i < TT * Np) {
                sb[i / Np][i % Np] = ld_in(&br[e]);
                if constexpr (!SUM) sc[i / Np][i % Np] = ld_in(&cr[e]);
            }
        }
        if (tid < 32) tile_edges(g, b, t0, min(TT, te - t0), seq, edge);
        __syncthreads();
        fetch(t0 + TT);

        // 2. the recurrence
        const uint32_t starts = edge[0], ends = edge[1];
#pragma unroll 1
        for (int g0 = 0; g0 < TT; g0 += L) {
            if constexpr (!SUM) {
                if (io.keep && g0 % kScanKeep == 0 && t0 + g0 < te && live)
                    store_pairs<S>(io.keep + (((size_t)b * ((g.T + kScanKeep - 1) / kScanKeep) + (t0 + g0) / kScanKeep) * g.D + c) * Np + n0, h);
            }
            const uint32_t in_group = ((starts | ends) >> g0) & (uint32_t)((1ull << L) - 1);
            float yp[L];
            auto token = [&](int j, bool edges) {
                const int t = g0 + j;
                const float2 q = dd[t][ch];
                float2 bb[S / 2];
                load_pairs<S>(bb, &sb[t][n0]);
                if (edges && (starts >> t & 1)) {
                    load_states<S>(h, g.h0 + ((size_t)seq[t] * g.D + c) * g.N, n0, g.N, live && g.h0);
#pragma unroll
                    for (int i = 0; i < S / 2; ++i) prod[i] = two(0.f);
                }
                float2 yy = two(0.f);
                float2 cc[S / 2];
                if constexpr (!SUM) load_pairs<S>(cc, &sc[t][n0]);
#pragma unroll
                for (int i = 0; i < S / 2; ++i) {
                    const float2 a = ex2_2(mul2(two(q.x), a2[i]));
                    h[i] = fma2(a, h[i], mul2(two(q.y), bb[i]));
                    if constexpr (SUM) prod[i] = mul2(prod[i], a);
                    else yy = fma2(cc[i], h[i], yy);
                }
                yp[j] = yy.x + yy.y;
                if constexpr (!SUM) {
                    if (edges && (ends >> t & 1) && io.hT)
                        store_states<S>(io.hT + ((size_t)seq[t] * g.D + c) * g.N, h, n0, g.N, live);
                }
            };
            if (in_group == 0) {
#pragma unroll
                for (int j = 0; j < L; ++j) token(j, false);
            } else {
#pragma unroll
                for (int j = 0; j < L; ++j) token(j, true);
            }
            if constexpr (!SUM) sy[g0 + l][ch] = lane_sum<L>(yp, lane);
        }
        __syncthreads();

        // 3. the results
        if constexpr (!SUM) {
#pragma unroll
            for (int e = 0; e < NV; ++e) {
                const int t = vt(e), q = vc(e);
                if (t0 + t < te && cg0 + q < g.Dg) {
                    float x[VEC], z[VEC], o[VEC];
                    xr[e].get(x);
                    zr[e].get(z);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        o[i] = fmaf(g.Dskip ? g.Dskip[c0 + q + i] : 0.f, x[i], sy[t][q + i]);
                        if (gated) o[i] *= z[i] * sigmoid(z[i]);
                    }
                    Vec<T, VEC> out;
                    out.set(o);
                    out.store(io.y.at(b, 0, t0 + t) + c0 + q);
                }
            }
        }
    }
    if constexpr (SUM) {
        if (live) {
            const size_t at = (((size_t)b * g.K + k) * g.D + c) * Np + n0;
            store_pairs<S>(io.segP + at, prod);
            store_pairs<S>(io.segH + at, h);
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

// One token a sequence: lanes of a channel take V states at a time (16 bytes where N and
// the states' alignment allow), so that a warp moves whole rows of the states, which are
// what this is bound by (HBM: states read and written once).
template <class T, int V>
__global__ void __launch_bounds__(256) k_scan_step(ScanDims g, ScanIo<T> io, int L)
{
    const long long i = (blockIdx.x * 256ll + threadIdx.x) / L;
    const int l = threadIdx.x & (L - 1);
    const bool live = i < (long long)g.B * g.D;   // the whole warp takes part in the sum
    const long long j = live ? i : 0;
    const int b = (int)(j / g.D), c = (int)(j - (long long)b * g.D), grp = c / g.Dg;
    const float x = ld_in(io.x.at(b, 0, 0) + c);
    float d = ld_in(io.dt.at(b, 0, 0) + c) + (g.bias ? g.bias[c] : 0.f), der;
    if (g.softplus) softplus(d, d, der);
    const float dx = d * x;
    const T *bp = io.b.at(b, grp, 0), *cp = io.c.at(b, grp, 0);
    const float *hi = g.h0 ? g.h0 + j * g.N : nullptr;
    float *ho = io.hT ? io.hT + j * g.N : nullptr;
    float y = 0.f;
    if (live) {
        for (int n = l * V; n < g.N; n += L * V) {
            Vec<float, V> hv, av;
            float h[V], a[V];
            hv.zero();
            if (hi) hv.load(hi + n);
            av.load(g.A + (size_t)c * g.N + n);
            hv.get(h);
            av.get(a);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                h[e] = fmaf(ex2(d * (a[e] * kLog2e)), h[e], dx * ld_in(bp + n + e));
                y = fmaf(ld_in(cp + n + e), h[e], y);
            }
            if (ho) {
                hv.set(h);
                hv.store(ho + n);
            }
        }
    }
    for (int o = L >> 1; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (live && l == 0) {
        y = fmaf(g.Dskip ? g.Dskip[c] : 0.f, x, y);
        if (io.z.p) {
            const float z = ld_in(io.z.at(b, 0, 0) + c);
            y *= z * sigmoid(z);
        }
        st_out(io.y.at(b, 0, 0) + c, y);
    }
}

// Time segments: while a row of blocks leaves SMs without work, at most one per 128 tokens.
int segments(const dn_scan_shape *s, int blocks)
{
    const int want = 4 * sm_count();
    int k = blocks >= want / 2 ? 1 : want / (blocks > 0 ? blocks : 1);
    const int most = (s->T + 127) / 128;
    if (k > most) k = most;
    if (k > 64) k = 64;
    return k < 1 ? 1 : k;
}

int scan_blocks(const dn_scan_shape *s, int CH)
{
    const int Dg = s->D / s->G;
    const long long n = (long long)s->B * s->G * ((Dg + CH - 1) / CH);
    return n > 0x3fffffff ? 0x3fffffff : (int)n;
}

int channels_of(int N)
{
    int ch = 0;
    scan_layout(N, [&](auto cfg) { ch = decltype(cfg)::CH; return cudaSuccess; });
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

template <class T, class Cfg, int VEC>
cudaError_t launch(const ScanCall &c, cudaStream_t st)
{
    ScanDims g = scan_dims(c);
    g.tiles = (g.Dg + Cfg::CH - 1) / Cfg::CH;
    g.K = segments(c.s, scan_blocks(c.s, Cfg::CH));
    const int TT = FwdTile<Cfg>::TT;
    g.seg = ((g.T + g.K - 1) / g.K + TT - 1) / TT * TT;
    g.K = (g.T + g.seg - 1) / g.seg;
    ScanIo<T> io = io_of<T>(c);
    const long long per = (long long)g.B * g.G * g.tiles;
    if (per * g.K > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (g.K > 1) {
        io.segP = (float *)c.ws;
        io.segH = io.segP + (size_t)g.B * g.K * g.D * Cfg::Np;
        k_scan_fwd<T, Cfg, VEC, true><<<(unsigned)(per * (g.K - 1)), kScanThreads, 0, st>>>(g, io);
    }
    k_scan_fwd<T, Cfg, VEC, false><<<(unsigned)(per * g.K), kScanThreads, 0, st>>>(g, io);
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
    return scan_layout(s->N, [&](auto cfg) {
        using Cfg = decltype(cfg);
        constexpr int VEC = FwdTile<Cfg>::EPT < 4 ? FwdTile<Cfg>::EPT : 4;
        const int bytes = VEC * sizeof(T);
        const bool v = (s->D / s->G) % VEC == 0 && can_vector(&io->x, sizeof(T), bytes) && can_vector(&io->dt, sizeof(T), bytes) &&
                       can_vector(&io->z, sizeof(T), bytes) && can_vector(&io->y, sizeof(T), bytes);
        return v ? launch<T, Cfg, VEC>(c, st) : launch<T, Cfg, 1>(c, st);
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
    int L = 1;
    while (L < 32 && L * V < g.N) L <<= 1;
    const long long blocks = ((long long)g.B * g.D * L + 255) / 256;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (V == 4) k_scan_step<T, 4><<<(unsigned)blocks, 256, 0, st>>>(g, io, L);
    else k_scan_step<T, 1><<<(unsigned)blocks, 256, 0, st>>>(g, io, L);
    return cudaPeekAtLastError();
}

}  // namespace

int scan_padded(int N)
{
    int np = 0;
    scan_layout(N, [&](auto cfg) { np = decltype(cfg)::Np; return cudaSuccess; });
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
    const int K = segments(s, scan_blocks(s, channels_of(s->N)));
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

// RMS norm of a row of d features with its output gate, or with the residual sum
// in front of it: forward and backward.
//
//     r = residual + s x (or x),  q = 1 / sqrt(mean r^2 + eps),  y = r q w silu(z)
//     g = dy w silu(z),  dr = q (g - r q^2 mean(g r)) + dsum,  dx = s dr,
//     dw = sum dy r q silu(z),  dz = dy r q w silu'(z),  ds = sum dr x
//
// Bound by HBM: every operand is read once and every result written once, in one
// pass; a row stays in registers between its loads and its results.  R threads
// share a row: part of a warp (sums by shuffles, several rows a warp) while a
// thread then holds at most 4 vectors, else one block.  mean r^2 and
// mean(g r) come out of one reduction.  Both sums, and the row, are float32.
// Measured, gate and rows of 128 bf16: forward 5.6 TB/s (83 % of a copy), backward
// 4.8 TB/s (71 %).  Residual, rows of 2048 bf16: forward 107 us for 8 x 4096 rows (74 %),
// backward 402 us (30 %), which spills: see k_norm_bwd.
#include "layers.h"

namespace gdn {
namespace lay {

namespace {

constexpr int kThreads = 256;
// Most blocks an SM of a pass: the backward's write partial sums, so that they are as many as
// run together (3; 4 were 162 us, 6 141 us, 3 138 us at 8 x 16 x 4096 x 128 with the gate, the only
// instance that the number and the register bound were measured on); the forward's are
// four rounds of six (24: 72 us; 12: 76 us; 48: 74 us at 4 x 16 x 8192 x 128).
constexpr long long kFwdBlocks = 24, kBwdBlocks = 3;

struct NormDims {
    int B, H, T, d, R;              // R: threads of a row
    int per_head;                   // grid.y = H, rows of one head only
    unsigned rows, chunk;           // rows of a grid.y slice, rows of a block
    float eps, inv_d;
};

// A thread's place in an array: its features of a row.  The thread's next row is `step` rows
// on: within one (batch, head) that is a step along t; only past its end is the row's place
// found anew (two divisions).
struct Row {
    int b, h, t;
    __device__ __forceinline__ void find(const NormDims &g, unsigned r)
    {
        const unsigned q = r / (unsigned)g.T;
        t = (int)(r - q * (unsigned)g.T);
        if (g.per_head) {
            b = (int)q;
            h = blockIdx.y;
        } else {
            b = (int)(q / (unsigned)g.H);
            h = (int)(q - (unsigned)b * (unsigned)g.H);
        }
    }
};

template <class T>
struct At {
    T *p;
    __device__ __forceinline__ void find(const View<T> &v, const Row &o, int i0) { p = v.p ? v.at(o.b, o.h, o.t) + i0 : nullptr; }
    __device__ __forceinline__ void step(const View<T> &v, int n) { p += n * v.t; }
};

// Sum of (a, b) over the R threads of a row.  WIDE: R = blockDim.x.
template <bool WIDE>
__device__ __forceinline__ float2 row_sum(float a, float b, int R, float2 *sm)
{
    const int top = WIDE ? 16 : R >> 1;
    for (int o = top; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if constexpr (WIDE) {
        const int warps = blockDim.x >> 5;
        __syncthreads();
        if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        a = b = 0.f;
        for (int i = 0; i < warps; ++i) {
            a += sm[i].x;
            b += sm[i].y;
        }
    }
    return make_float2(a, b);
}

// w of this thread's features: element e of vector v is feature (v R + lane) V + e
template <int V, int NV>
__device__ __forceinline__ void load_w(float (&f)[NV][V], const float *w, int d, int R, int lane, float none)
{
    const bool wide = V >= 4 && ((uintptr_t)w & 15u) == 0;   // d is a multiple of V
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int i = (v * R + lane) * V;
#pragma unroll
        for (int e = 0; e < V; ++e) f[v][e] = none;
        if (w && i < d) {
            if (wide) {
#pragma unroll
                for (int e = 0; e < V; e += 4) {
                    const float4 q = *reinterpret_cast<const float4 *>(w + i + e);
                    f[v][e] = q.x;
                    if (V >= 4) {
                        f[v][V >= 4 ? e + 1 : 0] = q.y;
                        f[v][V >= 4 ? e + 2 : 0] = q.z;
                        f[v][V >= 4 ? e + 3 : 0] = q.w;
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) f[v][e] = w[i + e];
            }
        }
    }
}

template <class T, int V, int NV>
__device__ __forceinline__ void load_row(Vec<T, V> (&q)[NV], const T *p, int d, int vs, int i0)
{
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        q[v].zero();
        if (i0 + v * vs < d) q[v].load(p + v * vs);
    }
}

template <class T, int V, int NV, bool WIDE, bool GATE, bool RES>
__global__ void __launch_bounds__(WIDE ? 1024 : kThreads)
    k_norm_fwd(NormDims g, View<const T> x, View<const T> z, View<const T> res, View<T> y, View<T> sum,
               const float *__restrict__ w, const float *__restrict__ rs)
{
    __shared__ float2 sm[32];
    const int R = WIDE ? blockDim.x : g.R, lane = WIDE ? threadIdx.x : threadIdx.x & (R - 1);
    const int grp = WIDE ? 0 : threadIdx.x / R, grps = WIDE ? 1 : kThreads / R;
    float wf[NV][V], sf[RES ? NV : 1][V];
    load_w<V, NV>(wf, w + (g.per_head ? (size_t)blockIdx.y * g.d : 0), g.d, R, lane, 0.f);
    if constexpr (RES) load_w<V, NV>(sf, rs, g.d, R, lane, 1.f);
    const unsigned r0 = blockIdx.x * g.chunk, r1 = min(r0 + g.chunk, g.rows);
    const int i0 = lane * V, vs = R * V;
    Row o;
    At<const T> ax, az, ae;
    At<T> ay, as;
    auto find = [&](unsigned r) {
        o.find(g, r);
        ax.find(x, o, i0);
        ay.find(y, o, i0);
        if constexpr (GATE) az.find(z, o, i0);
        if constexpr (RES) {
            ae.find(res, o, i0);
            as.find(sum, o, i0);
        }
    };
    find(min(r0 + grp, r1 - 1));
    for (unsigned rb = r0; rb < r1; rb += grps) {   // every thread of a warp takes part in the sums
        const unsigned r = rb + grp;
        const bool live = r < r1;
        Vec<T, V> xv[NV], zv[GATE ? NV : 1], ev[RES ? NV : 1];
        load_row<T, V, NV>(xv, ax.p, g.d, vs, i0);
        if constexpr (GATE) load_row<T, V, NV>(zv, az.p, g.d, vs, i0);
        if constexpr (RES) load_row<T, V, NV>(ev, ae.p, g.d, vs, i0);
        float f[NV][V], ss = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            xv[v].get(f[v]);
            if constexpr (RES) {
                float e[V];
                ev[v].get(e);
#pragma unroll
                for (int i = 0; i < V; ++i) f[v][i] = fmaf(sf[v][i], f[v][i], e[i]);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) ss = fmaf(f[v][i], f[v][i], ss);
        }
        const float q = rsqrtf(fmaf(row_sum<WIDE>(ss, 0.f, R, sm).x, g.inv_d, g.eps));
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (live && i0 + v * vs < g.d) {
                float out[V];
                Vec<T, V> ov;
                if constexpr (RES) {
                    if (as.p) {
                        ov.set(f[v]);
                        ov.store(as.p + v * vs);
                    }
                }
                if constexpr (GATE) {
                    float e[V];
                    zv[v].get(e);
#pragma unroll
                    for (int i = 0; i < V; ++i) out[i] = f[v][i] * q * wf[v][i] * (e[i] * sigmoid(e[i]));
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i) out[i] = f[v][i] * q * wf[v][i];
                }
                ov.set(out);
                ov.store(ay.p + v * vs);
            }
        }
        if (r + grps < r1) {
            o.t += grps;
            if (o.t < g.T) {
                ax.step(x, grps);
                ay.step(y, grps);
                if constexpr (GATE) az.step(z, grps);
                if constexpr (RES) {
                    ae.step(res, grps);
                    if (as.p) as.step(sum, grps);
                }
            } else {
                find(r + grps);
            }
        }
    }
}

struct NormGrad {
    float *part_w, *part_s;   // [grid.x][grid.y][d]
};

// RES: r is read from `sum`, x only for ds; else r = x.
// The bounds leave 80 registers (64 for a block a row).  Instances without a residual and with one vector a
// thread fit them or nearly; those with a residual, whose sums of dw and ds and five operands are all in
// registers, spill: 120 to 1400 bytes of stack with 8 bf16 an access, up to 600 with 4 float32.  Residual backward
// of 8 x 4096 rows: 477, 402, 948 us for 1024, 2048, 4096 bf16 features (bytes: 59, 119, 237 us), 161, 342, 659 us
// for float32 (119, 237, 475 us).
template <class T, int V, int NV, bool WIDE, bool GATE, bool RES>
__global__ void __launch_bounds__(WIDE ? 1024 : kThreads, WIDE ? 1 : 3)
    k_norm_bwd(NormDims g, View<const T> x, View<const T> z, View<const T> sum, View<const T> dy, View<const T> dsum,
               View<T> dx, View<T> dz, View<T> dres, const float *__restrict__ w, const float *__restrict__ rs,
               NormGrad pg)
{
    extern __shared__ float red[];   // partial sums of the groups of a block (not WIDE)
    __shared__ float2 sm[32];
    const int R = WIDE ? blockDim.x : g.R, lane = WIDE ? threadIdx.x : threadIdx.x & (R - 1);
    const int grp = WIDE ? 0 : threadIdx.x / R, grps = WIDE ? 1 : kThreads / R;
    float wf[NV][V], sf[RES ? NV : 1][V], aw[NV][V], as[RES ? NV : 1][V];
    load_w<V, NV>(wf, w + (g.per_head ? (size_t)blockIdx.y * g.d : 0), g.d, R, lane, 0.f);
    if constexpr (RES) load_w<V, NV>(sf, rs, g.d, R, lane, 1.f);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            aw[v][i] = 0.f;
            if constexpr (RES) as[v][i] = 0.f;
        }
    const unsigned r0 = blockIdx.x * g.chunk, r1 = min(r0 + g.chunk, g.rows);
    const int i0 = lane * V, vs = R * V;
    Row o;
    At<const T> ar, ad, az, ax, ae;     // r, dy, z, x (for ds), dsum
    At<T> bx, bz, br;                   // dx, dz, dresidual
    auto find = [&](unsigned r) {
        o.find(g, r);
        ar.find(RES ? sum : x, o, i0);
        ad.find(dy, o, i0);
        bx.find(dx, o, i0);
        if constexpr (GATE) {
            az.find(z, o, i0);
            bz.find(dz, o, i0);
        }
        if constexpr (RES) {
            ax.find(x, o, i0);
            ae.find(dsum, o, i0);
            br.find(dres, o, i0);
        }
    };
    find(min(r0 + grp, r1 - 1));
    for (unsigned rb = r0; rb < r1; rb += grps) {
        const unsigned r = rb + grp;
        const bool live = r < r1;
        Vec<T, V> rv[NV], dv[NV], zv[GATE ? NV : 1], xv[RES ? NV : 1], ev[RES ? NV : 1];
        load_row<T, V, NV>(rv, ar.p, g.d, vs, i0);
        load_row<T, V, NV>(dv, ad.p, g.d, vs, i0);
        if constexpr (GATE) load_row<T, V, NV>(zv, az.p, g.d, vs, i0);
        if constexpr (RES) {
#pragma unroll
            for (int v = 0; v < NV; ++v) xv[v].zero(), ev[v].zero();
            if (pg.part_s) load_row<T, V, NV>(xv, ax.p, g.d, vs, i0);
            if (ae.p) load_row<T, V, NV>(ev, ae.p, g.d, vs, i0);
        }
        float ss = 0.f, gr = 0.f, sig[GATE ? NV : 1][V];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float f[V], dyf[V], e[V];
            rv[v].get(f);
            dv[v].get(dyf);
            if constexpr (GATE) zv[v].get(e);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if constexpr (GATE) sig[v][i] = sigmoid(e[i]);
                const float gate = GATE ? e[i] * sig[GATE ? v : 0][i] : 1.f;
                ss = fmaf(f[i], f[i], ss);
                gr = fmaf(dyf[i] * wf[v][i] * gate, f[i], gr);
            }
        }
        const float2 s2 = row_sum<WIDE>(ss, gr, R, sm);
        const float q = rsqrtf(fmaf(s2.x, g.inv_d, g.eps)), m = q * q * s2.y * g.inv_d;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (live && i0 + v * vs < g.d) {
                float f[V], dyf[V], e[V], a[V], xo[V], zo[V];
                rv[v].get(f);
                dv[v].get(dyf);
                if constexpr (GATE) zv[v].get(e);
                if constexpr (RES) {
                    ev[v].get(a);
                    xv[v].get(xo);
                }
                Vec<T, V> ov;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float sg = GATE ? sig[GATE ? v : 0][i] : 1.f, gate = GATE ? e[i] * sg : 1.f, n = f[i] * q;
                    const float dn = dyf[i] * n;
                    aw[v][i] = fmaf(dn, gate, aw[v][i]);
                    if (GATE) zo[i] = dn * wf[v][i] * dsilu(e[i], sg);
                    float dr = q * fmaf(-f[i], m, dyf[i] * wf[v][i] * gate);
                    if constexpr (RES) {
                        dr += a[i];
                        as[v][i] = fmaf(dr, xo[i], as[v][i]);
                    }
                    f[i] = dr;
                }
                if constexpr (RES) {
                    if (br.p) {
                        ov.set(f);
                        ov.store(br.p + v * vs);
                    }
#pragma unroll
                    for (int i = 0; i < V; ++i) f[i] *= sf[v][i];
                }
                if (bx.p) {
                    ov.set(f);
                    ov.store(bx.p + v * vs);
                }
                if constexpr (GATE) {
                    if (bz.p) {
                        ov.set(zo);
                        ov.store(bz.p + v * vs);
                    }
                }
            }
        }
        if (r + grps < r1) {
            o.t += grps;
            if (o.t < g.T) {
                ar.step(RES ? sum : x, grps);
                ad.step(dy, grps);
                if (bx.p) bx.step(dx, grps);
                if constexpr (GATE) {
                    az.step(z, grps);
                    if (bz.p) bz.step(dz, grps);
                }
                if constexpr (RES) {
                    if (ax.p) ax.step(x, grps);
                    if (ae.p) ae.step(dsum, grps);
                    if (br.p) br.step(dres, grps);
                }
            } else {
                find(r + grps);
            }
        }
    }
    // this block's sums of dw (and ds): over its groups in order, then one row of partials
    const size_t at = ((size_t)blockIdx.x * gridDim.y + blockIdx.y) * g.d;
    for (int kind = 0; kind < (RES && pg.part_s ? 2 : 1); ++kind) {
        float *dst = (kind ? pg.part_s : pg.part_w) + at;
        if constexpr (WIDE) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const int i = (v * R + lane) * V + e;
                    if (i < g.d) dst[i] = kind && RES ? as[RES ? v : 0][e] : aw[v][e];
                }
        } else {
            const int span = R * NV * V;
            __syncthreads();
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int e = 0; e < V; ++e)
                    red[grp * span + (v * R + lane) * V + e] = kind && RES ? as[RES ? v : 0][e] : aw[v][e];
            __syncthreads();
            for (int i = threadIdx.x; i < g.d; i += kThreads) {
                float s = 0.f;
                for (int k = 0; k < grps; ++k) s += red[k * span + i];
                dst[i] = s;
            }
        }
    }
}

struct Shape {
    bool wide;
    int R, nv, threads;
};

// Threads of a row: a part of a warp while that leaves at most 4 vectors (16 single
// elements: 4) a thread, else a block of 128 .. 1024 threads.
Shape shape_of(int d, int V)
{
    const int n = (d + V - 1) / V;
    Shape s;
    if (n <= 32 * 4) {
        s.wide = false;
        s.R = 1;
        while (s.R < 32 && s.R < n) s.R <<= 1;
        s.nv = (n + s.R - 1) / s.R;
        s.threads = kThreads;
    } else {
        s.wide = true;
        s.R = 128;
        while (s.R < 1024 && s.R * (V == 1 ? 4 : 1) < n) s.R <<= 1;
        s.nv = (n + s.R - 1) / s.R;
        s.threads = s.R;
    }
    return s;
}

// Blocks of a pass whose partial sums leave the block (backward), as a multiple of the SMs.
unsigned grid_of(const dn_norm_shape *s, int per_block, bool bwd, unsigned &chunk, unsigned &rows)
{
    const int ny = s->w_per_head ? s->H : 1;
    const long long all = (long long)s->B * s->H * s->T / ny;
    rows = (unsigned)all;
    long long blocks = (all + per_block - 1) / per_block;
    const long long most = bwd ? kBwdBlocks * sm_count() / ny + 1 : kFwdBlocks * sm_count() / ny + 1;
    blocks = blocks < most ? blocks : most;
    if (blocks < 1) blocks = 1;
    chunk = (unsigned)((all + blocks - 1) / blocks);
    chunk = (chunk + per_block - 1) / per_block * per_block;
    return chunk ? (unsigned)((all + chunk - 1) / chunk) : 1;
}

template <class T>
bool vectors(const NormCall &c)
{
    constexpr int V = 16 / sizeof(T);
    const dn_view *all[] = {c.x, c.z, c.residual, c.sum, c.y, c.dy, c.dsum, c.dx, c.dz, c.dresidual};
    if (c.s->d % V) return false;
    for (const dn_view *v : all)
        if (!can_vector(v, sizeof(T), 16)) return false;
    return true;
}

template <class T, int V, int NV, bool WIDE, bool GATE, bool RES>
cudaError_t launch(const NormCall &c, const Shape &sh, bool bwd, cudaStream_t st)
{
    NormDims g;
    g.B = c.s->B; g.H = c.s->H; g.T = c.s->T; g.d = c.s->d; g.R = sh.R; g.per_head = c.s->w_per_head;
    g.eps = c.s->eps; g.inv_d = 1.f / (float)g.d;
    const int grps = WIDE ? 1 : kThreads / sh.R;
    const unsigned gx = grid_of(c.s, grps, bwd, g.chunk, g.rows);
    const dim3 grid(gx, c.s->w_per_head ? c.s->H : 1);
    const View<const T> x = view_of<const T>(c.x), z = view_of<const T>(c.z);
    if (!bwd) {
        k_norm_fwd<T, V, NV, WIDE, GATE, RES><<<grid, sh.threads, 0, st>>>(g, x, z, view_of<const T>(c.residual), view_of<T>(c.y),
                                                                        view_of<T>(c.sum), c.w, c.res_scale);
        return cudaPeekAtLastError();
    }
    NormGrad pg;
    const size_t n = (size_t)grid.x * grid.y * g.d;
    pg.part_w = c.part;
    pg.part_s = c.dres_scale ? c.part + n : nullptr;
    const size_t smem = WIDE ? 0 : (size_t)grps * sh.R * NV * V * sizeof(float);
    k_norm_bwd<T, V, NV, WIDE, GATE, RES><<<grid, sh.threads, smem, st>>>(
        g, x, z, view_of<const T>(c.sum), view_of<const T>(c.dy), view_of<const T>(c.dsum), view_of<T>(c.dx), view_of<T>(c.dz),
        view_of<T>(c.dresidual), c.w, c.res_scale, pg);
    ColSum rw, rs;
    rw.part = pg.part_w;
    rw.P = grid.x;
    rw.C = (long long)grid.y * g.d;
    rw.kinds = 1;
    rw.dst[0] = c.dw;
    rw.step[0] = 1;
    rs = rw;
    rs.part = pg.part_s;
    rs.P = (long long)grid.x * grid.y;
    rs.C = g.d;
    rs.dst[0] = c.dres_scale;
    return col_sum(rw, c.dres_scale ? &rs : nullptr, st);
}

template <class T, int V, int NV, bool WIDE>
cudaError_t by_flags(const NormCall &c, const Shape &sh, bool bwd, cudaStream_t st)
{
    const bool gate = c.z && c.z->data;
    const bool res = bwd ? (c.sum && c.sum->data) || c.res_scale || c.dres_scale || (c.dsum && c.dsum->data) ||
                               (c.dresidual && c.dresidual->data)
                         : (c.residual && c.residual->data) || c.res_scale || (c.sum && c.sum->data);
    if (gate) return res ? launch<T, V, NV, WIDE, true, true>(c, sh, bwd, st) : launch<T, V, NV, WIDE, true, false>(c, sh, bwd, st);
    return res ? launch<T, V, NV, WIDE, false, true>(c, sh, bwd, st) : launch<T, V, NV, WIDE, false, false>(c, sh, bwd, st);
}

template <class T>
cudaError_t run(const NormCall &c, bool bwd, cudaStream_t st)
{
    constexpr int V = 16 / sizeof(T);
    if (vectors<T>(c)) {
        const Shape s = shape_of(c.s->d, V);
        if (!s.wide) {
            if (s.nv == 1) return by_flags<T, V, 1, false>(c, s, bwd, st);
            if (s.nv == 2) return by_flags<T, V, 2, false>(c, s, bwd, st);
            return by_flags<T, V, 4, false>(c, s, bwd, st);
        }
        if (s.nv == 1) return by_flags<T, V, 1, true>(c, s, bwd, st);
        return by_flags<T, V, 4, true>(c, s, bwd, st);
    }
    const Shape s = shape_of(c.s->d, 1);
    if (!s.wide) return by_flags<T, 1, 4, false>(c, s, bwd, st);
    return by_flags<T, 1, 16, true>(c, s, bwd, st);
}

}  // namespace

// an upper bound over the variants: rows of d floats of one kind of partial sums
long long norm_part_rows(const dn_norm_shape *s)
{
    const int ny = s->w_per_head ? s->H : 1;
    return (kBwdBlocks * sm_count() / ny + 1) * ny;
}

cudaError_t norm_fwd(const NormCall &c, cudaStream_t st)
{
    return c.s->dtype == DN_F32 ? run<float>(c, false, st) : run<__nv_bfloat16>(c, false, st);
}

cudaError_t norm_bwd(const NormCall &c, cudaStream_t st)
{
    return c.s->dtype == DN_F32 ? run<float>(c, true, st) : run<__nv_bfloat16>(c, true, st);
}

}  // namespace lay
}  // namespace gdn

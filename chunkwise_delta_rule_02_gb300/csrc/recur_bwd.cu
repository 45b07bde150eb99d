// Gated linear recurrence: backward.
//
//     g = dy silu(z),  dh_t = g_t + a_{t+1} dh_{t+1},  q = m dh (u a^2 / s - a h_{t-1})
//     drg = q (1 - r),  dlam = sigmoid(lam) / softplus(lam) sum q,  r = sigmoid(rg + rg_bias)
//     dx = dh s i,  dig = dh s x i (1 - i),  i = sigmoid(ig + ig_bias),  dz = dy h silu'(z)
//
// (log a = -m: d log a = dh (a h_{t-1} - u a^2 / s), and m / s goes to 0 with m, so that no gradient is
// infinite where a is 1.)  The recurrence of dh runs from the end as the forward's does from the start: same
// blocks, runs and exchange (recur.cuh), in the opposite order.  A thread makes its run's h again from the state that
// the forward pass kept at the run's start, so that nothing of the forward recurrence has to be exchanged; what
// dh is multiplied with is in registers before the exchange.
#include "recur.cuh"

namespace gdn {
namespace lay {

namespace {

template <class T, bool WIDE, bool PACKED>
__global__ void __launch_bounds__(kRecurThreads) k_recur_bwd(RecurDims g, RecurIo<T> io)
{
    __shared__ RecurShared sm;
    __shared__ float2 red[3][kWarps][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = g.CL > 1 ? cluster_rank() : 0;
    const int id = blockIdx.x / g.CL, b = id / g.tiles, c = (id - b * g.tiles) * kChans + 2 * lane;
    const bool in0 = c < g.D, in1 = c + 1 < g.D;
    const int cc = in0 ? c : 0;
    const bool gated = io.z.p != nullptr;
    RecurParams par;
    float2 dk;
    par.load(g, c, in0, in1, &dk);
    const int te = PACKED ? g.cu[g.Nseq] : g.T;
    float2 carry = two(0.f);   // the gradient that reaches a token's state from behind it
    if (!PACKED && io.dhT) carry = load2(io.dhT + (size_t)b * g.D + c, in0, in1);
    const int span = kSpan * g.CL, steps = (te + span - 1) / span;
    const size_t kept = (g.T + kRun - 1) / kRun;
    float2 sq = two(0.f), sr = two(0.f), si = two(0.f);
    if (g.CL > 1) cluster_barrier();   // all of the cluster's blocks run before one writes to another

    for (int st = steps - 1; st >= 0; --st) {
        const int t = st * span + rank * kSpan + warp * kRun, n = max(0, min(kRun, te - t));
        Two<T, WIDE> x[kRun], r[kRun], i[kRun], z[kRun], dy[kRun];
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            const bool in = k < n;
            x[k].load(io.x.at(b, 0, in ? t + k : 0) + cc, in && in0, in && in1);
            r[k].load(io.rg.at(b, 0, in ? t + k : 0) + cc, in && in0, in && in1);
            i[k].load(io.ig.at(b, 0, in ? t + k : 0) + cc, in && in0, in && in1);
            dy[k].load(io.dy.at(b, 0, in ? t + k : 0) + cc, in && in0, in && in1);
            if (gated) z[k].load(io.z.at(b, 0, in ? t + k : 0) + cc, in && in0, in && in1);
        }
        uint32_t starts = 0, ends = 0;
        int seq = 0;
        if (PACKED) run_edges(g, t, n, starts, ends, seq);
        float2 h = n > 0 ? load2(io.keep + ((size_t)b * kept + t / kRun) * g.D + c, in0, in1) : two(0.f);

        // the run's states, and of each token what dh is multiplied with
        float2 a[kRun], gy[kRun], fq[kRun], f1[kRun], fx[kRun], fi[kRun];
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            const float2 rr = sigmoid2(add2(r[k].get(), par.rb)), m = mul2(par.km, rr);
            const float2 ii = sigmoid2(add2(i[k].get(), par.ib)), u = mul2(ii, x[k].get());
            float2 y, rs;
            decay_of(m, a[k], y, rs);
            const float2 s = mul2(y, rs);
            if (PACKED && (starts >> k & 1)) {
                const int q = __shfl_sync(0xffffffffu, seq, k);
                h = g.h0 ? load2(g.h0 + (size_t)q * g.D + c, in0, in1) : two(0.f);
            }
            // u a / s comes with m / s: m rs u a, which is 0 where m is
            const float2 ma = mul2(m, a[k]);
            fq[k] = mul2(ma, fma2(mul2(rs, u), a[k], mul2(two(-1.f), h)));
            f1[k] = fma2(two(-1.f), rr, two(1.f));
            fx[k] = mul2(s, ii);
            fi[k] = mul2(mul2(s, u), fma2(two(-1.f), ii, two(1.f)));
            h = fma2(a[k], h, mul2(s, u));
            gy[k] = dy[k].get();
            if (gated) {
                const float2 zz = z[k].get(), p = sigmoid2(zz);
                const float2 dz = mul2(mul2(gy[k], h), make_float2(dsilu(zz.x, p.x), dsilu(zz.y, p.y)));
                if (k < n) put_two<T, WIDE>(io.dz.at(b, 0, t + k) + cc, dz, in0, in1);
                gy[k] = mul2(gy[k], mul2(zz, p));
            }
            if (k >= n) {   // behind the end: nothing changes
                a[k] = two(1.f);
                gy[k] = two(0.f);
            }
        }
        float2 A = two(1.f), H = two(0.f);
#pragma unroll
        for (int k = kRun - 1; k >= 0; --k) {
            if (PACKED && (ends >> k & 1)) {
                A = two(-1.f);
                H = io.dhT ? load2(io.dhT + (size_t)__shfl_sync(0xffffffffu, seq, k) * g.D + c, in0, in1) : two(0.f);
            }
            A = mul2(A, a[k]);
            H = mul2(a[k], add2(gy[k], H));
        }
        float2 back = exchange(sm, st & 1, g.CL, g.CL - 1 - rank, kWarps - 1 - warp, A, H, carry);
#pragma unroll
        for (int k = kRun - 1; k >= 0; --k) {
            if (PACKED && (ends >> k & 1))
                back = io.dhT ? load2(io.dhT + (size_t)__shfl_sync(0xffffffffu, seq, k) * g.D + c, in0, in1) : two(0.f);
            const float2 dh = add2(gy[k], back), q = mul2(dh, fq[k]), drg = mul2(q, f1[k]), dig = mul2(dh, fi[k]);
            back = mul2(a[k], dh);
            if (PACKED && (starts >> k & 1) && io.dh0)
                store2(io.dh0 + (size_t)__shfl_sync(0xffffffffu, seq, k) * g.D + c, back, in0, in1);
            if (k < n) {
                put_two<T, WIDE>(io.dx.at(b, 0, t + k) + cc, mul2(dh, fx[k]), in0, in1);
                put_two<T, WIDE>(io.drg.at(b, 0, t + k) + cc, drg, in0, in1);
                put_two<T, WIDE>(io.dig.at(b, 0, t + k) + cc, dig, in0, in1);
                sq = add2(sq, q);
                sr = add2(sr, drg);
                si = add2(si, dig);
            }
        }
    }
    if (!PACKED && io.dh0 && rank == 0 && warp == 0) store2(io.dh0 + (size_t)b * g.D + c, carry, in0, in1);

    red[0][warp][lane] = mul2(sq, dk);
    red[1][warp][lane] = sr;
    red[2][warp][lane] = si;
    __syncthreads();
    if (warp < 3) {
        float2 v = red[warp][0][lane];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) v = add2(v, red[warp][w][lane]);
        store2(io.part + (((size_t)b * g.CL + rank) * 3 + warp) * g.D + c, v, in0, in1);
    }
}

// Initial states' gradients of empty sequences: those of the final ones.
__global__ void __launch_bounds__(256) k_recur_empty_grad(const int32_t *cu, int D, const float *from, float *to)
{
    const int s = blockIdx.x;
    if (cu[s] != cu[s + 1]) return;
    for (int c = threadIdx.x; c < D; c += 256) to[(size_t)s * D + c] = from ? from[(size_t)s * D + c] : 0.f;
}

template <class T>
cudaError_t bwd(const RecurCall &c, cudaStream_t st)
{
    const RecurDims g = recur_dims(c, true);
    RecurIo<T> io = {};
    const dn_recur_io *f = c.io;
    const dn_recur_grads *r = c.gr;
    io.x = view_of<const T>(&f->x); io.rg = view_of<const T>(&f->rg); io.ig = view_of<const T>(&f->ig); io.z = view_of<const T>(&f->z);
    io.dy = view_of<const T>(&r->dy); io.dx = view_of<T>(&r->dx); io.drg = view_of<T>(&r->drg); io.dig = view_of<T>(&r->dig);
    io.dz = view_of<T>(&r->dz);
    io.keep = c.keep; io.dhT = r->dhT; io.dh0 = r->dh0; io.part = c.part;
    const int e = sizeof(T);
    bool wide = g.D % 2 == 0;
    const dn_view *views[] = {&f->x, &f->rg, &f->ig, &f->z, &r->dy, &r->dx, &r->drg, &r->dig, &r->dz};
    for (const dn_view *v : views) wide = wide && can_vector(v, e, 2 * e);
    if (g.cu && io.dh0 && g.Nseq > 0) k_recur_empty_grad<<<g.Nseq, 256, 0, st>>>(g.cu, g.D, io.dhT, io.dh0);
    cudaError_t rc;
    if (g.cu) rc = wide ? recur_launch(k_recur_bwd<T, true, true>, g, st, io) : recur_launch(k_recur_bwd<T, false, true>, g, st, io);
    else rc = wide ? recur_launch(k_recur_bwd<T, true, false>, g, st, io) : recur_launch(k_recur_bwd<T, false, false>, g, st, io);
    if (rc != cudaSuccess) return rc;
    const ColSum s = {c.part, (long long)g.B * g.CL, g.D, 3, {r->dlam, r->drg_bias, r->dig_bias}, {1, 1, 1}};
    return col_sum(s, nullptr, st);
}

}  // namespace

cudaError_t recur_bwd(const RecurCall &c, cudaStream_t st) { return c.s->dtype == DN_F32 ? bwd<float>(c, st) : bwd<__nv_bfloat16>(c, st); }

}  // namespace lay
}  // namespace gdn

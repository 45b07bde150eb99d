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

template <class T, int Q, int MODE, bool PACKED>
__global__ void __launch_bounds__(32 * bwd_warps(sizeof(T))) k_recur_bwd(const __grid_constant__ RecurMaps maps, RecurDims g, RecurIo<T> io)
{
    constexpr int W = bwd_warps(sizeof(T)), S = bwd_stages(sizeof(T)), L = 32 / Q, R = kRun * Q;
    extern __shared__ __align__(128) char raw[];
    __shared__ RecurShared<W, Q> sm;
    __shared__ float2 red[3][W][L];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = g.CL > 1 ? cluster_rank() : 0;
    const int id = blockIdx.x / g.CL, b = id / g.tiles, c0 = (id - b * g.tiles) * (64 / Q), c = c0 + 2 * (lane % L), q = lane / L * kRun;
    const bool in0 = c < g.D, in1 = c + 1 < g.D;
    const bool gated = io.in[kZ].p != nullptr;
    Ring<T, W, Q, S, MODE> ring;
    ring.init(raw, sm.bar[warp], &io, &maps, gated ? 31 : 23, b, c0, g.D);
    const int te = PACKED ? g.cu[g.Nseq] : g.T;
    const int span = W * R * g.CL, steps = (te + span - 1) / span;
    const int first = (rank * W + warp) * R;
    auto token = [&](int st) { return (steps - 1 - st) * span + first; };   // step st handles the st-th span from the end
    for (int st = 0; st < S - 1; ++st) {
        if (st < steps) ring.ask(st, token(st), te - token(st));
        ring.asked();
    }
    RecurParams par;
    float2 dk;
    par.load(g, c, in0, in1, &dk);
    const bool far = par.far();
    float2 carry = two(0.f);   // the gradient that reaches a token's state from behind it
    if (!PACKED && io.dhT) carry = load2(io.dhT + (size_t)b * g.D + c, in0, in1);
    const size_t kept = (g.T + kRun - 1) / kRun;
    auto kept_at = [&](int st) {   // the state that enters this lane's run
        const int t = token(st) + q;
        return st < steps && t < te ? load2(io.keep + ((size_t)b * kept + t / kRun) * g.D + c, in0, in1) : two(0.f);
    };
    float2 next = kept_at(0);
    float2 sq = two(0.f), sr = two(0.f), si = two(0.f);
    Edges edges = {0, 0};
    if (g.CL > 1) cluster_barrier();   // all of the cluster's blocks run before one writes to another

    for (int st = 0; st < steps; ++st) {
        const int tw = token(st), nw = min(R, te - tw), t = tw + q, n = max(0, min(kRun, te - t));
        uint32_t starts = 0, ends = 0;
        if (PACKED) edges.find(g, tw, nw, t, n, starts, ends);
        float2 h = next;
        next = kept_at(st + 1);
        ring.get(st, tw, nw, g.status);

        // the run's states, and of each token what dh is multiplied with
        float2 a[kRun], gy[kRun], fq[kRun], f1[kRun], fx[kRun], fi[kRun];
        auto states = [&](auto wide) {
#pragma unroll
            for (int k = 0; k < kRun; ++k) {
                const float2 r = gate(ring.at(st, kRg, k), par.rb), m = mul2(par.km, r);
                const float2 i = gate(ring.at(st, kIg, k), par.ib), u = mul2(i, ring.at(st, kX, k));
                float2 y, rs;
                decay_of<decltype(wide)::value>(m, a[k], y, rs);
                const float2 s = mul2(y, rs), su = mul2(s, u);
                if (PACKED && (starts >> k & 1))
                    h = g.h0 ? load2(g.h0 + (size_t)seq_at(g.cu, g.Nseq, t + k) * g.D + c, in0, in1) : two(0.f);
                // u a / s comes with m / s: m rs u a, which is 0 where m is
                fq[k] = mul2(mul2(m, a[k]), sub2(mul2(mul2(rs, u), a[k]), h));
                f1[k] = sub2(two(1.f), r);
                fx[k] = mul2(s, i);
                fi[k] = mul2(su, sub2(two(1.f), i));
                h = fma2(a[k], h, su);
                gy[k] = ring.at(st, kDy, k);
                if (gated) {
                    const float2 z = ring.at(st, kZ, k), p = sigmoid2(z);
                    // silu'(z) = p (1 + z (1 - p))
                    const float2 ds = mul2(p, fma2(z, sub2(two(1.f), p), two(1.f)));
                    ring.put(st, kZ, k, mul2(mul2(gy[k], h), ds));
                    gy[k] = mul2(gy[k], mul2(z, p));
                }
            }
        };
        if (far) states(std::true_type{});
        else states(std::false_type{});
        if (n < kRun) {   // behind the end: nothing changes
#pragma unroll
            for (int k = 0; k < kRun; ++k) {
                if (k >= n) {
                    a[k] = two(1.f);
                    gy[k] = fq[k] = fi[k] = two(0.f);
                }
            }
        }
        float2 A = two(1.f), H = two(0.f);
#pragma unroll
        for (int k = kRun - 1; k >= 0; --k) {
            if (PACKED && (ends >> k & 1))
                H = io.dhT ? load2(io.dhT + (size_t)seq_at(g.cu, g.Nseq, t + k) * g.D + c, in0, in1) : two(0.f);
            A = mul2(A, a[k]);
            H = mul2(a[k], add2(gy[k], H));
        }
        A = make_float2(fmaxf(A.x, kLeast), fmaxf(A.y, kLeast));
        if (PACKED && ends) A = two(-1.f);
        float2 back = exchange<W, Q, PACKED, true>(sm, st & 1, g.CL, rank, A, H, carry);
        if (st + S - 1 < steps) ring.ask(st + S - 1, token(st + S - 1), te - token(st + S - 1));
        ring.asked();
#pragma unroll
        for (int k = kRun - 1; k >= 0; --k) {
            if (PACKED && (ends >> k & 1))
                back = io.dhT ? load2(io.dhT + (size_t)seq_at(g.cu, g.Nseq, t + k) * g.D + c, in0, in1) : two(0.f);
            const float2 dh = add2(gy[k], back), q = mul2(dh, fq[k]), drg = mul2(q, f1[k]), dig = mul2(dh, fi[k]);
            back = mul2(a[k], dh);
            if (PACKED && (starts >> k & 1) && io.dh0)
                store2(io.dh0 + (size_t)seq_at(g.cu, g.Nseq, t + k) * g.D + c, back, in0, in1);
            ring.put(st, kX, k, mul2(dh, fx[k]));
            ring.put(st, kRg, k, drg);
            ring.put(st, kIg, k, dig);
            if (k < n) {
                sq = add2(sq, q);
                sr = add2(sr, drg);
                si = add2(si, dig);
            }
        }
        ring.flush(st, gated ? 15 : 7, tw, nw);
    }
    ring.end();
    if (!PACKED && io.dh0 && rank == 0 && warp == 0 && lane < L) store2(io.dh0 + (size_t)b * g.D + c, carry, in0, in1);

    auto put = [&](int i, float2 v) {   // the sum over a warp's runs, in a fixed order
#pragma unroll
        for (int d = L; d < 32; d *= 2) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, d);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, d);
        }
        if (lane < L) red[i][warp][lane] = v;
    };
    put(0, mul2(sq, dk));
    put(1, sr);
    put(2, si);
    __syncthreads();
    if (warp < 3 && lane < L) {
        float2 v = red[warp][0][lane];
#pragma unroll
        for (int w = 1; w < W; ++w) v = add2(v, red[warp][w][lane]);
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
    io.in[kX] = view_of<const T>(&f->x); io.in[kRg] = view_of<const T>(&f->rg); io.in[kIg] = view_of<const T>(&f->ig);
    io.in[kZ] = view_of<const T>(&f->z); io.in[kDy] = view_of<const T>(&r->dy);
    io.out[kX] = view_of<T>(&r->dx); io.out[kRg] = view_of<T>(&r->drg); io.out[kIg] = view_of<T>(&r->dig); io.out[kZ] = view_of<T>(&r->dz);
    io.keep = c.keep; io.dhT = r->dhT; io.dh0 = r->dh0; io.part = c.part;
    if (g.cu && io.dh0 && g.Nseq > 0) k_recur_empty_grad<<<g.Nseq, 256, 0, st>>>(g.cu, g.D, io.dhT, io.dh0);
    constexpr int W = bwd_warps(sizeof(T)), S = bwd_stages(sizeof(T));
    const bool gated = io.in[kZ].p != nullptr;
    const int smem = S * (gated ? 5 : 4) * W * kRun * 64 * (int)sizeof(T);
    RecurMaps m = {};
    const int mode = recur_mode(m, io, gated ? 31 : 23, gated ? 15 : 7, g);
    const cudaError_t rc = recur_variant<T>(g, mode, [&](auto q, auto how, auto packed) {
        return recur_launch(k_recur_bwd<T, decltype(q)::value, decltype(how)::value, decltype(packed)::value>, g, 32 * W, smem, st, m, g, io);
    });
    if (rc != cudaSuccess) return rc;
    const ColSum s = {c.part, (long long)g.B * g.CL, g.D, 3, {r->dlam, r->drg_bias, r->dig_bias}, {1, 1, 1}};
    return col_sum(s, nullptr, st);
}

}  // namespace

cudaError_t recur_bwd(const RecurCall &c, cudaStream_t st) { return c.s->dtype == DN_F32 ? bwd<float>(c, st) : bwd<__nv_bfloat16>(c, st); }

}  // namespace lay
}  // namespace gdn

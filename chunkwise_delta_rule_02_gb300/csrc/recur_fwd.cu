// Gated linear recurrence: forward over tokens, and the single-token step.
//
// k_recur_fwd.  Per step every thread turns its kRun tokens of two channels into decays and
// inputs, composes their map, gets what enters the run from the exchange (recur.cuh), and
// steps through it.
#include "recur.cuh"

namespace gdn {
namespace lay {

namespace {

template <class T, int Q, int MODE, bool PACKED>
__global__ void __launch_bounds__(32 * fwd_warps(sizeof(T))) k_recur_fwd(const __grid_constant__ RecurMaps maps, RecurDims g, RecurIo<T> io)
{
    constexpr int W = fwd_warps(sizeof(T)), S = fwd_stages(sizeof(T)), L = 32 / Q, R = kRun * Q;
    extern __shared__ __align__(128) char raw[];
    __shared__ RecurShared<W, Q> sm;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = g.CL > 1 ? cluster_rank() : 0;
    const int id = blockIdx.x / g.CL, b = id / g.tiles, c0 = (id - b * g.tiles) * (64 / Q), c = c0 + 2 * (lane % L), q = lane / L * kRun;
    const bool in0 = c < g.D, in1 = c + 1 < g.D;
    const bool gated = io.in[kZ].p != nullptr;
    Ring<T, W, Q, S, MODE> ring;
    ring.init(raw, sm.bar[warp], &io, &maps, gated ? 15 : 7, b, c0, g.D);
    const int te = PACKED ? g.cu[g.Nseq] : g.T;   // malformed offsets: every sequence is empty
    const int span = W * R * g.CL, steps = (te + span - 1) / span;
    const int first = (rank * W + warp) * R;      // of the warp's tokens, in a step's span
    for (int st = 0; st < S - 1; ++st) {
        if (st < steps) ring.ask(st, st * span + first, te - st * span - first);
        ring.asked();
    }
    RecurParams par;
    par.load(g, c, in0, in1);
    const bool far = par.far();
    float2 carry = two(0.f);
    if (!PACKED && g.h0) carry = load2(g.h0 + (size_t)b * g.D + c, in0, in1);
    const size_t kept = (g.T + kRun - 1) / kRun;
    Edges edges = {0, 0};
    if (g.CL > 1) cluster_barrier();   // all of the cluster's blocks run before one writes to another

    for (int st = 0; st < steps; ++st) {
        const int tw = st * span + first, nw = min(R, te - tw), t = tw + q, n = max(0, min(kRun, te - t));
        uint32_t starts = 0, ends = 0;
        if (PACKED) edges.find(g, tw, nw, t, n, starts, ends);
        ring.get(st, tw, nw, g.status);
        float2 a[kRun], in[kRun], A = two(1.f), H = two(0.f);
        auto decays = [&](auto wide) {
#pragma unroll
            for (int k = 0; k < kRun; ++k) {
                const float2 m = mul2(par.km, gate(ring.at(st, kRg, k), par.rb));
                const float2 u = mul2(gate(ring.at(st, kIg, k), par.ib), ring.at(st, kX, k));
                float2 y, rs;
                decay_of<decltype(wide)::value>(m, a[k], y, rs);
                in[k] = mul2(mul2(y, rs), u);
            }
        };
        if (far) decays(std::true_type{});
        else decays(std::false_type{});
        if (n < kRun) {   // behind the end: nothing changes
#pragma unroll
            for (int k = 0; k < kRun; ++k) {
                if (k >= n) {
                    a[k] = two(1.f);
                    in[k] = two(0.f);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            if (PACKED && (starts >> k & 1)) {
                if (g.h0) in[k] = fma2(a[k], load2(g.h0 + (size_t)seq_at(g.cu, g.Nseq, t + k) * g.D + c, in0, in1), in[k]);
                H = in[k];
            } else {
                A = mul2(A, a[k]);
                H = fma2(a[k], H, in[k]);
            }
        }
        A = make_float2(fmaxf(A.x, kLeast), fmaxf(A.y, kLeast));
        if (PACKED && starts) A = two(-1.f);
        float2 h = exchange<W, Q, PACKED, false>(sm, st & 1, g.CL, rank, A, H, carry);
        if (st + S - 1 < steps) ring.ask(st + S - 1, tw + (S - 1) * span, te - tw - (S - 1) * span);
        ring.asked();
        if (io.keep && n > 0) store2(io.keep + ((size_t)b * kept + t / kRun) * g.D + c, h, in0, in1);
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            h = PACKED && (starts >> k & 1) ? in[k] : fma2(a[k], h, in[k]);
            if (PACKED && (ends >> k & 1) && io.hT) store2(io.hT + (size_t)seq_at(g.cu, g.Nseq, t + k) * g.D + c, h, in0, in1);
            float2 y = h;
            if (gated) {
                const float2 z = ring.at(st, kZ, k);
                y = mul2(h, mul2(z, sigmoid2(z)));
            }
            ring.put(st, kX, k, y);
        }
        ring.flush(st, 1 << kX, tw, nw);
    }
    if (!PACKED && io.hT && rank == 0 && warp == 0 && lane < L) store2(io.hT + (size_t)b * g.D + c, carry, in0, in1);
    ring.end();
}

// Final states of empty sequences: the initial ones.
__global__ void __launch_bounds__(256) k_recur_empty(const int32_t *cu, int D, const float *from, float *to)
{
    const int s = blockIdx.x;
    if (cu[s] != cu[s + 1]) return;
    for (int c = threadIdx.x; c < D; c += 256) to[(size_t)s * D + c] = from ? from[(size_t)s * D + c] : 0.f;
}

// Two neighbouring channels of a token, WIDE: one access, both channels exist.
template <class T, bool WIDE>
__device__ __forceinline__ float2 get_two(const T *p, bool in1)
{
    float f[2] = {0.f, 0.f};
    if constexpr (WIDE) {
        Vec<T, 2> v;
        v.load(p);
        v.get(f);
    } else {
        f[0] = ld_in(p);
        if (in1) f[1] = ld_in(p + 1);
    }
    return make_float2(f[0], f[1]);
}

// One token for each of B sequences.
template <class T, bool WIDE>
__global__ void __launch_bounds__(256) k_recur_step(RecurDims g, RecurIo<T> io, int pairs, long long all)
{
    const long long q = blockIdx.x * 256ll + threadIdx.x;
    if (q >= all) return;
    const int b = (int)(q / pairs), c = (int)(q - (long long)b * pairs) * 2;
    const bool in0 = true, in1 = c + 1 < g.D;
    const float2 x = get_two<T, WIDE>(io.in[kX].at(b, 0, 0) + c, in1), r = get_two<T, WIDE>(io.in[kRg].at(b, 0, 0) + c, in1);
    const float2 i = get_two<T, WIDE>(io.in[kIg].at(b, 0, 0) + c, in1);
    const float2 z = io.in[kZ].p ? get_two<T, WIDE>(io.in[kZ].at(b, 0, 0) + c, in1) : two(0.f);
    float2 h = g.h0 ? load2(g.h0 + (size_t)b * g.D + c, in0, in1) : two(0.f);
    RecurParams par;
    par.load(g, c, in0, in1);
    float2 a, y, rs;
    decay_of<true>(mul2(par.km, gate(r, par.rb)), a, y, rs);
    h = fma2(a, h, mul2(mul2(y, rs), mul2(gate(i, par.ib), x)));
    if (io.hT) store2(io.hT + (size_t)b * g.D + c, h, in0, in1);
    if (io.in[kZ].p) h = mul2(h, mul2(z, sigmoid2(z)));
    T *p = io.out[kX].at(b, 0, 0) + c;
    if constexpr (WIDE) {
        Vec<T, 2> v;
        const float f[2] = {h.x, h.y};
        v.set(f);
        v.store(p);
    } else {
        st_out(p, h.x);
        if (in1) st_out(p + 1, h.y);
    }
}

template <class T>
RecurIo<T> fwd_io(const RecurCall &c)
{
    RecurIo<T> r = {};
    r.in[kX] = view_of<const T>(&c.io->x); r.in[kRg] = view_of<const T>(&c.io->rg); r.in[kIg] = view_of<const T>(&c.io->ig);
    r.in[kZ] = view_of<const T>(&c.io->z); r.out[kX] = view_of<T>(&c.io->y);
    r.hT = c.io->hT;
    r.keep = c.keep;
    return r;
}

template <class T>
cudaError_t fwd(const RecurCall &c, cudaStream_t st)
{
    constexpr int W = fwd_warps(sizeof(T)), S = fwd_stages(sizeof(T));
    const RecurDims g = recur_dims(c, false);
    const RecurIo<T> io = fwd_io<T>(c);
    if (g.cu && io.hT && g.Nseq > 0) k_recur_empty<<<g.Nseq, 256, 0, st>>>(g.cu, g.D, g.h0, io.hT);
    const int sets = io.in[kZ].p ? 15 : 7, smem = S * (io.in[kZ].p ? 4 : 3) * W * kRun * 64 * (int)sizeof(T);
    RecurMaps m = {};
    const int mode = recur_mode(m, io, sets, 1 << kX, g);
    return recur_variant<T>(g, mode, [&](auto q, auto how, auto packed) {
        return recur_launch(k_recur_fwd<T, decltype(q)::value, decltype(how)::value, decltype(packed)::value>, g, 32 * W, smem, st, m, g, io);
    });
}

template <class T>
cudaError_t step(const RecurCall &c, cudaStream_t st)
{
    const RecurDims g = recur_dims(c, false);
    const RecurIo<T> io = fwd_io<T>(c);
    const int pairs = (g.D + 1) / 2;
    const long long all = (long long)g.B * pairs;
    const unsigned blocks = (unsigned)((all + 255) / 256);
    const int e = sizeof(T);
    const bool wide = c.s->D % 2 == 0 && can_vector(&c.io->x, e, 2 * e) && can_vector(&c.io->rg, e, 2 * e) && can_vector(&c.io->ig, e, 2 * e) &&
                      can_vector(&c.io->z, e, 2 * e) && can_vector(&c.io->y, e, 2 * e);
    if (wide) k_recur_step<T, true><<<blocks, 256, 0, st>>>(g, io, pairs, all);
    else k_recur_step<T, false><<<blocks, 256, 0, st>>>(g, io, pairs, all);
    return cudaPeekAtLastError();
}

}  // namespace

// Blocks that share a row's tokens: as many as run at once, and no more than there are spans.  Where 64-channel tiles leave
// three quarters of the places free all the same, tiles of 16.
RecurPlan recur_plan(const dn_recur_shape *s, bool bwd)
{
    const int e = s->dtype == DN_F32 ? 4 : 2, run = kRun * (bwd ? bwd_warps(e) : fwd_warps(e));
    const long long most = (long long)kResident * sm_count();
    RecurPlan p = {1, 1};
    for (p.Q = 1;; p.Q = 4) {
        const long long tiles = (long long)s->B * ((s->D + 64 / p.Q - 1) / (64 / p.Q));
        for (p.CL = 1; p.CL < kMaxCluster && tiles * p.CL * 2 <= most && (long long)p.CL * run * p.Q < s->T;) p.CL *= 2;
        if (p.Q > 1 || tiles * p.CL * 4 > most || s->D <= 16) return p;
    }
}

cudaError_t recur_fwd(const RecurCall &c, cudaStream_t st) { return c.s->dtype == DN_F32 ? fwd<float>(c, st) : fwd<__nv_bfloat16>(c, st); }
cudaError_t recur_step(const RecurCall &c, cudaStream_t st) { return c.s->dtype == DN_F32 ? step<float>(c, st) : step<__nv_bfloat16>(c, st); }

}  // namespace lay
}  // namespace gdn

// Gated linear recurrence: forward over tokens, and the single-token step.
//
// k_recur_fwd.  Per step of kSpan tokens a block has, every thread turns its kRun tokens of
// two channels into decays and inputs, composes their map, gets what enters the run from
// the exchange (recur.cuh), and steps through it.
#include <algorithm>

#include "recur.cuh"

namespace gdn {
namespace lay {

namespace {

template <class T, bool WIDE, bool PACKED>
__global__ void __launch_bounds__(kRecurThreads) k_recur_fwd(RecurDims g, RecurIo<T> io)
{
    __shared__ RecurShared sm;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = g.CL > 1 ? cluster_rank() : 0;
    const int id = blockIdx.x / g.CL, b = id / g.tiles, c = (id - b * g.tiles) * kChans + 2 * lane;
    const bool in0 = c < g.D, in1 = c + 1 < g.D;
    const int cc = in0 ? c : 0;
    const bool gated = io.z.p != nullptr;
    RecurParams par;
    par.load(g, c, in0, in1);
    const int te = PACKED ? g.cu[g.Nseq] : g.T;   // malformed offsets: every sequence is empty
    float2 carry = two(0.f);
    if (!PACKED && g.h0) carry = load2(g.h0 + (size_t)b * g.D + c, in0, in1);
    const int span = kSpan * g.CL, steps = (te + span - 1) / span;
    const size_t kept = (g.T + kRun - 1) / kRun;
    if (g.CL > 1) cluster_barrier();   // all of the cluster's blocks run before one writes to another

    for (int st = 0; st < steps; ++st) {
        const int t = st * span + rank * kSpan + warp * kRun, n = max(0, min(kRun, te - t));
        Two<T, WIDE> x[kRun], r[kRun], i[kRun], z[kRun];
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            const bool in = k < n;
            x[k].load(io.x.at(b, 0, in ? t + k : 0) + cc, in && in0, in && in1);
            r[k].load(io.rg.at(b, 0, in ? t + k : 0) + cc, in && in0, in && in1);
            i[k].load(io.ig.at(b, 0, in ? t + k : 0) + cc, in && in0, in && in1);
            if (gated) z[k].load(io.z.at(b, 0, in ? t + k : 0) + cc, in && in0, in && in1);
        }
        uint32_t starts = 0, ends = 0;
        int seq = 0;
        if (PACKED) run_edges(g, t, n, starts, ends, seq);
        float2 a[kRun], in[kRun], A = two(1.f), H = two(0.f);
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            const float2 m = mul2(par.km, sigmoid2(add2(r[k].get(), par.rb)));
            const float2 u = mul2(sigmoid2(add2(i[k].get(), par.ib)), x[k].get());
            float2 y, rs;
            decay_of(m, a[k], y, rs);
            in[k] = mul2(mul2(y, rs), u);
            if (k >= n) {   // behind the end: nothing changes
                a[k] = two(1.f);
                in[k] = two(0.f);
            }
            if (PACKED && (starts >> k & 1)) {
                const int s = __shfl_sync(0xffffffffu, seq, k);
                if (g.h0) in[k] = fma2(a[k], load2(g.h0 + (size_t)s * g.D + c, in0, in1), in[k]);
                A = two(-1.f);
                H = in[k];
            } else {
                A = mul2(A, a[k]);
                H = fma2(a[k], H, in[k]);
            }
        }
        float2 h = exchange(sm, st & 1, g.CL, rank, warp, A, H, carry);
        if (io.keep && n > 0) store2(io.keep + ((size_t)b * kept + t / kRun) * g.D + c, h, in0, in1);
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            h = PACKED && (starts >> k & 1) ? in[k] : fma2(a[k], h, in[k]);
            if (PACKED && (ends >> k & 1) && io.hT) store2(io.hT + (size_t)__shfl_sync(0xffffffffu, seq, k) * g.D + c, h, in0, in1);
            float2 y = h;
            if (gated) {
                const float2 zz = z[k].get();
                y = mul2(h, mul2(zz, sigmoid2(zz)));
            }
            if (k < n) put_two<T, WIDE>(io.y.at(b, 0, t + k) + cc, y, in0, in1);
        }
    }
    if (!PACKED && io.hT && rank == 0 && warp == 0) store2(io.hT + (size_t)b * g.D + c, carry, in0, in1);
}

// Final states of empty sequences: the initial ones.
__global__ void __launch_bounds__(256) k_recur_empty(const int32_t *cu, int D, const float *from, float *to)
{
    const int s = blockIdx.x;
    if (cu[s] != cu[s + 1]) return;
    for (int c = threadIdx.x; c < D; c += 256) to[(size_t)s * D + c] = from ? from[(size_t)s * D + c] : 0.f;
}

// One token for each of B sequences.
template <class T, bool WIDE>
__global__ void __launch_bounds__(256) k_recur_step(RecurDims g, RecurIo<T> io, int pairs, long long all)
{
    const long long q = blockIdx.x * 256ll + threadIdx.x;
    if (q >= all) return;
    const int b = (int)(q / pairs), c = (int)(q - (long long)b * pairs) * 2;
    const bool in0 = true, in1 = c + 1 < g.D;
    Two<T, WIDE> x, r, i, z;
    x.load(io.x.at(b, 0, 0) + c, in0, in1);
    r.load(io.rg.at(b, 0, 0) + c, in0, in1);
    i.load(io.ig.at(b, 0, 0) + c, in0, in1);
    if (io.z.p) z.load(io.z.at(b, 0, 0) + c, in0, in1);
    float2 h = g.h0 ? load2(g.h0 + (size_t)b * g.D + c, in0, in1) : two(0.f);
    RecurParams par;
    par.load(g, c, in0, in1);
    float2 a, y, rs;
    decay_of(mul2(par.km, sigmoid2(add2(r.get(), par.rb))), a, y, rs);
    h = fma2(a, h, mul2(mul2(y, rs), mul2(sigmoid2(add2(i.get(), par.ib)), x.get())));
    if (io.hT) store2(io.hT + (size_t)b * g.D + c, h, in0, in1);
    if (io.z.p) {
        const float2 zz = z.get();
        h = mul2(h, mul2(zz, sigmoid2(zz)));
    }
    put_two<T, WIDE>(io.y.at(b, 0, 0) + c, h, in0, in1);
}

template <class T>
RecurIo<T> fwd_io(const RecurCall &c)
{
    RecurIo<T> r = {};
    r.x = view_of<const T>(&c.io->x); r.rg = view_of<const T>(&c.io->rg); r.ig = view_of<const T>(&c.io->ig);
    r.z = view_of<const T>(&c.io->z); r.y = view_of<T>(&c.io->y);
    r.hT = c.io->hT;
    r.keep = c.keep;
    return r;
}

bool fwd_wide(const RecurCall &c)
{
    const int e = c.s->dtype == DN_F32 ? 4 : 2;
    return c.s->D % 2 == 0 && can_vector(&c.io->x, e, 2 * e) && can_vector(&c.io->rg, e, 2 * e) && can_vector(&c.io->ig, e, 2 * e) &&
           can_vector(&c.io->z, e, 2 * e) && can_vector(&c.io->y, e, 2 * e);
}

template <class T>
cudaError_t fwd(const RecurCall &c, cudaStream_t st)
{
    const RecurDims g = recur_dims(c, false);
    const RecurIo<T> io = fwd_io<T>(c);
    if (g.cu && io.hT && g.Nseq > 0) k_recur_empty<<<g.Nseq, 256, 0, st>>>(g.cu, g.D, g.h0, io.hT);
    const bool wide = fwd_wide(c);
    if (g.cu) return wide ? recur_launch(k_recur_fwd<T, true, true>, g, st, io) : recur_launch(k_recur_fwd<T, false, true>, g, st, io);
    return wide ? recur_launch(k_recur_fwd<T, true, false>, g, st, io) : recur_launch(k_recur_fwd<T, false, false>, g, st, io);
}

template <class T>
cudaError_t step(const RecurCall &c, cudaStream_t st)
{
    const RecurDims g = recur_dims(c, false);
    const RecurIo<T> io = fwd_io<T>(c);
    const int pairs = (g.D + 1) / 2;
    const long long all = (long long)g.B * pairs;
    const unsigned blocks = (unsigned)((all + 255) / 256);
    if (fwd_wide(c)) k_recur_step<T, true><<<blocks, 256, 0, st>>>(g, io, pairs, all);
    else k_recur_step<T, false><<<blocks, 256, 0, st>>>(g, io, pairs, all);
    return cudaPeekAtLastError();
}

}  // namespace

// Blocks that share a row's tokens: as many as leave two blocks an SM, and no more than there are spans.
int recur_cluster(const dn_recur_shape *s, bool)
{
    const long long tiles = (long long)s->B * ((s->D + kChans - 1) / kChans), most = 2ll * sm_count();
    int cl = 1;
    while (cl < kMaxCluster && tiles * cl * 2 <= most && (long long)cl * kSpan < s->T) cl *= 2;
    return cl;
}

cudaError_t recur_fwd(const RecurCall &c, cudaStream_t st) { return c.s->dtype == DN_F32 ? fwd<float>(c, st) : fwd<__nv_bfloat16>(c, st); }
cudaError_t recur_step(const RecurCall &c, cudaStream_t st) { return c.s->dtype == DN_F32 ? step<float>(c, st) : step<__nv_bfloat16>(c, st); }

}  // namespace lay
}  // namespace gdn

// Gated linear recurrence: forward over tokens, and the single-token step.
//
// k_recur_fwd.  Per step every thread turns its run's tokens of two channels into decays and
// inputs, composes their map, gets what enters the run from the exchange (recur.cuh), and
// steps through it.
//
// Bound by instruction issue: 43 instructions an element (three sigmoids, the series of the decay and the
// root are half of them) against 10 bytes of bf16 with the output gate.  8 x 4096 tokens of 2048 channels:
// 142 us, 4.8 TB/s of a copy's 6.7, 2.4 instructions a cycle and SM; 256 blocks on 152 SMs leave 15 % of
// the SMs' time empty.  4 x 8192 tokens: 143 us with the status word's clearing; one row of 16384 tokens, 1024 channels: 52 us, 11 steps of a
// barrier and an exchange each.
#include "recur.cuh"

namespace gdn {
namespace lay {

namespace {

template <class T, int Q, int MODE, bool PACKED>
__global__ void __launch_bounds__(32 * fwd_warps(sizeof(T), Q, MODE), kFwdResident) k_recur_fwd(const __grid_constant__ RecurMaps maps, RecurDims g, RecurIo<T> io)
{
    constexpr int W = fwd_warps(sizeof(T), Q, MODE), L = 32 / Q, R = kRun * Q;
    constexpr bool kShort = PACKED;   // one copy of each loop: these run fewer steps, and wait for instructions
    extern __shared__ __align__(128) char raw[];
    float4 *block = reinterpret_cast<float4 *>(raw);   // maps of the cluster's blocks, then the inputs
    __shared__ RecurShared<W, Q> sm;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, CL = Q < 4 ? 1 : g.CL;   // wider tiles are never shared
    const int rank = CL > 1 ? cluster_rank() : 0, id = blockIdx.x / CL, b = id / g.tiles, c0 = (id - b * g.tiles) * (64 / Q), c = c0 + 2 * (lane % L);
    const int q = warp * R + lane / L * kRun;     // of this lane's run, in a block's tokens
    const bool in0 = c < g.D, in1 = c + 1 < g.D;
    const bool gated = io.in[kZ].p != nullptr;
    Inputs<T, W, Q, MODE, false> inputs;
    inputs.init(raw + recur_block_bytes(CL, Q), sm.bar, &io, &maps, gated ? 15 : 7, b, c0, g.D);
    if (PACKED) wait_for_last();
    const int te = PACKED ? g.cu[g.Nseq] : g.T;   // malformed offsets: every sequence is empty
    const int span = W * R * CL, steps = (te + span - 1) / span;
    int t0 = rank * W * R;                        // the block's first token of a step
    for (int st = 0; st < 2; ++st) {
        if (st < steps) inputs.ask(st, t0 + st * span, te, g.short_in);
        inputs.asked();
    }
    RecurParams par;
    par.load(g, c, in0, in1);
    const bool far = par.far();
    float2 carry = two(0.f);
    if (!PACKED && g.h0) carry = load2(g.h0 + (size_t)b * g.D + c, in0, in1);
    if (warp == 0 && lane < L) sm.carry[0][lane] = carry;
    float *keep = io.keep ? io.keep + ((size_t)b * ((g.T + kRun - 1) / kRun) + (t0 + q) / kRun) * g.D + c : nullptr;
    T *py = io.out[kX].at(b, 0, t0 + q) + c;
    Edges edges;
    edges.init();
    int seq = 0;
    if (MODE == kTma) __syncthreads();   // the barriers exist
    if (CL > 1) cluster_barrier();     // all of the cluster's blocks run before one writes to another

    float2 h = carry;
    bool lost = false;
    for (int st = 0; st < steps; ++st, t0 += span) {
        const int t = t0 + q, n = te - t;   // tokens of the run that exist: 0 or less to kRun or more
        uint32_t starts = 0, ends = 0;
        if (PACKED) edges.find(g, t0 + warp * R, min(R, te - t0 - warp * R), t, min(kRun, n), starts, ends);
        inputs.get(st, g, par);
        float2 a[kRun], in[kRun], A = two(1.f), H = two(0.f);
        Vec<T, 2> z[kRun];
        const auto px = inputs.cells(st, kX, t), pr = inputs.cells(st, kRg, t), pi = inputs.cells(st, kIg, t), pz = inputs.cells(st, kZ, t);
        auto decays = [&](auto wide) {
#pragma unroll
            for (int k = 0; k < kRun; ++k) {
                const float2 m = mul2(par.km, gate(inputs.at(pr, k), par.rb));
                const float2 u = mul2(gate(inputs.at(pi, k), par.ib), inputs.at(px, k));
                float2 y, rs;
                decay_of<decltype(wide)::value>(m, a[k], y, rs);
                in[k] = mul2(mul2(y, rs), u);
            }
        };
        if (kShort || far) decays(std::true_type{});
        else decays(std::false_type{});
        if (gated) {
#pragma unroll
            for (int k = 0; k < kRun; ++k) z[k] = inputs.raw(pz, k);
        }
        if (n < kRun) {   // behind the end: nothing changes
#pragma unroll
            for (int k = 0; k < kRun; ++k) {
                if (k >= n) {
                    a[k] = two(1.f);
                    in[k] = two(0.f);
                }
            }
        }
        seq = edges.first;
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            if (PACKED && (starts >> k & 1)) {
                seq = edges.up(g.cu, seq, t + k);
                if (g.h0) in[k] = fma2(a[k], load2(g.h0 + (size_t)seq * g.D + c, in0, in1), in[k]);
                H = in[k];
            } else {
                A = mul2(A, a[k]);
                H = fma2(a[k], H, in[k]);
            }
        }
        A = make_float2(fmaxf(A.x, kLeast), fmaxf(A.y, kLeast));
        if (PACKED && starts) A = two(-1.f);
        h = exchange<W, Q, PACKED, false>(sm, block, st, CL, rank, A, H, carry, lost, g, [&] {
            if (st + 2 < steps) inputs.ask(st + 2, t0 + 2 * span, te, g.short_in);
            inputs.asked();
        });
        if (keep) {
            if (n > 0) store2(keep, h, in0, in1);
            keep += (size_t)(span / kRun) * g.D;
        }
        T *p = py;
        seq = edges.first;
        auto outputs = [&](auto whole) {
#pragma unroll
            for (int k = 0; k < kRun; ++k) {
                h = PACKED && (starts >> k & 1) ? in[k] : fma2(a[k], h, in[k]);
                if (PACKED && (ends >> k & 1) && io.hT) {
                    seq = edges.up(g.cu, seq, t + k);
                    store2(io.hT + (size_t)seq * g.D + c, h, in0, in1);
                }
                float2 y = h;
                if (gated) {
                    float f[2];
                    z[k].get(f);
                    const float2 zz = make_float2(f[0], f[1]);
                    y = mul2(h, mul2(zz, sigmoid2(zz)));
                }
                if (decltype(whole)::value || k < n) put_two<MODE>(p, y, in0, in1);
                p += io.out[kX].t;
            }
        };
        if (!kShort && n >= kRun) outputs(std::true_type{});
        else outputs(std::false_type{});
        py += span * io.out[kX].t;
        if (CL == 1) leave<W, Q, false>(sm, st & 1, h);
    }
    if (PACKED) pass_empty<W, L>(g, rank, CL, c, in0, in1, g.h0, io.hT);
    // what leaves the last run: a cluster's blocks all have it, a block alone its last warp
    if (!PACKED && io.hT) {
        if (CL > 1 || steps == 0) {
            if (rank == 0 && warp == 0 && lane < L) store2(io.hT + (size_t)b * g.D + c, carry, in0, in1);
        } else if (warp == W - 1 && lane >= 32 - L) {
            store2(io.hT + (size_t)b * g.D + c, h, in0, in1);
        }
    }
    inputs.drain(g.budget);
    if (CL > 1) leave_cluster(lost);
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
    constexpr int W = fwd_warps(sizeof(T), 1, kTma);
    const RecurDims g = recur_dims(c, false);
    const RecurIo<T> io = fwd_io<T>(c);
    const int arrays = io.in[kZ].p ? 4 : 3;
    RecurMaps m = {};
    const int mode = recur_mode(m, io, (1 << arrays) - 1, box_rows<W>(g.Q), g);
    return recur_variant(g, mode, [&](auto q, auto how, auto packed) {
        constexpr int Q = decltype(q)::value, M = decltype(how)::value, W = fwd_warps(sizeof(T), Q, M);
        const int smem = 2 * arrays * place_bytes(W, Q, M, sizeof(T)) + recur_block_bytes(g.CL, Q);
        return recur_launch(k_recur_fwd<T, Q, M, decltype(packed)::value>, g, 32 * W, smem, st, m, g, io);
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

// Narrower tiles as long as all blocks run at once, then blocks of a cluster that share a row's tokens, no more than there
// are spans: runs that share a warp exchange their maps more cheaply than blocks do.
RecurPlan recur_plan(const dn_recur_shape *s, bool bwd)
{
    const int e = s->dtype == DN_F32 ? 4 : 2, run = kRun * (bwd ? bwd_warps(e) : fwd_warps(e, 1, kTma));
    const long long most = (long long)(bwd ? kBwdResident : kFwdResident) * sm_count();
    auto tiles = [&](int Q) { return (long long)s->B * ((s->D + 64 / Q - 1) / (64 / Q)); };
    RecurPlan p = {1, 1};
    while (p.Q < 4 && tiles(2 * p.Q) <= most && (long long)run * p.Q < s->T) p.Q *= 2;
    if (p.Q == 4)
        while (p.CL < kMaxCluster && tiles(4) * p.CL * 2 <= most && (long long)p.CL * run * 4 < s->T) p.CL *= 2;
    return p;
}

cudaError_t recur_fwd(const RecurCall &c, cudaStream_t st) { return c.s->dtype == DN_F32 ? fwd<float>(c, st) : fwd<__nv_bfloat16>(c, st); }
cudaError_t recur_step(const RecurCall &c, cudaStream_t st) { return c.s->dtype == DN_F32 ? step<float>(c, st) : step<__nv_bfloat16>(c, st); }

}  // namespace lay
}  // namespace gdn

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
//
// Bound by latency at 12 warps an SM: six factors of 16 elements a thread are 96 of its 158 registers.  8 x 4096 tokens of
// 2048 channels, bf16 with output gate: 250 us, 18 bytes an element at 4.8 TB/s, 65 instructions an element at 1.9 a cycle and SM.
#include "recur.cuh"

namespace gdn {
namespace lay {

namespace {

template <class T, int Q, int MODE, bool PACKED>
__global__ void __launch_bounds__(32 * bwd_warps(sizeof(T)), kBwdResident) k_recur_bwd(const __grid_constant__ RecurMaps maps, RecurDims g, RecurIo<T> io)
{
    constexpr int W = bwd_warps(sizeof(T)), L = 32 / Q, R = kRun * Q;
    constexpr bool kShort = MODE != kTma || PACKED;   // one copy of each loop: these run fewer steps, and wait for instructions
    extern __shared__ __align__(128) char raw[];
    float4 *block = reinterpret_cast<float4 *>(raw);   // maps of the cluster's blocks, then the inputs
    __shared__ RecurShared<W, Q> sm;
    __shared__ float2 red[3][W][L];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, CL = Q < 4 ? 1 : g.CL;   // wider tiles are never shared
    const int rank = CL > 1 ? cluster_rank() : 0, id = blockIdx.x / CL, b = id / g.tiles, c0 = (id - b * g.tiles) * (64 / Q), c = c0 + 2 * (lane % L);
    const int q = warp * R + lane / L * kRun;     // of this lane's run, in a block's tokens
    const bool in0 = c < g.D, in1 = c + 1 < g.D;
    const bool gated = io.in[kZ].p != nullptr;
    Inputs<T, W, Q, MODE, true> inputs;
    inputs.init(raw + recur_block_bytes(CL, Q), sm.bar, &io, &maps, gated ? 31 : 23, b, c0, g.D);
    if (PACKED) wait_for_last();
    const int te = PACKED ? g.cu[g.Nseq] : g.T;
    const int span = W * R * CL, steps = (te + span - 1) / span;
    int t0 = (steps - 1) * span + rank * W * R;   // the block's first token of a step; step st handles the st-th span from the end
    const float *keep = io.keep + (size_t)b * ((g.T + kRun - 1) / kRun) * g.D + c;
    const int kept = ((q / kRun) * (64 / Q) + 2 * (lane % L)) * 4;   // of this lane's run, among a step's
    auto ask = [&](int st, int first) {   // step st, the block's tokens from `first`
        inputs.ask(st, first, te, g.short_in);
        if (MODE == kChunks) {
            const int t = first + q;
            const float *from = keep + (t < te ? (size_t)(t / kRun) * g.D : 0);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool in = t < te && (i ? in1 : in0);
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(sm100::smem_u32(inputs.kept(st) + kept + 4 * i)),
                             "l"(in ? from + i : io.keep), "r"(in ? 4 : 0)
                             : "memory");
            }
        }
    };
    for (int st = 0; st < 2; ++st) {
        if (st < steps) ask(st, t0 - st * span);
        inputs.asked();
    }
    RecurParams par;
    float2 dk;
    par.load(g, c, in0, in1, &dk);
    const bool far = par.far();
    float2 carry = two(0.f);   // the gradient that reaches a token's state from behind it
    if (!PACKED && io.dhT) carry = load2(io.dhT + (size_t)b * g.D + c, in0, in1);
    if (warp == 0 && lane < L) sm.carry[0][lane] = carry;
    float2 sq = two(0.f), sr = two(0.f), si = two(0.f);
    Edges edges;
    edges.init();
    int seq = 0;
    if (MODE == kTma) __syncthreads();   // the barriers exist
    if (CL > 1) cluster_barrier();     // all of the cluster's blocks run before one writes to another

    float2 back = carry;
    bool lost = false;
    for (int st = 0; st < steps; ++st, t0 -= span) {
        const int t = t0 + q, n = te - t;   // tokens of the run that exist: 0 or less to kRun or more
        uint32_t starts = 0, ends = 0;
        if (PACKED) edges.find(g, t0 + warp * R, min(R, te - t0 - warp * R), t, min(kRun, n), starts, ends);
        inputs.get(st, g, par);
        // the state that enters the run, with the inputs (loaded a step ahead into registers it cost the waits of shared memory behind it:
        // 41 of 290 us for 8 x 4096 tokens of 2048 channels)
        float2 h = *reinterpret_cast<const float2 *>(inputs.kept(st) + kept);

        // the run's states, and of each token what dh is multiplied with
        float2 a[kRun], gy[kRun], fq[kRun], f1[kRun], fx[kRun], fi[kRun];
        const auto px = inputs.cells(st, kX, t), pr = inputs.cells(st, kRg, t), pi = inputs.cells(st, kIg, t), pz = inputs.cells(st, kZ, t);
        const auto pd = inputs.cells(st, kDy, t);
        const bool whole = n >= kRun;
        seq = edges.first;
        auto states = [&](auto wide) {
            T *p = gated ? io.out[kZ].at(b, 0, t) + c : nullptr;
#pragma unroll
            for (int k = 0; k < kRun; ++k) {
                const float2 r = gate(inputs.at(pr, k), par.rb), m = mul2(par.km, r);
                const float2 i = gate(inputs.at(pi, k), par.ib), u = mul2(i, inputs.at(px, k));
                float2 y, rs;
                decay_of<decltype(wide)::value>(m, a[k], y, rs);
                const float2 s = mul2(y, rs), su = mul2(s, u);
                if (PACKED && (starts >> k & 1)) {
                    seq = edges.up(g.cu, seq, t + k);
                    h = g.h0 ? load2(g.h0 + (size_t)seq * g.D + c, in0, in1) : two(0.f);
                }
                // u a / s comes with m / s: m rs u a, which is 0 where m is
                fq[k] = mul2(mul2(m, a[k]), sub2(mul2(mul2(rs, u), a[k]), h));
                f1[k] = sub2(two(1.f), r);
                fx[k] = mul2(s, i);
                fi[k] = mul2(su, sub2(two(1.f), i));
                h = fma2(a[k], h, su);
                gy[k] = inputs.at(pd, k);
                if (gated) {
                    const float2 z = inputs.at(pz, k), pp = sigmoid2(z);
                    // silu'(z) = p (1 + z (1 - p))
                    const float2 ds = mul2(pp, fma2(z, sub2(two(1.f), pp), two(1.f)));
                    if (whole || k < n) put_two<MODE>(p, mul2(mul2(gy[k], h), ds), in0, in1);
                    p += io.out[kZ].t;
                    gy[k] = mul2(gy[k], mul2(z, pp));
                }
            }
        };
        if (kShort || far) states(std::true_type{});
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
        seq = edges.last;
#pragma unroll
        for (int k = kRun - 1; k >= 0; --k) {
            if (PACKED && (ends >> k & 1)) {
                seq = edges.down(g.cu, seq, t + k);
                H = io.dhT ? load2(io.dhT + (size_t)seq * g.D + c, in0, in1) : two(0.f);
            }
            A = mul2(A, a[k]);
            H = mul2(a[k], add2(gy[k], H));
        }
        A = make_float2(fmaxf(A.x, kLeast), fmaxf(A.y, kLeast));
        if (PACKED && ends) A = two(-1.f);
        back = exchange<W, Q, PACKED, true>(sm, block, st, CL, rank, A, H, carry, lost, g, [&] {
            if (st + 2 < steps) ask(st + 2, t0 - 2 * span);
            inputs.asked();
        });
        T *pdx = io.out[kX].at(b, 0, t + kRun - 1) + c, *pdr = io.out[kRg].at(b, 0, t + kRun - 1) + c, *pdi = io.out[kIg].at(b, 0, t + kRun - 1) + c;
        seq = edges.last;
        auto outputs = [&](auto all) {
#pragma unroll
            for (int k = kRun - 1; k >= 0; --k) {
                if (PACKED && (ends >> k & 1)) {
                    seq = edges.down(g.cu, seq, t + k);
                    back = io.dhT ? load2(io.dhT + (size_t)seq * g.D + c, in0, in1) : two(0.f);
                }
                const float2 dh = add2(gy[k], back), q = mul2(dh, fq[k]), drg = mul2(q, f1[k]), dig = mul2(dh, fi[k]);
                back = mul2(a[k], dh);
                if (PACKED && (starts >> k & 1) && io.dh0) {
                    seq = edges.down(g.cu, seq, t + k);
                    store2(io.dh0 + (size_t)seq * g.D + c, back, in0, in1);
                }
                if (decltype(all)::value || k < n) {
                    put_two<MODE>(pdx, mul2(dh, fx[k]), in0, in1);
                    put_two<MODE>(pdr, drg, in0, in1);
                    put_two<MODE>(pdi, dig, in0, in1);
                    sq = add2(sq, q);
                    sr = add2(sr, drg);
                    si = add2(si, dig);
                }
                pdx -= io.out[kX].t;
                pdr -= io.out[kRg].t;
                pdi -= io.out[kIg].t;
            }
        };
        if (!kShort && whole) outputs(std::true_type{});
        else outputs(std::false_type{});
        if (CL == 1) leave<W, Q, true>(sm, st & 1, back);
    }
    if (PACKED) pass_empty<W, L>(g, rank, CL, c, in0, in1, io.dhT, io.dh0);
    if (!PACKED && io.dh0) {
        if (CL > 1 || steps == 0) {
            if (rank == 0 && warp == 0 && lane < L) store2(io.dh0 + (size_t)b * g.D + c, carry, in0, in1);
        } else if (warp == 0 && lane < L) {
            store2(io.dh0 + (size_t)b * g.D + c, back, in0, in1);
        }
    }

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
        store2(io.part + (((size_t)b * CL + rank) * 3 + warp) * g.D + c, v, in0, in1);
    }
    inputs.drain(g.budget);
    if (CL > 1) leave_cluster(lost);
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
    constexpr int W = bwd_warps(sizeof(T));
    const bool gated = io.in[kZ].p != nullptr;
    RecurMaps m = {};
    const bool maps = g.T > 0 && tensor_map(&m.kept, true, c.keep, g.D, (g.T + kRun - 1) / kRun, g.B, g.D, (long long)((g.T + kRun - 1) / kRun) * g.D,
                                            64 / g.Q, W * g.Q, 0);
    const int mode = recur_mode(m, io, gated ? 31 : 23, box_rows<W>(g.Q), g, maps);
    const cudaError_t rc = recur_variant(g, mode, [&](auto q, auto how, auto packed) {
        constexpr int Q = decltype(q)::value, M = decltype(how)::value, W = bwd_warps(sizeof(T));
        const int smem = 2 * ((gated ? 5 : 4) * place_bytes(W, Q, M, sizeof(T)) + W * 64 * 4) + recur_block_bytes(g.CL, Q);
        return recur_launch(k_recur_bwd<T, Q, M, decltype(packed)::value>, g, 32 * W, smem, st, m, g, io);
    });
    if (rc != cudaSuccess) return rc;
    const ColSum s = {c.part, (long long)g.B * g.CL, g.D, 3, {r->dlam, r->drg_bias, r->dig_bias}, {1, 1, 1}};
    return col_sum(s, nullptr, st);
}

}  // namespace

cudaError_t recur_bwd(const RecurCall &c, cudaStream_t st) { return c.s->dtype == DN_F32 ? bwd<float>(c, st) : bwd<__nv_bfloat16>(c, st); }

}  // namespace lay
}  // namespace gdn

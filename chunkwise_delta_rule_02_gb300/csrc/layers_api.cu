// C ABI of the layer operators: argument checks, workspace layout, dispatch; and
// the two kernels they share (packed offsets, sums of partial results).
#include <string.h>

#include <atomic>

#include "layers.h"
#include "scan.cuh"

namespace gdn {
namespace lay {

namespace {

// One block: copies the offsets, or zeros if they are malformed; sets the status word.
__global__ void __launch_bounds__(256) k_offsets(const int32_t *cu, int N, int T, int32_t *out, uint32_t *status)
{
    int bad = 0;
    for (int i = threadIdx.x; i <= N; i += blockDim.x) {
        const int v = cu[i];
        if (i == 0 ? v != 0 : cu[i - 1] > v) bad = 1;
        if (i == N && v != T) bad = 1;
    }
    bad = __syncthreads_or(bad);
    for (int i = threadIdx.x; i <= N; i += blockDim.x) out[i] = bad ? 0 : cu[i];
    if (threadIdx.x == 0) *status = bad ? kStatusBadOffsets : kStatusOk;   // and clears what an earlier call left
}

// Columns of a block (one 32-byte sector of each row) and threads a column: each sums every
// kSumY-th row, then pairs of threads in a fixed tree.  8 x 16 threads for the convolution's
// 10240 columns of 16 rows: 7 us (8 x 64: 18 us; 32 x 32: 12 us); for the norm's 128 columns of
// 456 rows 8 x 64 is 0.7 us faster, the scan's training step 36 us slower.
constexpr int kSumX = 8, kSumY = 16;

__global__ void __launch_bounds__(kSumX *kSumY) k_col_sum(ColSum a, ColSum b, unsigned blocks_a)
{
    __shared__ float sm[kSumY][kSumX];
    const bool second = blockIdx.x >= blocks_a;
    // field by field: a reference to either would put the arguments into local memory
    const float *part = second ? b.part : a.part;
    const long long P = second ? b.P : a.P, C = second ? b.C : a.C, n = C * (second ? b.kinds : a.kinds);
    const long long col = (blockIdx.x - (second ? blocks_a : 0)) * (long long)kSumX + threadIdx.x;
    float v = 0.f;
    if (col < n) {
#pragma unroll 8
        for (long long p = threadIdx.y; p < P; p += kSumY) v += part[p * n + col];
    }
    sm[threadIdx.y][threadIdx.x] = v;
    for (int h = kSumY / 2; h > 0; h >>= 1) {
        __syncthreads();
        if (threadIdx.y < h) sm[threadIdx.y][threadIdx.x] += sm[threadIdx.y + h][threadIdx.x];
    }
    if (threadIdx.y == 0 && col < n) {
        const int k = (int)(col / C);
        float *dst = second ? b.dst[k] : a.dst[k];
        if (dst) dst[(col - k * C) * (second ? b.step[k] : a.step[k])] = sm[0][threadIdx.x];
    }
}

}  // namespace

cudaError_t check_offsets(const int32_t *cu, int N, int T, int32_t *out, uint32_t *status, cudaStream_t st)
{
    k_offsets<<<1, 256, 0, st>>>(cu, N, T, out, status);
    return cudaPeekAtLastError();
}

cudaError_t col_sum(const ColSum &a, const ColSum *b, cudaStream_t st)
{
    auto blocks = [](const ColSum &c) { return (unsigned)((c.C * c.kinds + kSumX - 1) / kSumX); };
    const unsigned na = blocks(a), nb = b ? blocks(*b) : 0;
    if (na + nb == 0) return cudaSuccess;
    k_col_sum<<<na + nb, dim3(kSumX, kSumY), 0, st>>>(a, b ? *b : a, na);
    return cudaPeekAtLastError();
}

int sm_count()
{
    // asked once a device: the answer does not change, and calls of a few microseconds ask several times
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 152;
    if (dev < kDevices && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 152;
    if (dev < kDevices) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

namespace {

bool aligned(const void *p, size_t n) { return ((uintptr_t)p % n) == 0; }
bool has(const dn_view *v) { return v && v->data; }
dn_status status_of(cudaError_t e) { return e == cudaSuccess ? DN_OK : DN_ERR_CUDA; }

constexpr int kMaxT = 1 << 30;   // token indices plus a tile stay in 32 bits

dn_status check_packed(const int32_t *cu, int B, int num_seqs)
{
    if (!cu) return DN_OK;
    if (B != 1 || num_seqs < 0 || num_seqs == INT32_MAX || !aligned(cu, 4)) return DN_ERR_INVALID_ARG;
    return DN_OK;
}

// ------------------------------------------------------------------ convolution
dn_status conv_shape_ok(const dn_conv_shape *s)
{
    if (!s || s->B < 1 || s->H < 1 || s->T < 0 || s->d < 1) return DN_ERR_INVALID_ARG;
    if (s->dtype != DN_F32 && s->dtype != DN_BF16) return DN_ERR_INVALID_ARG;
    if ((long long)s->H * s->d > (1 << 24) || s->T > kMaxT) return DN_ERR_UNSUPPORTED;
    if (s->width < 2 || s->width > 4) return DN_ERR_UNSUPPORTED;
    return check_packed(s->cu_seqlens, s->B, s->num_seqs);
}

struct ConvWs {
    size_t cu, part, total;
};

ConvWs conv_ws(const dn_conv_shape *s, bool bwd)
{
    ConvWs w;
    w.cu = 256;
    w.part = w.cu + (s->cu_seqlens ? align256(sizeof(int32_t) * ((size_t)s->num_seqs + 1)) : 0);
    w.total = w.part;
    if (bwd) w.total += align256(sizeof(float) * (size_t)conv_part_rows(s) * (s->width + 1) * s->H * s->d);
    return w;
}

dn_status conv_begin(ConvCall &c, const dn_conv_shape *s, bool bwd, void *ws, size_t ws_bytes, cudaStream_t st)
{
    const ConvWs l = conv_ws(s, bwd);
    if (!ws || !aligned(ws, 16) || ws_bytes < l.total) return DN_ERR_WORKSPACE;
    char *base = (char *)ws;
    c.s = s;
    c.N = s->cu_seqlens ? s->num_seqs : s->B;
    c.part = (float *)(base + l.part);
    if (s->cu_seqlens) {
        c.cu = (const int32_t *)(base + l.cu);
        return status_of(check_offsets(s->cu_seqlens, s->num_seqs, s->T, (int32_t *)(base + l.cu), (uint32_t *)ws, st));
    }
    return DN_OK;
}

// ------------------------------------------------------------------ norm
dn_status norm_shape_ok(const dn_norm_shape *s)
{
    if (!s || s->B < 1 || s->H < 1 || s->T < 0 || s->d < 1) return DN_ERR_INVALID_ARG;
    if (s->dtype != DN_F32 && s->dtype != DN_BF16) return DN_ERR_INVALID_ARG;
    if (!(s->eps >= 0.f)) return DN_ERR_INVALID_ARG;
    if (s->d > 16384) return DN_ERR_UNSUPPORTED;
    if ((double)s->B * s->H * s->T > 2147483647.0 || (s->w_per_head && s->H > 65535)) return DN_ERR_UNSUPPORTED;
    return DN_OK;
}

// ------------------------------------------------------------------ scan
constexpr int kMaxStates = 128;

dn_status scan_shape_ok(const dn_scan_shape *s)
{
    if (!s || s->B < 1 || s->T < 0 || s->D < 1 || s->N < 1 || s->G < 1 || s->D % s->G) return DN_ERR_INVALID_ARG;
    if (s->dtype != DN_F32 && s->dtype != DN_BF16) return DN_ERR_INVALID_ARG;
    if (s->N > kMaxStates || s->D > (1 << 24) || s->T > kMaxT) return DN_ERR_UNSUPPORTED;
    return check_packed(s->cu_seqlens, s->B, s->num_seqs);
}

size_t scan_offsets(const dn_scan_shape *s)
{
    return 256 + (s->cu_seqlens ? align256(sizeof(int32_t) * ((size_t)s->num_seqs + 1)) : 0);
}

size_t scan_saved(const dn_scan_shape *s)
{
    const size_t n = (size_t)s->B * ((s->T + keep_of(scan_padded(s->N)) - 1) / keep_of(scan_padded(s->N))) * s->D * scan_padded(s->N) * sizeof(float);
    return n ? n : 256;
}

dn_status scan_io_ok(const dn_scan_shape *s, const dn_scan_io *io, bool need_y)
{
    if (!io || !io->A) return DN_ERR_INVALID_ARG;
    const size_t e = s->dtype == DN_F32 ? 4 : 2;
    const float *params[] = {io->A, io->D, io->dt_bias, io->h0, io->hT};
    for (const float *p : params)
        if (!aligned(p, 4)) return DN_ERR_INVALID_ARG;
    if (s->T > 0 && (!io->x.data || !io->dt.data || !io->b.data || !io->c.data || (need_y && !io->y.data)))
        return DN_ERR_INVALID_ARG;
    const dn_view *views[] = {&io->x, &io->dt, &io->b, &io->c, &io->z, &io->y};
    for (const dn_view *v : views)
        if (v->data && !aligned(v->data, e)) return DN_ERR_INVALID_ARG;
    return DN_OK;
}

dn_status scan_begin(ScanCall &c, const dn_scan_shape *s, const dn_scan_io *io, size_t need, void *ws, size_t ws_bytes,
                     cudaStream_t st)
{
    const size_t head = scan_offsets(s);
    if (!ws || !aligned(ws, 16) || ws_bytes < head + need) return DN_ERR_WORKSPACE;
    memset(&c, 0, sizeof(c));
    c.s = s;
    c.io = io;
    c.Nseq = s->cu_seqlens ? s->num_seqs : s->B;
    c.ws = (char *)ws + head;
    if (s->cu_seqlens) {
        int32_t *cu = (int32_t *)((char *)ws + 256);
        c.cu = cu;
        return status_of(check_offsets(s->cu_seqlens, s->num_seqs, s->T, cu, (uint32_t *)ws, st));
    }
    return DN_OK;
}

}  // namespace
}  // namespace lay
}  // namespace gdn

using namespace gdn;
using namespace gdn::lay;

extern "C" {

size_t dn_conv_workspace_size(const dn_conv_shape *shape, int for_backward)
{
    return conv_shape_ok(shape) == DN_OK ? conv_ws(shape, for_backward != 0).total : 0;
}

dn_status dn_conv_fwd(const dn_conv_shape *shape, const dn_view *x, const float *w, const float *bias, const void *s0,
                      const dn_view *y, void *sT, void *ws, size_t ws_bytes, void *stream)
{
    dn_status rc = conv_shape_ok(shape);
    if (rc != DN_OK) return rc;
    const size_t e = shape->dtype == DN_F32 ? 4 : 2;
    if (!w || !aligned(w, 4) || !aligned(bias, 4) || !aligned(s0, e) || !aligned(sT, e)) return DN_ERR_INVALID_ARG;
    if (shape->T > 0 && (!has(x) || !has(y))) return DN_ERR_INVALID_ARG;
    if ((has(x) && !aligned(x->data, e)) || (has(y) && !aligned(y->data, e))) return DN_ERR_INVALID_ARG;
    ConvCall c;
    memset(&c, 0, sizeof(c));
    if ((rc = conv_begin(c, shape, false, ws, ws_bytes, (cudaStream_t)stream)) != DN_OK) return rc;
    c.x = x; c.y = y; c.w = w; c.bias = bias; c.s0 = s0; c.sT = sT;
    return status_of(conv_fwd(c, (cudaStream_t)stream));
}

dn_status dn_conv_bwd(const dn_conv_shape *shape, const dn_view *x, const float *w, const float *bias, const void *s0,
                      const dn_view *dy, const void *dsT, const dn_view *dx, float *dw, float *dbias, void *ds0,
                      void *ws, size_t ws_bytes, void *stream)
{
    dn_status rc = conv_shape_ok(shape);
    if (rc != DN_OK) return rc;
    const size_t e = shape->dtype == DN_F32 ? 4 : 2;
    if (!w || !dw || !aligned(w, 4) || !aligned(bias, 4) || !aligned(dw, 4) || !aligned(dbias, 4)) return DN_ERR_INVALID_ARG;
    if (!aligned(s0, e) || !aligned(dsT, e) || !aligned(ds0, e)) return DN_ERR_INVALID_ARG;
    if (shape->T > 0 && (!has(x) || !has(dy) || !has(dx))) return DN_ERR_INVALID_ARG;
    const dn_view *views[] = {x, dy, dx};
    for (const dn_view *v : views)
        if (has(v) && !aligned(v->data, e)) return DN_ERR_INVALID_ARG;
    ConvCall c;
    memset(&c, 0, sizeof(c));
    if ((rc = conv_begin(c, shape, true, ws, ws_bytes, (cudaStream_t)stream)) != DN_OK) return rc;
    c.x = x; c.dy = dy; c.dx = dx; c.w = w; c.bias = bias; c.s0 = s0; c.dsT = dsT; c.ds0 = ds0;
    c.dw = dw; c.dbias = dbias;
    return status_of(conv_bwd(c, (cudaStream_t)stream));
}

dn_status dn_conv_step(const dn_conv_shape *shape, const dn_view *x, const float *w, const float *bias,
                       const void *state_in, void *state_out, const dn_view *y, void *stream)
{
    dn_status rc = conv_shape_ok(shape);
    if (rc != DN_OK) return rc;
    const size_t e = shape->dtype == DN_F32 ? 4 : 2;
    if (shape->T != 1 || shape->cu_seqlens || !w || !has(x) || !has(y)) return DN_ERR_INVALID_ARG;
    if (!aligned(w, 4) || !aligned(bias, 4) || !aligned(state_in, e) || !aligned(state_out, e) || !aligned(x->data, e) ||
        !aligned(y->data, e))
        return DN_ERR_INVALID_ARG;
    ConvCall c;
    memset(&c, 0, sizeof(c));
    c.s = shape; c.N = shape->B;
    c.x = x; c.y = y; c.w = w; c.bias = bias; c.s0 = state_in; c.sT = state_out;
    return status_of(conv_step(c, (cudaStream_t)stream));
}

size_t dn_scan_workspace_size(const dn_scan_shape *shape, int for_backward)
{
    if (scan_shape_ok(shape) != DN_OK) return 0;
    return scan_offsets(shape) + (for_backward ? scan_bwd_bytes(shape) : scan_fwd_bytes(shape));
}

size_t dn_scan_saved_size(const dn_scan_shape *shape) { return scan_shape_ok(shape) == DN_OK ? scan_saved(shape) : 0; }

dn_status dn_scan_fwd(const dn_scan_shape *shape, const dn_scan_io *io, void *saved, size_t saved_bytes, void *ws,
                      size_t ws_bytes, void *stream)
{
    dn_status rc = scan_shape_ok(shape);
    if (rc != DN_OK) return rc;
    if ((rc = scan_io_ok(shape, io, true)) != DN_OK) return rc;
    if (saved && (!aligned(saved, 16) || saved_bytes < scan_saved(shape))) return DN_ERR_WORKSPACE;
    ScanCall c;
    if ((rc = scan_begin(c, shape, io, scan_fwd_bytes(shape), ws, ws_bytes, (cudaStream_t)stream)) != DN_OK) return rc;
    c.keep = (float *)saved;
    return status_of(scan_fwd(c, (cudaStream_t)stream));
}

dn_status dn_scan_bwd(const dn_scan_shape *shape, const dn_scan_io *io, const dn_scan_grads *grads, const void *saved,
                      size_t saved_bytes, void *ws, size_t ws_bytes, void *stream)
{
    dn_status rc = scan_shape_ok(shape);
    if (rc != DN_OK) return rc;
    if ((rc = scan_io_ok(shape, io, false)) != DN_OK) return rc;
    const size_t e = shape->dtype == DN_F32 ? 4 : 2;
    if (!grads || !grads->dA) return DN_ERR_INVALID_ARG;
    const float *params[] = {grads->dhT, grads->dA, grads->dD, grads->ddt_bias, grads->dh0};
    for (const float *p : params)
        if (!aligned(p, 4)) return DN_ERR_INVALID_ARG;
    if (shape->T > 0 && (!grads->dy.data || !grads->dx.data || !grads->ddt.data || !grads->db.data || !grads->dc.data ||
                         (io->z.data && !grads->dz.data)))
        return DN_ERR_INVALID_ARG;
    const dn_view *views[] = {&grads->dy, &grads->dx, &grads->ddt, &grads->db, &grads->dc, &grads->dz};
    for (const dn_view *v : views)
        if (v->data && !aligned(v->data, e)) return DN_ERR_INVALID_ARG;
    if (!saved || !aligned(saved, 16) || saved_bytes < scan_saved(shape)) return DN_ERR_WORKSPACE;
    ScanCall c;
    if ((rc = scan_begin(c, shape, io, scan_bwd_bytes(shape), ws, ws_bytes, (cudaStream_t)stream)) != DN_OK) return rc;
    c.gr = grads;
    c.keep = (float *)saved;
    return status_of(scan_bwd(c, (cudaStream_t)stream));
}

dn_status dn_scan_step(const dn_scan_shape *shape, const dn_scan_io *io, void *stream)
{
    dn_status rc = scan_shape_ok(shape);
    if (rc != DN_OK) return rc;
    if (shape->T != 1 || shape->cu_seqlens) return DN_ERR_INVALID_ARG;
    if ((rc = scan_io_ok(shape, io, true)) != DN_OK) return rc;
    ScanCall c;
    memset(&c, 0, sizeof(c));
    c.s = shape;
    c.io = io;
    c.Nseq = shape->B;
    return status_of(scan_step(c, (cudaStream_t)stream));
}

dn_status dn_norm_fwd(const dn_norm_shape *shape, const dn_view *x, const float *w, const dn_view *z,
                      const dn_view *residual, const float *res_scale, const dn_view *y, const dn_view *sum,
                      void *stream)
{
    dn_status rc = norm_shape_ok(shape);
    if (rc != DN_OK) return rc;
    const size_t e = shape->dtype == DN_F32 ? 4 : 2;
    if (!w || !aligned(w, 4) || !aligned(res_scale, 4)) return DN_ERR_INVALID_ARG;
    if ((has(sum) || res_scale) && !has(residual)) return DN_ERR_INVALID_ARG;
    if (shape->T == 0) return DN_OK;
    if (!has(x) || !has(y)) return DN_ERR_INVALID_ARG;
    const dn_view *views[] = {x, z, residual, y, sum};
    for (const dn_view *v : views)
        if (has(v) && !aligned(v->data, e)) return DN_ERR_INVALID_ARG;
    NormCall c;
    memset(&c, 0, sizeof(c));
    c.s = shape; c.x = x; c.z = z; c.residual = residual; c.res_scale = res_scale; c.y = y; c.sum = sum; c.w = w;
    return status_of(norm_fwd(c, (cudaStream_t)stream));
}

size_t dn_norm_workspace_size(const dn_norm_shape *shape)
{
    if (norm_shape_ok(shape) != DN_OK) return 0;
    return align256(2 * sizeof(float) * (size_t)norm_part_rows(shape) * shape->d);
}

dn_status dn_norm_bwd(const dn_norm_shape *shape, const dn_view *x, const float *w, const dn_view *z,
                      const float *res_scale, const dn_view *sum, const dn_view *dy, const dn_view *dsum,
                      const dn_view *dx, float *dw, const dn_view *dz, const dn_view *dresidual, float *dres_scale,
                      void *ws, size_t ws_bytes, void *stream)
{
    dn_status rc = norm_shape_ok(shape);
    if (rc != DN_OK) return rc;
    const size_t e = shape->dtype == DN_F32 ? 4 : 2;
    if (!w || !dw || !aligned(w, 4) || !aligned(dw, 4) || !aligned(res_scale, 4) || !aligned(dres_scale, 4))
        return DN_ERR_INVALID_ARG;
    const bool res = has(sum);
    if (!res && (res_scale || dres_scale || has(dsum) || has(dresidual))) return DN_ERR_INVALID_ARG;
    if (has(dz) && !has(z)) return DN_ERR_INVALID_ARG;
    if (shape->T > 0) {
        if (!has(dy) || (!has(dx) && !has(dresidual))) return DN_ERR_INVALID_ARG;
        if (!has(x) && (!res || dres_scale)) return DN_ERR_INVALID_ARG;
    }
    const dn_view *views[] = {x, z, sum, dy, dsum, dx, dz, dresidual};
    for (const dn_view *v : views)
        if (has(v) && !aligned(v->data, e)) return DN_ERR_INVALID_ARG;
    if (!ws || !aligned(ws, 16) || ws_bytes < dn_norm_workspace_size(shape)) return DN_ERR_WORKSPACE;
    NormCall c;
    memset(&c, 0, sizeof(c));
    c.s = shape; c.x = x; c.z = z; c.sum = sum; c.dy = dy; c.dsum = dsum; c.dx = dx; c.dz = dz; c.dresidual = dresidual;
    c.w = w; c.res_scale = res_scale; c.dw = dw; c.dres_scale = dres_scale; c.part = (float *)ws;
    if (shape->T == 0) {   // no rows: the sums are zero
        const size_t nw = (size_t)(shape->w_per_head ? shape->H : 1) * shape->d;
        if (cudaMemsetAsync(dw, 0, nw * 4, (cudaStream_t)stream) != cudaSuccess) return DN_ERR_CUDA;
        if (dres_scale && cudaMemsetAsync(dres_scale, 0, (size_t)shape->d * 4, (cudaStream_t)stream) != cudaSuccess)
            return DN_ERR_CUDA;
        return DN_OK;
    }
    return status_of(norm_bwd(c, (cudaStream_t)stream));
}

}  // extern "C"

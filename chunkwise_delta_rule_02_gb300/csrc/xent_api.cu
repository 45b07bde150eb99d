// C ABI of the linear softmax cross entropy: argument checks, workspace layout, dispatch.
#include <string.h>

#include "xent.h"

namespace gdn {
namespace xent {

namespace {

using lay::align256;

// Most bytes of a piece's logit gradients.  Every piece leaves a part of its last round of tiles idle, and the sums of dx are read and
// written once a piece; more than the L2 cache holds costs power, which is what the products are bound by: training step
// of 8192 tokens, 2048 features, 32768 entries with 64, 128, 256, 512 MB: 3.07, 2.81, 2.78, 2.84 ms.
constexpr long long kPieceBytes = 256ll << 20;

bool aligned(const void *p, size_t n) { return ((uintptr_t)p % n) == 0; }
bool has(const dn_view *v) { return v && v->data; }
dn_status status_of(cudaError_t e) { return e == cudaSuccess ? DN_OK : DN_ERR_CUDA; }

dn_status shape_ok(const dn_xent_shape *s)
{
    if (!s || s->B < 0 || s->T < 0 || s->K < 1 || s->V < 1) return DN_ERR_INVALID_ARG;
    if (s->dtype != DN_F32 && s->dtype != DN_BF16) return DN_ERR_INVALID_ARG;
    const double M = (double)s->B * s->T;
    // coordinates plus a tile in 32 bits, tiles in 31
    if (M > (1 << 30) || s->V > (1 << 30) || s->K > (1 << 24)) return DN_ERR_UNSUPPORTED;
    if ((M / 256 + 1) * (s->V / 256.0 + 1) > 2147483647.0 || (M / 256 + 1) * (s->K / 256.0 + 1) > 2147483647.0 ||
        (s->V / 256.0 + 1) * (s->K / 256.0 + 1) > 2147483647.0)
        return DN_ERR_UNSUPPORTED;
    return DN_OK;
}

// Rows as one bf16 matrix that a tensor map can read: of 16-byte aligned rows at one distance, and of whole 16 bytes, where a map's
// boxes are cut off (what lies behind a shorter row might be read)
bool direct(const dn_xent_shape *s, const dn_view *v, long long rows, long long per, long long &pitch)
{
    if (s->dtype != DN_BF16 || s->K % 8 || !aligned(v->data, 16)) return false;
    if (rows > per && (per > 1 ? v->batch != v->time * per : false)) return false;
    pitch = per > 1 || rows <= 1 ? v->time : v->batch;
    if (rows <= 1) pitch = (s->K + 7) / 8 * 8;
    return pitch >= s->K && pitch % 8 == 0 && pitch < (1ll << 38);
}

// Where everything lies in the workspace; fills `c`.  `base` null: the size only.
size_t layout(Call &c, const dn_xent_shape *s, const dn_view *x, const dn_view *w, bool bwd, char *base)
{
    memset(&c, 0, sizeof(c));
    c.s = s;
    c.x = x; c.w = w;
    c.M = s->B * s->T; c.K = s->K; c.V = s->V;
    c.planes = s->dtype == DN_F32 ? 3 : 1;
    size_t at = 256;
    auto take = [&](size_t bytes) -> char * {
        char *p = (char *)((uintptr_t)base + at);
        at += align256(bytes);
        return p;
    };
    c.status = (uint32_t *)base;
    const long long Kp = copy_pitch(c.K);
    auto operand = [&](Operand &o, bool &packed, const dn_view *v, long long rows, long long per) {
        packed = !v || !direct(s, v, rows, per, o.pitch);
        if (packed) {
            o.pitch = Kp;
            o.plane = rows * Kp;
            o.p = take((size_t)c.planes * rows * Kp * 2);
        } else {
            o.p = v->data;
        }
    };
    if (c.M == 0) return at;
    c.few = few_tokens(c.M, c.K, c.planes == 3);
    if (c.few) {
        const int blocks = few_blocks(c.M, c.K, c.V, bwd);
        if (bwd) {
            c.cut = (float *)take((size_t)blocks * c.M * c.K * 4);
        } else {
            c.row = (float *)take((size_t)c.M * 4);
            c.part = (float2 *)take((size_t)c.M * blocks * sizeof(float2));
        }
        return at;
    }
    // backward, x is copied in any case: with 0 for tokens without a target, so that what they hold does not get into dw
    operand(c.xo, c.pack_x, bwd ? nullptr : x, c.M, s->T);
    operand(c.wo, c.pack_w, w, c.V, c.V);
    if (!bwd) {
        c.row = (float *)take((size_t)c.M * 4);
        c.part = (float2 *)take((size_t)c.M * parts_of(c.M, c.V) * sizeof(float2));
    } else {
        long long n = kPieceBytes / (2ll * c.planes * c.M) / 256 * 256;
        const long long whole = (c.V + 255ll) / 256 * 256;
        if (n < 256) n = 256;
        if (n > whole) n = whole;
        c.piece = (int)n;
        c.d = take((size_t)c.planes * c.M * n * 2);
        if (n < c.V) c.acc = (float *)take((size_t)c.M * c.K * 4);
        // the last piece may be shorter, and cut otherwise
        size_t cut = 0;
        for (long long piece : {n, (c.V - 1) % n + 1}) {
            int dx, dw;
            cuts_of(c.M, c.K, (int)(piece < c.V ? piece : c.V), c.planes, dx, dw);
            const size_t room = (dx > 1 ? (size_t)dx * c.M * c.K : 0) + (dw > 1 ? (size_t)dw * piece * c.K : 0);
            if (room > cut) cut = room;
        }
        if (cut) c.cut = (float *)take(cut * 4);
        if (c.planes == 1 && c.K % 8) {
            c.dx_rows = take((size_t)c.M * Kp * 2);
            c.dw_rows = take((size_t)n * Kp * 2);
        }
    }
    return at;
}

dn_status views_ok(const dn_xent_shape *s, const dn_view *x, const dn_view *w)
{
    const size_t e = s->dtype == DN_F32 ? 4 : 2;
    if (!has(w) || !aligned(w->data, e)) return DN_ERR_INVALID_ARG;
    if (s->B > 0 && s->T > 0 && (!has(x) || !aligned(x->data, e))) return DN_ERR_INVALID_ARG;
    return DN_OK;
}

}  // namespace
}  // namespace xent
}  // namespace gdn

using namespace gdn;
using namespace gdn::xent;

extern "C" {

size_t dn_xent_workspace_size(const dn_xent_shape *shape, const dn_view *x, const dn_view *w, int for_backward)
{
    if (shape_ok(shape) != DN_OK || views_ok(shape, x, w) != DN_OK) return 0;
    Call c;
    return layout(c, shape, x, w, for_backward != 0, nullptr);
}

dn_status dn_xent_fwd(const dn_xent_shape *shape, const dn_view *x, const dn_view *w, const dn_view *targets, float *loss, float *lse,
                      void *ws, size_t ws_bytes, void *stream)
{
    dn_status rc = shape_ok(shape);
    if (rc != DN_OK) return rc;
    if ((rc = views_ok(shape, x, w)) != DN_OK) return rc;
    if (shape->B > 0 && shape->T > 0 &&
        (!has(targets) || !aligned(targets->data, 8) || !loss || !lse || !aligned(loss, 4) || !aligned(lse, 4)))
        return DN_ERR_INVALID_ARG;
    Call c;
    const size_t need = layout(c, shape, x, w, false, (char *)ws);
    if (!ws || !aligned(ws, 16) || ws_bytes < need) return DN_ERR_WORKSPACE;
    if (!lay::has_tensor_maps()) return DN_ERR_CUDA;
    c.targets = targets; c.loss = loss; c.lse = lse;
    return status_of(forward(c, (cudaStream_t)stream));
}

dn_status dn_xent_bwd(const dn_xent_shape *shape, const dn_view *x, const dn_view *w, const dn_view *targets, const float *lse,
                      const dn_view *dloss, const dn_view *dx, void *dw, void *ws, size_t ws_bytes, void *stream)
{
    dn_status rc = shape_ok(shape);
    if (rc != DN_OK) return rc;
    if ((rc = views_ok(shape, x, w)) != DN_OK) return rc;
    const size_t e = shape->dtype == DN_F32 ? 4 : 2;
    if (!dw || !aligned(dw, e)) return DN_ERR_INVALID_ARG;
    if (shape->B > 0 && shape->T > 0 &&
        (!has(targets) || !aligned(targets->data, 8) || !lse || !aligned(lse, 4) || !has(dloss) || !aligned(dloss->data, 4) || !has(dx) ||
         !aligned(dx->data, e)))
        return DN_ERR_INVALID_ARG;
    Call c;
    const size_t need = layout(c, shape, x, w, true, (char *)ws);
    if (!ws || !aligned(ws, 16) || ws_bytes < need) return DN_ERR_WORKSPACE;
    if (!lay::has_tensor_maps()) return DN_ERR_CUDA;
    c.targets = targets; c.lse = const_cast<float *>(lse); c.dloss = dloss; c.dx = dx; c.dw = dw;
    return status_of(backward(c, (cudaStream_t)stream));
}

}  // extern "C"

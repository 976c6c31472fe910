// layer_api.cpp -- C ABI of the layer operators (include/gdn_layer.h):
// host-side validation and launches.  Nothing here allocates device memory.
#include <math.h>

#include "gdn_layer.h"
#include "layer_check.hpp"
#include "layer_launch.hpp"

namespace {

using namespace layer_check;

int check_norm(const norm_problem* p) {
    if (!p || p->rows < 0 || p->D < 1 || !(p->eps >= 0.f) || !isfinite(p->eps) || !known(p->dtype))
        return GDR_ERR_INVALID;
    if (p->D > 8192 || p->rows > ((int64_t)1 << 40) / p->D) return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}
int check_act(const norm_problem* p) {
    return p->act == GDN_ACT_SILU || p->act == GDN_ACT_SIGMOID ? GDR_OK : GDR_ERR_INVALID;
}
int check_res(const norm_problem* p) {
    return p->res_dtype == p->dtype || p->res_dtype == GDR_F32 ? GDR_OK : GDR_ERR_INVALID;
}

layer::NormArgs norm_args(const norm_problem* p) {
    layer::NormArgs a{};
    a.rows = (long)p->rows; a.D = p->D; a.eps = p->eps;
    a.dtype = p->dtype; a.res_dtype = p->res_dtype; a.act = p->act;
    return a;
}

size_t norm_ws(const norm_problem* p) { return 4 * layer::norm_part_floats((long)p->rows, p->D); }

int check_dropout(const gdn_dropout* d, layer::Drop* out) {
    if (!d || !(d->p >= 0.0 && d->p <= 1.0) || ((uintptr_t)d->rng & 7)) return GDR_ERR_INVALID;
    const uint32_t t = (uint32_t)floor(d->p * 65536.0 + 0.5);
    *out = {d->seed, d->offset, d->rng, t, t < 65536 ? (float)(65536.0 / (65536.0 - t)) : 0.f};
    return GDR_OK;
}

// Both forms of the add norm; d NULL: no dropout.
int add_fwd(const norm_problem* p, const gdn_dropout* d, const layer::Drop& drop, const void* x, const void* res,
            const float* w, const float* scale, void* y, void* res_out, hipStream_t stream) {
    int st = check_norm(p);
    if (st != GDR_OK || (st = check_res(p)) != GDR_OK) return st;
    if (p->rows == 0) return GDR_OK;
    if (!x || !res || !w || !y || !res_out) return GDR_ERR_INVALID;
    const size_t es = size_of(p->dtype), rs = size_of(p->res_dtype), c = 4 * (size_t)p->D;
    const size_t n = (size_t)p->rows * p->D * es, m = (size_t)p->rows * p->D * rs;
    if (!buffers_ok({{x, n, es}, {res, m, rs}, {w, c, 4}, {scale, c, 4}, {drop.rng, 16, 8}},
                    {{{y, n, es}, 1}, {{res_out, m, rs}, 2}}))
        return GDR_ERR_INVALID;
    layer::NormArgs a = norm_args(p);
    a.x = x; a.res = res; a.w = w; a.scale = scale; a.y = y; a.res_out = res_out;
    a.dropped = d != nullptr; a.drop = drop;
    return status(layer::launch_add_norm_fwd(a, stream));
}
int add_bwd(const norm_problem* p, const gdn_dropout* d, const layer::Drop& drop, const void* dy, const void* dres,
            const void* res, const float* w, const void* x, const float* scale, void* dx, void* dres_out, float* dw,
            float* dscale, void* ws, size_t ws_bytes, hipStream_t stream) {
    int st = check_norm(p);
    if (st != GDR_OK || (st = check_res(p)) != GDR_OK) return st;
    if (!dw || !scale != !dscale) return GDR_ERR_INVALID;
    if (p->rows > 0 && (!dy || !res || !w || !dres_out || (scale && !x) || ((scale || d) && !dx))) return GDR_ERR_INVALID;
    const size_t es = size_of(p->dtype), rs = size_of(p->res_dtype), c = 4 * (size_t)p->D, need = norm_ws(p);
    const size_t n = (size_t)p->rows * p->D * es, m = (size_t)p->rows * p->D * rs;
    if ((st = check_ws(ws, ws_bytes, need)) != GDR_OK) return st;
    if (!buffers_ok({{dy, n, es}, {x, n, es}, {dres, m, rs}, {res, m, rs}, {w, c, 4}, {scale, c, 4}, {drop.rng, 16, 8}},
                    {{{dx, n, es}, 3}, {{dres_out, m, rs}, 12}, {{dw, c, 4}, 0}, {{dscale, c, 4}, 0},
                     {{ws, need, 16}, 0}}))
        return GDR_ERR_INVALID;
    layer::NormArgs a = norm_args(p);
    a.dy = dy; a.dres = dres; a.res = res; a.w = w; a.x = x; a.scale = scale; a.dx = dx; a.dres_out = dres_out;
    a.dw = dw; a.dscale = dscale; a.part = (float*)ws;
    a.dropped = d != nullptr; a.drop = drop;
    return status(layer::launch_add_norm_bwd(a, stream));
}

int check_glr(const glr_problem* p, layer::GlrArgs* a) {
    if (!p || p->B < 1 || p->T < 0 || p->D < 1 || !known(p->dtype)) return GDR_ERR_INVALID;
    int64_t n = (int64_t)p->B * p->T, nseq = p->B;
    if (p->cu_seqlens) {
        if (!p->cu_seqlens_host || p->B != 1 || p->N < 1 || p->cu_seqlens_host[0] != 0) return GDR_ERR_INVALID;
        for (int i = 0; i < p->N; i++)
            if (p->cu_seqlens_host[i + 1] < p->cu_seqlens_host[i]) return GDR_ERR_INVALID;
        if (p->cu_seqlens_host[p->N] != p->T) return GDR_ERR_INVALID;
        nseq = p->N;
    }
    if (n > (1 << 30) || p->D > (1 << 20)) return GDR_ERR_UNSUPPORTED;
    *a = layer::GlrArgs{};
    a->ntok = (long)n; a->nseq = (int)nseq; a->T = p->T; a->D = p->D; a->dtype = p->dtype; a->cu = p->cu_seqlens;
    a->polls = p->polls > 0 ? p->polls : 4096;
    // a launch has fewer than 2^32 threads: 4 a token (of whole segments of 192 or 128) and 128 channels
    if (layer::glr_threads(*a) >= (int64_t)1 << 32 || (n == 0 && nseq * p->D >= (int64_t)1 << 31))
        return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}

int64_t tiles(const layer::GlrArgs& a) { return (a.ntok + GLR_TILE - 1) / GLR_TILE; }

int check_step(int N, int64_t nslots, int dtype, const int32_t* slots) {
    if (N < 0 || nslots < 0 || !known(dtype)) return GDR_ERR_INVALID;
    if (!slots && N > nslots) return GDR_ERR_INVALID;
    return N > 65536 || nslots > INT32_MAX ? GDR_ERR_UNSUPPORTED : GDR_OK;
}

}  // namespace

extern "C" {

size_t norm_workspace_size(const norm_problem* p) { return check_norm(p) != GDR_OK ? 0 : norm_ws(p); }

int gated_norm_fwd(const norm_problem* p, const void* x, const void* z, const float* w, void* y, hipStream_t stream) {
    int st = check_norm(p);
    if (st != GDR_OK || (st = check_act(p)) != GDR_OK) return st;
    if (p->rows == 0) return GDR_OK;
    if (!x || !w || !y) return GDR_ERR_INVALID;
    const size_t es = size_of(p->dtype), n = (size_t)p->rows * p->D * es;
    if (!buffers_ok({{x, n, es}, {z, n, es}, {w, 4 * (size_t)p->D, 4}}, {{{y, n, es}, 3}})) return GDR_ERR_INVALID;
    layer::NormArgs a = norm_args(p);
    a.x = x; a.z = z; a.w = w; a.y = y;
    return status(layer::launch_gated_norm_fwd(a, stream));
}

int gated_norm_bwd(const norm_problem* p, const void* x, const void* z, const float* w, const void* dy, void* dx,
                   void* dz, float* dw, void* ws, size_t ws_bytes, hipStream_t stream) {
    int st = check_norm(p);
    if (st != GDR_OK || (st = check_act(p)) != GDR_OK) return st;
    if (!dw || (p->rows > 0 && (!x || !w || !dy || !dx || !z != !dz))) return GDR_ERR_INVALID;
    const size_t es = size_of(p->dtype), n = (size_t)p->rows * p->D * es, c = 4 * (size_t)p->D, need = norm_ws(p);
    if ((st = check_ws(ws, ws_bytes, need)) != GDR_OK) return st;
    if (!buffers_ok({{x, n, es}, {dy, n, es}, {z, n, es}, {w, c, 4}},
                    {{{dx, n, es}, 3}, {{dz, n, es}, 6}, {{dw, c, 4}, 0}, {{ws, need, 16}, 0}}))
        return GDR_ERR_INVALID;
    layer::NormArgs a = norm_args(p);
    a.x = x; a.z = z; a.w = w; a.dy = dy; a.dx = dx; a.dz = dz; a.dw = dw; a.part = (float*)ws;
    return status(layer::launch_gated_norm_bwd(a, stream));
}

int add_norm_fwd(const norm_problem* p, const void* x, const void* res, const float* w, const float* scale, void* y,
                 void* res_out, hipStream_t stream) {
    return add_fwd(p, nullptr, {}, x, res, w, scale, y, res_out, stream);
}

int add_norm_bwd(const norm_problem* p, const void* dy, const void* dres, const void* res, const float* w,
                 const void* x, const float* scale, void* dx, void* dres_out, float* dw, float* dscale, void* ws,
                 size_t ws_bytes, hipStream_t stream) {
    return add_bwd(p, nullptr, {}, dy, dres, res, w, x, scale, dx, dres_out, dw, dscale, ws, ws_bytes, stream);
}

int gdn_dropout_fwd(int64_t rows, int64_t D, gdr_dtype dtype, const gdn_dropout* d, const void* x, void* y,
                    hipStream_t stream) {
    layer::Drop drop;
    const int st = check_dropout(d, &drop);
    if (st != GDR_OK) return st;
    if (rows < 0 || D < 1 || !known(dtype)) return GDR_ERR_INVALID;
    if (D > (int64_t)1 << 40 || rows > ((int64_t)1 << 40) / D) return GDR_ERR_UNSUPPORTED;
    if (rows == 0) return GDR_OK;
    if (!x || !y) return GDR_ERR_INVALID;
    const size_t es = size_of(dtype), n = (size_t)rows * D * es;
    if (!buffers_ok({{x, n, es}, {drop.rng, 16, 8}}, {{{y, n, es}, 1}})) return GDR_ERR_INVALID;
    return status(layer::launch_dropout(dtype, x, y, rows, D, drop, stream));
}

int dropout_add_norm_fwd(const norm_problem* p, const gdn_dropout* d, const void* x, const void* res, const float* w,
                         const float* scale, void* y, void* res_out, hipStream_t stream) {
    layer::Drop drop;
    const int st = check_dropout(d, &drop);
    return st != GDR_OK ? st : add_fwd(p, d, drop, x, res, w, scale, y, res_out, stream);
}

int dropout_add_norm_bwd(const norm_problem* p, const gdn_dropout* d, const void* dy, const void* dres,
                         const void* res, const float* w, const void* x, const float* scale, void* dx, void* dres_out,
                         float* dw, float* dscale, void* ws, size_t ws_bytes, hipStream_t stream) {
    layer::Drop drop;
    const int st = check_dropout(d, &drop);
    return st != GDR_OK ? st
                        : add_bwd(p, d, drop, dy, dres, res, w, x, scale, dx, dres_out, dw, dscale, ws, ws_bytes, stream);
}

int64_t glr_num_states(const glr_problem* p) {
    layer::GlrArgs a;
    return check_glr(p, &a) != GDR_OK ? -1 : tiles(a);
}

size_t glr_workspace_size(const glr_problem* p) {
    layer::GlrArgs a;
    return check_glr(p, &a) != GDR_OK ? 0 : layer::glr_ws_bytes(a);
}

int glr_fwd(const glr_problem* p, const void* x, const float* g, const float* h0, void* h, float* ht, float* states,
            void* ws, size_t ws_bytes, hipStream_t stream) {
    layer::GlrArgs a;
    int st = check_glr(p, &a);
    if (st != GDR_OK) return st;
    if (a.ntok > 0 && (!x || !g || !h)) return GDR_ERR_INVALID;
    const size_t need = layer::glr_ws_bytes(a);
    if ((st = check_ws(ws, ws_bytes, need)) != GDR_OK) return st;
    const size_t es = size_of(a.dtype), n = (size_t)a.ntok * a.D, c = 4 * (size_t)a.nseq * a.D;
    if (!buffers_ok({{x, n * es, es}, {g, 4 * n, 4}, {h0, c, 4}, {a.cu, 4 * (size_t)(a.nseq + 1), 4}},
                    {{{h, n * es, es}, 0}, {{ht, c, 4}, 0}, {{states, 4 * (size_t)tiles(a) * a.D, 4}, 0},
                     {{ws, need, 16}, 0}}))
        return GDR_ERR_INVALID;
    a.x = x; a.g = g; a.h0 = h0; a.h = h; a.ht = ht; a.states = states; a.ws = ws;
    if (a.ntok == 0 && !ht) return GDR_OK;
    return status(layer::launch_glr_fwd(a, stream));
}

int glr_bwd(const glr_problem* p, const void* x, const float* g, const float* h0, const float* states, const void* dh,
            const float* dht, void* dx, float* dg, float* dh0, void* ws, size_t ws_bytes, hipStream_t stream) {
    layer::GlrArgs a;
    int st = check_glr(p, &a);
    if (st != GDR_OK) return st;
    if (a.ntok > 0 && (!x || !g || !states || !dh || !dx || !dg)) return GDR_ERR_INVALID;
    const size_t need = layer::glr_ws_bytes(a);
    if ((st = check_ws(ws, ws_bytes, need)) != GDR_OK) return st;
    const size_t es = size_of(a.dtype), n = (size_t)a.ntok * a.D, c = 4 * (size_t)a.nseq * a.D;
    if (!buffers_ok({{x, n * es, es}, {g, 4 * n, 4}, {h0, c, 4}, {states, 4 * (size_t)tiles(a) * a.D, 4},
                     {dh, n * es, es}, {dht, c, 4}, {a.cu, 4 * (size_t)(a.nseq + 1), 4}},
                    {{{dx, n * es, es}, 0}, {{dg, 4 * n, 4}, 0}, {{dh0, c, 4}, 0}, {{ws, need, 16}, 0}}))
        return GDR_ERR_INVALID;
    a.x = x; a.g = g; a.h0 = h0; a.states = (float*)states; a.dh = dh; a.dht = dht; a.dx = dx; a.dg = dg; a.dh0 = dh0;
    a.ws = ws;
    if (a.ntok == 0 && !dh0) return GDR_OK;
    return status(layer::launch_glr_bwd(a, stream));
}

int glr_step(int N, int D, int64_t nslots, gdr_dtype dtype, const void* x, const float* g, const int32_t* slots,
             float* state, void* h, hipStream_t stream) {
    int st = check_step(N, nslots, dtype, slots);
    if (st != GDR_OK) return st;
    if (D < 1) return GDR_ERR_INVALID;
    // a launch has fewer than 2^32 threads: 128 for every 512 channels of a row
    if (D > (1 << 20) || (int64_t)N * ((D + 511) / 512) >= 1 << 25) return GDR_ERR_UNSUPPORTED;
    if (N == 0) return GDR_OK;
    if (!x || !g || !h || (nslots > 0 && !state)) return GDR_ERR_INVALID;
    const size_t es = size_of(dtype), n = (size_t)N * D;
    if (!buffers_ok({{x, n * es, es}, {g, 4 * n, 4}, {slots, 4 * (size_t)N, 4}},
                    {{{h, n * es, es}, 1}, {{state, 4 * (size_t)nslots * D, 4}, 0}}))
        return GDR_ERR_INVALID;
    layer::StepArgs a{};
    a.N = N; a.D = D; a.nslots = (long)nslots; a.dtype = dtype;
    a.v = x; a.g = g; a.slots = slots; a.state = state; a.o = h;
    return status(layer::launch_glr_step(a, stream));
}

int gdr_step(int N, int HK, int HV, int K, int V, int64_t nslots, float scale, gdr_dtype dtype, const void* q,
             const void* k, const void* v, const float* g, const void* beta, const int32_t* slots, float* state,
             void* o, hipStream_t stream) {
    int st = check_step(N, nslots, dtype, slots);
    if (st != GDR_OK) return st;
    if (HK < 1 || HV < 1 || HV % HK != 0 || K < 1 || V < 1 || isnan(scale) || isinf(scale)) return GDR_ERR_INVALID;
    // a launch has fewer than 2^32 threads: 256 for every head where there are thousands of them
    if (K != V || (K != 64 && K != 128) || HV > 1024 || (int64_t)N * HV >= 1 << 24) return GDR_ERR_UNSUPPORTED;
    if (N == 0) return GDR_OK;
    if (!q || !k || !v || !g || !beta || !o || (nslots > 0 && !state)) return GDR_ERR_INVALID;
    const size_t es = size_of(dtype), nk = (size_t)N * HK * K * es, nv = (size_t)N * HV * V * es, nh = (size_t)N * HV;
    if (!buffers_ok({{v, nv, es}, {q, nk, es}, {k, nk, es}, {g, 4 * nh, 4}, {beta, nh * es, es},
                     {slots, 4 * (size_t)N, 4}},
                    {{{o, nv, es}, 1}, {{state, 4 * (size_t)nslots * HV * K * V, 4}, 0}}))
        return GDR_ERR_INVALID;
    layer::StepArgs a{};
    a.N = N; a.HK = HK; a.HV = HV; a.K = K; a.nslots = (long)nslots; a.dtype = dtype;
    a.scale = scale > 0.f ? scale : 1.0f / sqrtf((float)K);
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.slots = slots; a.state = state; a.o = o;
    return status(layer::launch_gdr_step(a, stream));
}

}  // extern "C"

// ffn_api.cpp -- C ABI of the gated feed-forward block (include/gdn_ffn.h):
// host-side validation, the workspace's layout and the launches.  Nothing here
// allocates device memory.
#include <limits.h>

#include <algorithm>

#include "ffn_launch.hpp"
#include "gdn_ffn.h"
#include "layer_check.hpp"

namespace {
using namespace layer_check;
using namespace ffn;

int check(const ffn_problem* p) {
    if (!p || p->T < 0 || p->D < 1 || p->F < 1 || !known(p->dtype)) return GDR_ERR_INVALID;
    if (p->act != GDN_FFN_SILU && p->act != GDN_FFN_SIGMOID && p->act != GDN_FFN_GELU) return GDR_ERR_INVALID;
    if (p->T > (1 << 24) || p->D > 65536 || p->F > 65536 || p->T * (p->D + 2LL * p->F) >= 1LL << 36)
        return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}

// Sizes as the products see them (rows padded to whole pieces of 16 bytes) and the
// workspace's parts, as offsets in bytes.
struct Plan {
    int T, D, F, e, piece;
    bool pad;
    size_t h, dgu, part, x, wg, wu, wd, dy, bytes;
    GradPlan grads;
};
Plan plan_of(const ffn_problem* p, bool bwd) {
    Plan l{};
    l.T = (int)p->T, l.e = (int)size_of(p->dtype), l.piece = 16 / l.e;
    l.D = (p->D + l.piece - 1) / l.piece * l.piece, l.F = (p->F + l.piece - 1) / l.piece * l.piece;
    l.pad = l.D != p->D || l.F != p->F;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) & ~(size_t)255;
        return o;
    };
    const size_t row = (size_t)l.T * l.F * l.e, xs = (size_t)l.T * l.D * l.e, ws = (size_t)l.D * l.F * l.e;
    size_t f = 0;
    auto most = [&](Kind k, int M, int N, int K) {
        const size_t n = part_floats(k, M, N, K, l.e);
        if (n > f) f = n;
    };
    if (bwd) {
        l.dgu = take(2 * row);
        most(DH, l.T, l.F, l.D);
        l.grads = grad_plan(l.T, l.D, l.F, l.e);
        f = std::max(f, grad_floats(l.grads, l.T, l.D, l.F));
    } else {
        l.h = take(row);   // not used by a call that keeps it
        most(GATE_UP, l.T, l.F, l.D);
        most(DOWN, l.T, l.D, l.F);
    }
    l.part = take(4 * f);
    if (l.pad && l.T > 0) {
        l.x = take(xs), l.wg = take(ws), l.wu = take(ws), l.wd = take(ws);
        if (bwd) l.dy = take(xs);
    }
    l.bytes = at;
    return l;
}

// Kept for the backward: gate and up [T][2 F] fp32, behind them h [T][F].
int64_t saved_width(const Plan& l) { return 2 * (int64_t)l.F + (int64_t)l.F * l.e / 4; }
size_t saved_bytes(const Plan& l) { return 4 * (size_t)l.T * saved_width(l); }
char* saved_h(const Plan& l, const float* saved) { return (char*)saved + 8 * (size_t)l.T * l.F; }

// Copies src into padded rows (and `rows_dst` of them) at dst, where it then is; not if its rows are as they have to be.
void pad(PadArgs& a, const void*& src, void* dst, int64_t rows, int64_t rows_dst, int cols, int cols_dst) {
    if (rows == rows_dst && cols == cols_dst && ((uintptr_t)src & 15) == 0) return;
    a.item[a.n++] = {src, dst, rows, rows_dst, cols, cols_dst};
    src = dst;
}

}  // namespace

extern "C" {

size_t ffn_workspace_size(const ffn_problem* p, int bwd) { return check(p) != GDR_OK ? 0 : plan_of(p, bwd != 0).bytes; }

int64_t ffn_saved_width(const ffn_problem* p) { return check(p) != GDR_OK ? -1 : saved_width(plan_of(p, false)); }

int gated_ffn_fwd(const ffn_problem* p, const void* x, const void* w_gate, const void* w_up, const void* w_down,
                  void* y, float* saved, void* ws, size_t ws_bytes, hipStream_t stream) {
    int st = check(p);
    if (st != GDR_OK) return st;
    if (p->T == 0) return GDR_OK;
    if (!x || !w_gate || !w_up || !w_down || !y) return GDR_ERR_INVALID;
    const Plan l = plan_of(p, false);
    if ((st = check_ws(ws, ws_bytes, l.bytes)) != GDR_OK) return st;
    const size_t es = l.e, in = l.pad ? es : 16, n = (size_t)l.T * p->D * es, w = (size_t)p->D * p->F * es;
    if (!buffers_ok({{x, n, in}, {w_gate, w, in}, {w_up, w, in}, {w_down, w, in}},
                    {{{y, n, es}, 0}, {{saved, saved_bytes(l), 16}, 0}, {{ws, l.bytes, 16}, 0}}))
        return GDR_ERR_INVALID;
    char* b = (char*)ws;
    hipError_t e = hipSuccess;
    if (l.pad) {
        PadArgs c{};
        pad(c, x, b + l.x, l.T, l.T, p->D, l.D);
        pad(c, w_gate, b + l.wg, p->F, p->F, p->D, l.D);
        pad(c, w_up, b + l.wu, p->F, p->F, p->D, l.D);
        pad(c, w_down, b + l.wd, p->D, p->D, p->F, l.F);
        if ((e = launch_pad(l.e, c, stream)) != hipSuccess) return status(e);
    }
    GemmArgs a{};
    a.act = p->act, a.part = (float*)(b + l.part);
    a.q = x, a.ldq = l.D, a.p0 = w_gate, a.p1 = w_up, a.ldp = l.D;
    a.M = l.T, a.N = l.F, a.K = l.D, a.rowsP = p->F;
    a.gu = saved, a.h = saved ? saved_h(l, saved) : b + l.h;
    if ((e = launch_gemm(p->dtype, GATE_UP, a, stream)) != hipSuccess) return status(e);
    a.q = a.h, a.ldq = l.F, a.p0 = w_down, a.p1 = nullptr, a.ldp = l.F;
    a.N = l.D, a.K = l.F, a.rowsP = p->D;
    a.out0 = y, a.ldo = p->D, a.osplit = INT_MAX, a.rows_out = l.T, a.cols_out = p->D;
    return status(launch_gemm(p->dtype, DOWN, a, stream));
}

int gated_ffn_bwd(const ffn_problem* p, const void* x, const void* w_gate, const void* w_up, const void* w_down,
                  const float* saved, const void* dy, void* dx, void* dw_gate, void* dw_up, void* dw_down, void* ws,
                  size_t ws_bytes, hipStream_t stream) {
    int st = check(p);
    if (st != GDR_OK) return st;
    if (!dw_gate != !dw_up) return GDR_ERR_INVALID;
    if (p->T > 0 && (!x || !w_gate || !w_up || !w_down || !saved || !dy)) return GDR_ERR_INVALID;
    const Plan l = plan_of(p, true);
    if ((st = check_ws(ws, ws_bytes, l.bytes)) != GDR_OK) return st;
    const size_t es = l.e, in = l.pad ? es : 16, n = (size_t)l.T * p->D * es, w = (size_t)p->D * p->F * es;
    if (!buffers_ok({{x, n, in}, {w_gate, w, in}, {w_up, w, in}, {w_down, w, in},
                     {saved, saved_bytes(l), 16}, {dy, n, in}},
                    {{{dx, n, es}, 0}, {{dw_gate, w, es}, 0}, {{dw_up, w, es}, 0}, {{dw_down, w, es}, 0},
                     {{ws, l.bytes, 16}, 0}}))
        return GDR_ERR_INVALID;
    if (!dx && !dw_gate && !dw_down) return GDR_OK;
    char* b = (char*)ws;
    hipError_t e = hipSuccess;
    if (l.pad && l.T > 0) {
        PadArgs c{};
        pad(c, x, b + l.x, l.T, l.T, p->D, l.D);
        pad(c, dy, b + l.dy, l.T, l.T, p->D, l.D);
        pad(c, w_gate, b + l.wg, p->F, l.F, p->D, l.D);
        pad(c, w_up, b + l.wu, p->F, l.F, p->D, l.D);
        pad(c, w_down, b + l.wd, p->D, l.D, p->F, l.F);
        if ((e = launch_pad(l.e, c, stream)) != hipSuccess) return status(e);
    }
    GemmArgs a{};
    a.act = p->act, a.part = (float*)(b + l.part), a.dgu = b + l.dgu, a.gu = (float*)saved;
    a.q = dy, a.ldq = l.D, a.p0 = w_down, a.ldp = l.F;
    a.M = l.T, a.N = l.F, a.K = l.D, a.rowsP = p->F;
    if ((e = launch_gemm(p->dtype, DH, a, stream)) != hipSuccess) return status(e);
    GemmArgs g[3];   // dx, dw of gate and up, dw of down
    for (GemmArgs& x : g) x = a, x.osplit = INT_MAX, x.p1 = nullptr;
    g[0].q = b + l.dgu, g[0].ldq = 2 * l.F, g[0].p0 = w_gate, g[0].p1 = w_up, g[0].psplit = l.F, g[0].ldp = l.D;
    g[0].M = l.T, g[0].N = l.D, g[0].K = 2 * l.F;
    g[0].out0 = dx, g[0].ldo = p->D, g[0].rows_out = l.T, g[0].cols_out = p->D;
    g[1].q = b + l.dgu, g[1].ldq = 2 * l.F, g[1].p0 = x, g[1].ldp = l.D;
    g[1].M = 2 * l.F, g[1].N = l.D, g[1].K = l.T;
    g[1].out0 = dw_gate, g[1].out1 = dw_up, g[1].osplit = l.F, g[1].ldo = p->D, g[1].rows_out = p->F, g[1].cols_out = p->D;
    g[2].q = dy, g[2].ldq = l.D, g[2].p0 = saved ? saved_h(l, saved) : nullptr, g[2].ldp = l.F;
    g[2].M = l.D, g[2].N = l.F, g[2].K = l.T;
    g[2].out0 = dw_down, g[2].ldo = p->F, g[2].rows_out = p->D, g[2].cols_out = p->F;
    e = launch_grads(p->dtype, l.grads, g, {dx != nullptr, dw_gate != nullptr, dw_down != nullptr}, a.part, stream);
    return status(e);
}

}  // extern "C"

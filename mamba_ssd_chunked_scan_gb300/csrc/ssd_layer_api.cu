// C ABI of the operators around the scan (residual norm, projection, gated recurrence):
// argument checks and dispatch.  Nothing here allocates device memory; every launch is asynchronous
// on the caller's stream.
#include "ssd_common.cuh"
#include "ssd_kernels.h"

using namespace ssd;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool known(int dtype) { return dtype == SSD_F32 || dtype == SSD_BF16 || dtype == SSD_E4M3; }
size_t elem(int dtype) { return dtype == SSD_F32 ? 4 : dtype == SSD_BF16 ? 2 : 1; }

// Whether [a, a + na) and [b, b + nb) share a byte (NULL shares none).
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && x < y + nb && y < x + na;
}
// Overlap other than being the same array with elements of the same size.
bool clash(const void* a, size_t na, const void* b, size_t nb) { return overlap(a, na, b, nb) && !(a == b && na == nb); }

// A workspace of `need` bytes, 256-byte aligned; none where only the status word would be in it (a wait that runs out is
// then not reported).
bool workspace_ok(const void* ws, size_t bytes, size_t need) {
    return ws ? bytes >= need && aligned(ws, 256) : need == sizeof(WsHeader);
}

// Types and width of the residual norm; SSD_OK or the status to return.
int check_norm(int64_t rows, int32_t width, int32_t dtype, int32_t residual_dtype) {
    if (rows < 0 || width < 1) return SSD_ERR_INVALID_ARG;
    if (dtype != SSD_F32 && dtype != SSD_BF16) return SSD_ERR_INVALID_ARG;
    if (residual_dtype != SSD_F32 && !(residual_dtype == SSD_BF16 && dtype == SSD_BF16)) return SSD_ERR_INVALID_ARG;
    if (width > kAddNormMaxWidth || rows >= ((int64_t)1 << 31)) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

// A (rows, width) matrix of `es`-byte elements with `stride` elements between rows.
struct Mat {
    const void* p;
    int64_t rows, width, stride;
    size_t es;
    size_t span() const { return p && rows ? ((size_t)(rows - 1) * stride + width) * es : 0; }
};
// Whether two matrices share an element.  Column ranges of one wider matrix lie
// inside each other's span without touching.
bool touch(const Mat& a, const Mat& b) {
    if (!overlap(a.p, a.span(), b.p, b.span())) return false;
    if (a.stride == b.stride && a.es == b.es) {
        const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
        const size_t pitch = (size_t)a.stride * a.es;
        const Mat& lo = x < y ? a : b;
        const Mat& hi = x < y ? b : a;
        const size_t off = (x < y ? y - x : x - y) % pitch;
        return !(off >= (size_t)lo.width * lo.es && off + (size_t)hi.width * hi.es <= pitch);
    }
    return true;
}

int check_scan(const ssd_gate_scan_params_t* p) {
    if (!p) return SSD_ERR_INVALID_ARG;
    if (p->batch < 1 || p->seqlen < 1 || p->width < 1 || p->ndocs < 0) return SSD_ERR_INVALID_ARG;
    if (p->dtype != SSD_F32 && p->dtype != SSD_BF16) return SSD_ERR_INVALID_ARG;
    if (p->g_stride < p->width || p->x_stride < p->width) return SSD_ERR_INVALID_ARG;
    if (p->ndocs > 0 && p->batch != 1) return SSD_ERR_INVALID_ARG;
    const int64_t big = (int64_t)1 << 31;
    // token offsets, tile numbers and the bytes between tokens are 32-bit; element offsets are 64-bit
    if (p->seqlen >= big - 256 || p->batch >= big || p->batch * p->seqlen >= big << 2 || p->g_stride >= big / 4 ||
        p->x_stride >= big / 4)
        return SSD_ERR_UNSUPPORTED;
    const int64_t tiles = ((p->seqlen + kScanMinTok - 1) / kScanMinTok) * ((p->width + kScanCh - 1) / kScanCh);
    if (tiles >= big / p->batch) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

int check_linear(const ssd_linear_params_t* p) {
    if (!p) return SSD_ERR_INVALID_ARG;
    if (p->m < 0 || p->n < 1 || p->k < 1 || p->ldx < p->k) return SSD_ERR_INVALID_ARG;
    if (p->dtype != SSD_BF16 && p->dtype != SSD_E4M3) return SSD_ERR_INVALID_ARG;
    if (p->act != SSD_ACT_NONE && p->act != SSD_ACT_SILU && p->act != SSD_ACT_GELU) return SSD_ERR_INVALID_ARG;
    const int unit = p->dtype == SSD_BF16 ? 8 : 16;   // elements per 16 bytes
    if (p->k % unit != 0 || p->ldx % unit != 0) return SSD_ERR_UNSUPPORTED;
    // tile numbers (parts of the contraction among them) and tile coordinates are 32-bit
    const int64_t big = (int64_t)1 << 30;
    if (p->m >= big || p->n >= big || p->k >= big || p->ldx >= big) return SSD_ERR_UNSUPPORTED;
    const int64_t tm = p->m / 64 + 1, tn = p->n / 64 + 1, tk = p->k / 64 + 1;
    if (tm > big / kLinearMaxSplits / tn || tm > big / kLinearMaxSplits / tk || tn > big / kLinearMaxSplits / tk) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

// Workspace of the projection's backward, in bytes from its start: the status word, dpre
// where it is not dy itself, the slabs' shares of dbias, and the parts of whichever product runs.
struct LinearBwdLayout {
    bool own_dpre;
    int64_t ldp;
    size_t dpre_off, shares_off, parts_off, total;
    LinearPlan dx, dw;
};
LinearBwdLayout linear_bwd_layout(const ssd_linear_params_t* p) {
    LinearBwdLayout l;
    l.own_dpre = p->act != SSD_ACT_NONE || p->n % 8 != 0;
    l.ldp = (p->n + 7) / 8 * 8;
    l.dpre_off = sizeof(WsHeader);
    l.shares_off = l.dpre_off + (l.own_dpre ? align_up((size_t)p->m * l.ldp * 2, 256) : 0);
    l.parts_off = l.shares_off + align_up((size_t)linear_dpre_slabs(p->m, p->n) * p->n * 4, 256);
    l.dx = linear_plan(p->m, p->k, (int64_t)p->n * 2, false);
    l.dw = linear_plan(p->n, p->k, p->m * 2, false);
    l.total = l.parts_off + (l.dx.parts_bytes > l.dw.parts_bytes ? l.dx.parts_bytes : l.dw.parts_bytes);
    return l;
}

// Fault injection (test aid): a cap on every bounded wait, in polls (0: an ordinary call), and how many loads a CTA issues;
// the recurrence: negative, no tile publishes its map.
struct Stall {
    uint32_t rounds = 0;
    int loads = 0;
};

int gate_scan_impl(const ssd_gate_scan_params_t* p, const void* g, const void* x, const float* initial_states,
                   const int32_t* cu_seqlens, void* y, float* final_states, void* workspace, size_t workspace_bytes,
                   void* stream, const Stall& stall) {
    const int rc = check_scan(p);
    if (rc != SSD_OK) return rc;
    if (!g || !x || !y || (p->ndocs > 0) != (cu_seqlens != nullptr)) return SSD_ERR_INVALID_ARG;
    const size_t es = elem(p->dtype);
    if (!aligned(g, es) || !aligned(x, es) || !aligned(y, es) || !aligned(initial_states, 4) ||
        !aligned(final_states, 4) || !aligned(cu_seqlens, 4))
        return SSD_ERR_INVALID_ARG;
    const size_t need = ssd_gate_scan_workspace_size(p);
    if (!workspace_ok(workspace, workspace_bytes, need)) return SSD_ERR_WORKSPACE;
    const int64_t rows = p->batch * p->seqlen, nst = p->ndocs > 0 ? p->ndocs : p->batch;
    const Mat in[] = {{g, rows, p->width, p->g_stride, es}, {x, rows, p->width, p->x_stride, es},
                      {initial_states, nst, p->width, p->width, 4}, {cu_seqlens, 1, p->ndocs + 1, p->ndocs + 1, 4}};
    const Mat out[] = {{y, rows, p->width, p->width, es}, {final_states, nst, p->width, p->width, 4},
                       {workspace, 1, (int64_t)need, (int64_t)need, 1}};
    for (int i = 0; i < 3; ++i) {
        for (const Mat& m : in)
            if (touch(out[i], m)) return SSD_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (touch(out[i], out[j])) return SSD_ERR_INVALID_ARG;
    }
    GateScanArgs a = {};
    a.batch = p->batch; a.seqlen = p->seqlen; a.width = p->width; a.dtype = p->dtype; a.ndocs = p->ndocs;
    a.g_stride = p->g_stride; a.x_stride = p->x_stride;
    a.g = g; a.x = x; a.init = initial_states; a.cu = cu_seqlens; a.y = y;
    a.enter = initial_states; a.leave = final_states;
    a.wait_iters = stall.rounds; a.loads = stall.loads; a.mute = stall.loads < 0;
    return launch_gate_scan(a, workspace, false, (cudaStream_t)stream) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

int linear_impl(const ssd_linear_params_t* p, const void* x, const void* w, const float* x_scales, const float* w_scales,
                const float* bias, const void* residual, void* y, void* pre, void* workspace, size_t workspace_bytes,
                void* stream, const Stall& stall) {
    const int rc = check_linear(p);
    if (rc != SSD_OK) return rc;
    const bool e4m3 = p->dtype == SSD_E4M3;
    if (e4m3 != (w_scales != nullptr) || (!e4m3 && x_scales) || (e4m3 && !x_scales && p->m > 0)) return SSD_ERR_INVALID_ARG;
    if (p->m == 0) return SSD_OK;
    if (!x || !w || !y) return SSD_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(x_scales, 4) || !aligned(w_scales, 4) || !aligned(bias, 4) ||
        !aligned(residual, 2) || !aligned(y, 2) || !aligned(pre, 2))
        return SSD_ERR_INVALID_ARG;
    const size_t es = elem(p->dtype);
    const LinearPlan plan = linear_plan(p->m, p->n, (int64_t)p->k * es, true);
    const size_t need = sizeof(WsHeader) + plan.parts_bytes;
    if (!workspace_ok(workspace, workspace_bytes, need)) return SSD_ERR_WORKSPACE;
    const Mat in[] = {{x, p->m, p->k, p->ldx, es}, {w, p->n, p->k, p->k, es}, {x_scales, 1, p->m, p->m, 4},
                      {w_scales, 1, p->n, p->n, 4}, {bias, 1, p->n, p->n, 4}};
    const Mat my = {y, p->m, p->n, p->n, 2}, mp = {pre, p->m, p->n, p->n, 2}, mr = {residual, p->m, p->n, p->n, 2},
              mw = {workspace, 1, (int64_t)need, (int64_t)need, 1};
    for (const Mat& m : in)
        if (touch(my, m) || touch(mp, m) || touch(mw, m)) return SSD_ERR_INVALID_ARG;
    if (touch(my, mp) || touch(mp, mr) || touch(mw, my) || touch(mw, mp) || touch(mw, mr) ||
        (y != residual && touch(my, mr)))
        return SSD_ERR_INVALID_ARG;
    LinearArgs a = {};
    a.m = p->m; a.n = p->n; a.k = p->k; a.dtype = p->dtype; a.act = p->act;
    a.x = {x, p->ldx, false};
    a.w = {w, p->k, false};
    a.x_scales = x_scales; a.w_scales = w_scales; a.bias = bias; a.residual = residual; a.y = y; a.pre = pre;
    a.wait_iters = stall.rounds; a.loads = (uint32_t)stall.loads;
    a.ws = (WsHeader*)workspace;
    a.parts = workspace ? (float*)((char*)workspace + sizeof(WsHeader)) : nullptr;
    return launch_linear(a, plan, (cudaStream_t)stream) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // namespace

extern "C" {

int ssd_add_norm(int64_t rows, int32_t width, int32_t dtype, int32_t residual_dtype, int32_t out_dtype,
                 const void* x, const void* residual, const float* weight, float eps, void* out, float* scales,
                 void* residual_out, float* rstd, void* stream) {
    if (!known(out_dtype)) return SSD_ERR_INVALID_ARG;
    const int rc = check_norm(rows, width, dtype, residual_dtype);
    if (rc != SSD_OK) return rc;
    if (out_dtype != dtype && out_dtype != SSD_E4M3) return SSD_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || eps > 3.0e38f) return SSD_ERR_INVALID_ARG;   // rejects NaN and inf
    if (rows == 0) return SSD_OK;
    if (!x || !weight || !out || (out_dtype == SSD_E4M3 && !scales)) return SSD_ERR_INVALID_ARG;
    if (!aligned(x, elem(dtype)) || !aligned(out, elem(out_dtype)) || !aligned(residual, elem(residual_dtype)) ||
        !aligned(residual_out, elem(residual_dtype)) || !aligned(weight, 4) || !aligned(scales, 4) || !aligned(rstd, 4))
        return SSD_ERR_INVALID_ARG;
    const size_t n = (size_t)rows * width, nx = n * elem(dtype), no = n * elem(out_dtype), nr = n * elem(residual_dtype);
    const size_t nw = (size_t)width * 4, ns = (size_t)rows * 4;
    if (out_dtype != SSD_E4M3) scales = nullptr;
    if (clash(out, no, x, nx) || clash(out, no, residual, nr) || clash(residual_out, nr, residual, nr) ||
        clash(residual_out, nr, x, nx) || overlap(residual_out, nr, out, no) || overlap(out, no, weight, nw) ||
        overlap(residual_out, nr, weight, nw))
        return SSD_ERR_INVALID_ARG;
    float* const small[2] = {scales, rstd};
    for (float* s : small)
        if (overlap(s, ns, x, nx) || overlap(s, ns, residual, nr) || overlap(s, ns, weight, nw) ||
            overlap(s, ns, out, no) || overlap(s, ns, residual_out, nr))
            return SSD_ERR_INVALID_ARG;
    if (overlap(scales, ns, rstd, ns)) return SSD_ERR_INVALID_ARG;
    AddNormArgs a;
    a.rows = rows; a.width = width; a.dtype = dtype; a.residual_dtype = residual_dtype; a.out_dtype = out_dtype;
    a.eps = eps; a.x = x; a.residual = residual; a.weight = weight; a.out = out; a.scales = scales;
    a.residual_out = residual_out; a.rstd = rstd;
    return launch_add_norm(a, (cudaStream_t)stream) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

size_t ssd_add_norm_bwd_workspace_size(int64_t rows, int32_t width) {
    if (rows < 1 || check_norm(rows, width, SSD_F32, SSD_F32) != SSD_OK) return 0;
    return (size_t)add_norm_bwd_shares(rows, width) * width * sizeof(float);
}

int ssd_add_norm_bwd(int64_t rows, int32_t width, int32_t dtype, int32_t residual_dtype, const void* dout,
                     const void* h, const float* weight, const float* rstd, const void* dresidual_out, void* dx,
                     void* dresidual, float* dweight, void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = check_norm(rows, width, dtype, residual_dtype);
    if (rc != SSD_OK) return rc;
    if (!dweight || !aligned(dweight, 4)) return SSD_ERR_INVALID_ARG;
    if (rows == 0)
        return cudaMemsetAsync(dweight, 0, (size_t)width * 4, (cudaStream_t)stream) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
    if (!dout || !h || !weight || !rstd || (!dx && !dresidual)) return SSD_ERR_INVALID_ARG;
    const size_t et = elem(dtype), er = elem(residual_dtype);
    if (!aligned(dout, et) || !aligned(dx, et) || !aligned(h, er) || !aligned(dresidual_out, er) ||
        !aligned(dresidual, er) || !aligned(weight, 4) || !aligned(rstd, 4))
        return SSD_ERR_INVALID_ARG;
    const size_t n = (size_t)rows * width, nt = n * et, nr = n * er, nw = (size_t)width * 4, ns = (size_t)rows * 4;
    const size_t need = ssd_add_norm_bwd_workspace_size(rows, width);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) return SSD_ERR_WORKSPACE;
    // dx and dresidual may each replace an incoming gradient of their own type
    if (clash(dx, nt, dout, nt) || overlap(dx, nt, h, nr) || clash(dx, nt, dresidual_out, nr) ||
        clash(dresidual, nr, dout, nt) || overlap(dresidual, nr, h, nr) || clash(dresidual, nr, dresidual_out, nr) ||
        overlap(dx, nt, dresidual, nr))
        return SSD_ERR_INVALID_ARG;
    struct { const void* p; size_t n; } const in[] = {{dout, nt}, {h, nr}, {dresidual_out, nr}, {weight, nw},
                                                      {rstd, ns}, {dx, nt}, {dresidual, nr}};
    for (const auto& b : in)
        if (overlap(dweight, nw, b.p, b.n) || overlap(workspace, need, b.p, b.n)) return SSD_ERR_INVALID_ARG;
    if (overlap(dx, nt, weight, nw) || overlap(dresidual, nr, weight, nw) || overlap(dx, nt, rstd, ns) ||
        overlap(dresidual, nr, rstd, ns) || overlap(dweight, nw, workspace, need))
        return SSD_ERR_INVALID_ARG;
    AddNormBwdArgs a;
    a.rows = rows; a.width = width; a.dtype = dtype; a.residual_dtype = residual_dtype;
    a.dout = dout; a.h = h; a.weight = weight; a.rstd = rstd; a.dres = dresidual_out;
    a.dx = dx; a.dres_out = dresidual; a.dweight = dweight; a.shares = (float*)workspace;
    return launch_add_norm_bwd(a, (cudaStream_t)stream) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

size_t ssd_gate_scan_workspace_size(const ssd_gate_scan_params_t* p) {
    if (check_scan(p) != SSD_OK) return 0;
    return gate_scan_workspace(p->batch, p->seqlen, p->width, p->dtype);
}

int ssd_gate_scan(const ssd_gate_scan_params_t* p, const void* g, const void* x, const float* initial_states,
                  const int32_t* cu_seqlens, void* y, float* final_states, void* workspace, size_t workspace_bytes,
                  void* stream) {
    return gate_scan_impl(p, g, x, initial_states, cu_seqlens, y, final_states, workspace, workspace_bytes, stream, Stall());
}

int ssd_gate_scan_fault_inject(const ssd_gate_scan_params_t* p, const void* g, const void* x, const float* initial_states,
                               const int32_t* cu_seqlens, void* y, float* final_states, void* workspace,
                               size_t workspace_bytes, int32_t loads, uint32_t max_wait_rounds, void* stream) {
    if (loads < -1 || max_wait_rounds < kMinInjectWaitRounds) return SSD_ERR_INVALID_ARG;
    if (!workspace) return SSD_ERR_WORKSPACE;
    return gate_scan_impl(p, g, x, initial_states, cu_seqlens, y, final_states, workspace, workspace_bytes, stream,
                          Stall{max_wait_rounds, loads});
}

int ssd_gate_scan_bwd(const ssd_gate_scan_params_t* p, const void* g, const void* x, const void* y,
                      const float* initial_states, const int32_t* cu_seqlens, const void* dy,
                      const float* dfinal_states, void* dg, void* dx, float* dinitial_states, void* workspace,
                      size_t workspace_bytes, void* stream) {
    const int rc = check_scan(p);
    if (rc != SSD_OK) return rc;
    if (!g || !x || !y || !dy || !dg || !dx || (p->ndocs > 0) != (cu_seqlens != nullptr)) return SSD_ERR_INVALID_ARG;
    const size_t es = elem(p->dtype);
    if (!aligned(g, es) || !aligned(x, es) || !aligned(y, es) || !aligned(dy, es) || !aligned(dg, es) ||
        !aligned(dx, es) || !aligned(initial_states, 4) || !aligned(dfinal_states, 4) || !aligned(dinitial_states, 4) ||
        !aligned(cu_seqlens, 4))
        return SSD_ERR_INVALID_ARG;
    const size_t need = ssd_gate_scan_workspace_size(p);
    if (!workspace_ok(workspace, workspace_bytes, need)) return SSD_ERR_WORKSPACE;
    const int64_t rows = p->batch * p->seqlen, nst = p->ndocs > 0 ? p->ndocs : p->batch;
    const int64_t w = p->width;
    const Mat in[] = {{g, rows, w, p->g_stride, es}, {x, rows, w, p->x_stride, es}, {y, rows, w, w, es}, {dy, rows, w, w, es},
                      {initial_states, nst, w, w, 4}, {dfinal_states, nst, w, w, 4},
                      {cu_seqlens, 1, p->ndocs + 1, p->ndocs + 1, 4}};
    const Mat out[] = {{dg, rows, w, p->g_stride, es}, {dx, rows, w, p->x_stride, es}, {dinitial_states, nst, w, w, 4},
                       {workspace, 1, (int64_t)need, (int64_t)need, 1}};
    for (int i = 0; i < 4; ++i) {
        for (const Mat& m : in)
            if (touch(out[i], m)) return SSD_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (touch(out[i], out[j])) return SSD_ERR_INVALID_ARG;
    }
    GateScanArgs a = {};
    a.batch = p->batch; a.seqlen = p->seqlen; a.width = p->width; a.dtype = p->dtype; a.ndocs = p->ndocs;
    a.g_stride = p->g_stride; a.x_stride = p->x_stride;
    a.g = g; a.x = x; a.init = initial_states; a.cu = cu_seqlens; a.y = const_cast<void*>(y);
    a.dy = dy; a.dg = dg; a.dx = dx; a.enter = dfinal_states; a.leave = dinitial_states;
    return launch_gate_scan(a, workspace, true, (cudaStream_t)stream) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

int ssd_gate_scan_step(int64_t batch, int32_t width, int32_t dtype, int64_t g_stride, int64_t x_stride, const void* g,
                       const void* x, const float* state_in, float* state_out, void* y, void* stream) {
    if (batch < 0 || width < 1 || g_stride < width || x_stride < width) return SSD_ERR_INVALID_ARG;
    if (dtype != SSD_F32 && dtype != SSD_BF16) return SSD_ERR_INVALID_ARG;
    if (batch == 0) return SSD_OK;
    if (batch >= ((int64_t)1 << 36) / width || g_stride >= (int64_t)1 << 31 || x_stride >= (int64_t)1 << 31) return SSD_ERR_UNSUPPORTED;
    if (!g || !x || !state_in || !state_out || !y) return SSD_ERR_INVALID_ARG;
    const size_t es = elem(dtype);
    if (!aligned(g, es) || !aligned(x, es) || !aligned(y, es) || !aligned(state_in, 4) || !aligned(state_out, 4))
        return SSD_ERR_INVALID_ARG;
    const Mat mg = {g, batch, width, g_stride, es}, mx = {x, batch, width, x_stride, es}, my = {y, batch, width, width, es};
    const Mat si = {state_in, batch, width, width, 4}, so = {state_out, batch, width, width, 4};
    if (touch(my, mg) || touch(my, mx) || touch(my, si) || touch(my, so) || touch(so, mg) || touch(so, mx) ||
        (state_in != state_out && touch(so, si)))
        return SSD_ERR_INVALID_ARG;
    GateStepArgs a;
    a.batch = batch; a.width = width; a.dtype = dtype; a.g_stride = g_stride; a.x_stride = x_stride;
    a.g = g; a.x = x; a.state_in = state_in; a.state_out = state_out; a.y = y;
    return launch_gate_scan_step(a, (cudaStream_t)stream) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

size_t ssd_linear_workspace_size(const ssd_linear_params_t* p) {
    if (check_linear(p) != SSD_OK) return 0;
    if (p->m == 0) return sizeof(WsHeader);
    return sizeof(WsHeader) + linear_plan(p->m, p->n, (int64_t)p->k * elem(p->dtype), true).parts_bytes;
}

size_t ssd_linear_bwd_workspace_size(const ssd_linear_params_t* p) {
    if (check_linear(p) != SSD_OK || p->dtype != SSD_BF16) return 0;
    return p->m == 0 ? sizeof(WsHeader) : linear_bwd_layout(p).total;
}

int ssd_linear_plan(const ssd_linear_params_t* p, int product, ssd_linear_plan_t* plan) {
    const int rc = check_linear(p);
    if (rc != SSD_OK) return rc;
    if (!plan || product < 0 || product > 2) return SSD_ERR_INVALID_ARG;
    if (product && p->dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    *plan = ssd_linear_plan_t();
    if (p->m == 0) return SSD_OK;
    const int64_t rows = product == 2 ? p->n : p->m, cols = product ? p->k : p->n;
    const int64_t kbytes = product == 0 ? (int64_t)p->k * elem(p->dtype) : product == 1 ? (int64_t)p->n * 2 : p->m * 2;
    const LinearPlan l = linear_plan(rows, cols, kbytes, product == 0);
    plan->tile_rows = l.pair ? 2 * kLinearTileRows : kLinearTileRows;
    plan->tile_cols = l.tile_n;
    plan->transposed = l.swap;
    plan->whole = l.whole;
    plan->splits = l.splits;
    const int64_t dr = l.swap ? cols : rows, dc = l.swap ? rows : cols;
    plan->tiles = ((dr + plan->tile_rows - 1) / plan->tile_rows) * ((dc + l.tile_n - 1) / l.tile_n);
    return SSD_OK;
}

int ssd_linear(const ssd_linear_params_t* p, const void* x, const void* w, const float* x_scales, const float* w_scales,
               const float* bias, const void* residual, void* y, void* pre, void* workspace, size_t workspace_bytes,
               void* stream) {
    return linear_impl(p, x, w, x_scales, w_scales, bias, residual, y, pre, workspace, workspace_bytes, stream, Stall());
}

int ssd_linear_fault_inject(const ssd_linear_params_t* p, const void* x, const void* w, const float* x_scales,
                            const float* w_scales, const float* bias, const void* residual, void* y, void* pre,
                            void* workspace, size_t workspace_bytes, int32_t loads, uint32_t max_wait_rounds, void* stream) {
    if (loads < 0 || max_wait_rounds < kMinInjectWaitRounds) return SSD_ERR_INVALID_ARG;
    if (!workspace) return SSD_ERR_WORKSPACE;
    return linear_impl(p, x, w, x_scales, w_scales, bias, residual, y, pre, workspace, workspace_bytes, stream,
                       Stall{max_wait_rounds, loads});
}

int ssd_linear_bwd(const ssd_linear_params_t* p, const void* x, const void* w, const void* pre, const void* dy, void* dx,
                   void* dw, float* dbias, void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = check_linear(p);
    if (rc != SSD_OK) return rc;
    if (p->dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    cudaStream_t st = (cudaStream_t)stream;
    if (!aligned(dw, 2) || !aligned(dbias, 4) || !aligned(dx, 2)) return SSD_ERR_INVALID_ARG;
    if (p->m == 0) {
        if (dw && cudaMemsetAsync(dw, 0, (size_t)p->n * p->k * 2, st) != cudaSuccess) return SSD_ERR_CUDA;
        if (dbias && cudaMemsetAsync(dbias, 0, (size_t)p->n * 4, st) != cudaSuccess) return SSD_ERR_CUDA;
        return SSD_OK;
    }
    if (!x || !w || !dy || (!dx && !dw && !dbias) || (p->act != SSD_ACT_NONE) != (pre != nullptr)) return SSD_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(dy, 16) || !aligned(pre, 2)) return SSD_ERR_INVALID_ARG;
    const LinearBwdLayout l = linear_bwd_layout(p);
    if (!workspace || workspace_bytes < l.total || !aligned(workspace, 256)) return SSD_ERR_WORKSPACE;
    const Mat in[] = {{x, p->m, p->k, p->ldx, 2}, {w, p->n, p->k, p->k, 2}, {pre, p->m, p->n, p->n, 2}, {dy, p->m, p->n, p->n, 2}};
    const Mat out[] = {{dx, p->m, p->k, p->k, 2}, {dw, p->n, p->k, p->k, 2}, {dbias, 1, p->n, p->n, 4},
                       {workspace, 1, (int64_t)l.total, (int64_t)l.total, 1}};
    for (int i = 0; i < 4; ++i) {
        for (const Mat& m : in)
            if (touch(out[i], m)) return SSD_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (touch(out[i], out[j])) return SSD_ERR_INVALID_ARG;
    }
    char* ws = (char*)workspace;
    // the first product clears the status word
    if (!dx && !dw && cudaMemsetAsync(ws, 0, sizeof(WsHeader), st) != cudaSuccess) return SSD_ERR_CUDA;
    LinearDpreArgs d = {};
    d.m = p->m; d.n = p->n; d.act = p->act; d.ldp = l.ldp; d.dy = dy; d.pre = pre;
    d.dpre = l.own_dpre && (dx || dw) ? ws + l.dpre_off : nullptr;
    d.shares = dbias ? (float*)(ws + l.shares_off) : nullptr;
    d.dbias = dbias;
    if ((d.dpre || dbias) && launch_linear_dpre(d, st) != cudaSuccess) return SSD_ERR_CUDA;
    const LinearOperand g = {l.own_dpre ? (const void*)(ws + l.dpre_off) : dy, l.own_dpre ? l.ldp : p->n, false};
    LinearArgs a = {};
    a.dtype = SSD_BF16; a.act = SSD_ACT_NONE;
    a.ws = (WsHeader*)workspace;
    a.parts = (float*)(ws + l.parts_off);
    if (dx) {   // (m, k) = dpre (m, n) w (n, k): w's contraction runs along its rows
        a.m = p->m; a.n = p->k; a.k = p->n; a.y = dx;
        a.x = g;
        a.w = {w, p->k, true};
        if (launch_linear(a, l.dx, st) != cudaSuccess) return SSD_ERR_CUDA;
    }
    if (dw) {   // (n, k) = dpre^T (n, m) x (m, k): both contractions run along the rows
        a.m = p->n; a.n = p->k; a.k = p->m; a.y = dw;
        a.x = {g.p, g.ld, true};
        a.keep_status = dx != nullptr;
        a.w = {x, p->ldx, true};
        if (launch_linear(a, l.dw, st) != cudaSuccess) return SSD_ERR_CUDA;
    }
    return SSD_OK;
}

}  // extern "C"

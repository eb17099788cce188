// C ABI of the operators around the scan (residual norm, projection, gated recurrence, the norms around a block and their
// 8-bit checkpoints):
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

// The same with x in 8-bit rows, which may start at any byte.
int check_linear_packed(const ssd_linear_params_t* p) {
    if (!p) return SSD_ERR_INVALID_ARG;
    if (p->ldx < p->k) return SSD_ERR_INVALID_ARG;
    if (p->dtype != SSD_BF16 || p->ldx >= (int64_t)1 << 30) return SSD_ERR_UNSUPPORTED;
    ssd_linear_params_t q = *p;
    q.ldx = q.k;
    return check_linear(&q);
}

// Workspace of the projection's backward, in bytes from its start: the status word, dpre
// where it is not dy itself, the slabs' shares of dbias, and the parts of whichever product runs.
struct LinearBwdLayout {
    bool own_dpre;
    int64_t ldp;
    size_t dpre_off, shares_off, parts_off, rows_off, inv_off, ones_off, total;
    LinearPlan dx, dw;
};
// expand: with room for x in bf16, its scales' factors' reciprocals and a row of ones.
LinearBwdLayout linear_bwd_layout(const ssd_linear_params_t* p, bool expand) {
    LinearBwdLayout l;
    l.own_dpre = p->act != SSD_ACT_NONE || p->n % 8 != 0;
    l.ldp = (p->n + 7) / 8 * 8;
    l.dpre_off = sizeof(WsHeader);
    l.shares_off = l.dpre_off + (l.own_dpre ? align_up((size_t)p->m * l.ldp * 2, 256) : 0);
    l.parts_off = l.shares_off + align_up((size_t)linear_dpre_slabs(p->m, p->n) * p->n * 4, 256);
    l.dx = linear_plan(p->m, p->k, (int64_t)p->n * 2, false);
    l.dw = linear_plan(p->n, p->k, p->m * 2, false);
    l.rows_off = l.parts_off + (l.dx.parts_bytes > l.dw.parts_bytes ? l.dx.parts_bytes : l.dw.parts_bytes);
    l.total = l.rows_off;
    if (expand) {
        l.rows_off = align_up(l.rows_off, 256);
        l.inv_off = align_up(l.rows_off + (size_t)p->m * p->k * 2, 256);
        l.ones_off = align_up(l.inv_off + (size_t)p->m * 4, 256);
        l.total = l.ones_off + (size_t)p->k * 4;
    }
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

// x_scales, pre_scales: x, pre are 8-bit rows; packed: x may be missing where dw is.
int linear_bwd_impl(const ssd_linear_params_t* p, const void* x, const float* x_scales, const void* w, const void* pre,
                    const float* pre_scales, const void* dy, void* dx, void* dw, float* dbias, void* workspace,
                    size_t workspace_bytes, void* stream, bool packed) {
    const int rc = x_scales ? check_linear_packed(p) : check_linear(p);
    if (rc != SSD_OK) return rc;
    if (p->dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    cudaStream_t st = (cudaStream_t)stream;
    if (!aligned(dw, 2) || !aligned(dbias, 4) || !aligned(dx, 2)) return SSD_ERR_INVALID_ARG;
    if (p->m == 0) {
        if (dw && cudaMemsetAsync(dw, 0, (size_t)p->n * p->k * 2, st) != cudaSuccess) return SSD_ERR_CUDA;
        if (dbias && cudaMemsetAsync(dbias, 0, (size_t)p->n * 4, st) != cudaSuccess) return SSD_ERR_CUDA;
        return SSD_OK;
    }
    if ((!x && (dw || x_scales || !packed)) || !w || !dy || (!dx && !dw && !dbias) || (p->act != SSD_ACT_NONE) != (pre != nullptr)) return SSD_ERR_INVALID_ARG;
    if ((pre_scales && !pre) || !aligned(x_scales, 4) || !aligned(pre_scales, 4)) return SSD_ERR_INVALID_ARG;
    if (!aligned(x, x_scales ? 1 : 16) || !aligned(w, 16) || !aligned(dy, 16) || !aligned(pre, pre_scales ? 1 : 2)) return SSD_ERR_INVALID_ARG;
    const LinearBwdLayout l = linear_bwd_layout(p, x_scales && dw);
    if (!workspace || workspace_bytes < l.total || !aligned(workspace, 256)) return SSD_ERR_WORKSPACE;
    const size_t ex = x_scales ? 1 : 2, ep = pre_scales ? 1 : 2;
    const Mat in[] = {{x, p->m, p->k, p->ldx, ex}, {w, p->n, p->k, p->k, 2}, {pre, p->m, p->n, p->n, ep}, {dy, p->m, p->n, p->n, 2},
                      {x_scales, 1, p->m, p->m, 4}, {pre_scales, 1, p->m, p->m, 4}};
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
    d.m = p->m; d.n = p->n; d.act = p->act; d.ldp = l.ldp; d.dy = dy; d.pre = pre; d.pre_scales = pre_scales;
    d.dpre = l.own_dpre && (dx || dw) ? ws + l.dpre_off : nullptr;
    d.shares = dbias ? (float*)(ws + l.shares_off) : nullptr;
    d.dbias = dbias;
    LinearDpreRows e = {};
    const bool factors = x_scales && dw && d.dpre;
    if (factors) {
        e.x_scales = x_scales;
        if (dx) {
            e.inv_factors = (float*)(ws + l.inv_off);
            e.ones = (float*)(ws + l.ones_off);
            e.k = p->k;
        }
    }
    PackArgs u = {};   // x as the products' operand
    if (x_scales && dw) {
        u.units = p->m; u.size = p->k; u.groups = 1; u.dtype = SSD_BF16; u.stride = p->ldx;
        u.codes = const_cast<void*>(x); u.scales = const_cast<float*>(x_scales); u.out = ws + l.rows_off;
        u.power_only = factors;
    }
    const bool together = u.out && (d.dpre || dbias) && unpack_flat_ctas(u) > 0;
    if (together) e.expand = u;
    if ((d.dpre || dbias) && launch_linear_dpre(d, e, st) != cudaSuccess) return SSD_ERR_CUDA;
    const LinearOperand g = {l.own_dpre ? (const void*)(ws + l.dpre_off) : dy, l.own_dpre ? l.ldp : p->n, false};
    LinearArgs a = {};
    a.dtype = SSD_BF16; a.act = SSD_ACT_NONE;
    a.ws = (WsHeader*)workspace;
    a.parts = (float*)(ws + l.parts_off);
    if (dx) {   // (m, k) = dpre (m, n) w (n, k): w's contraction runs along its rows
        a.m = p->m; a.n = p->k; a.k = p->n; a.y = dx;
        a.x = g;
        a.w = {w, p->k, true};
        a.x_scales = e.inv_factors;
        a.w_scales = e.ones;
        if (launch_linear(a, l.dx, st) != cudaSuccess) return SSD_ERR_CUDA;
        a.x_scales = a.w_scales = nullptr;
    }
    if (dw) {   // (n, k) = dpre^T (n, m) x (m, k): both contractions run along the rows
        a.m = p->n; a.n = p->k; a.k = p->m; a.y = dw;
        a.x = {g.p, g.ld, true};
        a.keep_status = dx != nullptr;
        a.w = {x, p->ldx, true};
        if (x_scales) {
            if (!together && launch_unpack(u, st) != cudaSuccess) return SSD_ERR_CUDA;
            a.w = {ws + l.rows_off, p->k, true};
        }
        if (launch_linear(a, l.dw, st) != cudaSuccess) return SSD_ERR_CUDA;
    }
    return SSD_OK;
}

// Units of 8-bit rows: rows, each of width / group columns' groups.
int check_rows(int64_t rows, int32_t width, int32_t group, int32_t dtype, int64_t stride, int32_t most) {
    if (rows < 0 || width < 1 || group < 1 || width % group != 0 || stride < width) return SSD_ERR_INVALID_ARG;
    if (dtype != SSD_F32 && dtype != SSD_BF16) return SSD_ERR_INVALID_ARG;
    const int64_t big = (int64_t)1 << 30;
    if (group > most || width >= big || stride >= big || rows >= 2 * big / (width / group)) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

int check_gate(const ssd_gate_norm_params_t* p, int64_t dz_stride) {
    if (!p) return SSD_ERR_INVALID_ARG;
    if (!(p->eps >= 0.f) || p->eps > 3.0e38f || dz_stride < p->width) return SSD_ERR_INVALID_ARG;
    if (dz_stride >= (int64_t)1 << 30) return SSD_ERR_UNSUPPORTED;
    return check_rows(p->rows, p->width, p->group_size, p->dtype, p->z_stride, kBlockNormMaxSize);
}

// gate, dgate: whether the call has them, and so their strides.
int check_block(const ssd_block_norm_params_t* p, bool gate, bool dgate) {
    if (!p) return SSD_ERR_INVALID_ARG;
    if (!(p->eps >= 0.f) || p->eps > 3.0e38f || !(p->scale >= -3.0e38f && p->scale <= 3.0e38f)) return SSD_ERR_INVALID_ARG;
    if (p->residual_dtype != SSD_F32 && !(p->residual_dtype == SSD_BF16 && p->dtype == SSD_BF16)) return SSD_ERR_INVALID_ARG;
    if (p->out_dtype != p->dtype && p->out_dtype != SSD_E4M3) return SSD_ERR_INVALID_ARG;
    if (dgate && p->dgate_stride < p->width) return SSD_ERR_INVALID_ARG;
    if (dgate && p->dgate_stride >= (int64_t)1 << 30) return SSD_ERR_UNSUPPORTED;
    return check_rows(p->rows, p->width, p->width, p->dtype, gate ? p->gate_stride : p->width, kBlockNormMaxSize);
}

// Whether an output shares an element with an input, or with an output before it.
template <int I, int O>
bool mixed(const Mat (&in)[I], const Mat (&out)[O]) {
    for (int i = 0; i < O; ++i) {
        for (const Mat& m : in)
            if (touch(out[i], m)) return true;
        for (int j = 0; j < i; ++j)
            if (touch(out[i], out[j])) return true;
    }
    return false;
}

// Whether each matrix starts on an element.
template <int N>
bool on_elements(const Mat (&m)[N]) {
    for (const Mat& x : m)
        if (!aligned(x.p, x.es)) return false;
    return true;
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
    return p->m == 0 ? sizeof(WsHeader) : linear_bwd_layout(p, false).total;
}

size_t ssd_linear_bwd_packed_workspace_size(const ssd_linear_params_t* p) {
    if (check_linear_packed(p) != SSD_OK) return 0;
    return p->m == 0 ? sizeof(WsHeader) : linear_bwd_layout(p, true).total;
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
    return linear_bwd_impl(p, x, nullptr, w, pre, nullptr, dy, dx, dw, dbias, workspace, workspace_bytes, stream, false);
}

int ssd_linear_bwd_packed(const ssd_linear_params_t* p, const void* x, const float* x_scales, const void* w, const void* pre,
                          const float* pre_scales, const void* dy, void* dx, void* dw, float* dbias, void* workspace,
                          size_t workspace_bytes, void* stream) {
    return linear_bwd_impl(p, x, x_scales, w, pre, pre_scales, dy, dx, dw, dbias, workspace, workspace_bytes, stream, true);
}

int ssd_pack_rows(int64_t rows, int32_t width, int32_t group_size, int32_t dtype, int64_t x_stride, const void* x, void* codes,
                  float* scales, void* stream) {
    const int rc = check_rows(rows, width, group_size, dtype, x_stride, kPackMaxSize);
    if (rc != SSD_OK || rows == 0) return rc;
    if (!x || !codes || !scales) return SSD_ERR_INVALID_ARG;
    const int groups = width / group_size;
    const Mat in[] = {{x, rows, width, x_stride, elem(dtype)}};
    const Mat out[] = {{codes, rows, width, width, 1}, {scales, rows, groups, groups, 4}};
    if (!on_elements(in) || !on_elements(out) || mixed(in, out)) return SSD_ERR_INVALID_ARG;
    PackArgs a = {};
    a.units = rows * groups; a.size = group_size; a.groups = groups; a.dtype = dtype; a.stride = x_stride;
    a.x = x; a.codes = codes; a.scales = scales;
    return launch_pack(a, (cudaStream_t)stream) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

int ssd_unpack_rows(int64_t rows, int32_t width, int32_t group_size, int32_t dtype, const void* codes, const float* scales,
                    void* out, void* stream) {
    const int rc = check_rows(rows, width, group_size, dtype, width, 1 << 30);
    if (rc != SSD_OK || rows == 0) return rc;
    if (!codes || !scales || !out) return SSD_ERR_INVALID_ARG;
    const int groups = width / group_size;
    const Mat in[] = {{codes, rows, width, width, 1}, {scales, rows, groups, groups, 4}};
    const Mat to[] = {{out, rows, width, width, elem(dtype)}};
    if (!on_elements(in) || !on_elements(to) || mixed(in, to)) return SSD_ERR_INVALID_ARG;
    PackArgs a = {};
    a.units = rows * groups; a.size = group_size; a.groups = groups; a.dtype = dtype; a.stride = width;
    a.codes = const_cast<void*>(codes); a.scales = const_cast<float*>(scales); a.out = out;
    return launch_unpack(a, (cudaStream_t)stream) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

int ssd_gate_norm_pack(const ssd_gate_norm_params_t* p, const void* y, const void* z, const float* weight, void* out, void* y_codes,
                       float* y_scales, void* z_codes, float* z_scales, void* stream) {
    const int rc = check_gate(p, p ? p->width : 0);
    if (rc != SSD_OK || p->rows == 0) return rc;
    if (!y || !z || !weight || !out || !y_codes || !y_scales || !z_codes || !z_scales) return SSD_ERR_INVALID_ARG;
    const int64_t r = p->rows, w = p->width, groups = w / p->group_size;
    const size_t es = elem(p->dtype);
    const Mat in[] = {{y, r, w, w, es}, {z, r, w, p->z_stride, es}, {weight, 1, w, w, 4}};
    const Mat to[] = {{out, r, w, w, es}, {y_codes, r, w, w, 1}, {z_codes, r, w, w, 1}, {y_scales, r, groups, groups, 4},
                      {z_scales, r, groups, groups, 4}};
    if (!on_elements(in) || !on_elements(to) || mixed(in, to)) return SSD_ERR_INVALID_ARG;
    BlockNormArgs a = {};
    a.units = r * groups; a.size = p->group_size; a.groups = (int)groups;
    a.dtype = a.residual_dtype = a.out_dtype = p->dtype;
    a.gate_stride = p->z_stride; a.scale = 1.f; a.eps = p->eps;
    a.x = y; a.gate = z; a.weight = weight; a.out = out;
    a.x_codes = y_codes; a.x_scales = y_scales; a.gate_codes = z_codes; a.gate_scales = z_scales;
    return launch_block_norm(a, (cudaStream_t)stream) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

size_t ssd_gate_norm_bwd_workspace_size(const ssd_gate_norm_params_t* p) {
    if (check_gate(p, p ? p->width : 0) != SSD_OK || p->rows == 0) return 0;
    return (size_t)block_norm_bwd_lines(p->rows, p->group_size, p->width / p->group_size) * p->width * sizeof(float);
}

int ssd_gate_norm_bwd(const ssd_gate_norm_params_t* p, const void* dout, const void* y, const float* y_scales, const void* z,
                      const float* z_scales, const float* weight, void* dy, void* dz, void* out, float* dweight,
                      void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = check_gate(p, p ? p->dz_stride : 0);
    if (rc != SSD_OK) return rc;
    const int64_t r = p->rows, w = p->width, groups = w / p->group_size;
    if (z_scales && p->z_stride != w) return SSD_ERR_INVALID_ARG;
    if (!dweight || !aligned(dweight, 4)) return SSD_ERR_INVALID_ARG;
    if (r == 0)
        return cudaMemsetAsync(dweight, 0, (size_t)w * 4, (cudaStream_t)stream) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
    if (!dout || !y || !z || !weight || !dy || !dz) return SSD_ERR_INVALID_ARG;
    const size_t es = elem(p->dtype), need = ssd_gate_norm_bwd_workspace_size(p);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) return SSD_ERR_WORKSPACE;
    const Mat in[] = {{dout, r, w, w, es}, {y, r, w, w, y_scales ? 1 : es}, {z, r, w, p->z_stride, z_scales ? 1 : es},
                      {y_scales, r, groups, groups, 4}, {z_scales, r, groups, groups, 4}, {weight, 1, w, w, 4}};
    const Mat to[] = {{dy, r, w, w, es}, {dz, r, w, p->dz_stride, es}, {out, r, w, w, es}, {dweight, 1, w, w, 4},
                      {workspace, 1, (int64_t)need, (int64_t)need, 1}};
    if (!on_elements(in) || !on_elements(to) || mixed(in, to)) return SSD_ERR_INVALID_ARG;
    BlockNormBwdArgs a = {};
    a.rows = r; a.size = p->group_size; a.groups = (int)groups;
    a.dtype = a.residual_dtype = p->dtype;
    a.gate_stride = p->z_stride; a.dgate_stride = p->dz_stride; a.scale = 1.f; a.eps = p->eps;
    a.dout = dout; a.x = y; a.x_scales = y_scales; a.gate = z; a.gate_scales = z_scales; a.weight = weight;
    a.dx = dy; a.dgate = dz; a.out = out; a.dweight = dweight; a.shares = (float*)workspace;
    a.share_lines = (int64_t)(need / (w * sizeof(float)));
    return launch_block_norm_bwd(a, (cudaStream_t)stream) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

int ssd_block_norm(const ssd_block_norm_params_t* p, const void* x, const void* gate, const void* residual, const float* weight,
                   const float* next_weight, void* residual_out, void* out, float* out_scales, void* x_codes, float* x_scales,
                   void* gate_codes, float* gate_scales, void* stream) {
    const int rc = check_block(p, gate != nullptr, false);
    if (rc != SSD_OK || p->rows == 0) return rc;
    const bool codes = p->out_dtype == SSD_E4M3;
    if (!x || !residual || !weight || !residual_out || (next_weight && (!out || (codes && !out_scales)))) return SSD_ERR_INVALID_ARG;
    if ((x_codes != nullptr) != (x_scales != nullptr) || (gate_codes != nullptr) != (gate_scales != nullptr) ||
        (gate_codes != nullptr) != (gate && x_codes))
        return SSD_ERR_INVALID_ARG;
    if (!next_weight) out = nullptr;
    if (!next_weight || !codes) out_scales = nullptr;
    const int64_t r = p->rows, w = p->width;
    const size_t es = elem(p->dtype), er = elem(p->residual_dtype);
    const Mat in[] = {{x, r, w, w, es}, {gate, r, w, p->gate_stride, es}, {weight, 1, w, w, 4}, {next_weight, 1, w, w, 4}};
    const Mat to[] = {{residual_out, r, w, w, er}, {out, r, w, w, elem(p->out_dtype)}, {out_scales, 1, r, r, 4}, {x_codes, r, w, w, 1},
                      {x_scales, 1, r, r, 4}, {gate_codes, r, w, w, 1}, {gate_scales, 1, r, r, 4}};
    const Mat res[] = {{residual, r, w, w, er}};
    if (!on_elements(in) || !on_elements(to) || !on_elements(res) || mixed(in, to)) return SSD_ERR_INVALID_ARG;
    for (const Mat& m : to)   // residual_out may be residual itself
        if (touch(m, res[0]) && m.p != residual) return SSD_ERR_INVALID_ARG;
    for (int k = 1; k < 7; ++k)
        if (to[k].p && touch(to[k], res[0])) return SSD_ERR_INVALID_ARG;
    BlockNormArgs a = {};
    a.units = r; a.size = p->width; a.groups = 1;
    a.dtype = p->dtype; a.residual_dtype = p->residual_dtype; a.out_dtype = p->out_dtype;
    a.gate_stride = p->gate_stride; a.scale = p->scale; a.eps = p->eps;
    a.x = x; a.gate = gate; a.residual = residual; a.weight = weight; a.next_weight = next_weight;
    a.residual_out = residual_out; a.out = out; a.out_scales = out_scales;
    a.x_codes = x_codes; a.x_scales = x_scales; a.gate_codes = gate_codes; a.gate_scales = gate_scales;
    return launch_block_norm(a, (cudaStream_t)stream) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

size_t ssd_block_norm_bwd_workspace_size(const ssd_block_norm_params_t* p) {
    if (check_block(p, false, false) != SSD_OK || p->rows == 0) return 0;
    return (size_t)block_norm_bwd_lines(p->rows, p->width, 1) * p->width * 2 * sizeof(float);
}

int ssd_block_norm_bwd(const ssd_block_norm_params_t* p, const void* dout, const void* dresidual_out, const void* x,
                       const float* x_scales, const void* gate, const float* gate_scales, const void* h, const float* h_scales,
                       const float* weight, const float* next_weight, void* dx, void* dgate, void* dresidual, float* dweight,
                       float* dnext_weight, void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = check_block(p, gate || dgate, gate || dgate);
    if (rc != SSD_OK) return rc;
    const int64_t r = p->rows, w = p->width;
    cudaStream_t st = (cudaStream_t)stream;
    if (gate_scales && p->gate_stride != w) return SSD_ERR_INVALID_ARG;
    if (!dweight || !aligned(dweight, 4) || !aligned(dnext_weight, 4) || (next_weight != nullptr) != (dnext_weight != nullptr))
        return SSD_ERR_INVALID_ARG;
    if (r == 0) {
        if (cudaMemsetAsync(dweight, 0, (size_t)w * 4, st) != cudaSuccess) return SSD_ERR_CUDA;
        if (dnext_weight && cudaMemsetAsync(dnext_weight, 0, (size_t)w * 4, st) != cudaSuccess) return SSD_ERR_CUDA;
        return SSD_OK;
    }
    if (!dresidual_out || !x || !weight || !dx || !dresidual || (gate != nullptr) != (dgate != nullptr) || (gate_scales && !gate) ||
        (next_weight != nullptr) != (dout != nullptr) || (next_weight && !h))
        return SSD_ERR_INVALID_ARG;
    if (!next_weight) {
        h = nullptr;
        h_scales = nullptr;
    }
    const size_t es = elem(p->dtype), er = elem(p->residual_dtype), need = ssd_block_norm_bwd_workspace_size(p);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) return SSD_ERR_WORKSPACE;
    const Mat in[] = {{dout, r, w, w, es}, {dresidual_out, r, w, w, er}, {x, r, w, w, x_scales ? 1 : es}, {x_scales, 1, r, r, 4},
                      {gate, r, w, p->gate_stride, gate_scales ? 1 : es}, {gate_scales, 1, r, r, 4}, {h, r, w, w, h_scales ? 1 : er},
                      {h_scales, 1, r, r, 4}, {weight, 1, w, w, 4}, {next_weight, 1, w, w, 4}};
    const Mat to[] = {{dx, r, w, w, es}, {dgate, r, w, p->dgate_stride, es}, {dresidual, r, w, w, er}, {dweight, 1, w, w, 4},
                      {dnext_weight, 1, w, w, 4}, {workspace, 1, (int64_t)need, (int64_t)need, 1}};
    if (!on_elements(in) || !on_elements(to) || mixed(in, to)) return SSD_ERR_INVALID_ARG;
    BlockNormBwdArgs a = {};
    a.rows = r; a.size = p->width; a.groups = 1;
    a.dtype = p->dtype; a.residual_dtype = p->residual_dtype;
    a.gate_stride = p->gate_stride; a.dgate_stride = p->dgate_stride; a.scale = p->scale; a.eps = p->eps;
    a.dout = dout; a.dres = dresidual_out; a.x = x; a.x_scales = x_scales; a.gate = gate; a.gate_scales = gate_scales;
    a.h = h; a.h_scales = h_scales; a.weight = weight; a.next_weight = next_weight;
    a.dx = dx; a.dgate = dgate; a.dres_out = dresidual; a.dweight = dweight; a.dnext_weight = dnext_weight;
    a.shares = (float*)workspace;
    a.share_lines = (int64_t)(need / (2 * w * sizeof(float)));
    return launch_block_norm_bwd(a, st) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"

// packed_api.cu -- the C ABI of the packed operators, the single-token step over slots and the gated
// norm's gradient (include/ssd.h): argument checks, workspace carving and dispatch.
#include <algorithm>

#include "../../include/ssd.h"
#include "api_util.cuh"
#include "norm_bwd.cuh"
#include "packed.cuh"
#include "slots.cuh"

using namespace ssd;

namespace {

int cuda_fail(const char *what)
{
    return api_fail(SSD_ERR_LAUNCH, "%s launch failed: %s", what, cudaGetErrorString(cudaGetLastError()));
}

int check_dtype(int dtype)
{
    return dtype == SSD_F32 || dtype == SSD_BF16 ? SSD_OK : api_fail(SSD_ERR_DTYPE, "unknown dtype %d", dtype);
}

int check_heads(int H, int P, int N, int G)
{
    if (H <= 0 || H > 65535 || G <= 0 || H % G != 0)
        return api_fail(SSD_ERR_SHAPE, "need 0 < H <= 65535, G > 0 and H %% G == 0 (H=%d, G=%d)", H, G);
    if (!api_pow2_dim(P) || !api_pow2_dim(N))
        return api_fail(SSD_ERR_SHAPE, "P and N must be 16, 32, 64 or 128 (P=%d, N=%d)", P, N);
    return SSD_OK;
}

int check_sizes(int nseq, int64_t total)
{
    if (nseq < 0 || total < 0 || total >= (1LL << 31) - 256)
        return api_fail(SSD_ERR_SHAPE, "nseq=%d and total=%lld must be >= 0, total below 2^31 - 256", nseq, (long long)total);
    return SSD_OK;
}

int check_plan(const void *plan, int nseq, int64_t total)
{
    const int rc = check_sizes(nseq, total);
    if (rc) return rc;
    if (!plan) return api_fail(SSD_ERR_NULL, "plan is NULL");
    if (!api_aligned(plan)) return api_fail(SSD_ERR_ALIGN, "plan must be 16-byte aligned");
    return SSD_OK;
}

// rows of `width` elements, 16-byte aligned, rs elements apart
int check_rows(const char *name, const void *ptr, int64_t rs, int64_t width, int dtype)
{
    if (!ptr) return api_fail(SSD_ERR_NULL, "%s is NULL", name);
    if (rs < width) return api_fail(SSD_ERR_STRIDE, "%s row stride %lld < row width %lld", name, (long long)rs, (long long)width);
    if (!api_aligned(ptr) || (rs * (int64_t)api_elem_size(dtype)) % 16 != 0)
        return api_fail(SSD_ERR_ALIGN, "%s must be 16-byte aligned with a 16-byte row stride", name);
    return SSD_OK;
}

int check_workspace(const void *ws, size_t have, size_t need)
{
    if (need == 0) return SSD_OK;
    if (!ws || have < need)
        return api_fail(SSD_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? have : (size_t)0);
    if (!api_aligned(ws, 256)) return api_fail(SSD_ERR_ALIGN, "workspace must be 256-byte aligned");
    return SSD_OK;
}

int status_or_fail(unsigned int **sp)
{
    *sp = api_status_ptr();
    return *sp ? SSD_OK : api_fail(SSD_ERR_LAUNCH, "no CUDA device available");
}

// Windows of the scan (packed.cuh): the tensor-core kernels run one CTA per SM and one (window, head
// pair) per CTA, so a pass takes about waves x (chunks per window + 2), the 2 standing for a CTA's fill
// and drain in chunks; more windows also mean more states handed on, so the fewest among equal costs
// are taken.  The chunk count is its upper bound (the device knows the true one and shares the
// chunks out evenly).  The CUDA-core kernels run two CTAs of one head each per SM.
struct ScanPlan {
    bool tc = false, carry = false;
    int nw = 0;
    size_t off_hin = 0, off_start = 0, off_dA = 0, bytes = 0;
};

ScanPlan scan_plan(int nseq, int64_t total, int64_t longest, int H, int P, int N, int G, int dtype)
{
    ScanPlan s;
    if (nseq <= 0 || H <= 0 || P <= 0 || N <= 0 || G <= 0) return s;
    // (without rows there is nothing that a TMA map could describe)
    s.tc = total > 0 && packed_scan_tc_shape(dtype, H, P, N, G) && !api_force_generic();
    const PackedLayout l = packed_layout(nseq, total);
    const int64_t chunks = s.tc ? l.m128 : l.m64;
    const int64_t units = s.tc ? H / 2 : H, slots = (int64_t)api_sm_count() * (s.tc ? 1 : 2);
    // a sequence is handed on between windows only if it has more than one chunk
    s.carry = std::min<int64_t>(longest, total) > (s.tc ? 128 : 64);
    int64_t best = -1;
    // (beyond four waves a window more changes nothing; chunks and windows x units fit 32 bits, whose quotients are the
    // cheaper ones: this runs in every call)
    const uint32_t nc = (uint32_t)chunks, un = (uint32_t)units, sl = (uint32_t)slots;
    const uint32_t most = (uint32_t)std::min<int64_t>(chunks, std::max<int64_t>(4, 4 * slots / units));
    for (uint32_t nw = 1; nw <= most; ++nw) {
        const uint32_t per = (nc + nw - 1) / nw, waves = (nw * un + sl - 1) / sl;
        const int64_t cost = (int64_t)waves * (per + 2);
        if (best < 0 || cost < best) { best = cost; s.nw = (int)nw; }
    }
    if (s.carry) {
        // S and the starts, the sums of dt A, and with many windows the entering states
        const size_t state = api_round256(sizeof(float) * (size_t)s.nw * H * P * N);
        const bool chain = s.nw > kMaxOwnWindows;
        s.off_start = state;
        s.off_hin = chain ? 2 * state : 0;
        s.off_dA = (chain ? 3 : 2) * state;
        s.bytes = s.off_dA + api_round256(sizeof(float) * (size_t)s.nw * H);
    }
    return s;
}

// Workspace of the scan's gradient: per chunk (room for m64) and head the states S then h, Gl then Gam;
// lam, dA and dD parts; per row and head dB and dC (all fp32)
struct ScanBwdPlan {
    int64_t nch = 0;
    size_t off_g = 0, off_lam = 0, off_pA = 0, off_pD = 0, off_dB = 0, off_dC = 0, bytes = 0;
};

ScanBwdPlan scan_bwd_plan(int nseq, int64_t total, int H, int P, int N)
{
    ScanBwdPlan s;
    if (nseq <= 0 || total < 0 || H <= 0 || P <= 0 || N <= 0) return s;
    s.nch = packed_layout(nseq, total).m64;
    const size_t states = api_round256(sizeof(float) * (size_t)H * s.nch * P * N);
    const size_t parts = api_round256(sizeof(float) * (size_t)H * s.nch);
    const size_t rows = api_round256(sizeof(float) * (size_t)total * H * N);
    s.off_g = states;
    s.off_lam = s.off_g + states;
    s.off_pA = s.off_lam + parts;
    s.off_pD = s.off_pA + parts;
    s.off_dB = s.off_pD + parts;
    s.off_dC = s.off_dB + rows;
    s.bytes = s.off_dC + rows;
    // (the tensor-core form's, where a call of these sizes may take it)
    if (P == 64 && N == 128 && total > 0) s.bytes = std::max(s.bytes, packed_grad_layout(nseq, total, H, api_sm_count()).bytes);
    return s;
}

}  // namespace

extern "C" {

size_t ssd_packed_plan_size(int nseq, int64_t total)
{
    return nseq < 0 || total < 0 ? 0 : packed_layout(nseq, total).bytes;
}

int ssd_packed_plan(const ssd_packed_plan_args *a, ssd_stream_t stream)
{
    if (!a) return api_fail(SSD_ERR_NULL, "args is NULL");
    int rc = check_plan(a->plan, a->nseq, a->total);
    if (rc) return rc;
    if (a->plan_bytes < packed_layout(a->nseq, a->total).bytes)
        return api_fail(SSD_ERR_WORKSPACE, "plan of %zu bytes needed, %zu given", packed_layout(a->nseq, a->total).bytes, a->plan_bytes);
    if (a->nseq > 0 && !a->cu_seqlens) return api_fail(SSD_ERR_NULL, "cu_seqlens is NULL");
    if (a->n_slots < 0 || a->max_seqlen < 0) return api_fail(SSD_ERR_SHAPE, "negative n_slots or max_seqlen");
    if (!a->slots && a->n_slots > 0 && a->n_slots < a->nseq)
        return api_fail(SSD_ERR_SHAPE, "without slots sequence i has slot i: n_slots=%d < nseq=%d", a->n_slots, a->nseq);
    if (a->slots && a->nseq > kPackedMaxSlotted)
        return api_fail(SSD_ERR_UNSUPPORTED, "a plan with slots takes at most %d sequences (nseq=%d)", kPackedMaxSlotted, a->nseq);
    PackedPlanParams p{};
    if ((rc = status_or_fail(&p.status))) return rc;
    p.nseq = a->nseq; p.total = a->total;
    p.max_seqlen = a->max_seqlen > 0 ? a->max_seqlen : a->total;
    p.cu = a->cu_seqlens; p.slots = a->slots; p.resume = a->resume;
    p.n_slots = a->slots ? a->n_slots : std::max(a->n_slots, a->nseq);
    p.plan = a->plan;
    if (launch_packed_plan(p, (cudaStream_t)stream)) return cuda_fail("plan");
    return api_ok();
}

int ssd_packed_conv_forward(const ssd_packed_conv_args *a, ssd_stream_t stream)
{
    if (!a) return api_fail(SSD_ERR_NULL, "args is NULL");
    int rc = check_dtype(a->dtype);
    if (rc || (rc = check_sizes(a->nseq, a->total))) return rc;
    const int V = a->dtype == SSD_BF16 ? 8 : 4;
    if (a->C_ch <= 0 || a->C_ch % V != 0) return api_fail(SSD_ERR_SHAPE, "C_ch=%d must be a positive multiple of %d", a->C_ch, V);
    if (a->nseq == 0) return api_ok();
    if ((rc = check_plan(a->plan, a->nseq, a->total))) return rc;
    if (a->total > 0) {
        if ((rc = check_rows("u", a->u, a->u_row_stride, a->C_ch, a->dtype))) return rc;
        if ((rc = check_rows("v", a->v, a->v_row_stride, a->C_ch, a->dtype))) return rc;
        if (a->u == a->v) return api_fail(SSD_ERR_SHAPE, "v must not overlap u");
    }
    if (!a->conv_w) return api_fail(SSD_ERR_NULL, "conv_w is NULL");
    if (!api_aligned(a->conv_w) || !api_aligned(a->tail_in) || !api_aligned(a->tail_out))
        return api_fail(SSD_ERR_ALIGN, "conv_w and the tails must be 16-byte aligned");
    PackedConvParams p{};
    if ((rc = status_or_fail(&p.status))) return rc;
    p.plan = packed_view(a->plan, a->nseq, a->total);
    p.u = a->u; p.urs = a->u_row_stride; p.w = a->conv_w; p.bias = a->conv_bias;
    p.tail_in = a->tail_in; p.tail_out = a->tail_out; p.v = a->v; p.vrs = a->v_row_stride; p.C_ch = a->C_ch;
    rc = launch_packed_conv(p, a->dtype, api_sm_count(), (cudaStream_t)stream);
    if (rc == 2) return api_fail(SSD_ERR_SHAPE, "packed conv grid too large");
    return rc ? cuda_fail("packed conv") : api_ok();
}

size_t ssd_packed_conv_backward_workspace_size(int nseq, int64_t total, int C_ch)
{
    if (nseq <= 0 || total < 0 || C_ch <= 0) return 0;
    const size_t parts = (size_t)packed_layout(nseq, total).m64 * C_ch;
    return api_round256(16 * parts) + api_round256(4 * parts);
}

int ssd_packed_conv_backward(const ssd_packed_conv_bwd_args *a, ssd_stream_t stream)
{
    if (!a) return api_fail(SSD_ERR_NULL, "args is NULL");
    int rc = check_dtype(a->dtype);
    if (rc || (rc = check_sizes(a->nseq, a->total))) return rc;
    const int HP = a->d_inner, GN = a->d_bc;
    if (HP <= 0 || GN <= 0 || HP % 8 != 0 || GN % 8 != 0 || HP > (1 << 22) || GN > (1 << 22))
        return api_fail(SSD_ERR_SHAPE, "d_inner=%d and d_bc=%d must be positive multiples of 8", HP, GN);
    const int C_ch = HP + 2 * GN;
    if (!a->conv_w || !a->dconv_w) return api_fail(SSD_ERR_NULL, "conv_w and dconv_w must not be NULL");
    const void *vec[] = {a->conv_w, a->dconv_w, a->tail_in, a->dx, a->dB, a->dC, a->dtail_out, a->du, a->dtail_in};
    for (const void *v : vec)
        if (!api_aligned(v)) return api_fail(SSD_ERR_ALIGN, "buffers must be 16-byte aligned");
    if (a->nseq == 0) {
        cudaError_t e = cudaMemsetAsync(a->dconv_w, 0, sizeof(float) * 4 * C_ch, (cudaStream_t)stream);
        if (e == cudaSuccess && a->dconv_bias) e = cudaMemsetAsync(a->dconv_bias, 0, sizeof(float) * C_ch, (cudaStream_t)stream);
        return e == cudaSuccess ? api_ok() : api_fail(SSD_ERR_LAUNCH, "%s", cudaGetErrorString(e));
    }
    if ((rc = check_plan(a->plan, a->nseq, a->total))) return rc;
    if (a->total > 0) {
        if ((rc = check_rows("u", a->u, a->u_row_stride, C_ch, a->dtype))) return rc;
        if (!a->dx || !a->dB || !a->dC || !a->du) return api_fail(SSD_ERR_NULL, "dx, dB, dC and du must not be NULL");
    }
    const size_t need = ssd_packed_conv_backward_workspace_size(a->nseq, a->total, C_ch);
    if ((rc = check_workspace(a->workspace, a->workspace_bytes, need))) return rc;
    PackedConvBwdParams p{};
    if ((rc = status_or_fail(&p.status))) return rc;
    p.plan = packed_view(a->plan, a->nseq, a->total);
    p.u = a->u; p.urs = a->u_row_stride; p.w = a->conv_w; p.bias = a->conv_bias; p.tail_in = a->tail_in;
    p.dx = a->dx; p.dB = a->dB; p.dC = a->dC; p.HP = HP; p.GN = GN; p.C_ch = C_ch;
    p.dtail_out = a->dtail_out; p.du = a->du; p.dtail_in = a->dtail_in; p.dw = a->dconv_w; p.dbias = a->dconv_bias;
    p.ws_dw = static_cast<float *>(a->workspace);
    p.ws_db = reinterpret_cast<float *>(static_cast<char *>(a->workspace) + api_round256(16 * (size_t)p.plan.m64 * C_ch));
    rc = launch_packed_conv_backward(p, a->dtype, (cudaStream_t)stream);
    if (rc == 2) return api_fail(SSD_ERR_SHAPE, "packed conv backward grid too large");
    return rc ? cuda_fail("packed conv backward") : api_ok();
}

size_t ssd_packed_scan_workspace_size(int nseq, int64_t total, int64_t max_seqlen, int H, int P, int N, int G, int dtype)
{
    if (nseq < 0 || total < 0) return 0;
    return scan_plan(nseq, total, max_seqlen > 0 ? max_seqlen : total, H, P, N, G, dtype).bytes;
}

int ssd_packed_scan_forward(const ssd_packed_scan_args *a, ssd_stream_t stream)
{
    if (!a) return api_fail(SSD_ERR_NULL, "args is NULL");
    int rc = check_dtype(a->dtype);
    if (rc || (rc = check_heads(a->H, a->P, a->N, a->G)) || (rc = check_sizes(a->nseq, a->total))) return rc;
    if (a->max_seqlen < 0) return api_fail(SSD_ERR_SHAPE, "negative max_seqlen");
    if (a->nseq == 0) return api_ok();
    if ((rc = check_plan(a->plan, a->nseq, a->total))) return rc;
    if (!a->A) return api_fail(SSD_ERR_NULL, "A is NULL");
    if (a->total > 0) {
        if ((rc = check_rows("x", a->x, a->x_row_stride, (int64_t)a->H * a->P, a->dtype))) return rc;
        if ((rc = check_rows("B", a->B, a->B_row_stride, (int64_t)a->G * a->N, a->dtype))) return rc;
        if ((rc = check_rows("C", a->C, a->C_row_stride, (int64_t)a->G * a->N, a->dtype))) return rc;
        if ((rc = check_rows("y", a->y, a->y_row_stride, (int64_t)a->H * a->P, a->dtype))) return rc;
        if (!a->dt) return api_fail(SSD_ERR_NULL, "dt is NULL");
        if (!api_aligned(a->dt, 8)) return api_fail(SSD_ERR_ALIGN, "dt must be 8-byte aligned");
    }
    if (!api_aligned(a->h_in) || !api_aligned(a->h_out)) return api_fail(SSD_ERR_ALIGN, "states must be 16-byte aligned");
    const ScanPlan sp = scan_plan(a->nseq, a->total, a->max_seqlen > 0 ? a->max_seqlen : a->total, a->H, a->P, a->N, a->G, a->dtype);
    if ((rc = check_workspace(a->workspace, a->workspace_bytes, sp.bytes))) return rc;
    PackedScanParams p{};
    if ((rc = status_or_fail(&p.status))) return rc;
    p.plan = packed_view(a->plan, a->nseq, a->total, a->max_seqlen > 0 ? a->max_seqlen : a->total);
    p.H = a->H; p.P = a->P; p.N = a->N; p.G = a->G;
    p.x = a->x; p.xrs = a->x_row_stride; p.B = a->B; p.Brs = a->B_row_stride; p.C = a->C; p.Crs = a->C_row_stride;
    p.dt = a->dt; p.A = a->A; p.D = a->D;
    p.dt_bias = a->dt_bias; p.dt_softplus = a->dt_softplus; p.dt_min = a->dt_min; p.dt_max = a->dt_max;
    p.h_in = a->h_in; p.h_out = a->h_out; p.y = a->y; p.yrs = a->y_row_stride;
    p.nw = sp.nw;
    if (sp.carry) {
        char *ws = static_cast<char *>(a->workspace);
        p.ws_S = reinterpret_cast<float *>(ws);
        p.ws_hin = sp.off_hin ? reinterpret_cast<float *>(ws + sp.off_hin) : nullptr;
        p.ws_start = reinterpret_cast<float *>(ws + sp.off_start);
        p.ws_dA = reinterpret_cast<float *>(ws + sp.off_dA);
    }
    p.wait_limit_ns = api_wait_limit_ns();
    p.test_drop_unit = api_take_drop_unit();
    rc = sp.tc ? launch_packed_scan_tc(p, sp.carry, (cudaStream_t)stream)
               : launch_packed_scan_generic(p, sp.carry, a->dtype, (cudaStream_t)stream);
    if (rc == 6) return api_fail(SSD_ERR_UNSUPPORTED, "no GPU kernel for this shape (P=%d N=%d)", a->P, a->N);
    return rc ? cuda_fail("packed scan") : api_ok();
}

size_t ssd_packed_scan_backward_workspace_size(int nseq, int64_t total, int H, int P, int N)
{
    return scan_bwd_plan(nseq, total, H, P, N).bytes;
}

int ssd_packed_scan_backward(const ssd_packed_scan_bwd_args *a, ssd_stream_t stream)
{
    if (!a) return api_fail(SSD_ERR_NULL, "args is NULL");
    cudaStream_t st = (cudaStream_t)stream;
    int rc = check_dtype(a->dtype);
    if (rc || (rc = check_heads(a->H, a->P, a->N, a->G)) || (rc = check_sizes(a->nseq, a->total))) return rc;
    if (!a->dA) return api_fail(SSD_ERR_NULL, "dA is NULL");
    if (a->nseq == 0) {
        cudaError_t e = cudaMemsetAsync(a->dA, 0, sizeof(float) * a->H, st);
        if (e == cudaSuccess && a->dD) e = cudaMemsetAsync(a->dD, 0, sizeof(float) * a->H, st);
        return e == cudaSuccess ? api_ok() : api_fail(SSD_ERR_LAUNCH, "%s", cudaGetErrorString(e));
    }
    if ((rc = check_plan(a->plan, a->nseq, a->total))) return rc;
    if (!a->A) return api_fail(SSD_ERR_NULL, "A is NULL");
    if (a->total > 0) {
        if ((rc = check_rows("x", a->x, a->x_row_stride, (int64_t)a->H * a->P, a->dtype))) return rc;
        if ((rc = check_rows("B", a->B, a->B_row_stride, (int64_t)a->G * a->N, a->dtype))) return rc;
        if ((rc = check_rows("C", a->C, a->C_row_stride, (int64_t)a->G * a->N, a->dtype))) return rc;
        if ((rc = check_rows("dy", a->dy, a->dy_row_stride, (int64_t)a->H * a->P, a->dtype))) return rc;
        if (!a->dt) return api_fail(SSD_ERR_NULL, "dt is NULL");
        if (!a->dx || !a->dB || !a->dC || !a->ddt) return api_fail(SSD_ERR_NULL, "dx, dB, dC and ddt must not be NULL");
    }
    const void *vec[] = {a->h_in, a->dh_out, a->dx, a->dB, a->dC, a->dh_in};
    for (const void *v : vec)
        if (!api_aligned(v)) return api_fail(SSD_ERR_ALIGN, "states and gradient outputs must be 16-byte aligned");
    const ScanBwdPlan pl = scan_bwd_plan(a->nseq, a->total, a->H, a->P, a->N);
    if ((rc = check_workspace(a->workspace, a->workspace_bytes, pl.bytes))) return rc;
    if (a->total > 0 && a->dtype == SSD_BF16 && a->P == 64 && a->N == 128) {
        const int ctas = api_sm_count();
        const PackedGradLayout l = packed_grad_layout(a->nseq, a->total, a->H, ctas);
        PackedGradParams q{};
        if ((rc = status_or_fail(&q.status))) return rc;
        q.plan = packed_view(a->plan, a->nseq, a->total);
        q.H = a->H; q.G = a->G;
        q.x = a->x; q.xrs = a->x_row_stride; q.B = a->B; q.Brs = a->B_row_stride; q.C = a->C; q.Crs = a->C_row_stride;
        q.dy = a->dy; q.dyrs = a->dy_row_stride;
        q.dt = a->dt; q.A = a->A; q.D = a->D; q.h_in = a->h_in; q.dh_out = a->dh_out;
        q.dx = a->dx; q.dB = a->dB; q.dC = a->dC; q.ddt = a->ddt; q.dA = a->dA; q.dD = a->dD; q.dh_in = a->dh_in;
        uint8_t *ws = static_cast<uint8_t *>(a->workspace);
        q.ws_img = ws;
        q.ws_part = reinterpret_cast<float *>(ws + l.off_part);
        q.ws_sums = reinterpret_cast<float *>(ws + l.off_sums);
        q.ws_pA = reinterpret_cast<float *>(ws + l.off_pA);
        q.ws_pD = reinterpret_cast<float *>(ws + l.off_pD);
        q.wait_limit_ns = api_wait_limit_ns();
        q.test_drop_unit = api_take_drop_unit();
        rc = launch_packed_grad_tc(q, ctas, st);
        if (rc == 2) return api_fail(SSD_ERR_SHAPE, "packed scan backward grid too large");
        return rc ? cuda_fail("packed scan backward") : api_ok();
    }
    int dev = 0, smem = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess)
        return api_fail(SSD_ERR_LAUNCH, "no CUDA device available");
    if (bwd_grad_smem_bytes(a->P, a->N) > (size_t)smem)
        return api_fail(SSD_ERR_UNSUPPORTED, "backward needs %zu bytes of shared memory, the device has %d", bwd_grad_smem_bytes(a->P, a->N), smem);
    const PackedPlan view = packed_view(a->plan, a->nseq, a->total);
    BwdParams p{};
    if ((rc = status_or_fail(&p.status))) return rc;
    p.b = 1; p.L = a->total; p.H = a->H; p.P = a->P; p.N = a->N; p.G = a->G;
    p.nch = pl.nch; p.cell_chunks = pl.nch;
    p.chunks = view.chunk64; p.seqs = view.seqs; p.hdr = view.hdr; p.nseq = a->nseq;
    p.x = a->x; p.xrs = a->x_row_stride; p.B = a->B; p.Brs = a->B_row_stride; p.C = a->C; p.Crs = a->C_row_stride;
    p.dy = a->dy; p.dyrs = a->dy_row_stride;
    p.dt = a->dt; p.A = a->A; p.D = a->D; p.h0 = a->h_in; p.dh_final = a->dh_out;
    p.dx = a->dx; p.dB = a->dB; p.dC = a->dC; p.ddt = a->ddt; p.dA = a->dA; p.dD = a->dD; p.dh0 = a->dh_in;
    char *ws = static_cast<char *>(a->workspace);
    p.ws_h = reinterpret_cast<float *>(ws);
    p.ws_g = reinterpret_cast<float *>(ws + pl.off_g);
    p.ws_lam = reinterpret_cast<float *>(ws + pl.off_lam);
    p.ws_pA = reinterpret_cast<float *>(ws + pl.off_pA);
    p.ws_pD = reinterpret_cast<float *>(ws + pl.off_pD);
    p.ws_dBh = reinterpret_cast<float *>(ws + pl.off_dB);
    p.ws_dCh = reinterpret_cast<float *>(ws + pl.off_dC);
    p.wait_limit_ns = api_wait_limit_ns();
    rc = launch_scan_backward(p, a->dtype, st);
    return rc ? cuda_fail("packed scan backward") : api_ok();
}

int ssd_decode_slots(const ssd_decode_slots_args *a, ssd_stream_t stream)
{
    if (!a) return api_fail(SSD_ERR_NULL, "args is NULL");
    int rc = check_dtype(a->dtype);
    if (rc || (rc = check_heads(a->H, a->P, a->N, a->G))) return rc;
    if (a->b < 0 || a->n_slots < 0) return api_fail(SSD_ERR_SHAPE, "negative b (%d) or n_slots (%d)", a->b, a->n_slots);
    if (a->b == 0) return api_ok();
    const int64_t C_ch = (int64_t)a->H * a->P + 2LL * a->G * a->N;
    if (!a->slots || !a->conv_w || !a->dt || !a->A || !a->tail_in || !a->tail_out || !a->h_in || !a->h_out)
        return api_fail(SSD_ERR_NULL, "slots, conv_w, dt, A, the tails and the states must not be NULL");
    if ((rc = check_rows("u", a->u, a->u_batch_stride, C_ch, a->dtype))) return rc;
    if ((rc = check_rows("y", a->y, a->y_batch_stride, (int64_t)a->H * a->P, a->dtype))) return rc;
    if (!api_aligned(a->conv_w) || !api_aligned(a->h_in) || !api_aligned(a->h_out) || !api_aligned(a->tail_in) || !api_aligned(a->tail_out))
        return api_fail(SSD_ERR_ALIGN, "conv_w, tails and states must be 16-byte aligned");
    SlotDecodeParams p{};
    if ((rc = status_or_fail(&p.status))) return rc;
    p.b = a->b; p.H = a->H; p.P = a->P; p.N = a->N; p.G = a->G; p.n_slots = a->n_slots; p.slots = a->slots;
    p.u = a->u; p.ubs = a->u_batch_stride; p.w = a->conv_w; p.bias = a->conv_bias;
    p.tail_in = a->tail_in; p.tail_out = a->tail_out; p.dt = a->dt; p.A = a->A; p.D = a->D;
    p.h_in = a->h_in; p.h_out = a->h_out; p.y = a->y; p.ybs = a->y_batch_stride;
    p.dt_bias = a->dt_bias; p.dt_softplus = a->dt_softplus; p.dt_min = a->dt_min; p.dt_max = a->dt_max;
    p.wait_limit_ns = api_wait_limit_ns();
    p.test_drop_unit = api_take_drop_unit();
    rc = launch_slot_decode(p, a->dtype, api_sm_count(), (cudaStream_t)stream);
    if (rc == 6) return api_fail(SSD_ERR_UNSUPPORTED, "no GPU kernel for this shape (b=%d H=%d P=%d N=%d G=%d)", a->b, a->H, a->P, a->N, a->G);
    return rc ? cuda_fail("slot decode") : api_ok();
}

size_t ssd_gated_rmsnorm_backward_workspace_size(int64_t rows, int d)
{
    if (rows <= 0 || d <= 0 || d % 8 != 0 || d > 8192) return 0;
    const NormBwdPlan pl = norm_bwd_plan(rows, d, api_sm_count());
    return api_round256(sizeof(float) * (size_t)pl.grid * pl.teams * d);
}

int ssd_gated_rmsnorm_backward(const ssd_gated_rmsnorm_bwd_args *a, ssd_stream_t stream)
{
    if (!a) return api_fail(SSD_ERR_NULL, "args is NULL");
    int rc = check_dtype(a->dtype);
    if (rc) return rc;
    const int d = a->d;
    if (a->rows < 0) return api_fail(SSD_ERR_SHAPE, "negative rows (%lld)", (long long)a->rows);
    if (d <= 0 || d % 8 != 0 || d > 8192) return api_fail(SSD_ERR_SHAPE, "d=%d must be a positive multiple of 8, at most 8192", d);
    const int group = a->group_size == 0 ? d : a->group_size;
    if (group <= 0 || group % 8 != 0 || d % group != 0)
        return api_fail(SSD_ERR_SHAPE, "group_size=%d must be a multiple of 8 that divides d=%d", a->group_size, d);
    if (!(a->eps >= 0.0f)) return api_fail(SSD_ERR_SHAPE, "eps must be >= 0");
    if (!a->dweight) return api_fail(SSD_ERR_NULL, "dweight is NULL");
    if (!api_aligned(a->dweight)) return api_fail(SSD_ERR_ALIGN, "dweight must be 16-byte aligned");
    if (a->rows == 0) {
        const cudaError_t e = cudaMemsetAsync(a->dweight, 0, sizeof(float) * d, (cudaStream_t)stream);
        return e == cudaSuccess ? api_ok() : api_fail(SSD_ERR_LAUNCH, "%s", cudaGetErrorString(e));
    }
    if ((rc = check_rows("dout", a->dout, a->dout_row_stride, d, a->dtype)) || (rc = check_rows("y", a->y, a->y_row_stride, d, a->dtype)) ||
        (rc = check_rows("z", a->z, a->z_row_stride, d, a->dtype)) || (rc = check_rows("dy", a->dy, a->dy_row_stride, d, a->dtype)) ||
        (rc = check_rows("dz", a->dz, a->dz_row_stride, d, a->dtype)))
        return rc;
    if (!a->weight) return api_fail(SSD_ERR_NULL, "weight is NULL");
    if (!api_aligned(a->weight)) return api_fail(SSD_ERR_ALIGN, "weight must be 16-byte aligned");
    const size_t need = ssd_gated_rmsnorm_backward_workspace_size(a->rows, d);
    if ((rc = check_workspace(a->workspace, a->workspace_bytes, need))) return rc;
    NormBwdParams p{};
    p.y = a->y; p.yrs = a->y_row_stride; p.z = a->z; p.zrs = a->z_row_stride; p.dout = a->dout; p.dors = a->dout_row_stride;
    p.w = a->weight; p.eps = a->eps; p.group = group;
    p.dy = a->dy; p.dyrs = a->dy_row_stride; p.dz = a->dz; p.dzrs = a->dz_row_stride; p.dw = a->dweight;
    p.ws = static_cast<float *>(a->workspace); p.rows = a->rows; p.d = d;
    return launch_gated_norm_backward(p, a->dtype, api_sm_count(), (cudaStream_t)stream) ? cuda_fail("norm backward") : api_ok();
}

}  // extern "C"

// packed_scan_generic.cu -- the selective scan over sequences laid end to end, on CUDA cores in fp32: both
// I/O types, any P and N, any heads.  (bf16 at P = 64, N = 128 has packed_scan_tc.cu.)
//
// The chunks (64 rows) of all sequences form one list, cut into nw windows of equal length; a CTA
// walks one window for one head, whatever sequences lie in it, so that work is shared out evenly
// whether the batch is one long sequence or many short ones.  In a chunk, with cs the running sum of
// dt A and h the state entering it:
//   y_i = sum_{j<=i} e^{cs_i - cs_j} dt_j (C_i . B_j) x_j + e^{cs_i} C_i h + D x_i
//   h   = e^{cs_last} h + sum_j dt_j e^{cs_last - cs_j} x_j B_j^T
// At a sequence's first chunk h is its slot's state or zero, after its last chunk h goes to its slot.
// Only a sequence that crosses from one window into the next has to be known beforehand: pass A forms
// what the window's chunks of that sequence leave (from a zero start), a chain over the windows turns
// that into the state entering each window, and pass C walks the windows.  Only differences of cs that
// are not positive are exponentiated.
// A thread forms 4 x 4 tiles of each product from shared memory.  The bound is the fp32 pipe and shared memory,
// 64 (N + P) + 4 N P multiply-adds per row and head over both passes, not the rows' bytes: 4000 rows of 8 heads
// (P = 64, N = 128) take 155 to 180 us, as they fall into sequences, 331 rows of 2 heads (P = N = 16) 21, most of it two launches.
#include <algorithm>

#include "packed.cuh"

namespace ssd {
namespace {

constexpr int kQ = 64;
constexpr int kThr = 256;
constexpr int kM = kQ + 1;        // row of the 64 x 64 matrix, padded

// acc[r][c] += sum_k a[(r0 + r rs) ars + k acs] b[k brs + (c0 + c cst) bcs]; the steps rs and cst put
// consecutive threads on consecutive rows or columns, so that a warp's reads fall in distinct banks
__device__ __forceinline__ void mm(float (&acc)[4][4], const float *a, int ars, int acs, const float *b, int brs, int bcs,
                                   int K, int r0, int rs, int c0, int cst)
{
#pragma unroll 4
    for (int k = 0; k < K; ++k) {
        float av[4], bv[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) av[r] = a[(r0 + r * rs) * ars + k * acs];
#pragma unroll
        for (int c = 0; c < 4; ++c) bv[c] = b[k * brs + (c0 + c * cst) * bcs];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[r][c] = fmaf(av[r], bv[c], acc[r][c]);
    }
}

__device__ __forceinline__ void zero(float (&acc)[4][4])
{
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[r][c] = 0.0f;
}

// rows in use of a chunk's tiles: the products take rows four at a time
__device__ __forceinline__ int tile_rows(int rows) { return (rows + 3) & ~3; }

// rows of cols elements into shared memory (row stride cols + 1), zeros past the chunk's rows up to tile_rows; cols is
// a multiple of 16 and rows are 16-byte aligned
template <typename T>
__device__ __forceinline__ void load_tile(float *dst, const T *src, int64_t rs, int rows, int cols)
{
    constexpr int V = 16 / (int)sizeof(T);
    const int nv = cols / V;
    for (int i = threadIdx.x; i < tile_rows(rows) * nv; i += kThr) {
        const int r = i / nv, c = i % nv * V;
        float *d = dst + r * (cols + 1) + c;
        if (r < rows) {
            const uint4 q = *reinterpret_cast<const uint4 *>(src + (int64_t)r * rs + c);
            if (sizeof(T) == 2) {
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) { d[2 * k] = bf16_lo(w[k]); d[2 * k + 1] = bf16_hi(w[k]); }
            } else {
                d[0] = __uint_as_float(q.x); d[1] = __uint_as_float(q.y);
                d[2] = __uint_as_float(q.z); d[3] = __uint_as_float(q.w);
            }
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) d[k] = 0.0f;
        }
    }
}

// dt of the chunk's rows and its running sum of dt A, by the first warp (two rows per lane)
__device__ __forceinline__ void load_dt(const PackedScanParams &p, int row0, int rows, int h, float *dts, float *cs)
{
    if (threadIdx.x >= 32) return;
    const int lane = threadIdx.x;
    const float A = p.A[h];
    float d[2], s[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int i = 2 * lane + k;
        d[k] = i < rows ? dt_effective(p.dt[((int64_t)row0 + i) * p.H + h], p.dt_bias, h, p.dt_softplus, p.dt_min, p.dt_max)
                        : 0.0f;
    }
    s[0] = d[0] * A;
    s[1] = fmaf(d[1], A, s[0]);
    float inc = s[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float t = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += t;
    }
    float ex = __shfl_up_sync(0xffffffffu, inc, 1);
    if (lane == 0) ex = 0.0f;
#pragma unroll
    for (int k = 0; k < 2; ++k) { dts[2 * lane + k] = d[k]; cs[2 * lane + k] = ex + s[k]; }
}

// h = e^{cs_last} h + sum_j (w o x)_j B_j^T for the chunk's rows in xs (already weighted) and bs
__device__ __forceinline__ void add_state(float *hs, const float *xw, const float *bs, int rows, int P, int N, float dec)
{
    const int ct = N / 4;
    for (int tile = threadIdx.x; tile < (P / 4) * ct; tile += kThr) {
        const int p0 = (tile / ct) * 4, n0 = tile % ct;
        float acc[4][4];
        zero(acc);
        mm(acc, xw, 1, P + 1, bs, N + 1, 1, rows, p0, 1, n0, ct);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float *e = hs + (p0 + r) * (N + 1) + n0 + c * ct;
                *e = fmaf(dec, *e, acc[r][c]);
            }
    }
}

// pass A: what the chunks of the sequence that leaves the window make of a zero state, and their decay
template <typename T>
__global__ void __launch_bounds__(kThr, 2) packed_state_kernel(PackedScanParams p)
{
    extern __shared__ float sm[];
    const int k = blockIdx.x, h = blockIdx.y, P = p.P, N = p.N;
    const int n = packed_n64(p.plan, p.status);
    const WindowTail t = window_tail<true>(p.plan, n, (n + p.nw - 1) / p.nw, k);
    if (!t.crosses) return;
    const int g = (int)((int64_t)h * p.G / p.H);
    float *xs = sm, *bs = xs + kQ * (P + 1), *hs = bs + kQ * (N + 1), *dts = hs + P * (N + 1), *cs = dts + kQ;
    for (int i = threadIdx.x; i < P * (N + 1); i += kThr) hs[i] = 0.0f;
    if (t.begins) {
        // the state that the sequence starts from, before its slot may be written
        const PackedSeq q = p.plan.seqs[t.seq];
        if (p.h_in && q.resume) {
            const float4 *src = reinterpret_cast<const float4 *>(p.h_in + ((int64_t)q.slot * p.H + h) * P * N);
            float4 *dst = reinterpret_cast<float4 *>(p.ws_start + ((int64_t)k * p.H + h) * P * N);
            for (int i = threadIdx.x; i < P * N / 4; i += kThr) dst[i] = src[i];
        }
    }
    float dA = 0.0f;
    for (int c = t.c0; c < t.c1; ++c) {
        const int4 d = p.plan.chunk64[c];
        const int rows = d.y & kChunkRows;
        __syncthreads();
        load_tile<T>(xs, reinterpret_cast<const T *>(p.x) + (int64_t)d.x * p.xrs + (int64_t)h * P, p.xrs, rows, P);
        load_tile<T>(bs, reinterpret_cast<const T *>(p.B) + (int64_t)d.x * p.Brs + (int64_t)g * N, p.Brs, rows, N);
        load_dt(p, d.x, rows, h, dts, cs);
        __syncthreads();
        const float tot = cs[kQ - 1];
        dA += tot;
        for (int i = threadIdx.x; i < rows * P; i += kThr) {
            const int j = i / P;
            xs[j * (P + 1) + i % P] *= dts[j] * expf(tot - cs[j]);
        }
        __syncthreads();
        add_state(hs, xs, bs, rows, P, N, expf(tot));
    }
    __syncthreads();
    float *dst = p.ws_S + ((int64_t)k * p.H + h) * P * N;
    for (int i = threadIdx.x; i < P * N; i += kThr) dst[i] = hs[i / N * (N + 1) + i % N];
    if (threadIdx.x == 0) p.ws_dA[(int64_t)k * p.H + h] = dA;
}

// pass C
template <typename T>
__global__ void __launch_bounds__(kThr) packed_output_kernel(PackedScanParams p)
{
    extern __shared__ float sm[];
    const int k = blockIdx.x, h = blockIdx.y, P = p.P, N = p.N, PN = P * N;
    const int n = packed_n64(p.plan, p.status);
    const int per = (n + p.nw - 1) / p.nw;
    const int64_t c0 = (int64_t)k * per, c1 = c0 + per < n ? c0 + per : n;
    if (c0 >= c1) return;
    const int g = (int)((int64_t)h * p.G / p.H);
    float *xs = sm, *bs = xs + kQ * (P + 1), *cq = bs + kQ * (N + 1), *hs = cq + kQ * (N + 1), *M = hs + P * (N + 1);
    float *dts = M + kQ * kM, *cs = dts + kQ;
    const float Dh = p.D ? p.D[h] : 0.0f;
    const int ctn = kQ / 4, ctp = P / 4;
    for (int64_t c = c0; c < c1; ++c) {
        const int4 d = p.plan.chunk64[c];
        const int rows = d.y & kChunkRows;
        __syncthreads();
        load_tile<T>(xs, reinterpret_cast<const T *>(p.x) + (int64_t)d.x * p.xrs + (int64_t)h * P, p.xrs, rows, P);
        load_tile<T>(bs, reinterpret_cast<const T *>(p.B) + (int64_t)d.x * p.Brs + (int64_t)g * N, p.Brs, rows, N);
        load_tile<T>(cq, reinterpret_cast<const T *>(p.C) + (int64_t)d.x * p.Crs + (int64_t)g * N, p.Crs, rows, N);
        load_dt(p, d.x, rows, h, dts, cs);
        if (c == c0 || (d.y & kChunkFirst)) {
            // a new sequence, or the window's first chunk of one that came before it
            if (d.y & kChunkFirst) {
                const float *src = window_start<true>(p, d, k, c1, h);
                for (int i = threadIdx.x; i < PN; i += kThr) hs[i / N * (N + 1) + i % N] = src ? src[i] : 0.0f;
            } else {
                for (int i = threadIdx.x; i < PN; i += kThr)
                    window_enter<true, 1>(p, d, k, per, h, i, 1, [&](int, float v) { hs[i / N * (N + 1) + i % N] = v; });
            }
        }
        __syncthreads();
        // M[i][j] = e^{cs_i - cs_j} dt_j (C_i . B_j), j <= i  (columns past the rows in use hold whatever lay there: masked)
        for (int tile = threadIdx.x; tile < (tile_rows(rows) / 4) * ctn; tile += kThr) {
            const int i0 = (tile / ctn) * 4, j0 = tile % ctn;
            float acc[4][4];
            zero(acc);
            if (j0 <= i0 + 3) mm(acc, cq, N + 1, 1, bs, 1, N + 1, N, i0, 1, j0, ctn);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int i = i0 + r, j = j0 + q * ctn;
                    M[i * kM + j] = j <= i ? acc[r][q] * expf(cs[i] - cs[j]) * dts[j] : 0.0f;
                }
        }
        __syncthreads();
        const float tot = cs[kQ - 1];
        T *yb = reinterpret_cast<T *>(p.y) + (int64_t)d.x * p.yrs + (int64_t)h * P;
        for (int tile = threadIdx.x; tile < (tile_rows(rows) / 4) * ctp; tile += kThr) {
            const int i0 = (tile / ctp) * 4, p0 = tile % ctp;
            float a1[4][4], a2[4][4];
            zero(a1);
            zero(a2);
            if (i0 < rows) {
                mm(a1, M, kM, 1, xs, P + 1, 1, i0 + 4, i0, 1, p0, ctp);
                mm(a2, cq, N + 1, 1, hs, 1, N + 1, N, i0, 1, p0, ctp);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = i0 + r;
                if (i >= rows) continue;
                const float e = expf(cs[i]);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int pp = p0 + q * ctp;
                    yb[(int64_t)i * p.yrs + pp] = from_f32<T>(fmaf(Dh, xs[i * (P + 1) + pp], fmaf(e, a2[r][q], a1[r][q])));
                }
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < rows * P; i += kThr) {
            const int j = i / P;
            xs[j * (P + 1) + i % P] *= dts[j] * expf(tot - cs[j]);
        }
        __syncthreads();
        add_state(hs, xs, bs, rows, P, N, expf(tot));
        if ((d.y & kChunkLast) && p.h_out && d.w >= 0) {
            __syncthreads();
            float *dst = p.h_out + ((int64_t)d.w * p.H + h) * PN;
            for (int i = threadIdx.x; i < PN; i += kThr) dst[i] = hs[i / N * (N + 1) + i % N];
        }
    }
}

// the state entering each window: st = the start of a sequence that begins in window k (its slot's state
// or zero), else the state that entered k;  h_in[k+1] = e^{dA_k} st + S_k.  One thread per four state elements.  What
// each window does is found by the threads side by side, kTails windows at a time, and S is loaded kAhead windows ahead
// (a window after the other waited for three dependent loads each: 37 us for 87 windows, 21 now).
constexpr int kTails = kThr, kAhead = 8;
template <bool k64>
__global__ void __launch_bounds__(kThr) packed_chain_kernel(PackedScanParams p)
{
    __shared__ int what[kTails];        // 1: a sequence leaves the window, 2: it begins there, 4: from the copy of its slot
    __shared__ float decay[kTails];
    const int PN = p.P * p.N, h = blockIdx.y;
    const int e = 4 * (blockIdx.x * blockDim.x + threadIdx.x);
    const int n = k64 ? packed_n64(p.plan, p.status) : packed_n128(p.plan, p.status);
    const int per = (n + p.nw - 1) / p.nw;
    const bool live = e < PN;
    const float4 zero4 = make_float4(0.f, 0.f, 0.f, 0.f);
    float4 st = zero4;
    for (int k0 = 0; k0 + 1 < p.nw; k0 += kTails) {
        const int kn = min(kTails, p.nw - 1 - k0);
        __syncthreads();
        if ((int)threadIdx.x < kn) {
            const int k = k0 + threadIdx.x;
            const WindowTail t = window_tail<k64>(p.plan, n, per, k);
            int w = 0;
            if (t.crosses) w = 1 | (t.begins ? 2 | (p.h_in && p.plan.seqs[t.seq].resume ? 4 : 0) : 0);
            what[threadIdx.x] = w;
            decay[threadIdx.x] = t.crosses ? expf(p.ws_dA[(int64_t)k * p.H + h]) : 0.0f;
        }
        __syncthreads();
        if (!live) continue;
        for (int i0 = 0; i0 < kn; i0 += kAhead) {
            float4 s[kAhead], b[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int w = i0 + i < kn ? what[i0 + i] : 0;
                const int64_t at = ((int64_t)(k0 + i0 + i) * p.H + h) * PN + e;
                s[i] = w & 1 ? *reinterpret_cast<const float4 *>(p.ws_S + at) : zero4;
                b[i] = w & 4 ? *reinterpret_cast<const float4 *>(p.ws_start + at) : zero4;
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int w = i0 + i < kn ? what[i0 + i] : 0;
                if (!(w & 1)) continue;
                if (w & 2) st = b[i];
                const float a = decay[i0 + i];
                st = make_float4(fmaf(a, st.x, s[i].x), fmaf(a, st.y, s[i].y), fmaf(a, st.z, s[i].z), fmaf(a, st.w, s[i].w));
                *reinterpret_cast<float4 *>(p.ws_hin + ((int64_t)(k0 + i0 + i + 1) * p.H + h) * PN + e) = st;
            }
        }
    }
}

template <typename T>
int launch_generic_t(const PackedScanParams &p, bool carry, cudaStream_t st)
{
    const int P = p.P, N = p.N;
    const size_t smA = sizeof(float) * ((size_t)kQ * (P + 1) + (size_t)kQ * (N + 1) + (size_t)P * (N + 1) + 2 * kQ);
    const size_t smC = smA + sizeof(float) * ((size_t)kQ * (N + 1) + (size_t)kQ * kM);
    static SmemLimit done_a, done_c;
    if (!allow_smem(packed_state_kernel<T>, (int)smA, done_a) || !allow_smem(packed_output_kernel<T>, (int)smC, done_c)) return 7;
    const dim3 grid((unsigned)p.nw, (unsigned)p.H);
    if (carry && p.nw > 1) {
        prof_begin(st, kKPackedState);
        packed_state_kernel<T><<<grid, kThr, smA, st>>>(p);
        prof_end(st, kKPackedState);
        const int rc = p.ws_hin ? launch_packed_chain(p, true, st) : 0;
        if (rc) return rc;
    }
    prof_begin(st, kKPackedOutput);
    packed_output_kernel<T><<<grid, kThr, smC, st>>>(p);
    prof_end(st, kKPackedOutput);
    return cudaGetLastError() == cudaSuccess ? 0 : 7;
}

}  // namespace

int launch_packed_chain(const PackedScanParams &p, bool k64, cudaStream_t st)
{
    const int quads = p.P * p.N / 4;
    const dim3 grid((unsigned)((quads + kThr - 1) / kThr), (unsigned)p.H);
    prof_begin(st, kKPackedChain);
    if (k64) packed_chain_kernel<true><<<grid, kThr, 0, st>>>(p);
    else packed_chain_kernel<false><<<grid, kThr, 0, st>>>(p);
    prof_end(st, kKPackedChain);
    return cudaGetLastError() == cudaSuccess ? 0 : 7;
}

int launch_packed_scan_generic(const PackedScanParams &p, bool carry, int dtype, cudaStream_t st)
{
    return dtype == 1 ? launch_generic_t<__nv_bfloat16>(p, carry, st) : launch_generic_t<float>(p, carry, st);
}

}  // namespace ssd

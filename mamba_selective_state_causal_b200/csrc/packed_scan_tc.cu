// packed_scan_tc.cu -- the selective scan over sequences laid end to end on the tensor cores: bf16 I/O,
// P = 64, N = 128, an even number of heads per group.
//
// The chunks (128 rows) of all sequences form one list, cut into nw windows of equal length
// (packed_scan_generic.cu has the decomposition); a CTA walks one window for two heads of a group, one
// CTA per SM, so that the pipeline fills and drains once per window and not once per sequence, and one
// long sequence and many short ones load the SMs alike.  In a chunk, with cs the running sum of dt A
// in log2 units and h the state entering it:
//   G  = C B^T                                          both heads
//   Pm = G o [e^{cs_i - cs_j} dt_j, j <= i]             TMEM -> TMEM, bf16
//   y  = Pm X + e^{cs_i} C h^T + D X                    h rounded to bf16 for this product only
//   h  = e^{cs_last} h + B^T (w o X),  w_j = dt_j e^{cs_last - cs_j}
// h stays in fp32 in TMEM, and leaves the kernel: w o X is split into its bf16 rounding and the bf16
// rounding of what that leaves, and both parts are multiplied (B is bf16 as given), so that a state
// is off by about 2^-17 of its terms instead of 2^-9.  y is rounded to bf16 anyway and takes single
// bf16 operands.
//
// A chunk of fewer than 128 rows is the last of its sequence.  Its loads bring rows of whatever
// lies behind it, possibly infinities or NaNs: the rows of X and B behind its end are cleared in shared
// memory before a product sums over them (C's and G's only reach rows of y that are not stored), dt
// is 0 there, and its y goes out row by row instead of by a TMA tile.
//
// All waits are bounded (tc::mbar_wait): on a timeout the CTA raises an abort flag, every thread
// unwinds, outstanding MMAs and loads are drained, TMEM is freed and the status word reports it.

#include <cuda.h>

#include "packed.cuh"
#include "scan_tc_util.cuh"

namespace ssd {
namespace {

using namespace tc;

constexpr int kQ = 128, kP = 64, kN = 128, kPN = kP * kN;

struct Maps {
    CUtensorMap x, B, C, y;
    CUtensorMap x64, B64;    // the same in boxes of 64 rows (pass A)
};

__device__ __forceinline__ void raise_timeout(const PackedScanParams &p, volatile int *abort)
{
    *abort = 1;
    atomicOr(p.status, kDevTimeout);
}

// w times 8 bf16 values: their bf16 rounding (on the integer pipe, ties away from zero; |w v| stays finite) and the
// bf16 rounding of what it leaves (on the conversion unit)
__device__ __forceinline__ void split8(uint4 v, float w, uint4 &hi, uint4 &lo)
{
    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
    uint32_t h[4], l[4];
    const float2 w2 = make_float2(w, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 q = mul2(unpack2(in[i]), w2);
        h[i] = pack_bf16x2_int(q.x, q.y);
        l[i] = pack_bf16x2(q.x - bf16_lo(h[i]), q.y - bf16_hi(h[i]));
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// dt as the scan uses it (dt_effective), with softplus(v) = max(v, 0) + log(1 + e^-|v|) from one exponential and one
// quotient: log(1 + e) = 2 artanh(s) = 2 (s + s^3 / 3 + s^5 / 5 + ..), s = e / (2 + e) <= 1/3, cut off at s^17 (1.4e-10 of
// it).  The scan warps take eight of them per lane and step: with log1p they, not the products, set pass A's pace.
__device__ __forceinline__ float dt_used(const PackedScanParams &p, float raw, float bias)
{
    float v = raw + bias;
    if (p.dt_softplus) {
        const float e = ex2(-fabsf(v) * kLog2e), q = __fdividef(e, 2.0f + e), q2 = q * q;
        float t = 1.0f / 17.0f;
        t = fmaf(t, q2, 1.0f / 15.0f);
        t = fmaf(t, q2, 1.0f / 13.0f);
        t = fmaf(t, q2, 1.0f / 11.0f);
        t = fmaf(t, q2, 1.0f / 9.0f);
        t = fmaf(t, q2, 1.0f / 7.0f);
        t = fmaf(t, q2, 1.0f / 5.0f);
        t = fmaf(t, q2, 1.0f / 3.0f);
        const float r = 2.0f * q;
        v = fmaxf(v, 0.0f) + fmaf(r * q2, t, r);
    }
    if (p.dt_max > 0.0f) v = fminf(fmaxf(v, p.dt_min), p.dt_max);
    return v;
}

// dt of rows 4 lane .. 4 lane + 3 of a chunk for the two heads ha, ha + 1, as the scan uses it (0 past its rows)
__device__ __forceinline__ void load_dt(const PackedScanParams &p, int row0, int rows, int lane, int ha, float2 (&d)[4])
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int i = 4 * lane + k;
        d[k] = i < rows ? *reinterpret_cast<const float2 *>(p.dt + ((int64_t)row0 + i) * p.H + ha) : make_float2(0.0f, 0.0f);
    }
}
__device__ __forceinline__ void use_dt(const PackedScanParams &p, int rows, int lane, float2 bias, float2 (&d)[4])
{
    if (!p.dt_bias && !p.dt_softplus && !(p.dt_max > 0.0f)) return;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (4 * lane + k < rows) {
            d[k].x = dt_used(p, d[k].x, bias.x);
            d[k].y = dt_used(p, d[k].y, bias.y);
        }
}

// Sums of dt A (log2 units) over the chunk's rows AFTER each row (rows 4 lane .. 4 lane + 3 of both heads), and over all
// of its rows.  Taken from the chunk's end, they are exact where they matter: a row near the end weighs most in the
// state that leaves the chunk, and its sum is short (differences of sums from the front were off by the rounding of the
// whole chunk's sum, three times the error of all else at A = -16).
__device__ __forceinline__ void chunk_sums(const float2 (&d)[4], float A2a, float A2b, int lane, float (&sa)[4], float (&sb)[4],
                                           float &ta, float &tb)
{
    float a[4], b[4], ia = 0.0f, ib = 0.0f;
#pragma unroll
    for (int k = 3; k >= 0; --k) {
        a[k] = d[k].x * A2a; ia += a[k];
        b[k] = d[k].y * A2b; ib += b[k];
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float qa = __shfl_down_sync(0xffffffffu, ia, o), qb = __shfl_down_sync(0xffffffffu, ib, o);
        if (lane + o < 32) { ia += qa; ib += qb; }
    }
    ta = __shfl_sync(0xffffffffu, ia, 0);
    tb = __shfl_sync(0xffffffffu, ib, 0);
    sa[3] = __shfl_down_sync(0xffffffffu, ia, 1);
    sb[3] = __shfl_down_sync(0xffffffffu, ib, 1);
    if (lane == 31) { sa[3] = 0.0f; sb[3] = 0.0f; }
#pragma unroll
    for (int k = 2; k >= 0; --k) { sa[k] = sa[k + 1] + a[k + 1]; sb[k] = sb[k + 1] + b[k + 1]; }
}

// =============================================================== pass A
// One CTA per (window, head pair) that a sequence leaves: S[n][(h,p)] = sum_j B[j][n] (w_h o X_h)[j][p] over the
// window's chunks of that sequence (all of 128 rows), accumulated in TMEM.  The rows are walked
// backwards, 64 at a time, so that the decay from each to the window's end is known when it is scaled.
// Warps 0..15 scale X into its two bf16 parts (the rounding in place, the rest beside it), warp 16 issues the
// products, warp 17 the loads, warps 18 and 19 run the dt sums of a head each, ahead of the others.
// 65536 rows of 32 heads: 97 to 99 us, 0.8 us per step of 64 rows and two heads, which the chain of load, scaling and
// product through five stages sets; the bytes (x and B once) would take 44.
constexpr int kStagesA = 5;
constexpr int kQA = 64;                  // rows of a step
constexpr uint32_t kBoxA = kQA * 128;    // 64 rows x 64 columns of bf16
constexpr int kScaleWarpsA = 16;
constexpr int kThreadsA = 32 * (kScaleWarpsA + 4);
constexpr uint32_t kStageA = 4 * kBoxA;   // B (2 boxes), X of head a and b

struct SmemA {
    uint8_t stage[kStagesA][kStageA];
    uint8_t rem[2][2 * kBoxA];            // the remainders of w o X of two steps
    float w[kStagesA][2][kQA];
    uint64_t full[kStagesA], w_ready[kStagesA], xw_ready[kStagesA], empty[kStagesA];
    uint64_t acc_full, fin;
    uint32_t tmem;
    int abort;
};

__global__ void __launch_bounds__(kThreadsA, 1)
packed_state_tc_kernel(const __grid_constant__ Maps maps, const PackedScanParams p)
{
    extern __shared__ __align__(1024) uint8_t sma_raw[];
    SmemA &s = *reinterpret_cast<SmemA *>((reinterpret_cast<uintptr_t>(sma_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hpairs = p.H / 2;
    const int ha = 2 * (int)(blockIdx.x % hpairs), k = (int)(blockIdx.x / hpairs);
    const int n = packed_n128(p.plan, p.status);
    const WindowTail wt = window_tail<false>(p.plan, n, (n + p.nw - 1) / p.nw, k);
    if (!wt.crosses) return;
    const int g = (int)((int64_t)ha * p.G / p.H);
    const int nc = (wt.c1 - wt.c0) * (kQ / kQA);     // steps
    const int row0 = p.plan.chunk128[wt.c0].x;       // the chunks are consecutive rows of one sequence
    const uint64_t lim = p.wait_limit_ns;

    if (wt.begins) {
        // the state that the sequence starts from, before its slot may be written
        const PackedSeq sq = p.plan.seqs[wt.seq];
        if (p.h_in && sq.resume) {
            const float4 *src = reinterpret_cast<const float4 *>(p.h_in + ((int64_t)sq.slot * p.H + ha) * kPN);
            float4 *dst = reinterpret_cast<float4 *>(p.ws_start + ((int64_t)k * p.H + ha) * kPN);
            for (int i = threadIdx.x; i < 2 * kPN / 4; i += kThreadsA) dst[i] = src[i];
        }
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStagesA; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.w_ready[i], 2);
            mbar_init(&s.xw_ready[i], kScaleWarpsA / 2);
            mbar_init(&s.empty[i], 1);
        }
        mbar_init(&s.acc_full, 1);
        mbar_init(&s.fin, 1);
        s.abort = 0;
        fence_mbar_init();
        prefetch_tmap(&maps.x64);
        prefetch_tmap(&maps.B64);
    }
    if (warp == 0) { tmem_alloc(&s.tmem, 128); tmem_relinquish(); }
    __syncthreads();
    tc_fence_after();
    const uint32_t tS = s.tmem;
    volatile int *abort = &s.abort;
    const bool live = (int64_t)blockIdx.x != p.test_drop_unit;

    if (warp < kScaleWarpsA) {
        // warps 0..7 take the even steps, 8..15 the odd ones
        const int hd = (warp >> 2) & 1, ti = 32 * (warp & 3) + lane, j = ti >> 1, c0 = 4 * (ti & 1);
        bool ok = true;
        for (int it = warp >> 3; it < nc; it += 2) {
            const int st = it % kStagesA;
            const uint32_t ph = (uint32_t)(it / kStagesA) & 1;
            // (the remainders' place is free once the step two before has been multiplied)
            ok = ewait(&s.w_ready[st], ph, abort, lim) &&
                 (it < 2 || ewait(&s.empty[(it - 2) % kStagesA], (uint32_t)((it - 2) / kStagesA) & 1, abort, lim)) &&
                 ewait(&s.full[st], ph, abort, lim);
            if (!ok) break;
            const float w = s.w[st][hd][j];
            uint8_t *xrow = s.stage[st] + (2 + hd) * kBoxA, *lrow = s.rem[it & 1] + hd * kBoxA;
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) {
                const uint32_t o = swz(j, c0 + cc);
                uint4 hi, lo;
                split8(lds128(xrow + o), w, hi, lo);
                sts128(xrow + o, hi);
                sts128(lrow + o, lo);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.xw_ready[st]);
        }
        if (!ok) {
            if (lane == 0) raise_timeout(p, abort);
        } else if (warp < 8) {
            if (ewait(&s.acc_full, 0, abort, lim)) {
                // lane quarter q holds state rows n = 32 q .. 32 q + 31; warp 4 hq + q takes head ha + hq
                tc_fence_after();
                const int q = warp & 3, hq = warp >> 2, nn = 32 * q + lane;
                const uint32_t lane_base = (uint32_t)(32 * q) << 16;
                float *dst = p.ws_S + ((int64_t)k * p.H + ha + hq) * kPN + nn;
#pragma unroll
                for (int c32 = 0; c32 < 2; ++c32) {
                    uint32_t a[32];
                    tmem_ld32(tS + lane_base + 64 * hq + 32 * c32, a);
                    tmem_wait_ld(a);
#pragma unroll
                    for (int pp = 0; pp < 32; ++pp) dst[(int64_t)(32 * c32 + pp) * kN] = __uint_as_float(a[pp]);
                }
            } else if (lane == 0) {
                raise_timeout(p, abort);
            }
        }
    } else if (warp == kScaleWarpsA) {
        // ================================================= issuing warp (the whole warp waits, lane 0 issues)
        const uint32_t id_s = idesc_bf16(128, 128, 1, 1);   // A = B^T (MN-major), B = w o X (MN-major)
        const uint32_t tSu = uniform(tS);
        bool ok = live;
        for (int it = 0; ok && it < nc; ++it) {
            const int st = it % kStagesA;
            ok = ewait(&s.xw_ready[st], (uint32_t)(it / kStagesA) & 1, abort, lim);
            if (!ok) break;
            tc_fence_after();
            const uint32_t sb = smem_u32(s.stage[0]) + uniform(st) * kStageA, sr = smem_u32(s.rem[0]) + uniform(it & 1) * 2 * kBoxA;
            if (elect_one()) {
                const uint64_t db = smem_desc(sb, kBoxA, 1024);
                const uint64_t dh = smem_desc(sb + 2 * kBoxA, kBoxA, 1024), dl = smem_desc(sr, kBoxA, 1024);
#pragma unroll
                for (int kk = 0; kk < kQA / 16; ++kk)
                    mma_ss(tSu, db + (uint64_t)(kk * 128), dh + (uint64_t)(kk * 128), id_s, it > 0 || kk > 0);
#pragma unroll
                for (int kk = 0; kk < kQA / 16; ++kk) mma_ss(tSu, db + (uint64_t)(kk * 128), dl + (uint64_t)(kk * 128), id_s, true);
                mma_commit(&s.empty[st]);
            }
            __syncwarp();
        }
        __syncwarp();
        if (elect_one()) {
            if (live && !ok) raise_timeout(p, abort);
            mma_commit(&s.acc_full);
            mma_commit(&s.fin);
            mbar_wait(&s.fin, 0, nullptr, 100000000ull);
        }
        __syncwarp();
    } else if (warp == kScaleWarpsA + 1) {
        // ================================================= loading warp: a stage is refilled once its product has read it
        // (kept off the issuing warp, which would otherwise wait for each product to end)
        int issued = 0;
        bool ok = live;
        for (int it = 0; ok && it < nc; ++it) {
            const int st = it % kStagesA;
            if (it >= kStagesA) {
                ok = ewait(&s.empty[st], (uint32_t)(it / kStagesA - 1) & 1, abort, lim);
                if (!ok) break;
            }
            if (lane == 0) {
                const int t0 = row0 + (nc - 1 - it) * kQA;
                uint8_t *sb = s.stage[st];
                mbar_arrive_expect_tx(&s.full[st], 4 * kBoxA);
                tma_load_3d(sb, &maps.B64, &s.full[st], g * kN, t0, 0);
                tma_load_3d(sb + kBoxA, &maps.B64, &s.full[st], g * kN + 64, t0, 0);
                tma_load_3d(sb + 2 * kBoxA, &maps.x64, &s.full[st], ha * kP, t0, 0);
                tma_load_3d(sb + 3 * kBoxA, &maps.x64, &s.full[st], (ha + 1) * kP, t0, 0);
            }
            ++issued;
            __syncwarp();
        }
        if (lane == 0) {
            if (live && !ok) raise_timeout(p, abort);
            // the last load issued into each stage lands before the CTA's shared memory is released (an
            // earlier one into the same stage has been waited on by the scaling warps)
            if (*abort)
                for (int it = issued > kStagesA ? issued - kStagesA : 0; it < issued; ++it)
                    mbar_wait(&s.full[it % kStagesA], (uint32_t)(it / kStagesA) & 1, nullptr, 100000000ull);
        }
        __syncwarp();
    } else {
        // one warp per head: w of every chunk, ready in registers before its place is free
        const int hd = warp - kScaleWarpsA - 2, h = ha + hd;
        const float A2 = p.A[h] * kLog2e;
        const bool used = p.dt_bias || p.dt_softplus || p.dt_max > 0.0f;
        const float bias = p.dt_bias ? p.dt_bias[h] : 0.0f;
        float suf = 0.0f;                   // sum of dt A (log2 units) after the chunks scanned so far
        // dt of four steps at a time, loaded while the four before them are used
        float dn[4][2], dc[4][2];
        auto load = [&](int it0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int it = min(it0 + e, nc - 1);
                const float *src = p.dt + ((int64_t)row0 + (int64_t)(nc - 1 - it) * kQA + 2 * lane) * p.H + h;
                dn[e][0] = src[0];
                dn[e][1] = src[p.H];
            }
        };
        bool ok = live;
        load(0);
#pragma unroll 1
        for (int it0 = 0; ok && it0 < nc; it0 += 4) {
#pragma unroll
            for (int e = 0; e < 4; ++e) { dc[e][0] = dn[e][0]; dc[e][1] = dn[e][1]; }
            if (it0 + 4 < nc) load(it0 + 4);
            // the four steps' sums side by side: one step's chain of shuffles alone took longer than its product
            float d[4][2], a1[4], inc[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    d[e][q] = used ? dt_used(p, dc[e][q], bias) : dc[e][q];
                a1[e] = d[e][1] * A2;
                inc[e] = a1[e] + d[e][0] * A2;
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float t = __shfl_down_sync(0xffffffffu, inc[e], o);
                    if (lane + o < 32) inc[e] += t;
                }
            float2 w2[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float after = __shfl_down_sync(0xffffffffu, inc[e], 1);
                if (lane == 31) after = 0.0f;
                const float tot = __shfl_sync(0xffffffffu, inc[e], 0);
                // decay from row j (exclusive) to the window's end: the rows after it in the step, and the later steps
                w2[e] = make_float2(d[e][0] * ex2(after + a1[e] + suf), d[e][1] * ex2(after + suf));
                if (it0 + e < nc) suf += tot;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int it = it0 + e;
                if (it >= nc) break;
                const int st = it % kStagesA;
                if (it >= kStagesA) {           // the scaling warps are done with w[st]
                    ok = ewait(&s.xw_ready[st], (uint32_t)(it / kStagesA - 1) & 1, abort, lim);
                    if (!ok) break;
                }
                reinterpret_cast<float2 *>(s.w[st][hd])[lane] = w2[e];
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.w_ready[st]);
            }
        }
        if (lane == 0) {
            if (live && !ok) raise_timeout(p, abort);
            if (ok && !*abort) p.ws_dA[(int64_t)k * p.H + h] = suf * kLn2;
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tS, 128);
}

// =============================================================== pass C
// One CTA per (window, head pair): 16 compute warps, an issuing warp, a store warp, a B/C warp and a scan warp.
// The output accumulator T of a chunk first receives Ys = C [h_a | h_b]^T, which the compute warps scale
// row by row by e^{cs_i}; Y = Pm X then accumulates onto it, so the epilogue only adds D x.  Per chunk c:
//   issuing warp: Pm written and T scaled -> Y_a, Y_b onto T; w o X ready -> S, both of its parts, onto the
//       state H; the state of chunk c+1 written -> Ys of chunk c+1
//   B/C warp: products done -> the B/C slot refilled with chunk c+2; G of chunk c+2 after Y of chunk c+1
//   store warp: y staged -> stored (TMA, or row by row for a short chunk), X of chunk c+2 into its slot
//   compute warp (lane quarter q = warp & 3, column slice cs = warp >> 2 of the 128 (head, p) columns):
//       T scaled; under Y, w o X into the C half of the B/C slot (spent once G and Ys have read C) and its
//       remainder into hp (spent once Ys has read it); under S, y and the masked decay of chunk c+1; then the state
//       step of chunk c+1 -- or, where a sequence ends, its state to its slot and the next one's start in its place
//   scan warp: the running sums of chunk c+1, ready in registers, into shared memory as soon as every warp has
//       used those of chunk c; it also starts the slot's state of a sequence about to begin into L2
// A chunk of fewer than 128 rows takes only the K-steps (of 16 rows) of Y and S that have rows.
// What bounds it: the compute warps' chain of steps, 4.7 us per chunk and head pair (T 0.3, w o X 0.7, waiting for Y
// 0.4, y 0.6, decay 1.3, state 0.9, waiting for Ys 0.3), with the tensor pipe active for 32 % of the time at 65536 rows
// and 25 % at 12001; the bytes would take 1.6.  65536 rows of 32 heads: 258 us, 8191 rows in 256 sequences 157.
// TMEM (512 columns): R0 = 0..127 G; R1 = 128..255 Pm_a | Pm_b (bf16); T = 256..383; H = 384..511 (rows n).
constexpr int kComputeWarps = 16;
constexpr int kThreadsC = 32 * (kComputeWarps + 4);

struct SmemC {
    uint8_t bc[2][4 * kBox];   // ring slot: C box 0, C box 1, B box 0, B box 1; later w o X in the C half
    uint8_t x[2][2 * kBox];    // X slot: head a box, head b box (X, then y)
    uint8_t hp[2 * kBox];      // bf16 state of head a, head b (rows n, cols p); later the remainder of w o X
    float cvs[2][kQ];          // sums of dt A (log2 units) after each row of the chunk, per head
    float dvs[2][kQ];          // dt, per head
    float fs[2][3 * 32];       // dt_j e^{cs_end(J) - cs_j} for the 32-row blocks J = 0..2
    int4 desc[2];              // descriptors of chunks c and c+1
    float tot[2];              // sums of dt A over the chunk
    uint64_t full_bc[2], full_x[2], g_done, ys_done, ymma_done, mma_done[2];
    uint64_t fin, fin2;
    uint64_t pmw, pm_ready, xw_ready, ys_go, scan_ready;
    uint64_t y_ready[2];
    uint32_t tmem;
    int abort;
};

__global__ void __launch_bounds__(kThreadsC, 1)
packed_output_tc_kernel(const __grid_constant__ Maps maps, const PackedScanParams p)
{
    extern __shared__ __align__(1024) uint8_t smc_raw[];
    SmemC &s = *reinterpret_cast<SmemC *>(smc_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int HP = p.H >> 1;
    const int ha = 2 * (int)(blockIdx.x % HP);   // head a; head b = ha + 1
    const int k = (int)(blockIdx.x / HP);
    const int g = (int)((int64_t)ha * p.G / p.H);
    const int nall = packed_n128(p.plan, p.status);
    const int per = (nall + p.nw - 1) / p.nw;
    const int64_t first = (int64_t)k * per;
    const int nc = (int)min((int64_t)per, nall - first);      // chunks of this window
    if (nc <= 0) return;
    const int4 *chunks = p.plan.chunk128 + first;
    const uint64_t lim = p.wait_limit_ns;

    // the 128B-swizzled tiles need a 1024-byte aligned base (no room to pad)
    if (smem_u32(smc_raw) & 1023u) {
        if (tid == 0) atomicOr(p.status, kDevUnsupported);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) { mbar_init(&s.full_bc[i], 1); mbar_init(&s.full_x[i], 1); }
        mbar_init(&s.g_done, 1);
        mbar_init(&s.ys_done, 1);
        mbar_init(&s.ymma_done, 1);
        mbar_init(&s.mma_done[0], 1);
        mbar_init(&s.mma_done[1], 1);
        mbar_init(&s.fin, 1);
        mbar_init(&s.fin2, 1);
        mbar_init(&s.pmw, kComputeWarps);
        mbar_init(&s.pm_ready, kComputeWarps);
        mbar_init(&s.xw_ready, kComputeWarps);
        mbar_init(&s.ys_go, kComputeWarps);
        mbar_init(&s.y_ready[0], kComputeWarps);
        mbar_init(&s.y_ready[1], kComputeWarps);
        mbar_init(&s.scan_ready, 1);
        s.abort = 0;
        fence_mbar_init();
        prefetch_tmap(&maps.x);
        prefetch_tmap(&maps.B);
        prefetch_tmap(&maps.C);
        prefetch_tmap(&maps.y);
    }
    if (warp == 0) { tmem_alloc(&s.tmem, 512); tmem_relinquish(); }
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = uniform(s.tmem);
    const uint32_t tG = tm, tPm = tm + 128, tT = tm + 256, tH = tm + 384;
    volatile int *abort = &s.abort;
    const bool live = (int64_t)blockIdx.x != p.test_drop_unit;

    if (warp < kComputeWarps) {
        // ================================================= compute warps
        const int q = warp & 3, cs = warp >> 2, hd = cs >> 1, p0 = 32 * (cs & 1);
        const int r = 32 * q + lane;             // chunk row / TMEM lane / state row n
        const uint32_t lane_base = (uint32_t)(32 * q) << 16;
        const int hh = ha + hd;
        auto fail = [&]() { if (lane == 0) raise_timeout(p, abort); };

        // thread (n = r, cs) owns h[p0 .. p0 + 31][n] of head hh
        auto store_state = [&](int slot, const uint32_t (&hv)[32]) {
            float *dst = p.h_out + ((int64_t)slot * p.H + hh) * kPN + (int64_t)p0 * kN + r;
#pragma unroll
            for (int pp = 0; pp < 32; ++pp) dst[pp * kN] = __uint_as_float(hv[pp]);
        };

        const float Dh = p.D ? p.D[hh] : 0.0f;

        // hv = the state entering a chunk: its bf16 copy feeds C h^T, then H = e^{cs_last} h, to which S is added
        auto state_step = [&](uint32_t (&hv)[32]) {
            uint8_t *dst = s.hp + hd * kBox;
#pragma unroll
            for (int c4 = 0; c4 < 4; ++c4) {
                uint4 v;
                v.x = pack_bf16x2(__uint_as_float(hv[8 * c4 + 0]), __uint_as_float(hv[8 * c4 + 1]));
                v.y = pack_bf16x2(__uint_as_float(hv[8 * c4 + 2]), __uint_as_float(hv[8 * c4 + 3]));
                v.z = pack_bf16x2(__uint_as_float(hv[8 * c4 + 4]), __uint_as_float(hv[8 * c4 + 5]));
                v.w = pack_bf16x2(__uint_as_float(hv[8 * c4 + 6]), __uint_as_float(hv[8 * c4 + 7]));
                sts128(dst + swz(r, (p0 >> 3) + c4), v);
            }
            const float dec = ex2(s.tot[hd]);
#pragma unroll
            for (int pp = 0; pp < 32; pp += 2) {
                const float2 q2 = mul2(make_float2(__uint_as_float(hv[pp]), __uint_as_float(hv[pp + 1])), make_float2(dec, dec));
                hv[pp] = __float_as_uint(q2.x); hv[pp + 1] = __float_as_uint(q2.y);
            }
            tmem_st32(tH + lane_base + 32 * cs, hv);
        };
        auto state_zero = [&]() {
            uint8_t *dst = s.hp + hd * kBox;
            uint32_t z[32];
#pragma unroll
            for (int pp = 0; pp < 32; ++pp) z[pp] = 0u;
#pragma unroll
            for (int c4 = 0; c4 < 4; ++c4) sts128(dst + swz(r, (p0 >> 3) + c4), make_uint4(0u, 0u, 0u, 0u));
            tmem_st32(tH + lane_base + 32 * cs, z);
        };
        // y = T + D x for 16 columns -> bf16, in place over x in the X slot (same swizzle as the y map)
        auto y_half = [&](uint8_t *xs, const uint32_t (&tv)[16], int hf) {
            uint8_t *dst = xs + hd * kBox;
#pragma unroll
            for (int c2 = 0; c2 < 2; ++c2) {
                uint8_t *a = dst + swz(r, (p0 >> 3) + 2 * hf + c2);
                uint4 v = lds128(a);
                uint32_t *vw = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
                for (int e2 = 0; e2 < 4; ++e2) {
                    const int i = 8 * c2 + 2 * e2;
                    vw[e2] = pack_bf16x2(fmaf(Dh, bf16_lo(vw[e2]), __uint_as_float(tv[i])),
                                         fmaf(Dh, bf16_hi(vw[e2]), __uint_as_float(tv[i + 1])));
                }
                sts128(a, v);
            }
        };

        // masked decay of the chunk whose sums are published: column blocks J = 2 (cs & 1) + jb of head
        // hd, rows of quarter q
        auto decay = [&](int rows) {
            if (32 * q >= rows) return;         // rows of y that are not stored
            const float csr = s.cvs[hd][r];
#pragma unroll 1
            for (int jb = 0; jb < 2; ++jb) {
                const int J = 2 * (cs & 1) + jb;
                if (32 * J >= rows) break;      // columns that no K-step of Y takes
                uint32_t pk[16];
                if (J < q) {
                    // below the diagonal: e^{cs_r - cs_j} = e^{cs_r - m_J} e^{m_J - cs_j}
                    const float E = ex2(s.cvs[hd][32 * J + 31] - csr);
                    const float2 E2 = make_float2(E, E);
                    uint32_t gv[32];
                    tmem_ld32(tG + lane_base + 32 * J, gv);
                    tmem_wait_ld(gv);
                    const float4 *f4 = reinterpret_cast<const float4 *>(&s.fs[hd][32 * J]);
#pragma unroll
                    for (int i4 = 0; i4 < 8; ++i4) {
                        const float4 f = f4[i4];
                        const float2 a = mul2(make_float2(__uint_as_float(gv[4 * i4]), __uint_as_float(gv[4 * i4 + 1])),
                                              mul2(make_float2(f.x, f.y), E2));
                        const float2 b = mul2(make_float2(__uint_as_float(gv[4 * i4 + 2]), __uint_as_float(gv[4 * i4 + 3])),
                                              mul2(make_float2(f.z, f.w), E2));
                        pk[2 * i4] = pack_bf16x2(a.x, a.y);
                        pk[2 * i4 + 1] = pack_bf16x2(b.x, b.y);
                    }
                } else if (J == q) {
                    // the diagonal block as 16x16 quarters: the two on the diagonal exponentiate each
                    // entry; the one below factors through the sum at the block's column 15
                    uint32_t gv[32];
                    tmem_ld32(tG + lane_base + 32 * J, gv);
                    tmem_wait_ld(gv);
                    const float *cvb = &s.cvs[hd][32 * J], *dvb = &s.dvs[hd][32 * J];
                    const float m16 = cvb[15];
                    const bool lo = lane < 16;
                    const float a_r = ex2(m16 - csr);                                   // <= 1 for lane >= 16
                    const float b_own = dvb[lane & 15] * ex2(cvb[lane & 15] - m16);     // <= dt for lane < 16
                    const int xo = lo ? 0 : 16;
#pragma unroll
                    for (int k4 = 0; k4 < 4; ++k4) {
                        const float4 c4 = *reinterpret_cast<const float4 *>(cvb + xo + 4 * k4), d4 = *reinterpret_cast<const float4 *>(dvb + xo + 4 * k4);
                        const float cc[4] = {c4.x, c4.y, c4.z, c4.w}, dd[4] = {d4.x, d4.y, d4.z, d4.w};
                        float vl[4], vh[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int kc = 4 * k4 + e;
                            const int x = xo + kc;
                            const float g_x = __uint_as_float(lo ? gv[kc] : gv[16 + kc]);
                            float t = g_x * ex2(cc[e] - csr) * dd[e];
                            t = x > lane ? 0.0f : t;
                            const float bk = __shfl_sync(0xffffffffu, b_own, kc);
                            vl[e] = lo ? t : __uint_as_float(gv[kc]) * (a_r * bk);
                            vh[e] = lo ? 0.0f : t;
                        }
                        pk[2 * k4] = pack_bf16x2(vl[0], vl[1]);
                        pk[2 * k4 + 1] = pack_bf16x2(vl[2], vl[3]);
                        pk[8 + 2 * k4] = pack_bf16x2(vh[0], vh[1]);
                        pk[9 + 2 * k4] = pack_bf16x2(vh[2], vh[3]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) pk[i] = 0u;
                }
                tmem_st16(tPm + lane_base + 16 * (2 * cs + jb), pk);
            }
        };

        // turn c: T, w o X and y of chunk c, then the state step and the masked decay of chunk c+1 (turn -1: those
        // of chunk 0 only, from the state that enters the window).  One copy of each: what the warps run through per
        // chunk has to stay in the instruction cache
#pragma unroll 1
        for (int c = -1; c < nc; ++c) {
          if (c >= 0) {
            uint8_t *xs = s.x[c & 1];

            // ---- T (= Ys of this chunk) *= e^{cs_r} on this warp's rows and columns
            if (!cwait(&s.ys_done, c & 1, abort, lim)) { fail(); break; }
            tc_fence_after();
            const int rows = s.desc[c & 1].y & kChunkRows;
            {
                const float e_r = ex2(s.tot[hd] - s.cvs[hd][r]);
                uint32_t tv[32];
                tmem_ld32(tT + lane_base + 32 * cs, tv);
                tmem_wait_ld(tv);
                const float2 e2 = make_float2(e_r, e_r);
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    const float2 q2 = mul2(make_float2(__uint_as_float(tv[i]), __uint_as_float(tv[i + 1])), e2);
                    tv[i] = __float_as_uint(q2.x); tv[i + 1] = __float_as_uint(q2.y);
                }
                tmem_st32(tT + lane_base + 32 * cs, tv);
            }
            // a short chunk: Y and S take K-steps of 16 rows; the rows of X behind the chunk's end in its last step are
            // cleared before Y sums over them, those of B before S does (G has read B: the decay waited for it)
            const int stop = (rows + 15) & ~15;
            if (rows < stop) {
                if (!cwait(&s.full_x[c & 1], (c >> 1) & 1, abort, lim)) { fail(); break; }
                for (int i = 32 * warp + lane; i < (stop - rows) * 16; i += 32 * kComputeWarps)
                    sts128(xs + ((i >> 3) & 1) * kBox + swz(rows + (i >> 4), i & 7), make_uint4(0u, 0u, 0u, 0u));
                fence_proxy_async_smem();
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.pm_ready);   // Pm written, T scaled, X's end cleared

            // ---- w o X of head hd: its bf16 rounding into the C half of this chunk's B/C slot (G and Ys have read
            //      C), the remainder into hp (Ys has read it), for S, which runs after Y
            if (!cwait(&s.full_x[c & 1], (c >> 1) & 1, abort, lim)) { fail(); break; }
            {
                const int ti = 32 * (warp & 7) + lane;
                const int j = ti >> 1, ch = 4 * (ti & 1);
                const float w = s.dvs[hd][j] * ex2(s.cvs[hd][j]);
                const uint8_t *src = xs + hd * kBox;
                uint8_t *dst = s.bc[c & 1] + hd * kBox, *rem = s.hp + hd * kBox;
#pragma unroll 1
                for (int u = 0; u < 4; ++u) {
                    const uint32_t o = swz(j, ch + u);
                    // (a row behind a short chunk's end is zero, whatever X holds there)
                    const uint4 v = j < rows ? lds128(src + o) : make_uint4(0u, 0u, 0u, 0u);
                    uint4 hi, lo;
                    split8(v, w, hi, lo);
                    sts128(dst + o, hi);
                    sts128(rem + o, lo);
                }
            }
            if (rows < stop) {
                if (!cwait(&s.full_bc[c & 1], (c >> 1) & 1, abort, lim)) { fail(); break; }
                for (int i = 32 * warp + lane; i < (stop - rows) * 16; i += 32 * kComputeWarps)
                    sts128(s.bc[c & 1] + (2 + ((i >> 3) & 1)) * kBox + swz(rows + (i >> 4), i & 7), make_uint4(0u, 0u, 0u, 0u));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.xw_ready);

            // ---- y of chunk c while S runs: Y is done, and every warp has read X for its w o X
            if (!(cwait(&s.ymma_done, c & 1, abort, lim) && cwait(&s.xw_ready, c & 1, abort, lim))) { fail(); break; }
            tc_fence_after();
            {
#pragma unroll 1
                for (int hf = 0; hf < 2; ++hf) {
                    uint32_t t0v[16];
                    tmem_ld16(tT + lane_base + 32 * cs + 16 * hf, t0v);
                    tmem_wait_ld(t0v);
                    y_half(xs, t0v, hf);
                }
            }
            fence_proxy_async_smem();   // y, read by the TMA store
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.y_ready[c & 1]);
          }
            // ---- the masked decay of chunk c+1 while S runs
            if (c + 1 < nc) {
                if (!(cwait(&s.scan_ready, (c + 1) & 1, abort, lim) && cwait(&s.g_done, (c + 1) & 1, abort, lim))) { fail(); break; }
                tc_fence_after();
                decay(s.desc[(c + 1) & 1].y & kChunkRows);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.pmw);
            }
            // ---- S is done too; the state step of chunk c+1
            if (c >= 0 && !cwait(&s.mma_done[c & 1], (c >> 1) & 1, abort, lim)) { fail(); break; }
            if (c + 1 < nc) {
                tc_fence_after();
                uint32_t hv[32];
                const int4 dn = s.desc[(c + 1) & 1];
                int slot = -1;
                bool ends = true;
                if (c >= 0) {
                    tmem_ld32(tH + lane_base + 32 * cs, hv);
                    tmem_wait_ld(hv);
                    ends = (s.desc[c & 1].y & kChunkLast) != 0;
                    if (p.h_out && ends) slot = s.desc[c & 1].w;
                }
                // where a sequence ends, its state goes to its slot and the next one's start takes its place; a
                // start from zero needs no registers, so that the old state can leave after Ys was let go
                const float *src = ends && (dn.y & kChunkFirst) ? window_start<false>(p, dn, k, first + nc, hh) : nullptr;
                const bool inside = ends && !(dn.y & kChunkFirst);      // (the window's first chunk of a sequence from before)
                if (inside)
                    window_enter<false, 32>(p, dn, k, per, hh, (int64_t)p0 * kN + r, kN, [&](int e, float v) { hv[e] = __float_as_uint(v); });
                if (src) {
                    if (slot >= 0) store_state(slot, hv);
#pragma unroll
                    for (int pp = 0; pp < 32; ++pp) hv[pp] = __float_as_uint(src[(p0 + pp) * kN + r]);
                }
                if (ends && !src && !inside) state_zero();
                else state_step(hv);
                tmem_wait_st();
                fence_proxy_async_smem();   // hp, read by Ys of chunk c+1
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.ys_go);
                if (slot >= 0 && !src) store_state(slot, hv);
            }
        }
        if (!__any_sync(0xffffffffu, *abort != 0)) {
            tc_fence_after();
            const int4 d = s.desc[(nc - 1) & 1];
            if ((d.y & kChunkLast) && p.h_out && d.w >= 0) {
                uint32_t hv[32];
                tmem_ld32(tH + lane_base + 32 * cs, hv);
                tmem_wait_ld(hv);
                store_state(d.w, hv);
            }
        }
    } else {
        // shared-memory descriptors of every operand tile, built once per slot: a K-step only adds
        // a constant to the start-address field (in 16-byte units; addresses stay below 256 KB)
        const uint32_t bc0 = smem_u32(s.bc[0]), bc1 = smem_u32(s.bc[1]);
        const uint32_t x0 = smem_u32(s.x[0]), x1 = smem_u32(s.x[1]);
        const uint64_t dC0 = smem_desc(bc0, 16, 1024), dC1 = smem_desc(bc1, 16, 1024);   // C, K-major
        const uint64_t dBk0 = smem_desc(bc0 + 2 * kBox, 16, 1024), dBk1 = smem_desc(bc1 + 2 * kBox, 16, 1024);  // B, K-major
        const uint64_t dBt0 = smem_desc(bc0 + 2 * kBox, kBox, 1024), dBt1 = smem_desc(bc1 + 2 * kBox, kBox, 1024);  // B^T, MN-major
        const uint64_t dX0 = smem_desc(x0, 0, 1024), dX1 = smem_desc(x1, 0, 1024);           // X of one head, MN-major, N = 64
        const uint64_t dXw0 = smem_desc(bc0, kBox, 1024), dXw1 = smem_desc(bc1, kBox, 1024);  // w o X, N = 128
        const uint64_t dHp = smem_desc(smem_u32(s.hp), kBox, 1024);                          // the states, then the remainder of w o X, N = 128
        constexpr uint64_t kBoxD = kBox >> 4;
        auto koff = [](int kk) -> uint64_t { return (uint64_t)((kk >> 2) * kBoxD + (kk & 3) * 2); };  // K-major K-step
        auto moff = [](int kk) -> uint64_t { return (uint64_t)(kk * 128); };                          // MN-major K-step
        auto issue_g = [&](int c) {
            const uint64_t dc = (c & 1) ? dC1 : dC0, db = (c & 1) ? dBk1 : dBk0;
            const uint32_t id_g = idesc_bf16(128, 128, 0, 0);
#pragma unroll 2
            for (int kk = 0; kk < 8; ++kk) mma_ss(tG, dc + koff(kk), db + koff(kk), id_g, kk > 0);
            mma_commit(&s.g_done);
        };
        // The whole warp waits (warp-uniform outcome); one lane issues.
        if (warp == kComputeWarps) {
            // ============================================= issuing warp: Y, S, Ys (and G of chunk 0)
            auto issue_ys = [&](int c) {
                const uint64_t dc = (c & 1) ? dC1 : dC0;
                const uint32_t id_ys = idesc_bf16(128, 128, 0, 1);    // A = C (K-major), B = hp (MN-major)
#pragma unroll 2
                for (int kk = 0; kk < 8; ++kk) mma_ss(tT, dc + koff(kk), dHp + moff(kk), id_ys, kk > 0);
                mma_commit(&s.ys_done);
            };
            const uint32_t id_pm = idesc_bf16(128, 64, 0, 1);     // A = Pm (TMEM), B = X (MN-major)
            const uint32_t id_s = idesc_bf16(128, 128, 1, 1);     // A = B^T (MN-major), B = w o X (MN-major)
            bool ok = live;
            if (ok) {
                ok = cwait(&s.full_bc[0], 0, abort, lim);
                if (ok) {
                    tc_fence_after();
                    if (elect_one()) issue_g(0);
                    __syncwarp();
                    ok = cwait(&s.ys_go, 0, abort, lim);
                    if (ok) {
                        tc_fence_after();
                        if (elect_one()) issue_ys(0);
                        __syncwarp();
                    }
                }
            }
            for (int c = 0; ok && c < nc; ++c) {
                ok = cwait(&s.pm_ready, c & 1, abort, lim) && cwait(&s.full_x[c & 1], (c >> 1) & 1, abort, lim);
                if (!ok) break;
                tc_fence_after();
                const int steps = (int)uniform(((s.desc[c & 1].y & kChunkRows) + 15) >> 4);
                if (elect_one()) {
                    const uint64_t dx = (c & 1) ? dX1 : dX0;
                    if (steps == 8) {
#pragma unroll 1
                        for (int hd2 = 0; hd2 < 2; ++hd2)
#pragma unroll 2
                            for (int kk = 0; kk < 8; ++kk)
                                mma_ts(tT + 64 * hd2, tPm + 64 * hd2 + kk * 8, dx + hd2 * kBoxD + moff(kk), id_pm, true);
                    } else {
#pragma unroll 1
                        for (int kk = 0; kk < steps; ++kk) {
                            mma_ts(tT, tPm + kk * 8, dx + moff(kk), id_pm, true);
                            mma_ts(tT + 64, tPm + 64 + kk * 8, dx + kBoxD + moff(kk), id_pm, true);
                        }
                    }
                    mma_commit(&s.ymma_done);
                }
                __syncwarp();
                ok = cwait(&s.xw_ready, c & 1, abort, lim);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t dbt = (c & 1) ? dBt1 : dBt0, dxw = (c & 1) ? dXw1 : dXw0;
                    if (steps == 8) {
#pragma unroll 2
                        for (int kk = 0; kk < 8; ++kk) mma_ss(tH, dbt + moff(kk), dxw + moff(kk), id_s, true);
#pragma unroll 2
                        for (int kk = 0; kk < 8; ++kk) mma_ss(tH, dbt + moff(kk), dHp + moff(kk), id_s, true);
                    } else {
#pragma unroll 1
                        for (int kk = 0; kk < steps; ++kk) {
                            mma_ss(tH, dbt + moff(kk), dxw + moff(kk), id_s, true);
                            mma_ss(tH, dbt + moff(kk), dHp + moff(kk), id_s, true);
                        }
                    }
                    mma_commit(&s.mma_done[c & 1]);
                }
                __syncwarp();
                if (c + 1 < nc) {
                    ok = cwait(&s.ys_go, (c + 1) & 1, abort, lim);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) issue_ys(c + 1);
                    __syncwarp();
                }
            }
            __syncwarp();
            if (elect_one()) {
                if (live && !ok) raise_timeout(p, abort);
                // every MMA of this warp complete before TMEM is freed
                mma_commit(&s.fin);
                wait_loop(&s.fin, 0, nullptr, 100000000ull);
            }
            __syncwarp();
        } else if (warp == kComputeWarps + 1) {
            // ============================================= store warp: y out, X in
            int x_issued = 0;   // lane 0's bookkeeping
            auto issue_x = [&](int c) {
                const int t0 = chunks[c].x;
                uint8_t *d = s.x[c & 1];
                uint64_t *bar = &s.full_x[c & 1];
                mbar_arrive_expect_tx(bar, 2 * kBox);
                tma_load_3d(d, &maps.x, bar, ha * kP, t0, 0);
                tma_load_3d(d + kBox, &maps.x, bar, (ha + 1) * kP, t0, 0);
                ++x_issued;
            };
            bool ok = live;
            if (ok && lane == 0) {
                issue_x(0);
                if (nc > 1) issue_x(1);
            }
            for (int c = 0; ok && c < nc; ++c) {
                const int4 d = chunks[c];
                const int rows = d.y & kChunkRows;
                uint8_t *xs = s.x[c & 1];
                // y staged: store it; once its slot has been read, X of chunk c+2 is loaded there
                ok = cwait(&s.y_ready[c & 1], (c >> 1) & 1, abort, lim);
                if (!ok) break;
                if (rows == kQ) {
                    if (lane == 0) {
                        tma_store_3d(&maps.y, xs, ha * kP, d.x, 0);
                        tma_store_3d(&maps.y, xs + kBox, (ha + 1) * kP, d.x, 0);
                        tma_store_commit();
                        if (c + 2 < nc) tma_store_wait_read<0>();
                    }
                } else {
                    // both heads' columns of a row are 256 consecutive bytes: two rows per step of the warp
                    __nv_bfloat16 *yr = reinterpret_cast<__nv_bfloat16 *>(p.y) + (int64_t)d.x * p.yrs + ha * kP + 8 * (lane & 15);
                    const uint8_t *src = xs + ((lane >> 3) & 1) * kBox;
                    for (int i = lane >> 4; i < rows; i += 2)
                        *reinterpret_cast<uint4 *>(yr + (int64_t)i * p.yrs) = lds128(src + swz(i, lane & 7));
                }
                __syncwarp();
                if (c + 2 < nc && lane == 0) issue_x(c + 2);
                __syncwarp();
            }
            if (lane == 0) {
                if (live && !ok) raise_timeout(p, abort);
                if (*abort) {
                    // the last load issued into each X slot lands before the CTA's shared memory is
                    // released (an earlier load into the same slot has been waited on by the compute warps)
                    for (int i = x_issued > 2 ? x_issued - 2 : 0; i < x_issued; ++i)
                        wait_loop(&s.full_x[i & 1], (i >> 1) & 1, nullptr, 100000000ull);
                }
                tma_store_wait<0>();
            }
            __syncwarp();
        } else if (warp == kComputeWarps + 3) {
            // ============================================= scan warp: lane l holds rows 4 l .. 4 l + 3
            const float A2a = p.A[ha] * kLog2e, A2b = p.A[ha + 1] * kLog2e;
            const float2 bias = p.dt_bias ? make_float2(p.dt_bias[ha], p.dt_bias[ha + 1]) : make_float2(0.0f, 0.0f);
            bool ok = live;
            int4 dn = chunks[0];
            float2 dt[4];
            load_dt(p, dn.x, dn.y & kChunkRows, lane, ha, dt);
            for (int c = 0; ok && c < nc; ++c) {
                const int4 d = dn;
                if (c + 1 < nc) dn = chunks[c + 1];
                use_dt(p, d.y & kChunkRows, lane, bias, dt);
                float ca[4], cb[4], ta, tb;
                chunk_sums(dt, A2a, A2b, lane, ca, cb, ta, tb);
                // the sum at the end of this lane's 32-row block (row 32 J + 31 = lane 8 J + 7)
                const float ea = __shfl_sync(0xffffffffu, ca[3], lane | 7), eb = __shfl_sync(0xffffffffu, cb[3], lane | 7);
                const float4 fa = make_float4(dt[0].x * ex2(ca[0] - ea), dt[1].x * ex2(ca[1] - ea),
                                              dt[2].x * ex2(ca[2] - ea), dt[3].x * ex2(ca[3] - ea));
                const float4 fb = make_float4(dt[0].y * ex2(cb[0] - eb), dt[1].y * ex2(cb[1] - eb),
                                              dt[2].y * ex2(cb[2] - eb), dt[3].y * ex2(cb[3] - eb));
                if (lane < 2 && c > 0 && (d.y & kChunkFirst)) {
                    const float *src = window_start<false>(p, d, k, first + nc, ha + lane);
                    if (src)
                        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"((uint32_t)(kPN * 4)) : "memory");
                }
                // every warp has used the sums of chunk c - 1 once all have written its w o X
                if (c > 0) {
                    ok = cwait(&s.xw_ready, (c - 1) & 1, abort, lim);
                    if (!ok) break;
                }
                reinterpret_cast<float4 *>(s.cvs[0])[lane] = make_float4(ca[0], ca[1], ca[2], ca[3]);
                reinterpret_cast<float4 *>(s.cvs[1])[lane] = make_float4(cb[0], cb[1], cb[2], cb[3]);
                reinterpret_cast<float4 *>(s.dvs[0])[lane] = make_float4(dt[0].x, dt[1].x, dt[2].x, dt[3].x);
                reinterpret_cast<float4 *>(s.dvs[1])[lane] = make_float4(dt[0].y, dt[1].y, dt[2].y, dt[3].y);
                if (lane < 24) {
                    reinterpret_cast<float4 *>(s.fs[0])[lane] = fa;
                    reinterpret_cast<float4 *>(s.fs[1])[lane] = fb;
                }
                if (lane == 0) { s.desc[c & 1] = d; s.tot[0] = ta; s.tot[1] = tb; }
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.scan_ready);
                if (c + 1 < nc) load_dt(p, dn.x, dn.y & kChunkRows, lane, ha, dt);
            }
            if (lane == 0 && live && !ok) raise_timeout(p, abort);
            __syncwarp();
        } else {
            // ============================================= B/C warp: B and C in, G of chunks 1..
            int bc_issued = 0;   // lane 0's bookkeeping
            auto issue_bc = [&](int c) {
                const int t0 = chunks[c].x;
                uint8_t *d = s.bc[c & 1];
                uint64_t *bar = &s.full_bc[c & 1];
                mbar_arrive_expect_tx(bar, 4 * kBox);
                tma_load_3d(d, &maps.C, bar, g * kN, t0, 0);
                tma_load_3d(d + kBox, &maps.C, bar, g * kN + 64, t0, 0);
                tma_load_3d(d + 2 * kBox, &maps.B, bar, g * kN, t0, 0);
                tma_load_3d(d + 3 * kBox, &maps.B, bar, g * kN + 64, t0, 0);
                ++bc_issued;
            };
            bool ok = live;
            if (ok) {
                if (lane == 0) {
                    issue_bc(0);
                    if (nc > 1) issue_bc(1);
                }
                if (nc > 1) {
                    ok = cwait(&s.pmw, 0, abort, lim) && cwait(&s.full_bc[1], 0, abort, lim);
                    if (ok) {
                        tc_fence_after();
                        if (elect_one()) issue_g(1);
                        __syncwarp();
                    }
                }
            }
            for (int c = 0; ok && c + 2 < nc; ++c) {
                // S of chunk c done: its B/C slot (C, B, w o X) is spent -- refill it with chunk c+2
                ok = cwait(&s.mma_done[c & 1], (c >> 1) & 1, abort, lim);
                if (!ok) break;
                if (lane == 0) issue_bc(c + 2);
                __syncwarp();
                // G of chunk c+2 once the warps have read G of chunk c+1, the slot has landed and Y of
                // chunk c+1 is done (G must not sit in front of it in the tensor pipe)
                ok = cwait(&s.pmw, (c + 1) & 1, abort, lim) &&
                     cwait(&s.full_bc[c & 1], ((c + 2) >> 1) & 1, abort, lim) &&
                     cwait(&s.ymma_done, (c + 1) & 1, abort, lim);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) issue_g(c + 2);
                __syncwarp();
            }
            __syncwarp();
            if (elect_one()) {
                if (live && !ok) raise_timeout(p, abort);
                mma_commit(&s.fin2);
                wait_loop(&s.fin2, 0, nullptr, 100000000ull);
            }
            __syncwarp();
            if (lane == 0) {
                if (*abort) {
                    for (int i = bc_issued > 2 ? bc_issued - 2 : 0; i < bc_issued; ++i)
                        wait_loop(&s.full_bc[i & 1], (i >> 1) & 1, nullptr, 100000000ull);
                }
            }
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tm, 512);
}

constexpr size_t kSmemA = sizeof(SmemA) + 1024;
constexpr size_t kSmemC = sizeof(SmemC);   // no alignment pad: the base is checked in the kernel
static_assert(kSmemC <= 232448, "pass C shared memory");
static_assert(kSmemA <= 232448, "pass A shared memory");

}  // namespace

bool packed_scan_tc_shape(int dtype, int H, int P, int N, int G)
{
    return dtype == 1 && P == kP && N == kN && G > 0 && H % G == 0 && (H / G) % 2 == 0;
}

int launch_packed_scan_tc(const PackedScanParams &p, bool carry, cudaStream_t st)
{
    EncodeTiledFn enc = encode_fn();
    if (!enc) return 7;
    Maps maps{};
    const int64_t gn = (int64_t)p.G * p.N, hp = (int64_t)p.H * p.P, rows = p.plan.total > 0 ? p.plan.total : 1;
    const bool hand_on = carry && p.nw > 1;
    if (p.plan.total > 0 &&
        (!encode_bf16(enc, &maps.x, p.x, hp, rows, 1, p.xrs, 0) || !encode_bf16(enc, &maps.B, p.B, gn, rows, 1, p.Brs, 0) ||
         (hand_on && (!encode_bf16(enc, &maps.x64, p.x, hp, rows, 1, p.xrs, 0, kQA) || !encode_bf16(enc, &maps.B64, p.B, gn, rows, 1, p.Brs, 0, kQA))) ||
         !encode_bf16(enc, &maps.C, p.C, gn, rows, 1, p.Crs, 0) || !encode_bf16(enc, &maps.y, p.y, hp, rows, 1, p.yrs, 0)))
        return 6;
    static SmemLimit done_a, done_c;
    if (!allow_smem(packed_state_tc_kernel, (int)kSmemA, done_a) || !allow_smem(packed_output_tc_kernel, (int)kSmemC, done_c)) return 7;
    const unsigned units = (unsigned)p.nw * (unsigned)(p.H / 2);
    if (hand_on) {
        prof_begin(st, kKPackedState);
        packed_state_tc_kernel<<<units, kThreadsA, kSmemA, st>>>(maps, p);
        prof_end(st, kKPackedState);
        const int rc = p.ws_hin ? launch_packed_chain(p, false, st) : 0;
        if (rc) return rc;
    }
    prof_begin(st, kKPackedOutput);
    packed_output_tc_kernel<<<units, kThreadsC, kSmemC, st>>>(maps, p);
    prof_end(st, kKPackedOutput);
    return cudaGetLastError() == cudaSuccess ? 0 : 7;
}

}  // namespace ssd

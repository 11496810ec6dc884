// packed_grad_tc.cu -- gradients of the selective scan over sequences laid end to end on the tensor
// cores: bf16 inputs, P = 64, N = 128.
//
// In chunks of 64 rows, with cs_i the running sum of dt A inside the chunk, lam the chunk's sum, h
// the state entering it and Gam the adjoint arriving at its last row (scan_bwd.cu has the formulas):
//   dx_j  = D dy_j + dt_j [ sum_{t>=j} E_tj CB_tj dy_t + e^{lam-cs_j} Gam B_j ]
//   dB_j  = sum_{t>=j} M_tj C_t + w_j x_j^T Gam           w_j = dt_j e^{lam-cs_j}
//   dC_t  = sum_{j<=t} M_tj B_j + e^{cs_t} dy_t^T h
//   with E_tj = e^{cs_t-cs_j}, CB = C B^T, M_tj = E_tj dt_j (dy_t . x_j)
// Three kernels (16384 rows of 32 heads, 9 sequences, the longest of 7000: 451 to 482 us on different machines; the bytes that go in and out
// would take 48, with h and Gam, which go through memory once, 210):
//   walk      the states and the adjoints, chunk after chunk, from the first or the last of a sequence,
//             kept in registers in fp32; only what the gradients multiply by leaves the kernel
//   gradient  a CTA takes the heads of a chunk one after the other: dB and dC, sums over the heads of a
//             group, stay in TMEM meanwhile, and C B^T is formed once
//   sums      dB and dC of the groups that were done in several blocks of heads; dA and dD
//
// Precision.  Products take bf16 operands with fp32 sums; x, dy, B and C are bf16 as given.  An operand
// that is not (the weighted x and dy, M, E o CB, and h and Gam) enters as its bf16 rounding plus the
// bf16 rounding of what that leaves, 16 significant bits, and of such pairs all but the product of the
// two remainders is formed: each term is off by about 2^-17.  State and adjoint are walked in fp32; where
// few rows or heads are summed, they enter <Gam, h>, dxI and YI (below) in three parts, 24 bits (two_parts).
//
// All waits are bounded (tc::mbar_wait): on a timeout the CTA raises an abort flag, every thread
// unwinds, copies and products in flight are drained, TMEM is freed and the status word reports it.
#include <algorithm>

#include "packed.cuh"
#include "scan_tc_util.cuh"

namespace ssd {
namespace {

using namespace tc;

constexpr int kQ = 64, kP = 64, kN = 128, kPN = kP * kN;
constexpr uint32_t kTile = 64 * 128;      // 64 rows of 128 bytes, 128B-swizzled
constexpr uint32_t kPiece = 128 * 128;    // a state's bf16 part: rows n, columns p, 128B-swizzled
// A state as the gradient's operand: kParts bf16 parts, each the rounding of what those before it leave
template <int kParts> constexpr uint32_t kImage = kParts * kPiece;
// Two parts where dA, one number per head, is made of many rows of many heads, three elsewhere: among random batches of
// few rows or few heads two parts left dA off by up to 1.3e-5 of 64 bits, three by 2.4e-6 (worst of 120).  From 1024
// rows of 16 heads on two are off by 1.9e-6 at 16384 rows of 32 heads, and in the worst batches known, of one-token
// sequences whose terms cancel, by 3.3e-6 in the middle and 9.7e-6 at most (4680 batches of 1024 to 4096 of them);
// three take 553 us instead of 453 at 16384 rows.  The rows are those of the sequences, which the device knows (the buffers of a captured batch may hold
// many more), so where the tensors have the rows for it the kernels hold both forms and the plan decides (9 sequences of
// 16384 rows in all 442 -> 451 us, one sequence 546 -> 535, on one machine).
constexpr int kManyRows = 1024, kManyHeads = 16;
inline bool either_form(int64_t total, int H) { return total >= kManyRows && H >= kManyHeads; }
template <bool kEither>
__device__ __forceinline__ bool two_parts(const PackedGradParams &p)
{
    return kEither && packed_ok(p.plan, p.status) && p.plan.hdr->rows >= kManyRows;
}

__device__ __forceinline__ void raise_timeout(const PackedGradParams &p, volatile int *abort)
{
    *abort = 1;
    atomicOr(p.status, kDevTimeout);
}

// 16 bytes into shared memory without passing through registers; zeros when they are not to be read
__device__ __forceinline__ void cp16(void *dst, const void *src, bool read)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(read ? 16u : 0u) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory"); }

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void bulk_store(void *dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes) : "memory");
}

// 8 TMEM columns of 32 lanes
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
// 16 columns of 16 lanes: thread l receives rows l / 4 (r[0..1], r[4..5]) and l / 4 + 8 (r[2..3], r[6..7]),
// columns 2 (l % 4) and the next (r[0..3]) and 8 further on (r[4..7])
__device__ __forceinline__ void tmem_ld_rows16(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld8(uint32_t (&r)[8])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :
                 : "memory");
}

// n K-steps, their operands' descriptors sa and sb apart
template <int n>
__device__ __forceinline__ void mma_steps(uint32_t d, uint64_t a, uint64_t b, uint32_t sa, uint32_t sb, uint32_t idesc, bool accumulate)
{
#pragma unroll
    for (int k = 0; k < n; ++k) mma_ss(d, a + (uint64_t)(k * sa), b + (uint64_t)(k * sb), idesc, accumulate || k > 0);
}

// fp32 pair -> its bf16 rounding and the bf16 rounding of what it leaves
__device__ __forceinline__ void split2(float2 v, uint32_t &hi, uint32_t &lo)
{
    hi = pack_bf16x2(v.x, v.y);
    lo = pack_bf16x2(v.x - bf16_lo(hi), v.y - bf16_hi(hi));
}
__device__ __forceinline__ void split_scaled8(uint4 v, float w, uint4 &hi, uint4 &lo)
{
    const float2 w2 = make_float2(w, w);
    split2(mul2(unpack2(v.x), w2), hi.x, lo.x);
    split2(mul2(unpack2(v.y), w2), hi.y, lo.y);
    split2(mul2(unpack2(v.z), w2), hi.z, lo.z);
    split2(mul2(unpack2(v.w), w2), hi.w, lo.w);
}

__device__ __forceinline__ int grad_chunks(const PackedGradParams &p) { return packed_n64(p.plan, p.status); }

// =============================================================== walk
// One CTA per (part of the chunk list, state or adjoint, head): a part begins and ends between sequences.  Per chunk
// the product S[n][p] = sum_j B[j][n] (w_j x_j[p]) (adjoint: C, e^{cs_j} dy) gets both parts of the weighted
// operand side by side as 128 columns, and the state follows in registers, h = e^lam h + S.  What enters each chunk
// goes out as the gradient kernel's operand, one bulk copy each.  What bounds it is a chunk's chain of waits,
// 1.2 us, times the chunks of the longest part (136 in that batch): 164 to 170 us, at 3.3 TB/s of states.
// Warps 0..7 keep the state (lane = n, 32 of p each), warps 8..15 fetch rows three chunks ahead and weigh them, warp
// 16 issues the products, warp 17 runs the sums of dt A, warp 18 the copies out.
constexpr int kWalkState = 8, kWalkScale = 8, kWalkThreads = 32 * (kWalkState + kWalkScale + 3);
template <int kParts> constexpr int kWalkStages = kParts == 2 ? 5 : 4;    // (what shared memory has room for)

template <int kParts>
struct SmemWalk {
    uint8_t op[kWalkStages<kParts>][2 * kTile];     // B (or C): columns 0..63, 64..127
    uint8_t xr[kWalkStages<kParts>][kTile];         // x (or dy) as given, each thread its own 16 bytes
    uint8_t xs[2][2 * kTile];               // the weighted x (or dy), and what its rounding leaves
    uint8_t img[2][kImage<kParts>];
    float w[8][kQ];
    float f[8];
    uint64_t w_ready[8], xs_ready[4], mma_done[4], acc_full[2], acc_free[2], img_ready[2], img_free[2], fin;
    uint32_t tmem;
    int abort;
};

// first chunk of the first sequence that begins at chunk k or later
__device__ __forceinline__ int sequence_begin(const PackedPlan &p, int n, int64_t k)
{
    if (k >= n) return n;
    const int4 d = p.chunk64[k];
    if (d.y & kChunkFirst) return (int)k;
    const PackedSeq s = p.seqs[d.z];
    return s.c64 + s.n64;
}

static_assert(sizeof(SmemWalk<2>) <= 232448 && sizeof(SmemWalk<3>) <= 232448, "the walk's shared memory");

template <int kParts>
__device__ __forceinline__ void grad_walk(const PackedGradParams &p, uint8_t *raw)
{
    SmemWalk<kParts> &s = *reinterpret_cast<SmemWalk<kParts> *>(raw);
    constexpr int kStages = kWalkStages<kParts>;
    constexpr uint32_t kImg = kImage<kParts>;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = (int)(blockIdx.x % p.H);
    const bool adj = blockIdx.x >= p.H;
    const int nch = grad_chunks(p);
    const int64_t per = (nch + gridDim.y - 1) / gridDim.y;
    const int ca = sequence_begin(p.plan, nch, blockIdx.y * per), cb = sequence_begin(p.plan, nch, (blockIdx.y + 1) * per);
    const int n = cb - ca;
    if (n <= 0) return;
    const int g = (int)((int64_t)h * p.G / p.H);
    const uint64_t lim = p.wait_limit_ns;
    const int4 *tab = p.plan.chunk64;
    auto chunk_of = [&](int it) { return adj ? cb - 1 - it : ca + it; };

    if (tid == 0) {
        for (int i = 0; i < 8; ++i) mbar_init(&s.w_ready[i], 1);
        for (int i = 0; i < 4; ++i) {
            mbar_init(&s.xs_ready[i], kWalkScale);
            mbar_init(&s.mma_done[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.acc_full[i], 1);
            mbar_init(&s.acc_free[i], kWalkState);
            mbar_init(&s.img_ready[i], kWalkState);
            mbar_init(&s.img_free[i], 1);
        }
        mbar_init(&s.fin, 1);
        s.abort = 0;
        fence_mbar_init();
    }
    if (warp == 0) { tmem_alloc(&s.tmem, 256); tmem_relinquish(); }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tS = s.tmem;
    volatile int *abort = &s.abort;
    bool ok = true;

    if (warp < kWalkState) {
        const int q = warp & 3, e = warp >> 2, nn = 32 * q + lane;      // state elements [32 e ..][nn]
        const uint32_t acc = tS + ((uint32_t)(32 * q) << 16) + 32 * e;
        float hv[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) hv[i] = 0.0f;
        int4 d = __ldg(tab + chunk_of(0));
#pragma unroll 1
        for (int it = 0; it < n; ++it) {
            const int b = it & 1;
            // the state that a sequence starts from (the adjoint that it ends with)
            if (d.y & (adj ? kChunkLast : kChunkFirst)) {
                const float *src = adj ? p.dh_out : p.h_in;
                const bool has = src && (adj || ((d.y & kChunkResume) && d.w >= 0));
                if (has) {
                    src += ((int64_t)(adj ? d.z : d.w) * p.H + h) * kPN + (int64_t)(32 * e) * kN + nn;
#pragma unroll
                    for (int i = 0; i < 32; ++i) hv[i] = __ldg(src + i * kN);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) hv[i] = 0.0f;
                }
            }
            // what enters the chunk
            if (it >= 2 && !(ok = cwait(&s.img_free[b], (uint32_t)((it >> 1) - 1) & 1, abort, lim))) break;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t v[kParts][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float2 r = make_float2(hv[8 * k + 2 * i], hv[8 * k + 2 * i + 1]);
#pragma unroll
                    for (int w = 0; w < kParts; ++w) {
                        v[w][i] = pack_bf16x2(r.x, r.y);
                        r = make_float2(r.x - bf16_lo(v[w][i]), r.y - bf16_hi(v[w][i]));
                    }
                }
#pragma unroll
                for (int w = 0; w < kParts; ++w) sts128(s.img[b] + w * kPiece + swz(nn, 4 * e + k), make_uint4(v[w][0], v[w][1], v[w][2], v[w][3]));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.img_ready[b]);
            const int4 dn = __ldg(tab + chunk_of(min(it + 1, n - 1)));
            if (!(ok = cwait(&s.w_ready[it & 7], (uint32_t)(it >> 3) & 1, abort, lim) && cwait(&s.acc_full[b], (uint32_t)(it >> 1) & 1, abort, lim))) break;
            tc_fence_after();
            const float f = s.f[it & 7];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t ah[16], al[16];
                tmem_ld16(acc + 128 * b + 16 * k, ah);
                tmem_ld16(acc + 128 * b + 64 + 16 * k, al);
                tmem_wait_ld(ah, al);
#pragma unroll
                for (int i = 0; i < 16; ++i) hv[16 * k + i] = fmaf(f, hv[16 * k + i], __uint_as_float(ah[i]) + __uint_as_float(al[i]));
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.acc_free[b]);
            if (adj && p.dh_in && (d.y & kChunkFirst)) {
                // a sequence that does not resume has no state to pass it on to
                const bool pass = p.h_in && (d.y & kChunkResume);
                float *dst = p.dh_in + ((int64_t)d.z * p.H + h) * kPN + (int64_t)(32 * e) * kN + nn;
#pragma unroll
                for (int i = 0; i < 32; ++i) dst[i * kN] = pass ? hv[i] : 0.0f;
            }
            d = dn;
        }
        if (!ok && lane == 0) raise_timeout(p, abort);
        __syncwarp();
    } else if (warp < kWalkState + kWalkScale) {
        // ================================================= fetch and weigh
        const int t = tid - 32 * kWalkState;
        const char *xg = static_cast<const char *>(adj ? p.dy : p.x) + 2 * (int64_t)h * kP;
        const char *og = static_cast<const char *>(adj ? p.C : p.B) + 2 * (int64_t)g * kN;
        const int64_t xrs = 2 * (adj ? p.dyrs : p.xrs), ors = 2 * (adj ? p.Crs : p.Brs);
        const int jx = t >> 3, cx = t & 7;             // 16 bytes of x: rows jx, jx + 32, columns 8 cx ..
        const int jo = t >> 4, co = t & 15;            // and of B: rows jo + 16 k, columns 8 co ..
        auto fetch = [&](int it) {
            if (it < n) {
                const int4 d = __ldg(tab + chunk_of(it));
                const int rows = d.y & kChunkRows, st = it % kStages;
                const char *xs = xg + d.x * xrs + 16 * cx, *os = og + d.x * ors + 16 * co;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int r = jx + 32 * k;
                    cp16(s.xr[st] + 128 * r + 16 * cx, r < rows ? xs + r * xrs : xg, r < rows);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = jo + 16 * k;
                    cp16(s.op[st] + (co >> 3) * kTile + swz(r, co & 7), r < rows ? os + r * ors : og, r < rows);
                }
            }
            cp_commit();
        };
#pragma unroll 1
        for (int it = 0; it < kStages - 2; ++it) fetch(it);
#pragma unroll 1
        for (int it = 0; it < n; ++it) {
            const int st = it % kStages, b = it & 1;
            cp_wait<kStages - 3>();
            if (!(ok = cwait(&s.w_ready[it & 7], (uint32_t)(it >> 3) & 1, abort, lim))) break;
            if (it >= 2 && !(ok = cwait(&s.mma_done[(it - 2) & 3], (uint32_t)((it - 2) >> 2) & 1, abort, lim))) break;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = jx + 32 * k;
                uint4 hi, lo;
                split_scaled8(lds128(s.xr[st] + 128 * r + 16 * cx), s.w[it & 7][r], hi, lo);
                sts128(s.xs[b] + swz(r, cx), hi);
                sts128(s.xs[b] + kTile + swz(r, cx), lo);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.xs_ready[it & 3]);
            fetch(it + kStages - 2);            // the stage of chunk it - 2
        }
        if (!ok && lane == 0) raise_timeout(p, abort);
        cp_wait<0>();
    } else if (warp == kWalkState + kWalkScale) {
        // ================================================= issuing warp
        const uint32_t id = idesc_bf16(128, 128, 1, 1);   // A = B^T (MN-major), B = the weighted rows and their remainders (MN-major)
        const uint32_t tSu = uniform(tS);
        const bool live = (int64_t)(blockIdx.y * gridDim.x + blockIdx.x) != p.test_drop_unit;
        for (int it = 0; live && it < n; ++it) {
            ok = cwait(&s.xs_ready[it & 3], (uint32_t)(it >> 2) & 1, abort, lim) &&
                 (it < 2 || cwait(&s.acc_free[it & 1], (uint32_t)((it >> 1) - 1) & 1, abort, lim));
            if (!ok) break;
            tc_fence_after();
            const uint32_t b = uniform(it & 1), st = uniform(it % kStages);
            if (elect_one()) {
                mma_steps<kQ / 16>(tSu + 128 * b, smem_desc(smem_u32(s.op[st]), kTile, 1024), smem_desc(smem_u32(s.xs[b]), kTile, 1024), 128, 128, id, false);
                mma_commit(&s.mma_done[it & 3]);
                mma_commit(&s.acc_full[b]);
            }
            __syncwarp();
        }
        __syncwarp();
        if (elect_one()) {
            if (!ok) raise_timeout(p, abort);
            mma_commit(&s.fin);
            mbar_wait(&s.fin, 0, nullptr, 100000000ull);
        }
        __syncwarp();
    } else if (warp == kWalkState + kWalkScale + 1) {
        // ================================================= the sums of dt A, four chunks at a time, the next four's dt in flight
        const float A2 = p.A[h] * kLog2e;
        float dn[4][2];
        auto load = [&](int it0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int4 d = __ldg(tab + chunk_of(min(it0 + e, n - 1)));
                const int rows = d.y & kChunkRows;
                const float *src = p.dt + ((int64_t)d.x + 2 * lane) * p.H + h;
                dn[e][0] = 2 * lane < rows ? src[0] : 0.0f;
                dn[e][1] = 2 * lane + 1 < rows ? src[p.H] : 0.0f;
                // the state of a sequence about to begin, on its way into L2
                const float *st = adj ? p.dh_out : p.h_in;
                if (lane == 0 && st && it0 + e < n && (d.y & (adj ? kChunkLast : kChunkFirst)) && (adj || ((d.y & kChunkResume) && d.w >= 0))) {
                    st += ((int64_t)(adj ? d.z : d.w) * p.H + h) * kPN;
                    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(st), "r"((uint32_t)(kPN * 4)) : "memory");
                }
            }
        };
        load(0);
#pragma unroll 1
        for (int it0 = 0; ok && it0 < n; it0 += 4) {
            float d0[4], d1[4], a0[4], a1[4], inc[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                d0[e] = dn[e][0]; d1[e] = dn[e][1];
                a0[e] = d0[e] * A2; a1[e] = d1[e] * A2;
                inc[e] = a0[e] + a1[e];
            }
            if (it0 + 4 < n) load(it0 + 4);
            if (adj) {
#pragma unroll
                for (int o = 1; o < 32; o <<= 1)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float t = __shfl_up_sync(0xffffffffu, inc[e], o);
                        if (lane >= o) inc[e] += t;
                    }
            } else {
#pragma unroll
                for (int o = 1; o < 32; o <<= 1)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float t = __shfl_down_sync(0xffffffffu, inc[e], o);
                        if (lane + o < 32) inc[e] += t;
                    }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int it = it0 + e;
                const float tot = __shfl_sync(0xffffffffu, inc[e], adj ? 31 : 0);
                float near = adj ? __shfl_up_sync(0xffffffffu, inc[e], 1) : __shfl_down_sync(0xffffffffu, inc[e], 1);
                if (lane == (adj ? 0 : 31)) near = 0.0f;
                if (it >= n) break;
                // adjoint: e^{cs_t}; state: dt_j e^{sum after j}
                const float2 w2 = adj ? make_float2(ex2(near + a0[e]), ex2(near + a0[e] + a1[e]))
                                      : make_float2(d0[e] * ex2(near + a1[e]), d1[e] * ex2(near));
                // the chunk eight before it has been weighed and its f used: the product of the chunk four before it waited for
                // the state warps to be done with the chunk six before it
                if (it >= 4 && !(ok = cwait(&s.mma_done[it & 3], (uint32_t)((it >> 2) - 1) & 1, abort, lim))) break;
                reinterpret_cast<float2 *>(s.w[it & 7])[lane] = w2;
                if (lane == 0) s.f[it & 7] = ex2(tot);
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.w_ready[it & 7]);
            }
        }
        if (!ok && lane == 0) raise_timeout(p, abort);
        __syncwarp();
    } else {
        // ================================================= copies out
#pragma unroll 1
        for (int it = 0; it < n; ++it) {
            const int b = it & 1;
            if (!(ok = cwait(&s.img_ready[b], (uint32_t)(it >> 1) & 1, abort, lim))) break;
            if (lane == 0) {
                bulk_store(p.ws_img + (((int64_t)chunk_of(it) * p.H + h) * 2 + (adj ? 1 : 0)) * (int64_t)kImg, s.img[b], kImg);
                tma_store_commit();
                // the copy before it has read its image
                tma_store_wait_read<1>();
                if (it >= 1) mbar_arrive(&s.img_free[b ^ 1]);
            }
            __syncwarp();
        }
        if (lane == 0) {
            if (!ok) raise_timeout(p, abort);
            tma_store_wait<0>();
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tS, 256);
}

template <bool kEither>
__global__ void __launch_bounds__(kWalkThreads, 1) packed_grad_walk_kernel(const __grid_constant__ PackedGradParams p)
{
    extern __shared__ __align__(1024) uint8_t sw_raw[];
    if (two_parts<kEither>(p)) grad_walk<2>(p, sw_raw);
    else grad_walk<3>(p, sw_raw);
}

// =============================================================== gradients
// The items (chunk, head), chunk after chunk, are dealt out in equal runs of blocks of heads, one CTA per SM: a CTA meets
// few chunks, loads C and B of a group once, and keeps dB and dC in TMEM through a block.
// Per item, on the tensor pipe: GX = dy x^T;  dxI = B Gam^T, YI = C h^T;  dB += Gam (w x), dC += h (e^{cs} dy);
// dx = (E CB)^T dy, dB += C^T M, dC += B^T M^T.  Warps 0..7: (M) E o CB and M in two parts, the row and column sums of
// M o CB; (A) x_j . dxI_j and dy_t . YI_t; (D) dx.  Warps 8..15, ahead of them: (S) w x and e^{cs} dy in two parts;
// (F) <Gam, h>.  (All 16 warps on one step after the other, each step waiting for its own latencies: 5.2 us per item
// and SM, 292 us for 8352 items; so 4.6 to 5.0.)
// M = 64 accumulators use 16 of each 32 TMEM lanes: GX and CB keep columns 16 k .. 16 k + 7 in the lower and the eight
// behind them in the upper 16, so that a warp's 16 rows and 16 columns lie on or off the triangle together; dxI and
// YI share their columns that way.  The sums that make ddt are finished by a warp of their own.
// TMEM: dB 0..63, dC 64..127 (lanes n, columns rows), dxI | YI 128..191 and 192..255, GX 256..287 and 288..319,
// dx 320..383, CB 384..415.  8352 items: 259 to 283 us on different machines, the tensor pipe active for 38 % of it.  Dealt
// out to two issuing warps it took 290 (the registers of a 21st warp), with products under lane == 0 430.
constexpr int kMathWarps = 8, kWeighWarps = 8, kGradWarps = kMathWarps + kWeighWarps, kGradThreads = 32 * (kGradWarps + 4);
constexpr uint32_t kColB = 0, kColC = 64, kColI = 128, kColG = 256, kColDx = 320, kColCB = 384;
constexpr uint32_t kUpper = 16u << 16;    // lanes 16..31 of each 32

template <int kParts> constexpr int kGradSlots = kParts == 2 ? 3 : 2;

template <int kParts>
struct SmemGrad {
    uint8_t cb[4 * kTile];                // C columns 0..63, 64..127, B likewise
    uint8_t xd[2][2 * kTile];             // x, dy of items i, i + 1
    uint8_t st[kGradSlots<kParts>][kImage<kParts>];           // Gam and h in turn
    uint8_t sc[4 * kTile];                // w x, its remainder, e^{cs} dy, its remainder
    uint8_t mk[4 * kTile];                // E o CB, its remainder, M, its remainder
    float cs[2][kQ], dt[2][kQ], suf[2][kQ];   // sums of dt A (log2 units) up to each row, dt, sums after each row
    uint64_t cb_full, cb_empty, xd_full[2], xd_empty[2], st_full[3], st_empty[3];
    uint64_t cs_ready[2], gx_done[2], in_done[2], cbt_done, sc_ready, inter_done, mk_ready, dx_done, intra_done, acc_free, res_ready;
    uint64_t sums_ready[2], sums_free[2], fin;
    uint32_t tmem;
    int abort;
};
static_assert(sizeof(SmemGrad<2>) <= 232448 && sizeof(SmemGrad<3>) <= 232448, "the gradient kernel's shared memory");

// partial sums of an item on their way to the warp that finishes them (in global memory: shared memory is full)
constexpr int kSumCol = 0, kSumRow = 256, kSumBe = 384, kSumAl = 512, kSumDiag = 640, kSumD = 704, kSumF = 768, kSumRes = 800, kSumFloats = 864;

// How the heads of the chunks are dealt out: in blocks of S heads of a group, nb blocks to a group.  The sums over the
// heads of a block are formed in TMEM, where each addition is cut off instead of rounded, so a block has at most
// kMaxBlock heads, added up in fp32 behind (blocks of 32 heads were off by 7.8e-6 of 64 bits, of 8 by 3.8e-6);
// a short batch gets smaller blocks, to load all SMs.
constexpr int kMaxBlock = 8;
struct GradSplit {
    int S, nb;
    int blocks, per;            // blocks in all (no more than chunks x heads), and per CTA
    __device__ __forceinline__ GradSplit(const PackedGradParams &p, int nch, int ctas)
    {
        const int R = p.H / p.G;
        const int64_t fair = (int64_t)nch * p.H / ctas;
        S = min(max(1, (int)min(fair, (int64_t)kMaxBlock)), R);
        nb = (R + S - 1) / S;
        blocks = nch * p.G * nb;
        per = (blocks + ctas - 1) / ctas;
    }
};

// The items of a CTA, in order, without those of empty sequences
struct Items {
    int v, end;                 // its blocks of heads
    int S, nb, G, R, it;
    int4 d;
    int chunk, h, h1;
    bool valid, first, last;    // first and last of its block
    bool enter, leave, tail;    // first and last of its chunk and group in this CTA; in the last block of them
    const int4 *tab;

    __device__ __forceinline__ void settle(bool fresh)
    {
        valid = false;
        while (v < end) {
            const int c = v / (G * nb), rem = v - c * (G * nb), blk = rem % nb;
            if (fresh || rem == 0) {
                d = __ldg(tab + c);
                chunk = c;
                if ((d.y & kChunkRows) == 0) { v = (c + 1) * (G * nb); continue; }
            }
            const int g = rem / nb;
            h = g * R + blk * S;
            h1 = min(h + S, (g + 1) * R);
            first = true;
            enter = fresh || blk == 0;
            last = h + 1 == h1;
            tail = blk == nb - 1 || v + 1 == end;
            leave = last && tail;
            valid = true;
            return;
        }
    }
    __device__ __forceinline__ Items(const PackedGradParams &p, const GradSplit &sp)
        : v((int)min((int64_t)blockIdx.x * sp.per, (int64_t)sp.blocks)), end(min(v + sp.per, sp.blocks)), S(sp.S), nb(sp.nb), G(p.G), R(p.H / p.G), it(0), d{}, chunk(0), h(0), h1(0), first(false), last(false), enter(false), leave(false), tail(false), tab(p.plan.chunk64)
    {
        settle(true);
    }
    __device__ __forceinline__ void next()
    {
        ++it;
        if (++h < h1) {
            first = enter = false;
            last = h + 1 == h1;
            leave = last && tail;
        } else {
            ++v;
            settle(false);
        }
    }
};

template <int kParts>
__device__ __forceinline__ void grad_items(const PackedGradParams &p, uint8_t *raw)
{
    SmemGrad<kParts> &s = *reinterpret_cast<SmemGrad<kParts> *>(raw);
    constexpr int kSlots = kGradSlots<kParts>;
    constexpr uint32_t kImg = kImage<kParts>;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const GradSplit split(p, grad_chunks(p), gridDim.x);
    Items m(p, split);
    if (!m.valid) return;           // nothing left, or nothing but empty sequences
    const int R = p.H / p.G;
    const uint64_t lim = p.wait_limit_ns;
    if (tid == 0) {
        mbar_init(&s.cb_full, 1); mbar_init(&s.cb_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.xd_full[i], 1); mbar_init(&s.xd_empty[i], kGradWarps);
            mbar_init(&s.cs_ready[i], 1); mbar_init(&s.gx_done[i], 1); mbar_init(&s.in_done[i], 1);
            mbar_init(&s.sums_ready[i], kGradWarps); mbar_init(&s.sums_free[i], 1);
        }
        for (int i = 0; i < kSlots; ++i) { mbar_init(&s.st_full[i], 1); mbar_init(&s.st_empty[i], 1 + kWeighWarps); }
        mbar_init(&s.cbt_done, 1); mbar_init(&s.sc_ready, kWeighWarps); mbar_init(&s.inter_done, 1);
        mbar_init(&s.mk_ready, kMathWarps); mbar_init(&s.dx_done, 1); mbar_init(&s.intra_done, 1);
        mbar_init(&s.acc_free, kMathWarps); mbar_init(&s.res_ready, kMathWarps); mbar_init(&s.fin, 1);
        s.abort = 0;
        fence_mbar_init();
    }
    if (warp == 0) { tmem_alloc(&s.tmem, 512); tmem_relinquish(); }
    // what lies behind the triangle
    for (int i = tid; i < (int)(4 * kTile / 16); i += kGradThreads) sts128(s.mk + 16 * i, make_uint4(0, 0, 0, 0));
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s.tmem;
    volatile int *abort = &s.abort;
    bool ok = true;

    if (warp < kMathWarps) {
        // ================================================= (M), (A), (D) of each item, dB and dC of each block
        const int q = warp & 3, e = warp >> 2, half = lane >> 4;
        const uint32_t lanes = (uint32_t)(32 * q) << 16;
        const int mrow = 16 * q + (lane & 15);         // row of an M = 64 accumulator
        float *sums = p.ws_sums + (int64_t)blockIdx.x * 2 * kSumFloats;
        uint32_t unit = 0, block = 0;
        // With states in three parts: what the two parts of M leave out on its diagonal, of the block's heads, added to dB
        // and dC in fp32.  Where every sequence is a token or two, dC_t is M_tt summed over the heads times B_t, and one
        // scalar's error, however the heads cancel, is all of dC_t's: 1.3e-5 at five sequences of one token without this.
        float res = 0.0f;
        for (; ok && m.valid; m.next()) {
            const int it = m.it, b = it & 1;
            const uint32_t ph = (uint32_t)(it >> 1) & 1;
            float *sm = sums + b * kSumFloats;
            // ---- (M)
            if (m.enter && !(ok = cwait(&s.cbt_done, unit++ & 1, abort, lim))) break;
            ok = cwait(&s.cs_ready[b], ph, abort, lim) && cwait(&s.gx_done[b], ph, abort, lim);
            if (ok && it > 0) ok = cwait(&s.intra_done, (uint32_t)(it - 1) & 1, abort, lim);
            if (ok && it > 1) ok = cwait(&s.sums_free[b], (uint32_t)((it >> 1) - 1) & 1, abort, lim);
            if (!ok) break;
            tc_fence_after();
            {
                const float ct = s.cs[b][mrow];
                float row = 0.0f;
                // columns 16 k .. of its rows 16 q ..: those behind the triangle stay zero
#pragma unroll 1
                for (int k = e; k <= q; k += 2) {
                    const int j0 = 16 * k + 8 * half;
                    uint32_t gx[8], cb[8];
                    tmem_ld8(tm + lanes + kColG + 32 * b + 8 * k, gx);
                    tmem_ld8(tm + lanes + kColCB + 8 * k, cb);
                    float cj[8], dj[8];
                    *reinterpret_cast<float4 *>(cj) = *reinterpret_cast<const float4 *>(&s.cs[b][j0]);
                    *reinterpret_cast<float4 *>(cj + 4) = *reinterpret_cast<const float4 *>(&s.cs[b][j0 + 4]);
                    *reinterpret_cast<float4 *>(dj) = *reinterpret_cast<const float4 *>(&s.dt[b][j0]);
                    *reinterpret_cast<float4 *>(dj + 4) = *reinterpret_cast<const float4 *>(&s.dt[b][j0 + 4]);
                    tmem_wait_ld8(gx);
                    tmem_wait_ld8(cb);
                    float kp[8], ec[8], mm[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float E = j0 + i <= mrow ? ex2(ct - cj[i]) : 0.0f, cbi = __uint_as_float(cb[i]);
                        const float eg = E * __uint_as_float(gx[i]);
                        ec[i] = E * cbi;
                        mm[i] = eg * dj[i];
                        kp[i] = eg * cbi;
                        if (j0 + i < mrow) row = fmaf(mm[i], cbi, row);
                    }
                    uint32_t hi[4], lo[4];
                    const uint32_t o = swz(mrow, (j0 >> 3));
#pragma unroll
                    for (int i = 0; i < 4; ++i) split2(make_float2(ec[2 * i], ec[2 * i + 1]), hi[i], lo[i]);
                    sts128(s.mk + o, make_uint4(hi[0], hi[1], hi[2], hi[3]));
                    sts128(s.mk + kTile + o, make_uint4(lo[0], lo[1], lo[2], lo[3]));
#pragma unroll
                    for (int i = 0; i < 4; ++i) split2(make_float2(mm[2 * i], mm[2 * i + 1]), hi[i], lo[i]);
                    sts128(s.mk + 2 * kTile + o, make_uint4(hi[0], hi[1], hi[2], hi[3]));
                    sts128(s.mk + 3 * kTile + o, make_uint4(lo[0], lo[1], lo[2], lo[3]));
                    if (k == q) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (j0 + i == mrow) {
                                sm[kSumDiag + mrow] = kp[i];
                                sm[kSumD + mrow] = __uint_as_float(gx[i]);
                                if (kParts == 3) res += mm[i] - (i & 1 ? bf16_hi(hi[i / 2]) : bf16_lo(hi[i / 2])) - (i & 1 ? bf16_hi(lo[i / 2]) : bf16_lo(lo[i / 2]));
                                if (kParts == 3 && m.last) {
                                    sm[kSumRes + mrow] = res;
                                    res = 0.0f;
                                }
                            }
                    }
                    // column sums over the 16 rows: each halving step keeps half of the columns and adds the partner's copy
                    // of them
                    float k4[4], k2[2];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bool up = lane & 8;
                        const float keep = up ? kp[i + 4] : kp[i], give = up ? kp[i] : kp[i + 4];
                        k4[i] = keep + __shfl_xor_sync(0xffffffffu, give, 8);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const bool up = lane & 4;
                        const float keep = up ? k4[i + 2] : k4[i], give = up ? k4[i] : k4[i + 2];
                        k2[i] = keep + __shfl_xor_sync(0xffffffffu, give, 4);
                    }
                    const bool up = lane & 2;
                    const float keep = up ? k2[1] : k2[0], give = up ? k2[0] : k2[1];
                    float kc = keep + __shfl_xor_sync(0xffffffffu, give, 2);
                    kc += __shfl_xor_sync(0xffffffffu, kc, 1);
                    // (lane bits 3, 2, 1 name the column of the eight)
                    if (!(lane & 1)) sm[kSumCol + 64 * q + j0 + ((lane >> 1) & 1) + ((lane >> 2) & 1) * 2 + ((lane >> 3) & 1) * 4] = kc;
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.mk_ready);
                row += __shfl_xor_sync(0xffffffffu, row, 16);
                if (lane < 16) sm[kSumRow + 64 * e + mrow] = row;
                if (kParts == 3 && m.last) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s.res_ready);
                }
            }
            // ---- (A)
            if (!(ok = cwait(&s.in_done[b], ph, abort, lim))) break;
            tc_fence_after();
            {
                float2 a = make_float2(0.0f, 0.0f);
                const uint8_t *v = s.xd[b] + half * kTile;
#pragma unroll 1
                for (int u = 0; u < 2; ++u) {
                    uint32_t r[16];
                    tmem_ld16(tm + lanes + kColI + 64 * b + 32 * e + 16 * u, r);
                    const uint4 v0 = lds128(v + swz(mrow, 4 * e + 2 * u)), v1 = lds128(v + swz(mrow, 4 * e + 2 * u + 1));
                    const uint32_t vv[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
                    tmem_wait_ld(r);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        a = fma2(make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), unpack2(vv[i]), a);
                }
                sm[(half ? kSumAl : kSumBe) + 64 * e + mrow] = a.x + a.y;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.sums_ready[b]);
            // ---- (D)
            if (!(ok = cwait(&s.dx_done, (uint32_t)it & 1, abort, lim))) break;
            tc_fence_after();
            {
                const float Dh = p.D ? __ldg(p.D + m.h) : 0.0f;
                const int rows = m.d.y & kChunkRows;
                float *dst = p.dx + (int64_t)m.d.x * ((int64_t)p.H * kP) + (int64_t)m.h * kP + 32 * e + 2 * (lane & 3);
                float dtj[2], ew[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int j = 16 * q + (lane >> 2) + 8 * u;
                    dtj[u] = s.dt[b][j];
                    ew[u] = ex2(s.suf[b][j]);
                }
#pragma unroll 1
                for (int w = 0; w < 2; ++w) {
                    uint32_t a[8], in[8];
                    tmem_ld_rows16(tm + lanes + kColDx + 32 * e + 16 * w, a);
                    tmem_ld_rows16(tm + lanes + kColI + 64 * b + 32 * e + 16 * w, in);
                    tmem_wait_ld8(a);
                    tmem_wait_ld8(in);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int j = 16 * q + (lane >> 2) + 8 * u;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float2 dy = unpack2(*reinterpret_cast<const uint32_t *>(s.xd[b] + kTile + swz(j, 4 * e + 2 * w + k) + 4 * (lane & 3)));
                            const float ax = __uint_as_float(a[4 * k + 2 * u]), ay = __uint_as_float(a[4 * k + 2 * u + 1]);
                            const float ix = __uint_as_float(in[4 * k + 2 * u]), iy = __uint_as_float(in[4 * k + 2 * u + 1]);
                            const float2 o = make_float2(fmaf(dtj[u], fmaf(ew[u], ix, ax), Dh * dy.x), fmaf(dtj[u], fmaf(ew[u], iy, ay), Dh * dy.y));
                            if (j < rows) *reinterpret_cast<float2 *>(dst + (int64_t)j * ((int64_t)p.H * kP) + 16 * w + 8 * k) = o;
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.xd_empty[b]);
            // ---- the block's dB and dC
            if (m.last) {
                if (kParts == 3 && !(ok = cwait(&s.res_ready, block++ & 1, abort, lim))) break;
                if (!(ok = cwait(&s.intra_done, (uint32_t)it & 1, abort, lim))) break;
                tc_fence_after();
                const int nn = 32 * q + lane, g = m.h / R, rows = m.d.y & kChunkRows;
                const __nv_bfloat16 *Bn = static_cast<const __nv_bfloat16 *>(p.B) + m.d.x * p.Brs + g * kN + nn;
                const __nv_bfloat16 *Cn = static_cast<const __nv_bfloat16 *>(p.C) + m.d.x * p.Crs + g * kN + nn;
                float *dB, *dC;
                int64_t rs;
                if (m.nb == 1) {
                    dB = p.dB + ((int64_t)m.d.x * p.G + g) * kN;
                    dC = p.dC + ((int64_t)m.d.x * p.G + g) * kN;
                    rs = (int64_t)p.G * kN;
                } else {
                    dB = p.ws_part + (int64_t)m.v * (2 * kQ * kN);
                    dC = dB + kQ * kN;
                    rs = kN;
                }
#pragma unroll 1
                for (int u = 0; u < 4; ++u) {
                    const int t0 = 32 * e + 8 * u;
                    uint32_t ab[8], ac[8];
                    tmem_ld8(tm + lanes + kColB + t0, ab);
                    tmem_ld8(tm + lanes + kColC + t0, ac);
                    // (three parts) what M's diagonal left out
                    float r[8];
                    __nv_bfloat16 bn[8], cn[8];
                    if (kParts == 3) {
                        *reinterpret_cast<float4 *>(r) = *reinterpret_cast<const float4 *>(sm + kSumRes + t0);
                        *reinterpret_cast<float4 *>(r + 4) = *reinterpret_cast<const float4 *>(sm + kSumRes + t0 + 4);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            bn[i] = t0 + i < rows ? __ldg(Bn + (t0 + i) * p.Brs) : __float2bfloat16(0.0f);
                            cn[i] = t0 + i < rows ? __ldg(Cn + (t0 + i) * p.Crs) : __float2bfloat16(0.0f);
                        }
                    }
                    tmem_wait_ld8(ab);
                    tmem_wait_ld8(ac);
                    if (u == 3) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&s.acc_free);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (t0 + i < rows) {
                            dB[(t0 + i) * rs + nn] = kParts == 3 ? fmaf(r[i], __bfloat162float(cn[i]), __uint_as_float(ab[i])) : __uint_as_float(ab[i]);
                            dC[(t0 + i) * rs + nn] = kParts == 3 ? fmaf(r[i], __bfloat162float(bn[i]), __uint_as_float(ac[i])) : __uint_as_float(ac[i]);
                        }
                }
            }
        }
        if (!ok && lane == 0) raise_timeout(p, abort);
        __syncwarp();
    } else if (warp < kGradWarps) {
        // ================================================= (S), (F) of each item
        const int t = tid - 32 * kMathWarps;
        float *sums = p.ws_sums + (int64_t)blockIdx.x * 2 * kSumFloats;
        for (; ok && m.valid; m.next()) {
            const int it = m.it, b = it & 1;
            const uint32_t ph = (uint32_t)(it >> 1) & 1;
            // ---- (S)
            if (!(ok = cwait(&s.xd_full[b], ph, abort, lim) && cwait(&s.cs_ready[b], ph, abort, lim))) break;
            if (it > 0 && !(ok = cwait(&s.inter_done, (uint32_t)(it - 1) & 1, abort, lim))) break;
#pragma unroll 1
            for (int u = 0; u < 2; ++u) {
                const int r = (t >> 3) + 32 * u, c = t & 7;
                const uint32_t o = swz(r, c);
                const uint4 x = lds128(s.xd[b] + o), dy = lds128(s.xd[b] + kTile + o);
                uint4 hi, lo;
                split_scaled8(x, s.dt[b][r] * ex2(s.suf[b][r]), hi, lo);
                sts128(s.sc + o, hi);
                sts128(s.sc + kTile + o, lo);
                split_scaled8(dy, ex2(s.cs[b][r]), hi, lo);
                sts128(s.sc + 2 * kTile + o, hi);
                sts128(s.sc + 3 * kTile + o, lo);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&s.sc_ready);
                mbar_arrive(&s.xd_empty[b]);
            }
            // ---- (F)
            const int ug = 2 * it, uh = 2 * it + 1;
            if (!(ok = cwait(&s.st_full[ug % kSlots], (uint32_t)(ug / kSlots) & 1, abort, lim) && cwait(&s.st_full[uh % kSlots], (uint32_t)(uh / kSlots) & 1, abort, lim))) break;
            const uint8_t *G = s.st[ug % kSlots], *h = s.st[uh % kSlots];
            float2 a = make_float2(0.0f, 0.0f);
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
                const uint32_t o = 16 * (t + 256 * k);
                uint4 gv[kParts], hv[kParts];
#pragma unroll
                for (int i = 0; i < kParts; ++i) { gv[i] = lds128(G + i * kPiece + o); hv[i] = lds128(h + i * kPiece + o); }
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    float2 g2[kParts], h2[kParts];
#pragma unroll
                    for (int i = 0; i < kParts; ++i) {
                        const uint32_t gw[4] = {gv[i].x, gv[i].y, gv[i].z, gv[i].w}, hw[4] = {hv[i].x, hv[i].y, hv[i].z, hv[i].w};
                        g2[i] = unpack2(gw[w]);
                        h2[i] = unpack2(hw[w]);
                    }
                    // the sum of a value's parts, smallest first
#pragma unroll
                    for (int i = kParts - 2; i >= 0; --i) {
                        g2[i] = make_float2(g2[i].x + g2[i + 1].x, g2[i].y + g2[i + 1].y);
                        h2[i] = make_float2(h2[i].x + h2[i + 1].x, h2[i].y + h2[i + 1].y);
                    }
                    a = fma2(g2[0], h2[0], a);
                }
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&s.st_empty[ug % kSlots]);
                mbar_arrive(&s.st_empty[uh % kSlots]);
            }
            float v = a.x + a.y;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (it > 1 && !(ok = cwait(&s.sums_free[b], (uint32_t)((it >> 1) - 1) & 1, abort, lim))) break;
            if (lane == 0) {
                sums[b * kSumFloats + kSumF + warp - kMathWarps] = v;
                mbar_arrive(&s.sums_ready[b]);
            }
            __syncwarp();
        }
        if (!ok && lane == 0) raise_timeout(p, abort);
        __syncwarp();
    } else if (warp == kGradWarps) {
        // ================================================= issuing warp (the whole warp waits, one lane issues)
        const uint32_t cC = smem_u32(s.cb), cB = cC + 2 * kTile;
        const uint64_t dCk = smem_desc(cC, 16, 1024), dBk = smem_desc(cB, 16, 1024);          // rows x K = n
        const uint64_t dBh = smem_desc(cB, 16, 2048);                                         // every other 8 rows of B
        const uint64_t dCm = smem_desc(cC, kTile, 1024), dBm = smem_desc(cB, kTile, 1024);    // M = n, K = rows
        const uint32_t id_g = idesc_bf16(64, 32, 0, 0), id_i = idesc_bf16(64, 64, 0, 1), id_x = idesc_bf16(64, 64, 1, 1);
        const uint32_t id_kk = idesc_bf16(128, 64, 0, 0), id_mm = idesc_bf16(128, 64, 1, 1), id_mk = idesc_bf16(128, 64, 1, 0);
        const uint32_t tu = uniform(tm);
        uint32_t unit = 0, block = 0;
        auto gx = [&](int it) -> bool {
            const uint32_t b = uniform(it & 1);
            if (!cwait(&s.xd_full[b], (uint32_t)(it >> 1) & 1, abort, lim)) return false;
            tc_fence_after();
            if (elect_one()) {
                const uint32_t x = smem_u32(s.xd[b]);
                const uint64_t dx = smem_desc(x, 16, 2048), dd = smem_desc(x + kTile, 16, 1024);     // (every other 8 rows of x)
#pragma unroll 1
                for (int hf = 0; hf < 2; ++hf)
                    mma_steps<4>(tu + kColG + 32 * b + hf * kUpper, dd, dx + (uint64_t)(hf * (1024 >> 4)), 2, 2, id_g, false);
                mma_commit(&s.gx_done[b]);
            }
            __syncwarp();
            return true;
        };
        auto from_states = [&](int it, bool first, bool enter) -> bool {
            const uint32_t b = uniform(it & 1), sg = uniform((2 * it) % kSlots), sh = uniform((2 * it + 1) % kSlots), acc = uniform(first ? 0 : 1);
            if (enter) {
                if (!cwait(&s.cb_full, unit & 1, abort, lim)) return false;
                ++unit;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) {
                        const int hf = k >> 1;
                        const uint64_t box = (uint64_t)((k & 1) * (kTile >> 4));
                        mma_steps<4>(tu + kColCB + hf * kUpper, dCk + box, dBh + box + (uint64_t)(hf * (1024 >> 4)), 2, 2, id_g, k & 1);
                    }
                    mma_commit(&s.cbt_done);
                }
                __syncwarp();
            }
            const uint32_t G = smem_u32(s.st[sg]), h = smem_u32(s.st[sh]);
            for (int w = 0; w < 2; ++w) {
                const int u = 2 * it + w;
                if (!cwait(&s.st_full[u % kSlots], (uint32_t)(u / kSlots) & 1, abort, lim)) return false;
                if (elect_one()) {
                    const uint64_t ds = smem_desc(w ? h : G, kTile, 1024);
                    const uint64_t da = w ? dCk : dBk;
#pragma unroll 1
                    for (int k = 0; k < 2 * kParts; ++k)      // every part, both halves of n
                        mma_steps<4>(tu + kColI + 64 * b + w * kUpper, da + (uint64_t)((k & 1) * (kTile >> 4)),
                                  ds + (uint64_t)((k >> 1) * (kPiece >> 4) + (k & 1) * 512), 2, 128, id_i, k > 0);
                }
                __syncwarp();
            }
            if (elect_one()) mma_commit(&s.in_done[b]);
            __syncwarp();
            if (!cwait(&s.sc_ready, (uint32_t)it & 1, abort, lim)) return false;
            if (first && block > 0 && !cwait(&s.acc_free, (block - 1) & 1, abort, lim)) return false;
            tc_fence_after();
            if (elect_one()) {
                // dB^T[n][j] += Gam^T[n][p] (w x)[j][p], dC^T likewise: M = n rows of the image, K = p
                const uint32_t sc = smem_u32(s.sc);
#pragma unroll 1
                for (int w = 0; w < 2; ++w) {
                    const uint64_t da = smem_desc(w ? h : G, 16, 1024), db = smem_desc(sc + (uint32_t)w * 2 * kTile, 16, 1024);
#pragma unroll 1
                    for (int part = 0; part < 3; ++part)
                        mma_steps<4>(tu + (w ? kColC : kColB), da + (uint64_t)(part == 2 ? kPiece >> 4 : 0), db + (uint64_t)(part == 1 ? kTile >> 4 : 0), 2, 2,
                                  id_kk, acc || part > 0);
                }
                mma_commit(&s.inter_done);
                mma_commit(&s.st_empty[sg]);
                mma_commit(&s.st_empty[sh]);
            }
            __syncwarp();
            if (first) ++block;
            return true;
        };
        Items nx = m;
        ok = gx(0) && from_states(0, true, true);
        while (ok && m.valid) {
            const int it = m.it;
            nx.next();
            if (!(ok = cwait(&s.mk_ready, (uint32_t)it & 1, abort, lim))) break;
            tc_fence_after();
            const uint32_t bi = uniform(it & 1);
            if (elect_one()) {
                const uint32_t mk = smem_u32(s.mk);
                const uint64_t de = smem_desc(mk, kTile, 1024), dm = smem_desc(mk + 2 * kTile, kTile, 1024), dmk = smem_desc(mk + 2 * kTile, 16, 1024);
                const uint64_t dd = smem_desc(smem_u32(s.xd[bi]) + kTile, kTile, 1024);
                const uint64_t lo = kTile >> 4;
#pragma unroll 1
                for (int part = 0; part < 2; ++part) mma_steps<4>(tu + kColDx, de + part * lo, dd, 128, 128, id_x, part);
                mma_commit(&s.dx_done);
#pragma unroll 1
                for (int part = 0; part < 2; ++part) {
                    mma_steps<4>(tu + kColB, dCm, dm + part * lo, 128, 128, id_mm, true);
                    mma_steps<4>(tu + kColC, dBm, dmk + part * lo, 128, 2, id_mk, true);
                }
                mma_commit(&s.intra_done);
                if (m.leave) mma_commit(&s.cb_empty);
            }
            __syncwarp();
            if (nx.valid && !(ok = gx(nx.it) && from_states(nx.it, nx.first, nx.enter))) break;
            m = nx;
        }
        __syncwarp();
        if (elect_one()) {
            if (!ok) raise_timeout(p, abort);
            mma_commit(&s.fin);
            mbar_wait(&s.fin, 0, nullptr, 100000000ull);
        }
        __syncwarp();
    } else if (warp == kGradWarps + 1) {
        // ================================================= x and dy, two items in flight; C and B of each unit
        uint32_t unit = 0;
        for (; ok && m.valid; m.next()) {
            const int it = m.it, b = it & 1, rows = m.d.y & kChunkRows;
            if (it >= 2 && !(ok = cwait(&s.xd_empty[b], (uint32_t)((it >> 1) - 1) & 1, abort, lim))) break;
            const char *xg = static_cast<const char *>(p.x) + 2 * (int64_t)m.h * kP, *dg = static_cast<const char *>(p.dy) + 2 * (int64_t)m.h * kP;
            const int c = lane & 7, r0 = lane >> 3;
#pragma unroll 4
            for (int k = 0; k < 16; ++k) {
                const int r = r0 + 4 * k;
                const int64_t row = r < rows ? (int64_t)m.d.x + r : 0;
                cp16(s.xd[b] + swz(r, c), xg + row * 2 * p.xrs + 16 * c, r < rows);
                cp16(s.xd[b] + kTile + swz(r, c), dg + row * 2 * p.dyrs + 16 * c, r < rows);
            }
            cp_commit();
            cp_wait<0>();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.xd_full[b]);
            if (m.enter) {
                // the unit before it has been multiplied
                if (unit > 0 && !(ok = cwait(&s.cb_empty, (unit - 1) & 1, abort, lim))) break;
                const int g = m.h / R;
                const char *Cg = static_cast<const char *>(p.C) + 2 * (int64_t)g * kN, *Bg = static_cast<const char *>(p.B) + 2 * (int64_t)g * kN;
                const int cc = lane & 15;
#pragma unroll 4
                for (int k = 0; k < 32; ++k) {
                    const int r = (lane >> 4) + 2 * k;
                    const int64_t row = r < rows ? (int64_t)m.d.x + r : 0;
                    const uint32_t o = (uint32_t)(cc >> 3) * kTile + swz(r, cc & 7);
                    cp16(s.cb + o, Cg + row * 2 * p.Crs + 16 * cc, r < rows);
                    cp16(s.cb + 2 * kTile + o, Bg + row * 2 * p.Brs + 16 * cc, r < rows);
                }
                cp_commit();
                cp_wait<0>();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.cb_full);
                ++unit;
            }
        }
        if (!ok && lane == 0) raise_timeout(p, abort);
        __syncwarp();
    } else if (warp == kGradWarps + 2) {
        // ================================================= Gam and h, three images in flight
        int issued = 0;
        for (; ok && m.valid; m.next()) {
            for (int w = 0; ok && w < 2; ++w) {
                const int u = 2 * m.it + w, k = u % kSlots;
                if (u >= kSlots && !(ok = cwait(&s.st_empty[k], (uint32_t)(u / kSlots - 1) & 1, abort, lim))) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&s.st_full[k], kImg);
                    bulk_load(s.st[k], p.ws_img + (((int64_t)m.chunk * p.H + m.h) * 2 + (w ? 0 : 1)) * (int64_t)kImg, kImg, &s.st_full[k]);
                }
                ++issued;
                __syncwarp();
            }
        }
        if (lane == 0) {
            if (!ok) raise_timeout(p, abort);
            // the last copy into each place lands before the CTA's shared memory is released
            for (int u = issued > kSlots ? issued - kSlots : 0; u < issued; ++u) mbar_wait(&s.st_full[u % kSlots], (uint32_t)(u / kSlots) & 1, nullptr, 100000000ull);
        }
        __syncwarp();
    } else {
        // ================================================= sums of dt A ahead of the items, ddt behind them
        Items ah = m;
        const float *sums = p.ws_sums + (int64_t)blockIdx.x * 2 * kSumFloats;
        auto scan = [&]() {
            const int b = ah.it & 1, rows = ah.d.y & kChunkRows;
            const float A2 = p.A[ah.h] * kLog2e;
            const float *src = p.dt + ((int64_t)ah.d.x + 2 * lane) * p.H + ah.h;
            const float d0 = 2 * lane < rows ? src[0] : 0.0f, d1 = 2 * lane + 1 < rows ? src[p.H] : 0.0f;
            const float a0 = d0 * A2, a1 = d1 * A2;
            float up = a0 + a1, dn = up;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float tu = __shfl_up_sync(0xffffffffu, up, o), td = __shfl_down_sync(0xffffffffu, dn, o);
                if (lane >= o) up += tu;
                if (lane + o < 32) dn += td;
            }
            float before = __shfl_up_sync(0xffffffffu, up, 1), after = __shfl_down_sync(0xffffffffu, dn, 1);
            if (lane == 0) before = 0.0f;
            if (lane == 31) after = 0.0f;
            reinterpret_cast<float2 *>(s.cs[b])[lane] = make_float2(before + a0, before + a0 + a1);
            reinterpret_cast<float2 *>(s.suf[b])[lane] = make_float2(after + a1, after);
            reinterpret_cast<float2 *>(s.dt[b])[lane] = make_float2(d0, d1);
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.cs_ready[b]);
        };
        for (int k = 0; k < 2 && ah.valid; ++k) { scan(); ah.next(); }
        for (; ok && m.valid; m.next()) {
            const int it = m.it, b = it & 1;
            const uint32_t ph = (uint32_t)(it >> 1) & 1;
            if (!(ok = cwait(&s.sums_ready[b], ph, abort, lim))) break;
            const float *sm = sums + b * kSumFloats;
            const float2 cs = reinterpret_cast<const float2 *>(s.cs[b])[lane], sf = reinterpret_cast<const float2 *>(s.suf[b])[lane];
            const float2 dt = reinterpret_cast<const float2 *>(s.dt[b])[lane];
            const float lam = s.cs[b][kQ - 1];
            float2 row = make_float2(0.0f, 0.0f), col = row, be = row, al = row;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k >= lane >> 3) {       // (rows 16 k .. reach columns 2 lane, 2 lane + 1)
                    const float2 c = reinterpret_cast<const float2 *>(sm + kSumCol + 64 * k)[lane];
                    col.x += c.x; col.y += c.y;
                }
                if (k < 2) {
                    const float2 r = reinterpret_cast<const float2 *>(sm + kSumRow + 64 * k)[lane];
                    const float2 u = reinterpret_cast<const float2 *>(sm + kSumBe + 64 * k)[lane], a = reinterpret_cast<const float2 *>(sm + kSumAl + 64 * k)[lane];
                    row.x += r.x; row.y += r.y;
                    be.x += u.x; be.y += u.y; al.x += a.x; al.y += a.y;
                }
            }
            const float2 dg = reinterpret_cast<const float2 *>(sm + kSumDiag)[lane], gd = reinterpret_cast<const float2 *>(sm + kSumD)[lane];
            float F = lane < kWeighWarps ? sm[kSumF + lane] : 0.0f;
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.sums_free[b]);
            // e^{lam-cs_j} x_j Gam B_j; and times dt_j
            be.x *= ex2(sf.x); be.y *= ex2(sf.y);
            const float b0 = dt.x * be.x, b1 = dt.y * be.y;
            // dl_t = sum_{t'>=t} (al_t' + row_t' - dt_t' (col_t' - diag_t')) + sum_{j<t} b_j + e^lam <Gam, h>
            const float v0 = fmaf(ex2(cs.x), al.x, row.x - dt.x * (col.x - dg.x)), v1 = fmaf(ex2(cs.y), al.y, row.y - dt.y * (col.y - dg.y));
            float sv = v0 + v1, pb = b0 + b1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float td = __shfl_down_sync(0xffffffffu, sv, o), tu = __shfl_up_sync(0xffffffffu, pb, o);
                if (lane + o < 32) sv += td;
                if (lane >= o) pb += tu;
                F += __shfl_xor_sync(0xffffffffu, F, o);
            }
            float svn = __shfl_down_sync(0xffffffffu, sv, 1), pbn = __shfl_up_sync(0xffffffffu, pb, 1);
            if (lane == 31) svn = 0.0f;
            if (lane == 0) pbn = 0.0f;
            const float in = ex2(lam) * F;
            const float l0 = svn + v1 + v0 + pbn + in, l1 = svn + v1 + pbn + b0 + in;
            const float A = p.A[m.h];
            const int rows = m.d.y & kChunkRows;
            float *dst = p.ddt + ((int64_t)m.d.x + 2 * lane) * p.H + m.h;
            if (2 * lane < rows) dst[0] = fmaf(A, l0, col.x + be.x);
            if (2 * lane + 1 < rows) dst[p.H] = fmaf(A, l1, col.y + be.y);
            float pa = fmaf(dt.x, l0, dt.y * l1), pd = gd.x + gd.y;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                pa += __shfl_xor_sync(0xffffffffu, pa, o);
                pd += __shfl_xor_sync(0xffffffffu, pd, o);
            }
            if (lane == 0) {
                p.ws_pA[(int64_t)m.h * p.plan.m64 + m.chunk] = pa;
                p.ws_pD[(int64_t)m.h * p.plan.m64 + m.chunk] = pd;
            }
            __syncwarp();
            if (ah.valid) {
                if (!(ok = cwait(&s.xd_empty[b], ph, abort, lim))) break;
                scan();
                ah.next();
            }
        }
        if (!ok && lane == 0) raise_timeout(p, abort);
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tm, 512);
}

template <bool kEither>
__global__ void __launch_bounds__(kGradThreads, 1) packed_grad_tc_kernel(const __grid_constant__ PackedGradParams p)
{
    extern __shared__ __align__(1024) uint8_t sg_raw[];
    if (two_parts<kEither>(p)) grad_items<2>(p, sg_raw);
    else grad_items<3>(p, sg_raw);
}

// =============================================================== sums
// The first kSumParts x units blocks: dB and dC of a (chunk, group) whose heads make several blocks, in their order; the H blocks
// behind them: dA and dD of a head, in a fixed order; the blocks behind those: dh_in of a sequence without chunks.
constexpr int kSumParts = 4;        // blocks to a unit

__global__ void __launch_bounds__(256) packed_grad_sum_kernel(const PackedGradParams p, int ctas)
{
    const int nch = grad_chunks(p);
    const int64_t units = p.plan.m64 * p.G;
    if (blockIdx.x < kSumParts * units) {
        const GradSplit sp(p, nch, ctas);
        const int64_t u = blockIdx.x / kSumParts;
        const int c = (int)(u / p.G), g = (int)(u % p.G);
        if (c >= nch || sp.nb == 1) return;
        const int4 d = p.plan.chunk64[c];
        const int rows = d.y & kChunkRows;
        for (int i = threadIdx.x + blockDim.x * (blockIdx.x % kSumParts); i < rows * (kN / 4); i += kSumParts * blockDim.x) {
            const int r = i / (kN / 4), n4 = i % (kN / 4);
            float4 sb = make_float4(0.f, 0.f, 0.f, 0.f), sc = sb;
#pragma unroll 4
            for (int b = 0; b < sp.nb; ++b) {
                const float4 *src = reinterpret_cast<const float4 *>(p.ws_part + (u * sp.nb + b) * (2 * kQ * kN) + r * kN) + n4;
                const float4 vb = src[0], vc = src[kQ * kN / 4];
                sb.x += vb.x; sb.y += vb.y; sb.z += vb.z; sb.w += vb.w;
                sc.x += vc.x; sc.y += vc.y; sc.z += vc.z; sc.w += vc.w;
            }
            const int64_t o = (((int64_t)d.x + r) * p.G + g) * kN;
            reinterpret_cast<float4 *>(p.dB + o)[n4] = sb;
            reinterpret_cast<float4 *>(p.dC + o)[n4] = sc;
        }
        return;
    }
    if (blockIdx.x >= kSumParts * units + p.H) {
        // a sequence without chunks starts from no state
        const int64_t q = blockIdx.x - kSumParts * units - p.H;
        if (!p.dh_in || !packed_ok(p.plan, p.status) || p.plan.seqs[q].n64 != 0) return;
        float4 *dst = reinterpret_cast<float4 *>(p.dh_in + q * p.H * kPN);
        for (int64_t i = threadIdx.x; i < (int64_t)p.H * (kPN / 4); i += blockDim.x) dst[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        return;
    }
    __shared__ float sa[256], sd[256];
    const int h = (int)(blockIdx.x - kSumParts * units);
    float a = 0.0f, d = 0.0f;
    for (int c = threadIdx.x; c < nch; c += blockDim.x)
        if (p.plan.chunk64[c].y & kChunkRows) {
            a += p.ws_pA[(int64_t)h * p.plan.m64 + c];
            d += p.ws_pD[(int64_t)h * p.plan.m64 + c];
        }
    sa[threadIdx.x] = a;
    sd[threadIdx.x] = d;
    __syncthreads();
    for (int o = 128; o > 0; o >>= 1) {
        if ((int)threadIdx.x < o) {
            sa[threadIdx.x] += sa[threadIdx.x + o];
            sd[threadIdx.x] += sd[threadIdx.x + o];
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        p.dA[h] = sa[0];
        if (p.dD) p.dD[h] = sd[0];
    }
}

}  // namespace

PackedGradLayout packed_grad_layout(int64_t nseq, int64_t total, int H, int ctas)
{
    // Blocks of heads, where a group has more than one (ceil(R / S) <= 2 R / S of them): of kMaxBlock at most
    // m64 H / 4, and of S < kMaxBlock, S = the fair share of m64 H / ctas rounded down, fewer than 4 ctas
    const int64_t m64 = packed_layout(nseq, total).m64, blocks = std::max<int64_t>(4 * ctas, 2 * m64 * H / kMaxBlock);
    auto round = [](size_t b) { return (b + 255) & ~size_t(255); };
    PackedGradLayout l;
    // The states' images: in two parts for all chunks, in three for those of fewer than kManyRows rows
    size_t images = (size_t)m64 * kImage<3>;
    if (either_form(total, H)) images = std::max((size_t)m64 * kImage<2>, (size_t)((kManyRows - 1) / kQ + nseq) * kImage<3>);
    l.off_part = images * H * 2;
    l.off_sums = l.off_part + (size_t)blocks * (2 * kQ * kN) * sizeof(float);
    l.off_pA = l.off_sums + round((size_t)ctas * 2 * kSumFloats * sizeof(float));
    l.off_pD = l.off_pA + round((size_t)m64 * H * sizeof(float));
    l.bytes = l.off_pD + round((size_t)m64 * H * sizeof(float));
    return l;
}

template <bool kEither>
static int launch_forms(const PackedGradParams &p, int ctas, cudaStream_t st)
{
    static SmemLimit walk_done, grad_done;
    constexpr size_t walk = kEither ? std::max(sizeof(SmemWalk<2>), sizeof(SmemWalk<3>)) : sizeof(SmemWalk<3>);
    constexpr size_t grad = kEither ? std::max(sizeof(SmemGrad<2>), sizeof(SmemGrad<3>)) : sizeof(SmemGrad<3>);
    if (!allow_smem(packed_grad_walk_kernel<kEither>, (int)walk, walk_done) || !allow_smem(packed_grad_tc_kernel<kEither>, (int)grad, grad_done))
        return 7;
    // parts of the chunk list: two waves of one CTA per SM, no more parts than sequences (they begin between sequences)
    const int64_t wide = 2 * (int64_t)p.H;
    const int64_t parts = std::max<int64_t>(1, std::min<int64_t>(p.plan.nseq, (2 * (int64_t)ctas + wide - 1) / wide));
    const int64_t units = kSumParts * p.plan.m64 * p.G + p.H + p.plan.nseq;
    if (units > 0x7fffffff) return 2;
    prof_begin(st, kKBwdChain);
    packed_grad_walk_kernel<kEither><<<dim3((unsigned)wide, (unsigned)parts), kWalkThreads, walk, st>>>(p);
    prof_end(st, kKBwdChain);
    prof_begin(st, kKBwdGrad);
    packed_grad_tc_kernel<kEither><<<(unsigned)ctas, kGradThreads, grad, st>>>(p);
    prof_end(st, kKBwdGrad);
    prof_begin(st, kKBwdReduce);
    packed_grad_sum_kernel<<<(unsigned)units, 256, 0, st>>>(p, ctas);
    prof_end(st, kKBwdReduce);
    return cudaGetLastError() == cudaSuccess ? 0 : 7;
}

int launch_packed_grad_tc(const PackedGradParams &p, int ctas, cudaStream_t st)
{
    return either_form(p.plan.total, p.H) ? launch_forms<true>(p, ctas, st) : launch_forms<false>(p, ctas, st);
}

}  // namespace ssd

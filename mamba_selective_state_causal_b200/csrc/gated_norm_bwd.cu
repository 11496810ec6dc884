// gated_norm_bwd.cu -- gradient of the block's output norm  out = v r w,  v = y silu(z),
// r = 1 / sqrt(mean over the channel group of v^2 + eps).  With g = dout w:
//   dv = r (g - v r^2 mean(g v)),   dy = dv silu(z),   dz = dv y silu'(z),   dw = sum over rows of dout v r,
//   silu(z) = z sg,  silu'(z) = sg (1 + z (1 - sg)),  sg = 1 / (1 + e^-z).
// A row is read once (y, z, dout) and written once (dy, dz): 5 d elements, the memory's rate is the
// bound.  A thread owns 8 channels; its pieces of the next kDepth rows stream by cp.async through its own
// slots of shared memory (48 KB per CTA, two CTAs per SM), so that loads never wait for the two sums
// over the group (of v^2 and of g v, both at once, in a fixed order).  Its share of dw stays in 8 registers
// over all the rows that its CTA walks, is written once per CTA, and is added over the CTAs by a second kernel
// in a fixed order: no atomics, the same result every time.  65536 rows of 2048: 222 to 253 us on
// different machines, 0.81 to 0.92 of the copy rate.
// Sums over a group: of 8 m channels, m threads.  m a power of two up to 32: shuffles among those
// lanes.  m a multiple of 32: shuffles, then the warps' sums through shared memory.  Any other m: every
// thread adds its group's m values in shared memory (rare widths, not tuned).
#include <algorithm>
#include <type_traits>

#include "norm_bwd.cuh"
#include "packed.cuh"

namespace ssd {
namespace {

constexpr int kV = 8;

__device__ __forceinline__ void cp16(void *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}

__device__ __forceinline__ void unpack8f(const uint4 &a, float (&v)[8])
{
    v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x); v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
    v[4] = bf16_lo(a.z); v[5] = bf16_hi(a.z); v[6] = bf16_lo(a.w); v[7] = bf16_hi(a.w);
}

// 8 elements in shared memory
template <typename T> struct Vec8;
template <> struct Vec8<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void fetch(const __nv_bfloat16 *p) { cp16(&a, p); }
    __device__ __forceinline__ void get(float (&v)[8]) const { unpack8f(a, v); }
    __device__ __forceinline__ static void put(__nv_bfloat16 *p, const float (&v)[8])
    {
        __stcs(reinterpret_cast<uint4 *>(p), make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                         pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
    }
};
template <> struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void fetch(const float *p) { cp16(&a, p); cp16(&b, p + 4); }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
    __device__ __forceinline__ static void put(float *p, const float (&v)[8])
    {
        __stcs(reinterpret_cast<float4 *>(p), make_float4(v[0], v[1], v[2], v[3]));
        __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
    }
};
template <typename T> constexpr int kDepth = 96 / (3 * (int)sizeof(Vec8<T>)) * 2;   // 4 rows of bf16, 2 of fp32: 192 bytes per thread

// One CTA: `teams` rows side by side, d / 8 threads each; it walks the rows blockIdx.x * teams + team, a grid apart.
// kMode: 0 groups of a power of two up to 32 threads, 1 of a multiple of 32, 2 any.
// kMost bounds the threads, and with them the registers.  Two CTAs of 256 threads per SM leave the 128 registers that
// a thread needs: 222 us at 65536 rows of 2048 in bf16 on one machine (6.0 TB/s), against 294 with three (80
// registers, a few of them spilled) and 335 with four.  Wider rows take one CTA per SM of 512 threads (122 registers;
// 4096 channels 0.8 to 0.9 of the copy rate), 640 (96; 5120 channels 0.7 to 0.8, with the 64 registers that 1024
// threads leave 0.33) or up to 1024 (spilled; 8192 channels 0.44).
template <typename T, int kMode, int kMost>
__global__ void __launch_bounds__(kMost, kMost == 256 ? 2 : 1) gated_norm_bwd_kernel(NormBwdParams p, int teams)
{
    extern __shared__ __align__(16) uint8_t raw[];
    constexpr int D = kDepth<T>;
    Vec8<T> *ring = reinterpret_cast<Vec8<T> *>(raw) + threadIdx.x;               // [D][3][threads]
    float2 *part = reinterpret_cast<float2 *>(raw + sizeof(Vec8<T>) * 3 * D * blockDim.x);   // mode 1: [2][warps]; mode 2: [2][threads]
    const int per = p.d / kV;                    // threads of a row
    const int team = threadIdx.x / per, i = threadIdx.x % per;
    const bool live = team < teams;
    const int m = p.group / kV;                  // threads of a group
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const float inv = 1.0f / (float)p.group;
    float2 wv[4] = {}, dw[4] = {};
    if (live) {
#pragma unroll
        for (int k = 0; k < 4; ++k) wv[k] = __ldg(reinterpret_cast<const float2 *>(p.w + kV * i) + k);
    }
    const int64_t step = (int64_t)gridDim.x * teams;
    const int64_t r0 = (int64_t)blockIdx.x * teams + team;
    // the rows of every team in step: the CTA's first row decides the number of turns, its own this thread's
    const int64_t first = (int64_t)blockIdx.x * teams;
    const int turns = first < p.rows ? (int)((p.rows - first + step - 1) / step) : 0;
    const int mine = live && r0 < p.rows ? (int)((p.rows - r0 + step - 1) / step) : 0;
    const T *yp = reinterpret_cast<const T *>(p.y) + r0 * p.yrs + kV * i, *zp = reinterpret_cast<const T *>(p.z) + r0 * p.zrs + kV * i;
    const T *op = reinterpret_cast<const T *>(p.dout) + r0 * p.dors + kV * i;
    T *dyp = reinterpret_cast<T *>(p.dy) + r0 * p.dyrs + kV * i, *dzp = reinterpret_cast<T *>(p.dz) + r0 * p.dzrs + kV * i;
    const int64_t ys = step * p.yrs, zs = step * p.zrs, os = step * p.dors, dys = step * p.dyrs, dzs = step * p.dzrs;
    const int nt = blockDim.x;
    auto fetch = [&](int k) {                    // rows are fetched in order: the pointers step along
        if (k < mine) {
            Vec8<T> *q = ring + (k % D) * 3 * nt;
            q[0].fetch(yp);
            q[nt].fetch(zp);
            q[2 * nt].fetch(op);
            yp += ys; zp += zs; op += os;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int k = 0; k < D; ++k) fetch(k);
#pragma unroll 1
    for (int k = 0; k < turns; ++k) {
        const bool on = k < mine;
        const Vec8<T> *q = ring + (k % D) * 3 * nt;
        asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");    // row k's group is the oldest
        float2 s = make_float2(0.f, 0.f);        // sums of v^2 and g v
        // until the outputs: sigma(z), silu(z), y and g of 4 pairs of channels
        float2 sg[4], si[4], y2[4], o2[4];
        if (on) {
            float y[8], z[8], o[8];
            q[0].get(y); q[nt].get(z); q[2 * nt].get(o);
            float2 vv = make_float2(0.f, 0.f), gv = vv;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y2[e] = make_float2(y[2 * e], y[2 * e + 1]);
                o2[e] = make_float2(o[2 * e], o[2 * e + 1]);
                sg[e] = make_float2(sigma_fast(z[2 * e]), sigma_fast(z[2 * e + 1]));
                si[e] = __fmul2_rn(make_float2(z[2 * e], z[2 * e + 1]), sg[e]);
                const float2 v = __fmul2_rn(y2[e], si[e]);
                vv = __ffma2_rn(v, v, vv);
                gv = __ffma2_rn(__fmul2_rn(o2[e], wv[e]), v, gv);
            }
            s = make_float2(vv.x + vv.y, gv.x + gv.y);
        }
        fetch(k + D);                            // into the slots just read, which are this thread's own
        if (kMode == 0) {
            for (int o = 1; o < m; o <<= 1) {
                s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
                s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
            }
        }
        if (kMode == 1) {
            // half of the lanes sum v^2, the other half g v: 5 exchanges for the two sums
            const bool up = (lane & 16) != 0;
            float t = up ? s.y : s.x;
            t += __shfl_xor_sync(0xffffffffu, up ? s.x : s.y, 16);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            float *b = reinterpret_cast<float *>(part + (k & 1) * warps);    // two in turn: one barrier per row
            if ((lane & 15) == 0) b[2 * warp + (up ? 1 : 0)] = t;
            __syncthreads();
            const int mw = m / 32;
            const float2 *b2 = part + (k & 1) * warps + warp / mw * mw;
            s = b2[0];
            if (mw == 8) {
#pragma unroll
                for (int e = 1; e < 8; ++e) s = __fadd2_rn(s, b2[e]);
            } else {
                for (int e = 1; e < mw; ++e) s = __fadd2_rn(s, b2[e]);
            }
        }
        if (kMode == 2) {
            float2 *b = part + (k & 1) * nt;
            b[threadIdx.x] = s;
            __syncthreads();
            if (live) {
                const int t0 = team * per + i / m * m;
                s = make_float2(0.f, 0.f);
                for (int e = 0; e < m; ++e) { const float2 t = b[t0 + e]; s.x += t.x; s.y += t.y; }
            }
        }
        if (on) {
            float a[8], b[8];
            const float rs = rsqrtf(fmaf(s.x, inv, p.eps));
            const float c = -rs * rs * (s.y * inv);
            const float2 rs2 = make_float2(rs, rs), c2 = make_float2(c, c);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 v = __fmul2_rn(y2[e], si[e]);
                const float2 dv = __fmul2_rn(rs2, __ffma2_rn(v, c2, __fmul2_rn(o2[e], wv[e])));
                const float2 da = __fmul2_rn(dv, si[e]);
                // silu'(z) = sg + si (1 - sg)
                const float2 one = make_float2(1.0f - sg[e].x, 1.0f - sg[e].y);
                const float2 db = __fmul2_rn(__fmul2_rn(dv, y2[e]), __ffma2_rn(si[e], one, sg[e]));
                a[2 * e] = da.x; a[2 * e + 1] = da.y;
                b[2 * e] = db.x; b[2 * e + 1] = db.y;
                dw[e] = __ffma2_rn(__fmul2_rn(o2[e], rs2), v, dw[e]);
            }
            Vec8<T>::put(dyp, a);
            Vec8<T>::put(dzp, b);
            dyp += dys; dzp += dzs;
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (live) {
        float4 *q = reinterpret_cast<float4 *>(p.ws + ((int64_t)blockIdx.x * teams + team) * p.d + kV * i);
        q[0] = make_float4(dw[0].x, dw[0].y, dw[1].x, dw[1].y);
        q[1] = make_float4(dw[2].x, dw[2].y, dw[3].x, dw[3].y);
    }
}

// dw: the CTAs' sums, added in a fixed order.  A CTA takes 32 channels, each of its 16 warps every 16th sum.
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(32 * kSumWarps) gated_norm_dw_kernel(NormBwdParams p, int parts)
{
    __shared__ float sm[kSumWarps][32];
    const int cl = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + cl;
    float acc = 0.0f;
    if (c < p.d) {
        for (int i0 = sl; i0 < parts; i0 += 8 * kSumWarps) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int i = i0 + k * kSumWarps;
                v[k] = i < parts ? p.ws[(int64_t)i * p.d + c] : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) acc += v[k];
        }
    }
    sm[sl][cl] = acc;
    __syncthreads();
    if (sl == 0 && c < p.d) {
        for (int k = 1; k < kSumWarps; ++k) acc += sm[k][cl];
        p.dw[c] = acc;
    }
}

template <typename T, int kMode, int kMost>
int launch_mode(const NormBwdParams &p, const NormBwdPlan &pl, cudaStream_t st)
{
    const size_t smem = sizeof(Vec8<T>) * 3 * kDepth<T> * pl.threads +
                        sizeof(float2) * 2 * (kMode == 0 ? 0 : kMode == 1 ? pl.threads / 32 : pl.threads);
    static SmemLimit done;
    if (!allow_smem(gated_norm_bwd_kernel<T, kMode, kMost>, (int)smem, done)) return 7;
    prof_begin(st, kKGatedNormBwd);
    gated_norm_bwd_kernel<T, kMode, kMost><<<(unsigned)pl.grid, pl.threads, smem, st>>>(p, pl.teams);
    gated_norm_dw_kernel<<<(unsigned)((p.d + 31) / 32), 32 * kSumWarps, 0, st>>>(p, pl.grid * pl.teams);
    prof_end(st, kKGatedNormBwd);
    return cudaGetLastError() == cudaSuccess ? 0 : 7;
}

template <typename T, int kMost>
int launch_t(const NormBwdParams &p, const NormBwdPlan &pl, cudaStream_t st)
{
    const int m = p.group / kV;
    // rows start at multiples of 32 threads, or their groups do not straddle warps
    const bool whole = (p.d / kV) % 32 == 0;
    if (m <= 32 && (m & (m - 1)) == 0) return launch_mode<T, 0, kMost>(p, pl, st);
    if (m % 32 == 0 && whole) return launch_mode<T, 1, kMost>(p, pl, st);
    return launch_mode<T, 2, kMost>(p, pl, st);
}

}  // namespace

// Threads: whole rows side by side up to 256 threads (wider rows: their own d / 8), rounded up to
// warps.  Grid: the 512 threads that fit an SM, on each of them, and no more than there are rows.
NormBwdPlan norm_bwd_plan(int64_t rows, int d, int sms)
{
    NormBwdPlan pl;
    const int per = d / kV;
    pl.teams = std::max(1, 256 / per);
    pl.threads = (pl.teams * per + 31) / 32 * 32;
    const int64_t need = (rows + pl.teams - 1) / pl.teams;
    pl.grid = (int)std::max<int64_t>(1, std::min<int64_t>(need, (int64_t)sms * std::max(1, 512 / pl.threads)));
    return pl;
}

int launch_gated_norm_backward(const NormBwdParams &p, int dtype, int sms, cudaStream_t st)
{
    const NormBwdPlan pl = norm_bwd_plan(p.rows, p.d, sms);
    const bool b = dtype == 1;
    if (pl.threads <= 256) return b ? launch_t<__nv_bfloat16, 256>(p, pl, st) : launch_t<float, 256>(p, pl, st);
    if (pl.threads <= 512) return b ? launch_t<__nv_bfloat16, 512>(p, pl, st) : launch_t<float, 512>(p, pl, st);
    if (pl.threads <= 640) return b ? launch_t<__nv_bfloat16, 640>(p, pl, st) : launch_t<float, 640>(p, pl, st);
    return b ? launch_t<__nv_bfloat16, 1024>(p, pl, st) : launch_t<float, 1024>(p, pl, st);
}

}  // namespace ssd

// gated_norm_bwd.cu -- gradient of the block's output norm  out = v r w,  v = y silu(z),
// r = 1 / sqrt(mean over the channel group of v^2 + eps).  With g = dout w:
//   dv = r (g - v r^2 mean(g v)),   dy = dv silu(z),   dz = dv y silu'(z),   dw = sum over rows of dout v r,
//   silu(z) = z sg,  silu'(z) = sg (1 + z (1 - sg)),  sg = 1 / (1 + e^-z).
// A row is read once (y, z, dout) and written once (dy, dz): 5 d elements, the memory's rate is the
// bound.  A thread owns 8 channels and keeps kRows rows of them in registers (three 16-byte loads per
// row in bf16) between the two sums over the group (of v^2 and of g v, both at once, in a fixed order)
// and the outputs; the next rows' loads come from the other CTAs of the SM.  Its share of dw stays in
// 8 registers over all the rows that its CTA walks, is written once per CTA, and is added over the
// CTAs by a second kernel in a fixed order: no atomics, the same result every time.
// Sums over a group: of 8 m channels, m threads.  m a power of two up to 32: shuffles among those
// lanes.  m a multiple of 32: shuffles, then the warps' sums through shared memory.  Any other m: every
// thread adds its group's m values in shared memory (rare widths, not tuned).
#include <algorithm>
#include <type_traits>

#include "norm_bwd.cuh"

namespace ssd {
namespace {

constexpr int kV = 8;

__device__ __forceinline__ void unpack8f(const uint4 &a, float (&v)[8])
{
    v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x); v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
    v[4] = bf16_lo(a.z); v[5] = bf16_hi(a.z); v[6] = bf16_lo(a.w); v[7] = bf16_hi(a.w);
}

// 8 elements as loaded, packed while they wait
template <typename T> struct Pack8;
template <> struct Pack8<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = __ldcs(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void get(float (&v)[8]) const { unpack8f(a, v); }
    __device__ __forceinline__ static void put(__nv_bfloat16 *p, const float (&v)[8])
    {
        __stcs(reinterpret_cast<uint4 *>(p), make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                         pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
    }
};
template <> struct Pack8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = __ldcs(reinterpret_cast<const float4 *>(p));
        b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    }
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

// sigma(z) with the hardware exponential (bf16) or the library's (fp32); -z is clamped so that the
// divisor stays finite (sigma is below 2e-35 there either way)
template <typename T> __device__ __forceinline__ float sigma(float z)
{
    return std::is_same<T, float>::value ? 1.0f / (1.0f + expf(fminf(-z, 80.0f)))
                                         : __fdividef(1.0f, 1.0f + __expf(fminf(-z, 80.0f)));
}

// One CTA: `teams` rows side by side, d / 8 threads each, kRows rows of each in registers at once.
// kMode: 0 groups of a power of two up to 32 threads, 1 of a multiple of 32, 2 any.
// kMost bounds the threads (rows wider than 4096 channels need up to 1024 and take one row at a time).
template <typename T, int kRows, int kMode, int kMost>
__global__ void __launch_bounds__(kMost) gated_norm_bwd_kernel(NormBwdParams p, int teams)
{
    extern __shared__ float2 part[];             // mode 1: [2][kRows][warps]; mode 2: [2][kRows][threads]
    const int per = p.d / kV;                    // threads of a row
    const int team = threadIdx.x / per, i = threadIdx.x % per;
    const bool live = team < teams;
    const int m = p.group / kV;                  // threads of a group
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const float inv = 1.0f / (float)p.group;
    float wv[8], dw[8] = {};
    if (live) {
#pragma unroll
        for (int k = 0; k < 8; ++k) wv[k] = __ldg(p.w + kV * i + k);
    }
    const T *yb = reinterpret_cast<const T *>(p.y) + kV * i, *zb = reinterpret_cast<const T *>(p.z) + kV * i;
    const T *ob = reinterpret_cast<const T *>(p.dout) + kV * i;
    const int64_t step = (int64_t)gridDim.x * teams * kRows;
    int buf = 0;
    for (int64_t base = (int64_t)blockIdx.x * teams * kRows; base < p.rows; base += step, buf ^= 1) {
        const int64_t r0 = base + (int64_t)team * kRows;
        Pack8<T> py[kRows], pz[kRows], po[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (live && r0 + r < p.rows) {
                py[r].load(yb + (r0 + r) * p.yrs);
                pz[r].load(zb + (r0 + r) * p.zrs);
                po[r].load(ob + (r0 + r) * p.dors);
            } else {
                py[r] = {}; pz[r] = {}; po[r] = {};
            }
        }
        float2 s[kRows];                         // sums of v^2 and g v
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            float y[8], z[8], o[8];
            py[r].get(y); pz[r].get(z); po[r].get(o);
            s[r] = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float v = y[k] * (z[k] * sigma<T>(z[k]));
                s[r].x = fmaf(v, v, s[r].x);
                s[r].y = fmaf(o[k] * wv[k], v, s[r].y);
            }
        }
        if (kMode <= 1) {
            const int span = kMode == 0 ? m : 32;
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                for (int o = 1; o < span; o <<= 1) {
                    s[r].x += __shfl_xor_sync(0xffffffffu, s[r].x, o);
                    s[r].y += __shfl_xor_sync(0xffffffffu, s[r].y, o);
                }
        }
        if (kMode == 1) {
            float2 *q = part + buf * kRows * warps;
            if (lane == 0) {
#pragma unroll
                for (int r = 0; r < kRows; ++r) q[r * warps + warp] = s[r];
            }
            __syncthreads();                     // one per step: the buffers alternate
            const int mw = m / 32, first = warp / mw * mw;
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                s[r] = make_float2(0.f, 0.f);
                for (int k = 0; k < mw; ++k) { const float2 t = q[r * warps + first + k]; s[r].x += t.x; s[r].y += t.y; }
            }
        }
        if (kMode == 2) {
            float2 *q = part + buf * kRows * blockDim.x;
#pragma unroll
            for (int r = 0; r < kRows; ++r) q[r * blockDim.x + threadIdx.x] = s[r];
            __syncthreads();
            const int first = live ? team * per + i / m * m : 0;
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                s[r] = make_float2(0.f, 0.f);
                if (live)
                    for (int k = 0; k < m; ++k) { const float2 t = q[r * blockDim.x + first + k]; s[r].x += t.x; s[r].y += t.y; }
            }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (!live || r0 + r >= p.rows) continue;
            float y[8], z[8], o[8], a[8], b[8];
            py[r].get(y); pz[r].get(z); po[r].get(o);
            const float rs = 1.0f / sqrtf(fmaf(s[r].x, inv, p.eps));
            const float c = rs * rs * (s[r].y * inv);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float sg = sigma<T>(z[k]), si = z[k] * sg, v = y[k] * si;
                const float dv = rs * fmaf(-v, c, o[k] * wv[k]);
                a[k] = dv * si;
                b[k] = dv * y[k] * (sg * fmaf(z[k], 1.0f - sg, 1.0f));
                dw[k] = fmaf(o[k] * rs, v, dw[k]);
            }
            Pack8<T>::put(reinterpret_cast<T *>(p.dy) + (r0 + r) * p.dyrs + kV * i, a);
            Pack8<T>::put(reinterpret_cast<T *>(p.dz) + (r0 + r) * p.dzrs + kV * i, b);
        }
    }
    if (live) {
        float4 *q = reinterpret_cast<float4 *>(p.ws + ((int64_t)blockIdx.x * teams + team) * p.d + kV * i);
        q[0] = make_float4(dw[0], dw[1], dw[2], dw[3]);
        q[1] = make_float4(dw[4], dw[5], dw[6], dw[7]);
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

template <typename T, int kRows, int kMode, int kMost>
int launch_mode(const NormBwdParams &p, const NormBwdPlan &pl, cudaStream_t st)
{
    const size_t smem = sizeof(float2) * 2 * kRows * (kMode == 0 ? 0 : kMode == 1 ? pl.threads / 32 : pl.threads);
    prof_begin(st, kKGatedNormBwd);
    gated_norm_bwd_kernel<T, kRows, kMode, kMost><<<(unsigned)pl.grid, pl.threads, smem, st>>>(p, pl.teams);
    gated_norm_dw_kernel<<<(unsigned)((p.d + 31) / 32), 32 * kSumWarps, 0, st>>>(p, pl.grid * pl.teams);
    prof_end(st, kKGatedNormBwd);
    return cudaGetLastError() == cudaSuccess ? 0 : 7;
}

template <typename T, int kRows, int kMost>
int launch_t(const NormBwdParams &p, const NormBwdPlan &pl, cudaStream_t st)
{
    const int m = p.group / kV;
    // rows start at multiples of 32 threads, or their groups do not straddle warps
    const bool whole = (p.d / kV) % 32 == 0;
    if (m <= 32 && (m & (m - 1)) == 0) return launch_mode<T, kRows, 0, kMost>(p, pl, st);
    if (m % 32 == 0 && whole) return launch_mode<T, kRows, 1, kMost>(p, pl, st);
    return launch_mode<T, kRows, 2, kMost>(p, pl, st);
}

}  // namespace

// Threads: whole rows side by side up to 256 threads (wider rows: their own d / 8), rounded up to
// warps.  Grid: what fits two CTAs' worth of 512 threads on each of the SMs, and no more than there are rows.
NormBwdPlan norm_bwd_plan(int64_t rows, int d, int dtype, int sms)
{
    NormBwdPlan pl;
    const int per = d / kV;
    pl.rows = per > 512 ? 1 : (dtype == 1 ? 4 : 2);
    pl.teams = std::max(1, 256 / per);
    pl.threads = (pl.teams * per + 31) / 32 * 32;
    const int64_t need = (rows + pl.teams * pl.rows - 1) / (pl.teams * pl.rows);
    pl.grid = (int)std::max<int64_t>(1, std::min<int64_t>(need, (int64_t)sms * std::max(1, 1024 / pl.threads)));
    return pl;
}

int launch_gated_norm_backward(const NormBwdParams &p, int dtype, int sms, cudaStream_t st)
{
    const NormBwdPlan pl = norm_bwd_plan(p.rows, p.d, dtype, sms);
    if (pl.rows == 1) return dtype == 1 ? launch_t<__nv_bfloat16, 1, 1024>(p, pl, st) : launch_t<float, 1, 1024>(p, pl, st);
    return dtype == 1 ? launch_t<__nv_bfloat16, 4, 512>(p, pl, st) : launch_t<float, 2, 512>(p, pl, st);
}

}  // namespace ssd

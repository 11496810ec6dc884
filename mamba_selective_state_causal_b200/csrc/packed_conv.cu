// packed_conv.cu -- the layer's causal convolution (kernel 4) and SiLU over sequences laid end to end,
// forward and backward:
//   z[t,c] = bias_c + sum_k w[c,k] u[t-3+k,c],   v = z sigma(z),
// where the rows before a sequence's first come from the 3-row buffer of its slot (zeros when it
// does not resume), never from the sequence that lies before it in the tensor.
//
// Forward.  A thread owns one 16-byte vector of channels over the rows of a 64-row chunk; they stream
// through its own kRing slots of shared memory by cp.async, which keeps 128 KB of loads in flight per SM
// without holding registers.  Every row is read once, plus three rows of halo per thread, and
// written once: the bound is the memory's rate.  The arithmetic and its order are the layer's
// convolution's, so that a packed sequence gets the same v bit for bit.  The thread of a sequence's
// first rows also writes its buffer: nobody else reads the slot's old one, so that tail_out may be
// tail_in.
#include <algorithm>

#include "packed.cuh"

namespace ssd {
namespace {

struct alignas(16) Vec16p { uint32_t w[4]; };

__device__ __forceinline__ Vec16p ld_rows(const void *p)
{
    Vec16p r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
                 : "l"(p));
    return r;
}

template <typename T> struct ConvVec;
template <> struct ConvVec<__nv_bfloat16> {
    static constexpr int kN = 8;
    __device__ __forceinline__ static void unpack(const Vec16p &v, float *f)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) { f[2 * i] = bf16_lo(v.w[i]); f[2 * i + 1] = bf16_hi(v.w[i]); }
    }
    __device__ __forceinline__ static Vec16p pack(const float *f)
    {
        Vec16p v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v.w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
        return v;
    }
    // weights and bias halved (exact): the sum is h = z / 2 and z sigma(z) = h + h tanh(h), one
    // hardware tanh (relative error about 2^-11) before the rounding to bf16 (2^-9)
    static constexpr float kPre = 0.5f;
    __device__ __forceinline__ static float silu(float h)
    {
        float t;
        asm("tanh.approx.f32 %0, %1;" : "=f"(t) : "f"(h));
        return fmaf(h, t, h);
    }
};
template <> struct ConvVec<float> {
    static constexpr int kN = 4;
    __device__ __forceinline__ static void unpack(const Vec16p &v, float *f)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v.w[i]);
    }
    __device__ __forceinline__ static Vec16p pack(const float *f)
    {
        Vec16p v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v.w[i] = __float_as_uint(f[i]);
        return v;
    }
    static constexpr float kPre = 1.0f;
    __device__ __forceinline__ static float silu(float z) { return z / (1.0f + expf(-z)); }
};

constexpr int kPackedConvThreads = 256;
constexpr int kRing = 16;          // rows in flight per thread

__device__ __forceinline__ void cp_row(void *smem, const void *gmem)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(gmem)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <typename T>
__global__ void __launch_bounds__(kPackedConvThreads, 2) packed_conv_kernel(PackedConvParams p)
{
    using IO = ConvVec<T>;
    constexpr int V = IO::kN;
    extern __shared__ Vec16p ring[];                        // [kRing][threads]
    const int ncv = p.C_ch / V;
    const int64_t gid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int c0 = (int)(gid % ncv) * V;
    const int64_t chunk = gid / ncv;
    int4 d;
    if (!packed_chunk64(p.plan, chunk, p.status, d)) return;
    const int n = d.y & kChunkRows;
    const bool head = (d.y & kChunkFirst) != 0;
    const T *u = reinterpret_cast<const T *>(p.u) + c0;
    const int64_t t0 = d.x;
    const T *up = u + t0 * p.urs;
    Vec16p *slot = ring + threadIdx.x;
    // one commit group per row (empty ones past the end keep the count uniform)
#pragma unroll
    for (int j = 0; j < kRing; ++j) {
        if (j < n) cp_row(slot + j * kPackedConvThreads, up + j * p.urs);
        cp_commit();
    }
    const bool kept = d.w >= 0;
    const int64_t tail = kept ? (int64_t)d.w * 3 * p.C_ch + c0 : 0;
    const T *tin = (p.tail_in && kept && (d.y & kChunkResume)) ? reinterpret_cast<const T *>(p.tail_in) + tail : nullptr;
    Vec16p m[3];                                            // rows t0 - 3 .. t0 - 1
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        if (!head) m[k] = ld_rows(u + (t0 - 3 + k) * p.urs);
        else if (tin) m[k] = *reinterpret_cast<const Vec16p *>(tin + k * p.C_ch);
        else m[k] = Vec16p{{0u, 0u, 0u, 0u}};
    }
    float w0[V], w1[V], w2[V], w3[V], bs[V];
    const float4 *wp = reinterpret_cast<const float4 *>(p.w + (int64_t)c0 * 4);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float4 q = __ldg(wp + i);
        w0[i] = IO::kPre * q.x; w1[i] = IO::kPre * q.y; w2[i] = IO::kPre * q.z; w3[i] = IO::kPre * q.w;
        bs[i] = p.bias ? IO::kPre * __ldg(p.bias + c0 + i) : 0.0f;
    }
    float m3[V], m2[V], m1[V];
    IO::unpack(m[0], m3);
    IO::unpack(m[1], m2);
    IO::unpack(m[2], m1);
    if (head && kept && p.tail_out) {
        // the last three rows of the sequence, or of its old buffer and it when it is shorter
        const PackedSeq s = p.plan.seqs[d.z];
        T *to = reinterpret_cast<T *>(p.tail_out) + tail;
#pragma unroll
        for (int r = 0; r < 3; ++r) {
            const int pos = s.len - 3 + r;                  // < 0: row 3 + pos of the old buffer
            Vec16p o;
            if (pos >= 0) {
                o = ld_rows(u + ((int64_t)s.row0 + pos) * p.urs);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) o.w[e] = pos == -3 ? m[0].w[e] : (pos == -2 ? m[1].w[e] : m[2].w[e]);
            }
            *reinterpret_cast<Vec16p *>(to + r * p.C_ch) = o;
        }
    }
    T *vp = reinterpret_cast<T *>(p.v) + t0 * p.vrs + c0;
    up += kRing * p.urs;
    for (int i0 = 0; i0 < n; i0 += kRing) {
#pragma unroll
        for (int j = 0; j < kRing; ++j) {
            if (i0 + j < n) {
                cp_wait<kRing - 1>();                       // row i0 + j has landed (its group is the oldest)
                float cur[V], out[V];
                IO::unpack(slot[j * kPackedConvThreads], cur);
                if (i0 + j + kRing < n) cp_row(slot + j * kPackedConvThreads, up);
                cp_commit();
                up += p.urs;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float z = bs[i];
                    z = fmaf(w0[i], m3[i], z);
                    z = fmaf(w1[i], m2[i], z);
                    z = fmaf(w2[i], m1[i], z);
                    z = fmaf(w3[i], cur[i], z);
                    out[i] = IO::silu(z);
                    m3[i] = m2[i]; m2[i] = m1[i]; m1[i] = cur[i];
                }
                *reinterpret_cast<Vec16p *>(vp) = IO::pack(out);
                vp += p.vrs;
            }
        }
    }
    cp_wait<0>();
}

template <typename T>
int launch_conv_t(const PackedConvParams &p, cudaStream_t st)
{
    const int64_t threads = p.plan.m64 * (p.C_ch / ConvVec<T>::kN);
    const int64_t blocks = (threads + kPackedConvThreads - 1) / kPackedConvThreads;
    if (blocks > 0x7fffffffLL) return 2;
    constexpr int smem = kRing * kPackedConvThreads * (int)sizeof(Vec16p);
    static std::atomic<int> done[64];
    if (!allow_smem(packed_conv_kernel<T>, smem, done)) return 7;
    prof_begin(st, kKPackedConv);
    packed_conv_kernel<T><<<(unsigned)blocks, kPackedConvThreads, smem, st>>>(p);
    prof_end(st, kKPackedConv);
    return cudaGetLastError() == cudaSuccess ? 0 : 7;
}

// ---------------------------------------------------------------- backward
// dz = dv sigma(z) (1 + z (1 - sigma(z)));  du[t] = sum_j w[3-j] dz[t+j] over the rows of t's own
// sequence (plus dLoss/d(buffer handed on) at its last three rows);  dw[k] = sum_t dz[t] u[t-3+k],
// dbias = sum_t dz[t];  the gradient of the buffer that a sequence starts from: row 3 + q (position
// q < 0) reaches the rows t <= q + 3 through tap q - t + 3.
// A thread owns 4 channels over a 64-row chunk and walks it forward with the window of u and of dz
// in registers: du[t-3] is complete once dz[t] is, so it runs three rows past the chunk (recomputing
// their dz) instead of handing dz between threads.  The next kBack rows of u and dv are on their
// way while kBack rows are worked on.  dw and dbias are summed over the thread's rows in fp32, written
// per chunk, and added over the chunks in a fixed order by a second kernel.
constexpr int kBack = 4;
constexpr int kConvBwdT = 128;

__device__ __forceinline__ float4 ld4(const float *q) { return __ldg(reinterpret_cast<const float4 *>(q)); }
__device__ __forceinline__ float4 ld4(const __nv_bfloat16 *q)
{
    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(q));
    return make_float4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y));
}
// 4 elements as loaded
template <typename T> struct Raw4;
template <> struct Raw4<float> {
    float4 v;
    __device__ __forceinline__ void load(const float *q) { v = __ldcs(reinterpret_cast<const float4 *>(q)); }
    __device__ __forceinline__ float4 get() const { return v; }
};
template <> struct Raw4<__nv_bfloat16> {
    uint2 v;
    __device__ __forceinline__ void load(const __nv_bfloat16 *q) { v = __ldg(reinterpret_cast<const uint2 *>(q)); }
    __device__ __forceinline__ float4 get() const { return make_float4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)); }
};

__device__ __forceinline__ float dz1(float dv, float w0, float w1, float w2, float w3, float b, float a3, float a2,
                                     float a1, float a0)
{
    float z = b;
    z = fmaf(w0, a3, z);
    z = fmaf(w1, a2, z);
    z = fmaf(w2, a1, z);
    z = fmaf(w3, a0, z);
    // sigma through the hardware exponential (relative error about 2^-21); -z is clamped so that the
    // divisor stays below 2^126 (sigma is below 2e-35 there either way)
    const float sg = __fdividef(1.0f, 1.0f + __expf(fminf(-z, 80.0f)));
    return dv * (sg * fmaf(z, 1.0f - sg, 1.0f));
}

template <typename T>
__global__ void __launch_bounds__(kConvBwdT, 3) packed_conv_bwd_kernel(PackedConvBwdParams p)
{
    const int np = p.C_ch >> 2;
    const int64_t gid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int c = 4 * (int)(gid % np);
    const int64_t chunk = gid / np;
    int4 d;
    if (!packed_chunk64(p.plan, chunk, p.status, d)) return;
    const PackedSeq s = p.plan.seqs[d.z];
    const bool head = (d.y & kChunkFirst) != 0;
    const int64_t t0 = d.x, se = (int64_t)s.row0 + s.len;
    const int n = d.y & kChunkRows;
    const int nt = n > 0 ? n + 3 : 0;
    const int nin = (int)min((int64_t)nt, se - t0);  // rows past the sequence's end have dz = 0
    const T *u = reinterpret_cast<const T *>(p.u) + c + t0 * p.urs;
    // dv of 4 channels, all in one of x, B and C
    const float *dv;
    int64_t dvs;
    if (c < p.HP) { dv = p.dx + c; dvs = p.HP; }
    else if (c < p.HP + p.GN) { dv = p.dB + (c - p.HP); dvs = p.GN; }
    else { dv = p.dC + (c - p.HP - p.GN); dvs = p.GN; }
    dv += t0 * dvs;
    Raw4<T> un[kBack];
    Raw4<float> dn[kBack];
    auto fetch = [&](int b0) {
#pragma unroll
        for (int j = 0; j < kBack; ++j) {
            if (b0 + j < nin) {
                un[j].load(u + (int64_t)(b0 + j) * p.urs);
                dn[j].load(dv + (int64_t)(b0 + j) * dvs);
            } else {
                un[j] = {};
                dn[j] = {};
            }
        }
    };
    fetch(0);
    const bool resumed = p.tail_in && s.slot >= 0 && s.resume;
    const T *tin = resumed ? reinterpret_cast<const T *>(p.tail_in) + (int64_t)s.slot * 3 * p.C_ch + c : nullptr;
    const float4 z4 = make_float4(0.f, 0.f, 0.f, 0.f);
    float4 a3, a2, a1;                      // u[t-3], u[t-2], u[t-1]
    if (!head) { a3 = ld4(u - 3 * p.urs); a2 = ld4(u - 2 * p.urs); a1 = ld4(u - p.urs); }
    else if (tin) { a3 = ld4(tin); a2 = ld4(tin + p.C_ch); a1 = ld4(tin + 2 * p.C_ch); }
    else { a3 = z4; a2 = z4; a1 = z4; }
    float wk[4][4];                         // [tap][channel]
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 q = __ldg(reinterpret_cast<const float4 *>(p.w) + c + i);
        wk[0][i] = q.x; wk[1][i] = q.y; wk[2][i] = q.z; wk[3][i] = q.w;
    }
    float bs[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) bs[i] = p.bias ? __ldg(p.bias + c + i) : 0.0f;
    float gw[4][4] = {}, gb[4] = {};
    float e3[4] = {}, e2[4] = {}, e1[4] = {};       // dz[t-3], dz[t-2], dz[t-1] (zero before t0: those rows' du is another thread's)
    float *du = p.du + t0 * p.C_ch + c;
    // the gradient of the buffer that the sequence starts from, with dz of its first three rows in e1, e2, e3
    auto put_tail = [&]() {
        float g[3][4] = {};
        if (resumed) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                g[0][i] = wk[0][i] * e3[i];
                g[1][i] = fmaf(wk[1][i], e3[i], wk[0][i] * e2[i]);
                g[2][i] = fmaf(wk[2][i], e3[i], fmaf(wk[1][i], e2[i], wk[0][i] * e1[i]));
            }
            if (p.dtail_out) {
                // a sequence of fewer than three rows hands rows of its old buffer on
#pragma unroll
                for (int q = 0; q < 3; ++q) {
                    const int r = q - s.len;            // row of the new buffer that holds old row q
                    if (r >= 0) {
                        const float4 x = ld4(p.dtail_out + ((int64_t)d.z * 3 + r) * p.C_ch + c);
                        g[q][0] += x.x; g[q][1] += x.y; g[q][2] += x.z; g[q][3] += x.w;
                    }
                }
            }
        }
#pragma unroll
        for (int q = 0; q < 3; ++q)
            *reinterpret_cast<float4 *>(p.dtail_in + ((int64_t)d.z * 3 + q) * p.C_ch + c) =
                make_float4(g[q][0], g[q][1], g[q][2], g[q][3]);
    };
    if (n == 0 && head && p.dtail_in) put_tail();
#pragma unroll 1
    for (int b0 = 0; b0 < nt; b0 += kBack) {
        Raw4<T> uc[kBack];
        Raw4<float> dc[kBack];
#pragma unroll
        for (int j = 0; j < kBack; ++j) { uc[j] = un[j]; dc[j] = dn[j]; }
        if (b0 + kBack < nt) fetch(b0 + kBack);
#pragma unroll
        for (int j = 0; j < kBack; ++j) {
            const int r = b0 + j;
            if (r < nt) {
                const float4 uu = uc[j].get(), dd = dc[j].get();
                const float x3[4] = {a3.x, a3.y, a3.z, a3.w}, x2[4] = {a2.x, a2.y, a2.z, a2.w};
                const float x1[4] = {a1.x, a1.y, a1.z, a1.w}, x0[4] = {uu.x, uu.y, uu.z, uu.w};
                const float dvv[4] = {dd.x, dd.y, dd.z, dd.w};
                float g[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // (a row past the sequence's end has dv = 0, its window may be anything finite: cleared)
                    float e0 = dz1(dvv[i], wk[0][i], wk[1][i], wk[2][i], wk[3][i], bs[i], x3[i], x2[i], x1[i], x0[i]);
                    e0 = r < nin ? e0 : 0.0f;
                    g[i] = fmaf(wk[0][i], e0, fmaf(wk[1][i], e1[i], fmaf(wk[2][i], e2[i], wk[3][i] * e3[i])));
                    if (r < n) {
                        gb[i] += e0;
                        gw[0][i] = fmaf(e0, x3[i], gw[0][i]);
                        gw[1][i] = fmaf(e0, x2[i], gw[1][i]);
                        gw[2][i] = fmaf(e0, x1[i], gw[2][i]);
                        gw[3][i] = fmaf(e0, x0[i], gw[3][i]);
                    }
                    e3[i] = e2[i]; e2[i] = e1[i]; e1[i] = e0;
                }
                if (r == 2 && head && p.dtail_in) put_tail();
                if (r >= 3) {
                    const int64_t back = t0 + r - 3 - (se - 3);     // row of the buffer handed on that du's row is
                    if (p.dtail_out && back >= 0) {
                        const float4 q = ld4(p.dtail_out + ((int64_t)d.z * 3 + back) * p.C_ch + c);
                        g[0] += q.x; g[1] += q.y; g[2] += q.z; g[3] += q.w;
                    }
                    __stcs(reinterpret_cast<float4 *>(du + (int64_t)(r - 3) * p.C_ch), make_float4(g[0], g[1], g[2], g[3]));
                }
                a3 = a2; a2 = a1; a1 = uu;
            }
        }
    }
    float4 *pw = reinterpret_cast<float4 *>(p.ws_dw) + chunk * p.C_ch + c;
#pragma unroll
    for (int i = 0; i < 4; ++i) pw[i] = make_float4(gw[0][i], gw[1][i], gw[2][i], gw[3][i]);
    *reinterpret_cast<float4 *>(p.ws_db + chunk * p.C_ch + c) = make_float4(gb[0], gb[1], gb[2], gb[3]);
}

// dw and dbias: the chunks' sums, added in a fixed order.  A CTA takes 32 channels; each of its 16
// warps adds every 16th chunk's, 4 loads ahead, then warp 0 adds the 16 sums in order.
constexpr int kRedWarps = 16;
__global__ void __launch_bounds__(32 * kRedWarps) packed_conv_reduce_kernel(PackedConvBwdParams p)
{
    __shared__ float4 sw[kRedWarps][32];
    __shared__ float sb[kRedWarps][32];
    const int cl = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + cl;
    const int nparts = packed_n64(p.plan, p.status);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float ab = 0.0f;
    if (c < p.C_ch) {
        for (int i0 = sl; i0 < nparts; i0 += 4 * kRedWarps) {
            float4 v[4];
            float b[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = i0 + k * kRedWarps;
                v[k] = i < nparts ? reinterpret_cast<const float4 *>(p.ws_dw)[(int64_t)i * p.C_ch + c] : make_float4(0.f, 0.f, 0.f, 0.f);
                b[k] = i < nparts ? p.ws_db[(int64_t)i * p.C_ch + c] : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                acc.x += v[k].x; acc.y += v[k].y; acc.z += v[k].z; acc.w += v[k].w;
                ab += b[k];
            }
        }
    }
    sw[sl][cl] = acc;
    sb[sl][cl] = ab;
    __syncthreads();
    if (sl == 0 && c < p.C_ch) {
        for (int k = 1; k < kRedWarps; ++k) {
            const float4 v = sw[k][cl];
            acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
            ab += sb[k][cl];
        }
        reinterpret_cast<float4 *>(p.dw)[c] = acc;
        if (p.dbias) p.dbias[c] = ab;
    }
}

}  // namespace

int launch_packed_conv(const PackedConvParams &p, int dtype, cudaStream_t st)
{
    if (p.plan.m64 == 0) return 0;
    return dtype == 1 ? launch_conv_t<__nv_bfloat16>(p, st) : launch_conv_t<float>(p, st);
}

int launch_packed_conv_backward(const PackedConvBwdParams &p, int dtype, cudaStream_t st)
{
    const int64_t n = p.plan.m64 * (p.C_ch / 4);
    const int64_t blocks = (n + kConvBwdT - 1) / kConvBwdT;
    if (blocks > 0x7fffffffLL) return 2;
    prof_begin(st, kKPackedConvBwd);
    if (blocks > 0) {
        if (dtype == 1) packed_conv_bwd_kernel<__nv_bfloat16><<<(unsigned)blocks, kConvBwdT, 0, st>>>(p);
        else packed_conv_bwd_kernel<float><<<(unsigned)blocks, kConvBwdT, 0, st>>>(p);
    }
    packed_conv_reduce_kernel<<<(unsigned)((p.C_ch + 31) / 32), 32 * kRedWarps, 0, st>>>(p);
    prof_end(st, kKPackedConvBwd);
    return cudaGetLastError() == cudaSuccess ? 0 : 7;
}

}  // namespace ssd

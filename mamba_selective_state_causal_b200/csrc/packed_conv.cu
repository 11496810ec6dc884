// packed_conv.cu -- the layer's causal convolution (kernel 4) and SiLU over sequences laid end to end,
// forward and backward:
//   z[t,c] = bias_c + sum_k w[c,k] u[t-3+k,c],   v = z sigma(z),
// where the rows before a sequence's first come from the 3-row buffer of its slot (zeros when it
// does not resume), never from the sequence that lies before it in the tensor.
//
// Forward.  A thread owns one 16-byte vector of channels over kTok consecutive rows of a 64-row
// chunk; its rows are loaded kAhead at a time into registers before any is used, which keeps 128 to
// 256 KB of loads in flight per SM.  Every row is read once, plus three rows of halo per thread, and
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

constexpr int kPackedConvThreads = 128;
constexpr int kAhead = 8;

template <typename T, int kTok>
__global__ void __launch_bounds__(kPackedConvThreads) packed_conv_kernel(PackedConvParams p)
{
    using IO = ConvVec<T>;
    constexpr int V = IO::kN;
    const int ncv = p.C_ch / V;
    const int64_t gid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int c0 = (int)(gid % ncv) * V;
    const int64_t part = gid / ncv;
    const int64_t chunk = part / (64 / kTok);
    const int r0 = (int)(part % (64 / kTok)) * kTok;
    if (chunk >= packed_n64(p.plan, p.status)) return;
    const int4 d = p.plan.chunk64[chunk];
    const int n = min(kTok, (d.y & kChunkRows) - r0);
    const bool head = (d.y & kChunkFirst) && r0 == 0;       // the first rows of a sequence (there may be none)
    if (n <= 0 && !head) return;
    const T *u = reinterpret_cast<const T *>(p.u) + c0;
    const bool kept = d.w >= 0;
    const int64_t tail = kept ? (int64_t)d.w * 3 * p.C_ch + c0 : 0;
    const T *tin = (p.tail_in && kept && (d.y & kChunkResume)) ? reinterpret_cast<const T *>(p.tail_in) + tail : nullptr;
    const int64_t t0 = (int64_t)d.x + r0;
    Vec16p m[3];                                            // rows t0 - 3 .. t0 - 1
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        if (!head) m[k] = ld_rows(u + (t0 - 3 + k) * p.urs);
        else if (tin) m[k] = *reinterpret_cast<const Vec16p *>(tin + k * p.C_ch);
        else m[k] = Vec16p{{0u, 0u, 0u, 0u}};
    }
    if (head && kept && p.tail_out) {
        // the last three rows of the sequence, or of its old buffer and it when it is shorter
        const PackedSeq s = p.plan.seqs[d.z];
        T *to = reinterpret_cast<T *>(p.tail_out) + tail;
        Vec16p o[3];
#pragma unroll
        for (int r = 0; r < 3; ++r) {
            const int pos = s.len - 3 + r;                  // < 0: row 3 + pos of the old buffer
            if (pos >= 0) o[r] = ld_rows(u + ((int64_t)s.row0 + pos) * p.urs);
            else o[r] = pos == -3 ? m[0] : (pos == -2 ? m[1] : m[2]);
        }
#pragma unroll
        for (int r = 0; r < 3; ++r) *reinterpret_cast<Vec16p *>(to + r * p.C_ch) = o[r];
    }
    if (n <= 0) return;
    const T *up = u + t0 * p.urs;
    Vec16p nx[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
        if (j < n) nx[j] = ld_rows(up + j * p.urs);
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
    T *vp = reinterpret_cast<T *>(p.v) + t0 * p.vrs + c0;
    for (int i0 = 0; i0 < n; i0 += kAhead) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (i0 + j < n) {
                float cur[V], out[V];
                IO::unpack(nx[j], cur);
                if (i0 + j + kAhead < n) nx[j] = ld_rows(up + (int64_t)(i0 + j + kAhead) * p.urs);
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
}

template <typename T, int kTok>
int launch_conv_tok(const PackedConvParams &p, cudaStream_t st)
{
    const int64_t threads = p.plan.m64 * (64 / kTok) * (p.C_ch / ConvVec<T>::kN);
    const int64_t blocks = (threads + kPackedConvThreads - 1) / kPackedConvThreads;
    if (blocks > 0x7fffffffLL) return 2;
    prof_begin(st, kKPackedConv);
    packed_conv_kernel<T, kTok><<<(unsigned)blocks, kPackedConvThreads, 0, st>>>(p);
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
// their dz) instead of handing dz between threads.  kBack rows of u (8 bytes) and dv (16 bytes) are
// in registers before they are used.  dw and dbias are summed over the thread's rows in fp32, written
// per chunk, and added over the chunks in a fixed order by a second kernel.
constexpr int kBack = 8;
constexpr int kConvBwdT = 128;

__device__ __forceinline__ float4 ld4(const float *q) { return __ldg(reinterpret_cast<const float4 *>(q)); }
__device__ __forceinline__ float4 ld4(const __nv_bfloat16 *q)
{
    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(q));
    return make_float4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y));
}

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
__global__ void __launch_bounds__(kConvBwdT) packed_conv_bwd_kernel(PackedConvBwdParams p)
{
    const int np = p.C_ch >> 2;
    const int64_t gid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int c = 4 * (int)(gid % np);
    const int64_t chunk = gid / np;
    if (chunk >= packed_n64(p.plan, p.status)) return;
    const int4 d = p.plan.chunk64[chunk];
    const PackedSeq s = p.plan.seqs[d.z];
    const bool head = (d.y & kChunkFirst) != 0;
    const int64_t t0 = d.x, t1 = t0 + (d.y & kChunkRows), se = (int64_t)s.row0 + s.len;
    const T *u = reinterpret_cast<const T *>(p.u) + c;
    // dv of 4 channels, all in one of x, B and C
    const float *dv;
    int64_t dvs;
    if (c < p.HP) { dv = p.dx + c; dvs = p.HP; }
    else if (c < p.HP + p.GN) { dv = p.dB + (c - p.HP); dvs = p.GN; }
    else { dv = p.dC + (c - p.HP - p.GN); dvs = p.GN; }
    const bool resumed = p.tail_in && s.slot >= 0 && s.resume;
    const T *tin = resumed ? reinterpret_cast<const T *>(p.tail_in) + (int64_t)s.slot * 3 * p.C_ch + c : nullptr;
    const float4 z4 = make_float4(0.f, 0.f, 0.f, 0.f);
    float4 a3, a2, a1;                      // u[t-3], u[t-2], u[t-1]
    if (!head) { a3 = ld4(u + (t0 - 3) * p.urs); a2 = ld4(u + (t0 - 2) * p.urs); a1 = ld4(u + (t0 - 1) * p.urs); }
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
    float f0[4] = {}, f1[4] = {}, f2[4] = {};       // dz of the sequence's first three rows, for its buffer
    const int n = (int)(t1 - t0);
    const int nt = n > 0 ? n + 3 : 0;
    const int nin = (int)min((int64_t)nt, se - t0);  // rows past the sequence's end have dz = 0
    for (int b0 = 0; b0 < nt; b0 += kBack) {
        float4 uu[kBack], dd[kBack];
#pragma unroll
        for (int j = 0; j < kBack; ++j) {
            const bool in = b0 + j < nin;
            uu[j] = in ? ld4(u + (t0 + b0 + j) * p.urs) : z4;
            dd[j] = in ? ld4(dv + (t0 + b0 + j) * dvs) : z4;
        }
#pragma unroll
        for (int j = 0; j < kBack; ++j) {
            const int r = b0 + j;
            if (r < nt) {
                const float x3[4] = {a3.x, a3.y, a3.z, a3.w}, x2[4] = {a2.x, a2.y, a2.z, a2.w};
                const float x1[4] = {a1.x, a1.y, a1.z, a1.w}, x0[4] = {uu[j].x, uu[j].y, uu[j].z, uu[j].w};
                const float dvv[4] = {dd[j].x, dd[j].y, dd[j].z, dd[j].w};
                float e0[4], g[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    e0[i] = r < nin ? dz1(dvv[i], wk[0][i], wk[1][i], wk[2][i], wk[3][i], bs[i], x3[i], x2[i], x1[i], x0[i]) : 0.0f;
                    g[i] = fmaf(wk[0][i], e0[i], fmaf(wk[1][i], e1[i], fmaf(wk[2][i], e2[i], wk[3][i] * e3[i])));
                    if (r < n) {
                        gb[i] += e0[i];
                        gw[0][i] = fmaf(e0[i], x3[i], gw[0][i]);
                        gw[1][i] = fmaf(e0[i], x2[i], gw[1][i]);
                        gw[2][i] = fmaf(e0[i], x1[i], gw[2][i]);
                        gw[3][i] = fmaf(e0[i], x0[i], gw[3][i]);
                    }
                    if (r == 0) f0[i] = e0[i];
                    if (r == 1) f1[i] = e0[i];
                    if (r == 2) f2[i] = e0[i];
                    e3[i] = e2[i]; e2[i] = e1[i]; e1[i] = e0[i];
                }
                if (r >= 3) {
                    const int64_t t = t0 + r - 3;
                    if (p.dtail_out && t >= se - 3) {
                        const float4 q = ld4(p.dtail_out + ((int64_t)d.z * 3 + (t - (se - 3))) * p.C_ch + c);
                        g[0] += q.x; g[1] += q.y; g[2] += q.z; g[3] += q.w;
                    }
                    *reinterpret_cast<float4 *>(p.du + t * p.C_ch + c) = make_float4(g[0], g[1], g[2], g[3]);
                }
                a3 = a2; a2 = a1; a1 = uu[j];
            }
        }
    }
    float4 *pw = reinterpret_cast<float4 *>(p.ws_dw) + chunk * p.C_ch + c;
#pragma unroll
    for (int i = 0; i < 4; ++i) pw[i] = make_float4(gw[0][i], gw[1][i], gw[2][i], gw[3][i]);
    *reinterpret_cast<float4 *>(p.ws_db + chunk * p.C_ch + c) = make_float4(gb[0], gb[1], gb[2], gb[3]);
    if (head && p.dtail_in) {
        float g[3][4] = {};
        if (resumed) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                g[0][i] = wk[0][i] * f0[i];
                g[1][i] = fmaf(wk[1][i], f0[i], wk[0][i] * f1[i]);
                g[2][i] = fmaf(wk[2][i], f0[i], fmaf(wk[1][i], f1[i], wk[0][i] * f2[i]));
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
    }
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
    return dtype == 1 ? launch_conv_tok<__nv_bfloat16, 64>(p, st) : launch_conv_tok<float, 64>(p, st);
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

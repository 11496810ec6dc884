// packed_conv.cu -- the layer's causal convolution (kernel 4) and SiLU over sequences laid end to end,
// forward and backward:
//   z[t,c] = bias_c + sum_k w[c,k] u[t-3+k,c],   v = z sigma(z),
// where the rows before a sequence's first come from the 3-row buffer of its slot (zeros when it
// does not resume), never from the sequence that lies before it in the tensor.
//
// Forward.  A thread owns one 16-byte vector of channels over the rows of a 64-row chunk; they stream
// through its own kRing slots of shared memory by cp.async, which keeps 128 KB of loads in flight per SM
// without holding registers.  Every row is read once, plus three rows of halo per thread, and
// written once: the bound is the memory's rate (65536 rows of 2304 channels: 106 to 111 us on different
// machines, 0.83 to 0.87 of the copy rate; in fp32 0.81).
// The arithmetic and its order are the layer's
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
    // weights and bias halved (exact): the sum is h = z / 2 and z sigma(z) = h + h tanh(h), with one hardware
    // tanh (relative error up to 2^-11).  What that costs v is absolute, up to 2^-11 |h|: less than the rounding to
    // bf16 (half a step, 2^-9 to 2^-8 of v) for positive z, more than it where h and h tanh(h) cancel (at z = -4 up to
    // 1.3 % of v, at z = -6, where v is -0.015, up to 10 %).  The layer's convolution has this form too, and a packed
    // sequence gets its bits; the gradients and the slot step take the accurate sigma.
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
__global__ void __launch_bounds__(kPackedConvThreads, 2) packed_conv_kernel(PackedConvParams p, int pieces)
{
    using IO = ConvVec<T>;
    constexpr int V = IO::kN;
    extern __shared__ Vec16p ring[];                        // [kRing][threads]
    const int ncv = p.C_ch / V;
    const int64_t gid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int c0 = (int)(gid % ncv) * V;
    const int64_t chunk = gid / ncv / pieces;
    const int r0 = (int)(gid / ncv % pieces) * (64 / pieces);
    int4 d;
    if (!packed_chunk64(p.plan, chunk, p.status, d)) return;
    const int n = min((d.y & kChunkRows) - r0, 64 / pieces);
    if (r0 > 0 && n <= 0) return;
    const bool head = (d.y & kChunkFirst) != 0 && r0 == 0;
    const T *u = reinterpret_cast<const T *>(p.u) + c0;
    const int64_t t0 = d.x + r0;
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
int launch_conv_t(const PackedConvParams &p, int sms, cudaStream_t st)
{
    // a chunk's rows in up to 8 pieces, while there are fewer CTAs than the SMs hold: what a small batch costs is one
    // thread's rows, one after the other (169 rows of 288 channels in fp32: 25 us in one piece, 9 in eight, the time of the call)
    const int64_t threads = p.plan.m64 * (p.C_ch / ConvVec<T>::kN);
    int pieces = 1;
    while (pieces < 8 && 2 * pieces * threads <= 2 * (int64_t)sms * kPackedConvThreads) pieces *= 2;
    const int64_t blocks = (pieces * threads + kPackedConvThreads - 1) / kPackedConvThreads;
    if (blocks > 0x7fffffffLL) return 2;
    constexpr int smem = kRing * kPackedConvThreads * (int)sizeof(Vec16p);
    static SmemLimit done;
    if (!allow_smem(packed_conv_kernel<T>, smem, done)) return 7;
    prof_begin(st, kKPackedConv);
    packed_conv_kernel<T><<<(unsigned)blocks, kPackedConvThreads, smem, st>>>(p, pieces);
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
// their dz) instead of handing dz between threads.  Its rows of u and dv stream through its own kBack
// slots of shared memory by cp.async (72 KB in flight per SM, no registers held).  dw and dbias are summed
// over the thread's rows in fp32, written per chunk, and added over the chunks in a fixed order by a second
// kernel.  16384 rows of 4352 channels: 140 to 154 us on different machines, 0.71 to 0.78 of the copy rate (8192 rows in
// fp32: 0.72).  By its counters neither the memory (67 %) nor the issue slots (62 %) are full: an SM holds 11 warps of
// 144 registers, which wait for their rows and for the sigma of one row after the other.
constexpr int kBack = 8;
constexpr int kConvBwdT = 128;

__device__ __forceinline__ float4 ld4(const float *q) { return __ldg(reinterpret_cast<const float4 *>(q)); }
__device__ __forceinline__ float4 ld4(const __nv_bfloat16 *q)
{
    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(q));
    return make_float4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y));
}
// 4 elements of u in shared memory
template <typename T> struct Raw4;
template <> struct Raw4<float> {
    float4 v;
    __device__ __forceinline__ float4 get() const { return v; }
};
template <> struct Raw4<__nv_bfloat16> {
    uint2 v;
    __device__ __forceinline__ float4 get() const { return make_float4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)); }
};
template <int kBytes>
__device__ __forceinline__ void cp_small(void *dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "n"(kBytes)
                 : "memory");
}

// two channels at a time (packed fp32 instructions: the arithmetic is what bounds this kernel)
struct F2x2 {
    float2 a, b;
};
__device__ __forceinline__ F2x2 pairs(float4 v) { return F2x2{make_float2(v.x, v.y), make_float2(v.z, v.w)}; }

// dz = dv sg (1 + z (1 - sg)), sg = sigma(z), z from the window x3 .. x0
__device__ __forceinline__ float2 dz2(float2 dv, const float2 (&w)[4], float2 b, float2 x3, float2 x2, float2 x1, float2 x0)
{
    float2 z = __ffma2_rn(w[0], x3, b);
    z = __ffma2_rn(w[1], x2, z);
    z = __ffma2_rn(w[2], x1, z);
    z = __ffma2_rn(w[3], x0, z);
    const float2 sg = make_float2(sigma_fast(z.x), sigma_fast(z.y));
    const float2 f = __ffma2_rn(z, make_float2(1.0f - sg.x, 1.0f - sg.y), make_float2(1.0f, 1.0f));
    return __fmul2_rn(dv, __fmul2_rn(sg, f));
}

template <typename T>
__global__ void __launch_bounds__(kConvBwdT, 3) packed_conv_bwd_kernel(PackedConvBwdParams p)
{
    extern __shared__ __align__(16) uint8_t cbr[];
    float4 *rd = reinterpret_cast<float4 *>(cbr) + threadIdx.x;                                  // [kBack][threads] dv
    Raw4<T> *ru = reinterpret_cast<Raw4<T> *>(cbr + sizeof(float4) * kBack * kConvBwdT) + threadIdx.x;   // [kBack][threads] u
    const int np = p.C_ch >> 2;
    const int64_t gid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int c = 4 * (int)(gid % np);
    const int64_t chunk = gid / np;
    int4 d;
    if (!packed_chunk64(p.plan, chunk, p.status, d)) return;
    const PackedSeq s = p.plan.seqs[d.z];
    const bool head = (d.y & kChunkFirst) != 0;
    const int64_t t0 = d.x;
    const int n = d.y & kChunkRows;
    const int left = (int)((int64_t)s.row0 + s.len - t0);   // rows to the sequence's end
    const int nin = n > 0 ? min(n + 3, left) : 0;           // rows past the sequence's end have dz = 0
    const T *u = reinterpret_cast<const T *>(p.u) + c + t0 * p.urs;
    // dv of 4 channels, all in one of x, B and C
    const float *dv;
    int64_t dvs;
    if (c < p.HP) { dv = p.dx + c; dvs = p.HP; }
    else if (c < p.HP + p.GN) { dv = p.dB + (c - p.HP); dvs = p.GN; }
    else { dv = p.dC + (c - p.HP - p.GN); dvs = p.GN; }
    dv += t0 * dvs;
    // row r of u and dv (in order: the pointers step along) into slot r % kBack; one commit group per row
    const T *uf = u;
    const float *df = dv;
    auto fetch = [&](int r, int sl) {
        if (r < nin) {
            cp_row(rd + sl * kConvBwdT, df);
            cp_small<(int)sizeof(Raw4<T>)>(ru + sl * kConvBwdT, uf);
            df += dvs;
            uf += p.urs;
        }
        cp_commit();
    };
#pragma unroll
    for (int j = 0; j < kBack; ++j) fetch(j, j);
    const bool resumed = p.tail_in && s.slot >= 0 && s.resume;
    const T *tin = resumed ? reinterpret_cast<const T *>(p.tail_in) + (int64_t)s.slot * 3 * p.C_ch + c : nullptr;
    const float4 z4 = make_float4(0.f, 0.f, 0.f, 0.f);
    const float2 z2 = make_float2(0.f, 0.f);
    F2x2 x3, x2, x1;                        // u[t-3], u[t-2], u[t-1]
    if (!head) { x3 = pairs(ld4(u - 3 * p.urs)); x2 = pairs(ld4(u - 2 * p.urs)); x1 = pairs(ld4(u - p.urs)); }
    else if (tin) { x3 = pairs(ld4(tin)); x2 = pairs(ld4(tin + p.C_ch)); x1 = pairs(ld4(tin + 2 * p.C_ch)); }
    else { x3 = x2 = x1 = F2x2{z2, z2}; }
    float2 wa[4], wb[4];                    // taps of the two channel pairs
    {
        const float4 q0 = __ldg(reinterpret_cast<const float4 *>(p.w) + c), q1 = __ldg(reinterpret_cast<const float4 *>(p.w) + c + 1);
        const float4 q2 = __ldg(reinterpret_cast<const float4 *>(p.w) + c + 2), q3 = __ldg(reinterpret_cast<const float4 *>(p.w) + c + 3);
        wa[0] = make_float2(q0.x, q1.x); wa[1] = make_float2(q0.y, q1.y); wa[2] = make_float2(q0.z, q1.z); wa[3] = make_float2(q0.w, q1.w);
        wb[0] = make_float2(q2.x, q3.x); wb[1] = make_float2(q2.y, q3.y); wb[2] = make_float2(q2.z, q3.z); wb[3] = make_float2(q2.w, q3.w);
    }
    F2x2 bs{z2, z2};
    if (p.bias) bs = pairs(make_float4(__ldg(p.bias + c), __ldg(p.bias + c + 1), __ldg(p.bias + c + 2), __ldg(p.bias + c + 3)));
    float2 gwa[4] = {}, gwb[4] = {}, gba = z2, gbb = z2;
    F2x2 e3{z2, z2}, e2{z2, z2}, e1{z2, z2};    // dz[t-3], dz[t-2], dz[t-1] (zero before t0: those rows' du is another thread's)
    float *du = p.du + t0 * p.C_ch + c;
    const int handed = p.dtail_out ? left : 0x7fffffff;   // du's row r - 3 also feeds row r - left of the buffer handed on, r >= left
    const float *dto = p.dtail_out ? p.dtail_out + (int64_t)d.z * 3 * p.C_ch + c : nullptr;
    // the gradient of the buffer that the sequence starts from, with dz of its first three rows in e3, e2, e1
    auto put_tail = [&]() {
        F2x2 g[3] = {{z2, z2}, {z2, z2}, {z2, z2}};
        if (resumed) {
            g[0] = F2x2{__fmul2_rn(wa[0], e3.a), __fmul2_rn(wb[0], e3.b)};
            g[1] = F2x2{__ffma2_rn(wa[1], e3.a, __fmul2_rn(wa[0], e2.a)), __ffma2_rn(wb[1], e3.b, __fmul2_rn(wb[0], e2.b))};
            g[2] = F2x2{__ffma2_rn(wa[2], e3.a, __ffma2_rn(wa[1], e2.a, __fmul2_rn(wa[0], e1.a))),
                        __ffma2_rn(wb[2], e3.b, __ffma2_rn(wb[1], e2.b, __fmul2_rn(wb[0], e1.b)))};
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                const int r = q - s.len;            // row of the new buffer that holds old row q, where the sequence is so short
                if (dto && r >= 0) {
                    const F2x2 x = pairs(ld4(dto + (int64_t)r * p.C_ch));
                    g[q].a = __fadd2_rn(g[q].a, x.a);
                    g[q].b = __fadd2_rn(g[q].b, x.b);
                }
            }
        }
#pragma unroll
        for (int q = 0; q < 3; ++q)
            *reinterpret_cast<float4 *>(p.dtail_in + ((int64_t)d.z * 3 + q) * p.C_ch + c) =
                make_float4(g[q].a.x, g[q].a.y, g[q].b.x, g[q].b.y);
    };
    // du of row r - 3, once dz of row r (e0) is known
    auto put_du = [&](int r, const F2x2 &e0) {
        F2x2 g{__ffma2_rn(wa[0], e0.a, __ffma2_rn(wa[1], e1.a, __ffma2_rn(wa[2], e2.a, __fmul2_rn(wa[3], e3.a)))),
               __ffma2_rn(wb[0], e0.b, __ffma2_rn(wb[1], e1.b, __ffma2_rn(wb[2], e2.b, __fmul2_rn(wb[3], e3.b))))};
        if (r >= handed) {
            const F2x2 x = pairs(ld4(dto + (int64_t)(r - left) * p.C_ch));
            g.a = __fadd2_rn(g.a, x.a);
            g.b = __fadd2_rn(g.b, x.b);
        }
        __stcs(reinterpret_cast<float4 *>(du), make_float4(g.a.x, g.a.y, g.b.x, g.b.y));
        du += p.C_ch;
    };
    if (n == 0 && head && p.dtail_in) put_tail();
#pragma unroll 1
    for (int b0 = 0; b0 < n; b0 += 4) {             // four rows bring the windows back to the same registers
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = b0 + j, sl = (b0 & (kBack - 1)) + j;
            if (r < n) {
                cp_wait<kBack - 1>();               // row r's group is the oldest
                const F2x2 x0 = pairs(ru[sl * kConvBwdT].get()), dd = pairs(rd[sl * kConvBwdT]);
                fetch(r + kBack, sl);
                const F2x2 e0{dz2(dd.a, wa, bs.a, x3.a, x2.a, x1.a, x0.a), dz2(dd.b, wb, bs.b, x3.b, x2.b, x1.b, x0.b)};
                gba = __fadd2_rn(gba, e0.a);
                gbb = __fadd2_rn(gbb, e0.b);
                gwa[0] = __ffma2_rn(e0.a, x3.a, gwa[0]); gwb[0] = __ffma2_rn(e0.b, x3.b, gwb[0]);
                gwa[1] = __ffma2_rn(e0.a, x2.a, gwa[1]); gwb[1] = __ffma2_rn(e0.b, x2.b, gwb[1]);
                gwa[2] = __ffma2_rn(e0.a, x1.a, gwa[2]); gwb[2] = __ffma2_rn(e0.b, x1.b, gwb[2]);
                gwa[3] = __ffma2_rn(e0.a, x0.a, gwa[3]); gwb[3] = __ffma2_rn(e0.b, x0.b, gwb[3]);
                if (r >= 3) put_du(r, e0);
                e3 = e2; e2 = e1; e1 = e0;
                x3 = x2; x2 = x1; x1 = x0;
                if (r == 2 && head && p.dtail_in) put_tail();
            }
        }
    }
    // three rows past the chunk: their dz completes du of its last rows
    if (n > 0) {
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            const int r = n + j;
            F2x2 e0{z2, z2};
            cp_wait<kBack - 1>();
            if (r < nin) {
                const int sl = r & (kBack - 1);
                const F2x2 x0 = pairs(ru[sl * kConvBwdT].get()), dd = pairs(rd[sl * kConvBwdT]);
                e0 = F2x2{dz2(dd.a, wa, bs.a, x3.a, x2.a, x1.a, x0.a), dz2(dd.b, wb, bs.b, x3.b, x2.b, x1.b, x0.b)};
                x3 = x2; x2 = x1; x1 = x0;
            }
            cp_commit();
            if (r >= 3) put_du(r, e0);
            e3 = e2; e2 = e1; e1 = e0;
            if (r == 2 && head && p.dtail_in) put_tail();
        }
    }
    cp_wait<0>();
    float4 *pw = reinterpret_cast<float4 *>(p.ws_dw) + chunk * p.C_ch + c;
    pw[0] = make_float4(gwa[0].x, gwa[1].x, gwa[2].x, gwa[3].x);
    pw[1] = make_float4(gwa[0].y, gwa[1].y, gwa[2].y, gwa[3].y);
    pw[2] = make_float4(gwb[0].x, gwb[1].x, gwb[2].x, gwb[3].x);
    pw[3] = make_float4(gwb[0].y, gwb[1].y, gwb[2].y, gwb[3].y);
    *reinterpret_cast<float4 *>(p.ws_db + chunk * p.C_ch + c) = make_float4(gba.x, gba.y, gbb.x, gbb.y);
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
    if (p.dtail_in && c < p.C_ch && packed_ok(p.plan, p.status)) {
        // sequences without chunks start from no buffer
        for (int q = sl; q < p.plan.nseq; q += kRedWarps)
            if (p.plan.seqs[q].n64 == 0)
                for (int r = 0; r < 3; ++r) p.dtail_in[((int64_t)q * 3 + r) * p.C_ch + c] = 0.0f;
    }
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

int launch_packed_conv(const PackedConvParams &p, int dtype, int sms, cudaStream_t st)
{
    if (p.plan.m64 == 0) return 0;
    return dtype == 1 ? launch_conv_t<__nv_bfloat16>(p, sms, st) : launch_conv_t<float>(p, sms, st);
}

int launch_packed_conv_backward(const PackedConvBwdParams &p, int dtype, cudaStream_t st)
{
    const int64_t n = p.plan.m64 * (p.C_ch / 4);
    const int64_t blocks = (n + kConvBwdT - 1) / kConvBwdT;
    if (blocks > 0x7fffffffLL) return 2;
    prof_begin(st, kKPackedConvBwd);
    if (blocks > 0) {
        static SmemLimit done_b, done_f;
        const int smem_b = (16 + 8) * kBack * kConvBwdT, smem_f = (16 + 16) * kBack * kConvBwdT;
        if (!(dtype == 1 ? allow_smem(packed_conv_bwd_kernel<__nv_bfloat16>, smem_b, done_b) : allow_smem(packed_conv_bwd_kernel<float>, smem_f, done_f)))
            return 7;
        if (dtype == 1) packed_conv_bwd_kernel<__nv_bfloat16><<<(unsigned)blocks, kConvBwdT, smem_b, st>>>(p);
        else packed_conv_bwd_kernel<float><<<(unsigned)blocks, kConvBwdT, smem_f, st>>>(p);
    }
    packed_conv_reduce_kernel<<<(unsigned)((p.C_ch + 31) / 32), 32 * kRedWarps, 0, st>>>(p);
    prof_end(st, kKPackedConvBwd);
    return cudaGetLastError() == cudaSuccess ? 0 : 7;
}

}  // namespace ssd

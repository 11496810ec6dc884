// decode_slots.cu -- one token of b streams whose states and conv buffers live in a pool of slots
// (continuous batching: the batch's streams are any slots in any order, padded with empty rows):
//   v = silu(bias + w0 tail[0] + w1 tail[1] + w2 tail[2] + w3 u),   tail' = [tail[1], tail[2], u]
//   h' = exp(dt A) h + dt x B^T,   y = C h' + D x           per head, x, B, C = v
// The bytes are the states': 2 P N 4 per stream and head, read and written once; the rest is small.
// A cluster of up to 8 CTAs serves one stream, each CTA a run of heads.  A CTA starts its first
// states into shared memory (one bulk copy of P N floats each, kStages in flight) before it forms
// the conv of its heads' x and their groups' B and C from the old buffer; then it updates state after
// state in place in shared memory and sends each back with one bulk copy.  The cluster is what lets
// the new conv buffer be written in the same launch, over the old one: B's and C's channels are read
// by all CTAs of the stream, and the barrier that every CTA arrives at after reading them (and waits
// for only before it writes) comes long after.  v is not rounded to the I/O type here: it stays in
// registers and shared memory, where the layer's packed convolution stores it.
#include <cooperative_groups.h>

#include "packed.cuh"
#include "slots.cuh"
#include "tc_ptx.cuh"

namespace ssd {
namespace {

using namespace tc;

constexpr int kSlotThreads = 256;
constexpr int kStages = 2;

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void bulk_store(void *dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;"
                 ::"l"(dst), "r"(smem_u32(src)), "r"(bytes) : "memory");
}

template <typename T>
__global__ void __launch_bounds__(kSlotThreads) decode_slots_kernel(SlotDecodeParams p)
{
    extern __shared__ __align__(128) uint8_t raw[];
    __shared__ uint64_t full[kStages];
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    const int ncta = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int bi = blockIdx.x / ncta, tid = threadIdx.x;
    const int P = p.P, N = p.N, PN = P * N;
    const int h0 = rank * p.heads_per_cta, h1 = min(p.H, h0 + p.heads_per_cta);
    const int din = p.H * P, C_ch = din + 2 * p.G * N;
    const uint32_t bytes = (uint32_t)PN * 4u;

    float *state = reinterpret_cast<float *>(raw);               // [kStages][P N]
    float *xs = state + kStages * PN;                             // [heads_per_cta][P]
    float *bc = xs + p.heads_per_cta * P;                         // [groups][2 N]

    // a slot out of range, or one that an earlier row of the batch has, leaves the row empty
    const int slot = p.slots[bi];
    bool twice = false;
    if (slot >= 0)
        for (int j = tid; j < bi; j += kSlotThreads) twice |= p.slots[j] == slot;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
    }
    const bool refused = __syncthreads_or(twice ? 1 : 0) != 0 || slot < -1 || slot >= p.n_slots;
    if (refused && tid == 0 && rank == 0) atomicOr(p.status, kDevIndex);
    T *y = reinterpret_cast<T *>(p.y) + (int64_t)bi * p.ybs;
    if (slot < 0 || refused) {                                    // the same for every CTA of the cluster
        for (int i = h0 * P + tid; i < h1 * P; i += kSlotThreads) y[i] = from_f32<T>(0.0f);
        return;
    }
    const float *hin = p.h_in + (int64_t)slot * p.H * PN;
    float *hout = p.h_out + (int64_t)slot * p.H * PN;
    if (tid == 0)
        for (int i = 0; i < kStages && h0 + i < h1; ++i) {
            mbar_arrive_expect_tx(&full[i], bytes);
            bulk_load(state + i * PN, hin + (int64_t)(h0 + i) * PN, bytes, &full[i]);
        }

    // conv + SiLU of the heads' x, then of B and C of the groups they use
    const T *u = reinterpret_cast<const T *>(p.u) + (int64_t)bi * p.ubs;
    const T *tin = reinterpret_cast<const T *>(p.tail_in) + (int64_t)slot * 3 * C_ch;
    T *tout = reinterpret_cast<T *>(p.tail_out) + (int64_t)slot * 3 * C_ch;
    auto conv = [&](int c, T &r1, T &r2, T &r3) {
        const float4 w = __ldg(reinterpret_cast<const float4 *>(p.w) + c);
        const T r0 = tin[c];
        r1 = tin[C_ch + c]; r2 = tin[2 * C_ch + c]; r3 = u[c];
        float z = p.bias ? __ldg(p.bias + c) : 0.0f;
        z = fmaf(w.x, to_f32(r0), z);
        z = fmaf(w.y, to_f32(r1), z);
        z = fmaf(w.z, to_f32(r2), z);
        z = fmaf(w.w, to_f32(r3), z);
        return z / (1.0f + expf(-z));
    };
    auto put = [&](int c, T r1, T r2, T r3) { tout[c] = r1; tout[C_ch + c] = r2; tout[2 * C_ch + c] = r3; };
    for (int i = tid; i < (h1 - h0) * P; i += kSlotThreads) {
        T r1, r2, r3;
        const int c = h0 * P + i;                                 // no other CTA reads or writes this channel
        xs[i] = conv(c, r1, r2, r3);
        put(c, r1, r2, r3);
    }
    const int g0 = h0 < h1 ? (int)((int64_t)h0 * p.G / p.H) : 0;
    const int g1 = h0 < h1 ? (int)((int64_t)(h1 - 1) * p.G / p.H) + 1 : 0;
    for (int i = tid; i < (g1 - g0) * 2 * N; i += kSlotThreads) {
        const int g = i / (2 * N), n = i % (2 * N);
        T r1, r2, r3;
        bc[i] = conv(n < N ? din + (g0 + g) * N + n : din + (p.G + g0 + g) * N + n - N, r1, r2, r3);
    }
    // this CTA has read the old buffer's B and C rows; it writes its share of the new ones below.
    // The new rows' values are read before the barrier, since any of them may change after it
    const int bcn = 2 * p.G * N, share = (bcn + ncta - 1) / ncta;
    constexpr int kKeep = 4;                                      // share <= kKeep * kSlotThreads (checked by the launcher)
    T k1[kKeep], k2[kKeep], k3[kKeep];
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
        const int i = tid + k * kSlotThreads, c = din + rank * share + i;
        if (i < share && rank * share + i < bcn) { k1[k] = tin[C_ch + c]; k2[k] = tin[2 * C_ch + c]; k3[k] = u[c]; }
    }
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

    const int warp = tid >> 5, lane = tid & 31;
    const int nq = N >> 2, sub = lane / nq, col = lane % nq, per = 32 / nq;
    int st = 0;
    uint32_t ph = 0;
    for (int h = h0; h < h1; ++h) {
        float *sm = state + st * PN;
        const float dt = dt_effective(p.dt[(int64_t)bi * p.H + h], p.dt_bias, h, p.dt_softplus, p.dt_min, p.dt_max);
        const float a = expf(dt * p.A[h]);
        const float Dh = p.D ? p.D[h] : 0.0f;
        const float *bg = bc + ((int)((int64_t)h * p.G / p.H) - g0) * 2 * N;
        const float4 Bv = reinterpret_cast<const float4 *>(bg)[col], Cv = reinterpret_cast<const float4 *>(bg + N)[col];
        const float *xh = xs + (h - h0) * P;
        const bool landed = mbar_wait(&full[st], ph, nullptr, p.wait_limit_ns);
        for (int r = warp * per + sub; r < P; r += (kSlotThreads / 32) * per) {
            float4 *cell = reinterpret_cast<float4 *>(sm + r * N) + col;
            float4 v = *cell;
            const float dx = dt * xh[r];
            v.x = fmaf(a, v.x, dx * Bv.x);
            v.y = fmaf(a, v.y, dx * Bv.y);
            v.z = fmaf(a, v.z, dx * Bv.z);
            v.w = fmaf(a, v.w, dx * Bv.w);
            *cell = v;
            float part = fmaf(Cv.x, v.x, fmaf(Cv.y, v.y, fmaf(Cv.z, v.z, Cv.w * v.w)));
            for (int o = 1; o < nq; o <<= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
            if (col == 0) y[h * P + r] = from_f32<T>(fmaf(Dh, xh[r], part));
        }
        fence_proxy_async_smem();
        if (!__syncthreads_and(landed)) {
            // a copy never came: nothing more is written, and what is on its way is waited for
            if (tid == 0) {
                atomicOr(p.status, kDevTimeout);
                for (int k = 0; k < kStages && h + k < h1; ++k)
                    mbar_wait(&full[(st + k) % kStages], st + k < kStages ? ph : ph ^ 1, nullptr, 100000000ull);
            }
            break;
        }
        if (tid == 0) {
            bulk_store(hout + (int64_t)h * PN, sm, bytes);
            tma_store_commit();
            if (h + kStages < h1) {
                tma_store_wait_read<0>();                         // the copy out has read this stage
                mbar_arrive_expect_tx(&full[st], bytes);
                bulk_load(sm, hin + (int64_t)(h + kStages) * PN, bytes, &full[st]);
            }
        }
        if (++st == kStages) { st = 0; ph ^= 1; }
    }
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
        const int i = tid + k * kSlotThreads, c = din + rank * share + i;
        if (i < share && rank * share + i < bcn) put(c, k1[k], k2[k], k3[k]);
    }
    if (tid == 0) tma_store_wait<0>();
}

template <typename T>
int launch_slots_t(const SlotDecodeParams &p, int cluster, size_t smem, cudaStream_t st)
{
    if (cudaFuncSetAttribute(decode_slots_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return 7;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)p.b * (unsigned)cluster);
    cfg.blockDim = dim3(kSlotThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)cluster;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    prof_begin(st, kKSlotDecode);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, decode_slots_kernel<T>, p);
    prof_end(st, kKSlotDecode);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? 0 : 7;
}

}  // namespace

int launch_slot_decode(SlotDecodeParams p, int dtype, cudaStream_t st)
{
    int cluster = 8;
    while (cluster > 1 && cluster > p.H) cluster /= 2;
    p.heads_per_cta = (p.H + cluster - 1) / cluster;
    // groups that a run of heads can touch
    const int hpg = p.H / p.G;
    const int groups = p.heads_per_cta / hpg + 2 < p.G ? p.heads_per_cta / hpg + 2 : p.G;
    const size_t smem = sizeof(float) * ((size_t)kStages * p.P * p.N + (size_t)p.heads_per_cta * p.P + (size_t)groups * 2 * p.N);
    if (smem > 220 * 1024) return 6;
    if ((2 * p.G * p.N + cluster - 1) / cluster > 4 * kSlotThreads) return 6;
    if ((int64_t)p.b * cluster > 0x7fffffffLL) return 6;
    return dtype == 1 ? launch_slots_t<__nv_bfloat16>(p, cluster, smem, st) : launch_slots_t<float>(p, cluster, smem, st);
}

}  // namespace ssd

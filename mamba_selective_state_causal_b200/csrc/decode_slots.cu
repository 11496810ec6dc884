// decode_slots.cu -- one token of b streams whose states and conv buffers live in a pool of slots
// (continuous batching: the batch's streams are any slots in any order, padded with empty rows):
//   v = silu(bias + w0 tail[0] + w1 tail[1] + w2 tail[2] + w3 u),   tail' = [tail[1], tail[2], u]
//   h' = exp(dt A) h + dt x B^T,   y = C h' + D x           per head, x, B, C = v
// The bytes are the states': 2 P N 4 per stream and head, read and written once; the rest is small.
// A cluster of up to 8 (few streams: 16) CTAs serves one stream, each CTA a run of heads.  A CTA starts its first
// states into shared memory (one bulk copy of P N floats each, kStages in flight) before it forms
// the conv of its heads' x and their groups' B and C from the old buffer; then it updates state after
// state in place in shared memory and sends each back with one bulk copy.  The cluster is what lets
// the new conv buffer be written in the same launch, over the old one: B's and C's channels are read
// by all CTAs of the stream, and the barrier that every CTA arrives at after reading them (and waits
// for only before it writes) comes long after.  A state moves in two halves of P / 2 rows (16 KB at P = 64,
// N = 128), three in flight per CTA and four CTAs per SM (all of them, up to 16, where the batch is so small
// that a CTA has its SM to itself); a buffer is refilled one piece after its copy out was started, so that nobody waits for that
// copy to have read it.  v is not rounded to the I/O type here: it stays in registers and shared memory, where
// the layer's packed convolution stores it.  256 streams of 32 heads (P = 64, N = 128): 100 to 102 us, 0.8 of the copy
// rate; two streams: the launch.
#include <algorithm>

#include <cooperative_groups.h>

#include "packed.cuh"
#include "slots.cuh"
#include "tc_ptx.cuh"

namespace ssd {
namespace {

using namespace tc;

constexpr int kSlotThreads = 256;
constexpr int kMaxStages = 16;

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

constexpr int kKeep = 4;             // turns of a CTA over its share of B's and C's channels that it keeps in registers

// nq = N / 4: lanes of a state row.  kLate: a share is longer than that.  (With the loop for the rest in every kernel 256
// streams of one group took 105 us instead of 101: at four CTAs per SM there is no register to spare.)
template <typename T, int nq, bool kLate>
__global__ void __launch_bounds__(kSlotThreads) decode_slots_kernel(SlotDecodeParams p)
{
    extern __shared__ __align__(128) uint8_t raw[];
    __shared__ uint64_t full[kMaxStages];
    const int kStages = p.stages;
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    const int ncta = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int bi = blockIdx.x / ncta, tid = threadIdx.x;
    const int P = p.P, PN = P * 4 * nq;
    constexpr int N = 4 * nq;
    const int R = P / 2, piece = R * N;                           // a state goes in two pieces of R rows
    const int h0 = rank * p.heads_per_cta, h1 = min(p.H, h0 + p.heads_per_cta);
    const int din = p.H * P, C_ch = din + 2 * p.G * N;
    const uint32_t bytes = (uint32_t)piece * 4u;
    const int np = 2 * (h1 - h0);                                 // pieces of this CTA's heads, one after the other

    float *state = reinterpret_cast<float *>(raw);               // [kStages][R N]
    float *xs = state + kStages * piece;                           // [heads_per_cta][P]
    float *hv = xs + p.heads_per_cta * P;                         // [heads_per_cta][4]: e^{dt A}, dt, D
    float *bc = hv + p.heads_per_cta * 4;                         // [groups][2 N]

    T *y = reinterpret_cast<T *>(p.y) + (int64_t)bi * p.ybs;
    const int slot = p.slots[bi];
    const bool inside = slot >= 0 && slot < p.n_slots;            // the same for every CTA of the cluster
    if (!inside) {
        if (slot != -1 && tid == 0 && rank == 0) atomicOr(p.status, kDevIndex);
        for (int i = h0 * P + tid; i < h1 * P; i += kSlotThreads) y[i] = from_f32<T>(0.0f);
        return;
    }
    const float *hin = p.h_in + ((int64_t)slot * p.H + h0) * PN;
    float *hout = p.h_out + ((int64_t)slot * p.H + h0) * PN;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
        for (int i = 0; i < kStages && i < np && (int64_t)blockIdx.x != p.test_drop_unit; ++i) {
            mbar_arrive_expect_tx(&full[i], bytes);
            bulk_load(state + i * piece, hin + (int64_t)i * piece, bytes, &full[i]);
        }
    }

    // conv + SiLU of the heads' x, then of B and C of the groups they use; two channels per thread and turn,
    // all of their loads in flight together
    const T *u = reinterpret_cast<const T *>(p.u) + (int64_t)bi * p.ubs;
    const T *tin = reinterpret_cast<const T *>(p.tail_in) + (int64_t)slot * 3 * C_ch;
    T *tout = reinterpret_cast<T *>(p.tail_out) + (int64_t)slot * 3 * C_ch;
    const int g0 = h0 < h1 ? (int)((int64_t)h0 * p.G / p.H) : 0;
    const int g1 = h0 < h1 ? (int)((int64_t)(h1 - 1) * p.G / p.H) + 1 : 0;
    const int nx = h0 < h1 ? (h1 - h0) * P : 0, nch = nx + (g1 - g0) * 2 * N;
    auto channel = [&](int i) {
        if (i < nx) return h0 * P + i;
        const int g = (i - nx) / (2 * N), n = (i - nx) % (2 * N);
        return n < N ? din + (g0 + g) * N + n : din + (p.G + g0 + g) * N + n - N;
    };
    bool twice = false;                                           // an earlier row of the batch has this slot
    for (int j = tid; j < bi; j += kSlotThreads) twice |= p.slots[j] == slot;
    for (int i0 = tid; i0 < nch; i0 += 2 * kSlotThreads) {
        T r[2][4];
        float4 w[2];
        float b[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int i = i0 + k * kSlotThreads;
            if (i < nch) {
                const int c = channel(i);
                r[k][0] = tin[c]; r[k][1] = tin[C_ch + c]; r[k][2] = tin[2 * C_ch + c]; r[k][3] = u[c];
                w[k] = __ldg(reinterpret_cast<const float4 *>(p.w) + c);
                b[k] = p.bias ? __ldg(p.bias + c) : 0.0f;
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int i = i0 + k * kSlotThreads;
            if (i < nch) {
                float z = b[k];
                z = fmaf(w[k].x, to_f32(r[k][0]), z);
                z = fmaf(w[k].y, to_f32(r[k][1]), z);
                z = fmaf(w[k].z, to_f32(r[k][2]), z);
                z = fmaf(w[k].w, to_f32(r[k][3]), z);
                (i < nx ? xs[i] : bc[i - nx]) = z / (1.0f + expf(-z));
            }
        }
    }
    for (int i = tid; i < h1 - h0; i += kSlotThreads) {
        const int h = h0 + i;
        const float dt = dt_effective(p.dt[(int64_t)bi * p.H + h], p.dt_bias, h, p.dt_softplus, p.dt_min, p.dt_max);
        reinterpret_cast<float4 *>(hv)[i] = make_float4(expf(dt * p.A[h]), dt, p.D ? p.D[h] : 0.0f, 0.0f);
    }
    // this CTA has read the old buffer's B and C rows; it writes its share of the new ones at the end.
    // The values of the first kKeep turns are read here, ahead of their use; those of more (kLate, many groups) at the end:
    // after the barrier no other CTA reads or writes them
    const int bcn = 2 * p.G * N, share = (bcn + ncta - 1) / ncta;
    T k1[kKeep], k2[kKeep], k3[kKeep];
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
        const int i = tid + k * kSlotThreads, c = din + rank * share + i;
        if (i < share && rank * share + i < bcn) { k1[k] = tin[C_ch + c]; k2[k] = tin[2 * C_ch + c]; k3[k] = u[c]; }
    }
    if (__syncthreads_or(twice ? 1 : 0)) {                        // the same for every CTA of the cluster
        if (tid == 0) {
            if (rank == 0) atomicOr(p.status, kDevIndex);
            for (int i = 0; i < kStages && i < np; ++i) mbar_wait(&full[i], 0, nullptr, p.wait_limit_ns);
        }
        for (int i = h0 * P + tid; i < h1 * P; i += kSlotThreads) y[i] = from_f32<T>(0.0f);
        return;
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

    const int warp = tid >> 5, lane = tid & 31;
    constexpr int per = 32 / nq, kRows = 4, kStep = (kSlotThreads / 32) * per;   // rows a warp, a thread, a turn of the CTA takes
    const int sub = lane / nq, col = lane % nq;
    const bool up = (lane & (nq / 2)) != 0, up2 = (lane & (nq / 4)) != 0;
    for (int k = 0; k < np; ++k) {
        const int st = k % kStages, h = h0 + (k >> 1), r0 = (k & 1) * R;
        float *sm = state + st * piece;
        const float4 he = reinterpret_cast<const float4 *>(hv)[h - h0];
        const float a = he.x, dt = he.y, Dh = he.z;
        const float *bg = bc + ((int)((int64_t)h * p.G / p.H) - g0) * 2 * N;
        const float4 Bv = reinterpret_cast<const float4 *>(bg)[col], Cv = reinterpret_cast<const float4 *>(bg + N)[col];
        const float *xh = xs + (h - h0) * P + r0;
        const bool landed = mbar_wait(&full[st], (uint32_t)(k / kStages) & 1, nullptr, p.wait_limit_ns);
        for (int rb = warp * per + sub; rb - sub < R; rb += kRows * kStep) {
            float4 v[kRows];
            float part[kRows];
#pragma unroll
            for (int e = 0; e < kRows; ++e)
                if (rb + e * kStep < R) v[e] = reinterpret_cast<const float4 *>(sm + (rb + e * kStep) * N)[col];
#pragma unroll
            for (int e = 0; e < kRows; ++e) {
                part[e] = 0.0f;
                if (rb + e * kStep < R) {
                    const float dx = dt * xh[rb + e * kStep];
                    v[e].x = fmaf(a, v[e].x, dx * Bv.x);
                    v[e].y = fmaf(a, v[e].y, dx * Bv.y);
                    v[e].z = fmaf(a, v[e].z, dx * Bv.z);
                    v[e].w = fmaf(a, v[e].w, dx * Bv.w);
                    reinterpret_cast<float4 *>(sm + (rb + e * kStep) * N)[col] = v[e];
                    part[e] = fmaf(Cv.x, v[e].x, fmaf(Cv.y, v[e].y, fmaf(Cv.z, v[e].z, Cv.w * v[e].w)));
                }
            }
            // the four rows' sums over their nq lanes in 3 + log2(nq / 4) exchanges: halves of the lanes take two rows
            // each, quarters one
            float k0 = up ? part[2] : part[0], k1 = up ? part[3] : part[1];
            k0 += __shfl_xor_sync(0xffffffffu, up ? part[0] : part[2], nq / 2);
            k1 += __shfl_xor_sync(0xffffffffu, up ? part[1] : part[3], nq / 2);
            float sum = up2 ? k1 : k0;
            sum += __shfl_xor_sync(0xffffffffu, up2 ? k0 : k1, nq / 4);
#pragma unroll
            for (int o = nq / 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const int r = rb + ((up ? 2 : 0) + (up2 ? 1 : 0)) * kStep;
            if ((col & (nq / 4 - 1)) == 0 && r < R) y[h * P + r0 + r] = from_f32<T>(fmaf(Dh, xh[r], sum));
        }
        fence_proxy_async_smem();
        if (!__syncthreads_and(landed)) {
            // a copy never came: this CTA writes no more states and no buffer, and what is on its way is waited for
            if (tid == 0) {
                atomicOr(p.status, kDevTimeout);
                for (int q = k; q < np && q < k + kStages - (k > 0 ? 1 : 0); ++q)
                    mbar_wait(&full[q % kStages], (uint32_t)(q / kStages) & 1, nullptr, 100000000ull);
                tma_store_wait<0>();
            }
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
            return;
        }
        if (tid == 0) {
            bulk_store(hout + (int64_t)k * piece, sm, bytes);
            tma_store_commit();
            if (k >= 1 && k - 1 + kStages < np) {
                const int q = k - 1 + kStages;                    // into the buffer of piece k - 1
                tma_store_wait_read<1>();                         // whose copy out has read it
                mbar_arrive_expect_tx(&full[q % kStages], bytes);
                bulk_load(state + (q % kStages) * piece, hin + (int64_t)q * piece, bytes, &full[q % kStages]);
            }
        }
    }
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
        const int i = tid + k * kSlotThreads, c = din + rank * share + i;
        if (i < share && rank * share + i < bcn) { tout[c] = k1[k]; tout[C_ch + c] = k2[k]; tout[2 * C_ch + c] = k3[k]; }
    }
    if (kLate) {
        for (int i = tid + kKeep * kSlotThreads; i < share && rank * share + i < bcn; i += kSlotThreads) {
            const int c = din + rank * share + i;
            const T a = tin[C_ch + c], b = tin[2 * C_ch + c], n = u[c];
            tout[c] = a; tout[C_ch + c] = b; tout[2 * C_ch + c] = n;
        }
    }
    for (int i = tid; i < nx; i += kSlotThreads) {                // x's channels: no other CTA reads or writes them
        const int c = h0 * P + i;
        const T a = tin[C_ch + c], b = tin[2 * C_ch + c], n = u[c];
        tout[c] = a; tout[C_ch + c] = b; tout[2 * C_ch + c] = n;
    }
    if (tid == 0) tma_store_wait<0>();
}

constexpr int kNotWide = -1;
constexpr int kRoom = 200 * 1024;         // shared memory of a CTA, at most

template <typename T, int nq, bool kLate>
int launch_slots_n(const SlotDecodeParams &p, int cluster, size_t smem, cudaStream_t st)
{
    static SmemLimit done;
    if (!allow_smem(decode_slots_kernel<T, nq, kLate>, cluster > 8 ? kRoom : (int)smem, done)) return 7;
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
    if (cluster > 8) {
        // asked once per device: how many such clusters run at a time, each CTA with an SM to itself (plus 1; more
        // streams than that would wait for others to end)
        static std::atomic<int> wide[64];
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 7;
        int w = wide[dev].load(std::memory_order_relaxed);
        if (w == 0) {
            int active = 0;
            cudaLaunchConfig_t most = cfg;
            most.dynamicSmemBytes = kRoom;
            if (cudaFuncSetAttribute(decode_slots_kernel<T, nq, kLate>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
                cudaOccupancyMaxActiveClusters(&active, decode_slots_kernel<T, nq, kLate>, &most) != cudaSuccess) {
                active = 0;
                cudaGetLastError();
            }
            w = active + 1;
            wide[dev].store(w, std::memory_order_relaxed);
        }
        if (p.b > w - 1) return kNotWide;
    }
    prof_begin(st, kKSlotDecode);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, decode_slots_kernel<T, nq, kLate>, p);
    prof_end(st, kKSlotDecode);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? 0 : 7;
}

template <typename T, int nq>
int launch_slots_q(const SlotDecodeParams &p, int cluster, size_t smem, cudaStream_t st)
{
    const bool late = (2 * p.G * p.N + cluster - 1) / cluster > kKeep * kSlotThreads;
    return late ? launch_slots_n<T, nq, true>(p, cluster, smem, st) : launch_slots_n<T, nq, false>(p, cluster, smem, st);
}

template <typename T>
int launch_slots_t(const SlotDecodeParams &p, int cluster, size_t smem, cudaStream_t st)
{
    switch (p.N) {
    case 16: return launch_slots_q<T, 4>(p, cluster, smem, st);
    case 32: return launch_slots_q<T, 8>(p, cluster, smem, st);
    case 64: return launch_slots_q<T, 16>(p, cluster, smem, st);
    default: return launch_slots_q<T, 32>(p, cluster, smem, st);
    }
}

}  // namespace

static int launch_slots(SlotDecodeParams p, int cluster, int dtype, int sms, cudaStream_t st)
{
    while (cluster > 1 && cluster > p.H) cluster /= 2;
    p.heads_per_cta = (p.H + cluster - 1) / cluster;
    // groups that a run of heads can touch
    const int hpg = p.H / p.G;
    const int groups = p.heads_per_cta / hpg + 2 < p.G ? p.heads_per_cta / hpg + 2 : p.G;
    const size_t small = sizeof(float) * ((size_t)p.heads_per_cta * (p.P + 4) + (size_t)groups * 2 * p.N);
    const size_t piece = sizeof(float) * (size_t)(p.P / 2) * p.N;
    const size_t room = kRoom;
    if (small + 3 * piece > room) return 6;
    const int np = 2 * p.heads_per_cta;
    p.stages = p.b * cluster <= sms ? (int)std::min<size_t>(std::min(np, kMaxStages), (room - small) / piece) : std::min(np, 3);
    const size_t smem = p.stages * piece + small;
    if ((int64_t)p.b * cluster > 0x7fffffffLL) return 6;
    return dtype == 1 ? launch_slots_t<__nv_bfloat16>(p, cluster, smem, st) : launch_slots_t<float>(p, cluster, smem, st);
}

int launch_slot_decode(const SlotDecodeParams &p, int dtype, int sms, cudaStream_t st)
{
    // 16 CTAs to a stream while the device runs so many clusters of 16 at a time: a CTA takes its heads one after the
    // other (64 heads, 5 streams: 23 us with 8 CTAs each, 12 with 16; 32 heads, 2 streams: 12 and 8)
    const int rc = 16 * (int64_t)p.b <= sms && p.H >= 16 ? launch_slots(p, 16, dtype, sms, st) : kNotWide;
    return rc == kNotWide ? launch_slots(p, 8, dtype, sms, st) : rc;
}

}  // namespace ssd

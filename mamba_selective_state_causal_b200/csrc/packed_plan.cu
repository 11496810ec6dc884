// packed_plan.cu -- the plan of a packed batch (packed.cuh), made on the device: two launches per
// batch, none per layer, no copy to the host, so that it can be captured and replayed with other
// offsets in the same buffers.
//
// The first kernel (one CTA) checks each sequence's offsets and slot and gives it its first chunk by
// a running sum over the sequences, 1024 at a time.  A slot that two sequences name goes to the
// first of them: the sequences are entered into a hash table over the slots in shared memory, each
// entry keeping the lowest sequence, and a sequence that does not find itself there loses its slot.
// The second kernel writes the chunks, each found by a binary search over the sequences' first chunks.
// Both are latency, once per batch: 4 us for one sequence, 6 for 24, 9 for 256, 32 for 4096 and 108 for 16384 (slots
// named; in a captured graph, a call of its own takes 10 to 14 of the host at least).
#include <algorithm>

#include "packed.cuh"

namespace ssd {
namespace {

constexpr int kPlanThreads = 1024;

__device__ __forceinline__ int hash_slot(int s, int mask) { return (int)(((unsigned)s * 2654435761u) >> 7) & mask; }

// inclusive sum over the CTA's 1024 threads, two values at once
__device__ __forceinline__ int2 block_sum(int2 v, int2 *part)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, v.x, o), b = __shfl_up_sync(0xffffffffu, v.y, o);
        if (lane >= o) { v.x += a; v.y += b; }
    }
    __syncthreads();                       // the previous tile's sums have been read
    if (lane == 31) part[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int2 t = part[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int a = __shfl_up_sync(0xffffffffu, t.x, o), b = __shfl_up_sync(0xffffffffu, t.y, o);
            if (lane >= o) { t.x += a; t.y += b; }
        }
        part[lane] = t;
    }
    __syncthreads();
    if (warp > 0) { v.x += part[warp - 1].x; v.y += part[warp - 1].y; }
    return v;
}

// inclusive maximum over the CTA's 1024 threads
__device__ __forceinline__ int block_max(int v, int *part)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v = max(v, a);
    }
    __syncthreads();
    if (lane == 31) part[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int t = part[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int a = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t = max(t, a);
        }
        part[lane] = t;
    }
    __syncthreads();
    if (warp > 0) v = max(v, part[warp - 1]);
    return v;
}

__global__ void __launch_bounds__(kPlanThreads) packed_seq_kernel(PackedPlanParams p, PackedSeq *seqs, int hash_size)
{
    extern __shared__ int table[];         // [hash_size] lowest sequence + 1 of a slot, 0 = free
    __shared__ int2 part[32];
    __shared__ int most[32];
    __shared__ int live;                   // rows of the sequences so far
    const int tid = threadIdx.x, mask = hash_size - 1;
    bool bad = false;
    if (tid == 0) live = 0;                // (a barrier of block_max lies before the first addition)
    if (p.slots) {
        for (int i = tid; i < hash_size; i += kPlanThreads) table[i] = 0;
        __syncthreads();
        for (int i = tid; i < p.nseq; i += kPlanThreads) {
            const int s = p.slots[i];
            if (s < 0 || s >= p.n_slots) continue;
            // at most half full, so that every search ends
            for (int e = hash_slot(s, mask), n = 0; n < hash_size; ++n, e = (e + 1) & mask) {
                const int old = atomicCAS(&table[e], 0, i + 1);
                if (old == 0) break;
                if (p.slots[old - 1] == s) { atomicMin(&table[e], i + 1); break; }
            }
        }
        __syncthreads();
    }
    int2 base = make_int2(0, 0);
    int behind = 0;                        // the highest offset of the tiles before
    for (int t = 0; t < p.nseq; t += kPlanThreads) {
        const int i = t + tid;
        // a sequence may not begin before the highest offset so far: sequences never share rows,
        // and the chunks of all of them fit the plan
        const int at = i < p.nseq ? p.cu[i] : -1;
        const int high = max(behind, block_max(at <= p.total ? at : -1, most));
        PackedSeq s{};
        int2 c = make_int2(0, 0);
        if (i < p.nseq) {
            const int a = at, b = p.cu[i + 1];
            const bool fits = a >= 0 && a >= high && b >= a && b <= p.total && (int64_t)b - a <= p.max_seqlen;
            bad |= !fits;
            s.row0 = fits ? a : 0;
            s.len = fits ? b - a : 0;
            s.slot = p.slots ? p.slots[i] : i;
            if (s.slot < -1 || s.slot >= p.n_slots) { bad = true; s.slot = -1; }
            if (p.slots && s.slot >= 0) {
                int found = 0;
                for (int e = hash_slot(s.slot, mask), n = 0; n < hash_size; ++n, e = (e + 1) & mask) {
                    found = table[e];
                    if (found == 0 || p.slots[found - 1] == s.slot) break;
                }
                if (found != i + 1) { bad = true; s.slot = -1; }
            }
            s.resume = p.resume ? (p.resume[i] != 0) : 1;
            if (s.slot < 0) s.resume = 0;
            if (fits && (s.len > 0 || s.slot >= 0)) {       // (nothing to do for one of no rows that is kept nowhere)
                s.n64 = max(1, (s.len + 63) / 64);
                s.n128 = max(1, (s.len + 127) / 128);
            }
            c = make_int2(s.n64, s.n128);
        }
        const int rows = __reduce_add_sync(0xffffffffu, s.len);
        if ((tid & 31) == 0 && rows > 0) atomicAdd(&live, rows);
        const int2 sum = block_sum(c, part);
        if (i < p.nseq) {
            s.c64 = base.x + sum.x - c.x;
            s.c128 = base.y + sum.y - c.y;
            seqs[i] = s;
        }
        base.x += part[31].x;
        base.y += part[31].y;
        behind = max(behind, most[31]);
    }
    if (bad) atomicOr(p.status, kDevIndex);
    if (tid == 0) {
        PackedHeader h{};
        h.magic = kPackedMagic; h.nseq = p.nseq; h.total = p.total; h.max_len = p.max_seqlen;
        h.n64 = base.x; h.n128 = base.y;
        h.rows = live;
        *static_cast<PackedHeader *>(p.plan) = h;
    }
}

// chunk k of Q rows: its sequence is the last one whose first chunk is at or before k (a sequence
// without chunks shares its first with the next, so it is never the last one)
template <int Q>
__device__ __forceinline__ void write_chunk(const PackedPlan &p, int k, int n, int4 *out)
{
    if (k >= n) return;
    int lo = 0, hi = p.nseq - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        const int first = Q == 64 ? p.seqs[mid].c64 : p.seqs[mid].c128;
        if (first <= k) lo = mid; else hi = mid - 1;
    }
    const PackedSeq s = p.seqs[lo];
    const int j = k - (Q == 64 ? s.c64 : s.c128);
    const int rows = max(0, min(Q, s.len - j * Q));
    const int count = Q == 64 ? s.n64 : s.n128;
    out[k] = make_int4(s.row0 + j * Q,
                       rows | (j == 0 ? kChunkFirst : 0) | (j == count - 1 ? kChunkLast : 0) | (s.resume ? kChunkResume : 0),
                       lo, s.slot);
}

__global__ void __launch_bounds__(256) packed_chunk_kernel(PackedPlan p, int4 *c64, int4 *c128)
{
    const int k = blockIdx.x * blockDim.x + threadIdx.x;
    write_chunk<64>(p, k, p.hdr->n64, c64);
    write_chunk<128>(p, k, p.hdr->n128, c128);
}

}  // namespace

int launch_packed_plan(const PackedPlanParams &p, cudaStream_t st)
{
    const PackedLayout l = packed_layout(p.nseq, p.total);
    char *b = static_cast<char *>(p.plan);
    int hash = 64;
    if (p.slots) while (hash < 2 * p.nseq) hash *= 2;
    const int smem = p.slots ? hash * (int)sizeof(int) : 0;
    static SmemLimit done;
    if (!allow_smem(packed_seq_kernel, 2 * kPackedMaxSlotted * (int)sizeof(int), done)) return 7;
    prof_begin(st, kKPackedPlan);
    packed_seq_kernel<<<1, kPlanThreads, smem, st>>>(p, reinterpret_cast<PackedSeq *>(b + l.off_seq), hash);
    if (l.m64 > 0)
        packed_chunk_kernel<<<(unsigned)((l.m64 + 255) / 256), 256, 0, st>>>(
            packed_view(p.plan, p.nseq, p.total), reinterpret_cast<int4 *>(b + l.off64),
            reinterpret_cast<int4 *>(b + l.off128));
    prof_end(st, kKPackedPlan);
    return cudaGetLastError() == cudaSuccess ? 0 : 7;
}

}  // namespace ssd

// packed.cuh -- sequences laid end to end in the rows of one tensor: the plan that the packed
// kernels walk, as it lies in device memory, and their parameters.
//
// A plan is made on the device from the sequences' offsets (packed_plan.cu) and serves every call
// and layer that works on the same batch: a header, one PackedSeq per sequence, and the
// sequences cut into chunks of 64 and of 128 rows.  A chunk never crosses a sequence, its rows are
// consecutive, and the chunks of a sequence follow one another, so that a kernel which takes
// chunks in order takes the sequences one after the other.  An empty sequence with a slot has one chunk
// of no rows (its state still moves from h_in to h_out); one without (a batch padded to a number of
// sequences) has none, nor has one whose offsets are refused.
#pragma once

#include "smem.cuh"
#include "ssd_common.cuh"

namespace ssd {

constexpr int kPackedMagic = 0x50414b31;

struct PackedHeader {
    int magic, nseq;
    int64_t total;
    int64_t max_len;        // no sequence is longer
    int n64, n128;          // chunks in use of each length
    int rows;               // rows of the sequences
    int pad[7];
};
static_assert(sizeof(PackedHeader) == 64, "packed header");

struct PackedSeq {
    int row0, len;          // first row, number of rows
    int slot;               // where its state and conv buffer live, or -1 (not kept)
    int resume;             // start from the slot's state (else from zero)
    int c64, c128;          // its first chunk of each length
    int n64, n128;          // its number of chunks
};
static_assert(sizeof(PackedSeq) == 32, "packed sequence");

// A chunk: x = first row, y = rows (0..128) | flags, z = sequence, w = slot or -1
constexpr int kChunkRows = 0xff, kChunkFirst = 1 << 8, kChunkLast = 1 << 9, kChunkResume = 1 << 10;

// Byte offsets of a plan's parts for nseq sequences in `total` rows.  A sequence of len rows has at
// most len / Q + 1 chunks of Q rows, hence at most total / Q + nseq of them in all.
struct PackedLayout {
    int64_t m64, m128;      // room for chunks
    size_t off_seq, off64, off128, bytes;
};

inline PackedLayout packed_layout(int64_t nseq, int64_t total)
{
    PackedLayout l;
    l.m64 = total / 64 + nseq;
    l.m128 = total / 128 + nseq;
    l.off_seq = sizeof(PackedHeader);
    l.off64 = l.off_seq + sizeof(PackedSeq) * (size_t)nseq;
    l.off128 = l.off64 + 16 * (size_t)l.m64;
    l.bytes = (l.off128 + 16 * (size_t)l.m128 + 255) & ~size_t(255);
    return l;
}

// A plan as a kernel receives it.
struct PackedPlan {
    const PackedHeader *hdr;
    const PackedSeq *seqs;
    const int4 *chunk64, *chunk128;
    int nseq;
    int64_t total;
    int64_t m64, m128;
    int64_t max_len;        // the bound that the call's launches were chosen by, or -1 (none)
};

inline PackedPlan packed_view(const void *plan, int nseq, int64_t total, int64_t max_len = -1)
{
    const PackedLayout l = packed_layout(nseq, total);
    const char *b = static_cast<const char *>(plan);
    return PackedPlan{reinterpret_cast<const PackedHeader *>(b), reinterpret_cast<const PackedSeq *>(b + l.off_seq),
                      reinterpret_cast<const int4 *>(b + l.off64), reinterpret_cast<const int4 *>(b + l.off128),
                      nseq, total, l.m64, l.m128, max_len};
}

// The number of 64- or 128-row chunks in use; 0 (and the status latched) when the plan in memory
// is not the one that the call was given sizes for, so that no row outside the tensors is touched.
__device__ __forceinline__ bool packed_ok(const PackedPlan &p, unsigned int *status)
{
    if (p.hdr->magic == kPackedMagic && p.hdr->nseq == p.nseq && p.hdr->total == p.total &&
        (p.max_len < 0 || p.hdr->max_len <= p.max_len))
        return true;
    if (threadIdx.x == 0) atomicOr(status, kDevIndex);
    return false;
}
__device__ __forceinline__ int packed_n64(const PackedPlan &p, unsigned int *status)
{
    return packed_ok(p, status) ? p.hdr->n64 : 0;
}
__device__ __forceinline__ int packed_n128(const PackedPlan &p, unsigned int *status)
{
    return packed_ok(p, status) ? p.hdr->n128 : 0;
}

// Descriptor of 64-row chunk k (k < m64), false past the chunks in use; the header's load and the
// descriptor's are in flight together
__device__ __forceinline__ bool packed_chunk64(const PackedPlan &p, int64_t k, unsigned int *status, int4 &d)
{
    if (k >= p.m64) return false;
    d = __ldg(p.chunk64 + k);
    return k < packed_n64(p, status);
}

struct PackedPlanParams {
    int nseq;
    int64_t total, max_seqlen;
    const int *cu, *slots, *resume;
    int n_slots;
    void *plan;
    unsigned int *status;
};

struct PackedConvParams {
    PackedPlan plan;
    const void *u;
    int64_t urs;
    const float *w, *bias;
    const void *tail_in;        // [slots][3][C_ch] or NULL
    void *tail_out;             // [slots][3][C_ch] or NULL
    void *v;
    int64_t vrs;
    int C_ch;
    unsigned int *status;
};

struct PackedConvBwdParams {
    PackedPlan plan;
    const void *u;
    int64_t urs;
    const float *w, *bias;
    const void *tail_in;
    const float *dx, *dB, *dC;  // [total][HP], [total][GN], [total][GN]
    int HP, GN, C_ch;
    const float *dtail_out;     // [nseq][3][C_ch] or NULL
    float *du, *dtail_in;       // [total][C_ch], [nseq][3][C_ch] or NULL
    float *ws_dw, *ws_db;       // [m64][C_ch][4], [m64][C_ch]
    float *dw, *dbias;
    unsigned int *status;
};

// The packed scan.  The chunks of all sequences are split into nw windows of consecutive chunks
// (per_window = ceil(chunks / nw), on the device); one CTA walks a window.
struct PackedScanParams {
    PackedPlan plan;
    int H, P, N, G;
    const void *x, *B, *C;
    int64_t xrs, Brs, Crs;
    const float *dt, *A, *D;
    const float *dt_bias;
    int dt_softplus;
    float dt_min, dt_max;
    const float *h_in;          // [slots][H][P][N] or NULL
    float *h_out;               // [slots][H][P][N] or NULL
    void *y;
    int64_t yrs;
    int nw;                     // windows
    float *ws_S;                // [nw][H][P][N] what the chunks before a window's end leave of its last sequence
    float *ws_hin;              // [nw][H][P][N] state entering the window, from the chain; NULL: few windows, each
                                // forms it for itself (window_enter)
    float *ws_start;            // [nw][H][P][N] state that a sequence which begins in the window and leaves it
                                // starts from, when it resumes: its slot may be written (h_out may be h_in) by
                                // the window where it ends before the one where it begins reads it
    float *ws_dA;               // [nw][H] sum of dt*A over those chunks
    unsigned int *status;
    uint64_t wait_limit_ns;
    int64_t test_drop_unit;
};

// The tensor-core gradient of the packed scan (packed_grad_tc.cu)
struct PackedGradParams {
    PackedPlan plan;
    int H, G;
    const void *x, *B, *C, *dy;
    int64_t xrs, Brs, Crs, dyrs;
    const float *dt, *A, *D;
    const float *h_in;          // [slots][H][P][N] or NULL
    const float *dh_out;        // [nseq][H][P][N] or NULL
    float *dx, *dB, *dC, *ddt, *dA, *dD, *dh_in;
    uint8_t *ws_img;            // [m64][H][2] h entering the chunk and Gam arriving at its last row, as operands
    float *ws_part;             // [blocks of heads][dB, dC][64][N]
    float *ws_sums;             // [CTAs][2] partial sums of an item
    float *ws_pA, *ws_pD;       // [H][m64]
    unsigned int *status;
    uint64_t wait_limit_ns;
    int64_t test_drop_unit;
};
struct PackedGradLayout {
    size_t off_part, off_sums, off_pA, off_pD, bytes;
};

// Whether window k hands a sequence on to window k + 1, and from which chunk of window k that
// sequence's state is built: c0 = first chunk (of the sequence, or of the window when the sequence
// began before it), c1 = end of the window.
struct WindowTail {
    bool crosses, begins;       // begins: the sequence's first chunk lies in the window
    int c0, c1, seq;
};

template <bool k64>
__device__ __forceinline__ WindowTail window_tail(const PackedPlan &p, int n, int per, int k)
{
    const int4 *tab = k64 ? p.chunk64 : p.chunk128;
    WindowTail t{};
    const int64_t a = (int64_t)k * per, b = a + per;
    if (b >= n) return t;       // the last window in use ends with the last sequence
    const int4 last = tab[b - 1];
    if (last.y & kChunkLast) return t;
    t.crosses = true;
    t.seq = last.z;
    const int sc = k64 ? p.seqs[last.z].c64 : p.seqs[last.z].c128;
    t.begins = sc >= a;
    t.c0 = t.begins ? sc : (int)a;
    t.c1 = (int)b;
    return t;
}

// The state that the chunk d, the first of its sequence, starts from in a window that ends at chunk
// c1: its slot's, the copy of it when the sequence leaves the window, or NULL (zero); of head h.
template <bool k64>
__device__ __forceinline__ const float *window_start(const PackedScanParams &p, int4 d, int window, int64_t c1, int h)
{
    if (!p.h_in || !(d.y & kChunkResume)) return nullptr;
    const int64_t PN = (int64_t)p.P * p.N;
    if (!(d.y & kChunkLast)) {
        const PackedSeq s = p.plan.seqs[d.z];
        if ((k64 ? s.c64 + s.n64 : s.c128 + s.n128) > c1) return p.ws_start + ((int64_t)window * p.H + h) * PN;
    }
    return p.h_in + ((int64_t)d.w * p.H + h) * PN;
}

// The state entering window k, whose first chunk d continues a sequence that began in window b, is
//   e^{dA_{k-1} + .. + dA_b} start + sum_w e^{dA_{k-1} + .. + dA_{w+1}} S_w,   b <= w < k:
// n elements of it, `stride` apart, from `at` on, of head h (of the chain's result where there is one).
template <bool k64, int n, typename F>
__device__ __forceinline__ void window_enter(const PackedScanParams &p, int4 d, int k, int per, int h, int64_t at, int stride, F put)
{
    const int64_t PN = (int64_t)p.P * p.N;
    if (p.ws_hin) {
        const float *src = p.ws_hin + ((int64_t)k * p.H + h) * PN + at;
#pragma unroll
        for (int e = 0; e < n; ++e) put(e, src[(int64_t)e * stride]);
        return;
    }
    const PackedSeq s = p.plan.seqs[d.z];
    const int b = (k64 ? s.c64 : s.c128) / per;
    float acc[n];
#pragma unroll
    for (int e = 0; e < n; ++e) acc[e] = 0.0f;
    float sum = 0.0f;
#pragma unroll 1
    for (int w = k - 1; w >= b; --w) {
        const float f = expf(sum);
        const float *src = p.ws_S + ((int64_t)w * p.H + h) * PN + at;
#pragma unroll
        for (int e = 0; e < n; ++e) acc[e] = fmaf(f, src[(int64_t)e * stride], acc[e]);
        sum += p.ws_dA[(int64_t)w * p.H + h];
    }
    if (p.h_in && s.resume) {
        const float f = expf(sum);
        const float *src = p.ws_start + ((int64_t)b * p.H + h) * PN + at;
#pragma unroll
        for (int e = 0; e < n; ++e) acc[e] = fmaf(f, src[(int64_t)e * stride], acc[e]);
    }
#pragma unroll
    for (int e = 0; e < n; ++e) put(e, acc[e]);
}

constexpr int kMaxOwnWindows = 16;         // up to so many windows each forms its entering state for itself

int launch_packed_plan(const PackedPlanParams &p, cudaStream_t st);
int launch_packed_conv(const PackedConvParams &p, int dtype, int sms, cudaStream_t st);
int launch_packed_conv_backward(const PackedConvBwdParams &p, int dtype, cudaStream_t st);
bool packed_scan_tc_shape(int dtype, int H, int P, int N, int G);
int launch_packed_scan_tc(const PackedScanParams &p, bool carry, cudaStream_t st);
int launch_packed_scan_generic(const PackedScanParams &p, bool carry, int dtype, cudaStream_t st);
PackedGradLayout packed_grad_layout(int64_t nseq, int64_t total, int H, int ctas);
int launch_packed_grad_tc(const PackedGradParams &p, int ctas, cudaStream_t st);
int launch_packed_chain(const PackedScanParams &p, bool k64, cudaStream_t st);
constexpr int kPackedMaxSlotted = 16384;   // sequences of one plan that names slots

}  // namespace ssd

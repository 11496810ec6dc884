// scan_tc_util.cuh -- what the tensor-core scans share: the 128B-swizzled 128 x 64 bf16 tile, packed
// fp32 arithmetic and bf16 rounding, warp-uniform bounded waits, and the TMA maps of row tensors.
#pragma once

#include <cuda.h>

#include "ssd_common.cuh"
#include "tc_ptx.cuh"

namespace ssd {
namespace tc {

constexpr uint32_t kBox = 128 * 64 * 2;   // one 128-row x 64-col bf16 TMA box (16 KB)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Bounded wait whose outcome is the same for every lane of the warp, so that
// the warp stays converged for the .sync.aligned TMEM instructions after it.
__device__ __forceinline__ bool ewait(uint64_t *bar, uint32_t parity, volatile int *abort, uint64_t limit_ns)
{
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, limit_ns));
}

// The same with the loop out of line, for kernels with many waits: with the loops in place the warps of the packed
// scan's output pass, some thirty waits, waited for instructions (298 against 282 us at 65536 rows of 32 heads).
[[maybe_unused]] static __device__ __noinline__ bool wait_loop(uint64_t *bar, uint32_t parity, volatile int *abort, uint64_t limit_ns)
{
    return mbar_wait(bar, parity, abort, limit_ns);
}
__device__ __forceinline__ bool cwait(uint64_t *bar, uint32_t parity, volatile int *abort, uint64_t limit_ns)
{
    const bool ok = mbar_try_wait(bar, parity) || wait_loop(bar, parity, abort, limit_ns);
    return __all_sync(0xffffffffu, ok);
}

// byte offset of 16-byte chunk c of row r in a 128B-swizzled tile of 128-byte rows
__device__ __forceinline__ uint32_t swz(int r, int c)
{
    return (uint32_t)((r >> 3) * 1024 + (r & 7) * 128 + ((c ^ (r & 7)) << 4));
}

__device__ __forceinline__ uint4 lds128(const uint8_t *p) { return *reinterpret_cast<const uint4 *>(p); }
__device__ __forceinline__ void sts128(uint8_t *p, uint4 v) { *reinterpret_cast<uint4 *>(p) = v; }


// fp32 pair -> bf16x2 by integer rounding (half an ulp added, ties away from zero), on the
// integer pipe so that it runs beside the conversion unit; inputs are finite
__device__ __forceinline__ uint32_t pack_bf16x2_int(float lo, float hi)
{
    return __byte_perm(__float_as_uint(lo) + 0x8000u, __float_as_uint(hi) + 0x8000u, 0x7632);
}

__device__ __forceinline__ uint32_t scale_bf16x2_int(uint32_t v, float w)
{
    return pack_bf16x2_int(bf16_lo(v) * w, bf16_hi(v) * w);
}

// two fp32 products / fused multiply-adds in one instruction (sm_100 packed fp32, through the
// CUDA float2 intrinsics, which leave the register pairing to the compiler); each lane rounds
// exactly as the scalar instruction does
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

__device__ __forceinline__ float2 unpack2(uint32_t v) { return make_float2(bf16_lo(v), bf16_hi(v)); }

// bf16 pair times w, rounded to nearest even (cvt)
__device__ __forceinline__ uint32_t scale_bf16x2_rn(uint32_t v, float2 w2)
{
    const float2 p = mul2(unpack2(v), w2);
    return pack_bf16x2(p.x, p.y);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                                  CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                  CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn()
{
    // looked up once per process (a function-local static is initialised thread-safely)
    static const EncodeTiledFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeTiledFn>(f);
        return (EncodeTiledFn) nullptr;
    }();
    return fn;
}

// [b][L][cols] view with element strides (rs, bs); box = 64 columns x 128 rows
inline bool encode_bf16(EncodeTiledFn enc, CUtensorMap *m, const void *base, int64_t cols, int64_t L, int b,
                 int64_t rs, int64_t bs, uint32_t box_rows = 128)
{
    if (b == 1) bs = rs * L;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)L, (cuuint64_t)b};
    const cuuint64_t strides[2] = {(cuuint64_t)rs * 2, (cuuint64_t)bs * 2};
    const cuuint32_t box[3] = {64, box_rows, 1};
    const cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}


}  // namespace tc
}  // namespace ssd

// moe_ops.cuh -- what the kernels around the expert layer (norms, router, FP4
// linear) share: element types, reductions and the layer's quantisers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include "moe.h"
#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {

using bf16 = __nv_bfloat16;

inline bool valid_dtype(int d) { return d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F32; }
inline size_t dtype_bytes(int d) { return d == MOE_DTYPE_F32 ? 4 : 2; }
inline bool aligned_to(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Every kernel here may be set up while the one before it in the stream still runs, which hides most of the 2 to 3 us
// between two launches: it is launched with launch(), calls launch_next() first of all, and in every thread
// wait_for_previous() -- which waits until all kernels before it are done and their stores visible -- before it reads what
// an earlier kernel may have written or writes anything.  A kernel that does not call launch_next() (anybody else's) is
// waited for as always.
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <class... P, class... A>
cudaError_t launch(void (*kernel)(P...), unsigned grid, int threads, size_t smem, int cluster, cudaStream_t s, const A &...args) {
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(grid);
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    cudaLaunchAttribute a[2];
    a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a[0].val.programmaticStreamSerializationAllowed = 1;
    a[1].id = cudaLaunchAttributeClusterDimension;
    a[1].val.clusterDim.x = cluster;
    a[1].val.clusterDim.y = a[1].val.clusterDim.z = 1;
    c.attrs = a;
    c.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&c, kernel, args...);
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ bf16 from_f32<bf16>(float v) { return __float2bfloat16_rn(v); }

// 16 bytes read once, kept out of L1 (which the parameters of every row stay in).
__device__ __forceinline__ uint4 ld_stream16(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// 16 bytes at a shared address, by an ordinary load that the compiler may move among others.
__device__ __forceinline__ uint4 ld_shared16(uint32_t at) {
    return *reinterpret_cast<const uint4 *>(__cvta_shared_to_generic(at));
}

// Asynchronous copy of `bytes` (16 or 32) to shared memory, past L1.
template <int bytes>
__device__ __forceinline__ void copy_async(uint32_t d, const void *src) {
#pragma unroll
    for (int i = 0; i < bytes; i += 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d + i), "l"(static_cast<const uint8_t *>(src) + i)
                     : "memory");
}

// Eight f32 values as four pairs: one instruction multiplies or adds a pair.
struct F8 {
    float2 p[4];
    __device__ __forceinline__ float get(int j) const { return (j & 1) ? p[j >> 1].y : p[j >> 1].x; }
    __device__ __forceinline__ void put(int j, float v) {   // j known at compile time
        if (j & 1) p[j >> 1].y = v;
        else p[j >> 1].x = v;
    }
    __device__ __forceinline__ void fill(float v) {
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] = make_float2(v, v);
    }
};
__device__ __forceinline__ float2 pair(float v) { return make_float2(v, v); }

// Eight neighbouring elements as they are in memory (16-byte aligned).
template <class S>
struct Raw8;
template <>
struct Raw8<bf16> {
    uint4 r;
    __device__ __forceinline__ void load(const bf16 *p) { r = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void load_once(const bf16 *p) { r = ld_stream16(p); }
    __device__ __forceinline__ void load_shared(uint32_t at) { r = ld_shared16(at); }
    __device__ __forceinline__ void store(bf16 *p) const { *reinterpret_cast<uint4 *>(p) = r; }
    __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(F8 &v) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) v.p[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
    }
    __device__ __forceinline__ void set(const F8 &v) {
        r = make_uint4(bf16x2(v.p[0].x, v.p[0].y), bf16x2(v.p[1].x, v.p[1].y), bf16x2(v.p[2].x, v.p[2].y),
                       bf16x2(v.p[3].x, v.p[3].y));
    }
};
template <>
struct Raw8<float> {
    float f[8];
    __device__ __forceinline__ void load(const float *p) {
        const float4 a = *reinterpret_cast<const float4 *>(p), b = *(reinterpret_cast<const float4 *>(p) + 1);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
    __device__ __forceinline__ void load_once(const float *p) { put(ld_stream16(p), ld_stream16(p + 4)); }
    __device__ __forceinline__ void load_shared(uint32_t at) { put(ld_shared16(at), ld_shared16(at + 16)); }
    __device__ __forceinline__ void put(const uint4 &a, const uint4 &b) {
        f[0] = __uint_as_float(a.x), f[1] = __uint_as_float(a.y), f[2] = __uint_as_float(a.z), f[3] = __uint_as_float(a.w);
        f[4] = __uint_as_float(b.x), f[5] = __uint_as_float(b.y), f[6] = __uint_as_float(b.z), f[7] = __uint_as_float(b.w);
    }
    __device__ __forceinline__ void store(float *p) const {
        *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
        *(reinterpret_cast<float4 *>(p) + 1) = make_float4(f[4], f[5], f[6], f[7]);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = 0.0f;
    }
    __device__ __forceinline__ void get(F8 &v) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) v.p[j] = make_float2(f[2 * j], f[2 * j + 1]);
    }
    __device__ __forceinline__ void set(const F8 &v) {
#pragma unroll
        for (int j = 0; j < 4; ++j) f[2 * j] = v.p[j].x, f[2 * j + 1] = v.p[j].y;
    }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// 2^e, e in [-126, 127].
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// FP8 group scale sf = amax / 448, the rounded quotient, and inv, by which v
// becomes q = v / sf: the rounded 448 / amax (within one more rounding of the
// division: a code differs where v is that near a tie).  The quotient by a
// constant is its product with the rounded reciprocal and one correction by
// the exact remainder (Brisebarre, Muller and Raina 2004; for 448 right for
// every mantissa; with a division 4096 x 7168 takes 45.5 us instead of 44.1).
// Below 2^-100, where the remainder would not stay normal and inv would pass
// the f32 range, v is brought up by 2^64.  An all-zero group has sf 0 and codes
// 0 (by any inv; it stays out of the branch, because the lanes past a row's end
// are such groups: 1 x 1408 f32 3.4 us, with them in it 3.8), one with an
// infinity sf infinity.
struct Fp8Scale {
    float sf, inv;
};
__device__ __forceinline__ Fp8Scale fp8_scale(float amax, F8 &v) {
    const float near = amax * (1.0f / 448.0f);
    const float rest = fminf(fmaf(-448.0f, near, amax), FLT_MAX);   // not a number for an infinity, which it leaves one
    Fp8Scale q{fmaf(rest, 1.0f / 448.0f, near), 448.0f / fmaxf(amax, 0x1p-100f)};
    if (__float_as_uint(amax) - 1u < 0x0D800000u - 1u) {   // 0 < amax < 2^-100
        q.sf = amax / 448.0f;
        q.inv = 448.0f / (amax * 0x1p64f);
#pragma unroll
        for (int j = 0; j < 4; ++j) v.p[j] = __fmul2_rn(v.p[j], pair(0x1p64f));
    }
    return q;
}

// UE8M0 code e + 127 of the smallest power of two 2^e with amax / 448 <= 2^e:
// 448 is 1.75 * 2^8, so with amax = m 2^x, e is x - 8 for m <= 1.75 and x - 7
// above; the addition carries into the exponent exactly for the latter.  At
// least 0 (all-zero groups among them), for infinities 247.
__device__ __forceinline__ int ue8m0_code(float amax) {
    return max(0, (int)((__float_as_uint(amax) + 0x001FFFFFu) >> 23) - 8);
}
// 2^-e of that code.
__device__ __forceinline__ float ue8m0_inverse(int code) { return __uint_as_float((uint32_t)(254 - code) << 23); }

}  // namespace moe

// cache8.cuh -- the paged 8-bit K/V cache: its geometry and argument checks
// (host) and the conversions of its 8-bit values (device).
//
// K and V lie in pages [n_pages, Hkv, page, d] of 8-bit values, head-major so
// that the rows of one head in one page are contiguous (page * d bytes): a
// decode CTA, which reads one head, streams whole lines of DRAM.  The rows of
// a page fall into blocks of `block` tokens; block b of head h has one fp32
// scale, [n_pages, Hkv, page / block], and a byte x stands for x * scale.
#pragma once

#include <cuda_fp16.h>

#include "device.cuh"
#include "internal.h"

namespace gqa {

// Programmatic dependent launch.  These kernels are short and follow one another (fork,
// copy, append, decode), so each is launched while its predecessor still runs and
// waits, before it touches memory, for that kernel to be complete: the launch costs
// then overlap.  Every thread calls dependents_may_launch() and wait_for_stream() first.
__device__ __forceinline__ void dependents_may_launch() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_stream() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <class Kernel, class... Args>
int launch_dependent(Kernel kern, dim3 grid, dim3 threads, size_t smem, cudaStream_t stream,
                     const char *what, const Args &...args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = threads;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return check_cuda(cudaLaunchKernelEx(&cfg, kern, args...), what);
}

struct Cache8 {
    void *k, *v;
    float *k_scale, *v_scale;
    int kind, n_pages, Hkv, page, d, block;
};

constexpr int kC8Rows = 16;          // page and block are multiples of this
constexpr int kC8MaxPage = 1024;
constexpr int kC8MaxBlock = 256;

// Geometry, then (need_ptrs) the pointers; GQA_OK or the error set.
int check_cache8(const Cache8 &c, bool need_ptrs);
// B rows of M page slots; M * page must fit an int.
int check_table(int B, int M, int page);

// The low and high byte pairs of a word of four 8-bit values as two f16 each,
// exactly.  e4m3 has 4 significant bits and exponents -9 .. 8; int8: byte x + 128
// in the low bits of the f16 1024 is 1152 + x.
template <bool kInt8>
__device__ __forceinline__ void to_f16x2(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if constexpr (kInt8) {
        const uint32_t x = w ^ 0x80808080u;
        const uint32_t a = __byte_perm(x, 0x64646464u, 0x4140), b = __byte_perm(x, 0x64646464u, 0x4342);
        const __half2 bias = __float2half2_rn(1152.0f);
        const __half2 l = __hsub2(*reinterpret_cast<const __half2 *>(&a), bias);
        const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&b), bias);
        lo = *reinterpret_cast<const uint32_t *>(&l);
        hi = *reinterpret_cast<const uint32_t *>(&h);
    } else {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi) : "r"(w));
    }
}

// Four 8-bit values -> fp32.
template <bool kInt8>
__device__ __forceinline__ void to_f32x4(uint32_t w, float (&f)[4]) {
    uint32_t a, b;
    to_f16x2<kInt8>(w, a, b);
    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&a));
    const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&b));
    f[0] = x.x;
    f[1] = x.y;
    f[2] = y.x;
    f[3] = y.y;
}

// Four fp32 -> 8-bit values, nearest even.  Beyond the range: the largest value
// of that sign; NaN stays NaN in e4m3 and becomes 0 in int8.
template <bool kInt8>
__device__ __forceinline__ uint32_t from_f32x4(float a, float b, float c, float d) {
    if constexpr (kInt8) {
        const int x = max(-127, min(127, __float2int_rn(a))), y = max(-127, min(127, __float2int_rn(b)));
        const int z = max(-127, min(127, __float2int_rn(c))), w = max(-127, min(127, __float2int_rn(d)));
        return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
    }
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// The same for |values| <= 127 (int8): adding 1.5 * 2^23 rounds to an integer, nearest
// even, and leaves it in the low bits.
template <bool kInt8>
__device__ __forceinline__ uint32_t from_small_f32x4(float a, float b, float c, float d) {
    if constexpr (kInt8) {
        const uint32_t x = __float_as_uint(__fadd_rn(a, 12582912.0f));
        const uint32_t y = __float_as_uint(__fadd_rn(b, 12582912.0f));
        const uint32_t z = __float_as_uint(__fadd_rn(c, 12582912.0f));
        const uint32_t w = __float_as_uint(__fadd_rn(d, 12582912.0f));
        return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
    }
    return from_f32x4<false>(a, b, c, d);
}

}  // namespace gqa

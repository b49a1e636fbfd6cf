// Loads and stores of io values (float32 or bfloat16) as floats, one at a time or 16 bytes at once.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace prism {
namespace io {

__device__ __forceinline__ float ld(const float *p) { return *p; }
__device__ __forceinline__ float ld(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st(float *p, float x) { *p = x; }
__device__ __forceinline__ void st(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// A unit of VEC consecutive io values: 16 bytes (VEC = 16 / sizeof(io_t)) or one value (VEC = 1).
template <typename io_t, int VEC>
struct Unit;
template <>
struct Unit<float, 4> {
    uint4 w;
    __device__ __forceinline__ void get(float (&f)[4]) const
    {
        f[0] = __uint_as_float(w.x), f[1] = __uint_as_float(w.y), f[2] = __uint_as_float(w.z), f[3] = __uint_as_float(w.w);
    }
    __device__ __forceinline__ void set(const float (&f)[4])
    {
        w = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};
template <>
struct Unit<__nv_bfloat16, 8> {
    uint4 w;
    static __device__ __forceinline__ void two(uint32_t x, float &a, float &b)
    {
        a = __uint_as_float(x << 16), b = __uint_as_float(x & 0xffff0000u);
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        two(w.x, f[0], f[1]), two(w.y, f[2], f[3]), two(w.z, f[4], f[5]), two(w.w, f[6], f[7]);
    }
    __device__ __forceinline__ void set(const float (&f)[8])
    {
        w = make_uint4(pack(f[0], f[1]), pack(f[2], f[3]), pack(f[4], f[5]), pack(f[6], f[7]));
    }
};
template <typename io_t>
struct Unit<io_t, 1> {
    io_t w;
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = ld(&w); }
    __device__ __forceinline__ void set(const float (&f)[1]) { st(&w, f[0]); }
};

template <typename io_t, int VEC>
__device__ __forceinline__ Unit<io_t, VEC> load_unit(const io_t *p)
{
    Unit<io_t, VEC> u;
    u.w = *reinterpret_cast<const decltype(u.w) *>(p);
    return u;
}
template <typename io_t, int VEC>
__device__ __forceinline__ void store_unit(io_t *p, const Unit<io_t, VEC> &u)
{
    *reinterpret_cast<decltype(u.w) *>(p) = u.w;
}

// Two fp32 operations in one instruction
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<uint64_t &>(r)) : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<uint64_t &>(r)) : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t &>(r))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)), "l"(reinterpret_cast<uint64_t &>(c)));
    return r;
}
}  // namespace io
}  // namespace prism

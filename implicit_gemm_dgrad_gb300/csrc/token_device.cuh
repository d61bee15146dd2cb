// Shared by the token operators (logprobs_sm103.cu, embed_sm103.cu): 16-byte
// vectors of fp16, bf16 or fp32 elements widened to fp32, token numbers of
// either width, and the argument checks of their C entry points.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/cdg.h"

namespace cdg {

template <typename T>
struct Elem;

template <>
struct Elem<float> {
    static __device__ __forceinline__ float get(float v) { return v; }
    static __device__ __forceinline__ float put(float v) { return v; }
};
template <>
struct Elem<__half> {
    static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<__nv_bfloat16> {
    static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};

// One 32-bit word of a vector: its two 16-bit values (or one fp32 value) widened.
template <typename T>
__device__ __forceinline__ void widen(uint32_t w, float *f);
template <>
__device__ __forceinline__ void widen<float>(uint32_t w, float *f)
{
    f[0] = __uint_as_float(w);
}
template <>
__device__ __forceinline__ void widen<__half>(uint32_t w, float *f)
{
    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    f[0] = v.x;
    f[1] = v.y;
}
template <>
__device__ __forceinline__ void widen<__nv_bfloat16>(uint32_t w, float *f)
{
    f[0] = __uint_as_float(w << 16);
    f[1] = __uint_as_float(w & 0xFFFF0000u);
}

template <typename T>
__device__ __forceinline__ uint32_t narrow(const float *f);
template <>
__device__ __forceinline__ uint32_t narrow<float>(const float *f)
{
    return __float_as_uint(f[0]);
}
template <>
__device__ __forceinline__ uint32_t narrow<__half>(const float *f)
{
    const __half2 v = __floats2half2_rn(f[0], f[1]);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t narrow<__nv_bfloat16>(const float *f)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(f[0], f[1]);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Elements of T in a 32-bit word and in a 16-byte vector.
template <typename T>
constexpr int kPerWord = 4 / static_cast<int>(sizeof(T));
template <typename T>
constexpr int kPerVec = 16 / static_cast<int>(sizeof(T));

template <typename T>
__device__ __forceinline__ void widen_vec(const uint4 &v, float (&f)[kPerVec<T>])
{
    widen<T>(v.x, f);
    widen<T>(v.y, f + kPerWord<T>);
    widen<T>(v.z, f + 2 * kPerWord<T>);
    widen<T>(v.w, f + 3 * kPerWord<T>);
}

template <typename T>
__device__ __forceinline__ uint4 narrow_vec(const float (&f)[kPerVec<T>])
{
    return make_uint4(narrow<T>(f), narrow<T>(f + kPerWord<T>), narrow<T>(f + 2 * kPerWord<T>),
                      narrow<T>(f + 3 * kPerWord<T>));
}

// Token i of an int32 or int64 list, or -1 when it lies outside [0, vocab).
__device__ __forceinline__ int token_at(const void *tokens, int index_bytes, long long i, int vocab)
{
    const long long t = index_bytes == 8 ? __ldg(static_cast<const long long *>(tokens) + i)
                                         : static_cast<long long>(__ldg(static_cast<const int *>(tokens) + i));
    return t >= 0 && t < vocab ? static_cast<int>(t) : -1;
}

// One vector of T read from any element address: the two aligned 16-byte
// blocks that hold it, joined by get().  [lo, hi) is the tensor; blocks that
// reach past it are read element by element, and of those only columns
// [0, cols) of the row, `col` being the vector's first (it may begin before the
// row or end after it; what lies there is any value).
template <typename T>
struct Shifted {
    uint4 a, b;
    uint32_t sh;  // bytes into a
    __device__ __forceinline__ void load(const T *p, const char *lo, const char *hi, int col, int cols)
    {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        sh = static_cast<uint32_t>(at) & 15u;
        const uintptr_t block = at - sh, end = block + (sh ? 32 : 16);
        if (block >= reinterpret_cast<uintptr_t>(lo) && end <= reinterpret_cast<uintptr_t>(hi)) {
            const uint4 *q = reinterpret_cast<const uint4 *>(block);
            a = __ldg(q);
            b = __ldg(q + (sh ? 1 : 0));
        } else {
            float f[kPerVec<T>];
#pragma unroll
            for (int e = 0; e < kPerVec<T>; ++e) f[e] = col + e >= 0 && col + e < cols ? Elem<T>::get(p[e]) : 0.0f;
            a = narrow_vec<T>(f);  // exact: the values are T's
            sh = 0;
        }
    }
    __device__ __forceinline__ uint4 get() const
    {
        uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        if (sh & 8u) {
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
        }
        if (sh & 4u) {
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
        }
        if constexpr (sizeof(T) == 2) {
            const uint32_t bits = (sh & 2u) * 8u;
            return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                              __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// ---------------------------------------------------------------- host side
// A launch that may begin while the one before it ends: its kernel waits
// (grid_dep_wait) before it touches memory.
template <typename... A>
cudaError_t launch_early(void (*kernel)(A...), dim3 grid, dim3 block, int smem, cudaStream_t s, const A &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

static inline int dtype_bytes(int dtype) { return dtype == CDG_F32 ? 4 : 2; }

static inline bool aligned_to(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Byte range of a tensor argument; overlap is tested between two of them.
struct Extent {
    const char *p;
    size_t n;
};
static inline Extent extent(const void *p, size_t n) { return Extent{static_cast<const char *>(p), p ? n : 0}; }
static inline bool overlap(const Extent &a, const Extent &b)
{
    return a.n && b.n && a.p < b.p + b.n && b.p < a.p + a.n;
}
// Bytes from the first to the last element of a rows x cols matrix of row stride ld.
static inline size_t matrix_bytes(long long rows, long long cols, long long ld, int esize)
{
    return rows > 0 ? static_cast<size_t>((rows - 1) * ld + cols) * static_cast<size_t>(esize) : 0;
}

// SM count of the current device (0 on an error); the runtime's own query takes
// a fifth of a launch, so the answer is kept per device.
static inline int sm_count()
{
    static std::atomic<int> known[64];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev >= 0 && dev < 64 && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev >= 0 && dev < 64) known[dev].store(sms, std::memory_order_relaxed);
    return sms;
}

}  // namespace cdg

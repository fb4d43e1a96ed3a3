// What the decode-step kernels share: 16-bit conversions, the programmatic-dependent-launch
// helper, the status word's address and the error text (defined in decode.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/decode.h"
#include "overlap.h"

namespace decode {

// Stores the message for decode_last_error() and returns `code`.
__attribute__((visibility("hidden"))) int fail(int code, const char* fmt, ...);
__attribute__((visibility("hidden"))) void clear_error();

// Address of the status word of the current device; nullptr (with the error stored) on failure.
__attribute__((visibility("hidden"))) uint32_t* status_word();

// Multiprocessors of the current device; 0 (with the error stored) on failure.
__attribute__((visibility("hidden"))) int sm_count();

// Devices for which a thread keeps what it has looked up or set once.
constexpr int kMaxDevices = 64;

// Programmatic dependent launch: dep_wait() returns once all earlier work on the stream has
// completed and its writes are visible; dep_launch() lets the next kernel of the stream be placed.
__device__ __forceinline__ void dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dep_launch()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                           cudaStream_t stream, int cluster, Args... args)
{
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                   cudaStream_t stream, Args... args)
{
    return launch_cluster(kernel, grid, block, smem, stream, 1, args...);
}

constexpr int64_t kSmShared = 233472;     // bytes of an SM, of which the system takes 1 KB a block
constexpr size_t kSpreadMost = kSmShared / 2 - 1024 + 256;

// Shared memory for `blocks` blocks, fewer than the GPU holds (`resident` an SM): so much that an SM
// takes no more of them than an even spread gives it, and leaves room for the next kernel's first
// ones.  Without it some SMs fill up while others stay idle: 7740 tokens of 8 + 1 heads of 64 take
// 7.3 us in the norm's kernel, 6.4 with it; 208 sequences of 5 tokens, one state each, 8.3 us in the
// step's, 6.9.
inline size_t spread(size_t smem, int64_t blocks, int sms, int resident)
{
    const int64_t each = (blocks + sms - 1) / sms;
    if (each >= resident) return smem;
    const size_t least = static_cast<size_t>(kSmShared / (each + 1) - 1024 + 256) & ~size_t(127);
    return least > smem ? least : smem;
}

// Allows a kernel as much shared memory as spread() asks for, once per thread and device.
template <auto kKernel>
cudaError_t allow_spread()
{
    static thread_local bool done[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < kMaxDevices && done[dev])) return e;
    e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSpreadMost);
    if (e == cudaSuccess && dev < kMaxDevices) done[dev] = true;
    return e;
}

// Copies a tensor's strides, 0 for a dimension of one element; false if one is not a multiple of
// `of`.
template <int N>
bool take_strides(int64_t (&to)[N], const int64_t (&from)[N], const int64_t (&sizes)[N], int64_t of)
{
    bool ok = true;
    for (int d = 0; d < N; ++d) {
        to[d] = sizes[d] > 1 ? from[d] : 0;
        ok = ok && to[d] % of == 0;
    }
    return ok;
}

// Refuses a call in which a written operand shares memory with another one.
inline int refuse_shared(std::initializer_list<Operand> written, std::initializer_list<Operand> read)
{
    const char *one = nullptr, *other = nullptr;
    if (!find_shared(written, read, one, other)) return DECODE_OK;
    return fail(DECODE_ERR_INVALID_ARG, "%s shares memory with %s", one, other);
}

inline bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

// ---- 16-bit types ------------------------------------------------------------------------------

template <typename T>
struct Half2;
template <>
struct Half2<__half> {
    __device__ static float2 unpack(uint32_t x)
    {
        return __half22float2(*reinterpret_cast<const __half2*>(&x));
    }
    __device__ static uint32_t pack(float lo, float hi)
    {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};
template <>
struct Half2<__nv_bfloat16> {
    __device__ static float2 unpack(uint32_t x)
    {
        return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
    }
    __device__ static uint32_t pack(float lo, float hi)
    {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};

// ---- asynchronous copies to shared memory: 16 bytes, of which the last may be zeros instead, or 4 ----

__device__ __forceinline__ uint32_t smem_addr(const void* p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---- pairs -----------------------------------------------------------------------------------------

// Pairs of fp32 values in one 64-bit register pair: fma.rn.f32x2 does two products at the issue
// cost of one.
__device__ __forceinline__ uint64_t pair(float x, float y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 halves(uint64_t x)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

}  // namespace decode

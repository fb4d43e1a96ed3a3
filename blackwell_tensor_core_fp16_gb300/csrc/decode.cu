// The status word and the error text of the decode-step operators (C ABI in include/decode.h).
#include <cstdarg>
#include <cstdio>
#include <string>

#include "decode_common.cuh"

namespace {

thread_local std::string t_error;
__device__ uint32_t d_status;

// Reads and clears a status word in one step, so that a bit that another stream sets meanwhile
// is either in `to` or still in the word.
__global__ void take_status_kernel(uint32_t* word, uint32_t* to) { *to = atomicExch(word, 0u); }

// A word of pinned host memory, one for each thread.
struct HostWord {
    uint32_t* p = nullptr;
    ~HostWord()
    {
        if (p != nullptr) cudaFreeHost(p);
    }
    cudaError_t get(uint32_t*& to)
    {
        cudaError_t e = cudaSuccess;
        if (p == nullptr) e = cudaHostAlloc(reinterpret_cast<void**>(&p), sizeof(*p), cudaHostAllocPortable);
        to = p;
        return e;
    }
};

}  // namespace

namespace decode {

int fail(int code, const char* fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    t_error = buf;
    return code;
}

void clear_error() { t_error.clear(); }

uint32_t* status_word()
{
    static thread_local uint32_t* cached[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && dev >= 0 && dev < kMaxDevices && cached[dev] != nullptr)
        return cached[dev];
    void* p = nullptr;
    if (e == cudaSuccess) e = cudaGetSymbolAddress(&p, d_status);
    if (e != cudaSuccess) {
        fail(DECODE_ERR_CUDA, "status word: %s", cudaGetErrorString(e));
        return nullptr;
    }
    if (dev >= 0 && dev < kMaxDevices) cached[dev] = static_cast<uint32_t*>(p);
    return static_cast<uint32_t*>(p);
}

int sm_count()
{
    static thread_local int cached[kMaxDevices] = {};
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && dev >= 0 && dev < kMaxDevices && cached[dev] > 0) return cached[dev];
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess || sms <= 0) {
        fail(DECODE_ERR_CUDA, "device query: %s", cudaGetErrorString(e));
        return 0;
    }
    if (dev >= 0 && dev < kMaxDevices) cached[dev] = sms;
    return sms;
}

}  // namespace decode

extern "C" {

const char* decode_last_error(void) { return t_error.c_str(); }

int decode_check_status(cudaStream_t stream, uint32_t* bits)
{
    decode::clear_error();
    if (bits == nullptr) return decode::fail(DECODE_ERR_INVALID_ARG, "bits is null");
    *bits = 0;
    // the word of the stream's device, which is made current meanwhile
    int before = 0, dev = 0;
    cudaError_t e = cudaGetDevice(&before);
    if (e == cudaSuccess) e = cudaStreamGetDevice(stream, &dev);
    if (e == cudaSuccess && dev != before) e = cudaSetDevice(dev);
    if (e != cudaSuccess)
        return decode::fail(DECODE_ERR_CUDA, "the stream's device: %s", cudaGetErrorString(e));
    static thread_local HostWord host;
    uint32_t* taken = nullptr;
    uint32_t* word = decode::status_word();
    if (word != nullptr) {
        e = host.get(taken);
        if (e == cudaSuccess) {
            *taken = 0;
            take_status_kernel<<<1, 1, 0, stream>>>(word, taken);
            e = cudaGetLastError();
        }
        if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
        if (e == cudaSuccess) *bits = *taken;
    }
    if (dev != before) cudaSetDevice(before);
    if (word == nullptr) return DECODE_ERR_CUDA;
    if (e != cudaSuccess)
        return decode::fail(DECODE_ERR_CUDA, "reading the status word: %s", cudaGetErrorString(e));
    return DECODE_OK;
}

}  // extern "C"

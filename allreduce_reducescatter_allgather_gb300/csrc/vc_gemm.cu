// Host side of the product kernel: tensor maps, and the count of waits that
// ran out.  Nothing here allocates or throws: C entry points call it.
#include <atomic>

#include "vc_gemm.cuh"
#include "vc_train.h"

namespace vc {

int sm_count();  // vc_api.cu

namespace gemm {

namespace {
__device__ unsigned g_timeouts = 0;
}

constexpr int kMaxDevices = 64;

// Looked up once per device (by two threads at once, if it so happens).
unsigned* timeout_counter() {
    static std::atomic<unsigned*> where[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    unsigned* at = where[dev].load(std::memory_order_relaxed);
    if (at == nullptr) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_timeouts) != cudaSuccess) return nullptr;
        at = static_cast<unsigned*>(p);
        where[dev].store(at, std::memory_order_relaxed);
    }
    return at;
}

int device_sms() { return sm_count(); }

namespace {

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                             const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                             const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled through the runtime (the library does not link the
// driver); looked up once.
EncodeFn encoder() {
    static std::atomic<EncodeFn> found;
    EncodeFn fn = found.load(std::memory_order_relaxed);
    if (fn == nullptr) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &r) == cudaSuccess &&
            r == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeFn>(p);
        found.store(fn, std::memory_order_relaxed);
    }
    return fn;
}

}  // namespace

// (a kernel that finds its places of the table taken sets its limit each time)
cudaError_t allow_smem(const void* kernel) {
    constexpr unsigned kPlaces = 256, kProbes = 16;
    static std::atomic<const void*> done[kMaxDevices][kPlaces];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    const unsigned first = (unsigned)(reinterpret_cast<uintptr_t>(kernel) >> 4) * 2654435761u >> 24;
    unsigned i = 0;
    const void* there = nullptr;
    for (; i < kProbes; ++i) {
        there = done[dev][(first + i) % kPlaces].load(std::memory_order_relaxed);
        if (there == kernel) return cudaSuccess;
        if (there == nullptr) break;
    }
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemPerBlock);
    if (e == cudaSuccess && i < kProbes)
        done[dev][(first + i) % kPlaces].compare_exchange_strong(there, kernel, std::memory_order_relaxed);
    return e;
}

bool encode_operand(CUtensorMap* map, const Operand& o, int batch, int box_rows) {
    EncodeFn fn = encoder();
    if (fn == nullptr) return false;
    // A stride is only meaningful with a second row (or matrix); the encoder
    // still wants a multiple of 16 bytes.
    const cuuint64_t row = o.outer > 1 ? (cuuint64_t)o.ld * 2 : (cuuint64_t)((o.inner + 7) / 8 * 16);
    const cuuint64_t mat = batch > 1 ? (cuuint64_t)o.batch_stride * 2 : row;
    const cuuint64_t dims[3] = {(cuuint64_t)o.inner, (cuuint64_t)o.outer, (cuuint64_t)batch};
    const cuuint64_t strides[2] = {row, mat};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
    const cuuint32_t step[3] = {1, 1, 1};
    return fn(map, o.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
              const_cast<void*>(o.data), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

// A block whose warps wait, for about half a millisecond, for what never
// comes, as a product kernel's would if a copy were lost: it gives up, ends
// and counts itself.  For tests of the report (VC_TEST_WAIT_OUT).
__global__ void __launch_bounds__(128) wait_out_kernel(unsigned* timeouts) {
    __shared__ __align__(8) uint64_t barrier;
    __shared__ int dead_word;
    volatile int* const dead = &dead_word;
    const unsigned bar = smem_u32(&barrier);
    if (threadIdx.x == 0) {
        mbar_init(bar, 1);
        *dead = 0;
    }
    __syncthreads();
    bool alive = true;
    for (int i = 0; alive && i < 1000; ++i) alive = warp_wait(bar, 0, dead, 1000000);
    __syncthreads();
    bury(dead, timeouts);
}

}  // namespace
}  // namespace gemm
}  // namespace vc

extern "C" vc_status_t vc_train_timeouts(unsigned* count) {
    if (count == nullptr) return VC_ERR_INVALID_ARGUMENT;
    const char* v = getenv("VC_TEST_FAIL_LAUNCH");
    if (v != nullptr && v[0] != '\0' && v[0] != '0') return VC_ERR_CUDA;
    const unsigned* p = vc::gemm::timeout_counter();
    if (p == nullptr) return VC_ERR_CUDA;
    const char* out = getenv("VC_TEST_WAIT_OUT");
    if (out != nullptr && out[0] != '\0' && out[0] != '0') {
        vc::gemm::wait_out_kernel<<<1, 128>>>(const_cast<unsigned*>(p));
        if (cudaGetLastError() != cudaSuccess) return VC_ERR_CUDA;
    }
    // (the copy alone would not wait for streams that do not block)
    if (cudaDeviceSynchronize() != cudaSuccess) return VC_ERR_CUDA;
    return cudaMemcpy(count, p, sizeof *count, cudaMemcpyDeviceToHost) == cudaSuccess
               ? VC_SUCCESS
               : VC_ERR_CUDA;
}

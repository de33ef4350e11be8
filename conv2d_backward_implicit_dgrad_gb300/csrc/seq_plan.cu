// What the sequence operators' plans share (include/seq.h): the device check,
// workspaces and the error word.
#include "seq_common.cuh"

namespace seq {

using dgrad::cuda_status;

dgrad_status_t open_plan(PlanBase *base) {
    int dev = 0, major = 0, minor = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&base->sm_count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return DGRAD_ERR_NO_DEVICE;
    }
    if (major != 10 || minor != 3) return DGRAD_ERR_NO_DEVICE;
    base->device = dev;
    base->err = nullptr;
    void *mem = nullptr;
    if (cudaMalloc(&mem, kErrorBytes) != cudaSuccess) {
        cudaGetLastError();
        return DGRAD_ERR_OOM;
    }
    if (cudaMemset(mem, 0, kErrorBytes) != cudaSuccess || cudaStreamSynchronize(nullptr) != cudaSuccess) {
        cudaGetLastError();
        cudaFree(mem);
        return DGRAD_ERR_CUDA;
    }
    base->err = static_cast<uint32_t *>(mem);
    return DGRAD_OK;
}

dgrad_status_t on_device(const PlanBase &base) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return DGRAD_ERR_CUDA;
    return dev == base.device ? DGRAD_OK : DGRAD_ERR_WRONG_DEVICE;
}

dgrad_status_t grow(void **mem, size_t *have, size_t want) {
    if (*have >= want) return DGRAD_OK;
    void *p = nullptr;
    const cudaError_t e = cudaMalloc(&p, want);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return e == cudaErrorMemoryAllocation ? DGRAD_ERR_OOM : cuda_status(e);
    }
    cudaFree(*mem);
    *mem = p;
    *have = want;
    return DGRAD_OK;
}

dgrad_status_t read_error(const PlanBase &base) {
    uint32_t word = 0;
    if (cudaMemcpy(&word, base.err, sizeof(word), cudaMemcpyDeviceToHost) != cudaSuccess) return DGRAD_ERR_CUDA;
    if (word == 0) return DGRAD_OK;
    if (cudaMemset(base.err, 0, sizeof(word)) != cudaSuccess) return DGRAD_ERR_CUDA;
    return DGRAD_ERR_INVALID_ARG;
}

void close_plan(const PlanBase &base, void *const *mems, int n) {
    int cur = -1;
    cudaGetDevice(&cur);
    if (cur != base.device) cudaSetDevice(base.device);
    cudaDeviceSynchronize();
    cudaFree(base.err);
    for (int i = 0; i < n; ++i) cudaFree(mems[i]);
    if (cur >= 0 && cur != base.device) cudaSetDevice(cur);
}

}  // namespace seq

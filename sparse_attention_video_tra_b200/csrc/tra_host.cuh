// tra_host.cuh -- host helpers of the entry points that launch kernels: TMA
// tensor maps, alignment checks, launch status, and the error word of the
// translation unit that includes it.
#pragma once
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/tra.h"
#include "tra_plan_impl.h"
#include "pipeline.cuh"

namespace {

// True if a runtime call succeeded.  An error is taken off the runtime's record,
// where launch_status() of the next call would find it.
bool cuda_ok(cudaError_t e)
{
    if (e == cudaSuccess) return true;
    cudaGetLastError();
    return false;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cuda_ok(cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q)) &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// [rows][D] bf16 rows, 128-row x 64-column boxes, 128-byte swizzle
bool make_row_map(CUtensorMap* m, const void* base, uint64_t rows, int D)
{
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)D * 2};
    const cuuint32_t box[2] = {64, 128};
    const cuuint32_t es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [heads*T][H][W][D] bf16 in natural token order, {64, tw, th, 1} boxes (one
// panel of one (1, th, tw) tile; coordinates past the grid read as zeros)
bool make_natural_map(CUtensorMap* m, const void* base, const tra::Geom& G)
{
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)G.D, (cuuint64_t)G.W, (cuuint64_t)G.H, (cuuint64_t)G.T * G.G};
    const cuuint64_t strides[3] = {(cuuint64_t)G.D * 2, (cuuint64_t)G.W * G.D * 2, (cuuint64_t)G.H * G.W * G.D * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)G.tw, (cuuint32_t)G.th, 1};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// the input map for the plan's layout
bool make_input_map(CUtensorMap* m, const void* base, const tra::Geom& G)
{
    return G.natural ? make_natural_map(m, base, G) : make_row_map(m, base, (uint64_t)G.G * G.N_pad, G.D);
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

tra_status launch_status()
{
    return cudaGetLastError() == cudaSuccess ? TRA_OK : TRA_ERR_CUDA;
}

template <class K>
bool set_smem(K kernel, int bytes)
{
    return cuda_ok(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
}

// streaming multiprocessors of the card
constexpr int kSMs = 148;

// largest dynamic shared memory a CTA may use on sm_100
constexpr int kMaxSmem = 232448;

// read and clear this translation unit's error word
bool take_error_word(unsigned int& word)
{
    unsigned int w = 0;
    if (!cuda_ok(cudaMemcpyFromSymbol(&w, tra::g_tra_error, sizeof w))) return false;
    if (w) {
        const unsigned int zero = 0;
        if (!cuda_ok(cudaMemcpyToSymbol(tra::g_tra_error, &zero, sizeof zero))) return false;
    }
    word |= w;
    return true;
}

// An identity of the current CUDA context that no other context of the process
// shares, not even the one that takes its place after cudaDeviceReset; 0 where
// it cannot be told.
uint64_t context_id()
{
    using GetCurrent = CUresult (*)(CUcontext*);
    using GetId = CUresult (*)(CUcontext, unsigned long long*);
    static GetCurrent get_current = nullptr;
    static GetId get_id = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *a = nullptr, *b = nullptr;
        cudaDriverEntryPointQueryResult qa, qb;
        if (cuda_ok(cudaGetDriverEntryPoint("cuCtxGetCurrent", &a, cudaEnableDefault, &qa)) &&
            cuda_ok(cudaGetDriverEntryPoint("cuCtxGetId", &b, cudaEnableDefault, &qb)) &&
            qa == cudaDriverEntryPointSuccess && qb == cudaDriverEntryPointSuccess) {
            get_current = reinterpret_cast<GetCurrent>(a);
            get_id = reinterpret_cast<GetId>(b);
        }
    });
    CUcontext ctx = nullptr;
    unsigned long long id = 0;
    if (!get_id || get_current(&ctx) != CUDA_SUCCESS || !ctx || get_id(ctx, &id) != CUDA_SUCCESS) return 0;
    return id + 1;
}

// Lets KERNEL (no static shared memory) use all of a CTA's shared memory, once
// per context: the attribute lives as long as the context, and setting it
// costs about as much as a launch.
template <auto KERNEL>
bool allow_max_smem()
{
    static std::atomic<uint64_t> done[64];                   // by device: the context it was last set in
    int dev = 0;
    if (!cuda_ok(cudaGetDevice(&dev))) return false;
    const uint64_t ctx = dev < 64 ? context_id() : 0;
    if (ctx && done[dev].load(std::memory_order_relaxed) == ctx) return true;
    if (!set_smem(KERNEL, kMaxSmem)) return false;
    if (ctx) done[dev].store(ctx, std::memory_order_relaxed);
    return true;
}

}  // namespace

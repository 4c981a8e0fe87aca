// abi.hip -- the C ABI of libmxfp4cvt (declared in include/mxfp4cvt.h): synchronous
// argument validation, then the call's kernel launches on the caller's stream (one per
// call, three for the NVFP4 quantizer, two for an expert map of many slots), all through
// launch_kernel.
#include <math.h>
#include <stdlib.h>
#include <string.h>

#include <atomic>
#include <mutex>

#include <hip/hip_ext.h>

#include "mxfp4cvt.h"
#include "common.h"

namespace mxfp4 {
hipError_t launch_quantize_rows(const uint16_t*, uint8_t*, uint8_t*, const int32_t*, int32_t,
                                int64_t, int64_t, hipStream_t);
hipError_t launch_fp8_rows(const uint8_t*, const uint8_t*, uint8_t*, uint8_t*, const int32_t*,
                           int32_t, int64_t, int64_t, hipStream_t);
hipError_t launch_fp8_cols(const uint8_t*, const uint8_t*, uint8_t*, uint8_t*, const int32_t*,
                           int32_t, int64_t, int64_t, WaitCtl, hipStream_t);
int64_t cols_block_capacity(int64_t M_cap, int32_t G);
hipError_t launch_fp8_gemm(const uint8_t*, const uint8_t*, const uint8_t*, const uint8_t*, uint16_t*,
                           const int32_t*, int32_t, int64_t, int64_t, int64_t, hipStream_t);
hipError_t launch_fp8_wgrad(const uint8_t*, const uint8_t*, const uint8_t*, const uint8_t*, uint16_t*,
                            const int32_t*, int32_t, int64_t, int64_t, int64_t, int64_t, hipStream_t);
hipError_t launch_nvfp4_quantize_rows(const uint16_t*, uint8_t*, uint8_t*, float*, const int32_t*, int32_t,
                                      int64_t, int64_t, bool, uint64_t, hipStream_t);
hipError_t launch_fp8q_cols(const uint16_t*, uint8_t*, uint8_t*, uint8_t*, uint8_t*, const int32_t*, int32_t, int64_t,
                            int64_t, WaitCtl, hipStream_t);
hipError_t launch_fp8q_rows(const uint16_t*, uint8_t*, uint8_t*, const int32_t*, int32_t, int64_t,
                            int64_t, hipStream_t);
hipError_t launch_route(const void*, bool, const float*, const uint8_t*, int32_t*, float*, int64_t, int32_t, int32_t,
                        int32_t, int32_t, int32_t, bool, bool, float, hipStream_t);
hipError_t launch_route_backward(const void*, bool, const int32_t*, const float*, void*, int64_t, int32_t, int32_t,
                                 bool, bool, float, hipStream_t);
int64_t expert_map_chunks(int64_t slots);
hipError_t launch_expert_map(const int32_t*, int32_t*, int32_t*, int32_t*, int32_t*, int64_t, int32_t, int32_t,
                             int64_t, hipStream_t);
hipError_t launch_dispatch_rows(const uint16_t*, const int32_t*, uint8_t*, uint8_t*, int64_t, int32_t, int64_t,
                                int64_t, hipStream_t);
hipError_t launch_dispatch_fp8_rows(const uint16_t*, const int32_t*, uint8_t*, float*, int64_t, int32_t, int64_t,
                                    int64_t, hipStream_t);
hipError_t launch_fp8_rows_f32(const uint16_t*, uint8_t*, float*, const int32_t*, int32_t, int64_t, int64_t,
                               hipStream_t);
hipError_t launch_block_gemm(const uint8_t*, const float*, const uint8_t*, const float*, uint16_t*, const int32_t*,
                             int32_t, int64_t, int64_t, int64_t, hipStream_t);
hipError_t launch_combine(const uint16_t*, const int32_t*, const float*, const uint16_t*, uint16_t*, int64_t, int32_t,
                          int64_t, int64_t, hipStream_t);
hipError_t launch_combine_backward(const uint16_t*, const uint16_t*, const int32_t*, const float*, uint16_t*, float*,
                                   int64_t, int32_t, int64_t, int64_t, hipStream_t);
}  // namespace mxfp4

namespace {

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Largest M_cap * K the kernels index: every byte count stays far inside int64.
constexpr int64_t kMaxElems = (int64_t)1 << 50;
// Largest K of the column conversion.
constexpr int64_t kMaxColsK = (int64_t)1 << 24;
// Largest N and K of the GEMM (its per-tile byte offsets are 32-bit).
constexpr int64_t kMaxGemmDim = (int64_t)1 << 20;
// Largest width * M_cap of a weight-gradient operand (its byte offsets are 32-bit).
constexpr int64_t kMaxWgradBytes = (int64_t)1 << 30;

mxfp4_status check_shape(int32_t G, int64_t M_cap, int64_t K, int64_t k_multiple)
{
    if (G < 1 || M_cap < 0 || K <= 0 || K % k_multiple != 0)
        return MXFP4_ERR_SHAPE;
    if (M_cap > 0 && K > kMaxElems / M_cap)
        return MXFP4_ERR_SHAPE;
    if (M_cap > INT32_MAX)                   // offsets are int32
        return MXFP4_ERR_SHAPE;
    return MXFP4_OK;
}

// Largest number of experts a router or an expert map takes, and of choices per token.
constexpr int32_t kMaxExperts = 1024;
constexpr int32_t kMaxChoices = 64;

// A call over the k choices of T tokens, rows of K elements, outputs or inputs of M_cap rows.
mxfp4_status check_tokens(int64_t T, int32_t k, int64_t M_cap, int64_t K, int64_t k_multiple)
{
    if (T < 0 || k < 1 || k > kMaxChoices || M_cap < 0 || K <= 0 || K > INT32_MAX || K % k_multiple != 0)
        return MXFP4_ERR_SHAPE;
    if (T > INT32_MAX / k || M_cap > INT32_MAX)      // positions are int32
        return MXFP4_ERR_SHAPE;
    if ((T > 0 && K > kMaxElems / T) || (M_cap > 0 && K > kMaxElems / M_cap))
        return MXFP4_ERR_SHAPE;
    return MXFP4_OK;
}

mxfp4_status check_route(int64_t T, int32_t E, int32_t k, int32_t score, float scale)
{
    if (T < 0 || T > INT32_MAX || E < 1 || E > kMaxExperts || k < 1 || k > kMaxChoices || k > E)
        return MXFP4_ERR_SHAPE;
    if (T > INT32_MAX / k || (score != MXFP4_SCORE_SOFTMAX && score != MXFP4_SCORE_SIGMOID))
        return MXFP4_ERR_SHAPE;
    return isfinite(scale) ? MXFP4_OK : MXFP4_ERR_SHAPE;
}

mxfp4_status from_hip(hipError_t e) { return e == hipSuccess ? MXFP4_OK : MXFP4_ERR_HIP; }

// ---- bounded-wait give-up status ----------------------------------------------------

// Set (to nonzero) by any column-kernel wave whose bounded wait ran out of polls; each
// device holds its own copy, zero when the code object loads.  Host code uses the
// address hipGetSymbolAddress gives for the device, never this name.
__device__ uint32_t wait_status;

constexpr int kMaxDevices = 64;
std::atomic<uint32_t*> status_addr[kMaxDevices];
std::mutex status_mu;
std::atomic<uint32_t> spin_limit{0};         // 0: the default

// The current device's status word address (looked up once per device).
hipError_t status_word(uint32_t** out)
{
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess)
        return e;
    if (dev < 0 || dev >= kMaxDevices)
        return hipErrorInvalidDevice;
    uint32_t* p = status_addr[dev].load(std::memory_order_acquire);
    if (!p) {
        std::lock_guard<std::mutex> lock(status_mu);
        p = status_addr[dev].load(std::memory_order_relaxed);
        if (!p) {
            e = hipGetSymbolAddress((void**)&p, HIP_SYMBOL(wait_status));
            if (e != hipSuccess)
                return e;
            status_addr[dev].store(p, std::memory_order_release);
        }
    }
    *out = p;
    return hipSuccess;
}

hipError_t wait_ctl(mxfp4::WaitCtl* w)
{
    const uint32_t lim = spin_limit.load(std::memory_order_relaxed);
    w->limit = lim ? lim : mxfp4::kDefaultSpinLimit;
    return status_word(&w->status);
}

// Copies the current device's status word to *flag, stream-ordered, and waits for it.
hipError_t read_status(uint32_t* flag, hipStream_t stream)
{
    uint32_t* p = nullptr;
    hipError_t e = status_word(&p);
    if (e == hipSuccess)
        e = hipMemcpyAsync(flag, p, sizeof(uint32_t), hipMemcpyDeviceToHost, stream);
    if (e == hipSuccess)
        e = hipStreamSynchronize(stream);
    return e;
}

// Timing events armed by mxfp4_time_next_launch on this thread.
thread_local hipEvent_t armed_start = nullptr;
thread_local hipEvent_t armed_stop = nullptr;

}  // namespace

hipError_t mxfp4::launch_kernel(const void* kernel, dim3 grid, dim3 block, void** args, hipStream_t stream,
                                bool last_of_call)
{
    hipEvent_t start = armed_start;
    hipEvent_t stop = last_of_call ? armed_stop : nullptr;
    if (!start && !stop)
        return hipLaunchKernel(kernel, grid, block, args, 0, stream);
    armed_start = nullptr;
    if (last_of_call)
        armed_stop = nullptr;
    return hipExtLaunchKernel(kernel, grid, block, args, 0, stream, start, stop, 0);
}

extern "C" {

mxfp4_status mxfp4_quantize_rows(const uint16_t* x_bf16, uint8_t* codes, uint8_t* scales,
                                 const int32_t* group_offsets, int32_t G, int64_t M_cap,
                                 int64_t K, hipStream_t stream)
{
    if (!x_bf16 || !codes || !scales || !group_offsets)
        return MXFP4_ERR_NULL;
    mxfp4_status st = check_shape(G, M_cap, K, 32);
    if (st != MXFP4_OK)
        return st;
    if (!aligned(x_bf16, 16) || !aligned(codes, 16) || !aligned(scales, 16) ||
        !aligned(group_offsets, 4))
        return MXFP4_ERR_ALIGN;
    if (M_cap == 0)
        return MXFP4_OK;
    return from_hip(mxfp4::launch_quantize_rows(x_bf16, codes, scales, group_offsets, G, M_cap,
                                                K, stream));
}

static mxfp4_status nvfp4_entry(const uint16_t* x_bf16, uint8_t* codes, uint8_t* scales_e4m3, float* tensor_amax,
                                const int32_t* group_offsets, int32_t G, int64_t M_cap, int64_t K, bool sr,
                                uint64_t seed, hipStream_t stream)
{
    if (!x_bf16 || !codes || !scales_e4m3 || !tensor_amax || !group_offsets)
        return MXFP4_ERR_NULL;
    mxfp4_status st = check_shape(G, M_cap, K, 16);
    if (st != MXFP4_OK)
        return st;
    if (!aligned(x_bf16, 16) || !aligned(codes, 16) || !aligned(scales_e4m3, 16) || !aligned(tensor_amax, 4) ||
        !aligned(group_offsets, 4))
        return MXFP4_ERR_ALIGN;
    return from_hip(mxfp4::launch_nvfp4_quantize_rows(x_bf16, codes, scales_e4m3, tensor_amax, group_offsets, G,
                                                      M_cap, K, sr, seed, stream));
}

mxfp4_status mxfp4_nvfp4_quantize_rows(const uint16_t* x_bf16, uint8_t* codes, uint8_t* scales_e4m3,
                                       float* tensor_amax, const int32_t* group_offsets, int32_t G,
                                       int64_t M_cap, int64_t K, hipStream_t stream)
{
    return nvfp4_entry(x_bf16, codes, scales_e4m3, tensor_amax, group_offsets, G, M_cap, K, false, 0, stream);
}

mxfp4_status mxfp4_nvfp4_quantize_rows_sr(const uint16_t* x_bf16, uint8_t* codes, uint8_t* scales_e4m3,
                                          float* tensor_amax, const int32_t* group_offsets, int32_t G,
                                          int64_t M_cap, int64_t K, uint64_t seed, hipStream_t stream)
{
    return nvfp4_entry(x_bf16, codes, scales_e4m3, tensor_amax, group_offsets, G, M_cap, K, true, seed, stream);
}

mxfp4_status mxfp4_to_fp8_rows(const uint8_t* codes, const uint8_t* scales, uint8_t* y_e4m3,
                               uint8_t* y_scales, const int32_t* group_offsets, int32_t G,
                               int64_t M_cap, int64_t K, hipStream_t stream)
{
    if (!codes || !scales || !y_e4m3 || !y_scales || !group_offsets)
        return MXFP4_ERR_NULL;
    mxfp4_status st = check_shape(G, M_cap, K, 128);
    if (st != MXFP4_OK)
        return st;
    if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(y_e4m3, 16) ||
        !aligned(y_scales, 16) || !aligned(group_offsets, 4))
        return MXFP4_ERR_ALIGN;
    if (M_cap == 0)
        return MXFP4_OK;
    return from_hip(mxfp4::launch_fp8_rows(codes, scales, y_e4m3, y_scales, group_offsets, G,
                                           M_cap, K, stream));
}

mxfp4_status mxfp4_to_fp8_cols_ragged(const uint8_t* codes, const uint8_t* scales,
                                      uint8_t* yT_e4m3, uint8_t* yT_scales,
                                      const int32_t* group_offsets, int32_t G, int64_t M_cap,
                                      int64_t K, hipStream_t stream)
{
    if (!codes || !scales || !yT_e4m3 || !yT_scales || !group_offsets)
        return MXFP4_ERR_NULL;
    mxfp4_status st = check_shape(G, M_cap, K, 128);
    if (st != MXFP4_OK)
        return st;
    if (K > kMaxColsK)                       // the kernel's per-strip row offsets are 32-bit
        return MXFP4_ERR_SHAPE;
    if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(yT_e4m3, 16) ||
        !aligned(yT_scales, 16) || !aligned(group_offsets, 4))
        return MXFP4_ERR_ALIGN;
    if (M_cap == 0)
        return MXFP4_OK;
    mxfp4::WaitCtl wc;
    hipError_t e = wait_ctl(&wc);
    if (e == hipSuccess)
        e = mxfp4::launch_fp8_cols(codes, scales, yT_e4m3, yT_scales, group_offsets, G, M_cap, K, wc, stream);
    return from_hip(e);
}

mxfp4_status mxfp4_bf16_to_fp8_rows(const uint16_t* x_bf16, uint8_t* y_e4m3, uint8_t* y_scales,
                                    const int32_t* group_offsets, int32_t G, int64_t M_cap,
                                    int64_t K, hipStream_t stream)
{
    if (!x_bf16 || !y_e4m3 || !y_scales || !group_offsets)
        return MXFP4_ERR_NULL;
    mxfp4_status st = check_shape(G, M_cap, K, 128);
    if (st != MXFP4_OK)
        return st;
    if (!aligned(x_bf16, 16) || !aligned(y_e4m3, 16) || !aligned(y_scales, 16) ||
        !aligned(group_offsets, 4))
        return MXFP4_ERR_ALIGN;
    if (M_cap == 0)
        return MXFP4_OK;
    return from_hip(mxfp4::launch_fp8q_rows(x_bf16, y_e4m3, y_scales, group_offsets, G, M_cap, K,
                                            stream));
}

mxfp4_status mxfp4_bf16_to_fp8_cols_ragged(const uint16_t* x_bf16, uint8_t* yT_e4m3,
                                           uint8_t* yT_scales, const int32_t* group_offsets,
                                           int32_t G, int64_t M_cap, int64_t K,
                                           hipStream_t stream)
{
    if (!x_bf16 || !yT_e4m3 || !yT_scales || !group_offsets)
        return MXFP4_ERR_NULL;
    mxfp4_status st = check_shape(G, M_cap, K, 128);
    if (st != MXFP4_OK)
        return st;
    if (K > kMaxColsK)                       // the kernel's per-strip row offsets are 32-bit
        return MXFP4_ERR_SHAPE;
    if (!aligned(x_bf16, 16) || !aligned(yT_e4m3, 16) || !aligned(yT_scales, 16) ||
        !aligned(group_offsets, 4))
        return MXFP4_ERR_ALIGN;
    if (M_cap == 0)
        return MXFP4_OK;
    mxfp4::WaitCtl wc;
    hipError_t e = wait_ctl(&wc);
    if (e == hipSuccess)
        e = mxfp4::launch_fp8q_cols(x_bf16, yT_e4m3, yT_scales, nullptr, nullptr, group_offsets, G, M_cap, K,
                                    wc, stream);
    return from_hip(e);
}

mxfp4_status mxfp4_bf16_to_fp8_rows_cols_ragged(const uint16_t* x_bf16, uint8_t* y_e4m3, uint8_t* y_scales,
                                                uint8_t* yT_e4m3, uint8_t* yT_scales,
                                                const int32_t* group_offsets, int32_t G, int64_t M_cap,
                                                int64_t K, hipStream_t stream)
{
    if (!x_bf16 || !y_e4m3 || !y_scales || !yT_e4m3 || !yT_scales || !group_offsets)
        return MXFP4_ERR_NULL;
    mxfp4_status st = check_shape(G, M_cap, K, 128);
    if (st != MXFP4_OK)
        return st;
    if (K > kMaxColsK)                       // the kernel's per-strip row offsets are 32-bit
        return MXFP4_ERR_SHAPE;
    if (!aligned(x_bf16, 16) || !aligned(y_e4m3, 16) || !aligned(y_scales, 16) || !aligned(yT_e4m3, 16) ||
        !aligned(yT_scales, 16) || !aligned(group_offsets, 4))
        return MXFP4_ERR_ALIGN;
    if (M_cap == 0)
        return MXFP4_OK;
    mxfp4::WaitCtl wc;
    hipError_t e = wait_ctl(&wc);
    if (e == hipSuccess)
        e = mxfp4::launch_fp8q_cols(x_bf16, yT_e4m3, yT_scales, y_e4m3, y_scales, group_offsets, G, M_cap, K,
                                    wc, stream);
    return from_hip(e);
}

mxfp4_status mxfp4_fp8_grouped_gemm(const uint8_t* a_e4m3, const uint8_t* a_scales,
                                    const uint8_t* w_e4m3, const uint8_t* w_scales,
                                    uint16_t* y_bf16, const int32_t* group_offsets, int32_t G,
                                    int64_t M_cap, int64_t N, int64_t K, hipStream_t stream)
{
    if (!a_e4m3 || !a_scales || !w_e4m3 || !w_scales || !y_bf16 || !group_offsets)
        return MXFP4_ERR_NULL;
    mxfp4_status st = check_shape(G, M_cap, K, 128);
    if (st != MXFP4_OK)
        return st;
    if (K > kMaxGemmDim || N <= 0 || N % 256 != 0 || N > kMaxGemmDim)
        return MXFP4_ERR_SHAPE;
    if (M_cap > 0 && N > kMaxElems / M_cap)          // output elements
        return MXFP4_ERR_SHAPE;
    if ((int64_t)G > kMaxElems / (N * K))             // weight elements
        return MXFP4_ERR_SHAPE;
    if (!aligned(a_e4m3, 16) || !aligned(a_scales, 16) || !aligned(w_e4m3, 16) ||
        !aligned(w_scales, 16) || !aligned(y_bf16, 16) || !aligned(group_offsets, 4))
        return MXFP4_ERR_ALIGN;
    if (M_cap == 0)
        return MXFP4_OK;
    return from_hip(mxfp4::launch_fp8_gemm(a_e4m3, a_scales, w_e4m3, w_scales, y_bf16, group_offsets,
                                           G, M_cap, N, K, stream));
}

mxfp4_status mxfp4_fp8_grouped_gemm_wgrad(const uint8_t* dyT_e4m3, const uint8_t* dyT_scales,
                                          const uint8_t* xT_e4m3, const uint8_t* xT_scales, uint16_t* dw_bf16,
                                          const int32_t* group_offsets, int32_t G, int64_t M_cap, int64_t N,
                                          int64_t K, hipStream_t stream)
{
    if (!dyT_e4m3 || !dyT_scales || !xT_e4m3 || !xT_scales || !dw_bf16 || !group_offsets)
        return MXFP4_ERR_NULL;
    mxfp4_status st = check_shape(G, M_cap, K, 256);
    if (st != MXFP4_OK)
        return st;
    if (N <= 0 || N % 256 != 0 || N > kMaxGemmDim || K > kMaxGemmDim)
        return MXFP4_ERR_SHAPE;
    if (M_cap > 0 && (N > kMaxWgradBytes / M_cap || K > kMaxWgradBytes / M_cap))
        return MXFP4_ERR_SHAPE;
    if ((int64_t)G > kMaxElems / (N * K))             // output elements
        return MXFP4_ERR_SHAPE;
    if (!aligned(dyT_e4m3, 16) || !aligned(dyT_scales, 16) || !aligned(xT_e4m3, 16) ||
        !aligned(xT_scales, 16) || !aligned(dw_bf16, 16) || !aligned(group_offsets, 4))
        return MXFP4_ERR_ALIGN;
    return from_hip(mxfp4::launch_fp8_wgrad(dyT_e4m3, dyT_scales, xT_e4m3, xT_scales, dw_bf16, group_offsets, G,
                                            M_cap, mxfp4::cols_block_capacity(M_cap, G), N, K, stream));
}

mxfp4_status mxfp4_route_topk(const void* logits, int32_t logits_f32, const float* bias, const uint8_t* row_mask,
                              int32_t* ids, float* weights, int64_t T, int32_t E, int32_t n_group,
                              int32_t topk_group, int32_t group_best, int32_t k, int32_t score, int32_t renorm,
                              float scale, hipStream_t stream)
{
    if (!logits || !ids || !weights)
        return MXFP4_ERR_NULL;
    mxfp4_status st = check_route(T, E, k, score, scale);
    if (st != MXFP4_OK)
        return st;
    if (n_group < 1 || n_group > 64 || E % n_group != 0 || topk_group < 1 || topk_group > n_group)
        return MXFP4_ERR_SHAPE;
    if (group_best < 1 || group_best > 2 || group_best > E / n_group || k > topk_group * (E / n_group))
        return MXFP4_ERR_SHAPE;
    if (!aligned(logits, 16) || !aligned(bias, 16) || !aligned(row_mask, 16) || !aligned(ids, 16) ||
        !aligned(weights, 16))
        return MXFP4_ERR_ALIGN;
    if (T == 0)
        return MXFP4_OK;
    return from_hip(mxfp4::launch_route(logits, logits_f32 != 0, bias, row_mask, ids, weights, T, E, n_group,
                                        topk_group, group_best, k, score == MXFP4_SCORE_SIGMOID, renorm != 0, scale,
                                        stream));
}

mxfp4_status mxfp4_route_topk_backward(const void* logits, int32_t logits_f32, const int32_t* ids,
                                       const float* dweights, void* dlogits, int64_t T, int32_t E, int32_t k,
                                       int32_t score, int32_t renorm, float scale, hipStream_t stream)
{
    if (!logits || !ids || !dweights || !dlogits)
        return MXFP4_ERR_NULL;
    mxfp4_status st = check_route(T, E, k, score, scale);
    if (st != MXFP4_OK)
        return st;
    if (!aligned(logits, 16) || !aligned(ids, 16) || !aligned(dweights, 16) || !aligned(dlogits, 16))
        return MXFP4_ERR_ALIGN;
    if (T == 0)
        return MXFP4_OK;
    return from_hip(mxfp4::launch_route_backward(logits, logits_f32 != 0, ids, dweights, dlogits, T, E, k,
                                                 score == MXFP4_SCORE_SIGMOID, renorm != 0, scale, stream));
}

int64_t mxfp4_expert_map_workspace(int64_t T, int32_t k, int32_t G)
{
    if (check_tokens(T, k, 0, 1, 1) != MXFP4_OK || G < 1 || G > kMaxExperts)
        return -1;
    return 4 * mxfp4::expert_map_chunks(T * k) * G;
}

mxfp4_status mxfp4_expert_map(const int32_t* ids, int32_t* group_offsets, int32_t* pos, int32_t* src,
                              void* workspace, int64_t T, int32_t k, int32_t first_expert, int32_t G, int64_t M_cap,
                              hipStream_t stream)
{
    if (!ids || !group_offsets || !pos)
        return MXFP4_ERR_NULL;
    const int64_t need = mxfp4_expert_map_workspace(T, k, G);
    if (need < 0 || first_expert < 0 || M_cap < 0 || M_cap > INT32_MAX)
        return MXFP4_ERR_SHAPE;
    if (need > 0 && !workspace)
        return MXFP4_ERR_NULL;
    if (!aligned(ids, 16) || !aligned(pos, 16) || !aligned(src, 16) || !aligned(workspace, 16) ||
        !aligned(group_offsets, 4))
        return MXFP4_ERR_ALIGN;
    return from_hip(mxfp4::launch_expert_map(ids, group_offsets, pos, src, static_cast<int32_t*>(workspace), T * k,
                                             first_expert, G, M_cap, stream));
}

mxfp4_status mxfp4_dispatch_rows(const uint16_t* x_bf16, const int32_t* pos, uint8_t* codes, uint8_t* scales,
                                 int64_t T, int32_t k, int64_t M_cap, int64_t K, hipStream_t stream)
{
    if (!x_bf16 || !pos || !codes || !scales)
        return MXFP4_ERR_NULL;
    mxfp4_status st = check_tokens(T, k, M_cap, K, 32);
    if (st != MXFP4_OK)
        return st;
    if (!aligned(x_bf16, 16) || !aligned(pos, 16) || !aligned(codes, 16) || !aligned(scales, 16))
        return MXFP4_ERR_ALIGN;
    if (T == 0 || M_cap == 0)
        return MXFP4_OK;
    return from_hip(mxfp4::launch_dispatch_rows(x_bf16, pos, codes, scales, T, k, M_cap, K, stream));
}

mxfp4_status mxfp4_dispatch_fp8_rows(const uint16_t* x_bf16, const int32_t* pos, uint8_t* y_e4m3, float* y_scales,
                                     int64_t T, int32_t k, int64_t M_cap, int64_t K, hipStream_t stream)
{
    if (!x_bf16 || !pos || !y_e4m3 || !y_scales)
        return MXFP4_ERR_NULL;
    mxfp4_status st = check_tokens(T, k, M_cap, K, 16);
    if (st != MXFP4_OK)
        return st;
    if (!aligned(x_bf16, 16) || !aligned(pos, 16) || !aligned(y_e4m3, 16) || !aligned(y_scales, 16))
        return MXFP4_ERR_ALIGN;
    if (T == 0 || M_cap == 0)
        return MXFP4_OK;
    return from_hip(mxfp4::launch_dispatch_fp8_rows(x_bf16, pos, y_e4m3, y_scales, T, k, M_cap, K, stream));
}

mxfp4_status mxfp4_bf16_to_fp8_rows_f32(const uint16_t* x_bf16, uint8_t* y_e4m3, float* y_scales,
                                        const int32_t* group_offsets, int32_t G, int64_t M_cap, int64_t K,
                                        hipStream_t stream)
{
    if (!x_bf16 || !y_e4m3 || !y_scales || !group_offsets)
        return MXFP4_ERR_NULL;
    mxfp4_status st = check_shape(G, M_cap, K, 16);
    if (st == MXFP4_OK && K > INT32_MAX)             // lanes of a row are counted in 32 bits
        st = MXFP4_ERR_SHAPE;
    if (st != MXFP4_OK)
        return st;
    if (!aligned(x_bf16, 16) || !aligned(y_e4m3, 16) || !aligned(y_scales, 16) || !aligned(group_offsets, 4))
        return MXFP4_ERR_ALIGN;
    if (M_cap == 0)
        return MXFP4_OK;
    return from_hip(mxfp4::launch_fp8_rows_f32(x_bf16, y_e4m3, y_scales, group_offsets, G, M_cap, K, stream));
}

mxfp4_status mxfp4_fp8_block_gemm(const uint8_t* a_e4m3, const float* a_scales, const uint8_t* w_e4m3,
                                  const float* w_scales, uint16_t* y_bf16, const int32_t* group_offsets, int32_t G,
                                  int64_t M_cap, int64_t N, int64_t K, hipStream_t stream)
{
    if (!a_e4m3 || !a_scales || !w_e4m3 || !w_scales || !y_bf16 || !group_offsets)
        return MXFP4_ERR_NULL;
    mxfp4_status st = check_shape(G, M_cap, K, 16);
    if (st != MXFP4_OK)
        return st;
    if (K > kMaxGemmDim || N <= 0 || N % 8 != 0 || N > kMaxGemmDim)
        return MXFP4_ERR_SHAPE;
    if (M_cap > 0 && N > kMaxElems / M_cap)          // output elements
        return MXFP4_ERR_SHAPE;
    if ((int64_t)G > kMaxElems / (N * K))             // weight elements
        return MXFP4_ERR_SHAPE;
    if (!aligned(a_e4m3, 16) || !aligned(a_scales, 16) || !aligned(w_e4m3, 16) || !aligned(w_scales, 16) ||
        !aligned(y_bf16, 16) || !aligned(group_offsets, 4))
        return MXFP4_ERR_ALIGN;
    if (M_cap == 0)
        return MXFP4_OK;
    return from_hip(mxfp4::launch_block_gemm(a_e4m3, a_scales, w_e4m3, w_scales, y_bf16, group_offsets, G, M_cap, N,
                                             K, stream));
}

mxfp4_status mxfp4_combine_rows(const uint16_t* y_bf16, const int32_t* pos, const float* weights,
                                const uint16_t* base_bf16, uint16_t* out_bf16, int64_t T, int32_t k, int64_t M_cap,
                                int64_t K, hipStream_t stream)
{
    if (!y_bf16 || !pos || !out_bf16)
        return MXFP4_ERR_NULL;
    mxfp4_status st = check_tokens(T, k, M_cap, K, 8);
    if (st != MXFP4_OK)
        return st;
    if (!aligned(y_bf16, 16) || !aligned(pos, 16) || !aligned(weights, 16) || !aligned(base_bf16, 16) ||
        !aligned(out_bf16, 16))
        return MXFP4_ERR_ALIGN;
    if (T == 0)
        return MXFP4_OK;
    return from_hip(mxfp4::launch_combine(y_bf16, pos, weights, base_bf16, out_bf16, T, k, M_cap, K, stream));
}

mxfp4_status mxfp4_combine_rows_backward(const uint16_t* dout_bf16, const uint16_t* y_bf16, const int32_t* pos,
                                         const float* weights, uint16_t* dy_bf16, float* dweights, int64_t T,
                                         int32_t k, int64_t M_cap, int64_t K, hipStream_t stream)
{
    if (!dout_bf16 || !y_bf16 || !pos || !weights || !dy_bf16 || !dweights)
        return MXFP4_ERR_NULL;
    mxfp4_status st = check_tokens(T, k, M_cap, K, 8);
    if (st != MXFP4_OK)
        return st;
    if (!aligned(dout_bf16, 16) || !aligned(y_bf16, 16) || !aligned(pos, 16) || !aligned(weights, 16) ||
        !aligned(dy_bf16, 16) || !aligned(dweights, 16))
        return MXFP4_ERR_ALIGN;
    if (T == 0)
        return MXFP4_OK;
    return from_hip(mxfp4::launch_combine_backward(dout_bf16, y_bf16, pos, weights, dy_bf16, dweights, T, k, M_cap, K,
                                                   stream));
}

int64_t mxfp4_cols_scale_capacity(int64_t M_cap, int64_t K, int32_t G)
{
    if (check_shape(G, M_cap, K, 128) != MXFP4_OK)
        return -1;
    return K * mxfp4::cols_block_capacity(M_cap, G);
}

mxfp4_status mxfp4_validate_offsets(const int32_t* group_offsets, int32_t G, int64_t M_cap,
                                    hipStream_t stream)
{
    if (!group_offsets)
        return MXFP4_ERR_NULL;
    if (G < 1 || M_cap < 0 || M_cap > INT32_MAX)
        return MXFP4_ERR_SHAPE;
    int32_t* h = (int32_t*)malloc(sizeof(int32_t) * ((size_t)G + 1));
    if (!h)
        return MXFP4_ERR_HIP;
    hipError_t e = hipMemcpyAsync(h, group_offsets, sizeof(int32_t) * ((size_t)G + 1),
                                  hipMemcpyDeviceToHost, stream);
    if (e == hipSuccess)
        e = hipStreamSynchronize(stream);
    mxfp4_status st = from_hip(e);
    if (st == MXFP4_OK) {
        if (h[0] != 0)
            st = MXFP4_ERR_SHAPE;
        for (int32_t g = 0; g < G && st == MXFP4_OK; ++g)
            if (h[g + 1] < h[g])
                st = MXFP4_ERR_SHAPE;
        if (st == MXFP4_OK && (int64_t)h[G] > M_cap)
            st = MXFP4_ERR_SHAPE;
    }
    free(h);
    if (st == MXFP4_OK) {
        uint32_t flag = 0;
        st = from_hip(read_status(&flag, stream));
        if (st == MXFP4_OK && flag)
            st = MXFP4_ERR_HIP;
    }
    return st;
}

mxfp4_status mxfp4_wait_status(hipStream_t stream)
{
    uint32_t flag = 0;
    hipError_t e = read_status(&flag, stream);
    if (e == hipSuccess && flag) {
        uint32_t* p = nullptr;
        static const uint32_t zero = 0;
        e = status_word(&p);
        if (e == hipSuccess)
            e = hipMemcpyAsync(p, &zero, sizeof(uint32_t), hipMemcpyHostToDevice, stream);
        if (e == hipSuccess)
            e = hipStreamSynchronize(stream);
    }
    if (e != hipSuccess)
        return MXFP4_ERR_HIP;
    return flag ? MXFP4_ERR_HIP : MXFP4_OK;
}

void mxfp4_set_wait_limit(uint32_t polls) { spin_limit.store(polls, std::memory_order_relaxed); }

mxfp4_status mxfp4_time_next_launch(hipEvent_t start, hipEvent_t stop)
{
    armed_start = start;
    armed_stop = stop;
    return MXFP4_OK;
}

const char* mxfp4_status_string(mxfp4_status status)
{
    switch (status) {
    case MXFP4_OK: return "MXFP4_OK";
    case MXFP4_ERR_NULL: return "MXFP4_ERR_NULL: a required pointer is NULL";
    case MXFP4_ERR_SHAPE: return "MXFP4_ERR_SHAPE: invalid G, M_cap or K";
    case MXFP4_ERR_ALIGN: return "MXFP4_ERR_ALIGN: a pointer is not 16-byte aligned";
    case MXFP4_ERR_HIP: return "MXFP4_ERR_HIP: HIP runtime error";
    }
    return "unknown status";
}

}  // extern "C"

// ssd_conv1d_step.cu -- the causal depthwise conv1d over decode and speculative
// windows, from a read slot, with a write slot for every token.
//
//   y[t, c] = act(bias[c] + sum_k weight[c, k] xin[t - (W-1) + k, c])
//   state after token t = xin[t - (W-2) .. t]
//
// A thread owns one channel of one request and slides the window over its tokens.
#include "pdl.cuh"
#include "ssd_internal.cuh"

namespace ssd {
namespace {

constexpr int kCsThreads = 128;

struct ConvStepParams {
    int64_t T;
    int32_t R, D, num_slots, silu;
    const int32_t *cu;
    ssd_conv_io io;
};

template <typename T, int W>
__global__ void __launch_bounds__(kCsThreads) conv1d_step_kernel(const __grid_constant__ ConvStepParams p) {
    pdl_wait();
    const ssd_conv_io &io = p.io;
    const int i = blockIdx.y, c = blockIdx.x * kCsThreads + threadIdx.x;
    const int64_t a = p.cu[i], b = p.cu[i + 1];
    if (b < a || a < 0 || b > p.T || (i == 0 && a != 0) || (i == p.R - 1 && b != p.T)) {
        if (c == 0) atomicOr(io.device_err, SSD_DEVERR_CU_SEQLENS);
        return;
    }
    if (c >= p.D || a == b) return;
    const T *x = static_cast<const T *>(io.x) + c;
    T *pool = static_cast<T *>(io.conv_pool), *y = static_cast<T *>(io.y) + c;
    const size_t slot = (size_t)p.D * (W - 1), off = (size_t)c * (W - 1);
    const int rs = io.read_slots ? io.read_slots[i] : -1;
    if (rs >= p.num_slots && c == 0) atomicOr(io.device_err, SSD_DEVERR_INIT_SLOT);
    T win[W];
    float w[W];
#pragma unroll
    for (int k = 0; k < W; ++k) {
        w[k] = io.weight[(size_t)c * W + k];
        if (k < W - 1) win[k] = rs >= 0 && rs < p.num_slots ? pool[rs * slot + off + k] : from_f32<T>(0.f);
    }
    const float bias = io.bias ? io.bias[c] : 0.f;
    for (int64_t t = a; t < b; ++t) {
        win[W - 1] = x[(size_t)t * p.D];
        float v = bias;
#pragma unroll
        for (int k = 0; k < W; ++k) v = fmaf(w[k], to_f32(win[k]), v);
        y[(size_t)t * p.D] = from_f32<T>(p.silu ? silu_f32(v) : v);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) win[k] = win[k + 1];
        const int ws = io.write_slots ? io.write_slots[t] : -1;
        if (ws >= p.num_slots) {
            if (c == 0) atomicOr(io.device_err, SSD_DEVERR_FINAL_SLOT);
        } else if (ws >= 0) {
#pragma unroll
            for (int k = 0; k < W - 1; ++k) pool[ws * slot + off + k] = win[k];
        }
    }
}

template <typename T>
cudaError_t launch_cs(const ConvStepParams &p, int W, cudaStream_t stream) {
    const dim3 grid((unsigned)((p.D + kCsThreads - 1) / kCsThreads), (unsigned)p.R), block(kCsThreads);
    switch (W) {
        case 2: return launch_after_prev(conv1d_step_kernel<T, 2>, grid, block, 0, stream, p);
        case 3: return launch_after_prev(conv1d_step_kernel<T, 3>, grid, block, 0, stream, p);
        case 4: return launch_after_prev(conv1d_step_kernel<T, 4>, grid, block, 0, stream, p);
        default: return cudaErrorInvalidValue;
    }
}

bool aligned_to(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" int ssd_varlen_conv1d_step(const ssd_conv_dims *d, const int32_t *cu_seqlens, const ssd_conv_io *io,
                                      cudaStream_t stream) {
    if (!d || !cu_seqlens || !io) return SSD_ERR_NULL;
    if (d->T < 0 || d->T > 0x7fffffffLL || d->R < 1 || d->R > 65535 || d->D < 1 || d->D > (1 << 24) ||
        d->num_slots < 0)
        return SSD_ERR_DIMS;
    if (d->dtype != SSD_DTYPE_BF16 && d->dtype != SSD_DTYPE_F32) return SSD_ERR_DTYPE;
    if (d->W < 2 || d->W > 4) return SSD_ERR_UNSUPPORTED;
    if (!io->weight || !io->device_err) return SSD_ERR_NULL;
    if (d->T > 0 && (!io->x || !io->y)) return SSD_ERR_NULL;
    if ((io->read_slots || io->write_slots) && (!io->conv_pool || d->num_slots < 1)) return SSD_ERR_NULL;
    const uintptr_t e = d->dtype == SSD_DTYPE_BF16 ? 2 : 4;
    const void *vec[] = {io->x, io->y, io->conv_pool};
    for (const void *ptr : vec)
        if (!aligned_to(ptr, e)) return SSD_ERR_ALIGN;
    const void *words[] = {cu_seqlens, io->weight, io->bias, io->read_slots, io->write_slots, io->device_err};
    for (const void *ptr : words)
        if (!aligned_to(ptr, 4)) return SSD_ERR_ALIGN;
    ConvStepParams p{};
    p.T = d->T;
    p.R = d->R;
    p.D = d->D;
    p.num_slots = d->num_slots;
    p.silu = d->silu ? 1 : 0;
    p.cu = cu_seqlens;
    p.io = *io;
    const cudaError_t err =
        d->dtype == SSD_DTYPE_BF16 ? launch_cs<__nv_bfloat16>(p, d->W, stream) : launch_cs<float>(p, d->W, stream);
    return err == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

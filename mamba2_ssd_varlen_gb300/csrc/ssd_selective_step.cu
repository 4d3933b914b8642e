// ssd_selective_step.cu -- the selective scan over decode and speculative
// windows, from a read slot, with a write slot for every token.
//
// A warp owns one channel of one request: lane l holds the states l, l + 32, ...
#include "pdl.cuh"
#include "selective.cuh"

namespace ssd {
namespace {

constexpr int kStepThreads = 128;

struct SelStepParams {
    SelShape s;
    const int32_t *cu;
    ssd_selective_step_io io;
};

template <typename T, int NPL>
__global__ void __launch_bounds__(kStepThreads) selective_step_kernel(const __grid_constant__ SelStepParams p) {
    pdl_wait();
    const SelShape &s = p.s;
    const ssd_selective_step_io &io = p.io;
    const int lane = threadIdx.x & 31, i = blockIdx.y;
    const int d = blockIdx.x * (kStepThreads / 32) + (threadIdx.x >> 5);
    const int64_t a = p.cu[i], b = p.cu[i + 1];
    if (b < a || a < 0 || b > s.T || (i == 0 && a != 0) || (i == s.R - 1 && b != s.T)) {
        if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(io.device_err, SSD_DEVERR_CU_SEQLENS);
        return;
    }
    if (d >= s.D || a == b) return;
    const bool first = d == 0 && lane == 0;
    const size_t dn = (size_t)s.D * s.N, off = (size_t)d * s.N;
    float h[NPL], A[NPL];
    const int rs = io.read_slots[i];
    if (rs >= s.num_slots && first) atomicOr(io.device_err, SSD_DEVERR_INIT_SLOT);
    const float *src = rs >= 0 && rs < s.num_slots ? io.state_pool + (size_t)rs * dn + off : nullptr;
#pragma unroll
    for (int k = 0; k < NPL; ++k) {
        const int n = lane + 32 * k;
        A[k] = n < s.N ? io.A[off + n] : 0.f;
        h[k] = src && n < s.N ? src[n] : 0.f;
    }
    const int g = d / (s.D / s.G);
    const float bias = io.delta_bias ? io.delta_bias[d] : 0.f, skip = io.D ? io.D[d] : 0.f;
    const T *u = static_cast<const T *>(io.u) + d, *dl = static_cast<const T *>(io.delta) + d;
    const T *B = static_cast<const T *>(io.B) + (size_t)g * s.N, *C = static_cast<const T *>(io.C) + (size_t)g * s.N;
    const T *z = io.z ? static_cast<const T *>(io.z) + d : nullptr;
    T *y = static_cast<T *>(io.y) + d;
    for (int64_t t = a; t < b; ++t) {
        const float dt = sel_step(to_f32(dl[t * s.ds]) + bias, s.softplus), uv = to_f32(u[t * s.us]), du = dt * uv;
        float acc = 0.f;
#pragma unroll
        for (int k = 0; k < NPL; ++k) {
            const int n = lane + 32 * k;
            if (n < s.N) {
                h[k] = fmaf(expf(dt * A[k]), h[k], du * to_f32(B[t * s.bs + n]));
                acc = fmaf(to_f32(C[t * s.cs + n]), h[k], acc);
            }
        }
        for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
        if (lane == 0) {
            if (io.D) acc = fmaf(skip, uv, acc);
            if (z) acc *= silu_f32(to_f32(z[t * s.zs]));
            y[t * s.ys] = from_f32<T>(acc);
        }
        const int ws = io.write_slots ? io.write_slots[t] : -1;
        if (ws >= s.num_slots) {
            if (first) atomicOr(io.device_err, SSD_DEVERR_FINAL_SLOT);
        } else if (ws >= 0) {
            float *dst = io.state_pool + (size_t)ws * dn + off;
#pragma unroll
            for (int k = 0; k < NPL; ++k)
                if (lane + 32 * k < s.N) dst[lane + 32 * k] = h[k];
        }
    }
}

template <typename T>
cudaError_t launch_step(const SelStepParams &p, cudaStream_t stream) {
    const dim3 grid((unsigned)((p.s.D + kStepThreads / 32 - 1) / (kStepThreads / 32)), (unsigned)p.s.R);
    if (p.s.N <= 32) return launch_after_prev(selective_step_kernel<T, 1>, grid, dim3(kStepThreads), 0, stream, p);
    if (p.s.N <= 64) return launch_after_prev(selective_step_kernel<T, 2>, grid, dim3(kStepThreads), 0, stream, p);
    return launch_after_prev(selective_step_kernel<T, 8>, grid, dim3(kStepThreads), 0, stream, p);
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" int ssd_varlen_selective_step(const ssd_selective_dims *d, const int32_t *cu_seqlens,
                                         const ssd_selective_step_io *io, cudaStream_t stream) {
    if (!d || !cu_seqlens || !io) return SSD_ERR_NULL;
    SelStepParams p{};
    const int rc = sel_shape(d, io->z != nullptr, &p.s);
    if (rc != SSD_OK) return rc;
    if (d->num_slots < 1) return SSD_ERR_DIMS;
    if (!io->A || !io->state_pool || !io->read_slots || !io->device_err) return SSD_ERR_NULL;
    if (d->T > 0 && (!io->u || !io->delta || !io->B || !io->C || !io->y)) return SSD_ERR_NULL;
    const uintptr_t e = d->dtype == SSD_DTYPE_BF16 ? 2 : 4;
    const void *vec[] = {io->u, io->delta, io->B, io->C, io->z, io->y};
    for (const void *ptr : vec)
        if (!sel_aligned(ptr, e)) return SSD_ERR_ALIGN;
    const void *words[] = {cu_seqlens, io->delta_bias, io->A, io->D, io->state_pool, io->read_slots, io->write_slots,
                           io->device_err};
    for (const void *ptr : words)
        if (!sel_aligned(ptr, 4)) return SSD_ERR_ALIGN;
    p.cu = cu_seqlens;
    p.io = *io;
    const cudaError_t err =
        d->dtype == SSD_DTYPE_BF16 ? launch_step<__nv_bfloat16>(p, stream) : launch_step<float>(p, stream);
    return err == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

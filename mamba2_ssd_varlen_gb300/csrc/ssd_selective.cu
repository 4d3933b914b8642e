// ssd_selective.cu -- the selective-scan (S6) prefill.
//
//   dt' = softplus(delta[t,d] + bias[d])
//   h[d,n] <- exp(dt' A[d,n]) h[d,n] + dt' u[t,d] B[t,g,n]
//   y[t,d] = (sum_n C[t,g,n] h[d,n] + D[d] u[t,d]) silu(z[t,d])
//
// A warp owns one channel of one request and walks its tokens: lane l holds the
// states l, l + 32, ...; the sum over n is a shuffle reduction.
#include "pdl.cuh"
#include "selective.cuh"

namespace ssd {
namespace {

constexpr int kSelThreads = 128;

struct SelParams {
    SelShape s;
    const int32_t *cu;
    ssd_selective_io io;
};

template <typename T, int NPL>
__global__ void __launch_bounds__(kSelThreads) selective_kernel(const __grid_constant__ SelParams p) {
    pdl_wait();
    const SelShape &s = p.s;
    const ssd_selective_io &io = p.io;
    const int lane = threadIdx.x & 31, i = blockIdx.y;
    const int d = blockIdx.x * (kSelThreads / 32) + (threadIdx.x >> 5);
    const int64_t a = p.cu[i], b = p.cu[i + 1];
    if (b < a || a < 0 || b > s.T || (i == 0 && a != 0) || (i == s.R - 1 && b != s.T)) {
        if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(io.device_err, SSD_DEVERR_CU_SEQLENS);
        return;
    }
    if (d >= s.D) return;
    const bool first = d == 0 && lane == 0;
    int64_t done = 0;
    const bool blocks = io.block_table != nullptr;
    bool table_ok = blocks;
    if (blocks && io.num_computed) {
        done = io.num_computed[i];
        if (done < 0 || done + (b - a) > 0x7fffffffLL) {
            if (first) atomicOr(io.device_err, SSD_DEVERR_NUM_COMPUTED);
            table_ok = false;
            done = 0;
        }
    }
    const size_t dn = (size_t)s.D * s.N, off = (size_t)d * s.N;
    float h[NPL], A[NPL];
    const float *src = nullptr;
    if (io.init_slots) {
        const int slot = io.init_slots[i];
        if (slot >= s.num_slots) {
            if (first) atomicOr(io.device_err, SSD_DEVERR_INIT_SLOT);
        } else if (slot >= 0) {
            src = io.state_pool + (size_t)slot * dn + off;
        }
    }
#pragma unroll
    for (int k = 0; k < NPL; ++k) {
        const int n = lane + 32 * k;
        A[k] = n < s.N ? io.A[off + n] : 0.f;
        h[k] = src && n < s.N ? src[n] : 0.f;
    }
    auto put = [&](float *base) {
#pragma unroll
        for (int k = 0; k < NPL; ++k)
            if (lane + 32 * k < s.N) base[off + lane + 32 * k] = h[k];
    };
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
        if (table_ok) {
            const int64_t pos = done + (t - a) + 1;
            if (pos % s.block_size == 0) {
                const int64_t col = pos / s.block_size - 1;
                if (col >= s.bt_width) {
                    if (first) atomicOr(io.device_err, SSD_DEVERR_BLOCK_TABLE);
                } else {
                    const int slot = io.block_table[(size_t)i * s.bt_width + col];
                    if (slot >= s.num_slots) {
                        if (first) atomicOr(io.device_err, SSD_DEVERR_BLOCK_SLOT);
                    } else if (slot >= 0) {
                        put(io.state_pool + (size_t)slot * dn);
                    }
                }
            }
        }
    }
    if (io.final_states) put(io.final_states + (size_t)i * dn);
    if (io.final_slots) {
        const int slot = io.final_slots[i];
        if (slot >= s.num_slots) {
            if (first) atomicOr(io.device_err, SSD_DEVERR_FINAL_SLOT);
        } else if (slot >= 0) {
            put(io.state_pool + (size_t)slot * dn);
        }
    }
}

template <typename T>
cudaError_t launch(const SelParams &p, cudaStream_t stream) {
    const dim3 grid((unsigned)((p.s.D + kSelThreads / 32 - 1) / (kSelThreads / 32)), (unsigned)p.s.R);
    if (p.s.N <= 32) return launch_after_prev(selective_kernel<T, 1>, grid, dim3(kSelThreads), 0, stream, p);
    if (p.s.N <= 64) return launch_after_prev(selective_kernel<T, 2>, grid, dim3(kSelThreads), 0, stream, p);
    return launch_after_prev(selective_kernel<T, 8>, grid, dim3(kSelThreads), 0, stream, p);
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" size_t ssd_varlen_selective_scan_workspace(const ssd_selective_dims *d) {
    (void)d;
    return 0;
}

extern "C" int ssd_varlen_selective_scan(const ssd_selective_dims *d, const int32_t *cu_seqlens,
                                         const ssd_selective_io *io, cudaStream_t stream) {
    if (!d || !cu_seqlens || !io) return SSD_ERR_NULL;
    SelParams p{};
    const int rc = sel_shape(d, io->z != nullptr, &p.s);
    if (rc != SSD_OK) return rc;
    if (!io->A || !io->device_err) return SSD_ERR_NULL;
    if (d->T > 0 && (!io->u || !io->delta || !io->B || !io->C || !io->y)) return SSD_ERR_NULL;
    if ((io->init_slots || io->final_slots || io->block_table) && (!io->state_pool || d->num_slots < 1))
        return SSD_ERR_NULL;
    if (io->block_table && (d->block_size < 1 || d->block_size % 16 != 0)) return SSD_ERR_BLOCK_SIZE;
    const uintptr_t e = d->dtype == SSD_DTYPE_BF16 ? 2 : 4;
    const void *vec[] = {io->u, io->delta, io->B, io->C, io->z, io->y};
    for (const void *ptr : vec)
        if (!sel_aligned(ptr, e)) return SSD_ERR_ALIGN;
    const void *words[] = {cu_seqlens,      io->delta_bias, io->A,           io->D,          io->num_computed, io->state_pool,
                           io->init_slots, io->final_slots, io->block_table, io->final_states, io->device_err};
    for (const void *ptr : words)
        if (!sel_aligned(ptr, 4)) return SSD_ERR_ALIGN;
    const size_t need = ssd_varlen_selective_scan_workspace(d);
    if (need && (!io->workspace || io->workspace_bytes < need || !sel_aligned(io->workspace, 16)))
        return SSD_ERR_WORKSPACE;
    p.cu = cu_seqlens;
    p.io = *io;
    const cudaError_t err = d->dtype == SSD_DTYPE_BF16 ? launch<__nv_bfloat16>(p, stream) : launch<float>(p, stream);
    return err == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

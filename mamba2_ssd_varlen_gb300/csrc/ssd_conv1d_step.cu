// ssd_conv1d_step.cu -- the causal depthwise conv1d over decode and speculative
// windows, from a read slot, with a write slot for every token.
//
//   y[t, c] = act(bias[c] + sum_k weight[c, k] xin[t - (W-1) + k, c])
//   state after token t = xin[t - (W-2) .. t]
//
// Bound by memory and, at serving sizes, by the launch.  A thread owns four neighbouring
// channels (one where the width or a pointer is off their boundary): a slot's W-1 inputs a
// channel are then 4 (W-1) neighbouring elements, W-1 vectors, which move between their
// order in the slot (channel by channel) and the window (input by input, held in fp32,
// where every element is exact) by the naming of registers.  A CTA takes several requests,
// one after the other with the weights in registers, the next one's state on its way: as
// many as leave one wave.  Measured at D = 5120, W = 4, bf16: 256 windows of one token
// 5.2 us (one request a CTA: 9.1), of four 15.8 us (60 MB; 56 % of the copy rate); eight
// channels a thread take 126 to 157 registers, 6.3 and 16.8 us.
#include <algorithm>

#include "pdl.cuh"
#include "resident.cuh"
#include "special.cuh"
#include "ssd_internal.cuh"

namespace ssd {
namespace {

constexpr int kCsThreads = 128;

struct ConvStepParams {
    int64_t T;
    int32_t R, D, num_slots, silu, tiles, rb;
    const int32_t *cu;
    ssd_conv_io io;
};

// kN (1 or 4) neighbouring elements as they lie in memory, moved as one; in fp32 they are exact, so that the window can be
// held there and handed back bit for bit.
template <typename T, int kN>
struct Raw {
    static_assert(kN == 1, "one element");
    T v;
    __device__ __forceinline__ void load(const T *p) { v = *p; }
    __device__ __forceinline__ void widen(float *x) const { x[0] = to_f32(v); }
    __device__ __forceinline__ static void store(T *p, const float *x) { *p = from_f32<T>(x[0]); }
    __device__ __forceinline__ static void store_exact(T *p, const float *x) {  // a rounding would rewrite a NaN's payload
        if constexpr (sizeof(T) == 2)
            *p = __ushort_as_bfloat16((unsigned short)(__float_as_uint(x[0]) >> 16));
        else
            *p = x[0];
    }
};
template <>
struct Raw<float, 4> {
    float4 v;
    __device__ __forceinline__ void load(const float *p) { v = *reinterpret_cast<const float4 *>(p); }
    __device__ __forceinline__ void widen(float *x) const { x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w; }
    __device__ __forceinline__ static void store(float *p, const float *x) {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    }
    __device__ __forceinline__ static void store_exact(float *p, const float *x) { store(p, x); }
};
template <>
struct Raw<__nv_bfloat16, 4> {
    uint2 v;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { v = *reinterpret_cast<const uint2 *>(p); }
    __device__ __forceinline__ void widen(float *x) const {
        x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xFFFF0000u);
        x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xFFFF0000u);
    }
    __device__ __forceinline__ static void store(__nv_bfloat16 *p, const float *x) {  // rounded
        const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
        *reinterpret_cast<uint2 *>(p) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
    __device__ __forceinline__ static void store_exact(__nv_bfloat16 *p, const float *x) {  // widened values: their upper halves
        *reinterpret_cast<uint2 *>(p) = make_uint2(__byte_perm(__float_as_uint(x[0]), __float_as_uint(x[1]), 0x7632),
                                                   __byte_perm(__float_as_uint(x[2]), __float_as_uint(x[3]), 0x7632));
    }
};

template <typename T, int W, int kN>
__global__ void __launch_bounds__(kCsThreads, 6) conv1d_step_kernel(const __grid_constant__ ConvStepParams p) {
    pdl_wait();
    const ssd_conv_io &io = p.io;
    const int lane = threadIdx.x & 31;
    const int i0 = (int)(blockIdx.x / p.tiles) * p.rb, count = min(p.rb, p.R - i0);
    const int c = ((int)(blockIdx.x % p.tiles) * kCsThreads + (int)threadIdx.x) * kN;
    const bool there = c < p.D;
    float w[kN * W], bias[kN];
#pragma unroll
    for (int e = 0; e < kN; ++e) bias[e] = there && io.bias ? io.bias[c + e] : 0.f;
    if constexpr (kN == 4) {
#pragma unroll
        for (int e = 0; e < kN * W; e += 4)
            *reinterpret_cast<float4 *>(w + e) = there ? *reinterpret_cast<const float4 *>(io.weight + (size_t)c * W + e)
                                                       : make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
#pragma unroll
        for (int e = 0; e < kN * W; ++e) w[e] = there ? io.weight[(size_t)c * W + e] : 0.f;
    }
    // lane q: the window and the read slot of request i0 + q
    int ma = 0, mb = 0, ms = -1;
    if (lane < count) {
        const int i = i0 + lane;
        ma = p.cu[i], mb = p.cu[i + 1];
        if (mb < ma || ma < 0 || mb > p.T || (i == 0 && ma != 0) || (i == p.R - 1 && mb != p.T)) {
            if (blockIdx.x % p.tiles == 0) atomicOr(io.device_err, SSD_DEVERR_CU_SEQLENS);
            ma = mb = 0;
        }
        if (mb > ma && io.read_slots) ms = io.read_slots[i];
        if (ms >= p.num_slots) {
            if (blockIdx.x % p.tiles == 0) atomicOr(io.device_err, SSD_DEVERR_INIT_SLOT);
            ms = -1;
        }
    }
    const T *x = static_cast<const T *>(io.x) + c;
    T *pool = static_cast<T *>(io.conv_pool), *y = static_cast<T *>(io.y) + c;
    const size_t slot = (size_t)p.D * (W - 1), off = (size_t)c * (W - 1);
    Raw<T, kN> state[W - 1], in;  // the slot's order: element e (W-1) + k is input k of channel e
    auto fetch = [&](int q) {     // the state and the first input of request i0 + q
        const int rs = __shfl_sync(0xffffffffu, ms, q), a = __shfl_sync(0xffffffffu, ma, q);
        const int b = __shfl_sync(0xffffffffu, mb, q);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            state[k] = {};
            if (rs >= 0 && there) state[k].load(pool + rs * slot + off + k * kN);
        }
        if (b > a && there) in.load(x + (size_t)a * p.D);
    };
    fetch(0);
    for (int q = 0; q < count; ++q) {
        const int a = __shfl_sync(0xffffffffu, ma, q), b = __shfl_sync(0xffffffffu, mb, q);
        float win[W][kN], flat[(W - 1) * kN];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) state[k].widen(flat + k * kN);
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
#pragma unroll
            for (int e = 0; e < kN; ++e) win[k][e] = flat[e * (W - 1) + k];
        in.widen(win[W - 1]);
        if (q + 1 < count) fetch(q + 1);  // on its way while this window is computed
        for (int t = a; t < b; ++t) {
            const int ws = io.write_slots ? io.write_slots[t] : -1;
            Raw<T, kN> ahead = {};
            if (t + 1 < b && there) ahead.load(x + (size_t)(t + 1) * p.D);
            float out[kN];
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                float v = bias[e];
#pragma unroll
                for (int k = 0; k < W; ++k) v = fmaf(w[e * W + k], win[k][e], v);
                out[e] = p.silu ? silu_sfu(v) : v;
            }
            if (there) Raw<T, kN>::store(y + (size_t)t * p.D, out);
            if (ws >= p.num_slots) {
                if (c == 0) atomicOr(io.device_err, SSD_DEVERR_FINAL_SLOT);
            } else if (ws >= 0 && there) {
#pragma unroll
                for (int i = 0; i < (W - 1) * kN; ++i) flat[i] = win[i % (W - 1) + 1][i / (W - 1)];
#pragma unroll
                for (int k = 0; k < W - 1; ++k)
                    Raw<T, kN>::store_exact(pool + ws * slot + off + k * kN, flat + k * kN);
            }
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
#pragma unroll
                for (int e = 0; e < kN; ++e) win[k][e] = win[k + 1][e];
            ahead.widen(win[W - 1]);
        }
    }
}

template <typename T, int W, int kN>
cudaError_t launch_cs_n(ConvStepParams &p, cudaStream_t stream) {
    constexpr auto kernel = conv1d_step_kernel<T, W, kN>;
    static int64_t cached[kResidentDevices] = {};
    int64_t resident = 0;
    const cudaError_t e = resident_ctas_at(cached, kernel, kCsThreads, 0, resident);
    if (e != cudaSuccess) return e;
    p.tiles = (p.D + kCsThreads * kN - 1) / (kCsThreads * kN);
    p.rb = (int)runs_of((int64_t)p.tiles * p.R, resident, 32);  // requests a CTA, with the weights in registers
    const int64_t ctas = (int64_t)p.tiles * ((p.R + p.rb - 1) / p.rb);
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_after_prev(kernel, dim3((unsigned)ctas), dim3(kCsThreads), 0, stream, p);
}

template <typename T, int W>
cudaError_t launch_cs_w(ConvStepParams &p, bool vec, cudaStream_t stream) {
    return vec ? launch_cs_n<T, W, 4>(p, stream) : launch_cs_n<T, W, 1>(p, stream);
}

bool aligned_to(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

template <typename T>
cudaError_t launch_cs(ConvStepParams &p, int W, cudaStream_t stream) {
    const bool vec = p.D % 4 == 0 && aligned_to(p.io.x, 4 * sizeof(T)) && aligned_to(p.io.y, 4 * sizeof(T)) &&
                     aligned_to(p.io.conv_pool, 4 * sizeof(T)) && aligned_to(p.io.weight, 16);
    switch (W) {
        case 2: return launch_cs_w<T, 2>(p, vec, stream);
        case 3: return launch_cs_w<T, 3>(p, vec, stream);
        case 4: return launch_cs_w<T, 4>(p, vec, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" int ssd_varlen_conv1d_step(const ssd_conv_dims *d, const int32_t *cu_seqlens, const ssd_conv_io *io,
                                      cudaStream_t stream) {
    if (!d || !cu_seqlens || !io) return SSD_ERR_NULL;
    if (d->T < 0 || d->T > 0x7fffffffLL || d->R < 1 || d->D < 1 || d->D > (1 << 24) ||
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

// ssd_selective_step.cu -- the selective scan over decode and speculative
// windows, from a read slot, with a write slot for every token.
//
// Bound by the states: N fp32 values a channel read once a window and written once a
// token.  QL lanes hold a channel, four neighbouring states each (one 16-byte access, the
// lanes of a channel a whole run of sectors), and CPG channels a lane group, so that a lane
// has CPG independent 16-byte loads in flight; each lane computes the step and the gate of
// one of its group's channels and hands them round by shuffles.  Rows of u, delta, z and y
// are read and written 32 neighbouring channels at a time.
#include "pdl.cuh"
#include "selective.cuh"
#include "special.cuh"

namespace ssd {
namespace {

constexpr int kStepThreads = 128;

struct SelStepParams {
    SelShape s;
    const int32_t *cu;
    ssd_selective_step_io io;
    int32_t vec;     // states: every four start on a 16-byte boundary
    int32_t bc_vec;  // B, C: every four start on a boundary of four elements
};

__device__ __forceinline__ float4 four(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 four(const __nv_bfloat16 *p) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xFFFF0000u));
}

// n of four neighbouring elements, zeros for the rest.
template <typename T>
__device__ __forceinline__ float4 some(const T *p, int n) {
    return make_float4(n > 0 ? to_f32(p[0]) : 0.f, n > 1 ? to_f32(p[1]) : 0.f, n > 2 ? to_f32(p[2]) : 0.f,
                       n > 3 ? to_f32(p[3]) : 0.f);
}

// QL lanes a channel with 4 NV states each (quad v of a lane: states 4 (l + QL v) ..), CPG channels a lane group.
template <typename T, int QL, int NV>
__global__ void __launch_bounds__(kStepThreads) selective_step_kernel(const __grid_constant__ SelStepParams p) {
    constexpr int GR = 32 / QL;               // lane groups of a warp
    constexpr int CPG = QL < 4 ? QL : 4;      // channels of a group
    constexpr int CW = GR * CPG;              // channels of a warp
    pdl_wait();
    const SelShape &s = p.s;
    const ssd_selective_step_io &io = p.io;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % QL, gr = lane / QL;
    const int tiles = (s.D / s.G + CW - 1) / CW * s.G;  // of CW channels, none over two groups of B and C
    const int64_t item = (int64_t)blockIdx.x * (kStepThreads / 32) + warp;
    if (item >= (int64_t)tiles * s.R) return;
    const int i = (int)(item / tiles), tile = (int)(item % tiles);
    const int dg = s.D / s.G, per_group = tiles / s.G, g = tile / per_group;
    const int d0 = g * dg + tile % per_group * CW, width = min(CW, (g + 1) * dg - d0);
    const bool first = tile == 0 && lane == 0;
    const int64_t a = p.cu[i], b = p.cu[i + 1];
    if (b < a || a < 0 || b > s.T || (i == 0 && a != 0) || (i == s.R - 1 && b != s.T)) {
        if (first) atomicOr(io.device_err, SSD_DEVERR_CU_SEQLENS);
        return;
    }
    if (a == b) return;
    const int rs = io.read_slots[i];
    if (rs >= s.num_slots && first) atomicOr(io.device_err, SSD_DEVERR_INIT_SLOT);
    const size_t dn = (size_t)s.D * s.N;
    const float *src = rs >= 0 && rs < s.num_slots ? io.state_pool + (size_t)rs * dn : nullptr;

    // channel k of the group: gr + GR k, so that a warp's access covers neighbouring channels
    float4 h[CPG][NV], A[CPG][NV];
#pragma unroll
    for (int k = 0; k < CPG; ++k) {
        const int ch = gr + GR * k;
        const size_t row = (size_t)(d0 + ch) * s.N;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int n0 = 4 * (l + QL * v), n = ch < width ? min(4, s.N - n0) : 0;
            const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p.vec) {
                h[k][v] = src && n > 0 ? four(src + row + n0) : zero;
                A[k][v] = n > 0 ? four(io.A + row + n0) : zero;
            } else {
                h[k][v] = src ? some(src + row + n0, n) : zero;
                A[k][v] = some(io.A + row + n0, n);
            }
        }
    }
    // the lane's own channel (lanes past CPG have none)
    const int own = gr + GR * l, d = d0 + own;
    const bool mine = l < CPG && own < width;
    const float bias = mine && io.delta_bias ? io.delta_bias[d] : 0.f, skip = mine && io.D ? io.D[d] : 0.f;
    const T *u = static_cast<const T *>(io.u) + d, *dl = static_cast<const T *>(io.delta) + d;
    const T *z = io.z ? static_cast<const T *>(io.z) + d : nullptr;
    const T *B = static_cast<const T *>(io.B) + (size_t)g * s.N, *C = static_cast<const T *>(io.C) + (size_t)g * s.N;
    T *y = static_cast<T *>(io.y) + d;
#pragma unroll
    for (int k = 0; k < CPG; ++k)
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            A[k][v].x *= kLog2e;
            A[k][v].y *= kLog2e;
            A[k][v].z *= kLog2e;
            A[k][v].w *= kLog2e;
        }
    // the next token's inputs are fetched while this one's states move
    float un = 0.f, dn1 = 0.f, zn = 0.f;
    float4 bn[NV], cn[NV];
    auto fetch = [&](int64_t t) {
        if (mine) {
            un = to_f32(u[t * s.us]);
            dn1 = to_f32(dl[t * s.ds]);
            if (z) zn = to_f32(z[t * s.zs]);
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int n0 = 4 * (l + QL * v), n = min(4, s.N - n0);
            const T *tb = B + t * s.bs + n0, *tc = C + t * s.cs + n0;
            if (p.bc_vec && n > 0) {
                bn[v] = four(tb);
                cn[v] = four(tc);
            } else {
                bn[v] = some(tb, n);
                cn[v] = some(tc, n);
            }
        }
    };
    fetch(a);
    for (int64_t t = a; t < b; ++t) {
        const float uv = un, zv = zn;
        float dt = dn1 + bias;
        if (s.softplus) {
            const float e = softplus_exp(dt);
            dt = softplus_end(dt, e, rcpf(e + 2.f));
        }
        const float du = dt * uv;
        float4 bv[NV], cv[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) bv[v] = bn[v], cv[v] = cn[v];
        const int ws = io.write_slots ? io.write_slots[t] : -1;
        if (t + 1 < b) fetch(t + 1);
        float acc[CPG];
#pragma unroll
        for (int k = 0; k < CPG; ++k) {
            const float dk = __shfl_sync(0xffffffffu, dt, gr * QL + k), uk = __shfl_sync(0xffffffffu, du, gr * QL + k);
            acc[k] = 0.f;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float4 &x = h[k][v];
                x.x = fmaf(ex2f(dk * A[k][v].x), x.x, uk * bv[v].x);
                x.y = fmaf(ex2f(dk * A[k][v].y), x.y, uk * bv[v].y);
                x.z = fmaf(ex2f(dk * A[k][v].z), x.z, uk * bv[v].z);
                x.w = fmaf(ex2f(dk * A[k][v].w), x.w, uk * bv[v].w);
                acc[k] = fmaf(x.x, cv[v].x, acc[k]);
                acc[k] = fmaf(x.y, cv[v].y, acc[k]);
                acc[k] = fmaf(x.z, cv[v].z, acc[k]);
                acc[k] = fmaf(x.w, cv[v].w, acc[k]);
            }
        }
        if (ws >= s.num_slots) {
            if (first) atomicOr(io.device_err, SSD_DEVERR_FINAL_SLOT);
        } else if (ws >= 0) {
#pragma unroll
            for (int k = 0; k < CPG; ++k) {
                const int ch = gr + GR * k;
                float *dst = io.state_pool + (size_t)ws * dn + (size_t)(d0 + ch) * s.N;
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const int n0 = 4 * (l + QL * v), n = ch < width ? min(4, s.N - n0) : 0;
                    const float4 x = h[k][v];
                    if (p.vec) {
                        if (n > 0) *reinterpret_cast<float4 *>(dst + n0) = x;
                    } else {
                        if (n > 0) dst[n0] = x.x;
                        if (n > 1) dst[n0 + 1] = x.y;
                        if (n > 2) dst[n0 + 2] = x.z;
                        if (n > 3) dst[n0 + 3] = x.w;
                    }
                }
            }
        }
        // sums over the QL lanes of a channel; lane k < CPG is left with channel k's
#pragma unroll
        for (int k = 0; k < CPG; ++k)
#pragma unroll
            for (int o = QL / 2; o >= CPG; o >>= 1) acc[k] += __shfl_xor_sync(0xffffffffu, acc[k], o);
#pragma unroll
        for (int o = CPG / 2; o >= 1; o >>= 1) {
            const bool up = (l & o) != 0;
#pragma unroll
            for (int k = 0; k < o; ++k) {
                const float lo = acc[k], hi = acc[k + o];
                acc[k] = (up ? hi : lo) + __shfl_xor_sync(0xffffffffu, up ? lo : hi, o);
            }
        }
        if (mine) {
            float v = fmaf(skip, uv, acc[0]);
            if (z) v *= silu_sfu(zv);
            y[t * s.ys] = from_f32<T>(v);
        }
    }
}

template <typename T, int QL, int NV>
cudaError_t launch_step_k(const SelStepParams &p, cudaStream_t stream) {
    constexpr int CW = 32 / QL * (QL < 4 ? QL : 4), kWarps = kStepThreads / 32;
    const int64_t items = (int64_t)((p.s.D / p.s.G + CW - 1) / CW) * p.s.G * p.s.R;
    if (items > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_after_prev(selective_step_kernel<T, QL, NV>, dim3((unsigned)((items + kWarps - 1) / kWarps)),
                             dim3(kStepThreads), 0, stream, p);
}

// Lanes a channel: enough for its states at four a lane.
template <typename T>
cudaError_t launch_step(const SelStepParams &p, cudaStream_t stream) {
    if (p.s.N <= 4) return launch_step_k<T, 1, 1>(p, stream);
    if (p.s.N <= 8) return launch_step_k<T, 2, 1>(p, stream);
    if (p.s.N <= 16) return launch_step_k<T, 4, 1>(p, stream);
    if (p.s.N <= 32) return launch_step_k<T, 8, 1>(p, stream);
    if (p.s.N <= 64) return launch_step_k<T, 16, 1>(p, stream);
    if (p.s.N <= 128) return launch_step_k<T, 32, 1>(p, stream);
    return launch_step_k<T, 32, 2>(p, stream);
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
    p.vec = d->N % 4 == 0 && sel_aligned(io->state_pool, 16) && sel_aligned(io->A, 16);
    auto fours = [&](const void *ptr, int64_t stride) {
        return sel_aligned(ptr, 4 * e) && stride % 4 == 0 && d->N % 4 == 0;
    };
    p.bc_vec = fours(io->B, p.s.bs) && fours(io->C, p.s.cs);
    const cudaError_t err =
        d->dtype == SSD_DTYPE_BF16 ? launch_step<__nv_bfloat16>(p, stream) : launch_step<float>(p, stream);
    return err == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

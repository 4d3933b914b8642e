// ssd_verify.cu -- verification of drafted tokens against the target's
// probabilities from given random numbers (speculative sampling).
//
// One CTA per window.  Thread 0 counts the accepted drafts; the CTA then draws
// the token that follows from one row's weights, held as whole multiples of
// 2^-40 so that their sums do not depend on the order: each thread sums a run of
// consecutive vocabulary entries, a scan over the threads finds the run that
// holds the mark, and its thread walks that run.
#include "pdl.cuh"
#include "ssd_internal.cuh"

namespace ssd {
namespace {

constexpr int kVerThreads = 256;

struct VerifyParams {
    int64_t T, ts, qs;
    int32_t R, V;
    const int32_t *cu;
    ssd_verify_io io;
};

// floor(2^40 min(max(w, 0), 1)), 0 for a NaN.  2^40 w is exact in fp32.
__device__ __forceinline__ uint64_t fixed_weight(float w) {
    return w > 0.f ? (uint64_t)__float2ull_rz(fminf(w, 1.f) * 1099511627776.f) : 0ull;
}

template <typename T>
__global__ void __launch_bounds__(kVerThreads) verify_kernel(const __grid_constant__ VerifyParams p) {
    pdl_wait();
    const ssd_verify_io &io = p.io;
    const int i = blockIdx.x, tid = threadIdx.x;
    const int64_t a = p.cu[i], b = p.cu[i + 1];
    if (b < a || a < 0 || b > p.T || (i == 0 && a != 0) || (i == p.R - 1 && b != p.T)) {
        if (tid == 0) atomicOr(io.device_err, SSD_DEVERR_CU_SEQLENS);
        return;
    }
    if (a == b) {
        if (tid == 0) io.accepted[i] = -1;
        return;
    }
    __shared__ int s_n, s_pick;
    __shared__ unsigned long long part[kVerThreads + 1];
    const T *P = static_cast<const T *>(io.target), *Q = static_cast<const T *>(io.draft);
    const int k = (int)(b - a - 1);
    if (tid == 0) {
        int n = 0;
        for (; n < k; ++n) {
            const int64_t t = a + n;
            const int x = io.tokens[t + 1];
            if (x < 0 || x >= p.V) {
                atomicOr(io.device_err, SSD_DEVERR_TOKEN);
                break;
            }
            const float q = Q ? to_f32(Q[t * p.qs + x]) : 1.f;
            if (!(io.accept_u[t + 1] * q < to_f32(P[t * p.ts + x]))) break;
        }
        s_n = n;
        s_pick = -1;
    }
    __syncthreads();
    const int n = s_n;
    const int64_t r = a + n;
    const T *pr = P + r * p.ts;
    bool residual = n < k;
    const int drafted = residual ? io.tokens[r + 1] : -1;
    auto weight = [&](int v) -> uint64_t {
        float w = to_f32(pr[v]);
        if (residual) {
            if (Q) w -= to_f32(Q[r * p.qs + v]);
            else if (v == drafted) w -= 1.f;
        }
        return fixed_weight(w);
    };
    const int run = (p.V + kVerThreads - 1) / kVerThreads;
    const int lo = min(tid * run, p.V), hi = min(lo + run, p.V);
    unsigned long long total = 0;
    for (;;) {
        uint64_t sum = 0;
        for (int v = lo; v < hi; ++v) sum += weight(v);
        part[tid + 1] = sum;
        if (tid == 0) part[0] = 0;
        __syncthreads();
        if (tid == 0)
            for (int j = 1; j <= kVerThreads; ++j) part[j] += part[j - 1];
        __syncthreads();
        total = part[kVerThreads];
        if (total != 0 || !residual) break;
        residual = false;  // no weight is positive after a rejection: the target's own
        __syncthreads();
    }
    if (total != 0) {
        const double f = (double)io.sample_u[i] * (double)total;
        unsigned long long mark = f >= 1.0 ? (unsigned long long)f : 0ull;  // also for a NaN
        mark = min(mark, total - 1);
        if (part[tid] <= mark && mark < part[tid + 1]) {
            unsigned long long c = part[tid];
            int v = lo;
            for (;; ++v) {
                c += weight(v);
                if (c > mark) break;
            }
            s_pick = v;
        }
    }
    __syncthreads();
    for (int j = tid; j < b - a; j += kVerThreads)
        io.out_tokens[a + j] = j < n ? io.tokens[a + j + 1] : j == n ? s_pick : -1;
    if (tid == 0) {
        io.accepted[i] = n;
        if (io.next_slots) io.next_slots[i] = io.write_slots[r];
    }
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" int ssd_varlen_verify(const ssd_verify_dims *d, const int32_t *cu_seqlens, const ssd_verify_io *io,
                                 cudaStream_t stream) {
    if (!d || !cu_seqlens || !io) return SSD_ERR_NULL;
    if (d->reserved != 0 || d->T < 0 || d->T > 0x7fffffffLL || d->R < 1 || d->R > 0x7ffffff || d->V < 1 ||
        d->V > (1 << 22))
        return SSD_ERR_DIMS;
    if (d->dtype != SSD_DTYPE_BF16 && d->dtype != SSD_DTYPE_F32) return SSD_ERR_DTYPE;
    const int64_t ts = d->target_stride ? d->target_stride : d->V, qs = d->draft_stride ? d->draft_stride : d->V;
    if (ts < d->V || ts > (1LL << 31) || (io->draft && (qs < d->V || qs > (1LL << 31)))) return SSD_ERR_DIMS;
    if (!io->accepted || !io->device_err) return SSD_ERR_NULL;
    if (d->T > 0 && (!io->target || !io->tokens || !io->accept_u || !io->sample_u || !io->out_tokens))
        return SSD_ERR_NULL;
    if (d->T > 0 && (io->write_slots != nullptr) != (io->next_slots != nullptr)) return SSD_ERR_NULL;
    const uintptr_t e = d->dtype == SSD_DTYPE_BF16 ? 2 : 4;
    auto ok = [](const void *ptr, uintptr_t al) { return ((uintptr_t)ptr & (al - 1)) == 0; };
    if (!ok(io->target, e) || !ok(io->draft, e)) return SSD_ERR_ALIGN;
    const void *words[] = {cu_seqlens,      io->tokens,     io->accept_u,   io->sample_u,  io->write_slots,
                           io->accepted, io->out_tokens, io->next_slots, io->device_err};
    for (const void *ptr : words)
        if (!ok(ptr, 4)) return SSD_ERR_ALIGN;
    VerifyParams p{};
    p.T = d->T;
    p.R = d->R;
    p.V = d->V;
    p.ts = ts;
    p.qs = qs;
    p.cu = cu_seqlens;
    p.io = *io;
    const dim3 grid((unsigned)d->R), block(kVerThreads);
    const cudaError_t err = d->dtype == SSD_DTYPE_BF16
                                ? launch_after_prev(verify_kernel<__nv_bfloat16>, grid, block, 0, stream, p)
                                : launch_after_prev(verify_kernel<float>, grid, block, 0, stream, p);
    return err == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

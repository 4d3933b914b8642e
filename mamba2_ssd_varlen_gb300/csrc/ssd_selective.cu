// ssd_selective.cu -- the selective-scan (S6) prefill.
//
//   dt' = softplus(delta[t,d] + bias[d])
//   h[d,n] <- exp(dt' A[d,n]) h[d,n] + dt' u[t,d] B[t,g,n]
//   y[t,d] = (sum_n C[t,g,n] h[d,n] + D[d] u[t,d]) silu(z[t,d])
//
// Every (token, channel, state) costs an exponential and four fp32 operations on the
// general pipe (two products, two multiply-adds); no part of it is a matrix product,
// because the decay differs for every channel and state.  The kernel is bound by
// instruction issue and those pipes, not by memory, so its shape is chosen to spend as
// few other instructions as possible:
//   - a CTA walks the tokens of one request for 32 channels of one group, L lanes a
//     channel, each with NP / L states in registers as packed fp32 pairs (two
//     multiply-adds an issue slot);
//   - u, delta, z and the rows of B and C arrive by tiles of 16 tokens through
//     asynchronous copies, a tile ahead; B and C are widened to fp32 once a tile;
//   - softplus, u dt', the skip term and the gate are computed by the L lanes of a channel
//     for different tokens, two at a time in packed pairs, and exchanged by shuffles.
#include "f32x2.cuh"
#include "pdl.cuh"
#include "selective.cuh"

namespace ssd {
namespace {

constexpr int kTile = 16;  // tokens staged at a time
constexpr int kCh = 32;    // channels of a CTA

struct SelParams {
    SelShape s;
    const int32_t *cu;
    ssd_selective_io io;
    int32_t tiles;   // channel tiles of a request: G * ceil((D / G) / 32)
    int32_t vec;     // u, delta, z: every tile row of a CTA starts on a 16-byte boundary
    int32_t bc_vec;  // B, C: every row does, and is whole 16-byte vectors
};

__device__ __forceinline__ void cp16(void *smem, const void *gmem) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(gmem)
                 : "memory");
}
__device__ __forceinline__ void cp4(void *smem, const void *gmem) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(gmem)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

template <typename T>
__device__ __forceinline__ void cp_elem(T *smem, const T *gmem) {
    if constexpr (sizeof(T) == 4) cp4(smem, gmem);
    else *smem = *gmem;  // two bytes: no asynchronous copy is that small
}

// Shared memory of a CTA.
template <typename T, int NP>
struct Smem {
    T raw[2][3][kTile][kCh];             // u, delta, z of two tiles
    T bc[2][2][kTile][NP];               // B and C as they come
    float f[2][kTile][NP];               // B and C of the tile at hand, fp32, zeros past N and past the tile
};

template <int L>
__device__ __forceinline__ void cta_sync() {
    if constexpr (L == 1) __syncwarp();
    else __syncthreads();
}

// L lanes a channel; lane = l * CW + c in a warp of CW = 32 / L channels.
template <typename T, int NP, int L>
__global__ void __launch_bounds__(kCh * L) selective_kernel(const __grid_constant__ SelParams p) {
    constexpr int NS = NP / L;               // states of a lane
    constexpr int NK = NS / 2;               // as packed pairs
    constexpr int CW = 32 / L;               // channels of a warp
    constexpr int OWN = L == 1 ? 4 : 2;      // tokens of a block whose step and gate a lane computes
    constexpr int TB = OWN * L;              // tokens of a block
    constexpr int THREADS = kCh * L;
    static_assert(NS >= 2 && kTile % TB == 0, "pairs of states, whole blocks");
    extern __shared__ __align__(16) uint8_t sel_smem[];
    Smem<T, NP> &sm = *reinterpret_cast<Smem<T, NP> *>(sel_smem);
    pdl_wait();
    const SelShape &s = p.s;
    const ssd_selective_io &io = p.io;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int l = lane / CW, c = warp * CW + lane % CW;  // this lane's share of the states, its channel in the tile
    const int i = (int)(blockIdx.x / p.tiles), tile = (int)(blockIdx.x % p.tiles);
    const int dg = s.D / s.G, per_group = p.tiles / s.G;
    const int g = tile / per_group, off = (tile % per_group) * kCh;
    const int width = min(kCh, dg - off);    // channels of this CTA
    const int d0 = g * dg + off, d = d0 + c;
    const bool mine = c < width;
    const bool first = tile == 0 && tid == 0;

    const int64_t a = p.cu[i], b = p.cu[i + 1];
    if (b < a || a < 0 || b > s.T || (i == 0 && a != 0) || (i == s.R - 1 && b != s.T)) {
        if (first) atomicOr(io.device_err, SSD_DEVERR_CU_SEQLENS);
        return;
    }
    const int len = (int)(b - a);
    int done = 0;
    bool table = io.block_table != nullptr;
    if (table && io.num_computed) {
        done = io.num_computed[i];
        if (done < 0 || (int64_t)done + len > 0x7fffffffLL) {
            if (first) atomicOr(io.device_err, SSD_DEVERR_NUM_COMPUTED);
            table = false;
            done = 0;
        }
    }

    const T *gu = static_cast<const T *>(io.u) + a * s.us + d0, *gd = static_cast<const T *>(io.delta) + a * s.ds + d0;
    const T *gz = io.z ? static_cast<const T *>(io.z) + a * s.zs + d0 : nullptr;
    const T *gb = static_cast<const T *>(io.B) + a * s.bs + (size_t)g * s.N;
    const T *gc = static_cast<const T *>(io.C) + a * s.cs + (size_t)g * s.N;
    T *gy = static_cast<T *>(io.y) + a * s.ys + d;

    // Tiles end at absolute multiples of kTile where block states are kept, so that a boundary ends its tile.
    const int lead = table ? done % kTile : 0;
    auto tile_begin = [&](int k) { return k == 0 ? 0 : k * kTile - lead; };
    auto stage = [&](int k) {  // asynchronous copies of tile k
        const int t0 = tile_begin(k), n = min(len, (k + 1) * kTile - lead) - t0, st = k & 1;
        constexpr int E = 16 / sizeof(T);    // elements of a vector
        if (p.vec) {
            constexpr int V = kCh / E;       // vectors of a row
            for (int q = tid; q < n * V; q += THREADS) {
                const int r = q / V, col = q % V * E;
                if (col >= width) continue;
                const size_t t = t0 + r;
                cp16(&sm.raw[st][0][r][col], gu + t * s.us + col);
                cp16(&sm.raw[st][1][r][col], gd + t * s.ds + col);
                if (gz) cp16(&sm.raw[st][2][r][col], gz + t * s.zs + col);
            }
        } else {
            for (int q = tid; q < n * kCh; q += THREADS) {
                const int r = q / kCh, col = q % kCh;
                if (col >= width) continue;
                const size_t t = t0 + r;
                cp_elem(&sm.raw[st][0][r][col], gu + t * s.us + col);
                cp_elem(&sm.raw[st][1][r][col], gd + t * s.ds + col);
                if (gz) cp_elem(&sm.raw[st][2][r][col], gz + t * s.zs + col);
            }
        }
        if (p.bc_vec) {
            const int V = s.N / E;
            for (int q = tid; q < n * V; q += THREADS) {
                const int r = q / V, col = q % V * E;
                cp16(&sm.bc[st][0][r][col], gb + (size_t)(t0 + r) * s.bs + col);
                cp16(&sm.bc[st][1][r][col], gc + (size_t)(t0 + r) * s.cs + col);
            }
        } else {
            for (int q = tid; q < n * s.N; q += THREADS) {
                const int r = q / s.N, col = q % s.N;
                cp_elem(&sm.bc[st][0][r][col], gb + (size_t)(t0 + r) * s.bs + col);
                cp_elem(&sm.bc[st][1][r][col], gc + (size_t)(t0 + r) * s.cs + col);
            }
        }
        cp_commit();
    };

    // The lane's states and decay rates (zeros past N and past the width: they stay zero).
    const size_t dn = (size_t)s.D * s.N, row = (size_t)d * s.N;
    const int n0 = l * NS;
    f2 h[NK], A[NK];
    {
        const float *src = nullptr;
        if (io.init_slots) {
            const int slot = io.init_slots[i];
            if (slot >= s.num_slots) {
                if (first) atomicOr(io.device_err, SSD_DEVERR_INIT_SLOT);
            } else if (slot >= 0) {
                src = io.state_pool + (size_t)slot * dn + row;
            }
        }
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            float hv[2], av[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int n = n0 + 2 * k + e;
                const bool ok = mine && n < s.N;
                hv[e] = ok && src ? src[n] : 0.f;
                av[e] = ok ? io.A[row + n] * kLog2e : 0.f;
            }
            h[k] = pk(hv[0], hv[1]);
            A[k] = pk(av[0], av[1]);
        }
    }
    const float bias = mine && io.delta_bias ? io.delta_bias[d] : 0.f, skip = mine && io.D ? io.D[d] : 0.f;
    auto put = [&](float *base) {
        if (!mine) return;
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            const float2 v = upk(h[k]);
            const int n = n0 + 2 * k;
            if (n < s.N) base[row + n] = v.x;
            if (n + 1 < s.N) base[row + n + 1] = v.y;
        }
    };

    const int tiles = (lead + len + kTile - 1) / kTile;
    if (len > 0) stage(0);
    for (int k = 0; k < tiles && len > 0; ++k) {
        const int t0 = tile_begin(k), n = min(len, (k + 1) * kTile - lead) - t0, st = k & 1;
        cp_wait_all();
        cta_sync<L>();  // tile k has landed; everybody is done with the buffers of tile k - 1
        if (k + 1 < tiles) stage(k + 1);
        for (int q = tid; q < 2 * kTile * NP; q += THREADS) {
            const int r = q / NP % kTile, col = q % NP;
            sm.f[q / (NP * kTile)][r][col] = r < n && col < s.N ? to_f32(sm.bc[st][q / (NP * kTile)][r][col]) : 0.f;
        }
        cta_sync<L>();
#pragma unroll 1
        for (int j0 = 0; j0 < n; j0 += TB) {
            // the steps of the lane's own tokens; zero past the tile, where they change nothing
            f2 dt[OWN / 2], du[OWN / 2], uv[OWN / 2];
#pragma unroll
            for (int q = 0; q < OWN / 2; ++q) {
                const int r = j0 + l * OWN + 2 * q;
                const bool v0 = r < n, v1 = r + 1 < n;
                uv[q] = pk(to_f32(sm.raw[st][0][r][c]), to_f32(sm.raw[st][0][r + 1][c]));
                f2 v = add2(pk(to_f32(sm.raw[st][1][r][c]), to_f32(sm.raw[st][1][r + 1][c])), dup2(bias));
                if (s.softplus) v = softplus2(v);
                const float2 x = upk(v), m = upk(mul2(v, uv[q]));
                dt[q] = pk(v0 ? x.x : 0.f, v1 ? x.y : 0.f);
                du[q] = pk(v0 ? m.x : 0.f, v1 ? m.y : 0.f);
            }
            float y[TB];
#pragma unroll
            for (int j = 0; j < TB; ++j) {
                const float2 dp = upk(dt[j % OWN / 2]), up = upk(du[j % OWN / 2]);
                float dv = j % 2 ? dp.y : dp.x, uu = j % 2 ? up.y : up.x;
                if constexpr (L > 1) {
                    dv = __shfl_sync(0xffffffffu, dv, j / OWN * CW + lane % CW);
                    uu = __shfl_sync(0xffffffffu, uu, j / OWN * CW + lane % CW);
                }
                const f2 dd = dup2(dv), ud = dup2(uu);
                const f2 *B = reinterpret_cast<const f2 *>(&sm.f[0][j0 + j][n0]);
                const f2 *C = reinterpret_cast<const f2 *>(&sm.f[1][j0 + j][n0]);
                f2 acc = 0;
#pragma unroll
                for (int q = 0; q < NK; q += 2) {
                    f2 b2[2], c2[2];
                    if constexpr (NK >= 2) {
                        const ulonglong2 bv = *reinterpret_cast<const ulonglong2 *>(B + q);
                        const ulonglong2 cv = *reinterpret_cast<const ulonglong2 *>(C + q);
                        b2[0] = bv.x, b2[1] = bv.y, c2[0] = cv.x, c2[1] = cv.y;
                    } else {
                        b2[0] = B[0], c2[0] = C[0];
                    }
#pragma unroll
                    for (int e = 0; e < (NK >= 2 ? 2 : 1); ++e) {
                        h[q + e] = fma2(ex2_2(mul2(dd, A[q + e])), h[q + e], mul2(ud, b2[e]));
                        acc = fma2(h[q + e], c2[e], acc);
                    }
                }
                const float2 r = upk(acc);
                y[j] = r.x + r.y;
            }
            // sums over the L lanes, each lane left with its own tokens'
#pragma unroll
            for (int w = L / 2; w >= 1; w /= 2) {
                const bool up = (l & w) != 0;
#pragma unroll
                for (int j = 0; j < OWN * w; ++j) {
                    const float lo = y[j], hi = y[j + OWN * w];
                    y[j] = (up ? hi : lo) + __shfl_xor_sync(0xffffffffu, up ? lo : hi, w * CW);
                }
            }
#pragma unroll
            for (int q = 0; q < OWN / 2; ++q) {
                const int r = j0 + l * OWN + 2 * q;
                f2 v = fma2(dup2(skip), uv[q], pk(y[2 * q], y[2 * q + 1]));
                if (!io.D) v = pk(y[2 * q], y[2 * q + 1]);
                if (gz) v = mul2(v, silu2(pk(to_f32(sm.raw[st][2][r][c]), to_f32(sm.raw[st][2][r + 1][c]))));
                const float2 o = upk(v);
                if (mine && r < n) gy[(size_t)(t0 + r) * s.ys] = from_f32<T>(o.x);
                if (mine && r + 1 < n) gy[(size_t)(t0 + r + 1) * s.ys] = from_f32<T>(o.y);
            }
        }
        if (table) {
            const int pos = done + t0 + n;
            if (pos % s.block_size == 0) {
                const int col = pos / s.block_size - 1;
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

template <typename T, int NP, int L>
cudaError_t launch_k(const SelParams &p, cudaStream_t stream) {
    constexpr size_t smem = sizeof(Smem<T, NP>);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(selective_kernel<T, NP, L>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return launch_after_prev(selective_kernel<T, NP, L>, dim3((unsigned)((int64_t)p.tiles * p.s.R)), dim3(kCh * L), smem,
                             stream, p);
}

#ifndef SEL_L16
#define SEL_L16 2
#endif

template <typename T>
cudaError_t launch(const SelParams &p, cudaStream_t stream) {
    const int64_t ctas = (int64_t)p.tiles * p.s.R;
    (void)ctas;
    if (p.s.N <= 8) return launch_k<T, 8, 2>(p, stream);
    if (p.s.N <= 16) return launch_k<T, 16, SEL_L16>(p, stream);
    if (p.s.N <= 32) return launch_k<T, 32, 4>(p, stream);
    if (p.s.N <= 64) return launch_k<T, 64, 8>(p, stream);
    if (p.s.N <= 128) return launch_k<T, 128, 8>(p, stream);
    return launch_k<T, 256, 8>(p, stream);
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
    if (io->block_table && (d->block_size < 1 || d->block_size % kTile != 0)) return SSD_ERR_BLOCK_SIZE;
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
    const int dg = d->D / d->G;
    const int64_t tiles = (int64_t)d->G * ((dg + kCh - 1) / kCh);
    if (tiles * d->R > 0x7fffffffLL) return SSD_ERR_DIMS;
    p.cu = cu_seqlens;
    p.io = *io;
    p.tiles = (int32_t)tiles;
    auto rows16 = [&](const void *ptr, int64_t stride, int64_t step) {  // rows and their parts on 16-byte boundaries
        return sel_aligned(ptr, 16) && stride * e % 16 == 0 && step * e % 16 == 0;
    };
    p.vec = rows16(io->u, p.s.us, dg) && rows16(io->delta, p.s.ds, dg) && (!io->z || rows16(io->z, p.s.zs, dg));
    p.bc_vec = rows16(io->B, p.s.bs, d->N) && rows16(io->C, p.s.cs, d->N);
    const cudaError_t err = d->dtype == SSD_DTYPE_BF16 ? launch<__nv_bfloat16>(p, stream) : launch<float>(p, stream);
    return err == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

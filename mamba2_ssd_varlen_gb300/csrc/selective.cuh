// selective.cuh -- what the selective scan's two kernels (prefill and windows) share.
#pragma once

#include "ssd_internal.cuh"

namespace ssd {

constexpr int kSelMaxN = 256;  // states a channel

// Sizes and strides of a call, strides resolved (no zeros).
struct SelShape {
    int64_t T;
    int32_t R, D, N, G, num_slots, block_size, bt_width, softplus;
    int64_t us, ds, bs, cs, zs, ys;  // elements between the rows of two tokens
};

// The step of one (token, channel): softplus of delta + bias, or the sum itself.
__device__ __forceinline__ float sel_step(float v, bool softplus) { return softplus ? softplus_f32(v) : v; }

// Validates the sizes; fills the shape with resolved strides.  Shared by both entry points.
inline int sel_shape(const ssd_selective_dims *d, bool has_z, SelShape *s) {
    if (d->reserved != 0) return SSD_ERR_DIMS;
    if (d->T < 0 || d->T > 0x7fffff00LL || d->R < 1 || d->D < 1 || d->D > (1 << 24) || d->N < 1 ||
        d->G < 1 || d->num_slots < 0 || d->block_size < 0 || d->block_table_width < 0)
        return SSD_ERR_DIMS;
    if (d->D % d->G != 0) return SSD_ERR_GROUPS;
    if (d->dtype != SSD_DTYPE_BF16 && d->dtype != SSD_DTYPE_F32) return SSD_ERR_DTYPE;
    if (d->N > kSelMaxN) return SSD_ERR_UNSUPPORTED;
    const int64_t gn = (int64_t)d->G * d->N;
    const int64_t given[6] = {d->u_stride, d->delta_stride, d->B_stride, d->C_stride, d->z_stride, d->y_stride};
    const int64_t row[6] = {d->D, d->D, gn, gn, d->D, d->D};
    int64_t use[6];
    for (int k = 0; k < 6; ++k) {
        use[k] = given[k] ? given[k] : row[k];
        if (k == 4 && !has_z) continue;  // the stride of an absent z is not looked at
        if (use[k] < row[k] || use[k] > (1LL << 31)) return SSD_ERR_DIMS;
    }
    s->T = d->T;
    s->R = d->R;
    s->D = d->D;
    s->N = d->N;
    s->G = d->G;
    s->num_slots = d->num_slots;
    s->block_size = d->block_size;
    s->bt_width = d->block_table_width;
    s->softplus = d->softplus != 0;
    s->us = use[0];
    s->ds = use[1];
    s->bs = use[2];
    s->cs = use[3];
    s->zs = use[4];
    s->ys = use[5];
    return SSD_OK;
}

inline bool sel_aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

}  // namespace ssd

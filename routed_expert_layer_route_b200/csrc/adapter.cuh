// adapter.cuh -- low-rank adapters of many requests beside one shared
// projection, and their gradients.
//
// Row t of a batch belongs to adapter a = adapter[t] (MOE_EMPTY_SLOT: none);
// adapter a holds A_a [r x din] and B_a [r x dout], both by rank:
//     u_t = s_a A_a x_t                 y_t = W x_t + b + B_a^T u_t
// and backwards, dy_t given:
//     v_t = s_a B_a dy_t                dx_t = W^T dy_t + A_a^T v_t
//     dA_a = sum_{t of a} v_t x_t^T     dB_a = sum_{t of a} u_t dy_t^T
// dx is the same contraction as y with W^T for W and A, B exchanged, and the
// two weight gradients are one contraction too, so three kernels do it all:
// the inner products (u, v), the projection (y, dx) and the sums of outer
// products (dA, dB).
#pragma once
#include "common.cuh"

namespace moe {

MOE_DEVINL float bf16_to_f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// The adapter of a row: -1 for none; an id outside [0, n) is recorded and
// taken as none.
MOE_DEVINL int adapter_of(const int32_t *adapter, int t, int n, int *status)
{
    const int a = __ldg(&adapter[t]);
    if ((unsigned)a < (unsigned)n)
        return a;
    if (a != MOE_EMPTY_SLOT)
        set_status(status, MOE_ERR_DEVICE_CHECK);
    return -1;
}

// ---------------------------------------------------------------------------
// Inner products: u[t][j] = s_a <x_t, A_a[j]>, 0 for rows without an adapter.
struct AdInnerArgs {
    const uint16_t *x;       // [T x din]
    const uint16_t *a;       // [n x r x din]
    const int32_t *adapter;  // [T]
    const float *scale;      // nullable [n]
    float *u;                // [T x r]
    int T, din, r, n;
    int *status;
};

// One warp for each (row, rank).
__global__ void __launch_bounds__(256) k_ad_inner(AdInnerArgs p)
{
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (i >= (int64_t)p.T * p.r)
        return;
    const int t = (int)(i / p.r), j = (int)(i % p.r);
    const int a = adapter_of(p.adapter, t, p.n, p.status);
    float s = 0.0f;
    if (a >= 0) {
        const uint16_t *x = p.x + (size_t)t * p.din, *w = p.a + ((size_t)a * p.r + j) * p.din;
        for (int k = lane; k < p.din; k += 32)
            s = fmaf(bf16_to_f32(x[k]), bf16_to_f32(w[k]), s);
        s = warp_sum(s) * (p.scale ? __ldg(&p.scale[a]) : 1.0f);
    }
    if (lane == 0)
        p.u[i] = s;
}

// ---------------------------------------------------------------------------
// The projection: y = x W^T + bias + sum_j u[t][j] B_a[j].  w nullptr: y
// holds the product already.
struct AdProductArgs {
    const uint16_t *x;       // [T x din]
    const uint16_t *w;       // nullable [dout x din]
    const float *bias;       // nullable [dout]
    const uint16_t *b;       // [n x r x dout]
    const int32_t *adapter;  // [T]
    const float *u;          // [T x r]
    void *y;                 // [T x dout]
    int y_bf16;
    int T, din, dout, r, n;
    int *status;
};

MOE_DEVINL void ad_store(const AdProductArgs &p, int t, int o, float v)
{
    const size_t i = (size_t)t * p.dout + o;
    if (p.bias)
        v += __ldg(&p.bias[o]);
    if (p.y_bf16) {
        uint16_t *y = static_cast<uint16_t *>(p.y) + i;
        *y = f32_to_bf16_rn(p.w ? v : v + bf16_to_f32(*y));
    } else {
        float *y = static_cast<float *>(p.y) + i;
        *y = p.w ? v : v + *y;
    }
}

// 64 x 64 outputs a CTA, 4 x 4 a thread, 16 values of K in shared memory at a time.
__global__ void __launch_bounds__(256) k_ad_product(AdProductArgs p)
{
    __shared__ float sx[16][65], sw[16][65];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int t0 = blockIdx.y * 64, o0 = blockIdx.x * 64;
    float acc[4][4] = {};
    if (p.w)
        for (int k0 = 0; k0 < p.din; k0 += 16) {
            for (int i = tid; i < 64 * 16; i += 256) {
                const int row = i >> 4, k = k0 + (i & 15);
                sx[i & 15][row] = t0 + row < p.T && k < p.din
                                      ? bf16_to_f32(p.x[(size_t)(t0 + row) * p.din + k])
                                      : 0.0f;
                sw[i & 15][row] = o0 + row < p.dout && k < p.din
                                      ? bf16_to_f32(p.w[(size_t)(o0 + row) * p.din + k])
                                      : 0.0f;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 16; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[i][j] = fmaf(sx[k][ty + 16 * i], sw[k][tx + 16 * j], acc[i][j]);
            __syncthreads();
        }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = t0 + ty + 16 * i;
        if (t >= p.T)
            continue;
        const int a = adapter_of(p.adapter, t, p.n, p.status);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int o = o0 + tx + 16 * j;
            if (o >= p.dout)
                continue;
            float v = acc[i][j];
            if (a >= 0)
                for (int q = 0; q < p.r; ++q)
                    v = fmaf(p.u[(size_t)t * p.r + q],
                             bf16_to_f32(p.b[((size_t)a * p.r + q) * p.dout + o]), v);
            ad_store(p, t, o, v);
        }
    }
}

// ---------------------------------------------------------------------------
// Sums of outer products: g[a][j][c] = sum_{t of a} u[t][j] z[t][c], rows in order.
struct AdOuterArgs {
    const float *u;          // [T x r]
    const uint16_t *z;       // [T x D]
    const int32_t *adapter;  // [T]
    float *g;                // [n x r x D]
    int T, D, r, n;
    int *status;
};

// One thread for each column of an (adapter, rank).
__global__ void __launch_bounds__(128) k_ad_outer(AdOuterArgs p)
{
    pdl_wait();
    pdl_trigger();
    const int c = blockIdx.x * 128 + threadIdx.x, j = blockIdx.y, a = blockIdx.z;
    if (c >= p.D)
        return;
    float s = 0.0f;
    for (int t = 0; t < p.T; ++t)
        if (__ldg(&p.adapter[t]) == a)
            s = fmaf(p.u[(size_t)t * p.r + j], bf16_to_f32(p.z[(size_t)t * p.D + c]), s);
    p.g[((size_t)a * p.r + j) * p.D + c] = s;
}

}  // namespace moe

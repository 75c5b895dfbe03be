// balance.cuh -- training a router: the balance and z losses of a route with
// the per-expert counts, and the gradient of the router logits through the
// routing weights and both losses.
//
// Losses (p_t = softmax(z_t), lse_t = log sum_e exp(z_te); N the tokens that
// count, n_e the routed slots of expert e over them, R = sum_e n_e):
//     P_e   = (1/N) sum_t p_te          f_e = n_e / R
//     L_bal = E sum_e f_e P_e           L_z = (1/N) sum_t lse_t^2
// Gradient (f held fixed, as counts are whole numbers), g the loss's gradient:
//     dz_te = g/N p_te (c_bal E (f_e - sum_j f_j p_tj) + 2 c_z lse_t)
// Routing weights ("Paper of the Week #3", section "The Receipt", Eq. 2):
// w_i = p_i / sum_{j in K2} p_j is a softmax over the k2 best experts, so with
// g_i = dL/dw_i (zero beside the routed slots)
//     dz_m = w_m (g_m - sum_i g_i w_i) for m in K2, 0 elsewhere.
// K2 is the token's given experts and, of the others, those of the largest
// logits, equal ones by the lower index -- the set Eq. 2 ranked, found again
// without its order.
//
// Both kernels give a token one warp and hold its E logits in registers, so
// each logit is read once; sums over a token are warp reductions in float32.
#pragma once
#include "common.cuh"

namespace moe {

constexpr int kBalWarps = 8;

// Element i of a lane's N values of a row: vectors of VEC values, lanes side by side.
template <int VEC>
MOE_DEVINL int row_index(int i, int lane)
{
    return (i / VEC) * (32 * VEC) + lane * VEC + (i % VEC);
}

// The row's logits, -inf behind its end.  VEC 4 needs E % 4 == 0.
template <int VEC, int N>
MOE_DEVINL void load_row(const float *z, int E, int lane, float (&v)[N])
{
    const float kNegInf = -__int_as_float(0x7f800000);
#pragma unroll
    for (int i = 0; i < N; i += VEC) {
        const int j = row_index<VEC>(i, lane);
        if (VEC == 4) {
            float4 q = make_float4(kNegInf, kNegInf, kNegInf, kNegInf);
            if (j < E)
                q = __ldcs(reinterpret_cast<const float4 *>(z + j));
            v[i] = q.x;
            v[i + 1] = q.y;
            v[i + 2] = q.z;
            v[i + 3] = q.w;
        } else {
            v[i] = j < E ? __ldcs(z + j) : kNegInf;
        }
    }
}

MOE_DEVINL float warp_max(float v)
{
    asm volatile("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(v));  // passes over NaN
    return v;
}

// ---------------------------------------------------------------------------
// Sums that CTAs add to are whole numbers, so their order does not show:
// counts as int32, sum_t p_te in steps of 2^-40 as 64 bits (T <= 2^20).
constexpr double kBalStep = 1099511627776.0;  // 2^40

struct BalanceArgs {
    const float *logits;        // [T x E]
    const int32_t *idx;         // [T x k1]
    const uint8_t *mask;        // nullable [T]
    int T, E, k1;
    float c_bal, c_z;
    int32_t *counts;            // out [E + 1]
    float *loss;                // out [3]
    float *prob;                // nullable out [E]
    unsigned long long *p_acc;  // [E] zero between calls
    int *n_acc;                 // [E + 1] zero between calls
    unsigned *arrive;           // zero between calls
    double *z_part;             // [grid]
    int *status;
};

template <int VEC, int N>
__global__ void __launch_bounds__(kBalWarps * 32) k_balance(BalanceArgs a)
{
    extern __shared__ uint8_t bal_smem[];
    float *sp = reinterpret_cast<float *>(bal_smem);   // [kBalWarps][E] probability sums
    int *sn = reinterpret_cast<int *>(sp + kBalWarps * a.E);  // [E + 1] counts
    __shared__ double sz[kBalWarps];
    __shared__ int last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float kNegInf = -__int_as_float(0x7f800000);
    const int E = a.E;
    for (int e = tid; e <= E; e += kBalWarps * 32)
        sn[e] = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();

    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        acc[i] = 0.0f;
    double zsum = 0.0;
    int tokens = 0;
    for (int t = blockIdx.x * kBalWarps + warp; t < a.T; t += gridDim.x * kBalWarps) {
        if (a.mask && !a.mask[t])
            continue;
        float v[N];
        load_row<VEC, N>(a.logits + (size_t)t * E, E, lane, v);
        const int e = lane < a.k1 ? a.idx[(size_t)t * a.k1 + lane] : MOE_EMPTY_SLOT;
        float m = kNegInf;
        bool some = false;  // a row of -inf alone has no distribution and does not count
#pragma unroll
        for (int i = 0; i < N; ++i) {
            m = fmaxf(m, v[i]);
            some |= !(v[i] == kNegInf);
        }
        if (!__any_sync(0xffffffffu, some))
            continue;
        m = warp_max(m);
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = __expf(v[i] - m);
            s += v[i];
        }
        s = warp_sum(s);
        const float inv = 1.0f / s;
#pragma unroll
        for (int i = 0; i < N; ++i)
            acc[i] = fmaf(v[i], inv, acc[i]);
        const double lse = (double)m + (double)logf(s);
        zsum += lse * lse;
        ++tokens;
        if ((unsigned)e < (unsigned)E)
            atomicAdd(&sn[e], 1);
        else if (e != MOE_EMPTY_SLOT)
            set_status(a.status, MOE_ERR_DEVICE_CHECK);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int j = row_index<VEC>(i, lane);
        if (j < E)
            sp[warp * E + j] = acc[i];
    }
    if (lane == 0) {
        sz[warp] = zsum;
        atomicAdd(&sn[E], tokens);
    }
    __syncthreads();
    for (int e = tid; e <= E; e += kBalWarps * 32) {
        if (sn[e])
            atomicAdd(&a.n_acc[e], sn[e]);
        if (e < E) {
            float p = 0.0f;
#pragma unroll
            for (int w = 0; w < kBalWarps; ++w)
                p += sp[w * E + e];
            if (p > 0.0f)  // a NaN shows in the z sum
                atomicAdd(&a.p_acc[e], __double2ull_rn((double)p * kBalStep));
        }
    }
    if (tid == 0) {
        double z = 0.0;
        for (int w = 0; w < kBalWarps; ++w)
            z += sz[w];
        a.z_part[blockIdx.x] = z;
    }
    __threadfence();
    __syncthreads();
    if (tid == 0)
        last = atomicAdd(a.arrive, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!last)
        return;
    // the last CTA: totals, the losses, and the accumulators back to zero
    __threadfence();
    double z = 0.0, rn = 0.0, fp = 0.0;
    for (int g = tid; g < gridDim.x; g += kBalWarps * 32)
        z += __ldcg(&a.z_part[g]);
    const int N_tok = __ldcg(&a.n_acc[E]);
    const double per = 1.0 / (kBalStep * (N_tok > 0 ? N_tok : 1));
    for (int e = tid; e < E; e += kBalWarps * 32) {
        const int n = __ldcg(&a.n_acc[e]);
        a.counts[e] = n;
        const double P = (double)__ldcg(&a.p_acc[e]) * per;
        sp[e] = (float)P;
        rn += n;
        fp += n * P;
    }
    __shared__ double red[3][kBalWarps];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        z += __shfl_xor_sync(0xffffffffu, z, o);
        rn += __shfl_xor_sync(0xffffffffu, rn, o);
        fp += __shfl_xor_sync(0xffffffffu, fp, o);
    }
    if (lane == 0) {
        red[0][warp] = z;
        red[1][warp] = rn;
        red[2][warp] = fp;
    }
    __syncthreads();
    z = rn = fp = 0.0;
    for (int w = 0; w < kBalWarps; ++w) {
        z += red[0][w];
        rn += red[1][w];
        fp += red[2][w];
    }
    const bool bad = z != z;
    if (a.prob)
        for (int e = tid; e < E; e += kBalWarps * 32)
            a.prob[e] = bad ? (float)z : sp[e];
    if (tid == 0) {
        const double bal = bad ? z : rn > 0.0 ? E * fp / rn : 0.0;
        const double zl = N_tok > 0 ? z / N_tok : 0.0;
        a.counts[E] = N_tok;
        a.loss[0] = (float)(a.c_bal * bal + a.c_z * zl);
        a.loss[1] = (float)bal;
        a.loss[2] = (float)zl;
        *a.arrive = 0u;
    }
    __syncthreads();
    for (int e = tid; e <= E; e += kBalWarps * 32) {
        a.n_acc[e] = 0;
        if (e < E)
            a.p_acc[e] = 0ull;
    }
}

inline size_t balance_smem_bytes(int E) { return sizeof(float) * kBalWarps * E + sizeof(int) * (E + 1); }

// ---------------------------------------------------------------------------
struct RouteBackArgs {
    const float *logits;   // [T x E]
    const int32_t *idx;    // [T x k1]
    const float *d_w;      // nullable [T x k1]
    const int32_t *counts; // nullable [E + 1]: the losses' part is added
    const float *d_loss;   // nullable (1)
    const uint8_t *mask;   // nullable [T]
    int T, E, k1, k2;
    float c_bal, c_z;
    void *dz;              // [T x E]
    int dz_bf16;
    int *status;           // nullable
};

// Order-preserving whole number of a float (0.0 and -0.0 alike, NaN last); 0 is below them all.
MOE_DEVINL unsigned order_key(float z)
{
    const unsigned u = __float_as_uint(z + 0.0f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

template <int N>
MOE_DEVINL int count_from(const unsigned (&key)[N], unsigned lo)
{
    int c = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
        c += key[i] >= lo;
    return __reduce_add_sync(0xffffffffu, c);
}

// The `need` largest of the warp's keys (0: not a candidate; at least `need`
// candidates, need >= 1), equal ones by the lower row index: bit i of the
// result marks this lane's element i.  Halves the interval of keys that holds
// the border until a key separates exactly `need` from the rest; where equal
// keys lie on the border, the lowest indices among them are taken one by one.
template <int VEC, int N>
MOE_DEVINL unsigned select_largest(const unsigned (&key)[N], int need, int lane)
{
    unsigned top = 0u;
#pragma unroll
    for (int i = 0; i < N; ++i)
        top = max(top, key[i]);
    unsigned lo = 1u;  // at least `need` keys are >= lo, fewer are >= hi
    if (need <= 32)    // 32 lanes' largest keys are all >= the least of them
        lo = max(lo, __reduce_min_sync(0xffffffffu, top));
    unsigned hi = __reduce_max_sync(0xffffffffu, top) + 1u;
    bool exact = false;
    while (hi - lo > 1u) {
        const unsigned mid = lo + (hi - lo) / 2u;
        const int c = count_from<N>(key, mid);
        if (c == need) {
            lo = mid;
            exact = true;
            break;
        }
        if (c > need)
            lo = mid;
        else
            hi = mid;
    }
    unsigned in = 0u;
    if (!exact && count_from<N>(key, lo) == need)
        exact = true;
    if (exact) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            in |= (unsigned)(key[i] >= lo) << i;
        return in;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        in |= (unsigned)(key[i] > lo) << i;
    int left = need - __reduce_add_sync(0xffffffffu, __popc(in));
    while (left-- > 0) {
        unsigned best = 0xffffffffu;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (key[i] == lo && !((in >> i) & 1u))
                best = min(best, (unsigned)row_index<VEC>(i, lane));
        best = __reduce_min_sync(0xffffffffu, best);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if ((unsigned)row_index<VEC>(i, lane) == best)
                in |= 1u << i;
    }
    return in;
}

template <int VEC, int N>
__global__ void __launch_bounds__(kBalWarps * 32) k_route_backward(RouteBackArgs a)
{
    extern __shared__ uint8_t rb_smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int E = a.E, Ep = (E + 3) & ~3;
    float *share = reinterpret_cast<float *>(rb_smem);         // [Ep] f_e
    float *gw = share + Ep + warp * Ep;                        // [Ep] of this warp: dL/dw, zero
    uint32_t *given = reinterpret_cast<uint32_t *>(share + (kBalWarps + 1) * Ep) + warp * 32;
    __shared__ int total;
    const float kNegInf = -__int_as_float(0x7f800000);
    for (int e = tid; e < (kBalWarps + 1) * Ep; e += kBalWarps * 32)
        share[e] = 0.0f;
    given[lane] = 0u;
    if (tid == 0)
        total = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    float per = 0.0f;  // d_loss / N
    if (a.counts) {
        int n = 0;
        for (int e = tid; e < E; e += kBalWarps * 32)
            n += __ldg(&a.counts[e]);
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0)
            atomicAdd(&total, n);
        __syncthreads();
        const float R = (float)max(total, 1);
        for (int e = tid; e < E; e += kBalWarps * 32)
            share[e] = (float)__ldg(&a.counts[e]) / R;
        per = (a.d_loss ? __ldg(a.d_loss) : 1.0f) / (float)max(__ldg(&a.counts[E]), 1);
        __syncthreads();
    }

    for (int t = blockIdx.x * kBalWarps + warp; t < a.T; t += gridDim.x * kBalWarps) {
        float v[N];
        bool some = false;
        if (!a.mask || a.mask[t]) {
            load_row<VEC, N>(a.logits + (size_t)t * E, E, lane, v);
#pragma unroll
            for (int i = 0; i < N; ++i)
                some |= !(v[i] == kNegInf);
        }
        float dz[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            dz[i] = 0.0f;
        if (__any_sync(0xffffffffu, some)) {
            float m = kNegInf;
#pragma unroll
            for (int i = 0; i < N; ++i)
                m = fmaxf(m, v[i]);
            m = warp_max(m);
            if (a.d_w) {
                // the given slots: their gradients (summed in slot order) and a bit each
                int e = lane < a.k1 ? a.idx[(size_t)t * a.k1 + lane] : MOE_EMPTY_SLOT;
                const float g = lane < a.k1 ? a.d_w[(size_t)t * a.k1 + lane] : 0.0f;
                if ((unsigned)e >= (unsigned)E) {
                    if (e != MOE_EMPTY_SLOT)
                        set_status(a.status, MOE_ERR_DEVICE_CHECK);
                    e = -1;
                }
                for (int s = 0; s < a.k1; ++s) {
                    if (lane == s && e >= 0) {
                        gw[e] += g;
                        given[e >> 5] |= 1u << (e & 31);
                    }
                    __syncwarp();
                }
                float gv[N];
                unsigned set = 0u;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int j = row_index<VEC>(i, lane);
                    gv[i] = 0.0f;
                    if (j < E) {
                        gv[i] = gw[j];
                        set |= ((given[j >> 5] >> (j & 31)) & 1u) << i;
                    }
                }
                __syncwarp();
                if (e >= 0) {
                    gw[e] = 0.0f;
                    given[e >> 5] = 0u;
                }
                __syncwarp();
                if (a.k2 >= E) {
                    set = 0xffffffffu;
                } else {
                    const int need = a.k2 - __reduce_add_sync(0xffffffffu, __popc(set));
                    if (need > 0) {
                        unsigned key[N];
#pragma unroll
                        for (int i = 0; i < N; ++i)
                            key[i] = row_index<VEC>(i, lane) < E && !((set >> i) & 1u)
                                         ? order_key(v[i])
                                         : 0u;
                        set |= select_largest<VEC, N>(key, need, lane);
                    }
                }
                // softmax over the set and its gradient
                float m2 = kNegInf;
                bool in_set = false;
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if ((set >> i) & 1u) {
                        m2 = fmaxf(m2, v[i]);
                        in_set |= !(v[i] == kNegInf);
                    }
                m2 = warp_max(m2);
                if (__any_sync(0xffffffffu, in_set)) {
                    float s2 = 0.0f, gs = 0.0f;
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        dz[i] = (set >> i) & 1u ? __expf(v[i] - m2) : 0.0f;
                        s2 += dz[i];
                        gs = fmaf(gv[i], dz[i], gs);
                    }
                    s2 = warp_sum(s2);
                    gs = warp_sum(gs) / s2;
                    const float inv = 1.0f / s2;
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        dz[i] = (set >> i) & 1u ? dz[i] * inv * (gv[i] - gs) : 0.0f;
                }
            }
            if (a.counts) {
                float s = 0.0f, fp = 0.0f;
                float f[N];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int j = row_index<VEC>(i, lane);
                    f[i] = j < E ? share[j] : 0.0f;
                    v[i] = __expf(v[i] - m);
                    s += v[i];
                    fp = fmaf(f[i], v[i], fp);
                }
                s = warp_sum(s);
                fp = warp_sum(fp);
                const float inv = 1.0f / s;
                const float lse = m + logf(s);
                const float cb = a.c_bal * (float)E;
                const float at = fmaf(-cb, fp * inv, 2.0f * a.c_z * lse);
#pragma unroll
                for (int i = 0; i < N; ++i)
                    dz[i] = fmaf(per * (v[i] * inv), fmaf(cb, f[i], at), dz[i]);
            }
        }
        // one rounding, to the output's type
#pragma unroll
        for (int i = 0; i < N; i += VEC) {
            const int j = row_index<VEC>(i, lane);
            if (j >= E)
                continue;
            const size_t o = (size_t)t * E + j;
            if (VEC == 4) {
                if (a.dz_bf16) {
                    const uint32_t lo = (uint32_t)f32_to_bf16_rn(dz[i]) |
                                        ((uint32_t)f32_to_bf16_rn(dz[i + 1]) << 16);
                    const uint32_t hi = (uint32_t)f32_to_bf16_rn(dz[i + 2]) |
                                        ((uint32_t)f32_to_bf16_rn(dz[i + 3]) << 16);
                    __stcs(reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.dz) + o),
                           make_uint2(lo, hi));
                } else {
                    __stcs(reinterpret_cast<float4 *>(static_cast<float *>(a.dz) + o),
                           make_float4(dz[i], dz[i + 1], dz[i + 2], dz[i + 3]));
                }
            } else if (a.dz_bf16) {
                static_cast<uint16_t *>(a.dz)[o] = f32_to_bf16_rn(dz[i]);
            } else {
                static_cast<float *>(a.dz)[o] = dz[i];
            }
        }
    }
}

inline size_t route_backward_smem_bytes(int E)
{
    return sizeof(float) * (kBalWarps + 1) * ((E + 3) & ~3) + sizeof(uint32_t) * 32 * kBalWarps;
}

}  // namespace moe

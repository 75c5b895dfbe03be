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
// T = 65536, E = 512: k_balance 28 us, 4.9 TB/s, bound by the read (76% of the
// copy bandwidth); k_route_backward with both parts, k1 = 5, k2 = 20, 85 us,
// bound by its instructions (about 950 a row, 400 of them on the half-rate
// comparison and logic pipe; reading and writing alone would take 32 us).  Rows
// with equal logits on the border take the general row, which raises the tied
// experts one by one: the weights' part alone takes 74 us for logits without ties,
// 411 us for logits in steps of 1/4, 231 us for equal ones (a new router's), and
// for 4096 rows of 1024 experts, k2 = 1023, 17 us and 1.1 ms.
// Small calls take 4 to 5 us, a launch and one pass of dependent loads.
#pragma once
#include "common.cuh"
#include "grouped.cuh"

namespace moe {

constexpr int kBalWarps = 8;
// CTAs of N values a lane that an SM holds (registers); a launch fills the
// device once and its warps take rows in turn
constexpr int row_ctas(int N) { return N <= 8 ? 4 : N <= 16 ? 3 : 2; }

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

// e^(z - m): the difference first, so that the largest logit's is exactly 1 (a
// fused multiply-add would leave a few last bits, which show where a weight of
// 1 cancels: k2 = 1 has no gradient through its weight at all); then the
// hardware's power of two (2^-22 relative).
constexpr float kLog2e = 1.4426950408889634f;
MOE_DEVINL float exp_from(float z, float m)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"((z - m) * kLog2e));
    return y;
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
    // WsKept's
    unsigned long long *p_acc;  // [E] zero between calls
    int *n_acc;                 // [E + 1] zero between calls
    unsigned *arrive;           // zero between calls
    double *z_part;             // [grid]
    int *status;
};

template <int VEC, int N>
__global__ void __launch_bounds__(kBalWarps * 32, row_ctas(N)) k_balance(BalanceArgs a)
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
    const int step = gridDim.x * kBalWarps;
    float next[N];  // the row after this one, on its way while this one is summed
    int next_e = MOE_EMPTY_SLOT;
    bool next_live = false;
    auto fetch = [&](int t) {
        next_live = t < a.T && (!a.mask || a.mask[t]);
        if (next_live) {
            load_row<VEC, N>(a.logits + (size_t)t * E, E, lane, next);
            next_e = lane < a.k1 ? a.idx[(size_t)t * a.k1 + lane] : MOE_EMPTY_SLOT;
        }
    };
    int t = blockIdx.x * kBalWarps + warp;
    fetch(t);
    for (; t < a.T; t += step) {
        float v[N];
        const bool live = next_live;
        const int e = next_e;
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = next[i];
        fetch(t + step);
        if (!live)
            continue;
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
            v[i] = exp_from(v[i], m);
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
constexpr int kRouteWarps = 8;
// as row_ctas; four CTAs spill a little and still win (65536 rows of 512: 85 us, 87 with three)
constexpr int route_ctas(int N) { return N <= 16 ? 4 : 2; }

struct RouteBackArgs {
    const float *logits;   // [T x E]
    const int32_t *idx;    // [T x k1]
    const float *d_w;      // nullable [T x k1]
    const int32_t *counts; // nullable [E + 1]: the losses' part is added
    const float *d_loss;   // nullable (1)
    const uint8_t *mask;   // nullable [T]
    int T, E, k1, k2;      // k1 <= k2 <= E
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

constexpr unsigned kGivenKey = 0xffffffffu;  // above every logit's key

// The key from which the warp's `want` largest keys begin (there are at least
// `want`, 1 <= want, and fewer of kGivenKey; top: no other key is above it).
// Halves the interval of keys that holds the border until a key separates
// exactly `want` from the rest; where equal keys lie on the border, the lowest
// row indices among them are raised to kGivenKey one by one.
template <int VEC, int N>
MOE_DEVINL unsigned border_key(unsigned (&key)[N], int want, unsigned top, int lane)
{
    unsigned lo = 1u, hi = top + 1u;  // at least `want` keys are >= lo, fewer are >= hi
    if (want <= 32) {                 // 32 lanes' largest keys are all >= the least of them
        unsigned mine = 0u;
#pragma unroll
        for (int i = 0; i < N; ++i)
            mine = max(mine, key[i]);
        lo = max(lo, __reduce_min_sync(0xffffffffu, mine));
        lo = min(lo, top);
    }
    while (hi - lo > 1u) {
        const unsigned mid = lo + (hi - lo) / 2u;
        const int c = count_from<N>(key, mid);
        if (c == want)
            return mid;
        if (c > want)
            lo = mid;
        else
            hi = mid;
    }
    // all keys between lo and hi are lo
    int left = want - count_from<N>(key, lo + 1u);
    if (count_from<N>(key, lo) - want == 0)
        return lo;
    while (left-- > 0) {
        unsigned best = 0xffffffffu;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (key[i] == lo)
                best = min(best, (unsigned)row_index<VEC>(i, lane));
        best = __reduce_min_sync(0xffffffffu, best);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if ((unsigned)row_index<VEC>(i, lane) == best)
                key[i] = kGivenKey;
    }
    return lo + 1u;
}

MOE_DEVINL float key_value(unsigned k)
{
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// The same border among a row's logits v themselves: true with thr where
// exactly `want` of them (1 <= want < the row's length, largest m) are >= thr;
// false where equal logits lie on the border.  The search first looks at each
// lane's three largest only -- three comparisons a step instead of N -- which
// finds the border unless a lane holds four of the `want` largest; a
// count over all elements says whether it did.
template <int N>
MOE_DEVINL bool border_value(const float (&v)[N], int want, float m, float &thr)
{
    const float kNegInf = -__int_as_float(0x7f800000);
    float a = kNegInf, b = kNegInf, c = kNegInf;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float t = fminf(a, v[i]);
        a = fmaxf(a, v[i]);
        const float u = fminf(b, t);
        b = fmaxf(b, t);
        c = fmaxf(c, u);
    }
    // at least `want` logits are >= lo's value, fewer are >= hi's
    unsigned lo = order_key(kNegInf), hi = order_key(m) + 1u;
    if (want <= 32) {  // 32 lanes' largest are all >= the least of them
        float least = a;
        asm volatile("redux.sync.min.f32 %0, %0, 0xffffffff;" : "+f"(least));
        lo = min(order_key(least), hi - 1u);
    }
    unsigned l3 = lo, h3 = hi;
    if (want <= 96)
        while (h3 - l3 > 1u) {
            const unsigned mid = l3 + (h3 - l3) / 2u;
            const float x = key_value(mid);
            // (one reduction: three votes' bit counts run at an eighth of the rate)
            const int n = __reduce_add_sync(0xffffffffu, (int)(a >= x) + (int)(b >= x) + (int)(c >= x));
            if (n == want) {
                thr = x;
                int all = 0;
#pragma unroll
                for (int i = 0; i < N; ++i)
                    all += v[i] >= x;
                if (__reduce_add_sync(0xffffffffu, all) == want)
                    return true;
                lo = mid;  // more than `want` are
                break;
            }
            if (n > want)
                l3 = mid;
            else
                h3 = mid;
        }
    while (hi - lo > 1u) {
        const unsigned mid = lo + (hi - lo) / 2u;
        const float x = key_value(mid);
        int n = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            n += v[i] >= x;
        n = __reduce_add_sync(0xffffffffu, n);
        if (n == want) {
            thr = x;
            return true;
        }
        if (n > want)
            lo = mid;
        else
            hi = mid;
    }
    thr = key_value(lo);
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
        n += v[i] >= thr;
    return __reduce_add_sync(0xffffffffu, n) == want;
}

// A lane's vector of a row in shared memory (padded to whole vectors).
template <int VEC>
MOE_DEVINL void smem_vec(const float *p, int E, int j, float (&v)[VEC])
{
    if (VEC == 4) {
        float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (j < E)
            q = *reinterpret_cast<const float4 *>(p + j);
        v[0] = q.x;
        v[1 % VEC] = q.y;
        v[2 % VEC] = q.z;
        v[3 % VEC] = q.w;
    } else {
        v[0] = j < E ? p[j] : 0.0f;
    }
}

// All of a lane's values.
template <int VEC, int N>
MOE_DEVINL void smem_row(const float *p, int E, int lane, float (&v)[N])
{
#pragma unroll
    for (int i = 0; i < N; i += VEC) {
        float q[VEC];
        smem_vec<VEC>(p, E, row_index<VEC>(i, lane), q);
#pragma unroll
        for (int k = 0; k < VEC; ++k)
            v[i + k] = q[k];
    }
}

template <int VEC, int N>
MOE_DEVINL void store_row(const RouteBackArgs &a, int t, int lane, const float (&v)[N])
{
    // one rounding, to the output's type
#pragma unroll
    for (int i = 0; i < N; i += VEC) {
        const int j = row_index<VEC>(i, lane);
        if (j >= a.E)
            continue;
        const size_t o = (size_t)t * a.E + j;
        if (VEC == 4) {
            if (a.dz_bf16)
                __stcs(reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.dz) + o),
                       make_uint2(pack_bf16x2(v[i], v[i + 1]), pack_bf16x2(v[i + 2], v[i + 3])));
            else
                __stcs(reinterpret_cast<float4 *>(static_cast<float *>(a.dz) + o),
                       make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]));
        } else if (a.dz_bf16) {
            static_cast<uint16_t *>(a.dz)[o] = f32_to_bf16_rn(v[i]);
        } else {
            static_cast<float *>(a.dz)[o] = v[i];
        }
    }
}

// One row whose K2 is not simply its k2 largest logits: equal logits on the
// border, or given experts that are not among the largest.  e: the lane's
// slot (-1: none); gw holds the slots' gradients at their experts.
template <int VEC, int N>
__device__ __noinline__ void route_row_general(const RouteBackArgs &a, int t, int e, float *gw,
                                               const float *share, int lane, float m, float per,
                                               float cb)
{
    const float kNegInf = -__int_as_float(0x7f800000);
    const int E = a.E;
    float v[N];
    load_row<VEC, N>(a.logits + (size_t)t * E, E, lane, v);
    unsigned key[N], thr;
    unsigned mine = 0u;  // given elements of this lane
    for (int s = 0; s < a.k1; ++s) {
        const int es = __shfl_sync(0xffffffffu, e, s);
        // row_index's inverse: the lane and element that hold expert es
        if (es >= 0 && (es / VEC) % 32 == lane)
            mine |= 1u << (es / (32 * VEC) * VEC + es % VEC);
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        key[i] = (mine >> i) & 1u ? kGivenKey : order_key(v[i]);
    float m2 = m;
    if (__reduce_add_sync(0xffffffffu, __popc(mine)) < a.k2) {
        thr = border_key<VEC, N>(key, a.k2, order_key(m), lane);
    } else {
        thr = kGivenKey;
        m2 = kNegInf;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (key[i] == kGivenKey)
                m2 = fmaxf(m2, v[i]);
        m2 = warp_max(m2);
        if (m2 == kNegInf) {  // weights of 0: nothing to differentiate
            thr = 1u;
#pragma unroll
            for (int i = 0; i < N; ++i)
                key[i] = 0u;
        }
    }
    float g[N], f[N];
    smem_row<VEC, N>(gw, E, lane, g);
    smem_row<VEC, N>(share, E, lane, f);
    float s = 0.0f, fp = 0.0f, s2 = 0.0f, gs = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float x = exp_from(v[i], m);
        const float w = key[i] >= thr ? exp_from(v[i], m2) : 0.0f;
        s += x;
        fp = fmaf(f[i], x, fp);
        s2 += w;
        if (key[i] >= thr)
            gs = fmaf(g[i], w, gs);
    }
    s = warp_sum(s);
    fp = warp_sum(fp);
    s2 = warp_sum(s2);
    gs = warp_sum(gs);
    const float inv2 = s2 == 0.0f ? 0.0f : 1.0f / s2;
    gs *= inv2;
    const float q = per / s;
    const float at = q * fmaf(-cb, fp / s, 2.0f * a.c_z * (m + logf(s))), qf = q * cb;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float x = exp_from(v[i], m);
        const float w = key[i] >= thr ? exp_from(v[i], m2) : 0.0f;
        v[i] = x * fmaf(qf, f[i], at);
        if (key[i] >= thr)
            v[i] = fmaf(w, inv2 * (g[i] - gs), v[i]);
    }
    store_row<VEC, N>(a, t, lane, v);
}

template <int VEC, int N>
__global__ void __launch_bounds__(kRouteWarps * 32, route_ctas(N)) k_route_backward(RouteBackArgs a)
{
    extern __shared__ __align__(16) uint8_t rb_smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int E = a.E, Ep = (E + 3) & ~3;
    float *share = reinterpret_cast<float *>(rb_smem);  // [Ep] f_e
    float *gw = share + Ep + warp * Ep;                 // [Ep] of this warp: dL/dw, zero between rows
    __shared__ unsigned long long total;
    const float kNegInf = -__int_as_float(0x7f800000);
    for (int e = tid; e < (kRouteWarps + 1) * Ep; e += kRouteWarps * 32)
        share[e] = 0.0f;
    if (tid == 0)
        total = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    float per = 0.0f;  // d_loss / N
    if (a.counts) {
        // 64 bits: counts summed over many batches may each come near 2^31
        unsigned long long n = 0;
        for (int e = tid; e < E; e += kRouteWarps * 32)
            n += (unsigned)__ldg(&a.counts[e]);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1)
            n += __shfl_xor_sync(0xffffffffu, n, o);
        if (lane == 0)
            atomicAdd(&total, n);
        __syncthreads();
        const float R = total ? (float)total : 1.0f;
        for (int e = tid; e < E; e += kRouteWarps * 32)
            share[e] = (float)__ldg(&a.counts[e]) / R;
        per = (a.d_loss ? __ldg(a.d_loss) : 1.0f) / (float)max(__ldg(&a.counts[E]), 1);
        __syncthreads();
    }
    const float cb = a.c_bal * (float)E;

    for (int t = blockIdx.x * kRouteWarps + warp; t < a.T; t += gridDim.x * kRouteWarps) {
        float v[N];  // the logits, then the gradient
        float m = kNegInf;
        bool live = !a.mask || a.mask[t];
        int e = MOE_EMPTY_SLOT;
        float ge = 0.0f, ze = kNegInf;  // the lane's slot: expert, gradient, logit
        if (live) {
            if (a.d_w && lane < a.k1) {
                e = a.idx[(size_t)t * a.k1 + lane];
                ge = a.d_w[(size_t)t * a.k1 + lane];
            }
            load_row<VEC, N>(a.logits + (size_t)t * E, E, lane, v);
            if ((unsigned)e >= (unsigned)E) {
                if (e != MOE_EMPTY_SLOT)
                    set_status(a.status, MOE_ERR_DEVICE_CHECK);
                e = -1;
                ge = 0.0f;
            } else {
                ze = __ldcg(a.logits + (size_t)t * E + e);
            }
#pragma unroll
            for (int i = 0; i < N; ++i)
                m = fmaxf(m, v[i]);
            m = warp_max(m);
            if (m == kNegInf) {  // -inf alone (no distribution) or NaN among it
                bool nan = false;
#pragma unroll
                for (int i = 0; i < N; ++i)
                    nan |= v[i] != v[i];
                live = __any_sync(0xffffffffu, nan);
            }
        }
        if (!live) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] = 0.0f;
            store_row<VEC, N>(a, t, lane, v);
            continue;
        }
        // K2 as "z >= thr"; the general row where that is not it
        float thr = -kNegInf;
        bool simple = true;
        if (a.d_w) {
            // the slots' gradients by expert; repeated experts add in slot order
            const unsigned same = __match_any_sync(0xffffffffu, e);
            const bool again = e >= 0 && (same & ((1u << lane) - 1u));  // not its expert's first
            if (e >= 0 && !again)
                gw[e] = ge;
            __syncwarp();
            if (__any_sync(0xffffffffu, again))
                for (int s = 0; s < a.k1; ++s) {
                    if (lane == s && again)
                        gw[e] += ge;
                    __syncwarp();
                }
            simple = a.k2 >= E || border_value<N>(v, a.k2, m, thr);
            if (a.k2 >= E)
                thr = kNegInf;
            simple = simple && !__any_sync(0xffffffffu, e >= 0 && !(ze >= thr));
        }
        if (!simple) {
            route_row_general<VEC, N>(a, t, e, gw, share, lane, m, per, cb);
        } else {
            // dz = e^(z - m) (1/S2 (g - sum g w) in K2  +  per/S (cb (f - sum f p) + 2 c_z lse))
            float s = 0.0f, fp = 0.0f, s2 = 0.0f;
            float gs = ge * (e >= 0 ? exp_from(ze, m) : 0.0f);
            // the exponentials are kept (their unit has an eighth of the rate),
            // f and g are read again
            float x[N];
#pragma unroll
            for (int i = 0; i < N; i += VEC) {
                float f[VEC];
                smem_vec<VEC>(share, E, row_index<VEC>(i, lane), f);
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    x[i + k] = exp_from(v[i + k], m);
                    s += x[i + k];
                    fp = fmaf(f[k], x[i + k], fp);
                    if (v[i + k] >= thr)
                        s2 += x[i + k];
                }
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) {
                s += __shfl_xor_sync(0xffffffffu, s, o);
                fp += __shfl_xor_sync(0xffffffffu, fp, o);
                s2 += __shfl_xor_sync(0xffffffffu, s2, o);
                gs += __shfl_xor_sync(0xffffffffu, gs, o);
            }
            const float inv2 = s2 == 0.0f ? 0.0f : 1.0f / s2;  // 0: no weights asked for
            gs *= inv2;
            const float inv = 1.0f / s, q = per * inv;
            const float at = q * fmaf(-cb, fp * inv, 2.0f * a.c_z * (m + logf(s))), qf = q * cb;
#pragma unroll
            for (int i = 0; i < N; i += VEC) {
                float f[VEC], g[VEC];
                smem_vec<VEC>(share, E, row_index<VEC>(i, lane), f);
                smem_vec<VEC>(gw, E, row_index<VEC>(i, lane), g);
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    float c = fmaf(qf, f[k], at);
                    if (v[i + k] >= thr)
                        c = fmaf(g[k] - gs, inv2, c);
                    v[i + k] = x[i + k] * c;
                }
            }
            store_row<VEC, N>(a, t, lane, v);
        }
        __syncwarp();
        if (e >= 0)
            gw[e] = 0.0f;
        __syncwarp();
    }
}

inline size_t route_backward_smem_bytes(int E)
{
    return sizeof(float) * (kRouteWarps + 1) * ((E + 3) & ~3);
}

}  // namespace moe

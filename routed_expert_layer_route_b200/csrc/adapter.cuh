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
// two weight gradients are one contraction too, so three steps do it all:
//   inner    u (or v) of every row, k_ad_inner;
//   product  y (or dx): k_ad_rows streams W once for up to kAdRows rows,
//            k_ad_gemm (adapter_gemm.cuh) runs on the tensor cores beyond;
//   outer    dA and dB in one launch, k_ad_outer.
//
// u passes between the steps as three bf16 parts, each the bf16 nearest to
// what the parts before it leave: together the 24 bits of a float32, so that
// u can be an operand of bf16 matrix instructions without the 2^-8 that one
// bf16 would cost the float32 outputs (two parts: 2^-17, which still shows).
#pragma once
#include "common.cuh"
#include "route.cuh"

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

constexpr int kAdParts = 3;
constexpr int kAdMaxR = 128;  // ranks

// The parts of u; a value beyond the finite numbers is all in the first, and a
// finite one that would round to an infinity has the largest bf16 there.
MOE_DEVINL void split_bf16(float v, uint16_t (&part)[kAdParts])
{
    part[0] = f32_to_bf16_rn(v);
    if ((part[0] & 0x7fffu) == 0x7f80u && fabsf(v) < __int_as_float(0x7f800000))
        part[0] -= 1;
    const bool finite = (part[0] & 0x7f80u) != 0x7f80u;
#pragma unroll
    for (int i = 1; i < kAdParts; ++i) {
        v -= bf16_to_f32(part[i - 1]);
        part[i] = finite ? f32_to_bf16_rn(v) : (uint16_t)0;
    }
}

// The parts' rows: kAdParts x rp values, rp = r rounded up to 16, zeros behind r.
MOE_DEVINL int ad_rp(int r) { return (r + 15) & ~15; }

// D (16 x 8, float32) += A (16 x 16) B (16 x 8), bf16.
MOE_DEVINL void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                         uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The matrix instructions' running sum rounds towards zero at each step of 16
// products, so what it loses grows with K.  One sum takes kAdSteps of them at most;
// the sums of a longer K are added up rounded.  u of 2500 rows at K = 4096 and 16384:
// 2.4e-7 off 64 bits, where sums of any length had 1.0e-6 and 4.4e-6 and a float32
// product has 1.5e-7 and 3.2e-7; 8192 rows of 4096, rank 32, take 2 us more with it
// (48 steps: 1 us, 7e-7).
constexpr int kAdSteps = 16;

MOE_DEVINL void cp_async16(uint32_t dst, const void *src, bool live)
{
    const int n = live ? 16 : 0;  // 0: zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
}
MOE_DEVINL void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
MOE_DEVINL void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
MOE_DEVINL void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// Fragments straight from row-major memory: a thread (g = lane / 4,
// q = lane % 4) loads the 16 bytes at K offset 32 c + 8 q of its row and feeds
// them to two matrix instructions as elements (2q, 2q+1, 2q+8, 2q+9) of each.
// That permutes K inside a chunk of 32, the same way for both operands, so
// the products pair up and their sum is the same set.
constexpr int kAdChunk = 32;

MOE_DEVINL uint4 ad_chunk(const uint16_t *row, int k, int K, bool live)
{
    return live && k < K ? __ldg(reinterpret_cast<const uint4 *>(row + k))
                         : make_uint4(0u, 0u, 0u, 0u);
}

// ---------------------------------------------------------------------------
// Rows grouped by adapter, in order inside a group (rows without one left
// out): one CTA of W warps, each warp a run of at most 32 IDS rows that its
// lanes hold, its counts of every adapter in shared memory of its own; then
// the counts' prefix over adapters and warps gives each warp its places.
// sg: ad_group_smem_bytes, zeroed here.
struct AdGroupArgs {
    const int32_t *adapter;  // [T]
    int32_t *offsets;        // [n + 1]
    int32_t *row;            // [offsets[n]]
    int T, n;
    int *status;
};

inline size_t ad_group_smem_bytes(int n, int warps) { return sizeof(int) * (size_t)n * (warps + 2); }

template <int W, int IDS>
MOE_DEVINL void ad_group(const AdGroupArgs &p, int *sg, int tid)
{
    __shared__ int scan[40];
    const int warp = tid >> 5, lane = tid & 31;
    int *start = sg + p.n * (W + 1);
    const int run = ((p.T + W - 1) / W + 31) & ~31;
    const int t0 = warp * run + lane;
    int id[IDS];  // every row of the run at once
    unsigned same[IDS];
#pragma unroll
    for (int i = 0; i < IDS; ++i)
        id[i] = 32 * i < run && t0 + 32 * i < p.T ? __ldg(&p.adapter[t0 + 32 * i]) : MOE_EMPTY_SLOT;
    for (int i = tid; i < p.n * (W + 1); i += W * 32)
        sg[i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < IDS; ++i) {
        if (32 * i >= run)
            break;
        if ((unsigned)id[i] >= (unsigned)p.n) {
            if (id[i] != MOE_EMPTY_SLOT)
                set_status(p.status, MOE_ERR_DEVICE_CHECK);
            id[i] = -1;
        }
        same[i] = __match_any_sync(0xffffffffu, id[i]);
        if (id[i] >= 0 && (int)__ffs(same[i]) - 1 == lane)
            sg[id[i] * (W + 1) + warp] += __popc(same[i]);
        __syncwarp();
    }
    __syncthreads();
    // per adapter: exclusive prefix over the warps and the total
    for (int a = tid; a < p.n; a += W * 32) {
        int sum = 0;
        for (int w = 0; w < W; ++w) {
            const int c = sg[a * (W + 1) + w];
            sg[a * (W + 1) + w] = sum;
            sum += c;
        }
        start[a] = sum;
    }
    __syncthreads();
    const int total = block_exclusive_scan(start, p.n, scan);
    for (int a = tid; a < p.n; a += W * 32)
        p.offsets[a] = start[a];
    if (tid == 0)
        p.offsets[p.n] = total;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < IDS; ++i) {
        if (32 * i >= run)
            break;
        const int a = id[i];
        int base = 0;
        if (a >= 0)
            base = start[a] + sg[a * (W + 1) + warp];
        __syncwarp();
        if (a >= 0) {
            p.row[base + __popc(same[i] & ((1u << lane) - 1u))] = t0 + 32 * i;
            if ((int)__ffs(same[i]) - 1 == lane)
                sg[a * (W + 1) + warp] += __popc(same[i]);
        }
        __syncwarp();
    }
}

constexpr int kAdGroupWarps = 32, kAdGroupIds = 16;
constexpr int kAdGroupMaxN = 256, kAdGroupMaxT = kAdGroupWarps * 32 * kAdGroupIds;

__global__ void __launch_bounds__(kAdGroupWarps * 32) k_ad_group(AdGroupArgs p)
{
    extern __shared__ int sg[];
    pdl_wait();
    pdl_trigger();
    ad_group<kAdGroupWarps, kAdGroupIds>(p, sg, threadIdx.x);
}

// ---------------------------------------------------------------------------
// Inner products: u[t][j] = s_a <x_t, A_a[j]>, 0 for rows without an adapter.
struct AdInnerArgs {
    const uint16_t *x;       // [T x din]
    const uint16_t *a;       // [n x r x din]
    const int32_t *adapter;  // [T]
    const int32_t *row;      // nullable: the rows in an order grouped by adapter,
    const int32_t *rows;     //   and how many those are (rows without adapter left out)
    const float *scale;      // nullable [n]
    uint16_t *parts;         // [T][kAdParts][rp]
    float *u_out;            // nullable [T x r]
    const float *conv;       // nullable [T x r]: given u to split into conv_parts
    uint16_t *conv_parts;    // [T][kAdParts][rp]
    int T, din, r, n;
    int zero_u;              // clear u_out in rows without an adapter (k_ad_inner_big)
    int lists;               // CTAs that share a row tile's adapters
    int inner_ctas;          // CTAs of the inner products; those behind them convert
    int grouping;            // one more CTA (of blockIdx.y 0) groups the rows
    AdGroupArgs group;
    int *status;
};

constexpr int kAdWarps = 8;            // warps, which split K
constexpr int kAdSmallGroupT = 2048;  // most rows that one of its CTAs groups

MOE_DEVINL void ad_put_parts(uint16_t *parts, int rp, int t, int j, float v)
{
    uint16_t q[kAdParts];
    split_bf16(v, q);
#pragma unroll
    for (int i = 0; i < kAdParts; ++i)
        parts[((size_t)t * kAdParts + i) * rp + j] = q[i];
}

// The CTAs behind the inner products: the given u into its parts, and zeros
// for rows without an adapter.
MOE_DEVINL void ad_convert(const AdInnerArgs &p, int tid)
{
    const int rp = ad_rp(p.r);
    const int64_t step =
        (int64_t)(gridDim.x - p.grouping - p.inner_ctas) * gridDim.y * blockDim.x;
    const int64_t first =
        ((int64_t)(blockIdx.x - p.inner_ctas) * gridDim.y + blockIdx.y) * blockDim.x + tid;
    // rows without an adapter
    for (int64_t i = first; p.zero_u && i < (int64_t)p.T * p.r; i += step)
        if ((unsigned)__ldg(&p.adapter[i / p.r]) >= (unsigned)p.n)
            p.u_out[i] = 0.0f;
    // eight ranks of a row at a time
    for (int64_t i = first; p.conv && i < (int64_t)p.T * (rp / 8); i += step) {
        const int t = (int)(i / (rp / 8)), j = (int)(i % (rp / 8)) * 8;
        uint16_t q[kAdParts][8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            uint16_t part[kAdParts];
            split_bf16(j + k < p.r ? __ldg(&p.conv[(size_t)t * p.r + j + k]) : 0.0f, part);
#pragma unroll
            for (int h = 0; h < kAdParts; ++h)
                q[h][k] = part[h];
        }
#pragma unroll
        for (int h = 0; h < kAdParts; ++h)
            *reinterpret_cast<uint4 *>(&p.conv_parts[((size_t)t * kAdParts + h) * rp + j]) =
                make_uint4(q[h][0] | (uint32_t)q[h][1] << 16, q[h][2] | (uint32_t)q[h][3] << 16,
                           q[h][4] | (uint32_t)q[h][5] << 16, q[h][6] | (uint32_t)q[h][7] << 16);
    }
}

// A tile's R <= 32 rows (st, -1: none) with their adapters (sa), and the
// distinct ones in order of appearance, by a match in one warp; all threads of
// the CTA, which gets their count.
template <int R>
MOE_DEVINL int ad_tile_list(const AdInnerArgs &p, int i0, int rows, int tid, int *sa, int *st,
                            int *list, int *count)
{
    if (tid < 32) {
        int t = -1, a = -1;
        if (tid < min(rows, R)) {
            t = p.row ? __ldcg(&p.row[i0 + tid]) : i0 + tid;
            if ((unsigned)t < (unsigned)p.T)
                a = adapter_of(p.adapter, t, p.n, p.status);
            else
                t = -1;
        }
        if (tid < R) {
            st[tid] = t;
            sa[tid] = a;
        }
        const unsigned same = __match_any_sync(0xffffffffu, a);
        const bool first = a >= 0 && (int)__ffs(same) - 1 == tid;
        const unsigned firsts = __ballot_sync(0xffffffffu, first);
        if (first)
            list[__popc(firsts & ((1u << tid) - 1u))] = a;
        if (tid == 0)
            *count = __popc(firsts);
    }
    __syncthreads();
    return *count;
}

// One CTA for 16 rows, 8 NT ranks (blockIdx.y) and every lists-th of the
// rows' distinct adapters.  Its warps take the chunks of K in turn, so the
// CTA reads whole 512-byte pieces of its rows, and add up through shared
// memory.  A pass over K for each distinct adapter computes all rows and
// keeps those that are its own: rows of one request mostly stand together,
// so a tile has one or two adapters; where every row has another (a decode
// batch), the lists spread the adapters, whose matrices have to be read
// anyway, over CTAs.  Bound by the reads of x and of the adapters.
template <int NT>
__global__ void __launch_bounds__(kAdWarps * 32, NT >= 8 ? 1 : 2) k_ad_inner(AdInnerArgs p)
{
    constexpr int MT = 1, kRows = 16;
    __shared__ float red[kAdWarps / 2][kRows][8 * NT + 1];
    __shared__ int sa[kRows], st[kRows];  // adapter and row
    __shared__ int s_list[kRows];
    __shared__ int s_count;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, q = lane & 3;
    const int rp = ad_rp(p.r);
    pdl_wait();
    pdl_trigger();
    if ((int)blockIdx.x >= p.inner_ctas) {
        if (p.grouping && blockIdx.x == gridDim.x - 1) {
            extern __shared__ int sg[];
            if (blockIdx.y == 0)
                ad_group<kAdWarps, kAdSmallGroupT / (kAdWarps * 32)>(p.group, sg, tid);
            return;
        }
        ad_convert(p, tid);
        return;
    }
    const int tiles = p.inner_ctas / p.lists;  // part 0 of all tiles first: most tiles have no more
    const int tile = blockIdx.x % tiles, part = blockIdx.x / tiles;
    const int i0 = tile * kRows, j0 = blockIdx.y * 8 * NT;
    const int rows = min(kRows, (p.row ? __ldcg(p.rows) : p.T) - i0);
    if (rows <= 0)
        return;
    const int count = ad_tile_list<kRows>(p, i0, rows, tid, sa, st, s_list, &s_count);
    const int nc = (p.din + kAdChunk - 1) / kAdChunk;
    const uint16_t *xr[2 * MT];
    bool has[2 * MT];
#pragma unroll
    for (int m = 0; m < 2 * MT; ++m) {
        const int t = st[8 * m + g];
        has[m] = t >= 0;
        xr[m] = p.x + (size_t)(has[m] ? t : 0) * p.din;
    }
    for (int l = part; l < count; l += p.lists) {
        const int a = s_list[l];
        const uint16_t *ap = p.a + ((size_t)a * p.r + j0 + g) * p.din;
        constexpr int kSegment = kAdWarps * kAdSteps / 2;  // chunks of one running sum of every warp
        for (int s0 = 0; s0 < nc; s0 += kSegment) {
            float acc[MT][NT][4];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    acc[m][i][0] = acc[m][i][1] = acc[m][i][2] = acc[m][i][3] = 0.0f;
            const int s1 = min(nc, s0 + kSegment);
#pragma unroll(NT <= 2 ? 8 : 4)
            for (int c = s0 + warp; c < s1; c += kAdWarps) {
                const int k = c * kAdChunk + 8 * q;
                uint4 u[2 * MT];
#pragma unroll
                for (int m = 0; m < 2 * MT; ++m)
                    u[m] = ad_chunk(xr[m], k, p.din, has[m]);
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const uint4 w = ad_chunk(ap + (size_t)i * 8 * p.din, k, p.din,
                                             j0 + 8 * i + g < p.r);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        mma_bf16(acc[m][i], u[2 * m].x, u[2 * m + 1].x, u[2 * m].y, u[2 * m + 1].y,
                                 w.x, w.y);
                        mma_bf16(acc[m][i], u[2 * m].z, u[2 * m + 1].z, u[2 * m].w, u[2 * m + 1].w,
                                 w.z, w.w);
                    }
                }
            }
            // the upper warps' sums of this adapter's rows, then the lower ones' added
#pragma unroll
            for (int half = 1; half >= 0; --half) {
                if (warp / (kAdWarps / 2) == half)
#pragma unroll
                    for (int m = 0; m < 2 * MT; ++m)
                        if (sa[8 * m + g] == a)
#pragma unroll
                            for (int i = 0; i < NT; ++i)
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    float &to =
                                        red[warp % (kAdWarps / 2)][8 * m + g][8 * i + 2 * q + h];
                                    const float v = acc[m / 2][i][2 * (m & 1) + h];
                                    to = half && s0 == 0 ? v : to + v;
                                }
                __syncthreads();
            }
        }
    }
    // the rows of this CTA's adapters (part 0: those without one too)
    for (int i = tid; i < kRows * 8 * NT; i += kAdWarps * 32) {
        const int row = i / (8 * NT), jj = i % (8 * NT), j = j0 + jj, t = st[row];
        if (t < 0 || j >= rp)
            continue;
        const int a = sa[row];
        bool mine = a < 0 && part == 0;
        for (int l = part; l < count; l += p.lists)
            mine |= s_list[l] == a;
        if (!mine)
            continue;
        float v = 0.0f;
        if (a >= 0) {
#pragma unroll
            for (int w = 0; w < kAdWarps / 2; ++w)
                v += red[w][row][jj];
            if (p.scale)
                v *= __ldg(&p.scale[a]);
        }
        ad_put_parts(p.parts, rp, t, j, j < p.r ? v : 0.0f);
        if (p.u_out && j < p.r)
            p.u_out[(size_t)t * p.r + j] = v;
    }
}

// The same for many rows (8 NT >= r of blockIdx.y): 32 rows a CTA and every
// lists-th of their adapters, one after another.  x and A_a stream through
// shared memory in stages of 128 values of K, four deep, by asynchronous
// copies that gather the rows (one bulk copy a row and stage was slower: 95
// against 33 us for 8192 rows of 4096, rank 32, the projection of 8 outputs
// included); a warp multiplies 16 rows with half of the ranks over a part of a
// stage, all its fragments loaded before the first product (a few warps hide
// little latency).  Meant to be bound by the read of x; it waits for its stages
// instead: 2.0 TB/s at rank 32 (8192 rows of 4096), a third of the copy bandwidth,
// and 1.1 TB/s at rank 64 (8192 rows of 2048), a sixth.  An adapter's matrix is
// read, from L2, once for each 32 rows that have it (64 rows would halve that but
// leave one CTA an SM: 43 against 33 us for the same rows).
constexpr int kAdBigWarps = 16;
constexpr int kAdBigGroupT = 4096;  // most rows that one of its CTAs groups

template <int NT>
struct AdBigShape {
    static constexpr int kRows = 32, kK = 128, kStages = 4;
    static constexpr int kPitch = kK * 2 + 16;  // bytes; 16 over: rows on other banks
    static constexpr int kStage = (kRows + 8 * NT) * kPitch;
    static constexpr int kBytes = kStages * kStage;
    static constexpr int kRedPitch = 8 * NT + 1;  // the halves' sums, in the stages' place
};

// An array that is to lie in local memory: the registers are the main loop's (64
// with two CTAs an SM; with 16 more values among them 8192 rows of 2048, rank 64,
// take 7 us more).
template <int N>
MOE_DEVINL float *ad_local(float (&v)[N])
{
    float *p = v;
    asm volatile("" : "+l"(p)::"memory");
    return p;
}

template <int NT>
__global__ void __launch_bounds__(kAdBigWarps * 32) k_ad_inner_big(AdInnerArgs p)
{
    using S = AdBigShape<NT>;
    constexpr int R = S::kRows;
    extern __shared__ __align__(16) uint8_t ab_smem[];
    __shared__ int sa[S::kRows], st[S::kRows], s_list[S::kRows];
    __shared__ int s_count;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rp = ad_rp(p.r);
    pdl_wait();
    pdl_trigger();
    if ((int)blockIdx.x >= p.inner_ctas) {
        if (p.grouping && blockIdx.x == gridDim.x - 1) {
            if (blockIdx.y == 0)
                ad_group<kAdBigWarps, kAdBigGroupT / (kAdBigWarps * 32)>(
                    p.group, reinterpret_cast<int *>(ab_smem), tid);
            return;
        }
        ad_convert(p, tid);
        return;
    }
    const int tiles = p.inner_ctas / p.lists;  // part 0 of all tiles first: most tiles have no more
    const int tile = blockIdx.x % tiles, part = blockIdx.x / tiles;
    const int i0 = tile * S::kRows, j0 = blockIdx.y * 8 * NT;
    const int rows = min(S::kRows, (p.row ? __ldcg(p.rows) : p.T) - i0);
    if (rows <= 0)
        return;
    const int count = ad_tile_list<S::kRows>(p, i0, rows, tid, sa, st, s_list, &s_count);
    const uint32_t sm = smem_addr(ab_smem);
    float *red = reinterpret_cast<float *>(ab_smem);
    const int ns = (p.din + S::kK - 1) / S::kK;
    constexpr int kMT = R / 16, kKG = kAdBigWarps / (2 * kMT);  // row tiles, parts of a stage
    constexpr int NH = NT / 2, KS = S::kK / 16 / kKG;           // instructions of N and of K
    constexpr int kSegment = kAdSteps / KS;                     // stages of one running sum
    const int mt = warp % kMT, nh = warp / kMT % 2, kh = warp / (2 * kMT);
    // this thread's vectors of a stage: column ck of row tid / 16 of x, then of
    // ranks tid / 16, + 32 of the adapter; nullptr: zeros
    constexpr int kVec = 1 + (NT + 3) / 4;
    const int ck = (tid & 15) * 8, r0 = tid >> 4;
    const uint32_t to0 = sm + r0 * S::kPitch + ck * 2;
    const uint16_t *src[kVec];
    src[0] = st[r0] >= 0 ? p.x + (size_t)st[r0] * p.din + ck : nullptr;
    for (int l = part; l < count; l += p.lists) {
        const int a = s_list[l];
#pragma unroll
        for (int v = 1; v < kVec; ++v) {
            const int j = j0 + r0 + 32 * (v - 1);
            src[v] = j < p.r && j < j0 + 8 * NT ? p.a + ((size_t)a * p.r + j) * p.din + ck : nullptr;
        }
        auto issue = [&](int s) {
            if (s < ns) {
                const uint32_t to = to0 + (s % S::kStages) * S::kStage;
                const bool in = s * S::kK + ck < p.din;
#pragma unroll
                for (int v = 0; v < kVec; ++v) {
                    if (r0 + 32 * v >= S::kRows + 8 * NT)
                        continue;
                    const bool live = in && src[v];
                    cp_async16(to + 32 * v * S::kPitch, live ? src[v] + s * S::kK : p.x, live);
                }
            }
            cp_async_commit();
        };
        float acc[NH][4];
        float done[NH * 4];  // sums of the segments before: in local memory, seldom used
#pragma unroll
        for (int i = 0; i < NH; ++i)
            acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
        __syncthreads();  // the adapter before is done with the stages
#pragma unroll
        for (int s = 0; s < S::kStages - 1; ++s)
            issue(s);
        for (int s0 = 0; s0 < ns; s0 += kSegment) {
            const int s1 = min(ns, s0 + kSegment);
            for (int s = s0; s < s1; ++s) {
                cp_async_wait<S::kStages - 2>();
                __syncthreads();
                issue(s + S::kStages - 1);
                const uint32_t at = sm + (s % S::kStages) * S::kStage + kh * KS * 32;
                uint32_t x[KS][4], w[KS][NH == 1 ? 1 : NH / 2][4];
#pragma unroll
                for (int kk = 0; kk < KS; ++kk) {
                    ldmatrix_x4(at + (mt * 16 + (lane & 15)) * S::kPitch + kk * 32 + (lane >> 4) * 16,
                                x[kk]);
                    if (NH == 1) {
                        const uint32_t addr = at + (S::kRows + nh * 8 + (lane & 7)) * S::kPitch +
                                              kk * 32 + ((lane >> 3) & 1) * 16;
                        asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];"
                                     : "=r"(w[kk][0][0]), "=r"(w[kk][0][1])
                                     : "r"(addr)
                                     : "memory");
                    } else {
#pragma unroll
                        for (int i = 0; i < NH / 2; ++i)  // two blocks of eight ranks
                            ldmatrix_x4(at + (S::kRows + nh * 8 * NH + i * 16 + (lane & 7) +
                                              (lane >> 4) * 8) * S::kPitch +
                                            kk * 32 + ((lane >> 3) & 1) * 16,
                                        w[kk][i]);
                    }
                }
#pragma unroll
                for (int kk = 0; kk < KS; ++kk)
#pragma unroll
                    for (int i = 0; i < NH; ++i)
                        mma_bf16(acc[i], x[kk][0], x[kk][1], x[kk][2], x[kk][3], w[kk][i / 2][2 * (i & 1)],
                                 w[kk][i / 2][2 * (i & 1) + 1]);
            }
            if (s1 < ns) {  // sums of a segment, added rounded
                float *to = ad_local(done);
#pragma unroll
                for (int i = 0; i < NH; ++i)
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        to[i * 4 + h] = s0 == 0 ? acc[i][h] : to[i * 4 + h] + acc[i][h];
                        acc[i][h] = 0.0f;
                    }
            }
        }
        cp_async_wait<0>();
        __syncthreads();
        if (ns > kSegment) {
            const float *from = ad_local(done);
#pragma unroll
            for (int i = 0; i < NH; ++i)
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    acc[i][h] += from[i * 4 + h];
        }
        // the parts of K meet
        if (kh > 0) {
            float *mine = red + (kh - 1) * R * S::kRedPitch;
#pragma unroll
            for (int i = 0; i < NH; ++i)
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    mine[(mt * 16 + (lane >> 2) + 8 * (h >> 1)) * S::kRedPitch + nh * 8 * NH + i * 8 +
                        2 * (lane & 3) + (h & 1)] = acc[i][h];
        }
        __syncthreads();
        if (kh > 0)
            continue;
        const float sc = p.scale ? __ldg(&p.scale[a]) : 1.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = mt * 16 + (lane >> 2) + 8 * h;
            if (sa[row] != a)
                continue;
            const int t = st[row];
#pragma unroll
            for (int i = 0; i < NH; ++i) {
                const int jj = nh * 8 * NH + i * 8 + 2 * (lane & 3), j = j0 + jj;
                if (j >= rp)
                    continue;
                // two ranks side by side (rp is even)
                float v0 = acc[i][2 * h], v1 = acc[i][2 * h + 1];
#pragma unroll
                for (int k = 0; k < kKG - 1; ++k) {
                    v0 += red[(k * R + row) * S::kRedPitch + jj];
                    v1 += red[(k * R + row) * S::kRedPitch + jj + 1];
                }
                v0 = j < p.r ? v0 * sc : 0.0f;
                v1 = j + 1 < p.r ? v1 * sc : 0.0f;
                uint16_t q0[kAdParts], q1[kAdParts];
                split_bf16(v0, q0);
                split_bf16(v1, q1);
#pragma unroll
                for (int k = 0; k < kAdParts; ++k)
                    *reinterpret_cast<uint32_t *>(
                        &p.parts[((size_t)t * kAdParts + k) * rp + j]) =
                        (uint32_t)q0[k] | ((uint32_t)q1[k] << 16);
                if (p.u_out) {
                    if (j < p.r)
                        p.u_out[(size_t)t * p.r + j] = v0;
                    if (j + 1 < p.r)
                        p.u_out[(size_t)t * p.r + j + 1] = v1;
                }
            }
        }
    }
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
    const uint16_t *parts;   // [T][kAdParts][rp] of u
    void *y;                 // [T x dout]
    int y_bf16;
    int T, din, dout, r, n;
    int segment;             // k_ad_gemm: most K blocks that one tensor-memory sum takes
    int splits;              // k_ad_gemm: parts of K; above 1 their sums go to partial
    float *partial;          // [tiles][splits][256 x kAGSplitCols]
    WsHeader *hdr;
};

// The adapter's part of one output: sum_j u_j B_a[j][o], in order of j.
MOE_DEVINL float ad_part(const AdProductArgs &p, int a, int t, int o)
{
    const int rp = ad_rp(p.r);
    const uint16_t *u = p.parts + (size_t)t * kAdParts * rp;
    const uint16_t *b = p.b + (size_t)a * p.r * p.dout + o;
    float v = 0.0f;
#pragma unroll 8
    for (int j = 0; j < p.r; ++j) {
        float x = bf16_to_f32(__ldcg(&u[j]));
#pragma unroll
        for (int i = 1; i < kAdParts; ++i)
            x += bf16_to_f32(__ldcg(&u[i * rp + j]));
        v = fmaf(x, bf16_to_f32(__ldg(&b[(size_t)j * p.dout])), v);
    }
    return v;
}

constexpr int kAdRows = 64;       // most rows of k_ad_rows
constexpr int kAdOneRanks = 16;   // most row-ranks of the one-launch form
struct AdOne {                    // what the one-launch form needs of the inner step
    const uint16_t *a;
    const float *scale;
    float *u_out;
};

// Few rows: one CTA for 16 outputs of 8 NT >= T rows.  W is the M side of the
// matrix instruction and is read once, straight into fragments, its chunks of
// K split over the warps and all of a phase's chunks in flight together; the
// rows are the N side, brought to shared memory a phase at a time by
// asynchronous copies.  The sums meet in shared memory, where the adapter's
// part joins: eight lanes a row (two vectors of eight outputs, a quarter of
// the ranks each), whose first rows of B_a are on their way from the start.
// Bound by the read of W and, from about 16 rows on, by each CTA's read of x
// from L2.
//
// After the inner kernel (ONE false), W x and B_a need nothing of it, so they
// come before the wait for it: the inner kernel lets this one start only after
// its own wait, when every earlier kernel (which may have made x) is complete.
// ONE: rows x ranks <= kAdOneRanks, one or a few rows; every CTA computes u
// itself, a rank to a warp in turn, which reads the rows' adapters once for
// each CTA (from L2) but saves a launch and its wait (one row, 2048 to 128,
// rank 16: 6.9 -> 5.2 us).
// 32 rows, 2048 to 2048, rank 16, each row its own adapter: 8.5 us with the
// inner launch, for 12.9 MB that have to be read (2.0 us).
template <int NT>
struct AdRowsShape {
    static constexpr int kDeep = NT <= 4 ? 8 : 4;              // chunks of a warp in a phase
    static constexpr int kPhase = kDeep * kAdWarps * kAdChunk;  // values of K
    static_assert(2 * kDeep <= kAdSteps, "a phase is one running sum");
    static constexpr int kPitch = kPhase * 2 + 64;  // bytes; 64 over: two rows on other banks
    static constexpr int kX = 8 * NT * kPitch;
    static constexpr int kRed = kAdWarps * 8 * NT * 17 * 4;
    // u takes the place of x: 8 NT rows of up to 128 ranks
    static constexpr int kBytes = (kX > 8 * NT * kAdMaxR * 4 ? kX : 8 * NT * kAdMaxR * 4) + kRed;
};

template <int NT, bool ONE>
__global__ void __launch_bounds__(kAdWarps * 32) k_ad_rows(AdProductArgs p, AdOne one)
{
    using S = AdRowsShape<NT>;
    extern __shared__ __align__(16) uint8_t ar_smem[];
    float *su = reinterpret_cast<float *>(ar_smem);  // [rows][r], after x
    float(*red)[8 * NT][17] =
        reinterpret_cast<float(*)[8 * NT][17]>(ar_smem + S::kBytes - S::kRed);
    __shared__ float su_one[ONE ? kAdOneRanks : 1];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, q = lane & 3;
    const int o0 = blockIdx.x * 16;
    if (ONE) {
        pdl_wait();
        pdl_trigger();
    }
    const bool lo_row = o0 + g < p.dout, hi_row = o0 + g + 8 < p.dout;
    const uint16_t *w0 = p.w + (size_t)(lo_row ? o0 + g : 0) * p.din;
    const uint16_t *w1 = p.w + (size_t)(hi_row ? o0 + g + 8 : 0) * p.din;
    const int K = p.w ? p.din : 0;
    const uint32_t sx = smem_addr(ar_smem);
    uint4 w[S::kDeep][2];
    auto fetch = [&](int k0) {
#pragma unroll
        for (int d = 0; d < S::kDeep; ++d) {
            const int k = k0 + (warp + d * kAdWarps) * kAdChunk + 8 * q;
            w[d][0] = ad_chunk(w0, k, K, lo_row);
            w[d][1] = ad_chunk(w1, k, K, hi_row);
        }
        for (int i = tid; i < 8 * NT * (S::kPhase / 8); i += kAdWarps * 32) {
            const int t = i / (S::kPhase / 8), c = i % (S::kPhase / 8) * 8;
            if (k0 + c >= ((K + kAdChunk - 1) & ~(kAdChunk - 1)))
                continue;  // behind the last chunk: not read
            const bool live = t < p.T && k0 + c < K;
            cp_async16(sx + t * S::kPitch + c * 2, p.x + (live ? (size_t)t * p.din + k0 + c : 0), live);
        }
        cp_async_commit();
    };
    if (K)
        fetch(0);
    // this thread's part of the adapters: row, vector of outputs, ranks jg, jg + 4, ...
    const int jg = tid & 3, ov = o0 + (tid >> 2 & 1) * 8;
    auto rank_row = [&](int a, int j) {
        return __ldg(reinterpret_cast<const uint4 *>(p.b + ((size_t)a * p.r + j) * p.dout + ov));
    };
    int a_of[(8 * NT + 31) / 32];
    uint4 b0[4];  // the first ranks of the first row
#pragma unroll
    for (int h = 0; h < (8 * NT + 31) / 32; ++h) {
        const int t = (tid >> 3) + 32 * h;
        a_of[h] = t < p.T && ov < p.dout ? adapter_of(p.adapter, t, p.n, &p.hdr->status) : -1;
    }
#pragma unroll
    for (int d = 0; d < 4; ++d)
        if (a_of[0] >= 0 && jg + 4 * d < p.r)
            b0[d] = rank_row(a_of[0], jg + 4 * d);
    if (ONE) {
        // u of the rows' ranks while W is on its way
        for (int i = warp; i < p.T * p.r; i += kAdWarps) {
            const int t = i / p.r, j = i % p.r;
            const int a = adapter_of(p.adapter, t, p.n, &p.hdr->status);
            float v = 0.0f;
            if (a >= 0) {
                const uint16_t *x = p.x + (size_t)t * p.din, *ar = one.a + ((size_t)a * p.r + j) * p.din;
#pragma unroll 8
                for (int k = 8 * lane; k < p.din; k += 256) {
                    const uint4 x8 = __ldg(reinterpret_cast<const uint4 *>(x + k));
                    const float xv[8] = {bf16lo(x8.x), bf16hi(x8.x), bf16lo(x8.y), bf16hi(x8.y),
                                         bf16lo(x8.z), bf16hi(x8.z), bf16lo(x8.w), bf16hi(x8.w)};
                    v = dot8_bf16(__ldg(reinterpret_cast<const uint4 *>(ar + k)), xv, v);
                }
                v = warp_sum(v);
                if (one.scale)
                    v *= __ldg(&one.scale[a]);
            }
            if (lane == 0) {
                su_one[i] = v;
                if (one.u_out && blockIdx.x == 0)
                    one.u_out[i] = v;
            }
        }
    }
    float acc[NT][4], sum[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int h = 0; h < 4; ++h)
            acc[i][h] = sum[i][h] = 0.0f;
    for (int k0 = 0; k0 < K; k0 += S::kPhase) {
        cp_async_wait<0>();
        __syncthreads();
#pragma unroll
        for (int d = 0; d < S::kDeep; ++d) {
            const int c = (warp + d * kAdWarps) * kAdChunk;
            if (k0 + c >= K)
                break;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const uint4 v = *reinterpret_cast<const uint4 *>(ar_smem + (8 * i + g) * S::kPitch +
                                                                 (c + 8 * q) * 2);
                mma_bf16(acc[i], w[d][0].x, w[d][1].x, w[d][0].y, w[d][1].y, v.x, v.y);
                mma_bf16(acc[i], w[d][0].z, w[d][1].z, w[d][0].w, w[d][1].w, v.z, v.w);
            }
        }
        __syncthreads();
        if (k0 + S::kPhase < K) {
            fetch(k0 + S::kPhase);
#pragma unroll
            for (int i = 0; i < NT; ++i)  // a phase's sums (kAdSteps at most), added rounded
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    sum[i][h] += acc[i][h];
                    acc[i][h] = 0.0f;
                }
        }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int h = 0; h < 4; ++h)
            acc[i][h] += sum[i][h];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        red[warp][8 * i + 2 * q][g] = acc[i][0];
        red[warp][8 * i + 2 * q + 1][g] = acc[i][1];
        red[warp][8 * i + 2 * q][g + 8] = acc[i][2];
        red[warp][8 * i + 2 * q + 1][g + 8] = acc[i][3];
    }
    if (!ONE) {
        pdl_wait();
        pdl_trigger();
        const int rp = ad_rp(p.r);
        for (int i = tid; i < p.T * p.r; i += kAdWarps * 32) {
            const uint16_t *u = p.parts + (size_t)(i / p.r) * kAdParts * rp + i % p.r;
            float v = bf16_to_f32(__ldcg(u));
#pragma unroll
            for (int k = 1; k < kAdParts; ++k)
                v += bf16_to_f32(__ldcg(u + k * rp));
            su[i] = v;
        }
    }
    __syncthreads();
    const float *us = ONE ? su_one : su;
#pragma unroll
    for (int h = 0; h < (8 * NT + 31) / 32; ++h) {
        const int t = (tid >> 3) + 32 * h, a = a_of[h];
        float s[8] = {};
        if (a >= 0)
            for (int j0 = 0; j0 < p.r; j0 += 16) {
                uint4 b[4];
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    if (j0 + jg + 4 * d < p.r)
                        b[d] = h == 0 && j0 == 0 ? b0[d] : rank_row(a, j0 + jg + 4 * d);
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    if (j0 + jg + 4 * d < p.r) {
                        const float u = us[t * p.r + j0 + jg + 4 * d];
                        s[0] = fmaf(u, bf16lo(b[d].x), s[0]);
                        s[1] = fmaf(u, bf16hi(b[d].x), s[1]);
                        s[2] = fmaf(u, bf16lo(b[d].y), s[2]);
                        s[3] = fmaf(u, bf16hi(b[d].y), s[3]);
                        s[4] = fmaf(u, bf16lo(b[d].z), s[4]);
                        s[5] = fmaf(u, bf16hi(b[d].z), s[5]);
                        s[6] = fmaf(u, bf16lo(b[d].w), s[6]);
                        s[7] = fmaf(u, bf16hi(b[d].w), s[7]);
                    }
            }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            s[k] += __shfl_xor_sync(0xffffffffu, s[k], 1);
            s[k] += __shfl_xor_sync(0xffffffffu, s[k], 2);
        }
        // each of the four lanes stores two of the eight outputs
        if (t >= p.T || ov >= p.dout || (!p.w && a < 0 && !p.bias))
            continue;
        float o[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float v = jg == 0 ? s[k] : jg == 1 ? s[2 + k] : jg == 2 ? s[4 + k] : s[6 + k];
            if (p.w) {
                float base = 0.0f;
#pragma unroll
                for (int wi = 0; wi < kAdWarps; ++wi)
                    base += red[wi][t][ov - o0 + 2 * jg + k];
                v += base;
            }
            if (p.bias)
                v += __ldg(&p.bias[ov + 2 * jg + k]);
            o[k] = v;
        }
        const size_t at = (size_t)t * p.dout + ov + 2 * jg;
        if (p.y_bf16) {
            uint32_t *y = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.y) + at);
            if (!p.w) {
                const uint32_t old = *y;
                o[0] += bf16lo(old);
                o[1] += bf16hi(old);
            }
            *y = (uint32_t)f32_to_bf16_rn(o[0]) | ((uint32_t)f32_to_bf16_rn(o[1]) << 16);
        } else {
            float2 *y = reinterpret_cast<float2 *>(static_cast<float *>(p.y) + at);
            if (!p.w) {
                const float2 old = *y;
                o[0] += old.x;
                o[1] += old.y;
            }
            *y = make_float2(o[0], o[1]);
        }
    }
}

}  // namespace moe

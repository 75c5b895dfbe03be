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
// u passes between the steps as two bf16 parts, hi = bf16(u) and
// lo = bf16(u - hi): together 16 bits of mantissa (an error below 2^-16
// relative), so that it can be an operand of bf16 matrix instructions without
// the 2^-8 a single bf16 would cost the float32 outputs.
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

// The two parts of u; a value beyond the finite numbers is all in hi.
MOE_DEVINL void split_bf16(float v, uint16_t &hi, uint16_t &lo)
{
    hi = f32_to_bf16_rn(v);
    const float h = bf16_to_f32(hi);
    lo = (hi & 0x7f80u) == 0x7f80u ? (uint16_t)0 : f32_to_bf16_rn(v - h);
}

// The parts' rows: [hi of rp ranks][lo of rp ranks], rp = r rounded up to 16,
// zeros behind r.
MOE_DEVINL int ad_rp(int r) { return (r + 15) & ~15; }

// D (16 x 8, float32) += A (16 x 16) B (16 x 8), bf16.
MOE_DEVINL void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                         uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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
// Inner products: u[t][j] = s_a <x_t, A_a[j]>, 0 for rows without an adapter.
struct AdInnerArgs {
    const uint16_t *x;       // [T x din]
    const uint16_t *a;       // [n x r x din]
    const int32_t *adapter;  // [T]
    const float *scale;      // nullable [n]
    uint16_t *parts;         // [T][2][rp]
    float *u_out;            // nullable [T x r]
    const float *conv;       // nullable [T x r]: given u to split into conv_parts
    uint16_t *conv_parts;    // [T][2][rp]
    int T, din, r, n;
    int *zero;               // nullable: zero_n counters to clear for the outer step
    int zero_n;
    int lists;               // CTAs that share a row tile's adapters
    int inner_ctas;          // CTAs of the inner products; those behind them convert
    int *status;
};

constexpr int kAdTile = 16;   // rows of a CTA (the matrix instruction's M)
constexpr int kAdWarps = 8;   // warps, which split K

// One CTA for 16 rows, 8 NT ranks (blockIdx.y) and every lists-th of the
// rows' distinct adapters.  Its warps take the chunks of K in turn, so the
// CTA reads whole 512-byte pieces of its rows, and add up through shared
// memory.  A pass over K for each distinct adapter computes all 16 rows and
// keeps those that are its own: rows of one request mostly stand together,
// so a tile has one or two adapters; where every row has another (a decode
// batch), the lists spread the adapters, whose matrices have to be read
// anyway, over CTAs.  Bound by the reads of x and of the adapters.
template <int NT>
__global__ void __launch_bounds__(kAdWarps * 32) k_ad_inner(AdInnerArgs p)
{
    __shared__ float red[kAdWarps][kAdTile][8 * NT + 1];
    __shared__ int sa[kAdTile];     // adapter of each row
    __shared__ int s_list[kAdTile];  // distinct adapters
    __shared__ int s_count;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, q = lane & 3;
    const int rp = ad_rp(p.r);
    pdl_wait();
    pdl_trigger();
    if ((int)blockIdx.x >= p.inner_ctas) {
        // the given u into its parts
        const int64_t all = (int64_t)p.T * rp;
        const int64_t step = (int64_t)(gridDim.x - p.inner_ctas) * gridDim.y * (kAdWarps * 32);
        const int64_t first = ((int64_t)(blockIdx.x - p.inner_ctas) * gridDim.y + blockIdx.y) *
                                  (kAdWarps * 32) + tid;
        for (int64_t i = first; i < p.zero_n; i += step)
            p.zero[i] = 0;
        for (int64_t i = first; p.conv && i < all; i += step) {
            const int t = (int)(i / rp), j = (int)(i % rp);
            uint16_t hi = 0, lo = 0;
            if (j < p.r)
                split_bf16(p.conv[(size_t)t * p.r + j], hi, lo);
            p.conv_parts[(size_t)t * 2 * rp + j] = hi;
            p.conv_parts[(size_t)t * 2 * rp + rp + j] = lo;
        }
        return;
    }
    const int tile = blockIdx.x / p.lists, part = blockIdx.x % p.lists;
    const int t0 = tile * kAdTile, j0 = blockIdx.y * 8 * NT;
    if (warp == 0) {
        int a = -1;
        if (lane < kAdTile && t0 + lane < p.T)
            a = adapter_of(p.adapter, t0 + lane, p.n, p.status);
        const unsigned same = __match_any_sync(0xffffffffu, a);
        const bool first = a >= 0 && (int)__ffs(same) - 1 == lane;
        const unsigned firsts = __ballot_sync(0xffffffffu, first);
        if (first)
            s_list[__popc(firsts & ((1u << lane) - 1u))] = a;
        if (lane < kAdTile)
            sa[lane] = a;
        if (lane == 0)
            s_count = __popc(firsts);
    }
    __syncthreads();
    const int count = s_count;
    const int nc = (p.din + kAdChunk - 1) / kAdChunk;
    const bool lo_row = t0 + g < p.T, hi_row = t0 + g + 8 < p.T;
    const uint16_t *x0 = p.x + (size_t)(lo_row ? t0 + g : 0) * p.din;
    const uint16_t *x1 = p.x + (size_t)(hi_row ? t0 + g + 8 : 0) * p.din;
    for (int l = part; l < count; l += p.lists) {
        const int a = s_list[l];
        float acc[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
            acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
        const uint16_t *ap = p.a + ((size_t)a * p.r + j0 + g) * p.din;
#pragma unroll(NT <= 2 ? 4 : NT <= 4 ? 2 : 1)
        for (int c = warp; c < nc; c += kAdWarps) {
            const int k = c * kAdChunk + 8 * q;
            const uint4 u0 = ad_chunk(x0, k, p.din, lo_row);
            const uint4 u1 = ad_chunk(x1, k, p.din, hi_row);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const uint4 w = ad_chunk(ap + (size_t)i * 8 * p.din, k, p.din,
                                         j0 + 8 * i + g < p.r);
                mma_bf16(acc[i], u0.x, u1.x, u0.y, u1.y, w.x, w.y);
                mma_bf16(acc[i], u0.z, u1.z, u0.w, u1.w, w.z, w.w);
            }
        }
        if (sa[g] == a)
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                red[warp][g][8 * i + 2 * q] = acc[i][0];
                red[warp][g][8 * i + 2 * q + 1] = acc[i][1];
            }
        if (sa[g + 8] == a)
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                red[warp][g + 8][8 * i + 2 * q] = acc[i][2];
                red[warp][g + 8][8 * i + 2 * q + 1] = acc[i][3];
            }
    }
    __syncthreads();
    // the rows of this CTA's adapters (part 0: those without one too)
    for (int i = tid; i < kAdTile * 8 * NT; i += kAdWarps * 32) {
        const int row = i / (8 * NT), jj = i % (8 * NT), j = j0 + jj, t = t0 + row;
        if (t >= p.T || j >= rp)
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
            for (int w = 0; w < kAdWarps; ++w)
                v += red[w][row][jj];
            if (p.scale)
                v *= __ldg(&p.scale[a]);
        }
        uint16_t hi, lo;
        split_bf16(j < p.r ? v : 0.0f, hi, lo);
        p.parts[(size_t)t * 2 * rp + j] = hi;
        p.parts[(size_t)t * 2 * rp + rp + j] = lo;
        if (p.u_out && j < p.r)
            p.u_out[(size_t)t * p.r + j] = v;
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
    const uint16_t *parts;   // [T][2][rp] of u
    void *y;                 // [T x dout]
    int y_bf16;
    int T, din, dout, r, n;
    WsHeader *hdr;
};

MOE_DEVINL void ad_store(const AdProductArgs &p, size_t i, float v)
{
    if (p.y_bf16) {
        uint16_t *y = static_cast<uint16_t *>(p.y) + i;
        *y = f32_to_bf16_rn(p.w ? v : v + bf16_to_f32(*y));
    } else {
        float *y = static_cast<float *>(p.y) + i;
        *y = p.w ? v : v + *y;
    }
}

// The adapter's part of one output: sum_j u_j B_a[j][o], in order of j.
MOE_DEVINL float ad_part(const AdProductArgs &p, int a, int t, int o)
{
    const int rp = ad_rp(p.r);
    const uint16_t *u = p.parts + (size_t)t * 2 * rp;
    const uint16_t *b = p.b + (size_t)a * p.r * p.dout + o;
    float v = 0.0f;
#pragma unroll 8
    for (int j = 0; j < p.r; ++j)
        v = fmaf(bf16_to_f32(__ldcg(&u[j])) + bf16_to_f32(__ldcg(&u[rp + j])),
                 bf16_to_f32(__ldg(&b[(size_t)j * p.dout])), v);
    return v;
}

constexpr int kAdRows = 64;  // most rows of k_ad_rows

// Few rows: one CTA for 16 outputs of 8 NT rows (blockIdx.y).  W is the M side
// of the matrix instruction and is read once, straight into fragments, its
// chunks of K split over the warps; the rows are the N side.  The sums meet
// in shared memory, where the adapter's part joins.  Bound by the read of W.
// W x needs nothing of the inner kernel, so it comes before the wait for it:
// the inner kernel lets this one start only after its own wait, when every
// earlier kernel (which may have made x) is complete.
template <int NT>
__global__ void __launch_bounds__(kAdWarps * 32) k_ad_rows(AdProductArgs p)
{
    __shared__ float red[kAdWarps][8 * NT][17];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, q = lane & 3;
    const int o0 = blockIdx.x * 16, t0 = blockIdx.y * 8 * NT;
    const int rows = min(8 * NT, p.T - t0);
    if (p.w) {
        float acc[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
            acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
        const bool lo_row = o0 + g < p.dout, hi_row = o0 + g + 8 < p.dout;
        const uint16_t *w0 = p.w + (size_t)(lo_row ? o0 + g : 0) * p.din;
        const uint16_t *w1 = p.w + (size_t)(hi_row ? o0 + g + 8 : 0) * p.din;
        const int nc = (p.din + kAdChunk - 1) / kAdChunk;
#pragma unroll(NT <= 2 ? 4 : 2)
        for (int c = warp; c < nc; c += kAdWarps) {
            const int k = c * kAdChunk + 8 * q;
            const uint4 u0 = ad_chunk(w0, k, p.din, lo_row);
            const uint4 u1 = ad_chunk(w1, k, p.din, hi_row);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int t = 8 * i + g;
                const uint4 v = ad_chunk(p.x + (size_t)(t < rows ? t0 + t : 0) * p.din, k, p.din,
                                         t < rows);
                mma_bf16(acc[i], u0.x, u1.x, u0.y, u1.y, v.x, v.y);
                mma_bf16(acc[i], u0.z, u1.z, u0.w, u1.w, v.z, v.w);
            }
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            red[warp][8 * i + 2 * q][g] = acc[i][0];
            red[warp][8 * i + 2 * q + 1][g] = acc[i][1];
            red[warp][8 * i + 2 * q][g + 8] = acc[i][2];
            red[warp][8 * i + 2 * q + 1][g + 8] = acc[i][3];
        }
    }
    pdl_wait();
    pdl_trigger();
    __syncthreads();
    for (int i = tid; i < 16 * rows; i += kAdWarps * 32) {
        const int t = t0 + (i >> 4), o = o0 + (i & 15);
        if (o >= p.dout)
            continue;
        const int a = adapter_of(p.adapter, t, p.n, &p.hdr->status);
        float v = 0.0f;
        if (p.w) {
#pragma unroll
            for (int w = 0; w < kAdWarps; ++w)
                v += red[w][i >> 4][i & 15];
            if (p.bias)
                v += __ldg(&p.bias[o]);
        } else {
            if (a < 0 && !p.bias)
                continue;
            if (p.bias)
                v = __ldg(&p.bias[o]);
        }
        if (a >= 0)
            v += ad_part(p, a, t, o);
        ad_store(p, (size_t)t * p.dout + o, v);
    }
}

// ---------------------------------------------------------------------------
// Sums of outer products: g[a][j][c] = sum_{t of a} u[t][j] z[t][c], for two
// problems (dA from v and x, dB from u and dy) over one grouping of the rows.
struct AdOuterProblem {
    const uint16_t *parts;  // [T][2][rp]
    const uint16_t *z;      // [T x D]
    float *g;               // [n x r x D]; nullptr: no such problem
    int D;
};
struct AdOuterArgs {
    AdOuterProblem pr[2];
    int dch0;                // column blocks of problem 0
    const int32_t *offsets;  // [n + 1] rows grouped by adapter (the counting sort)
    const int32_t *row;      // [offsets[n]]
    float *partial;          // pieces of adapters with several
    int *arrive;             // [n x column blocks x rank blocks], cleared by the inner step
    int rows;                // rows of one piece
    int T, r, n;
    int *status;
};

constexpr int kAdOutCols = 128;  // columns of a CTA: 16 for each of 8 warps
constexpr int kAdOutRows = 32;   // rows of a stage
constexpr int kAdOutStages = 4;
constexpr int kAdOutZPitch = kAdOutCols * 2 + 16;  // bytes; 16 over: rows on other banks
template <int MT>
struct AdOuterSmem {
    static constexpr int kUPitch = MT * 32 + 16;
    static constexpr int kStage = kAdOutRows * (kAdOutZPitch + 2 * kUPitch);
    static constexpr int kBytes = kAdOutStages * kStage;
};

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
MOE_DEVINL void ldmatrix_x4_t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// A CTA sums one piece (up to `rows` rows of one adapter) for 128 columns and
// 16 MT ranks (blockIdx.z): u^T is the M side and z the N side of the matrix
// instruction, K runs over the rows, which arrive by asynchronous copies four
// stages deep and are transposed on the way to registers.  Adapters of one
// piece are stored at once; the pieces of larger ones meet in scratch, where
// the last to arrive adds them in order, so results do not depend on timing.
// The pieces are found from the offsets on the device (the host knows only
// T): blockIdx.x counts them, adapters without rows have one that stores
// zeros, and CTAs behind the last leave.  Bound by the read of z.
template <int MT>
__global__ void __launch_bounds__(256) k_ad_outer(AdOuterArgs p)
{
    extern __shared__ __align__(16) uint8_t ao_smem[];
    __shared__ int s_item[6];  // adapter, first row, rows, pieces, first scratch piece, piece
    __shared__ int s_scan[32];
    __shared__ int s_last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();
    pdl_trigger();
    const int which = (int)blockIdx.y >= p.dch0;
    const AdOuterProblem pr = which ? p.pr[1] : p.pr[0];
    const int cb = blockIdx.y - (which ? p.dch0 : 0);
    const int rp = ad_rp(p.r);
    const int j0 = blockIdx.z * 16 * MT;

    // which piece: pieces before adapter e, and scratch pieces before it
    if (tid == 0)
        s_item[0] = -1;
    __syncthreads();
    {
        int base = 0, sbase = 0;
        for (int e0 = 0; e0 < p.n; e0 += 256) {
            const int e = e0 + tid;
            int first = 0, len = 0, np = 0;
            if (e < p.n) {
                first = __ldcg(&p.offsets[e]);
                len = __ldcg(&p.offsets[e + 1]) - first;
                np = len > p.rows ? (len + p.rows - 1) / p.rows : 1;
            }
            // scans of the pieces and of those that go through scratch
            int v = np, s = np > 1 ? np : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int a = __shfl_up_sync(0xffffffffu, v, o), b = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) {
                    v += a;
                    s += b;
                }
            }
            if (lane == 31) {
                s_scan[warp] = v;
                s_scan[16 + warp] = s;
            }
            __syncthreads();
            int wv = 0, wsum = 0, tv = 0, ts = 0;
            for (int w = 0; w < 8; ++w) {
                if (w < warp) {
                    wv += s_scan[w];
                    wsum += s_scan[16 + w];
                }
                tv += s_scan[w];
                ts += s_scan[16 + w];
            }
            const int start = base + wv + v - np;
            const int i = blockIdx.x;
            if (e < p.n && i >= start && i < start + np) {
                s_item[0] = e;
                s_item[5] = i - start;
                s_item[1] = first + s_item[5] * p.rows;
                s_item[2] = min(p.rows, len - s_item[5] * p.rows);
                s_item[3] = np;
                s_item[4] = sbase + wsum + s - (np > 1 ? np : 0);
            }
            base += tv;
            sbase += ts;
            __syncthreads();
            if (s_item[0] >= 0 || base > (int)blockIdx.x)
                break;
        }
    }
    const int a = s_item[0];
    if (a < 0)
        return;
    const int first = s_item[1], len = s_item[2], pieces = s_item[3];

    constexpr int kUP = AdOuterSmem<MT>::kUPitch, kStage = AdOuterSmem<MT>::kStage;
    const uint32_t sm = smem_addr(ao_smem);
    const int ns = (len + kAdOutRows - 1) / kAdOutRows;
    auto issue = [&](int s) {
        if (s < ns) {
            const uint32_t st = sm + (s % kAdOutStages) * kStage;
            // z: 32 rows x 16 vectors; u: 32 rows x 2 parts x 2 MT vectors
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = tid + 256 * h, rr = i >> 4, c = i & 15;
                const int m = s * kAdOutRows + rr;
                const int col = cb * kAdOutCols + c * 8;
                int t = 0;
                bool live = m < len;
                if (live)
                    t = __ldg(&p.row[first + m]);
                live = live && (unsigned)t < (unsigned)p.T;
                cp_async16(st + rr * kAdOutZPitch + c * 16,
                           pr.z + (live && col < pr.D ? (size_t)t * pr.D + col : 0),
                           live && col < pr.D);
            }
            for (int i = tid; i < kAdOutRows * 4 * MT; i += 256) {
                const int rr = i / (4 * MT), c = i % (4 * MT), half = c / (2 * MT), v = c % (2 * MT);
                const int m = s * kAdOutRows + rr;
                const int j = j0 + v * 8;
                int t = 0;
                bool live = m < len && j < rp;
                if (live)
                    t = __ldg(&p.row[first + m]);
                live = live && (unsigned)t < (unsigned)p.T;
                cp_async16(st + kAdOutRows * (kAdOutZPitch + half * kUP) + rr * kUP + v * 16,
                           pr.parts + (live ? (size_t)t * 2 * rp + half * rp + j : 0), live);
            }
        }
        cp_async_commit();
    };
    float acc[MT][2][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            acc[m][i][0] = acc[m][i][1] = acc[m][i][2] = acc[m][i][3] = 0.0f;
#pragma unroll
    for (int s = 0; s < kAdOutStages - 1; ++s)
        issue(s);
    for (int s = 0; s < ns; ++s) {
        cp_async_wait<kAdOutStages - 2>();
        __syncthreads();
        issue(s + kAdOutStages - 1);
        const uint32_t st = sm + (s % kAdOutStages) * kStage;
#pragma unroll
        for (int kk = 0; kk < kAdOutRows / 16; ++kk) {
            // z: four 8 x 8 blocks -- rows 0-7 and 8-15 of columns 0-7, then of 8-15
            uint32_t b[4];
            ldmatrix_x4_t(st + (kk * 16 + (lane & 15)) * kAdOutZPitch +
                              (warp * 16 + (lane >> 4) * 8) * 2,
                          b);
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    // u^T: ranks 0-7 and 8-15 of rows 0-7, then of rows 8-15
                    uint32_t u[4];
                    ldmatrix_x4_t(st + kAdOutRows * (kAdOutZPitch + half * kUP) +
                                      (kk * 16 + (lane & 7) + (lane >> 4) * 8) * kUP +
                                      (m * 16 + ((lane >> 3) & 1) * 8) * 2,
                                  u);
                    mma_bf16(acc[m][0], u[0], u[1], u[2], u[3], b[0], b[1]);
                    mma_bf16(acc[m][1], u[0], u[1], u[2], u[3], b[2], b[3]);
                }
        }
    }
    cp_async_wait<0>();

    const int gq = lane >> 2, q = lane & 3;
    const size_t plane = (size_t)p.r * pr.D;
    float *out = pr.g + (size_t)a * plane;
    // scratch: pieces of both problems, problem 0's first
    const size_t plane0 = p.pr[0].g ? (size_t)p.r * p.pr[0].D : 0;
    const size_t both = plane0 + (p.pr[1].g ? (size_t)p.r * p.pr[1].D : 0);
    float *mine = nullptr;
    if (pieces > 1) {
        mine = p.partial + (size_t)s_item[4] * both + (which ? plane0 : 0);
        out = mine + (size_t)s_item[5] * both;
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int j = j0 + m * 16 + gq + 8 * h;
                const int c = cb * kAdOutCols + warp * 16 + i * 8 + 2 * q;
                if (j < p.r && c < pr.D)
                    *reinterpret_cast<float2 *>(out + (size_t)j * pr.D + c) =
                        make_float2(acc[m][i][2 * h], acc[m][i][2 * h + 1]);
            }
    if (pieces == 1)
        return;
    __threadfence();
    __syncthreads();
    if (tid == 0) {
        int *cnt = p.arrive + ((size_t)a * gridDim.y + blockIdx.y) * gridDim.z + blockIdx.z;
        s_last = atomicAdd(cnt, 1) == pieces - 1;
    }
    __syncthreads();
    if (!s_last)
        return;
    __threadfence();
    for (int i = tid; i < 16 * MT * (kAdOutCols / 4); i += 256) {
        const int j = j0 + i / (kAdOutCols / 4), c = cb * kAdOutCols + (i % (kAdOutCols / 4)) * 4;
        if (j >= p.r || c >= pr.D)
            continue;
        const size_t o = (size_t)j * pr.D + c;
        float4 s = __ldcg(reinterpret_cast<const float4 *>(mine + o));
        for (int k = 1; k < pieces; ++k) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(mine + k * both + o));
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
        *reinterpret_cast<float4 *>(pr.g + (size_t)a * plane + o) = s;
    }
}

}  // namespace moe

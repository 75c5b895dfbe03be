// adapter_gemm.cuh -- the shared projection with its adapters on the tensor
// cores (tcgen05.mma on CTA pairs), for more rows than k_ad_rows takes.
//
//     Y [T x dout] = X W^T + sum over the adapters a of M_a U B_a
//
// with M_a the diagonal 0/1 matrix of the rows that are a's: the adapters'
// part is a contraction over (adapter, rank) appended to the one over din, so
// it lands in the same tensor-memory accumulator before the one store of y.
// A tile of 256 rows takes only the adapters that occur in it.  Its U operand
// is written by four warps of each CTA -- a row's own adapter's u, zeros for
// the others -- in its three bf16 parts, its B operand is a TMA copy of B_a as
// it lies in memory (16 ranks x outputs, the operand whose rows run along N).
// Each unit of 16 ranks costs three matrix instructions where din costs
// din / 16, so one adapter of rank 16 in a tile adds 3 to din / 16.
//
// Zeros do not silence a NaN or inf: 0 x inf is NaN, so a broken adapter
// would reach the other rows of its tile.  Every such product is a NaN, so
// the epilogue computes an output that came out NaN once more, from its own
// row and adapter alone.
//
// Where the tiles leave more than half of the pairs idle (few rows, or few
// outputs as a router has), K is split over several pairs, which leave their
// float32 sums in scratch; k_ad_join adds them in order and stores y (on all
// SMs, where the last CTA to arrive alone would wait for its reads longer
// than the split saves: 35 against 25 us for 4096 rows, 2048 to 128).
//
// The tensor cores' running float32 sum loses more at a step than a rounding:
// an output's error grows with K (1.9e-6 of the 2-norm at K = 2048, against
// 3.5e-7 for a float32 product).  Float32 outputs therefore take K in segments
// of kAGSegment blocks, each a sum of its own that the epilogue adds up,
// rounded, in registers (6.1e-7; BN = 128, whose two chunks of a warp fit
// there; 1 to 2 us more for 4096 rows, 2048 to 128).  A bf16 output takes all of
// K in one sum: its error against 64 bits stays the rounding's, 1.66e-3, and what
// the sum loses shows in the share of outputs that round to the neighbouring
// value, which grows with K: 0.12% at K = 2048, 0.23% at 4096, 0.45% at 8192,
// 0.89% at 16384 (a float32 product at 4096: 0.04%).
//
// The two CTAs of a pair share tiles of 256 rows x BN outputs: each holds its
// 128 rows of X and half of the outputs' rows of W in shared memory, and the
// accumulators of its 128 rows (two sets of BN columns, so the epilogue of
// one tile overlaps the next).  Tiles go to the pairs in turn, all column
// blocks of a row block side by side in time.  Roles of a CTA's 448 threads:
//   warps 0-3, 6-9  epilogue (two warps a quarter of the tensor-memory lanes)
//   warp 4          TMA producer of X and W
//   warp 5          tensor memory; one thread issues the MMAs (CTA 0) or says
//                   that U's copies have landed (CTA 1)
//   warps 10-13     the U operand, the list of a tile's adapters, TMA of B
// X and W need nothing of the inner kernel and are loaded while it runs (it
// lets this kernel start after its own wait); the U warps and the epilogue
// wait for it.  Every wait is bounded, as in gemm_pair.cuh.
//
// Bound by the matrix instructions for large tiles: 8192 rows, 4096 to 4096,
// bf16: 187 us of the call's 226 in here, 1.47 PFLOP/s.  A K block of a tile
// takes 0.36 to 0.38 us, a unit of adapters about 0.5 once the buffers that
// were ready are used up (one way from "empty" to the products and back),
// which is what many adapters in a tile cost: the same rows with every row
// another request's take 340 us.  U goes to its buffers by asynchronous copies
// that the MMA thread (in the other CTA a thread that passes it on) waits for
// and fences: with loads to registers, stores and a fence in the U threads,
// which waits for their next loads, a unit took 0.7 us and these rows 360.
// Small calls are bound by the chain of launches, set-up and waits: 15 us for
// 100 rows, 2048 to 2048.
#pragma once
#include "adapter.cuh"
#include "gemm_pair.cuh"

namespace moe {

constexpr int kAGRows = 256;    // rows of a pair's tile
constexpr int kAGSegment = 12;  // K blocks (768 values) of a float32 output's partial sum
constexpr int kAGThreads = 448;
constexpr int kAGWarpU = 10;    // first of the U warps
constexpr int kAGEpiWarps = 8;
constexpr int kAGUBufs = 4;     // buffers of U, a unit of 16 ranks each
constexpr int kAGBBufs = 8;     // buffers of B: a unit's copy starts kAGUBufs units ahead
constexpr int kAGTileA = 128 * kGBK * 2;  // 16 KB: a CTA's rows of one K block

template <int BN>
struct AGShape {
    static constexpr int kTileB = BN / 2 * kGBK * 2;     // a CTA's outputs of one K block
    static constexpr int kStage = kAGTileA + kTileB;
    static constexpr int kStages = BN == 256 ? 4 : 6;
    static constexpr int kUnitB = BN / 2 * 16 * 2;       // a CTA's outputs of one unit
    static constexpr int kUB = kAGUBufs * kAGTileA + kAGBBufs * kUnitB;
};

struct AGSync {
    uint64_t full[6];             // CTA 0: both CTAs' tiles of stage s landed
    uint64_t empty[6];            // each CTA: the MMAs reading stage s finished
    uint64_t ucopy[kAGUBufs];     // each CTA: its U warps' copies have landed
    uint64_t ufull[kAGUBufs];     // CTA 0: the other CTA's too
    uint64_t bfull[kAGBBufs];     // CTA 0: both CTAs' copies of B landed
    uint64_t uempty[kAGUBufs];    // each CTA: the MMAs reading the buffer finished
    uint64_t acc_full[2];         // each CTA: accumulator set b is complete
    uint64_t acc_empty[2];        // CTA 0: both epilogues have read set b
    uint64_t drained;             // each CTA: every MMA has completed
    uint64_t bye;                 // each CTA: the other CTA has finished
    int u_what[kAGUBufs];         // 1: a unit is in the buffer, + 2: the tile's last buffer
    uint32_t tmem_base;
    int abort;
    uint32_t bits[32];            // the adapters of a tile
    uint16_t list[kAGRows];
    int count;
};

template <int BN>
inline size_t ag_smem_bytes()
{
    return 1024 + (size_t)AGShape<BN>::kStages * AGShape<BN>::kStage +
           AGShape<BN>::kUB + sizeof(AGSync);
}

// Operand whose rows run along N (N contiguous), 128-byte swizzle: blocks of
// 64 N values x 8 K values (8 rows of 128 bytes); lbo from 64 values of N to
// the next, 1024 bytes from 8 values of K to the next.
MOE_DEVINL uint64_t umma_desc_mn_sw128(uint32_t saddr, uint32_t lbo)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(lbo >> 4) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

MOE_DEVINL void tma_load_3d_pair(void *dst, const CUtensorMap *map, int x, int y, int z,
                                 uint32_t bar_caddr)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_caddr), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// Arrive on `bar` (one of its counted arrivals) when this thread's copies so
// far have landed.
MOE_DEVINL void cp_async_arrive(uint64_t *bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

MOE_DEVINL void prefetch_tensormap(const CUtensorMap *m)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

MOE_DEVINL bool ag_aborted(const AGSync &sy) { return *(volatile const int *)&sy.abort != 0; }

// One output alone, in float32: its own adapter's part and the row's product
// with W.  A NaN on the way is the output's own and stays one.
__device__ __noinline__ float ag_one(const AdProductArgs &p, int a, int t, int o)
{
    const float part = a >= 0 ? ad_part(p, a, t, o) : 0.0f;
    if (!p.w || part != part)
        return part;
    const uint16_t *x = p.x + (size_t)t * p.din, *w = p.w + (size_t)o * p.din;
    float v = 0.0f;
    for (int k0 = 0; k0 < p.din && v == v; k0 += 64)
#pragma unroll
        for (int k = k0; k < k0 + 64; k += 8) {
            const uint4 a8 = ad_chunk(x, k, p.din, true), w8 = ad_chunk(w, k, p.din, true);
            const float xv[8] = {bf16lo(a8.x), bf16hi(a8.x), bf16lo(a8.y), bf16hi(a8.y),
                                 bf16lo(a8.z), bf16hi(a8.z), bf16lo(a8.w), bf16hi(a8.w)};
            v = dot8_bf16(w8, xv, v);
        }
    return v + part;
}

// A warp: the NaNs among 32 outputs from o on (v) of rows t0 + lane once more,
// each lane its own adapter's part of its row, the product with W of all rows
// by matrix instructions (fragments straight from memory).  A broken adapter
// makes every tile take this that it has a row in: 8192 rows of 4096 to 4096,
// one of 16 adapters all inf: 4.8 ms in runs of rows, 12.8 ms with the rows
// interleaved (214 output by output).
__device__ __noinline__ void ag_again(const AdProductArgs &p, float *v, int t0, int o)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3, t = t0 + lane;
    const int a = t < p.T ? adapter_of(p.adapter, t, p.n, nullptr) : -1;
    uint32_t left = 0;  // the outputs whose product is missing
    for (int j = 0; j < 32; ++j)
        if (t < p.T && o + j < p.dout && v[j] != v[j])
            left |= 1u << j;
    const int rp = ad_rp(p.r);
    const uint16_t *u = p.parts + (size_t)(a >= 0 ? t : 0) * kAdParts * rp;
#pragma unroll 1
    for (int j = 0; j < 32; j += 8) {  // eight outputs at a time
        if (!(left >> j & 0xffu))
            continue;
        float part[8] = {};
        const uint16_t *b = p.b + (size_t)(a >= 0 ? a : 0) * p.r * p.dout + o + j;
        for (int e = 0; e < (a >= 0 ? p.r : 0); ++e) {
            float x = bf16_to_f32(__ldcg(&u[e]));
#pragma unroll
            for (int i = 1; i < kAdParts; ++i)
                x += bf16_to_f32(__ldcg(&u[i * rp + e]));
            const uint4 w = __ldg(reinterpret_cast<const uint4 *>(b + (size_t)e * p.dout));
            const float wv[8] = {bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y),
                                 bf16lo(w.z), bf16hi(w.z), bf16lo(w.w), bf16hi(w.w)};
#pragma unroll
            for (int k = 0; k < 8; ++k)
                part[k] = fmaf(x, wv[k], part[k]);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (left >> (j + k) & 1u) {
                v[j + k] = part[k];
                if (part[k] != part[k])  // its own: it stays one
                    left &= ~(1u << (j + k));
            }
    }
    if (!p.w || !__any_sync(0xffffffffu, left != 0))
        return;
#pragma unroll 1
    for (int m = 0; m < 2; ++m) {  // rows t0 + 16 m + 0 .. 15
        const int ta = t0 + 16 * m + g, tb = ta + 8;
        float sum[4][4] = {};
        bool some = true;
#pragma unroll 1
        for (int c0 = 0; c0 < p.din && some; c0 += 8 * kAdChunk) {
            float acc[4][4] = {};
#pragma unroll 1
            for (int c = c0; c < min(p.din, c0 + 8 * kAdChunk); c += kAdChunk) {
                const int k = c + 8 * q;
                const uint4 xa = ad_chunk(p.x + (size_t)ta * p.din, k, p.din, ta < p.T);
                const uint4 xb = ad_chunk(p.x + (size_t)tb * p.din, k, p.din, tb < p.T);
                uint4 w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = ad_chunk(p.w + (size_t)(o + 8 * i + g) * p.din, k, p.din,
                                    o + 8 * i + g < p.dout);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mma_bf16(acc[i], xa.x, xb.x, xa.y, xb.y, w[i].x, w[i].y);
                    mma_bf16(acc[i], xa.z, xb.z, xa.w, xb.w, w[i].z, w[i].w);
                }
            }
            some = false;  // rows of NaN alone end here
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    sum[i][h] += acc[i][h];
                    some |= sum[i][h] == sum[i][h];
                }
            some = __any_sync(0xffffffffu, some);
        }
        // from the fragments to a row a lane
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const int from = (lane & 7) * 4 + (j & 7) / 2;
            const float lo = __shfl_sync(0xffffffffu, sum[j >> 3][j & 1], from);
            const float hi = __shfl_sync(0xffffffffu, sum[j >> 3][2 + (j & 1)], from);
            if ((left >> j & 1u) && lane >> 4 == m)
                v[j] += lane & 8 ? hi : lo;
        }
    }
}

MOE_DEVINL uint32_t ag_word(uint32_t w) { return w; }
MOE_DEVINL uint32_t ag_word(float w) { return __float_as_uint(w); }

// A lane holds N words of its own row (of 32 rows); four lanes (a quad)
// exchange vectors of four words so that vector 4 b + c of a lane becomes
// vector 4 b + (lane % 4) of the quad's row c: a store then writes 64 bytes of
// a row from a quad, whole sectors, where each lane's own row would give 32
// rows 16 bytes each.
template <int N, typename W>
MOE_DEVINL void ag_quad_rows(W (&v)[N])
{
    const int q = threadIdx.x & 3;
#pragma unroll
    for (int b = 0; b < N; b += 16) {
        // 4 x 4 transpose of vectors: halves across lanes 2 apart, then neighbours
#pragma unroll
        for (int s = 2; s >= 1; s >>= 1)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (!(c & s))
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        W &lo = v[b + 4 * c + k], &hi = v[b + 4 * (c | s) + k];
                        const W give = q & s ? lo : hi;
                        const W got = __shfl_xor_sync(0xffffffffu, give, s);
                        if (q & s)
                            lo = got;
                        else
                            hi = got;
                    }
    }
}

// Store what ag_quad_rows arranged: columns o .. o + 31 of rows r0 .. r0 + 31
// (below rows) of a matrix whose rows are ld values; columns below cols.
template <typename E, int N, typename W>
MOE_DEVINL void ag_put(E *base, int ld, int o, int r0, int lane, int rows, int cols, const W (&v)[N])
{
    constexpr int kPer = 16 / sizeof(E);  // values of a vector
#pragma unroll
    for (int b = 0; b < N; b += 16)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int row = r0 + (lane & ~3) + c, col = o + (b / 4 + (lane & 3)) * kPer;
            if (row < rows && col < cols) {
                uint4 q;
                q.x = ag_word(v[b + 4 * c]);
                q.y = ag_word(v[b + 4 * c + 1]);
                q.z = ag_word(v[b + 4 * c + 2]);
                q.w = ag_word(v[b + 4 * c + 3]);
                *reinterpret_cast<uint4 *>(base + (size_t)row * ld + col) = q;
            }
        }
}

template <int BN>
__global__ void __launch_bounds__(kAGThreads, 1)
    k_ad_gemm(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
              const __grid_constant__ CUtensorMap tm_b, AdProductArgs p)
{
    using S = AGShape<BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = g_align1024(smem_raw);
    uint8_t *ubuf = ring + (size_t)S::kStages * S::kStage;
    uint8_t *bbuf = ubuf + (size_t)kAGUBufs * kAGTileA;
    AGSync &sy = *reinterpret_cast<AGSync *>(ubuf + S::kUB);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank(), peer = rank ^ 1u;
    const bool lead = rank == 0;
    int *status = &p.hdr->status;

    if (tid == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(&sy.full[s], 1);
            mbar_init(&sy.empty[s], 1);
        }
        for (int b = 0; b < kAGUBufs; ++b) {
            mbar_init(&sy.ucopy[b], 128 + 1);  // the U threads' copies, u_what
            mbar_init(&sy.ufull[b], 1);
            mbar_init(&sy.uempty[b], 1);
        }
        for (int b = 0; b < kAGBBufs; ++b)
            mbar_init(&sy.bfull[b], 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sy.acc_full[b], 1);
            mbar_init(&sy.acc_empty[b], 2 * kAGEpiWarps);
        }
        mbar_init(&sy.drained, 1);
        mbar_init(&sy.bye, 1);
        sy.abort = 0;
        fence_mbar_init();
    }
    // U warps: the first tile's adapters, on their way during the set-up
    const int splits = p.splits;
    const int ncol = (p.dout + BN - 1) / BN, nrow = (p.T + kAGRows - 1) / kAGRows;
    // work items: (tile, split), the splits of a tile side by side
    const int items = nrow * ncol * splits, pairs = gridDim.x / 2, pair = blockIdx.x / 2;
    const int ut = tid - kAGWarpU * 32;  // U warps: this CTA's row of the tile
    int a_own = -1, a_peer = -1;
    auto load_ids = [&](int it) {
        const int t = it / splits / ncol * kAGRows + (int)rank * 128 + ut;
        const int tp = it / splits / ncol * kAGRows + (int)peer * 128 + ut;
        a_own = t < p.T ? adapter_of(p.adapter, t, p.n, status) : -1;
        a_peer = tp < p.T ? adapter_of(p.adapter, tp, p.n, status) : -1;
    };
    if (warp >= kAGWarpU && pair < items)
        load_ids(pair);
    if (warp == kGWarpTma && lane == 0) {
        if (p.w) {
            prefetch_tensormap(&tm_x);
            prefetch_tensormap(&tm_w);
        }
        prefetch_tensormap(&tm_b);
    }
    if (warp == kGWarpMma) {
        tmem_alloc_pair(&sy.tmem_base, 2 * BN);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = sy.tmem_base;

    const int nkb = p.w ? (p.din + kGBK - 1) / kGBK : 0;
    const int nks = (nkb + splits - 1) / splits;  // K blocks of a split
    const int nch = ad_rp(p.r) / 16;  // units of an adapter

    if (warp == kGWarpTma) {
        if (lane == 0) {
            uint32_t g = 0;
            for (int it = pair; it < items && !ag_aborted(sy); it += pairs) {
                const int i = it / splits, kb0 = it % splits * nks, kb1 = min(nkb, kb0 + nks);
                const int t0 = i / ncol * kAGRows + (int)rank * 128;
                const int o0 = i % ncol * BN + (int)rank * (BN / 2);
                for (int kb = kb0; kb < kb1; ++kb, ++g) {
                    const int s = g % S::kStages;
                    if (!mbar_wait_cluster(&sy.empty[s], ((g / S::kStages) & 1) ^ 1, status)) {
                        sy.abort = 1;
                        break;
                    }
                    uint8_t *st = ring + (size_t)s * S::kStage;
                    const uint32_t fb = cluster_addr(&sy.full[s], 0);
                    if (lead)  // both CTAs' bytes
                        mbar_arrive_expect_tx(&sy.full[s], 2 * S::kStage);
                    tma_load_2d_pair(st, &tm_x, kb * kGBK, t0, fb);
                    tma_load_2d_pair(st + kAGTileA, &tm_w, kb * kGBK, o0, fb);
                }
            }
            // CTA 0: every stage issued has landed before the CTA may leave
            if (lead)
                for (uint32_t r = g > (uint32_t)S::kStages ? g - S::kStages : 0; r < g; ++r)
                    mbar_wait(&sy.full[r % S::kStages], (r / S::kStages) & 1, status);
        }
    } else if (warp == kGWarpMma) {
        if (lane == 0 && lead) {
            uint32_t g = 0, ub = 0, bu = 0, itc = 0;
            const uint32_t idesc = umma_idesc_bf16(kAGRows, BN);
            const uint32_t idesc_mn = idesc | (1u << 16);  // B along N
            for (int it = pair; it < items && !ag_aborted(sy); it += pairs) {
                const int kb0 = it % splits * nks, kb1 = min(nkb, kb0 + nks);
                const int nseg = max(1, (kb1 - kb0 + p.segment - 1) / p.segment);
                for (int sg = 0; sg < nseg; ++sg, ++itc) {
                    const int buf = itc & 1;
                    const int kbs = kb0 + sg * p.segment, kbe = min(kb1, kbs + p.segment);
                    if (!mbar_wait_cluster(&sy.acc_empty[buf], ((itc >> 1) & 1) ^ 1, status)) {
                        sy.abort = 1;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t dt = tmem + buf * BN;
                    uint32_t acc = 0;
                    // adapters' units to come, with the last segment of the first split
                    bool more = it % splits == 0 && sg == nseg - 1;
                    auto unit = [&]() {
                        const int b = ub % kAGUBufs;
                        const uint32_t ph = (ub / kAGUBufs) & 1;
                        if (!mbar_wait(&sy.ucopy[b], ph, status) ||
                            !mbar_wait_cluster(&sy.ufull[b], ph, status)) {
                            sy.abort = 1;
                            return;
                        }
                        fence_proxy_async_smem();  // the copies, for the MMAs
                        tc_fence_after();
                        const int what = *(volatile int *)&sy.u_what[b];
                        const uint32_t st = smem_addr(ubuf + (size_t)b * kAGTileA);
                        if (what & 1) {
                            const int bb = bu % kAGBBufs;
                            if (!mbar_wait_cluster(&sy.bfull[bb], (bu / kAGBBufs) & 1, status)) {
                                sy.abort = 1;
                                return;
                            }
                            tc_fence_after();
                            ++bu;
                            const uint64_t bd =
                                umma_desc_mn_sw128(smem_addr(bbuf + (size_t)bb * S::kUnitB), 2048);
#pragma unroll
                            for (int k = 0; k < kAdParts; ++k) {
                                umma_bf16_pair(dt, umma_desc_sw128(st + k * 32), bd, idesc_mn, acc);
                                acc = 1;
                            }
                        }
                        umma_commit_pair_both(&sy.uempty[b]);
                        ++ub;
                        more = !(what & 2);
                    };
                    for (int kb = kbs; kb < kbe; ++kb, ++g) {
                        const int s = g % S::kStages;
                        if (!mbar_wait_cluster(&sy.full[s], (g / S::kStages) & 1, status)) {
                            sy.abort = 1;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t st = smem_addr(ring + (size_t)s * S::kStage);
#pragma unroll
                        for (int kk = 0; kk < kGBK / 16; ++kk) {
                            umma_bf16_pair(dt, umma_desc_sw128(st + kk * 32),
                                           umma_desc_sw128(st + kAGTileA + kk * 32), idesc, acc);
                            acc = 1;
                        }
                        umma_commit_pair_both(&sy.empty[s]);
                    }
                    // (units between the K blocks, at fixed places, cost 3 us more for
                    // 8192 rows of 4096 than they hid)
                    while (more && !ag_aborted(sy))
                        unit();
                    if (ag_aborted(sy))
                        break;
                    umma_commit_pair_both(&sy.acc_full[buf]);
                }
            }
            umma_commit_pair_both(&sy.drained);
            mbar_wait(&sy.drained, 0, status);
        } else if (lane == 0) {
            // CTA 1: tells CTA 0 of the units of U that have landed here
            uint32_t ub = 0;
            for (int it = pair; it < items && !ag_aborted(sy); it += pairs) {
                bool more = it % splits == 0;
                while (more) {
                    const int b = ub % kAGUBufs;
                    if (!mbar_wait(&sy.ucopy[b], (ub / kAGUBufs) & 1, status)) {
                        sy.abort = 1;
                        break;
                    }
                    fence_proxy_async_smem();
                    more = !(*(volatile int *)&sy.u_what[b] & 2);
                    mbar_arrive_cluster(cluster_addr(&sy.ufull[b], 0));
                    ++ub;
                }
            }
        }
    } else if (warp >= kAGWarpU) {
        // ------------------------------------------------------------ U and B
        const int rp = ad_rp(p.r);
        uint32_t ub = 0, bu = 0;  // units and copies of B so far
        bool waited = false;
        for (int it = pair; it < items; it += pairs) {
            if (it % splits)
                continue;  // the first split takes the adapters
            const int i = it / splits;
            // the tile's adapters, both CTAs' rows, in order of their number
            if (it != pair)
                load_ids(it);
            const int a = a_own, ap = a_peer;
            const int t = i / ncol * kAGRows + (int)rank * 128 + ut;
            if (ut < 32)
                sy.bits[ut] = 0u;
            named_bar_sync(1, 128);
            if (a >= 0)
                atomicOr(&sy.bits[a >> 5], 1u << (a & 31));
            if (ap >= 0)
                atomicOr(&sy.bits[ap >> 5], 1u << (ap & 31));
            named_bar_sync(1, 128);
            if (ut < 32) {
                uint32_t w = sy.bits[ut];
                int at = __popc(w), n = at;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, at, o);
                    if (ut >= o)
                        at += v;
                }
                int total = __shfl_sync(0xffffffffu, at, 31);
                at -= n;
                while (w) {
                    sy.list[at++] = (uint16_t)(ut * 32 + __ffs(w) - 1);
                    w &= w - 1;
                }
                // nothing to add and no product: one unit of zeros fills the accumulators
                if (total == 0 && !p.w) {
                    total = 1;
                    if (ut == 0)
                        sy.list[0] = 0;
                }
                if (ut == 0)
                    sy.count = total;
            }
            named_bar_sync(1, 128);
            const int units = sy.count * nch;
            const int o0 = i % ncol * BN + (int)rank * (BN / 2);
            const uint16_t *urow = p.parts + (size_t)(a >= 0 ? t : 0) * kAdParts * rp;
            // B of unit u (one thread).  Its buffer was unit u - kAGBBufs's, whose
            // MMAs are complete once U's buffer of unit u - kAGBBufs + kAGUBufs
            // has come back empty, so a unit's copy starts kAGUBufs units ahead
            int bl = 0, bj = 0;  // the next copy's adapter in the list and its first rank
            auto load_b = [&]() {
                const int e = sy.list[bl], j = bj, bb = bu % kAGBBufs;
                bj += 16;
                if (bj >= rp) {
                    bj = 0;
                    ++bl;
                }
                uint8_t *st = bbuf + (size_t)bb * S::kUnitB;
                const uint32_t fb = cluster_addr(&sy.bfull[bb], 0);
                if (lead)
                    mbar_arrive_expect_tx(&sy.bfull[bb], 2 * S::kUnitB);
                for (int c = 0; c < BN / 128; ++c)
                    tma_load_3d_pair(st + c * 2048, &tm_b, o0 + 64 * c, j, e, fb);
                ++bu;
            };
            if (ut == 0)
                for (int u = 0; u < min(units, kAGUBufs); ++u)
                    load_b();
            if (!waited) {
                pdl_wait();
                pdl_trigger();
                waited = true;
            }
            int u0 = 0, li = 0, j = 0;  // the unit: its adapter in the list, its first rank
            do {
                const int b = ub % kAGUBufs;
                const int e = u0 < units ? sy.list[li] : -1;
                // one lane waits for its warp
                int ok = 1;
                if (lane == 0)
                    ok = mbar_wait(&sy.uempty[b], ((ub / kAGUBufs) & 1) ^ 1, status);
                if (!__shfl_sync(0xffffffffu, ok, 0)) {
                    sy.abort = 1;
                    break;
                }
                const uint32_t st = smem_addr(ubuf + (size_t)b * kAGTileA) + ut * 128;
                const bool own = a >= 0 && a == e;
#pragma unroll
                for (int c = 0; c < 2 * kAdParts; ++c)
                    cp_async16(st + ((c ^ (ut & 7)) << 4), urow + c / 2 * rp + j + c % 2 * 8, own);
                cp_async_arrive(&sy.ucopy[b]);
                if (ut == 0) {
                    sy.u_what[b] = (e >= 0 ? 1 : 0) | (u0 + 1 >= units ? 2 : 0);
                    mbar_arrive(&sy.ucopy[b]);
                }
                if (ut == 0 && u0 + kAGUBufs < units)
                    load_b();
                j += 16;
                if (j >= rp) {
                    j = 0;
                    ++li;
                }
                ++ub;
                ++u0;
            } while (u0 < units);
            named_bar_sync(1, 128);  // the list has been read; all four warps see an abort
            if (ag_aborted(sy))
                break;
        }
        cp_async_commit();
        cp_async_wait<0>();
    } else {
        // ------------------------------------------------------------ epilogue
        const int lq = warp & 3, eh = warp >= 6;
        const uint32_t lane_addr = tmem + ((uint32_t)(lq * 32) << 16);
        uint32_t itc = 0;
        for (int it = pair; it < items; it += pairs, ++itc) {
            const int i = it / splits;
            const int row0 = i / ncol * kAGRows + (int)rank * 128;  // this CTA's first row
            const int t = row0 + lq * 32 + lane;
            const int o0 = i % ncol * BN;
            float *part = splits > 1 ? p.partial + ((size_t)it * 2 + rank) * 128 * BN : nullptr;
            const int kb0 = it % splits * nks, kb1 = min(nkb, kb0 + nks);
            const int nseg = max(1, (kb1 - kb0 + p.segment - 1) / p.segment);
            auto wait_full = [&]() {
                int ok = 1;
                if (lane == 0)
                    ok = mbar_wait_cluster(&sy.acc_full[itc & 1], (itc >> 1) & 1, status);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok)
                    sy.abort = 1;
                tc_fence_after();
                return ok != 0;
            };
            auto hand_back = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster(cluster_addr(&sy.acc_empty[itc & 1], 0));
            };
            // the segments before the last, rounded sums (this warp's two chunks)
            float sum[2][32];
            if (BN == 128) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        sum[c][j] = 0.0f;
                bool ok = true;
                for (int sg = 0; sg < nseg - 1 && ok; ++sg) {
                    ok = wait_full();
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float v[32];
                        __syncwarp();
                        tmem_ld32(lane_addr + (itc & 1) * BN + (eh + 2 * c) * 32, v);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            sum[c][j] += v[j];
                    }
                    hand_back();
                    ++itc;
                }
                if (!ok)
                    break;
            }
            if (it == pair) {  // only the stores wait for the kernels before
                pdl_wait();
                pdl_trigger();
            }
            if (!wait_full())
                break;
            const int buf = itc & 1;
#pragma unroll(BN == 128 ? 2 : 1)
            for (int cc = 0; cc < BN / 64; ++cc) {
                const int c = eh + 2 * cc, o = o0 + c * 32;
                if (o >= p.dout)
                    break;
                float v[32];
                __syncwarp();
                tmem_ld32(lane_addr + buf * BN + c * 32, v);
                if (BN == 128) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        v[j] += sum[cc & 1][j];
                }
                if (splits > 1) {
                    ag_quad_rows(v);
                    ag_put<float>(part, BN, c * 32, lq * 32, lane, 128, BN, v);
                    continue;
                }
                bool bad = false;
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    bad |= v[j] != v[j];
                if (__any_sync(0xffffffffu, bad && t < p.T)) {
                    // (through memory: nothing of the rare call costs the others registers)
                    constexpr int kSum = BN == 128 ? 32 : 0;
                    float w[32 + kSum];
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        w[j] = v[j];
                        if (BN == 128)
                            w[kSum + j] = sum[1][j];
                    }
                    ag_again(p, w, t - lane, o);
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        v[j] = w[j];
                        if (BN == 128)
                            sum[1][j] = w[kSum + j];
                    }
                }
                if (p.bias) {
#pragma unroll
                    for (int j = 0; j < 32; j += 8)
                        if (o + j < p.dout)
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                v[j + k] += __ldg(&p.bias[o + j + k]);
                }
                __syncwarp();
                if (p.y_bf16) {
                    uint32_t h[16];
                    if (p.w) {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            h[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
                    } else {
                        const uint4 *old = reinterpret_cast<const uint4 *>(
                            static_cast<const uint16_t *>(p.y) + (size_t)t * p.dout + o);
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            uint4 w = make_uint4(0u, 0u, 0u, 0u);
                            if (t < p.T && o + 2 * j < p.dout)
                                w = old[j / 4];
                            h[j] = pack_bf16x2(v[2 * j] + bf16lo(w.x), v[2 * j + 1] + bf16hi(w.x));
                            h[j + 1] = pack_bf16x2(v[2 * j + 2] + bf16lo(w.y), v[2 * j + 3] + bf16hi(w.y));
                            h[j + 2] = pack_bf16x2(v[2 * j + 4] + bf16lo(w.z), v[2 * j + 5] + bf16hi(w.z));
                            h[j + 3] = pack_bf16x2(v[2 * j + 6] + bf16lo(w.w), v[2 * j + 7] + bf16hi(w.w));
                        }
                    }
                    __syncwarp();
                    ag_quad_rows(h);
                    ag_put<uint16_t>(static_cast<uint16_t *>(p.y), p.dout, o, row0 + lq * 32, lane, p.T,
                                     p.dout, h);
                } else {
                    if (!p.w) {
                        const float4 *old = reinterpret_cast<const float4 *>(
                            static_cast<const float *>(p.y) + (size_t)t * p.dout + o);
#pragma unroll
                        for (int j = 0; j < 32; j += 4)
                            if (t < p.T && o + j < p.dout) {
                                const float4 w = old[j / 4];
                                v[j] += w.x;
                                v[j + 1] += w.y;
                                v[j + 2] += w.z;
                                v[j + 3] += w.w;
                            }
                    }
                    __syncwarp();
                    ag_quad_rows(v);
                    ag_put<float>(static_cast<float *>(p.y), p.dout, o, row0 + lq * 32, lane, p.T, p.dout,
                                  v);
                }
            }
            hand_back();
        }
    }
    // tensor memory goes back once every MMA has completed, and neither CTA's
    // shared memory goes away while the other may still reach it
    tc_fence_before();
    __syncthreads();
    if (warp == kGWarpMma) {
        if (lane == 0 && !lead)
            mbar_wait(&sy.drained, 0, status);
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem, 2 * BN);
    }
    if (tid == 0) {
        mbar_arrive_cluster(cluster_addr(&sy.bye, peer));
        mbar_wait_cluster(&sy.bye, 0, status);
    }
}

// ---------------------------------------------------------------------------
// y from the splits' sums: eight outputs of a row a thread, all splits' loads
// in flight, added in order of the splits.
constexpr int kAGSplitCols = 128;  // BN where K is split
constexpr int kAGMaxSplits = 8;

__global__ void __launch_bounds__(256) k_ad_join(AdProductArgs p)
{
    pdl_wait();
    pdl_trigger();
    const int nv = p.dout / 8, ncol = (p.dout + kAGSplitCols - 1) / kAGSplitCols;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)p.T * nv)
        return;
    const int t = (int)(i / nv), o = (int)(i % nv) * 8;
    const size_t tile = (size_t)(t / kAGRows) * ncol + o / kAGSplitCols;
    const float *q = p.partial + (tile * p.splits * kAGRows + t % kAGRows) * kAGSplitCols +
                     o % kAGSplitCols;
    float4 a[kAGMaxSplits], b[kAGMaxSplits];
#pragma unroll
    for (int s = 0; s < kAGMaxSplits; ++s)
        if (s < p.splits) {
            const float4 *r =
                reinterpret_cast<const float4 *>(q + (size_t)s * kAGRows * kAGSplitCols);
            a[s] = __ldcg(r);
            b[s] = __ldcg(r + 1);
        }
    float v[8] = {};
#pragma unroll
    for (int s = 0; s < kAGMaxSplits; ++s)
        if (s < p.splits) {
            v[0] += a[s].x;
            v[1] += a[s].y;
            v[2] += a[s].z;
            v[3] += a[s].w;
            v[4] += b[s].x;
            v[5] += b[s].y;
            v[6] += b[s].z;
            v[7] += b[s].w;
        }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if (v[k] != v[k])
            v[k] = ag_one(p, adapter_of(p.adapter, t, p.n, nullptr), t, o + k);
        if (p.bias)
            v[k] += __ldg(&p.bias[o + k]);
    }
    const size_t at = (size_t)t * p.dout + o;
    if (p.y_bf16) {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.y) + at) =
            make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                       pack_bf16x2(v[6], v[7]));
    } else {
        float4 *y = reinterpret_cast<float4 *>(static_cast<float *>(p.y) + at);
        y[0] = make_float4(v[0], v[1], v[2], v[3]);
        y[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}

}  // namespace moe

// adapter_outer.cuh -- the adapters' weight gradients on the tensor cores:
// sums of outer products over each adapter's rows,
//     g[a][j][c] = sum_{t of a} u[t][j] z[t][c],
// for two problems (dA from v and x, dB from u and dy) over one grouping of
// the rows.
//
// K runs over the rows, so both operands lie with K outermost (their other
// index contiguous): the gathered rows of z and of u's three bf16 parts go to
// shared memory as they are, by asynchronous copies into the 128-byte swizzled
// layout (blocks of 64 values x 8 rows), and tcgen05.mma reads them transposed.
// Ranks are the M side, 256 columns the N side.  Of the 128 lanes the upper 64
// take u's first part and the lower 64 the two smaller ones, in two
// instructions a step: (first, second) and (a block of zeros, third).  The
// tensor cores' running sum loses more at a step than a rounding, so the large
// sums get one step for 16 rows where all three parts in one would take three
// (relative error at 8192 rows 8.6e-7 where that gave 1.3e-6; a float32
// product 7.9e-7); the epilogue adds the halves.  What is lost grows with the
// steps, so one running sum takes kAOSegment stages at most, 48 steps; the sums of
// a longer piece are added up rounded in its output (dB of 131072 rows in two
// pieces: 7.7e-5 with one sum each, 7.6e-7 so; a float32 product 1.3e-6).  Pieces
// are that long beyond about 768 x 256 / (column and rank blocks) rows of one
// adapter; reading the sums out leaves the tensor cores idle (both gradients of
// 65536 rows of 4096 and 4096 columns, rank 64, one adapter, eight pieces: 799 us,
// 627 with one sum each).
//
// An infinity in z meets the zeros and, where u has fewer bits, parts of 0:
// the sums of its column come out NaN.  What came out NaN is computed once more
// from u itself (ao_again), so an infinity gives what the formula says and a NaN
// stays one.
//
// A CTA sums one piece (up to `rows` rows of one adapter) for 256 columns and
// 64 ranks (blockIdx.z).  Adapters of one piece are stored at once; the pieces
// of larger ones go to scratch, where k_ad_outer_join adds them in order, so
// results do not depend on timing.  The pieces are found from the offsets on
// the device (the host knows only T): blockIdx.x counts them, adapters without
// rows have one that stores zeros, and CTAs behind the last leave.  Meant to be
// bound by the read of z; two CTAs an SM, so that one's copies run under the
// other's start and end.  Both gradients of 8192 rows, 2048 and 2048 columns,
// rank 64, with their join: 37 us, 2 TB/s of z and the scratch pieces.
#pragma once
#include "adapter_gemm.cuh"

namespace moe {

struct AdOuterProblem {
    const uint16_t *parts;  // [T][kAdParts][rp]
    const uint16_t *z;      // [T x D]
    float *g;               // [n x r x D]; nullptr: no such problem
    int D;
};
struct AdOuterArgs {
    AdOuterProblem pr[2];
    int dch0;                // column blocks of problem 0
    const int32_t *offsets;  // [n + 1] rows grouped by adapter
    const int32_t *row;      // [offsets[n]]
    float *partial;          // pieces of adapters with several
    int rows;                // rows of one piece
    int T, r, n;
    int *status;
};

constexpr int kAOCols = 256, kAORanks = 64;  // of a CTA
constexpr int kAORows = 32;                  // of a stage
constexpr int kAOStages = 3;
constexpr int kAOWarps = 8;                  // producers, then epilogue; one more issues the MMAs
constexpr int kAOThreads = (kAOWarps + 1) * 32;
constexpr int kAOBlock = kAORows * 128;      // 64 values of every row
constexpr int kAOStage = (kAdParts + kAOCols / 64) * kAOBlock;

constexpr int kAOSegment = 24;  // stages that one tensor-memory sum takes

constexpr int kAOHalfPitch = kAOCols + 4;  // floats of a lower-half row on its way to the upper

struct AOSync {
    uint64_t full[kAOStages];   // every producer's copies of the stage have landed
    uint64_t empty[kAOStages];  // the MMAs reading it have completed
    uint64_t done;              // every MMA of the segment has completed
    uint32_t tmem_base;
    int abort, stop;            // stop: abort as warp 0 saw it, the same for all warps
};

// the zeros, the stages (afterwards the lower half's sums), the barriers
inline size_t ao_smem_bytes() { return 1024 + kAOBlock + (size_t)kAOStages * kAOStage + sizeof(AOSync); }
static_assert(kAORanks * kAOHalfPitch * 4 <= kAOStages * kAOStage, "the lower half fits the stages");

// Store or add what ag_quad_rows arranged: columns c .. c + 31 of ranks r0 ..
// r0 + 31.  Whether the warp stored a NaN (or an infinity).
MOE_DEVINL bool ao_put(float *out, int D, int c, int r0, int lane, int ranks, int cols,
                       const float (&v)[32], bool add)
{
    float bad = 0.0f;  // 0 x v
#pragma unroll
    for (int b = 0; b < 32; b += 16)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int row = r0 + (lane & ~3) + k, col = c + (b / 4 + (lane & 3)) * 4;
            if (row < ranks && col < cols) {
                float4 *to = reinterpret_cast<float4 *>(out + (size_t)row * D + col);
                float4 q = make_float4(v[b + 4 * k], v[b + 4 * k + 1], v[b + 4 * k + 2], v[b + 4 * k + 3]);
                if (add) {
                    const float4 old = *to;  // this thread's own
                    q.x += old.x;
                    q.y += old.y;
                    q.z += old.z;
                    q.w += old.w;
                }
                *to = q;
                bad = fmaf(q.x, 0.0f, fmaf(q.y, 0.0f, fmaf(q.z, 0.0f, fmaf(q.w, 0.0f, bad))));
            }
        }
    return __any_sync(0xffffffffu, bad != 0.0f);
}

// A warp: the NaNs among its stored sums once more, in float32 over the piece's
// rows: column blocks of 32 (the bits of `blocks`) of a lane's rank j (live:
// there is one), out its first column.  Ends early where every sum in question is
// a NaN.  Gradients of 8192 rows, 2048 and 2048 columns, rank 64: 0.4 ms with one
// infinity in x, 1.5 ms with a row of them, 0.2 ms where x is all NaN (88 us
// otherwise; looking for NaNs costs 0.2 to 0.4 us).
__device__ __noinline__ void ao_again(const uint16_t *parts, const uint16_t *z, int D, int cols,
                                      const int32_t *row, int len, int T, int rp, int j, bool live,
                                      uint32_t blocks, float *out)
{
    for (; blocks; blocks &= blocks - 1) {
        const int c = (__ffs(blocks) - 1) * 32;
        uint32_t left = 0;
        for (int k = 0; k < 32; ++k)
            if (live && c + k < cols && out[c + k] != out[c + k])
                left |= 1u << k;
        float s[32] = {};
#pragma unroll 1
        for (int m = 0; m < len; ++m) {
            const int t = __ldcg(&row[m]);
            if ((unsigned)t >= (unsigned)T)
                continue;
            float u = 0.0f;
            if (live)
#pragma unroll
                for (int i = 0; i < kAdParts; ++i)
                    u += bf16_to_f32(__ldcg(&parts[((size_t)t * kAdParts + i) * rp + j]));
#pragma unroll
            for (int k = 0; k < 32; k += 8)
                if (c + k < cols) {
                    const uint4 q = __ldg(reinterpret_cast<const uint4 *>(z + (size_t)t * D + c + k));
                    s[k] = fmaf(u, bf16lo(q.x), s[k]);
                    s[k + 1] = fmaf(u, bf16hi(q.x), s[k + 1]);
                    s[k + 2] = fmaf(u, bf16lo(q.y), s[k + 2]);
                    s[k + 3] = fmaf(u, bf16hi(q.y), s[k + 3]);
                    s[k + 4] = fmaf(u, bf16lo(q.z), s[k + 4]);
                    s[k + 5] = fmaf(u, bf16hi(q.z), s[k + 5]);
                    s[k + 6] = fmaf(u, bf16lo(q.w), s[k + 6]);
                    s[k + 7] = fmaf(u, bf16hi(q.w), s[k + 7]);
                }
            if ((m & 31) == 31) {
                bool more = false;
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    more |= (left >> k & 1u) && s[k] == s[k];
                if (!__any_sync(0xffffffffu, more))
                    break;
            }
        }
#pragma unroll
        for (int k = 0; k < 32; ++k)
            if (left >> k & 1u)
                out[c + k] = s[k];
    }
}

__global__ void __launch_bounds__(kAOThreads, 2) k_ad_outer(AdOuterArgs p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *zeros = g_align1024(smem_raw), *ring = zeros + kAOBlock;
    AOSync &sy = *reinterpret_cast<AOSync *>(ring + (size_t)kAOStages * kAOStage);
    __shared__ int s_item[6];  // adapter, first row, rows, pieces, first scratch piece, piece
    __shared__ int s_scan[2 * (kAOWarps + 1)];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < kAOStages; ++s) {
            mbar_init(&sy.full[s], kAOWarps * 32);
            mbar_init(&sy.empty[s], 1);
        }
        mbar_init(&sy.done, 1);
        sy.abort = 0;
        s_item[0] = -1;
        fence_mbar_init();
    }
    for (int i = tid; i < kAOBlock / 16; i += kAOThreads)
        reinterpret_cast<uint4 *>(zeros)[i] = make_uint4(0u, 0u, 0u, 0u);
    pdl_wait();
    pdl_trigger();
    __syncthreads();
    const int which = (int)blockIdx.y >= p.dch0;
    const AdOuterProblem pr = which ? p.pr[1] : p.pr[0];
    const int c0 = (blockIdx.y - (which ? p.dch0 : 0)) * kAOCols, j0 = blockIdx.z * kAORanks;
    const int rp = ad_rp(p.r);

    // which piece: pieces before adapter e, and scratch pieces before it
    {
        int base = 0, sbase = 0;
        for (int e0 = 0; e0 < p.n; e0 += kAOThreads) {
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
                s_scan[kAOWarps + 1 + warp] = s;
            }
            __syncthreads();
            int wv = 0, wsum = 0, tv = 0, ts = 0;
            for (int w = 0; w <= kAOWarps; ++w) {
                if (w < warp) {
                    wv += s_scan[w];
                    wsum += s_scan[kAOWarps + 1 + w];
                }
                tv += s_scan[w];
                ts += s_scan[kAOWarps + 1 + w];
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
    const size_t plane = (size_t)p.r * pr.D;
    float *out = pr.g + (size_t)a * plane;
    if (pieces > 1) {  // scratch pieces hold both problems, problem 0 first
        const size_t plane0 = p.pr[0].g ? (size_t)p.r * p.pr[0].D : 0;
        const size_t both = plane0 + (p.pr[1].g ? (size_t)p.r * p.pr[1].D : 0);
        out = p.partial + (size_t)(s_item[4] + s_item[5]) * both + (which ? plane0 : 0);
    }
    const int ranks = min(kAORanks, p.r - j0), cols = min(kAOCols, pr.D - c0);
    if (len <= 0) {  // no rows
        for (int i = tid; i < ranks * (cols / 4); i += kAOThreads)
            *reinterpret_cast<float4 *>(out + (size_t)(j0 + i / (cols / 4)) * pr.D + c0 +
                                        i % (cols / 4) * 4) = make_float4(0.f, 0.f, 0.f, 0.f);
        return;
    }
    if (warp == kAOWarps) {
        tmem_alloc(&sy.tmem_base, kAOCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sy.tmem_base;
    const int ns = (len + kAORows - 1) / kAORows;

    if (warp == kAOWarps) {
        // ------------------------------------------------------------ MMAs
        if (lane == 0) {
            // both operands along M and N; N in whole sixteens
            const uint32_t idesc =
                umma_idesc_bf16(128, (cols + 15) & ~15) | (1u << 15) | (1u << 16);
            uint32_t acc = 0;
            for (int s = 0; s < ns; ++s) {
                const int b = s % kAOStages;
                if (s % kAOSegment == 0)
                    acc = 0;
                if (!mbar_wait(&sy.full[b], (s / kAOStages) & 1, p.status)) {
                    sy.abort = 1;
                    break;
                }
                // the copies are ordinary writes to the tensor core's proxy; fenced
                // here, where no copy is in flight (the fence of a thread that
                // has some waits for them, which took away the stages' overlap)
                fence_proxy_async_smem();
                tc_fence_after();
                const uint32_t at = smem_addr(ring + (size_t)b * kAOStage);
                const int steps = (min(kAORows, len - s * kAORows) + 15) / 16;
                const uint32_t za = smem_addr(zeros);
                for (int k = 0; k < steps; ++k) {
                    const uint64_t zd =
                        umma_desc_mn_sw128(at + kAdParts * kAOBlock + k * 2048, kAOBlock);
                    // the parts' blocks lie one behind another; the zeros before
                    // them all, the third part as far behind the zeros as it lies
                    umma_bf16(tmem, umma_desc_mn_sw128(at + k * 2048, kAOBlock), zd, idesc, acc);
                    umma_bf16(tmem,
                              umma_desc_mn_sw128(za + k * 2048, at + 2 * kAOBlock - za), zd, idesc, 1);
                    acc = 1;
                }
                umma_commit(&sy.empty[b]);
                // (its sum is read before the next segment's first stage is full)
                if ((s + 1) % kAOSegment == 0 && s + 1 < ns)
                    umma_commit(&sy.done);
            }
            umma_commit(&sy.done);
            mbar_wait(&sy.done, (ns - 1) / kAOSegment & 1, p.status);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ copies
        // a warp's rows of a stage: warp, warp + 8, ...; lane: a vector of eight
        // columns of z, and (the first ones) of a part's ranks
        const uint32_t sm = smem_addr(ring);
        const int nc = min(rp - j0, kAORanks) / 8;  // vectors of a part
        const int part = lane / nc, ch = lane - part * nc;
        const bool pl = part < kAdParts, zl = lane * 8 < cols;
        const uint16_t *zp = pr.z + c0 + lane * 8;
        const uint16_t *up = pr.parts + (pl ? (size_t)part * rp + j0 + ch * 8 : 0);
        const uint32_t zo = kAdParts * kAOBlock + (lane >> 3) * kAOBlock;
        constexpr int kMine = kAORows / kAOWarps;
        auto ids = [&](int s) {  // lane i: the row of this warp's i-th
            const int m = s * kAORows + warp + kAOWarps * lane;
            return lane < kMine && m < len ? __ldg(&p.row[first + m]) : -1;
        };
        int next = ids(0);
        uint32_t again = 0;  // blocks of 32 columns with a NaN
        for (int s0 = 0; s0 < ns; s0 += kAOSegment) {
            for (int s = s0; s < min(ns, s0 + kAOSegment); ++s) {
                const int id = next;
                next = s + 1 < ns ? ids(s + 1) : -1;
                const int b = s % kAOStages;
                int w = 1;
                if (lane == 0)
                    w = mbar_wait(&sy.empty[b], ((s / kAOStages) & 1) ^ 1, p.status);
                if (!__shfl_sync(0xffffffffu, w, 0)) {
                    sy.abort = 1;
                    break;
                }
                const uint32_t at = sm + b * kAOStage;
#pragma unroll
                for (int i = 0; i < kMine; ++i) {
                    const int t = __shfl_sync(0xffffffffu, id, i);
                    const bool live = (unsigned)t < (unsigned)p.T;
                    const int row = warp + kAOWarps * i;
                    // zeros for rows behind the piece: they are multiplied too
                    cp_async16(at + zo + row * 128 + (((lane & 7) ^ (row & 7)) << 4),
                               live && zl ? zp + (size_t)t * pr.D : pr.z, live && zl);
                    if (pl)
                        cp_async16(at + part * kAOBlock + row * 128 + ((ch ^ (row & 7)) << 4),
                                   live ? up + (size_t)t * kAdParts * rp : pr.parts, live);
                }
                cp_async_arrive(&sy.full[b]);
            }
            cp_async_wait<0>();
            // -------------------------------------------------------- epilogue
            // warps 2, 3, 6, 7 hold the lower half of tensor memory's lanes and hand
            // their sums over; warps 0, 1, 4, 5 add them and store
            int w = 1;
            if (lane == 0)
                w = mbar_wait(&sy.done, s0 / kAOSegment & 1, p.status);
            const bool good = __shfl_sync(0xffffffffu, w, 0) && !*(volatile int *)&sy.abort;
            tc_fence_after();
            const int quarter = warp & 3, r0 = (quarter & 1) * 32;  // first rank of this warp's lanes
            const uint32_t from = tmem + ((uint32_t)(quarter * 32) << 16);
            float *half = reinterpret_cast<float *>(ring);
            if (good && quarter >= 2 && r0 < ranks)
                for (int c = warp >> 2; c * 32 < cols; c += 2) {
                    float v[32];
                    __syncwarp();
                    tmem_ld32(from + c * 32, v);
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        *reinterpret_cast<float4 *>(half + (r0 + lane) * kAOHalfPitch + c * 32 + j) =
                            make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                }
            named_bar_sync(1, kAOWarps * 32);
            if (good && quarter < 2 && r0 < ranks)
                for (int c = warp >> 2; c * 32 < cols; c += 2) {
                    float v[32];
                    __syncwarp();
                    tmem_ld32(from + c * 32, v);
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 h = *reinterpret_cast<const float4 *>(
                            half + (r0 + lane) * kAOHalfPitch + c * 32 + j);
                        v[j] += h.x;
                        v[j + 1] += h.y;
                        v[j + 2] += h.z;
                        v[j + 3] += h.w;
                    }
                    ag_quad_rows(v);
                    if (ao_put(out + (size_t)j0 * pr.D + c0, pr.D, c * 32, r0, lane, ranks, cols, v,
                               s0 > 0))
                        again |= 1u << c;
                }
            tc_fence_before();
            if (s0 + kAOSegment < ns) {
                if (tid == 0)
                    sy.stop = *(volatile int *)&sy.abort;
                named_bar_sync(1, kAOWarps * 32);  // the lower half has been read
                if (*(volatile int *)&sy.stop)
                    break;
            }
        }
        if (again) {
            __syncwarp();
            const AdOuterProblem q = which ? p.pr[1] : p.pr[0];
            const int r0 = (warp & 1) * 32;
            ao_again(q.parts, q.z + c0, q.D, cols, p.row + s_item[1], s_item[2], p.T, ad_rp(p.r),
                     j0 + r0 + lane, r0 + lane < ranks, again, out + (size_t)(j0 + r0 + lane) * q.D + c0);
        }
    }
    __syncthreads();
    if (warp == kAOWarps) {
        tc_fence_after();
        tmem_dealloc(tmem, kAOCols);
    }
}

// The pieces of adapter blockIdx.y added in order: four values a thread, eight
// pieces' loads in flight.
__global__ void __launch_bounds__(256) k_ad_outer_join(AdOuterArgs p)
{
    __shared__ int s_before;
    const int tid = threadIdx.x, a = blockIdx.y;
    if (tid == 0)
        s_before = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const int len = __ldcg(&p.offsets[a + 1]) - __ldcg(&p.offsets[a]);
    if (len <= p.rows)
        return;
    const int pieces = (len + p.rows - 1) / p.rows;
    // scratch pieces of the adapters before
    int before = 0;
    for (int e = tid; e < a; e += 256) {
        const int l = __ldcg(&p.offsets[e + 1]) - __ldcg(&p.offsets[e]);
        if (l > p.rows)
            before += (l + p.rows - 1) / p.rows;
    }
    before = __reduce_add_sync(0xffffffffu, before);
    if ((tid & 31) == 0 && before)
        atomicAdd(&s_before, before);
    __syncthreads();
    const size_t plane0 = p.pr[0].g ? (size_t)p.r * p.pr[0].D : 0;
    const size_t plane1 = p.pr[1].g ? (size_t)p.r * p.pr[1].D : 0, both = plane0 + plane1;
    const size_t o = ((size_t)blockIdx.x * 256 + tid) * 4;
    if (o >= both)
        return;
    const float *from = p.partial + (size_t)s_before * both + o;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int k0 = 0; k0 < pieces; k0 += 8) {
        float4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k0 + k < pieces)
                v[k] = __ldcg(reinterpret_cast<const float4 *>(from + (size_t)(k0 + k) * both));
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k0 + k < pieces) {
                s.x += v[k].x;
                s.y += v[k].y;
                s.z += v[k].z;
                s.w += v[k].w;
            }
    }
    float *to = o < plane0 ? p.pr[0].g + (size_t)a * plane0 + o
                           : p.pr[1].g + (size_t)a * plane1 + (o - plane0);
    *reinterpret_cast<float4 *>(to) = s;
}

}  // namespace moe

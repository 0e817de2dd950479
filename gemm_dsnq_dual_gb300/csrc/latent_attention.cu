// Attention of one new token per request over a paged latent cache.
//
//   out[b, h, :] = sum_j p_j k_j[0:DV],  p = softmax_j(scale * q[b, h] . k_j),  j < len_b
//
// All heads of a request share the cache rows: a row is key (DK columns) and
// value (its first DV columns) at once, so a row of 2 DK bytes serves
// 2 H (DK + DV) operations.  At 128 heads that is 242 operations per byte,
// about what the GPU has (measured copy bandwidth and bf16 matrix rate: 291),
// so both the copies and the tensor cores have to run without a pause.
//
// Work split: the tiles of 64 tokens of all requests are laid end to end and
// cut into equal runs, one per worker (a worker is one CTA per group of 64
// heads), so long requests are split over many workers and short ones share a
// worker, whatever the mix.  Every CTA works the cut out from the lengths on
// the device, so nothing is planned on the host and the call can be captured.
// A run that covers a whole request writes its output; the others leave
// (sum, max, unnormalized output) in fp32 in the workspace, at two slots per
// worker, and a second kernel joins them in the order of the tokens (no
// atomics: results do not depend on timing).
//
// One CTA, 64 heads, tiles of 64 tokens:
//   S [64 heads x 64 tokens]   = Q K^T     M = 64, N = 64; both K-major in shared memory
//   O^T [DV x 64 heads]       += V^T P^T   M = 128, N = 64; V^T is the same cache tile read
//                                          column-major, P is bf16 in shared memory
// O is kept transposed because TMEM has 512 columns: 64 heads x 512 values take
// DV/128 x 64 = 256 of them at full use of its 128 lanes, which leaves room for
// two S buffers; heads x DV at M = 64 would take all 512.
// P is rounded to bf16 (half a step, 2^-9 relative) because the tensor core
// takes bf16; sums, maxima and O stay in fp32, and the sum is of the unrounded p.
// Warps: 0 copies tiles (TMA), 1 issues the MMAs, 2..5 the softmax, the
// rescaling of O and the output.  S(n+1) is computed while softmax(n) runs.
// The running maximum is raised (and O rescaled) only when a row's maximum
// grew by more than 2^8: until then p <= 2^8 is harmless in fp32 and bf16.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "debug_check.cuh"
#include "dsnq_internal.h"
#include "tensor_host.h"
#include "tensor_ptx.cuh"

namespace dsnq {
namespace attn {

constexpr int kHeads = 64;            // heads of a CTA
constexpr int kTile = 64;             // tokens of a tile
constexpr int kChunkCols = 64;        // columns of a 128-byte swizzled chunk
constexpr int kChunkBytes = 64 * 128; // 64 rows
constexpr int kThreads = 192;
constexpr int kSoftWarps = 4;
constexpr int kMaxStages = 8;
constexpr int kMaxCtas = 160;         // bound of workers x head groups
constexpr int kTmemCols = 512;
constexpr int kTmemS = 256;           // first column of the two S buffers
constexpr float kRaise = 8.0f;        // log2 by which a maximum may grow before O is rescaled
constexpr int kMiscBytes = 2048;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Params {
    const int32_t* seq_lens;
    const int32_t* table;
    int64_t ld_table;
    int B, H, G, W;                   // requests, heads, head groups, workers
    int width, page_size, box_rows, num_pages;
    int64_t cap;                      // tokens the table can hold per request
    int ck, nblk;                     // 64-column chunks of a row, 128-column blocks of the value
    int stages;
    float scale_log2;
    __nv_bfloat16* out;
    int64_t ldo_b, ldo_h;
    float* lse;                       // NULL: not written
    int64_t ldl_b;
    int4* meta;                       // [W] (first request, its first tile, tiles of the worker, tiles of the request)
    float2* part_ml;                  // [W * 2][G][64] (max in log2 units, sum)
    float* part_o;                    // [W * 2][G][64][DV]
    uint64_t timeout_ns;
    uint32_t inject;
};

__device__ __forceinline__ int request_len(const Params& p, int b) {
    const int64_t n = p.seq_lens[b];
    return static_cast<int>(n < 0 ? 0 : (n > p.cap ? p.cap : n));
}
// Tiles of a request; an empty one counts as one (somebody writes its zeros).
__device__ __forceinline__ int tiles_of(int len) { return len > kTile ? (len + kTile - 1) / kTile : 1; }

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y,
                                            int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// D[tmem] (+)= A[smem] * B[smem]^T, bf16 x bf16 -> fp32 (elected lane).
__device__ __forceinline__ void tc_mma_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Shared-memory descriptor of the cache tile read column-major (M runs along
// the 64 columns of a 128-byte row, then to the next chunk; K runs down the
// rows): leading byte offset = the next 64 columns, stride byte offset = the
// next 8 rows, 128-byte swizzle.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t addr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((addr >> 4) & 0x3FFF);
    d |= static_cast<uint64_t>((kChunkBytes >> 4) & 0x3FFF) << 16;
    d |= static_cast<uint64_t>((1024 >> 4) & 0x3FFF) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

// Instruction descriptor of kind::f16: D fp32, A and B bf16; a_mn: A column-major.
constexpr uint32_t idesc_bf16(int m, int n, bool a_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
        ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
          "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A worker's run of tiles, request by request.
struct Run {
    int b, t0, left;                  // request, its first tile of the run, tiles left in the run
    bool first;
    int len, tiles, n;                // of the current request: tokens, tiles, tiles of this run
    __device__ __forceinline__ bool next(const Params& p) {
        if (left <= 0) return false;
        len = request_len(p, b);
        tiles = tiles_of(len);
        n = min(tiles - t0, left);
        return true;
    }
    __device__ __forceinline__ void advance() {
        left -= n;
        ++b;
        t0 = 0;
        first = false;
    }
};

__global__ void __launch_bounds__(kThreads, 1)
latent_attention_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_kv,
                        const Params p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tile_bytes = p.ck * kChunkBytes;
    uint8_t* q_s = smem;                                   // [ck][64 heads][128 B]
    uint8_t* p_s = q_s + tile_bytes;                       // [64 heads][128 B]
    uint8_t* kv_s = p_s + kChunkBytes;                     // [stages][ck][64 tokens][128 B]
    uint8_t* misc = kv_s + p.stages * tile_bytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(misc);    // [kMaxStages]
    uint64_t* empty = full + kMaxStages;                   // [kMaxStages]
    uint64_t* qfull = empty + kMaxStages;
    uint64_t* qempty = qfull + 1;
    uint64_t* sfull = qempty + 1;                          // [2]
    uint64_t* sempty = sfull + 2;                          // [2]
    uint64_t* pfull = sempty + 2;
    uint64_t* pempty = pfull + 1;
    uint64_t* xch = pempty + 1;                            // the softmax warps among themselves
    uint64_t* drain = xch + 1;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    int* run_s = reinterpret_cast<int*>(tmem_holder + 2);  // [3] the worker's first request, first tile, tiles
    int64_t* sums = reinterpret_cast<int64_t*>(tmem_holder + 6);   // [kThreads / 32]
    float* alpha_s = reinterpret_cast<float*>(sums + kThreads / 32);   // [2][64]
    float* inv_s = alpha_s + 2 * kHeads;                   // [64]
    int* raise_s = reinterpret_cast<int*>(inv_s + kHeads); // [2][4]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int w = blockIdx.x / p.G, g = blockIdx.x - w * p.G;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        mbar_init(smem_u32(qfull), 1);
        mbar_init(smem_u32(qempty), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sfull[i]), 1);
            mbar_init(smem_u32(&sempty[i]), kSoftWarps);
        }
        mbar_init(smem_u32(pfull), kSoftWarps);
        mbar_init(smem_u32(pempty), 1);
        mbar_init(smem_u32(xch), kSoftWarps);
        mbar_init(smem_u32(drain), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tma_prefetch_desc(&map_q);
        tma_prefetch_desc(&map_kv);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    grid_dependency_wait();
    allow_dependent_launch();
    bounds_self_test(p.inject);

    // The worker's run: total tiles T, then the request that holds tile
    // w * T / workers.  Thread t sums requests [t * per, (t + 1) * per).
    {
        const int per = (p.B + kThreads - 1) / kThreads;
        const int b0 = min(static_cast<int>(threadIdx.x) * per, p.B), b1 = min(b0 + per, p.B);
        int64_t mine = 0;
        for (int b = b0; b < b1; ++b) mine += tiles_of(request_len(p, b));
        int64_t inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += u;
        }
        if (lane == 31) sums[warp] = inc;
        __syncthreads();
        int64_t before = inc - mine, total = 0;
        for (int i = 0; i < kThreads / 32; ++i) {
            if (i < warp) before += sums[i];
            total += sums[i];
        }
        const int64_t workers = total < p.W ? total : p.W;
        const int64_t begin = w < workers ? w * total / workers : 0;
        const int64_t end = w < workers ? (w + 1) * total / workers : 0;
        if (threadIdx.x == 0 && end == begin) run_s[2] = 0;
        if (end > begin && begin >= before && begin < before + mine) {
            int64_t at = before;
            int b = b0, n = tiles_of(request_len(p, b));
            while (at + n <= begin) {
                at += n;
                n = tiles_of(request_len(p, ++b));
            }
            run_s[0] = b;
            run_s[1] = static_cast<int>(begin - at);
            run_s[2] = static_cast<int>(end - begin);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    const uint64_t tmo = p.timeout_ns;
    Run run;
    run.b = run_s[0];
    run.t0 = run_s[1];
    run.left = run_s[2];
    run.first = true;
    const bool idle = run.left == 0;
    if (idle) run.b = run.t0 = 0;
    if (threadIdx.x == 0 && g == 0)
        p.meta[w] = make_int4(run.b, run.t0, run.left, idle ? 0 : tiles_of(request_len(p, run.b)));

    if (warp == 0) {
        // ------------------------------------------------------- TMA producer
        const int pieces = kTile / p.box_rows;             // page pieces of a tile (1, 2, 4 or 8)
        const uint32_t piece_bytes = p.box_rows * 128;
        uint32_t n = 0, nq = 0;
        bool ok = true;
        for (; ok && run.next(p); run.advance()) {
            if (run.len == 0) continue;
            const int32_t* row = p.table + run.b * p.ld_table;
            // Entries of the next 32 / pieces tiles, one per lane.
            const int batch = 32 / pieces;
            int ids = 0;
            ok = wait_bounded(smem_u32(qempty), (nq & 1) ^ 1, abort_flag, tmo);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(smem_u32(qfull), tile_bytes);
            __syncwarp();
            if (lane < p.ck)
                tma_load_3d(smem_u32(q_s + lane * kChunkBytes), &map_q, smem_u32(qfull), lane * kChunkCols, g * kHeads,
                            run.b);
            ++nq;
            for (int i = 0; i < run.n; ++i, ++n) {
                const int tile = run.t0 + i;
                if (i % batch == 0) {
                    const int64_t tok = static_cast<int64_t>(tile) * kTile + static_cast<int64_t>(lane) * p.box_rows;
                    ids = 0;
                    if (tok < run.len) {
                        const int64_t e = tok / p.page_size;
                        if (bounds_ok(e < p.width)) ids = row[e];
                        if (ids < 0 || ids >= p.num_pages) {   // such pages read as zeros
                            atomicOr(&g_status, kStatusBounds);
                            ids = p.num_pages;
                        }
                    }
                }
                const int s = n % p.stages;
                ok = wait_bounded(smem_u32(&empty[s]), ((n / p.stages) & 1) ^ 1, abort_flag, tmo);
                if (!ok) break;
                const int tok0 = tile * kTile;
                const int live = min(pieces, (run.len - tok0 + p.box_rows - 1) / p.box_rows);
                const uint32_t fb = smem_u32(&full[s]);
                if ((p.inject & kInjectSkipLoad) && n == 0) continue;   // test hook: the waits on it run out
                if (lane == 0) mbar_arrive_expect_tx(fb, live * piece_bytes * p.ck);
                __syncwarp();
                const uint32_t dst = smem_u32(kv_s) + s * tile_bytes;
                for (int e = lane; e - lane < live * p.ck; e += 32) {
                    const bool on = e < live * p.ck;
                    const int piece = on ? e / p.ck : 0, c = on ? e - piece * p.ck : 0;
                    const int id = __shfl_sync(0xffffffffu, ids, (i % batch) * pieces + piece);
                    const int y = (tok0 + piece * p.box_rows) % p.page_size;
                    if (on) tma_load_3d(dst + c * kChunkBytes + piece * piece_bytes, &map_kv, fb, c * kChunkCols, y, id);
                }
            }
        }
        if (!ok) settle_ns(kAbortSettleNs);                // copies already issued land before the CTA goes
    } else if (warp == 1) {
        // --------------------------------------------------------- MMA issuer
        const uint32_t id_s = idesc_bf16(64, kTile, false), id_o = idesc_bf16(128, kHeads, true);
        uint32_t n = 0, nq = 0;
        int pend = -1;                                     // stage whose P V product is still to be issued
        bool pend_first = false, ok = true;
        const uint64_t q_desc = smem_desc_k_sw128(smem_u32(q_s)), p_desc = smem_desc_k_sw128(smem_u32(p_s));
        // O^T (+)= V^T P^T of tile n - 1.
        auto issue_pv = [&]() -> bool {
            if (!wait_bounded(smem_u32(pfull), (n - 1) & 1, abort_flag, tmo)) return false;
            tc_fence_after();
            const uint32_t v0 = smem_u32(kv_s) + pend * tile_bytes;
            for (int blk = 0; blk < p.nblk; ++blk) {
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    tc_mma_bf16(tmem + blk * kHeads, smem_desc_mn_sw128(v0 + blk * 2 * kChunkBytes + k * 16 * 128),
                                p_desc + k * 2, id_o, !(pend_first && k == 0));
            }
            tc_commit(smem_u32(&empty[pend]));
            tc_commit(smem_u32(pempty));
            return true;
        };
        for (; ok && run.next(p); run.advance()) {
            if (run.len == 0) continue;
            ok = wait_bounded(smem_u32(qfull), nq & 1, abort_flag, tmo);
            if (!ok) break;
            ++nq;
            for (int i = 0; i < run.n; ++i) {
                const int s = n % p.stages;
                ok = wait_bounded(smem_u32(&full[s]), (n / p.stages) & 1, abort_flag, tmo) &&
                     wait_bounded(smem_u32(&sempty[n & 1]), ((n >> 1) & 1) ^ 1, abort_flag, tmo);
                if (!ok) break;
                tc_fence_after();
                const uint64_t k_desc = smem_desc_k_sw128(smem_u32(kv_s) + s * tile_bytes);
                for (int c = 0; c < p.ck; ++c) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc_mma_bf16(tmem + kTmemS + (n & 1) * kTile, q_desc + c * (kChunkBytes >> 4) + k * 2,
                                    k_desc + c * (kChunkBytes >> 4) + k * 2, id_s, (c | k) != 0);
                }
                tc_commit(smem_u32(&sfull[n & 1]));
                if (i == run.n - 1) tc_commit(smem_u32(qempty));
                if (pend >= 0 && !(ok = issue_pv())) break;
                pend = s;
                pend_first = i == 0;
                ++n;
            }
        }
        if (ok && pend >= 0) ok = issue_pv();
        if (!ok) {                                         // MMAs already issued end before their memory goes
            tc_commit(smem_u32(drain));
            wait_drain(smem_u32(drain), 0, tmo);
        }
    } else {
        // ------------------------------------- softmax, rescaling and output
        const int quad = warp & 3;                         // TMEM lanes 32 * quad ..
        const uint32_t tl = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        const int st = threadIdx.x - 64;                   // 0..127
        // S at M = 64: row 16 * quad + i is lane 32 * quad + i, i < 16.
        const bool on = lane < 16;
        const int row = quad * 16 + (lane & 15);
        const int DV = p.nblk * 128;
        uint32_t n = 0, nx = 0;
        bool ok = true;
        // Barrier of the four warps.  An mbarrier, whose waits are bounded:
        // after an abort a warp may leave without the others.
        auto exchange = [&]() -> bool {
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(xch));
            return wait_bounded<true>(smem_u32(xch), nx++ & 1, abort_flag, tmo);
        };
        for (; ok && run.next(p); run.advance()) {
            const int b = run.b;
            const bool whole = run.t0 == 0 && run.n == run.tiles;
            if (run.len == 0) {
                // An empty request: zeros, and the logarithm of an empty sum.
                for (int e = st; e < kHeads * (DV / 8); e += 128) {
                    const int h = g * kHeads + e / (DV / 8), c = e % (DV / 8);
                    if (h < p.H && bounds_ok(b < p.B))
                        *reinterpret_cast<uint4*>(p.out + b * p.ldo_b + h * p.ldo_h + c * 8) = make_uint4(0, 0, 0, 0);
                }
                if (p.lse && st < kHeads && g * kHeads + st < p.H)
                    p.lse[b * p.ldl_b + g * kHeads + st] = __int_as_float(0xff800000);
                continue;
            }
            float m = __int_as_float(0xff800000), l = 0.f;  // maximum of the raw scores in use, sum of p
            for (int i = 0; i < run.n; ++i, ++n) {
                const int tok0 = (run.t0 + i) * kTile;
                const int valid = min(kTile, run.len - tok0);
                ok = wait_bounded(smem_u32(&sfull[n & 1]), (n >> 1) & 1, abort_flag, tmo);
                if (!ok) break;
                tc_fence_after();
                uint64_t sp[kTile / 2];
                tmem_ld_pairs<kTile>(tl + kTmemS + (n & 1) * kTile, sp);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sempty[n & 1]));
                float s[kTile];
#pragma unroll
                for (int j = 0; j < kTile / 2; ++j) {
                    const float2 f = as_float2(sp[j]);
                    s[2 * j] = f.x;
                    s[2 * j + 1] = f.y;
                }
                if (valid < kTile) {
#pragma unroll
                    for (int j = 0; j < kTile; ++j)
                        if (j >= valid) s[j] = __int_as_float(0xff800000);
                }
                float top = s[0];
#pragma unroll
                for (int j = 1; j < kTile; ++j) top = fmaxf(top, s[j]);
                // Raise the maximum when it grew too far (always on the first tile).
                float alpha = 1.f;
                bool raise = false;
                if (on && (top - m) * p.scale_log2 > kRaise) {
                    raise = i > 0;
                    alpha = exp2_fast((m - top) * p.scale_log2);
                    m = top;
                }
                if (on) alpha_s[(n & 1) * kHeads + row] = alpha;
                const bool any = __any_sync(0xffffffffu, raise);
                if (lane == 0) raise_s[(n & 1) * kSoftWarps + quad] = any;
                ok = exchange();
                if (!ok) break;
                const int* rs = raise_s + (n & 1) * kSoftWarps;
                if (rs[0] | rs[1] | rs[2] | rs[3]) {
                    ok = wait_bounded(smem_u32(pempty), (n & 1) ^ 1, abort_flag, tmo);   // product n - 1 is in O
                    if (!ok) break;
                    tc_fence_after();
                    l *= alpha;
                    const float* al = alpha_s + (n & 1) * kHeads;
                    for (int c = 0; c < p.nblk * kHeads; c += 16) {
                        uint32_t r[16];
                        tmem_ld16_issue(tl + c, r);
                        tmem_ld16_wait(r);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            r[j] = __float_as_uint(__uint_as_float(r[j]) * al[(c & (kHeads - 1)) + j]);
                        tmem_st16(tl + c, r);
                    }
                    tmem_wait_st();
                }
                const float off = m == __int_as_float(0xff800000) ? 0.f : m * p.scale_log2;
                uint32_t pk[kTile / 2];
                float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
                for (int j = 0; j < kTile / 2; ++j) {
                    const float e0 = exp2_fast(fmaf(s[2 * j], p.scale_log2, -off));
                    const float e1 = exp2_fast(fmaf(s[2 * j + 1], p.scale_log2, -off));
                    sum0 += e0;
                    sum1 += e1;
                    const __nv_bfloat162 h = __floats2bfloat162_rn(e0, e1);
                    memcpy(&pk[j], &h, 4);
                }
                l += sum0 + sum1;
                // P's buffer is free once product n - 1 is done.
                ok = n == 0 || wait_bounded(smem_u32(pempty), (n & 1) ^ 1, abort_flag, tmo);
                if (!ok) break;
                if (on) {
                    uint8_t* dst = p_s + row * 128;
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        *reinterpret_cast<uint4*>(dst + ((c ^ (row & 7)) << 4)) =
                            make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
                }
                if (valid < kTile) {
                    // Rows past the length hold whatever the page or the
                    // buffer held: 0 * NaN would reach O, so they become 0.
                    const int stage = n % p.stages;
                    ok = wait_bounded(smem_u32(&full[stage]), (n / p.stages) & 1, abort_flag, tmo);
                    if (!ok) break;
                    uint8_t* kv = kv_s + stage * tile_bytes;
                    const int per = (kTile - valid) * 8;   // 16-byte words of a chunk
                    for (int e = st; e < per * p.nblk * 2; e += 128) {
                        const int c = e / per, v = e - c * per;
                        *reinterpret_cast<uint4*>(kv + c * kChunkBytes + valid * 128 + v * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(pfull));
            }
            if (!ok) break;
            // ---- output of the request (or of this worker's part of it)
            ok = wait_bounded(smem_u32(pempty), (n & 1) ^ 1, abort_flag, tmo);
            if (!ok) break;
            tc_fence_after();
            const int head = g * kHeads + row;
            const float m2 = m == __int_as_float(0xff800000) ? m : m * p.scale_log2;
            const int64_t slot = (static_cast<int64_t>(w) * 2 + (run.first ? 0 : 1)) * p.G + g;
            if (on) {
                inv_s[row] = l > 0.f || l != l ? 1.0f / l : 0.f;
                if (whole) {
                    if (p.lse && head < p.H)
                        p.lse[b * p.ldl_b + head] = l == 0.f ? __int_as_float(0xff800000) : (m2 + log2f(l)) * kLn2;
                } else {
                    p.part_ml[slot * kHeads + row] = make_float2(m2, l);
                }
            }
            ok = exchange();                               // inv_s is next written after another exchange
            if (!ok) break;
            const int heads = min(kHeads, p.H - g * kHeads);
            for (int blk = 0; blk < p.nblk; ++blk) {
                const int dv = blk * 128 + quad * 32 + lane;
                for (int c = 0; c < heads; c += 16) {
                    uint32_t r[16];
                    tmem_ld16_issue(tl + blk * kHeads + c, r);
                    tmem_ld16_wait(r);
                    if (whole) {
                        __nv_bfloat16* o = p.out + b * p.ldo_b + static_cast<int64_t>(g * kHeads + c) * p.ldo_h + dv;
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (c + j < heads && bounds_ok(b < p.B && dv < DV))
                                o[j * p.ldo_h] = __float2bfloat16_rn(__uint_as_float(r[j]) * inv_s[c + j]);
                    } else {
                        float* o = p.part_o + (slot * kHeads + c) * DV + dv;
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (c + j < heads && bounds_ok(w < p.W && dv < DV)) o[j * DV] = __uint_as_float(r[j]);
                    }
                }
            }
            tc_fence_before();
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// ---------------------------------------------------------------------------
// Joins the parts of requests that more than one worker took.  A request is
// found at the first worker boundary inside it; its parts are that boundary's
// left neighbour's and those of the workers from there to its end, in the
// order of the tokens.
//   out = sum_k 2^(m_k - M) o_k / sum_k 2^(m_k - M) l_k,  M = max_k m_k
// Items: with few parts (<= 8) one warp per (head, 128 columns), eight heads'
// worth per CTA step; with many, eight warps share the parts of one.
// ---------------------------------------------------------------------------
constexpr int kJoinWarps = 8;
constexpr int kFewParts = 8;

__global__ void __launch_bounds__(kJoinWarps * 32)
latent_attention_join_kernel(const Params p) {
    grid_dependency_wait();
    allow_dependent_launch();
    bounds_self_test(p.inject);
    __shared__ int first_item[kMaxCtas + 1];               // running item count by boundary
    __shared__ int parts_s[kMaxCtas];
    __shared__ float4 red[kJoinWarps][32];
    __shared__ float red_l[kJoinWarps], red_m[kJoinWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int DV = p.nblk * 128;
    const int few_items = (p.H * p.nblk + kJoinWarps - 1) / kJoinWarps, many_items = p.H * p.nblk;

    if (threadIdx.x < static_cast<unsigned>(p.W)) {
        int parts = 0;
        const int w = threadIdx.x;
        if (w > 0) {
            const int4 me = p.meta[w], left = p.meta[w - 1];
            if (me.z > 0 && me.y > 0 && left.z >= me.y) {
                int covered = me.y, k = w;
                parts = 1;
                while (covered < me.w && k < p.W) {
                    covered += p.meta[k].z;
                    ++k;
                    ++parts;
                }
            }
        }
        parts_s[w] = parts;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int at = 0;
        for (int w = 0; w < p.W; ++w) {
            first_item[w] = at;
            at += parts_s[w] == 0 ? 0 : (parts_s[w] <= kFewParts ? few_items : many_items);
        }
        first_item[p.W] = at;
    }
    __syncthreads();
    int w = 0;
    for (int item = blockIdx.x; item < first_item[p.W]; item += gridDim.x) {
        while (item >= first_item[w + 1]) ++w;
        const int parts = parts_s[w];
        const bool few = parts <= kFewParts;
        const int sub = few ? (item - first_item[w]) * kJoinWarps + warp : item - first_item[w];
        const int step = few ? 1 : kJoinWarps, k0 = few ? 0 : warp;
        const bool on = sub < p.H * p.nblk;
        const int h = on ? sub / p.nblk : 0, blk = on ? sub - h * p.nblk : 0;
        const int g = h / kHeads, row = h - g * kHeads;
        const int4 me = p.meta[w];
        const int left_slot = p.meta[w - 1].z == me.y ? 0 : 1;
        auto slot_of = [&](int k) -> int64_t {             // part k's place in the workspace
            const int64_t s = k == 0 ? (w - 1) * 2 + left_slot : (w + k - 1) * 2;
            return (s * p.G + g) * kHeads + row;
        };
        float M = __int_as_float(0xff800000);
        for (int k = k0; k < parts; k += step) M = fmaxf(M, p.part_ml[slot_of(k)].x);
        if (!few) {
            if (lane == 0) red_m[warp] = M;
            __syncthreads();
            M = red_m[0];
#pragma unroll
            for (int i = 1; i < kJoinWarps; ++i) M = fmaxf(M, red_m[i]);
        }
        const float base = M == __int_as_float(0xff800000) ? 0.f : M;
        float L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = k0; k < parts; k += step) {
            const int64_t s = slot_of(k);
            const float2 ml = p.part_ml[s];
            const float4 o = *reinterpret_cast<const float4*>(p.part_o + s * DV + blk * 128 + lane * 4);
            const float f = exp2_fast(ml.x - base);
            L = fmaf(ml.y, f, L);
            acc.x = fmaf(o.x, f, acc.x);
            acc.y = fmaf(o.y, f, acc.y);
            acc.z = fmaf(o.z, f, acc.z);
            acc.w = fmaf(o.w, f, acc.w);
        }
        if (!few) {
            red[warp][lane] = acc;
            if (lane == 0) red_l[warp] = L;
            __syncthreads();
            if (warp == 0) {
#pragma unroll
                for (int i = 1; i < kJoinWarps; ++i) {
                    const float4 o = red[i][lane];
                    acc.x += o.x; acc.y += o.y; acc.z += o.z; acc.w += o.w;
                    L += red_l[i];
                }
            }
        }
        if (on && (few || warp == 0) && bounds_ok(me.x < p.B && h < p.H)) {
            const float inv = L > 0.f || L != L ? 1.0f / L : 0.f;
            const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
            const __nv_bfloat162 c = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
            uint2 v;
            memcpy(&v.x, &a, 4);
            memcpy(&v.y, &c, 4);
            *reinterpret_cast<uint2*>(p.out + me.x * p.ldo_b + h * p.ldo_h + blk * 128 + lane * 4) = v;
            if (p.lse && blk == 0 && lane == 0)
                p.lse[me.x * p.ldl_b + h] = L == 0.f ? __int_as_float(0xff800000) : (M + log2f(L)) * kLn2;
        }
        if (!few) __syncthreads();                         // the buffers are free for the next item
    }
}

// --------------------------------------------------------------------- host

// 3-D map of bf16 [n2][n1][n0] with strides ld2, ld1, 1 (elements); box 64
// columns x rows x 1, 128-byte swizzle, zeros outside.
bool make_map_3d(CUtensorMap* m, const void* base, int64_t n0, int64_t n1, int64_t n2, int64_t ld1, int64_t ld2, int rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(n0), static_cast<cuuint64_t>(n1), static_cast<cuuint64_t>(n2)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld1 * 2), static_cast<cuuint64_t>(ld2 * 2)};
    cuuint32_t box[3] = {kChunkCols, static_cast<cuuint32_t>(rows), 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Workers of a call (CTAs per head group), bounded by the device and by the
// most tiles that the tables can hold.
int64_t workers_for(int64_t B, int64_t G, int64_t cap, int64_t ctas) {
    const int64_t per = cap > kTile ? (cap + kTile - 1) / kTile : 1;
    int64_t w = ctas / G;
    if (w < 1) w = 1;
    return (w - 1) / per + 1 <= B ? w : B * per;           // min(w, B * per) without overflow
}

struct Layout {
    int64_t meta, ml, o, total;                            // byte offsets of the workspace's parts
};
Layout workspace_layout(int64_t W, int64_t G, int64_t DV) {
    Layout L;
    const int64_t slots = W * 2 * G * kHeads;
    L.meta = 0;
    L.ml = (W * 16 + 255) / 256 * 256;
    L.o = (L.ml + slots * 8 + 255) / 256 * 256;
    L.total = L.o + slots * DV * 4;
    return L;
}

dsnq_status check_sizes(int64_t B, int64_t H, int64_t DK, int64_t DV, int64_t width, int64_t page_size) {
    if (B < 0 || H <= 0 || DK <= 0 || DV <= 0 || width < 0 || page_size <= 0) return DSNQ_ERR_INVALID_ARG;
    if (DV > DK) return DSNQ_ERR_INVALID_ARG;
    if (DK % 64 || DV % 128 || DK > 576 || DV > 512 || H > 1024 || B > DSNQ_MAX_REQUESTS || page_size % 8 ||
        page_size > (1 << 20) || width > 0x7fffffffLL || width * page_size > 0x7fffff00LL)
        return DSNQ_ERR_UNSUPPORTED;
    return DSNQ_OK;
}

}  // namespace attn

bool take_attention_words(cudaStream_t s, unsigned int* v) {
    unsigned int w = 0, st = 0;
    const unsigned int zero = 0;
    if (!take_debug_word(s, &w)) return false;
    if (cudaMemcpyFromSymbolAsync(&st, g_status, sizeof(st), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess ||
        cudaMemcpyToSymbolAsync(g_status, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    *v = w | st;
    return true;
}

}  // namespace dsnq

using namespace dsnq;

extern "C" dsnq_status dsnq_paged_latent_attention_workspace_bytes(int64_t B, int64_t H, int64_t DV, int64_t table_width,
                                                                   int64_t page_size, int64_t* bytes) {
    const dsnq_status st = attn::check_sizes(B, H, DV, DV, table_width, page_size);
    if (st != DSNQ_OK) return st;
    const int64_t G = (H + attn::kHeads - 1) / attn::kHeads;
    const int64_t W = attn::workers_for(B, G, table_width * page_size, attn::kMaxCtas);
    if (bytes) *bytes = B == 0 ? 0 : attn::workspace_layout(W, G, DV).total;
    return DSNQ_OK;
}

extern "C" dsnq_status dsnq_paged_latent_attention(
    int64_t B, int64_t H, int64_t DK, int64_t DV, const void* q, int64_t ldq_tok, int64_t ldq_head, const void* cache,
    int64_t num_pages, int64_t page_size, int64_t ld_page, int64_t ld_row, const int32_t* block_table, int64_t table_width,
    int64_t ld_table, const int32_t* seq_lens, float scale, void* out, int64_t ldo_tok, int64_t ldo_head, float* lse,
    int64_t ldl_tok, void* workspace, int64_t workspace_bytes, void* stream) {
    using namespace dsnq::attn;
    dsnq_status st = check_sizes(B, H, DK, DV, table_width, page_size);
    if (st != DSNQ_OK) return st;
    if (num_pages < 1 || !(scale > 0.f && scale < 1.0e30f) || workspace_bytes < 0) return DSNQ_ERR_INVALID_ARG;
    if (num_pages > 0x7ffffffeLL || ld_row > (1LL << 36) || ld_page > (1LL << 38)) return DSNQ_ERR_UNSUPPORTED;
    if (B == 0) return DSNQ_OK;
    if (!q || !out || !seq_lens || !workspace || !cache || (table_width && !block_table))
        return DSNQ_ERR_INVALID_ARG;
    if ((H > 1 && (ldq_head < DK || ldo_head < DV)) || (B > 1 && (ldq_tok < DK || ldo_tok < DV || ld_table < table_width)) ||
        (B > 1 && lse && ldl_tok < H) || ld_row < DK || ld_page < (page_size - 1) * ld_row + DK)
        return DSNQ_ERR_INVALID_ARG;
    if (!aligned(q, 16) || ldq_tok % 8 || ldq_head % 8 || !aligned(cache, 16) || ld_page % 8 || ld_row % 8 ||
        !aligned(out, 16) || ldo_tok % 8 || ldo_head % 8 || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(lse, 4) || !aligned(workspace, 16))
        return DSNQ_ERR_MISALIGNED;
    const int64_t G = (H + kHeads - 1) / kHeads;
    const int64_t cap = table_width * page_size;
    if (workspace_bytes < workspace_layout(workers_for(B, G, cap, kMaxCtas), G, DV).total) return DSNQ_ERR_INVALID_ARG;
    const int sms = device_sm_count();
    if (sms <= 0) {
        cudaGetLastError();
        return DSNQ_ERR_CUDA;
    }
    Params p{};
    p.W = static_cast<int>(workers_for(B, G, cap, sms < kMaxCtas ? sms : kMaxCtas));
    p.seq_lens = seq_lens;
    p.table = block_table;
    p.ld_table = ld_table;
    p.B = static_cast<int>(B); p.H = static_cast<int>(H); p.G = static_cast<int>(G);
    p.width = static_cast<int>(table_width);
    p.page_size = static_cast<int>(page_size);
    p.num_pages = static_cast<int>(num_pages);
    p.cap = cap;
    p.box_rows = page_size % 64 == 0 ? 64 : page_size % 32 == 0 ? 32 : page_size % 16 == 0 ? 16 : 8;
    p.ck = static_cast<int>(DK / 64);
    p.nblk = static_cast<int>(DV / 128);
    const int64_t tile_bytes = static_cast<int64_t>(p.ck) * kChunkBytes;
    const int64_t fixed = 1024 + tile_bytes + kChunkBytes + kMiscBytes;
    int64_t stages = (227 * 1024 - fixed) / tile_bytes;
    if (stages > kMaxStages) stages = kMaxStages;
    p.stages = static_cast<int>(stages);
    const size_t smem = static_cast<size_t>(fixed + stages * tile_bytes);
    p.scale_log2 = scale * kLog2e;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.ldo_b = ldo_tok; p.ldo_h = ldo_head;
    p.lse = lse; p.ldl_b = ldl_tok;
    const Layout lay = workspace_layout(p.W, G, DV);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.meta = reinterpret_cast<int4*>(ws + lay.meta);
    p.part_ml = reinterpret_cast<float2*>(ws + lay.ml);
    p.part_o = reinterpret_cast<float*>(ws + lay.o);
    const uint64_t t = debug_wait_timeout_ns();
    p.timeout_ns = t ? t : kDefaultTimeoutNs;
    p.inject = debug_inject_flags();

    CUtensorMap mq, mk;
    // A lone token or head has no stride of its own: any valid one will do.
    const int64_t qh = H > 1 ? ldq_head : DK, qt = B > 1 ? ldq_tok : H * qh;
    if (!make_map_3d(&mq, q, DK, H, B, qh, qt, kHeads) ||
        !make_map_3d(&mk, cache, DK, page_size, num_pages, ld_row, ld_page, p.box_rows))
        return DSNQ_ERR_CUDA;
    if (!set_smem_attr(reinterpret_cast<const void*>(latent_attention_kernel), smem)) return DSNQ_ERR_CUDA;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    st = launch_result(launch_kernel(latent_attention_kernel, dim3(static_cast<unsigned>(p.W * G)), dim3(kThreads), smem, s,
                                     mq, mk, p));
    if (st != DSNQ_OK || p.W == 1) return st;
    const int64_t items = static_cast<int64_t>(p.W - 1) * H * p.nblk / kJoinWarps + 1;
    const int64_t grid = items < 4 * sms ? items : 4 * sms;
    return launch_result(launch_kernel(latent_attention_join_kernel, dim3(static_cast<unsigned>(grid)),
                                       dim3(kJoinWarps * 32), 0, s, p));
}

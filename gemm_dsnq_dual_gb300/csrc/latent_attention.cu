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
// worker, whatever the mix; requests that are about a worker's share each stay
// whole.  Every CTA works the cut out from the lengths on
// the device, so nothing is planned on the host and the call can be captured.
// A run that covers a whole request writes its output; the others leave
// (sum, max, output times that sum) in fp32 in the workspace, at two slots per
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
// P is rounded to bf16 (half a step, 2^-8 relative) because the tensor core
// takes bf16; sums, maxima and O stay in fp32.  O is divided by the sum of the
// rounded p, so that the weights add up to one and an output lies among the
// values it is made of; lse, and the weight of a part among the others, is of
// the unrounded sum.
// Warps: 0 copies tiles (TMA), 1 issues the products Q K^T, 6 the products P V,
// 2..5 do the softmax, the rescaling of O and the output.  S(n+1) is computed
// while softmax(n) runs.  Two issuing warps, because the two products wait for
// different things (a copy, a softmax): one warp that polls both barriers
// spends more time on the polls than the tensor core on the products.
// The running maximum is raised (and O rescaled) only when a row's maximum
// grew by more than 2^8: until then p <= 2^8 is harmless in fp32 and bf16.
// Shared memory (227 KB) holds q (72 KB at 64 heads x 576), P and two tiles and
// more: tiles come in pairs of 64-column chunks, each freed as soon as its
// product with P is done, so that the next tile's copies start early.
//
// Measured on GB300, 576 columns, between requests of 2048 and 8192 tokens, one
// to a worker: 1.61 us per tile and CTA at 16 heads, 1.73 at 64 (7.0 and 6.5
// TB/s over 152 CTAs: HBM bounds it), 1.70 at 128 heads, where two CTAs read
// each tile (3.3 TB/s).  There the products bound it: alone on an SM one of Q
// K^T takes 48 cycles and one of P V 61, so the 36 and 16 of a tile 2704 of its
// ~3500; the rest is the ring of two tiles, which refills as P V frees it.  Per
// call in a graph: 2 requests of 131071 tokens at 16 heads 59 us (floor 45), 128
// of 8000 at 48 heads, 512 columns, 191 us (159), 96 of mixed lengths at 128
// heads 105 us (44), one of 701 at 128 heads 13 us: ~1.8 us to the first copy,
// ~2.5 us to the first product and 4 to 7 us for parts and join do not shrink
// with the work.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "debug_check.cuh"
#include "group_quant.cuh"
#include "dsnq_internal.h"
#include "latent_tiles.cuh"
#include "tensor_host.h"
#include "tensor_ptx.cuh"

namespace dsnq {
namespace attn {

constexpr int kHeads = 64;            // heads of a CTA
constexpr int kTile = 64;             // tokens of a tile
constexpr int kChunkCols = 64;        // columns of a 128-byte swizzled chunk
constexpr int kChunkBytes = 64 * 128; // one chunk of a tile
constexpr int kPairBytes = 2 * kChunkBytes;
constexpr int kThreads = 224;
constexpr int kSoftWarps = 4;
constexpr int kMaxPairs = 13;         // slots of the ring of chunk pairs
constexpr int kMaxOdd = 3;            // slots of the ring of odd chunks
constexpr int kMaxCtas = 160;         // bound of workers x head groups
constexpr int kTmemCols = 512;
constexpr int kTmemS = 256;           // first column of the two S buffers
constexpr float kRaise = 8.0f;        // log2 by which a maximum may grow before O is rescaled
constexpr int kMiscBytes = 2048;
constexpr int kManyParts = 4;         // workers per request from which a CTA joins an item
constexpr int kRequestUnits = 2;      // what a request costs a worker beside its tiles, in tiles, at most

struct Params {
    const int32_t* seq_lens;
    const int32_t* table;
    int64_t ld_table;
    int B, H, G, W;                   // requests, heads, head groups, workers
    int W_full;                       // workers that the GPU has room for, whatever the tables hold
    int width, page_size, box_rows, num_pages;   // box_rows: tokens of one copy
    int64_t cap;                      // tokens the table can hold per request
    int ck, nblk;                     // 64-column chunks of a row, 128-column blocks of the value
    int q_rows;                       // rows of a chunk of q in shared memory (heads, a multiple of 8)
    int pair_slots, odd_slots;        // slots of the two rings
    float scale_log2;
    __nv_bfloat16* out;
    int64_t ldo_b, ldo_h;
    float* lse;                       // NULL: not written
    int64_t ldl_b;
    int2* meta;                       // [W] first request of the worker and its first tile there
    float2* part_ml;                  // [W * 2][G][64] (max in log2 units, sum)
    float* part_o;                    // [W * 2][G][nblk][16][128][4]: value block, four heads, value, head
    uint64_t timeout_ns;
    uint32_t inject;
};

__device__ __forceinline__ int clamp_len(const Params& p, int32_t n) {
    return n < 0 ? 0 : (n > p.cap ? static_cast<int>(p.cap) : n);
}
__device__ __forceinline__ int request_len(const Params& p, int b) { return clamp_len(p, p.seq_lens[b]); }
// Tiles of a request; an empty one counts as one (somebody writes its zeros).
__device__ __forceinline__ int tiles_of(int len) { return len > kTile ? (len + kTile - 1) / kTile : 1; }

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t y, int32_t w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %3, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(y), "r"(w)
        : "memory");
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t chunk, int32_t group,
                                            int32_t page, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(chunk), "r"(group), "r"(page), "l"(policy)
        : "memory");
}

// A place in a ring of shared-memory slots and the parity of its pass.
struct Place {
    int i = 0;
    uint32_t pass = 0;
    __device__ __forceinline__ void step(int slots) {
        if (++i == slots) {
            i = 0;
            pass ^= 1;
        }
    }
};

// Four steps of D[tmem] (+)= A[smem] * B[smem]^T, bf16 x bf16 -> fp32, K = 16
// each; A and B advance by ASTEP and BSTEP (16-byte units) a step, the first
// overwrites D when !accumulate.  One elected lane issues all four: with an
// election and 64-bit descriptor arithmetic for each, the issuing warp itself
// held the products back (61 cycles a step against 39).
template <int ASTEP, int BSTEP>
__device__ __forceinline__ void tc_mma4_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e, t;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.eq.b32 t, 0, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "add.u64 a, %1, %5;\n\tadd.u64 b, %2, %6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
        "add.u64 a, %1, %7;\n\tadd.u64 b, %2, %8;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
        "add.u64 a, %1, %9;\n\tadd.u64 b, %2, %10;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "n"(ASTEP), "n"(BSTEP), "n"(2 * ASTEP), "n"(2 * BSTEP),
        "n"(3 * ASTEP), "n"(3 * BSTEP)
        : "memory");
}

// Shared-memory descriptors.  A tile comes in pairs of 64-column chunks (16 KB)
// and, when the row has an odd number of chunks, one chunk (8 KB) by itself.  A
// pair lies as [8 groups of 8 tokens][2 chunks][8 tokens][128 bytes], 128-byte
// swizzle: one copy then takes whole groups of a page, whatever its size.  Read
// K-major (S = Q K^T), the next 8 tokens are a group (2 KB; odd chunk: 1 KB)
// on.  Read column-major (V^T: M runs along the 64 columns of a chunk and on to
// the next chunk, 1 KB on; K runs down the tokens), likewise.  `lead` and
// `stride` in bytes: to the next swizzle atom along the contiguous side, and to
// the next eight rows.
__device__ __forceinline__ uint64_t smem_desc_sw128(uint32_t addr, uint32_t lead, uint32_t stride) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((addr >> 4) & 0x3FFF);
    d |= static_cast<uint64_t>((lead >> 4) & 0x3FFF) << 16;
    d |= static_cast<uint64_t>((stride >> 4) & 0x3FFF) << 32;
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

// 16 lanes x 8 N columns of TMEM in the layout of matrix fragments: of each
// 8 columns, thread i gets columns 2 (i % 4), + 1 of lane i / 4 (r[0], r[1])
// and of lane i / 4 + 8 (r[2], r[3]).
__device__ __forceinline__ void tmem_ld_frag32(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void stmatrix_x4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

// Barrier of the softmax warps; returns whether any thread passed true.  A
// named barrier has no time limit, so every softmax warp reaches every one of
// them whether or not its waits succeeded (the counts depend on the run alone).
__device__ __forceinline__ bool soft_sync_or(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(v))
        : "memory");
    return r != 0;
}

// A worker's run of tiles, request by request: from tile t0 of request b up
// to (not including) tile t_end of request b_end.
struct Run {
    int b, t0, b_end, t_end;
    int32_t ahead;                    // seq_lens of request b: a trip to memory ahead of its use
    int len, tiles, n;                // of the current request: tokens, tiles, tiles of this run
    __device__ __forceinline__ bool next(const Params& p) {
        if (b > b_end || (b == b_end && t0 >= t_end)) return false;
        len = clamp_len(p, ahead);
        if (b + 1 < p.B) ahead = p.seq_lens[b + 1];
        tiles = tiles_of(len);
        n = (b == b_end ? t_end : tiles) - t0;
        return true;
    }
    __device__ __forceinline__ void advance() {
        ++b;
        t0 = 0;
    }
};

__global__ void __launch_bounds__(kThreads, 1)
latent_attention_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_pair,
                        const __grid_constant__ CUtensorMap map_odd, const Params p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int pairs = p.ck >> 1;
    const bool odd = p.ck & 1;
    const int q_bytes = p.ck * p.q_rows * 128;
    uint8_t* q_s = smem;                                   // [ck][q_rows][128 B]
    uint8_t* p_s = q_s + q_bytes;                          // [64 heads][128 B]
    uint8_t* pair_s = p_s + kChunkBytes;                   // [pair_slots][8 groups][2][8 tokens][128 B]
    uint8_t* odd_s = pair_s + p.pair_slots * kPairBytes;   // [odd_slots][8 groups][8 tokens][128 B]
    uint8_t* misc = odd_s + p.odd_slots * kChunkBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(misc);    // [kMaxPairs]
    uint64_t* empty = full + kMaxPairs;                    // [kMaxPairs]
    uint64_t* ofull = empty + kMaxPairs;                   // [kMaxOdd]
    uint64_t* oempty = ofull + kMaxOdd;                    // [kMaxOdd]
    uint64_t* qfull = oempty + kMaxOdd;
    uint64_t* qempty = qfull + 1;
    uint64_t* sfull = qempty + 1;                          // [2]
    uint64_t* sempty = sfull + 2;                          // [2]
    uint64_t* pfull = sempty + 2;
    uint64_t* pempty = pfull + 1;
    uint64_t* drain = pempty + 1;                          // [2] abort: products already issued
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    int* run_s = reinterpret_cast<int*>(tmem_holder + 2);  // [4] first request and tile, end request and tile
    int64_t* sums = reinterpret_cast<int64_t*>(tmem_holder + 6);   // [kThreads / 32]
    int* longest = reinterpret_cast<int*>(sums + kThreads / 32);   // [kThreads / 32 + 1]
    float* alpha_s = reinterpret_cast<float*>(longest + kThreads / 32 + 1);   // [64]
    float* inv_s = alpha_s + kHeads;                       // [64]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int w = blockIdx.x / p.G, g = blockIdx.x - w * p.G;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxPairs; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int s = 0; s < kMaxOdd; ++s) {
            mbar_init(smem_u32(&ofull[s]), 1);
            mbar_init(smem_u32(&oempty[s]), 1);
        }
        mbar_init(smem_u32(qfull), 1);
        mbar_init(smem_u32(qempty), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sfull[i]), 1);
            mbar_init(smem_u32(&sempty[i]), kSoftWarps);
        }
        mbar_init(smem_u32(pfull), kSoftWarps);
        mbar_init(smem_u32(pempty), 1);
        for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&drain[i]), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tma_prefetch_desc(&map_q);
        tma_prefetch_desc(&map_pair);
        if (odd) tma_prefetch_desc(&map_odd);
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

    // The worker's run.  Each request counts `lead` units, then one per tile;
    // worker w takes units [w U / workers, (w + 1) U / workers), and a cut
    // among a request's leading units is a cut before its first tile.  Thread
    // t sums requests [t * per, (t + 1) * per).  The leading units stand for
    // what a request costs beside its tiles (queries, pipeline fill, output:
    // ~3 us against ~1.5 us a tile); with less than that many tiles per worker
    // they would only leave workers idle.  Measured: 96 requests of mixed
    // lengths 105 us with 2 units, 107 with 3, 108 with 4, 160 with none; 200 up
    // to 1000 tokens, 16 heads, 23.0, 24.9 and 26.8; one request of 701 tokens
    // 14.2 us with 3, 12.8 with none.
    {
        const int per = (p.B + kThreads - 1) / kThreads;
        const int b0 = min(static_cast<int>(threadIdx.x) * per, p.B), b1 = min(b0 + per, p.B);
        int64_t mine = 0;
        int most = 0;
        for (int b = b0; b < b1; ++b) {
            const int t = tiles_of(request_len(p, b));
            mine += t;
            most = max(most, t);
        }
        most = __reduce_max_sync(0xffffffffu, most);
        int64_t inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += u;
        }
        if (lane == 31) {
            sums[warp] = inc;
            longest[warp] = most;
        }
        __syncthreads();
        int64_t before = inc - mine, tiles = 0;
        for (int i = 0; i < kThreads / 32; ++i) {
            if (i < warp) before += sums[i];
            tiles += sums[i];
            most = max(most, longest[i]);
        }
        // Requests a little longer than a worker's share go one to a worker,
        // uncut: cutting saves less than the parts and their join cost.  That
        // cost grows with the requests and heads that a join has to look at
        // (in tiles, one with an idle GPU, up to 10 with a fifth of it taken);
        // with less than kManyParts workers a request the join is the one of
        // few parts, at most 3 to 5 tiles.  Measured, cut against uncut, at
        // 128 heads (76 workers): one request of 2 tiles 12.3 and 12.5 us, of 3
        // 12.0 and 14.0, of 8 12.4 and 22.1; 4 of 3 15.2 and 14.8, of 5 15.6 and 18.0;
        // 16 of 10 30.9 and 29.3, of 16 32.8 and 39.4; 32 of 8 24.2 and 23.8, of 12
        // 26.2 and 30.8; 64 of 24 56.9 and 52.5.  At 16 heads (152): one of 2
        // 10.7 and 10.9, of 3 10.7 and 12.3; 64 of 4 15.7 and 14.8, of 7 17.8 and 19.6.  Over
        // 3660 mixes of 1 to 152 requests of 2 to 32 tiles the rule's choice
        // takes 1.2% more than the better one on average; a slack of 3 + h / 12,
        // whatever the number of requests, took 4%.
        const int h = min(p.H, kHeads), joined = 5 * p.B * h / (8 * p.W_full);
        const int slack = max(1, p.W < kManyParts * p.B ? min(joined, 3 + h / 32) : joined);
        const bool uncut = p.B <= p.W && most <= (tiles + p.W - 1) / p.W + slack;
        const int lead = tiles / p.W < kRequestUnits ? static_cast<int>(tiles / p.W) : kRequestUnits;
        const int64_t total = tiles + static_cast<int64_t>(lead) * p.B;
        before += static_cast<int64_t>(lead) * b0;
        mine += static_cast<int64_t>(lead) * (b1 - b0);
        const int64_t workers = total < p.W ? total : p.W;
        if (uncut && threadIdx.x < 2) {
            run_s[2 * threadIdx.x] = min(w + static_cast<int>(threadIdx.x), p.B);
            run_s[2 * threadIdx.x + 1] = 0;
        }
#pragma unroll
        for (int e = 0; e < 2 && !uncut; ++e) {
            const int64_t u = w + e < workers ? (w + e) * total / workers : total;
            if (threadIdx.x == 0 && u == total) {
                run_s[2 * e] = p.B;
                run_s[2 * e + 1] = 0;
            }
            if (u >= before && u < before + mine) {
                int64_t at = before;
                int b = b0, n = lead + tiles_of(request_len(p, b));
                while (at + n <= u) {
                    at += n;
                    n = lead + tiles_of(request_len(p, ++b));
                }
                run_s[2 * e] = b;
                run_s[2 * e + 1] = max(static_cast<int>(u - at) - lead, 0);
            }
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
    run.b_end = run_s[2];
    run.t_end = run_s[3];
    if (run.b < p.B) run.ahead = p.seq_lens[run.b];
    const int b_first = run.b;
    if (threadIdx.x == 0 && g == 0) p.meta[w] = make_int2(run.b, run.t0);

    // A whole warp's wait: all of its lanes go on or none (warp-wide
    // instructions follow), and the compiler sees that it is so.
    auto wait_uniform = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_bounded<true>(bar, parity, abort_flag, tmo));
    };
    // The same, asleep between polls: for the copying warp, which is ahead.
    auto wait_uniform_asleep = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_bounded(bar, parity, abort_flag, tmo));
    };

    if (warp == 0) {
        // ------------------------------------------------------- TMA producer
        // Tiles pass through L2 once (twice for two head groups), the parts are
        // to stay there for the join: with normal priority the parts of long
        // requests went to HBM (two of 131071 tokens wrote 5.2 MB there, now
        // 1.3).  Over eight caches in turn 128 x 8000 tokens take 191.3 us
        // against 196.7, two of 131071 59.3 against 62.0; over three caches in
        // turn, where a pass finds some of its rows still in L2, 189.4 and 59.1.
        uint64_t policy;
        asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
        const int pieces = kTile / p.box_rows;             // copies of a tile (1, 2, 4 or 8)
        const int batch = 32 / pieces;                     // tiles whose table entries the lanes hold
        uint32_t nq = 0;
        Place pp, po;
        bool ok = true, skip = (p.inject & kInjectSkipLoad) != 0;
        for (; ok && run.next(p); run.advance()) {
            if (run.len == 0) continue;
            const int32_t* row = p.table + run.b * p.ld_table;
            int ids = 0;
            ok = wait_uniform_asleep(smem_u32(qempty), (nq & 1) ^ 1);
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(smem_u32(qfull), q_bytes);
                tma_load_4d(smem_u32(q_s), &map_q, smem_u32(qfull), g * kHeads, run.b);
            }
            ++nq;
            for (int i = 0; ok && i < run.n; ++i) {
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
                const int tok0 = tile * kTile;
                const int live = min(pieces, (run.len - tok0 + p.box_rows - 1) / p.box_rows);
                const int id = __shfl_sync(0xffffffffu, ids, (i % batch) * pieces + (lane & (pieces - 1)));
                const int group = (tok0 + lane * p.box_rows) % p.page_size / 8;
                if (odd) {
                    ok = wait_uniform_asleep(smem_u32(&oempty[po.i]), po.pass ^ 1);
                    if (!ok) break;
                    const uint32_t fb = smem_u32(&ofull[po.i]);
                    if (lane == 0) mbar_arrive_expect_tx(fb, live * p.box_rows * 128);
                    __syncwarp();
                    if (lane < live)
                        tma_load_5d(smem_u32(odd_s) + po.i * kChunkBytes + lane * p.box_rows * 128, &map_odd, fb, p.ck - 1, group, id,
                                    policy);
                    po.step(p.odd_slots);
                }
                for (int j = 0; j < pairs; ++j) {
                    ok = wait_uniform_asleep(smem_u32(&empty[pp.i]), pp.pass ^ 1);
                    if (!ok) break;
                    const uint32_t fb = smem_u32(&full[pp.i]);
                    if (!skip) {                           // test hook: the first pair never comes, the waits on it run out
                        if (lane == 0) mbar_arrive_expect_tx(fb, live * p.box_rows * 256);
                        __syncwarp();
                        if (lane < live)
                            tma_load_5d(smem_u32(pair_s) + pp.i * kPairBytes + lane * p.box_rows * 256, &map_pair, fb, 2 * j, group,
                                        id, policy);
                    }
                    skip = false;
                    pp.step(p.pair_slots);
                }
            }
        }
        if (!ok) settle_ns(kAbortSettleNs);                // copies already issued land before the CTA goes
    } else if (warp == 1) {
        // ------------------------------------------------- products S = Q K^T
        // Chunk pair by chunk pair as they land.
        const uint32_t id_s = idesc_bf16(64, kTile, false);
        const uint64_t q_desc = smem_desc_sw128(smem_u32(q_s), 16, 1024);
        const uint32_t q_chunk = p.q_rows * 128 >> 4;      // descriptor step of a chunk of q
        Place po, pp;
        uint32_t n = 0, nq = 0;
        bool ok = true;
        for (; ok && run.next(p); run.advance()) {
            if (run.len == 0) continue;
            ok = wait_uniform(smem_u32(qfull), nq & 1);
            ++nq;
            for (int i = 0; ok && i < run.n; ++i, ++n) {
                ok = wait_uniform(smem_u32(&sempty[n & 1]), ((n >> 1) & 1) ^ 1);
                tc_fence_after();
                const uint32_t d = tmem + kTmemS + (n & 1) * kTile;
                if (odd && ok) {
                    ok = wait_uniform(smem_u32(&ofull[po.i]), po.pass);
                    if (!ok) break;
                    tc_mma4_bf16<2, 2>(d, q_desc + (p.ck - 1) * q_chunk, smem_desc_sw128(smem_u32(odd_s) + po.i * kChunkBytes, 16, 1024),
                                       id_s, 0);
                    tc_commit(smem_u32(&oempty[po.i]));
                    po.step(p.odd_slots);
                }
                for (int j = 0; ok && j < pairs; ++j) {
                    ok = wait_uniform(smem_u32(&full[pp.i]), pp.pass);
                    if (!ok) break;
                    const uint64_t kd = smem_desc_sw128(smem_u32(pair_s) + pp.i * kPairBytes, 16, 2048);
                    const uint64_t qd = q_desc + 2 * j * q_chunk;
                    tc_mma4_bf16<2, 2>(d, qd, kd, id_s, odd || j > 0);
                    tc_mma4_bf16<2, 2>(d, qd + q_chunk, kd + 64, id_s, 1);
                    if (j >= p.nblk) tc_commit(smem_u32(&empty[pp.i]));   // no part of the value
                    pp.step(p.pair_slots);
                }
                if (!ok) break;
                tc_commit(smem_u32(&sfull[n & 1]));
                if (i == run.n - 1) tc_commit(smem_u32(qempty));
            }
        }
        if (!ok) {                                         // products already issued end before their memory goes
            tc_commit(smem_u32(&drain[0]));
            wait_drain(smem_u32(&drain[0]), 0, tmo);
        }
    } else if (warp == 6) {
        // ------------------------------------------- products O^T += V^T P^T
        // They free the chunk pairs one by one.
        const int heads = min(kHeads, p.H - g * kHeads);
        const uint32_t id_o = idesc_bf16(128, (heads + 15) & ~15, true);
        const uint64_t p_desc = smem_desc_sw128(smem_u32(p_s), 16, 1024);
        Place pv;
        uint32_t n = 0;
        bool ok = true;
        for (; ok && run.next(p); run.advance()) {
            if (run.len == 0) continue;
            for (int i = 0; i < run.n; ++i, ++n) {
                ok = wait_uniform(smem_u32(pfull), n & 1);
                if (!ok) break;
                tc_fence_after();
                for (int blk = 0; blk < p.nblk; ++blk) {
                    tc_mma4_bf16<4096 / 16, 2>(tmem + blk * kHeads,
                                               smem_desc_sw128(smem_u32(pair_s) + pv.i * kPairBytes, 1024, 2048), p_desc, id_o, i > 0);
                    tc_commit(smem_u32(&empty[pv.i]));
                    pv.step(p.pair_slots);
                }
                tc_commit(smem_u32(pempty));
                for (int j = p.nblk; j < pairs; ++j) pv.step(p.pair_slots);
            }
        }
        if (!ok) {
            tc_commit(smem_u32(&drain[1]));
            wait_drain(smem_u32(&drain[1]), 0, tmo);
        }
    } else {
        // ------------------------------------- softmax, rescaling and output
        const int quad = warp & 3;                         // TMEM lanes 32 * quad ..
        const uint32_t tl = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        const int st = threadIdx.x - 64;                   // 0..127
        const float kNegInf = __int_as_float(0xff800000);
        // S at M = 64: row 16 * quad + i is lane 32 * quad + i, i < 16.  In
        // the fragment layout a thread holds 16 columns of two rows.
        const int row0 = quad * 16 + (lane >> 2), col0 = 2 * (lane & 3);   // the other row: row0 + 8
        // Where this lane's stmatrix row goes: matrices (rows 0-7, 8-15) x two
        // adjacent 8-column groups of the warp's 16 rows of P.
        const int p_row = quad * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
        const uint32_t p_addr = smem_u32(p_s) + p_row * 128;
        const int p_grp = lane >> 4, p_swz = lane & 7;
        const int DV = p.nblk * 128, heads = min(kHeads, p.H - g * kHeads);
        const bool mine = quad * 16 < heads;               // this warp's rows of S hold heads
        int zslot = 0;                                     // slot of tile n's first pair
        uint32_t n = 0;
        bool ok = true;                                    // false: only the barriers are kept up
        for (; run.next(p); run.advance()) {
            const int b = run.b;
            const bool whole = run.t0 == 0 && run.n == run.tiles;
            if (run.len == 0) {
                // An empty request: zeros, and the logarithm of an empty sum.
                for (int e = st; e < kHeads * (DV / 8); e += 128) {
                    const int h = g * kHeads + e / (DV / 8), c = e % (DV / 8);
                    if (h < p.H && bounds_ok(b < p.B))
                        *reinterpret_cast<uint4*>(p.out + b * p.ldo_b + h * p.ldo_h + c * 8) = make_uint4(0, 0, 0, 0);
                }
                if (p.lse && st < kHeads && g * kHeads + st < p.H) p.lse[b * p.ldl_b + g * kHeads + st] = kNegInf;
                continue;
            }
            // Of the two rows: maximum of the raw scores in use, and this
            // thread's share of the sums of p, unrounded and rounded.
            float m[2] = {kNegInf, kNegInf}, l[2] = {0.f, 0.f}, lr[2] = {0.f, 0.f};
            for (int i = 0; i < run.n; ++i, ++n) {
                const int valid = min(kTile, run.len - (run.t0 + i) * kTile);
                ok = ok && wait_uniform(smem_u32(&sfull[n & 1]), (n >> 1) & 1);
                tc_fence_after();
                float s[2][16];                            // [row][8 k + column]
                {
                    uint32_t r[2][16];
                    tmem_ld_frag32(tl + kTmemS + (n & 1) * kTile, r[0]);
                    tmem_ld_frag32(tl + kTmemS + (n & 1) * kTile + 32, r[1]);
                    tmem_ld16_wait(r[0]);
                    tmem_ld16_wait(r[1]);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {         // 8 column groups x 2 columns
                        s[0][j] = __uint_as_float(r[j >> 3][(j >> 1 & 3) * 4 + (j & 1)]);
                        s[1][j] = __uint_as_float(r[j >> 3][(j >> 1 & 3) * 4 + 2 + (j & 1)]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sempty[n & 1]));
                if (valid < kTile) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if ((j >> 1) * 8 + col0 + (j & 1) >= valid) s[0][j] = s[1][j] = kNegInf;
                }
                // Whether product n - 1 is done (then P's buffer and O are this
                // tile's) is looked at early: the test takes long, and mostly it is.
                bool pv_done = n == 0 || __all_sync(0xffffffffu, mbar_test(smem_u32(pempty), (n & 1) ^ 1));
                bool raise = false;
                float top[2];
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    float x[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = fmaxf(s[a][j], s[a][j + 8]);
                    top[a] = fmaxf(fmaxf(fmaxf(x[0], x[4]), fmaxf(x[1], x[5])), fmaxf(fmaxf(x[2], x[6]), fmaxf(x[3], x[7])));
                    top[a] = fmaxf(top[a], __shfl_xor_sync(0xffffffffu, top[a], 1));
                    top[a] = fmaxf(top[a], __shfl_xor_sync(0xffffffffu, top[a], 2));
                    raise |= row0 + 8 * a < heads && (top[a] - m[a]) * p.scale_log2 > kRaise;
                }
                if (i == 0) {
                    m[0] = top[0];
                    m[1] = top[1];
                    raise = false;
                }
                if (soft_sync_or(raise)) {
                    // Rare: some maximum grew too far; O and the sums follow.
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
                        float alpha = 1.f;
                        if (row0 + 8 * a < heads && (top[a] - m[a]) * p.scale_log2 > kRaise) {
                            alpha = exp2_fast((m[a] - top[a]) * p.scale_log2);
                            m[a] = top[a];
                            l[a] *= alpha;
                            lr[a] *= alpha;
                        }
                        if ((lane & 3) == 0) alpha_s[row0 + 8 * a] = alpha;
                    }
                    soft_sync_or(false);
                    if (!pv_done) ok = ok && wait_uniform(smem_u32(pempty), (n & 1) ^ 1);
                    pv_done = true;
                    tc_fence_after();
                    for (int c = 0; ok && c < p.nblk * kHeads; c += 16) {
                        uint32_t r[16];
                        tmem_ld16_issue(tl + c, r);
                        tmem_ld16_wait(r);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            r[j] = __float_as_uint(__uint_as_float(r[j]) * alpha_s[(c & (kHeads - 1)) + j]);
                        tmem_st16(tl + c, r);
                    }
                    tmem_wait_st();
                }
                uint32_t pk[2][8];
                if (mine) {
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
                        const float off = m[a] == kNegInf ? 0.f : m[a] * p.scale_log2;
                        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float e0 = exp2_fast(fmaf(s[a][2 * j], p.scale_log2, -off));
                            const float e1 = exp2_fast(fmaf(s[a][2 * j + 1], p.scale_log2, -off));
                            sum[j & 1] = add2(sum[j & 1], make_float2(e0, e1));
                            pk[a][j] = pack_bf16(e0, e1);
                        }
                        l[a] += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
                    }
                }
                if (!pv_done) ok = ok && wait_uniform(smem_u32(pempty), (n & 1) ^ 1);
                __syncwarp();
                if (ok) {
                    if (mine) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            stmatrix_x4(p_addr + (((2 * j + p_grp) ^ p_swz) << 4), pk[0][2 * j], pk[1][2 * j], pk[0][2 * j + 1],
                                        pk[1][2 * j + 1]);
                    }
                    if (valid < kTile) {
                        // Rows past the length hold whatever the page or the
                        // buffer held: 0 * NaN would reach O, so they become 0.
                        // (S of this tile is done, so its pairs have landed.)
                        for (int r = valid + (st >> 4); r < kTile; r += 8) {
                            int slot = zslot;
                            uint8_t* at = pair_s + (r >> 3) * 2048 + ((st >> 3) & 1) * 1024 + (r & 7) * 128 + (st & 7) * 16;
                            for (int j = 0; j < p.nblk; ++j) {
                                *reinterpret_cast<uint4*>(at + slot * kPairBytes) = make_uint4(0, 0, 0, 0);
                                if (++slot == p.pair_slots) slot = 0;
                            }
                        }
                    }
                }
                zslot += pairs;
                while (zslot >= p.pair_slots) zslot -= p.pair_slots;
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(pfull));
                if (mine) {
                    // The rounded sum, while the product runs.
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
                        float2 sum[2] = {make_float2(lr[a], 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            sum[j & 1] = add2(sum[j & 1], make_float2(__uint_as_float(pk[a][j] << 16),
                                                                      __uint_as_float(pk[a][j] & 0xffff0000u)));
                        lr[a] = (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
                    }
                }
            }
            // ---- output of the request (or of this worker's part of it)
            ok = ok && wait_uniform(smem_u32(pempty), (n & 1) ^ 1);
            tc_fence_after();
            const int64_t slot = (static_cast<int64_t>(w) * 2 + (b == b_first ? 0 : 1)) * p.G + g;
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                l[a] += __shfl_xor_sync(0xffffffffu, l[a], 1);
                lr[a] += __shfl_xor_sync(0xffffffffu, lr[a], 1);
                l[a] += __shfl_xor_sync(0xffffffffu, l[a], 2);
                lr[a] += __shfl_xor_sync(0xffffffffu, lr[a], 2);
                // A part's weights add up to its unrounded sum, which the join divides by.
                if ((lane & 3) == 0)
                    inv_s[row0 + 8 * a] = lr[a] > 0.f || lr[a] != lr[a] ? __fdividef(whole ? 1.0f : l[a], lr[a]) : 0.f;
            }
            soft_sync_or(false);                           // inv_s is next written after another tile's barrier
            __syncwarp();
            if (!ok) continue;
            if (whole) {
                // 32 values x 32 heads at a time, through the warp's own 2 KB
                // of P's buffer: stmatrix turns the fragments into rows of 32
                // values (16-byte chunks, chunk ^ (row / 2) % 4), which leave
                // as 16-byte stores, 64 bytes of each of eight heads at once.
                const uint32_t stage = smem_u32(p_s) + quad * 2048;
                const int halves = heads > 32 ? 2 : 1, its = p.nblk * halves;
                uint32_t r[2][2][16];
                auto fetch = [&](int it, uint32_t (&x)[2][16]) {
                    const uint32_t src = tl + (it / halves) * kHeads + (it % halves) * 32;
                    tmem_ld_frag32(src, x[0]);
                    tmem_ld_frag32(src + (16u << 16), x[1]);
                };
                auto put = [&](int it, const uint32_t (&x)[2][16]) {
                    const int blk = it / halves, h0 = (it % halves) * 32;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {          // eight heads
                        const float2 f = *reinterpret_cast<const float2*>(inv_s + h0 + q * 8 + col0);
                        uint32_t v[4];
#pragma unroll
                        for (int d = 0; d < 4; ++d)        // eight values
                            v[d] = pack_bf16(__uint_as_float(x[d >> 1][q * 4 + (d & 1) * 2]) * f.x,
                                             __uint_as_float(x[d >> 1][q * 4 + (d & 1) * 2 + 1]) * f.y);
                        const int hl = q * 8 + (lane & 7), d = lane >> 3;
                        stmatrix_x4_trans(stage + hl * 64 + ((d ^ ((hl >> 1) & 3)) << 4), v[0], v[1], v[2], v[3]);
                    }
                    __syncwarp();
                    __nv_bfloat16* o = p.out + b * p.ldo_b + blk * 128 + quad * 32 + (lane & 3) * 8;
                    uint4 v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int hl = j * 8 + (lane >> 2);
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(v[j].x), "=r"(v[j].y), "=r"(v[j].z), "=r"(v[j].w)
                                     : "r"(stage + hl * 64 + (((lane & 3) ^ ((hl >> 1) & 3)) << 4))
                                     : "memory");
                    }
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int head = h0 + j * 8 + (lane >> 2);
                        if (head < heads && bounds_ok(b < p.B))
                            *reinterpret_cast<uint4*>(o + static_cast<int64_t>(g * kHeads + head) * p.ldo_h) = v[j];
                    }
                };
                // The next fragments come from TMEM while these leave.
                fetch(0, r[0]);
                for (int it = 0; it < its; it += 2) {
                    tmem_ld16_wait(r[0][0]);
                    tmem_ld16_wait(r[0][1]);
                    if (it + 1 < its) fetch(it + 1, r[1]);
                    put(it, r[0]);
                    if (it + 1 >= its) break;
                    tmem_ld16_wait(r[1][0]);
                    tmem_ld16_wait(r[1][1]);
                    if (it + 2 < its) fetch(it + 2, r[0]);
                    put(it + 1, r[1]);
                }
            } else {
                // A part, in the order the registers hold it: 512 bytes a store,
                // 16 heads at a time with their factors in registers (read from
                // shared memory between the stores they cost 1.5 us a part).
                float4* o = reinterpret_cast<float4*>(p.part_o) + slot * p.nblk * 16 * 128 + quad * 32 + lane;
                for (int hg = 0; hg < heads; hg += 16) {
                    float4 f[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) f[j] = reinterpret_cast<const float4*>(inv_s + hg)[j];
                    uint32_t r[2][16];
                    auto fetch = [&](int blk, uint32_t (&x)[16]) { tmem_ld16_issue(tl + blk * kHeads + hg, x); };
                    auto put = [&](int blk, const uint32_t (&x)[16]) {
                        const int c = blk * 16 + hg / 4;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (bounds_ok(w < p.W && c + j < p.nblk * 16))
                                o[(c + j) * 128] =
                                    make_float4(__uint_as_float(x[4 * j]) * f[j].x, __uint_as_float(x[4 * j + 1]) * f[j].y,
                                                __uint_as_float(x[4 * j + 2]) * f[j].z, __uint_as_float(x[4 * j + 3]) * f[j].w);
                    };
                    fetch(0, r[0]);
                    for (int blk = 0; blk < p.nblk; blk += 2) {
                        tmem_ld16_wait(r[0]);
                        if (blk + 1 < p.nblk) fetch(blk + 1, r[1]);
                        put(blk, r[0]);
                        if (blk + 1 >= p.nblk) break;
                        tmem_ld16_wait(r[1]);
                        if (blk + 2 < p.nblk) fetch(blk + 2, r[0]);
                        put(blk + 1, r[1]);
                    }
                }
            }
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                const int row = row0 + 8 * a, head = g * kHeads + row;
                const float m2 = m[a] == kNegInf ? m[a] : m[a] * p.scale_log2;
                if ((lane & 3) != 0) continue;
                if (!whole) p.part_ml[slot * kHeads + row] = make_float2(m2, l[a]);
                else if (p.lse && head < p.H) p.lse[b * p.ldl_b + head] = l[a] == 0.f ? kNegInf : (m2 + log2f(l[a])) * kLn2;
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
// found at the first cut inside it; its parts are those of the worker before
// that cut and of the workers that begin inside it, in the order of the tokens.
//   out = sum_k 2^(m_k - M) o_k / sum_k 2^(m_k - M) l_k,  M = max_k m_k
// A part's value is read as it lies: 16 bytes are four heads of one value.  An
// item is four heads of one block of 128 values: SHARE = 1 gives it to one
// warp, for the few parts of a request in a large batch; SHARE = 8 gives it to
// the eight warps of a CTA, which take the parts in turn, for long requests
// that many workers share.  A warp has AHEAD parts on their way: the kernel
// takes as long as its trips to memory.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;

template <int SHARE, int AHEAD, int CTAS>
__global__ void __launch_bounds__(kJoinThreads, CTAS)
latent_attention_join_kernel(const Params p, const int by_cut) {
    grid_dependency_wait();
    allow_dependent_launch();
    bounds_self_test(p.inject);
    constexpr unsigned kAll = 0xffffffffu;
    __shared__ int first_s, parts_s, request_s[kJoinThreads];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = threadIdx.x;
    const float kNegInf = __int_as_float(0xff800000);
    const int quads = (p.H + 3) / 4, items = quads * p.nblk;
    const int per = (items + 8 / SHARE - 1) / (8 / SHARE); // CTAs of a request
    const int what = blockIdx.x / per;

    // The request: `what` itself, or the one whose first cut is the cut before
    // worker what + 1.  A cut before worker k lies inside request b when
    // meta[k] = (b, > 0); the cuts of a request are neighbours.
    static_assert(kMaxCtas <= kJoinThreads, "one thread per worker");
    const int2 me = t < p.W ? p.meta[t] : make_int2(-1, 0);
    request_s[t] = me.x;
    if (t == 0) {
        first_s = p.W;
        parts_s = 0;
    }
    __syncthreads();
    const int b = by_cut ? request_s[what + 1] : what;
    const bool cut = me.x == b && me.y > 0 && b < p.B;
    const unsigned votes = __ballot_sync(kAll, cut);
    if (lane == 0 && votes) {
        atomicMin(&first_s, warp * 32 + __ffs(votes) - 1);
        atomicAdd(&parts_s, __popc(votes));
    }
    __syncthreads();
    const int w = first_s, np = parts_s + 1;               // first cut inside the request, its parts
    if (np < 2 || (by_cut && w != what + 1)) return;
    const int sub = static_cast<int>(blockIdx.x) - what * per;
    const int item = SHARE == 1 ? sub * 8 + warp : sub;
    if (item >= items) return;                             // SHARE = 8: the whole CTA
    const int hq = item / p.nblk, blk = item - hq * p.nblk;
    const int g = hq * 4 / kHeads, hl = hq * 4 - g * kHeads;
    const int left_slot = request_s[w - 1] == b ? 0 : 1;
    auto slot_of = [&](int k) -> int64_t {                 // part k's place in the workspace
        return static_cast<int64_t>(k == 0 ? (w - 1) * 2 + left_slot : (w + k - 1) * 2) * p.G + g;
    };
    // Values 2 lane, + 1, 2 lane + 64, + 1 of the block.
    auto load = [&](int k, float4 (&o)[4]) {
        const float4* src = reinterpret_cast<const float4*>(p.part_o) + ((slot_of(k) * p.nblk + blk) * 16 + hl / 4) * 128 + 2 * lane;
        o[0] = src[0];
        o[1] = src[1];
        o[2] = src[64];
        o[3] = src[65];
    };
    const int k0 = SHARE == 1 ? 0 : warp, mine = np > k0 ? (np - k0 + SHARE - 1) / SHARE : 0;   // parts of this warp
    float M[4], L[4] = {0.f, 0.f, 0.f, 0.f}, acc[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        M[j] = kNegInf;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i][j] = 0.f;
    }
    for (int c = 0; c < mine; c += 32) {                   // 32 parts at a time, one's (max, sum) per lane
        const int cnt = min(32, mine - c);
        float4 o[AHEAD][4];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)                   // on their way while the factors are formed
            if (u < cnt) load(k0 + (c + u) * SHARE, o[u]);
        float f[4] = {kNegInf, kNegInf, kNegInf, kNegInf}, l[4] = {0.f, 0.f, 0.f, 0.f};
        if (lane < cnt) {
            const float4* ml = reinterpret_cast<const float4*>(p.part_ml + slot_of(k0 + (c + lane) * SHARE) * kHeads + hl);
            const float4 x = ml[0], y = ml[1];
            f[0] = x.x; f[1] = x.z; f[2] = y.x; f[3] = y.z;
            l[0] = x.y; l[1] = x.w; l[2] = y.y; l[3] = y.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float top = f[j];
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, s));
            top = fmaxf(top, M[j]);
            const float base = top == kNegInf ? 0.f : top, old = exp2_fast(M[j] - base);
            f[j] = exp2_fast(f[j] - base);
            L[j] = fmaf(L[j], old, warp_sum(f[j] * l[j]));
            M[j] = top;
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i][j] *= old;
        }
        auto add = [&](int k, const float4 (&x)[4]) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float fk = __shfl_sync(kAll, f[j], k);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float v = j == 0 ? x[i].x : j == 1 ? x[i].y : j == 2 ? x[i].z : x[i].w;
                    acc[i][j] = fmaf(v, fk, acc[i][j]);
                }
            }
        };
        for (int k = 0; k < cnt; k += AHEAD) {
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
                if (k + u < cnt) add(k + u, o[u]);
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
                if (k + AHEAD + u < cnt) load(k0 + (c + k + AHEAD + u) * SHARE, o[u]);
        }
    }
    if (SHARE > 1) {
        // The warps' results, merged by warp 0 in the order of the warps.
        __shared__ float4 red[8][4][32], red_m[8], red_l[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) red[warp][i][lane] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        if (lane == 0) {
            red_m[warp] = make_float4(M[0], M[1], M[2], M[3]);
            red_l[warp] = make_float4(L[0], L[1], L[2], L[3]);
        }
        __syncthreads();
        if (warp >= 4) return;
        // Warp i finishes value group i: its quarter of the item's values.
        float top[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            const float4 m = red_m[s];
            top[0] = fmaxf(top[0], m.x); top[1] = fmaxf(top[1], m.y);
            top[2] = fmaxf(top[2], m.z); top[3] = fmaxf(top[3], m.w);
        }
        float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j) L[j] = 0.f;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            const float4 m = red_m[s], q = red_l[s], x = red[s][warp][lane];
            const float sm[4] = {m.x, m.y, m.z, m.w}, sl[4] = {q.x, q.y, q.z, q.w}, sx[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float fk = exp2_fast(sm[j] - (top[j] == kNegInf ? 0.f : top[j]));
                L[j] = fmaf(sl[j], fk, L[j]);
                a[j] = fmaf(sx[j], fk, a[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            M[j] = top[j];
            const int h = hq * 4 + j, v = blk * 128 + (warp >> 1) * 64 + 2 * lane + (warp & 1);
            const float inv = L[j] > 0.f || L[j] != L[j] ? 1.0f / L[j] : 0.f;
            if (h < p.H && bounds_ok(b < p.B && v < p.nblk * 128))
                p.out[b * p.ldo_b + h * p.ldo_h + v] = __float2bfloat16_rn(a[j] * inv);
        }
        if (warp != 0) return;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int h = hq * 4 + j;
            const float inv = L[j] > 0.f || L[j] != L[j] ? 1.0f / L[j] : 0.f;
            if (h >= p.H || !bounds_ok(b < p.B)) continue;
            __nv_bfloat16* dst = p.out + b * p.ldo_b + h * p.ldo_h + blk * 128 + 2 * lane;
            *reinterpret_cast<uint32_t*>(dst) = pack_bf16(acc[0][j] * inv, acc[1][j] * inv);
            *reinterpret_cast<uint32_t*>(dst + 64) = pack_bf16(acc[2][j] * inv, acc[3][j] * inv);
        }
    }
    if (p.lse && blk == 0 && lane < 4 && hq * 4 + lane < p.H) {
        const float m = lane == 0 ? M[0] : lane == 1 ? M[1] : lane == 2 ? M[2] : M[3];
        const float l = lane == 0 ? L[0] : lane == 1 ? L[1] : lane == 2 ? L[2] : L[3];
        p.lse[b * p.ldl_b + hq * 4 + lane] = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
    }
}

// --------------------------------------------------------------------- host

bool encode_map(CUtensorMap* m, int rank, const void* base, const cuuint64_t* dims, const cuuint64_t* strides,
                const cuuint32_t* box) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// q as [request][chunk][head][64 columns]: one copy brings all chunks of 64
// heads (zeros past the last head).
bool make_q_map(CUtensorMap* m, const void* q, int64_t B, int64_t H, int64_t ck, int64_t ld_tok, int64_t ld_head, int rows) {
    const cuuint64_t dims[4] = {kChunkCols, static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(ck), static_cast<cuuint64_t>(B)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(ld_head * 2), kChunkCols * 2, static_cast<cuuint64_t>(ld_tok * 2)};
    const cuuint32_t box[4] = {kChunkCols, static_cast<cuuint32_t>(rows), static_cast<cuuint32_t>(ck), 1};
    return encode_map(m, 4, q, dims, strides, box);
}

// The cache as [page][group of 8 tokens][chunk][token][64 columns]: one copy
// brings `chunks` chunks of `rows` tokens (whole groups) of one page.
bool make_cache_map(CUtensorMap* m, const void* cache, int64_t pages, int64_t page_size, int64_t ck, int64_t ld_page,
                    int64_t ld_row, int rows, int chunks) {
    const cuuint64_t dims[5] = {kChunkCols, 8, static_cast<cuuint64_t>(ck), static_cast<cuuint64_t>(page_size / 8),
                                static_cast<cuuint64_t>(pages)};
    const cuuint64_t strides[4] = {static_cast<cuuint64_t>(ld_row * 2), kChunkCols * 2, static_cast<cuuint64_t>(ld_row * 16),
                                   static_cast<cuuint64_t>(ld_page * 2)};
    const cuuint32_t box[5] = {kChunkCols, 8, static_cast<cuuint32_t>(chunks), static_cast<cuuint32_t>(rows / 8), 1};
    return encode_map(m, 5, cache, dims, strides, box);
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
    L.ml = (W * 8 + 255) / 256 * 256;
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
    // Strides of a tensor map are below 2^40 bytes (the cache's 8-row groups: 16 ld_row).
    if (num_pages > 0x7ffffffeLL || ld_row >= (1LL << 36) || ld_page >= (1LL << 39) || ldq_tok >= (1LL << 39) ||
        ldq_head >= (1LL << 39))
        return DSNQ_ERR_UNSUPPORTED;
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
    const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
    p.W = static_cast<int>(workers_for(B, G, cap, ctas));
    p.W_full = ctas > G ? static_cast<int>(ctas / G) : 1;
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
    p.q_rows = static_cast<int>(H < kHeads ? (H + 7) / 8 * 8 : kHeads);
    // Shared memory: q, P, barriers, and the rest for the rings.  The MMA reads
    // 64 rows of q whatever H is: past the last chunk's rows it reads P's buffer
    // (rows of S that no head owns).
    const int64_t fixed = 1024 + static_cast<int64_t>(p.ck) * p.q_rows * 128 + kChunkBytes + kMiscBytes;
    int64_t room = 227 * 1024 - fixed;
    p.odd_slots = p.ck & 1 ? 2 : 0;
    p.pair_slots = static_cast<int>((room - p.odd_slots * kChunkBytes) / kPairBytes);
    if (p.pair_slots > kMaxPairs) p.pair_slots = kMaxPairs;
    if (p.odd_slots && room - p.pair_slots * kPairBytes >= kMaxOdd * kChunkBytes) p.odd_slots = kMaxOdd;
    const size_t smem = static_cast<size_t>(fixed + p.pair_slots * kPairBytes + p.odd_slots * kChunkBytes);
    p.scale_log2 = scale * kLog2e;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.ldo_b = ldo_tok; p.ldo_h = ldo_head;
    p.lse = lse; p.ldl_b = ldl_tok;
    const Layout lay = workspace_layout(p.W, G, DV);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.meta = reinterpret_cast<int2*>(ws + lay.meta);
    p.part_ml = reinterpret_cast<float2*>(ws + lay.ml);
    p.part_o = reinterpret_cast<float*>(ws + lay.o);
    const uint64_t t = debug_wait_timeout_ns();
    p.timeout_ns = t ? t : kDefaultTimeoutNs;
    p.inject = debug_inject_flags();

    CUtensorMap mq, mk, mo;
    // A lone token or head has no stride of its own: any valid one will do.
    const int64_t qh = H > 1 ? ldq_head : DK, qt = B > 1 ? ldq_tok : H * qh;
    if (!make_q_map(&mq, q, B, H, p.ck, qt, qh, p.q_rows) ||
        !make_cache_map(&mk, cache, num_pages, page_size, p.ck, ld_page, ld_row, p.box_rows, 2) ||
        !make_cache_map(&mo, cache, num_pages, page_size, p.ck, ld_page, ld_row, p.box_rows, 1))
        return DSNQ_ERR_CUDA;
    if (!set_smem_attr(reinterpret_cast<const void*>(latent_attention_kernel), smem)) return DSNQ_ERR_CUDA;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    st = launch_result(launch_kernel(latent_attention_kernel, dim3(static_cast<unsigned>(p.W * G)), dim3(kThreads), smem, s,
                                     mq, mk, mo, p));
    if (st != DSNQ_OK || p.W == 1) return st;
    // Few requests: a request has many parts, so a CTA joins each item.  Many:
    // a warp does, and no more requests can be split than there are cuts.
    // While all CTAs find room at once, each keeps more parts on their way
    // (registers, so fewer CTAs on an SM).  Measured, 2 parts ahead against 4:
    // 20 requests up to 8000 tokens, 128 heads (320 CTAs) 26.8 against 23.9 us,
    // 40 up to 4096 (640 CTAs) 31.5 against 33.4, 256 of 500, 16 heads (two
    // parts a request) 42.8 against 44.6; against 5, one request of 9000, 128
    // heads (128 CTAs) 19.4 against 18.0, eight up to 16000 (1024) 22.2 against 27.2.
    // With more CTAs than find room, three on an SM instead of two: 256 of 500,
    // 128 heads (1200 CTAs) 77.9 against 76.9 us, 40 up to 4096 (640) 30.3 against 30.9.
    const int64_t items = (H + 3) / 4 * p.nblk;
    const int by_cut = B > p.W - 1;
    const int64_t targets = by_cut ? p.W - 1 : B;
    const bool share = p.W >= kManyParts * B;
    const int64_t grid = targets * (share ? items : (items + 7) / 8);
    void (*join)(Params, int);
    if (share) join = p.W > 16 * B && grid <= sms ? latent_attention_join_kernel<8, 5, 1> : latent_attention_join_kernel<8, 2, 2>;
    else if (!by_cut && grid <= 3 * sms) join = latent_attention_join_kernel<1, 4, 1>;
    else join = grid <= 5 * sms ? latent_attention_join_kernel<1, 2, 2> : latent_attention_join_kernel<1, 2, 3>;
    return launch_result(launch_kernel(join, dim3(static_cast<unsigned>(grid)), dim3(kJoinThreads), 0, s, p, by_cut));
}

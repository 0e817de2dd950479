// Attention of one new token per request over a paged latent cache held in 8
// bits, and the same for a batch whose requests begin with the same tokens.
//
//   row j of the cache: s_j (codes_j | pe_j), codes e4m3, pe bf16, s_j fp32
//   out[b, h, :] = sum_j p_j s_j codes_j[0:DV],  p = softmax_j(scale * s_j q[b, h] . (codes_j | pe_j))
//
// The codes go to the tensor cores as they are; nothing is widened to 16 bits,
// neither in memory nor in shared memory, so a row costs its 8-bit bytes on the
// way in and in every read of it by a product.  What multiplies them is split
// instead, into two e4m3 numbers, x = hi + lo / 32, hi = e4m3(x), lo =
// e4m3(32 (x - hi)): eight significant bits, as many as bf16 has.
//   q: divided by a power of two per head (exact) so that its latent columns are
//      in [128, 256) at most; hi and lo then hold a bf16 exactly down to 2^-7 (hi's
//      last bit is 2^-9 there, lo's 2^-14), that is to 2^-14 of the head's largest;
//      what is smaller is off by at most 2^-15, 2^-22 of the largest.  hi and lo
//      are stacked along N, so a product reads a tile of the cache once.
//   p s: x = p_j s_j 2^-T with T a power of two per head and block of 32 tokens
//      such that the block's largest x lies in [128, 256]; the products put 2^T
//      back (block scales along K).  Rounded by at most 2^-8 of x (2^-4 of hi's
//      remainder, which is at most 2^-4 of x) or 2^-15 (half of lo's last bit),
//      at most 2^-22 of the block's largest.
// The position columns are a bf16 product into the same accumulators.  Scores,
// softmax statistics and outputs are fp32.  The outputs are divided by the sum
// of the p that the rounded x stand for, so that the weights add up to one
// (those of tokens whose scale is below 2^-8 of their block's largest count
// unrounded: they may have a large p and no value to speak of).
// The sums take p as x 2^T / s.  x below 2^-126 is lost and a block's 2^T is at
// least 2^-126 of the largest: with scales within a factor of 2^80 a token's p is
// then off by at most 2^-45 of the sum.
//
// One CTA, 64 heads (or 32 or 16 where CTAs would idle), tiles of 128 tokens:
//   S^T [128 tokens x (64 hi | 64 lo)]  = C Q^T        M = 128: a thread has a token
//   O^T [DV x 64 heads]                += C^T (p s)^T   M = 128, block-scaled; C^T is the
//                                                       same tile read column-major
// TMEM: O^T takes DV/128 x 64 columns, S^T 128, the block scales 8.  Measured
// alone on an SM, one product of S^T takes 69 cycles at 64 heads (52 at 16) and
// one of O^T 52 (45): 2900 cycles a tile at 64 heads and 576 columns, where the
// copy of a tile takes 3600 at this GPU's share of HBM per SM.
//
// Work split: jobs (a request, or as many rows of the whole batch against the
// common prefix as a CTA has heads) are laid end to end as tiles and cut into
// equal runs, one per worker (a CTA for each group of heads), on the device, from
// the lengths (prepare_kernel).  A run that
// covers a whole request writes its output; otherwise, and for all jobs of a
// batch with a common prefix, (max, sum, output times that sum) go to the
// workspace in fp32, and a second kernel joins them in the order of the tokens
// (no atomics: results do not depend on timing).
// The prefix: its rows are the (request, head) pairs of the batch laid end to
// end, so every tile of the prefix serves 64 rows whatever the number of heads.
//
// Measured (152 CTAs, requests of 2048 and 8192 tokens, per tile): 1.88 us at 16
// heads of 576 columns, where HBM needs 1.88; 2.17 at 48 of 512 (HBM 1.50), where the
// softmax warps bound it, two on each quarter of the SM, whose reads of shared
// memory and TMEM wait behind the products'; 2.71 at 64 of 576, where shared memory
// holds two tiles: the way from O^T of a tile over its freed slots, the copies
// into them, S^T and the softmax to the O^T two tiles on takes as long.
//
// Warps: 0 and 3 copy tiles (TMA), 1 issues S^T, 2 issues O^T, 4..11 do the softmax:
// warp w has tokens 32 (w % 4) .. of a tile (the TMEM lanes it can reach, and one
// block of 32 of the scales) and one half of the heads; they also write the
// output.  q is split beforehand, by a kernel of its own, and comes as one copy a
// job.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "debug_check.cuh"
#include "group_quant.cuh"
#include "dsnq_internal.h"
#include "latent_tiles.cuh"
#include "tensor_host.h"
#include "tensor_ptx.cuh"

namespace dsnq {
namespace attn8 {

using namespace attn;

constexpr int kHeads = 64;                  // rows (heads) of a CTA, at most
constexpr int kTile = 128;                  // tokens of a tile
constexpr int kChunkBytes = kTile * 128;    // 128 bytes of each row of a tile
constexpr int kPer = 32;                    // heads of a softmax warp, at most
constexpr int kSoftWarp0 = 4, kSoftWarps = 8, kSoftThreads = kSoftWarps * 32;
constexpr int kThreads = kSoftWarp0 * 32 + kSoftThreads;
constexpr int kMaxSlots = 13;               // slots of the rings of chunks
constexpr int kScaleSlots = 4;              // tiles whose row scales are kept; the rings hold at most three tiles
constexpr int kMaxCtas = 160;               // bound of workers x head groups
constexpr int kTmemCols = 512;
constexpr int kTmemS = 256;                 // first column of S^T
constexpr int kTmemSfa = 384, kTmemSfb = 388;   // block scales of C^T (ones) and of p s
constexpr int kStacked = 32;                // heads up to which hi and lo of p s stand side by side too
constexpr float kRaise = 32.0f;             // log2 by which a block may exceed the reference before O is rescaled
constexpr float kLeastScale = 0x1p-60f;
constexpr float kNothing = -3.402823466e38f; // log2 of p s of a token past the length: no finite one is lower
constexpr int kMiscBytes = 7168;
constexpr int kPBytes = kTile * 64;         // hi (or lo) of p s of a tile: 64 bytes a token
constexpr int kManyParts = 4;               // workers per job from which a CTA joins an item

struct Params {
    uint8_t* images;                  // [B * G + NP * G] of a job's split queries (see prepare_kernel)
    int image;                        // bytes of one
    const float* scales;
    int64_t ld_scale;                 // of a page
    const int32_t* seq_lens;
    const int32_t* table;
    int64_t ld_table;
    const int32_t* prefix_table;
    const int32_t* prefix_len;        // NULL: no common prefix
    int B, H, G, W;                   // requests, heads, head groups, workers
    int W_full;                       // workers that the GPU has room for, whatever the tables hold
    int hg;                           // log2 of the heads (rows) of a group
    int HR;                           // rows of a request against the prefix: heads, a multiple of 4
    int R, NP;                        // rows against the prefix; jobs of them (G groups each)
    int width, prefix_width, page_size, box_rows, num_pages;   // box_rows: tokens of one copy
    int64_t cap, prefix_cap;          // tokens the tables can hold
    int cc, pe, nblk;                 // 128-code chunks of a row, position chunk, 128-column blocks of the value
    int q_rows;                       // rows of hi (and of lo) that a chunk of q has room for
    int slots, odd_slots;             // slots of both rings, and of the odd chunks'
    int twin;                         // position columns share a slot with the last codes
    float scale_log2;
    __nv_bfloat16* out;
    int64_t ldo_b, ldo_h;
    float* lse;                       // NULL: not written
    int64_t ldl_b;
    int2* meta;                       // [W + 1] first job of the worker and its first tile there; the end
    float2* part_ml;                  // [part][64] (reference in log2 units, sum)
    float* part_o;                    // [part][nblk][16][128][4]: value block, four heads, value, head
    uint64_t timeout_ns;
    uint32_t inject;
};

__device__ __forceinline__ int clamp_len(int64_t cap, int32_t n) {
    return n < 0 ? 0 : (n > cap ? static_cast<int>(cap) : n);
}
// Tiles of a request; an empty one counts as one (somebody writes its zeros).
__device__ __forceinline__ int tiles_of(int len) { return len > kTile ? (len + kTile - 1) / kTile : 1; }

// Place of the part that worker w leaves of job j in the workspace.  With a
// prefix every job leaves its parts: along the runs j + w grows from part to
// part.  Otherwise only the first and the last job of a run can be cut.
__device__ __forceinline__ int64_t part_slot(const Params& p, int w, int j, bool first, int g) {
    return static_cast<int64_t>(p.prefix_len ? j + w : 2 * w + (first ? 0 : 1)) * p.G + g;
}

// Whether a part or an image lies in the workspace (the debug build's checks).
__device__ __forceinline__ bool part_ok(const Params& p, int64_t slot) {
    return slot >= 0 && slot < static_cast<int64_t>(p.prefix_len ? p.NP + p.B + p.W : 2 * p.W) * p.G;
}
__device__ __forceinline__ bool image_ok(const Params& p, int64_t image) {
    return image >= 0 && image < (static_cast<int64_t>(p.B) + p.NP) * p.G;
}

// The same value, of which the compiler knows nothing: it would otherwise make
// copies of a loop for either outcome of a test in it (the softmax had four, and
// the warps' code no room in the instruction cache).
__device__ __forceinline__ bool opaque(bool v) {
    uint32_t u = v;
    asm volatile("" : "+r"(u));
    return u != 0;
}

__device__ __forceinline__ bool elected() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t chunk, int32_t group,
                                            int32_t page, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(chunk), "r"(group), "r"(page), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void tma_prefetch_5d(const CUtensorMap* map, int32_t chunk, int32_t group, int32_t page, uint64_t policy) {
    asm volatile("cp.async.bulk.prefetch.tensor.5d.L2.global.tile.L2::cache_hint [%0, {%1, %1, %2, %3, %4}], %5;" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(0), "r"(chunk), "r"(group), "r"(page), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}
// 16 bytes into shared memory, and an arrival on the barrier when this thread's
// copies so far are there.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Instruction descriptors: D fp32, M = 128.  e4m3 x e4m3, both K-major; bf16 x
// bf16; and block-scaled e4m3 x e4m3 with both operands column-major, scales as
// powers of two, `block` the byte of B's scale words that holds this block's.
__device__ __forceinline__ uint32_t idesc_s(int n) { return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24); }
__device__ __forceinline__ uint32_t idesc_pe(int n) { return idesc_s(n) | (1u << 7) | (1u << 10); }
__device__ __forceinline__ uint32_t idesc_o(int n) {
    return (1u << 15) | (1u << 16) | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) | (8u << 24);
}

// Shared-memory descriptors as two words, of which the steps of a product change
// the lower one only.  The upper one: eight rows `stride` bytes on, version 1,
// swizzle code.
constexpr uint32_t desc_high(uint32_t stride, uint32_t swizzle) { return (stride >> 4) | 1u << 14 | swizzle << 29; }
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lead) { return ((addr >> 4) & 0x3FFF) | (lead >> 4) << 16; }
constexpr uint32_t kHighSw128 = desc_high(1024, 2);   // 128-byte rows and swizzle: chunks of the tile and of q
constexpr uint32_t kHighSw64 = desc_high(512, 4);     // 64-byte rows and swizzle: p s
constexpr uint32_t kHighRows16 = desc_high(128, 0);   // 16-byte rows: block scales

// Four steps of D (+)= A B^T along the 128 bytes of a chunk's rows, issued by
// one elected lane; the first overwrites D when !accumulate.
#define DSNQ_STEP(KIND, K)                                                                                             \
    "add.u32 x, %1, " K ";\n\tadd.u32 y, %2, " K ";\n\tmov.b64 a, {x, %5};\n\tmov.b64 b, {y, %5};\n\t"                \
    "@e tcgen05.mma.cta_group::1.kind::" KIND " [%0], a, b, %3, t;\n\t"
#define DSNQ_MMA4(KIND)                                                                                                \
    asm volatile(                                                                                                      \
        "{\n\t.reg .pred p, e, t;\n\t.reg .b64 a, b;\n\t.reg .b32 x, y;\n\t"                                           \
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\telect.sync _|e, 0xffffffff;\n\t"                            \
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"                                                            \
        "@e tcgen05.mma.cta_group::1.kind::" KIND " [%0], a, b, %3, p;\n\t"                                           \
        DSNQ_STEP(KIND, "2") DSNQ_STEP(KIND, "4") DSNQ_STEP(KIND, "6") "}" ::"r"(d_tmem),                              \
        "r"(a_low), "r"(b_low), "r"(idesc), "r"(accumulate), "n"(kHighSw128)                                           \
        : "memory")
__device__ __forceinline__ void tc_mma4_e4m3(uint32_t d_tmem, uint32_t a_low, uint32_t b_low, uint32_t idesc, uint32_t accumulate) {
    DSNQ_MMA4("f8f6f4");
}
__device__ __forceinline__ void tc_mma4_bf16(uint32_t d_tmem, uint32_t a_low, uint32_t b_low, uint32_t idesc, uint32_t accumulate) {
    DSNQ_MMA4("f16");
}
#undef DSNQ_MMA4
#undef DSNQ_STEP

// O^T (+)= C^T (p s)^T of one chunk of codes: four blocks of 32 tokens (4 KB of
// the tile, 2 KB of p s apart).  PAIR: of each block the product with hi and the
// one with lo (8 KB on), whose scales lie two columns on; otherwise one product
// with both, side by side.
template <bool PAIR>
__device__ __forceinline__ void tc_mma_scaled(uint32_t d_tmem, uint32_t a_low, uint32_t b_low, uint32_t idesc, uint32_t sfa,
                                              uint32_t sfb, uint32_t accumulate) {
#define DSNQ_MX "@e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X "
#define DSNQ_B(B) "add.u32 y, %2, " B ";\n\tmov.b64 b, {y, %9};\n\t"
#define DSNQ_STEP(A, B, ID)                                                                                            \
    "add.u32 x, %1, " A ";\n\tmov.b64 a, {x, %8};\n\tadd.u32 i, %3, " ID ";\n\t" DSNQ_B(B) DSNQ_MX "[%0], a, b, i, [%4], [%5], t;\n\t"
#define DSNQ_LOW(B) DSNQ_B(B) DSNQ_MX "[%0], a, b, i, [%4], [%6], t;\n\t"
#define DSNQ_ASM(STEPS)                                                                                                \
    asm volatile(                                                                                                      \
        "{\n\t.reg .pred p, e, t;\n\t.reg .b64 a, b;\n\t.reg .b32 i, x, y;\n\t"                                        \
        "setp.ne.b32 p, %7, 0;\n\tsetp.eq.b32 t, 0, 0;\n\telect.sync _|e, 0xffffffff;\n\t"                            \
        "mov.b64 a, {%1, %8};\n\tmov.b64 b, {%2, %9};\n\tmov.b32 i, %3;\n\t" DSNQ_MX "[%0], a, b, i, [%4], [%5], p;\n\t" \
        STEPS "}" ::"r"(d_tmem),                                                                                       \
        "r"(a_low), "r"(b_low), "r"(idesc), "r"(sfa), "r"(sfb), "r"(sfb + 2), "r"(accumulate), "n"(kHighSw128), "n"(kHighSw64) \
        : "memory")
    if (PAIR)
        DSNQ_ASM(DSNQ_LOW("512") DSNQ_STEP("256", "128", "16") DSNQ_LOW("640") DSNQ_STEP("512", "256", "32") DSNQ_LOW("768")
                     DSNQ_STEP("768", "384", "48") DSNQ_LOW("896"));
    else
        DSNQ_ASM(DSNQ_STEP("256", "128", "16") DSNQ_STEP("512", "256", "32") DSNQ_STEP("768", "384", "48"));
#undef DSNQ_ASM
#undef DSNQ_LOW
#undef DSNQ_STEP
#undef DSNQ_B
#undef DSNQ_MX
}

// 512 bytes of block scales into four TMEM columns of all lane quarters.
__device__ __forceinline__ void tc_copy_scales(uint32_t taddr, uint64_t desc) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
        "l"(desc)
        : "memory");
}

// 16 lanes x 16 columns of TMEM as matrix fragments: of each 8 columns, thread i
// gets columns 2 (i % 4), + 1 of lane i / 4 and of lane i / 4 + 8.
__device__ __forceinline__ void tmem_ld_frag16(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld8_wait(uint32_t (&r)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_ld4_issue(uint32_t taddr, uint32_t (&r)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld4_wait(uint32_t (&r)[4]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3])::"memory");
}
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t (&r)[4]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t (&r)[4]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%4], {%0, %1, %2, %3};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ float redux_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// hi = e4m3(x), lo = e4m3(32 (x - hi)) of two numbers (|x| <= 256: x - hi is at
// most 8, in half precision); `sum` gets hi + lo / 32.  (The conversion from
// fp32 pairs takes a third of the time of the one from half pairs, which the
// remainder uses because it is one.)
__device__ __forceinline__ __half2 half2_of(uint32_t codes) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
    return *reinterpret_cast<const __half2*>(&r);
}
__device__ __forceinline__ void split2(float2 x, uint32_t& hi, uint32_t& lo, __half2& sum) {
    uint16_t c;
    hi = e4m3x2(x);
    const __half2 h = half2_of(hi), d = __hmul2(__hsub2(__float22half2_rn(x), h), __float2half2_rn(32.f));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(*reinterpret_cast<const uint32_t*>(&d)));
    lo = c;
    sum = __hfma2(half2_of(lo), __float2half2_rn(0.03125f), h);
}
__device__ __forceinline__ float2 unpack_bf16(uint32_t v) { return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)); }

// The largest magnitude of eight bf16, as its bits (NaN above all others).
__device__ __forceinline__ uint32_t largest8(const uint4& v) {
    const uint32_t a = __vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), b = __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu);
    const uint32_t c = __vmaxu2(a, b);
    return max(c & 0xffffu, c >> 16);
}

// lg2.approx: off by at most 2^-22 here, and its inverse is taken from itself.
__device__ __forceinline__ float log2_fast(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Registers of a copying or issuing thread and of a softmax thread: together
// those that the CTA is launched with (168 each).  What does not fit goes to
// local memory, whose loads wait behind the products' reads of shared memory (16
// bytes are spilled at 48 rows, 76 at 64, none below).
// Measured, 88 and 208 against 72 and 216: 2.05 and 2.18 us a tile at 48 heads of
// 512 columns; sixteen softmax warps of half as many heads each, 56 and 104
// registers: 2.31.
constexpr int kRegsIssue = 88, kRegsSoft = 208;
static_assert(128 * kRegsIssue + kSoftThreads * kRegsSoft <= kThreads * 168, "registers of the CTA at its launch");

// wait_bounded<true> in a few instructions: the clock is first read after 64
// polls.  (The kernel's code has to stay small: the issuing warps run theirs
// once a tile, between passes of the softmax warps through theirs.)
__device__ __forceinline__ bool wait_polled(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t timeout_ns) {
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t n = 1; !mbar_try_wait(bar, parity); ++n) {
        if (n & 63) continue;
        if (*abort) return false;
        const uint64_t now = now_ns();
        if (n == 64) t0 = now;
        if (now - t0 > timeout_ns) {
            *abort = 1;
            atomicOr(&g_status, kStatusTimeout);
            return false;
        }
    }
    return true;
}

// Barriers of all softmax warps, and of the four that have the same heads
// (returns whether any of their threads passed true).  A named barrier has no
// time limit, so every softmax warp reaches every one of them whether or not
// its waits succeeded (the counts depend on the run alone).
__device__ __forceinline__ void soft_sync() { asm volatile("barrier.cta.sync 1, %0;" ::"n"(kSoftThreads) : "memory"); }
__device__ __forceinline__ bool half_sync_or(int half, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(v)), "r"(2 + half)
        : "memory");
    return r != 0;
}

// Where the chunks of the worker's n-th tile lie: chunk c of a tile is its first
// codes (c = 0), its position columns (c = 1, if any), its other codes.  Each of
// the two copying warps has a ring of its own, the even chunks' and the odd
// ones' (a slot's next copy is then always issued by the warp that waited for
// the one before: with one ring the parity of a phase would not say which pass
// it is).  S^T of a tile needs all of its chunks while the codes of the tile
// before wait for their product with p s, so there must be room for two tiles.
// With 512 codes, position columns and more than 32 heads there is not, by one
// slot or two: there (`twin`) a tile has four slots, and the last codes follow
// the position columns, which S^T is done with early, in one slot.
struct Chunks {
    int even = 0, odd = 0;            // places of the next even and odd chunk in their rings
    uint32_t passes = 0;              // parities of the rings' passes: bit 0 even, bit 1 odd
    int first_odd = 0;                // slot of the tile's first odd chunk
    // Chunk c, the chunks of a tile being taken in order.
    __device__ __forceinline__ void take(const Params& p, int c, int& slot, uint32_t& parity) {
        const bool r = c & 1, twin = opaque(p.twin);
        if (twin && c == 4) {
            slot = first_odd;
            parity = 1;
            return;
        }
        const int at = r ? odd : even, evens = p.slots - p.odd_slots;
        slot = twin ? 2 * at + r : at + (r ? evens : 0);
        parity = twin && c == 1 ? 0 : passes >> r & 1;
        if (c == 1) first_odd = slot;
        const bool wrap = at + 1 == (r ? p.odd_slots : evens);
        const int next = wrap ? 0 : at + 1;
        odd = r ? next : odd;
        even = r ? even : next;
        passes ^= static_cast<uint32_t>(wrap) << r;
    }
    // Slot of chunk c of the n-th tile.
    static __device__ __forceinline__ int slot_of(const Params& p, uint32_t n, int c) {
        if (p.twin) return static_cast<int>(n & 1) * 4 + (c == 4 ? 1 : c);
        const int r = c & 1, size = r ? p.odd_slots : p.slots - p.odd_slots, each = (p.cc + p.pe + 1 - r) >> 1;
        return static_cast<int>((n % size * each + (c >> 1)) % size) + (r ? p.slots - p.odd_slots : 0);
    }
};

// A worker's run of tiles, job by job: from tile t0 of job j up to (not
// including) tile t_end of job j_end.  Jobs below NP are rows against the
// prefix, job NP + b is request b.
struct Run {
    int j, t0, j_end, t_end;
    int plen;                         // tokens of the prefix
    int32_t ahead;                    // seq_lens of the next request: a trip to memory ahead of its use
    int len, tiles, n;                // of the current job: tokens, tiles, tiles of this run
    int count;                        // its rows in this CTA
    __device__ __forceinline__ bool next(const Params& p, int g) {
        if (j > j_end || (j == j_end && t0 >= t_end)) return false;
        const bool prefix = j < p.NP;
        len = prefix ? plen : clamp_len(p.cap, ahead);
        if (j + 1 >= p.NP && j + 1 < p.NP + p.B) ahead = p.seq_lens[j + 1 - p.NP];
        tiles = tiles_of(len);
        n = (j == j_end ? t_end : tiles) - t0;
        const int rows = prefix ? p.R - ((j * p.G + g) << p.hg) : p.H - (g << p.hg);
        count = max(0, min(1 << p.hg, rows));
        return true;
    }
    __device__ __forceinline__ bool live() const { return len > 0 && count > 0; }
    __device__ __forceinline__ void advance() {
        ++j;
        t0 = 0;
    }
};

// ---------------------------------------------------------------------------
// What the attention's CTAs would each do again.
//
// The first CTA shares out the work.  Each job counts `lead` units (what it costs
// beside its tiles: queries, pipeline fill, output), then one per tile; worker w
// takes units [w U / workers, (w + 1) U / workers), and a cut among a job's
// leading units is a cut before its first tile.  The jobs against the prefix come
// first.
//
// The others split the queries into images of what a job's CTA has in shared
// memory: codes of hi and of lo, chunk by chunk of 128, rows 128-byte swizzled,
// then the bf16 position columns divided by the same power of two, then the
// factors of the scores.  Image b G + g is that of group g's heads of request b;
// behind those come the prefix's, of as many (request, head) pairs each.  A warp takes
// a row; rows that pad an image keep what they hold (nothing of their columns is
// used).  In the attention's own warps, between the jobs, the split took 4.7 us a
// job of 64 heads.
// ---------------------------------------------------------------------------
constexpr int kPrepareThreads = 256;

__device__ void share_out(const Params& p) {
    constexpr int kWarps = kPrepareThreads / 32;
    __shared__ int64_t sums[kWarps], before_s[kPrepareThreads];
    __shared__ int longest[kWarps];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int plen = p.prefix_len ? clamp_len(p.prefix_cap, *p.prefix_len) : 0;
    // Thread t sums requests [t * per, (t + 1) * per).
    const int per = (p.B + kPrepareThreads - 1) / kPrepareThreads;
    const int b0 = min(t * per, p.B), b1 = min(b0 + per, p.B);
    int64_t mine = 0;
    int most = 0;
    for (int b = b0; b < b1; ++b) {
        const int n = tiles_of(clamp_len(p.cap, p.seq_lens[b]));
        mine += n;
        most = max(most, n);
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
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        if (i < warp) before += sums[i];
        tiles += sums[i];
        most = max(most, longest[i]);
    }
    const int ptiles = plen > 0 ? tiles_of(plen) : 0, pjobs = plen > 0 ? p.NP : 0;
    tiles += static_cast<int64_t>(pjobs) * ptiles;
    // Requests a little longer than a worker's share go one to a worker, uncut.
    const int h = min(p.H, 1 << p.hg), joined = 5 * p.B * h / (16 * p.W_full);
    const int slack = max(1, p.W < kManyParts * p.B ? min(joined, 2 + h / 64) : joined);
    const bool uncut = !p.prefix_len && p.B <= p.W && tiles > static_cast<int64_t>(most - slack - 1) * p.W;
    const int lead = tiles < p.W ? 0 : tiles < 2 * p.W ? 1 : 2;
    const int64_t front = static_cast<int64_t>(pjobs) * (lead + ptiles);   // units of the prefix
    const int64_t total = tiles + static_cast<int64_t>(lead) * (p.B + pjobs);
    before_s[t] = before + front + static_cast<int64_t>(lead) * b0;
    __syncthreads();
    const int workers = total < p.W ? static_cast<int>(total) : p.W;
    for (int w = t; w <= p.W; w += kPrepareThreads) {
        int2 cut = make_int2(p.NP + min(w, p.B), 0);       // uncut
        if (!uncut) {
            int64_t u = total;
            if (w < workers)                               // (a 32-bit division is a fraction of the 64-bit one)
                u = total < 1 << 24 ? static_cast<uint32_t>(w) * static_cast<uint32_t>(total) / static_cast<uint32_t>(workers)
                                    : w * total / workers;
            if (u == total) {
                cut.x = p.NP + p.B;
            } else if (u < front) {
                cut.x = static_cast<int>(u / (lead + ptiles));
                cut.y = max(static_cast<int>(u - static_cast<int64_t>(cut.x) * (lead + ptiles)) - lead, 0);
            } else {
                int k = 0;                                 // the last thread whose requests begin at or before u
#pragma unroll
                for (int o = kPrepareThreads / 2; o > 0; o >>= 1)
                    if (before_s[k + o] <= u) k += o;
                int64_t at = before_s[k];
                int b = k * per, n = lead + tiles_of(clamp_len(p.cap, p.seq_lens[b]));
                while (at + n <= u) {
                    at += n;
                    n = lead + tiles_of(clamp_len(p.cap, p.seq_lens[++b]));
                }
                cut = make_int2(p.NP + b, max(static_cast<int>(u - at) - lead, 0));
            }
        }
        if (bounds_ok(cut.x >= 0 && cut.x <= p.NP + p.B && cut.y >= 0)) p.meta[w] = cut;
    }
}

__global__ void __launch_bounds__(kPrepareThreads)
prepare_kernel(const Params p, const __nv_bfloat16* q, int64_t ldq_b, int64_t ldq_h) {
    grid_dependency_wait();
    allow_dependent_launch();
    bounds_self_test(p.inject);
    if (blockIdx.x == 0) {
        share_out(p);
        return;
    }
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x - 1) * (kPrepareThreads / 32) + (threadIdx.x >> 5);
    if (row >= static_cast<int64_t>(p.B) * p.H) return;
    const int b = static_cast<int>(row / p.H), h = static_cast<int>(row - static_cast<int64_t>(b) * p.H);
    const bool codes = lane * 16 < p.cc * 128, pos = p.pe && lane < 8;
    const __nv_bfloat16* src = q + b * ldq_b + h * ldq_h;
    uint4 x[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}, e = make_uint4(0, 0, 0, 0);
    if (codes) {
        x[0] = *reinterpret_cast<const uint4*>(src + lane * 16);
        x[1] = *reinterpret_cast<const uint4*>(src + lane * 16 + 8);
    }
    if (pos) e = *reinterpret_cast<const uint4*>(src + p.cc * 128 + lane * 8);
    // The largest magnitudes, as the bits of a bf16 (NaN above all others).
    const uint32_t top = __reduce_max_sync(0xffffffffu, max(largest8(x[0]), largest8(x[1])));
    const uint32_t etop = __reduce_max_sync(0xffffffffu, largest8(e));
    // 2^ex > largest / 256, so that 32 (x - hi) <= 256.  And the position columns
    // divided by it are below 2^25: the cache's are divided by its scale (2^60 for
    // a 1 behind a latent of zeros) and the sum of their 64 products has to stay
    // finite, which leaves 2^96 for them.  (Latent columns that this rounds away
    // are below 2^-39 of the position columns.)  The factor of the score times the
    // scale may then be subnormal, off by 2^-150, which is 2^-22 of a score at most.
    int ex = static_cast<int>(top >> 7) - 127 - 7;
    ex = max(max(ex, -100), static_cast<int>(etop >> 7) - 127 - 24);
    const bool finite = max(top, etop) < 0x7f80;
    if (!finite) ex = 0;
    const float inv = __int_as_float((127 - ex) << 23);
    const float factor = finite ? __int_as_float((127 + ex) << 23) * p.scale_log2 : __int_as_float(0x7fffffff);
    const uint32_t* xw = reinterpret_cast<const uint32_t*>(x);
    const uint32_t* ew = reinterpret_cast<const uint32_t*>(&e);
    uint32_t hi[4], lo[4], v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t h0, h1, l0, l1;
        __half2 s;
        split2(mul2(unpack_bf16(xw[2 * k]), make_float2(inv, inv)), h0, l0, s);
        split2(mul2(unpack_bf16(xw[2 * k + 1]), make_float2(inv, inv)), h1, l1, s);
        hi[k] = __byte_perm(h0, h1, 0x5410);
        lo[k] = __byte_perm(l0, l1, 0x5410);
        const float2 f = mul2(unpack_bf16(ew[k]), make_float2(inv, inv));
        v[k] = pack_bf16(f.x, f.y);
    }
    for (int to = 0; to < (p.NP ? 2 : 1); ++to) {
        const int64_t r = static_cast<int64_t>(b) * p.HR + h;
        const int64_t image = to ? static_cast<int64_t>(p.B) * p.G + (r >> p.hg) : static_cast<int64_t>(b) * p.G + (h >> p.hg);
        const int i = (to ? static_cast<int>(r) : h) & ((1 << p.hg) - 1);
        uint8_t* at = p.images + image * p.image;
        if (!bounds_ok(i < p.q_rows && image_ok(p, image))) continue;
        if (codes) {
            uint8_t* c = at + (lane >> 3) * 2 * p.q_rows * 128 + (((lane & 7) ^ (i & 7)) << 4);
            *reinterpret_cast<uint4*>(c + i * 128) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(c + (p.q_rows + i) * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        if (pos)
            *reinterpret_cast<uint4*>(at + p.cc * 2 * p.q_rows * 128 + i * 128 + ((lane ^ (i & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
        if (lane == 0) *reinterpret_cast<float*>(at + p.image - kHeads * 4 + i * 4) = factor;
    }
}

template <int NG>
__global__ void __launch_bounds__(kThreads, 1)
latent_attention_fp8_kernel(const __grid_constant__ CUtensorMap map_c, const Params p) {
    constexpr int HP = 16 * NG;                            // rows (heads) of a job, with those that pad it
    constexpr bool kPair = HP > kStacked;
    constexpr uint32_t kLow = kPair ? 0 : HP;              // columns from hi's part of O to lo's
    constexpr int hpp = HP / 2;                            // heads of a softmax warp, a multiple of eight
    constexpr int kBands = (hpp + 15) / 16;                // sixteens of them
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int q_chunk = 2 * p.q_rows * 128;                // bytes of a code chunk of q: hi, then lo
    const int cpt = p.cc + p.pe;                           // chunks of a tile
    uint8_t* q_s = smem;                                   // [cc][2 q_rows][128 B]
    uint8_t* qpe_s = q_s + p.cc * q_chunk;                 // [pe][q_rows][128 B]
    uint8_t* p_s = qpe_s + p.pe * p.q_rows * 128;          // hi, lo: [128 tokens][64 B]
    uint8_t* ring = p_s + 2 * kPBytes;                     // [slots][128 tokens][128 B]
    uint8_t* misc = ring + p.slots * kChunkBytes;
    uint8_t* sf_s = misc;                                  // [32][16 B] block scales of p s
    float* sc_s = reinterpret_cast<float*>(sf_s + 512);    // [kScaleSlots][128] row scales
    float* cq_s = sc_s + kScaleSlots * kTile;              // [64] factor of a head's scores
    float* bc_s = cq_s + kHeads;                           // [8 warps][32]{T, 2^(T - M)}; at a job's end {l, lr}
    float* mx_s = bc_s + kSoftWarps * 2 * kPer;            // [8 warps][32]
    float* al_s = mx_s + kSoftWarps * kPer;                // [64] factors of O
    uint64_t* full = reinterpret_cast<uint64_t*>(al_s + kHeads);   // [kMaxSlots]
    uint64_t* empty = full + kMaxSlots;                    // [kMaxSlots]
    uint64_t* scfull = empty + kMaxSlots;                  // [kScaleSlots]
    uint64_t* qfull = scfull + kScaleSlots;
    uint64_t* sfull = qfull + 1;
    uint64_t* sempty = sfull + 1;
    uint64_t* pfull = sempty + 1;
    uint64_t* pempty = pfull + 1;
    uint64_t* drain = pempty + 1;                          // [2] abort: products already issued
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int w = blockIdx.x / p.G, g = blockIdx.x - w * p.G;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxSlots; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int s = 0; s < kScaleSlots; ++s) mbar_init(smem_u32(&scfull[s]), 32);
        mbar_init(smem_u32(qfull), 1);
        mbar_init(smem_u32(sfull), 1);
        mbar_init(smem_u32(sempty), kSoftWarps);
        mbar_init(smem_u32(pfull), kSoftWarps);
        mbar_init(smem_u32(pempty), 1);
        for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&drain[i]), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tma_prefetch_desc(&map_c);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    if (warp >= kSoftWarp0 && warp < kSoftWarp0 + 4) {     // the scales of C^T are ones (for the product after pfull)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                         tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + kTmemSfa),
                     "r"(0x7f7f7f7f)
                     : "memory");
        tmem_wait_st();
    }
    grid_dependency_wait();
    allow_dependent_launch();
    bounds_self_test(p.inject);

    // The worker's run.
    const int2 from = p.meta[w], to = p.meta[w + 1];
    Run run;
    run.j = from.x;
    run.t0 = from.y;
    run.j_end = to.x;
    run.t_end = to.y;
    run.plen = p.prefix_len ? clamp_len(p.prefix_cap, *p.prefix_len) : 0;
    run.ahead = 0;
    if (run.j >= p.NP && run.j < p.NP + p.B) run.ahead = p.seq_lens[run.j - p.NP];
    const int j_first = run.j;
    const uint64_t tmo = p.timeout_ns;

    // A whole warp's wait: all of its lanes go on or none (warp-wide
    // instructions follow), and the compiler sees that it is so.
    auto wait_uniform = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_polled(bar, parity, abort_flag, tmo));
    };
    // The same, asleep between polls: for the copying warp, which is ahead.
    auto wait_uniform_asleep = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_bounded(bar, parity, abort_flag, tmo));
    };

    if (warp < kSoftWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == 0 || warp == 3) {
        // ------------------------------------------------------ TMA producers
        // Chunks in the order of their use by S^T, every other one from each of
        // the two warps (a copy takes a warp some 50 cycles, and small pages make
        // many): the first codes (and the tile's row scales), the position columns,
        // whose slot is free again when S^T is done with them, the other codes.  A request's tiles pass
        // through L2 once, so they leave it first; the prefix's are read by
        // every group of rows.
        uint64_t once, again;
        asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
        asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(again));
        const int pieces = kTile / p.box_rows;             // copies of a chunk (1, 2, 4, 8 or 16)
        const int batch = 32 / pieces;                     // tiles whose table entries the lanes hold
        const int odd = warp == 3;
        const int lines = p.twin ? 2 + odd : (cpt + 1 - odd) / 2;   // this warp's chunks of a tile
        const uint32_t to = smem_u32(ring) + lane * p.box_rows * 128;
        Chunks ch;
        uint32_t n = 0;
        bool ok = true, skip = !odd && (p.inject & kInjectSkipLoad) != 0;
#pragma unroll 1
        for (; ok && run.next(p, g); run.advance()) {
            if (!run.live()) continue;
            const bool prefix = run.j < p.NP;
            const int32_t* row = prefix ? p.prefix_table : p.table + (run.j - p.NP) * p.ld_table;
            const int width = prefix ? p.prefix_width : p.width;
            const uint64_t policy = prefix ? again : once;
            int ids = 0, offs = 0;
#pragma unroll 1
            for (int i = 0; ok && i < run.n; ++i, ++n) {
                const int tile = run.t0 + i;
                if (i % batch == 0) {
                    const int64_t tok = static_cast<int64_t>(tile) * kTile + static_cast<int64_t>(lane) * p.box_rows;
                    ids = offs = 0;
                    if (tok < run.len) {
                        const int e = static_cast<int>(tok) / p.page_size;
                        offs = static_cast<int>(tok) - e * p.page_size;
                        if (bounds_ok(e < width)) ids = row[e];
                        if (ids < 0 || ids >= p.num_pages) {   // such pages read as zeros
                            atomicOr(&g_status, kStatusBounds);
                            ids = p.num_pages;
                        }
                    }
                }
                const int live = min(pieces, (run.len - tile * kTile + p.box_rows - 1) / p.box_rows);
                const int from = (i % batch) * pieces + (lane & (pieces - 1));
                const int id = __shfl_sync(0xffffffffu, ids, from), in_page = __shfl_sync(0xffffffffu, offs, from);
#pragma unroll 1
                for (int k = 0; k < lines; ++k) {
                    const int c = odd && k == 2 ? 4 : 2 * k + odd;
                    const int chunk = c == 0 ? 0 : !p.pe ? c : c == 1 ? p.cc : c - 1;
                    int slot;
                    uint32_t parity;
                    ch.take(p, c, slot, parity);
                    ok = bounds_ok(slot >= 0 && slot < p.slots && chunk < cpt);
                    if (!ok) break;
                    // Barely two tiles of room: while it waits for the slot, the
                    // chunk comes as near as L2 (2.77 -> 2.69 us a tile at 64 heads
                    // of 576 columns; a whole tile ahead 2.87; with more room
                    // slower: 128 x 8000 tokens, 48 heads of 512, 148 -> 157 us).
                    if (opaque(p.twin) && lane < live && id < p.num_pages) tma_prefetch_5d(&map_c, chunk, in_page / 8, id, policy);
                    ok = wait_uniform_asleep(smem_u32(&empty[slot]), parity ^ 1);
                    if (!ok) break;
                    const uint32_t fb = smem_u32(&full[slot]);
                    if (!skip) {                           // test hook: the first chunk never comes, the waits on it run out
                        if (lane == 0) mbar_arrive_expect_tx(fb, live * p.box_rows * 128);
                        __syncwarp();
                        if (lane < live) tma_load_5d(to + slot * kChunkBytes, &map_c, fb, chunk, in_page / 8, id, policy);
                    }
                    skip = false;
                    if (c == 0) {
                        // Four row scales a lane.  (The tile that had their place
                        // has gone, since this chunk's slot is free.)
                        const int own = lane * 4 / p.box_rows;
                        const int page = __shfl_sync(0xffffffffu, id, own), first = __shfl_sync(0xffffffffu, in_page, own);
                        float* sc = sc_s + (n & (kScaleSlots - 1)) * kTile + lane * 4;
                        const uint32_t sb = smem_u32(&scfull[n & (kScaleSlots - 1)]);
                        if (own < live && page < p.num_pages) {
                            copy16(smem_u32(sc), p.scales + static_cast<int64_t>(page) * p.ld_scale + first + lane * 4 - own * p.box_rows);
                            copies_arrive(sb);
                        } else {
                            *reinterpret_cast<float4*>(sc) = make_float4(0.f, 0.f, 0.f, 0.f);
                            mbar_arrive(sb);
                        }
                    }
                }
            }
        }
        if (!ok) settle_ns(kAbortSettleNs);                // copies already issued land before the CTA goes
    } else if (warp == 1) {
        // ---------------------------------------------- products S^T = C Q^T
        // Chunk by chunk as they land.
        const uint32_t q_low = desc_low(smem_u32(q_s), 16), pe_low = desc_low(smem_u32(qpe_s), 16);
        const uint32_t d = tmem + kTmemS;
        Chunks ch;
        uint32_t n = 0, nq = 0;
        bool ok = true;
#pragma unroll 1
        for (; ok && run.next(p, g); run.advance()) {
            if (!run.live()) continue;
            // The job's queries, when the softmax has S^T of the job before: then
            // neither its queries nor their factors are read any more.
            ok = wait_uniform(smem_u32(sempty), (n & 1) ^ 1);
            if (!ok) break;
            if (elected()) {
                const uint32_t bytes = p.image - kHeads * 4;
                const int64_t at = run.j < p.NP ? static_cast<int64_t>(p.B + run.j) * p.G + g : static_cast<int64_t>(run.j - p.NP) * p.G + g;
                const uint8_t* src = p.images + (bounds_ok(image_ok(p, at)) ? at : 0) * p.image;
                mbar_arrive_expect_tx(smem_u32(qfull), p.image);
                bulk_load(smem_u32(q_s), src, bytes, smem_u32(qfull));
                bulk_load(smem_u32(cq_s), src + bytes, kHeads * 4, smem_u32(qfull));
            }
            __syncwarp();
            ok = wait_uniform(smem_u32(qfull), nq & 1);
            ++nq;
            // The output of the job before waits for its last O^T, this job's
            // softmax for the output: S^T comes second.
            ok = ok && wait_uniform(smem_u32(pempty), (n & 1) ^ 1);
#pragma unroll 1
            for (int i = 0; ok && i < run.n; ++i, ++n) {
                ok = wait_uniform(smem_u32(sempty), (n & 1) ^ 1);
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; ok && c < cpt; ++c) {
                    int slot;
                    uint32_t parity;
                    ch.take(p, c, slot, parity);
                    const int code = c == 0 ? 0 : c - p.pe;
                    const bool pe = c == 1 && opaque(p.pe);
                    ok = bounds_ok(slot >= 0 && slot < p.slots && code < p.cc && kTmemS + 2 * HP <= kTmemSfa);
                    if (!ok) break;
                    const uint32_t a = desc_low(smem_u32(ring) + slot * kChunkBytes, 16);
                    ok = wait_uniform(smem_u32(&full[slot]), parity);
                    if (!ok) break;
                    if (pe) tc_mma4_bf16(d, a, pe_low, idesc_pe(HP), 1);
                    else tc_mma4_e4m3(d, a, q_low + static_cast<uint32_t>(code * q_chunk >> 4), idesc_s(2 * HP), c > 0);
                    if (pe || code >= p.nblk) tc_commit(smem_u32(&empty[slot]));   // no part of the value
                }
                if (!ok) break;
                tc_commit(smem_u32(sfull));
            }
        }
        if (!ok) {                                         // products already issued end before their memory goes
            tc_commit(smem_u32(&drain[0]));
            wait_drain(smem_u32(&drain[0]), 0, tmo);
        }
    } else if (warp == 2) {
        // ----------------------------------------- products O^T += C^T (p s)^T
        // They free the chunks one by one.
        const uint32_t p_low = desc_low(smem_u32(p_s), kPBytes);
        const uint64_t sf_desc = static_cast<uint64_t>(kHighRows16) << 32 | desc_low(smem_u32(sf_s), 0);
        Chunks ch;
        uint32_t n = 0;
        bool ok = true;
#pragma unroll 1
        for (; ok && run.next(p, g); run.advance()) {
            if (!run.live()) continue;
#pragma unroll 1
            for (int i = 0; i < run.n; ++i, ++n) {
                ok = wait_uniform(smem_u32(pfull), n & 1);
                if (!ok) break;
                tc_fence_after();
                tc_copy_scales(tmem + kTmemSfb, sf_desc);
#pragma unroll 1
                for (int c = 0; c < cpt; ++c) {
                    int slot, code = c == 0 ? 0 : c - p.pe;
                    uint32_t parity;
                    if (opaque(p.twin)) {                  // the last codes first: their slot frees two loads one after the other
                        if (c == 4) break;
                        code = (c + 3) & 3;
                        slot = static_cast<int>(n & 1) * 4 + (0x1320 >> 4 * code & 3);
                    } else {
                        ch.take(p, c, slot, parity);
                        if (c == 1 && p.pe) continue;
                    }
                    if (code >= p.nblk) continue;
                    if (!bounds_ok(slot >= 0 && slot < p.slots && code * kHeads + (kPair ? HP : 2 * HP) <= kTmemS)) continue;
                    tc_mma_scaled<kPair>(tmem + code * kHeads, desc_low(smem_u32(ring) + slot * kChunkBytes, kChunkBytes), p_low,
                                         idesc_o(kPair ? HP : 2 * HP), tmem + kTmemSfa, tmem + kTmemSfb, i > 0);
                    tc_commit(smem_u32(&empty[slot]));
                }
                tc_commit(smem_u32(pempty));
            }
        }
        if (!ok) {
            tc_commit(smem_u32(&drain[1]));
            wait_drain(smem_u32(&drain[1]), 0, tmo);
        }
    }
    } else {
        // ------------------------------------- softmax, splitting q, output
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
        const int quad = warp & 3, sw = warp - kSoftWarp0, half = sw >> 2;
        const uint32_t tl = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        const int st = threadIdx.x - kSoftWarp0 * 32;      // 0..255
        const float kNegInf = __int_as_float(0xff800000);
        const int tok = quad * 32 + lane;                  // this thread's token of a tile
        const int DV = p.nblk * 128;
        float* bc = bc_s + sw * 2 * kPer;
        uint32_t n = 0, nq = 0;
        bool ok = true;                                    // false: only the barriers are kept up

        // Job by job: the output of the one before, the tiles of the next.
        Run next = run;
        bool started = false;
        float2 l[kPer / 2], lr[kPer / 2];                  // per head, this token's share of the sums of p: unrounded, rounded
        float M = 0.f;                                     // of head h0 + lane: what O and the sums are relative to (log2)
#pragma unroll 1
        while (true) {
            // The next job with tiles and rows.
            bool more = false;
#pragma unroll 1
            for (; next.next(p, g); next.advance()) {
                more = next.live();
                if (more) break;
                if (p.prefix_len || next.len > 0) continue;   // no part; the join knows
                // An empty request: zeros, and the logarithm of an empty sum.
                const int b = next.j - p.NP;
#pragma unroll 1
                for (int e = st; e < (DV / 8) << p.hg; e += kSoftThreads) {
                    const int h = (g << p.hg) + e / (DV / 8), c = e % (DV / 8);
                    if (h < p.H && bounds_ok(b >= 0 && b < p.B))
                        *reinterpret_cast<uint4*>(p.out + b * p.ldo_b + h * p.ldo_h + c * 8) = make_uint4(0, 0, 0, 0);
                }
                if (p.lse && st < 1 << p.hg && (g << p.hg) + st < p.H) p.lse[b * p.ldl_b + (g << p.hg) + st] = kNegInf;
            }
            if (started) {
                // ---- output of the job (or of this worker's part of it)
                const int b = run.j - p.NP, h0 = half * hpp;
                const bool whole = !p.prefix_len && run.t0 == 0 && run.n == run.tiles, mine = lane < hpp && h0 + lane < run.count;
                // Sums over the tokens: lane k gets head h0 + k's.
                float v[kPer], u[kPer];
#pragma unroll
                for (int k = 0; k < kPer / 2; ++k) {
                    v[2 * k] = l[k].x; v[2 * k + 1] = l[k].y;
                    u[2 * k] = lr[k].x; u[2 * k + 1] = lr[k].y;
                }
#pragma unroll
                for (int o = kPer / 2; o > 0; o >>= 1)
#pragma unroll
                    for (int k = 0; k < o; ++k) {
                        const bool odd = lane & o;
                        const float a = odd ? v[k] : v[k + o], c = odd ? u[k] : u[k + o];
                        v[k] = (odd ? v[k + o] : v[k]) + __shfl_xor_sync(0xffffffffu, a, o);
                        u[k] = (odd ? u[k + o] : u[k]) + __shfl_xor_sync(0xffffffffu, c, o);
                    }
                bc[lane] = v[0];
                bc[kPer + lane] = u[0];
                half_sync_or(half, false);
                late_self_test(p.inject, quad == 3);
                float ls = 0.f, lrs = 0.f;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    ls += bc_s[(half * 4 + q) * 2 * kPer + lane];
                    lrs += bc_s[(half * 4 + q) * 2 * kPer + kPer + lane];
                }
                // The next job's first tile writes T into bc in front of its own
                // barrier, and S^T of that tile waits for none of these reads.
                half_sync_or(half, false);
                // A part's weights add up to its unrounded sum, which the join divides by.
                if (mine) al_s[h0 + lane] = lrs > 0.f || lrs != lrs ? __fdividef(whole ? 1.0f : ls, lrs) : 0.f;
                __syncwarp();                                  // the same from each of the half's four warps
                ok = ok && wait_uniform(smem_u32(pempty), (n & 1) ^ 1);
                tc_fence_after();
                if (ok && whole) {
                    // 32 values x 32 heads at a time, through 2 KB of p's buffers
                    // for each warp: stmatrix turns the fragments into rows of 32
                    // values (16-byte chunks, chunk ^ (row / 2) % 4), which leave as
                    // 16-byte stores, 64 bytes of each of eight heads at once.
                    const uint32_t stage = smem_u32(p_s) + sw * 2048;
                    const int col0 = 2 * (lane & 3), hl0 = lane >> 2, head0 = (g << p.hg) + h0;
                    const int last = min(run.count - h0, hpp);
#pragma unroll 1
                    for (int blk = 0; blk < p.nblk; ++blk) {
                        uint32_t x[kBands][2][8];
                        const uint32_t src = tl + blk * kHeads + h0;
#pragma unroll
                        for (int k = 0; k < kBands; ++k)
#pragma unroll
                            for (int u = 0; u < 2; ++u) tmem_ld_frag16(src + 16 * k + (u * 16u << 16), x[k][u]);
                        if (kLow) {
                            uint32_t y[2][8];              // (a single band)
#pragma unroll
                            for (int u = 0; u < 2; ++u) tmem_ld_frag16(src + kLow + (u * 16u << 16), y[u]);
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                tmem_ld8_wait(x[0][u]);
                                tmem_ld8_wait(y[u]);
#pragma unroll
                                for (int e = 0; e < 8; ++e) x[0][u][e] = __float_as_uint(__uint_as_float(x[0][u][e]) + __uint_as_float(y[u][e]));
                            }
                        }
#pragma unroll
                        for (int k = 0; k < kBands; ++k) {
                            if (!kLow) {
                                tmem_ld8_wait(x[k][0]);
                                tmem_ld8_wait(x[k][1]);
                            }
#pragma unroll
                            for (int q = 0; q < 2; ++q) {  // eight heads; those past this half's are not stored
                                const float2 f = *reinterpret_cast<const float2*>(al_s + min(h0 + k * 16 + q * 8 + col0, kHeads - 2));
                                uint32_t v[4];
#pragma unroll
                                for (int d = 0; d < 4; ++d)    // eight values
                                    v[d] = pack_bf16(__uint_as_float(x[k][d >> 1][q * 4 + (d & 1) * 2]) * f.x,
                                                     __uint_as_float(x[k][d >> 1][q * 4 + (d & 1) * 2 + 1]) * f.y);
                                const int hl = k * 16 + q * 8 + (lane & 7), d = lane >> 3;
                                stmatrix_x4_trans(stage + hl * 64 + ((d ^ ((hl >> 1) & 3)) << 4), v[0], v[1], v[2], v[3]);
                            }
                        }
                        __syncwarp();
                        __nv_bfloat16* o = p.out + b * p.ldo_b + blk * 128 + quad * 32 + (lane & 3) * 8;
                        uint4 v[2 * kBands];
#pragma unroll
                        for (int j = 0; j < 2 * kBands; ++j)
                            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                         : "=r"(v[j].x), "=r"(v[j].y), "=r"(v[j].z), "=r"(v[j].w)
                                         : "r"(stage + (j * 8 + hl0) * 64 + (((lane & 3) ^ ((hl0 >> 1) & 3)) << 4))
                                         : "memory");
#pragma unroll
                        for (int j = 0; j < 2 * kBands; ++j)
                            if (j * 8 + hl0 < last && bounds_ok(b >= 0 && b < p.B))
                                *reinterpret_cast<uint4*>(o + static_cast<int64_t>(head0 + j * 8 + hl0) * p.ldo_h) = v[j];
                        __syncwarp();
                    }
                } else if (ok) {
                    // A part, in the order the registers hold it: 512 bytes a store.
                    const int64_t slot = part_slot(p, w, run.j, run.j == j_first, g);
                    float4* o = reinterpret_cast<float4*>(p.part_o) + slot * p.nblk * 16 * 128 + quad * 32 + lane;
#pragma unroll 1
                    for (int k = 0; 4 * k < hpp && h0 + 4 * k < run.count; ++k) {
                        const float4 f = *reinterpret_cast<const float4*>(al_s + h0 + 4 * k);
                        uint32_t x[4][4], y[4][4];
#pragma unroll
                        for (int blk = 0; blk < 4; ++blk) {
                            if (blk >= p.nblk) break;
                            tmem_ld4_issue(tl + blk * kHeads + h0 + 4 * k, x[blk]);
                            if (kLow) tmem_ld4_issue(tl + blk * kHeads + kLow + h0 + 4 * k, y[blk]);
                        }
#pragma unroll
                        for (int blk = 0; blk < 4; ++blk) {
                            if (blk >= p.nblk) break;
                            tmem_ld4_wait(x[blk]);
                            if (kLow) {
                                tmem_ld4_wait(y[blk]);
#pragma unroll
                                for (int u = 0; u < 4; ++u) x[blk][u] = __float_as_uint(__uint_as_float(x[blk][u]) + __uint_as_float(y[blk][u]));
                            }
                            if (!bounds_ok(part_ok(p, slot) && (h0 >> 2) + k < kHeads / 4)) continue;
                            o[(blk * 16 + (h0 >> 2) + k) * 128] =
                                make_float4(__uint_as_float(x[blk][0]) * f.x, __uint_as_float(x[blk][1]) * f.y, __uint_as_float(x[blk][2]) * f.z,
                                            __uint_as_float(x[blk][3]) * f.w);
                        }
                    }
                    if (quad == 0 && mine && bounds_ok(part_ok(p, slot))) p.part_ml[slot * kHeads + h0 + lane] = make_float2(M, ls);
                }
                const int head = (g << p.hg) + h0 + lane;
                if (ok && whole && p.lse && quad == 0 && mine && head < p.H)
                    p.lse[b * p.ldl_b + head] = ls == 0.f ? kNegInf : (M + log2f(ls)) * kLn2;
                tc_fence_before();
            }
            if (!more) break;
            run = next;
            next.advance();
            started = true;
            const int h0 = half * hpp;                     // this warp's first head
            const bool mine = lane < hpp && h0 + lane < run.count;   // this lane has a head: h0 + lane
            const float* cq = cq_s + h0;
#pragma unroll
            for (int k = 0; k < kPer / 2; ++k) l[k] = lr[k] = make_float2(0.f, 0.f);
#pragma unroll 1
            for (int i = 0; i < run.n; ++i, ++n) {
                const int valid = min(kTile, run.len - (run.t0 + i) * kTile);
                const bool in = tok < valid;
                const uint32_t sb = smem_u32(&scfull[n & (kScaleSlots - 1)]), sp = (n / kScaleSlots) & 1;
                // Shared memory answers in hundreds of cycles while the products
                // read it, so what can be asked for early is, and as little as
                // possible lies between S^T and the product that waits for p s.
                const bool landed = mbar_test(sb, sp);
                ok = opaque(ok && wait_uniform(smem_u32(sfull), n & 1));
                if (i == 0) ok = opaque(ok && wait_uniform(smem_u32(qfull), nq & 1));   // the factors of the scores
                if (!__all_sync(0xffffffffu, landed)) ok = opaque(ok && wait_uniform(sb, sp));
                tc_fence_after();
                float2 z[kPer / 2];                        // log2 of p s, up to the reference; then x
                float lg;
                {
                    const float sj = ok && in ? sc_s[(n & (kScaleSlots - 1)) * kTile + tok] : 1.f;
                    lg = log2_fast(fmaxf(sj, kLeastScale));
                    const float2 s2 = make_float2(sj, sj), lg2 = make_float2(lg, lg), down = make_float2(0.03125f, 0.03125f);
#pragma unroll
                    for (int k = 0; k < kPer / 16; ++k) {
                        if (16 * k >= hpp) break;
                        uint32_t a[16], c[16];
                        tmem_ld16_issue(tl + kTmemS + h0 + 16 * k, a);
                        tmem_ld16_issue(tl + kTmemS + HP + h0 + 16 * k, c);
                        tmem_ld16_wait(a);
                        tmem_ld16_wait(c);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float4 f = *reinterpret_cast<const float4*>(cq + 16 * k + 4 * j);
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const int e = 4 * j + 2 * u;
                                const float2 s = fma2(make_float2(__uint_as_float(c[e]), __uint_as_float(c[e + 1])), down,
                                                      make_float2(__uint_as_float(a[e]), __uint_as_float(a[e + 1])));
                                z[8 * k + 2 * j + u] = fma2(s, mul2(u ? make_float2(f.z, f.w) : make_float2(f.x, f.y), s2), lg2);
                            }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(sempty));
                const bool pv_done = n == 0 || mbar_test(smem_u32(pempty), (n & 1) ^ 1);
                if (opaque(valid < kTile)) {
#pragma unroll
                    for (int k = 0; k < kPer / 2; ++k)
                        if (!in) z[k] = make_float2(kNothing, kNothing);
                }
                // T of each head: x = 2^(z - T) <= 256, the block's largest at
                // least 128.  (Rounded to a whole number by adding 1.5 2^23.)
                uint32_t hi[kPer / 4], lo[kPer / 4];       // four heads each
                __half2 sum[kPer / 2];                     // x as rounded
#pragma unroll
                for (int k = 0; k < kPer / 4; ++k) {
                    if (4 * k >= hpp) break;
                    float2 T[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float2 top = make_float2(redux_max(z[2 * k + j].x), redux_max(z[2 * k + j].y));
                        T[j] = add2(add2(add2(top, make_float2(-7.5f, -7.5f)), make_float2(0x1.8p23f, 0x1.8p23f)),
                                    make_float2(-0x1.8p23f, -0x1.8p23f));
                    }
                    if (lane == 0) *reinterpret_cast<float4*>(bc + 4 * k) = make_float4(T[0].x, T[0].y, T[1].x, T[1].y);
                    uint32_t a2[2], c2[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int e = 2 * k + j;
                        const float2 y = fma2(T[j], make_float2(-1.f, -1.f), z[e]);
                        z[e] = make_float2(exp2_fast(y.x), exp2_fast(y.y));
                        split2(z[e], a2[j], c2[j], sum[e]);
                    }
                    hi[k] = __byte_perm(a2[0], a2[1], 0x5410);
                    lo[k] = __byte_perm(c2[0], c2[1], 0x5410);
                }
                __syncwarp();
                const float top = mine ? bc[lane] : kNothing;  // head h0 + lane's
                // What O and the sums are relative to.
                bool raise = false;
                if (opaque(i == 0)) {
                    mx_s[sw * kPer + lane] = top;
                    soft_sync();
                } else {
                    raise = half_sync_or(half, top - M > kRaise);
                    if (raise) {
                        mx_s[sw * kPer + lane] = top;
                        half_sync_or(half, false);
                    }
                }
                if (opaque(i == 0 || raise)) {
                    const float* mx = mx_s + half * 4 * kPer + lane;
                    const float to = fmaxf(fmaxf(mx[0], mx[kPer]), fmaxf(mx[2 * kPer], mx[3 * kPer]));
                    if (i == 0) {
                        M = to;
                    } else {
                        // Rare: some block grew too far; O and the sums follow.
                        float alpha = 1.f;
                        if (mine && to - M > kRaise) {
                            alpha = exp2_fast(M - to);
                            M = to;
                        }
                        if (mine) al_s[h0 + lane] = alpha; // the same from each of the half's four warps
                        __syncwarp();
#pragma unroll
                        for (int k = 0; k < kPer / 2; ++k) {
                            if (2 * k >= hpp) break;
                            const float2 by = *reinterpret_cast<const float2*>(al_s + h0 + 2 * k);
                            l[k] = mul2(l[k], by);
                            lr[k] = mul2(lr[k], by);
                        }
                        ok = opaque(ok && wait_uniform(smem_u32(pempty), (n & 1) ^ 1));
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; ok && c < p.nblk * (kLow ? 2 : 1); ++c)
#pragma unroll 1
                            for (int k = 0; 4 * k < hpp; ++k) {
                                uint32_t r[4];
                                const uint32_t at = tl + (kLow ? (c >> 1) * kHeads + (c & 1) * kLow : c * kHeads) + h0 + 4 * k;
                                tmem_ld4(at, r);
#pragma unroll
                                for (int j = 0; j < 4; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * al_s[h0 + 4 * k + j]);
                                tmem_st4(at, r);
                            }
                        tmem_wait_st();
                    }
                }
                const int up = static_cast<int>(fmaxf(fminf(top - M, 127.f), -126.f));
                bc[kPer + lane] = __int_as_float((up + 127) << 23);
                if (!__all_sync(0xffffffffu, pv_done)) ok = opaque(ok && wait_uniform(smem_u32(pempty), (n & 1) ^ 1));
                if (opaque(ok)) {
                    // hi of the heads, then lo: in the same row of 64 bytes or in a
                    // buffer of its own.  A quarter of the warp's lanes fill all
                    // banks with 16 bytes each.
                    uint8_t* at = p_s + tok * 64;
                    const int swz = (tok >> 1) & 3, below = kPair ? kPBytes : 0, beside = kPair ? 0 : HP;
                    if (hpp % 16 == 0) {
#pragma unroll
                        for (int k = 0; k < kPer / 16; ++k) {
                            if (16 * k >= hpp) break;
                            const int v = (h0 >> 4) + k, u = v + (beside >> 4);
                            *reinterpret_cast<uint4*>(at + ((v ^ swz) << 4)) = make_uint4(hi[4 * k], hi[4 * k + 1], hi[4 * k + 2], hi[4 * k + 3]);
                            *reinterpret_cast<uint4*>(at + below + ((u ^ swz) << 4)) =
                                make_uint4(lo[4 * k], lo[4 * k + 1], lo[4 * k + 2], lo[4 * k + 3]);
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < kPer / 4; ++k) {
                            if (4 * k >= hpp) break;
                            const int v = h0 + 4 * k, u = v + beside;   // four heads: four bytes
                            *reinterpret_cast<uint32_t*>(at + (((v >> 4) ^ swz) << 4) + (v & 12)) = hi[k];
                            *reinterpret_cast<uint32_t*>(at + below + (((u >> 4) ^ swz) << 4) + (u & 12)) = lo[k];
                        }
                    }
                    if (mine) {
                        const int h = h0 + lane, u = kPair ? h + 64 : h + HP;   // rows of the scales
                        sf_s[(h & 31) * 16 + (h >> 5) * 4 + quad] = static_cast<uint8_t>(up + 127);
                        sf_s[(u & 31) * 16 + (u >> 5) * 4 + quad] = static_cast<uint8_t>(max(up + 127 - 5, 0));
                    }
                    if (opaque(valid < kTile)) {
                        // Rows past the length hold whatever the page or the
                        // buffer held: 0 * NaN would reach O, so their codes become 0.
                        // (S^T of this tile is done, so its chunks have landed.)
#pragma unroll 1
                        for (int c = 0; c < cpt; ++c) {
                            if ((c == 1 && p.pe) || c - (c > 0 ? p.pe : 0) >= p.nblk) continue;
                            const int slot = Chunks::slot_of(p, n, c);
                            if (!bounds_ok(slot >= 0 && slot < p.slots)) continue;
#pragma unroll 1
                            for (int r = valid + (st >> 3); r < kTile; r += kSoftThreads / 8)
                                *reinterpret_cast<uint4*>(ring + slot * kChunkBytes + r * 128 + (st & 7) * 16) = make_uint4(0, 0, 0, 0);
                        }
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(pfull));
                // The sums, while the product runs.  Tokens whose values are far
                // below their neighbours' count unrounded.
                const bool tiny = lg < redux_max(in ? lg : -1.0e30f) - 8.f;
                const float inv_s = exp2_fast(-lg);
#pragma unroll
                for (int k = 0; k < kPer / 4; ++k) {
                    if (4 * k >= hpp) break;
                    const float4 f = *reinterpret_cast<const float4*>(bc + kPer + 4 * k);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int e = 2 * k + j;
                        const float2 w = mul2(j ? make_float2(f.z, f.w) : make_float2(f.x, f.y), make_float2(inv_s, inv_s));
                        float2 r = __half22float2(sum[e]);
                        r = make_float2(tiny ? z[e].x : r.x, tiny ? z[e].y : r.y);
                        l[e] = fma2(z[e], w, l[e]);
                        lr[e] = fma2(r, w, lr[e]);
                    }
                }
                __syncwarp();                              // bc is read
            }
            ++nq;
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
// Joins the parts of a job in the order of the tokens, the prefix's before the
// request's own:
//   out = sum_k 2^(m_k - M) o_k / sum_k 2^(m_k - M) l_k,  M = max_k m_k
// The parts of job j are those of the workers from the last one that begins at
// or before its first tile up to the last one that begins inside it.  Without a
// prefix only requests with two or more parts are joined (by_cut: found at the
// first cut inside them); with one, all of them.
// A part's value is read as it lies: 16 bytes are four heads of one value.  An
// item is four heads of one block of 128 values: SHARE = 1 gives it to one
// warp, for few parts; SHARE = 8 gives it to the eight warps of a CTA, which
// take the parts in turn, for jobs that many workers share.  A warp has AHEAD
// parts on their way: the kernel takes as long as its trips to memory.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;

template <bool PREFIX, int SHARE, int AHEAD, int CTAS>
__global__ void __launch_bounds__(kJoinThreads, CTAS)
latent_attention_fp8_join_kernel(const Params p, const int by_cut) {
    grid_dependency_wait();
    allow_dependent_launch();
    bounds_self_test(p.inject);
    constexpr unsigned kAll = 0xffffffffu;
    __shared__ int2 meta_s[kJoinThreads];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = threadIdx.x;
    const float kNegInf = __int_as_float(0xff800000);
    const int quads = (p.H + 3) / 4, items = quads * p.nblk;
    const int per = (items + 8 / SHARE - 1) / (8 / SHARE); // CTAs of a request
    const int what = blockIdx.x / per;

    static_assert(kMaxCtas <= kJoinThreads, "one thread per worker");
    const int2 me = t < p.W ? p.meta[t] : make_int2(0x7fffffff, 0);
    meta_s[t] = me;
    __syncthreads();
    int b = what;
    if (by_cut) {                                          // the request of the cut before worker what + 1, at its first cut
        const int2 cut = meta_s[what + 1];
        b = cut.x - p.NP;
        if (b >= p.B || cut.y == 0 || (meta_s[what].x == cut.x && meta_s[what].y > 0)) return;
    }
    // First worker and number of parts of a job.
    auto parts_of = [&](int j, int& w0) {
        const int before = __syncthreads_count(me.x < j || (me.x == j && me.y == 0));
        const int upto = __syncthreads_count(me.x <= j);
        w0 = before - 1;
        return upto - before + 1;
    };
    int w1 = 0, w2, n1 = 0;
    const int sub = static_cast<int>(blockIdx.x) - what * per;
    const int item = SHARE == 1 ? sub * 8 + warp : sub;
    const int hq = min(item, items - 1) / p.nblk, blk = item - hq * p.nblk;
    int g1 = 0, hl1 = 0, j1 = 0;
    const int j2 = p.NP + b, g2 = hq * 4 >> p.hg, hl2 = hq * 4 - (g2 << p.hg);
    int n2 = parts_of(j2, w2);
    if (PREFIX) {
        if (clamp_len(p.cap, p.seq_lens[b]) == 0) n2 = 0;  // an empty request leaves none
        if (clamp_len(p.prefix_cap, *p.prefix_len) > 0) {
            // The rows of four heads lie in one group; a CTA's items may lie in two
            // jobs, so each warp finds its own.
            const int r = b * p.HR + hq * 4, rg = r >> p.hg;
            j1 = rg / p.G;
            g1 = rg - j1 * p.G;
            hl1 = r - (rg << p.hg);
            int before = 0, upto = 0;
            for (int k = lane; k < p.W; k += 32) {
                const int2 m = meta_s[k];
                before += m.x < j1 || (m.x == j1 && m.y == 0);
                upto += m.x <= j1;
            }
            before = __reduce_add_sync(kAll, before);
            upto = __reduce_add_sync(kAll, upto);
            w1 = before - 1;
            n1 = upto - before + 1;
        }
    } else if (n2 < 2) {
        return;
    }
    if (item >= items) return;                             // SHARE = 8: the whole CTA
    const int np = n1 + n2;
    auto slot_of = [&](int k) -> int64_t {                 // part k's place in the workspace
        if (!PREFIX) return part_slot(p, w2 + k, j2, k > 0 || meta_s[w2].x == j2, g2);
        const bool front = k < n1;
        return part_slot(p, front ? w1 + k : w2 + k - n1, front ? j1 : j2, false, front ? g1 : g2);
    };
    auto row_of = [&](int k) { return PREFIX && k < n1 ? hl1 : hl2; };
    // Values 2 lane, + 1, 2 lane + 64, + 1 of the block.
    auto load = [&](int k, float4 (&o)[4]) {
        if (!bounds_ok(part_ok(p, slot_of(k)) && row_of(k) < kHeads && blk < p.nblk)) return;
        const float4* src = reinterpret_cast<const float4*>(p.part_o) + ((slot_of(k) * p.nblk + blk) * 16 + row_of(k) / 4) * 128 + 2 * lane;
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
        for (int u = 0; u < AHEAD; ++u)                    // on their way while the factors are formed
            if (u < cnt) load(k0 + (c + u) * SHARE, o[u]);
        float f[4] = {kNegInf, kNegInf, kNegInf, kNegInf}, l[4] = {0.f, 0.f, 0.f, 0.f};
        if (lane < cnt && bounds_ok(part_ok(p, slot_of(k0 + (c + lane) * SHARE)) && row_of(k0 + (c + lane) * SHARE) + 4 <= kHeads)) {
            const int k = k0 + (c + lane) * SHARE;
            const float4* ml = reinterpret_cast<const float4*>(p.part_ml + slot_of(k) * kHeads + row_of(k));
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
        // The warps' results, merged in the order of the warps.
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

// The cache as [page][group of 8 tokens][chunk][token][128 bytes]: one copy
// brings one chunk of `rows` tokens (whole groups) of one page.
bool make_cache_map(CUtensorMap* m, const void* cache, int64_t pages, int64_t page_size, int64_t chunks, int64_t ld_page,
                    int64_t ld_row, int rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[5] = {128, 8, static_cast<cuuint64_t>(chunks), static_cast<cuuint64_t>(page_size / 8),
                                static_cast<cuuint64_t>(pages)};
    const cuuint64_t strides[4] = {static_cast<cuuint64_t>(ld_row), 128, static_cast<cuuint64_t>(ld_row * 8),
                                   static_cast<cuuint64_t>(ld_page)};
    const cuuint32_t box[5] = {128, 8, 1, static_cast<cuuint32_t>(rows / 8), 1};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void*>(cache), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t tiles_for(int64_t cap) { return cap > kTile ? (cap + kTile - 1) / kTile : 1; }

// What a call comes to before anything is known about the lengths.
struct Shape {
    int64_t B, H, K, P, DV, width, page_size;
    bool prefix;
    int64_t prefix_width;
};
struct Plan {
    int64_t hg, G, HR, R, NP, W, parts, rows, images, image;
};
Plan plan_for(const Shape& s, int64_t ctas, int hg) {
    Plan x{};
    const int64_t heads = 1 << hg;
    x.hg = hg;
    x.G = (s.H + heads - 1) / heads;
    x.HR = (s.H + 3) / 4 * 4;
    int64_t tiles = 0;
    if (s.prefix && s.prefix_width > 0) {
        x.R = s.B * x.HR;
        x.NP = ((x.R + heads - 1) / heads + x.G - 1) / x.G;
        tiles = x.NP * tiles_for(s.prefix_width * s.page_size);
    }
    // Workers: bounded by the device and by the most tiles that the tables can hold.
    const int64_t per = tiles_for(s.width * s.page_size);
    x.W = ctas / x.G;
    if (x.W < 1) x.W = 1;
    if ((x.W - 1) / per + 1 > s.B) {                       // min(W, tiles + B * per) without overflow
        tiles += s.B * per;
        if (tiles < x.W) x.W = tiles;
    }
    x.parts = (s.prefix ? x.NP + s.B + x.W : 2 * x.W) * x.G;
    const int64_t most = x.NP ? x.R : s.H;                 // rows that a CTA can get
    x.rows = most < heads ? (most + 15) / 16 * 16 : heads;
    x.images = (s.B + x.NP) * x.G;
    x.image = (2 * s.K / 128 + (s.P ? 1 : 0)) * x.rows * 128 + kHeads * 4;
    return x;
}

// Heads of a group (rows of a CTA): 64, whose products cost the least a head, or
// fewer while that gives every job a CTA of its own and few tiles: a tile of 16
// heads takes two thirds of the time of one of 64, and its output or part a
// quarter.  By what the tables can hold, which bounds the lengths; where they hold
// far more (131072 tokens each) the short requests below get 64 heads: 1 x 701
// 17.0 us, 16 x 2000 40.5, 32 x 500 24.2, 4 behind 900 22.1.  Measured, us, with
// tables as wide as the requests, 16 / 32 / 64 heads (* the rule's choice) of
//   1 request of 701 tokens, 128 heads      15.4* / 16.4 / 19.0
//   1 x 4000, 128                           16.4* / 17.6 / 20.0
//   4 x 2400, 128                           24.6 / 22.6* / 24.6
//   16 x 2000, 128                          40.5 / 32.8* / 41.0
//   32 x 500, 128                           32.3 / 20.5* / 24.1
//   64 x 500, 128 (256 jobs of 32 heads)    51.3 / 36.4 / 27.2*
//   1 x 64000, 128 (2000 tiles of 32)       62.0 / 41.4 / 36.9*
//   4 behind a prefix of 900, 128           19.5* / 20.0 / 22.6
//   8 behind a prefix of 2000, 128          30.7 / 24.8* / 30.0
Plan plan_of(const Shape& s, int64_t ctas) {
    for (int hg = 4; hg < 6; ++hg) {
        const Plan x = plan_for(s, ctas, hg);
        const int64_t jobs = (x.NP + s.B) * x.G;
        const int64_t tiles = (x.NP * tiles_for(s.prefix_width * s.page_size) + s.B * tiles_for(s.width * s.page_size)) * x.G;
        if (jobs <= ctas && tiles <= (hg == 4 ? 2 : 8) * ctas) return x;
    }
    return plan_for(s, ctas, 6);
}

struct Layout {
    int64_t meta, ml, o, images, total;                    // byte offsets of the workspace's parts
};
Layout workspace_layout(const Plan& x, int64_t DV) {
    Layout L;
    L.meta = 0;
    L.ml = ((x.W + 1) * 8 + 255) / 256 * 256;
    L.o = (L.ml + x.parts * kHeads * 8 + 255) / 256 * 256;
    L.images = L.o + x.parts * kHeads * DV * 4;
    L.total = L.images + x.images * x.image;
    return L;
}

dsnq_status check_sizes(const Shape& s) {
    if (s.B < 0 || s.H <= 0 || s.K <= 0 || s.P < 0 || s.DV <= 0 || s.width < 0 || s.prefix_width < 0 || s.page_size <= 0)
        return DSNQ_ERR_INVALID_ARG;
    if (s.DV > s.K) return DSNQ_ERR_INVALID_ARG;
    if (s.K % 128 || s.K > 512 || (s.P != 0 && s.P != 64) || s.DV % 128 || s.H > 1024 || s.B > DSNQ_MAX_REQUESTS || s.page_size % 8 ||
        s.page_size > (1 << 20) || s.width > 0x7fffffffLL || s.width * s.page_size > 0x7fffff00LL || s.prefix_width > 0x7fffffffLL ||
        s.prefix_width * s.page_size > 0x7fffff00LL)
        return DSNQ_ERR_UNSUPPORTED;
    return DSNQ_OK;
}

// What a call asks for: of the widest row, on the largest GPU (a smaller one may
// choose larger groups).
int64_t workspace_needed(Shape s) {
    s.K = 512;
    s.P = 64;
    int64_t most = 0;
    for (int hg = 4; hg <= 6; ++hg) {
        const int64_t n = workspace_layout(plan_for(s, kMaxCtas, hg), s.DV).total;
        if (hg >= plan_of(s, kMaxCtas).hg && n > most) most = n;
    }
    return most;
}
dsnq_status workspace_bytes_of(const Shape& s, int64_t* bytes) {
    const dsnq_status st = check_sizes(s);
    if (st != DSNQ_OK) return st;
    if (bytes) *bytes = s.B == 0 ? 0 : workspace_needed(s);
    return DSNQ_OK;
}

struct Tensors {
    const void* q;
    int64_t ldq_tok, ldq_head;
    const void* cache;
    int64_t num_pages, ld_page, ld_row;
    const float* scales;
    int64_t ld_scale;
    const int32_t *prefix_table, *prefix_len, *table;
    int64_t ld_table;
    const int32_t* seq_lens;
    float scale;
    void* out;
    int64_t ldo_tok, ldo_head;
    float* lse;
    int64_t ldl_tok;
    void* workspace;
    int64_t workspace_bytes;
};

dsnq_status attention(const Shape& z, const Tensors& t, cudaStream_t s) {
    dsnq_status st = check_sizes(z);
    if (st != DSNQ_OK) return st;
    if (t.num_pages < 1 || !(t.scale > 0.f && t.scale < 1.0e30f) || t.workspace_bytes < 0) return DSNQ_ERR_INVALID_ARG;
    // Strides of a tensor map are below 2^40 bytes (the cache's 8-row groups: 8 ld_row).
    if (t.num_pages > 0x7ffffffeLL || t.ld_row >= (1LL << 37) || t.ld_page >= (1LL << 40) || t.ld_scale >= (1LL << 38) ||
        t.ldq_tok >= (1LL << 39) || t.ldq_head >= (1LL << 39))
        return DSNQ_ERR_UNSUPPORTED;
    if (z.B == 0) return DSNQ_OK;
    if (!t.q || !t.out || !t.seq_lens || !t.workspace || !t.cache || !t.scales || (z.width && !t.table) ||
        (z.prefix && (!t.prefix_len || (z.prefix_width && !t.prefix_table))))
        return DSNQ_ERR_INVALID_ARG;
    const int64_t DK = z.K + z.P, row = z.K + 2 * z.P;
    if ((z.H > 1 && (t.ldq_head < DK || t.ldo_head < z.DV)) ||
        (z.B > 1 && (t.ldq_tok < DK || t.ldo_tok < z.DV || t.ld_table < z.width)) || (z.B > 1 && t.lse && t.ldl_tok < z.H) ||
        t.ld_row < row || t.ld_page < (z.page_size - 1) * t.ld_row + row || (t.num_pages > 1 && t.ld_scale < z.page_size))
        return DSNQ_ERR_INVALID_ARG;
    if (!aligned(t.q, 16) || t.ldq_tok % 8 || t.ldq_head % 8 || !aligned(t.cache, 16) || t.ld_page % 16 || t.ld_row % 16 ||
        !aligned(t.scales, 16) || t.ld_scale % 4 || !aligned(t.out, 16) || t.ldo_tok % 8 || t.ldo_head % 8 || !aligned(t.table, 4) ||
        !aligned(t.prefix_table, 4) || !aligned(t.prefix_len, 4) || !aligned(t.seq_lens, 4) || !aligned(t.lse, 4) ||
        !aligned(t.workspace, 16))
        return DSNQ_ERR_MISALIGNED;
    if (t.workspace_bytes < workspace_needed(z)) return DSNQ_ERR_INVALID_ARG;
    const int sms = device_sm_count();
    if (sms <= 0) {
        cudaGetLastError();
        return DSNQ_ERR_CUDA;
    }
    const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
    const Plan x = plan_of(z, ctas);
    Params p{};
    p.scales = t.scales; p.ld_scale = t.ld_scale;
    p.seq_lens = t.seq_lens;
    p.table = t.table; p.ld_table = t.ld_table;
    p.prefix_table = t.prefix_table;
    p.prefix_len = z.prefix ? t.prefix_len : nullptr;
    p.B = static_cast<int>(z.B); p.H = static_cast<int>(z.H); p.G = static_cast<int>(x.G); p.W = static_cast<int>(x.W);
    p.hg = static_cast<int>(x.hg);
    p.W_full = ctas > x.G ? static_cast<int>(ctas / x.G) : 1;
    p.HR = static_cast<int>(x.HR); p.R = static_cast<int>(x.R); p.NP = static_cast<int>(x.NP);
    p.width = static_cast<int>(z.width);
    p.prefix_width = static_cast<int>(z.prefix_width);
    p.page_size = static_cast<int>(z.page_size);
    p.num_pages = static_cast<int>(t.num_pages);
    p.cap = z.width * z.page_size;
    p.prefix_cap = z.prefix_width * z.page_size;
    p.box_rows = z.page_size % 128 == 0 ? 128 : z.page_size % 64 == 0 ? 64 : z.page_size % 32 == 0 ? 32 : z.page_size % 16 == 0 ? 16 : 8;
    p.cc = static_cast<int>(z.K / 128);
    p.pe = z.P ? 1 : 0;
    p.nblk = static_cast<int>(z.DV / 128);
    p.q_rows = static_cast<int>(x.rows);
    // Shared memory: q, p s, scales and barriers, and the rest for the rings, up
    // to the three tiles whose row scales have a place.
    const int64_t fixed = 1024 + static_cast<int64_t>(2 * p.cc + p.pe) * p.q_rows * 128 + 2 * kPBytes + kMiscBytes;
    const int cpt = p.cc + p.pe;
    p.slots = static_cast<int>((227 * 1024 - fixed) / kChunkBytes);
    if (p.slots > 3 * cpt) p.slots = 3 * cpt;
    if (p.slots > kMaxSlots) p.slots = kMaxSlots;
    p.twin = p.slots < 2 * cpt;                            // 512 codes, position columns, more than 32 heads
    if (p.twin && (cpt != 5 || p.slots < 8)) return DSNQ_ERR_UNSUPPORTED;
    if (p.twin) p.slots = 8;
    // The rings hold two tiles or more each.
    const int odd = cpt / 2, share_odd = p.slots * odd / cpt;
    p.odd_slots = share_odd > 2 * odd ? share_odd : 2 * odd;
    const size_t smem = static_cast<size_t>(fixed + p.slots * kChunkBytes);
    p.scale_log2 = t.scale * kLog2e;
    p.out = static_cast<__nv_bfloat16*>(t.out);
    p.ldo_b = t.ldo_tok; p.ldo_h = t.ldo_head;
    p.lse = t.lse; p.ldl_b = t.ldl_tok;
    const Layout lay = workspace_layout(x, z.DV);
    uint8_t* ws = static_cast<uint8_t*>(t.workspace);
    p.meta = reinterpret_cast<int2*>(ws + lay.meta);
    p.part_ml = reinterpret_cast<float2*>(ws + lay.ml);
    p.part_o = reinterpret_cast<float*>(ws + lay.o);
    p.images = ws + lay.images;
    p.image = static_cast<int>(x.image);
    const uint64_t limit = debug_wait_timeout_ns();
    p.timeout_ns = limit ? limit : kDefaultTimeoutNs;
    p.inject = debug_inject_flags();

    CUtensorMap mc;
    if (!make_cache_map(&mc, t.cache, t.num_pages, z.page_size, cpt, t.ld_page, t.ld_row, p.box_rows)) return DSNQ_ERR_CUDA;
    void (*kern)(CUtensorMap, Params) = p.q_rows <= 16   ? latent_attention_fp8_kernel<1>
                                        : p.q_rows <= 32 ? latent_attention_fp8_kernel<2>
                                        : p.q_rows <= 48 ? latent_attention_fp8_kernel<3>
                                                         : latent_attention_fp8_kernel<4>;
    if (!set_smem_attr(reinterpret_cast<const void*>(kern), smem)) return DSNQ_ERR_CUDA;
    const int64_t rows = z.B * z.H, per = kPrepareThreads / 32;
    st = launch_result(launch_kernel(prepare_kernel, dim3(static_cast<unsigned>(1 + (rows + per - 1) / per)), dim3(kPrepareThreads), 0, s,
                                     p, static_cast<const __nv_bfloat16*>(t.q), t.ldq_tok, t.ldq_head));
    if (st != DSNQ_OK) return st;
    st = launch_result(launch_kernel(kern, dim3(static_cast<unsigned>(p.W * p.G)), dim3(kThreads), smem, s, mc, p));
    if (st != DSNQ_OK || (p.W == 1 && !z.prefix)) return st;
    // Few jobs: a request has many parts, so a CTA joins each item.  Many: a
    // warp does, and without a prefix no more requests can be split than there
    // are cuts.  While all CTAs find room at once, each keeps more parts on
    // their way (registers, so fewer CTAs on an SM).
    const int64_t items = (z.H + 3) / 4 * p.nblk, jobs = x.NP + z.B;
    const int by_cut = !z.prefix && z.B > p.W - 1;
    const int64_t targets = by_cut ? p.W - 1 : z.B;
    const bool share = p.W >= kManyParts * jobs;
    const int64_t grid = targets * (share ? items : (items + 7) / 8);
    void (*join)(Params, int);
    if (z.prefix) {
        if (share) join = p.W > 16 * jobs && grid <= sms ? latent_attention_fp8_join_kernel<true, 8, 5, 1>
                                                         : latent_attention_fp8_join_kernel<true, 8, 2, 2>;
        else join = grid <= 3 * sms ? latent_attention_fp8_join_kernel<true, 1, 4, 1> : latent_attention_fp8_join_kernel<true, 1, 2, 2>;
    } else {
        if (share) join = p.W > 16 * jobs && grid <= sms ? latent_attention_fp8_join_kernel<false, 8, 5, 1>
                                                         : latent_attention_fp8_join_kernel<false, 8, 2, 2>;
        else if (!by_cut && grid <= 3 * sms) join = latent_attention_fp8_join_kernel<false, 1, 4, 1>;
        else join = grid <= 5 * sms ? latent_attention_fp8_join_kernel<false, 1, 2, 2> : latent_attention_fp8_join_kernel<false, 1, 2, 3>;
    }
    return launch_result(launch_kernel(join, dim3(static_cast<unsigned>(grid)), dim3(kJoinThreads), 0, s, p, by_cut));
}

}  // namespace attn8

bool take_attention_fp8_words(cudaStream_t s, unsigned int* v) {
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

extern "C" dsnq_status dsnq_paged_latent_attention_fp8_workspace_bytes(int64_t B, int64_t H, int64_t DV, int64_t table_width,
                                                                       int64_t page_size, int64_t* bytes) {
    return attn8::workspace_bytes_of({B, H, 512, 64, DV, table_width, page_size, false, 0}, bytes);
}

extern "C" dsnq_status dsnq_shared_prefix_latent_attention_fp8_workspace_bytes(
    int64_t B, int64_t H, int64_t DV, int64_t prefix_width, int64_t table_width, int64_t page_size, int64_t* bytes) {
    return attn8::workspace_bytes_of({B, H, 512, 64, DV, table_width, page_size, true, prefix_width}, bytes);
}

extern "C" dsnq_status dsnq_paged_latent_attention_fp8(
    int64_t B, int64_t H, int64_t K, int64_t P, int64_t DV, const void* q, int64_t ldq_tok, int64_t ldq_head, const void* cache,
    int64_t num_pages, int64_t page_size, int64_t ld_page, int64_t ld_row, const float* scales, int64_t ld_scale,
    const int32_t* block_table, int64_t table_width, int64_t ld_table, const int32_t* seq_lens, float scale, void* out, int64_t ldo_tok,
    int64_t ldo_head, float* lse, int64_t ldl_tok, void* workspace, int64_t workspace_bytes, void* stream) {
    return attn8::attention({B, H, K, P, DV, table_width, page_size, false, 0},
                            {q, ldq_tok, ldq_head, cache, num_pages, ld_page, ld_row, scales, ld_scale, nullptr, nullptr, block_table,
                             ld_table, seq_lens, scale, out, ldo_tok, ldo_head, lse, ldl_tok, workspace, workspace_bytes},
                            static_cast<cudaStream_t>(stream));
}

extern "C" dsnq_status dsnq_shared_prefix_latent_attention_fp8(
    int64_t B, int64_t H, int64_t K, int64_t P, int64_t DV, const void* q, int64_t ldq_tok, int64_t ldq_head, const void* cache,
    int64_t num_pages, int64_t page_size, int64_t ld_page, int64_t ld_row, const float* scales, int64_t ld_scale,
    const int32_t* prefix_table, int64_t prefix_width, const int32_t* prefix_len, const int32_t* block_table, int64_t table_width,
    int64_t ld_table, const int32_t* seq_lens, float scale, void* out, int64_t ldo_tok, int64_t ldo_head, float* lse, int64_t ldl_tok,
    void* workspace, int64_t workspace_bytes, void* stream) {
    return attn8::attention({B, H, K, P, DV, table_width, page_size, true, prefix_width},
                            {q, ldq_tok, ldq_head, cache, num_pages, ld_page, ld_row, scales, ld_scale, prefix_table, prefix_len,
                             block_table, ld_table, seq_lens, scale, out, ldo_tok, ldo_head, lse, ldl_tok, workspace, workspace_bytes},
                            static_cast<cudaStream_t>(stream));
}

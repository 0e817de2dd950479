// The steps between the pre-projection and the attention of a decode step:
// block tables and slots from request lengths, per-head RMSNorm with rotary
// positions, and the write of normalized, rotated latent rows into the paged
// cache, in bf16 or in 8 bits, with the way back from 8 bits.
//
// Rotary positions: the pair (a, b) of frequency i at position p becomes
//   (a cos t - b sin t, b cos t + a sin t) * rope_scale,   t = p * inv_freq[i].
// At position 10^6 an fp32 product p * inv_freq is off by up to 0.06 rad.
// Positions are whole, so only the fraction of a turn that one position adds
// matters: it is taken from inv_freq once, as a 64-bit fixed-point number;
// times the position modulo 2^64 it is the fraction of a turn at that position
// (off by 2^-64 per position), and only that goes to fp32 (sincospif).  The
// table of a token's angles is formed once per CTA or warp, in shared memory,
// and used for all its heads.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "debug_check.cuh"
#include "dsnq_internal.h"
#include "group_quant.cuh"
#include "tensor_host.h"

namespace dsnq {
namespace {

__device__ unsigned int g_rope_status;   // kStatusBounds: a slot outside the cache was given

constexpr int kChunk = 8;                // bf16 per 16-byte chunk
constexpr int kMaxRope = 256;            // rotated columns
constexpr int kMaxWidth = 1024;          // columns of a head or cache row

__device__ __forceinline__ uint4 pack8(const float2 (&f)[4]) {
    uint4 v;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[i].x, f[i].y);
    return v;
}

struct Rope {
    const int64_t* positions;   // [M]
    const double* inv_freq;     // [dim / 2]
    int off, dim;               // rotated columns [off, off + dim)
    int half;                   // pairs (i, i + dim/2) instead of (2i, 2i + 1)
    float scale;                // factor of cos and sin
    float sign;                 // -1 rotates back
};

// The turns that one position adds, modulo 1, as a 64-bit fraction: the
// frequency's 53-bit mantissa times round(2^66 / (2 pi)), shifted by its
// exponent.  In whole numbers, since the fp64 units are few (in fp64 it was a
// seventh of the time of a prompt's cache write: 8191 rows in 6.9 us, now 6.0).
__device__ __forceinline__ uint64_t turn_step(double inv_freq) {
    constexpr uint64_t kTurn = 11743562013128004906ull;
    const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(inv_freq));
    const int exp = static_cast<int>(bits >> 52) & 0x7ff;
    if (exp == 0) return 0;                        // below 2^-1022
    const uint64_t mant = (bits & 0xfffffffffffffull) | 0x10000000000000ull;
    const uint64_t hi = __umul64hi(mant, kTurn), lo = mant * kTurn;
    const int shift = 54 - (exp - 1023);           // turns * 2^64 = (hi:lo) >> shift
    const uint64_t f = shift >= 128 ? 0 : shift >= 64 ? hi >> (shift - 64) : shift > 0 ? (hi << (64 - shift)) | (lo >> shift)
                       : shift > -64 ? lo << -shift : 0;
    return bits >> 63 ? 0 - f : f;
}

// (cos, sin) * scale at position pos of the frequency with that step.
__device__ __forceinline__ float2 rope_angle(const Rope& r, uint64_t step, int64_t pos) {
    const int64_t turn = static_cast<int64_t>(step * static_cast<uint64_t>(pos));   // in [-1/2, 1/2) turns
    float s, c;
    sincospif(__ll2float_rn(turn) * 0x1p-63f, &s, &c);
    return make_float2(c * r.scale, s * (r.scale * r.sign));
}

// The values of a chunk whose first column is `q` of the rotated range, given
// its own values x and, for the half layout, its partner chunk's values y.
template <bool HALF>
__device__ __forceinline__ void rotate_chunk(const Rope& r, const float2* cs, int q, float2 (&x)[4],
                                             const float2 (&y)[4]) {
    if (!HALF) {
        const float2* t = cs + (q >> 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 a = x[i], w = t[i];
            x[i] = make_float2(a.x * w.x - a.y * w.y, a.y * w.x + a.x * w.y);
        }
        return;
    }
    const int hd = r.dim >> 1;
    const bool low = q < hd;                       // first members of the pairs
    const float2* t = cs + (low ? q : q - hd);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 w0 = t[2 * i], w1 = t[2 * i + 1];
        const float s0 = low ? -w0.y : w0.y, s1 = low ? -w1.y : w1.y;
        x[i] = make_float2(x[i].x * w0.x + y[i].x * s0, x[i].y * w1.x + y[i].y * s1);
    }
}

__device__ __forceinline__ float sum_squares(const float2 (&x)[4]) {
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) s = fma2(x[i], x[i], s);
    return s.x + s.y;
}

__device__ __forceinline__ void scale_by(float2 (&x)[4], float r, const uint4& gamma_raw, bool weighted) {
    const float2 r2 = make_float2(r, r);
    float2 g[4];
    if (weighted) unpack8(gamma_raw, g);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] = mul2(x[i], r2);
        if (weighted) x[i] = mul2(x[i], g[i]);
    }
}

// --------------------------------------------------------- head norm + rotary
struct HeadArgs {
    const __nv_bfloat16* x;
    __nv_bfloat16* out;
    const __nv_bfloat16* gamma;          // NULL: no weight
    int64_t ldx_tok, ldx_head, ldo_tok, ldo_head;
    int64_t M;
    int H, D;
    int head_blocks, heads_per_block;    // CTAs per token, heads of each
    int norm;
    float d_f, eps;
    Rope rope;
    uint32_t inject;
};

constexpr int kHeadWarps = 8;

// LPR lanes hold one head's row (CPL chunks of 16 bytes each, chunk
// lane + j * LPR), so a warp works on 32 / LPR heads at once, and takes U such
// rows a step, all requested before the first is worked on.  A CTA takes heads
// of one token: its first dim/2 threads form the token's angles while the
// first rows are on their way.  Bound by HBM for many tokens: four CTAs per SM
// (64 registers) with 64 bytes a thread on their way keep 64 KB in flight.
// Measured: 4096 x 48 x 512 in 61.5 us (6.5 TB/s, 98% of the copy bandwidth;
// 86 us with one row a warp in flight), 1 x 128 x 192 in 2.1 us.
// HALF: pairs (i, i + dim/2), whose partner chunk is loaded beside the own one,
// in registers of its own: at 257 to 512 columns a warp then has one row in
// flight and an SM two CTAs, and 4096 x 48 x 512 take 108 us (3.7 TB/s).
template <int LPR, int CPL, bool HALF>
__global__ void __launch_bounds__(kHeadWarps * 32, CPL * (HALF ? 2 : 1) <= 2 ? 4 : CPL * (HALF ? 2 : 1) <= 4 ? 2 : 1)
head_norm_rope_kernel(const HeadArgs a) {
    grid_dependency_wait();
    allow_dependent_launch();
    bounds_self_test(a.inject);
    constexpr int kRows = 32 / LPR;      // heads per warp and row
    constexpr int U = CPL >= 4 ? 1 : 4 / (CPL * (HALF ? 2 : 1));
    __shared__ float2 cs[kMaxRope / 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane % LPR, sub = lane / LPR;
    const int64_t m = blockIdx.x / a.head_blocks;
    const int h0 = static_cast<int>(blockIdx.x - m * a.head_blocks) * a.heads_per_block;
    const int h1 = min(h0 + a.heads_per_block, a.H);
    const int chunks = a.D / kChunk;
    const int c_lo = a.rope.off / kChunk, c_n = a.rope.dim / kChunk;

    bool live[CPL], rot[CPL];
    int pcol[CPL];
    uint4 graw[CPL], pgraw[CPL];
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
        const int c = l + j * LPR, q = c - c_lo;
        live[j] = c < chunks;
        rot[j] = live[j] && c >= c_lo && c < c_lo + c_n;
        pcol[j] = (HALF && rot[j] ? (q < c_n / 2 ? c + c_n / 2 : c - c_n / 2) : c) * kChunk;
        graw[j] = pgraw[j] = make_uint4(0, 0, 0, 0);
        if (a.gamma && live[j]) {
            graw[j] = *reinterpret_cast<const uint4*>(a.gamma + c * kChunk);
            if (HALF) pgraw[j] = *reinterpret_cast<const uint4*>(a.gamma + pcol[j]);
        }
    }

    uint4 raw[U][CPL], praw[U][CPL];
    constexpr int kStep = kHeadWarps * kRows;              // heads of a row of the CTA
    auto load = [&](int h) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const __nv_bfloat16* row = a.x + m * a.ldx_tok + static_cast<int64_t>(h + u * kStep) * a.ldx_head;
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                raw[u][j] = praw[u][j] = make_uint4(0, 0, 0, 0);
                const int col = (l + j * LPR) * kChunk;
                if (h + u * kStep < h1 && live[j] && bounds_ok(m < a.M && h + u * kStep < a.H && col + kChunk <= a.D &&
                                                               pcol[j] + kChunk <= a.D)) {
                    raw[u][j] = *reinterpret_cast<const uint4*>(row + col);
                    if (HALF && rot[j]) praw[u][j] = *reinterpret_cast<const uint4*>(row + pcol[j]);
                }
            }
        }
    };

    load(h0 + warp * kRows + sub);
    if (threadIdx.x < static_cast<unsigned>(a.rope.dim / 2))
        cs[threadIdx.x] = rope_angle(a.rope, turn_step(a.rope.inv_freq[threadIdx.x]), a.rope.positions[m]);
    __syncthreads();

    for (int base = h0 + warp * kRows; base < h1; base += U * kStep) {
        // In place, a lane's partner chunk is another lane's output: every
        // lane has its rows in registers before any lane stores.
        __syncwarp();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = base + sub + u * kStep;
            float2 x[CPL][4], y[CPL][4];
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                unpack8(raw[u][j], x[j]);
                if (HALF) unpack8(praw[u][j], y[j]);
            }
            if (a.norm) {
                float ssq = 0.f;
#pragma unroll
                for (int j = 0; j < CPL; ++j) ssq += sum_squares(x[j]);
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) ssq += __shfl_xor_sync(0xffffffffu, ssq, o);
                const float r = 1.0f / sqrtf(ssq / a.d_f + a.eps);
#pragma unroll
                for (int j = 0; j < CPL; ++j) {
                    scale_by(x[j], r, graw[j], a.gamma != nullptr);
                    if (HALF) scale_by(y[j], r, pgraw[j], a.gamma != nullptr);
                }
            }
            if (h >= h1) continue;
            __nv_bfloat16* row = a.out + m * a.ldo_tok + static_cast<int64_t>(h) * a.ldo_head;
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                const int col = (l + j * LPR) * kChunk;
                if (!live[j] || !bounds_ok(m < a.M && h < a.H && col + kChunk <= a.D)) continue;
                if (rot[j]) rotate_chunk<HALF>(a.rope, cs, col - a.rope.off, x[j], y[j]);
                *reinterpret_cast<uint4*>(row + col) = pack8(x[j]);
            }
        }
        if (base + U * kStep < h1) load(base + U * kStep + sub);
    }
}

template <int LPR, int CPL>
dsnq_status launch_heads(HeadArgs& a, int sms, cudaStream_t s) {
    // Heads per CTA: one row of its warps when tokens are few (a decode row is
    // bound by latency), the whole token once the tokens alone fill the GPU.
    const int step = kHeadWarps * (32 / LPR);
    int64_t blocks = (a.H + step - 1) / step;
    const int64_t want = (8LL * sms + a.M - 1) / a.M;      // CTAs per token that give every SM eight
    if (blocks > want) blocks = want;
    const int64_t steps = ((a.H + step - 1) / step + blocks - 1) / blocks;
    a.heads_per_block = static_cast<int>(steps * step);
    a.head_blocks = (a.H + a.heads_per_block - 1) / a.heads_per_block;
    const int64_t grid = a.M * a.head_blocks;
    if (grid > 0x7fffffffLL) return DSNQ_ERR_UNSUPPORTED;
    return launch_result(launch_kernel(a.rope.half ? head_norm_rope_kernel<LPR, CPL, true> : head_norm_rope_kernel<LPR, CPL, false>,
                                       dim3(static_cast<unsigned>(grid)), dim3(kHeadWarps * 32), 0, s, a));
}

// --------------------------------------------------------- latent cache write
struct WriteArgs {
    const __nv_bfloat16* kv;
    const __nv_bfloat16* pe;
    const __nv_bfloat16* gamma;
    int64_t ldkv, ldpe;
    int64_t M;
    int K, W;                            // latent columns, row columns (latent + position part)
    const int64_t* slots;
    void* cache;                         // bf16, or bytes: K codes, then the position columns as bf16
    int64_t ld_page, ld_row, num_slots;  // strides in elements of the cache
    float* scales;                       // 8 bits: one a row
    int64_t ld_scale;
    int page_size;
    int norm;
    float k_f, eps;
    Rope rope;
    uint32_t inject;
};

constexpr int kWriteWarps = 4;
constexpr float kLeastScale = 0x1p-60f;  // of a row in 8 bits: an all-zero latent leaves its position columns finite

// One warp per row; lane l holds chunks l, l + 32, ... of the concatenated
// row.  The row is requested before its slot and position are known (they
// decide only where and by how much), so a row costs one trip to memory; four
// CTAs or more per SM hide it.  Measured: 8191 normalized rows of 576 in 6.0 us
// (3.1 TB/s: two and a quarter waves of one trip each), 32768 in 20.6 us, 32
// in 2.3 us; half pairs, whose partner chunks are loaded a second time, 7.9 us
// for 8191 rows and 28.5 for 32768.  For many rows the instructions bound it
// (~520 a row: the third of a row's three passes holds 8 chunks of 32, and the
// angles take a pass of their own).  Warps that stride over the rows and request
// the next one early need registers of a CTA per SM: 6.7 us at 8191 rows, 19.9
// at 32768.
//
// FP8: the row leaves as s (codes | position columns / s), s = max |latent| /
// 448 of the rotated row, in fp32; one scale a row, since the attention's
// products sum over the whole row before a factor can be applied, and e4m3
// keeps its 4 bits down to 2^-15 of the largest.  Codes are those of the IEEE
// quotient; the position columns' quotients are rounded once to bf16.
template <int CPL, bool HALF, bool FP8>
__global__ void __launch_bounds__(kWriteWarps * 32, HALF ? 4 : 6)
latent_cache_write_kernel(const WriteArgs a) {
    grid_dependency_wait();
    allow_dependent_launch();
    bounds_self_test(a.inject);
    __shared__ float2 cs_all[kWriteWarps][kMaxRope / 2];
    __shared__ uint64_t steps[kMaxRope / 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float2* cs = cs_all[warp];
    const int64_t m = static_cast<int64_t>(blockIdx.x) * kWriteWarps + warp;
    const bool in = m < a.M;
    const int c_lo = a.rope.off / kChunk, c_n = a.rope.dim / kChunk;
    bool live[CPL], rot[CPL];
    uint4 raw[CPL], praw[CPL], graw[CPL], pgraw[CPL];
    int pcol[CPL];
    const int64_t slot = in ? a.slots[m] : -1;
    const int64_t pos = in && a.rope.dim ? a.rope.positions[m] : 0;
    auto at = [&](int col) {
        return col < a.K ? a.kv + m * a.ldkv + col : a.pe + m * a.ldpe + (col - a.K);
    };
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
        const int c = lane + j * 32, col = c * kChunk, q = c - c_lo;
        live[j] = col < a.W;
        rot[j] = live[j] && c >= c_lo && c < c_lo + c_n;
        pcol[j] = HALF && rot[j] ? (q < c_n / 2 ? c + c_n / 2 : c - c_n / 2) * kChunk : col;
        raw[j] = praw[j] = graw[j] = pgraw[j] = make_uint4(0, 0, 0, 0);
        if (in && live[j] && bounds_ok(col + kChunk <= a.W && pcol[j] + kChunk <= a.W)) {
            raw[j] = *reinterpret_cast<const uint4*>(at(col));
            if (HALF && rot[j]) praw[j] = *reinterpret_cast<const uint4*>(at(pcol[j]));
            if (a.gamma && col < a.K) graw[j] = *reinterpret_cast<const uint4*>(a.gamma + col);
            if (HALF && a.gamma && pcol[j] < a.K) pgraw[j] = *reinterpret_cast<const uint4*>(a.gamma + pcol[j]);
        }
    }
    for (int i = threadIdx.x; i < a.rope.dim / 2; i += kWriteWarps * 32) steps[i] = turn_step(a.rope.inv_freq[i]);
    __syncthreads();
    if (slot < 0) return;                // a padded row, or none
    if (slot >= a.num_slots) {
        if (lane == 0) atomicOr(&g_rope_status, kStatusBounds);
        return;
    }
    for (int i = lane; i < a.rope.dim / 2; i += 32) cs[i] = rope_angle(a.rope, steps[i], pos);
    __syncwarp();
    float2 x[CPL][4];
#pragma unroll
    for (int j = 0; j < CPL; ++j) unpack8(raw[j], x[j]);
    float r = 1.f;
    if (a.norm) {
        float ssq = 0.f;
#pragma unroll
        for (int j = 0; j < CPL; ++j)
            if ((lane + j * 32) * kChunk < a.K) ssq += sum_squares(x[j]);
        r = 1.0f / sqrtf(warp_sum(ssq) / a.k_f + a.eps);
    }
    // Slots mostly fit 32 bits, whose division is a fraction of the 64-bit one.
    const int64_t page = slot <= 0xffffffffLL ? static_cast<uint32_t>(slot) / static_cast<uint32_t>(a.page_size) : slot / a.page_size;
    const int64_t in_page = slot - page * a.page_size, at_row = page * a.ld_page + in_page * a.ld_row;
    uint32_t top = 0;                    // largest magnitude among the latent columns, as bits (NaN above all)
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
        const int col = (lane + j * 32) * kChunk;
        if (!live[j] || !bounds_ok(col + kChunk <= a.W)) continue;
        if (a.norm && col < a.K) scale_by(x[j], r, graw[j], a.gamma != nullptr);
        if (rot[j]) {
            float2 y[4];
            if (HALF) {
                unpack8(praw[j], y);
                if (a.norm && pcol[j] < a.K) scale_by(y, r, pgraw[j], a.gamma != nullptr);
            }
            rotate_chunk<HALF>(a.rope, cs, col - a.rope.off, x[j], y);
        }
        if (!FP8) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.cache) + at_row + col) = pack8(x[j]);
        if (FP8 && col < a.K) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                top = max(top, max(__float_as_uint(x[j][i].x) & 0x7fffffffu, __float_as_uint(x[j][i].y) & 0x7fffffffu));
        }
    }
    if (!FP8) return;
    top = __reduce_max_sync(0xffffffffu, top);
    // A NaN or an infinity among the latent columns makes the row NaN.
    const float scale = top < 0x7f800000u ? fmaxf(group_scale(__uint_as_float(top)), kLeastScale) : __int_as_float(0x7fffffff);
    const GroupQuant gq = group_quant_from(scale, group_recip(scale));
    uint8_t* row = static_cast<uint8_t*>(a.cache) + at_row;
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
        const int col = (lane + j * 32) * kChunk;
        if (!live[j] || !bounds_ok(col + kChunk <= a.W)) continue;
        if (col < a.K) {
            bool ok;
            uint2 codes = quant8_bracket(x[j], gq, ok);
            if (!ok) codes = quant8_divide(x[j], scale);
            *reinterpret_cast<uint2*>(row + col) = codes;
        } else {
            // The same bracket: where both ends round to the same bf16, the
            // quotient does (below 2^-126, where the ends' own roundings show, to
            // 2^-149).  The division alone: 9.1 us for 8191 rows, now 8.6.
            float2 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = mul2(x[j][i], gq.ylo);
            uint4 pe = pack8(v);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = mul2(x[j][i], gq.yhi);
            const uint4 hi = pack8(v);
            if (pe.x != hi.x || pe.y != hi.y || pe.z != hi.z || pe.w != hi.w || gq.exact || scale != scale) {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = make_float2(__fdiv_rn(x[j][i].x, scale), __fdiv_rn(x[j][i].y, scale));
                pe = pack8(v);
            }
            *reinterpret_cast<uint4*>(row + a.K + (col - a.K) * 2) = pe;
        }
    }
    if (lane == 0) a.scales[page * a.ld_scale + in_page] = scale;
}

// -------------------------------------------------- latent cache read (8 bits)
struct ReadArgs {
    const uint8_t* cache;
    const float* scales;
    int64_t ld_page, ld_row, ld_scale;   // bytes, bytes, floats
    int num_pages, page_size;
    int K, W;                            // latent columns, columns of an output row
    const int32_t* table;
    int64_t ld_table;
    int B, width;
    const int32_t* row_starts;           // [B + 1]
    const int32_t* first;                // first token of each request, NULL: 0
    __nv_bfloat16* out;
    int64_t ldo;
    int64_t rows;
    uint32_t recip;                      // ceil(2^32 / chunks of a row)
    uint32_t inject;
};

constexpr int kReadThreads = 128;

// A CTA takes ROWS rows of the output: each of its first threads finds one row's
// request (the last that begins at or before it), page and scale, then all of
// them take the rows' chunks of 8 columns one after the other, U on their way at
// once.  Bound by HBM: 1.8 KB a row in and out.
template <int ROWS, int U>
__global__ void __launch_bounds__(kReadThreads)
latent_cache_read_fp8_kernel(const ReadArgs a) {
    grid_dependency_wait();
    allow_dependent_launch();
    bounds_self_test(a.inject);
    __shared__ int64_t at_s[ROWS];  // byte offset of the row in the cache, -1: zeros, -2: not written
    __shared__ float scale_s[ROWS];
    const int t = threadIdx.x;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * ROWS;
    if (t < ROWS) {
        const int64_t r = r0 + t;
        int64_t at = -2;
        float scale = 0.f;
        if (r < a.rows && r >= a.row_starts[0] && r < a.row_starts[a.B]) {
            int lo = 0, hi = a.B;        // row_starts[lo] <= r < row_starts[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (a.row_starts[mid] <= r) lo = mid;
                else hi = mid;
            }
            const int64_t tok = r - a.row_starts[lo] + (a.first ? a.first[lo] : 0);
            int id = -1;
            if (tok >= 0 && tok < static_cast<int64_t>(a.width) * a.page_size) id = a.table[lo * a.ld_table + tok / a.page_size];
            at = -1;
            if (id >= 0 && id < a.num_pages) {
                const int64_t in_page = tok % a.page_size;
                at = id * a.ld_page + in_page * a.ld_row;
                scale = a.scales[id * a.ld_scale + in_page];
            } else {
                atomicOr(&g_rope_status, kStatusBounds);
            }
        }
        at_s[t] = at;
        scale_s[t] = scale;
    }
    __syncthreads();
    const int chunks = a.W / kChunk, items = ROWS * chunks;
    for (int base = t; base < items; base += U * kReadThreads) {
        uint4 raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int e = base + u * kReadThreads;
            raw[u] = make_uint4(0, 0, 0, 0);
            if (e >= items) continue;
            const int row = static_cast<int>(__umulhi(static_cast<uint32_t>(e), a.recip)), col = (e - row * chunks) * kChunk;
            const int64_t at = at_s[row];
            if (at < 0 || !bounds_ok(col + kChunk <= a.W)) continue;
            if (col < a.K) {
                const uint2 v = *reinterpret_cast<const uint2*>(a.cache + at + col);
                raw[u].x = v.x;
                raw[u].y = v.y;
            } else {
                raw[u] = *reinterpret_cast<const uint4*>(a.cache + at + a.K + (col - a.K) * 2);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int e = base + u * kReadThreads;
            if (e >= items) continue;
            const int row = static_cast<int>(__umulhi(static_cast<uint32_t>(e), a.recip)), col = (e - row * chunks) * kChunk;
            if (at_s[row] == -2) continue;
            const float2 s = make_float2(scale_s[row], scale_s[row]);
            float2 f[4];
            if (col < a.K) {
                const uint32_t w[2] = {raw[u].x, raw[u].y};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i >> 1] >> (i & 1) * 16), __NV_E4M3);
                    f[i] = __half22float2(__half2(h));
                }
            } else {
                unpack8(raw[u], f);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = mul2(f[i], s);
            *reinterpret_cast<uint4*>(a.out + (r0 + row) * a.ldo + col) = pack8(f);
        }
    }
}

// ------------------------------------------------------- block tables, slots
struct ExtendArgs {
    int B, rows, page_size, width;       // requests, token rows, tokens per page, table columns
    int F;                               // free pages listed
    const int32_t* seq_lens;
    const int32_t* new_tokens;           // NULL: one each
    const int32_t* free_pages;
    int32_t* table;
    int64_t ld_table;
    int32_t* new_lens;
    int32_t* row_starts;
    int64_t* positions;
    int64_t* slots;
    int32_t* counts;
    uint32_t inject;
};

constexpr int kExtendThreads = 512;

// Exclusive sum of one value per thread over the CTA; *total gets the sum.
// One barrier: every thread adds the warps' sums before its own itself.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* warp_sums, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    int64_t before = inc - v, sum = 0;
#pragma unroll
    for (int i = 0; i < kExtendThreads / 32; ++i) {
        if (i < warp) before += warp_sums[i];
        sum += warp_sums[i];
    }
    *total = sum;
    return before;
}

// Every CTA forms the sums over all requests in shared memory (they are few
// and in L2; a second launch would cost more), then takes its strip of the
// requests (table, lengths) and of the token rows (positions, slots).  A
// row's page is read from the entries the request already held, or straight
// from the free list, never from an entry that another CTA writes.
// Bound by latency: two trips to memory (lengths, then page ids) and three
// barriers.  Measured: 48 requests 3.7 us, 1000 requests with 20000 rows 6.2 us.
__global__ void __launch_bounds__(kExtendThreads)
extend_tables_kernel(const ExtendArgs a) {
    grid_dependency_wait();
    allow_dependent_launch();
    bounds_self_test(a.inject);
    extern __shared__ int32_t sums[];
    int32_t* old_s = sums;               // [B] tokens so far
    int32_t* row_s = old_s + a.B;        // [B] first row, at most `rows`
    int32_t* page_s = row_s + a.B;       // [B] first free page, at most F
    int32_t* new_s = page_s + a.B;       // [B] tokens after the step
    __shared__ int64_t warp_rows[kExtendThreads / 32], warp_pages[kExtendThreads / 32];
    const int t = threadIdx.x, lane = t & 31;
    const int per = (a.B + kExtendThreads - 1) / kExtendThreads;
    const int b0 = min(t * per, a.B), b1 = min(b0 + per, a.B);
    const int64_t cap = static_cast<int64_t>(a.width) * a.page_size;     // below 2^31
    const uint32_t ps = a.page_size;
    auto pages_of = [&](int32_t len) -> int32_t { return static_cast<int32_t>((static_cast<uint32_t>(len) + ps - 1) / ps); };

    // Each thread works on its own requests' entries up to the last barrier.
    int64_t n = 0, total_rows, total_pages;
    for (int b = b0; b < b1; ++b) {
        const int32_t len = a.seq_lens[b], want = a.new_tokens ? a.new_tokens[b] : 1;
        old_s[b] = static_cast<int32_t>(len < 0 ? 0 : (len > cap ? cap : len));
        row_s[b] = want < 0 ? 0 : want;
        n += row_s[b];
    }
    int64_t start = block_scan(n, warp_rows, &total_rows), pages = 0;
    for (int b = b0; b < b1; ++b) {
        const int32_t want = row_s[b], len = old_s[b];
        row_s[b] = static_cast<int32_t>(start < a.rows ? start : a.rows);
        // The tokens that have a row and a place in the table.
        const int64_t fit = min(static_cast<int64_t>(min(want, a.rows - row_s[b])), cap - len);
        new_s[b] = static_cast<int32_t>(len + fit);
        page_s[b] = pages_of(new_s[b]) - pages_of(len);
        pages += page_s[b];
        start += want;
    }
    int64_t page = block_scan(pages, warp_pages, &total_pages);
    for (int b = b0; b < b1; ++b) {
        const int32_t need = page_s[b];
        page_s[b] = static_cast<int32_t>(page < a.F ? page : a.F);
        page += need;
        const int32_t got = min(need, a.F - page_s[b]);
        const int64_t backed = static_cast<int64_t>(pages_of(old_s[b]) + got) * ps;
        if (backed < new_s[b]) new_s[b] = static_cast<int32_t>(backed);
    }
    __syncthreads();
    const int live_rows = static_cast<int>(total_rows < a.rows ? total_rows : a.rows);

    if (blockIdx.x == 0 && t == 0) {
        a.row_starts[a.B] = live_rows;
        a.counts[0] = static_cast<int32_t>(total_pages < a.F ? total_pages : a.F);
        a.counts[1] = static_cast<int32_t>(total_pages < 0x7fffffff ? total_pages : 0x7fffffff);
    }

    // Token rows.
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * kExtendThreads + t; r < a.rows;
         r += static_cast<int64_t>(gridDim.x) * kExtendThreads) {
        const int row = static_cast<int>(r);
        int64_t pos = 0, slot = -1;
        if (row < live_rows) {
            // The last request whose first row is at most `row` (requests
            // without tokens share their successor's first row and lose).
            int lo = 0, hi = a.B;        // row_s[lo] <= row, row_s[hi] > row
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (row_s[mid] <= row) lo = mid;
                else hi = mid;
            }
            const int32_t len = old_s[lo];
            pos = static_cast<int64_t>(len) + (row - row_s[lo]);
            if (pos < new_s[lo]) {
                const int32_t p = static_cast<int32_t>(static_cast<uint32_t>(pos) / ps), k = p - pages_of(len);
                int32_t id = -1;
                if (bounds_ok(p < a.width && (k < 0 || page_s[lo] + k < a.F)))
                    id = k < 0 ? a.table[lo * a.ld_table + p] : a.free_pages[page_s[lo] + k];
                if (id >= 0) slot = static_cast<int64_t>(id) * ps + (pos - static_cast<int64_t>(p) * ps);
            }
        }
        a.positions[row] = pos;
        a.slots[row] = slot;
    }

    // Requests: one per thread; a request's new pages are stored by its whole
    // warp when they are many (a prompt), by its thread otherwise.
    for (int bw = blockIdx.x * kExtendThreads + (t & ~31); bw < a.B; bw += gridDim.x * kExtendThreads) {
        const int b = bw + lane;
        int got = 0, held = 0, from = 0;
        if (b < a.B) {
            held = pages_of(old_s[b]);
            from = page_s[b];
            got = pages_of(new_s[b]) - held;
            a.new_lens[b] = new_s[b];
            a.row_starts[b] = row_s[b];
            if (got <= 2)
                for (int k = 0; k < got; ++k)
                    if (bounds_ok(held + k < a.width && from + k < a.F))
                        a.table[b * a.ld_table + held + k] = a.free_pages[from + k];
        }
        unsigned many = __ballot_sync(0xffffffffu, got > 2);
        while (many) {
            const int src = __ffs(many) - 1;
            many &= many - 1;
            const int g = __shfl_sync(0xffffffffu, got, src), hd = __shfl_sync(0xffffffffu, held, src);
            const int f = __shfl_sync(0xffffffffu, from, src);
            for (int k = lane; k < g; k += 32)
                if (bounds_ok(hd + k < a.width && f + k < a.F))
                    a.table[(bw + src) * a.ld_table + hd + k] = a.free_pages[f + k];
        }
    }
}

dsnq_status check_rope(int64_t width, int64_t off, int64_t dim, int32_t layout, float scale) {
    if (dim < 0 || off < 0 || dim > width || off > width - dim) return DSNQ_ERR_INVALID_ARG;
    if (layout != DSNQ_ROPE_INTERLEAVED && layout != DSNQ_ROPE_HALF) return DSNQ_ERR_INVALID_ARG;
    if (!(scale > -3.0e38f && scale < 3.0e38f)) return DSNQ_ERR_INVALID_ARG;      // also rejects NaN
    if (dim % 16 || off % kChunk || dim > kMaxRope) return DSNQ_ERR_UNSUPPORTED;
    return DSNQ_OK;
}

}  // namespace

bool take_rope_cache_words(cudaStream_t s, unsigned int* v) {
    unsigned int w = 0, st = 0;
    const unsigned int zero = 0;
    if (!take_debug_word(s, &w)) return false;
    if (cudaMemcpyFromSymbolAsync(&st, g_rope_status, sizeof(st), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess ||
        cudaMemcpyToSymbolAsync(g_rope_status, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    *v = w | st;
    return true;
}

}  // namespace dsnq

using namespace dsnq;

extern "C" dsnq_status dsnq_head_rmsnorm_rope(
    int64_t M, int64_t H, int64_t D, const void* x, int64_t ldx_tok, int64_t ldx_head, int32_t normalize,
    const void* gamma, float eps, const int64_t* positions, const double* inv_freq, int64_t rope_offset,
    int64_t rope_dim, dsnq_rope_layout layout, float rope_scale, int32_t inverse, void* out, int64_t ldo_tok,
    int64_t ldo_head, void* stream) {
    if (M < 0 || H <= 0 || D <= 0) return DSNQ_ERR_INVALID_ARG;
    if (normalize && (!(eps >= 0.f) || eps > 3.0e38f)) return DSNQ_ERR_INVALID_ARG;   // also rejects NaN
    if (!normalize && gamma) return DSNQ_ERR_INVALID_ARG;
    if (D % kChunk || D > kMaxWidth || H > 65535 || M > 0x7fffffffLL) return DSNQ_ERR_UNSUPPORTED;
    dsnq_status st = check_rope(D, rope_offset, rope_dim, layout, rope_scale);
    if (st != DSNQ_OK) return st;
    if (M == 0) return DSNQ_OK;
    if (!x || !out || (rope_dim && (!positions || !inv_freq))) return DSNQ_ERR_INVALID_ARG;
    if ((H > 1 && (ldx_head < D || ldo_head < D)) || (M > 1 && (ldx_tok < D || ldo_tok < D))) return DSNQ_ERR_INVALID_ARG;
    // In place only row by row: with other strides a row would meet another's output.
    if (x == out && ((H > 1 && ldx_head != ldo_head) || (M > 1 && ldx_tok != ldo_tok))) return DSNQ_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(out, 16) || ldx_tok % kChunk || ldx_head % kChunk || ldo_tok % kChunk ||
        ldo_head % kChunk || (gamma && !aligned(gamma, 16)) || !aligned(positions, 8) || !aligned(inv_freq, 8))
        return DSNQ_ERR_MISALIGNED;
    const int sms = device_sm_count();
    if (sms <= 0) {
        cudaGetLastError();
        return DSNQ_ERR_CUDA;
    }
    HeadArgs a{};
    a.x = static_cast<const __nv_bfloat16*>(x);
    a.out = static_cast<__nv_bfloat16*>(out);
    a.gamma = static_cast<const __nv_bfloat16*>(gamma);
    a.ldx_tok = ldx_tok; a.ldx_head = ldx_head; a.ldo_tok = ldo_tok; a.ldo_head = ldo_head;
    a.M = M; a.H = static_cast<int>(H); a.D = static_cast<int>(D);
    a.norm = normalize ? 1 : 0;
    a.d_f = static_cast<float>(D); a.eps = eps;
    a.rope = Rope{positions, inv_freq, static_cast<int>(rope_offset), static_cast<int>(rope_dim),
                  layout == DSNQ_ROPE_HALF, rope_scale, inverse ? -1.0f : 1.0f};
    a.inject = debug_inject_flags();
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (D <= 64) return launch_heads<8, 1>(a, sms, s);
    if (D <= 128) return launch_heads<16, 1>(a, sms, s);
    if (D <= 256) return launch_heads<32, 1>(a, sms, s);
    if (D <= 512) return launch_heads<32, 2>(a, sms, s);
    return launch_heads<32, 4>(a, sms, s);
}

namespace dsnq {
namespace {

// What the writes in bf16 and in 8 bits have in common; `row` is the length of
// a cache row and `unit` the multiple of its strides, in elements of the cache.
dsnq_status check_write(WriteArgs& a, int64_t M, int64_t K, int64_t P, const void* kv, int64_t ldkv, const void* pe, int64_t ldpe,
                        int32_t normalize, const void* gamma, float eps, const int64_t* positions, const double* inv_freq,
                        int64_t rope_offset, int64_t rope_dim, dsnq_rope_layout layout, float rope_scale, const int64_t* slots,
                        void* cache, int64_t num_pages, int64_t page_size, int64_t ld_page, int64_t ld_row, int64_t row, int64_t unit) {
    if (M < 0 || K <= 0 || P < 0 || num_pages < 0 || page_size <= 0) return DSNQ_ERR_INVALID_ARG;
    if (normalize && (!(eps >= 0.f) || eps > 3.0e38f)) return DSNQ_ERR_INVALID_ARG;   // also rejects NaN
    if (!normalize && gamma) return DSNQ_ERR_INVALID_ARG;
    if (K % kChunk || P % kChunk || K > kMaxWidth || P > kMaxWidth || K + P > kMaxWidth || M > 0x7fffffffLL ||
        page_size > (1 << 20) || num_pages > 0x7fffffffLL || ld_row > (1LL << 40))
        return DSNQ_ERR_UNSUPPORTED;
    const int64_t W = K + P;
    dsnq_status st = check_rope(W, rope_offset, rope_dim, layout, rope_scale);
    if (st != DSNQ_OK) return st;
    if (M == 0) return DSNQ_OK;
    if (!kv || (P && !pe) || !slots || (num_pages && !cache) || (rope_dim && (!positions || !inv_freq)))
        return DSNQ_ERR_INVALID_ARG;
    if ((M > 1 && (ldkv < K || (P && ldpe < P))) || ld_row < row || ld_page < (page_size - 1) * ld_row + row)
        return DSNQ_ERR_INVALID_ARG;
    if (!aligned(kv, 16) || ldkv % kChunk || (P && (!aligned(pe, 16) || ldpe % kChunk)) || !aligned(cache, 16) ||
        ld_page % unit || ld_row % unit || (gamma && !aligned(gamma, 16)) || !aligned(slots, 8) ||
        !aligned(positions, 8) || !aligned(inv_freq, 8))
        return DSNQ_ERR_MISALIGNED;
    a.kv = static_cast<const __nv_bfloat16*>(kv);
    a.pe = static_cast<const __nv_bfloat16*>(pe);
    a.gamma = static_cast<const __nv_bfloat16*>(gamma);
    a.ldkv = ldkv; a.ldpe = ldpe;
    a.M = M; a.K = static_cast<int>(K); a.W = static_cast<int>(W);
    a.slots = slots;
    a.cache = cache;
    a.ld_page = ld_page; a.ld_row = ld_row;
    a.num_slots = num_pages * page_size;
    a.page_size = static_cast<int>(page_size);
    a.norm = normalize ? 1 : 0;
    a.k_f = static_cast<float>(K); a.eps = eps;
    a.rope = Rope{positions, inv_freq, static_cast<int>(rope_offset), static_cast<int>(rope_dim),
                  layout == DSNQ_ROPE_HALF, rope_scale, 1.0f};
    a.inject = debug_inject_flags();
    return DSNQ_OK;
}

template <bool HALF, bool FP8>
dsnq_status launch_write(const WriteArgs& a, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>((a.M + kWriteWarps - 1) / kWriteWarps)), block(kWriteWarps * 32);
    void (*kern)(WriteArgs) = a.W <= 256   ? latent_cache_write_kernel<1, HALF, FP8>
                              : a.W <= 512 ? latent_cache_write_kernel<2, HALF, FP8>
                              : a.W <= 768 ? latent_cache_write_kernel<3, HALF, FP8>
                                           : latent_cache_write_kernel<4, HALF, FP8>;
    return launch_result(launch_kernel(kern, grid, block, 0, s, a));
}

}  // namespace
}  // namespace dsnq

extern "C" dsnq_status dsnq_latent_cache_write(
    int64_t M, int64_t K, int64_t P, const void* kv, int64_t ldkv, const void* pe, int64_t ldpe, int32_t normalize,
    const void* gamma, float eps, const int64_t* positions, const double* inv_freq, int64_t rope_offset,
    int64_t rope_dim, dsnq_rope_layout layout, float rope_scale, const int64_t* slots, void* cache, int64_t num_pages,
    int64_t page_size, int64_t ld_page, int64_t ld_row, void* stream) {
    WriteArgs a{};
    const dsnq_status st = check_write(a, M, K, P, kv, ldkv, pe, ldpe, normalize, gamma, eps, positions, inv_freq, rope_offset, rope_dim,
                                       layout, rope_scale, slots, cache, num_pages, page_size, ld_page, ld_row, K + P, kChunk);
    if (st != DSNQ_OK || M == 0) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return layout == DSNQ_ROPE_HALF ? launch_write<true, false>(a, s) : launch_write<false, false>(a, s);
}

extern "C" dsnq_status dsnq_latent_cache_write_fp8(
    int64_t M, int64_t K, int64_t P, const void* kv, int64_t ldkv, const void* pe, int64_t ldpe, int32_t normalize,
    const void* gamma, float eps, const int64_t* positions, const double* inv_freq, int64_t rope_offset,
    int64_t rope_dim, dsnq_rope_layout layout, float rope_scale, const int64_t* slots, void* cache, int64_t num_pages,
    int64_t page_size, int64_t ld_page, int64_t ld_row, float* scales, int64_t ld_scale, void* stream) {
    WriteArgs a{};
    const dsnq_status st = check_write(a, M, K, P, kv, ldkv, pe, ldpe, normalize, gamma, eps, positions, inv_freq, rope_offset, rope_dim,
                                       layout, rope_scale, slots, cache, num_pages, page_size, ld_page, ld_row, K + 2 * P, 16);
    if (st != DSNQ_OK) return st;
    if (K % 16) return DSNQ_ERR_UNSUPPORTED;
    if (M == 0) return DSNQ_OK;
    if (num_pages && !scales) return DSNQ_ERR_INVALID_ARG;
    if (num_pages > 1 && ld_scale < page_size) return DSNQ_ERR_INVALID_ARG;
    if (!aligned(scales, 4)) return DSNQ_ERR_MISALIGNED;
    a.scales = scales;
    a.ld_scale = ld_scale;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return layout == DSNQ_ROPE_HALF ? launch_write<true, true>(a, s) : launch_write<false, true>(a, s);
}

extern "C" dsnq_status dsnq_latent_cache_read_fp8(
    int64_t B, int64_t rows, int64_t K, int64_t P, const void* cache, int64_t num_pages, int64_t page_size, int64_t ld_page,
    int64_t ld_row, const float* scales, int64_t ld_scale, const int32_t* block_table, int64_t table_width, int64_t ld_table,
    const int32_t* row_starts, const int32_t* first, void* out, int64_t ldo, void* stream) {
    if (B < 0 || rows < 0 || K <= 0 || P < 0 || num_pages < 0 || page_size <= 0 || table_width < 0) return DSNQ_ERR_INVALID_ARG;
    if (K % 16 || P % kChunk || K > kMaxWidth || P > kMaxWidth || K + P > kMaxWidth || B > DSNQ_MAX_REQUESTS || rows > 0x7fffffffLL ||
        page_size > (1 << 20) || num_pages > 0x7fffffffLL || table_width > 0x7fffffffLL || table_width * page_size > 0x7fffffffLL ||
        ld_row > (1LL << 40))
        return DSNQ_ERR_UNSUPPORTED;
    if (B == 0 || rows == 0) return DSNQ_OK;
    const int64_t row = K + 2 * P, W = K + P;
    if (!row_starts || !out || (num_pages && (!cache || !scales)) || (table_width && !block_table)) return DSNQ_ERR_INVALID_ARG;
    if ((rows > 1 && ldo < W) || (B > 1 && ld_table < table_width) || ld_row < row || ld_page < (page_size - 1) * ld_row + row ||
        (num_pages > 1 && ld_scale < page_size))
        return DSNQ_ERR_INVALID_ARG;
    if (!aligned(cache, 16) || ld_page % 16 || ld_row % 16 || !aligned(scales, 4) || !aligned(block_table, 4) || !aligned(row_starts, 4) ||
        !aligned(first, 4) || !aligned(out, 16) || ldo % kChunk)
        return DSNQ_ERR_MISALIGNED;
    ReadArgs a{};
    a.cache = static_cast<const uint8_t*>(cache);
    a.scales = scales;
    a.ld_page = ld_page; a.ld_row = ld_row; a.ld_scale = ld_scale;
    a.num_pages = static_cast<int>(num_pages); a.page_size = static_cast<int>(page_size);
    a.K = static_cast<int>(K); a.W = static_cast<int>(W);
    a.table = block_table; a.ld_table = ld_table;
    a.B = static_cast<int>(B); a.width = static_cast<int>(table_width);
    a.row_starts = row_starts;
    a.first = first;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.ldo = ldo; a.rows = rows;
    const uint32_t chunks = static_cast<uint32_t>(W / kChunk);
    a.recip = static_cast<uint32_t>((0x100000000ull + chunks - 1) / chunks);   // exact for the few thousand items of a CTA
    a.inject = debug_inject_flags();
    // Few rows: small CTAs with all of their chunks on the way at once; many: fewer
    // registers, so more CTAs on an SM.  Per call in a graph, 8 rows and 5 chunks
    // against 16 and 3, us: 400 rows of 576 columns 3.6 and 4.6, 4000 4.1 and 5.1,
    // 12000 both 5.7, 80000 28.6 and 27.1; 8000 of 192 4.1 and 3.6.  (32 rows a CTA
    // of 256 threads with 6 chunks: 5.9 and, for 120003 rows, 34.4; now 4.3 and 30.8,
    // 85% of the measured copy bandwidth.)
    const bool few = rows <= 6144;
    const int64_t per = few ? 8 : 16;
    return launch_result(launch_kernel(few ? latent_cache_read_fp8_kernel<8, 5> : latent_cache_read_fp8_kernel<16, 3>,
                                       dim3(static_cast<unsigned>((rows + per - 1) / per)), dim3(kReadThreads), 0,
                                       static_cast<cudaStream_t>(stream), a));
}

extern "C" dsnq_status dsnq_extend_block_tables(
    int64_t B, int64_t rows, int64_t page_size, const int32_t* seq_lens, const int32_t* new_tokens,
    const int32_t* free_pages, int64_t num_free, int32_t* block_table, int64_t table_width, int64_t ld_table,
    int32_t* new_lens, int32_t* row_starts, int64_t* positions, int64_t* slots, int32_t* counts, void* stream) {
    if (B < 0 || rows < 0 || page_size <= 0 || num_free < 0 || table_width < 0) return DSNQ_ERR_INVALID_ARG;
    if (B > DSNQ_MAX_REQUESTS || rows > 0x7fffffffLL || num_free > 0x7fffffffLL || page_size > (1 << 20) ||
        table_width > 0x7fffffffLL || table_width * page_size > 0x7fffffffLL)
        return DSNQ_ERR_UNSUPPORTED;
    if (!row_starts || !counts || (B && (!seq_lens || !new_lens)) || (B && table_width && !block_table) ||
        (num_free && !free_pages) || (rows && (!positions || !slots)))
        return DSNQ_ERR_INVALID_ARG;
    if (B > 1 && ld_table < table_width) return DSNQ_ERR_INVALID_ARG;
    // Every CTA reads the lengths, so no output may take their place.
    if (B && (new_lens == seq_lens || new_lens == new_tokens || row_starts == seq_lens || row_starts == new_tokens))
        return DSNQ_ERR_INVALID_ARG;
    if ((rows && positions == slots) || (B && new_lens == row_starts)) return DSNQ_ERR_INVALID_ARG;
    if (!aligned(seq_lens, 4) || !aligned(new_tokens, 4) || !aligned(free_pages, 4) || !aligned(block_table, 4) ||
        !aligned(new_lens, 4) || !aligned(row_starts, 4) || !aligned(positions, 8) || !aligned(slots, 8) ||
        !aligned(counts, 4))
        return DSNQ_ERR_MISALIGNED;
    ExtendArgs a{};
    a.B = static_cast<int>(B); a.rows = static_cast<int>(rows);
    a.page_size = static_cast<int>(page_size); a.width = static_cast<int>(table_width);
    a.F = static_cast<int>(num_free);
    a.seq_lens = seq_lens; a.new_tokens = new_tokens; a.free_pages = free_pages;
    a.table = block_table; a.ld_table = ld_table;
    a.new_lens = new_lens; a.row_starts = row_starts; a.positions = positions; a.slots = slots; a.counts = counts;
    a.inject = debug_inject_flags();
    const int sms = device_sm_count();
    if (sms <= 0) {
        cudaGetLastError();
        return DSNQ_ERR_CUDA;
    }
    int64_t grid = ((rows > B ? rows : B) + kExtendThreads - 1) / kExtendThreads;
    grid = grid < 1 ? 1 : (grid > sms ? sms : grid);
    const size_t smem = static_cast<size_t>(4 * B) * sizeof(int32_t);
    static_assert(4 * DSNQ_MAX_REQUESTS * sizeof(int32_t) <= 128 * 1024, "four words per request in shared memory");
    // The limit without the attribute is 48 KB with the static part.
    if (smem > 32 * 1024 && !set_smem_attr(reinterpret_cast<const void*>(extend_tables_kernel), smem)) return DSNQ_ERR_CUDA;
    return launch_result(launch_kernel(extend_tables_kernel, dim3(static_cast<unsigned>(grid)), dim3(kExtendThreads), smem,
                                       static_cast<cudaStream_t>(stream), a));
}

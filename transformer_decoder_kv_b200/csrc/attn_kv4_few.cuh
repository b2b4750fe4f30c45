// Attention over a 4-bit cache for units of few query rows (decoding tokens, and the heads of a
// group that share a K/V head): k_attn_kv4_few<NT, PAIR>, up to 8 NT unit rows (4 with PAIR).
//
// The cache's 72 bytes per key are little beside the instructions a key takes (one row: about 12 per key and
// head, 66 % of the issue slots, 4.3 TB/s at 256 streams x 4096 keys x 16 heads; 7 rows: 2.6 TB/s), so those
// are what is saved. The codes go to the tensor cores (mma.sync m16n8k16, f16) as the integers they are;
// tcgen05 would need them unpacked into shared memory for tiles of 128 rows, and here 1 to 16 rows
// meet each key once.
//
//   S^T = K Q^T   A = 16 keys x 64 dims, B = 64 dims x 8 columns. A nibble masked out of its word and
//                 read as f16 bits is n 2^-24 (or 16 n 2^-24), a subnormal number that the tensor
//                 cores take exactly: no conversion. Q is scaled by a power of two per row and split
//                 into an integer of up to 2048 and a remainder of at most 1 / 2, both in f16 (together
//                 within 2^-23 of the row's largest element; dims met as 16 n are divided by 16).
//                 The code is n - 8, so sum(q n) - 8 sum(q) is wanted: of the integer parts that is exact
//                 in f32 (below 2^20 for the 32 dims of a group) and the accumulators just start at
//                 -8 sum; the remainders' correction is added to the result. One accumulator per
//                 group; the key's two scales and the row's factor are applied in f32.
//   softmax       running maximum per unit row and warp, p = exp2(s - m + 12), f32 sums.
//   O^T += V^T P^T  A = 64 dims x 16 keys: code times scale, 3 + 8 significant bits, exact in f16
//                 after the warp's power of two 2^(9 - E) (E follows the largest scale met so far);
//                 B = p in f16 high and low parts. Each chunk of 64 keys sums into fresh
//                 accumulators that are added to the running f32 sums by ordinary fma, so that the
//                 tensor cores' truncation does not build up over a long cache.
//
// E is shared by rows that see different keys, and f16 holds scales from 2^E down to 2^(E - 24) exactly. A
// warp that met scales further apart throws its sums away and takes its keys again in a plain f32 loop (64
// streams x 4096 keys x 16 heads 1.4 ms where all warps do, instead of 78 us); ordinary caches hold none, and
// looking for them in every chunk, to leave only that chunk to a plain loop, took 2 % of every call.
//
// With up to 4 unit rows (PAIR) columns 2 r and 2 r + 1 are row r's high and low parts: half the
// products and half the softmax of the general form, where both parts take a product of their own.
//
// Fragment layouts decide the rest. Row r of S^T's 8-row halves is key (r >> 1) + 4 (r & 1), so that
// after a transposing movmatrix a thread holds P^T's keys t, t + 4 (t + 8, t + 12) of its quad lane t, and
// V's words of those keys are read without bank conflicts. A V word holds 8 dims of one key; two prmt
// of the words of keys t and t + 4 give pairs along the keys, as the A fragment wants them.
//
// A warp owns every fourth chunk of 64 keys of the block's range and copies it into its own ring of
// shared memory with cp.async, one chunk ahead; warps meet only at the end.
#pragma once

#include <cuda_fp16.h>

#include "attn_rows.cuh"

namespace dec {

constexpr int kFewChunk = 64;
constexpr int kFewWarps = 4;
constexpr int kFewStages = 2;
constexpr int kFewStageBytes = kFewChunk * 2 * kKv4RowBytes;   // K codes, V codes, K scales, V scales
constexpr int kFewSpan = 24;             // scales from 2^E down to 2^(E - 24) are exact
constexpr int kFewK = 0, kFewV = kFewChunk * 32, kFewKs = 2 * kFewChunk * 32, kFewVs = kFewKs + kFewChunk * 4;

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// d = a b + c
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0,
                                        float c1, float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    mma_f16(d, a, b0, b1, d[0], d[1], d[2], d[3]);
}
// 2^x, off by 2 ulp at most; results below 2^-126 are 0.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

// f16 high and low parts of two values: hi + lo is within 2^-22 of each.
__device__ __forceinline__ void split_f16(float x, float y, uint32_t& hi, uint32_t& lo) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    hi = h2_bits(h);
    lo = h2_bits(__floats2half2_rn(x - f.x, y - f.y));
}

// Four dims of two keys (the 16-bit halves of u, V's layout: codes at bits 2, 6, 10 and around 14) times
// the keys' scales s: x = 1 + n / 16 by its bits, then x (16 s) - 1.5 (16 s) = (n - 8) s, exact: 1.5 times 8
// significant bits is 10, the result has 11.
__device__ __forceinline__ void kv4_values(uint32_t u, __half2 s16, __half2 c, uint32_t* v) {
    const uint32_t x[4] = {u << 4, u, u >> 4, __byte_perm(u, 0, 0x2301)};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = h2_bits(__hfma2(bits_h2((x[i] & 0x03c003c0u) | 0x3c003c00u), s16, c));
}

// Positions j0 .. j0 + 31 a query at position p sees, as bits.
__device__ __forceinline__ uint32_t visible_bits(long long j0, long long p, int window, int sinks) {
    auto below = [](long long n) -> uint32_t {      // the lowest n bits
        return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
    };
    uint32_t m = below(p + 1 - j0);
    if (window > 0) m &= ~below(p - window + 1 - j0) | below(sinks - j0);
    return m;
}

template <int NT, bool PAIR>
static __global__ void __launch_bounds__(kFewWarps * 32) k_attn_kv4_few(const RowsAttnArgs a) {
    static_assert(!PAIR || NT == 1, "paired columns: one column tile");
    constexpr int UR = PAIR ? 4 : 8 * NT;
    constexpr int NB = PAIR ? 1 : 2;         // unit rows a thread holds scores of, per column tile
    constexpr int MT = kFewChunk / 16;
    extern __shared__ __align__(128) unsigned char few_smem[];
    __shared__ float sm_m[kFewWarps][UR], sm_l[kFewWarps][UR];
    __shared__ __align__(8) uint32_t sm_vs[kFewWarps][2][kFewChunk / 2];      // V scales of a chunk, f16, by group

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    pdl_wait();
    const StreamRows s = stream_rows(a.r, a.v, blockIdx.z);
    const int n_tiles = gridDim.y / a.v.heads;
    const int hk = blockIdx.y / n_tiles;
    const UnitKeys k = unit_keys<UR, kFewChunk>(a, s, blockIdx.y % n_tiles);
    const int sp = blockIdx.x;
    if (k.n_u == 0 || sp >= k.splits) return;
    const int c_end = split_begin(k, sp + 1);
    const int c0 = split_begin(k, sp) + warp;

    // ---- the ring ----
    unsigned char* ring = few_smem + warp * kFewStages * kFewStageBytes;
    const int pr_mask = a.v.page_rows - 1;
    const int part = a.v.page_rows * kKv4RowBytes;               // bytes of a block's K part
    const unsigned page_bytes = static_cast<unsigned>(a.v.heads) * 2u * part;
    const unsigned char* base = a.cache + static_cast<long long>(hk) * 2 * part;
    const int end = static_cast<int>(k.end);
    const int* tab = a.v.table ? a.v.table + s.slot * a.v.pages_per_slot : nullptr;
    // Lane: pieces of the chunk's 16-row quarter lane / 8, by 8 lanes each.
    const int sub = lane & 7, qrow = (lane >> 3) * 16;
    const int scale_off = a.v.page_rows * 32 + (sub & 3) * 16 + ((sub & 4) ? part : 0);
    // Page of the lane's quarter of a chunk, -1 where there are no rows.
    auto quarter_page = [&](int c) {
        int p = -1;
        const int j = unit_chunk(k, c) * kFewChunk + qrow;
        if (c < c_end && j < end) {
            p = tab ? tab[j >> a.v.shift] : s.slot * a.v.pages_per_slot + (j >> a.v.shift);
            if (static_cast<unsigned>(p) >= static_cast<unsigned>(a.v.n_pages)) p = -1;
        }
        return p;
    };
    int pg = quarter_page(c0);

    // the queries of column g of each tile, dims 8 t .. 8 t + 7 of both groups, fetched meanwhile
    float qx[NT][2][8];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int u = PAIR ? g >> 1 : nt * 8 + g;
        if (u < k.n_u) {
            const int ur = k.u0 + u, i = ur / a.group, h = hk * a.group + ur % a.group;
            const float4* q = reinterpret_cast<const float4*>(a.q + static_cast<long long>(s.row0 + i) * a.q_ld +
                                                              h * kHeadDim + 8 * t);
#pragma unroll
            for (int gr = 0; gr < 2; ++gr) {
                const float4 x0 = q[gr * 8], x1 = q[gr * 8 + 1];
                float* x = qx[nt][gr];
                x[0] = x0.x, x[1] = x0.y, x[2] = x0.z, x[3] = x0.w;
                x[4] = x1.x, x[5] = x1.y, x[6] = x1.z, x[7] = x1.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) qx[nt][0][j] = qx[nt][1][j] = 0.0f;
        }
    }
    uint32_t bad[2] = {0, 0};              // per stage: lanes whose quarter has no page
    auto issue = [&](int c, int stage) {
        if (c < c_end) {
            unsigned char* dst = ring + stage * kFewStageBytes;
            const int r = (unit_chunk(k, c) * kFewChunk + qrow) & pr_mask;
            const unsigned char* blk = base + static_cast<unsigned long long>(static_cast<unsigned>(pg)) * page_bytes;
            const unsigned char* src = blk + (r * 32 + sub * 16);
            if (pg >= 0) {
                unsigned char* d = dst + qrow * 32 + sub * 16;
#pragma unroll
                for (int i = 0; i < 4; ++i) cp_async16(d + kFewK + i * 128, src + i * 128);
                src += part;
#pragma unroll
                for (int i = 0; i < 4; ++i) cp_async16(d + kFewV + i * 128, src + i * 128);
                cp_async16(dst + ((sub & 4) ? kFewVs : kFewKs) + qrow * 4 + (sub & 3) * 16, blk + (r * 4 + scale_off));
            }
            const uint32_t m = __ballot_sync(0xffffffffu, pg < 0);
            if (stage) bad[1] = m; else bad[0] = m;
            pg = quarter_page(c + kFewWarps);
        }
        cp_async_commit();
    };
    issue(c0, 0);

    // ---- Q^T fragments ----
    uint32_t qf[NB][NT][4][2];             // PAIR: one part per column; else high, low
    // score factors of this thread's rows; -8 sum(q) of columns 2 t, 2 t + 1: where the accumulators
    // start, and (not PAIR) the remainders' part
    float qs[NT][NB], off[NT][2][2], rem[NT][2][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const float (&x)[2][8] = qx[nt];
        float mx = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fmaxf(fabsf(x[0][j]), fabsf(x[1][j])));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // the row's largest element goes to [2^10, 2^11); rows below 2^-100 are taken as that small
        const int e = max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -100);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 10 - e) << 23);
        const float down = (e > 112 ? INFINITY : __uint_as_float(static_cast<uint32_t>(127 - 10 + 24 + e) << 23)) *
                           (0.125f * kLog2e);
        float sum[2][2] = {};                // [group][integer part (PAIR: this column's part), remainder]
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            const float* y = x[ks >> 1];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int j = (ks & 1) * 2 + b;
                const float f = b ? 0.0625f : 1.0f;
                const float y0 = y[j] * up, y1 = y[j + 4] * up, h0 = rintf(y0), h1 = rintf(y1);
                const __half2 hi = __floats2half2_rn(h0 * f, h1 * f), lo = __floats2half2_rn((y0 - h0) * f, (y1 - h1) * f);
                const float2 lf = __half22float2(lo);
                const float sh = h0 + h1, sl = (lf.x + lf.y) * (b ? 16.0f : 1.0f);
                if (PAIR) {
                    qf[0][nt][ks][b] = h2_bits((g & 1) ? lo : hi);
                    sum[ks >> 1][0] += (g & 1) ? sl : sh;
                } else {
                    qf[0][nt][ks][b] = h2_bits(hi);
                    qf[NB - 1][nt][ks][b] = h2_bits(lo);
                    sum[ks >> 1][0] += sh;
                    sum[ks >> 1][1] += sl;
                }
            }
        }
#pragma unroll
        for (int gr = 0; gr < 2; ++gr)
#pragma unroll
            for (int part = 0; part < (PAIR ? 1 : 2); ++part) {
                float v = sum[gr][part];
                v += __shfl_xor_sync(0xffffffffu, v, 1);
                v += __shfl_xor_sync(0xffffffffu, v, 2);
                v *= -8.0f / 16777216.0f;
                (part ? rem : off)[nt][gr][0] = __shfl_sync(0xffffffffu, v, 8 * t);
                (part ? rem : off)[nt][gr][1] = __shfl_sync(0xffffffffu, v, 8 * t + 4);
            }
        qs[nt][0] = __shfl_sync(0xffffffffu, down, 8 * t);
        if (!PAIR) qs[nt][NB - 1] = __shfl_sync(0xffffffffu, down, 8 * t + 4);
    }

    // ---- running state: unit row 8 nt + 2 t + b (PAIR: t); O^T dims 8 g + 2 mt, + 1 ----
    auto row_of = [&](int nt, int b) { return PAIR ? t : nt * 8 + 2 * t + b; };
    float m[NT][NB], rf[NT][NB], l[NT][NB], o[NT][4][4];     // maximum, reference of the weights, sum, values
    int E = -100;                          // V is held times 2^(9 - E)
    uint32_t low = 0xffffffffu;            // the lane's smallest V scales that are not 0, less 1, by group
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            m[nt][b] = rf[nt][b] = -INFINITY;
            l[nt][b] = 0.0f;
        }
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[nt][mt][j] = 0.0f;
    }
    const long long p_first = s.pos0 + k.u0 / a.group, p_last = s.pos0 + (k.u0 + k.n_u - 1) / a.group;
    // chunks whose 64 keys all rows see: below, and above or within the sinks
    const int full_hi = static_cast<int>(min(p_first - (kFewChunk - 1), 0x7fffff00ll));
    const int full_lo = a.window == 0 ? 0 : static_cast<int>(max(0ll, min(p_last - a.window + 1, 0x7fffff00ll)));
    // keys below, past the sinks: no row sees them
    const int seen_lo = a.window > 0 ? static_cast<int>(max(0ll, min(p_first - a.window + 1, 0x7fffff00ll))) : 0;
    const int key_a = (g >> 1) + 4 * (g & 1);           // key of S^T row g of a 16-key half

    int stage = 0;
    for (int c = c0; c < c_end; c += kFewWarps) {
        issue(c + kFewWarps, stage ^ 1);
        cp_async_wait<kFewStages - 1>();
        __syncwarp();
        const unsigned char* st = ring + stage * kFewStageBytes;
        const int j0 = unit_chunk(k, c) * kFewChunk;
        const uint32_t miss = stage ? bad[1] : bad[0];
        const bool full = miss == 0 && j0 <= full_hi && (j0 >= full_lo || j0 + kFewChunk <= a.sinks);

        // this thread's rows: the keys of this chunk they see
        uint32_t vis[NT][NB][2];
        uint32_t have[2] = {0xffffffffu, 0xffffffffu};
        if (full) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int b = 0; b < NB; ++b) vis[nt][b][0] = vis[nt][b][1] = 0xffffffffu;
        } else {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                have[w] = ((miss >> (16 * w)) & 1u ? 0u : 0xffffu) | ((miss >> (16 * w)) & 0x100u ? 0u : 0xffff0000u);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        vis[nt][b][w] = visible_bits(j0 + 32 * w, s.pos0 + (k.u0 + row_of(nt, b)) / a.group, a.window,
                                                     a.sinks) & have[w];
            }
        }

        // V scales, lane = two keys 4 apart: f16 of 16 times scale 2^(9 - E), 0 for keys that no row sees
        // (whose bits may be anything), and for a scale that is not a number (those keys' outputs are
        // set below). Kept in the order their readers want: keys 16 i + t, + 4, + 8, + 12 of quad lane t
        // side by side. (A row never written may hold a negative scale: magnitudes are compared.)
        float fac = 1.0f;
        uint32_t any_nan;
        const int vkey = (lane >> 3) * 16 + ((lane >> 1) & 3) + 8 * (lane & 1);
        uint32_t vw[2];
        {
            float z[2][2], big = 0.0f;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const int key = vkey + 4 * w;
                vw[w] = *reinterpret_cast<const uint32_t*>(st + kFewVs + key * 4);
                if (!full) {
                    const int j = j0 + key;
                    const bool seen = (((lane & 16) ? have[1] : have[0]) >> (key & 31) & 1u) && j <= p_last &&
                                      (j >= seen_lo || j < a.sinks);
                    vw[w] = seen ? vw[w] : 0u;
                }
                low = __vminu2(low, vw[w] - 0x00010001u);          // (a zero gives 0xfffe or more)
                z[w][0] = __uint_as_float(vw[w] << 16);
                z[w][1] = __uint_as_float(vw[w] & 0xffff0000u);
                big = fmaxf(big, fmaxf(fabsf(z[w][0]), fabsf(z[w][1])));
            }
            // (stored scales are below 2^126: four of them stay finite)
            any_nan = __ballot_sync(0xffffffffu, !((fabsf(z[0][0]) + fabsf(z[0][1])) + (fabsf(z[1][0]) + fabsf(z[1][1])) < INFINITY));
            if (any_nan) {
                big = 0.0f;
#pragma unroll
                for (int w = 0; w < 2; ++w)
#pragma unroll
                    for (int gr = 0; gr < 2; ++gr) {
                        if (!(fabsf(z[w][gr]) < INFINITY)) z[w][gr] = 0.0f;
                        big = fmaxf(big, fabsf(z[w][gr]));
                    }
            }
            const int e = max(static_cast<int>(__reduce_max_sync(0xffffffffu, __float_as_uint(big)) >> 23) - 127, -100);
            if (e > E) {
                fac = E < e - 120 ? 0.0f : __uint_as_float(static_cast<uint32_t>(127 + E - e) << 23);
                E = e;
            }
            const float up = __uint_as_float(static_cast<uint32_t>(127 + 13 - E) << 23);
#pragma unroll
            for (int gr = 0; gr < 2; ++gr)
                sm_vs[warp][gr][lane] = h2_bits(__floats2half2_rn(z[0][gr] * up, z[1][gr] * up));
        }
        __syncwarp();

        // ---- scores: sc[..][mt][j] of keys 16 mt + key_a + 8 j ----
        float sc[NT][NB][MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            uint32_t ka[4][4];              // A fragments of the four 16-dim steps
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
                const uint2 w = *reinterpret_cast<const uint2*>(st + kFewK + (mt * 16 + hi * 8 + key_a) * 32 + t * 8);
                const uint32_t x8 = w.x >> 8, y8 = w.y >> 8;
                ka[0][hi] = w.x & 0x000f000fu, ka[0][2 + hi] = w.x & 0x00f000f0u;
                ka[1][hi] = x8 & 0x000f000fu, ka[1][2 + hi] = x8 & 0x00f000f0u;
                ka[2][hi] = w.y & 0x000f000fu, ka[2][2 + hi] = w.y & 0x00f000f0u;
                ka[3][hi] = y8 & 0x000f000fu, ka[3][2 + hi] = y8 & 0x00f000f0u;
            }
            float ks0[2], ks1[2];           // the keys' scales
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(st + kFewKs + (mt * 16 + 8 * j + key_a) * 4);
                ks0[j] = __uint_as_float(w << 16);
                ks1[j] = __uint_as_float(w & 0xffff0000u);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float d0[4], d1[4];
                const float* c0v = off[nt][0];
                const float* c1v = off[nt][1];
                mma_f16(d0, ka[0], qf[0][nt][0][0], qf[0][nt][0][1], c0v[0], c0v[1], c0v[0], c0v[1]);
                mma_f16(d1, ka[2], qf[0][nt][2][0], qf[0][nt][2][1], c1v[0], c1v[1], c1v[0], c1v[1]);
                mma_f16(d0, ka[1], qf[0][nt][1][0], qf[0][nt][1][1]);
                mma_f16(d1, ka[3], qf[0][nt][3][0], qf[0][nt][3][1]);
                if (!PAIR) {
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks) {
                        mma_f16(d0, ka[ks], qf[NB - 1][nt][ks][0], qf[NB - 1][nt][ks][1]);
                        mma_f16(d1, ka[2 + ks], qf[NB - 1][nt][2 + ks][0], qf[NB - 1][nt][2 + ks][1]);
                    }
                }
                // (the raw sums are below 1: no scale takes them out of f32's range)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (PAIR) {
                        const float r0 = d0[2 * j] + d0[2 * j + 1], r1 = d1[2 * j] + d1[2 * j + 1];
                        sc[nt][0][mt][j] = fmaf(r1, ks1[j], r0 * ks0[j]) * qs[nt][0];
                    } else {
                        // both rows of the thread at once
                        const float2 r0 = add2(make_float2(d0[2 * j], d0[2 * j + 1]), make_float2(rem[nt][0][0], rem[nt][0][1]));
                        const float2 r1 = add2(make_float2(d1[2 * j], d1[2 * j + 1]), make_float2(rem[nt][1][0], rem[nt][1][1]));
                        const float2 x = fma2(r1, make_float2(ks1[j], ks1[j]), mul2(r0, make_float2(ks0[j], ks0[j])));
                        const float2 y = mul2(x, make_float2(qs[nt][0], qs[nt][NB - 1]));
                        sc[nt][0][mt][j] = y.x;
                        sc[nt][NB - 1][mt][j] = y.y;
                    }
                }
            }
        }
        if (!full) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            if (!((vis[nt][b][mt >> 1] >> ((mt & 1) * 16 + j * 8 + key_a)) & 1u))
                                sc[nt][b][mt][j] = -INFINITY;
        }

        // ---- softmax ----
        uint32_t ph[NT][MT][2], pl[PAIR ? 1 : NT][MT][2];       // B fragments of P^T (PAIR: both parts in ph)
        float corr[NT][NB];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float mx = -INFINITY;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) mx = fmaxf(mx, fmaxf(sc[nt][b][mt][0], sc[nt][b][mt][1]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                const float mn = fmaxf(m[nt][b], mx);
                // Weights are 2^(s - ref): ref 12 below the maximum keeps small ones in f16's range
                // (at the maximum itself where f32 no longer resolves 12); before anything is seen
                // ref 0 makes every term 0.
                const float ref = mn == -INFINITY ? 0.0f : fabsf(mn) < 65536.0f ? mn - 12.0f : mn;
                corr[nt][b] = ex2(rf[nt][b] - ref);
                m[nt][b] = mn;
                rf[nt][b] = mn == -INFINITY ? -INFINITY : ref;
                float sum = 0.0f;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        sc[nt][b][mt][j] = ex2(sc[nt][b][mt][j] - ref);
                        sum += sc[nt][b][mt][j];
                    }
                l[nt][b] = fmaf(l[nt][b], corr[nt][b], sum);
                corr[nt][b] *= fac;
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if (PAIR) {
                    uint32_t h, lo;          // keys j = 0, 1; then (high, low) of each
                    split_f16(sc[nt][0][mt][0], sc[nt][0][mt][1], h, lo);
                    ph[nt][mt][0] = movmatrix_trans(__byte_perm(h, lo, 0x5410));
                    ph[nt][mt][1] = movmatrix_trans(__byte_perm(h, lo, 0x7632));
                } else {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t h, lo;
                        split_f16(sc[nt][0][mt][j], sc[nt][NB - 1][mt][j], h, lo);
                        ph[nt][mt][j] = movmatrix_trans(h);
                        pl[nt][mt][j] = movmatrix_trans(lo);
                    }
                }
            }
        }

        // ---- values ----
        float d[NT][4][4];
#pragma unroll
        for (int ks = 0; ks < MT; ++ks) {
            const unsigned char* vp = st + kFewV + ks * 512 + t * 32 + g * 4;
            const uint32_t w0 = *reinterpret_cast<const uint32_t*>(vp), w1 = *reinterpret_cast<const uint32_t*>(vp + 128);
            const uint32_t w2 = *reinterpret_cast<const uint32_t*>(vp + 256);
            const uint32_t w3 = *reinterpret_cast<const uint32_t*>(vp + 384);
            const uint2 vs = *reinterpret_cast<const uint2*>(&sm_vs[warp][g >> 2][ks * 8 + t * 2]);
            // pairs along the keys: low and high halves of two keys' words side by side
            const __half2 s0 = bits_h2(vs.x), s1 = bits_h2(vs.y), c15 = __float2half2_rn(-1.5f);
            const __half2 z0 = __hmul2(s0, c15), z1 = __hmul2(s1, c15);
            uint32_t d01[8], d23[8];
            kv4_values(__byte_perm(w0, w1, 0x5410), s0, z0, d01);
            kv4_values(__byte_perm(w0, w1, 0x7632), s0, z0, d01 + 4);
            kv4_values(__byte_perm(w2, w3, 0x5410), s1, z1, d23);
            kv4_values(__byte_perm(w2, w3, 0x7632), s1, z1, d23 + 4);
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                const uint32_t va[4] = {d01[2 * mt], d01[2 * mt + 1], d23[2 * mt], d23[2 * mt + 1]};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if (ks == 0)
                        mma_f16(d[nt][mt], va, ph[nt][0][0], ph[nt][0][1], 0.0f, 0.0f, 0.0f, 0.0f);
                    else
                        mma_f16(d[nt][mt], va, ph[nt][ks][0], ph[nt][ks][1]);
                    if (!PAIR) mma_f16(d[nt][mt], va, pl[nt][ks][0], pl[nt][ks][1]);
                }
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    const float2 y = fma2(make_float2(o[nt][mt][j], o[nt][mt][j + 1]),
                                          make_float2(corr[nt][0], corr[nt][NB - 1]),
                                          make_float2(d[nt][mt][j], d[nt][mt][j + 1]));
                    o[nt][mt][j] = y.x;
                    o[nt][mt][j + 1] = y.y;
                }
        if (any_nan) {                     // a seen key whose V group is not a number
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                // of keys 32 w .. 32 w + 31: those with such a scale, from the lanes that hold them
                uint32_t bits = 0;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t n0 = __ballot_sync(0xffffffffu, (vw[i] & 0x7f80u) == 0x7f80u);
                    const uint32_t n1 = __ballot_sync(0xffffffffu, (vw[i] & 0x7f800000u) == 0x7f800000u);
                    const uint32_t n = g < 4 ? n0 : n1;
                    for (int x = 16 * w; x < 16 * w + 16; ++x)
                        if ((n >> x) & 1u) bits |= 1u << (((x >> 3) & 1) * 16 + ((x >> 1) & 3) + 8 * (x & 1) + 4 * i);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        if (vis[nt][b][w] & bits) {
#pragma unroll
                            for (int mt = 0; mt < 4; ++mt) o[nt][mt][b] = o[nt][mt][b + 2] = __uint_as_float(0x7fc00000u);
                        }
            }
        }
        __syncwarp();
        stage ^= 1;
    }
    cp_async_wait<0>();
    __syncthreads();

    float back = __uint_as_float(static_cast<uint32_t>(127 + E - 9) << 23);
    if (__any_sync(0xffffffffu, static_cast<int>(min(low & 0xffffu, low >> 16)) + 1 < (127 + E - kFewSpan) << 7)) {
        // ---- plain loop: thread = a word of 8 dims, the rows of its quad lane ----
        float q[NT][NB][8];
        back = 1.0f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int ur = k.u0 + min(row_of(nt, b), k.n_u - 1), h = hk * a.group + ur % a.group;
                const float* src = a.q + static_cast<long long>(s.row0 + ur / a.group) * a.q_ld + h * kHeadDim + 8 * g;
#pragma unroll
                for (int n = 0; n < 8; ++n) q[nt][b][n] = src[n];
                rf[nt][b] = -INFINITY;
                m[nt][b] = INFINITY;               // (weights of at most 1)
                l[nt][b] = 0.0f;
            }
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[nt][mt][j] = 0.0f;
        }
        for (int c = c0; c < c_end; c += kFewWarps)
            for (int x = 0; x < kFewChunk; ++x) {
                const int j = unit_chunk(k, c) * kFewChunk + x;
                if (j >= end) break;
                const int page = tab ? tab[j >> a.v.shift] : s.slot * a.v.pages_per_slot + (j >> a.v.shift);
                if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.v.n_pages)) continue;
                const unsigned char* blk = base + static_cast<unsigned long long>(static_cast<unsigned>(page)) * page_bytes;
                const int r = j & pr_mask, at = a.v.page_rows * 32 + r * 4 + (g >> 2) * 2;
                const uint32_t kc = *reinterpret_cast<const uint32_t*>(blk + r * 32 + ((g & 3) * 2 + (g >> 2)) * 4);
                uint32_t vc = *reinterpret_cast<const uint32_t*>(blk + part + r * 32 + g * 4);
                vc = ((vc >> 2) & 0x3fff3fffu) | ((vc << 14) & 0xc000c000u);
                const float ks = __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(blk + at)) << 16);
                const float vs = __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(blk + part + at)) << 16);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        float sc = 0.0f;
#pragma unroll
                        for (int n = 0; n < 8; ++n)
                            sc = fmaf(ks * static_cast<float>(static_cast<int>((kc >> (4 * n)) & 15u) - 8), q[nt][b][n], sc);
                        sc += __shfl_xor_sync(0xffffffffu, sc, 4);
                        sc += __shfl_xor_sync(0xffffffffu, sc, 8);
                        sc = (sc + __shfl_xor_sync(0xffffffffu, sc, 16)) * (0.125f * kLog2e);
                        const long long p = s.pos0 + (k.u0 + row_of(nt, b)) / a.group;
                        if (!(j <= p && (a.window == 0 || j > p - a.window || j < a.sinks))) sc = -INFINITY;
                        const float mn = fmaxf(rf[nt][b], sc), ref = mn == -INFINITY ? 0.0f : mn;
                        const float cr = ex2(rf[nt][b] - ref), w = ex2(sc - ref);
                        rf[nt][b] = mn;
                        l[nt][b] = fmaf(l[nt][b], cr, g == 0 ? w : 0.0f);
#pragma unroll
                        for (int n = 0; n < 8; ++n) {
                            float& on = o[nt][n >> 1][(n & 1) * 2 + b];
                            on *= cr;
                            if (w != 0.0f) on = fmaf(w, vs * static_cast<float>(static_cast<int>((vc >> (4 * n)) & 15u) - 8), on);
                        }
                    }
            }
    }

    // ---- join the warps: O as [unit row][dim], each warp's sums scaled back ----
    float* so = reinterpret_cast<float*>(few_smem) + warp * UR * (kHeadDim + 4);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float sum = l[nt][b];
            sum += __shfl_xor_sync(0xffffffffu, sum, 4);
            sum += __shfl_xor_sync(0xffffffffu, sum, 8);
            sum += __shfl_xor_sync(0xffffffffu, sum, 16);
            const int u = row_of(nt, b);
            const RowScale f = row_scale(m[nt][b], rf[nt][b]);
            if (g == 0) {
                sm_m[warp][u] = f.ref;
                sm_l[warp][u] = sum * f.mul;
            }
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                const float x = PAIR ? o[nt][mt][0] + o[nt][mt][1] : o[nt][mt][b];
                const float y = PAIR ? o[nt][mt][2] + o[nt][mt][3] : o[nt][mt][b + 2];
                *reinterpret_cast<float2*>(so + u * (kHeadDim + 4) + 8 * g + 2 * mt) =
                    make_float2(x * (back * f.mul), y * (back * f.mul));
            }
        }
    __syncthreads();
    for (int x = tid; x < k.n_u * (kHeadDim / 4); x += kFewWarps * 32) {
        const int u = x / (kHeadDim / 4), d4 = x % (kHeadDim / 4);
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) mx = fmaxf(mx, sm_m[w][u]);
        float L = 0.0f;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) {
            const float e = sm_m[w][u] == -INFINITY ? 0.0f : exp2f(sm_m[w][u] - mx);
            L = fmaf(e, sm_l[w][u], L);
            const float4 ow = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(few_smem) +
                                                               (w * UR + u) * (kHeadDim + 4) + d4 * 4);
            if (e != 0.0f) {
                acc.x = fmaf(e, ow.x, acc.x);
                acc.y = fmaf(e, ow.y, acc.y);
                acc.z = fmaf(e, ow.z, acc.z);
                acc.w = fmaf(e, ow.w, acc.w);
            }
        }
        store_unit_row(a, k, s, hk, sp, u, d4, mx, L, acc);
    }
}

inline size_t few_smem_bytes(int unit_rows) {
    const size_t ring = size_t(kFewWarps) * kFewStages * kFewStageBytes;
    const size_t join = size_t(kFewWarps) * unit_rows * (kHeadDim + 4) * sizeof(float);
    return ring > join ? ring : join;
}

}  // namespace dec

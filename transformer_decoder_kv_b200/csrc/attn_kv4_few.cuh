// Attention over a 4-bit cache for units of few query rows (decoding tokens, and the heads of a
// group that share a K/V head): k_attn_kv4_few<NT>, up to 8 NT unit rows.
//
// Bound by the cache's 72 bytes per key, so the work per key must stay small: the codes go to the
// tensor cores (mma.sync m16n8k16, f16) as the integers they are. tcgen05 would need the codes
// unpacked into shared memory for tiles of 128 rows; here 1 to 16 rows meet each key once, and the
// unpacked codes stay in the registers of the warp that read them.
//
//   S^T = K Q^T   A = 16 keys x 64 dims (codes, exact in f16), B = 64 dims x 8 unit rows. Q is scaled
//                 by a power of two per row and split into f16 high and low parts (22 bits), the two
//                 products accumulate in f32, one accumulator per group of 32 dims, and the key's
//                 two scales and the row's factor are applied to them in f32.
//   softmax       running maximum per unit row and warp, p = exp2(s - m + 12), f32 sums.
//   O^T += V^T P^T  A = 64 dims x 16 keys: code times scale, 3 + 8 significant bits, exact in f16
//                 after the warp's power of two 2^-E (E follows the largest scale met so far);
//                 B = p in f16 high and low parts. Each chunk of 32 keys sums into fresh
//                 accumulators that are added to the running f32 sums by ordinary fma, so that the
//                 tensor cores' truncation does not build up over a long cache.
//
// Fragment layouts decide the rest. Row r of S^T's 8-row halves is key (r >> 1) + 4 (r & 1), so that
// after a transposing movmatrix a thread holds P^T's keys t, t + 4 (t + 8, t + 12) of its quad lane t, and
// V's words of those keys are read without bank conflicts. A V word holds 8 dims of one key; two prmt
// of the words of keys t and t + 4 give pairs along the keys, as the A fragment wants them.
//
// A warp owns every fourth chunk of 32 keys of the block's range and copies it into its own ring of
// shared memory with cp.async, kStages - 1 chunks ahead; warps meet only at the end.
#pragma once

#include <cuda_fp16.h>

#include "attn_rows.cuh"

namespace dec {

constexpr int kFewChunk = 32;
constexpr int kFewWarps = 4;
constexpr int kFewStages = 3;
constexpr int kFewStageBytes = kFewChunk * 2 * kKv4RowBytes;   // K codes, V codes, K scales, V scales
constexpr int kFewK = 0, kFewV = kFewChunk * 32, kFewKs = 2 * kFewChunk * 32, kFewVs = kFewKs + kFewChunk * 4;

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// Codes of nibbles j and j + 4 of a word as f16 pairs p[j], j = 0..3. 0x6400 | n is 1024 + n; a nibble
// four bits up gives 1024 + 16 n, halved down by one fma.
__device__ __forceinline__ void kv4_pairs(uint32_t w, uint32_t* p) {
    const __half2 sub = bits_h2(0x64086408u);                              // 1032
    const __half2 s16 = bits_h2(0x2c002c00u), sub16 = bits_h2(0xd480d480u);   // 1 / 16, -72
    const uint32_t w8 = w >> 8;
    p[0] = h2_bits(__hsub2(bits_h2((w & 0x000f000fu) | 0x64006400u), sub));
    p[1] = h2_bits(__hfma2(bits_h2((w & 0x00f000f0u) | 0x64006400u), s16, sub16));
    p[2] = h2_bits(__hsub2(bits_h2((w8 & 0x000f000fu) | 0x64006400u), sub));
    p[3] = h2_bits(__hfma2(bits_h2((w8 & 0x00f000f0u) | 0x64006400u), s16, sub16));
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

template <int NT>
static __global__ void __launch_bounds__(kFewWarps * 32) k_attn_kv4_few(const RowsAttnArgs a) {
    constexpr int UR = 8 * NT;
    extern __shared__ __align__(128) unsigned char few_smem[];
    __shared__ float sm_m[kFewWarps][UR], sm_l[kFewWarps][UR];
    __shared__ uint32_t sm_vs[kFewWarps][2][kFewChunk / 2];      // V scales of a chunk, f16, by group

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
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
    // Pages of the two 16-row halves of a chunk (-1: no rows there)
    auto half_page = [&](int c, int half) {
        const long long j = static_cast<long long>(unit_chunk(k, c)) * kFewChunk + half * 16;
        return c < c_end && j < k.end ? kv_page(a.v, s.slot, static_cast<int>(j) >> a.v.shift) : -1;
    };
    int pg0 = half_page(c0, 0), pg1 = half_page(c0, 1);
    uint32_t bad = 0;                      // two bits per stage: halves without a page
    const int pr_mask = a.v.page_rows - 1;
    auto issue = [&](int c, int stage) {
        if (c < c_end) {
            unsigned char* dst = ring + stage * kFewStageBytes;
            const int j = unit_chunk(k, c) * kFewChunk;
            const int part = a.v.page_rows * kKv4RowBytes;       // bytes of a block's K part
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int pg = half ? pg1 : pg0;
                if (pg < 0) continue;
                const int pr = (j + half * 16) & pr_mask;
                const unsigned char* blk = a.cache + kv4_block(a.v, pg, hk);
                cp_async16(dst + kFewK + half * 512 + lane * 16, blk + pr * 32 + lane * 16);
                cp_async16(dst + kFewV + half * 512 + lane * 16, blk + part + pr * 32 + lane * 16);
                if (lane < 8)
                    cp_async16(dst + (lane < 4 ? kFewKs : kFewVs) + half * 64 + (lane & 3) * 16,
                               blk + (lane < 4 ? 0 : part) + a.v.page_rows * 32 + pr * 4 + (lane & 3) * 16);
            }
            bad = (bad & ~(3u << (2 * stage))) | (((pg0 < 0 ? 1u : 0u) | (pg1 < 0 ? 2u : 0u)) << (2 * stage));
            pg0 = half_page(c + kFewWarps, 0);
            pg1 = half_page(c + kFewWarps, 1);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kFewStages - 1; ++i) issue(c0 + i * kFewWarps, i);

    // ---- Q^T fragments: unit row g of each tile, dims 8 t .. 8 t + 7 of both groups ----
    uint32_t qh[NT][4][2], ql[NT][4][2];
    float qs[NT][2];                       // score factors of unit rows 2 t, 2 t + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int u = nt * 8 + g;
        float x[2][8];
        if (u < k.n_u) {
            const int ur = k.u0 + u, i = ur / a.group, h = hk * a.group + ur % a.group;
            const float4* q = reinterpret_cast<const float4*>(a.q + static_cast<long long>(s.row0 + i) * a.q_ld +
                                                              h * kHeadDim + 8 * t);
#pragma unroll
            for (int gr = 0; gr < 2; ++gr) {
                const float4 x0 = q[gr * 8], x1 = q[gr * 8 + 1];
                x[gr][0] = x0.x, x[gr][1] = x0.y, x[gr][2] = x0.z, x[gr][3] = x0.w;
                x[gr][4] = x1.x, x[gr][5] = x1.y, x[gr][6] = x1.z, x[gr][7] = x1.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[0][j] = x[1][j] = 0.0f;
        }
        float mx = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fmaxf(fabsf(x[0][j]), fabsf(x[1][j])));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // the row's largest element goes to [2^10, 2^11); rows below 2^-100 are taken as that small
        const int e = max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -100);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 10 - e) << 23);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - 10 + e) << 23) * (0.125f * kLog2e);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            const float* y = x[ks >> 1];
            const int j = (ks & 1) * 2;
            split_f16(y[j] * up, y[j + 4] * up, qh[nt][ks][0], ql[nt][ks][0]);
            split_f16(y[j + 1] * up, y[j + 5] * up, qh[nt][ks][1], ql[nt][ks][1]);
        }
        qs[nt][0] = __shfl_sync(0xffffffffu, down, 8 * t);
        qs[nt][1] = __shfl_sync(0xffffffffu, down, 8 * t + 4);
    }

    // ---- running state: unit rows 8 nt + 2 t, + 1; O^T dims 8 g + 2 mt, + 1 ----
    float m[NT][2], l[NT][2], o[NT][4][4];
    int E = -1000;                         // V is held times 2^(11 - E)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[nt][mt][j] = 0.0f;
    }
    const long long p_first = s.pos0 + k.u0 / a.group, p_last = s.pos0 + (k.u0 + k.n_u - 1) / a.group;
    const int key_a = (g >> 1) + 4 * (g & 1);           // key of S^T row g of a 16-key half

    int stage = 0;
    for (int c = c0; c < c_end; c += kFewWarps) {
        issue(c + (kFewStages - 1) * kFewWarps, stage == 0 ? kFewStages - 1 : stage - 1);
        cp_async_wait<kFewStages - 1>();
        __syncwarp();
        const unsigned char* st = ring + stage * kFewStageBytes;
        const long long j0 = static_cast<long long>(unit_chunk(k, c)) * kFewChunk;
        const uint32_t halves = (bad >> (2 * stage)) & 3u;
        const uint32_t have = ((halves & 1u) ? 0u : 0xffffu) | ((halves & 2u) ? 0u : 0xffff0000u);

        // rows 2 t, 2 t + 1 of each tile: the keys of this chunk they see
        uint32_t vis[NT][2];
        const bool full = have == 0xffffffffu && j0 + 31 <= p_first &&
                          (a.window == 0 || j0 > p_last - a.window || j0 + 31 < a.sinks);
        if (full) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) vis[nt][0] = vis[nt][1] = 0xffffffffu;
        } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const long long p = s.pos0 + (k.u0 + nt * 8 + 2 * t + b) / a.group;
                    vis[nt][b] = visible_bits(j0, p, a.window, a.sinks) & have;
                }
        }

        // V scales: lane = key; f16 of scale 2^(11 - E), 0 for keys without a page, no unit row or a
        // scale that is not a number (those keys' outputs are set below)
        float fac = 1.0f;
        uint32_t nan0, nan1;
        {
            uint32_t w = *reinterpret_cast<const uint32_t*>(st + kFewVs + lane * 4);
            const bool dead = !((have >> lane) & 1u) || j0 + lane > p_last;
            if (dead) w = 0;
            nan0 = __ballot_sync(0xffffffffu, (w & 0x7f80u) == 0x7f80u);
            nan1 = __ballot_sync(0xffffffffu, (w & 0x7f800000u) == 0x7f800000u);
            if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
            if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
            const uint32_t big = __reduce_max_sync(0xffffffffu, max(w & 0xffffu, w >> 16));
            const int e = static_cast<int>(big >> 7) - 127;
            if (big != 0 && e > E) {
                fac = E < e - 120 ? 0.0f : __uint_as_float(static_cast<uint32_t>(127 + E - e) << 23);
                E = e;
            }
            auto scaled = [&](uint32_t b) {            // bf16 bits -> f32 of value 2^(11 - E)
                const int ne = static_cast<int>(b >> 7) - E + 11;
                return b == 0 || ne <= 0 ? 0.0f : __uint_as_float((static_cast<uint32_t>(ne) << 23) | ((b & 0x7fu) << 16));
            };
            // slot of key 16 a + 4 i + t in the order its reader wants: 16 a + 4 t + i
            const int at = (lane & 16) | ((lane & 3) << 2) | ((lane >> 2) & 3);
            reinterpret_cast<__half*>(sm_vs[warp][0])[at] = __float2half_rn(scaled(w & 0xffffu));
            reinterpret_cast<__half*>(sm_vs[warp][1])[at] = __float2half_rn(scaled(w >> 16));
        }
        __syncwarp();

        // ---- scores ----
        float sc[NT][2][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
            uint32_t ka[4][4];              // A fragments of the four 16-dim steps
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
                const uint2 w = *reinterpret_cast<const uint2*>(st + kFewK + (mt * 16 + hi * 8 + key_a) * 32 + t * 8);
                uint32_t p0[4], p1[4];
                kv4_pairs(w.x, p0);
                kv4_pairs(w.y, p1);
                ka[0][hi] = p0[0], ka[0][2 + hi] = p0[1], ka[1][hi] = p0[2], ka[1][2 + hi] = p0[3];
                ka[2][hi] = p1[0], ka[2][2 + hi] = p1[1], ka[3][hi] = p1[2], ka[3][2 + hi] = p1[3];
            }
            const uint32_t wa = *reinterpret_cast<const uint32_t*>(st + kFewKs + (mt * 16 + key_a) * 4);
            const uint32_t wb = *reinterpret_cast<const uint32_t*>(st + kFewKs + (mt * 16 + 8 + key_a) * 4);
            const float ka0 = __uint_as_float(wa << 16), ka1 = __uint_as_float(wa & 0xffff0000u);
            const float kb0 = __uint_as_float(wb << 16), kb1 = __uint_as_float(wb & 0xffff0000u);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float d0[4] = {0.0f, 0.0f, 0.0f, 0.0f}, d1[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    mma_f16(d0, ka[ks], ql[nt][ks][0], ql[nt][ks][1]);
                    mma_f16(d1, ka[2 + ks], ql[nt][2 + ks][0], ql[nt][2 + ks][1]);
                }
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    mma_f16(d0, ka[ks], qh[nt][ks][0], qh[nt][ks][1]);
                    mma_f16(d1, ka[2 + ks], qh[nt][2 + ks][0], qh[nt][2 + ks][1]);
                }
                // the row's factor first: scale times raw sum could leave f32's range
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float f = qs[nt][j & 1];
                    sc[nt][mt][j] = fmaf(d1[j] * f, j < 2 ? ka1 : kb1, (d0[j] * f) * (j < 2 ? ka0 : kb0));
                }
            }
        }
        if (!full) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (!((vis[nt][j & 1] >> (mt * 16 + (j >> 1) * 8 + key_a)) & 1u)) sc[nt][mt][j] = -INFINITY;
        }

        // ---- softmax ----
        uint32_t ph[NT][2][2], pl[NT][2][2];
        float corr[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float mx = fmaxf(fmaxf(sc[nt][0][b], sc[nt][0][b + 2]), fmaxf(sc[nt][1][b], sc[nt][1][b + 2]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                const float mn = fmaxf(m[nt][b], mx);
                // nothing seen yet: exp2(-inf - 0) = 0 keeps every term 0
                const float base = mn == -INFINITY ? 0.0f : mn;
                corr[nt][b] = exp2f(m[nt][b] - base);
                m[nt][b] = mn;
                float sum = 0.0f;
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    sc[nt][mt][b] = exp2f(sc[nt][mt][b] - base + 12.0f);
                    sc[nt][mt][b + 2] = exp2f(sc[nt][mt][b + 2] - base + 12.0f);
                    sum += sc[nt][mt][b] + sc[nt][mt][b + 2];
                }
                l[nt][b] = fmaf(l[nt][b], corr[nt][b], sum);
                corr[nt][b] *= fac;
            }
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                uint32_t h0, l0, h1, l1;
                split_f16(sc[nt][mt][0], sc[nt][mt][1], h0, l0);
                split_f16(sc[nt][mt][2], sc[nt][mt][3], h1, l1);
                ph[nt][mt][0] = movmatrix_trans(h0);
                ph[nt][mt][1] = movmatrix_trans(h1);
                pl[nt][mt][0] = movmatrix_trans(l0);
                pl[nt][mt][1] = movmatrix_trans(l1);
            }
        }

        // ---- values ----
        uint32_t va[2][4][4];              // A fragments: 16-key step, dim tile
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const unsigned char* vp = st + kFewV + ks * 512 + t * 32 + g * 4;
            const uint32_t w0 = *reinterpret_cast<const uint32_t*>(vp), w1 = *reinterpret_cast<const uint32_t*>(vp + 128);
            const uint32_t w2 = *reinterpret_cast<const uint32_t*>(vp + 256);
            const uint32_t w3 = *reinterpret_cast<const uint32_t*>(vp + 384);
            const uint2 vs = *reinterpret_cast<const uint2*>(&sm_vs[warp][g >> 2][ks * 8 + t * 2]);
            // pairs along the keys: low and high halves of two keys' words side by side
            uint32_t d01[8], d23[8];
            kv4_pairs(__byte_perm(w0, w1, 0x5410), d01);
            kv4_pairs(__byte_perm(w0, w1, 0x7632), d01 + 4);
            kv4_pairs(__byte_perm(w2, w3, 0x5410), d23);
            kv4_pairs(__byte_perm(w2, w3, 0x7632), d23 + 4);
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                va[ks][mt][0] = h2_bits(__hmul2(bits_h2(d01[2 * mt]), bits_h2(vs.x)));
                va[ks][mt][1] = h2_bits(__hmul2(bits_h2(d01[2 * mt + 1]), bits_h2(vs.x)));
                va[ks][mt][2] = h2_bits(__hmul2(bits_h2(d23[2 * mt]), bits_h2(vs.y)));
                va[ks][mt][3] = h2_bits(__hmul2(bits_h2(d23[2 * mt + 1]), bits_h2(vs.y)));
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma_f16(d, va[0][mt], pl[nt][0][0], pl[nt][0][1]);
                mma_f16(d, va[1][mt], pl[nt][1][0], pl[nt][1][1]);
                mma_f16(d, va[0][mt], ph[nt][0][0], ph[nt][0][1]);
                mma_f16(d, va[1][mt], ph[nt][1][0], ph[nt][1][1]);
#pragma unroll
                for (int j = 0; j < 4; ++j) o[nt][mt][j] = fmaf(o[nt][mt][j], corr[nt][j & 1], d[j]);
            }
        if (nan0 | nan1) {                 // a seen key whose V group is not a number
            const uint32_t bits = g < 4 ? nan0 : nan1;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    if (vis[nt][b] & bits) {
#pragma unroll
                        for (int mt = 0; mt < 4; ++mt) o[nt][mt][b] = o[nt][mt][b + 2] = __uint_as_float(0x7fc00000u);
                    }
        }
        __syncwarp();
        stage = stage + 1 == kFewStages ? 0 : stage + 1;
    }
    cp_async_wait<0>();
    __syncthreads();

    // ---- join the warps: O as [unit row][dim], each warp's sums scaled back by 2^(E - 11) ----
    float* so = reinterpret_cast<float*>(few_smem) + warp * UR * (kHeadDim + 4);
    // 2^(E - 11) in two factors, so that neither leaves f32's range
    const int es = max(E - 11, -250), ea = es / 2, eb = es - ea;
    const float fa = __uint_as_float(static_cast<uint32_t>(127 + ea) << 23);
    const float fb = __uint_as_float(static_cast<uint32_t>(127 + eb) << 23);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            float sum = l[nt][b];
            sum += __shfl_xor_sync(0xffffffffu, sum, 4);
            sum += __shfl_xor_sync(0xffffffffu, sum, 8);
            sum += __shfl_xor_sync(0xffffffffu, sum, 16);
            const int u = nt * 8 + 2 * t + b;
            if (g == 0) {
                sm_m[warp][u] = m[nt][b];
                sm_l[warp][u] = sum;
            }
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
                *reinterpret_cast<float2*>(so + u * (kHeadDim + 4) + 8 * g + 2 * mt) =
                    make_float2(o[nt][mt][b] * fa * fb, o[nt][mt][b + 2] * fa * fb);
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
        const int ur = k.u0 + u, h = hk * a.group + ur % a.group;
        const long long row = s.row0 + ur / a.group;
        if (k.splits == 1) {
            const bool ok = L > 0.0f && isfinite(L);
            *reinterpret_cast<float4*>(a.out + row * a.out_ld + h * kHeadDim + d4 * 4) =
                ok ? make_float4(acc.x / L, acc.y / L, acc.z / L, acc.w / L) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        } else {
            float* p = a.part + ((row * a.heads + h) * a.S + sp) * kPartStride;
            if (d4 == 0) *reinterpret_cast<float2*>(p) = make_float2(mx, L);
            *reinterpret_cast<float4*>(p + 4 + d4 * 4) = acc;
        }
    }
}

inline size_t few_smem_bytes(int nt) {
    const size_t ring = size_t(kFewWarps) * kFewStages * kFewStageBytes;
    const size_t join = size_t(kFewWarps) * 8 * nt * (kHeadDim + 4) * sizeof(float);
    return ring > join ? ring : join;
}

}  // namespace dec

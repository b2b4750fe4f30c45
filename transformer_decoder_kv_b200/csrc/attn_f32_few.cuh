// Attention over f32 caches for units of one or two query rows (decoding tokens without grouped heads):
// k_attn_f32_few<R>, up to R unit rows; attn_f32_mma.cuh takes more.
//
// Bound by the cache's 512 bytes per key: 64 streams x 4096 keys x 16 heads take 327 us, 6.6 TB/s, and 256 x
// 8192 x 2 303 us, 7.1 TB/s. At HBM's rate a key leaves an SM time for about 90 instructions, and on CUDA cores
// a key takes about 8 per unit row, so nothing is staged and no product goes to the tensor cores: a warp loads
// 16 keys of K and of V (a row per 16 lanes, 16 bytes a lane) straight into registers, 8 KB in flight
// per warp, the next chunk's K while it works on V and the next V while it works on K.
//
//   scores   each lane multiplies its 4 dims; the 8 partial sums of a half-warp's 8 keys are added
//            across its 16 lanes by exchanging halves (8 shuffles for 8 keys), which leaves each lane
//            the score of one key.
//   softmax  running maximum and sum per unit row and warp, f32 throughout.
//   values   each key's weight goes back to its half-warp by one shuffle, 4 fma per key and lane.
//
// A warp owns every fourth chunk of the block's range; warps meet only at the end.
#pragma once

#include "attn_rows.cuh"

namespace dec {

constexpr int kF32Chunk = 16;
constexpr int kF32Warps = 4;

// (One row: five blocks per SM instead of four, 32 streams x 448 keys x 20 heads 30.6 -> 25.6 us; six spill.)
template <int R>
static __global__ void __launch_bounds__(kF32Warps * 32, R == 1 ? 5 : 4) k_attn_f32_few(const RowsAttnArgs a) {
    __shared__ float sm_m[kF32Warps][R], sm_l[kF32Warps][R];
    __shared__ __align__(16) float sm_o[kF32Warps][R][kHeadDim];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, half = lane >> 4, d4 = lane & 15;
    pdl_wait();
    const StreamRows s = stream_rows(a.r, a.v, blockIdx.z);
    const int n_tiles = gridDim.y / a.v.heads;
    const int hk = blockIdx.y / n_tiles;
    const UnitKeys k = unit_keys<R, kF32Chunk>(a, s, blockIdx.y % n_tiles);
    const int sp = blockIdx.x;
    if (k.n_u == 0 || sp >= k.splits) return;
    const int c_end = split_begin(k, sp + 1);
    const int end = static_cast<int>(k.end);

    // (scores are taken to the log2 domain)
    float4 q[R];
    float o[R][4], m[R], l[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        q[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (r < k.n_u) {
            const int ur = k.u0 + r, h = hk * a.group + ur % a.group;
            q[r] = *(reinterpret_cast<const float4*>(a.q + static_cast<long long>(s.row0 + ur / a.group) * a.q_ld +
                                                     h * kHeadDim) + d4);
        }
        o[r][0] = o[r][1] = o[r][2] = o[r][3] = l[r] = 0.0f;
        m[r] = -INFINITY;
    }

    const int* tab = a.v.table ? a.v.table + s.slot * a.v.pages_per_slot : nullptr;
    const long long page_floats = static_cast<long long>(a.v.heads) * a.v.page_rows * kHeadDim;
    const long long head_off = static_cast<long long>(hk) * a.v.page_rows * kHeadDim + lane * 4;
    const int pr_mask = a.v.shift == 31 ? 0x7fffffff : a.v.page_rows - 1;
    // Offset of a chunk's rows in the pools (this lane's part), -1 where there are no rows.
    auto place = [&](int c) -> long long {
        if (c >= c_end) return -1;
        const int j = unit_chunk(k, c) * kF32Chunk;
        if (j >= end) return -1;
        const int p = tab ? tab[j >> a.v.shift] : s.slot * a.v.pages_per_slot + (j >> a.v.shift);
        if (static_cast<unsigned>(p) >= static_cast<unsigned>(a.v.n_pages)) return -1;
        return p * page_floats + head_off + static_cast<long long>(j & pr_mask) * kHeadDim;
    };
    // Keys 2 i + half of a chunk; rows at or beyond `end` are not read.
    auto load = [&](float4 (&x)[8], const float* pool, long long at, int c) {
        const int n = c < c_end ? end - unit_chunk(k, c) * kF32Chunk - half : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (at >= 0 && 2 * i < n) x[i] = __ldg(reinterpret_cast<const float4*>(pool + at + i * 2 * kHeadDim));
        }
    };

    const long long p_first = s.pos0 + k.u0 / a.group, p_last = s.pos0 + (k.u0 + k.n_u - 1) / a.group;
    const int full_hi = static_cast<int>(min(p_first - (kF32Chunk - 1), 0x7fffff00ll));
    const int full_lo = a.window == 0 ? 0 : static_cast<int>(max(0ll, min(p_last - a.window + 1, 0x7fffff00ll)));
    // after the exchange this lane holds key 2 ((lane >> 1) & 7, bits in the order 3 2 1) + half
    const int my_i = ((lane >> 3) & 1) * 4 + ((lane >> 2) & 1) * 2 + ((lane >> 1) & 1);
    const int my_key = 2 * my_i + half;

    int c = split_begin(k, sp) + warp;
    float4 kk[8], vv[8];
    long long at = place(c), at_next = place(c + kF32Warps);
    load(kk, a.k, at, c);
    load(vv, a.vv, at, c);
    for (; c < c_end; c += kF32Warps) {
        const int j0 = unit_chunk(k, c) * kF32Chunk;
        const bool full = at >= 0 && j0 <= full_hi && j0 + kF32Chunk <= end && (j0 >= full_lo || j0 + kF32Chunk <= a.sinks);
        float sc[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float part[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                part[i] = fmaf(kk[i].w, q[r].w, fmaf(kk[i].z, q[r].z, fmaf(kk[i].y, q[r].y, kk[i].x * q[r].x)));
            const bool up8 = lane & 8, up4 = lane & 4, up2 = lane & 2;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float send = up8 ? part[i] : part[i + 4], keep = up8 ? part[i + 4] : part[i];
                part[i] = keep + __shfl_xor_sync(0xffffffffu, send, 8);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float send = up4 ? part[i] : part[i + 2], keep = up4 ? part[i + 2] : part[i];
                part[i] = keep + __shfl_xor_sync(0xffffffffu, send, 4);
            }
            const float send = up2 ? part[0] : part[1], keep = up2 ? part[1] : part[0];
            part[0] = keep + __shfl_xor_sync(0xffffffffu, send, 2);
            sc[r] = (part[0] + __shfl_xor_sync(0xffffffffu, part[0], 1)) * (0.125f * kLog2e);
        }
        load(kk, a.k, at_next, c + kF32Warps);
        const long long at_after = place(c + 2 * kF32Warps);
        if (!full) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const long long p = s.pos0 + (k.u0 + r) / a.group, j = j0 + my_key;
                const bool vis = at >= 0 && j <= p && j < end && (a.window == 0 || j > p - a.window || j < a.sinks);
                if (!vis) sc[r] = -INFINITY;
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float mx = fmaxf(sc[r], __shfl_xor_sync(0xffffffffu, sc[r], 2));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float mn = fmaxf(m[r], mx), base = mn == -INFINITY ? 0.0f : mn;
            const float corr = exp2f(m[r] - base), w = exp2f(sc[r] - base);
            m[r] = mn;
            l[r] = fmaf(l[r], corr, w);          // each key is held by two lanes: halved at the end
#pragma unroll
            for (int j = 0; j < 4; ++j) o[r][j] *= corr;
            sc[r] = w;
        }
        // a key without weight adds nothing, whatever it holds
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float w = __shfl_sync(0xffffffffu, sc[r], (lane & 16) | (i << 1));
                if (w != 0.0f) {
                    o[r][0] = fmaf(w, vv[i].x, o[r][0]);
                    o[r][1] = fmaf(w, vv[i].y, o[r][1]);
                    o[r][2] = fmaf(w, vv[i].z, o[r][2]);
                    o[r][3] = fmaf(w, vv[i].w, o[r][3]);
                }
            }
        load(vv, a.vv, at_next, c + kF32Warps);
        at = at_next;
        at_next = at_after;
    }

    // ---- join the half-warps, then the warps ----
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float sum = warp_sum(l[r]) * 0.5f;
        if (lane == 0) {
            sm_m[warp][r] = m[r];
            sm_l[warp][r] = sum;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) o[r][j] += __shfl_xor_sync(0xffffffffu, o[r][j], 16);
        if (half == 0) *reinterpret_cast<float4*>(&sm_o[warp][r][d4 * 4]) = make_float4(o[r][0], o[r][1], o[r][2], o[r][3]);
    }
    __syncthreads();
    for (int x = tid; x < k.n_u * 16; x += kF32Warps * 32) {
        const int u = x >> 4, e4 = x & 15;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kF32Warps; ++w) mx = fmaxf(mx, sm_m[w][u]);
        float L = 0.0f;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kF32Warps; ++w) {
            const float e = sm_m[w][u] == -INFINITY ? 0.0f : exp2f(sm_m[w][u] - mx);
            L = fmaf(e, sm_l[w][u], L);
            const float4 ow = *reinterpret_cast<const float4*>(&sm_o[w][u][e4 * 4]);
            if (e != 0.0f) {
                acc.x = fmaf(e, ow.x, acc.x);
                acc.y = fmaf(e, ow.y, acc.y);
                acc.z = fmaf(e, ow.z, acc.z);
                acc.w = fmaf(e, ow.w, acc.w);
            }
        }
        store_unit_row(a, k, s, hk, sp, u, e4, mx, L, acc);
    }
}

}  // namespace dec

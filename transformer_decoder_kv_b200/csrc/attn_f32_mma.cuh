// Attention over f32 caches for units of several query rows (the heads of a group that share a K/V
// head, a few tokens of a stream): k_attn_f32_mma<NT>, up to 8 NT unit rows.
//
// Bound by the cache's 512 bytes per key, as the CUDA-core kernel for fewer rows, whose 8 instructions per
// key and row are too many from a few rows on. Here the products go to the tensor cores (mma.sync
// m16n8k16, f16; a key meets 3 to 16 rows once, so its split halves stay in the registers of the warp
// that loaded it, and tcgen05's tiles of 128 rows would stand nearly empty): K, V and Q are scaled by
// powers of two and split into f16 high and low parts (22 bits), three products each, f32 sums;
// the product of two low parts, below 2^-22, is left out. About 23 instructions per key; 256 streams x
// 8192 keys x 2 heads take 400 us with 7 rows (5.4 TB/s; 689 on CUDA cores) and 498 with 16.
//
// Fragments as in the 4-bit kernel: S^T = K Q^T with keys in the rows, softmax per column, P^T by movmatrix,
// O^T += V^T P^T with 8 dims per quad lane and each chunk's sums in fresh accumulators. A 16-byte load is
// a key's four dims of one 16-dim step (K), or half of its 8 dims (V); V's pairs along the keys come from
// the conversion of two keys' values at once.
//
// The powers of two of K and V stand while every key's largest value stays between 2^-2 and f16's end, where
// 22 bits are left of it; a chunk outside (the first one, to begin with, and one with keys that no row sees)
// is looked at more closely and may set them anew. A chunk whose keys lie 2^12 apart, or that holds a NaN or
// an infinity, is computed by a plain f32 loop: a matrix product would take it to rows that do not see it. From
// a plain chunk on, or from one that needs a smaller power of two than those before, the sums are kept in a
// scale of their own, 2^-16, in which f32 holds those of all finite values.
#pragma once

#include "attn_f32_few.cuh"
#include "attn_kv4_few.cuh"

namespace dec {

constexpr int kMmaOwnScale = 26;           // o is held times 2^(10 - 26)
constexpr int kMmaSpan = 12;               // keys' largest values from 2^e down to 2^(e - 12)

template <int NT>
static __global__ void __launch_bounds__(kF32Warps * 32) k_attn_f32_mma(const RowsAttnArgs a) {
    constexpr int UR = 8 * NT;
    __shared__ float sm_m[kF32Warps][UR], sm_l[kF32Warps][UR];
    __shared__ __align__(16) float sm_o[kF32Warps][UR][kHeadDim + 4];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    pdl_wait();
    const StreamRows s = stream_rows(a.r, a.v, blockIdx.z);
    const int n_tiles = gridDim.y / a.v.heads;
    const int hk = blockIdx.y / n_tiles;
    const UnitKeys k = unit_keys<UR, kF32Chunk>(a, s, blockIdx.y % n_tiles);
    const int sp = blockIdx.x;
    if (k.n_u == 0 || sp >= k.splits) return;
    const int c_end = split_begin(k, sp + 1);
    const int end = static_cast<int>(k.end);

    // ---- the chunks' loads ----
    const int* tab = a.v.table ? a.v.table + s.slot * a.v.pages_per_slot : nullptr;
    const long long page_floats = static_cast<long long>(a.v.heads) * a.v.page_rows * kHeadDim;
    const long long head_off = static_cast<long long>(hk) * a.v.page_rows * kHeadDim;
    const int pr_mask = a.v.shift == 31 ? 0x7fffffff : a.v.page_rows - 1;
    const long long p_first = s.pos0 + k.u0 / a.group, p_last = s.pos0 + (k.u0 + k.n_u - 1) / a.group;
    // keys below, past the sinks: no row sees them
    const int seen_lo = a.window > 0 ? static_cast<int>(max(0ll, min(p_first - a.window + 1, 0x7fffff00ll))) : 0;
    // Offset of a chunk's first row in the pools, -1 where there are no rows.
    auto place = [&](int c) -> long long {
        if (c >= c_end) return -1;
        const int j = unit_chunk(k, c) * kF32Chunk;
        if (j >= end) return -1;
        const int p = tab ? tab[j >> a.v.shift] : s.slot * a.v.pages_per_slot + (j >> a.v.shift);
        if (static_cast<unsigned>(p) >= static_cast<unsigned>(a.v.n_pages)) return -1;
        return p * page_floats + head_off + static_cast<long long>(j & pr_mask) * kHeadDim;
    };
    auto row4 = [&](const float* pool, long long at, int j0, int key, int d) {
        const int j = j0 + key;
        const bool live = at >= 0 && j < end && (j >= seen_lo || j < a.sinks);
        return live ? __ldg(reinterpret_cast<const float4*>(pool + at + key * kHeadDim + d)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    };
    float4 kk[2][4], vv[4][2];
    auto load_k = [&](int c, long long at) {       // keys g, g + 8; dims 16 ks + 4 t
        const int j0 = c < c_end ? unit_chunk(k, c) * kF32Chunk : 0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) kk[h][ks] = row4(a.k, at, j0, g + 8 * h, 16 * ks + 4 * t);
    };
    auto load_v = [&](int c, long long at) {       // keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9; dims 8 g
        const int j0 = c < c_end ? unit_chunk(k, c) * kF32Chunk : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) vv[i][h] = row4(a.vv, at, j0, 2 * t + (i & 1) + 8 * (i >> 1), 8 * g + 4 * h);
    };
    int c = split_begin(k, sp) + warp;
    long long at = place(c), at_next = place(c + kF32Warps);
    load_k(c, at);
    load_v(c, at);

    // ---- Q^T fragments: column g of each tile ----
    uint32_t qh[NT][4][2], ql[NT][4][2];
    float qs[NT][2];                               // score factors of rows 8 nt + 2 t, + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int u = nt * 8 + g;
        float4 x[4];
        float mx = 0.0f;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            x[ks] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (u < k.n_u) {
                const int ur = k.u0 + u, h = hk * a.group + ur % a.group;
                x[ks] = *reinterpret_cast<const float4*>(a.q + static_cast<long long>(s.row0 + ur / a.group) * a.q_ld +
                                                         h * kHeadDim + 16 * ks + 4 * t);
            }
            mx = fmaxf(mx, fmaxf(fmaxf(fabsf(x[ks].x), fabsf(x[ks].y)), fmaxf(fabsf(x[ks].z), fabsf(x[ks].w))));
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // the row's largest element goes to [2^10, 2^11); rows below 2^-100 are taken as that small
        const int e = max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -100);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 10 - e) << 23);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - 10 + e) << 23) * (0.125f * kLog2e);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            split_f16(x[ks].x * up, x[ks].y * up, qh[nt][ks][0], ql[nt][ks][0]);
            split_f16(x[ks].z * up, x[ks].w * up, qh[nt][ks][1], ql[nt][ks][1]);
        }
        qs[nt][0] = __shfl_sync(0xffffffffu, down, 8 * t);
        qs[nt][1] = __shfl_sync(0xffffffffu, down, 8 * t + 4);
    }

    // ---- running state: unit rows 8 nt + 2 t + b; O^T dims 8 g + 2 mt, + 1 ----
    float m[NT][2], rf[NT][2], l[NT][2], o[NT][4][4];       // maximum, reference of the weights, sum, values
    int ek = -100, E = -100;                       // K is held times 2^(10 - ek), V times 2^(10 - E)
    bool own = false;                              // o is held times 2^-16, or else as V
    float kscale = __uint_as_float(static_cast<uint32_t>(127 - 110) << 23);      // 2^(ek - 10)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            m[nt][b] = rf[nt][b] = -INFINITY;
            l[nt][b] = 0.0f;
        }
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[nt][mt][j] = 0.0f;
    }
    const int full_hi = static_cast<int>(min(p_first - (kF32Chunk - 1), 0x7fffff00ll));
    const int full_lo = a.window == 0 ? 0 : static_cast<int>(max(0ll, min(p_last - a.window + 1, 0x7fffff00ll)));
    auto pow2 = [](int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); };
    // f16 parts of two values times `up`; `big` follows the largest high part (NaN stays)
    auto halves = [](float x, float y, float up, uint32_t& hi, uint32_t& lo, __half2& big) {
        const float2 v = mul2(make_float2(x, y), make_float2(up, up));
        const __half2 h = __floats2half2_rn(v.x, v.y);
        const float2 f = __half22float2(h);
        hi = h2_bits(h);
        lo = h2_bits(__floats2half2_rn(v.x - f.x, v.y - f.y));
        big = __hmax2_nan(big, __habs2(h));
    };
    for (; c < c_end; c += kF32Warps) {
        const int j0 = unit_chunk(k, c) * kF32Chunk;
        const bool full = at >= 0 && j0 <= full_hi && j0 + kF32Chunk <= end && (j0 >= full_lo || j0 + kF32Chunk <= a.sinks);
        uint32_t vis[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                vis[nt][b] = 0xffffu;
                if (!full) {
                    const long long p = s.pos0 + (k.u0 + nt * 8 + 2 * t + b) / a.group;
                    vis[nt][b] = at < 0 ? 0u : visible_bits(j0, min(p, static_cast<long long>(end) - 1), a.window, a.sinks) & 0xffffu;
                    // (the window is measured from the row's own position, which may lie past the slot's end)
                    if (a.window > 0 && p >= end) vis[nt][b] &= visible_bits(j0, p, a.window, a.sinks);
                }
            }

        // ---- K and V to f16 ----
        uint32_t kh[4][4], kl[4][4], vh[4][4], vl[4][4];      // A fragments per 16-dim step, per dim tile
        float fac = 1.0f;
        bool plain = false;
        auto convert = [&]() {
            const float ku = pow2(10 - ek), vu = pow2(10 - E);
            const __half2 zero = __float2half2_rn(0.0f);
            __half2 bk[2] = {zero, zero}, bv[2] = {zero, zero};          // largest halves by key
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    halves(kk[h][ks].x, kk[h][ks].y, ku, kh[ks][h], kl[ks][h], bk[h]);
                    halves(kk[h][ks].z, kk[h][ks].w, ku, kh[ks][2 + h], kl[ks][2 + h], bk[h]);
                }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i) {      // keys 2 t, 2 t + 1, then + 8
                    const float4 x = vv[2 * i][h], y = vv[2 * i + 1][h];
                    halves(x.x, y.x, vu, vh[2 * h][2 * i], vl[2 * h][2 * i], bv[i]);
                    halves(x.y, y.y, vu, vh[2 * h][2 * i + 1], vl[2 * h][2 * i + 1], bv[i]);
                    halves(x.z, y.z, vu, vh[2 * h + 1][2 * i], vl[2 * h + 1][2 * i], bv[i]);
                    halves(x.w, y.w, vu, vh[2 * h + 1][2 * i + 1], vl[2 * h + 1][2 * i + 1], bv[i]);
                }
            // (of the lane's part of each key: a smaller part is looked at, too; a NaN fails the first test)
            const __half2 big = __hmax2_nan(__hmax2_nan(bk[0], bk[1]), __hmax2_nan(bv[0], bv[1]));
            const __half2 low = __hmin2(__hmin2(bk[0], bk[1]), __hmin2(bv[0], bv[1]));
            const bool fits = __hblt2(big, bits_h2(0x7c007c00u)) && __hbge2(low, bits_h2(0x34003400u));
            return __any_sync(0xffffffffu, !fits);
        };
        if (convert()) {
            // each key's largest magnitude, as bits (a NaN's are above all); the smallest of those above 0, less 1
            uint32_t top[2], least[2];             // K, V
            auto mag = [](const float4& x) {
                return max(max(__float_as_uint(fabsf(x.x)), __float_as_uint(fabsf(x.y))),
                           max(__float_as_uint(fabsf(x.z)), __float_as_uint(fabsf(x.w))));
            };
            top[0] = top[1] = 0u;
            least[0] = least[1] = 0xffffffffu;
#pragma unroll
            for (int i = 0; i < 6; ++i) {
                uint32_t x;
                if (i < 2) {
                    x = max(max(mag(kk[i][0]), mag(kk[i][1])), max(mag(kk[i][2]), mag(kk[i][3])));
                    x = max(x, __shfl_xor_sync(0xffffffffu, x, 1));
                    x = max(x, __shfl_xor_sync(0xffffffffu, x, 2));
                } else {
                    x = max(mag(vv[i - 2][0]), mag(vv[i - 2][1]));
                    x = max(x, __shfl_xor_sync(0xffffffffu, x, 4));
                    x = max(x, __shfl_xor_sync(0xffffffffu, x, 8));
                    x = max(x, __shfl_xor_sync(0xffffffffu, x, 16));
                }
                top[i >= 2] = max(top[i >= 2], x);
                least[i >= 2] = min(least[i >= 2], x - 1u);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                top[i] = __reduce_max_sync(0xffffffffu, top[i]);
                least[i] = __reduce_min_sync(0xffffffffu, least[i]);
                const int t2 = static_cast<int>(top[i] & 0x7f800000u) - (kMmaSpan << 23);
                plain |= top[i] >= 0x7f800000u || (t2 > 0 && least[i] < static_cast<uint32_t>(t2) - 1u);
            }
            if (!plain) {
                if (top[0]) ek = max(static_cast<int>(top[0] >> 23) - 127, -100);
                kscale = pow2(ek - 10);
                const int e = max(static_cast<int>(top[1] >> 23) - 127, -100);
                if (!own && top[1]) {
                    // smaller than the sums' scale leaves bits for, or far from 1: the sums' own scale
                    own = e > 40 || e < -40 || static_cast<int>(least[1] >> 23) - 127 < E - kMmaSpan;
                    const int to = own ? kMmaOwnScale : max(E, e);
                    fac = E < to - 120 ? 0.0f : pow2(E - to);              // (E is -100 before any value)
                    E = max(E, e);
                }
                if (own && top[1]) E = e;
                convert();
            }
        }
        const long long at_after = place(c + 2 * kF32Warps);

        if (!plain) {
            load_k(c + kF32Warps, at_next);
            load_v(c + kF32Warps, at_next);
            // ---- scores of keys g, g + 8 ----
            float sc[NT][2][2];                    // [tile][row b][key]
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    mma_f16(d, kl[ks], qh[nt][ks][0], qh[nt][ks][1]);
                    mma_f16(d, kh[ks], ql[nt][ks][0], ql[nt][ks][1]);
                }
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) mma_f16(d, kh[ks], qh[nt][ks][0], qh[nt][ks][1]);
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const float x = (d[2 * j + b] * qs[nt][b]) * kscale;
                        sc[nt][b][j] = full || ((vis[nt][b] >> (g + 8 * j)) & 1u) ? x : -INFINITY;
                    }
            }
            // ---- softmax ----
            uint32_t ph[NT][2], pl[NT][2];
            float corr[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    float mx = fmaxf(sc[nt][b][0], sc[nt][b][1]);
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    const float mn = fmaxf(m[nt][b], mx);
                    // the weights' reference: 12 below the maximum, as in the 4-bit kernel
                    const float ref = mn == -INFINITY ? 0.0f : fabsf(mn) < 65536.0f ? mn - 12.0f : mn;
                    corr[nt][b] = ex2(rf[nt][b] - ref);
                    m[nt][b] = mn;
                    rf[nt][b] = mn == -INFINITY ? -INFINITY : ref;
                    sc[nt][b][0] = ex2(sc[nt][b][0] - ref);
                    sc[nt][b][1] = ex2(sc[nt][b][1] - ref);
                    l[nt][b] = fmaf(l[nt][b], corr[nt][b], sc[nt][b][0] + sc[nt][b][1]);
                    corr[nt][b] *= fac;
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t h, lo;
                    split_f16(sc[nt][0][j], sc[nt][1][j], h, lo);
                    ph[nt][j] = movmatrix_trans(h);
                    pl[nt][j] = movmatrix_trans(lo);
                }
            }
            // ---- values ----
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) {
                    float d[4];
                    mma_f16(d, vl[mt], ph[nt][0], ph[nt][1], 0.0f, 0.0f, 0.0f, 0.0f);
                    mma_f16(d, vh[mt], pl[nt][0], pl[nt][1]);
                    mma_f16(d, vh[mt], ph[nt][0], ph[nt][1]);
                    if (own) {
                        const float df = pow2(E - kMmaOwnScale);
#pragma unroll
                        for (int j = 0; j < 4; ++j) d[j] *= df;
                    }
#pragma unroll
                    for (int j = 0; j < 4; j += 2) {
                        const float2 y = fma2(make_float2(o[nt][mt][j], o[nt][mt][j + 1]), make_float2(corr[nt][0], corr[nt][1]),
                                              make_float2(d[j], d[j + 1]));
                        o[nt][mt][j] = y.x;
                        o[nt][mt][j + 1] = y.y;
                    }
                }
        } else {
            // ---- plain loop: every quad lane takes all keys of its rows, lanes g = 0 their sums ----
            const float vs = pow2(10 - kMmaOwnScale);
            if (!own) {
                own = true;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                        for (int j = 0; j < 4; ++j) o[nt][mt][j] *= pow2(E - kMmaOwnScale);
            }
            for (int x = 0; x < kF32Chunk; ++x) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        if (!((vis[nt][b] >> x) & 1u)) continue;
                        const int ur = k.u0 + min(nt * 8 + 2 * t + b, k.n_u - 1), h = hk * a.group + ur % a.group;
                        const float* q = a.q + static_cast<long long>(s.row0 + ur / a.group) * a.q_ld + h * kHeadDim;
                        const float* kr = a.k + at + x * kHeadDim;
                        float sum = 0.0f;
                        for (int d = 0; d < kHeadDim; ++d) sum = fmaf(kr[d], q[d], sum);
                        sum *= 0.125f * kLog2e;
                        const float mn = fmaxf(m[nt][b], sum);
                        const float ref = mn == -INFINITY ? 0.0f : fabsf(mn) < 65536.0f ? mn - 12.0f : mn;
                        const float cr = ex2(rf[nt][b] - ref), w = ex2(sum - ref);
                        m[nt][b] = mn;
                        rf[nt][b] = mn == -INFINITY ? -INFINITY : ref;
                        l[nt][b] = fmaf(l[nt][b], cr, g == 0 ? w : 0.0f);
                        const float* vr = a.vv + at + x * kHeadDim + 8 * g;
#pragma unroll
                        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                float& oi = o[nt][mt][2 * j + b];
                                oi *= cr;
                                if (w != 0.0f) oi = fmaf(w, vr[2 * mt + j] * vs, oi);
                            }
                    }
            }
            __syncwarp();
            load_k(c + kF32Warps, at_next);
            load_v(c + kF32Warps, at_next);
        }
        at = at_next;
        at_next = at_after;
    }

    // ---- join the warps ----
    const float back = pow2((own ? kMmaOwnScale : E) - 10);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            float sum = l[nt][b];
            sum += __shfl_xor_sync(0xffffffffu, sum, 4);
            sum += __shfl_xor_sync(0xffffffffu, sum, 8);
            sum += __shfl_xor_sync(0xffffffffu, sum, 16);
            const int u = nt * 8 + 2 * t + b;
            const RowScale f = row_scale(m[nt][b], rf[nt][b]);
            if (g == 0) {
                sm_m[warp][u] = f.ref;
                sm_l[warp][u] = sum * f.mul;
            }
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
                *reinterpret_cast<float2*>(&sm_o[warp][u][8 * g + 2 * mt]) =
                    make_float2(o[nt][mt][b] * (back * f.mul), o[nt][mt][b + 2] * (back * f.mul));
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

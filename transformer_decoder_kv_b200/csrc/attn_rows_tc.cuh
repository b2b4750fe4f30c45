// Attention of many query rows per K/V head (prompt chunks, whole prompts) on the 5th-generation
// tensor cores: k_attn_rows_tc<KV4>, units of 128 unit rows against tiles of 128 keys.
//
//   S = Q K^T   tcgen05.mma kind::f16, M = 128 unit rows, N = 128 keys, accumulators in TMEM. Q is
//               scaled by a power of two per row and split into f16 high and low parts (22 bits). K of
//               a 4-bit cache is code times scale, 3 + 8 significant bits: exact in f16 after a power
//               of two per tile; K of an f32 cache is scaled and split like Q (the product of the two
//               low parts, below 2^-22, is left out).
//   softmax     two threads per row, 64 columns each: running maximum (joined through shared memory),
//               p = exp2(s - m + 12), f32 sums; p in f16 high and low parts goes back to TMEM over the
//               scores it came from.
//   O = P V     A = P from TMEM, B = V as it lies (rows of 64 dims: an MN-major operand), N = 64. Each
//               tile's product is read back and added to the running f32 sums in registers, scaled by
//               the change of the maximum, so that the tensor cores' truncation does not build up.
//
// A block (256 threads, two per SM) goes through load, unpack, MMA, softmax, MMA, add one after the
// other; the other block of the SM fills the gaps. An M128 N128 K16 MMA takes 65 SM cycles and an
// M128 N64 K16 one 45 to 49 (measured), 1240 per tile of a 4-bit cache; the softmax's instructions, about
// 8 per score, are the larger part of a tile's time.
//
// A tile that holds a NaN or an infinity in K or V, at a position that some row sees, is computed by a
// plain f32 loop instead: in a matrix product it would reach the rows that do not see it.
#pragma once

#include "attn_kv4_few.cuh"
#include "head_tc.cuh"

namespace dec {

constexpr int kRtRows = 128, kRtKeys = 128, kRtThreads = 256;
constexpr int kRtPlane = kRtRows * 128;           // one f16 operand plane: 128 rows of 64 dims
constexpr uint32_t kRtTmemCols = 256;             // S / P 0..127, O 128..191
template <bool KV4>
constexpr int rt_smem_bytes() {
    return (2 + (KV4 ? 2 : 4)) * kRtPlane + 1024;
}

__device__ __forceinline__ void umma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// A from TMEM: 128 lanes, two consecutive k per 32-bit column
__device__ __forceinline__ void umma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// f32 accumulator, f16 operands, M = 128, N = n; b_mn: B is given as rows of N values per k
__host__ __device__ constexpr uint32_t idesc_f16(int n, bool b_mn) {
    return (1u << 4) | (uint32_t(b_mn) << 16) | (uint32_t(n >> 3) << 17) | (uint32_t(128 >> 4) << 24);
}

__device__ __forceinline__ void tmem_ld32(uint32_t addr, float (&r)[32]) {
    uint32_t x[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]), "=r"(x[8]),
          "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15]), "=r"(x[16]),
          "=r"(x[17]), "=r"(x[18]), "=r"(x[19]), "=r"(x[20]), "=r"(x[21]), "=r"(x[22]), "=r"(x[23]), "=r"(x[24]),
          "=r"(x[25]), "=r"(x[26]), "=r"(x[27]), "=r"(x[28]), "=r"(x[29]), "=r"(x[30]), "=r"(x[31])
        : "r"(addr)
        : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = __uint_as_float(x[i]);
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&x)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(x[0]),
        "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]), "r"(x[8]), "r"(x[9]), "r"(x[10]),
        "r"(x[11]), "r"(x[12]), "r"(x[13]), "r"(x[14]), "r"(x[15]), "r"(x[16]), "r"(x[17]), "r"(x[18]), "r"(x[19]),
        "r"(x[20]), "r"(x[21]), "r"(x[22]), "r"(x[23]), "r"(x[24]), "r"(x[25]), "r"(x[26]), "r"(x[27]), "r"(x[28]),
        "r"(x[29]), "r"(x[30]), "r"(x[31]), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void pair_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// One row's (or key's) 16-byte chunk c of a 128-byte-swizzled operand plane.
__device__ __forceinline__ uint4* rt_chunk(unsigned char* plane, int row, int c) {
    return reinterpret_cast<uint4*>(plane + row * 128 + ((c ^ (row & 7)) << 4));
}
// Dims 8 w .. 8 w + 7 of a row in two f16 planes. The 4-bit cache's words unpack to the order
// 0 4 1 5 2 6 3 7, so its queries are laid out in that order too (PERM).
template <bool PERM>
__device__ __forceinline__ void rt_store_split(unsigned char* hi, unsigned char* lo, int row, int w, const float* x) {
    uint4 h, l;
    constexpr int o[8] = {0, PERM ? 4 : 1, PERM ? 1 : 2, PERM ? 5 : 3, PERM ? 2 : 4, PERM ? 6 : 5, PERM ? 3 : 6, 7};
    split_f16(x[o[0]], x[o[1]], h.x, l.x);
    split_f16(x[o[2]], x[o[3]], h.y, l.y);
    split_f16(x[o[4]], x[o[5]], h.z, l.z);
    split_f16(x[o[6]], x[o[7]], h.w, l.w);
    *rt_chunk(hi, row, w) = h;
    *rt_chunk(lo, row, w) = l;
}

// Values of dims d .. d + 3 of one cached row, as f32.
template <bool KV4>
__device__ __forceinline__ float4 rt_row4(const RowsAttnArgs& a, bool v, int page, int hk, int pr, int d) {
    if (!KV4) {
        const float* pool = v ? a.vv : a.k;
        return *reinterpret_cast<const float4*>(pool + kvf_block(a.v, page, hk) + static_cast<long long>(pr) * kHeadDim + d);
    }
    const unsigned char* blk = a.cache + kv4_block(a.v, page, hk) + (v ? a.v.page_rows * kKv4RowBytes : 0);
    const int w = d >> 3;
    uint32_t x = *reinterpret_cast<const uint32_t*>(blk + pr * 32 + (v ? w : (w & 3) * 2 + (w >> 2)) * 4);
    if (v) x = ((x >> 2) & 0x3fff3fffu) | ((x << 14) & 0xc000c000u);
    x >>= (d & 4) * 4;
    const uint16_t sb = *reinterpret_cast<const uint16_t*>(blk + a.v.page_rows * 32 + pr * 4 + (w >> 2) * 2);
    const float s = __uint_as_float(static_cast<uint32_t>(sb) << 16);
    auto val = [&](int i) { return s * static_cast<float>(static_cast<int>((x >> (4 * i)) & 15u) - 8); };
    return make_float4(val(0), val(1), val(2), val(3));
}

template <bool KV4>
static __global__ void __launch_bounds__(kRtThreads, 2) k_attn_rows_tc(const RowsAttnArgs a) {
    extern __shared__ unsigned char rt_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(rt_raw) + 1023) &
                                                           ~static_cast<uintptr_t>(1023));
    unsigned char* sQ = smem;                                    // high, low
    unsigned char* sK = smem + 2 * kRtPlane;                     // high (, low)
    unsigned char* sV = sK + (KV4 ? 1 : 2) * kRtPlane;
    __shared__ __align__(8) uint64_t bar_s, bar_o;
    __shared__ uint32_t s_tmem;
    __shared__ float sm_f[kRtRows], sm_x[2][kRtRows];            // row factors; column halves' maxima, sums
    __shared__ uint32_t sm_kmax[2][8], sm_vmax[2][8], sm_bad[2][8], sm_nan[2][8];   // of a tile, per loading warp
    __shared__ int s_fail;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const StreamRows s = stream_rows(a.r, a.v, blockIdx.z);
    const int n_tiles = gridDim.y / a.v.heads;
    const int hk = blockIdx.y / n_tiles;
    const UnitKeys k = unit_keys<kRtRows, kRtKeys>(a, s, blockIdx.y % n_tiles);
    const int sp = blockIdx.x;
    if (k.n_u == 0 || sp >= k.splits) return;
    const int c0 = split_begin(k, sp), c_end = split_begin(k, sp + 1);
    const int end = static_cast<int>(k.end);
    const long long p_first = s.pos0 + k.u0 / a.group, p_last = s.pos0 + (k.u0 + k.n_u - 1) / a.group;
    const long long seen_lo = a.window > 0 ? p_first - a.window + 1 : 0;     // keys below, past the sinks: no row sees them

    if (tid == 0) {
        mbar_init(&bar_s, 1);
        mbar_init(&bar_o, 1);
        mbar_fence_init();
        s_fail = 0;
    }
    if (warp == 0) {
        tmem_alloc(&s_tmem, kRtTmemCols);
        tmem_relinquish();
    }

    // ---- keys: thread = key tid / 2 of a tile, half of its dims ----
    const int kr = tid >> 1, kh = tid & 1;
    const int* tab = a.v.table ? a.v.table + s.slot * a.v.pages_per_slot : nullptr;
    const int pr_mask = a.v.shift == 31 ? 0x7fffffff : a.v.page_rows - 1;
    auto key_page = [&](int c) {                   // page of this thread's key, -1 where no row sees one
        if (c >= c_end) return -1;
        const int j = unit_chunk(k, c) * kRtKeys + kr;
        if (j >= end || (j < seen_lo && j >= a.sinks)) return -1;
        const int p = tab ? tab[j >> a.v.shift] : s.slot * a.v.pages_per_slot + (j >> a.v.shift);
        return static_cast<unsigned>(p) < static_cast<unsigned>(a.v.n_pages) ? p : -1;
    };
    uint4 kc, vc;                                  // KV4: codes of 32 dims
    uint32_t ksw, vsw;                             // KV4: scales
    float4 kf[KV4 ? 1 : 8], vf[KV4 ? 1 : 8];       // f32: 32 dims
    auto load = [&](int c, int page) {
        const int pr = (unit_chunk(k, c) * kRtKeys + kr) & pr_mask;
        if (KV4) {
            kc = vc = make_uint4(0, 0, 0, 0);
            ksw = vsw = 0;
            if (page >= 0) {
                const int part = a.v.page_rows * kKv4RowBytes;
                const unsigned char* blk = a.cache + kv4_block(a.v, page, hk);
                kc = *reinterpret_cast<const uint4*>(blk + pr * 32 + kh * 16);
                vc = *reinterpret_cast<const uint4*>(blk + part + pr * 32 + kh * 16);
                ksw = *reinterpret_cast<const uint32_t*>(blk + a.v.page_rows * 32 + pr * 4);
                vsw = *reinterpret_cast<const uint32_t*>(blk + part + a.v.page_rows * 32 + pr * 4);
            }
        } else {
            const long long off = page < 0 ? 0 : kvf_block(a.v, page, hk) + static_cast<long long>(pr) * kHeadDim + kh * 32;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                kf[i] = vf[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (page >= 0) {
                    kf[i] = __ldg(reinterpret_cast<const float4*>(a.k + off) + i);
                    vf[i] = __ldg(reinterpret_cast<const float4*>(a.vv + off) + i);
                }
            }
        }
    };
    // Largest magnitudes of the loaded tile (f32 bits), what is not finite, and 16-key blocks without a
    // page, per loading warp (its 16 keys) into buffer `buf`.
    auto survey = [&](int c, int page, int buf) {
        uint32_t km = 0, vm = 0, nan = 0;
        auto take = [&](uint32_t bits, uint32_t& m) {
            if (bits >= 0x7f800000u) nan = 1; else m = max(m, bits);
        };
        if (KV4) {
            take(ksw << 16, km), take(ksw & 0xffff0000u, km);
            take(vsw << 16, vm), take(vsw & 0xffff0000u, vm);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                take(__float_as_uint(fabsf(kf[i].x)), km), take(__float_as_uint(fabsf(kf[i].y)), km);
                take(__float_as_uint(fabsf(kf[i].z)), km), take(__float_as_uint(fabsf(kf[i].w)), km);
                take(__float_as_uint(fabsf(vf[i].x)), vm), take(__float_as_uint(fabsf(vf[i].y)), vm);
                take(__float_as_uint(fabsf(vf[i].z)), vm), take(__float_as_uint(fabsf(vf[i].w)), vm);
            }
        }
        km = __reduce_max_sync(0xffffffffu, km);
        vm = __reduce_max_sync(0xffffffffu, vm);
        nan = __reduce_max_sync(0xffffffffu, nan);
        // a key may be left out as unseen in a block that has a page: only the page decides here
        uint32_t bad = 0;
        if (c < c_end) {
            const int j = unit_chunk(k, c) * kRtKeys + warp * 16;
            if (j < end) {
                const int p = tab ? tab[j >> a.v.shift] : s.slot * a.v.pages_per_slot + (j >> a.v.shift);
                bad = static_cast<unsigned>(p) >= static_cast<unsigned>(a.v.n_pages);
            }
        }
        (void)page;
        if (lane == 0) {
            sm_kmax[buf][warp] = km;
            sm_vmax[buf][warp] = vm;
            sm_nan[buf][warp] = nan;
            sm_bad[buf][warp] = bad;
        }
    };

    int page = key_page(c0);
    load(c0, page);

    // ---- queries: thread = row tid / 2, half of its dims ----
    {
        float x[32];
        float mx = 0.0f;
        if (kr < k.n_u) {
            const int ur = k.u0 + kr, h = hk * a.group + ur % a.group;
            const float4* q = reinterpret_cast<const float4*>(a.q + static_cast<long long>(s.row0 + ur / a.group) * a.q_ld +
                                                              h * kHeadDim + kh * 32);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 y = q[i];
                x[4 * i] = y.x, x[4 * i + 1] = y.y, x[4 * i + 2] = y.z, x[4 * i + 3] = y.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) mx = fmaxf(mx, fabsf(x[i]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        // the row's largest element goes to [2^10, 2^11); rows below 2^-100 are taken as that small
        const int e = max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -100);
        const float up = pow2i(10 - e);
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] *= up;
#pragma unroll
        for (int w = 0; w < 4; ++w) rt_store_split<KV4>(sQ, sQ + kRtPlane, kr, kh * 4 + w, x + 8 * w);
        if (kh == 0) sm_f[kr] = pow2i(e - 10) * (0.125f * kLog2e);
    }
    survey(c0, page, 0);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;

    // ---- rows: thread = row 32 (warp % 4) + lane, columns 64 half .. of S and 32 half .. of O ----
    const int half = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t t_s = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + half * 64;
    const uint32_t t_o = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 128 + half * 32;
    const float f_row = sm_f[row];
    const long long p_row = s.pos0 + (k.u0 + min(row, k.n_u - 1)) / a.group;
    float o[32], m = -INFINITY, ref_old = -INFINITY, l = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = 0.0f;
    int E = -100;                                  // V is held times 2^(vbits - E)
    constexpr int vbits = KV4 ? 9 : 10;
    uint32_t ph = 0;                               // MMA rounds done: the barriers' phase

    for (int c = c0; c < c_end; ++c) {
        const int buf = (c - c0) & 1;
        const int j0 = unit_chunk(k, c) * kRtKeys;
        if (!KV4 && c > c0) {
            load(c, page);
            survey(c, page, buf);
            __syncthreads();
        }
        uint32_t km = 0, vm = 0, nan = 0, bad = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            km = max(km, sm_kmax[buf][w]);
            vm = max(vm, sm_vmax[buf][w]);
            nan |= sm_nan[buf][w];
            bad |= sm_bad[buf][w] << w;
        }
        const int ek = max(static_cast<int>(km >> 23) - 127, -100);
        const int ev = max(static_cast<int>(vm >> 23) - 127, -100);
        const int E_new = max(E, ev);
        const float fac = E < E_new - 120 ? 0.0f : pow2i(E - E_new);
        E = E_new;

        // this row's keys: 32-column masks, unless every row sees the whole tile
        const bool full = bad == 0 && j0 + kRtKeys - 1 <= p_first && j0 + kRtKeys <= end &&
                          (a.window == 0 || j0 > p_last - a.window || j0 + kRtKeys <= a.sinks);
        auto seen_bits = [&](int b) {              // columns 32 b .. 32 b + 31 of the tile
            uint32_t v = visible_bits(j0 + 32 * b, min(p_row, k.end - 1), a.window, a.sinks);
            // the window is measured from the row's own position, which may lie past the slot's end
            if (a.window > 0 && p_row >= k.end) v &= visible_bits(j0 + 32 * b, p_row, a.window, a.sinks);
            const uint32_t miss = (bad >> (2 * b)) & 3u;
            return v & ~(((miss & 1u) ? 0xffffu : 0u) | ((miss & 2u) ? 0xffff0000u : 0u));
        };

        if (nan) {
            // ---- plain loop over the tile ----
            float corr = 1.0f;
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= fac;
            const int ur = k.u0 + min(row, k.n_u - 1), h = hk * a.group + ur % a.group;
            const float* q = a.q + static_cast<long long>(s.row0 + ur / a.group) * a.q_ld + h * kHeadDim;
            const float vs = pow2i(vbits - E);
            for (int x = 0; x < kRtKeys; ++x) {
                if (!((seen_bits(x >> 5) >> (x & 31)) & 1u)) continue;
                const int j = j0 + x;
                const int p = tab ? tab[j >> a.v.shift] : s.slot * a.v.pages_per_slot + (j >> a.v.shift);
                const int pr = j & pr_mask;
                float sc = 0.0f;
                for (int d = 0; d < kHeadDim; d += 4) {
                    const float4 kv = rt_row4<KV4>(a, false, p, hk, pr, d);
                    const float4 qv = *reinterpret_cast<const float4*>(q + d);
                    sc = fmaf(kv.w, qv.w, fmaf(kv.z, qv.z, fmaf(kv.y, qv.y, fmaf(kv.x, qv.x, sc))));
                }
                sc *= 0.125f * kLog2e;
                const float mn = fmaxf(m, sc);
                const float ref = mn == -INFINITY ? 0.0f : fabsf(mn) < 65536.0f ? mn - 12.0f : mn;
                corr = ex2(ref_old - ref);
                const float w = ex2(sc - ref);
                m = mn;
                ref_old = mn == -INFINITY ? -INFINITY : ref;
                l = fmaf(l, corr, half == 0 ? w : 0.0f);
#pragma unroll
                for (int i4 = 0; i4 < 8; ++i4) {
                    const float4 v = rt_row4<KV4>(a, true, p, hk, pr, half * 32 + i4 * 4);
                    // KV4's columns: dims 0 4 1 5 2 6 3 7 of each word
                    const int b0 = KV4 ? (i4 >> 1) * 8 + (i4 & 1) : i4 * 4, st = KV4 ? 2 : 1;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float vi = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
                        float& oi = o[b0 + i * st];
                        oi *= corr;
                        if (w != 0.0f) oi = fmaf(w, vi * vs, oi);
                    }
                }
            }
            page = key_page(c + 1);
            if (KV4) {
                if (c + 1 < c_end) load(c + 1, page);
                survey(c + 1, page, buf ^ 1);
            }
            __syncthreads();
            continue;
        }

        // ---- unpack the tile ----
        if (KV4) {
            // times 2^(10 - ek), and 16 times 2^(9 - E)
            auto pair = [](uint32_t bits, float up) { return __float2half2_rn(__uint_as_float(bits) * up); };
            const float ku = pow2i(10 - ek), vu = pow2i(13 - E);
            const __half2 k0 = pair(ksw << 16, ku), k1 = pair(ksw & 0xffff0000u, ku);
            const __half2 v0 = pair((kh ? vsw & 0xffff0000u : vsw << 16), vu), z0 = __hmul2(v0, __float2half2_rn(-1.5f));
            const uint32_t kw[4] = {kc.x, kc.y, kc.z, kc.w}, vw[4] = {vc.x, vc.y, vc.z, vc.w};
            const __half2 sub = bits_h2(0x64086408u), s16 = bits_h2(0x2c002c00u), sub16 = bits_h2(0xd480d480u);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                // K: words 2 kh + w / 2 (+ 4 for odd w). 0x6400 | n is 1024 + n; a nibble four bits up
                // gives 1024 + 16 n
                const __half2 sc = (w & 1) ? k1 : k0;
                const uint32_t x = kw[w], x8 = x >> 8;
                uint4 r;
                r.x = h2_bits(__hmul2(__hsub2(bits_h2((x & 0x000f000fu) | 0x64006400u), sub), sc));
                r.y = h2_bits(__hmul2(__hfma2(bits_h2((x & 0x00f000f0u) | 0x64006400u), s16, sub16), sc));
                r.z = h2_bits(__hmul2(__hsub2(bits_h2((x8 & 0x000f000fu) | 0x64006400u), sub), sc));
                r.w = h2_bits(__hmul2(__hfma2(bits_h2((x8 & 0x00f000f0u) | 0x64006400u), s16, sub16), sc));
                *rt_chunk(sK, kr, 2 * kh + (w >> 1) + 4 * (w & 1)) = r;
                // V: words 4 kh + w, nibbles i and 4 + i of the halves: the order 0 4 1 5 2 6 3 7 again
                uint32_t v[4];
                kv4_values(vw[w], v0, z0, v);
                *rt_chunk(sV, kr, 4 * kh + w) = make_uint4(v[0], v[1], v[2], v[3]);
            }
        } else {
            const float ku = pow2i(10 - ek), vu = pow2i(10 - E);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                float x[8];
                const float4 a0 = kf[2 * w], a1 = kf[2 * w + 1], b0 = vf[2 * w], b1 = vf[2 * w + 1];
                x[0] = a0.x * ku, x[1] = a0.y * ku, x[2] = a0.z * ku, x[3] = a0.w * ku;
                x[4] = a1.x * ku, x[5] = a1.y * ku, x[6] = a1.z * ku, x[7] = a1.w * ku;
                rt_store_split<false>(sK, sK + kRtPlane, kr, kh * 4 + w, x);
                x[0] = b0.x * vu, x[1] = b0.y * vu, x[2] = b0.z * vu, x[3] = b0.w * vu;
                x[4] = b1.x * vu, x[5] = b1.y * vu, x[6] = b1.z * vu, x[7] = b1.w * vu;
                rt_store_split<false>(sV, sV + kRtPlane, kr, kh * 4 + w, x);
            }
        }
        fence_async_smem();
        __syncthreads();
        if (s_fail) break;                         // (uniform: set before a barrier, never cleared)

        // ---- S = Q K^T: low parts first ----
        if (tid == 0) {
            tc_fence_after();
            constexpr uint32_t id = idesc_f16(kRtKeys, false);
            const uint64_t qh = smem_desc_sw128(sQ), ql = smem_desc_sw128(sQ + kRtPlane), kd = smem_desc_sw128(sK);
            if (!KV4) {
                const uint64_t kl = smem_desc_sw128(sK + kRtPlane);
#pragma unroll
                for (int i = 0; i < 4; ++i) umma_f16_ss(tmem, qh + 2 * i, kl + 2 * i, id, i > 0);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) umma_f16_ss(tmem, ql + 2 * i, kd + 2 * i, id, !KV4 || i > 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) umma_f16_ss(tmem, qh + 2 * i, kd + 2 * i, id, 1);
            umma_commit(&bar_s);
        }
        page = key_page(c + 1);
        if (KV4 && c + 1 < c_end) load(c + 1, page);
        if (!mbar_wait_bounded(&bar_s, ph, nullptr)) s_fail = 1;
        tc_fence_after();

        // ---- softmax ----
        const float f = fmaxf(f_row * pow2i(ek - 10), 1.1754944e-38f);
        float raw = -INFINITY;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            float x[32];
            tmem_ld32(t_s + 32 * b, x);
            if (full) {
#pragma unroll
                for (int i = 0; i < 32; ++i) raw = fmaxf(raw, x[i]);
            } else {
                const uint32_t v = seen_bits(2 * half + b);
#pragma unroll
                for (int i = 0; i < 32; ++i) raw = fmaxf(raw, (v >> i) & 1u ? x[i] : -INFINITY);
            }
        }
        sm_x[half][row] = raw;
        pair_sync(1 + (warp & 3));
        raw = fmaxf(raw, sm_x[half ^ 1][row]);
        const float mn = fmaxf(m, raw * f);
        const bool far = !(fabsf(mn) < 65536.0f) && mn != -INFINITY;
        const float ref = mn == -INFINITY ? 0.0f : far ? mn : mn - 12.0f;
        const float corr = ex2(ref_old - ref);
        m = mn;
        ref_old = mn == -INFINITY ? -INFINITY : ref;
        float sum = 0.0f;
        // (far from 0, where f32 does not resolve 12, the product is rounded first, as the maximum's was)
        const bool two_steps = __any_sync(0xffffffffu, far);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            float x[32];
            tmem_ld32(t_s + 32 * b, x);
            const uint32_t v = full ? 0xffffffffu : seen_bits(2 * half + b);
            if (two_steps) {
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = ex2(__fadd_rn(__fmul_rn(x[i], f), -ref));
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = ex2(fmaf(x[i], f, -ref));
            }
            if (!full) {
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = (v >> i) & 1u ? x[i] : 0.0f;
            }
            uint32_t p[32];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                sum += x[2 * i] + x[2 * i + 1];
                split_f16(x[2 * i], x[2 * i + 1], p[i], p[16 + i]);
            }
            tmem_st32(t_s + 32 * b, p);            // 16 columns of high parts, 16 of low parts
        }
        l = fmaf(l, corr, sum);
        tmem_st_wait();
        if (KV4) survey(c + 1, page, buf ^ 1);
        tc_fence_before();
        __syncthreads();

        // ---- O = P V ----
        if (tid == 0) {
            tc_fence_after();
            constexpr uint32_t id = idesc_f16(kHeadDim, true);
            const uint64_t vd = smem_desc_sw128(sV), vl = smem_desc_sw128(sV + (KV4 ? 0 : kRtPlane));
#pragma unroll
            for (int i = 0; i < 8; ++i)            // 16 keys: block i / 2 of 32, step i % 2; 2048 bytes of V
                umma_f16_ts(tmem + 128, tmem + (i >> 1) * 32 + 16 + (i & 1) * 8, vd + 128 * i, id, i > 0);
            if (!KV4) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    umma_f16_ts(tmem + 128, tmem + (i >> 1) * 32 + (i & 1) * 8, vl + 128 * i, id, 1);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                umma_f16_ts(tmem + 128, tmem + (i >> 1) * 32 + (i & 1) * 8, vd + 128 * i, id, 1);
            umma_commit(&bar_o);
        }
        if (!mbar_wait_bounded(&bar_o, ph, nullptr)) s_fail = 1;
        ph ^= 1u;
        tc_fence_after();
        {
            float d[32];
            tmem_ld32(t_o, d);
            const float cf = corr * fac;
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = fmaf(o[i], cf, d[i]);
        }
        tc_fence_before();
    }
    // ---- finish ----
    __syncthreads();
    sm_x[half][row] = l;
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, kRtTmemCols);
    if (row >= k.n_u) return;
    // a wait that gave up leaves the rows' sums NaN, their outputs 0
    const float L = s_fail ? __uint_as_float(0x7fc00000u) : l + sm_x[half ^ 1][row];
    const float back = pow2i(E - vbits);
    float y[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const int w = i >> 3, d = i & 7;           // dim d of the word sits in column 2 (d % 4) + d / 4
        y[i] = (KV4 ? o[w * 8 + (d & 3) * 2 + (d >> 2)] : o[i]) * back;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float4 v = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
        store_unit_row(a, k, s, hk, sp, row, half * 8 + i, ref_old, L, v);
    }
}

}  // namespace dec

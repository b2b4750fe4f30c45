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
// A block (256 threads, two per SM) alternates between its softmax and the two products. The thread
// that issues a product is held for as long as the product runs, so the warps share the rest: warp 0
// issues P V while warps 4..7 unpack the next tile's K, then warp 4 issues Q K^T while warps 0..3 unpack
// its V; the other block of the SM fills the gaps. A 4-bit cache's tile is copied into shared memory by
// cp.async a tile ahead; an f32 tile goes through registers, half a key per thread. An M128 N128 K16 MMA
// takes 65 SM cycles and an M128 N64 K16 one 45 to 49 (measured), 1240 per tile of a 4-bit cache; the
// softmax, about 6 instructions per score and an exp2 unit that takes 1024 cycles per tile, is the larger
// part of a tile's time. 16 streams' chunks of 128 rows over 4096 keys, 14 heads over 2: 156 us, 190 TFLOP/s
// counted once (f32: 286 us, 104); a warp of its own for the issue, a queue of work on the device and 96
// registers for more warps were all slower.
//
// All rows share a tile's powers of two, also for keys that only some of them see. Of a 4-bit cache f16 holds
// scales down to 2^-24 of the tile's largest exactly, of an f32 cache 22 bits of every key's largest value down
// to 2^-12 of the tile's. A tile with keys further apart, or with a NaN or an infinity at a position that some
// row sees, is computed by a plain f32 loop instead (as long as 60 to 90 tiles). From a plain tile on, or from one that needs a smaller
// power of two of V than those before, the sums are kept in a scale of their own, 2^-16, in which f32 holds
// those of all finite values.
#pragma once

#include "attn_kv4_few.cuh"
#include "head_tc.cuh"

namespace dec {

constexpr int kRtRows = 128, kRtKeys = 128, kRtThreads = 256;
constexpr int kRtPlane = kRtRows * 128;           // one f16 operand plane: 128 rows of 64 dims
constexpr uint32_t kRtTmemCols = 256;             // S / P 0..127, O 128..191
// a tile of a 4-bit cache as it lies: K codes, V codes, K scales, V scales
constexpr int kRtStage = kRtKeys * 2 * kKv4RowBytes;
constexpr int kRtSpan4 = 24, kRtSpan = 12;        // scales, and keys' largest values: from 2^e down to 2^(e - span)
constexpr int kRtV = kRtKeys * 32, kRtKs = 2 * kRtKeys * 32, kRtVs = kRtKs + kRtKeys * 4;
template <bool KV4>
constexpr int rt_smem_bytes() {
    return (2 + (KV4 ? 2 : 4)) * kRtPlane + (KV4 ? 2 * kRtStage : 0) + 1024;
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
__device__ __forceinline__ void tmem_ld16(uint32_t addr, float (&r)[16]) {
    uint32_t x[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]), "=r"(x[8]),
          "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15])
        : "r"(addr)
        : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __uint_as_float(x[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&x)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(x[0]),
        "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]), "r"(x[8]), "r"(x[9]), "r"(x[10]),
        "r"(x[11]), "r"(x[12]), "r"(x[13]), "r"(x[14]), "r"(x[15]), "r"(addr)
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
    unsigned char* stages = sV + kRtPlane;                       // KV4: two
    __shared__ __align__(8) uint64_t bar_s, bar_o;
    __shared__ uint32_t s_tmem;
    __shared__ float sm_f[kRtRows], sm_x[2][kRtRows];            // row factors; column halves' maxima, sums
    __shared__ uint32_t sm_bad[2][8];                            // of a tile's 16-key blocks: no page
    __shared__ uint32_t sm_mag[4][8];                            // f32: magnitudes of K, of V; the smallest
    __shared__ int s_fail;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();
    const StreamRows s = stream_rows(a.r, a.v, blockIdx.z);
    const int n_tiles = gridDim.y / a.v.heads;
    const int hk = blockIdx.y / n_tiles;
    const UnitKeys k = unit_keys<kRtRows, kRtKeys>(a, s, blockIdx.y % n_tiles);
    const int sp = blockIdx.x;
    if (k.n_u == 0 || sp >= k.splits) return;
    const int c0 = split_begin(k, sp), c_end = split_begin(k, sp + 1);
    const int end = static_cast<int>(k.end);
    const long long p_first = s.pos0 + k.u0 / a.group, p_last = s.pos0 + (k.u0 + k.n_u - 1) / a.group;
    // keys below, past the sinks: no row sees them
    const int seen_lo = a.window > 0 ? static_cast<int>(max(0ll, min(p_first - a.window + 1, 0x7fffff00ll))) : 0;

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

    // ---- keys ----
    // a 4-bit tile: thread = key ku, fetched and K unpacked by warps 4..7, V unpacked by warps 0..3; an f32
    // tile: thread = half kh of key ku's dims
    const int ku = KV4 ? tid & 127 : tid >> 1, kh = tid & 1;
    const bool k_side = warp >= 4;
    const int* tab = a.v.table ? a.v.table + s.slot * a.v.pages_per_slot : nullptr;
    const int pr_mask = a.v.shift == 31 ? 0x7fffffff : a.v.page_rows - 1;
    // Table entry of a key below `end` (not yet checked: the value is first used a tile later), -1 beyond.
    auto page_entry = [&](int j) { return tab ? tab[j >> a.v.shift] : s.slot * a.v.pages_per_slot + (j >> a.v.shift); };
    auto checked = [&](int p) { return static_cast<unsigned>(p) < static_cast<unsigned>(a.v.n_pages) ? p : -1; };
    auto key_page = [&](int c) {
        int p = -1;
        if (c < c_end) {
            const int j = unit_chunk(k, c) * kRtKeys + ku;
            if (j < end) p = page_entry(j);
        }
        return p;
    };
    auto seen = [&](int j) { return j < end && (j >= seen_lo || j < a.sinks); };
    // Copies the tile into its stage (4-bit cache), and notes its blocks without a page.
    auto stage_tile = [&](int c, int entry) {
        if (KV4 && !k_side) return;
        const int buf = (c - c0) & 1, pg = checked(entry);
        if (c < c_end) {
            if (KV4 && pg >= 0) {
                const int pr = (unit_chunk(k, c) * kRtKeys + ku) & pr_mask;
                const int part = a.v.page_rows * kKv4RowBytes;
                const unsigned char* src = a.cache + kv4_block(a.v, pg, hk) + pr * 32;
                unsigned char* dst = stages + buf * kRtStage + ku * 32;
                cp_async16(dst, src);
                cp_async16(dst + 16, src + 16);
                cp_async16(dst + kRtV, src + part);
                cp_async16(dst + kRtV + 16, src + part + 16);
                if ((ku & 3) == 0) {               // four keys' scales
                    src += a.v.page_rows * 32 - pr * 28;
                    dst = stages + buf * kRtStage + kRtKs + ku * 4;
                    cp_async16(dst, src);
                    cp_async16(dst + (kRtVs - kRtKs), src + part);
                }
            }
            if ((ku & 15) == 0) sm_bad[buf][ku >> 4] = pg < 0 && unit_chunk(k, c) * kRtKeys + ku < end;
        }
        if (KV4) cp_async_commit();
    };

    const int page = key_page(c0);
    int page1 = key_page(c0 + 1), page2 = key_page(c0 + 2);

    // ---- queries: thread = row tid / 2, half of its dims ----
    {
        const int qr = tid >> 1;
        float x[32];
        float mx = 0.0f;
        if (qr < k.n_u) {
            const int ur = k.u0 + qr, h = hk * a.group + ur % a.group;
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
        stage_tile(c0, page);                      // (the queries are on their way)
        stage_tile(c0 + 1, page1);
#pragma unroll
        for (int i = 0; i < 32; ++i) mx = fmaxf(mx, fabsf(x[i]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        // the row's largest element goes to [2^10, 2^11); rows below 2^-100 are taken as that small
        const int e = max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -100);
        const float up = pow2i(10 - e);
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] *= up;
#pragma unroll
        for (int w = 0; w < 4; ++w) rt_store_split<KV4>(sQ, sQ + kRtPlane, qr, kh * 4 + w, x + 8 * w);
        if (kh == 0) sm_f[qr] = pow2i(e - 10) * (0.125f * kLog2e);
    }

    // ---- rows: thread = row 32 (warp % 4) + lane, columns 64 half .. of S and 32 half .. of O ----
    const int half = warp >> 2, row = (warp & 3) * 32 + lane;
    const long long p_row = s.pos0 + (k.u0 + min(row, k.n_u - 1)) / a.group;
    float o[32], m = -INFINITY, ref_old = -INFINITY, l = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = 0.0f;
    constexpr int vbits = KV4 ? 9 : 10;
    constexpr int own_scale = vbits + 16;
    int ek = -100, E = -100;                       // K is held times 2^(10 - ek), V times 2^(vbits - E)
    bool own = false;                              // O is held times 2^-16, or else as V
    float fac = 1.0f, df = 1.0f;                   // what the last change of scale makes of O, and P V's scale
    // For a tile whose V has the largest exponent e; `small`: some key is too small for the scale so far.
    auto set_scale = [&](int e, bool small, bool plain) {
        if (!own) {
            own = plain || e > 40 || e < -40 || small;
            const int to = own ? own_scale : max(E, e);
            fac = E < to - 120 ? 0.0f : pow2i(E - to);         // (E is -100 before any value)
            if (!plain) E = max(E, e);
        }
        if (own && !plain) E = min(max(e, -100), 123);
        if (own) df = pow2i(E - own_scale);
    };
    uint32_t bad = 0;                              // blocks of the tile at hand without a page

    // Looks a tile over before its K is unpacked: powers of two, blocks without a page. True when
    // something that a row sees is not finite, or its scales are too far apart.
    auto survey4 = [&](int c) {
        const int buf = (c - c0) & 1, j0 = unit_chunk(k, c) * kRtKeys;
        bad = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) bad |= sm_bad[buf][w] << w;
        const bool live = bad == 0 && j0 + kRtKeys <= end && (j0 >= seen_lo || j0 + kRtKeys <= a.sinks);
        const unsigned char* st = stages + buf * kRtStage + lane * 16;
        const uint4 kv = *reinterpret_cast<const uint4*>(st + kRtKs), vv = *reinterpret_cast<const uint4*>(st + kRtVs);
        const uint32_t kw[4] = {kv.x, kv.y, kv.z, kv.w}, vw[4] = {vv.x, vv.y, vv.z, vv.w};
        uint32_t km = 0, vm = 0, kl = 0xffffffffu, vl = 0xffffffffu;     // largest; smallest above 0, less 1, by group
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (live || (seen(j0 + lane * 4 + i) && !((bad >> (lane >> 2)) & 1u))) {
                km = __vmaxu2(km, kw[i]);
                vm = __vmaxu2(vm, vw[i]);
                kl = __vminu2(kl, kw[i] - 0x00010001u);            // (a zero gives 0xfffe or more)
                vl = __vminu2(vl, vw[i] - 0x00010001u);
            }
        km = __reduce_max_sync(0xffffffffu, max(km & 0xffffu, km >> 16));
        vm = __reduce_max_sync(0xffffffffu, max(vm & 0xffffu, vm >> 16));
        const int ke = static_cast<int>(km >> 7) - 127, e = static_cast<int>(vm >> 7) - 127;
        const int kleast = static_cast<int>((min(kl & 0xffffu, kl >> 16) + 1u) >> 7) - 127;
        const int least = static_cast<int>((min(vl & 0xffffu, vl >> 16) + 1u) >> 7) - 127;
        bool plain = max(km, vm) >= 0x7f80u;
        plain |= __any_sync(0xffffffffu, kleast < ke - kRtSpan4 || least < e - kRtSpan4);
        if (!plain) ek = max(ke, -100);
        if (plain || vm) set_scale(e, __any_sync(0xffffffffu, least < E - kRtSpan4), plain);
        return plain;
    };
    auto live_key = [&](int c) {
        return seen(unit_chunk(k, c) * kRtKeys + ku) && !((bad >> (ku >> 4)) & 1u);
    };
    // Unpacks K (times 2^(10 - ek)).
    auto unpack_k4 = [&](int c) {
        const unsigned char* st = stages + ((c - c0) & 1) * kRtStage;
        const uint32_t ksw = live_key(c) ? *reinterpret_cast<const uint32_t*>(st + kRtKs + ku * 4) : 0u;
        const float up = pow2i(10 - ek);
        const __half2 k0 = __float2half2_rn(__uint_as_float(ksw << 16) * up);
        const __half2 k1 = __float2half2_rn(__uint_as_float(ksw & 0xffff0000u) * up);
        const __half2 sub = bits_h2(0x64086408u), s16 = bits_h2(0x2c002c00u), sub16 = bits_h2(0xd480d480u);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const uint4 kc = *reinterpret_cast<const uint4*>(st + ku * 32 + hf * 16);
            const uint32_t kw[4] = {kc.x, kc.y, kc.z, kc.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                // words 2 hf + w / 2 (+ 4 for odd w). 0x6400 | n is 1024 + n; a nibble four bits up
                // gives 1024 + 16 n
                const __half2 sc = (w & 1) ? k1 : k0;
                const uint32_t x = kw[w], x8 = x >> 8;
                uint4 r;
                r.x = h2_bits(__hmul2(__hsub2(bits_h2((x & 0x000f000fu) | 0x64006400u), sub), sc));
                r.y = h2_bits(__hmul2(__hfma2(bits_h2((x & 0x00f000f0u) | 0x64006400u), s16, sub16), sc));
                r.z = h2_bits(__hmul2(__hsub2(bits_h2((x8 & 0x000f000fu) | 0x64006400u), sub), sc));
                r.w = h2_bits(__hmul2(__hfma2(bits_h2((x8 & 0x00f000f0u) | 0x64006400u), s16, sub16), sc));
                *rt_chunk(sK, ku, 2 * hf + (w >> 1) + 4 * (w & 1)) = r;
            }
        }
    };
    // Unpacks V (16 times the scale is 2^(13 - E) times it). A word's nibbles i and 4 + i come out
    // paired: the order 0 4 1 5 2 6 3 7 again.
    auto unpack_v4 = [&](int c) {
        const unsigned char* st = stages + ((c - c0) & 1) * kRtStage;
        const uint32_t vsw = live_key(c) ? *reinterpret_cast<const uint32_t*>(st + kRtVs + ku * 4) : 0u;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const uint4 vc = *reinterpret_cast<const uint4*>(st + kRtV + ku * 32 + hf * 16);
            const __half2 v0 = __float2half2_rn(__uint_as_float(hf ? vsw & 0xffff0000u : vsw << 16) * pow2i(13 - E));
            const __half2 z0 = __hmul2(v0, __float2half2_rn(-1.5f));
            const uint32_t vw[4] = {vc.x, vc.y, vc.z, vc.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t v[4];
                kv4_values(vw[w], v0, z0, v);
                *rt_chunk(sV, ku, 4 * hf + w) = make_uint4(v[0], v[1], v[2], v[3]);
            }
        }
    };
    // f32: this thread's 32 dims of K or V, 0 where no row sees the key.
    auto load_f32 = [&](int c, int entry, const float* pool, float4 (&x)[8]) {
        const int j = unit_chunk(k, c) * kRtKeys + ku, pg = checked(entry);
        const bool live = pg >= 0 && seen(j);
        const float4* src = reinterpret_cast<const float4*>(
            pool + (live ? kvf_block(a.v, pg, hk) + static_cast<long long>(j & pr_mask) * kHeadDim + kh * 32 : 0));
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = live ? __ldg(src + i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    };
    // f32: largest magnitude, as bits (a NaN's are above all).
    auto magnitude = [&](const float4 (&x)[8]) {
        uint32_t g = 0;
#pragma unroll
        for (int n = 0; n < 8; ++n)
            g = max(max(max(g, __float_as_uint(fabsf(x[n].x))), __float_as_uint(fabsf(x[n].y))),
                    max(__float_as_uint(fabsf(x[n].z)), __float_as_uint(fabsf(x[n].w))));
        return g;
    };
    // f32: scales, splits and stores.
    auto store_f32 = [&](unsigned char* plane, const float4 (&x)[8], float up) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float4 u = x[2 * w], v = x[2 * w + 1];
            const float y[8] = {u.x * up, u.y * up, u.z * up, u.w * up, v.x * up, v.y * up, v.z * up, v.w * up};
            rt_store_split<false>(plane, plane + kRtPlane, ku, kh * 4 + w, y);
        }
    };
    float4 vf[KV4 ? 1 : 8];                        // f32: the next tile's V

    // Gets tile c ready for its scores: looks it over, and K into sK (every thread is done with the last
    // tile's scores), an f32 V into registers. True when something that a row sees is not finite, or its
    // keys are too far apart: the tile is left to the plain loop. All threads return the same.
    auto prepare = [&](int c, int entry) -> bool {
        fac = 1.0f;
        bool plain = false;
        if constexpr (KV4) {
            plain = survey4(c);
            if (!plain && k_side) unpack_k4(c);
            fence_async_smem();
            __syncthreads();
        } else {
            // The powers of two stand while the values, held below 2^11 when they were set, stay below 2^15
            // (2^16 itself would not do: f16 ends at 65504) and every key's largest at 2^-2 or more; a tile
            // beyond them (the first one, to begin with) sets them anew.
            float4 x[8];
            load_f32(c, entry, a.k, x);
            uint32_t km = magnitude(x);
            store_f32(sK, x, pow2i(10 - ek));
            load_f32(c, entry, a.vv, vf);
            uint32_t vm = magnitude(vf);
            // (of half a key: a smaller half is looked at, too)
            const uint32_t klow = static_cast<uint32_t>(127 + ek - kRtSpan) << 23;
            const uint32_t vlow = static_cast<uint32_t>(127 + E - kRtSpan) << 23;
            constexpr uint32_t range = (kRtSpan + 5) << 23;
            fence_async_smem();
            if (__syncthreads_or(c == c0 || (km && km - klow >= range) || (vm && vm - vlow >= range))) {
                km = max(km, __shfl_xor_sync(0xffffffffu, km, 1));
                vm = max(vm, __shfl_xor_sync(0xffffffffu, vm, 1));
                // largest of all keys, smallest above 0 less 1
                const uint32_t kl = __reduce_min_sync(0xffffffffu, km - 1u), vl = __reduce_min_sync(0xffffffffu, vm - 1u);
                km = __reduce_max_sync(0xffffffffu, km);
                vm = __reduce_max_sync(0xffffffffu, vm);
                if (lane == 0) sm_mag[0][warp] = km, sm_mag[1][warp] = vm, sm_mag[2][warp] = kl, sm_mag[3][warp] = vl;
                __syncthreads();
                uint32_t kleast = kl, least = vl;
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    km = max(km, sm_mag[0][w]);
                    vm = max(vm, sm_mag[1][w]);
                    kleast = min(kleast, sm_mag[2][w]);
                    least = min(least, sm_mag[3][w]);
                }
                const int ke = static_cast<int>(km >> 23) - 127, e = static_cast<int>(vm >> 23) - 127;
                const int kmin = static_cast<int>(kleast >> 23) - 127, vmin = static_cast<int>(least >> 23) - 127;
                plain = max(km, vm) >= 0x7f800000u || kmin < ke - kRtSpan || vmin < e - kRtSpan;
                if (plain || vm) set_scale(e, vmin < E - kRtSpan, plain);
                if (!plain) {
                    if (km) ek = min(max(ke, -100), 123);
                    load_f32(c, entry, a.k, x);
                    store_f32(sK, x, pow2i(10 - ek));
                }
                fence_async_smem();
                __syncthreads();
            }
            bad = 0;
#pragma unroll
            for (int w = 0; w < 8; ++w) bad |= sm_bad[(c - c0) & 1][w] << w;
        }
        return plain;
    };

    if (KV4) cp_async_wait<0>();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const uint32_t t_s = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + half * 64;
    const uint32_t t_o = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 128 + half * 32;
    const float f_row = sm_f[row];
    uint32_t ph_s = 0, ph_o = 0;                   // the barriers' phases
    // S = Q K^T, low parts first (issued by warp 4)
    auto start_scores = [&]() {
        if (tid != 128) return;
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
    };
    // V of tile c into sV; every thread has seen the last P V end.
    auto store_v = [&](int c) {
        if constexpr (KV4) {
            if (!k_side) unpack_v4(c);
        } else {
            store_f32(sV, vf, pow2i(10 - E));
        }
    };
    bool plain = false;
    if (c0 < c_end) {
        plain = prepare(c0, page);
        if (!plain) {
            start_scores();
            store_v(c0);
        }
    }

    for (int c = c0; c < c_end; ++c) {
        const int j0 = unit_chunk(k, c) * kRtKeys;
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
        uint32_t cols[2] = {0xffffffffu, 0xffffffffu};      // this thread's columns
        if (!full) cols[0] = seen_bits(2 * half), cols[1] = seen_bits(2 * half + 1);
        float corr = 1.0f;
        if (!plain) {
            if (!mbar_wait_bounded(&bar_s, ph_s, nullptr)) s_fail = 1;
            ph_s ^= 1u;
            tc_fence_after();

            // ---- softmax ----
            const float f = fmaxf(f_row * pow2i(ek - 10), 1.1754944e-38f);
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float x[32];
                tmem_ld32(t_s + 32 * b, x);
                if (!full) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] = cols[b] & (1u << i) ? x[i] : -INFINITY;
                }
#pragma unroll
                for (int i = 0; i < 32; i += 8)
#pragma unroll
                    for (int n = 0; n < 4; ++n) mx[n] = fmaxf(mx[n], fmaxf(x[i + 2 * n], x[i + 2 * n + 1]));
            }
            float raw = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            sm_x[half][row] = raw;
            pair_sync(1 + (warp & 3));
            raw = fmaxf(raw, sm_x[half ^ 1][row]);
            const float mn = fmaxf(m, raw * f);
            const bool far = !(fabsf(mn) < 65536.0f) && mn != -INFINITY;
            const float ref = mn == -INFINITY ? 0.0f : far ? mn : mn - 12.0f;
            corr = ex2(ref_old - ref);
            m = mn;
            ref_old = mn == -INFINITY ? -INFINITY : ref;
            float2 sum = make_float2(0.0f, 0.0f);
            // (far from 0, where f32 does not resolve 12, the product is rounded first, as the maximum's was)
            const bool two_steps = __any_sync(0xffffffffu, far);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                float x[16];
                tmem_ld16(t_s + 16 * b, x);
                if (two_steps) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = ex2(__fadd_rn(__fmul_rn(x[i], f), -ref));
                } else {
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float2 y = fma2(make_float2(x[i], x[i + 1]), make_float2(f, f), make_float2(-ref, -ref));
                        x[i] = ex2(y.x);
                        x[i + 1] = ex2(y.y);
                    }
                }
                if (!full) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = cols[b >> 1] & (1u << ((b & 1) * 16 + i)) ? x[i] : 0.0f;
                }
                uint32_t p[16];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 y = make_float2(x[2 * i], x[2 * i + 1]);
                    sum = add2(sum, y);
                    const __half2 h = __floats2half2_rn(y.x, y.y);
                    const float2 hf = __half22float2(h), r = fma2(hf, make_float2(-1.0f, -1.0f), y);
                    p[i] = h2_bits(h);
                    p[8 + i] = h2_bits(__floats2half2_rn(r.x, r.y));
                }
                tmem_st16(t_s + 16 * b, p);        // 8 columns of high parts, 8 of low parts
            }
            l = fmaf(l, corr, sum.x + sum.y);
            tmem_st_wait();
        } else {
            // ---- plain loop over the tile ----
            const int ur = k.u0 + min(row, k.n_u - 1), h = hk * a.group + ur % a.group;
            const float* q = a.q + static_cast<long long>(s.row0 + ur / a.group) * a.q_ld + h * kHeadDim;
            const float vs = pow2i(vbits - own_scale);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= fac;
            for (int x = 0; x < kRtKeys; ++x) {
                if (!((seen_bits(x >> 5) >> (x & 31)) & 1u)) continue;
                const int j = j0 + x, p = page_entry(j), pr = j & pr_mask;
                float sc = 0.0f;
                for (int d = 0; d < kHeadDim; d += 4) {
                    const float4 kv = rt_row4<KV4>(a, false, p, hk, pr, d);
                    const float4 qv = *reinterpret_cast<const float4*>(q + d);
                    sc = fmaf(kv.w, qv.w, fmaf(kv.z, qv.z, fmaf(kv.y, qv.y, fmaf(kv.x, qv.x, sc))));
                }
                sc *= 0.125f * kLog2e;
                const float mn = fmaxf(m, sc);
                const float ref = mn == -INFINITY ? 0.0f : fabsf(mn) < 65536.0f ? mn - 12.0f : mn;
                const float cr = ex2(ref_old - ref), w = ex2(sc - ref);
                m = mn;
                ref_old = mn == -INFINITY ? -INFINITY : ref;
                l = fmaf(l, cr, half == 0 ? w : 0.0f);
#pragma unroll
                for (int i4 = 0; i4 < 8; ++i4) {
                    const float4 v = rt_row4<KV4>(a, true, p, hk, pr, half * 32 + i4 * 4);
                    // KV4's columns: dims 0 4 1 5 2 6 3 7 of each word
                    const int b0 = KV4 ? (i4 >> 1) * 8 + (i4 & 1) : i4 * 4, st = KV4 ? 2 : 1;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float vi = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
                        float& oi = o[b0 + i * st];
                        oi *= cr;
                        if (w != 0.0f) oi = fmaf(w, vi * vs, oi);
                    }
                }
            }
        }
        if (KV4) cp_async_wait<0>();
        fence_async_smem();                        // V's unpacked values
        tc_fence_before();
        __syncthreads();
        if (s_fail) break;                         // (set before a barrier, never cleared)
        if (!plain && tid == 0) {
            // ---- O = P V ----
            tc_fence_after();
            constexpr uint32_t id = idesc_f16(kHeadDim, true);
            const uint64_t vd = smem_desc_sw128(sV), vl = smem_desc_sw128(sV + (KV4 ? 0 : kRtPlane));
#pragma unroll
            for (int i = 0; i < 8; ++i)            // 16 keys: 8 + 8 columns of P, 2048 bytes of V
                umma_f16_ts(tmem + 128, tmem + i * 16 + 8, vd + 128 * i, id, i > 0);
            if (!KV4) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    umma_f16_ts(tmem + 128, tmem + i * 16, vl + 128 * i, id, 1);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                umma_f16_ts(tmem + 128, tmem + i * 16, vd + 128 * i, id, 1);
            umma_commit(&bar_o);
        }
        const bool running = !plain, more = c + 1 < c_end;
        const float cf = corr * fac, df_now = df;  // (of this tile: preparing the next one may change them)
        const bool own_now = own;
        plain = more && prepare(c + 1, page1);
        if (running) {
            if (!mbar_wait_bounded(&bar_o, ph_o, nullptr)) s_fail = 1;
            ph_o ^= 1u;
            tc_fence_after();
        }
        if (more && !plain) start_scores();        // (over the columns that P V has read)
        if (running) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float d[16];
                tmem_ld16(t_o + 16 * b, d);
                if (own_now) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) d[i] *= df_now;
                }
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    float* x = o + 16 * b + i;
                    const float2 y = fma2(make_float2(x[0], x[1]), make_float2(cf, cf), make_float2(d[i], d[i + 1]));
                    x[0] = y.x;
                    x[1] = y.y;
                }
            }
            tc_fence_before();
        }
        if (more && !plain) store_v(c + 1);
        stage_tile(c + 2, page2);                  // (the stage's last tile is unpacked)
        page1 = page2;
        page2 = key_page(c + 3);
    }
    // ---- finish ----
    __syncthreads();
    sm_x[half][row] = l;
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, kRtTmemCols);
    if (row >= k.n_u) return;
    // a wait that gave up leaves the rows' sums NaN, their outputs 0
    const RowScale f = row_scale(m, ref_old);
    const float L = s_fail ? __uint_as_float(0x7fc00000u) : (l + sm_x[half ^ 1][row]) * f.mul;
    const float back = pow2i((own ? own_scale : E) - vbits) * f.mul;
    float y[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const int w = i >> 3, d = i & 7;           // dim d of the word sits in column 2 (d % 4) + d / 4
        y[i] = (KV4 ? o[w * 8 + (d & 3) * 2 + (d >> 2)] : o[i]) * back;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        store_unit_row(a, k, s, hk, sp, row, half * 8 + i, f.ref, L,
                       make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]));
}

}  // namespace dec

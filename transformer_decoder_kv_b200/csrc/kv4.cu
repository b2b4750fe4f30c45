// 4-bit K/V cache: quantising rows as they are stored (dec_kv4_write) and reading them back
// (dec_kv4_read).
//
// Per (row, K/V head, group of 32 dims): a = max |x|, s = bf16(a / 7), c = round(x / s) to the
// nearest integer, ties to even; value c s. a / 7 is the f32 quotient or a times the f32 next to 1 / 7, as the
// call asks: next to a border of bf16 the two give neighbouring scales. The scale is rounded before the codes
// are chosen, so |x - c s| <= s / 2 holds whatever its rounding (a / s <= 7 (1 + 2^-8 + 2^-22) rounds to 7),
// and bf16 keeps f32's range. c s has 3 + 8 significant bits: exact in f32, and in f16 up to a power of two.
//
// The code is decided exactly: c0, the integer next to x * (1 / s) in f32, is within one of it, and
// e = x - c0 s is exact in f32 (fma; c0 s has 11 significant bits and cancels x's leading ones;
// s >= 2^-126 keeps the last bit of c0 s above the subnormal grid), so comparing e with +-s / 2 settles
// borders and ties; only an element within rounding of a border needs more than the comparison.
//
// One lane takes 8 consecutive dims: 8 lanes are one (row, head) of K or V, 4 lanes one scale. Bound by
// memory: 512 bytes read and 72 written per (row, K/V head), the reverse for reading back. A lane has
// kTasks rows of K and V in flight (32 bytes each, one 256-bit access where the rows are 32-byte
// aligned), and a code takes about 8 instructions.
#include "kv_rows.cuh"

using namespace dec;

namespace {

constexpr int kThreads = 256;
constexpr int kTasks = 2;                          // (row, head) pairs per 8 lanes
constexpr int kGroups = kThreads / 8 * kTasks;     // (row, head) pairs per block

struct F8 {
    float v[8];
};
// 32 bytes of a row; WIDE: 32-byte aligned.
template <bool WIDE>
__device__ __forceinline__ F8 load8(const float* p) {
    F8 x;
    if (WIDE) {
        asm("ld.global.nc.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
            : "=f"(x.v[0]), "=f"(x.v[1]), "=f"(x.v[2]), "=f"(x.v[3]), "=f"(x.v[4]), "=f"(x.v[5]), "=f"(x.v[6]), "=f"(x.v[7])
            : "l"(p));
    } else {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
        x.v[0] = a.x, x.v[1] = a.y, x.v[2] = a.z, x.v[3] = a.w, x.v[4] = b.x, x.v[5] = b.y, x.v[6] = b.z, x.v[7] = b.w;
    }
    return x;
}
template <bool WIDE>
__device__ __forceinline__ void store8(float* p, const F8& x) {
    if (WIDE) {
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x.v[0]), "f"(x.v[1]),
                     "f"(x.v[2]), "f"(x.v[3]), "f"(x.v[4]), "f"(x.v[5]), "f"(x.v[6]), "f"(x.v[7])
                     : "memory");
    } else {
        reinterpret_cast<float4*>(p)[0] = make_float4(x.v[0], x.v[1], x.v[2], x.v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(x.v[4], x.v[5], x.v[6], x.v[7]);
    }
}

// Word of 8 codes + 8 and the bf16 bits of their scale, the group's four lanes together.
__device__ __forceinline__ uint32_t kv4_quantise(const F8& x, unsigned mask, bool product, uint32_t& scale) {
    float a = 0.0f;
    float2 z = make_float2(0.0f, 0.0f);            // 0 while everything is finite
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        a = fmaxf(a, fmaxf(fabsf(x.v[j]), fabsf(x.v[j + 1])));
        z = fma2(make_float2(x.v[j], x.v[j + 1]), make_float2(0.0f, 0.0f), z);
    }
    if (!(z.x + z.y == 0.0f)) a = INFINITY;
    a = fmaxf(a, __shfl_xor_sync(mask, a, 1));
    a = fmaxf(a, __shfl_xor_sync(mask, a, 2));
    scale = 0x7fc0u;
    if (!(a < INFINITY)) return 0x88888888u;
    const uint32_t u = __float_as_uint(product ? __fmul_rn(a, 1.0f / 7.0f) : __fdiv_rn(a, 7.0f));
    scale = (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
    if (scale < 0x0080u) {
        scale = 0;
        return 0x88888888u;
    }
    const float s = __uint_as_float(scale << 16), inv = 1.0f / s, h = 0.5f * s;
    // t = 1.5 2^23 + c: its low bits are c's (two's complement)
    constexpr float kMagic = 12582912.0f;
    uint32_t n[8];
    float e[8], far = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const float2 v = make_float2(x.v[j], x.v[j + 1]);
        const float2 t = fma2(v, make_float2(inv, inv), make_float2(kMagic, kMagic));
        const float2 c = add2(t, make_float2(-kMagic, -kMagic));
        const float2 r = fma2(c, make_float2(-s, -s), v);
        n[j] = __float_as_uint(t.x), n[j + 1] = __float_as_uint(t.y);
        e[j] = r.x, e[j + 1] = r.y;
        far = fmaxf(far, fmaxf(fabsf(r.x), fabsf(r.y)));
    }
    if (far >= h) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t odd = n[j] & 1u;
            if (e[j] > h || (e[j] == h && odd)) n[j] += 1;
            if (e[j] < -h || (e[j] == -h && odd)) n[j] -= 1;
        }
    }
    // two codes to a byte, four bytes to the word
    uint32_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t hi = n[2 * j + 1] * 16u;
        b[j] = (n[2 * j] & 15u) | (hi & ~15u);
    }
    const uint32_t w = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    return w ^ 0x88888888u;                        // (c + 8) & 15
}

// The values of 8 codes + 8 of one scale. A nibble masked out at bit 8 (or 12) under the exponent of
// 2^15 (2^11) is 2^15 + n (2^11 + n); one fma takes it to (n - 8) s, exactly: 2^15 + 8 times the scale's 8
// significant bits has 21. Scales whose product with it would leave f32 go the long way.
__device__ __forceinline__ F8 kv4_dequantise(uint32_t w, float s) {
    F8 y;
    if (s >= 1e30f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y.v[j] = s * static_cast<float>(static_cast<int>((w >> (4 * j)) & 15u) - 8);
        return y;
    }
    const float2 c = make_float2(-32776.0f * s, -2056.0f * s);
    const uint32_t x[4] = {w << 8, w, w >> 8, w >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = fma2(make_float2(__uint_as_float((x[i] & 0x00000f00u) | 0x47000000u),
                                          __uint_as_float((x[i] & 0x0000f000u) | 0x45000000u)),
                              make_float2(s, s), c);
        y.v[2 * i] = v.x, y.v[2 * i + 1] = v.y;
    }
    return y;
}

// A block's tile: 2^lh heads x 64 / 2^lh rows, so that a lane group finds its row and head by shifts
// and several heads share a row's place. lh: the largest power of two (up to 16) that divides the
// heads; no lane group is left without a head.
template <bool WRITE, bool WIDE>
__global__ void __launch_bounds__(kThreads) k_kv4_rows(const KvViewDev v, const KvRowsDev r, float* __restrict__ k,
                                                       float* __restrict__ vv, long long ld,
                                                       unsigned char* __restrict__ cache, int lh, bool product) {
    pdl_wait();
    const StreamRows s = stream_rows(r, v, blockIdx.y);
    const int head_blocks = v.heads >> lh, row_block = blockIdx.x / head_blocks;
    const int head_block = blockIdx.x - row_block * head_blocks;
    const int row0 = row_block * (kGroups >> lh);
    if (row0 >= s.n) return;
    const int l8 = threadIdx.x & 7;
    const unsigned mask = 0xffu << (threadIdx.x & 24);
    const int part = v.page_rows * kKv4RowBytes;
    const unsigned page_bytes = static_cast<unsigned>(v.heads) * 2u * part;
    F8 x[kTasks][2];
    float* src[kTasks][2];                         // null: no such row
    unsigned char* blk[kTasks];                    // null: no place, nothing to store or zeros to read
    int pr[kTasks];
#pragma unroll
    for (int i = 0; i < kTasks; ++i) {
        const int g = (threadIdx.x >> 3) + i * (kThreads / 8);
        const int row = row0 + (g >> lh), head = (head_block << lh) + (g & ((1 << lh) - 1));
        blk[i] = nullptr;
        src[i][0] = nullptr;
        if (row >= s.n) continue;                  // (8 lanes alike)
        int page = 0;
        if (kv_place(v, s, row, page, pr[i]))
            blk[i] = cache + static_cast<unsigned long long>(static_cast<unsigned>(page)) * page_bytes + head * (2 * part);
        if (WRITE && !blk[i]) continue;
        const long long off = static_cast<long long>(s.row0 + row) * ld + (head * kHeadDim + l8 * 8);
        src[i][0] = k + off;
        src[i][1] = vv + off;
        if (WRITE) {
            x[i][0] = load8<WIDE>(src[i][0]);
            x[i][1] = load8<WIDE>(src[i][1]);
        }
    }
    // K words sit in the order 0 4 1 5 2 6 3 7, so that one 8-byte load of the attention kernels gives 8
    // dims of each scale's group; V's halves are kept rotated left by 2, as they unpack them
    const int kw = ((l8 & 3) * 2 + (l8 >> 2)) * 4, vw = part + l8 * 4, sw = v.page_rows * 32 + (l8 >> 2) * 2;
    if (WRITE) {
#pragma unroll
        for (int i = 0; i < kTasks; ++i) {
            if (!src[i][0]) continue;
            unsigned char* codes = blk[i] + pr[i] * 32;
            unsigned char* scale = blk[i] + sw + pr[i] * 4;
            uint32_t sk, sv;
            *reinterpret_cast<uint32_t*>(codes + kw) = kv4_quantise(x[i][0], mask, product, sk);
            const uint32_t w = kv4_quantise(x[i][1], mask, product, sv);
            *reinterpret_cast<uint32_t*>(codes + vw) = ((w << 2) & 0xfffcfffcu) | ((w >> 14) & 0x00030003u);
            if ((l8 & 3) == 0) {
                *reinterpret_cast<uint16_t*>(scale) = static_cast<uint16_t>(sk);
                *reinterpret_cast<uint16_t*>(scale + part) = static_cast<uint16_t>(sv);
            }
        }
    } else {
        uint32_t w[kTasks][2], sc[kTasks][2];
#pragma unroll
        for (int i = 0; i < kTasks; ++i) {
            w[i][0] = w[i][1] = sc[i][0] = sc[i][1] = 0;       // (a row without a place: scale 0 gives zeros)
            if (!blk[i]) continue;
            const unsigned char* codes = blk[i] + pr[i] * 32;
            const unsigned char* scale = blk[i] + sw + pr[i] * 4;
            w[i][0] = *reinterpret_cast<const uint32_t*>(codes + kw);
            w[i][1] = *reinterpret_cast<const uint32_t*>(codes + vw);
            sc[i][0] = *reinterpret_cast<const uint16_t*>(scale);
            sc[i][1] = *reinterpret_cast<const uint16_t*>(scale + part);
        }
#pragma unroll
        for (int i = 0; i < kTasks; ++i) {
            if (!src[i][0]) continue;
            store8<WIDE>(src[i][0], kv4_dequantise(w[i][0], __uint_as_float(sc[i][0] << 16)));
            const uint32_t y = ((w[i][1] >> 2) & 0x3fff3fffu) | ((w[i][1] << 14) & 0xc000c000u);
            store8<WIDE>(src[i][1], kv4_dequantise(y, __uint_as_float(sc[i][1] << 16)));
        }
    }
}

template <bool WRITE>
dec_status kv4_rows(const char* who, const dec_kv_view* view, const dec_kv_rows* rows, float* k, float* v, int64_t ld,
                    unsigned char* cache, int32_t scale_rule, void* stream) {
    const char* bad = view_problem(view, true);
    if (!bad) bad = rows_problem(rows);
    if (!bad && (!k || !v || !cache)) bad = "null pointer";
    if (!bad && (ld < static_cast<int64_t>(view->n_kv_heads) * kHeadDim || (ld & 3)))
        bad = "ld must be a multiple of 4 and at least n_kv_heads * 64";
    if (!bad && !(aligned16(k) && aligned16(v) && aligned16(cache))) bad = "k, v and cache must be 16-byte aligned";
    if (!bad && scale_rule != DEC_KV4_SCALE_QUOTIENT && scale_rule != DEC_KV4_SCALE_PRODUCT) bad = "unknown scale_rule";
    if (bad) return rows_fail(who, DEC_EINVAL, bad);
    int lh = 0;
    while (lh < 4 && view->n_kv_heads % (2 << lh) == 0) ++lh;
    const long long rows_per = kGroups >> lh;
    const long long blocks = (rows->max_rows + rows_per - 1) / rows_per * (view->n_kv_heads >> lh);
    if (blocks > 0x7fffffffll) return rows_fail(who, DEC_EINVAL, "max_rows * n_kv_heads is too large");
    const bool wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) | static_cast<uintptr_t>(ld * 4)) & 31) == 0;
    const cudaError_t e = rows_launch(wide ? k_kv4_rows<WRITE, true> : k_kv4_rows<WRITE, false>,
                                      dim3(static_cast<unsigned>(blocks), rows->batch), kThreads, 0,
                                      static_cast<cudaStream_t>(stream), view_dev(*view), rows_dev(*rows), k, v,
                                      static_cast<long long>(ld), cache, lh, scale_rule == DEC_KV4_SCALE_PRODUCT);
    if (e != cudaSuccess) return rows_cuda_fail(who, e, "k_kv4_rows launch");
    return DEC_OK;
}

}  // namespace

extern "C" {

size_t dec_kv4_bytes(const dec_kv_view* view) {
    if (view_problem(view, true)) return 0;
    return static_cast<size_t>(view->n_pages) * view->n_kv_heads * view->page_rows * (2 * kKv4RowBytes);
}

dec_status dec_kv4_write(const dec_kv_view* view, const dec_kv_rows* rows, const float* k, const float* v, int64_t ld,
                         void* cache, void* stream) {
    return kv4_rows<true>("dec_kv4_write", view, rows, const_cast<float*>(k), const_cast<float*>(v), ld,
                          static_cast<unsigned char*>(cache), DEC_KV4_SCALE_QUOTIENT, stream);
}

dec_status dec_kv4_write_scaled(const dec_kv_view* view, const dec_kv_rows* rows, const float* k, const float* v,
                                int64_t ld, void* cache, int32_t scale_rule, void* stream) {
    return kv4_rows<true>("dec_kv4_write_scaled", view, rows, const_cast<float*>(k), const_cast<float*>(v), ld,
                          static_cast<unsigned char*>(cache), scale_rule, stream);
}

dec_status dec_kv4_read(const dec_kv_view* view, const dec_kv_rows* rows, const void* cache, float* k_out,
                        float* v_out, int64_t ld, void* stream) {
    return kv4_rows<false>("dec_kv4_read", view, rows, k_out, v_out, ld,
                           static_cast<unsigned char*>(const_cast<void*>(cache)), DEC_KV4_SCALE_QUOTIENT, stream);
}

}  // extern "C"

// 4-bit K/V cache: quantising rows as they are stored (dec_kv4_write) and reading them back
// (dec_kv4_read).
//
// Per (row, K/V head, group of 32 dims): a = max |x|, s = bf16(a / 7), c = round(x / s) to the
// nearest integer, ties to even; value c s. The scale is rounded before the codes are chosen, so
// |x - c s| <= s / 2 holds whatever its rounding (a / s <= 7 (1 + 2^-8) rounds to 7), and bf16 keeps
// f32's range. c s has 3 + 8 significant bits: exact in f32, and in f16 up to a power of two.
//
// The code is decided exactly: c0 = rint(x * (1 / s)) is within one of it, and e = x - c0 s is exact
// in f32 (fma; c0 s has 11 significant bits and cancels x's leading ones; s >= 2^-126 keeps the last
// bit of c0 s above the subnormal grid), so comparing e with +-s / 2 settles borders and ties.
//
// One lane takes 8 consecutive dims: 8 lanes are one (row, head) of K or V, 4 lanes one scale.
// Bound by memory: 512 bytes read and 72 written per (row, K/V head), the reverse for reading back.
#include "kv_rows.cuh"

using namespace dec;

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int kv4_code(float x, float s, float inv) {
    float c = rintf(x * inv);
    c = fminf(fmaxf(c, -7.0f), 7.0f);
    const float e = fmaf(-c, s, x), h = 0.5f * s;
    int ci = static_cast<int>(c);
    if (e > h || (e == h && (ci & 1))) ci += 1;
    if (e < -h || (e == -h && (ci & 1))) ci -= 1;
    return min(max(ci, -7), 7);
}

template <bool WRITE>
__global__ void __launch_bounds__(kThreads) k_kv4_rows(const KvViewDev v, const KvRowsDev r, float* __restrict__ k,
                                                       float* __restrict__ vv, long long ld,
                                                       unsigned char* __restrict__ cache) {
    const int b = blockIdx.y;
    const StreamRows s = stream_rows(r, v, b);
    const int l8 = threadIdx.x & 7;
    const long long task = static_cast<long long>(blockIdx.x) * (kThreads / 8) + (threadIdx.x >> 3);
    // tasks: (row, head), head fastest; a group of 8 lanes leaves or stays together
    const int i = static_cast<int>(task / v.heads), head = static_cast<int>(task % v.heads);
    if (i >= s.n) return;
    int page = 0, pr = 0;
    const bool ok = kv_place(v, s, i, page, pr);
    if (WRITE && !ok) return;
    const unsigned mask = 0xffu << (threadIdx.x & 24);
    unsigned char* blk = cache + kv4_block(v, ok ? page : 0, head);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float4* x = reinterpret_cast<float4*>((which ? vv : k) + static_cast<long long>(s.row0 + i) * ld +
                                              head * kHeadDim + l8 * 8);
        unsigned char* part = blk + which * v.page_rows * kKv4RowBytes;
        // K words sit in the order 0 4 1 5 2 6 3 7, so that one 8-byte load of the attention kernels
        // gives 8 dims of each scale's group
        const int word = which ? l8 : (l8 & 3) * 2 + (l8 >> 2);
        uint32_t* codes = reinterpret_cast<uint32_t*>(part + pr * 32 + word * 4);
        uint16_t* scale = reinterpret_cast<uint16_t*>(part + v.page_rows * 32 + pr * 4 + (l8 >> 2) * 2);
        if (WRITE) {
            const float4 x0 = x[0], x1 = x[1];
            const float e[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
            float a = 0.0f;
            bool finite = true;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                a = fmaxf(a, fabsf(e[j]));
                finite = finite && fabsf(e[j]) <= 3.402823466e38f;
            }
            if (!finite) a = INFINITY;
            a = fmaxf(a, __shfl_xor_sync(mask, a, 1));
            a = fmaxf(a, __shfl_xor_sync(mask, a, 2));
            uint32_t w = 0x88888888u, sb = 0x7fc0u;
            if (a < INFINITY) {
                const float q = __fdiv_rn(a, 7.0f);
                const uint32_t u = __float_as_uint(q);
                sb = (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
                if (sb < 0x0080u) sb = 0;
                if (sb) {
                    const float sc = __uint_as_float(sb << 16), inv = 1.0f / sc;
                    w = 0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) w |= static_cast<uint32_t>(kv4_code(e[j], sc, inv) + 8) << (4 * j);
                }
            }
            // V's halves are kept rotated left by 2, as the attention kernels unpack them
            *codes = which ? ((w << 2) & 0xfffcfffcu) | ((w >> 14) & 0x00030003u) : w;
            if ((l8 & 3) == 0) *scale = static_cast<uint16_t>(sb);
        } else {
            float e[8];
            uint32_t w = ok ? *codes : 0x88888888u;
            if (which && ok) w = ((w >> 2) & 0x3fff3fffu) | ((w << 14) & 0xc000c000u);
            const float sc = ok ? __uint_as_float(static_cast<uint32_t>(*scale) << 16) : 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = sc * static_cast<float>(static_cast<int>((w >> (4 * j)) & 15u) - 8);
            x[0] = make_float4(e[0], e[1], e[2], e[3]);
            x[1] = make_float4(e[4], e[5], e[6], e[7]);
        }
    }
}

template <bool WRITE>
dec_status kv4_rows(const char* who, const dec_kv_view* view, const dec_kv_rows* rows, float* k, float* v, int64_t ld,
                    unsigned char* cache, void* stream) {
    const char* bad = view_problem(view, true);
    if (!bad) bad = rows_problem(rows);
    if (!bad && (!k || !v || !cache)) bad = "null pointer";
    if (!bad && (ld < static_cast<int64_t>(view->n_kv_heads) * kHeadDim || (ld & 3)))
        bad = "ld must be a multiple of 4 and at least n_kv_heads * 64";
    if (!bad && !(aligned16(k) && aligned16(v) && aligned16(cache))) bad = "k, v and cache must be 16-byte aligned";
    if (bad) return rows_fail(who, DEC_EINVAL, bad);
    const long long tasks = static_cast<long long>(rows->max_rows) * view->n_kv_heads;
    const long long blocks = (tasks + kThreads / 8 - 1) / (kThreads / 8);
    if (blocks > 0x7fffffffll) return rows_fail(who, DEC_EINVAL, "max_rows * n_kv_heads is too large");
    k_kv4_rows<WRITE><<<dim3(static_cast<unsigned>(blocks), rows->batch), kThreads, 0,
                        static_cast<cudaStream_t>(stream)>>>(view_dev(*view), rows_dev(*rows), k, v, ld, cache);
    const cudaError_t e = cudaGetLastError();
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
                          static_cast<unsigned char*>(cache), stream);
}

dec_status dec_kv4_read(const dec_kv_view* view, const dec_kv_rows* rows, const void* cache, float* k_out,
                        float* v_out, int64_t ld, void* stream) {
    return kv4_rows<false>("dec_kv4_read", view, rows, k_out, v_out, ld,
                           static_cast<unsigned char*>(const_cast<void*>(cache)), stream);
}

}  // extern "C"

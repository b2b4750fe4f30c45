// Row batches over a K/V cache in caller memory: the device view of dec_kv_view / dec_kv_rows,
// the 4-bit cache's layout, and the host-side checks shared by the entry points.
#pragma once

#include <string>

#include "../../include/dec.h"
#include "common.cuh"

void dec_set_thread_error(const char* msg);

namespace dec {

// ---- 4-bit cache layout ------------------------------------------------------------------
// One (page, head) block, pr rows:  K codes pr x 32 | K scales pr x 4 | V codes pr x 32 | V scales
// pr x 4. Per row and head K and V take 72 bytes; a block is one contiguous run, and every part of
// it starts on a 16-byte boundary (pr is a multiple of 16).
constexpr int kKv4Group = 32;        // dims per scale
constexpr int kKv4RowBytes = 36;     // codes and scales of one row of K (or V)

struct KvRowsDev {
    int batch, n_rows, max_rows;
    const int* row_start;   // null: row b belongs to stream b
    const int* slots;       // null: slot b
    const int* lens;
};

struct KvViewDev {
    int heads;              // K/V heads
    int shift;              // log2(page_rows), or 31 for one page of any size per slot
    int page_rows, pages_per_slot, n_slots, n_pages;
    const int* table;
};

// Rows of one slot.
__host__ __device__ __forceinline__ long long kv_capacity(const KvViewDev& v) {
    return static_cast<long long>(v.page_rows) * v.pages_per_slot;
}

// The rows of stream b: first row of the buffers, count (at most max_rows), slot, and the position
// of the first row. Malformed entries give an empty stream or rows without a place, never an
// access out of range.
struct StreamRows {
    int row0, n, slot;
    long long pos0;
};
__host__ __device__ __forceinline__ StreamRows stream_rows(const KvRowsDev& r, const KvViewDev& v, int b) {
    StreamRows s;
    int r0 = b, r1 = b + 1;
    if (r.row_start) {
        r0 = r.row_start[b];
        r1 = r.row_start[b + 1];
    }
    s.slot = r.slots ? r.slots[b] : b;
    const int len = r.lens[b];
    r0 = min(max(r0, 0), r.n_rows);
    r1 = min(max(r1, 0), r.n_rows);
    s.row0 = r0;
    const int all = max(r1 - r0, 0);
    s.n = min(all, r.max_rows);
    s.pos0 = static_cast<long long>(len) - all;
    if (s.slot < 0 || s.slot >= v.n_slots) s.slot = -1;
    return s;
}

// Physical page of a logical page of a slot (both in range), or -1.
__host__ __device__ __forceinline__ int kv_page(const KvViewDev& v, int slot, int lp) {
    const int at = slot * v.pages_per_slot + lp;
    const int p = v.table ? v.table[at] : at;
    return (p >= 0 && p < v.n_pages) ? p : -1;
}

// Page and row in it of the stream's i-th row; false where the row has no place.
__host__ __device__ __forceinline__ bool kv_place(const KvViewDev& v, const StreamRows& s, int i, int& page, int& pr) {
    const long long pos = s.pos0 + i;
    if (s.slot < 0 || pos < 0 || pos >= kv_capacity(v)) return false;
    page = kv_page(v, s.slot, static_cast<int>(pos) >> v.shift);
    pr = v.shift == 31 ? static_cast<int>(pos) : static_cast<int>(pos) & (v.page_rows - 1);
    return page >= 0;
}

// Byte offset of a (page, head) block of a 4-bit pool, float offset of one of an f32 pool.
__host__ __device__ __forceinline__ long long kv4_block(const KvViewDev& v, int page, int head) {
    return (static_cast<long long>(page) * v.heads + head) * v.page_rows * (2 * kKv4RowBytes);
}
__host__ __device__ __forceinline__ long long kvf_block(const KvViewDev& v, int page, int head) {
    return (static_cast<long long>(page) * v.heads + head) * v.page_rows * kHeadDim;
}

// Packed f32 pairs: a * b + c, a * b and a + b on both halves.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 d, a, b;\n\t"
        "mov.b64 {%0, %1}, d;}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 d, a, b;\n\t"
        "mov.b64 {%0, %1}, d;}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// ---- host-side checks ----------------------------------------------------------------------

inline dec_status rows_fail(const char* who, dec_status st, const std::string& msg) {
    dec_set_thread_error((std::string(who) + ": " + msg).c_str());
    return st;
}
inline dec_status rows_cuda_fail(const char* who, cudaError_t e, const char* what) {
    return rows_fail(who, DEC_ECUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

// Message of what is wrong with a view, or null. kv4: pages of 16, 32 or 64 rows only.
inline const char* view_problem(const dec_kv_view* v, bool kv4) {
    if (!v) return "null view";
    if (v->n_kv_heads < 1 || v->n_kv_heads > 65535) return "n_kv_heads must be in [1, 65535]";
    if (v->pages_per_slot < 1 || v->n_slots < 1 || v->n_pages < 1 || v->page_rows < 1)
        return "page_rows, pages_per_slot, n_slots and n_pages must be >= 1";
    const bool pow2 = v->page_rows == 16 || v->page_rows == 32 || v->page_rows == 64;
    if (!pow2 && (kv4 || v->table || v->pages_per_slot != 1))
        return "page_rows must be 16, 32 or 64 (an f32 cache without a table may have one page of any size per slot)";
    if (static_cast<long long>(v->page_rows) * v->pages_per_slot > 0x7fffff00ll) return "a slot holds too many rows";
    if (static_cast<long long>(v->n_slots) * v->pages_per_slot > 0x7fffffffll) return "too many logical pages";
    if (!v->table && static_cast<long long>(v->n_slots) * v->pages_per_slot > v->n_pages)
        return "without a table n_pages must hold n_slots * pages_per_slot pages";
    if (!aligned4(v->table)) return "table must be 4-byte aligned";
    return nullptr;
}

inline const char* rows_problem(const dec_kv_rows* r) {
    if (!r) return "null rows";
    if (!r->lens) return "null lens";
    if (!aligned4(r->row_start) || !aligned4(r->slots) || !aligned4(r->lens))
        return "row_start, slots and lens must be 4-byte aligned";
    if (r->batch < 1 || r->batch > 65535) return "batch must be in [1, 65535]";
    if (r->n_rows < 1) return "n_rows must be >= 1";
    if (r->max_rows < 1 || r->max_rows > r->n_rows) return "max_rows must be in [1, n_rows]";
    if (!r->row_start && (r->max_rows != 1 || r->n_rows < r->batch))
        return "without row_start every stream has one row (max_rows 1, n_rows >= batch)";
    return nullptr;
}

inline KvViewDev view_dev(const dec_kv_view& v) {
    KvViewDev d;
    d.heads = v.n_kv_heads;
    d.page_rows = v.page_rows;
    d.shift = v.page_rows == 16 ? 4 : v.page_rows == 32 ? 5 : v.page_rows == 64 ? 6 : 31;
    d.pages_per_slot = v.pages_per_slot;
    d.n_slots = v.n_slots;
    d.n_pages = v.n_pages;
    d.table = v.table;
    return d;
}
inline KvRowsDev rows_dev(const dec_kv_rows& r) {
    return KvRowsDev{r.batch, r.n_rows, r.max_rows, r.row_start, r.slots, r.lens};
}

// Launch whose blocks may be set up while the kernel before them on the stream ends; each kernel
// waits for it (griddepcontrol) before it reads anything.
template <typename... P, typename... Args>
cudaError_t rows_launch(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace dec

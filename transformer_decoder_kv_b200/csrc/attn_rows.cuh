// Attention of a row batch's queries with a sliding window and sinks: what its kernels share.
//
// A query at position p sees key j iff j <= p and (window == 0 or j > p - window or j < sinks):
// s_j = q . k_j / 8, p_j = exp(s_j - max), out = sum_j p_j v_j / sum_j p_j, zeros where the sum is
// not finite and positive.
//
// Work: the query rows of one (stream, K/V head) - row i of the stream and head g of the group are
// unit row i * group + g - are cut into units of UR rows. A unit's keys are the chunks (of CK
// positions) that any of its rows sees: the sinks' chunks, then the window's. They are split over
// at most S blocks; with more than one, each block leaves its running maximum, sum and weighted
// values per row in the workspace and k_attn_merge joins them in split order, so the result does
// not depend on the order in which blocks run.
#pragma once

#include "kv_rows.cuh"

namespace dec {

constexpr int kPartStride = 68;            // m (log2 domain), l, 2 unused, o[64]
constexpr int kRowsMaxSplits = 64;
constexpr int kRowsSms = 148;              // B200
constexpr float kLog2e = 1.4426950408889634f;

struct RowsAttnArgs {
    KvViewDev v;
    KvRowsDev r;
    const float* q;
    long long q_ld;
    int heads, group;            // query heads, query heads per K/V head
    const unsigned char* cache;  // 4-bit pool, or
    const float* k;              // f32 pools
    const float* vv;
    int window, sinks;
    float* out;
    long long out_ld;
    float* part;                 // [n_rows * heads, S] partial states
    int S;                       // splits launched per unit
    int per_split;               // chunks that make a split
};

// The keys of unit rows [u0, u0 + UR) of a stream in chunks of CK: chunks 0 .. sink_chunks - 1 and
// first .. first + (total - sink_chunks) - 1.
struct UnitKeys {
    int u0, n_u;              // unit rows (n_u 0: none)
    int sink_chunks, first, total;
    long long end;            // keys at or beyond end are not visible to any row
    int splits;               // blocks that take part
};

template <int UR, int CK>
__host__ __device__ __forceinline__ UnitKeys unit_keys(const RowsAttnArgs& a, const StreamRows& s, int unit) {
    UnitKeys k{};
    const long long all = static_cast<long long>(s.n) * a.group;
    const long long u0 = static_cast<long long>(unit) * UR;
    k.splits = 1;
    if (u0 >= all) return k;
    k.u0 = static_cast<int>(u0);
    k.n_u = static_cast<int>(all - u0 < UR ? all - u0 : UR);
    const long long p_first = s.pos0 + k.u0 / a.group, p_last = s.pos0 + (k.u0 + k.n_u - 1) / a.group;
    const long long cap = kv_capacity(a.v);
    k.end = p_last + 1 < cap ? p_last + 1 : cap;
    if (s.slot < 0 || k.end <= 0) {
        k.end = 0;
        return k;
    }
    long long lo = a.window > 0 && p_first - a.window + 1 > 0 ? p_first - a.window + 1 : 0;
    if (lo > k.end) lo = k.end;      // a window beyond the slot's last row: only the sinks are left
    const long long se = a.sinks < lo ? a.sinks : lo;
    int sc = static_cast<int>((se + CK - 1) / CK), fc = static_cast<int>(lo / CK);
    if (sc >= fc) {                  // the sinks reach the window's first chunk
        fc = se > 0 ? 0 : fc;
        sc = 0;
    }
    k.sink_chunks = sc;
    k.first = fc;
    k.total = sc + static_cast<int>((k.end + CK - 1) / CK) - fc;
    const int most = (k.total + a.per_split - 1) / a.per_split;
    k.splits = most < 1 ? 1 : (most < a.S ? most : a.S);
    return k;
}
__host__ __device__ __forceinline__ int unit_chunk(const UnitKeys& k, int t) {
    return t < k.sink_chunks ? t : k.first + t - k.sink_chunks;
}

// Chunks [begin, end) of split sp.
__host__ __device__ __forceinline__ int split_begin(const UnitKeys& k, int sp) {
    return static_cast<int>(static_cast<long long>(k.total) * sp / k.splits);
}

// The kernels on tensor cores weigh a key by 2^(s - ref) with ref 12 below the running maximum m (at it from 2^16
// on): for the joins and the output the sums go to weights of at most 1, where they are finite as long as
// f32 holds them at all. (ref + 12 is exact: a multiple of ref's last bit below 2^16.)
struct RowScale {
    float ref, mul;
};
__device__ __forceinline__ RowScale row_scale(float m, float ref) {
    return fabsf(m) < 65536.0f ? RowScale{ref + 12.0f, 1.0f / 4096.0f} : RowScale{ref, 1.0f};
}

// A block's result of unit row u, dims 4 d4 .. 4 d4 + 3: the output, or this split's partial state.
__device__ __forceinline__ void store_unit_row(const RowsAttnArgs& a, const UnitKeys& k, const StreamRows& s, int hk,
                                               int sp, int u, int d4, float m, float l, float4 o) {
    const int ur = k.u0 + u, h = hk * a.group + ur % a.group;
    const long long row = s.row0 + ur / a.group;
    if (k.splits == 1) {
        const bool ok = l > 0.0f && isfinite(l);
        *reinterpret_cast<float4*>(a.out + row * a.out_ld + h * kHeadDim + d4 * 4) =
            ok ? make_float4(o.x / l, o.y / l, o.z / l, o.w / l) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    } else {
        float* p = a.part + ((row * a.heads + h) * a.S + sp) * kPartStride;
        if (d4 == 0) *reinterpret_cast<float2*>(p) = make_float2(m, l);
        *reinterpret_cast<float4*>(p + 4 + d4 * 4) = o;
    }
}

// Chunks (of ck) of the widest unit of at most `rows` query rows, from the sizes the host knows.
inline long long rows_max_chunks(const KvViewDev& v, long long rows, int window, int sinks, int ck) {
    const long long cap = kv_capacity(v);
    long long keys = cap;
    if (window > 0) {
        const long long seen = static_cast<long long>(window) + rows + ck;
        keys = seen < cap ? seen : cap;
    }
    const long long extra = window > 0 && sinks > 0 ? (sinks < cap ? sinks : cap) : 0;
    const long long whole = (cap + ck - 1) / ck, c = (keys + ck - 1) / ck + (extra + ck - 1) / ck;
    return c < whole ? (c < 1 ? 1 : c) : whole;
}

// Joins the splits' partial states of each (row, head): a half-warp each, 16 bytes a lane. Eight splits'
// states are fetched at once, so a row costs about one round trip per eight splits.
template <int UR, int CK>
static __global__ void __launch_bounds__(128) k_attn_merge(const RowsAttnArgs a) {
    pdl_wait();
    const int d4 = threadIdx.x & 15;
    const StreamRows s = stream_rows(a.r, a.v, blockIdx.z);
    const int i = blockIdx.x * 8 + (threadIdx.x >> 4), h = blockIdx.y;
    if (i >= s.n) return;
    const UnitKeys k = unit_keys<UR, CK>(a, s, (i * a.group + h % a.group) / UR);
    if (k.splits <= 1) return;
    const long long row = s.row0 + i;
    const float* p = a.part + (row * a.heads + h) * a.S * kPartStride;
    float m = -INFINITY, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int sp0 = 0; sp0 < k.splits; sp0 += 8) {
        float2 ml[8];
        float4 x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            ml[j] = make_float2(-INFINITY, 0.0f);
            x[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (sp0 + j < k.splits) {
                ml[j] = __ldcg(reinterpret_cast<const float2*>(p + (sp0 + j) * kPartStride));
                x[j] = __ldcg(reinterpret_cast<const float4*>(p + (sp0 + j) * kPartStride + 4) + d4);
            }
        }
        float mn = m;
#pragma unroll
        for (int j = 0; j < 8; ++j) mn = fmaxf(mn, ml[j].x);
        const float corr = m == -INFINITY ? 0.0f : exp2f(m - mn);
        m = mn;
        l *= corr;
        o.x *= corr, o.y *= corr, o.z *= corr, o.w *= corr;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float w = ml[j].x == -INFINITY ? 0.0f : exp2f(ml[j].x - m);
            l = fmaf(w, ml[j].y, l);   // (a sum that is not a number stays one)
            if (w != 0.0f) {           // a split without weight adds nothing, whatever its values are
                o.x = fmaf(w, x[j].x, o.x);
                o.y = fmaf(w, x[j].y, o.y);
                o.z = fmaf(w, x[j].z, o.z);
                o.w = fmaf(w, x[j].w, o.w);
            }
        }
    }
    const bool ok = l > 0.0f && isfinite(l);
    *(reinterpret_cast<float4*>(a.out + row * a.out_ld + h * kHeadDim) + d4) =
        ok ? make_float4(o.x / l, o.y / l, o.z / l, o.w / l) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
}

}  // namespace dec

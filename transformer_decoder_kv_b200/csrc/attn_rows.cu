// dec_attention_kv4 and dec_attention_window: argument checks, the choice of kernel and split, and
// the launches (kernels: attn_rows.cuh, attn_kv4_few.cuh).
#include <algorithm>

#include "attn_kv4_few.cuh"
#include "attn_rows.cuh"

using namespace dec;

namespace {

template <bool KV4>
__global__ void __launch_bounds__(128) k_attn_rows(const RowsAttnArgs a) {
    const int lane = threadIdx.x & 31;
    const StreamRows s = stream_rows(a.r, a.v, blockIdx.z);
    const int i = blockIdx.x * 4 + (threadIdx.x >> 5), h = blockIdx.y;
    if (i >= s.n) return;
    const int hk = h / a.group;
    const long long row = s.row0 + i;
    const float2 q = *reinterpret_cast<const float2*>(a.q + row * a.q_ld + h * kHeadDim + 2 * lane);
    const long long p = s.pos0 + i;
    float m = -INFINITY, l = 0.0f, o0 = 0.0f, o1 = 0.0f;
    const long long end = s.slot < 0 ? 0 : min(p + 1, kv_capacity(a.v));
    const long long lo = a.window > 0 ? max(0ll, p - a.window + 1) : 0;
    long long j = a.sinks > 0 ? 0 : lo;
    while (j < end) {
        if (j < lo && j >= a.sinks) {
            j = lo;
            continue;
        }
        const int page = kv_page(a.v, s.slot, static_cast<int>(j) >> a.v.shift);
        const int pr = a.v.shift == 31 ? static_cast<int>(j) : static_cast<int>(j) & (a.v.page_rows - 1);
        ++j;
        if (page < 0) continue;
        float2 k, v;
        if (KV4) {
            const unsigned char* blk = a.cache + kv4_block(a.v, page, hk);
            auto get = [&](const unsigned char* part) {
                const int c = part[pr * 32 + lane];
                const float sc = __uint_as_float(
                    static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(part + a.v.page_rows * 32 + pr * 4 +
                                                                             (lane >> 4) * 2)) << 16);
                return make_float2(sc * static_cast<float>((c & 15) - 8), sc * static_cast<float>((c >> 4) - 8));
            };
            k = get(blk);
            v = get(blk + a.v.page_rows * kKv4RowBytes);
        } else {
            const long long off = kvf_block(a.v, page, hk) + static_cast<long long>(pr) * kHeadDim + 2 * lane;
            k = *reinterpret_cast<const float2*>(a.k + off);
            v = *reinterpret_cast<const float2*>(a.vv + off);
        }
        const float sc = warp_sum(fmaf(q.x, k.x, q.y * k.y)) * 0.125f;
        const float mn = fmaxf(m, sc);
        const float corr = m == mn ? 1.0f : expf(m - mn);
        const float w = sc == -INFINITY ? 0.0f : expf(sc - mn);
        l = fmaf(l, corr, w);
        if (w != 0.0f) {
            o0 = fmaf(w, v.x, o0 * corr);
            o1 = fmaf(w, v.y, o1 * corr);
        }
        m = mn;
    }
    const bool ok = l > 0.0f && isfinite(l);
    *reinterpret_cast<float2*>(a.out + row * a.out_ld + h * kHeadDim + 2 * lane) =
        ok ? make_float2(o0 / l, o1 / l) : make_float2(0.0f, 0.0f);
}

// Launch shape of a batch: unit rows per block, splits per unit.
struct RowsPlan {
    int unit_rows, tiles, S, min_chunks;
};

RowsPlan rows_plan(const dec_kv_view& view, const dec_kv_rows& rows, int n_heads, int window, int sinks) {
    RowsPlan p;
    const int group = n_heads / view.n_kv_heads;
    const long long u = static_cast<long long>(rows.max_rows) * group;
    p.unit_rows = u <= 4 ? 4 : u <= 8 ? 8 : 16;
    p.tiles = static_cast<int>((u + p.unit_rows - 1) / p.unit_rows);
    const long long units = static_cast<long long>(rows.batch) * view.n_kv_heads * p.tiles;
    const long long chunks = rows_max_chunks(view_dev(view), rows.max_rows, window, sinks, kFewChunk);
    p.min_chunks = kFewWarps;
    // Fewest (waves of resident blocks) x (rounds of chunks per warp, and one for the block's start and
    // end); a merge costs about one more.
    const long long slots = kRowsSms * (p.unit_rows == 4 ? 4 : p.unit_rows == 8 ? 3 : 2);
    long long best = 0;
    for (int S = 1; S <= kRowsMaxSplits && (S == 1 || chunks / S >= p.min_chunks); ++S) {
        const long long rounds = ((chunks + S - 1) / S + kFewWarps - 1) / kFewWarps;
        const long long cost = (units * S + slots - 1) / slots * (rounds + 1) + (S > 1);
        if (S == 1 || cost < best) best = cost, p.S = S;
    }
    return p;
}

template <typename K, typename... Args>
cudaError_t launch_after(K kern, dim3 grid, dim3 block, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int NT, bool PAIR>
cudaError_t launch_kv4_few(const RowsAttnArgs& a, const RowsPlan& p, cudaStream_t st) {
    constexpr int UR = PAIR ? 4 : 8 * NT;
    static_assert(kFewWarps * kFewStages * kFewStageBytes <= 48 * 1024, "no opt-in needed");
    k_attn_kv4_few<NT, PAIR><<<dim3(p.S, a.v.heads * p.tiles, a.r.batch), kFewWarps * 32, few_smem_bytes(UR), st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.S == 1) return e;
    return launch_after(k_attn_merge<UR, kFewChunk>, dim3((a.r.max_rows + 3) / 4, a.heads, a.r.batch), dim3(128), st, a);
}

template <bool KV4>
dec_status attn_rows(const char* who, const dec_kv_view* view, const dec_kv_rows* rows, const float* q, int64_t q_ld,
                     int32_t n_heads, const void* cache, const float* k, const float* v, int32_t window,
                     int32_t sinks, float* out, int64_t out_ld, void* workspace, size_t workspace_bytes,
                     void* stream) {
    const char* bad = view_problem(view, KV4);
    if (!bad) bad = rows_problem(rows);
    if (!bad && (!q || !out || !workspace || (KV4 ? !cache : (!k || !v)))) bad = "null pointer";
    if (!bad && (n_heads < 1 || n_heads > 65535 || n_heads % view->n_kv_heads))
        bad = "n_heads must be a multiple of n_kv_heads, at most 65535";
    if (!bad && (window < 0 || sinks < 0)) bad = "window and sinks must be >= 0";
    const int64_t d = static_cast<int64_t>(n_heads) * kHeadDim;
    if (!bad && (q_ld < d || out_ld < d || ((q_ld | out_ld) & 3)))
        bad = "q_ld and out_ld must be multiples of 4 and at least n_heads * 64";
    if (!bad && !(aligned16(q) && aligned16(out) && aligned16(workspace) && aligned16(cache) && aligned16(k) &&
                  aligned16(v)))
        bad = "q, out, workspace and the caches must be 16-byte aligned";
    if (!bad && (static_cast<long long>(rows->max_rows) * n_heads + 4 * view->n_kv_heads) / 4 > 65535)
        bad = "max_rows * n_heads is too large";
    if (!bad && workspace_bytes < dec_attention_rows_workspace_size(view, rows, n_heads)) bad = "workspace too small";
    if (bad) return rows_fail(who, DEC_EINVAL, bad);
    RowsAttnArgs a{};
    a.v = view_dev(*view);
    a.r = rows_dev(*rows);
    a.q = q;
    a.q_ld = q_ld;
    a.heads = n_heads;
    a.group = n_heads / view->n_kv_heads;
    a.cache = static_cast<const unsigned char*>(cache);
    a.k = k;
    a.vv = v;
    a.window = window;
    a.sinks = sinks;
    a.out = out;
    a.out_ld = out_ld;
    const RowsPlan plan = rows_plan(*view, *rows, n_heads, window, sinks);
    a.part = static_cast<float*>(workspace);
    a.S = plan.S;
    a.min_chunks = plan.min_chunks;
    if (KV4) {
        const cudaStream_t st = static_cast<cudaStream_t>(stream);
        const cudaError_t e = plan.unit_rows == 4   ? launch_kv4_few<1, true>(a, plan, st)
                              : plan.unit_rows == 8 ? launch_kv4_few<1, false>(a, plan, st)
                                                    : launch_kv4_few<2, false>(a, plan, st);
        return e == cudaSuccess ? DEC_OK : rows_cuda_fail(who, e, "k_attn_kv4_few launch");
    }
    k_attn_rows<KV4><<<dim3((rows->max_rows + 3) / 4, n_heads, rows->batch), 128, 0,
                       static_cast<cudaStream_t>(stream)>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return rows_cuda_fail(who, e, "k_attn_rows launch");
    return DEC_OK;
}

}  // namespace

extern "C" {

size_t dec_attention_rows_workspace_size(const dec_kv_view* view, const dec_kv_rows* rows, int32_t n_heads) {
    if (view_problem(view, false) || rows_problem(rows) || n_heads < 1 || n_heads % view->n_kv_heads) return 0;
    const RowsPlan p = rows_plan(*view, *rows, n_heads, 0, 0);
    return 256 + (p.S > 1 ? static_cast<size_t>(rows->n_rows) * n_heads * p.S * kPartStride * sizeof(float) : 0);
}

dec_status dec_attention_kv4(const dec_kv_view* view, const dec_kv_rows* rows, const float* q, int64_t q_ld,
                             int32_t n_heads, const void* cache, int32_t window, int32_t sinks, float* out,
                             int64_t out_ld, void* workspace, size_t workspace_bytes, void* stream) {
    return attn_rows<true>("dec_attention_kv4", view, rows, q, q_ld, n_heads, cache, nullptr, nullptr, window, sinks,
                           out, out_ld, workspace, workspace_bytes, stream);
}

dec_status dec_attention_window(const dec_kv_view* view, const dec_kv_rows* rows, const float* q, int64_t q_ld,
                                int32_t n_heads, const float* k, const float* v, int32_t window, int32_t sinks,
                                float* out, int64_t out_ld, void* workspace, size_t workspace_bytes, void* stream) {
    return attn_rows<false>("dec_attention_window", view, rows, q, q_ld, n_heads, nullptr, k, v, window, sinks, out,
                            out_ld, workspace, workspace_bytes, stream);
}

}  // extern "C"

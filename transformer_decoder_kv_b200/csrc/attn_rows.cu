// dec_attention_kv4 and dec_attention_window: argument checks, the choice of kernel and split, and
// the launches (kernels: attn_kv4_few.cuh, attn_f32_few.cuh, attn_f32_mma.cuh, attn_rows_tc.cuh; the
// join of splits: attn_rows.cuh).
#include <algorithm>

#include "attn_f32_few.cuh"
#include "attn_f32_mma.cuh"
#include "attn_kv4_few.cuh"
#include "attn_rows.cuh"
#include "attn_rows_tc.cuh"

using namespace dec;

namespace {

// Launch shape of a batch: unit rows per block, units per (stream, K/V head), splits per unit.
struct RowsPlan {
    bool tc;
    int unit_rows, resident, warps, chunk, least;    // blocks per SM; warps that share a block's chunks;
                                                     // keys per chunk; fewest chunks worth a split
    int group;
    long long tiles, units;
    int most_splits;                                 // what the workspace is sized for
    int S, per_split;
};

// Unit rows: the smallest few-row variant that holds a stream's rows of one group, several units of the
// widest one, and the tensor-core tiles of 128 rows where those take longer. Measured on B200, us.
//   4-bit cache, units against tiles (a further unit of 16 rows adds 27, the tile does not change):
//     32 streams x 1024 rows x 16 heads, 32 rows 56 / 86, 48 rows 83 / 87; 32 x 2048 x 2, 63 rows 26 / 29
//   f32 cache, the same streams: 32 rows (two units of 16) 137 / 208, a third unit would add 60
//   f32 cache, CUDA cores against mma.sync: 256 streams x 4096 x 4 heads, 3 rows 364 / 390; 256 x 8192 x 1,
//     4 rows 226 / 204; 256 x 8192 x 2, 7 rows 689 / 401, 16 rows 1306 / 491
// The bound on the splits does not depend on the window.
RowsPlan rows_shape(bool kv4, const dec_kv_view& view, const dec_kv_rows& rows, int n_heads) {
    RowsPlan p{};
    p.group = n_heads / view.n_kv_heads;
    const long long u = static_cast<long long>(rows.max_rows) * p.group;
    p.tc = u > (kv4 ? 64 : 32);
    if (p.tc) {
        p.unit_rows = kRtRows;
        p.resident = 2, p.warps = 1, p.chunk = kRtKeys, p.least = 1;
    } else if (kv4) {
        p.unit_rows = u <= 4 ? 4 : u <= 8 ? 8 : 16;
        p.resident = u <= 4 ? 4 : u <= 8 ? 3 : 2;
        p.warps = kFewWarps, p.chunk = kFewChunk, p.least = kFewWarps;
    } else {
        p.unit_rows = u <= 1 ? 1 : u <= 2 ? 2 : u <= 8 ? 8 : 16;
        p.resident = u <= 1 ? 5 : u <= 2 ? 4 : 2;
        p.warps = kF32Warps, p.chunk = kF32Chunk, p.least = 2 * kF32Warps;
    }
    p.tiles = (u + p.unit_rows - 1) / p.unit_rows;
    p.units = static_cast<long long>(rows.batch) * view.n_kv_heads * p.tiles;
    const long long slots = static_cast<long long>(kRowsSms) * p.resident;
    const long long all = rows_max_chunks(view_dev(view), 1, 0, 0, p.chunk);
    p.most_splits = static_cast<int>(std::max(
        1ll, std::min({static_cast<long long>(kRowsMaxSplits), (p.tc ? 8 : 2) * slots / p.units, all / p.least})));
    return p;
}

// Splits: the fewest (waves of resident blocks) x (rounds of chunks per block, and its start and end), a
// merge counting as one more round. For the tensor-core tiles, whose blocks are few and long:
//   - a batch whose n_rows falls short of batch * max_rows has about as many units as its rows fill, and
//     their blocks differ in length, so its waves are counted in parts (16 chunks of 5 to 128 rows over 513
//     to 4129 keys: 63 us, where whole waves of full streams had given 5 splits and 69 us; 4 would take 60);
//   - elsewhere of the splits within a tenth of the best the finest is taken;
//   - where the splits make more than one wave their length is fixed, so that the blocks of short and long
//     streams are alike (in one wave a short stream is rather split as often as it can be).
void rows_splits(RowsPlan& p, const dec_kv_view& view, const dec_kv_rows& rows, int window, int sinks) {
    const long long span = std::min<long long>(rows.max_rows, p.unit_rows / p.group + 1);
    const int chunks = static_cast<int>(rows_max_chunks(view_dev(view), span, window, sinks, p.chunk));
    const int most = std::max(1, std::min(p.most_splits, chunks / p.least));
    const long long slots = static_cast<long long>(kRowsSms) * p.resident, start = p.tc ? 2 : 1;
    long long units = p.units;
    bool parts = false;
    if (p.tc && rows.batch > 1) {
        const long long filled = view.n_kv_heads * (static_cast<long long>(rows.n_rows) * p.group / p.unit_rows + rows.batch / 2);
        parts = 10 * filled < 9 * units;
        if (parts) units = std::max(1ll, filled);
    }
    auto cost = [&](long long S) {                 // in sixteenths of a round
        const long long rounds = ((chunks + S - 1) / S + p.warps - 1) / p.warps + start;
        const long long waves = parts ? 16 * std::max(slots, units * S) / slots : (units * S + slots - 1) / slots * 16;
        return waves * rounds + (S > 1 ? 16 : 0);
    };
    p.S = 1;
    long long best = most > 1 ? cost(1) : 0;
    for (int S = 2; S <= most; ++S) {
        const long long c = cost(S);
        if (c < best) best = c, p.S = S;
    }
    if (p.tc && !parts)
        for (int S = most; S > p.S; --S)
            if (10 * cost(S) <= 11 * best) p.S = S;
    p.per_split = !p.tc ? p.least : units * p.S <= slots ? 2 : (chunks + p.S - 1) / p.S;
}

size_t rows_workspace(const RowsPlan& p, const dec_kv_rows& rows, int n_heads) {
    return 256 + (p.most_splits > 1
                      ? static_cast<size_t>(rows.n_rows) * n_heads * p.most_splits * kPartStride * sizeof(float)
                      : 0);
}

template <int UR, int CK>
cudaError_t launch_merge(const RowsAttnArgs& a, const RowsPlan& p, cudaStream_t st) {
    if (p.S == 1) return cudaSuccess;
    return rows_launch(k_attn_merge<UR, CK>, dim3((a.r.max_rows + 7) / 8, a.heads, a.r.batch), 128, 0, st, a);
}

template <typename K>
cudaError_t launch_units(K kern, const RowsAttnArgs& a, const RowsPlan& p, int threads, size_t smem, cudaStream_t st) {
    return rows_launch(kern, dim3(p.S, static_cast<unsigned>(a.v.heads * p.tiles), a.r.batch), threads, smem, st, a);
}

template <int NT, bool PAIR>
cudaError_t launch_kv4_few(const RowsAttnArgs& a, const RowsPlan& p, cudaStream_t st) {
    constexpr int UR = PAIR ? 4 : 8 * NT;
    static_assert(kFewWarps * kFewStages * kFewStageBytes <= 48 * 1024, "no opt-in needed");
    const cudaError_t e = launch_units(k_attn_kv4_few<NT, PAIR>, a, p, kFewWarps * 32, few_smem_bytes(UR), st);
    return e == cudaSuccess ? launch_merge<UR, kFewChunk>(a, p, st) : e;
}

template <bool KV4>
cudaError_t launch_rows_tc(const RowsAttnArgs& a, const RowsPlan& p, cudaStream_t st) {
    thread_local int attr_dev = -1;
    cudaError_t e = prefer_max_shared_once(k_attn_rows_tc<KV4>, attr_dev, rt_smem_bytes<KV4>());
    if (e == cudaSuccess) e = launch_units(k_attn_rows_tc<KV4>, a, p, kRtThreads, rt_smem_bytes<KV4>(), st);
    return e == cudaSuccess ? launch_merge<kRtRows, kRtKeys>(a, p, st) : e;
}

template <int R>
cudaError_t launch_f32_few(const RowsAttnArgs& a, const RowsPlan& p, cudaStream_t st) {
    const cudaError_t e = launch_units(k_attn_f32_few<R>, a, p, kF32Warps * 32, 0, st);
    return e == cudaSuccess ? launch_merge<R, kF32Chunk>(a, p, st) : e;
}

template <int NT>
cudaError_t launch_f32_mma(const RowsAttnArgs& a, const RowsPlan& p, cudaStream_t st) {
    const cudaError_t e = launch_units(k_attn_f32_mma<NT>, a, p, kF32Warps * 32, 0, st);
    return e == cudaSuccess ? launch_merge<8 * NT, kF32Chunk>(a, p, st) : e;
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
    RowsPlan plan{};
    if (!bad) {
        plan = rows_shape(KV4, *view, *rows, n_heads);
        if (workspace_bytes < dec_attention_rows_workspace_size(view, rows, n_heads)) bad = "workspace too small";
        if (plan.tiles * view->n_kv_heads > 65535) bad = "max_rows * n_heads is too large";
    }
    if (bad) return rows_fail(who, DEC_EINVAL, bad);
    rows_splits(plan, *view, *rows, window, sinks);
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
    a.part = static_cast<float*>(workspace);
    a.S = plan.S;
    a.per_split = plan.per_split;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (plan.unit_rows == kRtRows)
        e = launch_rows_tc<KV4>(a, plan, st);
    else if (KV4)
        e = plan.unit_rows == 4   ? launch_kv4_few<1, true>(a, plan, st)
            : plan.unit_rows == 8 ? launch_kv4_few<1, false>(a, plan, st)
                                  : launch_kv4_few<2, false>(a, plan, st);
    else
        e = plan.unit_rows == 1   ? launch_f32_few<1>(a, plan, st)
            : plan.unit_rows == 2 ? launch_f32_few<2>(a, plan, st)
            : plan.unit_rows == 8 ? launch_f32_mma<1>(a, plan, st)
                                  : launch_f32_mma<2>(a, plan, st);
    return e == cudaSuccess ? DEC_OK : rows_cuda_fail(who, e, "attention kernel launch");
}

}  // namespace

extern "C" {

size_t dec_attention_rows_workspace_size(const dec_kv_view* view, const dec_kv_rows* rows, int32_t n_heads) {
    if (view_problem(view, false) || rows_problem(rows) || n_heads < 1 || n_heads % view->n_kv_heads) return 0;
    return std::max(rows_workspace(rows_shape(false, *view, *rows, n_heads), *rows, n_heads),
                    rows_workspace(rows_shape(true, *view, *rows, n_heads), *rows, n_heads));
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

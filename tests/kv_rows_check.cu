// Host-only check of the row batch's index arithmetic (csrc/kv_rows.cuh): whatever the device
// arrays hold, every place that kv_place returns lies inside the pool, rows lie inside the row
// buffers, and well-formed batches get exactly their rows. Prints "ok".
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "attn_rows.cuh"

void dec_set_thread_error(const char*) {}

using namespace dec;

#define CHECK(c)                                             \
    do {                                                     \
        if (!(c)) {                                          \
            std::printf("line %d: %s\n", __LINE__, #c);      \
            return 1;                                        \
        }                                                    \
    } while (0)

static unsigned seed = 12345;
static unsigned rnd() { return seed = seed * 1664525u + 1013904223u; }
static int wild() {
    static const int v[] = {0, 1, -1, 5, 31, 32, 63, 64, 1000, -1000, 0x7fffffff, -0x7fffffff - 1, 0x7ffffff0};
    return v[(rnd() >> 8) % (sizeof(v) / sizeof(v[0]))];
}

// A unit's chunks hold every key that one of its rows sees exactly once, end inside the slot, and
// are shared out completely among the splits; the launch bound covers them.
template <int UR, int CK>
static int check_units() {
    for (int rep = 0; rep < 3000; ++rep) {
        const int page_rows = rep % 3 ? 16 << (rep % 3) : 16, pages = 1 + static_cast<int>((rnd() >> 8) % 40);
        dec_kv_view v{1, page_rows, pages, 1, pages, nullptr};
        RowsAttnArgs a{};
        a.v = view_dev(v);
        a.group = 1 + static_cast<int>((rnd() >> 8) % 9);
        a.heads = a.group;
        a.window = (rnd() >> 8) % 3 ? static_cast<int>((rnd() >> 8) % 300) : 0;
        a.sinks = (rnd() >> 8) % 2 ? static_cast<int>((rnd() >> 8) % 90) : 0;
        a.S = 1 + static_cast<int>((rnd() >> 8) % 9);
        a.per_split = 1 + static_cast<int>((rnd() >> 8) % 5);
        StreamRows s;
        s.row0 = 0;
        s.n = 1 + static_cast<int>((rnd() >> 8) % 70);
        s.slot = 0;
        const long long cap = kv_capacity(a.v);
        s.pos0 = static_cast<long long>((rnd() >> 8) % (cap + 40)) - 30;
        const int units = (s.n * a.group + UR - 1) / UR;
        for (int unit = 0; unit <= units; ++unit) {
            const UnitKeys k = unit_keys<UR, CK>(a, s, unit);
            CHECK(unit < units ? k.n_u >= 1 && k.n_u <= UR : k.n_u == 0);
            if (!k.n_u) continue;
            CHECK(k.splits >= 1 && k.splits <= a.S && k.end <= cap && k.total >= 0);
            CHECK(k.total <= rows_max_chunks(a.v, UR / a.group + 1, a.window, a.sinks, CK));
            CHECK(split_begin(k, 0) == 0 && split_begin(k, k.splits) == k.total);
            std::vector<int> seen(cap + CK, 0);
            for (int sp = 0; sp < k.splits; ++sp)
                for (int t = split_begin(k, sp); t < split_begin(k, sp + 1); ++t)
                    for (int j = 0; j < CK; ++j) {
                        const long long at = static_cast<long long>(unit_chunk(k, t)) * CK + j;
                        CHECK(at >= 0 && at < cap + CK);
                        seen[at] += 1;
                    }
            for (int u = k.u0; u < k.u0 + k.n_u; ++u) {
                const long long p = s.pos0 + u / a.group;
                for (long long j = 0; j < cap; ++j) {
                    const bool vis = j <= p && (a.window == 0 || j > p - a.window || j < a.sinks);
                    CHECK(!vis || (seen[j] == 1 && j < k.end));
                    CHECK(seen[j] <= 1);
                }
            }
        }
    }
    return 0;
}

int main() {
    if (check_units<4, 64>() || check_units<16, 64>() || check_units<8, 16>() || check_units<16, 16>() || check_units<1, 16>() || check_units<128, 128>()) return 1;
    const int shapes[][4] = {{16, 3, 4, 12}, {32, 1, 1, 1}, {64, 7, 5, 40}, {300, 1, 6, 6}, {16, 130000, 900, 5}};
    for (const auto& sh : shapes) {
        for (int paged = 0; paged < 2; ++paged) {
            dec_kv_view v{3, sh[0], sh[1], sh[2], sh[3], nullptr};
            if (sh[0] == 300 && paged) continue;
            if (!paged) v.n_pages = v.n_slots * v.pages_per_slot;
            std::vector<int> table(static_cast<size_t>(v.n_slots) * v.pages_per_slot);
            for (auto& t : table) t = (rnd() >> 9) % 3 ? static_cast<int>((rnd() >> 4) % v.n_pages) : wild();
            if (paged) v.table = table.data();
            CHECK(view_problem(&v, false) == nullptr);
            const KvViewDev d = view_dev(v);
            const long long pool = static_cast<long long>(v.n_pages) * 3 * v.page_rows;
            for (int rep = 0; rep < 4000; ++rep) {
                const int B = 3, n_rows = 9;
                int start[4], slots[3], lens[3];
                for (int& x : start) x = (rnd() >> 9) % 2 ? static_cast<int>((rnd() >> 5) % 10) : wild();
                for (int& x : slots) x = (rnd() >> 9) % 2 ? static_cast<int>((rnd() >> 5) % v.n_slots) : wild();
                for (int& x : lens) x = (rnd() >> 9) % 2 ? static_cast<int>((rnd() >> 5) % 70) : wild();
                dec_kv_rows r{B, n_rows, 1 + static_cast<int>((rnd() >> 6) % n_rows), rep % 5 ? start : nullptr,
                              rep % 3 ? slots : nullptr, lens};
                if (!r.row_start) r.max_rows = 1;
                CHECK(rows_problem(&r) == nullptr);
                const KvRowsDev rd = rows_dev(r);
                for (int b = 0; b < B; ++b) {
                    const StreamRows s = stream_rows(rd, d, b);
                    CHECK(s.n >= 0 && s.n <= r.max_rows);
                    CHECK(s.n == 0 || (s.row0 >= 0 && s.row0 + s.n <= n_rows));
                    CHECK(s.slot >= -1 && s.slot < v.n_slots);
                    for (int i = 0; i < s.n; ++i) {
                        int page = -5, pr = -5;
                        if (!kv_place(d, s, i, page, pr)) continue;
                        CHECK(page >= 0 && page < v.n_pages && pr >= 0 && pr < v.page_rows);
                        for (int h = 0; h < 3; ++h) {
                            CHECK(kvf_block(d, page, h) / kHeadDim + pr < pool);
                            CHECK(kv4_block(d, page, h) + static_cast<long long>(v.page_rows) * 72 <= pool * 72);
                        }
                    }
                }
            }
        }
    }
    // a well-formed ragged batch: stream 1 holds rows 2..5 at positions 29..32 of slot 2
    const int start[] = {0, 2, 6, 6}, slots[] = {0, 2, 1}, lens[] = {2, 33, 0};
    dec_kv_view v{2, 16, 3, 3, 9, nullptr};
    dec_kv_rows r{3, 8, 4, start, slots, lens};
    const KvViewDev d = view_dev(v);
    const StreamRows s = stream_rows(rows_dev(r), d, 1);
    CHECK(s.row0 == 2 && s.n == 4 && s.slot == 2 && s.pos0 == 29);
    int page, pr;
    CHECK(kv_place(d, s, 3, page, pr) && page == 2 * 3 + 2 && pr == 0);
    CHECK(kv_place(d, s, 0, page, pr) && page == 2 * 3 + 1 && pr == 13);
    CHECK(stream_rows(rows_dev(r), d, 2).n == 0);
    std::printf("ok\n");
    return 0;
}

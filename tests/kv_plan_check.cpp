// Host check of the paged cache's index arithmetic (kv_plan.h): every row lies
// in its page and is given to one slot only, bad entries give -1 and are never
// followed, and the attention's units are shared out completely. Prints "ok".
#include <stdio.h>
#include <stdlib.h>

#include <set>
#include <vector>

#include "kv_plan.h"

#define CHECK(x)                                                  \
    do {                                                          \
        if (!(x)) {                                               \
            printf("line %d: %s does not hold\n", __LINE__, #x); \
            exit(1);                                              \
        }                                                         \
    } while (0)

using namespace dq;

static void rows(int pages, int page_size, int per_seq, int heads) {
    KvGeom g{make_kvdiv((uint32_t)page_size), pages, per_seq, heads};
    std::vector<int32_t> table((size_t)per_seq);
    for (int i = 0; i < per_seq; ++i) table[i] = (i * 7 + 3) % pages;
    std::set<int32_t> seen;
    for (int t = 0; t < per_seq * page_size; ++t)
        for (int h = 0; h < heads; ++h) {
            const int32_t r = kv_row(table.data(), (uint32_t)t, h, g);
            CHECK(r == (table[t / page_size] * heads + h) * page_size + t % page_size);
            CHECK(r >= 0 && r < pages * heads * page_size);
            if (per_seq <= pages && pages % 7) CHECK(seen.insert(r).second);
        }
    // beyond the table: never read (the sanitizer watches), no row
    CHECK(kv_row(table.data(), (uint32_t)(per_seq * page_size), 0, g) == -1);
    CHECK(kv_row(table.data(), 0xffffffffu, 0, g) == -1);
    for (int32_t bad : {-1, pages, pages + 1, INT32_MIN, INT32_MAX}) {
        table[0] = bad;
        CHECK(kv_row(table.data(), 0, heads - 1, g) == -1);
    }
}

static void pairs(int D, int R, bool il) {
    std::set<int> seen;
    for (int i = 0; i < D / 2; ++i) {
        int a, b;
        kv_pair(i, D, R, il, &a, &b);
        CHECK(a >= 0 && b >= 0 && a < D && b < D);
        CHECK(seen.insert(a).second && seen.insert(b).second);
        CHECK((i < R / 2) == (a < R) && (i < R / 2) == (b < R));
        if (i < R / 2) CHECK(il ? (a == 2 * i && b == 2 * i + 1) : (a == i && b == i + R / 2));
    }
}

static void shares(int64_t units, int W) {
    const KvShare s = kv_share(units, W);
    CHECK(s.workers >= (units > 0) && s.workers <= W && s.workers <= units);
    if (units == 0) return;
    CHECK(kv_first(0, s) == 0 && kv_first(s.workers, s) == units);
    int64_t least = units, most = 0;
    for (int w = 0; w < s.workers; ++w) {
        const int64_t a = kv_first(w, s), b = kv_first(w + 1, s);
        CHECK(a < b);  // every worker has something
        if (w + 1 < s.workers) least = b - a < least ? b - a : least;
        most = b - a > most ? b - a : most;
        for (int64_t u = a; u < b; ++u) CHECK(kv_worker(u, s) == w);
    }
    CHECK(most - least <= 1);
    CHECK(most <= (units + W - 1) / W);  // no worker has more than the evenest share
}

int main() {
    for (int ps : {1, 2, 8, 16, 24, 37, 128}) rows(11, ps, 9, 3);
    rows(1, 5, 1, 1);
    for (uint32_t d : {1u, 2u, 3u, 24u, 127u, 65535u, 0x40000000u}) {
        const KvDiv f = make_kvdiv(d);
        for (uint64_t n : {0ull, 1ull, (unsigned long long)d - 1, (unsigned long long)d, 0x7fffffffull, 0xffffffffull})
            CHECK(kv_div((uint32_t)n, f) == (uint32_t)n / d);
    }
    for (int D : {2, 16, 80, 96, 256})
        for (int R = 2; R <= D; R += 2) {
            pairs(D, R, false);
            pairs(D, R, true);
        }
    for (int W : {1, 2, 3, 255, 512, 768})
        for (int64_t u : {0ll, 1ll, 2ll, 7ll, 511ll, 512ll, 513ll, 4099ll, 38001ll}) shares(u, W);
    for (int n : {0, 1, 127, 128, 129, 5000})
        for (int w : {0, 1, 128, 1000, 6000}) {
            const int first = kv_first_token(n, w), units = kv_units(n, w);
            CHECK(first >= 0 && first <= n && (w == 0 ? first == 0 : n - first <= w));
            CHECK((int64_t)units * kKvUnit >= n - first && (int64_t)(units - 1) * kKvUnit < n - first);
        }
    printf("ok\n");
    return 0;
}

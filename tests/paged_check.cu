// Host-only check of how the paged attention shares out its work (no GPU needed; built by
// tests/test_paged_host.py with nvcc).  For batches drawn from a seed it walks the ranges of all shares as the kernels
// do and prints: batches, pieces, and how many of each kind of mistake it found: keys of a unit that no share or two
// take, units without keys not taken once, a partial result in the wrong slot or out of order (the join could not
// find it), and shares with much more than their part of the work.
#include <algorithm>
#include <cstdio>
#include <random>
#include <vector>

#include "paged_sched.cuh"
using namespace attn;
using namespace attn::paged;

static long long batches, pieces, holes, twice, empty_wrong, slot_wrong, chain_wrong, heavy, lane_wrong;

template <int kUnitCost, int kStep, int kLeast, int kShare>
void check(const std::vector<int> &lens, const std::vector<int> &news, bool packed, int tokens, int heads, int causal, int ctas)
{
    PagedSeqs s = {};
    std::vector<int> cu(1, 0);
    for (int m : news) cu.push_back(cu.back() + m);
    s.lens = lens.data();
    s.cu = packed ? cu.data() : nullptr;
    s.b = int(lens.size());
    s.s_q = news[0];
    s.tokens = cu.back();
    s.cap = 1 << 30;
    const Sched<kUnitCost> sc = {s, tokens, heads, causal};
    bool bad = false;
    std::vector<int64_t> base(1, 0);
    for (int n = 0; n < s.b; ++n) base.push_back(base.back() + sc.cost(sc.units(n, &bad)));
    const int64_t total = base.back();
    const int n_cta = Sched<kUnitCost>::template shares<kShare>(total, ctas);
    auto at = [&](int c, int *n, int *x, int *t, int *k) {
        const int64_t pos = Sched<kUnitCost>::border(total, n_cta, c);
        *n = s.b;
        *x = *t = *k = 0;
        if (pos >= total) return;
        *n = int(std::upper_bound(base.begin(), base.end(), pos) - base.begin()) - 1;
        sc.template locate<kStep, kLeast>(sc.units(*n, &bad), pos - base[*n], x, t, k);
    };
    ++batches;
    // the state of the walk over all shares in order
    int un = -1, ux = 0, ut = 0, done = 0;
    bool open = false;  // a unit begun and not ended
    std::vector<std::vector<int>> taken(s.b);  // times a unit's end was reached
    for (int n = 0; n < s.b; ++n) taken[n].assign(size_t(heads) * sc.units(n, &bad).nt, 0);
    for (int c = 0; c < n_cta; ++c) {
        Range r;
        r.any = total > 0;
        at(c, &r.n0, &r.x0, &r.t0, &r.k0);
        at(c + 1, &r.n1, &r.x1, &r.t1, &r.k1);
        Walk<kUnitCost> w(sc, r);
        int64_t load = 0;
        int in_share = 0;
        bool went_on = false;
        while (w.next()) {
            ++pieces;
            load += w.k1 - w.k0 + kUnitCost;
            if (went_on) ++slot_wrong;  // a piece that others follow has to be the share's last
            if (w.k0 > 0) {
                if (in_share > 0) ++slot_wrong;  // a piece that goes on from another share: the first
                if (!open || w.n != un || w.x != ux || w.t != ut) ++chain_wrong;
                else if (w.k0 > done) ++holes;
                else if (w.k0 < done) ++twice;
            } else if (open) {
                ++holes;
            }
            if (w.k0 % kStep || (w.k1 % kStep && w.k1 != w.all)) ++slot_wrong;
            un = w.n; ux = w.x; ut = w.t; done = w.k1;
            open = !w.ends();
            went_on = open;
            if (!open) ++taken[w.n][size_t(w.x) * w.u.nt + w.t];
            ++in_share;
        }
        const int64_t part = (total + n_cta - 1) / n_cta;
        // (borders are fractions of 2^-32 of the work, of which the last share gets what is rounded off)
        if (load > part + total / (int64_t(1) << 32) * n_cta + n_cta + 2 * kLeast + 2 * kStep + kUnitCost * (in_share + 1)) ++heavy;
    }
    if (open) ++holes;
    for (auto &v : taken)
        for (int k : v) {
            if (k == 0) ++empty_wrong;
            if (k > 1) ++twice;
        }
    if (bad) ++chain_wrong;
}

// Every share of every lane has one CTA, and every CTA a number of its own.
static void check_lanes(int heads, int ctas)
{
    std::vector<int> numbers(ctas, 0), shares(ctas, 0);
    for (int c = 0; c < ctas; ++c) {
        const Lanes x(heads, ctas, c);
        if (x.lanes < 1 || heads % x.lanes || x.lane >= x.lanes || x.per < 1 || x.share > x.per || x.me < 0 || x.me >= ctas) {
            ++lane_wrong;
            continue;
        }
        ++numbers[x.me];
        if (x.share < x.per) {
            if (x.me != x.lane * x.per + x.share) ++lane_wrong;
            ++shares[x.me];
        }
    }
    const Lanes x(heads, ctas, 0);
    for (int c = 0; c < ctas; ++c)
        if (numbers[c] != 1 || shares[c] != (c < x.per * x.lanes)) ++lane_wrong;
    if (x.per * x.lanes * 20 < ctas * 19) ++lane_wrong;  // at most a twentieth of the CTAs without work
}

int main()
{
    for (int heads = 1; heads < 400; ++heads)
        for (int ctas : {304, 456}) check_lanes(heads, ctas);
    std::mt19937 rng(5);
    auto upto = [&](int n) { return int(rng() % unsigned(n + 1)); };
    for (int i = 0; i < 4000; ++i) {
        const int b = 1 + upto(i % 10 == 0 ? 400 : 12), big = i % 3 == 0 ? 200 : i % 3 == 1 ? 3000 : 40000;
        std::vector<int> lens, news;
        const bool packed = i % 4 != 0;
        const int fixed = 1 + upto(i % 2 ? 3 : 600);
        for (int n = 0; n < b; ++n) {
            lens.push_back(upto(3) ? upto(big) : upto(20));
            news.push_back(!packed ? fixed : upto(4) == 0 ? 0 : upto(2) ? 1 + upto(5) : upto(i % 5 ? 700 : 5000));
            if (news.back() > lens.back() && upto(3)) lens.back() += news.back();
        }
        if (b > 1 && packed) news[0] = std::max(news[0], 1);
        check<384, 64, 64, 256>(lens, news, packed, 1 + upto(15), 1 + upto(40), i & 1, 456);
        check<384, 128, 128, 256>(lens, news, packed, 1 + upto(15), 1 + upto(7), i & 1, 608);
        check<256, 128, 512, 1024>(lens, news, packed, 1 + upto(255), 1 + upto(40), i & 1, 152);
    }
    // no tokens at all, and a cost past 32 bits
    check<384, 64, 64, 256>({5, 0}, {0, 0}, true, 2, 3, 1, 456);
    check<256, 128, 512, 1024>({1 << 30, 1 << 29}, {200000, 100000}, true, 8, 128, 1, 152);
    printf("batches %lld pieces %lld holes %lld twice %lld empty %lld slot %lld chain %lld heavy %lld lanes %lld\n", batches, pieces, holes,
           twice, empty_wrong, slot_wrong, chain_wrong, heavy, lane_wrong);
    return 0;
}

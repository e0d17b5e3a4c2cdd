// Host-only: the check of tests/paged_check.cu over the launches that there are.  The kernel for few rows runs 304
// or 456 CTAs, which neighbouring heads share out alike (Lanes): a lane of them walks its own shares, in steps of
// 64 or 128 keys; the tensor-core kernel runs 152.
#define main other_main
#include "paged_check.cu"
#undef main

template <int kStep> static void lane(std::mt19937 &rng, const std::vector<int> &lens, const std::vector<int> &news, bool packed, int causal, int ctas)
{
    const int blocks = 1 + int(rng() % 40);  // head blocks
    const Lanes x(blocks, ctas, 0);
    check<384, kStep, kStep, 256>(lens, news, packed, 1 + int(rng() % 16), blocks / x.lanes, causal, x.per);
}

int main()
{
    std::mt19937 rng(6);
    auto upto = [&](int n) { return int(rng() % unsigned(n + 1)); };
    for (int i = 0; i < 3000; ++i) {
        const int b = 1 + upto(i % 10 == 0 ? 1000 : 40), big = i % 3 == 0 ? 200 : i % 3 == 1 ? 3000 : 40000;
        std::vector<int> lens, news;
        const bool packed = i % 4 != 0;
        const int fixed = 1 + upto(i % 2 ? 3 : 40);
        for (int n = 0; n < b; ++n) {
            lens.push_back(upto(3) ? upto(big) : upto(20));
            news.push_back(!packed ? fixed : upto(4) == 0 ? 0 : upto(2) ? 1 + upto(5) : upto(700));
        }
        if (packed) news[0] = std::max(news[0], 1);
        lane<64>(rng, lens, news, packed, i & 1, 304);
        lane<128>(rng, lens, news, packed, i & 1, 304);
        lane<128>(rng, lens, news, packed, i & 1, 456);
        check<256, 128, 512, 1024>(lens, news, packed, 1 + upto(255), 1 + upto(40), i & 1, 152);
    }
    printf("batches %lld pieces %lld holes %lld twice %lld empty %lld slot %lld chain %lld heavy %lld\n", batches, pieces, holes, twice, empty_wrong,
           slot_wrong, chain_wrong, heavy);
    return 0;
}

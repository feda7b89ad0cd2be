// Host-side check of scored decode's cut (ScoredCut in decode_kernel.cuh): for
// many length mixes, head counts, grids and piece sizes, the ranges
// start_unit(c) .. start_unit(c + 1) must partition the units in order and
// range_of(u, s) must name the range holding unit u of segment s; while the
// grid has a warp for every piece, each range lies in one segment and holds at
// most `per` units.  Prints "ok" or the first violation; exit status 0 / 1.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "decode_kernel.cuh"

using pagedkv::dec::ScoredCut;

static int check(const std::vector<int>& nb, int H, int W, int per) {
    const int B = (int)nb.size();
    std::vector<int> pre(B + 1, 0), pcs(B + 1, 0);
    for (int b = 0; b < B; ++b) {
        pre[b + 1] = pre[b] + nb[b];
        pcs[b + 1] = pcs[b] + (nb[b] + per - 1) / per;
    }
    const int U = pre[B] * H;
    const ScoredCut cut(pre.data(), pcs.data(), B, H, W, per);
    std::vector<int> owner(U, -1);
    for (int c = 0, end = 0; c < W; ++c) {
        const int u0 = cut.start_unit(c), u1 = cut.start_unit(c + 1);
        if (u0 != end || u1 < u0 || u1 > U) {
            std::printf("B=%d H=%d W=%d per=%d: range %d is %d..%d after %d\n", B, H, W, per, c, u0, u1, end);
            return 1;
        }
        if (cut.aligned && u1 - u0 > per) {
            std::printf("range %d holds %d units of %d\n", c, u1 - u0, per);
            return 1;
        }
        for (int u = u0; u < u1; ++u) owner[u] = c;
        end = u1;
        if (c == W - 1 && end != U) {
            std::printf("B=%d H=%d W=%d per=%d: the last range ends at %d of %d\n", B, H, W, per, end, U);
            return 1;
        }
    }
    for (int b = 0; b < B; ++b)
        for (int g = 0; g < H; ++g)
            for (int k = 0; k < nb[b]; ++k) {
                const int s = b * H + g, u = pre[b] * H + g * nb[b] + k;
                if (cut.range_of(u, s) != owner[u]) {
                    std::printf("unit %d of segment %d: range_of %d, held by %d\n", u, s,
                                cut.range_of(u, s), owner[u]);
                    return 1;
                }
                if (cut.aligned && k > 0 && k % per != 0 && owner[u] != owner[u - 1]) {
                    std::printf("segment %d is cut inside a piece\n", s);
                    return 1;
                }
                if (cut.aligned && k == 0 && u > 0 && owner[u] == owner[u - 1]) {
                    std::printf("range %d holds two segments\n", owner[u]);
                    return 1;
                }
            }
    return 0;
}

int main() {
    std::srand(4321);
    long long cases = 0, aligned = 0;
    for (int trial = 0; trial < 300; ++trial) {
        const int B = 1 + std::rand() % (trial % 2 ? 300 : 12);
        std::vector<int> nb(B);
        for (int b = 0; b < B; ++b) {
            const int kind = std::rand() % 10;
            nb[b] = kind == 0 ? 0 : kind < 6 ? std::rand() % 8 : std::rand() % 200;
        }
        for (int H : {1, 2, 8})
            for (int W : {4, 96, 608, 1824})
                for (int per : {2, 4}) {
                    if (check(nb, H, W, per)) return 1;
                    ++cases;
                }
        aligned += nb.size() < 12;
    }
    std::printf("ok %lld cases\n", cases);
    return aligned > 0 ? 0 : 1;
}

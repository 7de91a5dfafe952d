// Schedules of k_pair_gemm, one line per "M N k_steps mx" of the input: bn pairs whole-waves tail split bytes.
#include <cstdio>

#include "../qlora_parameter_efficient_b200/csrc/pair_schedule.cuh"

int main() {
    long long m, n, k;
    int mx;
    while (scanf("%lld %lld %lld %d", &m, &n, &k, &mx) == 4) {
        const qlora::PairSched g = qlora::pair_schedule(m, n, k, mx, 74);
        const long long tiles = (m + 255) / 256 * ((n + g.bn - 1) / g.bn);
        printf("%d %d %lld %d %d %zu\n", g.bn, g.pairs, tiles / 74, g.tail, g.split, g.bytes());
    }
}

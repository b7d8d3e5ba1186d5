// Prints the host's plans (no GPU), one line for each line of standard input:
//   back rows cols elem mats num_sms -> threads_per_row eights_per_thread rows_per_block slots cluster ctas smem bytes
//   fp4 M N K num_sms pairs -> pair bn tiles_m tiles_n parts splits ws_bytes
// Read by tests/test_plans.py.
#include <cstdio>
#include <cstring>
#include "norm_fp4_plan.cuh"

using namespace fp8bs;

int main()
{
    char what[16];
    while (std::scanf("%15s", what) == 1) {
        if (std::strcmp(what, "fp4") == 0) {
            long long M, N, K;
            int sms, pairs;
            if (std::scanf("%lld %lld %lld %d %d", &M, &N, &K, &sms, &pairs) != 5) return 1;
            const Fp4Plan p = plan_fp4(M, N, K, sms, pairs != 0);
            std::printf("%d %d %d %d %d %d %zu\n", p.pair ? 1 : 0, p.bn, p.tiles_m, p.tiles_n, p.parts, p.splits, p.ws_bytes);
        } else if (std::strcmp(what, "back") == 0) {
            long long rows, cols;
            int elem, mats, sms;
            if (std::scanf("%lld %lld %d %d %d", &rows, &cols, &elem, &mats, &sms) != 5) return 1;
            const BackPlan b = plan_back(rows, cols, elem, mats, sms);
            std::printf("%d %d %d %d %d %lld %u %zu\n", b.shape.tx, b.shape.vpt, b.ty, b.slots, b.cluster, (long long)b.grid,
                        b.smem, b.bytes);
        } else {
            return 1;
        }
    }
    return 0;
}

// Prints how calls of the 4-bit weight operators are laid out: one line "M K group C gated" in, one line
// "kernel a b c d" out ("few pl nw passes rows depth lds", "mid ntl stages scales", "gemm large").
#include <stdio.h>

#include "w4_plan.hpp"

int main() {
    long M, K, group, C;
    int gated;
    while (scanf("%ld %ld %ld %ld %d", &M, &K, &group, &C, &gated) == 5) {
        const long N = gated ? 2 * C : C;
        qlin::W4FewPlan f;
        qlin::W4MidPlan m;
        if (qlin::w4_few_plan(M, K, group, C, gated, f))
            printf("few %d %d %d %d %d %u\n", f.pl, f.nw, f.passes, f.rows, f.depth, f.lds);
        else if (qlin::w4_mid_plan(M, K, group, C, gated, m) && qlin::w4_use_mid(M, N, K, group, m))
            printf("mid %d %d %u\n", m.ntl, m.stages, m.scales);
        else
            printf("gemm %ld\n", (long)qlin::w4_gemm_plan(M, N, K).large);
    }
    return 0;
}

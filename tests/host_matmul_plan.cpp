// Host-side driver for the planning rules of the 8-bit products in qg_matmul_plan.h,
// built with the host compiler alone: nothing here touches a GPU.  One query per input
// line, "R E I O bf16 gated direct fits ncu" -> "tile kind parts head head_kind bm".
#include "qg_matmul_plan.h"

#include <cstdio>

int main()
{
    qg::MatmulSizes p{};
    int bf16, gated, direct, fits;
    long long ncu;
    while (std::scanf("%d %d %d %d %d %d %d %d %lld", &p.R, &p.E, &p.I, &p.O, &bf16, &gated,
                      &direct, &fits, &ncu) == 9) {
        p.bf16 = bf16 != 0;
        p.gated = gated != 0;
        const qg::MatmulPlan m = qg::plan_matmul(p, fits != 0, direct != 0, ncu);
        std::printf("%d %d %d %d %d %d\n", m.tile, m.plan.kind, m.plan.parts, m.plan.head,
                    m.plan.head_kind, m.bm);
    }
    return 0;
}

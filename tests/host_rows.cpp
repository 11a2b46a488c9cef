// Host-side driver for qg_rows.h.  One query per input line, two sets of rows:
//   p n width ld  p n width ld   -> 1 if they share a byte, else 0
#include "qg_rows.h"

#include <cstdio>

int main()
{
    qg::Rows r[2];
    for (;;) {
        for (auto &v : r) {
            unsigned long long p;
            if (std::scanf("%llu %lld %lld %lld", &p, &v.n, &v.width, &v.ld) != 4) return 0;
            v.p = p;
        }
        std::printf("%d\n", qg::overlap(r[0], r[1]));
    }
}

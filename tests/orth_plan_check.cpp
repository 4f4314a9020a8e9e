// Host-only check of which sizes the orthogonalised update takes in one launch
// (csrc/bstq_orth_plan.h): reads lines "m n widest" on stdin and prints whether and
// with how many blocks to a cluster.  Built and run by tests/test_orthogonalize.py.
#include <cstdio>

#include "bstq_orth_plan.h"

int main()
{
    long long m, n;
    int widest;
    while (std::scanf("%lld %lld %d", &m, &n, &widest) == 3)
        std::printf("%d %d\n", (int)bstq::is_small(m, n, widest), bstq::cluster_of(m < n ? n : m));
    return 0;
}

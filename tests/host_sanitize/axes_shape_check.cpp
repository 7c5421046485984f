// The launches that the rotation with several axes makes (axes.h), for the sizes on standard input: a line
// "f32 halves vector batch tokens q_heads k_heads head_dim pairs axes" gives a line "planes together jobs
// launch_tokens groups", groups being the workgroups of the largest launch.  Built for the host alone.
#include <cstdio>

#include "axes.h"

using namespace ltx3drope;

int main() {
    unsigned f32, halves, vector, batch, tokens, q_heads, k_heads, head_dim, pairs, axes;
    while (std::scanf("%u %u %u %u %u %u %u %u %u %u", &f32, &halves, &vector, &batch, &tokens, &q_heads, &k_heads,
                      &head_dim, &pairs, &axes) == 10) {
        AxesProblem p{};
        for (AxesTensor* t : {&p.q, &p.k}) {
            t->heads = t == &p.q ? q_heads : k_heads;
            t->in_head = t->out_head = head_dim;
        }
        p.f32 = f32 != 0;
        p.halves = halves != 0;
        p.vector = vector;
        p.batch = batch;
        p.tokens = tokens;
        p.head_dim = head_dim;
        p.pairs = pairs;
        p.axes = axes;
        const AxesShape s = axes_shape(p);
        const unsigned most = axes_launch_tokens(s);
        std::printf("%u %u %u %u %u\n", s.segments + s.copies, s.together, axes_jobs(s), most,
                    axes_launch_groups(s, tokens < most ? tokens : most));
    }
    return 0;
}

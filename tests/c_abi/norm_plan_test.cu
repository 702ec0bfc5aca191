/* The block norms' plans (norm_plan of seq_norm.cuh), on the host alone: every
 * plan that is taken fits a block's shared memory, has clusters and covers the
 * channels and positions.  Prints the plans that do not, and a count. */
#include <cstdio>

#include "seq_norm.cuh"

using namespace spconv::seq;

int main() {
    static float some;
    long plans = 0, wide = 0, bad = 0;
    for (int dtype : {SPCONV_F32, SPCONV_BF16, SPCONV_F16})
        for (int extra : {0, 8})
            for (bool vec : {true, false})
                for (int inputs = 1; inputs <= (extra ? kNormInputs : 3); ++inputs)
                    for (int L : {1, 3, 8, 9, 16, 24, 33, 64, 1000, 4096})
                        for (int C = 1; C < 70000; C += C < 4200 ? 1 : 61) {
                            NormParams p{};
                            for (int i = 0; i < inputs; ++i) p.in[i] = &some;
                            p.N = 3, p.C = C, p.L = L;
                            const int W = norm_plan(p, dtype, extra, vec), V = 16 / (int)dtype_size(dtype);
                            ++plans;
                            if (W == 0) {
                                ++wide;
                                continue;
                            }
                            const int rows = kNormThreads / W;
                            const bool good = p.shared <= kNormShared && p.clusters >= 1 && p.stages >= 1 && p.R >= 1 &&
                                              p.ranks <= kNormRanks && (int64_t)p.per * p.ranks >= C && rows * p.R >= p.per &&
                                              (int64_t)p.tiles * W * V >= L;
                            if (!good && ++bad <= 20)
                                std::printf("type %d, gradients %d, whole rows %d, %d inputs, C %d, L %d: W %d, %d blocks of %d runs, "
                                            "%d stages, %d bytes, %d clusters\n",
                                            dtype, extra != 0, vec, inputs, C, L, W, p.ranks, p.R, p.stages, p.shared, p.clusters);
                        }
    std::printf("%ld plans, %ld without a cluster that holds the channels, %ld bad\n", plans, wide, bad);
    return bad != 0;
}

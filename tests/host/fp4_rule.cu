// Prints, for every five numbers on the command line (block, tokens a tile, tiles, stages, SMs), what fp4_few.cuh makes of such a product: CTAs a
// tile, places of the ring, bytes of shared memory, and bytes of a stage and of what a CTA is sent.
#include <cstdio>
#include <cstdlib>

#include "fp4_few.cuh"

int main(int argc, char** argv) {
    for (int i = 1; i + 4 < argc; i += 5) {
        int v[5];
        for (int j = 0; j < 5; ++j) v[j] = std::atoi(argv[i + j]);
        const sgemv::FewPlan f = sgemv::few_plan(v[0], v[1], v[2], v[3], v[4]);
        std::printf("%d %d %d %d %d\n", f.split, f.ring, f.smem, sgemv::few_stage_bytes(v[0], v[1]), f.split > 1 ? sgemv::few_sent(v[1], f.split) : 0);
    }
}

// Prints, for every seven numbers on the command line (dim, KV heads, query heads a KV head, requests, new tokens, the most of a
// request, SMs), the rows past which a request is the chunk kernel's (kv_common.cuh), -1 where none is.
#include <cstdio>
#include <cstdlib>

#include "kv_common.cuh"

int main(int argc, char** argv) {
    for (int i = 1; i + 6 < argc; i += 7) {
        int v[7];
        for (int j = 0; j < 7; ++j) v[j] = std::atoi(argv[i + j]);
        const int rows = sgemv::chunk_threshold(v[0], v[1], v[2], v[3], v[4], v[5], v[6]);
        std::printf("%d\n", rows == INT_MAX ? -1 : rows);
    }
}

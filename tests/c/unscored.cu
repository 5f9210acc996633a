// Every thread of every block over an entry, giving up at each tile in turn (host code only): the keys
// that were scored before and those left -inf are all of the entry's, each once, and nothing else.
#include <cstdio>
#include <vector>

#include "unscored.cuh"

int main() {
    const uint32_t kTile = 128, sets[] = {1, 2, 4};
    for (uint32_t kv_len : {1u, 127u, 128u, 129u, 1000u, 4097u})
        for (uint32_t blocks : {1u, 2u, 3u, 7u})
            for (uint32_t n : sets)
                for (uint32_t give_up = 0; give_up < 12; ++give_up) {
                    const uint32_t tiles = (kv_len + kTile - 1) / kTile;
                    std::vector<float> out(kv_len + 2 * kTile, 5.0f);
                    std::vector<int> times(kv_len + 2 * kTile, 0);
                    for (uint32_t b = 0; b < blocks; ++b) {
                        const uint32_t mine = b < tiles ? (tiles - b + blocks - 1) / blocks : 0;
                        for (uint32_t set = 0; set < n; ++set)
                            for (uint32_t t = 0; t < kTile; ++t) {
                                uint32_t it = set, j = (b + set * blocks) * kTile + t;
                                for (; it < mine && it < give_up; it += n, j += n * blocks * kTile)
                                    if (j < kv_len) out[j] = 1.0f, ++times[j];
                                if (it < mine) {
                                    std::vector<float> left(out.size(), 5.0f);
                                    dsrows::unscored(left.data(), it, mine, n, j, n * blocks * kTile, kv_len);
                                    for (size_t k = 0; k < left.size(); ++k)
                                        if (left[k] != 5.0f) out[k] = left[k], ++times[k];
                                }
                            }
                    }
                    for (uint32_t k = 0; k < out.size(); ++k) {
                        const bool scored = k / kTile / blocks < give_up;
                        const float want = k >= kv_len ? 5.0f : scored ? 1.0f : -INFINITY;
                        if (out[k] != want || times[k] != (k < kv_len ? 1 : 0)) {
                            printf("key %u of %u: %g, %d times (%u blocks, %u sets, given up at %u)\n", k, kv_len, out[k],
                                   times[k], blocks, n, give_up);
                            return 1;
                        }
                    }
                }
    printf("every key once\n");
    return 0;
}

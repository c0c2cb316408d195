// Replays, through the address functions that the kernels call, what extent_check_f8.cpp leaves out: rows past a tile's last, gathered
// rows, and scales. Each lane's load of each block lies inside an aligned chunk that holds an element, or behind the
// descriptor with and without the block's offset, and no sum passes 32 bits.
//   extent_check_f8_rows rows ROWS K LD TILE        a tile of TILE rows of which the last of ROWS fill a part
//   extent_check_f8_rows gather ROWS K LD TILE      rows taken from anywhere in a matrix of ROWS
//   extent_check_f8_rows scales ROWS BLOCKS S_ROW S_COL
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <vector>

#include "tile_addressing.h"

using namespace regtile::addr;

static int fail(const char *what, long long a, long long b) {
    printf("FAIL %s: %lld %lld\n", what, a, b);
    return 1;
}

// Rows `from` (of the descriptor's) of one tile; `end`: bytes from its base to behind the last element
static int tile(const std::vector<int64_t> &from, int height, int K, int64_t ld, uint32_t span, int64_t end) {
    const int used = (int)from.size(), blocks = (K + 127) / 128;
    for (int kb = 0; kb < blocks; kb += (blocks > 3 && kb == 0) ? blocks - 2 : 1) {
        std::vector<int64_t> slot(height * 8, -2);
        for (int q = 0; q < height / 8; ++q)
            for (int lane = 0; lane < 64; ++lane) {
                const int r = f8_row(q, lane);
                const uint32_t of_lane = f8_row_lane(q, lane, used, from[r < used ? r : used - 1], ld), of_block = f8_block(false, kb, ld);
                const uint64_t at = (uint64_t)of_lane + of_block;
                if (at >> 32) return fail("past 32 bits", (long long)at, kb);
                if (r >= used && (of_lane < span || at < span)) return fail("a row past the last is loaded", r, (long long)at);
                if (at % 16) return fail("alignment", (long long)at, kb);
                if (at < span && (int64_t)at >= end) return fail("chunk without an element", (long long)at, end);
                if (slot[q * 64 + lane] != -2) return fail("slot twice", q, lane);
                slot[q * 64 + lane] = at < span ? (int64_t)at : -1;
            }
        for (int i = 0; i < used; ++i)
            for (int k = 0; k < 128 && kb * 128 + k < K; ++k)
                if (slot[i * 8 + (k / 16 ^ slab_key<8, 16>(i))] != from[i] * ld + (kb * 128 + k) / 16 * 16) return fail("element", i, kb * 128 + k);
    }
    return 0;
}

static int rows(bool gather, int64_t n, int K, int64_t ld, int height) {
    if (!f8_reach(false, gather ? n : 256, K, ld)) {
        printf("not taken\n");
        return 0;
    }
    uint64_t seed = 12345;
    for (int used = 1; used <= height; used = used < height && used * 3 > height ? height : used * 3) {
        std::vector<int64_t> from;
        int64_t last = used - 1;
        for (int i = 0; i < used; ++i) {
            seed = seed * 6364136223846793005ull + 1442695040888963407ull;
            from.push_back(!gather ? i : i == 0 ? n - 1 : i == 1 ? 0 : (int64_t)(seed >> 33) % n);
        }
        if (!gather && used > n) break;
        if (gather) last = n - 1;
        if (tile(from, height, K, ld, f8_span(last + 1, ld, K), last * ld + K)) return 1;
        if (used == height) break;
    }
    printf("ok\n");
    return 0;
}

static int scales(int64_t n, int64_t blocks, int64_t s_row, int64_t s_col) {
    if (!f8_scales_reach(n, s_row, blocks, s_col)) {
        printf("not taken\n");
        return 0;
    }
    const int step = f8_scale_step(s_col);
    const int64_t rs[4] = {0, n / 2, n - 1, n > 1 ? 1 : 0}, ks[4] = {0, blocks / 2, blocks - 1, blocks > 1 ? 1 : 0};
    for (int64_t r : rs)
        for (int64_t k : ks) {
            const uint64_t at = (uint64_t)f8_scale_lane(r, s_row) + f8_scale_block((int)k, step);
            if ((int64_t)at != (r * s_row + k * s_col) * 4) return fail("scale", r, k);
            if (at + 4 > 0x7FFFFFFFull) return fail("scale past the descriptor", r, k);
        }
    printf("ok\n");
    return 0;
}

int main(int argc, char **argv) {
    if (argc != 6) return 2;
    const int64_t a = atoll(argv[2]), b = atoll(argv[3]), c = atoll(argv[4]), d = atoll(argv[5]);
    if (strcmp(argv[1], "scales") == 0) return scales(a, b, c, d);
    return rows(strcmp(argv[1], "gather") == 0, a, (int)b, c, (int)d);
}

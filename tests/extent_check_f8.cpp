// Replays the DMA of the 8-bit float tiles on the host, through the address functions that the kernels call. For one
// operand of one problem: every lane's load of every block of the first and the last tile either lies wholly inside
// an aligned chunk of 16 bytes that holds an element of the matrix's span, or past the descriptor (zeros); every element of
// the tile arrives in its LDS slot; and no two lanes fill the same slot.
//   extent_check_f8 kc ROWS K LD TILE     K-contiguous rows, tiles of TILE rows
//   extent_check_f8 nn K N LD TILE        K x N, tiles of TILE columns
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

template <int BN>
static int check(bool nn, int64_t rows, int K, int64_t ld) {
    const int blocks = (K + 127) / 128, tiles = (int)((rows + BN - 1) / BN);
    if (!f8_reach(nn, 256, K, ld)) {
        printf("not taken\n");
        return 0;
    }
    for (int t = 0; t < tiles; t += tiles > 1 ? tiles - 1 : 1) {
        const int first = t * BN, n = (int)(rows - first < BN ? rows - first : BN);
        // bytes from the descriptor's base to behind the matrix's last element, and that chunk's end
        const int64_t end = nn ? (int64_t)(K - 1) * ld + (rows - first) : (int64_t)(rows - first - 1) * ld + K;
        const uint32_t span = nn ? f8_span(K, ld, (int)(rows - first)) : f8_span(n, ld, K);
        if ((int64_t)span > (end + 15) / 16 * 16) return fail("span", span, end);
        for (int kb = 0; kb < blocks; kb += (blocks > 3 && kb == 0) ? blocks - 2 : 1) {
            std::vector<int64_t> slot(BN * 8, -2);
            for (int q = 0; q < BN / 8; ++q)
                for (int lane = 0; lane < 64; ++lane) {
                    const int r = f8_row(q, lane);
                    const uint64_t at = (uint64_t)(nn ? f8_nn_lane<BN>(q, lane, n, ld) : f8_lane(q, lane, r < n ? r : n - 1, ld)) + f8_block(nn, kb, ld);
                    if (at >> 32) return fail("past 32 bits", (long long)at, kb);
                    if (at % 16) return fail("alignment", (long long)at, kb);
                    if (at < span && (int64_t)at >= end) return fail("chunk without an element", (long long)at, end);
                    int64_t &s = slot[q * 64 + lane];
                    if (s != -2) return fail("slot twice", q, lane);
                    s = at < span ? (int64_t)at : -1;
                }
            for (int i = 0; i < n; ++i)
                for (int k = 0; k < 128 && kb * 128 + k < K; ++k) {
                    const int64_t want = nn ? (int64_t)(kb * 128 + k) * ld + i : (int64_t)i * ld + kb * 128 + k;
                    const int c = nn ? i / 16 : k / 16;
                    const int at = nn ? k * (BN / 16) + (c ^ f8_nn_key<BN>(k)) : i * 8 + (c ^ slab_key<8, 16>(i));
                    if (slot[at] != want / 16 * 16) return fail("element", i, kb * 128 + k);
                }
        }
    }
    printf("ok\n");
    return 0;
}

int main(int argc, char **argv) {
    if (argc != 6) return 2;
    const bool nn = strcmp(argv[1], "nn") == 0;
    const int64_t a = atoll(argv[2]), b = atoll(argv[3]), ld = atoll(argv[4]);
    const int tile = atoi(argv[5]);
    const int64_t rows = nn ? b : a;
    const int K = (int)(nn ? a : b);
    return tile == 64 ? check<64>(nn, rows, K, ld) : tile == 128 ? check<128>(nn, rows, K, ld) : check<256>(nn, rows, K, ld);
}

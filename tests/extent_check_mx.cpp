// extent_check_mx.cpp -- host replay of what the block-scaled (MX) kernels compute from their sizes.
//
// extent_check.cpp with the block-scaled kernels' paths added; the checks of an access are its own
// (included here with its main renamed).
//   extent_check_mx units <cols>          units of 8 columns of a converted row: every column in one unit,
//                                         and no unit without one
//   extent_check_mx bytes <0|1> <cols>    bytes of a row's codes (1: fp4): the last code in the last of them
//   extent_check_mx one|force <nt|nn|tn|tt> M N K lda ldc
//                                         the descriptors of gemm_mx_dma.hip and gemm_mx_codes.hip: every
//                                         access of A and C, on each tile that the launchers may take
//                                         (force: 256-wide tiles, whatever the admission rules say)
//   extent_check_mx sweep <seed> <count>  seeded shapes, leading dimensions up to the descriptors' limits
#define main extent_check_main
#include "extent_check.cpp"
#undef main

namespace {

int check_units(int cols) {
    const int64_t n = addr::mx_units(cols);
    if (n < 1 || (n - 1) * 8 >= cols || n * 8 < cols) {
        std::printf("VIOLATION %lld units for %d columns\n", (long long)n, cols);
        return 1;
    }
    std::printf("%lld units\n", (long long)n);
    return 0;
}

int check_bytes(bool fp4, int cols) {
    const int64_t n = addr::mx_row_bytes(fp4, cols), per = fp4 ? 2 : 1;
    if (n < 1 || n > 2147483647 || (n - 1) * per >= cols || n * per < cols) {
        std::printf("VIOLATION %lld bytes for %d columns\n", (long long)n, cols);
        return 1;
    }
    std::printf("%lld bytes\n", (long long)n);
    return 0;
}

// A product on t-wide tiles. A is read as the 16-bit DMA kernel reads it; C is the caller's, or the
// workspace's parts (M x N, no padding).
void check_tile(bool ta, int M, int N, int K, int64_t lda, int64_t ldc, int t, bool parts) {
    if (ta)
        check_mn_operand("A", M, K, lda, t);
    else
        check_kc_operand<32>("A", M, K, lda, t);
    check_c<32>(M, N, parts ? N : ldc, t);
}

bool check_mx(bool ta, bool tb, int M, int N, int K, int64_t lda, int64_t ldc) {
    if (g_force) {
        check_tile(ta, M, N, K, lda, ldc, 256, true);
        return true;
    }
    if (!addr::mx_dma_takes(ta, tb, M, N, K, lda, ldc)) return false;
    const int t = addr::dma_tile(M, N);
    check_tile(ta, M, N, K, lda, ldc, t, false);
    if (t == 128) check_tile(ta, M, N, K, lda, ldc, t, true);
    if (addr::mx_wide_parts(ta, M, N, K, lda) > 1) check_tile(ta, M, N, K, lda, ldc, 256, true);
    return true;
}

int report(long taken) {
    std::printf("taken %ld loads %ld stores %ld violations %ld\n", taken, g_loads, g_stores, g_violations);
    return g_violations ? 1 : 0;
}

int sweep(uint64_t seed, int count) {
    std::mt19937_64 rng(seed);
    const int sizes[] = {1, 2, 8, 24, 32, 64, 72, 96, 127, 128, 129, 160, 255, 256, 257, 264, 384, 512, 1000, 1504, 2049, 8224};
    const int depths[] = {8, 32, 64, 72, 96, 128, 777, 1000, 1504, 8192, 8288, 8320};
    auto pick = [&](auto &of) { return of[rng() % (sizeof of / sizeof of[0])]; };
    long taken = 0;
    for (int c = 0; c < count; ++c) {
        const bool ta = rng() & 1, tb = rng() & 1;
        const int M = pick(sizes), N = pick(sizes), K = pick(depths);
        const int64_t pad[] = {0, 8, 4096, int64_t(1) << 21, int64_t(1) << 22, (int64_t(1) << 22) + 4096, int64_t(3) << 21, int64_t(1) << 23};
        const int64_t lda = (ta ? M : K) + pick(pad), ldc = N + (rng() % 3 ? 0 : (int64_t)(rng() % 5));
        taken += check_mx(ta, tb, M, N, K, lda, ldc);
    }
    return report(taken);
}

}  // namespace

int main(int argc, char **argv) {
    if (argc == 8 && (std::strcmp(argv[1], "one") == 0 || std::strcmp(argv[1], "force") == 0)) {
        g_force = std::strcmp(argv[1], "force") == 0;
        return report(check_mx(argv[2][0] == 't', argv[2][1] == 't', std::atoi(argv[3]), std::atoi(argv[4]), std::atoi(argv[5]),
                               std::atoll(argv[6]), std::atoll(argv[7])));
    }
    if (argc == 4 && std::strcmp(argv[1], "sweep") == 0) return sweep(std::strtoull(argv[2], nullptr, 10), std::atoi(argv[3]));
    if (argc == 3 && std::strcmp(argv[1], "units") == 0) return check_units(std::atoi(argv[2]));
    if (argc == 4 && std::strcmp(argv[1], "bytes") == 0) return check_bytes(std::atoi(argv[2]) != 0, std::atoi(argv[3]));
    std::fprintf(stderr, "usage: extent_check_mx units <cols> | bytes <0|1> <cols> | one|force <nt|nn|tn|tt> M N K lda ldc | sweep <seed> <count>\n");
    return 2;
}

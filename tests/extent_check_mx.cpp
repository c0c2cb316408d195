// extent_check_mx.cpp -- host replay of what the block-scaled (MX) kernels compute from their sizes.
//
// extent_check.cpp with the block-scaled kernels' paths added; the checks of an access are its own
// (included here with its main renamed).
//   extent_check_mx units <cols>          units of 8 columns of a converted row: every column in one unit,
//                                         and no unit without one
//   extent_check_mx bytes <0|1> <cols>    bytes of a row's codes (1: fp4): the last code in the last of them
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

}  // namespace

int main(int argc, char **argv) {
    if (argc == 3 && std::strcmp(argv[1], "units") == 0) return check_units(std::atoi(argv[2]));
    if (argc == 4 && std::strcmp(argv[1], "bytes") == 0) return check_bytes(std::atoi(argv[2]) != 0, std::atoi(argv[3]));
    std::fprintf(stderr, "usage: extent_check_mx units <cols> | bytes <0|1> <cols>\n");
    return 2;
}

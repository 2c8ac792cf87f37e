// Prints the form that the rules of vocab.h give each shape (n vocab dim in_place,
// four arguments a shape): pieces, the last one's rows, and the tile and splits of
// the two gradients' sums, in the first piece and in the last.
#include <cstdio>
#include <cstdlib>

#include "vocab.h"

int main(int argc, char **argv) {
    using namespace zdo;
    for (int i = 1; i + 3 < argc; i += 4) {
        const int64_t n = std::atoll(argv[i]), vocab = std::atoll(argv[i + 1]), dim = std::atoll(argv[i + 2]);
        const bool in_place = std::atoi(argv[i + 3]) != 0;
        const CeLayout l = ce_layout(n, vocab, dim, in_place);
        const int64_t pieces = ceil_div(vocab, l.piece), last = vocab - (pieces - 1) * l.piece;
        auto tile = [](int64_t m, int64_t rows, int64_t splits) { return wide_tiles(m, rows, splits) ? 256 : 128; };
        std::printf("%lld %s, last %lld; sum %d/%lld, rows %d/%lld%s\n", (long long)pieces,
                    in_place ? "in place" : "copied", (long long)last, tile(dim, n, l.splits), (long long)l.splits,
                    tile(dim, l.piece, l.row_splits), (long long)l.row_splits,
                    tile(dim, last, l.row_splits) == tile(dim, l.piece, l.row_splits) ? "" : " (last otherwise)");
    }
    return 0;
}

// The order in which a block of kda_scan goes through its tiles; plain C++, so that a host can go through it as well.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define KDA_SCAN_COURSE __device__ __forceinline__
#else
#define KDA_SCAN_COURSE inline
#endif

namespace kda {
namespace scan {

struct tile {
    int n, p, count;   // sequence, position in the direction of the scan (-1: no tile), tiles of the sequence
    int a, b;          // the sequence's tokens
    int block;         // of channels
    int first;         // slot of the sequence's first tile
};

// From a tile (none before the first) to the next one: of the same chain where a block takes whole chains, else the first one that
// item(&t) finds, which sets n, p (-1: an item without a tile), a, b and block and is false behind the last item.  There p is -1,
// and stays so however often the next tile is asked for: a tile that is asked for is one that somebody waits for.
template <int L, typename Item> KDA_SCAN_COURSE void next_tile(tile &t, bool chains, bool back, Item &&item) {
    if (chains && t.p + 1 < t.count) {
        ++t.p;
        return;
    }
    do {
        t.p = -1;
        if (!item(&t)) {
            t.count = 0;  // (of the last chain: its tiles do not begin again)
            return;
        }
    } while (t.p < 0);
    t.count = (t.b - t.a + L - 1) / L;
    t.first = t.a / L + t.n;
    if (back && !chains && t.count > 0) t.p = t.count - 1 - t.p;  // positions count in the direction of the scan
}

}  // namespace scan
}  // namespace kda

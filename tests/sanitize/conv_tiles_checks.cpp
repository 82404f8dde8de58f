// Which tiles of a packed convolution touch a prompt's history, walked as the
// kernel walks them, against the tiles whose arrival publishes the new head:
// every prompt start and length over a few tiles, every width and tile size.
// A tile that reads the head or the ring uncounted could do so after the head
// has moved.  Host code only; built with g++ by tests/test_conv_tiles.py.
#include <cstdio>
#include <cstdlib>
#include <set>

#include "mixer.h"

static long g_prompts = 0, g_fail = 0;

static void check(bool ok, const char *what, int W, int tile, int start, int end, int at) {
    if (ok) return;
    if (++g_fail <= 10)
        std::fprintf(stderr, "FAIL %s: W %d, tile %d, prompt %d..%d, tile number %d\n", what, W, tile, start, end, at);
}

int main() {
    for (int W = 2; W <= 4; ++W)
        for (int tile = 4; tile <= 32; tile *= 2)
            for (int start = 0; start < 2 * tile; ++start)
                for (int end = start + 1; end <= start + 4 * tile + 1; ++end) {
                    ++g_prompts;
                    const rssm::HistoryTiles counted(start, end, W, tile);
                    std::set<int> arrive;
                    for (int n = start / tile; n * tile < end; ++n) {
                        // the tile's first token of the prompt: its window of W - 1 inputs comes from the
                        // ring where it reaches back past the prompt's start
                        const int entry = n * tile > start ? n * tile : start;
                        bool touches = entry - (W - 1) < start;
                        // the last W - 1 inputs go into the ring
                        for (int t = entry; t < end && t < (n + 1) * tile; ++t) touches |= t >= end - (W - 1);
                        if (touches) check(counted.has(n), "not counted", W, tile, start, end, n);
                        if (counted.has(n)) arrive.insert(n);
                    }
                    check((int)arrive.size() == counted.count(), "arrivals", W, tile, start, end, counted.count());
                }
    std::printf("%ld prompts, %ld failed\n", g_prompts, g_fail);
    return g_fail != 0;
}

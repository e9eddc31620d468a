// Host simulation of an eviction's choice for one request and head: the search
// of the border key by the range arithmetic that the kernel uses, then the numbering.
// Reads any number of cases from stdin: log2 of the bins, n, budget, n_recent, n_sink, then n weights as bit patterns.
// Prints for each the passes taken and the kept slots, or "endless" if the passes do not end.
#include <cstdio>
#include <vector>

#include "../event_driven_persistent_b200/csrc/kv_shared.h"

using namespace et;

int main() {
    int log_bins, n, budget, recent, sink;
    while (scanf("%d %d %d %d %d", &log_bins, &n, &budget, &recent, &sink) == 5) {
        std::vector<uint32_t> key(n);
        for (auto& k : key) {
            uint32_t bits;
            if (scanf("%u", &bits) != 1) return 1;
            k = kv_weight_key(bits);
        }
        const int c0 = sink, c1 = n - recent;  // the slots that compete; the others have key 0
        uint32_t lo = 0xFFFFFFFFu, hi = 0, need = budget - recent - sink;
        for (int i = 0; i < n; ++i) {
            if (i < c0 || i >= c1) key[i] = 0;
            if (key[i] - 1 < lo) lo = key[i] - 1;
            if (key[i] > hi) hi = key[i];
        }
        ++lo;
        const bool none = need == 0;
        bool all_in = false, endless = false;
        int pass = 0;
        for (; need; ++pass) {
            if ((endless = pass == kv_border_passes(log_bins))) break;
            const uint32_t range = hi - lo;
            const int shift = kv_border_shift(range, log_bins);
            std::vector<uint32_t> bins((size_t)1 << log_bins);
            for (uint32_t k : key)
                if (k - lo <= range) {
                    if ((k - lo) >> shift >= bins.size()) return printf("bin %u of %zu\n", (k - lo) >> shift, bins.size()), 1;
                    ++bins[(k - lo) >> shift];
                }
            uint32_t above = 0;
            int bin = (int)bins.size() - 1;
            while (bin >= 0 && above + bins[bin] < need) above += bins[bin--];
            if (bin < 0) return printf("no border\n"), 1;
            need -= above;
            lo += (uint32_t)bin << shift;
            if (bins[bin] == need) {
                all_in = true;
                ++pass;
                break;
            }
            if (shift == 0) {
                ++pass;
                break;
            }
            hi = kv_border_end(lo, hi, shift);
        }
        if (endless) {
            printf("endless\n");
            continue;
        }
        printf("%d", pass);
        uint32_t ties = 0;
        for (int i = 0; i < n; ++i) {
            bool stays = i < c0 || i >= c1;
            if (!stays && !none) stays = key[i] > lo || (key[i] == lo && (all_in || ties++ < need));
            if (stays) printf(" %d", i);
        }
        printf("\n");
    }
    return 0;
}

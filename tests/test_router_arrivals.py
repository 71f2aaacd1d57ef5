"""How the router's workgroups find out which of them ends last (csrc/arrival.h), in every
order: one call's, whatever calls went before it, and after calls that overlapped."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gradient_aggregation_amd", "csrc")

PROGRAM = r"""
#include <algorithm>
#include <cstdio>
#include <utility>
#include <vector>
#include "arrival.h"

typedef std::vector<std::pair<int, unsigned>> Order;      // (call, workgroup), as they arrive

// Workgroups of calls of `sizes` in every order; f(order).
template <typename F>
void every(const std::vector<unsigned>& sizes, F f) {
    Order o;
    for (int c = 0; c < (int)sizes.size(); ++c)
        for (unsigned i = 0; i < sizes[c]; ++i) o.push_back({c, i});
    do f(o); while (std::next_permutation(o.begin(), o.end()));
}

// The arrivals that are taken for the last ones.
template <bool RESET>
int ends(const Order& o, const std::vector<unsigned>& sizes, uint32_t& count, bool& at_end) {
    int found = 0;
    for (size_t j = 0; j < o.size(); ++j) {
        const unsigned n = sizes[o[j].first];
        bool last;
        if (RESET) {           // counting to n, and then back to 0
            last = ++count == n;
            if (last) count = 0;
        } else {
            count += ga::arrival(o[j].second, n);
            last = count == 0;
        }
        found += last;
        at_end = last && j + 1 == o.size();
    }
    return found;
}

int main() {
    long orders = 0, spoilt = 0;
    for (unsigned a = 1; a <= 4; ++a)
        for (unsigned b = 1; b <= 4; ++b)
            every({a, b}, [&](const Order& o) {
                uint32_t count = 0, other = 0;
                bool at_end;
                ends<false>(o, {a, b}, count, at_end);
                if (count != 0) std::printf("%u and %u workgroups leave %u\n", a, b, count);
                ends<true>(o, {a, b}, other, at_end);
                spoilt += other != 0;
                ++orders;
            });
    for (unsigned n = 1; n <= 7; ++n)
        every({n}, [&](const Order& o) {
            uint32_t count = 0;
            bool at_end = false;
            if (ends<false>(o, {n}, count, at_end) != 1 || !at_end || count != 0) std::printf("%u workgroups: not the last one\n", n);
            ++orders;
        });
    for (uint32_t n = 1; n < 100000; n = n * 3 + 1) {
        uint32_t sum = 0;
        for (uint32_t i = 0; i < n; ++i) sum += ga::arrival(i, n);
        if (sum != 0) std::printf("%u workgroups add up to %u\n", n, sum);
    }
    std::printf("%ld orders, %ld spoilt by a count that is reset\n", orders, spoilt);
}
"""


def test_every_order_of_arrivals(tmp_path):
    src = tmp_path / "arrivals.cpp"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I" + CSRC, str(src), "-o", str(tmp_path / "arrivals")], check=True)
    out = subprocess.run([str(tmp_path / "arrivals")], check=True, capture_output=True, text=True).stdout.split("\n")
    assert len(out) == 2, out                  # no fault among them
    orders, spoilt = (int(w) for w in out[0].split() if w.isdigit())
    assert orders > 50000 and spoilt > 0      # the count that is reset is what this tells apart

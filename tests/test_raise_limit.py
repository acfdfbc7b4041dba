"""The limit that threads raise together (a kernel's dynamic shared memory, with a fake of the call that sets it)."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int4_block_quantized_matmulnbits_b200",
                    "csrc")

# Thread A asks for 200 and has set it when thread B, which asks for 100, starts; A notes it only when B is done, or
# when B has had half a second: unguarded, B sets 100 behind A's 200, and A's note says 200.
PROGRAM = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <initializer_list>
#include <thread>
#include "raise_limit.h"

int main() {
    int known = 0;
    std::atomic<int> limit{0}, a_set{0}, b_done{0};
    auto ask = [&](int want, bool first) {
        return mnb::raise_limit(&known, want, [&](int n) {
            limit = n;
            if (first) {
                a_set = 1;
                for (int i = 0; i < 500 && !b_done; i++)
                    std::this_thread::sleep_for(std::chrono::milliseconds(1));
            }
            return 0;
        });
    };
    std::thread a([&] { ask(200, true); });
    std::thread b([&] {
        while (!a_set)
            std::this_thread::yield();
        ask(100, false);
        b_done = 1;
    });
    a.join(), b.join();
    std::printf("%d %d\n", (int)limit, known);
    // an error is no raise: the next one tries again
    const int failed = mnb::raise_limit(&known, 300, [](int) { return 7; });
    int calls = 0;
    for (int want : {300, 300, 250, 301})
        mnb::raise_limit(&known, want, [&](int n) { limit = n; calls++; return 0; });
    std::printf("%d %d %d %d\n", failed, (int)limit, known, calls);
    return 0;
}
"""


def test_threads_do_not_lower_one_anothers_limit(tmp_path):
    src = tmp_path / "r.cpp"
    src.write_text(PROGRAM)
    subprocess.check_call(["g++", "-std=c++17", "-pthread", "-I", CSRC, str(src), "-o", str(tmp_path / "r")])
    out = subprocess.check_output([str(tmp_path / "r")], timeout=60, text=True).split("\n")
    assert out[0] == "200 200"
    assert out[1] == "7 301 301 2"

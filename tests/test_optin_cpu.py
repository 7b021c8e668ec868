"""The shared-memory limits that launches raise, under two host threads: the
limit in force is never below the one noted, and never falls."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
#include "moe_optin.h"

int main() {
    std::atomic<size_t> limit{0};
    int bad = 0;
    for (int round = 0; round < 20; ++round) {
        moe::OptIn optin;
        limit = 0;
        // each attribute call takes a while before (the small one) or after (the large one) it acts
        auto small = [&](size_t n) { std::this_thread::sleep_for(std::chrono::milliseconds(4)); limit = n; return 0; };
        auto large = [&](size_t n) { limit = n; std::this_thread::sleep_for(std::chrono::milliseconds(8)); return 0; };
        std::thread a([&] { optin.raise(7, 50, small); });
        std::thread b([&] { std::this_thread::sleep_for(std::chrono::milliseconds(1)); optin.raise(7, 130, large); });
        a.join();
        b.join();
        optin.raise(7, 130, large);  // a launch that needs 130: the limit must reach it
        bad += limit < 130;
        optin.raise(7, 60, small);  // a smaller one changes nothing
        bad += limit < 130;
        if (optin.raise(8, 10, [&](size_t) { return 5; }) != 5) ++bad;  // a failure is handed on
        bool again = false;
        optin.raise(8, 10, [&](size_t) { again = true; return 0; });  // and not noted as done
        bad += !again;
    }
    std::printf("%d\n", bad);
    return bad != 0;
}
"""


def test_two_threads_raise_one_limit(tmp_path):
    src, exe = tmp_path / "optin.cpp", tmp_path / "optin"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I",
                    os.path.join(ROOT, "expert_ffn_router_b200", "csrc"), str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout

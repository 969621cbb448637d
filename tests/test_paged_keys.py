"""The bounds arithmetic of the attention kernels (csrc/keys.hpp), built for
the host with undefined behaviour trapped: for every window that the call
accepts and positions at the ends of their range, the same keys as 64-bit
arithmetic gives, and no sum that leaves 32 bits."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_kv_cache_sz_amd", "csrc")

PROGRAM = r"""
#include "keys.hpp"
#include <cstdio>
#include <initializer_list>

int main()
{
    const int64_t top = sz::kMaxTokens;
    const int64_t sizes[] = {0, 1, 2, 3, 5, 10, 63, 64, 65, 1000, top / 2, top - 2, top - 1, top};
    const int64_t windows[] = {0, 1, 2, 3, 16, 64, 1000, top / 2, top - 2, top - 1, top, top + 1, top + 64,
                               2 * top - 64, 2 * top - 4, 2 * top - 3, 2 * top - 2, 2 * top - 1};
    int checked = 0;
    for (int64_t len : sizes)
        for (int64_t n : sizes)
            for (int64_t w : windows)
                for (int64_t i : {(int64_t)0, n / 2, n - 1}) {
                    if (i < 0 || i >= n) continue;
                    const int64_t p = len - n + i, from = w > 0 && p - w + 1 > 0 ? p - w + 1 : 0;
                    const int64_t got = sz::first_seen((int32_t)p, sz::window_keys((uint32_t)w));
                    if (got != from) {
                        printf("len %lld new %lld token %lld window %lld: first key %lld, not %lld\n", (long long)len,
                               (long long)n, (long long)i, (long long)w, (long long)got, (long long)from);
                        return 1;
                    }
                    ++checked;
                }
    printf("checked %d\n", checked);
    return 0;
}
"""


def test_first_keys_over_the_whole_range(tmp_path):
    source, program = tmp_path / "keys.cpp", tmp_path / "keys"
    source.write_text(PROGRAM)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", CSRC,
                           str(source), "-o", str(program)])
    run = subprocess.run([str(program)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout + run.stderr
    assert run.stdout.startswith("checked ")



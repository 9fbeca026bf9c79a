"""Host arithmetic of the microscaled formats' launches at the ends of its range (CPU): the
library's header is compiled with static assertions, where an overflow is an error."""
import os
import subprocess

from sharded_mixed_precision_shard_amd import _build

SOURCE = r"""
#include "zs_mx.h"
using namespace zs_detail;
// a tile's 256 rows below 2^31 bytes apart in all
static_assert(mx_rows_reach(0, 256) && mx_rows_reach((1 << 22) - 1, 256), "");
static_assert(!mx_rows_reach(1 << 22, 256), "");
// a single row's distance to the next is any number that the argument checks let through
constexpr bool none() {
    for (int e = 22; e < 60; ++e)
        if (mx_rows_reach(int64_t(1) << e, 256) || mx_rows_reach((int64_t(1) << e) + 8, 256) ||
            mx_rows_reach((int64_t(1) << e) + (int64_t(1) << (e - 1)), 256))
            return false;
    return true;
}
static_assert(none(), "");
"""


def test_distances_of_rows_do_not_overflow(tmp_path):
    src = tmp_path / "reach.cpp"
    src.write_text(SOURCE)
    subprocess.run([_build.hipcc(), "-x", "hip", "--offload-arch=" + _build.ARCH,
                    "--offload-host-only", "-std=c++17", "-fsyntax-only",
                    "-I", os.path.join(_build.PKG_DIR, "csrc"), "-I", _build.INCLUDE_DIR,
                    str(src)], check=True, capture_output=True, text=True)

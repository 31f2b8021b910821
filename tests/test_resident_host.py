"""The launchers' memory of how many clusters run at once (no GPU needed), compiled from its source:
one count for each device, asked for until it is known, from any thread."""
import subprocess

PROGRAM = r"""
#include <cassert>
#include <cstdio>
#include <thread>
#include <vector>
#include "%s/resident.h"
int main()
{
    lnq::ResidentClusters r;
    int asked = 0;
    auto query = [&](int n) { return [&asked, n]() { ++asked; return n; }; };
    assert(r.get(0, 5, query(0)) == 5 && asked == 1);      // a failed query is not kept
    assert(r.get(0, 5, query(74)) == 74 && asked == 2);
    assert(r.get(0, 5, query(1)) == 74 && asked == 2);
    assert(r.get(1, 5, query(70)) == 70 && asked == 3);    // another device has its own
    assert(r.get(0, 5, query(1)) == 74 && r.get(1, 5, query(1)) == 70 && asked == 3);
    assert(r.get(-1, 5, query(9)) == 9 && r.get(1 << 20, 5, query(8)) == 8 && asked == 5);
    assert(r.get(-1, 5, query(7)) == 7);                   // no place to keep it
    lnq::ResidentClusters many;
    std::vector<std::thread> ts;
    for (int k = 0; k < 8; ++k)
        ts.emplace_back([&many]() {
            for (int i = 0; i < 64 * 1000; ++i)
                assert(many.get(i %% 64, 1, [i]() { return 100 + i %% 64; }) == 100 + i %% 64);
        });
    for (auto &t : ts)
        t.join();
    std::puts("ok");
}
"""


def test_counts_are_kept_per_device(tmp_path):
    from post_weight_quantization_guided_b200 import build
    src = tmp_path / "resident.cpp"
    src.write_text(PROGRAM % build.CSRC)
    exe = tmp_path / "resident"
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-pthread", str(src), "-o", str(exe)])
    assert subprocess.check_output([str(exe)], text=True) == "ok\n"


def test_no_launcher_keeps_a_plain_static():
    """Host state that outlives a call is atomic or guarded: no plain static number."""
    import glob
    import re
    from post_weight_quantization_guided_b200 import build
    for path in sorted(glob.glob(build.CSRC + "/*.cu")):
        found = re.findall(r"^\s+static (?:int|long|bool|unsigned|uint32_t|int64_t) \w+(?:\[\w+\])?\s*(?:=|;)",
                           open(path).read(), re.M)
        assert not found, (path, found)

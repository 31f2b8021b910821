"""The host's part of lnq_fp4_check (no GPU needed), compiled from its source with a stand-in for the
device: slots of streams, and what each stream has been told of."""
import os
import subprocess

from conftest import ROOT

PROGRAM = r"""
#include <assert.h>
#include <stdio.h>
#include <set>
#include <thread>
#include <vector>
#include "%(csrc)s/fp4_report.cu"
using namespace lnq;
static cudaStream_t handle(uintptr_t k) { return reinterpret_cast<cudaStream_t>(k); }
int main()
{
    // the default stream under both its names; as many others as there are slots, each its own, for
    // two threads that ask at once
    assert(fp4_report_slot(nullptr) == 0 && fp4_report_slot(cudaStreamLegacy) == 0);
    std::vector<int> a(kFp4ReportSlots - 1), b(a);
    auto ask = [](std::vector<int> &v) {
        for (size_t k = 0; k < v.size(); ++k)
            v[k] = fp4_report_slot(handle(0x500000 + 64 * k));
    };
    std::thread t1(ask, std::ref(a)), t2(ask, std::ref(b));
    t1.join(), t2.join();
    assert(a == b);
    std::set<int> distinct(a.begin(), a.end());
    assert(distinct.size() == a.size() && *distinct.begin() == 1 && *distinct.rbegin() == kFp4ReportSlots - 1);
    // one more shares a slot, always the same one
    const int shared = fp4_report_slot(handle(0x900000));
    assert(shared >= 1 && shared < kFp4ReportSlots && shared == fp4_report_slot(handle(0x900000)));

    cudaStream_t s = handle(0x500000), u = handle(0x500040);
    assert(!fp4_report_news(0, s, Fp4GiveUps{0, 0, 5}));   // others' give-ups
    assert(fp4_report_news(0, s, Fp4GiveUps{2, 0, 7}));    // its own, once
    assert(!fp4_report_news(0, s, Fp4GiveUps{2, 0, 9}));
    assert(fp4_report_news(0, nullptr, Fp4GiveUps{0, 0, 9}));   // the device's
    assert(!fp4_report_news(0, cudaStreamLegacy, Fp4GiveUps{0, 0, 9}));
    assert(fp4_report_news(1, nullptr, Fp4GiveUps{0, 0, 1}));   // of each device
    assert(fp4_report_news(0, u, Fp4GiveUps{0, 1, 10}) && fp4_report_news(0, s, Fp4GiveUps{2, 1, 10}));
    assert(!fp4_report_news(0, u, Fp4GiveUps{0, 1, 10}) && !fp4_report_news(0, s, Fp4GiveUps{2, 1, 10}));
    assert(!fp4_report_news(0, s, Fp4GiveUps{1, 0, 8}));   // read before, told after: nothing new
    assert(fp4_report_news(0, s, Fp4GiveUps{3, 1, 11}));
    // counts run over
    assert(fp4_report_news(0, handle(0x500080), Fp4GiveUps{0x7FFFFFFFu, 0, 0}));
    assert(fp4_report_news(0, handle(0x500080), Fp4GiveUps{0xFFFFFFF0u, 0, 0}));
    assert(fp4_report_news(0, handle(0x500080), Fp4GiveUps{3u, 0, 0}));
    // the per-thread default stream: one for each thread
    assert(fp4_report_news(0, cudaStreamPerThread, Fp4GiveUps{1, 0, 0}));
    std::thread([] { assert(fp4_report_news(0, cudaStreamPerThread, Fp4GiveUps{1, 0, 0})); }).join();
    assert(!fp4_report_news(0, cudaStreamPerThread, Fp4GiveUps{1, 0, 0}));
    puts("ok");
}
"""


def test_slots_and_reports(tmp_path):
    from post_weight_quantization_guided_b200 import build
    src = tmp_path / "report.cu"
    src.write_text(PROGRAM % {"csrc": build.CSRC})
    exe = tmp_path / "report"
    subprocess.check_call([build.NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17",
                           "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    assert subprocess.check_output([str(exe)], text=True) == "ok\n"

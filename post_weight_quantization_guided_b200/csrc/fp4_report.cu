// fp4_report.cu -- which give-ups of the 4-bit products a stream has been told of (lnq_fp4_check).
//
// The device only ever adds to its counts, so nothing is erased while somebody else reads. What a
// stream has been told of is kept here, and only where a count is not zero: in a process whose waits
// never give up the table stays empty.
#include <atomic>
#include <mutex>

#include "fp4.cuh"

namespace lnq {
namespace {

struct Told {
    int device;
    uintptr_t stream;
    Fp4GiveUps counts;
};
constexpr int kMaxTold = 4096;
std::mutex g_mu;
Told g_told[kMaxTold];
int g_num_told = 0;

// The default stream's two names are one, and the per-thread default stream is one for each thread.
uintptr_t stream_key(cudaStream_t s)
{
    static thread_local char mine;
    if (s == cudaStreamPerThread)
        return reinterpret_cast<uintptr_t>(&mine);
    return s == cudaStreamLegacy ? 0 : reinterpret_cast<uintptr_t>(s);
}

bool newer(uint32_t now, uint32_t told) { return static_cast<int32_t>(now - told) > 0; }

}  // namespace

// Slot 0 is the default stream's. Another stream's is the first free one from a place that its handle
// gives, for good; when none is free, that place, which it then shares.
int fp4_report_slot(cudaStream_t s)
{
    static std::atomic<uintptr_t> owner[kFp4ReportSlots];
    const uintptr_t key = stream_key(s);
    if (key == 0)
        return 0;
    const int home = 1 + static_cast<int>((static_cast<uint64_t>(key) * 0x9E3779B97F4A7C15ull >> 32) %
                                          (kFp4ReportSlots - 1));
    for (int k = 0, at = home; k < kFp4ReportSlots - 1; ++k) {
        uintptr_t free = 0;
        if (owner[at].load(std::memory_order_relaxed) == key ||
            owner[at].compare_exchange_strong(free, key, std::memory_order_relaxed) || free == key)
            return at;
        at = at + 1 == kFp4ReportSlots ? 1 : at + 1;
    }
    return home;
}

bool fp4_report_news(int device, cudaStream_t s, const Fp4GiveUps &now)
{
    const uintptr_t key = stream_key(s);
    std::lock_guard<std::mutex> lk(g_mu);
    Told *t = nullptr;
    for (int k = 0; k < g_num_told && t == nullptr; ++k)
        if (g_told[k].device == device && g_told[k].stream == key)
            t = &g_told[k];
    const Fp4GiveUps told = t != nullptr ? t->counts : Fp4GiveUps{0u, 0u, 0u};
    const bool news = key == 0 ? newer(now.all, told.all)
                               : newer(now.own, told.own) || newer(now.captured, told.captured);
    if (!news)
        return false;
    if (t == nullptr && g_num_told < kMaxTold) {  // a full table: told again, never too little
        t = &g_told[g_num_told++];
        t->device = device;
        t->stream = key;
    }
    if (t != nullptr)
        t->counts = now;
    return true;
}

}  // namespace lnq

// launch_order.h -- host-side bookkeeping of programmatic dependent launch
// for the decode kernel family (host code only, no CUDA dependency).
//
// Decode-family launches with host positions (decode steps, short chunks)
// signal their dependents at kernel start, and every one of their thread
// blocks waits for the previous kernel on the stream before it exits, so a
// launch that has finished implies that its predecessor has.  When launch X
// starts, the launches that may still run are N, N-1, ..., N-k (N the one just
// before X) such that all thread blocks of N-k+1..N were resident together
// with one of N-k: none of them can have exited while N-k runs, and X starts
// only once every block of N has started.  The walk back from N therefore
// stops where the blocks counted so far plus one would exceed what the device
// holds at once, at a launch that signals only after its own wait (nothing
// before it still runs), or at a barrier: a kernel that never signals early
// (the prefill kernels, reset) or a synchronisation of the stream, after which
// nothing enqueued earlier still runs when the next launch starts.
//
// X must load only after its own wait the cache rows that those launches
// append to X's layer: at most the sum of their new tokens per sequence, just
// below X's first new slot (positions only grow between barriers).
#pragma once

#include <algorithm>
#include <atomic>
#include <cstddef>
#include <cstdint>
#include <deque>
#include <iterator>
#include <mutex>
#include <unordered_map>

namespace qa {

// A stream by what its handle stands for.  The legacy default stream (NULL, or
// the handle 1) and the per-thread one (2) have the same handle on every device,
// and the latter in every thread, but each device, and each thread, has its own.
// `capture`: the id of the capture that the stream's launches go into (0: they
// run).  Captured launches are ordered among themselves (a graph's first kernels
// start after everything before its replay).  They do not end what the stream
// still runs: a walk of its own launches passes over them, counting the rows
// that they append as if they had run.
struct StreamRef {
    uintptr_t handle;
    uint64_t thread = 0;  // of the per-thread stream
    uint64_t capture;
    int device;

    StreamRef(const void *stream, int device_ = 0, uint64_t capture_ = 0)
        : handle(reinterpret_cast<uintptr_t>(stream)), capture(capture_), device(device_) {
        if (handle == 1) handle = 0;
        if (handle == 2) thread = this_thread();
    }
    bool operator==(const StreamRef &o) const {  // the same stream
        return handle == o.handle && thread == o.thread && device == o.device;
    }
    struct Hash {
        size_t operator()(const StreamRef &r) const {
            return std::hash<uint64_t>()(r.handle ^ (r.thread << 40) ^ (static_cast<uint64_t>(r.device) << 56));
        }
    };

  private:
    static uint64_t this_thread() {  // ids are not used again, unlike the system's
        static std::atomic<uint64_t> threads{0};
        thread_local const uint64_t id = ++threads;
        return id;
    }
};

class LaunchOrder {
  public:
    // Guard value meaning "every cache row may still be written".
    static constexpr int kGuardAll = 1 << 30;

    // Records a launch of `ctas` thread blocks on `stream` that appends up to
    // `tmax` tokens per sequence to (cache, layer), and returns its guard: the
    // number of rows below its first new slot that launches possibly still
    // running append to the same (cache, layer).  early: the launch signals its
    // dependents before waiting for its predecessor.  resident_max: the most
    // thread blocks of this family the device holds at once.
    int admit(const StreamRef &stream, const void *cache, int layer, int ctas, int tmax, bool early,
              int64_t resident_max) {
        std::lock_guard<std::mutex> lock(mu_);
        Hist &h = hist(stream);
        int64_t guard = 0, resident = 0;
        bool bounded = false;
        for (auto it = h.recs.rbegin(); it != h.recs.rend(); ++it) {
            if (it->cache == cache && it->layer == layer) guard += it->tmax;
            if (it->passed) continue;
            if (!it->early) {  // it waited before signalling: nothing before it still runs
                bounded = true;
                break;
            }
            resident += it->ctas;  // all of its blocks resident while anything before it runs
            if (resident + 1 > resident_max) {
                bounded = true;
                break;
            }
        }
        if (!bounded && h.truncated) guard = kGuardAll;  // the older launches are not known
        h.add({cache, layer, std::max(ctas, 1), tmax, early, false});
        if (stream.capture != 0) streams_[0][stream].add({cache, layer, 0, tmax, true, true});
        return static_cast<int>(std::min<int64_t>(guard, kGuardAll));
    }

    // True when no launch that may still run when the next launch on `stream`
    // starts appends to (cache, layer): the same walk as admit, nothing recorded.
    // A launch for which this holds may read that layer's device lengths
    // before its own wait.
    bool layer_settled(const StreamRef &stream, const void *cache, int layer, int64_t resident_max) {
        std::lock_guard<std::mutex> lock(mu_);
        const Hist *found = find(stream);
        if (!found) return true;
        const Hist &h = *found;
        int64_t resident = 0;
        for (auto it = h.recs.rbegin(); it != h.recs.rend(); ++it) {
            if (it->cache == cache && it->layer == layer) return false;
            if (it->passed) continue;
            if (!it->early) return true;
            resident += it->ctas;
            if (resident + 1 > resident_max) return true;
        }
        return !h.truncated;
    }

    // What the next launch on `stream` may run beside: 0 nothing (no launch
    // recorded since the last barrier), 1 launches of other layers only, 2 a
    // launch that appends to (cache, layer).
    int in_flight(const StreamRef &stream, const void *cache, int layer, int64_t resident_max) {
        {
            std::lock_guard<std::mutex> lock(mu_);
            const Hist *found = find(stream);
            if (!found || found->recs.empty()) return 0;
        }
        return layer_settled(stream, cache, layer, resident_max) ? 1 : 2;
    }

    // A kernel that never signals early was enqueued on `stream`, or the
    // stream was synchronised.
    void barrier(const StreamRef &stream) {
        std::lock_guard<std::mutex> lock(mu_);
        if (find(stream)) streams_[stream.capture != 0].erase(stream);
    }

    // The device was synchronised (kAllDevices: all of them).
    static constexpr int kAllDevices = -1;
    void clear(int device = kAllDevices) {
        std::lock_guard<std::mutex> lock(mu_);
        auto &run = streams_[0];  // (a synchronisation cannot be part of a capture)
        for (auto it = run.begin(); it != run.end();)
            it = device == kAllDevices || it->first.device == device ? run.erase(it) : std::next(it);
    }

    // Launches kept per stream; the walk needs at most resident_max of them.
    static constexpr size_t kCap = size_t(1) << 14;

  private:
    struct Rec {
        const void *cache;
        int layer, ctas, tmax;
        bool early;
        bool passed;  // captured, in the record of what the stream runs
    };
    struct Hist {
        std::deque<Rec> recs;
        bool truncated = false;
        uint64_t capture = 0;
        void add(const Rec &r) {
            recs.push_back(r);
            if (recs.size() > kCap) {
                recs.pop_front();
                truncated = true;
            }
        }
    };
    const Hist *find(const StreamRef &stream) const {
        const auto &map = streams_[stream.capture != 0];
        const auto found = map.find(stream);
        return found == map.end() || found->second.capture != stream.capture ? nullptr : &found->second;
    }
    Hist &hist(const StreamRef &stream) {
        Hist &h = streams_[stream.capture != 0][stream];
        if (h.capture != stream.capture) h = Hist{};  // of an earlier capture
        h.capture = stream.capture;
        return h;
    }
    std::mutex mu_;
    // What each stream runs, and what goes into its capture.
    std::unordered_map<StreamRef, Hist, StreamRef::Hash> streams_[2];
};

}  // namespace qa

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
//
// That is the order of a stream that runs.  In a capture the graph's edges take its
// place, and X may follow a launch of another stream, whose event its own has waited
// for: such an edge is programmatic too, so X may start beside that launch and what
// that one ran beside.  Where X follows a node of this library that is not its stream's
// last one, nothing is known to have finished: the stream's record begins anew, as
// one whose older launches are not known.
#pragma once

#include <algorithm>
#include <atomic>
#include <cstddef>
#include <cstdint>
#include <deque>
#include <iterator>
#include <mutex>
#include <unordered_map>
#include <unordered_set>
#include <vector>

namespace qa {

// Whether steps overlap earlier kernels of their stream (qa_set_early_reads).
bool early_reads();

// A stream by what its handle stands for.  The legacy default stream (NULL, or
// the handle 1) and the per-thread one (2) have the same handle on every device,
// and the latter in every thread, but each device, and each thread, has its own.
// `capture`: the id of the capture that the stream's launches go into (0: they
// run).  Captured launches are ordered among themselves (a graph's first kernels
// start after everything before its replay).  They do not end what the stream
// still runs: a walk of its own launches passes over them, counting the rows
// that they append as if they had run.
// `after`: in a capture, the graph's nodes that the next launch follows.
struct StreamRef {
    uintptr_t handle;
    uint64_t thread = 0;  // of the per-thread stream
    uint64_t capture;
    int device;
    std::vector<uintptr_t> after;

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
        const bool stray = strays(stream);
        Hist &h = hist(stream);
        if (stray) {
            h.recs.clear();
            h.truncated = true;
        }
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
        h.add({cache, layer, std::max(ctas, 1), tmax, early, false, next_++});
        if (stream.capture != 0) streams_[0][stream].add({cache, layer, 0, tmax, true, true, next_++});
        return static_cast<int>(std::min<int64_t>(guard, kGuardAll));
    }

    // True when no launch that may still run when the next launch on `stream`
    // starts appends to (cache, layer): the same walk as admit, nothing recorded.
    // A launch for which this holds may read that layer's device lengths
    // before its own wait.
    bool layer_settled(const StreamRef &stream, const void *cache, int layer, int64_t resident_max) {
        std::lock_guard<std::mutex> lock(mu_);
        if (strays(stream)) return false;
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
            if (!strays(stream) && (!found || found->recs.empty())) return 0;
        }
        return layer_settled(stream, cache, layer, resident_max) ? 1 : 2;
    }

    // A kernel that never signals early was enqueued on `stream`, or the
    // stream was synchronised.
    void barrier(const StreamRef &stream) {
        std::lock_guard<std::mutex> lock(mu_);
        if (!find(stream)) return;
        if (stream.capture == 0) {
            streams_[0].erase(stream);
            return;
        }
        Hist &h = hist(stream);  // (another stream may yet follow its nodes)
        h.recs.clear();
        h.truncated = false;
    }

    // An admitted launch has become the node that `stream` now follows.
    void captured(const StreamRef &stream) {
        std::lock_guard<std::mutex> lock(mu_);
        if (stream.capture == 0 || stream.after.size() != 1) return;
        Hist &h = hist(stream);
        h.last = stream.after[0];
        h.nodes.insert(h.last);
    }

    // A call that admits launches before it makes them: its records, until it is over, are
    // of launches that a synchronisation may not have seen.
    class Call {
      public:
        explicit Call(LaunchOrder &order) : order_(order) {
            std::lock_guard<std::mutex> lock(order_.mu_);
            first_ = order_.next_++;
            order_.calls_.push_back(first_);
        }
        ~Call() {
            std::lock_guard<std::mutex> lock(order_.mu_);
            order_.calls_.erase(std::find(order_.calls_.begin(), order_.calls_.end(), first_));
        }
        Call(const Call &) = delete;

      private:
        LaunchOrder &order_;
        uint64_t first_;
    };

    // Every launch recorded before the one of this number has been enqueued.
    uint64_t mark() {
        std::lock_guard<std::mutex> lock(mu_);
        return calls_.empty() ? next_ : *std::min_element(calls_.begin(), calls_.end());
    }

    // The calling thread has synchronised the device (kAllDevices: all of them): what it
    // had launched there has finished, and what any thread had enqueued at a mark() before.
    // Other records of other threads stay: they may have launched since, or be about to
    // launch.  Without the finished ones a walk goes further back, never less far.
    static constexpr int kAllDevices = -1;
    void clear(int device = kAllDevices, uint64_t mark = 0) {
        const uint64_t me = StreamRef::this_thread();
        std::lock_guard<std::mutex> lock(mu_);
        auto &run = streams_[0];  // (a synchronisation cannot be part of a capture)
        for (auto it = run.begin(); it != run.end();) {
            Hist &h = it->second;
            if (device != kAllDevices && it->first.device != device) {
                ++it;
                continue;
            }
            const bool mine = !h.shared && !h.recs.empty() && h.recs.front().thread == me;
            h.recs.erase(std::remove_if(h.recs.begin(), h.recs.end(), [&](const Rec &r) { return r.thread == me || r.number < mark; }),
                         h.recs.end());
            if (mine || h.lost < mark) h.truncated = false;
            it = h.recs.empty() && !h.truncated ? run.erase(it) : std::next(it);
        }
    }

    // Launches kept per stream; the walk needs at most resident_max of them.
    static constexpr size_t kCap = size_t(1) << 14;

  private:
    struct Rec {
        const void *cache;
        int layer, ctas, tmax;
        bool early;
        bool passed;  // captured, in the record of what the stream runs
        uint64_t number;
        uint64_t thread = StreamRef::this_thread();  // that launches it
    };
    struct Hist {
        std::deque<Rec> recs;
        bool truncated = false;
        uint64_t lost = 0;    // the last record that went
        bool shared = false;  // several threads' launches
        uint64_t capture = 0;
        uintptr_t last = 0;                   // in a capture: the node of its last admitted launch
        std::unordered_set<uintptr_t> nodes;  // and of all of them
        void add(const Rec &r) {
            shared = shared || (!recs.empty() && recs.back().thread != r.thread);
            recs.push_back(r);
            if (recs.size() > kCap) {
                lost = recs.front().number;
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
    // Whether the next launch follows an admitted one other than its stream's last.
    bool strays(const StreamRef &stream) const {
        if (stream.capture == 0) return false;
        const Hist *own = find(stream);
        for (const uintptr_t node : stream.after) {
            if (own && own->last == node) continue;
            for (const auto &h : streams_[1])
                if (h.second.capture == stream.capture && h.second.nodes.count(node)) return true;
        }
        return false;
    }
    Hist &hist(const StreamRef &stream) {
        Hist &h = streams_[stream.capture != 0][stream];
        if (h.capture != stream.capture) h = Hist{};  // of an earlier capture
        h.capture = stream.capture;
        return h;
    }
    std::mutex mu_;
    uint64_t next_ = 1;            // the number of the next record
    std::vector<uint64_t> calls_;  // under way: numbers below all of their records'
    // What each stream runs, and what goes into its capture.
    std::unordered_map<StreamRef, Hist, StreamRef::Hash> streams_[2];
};

}  // namespace qa

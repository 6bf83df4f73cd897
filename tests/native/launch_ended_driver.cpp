// What qa::LaunchOrder keeps of threads that have ended, one command per input line; cache
// 7, layer 0, 10 thread blocks a launch, 304 resident at most.
//   threads <n> <handle>   n threads, one after the other, launch on the stream once each and end
//   calls <n> <handle>     the same, but each is still in its call: it has recorded its launch
//                          and not made it (they wait for `go`)
//   go                     those calls are over, and the threads
//   launch <handle>        this thread launches
//   mark
//   clear                  this thread has synchronised, after the mark
//   settled                -> on how many of all those threads' streams the layer is settled
//   stream <handle>        -> 0 | 1: whether it is on this thread's
#include <condition_variable>
#include <iostream>
#include <list>
#include <memory>
#include <mutex>
#include <sstream>
#include <string>
#include <thread>
#include <vector>

#include "launch_order.h"

int main() {
    qa::LaunchOrder order;
    const void *cache = reinterpret_cast<const void *>(7);
    std::vector<qa::StreamRef> refs;
    std::vector<std::thread> waiting;
    std::mutex mu;
    std::condition_variable cv;
    int in_call = 0;
    bool go = false;
    uint64_t mark = 0;
    std::string line;
    auto admit = [&](const qa::StreamRef &at) { order.admit(at, cache, 0, 10, 1, true, 304); };
    while (std::getline(std::cin, line)) {
        std::istringstream in(line);
        std::string cmd;
        int n = 0;
        uintptr_t handle = 0;
        in >> cmd;
        if (cmd == "threads" || cmd == "calls") in >> n;
        in >> handle;
        const void *stream = reinterpret_cast<const void *>(handle);
        if (cmd == "threads") {
            for (int i = 0; i < n; ++i)
                std::thread([&] {
                    refs.emplace_back(stream);
                    admit(refs.back());
                }).join();
        } else if (cmd == "calls") {
            for (int i = 0; i < n; ++i) {
                std::unique_lock<std::mutex> lock(mu);
                waiting.emplace_back([&, stream] {
                    std::unique_lock<std::mutex> inner(mu);
                    const qa::LaunchOrder::Call call(order);
                    refs.emplace_back(stream);
                    admit(refs.back());
                    ++in_call;
                    cv.notify_all();
                    cv.wait(inner, [&] { return go; });
                });
                cv.wait(lock, [&] { return in_call == static_cast<int>(waiting.size()); });
            }
        } else if (cmd == "go") {
            {
                std::lock_guard<std::mutex> lock(mu);
                go = true;
            }
            cv.notify_all();
            for (std::thread &t : waiting) t.join();
            waiting.clear();
            in_call = 0;
            go = false;
        } else if (cmd == "launch") {
            admit(qa::StreamRef(stream));
        } else if (cmd == "mark") {
            mark = order.mark();
        } else if (cmd == "clear") {
            order.clear(qa::LaunchOrder::kAllDevices, mark);
        } else if (cmd == "settled") {
            int k = 0;
            for (const qa::StreamRef &at : refs) k += order.layer_settled(at, cache, 0, 304);
            std::cout << k << "\n";
        } else if (cmd == "stream") {
            std::cout << order.layer_settled(qa::StreamRef(stream), cache, 0, 304) << "\n";
        }
    }
    return 0;
}

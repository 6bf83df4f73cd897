// Two threads' records in qa::LaunchOrder, one command per input line:
//   admit <thread 0|1> <stream> <layer> <early 0|1>   -> guard
//   clear <thread 0|1>                                (that thread has synchronised)
//   settled <stream> <layer>                          -> 0 | 1
#include <condition_variable>
#include <functional>
#include <iostream>
#include <mutex>
#include <sstream>
#include <string>
#include <thread>

#include "launch_order.h"

// A thread that runs what it is given, one thing at a time.
struct Worker {
    std::mutex mu;
    std::condition_variable cv;
    std::function<void()> job;
    bool stop = false;
    std::thread th{[this] {
        std::unique_lock<std::mutex> lock(mu);
        for (;;) {
            cv.wait(lock, [&] { return job || stop; });
            if (!job) return;
            job();
            job = nullptr;
            cv.notify_all();
        }
    }};
    void run(std::function<void()> f) {
        std::unique_lock<std::mutex> lock(mu);
        job = std::move(f);
        cv.notify_all();
        cv.wait(lock, [&] { return !job; });
    }
    ~Worker() {
        {
            std::lock_guard<std::mutex> lock(mu);
            stop = true;
        }
        cv.notify_all();
        th.join();
    }
};

int main() {
    qa::LaunchOrder order;
    Worker workers[2];
    const void *cache = &order;
    std::string line;
    while (std::getline(std::cin, line)) {
        std::istringstream in(line);
        std::string cmd;
        int thread = 0, layer = 0, early = 1;
        uintptr_t stream = 0;
        in >> cmd;
        if (cmd == "admit") {
            in >> thread >> stream >> layer >> early;
            workers[thread].run([&] {
                std::cout << order.admit(reinterpret_cast<const void *>(stream), cache, layer, 10, 1, early != 0, 304) << "\n";
            });
        } else if (cmd == "clear") {
            in >> thread;
            workers[thread].run([&] { order.clear(); });
        } else if (cmd == "settled") {
            in >> stream >> layer;
            std::cout << order.layer_settled(reinterpret_cast<const void *>(stream), cache, layer, 304) << "\n";
        }
    }
    return 0;
}

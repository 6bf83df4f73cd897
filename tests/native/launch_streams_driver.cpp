// Command-line driver of qa::LaunchOrder for streams of several devices and
// threads, one command per line (handles: 0 and 1 the legacy default stream, 2 the
// per-thread one); cache 7, layer 0 throughout:
//   admit <handle> <device> <thread> <ctas> [<capture>]  -> guard (304 blocks resident at most)
//   settled <handle> <device> <thread> 0 [<capture>]     -> 0 | 1
//   barrier <handle> <device> <thread> 0 [<capture>]
//   clear <device>
// thread 0 is this one, 1 a new one.
#include <cstdint>
#include <iostream>
#include <sstream>
#include <string>
#include <thread>

#include "launch_order.h"

int main() {
    qa::LaunchOrder order;
    const void *cache = reinterpret_cast<const void *>(7);
    std::string line;
    while (std::getline(std::cin, line)) {
        std::istringstream in(line);
        std::string cmd;
        unsigned long long handle = 0, capture = 0;
        int device = 0, thread = 0, ctas = 0;
        in >> cmd;
        if (cmd == "clear") {
            in >> device;
            order.clear(device);
            continue;
        }
        in >> handle >> device >> thread >> ctas >> capture;
        auto call = [&] {
            const qa::StreamRef at(reinterpret_cast<const void *>(handle), device, capture);
            if (cmd == "admit") std::cout << order.admit(at, cache, 0, ctas, 1, true, 304) << "\n";
            if (cmd == "settled") std::cout << order.layer_settled(at, cache, 0, 304) << "\n";
            if (cmd == "barrier") order.barrier(at);
        };
        if (thread) std::thread(call).join();
        else call();
    }
    return 0;
}

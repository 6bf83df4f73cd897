// Command-line driver of qa::LaunchOrder for captures whose streams follow each other's
// launches, one command per line; cache 7, 10 thread blocks a launch, 304 resident at most.
// <nodes>: those that the stream follows, "-" for none, "a,b" for two.
//   admit <stream> <capture> <layer> <early 0|1> <nodes> <node>  -> guard; it becomes <node>
//   settled <stream> <capture> <layer> <nodes>                   -> 0 | 1
//   inflight <stream> <capture> <layer> <nodes>                  -> 0 | 1 | 2
//   barrier <stream> <capture> <nodes>
#include <cstdint>
#include <iostream>
#include <sstream>
#include <string>

#include "launch_order.h"

int main() {
    qa::LaunchOrder order;
    const void *cache = reinterpret_cast<const void *>(7);
    std::string line;
    while (std::getline(std::cin, line)) {
        std::istringstream in(line);
        std::string cmd, nodes, node;
        unsigned long long stream = 0, capture = 0;
        int layer = 0, early = 1;
        in >> cmd >> stream >> capture;
        if (cmd != "barrier") in >> layer;
        if (cmd == "admit") in >> early;
        in >> nodes;
        qa::StreamRef at(reinterpret_cast<const void *>(stream), 0, capture);
        for (std::istringstream list(nodes); nodes != "-" && std::getline(list, node, ',');)
            at.after.push_back(std::stoul(node));
        if (cmd == "admit") {
            std::cout << order.admit(at, cache, layer, 10, 1, early != 0, 304) << "\n";
            in >> node;
            at.after = {std::stoul(node)};
            order.captured(at);
        } else if (cmd == "settled") {
            std::cout << order.layer_settled(at, cache, layer, 304) << "\n";
        } else if (cmd == "inflight") {
            std::cout << order.in_flight(at, cache, layer, 304) << "\n";
        } else {
            order.barrier(at);
        }
    }
    return 0;
}

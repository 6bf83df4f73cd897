// Command-line driver of csrc/q4_plan.h for the CPU tests, one command per line:
//   decode <D> <groups> <held 1..13> <n> <keys>*n   -> cluster, then the splits
//   parts <window> <D> <G> <Hkv> <sms> <n> (<start> <len>)*n
//                                      -> 1 when cut, heads an item, (run, lo, hi) per part
//   runs <window> <D> <G> <Hkv> <sms> <n> <start len>*n
//     -> span before, span after, then "seq first len" of every run
#include <iostream>
#include <sstream>
#include <string>
#include <vector>

#include "q4_plan.h"

int main() {
    std::string line;
    while (std::getline(std::cin, line)) {
        std::istringstream in(line);
        std::string cmd;
        in >> cmd;
        if (cmd == "decode") {
            int D, groups, n, held[qa::kQ4MaxSplits + 1] = {}, keys[qa::kQ4MaxSeqPerLaunch];
            in >> D >> groups;
            for (int S = 1; S <= qa::kQ4MaxSplits; ++S) in >> held[S];
            in >> n;
            for (int i = 0; i < n; ++i) in >> keys[i];
            qa::DecodePlan plan;
            qa::plan_decode(D, held, groups, n, keys, plan);
            std::cout << plan.cluster;
            for (int i = 0; i < n; ++i) std::cout << " " << plan.splits[i];
            std::cout << "\n";
        } else if (cmd == "parts") {
            int window, D, G, Hkv, sms, n, hpi = 0;
            in >> window >> D >> G >> Hkv >> sms >> n;
            std::vector<int> start(n);
            std::vector<qa::QueryRun> runs;
            for (int i = 0; i < n; ++i) {
                int len;
                in >> start[i] >> len;
                runs.push_back({i, 0, len});
            }
            std::vector<qa::KeyPart> parts;
            std::cout << qa::plan_parts(runs, start.data(), window, D, G, Hkv, sms, 8, parts, hpi) << " " << hpi;
            for (const qa::KeyPart &k : parts) std::cout << " " << k.run << " " << k.lo << " " << k.hi;
            std::cout << "\n";
        } else if (cmd == "runs") {
            int window, D, G, Hkv, sms, n;
            in >> window >> D >> G >> Hkv >> sms >> n;
            std::vector<int> start(n);
            std::vector<qa::QueryRun> runs;
            for (int i = 0; i < n; ++i) {
                int len;
                in >> start[i] >> len;
                runs.push_back({i, 0, len});
            }
            std::vector<int> load;
            int workers, copies, blocks = 0;
            for (const qa::QueryRun &r : runs) blocks += (r.len + 127) / 128;
            qa::prefill_form(blocks, D, G, Hkv, sms, workers, copies);
            std::cout << qa::prefill_span(runs, start.data(), window, copies, workers, load) << " ";
            qa::plan_runs(runs, start.data(), window, D, G, Hkv, sms, 8);
            std::cout << qa::prefill_span(runs, start.data(), window, copies, workers, load);
            for (const qa::QueryRun &r : runs) std::cout << " " << r.seq << " " << r.first << " " << r.len;
            std::cout << "\n";
        }
    }
    return 0;
}

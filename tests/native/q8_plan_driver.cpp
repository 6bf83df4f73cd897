// Command-line driver of csrc/q8_tail.h and csrc/q8_plan.h for the CPU tests, one
// command per line:
//   tail (<blk> <rows> <sealed>)*2 <start> <end> <keep> -> from, from_rows, dst, then the next state
//   of (<blk> <rows> <sealed>)*2 <blk> <row> <raw>      -> the buffer, or -1
//   step <sms> <Hkv> <most> <n> <work>*n                -> the largest number of splits, then each
//   work <D> <full> <n_blocks>                          -> blocks
#include <iostream>
#include <sstream>
#include <string>
#include <vector>

#include "q8_plan.h"
#include "q8_tail.h"

int main() {
    std::string line;
    while (std::getline(std::cin, line)) {
        std::istringstream in(line);
        std::string cmd;
        in >> cmd;
        qa::Q8Tail t{};
        if (cmd == "tail" || cmd == "of")
            for (int i = 0; i < 2; ++i) in >> t.blk[i] >> t.rows[i] >> t.sealed[i];
        if (cmd == "tail") {
            int start, end, keep;
            in >> start >> end >> keep;
            const qa::Q8TailPlan p = qa::q8_plan_tail(t, start, end, keep != 0);
            std::cout << p.from << " " << p.from_rows << " " << p.dst;
            for (int i = 0; i < 2; ++i) std::cout << " " << p.next.blk[i] << " " << p.next.rows[i] << " " << p.next.sealed[i];
        } else if (cmd == "of") {
            int blk, row, raw;
            in >> blk >> row >> raw;
            std::cout << qa::q8_tail_of(t, blk, row, raw != 0);
        } else if (cmd == "step") {
            int sms, hkv, most, n;
            in >> sms >> hkv >> most >> n;
            std::vector<int> work(n), splits(n);
            for (int &w : work) in >> w;
            std::cout << qa::q8_plan_step(sms, hkv, most, n, work.data(), splits.data());
            for (int s : splits) std::cout << " " << s;
        } else {
            int D, full, n;
            in >> D >> full >> n;
            std::cout << qa::q8_step_work(D, full, n);
        }
        std::cout << "\n";
    }
}

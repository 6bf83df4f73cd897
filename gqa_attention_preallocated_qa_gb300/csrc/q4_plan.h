// q4_plan.h -- how the 4-bit cache's launches are cut: splits of a decode step
// and runs of query blocks of a prefill (host code only, no CUDA dependency).
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>
#include <vector>

namespace qa {

constexpr int kQ4Chunk = 32;       // keys of one warp's part of a stage of the decode kernel
constexpr int kQ4DecodeWarps = 8;  // warps of a decode CTA
constexpr int kQ4MaxSplits = 13;   // splits of one (sequence, kv head) = CTAs of one cluster

constexpr int kQ4MaxSeqPerLaunch = 64;  // sequences carried in the parameters of one launch

// How a decode launch is cut: splits[i] CTAs work on each kv head (and head
// group) of sequence i, and clusters are of `cluster` CTAs, which every
// splits[i] divides.
struct DecodePlan {
    int cluster = 1;
    int splits[kQ4MaxSeqPerLaunch];
};

// A CTA costs a fixed part (its prologue and the merge) and a part per stage of
// 256 keys; CTAs that share an SM slow each other down.  Fitted on GB300 (D =
// 128, steps apart from each other, 512 to 16384 keys, 8 to 192 groups): 2.6 us
// + 1.1 us a stage for a CTA alone on its SM, 3.6 + 1.85 for two; at D = 64 a
// stage costs 0.66 times that.  CTAs get SMs of their own as long as the launch
// has at most 96 of them, or 128 in clusters of up to 4.
inline bool decode_alone(int cluster, int64_t ctas) { return ctas <= (cluster <= 4 ? 128 : 96); }
inline float decode_cta_us(int D, bool alone, int stages) {
    const float stage = D == 128 ? 1.f : 0.66f;
    return alone ? 2.6f + 1.1f * stage * stages : 3.6f + 1.85f * stage * stages;
}

// The plan of least cost for n sequences of keys[i] cached keys (in falling
// order), `groups` kv heads x head groups each.  Either every sequence has the
// same number of splits, all clusters on the device at once (held[S] clusters of
// S CTAs; the fewest splits among equals; B = 4, 8 kv heads: 4 splits at 2048
// keys take 7.8 us and 8 take 8.4; at 16384 keys 23.2 and 21.4); a short
// sequence's CTAs may then be left without keys.  Or, for mixed lengths, the
// longest has 2, 4 or 8 and the others as few (1, 2, 4, 8) as give no CTA more
// stages than the longest's.  A launch takes as long as its longest CTA; one of
// more CTAs than the device holds at least as long as their sum shared out and
// then its shortest, which starts last.  (8 kv heads, D = 128: one sequence of
// 16384 keys beside 3 of 2048 and 4 of 512 takes 14.8 us, with 4 splits each
// 23.5; 24 of 8000 down to 1 key 19.2, unsplit 40.4; 4 of 8192 beside 60 of 512,
// with 4 splits and 1, 25.6, unsplit 42.1.)
inline void plan_decode(int D, const int *held, int groups, int n, const int *keys, DecodePlan &plan) {
    int chunks[kQ4MaxSeqPerLaunch];
    for (int i = 0; i < n; ++i) chunks[i] = (keys[i] + kQ4Chunk - 1) / kQ4Chunk;
    plan.cluster = 1;
    std::fill(plan.splits, plan.splits + n, 1);
    if (!held) return;
    auto stages = [](int chunks, int S) { return (chunks + S * kQ4DecodeWarps - 1) / (S * kQ4DecodeWarps); };
    auto cost = [&](int S, const int *splits, int64_t ctas) {
        const float longest = decode_cta_us(D, decode_alone(S, ctas), stages(chunks[0], splits[0]));
        if ((ctas + S - 1) / S <= held[S]) return longest;
        float sum = 0.f;
        for (int i = 0; i < n; ++i) sum += splits[i] * decode_cta_us(D, false, stages(chunks[i], splits[i]));
        return std::max(longest, sum * groups / (held[S] * S) + decode_cta_us(D, false, stages(chunks[n - 1], splits[n - 1])));
    };
    float least = 1e30f;
    int s[kQ4MaxSeqPerLaunch];
    const int64_t total = static_cast<int64_t>(groups) * n;
    for (int S = 1; S <= kQ4MaxSplits && (S == 1 || S <= chunks[0]); ++S) {
        if (S > 1 && held[S] < total) continue;
        std::fill(s, s + n, S);
        const float us = cost(S, s, total * S);
        if (us < least - 0.01f) {
            least = us;
            plan.cluster = S;
        }
    }
    std::fill(plan.splits, plan.splits + n, plan.cluster);
    for (int S = 2; S <= 8 && S <= chunks[0] && held[S] > 0; S *= 2) {
        const int most = stages(chunks[0], S) * kQ4DecodeWarps;  // chunks of a CTA
        int64_t ctas = 0;
        for (int i = 0; i < n; ++i) {
            s[i] = 1;
            while (s[i] * most < chunks[i]) s[i] *= 2;
            ctas += static_cast<int64_t>(groups) * s[i];
        }
        if (s[0] < S || s[n - 1] == S) continue;  // a smaller cluster's, or equal splits
        // 0.3 us for what the fit leaves out
        const float us = cost(S, s, ctas);
        if (us < least - 0.3f) {
            least = us;
            plan.cluster = S;
            std::copy(s, s + n, plan.splits);
        }
    }
}

// Whether a sequence's new tokens go through the decode kernel, eight at a time,
// or through the prefill kernel on the dequantised cache, where up to 128 tokens
// cost the same.  (8 kv heads, 32 query heads, D = 128, eight tokens / prefill
// kernel: nothing cached 4.0 / 12.5 us for one sequence, 5.6 / 14.5 for four,
// 14 / 29 for 16; 512 keys 4.7 / 23, 7.4 / 25, 21 / 56; 2048 keys 7.0 / 26,
// 12.5 / 45, 37 / 115; 16384 keys 17.9 / 62, 53 / 179, 198 / 661.)
constexpr int kQ4MaxTokens = 8;  // new tokens per sequence of one decode launch
inline bool few_tokens(int start, int ntok, int window) {
    const int keys = window > 0 ? std::min(start, window) : start;
    return ntok <= kQ4MaxTokens * (keys < 512 ? 2 : 3);
}

// A prefill's rows (K4): warps of a CTA, one CTA per SM, each with a ring of two
// stages that hold one share of a token's query, key and value rows.
constexpr int kQ4RowWarps = 16;
constexpr size_t kQ4RowSmemMost = 200 * 1024 + 128;
inline size_t q4_prefill_rows_smem(int Hq, int Hkv, int D, int parts) {
    const size_t stage = (static_cast<size_t>(Hq / parts + 2 * (Hkv / parts)) * D * 2 + 127) & ~static_cast<size_t>(127);
    return static_cast<size_t>(kQ4RowWarps) * 2 * stage + 128;
}

// Shares that a token is cut into, by heads (0: no number of them fits): the
// fewest that fit (two at 32 + 2 x 8 heads of 128), and four as long as every
// share still has a warp of its own.  A power of two, and at most one for each
// warp of a CTA: a warp steps by gridDim * (warps / shares) tokens.  (Prefill of 256 tokens: 14.5 us with four
// shares and 16.6 with two; of 1024: 29.5 and 27.0; eight leave lanes idle.)
inline int q4_row_parts(int Hq, int Hkv, int D, int64_t T, int sms) {
    int parts = 1;
    while (q4_prefill_rows_smem(Hq, Hkv, D, parts) > kQ4RowSmemMost) {
        parts *= 2;
        if (parts > kQ4RowWarps || Hkv % parts) return 0;
    }
    while (parts < 4 && Hkv % (2 * parts) == 0 && 2 * T * parts <= static_cast<int64_t>(sms) * kQ4RowWarps) parts *= 2;
    return parts;
}

// A run of query blocks of one sequence of a prefill launch: rows first ..
// first + len - 1 of its new tokens.
struct QueryRun {
    int seq, first, len;
};

// Time of the prefill attention of `runs` in units of key tiles: its items are
// dealt out level by level (the block within its run, the highest first), then
// by run, to `workers` in snake order; a block costs its key tiles and about
// one more.  `copies`: items of a block (kv heads and head groups).
inline int prefill_span(const std::vector<QueryRun> &runs, const int *start, int window, int copies, int workers,
                        std::vector<int> &load) {
    load.assign(workers, 0);
    int levels = 0, idx = 0;
    for (const QueryRun &r : runs) levels = std::max(levels, (r.len + 127) / 128);
    for (int lvl = levels - 1; lvl >= 0; --lvl)
        for (const QueryRun &r : runs) {
            if (r.len <= lvl * 128) continue;
            const int pos = start[r.seq] + r.first + lvl * 128;
            const int from = window > 0 ? std::max(0, pos + 1 - window) / 128 : 0;
            const int tiles = (pos + std::min(r.len - 1 - lvl * 128, 127)) / 128 + 1 - from + 1;
            for (int k = 0; k < copies; ++k, ++idx) {
                const int round = idx / workers, at = idx % workers;
                load[round & 1 ? workers - 1 - at : at] += tiles;
            }
        }
    return *std::max_element(load.begin(), load.end());
}

// The form that a launch of so many query blocks takes: pairs of CTAs on four
// heads when every pair gets an item, else CTAs on two heads, or on one when
// there are fewer items than SMs.  copies: items of a block.
inline void prefill_form(int blocks, int D, int G, int Hkv, int sms, int &workers, int &copies) {
    workers = sms / 2;
    copies = Hkv * (G / 4);
    if (D == 128 && G % 4 == 0 && blocks * copies >= workers) return;
    workers = sms;
    copies = Hkv * ((G + 1) / 2);
    if (G > 1 && blocks * copies < workers) copies = Hkv * G;
}

// The runs a prefill launch is made of.  The kernel deals its items out by the
// block's place in its run, which is their weight when every sequence starts at
// 0; behind caches of different lengths it is not, and heavy blocks dealt late
// leave most of the device idle at the end.  So the sequences may go in by falling
// start, and the ones that start lowest may be cut into shorter runs (up to the
// 8 of a launch), whose blocks then come later.  Results are the same bits: an
// item does not depend on its neighbours.  (777 tokens behind 4099 and 1001
// behind 1025, 32 / 8 heads: 124 us as two runs, 86 us cut.)
inline void plan_runs(std::vector<QueryRun> &runs, const int *start, int window, int D, int G, int Hkv, int sms,
                      int max_runs) {
    bool same = true;
    int blocks = 0;
    for (const QueryRun &r : runs) {
        same = same && start[r.seq] == start[runs[0].seq];
        blocks += (r.len + 127) / 128;
    }
    int workers, copies;
    prefill_form(blocks, D, G, Hkv, sms, workers, copies);
    // One item or less per worker: no order matters.  Many per worker: none helps
    // much, and trying them would cost the host more.
    const int64_t items = static_cast<int64_t>(blocks) * copies;
    if (same || items <= workers || items > 16 * static_cast<int64_t>(workers)) return;
    std::vector<int> load;
    std::vector<QueryRun> best = runs;
    int least = prefill_span(runs, start, window, copies, workers, load);
    std::stable_sort(runs.begin(), runs.end(),
                     [&](const QueryRun &x, const QueryRun &y) { return start[x.seq] > start[y.seq]; });
    int span = prefill_span(runs, start, window, copies, workers, load);
    if (span < least) {
        least = span;
        best = runs;
    }
    for (size_t cut = 1; cut <= runs.size(); ++cut)        // the last `cut` sequences
        for (int m : {1, 2, 3, 4, 6, 8}) {                  // into runs of m blocks
            std::vector<QueryRun> tried(runs.begin(), runs.end() - cut);
            for (size_t i = runs.size() - cut; i < runs.size(); ++i)
                for (int at = (runs[i].len - 1) / (128 * m) * (128 * m); at >= 0; at -= 128 * m)
                    tried.push_back({runs[i].seq, at, std::min(128 * m, runs[i].len - at)});
            if (tried.size() > static_cast<size_t>(max_runs) || tried.size() == runs.size()) continue;
            span = prefill_span(tried, start, window, copies, workers, load);
            if (span < least) {
                least = span;
                best = tried;
            }
        }
    runs = best;
}

// A key tile of the one-CTA prefill kernel with h heads an item, us.
inline float tile_us(int D, int h) { return h == 2 ? (D == 128 ? 1.75f : 1.45f) : (D == 128 ? 1.3f : 1.2f); }

// Whether a launch that has fewer two-head items than SMs, but more one-head
// items, does better with two heads: one round of 1.75 us a key tile instead of
// two of 1.3.  (32 / 8 heads, D = 128: 8
// sequences of 128 tokens behind 16384 keys 458 -> 336 us, 5 of 100 behind 2048
// 72 -> 55, 4 prompts of 256 21.2 -> 20.4.)
inline bool two_heads(const std::vector<QueryRun> &runs, const int *start, int window, int D, int G, int Hkv, int sms) {
    int blocks = 0;
    for (const QueryRun &r : runs) blocks += (r.len + 127) / 128;
    const int64_t items = static_cast<int64_t>(blocks) * Hkv * (G / 2);
    if (G < 2 || items >= sms || 2 * items <= sms) return false;
    std::vector<int> load;
    const int two = prefill_span(runs, start, window, Hkv * (G / 2), sms, load);
    const int one = prefill_span(runs, start, window, Hkv * G, sms, load);
    return two * tile_us(D, 2) < one * tile_us(D, 1);
}

// A part of a run's keys: tiles lo .. hi - 1 of 128.
struct KeyPart {
    int run, lo, hi;
};

// Cuts the keys of few query blocks behind many keys into parts, so that the
// device's SMs share them, and says how many query heads an item takes; false
// when it does not pay.  Fitted on GB300 (D = 128; 1 to 4 sequences of 40 to 512
// tokens behind 1000 to 65536 keys): a key tile takes 1.75 us with two heads and
// 1.3 with one (the launch without parts: one head an item here), the join 5 us
// and 0.2 ns for each part of a row and head.  (32 / 8 heads, 128 tokens behind
// 16384 keys: 196 us without, 8 parts of two heads 68, 4 of one head 80; behind
// 2048 keys 39 and 33; behind 1000 keys 27.6, and 31.5 with 2 parts.  8 / 1 heads
// behind 16384 keys: 183, 8 parts of two heads 52, of one head 44.)
inline bool plan_parts(const std::vector<QueryRun> &runs, const int *start, int window, int D, int G, int Hkv, int sms,
                       int max_parts, std::vector<KeyPart> &parts, int &hpi) {
    const int nruns = static_cast<int>(runs.size());
    if (nruns == 0 || 2 * nruns > max_parts) return false;
    int blocks[kQ4MaxSeqPerLaunch], from[kQ4MaxSeqPerLaunch], tiles[kQ4MaxSeqPerLaunch];
    int total = 0, most = 0, rows = 0;
    for (int i = 0; i < nruns; ++i) {
        const int pos = start[runs[i].seq] + runs[i].first;
        blocks[i] = (runs[i].len + 127) / 128;
        from[i] = window > 0 ? std::max(0, pos + 1 - window) / 128 : 0;
        tiles[i] = pos / 128 + 1 - from[i];  // of the first block, up to the one its first row is in
        total += blocks[i];
        rows += runs[i].len;
        most = std::max(most, tiles[i] + blocks[i] - 1);
    }
    // Parts of run i when the most are n.  A later block's window starts up to
    // blocks - 1 tiles later: every part of it keeps a tile at least.
    auto cut = [&](int i, int n) {
        int m = std::min(n, tiles[i]);
        while (m > 1 && window > 0 && tiles[i] / m <= blocks[i]) --m;
        return m;
    };
    float least = tile_us(D, 1) * most - 1.f;
    int best = 1;
    for (int h = std::min(G, 2); h >= 1; --h) {
        const int items = total * Hkv * (G / h);
        for (int n = 2; n * nruns <= max_parts && n * items <= sms; ++n) {
            int longest = 0;
            for (int i = 0; i < nruns; ++i) {
                const int m = cut(i, n);
                longest = std::max(longest, (tiles[i] + m - 1) / m + blocks[i] - 1);
            }
            const float us = tile_us(D, h) * longest + 5.f + 0.2e-3f * (D / 128.f) * rows * (Hkv * G) * n;
            if (us < least) {
                least = us;
                best = n;
                hpi = h;
            }
        }
    }
    if (best == 1) return false;
    parts.clear();
    for (int i = 0; i < nruns; ++i)
        for (int k = 0, m = cut(i, best); k < m; ++k)
            parts.push_back({i, from[i] + static_cast<int>(int64_t(tiles[i]) * k / m),
                             k == m - 1 ? 1 << 30 : from[i] + static_cast<int>(int64_t(tiles[i]) * (k + 1) / m)});
    return true;
}

}  // namespace qa

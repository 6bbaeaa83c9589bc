// Whether two views of heads share a byte (host code, without CUDA: the tests compile it by itself).
#ifndef NVFP4_HEADS_OVERLAP_H
#define NVFP4_HEADS_OVERLAP_H

#include <cstdint>
#include <utility>

namespace nvfp4 {

// The bytes of a view: runs of `run` bytes, n[0] groups step[0] apart of n[1] runs step[1] apart (step[0] >=
// step[1]); the levels that are not needed are left out.
struct Runs {
    int64_t at, run;
    int levels;
    int64_t n[2], step[2];

    Runs(const void* data, int64_t heads, int64_t tokens, int64_t head_bytes, int64_t head_step, int64_t token_step)
        : at(static_cast<int64_t>(reinterpret_cast<intptr_t>(data))), run(head_bytes), levels(0)
    {
        if (tokens > 1 && token_step > 0) n[levels] = tokens, step[levels++] = token_step;
        if (heads > 1 && head_step > 0) n[levels] = heads, step[levels++] = head_step;
        if (levels == 2 && step[0] < step[1]) {
            std::swap(n[0], n[1]);
            std::swap(step[0], step[1]);
        }
        // runs that touch are one
        while (levels > 0 && step[levels - 1] <= run) {
            --levels;
            run += (n[levels] - 1) * step[levels];
        }
    }
    int64_t extent(int level) const  // of what lies below `level`
    {
        int64_t e = run;
        for (int i = level; i < levels; ++i) e += (n[i] - 1) * step[i];
        return e;
    }
};

// a's runs from level la on, at `at`, against b's from lb on at 0.  `tries` bounds the search between views of unlike
// strides that lie in one another without sharing a byte: behind it they count as apart.
inline bool runs_meet(const Runs& a, int la, int64_t at, const Runs& b, int lb, int& tries)
{
    const int64_t ea = a.extent(la), eb = b.extent(lb);
    if (at >= eb || at + ea <= 0) return false;
    const bool more_a = la < a.levels, more_b = lb < b.levels;
    if (!more_a && !more_b) return true;
    const int64_t step_a = more_a ? a.step[la] : 0, step_b = more_b ? b.step[lb] : 0;
    const int64_t step = step_a > step_b ? step_a : step_b;
    // the groups of the larger step, one by one; with equal steps only their distance counts
    const bool split_a = step_a == step, split_b = step_b == step;
    const int64_t wa = split_a ? a.extent(la + 1) : ea, wb = split_b ? b.extent(lb + 1) : eb;
    int64_t low = split_b ? -(b.n[lb] - 1) : 0, high = split_a ? a.n[la] - 1 : 0;
    // at + d step in (-wa, wb)
    const int64_t above = -wa - at, below = wb - at;
    const int64_t first = (above >= 0 ? above / step : -((-above + step - 1) / step)) + 1;
    const int64_t last = below > 0 ? (below - 1) / step : -((-below) / step) - 1;
    if (first > low) low = first;
    if (last < high) high = last;
    for (int64_t d = low; d <= high; ++d) {
        if (--tries < 0) return false;
        if (runs_meet(a, la + split_a, at + d * step, b, lb + split_b, tries)) return true;
    }
    return false;
}

inline bool runs_meet(const Runs& a, const Runs& b)
{
    int tries = 4096;
    return runs_meet(a, 0, a.at - b.at, b, 0, tries);
}

}  // namespace nvfp4

#endif

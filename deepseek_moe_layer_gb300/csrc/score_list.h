// score_list.h -- how long the scores' list of (tile, accumulator) can be.  Plain C++ (host only).
#pragma once

namespace moe {

// T tokens in groups of `tt`; a group is cut into a part for each of its sequences (B of them with
// tokens of any number each, or 0: one per token), a part has ceil(n / keys) tiles at most and an
// accumulator per `gtok` of its tokens for each.  An end of a sequence cuts at most one group once more.
inline long long score_list_bound(long long T, long long B, int tt, int gtok, long long n, int keys) {
    const long long groups = (T + tt - 1) / tt, ends = (B < T ? B : T) - 1;
    const long long parts = groups + (ends > 0 ? ends : 0);
    const long long cut = parts < T ? parts : T;  // (a part has a token)
    return cut * ((n + keys - 1) / keys) * ((tt + gtok - 1) / gtok);
}

}  // namespace moe

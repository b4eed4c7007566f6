// paged.cuh -- device helpers of the operators over a paged cache: which sequence a token belongs to,
// asynchronous 16-byte copies, waits, the issue of UMMAs.
#pragma once

#include "common.cuh"

namespace moe {

// A cache of `pages` pages of `page` rows; sequence b's position j lies in row j % page of page
// table[b * width + j / page].
struct Paged {
    const int32_t* table;
    int width, page;
    long long pages;
};

// Sequences of tokens: sequence b's are cu[b] .. cu[b + 1] - 1, or token b alone without cu.  (cu may
// be a copy in shared memory.)
struct Sequences {
    const int32_t* cu;       // [B + 1] or nullptr
    const int32_t* lengths;  // [T] positions a token may see
    int B, T;
    int most;                // positions a table row has room for
};

MOE_DEV int seq_tokens(const Sequences& q) {  // tokens that belong to a sequence
    return q.cu ? max(0, min(q.T, q.cu[q.B])) : q.T;
}
// The sequence of token t < seq_tokens(): the last b with cu[b] <= t.
MOE_DEV int seq_of(const Sequences& q, int t) {
    if (!q.cu) return t;
    int lo = 0, hi = q.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (q.cu[mid] <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}
MOE_DEV int seq_end(const Sequences& q, int b) { return q.cu ? min(q.T, q.cu[b + 1]) : b + 1; }
MOE_DEV int seq_length(const Sequences& q, int t) { return max(0, min(q.most, __ldg(q.lengths + t))); }

// 16 bytes global -> shared, of which the first `bytes` (16 or 0) are read and the rest is zero.
MOE_DEV void copy16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
MOE_DEV void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
MOE_DEV void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Whether the phase with this parity has completed, without waiting (try_wait suspends the thread
// until it has, or for some microseconds: copies that are announced behind it arrive late).
MOE_DEV bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// mbar_wait with a clock that is looked at only after some microseconds: a try returns after a while
// of its own accord, so waits go round more than once, and a warp that waits takes issue slots
// from those that share its scheduler (23 instructions a round with the clock in it, 5 without).
MOE_DEV bool mbar_wait_lean(uint64_t* bar, uint32_t parity, volatile int* abort) {
#pragma unroll 1
    for (int i = 0; i < 256; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return mbar_wait(bar, parity, abort);
}
// One lane of a converged warp, always the same.  UMMAs are issued by a warp that runs its loops
// converged, with the issue alone inside `if (elect_lane())`: the operands then are warp-uniform
// (four UMMAs of 128 x 128 x 16 by a CTA pair, with a wait and a commit: 142 clocks; in a loop
// that lane 0 runs alone 272).
MOE_DEV bool elect_lane() {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok));
    return ok != 0;
}
// Waits for the thread's TMEM loads, of which r is one: no use of r can move ahead of the wait.
MOE_DEV void tmem_ready(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
MOE_DEV void tmem_ready(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                   "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
// What this thread wrote to shared memory becomes visible to the tensor cores and the bulk copies.
MOE_DEV void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

}  // namespace moe

// indexer_scores.cu -- the indexer's scores of the cached positions on the 5th-generation tensor
// cores:
//     out[t, j] = ks_j * sum_h w[t, h] * max(q[t, h] . k_j, 0)    j < lengths[t], else -inf
// with index keys k_j of 128 columns in a paged cache, bf16 or e4m3 (ks_j: a scale per key).
//
// Keys lie on the tensor cores' M side (128 per tile) and (token, head) pairs on the N side: a
// thread then holds one key's dot products with all heads, the sum over the heads is its own
// and a token's scores leave as consecutive numbers.  A group is `tt` consecutive tokens (e4m3 up to 512
// columns, bf16 384), whose queries stay in shared memory while key tiles stream past them; tokens of
// several sequences in one group are taken sequence by sequence, with the columns of that
// sequence's tokens only.  Columns run in accumulators of up to 128 (whole tokens), four in
// TMEM with four warps each, so that the epilogue (a maximum and half a packed multiply-add per
// product) runs beside the UMMAs of the accumulators ahead and four of its warps share a scheduler
// (4096 x 16384 in 770 us; 1288 with two and 32 columns loaded ahead, 1016 with four and 16 ahead,
// 955 with eight accumulators of 64 columns; 637 with the runs below, 548 now).
//
// Work is one list of (tile, accumulator) over all groups and their sequences, as many tiles as the
// tokens can see, cut into equal runs, one per CTA (units of as many tiles, some of them out of sight:
// 64 sequences of 8192 to 32768 positions 59 us, 42 so).
//
// What bounds long prompts is the epilogue's instructions: 59% of issue slots and 55% of the pipe that
// takes the maxima at half rate, the tensor cores 35% (4096 x 16384 with 64 heads, e4m3: 548 us, 1755
// TFLOP/s).  Columns loaded ahead with more registers for it (563), an issuer per accumulator (563), an
// accumulator handed back before its last columns are weighed (543, but 64 sequences 41 -> 44) gain
// nothing.  64 sequences of up to 32768 positions: 41 us, of which 8 are start and end; HBM at 5.5 TB/s.
//
// Warp roles (768 threads, one CTA per SM): warps 0..15 epilogue (warp % 4 = TMEM lane quarter, warp / 4 =
// accumulator), 16..19 key copies (16-byte asynchronous copies, so that pages of any size and any order
// do; rows without a page or behind the end are zeros; a warp takes every fourth tile, so that
// four are in flight, and looks its next one's pages up meanwhile), 20 and 21 issue the UMMAs of every
// other accumulator (an issuer's waits and commits take as long as the UMMAs), 22 and 23 queries and
// weights.  Every wait is bounded.
#include <mutex>

#include "launch.h"
#include "paged.cuh"
#include "score_list.h"

namespace moe {

__device__ unsigned int g_scores_status;

namespace {

constexpr int kD = 128;             // columns of an index key
constexpr int kKeys = 128;          // keys per tile
constexpr int kAccCols = 128;       // of them per accumulator
constexpr int kAccs = 4;
constexpr int kEpiWarps = 4 * kAccs, kLoadWarps = 4, kMmaWarps = 2, kQueryWarps = 2;
constexpr int kMmaWarp = kEpiWarps + kLoadWarps, kQueryWarp = kMmaWarp + kMmaWarps;
constexpr int kThreads = 32 * (kQueryWarp + kQueryWarps);

template <bool F8>
struct Cfg {
    static constexpr int kRowBytes = F8 ? kD : 2 * kD;
    static constexpr int kBlocks = kRowBytes / 128;         // 128-byte blocks of a row
    static constexpr int kCols = F8 ? 512 : 384;            // (token, head) columns of a group
    static constexpr int kQBytes = kCols * kRowBytes;
    static constexpr int kStageBytes = kKeys * kRowBytes;
    static constexpr int kStages = F8 ? 8 : 4;
    static_assert(kStages % kLoadWarps == 0, "a stage is one warp's, so its waits are in order");
    // Which keys of a tile are there, and their scales, for the epilogue: written before the tile is
    // announced, read until its last accumulator is.  A place is taken again kRing tiles later, when
    // the UMMAs of tile kRing - kStages behind are done, which had waited for all but kAccs of the
    // accumulators before theirs.
    static constexpr int kRing = 16;
    static_assert(kRing - kStages > kAccs, "the epilogue is done with a place that is taken again");
    static constexpr int kStageOff = kQBytes;
    static constexpr int kWOff = kStageOff + kStages * kStageBytes;
    static constexpr int kLenOff = kWOff + 4 * kCols;       // a group's lengths
    static constexpr int kScaleOff = kLenOff + 4 * (kCols / 16);
    static constexpr int kThereOff = kScaleOff + (F8 ? 4 * kKeys * kRing : 0);
    static constexpr int kBarOff = kThereOff + 16 * kRing;
    // full, empty, known (per place of the ring), query full, query empty, accumulator full, empty, done
    static constexpr int kBars = 2 * kStages + kRing + 2 + 2 * kAccs + 1;
    static constexpr int kMiscOff = kBarOff + 8 * kBars;
    static constexpr int kSmemBytes = kMiscOff + 16;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
    // fp32 accumulator (bits 4-5 = 1); A and B bf16 (bits 7-9, 10-12 = 1) or e4m3 (0); both K-major
    static constexpr uint32_t kIdesc0 =
        (1u << 4) | (F8 ? 0u : (1u << 7) | (1u << 10)) | ((128u >> 4) << 24);
};

struct Params {
    Paged keys;
    Sequences seq;
    const uint8_t* k;        // rows of kRowBytes
    const float* ks;         // F8: [rows] scales
    const uint8_t* q;        // [T, H, kD]
    const float* w;          // [T, H]
    int H, Hp;               // heads; the same rounded up to 16
    int n;                   // positions of an output row
    float* out;              // [T, ld]
    long long ld;
    int tt, gtok;            // tokens of a group, of an accumulator
};

MOE_DEV void umma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                     uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

MOE_DEV void record_timeout(volatile int* abort) {
    *abort = 1;
    atomicCAS(&g_scores_status, 0u, kStatusTimeout);
}

// The part of a group (tokens u0 .. u1 - 1) that belongs to one sequence: tokens t0 .. t1 - 1 of
// sequence b, `accs` accumulators for each of the tiles that one of them can see; c0 .. c1 - 1 of
// these tiles are this CTA's.
struct Part {
    int b, u0, u1, t0, t1, accs, tiles, c0, c1;
};
MOE_DEV void part_at(const Params& p, int tokens, int t, Part& r) {
    r.u0 = t - t % p.tt;
    r.u1 = min(tokens, r.u0 + p.tt);
    r.b = seq_of(p.seq, t);
    r.t0 = t;
    r.t1 = max(t + 1, min(r.u1, seq_end(p.seq, r.b)));
    int most = 0;
    for (int i = r.t0; i < r.t1; ++i) most = max(most, seq_length(p.seq, i));
    r.tiles = (min(most, p.n) + kKeys - 1) / kKeys;
    r.accs = (r.t1 - r.t0 + p.gtok - 1) / p.gtok;
}

// A CTA's run lo .. hi - 1 of the list, from the part at token t, the list's entry `at`, on.
struct Start {
    long long lo, hi, at;
    int t, pad;
};
// Its parts, in order; every thread that walks sees the same ones.
struct Walk {
    Start s;
    int tokens;
    MOE_DEV Walk(const Start& st, int tokens) : s(st), tokens(tokens) {}
    MOE_DEV bool part(const Params& p, Part& r) {
        while (s.t < tokens && s.at < s.hi) {
            part_at(p, tokens, s.t, r);
            // a tile is the run's that holds its first accumulator
            const auto from = [&](long long x) {
                const long long d = x - s.at;
                return d <= 0 ? 0 : d >= (long long)r.tiles * r.accs
                           ? r.tiles : (int)((unsigned)(d + r.accs - 1) / (unsigned)r.accs);
            };
            r.c0 = from(s.lo);
            r.c1 = from(s.hi);
            s.at += (long long)r.tiles * r.accs;
            s.t = r.t1;
            if (r.c0 < r.c1) return true;
        }
        return false;
    }
};

// The key tiles of a run, in order.
struct Tiles {
    Walk w;
    Part r;
    int c;
    bool more;
    MOE_DEV Tiles(const Params& p, const Start& st, int tokens) : w(st, tokens) {
        more = w.part(p, r);
        c = more ? r.c0 : 0;
    }
    MOE_DEV void next(const Params& p) {
        if (++c < r.c1) return;
        more = w.part(p, r);
        c = r.c0;
    }
};

// sum += 16 products' maximum with 0 times their heads' weights.
MOE_DEV void weigh16(const uint32_t* v, const float* w, float2& s0, float2& s1) {
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
        const float4 q = *reinterpret_cast<const float4*>(w + e);
        float x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[k] = __uint_as_float(v[e + k]);
            asm("max.NaN.f32 %0, %0, 0f00000000;" : "+f"(x[k]));
        }
        s0 = __ffma2_rn(make_float2(x[0], x[1]), make_float2(q.x, q.y), s0);
        s1 = __ffma2_rn(make_float2(x[2], x[3]), make_float2(q.z, q.w), s1);
    }
}

// The products of heads that are not there: 0, where an infinite key makes them NaN.
MOE_DEV void clear_last(uint32_t* v, int n) {
#pragma unroll
    for (int e = 0; e < 16; ++e)
        if (e >= 16 - n) v[e] = 0u;
}

// HP: the heads, for loops of known length in the epilogue, or 0 for any number of them
// (4096 x 16384 with 64 heads: 615 us with 0, 548 with 64; 3 ragged prompts with 32: 47 and 44).
// 16 and 128 also divide an accumulator; they were not measured and take the loop of any length.
template <bool F8, int HP>
__global__ void __launch_bounds__(kThreads, 1) scores_kernel(const Params p) {
    using C = Cfg<F8>;
    extern __shared__ __align__(1024) uint8_t smem[];
    float* wts = reinterpret_cast<float*>(smem + C::kWOff);
    int* lens = reinterpret_cast<int*>(smem + C::kLenOff);
    float* scales = reinterpret_cast<float*>(smem + C::kScaleOff);
    uint32_t* there = reinterpret_cast<uint32_t*>(smem + C::kThereOff);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
    uint64_t* empty = full + C::kStages;
    uint64_t* known = empty + C::kStages;
    uint64_t* qfull = known + C::kRing;
    uint64_t* qempty = qfull + 1;
    uint64_t* afull = qfull + 2;
    uint64_t* aempty = afull + kAccs;
    uint64_t* done = aempty + kAccs;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
    volatile int* abort = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // entries of the list of this thread's groups (asked for before the set-up waits for anything)
    const int tokens = seq_tokens(p.seq);
    const int groups = (tokens + p.tt - 1) / p.tt, per = (groups + kThreads - 1) / kThreads;
    const int a = min((long long)tokens, (long long)threadIdx.x * per * p.tt);
    const int z = min((long long)tokens, (long long)a + (long long)per * p.tt);
    long long mine = 0;
    {
        Part r;
        for (int t = a; t < z; t = r.t1) {
            part_at(p, tokens, t, r);
            mine += (long long)r.tiles * r.accs;
        }
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kMmaWarps);
        }
        for (int i = 0; i < C::kRing; ++i) mbar_init(&known[i], 1);
        mbar_init(qfull, 32 * kQueryWarps);
        mbar_init(qempty, kMmaWarps + kEpiWarps);  // the unit's last UMMAs, and the weights read
        for (int i = 0; i < kAccs; ++i) {
            mbar_init(&afull[i], 1);
            mbar_init(&aempty[i], 4);
        }
        mbar_init(done, kMmaWarps);
        *abort = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) tmem_alloc(tmem_slot, 512);
    // this CTA's run: a prefix sum over the groups, through what will hold the queries
    Start* start = reinterpret_cast<Start*>(smem + 256);
    {
        long long* scan = reinterpret_cast<long long*>(smem);
        long long incl = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) scan[warp] = incl;
        if (threadIdx.x == 0) start->lo = start->hi = start->at = 0, start->t = tokens;
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (__any_sync(0xFFFFFFFFu, mine > 0)) {
            long long upto = lane < kThreads / 32 ? scan[lane] : 0;
            for (int o = 1; o < 32; o <<= 1) {
                const long long v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
                if (lane >= o) upto += v;
            }
            const long long total = __shfl_sync(0xFFFFFFFFu, upto, 31);
            const long long before = (warp ? __shfl_sync(0xFFFFFFFFu, upto, max(warp, 1) - 1) : 0) + incl - mine;
            long long lo, hi;
            if (total < (1 << 22)) {  // (64-bit divisions take a microsecond)
                lo = (unsigned)total * blockIdx.x / gridDim.x;
                hi = (unsigned)total * (blockIdx.x + 1) / gridDim.x;
            } else {
                lo = total * blockIdx.x / gridDim.x;
                hi = total * (blockIdx.x + 1) / gridDim.x;
            }
            if (lo < hi && before <= lo && lo < before + mine) {
                long long at = before;
                Part r;
                for (int t = a; t < z; t = r.t1) {
                    part_at(p, tokens, t, r);
                    const long long n = (long long)r.tiles * r.accs;
                    if (at <= lo && lo < at + n) {
                        start->lo = lo;
                        start->hi = hi;
                        start->at = at;
                        start->t = t;
                    }
                    at += n;
                }
            }
        }
    }
    __syncthreads();
    const uint32_t tmem = *tmem_slot;
    const Start st = *start;
    __syncthreads();  // (where it was, queries come)
    const int gtok = p.gtok;
    bool ok = true;
    const auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        if (__all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort))) return true;
        if (lane == 0) record_timeout(abort);
        return ok = false;
    };

    if (warp >= kEpiWarps && warp < kMmaWarp) {
        // ================================ key copies ================================
        constexpr int kPer = C::kRowBytes / 16;   // 16-byte pieces of a row
        constexpr int kRows = 32 / kPer;          // rows that a warp copies at once
        const int piece = lane % kPer, sub = lane / kPer;
        const uint32_t dst0 = (piece / 8) * (kKeys * 128) + sub * 128;
        Tiles tile(p, st, tokens);
        uint32_t it = 0;
        for (; (int)it < warp - kEpiWarps && tile.more; ++it) tile.next(p);
        int id[4], off[4];                        // page and row in it of the keys 32 k + lane
        const auto ask = [&] {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int pos = tile.c * kKeys + 32 * k + lane;
                const unsigned at = (unsigned)pos / (unsigned)p.keys.page;
                off[k] = pos - (int)(at * (unsigned)p.keys.page);
                id[k] = pos < p.seq.most
                            ? __ldg(p.keys.table + (long long)tile.r.b * p.keys.width + at) : -1;
            }
        };
        if (tile.more) ask();
        while (tile.more) {
            const uint32_t s = it % C::kStages, ring = it % C::kRing;
            int row[4];
            float ks[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                row[k] = (unsigned)id[k] < (unsigned long long)p.keys.pages ? id[k] * p.keys.page + off[k] : -1;
                if (F8) ks[k] = row[k] >= 0 ? __ldg(p.ks + row[k]) : 0.0f;
            }
            if (!wait(&empty[s], ((it / C::kStages) & 1u) ^ 1u)) break;
            const uint32_t to = smem_u32(smem + C::kStageOff + s * C::kStageBytes) + dst0;
#pragma unroll
            for (int i = 0; i < kKeys / kRows; ++i) {
                const int at = __shfl_sync(0xFFFFFFFFu, row[i * kRows / 32], (i * kRows + sub) & 31);
                copy16(to + i * kRows * 128 + (((piece & 7) ^ ((i * kRows + sub) & 7)) << 4),
                       p.k + (long long)max(at, 0) * C::kRowBytes + piece * 16, at < 0 ? 0u : 16u);
            }
            copy_commit();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (F8) scales[ring * kKeys + 32 * k + lane] = ks[k];
                const uint32_t bits = __ballot_sync(0xFFFFFFFFu, row[k] >= 0);
                if (lane == 0) there[ring * 4 + k] = bits;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&known[ring]);
            it += kLoadWarps;
            for (int k = 0; k < kLoadWarps && tile.more; ++k) tile.next(p);
            if (tile.more) ask();
            copy_wait<0>();
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[s]);
        }
        copy_wait<0>();
    } else if (warp >= kQueryWarp) {
        // ============================ queries and weights ============================
        const int tid = (int)threadIdx.x - 32 * kQueryWarp;
        Walk w(st, tokens);
        Part r;
        bool more = w.part(p, r);
        for (uint32_t n = 0; more; ++n) {
            const int u0 = r.u0, u1 = r.u1;
            if (!wait(qempty, (n & 1u) ^ 1u)) break;
            const uint32_t base = smem_u32(smem);
            constexpr int kPer = C::kRowBytes / 16;
            const int rows = (u1 - u0) * p.Hp;
            const int piece = tid % kPer;
            const uint32_t dst = base + (piece / 8) * (C::kCols * 128);
            const uint8_t* q = p.q + (long long)u0 * p.H * C::kRowBytes + piece * 16;
            const float* w0 = p.w + (long long)u0 * p.H;
            if (p.H == p.Hp) {  // (rows as they lie)
#pragma unroll 8
                for (int rr = tid / kPer; rr < rows; rr += 32 * kQueryWarps / kPer)
                    copy16(dst + rr * 128 + (((piece & 7) ^ (rr & 7)) << 4), q + rr * C::kRowBytes, 16u);
                copy_commit();
                for (int i = tid; i < rows; i += 32 * kQueryWarps) wts[i] = __ldg(w0 + i);
            } else {
#pragma unroll 4
                for (int rr = tid / kPer; rr < rows; rr += 32 * kQueryWarps / kPer) {
                    const int t = rr / p.Hp, h = rr % p.Hp;
                    copy16(dst + rr * 128 + (((piece & 7) ^ (rr & 7)) << 4),
                           q + (t * p.H + (h < p.H ? h : 0)) * C::kRowBytes, h < p.H ? 16u : 0u);
                }
                copy_commit();
                for (int i = tid; i < rows; i += 32 * kQueryWarps) {
                    const int t = i / p.Hp, h = i % p.Hp;
                    wts[i] = h < p.H ? __ldg(w0 + t * p.H + h) : 0.0f;
                }
            }
            for (int t = tid; t < u1 - u0; t += 32 * kQueryWarps) lens[t] = seq_length(p.seq, u0 + t);
            copy_wait<0>();
            fence_async_shared();
            mbar_arrive(qfull);
            do more = w.part(p, r);
            while (more && r.u0 == u0);
            // the next group's on their way to L2
            if (more)
                for (int i = tid; i < (r.u1 - r.u0) * p.H * (C::kRowBytes / 128); i += 32 * kQueryWarps)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(p.q + (long long)r.u0 * p.H * C::kRowBytes +
                                                                 i * 128)
                                 : "memory");
        }
    } else if (warp >= kMmaWarp) {
        // ================================ UMMA issuers ================================
        const uint32_t mine = warp - kMmaWarp;  // accumulators of this parity
        uint32_t it = 0, acc = 0;
        const uint64_t dq = sdesc_k128(smem_u32(smem)), dk = sdesc_k128(smem_u32(smem + C::kStageOff));
        Walk w(st, tokens);
        Part r;
        bool more = w.part(p, r);
        for (uint32_t n = 0; more && ok; ++n) {
            const int u0 = r.u0;
            if (!wait(qfull, n & 1u)) break;
            do {
                const int accs = r.accs;
                for (int c = r.c0; c < r.c1 && ok; ++c, ++it, acc += accs) {
                    const uint32_t s = it % C::kStages;
                    int k = (int)((mine - acc) & (kMmaWarps - 1));
                    bool here = mbar_test(&aempty[(acc + k) & (kAccs - 1)], (((acc + k) / kAccs) & 1u) ^ 1u);
                    if (!wait(&full[s], (it / C::kStages) & 1u)) break;
                    tc_fence_after();
                    const uint64_t da = dk + (uint64_t)(s * (C::kStageBytes / 16));
                    for (; k < accs; k += kMmaWarps) {
                        const uint32_t a1 = acc + k, ab = a1 & (kAccs - 1), a2 = a1 + kMmaWarps;
                        if (!__all_sync(0xFFFFFFFFu, here) && !wait(&aempty[ab], ((a1 / kAccs) & 1u) ^ 1u)) break;
                        here = mbar_test(&aempty[a2 & (kAccs - 1)], ((a2 / kAccs) & 1u) ^ 1u);
                        tc_fence_after();
                        const int t = r.t0 + k * gtok, cols = min(gtok, r.t1 - t) * p.Hp;
                        const uint32_t idesc = C::kIdesc0 | ((uint32_t)(cols >> 3) << 17);
                        const uint64_t db = dq + (uint64_t)((t - u0) * p.Hp * 8);
                        if (elect_lane()) {
#pragma unroll
                            for (int blk = 0; blk < C::kBlocks; ++blk)
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const uint64_t a = da + (uint64_t)(blk * (kKeys * 128 / 16) + 2 * e);
                                    const uint64_t b = db + (uint64_t)(blk * (C::kCols * 128 / 16) + 2 * e);
                                    if (F8) umma_f8(tmem + ab * kAccCols, a, b, idesc, blk + e > 0);
                                    else umma_bf16(tmem + ab * kAccCols, a, b, idesc, blk + e > 0);
                                }
                            umma_commit(&afull[ab]);
                        }
                        __syncwarp();
                    }
                    if (ok && elect_lane()) umma_commit(&empty[s]);
                    __syncwarp();
                }
                more = w.part(p, r);
            } while (more && ok && r.u0 == u0);
            if (ok && elect_lane()) umma_commit(qempty);
            __syncwarp();
        }
        if (elect_lane()) umma_commit(done);  // no UMMA is left when the CTA frees its TMEM
        __syncwarp();
        mbar_wait(done, 0u, nullptr, 100000000ull);
    } else {
        // ================================= epilogue =================================
        const int quarter = warp & 3;
        const uint32_t mine = warp >> 2;  // its accumulator
        const uint32_t ta0 = tmem + ((uint32_t)(quarter * 32) << 16) + mine * kAccCols;
        // what no token of a part can see, 4096 positions per warp
        const int runs = (int)(((long long)p.n + 4095) / 4096);
        for (long long f = (long long)blockIdx.x * kEpiWarps + warp; f < (long long)tokens * runs;
             f += (long long)gridDim.x * kEpiWarps) {
            const int t = (int)(f / runs), b = seq_of(p.seq, t), u0 = t - t % p.tt;
            const int t0 = p.seq.cu ? min(t, max(u0, p.seq.cu[b])) : t;
            Part r;
            part_at(p, tokens, t0, r);
            const int at = (int)(f % runs) * 4096, j1 = at + min(p.n - at, 4096);
            for (int j = max(at, r.tiles * kKeys) + lane; j < j1; j += 32)
                p.out[(long long)t * p.ld + j] = -__int_as_float(0x7F800000);
        }
        uint32_t it = 0, acc = 0;
        Walk walk(st, tokens);
        Part r;
        bool more = walk.part(p, r);
        for (uint32_t n = 0; more && ok; ++n) {
            const int u0 = r.u0;
            if (!wait(qfull, n & 1u)) break;  // (the weights and lengths)
            do {
                const int accs = r.accs;
                // of the accumulator `was` of a tile (always the same one, where a tile has kAccs)
                int was = -1, cnt = 0, pos = r.c0 * kKeys + quarter * 32 + lane;
                const float* w0 = wts;
                const int* len = lens;
                float* out0 = p.out;
                for (int c = r.c0; c < r.c1 && ok; ++c, ++it, acc += accs, pos += kKeys) {
                    const uint32_t ring = it % C::kRing;
                    int hidden = 0x7FFFFFFF;  // the key's position, if it is there
                    float ks = 1.0f;
                    // the tile's accumulators k with (acc + k) % kAccs == mine
                    for (int k = (int)((mine - acc) & (kAccs - 1)), told = 0; k < accs; k += kAccs) {
                        if (k != was) {
                            was = k;
                            const int t = r.t0 + k * gtok;
                            cnt = min(gtok, r.t1 - t);
                            w0 = wts + (t - u0) * p.Hp;
                            len = lens + (t - u0);
                            out0 = p.out + (long long)t * p.ld;
                        }
                        if (!told) {
                            if (!wait(&known[ring], (it / C::kRing) & 1u)) break;
                            if (there[ring * 4 + quarter] >> lane & 1u) hidden = pos;
                            if (F8) ks = scales[ring * kKeys + 32 * quarter + lane];
                            told = 1;
                        }
                        if (!wait(&afull[mine], ((acc + k) / kAccs) & 1u)) break;
                        tc_fence_after();
                        uint32_t ta = ta0;
                        const float* w = w0;
                        float* out = out0 + pos;
                        const auto put = [&](int i, float2 s0, float2 s1) {
                            const float sum = (s0.x + s0.y) + (s1.x + s1.y);
                            if (pos < p.n) *out = hidden < len[i] ? sum * ks : -__int_as_float(0x7F800000);
                        };
                        if constexpr (HP != 0) {
#pragma unroll
                            for (int i = 0; i < kAccCols / HP; ++i, out += p.ld) {
                                if (i >= cnt) break;
                                float2 s0 = make_float2(0.0f, 0.0f), s1 = s0;
#pragma unroll
                                for (int h = i * HP; h < i * HP + HP; h += 32) {
                                    uint32_t v[32];
                                    tmem_ld32(ta + (uint32_t)h, v);
                                    tmem_ready(v);
                                    weigh16(v, w + h, s0, s1);
                                    weigh16(v + 16, w + h + 16, s0, s1);
                                }
                                put(i, s0, s1);
                            }
                        } else {
                            const int absent = p.Hp - p.H;  // of a token's last 16 columns
                            for (int i = 0; i < cnt; ++i, out += p.ld) {
                                float2 s0 = make_float2(0.0f, 0.0f), s1 = s0;
                                int h = p.Hp;
                                for (; h >= 32; h -= 32, ta += 32, w += 32) {
                                    uint32_t v[32];
                                    tmem_ld32(ta, v);
                                    tmem_ready(v);
                                    if (h == 32 && absent) clear_last(v + 16, absent);
                                    weigh16(v, w, s0, s1);
                                    weigh16(v + 16, w + 16, s0, s1);
                                }
                                if (h) {
                                    uint32_t v[16];
                                    tmem_ld16(ta, v);
                                    tmem_ready(v);
                                    if (absent) clear_last(v, absent);
                                    weigh16(v, w, s0, s1);
                                    ta += 16;
                                    w += 16;
                                }
                                put(i, s0, s1);
                            }
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&aempty[mine]);
                    }
                }
                more = walk.part(p, r);
            } while (more && ok && r.u0 == u0);
            __syncwarp();
            if (lane == 0) mbar_arrive(qempty);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <bool F8, int HP>
cudaError_t run(const ScoresArgs& a, cudaStream_t s) {
    using C = Cfg<F8>;
    static DeviceOnce once;
    const cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(scores_kernel<F8, HP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    C::kSmemBytes);
    });
    if (e != cudaSuccess) return e;
    Params p = {};
    p.keys = {a.table, a.width, a.page, a.pages};
    const long long room = (long long)a.width * a.page;
    p.seq = {a.cu, a.lengths, a.B, (int)a.T, (int)(room < 0x7FFFFF00 ? room : 0x7FFFFF00)};
    p.k = static_cast<const uint8_t*>(a.keys);
    p.ks = a.key_scales;
    p.q = static_cast<const uint8_t*>(a.q);
    p.w = a.weights;
    p.H = a.H;
    p.Hp = (a.H + 15) / 16 * 16;
    p.n = a.n;
    p.out = a.out;
    p.ld = a.ld;
    p.gtok = kAccCols / p.Hp;
    // tokens of a group: what a sequence has on average, as far as the columns go
    const int avg = a.cu ? (int)((a.T + a.B - 1) / a.B) : 1;
    p.tt = C::kCols / p.Hp;
    if (avg < p.tt) p.tt = avg;
    // no more CTAs than the list can have entries
    const long long most = score_list_bound(a.T, a.cu ? a.B : 0, p.tt, p.gtok, a.n, kKeys);
    const long long grid = most < num_sms() ? most : num_sms();
    return launch_kernel(scores_kernel<F8, HP>, dim3((unsigned)grid), dim3(kThreads), (size_t)C::kSmemBytes,
                         s, p);
}

}  // namespace

cudaError_t launch_scores(const ScoresArgs& a, cudaStream_t s) {
    if (a.key_scales)
        return a.H == 64 ? run<true, 64>(a, s) : a.H == 32 ? run<true, 32>(a, s) : run<true, 0>(a, s);
    return a.H == 64 ? run<false, 64>(a, s) : a.H == 32 ? run<false, 32>(a, s) : run<false, 0>(a, s);
}

cudaError_t read_scores_status(unsigned int* out, int clear, cudaStream_t s) {
    cudaError_t err = cudaMemcpyFromSymbolAsync(out, g_scores_status, sizeof(unsigned int), 0,
                                                cudaMemcpyDeviceToHost, s);
    if (err != cudaSuccess) return err;
    err = cudaStreamSynchronize(s);
    if (err != cudaSuccess || !clear) return err;
    const unsigned int zero = 0;
    err = cudaMemcpyToSymbolAsync(g_scores_status, &zero, sizeof(unsigned int), 0,
                                  cudaMemcpyHostToDevice, s);
    if (err != cudaSuccess) return err;
    return cudaStreamSynchronize(s);
}

}  // namespace moe

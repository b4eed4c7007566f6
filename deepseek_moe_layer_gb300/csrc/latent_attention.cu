// latent_attention.cu -- attention over a paged cache of one latent row per position, absorbed form,
// on the 5th-generation tensor cores:
//     o[t, h] = sum_j p_j c_j[0:512],   p = softmax_j(scale * q[t, h] . c_j),   c_j 576 columns
// over the first lengths[t] positions of token t's sequence, or over the selected ones inds[t, :].
// All heads read the same rows: a cache row is loaded once and is key and value of every head.
//
// One pass over the positions with the softmax's running maximum m and sum l per (token, head) row,
// both fp32 and in base 2.  The maximum is a reference only: it moves (and the sums are
// rescaled) when a score passes it by more than 8, so p <= 2^8 and the rescaling of 512 columns of
// TMEM is rare.  p is rounded to bf16 for the second product (at most 2^-8 of each term, the inputs'
// own precision); l sums the fp32 values.
//
// 128 rows x 512 fp32 columns of o are all of an SM's TMEM, so a CTA pair shares them: each CTA
// has 64 rows, and cta_group::2 UMMAs with M = 128 run both halves at the full rate (a CTA's 64 rows
// lie in lanes 0..63 for the first half of N and in lanes 64..127 for the second).  A tile is 128
// positions.  s = q c^T (N = 128, K = 576): each CTA holds 64 of the positions as the K-major B
// operand.  o += p c (N = 512 as two UMMAs of 256, K = 128): each CTA holds half of the columns of
// all 128 positions, the same swizzled rows read as an MN-major B operand.  (N = 64 takes as long as
// N = 128, 36 clocks, so tiles of 64 positions spend twice the time on s.)
//
// q, one tile of keys, its values and p fill shared memory, so every operand block has one place and goes
// round once a tile: freed by its UMMAs, copied (1900 .. 2100 clocks), waited for, used.  That bounds a
// long call: 3400 clocks a tile, where the UMMAs take 2340 and the copies, at the 15.5 TB/s that they reach
// alone, 2500 (a pair loads 278 KB per tile where 147 KB are unique, the rest a second time from L2): 2048
// tokens x 2048 selected 871 us, 10.5 TB/s copied, 1340 TFLOP/s (955 us after some seconds, under the power
// cap); 64 sequences of up to 16384 positions 164 us (185), 8.8 TB/s copied, 4.6 of them from HBM.  Values
// copied out of the pair's keys instead would have to wait for the last tile's second product and hold the
// keys' places meanwhile.
//
// Work is one list of tiles over all segments (up to 128 / H consecutive tokens of a sequence;
// one token with a selection), cut into equal runs, one per pair, so that sequences of any
// lengths fill the device; a segment cut apart leaves partial sums (m, l, o in fp32) that a second
// kernel joins in the order of the pairs: equal calls give equal bits.  Where whole segments give
// a longest run that is no longer than an equal one and the cost of cutting (kCutTiles), runs are
// whole segments; where there are two pairs or more for each, pieces of one segment each (kTries).
//
// Warp roles (1024 threads): warps 0..7 softmax, rescaling and epilogue (a row's 128 positions are
// four threads': TMEM lane half x half of its columns), 8 and 9 issue the two products' UMMAs (of the
// pair's even CTA; one warp for both waits for barriers as long as the tensor cores work), 10
// finds the rows of the tiles ahead, 11 and 29..31 load the queries, 12..20 copy the K-major rows, a
// block of 64 columns each, 21..28 the MN-major columns, 16 positions each (16-byte asynchronous
// copies, so pages of any size and selected rows are alike; absent rows are zeros).  A copying warp has one place in shared
// memory: it waits until that is free, copies, waits for the data and announces it.  p goes
// through two blocks of 64 positions that are freed and filled apart, so that the second product of
// a tile follows on the last one's.  Every wait is bounded.
#include <mutex>

#include "launch.h"
#include "paged.cuh"

namespace moe {

__device__ unsigned int g_attention_status;

namespace {

constexpr int kWidth = 576, kLatent = 512;
constexpr int kRowBytes = 2 * kWidth;
constexpr int kTile = 128;                      // positions per tile
constexpr int kRows = 128;                      // (token, head) rows of a pair
constexpr int kSoftWarps = 8, kMmaWarp = 8, kFindWarp = 10, kQWarp = 11, kKWarp = 12;
constexpr int kSoftThreads = 32 * kSoftWarps;
// Operand blocks are freed one by one (their copies take as long as a tile) and waited for in
// groups (a wait costs the issuing warp more than a block's UMMAs take).
constexpr int kKBlocks = 9, kKGroups = 3;       // 64 columns of this CTA's 64 positions
constexpr int kVChunks = 8, kVGroups = 4;       // 16 positions, this CTA's 256 columns
constexpr int kKPer = kKBlocks / kKGroups, kVPer = kVChunks / kVGroups;
constexpr int kVWarp = kKWarp + kKBlocks, kEndWarp = kVWarp + kVChunks;
constexpr int kQWarps = 4;                      // kQWarp and those from kEndWarp on
constexpr int kThreads = 32 * 32;               // whole warpgroups
constexpr int kLowRegs = 56, kHighRegs = 88;    // 88 * 256 + 56 * 768 = 64 * 1024

constexpr int kQOff = 0, kQBlock = 64 * 128;    // 9 blocks of [64 rows x 64 columns]
constexpr int kKOff = kQOff + 9 * kQBlock, kKBlock = 64 * 128;
constexpr int kVOff = kKOff + kKBlocks * kKBlock, kVBlock = kTile * 128;  // 4 of [128 x 64 columns]
constexpr int kPOff = kVOff + 4 * kVBlock, kPBlock = 64 * 128;  // 2 of [64 rows x 64 positions]
constexpr int kBarOff = kPOff + 2 * kPBlock;
// q full, q empty, o free, done, p free, pv done; p full, s full, s free (2 each); k full, k empty;
// v full, v empty; rows full, rows empty (2 each); masks (4)
constexpr int kBars = 6 + 6 + kKGroups + kKBlocks + kVGroups + kVChunks + 4 + 4;
constexpr int kXchOff = kBarOff + 8 * kBars;    // a float per softmax thread: maxima, sums
constexpr int kRowOff = kXchOff + 4 * kSoftThreads;      // [2][128] rows of the cache
constexpr int kMaskOff = kRowOff + 2 * 4 * kTile;  // [4][4] words
constexpr int kScanOff = kMaskOff + 64;         // 32 x int64
constexpr int kSchedOff = kScanOff + 256;       // Start (40 bytes)
constexpr int kMiscOff = kSchedOff + 48;        // TMEM address, abort, the peer's TMEM address
constexpr int kSmemBytes = kMiscOff + 16;
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
static_assert(kThreads == 32 * (kEndWarp + kQWarps - 1), "every warp has a role");
static_assert(kVPer == 2 && kVGroups == 4, "descriptors of the second product");

constexpr uint32_t kSCol = 256;                 // TMEM columns: o 0..255, s 2 x 64
constexpr uint32_t kIdescS = idesc_bf16(128, 128);
constexpr uint32_t kIdescO = idesc_bf16(128, 256) | (1u << 16);  // B is MN-major
constexpr float kInf = __builtin_huge_valf();
constexpr float kLag = 8.0f;                    // how far a score may pass the reference (base 2)

constexpr int kMaxPairs = 76;
constexpr int kMinTiles = 1;                    // tiles of a pair at least
// What cutting costs a call, in tiles: partial sums written (2 us) and joined (8 us).  64 segments of
// 16 tiles on 76 pairs: 62 us cut into runs of 13 or 14 tiles, 47 us whole.
constexpr int kCutTiles = 6;
// What a run pays for holding the border of two segments, in tiles: a piece's partial sums written, the next
// one's queries and first rows (17 sequences of up to 3001 positions: runs of 4 tiles take 37000 clocks within
// a segment, 54000 across a border).  So pieces of one segment each, up to so many tiles longer than an equal
// run, go before runs across borders where the pairs suffice for them: 38 us without, 34 with.
constexpr int kTries = 4;
// A piece's partial sums: o as the epilogue's warps hold it, in blocks of 32 rows x 16 columns
// ([CTA][warp][8]), a block as [4][32 rows][4 columns], so that stores and the join's loads are whole
// lines; then m and l of the 128 rows.
constexpr int kBlockFloats = 32 * 16, kBlocks = kRows * kLatent / kBlockFloats;
constexpr int kPartFloats = kRows * (kLatent + 2);

struct Params {
    Paged cache;
    Sequences seq;
    const uint8_t* rows;
    const uint16_t* q;
    long long q_token, q_head;   // strides in elements
    int H, tt;                   // heads; tokens of a segment at most
    float scale;                 // times log2(e)
    const int32_t* inds;         // [T, k] or nullptr
    int k;
    uint16_t* out;               // [T, H, 512]
    float* lse;                  // [T, H] or nullptr
    float* part;                 // [2 pairs][kPartFloats]
    int4* meta;                  // [2 pairs] valid, token, tokens, last piece of its segment
    int pairs;
};

MOE_DEV void record_timeout(volatile int* abort) {
    *abort = 1;
    atomicCAS(&g_attention_status, 0u, kStatusTimeout);
}

// A segment: tokens t .. t + n - 1 of sequence b, which see up to `see` positions; `len` positions (or
// entries of its selection) in `tiles` tiles (one, all masked, where it sees nothing).
struct Seg {
    int t, n, b, see, len, tiles;
};
// `near`: the lengths of tokens from 0 on in shared memory, or nullptr.
MOE_DEV Seg segment(const Params& p, const Sequences& q, int t, int b, const volatile int32_t* near = nullptr) {
    Seg s;
    s.t = t;
    s.b = b;
    s.n = max(1, min(p.tt, seq_end(q, b) - t));
    s.see = 0;
    if (near)
        for (int i = 0; i < s.n; ++i) s.see = max(s.see, min(q.most, near[t + i]));
    else
        for (int i = 0; i < s.n; ++i) s.see = max(s.see, seq_length(q, t + i));
    s.len = p.inds ? min(s.see, p.k) : s.see;
    s.tiles = max(1, (s.len + kTile - 1) / kTile);
    return s;
}

// A pair's run: its first segment, the tile in it, and at most so many segments and tiles.
struct Start {
    Seg s;
    int tile, segments;
    long long left;
};

// The pieces of a pair's run, in order.
struct Walk {
    int t, b, tile, segments;
    long long left;
    Seg s;
    int i0, i1;  // tiles of the piece
    MOE_DEV Walk(const Start& st)
        : t(-1), b(0), tile(st.tile), segments(st.segments), left(st.left), s(st.s) {}
    MOE_DEV bool next(const Params& p) {
        if (left <= 0 || segments <= 0) return false;
        --segments;
        if (t >= 0) {  // (the first segment is at hand)
            if (t >= p.seq.T) return false;  // (ends of sequences that do not ascend)
            b = s.b;
            if (!p.seq.cu) b = t;
            else while (b < p.seq.B - 1 && t >= seq_end(p.seq, b)) ++b;
            s = segment(p, p.seq, t, b);
        }
        i0 = tile;
        i1 = (int)min((long long)s.tiles, i0 + left);
        left -= i1 - i0;
        tile = 0;
        t = s.t + s.n;
        return true;
    }
    MOE_DEV bool begins() const { return i0 == 0; }
    MOE_DEV bool ends() const { return i1 == s.tiles; }
};

// The entry e of a segment's list: a position, or what its selection holds; -1 behind its end.
MOE_DEV int entry(const Params& p, const Seg& s, int e) {
    if (e >= s.len) return -1;
    return p.inds ? __ldg(p.inds + (long long)s.t * p.k + e) : e;
}

// What the barriers hand over between the CTAs of a pair are operands that their writers have
// fenced for the asynchronous proxy and TMEM under the tcgen05 fences; no thread reads what
// another CTA's thread wrote with ordinary stores.  So arrivals and waits have the default scope
// (cluster scope on both, measured at 2048 tokens x 2048 selected: 2680 us against 2013).
MOE_DEV void arrive_even(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(mapa_shared(bar, 0)) : "memory");
}
// Every lane; false (in every lane) when a wait gave up.
MOE_DEV bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort) {
    if (__all_sync(0xFFFFFFFFu, mbar_wait_lean(bar, parity, abort))) return true;
    if ((threadIdx.x & 31) == 0) record_timeout(abort);
    return false;
}

// MN-major operand in the 128-byte swizzle: blocks of 64 columns kVBlock apart, groups of 8 rows
// (along K) 1024 bytes apart.
MOE_DEV uint64_t sdesc_mn128(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(kVBlock >> 4) << 16) |
           ((uint64_t)(1024u >> 4) << 32) | ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}

MOE_DEV float exp2_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What the sums are multiplied by: 1 / l, 0 without any position, NaN where all scores are -inf.
MOE_DEV float over(float l, float m) {
    return l == 0.0f ? 0.0f : m == -kInf ? __int_as_float(0x7FFFFFFF) : 1.0f / l;
}

// Barrier of the softmax threads: whether v holds for one of them.
MOE_DEV bool soft_any(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred a, b;\n\t"
        "setp.ne.b32 a, %1, 0;\n\t"
        "bar.red.or.pred b, 1, %2, a;\n\t"
        "selp.u32 %0, 1, 0, b;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "n"(kSoftThreads)
        : "memory");
    return r != 0;
}

// The lowest n bits.
MOE_DEV uint32_t low_bits(int n) { return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u; }

// Two bf16 numbers with infinities and NaN as 0.
MOE_DEV uint32_t finite2(uint32_t v) {
    if ((v & 0x7F80u) == 0x7F80u) v &= 0xFFFF0000u;
    if ((v & 0x7F800000u) == 0x7F800000u) v &= 0xFFFFu;
    return v;
}

// Tiles of the tokens a .. z - 1 (of those that begin a segment).
template <class F>
MOE_DEV void for_segments(const Params& p, const Sequences& q, const volatile int32_t* near, int a, int z, F&& f) {
    if (a >= z) return;
    int b = seq_of(q, a);
    for (int t = a; t < z; ++t) {
        if (!q.cu) b = t;
        else while (b < q.B - 1 && t >= seq_end(q, b)) ++b;
        const int first = q.cu ? q.cu[b] : t;
        if ((t - first) % p.tt == 0) f(segment(p, q, t, b, near));
    }
}

// FEW: there may be at most half as many segments as pairs (the code of their pieces alone costs the other
// calls 0.6 us of set-up: one token of 4096 positions 18.6 us without, 19.2 with).
template <bool FEW>
__global__ void __launch_bounds__(kThreads, 1) attention_kernel(const Params p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kBarOff);
    uint64_t *qfull = bars, *qempty = bars + 1, *ofree = bars + 2, *done = bars + 3;
    uint64_t *pfree = bars + 4, *pvdone = bars + 5, *pfull = bars + 6, *sfull = bars + 8, *sfree = bars + 10;
    uint64_t *kfull = bars + 12, *kempty = kfull + kKGroups;
    uint64_t *vfull = kempty + kKBlocks, *vempty = vfull + kVGroups;
    uint64_t *rfull = vempty + kVChunks, *rempty = rfull + 2, *mfull = rempty + 2;
    float* xch = reinterpret_cast<float*>(smem + kXchOff);
    volatile int32_t* rowat = reinterpret_cast<volatile int32_t*>(smem + kRowOff);
    volatile uint32_t* mask = reinterpret_cast<volatile uint32_t*>(smem + kMaskOff);
    unsigned long long* scan = reinterpret_cast<unsigned long long*>(smem + kScanOff);
    int* tops = reinterpret_cast<int*>(smem + kXchOff);  // (before the softmax needs it)
    Start* sched = reinterpret_cast<Start*>(smem + kSchedOff);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kMiscOff);
    volatile int* abort = reinterpret_cast<volatile int*>(smem + kMiscOff + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int crank = (int)cluster_rank(), pair = (int)(blockIdx.x >> 1);

    // ---- set-up ----
    // tiles, segments (from bit 40 on) and the longest segment of this thread's tokens; the sequences'
    // ends and the tokens' lengths are looked at in shared memory, where the first rows will be
    Sequences seq = p.seq;
    const volatile int32_t* near = nullptr;
    if (seq.cu && seq.B < 4 * kVBlock / 4) {
        int32_t* ends = reinterpret_cast<int32_t*>(smem + kVOff);
        const bool hold = FEW && seq.T <= kThreads;
        const int length = hold && (int)threadIdx.x < seq.T ? __ldg(p.seq.lengths + threadIdx.x) : 0;
        for (int i = threadIdx.x; i <= seq.B; i += kThreads) ends[i] = __ldg(p.seq.cu + i);
        seq.cu = ends;
        if (hold) {
            int32_t* lengths = reinterpret_cast<int32_t*>(smem + kKOff);
            lengths[threadIdx.x] = length;
            near = lengths;
        }
        __syncthreads();
    }
    const int tokens = seq_tokens(seq);
    const int per = (tokens + kThreads - 1) / kThreads;
    const int a = min(tokens, (int)threadIdx.x * per), z = min(tokens, a + per);
    unsigned long long mine = 0;
    int longest = 0;
    for_segments(p, seq, near, a, z, [&](const Seg& s) {
        mine += (unsigned)s.tiles + (1ull << 40);
        longest = max(longest, s.tiles);
    });
    if (threadIdx.x == 0) {
        // the barriers that the issuer waits on are the even CTA's, with arrivals from both
        mbar_init(qfull, 2 * kQWarps);
        mbar_init(qempty, 1);
        mbar_init(ofree, 2 * kSoftWarps);
        mbar_init(done, 2);
        mbar_init(pfree, 1);
        mbar_init(pvdone, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&pfull[i], kSoftWarps);  // half of the warps of both CTAs
            mbar_init(&sfull[i], 1);
            mbar_init(&sfree[i], 2 * kSoftWarps);
            mbar_init(&rfull[i], 1);
            mbar_init(&rempty[i], kKBlocks + kVChunks);
        }
        for (int i = 0; i < kKGroups; ++i) mbar_init(&kfull[i], 2 * kKPer);
        for (int i = 0; i < kVGroups; ++i) mbar_init(&vfull[i], 2 * kVPer);
        for (int i = 0; i < kKBlocks; ++i) mbar_init(&kempty[i], 1);
        for (int i = 0; i < kVChunks; ++i) mbar_init(&vempty[i], 1);
        for (int i = 0; i < 4; ++i) mbar_init(&mfull[i], 1);
        *abort = 0;
        sched->left = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) tmem_alloc_pair(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // the pair's UMMAs address the same columns in both CTAs: each tells the other its address
    if (threadIdx.x == 0)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(tmem_slot + 2, (uint32_t)(crank ^ 1))),
                     "r"(tmem)
                     : "memory");
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    // this pair's run of the list of tiles: a prefix sum over the tokens (tiles in the low 40 bits,
    // segments above) and the longest segment
    {
        constexpr unsigned long long kTiles = (1ull << 40) - 1;
        unsigned long long incl = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += v;
        }
        const int warp_longest = (int)__reduce_max_sync(0xFFFFFFFFu, (unsigned)longest);
        if (lane == 31) {
            scan[warp] = incl;
            tops[warp] = warp_longest;
        }
        __syncthreads();
        if (__any_sync(0xFFFFFFFFu, a < z)) {  // (a few tokens are one warp's)
            unsigned long long upto = scan[lane];
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned long long v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
                if (lane >= o) upto += v;
            }
            const unsigned top = __reduce_max_sync(0xFFFFFFFFu, (unsigned)tops[lane]);
            const unsigned long long all = __shfl_sync(0xFFFFFFFFu, upto, 31);
            const unsigned long long before =
                (warp ? __shfl_sync(0xFFFFFFFFu, upto, max(warp, 1) - 1) : 0) + incl - mine;
            const long long total = (long long)(all & kTiles);
            const unsigned segs = (unsigned)(all >> 40), pairs = (unsigned)p.pairs;
            // 32-bit divisions where they do (64-bit ones take a microsecond)
            const bool small = total < (1 << 24);
            const unsigned fair = small ? (unsigned)total / pairs : 0u;
            const unsigned whole_runs = min(segs, pairs);
            const unsigned longest_run = small ? (segs + pairs - 1) / pairs * top : 0xFFFFFFFFu;
            const bool whole = small && longest_run <= fair + kCutTiles &&
                               (segs <= pairs || (long long)top * segs == total);
            // pieces of one segment each, of up to fair + 1 .. fair + kTries tiles: how many each would give
            // (in 16 bits), and the shortest that the pairs suffice for
            int most = 0;
            if (FEW && !whole && segs > 1 && 2 * segs <= pairs && tokens <= kThreads && total < (1 << 16)) {
                int shift = 0;
                unsigned long long before2 = 0, pieces = 0;
                const unsigned tiles = (unsigned)(mine & kTiles);
                if (mine) {  // (a thread has one token)
#pragma unroll
                    for (int c = 0; c < kTries; ++c)
                        pieces += (unsigned long long)((tiles + fair + c) / (fair + 1 + c)) << (16 * c);
                }
                unsigned long long incl2 = pieces;
                for (int o = 1; o < 32; o <<= 1) {
                    const unsigned long long v = __shfl_up_sync(0xFFFFFFFFu, incl2, o);
                    if (lane >= o) incl2 += v;
                }
                unsigned long long all2 = __shfl_sync(0xFFFFFFFFu, incl2, 31);
                const int warps = (tokens + 31) / 32;  // that have tokens
                if (warps > 1) {
                    unsigned long long* scan2 = reinterpret_cast<unsigned long long*>(smem + kXchOff + 256);
                    if (lane == 31) scan2[warp] = incl2;
                    asm volatile("bar.sync 2, %0;" ::"r"(32 * warps) : "memory");
                    all2 = 0;
                    for (int i = 0; i < warps; ++i) {
                        if (i < warp) before2 += scan2[i];
                        all2 += scan2[i];
                    }
                }
                before2 += incl2 - pieces;
#pragma unroll
                for (int c = kTries - 1; c >= 0; --c)
                    if (((all2 >> (16 * c)) & 0xFFFFu) <= pairs) {
                        most = (int)fair + 1 + c;
                        shift = 16 * c;
                    }
                const int i = pair - (int)((before2 >> shift) & 0xFFFFu), n = (int)((pieces >> shift) & 0xFFFFu);
                if (most && mine && i >= 0 && i < n) {
                    for_segments(p, seq, near, a, z, [&](const Seg& s) { sched->s = s; });
                    sched->tile = (int)tiles * i / n;
                    sched->segments = 1;
                    sched->left = (int)tiles * (i + 1) / n - (int)tiles * i / n;
                }
            }
            long long lo = 0, hi = 0, mine0, mine1;
            if (whole) {
                if ((unsigned)pair < whole_runs) {
                    lo = segs * (unsigned)pair / whole_runs;
                    hi = segs * (unsigned)(pair + 1) / whole_runs;
                }
                mine0 = (long long)(before >> 40);
                mine1 = (long long)((before + mine) >> 40);
            } else {
                if (small) {
                    const unsigned runs = max(1u, min(pairs, (unsigned)total / kMinTiles));
                    if ((unsigned)pair < runs) {
                        lo = (unsigned)total * pair / runs;
                        hi = (unsigned)total * (pair + 1) / runs;
                    }
                } else {
                    lo = total * pair / pairs;
                    hi = total * (pair + 1) / pairs;
                }
                mine0 = (long long)(before & kTiles);
                mine1 = (long long)((before + mine) & kTiles);
            }
            if (!most && lo < hi && mine0 <= lo && lo < mine1) {
                long long at = mine0;
                for_segments(p, seq, near, a, z, [&](const Seg& s) {
                    const int n = whole ? 1 : s.tiles;
                    if (at <= lo && lo < at + n) {
                        sched->s = s;
                        sched->tile = (int)(lo - at);
                        sched->segments = whole ? (int)(hi - lo) : 0x7FFFFFFF;
                        sched->left = whole ? 0x7FFFFFFFFFFFll : hi - lo;
                    }
                    at += n;
                });
            }
        }
    }
    __syncthreads();
    // the peer's barriers are initialised and its TMEM allocated
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    Start st = *sched;
    if (tmem_slot[2] != tmem) {
        st.left = 0;
        if (threadIdx.x == 0) atomicCAS(&g_attention_status, 0u, kStatusPairTmem);
    }
    Walk w(st);
    uint32_t g = 0;  // tiles so far
    bool ok = true;

    if (warp >= kSoftWarps) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLowRegs));
    if (warp >= kKWarp && warp < kVWarp) {
        // ============== rows as keys: 64 columns of this CTA's 64 positions ==============
        const int j = warp - kKWarp, sub = lane >> 3, ch = lane & 7;
        const uint32_t dst = smem_u32(smem + kKOff + j * kKBlock) + sub * 128;
        const uint8_t* src = p.rows + j * 128 + ch * 16;
        while (ok && w.next(p)) {
            for (int i = w.i0; i < w.i1; ++i, ++g) {
                if (!(ok = wait_all(&rfull[g & 1u], (g >> 1) & 1u, abort))) break;
                const volatile int32_t* rows = rowat + (g & 1u) * kTile + crank * 64;
                const int32_t own0 = rows[lane], own1 = rows[32 + lane];
                __syncwarp();
                if (lane == 0) mbar_arrive(&rempty[g & 1u]);
                if (!(ok = wait_all(&kempty[j], (g & 1u) ^ 1u, abort))) break;
#pragma unroll
                for (int h = 0; h < 16; ++h) {
                    const int32_t at = __shfl_sync(0xFFFFFFFFu, h < 8 ? own0 : own1, (4 * h + sub) & 31);
                    copy16(dst + h * 512 + ((ch ^ ((4 * h + sub) & 7)) << 4),
                           src + (long long)max(at, 0) * kRowBytes, at < 0 ? 0u : 16u);
                }
                copy_commit();
                copy_wait<0>();
                fence_async_shared();
                __syncwarp();
                if (lane == 0) arrive_even(&kfull[j / kKPer]);
            }
        }
    } else if (warp >= kVWarp && warp < kEndWarp) {
        // ============ rows as values: 16 positions, half of the 512 columns ============
        const int c = warp - kVWarp, blk = lane >> 3, ch = lane & 7;
        // block 0, 1: this CTA's 128 columns of the first 256; 2, 3: of the last 256
        const int col = (blk >> 1) * 256 + crank * 128 + (blk & 1) * 64;
        const uint32_t dst = smem_u32(smem + kVOff) + blk * kVBlock + c * 2048;
        const uint8_t* src = p.rows + col * 2 + ch * 16;
        while (ok && w.next(p)) {
            // a row that not every token of the segment sees meets zeros of p; an infinity or a
            // NaN in it must not
            int fewest = 0x7FFFFFFF;
            if (w.s.n > 1)
                for (int i = 0; i < w.s.n; ++i) fewest = min(fewest, seq_length(p.seq, w.s.t + i));
            for (int i = w.i0; i < w.i1; ++i, ++g) {
                if (!(ok = wait_all(&rfull[g & 1u], (g >> 1) & 1u, abort))) break;
                const int32_t own = rowat[(g & 1u) * kTile + 16 * c + (lane & 15)];
                __syncwarp();
                if (lane == 0) mbar_arrive(&rempty[g & 1u]);
                if (!(ok = wait_all(&vempty[c], (g & 1u) ^ 1u, abort))) break;
                const int first = i * kTile + 16 * c;
                if (first + 15 < fewest || first >= w.s.len) {
#pragma unroll
                    for (int rr = 0; rr < 16; ++rr) {
                        const int32_t at = __shfl_sync(0xFFFFFFFFu, own, rr);
                        copy16(dst + rr * 128 + ((ch ^ (rr & 7)) << 4),
                               src + (long long)max(at, 0) * kRowBytes, at < 0 ? 0u : 16u);
                    }
                    copy_commit();
                    copy_wait<0>();
                } else {
#pragma unroll 4
                    for (int rr = 0; rr < 16; ++rr) {
                        const int32_t at = __shfl_sync(0xFFFFFFFFu, own, rr);
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (at >= 0) v = __ldg(reinterpret_cast<const uint4*>(src + (long long)at * kRowBytes));
                        if (first + rr >= fewest)
                            v = make_uint4(finite2(v.x), finite2(v.y), finite2(v.z), finite2(v.w));
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         dst + rr * 128 + ((ch ^ (rr & 7)) << 4)),
                                     "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                                     : "memory");
                    }
                }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) arrive_even(&vfull[c / kVPer]);
            }
        }
    } else if (warp == kFindWarp) {
        // ====================== the rows of the tiles ahead, and which are there ======================
        // Three tiles are under way: entries asked for, pages asked for, rows handed on.  A load
        // waits behind the copies for as long as a tile takes (one tile at a time, with its two
        // loads one after the other: 2048 x 2048 selected 1353 us).
        bool more = w.next(p), asked = false, paged = false;
        int i = w.i0, e[4], b = 0, see = 0, id[4], off[4];
        while (more || asked || paged) {
            const bool ask = more;
            int e2[4], b2 = 0, see2 = 0, id2[4], off2[4];
            if (ask) {
#pragma unroll
                for (int c = 0; c < 4; ++c) e2[c] = entry(p, w.s, i * kTile + 32 * c + lane);
                b2 = w.s.b;
                see2 = w.s.see;
            }
            if (asked) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const unsigned at = (unsigned)e[c] / (unsigned)p.cache.page;
                    off2[c] = e[c] - (int)(at * (unsigned)p.cache.page);
                    id2[c] = e[c] >= 0 && e[c] < see
                                 ? __ldg(p.cache.table + (long long)b * p.cache.width + at) : -1;
                }
            }
            if (paged) {
                int32_t row[4];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    row[c] = (unsigned)id[c] < (unsigned long long)p.cache.pages ? id[c] * p.cache.page + off[c] : -1;
                // this CTA's 64 rows on their way to L2: they are copied a tile or two later (line by
                // line: a bulk prefetch of a row takes its lane 90 clocks).  Not the rows that a
                // prompt's tokens select: they are there from its other tokens (2048 x 2048
                // 909 us with, 881 without; 64 sequences' 2048 of 16384 46 with, 48 without)
                const bool fetch = !p.inds || !p.seq.cu;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int32_t at = crank ? row[2 + c] : row[c];
                    const uint8_t* r = p.rows + (long long)at * kRowBytes;
                    if (fetch && at >= 0)
#pragma unroll
                        for (int k = 0; k < kRowBytes; k += 128)
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(r + k) : "memory");
                }
                if (!wait_all(&rempty[g & 1u], ((g >> 1) & 1u) ^ 1u, abort)) { ok = false; break; }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    rowat[(g & 1u) * kTile + 32 * c + lane] = row[c];
                    const uint32_t there = __ballot_sync(0xFFFFFFFFu, row[c] >= 0);
                    // (its last reader was the softmax of four tiles ago: the copies that have read
                    // the rows of two tiles ago had waited for the second product of four tiles ago)
                    if (lane == 0) mask[(g & 3u) * 4 + c] = there;
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&rfull[g & 1u]);
                    mbar_arrive(&mfull[g & 3u]);
                }
                ++g;
            }
            if (ask && ++i == w.i1) {
                more = w.next(p);
                i = w.i0;
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                e[c] = e2[c];
                id[c] = id2[c];
                off[c] = off2[c];
            }
            b = b2;
            see = see2;
            paged = asked;
            asked = ask;
        }
    } else if (warp == kQWarp || warp >= kEndWarp) {
        // ================================== queries ==================================
        const int r0 = 16 * (warp == kQWarp ? 0 : warp - kEndWarp + 1);  // of the CTA's 64 rows
        const int sub = lane >> 3, ch = lane & 7;
        const uint32_t dst = smem_u32(smem + kQOff) + (r0 + sub) * 128;
        const auto row_of = [&](const Seg& q, int gr) {
            return p.q + (q.t + gr / p.H) * p.q_token + (gr % p.H) * p.q_head;
        };
        bool more = w.next(p);
        for (uint32_t n = 0; more; ++n) {
            const Seg q = w.s;
            more = w.next(p);
            if (!(ok = wait_all(qempty, (n & 1u) ^ 1u, abort))) break;
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                const int gr = crank * 64 + r0 + r + sub;
                const bool live = gr < q.n * p.H;
                const uint16_t* src = live ? row_of(q, gr) : p.q;
#pragma unroll
                for (int j = 0; j < 9; ++j)
                    copy16(dst + r * 128 + ((ch ^ ((r + sub) & 7)) << 4) + j * kQBlock, src + j * 64 + ch * 8,
                           live ? 16u : 0u);
            }
            copy_commit();
            copy_wait<0>();
            fence_async_shared();
            __syncwarp();
            if (lane == 0) arrive_even(qfull);
            // the next piece's on their way to L2
            if (more)
                for (int i = lane; i < 16 * 9; i += 32) {
                    const int gr = crank * 64 + r0 + i / 9;
                    if (gr < w.s.n * p.H)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(row_of(w.s, gr) + i % 9 * 64) : "memory");
                }
        }
    } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
        // ================================ UMMA issuers ================================
        // (the next block's barrier is looked at before a block is issued: a look takes 90 clocks)
        if (crank == 0) {
            if (warp == kMmaWarp) {
                const uint64_t dq = sdesc_k128(smem_u32(smem + kQOff)), dk = sdesc_k128(smem_u32(smem + kKOff));
                for (uint32_t n = 0; ok && w.next(p); ++n) {
                    ok = wait_all(qfull, n & 1u, abort);
                    for (int i = w.i0; ok && i < w.i1; ++i, ++g) {
                        const uint32_t b = g & 1u;
                        bool here = mbar_test(&kfull[0], g & 1u);
                        if (!(ok = wait_all(&sfree[b], ((g >> 1) & 1u) ^ 1u, abort))) break;
#pragma unroll 1
                        for (int j = 0; j < kKGroups; ++j) {
                            if (!__all_sync(0xFFFFFFFFu, here) && !(ok = wait_all(&kfull[j], g & 1u, abort))) break;
                            if (j + 1 < kKGroups) here = mbar_test(&kfull[j + 1], g & 1u);
                            tc_fence_after();
                            const uint64_t da = dq + (uint64_t)(j * kKPer * (kQBlock / 16));
                            const uint64_t db = dk + (uint64_t)(j * kKPer * (kKBlock / 16));
                            if (elect_lane()) {
#pragma unroll
                                for (int c = 0; c < kKPer; ++c) {
#pragma unroll
                                    for (int k = 0; k < 4; ++k)
                                        umma_bf16_pair(tmem + kSCol + 64 * b,
                                                       da + (uint64_t)(c * (kQBlock / 16) + 2 * k),
                                                       db + (uint64_t)(c * (kKBlock / 16) + 2 * k), kIdescS,
                                                       j + c + k > 0);
                                    umma_commit_pair(&kempty[j * kKPer + c], 3);
                                }
                                if (j == kKGroups - 1) {
                                    umma_commit_pair(&sfull[b], 3);
                                    if (i == w.i1 - 1) umma_commit_pair(qempty, 3);
                                }
                            }
                            __syncwarp();
                        }
                    }
                }
            } else {
                const uint64_t dp = sdesc_k128(smem_u32(smem + kPOff)), dv = sdesc_mn128(smem_u32(smem + kVOff));
                for (uint32_t n = 0; ok && w.next(p); ++n) {
                    for (int i = w.i0; ok && i < w.i1; ++i, ++g) {
                        const bool first = i == w.i0;
                        if (first && !(ok = wait_all(ofree, (n & 1u) ^ 1u, abort))) break;
                        bool here = mbar_test(&vfull[0], g & 1u);
                        if (!(ok = wait_all(&pfull[0], g & 1u, abort))) break;
#pragma unroll 1
                        for (int j = 0; j < kVGroups; ++j) {
                            if (!__all_sync(0xFFFFFFFFu, here) && !(ok = wait_all(&vfull[j], g & 1u, abort))) break;
                            if (j + 1 < kVGroups) here = mbar_test(&vfull[j + 1], g & 1u);
                            if (j == kVGroups / 2 && !(ok = wait_all(&pfull[1], g & 1u, abort))) break;
                            tc_fence_after();
                            // 32 positions: half a block of p's columns, 4096 bytes of rows
                            const uint64_t da = dp + (uint64_t)((j >> 1) * (kPBlock / 16) + 4 * (j & 1));
                            const uint64_t db = dv + (uint64_t)(j * (kVPer * 2048 / 16));
                            if (elect_lane()) {
#pragma unroll
                                for (int c = 0; c < kVPer; ++c) {
#pragma unroll
                                    for (int half = 0; half < 2; ++half)
                                        umma_bf16_pair(tmem + 128 * half, da + (uint64_t)(2 * c),
                                                       db + (uint64_t)(half * 2 * (kVBlock / 16) + c * (2048 / 16)),
                                                       kIdescO, !first || j + c > 0);
                                    umma_commit_pair(&vempty[j * kVPer + c], 3);
                                }
                                if (j == kVGroups / 2 - 1) umma_commit_pair(pfree, 3);
                                if (j == kVGroups - 1) umma_commit_pair(pvdone, 3);
                            }
                            __syncwarp();
                        }
                    }
                }
            }
            if (elect_lane()) umma_commit_pair(done, 1);  // no UMMA is left when the pair frees its TMEM
            __syncwarp();
            mbar_wait(done, 0u, nullptr, 100000000ull);
        }
    } else if (warp < kSoftWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kHighRegs));
        // ======================= softmax, rescaling and epilogue =======================
        // thread: row, half of the tile's positions (TMEM lane >= 64), half of those (set)
        const int L = (int)threadIdx.x, set = warp >> 2, lane128 = L & 127;
        const int row = lane128 & 63, half = lane128 >> 6;
        const int gr = crank * 64 + row;
        const uint32_t lane0 = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        uint64_t* pgone = half ? pvdone : pfree;  // the last tile's p of this half has been read
        if (crank == 0 && L == 0) p.meta[2 * pair] = p.meta[2 * pair + 1] = make_int4(0, 0, 0, 0);
        const auto of_row = [&](float v, auto&& f) {  // f over the row's four threads
            return f(f(v, xch[L ^ 64]), f(xch[L ^ 128], xch[L ^ 192]));
        };
        for (; ok && w.next(p);) {
            const bool live = gr < w.s.n * p.H;
            const int tok = w.s.t + gr / p.H, head = gr % p.H;
            const int see = !live ? 0 : p.inds ? w.s.len : seq_length(p.seq, tok);
            float m = -kInf, l = 0.0f;
            uint32_t seen = 0;  // whether there was any position
            for (int i = w.i0; i < w.i1; ++i, ++g) {
                const uint32_t b = g & 1u;
                // (a warp whose wait gave up keeps to the softmax barriers until all know)
                ok = ok && wait_all(&mfull[g & 3u], (g >> 2) & 1u, abort) &&
                     wait_all(&sfull[b], (g >> 1) & 1u, abort);
                tc_fence_after();
                float x[32];
                {
                    uint32_t v[32];
                    tmem_ld32(lane0 + kSCol + 64 * b + 32 * set, v);
                    tmem_ready(v);
#pragma unroll
                    for (int c = 0; c < 32; ++c) x[c] = __uint_as_float(v[c]) * p.scale;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && ok) arrive_even(&sfree[b]);
                const uint32_t bits = mask[(g & 3u) * 4 + 2 * half + set] &
                                      low_bits(see - i * kTile - half * 64 - set * 32);
                seen |= bits;
                if (!__all_sync(0xFFFFFFFFu, bits == 0xFFFFFFFFu)) {
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (!((bits >> c) & 1u)) x[c] = -kInf;
                }
                float mx = fmaxf(x[0], x[1]);
#pragma unroll
                for (int c = 2; c < 32; ++c) mx = fmaxf(mx, x[c]);
                if (soft_any(!ok || mx > m + kLag)) {
                    xch[L] = mx;
                    if (soft_any(!ok)) { ok = false; break; }
                    mx = of_row(mx, [](float u, float v) { return fmaxf(u, v); });
                    const float to = mx > m + kLag ? mx : m;
                    const float f = to == m ? 1.0f : exp2_of(m - to);
                    m = to;
                    l *= f;
                    if (i > w.i0) {
                        // o of the tiles so far; the next product waits for this tile's p
                        ok = wait_all(pvdone, (g & 1u) ^ 1u, abort);
                        if (__any_sync(0xFFFFFFFFu, f != 1.0f)) {
                            tc_fence_after();
#pragma unroll 1
                            for (uint32_t c = 128 * set; c < 128u * set + 128u; c += 16) {
                                uint32_t o[16];
                                tmem_ld16(lane0 + c, o);
                                tmem_ready(o);
#pragma unroll
                                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                                tmem_st16(lane0 + c, o);
                            }
                            tmem_st_wait();
                            tc_fence_before();
                        }
                    }
                    // (nor may a warp hand over its p, or write its sum there, before the others are done)
                    if (soft_any(!ok)) { ok = false; break; }
                }
                const float ref = m == -kInf ? 0.0f : m;
                uint32_t pk[16];
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                    const float p0 = exp2_of(x[c] - ref), p1 = exp2_of(x[c + 1] - ref);
                    l += p0 + p1;
                    pk[c / 2] = pack_bf16x2(p0, p1);
                }
                ok = ok && wait_all(pgone, (g & 1u) ^ 1u, abort);
                const uint32_t dst = smem_u32(smem + kPOff + half * kPBlock) + row * 128;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                     dst + (((4 * set + c) ^ (row & 7)) << 4)),
                                 "r"(pk[4 * c]), "r"(pk[4 * c + 1]), "r"(pk[4 * c + 2]), "r"(pk[4 * c + 3])
                                 : "memory");
                fence_async_shared();
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && ok) arrive_even(&pfull[half]);
            }
            ok = ok && wait_all(pvdone, (g - 1) & 1u, abort);
            // scores that are all -inf are told from no positions by their sum, 0 otherwise
            if (m == -kInf && seen) l += 1.0f;
            xch[L] = l;
            if (soft_any(!ok)) { ok = false; break; }
            l = of_row(l, [](float u, float v) { return u + v; });
            tc_fence_after();
            const bool whole = w.begins() && w.ends();
            const int slot = 2 * pair + (w.begins() ? 1 : 0);
            float* part = p.part + (long long)slot * kPartFloats;
            const float f = whole ? over(l, m) : 1.0f;
            if (live && half == 0 && set == 0) {
                if (whole) {
                    if (p.lse)
                        p.lse[(long long)tok * p.H + head] =
                            l == 0.0f ? -kInf : (m + log2f(l)) * 0.693147180559945f;
                } else {
                    part[kRows * kLatent + gr] = m;
                    part[kRows * kLatent + kRows + gr] = l;
                }
            }
            if (crank == 0 && L == 0 && !whole)
                p.meta[slot] = make_int4(1, w.s.t, w.s.n, w.ends() ? 1 : 0);
            // 32 rows of 64 bytes at a time through this warp's part of p's place (its last reader is
            // done, its next writers are these warps), so that a store has 64 consecutive bytes of 8
            // rows: a row per lane takes the stores four times as long
            const uint32_t stage = smem_u32(smem + kPOff) + warp * 2048;
            const int col0 = set * 256 + half * 128;
            const int first = crank * 64 + (warp & 1) * 32;  // of the warp's rows
            const int rows = w.s.n * p.H;
            const long long out0 = (long long)w.s.t * p.H;
            const auto put = [&](const uint32_t (&v)[16], int col) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                     stage + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)),
                                 "r"(v[4 * k]), "r"(v[4 * k + 1]), "r"(v[4 * k + 2]), "r"(v[4 * k + 3])
                                 : "memory");
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = 8 * k + (lane >> 2);
                    uint4 q;
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                                 : "r"(stage + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4))
                                 : "memory");
                    if (first + r < rows)
                        *reinterpret_cast<uint4*>(p.out + (out0 + first + r) * kLatent + col + (lane & 3) * 8) = q;
                }
                __syncwarp();
            };
            if (whole) {
#pragma unroll 1
                for (int c = 0; c < 128; c += 32) {
                    uint32_t o[32], v[16];
                    tmem_ld32(lane0 + (uint32_t)(128 * set + c), o);
                    tmem_ready(o);
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        v[k] = pack_bf16x2(__uint_as_float(o[2 * k]) * f, __uint_as_float(o[2 * k + 1]) * f);
                    put(v, col0 + c);
                }
            } else {
                uint4* at = reinterpret_cast<uint4*>(part + (crank * kSoftWarps + warp) * 8 * kBlockFloats) + lane;
#pragma unroll 2
                for (int c = 0; c < 128; c += 16) {
                    uint32_t o[16];
                    tmem_ld16(lane0 + (uint32_t)(128 * set + c), o);
                    tmem_ready(o);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        at[c * 8 + 32 * k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_even(ofree);
        }
    }

    pdl_launch_dependents();
    tc_fence_before();
    __syncthreads();
    // neither CTA leaves while the other's UMMAs or arrivals may still touch its memory
    cluster_sync();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// Joins the pieces of the blockIdx.y-th segment that was cut apart: its first piece is the second
// slot of some pair, the others the first slots of the pairs behind it.  A lane has a row of a block.
// SPLIT 1: a warp takes a block and all its pieces, in their order.  SPLIT 8: eight warps share the
// pieces of one block (warp w: w, w + 8, ..) and join their sums in the order of the warps; for
// the few tokens whose pieces are many (one token of 4096 positions: 30 us with SPLIT 1, 19 with 8).
constexpr int kJoinWarps = 4;
constexpr int kJoinFew = 8;  // tokens up to which SPLIT is 8
template <int SPLIT>
__global__ void __launch_bounds__(SPLIT == 1 ? 32 * kJoinWarps : 32 * SPLIT) join_kernel(const Params p) {
    __shared__ float held[SPLIT == 1 ? 1 : SPLIT][18][32];
    pdl_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int want = (int)blockIdx.y, owner = -1;
    for (int q = 0; q < p.pairs && owner < 0; q += 32) {
        const bool cut = q + lane < p.pairs && p.meta[2 * (q + lane) + 1].x != 0;
        uint32_t any = __ballot_sync(0xFFFFFFFFu, cut);
        const int cnt = __popc(any);
        if (want >= cnt) { want -= cnt; continue; }
        while (want-- > 0) any &= any - 1;
        owner = q + __ffs(any) - 1;
    }
    if (owner < 0) return;
    const int4 first = p.meta[2 * owner + 1];
    const int blk = SPLIT == 1 ? (int)blockIdx.x * kJoinWarps + w : (int)blockIdx.x;
    const int warp = (blk >> 3) & (kSoftWarps - 1), quarter = warp & 3;
    const int row = (blk >> 6) * 64 + (quarter & 1) * 32 + lane;
    const int col = (warp >> 2) * 256 + (quarter >> 1) * 128 + (blk & 7) * 16;
    // the pieces behind the first: up to the one that ends the segment
    int pieces = 0;
    for (int q = 1; owner + q < p.pairs && !pieces; q += 32) {
        const bool in = owner + q + lane < p.pairs;
        const int4 m = in ? p.meta[2 * (owner + q + lane)] : make_int4(0, 0, 0, 0);
        const uint32_t last = __ballot_sync(0xFFFFFFFFu, m.x && m.w);
        const uint32_t gone = __ballot_sync(0xFFFFFFFFu, !m.x);
        const int e = last ? __ffs(last) - 1 : 32;
        if (gone & low_bits(e)) return;  // (a pair gave up)
        if (last) pieces = q + e + 1;
    }
    if (!pieces || row - lane >= first.z * p.H) return;
    const float* const p0 = p.part + (long long)(2 * owner + 1) * kPartFloats;
    const float* const p1 = p.part + (long long)(2 * owner) * kPartFloats;  // + 2 i pieces for i > 0
    const auto at = [&](int i) { return i == 0 ? p0 : p1 + (long long)(2 * i) * kPartFloats; };
    // (one pass with a running maximum, so that all of a piece's loads go out at once)
    float m = -kInf, l = 0.0f, acc[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) acc[c] = 0.0f;
#pragma unroll 4
    for (int i = SPLIT == 1 ? 0 : w; i < pieces; i += SPLIT) {
        const float* const a = at(i);
        const float mi = a[kRows * kLatent + row], li = a[kRows * kLatent + kRows + row];
        const float4* o = reinterpret_cast<const float4*>(a + blk * kBlockFloats) + lane;
        const float to = fmaxf(m, mi);
        const float f = mi == to ? 1.0f : exp2_of(mi - to);
        const float g = m == to ? 1.0f : exp2_of(m - to);
        m = to;
        l = fmaf(f, li, l * g);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 v = o[32 * k];
            acc[4 * k] = fmaf(f, v.x, acc[4 * k] * g);
            acc[4 * k + 1] = fmaf(f, v.y, acc[4 * k + 1] * g);
            acc[4 * k + 2] = fmaf(f, v.z, acc[4 * k + 2] * g);
            acc[4 * k + 3] = fmaf(f, v.w, acc[4 * k + 3] * g);
        }
    }
    if constexpr (SPLIT > 1) {
#pragma unroll
        for (int c = 0; c < 16; ++c) held[w][c][lane] = acc[c];
        held[w][16][lane] = m;
        held[w][17][lane] = l;
        __syncthreads();
        if (w) return;
        for (int k = 0; k < SPLIT; ++k) m = fmaxf(m, held[k][16][lane]);
        l = 0.0f;
#pragma unroll
        for (int c = 0; c < 16; ++c) acc[c] = 0.0f;
        for (int k = 0; k < SPLIT; ++k) {
            const float mi = held[k][16][lane];
            const float f = mi == m ? 1.0f : exp2_of(mi - m);
            l = fmaf(f, held[k][17][lane], l);
#pragma unroll
            for (int c = 0; c < 16; ++c) acc[c] = fmaf(f, held[k][c][lane], acc[c]);
        }
    }
    if (row >= first.z * p.H) return;
    const float f = over(l, m);
    const long long o = (long long)first.y * p.H + row;
    uint32_t r[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) r[c] = pack_bf16x2(acc[2 * c] * f, acc[2 * c + 1] * f);
    uint4* d = reinterpret_cast<uint4*>(p.out + o * kLatent + col);
    d[0] = make_uint4(r[0], r[1], r[2], r[3]);
    d[1] = make_uint4(r[4], r[5], r[6], r[7]);
    if (p.lse && col == 0) p.lse[o] = l == 0.0f ? -kInf : (m + log2f(l)) * 0.693147180559945f;
}

}  // namespace

int attention_pairs(long long T, long long entries) {
    const long long tiles = T * ((entries + kTile - 1) / kTile > 0 ? (entries + kTile - 1) / kTile : 1);
    const long long runs = tiles / kMinTiles;
    return (int)(runs < 1 ? 1 : runs > kMaxPairs ? kMaxPairs : runs);
}
size_t attention_ws_bytes(int pairs) {
    return (size_t)pairs * 2 * (kPartFloats * sizeof(float) + sizeof(int4));
}

namespace {

Params params_of(const AttentionArgs& a, int pairs) {
    const long long room = (long long)a.width * a.page;
    Params p = {};
    p.cache = {a.table, a.width, a.page, a.pages};
    p.seq = {a.cu, a.lengths, a.B, (int)a.T, (int)room};
    p.rows = static_cast<const uint8_t*>(a.rows);
    p.q = static_cast<const uint16_t*>(a.q);
    p.q_token = a.q_token;
    p.q_head = a.q_head;
    p.H = a.H;
    p.tt = a.inds || !a.cu ? 1 : kRows / a.H;
    p.scale = a.scale * 1.44269504088896f;
    p.inds = a.inds;
    p.k = a.k;
    p.out = static_cast<uint16_t*>(a.out);
    p.lse = a.lse;
    p.pairs = pairs;
    p.part = static_cast<float*>(a.ws);
    p.meta = reinterpret_cast<int4*>(p.part + (size_t)pairs * 2 * kPartFloats);
    return p;
}

}  // namespace

cudaError_t attention_plan(AttentionArgs& a) {
    static DeviceOnce once;
    static int resident[DeviceOnce::kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= DeviceOnce::kMaxDevices) return cudaErrorInvalidDevice;
    e = once.run([&] {
        cudaError_t err = cudaSuccess;
        for (auto kernel : {attention_kernel<false>, attention_kernel<true>})
            if (err == cudaSuccess)
                err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
        if (err != cudaSuccess) return err;
        // as many pairs as the device can hold at once (an SM left over in a GPC takes none)
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * kMaxPairs);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmemBytes;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        err = cudaOccupancyMaxActiveClusters(&n, attention_kernel<true>, &cfg);
        if (err == cudaSuccess) resident[dev] = n > 0 ? n : 1;
        return err;
    });
    if (e != cudaSuccess) return e;
    a.pairs = attention_pairs(a.T, a.inds ? a.k : (long long)a.width * a.page);
    if (resident[dev] < a.pairs) a.pairs = resident[dev];
    return cudaSuccess;
}

cudaError_t launch_attention(const AttentionArgs& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * a.pairs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // (of several tokens a segment may hold some, so there may be as few segments as sequences)
    const bool few = a.T > 1 && 2 * (a.inds || !a.cu ? a.T : (long long)a.B) <= a.pairs;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, few ? attention_kernel<true> : attention_kernel<false>,
                                             params_of(a, a.pairs));
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_attention_join(const AttentionArgs& a, cudaStream_t s) {
    const long long cut = a.T < a.pairs - 1 ? a.T : a.pairs - 1;  // segments that may be cut apart
    if (a.T <= kJoinFew)
        return launch_kernel(join_kernel<8>, dim3((unsigned)kBlocks, (unsigned)cut), dim3(32 * 8), 0, s,
                             params_of(a, a.pairs));
    return launch_kernel(join_kernel<1>, dim3((unsigned)(kBlocks / kJoinWarps), (unsigned)cut),
                         dim3(32 * kJoinWarps), 0, s, params_of(a, a.pairs));
}

cudaError_t read_attention_status(unsigned int* out, int clear, cudaStream_t s) {
    cudaError_t err = cudaMemcpyFromSymbolAsync(out, g_attention_status, sizeof(unsigned int), 0,
                                                cudaMemcpyDeviceToHost, s);
    if (err != cudaSuccess) return err;
    err = cudaStreamSynchronize(s);
    if (err != cudaSuccess || !clear) return err;
    const unsigned int zero = 0;
    err = cudaMemcpyToSymbolAsync(g_attention_status, &zero, sizeof(unsigned int), 0,
                                  cudaMemcpyHostToDevice, s);
    if (err != cudaSuccess) return err;
    return cudaStreamSynchronize(s);
}

}  // namespace moe

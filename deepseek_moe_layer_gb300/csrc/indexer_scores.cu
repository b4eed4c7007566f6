// indexer_scores.cu -- the indexer's scores of the cached positions on the 5th-generation tensor
// cores:
//     out[t, j] = ks_j * sum_h w[t, h] * max(q[t, h] . k_j, 0)    j < lengths[t], else -inf
// with index keys k_j of 128 columns in a paged cache, bf16 or e4m3 (ks_j: a scale per key).
//
// Keys lie on the tensor cores' M side (128 per tile) and (token, head) pairs on the N side: a
// thread then holds one key's dot products with all heads, the sum over the heads is its own
// and a token's scores leave as consecutive numbers.  A unit is `tt` consecutive tokens (up to 512
// columns, of bf16 384, in shared memory for the whole unit) and `kc` key tiles that stream past them; tokens
// of several sequences in one unit are taken sequence by sequence, with the columns of that
// sequence's tokens only.  Columns run in groups of up to 128 (whole tokens) through four TMEM
// accumulators of four warps each, so that the epilogue (a maximum and half a packed
// multiply-add per product) runs beside the UMMAs of the groups ahead and four of its warps share
// a scheduler (4096 x 16384 in 770 us; 1288 with two and 32 columns loaded ahead, 1016 with four and
// 16 ahead, 955 with eight accumulators of 64 columns).
//
// Warp roles (768 threads, one CTA per SM, persistent over units): warps 0..15 epilogue (warp % 4 =
// TMEM lane quarter, warp / 4 = accumulator), 16..19 key copies (16-byte asynchronous copies, so that
// pages of any size and any order do; rows without a page or behind the end are zeros; a warp takes
// every fourth tile, so that four are in flight, and looks its next one's pages up meanwhile), 20 and 21 issue the UMMAs of
// every other accumulator (an issuer's waits and commits take as long as the UMMAs), 22 and 23
// queries and weights.  Every
// wait is bounded.
#include <mutex>

#include "launch.h"
#include "paged.cuh"

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
    static constexpr int kCols = F8 ? 512 : 384;            // (token, head) columns of a unit
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
    static constexpr int kLenOff = kWOff + 4 * kCols;       // a unit's lengths
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
    int tt, kc;              // tokens of a unit, key tiles of a unit
    int tiles;               // key tiles of n
    long long units;
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

// The part of a unit that belongs to one sequence: tokens t0 .. t1 - 1 of sequence b, key tiles
// c0 .. c1 - 1 hold positions that one of them may see.
struct Part {
    int b, t0, t1, c0, c1;
};
// Walks a unit's parts; every thread that walks sees the same ones.
struct Unit {
    int u0, u1, c0, c1, next;
    MOE_DEV Unit(const Params& p, long long u, int tokens) {
        const int chunks = (p.tiles + p.kc - 1) / p.kc;
        u0 = (int)(u / chunks) * p.tt;
        u1 = min(tokens, u0 + p.tt);
        c0 = (int)(u % chunks) * p.kc;
        c1 = min(p.tiles, c0 + p.kc);
        next = u0;
    }
    MOE_DEV bool part(const Params& p, Part& r) {
        if (next >= u1) return false;
        r.t0 = next;
        r.b = seq_of(p.seq, next);
        r.t1 = max(next + 1, min(u1, seq_end(p.seq, r.b)));
        next = r.t1;
        int most = 0;
        for (int t = r.t0; t < r.t1; ++t) most = max(most, seq_length(p.seq, t));
        r.c0 = c0;
        r.c1 = max(c0, min(c1, (min(most, p.n) + kKeys - 1) / kKeys));
        return true;
    }
};

// The key tiles of a CTA's units, in order.
struct Tiles {
    long long u;
    int tokens, c;
    bool more;
    Unit un;
    Part r;
    MOE_DEV Tiles(const Params& p, int tokens) : u(blockIdx.x), tokens(tokens), un(p, blockIdx.x, tokens) {
        r.c0 = r.c1 = 0;
        c = 0;
        more = u < p.units;
        step(p);
    }
    MOE_DEV void step(const Params& p) {  // to a tile, or to the end
        while (more && c >= r.c1) {
            if (un.part(p, r)) {
                c = r.c0;
            } else {
                u += gridDim.x;
                more = u < p.units;
                if (more) un = Unit(p, u, tokens);
            }
        }
    }
    MOE_DEV void next(const Params& p) {
        ++c;
        step(p);
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

template <bool F8>
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
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int tokens = seq_tokens(p.seq);
    const int gtok = kAccCols / p.Hp;  // tokens of an accumulator
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
        Tiles tile(p, tokens);
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
            const uint32_t st = smem_u32(smem + C::kStageOff + s * C::kStageBytes) + dst0;
#pragma unroll
            for (int i = 0; i < kKeys / kRows; ++i) {
                const int at = __shfl_sync(0xFFFFFFFFu, row[i * kRows / 32], (i * kRows + sub) & 31);
                copy16(st + i * kRows * 128 + (((piece & 7) ^ ((i * kRows + sub) & 7)) << 4),
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
        uint32_t n = 0;
        for (long long u = blockIdx.x; u < p.units; u += gridDim.x, ++n) {
            Unit un(p, u, tokens);
            if (!wait(qempty, (n & 1u) ^ 1u)) break;
            const uint32_t base = smem_u32(smem);
            constexpr int kPer = C::kRowBytes / 16;
            const int rows = max(0, un.u1 - un.u0) * p.Hp;
            const int piece = tid % kPer;
#pragma unroll 8
            for (int rr = tid / kPer; rr < rows; rr += 32 * kQueryWarps / kPer) {
                const int t = rr / p.Hp, h = rr % p.Hp;
                const long long at = ((long long)(un.u0 + t) * p.H + (h < p.H ? h : 0)) * C::kRowBytes;
                copy16(base + (piece / 8) * (C::kCols * 128) + rr * 128 + (((piece & 7) ^ (rr & 7)) << 4),
                       p.q + at + piece * 16, h < p.H ? 16u : 0u);
            }
            copy_commit();
            for (int i = tid; i < rows; i += 32 * kQueryWarps) {
                const int t = i / p.Hp, h = i % p.Hp;
                wts[i] = h < p.H ? __ldg(p.w + (long long)(un.u0 + t) * p.H + h) : 0.0f;
            }
            for (int t = tid; t < un.u1 - un.u0; t += 32 * kQueryWarps) lens[t] = seq_length(p.seq, un.u0 + t);
            copy_wait<0>();
            fence_async_shared();
            mbar_arrive(qfull);
        }
    } else if (warp >= kMmaWarp) {
        // ================================ UMMA issuers ================================
        const uint32_t mine = warp - kMmaWarp;  // accumulators of this parity
        uint32_t it = 0, acc = 0, n = 0;
        const uint64_t dq = sdesc_k128(smem_u32(smem)), dk = sdesc_k128(smem_u32(smem + C::kStageOff));
        for (long long u = blockIdx.x; u < p.units && ok; u += gridDim.x, ++n) {
            Unit un(p, u, tokens);
            if (!wait(qfull, n & 1u)) break;
            Part r;
            while (ok && un.part(p, r)) {
                const int accs = (r.t1 - r.t0 + gtok - 1) / gtok;  // of a tile
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
                        const uint64_t db = dq + (uint64_t)((t - un.u0) * p.Hp * 8);
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
            }
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
        uint32_t it = 0, acc = 0, n = 0;
        for (long long u = blockIdx.x; u < p.units && ok; u += gridDim.x, ++n) {
            Unit un(p, u, tokens);
            if (!wait(qfull, n & 1u)) break;  // (the weights and lengths)
            Part r;
            while (ok && un.part(p, r)) {
                const int accs = (r.t1 - r.t0 + gtok - 1) / gtok;  // of a tile
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
                            w0 = wts + (t - un.u0) * p.Hp;
                            len = lens + (t - un.u0);
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
                        for (int i = 0; i < cnt; ++i, out += p.ld) {
                            float2 s0 = make_float2(0.0f, 0.0f), s1 = s0;
                            int h = p.Hp;
                            for (; h >= 32; h -= 32, ta += 32, w += 32) {
                                uint32_t v[32];
                                tmem_ld32(ta, v);
                                tmem_ready(v);
                                weigh16(v, w, s0, s1);
                                weigh16(v + 16, w + 16, s0, s1);
                            }
                            if (h) {
                                uint32_t v[16];
                                tmem_ld16(ta, v);
                                tmem_ready(v);
                                weigh16(v, w, s0, s1);
                                ta += 16;
                                w += 16;
                            }
                            const float sum = (s0.x + s0.y) + (s1.x + s1.y);
                            if (pos < p.n) *out = hidden < len[i] ? sum * ks : -__int_as_float(0x7F800000);
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&aempty[mine]);
                    }
                }
                if (!ok) break;
                // what no token of the part may see
                const int e0 = max(r.c1, un.c0) * kKeys, e1 = min(p.n, un.c1 * kKeys);
                for (int t = r.t0; t < r.t1; ++t)
                    for (int j = e0 + (int)threadIdx.x; j < e1; j += 32 * kEpiWarps)
                        p.out[(long long)t * p.ld + j] = -__int_as_float(0x7F800000);
            }
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

template <bool F8>
cudaError_t run(const ScoresArgs& a, cudaStream_t s) {
    using C = Cfg<F8>;
    static DeviceOnce once;
    const cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(scores_kernel<F8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
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
    p.tiles = (a.n + kKeys - 1) / kKeys;
    // tokens of a unit: what a sequence has on average, as far as the columns go
    const int avg = a.cu ? (int)((a.T + a.B - 1) / a.B) : 1;
    p.tt = C::kCols / p.Hp;
    if (avg < p.tt) p.tt = avg;
    const long long groups = (a.T + p.tt - 1) / p.tt;
    // key tiles of a unit: the number of rounds of units times their clocks, at the least (queries
    // loaded, then 280 clocks per accumulator and tile, or what 128 keys take from HBM)
    const int accs = (p.tt + kAccCols / p.Hp - 1) / (kAccCols / p.Hp);
    const long long tile = accs * 280 > 3 * C::kRowBytes * 2 ? accs * 280 : 3 * C::kRowBytes * 2;
    const long long query = p.tt * p.Hp > kAccCols ? 3000 + p.tt * p.Hp * C::kRowBytes / 32 : 300;
    long long best = -1;
    for (long long cuts = 1; cuts <= p.tiles; cuts += 1 + cuts / 8) {
        const long long kc = (p.tiles + cuts - 1) / cuts;
        const long long units = groups * ((p.tiles + kc - 1) / kc);
        const long long t = (units + num_sms() - 1) / num_sms() * (query + kc * tile);
        // (as long, and more units: sequences of different lengths even out)
        if (best < 0 || t <= best) {
            best = t;
            p.kc = (int)kc;
        }
    }
    p.units = groups * ((p.tiles + p.kc - 1) / p.kc);
    long long grid = num_sms();
    if (p.units < grid) grid = p.units;
    return launch_kernel(scores_kernel<F8>, dim3((unsigned)grid), dim3(kThreads), (size_t)C::kSmemBytes,
                         s, p);
}

}  // namespace

cudaError_t launch_scores(const ScoresArgs& a, cudaStream_t s) {
    return a.key_scales ? run<true>(a, s) : run<false>(a, s);
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

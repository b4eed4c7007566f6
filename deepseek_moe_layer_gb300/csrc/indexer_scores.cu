// indexer_scores.cu -- the indexer's scores of the cached positions on the 5th-generation tensor
// cores:
//     out[t, j] = ks_j * sum_h w[t, h] * max(q[t, h] . k_j, 0)    j < lengths[t], else -inf
// with index keys k_j of 128 columns in a paged cache, bf16 or e4m3 (ks_j: a scale per key).
//
// Keys lie on the tensor cores' M side (128 per tile) and (token, head) pairs on the N side: a
// thread then holds one key's dot products with all heads, the sum over the heads is its own
// and a token's scores leave as consecutive numbers.  A unit is `tt` consecutive tokens (up to 512
// columns, in shared memory for the whole unit) and `kc` key tiles that stream past them; tokens
// of several sequences in one unit are taken sequence by sequence, with the columns of that
// sequence's tokens only.  Columns run in groups of up to 256 (whole tokens) through two TMEM
// accumulators of 256, so the epilogue of one overlaps the UMMAs of the next.
//
// Warp roles (448 threads, one CTA per SM, persistent over units): warps 0..7 epilogue (warp % 4 =
// TMEM lane quarter, warp / 4 takes every other token), 8..11 key copies (16-byte asynchronous
// copies, so that pages of any size and any order do; rows without a page or behind the end are
// zeros), 12 UMMA issuer, 13 queries and weights.  Every wait is bounded.
#include <mutex>

#include "launch.h"
#include "paged.cuh"

namespace moe {

__device__ unsigned int g_scores_status;

namespace {

constexpr int kD = 128;             // columns of an index key
constexpr int kKeys = 128;          // keys per tile
constexpr int kCols = 512;          // (token, head) columns of a unit
constexpr int kGroupCols = 256;     // of them per accumulator
constexpr int kEpiWarps = 8, kLoadWarps = 4;
constexpr int kMmaWarp = kEpiWarps + kLoadWarps, kQueryWarp = kMmaWarp + 1;
constexpr int kThreads = 32 * (kQueryWarp + 1);

template <bool F8>
struct Cfg {
    static constexpr int kRowBytes = F8 ? kD : 2 * kD;
    static constexpr int kBlocks = kRowBytes / 128;         // 128-byte blocks of a row
    static constexpr int kQBytes = kCols * kRowBytes;
    static constexpr int kStageBytes = kKeys * kRowBytes;
    static constexpr int kStages = F8 ? 8 : 3;
    static constexpr int kLag = F8 ? 4 : 1;                 // tiles in flight behind the newest
    static constexpr int kStageOff = kQBytes;
    static constexpr int kWOff = kStageOff + kStages * kStageBytes;
    static constexpr int kBarOff = kWOff + 4 * kCols;
    // full, empty, query full, query empty, accumulator full (2), empty (2), done
    static constexpr int kBars = 2 * kStages + 2 + 4 + 1;
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

template <bool F8>
__global__ void __launch_bounds__(kThreads, 1) scores_kernel(const Params p) {
    using C = Cfg<F8>;
    extern __shared__ __align__(1024) uint8_t smem[];
    float* wts = reinterpret_cast<float*>(smem + C::kWOff);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
    uint64_t* empty = full + C::kStages;
    uint64_t* qfull = empty + C::kStages;
    uint64_t* qempty = qfull + 1;
    uint64_t* afull = qfull + 2;
    uint64_t* aempty = afull + 2;
    uint64_t* done = aempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
    volatile int* abort = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], kLoadWarps);
            mbar_init(&empty[s], 1);
        }
        mbar_init(qfull, 32);
        mbar_init(qempty, 1 + kEpiWarps);  // the unit's last UMMA, and the weights read
        for (int i = 0; i < 2; ++i) {
            mbar_init(&afull[i], 1);
            mbar_init(&aempty[i], kEpiWarps);
        }
        mbar_init(done, 1);
        *abort = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int tokens = seq_tokens(p.seq);
    const int gtok = max(1, kGroupCols / p.Hp);  // tokens of an accumulator

    if (warp >= kEpiWarps && warp < kMmaWarp) {
        // ================================ key copies ================================
        const int w = warp - kEpiWarps;  // rows 32 w .. 32 w + 31 of a tile
        constexpr int kPer = C::kRowBytes / 16;   // 16-byte pieces of a row
        constexpr int kRows = 32 / kPer;          // rows that a warp copies at once
        uint32_t it = 0, posted = 0;              // tiles copied, tiles announced
        bool ok = true;
        const auto post = [&] {
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[posted % C::kStages]);
            ++posted;
        };
        for (long long u = blockIdx.x; u < p.units && ok; u += gridDim.x) {
            Unit un(p, u, tokens);
            Part r;
            while (ok && un.part(p, r)) {
                for (int c = r.c0; c < r.c1; ++c, ++it) {
                    const uint32_t s = it % C::kStages;
                    const int pos = c * kKeys + 32 * w + lane;
                    const long long mine = pos < p.seq.most ? paged_row(p.keys, r.b, pos) : -1;
                    if (!__all_sync(0xFFFFFFFFu,
                                    mbar_test(&empty[s], ((it / C::kStages) & 1u) ^ 1u))) {
                        // no slot yet: what has been asked for is announced before the wait
                        copy_wait<0>();
                        while (posted < it) post();
                        if (!__all_sync(0xFFFFFFFFu,
                                        mbar_wait(&empty[s], ((it / C::kStages) & 1u) ^ 1u, abort))) {
                            if (lane == 0) record_timeout(abort);
                            ok = false;
                            break;
                        }
                    }
                    __syncwarp();
                    const uint32_t st = smem_u32(smem + C::kStageOff + s * C::kStageBytes);
#pragma unroll
                    for (int i = 0; i < 32 / kRows; ++i) {
                        const int rr = i * kRows + lane / kPer, piece = lane % kPer;
                        const long long row = __shfl_sync(0xFFFFFFFFu, mine, rr);
                        const int tr = 32 * w + rr;
                        copy16(st + (piece / 8) * (kKeys * 128) + tr * 128 + (((piece & 7) ^ (tr & 7)) << 4),
                               p.k + (row < 0 ? 0 : row) * C::kRowBytes + piece * 16, row < 0 ? 0u : 16u);
                    }
                    copy_commit();
                    if (it - posted >= C::kLag) {
                        copy_wait<C::kLag>();
                        post();
                    }
                }
            }
        }
        copy_wait<0>();
        while (posted < it) post();
    } else if (warp == kQueryWarp) {
        // ============================ queries and weights ============================
        uint32_t n = 0;
        for (long long u = blockIdx.x; u < p.units; u += gridDim.x, ++n) {
            Unit un(p, u, tokens);
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(qempty, (n & 1u) ^ 1u, abort))) {
                if (lane == 0) record_timeout(abort);
                break;
            }
            const uint32_t base = smem_u32(smem);
            constexpr int kPer = C::kRowBytes / 16;
            const int rows = (un.u1 - un.u0) * p.Hp;
            for (int i = lane; i < rows * kPer; i += 32) {
                const int rr = i / kPer, piece = i % kPer;
                const int t = rr / p.Hp, h = rr % p.Hp;
                const long long at = ((long long)(un.u0 + t) * p.H + (h < p.H ? h : 0)) * C::kRowBytes;
                copy16(base + (piece / 8) * (kCols * 128) + rr * 128 + (((piece & 7) ^ (rr & 7)) << 4),
                       p.q + at + piece * 16, h < p.H ? 16u : 0u);
            }
            copy_commit();
            for (int i = lane; i < rows; i += 32) {
                const int t = i / p.Hp, h = i % p.Hp;
                wts[i] = h < p.H ? __ldg(p.w + (long long)(un.u0 + t) * p.H + h) : 0.0f;
            }
            copy_wait<0>();
            fence_async_shared();
            mbar_arrive(qfull);
        }
    } else if (warp == kMmaWarp) {
        // ================================ UMMA issuer ================================
        uint32_t it = 0, acc = 0, n = 0;
        bool ok = true;
        const auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
            if (__all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort))) return true;
            if (lane == 0) record_timeout(abort);
            return ok = false;
        };
        const uint64_t dq = sdesc_k128(smem_u32(smem)), dk = sdesc_k128(smem_u32(smem + C::kStageOff));
        for (long long u = blockIdx.x; u < p.units && ok; u += gridDim.x, ++n) {
            Unit un(p, u, tokens);
            if (!wait(qfull, n & 1u)) break;
            Part r;
            while (ok && un.part(p, r)) {
                for (int c = r.c0; c < r.c1 && ok; ++c, ++it) {
                    const uint32_t s = it % C::kStages;
                    if (!wait(&full[s], (it / C::kStages) & 1u)) break;
                    const uint64_t da = dk + (uint64_t)(s * (C::kStageBytes / 16));
                    for (int t = r.t0; t < r.t1; t += gtok, ++acc) {
                        const uint32_t ab = acc & 1u;
                        if (!wait(&aempty[ab], ((acc >> 1) & 1u) ^ 1u)) break;
                        tc_fence_after();
                        const int cols = min(gtok, r.t1 - t) * p.Hp;
                        const uint32_t idesc = C::kIdesc0 | ((uint32_t)(cols >> 3) << 17);
                        const uint64_t db = dq + (uint64_t)((t - un.u0) * p.Hp * 8);
                        if (elect_lane()) {
#pragma unroll
                            for (int blk = 0; blk < C::kBlocks; ++blk)
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const uint64_t a = da + (uint64_t)(blk * (kKeys * 128 / 16) + 2 * k);
                                    const uint64_t b = db + (uint64_t)(blk * (kCols * 128 / 16) + 2 * k);
                                    if (F8) umma_f8(tmem + ab * kGroupCols, a, b, idesc, blk + k > 0);
                                    else umma_bf16(tmem + ab * kGroupCols, a, b, idesc, blk + k > 0);
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
        const int quarter = warp & 3, set = warp >> 2;
        const uint32_t taddr0 = tmem + ((uint32_t)(quarter * 32) << 16);
        uint32_t acc = 0, n = 0;
        bool ok = true;
        for (long long u = blockIdx.x; u < p.units && ok; u += gridDim.x, ++n) {
            Unit un(p, u, tokens);
            // (the weights are read behind this wait)
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(qfull, n & 1u, abort))) {
                if (lane == 0) record_timeout(abort);
                break;
            }
            Part r;
            while (ok && un.part(p, r)) {
                for (int c = r.c0; c < r.c1 && ok; ++c) {
                    const int pos = c * kKeys + quarter * 32 + lane;
                    const long long row = pos < p.seq.most ? paged_row(p.keys, r.b, pos) : -1;
                    float ks = 1.0f;
                    if (F8 && row >= 0) ks = __ldg(p.ks + row);
                    for (int t = r.t0; t < r.t1; t += gtok, ++acc) {
                        const uint32_t ab = acc & 1u;
                        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&afull[ab], (acc >> 1) & 1u, abort))) {
                            if (lane == 0) record_timeout(abort);
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const int cnt = min(gtok, r.t1 - t);
                        for (int i = (int)((set + acc) & 1u); i < cnt; i += 2) {
                            const uint32_t ta = taddr0 + ab * kGroupCols + (uint32_t)(i * p.Hp);
                            const float* w = wts + (t + i - un.u0) * p.Hp;
                            float sum = 0.0f;
                            for (int h = 0; h < p.Hp; h += 16) {
                                uint32_t v[16];
                                tmem_ld16(ta + (uint32_t)h, v);
                                float wv[16];
#pragma unroll
                                for (int e = 0; e < 16; e += 4)
                                    *reinterpret_cast<float4*>(wv + e) =
                                        *reinterpret_cast<const float4*>(w + h + e);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    float x = __uint_as_float(v[e]);
                                    asm("max.NaN.f32 %0, %0, 0f00000000;" : "+f"(x));
                                    sum = fmaf(x, wv[e], sum);
                                }
                            }
                            if (pos < p.n)
                                p.out[(long long)(t + i) * p.ld + pos] =
                                    row >= 0 && pos < seq_length(p.seq, t + i)
                                        ? sum * ks
                                        : -__int_as_float(0x7F800000);
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&aempty[ab]);
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
    p.tt = kCols / p.Hp;
    if (avg < p.tt) p.tt = avg;
    const long long groups = (a.T + p.tt - 1) / p.tt;
    // key tiles of a unit: eight units per SM where there are as many, so that sequences of
    // different lengths even out, and no more than 64
    long long kc = groups * p.tiles / (8 * num_sms());
    p.kc = (int)(kc < 1 ? 1 : kc > 64 ? 64 : kc);
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

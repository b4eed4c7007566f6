// gemm_scaled.cu -- products of block-scaled e4m3 matrices on the 5th-generation tensor cores:
//   kLinear : y[r, n]  = sum_b sx[r, b] sw[n/128, b] (sum_{k in block b} x[r, k] w[n, k])
//             (the dense product and the experts' down product; bf16 or fp32 out)
//   kSwiglu : h[r, j]  = silu(g) * u with g, u two such sums over the gate and the up rows,
//             written as e4m3 codes with a power-of-two scale for each row and 128 features
// x [rows, K] and w [F, K] hold e4m3 codes, sx [rows, ceil(K/128)] and sw [ceil(F/128),
// ceil(K/128)] any fp32 scales.
//
// Groups and tiles follow the expert GEMMs: E routed groups (rows offsets[g] .. offsets[g+1])
// and optionally the shared expert as group E, or a single group; a tile is 128 token rows x
// 256 weight rows (kSwiglu: 128 gate rows and the same 128 up rows), tokens fastest, derived
// from the offsets on the device.
//
// The scales vary along K, so the sum cannot stay in TMEM: every 128-wide k-block is one
// UMMA group (128 x 256 x 128, four K = 32 steps) into one of two TMEM buffers, and sixteen
// warps fold the finished buffer into fp32 sums in registers with one multiply-add per element
// (two per instruction) while the tensor core fills the other.  A row is one thread's, so the
// row scale is a register and the weight scale is uniform over a warp's columns.
//
// Warp roles (384 threads, one CTA per SM, persistent over tiles): warp 0 TMA producer,
// warp 1 TMEM owner and UMMA issuer, warps 4..19 scaling and epilogue (warp % 4 = TMEM lane
// quarter, (warp - 4) / 4 = quarter of the columns; warps 2 and 3 only lend their registers).
// Sixteen warps of 64 sums rather than eight of 128: four per scheduler hide each other's TMEM
// and barrier latency, and the sums stay in registers.  Every wait is bounded, as in the expert GEMMs.
#include <mutex>

#include "launch.h"
#include "scaled.cuh"

namespace moe {

__device__ unsigned int g_scaled_status;

namespace {

enum { kLinear = 0, kSwiglu = 1 };

constexpr int kThreads = 640;
constexpr int kEpiWarps = 16;
constexpr int kEpiWarp0 = 4;  // first of them: four whole warpgroups
constexpr int kParts = 4;     // warps per TMEM lane quarter, each a quarter of the columns
constexpr int kBK = 128;                        // codes per 128-byte swizzled row = one k-block
constexpr int kABytes = 128 * kBK;
constexpr int kBBytes = 256 * kBK;
constexpr int kStageBytes = kABytes + kBBytes;  // 48 KB
constexpr int kStages = 4;
constexpr int kMaxGroups = 1025;
constexpr int kBarOff = kStages * kStageBytes;
constexpr int kNumBars = 2 * kStages + 2 + 2 + 1 + 4;  // full, empty, tfull, tempty, done, pair
constexpr int kMiscOff = kBarOff + 8 * kNumBars;
constexpr int kPrefixOff = (kMiscOff + 16 + 15) / 16 * 16;
constexpr int kRowOffOff = kPrefixOff + 4 * (kMaxGroups + 1);
constexpr int kAmaxOff = (kRowOffOff + 4 * (kMaxGroups + 1) + 15) / 16 * 16;
constexpr int kRagOff = kAmaxOff + 4 * 2 * kParts * 128;
constexpr int kRagLd = 9;  // floats per row of a warp's 32 x 8 piece: no bank conflicts by row
constexpr int kSmemBytes = kRagOff + 4 * kEpiWarps * 32 * kRagLd + 1024;  // + stage alignment
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");

// kind::f8f6f4: fp32 accumulator (bits 4-5 = 1), e4m3 A and B (formats 0), both K-major,
// N >> 3 at bits 17-22, M >> 4 at bits 24-28.
constexpr uint32_t kIdesc = (1u << 4) | ((256u >> 3) << 17) | ((128u >> 4) << 24);

struct Params {
    const int32_t* offsets;  // [E + 1], or nullptr: one group of `single_rows` rows
    long long single_rows;
    int E, has_shared;
    long long shared_rows;   // T
    long long shared_row0;   // first row of the shared group in x and in the output
    int nkb;                 // k-blocks
    int F;                   // outputs (kSwiglu: features) per group
    const float* sx;         // [rows, nkb]
    const float* sw0;        // [groups * ceil(F/128), nkb]: weights, or gate
    const float* sw1;        // kSwiglu: up
    const float* ssw0;       // the shared expert's
    const float* ssw1;
    void* out;               // kLinear: bf16 or fp32 [rows, ld]; kSwiglu: codes [rows, F]
    long long ld;
    int f32;                 // kLinear: fp32 out
    int vec;                 // kLinear: rows of `out` are 32-byte aligned
    float* out_scale;        // kSwiglu: [rows, F / 128]
};

MOE_DEV void umma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(kIdesc), "r"(accumulate)
        : "memory");
}

// Waits for this thread's TMEM loads; the registers pass through it so that no use of them
// moves ahead of the wait.
MOE_DEV void tmem_wait16(uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.wait::ld.sync.aligned;"
        : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
          "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
          "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
        :
        : "memory");
}

// acc (two fp32) += (lo, hi) * f, both lanes of f the same factor.
MOE_DEV void fma_pair(unsigned long long& acc, uint32_t lo, uint32_t hi, unsigned long long f) {
    asm("{\n\t.reg .b64 t;\n\t"
        "mov.b64 t, {%1, %2};\n\t"
        "fma.rn.f32x2 %0, t, %3, %0;\n\t}"
        : "+l"(acc)
        : "r"(lo), "r"(hi), "l"(f));
}
MOE_DEV unsigned long long both(float f) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(f));
    return r;
}
MOE_DEV unsigned long long pair_of(float lo, float hi) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
// An infinity has no e4m3 code: it becomes NaN, and leaves the block's scale to the others.
MOE_DEV float nan_for_inf(float v) {
    return fabsf(v) == __int_as_float(0x7F800000) ? __int_as_float(0x7FFFFFFF) : v;
}
MOE_DEV float lo_of(unsigned long long v) { return __uint_as_float((uint32_t)v); }
MOE_DEV float hi_of(unsigned long long v) { return __uint_as_float((uint32_t)(v >> 32)); }

// acc (16 sums) += 16 TMEM columns of the thread's lane * f.
MOE_DEV void fold16(unsigned long long* acc, const uint32_t (&r)[16], float f) {
    const unsigned long long ff = both(f);
#pragma unroll
    for (int i = 0; i < 8; ++i) fma_pair(acc[i], r[2 * i], r[2 * i + 1], ff);
}

// One 32-byte store (a whole sector).
MOE_DEV void st_global_32B(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

MOE_DEV void record_timeout(volatile int* abort) {
    *abort = 1;
    atomicCAS(&g_scaled_status, 0u, kStatusTimeout);
}

struct Tile {
    int g, f, rows;   // group (E = shared), feature tile, valid token rows
    bool shared;
    long long row;    // first row, in x and in the output
};

MOE_DEV long long rows_of(const Params& p, const int32_t* rowoff, int g) {
    if (!p.offsets) return p.single_rows;
    return g == p.E ? p.shared_rows : (long long)(rowoff[g + 1] - rowoff[g]);
}

MOE_DEV Tile tile_at(const Params& p, const int32_t* prefix, const int32_t* rowoff, int ngroups,
                     int t) {
    int lo = 0, hi = ngroups - 1;  // largest g with prefix[g] <= t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= t) lo = mid; else hi = mid - 1;
    }
    Tile ti;
    ti.g = lo;
    ti.shared = p.offsets && lo == p.E;
    const long long rows = rows_of(p, rowoff, lo);
    const int mt = (int)((rows + 127) / 128);
    const int local = t - prefix[lo];
    const long long r0 = (long long)(local % mt) * 128;
    ti.f = local / mt;
    ti.rows = (int)(rows - r0 < 128 ? rows - r0 : 128);
    ti.row = (ti.shared ? p.shared_row0 : p.offsets ? (long long)rowoff[lo] : 0) + r0;
    return ti;
}

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    scaled_gemm_kernel(const __grid_constant__ CUtensorMap tm_x,     // boxes of 128 rows
                       const __grid_constant__ CUtensorMap tm_x32,   // boxes of 32 rows
                       const __grid_constant__ CUtensorMap tm_w0,
                       const __grid_constant__ CUtensorMap tm_w1,
                       const __grid_constant__ CUtensorMap tm_s0,
                       const __grid_constant__ CUtensorMap tm_s1, const Params p) {
    constexpr int kFeat = MODE == kSwiglu ? 128 : 256;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kBarOff);
    uint64_t* empty = full + kStages;
    uint64_t* tfull = empty + kStages;
    uint64_t* tempty = tfull + 2;
    uint64_t* done = tempty + 2;
    uint64_t* pair = done + 1;  // kSwiglu: the warps of a lane quarter exchange row maxima
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kMiscOff);
    volatile int* abort = reinterpret_cast<volatile int*>(smem + kMiscOff + 4);
    int32_t* prefix = reinterpret_cast<int32_t*>(smem + kPrefixOff);
    int32_t* rowoff = reinterpret_cast<int32_t*>(smem + kRowOffOff);
    float* rag = reinterpret_cast<float*>(smem + kRagOff);
    float* amax = reinterpret_cast<float*>(smem + kAmaxOff);  // [tile parity][part][row]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ngroups = p.offsets ? p.E + p.has_shared : 1;
    const int ftiles = (p.F + kFeat - 1) / kFeat;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], kEpiWarps);
        }
        mbar_init(done, 1);
        for (int q = 0; q < 4; ++q) mbar_init(&pair[q], kParts);
        *abort = 0;
        fence_mbar_init();
        prefetch_tmap(&tm_x);
        prefetch_tmap(&tm_x32);
        prefetch_tmap(&tm_w0);
        if (MODE == kSwiglu) prefetch_tmap(&tm_w1);
    }
    if (warp == 1) tmem_alloc(tmem_slot, 512);
    pdl_wait();
    if (p.offsets)
        for (int i = threadIdx.x; i <= p.E; i += blockDim.x) rowoff[i] = p.offsets[i];
    __syncthreads();
    if (warp == 0) {
        const int per = (ngroups + 31) / 32;
        const int g0 = lane * per, g1 = min(ngroups, g0 + per);
        int local = 0;
        for (int g = g0; g < g1; ++g)
            local += (int)((rows_of(p, rowoff, g) + 127) / 128) * ftiles;
        int incl = local;
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, incl, off);
            if (lane >= off) incl += v;
        }
        int run = incl - local;
        for (int g = g0; g < g1; ++g) {
            prefix[g] = run;
            run += (int)((rows_of(p, rowoff, g) + 127) / 128) * ftiles;
        }
        if (lane == 31) prefix[ngroups] = incl;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int total = prefix[ngroups];

    // 640 threads at 96 registers: the scaling warps take from the other four
    // (64 * 128 + 104 * 512 = 96 * 640)
    if (warp < kEpiWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 0) {
        // =============================== TMA producer ===============================
        if (lane == 0) {
            const uint64_t pol_w = policy_evict_first(), pol_x = policy_evict_last();
            int it = 0, s = 0;
            uint32_t ph = 0u;
            bool ok = true;
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
                const Tile ti = tile_at(p, prefix, rowoff, ngroups, t);
                const CUtensorMap* w0 = ti.shared ? &tm_s0 : &tm_w0;
                const CUtensorMap* w1 = ti.shared ? &tm_s1 : &tm_w1;
                const int wrow = (ti.shared || !p.offsets ? 0 : ti.g * p.F) + ti.f * kFeat;
                // only the rows the tile has (32 at a time): the others' products are unused
                const int boxes = ti.rows > 96 ? 4 : (ti.rows + 31) / 32;
                for (int kb = 0; kb < p.nkb; ++kb, ++it) {
                    if (it > 0 && ++s == kStages) { s = 0; ph ^= 1u; }
                    if (!mbar_wait(&empty[s], ph ^ 1u, abort)) {
                        record_timeout(abort);
                        ok = false;
                        break;
                    }
                    uint8_t* st = smem + s * kStageBytes;
                    mbar_arrive_expect_tx(&full[s], (uint32_t)(boxes * 32 * kBK + kBBytes));
                    if (MODE == kSwiglu) {
                        tma_load_2d(st + kABytes, w0, &full[s], kb * kBK, wrow, pol_w);
                        tma_load_2d(st + kABytes + kBBytes / 2, w1, &full[s], kb * kBK, wrow, pol_w);
                    } else {
                        tma_load_2d(st + kABytes, w0, &full[s], kb * kBK, wrow, pol_w);
                    }
                    if (boxes == 4)
                        tma_load_2d(st, &tm_x, &full[s], kb * kBK, (int)ti.row, pol_x);
                    else
                        for (int b = 0; b < boxes; ++b)
                            tma_load_2d(st + b * 32 * kBK, &tm_x32, &full[s], kb * kBK,
                                        (int)ti.row + 32 * b, pol_x);
                }
            }
            // no copy may land after the CTA has gone
            for (int i = it > kStages ? it - kStages : 0; i < it; ++i)
                mbar_wait(&full[i % kStages], (uint32_t)(i / kStages) & 1u, nullptr, 100000000ull);
        }
    } else if (warp == 1) {
        // ================================ UMMA issuer ===============================
        if (lane == 0) {
            int it = 0, s = 0;
            uint32_t ph = 0u;
            bool ok = true;
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
                for (int kb = 0; kb < p.nkb; ++kb, ++it) {
                    if (it > 0 && ++s == kStages) { s = 0; ph ^= 1u; }
                    const int b = it & 1;
                    if (!mbar_wait(&tempty[b], (((uint32_t)it >> 1) & 1u) ^ 1u, abort) ||
                        !mbar_wait(&full[s], ph, abort)) {
                        record_timeout(abort);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t xs = smem_u32(smem + s * kStageBytes);
                    const uint64_t dx = sdesc_k128(xs), dw = sdesc_k128(xs + kABytes);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)  // 32 codes = 32 bytes further each
                        umma_e4m3(tmem + (uint32_t)(b * 256), dx + (uint64_t)(2 * kk),
                                  dw + (uint64_t)(2 * kk), kk > 0 ? 1u : 0u);
                    umma_commit(&empty[s]);
                    umma_commit(&tfull[b]);
                }
            }
            if (it > 0) {  // every UMMA issued has finished before TMEM is given back
                umma_commit(done);
                mbar_wait(done, 0u, nullptr, 100000000ull);
            }
        }
    }
    } else {
        // ============================ scaling and epilogue ==========================
        asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        const int q = warp & 3, part = (warp - kEpiWarp0) >> 2;
        const int r = q * 32 + lane;  // the thread's row of the tile
        const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16);
        // the warp's two chunks of 32 columns: 32 gate and 32 up, or 64 in a row
        const int c0 = MODE == kSwiglu ? 32 * part : 64 * part;
        const int c1 = MODE == kSwiglu ? 128 + 32 * part : 64 * part + 32;
        const int wblocks = (p.F + 127) / 128;
        int it = 0, lt = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < total; t += gridDim.x, ++lt) {
            const Tile ti = tile_at(p, prefix, rowoff, ngroups, t);
            const bool mine = r < ti.rows;
            const bool idle = q * 32 >= ti.rows;  // no row of this warp is in the tile
            const float* sx = p.sx + (ti.row + (mine ? r : 0)) * p.nkb;
            const long long wb = (long long)(ti.shared || !p.offsets ? 0 : ti.g) * wblocks +
                                 (MODE == kSwiglu ? ti.f : min(2 * ti.f + part / 2, wblocks - 1));
            const float* sw0 = (ti.shared ? p.ssw0 : p.sw0) + wb * p.nkb;
            const float* sw1 = MODE == kSwiglu ? (ti.shared ? p.ssw1 : p.sw1) + wb * p.nkb : sw0;
            unsigned long long acc[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[i] = 0ull;
            float x_next = sx[0], w0_next = sw0[0], w1_next = MODE == kSwiglu ? sw1[0] : 0.0f;
            for (int kb = 0; kb < p.nkb; ++kb, ++it) {
                const float f0 = x_next * w0_next, f1 = MODE == kSwiglu ? x_next * w1_next : f0;
                if (kb + 1 < p.nkb) {
                    x_next = sx[kb + 1];
                    w0_next = sw0[kb + 1];
                    if (MODE == kSwiglu) w1_next = sw1[kb + 1];
                }
                const int b = it & 1;
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(&tfull[b], ((uint32_t)it >> 1) & 1u, abort))) {
                    record_timeout(abort);
                    ok = false;
                    break;
                }
                if (!idle) {
                    tc_fence_after();
                    const uint32_t col = taddr + (uint32_t)(b * 256);
                    uint32_t u[16], v[16];
                    tmem_ld16(col + (uint32_t)c0, u);
                    tmem_wait16(u);
                    tmem_ld16(col + (uint32_t)c0 + 16u, v);
                    fold16(acc, u, f0);
                    tmem_wait16(v);
                    tmem_ld16(col + (uint32_t)c1, u);
                    fold16(acc + 8, v, f0);
                    tmem_wait16(u);
                    tmem_ld16(col + (uint32_t)c1 + 16u, v);
                    fold16(acc + 16, u, f1);
                    tmem_wait16(v);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&tempty[b]);
                    fold16(acc + 24, v, f1);
                } else if (lane == 0) {
                    mbar_arrive(&tempty[b]);
                }
            }
            if (!ok) break;
            if constexpr (MODE == kSwiglu) {
                // h over the gate sums' registers, the row's maximum with the other parts
                float m = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float h0 = nan_for_inf(silu(lo_of(acc[i])) * lo_of(acc[16 + i]));
                    const float h1 = nan_for_inf(silu(hi_of(acc[i])) * hi_of(acc[16 + i]));
                    m = fmaxf(m, fmaxf(fabsf(h0), fabsf(h1)));
                    acc[i] = pair_of(h0, h1);
                }
                float* am = amax + (lt & 1) * (kParts * 128) + r;
                am[part * 128] = m;
                __syncwarp();
                if (lane == 0) mbar_arrive(&pair[q]);
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(&pair[q], (uint32_t)lt & 1u, abort))) {
                    record_timeout(abort);
                    break;
                }
#pragma unroll
                for (int o = 0; o < kParts; ++o) m = fmaxf(m, am[o * 128]);
                float s, inv;
                block_scale(m, s, inv);
                if (mine) {
                    uint32_t w[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        w[j] = cvt_e4m3x4(lo_of(acc[2 * j]) * inv, hi_of(acc[2 * j]) * inv,
                                          lo_of(acc[2 * j + 1]) * inv, hi_of(acc[2 * j + 1]) * inv);
                    st_global_32B(static_cast<uint8_t*>(p.out) + (ti.row + r) * p.F + ti.f * 128 +
                                      32 * part,
                                  w);
                    if (part == 0) p.out_scale[(ti.row + r) * (p.F / 128) + ti.f] = s;
                }
            } else {
                const int n0 = ti.f * 256 + 64 * part;
                if (p.vec && n0 + 64 <= p.F) {
                    if (mine && p.f32) {
                        float* o = static_cast<float*>(p.out) + (ti.row + r) * p.ld + n0;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            uint32_t w[8];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                w[2 * j] = __float_as_uint(lo_of(acc[4 * i + j]));
                                w[2 * j + 1] = __float_as_uint(hi_of(acc[4 * i + j]));
                            }
                            st_global_32B(o + 8 * i, w);
                        }
                    } else if (mine) {
                        uint16_t* o = static_cast<uint16_t*>(p.out) + (ti.row + r) * p.ld + n0;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t w[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                w[j] = pack_bf16x2(lo_of(acc[8 * i + j]), hi_of(acc[8 * i + j]));
                            st_global_32B(o + 16 * i, w);
                        }
                    }
                } else if (!idle) {
                    // rows without 32-byte alignment, or the last columns: eight columns at a
                    // time through shared memory, so that a store covers eight columns of four
                    // rows instead of one of 32
                    float* piece = rag + (warp - kEpiWarp0) * (32 * kRagLd);
                    const int pr = lane >> 3, pc = lane & 7;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            piece[lane * kRagLd + 2 * j] = lo_of(acc[4 * i + j]);
                            piece[lane * kRagLd + 2 * j + 1] = hi_of(acc[4 * i + j]);
                        }
                        __syncwarp();
                        const int n = n0 + 8 * i + pc;
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int rr = 4 * k + pr;
                            if (q * 32 + rr < ti.rows && n < p.F) {
                                const long long at = (ti.row + q * 32 + rr) * p.ld + n;
                                const float v = piece[rr * kRagLd + pc];
                                if (p.f32) static_cast<float*>(p.out)[at] = v;
                                else static_cast<uint16_t*>(p.out)[at] = (uint16_t)pack_bf16x2(v, 0.0f);
                            }
                        }
                    }
                }
            }
        }
    }

    pdl_launch_dependents();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    return fn;
}

// Codes [rows, cols], rows `ld` bytes apart, in boxes of 128 columns x box_rows rows with the
// 128-byte swizzle; what lies outside reads as zero.
bool code_map(CUtensorMap* m, const void* base, long long rows, long long cols, long long ld,
              int box_rows) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)(rows < 1 ? 1 : rows)};
    const cuuint64_t strides[1] = {(cuuint64_t)ld};
    const cuuint32_t box[2] = {(cuuint32_t)kBK, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE>
cudaError_t run(const ScaledGemmArgs& a, cudaStream_t s) {
    static DeviceOnce attr_once;
    cudaError_t err = attr_once.run([] {
        return cudaFuncSetAttribute(scaled_gemm_kernel<MODE>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    });
    if (err != cudaSuccess) return err;
    const int wbox = MODE == kSwiglu ? 128 : 256;
    const long long wrows = (long long)(a.offsets ? a.E : 1) * a.F;
    CUtensorMap x, x32, w0, w1, s0, s1;
    bool ok = code_map(&x, a.x, a.rows, a.K, a.ldx, 128) &&
              code_map(&x32, a.x, a.rows, a.K, a.ldx, 32) &&
              code_map(&w0, a.w.w0, wrows, a.K, a.K, wbox);
    w1 = s0 = s1 = w0;
    if (ok && a.w.w1) ok = code_map(&w1, a.w.w1, wrows, a.K, a.K, wbox);
    if (ok && a.has_shared) ok = code_map(&s0, a.ws.w0, a.F, a.K, a.K, wbox);
    if (ok && a.has_shared && a.ws.w1) ok = code_map(&s1, a.ws.w1, a.F, a.K, a.K, wbox);
    if (!ok) return cudaErrorInvalidValue;

    Params p = {};
    p.offsets = a.offsets;
    p.single_rows = a.rows;
    p.E = a.E;
    p.has_shared = a.has_shared;
    p.shared_rows = a.shared_rows;
    p.shared_row0 = a.shared_row0;
    p.nkb = (a.K + kBK - 1) / kBK;
    p.F = a.F;
    p.sx = a.sx;
    p.sw0 = a.w.s0;
    p.sw1 = a.w.s1;
    p.ssw0 = a.ws.s0;
    p.ssw1 = a.ws.s1;
    p.out = a.out;
    p.ld = a.F;
    p.f32 = a.f32;
    p.vec = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0 && a.F % (a.f32 ? 8 : 16) == 0;
    p.out_scale = a.out_scale;

    // at most this many tiles (the offsets are on the device): a group adds one ragged tile
    const long long ft = (a.F + (MODE == kSwiglu ? 127 : 255)) / (MODE == kSwiglu ? 128 : 256);
    const long long mt = a.offsets ? a.shared_row0 / 128 + a.E + (a.shared_rows + 127) / 128
                                   : (a.rows + 127) / 128;
    long long grid = num_sms();
    if (mt * ft < grid) grid = mt * ft;
    if (grid < 1) return cudaSuccess;
    return launch_kernel(scaled_gemm_kernel<MODE>, dim3((unsigned)grid), dim3(kThreads),
                         (size_t)kSmemBytes, s, x, x32, w0, w1, s0, s1, p);
}

}  // namespace

cudaError_t launch_scaled_gemm(const ScaledGemmArgs& a, cudaStream_t s) {
    return a.swiglu ? run<kSwiglu>(a, s) : run<kLinear>(a, s);
}

cudaError_t read_scaled_status(unsigned int* out, int clear, cudaStream_t s) {
    cudaError_t err = cudaMemcpyFromSymbolAsync(out, g_scaled_status, sizeof(unsigned int), 0,
                                                cudaMemcpyDeviceToHost, s);
    if (err != cudaSuccess) return err;
    err = cudaStreamSynchronize(s);
    if (err != cudaSuccess || !clear) return err;
    const unsigned int zero = 0;
    err = cudaMemcpyToSymbolAsync(g_scaled_status, &zero, sizeof(unsigned int), 0,
                                  cudaMemcpyHostToDevice, s);
    if (err != cudaSuccess) return err;
    return cudaStreamSynchronize(s);
}

}  // namespace moe

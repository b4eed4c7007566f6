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
// two halves of 128 weight rows (kSwiglu: 128 gate rows and the same up rows), tokens fastest,
// derived from the offsets on the device.
//
// The scales vary along K, so the sum cannot stay in TMEM: a k-block of 128 is one group of
// UMMAs (128 x 256 x 128, four K = 32 steps) into one of two TMEM buffers, and eight warps fold
// the finished buffer into fp32 sums in registers, one multiply-add per element (two per
// instruction), while the tensor core fills the other.  A row is one thread's, so the row scale
// times the weight scale is one factor per thread, half and k-block.  (Scales whose fp32 product is
// no normal number: factor_class.)
//
// What bounds a long product is the way round a buffer: UMMA issue, completion, TMEM loads and
// multiply-adds, the buffer's release (410 .. 470, 500 .. 600, 450 .. 490 and 190 cycles by the
// clock; with the 150 .. 350 that the trace does not place about 1900 for each of the two buffers,
// so some 950 .. 1000 per k-block against the UMMAs' own 512): 8192 x 4096 x 7168 takes 212 us, 170
// with the scaling left out, 107 for the UMMAs alone.  Tried and slower there: sixteen warps of 64 columns (242 us), halves of 128
// columns with barriers, issuers or warps of their own (261 .. 277), an issuer per buffer (225),
// looking at the next k-block's barriers between UMMAs (223), CTA pairs with cta_group::2 (513:
// the way round crosses the cluster twice).
//
// Warp roles (384 threads, one CTA per SM, persistent over tiles): warp 0 TMA producer, warp 1
// TMEM owner and UMMA issuer, warps 2 and 3 multiply the scales ahead of the others, warps 4..11
// scaling and epilogue: warp % 4 = TMEM lane quarter, (warp - 4) / 4 = part, the first or last 64
// columns of each half (kSwiglu: of the gate and of the up rows, so silu(g) * u stays in the
// thread).  Every wait is bounded, as in the expert GEMMs.
#include <mutex>

#include "launch.h"
#include "scaled.cuh"

namespace moe {

__device__ unsigned int g_scaled_status;

namespace {

enum { kLinear = 0, kSwiglu = 1 };

constexpr int kEpiWarps = 8;
constexpr int kEpiWarp0 = 4;                   // first of them: whole warpgroups
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
// Columns of each half that a warp sums: 64, or with FEW (tiles of 32 rows) 16.
template <int FEW>
constexpr int kRun = FEW ? 16 : 64;
constexpr int kPartLd = 260;                   // SPLIT: floats per row of a CTA's partial sums
constexpr int kLowRegs = 56, kHighRegs = 224;  // 56 * 128 + 224 * 256 = 168 * 384
constexpr int kBK = 128;                       // codes per 128-byte swizzled row = one k-block
constexpr int kMaxGroups = 1025;
constexpr int kFKb = 4;                        // k-blocks of factors per slot
constexpr int kFSlots = 2;                     // a power of two
constexpr int kFacFloats = kFKb * 2 * 128;     // [k-block][half][row]
constexpr int kRagLd = 5;  // floats per row of a warp's 32 x 4 piece: no bank conflicts by row

constexpr int kABytes = 128 * kBK;
constexpr int kBBytes = 128 * kBK;             // per half
constexpr int kStageBytes = kABytes + 2 * kBBytes;
constexpr int kStages = 4;
constexpr int kBarOff = kStages * kStageBytes;
// full, empty, tfull, tempty, done, row maxima, ffull, fempty, decided
constexpr int kNumBars = 2 * kStages + 2 + 2 + 1 + 4 + 2 * kFSlots + 1;
constexpr int kMiscOff = kBarOff + 8 * kNumBars;  // TMEM address, abort, lost
constexpr int kPrefixOff = (kMiscOff + 16 + 15) / 16 * 16;
constexpr int kRowOffOff = kPrefixOff + 4 * (kMaxGroups + 1);
constexpr int kFacOff = (kRowOffOff + 4 * (kMaxGroups + 1) + 15) / 16 * 16;
constexpr int kEpiOff = kFacOff + 4 * kFSlots * kFacFloats;
constexpr int kEpiBytes = 4 * kEpiWarps * 32 * kRagLd;  // kLinear: pieces; kSwiglu: row maxima
constexpr int kSmemBytes = kEpiOff + kEpiBytes + 1024;  // + alignment of the stages
static_assert(kEpiBytes >= 4 * 2 * 2 * 128, "room for the row maxima");
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");

// kind::f8f6f4: fp32 accumulator (bits 4-5 = 1), e4m3 A and B (formats 0), both K-major,
// N >> 3 at bits 17-22 (256), M >> 4 at bits 24-28 (128).
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
    int f32;                 // kLinear: fp32 out (not FEW: the experts' rows are bf16)
    int vec;                 // kLinear: rows of `out` are 32-byte aligned
    float* out_scale;        // kSwiglu: [rows, F / 128]
    int split;               // SPLIT: CTAs per tile (the cluster's size), k-blocks shared out
};

// One k-block: four K = 32 steps (32 codes = 32 bytes further each) into one buffer, then the
// arrivals on `tfull` (the buffer is done) and `empty` (the stage has been read).
MOE_DEV void umma_block(uint32_t d_tmem, uint64_t dx, uint64_t dw, uint64_t* tfull, uint64_t* empty) {
    asm volatile(
        "{\n\t.reg .pred t;\n\t"
        "setp.eq.b32 t, 0, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %9, !t;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %3, %4, %9, t;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %5, %6, %9, t;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %7, %8, %9, t;\n\t"
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%10];\n\t"
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%11];\n\t}" ::"r"(
            d_tmem),
        "l"(dx), "l"(dw), "l"(dx + 2), "l"(dw + 2), "l"(dx + 4), "l"(dw + 4), "l"(dx + 6), "l"(dw + 6),
        "r"(kIdesc), "r"(smem_u32(tfull)), "r"(smem_u32(empty))
        : "memory");
}

// An infinity has no e4m3 code: it becomes NaN, and leaves the block's scale to the others.
MOE_DEV float nan_for_inf(float v) {
    return fabsf(v) == __int_as_float(0x7F800000) ? __int_as_float(0x7FFFFFFF) : v;
}

// 16 TMEM columns of the thread's lane, loaded and waited for in one statement: no use of the
// registers can move ahead of the wait.
MOE_DEV void tmem_get16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// acc (16 sums) += 16 TMEM columns of the thread's lane * f.
MOE_DEV void fold16(float* acc, const uint32_t (&r)[16], float f) {
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        const float2 v = __ffma2_rn(make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])),
                                    make_float2(f, f), make_float2(acc[i], acc[i + 1]));
        acc[i] = v.x;
        acc[i + 1] = v.y;
    }
}

// A block's sum is 0 or between 2^-18 and 2^25, so it can make a normal number with two scales
// whose own fp32 product is none: such a factor has lost what its scales hold.  A CTA that met one
// goes over its tiles a second time and writes them again, now three times over the k-blocks of
// each: with the factors too large for fp32 (kLarge: less 2^128), with those too small (kSmall:
// times 2^100) and with all the others, each time 0 for the rest.  The sums are put right in
// between; the loop over the k-blocks is the same one (a branch for it in there, or a second loop:
// 8192 x 4096 x 7168 231 .. 269 us against 210).
enum { kLarge = 0, kSmall = 1, kUsual = 2 };
constexpr float kFltMax = 0x1.fffffep127f;

MOE_DEV int factor_class(float f, float a, float g) {
    const float v = fabsf(f);
    if (v < 0x1p-126f && a != 0.0f && g != 0.0f) return kSmall;
    return v > kFltMax && fabsf(a) <= kFltMax && fabsf(g) <= kFltMax ? kLarge : kUsual;
}

// The factor of the scales a and g in the sweep `cls` of a second time.  A small one's scales are
// both below 2^23, a large one's both at least 1.
MOE_DEV float class_factor(float a, float g, int cls) {
    const float f = a * g;
    if (factor_class(f, a, g) != cls) return 0.0f;
    if (cls == kLarge) return (a * 0x1p-64f) * (g * 0x1p-64f);
    return cls == kSmall ? (a * 0x1p50f) * (g * 0x1p50f) : f;
}

// What a sweep left, as the next one needs it.  After the large factors a sum is 0, or so large
// that the small ones do not move it, neither by what they are nor by 2^100 times that; so the
// second step leaves it alone, and the others leave 2^100.
MOE_DEV float after_sweep(float v, int cls) {
    if (cls == kLarge) return v * 0x1p64f * 0x1p64f;
    return cls == kSmall && fabsf(v) < 0x1p60f ? v * 0x1p-100f : v;
}

// One 32-byte store (a whole sector).
MOE_DEV void st_global_32B(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// What the scaling warps wait on and free: the two buffers in TMEM and the factor slots, with the
// k-blocks and the slots taken so far.
struct Rings {
    uint64_t *tfull, *tempty, *ffull, *fempty;
    uint32_t it, fn;
};

// One tile's sums of a warp over n k-blocks: its RUN columns of each half times the factor of
// the thread's row (f: the first half's in slot 0) are added to acc.  LIVE false (no row of the
// warp is in the tile): only the waiting.  False when a wait gave up (then in every lane).
template <int RUN, bool LIVE>
MOE_DEV bool sums(float (&acc)[2 * RUN], int n, Rings& rg, const float* f, uint32_t taddr,
                  volatile int* abort) {
    const int lane = threadIdx.x & 31;
    int fi = 0;
#pragma unroll 1
    for (int kb = 0; kb < n; ++kb, ++rg.it) {
        const uint32_t b = rg.it & 1u, s = rg.fn & (kFSlots - 1);
        if (fi == 0 && !__all_sync(0xFFFFFFFFu, mbar_wait(&rg.ffull[s], (rg.fn / kFSlots) & 1u, abort)))
            return false;
        const float* g = f + s * kFacFloats + fi * 256;
        const float f0 = g[0], f1 = g[128];
        if (++fi == kFKb || kb == n - 1) {
            fi = 0;
            ++rg.fn;
            __syncwarp();
            if (lane == 0) mbar_arrive(&rg.fempty[s]);
        }
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&rg.tfull[b], (rg.it >> 1) & 1u, abort))) return false;
        if (LIVE) {
            tc_fence_after();
            uint32_t u[16];
#pragma unroll
            for (int c = 0; c < 2 * RUN; c += 16) {
                tmem_get16(taddr + b * 256u + (uint32_t)(c < RUN ? c : c - RUN + 128), u);
                if (c == 2 * RUN - 16) {  // the last load: the buffer is free before the last sums
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&rg.tempty[b]);
                }
                fold16(acc + c, u, c < RUN ? f0 : f1);
            }
        } else if (lane == 0) {
            mbar_arrive(&rg.tempty[b]);
        }
    }
    return true;
}

MOE_DEV float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
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

template <int TR>
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
    const int mt = (int)((rows + TR - 1) / TR);
    const int local = t - prefix[lo];
    const long long r0 = (long long)(local % mt) * TR;
    ti.f = local / mt;
    ti.rows = (int)(rows - r0 < TR ? rows - r0 : TR);
    ti.row = (ti.shared ? p.shared_row0 : p.offsets ? (long long)rowoff[lo] : 0) + r0;
    return ti;
}

// SPLIT: adds the partial sums of a tile's CTAs (their shared memory at `part`, in rank order)
// and writes the rows rank, rank + split, ..: a warp per row, a lane four columns of each half.
template <int MODE, int FEW>
MOE_DEV void join_rows(const Params& p, const Tile& ti, const float* part, int rank) {
    const bool f32 = !FEW && p.f32;
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - kEpiWarp0;
    for (int r = rank + p.split * w; r < ti.rows; r += p.split * kEpiWarps) {
        const float* at = part + r * kPartLd + 4 * lane;
        float4 x[8], y[8];
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (c < p.split) {
                const uint32_t from = mapa_shared(at, (uint32_t)c);
                x[c] = ld_cluster_f4(from);
                y[c] = ld_cluster_f4(from + 512u);
            }
        float g[4] = {0.0f, 0.0f, 0.0f, 0.0f}, u[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (c < p.split) {
                g[0] += x[c].x; g[1] += x[c].y; g[2] += x[c].z; g[3] += x[c].w;
                u[0] += y[c].x; u[1] += y[c].y; u[2] += y[c].z; u[3] += y[c].w;
            }
        const long long row = ti.row + r;
        if constexpr (MODE == kSwiglu) {
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                g[i] = nan_for_inf(silu(g[i]) * u[i]);
                m = fmaxf(m, fabsf(g[i]));
            }
#pragma unroll
            for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
            float s, inv;
            block_scale(m, s, inv);
            *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + row * p.F + ti.f * 128 +
                                         4 * lane) =
                cvt_e4m3x4(g[0] * inv, g[1] * inv, g[2] * inv, g[3] * inv);
            if (lane == 0) p.out_scale[row * (p.F / 128) + ti.f] = s;
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float* v = h ? u : g;
                const int n = ti.f * 256 + 128 * h + 4 * lane;
                if (f32) {
                    float* o = static_cast<float*>(p.out) + row * p.ld + n;
                    if (p.vec && n + 4 <= p.F) {
                        *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (n + i < p.F) o[i] = v[i];
                    }
                } else {
                    uint16_t* o = static_cast<uint16_t*>(p.out) + row * p.ld + n;
                    const uint32_t a = pack_bf16x2(v[0], v[1]), b = pack_bf16x2(v[2], v[3]);
                    if (p.vec && n + 4 <= p.F) {
                        *reinterpret_cast<uint2*>(o) = make_uint2(a, b);
                    } else {
                        if (n < p.F) o[0] = (uint16_t)a;
                        if (n + 1 < p.F) o[1] = (uint16_t)(a >> 16);
                        if (n + 2 < p.F) o[2] = (uint16_t)b;
                        if (n + 3 < p.F) o[3] = (uint16_t)(b >> 16);
                    }
                }
            }
        }
    }
}

template <int MODE, int FEW, int SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    scaled_gemm_kernel(const __grid_constant__ CUtensorMap tm_x,     // boxes of 128 rows (FEW: 8)
                       const __grid_constant__ CUtensorMap tm_x32,   // boxes of 32 rows
                       const __grid_constant__ CUtensorMap tm_w0,
                       const __grid_constant__ CUtensorMap tm_w1,
                       const __grid_constant__ CUtensorMap tm_s0,
                       const __grid_constant__ CUtensorMap tm_s1, const Params p) {
    constexpr int kFeat = MODE == kSwiglu ? 128 : 256;
    constexpr int kTile = FEW ? 32 : 128;  // token rows
    constexpr int RUN = kRun<FEW>;
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
    uint64_t* ffull = pair + 4;
    uint64_t* fempty = ffull + kFSlots;
    uint64_t* decided = fempty + kFSlots;
    volatile int* lost = reinterpret_cast<volatile int*>(smem + kMiscOff + 8);
    float* fac = reinterpret_cast<float*>(smem + kFacOff);
    float* rag = reinterpret_cast<float*>(smem + kEpiOff);
    float* amax = rag;          // kSwiglu: [tile parity][warps of a row][row]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ngroups = p.offsets ? p.E + p.has_shared : 1;
    const int ftiles = (p.F + kFeat - 1) / kFeat;
    // SPLIT: a cluster per tile, each CTA its share of the k-blocks
    const int rank = SPLIT ? (int)cluster_rank() : 0;
    const int tstart = SPLIT ? (int)blockIdx.x / p.split : (int)blockIdx.x;
    const int tstep = SPLIT ? (int)gridDim.x / p.split : (int)gridDim.x;
    const int kb0 = SPLIT ? p.nkb * rank / p.split : 0;
    const int kb1 = SPLIT ? p.nkb * (rank + 1) / p.split : p.nkb;

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
        for (int q = 0; q < 4; ++q) mbar_init(&pair[q], FEW ? kEpiWarps : 2);
        for (int f = 0; f < kFSlots; ++f) {
            mbar_init(&ffull[f], 64);
            mbar_init(&fempty[f], kEpiWarps);
        }
        mbar_init(decided, 64);
        *abort = 0;
        *lost = 0;
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
            local += (int)((rows_of(p, rowoff, g) + kTile - 1) / kTile) * ftiles;
        int incl = local;
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, incl, off);
            if (lane >= off) incl += v;
        }
        int run = incl - local;
        for (int g = g0; g < g1; ++g) {
            prefix[g] = run;
            run += (int)((rows_of(p, rowoff, g) + kTile - 1) / kTile) * ftiles;
        }
        if (lane == 31) prefix[ngroups] = incl;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int total = prefix[ngroups];

    // 384 threads at 168 registers: the scaling warps take from the other four
    if (warp < kEpiWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLowRegs));
    if (warp == 0) {
        // =============================== TMA producer ===============================
        if (lane == 0) {
            const uint64_t pol_w = policy_evict_first(), pol_x = policy_evict_last();
            int it = 0, s = 0;
            uint32_t ph = 0u;
            bool ok = true;
            int sweeps = 1;
            for (int pass = 0; pass < 2 && ok; ++pass, sweeps = 3) {
                if (pass && !(mbar_wait(decided, 0u, abort) && *lost)) break;
                for (int t = tstart; t < total && ok; t += tstep) {
                    const Tile ti = tile_at<kTile>(p, prefix, rowoff, ngroups, t);
                    const CUtensorMap* w0 = ti.shared ? &tm_s0 : &tm_w0;
                    const CUtensorMap* w1 = ti.shared ? &tm_s1 : &tm_w1;
                    const int wrow = (ti.shared || !p.offsets ? 0 : ti.g * p.F) + ti.f * kFeat;
                    // only the rows the tile has (32 at a time): the others' products are unused.
                    // FEW: the same rows in every lane quarter, 8 or 32 of them (one token's
                    // experts: 84 -> 74 us)
                    const int boxes = FEW || ti.rows > 96 ? 4 : (ti.rows + 31) / 32;
                    const int per = FEW && ti.rows <= 8 ? 8 : 32;
                    for (int sweep = 0; sweep < sweeps && ok; ++sweep)
                        for (int kb = kb0; kb < kb1; ++kb, ++it) {
                            if (it > 0 && ++s == kStages) { s = 0; ph ^= 1u; }
                            if (!mbar_wait(&empty[s], ph ^ 1u, abort)) {
                                record_timeout(abort);
                                ok = false;
                                break;
                            }
                            uint8_t* st = smem + s * kStageBytes;
                            const int kx = kb * kBK;
                            mbar_arrive_expect_tx(&full[s],
                                                  (uint32_t)(boxes * per * kBK + 2 * kBBytes));
                            tma_load_2d(st + kABytes, w0, &full[s], kx, wrow, pol_w);
                            tma_load_2d(st + kABytes + kBBytes, MODE == kSwiglu ? w1 : w0,
                                        &full[s], kx, MODE == kSwiglu ? wrow : wrow + 128, pol_w);
                            if (!FEW && boxes == 4)
                                tma_load_2d(st, &tm_x, &full[s], kx, (int)ti.row, pol_x);
                            else
                                for (int b = 0; b < boxes; ++b)
                                    tma_load_2d(st + b * 32 * kBK, per == 8 ? &tm_x : &tm_x32,
                                                &full[s], kx, (int)ti.row + (FEW ? 0 : 32 * b),
                                                pol_x);
                        }
                }
            }
            // no copy may land after the CTA has gone
            for (int i = it > kStages ? it - kStages : 0; i < it; ++i)
                mbar_wait(&full[i % kStages], (uint32_t)(i / kStages) & 1u, nullptr, 100000000ull);
        }
    } else if (warp == 1) {
        // ================================ UMMA issuer ===============================
        // (few instructions between a buffer's release and its next UMMA: they are on the way
        // round)
        if (lane == 0) {
            const int mine = tstart < total ? (total - 1 - tstart) / tstep + 1 : 0;
            const int n = SPLIT ? (mine > 0 ? kb1 - kb0 : 0) : mine * p.nkb;
            const uint64_t dx = sdesc_k128(smem_u32(smem)), dw = sdesc_k128(smem_u32(smem) + kABytes);
            constexpr uint64_t kStep = kStageBytes >> 4;  // descriptors count 16 bytes
            uint64_t ax = dx, aw = dw;
            uint32_t ph = 0u, it = 0u, end = (uint32_t)n;
            int s = 0;
#pragma unroll 1
            for (;; ++it) {
                if (it == end) {  // (3 n + n at most: a second time)
                    if (it != (uint32_t)n || !(mbar_wait(decided, 0u, abort) && *lost)) break;
                    end *= 4u;
                }
                const uint32_t b = it & 1u;
                if (!mbar_wait(&full[s], ph, abort) ||
                    !mbar_wait(&tempty[b], ((it >> 1) & 1u) ^ 1u, abort)) {
                    record_timeout(abort);
                    break;
                }
                tc_fence_after();
                umma_block(tmem + b * 256u, ax, aw, &tfull[b], &empty[s]);
                ax += kStep;
                aw += kStep;
                if (++s == kStages) {
                    s = 0;
                    ph ^= 1u;
                    ax = dx;
                    aw = dw;
                }
            }
            // every UMMA issued has finished before TMEM is given back
            if (n > 0) {
                umma_commit(done);
                mbar_wait(done, 0u, nullptr, 100000000ull);
            }
        }
    } else {
        // ============================== scale factors ===============================
        // fac[k-block][half][row] = sx[row] * sw[half], kFKb k-blocks per slot, ahead of the
        // scaling warps: a row's scales are read once and in 16 bytes, not by every warp of
        // the row in every k-block (32 lines per load)
        const int w = threadIdx.x - 64;
        const int wblocks = (p.F + 127) / 128;
        const bool vec = ((p.nkb | kb0) & 3) == 0 && (reinterpret_cast<uintptr_t>(p.sx) & 15) == 0;
        int n = 0;
        bool ok = true;
        int sweeps = 1;
        for (int pass = 0; pass < 2 && ok; ++pass, sweeps = 3) {
            if (pass) {
                mbar_arrive(decided);
                if (!(mbar_wait(decided, 0u, abort) && *lost)) break;
            }
            for (int t = tstart; t < total && ok; t += tstep) {
                const Tile ti = tile_at<kTile>(p, prefix, rowoff, ngroups, t);
                const long long wb = (long long)(ti.shared || !p.offsets ? 0 : ti.g) * wblocks;
                const float* sw0 = ti.shared ? p.ssw0 : p.sw0;
                const float* sw1 = MODE == kSwiglu ? (ti.shared ? p.ssw1 : p.sw1) : sw0;
                sw0 += (wb + (MODE == kSwiglu ? ti.f : 2 * ti.f)) * p.nkb;
                sw1 += (wb + (MODE == kSwiglu ? ti.f : min(2 * ti.f + 1, wblocks - 1))) * p.nkb;
                const float* sx = p.sx + ti.row * p.nkb;
                const int last = ti.rows - 1;
                for (int sweep = 0; sweep < sweeps && ok; ++sweep)
                    for (int kb = kb0; kb < kb1; kb += kFKb, ++n) {
                        const int s = n % kFSlots;
                        float a[2][kFKb];  // rows w and w + 64 (FEW: the lane's)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int r = min(FEW ? w & 31 : w + 64 * j, last);
                            const float* x = sx + (long long)r * p.nkb + kb;
                            if (vec) {
                                *reinterpret_cast<float4*>(a[j]) = *reinterpret_cast<const float4*>(x);
                            } else {
#pragma unroll
                                for (int i = 0; i < kFKb; ++i) a[j][i] = kb + i < kb1 ? x[i] : 0.0f;
                            }
                        }
                        if (!mbar_wait(&fempty[s], (((uint32_t)n / kFSlots) & 1u) ^ 1u, abort)) {
                            record_timeout(abort);
                            ok = false;
                            break;
                        }
                        float* f = fac + s * kFacFloats + w;
                        float low = 1.0f, high = 1.0f;
#pragma unroll
                        for (int i = 0; i < kFKb; ++i) {
                            if (kb + i >= kb1) break;
                            const float g0 = sw0[kb + i], g1 = sw1[kb + i];
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const float x = a[j][i];
                                const float f0 = pass ? class_factor(x, g0, sweep) : x * g0;
                                const float f1 = pass ? class_factor(x, g1, sweep) : x * g1;
                                f[i * 256 + 64 * j] = f0;
                                f[i * 256 + 128 + 64 * j] = f1;
                                low = fminf(low, fminf(fabsf(f0), fabsf(f1)));
                                high = fmaxf(high, fmaxf(fabsf(f0), fabsf(f1)));
                            }
                        }
                        if (!(low >= 0x1p-126f && high <= kFltMax) && !pass) {  // (or scales of 0)
#pragma unroll
                            for (int i = 0; i < kFKb; ++i) {
                                if (kb + i >= kb1) break;
                                const float g0 = sw0[kb + i], g1 = sw1[kb + i];
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    const float x = a[j][i];
                                    if (factor_class(x * g0, x, g0) != kUsual ||
                                        factor_class(x * g1, x, g1) != kUsual)
                                        *lost = 1;
                                }
                            }
                        }
                        mbar_arrive(&ffull[s]);
                    }
            }
        }
    }
    if constexpr (SPLIT) {  // around the join of the scaling warps
        __syncwarp();
        cluster_sync();
        cluster_sync();
    }
    } else {
        // ============================ scaling and epilogue ==========================
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kHighRegs));
        const int q = warp & 3, part = (warp - kEpiWarp0) >> 2;
        const int c0 = FEW ? 16 * (2 * q + part) : 64 * part;  // the warp's columns of a half
        const int wr = FEW ? 0 : q * 32;                       // its first row
        const int r = wr + lane;                               // the thread's row of the tile
        const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)c0;
        const bool f32 = !FEW && p.f32;
        Rings rg = {tfull, tempty, ffull, fempty, 0u, 0u};
        int lt = 0;  // tiles so far
        bool ok = true;
        int sweeps = 1;
        for (int pass = 0; pass < 2 && ok; ++pass, sweeps = 3) {
            // (every factor of the tiles has been waited for, and with them what `lost` says)
            __syncwarp();
            if (pass && !*lost) break;
            for (int t = tstart; t < total; t += tstep, ++lt) {
                const Tile ti = tile_at<kTile>(p, prefix, rowoff, ngroups, t);
                const bool mine = r < ti.rows;
                const bool idle = wr >= ti.rows;  // no row of this warp is in the tile
                float acc[2 * RUN];
#pragma unroll
                for (int i = 0; i < 2 * RUN; ++i) acc[i] = 0.0f;
                for (int sweep = 0; sweep < sweeps && ok; ++sweep) {
                    ok = idle ? sums<RUN, false>(acc, kb1 - kb0, rg, fac + r, taddr, abort)
                              : sums<RUN, true>(acc, kb1 - kb0, rg, fac + r, taddr, abort);
                    if (sweeps > 1) {
#pragma unroll
                        for (int i = 0; i < 2 * RUN; ++i) acc[i] = after_sweep(acc[i], sweep);
                    }
                }
                if (!ok) {
                    record_timeout(abort);
                    break;
                }
                if constexpr (SPLIT) {
                    // into this CTA's shared memory (every copy into it has been consumed, and no
                    // second time will follow)
                    float* row = reinterpret_cast<float*>(smem) + r * kPartLd + c0;
                    if (mine && !(*lost && sweeps == 1))
#pragma unroll
                        for (int i = 0; i < 2 * RUN; i += 4)
                            *reinterpret_cast<float4*>(row + (i < RUN ? i : i - RUN + 128)) =
                                make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
                    break;  // one tile per cluster
                }
                else if constexpr (MODE == kSwiglu) {
                    // h over the gate sums' registers, the row's maximum with the other parts
                    float m = 0.0f;
#pragma unroll
                    for (int i = 0; i < RUN; ++i) {
                        acc[i] = nan_for_inf(silu(acc[i]) * acc[RUN + i]);
                        m = fmaxf(m, fabsf(acc[i]));
                    }
                    float* am = amax + (lt & 1) * 256 + r;
                    uint64_t* bar = FEW ? &pair[0] : &pair[q];
                    am[FEW ? 32 * (2 * q + part) : 128 * part] = m;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar);
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar, (uint32_t)lt & 1u, abort));
                    if (!ok) {
                        record_timeout(abort);
                        break;
                    }
#pragma unroll
                    for (int o = 0; o < 256; o += kTile) m = fmaxf(m, am[o]);
                    float s, inv;
                    block_scale(m, s, inv);
                    if (mine) {
                        uint8_t* o = static_cast<uint8_t*>(p.out) + (ti.row + r) * p.F + ti.f * 128 + c0;
                        if constexpr (FEW) {
                            *reinterpret_cast<uint4*>(o) = make_uint4(
                                cvt_e4m3x4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv),
                                cvt_e4m3x4(acc[4] * inv, acc[5] * inv, acc[6] * inv, acc[7] * inv),
                                cvt_e4m3x4(acc[8] * inv, acc[9] * inv, acc[10] * inv, acc[11] * inv),
                                cvt_e4m3x4(acc[12] * inv, acc[13] * inv, acc[14] * inv, acc[15] * inv));
                        } else {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                uint32_t w[8];
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
                                    const float* x = acc + 32 * i + 4 * j;
                                    w[j] = cvt_e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
                                }
                                st_global_32B(o + 32 * i, w);
                            }
                        }
                        if (c0 == 0) p.out_scale[(ti.row + r) * (p.F / 128) + ti.f] = s;
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int n0 = ti.f * 256 + 128 * h + c0;
                        const float* sum = acc + RUN * h;
                        if (p.vec && n0 + RUN <= p.F) {
                            if (mine && f32) {
                                float* o = static_cast<float*>(p.out) + (ti.row + r) * p.ld + n0;
#pragma unroll
                                for (int i = 0; i < RUN / 8; ++i) {
                                    uint32_t w[8];
#pragma unroll
                                    for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(sum[8 * i + j]);
                                    st_global_32B(o + 8 * i, w);
                                }
                            } else if (mine) {
                                uint16_t* o = static_cast<uint16_t*>(p.out) + (ti.row + r) * p.ld + n0;
#pragma unroll
                                for (int i = 0; i < RUN / 16; ++i) {
                                    uint32_t w[8];
#pragma unroll
                                    for (int j = 0; j < 8; ++j)
                                        w[j] = pack_bf16x2(sum[16 * i + 2 * j], sum[16 * i + 2 * j + 1]);
                                    st_global_32B(o + 16 * i, w);
                                }
                            }
                        } else if (!idle && n0 < p.F) {
                            // rows without 32-byte alignment, or the last columns: four columns at
                            // a time through shared memory, so that a store covers four columns of
                            // eight rows instead of one of 32
                            float* piece = rag + (warp - kEpiWarp0) * (32 * kRagLd);
                            const int pr = lane >> 2, pc = lane & 3;
#pragma unroll
                            for (int i = 0; i < RUN / 4; ++i) {
                                __syncwarp();
#pragma unroll
                                for (int j = 0; j < 4; ++j) piece[lane * kRagLd + j] = sum[4 * i + j];
                                __syncwarp();
                                const int n = n0 + 4 * i + pc;
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const int rr = 8 * k + pr;
                                    if (wr + rr < ti.rows && n < p.F) {
                                        const long long at = (ti.row + wr + rr) * p.ld + n;
                                        const float v = piece[rr * kRagLd + pc];
                                        if (f32) static_cast<float*>(p.out)[at] = v;
                                        else static_cast<uint16_t*>(p.out)[at] = (uint16_t)pack_bf16x2(v, 0.0f);
                                    }
                                }
                            }
                        }
                    }
                }
            }
        }
        if constexpr (SPLIT) {
            __syncwarp();
            cluster_sync();  // all partial sums are written
            if (tstart < total)
                join_rows<MODE, FEW>(p, tile_at<kTile>(p, prefix, rowoff, ngroups, tstart),
                                reinterpret_cast<const float*>(smem), rank);
            __syncwarp();
            cluster_sync();  // and read: the CTAs may leave
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

// At most this many tiles of `tr` token rows (the offsets are on the device): a group that has
// rows adds one ragged tile.
long long max_tiles(const ScaledGemmArgs& a, long long tr) {
    const long long per = a.swiglu ? 128 : 256, ft = (a.F + per - 1) / per;
    if (!a.offsets) return (a.rows + tr - 1) / tr * ft;
    const long long P = a.shared_row0, hit = P < a.E ? P : a.E;
    return (P / tr + hit + (a.shared_rows + tr - 1) / tr) * ft;
}

template <int MODE, int FEW, int SPLIT>
cudaError_t run(const ScaledGemmArgs& a, int split, cudaStream_t s) {
    static DeviceOnce attr_once;
    cudaError_t err = attr_once.run([] {
        return cudaFuncSetAttribute(scaled_gemm_kernel<MODE, FEW, SPLIT>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    });
    if (err != cudaSuccess) return err;
    const int wbox = 128;
    const long long wrows = (long long)(a.offsets ? a.E : 1) * a.F;
    CUtensorMap x, x32, w0, w1, s0, s1;
    bool ok = code_map(&x, a.x, a.rows, a.K, a.ldx, FEW ? 8 : 128) &&
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

    p.split = split;
    const long long tiles = max_tiles(a, FEW ? 32 : 128);
    if (tiles < 1) return cudaSuccess;
    if constexpr (SPLIT) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(tiles * split), 1, 1);
        cfg.blockDim = dim3(kThreads, 1, 1);
        cfg.dynamicSmemBytes = kSmemBytes;
        cfg.stream = s;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)split;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = pdl_enabled() ? 2 : 1;
        err = cudaLaunchKernelEx(&cfg, scaled_gemm_kernel<MODE, FEW, SPLIT>, x, x32, w0, w1, s0, s1, p);
        return err != cudaSuccess ? err : cudaGetLastError();
    } else {
        const long long sms = num_sms();
        return launch_kernel(scaled_gemm_kernel<MODE, FEW, SPLIT>,
                             dim3((unsigned)(tiles < sms ? tiles : sms)), dim3(kThreads),
                             (size_t)kSmemBytes, s, x, x32, w0, w1, s0, s1, p);
    }
}

template <int MODE>
cudaError_t choose(const ScaledGemmArgs& a, cudaStream_t s) {
    // Experts with few rows: tiles of 32 rows, the same rows in every lane quarter, so that all
    // scaling warps share the columns instead of two of them doing all (64 experts, 7168 x 2048,
    // up to 8 / 24 / 32 rows per expert on average: 413 / 472 / 536 us against 473 / 505 / 514 for
    // tiles of 128 rows).  A single group's product keeps tiles of 128, though the others would be the
    // faster ones by now for up to 32 rows (32 x 32768 x 2048: 12.6 us against 11.7, 8 rows 12.1
    // against 11.1, 1 x 2112 x 7168 9.1 against 8.3).
    const bool few = a.offsets && a.shared_row0 <= (long long)24 * a.E;
    // Too few tiles for the SMs: 2, 4 or 8 CTAs share a tile's k-blocks (two at least each) and
    // join their sums through the cluster's shared memory, in rank order, if that spares a CTA
    // at least six k-blocks, which the join costs (1 x 2112 x 7168: 9.1 us against 29.4 for a CTA
    // per tile; 128 x 16384 x 2048, two CTAs: 14.4 against 14.6; 600 x 3840 x 1024, where two
    // would spare four k-blocks: 11.8 against 10.1).
    const long long tiles = max_tiles(a, few ? 32 : 128), sms = num_sms();
    const int nkb = (a.K + kBK - 1) / kBK;
    int split = 1;
    while (split < 8 && tiles * split * 2 <= sms && nkb >= 4 * split) split *= 2;
    if (nkb - nkb / split < 6) split = 1;
    if (split > 1) return few ? run<MODE, 1, 1>(a, split, s) : run<MODE, 0, 1>(a, split, s);
    return few ? run<MODE, 1, 0>(a, 1, s) : run<MODE, 0, 0>(a, 1, s);
}

}  // namespace

cudaError_t launch_scaled_gemm(const ScaledGemmArgs& a, cudaStream_t s) {
    return a.swiglu ? choose<kSwiglu>(a, s) : choose<kLinear>(a, s);
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

// quant.cu -- rows (or 128 x 128 blocks) of bf16 / fp32 numbers to e4m3 codes with one scale for
// each block of 128.
//
// For a block with largest finite magnitude A the scale is the smallest power of two s >= 2^-126
// with A / s <= 448 (the largest e4m3 number), 1 for a block of zeros, and the codes are x / s
// rounded to nearest, ties to even.  A power of two makes x / s exact, so a code is the one
// rounding of its input; NaN and +-inf become the e4m3 NaN and leave the scale to the rest of
// their block.
//
// Rows: half a warp per block of 128 (8 elements per lane, 16 B of bf16 or 32 B of fp32), so the
// maximum is four shuffles; each half warp takes kPer blocks with all their loads in flight.
#include "launch.h"
#include "scaled.cuh"

namespace moe {
namespace {

constexpr float kInf = __builtin_huge_valf();

template <bool BF16>
MOE_DEV void load8(const void* p, long long at, float (&v)[8]) {
    if constexpr (BF16) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at));
        const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(u[i]);
            v[2 * i + 1] = bf16_hi(u[i]);
        }
    } else {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
        const float4 a = __ldg(q), b = __ldg(q + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
}

// Largest magnitude of eight numbers; NaN is skipped (fmaxf), infinities are not.
MOE_DEV float amax8(const float (&v)[8]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
    return m;
}
MOE_DEV float amax8_finite(const float (&v)[8]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]) < kInf ? fabsf(v[i]) : 0.0f);
    return m;
}

MOE_DEV uint2 codes8(const float (&v)[8], float inv) {
    return make_uint2(cvt_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                      cvt_e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
}
MOE_DEV void inf_to_nan(float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (fabsf(v[i]) == kInf) v[i] = __int_as_float(0x7FFFFFFF);
}

// Rows, plain or of a dispatch:
//   kGather : output row j < P is row perm[j] / K of x when j < *dispatched (else it is left
//             alone), and row P + t is row t for the shared rows;
//   kScatter: the same rows from the tokens' side: row t of x is quantised once and written to
//             the slots inv[t K + k] >= 0, and to P + t.
enum { kPlain = 0, kGather = 1, kScatter = 2 };
struct QuantRows {
    const void* x;
    unsigned units;      // half warps with work: rows * ceil(nb / kPer)
    unsigned upr;        // of them per row
    long long ld;        // elements between rows of x
    int n, nb;           // columns (a multiple of 16), blocks of 128 per row
    uint8_t* codes;      // [rows, n]
    float* scales;       // [rows, nb]
    const int32_t* perm; // kGather
    const int32_t* dispatched;
    const int32_t* inv;  // kScatter
    long long P;
    int K, shared;
};

constexpr int kPer = 4;

template <bool BF16, int FORM>
__global__ void __launch_bounds__(256) quant_rows_kernel(const QuantRows a) {
    const int lane = threadIdx.x & 15;
    const unsigned unit = blockIdx.x * 16u + (threadIdx.x >> 4);
    const unsigned r = unit / a.upr;
    const int b0 = (int)(unit - r * a.upr) * kPer;
    const long long row = r;
    bool on = unit < a.units;
    pdl_launch_dependents();
    pdl_wait();  // the dispatch or x come from the kernels before
    long long src = row;
    if (FORM == kGather && on) {
        if (src >= a.P) src -= a.P;
        else if (src < *a.dispatched) src = a.perm[src] / a.K;
        else on = false;
    }
    float v[kPer][8];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        const int col = (b0 + u) * 128 + lane * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] = 0.0f;
        if (on && col < a.n) load8<BF16>(a.x, src * a.ld + col, v[u]);
    }
    uint2 q[kPer];
    float sc[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        float m = amax8(v[u]);
#pragma unroll
        for (int off = 8; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
        if (__any_sync(0xFFFFFFFFu, m == kInf)) {  // an infinity in one of the warp's two blocks
            m = amax8_finite(v[u]);
#pragma unroll
            for (int off = 8; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
            inf_to_nan(v[u]);
        }
        float inv;
        block_scale(m, sc[u], inv);
        q[u] = codes8(v[u], inv);
    }
    if (!on) return;
    auto put = [&](long long to) {
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int col = (b0 + u) * 128 + lane * 8;
            if (col < a.n) *reinterpret_cast<uint2*>(a.codes + to * a.n + col) = q[u];
            if (lane == 0 && b0 + u < a.nb) a.scales[to * a.nb + b0 + u] = sc[u];
        }
    };
    if (FORM == kScatter) {
        for (int k = 0; k < a.K; ++k) {
            const int32_t to = __ldg(a.inv + row * a.K + k);
            if (to >= 0) put(to);
        }
        if (a.shared) put(a.P + row);
    } else {
        put(row);
    }
}

// inv[perm[j]] = j for the dispatched slots (the others' pairs keep what inv held).
__global__ void __launch_bounds__(256) invert_kernel(const int32_t* perm, const int32_t* dispatched,
                                                     int P, int32_t* inv) {
    const int j = (int)(blockIdx.x * 256u + threadIdx.x);
    if (j < P && j < *dispatched) inv[perm[j]] = j;
}

// 128 x 128 blocks (weights): one CTA per block, its 16 half warps take eight rows each and
// keep them in registers between the maximum and the codes.
template <bool BF16>
__global__ void __launch_bounds__(256) quant_square_kernel(const void* x, long long rows,
                                                           long long ld, int n, int nb,
                                                           uint8_t* codes, float* scales) {
    __shared__ float part[8];
    const int lane = threadIdx.x & 15, hw = threadIdx.x >> 4;
    const long long br = blockIdx.x / nb;
    const int bc = (int)(blockIdx.x - br * nb);
    const int col = bc * 128 + lane * 8;
    pdl_launch_dependents();
    pdl_wait();
    float v[8][8];
    float m = 0.0f;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        const long long r = br * 128 + u * 16 + hw;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] = 0.0f;
        if (r < rows && col < n) load8<BF16>(x, r * ld + col, v[u]);
        m = fmaxf(m, amax8(v[u]));
    }
    if (__syncthreads_or(m == kInf)) {
        m = 0.0f;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            m = fmaxf(m, amax8_finite(v[u]));
            inf_to_nan(v[u]);
        }
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = fmaxf(m, part[w]);
    float s, inv;
    block_scale(m, s, inv);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        const long long r = br * 128 + u * 16 + hw;
        if (r < rows && col < n)
            *reinterpret_cast<uint2*>(codes + r * n + col) = codes8(v[u], inv);
    }
    if (threadIdx.x == 0) scales[br * nb + bc] = s;
}

QuantRows quant_rows(const void* x, long long rows, long long ld, int n, uint8_t* codes,
                     float* scales) {
    QuantRows a = {};
    a.x = x;
    a.nb = (n + 127) / 128;
    a.upr = (unsigned)((a.nb + kPer - 1) / kPer);
    a.units = (unsigned)(rows * a.upr);  // fewer than 2^31 blocks: checked by the caller
    a.ld = ld;
    a.n = n;
    a.codes = codes;
    a.scales = scales;
    return a;
}

}  // namespace

cudaError_t launch_quantize_rows(const void* x, int bf16, long long rows, int n, long long ld,
                                 uint8_t* codes, float* scales, cudaStream_t s) {
    const QuantRows a = quant_rows(x, rows, ld, n, codes, scales);
    const unsigned grid = (a.units + 15) / 16;
    return bf16 ? launch_kernel(quant_rows_kernel<true, kPlain>, dim3(grid), dim3(256), 0, s, a)
                : launch_kernel(quant_rows_kernel<false, kPlain>, dim3(grid), dim3(256), 0, s, a);
}

cudaError_t launch_quantize_square(const void* x, int bf16, long long rows, int n, long long ld,
                                   uint8_t* codes, float* scales, cudaStream_t s) {
    const int nb = (n + 127) / 128;
    const unsigned grid = (unsigned)((rows + 127) / 128 * nb);
    return bf16 ? launch_kernel(quant_square_kernel<true>, dim3(grid), dim3(256), 0, s, x, rows, ld,
                                n, nb, codes, scales)
                : launch_kernel(quant_square_kernel<false>, dim3(grid), dim3(256), 0, s, x, rows,
                                ld, n, nb, codes, scales);
}

cudaError_t launch_invert(const int32_t* perm, const int32_t* offsets, int E, long long P,
                          int32_t* inv, cudaStream_t s) {
    const cudaError_t err = cudaMemsetAsync(inv, 0xFF, sizeof(int32_t) * (size_t)P, s);
    if (err != cudaSuccess) return err;
    invert_kernel<<<(unsigned)((P + 255) / 256), 256, 0, s>>>(perm, offsets + E, (int)P, inv);
    return cudaGetLastError();
}

cudaError_t launch_quantize_dispatched(const void* x, const int32_t* perm, const int32_t* offsets,
                                       const int32_t* inv, int E, int K, long long P,
                                       long long shared_rows, int d, uint8_t* codes, float* scales,
                                       cudaStream_t s) {
    QuantRows a = quant_rows(x, inv ? P / K : P + shared_rows, d, d, codes, scales);
    a.perm = perm;
    a.dispatched = offsets + E;
    a.inv = inv;
    a.P = P;
    a.K = K;
    a.shared = shared_rows > 0;
    const dim3 grid((a.units + 15) / 16);
    return inv ? launch_kernel(quant_rows_kernel<true, kScatter>, grid, dim3(256), 0, s, a)
               : launch_kernel(quant_rows_kernel<true, kGather>, grid, dim3(256), 0, s, a);
}

}  // namespace moe

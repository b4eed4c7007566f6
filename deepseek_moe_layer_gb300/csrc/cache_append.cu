// cache_append.cu -- new tokens' rows into a paged cache, and the rotation of their queries.
//
// Row t of x (W columns): y = x normalised in its first Nc columns (RMS: x / rms(x) * w; with a
// bias the layer norm: (x - mean) / std * w + b), the R columns from r0 on turned pair by pair by
// the angle positions[t] * inv_freq[i], then rounded once, to bf16 or to e4m3 codes with one
// power-of-two scale per 128 columns, into row slots[t] of the cache.  Sums and values in fp32.  The
// angle is formed in turns from whole numbers (turn_of): at position 10^6 an fp32 product is off by
// 0.03 radians, and the device's 64-bit floating-point rate is a hundredth of its 32-bit one (4001 index
// keys: 18 us with angles in fp64, 7.7 so).
//
// The bound of a prompt's rows is memory (8192 rows of 576 columns with 128 heads' rotations move 287 MB),
// of a few tokens the launch.  A row is a warp's, 8 columns per lane and step, its sums five shuffles; queries
// go through blocks of their own, which make their tokens' cosines and sines once in shared memory
// while the first columns are on their way.  Measured: 287 MB in 65 us (4.4 TB/s), one token in 3.6 us;
// with 2 or 8 pieces in flight per thread instead of 4 68 and 88 us, with 3, 5 or 6 blocks per SM 68 .. 71.
// The lanes that hold rotated columns compute their angles one after the other (8 of 32 lanes, 4 or 8
// angles each, where a row has 64 rotated columns), which short rows in large numbers show.
#include "launch.h"
#include "scaled.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerBlock = kThreads / 32;
constexpr int kMaxChunks = 4;      // of 8 columns per lane: rows up to 1024 columns
constexpr int kMaxAngles = 2048;   // of a query block: tokens * R / 2
constexpr int kQueryUnits = 4;     // 16-byte columns (or pairs of them) in flight per thread

// cos and sin of the angle pos * f.  In turns it is pos * g with g = f / (2 pi), of which only what
// lies behind the point counts: g is held in units of 2^-64 turns (rounded down, off by less than two for
// f < 1 and twice as much with every doubling), and its product with pos modulo 2^64 is exact.  So the angle is
// off by less than 2^-25 turns at every position for f < 64: 2^-26 from its rounding to fp32, the rest from g.  (Sums of
// fp32 products with their errors: 2^-22.7 turns at 2^26, 2^-18 at 2^31.)
MOE_DEV void turn_of(int pos, float f, float& c, float& s) {
    constexpr uint64_t kTurn = 0x28BE60DB9391054Aull;  // 2^64 / (2 pi)
    const uint32_t bits = __float_as_uint(f), m = (bits | 0x800000u) << 8;
    const int e = (int)(bits >> 23 & 255u) - 126;      // |f| = m 2^(e - 32)
    uint64_t g = (uint64_t)(uint32_t)(kTurn >> 32) * m + __umulhi((uint32_t)kTurn, m);
    g = e > 0 ? g << min(e, 63) : g >> min(-e, 63);
    const uint64_t a = (uint64_t)(long long)pos * g;
    float t = fmaf((float)(uint32_t)a, 0x1p-63f, (float)(int)(a >> 32) * 0x1p-31f);  // half turns
    if (e == 129) t = f - f;                           // no finite frequency
    sincospif(t, &s, &c);
    if ((int)bits < 0) s = -s;
}

MOE_DEV void unpack8(const uint4& q, float (&v)[8]) {
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(u[i]);
        v[2 * i + 1] = bf16_hi(u[i]);
    }
}
MOE_DEV uint4 pack8(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
}

// Eight columns of one row from column c on, normalised where they belong to the first Nc.
MOE_DEV void normalise(const AppendArgs& a, int c, float mean, float r, float (&v)[8]) {
    if (c >= a.norm_cols) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = (v[i] - mean) * r * __ldg(a.norm_weight + c + i);
        if (a.norm_bias) v[i] += __ldg(a.norm_bias + c + i);
    }
}

template <bool F8>
MOE_DEV void append_row(const AppendArgs& a, long long t) {
    const int lane = threadIdx.x & 31;
    const long long slot = __ldg(a.slots + t);
    if (slot < 0 || slot >= a.rows) return;
    const uint16_t* x = static_cast<const uint16_t*>(a.x) + t * a.ldx;
    const int chunks = a.W / 8;
    uint4 raw[kMaxChunks];
#pragma unroll
    for (int i = 0; i < kMaxChunks; ++i) {
        const int c = lane + 32 * i;
        raw[i] = c < chunks ? __ldg(reinterpret_cast<const uint4*>(x) + c) : make_uint4(0, 0, 0, 0);
    }
    float mean = 0.0f, r = 1.0f;
    if (a.norm_cols) {
        // the mean first and then the squares about it: a row far from 0 keeps its digits
        float sum = 0.0f;
        if (a.norm_bias) {
#pragma unroll
            for (int i = 0; i < kMaxChunks; ++i)
                if (8 * (lane + 32 * i) < a.norm_cols) {
                    float v[8];
                    unpack8(raw[i], v);
#pragma unroll
                    for (int k = 0; k < 8; ++k) sum += v[k];
                }
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            mean = sum / (float)a.norm_cols;
            sum = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kMaxChunks; ++i)
            if (8 * (lane + 32 * i) < a.norm_cols) {
                float v[8];
                unpack8(raw[i], v);
#pragma unroll
                for (int k = 0; k < 8; ++k) sum += (v[k] - mean) * (v[k] - mean);
            }
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        r = rsqrtf(sum / (float)a.norm_cols + a.eps);
    }
    const int pos = a.R ? __ldg(a.positions + t) : 0;
#pragma unroll
    for (int i = 0; i < kMaxChunks; ++i) {
        const int c = 8 * (lane + 32 * i);
        if (32 * i >= chunks) break;
        float v[8];
        unpack8(raw[i], v);
        normalise(a, c, mean, r, v);
        const int at = c - a.rope_at;
        if (at >= 0 && at < a.R) {
            if (a.interleaved) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float cs, sn;
                    turn_of(pos, __ldg(a.inv_freq + at / 2 + k), cs, sn);
                    const float u = v[2 * k], w = v[2 * k + 1];
                    v[2 * k] = u * cs - w * sn;
                    v[2 * k + 1] = w * cs + u * sn;
                }
            } else {
                // the other half of each pair lies R / 2 columns away
                const bool low = at < a.R / 2;
                const int oc = low ? c + a.R / 2 : c - a.R / 2;
                float o[8];
                unpack8(__ldg(reinterpret_cast<const uint4*>(x + oc)), o);
                normalise(a, oc, mean, r, o);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    float cs, sn;
                    turn_of(pos, __ldg(a.inv_freq + (low ? at : at - a.R / 2) + k), cs, sn);
                    v[k] = low ? v[k] * cs - o[k] * sn : v[k] * cs + o[k] * sn;
                }
            }
        }
        if constexpr (F8) {
            // 16 lanes hold a block of 128; infinities become NaN and leave the scale to the others
            float m = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (fabsf(v[k]) == __int_as_float(0x7F800000)) v[k] = __int_as_float(0x7FFFFFFF);
                m = fmaxf(m, fabsf(v[k]));
            }
#pragma unroll
            for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            float s, inv;
            block_scale(m, s, inv);
            if (c < a.W) {
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.cache) + slot * a.W + c) =
                    make_uint2(cvt_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                               cvt_e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
                if ((lane & 15) == 0) a.scales[slot * (a.W / 128) + c / 128] = s;
            }
        } else if (c < a.W) {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.cache) + slot * a.W + c) = pack8(v);
        }
    }
}

// `per` tokens' queries, all their heads.  A unit is 8 columns (interleaved pairs) or 8 columns and
// the 8 that lie R / 2 further on.
MOE_DEV void rotate_queries(const AppendArgs& a, long long t0, int tokens) {
    __shared__ float2 turn[kMaxAngles];
    const int half = a.R / 2;
    const int upr = a.interleaved ? a.R / 8 : a.R / 16;  // units of a head
    const int units = tokens * a.H * upr;
    const uint16_t* q = static_cast<const uint16_t*>(a.q);
    uint16_t* out = static_cast<uint16_t*>(a.q_out);
    bool made = false;
    for (int u0 = threadIdx.x; u0 - (int)threadIdx.x < units; u0 += kThreads * kQueryUnits) {
        uint4 lo[kQueryUnits], hi[kQueryUnits];
        long long dst[kQueryUnits];
        int ang[kQueryUnits];
#pragma unroll
        for (int i = 0; i < kQueryUnits; ++i) {
            const int u = u0 + i * kThreads;
            if (u < units) {
                const int j = u % upr, th = u / upr, h = th % a.H, t = th / a.H;
                const uint16_t* s = q + (t0 + t) * a.q_token + (long long)h * a.q_head + 8 * j;
                dst[i] = (t0 + t) * a.o_token + (long long)h * a.o_head + 8 * j;
                ang[i] = t * half + (a.interleaved ? 4 * j : 8 * j);
                lo[i] = __ldg(reinterpret_cast<const uint4*>(s));
                if (!a.interleaved) hi[i] = __ldg(reinterpret_cast<const uint4*>(s + half));
            }
        }
        if (!made) {
            for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
                float c, s;
                turn_of(__ldg(a.positions + t0 + i / half), __ldg(a.inv_freq + i % half), c, s);
                turn[i] = make_float2(c, s);
            }
            __syncthreads();
            made = true;
        }
#pragma unroll
        for (int i = 0; i < kQueryUnits; ++i) {
            if (u0 + i * kThreads >= units) break;
            float v[8];
            unpack8(lo[i], v);
            if (a.interleaved) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 cs = turn[ang[i] + k];
                    const float x = v[2 * k], y = v[2 * k + 1];
                    v[2 * k] = x * cs.x - y * cs.y;
                    v[2 * k + 1] = y * cs.x + x * cs.y;
                }
            } else {
                float w[8];
                unpack8(hi[i], w);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 cs = turn[ang[i] + k];
                    const float x = v[k], y = w[k];
                    v[k] = x * cs.x - y * cs.y;
                    w[k] = y * cs.x + x * cs.y;
                }
                *reinterpret_cast<uint4*>(out + dst[i] + half) = pack8(w);
            }
            *reinterpret_cast<uint4*>(out + dst[i]) = pack8(v);
        }
    }
}

template <bool F8>
__global__ void __launch_bounds__(kThreads, 4) append_kernel(const AppendArgs a, unsigned row_blocks, int per) {
    if (blockIdx.x < row_blocks) {
        const long long t = (long long)blockIdx.x * kRowsPerBlock + (threadIdx.x >> 5);
        if (t < a.T) append_row<F8>(a, t);
    } else {
        const long long t0 = (long long)(blockIdx.x - row_blocks) * per;
        rotate_queries(a, t0, (int)min((long long)per, a.T - t0));
    }
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, cudaStream_t s) {
    const unsigned row_blocks = (unsigned)((a.T + kRowsPerBlock - 1) / kRowsPerBlock);
    unsigned q_blocks = 0;
    int per = 1;
    if (a.q) {
        // tokens per query block: enough units for its threads, within the table of angles
        const int upr = a.H * (a.interleaved ? a.R / 8 : a.R / 16);
        while (per * 2 * upr <= kThreads * kQueryUnits && per * a.R <= kMaxAngles && per * 2 <= a.T) per *= 2;
        q_blocks = (unsigned)((a.T + per - 1) / per);
    }
    return launch_kernel(a.scales ? append_kernel<true> : append_kernel<false>, dim3(row_blocks + q_blocks),
                         dim3(kThreads), 0, s, a, row_blocks, per);
}

}  // namespace moe

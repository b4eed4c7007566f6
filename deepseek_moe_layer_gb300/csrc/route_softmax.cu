// route_softmax.cu -- the group-limited softmax gate: softmax over ALL experts, selection by
// probability (plus an optional bias for balance) inside the best groups, weights that are the
// probabilities themselves or renormalised over the selection.
//
// For a row of logits l (a NaN counts as -inf), m = max_j l_j and Z = sum_j exp(l_j - m):
//     p_j = exp(l_j - m) / Z                         (all 0 when m = -inf; the +inf logits
//                                                     share the probability when m = +inf)
//     v_j = p_j + b_j                                (b = 0 without a bias; NaN counts as -inf)
//     group score = max of v over the group; the topk_group best groups stay, lower index
//                   first among equal scores; experts of the other groups are never selected
//     the K largest v, larger first, lower index first among equals
//     w_k = p_k, divided by sum of the selected p when K > 1 and norm is set (0 when that sum
//           is 0), times the scaling factor
//
// Selection is exact.  Without a bias it compares the logits themselves (softmax is strictly
// increasing).  With a bias v is computed in fp32, and where two neighbours in the order stand
// closer than its rounding can tell (kNear below) the row is selected again in fp64.
//
// One warp per row; lane l holds experts l, l + 32, ... so that a row is read in whole lines.
// An arg-max is one redux.max over order-preserving keys and one redux.min over the indices of
// the maxima.
#include "common.cuh"
#include "launch.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;

// Order-preserving keys: -0 == +0, NaN as -inf; 0 is below every value and marks a slot that
// cannot be selected.
MOE_DEV uint32_t order_key(float f) {
    if (f != f) f = __int_as_float(0xFF800000);
    const uint32_t u = __float_as_uint(f + 0.0f);  // -0 + 0 = +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
MOE_DEV unsigned long long order_key(double f) {
    if (f != f) f = -__longlong_as_double(0x7FF0000000000000ll);
    const unsigned long long u = (unsigned long long)__double_as_longlong(f + 0.0);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

MOE_DEV uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kFull, v); }
MOE_DEV unsigned long long warp_max(unsigned long long v) {
    const uint32_t hi = (uint32_t)(v >> 32);
    const uint32_t top = __reduce_max_sync(kFull, hi);
    const uint32_t lo = __reduce_max_sync(kFull, hi == top ? (uint32_t)v : 0u);
    return ((unsigned long long)top << 32) | lo;
}
template <typename T>
MOE_DEV T warp_sum(T v) {
#pragma unroll
    for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
    return v;
}

MOE_DEV float exp_of(float x) { return expf(x); }
MOE_DEV double exp_of(double x) { return exp(x); }

// The row's selection with values in V (float or double) and keys in Key.  On return lane k < K
// holds the k-th selected expert and its probability.  Returns, with NEAR, whether some order
// that decided the result was closer than fp32 can tell (the same in every lane).
template <int EPL, typename V, typename Key, bool NEAR>
MOE_DEV bool select_row(const RouteArgs& a, const float (&l)[EPL], float m, int lane, int& my_idx,
                        V& my_p) {
    const int E = a.E, G = a.n_group, K = a.top_k, eg = E / G;
    const float inf = __int_as_float(0x7F800000);
    V e[EPL];
    V z = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        // m = -inf: every probability 0; m = +inf: the limit, shared by the +inf logits
        e[i] = m == inf ? (l[i] == inf ? (V)1 : (V)0)
                        : m == -inf ? (V)0 : exp_of((V)l[i] - (V)m);
        if (lane + 32 * i >= E) e[i] = 0;
        z += e[i];
    }
    z = warp_sum(z);
    const V rz = z > 0 ? (V)1 / z : (V)0;
    Key key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int x = lane + 32 * i;
        e[i] *= rz;
        if constexpr (NEAR || sizeof(V) == 8)
            key[i] = x < E ? order_key(e[i] + (V)a.bias[x]) : (Key)0;
        else
            key[i] = x < E ? order_key(l[i]) : (Key)0;
    }
    const float pmax = (float)rz;  // the largest probability (exp(0) / Z)
    // fp32: p is off by at most EPL + 11 halves of 2^-23 of itself (EPL + 4 sums of Z, expf's
    // two steps, the reciprocal, the product, to first order), v by 2^-24 |v| more; two values
    // further apart than twice that stand in their true order
    constexpr float kNear = (EPL + 12) * 0x1p-23f;
    bool near = false;

    if (G > a.topk_group) {
        Key mine = 0;  // lane g (< G): the key of group g's best expert
        for (int g = 0; g < G; ++g) {
            Key b = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const int x = lane + 32 * i;
                if (x >= g * eg && x < (g + 1) * eg && key[i] > b) b = key[i];
            }
            b = warp_max(b);
            if (lane == g) mine = b;
        }
        int rank = 0;
        for (int h = 0; h < G; ++h) {
            const Key o = __shfl_sync(kFull, mine, h);
            rank += o > mine || (o == mine && h < lane);
        }
        const unsigned kept = __ballot_sync(kFull, lane < G && rank < a.topk_group);
        if constexpr (NEAR) {
            const unsigned last = __ballot_sync(kFull, lane < G && rank == a.topk_group - 1);
            const unsigned next = __ballot_sync(kFull, lane < G && rank == a.topk_group);
            const uint32_t k0 = __shfl_sync(kFull, mine, __ffs(last) - 1);
            const uint32_t k1 = __shfl_sync(kFull, mine, __ffs(next) - 1);
            const float v0 = __uint_as_float((k0 & 0x80000000u) ? (k0 & 0x7FFFFFFFu) : ~k0);
            const float v1 = __uint_as_float((k1 & 0x80000000u) ? (k1 & 0x7FFFFFFFu) : ~k1);
            near = !(v0 - v1 > kNear * pmax + 0x1p-22f * fabsf(v0));
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int x = lane + 32 * i;
            if (x < E && !((kept >> (x / eg)) & 1u)) key[i] = 0;
        }
    }

    // lane's best slot; only the lane whose slot was taken looks again
    Key bk = 0;
    int bi = 0;
    V bp = 0;
    auto look = [&] {
        bk = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (key[i] > bk) {
                bk = key[i];
                bi = i;
                bp = e[i];
            }
    };
    look();
    float before = 0.0f;  // NEAR: the value taken last
    const int selectable = min(a.topk_group, G) * eg;
    const int rounds = NEAR && K < selectable ? K + 1 : K;
    for (int r = 0; r < rounds; ++r) {
        const Key top = warp_max(bk);
        const unsigned x = (unsigned)(lane + 32 * bi);
        const unsigned w = __reduce_min_sync(kFull, bk == top ? x : 0xFFFFFFFFu);
        const V p = __shfl_sync(kFull, bp, (int)(w & 31u));
        if constexpr (NEAR) {
            const uint32_t t = (uint32_t)top;
            const float v = __uint_as_float((t & 0x80000000u) ? (t & 0x7FFFFFFFu) : ~t);
            if (r > 0) near |= !(before - v > kNear * pmax + 0x1p-22f * fabsf(before));
            before = v;
        }
        if (r < K && lane == r) {
            my_idx = (int)w;
            my_p = p;
        }
        if (bk == top && x == w) {
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (i == bi) key[i] = 0;
            look();
        }
    }
    return near;
}

template <int EPL>
__global__ void __launch_bounds__(256, EPL <= 8 ? 3 : 1) route_grouped_kernel(const RouteArgs a) {
    pdl_launch_dependents();
    pdl_wait();  // the logits come from the kernel before
    const int lane = threadIdx.x & 31, E = a.E, K = a.top_k;
    const long long nwarps = (long long)gridDim.x * 8;
    for (long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); row < a.rows;
         row += nwarps) {
        float l[EPL];
        float m = __int_as_float(0xFF800000);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int x = lane + 32 * i;
            float v = 0.0f;
            if (x < E) {
                if (a.bf16) {
                    v = __uint_as_float(
                        (uint32_t) static_cast<const unsigned short*>(a.logits)[row * E + x] << 16);
                } else {
                    const float* q = static_cast<const float*>(a.logits) + row * E + x;
                    for (int s = 0; s < a.nsplit; ++s) v += q[(long long)s * a.split_stride];
                }
                if (a.logit_offset) v += a.logit_offset[x];
                if (a.logits_out) a.logits_out[row * E + x] = v;
                if (v != v) v = __int_as_float(0xFF800000);
                m = fmaxf(m, v);
            }
            l[i] = v;
        }
#pragma unroll
        for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));

        int idx = 0;
        float p = 0.0f;
        if (a.bias) {
            if (select_row<EPL, float, uint32_t, true>(a, l, m, lane, idx, p)) {
                double pd = 0.0;
                select_row<EPL, double, unsigned long long, false>(a, l, m, lane, idx, pd);
                p = (float)pd;
            }
        } else {
            select_row<EPL, float, uint32_t, false>(a, l, m, lane, idx, p);
        }
        if (a.norm && K > 1) {
            const float sum = warp_sum(lane < K ? p : 0.0f);
            p = sum > 0.0f ? p / sum : 0.0f;
        }
        if (lane < K) {
            a.inds[row * K + lane] = idx;
            a.scores[row * K + lane] = p * a.scale;
        }
    }
}

template <int EPL>
cudaError_t launch_epl(const RouteArgs& a, cudaStream_t s) {
    const long long want = (a.rows + 7) / 8;
    const long long cap = (long long)(EPL <= 8 ? 3 : 1) * num_sms();
    return launch_kernel(route_grouped_kernel<EPL>, dim3((unsigned)(want < cap ? want : cap)),
                         dim3(256), 0, s, a);
}

}  // namespace

cudaError_t launch_route_grouped(const RouteArgs& a, cudaStream_t s) {
    if (a.rows == 0) return cudaSuccess;
    switch ((a.E + 31) / 32) {
        case 1: return launch_epl<1>(a, s);
        case 2: return launch_epl<2>(a, s);
        case 3: return launch_epl<3>(a, s);
        case 4: return launch_epl<4>(a, s);
        case 5: return launch_epl<5>(a, s);
        case 6: return launch_epl<6>(a, s);
        case 7: return launch_epl<7>(a, s);
        case 8: return launch_epl<8>(a, s);
        default: break;
    }
    return a.E <= 512 ? launch_epl<16>(a, s) : launch_epl<32>(a, s);
}

}  // namespace moe

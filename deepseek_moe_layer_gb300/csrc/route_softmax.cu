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
// Selection is exact.  Without a bias it compares the logits themselves: softmax is strictly
// increasing, and where p tells two experts no longer apart (finite logits beside a +inf one, whose
// p are all 0) the larger logit still comes first.  With a bias v is computed in fp32, and where that cannot tell the order (two
// neighbours among the chosen, or the last of them and any of the others, closer than far_apart
// below) the row is selected again in fp64.
//
// One warp per row; lane l holds the experts l EPL, .. l EPL + EPL - 1.  An arg-max is one
// redux.max over order-preserving keys and one redux.min over the indices of the maxima; a group
// that is a power of two of whole lanes has its maximum after that many shuffles, any other one
// after a redux of its own.  What bounds a large batch is instruction issue (848 a row with 160
// experts, 6 chosen from 3 of 8 groups; the issue slots are three quarters full) with enough rows
// under way to hide the chain of some thirty warp steps: the gate without a bias carries neither
// probabilities nor the fp64 path, and that path is a function of its own that reads the row
// again, so that it takes no registers.  16384 such rows: 15.6 us (10.5 MB of logits: 1.7 us), with
// a bias 22.5 .. 29; 16384 x 256, 8 from 4 of 8 groups, with a bias 33 .. 47, as few or many of the
// rows go through fp64 (one of them is ten times a row's time, which shows when it comes last).
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

// exp(l - m), or the limit of the probabilities' numerators: shared by the +inf logits when
// m = +inf, 0 when m = -inf.
template <typename V>
MOE_DEV V numerator(float l, float m) {
    const float inf = __int_as_float(0x7F800000);
    if (m == inf) return l == inf ? (V)1 : (V)0;
    if (m == -inf) return (V)0;
    return exp_of((V)l - (V)m);
}

MOE_DEV float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// The logit of expert x: the partial sums in split order, plus the optional offset.
MOE_DEV float logit(const RouteArgs& a, long long row, int x) {
    float v = 0.0f;
    if (a.bf16) {
        v = __uint_as_float((uint32_t) static_cast<const unsigned short*>(a.logits)[row * a.E + x] << 16);
    } else {
        const float* q = static_cast<const float*>(a.logits) + row * a.E + x;
        for (int s = 0; s < a.nsplit; ++s) v += q[(long long)s * a.split_stride];
    }
    return a.logit_offset ? v + a.logit_offset[x] : v;
}

// Sets the keys of the dropped groups' experts to 0.  Returns the kept groups' border: the last
// kept and the best dropped group's keys.
template <int EPL, typename Key>
MOE_DEV void keep_groups(const RouteArgs& a, Key (&key)[EPL], int lane, Key& last, Key& next) {
    const int G = a.n_group, E = a.E, eg = E / G;
    const int lpg = eg % EPL == 0 ? eg / EPL : 0;  // lanes per group
    const bool whole = lpg > 0 && (lpg & (lpg - 1)) == 0;
    Key mine = 0;  // lane g (< G): the key of group g's best expert
    if (whole) {
        Key b = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) b = key[i] > b ? key[i] : b;
        for (int off = 1; off < lpg; off <<= 1) {
            const Key o = __shfl_xor_sync(kFull, b, off);
            b = o > b ? o : b;
        }
        mine = __shfl_sync(kFull, b, min(lane, G - 1) * lpg);
    } else {
        for (int g = 0; g < G; ++g) {
            Key b = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const int x = lane * EPL + i;
                if (x >= g * eg && x < (g + 1) * eg && key[i] > b) b = key[i];
            }
            b = warp_max(b);
            if (lane == g) mine = b;
        }
    }
    int rank = 0;
    for (int h = 0; h < G; ++h) {
        const Key o = __shfl_sync(kFull, mine, h);
        rank += o > mine || (o == mine && h < lane);
    }
    if (lane >= G) rank = 64;
    const unsigned kept = __ballot_sync(kFull, rank < a.topk_group);
    last = __shfl_sync(kFull, mine, __ffs(__ballot_sync(kFull, rank == a.topk_group - 1)) - 1);
    next = __shfl_sync(kFull, mine, __ffs(__ballot_sync(kFull, rank == a.topk_group)) - 1);
    if (whole) {
        const bool in = (kept >> min(lane / lpg, 31)) & 1u;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (!in) key[i] = 0;
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (!((kept >> min((lane * EPL + i) / eg, 31)) & 1u)) key[i] = 0;
    }
}

// A lane's best slot, which the arg-max rounds take from.
template <int EPL, typename Key>
MOE_DEV void look(const Key (&key)[EPL], Key& bk, int& bi) {
    bk = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (key[i] > bk) {
            bk = key[i];
            bi = i;
        }
}

// One round: the expert with the largest key, the lowest index first among equals; its slot is
// taken out.  `top`: its key.
template <int EPL, typename Key>
MOE_DEV int take(Key (&key)[EPL], Key& bk, int& bi, int lane, Key& top) {
    top = warp_max(bk);
    const unsigned x = (unsigned)(lane * EPL + bi);
    const unsigned w = __reduce_min_sync(kFull, bk == top ? x : 0xFFFFFFFFu);
    if (bk == top && x == w) {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (i == bi) key[i] = 0;
        look(key, bk, bi);
    }
    return (int)w;
}

// The row again in fp64: the lane's expert and its probability.  Not inlined, so that its
// registers do not count for the rows that never come here.
template <int EPL>
__device__ __noinline__ void select_exact(const RouteArgs& a, long long row, int* idx, float* p) {
    const int lane = threadIdx.x & 31;
    float l[EPL];
    float m = __int_as_float(0xFF800000);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int x = lane * EPL + i;
        l[i] = x < a.E ? logit(a, row, x) : __int_as_float(0xFF800000);
        if (l[i] != l[i]) l[i] = __int_as_float(0xFF800000);
        m = fmaxf(m, l[i]);
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
    double z = 0.0, e[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        e[i] = lane * EPL + i < a.E ? numerator<double>(l[i], m) : 0.0;
        z += e[i];
    }
    z = warp_sum(z);
    const double rz = z > 0.0 ? 1.0 / z : 0.0;
    unsigned long long key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int x = lane * EPL + i;
        key[i] = x < a.E ? order_key(e[i] * rz + (double)a.bias[x]) : 0ull;
    }
    unsigned long long last, next, bk, top;
    int bi = 0;
    if (a.n_group > a.topk_group) keep_groups(a, key, lane, last, next);
    look(key, bk, bi);
    for (int r = 0; r < a.top_k; ++r) {
        const int w = take(key, bk, bi, lane, top);
        if (lane == r) *idx = w;
    }
    if (lane < a.top_k) {
        float v = logit(a, row, *idx);
        if (v != v) v = __int_as_float(0xFF800000);
        *p = (float)(z > 0.0 ? numerator<double>(v, m) / z : 0.0);
    }
}

// Above this gap two fp32 values v = p + b stand in their true order.  In units of 2^-24: an own
// numerator is off by 4 of itself (expf), its product and Z's reciprocal by 2 more, and the rounding
// of l - m by |l - m| of it, with x exp(-x) < 0.4 of the largest; Z by 4, by EPL + 4 sums and by the
// mean of |l - m| under p (< 5 with 1024 experts), which moves both values alike and so counts for
// their difference; the two sums with the bias by |v| each.
template <int EPL>
MOE_DEV float far_apart(float p, float q, float pmax, float v) {
    return 0x1p-24f * (6.0f * (p + q) + (EPL + 13) * fabsf(p - q) + 0.8f * pmax + 2.0f * fabsf(v)) *
           1.001f;
}

template <int EPL, bool BIAS>
__global__ void __launch_bounds__(256, EPL <= 8 ? (BIAS ? 4 : 5) : 1)
    route_grouped_kernel(const __grid_constant__ RouteArgs a) {
    pdl_launch_dependents();
    pdl_wait();  // the logits come from the kernel before
    const int lane = threadIdx.x & 31, E = a.E, K = a.top_k;
    const long long nwarps = (long long)gridDim.x * 8;
    for (long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); row < a.rows;
         row += nwarps) {
        uint32_t key[EPL];  // of the logits (0: no expert)
        uint32_t mk = 0;
        const bool plain = !a.bf16 && a.nsplit == 1 && !a.logit_offset;
        const float* q = static_cast<const float*>(a.logits) + row * E;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int x = lane * EPL + i;
            key[i] = 0;
            if (x < E) {
                const float v = plain ? q[x] : logit(a, row, x);
                if (a.logits_out) a.logits_out[row * E + x] = v;
                key[i] = order_key(v);
                mk = max(mk, key[i]);
            }
        }
        const float m = key_value(warp_max(mk));
        float z = 0.0f, e[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            e[i] = key[i] ? numerator<float>(key_value(key[i]), m) : 0.0f;
            z += e[i];
        }
        z = warp_sum(z);
        const float rz = z > 0.0f ? 1.0f / z : 0.0f;  // also the largest probability
        if (BIAS) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const int x = lane * EPL + i;
                e[i] *= rz;
                if (x < E) key[i] = order_key(e[i] + __ldg(a.bias + x));
            }
        }
        bool near = false;
        if (a.n_group > a.topk_group) {
            uint32_t last, next;
            keep_groups(a, key, lane, last, next);
            const float v = key_value(last);
            if (BIAS) near = !(v - key_value(next) > far_apart<EPL>(rz, 0.0f, rz, v) + far_apart<EPL>(rz, rz, rz, v));
        }
        uint32_t bk, top;
        int bi = 0, idx = 0;
        look(key, bk, bi);
        float p = 0.0f, before = 0.0f, pb = 0.0f;
        for (int r = 0; r < K; ++r) {
            float pe = 0.0f;
            if (BIAS) {
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (i == bi) pe = e[i];
            }
            const int w = take(key, bk, bi, lane, top);
            const float v = key_value(top);
            if (BIAS) {
                pe = __shfl_sync(kFull, pe, w / EPL);
                if (r > 0) near |= !(before - v > far_apart<EPL>(pb, pe, rz, before));
                before = v;
                pb = pe;
            }
            if (lane == r) {
                idx = w;
                p = BIAS ? pe : v;
            }
        }
        if (BIAS && K < a.topk_group * (E / a.n_group)) {
            // the last one chosen has to stand clear of all the others, not of the best of them
            // alone: one further behind with a larger p is off by more (the bound is convex in p,
            // so its ends 0 and rz cover them all; each one's own p decides where they do not)
            if (!(before - key_value(warp_max(bk)) > fmaxf(far_apart<EPL>(pb, 0.0f, rz, before),
                                                           far_apart<EPL>(pb, rz, rz, before)))) {
                bool close = false;
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    close |= key[i] && !(before - key_value(key[i]) > far_apart<EPL>(pb, e[i], rz, before));
                near |= __any_sync(kFull, close);
            }
        }
        if (BIAS) {
            if (near) select_exact<EPL>(a, row, &idx, &p);
        } else {
            p = numerator<float>(p, m) * rz;  // p held the logit
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
    // a row per warp: rows that go through fp64 (some ten times a row's time) are overtaken by the
    // others, and the scheduler spreads the rest better than a stride (16384 x 160: 18.2 -> 15.6 us)
    const long long want = (a.rows + 7) / 8;
    const dim3 grid((unsigned)(want < 0x7FFFFFFF ? want : 0x7FFFFFFF));
    return a.bias ? launch_kernel(route_grouped_kernel<EPL, true>, grid, dim3(256), 0, s, a)
                  : launch_kernel(route_grouped_kernel<EPL, false>, grid, dim3(256), 0, s, a);
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

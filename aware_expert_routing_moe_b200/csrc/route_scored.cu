// Routing with scores, balance bias and expert groups (sm_100a).
//
// route_choose_kernel : a warp per token: scores, group values, top-k,
//                       weights; per run of tokens, how many chose each expert.
// route_lists_kernel  : expert-major token lists from the choices: a block
//                       per run of tokens; an entry's place is the expert's
//                       first place + the entries of earlier runs + its rank
//                       among the run's tokens (bit masks, no atomics on
//                       places: the lists do not depend on scheduling).
// Batches of up to ONE_LAUNCH tokens get their lists from the last block of
// the first kernel to finish.
//
// The choice is that of the values c = s + bias in fp64, equal values to the
// lower index.  The scores are computed in fp64 by a short exp and a
// reciprocal (about 25 operations an expert); the warp then ranks 28-bit
// images of the values, which one warp reduction each finds the largest of,
// and ranks the fp64 values themselves only for a token in which two
// neighbours of the order it uses are too close for that: about one random
// token in 10^4 with fp32 logits, and every exact tie, which logits of bf16
// precision have in 22 to 37 % of tokens (64 to 256 experts, k = 8).  Without
// a bias, and with groups valued by their best expert, the logits rank (a
// score is monotone in its logit) and no score but the chosen ones is
// computed, except among logits so near 0 that fp64 scores are equal.
//
// Bound by instructions: 1970 a token with 256 experts in 8 groups, sigmoid
// scores and a bias (1570 without the groups, 1110 where the logits rank).
// Measured: 1 token 8.6 us, 77 tokens (128 experts) 8.9 us, 8192 tokens 40 us
// (under ncu the choice 28, the lists 12.5).  Exact ties: 8192 tokens, 128
// experts, softmax 27 us with bf16-valued logits, 20 with fp32 ones.  With
// fp32 scores and fp64 only for close calls a long batch took as long: some
// token of it always needed fp64, at the latency of the whole fp64 path.
#include <cfloat>
#include <cmath>

#include "blocks.h"

namespace moe {
namespace {

constexpr unsigned ALL = 0xffffffffu;
constexpr int SUB = 32;          // tokens whose choices of one expert are one 32-bit mask
constexpr int RUNS_MAX = 256;    // runs of tokens (blocks) of a long batch
constexpr int THREADS = 512;     // of both kernels
constexpr int WARPS = THREADS / 32;
// One launch up to this many tokens, a token per warp; the last block's work
// grows with the batch, and above it the second kernel is cheaper.
constexpr int ONE_LAUNCH = 512;

// Tokens per block of the first kernel.
int run_tokens(int B) {
    if (B <= ONE_LAUNCH) return WARPS;
    const int subs = (B + SUB - 1) / SUB;
    return SUB * ((subs + RUNS_MAX - 1) / RUNS_MAX);
}

// The histograms of a workspace start behind what any entry point keeps from
// call to call in it.
constexpr size_t HIST_OFFSET = MOE_GEMM_WORKSPACE_BYTES;
static_assert(sizeof(Counters) <= HIST_OFFSET && sizeof(BlocksControl) <= HIST_OFFSET, "kept counters");
static_assert(sizeof(BlocksControl) % 256 == 0, "workspace sizes are multiples of 256 bytes");

// Counts of a run: whole 16-byte pieces.
__host__ __device__ constexpr int hist_pitch(int E) { return (E + 7) / 8 * 8; }

struct RouteArgs {
    const float *logits, *bias;
    int B, E, k, run, runs, one_launch;
    moe_scoring_t rule;
    int32_t *sel_idx;
    float *sel_w;
    unsigned *ticket;  // blocks finished (one launch)
    uint16_t *hist;    // [runs][hist_pitch(E)]
    moe_lists_t lists;
};

// Largest value over the warp; the lowest index among equal ones (value
// -inf: no candidate).
__device__ __forceinline__ void warp_best(double &v, int &e) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        const double ov = __shfl_xor_sync(ALL, v, o);
        const int oe = __shfl_xor_sync(ALL, e, o);
        if (ov > v || (ov == v && oe < e)) {
            v = ov;
            e = oe;
        }
    }
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(ALL, v, o);
    return v;
}
__device__ __forceinline__ float warp_maxf(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(ALL, v, o));
    return v;
}

// Adding this to |v| < 2^31 rounds v to an integer, found in the low word.
constexpr double ROUND = 6755399441055744.0;  // 1.5 * 2^52

// exp(x) for x <= 0 in fp64: x = n ln2 + r with ln2 split into its first 32
// bits and a tail, the Taylor series of exp(r) to degree 12 (|r| <= 0.347:
// the rest is below 2e-16), 2^n through the exponent field.  -700 <= x.
__device__ __forceinline__ double exp_neg(double x) {
    const double t = fma(x, 1.4426950408889634, ROUND), n = t - ROUND;
    double r = fma(n, -2977044472.0 / 4294967296.0, x);
    r = fma(n, 4.2009150726810846e-11, r);
    double p = 1.0 / 479001600.0;
    p = fma(p, r, 1.0 / 39916800.0);
    p = fma(p, r, 1.0 / 3628800.0);
    p = fma(p, r, 1.0 / 362880.0);
    p = fma(p, r, 1.0 / 40320.0);
    p = fma(p, r, 1.0 / 5040.0);
    p = fma(p, r, 1.0 / 720.0);
    p = fma(p, r, 1.0 / 120.0);
    p = fma(p, r, 1.0 / 24.0);
    p = fma(p, r, 1.0 / 6.0);
    p = fma(p, r, 0.5);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    return __hiloint2double(__double2hiint(p) + (__double2loint(t) << 20), __double2loint(p));
}
// 1 / y for 1 <= y <= 2: an fp32 reciprocal and two Newton steps.
__device__ __forceinline__ double reciprocal(double y) {
    double r = static_cast<double>(__fdividef(1.0f, static_cast<float>(y)));
    r = fma(r, fma(-y, r, 1.0), r);
    return fma(r, fma(-y, r, 1.0), r);
}
// Scores below exp(-700), 1e-304, are 0 (both kinds).
__device__ __forceinline__ double sigmoid(float l) {
    const double z = exp_neg(static_cast<double>(fmaxf(-fabsf(l), -700.0f)));
    const double r = reciprocal(1.0 + z);
    return l >= 0.0f ? r : l >= -700.0f ? z * r : 0.0;
}
// exp(l - top)
__device__ __forceinline__ double exp_from(float l, float top) {
    const double x = static_cast<double>(l) - static_cast<double>(top);
    return x >= -700.0 ? exp_neg(x) : 0.0;
}
__device__ __forceinline__ int round_int(double v) { return __double2loint(v + ROUND); }

// Logits for which fp64 scores keep the order of the logits: not near 1 for
// sigmoid scores, at most 600 below the largest for softmax.  Below
// TINY_LOGIT neighbouring fp32 values can be nearer than fp64 scores tell
// (from it on they are 2^-40 apart, and l - top is rounded by 2^-44 at most):
// close calls among such logits are decided by the scores.
constexpr float TOP_LOGIT = 16.0f, LOW_LOGIT = -600.0f, TINY_LOGIT = 1.0f / 65536.0f;
// Images: 28 bits of value (1 to 2^27 + 1; a unit is 2^-26 to 2^-25 of the
// bound on the values' magnitude) over 4 bits of slot.  Rounding moves a value
// by half a unit, so two that are more than NEAR units apart are in order;
// sums of two, SUM_NEAR.
constexpr int SLOT_BITS = 4, NEAR = 2, SUM_NEAR = 4;

// Experts lane + 32 i, i < NI.
template <int NI>
struct Token {
    double c[NI];       // values; -inf: not to choose from
    unsigned image[NI]; // 0: not to choose from

    // Groups whose experts stay, and the choice (lane j: the j-th expert,
    // -1 none), by the images; false: too close to call.
    __device__ __forceinline__ bool by_image(const RouteArgs &a, const int (&group)[NI], unsigned *row, int &mine) {
        const int lane = threadIdx.x & 31;
        bool sure = true;
        if (a.rule.groups > 1) {
            const int G = a.rule.groups, per = a.E / G;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int e = lane + 32 * i;
                if (e < a.E) row[e + group[i]] = image[i] >> SLOT_BITS;  // groups skewed by a bank each
            }
            __syncwarp();
            unsigned b1 = 0u, b2 = 0u;
            if (lane < G) {
                const unsigned *mem = row + lane * (per + 1);
#pragma unroll 8
                for (int j = 0; j < per; ++j) {
                    const unsigned v = mem[j];
                    b2 = max(b2, min(b1, v));
                    b1 = max(b1, v);
                }
            }
            // a group of one such expert has half the sum: too close to say
            const bool two = a.rule.group_best == 2;
            if (two && __any_sync(ALL, b1 != 0u && b2 == 0u)) return false;
            unsigned value = two ? b1 + b2 : b1, keep = 0u, before = 0xffffffffu;
            const unsigned near = two ? SUM_NEAR : NEAR;
            for (int j = 0; j <= a.rule.top_groups; ++j) {
                const unsigned m = __reduce_max_sync(ALL, value);
                if (m == 0u) break;
                sure = sure && before - m > near;
                before = m;
                if (j == a.rule.top_groups) break;
                const int g = __ffs(__ballot_sync(ALL, value == m)) - 1;
                keep |= 1u << g;
                if (lane == g) value = 0u;
            }
            if (!sure) return false;
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if (!((keep >> group[i]) & 1u)) image[i] = 0u;
        }
        unsigned best = 0u, before = 0xffffffffu;
#pragma unroll
        for (int i = 0; i < NI; ++i) best = max(best, image[i]);
        mine = -1;
        for (int j = 0; j <= a.k; ++j) {
            const unsigned m = __reduce_max_sync(ALL, best);
            if (m == 0u) break;
            const unsigned who = __ballot_sync(ALL, best == m);
            sure = sure && (before >> SLOT_BITS) - (m >> SLOT_BITS) > NEAR && (who & (who - 1u)) == 0u;
            before = m;
            if (j == a.k) break;
            if (lane == j) mine = (__ffs(who) - 1) + 32 * static_cast<int>((1u << SLOT_BITS) - 1u - (m & ((1u << SLOT_BITS) - 1u)));
            best = 0u;
#pragma unroll
            for (int i = 0; i < NI; ++i) {  // (another lane's equal image makes the token unsure)
                if (image[i] == m) image[i] = 0u;
                best = max(best, image[i]);
            }
        }
        return sure;
    }
};

// The scores of logits c (-inf: not to choose from), in their place.
template <int NI>
__device__ __forceinline__ void to_scores(double (&c)[NI], bool sig, float shift) {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        if (c[i] == -INFINITY) continue;
        const float l = static_cast<float>(c[i]);
        c[i] = sig ? sigmoid(l) : exp_from(l, shift);
        sum += c[i];
    }
    if (sig) return;
    const double inv = 1.0 / warp_sum(sum);  // (not of a token that has no expert: its images are sure)
#pragma unroll
    for (int i = 0; i < NI; ++i)
        if (c[i] > -INFINITY) c[i] *= inv;
}

// The same by the values c (overwritten); logits (by_logit) by their scores
// where a tiny one has another near it.
template <int NI>
__device__ __noinline__ int by_value(const RouteArgs &a, double (&c)[NI], double *row, bool by_logit, float shift) {
    if (by_logit) {
        bool tiny = false;
        int near_zero = 0;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const bool near = fabs(c[i]) < TINY_LOGIT;
            near_zero += near;
            tiny = tiny || (near && c[i] != 0.0);
        }
        if (__any_sync(ALL, tiny) && __reduce_add_sync(ALL, near_zero) > 1)
            to_scores<NI>(c, a.rule.score == MOE_SCORE_SIGMOID, shift);
    }
    const int lane = threadIdx.x & 31;
    const int G = a.rule.groups, per = a.E / G;
    if (G > 1) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (lane + 32 * i < a.E) row[lane + 32 * i] = c[i];
        __syncwarp();
        double b1 = -INFINITY, b2 = -INFINITY;
        if (lane < G)
            for (int j = 0; j < per; ++j) {
                const double v = row[lane * per + j];
                if (v > b1) {
                    b2 = b1;
                    b1 = v;
                } else if (v > b2) b2 = v;
            }
        double value = b1;
        if (a.rule.group_best == 2 && b2 > -INFINITY) value += b2;
        unsigned keep = 0;
        for (int j = 0; j < a.rule.top_groups; ++j) {
            double v = (keep >> lane) & 1u ? -INFINITY : value;
            int g = lane;
            warp_best(v, g);
            if (v > -INFINITY) keep |= 1u << g;
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E && !((keep >> (e / per)) & 1u)) c[i] = -INFINITY;
        }
    }
    int mine = -1;
    for (int j = 0; j < a.k; ++j) {
        double v = -INFINITY;
        int e = 1 << 20;
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (c[i] > v) {
                v = c[i];
                e = lane + 32 * i;
            }
        warp_best(v, e);
        if (v == -INFINITY) break;
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (lane + 32 * i == e) c[i] = -INFINITY;
        if (lane == j) mine = e;
    }
    return mine;
}

__device__ __forceinline__ float clean_logit(float v) { return v != v ? -INFINITY : fminf(v, FLT_MAX); }

template <int NI>
__device__ __forceinline__ void load_logits(const RouteArgs &a, int b, int last, float (&l)[NI]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < NI; ++i)
        l[i] = b < last && lane + 32 * i < a.E ? __ldg(a.logits + static_cast<size_t>(b) * a.E + lane + 32 * i) : -INFINITY;
}

// A token's choice and weights by one warp.
template <int NI>
__device__ __forceinline__ void choose(const RouteArgs &a, int b, const int (&group)[NI], const float (&bias)[NI],
                                       double unit, const float (&raw)[NI], unsigned *s_hist, double *row, int *s_sel,
                                       float *s_w) {
    const int lane = threadIdx.x & 31;
    const bool sig = a.rule.score == MOE_SCORE_SIGMOID;
    const float *logits = a.logits + static_cast<size_t>(b) * a.E;
    Token<NI> t;
    float l[NI], top = -INFINITY, low = INFINITY;
#pragma unroll
    for (int i = 0; i < NI; ++i) l[i] = clean_logit(raw[i]);
    // with a bias, or groups valued by two experts, the values rank
    const bool may_logit = a.bias == nullptr && (a.rule.groups == 1 || a.rule.group_best == 1);
    if (may_logit || !sig) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            top = fmaxf(top, l[i]);
            if (l[i] > -INFINITY) low = fminf(low, l[i]);
        }
        top = warp_maxf(top);
        low = -warp_maxf(-low);
    }
    const float shift = sig || top == -INFINITY ? 0.0f : top;
    const bool by_logit = may_logit && (!sig || top <= TOP_LOGIT) && low - shift >= LOW_LOGIT;
    // softmax: the sum of exp(l - top)
    double z = 1.0;
    if (!sig && !(by_logit && a.rule.renorm)) {
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            t.c[i] = l[i] > -INFINITY ? exp_from(l[i], shift) : 0.0;
            sum += t.c[i];
        }
        z = warp_sum(sum);
    }
    constexpr unsigned LAST_SLOT = (1u << SLOT_BITS) - 1u;
    if (by_logit) {
        // images of the upper 64 units of logit; what lies below is equal
        const double base = 64.0 - static_cast<double>(top);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            t.c[i] = static_cast<double>(l[i]);
            const int u = round_int(fmax(t.c[i] + base, 0.0) * 1048576.0) + 1;
            t.image[i] = l[i] > -INFINITY ? static_cast<unsigned>(u) << SLOT_BITS | (LAST_SLOT - i) : 0u;
        }
    } else {
        const double inv = sig ? 1.0 : z > 0.0 ? 1.0 / z : 0.0;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const double s = sig ? sigmoid(l[i]) : t.c[i] * inv;
            t.c[i] = l[i] > -INFINITY ? s + static_cast<double>(bias[i]) : -INFINITY;
            const int u = round_int(l[i] > -INFINITY ? t.c[i] * unit : 0.0) + (1 << 26) + 1;
            t.image[i] = l[i] > -INFINITY ? static_cast<unsigned>(u) << SLOT_BITS | (LAST_SLOT - i) : 0u;
        }
    }
    int mine;
    if (!t.by_image(a, group, reinterpret_cast<unsigned *>(row), mine)) {
        double c[NI];  // a copy: the values themselves stay in registers
#pragma unroll
        for (int i = 0; i < NI; ++i) c[i] = t.c[i];
        mine = by_value<NI>(a, c, row, by_logit, shift);
    }
    // lane j: the score of its expert
    double s = 0.0;
    if (mine >= 0) {
        const float v = clean_logit(__ldg(logits + mine));
        s = sig ? sigmoid(v) : exp_from(v, shift);
    }
    const double sum = a.rule.renorm ? warp_sum(s) : z;
    if (lane < a.k) {
        // rounded once, at the end
        const float w = mine >= 0 && sum > 0.0 ? static_cast<float>(s / sum * static_cast<double>(a.rule.scale)) : 0.0f;
        a.sel_idx[static_cast<size_t>(b) * a.k + lane] = mine;
        a.sel_w[static_cast<size_t>(b) * a.k + lane] = w;
        if (a.runs == 1) {
            s_sel[b * a.k + lane] = mine;
            s_w[b * a.k + lane] = w;
        }
        if (mine >= 0 && !a.one_launch) atomicAdd(s_hist + mine, 1u);
    }
}

// ---------------------------------------------------------------- lists --
struct ListsShared {
    int total[SE_MAX], before[SE_MAX], place[SE_MAX], wsum[WARPS];
    unsigned mask[SE_MAX];
    int sel[WARPS * K_MAX];  // the choices of a batch that is one block
    float w[WARPS * K_MAX];
};

// Inclusive scan over the block's threads.
__device__ int block_scan(int v, int *wsum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(ALL, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) wsum[warp] = v;
    __syncthreads();
    int base = 0;
    for (int w = 0; w < warp; ++w) base += wsum[w];
    __syncthreads();
    return v + base;
}

// Masks of the SUB tokens from t0 (their choices), then fn(expert, token,
// pair) for each choice.
template <class Fn>
__device__ __forceinline__ void each_choice(const RouteArgs &a, int t0, int last, ListsShared &sh, Fn fn) {
    const int p = threadIdx.x, t = p / a.k;  // at most 512 pairs: one a thread
    const size_t pair = static_cast<size_t>(t0) * a.k + p;
    int e = -1;
    if (p < min(SUB, last - t0) * a.k) e = a.runs == 1 ? sh.sel[p] : __ldcg(a.sel_idx + pair);
    if (e >= 0) atomicOr(sh.mask + e, 1u << t);
    __syncthreads();
    if (e >= 0) fn(e, t, pair);
    __syncthreads();
}

// The lists' entries of tokens [first, last), and what one block (`head`)
// writes for all.  Expert counts come from the runs' histograms, or, for one
// launch, from the choices.
__device__ void write_lists(const RouteArgs &a, ListsShared &sh, int first, int last, bool head) {
    const int tid = threadIdx.x;  // SE_MAX threads: one an expert
    sh.total[tid] = sh.before[tid] = 0;
    sh.mask[tid] = 0u;
    __syncthreads();
    if (a.one_launch) {
        for (int t0 = 0; t0 < a.B; t0 += SUB) {
            each_choice(a, t0, a.B, sh, [](int, int, size_t) {});
            sh.total[tid] += __popc(sh.mask[tid]);
            sh.mask[tid] = 0u;
            __syncthreads();
        }
    } else {
        // eight experts a thread, several runs at once
        const int pieces = hist_pitch(a.E) / 8, parts = THREADS / pieces, part = tid / pieces, at = tid - part * pieces;
        int total[8] = {}, before[8] = {};
        if (part < parts) {
            const uint4 *h = reinterpret_cast<const uint4 *>(a.hist) + at;
#pragma unroll 8
            for (int r = part; r < a.runs; r += parts) {
                const uint4 v = __ldcg(h + r * pieces);
                const unsigned w[4] = {v.x, v.y, v.z, v.w};
                const bool earlier = r < static_cast<int>(blockIdx.x);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int n = (w[i / 2] >> (16 * (i & 1))) & 0xffffu;
                    total[i] += n;
                    before[i] += earlier ? n : 0;
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                atomicAdd(sh.total + at * 8 + i, total[i]);
                atomicAdd(sh.before + at * 8 + i, before[i]);
            }
        }
        __syncthreads();
    }
    const int n = tid < a.E ? sh.total[tid] : 0;
    const int end = block_scan(n, sh.wsum), slot = block_scan(n > 0 ? 1 : 0, sh.wsum);
    __shared__ int s_end, s_slots;
    if (tid == THREADS - 1) {
        s_end = end;
        s_slots = slot;
    }
    sh.place[tid] = end - n + sh.before[tid];
    __syncthreads();
    if (head && tid < a.E) {
        if (n > 0) {
            a.lists.active[slot - 1] = tid;
            a.lists.offsets[slot - 1] = end - n;
        }
        if (tid >= s_slots) a.lists.active[tid] = -1;
        if (tid >= s_slots) a.lists.offsets[tid] = s_end;
        if (tid == 0) {
            a.lists.offsets[a.E] = s_end;
            *a.lists.n_active = s_slots;
        }
    }
    const int all = a.B * a.k, blocks = a.one_launch ? 1 : gridDim.x, me = a.one_launch ? 0 : blockIdx.x;
    for (int p = s_end + me * THREADS + tid; p < all; p += blocks * THREADS) {
        a.lists.tok[p] = -1;
        a.lists.w[p] = 0.0f;
    }
    for (int t0 = first; t0 < last; t0 += SUB) {
        each_choice(a, t0, last, sh, [&](int e, int t, size_t pair) {
            const int p = sh.place[e] + __popc(sh.mask[e] & ((1u << t) - 1u));
            a.lists.tok[p] = t0 + t;
            a.lists.w[p] = a.runs == 1 ? sh.w[pair] : __ldcg(a.sel_w + pair);
        });
        sh.place[tid] += __popc(sh.mask[tid]);
        sh.mask[tid] = 0u;
        __syncthreads();
    }
}
static_assert(THREADS == SE_MAX && SUB * K_MAX <= THREADS, "a thread per expert, and per choice of SUB tokens");

template <int NI>
__global__ void __launch_bounds__(THREADS, NI <= 8 ? 2 : 1) route_choose_kernel(const __grid_constant__ RouteArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ ListsShared sh;
    __shared__ int s_last;
    unsigned *s_hist = reinterpret_cast<unsigned *>(sh.total);
    double *s_row = reinterpret_cast<double *>(smem);  // [warp][E + groups], groups only
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    s_hist[threadIdx.x] = 0;
    const float inv_per = static_cast<float>(a.rule.groups) / static_cast<float>(a.E);
    int group[NI];
    float bias[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e = lane + 32 * i;
        // e / per for small integers: (e + 1/2) / per is never near one
        group[i] = a.rule.groups > 1 ? __float2int_rz((static_cast<float>(min(e, a.E - 1)) + 0.5f) * inv_per) : 0;
        bias[i] = a.bias != nullptr && e < a.E ? __ldg(a.bias + e) : 0.0f;
    }
    // images: scores are at most 1, so values are below 1 + the largest bias
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) most = fmaxf(most, fabsf(bias[i]));
    most = 1.0f + warp_maxf(most);
    const int ex = static_cast<int>(__float_as_uint(most) >> 23) - 126;  // most < 2^ex
    const double unit = __hiloint2double((1023 + 26 - ex) << 20, 0);
    __syncthreads();
    const int first = blockIdx.x * a.run, last = min(first + a.run, a.B);
    // the next token's logits are on their way while a token is done
    float raw[NI], next[NI];
    load_logits<NI>(a, first + warp, last, next);
    for (int b = first + warp; b < last; b += WARPS) {
#pragma unroll
        for (int i = 0; i < NI; ++i) raw[i] = next[i];
        load_logits<NI>(a, b + WARPS, last, next);
        choose<NI>(a, b, group, bias, unit, raw, s_hist, s_row + static_cast<size_t>(warp) * (a.E + a.rule.groups), sh.sel, sh.w);
    }
    __syncthreads();
    if (!a.one_launch) {
        const int pitch = hist_pitch(a.E);
        if (threadIdx.x < pitch)
            a.hist[static_cast<size_t>(blockIdx.x) * pitch + threadIdx.x] = static_cast<uint16_t>(s_hist[threadIdx.x]);
        return;
    }
    if (a.runs == 1) {
        write_lists(a, sh, 0, a.B, true);
        return;
    }
    // the last block to finish writes the lists (the ticket wraps to 0)
    if (threadIdx.x == 0) {
        __threadfence();
        s_last = atomicInc(a.ticket, gridDim.x - 1) == gridDim.x - 1;
        __threadfence();
    }
    __syncthreads();
    if (s_last) write_lists(a, sh, 0, a.B, true);
}

__global__ void __launch_bounds__(THREADS) route_lists_kernel(const __grid_constant__ RouteArgs a) {
    __shared__ ListsShared sh;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int first = blockIdx.x * a.run;
    write_lists(a, sh, first, min(first + a.run, a.B), blockIdx.x == 0);
}

template <int NI>
cudaError_t launch_choose(const RouteArgs &a, cudaStream_t s) {
    const size_t smem = a.rule.groups > 1 ? static_cast<size_t>(WARPS) * (a.E + a.rule.groups) * 8 : 0;
    static bool configured[MAX_DEVICES] = {};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= MAX_DEVICES) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        err = cudaFuncSetAttribute(route_choose_kernel<NI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   WARPS * (SE_MAX + 32) * 8);
        if (err != cudaSuccess) return err;
        configured[dev] = true;
    }
    route_choose_kernel<NI><<<a.runs, THREADS, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t route_ws_bytes(const moe_dims_t &d) {
    const size_t run = run_tokens(d.B), runs = (d.B + run - 1) / run;
    return d.B <= ONE_LAUNCH ? sizeof(BlocksControl) : (HIST_OFFSET + runs * hist_pitch(d.E) * 2 + 255) / 256 * 256;
}

cudaError_t launch_route_scored(const float *logits, const float *bias, const moe_dims_t &d,
                                const moe_scoring_t &r, int32_t *sel_idx, float *sel_w, const moe_lists_t &l,
                                void *ws, cudaStream_t s) {
    RouteArgs a = {};
    BlocksControl *control = static_cast<BlocksControl *>(ws);
    a.logits = logits;
    a.bias = bias;
    a.B = d.B;
    a.E = d.E;
    a.k = d.k;
    a.run = run_tokens(d.B);
    a.runs = (d.B + a.run - 1) / a.run;
    a.one_launch = d.B <= ONE_LAUNCH;
    a.rule = r;
    a.sel_idx = sel_idx;
    a.sel_w = sel_w;
    a.ticket = &control->ticket;
    a.hist = reinterpret_cast<uint16_t *>(static_cast<unsigned char *>(ws) + HIST_OFFSET);
    a.lists = l;
    cudaError_t err = a.E <= 32    ? launch_choose<1>(a, s)
                      : a.E <= 64  ? launch_choose<2>(a, s)
                      : a.E <= 128 ? launch_choose<4>(a, s)
                      : a.E <= 256 ? launch_choose<8>(a, s)
                                   : launch_choose<16>(a, s);
    if (err != cudaSuccess || a.one_launch) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.runs);
    cfg.blockDim = dim3(THREADS);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, route_lists_kernel, a);
}

}  // namespace moe

// Routing with scores, balance bias and expert groups (sm_100a).
//
// route_choose_kernel : a warp per token: scores, group values, top-k,
//                       weights; per run of tokens, how many chose each expert.
// route_lists_kernel  : expert-major token lists from the choices: a block
//                       per run of tokens; an entry's place is the expert's
//                       first place + the entries of earlier runs + its rank
//                       among the run's tokens (bit masks, no atomics on
//                       places: the lists do not depend on scheduling).  A
//                       batch that is one run gets its lists in the first
//                       kernel.
//
// The choice is that of the values c = s + bias in fp64 (equal values to the
// lower index).  The warp ranks fp32 values instead and checks that every
// two neighbours of the order it uses, the first expert left out among them,
// are further apart than the fp32 errors; a token that fails the check (a
// few in 10^5 of random ones, and every exact tie) is done again in fp64.
// Without a bias, and with groups valued by their best expert, the logits
// themselves rank (a score is monotone in its logit).
#include <cfloat>
#include <cmath>

#include "blocks.h"
#include "route_dev.cuh"

namespace moe {
namespace {

constexpr unsigned ALL = FULL;
constexpr int SUB = 64;          // tokens whose choices of one expert are one 64-bit mask
constexpr int RUNS_MAX = 128;    // runs of tokens (blocks)
constexpr int ONE_RUN = 128;     // 4 tokens a warp, but one launch
constexpr int CHOOSE_THREADS = 1024;
constexpr int LISTS_THREADS = 1024;

// Tokens per run: a multiple of SUB that leaves at most RUNS_MAX runs; up to
// ONE_RUN tokens are one.
int run_tokens(int B) {
    if (B <= ONE_RUN) return ONE_RUN;
    const int subs = (B + SUB - 1) / SUB;
    return SUB * ((subs + RUNS_MAX - 1) / RUNS_MAX);
}

// Values of a token's row in shared memory: skewed by one every 32, so that
// lanes which walk runs of experts meet different banks.
__host__ __device__ constexpr int row_values(int E) { return E + E / 32 + 1; }

struct RouteArgs {
    const float *logits, *bias;
    int B, E, k, run, runs;
    moe_scoring_t rule;
    int32_t *sel_idx;
    float *sel_w;
    int32_t *hist;  // [runs][E]
    moe_lists_t lists;
};

// Largest value over the warp; the lowest expert index among equal ones
// (value -inf: no candidate).
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

// A token in fp64.
template <int NI>
__device__ __noinline__ void token_exact(const RouteArgs &a, int b, unsigned *s_hist, double *s_row) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.rule.groups, per = a.E / G;
            double s[NI], c[NI];
            float l[NI];
            double top = -INFINITY;
    #pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int e = lane + 32 * i;
                float v = e < a.E ? __ldg(a.logits + static_cast<size_t>(b) * a.E + e) : -INFINITY;
                v = v != v ? -INFINITY : fminf(v, FLT_MAX);
                l[i] = v;
                top = fmax(top, static_cast<double>(v));
            }
            if (a.rule.score == MOE_SCORE_SOFTMAX) {
                int dummy = 0;
                warp_best(top, dummy);
                double sum = 0.0;
    #pragma unroll
                for (int i = 0; i < NI; ++i) {
                    s[i] = l[i] > -INFINITY ? exp(static_cast<double>(l[i]) - top) : 0.0;
                    sum += s[i];
                }
                sum = warp_sum(sum);
    #pragma unroll
                for (int i = 0; i < NI; ++i) s[i] = s[i] / sum;
            } else {
    #pragma unroll
                for (int i = 0; i < NI; ++i) s[i] = 1.0 / (1.0 + exp(-static_cast<double>(l[i])));
            }
    #pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int e = lane + 32 * i;
                const double beta = a.bias != nullptr && e < a.E ? static_cast<double>(__ldg(a.bias + e)) : 0.0;
                c[i] = l[i] > -INFINITY ? s[i] + beta : -INFINITY;
            }
            if (G > 1) {
                // lane g sums the best of group g (rows skewed by one value every 32)
                double *row = s_row + static_cast<size_t>(warp) * row_values(a.E);
                __syncwarp();
    #pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const int e = lane + 32 * i;
                    if (e < a.E) row[e + (e >> 5)] = c[i];
                }
                __syncwarp();
                double b1 = -INFINITY, b2 = -INFINITY;
                if (lane < G) {
                    for (int j = 0; j < per; ++j) {
                        const int e = lane * per + j;
                        const double v = row[e + (e >> 5)];
                        if (v > b1) {
                            b2 = b1;
                            b1 = v;
                        } else if (v > b2) b2 = v;
                    }
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
            int mine = -1;        // lane j: the j-th chosen expert and its score
            double score = 0.0;
            for (int j = 0; j < a.k; ++j) {
                double v = -INFINITY, sv = 0.0;
                int e = 1 << 20;
    #pragma unroll
                for (int i = 0; i < NI; ++i)
                    if (c[i] > v) {
                        v = c[i];
                        e = lane + 32 * i;
                        sv = s[i];
                    }
                const int own = e;
                warp_best(v, e);
                if (v == -INFINITY) break;
                sv = __shfl_sync(ALL, sv, e & 31);
                if (own == e) {
    #pragma unroll
                    for (int i = 0; i < NI; ++i)
                        if (lane + 32 * i == e) c[i] = -INFINITY;
                    atomicAdd(s_hist + e, 1u);
                }
                if (lane == j) {
                    mine = e;
                    score = sv;
                }
            }
            const double sum = a.rule.renorm ? warp_sum(score) : 1.0;
            if (lane < a.k) {
                a.sel_idx[static_cast<size_t>(b) * a.k + lane] = mine;
                a.sel_w[static_cast<size_t>(b) * a.k + lane] =
                    mine >= 0 && sum > 0.0 ? static_cast<float>(score / sum * static_cast<double>(a.rule.scale)) : 0.0f;
            }
}

// fp32 errors, in units of 2^-24: exp_own (1 ulp = 2 units), the sum 1 + z,
// and a division good to 2 ulp give a sigmoid within 8 units of itself; a
// softmax adds the errors of the sum's terms (2) and of the sum, taken in
// fp64, and stays within 8.  Adding the bias rounds once more.
constexpr float ERR = 5.9604645e-8f * 9.0f;
// Logits: scores differ in fp64 when their logits do, by more than
// NEAR_LOGIT and inside these limits.
constexpr float NEAR_LOGIT = 1e-9f, TOP_LOGIT = 16.0f, LOW_LOGIT = -600.0f;

// The lane's best candidate.
template <int NI>
__device__ __forceinline__ void lane_best(const float (&c)[NI], int lane, float &v, int &e) {
    v = -INFINITY;
    e = 1 << 20;
#pragma unroll
    for (int i = 0; i < NI; ++i)
        if (c[i] > v) {
            v = c[i];
            e = lane + 32 * i;
        }
}

// Experts lane + 32 i, i < NI; false: the token has to be decided in fp64
// (nothing has been written).
template <int NI>
__device__ __forceinline__ bool token_fast(const RouteArgs &a, int b, unsigned *s_hist, float *row) {
    const int lane = threadIdx.x & 31;
    const int G = a.rule.groups;
    const bool sigmoid = a.rule.score == MOE_SCORE_SIGMOID;
    const bool by_logit = a.bias == nullptr && (G == 1 || a.rule.group_best == 1);
    float l[NI], s[NI], c[NI];
    float top = -INFINITY, low = INFINITY;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e = lane + 32 * i;
        const float v = e < a.E ? __ldg(a.logits + static_cast<size_t>(b) * a.E + e) : -INFINITY;
        l[i] = v != v ? -INFINITY : fminf(v, FLT_MAX);
        top = fmaxf(top, l[i]);
    }
    top = float_of_ord(__reduce_max_sync(ALL, ord_of(top)));
    float shift = 0.0f, bound = 1.0f;  // bound: no score is larger
    double z = 1.0;
    if (sigmoid) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const float x = exp_own(-fabsf(l[i]));  // 0 for -inf
            s[i] = __fdividef(l[i] >= 0.0f ? 1.0f : x, 1.0f + x);
        }
        if (top > TOP_LOGIT && by_logit) return false;
    } else {
        shift = top > -INFINITY ? top : 0.0f;
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            s[i] = exp_own(l[i] - shift);
            sum += static_cast<double>(s[i]);
        }
        z = warp_sum(sum);
        const float inv = z > 0.0 ? static_cast<float>(1.0 / z) : 0.0f;
        bound = inv;
        if (!by_logit) {
#pragma unroll
            for (int i = 0; i < NI; ++i) s[i] *= inv;
        }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e = lane + 32 * i;
        if (by_logit) c[i] = l[i];
        else {
            const float beta = a.bias != nullptr && e < a.E ? __ldg(a.bias + e) : 0.0f;
            c[i] = l[i] > -INFINITY ? s[i] + beta : -INFINITY;
            bound = fmaxf(bound, c[i] > -INFINITY ? fabsf(c[i]) : 0.0f);
        }
    }
    // two values further apart than this are in order
    float near = NEAR_LOGIT;
    if (!by_logit) near = 2.0f * ERR * __uint_as_float(__reduce_max_sync(ALL, __float_as_uint(bound)));
    bool sure = true;
    if (G > 1) {
        const int per = a.E / G;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E) row[e + (e >> 5)] = c[i];
        }
        __syncwarp();
        float b1 = -INFINITY, b2 = -INFINITY;
        if (lane < G) {
#pragma unroll 8
            for (int j = 0; j < per; ++j) {
                const int e = lane * per + j;
                const float v = row[e + (e >> 5)];
                b2 = fmaxf(b2, fminf(b1, v));
                b1 = fmaxf(b1, v);
            }
        }
        float value = b1;
        if (a.rule.group_best == 2 && b2 > -INFINITY) value += b2;
        // a sum of two values rounds once more: three times the distance
        const float gnear = a.rule.group_best == 2 ? 3.0f * near : near;
        unsigned keep = 0;
        float before = INFINITY;
        for (int j = 0; j <= a.rule.top_groups; ++j) {
            const unsigned o = (keep >> lane) & 1u || lane >= G ? 0u : ord_of(value);
            const unsigned m = __reduce_max_sync(ALL, o);
            const float v = m == 0u ? -INFINITY : float_of_ord(m);
            if (v == -INFINITY) break;
            sure = sure && (before - v > gnear || (by_logit && before == v));
            before = v;
            if (j < a.rule.top_groups) keep |= 1u << (__ffs(__ballot_sync(ALL, o == m)) - 1);
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E && !((keep >> (e / per)) & 1u)) c[i] = -INFINITY;
        }
    }
    int mine = -1;  // lane j: the j-th chosen expert and its score
    float score = 0.0f, v, before = INFINITY;
    int e;
    lane_best<NI>(c, lane, v, e);
    for (int j = 0; j <= a.k; ++j) {
        const unsigned o = v == -INFINITY ? 0u : ord_of(v);
        const unsigned m = __reduce_max_sync(ALL, o);
        if (m == 0u) break;
        const float best = float_of_ord(m);
        sure = sure && (before - best > near || (by_logit && before == best));
        before = best;
        low = fminf(low, best);
        if (j == a.k) break;
        const int win = static_cast<int>(__reduce_min_sync(ALL, o == m ? static_cast<unsigned>(e) : 0xffffffffu));
        float sv = 0.0f;
        if (win == e) {
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if (lane + 32 * i == e) {
                    sv = s[i];
                    c[i] = -INFINITY;
                }
            lane_best<NI>(c, lane, v, e);
        }
        sv = __shfl_sync(ALL, sv, win & 31);
        if (lane == j) {
            mine = win;
            score = sv;
        }
    }
    if (by_logit) sure = sure && low - shift > LOW_LOGIT;
    // scores that fp32 cannot hold (exp_own gives 0 below -87) weigh in fp64
    if (!sure || __any_sync(ALL, mine >= 0 && score < 1e-30f)) return false;
    const double sum = a.rule.renorm ? warp_sum(static_cast<double>(score)) : (sigmoid || !by_logit ? 1.0 : z);
    if (lane < a.k) {
        a.sel_idx[static_cast<size_t>(b) * a.k + lane] = mine;
        a.sel_w[static_cast<size_t>(b) * a.k + lane] =
            mine >= 0 ? static_cast<float>(static_cast<double>(score) * static_cast<double>(a.rule.scale) / sum) : 0.0f;
        if (mine >= 0) atomicAdd(s_hist + mine, 1u);
    }
    return true;
}

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
    if (warp == 0) {
        int w = wsum[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(ALL, w, o);
            if (lane >= o) w += u;
        }
        wsum[lane] = w;
    }
    __syncthreads();
    const int r = v + (warp > 0 ? wsum[warp - 1] : 0);
    __syncthreads();
    return r;
}

// The lists of the block's run (all the block's threads).
__device__ void lists_of_run(const RouteArgs &a) {
    __shared__ int s_total[SE_MAX], s_before[SE_MAX], s_place[SE_MAX], wsum[32];
    __shared__ unsigned long long s_mask[SE_MAX];
    const int tid = threadIdx.x;
    for (int e = tid; e < SE_MAX; e += LISTS_THREADS) {
        s_total[e] = s_before[e] = 0;
        s_mask[e] = 0ull;
    }
    __syncthreads();
    // the run counts, several runs at once
    const int parts = LISTS_THREADS / a.E, part = tid / a.E, ex = tid - part * a.E;
    if (part < parts) {
        int total = 0, before = 0;
        for (int r = part; r < a.runs; r += parts) {
            const int h = a.hist[static_cast<size_t>(r) * a.E + ex];
            total += h;
            if (r < static_cast<int>(blockIdx.x)) before += h;
        }
        if (total) atomicAdd(s_total + ex, total);
        if (before) atomicAdd(s_before + ex, before);
    }
    __syncthreads();
    const int n = tid < a.E ? s_total[tid] : 0;
    const int end = block_scan(n, wsum), slot = block_scan(n > 0 ? 1 : 0, wsum);
    __shared__ int s_end, s_slots;
    if (tid == LISTS_THREADS - 1) {
        s_end = end;
        s_slots = slot;
    }
    if (tid < a.E) s_place[tid] = end - n + s_before[tid];
    __syncthreads();
    if (blockIdx.x == 0 && tid < a.E) {
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
    const int first = blockIdx.x * a.run, last = min(first + a.run, a.B);
    const long long all = static_cast<long long>(a.B) * a.k;
    for (long long p = s_end + static_cast<long long>(blockIdx.x) * LISTS_THREADS + tid; p < all;
         p += static_cast<long long>(gridDim.x) * LISTS_THREADS) {
        a.lists.tok[p] = -1;
        a.lists.w[p] = 0.0f;
    }
    for (int t0 = first; t0 < last; t0 += SUB) {
        const int pairs = min(SUB, last - t0) * a.k;  // at most 1024
        int e = -1, t = 0;
        if (tid < pairs) {
            t = tid / a.k;
            e = a.sel_idx[static_cast<size_t>(t0) * a.k + tid];
            if (e >= 0) atomicOr(s_mask + e, 1ull << t);
        }
        __syncthreads();
        if (e >= 0) {
            const int p = s_place[e] + __popcll(s_mask[e] & ((1ull << t) - 1ull));
            a.lists.tok[p] = t0 + t;
            a.lists.w[p] = a.sel_w[static_cast<size_t>(t0) * a.k + tid];
        }
        __syncthreads();
        if (tid < a.E) {
            s_place[tid] += __popcll(s_mask[tid]);
            s_mask[tid] = 0ull;
        }
        __syncthreads();
    }
}

template <int NI>
__global__ void __launch_bounds__(CHOOSE_THREADS, 1) route_choose_kernel(const __grid_constant__ RouteArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ unsigned char smem[];
    unsigned *s_hist = reinterpret_cast<unsigned *>(smem);          // [E]
    double *s_row = reinterpret_cast<double *>(smem + SE_MAX * 4);  // [warp][row_values(E)], groups only
    const int warp = threadIdx.x >> 5;
    for (int e = threadIdx.x; e < a.E; e += CHOOSE_THREADS) s_hist[e] = 0;
    __syncthreads();
    const int first = blockIdx.x * a.run, last = min(first + a.run, a.B);
    for (int b = first + warp; b < last; b += CHOOSE_THREADS / 32)
        if (!token_fast<NI>(a, b, s_hist, reinterpret_cast<float *>(s_row + static_cast<size_t>(warp) * row_values(a.E))))
            token_exact<NI>(a, b, s_hist, s_row);
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += CHOOSE_THREADS) a.hist[static_cast<size_t>(blockIdx.x) * a.E + e] = s_hist[e];
    if (a.runs == 1) {
        __threadfence_block();
        __syncthreads();
        lists_of_run(a);
    }
}

__global__ void __launch_bounds__(LISTS_THREADS, 1) route_lists_kernel(const __grid_constant__ RouteArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    lists_of_run(a);
}

template <int NI>
cudaError_t launch_choose(const RouteArgs &a, cudaStream_t s) {
    const size_t rows = a.rule.groups > 1 ? static_cast<size_t>(CHOOSE_THREADS / 32) * row_values(a.E) * 8 : 0;
    const size_t smem = SE_MAX * 4 + rows;
    static bool configured[MAX_DEVICES] = {};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= MAX_DEVICES) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        err = cudaFuncSetAttribute(route_choose_kernel<NI>, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
        if (err != cudaSuccess) return err;
        configured[dev] = true;
    }
    route_choose_kernel<NI><<<a.runs, CHOOSE_THREADS, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t route_ws_bytes(const moe_dims_t &d) {
    const size_t run = run_tokens(d.B), runs = (d.B + run - 1) / run;
    return (sizeof(BlocksControl) + runs * d.E * 4 + 255) / 256 * 256;
}

cudaError_t launch_route_scored(const float *logits, const float *bias, const moe_dims_t &d,
                                const moe_scoring_t &r, int32_t *sel_idx, float *sel_w, const moe_lists_t &l,
                                void *ws, cudaStream_t s) {
    RouteArgs a = {};
    a.logits = logits;
    a.bias = bias;
    a.B = d.B;
    a.E = d.E;
    a.k = d.k;
    a.run = run_tokens(d.B);
    a.runs = (d.B + a.run - 1) / a.run;
    a.rule = r;
    a.sel_idx = sel_idx;
    a.sel_w = sel_w;
    a.hist = reinterpret_cast<int32_t *>(static_cast<unsigned char *>(ws) + sizeof(BlocksControl));
    a.lists = l;
    cudaError_t err = a.E <= 32    ? launch_choose<1>(a, s)
                      : a.E <= 64  ? launch_choose<2>(a, s)
                      : a.E <= 128 ? launch_choose<4>(a, s)
                      : a.E <= 256 ? launch_choose<8>(a, s)
                                   : launch_choose<16>(a, s);
    if (err != cudaSuccess) return err;
    if (a.runs == 1) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.runs);
    cfg.blockDim = dim3(LISTS_THREADS);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, route_lists_kernel, a);
}

}  // namespace moe

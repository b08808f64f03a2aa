// Block-scaled e4m3 quantisation and the expert FFN's combine (sm_100a).
//
// quantize_rows_kernel  : one scale per 128 columns of a row (activations)
// quantize_tiles_kernel : one scale per 128 x 128 block (weights)
// combine_kernel        : y[t] = sum of w[p] * yp[p] over the token's list
//                         entries, in list order (no atomics: the result
//                         does not depend on scheduling)
//
// A block's scale is the smallest power of two s with max|x| <= 448 s (448:
// the largest e4m3 value), 1 for a block of zeros.  Dividing by a power of
// two is exact, so the only rounding is the one to e4m3 (nearest even) and
// the result is fixed bit by bit, whatever computes it.
//
// Bound by HBM: each value is read once and a byte written.  Measured: 4096
// x 2048 bf16 rows 6.4 us with inputs from HBM (25.4 MB, 4.0 TB/s: a short
// launch), 4.9 us where they stay in L2; 128 matrices of 768 x 2048 bf16 89 us
// (604 MB, 6.8 TB/s, 1.04 of the measured copy rate).
#include <cuda_bf16.h>

#include "blocks.h"

namespace moe {
namespace {

constexpr unsigned ALL = 0xffffffffu;
constexpr unsigned INF_BITS = 0x7f800000u;  // magnitude bits of fp32 infinity; NaN above
// Rows from which a warp takes 2048 (bf16) or 1024 (fp32) columns instead of
// 512 (2048 columns, bf16: 2048 rows 4.3 against 4.1 us, 4096 rows 6.5 and
// 6.5, 8192 rows 9.5 against 11.2; fp32: 5.5 against 5.4, 7.9 against 8.1,
// 13.7 against 14.8).
constexpr long long WIDE_ROWS = 2048;

// Exponent e of the scale 2^e for a block whose largest magnitude is top
// (its fp32 bits): top = m 2^(x-127), 1 <= m < 2; 448 = 1.75 * 2^8, so
// e = x - 127 - 8, plus one when m > 1.75.  Below 2^-112 the scale stays
// 2^-120: its reciprocal must be a normal number.
__device__ __forceinline__ int scale_exp(unsigned top_bits) {
    if (top_bits == 0u) return 0;
    const int e = static_cast<int>(top_bits >> 23) - 135 + ((top_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e < -120 ? -120 : e;
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// four values scaled by inv (a power of two) -> four e4m3 bytes
__device__ __forceinline__ unsigned pack4(float a, float b, float c, float d, float inv) {
    unsigned short lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b * inv), "f"(a * inv));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d * inv), "f"(c * inv));
    return static_cast<unsigned>(lo) | (static_cast<unsigned>(hi) << 16);
}

// The largest finite magnitude among two (fp32 bits), and x with an infinity
// made NaN.
__device__ __forceinline__ unsigned finite_max(unsigned top, unsigned bits) {
    bits &= 0x7fffffffu;
    return bits < INF_BITS ? max(top, bits) : top;
}
__device__ __forceinline__ unsigned inf_to_nan(unsigned bits) {
    return (bits & 0x7fffffffu) == INF_BITS ? 0x7fffffffu : bits;
}

// A lane's 16 columns: raw loads, the largest magnitude, and the four words
// of e4m3 values.  Where the largest magnitude is not finite, `settle` makes
// infinities NaN and gives the largest finite one.
template <typename T>
struct Lane16;
template <>
struct Lane16<float> {
    float4 v[4];
    __device__ __forceinline__ void load(const float *p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __ldg(reinterpret_cast<const float4 *>(p) + i);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __device__ __forceinline__ unsigned top() const {
        unsigned t = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            t = max(max(t, max(__float_as_uint(v[i].x) & 0x7fffffffu, __float_as_uint(v[i].y) & 0x7fffffffu)),
                    max(__float_as_uint(v[i].z) & 0x7fffffffu, __float_as_uint(v[i].w) & 0x7fffffffu));
        return t;
    }
    __device__ __forceinline__ unsigned settle() {
        unsigned t = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float *f[4] = {&v[i].x, &v[i].y, &v[i].z, &v[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const unsigned b = __float_as_uint(*f[j]);
                t = finite_max(t, b);
                *f[j] = __uint_as_float(inf_to_nan(b));
            }
        }
        return t;
    }
    __device__ __forceinline__ uint4 pack(float inv) const {
        return make_uint4(pack4(v[0].x, v[0].y, v[0].z, v[0].w, inv), pack4(v[1].x, v[1].y, v[1].z, v[1].w, inv),
                          pack4(v[2].x, v[2].y, v[2].z, v[2].w, inv), pack4(v[3].x, v[3].y, v[3].z, v[3].w, inv));
    }
};
template <>
struct Lane16<__nv_bfloat16> {
    uint4 v[2];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        v[0] = __ldg(reinterpret_cast<const uint4 *>(p));
        v[1] = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
    }
    __device__ __forceinline__ void zero() { v[0] = v[1] = make_uint4(0u, 0u, 0u, 0u); }
    static __device__ __forceinline__ unsigned top2(unsigned w) { return max((w << 16) & 0x7fffffffu, w & 0x7fff0000u); }
    __device__ __forceinline__ unsigned top() const {
        return max(max(max(top2(v[0].x), top2(v[0].y)), max(top2(v[0].z), top2(v[0].w))),
                   max(max(top2(v[1].x), top2(v[1].y)), max(top2(v[1].z), top2(v[1].w))));
    }
    __device__ __forceinline__ unsigned settle() {
        unsigned t = 0u;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            unsigned *w[4] = {&v[i].x, &v[i].y, &v[i].z, &v[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const unsigned lo = *w[j] << 16, hi = *w[j] & 0xffff0000u;
                t = finite_max(finite_max(t, lo), hi);
                *w[j] = (inf_to_nan(lo) >> 16) | (inf_to_nan(hi) & 0xffff0000u);
            }
        }
        return t;
    }
    static __device__ __forceinline__ unsigned pack2(unsigned a, unsigned b, float inv) {
        return pack4(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u), __uint_as_float(b << 16),
                     __uint_as_float(b & 0xffff0000u), inv);
    }
    __device__ __forceinline__ uint4 pack(float inv) const {
        return make_uint4(pack2(v[0].x, v[0].y, inv), pack2(v[0].z, v[0].w, inv), pack2(v[1].x, v[1].y, inv),
                          pack2(v[1].z, v[1].w, inv));
    }
};

// A block's 128 x 128 tile that holds an infinity or NaN, read again (out of
// line: the kept values would cost a third more registers): row r0 + 32 i,
// column c of the thread's values at x + 32 i pitch.
template <typename T>
__device__ __noinline__ void round_tile(const T *x, uint8_t *q, float *scale, int rows, int pitch, bool inside,
                                        unsigned *s_top) {
    Lane16<T> v;
    unsigned top = 0u;
#pragma unroll 1
    for (int i = 0; i < 4; ++i)
        if (inside && 32 * i < rows) {
            v.load(x + 32ll * i * pitch);
            top = max(top, v.settle());
        }
    top = __reduce_max_sync(ALL, top);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = top;
    __syncthreads();
    for (int i = 0; i < 8; ++i) top = max(top, s_top[i]);
    const int e = scale_exp(top);
#pragma unroll 1
    for (int i = 0; i < 4; ++i)
        if (inside && 32 * i < rows) {
            v.load(x + 32ll * i * pitch);
            v.settle();
            *reinterpret_cast<uint4 *>(q + 32ll * i * pitch) = v.pack(pow2(-e));
        }
    if (threadIdx.x == 0) *scale = pow2(e);
}

// A warp per SPAN * 512 columns of a row: 16 columns a lane and chunk of 512
// (16-byte loads and one 16-byte store), eight lanes a block of 128, the
// chunks' loads in flight together.  Scale of row r, block j at
// scale[r * pitch + j].
template <typename T, int SPAN>
__global__ void __launch_bounds__(256, SPAN > 1 ? 4 : 1) quantize_rows_kernel(const T *__restrict__ x, unsigned rows, int cols,
                                                            unsigned spans, const int32_t *__restrict__ src, int n_src,
                                                            uint8_t *__restrict__ q, float *__restrict__ scale,
                                                            int pitch, int32_t *__restrict__ zero, int n_zero) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const unsigned warps = gridDim.x * 8;
    if (zero != nullptr)
        for (int i = blockIdx.x * 256 + threadIdx.x; i < n_zero; i += gridDim.x * 256) zero[i] = 0;
    const unsigned items = rows * spans;
    for (unsigned b = blockIdx.x * 8 + (threadIdx.x >> 5); b < items; b += warps) {
        const unsigned r = b / spans;
        const int c0 = static_cast<int>(b - r * spans) * SPAN * 512 + lane * 16;
        long long from = r;
        if (src != nullptr) {
            from = __ldg(src + r);
            if (from < 0 || from >= n_src) continue;  // past the last entry (or a bad list, reported by the product)
        }
        Lane16<T> v[SPAN];
#pragma unroll
        for (int u = 0; u < SPAN; ++u) {
            if (c0 + u * 512 < cols) v[u].load(x + from * cols + c0 + u * 512);
            else v[u].zero();
        }
        uint8_t *const qr = q + static_cast<long long>(r) * cols;
        float *const sr = scale + static_cast<long long>(r) * pitch;
#pragma unroll
        for (int u = 0; u < SPAN; ++u) {
            const int c = c0 + u * 512;
            unsigned top = v[u].top();
#pragma unroll
            for (int o = 4; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(ALL, top, o));
            if (__any_sync(ALL, top >= INF_BITS)) {  // rare; all lanes together, for the shuffles
                top = v[u].settle();
#pragma unroll
                for (int o = 4; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(ALL, top, o));
            }
            const int e = scale_exp(top);
            if (c < cols) {
                *reinterpret_cast<uint4 *>(qr + c) = v[u].pack(pow2(-e));
                if ((lane & 7) == 0) sr[c / BLK] = pow2(e);
            }
        }
        if (b + warps < b) break;  // the counter would wrap
    }
}

// A block of 256 threads per 128 x 128 tile: eight lanes a row, 32 rows at a
// time, all of the tile's loads in flight at once.
template <typename T>
__global__ void __launch_bounds__(256) quantize_tiles_kernel(const T *__restrict__ x, int rows, int cols, int rb,
                                                             int cb, uint8_t *__restrict__ q,
                                                             float *__restrict__ scale) {
    __shared__ unsigned s_top[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned tile = blockIdx.x, line = tile / cb;
    const int bc = static_cast<int>(tile - line * cb), br = static_cast<int>(line % rb);
    const long long base = static_cast<long long>(line / rb) * rows * cols;
    const int c = bc * BLK + (lane & 7) * 16, r0 = br * BLK + warp * 4 + (lane >> 3);
    Lane16<T> v[4];
    unsigned top = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + 32 * i;
        if (r < rows && c < cols) v[i].load(x + base + static_cast<long long>(r) * cols + c);
        else v[i].zero();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, v[i].top());
    top = __reduce_max_sync(ALL, top);
    if (lane == 0) s_top[warp] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, s_top[i]);
    if (top >= INF_BITS) {  // the same for the whole block
        const long long at = base + static_cast<long long>(r0) * cols + c;
        round_tile(x + at, q + at, scale + tile, rows - r0, cols, c < cols, s_top);
        return;
    }
    const int e = scale_exp(top);
    const float inv = pow2(-e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + 32 * i;
        if (r < rows && c < cols)
            *reinterpret_cast<uint4 *>(q + base + static_cast<long long>(r) * cols + c) = v[i].pack(inv);
    }
    if (threadIdx.x == 0) scale[tile] = pow2(e);
}

// One block per token.  yp, cnt and inv are the kernel's before, which may
// still run when this one starts: no load of theirs may be taken for one of
// unchanging memory and move in front of the wait.
__global__ void __launch_bounds__(256) combine_kernel(const float *yp, const float *w, const int32_t *cnt,
                                                      const int32_t *inv, int d, int k, void *y, int y_bf16) {
    __shared__ int s_p[K_MAX];
    __shared__ float s_w[K_MAX];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int t = blockIdx.x;
    const int n = min(cnt[t], k);
    if (threadIdx.x < n) {  // entries in ascending order
        const int p = inv[static_cast<size_t>(t) * k + threadIdx.x];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += inv[static_cast<size_t>(t) * k + j] < p ? 1 : 0;
        s_p[rank] = p;
        s_w[rank] = w[p];
    }
    __syncthreads();
    for (int c = threadIdx.x * 4; c < d; c += blockDim.x * 4) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int j = 0; j < n; ++j) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(yp + static_cast<size_t>(s_p[j]) * d + c));
            s.x = fmaf(s_w[j], v.x, s.x);
            s.y = fmaf(s_w[j], v.y, s.y);
            s.z = fmaf(s_w[j], v.z, s.z);
            s.w = fmaf(s_w[j], v.w, s.w);
        }
        const size_t at = static_cast<size_t>(t) * d + c;
        if (y_bf16) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
            uint2 o;
            o.x = *reinterpret_cast<const unsigned *>(&lo);
            o.y = *reinterpret_cast<const unsigned *>(&hi);
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(y) + at) = o;
        } else {
            *reinterpret_cast<float4 *>(static_cast<float *>(y) + at) = s;
        }
    }
}

}  // namespace

namespace {
template <typename T, int SPAN>
cudaError_t launch_span(const void *x, long long rows, int cols, const int32_t *src, int n_src, uint8_t *q, float *scale,
                        int pitch, int32_t *zero, int n_zero, cudaStream_t s) {
    const unsigned spans = (cols + SPAN * 512 - 1) / (SPAN * 512);
    const long long blocks = (rows * spans + 7) / 8;
    const unsigned grid = static_cast<unsigned>(blocks < 148 * 32 ? blocks : 148 * 32);
    quantize_rows_kernel<T, SPAN><<<grid, 256, 0, s>>>(static_cast<const T *>(x), static_cast<unsigned>(rows), cols, spans,
                                                       src, n_src, q, scale, pitch, zero, n_zero);
    return cudaGetLastError();
}
cudaError_t launch_rows(const void *x, int type, long long rows, int cols, const int32_t *src, int n_src, uint8_t *q,
                        float *scale, int pitch, int32_t *zero, int n_zero, cudaStream_t s) {
    // many rows: the row index (and the gathered row's) once for 1024 or
    // 2048 columns; few: as many warps as there are chunks
    const bool many = rows >= WIDE_ROWS;
    if (type == MOE_BF16)
        return many ? launch_span<__nv_bfloat16, 4>(x, rows, cols, src, n_src, q, scale, pitch, zero, n_zero, s)
                    : launch_span<__nv_bfloat16, 1>(x, rows, cols, src, n_src, q, scale, pitch, zero, n_zero, s);
    return many ? launch_span<float, 2>(x, rows, cols, src, n_src, q, scale, pitch, zero, n_zero, s)
                : launch_span<float, 1>(x, rows, cols, src, n_src, q, scale, pitch, zero, n_zero, s);
}
}  // namespace

cudaError_t launch_quantize_dispatch(const void *x, int type, int64_t rows, int cols, const int32_t *src, int n_src,
                                     uint8_t *q, float *scale, int32_t *zero, int n_zero, cudaStream_t s) {
    return launch_rows(x, type, rows, cols, src, n_src, q, scale, scale_pitch(cols), zero, n_zero, s);
}

cudaError_t launch_quantize(const void *x, int type, int64_t batch, int64_t rows, int64_t cols, int block_rows,
                            uint8_t *q, float *scale, cudaStream_t s) {
    const int cb = blocks_of(static_cast<int>(cols)), c = static_cast<int>(cols);
    if (block_rows == 1) return launch_rows(x, type, batch * rows, c, nullptr, 0, q, scale, cb, nullptr, 0, s);
    const int rb = blocks_of(static_cast<int>(rows)), r = static_cast<int>(rows);
    const unsigned grid = static_cast<unsigned>(batch * rb * cb);
    if (type == MOE_BF16)
        quantize_tiles_kernel<<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16 *>(x), r, c, rb, cb, q, scale);
    else
        quantize_tiles_kernel<<<grid, 256, 0, s>>>(static_cast<const float *>(x), r, c, rb, cb, q, scale);
    return cudaGetLastError();
}

cudaError_t launch_combine(const float *yp, const float *w, const int32_t *cnt, const int32_t *inv, int B, int d,
                           int k, void *y, int y_bf16, cudaStream_t s) {
    const int threads = d >= 1024 ? 256 : 64;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(B);
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, combine_kernel, yp, w, cnt, inv, d, k, y, y_bf16);
}

}  // namespace moe

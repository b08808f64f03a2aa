// Block-scaled 8-bit expert products (sm_100a): y = W[e] x per list entry,
// e4m3 operands, one fp32 scale per 128 columns of an activation row and per
// 128 x 128 block of a weight matrix, on the 5th-generation tensor cores.
//
// A tile is up to 128 list entries of one expert (the MMA's M, TMEM lanes)
// by 256 weight rows (its N): for a plain product 256 rows of W, for the
// gate/up product 128 rows of Wgate and the same 128 of Wup.  Scales change
// every 128 columns, so the sum over a column block is formed in TMEM by
// four MMAs of K = 32 and added, times the row's and the block's scale, to
// fp32 accumulators in registers: thread (row, column half) of the eight
// epilogue warps holds 128 of the row's 256 sums.  With the entries on the
// lanes a row's scale is one register, and SwiGLU, the largest magnitude of
// a block of h and its rounding to e4m3 stay inside a thread (two threads
// share a block).  Two TMEM buffers of 256 columns let the MMAs of the next
// column block run while one is added.
//
// Persistent CTAs, one per SM, take tiles round robin.  Roles: warps 0-7
// epilogue, warp 8 loads (weights as TMA boxes, activation rows gathered
// four at a time by list entry), warp 9 issues the MMAs.  Every wait is
// bounded; past the limit the CTA records an error, lets its copies and
// MMAs land and leaves.
#include <cuda_bf16.h>

#include "blocks.h"
#include "tcgen05.cuh"

namespace moe {
namespace {

constexpr unsigned ALL = 0xffffffffu;
constexpr int TILE_M = 128;       // list entries per tile
constexpr int TILE_N = 256;       // weight rows per tile (128 + 128 for gate/up)
constexpr int W_STAGE = TILE_N * BLK;  // weight bytes of a stage: 256 rows x 128 columns
constexpr int A_STAGE = TILE_M * BLK;
constexpr int STAGE = W_STAGE + A_STAGE;
constexpr int STAGES = 4;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = (EPI_WARPS + 2) * 32;
constexpr int OUT_PITCH = 80;     // bytes of a staged output row: 64 and a pad that spreads the banks
constexpr int OUT_STAGE = 32 * OUT_PITCH;
constexpr unsigned long long DRAIN_NS = 1000000000ull;

struct Ctl {
    unsigned long long full[STAGES], empty[STAGES];
    unsigned long long part_full[2], part_free[2];
    unsigned long long mma_done;
    volatile int abort_flag;
    int n_slots, n_tiles;
    uint32_t tmem;
    float top[2][2][TILE_M];  // [tile parity][column half][row]: largest |h|
    int act[SE_MAX], off[SE_MAX + 1], mt[SE_MAX + 1];  // expert, first entry, first m-tile of a slot
};
constexpr int SMEM_BYTES = 1024 + STAGES * STAGE + EPI_WARPS * OUT_STAGE + static_cast<int>(sizeof(Ctl));
static_assert(SMEM_BYTES <= 232448, "shared memory budget");

// ---------------------------------------------------------------- PTX --
__device__ __forceinline__ uint32_t saddr(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ unsigned long long clock_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
__device__ __forceinline__ void bar_init(unsigned long long *b, unsigned n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_expect(unsigned long long *b, unsigned bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(unsigned long long *b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(b)) : "memory");
}
__device__ __forceinline__ bool bar_try(unsigned long long *b, unsigned parity) {
    unsigned ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(saddr(b)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void load_box(void *dst, const CUtensorMap *map, int c, int r, int e,
                                         unsigned long long *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(saddr(dst)),
        "l"(reinterpret_cast<unsigned long long>(map)), "r"(c), "r"(r), "r"(e), "r"(saddr(bar))
        : "memory");
}
__device__ __forceinline__ void load_rows4(void *dst, const CUtensorMap *map, int c, const int (&r)[4],
                                           unsigned long long *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(saddr(dst)),
        "l"(reinterpret_cast<unsigned long long>(map)), "r"(c), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
        "r"(saddr(bar))
        : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}
// Instruction descriptor of kind::f8f6f4: e4m3 A and B (format code 0), fp32
// accumulator, both K-major, M = 128, N = 256.
constexpr uint32_t IDESC = (1u << 4) | (static_cast<uint32_t>(TILE_N >> 3) << 17) |
                           (static_cast<uint32_t>(TILE_M >> 4) << 24);
__device__ __forceinline__ void umma_e4m3(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(IDESC), "r"(accumulate)
        : "memory");
}
// 32 consecutive fp32 columns of the warp's 32 TMEM lanes
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

// Bounded wait on an mbarrier phase; false once the CTA has given up.
__device__ bool wait_bar(unsigned long long *b, unsigned parity, Ctl *ctl, const ProductArgs &a, int code) {
    if (bar_try(b, parity)) return true;
    const unsigned long long t0 = clock_ns();
    for (;;) {
        if (bar_try(b, parity)) return true;
        if (ctl->abort_flag) return false;
        if (clock_ns() - t0 > a.wait_ns) {
            atomicCAS(a.error, 0, code);
            ctl->abort_flag = 1;
            return false;
        }
    }
}

// --------------------------------------------------------------- tiles --
struct Tile {
    int slot, e, p0, n, nb;  // slot, expert, first entry, entries, column tile
};
// Tile t: slots in order, within a slot the column tiles, within one the
// m-tiles (neighbouring CTAs then share weights in L2).
__device__ __forceinline__ Tile tile_at(int t, int nbt, const Ctl *ctl) {
    int lo = 0, hi = ctl->n_slots - 1;
    const int v = t / nbt;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (ctl->mt[mid] <= v) lo = mid;
        else hi = mid - 1;
    }
    const int mts = ctl->mt[lo + 1] - ctl->mt[lo];
    const int r = t - ctl->mt[lo] * nbt;
    Tile x;
    x.slot = lo;
    x.e = ctl->act[lo];
    x.nb = r / mts;
    const int m = r - x.nb * mts;
    x.p0 = ctl->off[lo] + m * TILE_M;
    x.n = min(TILE_M, ctl->off[lo + 1] - x.p0);
    return x;
}

// Slots with no entries hold no m-tile; the search above never lands on one
// because it takes the last slot whose first m-tile is at most v.

// The call's slots from the lists, checked before anything indexes with
// them: inconsistent lists run as an empty call and are recorded.
__device__ void build_slots(Ctl *ctl, const ProductArgs &a, int nbt) {
    __shared__ int s_bad;
    const int most = min(a.E, a.B * a.k);
    if (threadIdx.x == 0) s_bad = 0;
    __syncthreads();
    int n = __ldg(a.n_active);
    if (n < 0 || n > most) {
        n = 0;
        if (threadIdx.x == 0) s_bad = 1;
    }
    for (int i = threadIdx.x; i <= n; i += blockDim.x) {
        const int o = __ldg(a.offsets + i);
        ctl->off[i] = o;
        bool bad = o < 0 || o > a.B * a.k || (i == 0 && n > 0 && o != 0);
        if (i < n) {
            const int e = __ldg(a.active + i), next = __ldg(a.offsets + i + 1);
            ctl->act[i] = e;
            bad = bad || e < 0 || e >= a.E || next < o || next - o > a.B;
        }
        if (bad) s_bad = 1;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        if (s_bad) n = 0;
        int run = 0;
        for (int i0 = 0; i0 < n; i0 += 32) {
            const int i = i0 + threadIdx.x;
            int v = i < n ? (ctl->off[i + 1] - ctl->off[i] + TILE_M - 1) / TILE_M : 0;
            const int mine = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(ALL, v, o);
                if (static_cast<int>(threadIdx.x) >= o) v += u;
            }
            if (i < n) ctl->mt[i] = run + v - mine;
            run += __shfl_sync(ALL, v, 31);
        }
        if (threadIdx.x == 0) {
            ctl->mt[n] = run;
            ctl->n_slots = n;
            ctl->n_tiles = run * nbt;
            if (s_bad && blockIdx.x == 0) atomicCAS(a.error, 0, DEV_BAD_LISTS);
        }
    }
    __syncthreads();
}

// --------------------------------------------------------------- roles --
__device__ void producer(unsigned char *ring, Ctl *ctl, const ProductMaps &maps, const ProductArgs &a, int nbt,
                         int kb) {
    const int lane = threadIdx.x & 31;
    const int last_row = (a.by_pair ? a.B * a.k : a.B) - 1;
    unsigned it = 0;
    for (int t = blockIdx.x; t < ctl->n_tiles; t += gridDim.x) {
        const Tile x = tile_at(t, nbt, ctl);
        int rows[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // rows past the tile's end repeat its last one (their sums are not used)
            const int p = x.p0 + min(lane * 4 + j, x.n - 1);
            int r = a.by_pair ? p : __ldg(a.tok + p);
            if (r < 0 || r > last_row) {
                atomicCAS(a.error, 0, DEV_BAD_LISTS);
                r = 0;
            }
            rows[j] = r;
        }
        const int groups = (x.n + 3) >> 2;
        const int r0 = a.kind == PRODUCT_SWIGLU ? x.nb * BLK : x.nb * TILE_N;
        const int r1 = a.kind == PRODUCT_SWIGLU ? r0 : r0 + BLK;
        for (int j = 0; j < kb; ++j, ++it) {
            const int st = it % STAGES;
            unsigned char *w = ring + st * STAGE;
            const bool ok = it < STAGES || wait_bar(&ctl->empty[st], ((it / STAGES) - 1) & 1, ctl, a, DEV_TIMEOUT_EMPTY);
            if (!__all_sync(ALL, ok)) goto drain;
            if (lane == 0) {
                bar_expect(&ctl->full[st], W_STAGE + groups * 4 * BLK);
                load_box(w, &maps.b0, j * BLK, r0, x.e, &ctl->full[st]);
                load_box(w + W_STAGE / 2, &maps.b1, j * BLK, r1, x.e, &ctl->full[st]);
            }
            __syncwarp();
            if (lane < groups) load_rows4(w + W_STAGE + lane * 4 * BLK, &maps.a, j * BLK, rows, &ctl->full[st]);
            __syncwarp();
        }
    }
drain:
    // copies in flight land before the CTA's shared memory goes away
    if (lane == 0) {
        const unsigned long long t0 = clock_ns();
        for (unsigned i = it > STAGES ? it - STAGES : 0; i < it; ++i)
            while (!bar_try(&ctl->full[i % STAGES], (i / STAGES) & 1) && clock_ns() - t0 < DRAIN_NS) {
            }
    }
    __syncwarp();
}

__device__ void issuer(unsigned char *ring, Ctl *ctl, const ProductArgs &a, int kb) {
    unsigned it = 0;
    const uint32_t tmem = ctl->tmem;
    const bool leader = elect_one();
    for (int t = blockIdx.x; t < ctl->n_tiles; t += gridDim.x) {
        for (int j = 0; j < kb; ++j, ++it) {
            const int st = it % STAGES, buf = it & 1;
            bool ok = it < 2 || wait_bar(&ctl->part_free[buf], ((it >> 1) - 1) & 1, ctl, a, DEV_TIMEOUT_DEP);
            ok = ok && wait_bar(&ctl->full[st], (it / STAGES) & 1, ctl, a, DEV_TIMEOUT_FULL);
            if (!__all_sync(ALL, ok)) goto drain;
            tc_fence_after();
            if (leader) {
                const uint64_t b = umma_desc(saddr(ring + st * STAGE));
                const uint64_t x = umma_desc(saddr(ring + st * STAGE + W_STAGE));
#pragma unroll
                for (int s = 0; s < 4; ++s)  // 32 columns = 32 bytes each
                    umma_e4m3(tmem + buf * TILE_N, x + 2 * s, b + 2 * s, s > 0);
                umma_commit(saddr(&ctl->empty[st]));
                umma_commit(saddr(&ctl->part_full[buf]));
            }
            __syncwarp();
        }
    }
drain:
    if (leader) {
        umma_commit(saddr(&ctl->mma_done));
        const unsigned long long t0 = clock_ns();
        while (!bar_try(&ctl->mma_done, 0) && clock_ns() - t0 < DRAIN_NS) {
        }
    }
    __syncwarp();
}

__device__ __forceinline__ void epi_bar() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// 32 rows x 64 bytes of a warp's output through shared memory: lane l wrote
// its row's four 16-byte pieces; rows go out as whole 64-byte runs.
__device__ __forceinline__ void store_chunk(unsigned char *stage, const uint4 (&v)[4], char *out, size_t pitch,
                                            int rows, int lane, int bytes) {
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4 *>(stage + lane * OUT_PITCH + i * 16) = v[i];
    __syncwarp();
    const int piece = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 2);
        if (r < rows && piece * 16 < bytes)
            *reinterpret_cast<uint4 *>(out + static_cast<size_t>(r) * pitch + piece * 16) =
                *reinterpret_cast<const uint4 *>(stage + r * OUT_PITCH + piece * 16);
    }
    __syncwarp();
}

__device__ __forceinline__ unsigned pack_e4m3(float a, float b, float c, float d) {
    unsigned short lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<unsigned>(lo) | (static_cast<unsigned>(hi) << 16);
}
__device__ __forceinline__ unsigned pack_bf16(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const unsigned *>(&v);
}

__device__ void epilogue(unsigned char *out_stage, Ctl *ctl, const ProductArgs &a, int nbt, int kb) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quarter = warp & 3, half = warp >> 2;  // TMEM lanes 32 quarter .., columns 64 half .. of each matrix
    const int row = quarter * 32 + lane;
    const uint32_t tbase = ctl->tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * 64;
    const int rb = (a.rows + BLK - 1) / BLK;
    unsigned char *stage = out_stage + warp * OUT_STAGE;
    bool dead = false;
    unsigned it = 0;
    int parity = 0;
    for (int t = blockIdx.x; t < ctl->n_tiles; t += gridDim.x, parity ^= 1) {
        const Tile x = tile_at(t, nbt, ctl);
        const bool live = quarter * 32 < x.n;  // the warp holds rows of the tile
        const int p = x.p0 + min(row, x.n - 1);
        int ar = a.by_pair ? p : __ldg(a.tok + p);
        if (ar < 0 || ar >= (a.by_pair ? a.B * a.k : a.B)) ar = 0;  // recorded by the producer
        const float *as = a.as + static_cast<size_t>(ar) * kb;
        const int nb0 = a.kind == PRODUCT_SWIGLU ? x.nb : 2 * x.nb;
        const int nb1 = a.kind == PRODUCT_SWIGLU ? x.nb : min(2 * x.nb + 1, rb - 1);
        const float *s0 = a.bs0 + (static_cast<size_t>(x.e) * rb + nb0) * kb;
        const float *s1 = a.bs1 + (static_cast<size_t>(x.e) * rb + nb1) * kb;
        float c0[64], c1[64];
#pragma unroll
        for (int i = 0; i < 64; ++i) c0[i] = c1[i] = 0.0f;
        float fa = __ldg(as), f0 = __ldg(s0), f1 = __ldg(s1);
        for (int j = 0; j < kb; ++j, ++it) {
            const int buf = it & 1;
            const float m0 = fa * f0, m1 = fa * f1;
            if (j + 1 < kb) {
                fa = __ldg(as + j + 1);
                f0 = __ldg(s0 + j + 1);
                f1 = __ldg(s1 + j + 1);
            }
            if (!__all_sync(ALL, !dead && wait_bar(&ctl->part_full[buf], (it >> 1) & 1, ctl, a, DEV_TIMEOUT_FULL)))
                dead = true;
            if (!dead) {
                tc_fence_after();
                if (live) {
                    const uint32_t col = tbase + buf * TILE_N;
                    uint32_t v[32];
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        tmem_ld32(col + q * 32, v);
#pragma unroll
                        for (int i = 0; i < 32; ++i) c0[q * 32 + i] = fmaf(__uint_as_float(v[i]), m0, c0[q * 32 + i]);
                        tmem_ld32(col + 128 + q * 32, v);
#pragma unroll
                        for (int i = 0; i < 32; ++i) c1[q * 32 + i] = fmaf(__uint_as_float(v[i]), m1, c1[q * 32 + i]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&ctl->part_free[buf]);
            }
        }
        const int rows_here = min(32, x.n - quarter * 32);
        if (a.kind == PRODUCT_SWIGLU) {
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < 64; ++i) {
                c0[i] = c0[i] / (1.0f + expf(-c0[i])) * c1[i];
                top = fmaxf(top, fabsf(c0[i]));
            }
            ctl->top[parity][half][row] = top;
            epi_bar();
            if (live && !dead) {
                top = fmaxf(ctl->top[parity][0][row], ctl->top[parity][1][row]);
                const unsigned tb = __float_as_uint(top);
                int e = tb == 0u ? 0 : static_cast<int>(tb >> 23) - 135 + ((tb & 0x7fffffu) > 0x600000u ? 1 : 0);
                e = e < -120 ? -120 : e;
                const float inv = __int_as_float((127 - e) << 23);
                uint4 o[4];
                unsigned *w = reinterpret_cast<unsigned *>(o);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    w[i] = pack_e4m3(c0[4 * i] * inv, c0[4 * i + 1] * inv, c0[4 * i + 2] * inv, c0[4 * i + 3] * inv);
                const int f = x.nb * BLK + half * 64;
                const size_t at = static_cast<size_t>(x.p0 + quarter * 32);
                store_chunk(stage, o, reinterpret_cast<char *>(a.hq) + at * a.rows + f, a.rows, rows_here, lane,
                            a.rows - f);
                if (row < x.n && half == 0) a.hs[static_cast<size_t>(p) * rb + x.nb] = __int_as_float((127 + e) << 23);
                if (x.nb == 0 && half == 0 && a.cnt != nullptr && row < x.n) {
                    const int c = atomicAdd(a.cnt + ar, 1);  // by_pair is 0: ar is the entry's token
                    if (c < a.k) a.inv[static_cast<size_t>(ar) * a.k + c] = p;
                    else atomicCAS(a.error, 0, DEV_BAD_LISTS);
                }
            }
        } else if (live && !dead) {
            const size_t at = static_cast<size_t>(x.p0 + quarter * 32) * a.rows;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const float(&c)[64] = m == 0 ? c0 : c1;
                const int n0 = x.nb * TILE_N + m * BLK + half * 64;
                uint4 o[4];
                unsigned *w = reinterpret_cast<unsigned *>(o);
                if (a.out_bf16) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) w[i] = pack_bf16(c[q * 32 + 2 * i], c[q * 32 + 2 * i + 1]);
                        store_chunk(stage, o, static_cast<char *>(a.out) + (at + n0 + q * 32) * 2,
                                    static_cast<size_t>(a.rows) * 2, rows_here, lane, (a.rows - n0 - q * 32) * 2);
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(c[q * 16 + i]);
                        store_chunk(stage, o, static_cast<char *>(a.out) + (at + n0 + q * 16) * 4,
                                    static_cast<size_t>(a.rows) * 4, rows_here, lane, (a.rows - n0 - q * 16) * 4);
                    }
                }
            }
        }
    }
}

__global__ void __launch_bounds__(THREADS, 1) product_kernel(const __grid_constant__ ProductMaps maps,
                                                             const __grid_constant__ ProductArgs a) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char *ring =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char *out_stage = ring + STAGES * STAGE;
    Ctl *ctl = reinterpret_cast<Ctl *>(out_stage + EPI_WARPS * OUT_STAGE);
    const int warp = threadIdx.x >> 5;
    const int kb = (a.K + BLK - 1) / BLK;
    const int nbt = a.kind == PRODUCT_SWIGLU ? (a.rows + BLK - 1) / BLK : (a.rows + TILE_N - 1) / TILE_N;
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            bar_init(&ctl->full[i], 1);
            bar_init(&ctl->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&ctl->part_full[i], 1);
            bar_init(&ctl->part_free[i], EPI_WARPS);
        }
        bar_init(&ctl->mma_done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        ctl->abort_flag = 0;
    }
    if (warp == EPI_WARPS + 1) tmem_alloc(saddr(&ctl->tmem), 512);
    tc_fence_before();
    build_slots(ctl, a, nbt);  // ends in a block barrier
    tc_fence_after();
    if (warp < EPI_WARPS) epilogue(out_stage, ctl, a, nbt, kb);
    else if (warp == EPI_WARPS) producer(ring, ctl, maps, a, nbt, kb);
    else issuer(ring, ctl, a, kb);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == EPI_WARPS + 1) tmem_dealloc(ctl->tmem, 512);
}

}  // namespace

cudaError_t launch_product(const ProductMaps &maps, const ProductArgs &a, cudaStream_t s) {
    // per device: the SM count, and the shared-memory attribute set
    static int sms[MAX_DEVICES] = {};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= MAX_DEVICES) return cudaErrorInvalidDevice;
    if (sms[dev] == 0) {
        int n = 0;
        err = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (err != cudaSuccess) return err;
        err = cudaFuncSetAttribute(product_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
        if (err != cudaSuccess) return err;
        sms[dev] = n;
    }
    product_kernel<<<sms[dev], THREADS, SMEM_BYTES, s>>>(maps, a);
    return cudaGetLastError();
}

}  // namespace moe

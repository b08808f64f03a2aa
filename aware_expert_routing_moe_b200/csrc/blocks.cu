// Block-scaled 8-bit expert products (sm_100a): y = W[e] x per list entry,
// e4m3 operands, one fp32 scale per 128 columns of an activation row and per
// 128 x 128 block of a weight matrix, on the 5th-generation tensor cores.
//
// A tile is some list entries of one expert by 256 weight rows: for a plain
// product 256 rows of W, for the gate/up product 128 rows of Wgate and the
// same 128 of Wup.  Scales change every 128 columns, so the sum over a column
// block is formed in TMEM by MMAs of K = 32 and added, times the row's and
// the block's scale, to fp32 accumulators in the registers of eight epilogue
// warps; several TMEM buffers let the MMAs of the next blocks run meanwhile.
//
// Few entries (up to 16 a tile): the weights are the MMA's M (two MMAs of
// 128 rows), the entries its N.  An MMA then costs what its entries cost:
// with the entries as a half-empty M of 128 the decode kernels drew 990 W and
// lost a sixth of their speed to the power cap (8 tokens, Qwen3-235B shape,
// back to back: 174 us against 150 in a short run).  A thread holds one
// weight row of both matrices for 8 entries.
// Many entries (up to 128 a tile): the entries are M (TMEM lanes), the 256
// weight rows N.  An entry's scale is then one register, and SwiGLU, the
// largest magnitude of a block of h and its rounding to e4m3 stay inside a
// thread: thread (entry, column half) holds 128 of the entry's 256 sums.
//
// A call is one phase (a plain product) or two (gate/up, then down, whose
// activations are the first phase's h).  Persistent CTAs, one per SM, claim
// tiles from a counter, all of the first phase's before the second's; a down
// tile waits until its entries' gate/up tiles are counted done.  A tile is
// claimed only by a running CTA, so no wait depends on a CTA that has not
// started.  The last CTA puts the counters back to zero.
//
// Roles: warps 0-7 epilogue; warp 8 weights (TMA boxes; they do not wait for
// the tile's activations); warp 9 MMAs; warp 10 activation rows (boxes of 32
// where they are consecutive, else gathered four at a time) and the scales of
// each column block, copied to a ring of their own, so that no global load
// latency sits in the epilogue's loop; warp 11 claims tiles and publishes
// finished ones.  Every wait is bounded; past the limit the CTA records an
// error, lets its copies and MMAs land and leaves.
//
// What bounds it, measured.  Few entries: HBM.  Expert FFN, Qwen3-30B shape,
// 16 tokens: 62 us for 321 MB (58 of it this kernel, 312 MB read, 5.4 TB/s,
// tensor pipe 4 % busy); 1 token 25 us, of which the chain of latencies
// (claim, first copies, gate/up, publication, down, combine) is about 20;
// Qwen3-235B shape, 8 tokens: 134 us, 6.3 TB/s.  Many entries: the copies from
// L2 and the additions.  A stage of 48 KB takes about 970 cycles to arrive,
// its four MMAs 512, the additions 500 to 1100: product 2000 x 4096 x 4096
// 52 us (1.29 PFLOP/s), expert FFN with 4096 tokens 376 us.  Pairs of CTAs
// (cta_group::2), which halve the weight copies, were no faster: then the
// sub-partition that issues the MMAs falls behind with its additions.
#include <cuda_bf16.h>

#include "blocks.h"
#include "tcgen05.cuh"

namespace moe {
namespace {

constexpr unsigned ALL = 0xffffffffu;
constexpr int TILE_MANY = 128, TILE_FEW = 16;  // list entries per tile
constexpr int TILE_N = 256;       // weight rows per tile (128 + 128 for gate/up)
constexpr int W_STAGE = TILE_N * BLK;  // weight bytes of a stage: 256 rows x 128 columns
constexpr int EPI_WARPS = 8;
constexpr int THREADS = (EPI_WARPS + 4) * 32;
// Registers a thread: the block starts with 168 (384 threads); with many
// entries the four copy and issue warps give theirs up for the epilogue's
// accumulators.
constexpr int REGS_EPI = 224, REGS_COPY = 56;
static_assert(256 * REGS_EPI + 128 * REGS_COPY <= THREADS * 168, "register split");
constexpr int OUT_PITCH = 80;     // bytes of a staged output row: 64 and a pad that spreads the banks
constexpr int OUT_STAGE = 32 * OUT_PITCH;
constexpr int SGROUP = 4;         // column blocks whose scales are copied together (16 bytes a row)
constexpr int SCALES = 3;         // such groups in flight
constexpr int TILES = 2;          // tiles claimed ahead
constexpr int PUBS = 4;           // tiles claimed and not yet published, at most
// Tiles are of 16 entries up to FEW_AVERAGE entries an expert on average
// (expert FFN, d 2048, d_ff 1024, 64 experts: 12 entries 78.8 against 85.3 us
// with tiles of 128, 20 entries 86.2 and 88.8, 24 entries 95.9 and 90.1; of
// 64 entries, as an N of up to 64, 82.2, 92.6 and 96.4), and where an expert
// has at most two such tiles (32 tokens, 8 experts: 32.7 against 37.8 us).
constexpr int FEW_AVERAGE = 20;
constexpr int BOX_ROWS = 32;      // activation rows per copy where they are consecutive
constexpr unsigned long long DRAIN_CYCLES = 2000000000ull;  // 1 s

// A kernel for tiles of AR entries: AR activation rows per stage; with few
// entries two more stages fit, and four TMEM buffers.
template <int AR>
struct Ring {
    static constexpr bool FEW = AR == TILE_FEW;
    static constexpr int A_STAGE = AR * BLK;
    static constexpr int STAGE = W_STAGE + A_STAGE;
    static constexpr int STAGES = FEW ? 6 : 4;
    static constexpr int OUT_BYTES = FEW ? AR * BLK : EPI_WARPS * OUT_STAGE;  // h of a tile, or a piece a warp
    static constexpr int BOX = AR < BOX_ROWS ? AR : BOX_ROWS;  // rows per copy
    static constexpr int BUFS = FEW ? 4 : 2;          // TMEM buffers
    static constexpr int BUF_COLS = 512 / BUFS;       // two blocks of entries, or 256 weight rows
};

enum : int { TILE_END = 2 };
struct Tile {
    int phase, e, p0, n, nb, mt;  // phase (TILE_END: no more), expert, first entry, entries, column tile, m-tile
    int ready;                    // down: its gate/up tiles were done when it was claimed
};

struct Ctl {
    unsigned long long full[6], empty[6];
    unsigned long long part_full[4], part_free[4];
    unsigned long long scale_full[SCALES], scale_free[SCALES];
    unsigned long long tile_full[TILES], tile_free[TILES];
    unsigned long long pub_full[PUBS];
    unsigned long long mma_done;
    volatile int abort_flag;
    int n_slots, m_tiles;
    unsigned fills[2];  // stages filled with weights, with rows
    uint32_t tmem;
    Tile tile[TILES];
    int rows[TILES][TILE_MANY];          // activation row of each entry of a claimed tile
    Tile own[EPI_WARPS];              // many entries: each epilogue warp's tile, out of its registers
    unsigned handed[EPI_WARPS];       // and the gate/up tiles it has handed over
    int pub_mt[PUBS];                    // m-tile of a finished gate/up tile
    float4 scale[SCALES][TILE_MANY];     // each row's scales of a group of column blocks
    float wscale[SCALES][2][SGROUP];  // and the two weight blocks'
    float top[4][TILE_MANY];          // largest |h|: [column half][entry], few entries: [quarter of the rows][entry]
    int off[SE_MAX + 1];              // first entry of a slot, its first m-tile, its expert
    uint16_t mt[SE_MAX + 1], act[SE_MAX];
};
template <int AR>
constexpr int smem_bytes() {
    return 1024 + Ring<AR>::STAGES * Ring<AR>::STAGE + Ring<AR>::OUT_BYTES + static_cast<int>(sizeof(Ctl));
}
static_assert(ST_MAX * K_MAX / TILE_MANY + SE_MAX < 65536 && (FEW_AVERAGE + TILE_FEW) * SE_MAX / TILE_FEW < 65536,
              "m-tile numbers are 16 bits");
static_assert(smem_bytes<TILE_MANY>() <= 232448 - 64 && smem_bytes<TILE_FEW>() <= 232448 - 64, "shared memory budget");
// ---------------------------------------------------------------- PTX --
__device__ __forceinline__ uint32_t saddr(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
// Time for the bounded waits: SM cycles at the highest clock, so that a limit
// is never shorter than asked for (reading the global timer instead costs
// every wait that does not succeed at once several hundred nanoseconds).
constexpr unsigned long long CYCLES_PER_NS = 2;
__device__ __forceinline__ unsigned long long cycles() { return static_cast<unsigned long long>(clock64()); }
__device__ __forceinline__ void bar_init(unsigned long long *b, unsigned n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_expect(unsigned long long *b, unsigned bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(unsigned long long *b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(b)) : "memory");
}
__device__ __forceinline__ void copy16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(saddr(dst)), "l"(src) : "memory");
}
// four bytes global -> shared; arrive on b when this thread's copies land
__device__ __forceinline__ void copy4(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(saddr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_arrive(unsigned long long *b) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(saddr(b)) : "memory");
}
__device__ __forceinline__ int ld_acquire(const int32_t *p) {
    int v;
    asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void add_release(int32_t *p) {
    asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(p) : "memory");
}
// orders generic-proxy accesses with the TMA copies of this or another CTA
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async;" ::: "memory"); }
// c (two floats) += a (two floats) * b
__device__ __forceinline__ void fma2(float &c0, float &c1, uint32_t a0, uint32_t a1, float b) {
    asm("{\n\t.reg .b64 a, b, c;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmov.b64 c, {%0, %1};\n\t"
        "fma.rn.f32x2 c, a, b, c;\n\t"
        "mov.b64 {%0, %1}, c;\n\t}"
        : "+f"(c0), "+f"(c1)
        : "r"(a0), "r"(a1), "f"(b));
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
// The same without the wait that try_wait may take before it says no.
__device__ __forceinline__ bool bar_test(unsigned long long *b, unsigned parity) {
    unsigned ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
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
__device__ __forceinline__ void load_rows(void *dst, const CUtensorMap *map, int c, int r, unsigned long long *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(saddr(dst)),
        "l"(reinterpret_cast<unsigned long long>(map)), "r"(c), "r"(r), "r"(saddr(bar))
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
// accumulator, both K-major, M = 128, N = n (a multiple of 16).
__device__ __forceinline__ uint32_t idesc_e4m3(int n) {
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (128u >> 4 << 24);
}
__device__ __forceinline__ void umma_e4m3(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// 32 consecutive fp32 columns of the warp's 32 TMEM lanes; the registers
// hold them after tmem_wait, which also waits for the loads issued before
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

// eight columns from each of two places, waited for
__device__ __forceinline__ void tmem_ld8x2(uint32_t t0, uint32_t t1, float (&u)[8], float (&v)[8]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%16];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%17];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(t0), "r"(t1)
        : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        u[i] = __uint_as_float(r[i]);
        v[i] = __uint_as_float(r[8 + i]);
    }
}

// Bounded wait on an mbarrier phase; false once the CTA has given up.
__device__ __forceinline__ bool wait_slow(unsigned long long *b, unsigned parity, Ctl *ctl, const ProductArgs &a, int code) {
    const unsigned long long t0 = cycles();
    for (;;) {
        if (bar_try(b, parity)) return true;
        if (ctl->abort_flag) return false;
        if (cycles() - t0 > a.wait_ns * CYCLES_PER_NS) {
            atomicCAS(a.error, 0, code);
            ctl->abort_flag = 1;
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_bar(unsigned long long *b, unsigned parity, Ctl *ctl, const ProductArgs &a,
                                         int code) {
    return bar_try(b, parity) || wait_slow(b, parity, ctl, a, code);
}

// --------------------------------------------------------------- tiles --
// Tile t of a phase with nbt column tiles: slots in order, within a slot the
// column tiles, within one the m-tiles (CTAs that run together then share
// weights in L2).  A slot without entries holds no m-tile: the search takes
// the last slot whose first m-tile is at most t / nbt.
template <int AR>
__device__ Tile tile_at(int t, int phase, int nbt, const Ctl *ctl) {
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
    x.phase = phase;
    x.e = ctl->act[lo];
    x.nb = r / mts;
    const int m = r - x.nb * mts;
    x.mt = ctl->mt[lo] + m;
    x.p0 = ctl->off[lo] + m * AR;
    x.n = min(AR, ctl->off[lo + 1] - x.p0);
    return x;
}

// The call's slots from the lists, checked before anything indexes with
// them: inconsistent lists run as an empty call and are recorded.
template <int AR>
__device__ void build_slots(Ctl *ctl, const ProductArgs &a) {
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
            ctl->act[i] = static_cast<uint16_t>(e);
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
            int v = i < n ? (ctl->off[i + 1] - ctl->off[i] + AR - 1) / AR : 0;
            const int mine = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(ALL, v, o);
                if (static_cast<int>(threadIdx.x) >= o) v += u;
            }
            if (i < n) ctl->mt[i] = static_cast<uint16_t>(run + v - mine);
            run += __shfl_sync(ALL, v, 31);
        }
        if (threadIdx.x == 0) {
            ctl->mt[n] = static_cast<uint16_t>(run);
            ctl->n_slots = n;
            ctl->m_tiles = run;
            if (s_bad && blockIdx.x == 0) atomicCAS(a.error, 0, DEV_BAD_LISTS);
        }
    }
    __syncthreads();
}

__device__ __forceinline__ int column_tiles(const ProductPhase &p) {
    return p.kind == PRODUCT_SWIGLU ? (p.rows + BLK - 1) / BLK : (p.rows + TILE_N - 1) / TILE_N;
}

// The next tile of the CTA's sequence; false: none (or given up).
struct TileCursor {
    unsigned i = 0;
    __device__ __forceinline__ bool next(Ctl *ctl, const ProductArgs &a, Tile &x) {
        const int s = i % TILES;
        if (!wait_bar(&ctl->tile_full[s], (i / TILES) & 1, ctl, a, DEV_TIMEOUT_FULL)) return false;
        x = ctl->tile[s];
        return true;
    }
    __device__ __forceinline__ void release(Ctl *ctl) {
        bar_arrive(&ctl->tile_free[i % TILES]);
        ++i;
    }
};

// --------------------------------------------------------------- roles --
// Claims tiles ahead of the other roles (with the activation rows of their
// entries), and publishes finished gate/up tiles: the fence before a
// publication takes a microsecond that the epilogue does not wait for.
template <int AR>
__device__ void scheduler(Ctl *ctl, const ProductArgs &a) {
    const int lane = threadIdx.x & 31;
    const int nbt0 = column_tiles(a.phase[0]), t0 = ctl->m_tiles * nbt0;
    const int nbt1 = a.phases > 1 ? column_tiles(a.phase[1]) : 0, total = t0 + ctl->m_tiles * nbt1;
    unsigned claimed = 0, published = 0, to_publish = 0;
    bool open = true, waited = false;
    unsigned long long since = cycles();
    while (open || published < to_publish) {
        bool idle = true;
        const int s = claimed % TILES;
        bool slot = false;
        if (open && to_publish - published < PUBS) slot = __all_sync(ALL, claimed < TILES || bar_test(&ctl->tile_free[s], (claimed / TILES - 1) & 1));
        if (slot) {
            int t = 0;
            if (lane == 0) t = atomicAdd(a.next_tile, 1);
            t = __shfl_sync(ALL, t, 0);
            Tile x;
            x.phase = TILE_END;
            x.n = x.ready = 0;
            if (t < 0) {  // a workspace that was not zero-filled
                if (lane == 0) atomicCAS(a.error, 0, DEV_BAD_LISTS);
            } else if (t < t0) x = tile_at<AR>(t, 0, nbt0, ctl);
            else if (t < total) x = tile_at<AR>(t - t0, 1, nbt1, ctl);
            int tok[4];
            if (x.phase != TILE_END) {
                const bool by_pair = a.phase[x.phase].by_pair != 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    // rows past the tile's end repeat its last one (their sums are not used)
                    const int p = x.p0 + min(lane + 32 * q, x.n - 1);
                    int r = p;
                    if (!by_pair || x.phase == 0) {
                        tok[q] = __ldg(a.tok + p);
                        if (tok[q] < 0 || tok[q] >= a.B) {
                            atomicCAS(a.error, 0, DEV_BAD_LISTS);
                            tok[q] = -1;
                        }
                        if (!by_pair) r = max(tok[q], 0);
                    }
                    ctl->rows[s][lane + 32 * q] = r;
                }
                if (x.phase == 1) {
                    if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");  // the counts are zero
                    waited = true;
                    x.ready = ld_acquire(a.done + x.mt) >= nbt0;
                }
            }
            if (lane == 0) ctl->tile[s] = x;
            __syncwarp();
            if (lane == 0) bar_arrive(&ctl->tile_full[s]);
            ++claimed;
            open = x.phase != TILE_END;
            if (a.phases > 1 && x.phase == 0) {
                ++to_publish;
                if (x.nb == 0) {  // the entries of each token, for the combine
                    if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
                    waited = true;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int p = x.p0 + lane + 32 * q;
                        if (lane + 32 * q >= x.n || tok[q] < 0) continue;
                        const int c = atomicAdd(a.cnt + tok[q], 1);
                        if (c < a.k) a.inv[static_cast<size_t>(tok[q]) * a.k + c] = p;
                        else atomicCAS(a.error, 0, DEV_BAD_LISTS);
                    }
                }
            }
            idle = false;
        }
        if (published < to_publish && __all_sync(ALL, bar_test(&ctl->pub_full[published % PUBS], (published / PUBS) & 1))) {
            if (lane == 0) {
                const int mt = ctl->pub_mt[published % PUBS];
                // h and its scales, written by the epilogue's threads, are in
                // memory for the copies of any CTA before the tile counts
                fence_async();
                __threadfence();
                add_release(a.done + mt);
            }
            __syncwarp();
            ++published;
            idle = false;
        }
        if (!idle) since = cycles();
        else if (__any_sync(ALL, ctl->abort_flag || cycles() - since > a.wait_ns * CYCLES_PER_NS)) {
            if (lane == 0 && !ctl->abort_flag) {
                atomicCAS(a.error, 0, DEV_TIMEOUT_EMPTY);
                ctl->abort_flag = 1;
            }
            return;
        }
    }
}

// Lets the copies in flight land before the CTA leaves: after a wait that ran
// out, one of the two copying roles may have filled stages that the other has
// not; its arrival is made up for.
template <int STAGES>
__device__ void drain_fills(Ctl *ctl) {
    const unsigned w = ctl->fills[0], r = ctl->fills[1], lo = min(w, r), hi = max(w, r);
    for (unsigned i = lo; i < hi; ++i) bar_arrive(&ctl->full[i % STAGES]);
    const unsigned long long t0 = cycles();
    for (unsigned i = hi > STAGES ? hi - STAGES : 0; i < hi; ++i)
        while (!bar_try(&ctl->full[i % STAGES], (i / STAGES) & 1) && cycles() - t0 < DRAIN_CYCLES) {
        }
}

template <int AR>
__device__ unsigned weights_role(unsigned char *ring, Ctl *ctl, const ProductMaps &maps, const ProductArgs &a) {
    using R = Ring<AR>;
    TileCursor cur;
    Tile x;
    unsigned it = 0;
    while (cur.next(ctl, a, x)) {
        cur.release(ctl);
        if (x.phase == TILE_END) return it;
        const ProductPhase &ph = a.phase[x.phase];
        const int kb = (ph.K + BLK - 1) / BLK;
        const int r0 = ph.kind == PRODUCT_SWIGLU ? x.nb * BLK : x.nb * TILE_N;
        const int r1 = ph.kind == PRODUCT_SWIGLU ? r0 : r0 + BLK;
        const CUtensorMap *m0 = &maps.phase[x.phase].b0, *m1 = &maps.phase[x.phase].b1;
        for (int j = 0; j < kb; ++j, ++it) {
            const int st = it % R::STAGES;
            unsigned char *w = ring + st * R::STAGE;
            if (it >= R::STAGES && !wait_bar(&ctl->empty[st], (it / R::STAGES - 1) & 1, ctl, a, DEV_TIMEOUT_EMPTY))
                return it;
            bar_expect(&ctl->full[st], W_STAGE);
            load_box(w, m0, j * BLK, r0, x.e, &ctl->full[st]);
            load_box(w + W_STAGE / 2, m1, j * BLK, r1, x.e, &ctl->full[st]);
        }
    }
    return it;
}

template <int AR>
__device__ unsigned rows_role(unsigned char *ring, Ctl *ctl, const ProductMaps &maps, const ProductArgs &a) {
    using R = Ring<AR>;
    const int lane = threadIdx.x & 31;
    TileCursor cur;
    Tile x;
    unsigned it = 0, sg = 0;
    int st = 0;
    unsigned phase = 0;  // of stage st's present fill
    // the activations are the previous kernel's
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (;;) {
        if (!__all_sync(ALL, cur.next(ctl, a, x))) return it;
        int rows[4], srow[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            rows[q] = ctl->rows[cur.i % TILES][lane * 4 + q];
            srow[q] = ctl->rows[cur.i % TILES][lane + 32 * q];
        }
        __syncwarp();
        if (lane == 0) cur.release(ctl);
        else ++cur.i;
        if (x.phase == TILE_END) return it;
        const ProductPhase &ph = a.phase[x.phase];
        const int kb = (ph.K + BLK - 1) / BLK, rb = (ph.rows + BLK - 1) / BLK;
        if (x.phase == 1) {
            // the entries' gate/up tiles are all done
            bool ok = true;
            if (lane == 0 && !x.ready) {
                const int need = column_tiles(a.phase[0]);
                const unsigned long long t0 = cycles();
                while (ok && ld_acquire(a.done + x.mt) < need) {
                    ok = !ctl->abort_flag;
                    if (ok && cycles() - t0 > a.wait_ns * CYCLES_PER_NS) {
                        atomicCAS(a.error, 0, DEV_TIMEOUT_DEP);
                        ctl->abort_flag = 1;
                        ok = false;
                    }
                }
            }
            if (!__all_sync(ALL, ok)) return it;
            fence_async();
        }
        // lane l copies the scales of rows l, l + 32, ..., and gathers rows 4 l ..
        const float *src[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) src[q] = ph.as + srow[q] * static_cast<size_t>(ph.as_pitch);
        // lanes 0-3 and 4-7: a group's scales of the two weight blocks
        const int nb = ph.kind == PRODUCT_SWIGLU ? x.nb : min(2 * x.nb + (lane >> 2), rb - 1);
        const float *wsrc = (lane < 4 ? ph.bs0 : ph.bs1) + (static_cast<size_t>(x.e) * rb + nb) * kb;
        const bool wide = (ph.as_pitch & 3) == 0;
        // consecutive rows in boxes, scattered ones four at a time
        const int first = __shfl_sync(ALL, rows[0], 0);
        bool run = true;
#pragma unroll
        for (int q = 0; q < 4; ++q) run = run && rows[q] == first + min(lane * 4 + q, x.n - 1);
        const bool box = __all_sync(ALL, run);
        const int copies = box ? (x.n + R::BOX - 1) / R::BOX : (x.n + 3) >> 2;
        const unsigned copy_bytes = box ? R::BOX * BLK : 4 * BLK, bytes = copies * copy_bytes;
        const CUtensorMap *m = box ? &maps.phase[x.phase].ab : &maps.phase[x.phase].a;
        for (int j = 0; j < kb; ++j) {
            if (j % SGROUP == 0) {
                const unsigned sc = sg % SCALES;
                if (sg >= SCALES && !__all_sync(ALL, wait_bar(&ctl->scale_free[sc], (sg / SCALES - 1) & 1, ctl, a, DEV_TIMEOUT_EMPTY)))
                    return it;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int r = lane + 32 * q;
                    if (r >= x.n) break;
                    if (wide) copy16(&ctl->scale[sc][r], src[q] + j);
                    else
                        for (int i = 0; i < SGROUP && j + i < kb; ++i)
                            copy4(reinterpret_cast<float *>(&ctl->scale[sc][r]) + i, src[q] + j + i);
                }
                if (lane < 8 && j + (lane & 3) < kb) copy4(&ctl->wscale[sc][lane >> 2][lane & 3], wsrc + j + (lane & 3));
                copies_arrive(&ctl->scale_full[sc]);
                ++sg;
            }
            unsigned long long *full = &ctl->full[st];
            if (it >= R::STAGES && !__all_sync(ALL, wait_bar(&ctl->empty[st], phase ^ 1, ctl, a, DEV_TIMEOUT_EMPTY))) return it;
            if (lane == 0) bar_expect(full, bytes);
            __syncwarp();
            if (lane < copies) {
                unsigned char *d = ring + st * R::STAGE + W_STAGE + lane * copy_bytes;
                if (box) load_rows(d, m, j * BLK, first + lane * R::BOX, full);
                else load_rows4(d, m, j * BLK, rows, full);
            }
            ++it;
            if (++st == R::STAGES) {
                st = 0;
                phase ^= 1;
            }
        }
    }
}

template <int AR>
__device__ void issue_role(unsigned char *ring, Ctl *ctl, const ProductArgs &a) {
    using R = Ring<AR>;
    const uint32_t tmem = ctl->tmem;
    TileCursor cur;
    Tile x;
    unsigned it = 0;
    while (cur.next(ctl, a, x)) {
        cur.release(ctl);
        if (x.phase == TILE_END) return;
        const int kb = (a.phase[x.phase].K + BLK - 1) / BLK;
        for (int j = 0; j < kb; ++j, ++it) {
            const int st = it % R::STAGES, buf = it % R::BUFS;
            if (it >= R::BUFS && !wait_bar(&ctl->part_free[buf], (it / R::BUFS - 1) & 1, ctl, a, DEV_TIMEOUT_DEP)) return;
            if (!wait_bar(&ctl->full[st], (it / R::STAGES) & 1, ctl, a, DEV_TIMEOUT_FULL)) return;
            tc_fence_after();
            const uint64_t w = umma_desc(saddr(ring + st * R::STAGE));
            const uint64_t v = umma_desc(saddr(ring + st * R::STAGE + W_STAGE));
            const uint32_t d = tmem + buf * R::BUF_COLS;
            if constexpr (R::FEW) {
                const uint64_t w1 = umma_desc(saddr(ring + st * R::STAGE + W_STAGE / 2));
                constexpr int N = TILE_FEW;
#pragma unroll
                for (int s = 0; s < 4; ++s) {  // 32 columns = 32 bytes each
                    umma_e4m3(d, w + 2 * s, v + 2 * s, idesc_e4m3(N), s > 0);
                    umma_e4m3(d + TILE_FEW, w1 + 2 * s, v + 2 * s, idesc_e4m3(N), s > 0);
                }
            } else {
#pragma unroll
                for (int s = 0; s < 4; ++s) umma_e4m3(d, v + 2 * s, w + 2 * s, idesc_e4m3(TILE_N), s > 0);
            }
            umma_commit(saddr(&ctl->empty[st]));
            umma_commit(saddr(&ctl->part_full[buf]));
        }
    }
}

__device__ __forceinline__ void epi_bar() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
// all epilogue threads meet; true if any of them says so
__device__ __forceinline__ bool epi_any(bool v) {
    unsigned r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 2, 256, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<unsigned>(v))
        : "memory");
    return r != 0;
}

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

// c[0 .. 32) += v * m
__device__ __forceinline__ void add32(float *c, const uint32_t (&v)[32], float m) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) fma2(c[i], c[i + 1], v[i], v[i + 1], m);
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

// 64 output columns n0 .. of the warp's rows
__device__ __forceinline__ void store_out(unsigned char *stage, const float (&c)[64], const ProductPhase &ph, size_t row0,
                                          int n0, int rows_here, int lane) {
    uint4 o[4];
    unsigned *w = reinterpret_cast<unsigned *>(o);
    const size_t at = row0 * ph.rows + n0;
    if (ph.out_bf16) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = pack_bf16(c[q * 32 + 2 * i], c[q * 32 + 2 * i + 1]);
            store_chunk(stage, o, static_cast<char *>(ph.out) + (at + q * 32) * 2, static_cast<size_t>(ph.rows) * 2,
                        rows_here, lane, (ph.rows - n0 - q * 32) * 2);
        }
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(c[q * 16 + i]);
            store_chunk(stage, o, static_cast<char *>(ph.out) + (at + q * 16) * 4, static_cast<size_t>(ph.rows) * 4,
                        rows_here, lane, (ph.rows - n0 - q * 16) * 4);
        }
    }
}

// The n-th finished gate/up tile, for the warp that publishes: all epilogue
// warps, after their stores.  (A slot comes round again only once the tile
// that had it is published: no more are claimed before.)
__device__ __forceinline__ void hand_over(Ctl *ctl, unsigned n, int mt) {
    if (threadIdx.x == 0) ctl->pub_mt[n % PUBS] = mt;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) bar_arrive(&ctl->pub_full[n % PUBS]);
}

__device__ __forceinline__ int scale_exponent(float top) {
    const unsigned tb = __float_as_uint(top);
    const int e = tb == 0u ? 0 : static_cast<int>(tb >> 23) - 135 + ((tb & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e < -120 ? -120 : e;
}
// silu(g) u, NaN where it is not finite: e4m3 has no infinity, and cvt would
// make one the largest finite value.  The fast exp and division are good to a
// few units of fp32, and h is about to be rounded to 4 bits; the exact ones
// leave y no nearer to a plain fp32 computation (24 random cases, fp32 y:
// 1.3e-5 from 64 bits with these, 1.0e-5 with the exact ones, 5.8e-5 the plain
// form) and cost 26 us of 111 (333 tokens) and 28 of 445 (4096 tokens).
__device__ __forceinline__ float swiglu(float g, float u) {
    const float h = __fdividef(g, 1.0f + __expf(-g)) * u;
    return fmaf(h, 0.0f, h);
}

// Few entries: thread (weight row, entry half) holds the row of both
// matrices for up to 8 entries.
__device__ __forceinline__ void epilogue_few(unsigned char *out_stage, Ctl *ctl, const ProductArgs &a) {
    using R = Ring<TILE_FEW>;
    constexpr int HALF = TILE_FEW / 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quarter = warp & 3, half = warp >> 2;
    const int m = quarter * 32 + lane;  // row of either matrix
    bool dead = false;
    unsigned it = 0, gu = 0, sg = 0;
    TileCursor cur;
    Tile x;
    for (;;) {
        dead = dead || !cur.next(ctl, a, x);
        if (epi_any(dead)) return;  // together, so that none is left at a barrier
        __syncwarp();
        if (lane == 0) cur.release(ctl);
        else ++cur.i;
        if (x.phase == TILE_END) return;
        const ProductPhase &ph = a.phase[x.phase];
        const int kb = (ph.K + BLK - 1) / BLK;
        const int first = half * HALF, n = min(HALF, x.n - first);  // the warp's entries (n <= 0: none)
        const uint32_t tbase = ctl->tmem + (static_cast<uint32_t>(quarter * 32) << 16) + first;
        float c0[HALF], c1[HALF];
#pragma unroll
        for (int i = 0; i < HALF; ++i) c0[i] = c1[i] = 0.0f;
        for (int j = 0; j < kb; ++j, ++it) {
            const int buf = it % R::BUFS, sc = sg % SCALES;
            bool ok = !dead;
            if (j % SGROUP == 0) ok = ok && wait_bar(&ctl->scale_full[sc], (sg / SCALES) & 1, ctl, a, DEV_TIMEOUT_FULL);
            ok = ok && wait_bar(&ctl->part_full[buf], (it / R::BUFS) & 1, ctl, a, DEV_TIMEOUT_FULL);
            dead = !__all_sync(ALL, ok);
            const bool last = j % SGROUP == SGROUP - 1 || j + 1 == kb;  // of the group
            sg += last;
            if (dead) continue;
            tc_fence_after();
            const float w0 = ctl->wscale[sc][0][j % SGROUP], w1 = ctl->wscale[sc][1][j % SGROUP];
            const float *as = reinterpret_cast<const float *>(&ctl->scale[sc][first]) + j % SGROUP;
            if (n > 0) {
                float u[HALF], v[HALF];
                tmem_ld8x2(tbase + buf * R::BUF_COLS, tbase + buf * R::BUF_COLS + TILE_FEW, u, v);
#pragma unroll
                for (int i = 0; i < HALF; ++i) {
                    const float f = as[i * SGROUP];
                    c0[i] = fmaf(u[i], f * w0, c0[i]);
                    c1[i] = fmaf(v[i], f * w1, c1[i]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                bar_arrive(&ctl->part_free[buf]);
                if (last) bar_arrive(&ctl->scale_free[sc]);
            }
        }
        if (ph.kind == PRODUCT_SWIGLU) {
#pragma unroll
            for (int i = 0; i < HALF; ++i) {
                if (i < n) {  // the same for the whole warp
                    c0[i] = swiglu(c0[i], c1[i]);
                    const unsigned t = __reduce_max_sync(ALL, __float_as_uint(fmaxf(0.0f, fabsf(c0[i]))));  // (of NaN: 0)
                    if (lane == 0) ctl->top[quarter][first + i] = __uint_as_float(t);
                }
            }
            epi_bar();
#pragma unroll
            for (int i = 0; i < HALF; ++i) {
                if (i < n) {
                    const int c = first + i;
                    const int e = scale_exponent(fmaxf(fmaxf(ctl->top[0][c], ctl->top[1][c]), fmaxf(ctl->top[2][c], ctl->top[3][c])));
                    out_stage[c * BLK + m] =
                        static_cast<unsigned char>(pack_e4m3(c0[i] * __int_as_float((127 - e) << 23), 0.f, 0.f, 0.f));
                    if (m == 0 && !dead)
                        ph.hs[static_cast<size_t>(x.p0 + c) * ph.hs_pitch + x.nb] = __int_as_float((127 + e) << 23);
                }
            }
            epi_bar();
            const int f0 = x.nb * BLK;
            for (int i = threadIdx.x; i < x.n * 8 && !dead; i += 32 * EPI_WARPS) {
                const int c = i >> 3, f = (i & 7) * 16;
                if (f0 + f < ph.rows)
                    *reinterpret_cast<uint4 *>(ph.hq + static_cast<size_t>(x.p0 + c) * ph.rows + f0 + f) =
                        *reinterpret_cast<const uint4 *>(out_stage + c * BLK + f);
            }
            if (a.phases > 1 && !dead) hand_over(ctl, gu++, x.mt);
        } else if (!dead) {
            // a warp's lanes are neighbours in the output row: whole lines
            const int r0 = x.nb * TILE_N + m;
            const bool in0 = r0 < ph.rows, in1 = r0 + BLK < ph.rows;
            const size_t at = static_cast<size_t>(x.p0 + first) * ph.rows + r0;
#pragma unroll
            for (int i = 0; i < HALF; ++i) {
                if (i < n) {
                    const size_t o = at + static_cast<size_t>(i) * ph.rows;
                    if (ph.out_bf16) {
                        __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(ph.out);
                        if (in0) y[o] = __float2bfloat16_rn(c0[i]);
                        if (in1) y[o + BLK] = __float2bfloat16_rn(c1[i]);
                    } else {
                        float *y = static_cast<float *>(ph.out);
                        if (in0) y[o] = c0[i];
                        if (in1) y[o + BLK] = c1[i];
                    }
                }
            }
        }
    }
}

// Many entries: thread (entry, column half).
__device__ __forceinline__ void epilogue_many(unsigned char *out_stage, Ctl *ctl, const ProductArgs &a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quarter = warp & 3, half = warp >> 2;  // TMEM lanes 32 quarter .., columns 64 half .. of each matrix
    const int row = quarter * 32 + lane;
    const uint32_t tbase = ctl->tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * 64;
    unsigned char *stage = out_stage + warp * OUT_STAGE;
    bool dead = false;
    unsigned it = 0, sg = 0;
    if (lane == 0) ctl->handed[warp] = 0;
    TileCursor cur;
    Tile x;
    for (;;) {
        dead = dead || !cur.next(ctl, a, x);
        if (epi_any(dead)) return;  // together, so that none is left at a barrier
        __syncwarp();
        if (lane == 0) cur.release(ctl);
        else ++cur.i;
        if (x.phase == TILE_END) return;
        const int kb = (a.phase[x.phase].K + BLK - 1) / BLK;
        const bool live = quarter * 32 < x.n;  // the warp holds rows of the tile
        if (lane == 0) ctl->own[warp] = x;
        __syncwarp();
        float c0[64], c1[64];
#pragma unroll
        for (int i = 0; i < 64; ++i) c0[i] = c1[i] = 0.0f;
        for (int j = 0; j < kb; ++j, ++it) {
            const int buf = it & 1, sc = sg % SCALES;
            bool ok = !dead;
            if (j % SGROUP == 0) ok = ok && wait_bar(&ctl->scale_full[sc], (sg / SCALES) & 1, ctl, a, DEV_TIMEOUT_FULL);
            ok = ok && wait_bar(&ctl->part_full[buf], (it >> 1) & 1, ctl, a, DEV_TIMEOUT_FULL);
            dead = !__all_sync(ALL, ok);
            const bool last = j % SGROUP == SGROUP - 1 || j + 1 == kb;  // of the group
            sg += last;
            if (dead) continue;
            tc_fence_after();
            if (live) {
                const uint32_t col = tbase + buf * TILE_N;
                // a load is in flight while the one before is added; the
                // buffer goes back to the MMAs before the last additions
                uint32_t u[32], v[32];
                tmem_ld32(col, u);
                const float f = reinterpret_cast<const float *>(&ctl->scale[sc][row])[j % SGROUP];
                const float m0 = f * ctl->wscale[sc][0][j % SGROUP], m1 = f * ctl->wscale[sc][1][j % SGROUP];
                tmem_wait(u);
                tmem_ld32(col + 32, v);
                add32(c0, u, m0);
                tmem_wait(v);
                tmem_ld32(col + 128, u);
                add32(c0 + 32, v, m0);
                tmem_wait(u);
                tmem_ld32(col + 160, v);
                add32(c1, u, m1);
                tmem_wait(v);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(&ctl->part_free[buf]);
                    if (last) bar_arrive(&ctl->scale_free[sc]);
                }
                add32(c1 + 32, v, m1);
            } else {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(&ctl->part_free[buf]);
                    if (last) bar_arrive(&ctl->scale_free[sc]);
                }
            }
        }
        const volatile Tile *own = &ctl->own[warp];
        x.phase = own->phase;
        x.p0 = own->p0;
        x.n = own->n;
        x.nb = own->nb;
        const ProductPhase &ph = a.phase[x.phase];
        const int rows_here = min(32, x.n - quarter * 32);
        const size_t row0 = static_cast<size_t>(x.p0 + quarter * 32);
        if (ph.kind == PRODUCT_SWIGLU) {
            float top = 0.0f;
            if (live) {
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    c0[i] = swiglu(c0[i], c1[i]);
                    top = fmaxf(top, fabsf(c0[i]));
                }
            }
            // (read again only after the next tile's meeting)
            ctl->top[half][row] = top;
            epi_bar();
            if (live && !dead) {
                top = fmaxf(ctl->top[0][row], ctl->top[1][row]);
                const int e = scale_exponent(top);
                const float inv = __int_as_float((127 - e) << 23);
                uint4 o[4];
                unsigned *w = reinterpret_cast<unsigned *>(o);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    w[i] = pack_e4m3(c0[4 * i] * inv, c0[4 * i + 1] * inv, c0[4 * i + 2] * inv, c0[4 * i + 3] * inv);
                const int f = x.nb * BLK + half * 64;
                store_chunk(stage, o, reinterpret_cast<char *>(ph.hq) + row0 * ph.rows + f, ph.rows, rows_here, lane,
                            ph.rows - f);
                if (row < x.n && half == 0)
                    ph.hs[static_cast<size_t>(x.p0 + row) * ph.hs_pitch + x.nb] = __int_as_float((127 + e) << 23);
            }
            if (!dead) {
                const unsigned n = const_cast<volatile unsigned *>(ctl->handed)[warp];
                __syncwarp();
                if (lane == 0) ctl->handed[warp] = n + 1;
                hand_over(ctl, n, own->mt);
            }
        } else if (live && !dead) {
            const int n0 = x.nb * TILE_N + half * 64;
            store_out(stage, c0, ph, row0, n0, rows_here, lane);
            store_out(stage, c1, ph, row0, n0 + BLK, rows_here, lane);
        }
    }
}

template <int AR>
__global__ void __launch_bounds__(THREADS, 1) product_kernel(const __grid_constant__ ProductMaps maps,
                                                             const __grid_constant__ ProductArgs a) {
    using R = Ring<AR>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *ring =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char *out_stage = ring + R::STAGES * R::STAGE;
    Ctl *ctl = reinterpret_cast<Ctl *>(out_stage + R::OUT_BYTES);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < R::STAGES; ++i) {
            bar_init(&ctl->full[i], 2);  // weights and rows
            bar_init(&ctl->empty[i], 1);
        }
        for (int i = 0; i < R::BUFS; ++i) {
            bar_init(&ctl->part_full[i], 1);
            bar_init(&ctl->part_free[i], EPI_WARPS);
        }
        for (int i = 0; i < SCALES; ++i) {
            bar_init(&ctl->scale_full[i], 32);
            bar_init(&ctl->scale_free[i], EPI_WARPS);
        }
        for (int i = 0; i < TILES; ++i) {
            bar_init(&ctl->tile_full[i], 1);
            bar_init(&ctl->tile_free[i], EPI_WARPS + 3);
        }
        for (int i = 0; i < PUBS; ++i) bar_init(&ctl->pub_full[i], EPI_WARPS);
        bar_init(&ctl->mma_done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        ctl->abort_flag = 0;
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == EPI_WARPS + 1) tmem_alloc(saddr(&ctl->tmem), 512);
    tc_fence_before();
    build_slots<AR>(ctl, a);  // ends in a block barrier
    tc_fence_after();
    if (warp < EPI_WARPS) {
        if constexpr (!R::FEW) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_EPI));
        if constexpr (R::FEW) epilogue_few(out_stage, ctl, a);
        else epilogue_many(out_stage, ctl, a);
    } else {
        if constexpr (!R::FEW) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_COPY));
        if (warp == EPI_WARPS) {
            if (elect_one()) ctl->fills[0] = weights_role<AR>(ring, ctl, maps, a);
        } else if (warp == EPI_WARPS + 1) {
            if (elect_one()) {
                issue_role<AR>(ring, ctl, a);
                umma_commit(saddr(&ctl->mma_done));
                const unsigned long long t0 = cycles();
                while (!bar_try(&ctl->mma_done, 0) && cycles() - t0 < DRAIN_CYCLES) {
                }
            }
        } else if (warp == EPI_WARPS + 2) {
            const unsigned n = rows_role<AR>(ring, ctl, maps, a);
            if ((threadIdx.x & 31) == 0) ctl->fills[1] = n;
            asm volatile("cp.async.wait_all;" ::: "memory");
        } else {
            scheduler<AR>(ctl, a);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == EPI_WARPS + 1) tmem_dealloc(ctl->tmem, 512);
    if (threadIdx.x == 0) {
        drain_fills<R::STAGES>(ctl);
        __threadfence();
        if (atomicAdd(a.exits, 1) == static_cast<int>(gridDim.x) - 1) {
            *a.next_tile = 0;
            *a.exits = 0;
        }
    }
}

template <int AR>
cudaError_t launch_ar(const ProductMaps &maps, const ProductArgs &a, cudaStream_t s) {
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
        err = cudaFuncSetAttribute(product_kernel<AR>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<AR>());
        if (err != cudaSuccess) return err;
        if (!Ring<AR>::FEW) {  // setmaxnreg.inc would wait for ever for more registers than the launch has
            cudaFuncAttributes at;
            err = cudaFuncGetAttributes(&at, product_kernel<AR>);
            if (err != cudaSuccess) return err;
            if (at.numRegs * THREADS < 256 * REGS_EPI + 128 * REGS_COPY) return cudaErrorInvalidConfiguration;
        }
        sms[dev] = n;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sms[dev]);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem_bytes<AR>();
    cfg.stream = s;
    // after the quantisation kernel: claim tiles and stream weights meanwhile
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.phases > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, product_kernel<AR>, maps, a);
}

}  // namespace

int product_tile_entries(const moe_dims_t &d) {
    const long long pairs = static_cast<long long>(d.B) * d.k, experts = d.E < pairs ? d.E : pairs;
    return d.B <= 2 * TILE_FEW || pairs <= FEW_AVERAGE * experts ? TILE_FEW : TILE_MANY;
}
// Large tiles take their rows from copies in list order; small ones gather
// them by token, four at a time.
bool product_dispatch(const moe_dims_t &d) { return product_tile_entries(d) == TILE_MANY; }
int product_box_rows(const moe_dims_t &d) {
    const int n = product_tile_entries(d);
    return n < BOX_ROWS ? n : BOX_ROWS;
}

cudaError_t launch_product(const ProductMaps &maps, const ProductArgs &a, cudaStream_t s) {
    return a.tile_entries == TILE_FEW ? launch_ar<TILE_FEW>(maps, a, s) : launch_ar<TILE_MANY>(maps, a, s);
}

}  // namespace moe

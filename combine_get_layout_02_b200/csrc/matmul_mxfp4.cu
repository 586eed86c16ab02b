// The experts' product on MXFP4 rows: y[r, :] = A[r, :] W[e(r), :, :]^T, sums in
// binary32, BF16 out (format in mxfp4.cuh).
//
// Tensor cores: tcgen05.mma kind::mxf4 with block scales (32 values a scale,
// 64 values an instruction), cta_group::2: a pair of blocks on neighbouring SMs
// works on one tile of 256 output features.  The weights are the M side, 128
// features in each block; the tokens are the N side, half of the tile's rows in
// each block's shared memory, whose width goes by the expert's rows, 16 at a
// time: few rows cost few columns, and each weight tile is read once for up to
// `nt` rows.  Persistent pairs walk the list of (expert, rows, features) tiles;
// each block makes the list's prefix sums from expert_offset for itself.
// One block:
//   warp 0, 9   TMA: a ring of stages of 256 values (128 bytes) a row, 128-byte
//               swizzle; 0 the weights, 9 the tokens
//   warp 1, 10  in the pair's first block, for both: 1 issues the MMAs, 4 a stage,
//               10 the copies of the scales from shared memory to TMEM (tcgen05.cp)
//   warps 2, 11 the weights' scales (11: see the launcher), 3 and 8 the tokens':
//               global rows -> the 512-byte blocks that tcgen05.cp wants (row r's word
//               at (r % 32) * 16 + (r / 32) * 4)
//   warps 4-7   TMEM -> registers -> transposed through shared memory -> BF16 rows,
//               while the next tile's MMAs run
// Why pairs: one block alone (128 x 208) moves 45 KB a stage into shared memory and
// reads them out again in 700 cycles of its 128 bytes a cycle, where the MMAs need
// 416; a pair holds half the tokens' rows each (131072 x 2048 -> 7168 over 256
// experts: 2.37 ms with single blocks, 1.26 ms with pairs at that step).
// Scales stay in their rows in memory, [rows, in / 32], because a tile starts at
// any row of the receive buffer; a warp reads 32 bytes of each row, four stages'
// worth, one such chunk ahead.
// Where tiles are few (see the launcher), two or four pairs share one, a part of K
// each, and join their sums in order through distributed shared memory.
//
// What bounds it (B200; floors at the measured 6.53 TB/s copy and four times the
// measured bf16 rate; short runs of a few ms, over several cards): few rows an
// expert, the weights' bytes: 4 rows, 7168 -> 4096, 256 experts 611 to 625 us
// against 602; 128 rows 667 to 695 against 672, and 757 to 873 when run for
// seconds, where the 1000 W cap takes the clock to 1.0 GHz.  Many rows: no single
// unit.  512 rows an expert, 2048 -> 7168: 0.99 to 1.05 ms (1.15 to 1.25 in a long
// run) against 615 us; the tensor pipe is active half of the time, the SMs take 45
// bytes a cycle from L2 of the 64 they could, DRAM is at 45%.  In long runs the
// MMAs without loads took 0.82 ms, with all weights in L2 1.05, and more columns a
// tile, which take fewer bytes, less (160, 192, 208: 1.35, 1.23, 1.16 ms); two
// accumulators and the scales fill TMEM at 208.  One row, 7168 -> 4096: 12 us;
// with 1024 values it is 7, the launch, the tables, the first loads and the stores.
//
// Every wait is bounded (about a second, then CGL_ETIMEOUT): the pair's roles leave
// their loops, MMAs in flight are waited for, copies and arrivals under way get
// 0.15 s to land before either block leaves, TMEM is freed.
#include <cuda.h>

#include "mxfp4.cuh"
#include "launch.h"

namespace cgl {

namespace {

constexpr uint32_t kErrTimeout = 1u << CGL_ETIMEOUT;
constexpr long long kWaitCycles = 1ll << 31;
constexpr long long kLandCycles = 1ll << 28;
constexpr int kThreads = 384;
constexpr int kStageK = 256;              // values a stage
constexpr int kChunk = 4;                 // stages a chunk of scales (1024 values, 32 bytes a row)
constexpr int kM = 128;                   // features a tile
constexpr int kMaxStages = 12;
constexpr int kMaxNt = 208;               // 2 accumulators of 208 columns + 4 stages' scales = 512 columns
constexpr int kOutBytes = 4 * 2048;       // the epilogue's 32 x 32 BF16 blocks, one a warp
constexpr size_t kSmemLimit = 226 * 1024; // dynamic part: 227 KiB less the static part
constexpr uint32_t kABytes = kM * kStageK / 2;
constexpr uint32_t kChunkA = kChunk * 1024;   // bytes of a chunk of the weights' scales, 512 for 128 rows x 4

struct Params {
    const uint8_t *sa, *sw;
    const int32_t *off;
    uint16_t *y;
    uint32_t *status;
    int64_t rows, cap;
    int E, F, K;
    int nt;          // most token columns a tile (of the pair)
    int nb;          // 128-row scale blocks of the token side (1 or 2)
    int box;         // token rows a TMA box
    int stages;
    int chunks;      // chunks of scales in shared memory
    int sfwarps;     // warps for the weights' scales (1 or 2)
    int split;       // pairs that share a tile, each a part of K (one cluster)
    int wide;        // y's rows allow 16-byte stores
    int aligned;     // every scale row starts at a 16-byte boundary
    uint32_t stage_bytes, chunk_bytes;
    long long wait_cycles;   // a wait's limit: kWaitCycles, less in the self-test
};

// ---- barriers, TMA, tcgen05 ----------------------------------------------------------------

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\n"
        "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n"
        "selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// Half of what a barrier counts is done by the pair's other block (arrivals,
// copies' bytes, commits), so every wait has cluster scope; this fence after it
// makes what the others wrote to shared memory before they arrived theirs to read.
// It is restricted to shared memory, as is its counterpart in bar_arrive_smem: an
// acquire or release of all memory at that scope holds a warp until its loads in
// flight are there (4 rows an expert, 7168 -> 4096: 910 us with those, 620 with
// these; 128 rows 909 and 689; 512 rows, 2048 -> 7168: 1256 and 1037).
__device__ __forceinline__ void fence_acquire_smem() {
    asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// The same shared-memory address in another block of the cluster.
__device__ __forceinline__ uint32_t in_block(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Arrive at a barrier of the pair's first block, from either block.  _tmem hands
// back TMEM that tcgen05.ld has read: execution order is all that needs, with
// tcgen05's fences on both sides.  _smem announces what this warp wrote to its
// own shared memory (after a proxy fence), which the tensor core reads on behalf
// of a thread of the first block.
__device__ __forceinline__ void bar_arrive_tmem(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_arrive_smem(uint32_t bar) {
    asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Whether a phase has ended, without waiting (where it has, fence_acquire_smem is still to come).
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\n"
        "mbarrier.test_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n"
        "selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Tells both blocks of the pair that a wait has run out: a word in each one's shared memory.
__device__ __forceinline__ void give_up(volatile int *abort, uint32_t *status) {
    const uint32_t word = smem_u32(const_cast<const int *>(abort));
    *abort = 1;
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(in_block(word, cluster_rank() ^ 1)), "r"(1) : "memory");
    report(status, kErrTimeout);
}

// Bounded wait for a phase; false once this wait or another of the pair has given up.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int *abort, const Params &p) {
    if (!bar_try(bar, parity)) {
        const long long start = clock64();
        while (!bar_try(bar, parity)) {
            if (*abort) return false;
            if (clock64() - start > p.wait_cycles) {
                give_up(abort, p.status);
                return false;
            }
        }
    }
    fence_acquire_smem();
    return true;
}

// One lane of a converged warp, always the same.  Copies and MMAs issued by the
// elected lane took 300 cycles a stage, inside `if (lane == 0)` 1300.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xFFFFFFFF;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}

// Tile loads into this block; the barrier may be the first block's.
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// Shared-memory descriptors: rows of 128 bytes in the 128-byte swizzle (groups
// of eight rows 1024 bytes apart), and the unswizzled 32 x 16-byte block of
// scales (groups of eight rows 128 bytes apart).
__device__ __forceinline__ uint64_t desc_rows(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_scales(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (8ull << 32) | (1ull << 46);
}

// Instruction descriptor: E2M1 x E2M1, UE8M0 scales, M = 256, N columns, the
// scale bytes `id` and id + 1 of each word.
__device__ __forceinline__ uint32_t instr_desc(int n, uint32_t id) {
    return (id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | (1u << 28) | (id << 29);
}

__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.u32 p, %6, 0;\n"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void scales_to_tmem(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// Arrive, once this thread's MMAs and copies so far have ended, at a barrier of both blocks or of this one.
__device__ __forceinline__ void mma_commit_both(uint32_t bar, uint32_t lead) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"((uint16_t)(3u << lead))
                 : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 16 lanes x 32 columns: of each eight columns, r[0], r[1] are row lane / 4 and
// columns 2 (lane % 4) and the next, r[2], r[3] the same of row lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t r[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Four 8 x 8 blocks of 16-bit values, transposed: lane i gives the address of row i % 8 of block i / 8.
__device__ __forceinline__ void stmatrix_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---- the list of tiles -----------------------------------------------------------------------

// Rows [r0, r0 + m) of expert e.  `bad`: offsets that run backwards or out of the
// buffer.  Where no expert's are, the experts' rows are apart and in the buffer.
__device__ __forceinline__ void expert_rows(const Params &p, int e, int &r0, int &m, bool &bad) {
    if (p.off == nullptr) {
        r0 = 0;
        m = (int)p.rows;
        return;
    }
    const int64_t a = __ldg(p.off + e), b = __ldg(p.off + e + 1), n = b - a;
    if (a < 0 || n < 0 || (p.cap == 0 && b > p.rows)) bad = true;
    r0 = (int)(p.cap > 0 ? e * p.cap : a);
    m = (int)(p.cap > 0 && n > p.cap ? p.cap : n);
}

// One tile: features [f0, f0 + 128) of expert e in this block (the pair's 256
// side by side; f0 may be past the last one), token rows [row0, row0 + n).
struct Tiles {
    const int32_t *first, *row0s, *counts, *pers;   // shared: tiles' prefix sums over experts, rows, rows a tile
    int ftiles, rank, last;                  // last: tiles of rows in all
    int q, ft, dq, dft;                      // the tile of rows and of features, and the step from one tile to the next
    int e, begin, end, per, rows0, stop;     // expert: its tiles of rows, rows a tile, its rows
    int f0, row0, n;

    __device__ __forceinline__ void start(const Params &p, const int32_t *tables) {
        first = tables;
        row0s = tables + p.E + 1;
        counts = row0s + p.E;
        pers = counts + p.E;
        ftiles = (p.F + 2 * kM - 1) / (2 * kM);
        rank = (int)(blockIdx.x & 1);
        last = first[p.E];
        const int per_cluster = 2 * p.split, pair = blockIdx.x / per_cluster, pairs = gridDim.x / per_cluster;
        q = pair / ftiles, ft = pair % ftiles;
        dq = pairs / ftiles, dft = pairs % ftiles;
        e = -1, begin = end = 0;
        place();
    }
    __device__ __forceinline__ bool valid() const { return q < last; }
    __device__ __forceinline__ void next() {
        q += dq;
        ft += dft;
        if (ft >= ftiles) ft -= ftiles, ++q;
        place();
    }
    __device__ __forceinline__ void place() {
        if (q >= last) return;
        if (q >= end) {
            do {
                begin = end;
                end = first[++e + 1];
            } while (end <= q);
            per = pers[e];
            rows0 = row0s[e];
            stop = rows0 + counts[e];
        }
        f0 = (2 * ft + rank) * kM;
        row0 = rows0 + (q - begin) * per;
        n = stop - row0 < per ? stop - row0 : per;
    }
    __device__ __forceinline__ int columns() const { return (n + 15) & ~15; }
};

// ---- scales ----------------------------------------------------------------------------------

// Sixteen bytes at `q`, those outside the array [begin, end) zero.
__device__ __noinline__ uint4 edge16(const uint8_t *q, const uint8_t *begin, const uint8_t *end) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (q + i >= begin && q + i < end) w[i / 4] |= (uint32_t)__ldg(q + i) << (8 * (i % 4));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The 16-byte pieces around a chunk of a scale row (32 bytes from p, `valid` of
// them in the row), which may start anywhere.  A lane loads a row: each load
// touches 32 lines whatever its width, so it is as wide as it can be (64 experts
// of 128 rows, 7200 -> 2048: 115 us, with 4-byte words 175; 7168 takes 99).
__device__ __forceinline__ void load_scales(const uint8_t *p, int valid, const uint8_t *begin, const uint8_t *end, uint32_t w[12]) {
    const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        uint4 a = make_uint4(0, 0, 0, 0);
        if (16 * i < off + valid) {
            const uint8_t *q = p - off + 16 * i;
            a = q >= begin && q + 16 <= end ? __ldg(reinterpret_cast<const uint4 *>(q)) : edge16(q, begin, end);
        }
        w[4 * i] = a.x, w[4 * i + 1] = a.y, w[4 * i + 2] = a.z, w[4 * i + 3] = a.w;
    }
}

// The chunk's bytes out of those pieces; what is behind `valid` becomes zero.
__device__ __forceinline__ void shift_scales(const uint32_t w[12], const uint8_t *p, int valid, uint32_t v[8]) {
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15);
    uint32_t t[10];
#pragma unroll
    for (int i = 0; i < 10; ++i) t[i] = (off & 8) ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 9; ++i) t[i] = (off & 4) ? t[i + 1] : t[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __funnelshift_r(t[i], t[i + 1], 8 * (off & 3));
    if (valid < 32) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (valid - 4 * i < 4) v[i] &= valid > 4 * i ? (1u << (8 * (valid - 4 * i))) - 1u : 0u;
    }
}

// ---- results ---------------------------------------------------------------------------------

// Another pair's sums of a tile: for each 32 columns and each epilogue warp its
// 32 registers, 128 bytes (a lane each) a register.
__host__ __device__ __forceinline__ uint32_t part_bytes(int nt) { return (uint32_t)((nt + 31) / 32) * (4 * 32 * 32 * 4); }
__device__ __forceinline__ int part_index(int column, int quarter, int lane) { return ((column / 32) * 4 + quarter) * 1024 + lane; }

__device__ __forceinline__ void dump_tile(const Tiles &tile, uint32_t d, int quarter, int lane, uint32_t part) {
    d += (uint32_t)(quarter * 32) << 16;
    const int columns = tile.columns();
    for (int c = 0; c < columns; c += 32) {
        uint32_t r[2][16];
        __syncwarp();
        tmem_ld_16x32(d + c, r[0]);
        tmem_ld_16x32(d + c + (16u << 16), r[1]);
        tmem_ld_wait();
        const uint32_t to = part + 4 * part_index(c, quarter, lane);
#pragma unroll
        for (int j = 0; j < 32; ++j)
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to + 128 * j), "r"(r[j / 16][j % 16]) : "memory");
    }
}

// A warp's 32 features of the tile, `parts` other pairs' sums added to this one's, as BF16 rows of y.
__device__ __forceinline__ void store_tile(const Params &p, const Tiles &tile, uint32_t d, int quarter, int lane, uint32_t out,
                                           uint8_t *out_ptr, const float *part, int parts) {
    const int f = tile.f0 + quarter * 32;
    const uint32_t mine = out + quarter * 2048;
    const uint8_t *mine_ptr = out_ptr + quarter * 2048;
    d += (uint32_t)(quarter * 32) << 16;
    const int columns = tile.columns();
    for (int c = 0; c < columns; c += 32) {
        // 32 features x 32 tokens -> [token][feature], 64 bytes a token, its
        // 16-byte pieces exchanged by the token's number so that neither side
        // meets a bank twice
        uint32_t r[2][16];
        tmem_ld_16x32(d + c, r[0]);
        tmem_ld_16x32(d + c + (16u << 16), r[1]);
        tmem_ld_wait();
        for (int i = 0; i < parts; ++i) {
            const float *q = part + (size_t)i * (part_bytes(p.nt) / 4) + part_index(c, quarter, lane);
#pragma unroll
            for (int j = 0; j < 32; ++j) r[j / 16][j % 16] = __float_as_uint(__uint_as_float(r[j / 16][j % 16]) + q[32 * j]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int u = 0; u < 4; u += 2) {
                const int token = 8 * (u + (lane >> 4)) + (lane & 7), piece = 2 * h + ((lane >> 3) & 1);
                uint32_t b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    b[i] = cvt_bf16x2(__uint_as_float(r[h][4 * u + 2 * i]), __uint_as_float(r[h][4 * u + 2 * i + 1]));
                stmatrix_trans(mine + token * 64 + ((piece ^ ((token >> 1) & 3)) << 4), b[0], b[1], b[2], b[3]);
            }
        __syncwarp();
        const int there = tile.n - c < 32 ? tile.n - c : 32;
        uint16_t *y = p.y + ((int64_t)tile.row0 + c) * p.F + f;
        if (p.wide) {
            const int piece = lane & 3;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int token = 8 * i + (lane >> 2);
                const uint4 v = *reinterpret_cast<const uint4 *>(mine_ptr + token * 64 + ((piece ^ ((token >> 1) & 3)) << 4));
                if (token < there && f + 8 * piece < p.F) *reinterpret_cast<uint4 *>(y + (int64_t)token * p.F + 8 * piece) = v;
            }
        } else if (f + lane < p.F) {
            for (int token = 0; token < there; ++token)
                y[(int64_t)token * p.F + lane] = *reinterpret_cast<const uint16_t *>(
                    mine_ptr + token * 64 + (((lane >> 3) ^ ((token >> 1) & 3)) << 4) + 2 * (lane & 7));
        }
        __syncwarp();
    }
}

// ---- the kernel ------------------------------------------------------------------------------

__global__ void __launch_bounds__(kThreads, 1)
matmul_mxfp4_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    // full, sffull and accfree count for the pair, in its first block; empty, sffree and accfull are told to both
    __shared__ uint64_t s_full[kMaxStages], s_empty[kMaxStages], s_sffull[3], s_sffree[3], s_accfull[2], s_accfree[2], s_drain[2];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort_word;
    volatile int *abort = &s_abort_word;

    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank(), lead = rank & ~1u;   // lead: the pair's first block
    const bool first = rank == lead;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *ring_ptr = smem_raw + (ring - smem_u32(smem_raw));
    const uint32_t sf_ring = ring + p.stages * p.stage_bytes, out = sf_ring + p.chunks * p.chunk_bytes;
    uint8_t *sf_ptr = ring_ptr + (size_t)p.stages * p.stage_bytes, *out_ptr = sf_ptr + (size_t)p.chunks * p.chunk_bytes;
    int32_t *tables = reinterpret_cast<int32_t *>(out_ptr + kOutBytes);

    if (warp == 0) {   // a lane each: one thread alone took 1000 cycles
        if (lane < p.stages) {
            bar_init(smem_u32(&s_full[lane]), 2);   // the copies' bytes, the scales in TMEM
            bar_init(smem_u32(&s_empty[lane]), 1);
        }
        if (lane < p.chunks) {
            bar_init(smem_u32(&s_sffull[lane]), 2 * (1 + p.nb));   // the scale warps of both blocks
            bar_init(smem_u32(&s_sffree[lane]), 1);
        }
        if (lane < 2) {
            bar_init(smem_u32(&s_accfull[lane]), 1);
            bar_init(smem_u32(&s_accfree[lane]), 8);   // the epilogue warps of both blocks
            bar_init(smem_u32(&s_drain[lane]), 1);
        }
        if (lane == 0) {
            s_abort_word = 0;
            asm volatile("prefetch.tensormap [%0];" ::"l"(&map_a) : "memory");
            asm volatile("prefetch.tensormap [%0];" ::"l"(&map_w) : "memory");
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    griddep_wait();

    // tables: first[E + 1] (tiles of nt rows before each expert), row0[E], rows[E], rows a tile[E]
    bool bad = false;
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        int r0, m;
        expert_rows(p, e, r0, m, bad);
        tables[p.E + 1 + e] = r0;
        tables[2 * p.E + 1 + e] = m;
        // rows of a tile: the expert's, in equal parts of at most nt, rounded up to 16
        const uint32_t parts = ((uint32_t)m + p.nt - 1) / p.nt;
        tables[3 * p.E + 1 + e] = parts > 0 ? (int)((((uint32_t)m + parts - 1) / parts + 15) & ~15u) : 0;
    }
    // bad offsets: no tiles at all, for the sums below hold only where rows do not overlap
    const bool refused = __syncthreads_or(bad) != 0;
    if (bad && blockIdx.x == 0) report(p.status, kErrRange);
    if (refused) {
        for (int e = threadIdx.x; e <= p.E; e += blockDim.x) tables[e] = 0;
    } else if (warp == 0) {
        const int per = (p.E + 31) / 32, e0 = lane * per, e1 = e0 + per < p.E ? e0 + per : p.E;
        int sum = 0;
        for (int e = e0; e < e1; ++e) sum += ((uint32_t)tables[2 * p.E + 1 + e] + p.nt - 1) / p.nt;
        int before = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, before, o);
            if (lane >= o) before += v;
        }
        before -= sum;
        for (int e = e0; e < e1; ++e) {
            tables[e] = before;
            before += ((uint32_t)tables[2 * p.E + 1 + e] + p.nt - 1) / p.nt;
        }
        if (e0 < p.E && e1 == p.E) tables[p.E] = before;
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    // this pair's stages [k0, k1), whole chunks of scales
    const int ksteps = (p.K + kStageK - 1) / kStageK, kchunks = (ksteps + kChunk - 1) / kChunk;
    const int c0 = kchunks * (int)(rank >> 1) / p.split, c1 = kchunks * (int)((rank >> 1) + 1) / p.split;
    const int k0 = c0 * kChunk, k1 = c1 * kChunk < ksteps ? c1 * kChunk : ksteps;

    Tiles tile;
    bool done = false;
    if (warp == 0 || warp == 9) {
        int s = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (tile.start(p, tables); ok && tile.valid(); tile.next()) {
            const int half = tile.columns() / 2, boxes = (half + p.box - 1) / p.box;
            const uint32_t box_bytes = p.box * (kStageK / 2);
            const int row0 = tile.row0 + tile.rank * half;
            for (int k = k0; k < k1; ++k) {
                ok = __all_sync(0xFFFFFFFFu, bar_wait(smem_u32(&s_empty[s]), phase ^ 1, abort, p));
                if (!ok) break;
                const uint32_t base = ring + s * p.stage_bytes, bar = in_block(smem_u32(&s_full[s]), lead);
                if (warp == 0) {
                    if (elect_one()) {
                        if (first) bar_expect(smem_u32(&s_full[s]), 2 * (kABytes + boxes * box_bytes));
                        tma_3d(base, &map_w, k * (kStageK / 2), tile.f0, tile.e, bar);
                    }
                } else if (elect_one()) {
                    for (int b = 0; b < boxes; ++b)
                        tma_2d(base + kABytes + b * box_bytes, &map_a, k * (kStageK / 2), row0 + b * p.box, bar);
                }
                __syncwarp();
                if (++s == p.stages) s = 0, phase ^= 1;
            }
        }
        // Once more round the ring, a lane a place: the last releases are arrivals from
        // the first block, and a block must not leave before they have reached its barriers.
        if (ok && warp == 0 && lane < p.stages) bar_wait(smem_u32(&s_empty[lane]), lane < s ? phase : phase ^ 1, abort, p);
    } else if ((warp == 1 || warp == 10) && first) {
        // What bounds this loop is its instructions: 20 to 30 cycles for each that it
        // issues, as much for each branch.  Hence two warps, a wait that is asked for
        // a stage ahead, and K's tail run as zeros.  A stage's scales have a place of
        // their own in TMEM (its place in the ring): the MMAs that read it before had
        // ended when the stage was free.
        const bool mma = warp == 1;
        const uint32_t full0 = smem_u32(&s_full[0]), empty0 = smem_u32(&s_empty[0]);
        const uint32_t sf0 = tmem + 2 * p.nt, sf_cols = 8 + 8 * p.nb, nb = p.nb, stages = p.stages, stage_bytes = p.stage_bytes;
        uint32_t s = 0, base = ring, tsf = sf0, phase = 0;      // ring position
        bool ok = true, any = false;
        tile.start(p, tables);
        if (mma) {
            uint32_t acc = 0, accphase = 0;
            bool ready = false;
            for (; ok && tile.valid(); tile.next()) {
                const uint32_t i0 = instr_desc(tile.columns(), 0), i2 = instr_desc(tile.columns(), 2);
                ok = bar_wait(smem_u32(&s_accfree[acc]), accphase ^ 1, abort, p);
                const uint32_t d = tmem + acc * p.nt;
                for (int k = k0; k < k1; ++k) {
                    if (!ready) ok = ok && bar_wait(full0 + 8 * s, phase, abort, p);
                    tc_fence_after();
                    const uint32_t empty = empty0 + 8 * s, ta = tsf, tb = tsf + 8;
                    const uint64_t da = desc_rows(base), db = desc_rows(base + kABytes);
                    ++s, base += stage_bytes, tsf += sf_cols;
                    if (s == stages) s = 0, base = ring, tsf = sf0, phase ^= 1;
                    ready = bar_test(full0 + 8 * s, phase);
                    fence_acquire_smem();
                    if (elect_one() && ok) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)     // 64 values: 32 bytes (two units) of each row
                            mma_mxf4(d, da + 2 * i, db + 2 * i, (i & 1) ? i2 : i0, ta + 4 * (i >> 1), tb + 4 * (i >> 1) * nb,
                                     i > 0 || k > k0);
                        mma_commit_both(empty, lead);
                    }
                }
                if (elect_one() && ok) mma_commit_both(smem_u32(&s_accfull[acc]), lead);
                any = true;
                ok = __all_sync(0xFFFFFFFFu, ok);
                acc ^= 1;
                if (acc == 0) accphase ^= 1;
            }
        } else {
            uint32_t ch = 0, chphase = 0;
            for (; ok && tile.valid(); tile.next()) {
                const bool two = tile.columns() > 128;
                for (int k = k0; k < k1; k += kChunk) {
                    ok = ok && bar_wait(smem_u32(&s_sffull[ch]), chphase, abort, p);
                    const uint32_t sf = sf_ring + ch * p.chunk_bytes;
                    const uint64_t sa = desc_scales(sf), sb = desc_scales(sf + kChunkA);
#pragma unroll
                    for (int j = 0; j < kChunk; ++j) {
                        if (k + j >= k1) break;
                        ok = ok && bar_wait(empty0 + 8 * s, phase ^ 1, abort, p);
                        tc_fence_after();
                        if (elect_one() && ok) {
#pragma unroll
                            for (int w = 0; w < 2; ++w) {   // 512 bytes (32 descriptor units) a block
                                scales_to_tmem(tsf + 4 * w, sa + 32 * (2 * j + w));
                                scales_to_tmem(tsf + 8 + 4 * w * nb, sb + 32 * (2 * j + w) * nb);
                                if (two) scales_to_tmem(tsf + 8 + 4 * (w * nb + 1), sb + 32 * ((2 * j + w) * nb + 1));
                            }
                            mma_commit(full0 + 8 * s);
                        }
                        ++s, tsf += sf_cols;
                        if (s == stages) s = 0, tsf = sf0, phase ^= 1;
                    }
                    if (elect_one() && ok) mma_commit_both(smem_u32(&s_sffree[ch]), lead);
                    any = true;
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    if (++ch == p.chunks) ch = 0, chphase ^= 1;
                }
            }
        }
        if (any) {   // every MMA and copy has ended before TMEM is freed
            const uint32_t drain = smem_u32(&s_drain[mma ? 0 : 1]);
            __syncwarp();
            if (elect_one()) mma_commit(drain);
            __syncwarp();
            const long long start = clock64();
            while (!bar_try(drain, 0) && clock64() - start < kWaitCycles) {}
        }
    } else if (warp == 2 || warp == 3 || warp == 8 || warp == 11) {
        const bool weights = warp == 2 || warp == 11;
        const int block = warp == 8 ? 1 : 0;   // 128-row block of the token side
        const int odd = warp == 11 ? 1 : 0, stride = weights ? p.sfwarps : 1;   // which of the chunks
        if (weights ? odd < p.sfwarps : block < p.nb) {
            const int row_bytes = p.K / 32;
            int ch = odd, chunk = c0;
            uint32_t phase = 0;
            uint32_t raw[4][12], v[4][8];   // the chunk ahead, in flight, and the present one
            const uint8_t *const begin = weights ? p.sw : p.sa;
            const uint8_t *const end = begin + (weights ? (int64_t)p.E * p.F : p.rows) * row_bytes;
            // this lane's first row of a tile's chunk; rows 32 apart, `rows` of 128 there
            const auto chunk_at = [&](const Tiles &t, int c, int &rows, int &valid) {
                rows = (weights ? p.F - t.f0 : t.n - block * 128) - lane;
                valid = row_bytes - c * 32 < 32 ? row_bytes - c * 32 : 32;
                return begin + (weights ? (int64_t)t.e * p.F + t.f0 : (int64_t)t.row0 + block * 128) * row_bytes +
                       (int64_t)lane * row_bytes + c * 32;
            };
            const auto load = [&](const Tiles &t, int c) {
                int rows, valid;
                const uint8_t *at = chunk_at(t, c, rows, valid);
                if (p.aligned) {   // the plain form, for its fewer instructions
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 *q = reinterpret_cast<const uint4 *>(at + (int64_t)(32 * i) * row_bytes);
                        uint4 a = make_uint4(0, 0, 0, 0), b = a;
                        if (32 * i < rows) {
                            a = __ldg(q);
                            if (valid > 16) b = __ldg(q + 1);
                        }
                        raw[i][0] = a.x, raw[i][1] = a.y, raw[i][2] = a.z, raw[i][3] = a.w;
                        raw[i][4] = b.x, raw[i][5] = b.y, raw[i][6] = b.z, raw[i][7] = b.w;
                    }
                    return;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    load_scales(at + (int64_t)(32 * i) * row_bytes, 32 * i < rows ? valid : -16, begin, end, raw[i]);
            };
            // the weights' scales of a tile lie in one piece: asked into L2 a tile
            // ahead, since a load that has to queue behind the ring's own copies
            // comes too late (one chunk in flight a warp)
            const auto to_l2 = [&](const Tiles &t) {
                if (!weights || odd || lane != 0 || !t.valid()) return;
                const int there = p.F - t.f0 < kM ? p.F - t.f0 : kM;
                if (there <= 0) return;
                const uintptr_t a = reinterpret_cast<uintptr_t>(p.sw + ((int64_t)t.e * p.F + t.f0) * row_bytes);
                const uintptr_t a0 = (a + 15) & ~(uintptr_t)15, a1 = (a + (int64_t)there * row_bytes) & ~(uintptr_t)15;
                if (a1 > a0) prefetch_l2_bulk(reinterpret_cast<const void *>(a0), (uint32_t)(a1 - a0));
            };
            const auto step = [&](Tiles &t, int &c) {
                if (++c < c1) return;
                c = c0;
                t.next();
                Tiles after = t;
                after.next();
                to_l2(after);
            };
            tile.start(p, tables);
            to_l2(tile);
            if (tile.valid()) {
                Tiles second = tile;
                second.next();
                to_l2(second);
            }
            // one copy of each part of the loop: its instructions are what the
            // block's other warps wait for in the instruction cache
            Tiles ahead = tile;
            int ahead_chunk = c0, steps = odd;
            bool ok = true;
            for (bool have = false;; have = true, steps = stride) {
#pragma unroll 1
                for (int i = 0; i < steps && ahead.valid(); ++i) step(ahead, ahead_chunk);
                if (have) {
                    if (p.aligned) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int j = 0; j < 8; ++j) v[i][j] = raw[i][j];
                    } else {
                        int rows, valid;
                        const uint8_t *at = chunk_at(tile, chunk, rows, valid);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            shift_scales(raw[i], at + (int64_t)(32 * i) * row_bytes, 32 * i < rows ? valid : 0, v[i]);
                    }
                }
                if (ahead.valid()) load(ahead, ahead_chunk);
                if (have) {
                    ok = __all_sync(0xFFFFFFFFu, bar_wait(smem_u32(&s_sffree[ch]), phase ^ 1, abort, p));
                    if (!ok) break;
                    uint8_t *to = sf_ptr + (size_t)ch * p.chunk_bytes + (weights ? 0 : kChunkA + 512 * block) + lane * 16;
                    const int pitch = 512 * (weights ? 1 : p.nb);
#pragma unroll
                    for (int j = 0; j < 8; ++j)   // 128 values each; past the row's end zeros that nothing reads
                        *reinterpret_cast<uint4 *>(to + j * pitch) = make_uint4(v[0][j], v[1][j], v[2][j], v[3][j]);
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) bar_arrive_smem(in_block(smem_u32(&s_sffull[ch]), lead));
                    ch += stride;
                    if (ch >= p.chunks) ch -= p.chunks, phase ^= 1;
                }
                if (!ahead.valid()) break;
                tile = ahead;
                chunk = ahead_chunk;
            }
            // the last releases of this ring, as those of the stages' (warp 3 has filled every place of it)
            if (ok && warp == 3 && lane < p.chunks) bar_wait(smem_u32(&s_sffree[lane]), lane < ch ? phase : phase ^ 1, abort, p);
        }
    } else if (warp >= 4 && warp < 8) {
        int acc = 0;
        uint32_t accphase = 0;
        for (tile.start(p, tables); tile.valid(); tile.next()) {
            done = __all_sync(0xFFFFFFFFu, bar_wait(smem_u32(&s_accfull[acc]), accphase, abort, p));
            if (!done || p.split > 1) break;
            tc_fence_after();
            store_tile(p, tile, tmem + acc * p.nt, warp & 3, lane, out, out_ptr, nullptr, 0);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive_tmem(in_block(smem_u32(&s_accfree[acc]), lead));
            acc ^= 1;
            if (acc == 0) accphase ^= 1;
        }
    }
    if (p.split > 1) {
        // One tile a cluster.  Once every pair's MMAs have ended the rings are free:
        // the others lay their sums into the first pair's, register by register, and
        // it adds them to its own in the pairs' order.
        __syncwarp();
        cluster_sync();
        const bool epilogue = warp >= 4 && warp < 8 && done;   // done: this pair's part of a tile is in TMEM
        if (epilogue && rank >= 2) {
            tc_fence_after();
            const uint32_t part = in_block(ring + (rank / 2 - 1) * part_bytes(p.nt), rank & 1);
            dump_tile(tile, tmem, warp & 3, lane, part);
        }
        __syncwarp();
        cluster_sync();
        if (epilogue && rank < 2) {
            tc_fence_after();
            store_tile(p, tile, tmem, warp & 3, lane, out, out_ptr, reinterpret_cast<const float *>(ring_ptr), p.split - 1);
        }
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync();   // the pair's memory, barriers and TMEM stay until both are done
    // Without an error the MMA warp has waited for every copy of both blocks.  With
    // one, whichever role it was that gave up, copies and commits may still be under
    // way; none was issued after the barrier above, and they get 2^28 cycles to land.
    if (*abort)
        for (const long long start = clock64(); clock64() - start < kLandCycles;) {}
    __syncwarp();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeTiled>(f);
    }();
    return fn;
}

// Rows of codes as bytes: [planes][rows][row_bytes], boxes of 128 bytes x box_rows, zeros outside.
bool make_map(CUtensorMap *map, const void *p, int64_t row_bytes, int64_t rows, int64_t planes, int box_rows) {
    const cuuint64_t dims[3] = {(cuuint64_t)row_bytes, (cuuint64_t)rows, (cuuint64_t)planes};
    const cuuint64_t strides[2] = {(cuuint64_t)row_bytes, (cuuint64_t)(row_bytes * rows)};
    const cuuint32_t box[3] = {kStageK / 2, (cuuint32_t)box_rows, 1}, step[3] = {1, 1, 1};
    const EncodeTiled fn = encode_tiled();
    return fn != nullptr && fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, planes > 0 ? 3 : 2, const_cast<void *>(p), dims, strides, box,
                               step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cgl_status launch_matmul_mxfp4(const uint8_t *a, const uint8_t *sa, int64_t rows, const uint8_t *w, const uint8_t *sw,
                               int E, int F, int K, const int32_t *off, int64_t cap, uint16_t *y, int num_sms,
                               uint32_t *status, cudaStream_t stream, int64_t wait_cycles) {
    if (rows == 0) return CGL_OK;
    Params p = {};
    p.sa = sa, p.sw = sw, p.off = off, p.y = y, p.status = status;
    p.rows = rows, p.cap = cap, p.E = E, p.F = F, p.K = K;
    p.wait_cycles = wait_cycles < 0 || wait_cycles > kWaitCycles ? kWaitCycles : wait_cycles;
    // Columns a tile: a quarter over the mean rows of an expert (a padded one's
    // capacity), so that few experts need two tiles.
    const int64_t mean = (rows + E - 1) / E, want = cap > 0 ? cap : mean + mean / 4 + 8;
    p.nt = want >= kMaxNt ? kMaxNt : want <= 32 ? 32 : (int)((want + 15) / 16 * 16);
    p.nb = p.nt > 128 ? 2 : 1;
    p.box = p.nt > 64 ? 32 : 16;
    p.stage_bytes = kABytes + (p.nt / 2 + p.box - 1) / p.box * p.box * (kStageK / 2);
    p.chunk_bytes = kChunkA * (1 + p.nb);
    const size_t tables = (size_t)(4 * E + 1) * 4;
    const size_t room = kSmemLimit - 1024 - kOutBytes - tables;
    int stages = (int)((room - 2 * p.chunk_bytes) / p.stage_bytes);
    const int by_tmem = (512 - 2 * p.nt) / (8 + 8 * p.nb);
    if (stages > by_tmem) stages = by_tmem;
    if (stages > kMaxStages) stages = kMaxStages;
    p.chunks = room - (size_t)stages * p.stage_bytes >= 3 * p.chunk_bytes ? 3 : 2;
    p.stages = stages;
    p.aligned = K % 512 == 0 && ((reinterpret_cast<uintptr_t>(sa) | reinterpret_cast<uintptr_t>(sw)) & 15) == 0;
    // Few rows an expert: the weights come fast, and one warp for their scales is
    // what the ring waits for.  64 experts, one warp and two: 7168 -> 2048 with 16 rows
    // (32 columns a tile) 94 and 86 us, 64 rows (96) 99 and 91, 134 rows (176) 105 and
    // 102; 2048 -> 7168 with 112 rows (160) 98 and 97, 134 rows 102 and 100.  At 208
    // columns there is nothing between them (150 rows 109 and 110, 110 and 113; 512
    // rows 246 and 245, 267 and 267), and the block does without the warp.
    p.sfwarps = p.nt <= 176 ? 2 : 1;
    p.wide = F % 8 == 0 && (reinterpret_cast<uintptr_t>(y) & 15) == 0;
    const size_t smem = 1024 + (size_t)stages * p.stage_bytes + (size_t)p.chunks * p.chunk_bytes + kOutBytes + tables;

    CUtensorMap map_a, map_w;
    if (!make_map(&map_a, a, K / 2, rows, 0, p.box) || !make_map(&map_w, w, K / 2, F, E, kM)) return CGL_ECUDA;
    if (!ensure_smem_attr((const void *)matmul_mxfp4_kernel, smem)) return CGL_ECUDA;
    const int sms = device_sm_count();
    if (sms <= 0) return CGL_ECUDA;
    const int64_t ftiles = (F + 2 * kM - 1) / (2 * kM);
    const int64_t most = ((rows + p.nt - 1) / p.nt + (rows < E ? rows : E)) * ftiles;   // no more tiles than this
    int64_t pairs = (num_sms > 0 && num_sms < sms ? num_sms : sms) / 2;
    if (pairs < 1) pairs = 1;
    // Where `most` tiles would leave three quarters or half of the pairs without work,
    // four or two pairs share one, a part of K each (whole chunks of scales), as long as
    // their sums fit into the first pair's ring.  `most` is known without the offsets and
    // may be twice the tiles there are: one row, 7168 -> 4096, has 16 tiles, counts as 32
    // and runs as two pairs a tile (12 and 16 stages).
    p.split = 1;
    for (int split = 4; split > 1 && p.split == 1; split /= 2)
        if (most * split <= pairs && (K + kStageK * kChunk - 1) / (kStageK * kChunk) >= split &&
            (split - 1) * part_bytes(p.nt) <= (uint32_t)stages * p.stage_bytes)
            p.split = split;
    if (pairs > most) pairs = most;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * pairs * p.split));
    cfg.blockDim = dim3(p.sfwarps == 2 ? kThreads : kThreads - 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2 * p.split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, matmul_mxfp4_kernel, map_a, map_w, p) == cudaSuccess ? CGL_OK : CGL_ECUDA;
}

}  // namespace cgl

// The experts' product on BF16 rows with bias, activation and residual, and its
// gradients (formulas at cgl_matmul_bf16 in cgl.h).  With e the expert of row r:
//   forward  z[r, f]  = sum_k w[e, f, k] a[r, k]      y = act(z + bias) + residual
//   grad_a   da[r, k] = sum_f w[e, f, k] dz[r, f]     dz = grad_y act'(z), slope.cu
//   grad_w   dw[f, k] = sum_r a[r, k] dz[r, f]        over the rows of one expert
// One kernel computes all three as out[n, m] = sum_c X[m, c] Y[n, c]: m the features
// that lie side by side in the result's rows, n the rows.  X is w, w and a, Y is a, dz
// and dz; c is the inner dimension of an operand's rows in memory (K-major) for both
// in the forward and for Y in grad_a, the outer one (MN-major) for the others, which
// the tensor core reads either way.
//
// Tensor cores: tcgen05.mma kind::f16, cta_group::2: a pair of blocks on
// neighbouring SMs works on one tile of 256 features, 128 in each block, and of up
// to 256 rows, half of them in each block's shared memory.  The rows of an expert
// are cut into equal parts of at most `nt`, rounded up to 16: few rows cost few
// columns.  Persistent pairs walk the list of tiles; each block makes the list's
// prefix sums from expert_offset for itself.  One block:
//   warps 0, 2  TMA: a ring of stages of 64 values of c, 128-byte swizzle; 0 X, 2 Y
//   warp 1      in the pair's first block, for both: the MMAs, 4 a stage
//   warp 3      grad_w: an expert's rows end inside a stage, what lies behind them (the
//               next expert's, or anything) becomes zero before the MMAs read it
//   warps 4-11  TMEM -> registers -> bias, activation, residual -> transposed through
//               shared memory -> BF16 rows, while the next tile's MMAs run; two warps
//               for each 32 lanes of TMEM, 32 columns in turn
// A gated product has gate and up features 16 by 16 in the tile's rows, so that both
// come to the same lane.  Where tiles are few (see plan), two to four pairs share one,
// a part of c each, and join their sums in order through distributed shared memory.
//
// What bounds it (B200; floors at the measured 6.55 TB/s copy and 1656 TFLOP/s burst,
// 1396 sustained).  Few rows an expert, the weights' bytes: 4 rows, 256 experts, 7168 ->
// 2 x 2048 gated 2.07 ms (7.1 TB/s, the floor 2.26 being that of a copy); 128 rows 2.29 to 2.45
// ms in short runs (floor 2.39), 2.6 to 3.0 at the 1000 W cap.  Many rows, the tensor cores
// and in long runs the cap: 8192^3 676 to 707 us in a short run by the card (1555 to 1626
// TFLOP/s; cuBLAS 662 to 671), 780 to 849 in a long one (750 to 802); grad_a 676 to 852 and 839 to
// 849, grad_w 702 to 835 and 890 to 929.  512 rows an expert, 2048 -> 7168, 16 experts: 168 us
// with the tensor pipe active 79% of the time, 12.1 waves of tiles in 13; a tile of
// 200 columns takes 71 bytes a cycle and SM from L2, whose ports carry 64.  One row, 7168
// -> 4096: 17.5 us, 9 of bytes and 5.5 for a call without work; 128 rows 21.6 (cuBLAS
// 14); both are 16 tiles of three pairs, 96 of 148 SMs.  Sums are binary32, but the
// tensor cores cut each addition towards zero: 1.5e-6 off (root mean square) for 1520
// terms whose sum is about 1, where rounded additions are 8e-8 off.
//
// Every wait is bounded (about a second, then CGL_ETIMEOUT): the pair's roles leave
// their loops, MMAs in flight are waited for, copies and arrivals under way get
// 0.15 s to land before either block leaves, TMEM is freed.
#include <cuda.h>

#include <cmath>
#include <mutex>

#include "matmul_bf16.cuh"
#include "launch.h"

namespace cgl {

namespace {

constexpr uint32_t kErrTimeout = 1u << CGL_ETIMEOUT;
constexpr long long kWaitCycles = 1ll << 31;
constexpr long long kLandCycles = 1ll << 28;
constexpr int kEpilogue = 8;               // warps
constexpr int kThreads = 128 + 32 * kEpilogue;
constexpr int kStageC = 64;                // values of c a stage
constexpr int kM = 128;                    // features a block
constexpr int kMaxNt = 256;                // 2 accumulators of 256 columns fill TMEM
constexpr int kMaxStages = 12;
constexpr int kBand = 8;                   // tiles of rows
constexpr int kOutBytes = kEpilogue * 2048;   // the epilogue's 32 x 32 BF16 blocks, one a warp
constexpr size_t kSmemLimit = 226 * 1024;  // dynamic part: 227 KiB less the static part
constexpr uint32_t kXBytes = kM * kStageC * 2;
constexpr uint32_t kChunkBytes = 64 * 128;    // MN-major: 64 values of c, each 64 neighbours (128 bytes)

enum Mode { kForward, kGated, kGradA, kGradW };

struct Params {
    const int32_t *off;
    const uint16_t *bias, *residual;
    uint16_t *y;
    void *preact;
    uint32_t *status;
    int64_t rows, cap;
    int E;
    int M;           // columns of the result
    int N;           // grad_w: rows of the result an expert
    int C;           // values of c (grad_w: the expert's rows)
    int act;
    int preact_wide; // binary32
    int nt;          // most columns of the accumulator a tile
    int box;         // rows a TMA box of Y (K-major)
    int stages;
    int split;       // pairs that share a tile, each a part of c (one cluster)
    int wide;        // y's, residual's and preact's rows allow 16-byte accesses
    uint32_t stage_bytes;
    long long wait_cycles;
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
// Half of what a barrier counts is done by the pair's other block, so every wait
// has cluster scope; the fence after it and its counterpart in bar_arrive_smem are
// restricted to shared memory, since fences of all memory at that scope hold a
// warp until its loads in flight are there.
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
// Arrive at a barrier of either block of the pair.  _tmem hands back TMEM that
// tcgen05.ld has read: execution order is all that needs, with tcgen05's fences on
// both sides.  _smem announces what this warp wrote to its own shared memory (after a
// proxy fence), which the tensor core reads on behalf of a thread of the first block.
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

// One lane of a converged warp, always the same.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xFFFFFFFF;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}

// Tile loads into this block; the barrier may be the first block's.
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int u, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(u), "r"(bar)
        : "memory");
}

// Shared-memory descriptors, 128-byte swizzle.  K-major: rows of 128 bytes, groups
// of eight rows 1024 bytes apart.  MN-major: 64 neighbours (128 bytes) for each c,
// groups of eight c 1024 bytes apart, the next 64 neighbours a chunk further.
__device__ __forceinline__ uint64_t desc_k(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(kChunkBytes >> 4) << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// Instruction descriptor: BF16 x BF16, binary32 sums, M = 256, N columns; which operands are MN-major.
template <int MODE>
__device__ __forceinline__ uint32_t instr_desc(int n) {
    constexpr uint32_t x_mn = MODE == kGradA || MODE == kGradW, y_mn = MODE == kGradW;
    return (1u << 4) | (1u << 7) | (1u << 10) | (x_mn << 15) | (y_mn << 16) | ((uint32_t)(n >> 3) << 17) | (16u << 24);
}
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive, once this thread's MMAs so far have ended, at a barrier of both blocks or of this one.
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
__device__ __forceinline__ void stmatrix_trans(uint32_t addr, const uint32_t b[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(b[0]), "r"(b[1]),
                 "r"(b[2]), "r"(b[3])
                 : "memory");
}
__device__ __forceinline__ void ldmatrix_trans(uint32_t addr, uint32_t b[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---- the list of tiles -----------------------------------------------------------------------

// One tile: features [f0, ...) of this block (f0 may be past the last one), rows
// [row0, row0 + n) of the result, stages [k0, k1) of c for this pair, from c0 on.
template <int MODE>
struct Tiles {
    static constexpr int kFeatures = MODE == kGated ? kM / 2 : kM;   // results a block
    const int32_t *first, *row0s, *counts, *pers;   // shared: tiles' prefix sums over experts, rows, rows a tile
    int mtiles, rank, last;                  // last: tiles of rows in all
    int q, mt, dq, dmt;                      // the tile of rows and of features, and the step from one tile to the next
    int e, begin, end, per, rows0, stop;     // expert: its tiles of rows, rows a tile, its rows
    int f0, row0, n;
    int k0, k1, c0, tail;                    // tail: values of c in the last stage (grad_w), 0: no part of it is behind the rows
    int part, split, ntiles;

    __device__ __forceinline__ void start(const Params &p, const int32_t *tables) {
        first = tables;
        row0s = tables + p.E + 1;
        counts = row0s + p.E;
        pers = counts + p.E;
        mtiles = (p.M + 2 * kFeatures - 1) / (2 * kFeatures);
        rank = (int)(blockIdx.x & 1);
        part = (int)(cluster_rank() >> 1), split = p.split;
        ntiles = (p.N + p.nt - 1) / p.nt;
        last = first[p.E];
        const int per_cluster = 2 * p.split, pair = blockIdx.x / per_cluster, pairs = gridDim.x / per_cluster;
        q = pair / mtiles, mt = pair % mtiles;
        dq = pairs / mtiles, dmt = pairs % mtiles;
        e = -1, begin = end = 0;
        c0 = tail = 0;
        if (MODE != kGradW) {
            const int steps = (p.C + kStageC - 1) / kStageC;
            k0 = (int)((int64_t)steps * part / split), k1 = (int)((int64_t)steps * (part + 1) / split);
        } else {
            per = p.nt, stop = p.N;
        }
        place();
    }
    __device__ __forceinline__ bool valid() const { return q < last; }
    __device__ __forceinline__ void next() {
        q += dq;
        mt += dmt;
        if (mt >= mtiles) mt -= mtiles, ++q;
        place();
    }
    __device__ __forceinline__ void place() {
        if (q >= last) return;
        if (MODE == kGradW) {
            e = q / ntiles;
            row0 = (q - e * ntiles) * per;
            c0 = row0s[e];
            const int m = counts[e], steps = (int)(((uint32_t)m + kStageC - 1) / kStageC);
            k0 = (int)((int64_t)steps * part / split), k1 = (int)((int64_t)steps * (part + 1) / split);
            tail = k1 == steps ? m % kStageC : 0;
        } else {
            if (q >= end) {
                do {
                    begin = end;
                    end = first[++e + 1];
                } while (end <= q);
                per = pers[e];
                rows0 = row0s[e];
                stop = rows0 + counts[e];
            }
            // An expert's tiles in bands of kBand tiles of rows, a band's tiles of features one
            // after the other: the pairs at work at one time share the weights of few features
            // and the rows of one band, rather than all weights and two tiles of rows.
            int row = q - begin, m = mt;
            if (end - begin > 1) {
                const int i = row * mtiles + mt, band = i / (kBand * mtiles), j = i - band * kBand * mtiles;
                const int high = end - begin - band * kBand < kBand ? end - begin - band * kBand : kBand;
                m = j / high;
                row = band * kBand + j - m * high;
            }
            row0 = rows0 + row * per;
            f0 = (2 * m + rank) * kFeatures;
        }
        if (MODE == kGradW) f0 = (2 * mt + rank) * kFeatures;
        n = stop - row0 < per ? stop - row0 : per;
    }
    __device__ __forceinline__ int columns() const { return (n + 15) & ~15; }
    __device__ __forceinline__ bool any() const { return k1 > k0; }
    __device__ __forceinline__ int tail_at(int k) const { return MODE == kGradW && k == k1 - 1 ? tail : 0; }
};

// ---- results ---------------------------------------------------------------------------------

// Another pair's sums of a tile: for each 32 columns and each 32 lanes of TMEM
// 32 registers, four of them 512 bytes (sixteen a lane).
__host__ __device__ __forceinline__ uint32_t part_bytes(int nt) { return (uint32_t)((nt + 31) / 32) * (4 * 32 * 32 * 4); }
__device__ __forceinline__ int part_index(int column, int quarter, int lane) { return ((column / 32) * 4 + quarter) * 1024 + lane * 4; }

// A warp's share of a tile: 32 lanes of TMEM (`quarter`), every second block of 32 columns.
template <int MODE>
__device__ __forceinline__ void dump_tile(const Tiles<MODE> &tile, bool any, uint32_t d, int quarter, int half, int lane, uint32_t part) {
    d += (uint32_t)(quarter * 32) << 16;
    const int columns = tile.columns();
    for (int c = 32 * half; c < columns; c += 32 * (kEpilogue / 4)) {
        uint32_t r[2][16] = {};
        __syncwarp();
        if (any) {
            tmem_ld_16x32(d + c, r[0]);
            tmem_ld_16x32(d + c + (16u << 16), r[1]);
            tmem_ld_wait();
        }
        const uint32_t to = part + 4 * part_index(c, quarter, lane);
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
            const uint32_t *v = &r[j / 16][j % 16];
            asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to + 128 * j), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
        }
    }
}

// A warp's block of 32 rows x 32 features in shared memory: 64 bytes a row, its 16-byte
// pieces exchanged by the row's number so that neither side meets a bank twice.
__device__ __forceinline__ int block_at(int row, int piece) { return row * 64 + ((piece ^ ((row >> 1) & 3)) << 4); }

// The block to global memory (or from it): rows `there`, PIECES pieces of eight
// features; column(i) is where the block's feature i stands in a row, -1 nowhere.
template <int PIECES, bool STORE, typename Column>
__device__ __forceinline__ void move_block(uint8_t *block, uint16_t *base, int64_t ld, int there, int lane, bool wide, Column column) {
    if (wide) {
        const int piece = lane % PIECES, col = column(8 * piece);
        constexpr int kRows = 32 / PIECES;   // a step
        uint4 v[PIECES] = {};
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int row = kRows * i + lane / PIECES;
            uint4 *g = reinterpret_cast<uint4 *>(base + row * ld + col);
            if (row < there && col >= 0) {
                if (STORE) *g = *reinterpret_cast<uint4 *>(block + block_at(row, piece));
                else v[i] = *g;
            }
        }
        if (!STORE)
#pragma unroll
            for (int i = 0; i < PIECES; ++i) *reinterpret_cast<uint4 *>(block + block_at(kRows * i + lane / PIECES, piece)) = v[i];
    } else if (lane < 8 * PIECES) {
        // a feature a lane, eight rows in flight
        const int col = column(lane);
        uint16_t *g = base + col;
        if (col >= 0)
#pragma unroll 1
            for (int row = 0; row < there; row += 8, g += 8 * ld) {
                uint16_t v[8] = {};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint16_t *s = reinterpret_cast<uint16_t *>(block + block_at(row + i, lane >> 3)) + (lane & 7);
                    if (STORE) v[i] = *s;
                    else if (row + i < there) v[i] = g[i * ld];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint16_t *s = reinterpret_cast<uint16_t *>(block + block_at(row + i, lane >> 3)) + (lane & 7);
                    if (!STORE) *s = v[i];
                    else if (row + i < there) g[i * ld] = v[i];
                }
            }
    }
}

template <int MODE>
__device__ __forceinline__ void store_tile(const Params &p, const Tiles<MODE> &tile, bool any, uint32_t d, int quarter, int half, int lane,
                                           uint32_t out, uint8_t *out_ptr, const float *part, int parts) {
    constexpr bool kGate = MODE == kGated, kSum = MODE == kGradA || MODE == kGradW;   // kSum: the sums are the result
    constexpr int kPieces = kGate ? 2 : 4;
    const int f = tile.f0 + quarter * (kGate ? 16 : 32);
    const uint32_t mine = out + (half * 4 + quarter) * 2048;
    uint8_t *mine_ptr = out_ptr + (half * 4 + quarter) * 2048;
    d += (uint32_t)(quarter * 32) << 16;
    const int columns = tile.columns();
    const auto plain = [&](int i) { return f + i < p.M ? f + i : -1; };
    float b[2][2] = {};   // bias of row lane / 4 + 8 i of the 16 rows h
    if (!kSum && p.bias != nullptr) {
        const uint16_t *q = p.bias + (int64_t)tile.e * (kGate ? 2 * p.M : p.M);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int at = f + (kGate ? 0 : 16 * h) + 8 * i + (lane >> 2);
                if (at < p.M) b[h][i] = widen16(__ldg(q + (kGate ? h * p.M : 0) + at));
            }
    }
    for (int c = 32 * half; c < columns; c += 32 * (kEpilogue / 4)) {
        const int there = tile.n - c < 32 ? tile.n - c : 32;
        const int64_t r0 = (MODE == kGradW ? (int64_t)tile.e * p.N : 0) + tile.row0 + c;   // the block's first row
        if (!kSum && p.residual != nullptr) {
            move_block<kPieces, false>(mine_ptr, const_cast<uint16_t *>(p.residual) + r0 * p.M, p.M, there, lane, p.wide, plain);
            __syncwarp();
        }
        uint32_t raw[2][16] = {};
        if (any) {
            tmem_ld_16x32(d + c, raw[0]);
            tmem_ld_16x32(d + c + (16u << 16), raw[1]);
            tmem_ld_wait();
        }
        float r[2][16];
#pragma unroll
        for (int j = 0; j < 32; ++j) r[j / 16][j % 16] = __uint_as_float(raw[j / 16][j % 16]);
        for (int i = 0; i < parts; ++i) {
            const float *q = part + (size_t)i * (part_bytes(p.nt) / 4) + part_index(c, quarter, lane);
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(q + 32 * j);
                float *to = &r[j / 16][j % 16];
                to[0] += v.x, to[1] += v.y, to[2] += v.z, to[3] += v.w;
            }
        }
        const int token = 8 * (lane >> 4) + (lane & 7), piece = (lane >> 3) & 1;   // this lane's address for (ld|st)matrix
        if (!kSum) {
#pragma unroll
            for (int j = 0; j < 32; ++j) r[j / 16][j % 16] += b[j / 16][(j >> 1) & 1];
            if (p.preact != nullptr && p.preact_wide) {
                // eight neighbours a row and register, 32 bytes: whole sectors as they are
                const int64_t ld = kGate ? 2 * p.M : p.M;
                float *q = static_cast<float *>(p.preact) + r0 * ld;
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const int row = 8 * ((j % 16) >> 2) + 2 * (lane & 3) + (j & 1);
                    const int at = f + (kGate ? 0 : 16 * (j / 16)) + 8 * ((j >> 1) & 1) + (lane >> 2);
                    if (row < there && at < p.M) q[row * ld + (kGate ? (j / 16) * p.M : 0) + at] = r[j / 16][j % 16];
                }
            } else if (p.preact != nullptr) {
                uint32_t keep[2][4][2] = {};   // the residual's block is in the same place
                if (p.residual != nullptr) {
#pragma unroll
                    for (int h = 0; h < (kGate ? 1 : 2); ++h)
#pragma unroll
                        for (int u = 0; u < 4; u += 2) ldmatrix_trans(mine + block_at(8 * u + token, 2 * h + piece), &keep[h][u][0]);
                    __syncwarp();
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int u = 0; u < 4; u += 2) {
                        uint32_t v[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[i] = cvt_bf16x2(r[h][4 * u + 2 * i], r[h][4 * u + 2 * i + 1]);
                        stmatrix_trans(mine + block_at(8 * u + token, 2 * h + piece), v);
                    }
                __syncwarp();
                const int64_t ld = kGate ? 2 * p.M : p.M;
                uint16_t *q = static_cast<uint16_t *>(p.preact) + r0 * ld;
                if (kGate)   // sixteen gate, sixteen up
                    move_block<4, true>(mine_ptr, q, ld, there, lane, p.wide, [&](int i) { return f + i % 16 < p.M ? i / 16 * p.M + f + i % 16 : -1; });
                else
                    move_block<4, true>(mine_ptr, q, ld, there, lane, p.wide, plain);
                __syncwarp();
                if (p.residual != nullptr) {
#pragma unroll
                    for (int h = 0; h < (kGate ? 1 : 2); ++h)
#pragma unroll
                        for (int u = 0; u < 4; u += 2) stmatrix_trans(mine + block_at(8 * u + token, 2 * h + piece), &keep[h][u][0]);
                    __syncwarp();
                }
            }
            if (kGate) {
#pragma unroll
                for (int j = 0; j < 16; ++j) r[0][j] = r[0][j] * sigmoid(r[0][j]) * r[1][j];
            } else if (p.act == CGL_ACT_RELU) {
#pragma unroll
                for (int j = 0; j < 32; ++j) r[j / 16][j % 16] = relu(r[j / 16][j % 16]);
            } else if (p.act == CGL_ACT_SILU) {
#pragma unroll
                for (int j = 0; j < 32; ++j) r[j / 16][j % 16] *= sigmoid(r[j / 16][j % 16]);
            } else if (p.act == CGL_ACT_GELU) {
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    float bell;
                    r[j / 16][j % 16] *= normal_cdf(r[j / 16][j % 16], bell);
                }
            }
            if (p.residual != nullptr) {
#pragma unroll
                for (int h = 0; h < (kGate ? 1 : 2); ++h)
#pragma unroll
                    for (int u = 0; u < 4; u += 2) {
                        uint32_t v[4];
                        ldmatrix_trans(mine + block_at(8 * u + token, 2 * h + piece), v);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            r[h][4 * u + 2 * i] += bf16_lo(v[i]);
                            r[h][4 * u + 2 * i + 1] += bf16_hi(v[i]);
                        }
                    }
                __syncwarp();
            }
        }
#pragma unroll
        for (int h = 0; h < (kGate ? 1 : 2); ++h)
#pragma unroll
            for (int u = 0; u < 4; u += 2) {
                uint32_t v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = cvt_bf16x2(r[h][4 * u + 2 * i], r[h][4 * u + 2 * i + 1]);
                stmatrix_trans(mine + block_at(8 * u + token, 2 * h + piece), v);
            }
        __syncwarp();
        move_block<kPieces, true>(mine_ptr, p.y + r0 * p.M, p.M, there, lane, p.wide, plain);
        __syncwarp();
    }
}

// ---- the kernel ------------------------------------------------------------------------------

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1)
matmul_bf16_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_y, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    // full and accfree count for the pair, in its first block; empty and accfull are told to both; tail is each block's own
    __shared__ uint64_t s_full[kMaxStages], s_empty[kMaxStages], s_tail[kMaxStages], s_accfull[2], s_accfree[2], s_drain;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort_word;
    volatile int *abort = &s_abort_word;

    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank(), lead = rank & ~1u;   // lead: the pair's first block
    const bool first = rank == lead;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *ring_ptr = smem_raw + (ring - smem_u32(smem_raw));
    const uint32_t out = ring + p.stages * p.stage_bytes;
    uint8_t *out_ptr = ring_ptr + (size_t)p.stages * p.stage_bytes;
    int32_t *tables = reinterpret_cast<int32_t *>(out_ptr + kOutBytes);

    if (warp == 0) {   // a lane each
        if (lane < p.stages) {
            bar_init(smem_u32(&s_full[lane]), MODE == kGradW ? 2 : 1);   // grad_w: a stage with a tail has an arrival of each block
            bar_init(smem_u32(&s_empty[lane]), 1);
            bar_init(smem_u32(&s_tail[lane]), 1);
        }
        if (lane < 2) {
            bar_init(smem_u32(&s_accfull[lane]), 1);
            bar_init(smem_u32(&s_accfree[lane]), 2 * kEpilogue);   // the epilogue warps of both blocks
        }
        if (lane == 0) {
            bar_init(smem_u32(&s_drain), 1);
            s_abort_word = 0;
            asm volatile("prefetch.tensormap [%0];" ::"l"(&map_x) : "memory");
            asm volatile("prefetch.tensormap [%0];" ::"l"(&map_y) : "memory");
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    griddep_wait();

    // tables: first[E + 1] (tiles of rows before each expert), row0[E], rows[E], rows a tile[E]
    const int ntiles = MODE == kGradW ? (p.N + p.nt - 1) / p.nt : 0;
    bool bad = false;
    for (int e = threadIdx.x; e < p.E; e += kThreads) {
        int r0, m;
        expert_rows(p.off, p.rows, p.cap, e, r0, m, bad);
        tables[p.E + 1 + e] = r0;
        tables[2 * p.E + 1 + e] = m;
        // rows of a tile: the expert's, in equal parts of at most nt, rounded up to 16
        const uint32_t parts = ((uint32_t)m + p.nt - 1) / p.nt;
        tables[3 * p.E + 1 + e] = parts > 0 ? (int)((((uint32_t)m + parts - 1) / parts + 15) & ~15u) : 0;
    }
    // bad offsets: no tiles at all, for the sums below hold only where rows do not overlap
    const bool refused = __syncthreads_or(bad) != 0;
    if (bad && blockIdx.x == 0) report(p.status, kErrRange);
    if (refused || MODE == kGradW) {
        for (int e = threadIdx.x; e <= p.E; e += kThreads) tables[e] = refused ? 0 : e * ntiles;
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

    Tiles<MODE> tile;
    bool done = false;
    if (warp == 0 || warp == 2) {
        int s = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (tile.start(p, tables); ok && tile.valid(); tile.next()) {
            const int half = tile.columns() / 2, box = MODE == kGradW ? 64 : p.box, boxes = (half + box - 1) / box;
            const uint32_t box_bytes = box * (kStageC * 2);
            const int row0 = tile.row0 + tile.rank * half;
            for (int k = tile.k0; k < tile.k1; ++k) {
                ok = __all_sync(0xFFFFFFFFu, bar_wait(smem_u32(&s_empty[s]), phase ^ 1, abort, p));
                if (!ok) break;
                const bool own = tile.tail_at(k) != 0;   // warp 3 of each block comes between
                const uint32_t base = ring + s * p.stage_bytes;
                const uint32_t bar = own ? in_block(smem_u32(&s_tail[s]), rank) : in_block(smem_u32(&s_full[s]), lead);
                if (elect_one()) {
                    if (warp == 0) {
                        const uint32_t bytes = kXBytes + boxes * box_bytes;
                        if (own) {
                            bar_expect(smem_u32(&s_tail[s]), bytes);
                        } else if (first) {
                            if (MODE == kGradW) bar_arrive_tmem(bar);
                            bar_expect(smem_u32(&s_full[s]), 2 * bytes);
                        }
                        const int x = k * kStageC;
                        if (MODE == kForward) {
                            tma_3d(base, &map_x, x, tile.f0, tile.e, bar);
                        } else if (MODE == kGated) {
#pragma unroll
                            for (int b = 0; b < 4; ++b) tma_4d(base + b * 4096, &map_x, x, tile.f0 + 16 * b, 0, tile.e, bar);
                        } else if (MODE == kGradA) {
#pragma unroll
                            for (int b = 0; b < 2; ++b) tma_3d(base + b * kChunkBytes, &map_x, tile.f0 + 64 * b, x, tile.e, bar);
                        } else {
#pragma unroll
                            for (int b = 0; b < 2; ++b) tma_2d(base + b * kChunkBytes, &map_x, tile.f0 + 64 * b, tile.c0 + x, bar);
                        }
                    } else {
                        for (int b = 0; b < boxes; ++b) {
                            if (MODE == kGradW) tma_2d(base + kXBytes + b * box_bytes, &map_y, row0 + b * box, tile.c0 + k * kStageC, bar);
                            else tma_2d(base + kXBytes + b * box_bytes, &map_y, k * kStageC, row0 + b * box, bar);
                        }
                    }
                }
                __syncwarp();
                if (++s == p.stages) s = 0, phase ^= 1;
            }
        }
        // Once more round the ring, a lane a place: the last releases are arrivals from
        // the first block, and a block must not leave before they have reached its barriers.
        if (ok && warp == 0 && lane < p.stages) bar_wait(smem_u32(&s_empty[lane]), lane < s ? phase : phase ^ 1, abort, p);
    } else if (warp == 1 && first) {
        // A stage's wait is asked for a stage ahead.
        const uint32_t full0 = smem_u32(&s_full[0]), empty0 = smem_u32(&s_empty[0]);
        const uint32_t stages = p.stages, stage_bytes = p.stage_bytes;
        uint32_t s = 0, base = ring, phase = 0;      // ring position
        uint32_t acc = 0, accphase = 0;
        bool ok = true, any = false, ready = false;
        for (tile.start(p, tables); ok && tile.valid(); tile.next()) {
            if (!tile.any()) continue;
            const uint32_t idesc = instr_desc<MODE>(tile.columns());
            ok = bar_wait(smem_u32(&s_accfree[acc]), accphase ^ 1, abort, p);
            const uint32_t d = tmem + acc * p.nt;
            for (int k = tile.k0; k < tile.k1; ++k) {
                if (!ready) ok = ok && bar_wait(full0 + 8 * s, phase, abort, p);
                tc_fence_after();
                const uint32_t empty = empty0 + 8 * s;
                const uint64_t dx = MODE == kForward || MODE == kGated ? desc_k(base) : desc_mn(base);
                const uint64_t dy = MODE == kGradW ? desc_mn(base + kXBytes) : desc_k(base + kXBytes);
                // 16 values of c an instruction: 32 bytes (two units) of each row, or 16 rows (128 units)
                constexpr uint64_t sx = MODE == kForward || MODE == kGated ? 2 : 128, sy = MODE == kGradW ? 128 : 2;
                const int tail = tile.tail_at(k);
                ++s, base += stage_bytes;
                if (s == stages) s = 0, base = ring, phase ^= 1;
                ready = bar_test(full0 + 8 * s, phase);
                fence_acquire_smem();
                if (elect_one() && ok) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (MODE != kGradW || tail == 0 || 16 * i < tail) mma_bf16(d, dx + sx * i, dy + sy * i, idesc, i > 0 || k > tile.k0);
                    mma_commit_both(empty, lead);
                }
            }
            if (elect_one() && ok) mma_commit_both(smem_u32(&s_accfull[acc]), lead);
            any = true;
            ok = __all_sync(0xFFFFFFFFu, ok);
            acc ^= 1;
            if (acc == 0) accphase ^= 1;
        }
        if (any) {   // every MMA has ended before TMEM is freed
            const uint32_t drain = smem_u32(&s_drain);
            __syncwarp();
            if (elect_one()) mma_commit(drain);
            __syncwarp();
            const long long start = clock64();
            while (!bar_try(drain, 0) && clock64() - start < kWaitCycles) {}
        }
    } else if (MODE == kGradW && warp == 3) {
        int s = 0;
        uint32_t phases = 0;   // of each place's tail barrier
        bool ok = true;
        for (tile.start(p, tables); ok && tile.valid(); tile.next()) {
            if (tile.tail != 0 && tile.any()) {
                const int at = (s + tile.k1 - 1 - tile.k0) % p.stages;
                ok = __all_sync(0xFFFFFFFFu, bar_wait(smem_u32(&s_tail[at]), (phases >> at) & 1, abort, p));
                if (!ok) break;
                phases ^= 1u << at;
                const int chunks = 2 + (tile.columns() / 2 + 63) / 64, c0 = tile.tail, rows = ((c0 + 15) & ~15) - c0;
                uint8_t *stage = ring_ptr + (size_t)at * p.stage_bytes;
                for (int i = lane; i < chunks * rows * 8; i += 32)
                    *reinterpret_cast<uint4 *>(stage + (i / (rows * 8)) * kChunkBytes + c0 * 128 + (i % (rows * 8)) * 16) = make_uint4(0, 0, 0, 0);
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) bar_arrive_smem(in_block(smem_u32(&s_full[at]), lead));
            }
            s = (s + tile.k1 - tile.k0) % p.stages;
        }
    } else if (warp >= 4) {
        int acc = 0;
        uint32_t accphase = 0;
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        for (tile.start(p, tables); tile.valid(); tile.next()) {
            const bool any = tile.any();
            done = !any || __all_sync(0xFFFFFFFFu, bar_wait(smem_u32(&s_accfull[acc]), accphase, abort, p));
            if (!done || p.split > 1) break;
            tc_fence_after();
            store_tile<MODE>(p, tile, any, tmem + acc * p.nt, quarter, half, lane, out, out_ptr, nullptr, 0);
            if (!any) continue;
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
        const bool epilogue = warp >= 4 && done;   // done: this pair's part of a tile is in TMEM, or it has none
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        if (epilogue && rank >= 2) {
            tc_fence_after();
            const uint32_t part = in_block(ring + (rank / 2 - 1) * part_bytes(p.nt), rank & 1);
            dump_tile<MODE>(tile, tile.any(), tmem, quarter, half, lane, part);
        }
        __syncwarp();
        cluster_sync();
        if (epilogue && rank < 2) {
            tc_fence_after();
            store_tile<MODE>(p, tile, tile.any(), tmem, quarter, half, lane, out, out_ptr, reinterpret_cast<const float *>(ring_ptr), p.split - 1);
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

// A BF16 array of `rank` dimensions, innermost first, strides in values from the second on; zeros outside.
bool make_map(CUtensorMap *map, const void *p, int rank, const int64_t *dims, const int64_t *strides, const int *box) {
    cuuint64_t d[4], s[4];
    cuuint32_t b[4], step[4] = {1, 1, 1, 1};
    for (int i = 0; i < rank; ++i) d[i] = (cuuint64_t)dims[i], b[i] = (cuuint32_t)box[i];
    for (int i = 1; i < rank; ++i) s[i - 1] = (cuuint64_t)strides[i - 1] * 2;
    const EncodeTiled fn = encode_tiled();
    return fn != nullptr && fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(p), d, s, b, step,
                               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How many clusters of `size` blocks run at once (0 on error); asked once for each size and kernel, with
// all the shared memory a block may have: these blocks come one to an SM whatever they take.
int clusters_at_once(const void *kernel, int size, size_t smem) {
    static std::mutex mu;
    static struct { const void *kernel; int device, size, n; } seen[64];
    static int count = 0;
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess || !ensure_smem_attr(kernel, smem)) return 0;
    std::lock_guard<std::mutex> lk(mu);
    for (int i = 0; i < count; ++i)
        if (seen[i].kernel == kernel && seen[i].device == device && seen[i].size == size) return seen[i].n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(size);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();   // not this launch's
        return 0;
    }
    if (count < 64) seen[count++] = {kernel, device, size, n};
    return n;
}

int pairs_of(int num_sms) {
    const int sms = device_sm_count(), n = (num_sms > 0 && num_sms < sms ? num_sms : sms) / 2;
    return n < 1 ? 1 : n;
}

// Shared memory for tiles of p.nt columns: the ring's stages, then the rest.
template <int MODE>
size_t lay_out(Params &p) {
    const size_t tables = (size_t)(4 * p.E + 1) * 4;
    const int y_rows = MODE == kGradW ? (p.nt / 2 + 63) / 64 * 64 : (p.nt / 2 + p.box - 1) / p.box * p.box;
    p.stage_bytes = kXBytes + y_rows * (kStageC * 2);
    const int stages = (int)((kSmemLimit - 1024 - kOutBytes - tables) / p.stage_bytes);
    p.stages = stages < kMaxStages ? stages : kMaxStages;
    return 1024 + (size_t)p.stages * p.stage_bytes + kOutBytes + tables;
}

int box_rows(int nt) { return nt > 128 ? 32 : nt > 64 ? 16 : 8; }

// Columns a tile and pairs that share one (p.nt, p.split), by what the call would take
// in cycles: waves of tiles, a stage of 512 cycles at 256 columns (the MMAs) and not
// below 370 (a block's 16 KiB of X from DRAM), 2000 and 10 a column for a tile's
// epilogue, 1500 and 40 a column for joining pairs' sums.  An expert's rows are cut into
// equal parts, so a tile's columns are those of its part (of the mean one; grad_w's
// tiles are whole) and a width is worth what it makes of the number of parts.  Narrow
// tiles read X more often, wide ones leave pairs without work: 2000 rows, 512 -> 512:
// 64 columns 9.5 us, 256 11.0; 2048 rows, 2048 -> 7168: 113 and 49; 16 experts of 256
// rows, 2048 -> 2048: 208 columns 60 us, 256 46.  Pairs share a tile where that leaves
// each four stages, all clusters run at once and the sums fit into the first pair's
// ring.  `guess` and `most`: tiles of rows of that many columns, as expected and at most;
// `exact`: the guess is right.  Where it may not be, a narrower width has to promise 3%:
// grad_a of 16 experts of 512 rows, 2048 -> 7168: 240 columns 254 us, 256 212.
template <int MODE, typename Guess, typename Most>
void plan(Params &p, int widest, int64_t mtiles, int64_t steps, int64_t rows, int64_t pairs, bool exact, Guess guess, Most most) {
    static const int widths[] = {32, 64, 96, 128, 160, 192, 208, 224, 240, 256};
    double best = 0;
    int nt = 0, split = 1;
    for (int i = 10; i >= 0; --i) {   // the widest first: of equals it stays
        p.nt = i == 10 ? widest : widths[i];
        if (i < 10 && p.nt >= widest) continue;
        if (MODE == kGradW && p.nt % 64 != 0) continue;   // 64 columns a chunk: others load as many
        if (MODE != kGradW) p.box = box_rows(p.nt);
        const double parts = (double)guess(p.nt), tiles = parts * mtiles;
        int part = p.nt;
        if (MODE != kGradW && rows <= parts * (p.nt - 16)) part = ((int)std::ceil(rows / parts) + 15) / 16 * 16;
        const double out = 2000 + 10 * part, stage = 2 * part > 370 + part / 2 ? 2 * part : 370 + part / 2;
        for (int k = 1; k <= 4; ++k) {
            if (k > 1 && (tiles * k > pairs || steps < 4 * k)) break;
            const double waves = k > 1 ? 1 : std::ceil(tiles / pairs), sums = ((steps + k - 1) / k) * stage;
            const double t = waves * (sums > out ? sums : out) + out + (k > 1 ? 1500 + 40 * part : 0);
            if (nt != 0 && t >= (exact || p.nt == nt ? best : 0.97 * best)) continue;
            if (k > 1) {
                const size_t smem = lay_out<MODE>(p);
                if (most(p.nt) * mtiles * k > pairs || (k - 1) * part_bytes(p.nt) > (uint32_t)p.stages * p.stage_bytes ||
                    most(p.nt) * mtiles > clusters_at_once((const void *)matmul_bf16_kernel<MODE>, 2 * k, smem))
                    break;
            }
            best = t, nt = p.nt, split = k;
        }
    }
    p.nt = nt, p.split = split;
    if (MODE != kGradW) p.box = box_rows(nt);
}

// The launch, for `most` tiles (at least as many as there are).
template <int MODE>
cgl_status launch(Params &p, const CUtensorMap &map_x, const CUtensorMap &map_y, int64_t most, int64_t pairs, cudaStream_t stream) {
    const auto kernel = matmul_bf16_kernel<MODE>;
    const size_t smem = lay_out<MODE>(p);
    if (!ensure_smem_attr((const void *)kernel, smem)) return CGL_ECUDA;
    if (pairs > most) pairs = most;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * pairs * p.split));
    cfg.blockDim = dim3(kThreads);
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
    return cudaLaunchKernelEx(&cfg, kernel, map_x, map_y, p) == cudaSuccess ? CGL_OK : CGL_ECUDA;
}

// The plan for a product whose rows are the experts' (sizes alone are known here); returns the most tiles there can be.
template <int MODE>
int64_t plan_rows(Params &p, const MatmulArgs &m, int64_t pairs) {
    // a quarter over the mean rows of an expert (a padded one's capacity), so that few experts need two tiles
    const int64_t mean = (m.rows + m.E - 1) / m.E, want = m.cap > 0 ? m.cap : m.off == nullptr || m.E == 1 ? mean : mean + mean / 4 + 8;
    const int widest = want >= kMaxNt ? kMaxNt : want <= 32 ? 32 : (int)((want + 15) / 16 * 16);
    const int64_t mtiles = (p.M + 2 * Tiles<MODE>::kFeatures - 1) / (2 * Tiles<MODE>::kFeatures), some = m.rows < m.E ? m.rows : m.E;
    const auto guess = [&](int nt) {
        if (m.cap > 0) return (double)m.E * ((m.cap + nt - 1) / nt);
        if (some == 1) return (double)((m.rows + nt - 1) / nt);
        // an expert's rows within an eighth of their mean, each number as likely: the mean of the tiles that takes
        const double mean = (double)m.rows / some / nt, a = mean * 0.875, b = mean * 1.125;
        const auto sum = [](double x) { const double n = std::floor(x); return n * (n + 1) / 2 + (x - n) * (n + 1); };   // of ceil, from 0 to x
        return some * (b <= 1 ? 1.0 : (sum(b) - sum(a)) / (b - a));
    };
    // with a row in each expert and the others in whole tiles
    const auto most = [&](int nt) { return some + (m.rows - some) / nt; };
    plan<MODE>(p, widest, mtiles, (p.C + kStageC - 1) / kStageC, m.cap > 0 ? m.E * m.cap : m.rows, pairs, m.cap > 0 || some == 1, guess, most);
    return most(p.nt) * mtiles;
}

Params params(const MatmulArgs &m) {
    Params p = {};
    p.off = m.off, p.status = m.status, p.rows = m.rows, p.cap = m.cap, p.E = m.E;
    p.N = 1, p.wait_cycles = m.wait_cycles < 0 || m.wait_cycles > kWaitCycles ? kWaitCycles : m.wait_cycles;
    return p;
}

bool rows_wide(const void *p, int64_t ld, int item) { return ld * item % 16 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

cgl_status launch_matmul_bf16(const MatmulArgs &m, const uint16_t *bias, const uint16_t *residual, uint16_t *y, void *preact,
                              bool preact_f32, cudaStream_t stream) {
    if (m.rows == 0) return CGL_OK;
    const bool gated = m.act == CGL_ACT_SWIGLU;
    Params p = params(m);
    p.bias = bias, p.residual = residual, p.y = y, p.preact = preact, p.preact_wide = preact_f32;
    p.act = m.act, p.M = gated ? m.F / 2 : m.F, p.C = m.K;
    const int64_t pairs = pairs_of(m.num_sms), most = gated ? plan_rows<kGated>(p, m, pairs) : plan_rows<kForward>(p, m, pairs);
    p.wide = rows_wide(y, p.M, 2) && rows_wide(residual, p.M, 2) && (preact_f32 || rows_wide(preact, p.M, 2));
    CUtensorMap map_x, map_y;
    const int64_t wd[4] = {m.K, p.M, gated ? 2 : m.E, m.E}, ws[3] = {m.K, (int64_t)p.M * m.K, (int64_t)m.F * m.K};
    const int wb[4] = {kStageC, gated ? 16 : kM, gated ? 2 : 1, 1};
    const int64_t ad[2] = {m.K, m.rows}, as[1] = {m.K};
    const int ab[2] = {kStageC, p.box};
    if (!make_map(&map_x, m.w, gated ? 4 : 3, wd, ws, wb) || !make_map(&map_y, m.a, 2, ad, as, ab)) return CGL_ECUDA;
    return gated ? launch<kGated>(p, map_x, map_y, most, pairs, stream) : launch<kForward>(p, map_x, map_y, most, pairs, stream);
}

cgl_status launch_matmul_bf16_backward(const MatmulArgs &m, const uint16_t *grad_y, const void *preact, bool preact_f32, uint16_t *grad_a,
                                       uint16_t *grad_w, uint16_t *grad_bias, void *ws, cudaStream_t stream) {
    const uint16_t *dz;
    int64_t ld;
    const cgl_status st = launch_slope(m, grad_y, preact, preact_f32, grad_a != nullptr || grad_w != nullptr, grad_bias, ws, &dz, &ld, stream);
    if (st != CGL_OK) return st;
    CUtensorMap map_x, map_y;
    const int64_t pairs = pairs_of(m.num_sms);
    if (grad_a != nullptr && m.rows > 0) {
        Params p = params(m);
        p.y = grad_a, p.M = m.K, p.C = m.F;
        const int64_t most = plan_rows<kGradA>(p, m, pairs);
        p.wide = 1;   // K % 8 == 0, grad_a 16-byte aligned
        const int64_t wd[3] = {m.K, m.F, m.E}, wst[2] = {m.K, (int64_t)m.F * m.K}, zd[2] = {m.F, m.rows};
        const int wb[3] = {64, kStageC, 1}, zb[2] = {kStageC, p.box};
        if (!make_map(&map_x, m.w, 3, wd, wst, wb) || !make_map(&map_y, dz, 2, zd, &ld, zb)) return CGL_ECUDA;
        const cgl_status r = launch<kGradA>(p, map_x, map_y, most, pairs, stream);
        if (r != CGL_OK) return r;
    }
    if (grad_w != nullptr) {
        Params p = params(m);
        p.y = grad_w, p.M = m.K, p.N = m.F;
        p.wide = 1;
        const int64_t mtiles = (m.K + 2 * kM - 1) / (2 * kM);
        const auto tiles = [&](int nt) { return (int64_t)m.E * ((m.F + nt - 1) / nt); };
        plan<kGradW>(p, kMaxNt, mtiles, (m.rows / m.E + kStageC - 1) / kStageC, 0, pairs, true, tiles, tiles);
        const int64_t rows = m.rows > 0 ? m.rows : 1;   // without rows nothing is loaded, and a map needs one
        const int64_t ad[2] = {m.K, rows}, as[1] = {m.K}, zd[2] = {m.F, rows};
        const int box[2] = {64, kStageC};
        if (!make_map(&map_x, m.rows > 0 ? m.a : m.w, 2, ad, as, box) || !make_map(&map_y, m.rows > 0 ? dz : m.w, 2, zd, &ld, box)) return CGL_ECUDA;
        return launch<kGradW>(p, map_x, map_y, tiles(p.nt) * mtiles, pairs, stream);
    }
    return CGL_OK;
}

}  // namespace cgl

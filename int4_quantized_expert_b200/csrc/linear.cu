// bf16 matrix products for the linear and grouped linear operators, on the
// 5th-generation tensor cores.
//
// One kernel computes, per matrix e (one expert, or the only matrix),
//   LIN_FWD  y[r][n]  = sum_k x[r][k] W[n][k]     (then bias, activation, residual)
//   LIN_DX   dx[r][k] = sum_n dy[r][n] W[n][k]
//   LIN_DW   dw[n][k] = sum_r dy[r][n] x[r][k]
// as D[lane][col] = sum_c A[lane][c] B[col][c]: the output feature that is
// contiguous in memory is the lane (M = 128) and the output row the column
// (up to 256), so a warp's stores run along rows of the output.  The
// contracted index c is contiguous in memory for both operands of LIN_FWD and
// for B of LIN_DX (K-major tiles); W of LIN_DX and both operands of LIN_DW
// have it as their row index and are fed as MN-major tiles straight from the
// same row-major matrices: no operand is transposed or copied beforehand.
//
// Tiles: 128 features x up to bn columns, steps of 64 along c, through a ring
// of TMA-filled slots (A 16 KB, B bn x 128 B, 128-byte swizzle).  D is fp32 in
// tensor memory, whose 512 columns are handed out in turn, so a tile's epilogue
// overlaps the next tile's MMAs.  TMA's zero fill pads c, features and rows at
// the tensors' edges; what it cannot pad is the end of an expert's rows inside the
// tensor when c runs over rows (LIN_DW): warp 2 zeroes those rows of both operands
// in the slot before the MMAs read it, so rows of the next expert -- which may
// hold NaN -- never enter.
//
// LIN_PAIR: two CTAs of a cluster share a tile of 256 features x up to 256
// columns.  Each loads its 128 features of A and its half of B's rows, and one
// thread of the pair issues MMAs over both.  A CTA alone moves 48 KB into and
// out of its shared memory for a step of 128 x 256 x 64, 768 cycles at 128
// bytes a cycle, against 512 cycles of MMAs; a CTA of a pair moves 32 KB for
// the same MMAs.
//
// An expert's rows are cut into equal chunks of at most bn rows (rounded up to
// 16, pairs: 32), not into full chunks and a tail: a tail of a few rows would
// stream a whole weight tile for them.  A pair's tile may have up to 320 rows, as
// two accumulators (192 columns and the rest) under one pass over the weights: 300
// rows in two tiles of 160 would load the weights twice, and the 64 bytes a cycle
// that an SM can load are what bounds narrow tiles.  Each CTA derives the list from
// the offsets by a scan over the (at most 256) experts.
//
// LIN_PAIR_SPLIT: where there are few such tiles, two to four pairs of a cluster
// share one's contraction, as in LIN_SPLIT below; their rings take the sums once all
// are past their MMAs.
//
// LIN_SPLIT: when there are few tiles, a CTA takes one of up to 128 columns, or a
// cluster of up to 8 CTAs shares the contraction of one of up to 192 and each
// finishes a part of the tile.  Partial sums are sent to the CTA that finishes them
// (st.async to its shared memory, counted by a barrier there; its own are plain
// stores) and added in rank order: no scratch, no atomics, the same bits every
// time.  Short calls are bound by latency or by the weights' bytes, so what counts
// is how soon a call's loads follow the last call's: where half of an SM's shared
// memory is enough, the next call's CTAs (programmatic dependent launch) are set up
// and waiting beside this one's.
//
// Without offsets, a CTA knows its weights before it has waited for the kernel
// before it, and asks for a ring's worth of them to be brought into L2.
//
// Warps: 0 TMA producer, 1 MMA issuer, 2 slot hand-over (LIN_DW: zeroes rows;
// LIN_PAIR: tells the MMA issuer's CTA that its own half has landed), 3
// tensor-memory allocation and tile scheduler, 4-11 epilogue.  The scheduler
// works out the tiles after a CTA's first, some 700 cycles of divisions and
// searches each, ahead of the other warps: loads and MMAs of full tiles take the
// same time, so what either loses between tiles is not made up again.  The single
// threads of warps 0 and 1 are picked by elect.sync and run their loops alone:
// under `lane == 0` a step's three loads took 708 cycles to issue, against the
// MMAs' 512, and with loops run by the whole warp on shuffled (uniform) values a
// step of loads and MMAs took 710; this way it takes 530.
#include <cuda.h>

#include <atomic>
#include <cstdint>
#include <type_traits>

#include "activation.cuh"
#include "linear.cuh"
#include "tcgen05.cuh"

namespace moe {

constexpr int LN_THREADS = 384;
constexpr int LN_EPI_WARPS = 8, LN_EPI_THREADS = 32 * LN_EPI_WARPS;
constexpr int LN_MAX_STAGES = 10;
constexpr int LN_TILES = 4;               // tiles scheduled ahead
constexpr int LN_ACCS = 4;                // accumulators in use at a time
constexpr int LN_SUB = 192;               // columns of the first accumulator of a tile of more than 256
constexpr int LN_MAX_E = 256;             // one thread per expert in the scan
constexpr int LN_A_BYTES = 128 * 64 * 2;  // 16 KB
constexpr int LN_RING_BYTES = 196608;     // the ring of a CTA that has an SM to itself
constexpr int LN_HALF_RING_BYTES = 109568;   // of one that shares it with another, with the sums it is sent
constexpr int LN_STG_BYTES = 32 * 64;     // an epilogue warp's staging buffer: 32 columns x 32 features, bf16

// What the kernels report (moe_linear_device_status): DEV_* values or-ed into one word per device.
static __device__ int32_t g_linear_status;

// What a query has taken from it.  Reading and clearing are one step: kernels of
// other streams report, and other threads query, at any time between two steps.
static __device__ int32_t g_linear_taken;
static __global__ void take_status_kernel() { g_linear_taken = atomicExch(&g_linear_status, DEV_OK); }

// How CTAs share tiles: one tile each, a cluster per tile along the contraction,
// two CTAs per tile of 256 features, or a cluster of pairs per such tile.
enum LinShare { LIN_ONE, LIN_SPLIT, LIN_PAIR, LIN_PAIR_SPLIT };
__host__ __device__ constexpr bool is_pair(int share) { return share == LIN_PAIR || share == LIN_PAIR_SPLIT; }
__host__ __device__ constexpr bool is_split(int share) { return share == LIN_SPLIT || share == LIN_PAIR_SPLIT; }

struct alignas(16) Tile {
    int e, f0;            // expert (-1: there is no tile), the CTA's first feature
    int col0, ncols;      // output rows (LIN_FWD, LIN_DX: rows; LIN_DW: n) of the tile
    int c0, k0, k1, clen; // contraction: first row (LIN_DW), steps [k0, k1), length
};

struct LinSmem {
    uint64_t full[LN_MAX_STAGES];    // TMA data of the slot landed (tx counted)
    uint64_t empty[LN_MAX_STAGES];   // the slot's MMAs completed
    uint64_t ready[LN_MAX_STAGES];   // LIN_DW, LIN_PAIR: warp 2 (of both CTAs) handed the slot over
    uint64_t drained;                // all MMAs of this CTA (pair) completed
    uint64_t acc_full[LN_ACCS];      // accumulator holds a finished tile
    uint64_t acc_empty[LN_ACCS];     // epilogue (of both CTAs) finished reading the accumulator
    uint64_t sums_full;              // LIN_SPLIT: all partial sums that are sent here have landed
    uint64_t tile_full[LN_TILES];    // the scheduler wrote the tile
    uint64_t tile_empty[LN_TILES];   // all that use it have read it
    Tile tiles[LN_TILES];
    uint32_t tmem_base;
    int32_t status;                  // of this CTA; joined into g_linear_status at the end
    int32_t first[LN_MAX_E + 1];     // chunks before each expert (LIN_FWD, LIN_DX)
    int32_t begin[LN_MAX_E];         // the expert's rows
    int32_t count[LN_MAX_E];
    int32_t warp_sum[LN_THREADS / 32];
};
// behind it, unless SPLIT: the epilogue warps' staging buffers
constexpr int LN_STG_OFFSET = (int(sizeof(LinSmem)) + 127) & ~127;
constexpr int LN_SMEM_BYTES = 1024 + LN_RING_BYTES + LN_STG_OFFSET + LN_EPI_WARPS * LN_STG_BYTES;
static_assert(LN_SMEM_BYTES <= 232448, "shared memory of a block");
static_assert(2 * (1024 + 1024 + LN_HALF_RING_BYTES + LN_STG_OFFSET) <= 233472, "two blocks on an SM");
constexpr int LN_FULL_RING_BYTES = 232448 - 1024 - LN_STG_OFFSET;   // of a split tile's CTA that has an SM to itself

// Shared-memory matrix descriptor of an MN-major tile with the 128-byte
// swizzle: rows of 64 values along M or N (128 bytes), one per c; 8 c are
// 1024 bytes, the next 64 values along M or N one box of 64 c (8192 bytes)
// further (leading byte offset).  16 c are 2048 bytes (+128 encoded).
__device__ __forceinline__ uint64_t sw128_desc_mn(uint32_t addr) {
    return uint64_t((addr >> 4) & 0x3FFFu) | (512ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// Whether an expert's two offsets are a range of the rows.
__device__ __forceinline__ bool in_order(int begin, int end, int rows) {
    return begin >= 0 && end >= begin && end <= rows;
}

// Chunks of an expert's rows.  Tiles of up to 320 rows save a pass over the
// weights where few chunks of up to 256 would be narrow.
__device__ __forceinline__ int row_chunks(int rows, int bn) {
    if (bn <= 256) return (rows + bn - 1) / bn;
    const int c = (rows + 255) >> 8, wide = (rows + 319) / 320;
    return c <= 4 ? wide : c;
}

// The columns of tensor memory of each accumulator in turn: wherever the last
// one ended, or from the start again.
struct AccColumns {
    int head = 0;
    __device__ __forceinline__ int next(int width) {
        const int first = head + width > 512 ? 0 : head;
        head = first + width;
        return first;
    }
};

template <int MODE, int SHARE>
__device__ __forceinline__ Tile get_tile(int tile, const LinSmem* sm, const LinParams& p, int rank) {
    // Expert by expert, so that its rows are in L2 for all of their tiles; within
    // an expert feature blocks in groups of 2048 features, chunk by chunk within a
    // group: the concurrent tiles of 148 CTAs then share 2048 features and 9 row
    // chunks.
    constexpr bool PAIR = is_pair(SHARE), SPLIT = is_split(SHARE);
    Tile t;
    int n, before;                         // the expert's chunks (LIN_DW: column blocks), those before it
    const int unit = tile / p.n_fblocks;   // not the tile's chunk, but one of its expert's
    if (MODE == LIN_DW) {
        n = (p.NC + p.bn - 1) / p.bn;
        t.e = unit / n;
        before = t.e * n;
    } else {
        int lo = 0, hi = p.E;              // the last expert whose first chunk is <= unit
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (sm->first[mid] <= unit) lo = mid; else hi = mid;
        }
        t.e = lo;
        before = sm->first[lo];
        n = sm->first[lo + 1] - before;
    }
    const int gf = min(PAIR ? 8 : 16, p.n_fblocks);
    const int in_e = tile - before * p.n_fblocks, g = in_e / (n * gf), r = in_e - g * n * gf;
    const int gsize = min(gf, p.n_fblocks - g * gf), i = r / gsize, fb = g * gf + (r - i * gsize);
    t.f0 = 128 * (PAIR ? 2 * fb + (rank & 1) : fb);
    if (MODE == LIN_DW) {
        t.col0 = i * p.bn;
        t.ncols = min(p.bn, p.NC - t.col0);
        t.c0 = sm->begin[t.e];
        t.clen = sm->count[t.e];
    } else {
        const int cnt = sm->count[t.e];
        const int align = PAIR ? 31 : 15;   // of the MMA's N
        const int size = ((cnt + n - 1) / n + align) & ~align;
        t.col0 = sm->begin[t.e] + i * size;
        t.ncols = min(size, cnt - i * size);
        t.c0 = 0;
        t.clen = p.C;
    }
    const int nk = (t.clen + 63) >> 6;
    const int part = PAIR ? rank >> 1 : rank;
    t.k0 = SPLIT ? nk * part / p.split : 0;
    t.k1 = SPLIT ? nk * (part + 1) / p.split : nk;
    return t;
}

// Eight neighbouring features of one output row (LIN_SPLIT): bias, pre-activation,
// activation, residual, rounding, store.  idx: of the first one in the output.
template <int MODE>
__device__ __forceinline__ void finish8(const LinParams& p, int64_t idx, float (&v)[8], const uint4& bias,
                                        const uint4& res) {   // bias, res: read where p has them
    if (MODE == LIN_FWD) {
        if (p.bias) {
            float t[8];
            unpack8(bias, t);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += t[i];
        }
        if (p.preact) *reinterpret_cast<uint4*>(p.preact + idx) = pack8(v);
        act_values(p.act, v);
        if (p.residual) {
            float t[8];
            unpack8(res, t);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += t[i];
        }
    }
    if (p.out_fp32) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + idx);
        o[0] = make_float4(v[0], v[1], v[2], v[3]);
        o[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<bf16*>(p.out) + idx) = pack8(v);
    }
}

// 32 lanes x 32 columns of an accumulator as fragments (tmem_ld_frag): v[h] has
// the lanes 16 h .. 16 h + 15.
__device__ __forceinline__ void tmem_ld_block(uint32_t taddr, uint32_t (&v)[2][16]) {
    tmem_ld_frag(taddr, v[0]);
    tmem_ld_frag(taddr + (16u << 16), v[1]);
}

// The same of a block of 32 features (from f0) x up to ncols columns, output
// rows row .., held as fragments.  Rows of the output are stored and rows of
// the residual loaded as 16-byte pieces, four lanes to a row; between these and
// the fragments they are transposed by stmatrix / ldmatrix through the warp's
// staging buffer of 64-byte rows (piece q of row r at q ^ (r / 2 % 4): the eight
// rows of a matrix, and the two rows that eight lanes read, take distinct
// banks).  Against 4-byte shared-memory stores of the fp32 values and 32-byte
// loads this is a third of the shared-memory traffic.
template <int MODE>
__device__ __forceinline__ void finish_block(const LinParams& p, float (&a)[2][16], int64_t row, int ncols, int f0,
                                             uint32_t stage, int lane) {
    const int f = f0 + 8 * (lane & 3);          // this lane's piece of rows 8 i + lane / 4
    const int rl = lane >> 2;
    const bool fok = f < p.F;                   // F is a multiple of 8
    const uint32_t piece = stage + rl * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);                // + 512 i
    const uint32_t mat = stage + (lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4);         // + 512 i
    // two columns of one feature in a register: what row t / 4 (+ 8 b + 16 h) of
    // the fragments has at columns 8 i + 2 (t % 4) and + 1
    auto store_rows = [&](bf16* out) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t m[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                m[q] = pack_bf16x2(a[q >> 1][4 * i + 2 * (q & 1)], a[q >> 1][4 * i + 2 * (q & 1) + 1]);
            st_matrix4_t(mat + 512 * i, m);
        }
        __syncwarp();
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = ld_shared_v4_at(piece + 512 * i);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (fok && 8 * i + rl < ncols) *reinterpret_cast<uint4*>(out + (row + 8 * i + rl) * p.F + f) = v[i];
    };
    uint4 res[4];
    if (MODE == LIN_FWD) {
        if (p.residual) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                res[i] = make_uint4(0, 0, 0, 0);
                if (fok && 8 * i + rl < ncols)
                    res[i] = *reinterpret_cast<const uint4*>(p.residual + (row + 8 * i + rl) * p.F + f);
            }
        }
        if (p.bias) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int fq = f0 + 8 * q + rl;
                const float b = fq < p.F ? __bfloat162float(p.bias[fq]) : 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[q >> 1][4 * i + 2 * (q & 1)] += b;
                    a[q >> 1][4 * i + 2 * (q & 1) + 1] += b;
                }
            }
        }
        if (p.preact) store_rows(p.preact);
        act_values(p.act, a[0]);
        act_values(p.act, a[1]);
        if (p.residual) {
#pragma unroll
            for (int i = 0; i < 4; ++i) st_shared_v4_at(piece + 512 * i, res[i]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t m[4];
                ld_matrix4_t(mat + 512 * i, m);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    a[q >> 1][4 * i + 2 * (q & 1)] += bf16_lo(m[q]);
                    a[q >> 1][4 * i + 2 * (q & 1) + 1] += bf16_hi(m[q]);
                }
            }
            __syncwarp();
        }
    }
    if (!p.out_fp32) {
        store_rows(static_cast<bf16*>(p.out));
        return;
    }
    // eight lanes hold the 32 bytes of eight features of a column
    float* out = static_cast<float*>(p.out) + row * p.F + f0 + rl;
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int c = 8 * i + 2 * (lane & 3) + j;
                if (f0 + 8 * q < p.F && c < ncols)
                    out[int64_t(c) * p.F + 8 * q] = a[q >> 1][4 * i + 2 * (q & 1) + j];
            }
}

template <int MODE, int SHARE>
__global__ void __launch_bounds__(LN_THREADS, SHARE == LIN_SPLIT ? 2 : 1) linear_kernel(const __grid_constant__ CUtensorMap tm_a,
                                                               const __grid_constant__ CUtensorMap tm_b, LinParams p) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* base = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    LinSmem* sm = reinterpret_cast<LinSmem*>(base + p.ring_bytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr bool A_MN = MODE != LIN_FWD, B_MN = MODE == LIN_DW;
    constexpr bool PAIR = is_pair(SHARE), SPLIT = is_split(SHARE);
    constexpr bool HAND_OVER = PAIR || MODE == LIN_DW;
    const int stage_bytes = LN_A_BYTES + (PAIR ? p.bn / 2 : p.bn) * 128;
    uint32_t rank = 0;
    if (SHARE != LIN_ONE) asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    // of a pair: the CTA's half of the features, the rank of the one that issues the
    // MMAs, both as a mask; the CTA's (pair's) part of a split contraction
    const uint32_t half = PAIR ? rank & 1 : 0, lead = rank & ~1u, both_ctas = 3u << lead, part = PAIR ? rank >> 1 : rank;
    const bool leader = half == 0;

    griddep_launch_dependents();
    if (warp == 0) {
        if (lane < LN_MAX_STAGES) {
            mbar_init(&sm->full[lane], 1);
            mbar_init(&sm->empty[lane], 1);
            mbar_init(&sm->ready[lane], PAIR ? 2 : 1);
            if (lane < LN_TILES) {   // read by warps 0, 1 (where it issues), 2 (where it hands over) and the epilogue's
                mbar_init(&sm->tile_full[lane], 1);
                mbar_init(&sm->tile_empty[lane], 1 + leader + HAND_OVER + LN_EPI_WARPS);
            }
        } else if (lane < LN_MAX_STAGES + LN_ACCS) {
            mbar_init(&sm->acc_full[lane - LN_MAX_STAGES], 1);
            mbar_init(&sm->acc_empty[lane - LN_MAX_STAGES], PAIR ? 2 * LN_EPI_WARPS : LN_EPI_WARPS);
        } else if (lane == LN_MAX_STAGES + LN_ACCS) {
            mbar_init(&sm->drained, 1);
            mbar_init(&sm->sums_full, 1 + LN_EPI_WARPS);   // the bytes that others send; this CTA's own epilogue warps
            sm->status = DEV_OK;
        } else if (lane == LN_MAX_STAGES + LN_ACCS + 1) {
            prefetch_tmap(&tm_a);
            prefetch_tmap(&tm_b);
        }
        fence_barrier_init();
    }
    if (warp == 3) {
        tmem_alloc<PAIR>(&sm->tmem_base, p.tmem_cols);
        tmem_relinquish<PAIR>();
    }
    if (p.offsets) griddep_wait();

    // the row ranges, and for LIN_FWD / LIN_DX the chunks before each expert
    int chunks = 0;
    bool bad = false;
    if (int(threadIdx.x) < p.E) {
        int b = 0, c = p.rows;
        if (p.offsets) {
            b = p.offsets[threadIdx.x];
            const int end = p.offsets[threadIdx.x + 1];
            if (in_order(b, end, p.rows)) {
                c = end - b;
            } else {
                b = c = 0;
                bad = true;
                if (blockIdx.x == 0) atomicOr(&g_linear_status, DEV_BAD_EXPERT);
            }
        }
        sm->begin[threadIdx.x] = b;
        sm->count[threadIdx.x] = c;
        chunks = p.offsets ? row_chunks(c, p.bn) : p.chunks;
    }
    if (MODE != LIN_DW) {
        int incl = chunks;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) sm->warp_sum[warp] = incl;
        __syncthreads();
        int before = 0;
        for (int i = 0; i < warp; ++i) before += sm->warp_sum[i];
        if (int(threadIdx.x) < p.E) {
            sm->first[threadIdx.x + 1] = before + incl;
            if (threadIdx.x == 0) sm->first[0] = 0;
        }
    }
    tc_fence_before();
    // Where two offsets are out of order, ranges that are in order by themselves may
    // overlap.  Those that overlap an earlier one count as empty too: a grid of split
    // tiles has room for the chunks of ranges that are apart and no more.
    if (__syncthreads_or(bad)) {
        if (int(threadIdx.x) < p.E) {
            const int b = sm->begin[threadIdx.x], end = b + sm->count[threadIdx.x];
            bool overlaps = false;
            for (int i = 0; i < int(threadIdx.x) && !overlaps; ++i) {
                const int bi = p.offsets[i], ei = p.offsets[i + 1];
                overlaps = in_order(bi, ei, p.rows) && max(b, bi) < min(end, ei);
            }
            if (overlaps) {
                sm->count[threadIdx.x] = 0;
                if (blockIdx.x == 0) atomicOr(&g_linear_status, DEV_BAD_EXPERT);
            }
        }
        __syncthreads();
        if (MODE != LIN_DW && threadIdx.x == 0)
            for (int e = 0; e < p.E; ++e) sm->first[e + 1] = sm->first[e] + row_chunks(sm->count[e], p.bn);
        __syncthreads();
    }
    // the other CTAs' barriers are initialized (a pair's allocations done)
    if (PAIR || (SPLIT && p.split > 1)) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = sm->tmem_base;
    const int n_units = MODE == LIN_DW ? p.E * ((p.NC + p.bn - 1) / p.bn) : sm->first[p.E];
    const int n_tiles = n_units * p.n_fblocks;
    const int tile0 = int(blockIdx.x) / ((PAIR ? 2 : 1) * (SPLIT ? p.split : 1));
    const int tstep = PAIR ? int(gridDim.x) / 2 : int(gridDim.x);
    // the accumulators of a tile: MMA's N, and the rows of B (the columns of D)
    // that this CTA loads
    constexpr bool WIDE = SHARE == LIN_PAIR && MODE != LIN_DW;
    auto subs = [](const Tile& t) { return WIDE && t.ncols > 256 ? 2 : 1; };
    auto sub_cols = [&](const Tile& t, int i) { return subs(t) == 1 ? t.ncols : i == 0 ? LN_SUB : t.ncols - LN_SUB; };
    auto mma_n = [](int ncols) { return PAIR ? (ncols + 31) & ~31 : (ncols + 15) & ~15; };
    auto b_rows = [&](int ncols) { return PAIR ? mma_n(ncols) / 2 : ncols; };
    auto b_boxes = [&](int ncols) { return (b_rows(ncols) + p.box - 1) / p.box; };

    // the CTA's first tile is worked out by every warp, the others come from the scheduler
    Tile t = {-1};
    if (tile0 < n_tiles) t = get_tile<MODE, SHARE>(tile0, sm, p, rank);
    uint32_t tiles_read = 0;
    auto advance = [&](bool whole_warp) {
        if (SPLIT) {
            t.e = -1;
            return;
        }
        const uint32_t i = tiles_read % LN_TILES;
        if (mbar_wait(&sm->tile_full[i], (tiles_read / LN_TILES) & 1, &sm->status)) t = sm->tiles[i];
        else t.e = -1;
        ++tiles_read;
        if (whole_warp) __syncwarp();
        if (!whole_warp || lane == 0) mbar_arrive(&sm->tile_empty[i]);
    };

    auto out_row = [&](const Tile& t) { return MODE == LIN_DW ? int64_t(t.e) * p.NC + t.col0 : int64_t(t.col0); };

    // SPLIT: a unit is eight features and four columns of the tile; each CTA
    // finishes `units` of them in a row (the last ones fewer).  Sums lie in
    // [sender][unit][feature, turned by the unit][4 columns]: 16-byte pieces that
    // the eight units a warp reads at a time have in different banks.
    const int64_t split_row = SPLIT ? out_row(t) : 0;
    const int n_sums = (t.ncols + 3) / 4 * 16, units = (n_sums + p.split - 1) / p.split;
    const int my_units = max(0, min(units, n_sums - int(part) * units));
    unsigned char* sums_at = !PAIR && p.split > 1 ? reinterpret_cast<unsigned char*>(sm) + LN_STG_OFFSET : base;
    // A thread finishes eight features of a column at a time, LN_EPI_THREADS / 4
    // units apart: its features stay the same.  The bias and the first residual are
    // loaded under the sums, each next residual under the piece before.
    const int i0 = int(threadIdx.x) - 128;
    const int split_f = t.f0 + 8 * ((int(part) * units + (i0 >> 2)) & 15);
    auto split_col = [&](int i) { return 4 * ((int(part) * units + (i >> 2)) >> 4) + (i & 3); };
    uint4 bias0 = make_uint4(0, 0, 0, 0), res0 = bias0;
    auto load_residual = [&](int i) {
        if (MODE == LIN_FWD && p.residual && i < 4 * my_units && split_col(i) < t.ncols && split_f < p.F)
            res0 = *reinterpret_cast<const uint4*>(p.residual + (split_row + split_col(i)) * p.F + split_f);
    };
    if (!p.offsets) {
        if (MODE != LIN_DW && warp == 0 && t.e >= 0 && elect_one()) {
            for (int kk = t.k0; kk < t.k1 && kk < t.k0 + p.stages; ++kk) {
                if (MODE == LIN_FWD) {
                    tma_prefetch_3d(&tm_a, kk * 64, t.f0, t.e);
                } else {
                    tma_prefetch_3d(&tm_a, t.f0, kk * 64, t.e);
                    tma_prefetch_3d(&tm_a, t.f0 + 64, kk * 64, t.e);
                }
            }
        }
        __syncwarp();
        griddep_wait();
    }

    if (warp == 0) {
        // ------------------------------ TMA producer ------------------------------
        if (elect_one()) {
            uint32_t slot = 0, par = 1, filled = 0;
            bool ok = true;
            for (; t.e >= 0 && ok; advance(false)) {
                const int n0 = sub_cols(t, 0), n1 = subs(t) > 1 ? t.ncols - n0 : 0;
                const int boxes0 = b_boxes(n0), boxes = boxes0 + (WIDE ? b_boxes(n1) : 0);
                const int row = t.col0 + int(half) * b_rows(n0);
                const int row1 = t.col0 + n0 + int(half) * b_rows(n1) - boxes0 * p.box;   // so box i is at row1 + i * p.box
                const int box_bytes = p.box * 128;
                const uint32_t bytes = LN_A_BYTES + boxes * box_bytes;
                for (int kk = t.k0; kk < t.k1; ++kk) {
                    if (!mbar_wait(&sm->empty[slot], par, &sm->status)) { ok = false; break; }
                    unsigned char* sa = base + slot * stage_bytes;
                    unsigned char* sb = sa + LN_A_BYTES;
                    uint64_t* bar = &sm->full[slot];
                    const int c = t.c0 + kk * 64;
                    mbar_arrive_expect_tx(bar, bytes);
                    if (MODE == LIN_FWD) {
                        tma_load_3d(sa, &tm_a, bar, c, t.f0, t.e);
                    } else if (MODE == LIN_DX) {
                        tma_load_3d(sa, &tm_a, bar, t.f0, c, t.e);
                        tma_load_3d(sa + 8192, &tm_a, bar, t.f0 + 64, c, t.e);
                    } else {
                        tma_load_2d(sa, &tm_a, bar, t.f0, c);
                        tma_load_2d(sa + 8192, &tm_a, bar, t.f0 + 64, c);
                    }
                    for (int i = 0; i < boxes; ++i) {
                        if (B_MN) tma_load_2d(sb + i * 8192, &tm_b, bar, row + i * 64, c);
                        else tma_load_2d(sb + i * box_bytes, &tm_b, bar, c, (!WIDE || i < boxes0 ? row : row1) + i * p.box);
                    }
                    ++filled;
                    if (++slot == uint32_t(p.stages)) { slot = 0; par ^= 1; }
                }
            }
            // wind down: wait (bounded) for the loads still in flight to land
            for (uint32_t i = 0; i < uint32_t(p.stages) && i < filled; ++i) {
                const uint32_t j = filled - 1 - i;
                mbar_wait(&sm->full[j % p.stages], (j / p.stages) & 1, nullptr);
            }
        }
    } else if (warp == 1) {
        // ------------------------------ MMA issuer ------------------------------
        if (leader && elect_one()) {
            uint32_t slot = 0, par = 0, n = 0, done = 0;   // accumulators begun; known to be free again
            uint32_t held = 0;                             // columns of the last four: first / 32 and width / 32 - 1
            AccColumns cols;
            bool ok = true;
            const uint32_t idesc_m = tc_idesc_fmt(PAIR ? 256 : 128, 0, 1u) | (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u);
            // the columns of the next accumulator, once they are free: the one
            // that had its barrier before and all that had these columns are read
            auto take = [&](int nn) {
                const int width = (nn + 31) & ~31, first = cols.next(width);
                uint32_t need = n >= LN_ACCS ? n - LN_ACCS + 1 : 0;
                for (uint32_t j = max(done, need); j < n; ++j) {
                    const uint32_t h = held >> (8 * (j % LN_ACCS));
                    const int hf = 32 * (h & 15), hw = 32 * ((h >> 4 & 15) + 1);
                    if (first < hf + hw && hf < first + width) need = j + 1;
                }
                for (; done < need && ok; ++done)
                    ok = mbar_wait(&sm->acc_empty[done % LN_ACCS], (done / LN_ACCS) & 1, &sm->status);
                const int at = 8 * (n % LN_ACCS);
                held = (held & ~(255u << at)) | uint32_t((first >> 5) | ((width >> 5) - 1) << 4) << at;
                ++n;
                return tmem + first;
            };
            // the steps of a tile, with one or two accumulators
            auto steps = [&](auto two, uint32_t d0, uint32_t idesc0, uint32_t d1, uint32_t idesc1) {
                for (int kk = t.k0; kk < t.k1; ++kk) {
                    if (!mbar_wait(HAND_OVER ? &sm->ready[slot] : &sm->full[slot], par, &sm->status)) return false;
                    const int left = t.clen - kk * 64;
                    // the peer's zeroes: this wait acquires at CTA scope only
                    if (PAIR && MODE == LIN_DW && left < 64) asm volatile("fence.acq_rel.cluster;" ::: "memory");
                    tc_fence_after();
                    const unsigned char* sa = base + slot * stage_bytes;
                    const uint64_t ad = A_MN ? sw128_desc_mn(smem_u32(sa)) : sw128_desc(sa);
                    const uint64_t bd = B_MN ? sw128_desc_mn(smem_u32(sa + LN_A_BYTES)) : sw128_desc(sa + LN_A_BYTES);
#pragma unroll
                    for (int k16 = 0; k16 < 4; ++k16)
                        if (k16 * 16 < left) {
                            const uint64_t a = ad + (A_MN ? 128 : 2) * k16, b = bd + (B_MN ? 128 : 2) * k16;
                            const uint32_t accumulate = kk != t.k0 || k16 != 0;
                            if (PAIR) umma_pair(d0, a, b, idesc0, accumulate);
                            else umma<false>(d0, a, b, idesc0, accumulate);
                            if (decltype(two)::value) umma_pair(d1, a, b + (LN_SUB / 2 * 128 >> 4), idesc1, accumulate);
                        }
                    if (PAIR) umma_commit_pair(&sm->empty[slot], both_ctas);
                    else umma_commit(&sm->empty[slot]);
                    if (++slot == uint32_t(p.stages)) { slot = 0; par ^= 1; }
                }
                return true;
            };
            for (; t.e >= 0 && ok; advance(false)) {
                if (t.k0 >= t.k1) continue;   // nothing to contract: the epilogue writes zeros
                const int n0 = mma_n(sub_cols(t, 0)), n1 = subs(t) > 1 ? mma_n(sub_cols(t, 1)) : 0;
                const uint32_t idesc0 = idesc_m | uint32_t(n0 >> 3) << 17, idesc1 = idesc_m | uint32_t(n1 >> 3) << 17;
                const uint32_t d0 = take(n0), d1 = WIDE && n1 ? take(n1) : 0;
                if (!ok) break;
                tc_fence_after();
                if (WIDE && n1) ok = steps(std::true_type{}, d0, idesc0, d1, idesc1);
                else ok = steps(std::false_type{}, d0, idesc0, 0, 0);
                if (!ok) break;
                if (WIDE && n1) umma_commit_pair(&sm->acc_full[(n - 2) % LN_ACCS], both_ctas);
                if (PAIR) umma_commit_pair(&sm->acc_full[(n - 1) % LN_ACCS], both_ctas);
                else umma_commit(&sm->acc_full[(n - 1) % LN_ACCS]);
            }
            // wind down: wait (bounded) for the last MMAs
            if (PAIR) umma_commit_pair(&sm->drained, both_ctas);
            else umma_commit(&sm->drained);
            mbar_wait(&sm->drained, 0, nullptr);
        }
    } else if (warp == 2 && HAND_OVER) {
        // ---------------- hand the slots over to the MMA issuer ----------------
        uint32_t slot = 0, par = 0;
        bool ok = true;
        for (; t.e >= 0 && ok; advance(true)) {
            const int boxes = b_boxes(t.ncols);   // LIN_DW
            for (int kk = t.k0; kk < t.k1; ++kk) {
                if (!mbar_wait(&sm->full[slot], par, &sm->status)) { ok = false; break; }
                const int left = t.clen - kk * 64;
                const bool ragged = MODE == LIN_DW && left < 64 && (left & 15);
                if (ragged) {
                    // zero the rows past the expert's end.  A box is 64 rows of
                    // 128 bytes; the swizzle moves 16-byte chunks within a row
                    // only.  The MMAs read up to the next multiple of 16 rows.
                    unsigned char* sa = base + slot * stage_bytes;
                    const int chunks16 = ((16 - (left & 15)) * 128) / 16;
                    for (int b = 0; b < 2 + boxes; ++b)
                        for (int i = lane; i < chunks16; i += 32)
                            st_shared_v4(sa + b * 8192 + left * 128 + i * 16, make_uint4(0, 0, 0, 0));
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) {
                    if (PAIR && ragged) mbar_arrive_at<true>(&sm->ready[slot], lead);
                    else if (PAIR) mbar_arrive_at(&sm->ready[slot], lead);
                    else mbar_arrive(&sm->ready[slot]);
                }
                if (++slot == uint32_t(p.stages)) { slot = 0; par ^= 1; }
            }
        }
    } else if (warp == 3 && !SPLIT) {
        // ------------------------------ tile scheduler ------------------------------
        if (lane == 0 && tile0 < n_tiles) {
            int tile = tile0;
            for (uint32_t i = 0; tile < n_tiles; ++i) {
                tile += tstep;
                Tile next = {-1};
                if (tile < n_tiles) next = get_tile<MODE, SHARE>(tile, sm, p, rank);
                if (!mbar_wait(&sm->tile_empty[i % LN_TILES], ((i / LN_TILES) & 1) ^ 1, &sm->status)) break;
                sm->tiles[i % LN_TILES] = next;
                mbar_arrive(&sm->tile_full[i % LN_TILES]);
            }
        }
    } else if (warp >= 4) {
        // ------------------------------ epilogue ------------------------------
        const int ew = warp & 3;                 // TMEM lanes 32 ew .. 32 ew + 31
        const uint32_t stage = smem_u32(sm) + LN_STG_OFFSET + (warp - 4) * LN_STG_BYTES;
        uint32_t n = 0;
        AccColumns cols;
        for (bool ok = true; t.e >= 0 && ok; advance(true)) {
            const bool any = t.k0 < t.k1;
            const int64_t row0 = out_row(t);
            if (SPLIT) {
                if (threadIdx.x == 128) mbar_arrive_expect_tx(&sm->sums_full, (p.split - 1) * my_units * 128);
                if (MODE == LIN_FWD && p.bias && split_f < p.F) bias0 = *reinterpret_cast<const uint4*>(p.bias + split_f);
                load_residual(i0);
                bool got = any;
                if (any) {
                    got = mbar_wait(&sm->acc_full[0], 0, &sm->status);
                    tc_fence_after();
                }
                // pairs' sums reuse the rings: every pair is past its loads and MMAs
                if (PAIR) { __syncwarp(); cluster_sync(); }
                // 16-byte pieces of one feature and four columns, also after a
                // wait that gave up: the others count on them
                const uint32_t sums = smem_u32(sums_at);
                for (int cc = (warp - 4) >> 2; cc * 32 < t.ncols; cc += 2) {
                    uint32_t v[32];
                    if (got) {
                        tmem_ld32(tmem + (uint32_t(32 * ew) << 16) + cc * 32, v);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = 0u;
                    }
                    const int u = cc * 128 + 4 * ew + (lane >> 3);
                    int owner = u / units, at = u - owner * units;
#pragma unroll
                    for (int g = 0; g < 8; ++g) {
                        if (cc * 32 + 4 * g < t.ncols) {
                            const uint32_t to = sums + ((part * units + at) * 8 + ((lane + at) & 7)) * 16;
                            if (owner == int(part))
                                st_shared_v4_at(to, make_uint4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]));
                            else
                                st_async_v4(to, PAIR ? 2 * owner + half : owner, &sm->sums_full, v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
                        }
                        at += 16;
                        while (at >= units) { at -= units; ++owner; }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->sums_full);
                break;     // a split tile is its cluster's only one
            }
            for (int sub = 0; sub < subs(t); ++sub) {
                const int ncols = sub_cols(t, sub);
                const int64_t row = row0 + (sub ? LN_SUB : 0);
                uint32_t taddr = tmem + (uint32_t(32 * ew) << 16);
                if (any) {
                    taddr += cols.next((mma_n(ncols) + 31) & ~31);
                    if (!mbar_wait(&sm->acc_full[n % LN_ACCS], (n / LN_ACCS) & 1, &sm->status)) { ok = false; break; }
                    tc_fence_after();
                }
                // every other 32 columns for each of the two warps of these lanes
                auto release = [&] {
                    tc_fence_before();
                    __syncwarp();
                    if (any && lane == 0) {
                        if (PAIR) mbar_arrive_at(&sm->acc_empty[n % LN_ACCS], lead);
                        else mbar_arrive(&sm->acc_empty[n % LN_ACCS]);
                    }
                };
                const int nb = (ncols + 31) >> 5;
                int cc = (warp - 4) >> 2;
                uint32_t v[2][16];
                if (cc >= nb) release();
                else if (any) tmem_ld_block(taddr + cc * 32, v);
                for (; cc < nb; cc += 2) {
                    float a[2][16];
                    if (any) tmem_wait_ld(v);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int j = 0; j < 16; ++j) a[h][j] = any ? __uint_as_float(v[h][j]) : 0.0f;
                    // the next block's load runs under this block's arithmetic and
                    // stores; after the last one the accumulator is free
                    if (cc + 2 >= nb) release();
                    else if (any) tmem_ld_block(taddr + cc * 32 + 64, v);
                    finish_block<MODE>(p, a, row + cc * 32, ncols - cc * 32, t.f0 + ew * 32, stage, lane);
                }
                if (any) ++n;
            }
        }
    }
    bool landed = true;
    if (SPLIT) {
        __syncwarp();
        if (PAIR && (warp < 4 || t.e < 0)) cluster_sync();
        if (!PAIR && p.split > 1) cluster_arrive();   // this CTA has sent what it sends
        if (warp >= 4 && t.e >= 0) {
            landed = mbar_wait(&sm->sums_full, 0, &sm->status);
            for (int i = i0; i < 4 * my_units; i += LN_EPI_THREADS) {
                const uint4 res = res0;
                load_residual(i + LN_EPI_THREADS);
                const int at = i >> 2;
                uint32_t q = smem_u32(sums_at) + at * 128 + (i & 3) * 4;
                float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
                for (int s = 0; s < p.split; ++s, q += units * 128)
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] += ld_shared_f32_at(q + ((j + at) & 7) * 16);
                if (split_col(i) < t.ncols && split_f < p.F)
                    finish8<MODE>(p, (split_row + split_col(i)) * p.F + split_f, v, bias0, res);
            }
        }
        __syncwarp();
        if (!PAIR && p.split > 1) cluster_wait();
    }
    if (PAIR) {
        __syncwarp();
        cluster_sync();                          // the pair's MMAs and remote arrivals are over
        // ... and the last commit, which arrives in both CTAs, has arrived here
        if (threadIdx.x == 32) mbar_wait(&sm->drained, 0, nullptr);
    }
    // a wait that gave up: all has been sent, and lands before this CTA leaves
    if (SPLIT && !landed) mbar_wait(&sm->sums_full, 0, nullptr);
    tc_fence_before();
    __syncthreads();
    if (warp == 3) {
        tc_fence_after();
        tmem_dealloc<PAIR>(tmem, p.tmem_cols);
    }
    if (threadIdx.x == 0 && sm->status != DEV_OK) atomicOr(&g_linear_status, sm->status);
}

// ---------------------------------------------------------------------------
// dz = dy * act'(z) and dbias = sum over the rows of dz (unrounded)
//
// dz is rounded to bf16 for the products that read it, whose operands are bf16
// (dy of a layer without activation has that type too); dbias takes it before.
//
// HBM-bound: dy and z are read once, dz is written once, the column sums ride
// along.  A cluster of AG_SPLIT CTAs takes a strip of AG_COLS columns: 8 threads
// x 16 bytes a row (one 128-byte line), 32 rows at a time, each CTA a part of
// the rows.  A thread sums its rows in fp32, the CTA its row lanes and the
// cluster its CTAs in a fixed order.  4099 x 5120 with GELU: 24 us, 5.2 TB/s;
// strips of 32 and 128 columns, 512 threads and two or eight rows in flight a
// thread all took 28 to 37 us.  Five CTAs to an SM (48 registers) run these 640 at
// once; left to itself the compiler takes 64 registers, and the last 48 CTAs run
// alone: 33 us.
// ---------------------------------------------------------------------------
constexpr int AG_THREADS = 256, AG_SPLIT = 8, AG_COLS = 64, AG_ROWS = AG_THREADS * 8 / AG_COLS;

template <bool DZ, bool DB>
__global__ void __launch_bounds__(AG_THREADS, 5) act_grad_kernel(const bf16* __restrict__ dy,
                                                                 const bf16* __restrict__ z, int T, int N, int act,
                                                                 bf16* __restrict__ dz, void* __restrict__ dbias,
                                                                 int dbias_fp32) {
    __shared__ float part[AG_ROWS][AG_COLS + 1];
    __shared__ float sums[AG_COLS];
    griddep_launch_dependents();
    griddep_wait();
    const int split = blockIdx.x % AG_SPLIT, n0 = int(blockIdx.x / AG_SPLIT) * AG_COLS;
    const int c8 = threadIdx.x % (AG_COLS / 8), rl = threadIdx.x / (AG_COLS / 8);
    const int col = n0 + 8 * c8;
    const int r0 = int(int64_t(T) * split / AG_SPLIT), r1 = int(int64_t(T) * (split + 1) / AG_SPLIT);
    float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (col < N) {   // N is a multiple of 8
#pragma unroll 4
        for (int r = r0 + rl; r < r1; r += AG_ROWS) {
            const int64_t idx = int64_t(r) * N + col;
            float v[8];
            unpack8(*reinterpret_cast<const uint4*>(dy + idx), v);
            if (DZ) {
                float zv[8];
                unpack8(*reinterpret_cast<const uint4*>(z + idx), zv);
                act_slopes(act, v, zv);
                if (dz) *reinterpret_cast<uint4*>(dz + idx) = pack8(v);
            }
            if (DB)
#pragma unroll
                for (int i = 0; i < 8; ++i) s[i] += v[i];
        }
    }
    if (!DB) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) part[rl][8 * c8 + i] = s[i];
    __syncthreads();
    if (threadIdx.x < AG_COLS) {
        float t = 0.0f;
        for (int i = 0; i < AG_ROWS; ++i) t += part[i][threadIdx.x];
        sums[threadIdx.x] = t;
    }
    cluster_sync();
    const int n = n0 + int(threadIdx.x);
    if (split == 0 && threadIdx.x < AG_COLS && n < N) {
        float t = 0.0f;
        for (int i = 0; i < AG_SPLIT; ++i) t += ld_dsmem_f32(&sums[threadIdx.x], i);
        if (dbias_fp32) static_cast<float*>(dbias)[n] = t;
        else static_cast<bf16*>(dbias)[n] = __float2bfloat16_rn(t);
    }
    cluster_sync();
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            ptr = nullptr;
        return reinterpret_cast<EncodeTiledFn>(ptr);
    }();
    return fn;
}

// bf16 [mats, rows, inner] (mats = 0: 2-D [rows, inner]), boxes of 64 values x
// box_rows rows with the 128-byte swizzle; reads past an edge give zeros.
bool make_map(CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t rows, uint64_t mats, uint32_t box_rows) {
    const EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {inner, rows, mats};
    const cuuint64_t strides[2] = {inner * 2, inner * rows * 2};
    const cuuint32_t box[3] = {64, box_rows, 1}, step[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, mats ? 3 : 2, const_cast<void*>(ptr), dims, strides, box, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

moe_status sm_count(int* sms) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return MOE_ERR_CUDA;
    return MOE_OK;
}

template <typename... KArgs, typename... Args>
moe_status launch_cluster(void (*kernel)(KArgs...), unsigned grid, unsigned block, size_t smem, unsigned cluster,
                          cudaStream_t stream, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...));
}

// Chunks of all rows for pairs: the fewest that take the least time, counted as
// rounds of tiles over the pairs times the cycles of a step, which are those of
// the MMAs (2 a column) or of the loads (128 rows of A and half of the columns,
// 64 bytes a cycle), whichever are more, and at least 480 (a step's latencies).
// A tile of more than 256 leaves the tensor cores idle for about 5000 cycles at
// its end, until its first accumulator has been read.
int pair_chunks(int rows, int n_fblocks, int steps, int pairs) {
    const int least = int(ceil_div(rows, 320)), most = int(ceil_div(rows, 256)) + 8;
    int best = least;
    int64_t best_time = INT64_MAX;
    for (int c = least; c <= most; ++c) {
        const int n = (int(ceil_div(rows, c)) + 31) & ~31;
        if ((c - 1) * n >= rows) continue;   // no chunk may be empty
        const int64_t tile = int64_t(steps) * (n > 256 ? 2 * n : n < 224 ? 480 : n + 256) + (n > 256 ? 5000 : 0);
        const int64_t time = ceil_div(int64_t(c) * n_fblocks, pairs) * tile;
        if (time < best_time) best = c, best_time = time;
    }
    return best;
}

// Shared memory of a split tile's CTA: its ring and, with more than one CTA, the
// sums that it is sent; half of an SM's for tiles of up to 64 columns.
struct SplitSmem {
    int stages, ring, total;
    SplitSmem(int bn, int split) {
        const int stage = LN_A_BYTES + bn * 128, sums = split > 1 ? split * ((4 * bn + split - 1) / split) * 128 : 0;
        stages = ((bn <= 64 ? LN_HALF_RING_BYTES : LN_FULL_RING_BYTES) - sums) / stage;
        if (stages > LN_MAX_STAGES) stages = LN_MAX_STAGES;
        ring = stages * stage;
        if (split == 1 && ring < bn * 512) ring = bn * 512;   // a tile's own sums reuse the ring
        total = 1024 + ring + LN_STG_OFFSET + sums;
    }
};

// The clusters of `split` CTAs that a device holds at once, one CTA to an SM: 33 of
// 4 on 148 SMs, because a cluster stays within a GPC.  0 if it cannot be found out.
int max_clusters(int split) {
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices][9];   // + 1
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= kDevices) return 0;
    const int have = known[dev][split].load(std::memory_order_relaxed);
    if (have) return have - 1;
    auto kernel = linear_kernel<LIN_FWD, LIN_SPLIT>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(split));
    cfg.blockDim = dim3(LN_THREADS);
    cfg.dynamicSmemBytes = size_t(SplitSmem(128, split).total);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(split);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (allow_max_smem(kernel) != MOE_OK || cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) return 0;
    known[dev][split].store(n + 1, std::memory_order_relaxed);
    return n;
}

// How a call's tiles are shared out, by an estimate of the cycles it takes.  A tile's
// steps take their loads (64 bytes a cycle for an SM) or MMAs, whichever take
// longer, and at least 480 each; its epilogue takes 20 cycles a column and more
// with activation, residual or pre-activations, and 50 more through the sums of
// LIN_SPLIT, over its CTAs.  Rounds of tiles over the SMs take
// the longer of the two, all loops at least what the weights take from HBM at 3400
// bytes a cycle (an eighth more where no SM has two CTAs: one to an SM, they end
// 10 % apart; 16 x 5120 -> 16384 takes 32.2 us in 128 CTAs and 28.9 in 256); then
// come the last epilogue and what a kernel costs before and after.  The constants
// were measured on 64 to 16384 features and contractions of 64 to 16384.
template <int MODE>
moe_status launch_mode(const bf16* a, const bf16* b, int32_t N, int32_t K, LinParams p, int sms, cudaStream_t stream) {
    constexpr bool DW = MODE == LIN_DW;
    const int experts = p.E < p.rows ? p.E : p.rows;
    const int per_expert = int(ceil_div(p.rows, p.E)), steps = int(ceil_div(DW ? per_expert : p.C, 64));
    const int fb = int(ceil_div(p.F, 128)), fb2 = int(ceil_div(p.F, 256));
    // chunks of all rows (LIN_DW: blocks of all columns), at most
    auto units = [&](int bn) {
        return DW ? int64_t(p.E) * ceil_div(N, bn) : p.offsets ? int64_t(p.rows) / bn + experts : ceil_div(p.rows, bn);
    };
    // columns that a tile may have: as many as there are, or as an expert has rows
    // on average -- and not below 64 then, since many rows of one expert in narrow
    // tiles would stream its weights through every SM again and again
    const int cols = DW ? N : !p.offsets || p.rows <= 64 ? p.rows : per_expert > 64 ? per_expert : 64;

    int share = LIN_ONE, pair_split_chunks = 0;
    p.bn = DW || cols > 32 ? (cols <= 64 ? 64 : cols <= 128 ? 128 : 256) : cols <= 16 ? 16 : 32;
    p.split = 1;
    const int64_t hbm = DW ? 0 : int64_t(p.offsets ? experts : 1) * N * K * 2 / 3400;
    auto loop = [&](int64_t cycles, bool shared_sms) {
        const int64_t least = shared_sms ? hbm : hbm + hbm / 8;
        return cycles > least ? cycles : least;
    };
    const int column = 20 + (p.preact ? 10 : 0) + (p.residual ? 10 : 0) + (p.act == MOE_ACT_GELU ? 16 : p.act ? 8 : 0);
    auto rounds = [&](int64_t n, int64_t tile_loop, int64_t epilogue) {
        return loop(n * (tile_loop > epilogue ? tile_loop : epilogue), false) + epilogue;
    };
    int64_t best = rounds(ceil_div(units(p.bn) * fb, sms), steps * int64_t(p.bn < 112 ? 480 : 256 + 2 * p.bn),
                          column * p.bn) + 4000;
    // (experts of fewer rows on average too: some have more)
    if (cols > (p.offsets && !DW ? 64 : 128)) {
        p.chunks = DW || p.offsets ? 0 : pair_chunks(p.rows, fb2, steps, sms / 2);
        const int64_t n = p.chunks ? p.chunks : units(256), width = p.chunks ? (ceil_div(p.rows, p.chunks) + 31) & ~31 : 256;
        const int64_t step = width > 256 ? 2 * width : width < 224 || cols < 224 ? 480 : 256 + width;
        const int64_t time = rounds(ceil_div(n * fb2, sms / 2), steps * step, column * width) + 4500;
        if (time < best) best = time, share = LIN_PAIR;
    }
    if (cols > 128 && !p.offsets) {
        const int least = int(ceil_div(DW ? N : p.rows, 256));
        for (int c = least; c <= (DW ? least : least + 2); ++c) {
            const int width = DW ? 256 : int(ceil_div(p.rows, c) + 31) & ~31;
            if (!DW && (c - 1) * width >= p.rows) continue;   // no chunk may be empty
            for (int q = 2; q <= 4 && q <= steps; ++q) {
                if (max_clusters(2 * q) < c * fb2) break;
                const int64_t time = loop(ceil_div(steps, q) * (width < 224 ? 480 : 256 + width), false) +
                                     (column + 50 / q) * width + 6000 + 300 * q;
                if (time < best) best = time, share = LIN_PAIR_SPLIT, p.split = q, pair_split_chunks = c;
            }
        }
    }
    for (int bn = DW || (p.offsets && p.rows > 64) ? 64 : 16; bn <= 192; bn += DW ? 64 : 16) {
        const int64_t all = units(bn) * fb;
        if (all > 8 * sms) {
            if (bn >= cols) break;
            continue;
        }
        const int tiles = int(all);
        // as many CTAs to a tile as two to an SM or one to an SM allow, or one;
        // wider than 128, a tile that is not split is a pair's or another kernel's
        for (int per_sm = bn <= 64 ? 2 : 1, last = 0; tiles <= sms && per_sm >= 0; --per_sm) {
            int s = per_sm ? per_sm * sms / tiles : 1;
            if (s > 8) s = 8;
            if (s > steps) s = steps;
            while (s > 1 && (bn <= 64 ? 2 : 1) * max_clusters(s) < tiles) --s;
            if (s == last || (s == 1 && bn > 128)) continue;
            last = s;
            const bool shared_sms = s * tiles > sms;
            const int load = (shared_sms ? 2 : 1) * (256 + 2 * bn);
            const int64_t time = loop(int64_t((steps + s - 1) / s) * (load < 480 ? 480 : load), shared_sms) +
                                 (column + 50 / s) * bn + (s > 1 ? 5000 + 150 * s : 2500);
            if (time < best) best = time, share = LIN_SPLIT, p.bn = bn, p.split = s;
        }
        // more tiles than SMs, two CTAs to an SM: one's epilogue under the other's loads
        if (bn <= 64 && tiles > sms) {
            const int load = 2 * (256 + 2 * bn);
            const int64_t time = loop((tiles + 2 * sms - 1) / (2 * sms) * (int64_t(steps) * (load < 480 ? 480 : load) + (column + 50) * bn + 2500),
                                      true) + 2500;
            if (time < best) best = time, share = LIN_SPLIT, p.bn = bn, p.split = 1;
        }
        if (bn >= cols) break;
    }

    int64_t n_units = units(p.bn);
    int smem = LN_SMEM_BYTES, cluster = 1, stage = LN_A_BYTES + p.bn * 128;
    if (share == LIN_PAIR_SPLIT) {
        cluster = 2 * p.split;
        p.bn = 256;
        p.chunks = pair_split_chunks;
        n_units = p.chunks;
        stage = LN_A_BYTES + p.bn / 2 * 128;
    } else if (share == LIN_PAIR) {
        cluster = 2;
        p.bn = 256;
        n_units = units(256);
        if (!DW && p.offsets) p.bn = 320;
        if (!DW && !p.offsets) {
            n_units = p.chunks;
            if (ceil_div(p.rows, p.chunks) > 256) p.bn = 320;
        }
        stage = LN_A_BYTES + p.bn / 2 * 128;
    } else {
        p.chunks = int(ceil_div(p.rows, p.bn));
    }
    if (share == LIN_SPLIT) {
        const SplitSmem sizes(p.bn, p.split);
        cluster = p.split;
        p.stages = sizes.stages;
        p.ring_bytes = sizes.ring;
        smem = sizes.total;
        p.tmem_cols = p.bn <= 32 ? 32 : p.bn <= 64 ? 64 : p.bn <= 128 ? 128 : 256;
    } else {
        p.stages = LN_RING_BYTES / stage < LN_MAX_STAGES ? LN_RING_BYTES / stage : LN_MAX_STAGES;
        p.ring_bytes = p.stages * stage;
        p.tmem_cols = 512;
    }
    p.n_fblocks = is_pair(share) ? fb2 : fb;
    p.box = DW ? 64 : is_pair(share) ? 32 : share == LIN_SPLIT || p.bn < 64 ? p.bn : 64;

    CUtensorMap ta, tb;
    const bool ok = DW ? make_map(&ta, a, K, p.rows, 0, 64) && make_map(&tb, b, N, p.rows, 0, 64)
                       : make_map(&ta, a, K, N, p.E, MODE == LIN_FWD ? 128 : 64) &&
                             make_map(&tb, b, p.C, p.rows, 0, p.box);
    if (!ok) return MOE_ERR_CUDA;
    auto kernel = share == LIN_PAIR         ? linear_kernel<MODE, LIN_PAIR>
                  : share == LIN_PAIR_SPLIT ? linear_kernel<MODE, LIN_PAIR_SPLIT>
                  : share == LIN_SPLIT      ? linear_kernel<MODE, LIN_SPLIT>
                                            : linear_kernel<MODE, LIN_ONE>;
    if (allow_max_smem(kernel) != MOE_OK || prefer_smem(kernel) != MOE_OK) return MOE_ERR_CUDA;
    const int64_t tiles = n_units * p.n_fblocks;
    const int64_t grid = is_split(share) ? tiles : tiles < sms / cluster ? tiles : sms / cluster;
    return launch_cluster(kernel, unsigned(grid * cluster), LN_THREADS, size_t(smem), unsigned(cluster), stream, ta, tb, p);
}

}  // namespace

moe_status launch_linear(int mode, const bf16* a, const bf16* b, int32_t N, int32_t K, LinParams p,
                         cudaStream_t stream) {
    if (p.rows == 0) return MOE_OK;
    int sms = 148;
    if (sm_count(&sms) != MOE_OK) return MOE_ERR_CUDA;
    p.F = mode == LIN_FWD ? N : K;
    p.C = mode == LIN_FWD ? K : N;
    p.NC = N;
    if (mode == LIN_FWD) return launch_mode<LIN_FWD>(a, b, N, K, p, sms, stream);
    if (mode == LIN_DX) return launch_mode<LIN_DX>(a, b, N, K, p, sms, stream);
    return launch_mode<LIN_DW>(a, b, N, K, p, sms, stream);
}

moe_status launch_act_grad(const bf16* dy, const bf16* z, int32_t T, int32_t N, int32_t act, bf16* dz, void* dbias,
                           int32_t dbias_fp32, cudaStream_t stream) {
    const unsigned grid = unsigned(ceil_div(N, AG_COLS) * AG_SPLIT);
    if (z && dbias)
        return launch_cluster(act_grad_kernel<true, true>, grid, AG_THREADS, 0, AG_SPLIT, stream, dy, z, T, N, act, dz,
                              dbias, dbias_fp32);
    if (z)
        return launch_cluster(act_grad_kernel<true, false>, grid, AG_THREADS, 0, AG_SPLIT, stream, dy, z, T, N, act,
                              dz, dbias, dbias_fp32);
    return launch_cluster(act_grad_kernel<false, true>, grid, AG_THREADS, 0, AG_SPLIT, stream, dy, z, T, N, act, dz,
                          dbias, dbias_fp32);
}

moe_status set_wait_limit_linear(uint32_t cycles) {
    return cuda_status(cudaMemcpyToSymbol(c_wait_limit, &cycles, sizeof(cycles)));
}

moe_status linear_device_status(cudaStream_t stream) {
    static std::mutex mu;   // g_linear_taken belongs to one query at a time
    if (cudaStreamSynchronize(stream) != cudaSuccess) return MOE_ERR_CUDA;   // not under the lock
    std::lock_guard<std::mutex> lock(mu);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = cfg.blockDim = dim3(1);
    cfg.stream = stream;
    int32_t v = 0;
    // this launch's own result: an error that some call before left behind must not cost a report
    if (cudaLaunchKernelEx(&cfg, take_status_kernel) != cudaSuccess ||
        cudaMemcpyFromSymbolAsync(&v, g_linear_taken, sizeof(v), 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
        cudaStreamSynchronize(stream) != cudaSuccess)
        return MOE_ERR_CUDA;
    if (v == DEV_OK) return MOE_OK;
    return v & DEV_TIMEOUT ? MOE_ERR_TIMEOUT : MOE_ERR_INVALID_ARG;
}

}  // namespace moe

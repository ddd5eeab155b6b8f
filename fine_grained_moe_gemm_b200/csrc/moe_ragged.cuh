// Matrix products grouped by expert with ragged sizes, on CTA pairs.
//
// Rows sorted by group; off[g] .. off[g+1] are group g's rows.  Three products:
//   RAG_NT  y[r, n]     = sum_k x[r, k] w[g(r), n, k]      (w as nn.Linear keeps it)
//   RAG_NN  y[r, n]     = sum_k x[r, k] w[g(r), k, n]      (the input gradient, same w)
//   RAG_TN  dw[g, n, k] = sum_{r in g} dy[r, n] x[r, k]    (the weight gradient)
// in 16-bit types with fp32 sums, and RAG_NT in 8-bit integers with exact 32-bit sums
// and one scale per row and per output channel.
//
// Tiling.  The output's feature axis n is M of the tensor-core tile (256 per CTA
// pair, 128 per SM), the ragged row axis (TN: the k axis) is N, up to 256 wide.  A
// group's rows then cost MMA width only in steps of 32, where rows as M would pad
// every group to 128 or 256 of them.  A group of more than P.bn rows (256, or 128 where
// the product has too few tiles for every SM) is cut into equal chunks.  Each SM loads
// its own 128 features and half of the chunk's rows.  An accumulator is 256 TMEM columns,
// so two fit: the epilogue of one item overlaps the products of the next.
//
// NN and TN read operands whose summed axis is the row axis of memory: their tiles
// are MN-major in shared memory (64 elements of the free axis by 64 of the summed
// one per 8 KB block).  TN sums over a group's rows, which end inside a 64-row block:
// a warp zeroes the rows behind the group's last in both tiles before the MMA may
// read them (zero in one only would keep a NaN of the next group).
//
// Nothing is scheduled on the host: every CTA builds the groups' item counts in
// shared memory from the offsets and walks the items with the stride of the grid.
//
// Measured (B200).  8192^3, one group: bf16 750 us (tensor pipe 98 % active, 1.24 GHz
// under the power cap), int8 340 us.  256 groups of 4 rows, 7168 -> 2048: 1142 us, HBM at
// 99 % of the copy rate.  32768 rows in 256 groups, gradients of 2048 x 7168 in bf16: 2089
// us, bound by storing 7.5 GB.
#pragma once

#include <cuda_fp16.h>

#include "moe_gemm2.cuh"

namespace moe {

constexpr int RAG_SLOT = 128 * 128;       // half of a stage: 128 features (rows) x 128 bytes of the summed axis
constexpr int RAG_TN_BLOCK = 64 * 128;    // one 64 x 64 block of an MN-major tile
// Warps: 0 and 1 load A, 2 loads B (a thread issues one TMA instruction every few hundred
// cycles whatever its size, and a block of 64 is consumed in about 700), 4 issues the MMAs,
// 5 zeroes TN's tail rows, 8-15 are the epilogue (3, 6 and 7 fill up their warpgroups).
// Every loading warp has bytes in every block: one that only followed the others could fall
// two rounds of the ring behind, and a wait for a phase of a barrier that is two phases
// further never ends.
constexpr int RAG_EPI_WARP0 = 8;
constexpr int RAG_EPI_WARPS = 8;
constexpr int RAG_THREADS = (RAG_EPI_WARP0 + RAG_EPI_WARPS) * 32;
constexpr int RAG_BAND = 8;               // chunks whose items run together (L2)

// The tensor core cuts each partial sum off instead of rounding it: after every 16 terms a sum
// loses up to 2^-23 of its value, always towards zero, so m terms of one sign come out small by up
// to m * 2^-27 (measured: 6.4e-9 m, 6.7e-3 at 2^20 terms; terms of both signs about a sixth).
// With PROMOTE the tensor core sums RAG_SEGMENT terms at a time and the epilogue adds the
// segments in fp32 registers, rounding to nearest.  fp32 results take such segments always.  A 16-bit
// one needs them only where the loss could pass an eighth of its half step, and then as long as that
// (RAG_LONG: P.whole blocks).  With segments of 512 terms an f16 product of 4096 x 4096 x 18432 took
// 479 us, with these or none 474; with segments for every 16-bit sum gradients of 32768 rows in 256
// groups, 2048 x 7168 in bf16, took 2700 us in place of 2100.
constexpr int RAG_SEGMENT = 512;
// The segments' sums take 128 registers of an epilogue thread, so PROMOTE (and an int8
// product, whose scales and next item go along: 2 % on short sums) moves
// registers from warps 0-7 to warps 8-15: 256 x 56 + 256 x 200 = 512 x 128, the
// registers that the CTA was launched with (launch_ragged checks that it was).
constexpr int RAG_REGS_LAUNCH = 128, RAG_REGS_CONTROL = 56, RAG_REGS_EPILOGUE = 200;

template <int DIR>
struct RagCfg {
    // a staging tile of the epilogue, per warp: 32 rows of 64 (NT, NN) or 128 bytes
    static constexpr int STAGING = DIR == RAG_TN ? 4096 : 2048;
    static constexpr int SCALES = DIR == RAG_NT ? 512 : 0;  // int8: the scales of four chunks of 32 rows, per warp
    static constexpr int STAGES = DIR == RAG_TN ? 5 : 6;
    static constexpr int RING = STAGES * 2 * RAG_SLOT;
    static constexpr int TABLE = 3 * RAG_MAX_GROUPS * 4 + 16;  // first row, rows, first item of each group
    static constexpr int BARS = 2 * STAGES + (DIR == RAG_TN ? 2 * STAGES : 0) + 5;
    static constexpr int MISC = (BARS * 8 + (3 + RAG_THREADS / 32) * 4 + 15) / 16 * 16;
    static constexpr int SMEM_BYTES = 1024 + RING + RAG_EPI_WARPS * (STAGING + SCALES) + TABLE + MISC;
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory of one CTA");
};

// One unit of work of a CTA pair.
struct RagItem {
    int g;        // group
    int m;        // 256-feature tile
    int row0;     // first row (TN: the group's first row)
    int rows;     // rows of the chunk (TN: rows of the group, the summed length)
    int col0;     // TN: first column of dw
    int width;    // valid columns of the tile: rows of the chunk (TN: columns of dw)
    int chunks;   // chunks of the group that read the same weights
};

struct RagTable {
    int* start;   // [groups] first row
    int* count;   // [groups] rows
    int* first;   // [groups + 1] first item
};

// Chunks of a group of `rows` rows (TN: column tiles of its dw), and its items.
template <int DIR>
__device__ __forceinline__ int rag_chunks(const RaggedArgs& P, int rows) {
    return ((DIR == RAG_TN ? P.k : rows) + P.bn - 1) >> P.bn_shift;
}
template <int DIR>
__device__ __forceinline__ int rag_items_of(const RaggedArgs& P, int rows) {
    return ((P.n + 255) >> 8) * rag_chunks<DIR>(P, rows);
}

// Fills the table from the offsets (all THREADS threads of the CTA; the caller
// synchronises).  A group whose offsets decrease or leave [0, rows], or that starts before an
// earlier group's end, has no rows and sets MOE_DEVERR_BAD_ROWS: groups never share rows, so no
// two tiles store the same ones and the rows of all groups are at most `rows`, which bounds the
// tiles that the host launches for.  Groups that share rows have a decrease between them, so
// offsets without a bad group of their own need no more than the first look; else one thread
// goes through them all.
// `head` is what rag_first_offsets loaded: the caller does so before everything else, as the
// loads' latency is most of what a CTA waits for before its first tile.
__device__ __forceinline__ int2 rag_first_offsets(const RaggedArgs& P) {
    const int tid = threadIdx.x;
    return P.offsets && tid < P.groups ? make_int2(__ldg(P.offsets + tid), __ldg(P.offsets + tid + 1)) : make_int2(0, P.rows);
}

template <int THREADS, typename ItemsOf>
__device__ __forceinline__ void rag_build_table(const RaggedArgs& P, const RagTable& t, int* warp_sums, int2 head,
                                                ItemsOf items_of) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (P.groups + THREADS - 1) / THREADS;  // consecutive groups of a thread
    const int g0 = tid * per;
    int sum = 0;
    bool bad = false;
    for (int g = g0; g < min(g0 + per, P.groups); ++g) {
        int a = head.x, b = head.y;  // per == 1: the thread's group
        if (per > 1) {
            a = __ldg(P.offsets + g);
            b = __ldg(P.offsets + g + 1);
        }
        if (a < 0 || b < a || b > P.rows) {
            bad = true;
            a = b = 0;
        }
        t.start[g] = a;
        t.count[g] = b - a;
        t.first[g] = sum;  // within the thread, for now
        sum += items_of(b - a);
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sums[warp] = incl;
    if (__syncthreads_or(bad)) {
        if (tid != 0) return;
        if (blockIdx.x == 0) set_dev_error(MOE_DEVERR_BAD_ROWS);
        int end = 0, items = 0;
        for (int g = 0; g < P.groups; ++g) {
            int a = __ldg(P.offsets + g), b = __ldg(P.offsets + g + 1);
            if (a < end || b < a || b > P.rows) a = b = 0;
            else end = b;
            t.start[g] = a;
            t.count[g] = b - a;
            t.first[g] = items;
            items += items_of(b - a);
        }
        t.first[P.groups] = items;
        return;
    }
    int base = incl - sum;
    for (int w = 0; w < warp; ++w) base += warp_sums[w];
    for (int g = g0; g < min(g0 + per, P.groups); ++g) t.first[g] += base;
    if (tid == THREADS - 1) t.first[P.groups] = base + sum;
}

// The group of item i: the largest g with first[g] <= i.
__device__ __forceinline__ int rag_group(const RagTable& t, int groups, int i) {
    int lo = 0, hi = groups - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first[mid] <= i) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// n / d for 0 <= n < 2^20, from inv = 1 / d: (n + 1/2) / d is at least 1 / (2 d) from every
// integer, and the product (1 / d to two ulps, one rounding) less than 2^-21 of it off.
__device__ __forceinline__ int quotient(int n, float inv) { return (int)(((float)n + 0.5f) * inv); }

// The first of `blocks` < 2^20 blocks that part p of P.split takes: equal shares, the first
// ones a block longer.
__device__ __forceinline__ int rag_share(const RaggedArgs& P, int blocks, int p) {
    const int each = quotient(blocks, __fdividef(1.0f, (float)P.split));
    return p * each + min(p, blocks - each * P.split);
}

// Items in increasing order.  A group's items run in bands of RAG_BAND chunks (TN: column
// tiles), a band's chunks together over the feature tiles: at any time the pairs work on a
// block of about RAG_BAND chunks x 9 tiles whose operands L2 holds.
// What depends on the group is kept from item to item, and the divisions inside it are
// products with reciprocals: found anew for each item (a bisection and three divisions) an
// item cost the epilogue 1200 clocks, a quarter of a weight gradient's over 128 rows.
template <int DIR>
struct RagWalk {
    const RaggedArgs& P;
    const RagTable& t;
    int g = -1, next = 0;         // the group and the first item behind it
    int first, start, count;
    int nc, w;                    // its chunks, and rows of a chunk
    float per_chunks;             // one band: 1 / nc
    int band_items, tail;         // several: items of a full band, chunks of the last
    float per_band, per_tail;     // and 1 / each

    __device__ __forceinline__ RagWalk(const RaggedArgs& p, const RagTable& table) : P(p), t(table) {}

    __device__ __forceinline__ void enter(int i) {
        g = g + 1 < P.groups && t.first[g + 2 <= P.groups ? g + 2 : P.groups] > i ? g + 1 : rag_group(t, P.groups, i);
        first = t.first[g];
        next = t.first[g + 1];
        start = t.start[g];
        count = t.count[g];
        nc = rag_chunks<DIR>(P, count);
        w = DIR == RAG_TN || nc == 1 ? P.bn : ((count + nc - 1) / nc + 31) & ~31;  // equal chunks, at most bn rows
        if (nc <= RAG_BAND) {
            per_chunks = __fdividef(1.0f, (float)nc);
        } else {
            band_items = RAG_BAND * ((P.n + 255) >> 8);
            tail = ((nc - 1) & (RAG_BAND - 1)) + 1;
            per_band = __fdividef(1.0f, (float)band_items);
            per_tail = __fdividef(1.0f, (float)tail);
        }
    }

    __device__ __forceinline__ RagItem at(int i) {
        if (i >= next) enter(i);
        RagItem it;
        int local = i - first, band = 0;
        if (nc <= RAG_BAND) {
            it.m = quotient(local, per_chunks);
            local -= it.m * nc;
        } else {
            band = local < 1 << 20 ? quotient(local, per_band) : local / band_items;
            local -= band * band_items;
            const bool full = (band + 1) * RAG_BAND <= nc;
            it.m = full ? local / RAG_BAND : quotient(local, per_tail);
            local -= it.m * (full ? RAG_BAND : tail);
        }
        const int c = band * RAG_BAND + local;
        it.g = g;
        it.chunks = nc;
        if (DIR == RAG_TN) {
            it.row0 = start;
            it.rows = count;
            it.col0 = c * w;
            it.width = min(w, P.k - it.col0);
        } else {
            it.row0 = start + c * w;
            it.rows = it.width = min(w, count - c * w);
            it.col0 = 0;
        }
        return it;
    }
};

// Blocks of 128 bytes (NT; NN, TN: of 64 rows) of the summed axis an item reads.
template <int DIR, bool I8>
__device__ __forceinline__ int rag_blocks(const RaggedArgs& P, const RagItem& it) {
    if (DIR == RAG_TN) return (it.rows + 63) >> 6;
    return I8 ? (P.k + 127) >> 7 : (P.k + 63) >> 6;
}

// Width of the MMA: the item's, in steps of 32 (NT, NN) or of the 64-column blocks of
// both CTAs (TN; the loads fill columns past dw's last with zeros).
template <int DIR>
__device__ __forceinline__ int rag_mma_n(const RagItem& it) {
    return DIR == RAG_TN ? (it.width + 127) & ~127 : (it.width + 31) & ~31;
}

// MN-major operand tile in 128-byte-swizzled 64 x 64 blocks: 8 rows of the summed axis
// are 1024 bytes (stride byte offset), the next 64 elements of the free axis RAG_TN_BLOCK
// further (leading byte offset).
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(RAG_TN_BLOCK >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// Instruction descriptor: kind::f16 (fp32 sums; `fmt` 0 = f16, 1 = bf16) or kind::i8
// (32-bit sums of signed 8-bit operands); bits 15 / 16 say that A / B is MN-major.
template <int DIR, bool I8>
__device__ __forceinline__ uint32_t rag_idesc(uint32_t fmt, uint32_t M, uint32_t N) {
    const uint32_t d_fmt = I8 ? 2u : 1u, ab = I8 ? 1u : fmt;
    return (d_fmt << 4) | (ab << 7) | (ab << 10) | (DIR != RAG_NT ? 1u << 15 : 0u) | (DIR == RAG_TN ? 1u << 16 : 0u) |
           ((N >> 3) << 17) | ((M >> 4) << 24);
}

__device__ __forceinline__ void mma2_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 3-D tiled load (x inner, y, z) counted on an mbarrier of either CTA of the pair.  No multicast.
__device__ __forceinline__ void tma_load_3d_pair(void* smem_dst, const CUtensorMap* map, int x, int y, int z,
                                                 uint32_t mbar_cluster, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(mbar_cluster), "l"(policy)
        : "memory");
}

// The wait of the MMA issuer for a stage that warps of both CTAs hand over (acquire at
// cluster scope: the peer's zeroed rows are then visible); else as mbar_wait_bounded.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ bool mbar_wait_bounded_cluster(uint64_t* bar, uint32_t parity, volatile int* abort,
                                                          uint64_t limit_ns = 2000000000ull) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait_cluster(bar, parity)) return true;
        if ((it & 63u) == 0) {
            if (*abort) return false;
            if (global_timer_ns() - t0 > limit_ns) {
                set_dev_error(MOE_DEVERR_TIMEOUT);
                *abort = 1;
                return false;
            }
        }
    }
}

// A wait that may begin many items before its own: the limit counts from the last change of
// *progress (the item that the loads have come to), else as mbar_wait_bounded.
__device__ __forceinline__ bool mbar_wait_following(uint64_t* bar, uint32_t parity, volatile int* abort,
                                                    volatile int* progress, uint64_t limit_ns = 2000000000ull) {
    int seen = *progress;
    uint64_t t0 = global_timer_ns();
    for (uint32_t it = 0;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) == 0) {
            if (*abort) return false;
            const int now = *progress;
            if (now != seen) {
                seen = now;
                t0 = global_timer_ns();
            } else if (global_timer_ns() - t0 > limit_ns) {
                set_dev_error(MOE_DEVERR_TIMEOUT);
                *abort = 1;
                return false;
            }
        }
    }
}

// Before a CTA that gave up a wait leaves: a role may have issued loads up to the moment when another
// set the flag, and they must not land in the next CTA's memory.  A load lands within
// microseconds, whatever its barrier is waiting for; a millisecond is the limit.
__device__ __forceinline__ void settle_copies(volatile int* abort) {
    if (!*abort) return;
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 1000000ull) __nanosleep(1000);
}

// fp32 -> 16-bit bits, one rounding to nearest even.
template <bool BF16>
__device__ __forceinline__ uint32_t rag_pack2(float a, float b) {
    if (BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t rag_pack2(float a, float b, int bf16) {
    return bf16 ? rag_pack2<true>(a, b) : rag_pack2<false>(a, b);
}
__device__ __forceinline__ float rag_unpack(uint16_t v, int bf16) {
    if (bf16) return __uint_as_float((uint32_t)v << 16);
    return __half2float(__ushort_as_half(v));
}

// Epilogue of NT / NN for 32 columns (rows of y) of a warp's 32 features: v[j] is
// feature f0 + lane of row row0 + j, j < valid.  The values pass through the warp's
// 2 KB of `stage`, so that a lane stores 16 bytes and the warp several rows' pieces (64
// bytes in 16 bits, 128 in fp32) with one instruction.
__device__ __forceinline__ void rag_store_rows_f32(const RaggedArgs& P, uint8_t* stage, int row0, int valid, int f0,
                                                   const float (&v)[32]) {
    const int lane = threadIdx.x & 31;
    const int f = f0 + (lane & 7) * 4;  // n is a multiple of 8: a piece is inside or outside
    float* st = reinterpret_cast<float*>(stage);
#pragma unroll
    for (int h = 0; h < 2; ++h) {       // 16 rows at a time
#pragma unroll
        for (int j = 0; j < 16; ++j) st[j * 32 + lane] = v[16 * h + j];
        __syncwarp();
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
            const int j = i * 4 + (lane >> 3);
            if (16 * h + j < valid && f < P.n) {
                float4 s = *reinterpret_cast<const float4*>(st + j * 32 + (lane & 7) * 4);
                float4* y = reinterpret_cast<float4*>(static_cast<float*>(P.y) + (size_t)(row0 + 16 * h + j) * P.ldy + f);
                if (P.accumulate) {
                    const float4 o = *y;
                    s = make_float4(o.x + s.x, o.y + s.y, o.z + s.z, o.w + s.w);
                }
                *y = s;
            }
        }
        __syncwarp();
    }
}

// 16-bit results.  A word of the stage holds two rows' values of one feature (one
// conversion and one store for two values); a lane takes eight features of a pair of rows
// back and parts them.  Reading the two 16-byte halves in the other order on odd pairs
// keeps a quarter warp on different banks.
template <bool BF16>
__device__ __forceinline__ void rag_store_rows_h16(const RaggedArgs& P, uint8_t* stage, int row0, int valid, int f0,
                                                   const float (&v)[32]) {
    const int lane = threadIdx.x & 31;
    uint32_t* st = reinterpret_cast<uint32_t*>(stage);
#pragma unroll
    for (int j = 0; j < 16; ++j) st[j * 32 + lane] = rag_pack2<BF16>(v[2 * j], v[2 * j + 1]);
    __syncwarp();
    const int part = lane & 3, odd = (lane >> 2) & 1;
    if (f0 + part * 8 < P.n) {
        uint16_t* y = static_cast<uint16_t*>(P.y) + (size_t)(row0 + 2 * (lane >> 2)) * P.ldy + f0 + part * 8;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = 16 * i + 2 * (lane >> 2);  // the pair's first row
            const uint4* src = reinterpret_cast<const uint4*>(st + (j >> 1) * 32 + part * 8);
            const uint4 p = src[odd], q = src[odd ^ 1];
            const uint4 lo = odd ? q : p, hi = odd ? p : q;
            if (j < valid)
                *reinterpret_cast<uint4*>(y + (size_t)(16 * i) * P.ldy) =
                    make_uint4(__byte_perm(lo.x, lo.y, 0x5410), __byte_perm(lo.z, lo.w, 0x5410),
                               __byte_perm(hi.x, hi.y, 0x5410), __byte_perm(hi.z, hi.w, 0x5410));
            if (j + 1 < valid)
                *reinterpret_cast<uint4*>(y + (size_t)(16 * i + 1) * P.ldy) =
                    make_uint4(__byte_perm(lo.x, lo.y, 0x7632), __byte_perm(lo.z, lo.w, 0x7632),
                               __byte_perm(hi.x, hi.y, 0x7632), __byte_perm(hi.z, hi.w, 0x7632));
        }
    }
    __syncwarp();
}

__device__ __forceinline__ void rag_store_rows(const RaggedArgs& P, uint8_t* stage, int row0, int valid, int f0,
                                               const float (&v)[32]) {
    const int lane = threadIdx.x & 31;
    if (P.out == MOE_F32) {
        rag_store_rows_f32(P, stage, row0, valid, f0, v);
    } else if (P.accumulate) {  // added in fp32 and rounded once: in place, two bytes a lane
        const int bf16 = P.out == MOE_BF16;
        if (f0 + lane < P.n) {
            uint16_t* y = static_cast<uint16_t*>(P.y) + (size_t)row0 * P.ldy + f0 + lane;
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (j < valid) {
                    uint16_t* p = y + (size_t)j * P.ldy;
                    const float s = rag_unpack(*p, bf16) + v[j];
                    *p = (uint16_t)(rag_pack2(s, s, bf16) & 0xffffu);
                }
        }
    } else if (P.out == MOE_BF16) {
        rag_store_rows_h16<true>(P, stage, row0, valid, f0, v);
    } else {
        rag_store_rows_h16<false>(P, stage, row0, valid, f0, v);
    }
}

// Epilogue of TN: lane holds row f0 + lane of dw, columns c0 .. (32 fp32 values, or 64
// 16-bit ones already packed); the warp's 4 KB tile is staged (16-byte pieces swizzled by
// the row, free of bank conflicts) and stored as whole 128-byte pieces of rows.
__device__ __forceinline__ void rag_stage_piece(uint8_t* stage, int piece, uint4 v) {
    const int lane = threadIdx.x & 31;
    *reinterpret_cast<uint4*>(stage + lane * 128 + ((piece ^ (lane & 7)) << 4)) = v;
}
// 32 columns of the lane's row in 16 bits, from piece p0 on
__device__ __forceinline__ void rag_stage_h16(uint8_t* stage, int p0, const float (&v)[32], int bf16) {
#pragma unroll
    for (int p = 0; p < 4; ++p)
        rag_stage_piece(stage, p0 + p, make_uint4(rag_pack2(v[8 * p], v[8 * p + 1], bf16), rag_pack2(v[8 * p + 2], v[8 * p + 3], bf16),
                                                  rag_pack2(v[8 * p + 4], v[8 * p + 5], bf16), rag_pack2(v[8 * p + 6], v[8 * p + 7], bf16)));
}
__device__ __forceinline__ uint4 rag_staged(const uint8_t* stage, int row, int piece) {
    return *reinterpret_cast<const uint4*>(stage + row * 128 + ((piece ^ (row & 7)) << 4));
}

template <bool F32>
__device__ __forceinline__ void rag_store_f32_tile(const RaggedArgs& P, uint8_t* stage, size_t base, int f0, int c0,
                                                   const float (&v)[32]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        rag_stage_piece(stage, i, make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                             __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3])));
    __syncwarp();
    const int piece = lane & 7, col = c0 + piece * 4;
    if (col < P.k) {
#pragma unroll 2
        for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + (lane >> 3);
            if (f0 + r >= P.n) break;
            const uint4 u = rag_staged(stage, r, piece);
            float4 s = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z),
                                   __uint_as_float(u.w));
            const size_t at = base + (size_t)(f0 + r) * P.k + col;
            if (F32) {
                float4* p = reinterpret_cast<float4*>(static_cast<float*>(P.y) + at);
                if (P.accumulate) {
                    const float4 o = *p;
                    s = make_float4(o.x + s.x, o.y + s.y, o.z + s.z, o.w + s.w);
                }
                *p = s;
            } else {  // 16-bit accumulate: added in fp32, rounded once
                const int bf16 = P.out == MOE_BF16;
                uint2* p = reinterpret_cast<uint2*>(static_cast<uint16_t*>(P.y) + at);
                const uint2 o = *p;
                s.x += rag_unpack((uint16_t)o.x, bf16);
                s.y += rag_unpack((uint16_t)(o.x >> 16), bf16);
                s.z += rag_unpack((uint16_t)o.y, bf16);
                s.w += rag_unpack((uint16_t)(o.y >> 16), bf16);
                *p = make_uint2(rag_pack2(s.x, s.y, bf16), rag_pack2(s.z, s.w, bf16));
            }
        }
    }
    __syncwarp();
}

__device__ __forceinline__ void rag_store_h16_tile(const RaggedArgs& P, uint8_t* stage, size_t base, int f0, int c0) {
    const int lane = threadIdx.x & 31;
    __syncwarp();
    const int piece = lane & 7, col = c0 + piece * 8;
    if (col < P.k) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + (lane >> 3);
            if (f0 + r < P.n)
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(P.y) + base + (size_t)(f0 + r) * P.k + col) =
                    rag_staged(stage, r, piece);
        }
    }
    __syncwarp();
}

__device__ __forceinline__ uint32_t cluster_id() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(r));
    return r;
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// An integer sum times its two scales.  Their product alone can leave the normal numbers where the
// result does not, so the sum meets the channel's scale first; z times it keeps its 24 bits (below
// the normal numbers it is a multiple of their step, exact), and with |z| <= 2^30 it is finite below
// RAG_SCALE_FIRST.  A larger scale comes last: if z times the row's overflows then, so does the result.
// NaN and infinity come last too.  first * last is the scale, one of them 1.
constexpr float RAG_SCALE_FIRST = 0x1p97f;
__device__ __forceinline__ float rag_scale_first(float sw) { return fabsf(sw) < RAG_SCALE_FIRST ? sw : 1.0f; }
__device__ __forceinline__ float rag_scale_last(float sw) { return fabsf(sw) < RAG_SCALE_FIRST ? 1.0f : sw; }
__device__ __forceinline__ float rag_scaled(int z, float sx, float sw) {
    return (float)z * rag_scale_first(sw) * sx * rag_scale_last(sw);
}

// Four values of a row, added to what is there with accumulate, rounded once.
__device__ __forceinline__ void rag_store4(const RaggedArgs& P, size_t at, float4 s) {
    if (P.out == MOE_F32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(P.y) + at);
        if (P.accumulate) {
            const float4 o = *p;
            s = make_float4(o.x + s.x, o.y + s.y, o.z + s.z, o.w + s.w);
        }
        *p = s;
        return;
    }
    const int bf16 = P.out == MOE_BF16;
    uint2* p = reinterpret_cast<uint2*>(static_cast<uint16_t*>(P.y) + at);
    if (P.accumulate) {
        const uint2 o = *p;
        s.x += rag_unpack((uint16_t)o.x, bf16);
        s.y += rag_unpack((uint16_t)(o.x >> 16), bf16);
        s.z += rag_unpack((uint16_t)o.y, bf16);
        s.w += rag_unpack((uint16_t)(o.y >> 16), bf16);
    }
    *p = make_uint2(rag_pack2(s.x, s.y, bf16), rag_pack2(s.z, s.w, bf16));
}

// A tile whose summed axis P.split CTAs of a cluster share: each has written its part to its
// shared memory (NT, NN: [column][128 features], TN: [feature][bn + 4] values, integers as
// bits), CTA first_rank + rank_step p holds part p.  CTA number `part` adds its share of the
// tile's rows over all parts, in the parts' order, and stores it.  A lane takes one piece of
// four values of a row, warp w of eight one row at a time (TN with 64 columns: two).
template <int DIR, bool I8>
__device__ __forceinline__ void rag_store_parts(const RaggedArgs& P, const uint8_t* ring, int first_rank, int rank_step,
                                                int part, int w, int g, int f0, int row0, int col0, int width) {
    const int lane = threadIdx.x & 31;
    const uint32_t base = smem_u32(ring);
    const int n_rows = DIR == RAG_TN ? max(0, min(128, P.n - f0)) : width;  // rows of the output's tile
    const int n_vec = (DIR == RAG_TN ? width : min(128, P.n - f0)) / 4;      // its pieces of four (none behind n)
    const int pitch = DIR == RAG_TN ? P.bn + 4 : 128;
    const int r0 = P.split == 1 ? 0 : n_rows * part / P.split, r1 = P.split == 1 ? n_rows : n_rows * (part + 1) / P.split;
    const bool two = DIR == RAG_TN && P.bn == 64;
    for (int r = r0 + (two ? 2 * w + (lane >> 4) : w); r < r1; r += two ? 16 : 8) {
        for (int v = two ? lane & 15 : lane; v < n_vec; v += 32) {
            const uint32_t at = (uint32_t)(r * pitch + v * 4) * 4;
            float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            int4 z = make_int4(0, 0, 0, 0);
            if (P.split == 1) {
                s = *reinterpret_cast<const float4*>(ring + at);
                z = make_int4(__float_as_int(s.x), __float_as_int(s.y), __float_as_int(s.z), __float_as_int(s.w));
            } else {
                for (int p0 = 0; p0 < P.split; p0 += 8) {  // (a part without blocks is zero)
                    float4 u[8];                           // loads of eight parts under way together
#pragma unroll
                    for (int p = 0; p < 8; ++p) {
                        u[p] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        if (p0 + p < P.split)
                            u[p] = ld_cluster_f4(mapa_shared(base + at, (uint32_t)(first_rank + rank_step * (p0 + p))));
                    }
#pragma unroll
                    for (int p = 0; p < 8; ++p) {
                        if (I8) {
                            z.x += __float_as_int(u[p].x);
                            z.y += __float_as_int(u[p].y);
                            z.z += __float_as_int(u[p].z);
                            z.w += __float_as_int(u[p].w);
                        } else {
                            s = make_float4(s.x + u[p].x, s.y + u[p].y, s.z + u[p].z, s.w + u[p].w);
                        }
                    }
                }
            }
            if (DIR == RAG_TN) {
                rag_store4(P, ((size_t)g * P.n + f0 + r) * P.k + col0 + v * 4, s);
            } else {
                if (I8) {
                    const float sx = __ldg(P.sx + row0 + r);
                    const float* sw = P.sw + (size_t)g * P.n + f0 + v * 4;
                    s = make_float4(rag_scaled(z.x, sx, __ldg(sw)), rag_scaled(z.y, sx, __ldg(sw + 1)),
                                    rag_scaled(z.z, sx, __ldg(sw + 2)), rag_scaled(z.w, sx, __ldg(sw + 3)));
                }
                rag_store4(P, (size_t)(row0 + r) * P.ldy + f0 + v * 4, s);
            }
        }
    }
}

// A position in a ring of N slots.
template <int N>
struct RagCursor {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++slot == N) {
            slot = 0;
            phase ^= 1u;
        }
    }
    __device__ __forceinline__ void skip(int n) {  // n >= 0
        const int at = slot + n;
        phase ^= (uint32_t)((at / N) & 1);
        slot = at % N;
    }
};

// (a0, a1) += (b0, b1), in place and in order: the volatile keeps the next TMEM load
// behind it, whose registers would come on top of the sums'.
__device__ __forceinline__ void add2(float& a0, float& a1, float b0, float b1) {
    asm volatile(
        "{\n\t.reg .b64 pa, pb;\n\t"
        "mov.b64 pa, {%0, %1};\n\t"
        "mov.b64 pb, {%2, %3};\n\t"
        "add.rn.f32x2 pa, pa, pb;\n\t"
        "mov.b64 {%0, %1}, pa;\n\t}"
        : "+f"(a0), "+f"(a1)
        : "f"(b0), "f"(b1));
}

__device__ __forceinline__ void mul2(float& a0, float& a1, float b0, float b1) {
    asm("{\n\t.reg .b64 pa, pb;\n\t"
        "mov.b64 pa, {%0, %1};\n\t"
        "mov.b64 pb, {%2, %3};\n\t"
        "mul.rn.f32x2 pa, pa, pb;\n\t"
        "mov.b64 {%0, %1}, pa;\n\t}"
        : "+f"(a0), "+f"(a1)
        : "f"(b0), "f"(b1));
}

// One lane of a converged warp, in the form that tells the compiler that no other runs
// the code behind it: TMA and MMA operands then go straight to uniform registers.  With
// `lane == 0` instead the 8192^3 product took 812 us instead of 754, and 415 instead of
// 348 in 8-bit integers.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void rag_arrive(uint32_t bar_cluster, uint32_t count) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0], %1;" ::"r"(bar_cluster), "r"(count) : "memory");
}

// Whether the two halves of the epilogue's warps take whole tiles in turn, one accumulator
// each, instead of half of every tile's columns.  After a sum of at most 256 bytes the
// epilogue is what a tile waits for, and its latencies (the wait, the first load, the
// hand-over) then run side by side; a group's narrow tiles leave no warp without columns.
// In turn against halves, in us:
//   214 groups, 7210 rows, n 3352, k 64     bf16 49.8 / 57.8   fp32 59.4 / 82.1
//   the same, int8, k 128                   bf16 52.9 / 71.5   fp32 66.6 / 87.4
//   64 groups, 65536 rows, n 2048, k 64     bf16 74.6 / 87.5   fp32  130 / 143
//   the same, int8, k 128                   bf16 94.7 / 105    fp32  151 / 159
//   the same, bf16, k 512                   bf16  136 / 134    fp32  179 / 175
//   1 group, 65536 rows, n 2048, k 128      bf16 77.8 / 75.1   fp32  122 / 119
//   8 groups, 4096 rows, n 4096, k 64       fp32 23.2 / 22.4 (3.5 tiles a pair: a last
//                                           tile's epilogue takes twice as long)
template <bool I8>
__device__ __forceinline__ bool rag_alternate(const RaggedArgs& P, int total, int pairs) {
    return P.groups > 1 && P.k <= (I8 ? 256 : 128) && total >= 6 * pairs;
}

// MODE: RAG_PLAIN; RAG_PROMOTE, fp32 results of long sums; RAG_LONG, 16-bit results of sums of
// which some are longer than P.whole blocks; RAG_SPLIT, one tile a cluster of P.split pairs that
// share its summed axis (rag_store_parts), where a product has few tiles.
template <int DIR, bool I8, int MODE>
__global__ void __launch_bounds__(RAG_THREADS, 1) moe_ragged_kernel(const __grid_constant__ RaggedArgs P) {
    using C = RagCfg<DIR>;
    constexpr bool SPLIT = MODE == RAG_SPLIT;
    constexpr bool PROMOTE = MODE != RAG_PLAIN;  // sums in the epilogue's registers
    constexpr bool AHEAD = I8 && !PROMOTE;       // the scales are loaded a tile ahead
    constexpr bool REGS = PROMOTE || I8;         // the epilogue needs more than an equal share of registers
    constexpr int ST = C::STAGES;
    const int2 head = rag_first_offsets(P);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* ring = smem;
    uint8_t* staging = smem + C::RING;
    RagTable tab;
    tab.start = reinterpret_cast<int*>(staging + RAG_EPI_WARPS * (C::STAGING + C::SCALES));
    tab.count = tab.start + RAG_MAX_GROUPS;
    tab.first = tab.count + RAG_MAX_GROUPS;
    uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(tab.start) + C::TABLE);
    uint64_t* full = bars;                 // leader: both CTAs' bytes of the stage are there
    uint64_t* empty = full + ST;           // both: stage consumed
    uint64_t* tfull = empty + ST;          // [2] both: accumulator written
    uint64_t* tempty = tfull + 2;          // [2] leader: accumulator read by both epilogues
    uint64_t* drain = tempty + 2;
    uint64_t* landed = drain + 1;          // TN, blocks with tail rows, both: this CTA's bytes
    uint64_t* peer_done = landed + ST;     // TN, blocks with tail rows, leader: the peer's tail is zeroed
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::BARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* progress = reinterpret_cast<volatile int*>(tmem_slot + 2);  // TN: the item being loaded
    int* warp_sums = reinterpret_cast<int*>(tmem_slot + 3);  // [RAG_THREADS / 32]

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t crank = cluster_ctarank();
    const uint32_t rank = crank & 1u, pair0 = crank & ~1u;  // side of the pair, and its leader's rank
    const uint16_t pair_mask = (uint16_t)(3u << pair0);
    const int part = (int)(crank >> 1);
    const bool leader = rank == 0;

    if (threadIdx.x < C::BARS) {
        // the two accumulators are released by every epilogue warp of both CTAs
        const bool is_tempty = &bars[threadIdx.x] == tempty || &bars[threadIdx.x] == tempty + 1;
        mbar_init(&bars[threadIdx.x], is_tempty ? 2 * RAG_EPI_WARPS : 1);
        fence_mbar_init();
    } else if (threadIdx.x == RAG_THREADS - 1) {
        *abort_flag = 0;
        *progress = -1;
        tma_prefetch_desc(&P.a);
        tma_prefetch_desc(&P.b64);
        if (DIR != RAG_TN) {
            tma_prefetch_desc(&P.b128);
            tma_prefetch_desc(&P.b16);
        }
    }
    if (warp == 4) tmem_alloc_pair(tmem_slot);
    rag_build_table<RAG_THREADS>(P, tab, warp_sums, head, [&](int rows) { return rag_items_of<DIR>(P, rows); });
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // both CTAs' barriers initialised and TMEM allocated
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int total = tab.first[P.groups];
    const int first = SPLIT ? (int)cluster_id() : blockIdx.x >> 1;
    const int n_clusters = SPLIT ? 1 << 30 : gridDim.x >> 1;  // SPLIT: one item at most
    const int seg_blocks = I8 ? 1 << 30 : MODE == RAG_LONG ? P.whole : RAG_SEGMENT / 64;
    // this pair's blocks of an item's
    auto begin = [&](int blocks) { return SPLIT ? rag_share(P, blocks, part) : 0; };
    auto end = [&](int blocks) { return SPLIT ? rag_share(P, blocks, part + 1) : blocks; };
    // whether the epilogue adds up an item's segments
    auto segmented = [&](int blocks) { return MODE == RAG_LONG ? blocks > P.whole : PROMOTE; };

    if (warp < RAG_EPI_WARP0) {
        if (REGS) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(RAG_REGS_CONTROL));
        if (warp < 4) {
            // ---------------------------------------------------- loads (both CTAs)
            // warp 0: A (NN, TN: its first 64 features), 1: A's other 64, 2: B
            const bool works = warp == 0 || warp == 2 || (warp == 1 && DIR != RAG_NT);
            if (works && elect_one()) {
                const bool is_a = warp < 2;
                const int half = (warp & 1) * 64;  // of A
                const uint64_t pol_stream = l2_policy_evict_first();
                const uint64_t pol_keep = l2_policy_evict_last();
                const uint64_t pol_normal = l2_policy_evict_normal();
                const uint32_t full0 = mapa_shared(smem_u32(full), pair0);
                const uint32_t landed0 = mapa_shared(smem_u32(landed), crank);
                RagCursor<ST> at;
                RagWalk<DIR> walk(P, tab);
                for (int i = first; i < total; i += n_clusters) {
                    const RagItem it = walk.at(i);
                    if (DIR == RAG_TN && warp == 0) *progress = i;
                    const int blocks = rag_blocks<DIR, I8>(P, it);
                    const int f0 = it.m * 256 + (int)rank * 128;
                    const int nh = rag_mma_n<DIR>(it) / 2;  // this CTA's columns of the tile
                    // weights that one chunk reads stream; those of several chunks stay for the others
                    const uint64_t policy = DIR == RAG_TN || !is_a ? pol_normal : it.chunks > 1 ? pol_keep : pol_stream;
                    // rows of the smallest box that holds this CTA's rows (NT, NN)
                    const int box = nh > 64 ? 128 : nh > 16 ? 64 : 16;
                    const CUtensorMap* bmap = nh > 64 ? &P.b128 : nh > 16 ? &P.b64 : &P.b16;
                    const bool second = nh > 64;                 // TN: B has a second 64-column block
                    const uint32_t bytes =
                        RAG_SLOT + (DIR == RAG_TN ? (second ? 2u : 1u) * RAG_TN_BLOCK : (uint32_t)box * 128u);
                    const int brow = it.row0 + (int)rank * nh;
                    bool ok = true;
                    for (int kb = begin(blocks); kb < end(blocks); ++kb) {
                        if (!mbar_wait_bounded(&empty[at.slot], at.phase ^ 1u, abort_flag)) { ok = false; break; }
                        uint8_t* dst = ring + at.slot * 2 * RAG_SLOT + (is_a ? 0 : RAG_SLOT) + half * 128;
                        // a block whose last rows belong to the next group is counted where it lies,
                        // for the warp that zeroes them; the others on the leader's barrier
                        const bool tail = DIR == RAG_TN && kb == blocks - 1 && (it.rows & 15);
                        const uint32_t bar = (tail ? landed0 : full0) + (uint32_t)(at.slot * 8);
                        if (warp == 0) {
                            if (tail) mbar_arrive_expect_tx(&landed[at.slot], bytes);
                            else if (leader) mbar_arrive_expect_tx(&full[at.slot], 2u * bytes);
                        }
                        if (DIR == RAG_TN) {
                            if (is_a) {
                                tma_load_2d_pair(dst, &P.a, f0 + half, it.row0 + kb * 64, bar, policy);
                            } else {
                                const int x = it.col0 + (int)rank * nh, y = it.row0 + kb * 64;
                                tma_load_2d_pair(dst, &P.b64, x, y, bar, policy);
                                if (second) tma_load_2d_pair(dst + RAG_TN_BLOCK, &P.b64, x + 64, y, bar, policy);
                            }
                        } else if (!is_a) {
                            tma_load_2d_pair(dst, bmap, kb * (I8 ? 128 : 64), brow, bar, policy);
                        } else if (DIR == RAG_NT) {
                            tma_load_3d_pair(dst, &P.a, kb * (I8 ? 128 : 64), f0, it.g, bar, policy);
                        } else {
                            tma_load_3d_pair(dst, &P.a, f0 + half, kb * 64, it.g, bar, policy);
                        }
                        at.next();
                    }
                    if (!ok) break;
                }
            }
        } else if (warp == 4) {
            if (leader && elect_one()) {
                // ------------------------------------------------ 2-SM MMA issuer
                RagCursor<ST> at;
                uint32_t acc_phase = 0;  // bit b: phase of accumulator b
                int buf = 0;
                bool issued = false;
                // one step sums 32 bytes of a K-major row, or 16 rows (2048 bytes) of an MN-major tile
                constexpr uint64_t a_step = DIR == RAG_NT ? 2 : 128, b_step = DIR == RAG_TN ? 128 : 2;
                constexpr int per_step = I8 ? 32 : 16;
                constexpr uint64_t stage_step = 2 * RAG_SLOT / 16;
                const uint32_t ring_addr = smem_u32(ring);
                const uint64_t ad0 = DIR == RAG_NT ? smem_desc_sw128(ring_addr) : smem_desc_mn_sw128(ring_addr);
                const uint64_t bd0 = DIR == RAG_TN ? smem_desc_mn_sw128(ring_addr + RAG_SLOT)
                                                   : smem_desc_sw128(ring_addr + RAG_SLOT);
                bool ok = true;
                RagWalk<DIR> walk(P, tab);
                for (int i = first; ok && i < total; i += n_clusters) {
                    const RagItem it = walk.at(i);
                    const int blocks = rag_blocks<DIR, I8>(P, it);
                    // elements of the summed axis in the last block (TN: rows past it are zero up to a
                    // multiple of 16; NT, NN: the loads filled in zeros)
                    const int last = (DIR == RAG_TN ? it.rows : P.k) - (blocks - 1) * 4 * per_step;
                    const uint32_t idesc = rag_idesc<DIR, I8>((uint32_t)P.bf16, 256, (uint32_t)rag_mma_n<DIR>(it));
                    const int stop = end(blocks);
                    for (int kb0 = begin(blocks), kb1; kb0 < stop; kb0 = kb1) {
                        kb1 = segmented(blocks) ? kb0 + min(seg_blocks, stop - kb0) : stop;
                        if (!mbar_wait_bounded(&tempty[buf], ((acc_phase >> buf) & 1u) ^ 1u, abort_flag)) { ok = false; break; }
                        const uint32_t d = tmem_base + (uint32_t)(buf * 256);
                        for (int kb = kb0; kb < kb1; ++kb) {
                            if (!mbar_wait_bounded(&full[at.slot], at.phase, abort_flag)) { ok = false; break; }
                            tc_fence_after();
                            const uint64_t ad = ad0 + stage_step * at.slot, bd = bd0 + stage_step * at.slot;
                            const int steps = kb == blocks - 1 ? (last + per_step - 1) / per_step : 4;
                            if (steps == 4) {
#pragma unroll
                                for (int s = 0; s < 4; ++s) {
                                    const uint32_t accum = (kb > kb0 || s != 0) ? 1u : 0u;
                                    if (I8) mma2_i8(d, ad + a_step * s, bd + b_step * s, idesc, accum);
                                    else mma2_bf16(d, ad + a_step * s, bd + b_step * s, idesc, accum);
                                }
                            } else {
                                for (int s = 0; s < steps; ++s) {
                                    const uint32_t accum = (kb > kb0 || s != 0) ? 1u : 0u;
                                    if (I8) mma2_i8(d, ad + a_step * s, bd + b_step * s, idesc, accum);
                                    else mma2_bf16(d, ad + a_step * s, bd + b_step * s, idesc, accum);
                                }
                            }
                            mma2_commit_pair(&empty[at.slot], pair_mask);
                            issued = true;
                            at.next();
                        }
                        if (!ok) break;
                        mma2_commit_pair(&tfull[buf], pair_mask);
                        acc_phase ^= 1u << buf;
                        buf ^= 1;
                    }
                }
                if (*abort_flag && issued) {
                    mma2_commit_local(drain);
                    volatile int dummy = 0;
                    mbar_wait_bounded(drain, 0, &dummy, 100000000ull);
                }
            }
        } else if (warp == 5 && DIR == RAG_TN) {
            // ---------------------------------------------------- tail rows (both CTAs)
            RagCursor<ST> at;
            uint32_t ph = 0;  // bit s: phase of the stage's landed and peer_done
            const uint32_t peer0 = mapa_shared(smem_u32(peer_done), pair0);
            RagWalk<DIR> walk(P, tab);
            for (int i = first; i < total; i += n_clusters) {
                const RagItem it = walk.at(i);
                const int blocks = rag_blocks<DIR, I8>(P, it);
                const int mine = end(blocks) - begin(blocks);
                if ((it.rows & 15) == 0 || end(blocks) < blocks || mine == 0) {
                    at.skip(mine);
                    continue;
                }
                at.skip(mine - 1);
                // Items without tail rows are passed over at once, so this wait begins when the last
                // tail was done and may span any number of them.
                // Every lane waits: each then sees the landed bytes before it overwrites some.
                const bool ok = mbar_wait_following(&landed[at.slot], (ph >> at.slot) & 1u, abort_flag, progress);
                if (!__all_sync(0xffffffffu, ok)) break;
                const int r0 = it.rows - (blocks - 1) * 64;  // rows of the group in this block
                const int n = ((r0 + 15) & ~15) - r0;
                for (int j = lane; j < n * 32; j += 32) {    // a row is 128 bytes of each 64 x 64 block
                    const int row = r0 + (j >> 5), blk = (j >> 3) & 3, piece = j & 7;
                    *reinterpret_cast<uint4*>(ring + at.slot * 2 * RAG_SLOT + blk * RAG_TN_BLOCK + row * 128 + piece * 16) =
                        make_uint4(0, 0, 0, 0);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (!leader) {
                    if (lane == 0) mbar_arrive_cluster_release(peer0 + (uint32_t)(at.slot * 8));
                } else {
                    int got = 0;
                    if (lane == 0) got = mbar_wait_bounded_cluster(&peer_done[at.slot], (ph >> at.slot) & 1u, abort_flag);
                    if (!__shfl_sync(0xffffffffu, got, 0)) break;
                    if (lane == 0) mbar_arrive(&full[at.slot]);
                }
                ph ^= 1u << at.slot;
                at.next();
            }
        }
        if (SPLIT) {
            __syncwarp();
            cluster_sync_all();  // the parts' meeting, as in the epilogue
        }
    } else {
        // ------------------------------------------------------------ epilogue (both CTAs, own TMEM)
        if (REGS) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(RAG_REGS_EPILOGUE));
        const int q = warp & 3;                          // TMEM lane quarter of this warp
        const int half = (warp - RAG_EPI_WARP0) >> 2;
        uint8_t* stage = staging + (warp - RAG_EPI_WARP0) * C::STAGING;
        float* scales = reinterpret_cast<float*>(staging + RAG_EPI_WARPS * C::STAGING + (warp - RAG_EPI_WARP0) * C::SCALES);
        const uint32_t tempty0 = mapa_shared(smem_u32(&tempty[0]), pair0);
        uint32_t acc_phase = 0;
        const bool alternate = !PROMOTE && DIR != RAG_TN && rag_alternate<I8>(P, total, n_clusters);
        int buf = alternate ? half : 0;
        auto wait_acc = [&]() -> bool {
            int got = 0;
            if (lane == 0) got = mbar_wait_bounded(&tfull[buf], (acc_phase >> buf) & 1u, abort_flag) ? 1 : 0;
            got = __shfl_sync(0xffffffffu, got, 0);
            if (got) tc_fence_after();
            return got != 0;
        };
        auto release_acc = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) rag_arrive(tempty0 + (uint32_t)(buf * 8), alternate ? 2u : 1u);  // half the warps: twice each
            acc_phase ^= 1u << buf;
            buf ^= alternate ? 0 : 1;
        };
        RagWalk<DIR> walk(P, tab);
        // The scales of an int8 product come a tile ahead, and reach every lane through shared
        // memory once a tile: 65536 x 2048 x 128 took 125 us with a load and a meeting of the
        // warp for each 32 rows, 97 us so (75 us the bf16 product of the same output).
        RagItem ahead = {};
        const int chunks0 = alternate ? 0 : half;
        const int item0 = alternate ? first + half * n_clusters : first, item_step = alternate ? 2 * n_clusters : n_clusters;
        float sw_ahead = 0.0f, sx_ahead[4] = {};
        auto load_scales = [&](int i) {  // lane l: feature l of the warp, and rows l of its chunks of 32
            if (i >= total) return;
            ahead = walk.at(i);
            const int f = ahead.m * 256 + (int)rank * 128 + q * 32 + lane;
            if (f < P.n) sw_ahead = __ldg(P.sw + (size_t)ahead.g * P.n + f);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int r = 32 * (chunks0 + 2 * c) + lane;
                if (r < ahead.width) sx_ahead[c] = __ldg(P.sx + ahead.row0 + r);
            }
        };
        if (AHEAD) load_scales(item0);
        for (int i = item0; i < total; i += item_step) {
            const RagItem it = AHEAD ? ahead : walk.at(i);
            const int f0 = it.m * 256 + (int)rank * 128 + q * 32;
            const size_t base = (size_t)it.g * P.n * P.k;  // TN: the group's dw
            if (DIR == RAG_TN && it.rows == 0) {
                if (!P.accumulate && !SPLIT) {  // zeros, a row of the warp's 32 after the other; k is a multiple of 8
                    const int e = P.out == MOE_F32 ? 4 : 2, pieces = it.width * e / 16;
                    const int n = max(0, min(32, P.n - f0)) * pieces;
                    uint8_t* tile = static_cast<uint8_t*>(P.y) + (base + (size_t)f0 * P.k + it.col0) * e;
#pragma unroll 4
                    for (int j = 32 * half + lane; j < n; j += 64) {
                        const int r = pieces == 32 ? j >> 5 : pieces == 64 ? j >> 6 : j / pieces;
                        *reinterpret_cast<uint4*>(tile + (size_t)r * P.k * e + (j - r * pieces) * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
                if (!SPLIT) continue;  // (SPLIT: the parts are zero)
            }
            const uint32_t lanes = tmem_base + ((uint32_t)(q * 32) << 16);
            if (segmented(rag_blocks<DIR, I8>(P, it))) {
                // this warp's columns: chunks of 32, every other one; two neighbours where a stored
                // piece is 64 columns
                const bool pieces64 = DIR == RAG_TN && MODE == RAG_LONG && !P.accumulate;
                auto column = [&](int c) { return pieces64 ? 128 * (c >> 1) + 64 * half + 32 * (c & 1) : 32 * (half + 2 * c); };
                const int blocks = rag_blocks<DIR, I8>(P, it), mine = end(blocks) - begin(blocks);
                const int segs = I8 ? (mine > 0 ? 1 : 0) : (mine + seg_blocks - 1) / seg_blocks;
                float sum[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[c][j] = 0.0f;
                bool ok = true;
                for (int sg = 0; sg < segs; ++sg) {
                    if (!wait_acc()) { ok = false; break; }
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int c0 = column(c);
                        if (c0 < it.width) {
                            float v[32];
                            tmem_ld32(lanes + (uint32_t)(buf * 256 + c0), v);
#pragma unroll
                            for (int j = 0; j < 32; j += 2) {
                                if (I8) {  // one segment, of integers
                                    sum[c][j] = v[j];
                                    sum[c][j + 1] = v[j + 1];
                                } else {
                                    add2(sum[c][j], sum[c][j + 1], v[j], v[j + 1]);
                                }
                            }
                        }
                    }
                    release_acc();
                }
                if (!ok) break;
                if (SPLIT) {
                    // the last accumulator is written, so every load has been consumed: the ring is free
                    float* parts = reinterpret_cast<float*>(ring);
                    const int f = q * 32 + lane;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int c0 = 32 * (half + 2 * c);
                        if (c0 < it.width) {
                            if (DIR == RAG_TN) {
#pragma unroll
                                for (int j = 0; j < 32; j += 4)
                                    *reinterpret_cast<float4*>(parts + f * (P.bn + 4) + c0 + j) =
                                        make_float4(sum[c][j], sum[c][j + 1], sum[c][j + 2], sum[c][j + 3]);
                            } else {
#pragma unroll
                                for (int j = 0; j < 32; ++j) parts[(c0 + j) * 128 + f] = sum[c][j];
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int c0 = column(c);
                        if (c0 < it.width) {
                            if (DIR != RAG_TN) {
                                if (MODE == RAG_LONG) rag_store_rows(P, stage, it.row0 + c0, it.width - c0, f0, sum[c]);
                                else rag_store_rows_f32(P, stage, it.row0 + c0, it.width - c0, f0, sum[c]);
                            } else if (MODE == RAG_PROMOTE) {
                                rag_store_f32_tile<true>(P, stage, base, f0, it.col0 + c0, sum[c]);
                            } else if (P.accumulate) {
                                rag_store_f32_tile<false>(P, stage, base, f0, it.col0 + c0, sum[c]);
                            } else {  // a piece is two chunks, or the tile ends in its first
                                rag_stage_h16(stage, 4 * (c & 1), sum[c], P.out == MOE_BF16);
                                if ((c & 1) || c0 + 32 >= it.width) rag_store_h16_tile(P, stage, base, f0, it.col0 + (c0 & ~63));
                            }
                        }
                    }
                }
                continue;
            }
            const float first_scale = rag_scale_first(sw_ahead), last_scale = rag_scale_last(sw_ahead);
            if (AHEAD) {
#pragma unroll
                for (int c = 0; c < 4; ++c) scales[32 * c + lane] = sx_ahead[c];
                __syncwarp();
                load_scales(i + item_step);
            }
            if (!wait_acc()) break;
            const uint32_t t0 = lanes + (uint32_t)(buf * 256);
            if (DIR == RAG_TN) {
                for (int c0 = 64 * half; c0 < it.width && f0 < P.n; c0 += 128) {
                    float v[32];
                    const bool wide = P.out != MOE_F32 && !P.accumulate;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        tmem_ld32(t0 + (uint32_t)(c0 + 32 * h), v);
                        if (wide) {
                            rag_stage_h16(stage, 4 * h, v, P.out == MOE_BF16);
                        } else if (P.out == MOE_F32) {
                            rag_store_f32_tile<true>(P, stage, base, f0, it.col0 + c0 + 32 * h, v);
                        } else {
                            rag_store_f32_tile<false>(P, stage, base, f0, it.col0 + c0 + 32 * h, v);
                        }
                    }
                    if (wide) rag_store_h16_tile(P, stage, base, f0, it.col0 + c0);
                }
            } else {
                for (int h = chunks0;; ++h) {  // the warp's chunks of 32 columns: every other one from h on
                    for (int c0 = 32 * h; c0 < it.width && f0 < P.n; c0 += 64) {
                        float v[32];
                        tmem_ld32(t0 + (uint32_t)c0, v);
                        if (I8) {
                            const float* st = scales + (c0 >> 6) * 32;
#pragma unroll
                            for (int j = 0; j < 32; j += 4) {
                                const float4 s4 = *reinterpret_cast<const float4*>(st + j);
#pragma unroll
                                for (int l = 0; l < 4; ++l) v[j + l] = (float)__float_as_int(v[j + l]);
                                mul2(v[j], v[j + 1], first_scale, first_scale);
                                mul2(v[j + 2], v[j + 3], first_scale, first_scale);
                                mul2(v[j], v[j + 1], s4.x, s4.y);
                                mul2(v[j + 2], v[j + 3], s4.z, s4.w);
                                mul2(v[j], v[j + 1], last_scale, last_scale);
                                mul2(v[j + 2], v[j + 3], last_scale, last_scale);
                            }
                        }
                        rag_store_rows(P, stage, it.row0 + c0, it.width - c0, f0, v);
                    }
                    if (!alternate || h == 1) break;
                    if (AHEAD && it.width > 32) {
                        __syncwarp();
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int r = 32 + 64 * c + lane;
                            if (r < it.width) scales[32 * c + lane] = __ldg(P.sx + it.row0 + r);
                        }
                        __syncwarp();
                    }
                }
            }
            release_acc();
        }
        if (SPLIT) {
            __syncwarp();
            cluster_sync_all();  // every part is in its CTA's shared memory
            if (first < total && !*abort_flag) {
                const RagItem it = walk.at(first);
                if (DIR != RAG_TN || it.rows > 0 || !P.accumulate)
                    rag_store_parts<DIR, I8>(P, ring, (int)rank, 2, part, warp - RAG_EPI_WARP0, it.g,
                                             it.m * 256 + (int)rank * 128, it.row0, it.col0, it.width);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    settle_copies(abort_flag);
    cluster_sync_all();  // no CTA leaves while its peer may still signal it or read its part
    if (warp == 4) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base);
    }
}

}  // namespace moe

// The products of moe_ragged.cuh where they have too few tiles to occupy the GPU: few
// rows, narrow outputs, or a weight gradient of few tiles over many rows.
//
// Tiles are smaller than there (128 features by P.bn <= 128 columns, one CTA each) and the summed
// axis is cut over the P.split <= 16 CTAs of a cluster, one tile a cluster.  Each CTA sums its
// part; the parts meet through distributed shared memory: after a cluster barrier CTA s
// adds its share of the tile's rows over all parts, in the parts' order, and stores it.
// No workspace, no atomics, the same result every time.
//
// Sums stay in fp32 registers of the epilogue (segments of RAG_SEGMENT terms, as PROMOTE
// there) or in 32-bit integers.
//
// Measured (B200): 16 rows, 18432 -> 7168 in int8, two CTAs a tile: 26 us, of which the 132
// MB of weights stream for 20 (6.7 TB/s), 3 pass before the first and 3 after the last; in
// 56 tiles without a split 35 us.  256 rows in 16 groups, 256 -> 128: 5.7 us, all latency.
#pragma once

#include "moe_ragged.cuh"

namespace moe {

// Warps: 0-2 load, 4 issues the MMAs, 5 zeroes TN's tail rows, 8-15 are the epilogue, as in
// moe_ragged.cuh.
constexpr int SPLIT_EPI_WARP0 = 8;
constexpr int SPLIT_EPI_WARPS = 8;
constexpr int SPLIT_THREADS = (SPLIT_EPI_WARP0 + SPLIT_EPI_WARPS) * 32;
constexpr int SPLIT_MAX_STAGES = 12;
constexpr int SPLIT_TMEM_COLS = 256;  // two accumulators of 128 columns
constexpr int SPLIT_BARS = 3 * SPLIT_MAX_STAGES + 5;
constexpr int SPLIT_MISC = (SPLIT_BARS * 8 + (2 + SPLIT_THREADS / 32) * 4 + 15) / 16 * 16;
constexpr int SPLIT_TABLE = 3 * RAG_MAX_GROUPS * 4 + 16;

// Bytes of the ring, which also holds the finished part of the tile: 128 x bn values, a
// row 16 bytes longer in TN so that its 16-byte pieces miss each other's banks.
constexpr int split_ring_bytes(int bn, int stages) {
    const int ring = stages * (RAG_SLOT + bn * 128), part = 128 * (bn + 4) * 4;
    return ring > part ? ring : part;
}
constexpr int split_smem_bytes(int bn, int stages) {
    return 1024 + split_ring_bytes(bn, stages) + SPLIT_TABLE + SPLIT_MISC;
}

__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar,
                                            uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void mma_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

template <int DIR, bool I8>
__global__ void __launch_bounds__(SPLIT_THREADS, 1) moe_split_kernel(const __grid_constant__ RaggedArgs P) {
    const int2 head = rag_first_offsets(P);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* ring = smem;
    const int bn = P.bn, stages = P.stages;
    const int stage_bytes = RAG_SLOT + bn * 128;
    RagTable tab;
    tab.start = reinterpret_cast<int*>(smem + split_ring_bytes(bn, stages));
    tab.count = tab.start + RAG_MAX_GROUPS;
    tab.first = tab.count + RAG_MAX_GROUPS;
    uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(tab.start) + SPLIT_TABLE);
    uint64_t* full = bars;                           // stage ready for the MMA
    uint64_t* empty = full + SPLIT_MAX_STAGES;       // stage consumed
    uint64_t* landed = empty + SPLIT_MAX_STAGES;     // TN: the stage's bytes, in the block with tail rows
    uint64_t* tfull = landed + SPLIT_MAX_STAGES;     // [2] accumulator written
    uint64_t* tempty = tfull + 2;                    // [2] accumulator read
    uint64_t* drain = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + SPLIT_BARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* warp_sums = reinterpret_cast<int*>(tmem_slot + 2);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();

    if (threadIdx.x < SPLIT_BARS) {
        const uint64_t* b = &bars[threadIdx.x];
        mbar_init(&bars[threadIdx.x], b == tempty || b == tempty + 1 ? SPLIT_EPI_WARPS : 1);
        fence_mbar_init();
    } else if (threadIdx.x == SPLIT_THREADS - 1) {
        *abort_flag = 0;
        tma_prefetch_desc(&P.a);
        tma_prefetch_desc(&P.b64);
    }
    if (warp == 4) tmem_alloc<SPLIT_TMEM_COLS>(tmem_slot);
    const int mt = (P.n + 127) >> 7;
    rag_build_table<SPLIT_THREADS>(P, tab, warp_sums, head, [&](int rows) {
        return mt * rag_chunks<DIR>(P, rows);
    });
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    // This cluster's tile.  The grid is an upper bound: clusters behind the last tile leave.
    // (Every division here is on the way to the first load; a run-time one costs about 150 clocks.)
    const int tile = (int)cluster_id();
    const bool work = tile < tab.first[P.groups];
    int g = 0, f0 = 0, row0 = 0, rows = 0, col0 = 0, width = 0;
    if (work) {
        g = rag_group(tab, P.groups, tile);
        const int local = tile - tab.first[g];
        row0 = tab.start[g];
        rows = tab.count[g];
        const int nc = rag_chunks<DIR>(P, rows);
        // chunks that share weights run together
        const int m = nc == 1 ? local : local < 1 << 20 ? quotient(local, __fdividef(1.0f, (float)nc)) : local / nc;
        const int c = local - m * nc;
        f0 = m * 128;
        if (DIR == RAG_TN) {
            col0 = c * bn;
            width = min(bn, P.k - col0);
        } else {
            const int w = nc == 1 ? bn : ((rows + nc - 1) / nc + 15) & ~15;  // equal chunks
            row0 += c * w;
            width = min(w, rows - c * w);
        }
    }
    constexpr int block_k = I8 ? 128 : 64;
    constexpr int seg_blocks = I8 ? 1 << 30 : RAG_SEGMENT / 64;
    const int len = DIR == RAG_TN ? rows : P.k;
    const int all_blocks = work ? (len + block_k - 1) / block_k : 0;
    const int kb0 = P.split == 1 ? 0 : rag_share(P, all_blocks, rank);
    const int kb1 = P.split == 1 ? all_blocks : rag_share(P, all_blocks, rank + 1);
    const int mma_n = DIR == RAG_TN ? (width + 63) & ~63 : (width + 15) & ~15;

    const int q = warp & 3, half = (warp - SPLIT_EPI_WARP0) >> 2;
    bool ok = true;

    if (warp < 4) {
        const bool works = warp == 0 || warp == 2 || (warp == 1 && DIR != RAG_NT);
        if (works && elect_one()) {
            const bool is_a = warp < 2;
            const int half = (warp & 1) * 64;  // of A
            // weights that one chunk reads stream; those of several chunks stay for the others
            const uint64_t policy = DIR == RAG_TN || !is_a ? l2_policy_evict_normal()
                                    : tab.count[g] > bn   ? l2_policy_evict_last() : l2_policy_evict_first();
            const bool second = mma_n > 64;  // TN: B has a second 64-column block
            const uint32_t bytes = RAG_SLOT + (DIR == RAG_TN ? (second ? 2u : 1u) * RAG_TN_BLOCK : (uint32_t)bn * 128u);
            int slot = 0;
            uint32_t phase = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait_bounded(&empty[slot], phase ^ 1u, abort_flag)) break;
                uint8_t* dst = ring + slot * stage_bytes + (is_a ? 0 : RAG_SLOT) + half * 128;
                const bool tail = DIR == RAG_TN && kb == all_blocks - 1 && (rows & 15);
                uint64_t* bar = tail ? &landed[slot] : &full[slot];
                if (warp == 0) mbar_arrive_expect_tx(bar, bytes);
                if (DIR == RAG_TN) {
                    if (is_a) {
                        tma_load_2d(dst, &P.a, f0 + half, row0 + kb * 64, bar, policy);
                    } else {
                        tma_load_2d(dst, &P.b64, col0, row0 + kb * 64, bar, policy);
                        if (second) tma_load_2d(dst + RAG_TN_BLOCK, &P.b64, col0 + 64, row0 + kb * 64, bar, policy);
                    }
                } else if (!is_a) {
                    tma_load_2d(dst, &P.b64, kb * block_k, row0, bar, policy);
                } else if (DIR == RAG_NT) {
                    tma_load_3d(dst, &P.a, kb * block_k, f0, g, bar, policy);
                } else {
                    tma_load_3d(dst, &P.a, f0 + half, kb * 64, g, bar, policy);
                }
                if (++slot == stages) { slot = 0; phase ^= 1u; }
            }
        }
    } else if (warp == 4) {
        if (elect_one()) {
            constexpr uint64_t a_step = DIR == RAG_NT ? 2 : 128, b_step = DIR == RAG_TN ? 128 : 2;
            constexpr int per_step = I8 ? 32 : 16;
            const uint32_t ring_addr = smem_u32(ring);
            const uint64_t ad0 = DIR == RAG_NT ? smem_desc_sw128(ring_addr) : smem_desc_mn_sw128(ring_addr);
            const uint64_t bd0 = DIR == RAG_TN ? smem_desc_mn_sw128(ring_addr + RAG_SLOT)
                                               : smem_desc_sw128(ring_addr + RAG_SLOT);
            const uint64_t stage_step = (uint64_t)(stage_bytes >> 4);
            const uint32_t idesc = rag_idesc<DIR, I8>((uint32_t)P.bf16, 128, (uint32_t)mma_n);
            int slot = 0, buf = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool fine = true, issued = false;
            for (int s0 = kb0; fine && s0 < kb1; s0 += min(seg_blocks, kb1 - s0)) {
                const int s1 = s0 + min(seg_blocks, kb1 - s0);
                if (!mbar_wait_bounded(&tempty[buf], ((acc_phase >> buf) & 1u) ^ 1u, abort_flag)) break;
                const uint32_t d = tmem_base + (uint32_t)(buf * 128);
                for (int kb = s0; kb < s1; ++kb) {
                    if (!mbar_wait_bounded(&full[slot], phase, abort_flag)) { fine = false; break; }
                    tc_fence_after();
                    const uint64_t ad = ad0 + stage_step * slot, bd = bd0 + stage_step * slot;
                    const int steps = min(4, (len - kb * block_k + per_step - 1) / per_step);
                    if (steps == 4) {
#pragma unroll
                        for (int s = 0; s < 4; ++s) {
                            const uint32_t accum = (kb > s0 || s != 0) ? 1u : 0u;
                            if (I8) mma_i8(d, ad + a_step * s, bd + b_step * s, idesc, accum);
                            else mma_bf16(d, ad + a_step * s, bd + b_step * s, idesc, accum);
                        }
                    } else {
                        for (int s = 0; s < steps; ++s) {
                            const uint32_t accum = (kb > s0 || s != 0) ? 1u : 0u;
                            if (I8) mma_i8(d, ad + a_step * s, bd + b_step * s, idesc, accum);
                            else mma_bf16(d, ad + a_step * s, bd + b_step * s, idesc, accum);
                        }
                    }
                    mma_commit(&empty[slot]);
                    issued = true;
                    if (++slot == stages) { slot = 0; phase ^= 1u; }
                }
                if (!fine) break;
                mma_commit(&tfull[buf]);
                acc_phase ^= 1u << buf;
                buf ^= 1;
            }
            if (*abort_flag && issued) {
                mma_commit(drain);
                volatile int dummy = 0;
                mbar_wait_bounded(drain, 0, &dummy, 100000000ull);
            }
        }
    } else if (warp == 5) {
        if (DIR == RAG_TN && kb1 == all_blocks && kb1 > kb0 && (rows & 15)) {
            // this CTA has the group's last rows: zeros behind them (see moe_ragged.cuh)
            const int slot = (kb1 - 1 - kb0) % stages;
            if (__all_sync(0xffffffffu, mbar_wait_bounded(&landed[slot], 0, abort_flag))) {
                const int r0 = rows - (kb1 - 1) * 64, n = ((r0 + 15) & ~15) - r0;
                const int blocks = 2 + (mma_n > 64 ? 2 : 1);
                for (int j = lane; j < n * blocks * 8; j += 32) {
                    const int row = r0 + j / (blocks * 8), blk = (j >> 3) % blocks, piece = j & 7;
                    *reinterpret_cast<uint4*>(ring + slot * stage_bytes + blk * RAG_TN_BLOCK + row * 128 + piece * 16) =
                        make_uint4(0, 0, 0, 0);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[slot]);
            }
        }
    } else if (warp >= SPLIT_EPI_WARP0) {
        // ------------------------------------------------------------ the part's sums
        float sum[2][32];  // this thread's feature, columns 32 (half + 2 c) + j; integers as bits
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j) sum[c][j] = 0.0f;
        int buf = 0;
        uint32_t acc_phase = 0;
        for (int s0 = kb0; s0 < kb1; s0 += min(seg_blocks, kb1 - s0)) {
            int got = 0;
            if (lane == 0) got = mbar_wait_bounded(&tfull[buf], (acc_phase >> buf) & 1u, abort_flag) ? 1 : 0;
            got = __shfl_sync(0xffffffffu, got, 0);
            if (!got) { ok = false; break; }
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int c0 = 32 * (half + 2 * c);
                if (c0 < width) {
                    float v[32];
                    tmem_ld32(tmem_base + (uint32_t)(buf * 128 + c0) + ((uint32_t)(q * 32) << 16), v);
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        if (I8) {  // one segment
                            sum[c][j] = v[j];
                            sum[c][j + 1] = v[j + 1];
                        } else {
                            add2(sum[c][j], sum[c][j + 1], v[j], v[j + 1]);
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[buf]);
            acc_phase ^= 1u << buf;
            buf ^= 1;
        }
        // The last accumulator is written, so every load has been consumed: the ring is free.
        // A CTA without blocks has loaded nothing.
        // NT, NN: part[column][feature]; TN: part[feature][column], rows of bn + 4.
        if (ok) {
            float* part = reinterpret_cast<float*>(ring);
            const int f = q * 32 + lane;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int c0 = 32 * (half + 2 * c);
                if (c0 < width) {
                    if (DIR == RAG_TN) {
#pragma unroll
                        for (int j = 0; j < 32; j += 4)
                            *reinterpret_cast<float4*>(part + f * (bn + 4) + c0 + j) =
                                make_float4(sum[c][j], sum[c][j + 1], sum[c][j + 2], sum[c][j + 3]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (c0 + j < bn) part[(c0 + j) * 128 + f] = sum[c][j];
                    }
                }
            }
        }
    }

    // All parts are in their CTAs' shared memory.  (A CTA that gave up has set the error word; its
    // peers go on with what is there.)
    const bool stores = warp >= SPLIT_EPI_WARP0 && work && !(all_blocks == 0 && P.accumulate);
    __syncwarp();
    if (P.split > 1) cluster_sync_all();
    else if (stores) named_bar_sync(1, SPLIT_EPI_WARPS * 32);
    if (stores && !*abort_flag) {
        rag_store_parts<DIR, I8>(P, ring, 0, 1, rank, warp - SPLIT_EPI_WARP0, g, f0, row0, col0, width);
    }
    __syncwarp();
    if (P.split > 1) cluster_sync_all();  // no CTA leaves while another reads its part
    tc_fence_before();
    __syncthreads();
    if (warp == 4) {
        tc_fence_after();
        tmem_dealloc<SPLIT_TMEM_COLS>(tmem_base);
        settle_copies(abort_flag);
    }
}

}  // namespace moe

// C ABI of the products grouped by expert and the row operators around them
// (include/moe.h): argument checks, tensor maps, launches.  Host code only.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "../../include/moe.h"
#include "moe_host.h"
#include "moe_launch.h"

using namespace moe;

namespace {

constexpr int kMaxWidth = 65536;     // n, k: 128 * 128 * 65536 = 2^30, so 8-bit sums stay inside 32 bits
constexpr int kMaxRows = 1 << 24;    // items of all groups stay inside 32 bits
constexpr int kMaxQuantWidth = 32768;  // a row in registers: 512 threads of four 16-value pieces
// Clocks besides the blocks': of a pair kernel's launch and of each of its tiles, of each
// round of the split kernel (whose CTAs start anew for every tile), of the meeting of parts
// and of each of their columns.
constexpr int kPairClocks = 6000, kPairTileClocks = 2500, kSplitTileClocks = 8000, kMeetClocks = 1500, kMeetColumnClocks = 17;
// Terms that the tensor core may sum alone for a 16-bit result: it then comes out small by at most
// 2^-27 of its value a term, an eighth of its half step (2^-11 and 2^-8).
constexpr int kWholeF16 = 1 << 13, kWholeBF16 = 1 << 16;
constexpr int64_t kMaxLd = 1ll << 36;

int size_of(moe_dtype t) { return t == MOE_F32 ? 4 : 2; }
bool is_float(moe_dtype t) { return t == MOE_F32 || t == MOE_BF16 || t == MOE_F16; }
moe_status refused(moe_dtype t) { return is_float(t) || t == MOE_E4M3 ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
// distance of rows: holds a row and keeps every row on a 16-byte boundary
bool good_ld(int64_t ld, int width, int elem) { return ld >= width && ld <= kMaxLd && (ld * elem) % 16 == 0; }

// Whether two matrices of `rows` rows share bytes (p: address, ld: bytes from row to row, w:
// bytes of a row).  Columns of one wider buffer do not; different row distances over a
// common range count as sharing.
struct Rows {
    const void* p;
    int64_t ld, w;
};
bool share(const Rows& a, const Rows& b, int rows) {
    const int64_t pa = (int64_t)reinterpret_cast<uintptr_t>(a.p), pb = (int64_t)reinterpret_cast<uintptr_t>(b.p);
    const int64_t ea = pa + (rows - 1) * a.ld + a.w, eb = pb + (rows - 1) * b.ld + b.w;
    if (ea <= pb || eb <= pa) return false;
    if (a.ld != b.ld) return true;
    const int64_t d = ((pb - pa) % a.ld + a.ld) % a.ld;  // b's columns start d bytes behind a's
    return d < a.w || a.ld - d < b.w;
}
bool same(const Rows& a, const Rows& b) { return a.p == b.p && a.ld == b.ld; }
// one block of bytes against rows
bool share(const void* p, size_t bytes, const Rows& r, int rows) {
    return share(Rows{p, (int64_t)bytes, (int64_t)bytes}, Rows{r.p, (rows - 1) * r.ld + r.w, (rows - 1) * r.ld + r.w}, 1);
}
// the same of a vector that may be absent (offsets, scales, coefficients, a count)
bool vector_in(const void* p, int64_t count, const Rows& r, int rows) { return p && share(p, (size_t)count * 4, r, rows); }

// Shapes and flags that every product checks; k_step: elements of 16 bytes of the operands.
moe_status check_product(int groups, int rows, int n, int k, int k_step, const int32_t* offsets, moe_dtype out,
                         moe_dtype operands, int accumulate) {
    if (groups < 1 || groups > RAG_MAX_GROUPS || rows < 0 || rows > kMaxRows) return MOE_ERR_INVALID_ARG;
    if (n < 8 || n > kMaxWidth || n % 8 != 0 || k < k_step || k > kMaxWidth || k % k_step != 0)
        return MOE_ERR_INVALID_ARG;
    if ((!offsets && groups != 1) || !aligned4(offsets) || (accumulate != 0 && accumulate != 1))
        return MOE_ERR_INVALID_ARG;
    if (!is_float(out)) return MOE_ERR_INVALID_ARG;
    if (out != MOE_F32 && out != operands) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// Tiled map of 128-byte-swizzled boxes over [depth][rows][cols] (depth 0: two
// dimensions), rows ld elements apart; elements outside read as zero.
bool map_box(CUtensorMap* m, CUtensorMapDataType dt, int elem, const void* p, uint64_t depth, uint64_t rows,
             uint64_t cols, uint64_t ld, uint32_t box_rows) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[3] = {cols, rows, depth};
    const cuuint64_t strides[2] = {ld * elem, ld * elem * rows};
    const cuuint32_t box[3] = {(cuuint32_t)(128 / elem), box_rows, 1};
    const cuuint32_t ones[3] = {1, 1, 1};
    return enc(m, dt, depth ? 3 : 2, const_cast<void*>(p), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

CUtensorMapDataType map_type(moe_dtype t) {
    return t == MOE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

// Which kernel runs a product, from what the host knows: the sizes, not the offsets.
//
// pair: moe_ragged_kernel, tiles of 256 features x bn columns on CTA pairs, with split > 1 the
// summed axis over that many pairs; else moe_split_kernel, tiles of 128 x bn on single CTAs
// with the summed axis over `split` of them.  Both take a block of 128 bytes of the summed
// axis at a time, and a CTA gets about 45 bytes a clock into shared memory, so a block of a
// tile with c columns a CTA costs (128 + c) * 128 / 45 clocks, and a product its rounds of
// tiles times its blocks.  The cheapest of the choices runs; a split also pays for its
// meeting.  Measured (us; the choice first):
//   222 rows, n 3272, k 18432         four pairs of 256 columns 32, two of 128 44, two CTAs 46, no split 65
//   16 rows, 7168, 18432, int8        two CTAs of 16 columns 25.5, two pairs 27.5, no split 35
//   1024 rows, 7168, 2048             pairs of 256 columns 26, of 128 30, single CTAs 56
//   512 rows in 8 groups, 2048, 1024  pairs of 128 columns 8.8, single CTAs 10.1
//   1785 rows, 256, 2688              four pairs of 128 11.2, four CTAs 10.9, no split 12.7
//   gradient 544 x 488, 47337 rows    eight pairs 46, six CTAs 64, pairs without a split 190
struct ProductPlan {
    bool pair;
    int grid;         // pair: CTAs
    int bn, split;
    long long tiles;  // split kernel: at most
};

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// chunks of at most w rows that the groups of a NT / NN product can have
long long chunks_of(int groups, int rows, int w) {
    return groups == 1 ? ceil_div(rows, w) : rows / w + (groups < rows ? groups : rows);
}

ProductPlan plan_product(int dir, bool i8, int groups, int rows, int n, int k, int n_sm) {
    const int sms = n_sm & ~1;
    const long long mean = ceil_div(rows, groups < rows ? groups : rows);  // rows of a group that has some
    const int blocks = (int)(dir == RAG_TN ? ceil_div(mean, 64) : ceil_div(k, i8 ? 128 : 64));
    // columns a tile has in fact: no more than a chunk has rows
    auto wide = [&](int bn) { return dir == RAG_TN || mean >= bn ? bn : (int)((mean + 31) & ~31ll); };
    auto columns = [&](int bn) { return dir == RAG_TN ? groups * ceil_div(k, bn) : chunks_of(groups, rows, bn); };
    ProductPlan best = {};
    double best_cost = 0.0;
    auto offer = [&](bool pair, int bn, int split, long long tiles, int at_once, int once, int each) {
        const double rounds = (double)((tiles + at_once - 1) / at_once);
        const double cost = once + rounds * ((blocks + split - 1) / split * ((128 + (pair ? wide(bn) / 2 : bn)) * 128 / 45) + each);
        if (best_cost > 0.0 && cost >= best_cost) return;
        best_cost = cost;
        best.pair = pair;
        best.bn = bn;
        best.split = split;
        best.tiles = tiles;
        best.grid = (int)(split > 1 ? 2 * split * tiles : 2 * tiles < sms ? 2 * tiles : sms);
    };
    for (int bn = 256; bn >= 128; bn /= 2) {
        const long long tiles = columns(bn) * ceil_div(n, 256);
        offer(true, bn, 1, tiles, sms / 2, kPairClocks, kPairTileClocks);
        if (tiles >= 2 * sms) return best;  // rounds enough for the rest of the last not to matter
    }
    // a split: parts of four blocks at least (a shorter one is over before its pipeline is full),
    // and every cluster running at once
    const int* at_once = split_clusters();
    for (int bn = 256; bn >= 128; bn /= 2) {
        const long long tiles = columns(bn) * ceil_div(n, 256);
        for (int split = 2; 2 * split <= SPLIT_MAX_CLUSTER && 4 * split <= blocks && tiles <= at_once[2 * split]; ++split)
            offer(true, bn, split, tiles, at_once[2 * split], kPairClocks, kPairTileClocks + kMeetClocks + bn * kMeetColumnClocks);
    }
    for (int bn = 128; bn >= (dir == RAG_TN ? 64 : 16); bn /= 2) {
        const long long tiles = columns(bn) * ceil_div(n, 128);
        for (int split = 1; split <= SPLIT_MAX_CLUSTER && (split == 1 || 4 * split <= blocks); ++split) {
            if (split > 1 && tiles > at_once[split]) break;
            if (at_once[split] > 0)
                offer(false, bn, split, tiles, at_once[split], split > 1 ? kMeetClocks + bn * kMeetColumnClocks : 0,
                      kSplitTileClocks);
        }
    }
    return best;
}

moe_status run_product(int dir, bool i8, RaggedArgs* a, const ProductPlan& p, cudaStream_t s) {
    a->bn = p.bn;
    while ((1 << a->bn_shift) < p.bn) ++a->bn_shift;
    a->split = p.split;
    a->whole = (a->out == MOE_F16 ? kWholeF16 : kWholeBF16) / 64;
    return cuda_status(p.pair ? launch_ragged(dir, i8, a, p.grid, s) : launch_split(dir, i8, a, p.tiles, s));
}

moe_status product(bool i8, moe_dtype t, int groups, int rows, int n, int k, const void* x, int64_t ldx, const void* w,
                   int transpose_w, const float* sx, const float* sw, const int32_t* offsets, void* y, int64_t ldy,
                   moe_dtype out, int accumulate, moe_stream_t stream) {
    DevInfo di;
    const moe_status st = check_device(&di);
    if (st != MOE_OK) return st;
    RaggedArgs a;
    memset(&a, 0, sizeof(a));
    const int elem = i8 ? 1 : 2;
    const CUtensorMapDataType dt = i8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : map_type(t);
    const int dir = transpose_w ? RAG_NN : RAG_NT;
    const ProductPlan plan = plan_product(dir, i8, groups, rows, n, k, di.sm_count);
    bool ok = transpose_w ? map_box(&a.a, dt, elem, w, groups, k, n, n, 64)
                          : map_box(&a.a, dt, elem, w, groups, n, k, k, 128);
    if (plan.pair) {
        ok = ok && map_box(&a.b128, dt, elem, x, 0, rows, k, ldx, 128) &&
             map_box(&a.b64, dt, elem, x, 0, rows, k, ldx, 64) && map_box(&a.b16, dt, elem, x, 0, rows, k, ldx, 16);
    } else {
        ok = ok && map_box(&a.b64, dt, elem, x, 0, rows, k, ldx, plan.bn);
    }
    if (!ok) return MOE_ERR_CUDA;
    a.offsets = offsets;
    a.groups = groups;
    a.rows = rows;
    a.n = n;
    a.k = k;
    a.bf16 = t == MOE_BF16;
    a.y = y;
    a.ldy = ldy;
    a.out = out;
    a.accumulate = accumulate;
    a.sx = sx;
    a.sw = sw;
    return run_product(dir, i8, &a, plan, (cudaStream_t)stream);
}

}  // namespace

extern "C" {

moe_status moe_grouped_mm(int groups, int rows, int n, int k, moe_dtype dtype, const void* x, int64_t ldx,
                          const void* w, int transpose_w, const int32_t* offsets, void* y, int64_t ldy,
                          moe_dtype y_dtype, int accumulate, moe_stream_t stream) {
    NvtxRange nv("moe.grouped_mm");
    if (dtype != MOE_BF16 && dtype != MOE_F16) return refused(dtype);
    const moe_status st = check_product(groups, rows, n, k, 8, offsets, y_dtype, dtype, accumulate);
    if (st != MOE_OK) return st;
    if (transpose_w != 0 && transpose_w != 1) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!x || !w || !y || !aligned16(x) || !aligned16(w) || !aligned16(y)) return MOE_ERR_INVALID_ARG;
    if (!good_ld(ldx, k, 2) || !good_ld(ldy, n, size_of(y_dtype))) return MOE_ERR_INVALID_ARG;
    const Rows rx = {x, ldx * 2, k * 2}, ry = {y, ldy * size_of(y_dtype), n * size_of(y_dtype)};
    if (share(rx, ry, rows) || share(w, (size_t)groups * n * k * 2, ry, rows) || vector_in(offsets, groups + 1, ry, rows))
        return MOE_ERR_INVALID_ARG;
    return product(false, dtype, groups, rows, n, k, x, ldx, w, transpose_w, nullptr, nullptr, offsets, y, ldy,
                   y_dtype, accumulate, stream);
}

moe_status moe_grouped_mm_int8(int groups, int rows, int n, int k, const int8_t* q, const float* sx, const int8_t* w,
                               const float* sw, const int32_t* offsets, void* y, int64_t ldy, moe_dtype y_dtype,
                               int accumulate, moe_stream_t stream) {
    NvtxRange nv("moe.grouped_mm_int8");
    const moe_status st = check_product(groups, rows, n, k, 16, offsets, y_dtype, y_dtype, accumulate);
    if (st != MOE_OK) return st;
    if (rows == 0) return MOE_OK;
    if (!q || !w || !y || !sx || !sw || !aligned16(q) || !aligned16(w) || !aligned16(y) || !aligned4(sx) ||
        !aligned4(sw) || !good_ld(ldy, n, size_of(y_dtype)))
        return MOE_ERR_INVALID_ARG;
    const Rows rq = {q, k, k}, ry = {y, ldy * size_of(y_dtype), n * size_of(y_dtype)};
    if (share(rq, ry, rows) || share(w, (size_t)groups * n * k, ry, rows) || vector_in(offsets, groups + 1, ry, rows) ||
        vector_in(sx, rows, ry, rows) || vector_in(sw, (int64_t)groups * n, ry, rows))
        return MOE_ERR_INVALID_ARG;
    return product(true, y_dtype, groups, rows, n, k, q, k, w, 0, sx, sw, offsets, y, ldy, y_dtype, accumulate, stream);
}

moe_status moe_grouped_wgrad(int groups, int rows, int n, int k, moe_dtype dtype, const void* dy, int64_t lddy,
                             const void* x, int64_t ldx, const int32_t* offsets, void* dw, moe_dtype dw_dtype,
                             int accumulate, moe_stream_t stream) {
    NvtxRange nv("moe.grouped_wgrad");
    if (dtype != MOE_BF16 && dtype != MOE_F16) return refused(dtype);
    moe_status st = check_product(groups, rows, n, k, 8, offsets, dw_dtype, dtype, accumulate);
    if (st != MOE_OK) return st;
    if (!dw || !aligned16(dw)) return MOE_ERR_INVALID_ARG;
    if (rows && (!dy || !x || !aligned16(dy) || !aligned16(x) || !good_ld(lddy, n, 2) || !good_ld(ldx, k, 2)))
        return MOE_ERR_INVALID_ARG;
    const size_t dw_bytes = (size_t)groups * n * k * size_of(dw_dtype);
    if (rows && (share(dw, dw_bytes, Rows{dy, lddy * 2, n * 2}, rows) || share(dw, dw_bytes, Rows{x, ldx * 2, k * 2}, rows)))
        return MOE_ERR_INVALID_ARG;
    if (vector_in(offsets, groups + 1, Rows{dw, (int64_t)dw_bytes, (int64_t)dw_bytes}, 1)) return MOE_ERR_INVALID_ARG;
    DevInfo di;
    if ((st = check_device(&di)) != MOE_OK) return st;
    if (rows == 0) {  // a sum of nothing
        if (accumulate) return MOE_OK;
        const cudaError_t e = cudaMemsetAsync(dw, 0, dw_bytes, (cudaStream_t)stream);
        if (e != cudaSuccess) cudaGetLastError();  // not left for the next call's check
        return cuda_status(e);
    }
    RaggedArgs a;
    memset(&a, 0, sizeof(a));
    if (!map_box(&a.a, map_type(dtype), 2, dy, 0, rows, n, lddy, 64) ||
        !map_box(&a.b64, map_type(dtype), 2, x, 0, rows, k, ldx, 64))
        return MOE_ERR_CUDA;
    a.b128 = a.b16 = a.b64;
    a.offsets = offsets;
    a.groups = groups;
    a.rows = rows;
    a.n = n;
    a.k = k;
    a.bf16 = dtype == MOE_BF16;
    a.y = dw;
    a.out = dw_dtype;
    a.accumulate = accumulate;
    return run_product(RAG_TN, false, &a, plan_product(RAG_TN, false, groups, rows, n, k, di.sm_count), (cudaStream_t)stream);
}

moe_status moe_swiglu(int rows, int width, moe_dtype dtype, const void* gate, int64_t ld_gate, const void* up,
                      int64_t ld_up, const float* coef, const int32_t* n_rows, void* h, int64_t ld_h,
                      moe_stream_t stream) {
    NvtxRange nv("moe.swiglu");
    if (!is_float(dtype)) return refused(dtype);
    if (rows < 0 || rows > kMaxRows || width < 8 || width > kMaxWidth || width % 8 != 0) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    const int e = size_of(dtype);
    if (!gate || !up || !h || !aligned16(gate) || !aligned16(up) || !aligned16(h) || !aligned4(coef) ||
        !aligned4(n_rows) || !good_ld(ld_gate, width, e) || !good_ld(ld_up, width, e) || !good_ld(ld_h, width, e))
        return MOE_ERR_INVALID_ARG;
    const int64_t wide = (int64_t)width * e;
    const Rows rg = {gate, ld_gate * e, wide}, ru = {up, ld_up * e, wide}, rh = {h, ld_h * e, wide};
    if ((share(rg, rh, rows) && !same(rg, rh)) || (share(ru, rh, rows) && !same(ru, rh))) return MOE_ERR_INVALID_ARG;
    if (vector_in(coef, rows, rh, rows) || vector_in(n_rows, 1, rh, rows)) return MOE_ERR_INVALID_ARG;
    DevInfo di;
    const moe_status st = check_device(&di);
    if (st != MOE_OK) return st;
    SwigluArgs a;
    memset(&a, 0, sizeof(a));
    a.gate = gate;
    a.up = up;
    a.out0 = h;
    a.coef = coef;
    a.n_rows = n_rows;
    a.ld_gate = ld_gate;
    a.ld_up = ld_up;
    a.ld_out0 = ld_h;
    a.rows = rows;
    a.width = width;
    return cuda_status(launch_swiglu(false, dtype, a, di.sm_count, (cudaStream_t)stream));
}

moe_status moe_swiglu_backward(int rows, int width, moe_dtype dtype, const void* dh, int64_t ld_dh, const void* gate,
                               int64_t ld_gate, const void* up, int64_t ld_up, const float* coef,
                               const int32_t* n_rows, void* dgate, int64_t ld_dgate, void* dup, int64_t ld_dup,
                               float* dcoef, moe_stream_t stream) {
    NvtxRange nv("moe.swiglu_backward");
    if (!is_float(dtype)) return refused(dtype);
    if (rows < 0 || rows > kMaxRows || width < 8 || width > kMaxWidth || width % 8 != 0) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    const int e = size_of(dtype);
    if (!dh || !gate || !up || !dgate || !dup || !aligned16(dh) || !aligned16(gate) || !aligned16(up) ||
        !aligned16(dgate) || !aligned16(dup) || !aligned4(coef) || !aligned4(n_rows) || !aligned4(dcoef) ||
        !good_ld(ld_dh, width, e) || !good_ld(ld_gate, width, e) || !good_ld(ld_up, width, e) ||
        !good_ld(ld_dgate, width, e) || !good_ld(ld_dup, width, e))
        return MOE_ERR_INVALID_ARG;
    const int64_t wide = (int64_t)width * e;
    const Rows in[3] = {{dh, ld_dh * e, wide}, {gate, ld_gate * e, wide}, {up, ld_up * e, wide}};
    const Rows out[2] = {{dgate, ld_dgate * e, wide}, {dup, ld_dup * e, wide}};
    if (share(out[0], out[1], rows)) return MOE_ERR_INVALID_ARG;
    for (const Rows& i : in)
        for (const Rows& o : out)
            if (share(i, o, rows) && !same(i, o)) return MOE_ERR_INVALID_ARG;
    for (const Rows& o : out)
        if (vector_in(coef, rows, o, rows) || vector_in(n_rows, 1, o, rows) || vector_in(dcoef, rows, o, rows))
            return MOE_ERR_INVALID_ARG;
    if (dcoef) {  // may be coef itself: a row's threads have read it before its sum is complete
        const Rows rc = {dcoef, (int64_t)rows * 4, (int64_t)rows * 4};
        for (const Rows& i : in)
            if (vector_in(dcoef, rows, i, rows)) return MOE_ERR_INVALID_ARG;
        if ((coef != dcoef && vector_in(coef, rows, rc, 1)) || vector_in(n_rows, 1, rc, 1)) return MOE_ERR_INVALID_ARG;
    }
    DevInfo di;
    const moe_status st = check_device(&di);
    if (st != MOE_OK) return st;
    SwigluArgs a;
    memset(&a, 0, sizeof(a));
    a.gate = gate;
    a.up = up;
    a.dh = dh;
    a.out0 = dgate;
    a.out1 = dup;
    a.coef = coef;
    a.dcoef = dcoef;
    a.n_rows = n_rows;
    a.ld_gate = ld_gate;
    a.ld_up = ld_up;
    a.ld_dh = ld_dh;
    a.ld_out0 = ld_dgate;
    a.ld_out1 = ld_dup;
    a.rows = rows;
    a.width = width;
    return cuda_status(launch_swiglu(true, dtype, a, di.sm_count, (cudaStream_t)stream));
}

moe_status moe_quantize_int8(const void* x, moe_dtype dtype, int64_t ldx, int rows, int k, const int32_t* n_rows,
                             int8_t* q, float* sx, moe_stream_t stream) {
    NvtxRange nv("moe.quantize_int8");
    if (!is_float(dtype)) return refused(dtype);
    if (rows < 0 || rows > kMaxRows || k < 16 || k > kMaxQuantWidth || k % 16 != 0) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!x || !q || !sx || !aligned16(x) || !aligned16(q) || !aligned4(sx) || !aligned4(n_rows) ||
        !good_ld(ldx, k, size_of(dtype)))
        return MOE_ERR_INVALID_ARG;
    const Rows rx = {x, ldx * size_of(dtype), (int64_t)k * size_of(dtype)}, rq = {q, k, k};
    const Rows rs = {sx, (int64_t)rows * 4, (int64_t)rows * 4};
    if (share(q, (size_t)rows * k, rx, rows) || vector_in(sx, rows, rx, rows) || vector_in(sx, rows, rq, rows) ||
        vector_in(n_rows, 1, rq, rows) || vector_in(n_rows, 1, rs, 1))
        return MOE_ERR_INVALID_ARG;
    DevInfo di;
    const moe_status st = check_device(&di);
    if (st != MOE_OK) return st;
    return cuda_status(
        launch_quantize_int8(x, dtype, ldx, rows, k, n_rows, q, sx, di.sm_count, (cudaStream_t)stream));
}

}  // extern "C"

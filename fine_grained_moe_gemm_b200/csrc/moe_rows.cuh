// Row operators around the grouped products: SwiGLU with its gradient, and the
// per-row int8 codes.  All three are bound by HBM at large sizes: every value is read
// once and written once, in 16-byte pieces, and the row sums stay in registers.
#pragma once

#include <cuda_fp16.h>

#include "moe_device.cuh"
#include "moe_launch.h"

namespace moe {

constexpr int ROWS_THREADS = 256;

// Rows to compute: all, or the device count (outside [0, rows]: none, and an error bit).
__device__ __forceinline__ int rows_to_compute(const int* n_rows, int rows) {
    if (!n_rows) return rows;
    const int n = __ldg(n_rows);
    if (n >= 0 && n <= rows) return n;
    if (blockIdx.x == 0 && threadIdx.x == 0) set_dev_error(MOE_DEVERR_BAD_ROWS);
    return 0;
}

template <typename T>
struct Vec16 {  // 16 bytes of T as floats
    static constexpr int N = 16 / (int)sizeof(T);
    float v[N];
};

__device__ __forceinline__ void vec_load(const float* p, Vec16<float>& o) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    o.v[0] = u.x; o.v[1] = u.y; o.v[2] = u.z; o.v[3] = u.w;
}
__device__ __forceinline__ void vec_load(const __nv_bfloat16* p, Vec16<__nv_bfloat16>& o) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o.v[2 * i] = __uint_as_float(w[i] << 16);
        o.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void vec_load(const __half* p, Vec16<__half>& o) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        o.v[2 * i] = f.x;
        o.v[2 * i + 1] = f.y;
    }
}
// each value rounded once, to nearest even
__device__ __forceinline__ void vec_store(float* p, const Vec16<float>& o) {
    *reinterpret_cast<float4*>(p) = make_float4(o.v[0], o.v[1], o.v[2], o.v[3]);
}
__device__ __forceinline__ void vec_store(__nv_bfloat16* p, const Vec16<__nv_bfloat16>& o) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(o.v[2 * i], o.v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void vec_store(__half* p, const Vec16<__half>& o) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(o.v[2 * i], o.v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// sigmoid(z): exp(-z) overflows to infinity below -88 and the quotient is then 0, off by
// less than the smallest normal number.  16-bit values take the fast exponential and
// quotient (a few fp32 ulps, far below their half step); fp32 ones the accurate ones.
template <typename T>
__device__ __forceinline__ float row_sigmoid(float z) {
    if (sizeof(T) == 4) return 1.0f / (1.0f + expf(-z));
    return __fdividef(1.0f, 1.0f + __expf(-z));
}

// h = c * silu(gate) * up.  tx threads (a power of two) share a row, ROWS_THREADS / tx rows
// a CTA.  h may be gate or up: a thread writes only pieces it has read.
template <typename T>
__global__ void __launch_bounds__(ROWS_THREADS) swiglu_kernel(const __grid_constant__ SwigluArgs A, int tx) {
    constexpr int V = Vec16<T>::N;
    const int t = threadIdx.x & (tx - 1);
    const int ty = ROWS_THREADS / tx;
    const int rows = rows_to_compute(A.n_rows, A.rows);
    for (int r = blockIdx.x * ty + threadIdx.x / tx; r < rows; r += gridDim.x * ty) {
        const T* g = static_cast<const T*>(A.gate) + (size_t)r * A.ld_gate;
        const T* u = static_cast<const T*>(A.up) + (size_t)r * A.ld_up;
        T* h = static_cast<T*>(A.out0) + (size_t)r * A.ld_out0;
        const float c = A.coef ? A.coef[r] : 1.0f;
        for (int i = t * V; i < A.width; i += tx * V) {
            Vec16<T> a, b;
            vec_load(g + i, a);
            vec_load(u + i, b);
#pragma unroll
            for (int j = 0; j < V; ++j) a.v[j] = c * (a.v[j] * row_sigmoid<T>(a.v[j]) * b.v[j]);
            vec_store(h + i, a);
        }
    }
}

// dgate = c dh up (s + silu (1 - s)), dup = c dh silu, dcoef = sum dh silu up, with
// s = sigmoid(gate), silu = gate s.  dgate may be gate and dup may be up or dh.
// Bound by HBM: 131072 rows of 2048 in bf16 (2.7 GB) take 419 us, 98 % of the copy rate.
// With one warp to a row the sum needs no barrier; two, four or eight warps take 440, 450
// and 483 us, and two or four pieces of a thread loaded together 474 and 540 us (fewer
// warps fit).
template <typename T>
__global__ void __launch_bounds__(ROWS_THREADS) swiglu_backward_kernel(const __grid_constant__ SwigluArgs A, int tx) {
    constexpr int V = Vec16<T>::N;
    __shared__ float part[2][ROWS_THREADS / 32];
    const int t = threadIdx.x & (tx - 1);
    const int ty = ROWS_THREADS / tx;
    const int rows = rows_to_compute(A.n_rows, A.rows);
    int flip = 0;
    // every thread of the CTA makes the same number of turns (the reduction may synchronise)
    for (int r0 = blockIdx.x * ty; r0 < rows; r0 += gridDim.x * ty) {
        const int r = r0 + threadIdx.x / tx;
        float dot = 0.0f;
        if (r < rows) {
            const T* g = static_cast<const T*>(A.gate) + (size_t)r * A.ld_gate;
            const T* u = static_cast<const T*>(A.up) + (size_t)r * A.ld_up;
            const T* d = static_cast<const T*>(A.dh) + (size_t)r * A.ld_dh;
            T* dg = static_cast<T*>(A.out0) + (size_t)r * A.ld_out0;
            T* du = static_cast<T*>(A.out1) + (size_t)r * A.ld_out1;
            const float c = A.coef ? A.coef[r] : 1.0f;
            for (int i = t * V; i < A.width; i += tx * V) {
                Vec16<T> a, b, e;
                vec_load(g + i, a);
                vec_load(u + i, b);
                vec_load(d + i, e);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float s = row_sigmoid<T>(a.v[j]);
                    const float act = a.v[j] * s;
                    const float ce = c * e.v[j];
                    dot = fmaf(e.v[j] * act, b.v[j], dot);
                    a.v[j] = ce * b.v[j] * fmaf(act, 1.0f - s, s);
                    b.v[j] = ce * act;
                }
                vec_store(dg + i, a);
                vec_store(du + i, b);
            }
        }
        if (A.dcoef) {  // fixed order: lanes by a butterfly, then the row's warps one after another
            for (int o = min(tx, 32) >> 1; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
            if (tx > 32) {
                if ((threadIdx.x & 31) == 0) part[flip][threadIdx.x >> 5] = dot;
                __syncthreads();
                if (t == 0) {
                    for (int w = 1; w < (tx >> 5); ++w) dot += part[flip][(threadIdx.x >> 5) + w];
                }
                flip ^= 1;  // the next row's partials do not overwrite these before they are read
            }
            if (t == 0 && r < rows) A.dcoef[r] = dot;
        }
    }
}

// ---------------------------------------------------------------- int8 codes
// Sixteen values as they lie in memory, and pairs of them in fp32.
template <typename T>
struct Raw16 {
    uint4 u[sizeof(T)];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T); ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ uint32_t word(int i) const {
        const uint4& v = u[i >> 2];
        return (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
    }
    // values 2 i and 2 i + 1
    __device__ __forceinline__ float2 pair(int i) const;
    // Largest magnitude by its bits: non-negative floats order as integers, and a NaN's
    // bits lie above infinity's, so it wins.  `m` starts at 0; 16-bit types keep a maximum
    // for each half of a word.
    __device__ __forceinline__ uint32_t magnitude(uint32_t m) const;
};
template <> __device__ __forceinline__ float2 Raw16<float>::pair(int i) const {
    return make_float2(__uint_as_float(word(2 * i)), __uint_as_float(word(2 * i + 1)));
}
template <> __device__ __forceinline__ float2 Raw16<__nv_bfloat16>::pair(int i) const {
    return make_float2(__uint_as_float(word(i) << 16), __uint_as_float(word(i) & 0xffff0000u));
}
template <> __device__ __forceinline__ float2 Raw16<__half>::pair(int i) const {
    const uint32_t w = word(i);
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <> __device__ __forceinline__ uint32_t Raw16<float>::magnitude(uint32_t m) const {
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, word(i) & 0x7fffffffu);
    return m;
}
template <> __device__ __forceinline__ uint32_t Raw16<__nv_bfloat16>::magnitude(uint32_t m) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, word(i) & 0x7fff7fffu);
    return m;
}
template <> __device__ __forceinline__ uint32_t Raw16<__half>::magnitude(uint32_t m) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, word(i) & 0x7fff7fffu);
    return m;
}
// fp32 bits of a thread's maximum
template <typename T>
__device__ __forceinline__ uint32_t magnitude_f32(uint32_t m) { return m; }
template <>
__device__ __forceinline__ uint32_t magnitude_f32<__nv_bfloat16>(uint32_t m) { return max(m & 0xffffu, m >> 16) << 16; }
template <>
__device__ __forceinline__ uint32_t magnitude_f32<__half>(uint32_t m) {
    return __float_as_uint(__half2float(__ushort_as_half((unsigned short)max(m & 0xffffu, m >> 16))));
}

// The integer nearest to the real quotient x / s, ties to even, in [-127, 127]: the
// checked form of code_word below for one value.
__device__ __forceinline__ int code_of(float x, float s, float inv) {
    float c = rintf(x * inv);
    const float rem = fmaf(-c, s, x);
    const float twice = 2.0f * fabsf(rem);
    if (twice > s || (twice == s && ((int)c & 1))) c += copysignf(1.0f, rem);
    return (int)fminf(fmaxf(c, -127.0f), 127.0f);
}

// Four codes in a word.  t = x / s + 1.5 2^23 rounds the quotient to an integer c whose low
// byte is t's; x * (1/s) is off by less than 3e-5, so c is the nearest integer or one off
// next to a tie.  x - c s is exact in fp32 (a multiple of an ulp of s or of x, no larger
// than s): below s / 2 it proves c, and `worst` keeps the largest for that test.  Six
// instructions a value (two values at a time in fp32x2); the tie's own test for each value
// would take twelve, and at 6.5 TB/s a value has sixteen issue slots.
__device__ __forceinline__ uint32_t code_word(float2 x0, float2 x1, float s, float inv, float& worst) {
    const float magic = 12582912.0f;
    float t0 = magic, t1 = magic, t2 = magic, t3 = magic;
    fma2(t0, t1, x0.x, x0.y, inv, inv);
    fma2(t2, t3, x1.x, x1.y, inv, inv);
    float r0 = x0.x, r1 = x0.y, r2 = x1.x, r3 = x1.y;
    fma2(r0, r1, magic - t0, magic - t1, s, s);
    fma2(r2, r3, magic - t2, magic - t3, s, s);
    worst = fmaxf(fmaxf(worst, fabsf(r0)), fabsf(r1));
    worst = fmaxf(fmaxf(worst, fabsf(r2)), fabsf(r3));
    const uint32_t lo = __byte_perm(__float_as_uint(t0), __float_as_uint(t1), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(t2), __float_as_uint(t3), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}

// sx[r] = max |x[r]| * (1/127) (1 if that is zero), q = codes.  tx threads (a power of two,
// a warp at least) share a row, which stays in registers between the two passes: NV
// pieces of 16 values a thread.  Bound by HBM: 16384 rows of 7168 in bf16 (352 MB) take
// 58-64 us; 69 when the next row's loads wait for this one's stores, and with 64, 128 or 512
// threads to a row instead of 256 (7, 4 or 1 pieces each) 65, 69 and 98.  Few rows take one
// piece a thread: 128 rows 3.7 us, with two 4.8.
template <typename T, int NV>
__global__ void __launch_bounds__(512) quantize_int8_kernel(const T* __restrict__ x, long long ldx, int n, int k,
                                                            const int* n_rows, int8_t* __restrict__ q,
                                                            float* __restrict__ sx, int tx) {
    __shared__ uint32_t part[2][16];
    const int t = threadIdx.x & (tx - 1);
    const int ty = blockDim.x / tx;
    const int rows = rows_to_compute(n_rows, n);
    int flip = 0;
    Raw16<T> v[NV], next[NV];
    auto load = [&](Raw16<T>(&d)[NV], int r) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * tx) * 16;
            if (r < rows && c < k) d[i].load(x + (size_t)r * ldx + c);
        }
    };
    load(next, blockIdx.x * ty + threadIdx.x / tx);
    for (int r0 = blockIdx.x * ty; r0 < rows; r0 += gridDim.x * ty) {
        const int r = r0 + threadIdx.x / tx;
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            v[i] = next[i];
            if (r < rows && (t + i * tx) * 16 < k) m = v[i].magnitude(m);
        }
        load(next, r + gridDim.x * ty);  // under way while this row is worked on
        m = __reduce_max_sync(0xffffffffu, magnitude_f32<T>(m));
        if (tx > 32) {
            if ((threadIdx.x & 31) == 0) part[flip][threadIdx.x >> 5] = m;
            __syncthreads();
            const int w0 = (threadIdx.x / tx) * (tx >> 5);
            for (int w = 0; w < (tx >> 5); ++w) m = max(m, part[flip][w0 + w]);
            flip ^= 1;
        }
        if (r >= rows) continue;
        float s = __fmul_rn(__uint_as_float(m), 1.0f / 127.0f);
        if (s == 0.0f) s = 1.0f;
        if (t == 0) sx[r] = s;
        // an infinity or a NaN in the row: the scale is not finite and the codes are zero
        const bool bad = !(s < __uint_as_float(0x7f800000u));
        // tiny scales: x and s times 2^64 (exact), so that 1/s and x - c s stay normal
        const bool tiny = s < 0x1p-60f;
        const float lift = tiny ? 0x1p64f : 1.0f;
        const float ss = s * lift, inv = 1.0f / ss;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * tx) * 16;
            if (c >= k) continue;
            uint32_t w[4];
            float worst = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = code_word(v[i].pair(2 * j), v[i].pair(2 * j + 1), ss, inv, worst);
            if (bad || tiny || !(worst < 0.5f * ss)) {  // a tie or a code one off (about 1 in 10^5 values): each checked
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 a = v[i].pair(2 * j), b = v[i].pair(2 * j + 1);
                    const float f[4] = {a.x, a.y, b.x, b.y};
                    uint32_t u = 0;
#pragma unroll
                    for (int l = 0; l < 4; ++l)
                        u |= bad ? 0u : (uint32_t)(code_of(f[l] * lift, ss, inv) & 0xff) << (8 * l);
                    w[j] = u;
                }
            }
            *reinterpret_cast<uint4*>(q + (size_t)r * k + c) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

}  // namespace moe

// q4_mx_pack.cu -- quantise to the microscaled 4-bit format and back.
//
// Per group of 32 weights with largest magnitude a: the exponent byte is
// floor(log2 a) - 2 + 127, at least 0 (e2m1's largest value 6 = 1.5 * 2^2 then
// covers [4, 8) * scale up to saturation), and each code is w * 2^(127 - byte)
// rounded to the nearest e2m1 value, ties to the even code, saturating at 6.
// The byte is a's exponent field minus 2, and the division is a product with a
// power of two, so every step but the one rounding is exact and the result is
// that of any serial IEEE implementation.  A group with an infinity or NaN
// gets byte 255 (NaN); rows and columns that pad a block hold zeros, byte 0.
//
// Both directions are bound by memory.  A CTA of 256 threads owns one block:
// 16 threads a row, 8 weights each, 16 rows a pass, so that a pass writes 1 KB
// of codes in one piece and every thread has its 8 passes' loads in flight.
#include <algorithm>

#include "q4_mx.cuh"

namespace q4 {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerPass = kThreads / 16;
constexpr int kPasses = kMxBlock / kRowsPerPass;

// Eight consecutive weights as binary32; kVector: one or two 16-byte loads.
template <typename T, bool kVector>
__device__ __forceinline__ void load8(const T* p, int64_t first, int64_t count, int64_t extent, float (&v)[8]) {
    if (kVector) {
        constexpr int kWords = 8 * sizeof(T) / 16;
        union {
            uint4 q[kWords];
            T t[8];
        } u;
#pragma unroll
        for (int i = 0; i < kWords; ++i) u.q[i] = make_uint4(0, 0, 0, 0);
        if (count >= 8 && Q4_IN_BOUNDS(first, 8, extent)) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) u.q[i] = __ldcs(reinterpret_cast<const uint4*>(p + first) + i);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = Element<T>::get(u.t[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = i < count && Q4_IN_BOUNDS(first + i, 1, extent) ? Element<T>::get(p[first + i]) : 0.0f;
    }
}

// Eight binary32 values as e2m1 codes, the first in the low nibble.
__device__ __forceinline__ uint32_t to_e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Four code bytes as eight binary16 values (exact).
__device__ __forceinline__ void from_e2m1x8(uint32_t codes, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
}

template <typename T, bool kVector>
__global__ void __launch_bounds__(kThreads)
    pack_mx_kernel(const T* __restrict__ w, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int64_t E,
                   int64_t N, int64_t K, int64_t Nb, int64_t Kb) {
    const int64_t block = blockIdx.x, kb = block % Kb, nb = block / Kb % Nb, e = block / Kb / Nb;
    const int part = threadIdx.x % 16, row0 = threadIdx.x / 16;
    const int64_t k = kb * kMxBlock + 8 * part;
    float v[kPasses][8];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int64_t n = nb * kMxBlock + row0 + i * kRowsPerPass;
        const int64_t count = n < N ? K - k : 0;
        load8<T, kVector>(w, (e * N + n) * K + k, count, E * N * K, v[i]);
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        uint32_t top = 0;  // largest magnitude, as the bits of a non-negative number
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        const uint32_t field = top >> 23;
        const uint32_t byte = field == 255u ? 255u : field > 2u ? field - 2u : 0u;
        const float inverse = byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
        uint32_t packed = 0;
        if (byte != 255u) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] *= inverse;
            packed = to_e2m1x8(v[i]);
        }
        // the row's four exponent bytes, gathered by the first of its 16 threads
        const int first = threadIdx.x & 16;
        const uint32_t b0 = __shfl_sync(0xFFFFFFFFu, byte, first), b1 = __shfl_sync(0xFFFFFFFFu, byte, first + 4),
                       b2 = __shfl_sync(0xFFFFFFFFu, byte, first + 8),
                       b3 = __shfl_sync(0xFFFFFFFFu, byte, first + 12);
        const int row = row0 + i * kRowsPerPass;
        const int64_t at = block * kMxCodeBytes + row * 64 + 4 * part;
        if (Q4_IN_BOUNDS(at, 4, E * Nb * Kb * kMxCodeBytes)) *reinterpret_cast<uint32_t*>(codes + at) = packed;
        const int64_t sat = block * kMxScaleBytes + mx_scale_at(row, 0);
        if (part == 0 && Q4_IN_BOUNDS(sat, 4, E * Nb * Kb * kMxScaleBytes))
            *reinterpret_cast<uint32_t*>(scales + sat) = b0 | b1 << 8 | b2 << 16 | b3 << 24;
    }
}

template <typename T, bool kVector>
__global__ void __launch_bounds__(kThreads)
    dequant_mx_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, T* __restrict__ w,
                      int64_t E, int64_t N, int64_t K, int64_t Nb, int64_t Kb) {
    const int64_t block = blockIdx.x, kb = block % Kb, nb = block / Kb % Nb, e = block / Kb / Nb;
    const int part = threadIdx.x % 16, row0 = threadIdx.x / 16;
    const int64_t k = kb * kMxBlock + 8 * part;
    uint32_t packed[kPasses], byte[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int row = row0 + i * kRowsPerPass;
        const int64_t at = block * kMxCodeBytes + row * 64 + 4 * part;
        const int64_t sat = block * kMxScaleBytes + mx_scale_at(row, part / 4);
        packed[i] = Q4_IN_BOUNDS(at, 4, E * Nb * Kb * kMxCodeBytes)
                        ? __ldcs(reinterpret_cast<const uint32_t*>(codes + at)) : 0u;
        byte[i] = Q4_IN_BOUNDS(sat, 1, E * Nb * Kb * kMxScaleBytes) ? __ldg(scales + sat) : 0u;
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int64_t n = nb * kMxBlock + row0 + i * kRowsPerPass;
        if (n >= N || k >= K) continue;
        uint32_t h[4];
        from_e2m1x8(packed[i], h);
        const float scale = mx_scale_value(byte[i]);
        constexpr int kWords = 8 * sizeof(T) / 16;
        union {
            uint4 q[kWords];
            T t[8];
        } u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
            u.t[2 * j] = Element<T>::put(f.x * scale);
            u.t[2 * j + 1] = Element<T>::put(f.y * scale);
        }
        const int64_t first = (e * N + n) * K + k;
        if (kVector) {
            if (Q4_IN_BOUNDS(first, 8, E * N * K)) {
#pragma unroll
                for (int j = 0; j < kWords; ++j) __stcs(reinterpret_cast<uint4*>(w + first) + j, u.q[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (k + j < K && Q4_IN_BOUNDS(first + j, 1, E * N * K)) w[first + j] = u.t[j];
        }
    }
}

template <typename T>
cudaError_t pack_as(const void* w, uint8_t* codes, uint8_t* scales, int64_t E, int64_t N, int64_t K, cudaStream_t s) {
    const int64_t Nb = mx_blocks(N), Kb = mx_blocks(K);
    const unsigned grid = static_cast<unsigned>(E * Nb * Kb);
    // rows that are whole 8-weight pieces load 16 bytes at a time
    if (K % 8 == 0)
        pack_mx_kernel<T, true><<<grid, kThreads, 0, s>>>(static_cast<const T*>(w), codes, scales, E, N, K, Nb, Kb);
    else
        pack_mx_kernel<T, false><<<grid, kThreads, 0, s>>>(static_cast<const T*>(w), codes, scales, E, N, K, Nb, Kb);
    return cudaGetLastError();
}

template <typename T>
cudaError_t dequant_as(const uint8_t* codes, const uint8_t* scales, void* w, int64_t E, int64_t N, int64_t K,
                       cudaStream_t s) {
    const int64_t Nb = mx_blocks(N), Kb = mx_blocks(K);
    const unsigned grid = static_cast<unsigned>(E * Nb * Kb);
    if (K % 8 == 0)
        dequant_mx_kernel<T, true><<<grid, kThreads, 0, s>>>(codes, scales, static_cast<T*>(w), E, N, K, Nb, Kb);
    else
        dequant_mx_kernel<T, false><<<grid, kThreads, 0, s>>>(codes, scales, static_cast<T*>(w), E, N, K, Nb, Kb);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_pack_mx(const void* w, int type, uint8_t* codes, uint8_t* scales, int64_t E, int64_t N,
                           int64_t K, cudaStream_t s) {
    if (type == Q4_F32) return pack_as<float>(w, codes, scales, E, N, K, s);
    if (type == Q4_BF16) return pack_as<__nv_bfloat16>(w, codes, scales, E, N, K, s);
    return pack_as<__half>(w, codes, scales, E, N, K, s);
}

cudaError_t launch_dequant_mx(const uint8_t* codes, const uint8_t* scales, void* w, int type, int64_t E,
                              int64_t N, int64_t K, cudaStream_t s) {
    if (type == Q4_F32) return dequant_as<float>(codes, scales, w, E, N, K, s);
    if (type == Q4_BF16) return dequant_as<__nv_bfloat16>(codes, scales, w, E, N, K, s);
    return dequant_as<__half>(codes, scales, w, E, N, K, s);
}

Q4_DEFINE_TAKE_BOUNDS(mx_pack)

}  // namespace q4

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
// Both directions are bound by memory: on B200 6.7 TB/s for a binary32 matrix
// of 16384 x 8192 (91 us), 5.9 TB/s for a bfloat16 one of 57344 x 8192 (202 us;
// the instructions for each weight bound it there), 6.4 and 6.6 TB/s back.
// A CTA of 256 threads owns part of a block.  Where rows are whole 16-byte
// pieces, 16 threads share a row, 8 weights each, and every thread has all its
// rows' loads in flight.  Else (K not a multiple of 8), and for a
// binary32 dequant whose 32 bytes a thread would leave gaps in each store, a
// warp takes a row and lane l the weights l, l + 32, l + 64, l + 96: loads and
// stores of whole lines whatever the alignment.
#include <algorithm>
#include <cstring>

#include "q4_mx.cuh"

namespace q4 {
namespace {

constexpr int kThreads = 256;
// Rows of a block that a CTA owns: few, so that small matrices use every SM.
// A 2-byte type in kManyBlocks blocks or more does better with wider pieces
// (57344 x 8192 bfloat16): packing takes two blocks of k a CTA (202 us, one
// block 259), writing values back 64 rows (179 us, 32 rows 211).
constexpr int kFew = 32;
constexpr int kMany = 64;
constexpr int64_t kManyBlocks = 1024;

// The block of a CTA, one of `parts` of that block (there are fewer than 2^24).
struct Place {
    uint32_t kb, nb, e;
    __device__ Place(uint32_t Nb, uint32_t Kb, uint32_t parts) {
        const uint32_t block = blockIdx.x / parts, row = block / Kb;
        kb = block - row * Kb;
        e = row / Nb;
        nb = row - e * Nb;
    }
};

// Eight consecutive weights as they are stored.
template <typename T>
struct Eight {
    static constexpr int kWords = 8 * sizeof(T) / 16;
    union {
        uint4 q[kWords];
        uint32_t w[4 * kWords];
    };
    // zeros where the row has ended
    __device__ void load(const T* p, bool in) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) q[i] = in ? __ldcs(reinterpret_cast<const uint4*>(p) + i) : make_uint4(0, 0, 0, 0);
    }
    // Bits of the largest magnitude as a binary32; above those of infinity if
    // there is a NaN.  Magnitudes order as their bits do, two of 16 bits at a time.
    __device__ uint32_t top() const {
        if (sizeof(T) == 4) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 4 * kWords; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
            return m;
        }
        uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
        for (int i = 1; i < 4 * kWords; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
        const uint32_t one = max(m & 0xFFFFu, m >> 16);
        return __float_as_uint(value16(one));
    }
    static __device__ float value16(uint32_t bits) {
        if (sizeof(T) == 4) return 0.0f;
        T t;
        const uint16_t h = static_cast<uint16_t>(bits);
        memcpy(&t, &h, 2);
        return Element<T>::get(t);
    }
    __device__ float get(int i) const {
        if (sizeof(T) == 4) return __uint_as_float(w[i]);
        return value16(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu);
    }
};

// The exponent byte of a group whose largest magnitude has these bits, and
// 2^(127 - byte) (0 for the byte of NaN).
__device__ __forceinline__ uint32_t group_byte(uint32_t top) {
    const uint32_t field = top >> 23;
    return field == 255u ? 255u : field > 2u ? field - 2u : 0u;
}
__device__ __forceinline__ float group_inverse(uint32_t byte) {
    return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
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

// Two of either, the first in the low nibble.
__device__ __forceinline__ uint32_t to_e2m1x2(float a, float b) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.u32.u8 %0, b0;\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 from_e2m1x2(uint32_t codes) {
    uint32_t h;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t}"
        : "=r"(h)
        : "r"(codes));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
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

// kWide: blocks of k that a CTA covers, so that it reads rows in pieces of 512 bytes.
template <typename T, int kRows, int kWide>
__global__ void __launch_bounds__(kThreads)
    pack_mx_kernel(const T* __restrict__ w, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int64_t E,
                   int64_t N, int64_t K, int64_t Nb, int64_t Kb) {
    constexpr int kParts = kMxBlock / kRows, kRowsPerPass = kThreads / (16 * kWide), kPasses = kRows / kRowsPerPass;
    const Place place(static_cast<uint32_t>(Nb), static_cast<uint32_t>((Kb + kWide - 1) / kWide), kParts);
    const int part = threadIdx.x % 16, row0 = blockIdx.x % kParts * kRows + threadIdx.x / (16 * kWide);
    const int64_t nb = place.nb, e = place.e, kb = place.kb * kWide + threadIdx.x / 16 % kWide;
    const int64_t block = (e * Nb + nb) * Kb + kb, k = kb * kMxBlock + 8 * part;
    const int64_t n0 = nb * kMxBlock + row0, first = (e * N + n0) * K + k;
    const int rows = k < K ? static_cast<int>(min(N - n0, static_cast<int64_t>(kMxBlock))) : 0;
    Eight<T> v[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const bool in = i * kRowsPerPass < rows && Q4_IN_BOUNDS(first + i * kRowsPerPass * K, 8, E * N * K);
        v[i].load(w + first + i * kRowsPerPass * K, in);
    }
    const int64_t at0 = block * kMxCodeBytes + row0 * 64 + 4 * part;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        uint32_t top = v[i].top();
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        const uint32_t byte = group_byte(top);
        const float inverse = group_inverse(byte);
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = v[i].get(j) * inverse;
        const uint32_t packed = byte == 255u ? 0u : to_e2m1x8(f);
        if (kb >= Kb) continue;
        const int row = row0 + i * kRowsPerPass;
        const int64_t at = at0 + i * kRowsPerPass * 64, sat = block * kMxScaleBytes + mx_scale_at(row, part / 4);
        if (Q4_IN_BOUNDS(at, 4, E * Nb * Kb * kMxCodeBytes)) *reinterpret_cast<uint32_t*>(codes + at) = packed;
        if (part % 4 == 0 && Q4_IN_BOUNDS(sat, 1, E * Nb * Kb * kMxScaleBytes)) scales[sat] = static_cast<uint8_t>(byte);
    }
}

template <typename T, int kRows>
__global__ void __launch_bounds__(kThreads)
    dequant_mx_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, T* __restrict__ w,
                      int64_t E, int64_t N, int64_t K, int64_t Nb, int64_t Kb) {
    constexpr int kParts = kMxBlock / kRows, kRowsPerPass = kThreads / 16, kPasses = kRows / kRowsPerPass;
    const Place place(static_cast<uint32_t>(Nb), static_cast<uint32_t>(Kb), kParts);
    const int part = threadIdx.x % 16, row0 = blockIdx.x % kParts * kRows + threadIdx.x / 16;
    const int64_t nb = place.nb, e = place.e, kb = place.kb;
    const int64_t block = (e * Nb + nb) * Kb + kb, k = kb * kMxBlock + 8 * part;
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
        if (Q4_IN_BOUNDS(first, 8, E * N * K)) {
#pragma unroll
            for (int j = 0; j < kWords; ++j) __stcs(reinterpret_cast<uint4*>(w + first) + j, u.q[j]);
        }
    }
}

// The row-a-warp forms: warp w of the CTA takes rows w, w + 8, ...
constexpr int kRowWarps = kThreads / 32;
constexpr int kRowBatch = 4;  // rows whose loads are in flight together

template <typename T>
__global__ void __launch_bounds__(kThreads)
    pack_mx_rows_kernel(const T* __restrict__ w, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                        int64_t E, int64_t N, int64_t K, int64_t Nb, int64_t Kb) {
    constexpr int kParts = kMxBlock / kFew;
    const Place place(static_cast<uint32_t>(Nb), static_cast<uint32_t>(Kb), kParts);
    const int64_t nb = place.nb, e = place.e, kb = place.kb, block = (e * Nb + nb) * Kb + kb;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t k0 = kb * kMxBlock + lane;
    const int top = blockIdx.x % kParts * kFew;
    for (int r0 = top + warp; r0 < top + kFew; r0 += kRowWarps * kRowBatch) {
        float v[kRowBatch][4];
#pragma unroll
        for (int i = 0; i < kRowBatch; ++i) {
            const int64_t n = nb * kMxBlock + r0 + i * kRowWarps;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int64_t k = k0 + 32 * g, at = (e * N + n) * K + k;
                v[i][g] = n < N && k < K && Q4_IN_BOUNDS(at, 1, E * N * K) ? Element<T>::get(__ldcs(w + at)) : 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < kRowBatch; ++i) {
            const int row = r0 + i * kRowWarps;
            uint32_t bytes = 0, code[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const uint32_t byte =
                    group_byte(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v[i][g]) & 0x7FFFFFFFu));
                bytes |= byte << (8 * g);
                // the pair's byte, in both lanes
                const float mine = v[i][g] * group_inverse(byte), other = __shfl_xor_sync(0xFFFFFFFFu, mine, 1);
                code[g] = byte == 255u ? 0u : lane & 1 ? to_e2m1x2(other, mine) : to_e2m1x2(mine, other);
            }
            // even lanes write groups 0 and 1, odd lanes 2 and 3
            const int64_t at = block * kMxCodeBytes + row * 64 + (lane & 1) * 32 + lane / 2;
            if (Q4_IN_BOUNDS(at, 17, E * Nb * Kb * kMxCodeBytes)) {
                codes[at] = static_cast<uint8_t>(lane & 1 ? code[2] : code[0]);
                codes[at + 16] = static_cast<uint8_t>(lane & 1 ? code[3] : code[1]);
            }
            const int64_t sat = block * kMxScaleBytes + mx_scale_at(row, 0);
            if (lane == 0 && Q4_IN_BOUNDS(sat, 4, E * Nb * Kb * kMxScaleBytes))
                *reinterpret_cast<uint32_t*>(scales + sat) = bytes;
        }
    }
}

// kFour: rows are whole pieces of four weights; lane l then takes 4 l .. 4 l + 3.
template <typename T, bool kFour>
__global__ void __launch_bounds__(kThreads)
    dequant_mx_rows_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                           T* __restrict__ w, int64_t E, int64_t N, int64_t K, int64_t Nb, int64_t Kb) {
    constexpr int kParts = kMxBlock / kFew;
    const Place place(static_cast<uint32_t>(Nb), static_cast<uint32_t>(Kb), kParts);
    const int64_t nb = place.nb, e = place.e, kb = place.kb, block = (e * Nb + nb) * Kb + kb;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t k0 = kb * kMxBlock + lane;
    constexpr int kRows = kFew / kRowWarps;
    const int top = blockIdx.x % kParts * kFew;
    // the codes of group l / 8 that lane l holds of a row: two bytes
    uint32_t held[kRows], bytes[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int row = top + warp + i * kRowWarps;
        const int64_t at = block * kMxCodeBytes + row * 64 + 2 * lane, sat = block * kMxScaleBytes + mx_scale_at(row, 0);
        held[i] = Q4_IN_BOUNDS(at, 2, E * Nb * Kb * kMxCodeBytes)
                      ? __ldcs(reinterpret_cast<const uint16_t*>(codes + at)) : 0u;
        bytes[i] = Q4_IN_BOUNDS(sat, 4, E * Nb * Kb * kMxScaleBytes)
                       ? __ldg(reinterpret_cast<const uint32_t*>(scales + sat)) : 0u;
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t n = nb * kMxBlock + top + warp + i * kRowWarps;
        if (n >= N) break;
        if constexpr (kFour) {
            const float scale = mx_scale_value(bytes[i] >> (8 * (lane / 8)) & 255u);
            const float2 a = from_e2m1x2(held[i]), b = from_e2m1x2(held[i] >> 8);
            union {
                uint2 two;
                uint4 four;
                T t[4];
            } u;
            u.t[0] = Element<T>::put(a.x * scale);
            u.t[1] = Element<T>::put(a.y * scale);
            u.t[2] = Element<T>::put(b.x * scale);
            u.t[3] = Element<T>::put(b.y * scale);
            const int64_t k = kb * kMxBlock + 4 * lane, at = (e * N + n) * K + k;
            if (k < K && Q4_IN_BOUNDS(at, 4, E * N * K)) {
                if (sizeof(T) == 4)
                    __stcs(reinterpret_cast<uint4*>(w + at), u.four);
                else
                    __stcs(reinterpret_cast<uint2*>(w + at), u.two);
            }
        } else {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                // weight lane + 32 g: nibble lane % 4 of the lane 8 g + lane / 4
                const uint32_t pair = __shfl_sync(0xFFFFFFFFu, held[i], 8 * g + lane / 4);
                const float f = from_e2m1x2(pair >> (4 * (lane & 3))).x;
                const int64_t k = k0 + 32 * g, at = (e * N + n) * K + k;
                if (k < K && Q4_IN_BOUNDS(at, 1, E * N * K))
                    __stcs(w + at, Element<T>::put(f * mx_scale_value(bytes[i] >> (8 * g) & 255u)));
            }
        }
    }
}

template <typename T>
cudaError_t pack_as(const void* w, uint8_t* codes, uint8_t* scales, int64_t E, int64_t N, int64_t K, cudaStream_t s) {
    const int64_t Nb = mx_blocks(N), Kb = mx_blocks(K);
    const T* src = static_cast<const T*>(w);
    const unsigned few = static_cast<unsigned>(E * Nb * Kb * (kMxBlock / kFew));
    if (K % 8 != 0)
        pack_mx_rows_kernel<T><<<few, kThreads, 0, s>>>(src, codes, scales, E, N, K, Nb, Kb);
    else if (sizeof(T) == 2 && E * Nb * Kb >= kManyBlocks)
        pack_mx_kernel<T, kFew, 2><<<static_cast<unsigned>(E * Nb * ((Kb + 1) / 2) * (kMxBlock / kFew)), kThreads, 0, s>>>(
            src, codes, scales, E, N, K, Nb, Kb);
    else
        pack_mx_kernel<T, kFew, 1><<<few, kThreads, 0, s>>>(src, codes, scales, E, N, K, Nb, Kb);
    return cudaGetLastError();
}

template <typename T>
cudaError_t dequant_as(const uint8_t* codes, const uint8_t* scales, void* w, int64_t E, int64_t N, int64_t K,
                       cudaStream_t s) {
    const int64_t Nb = mx_blocks(N), Kb = mx_blocks(K);
    T* dst = static_cast<T*>(w);
    const unsigned few = static_cast<unsigned>(E * Nb * Kb * (kMxBlock / kFew));
    if (K % 8 == 0 && sizeof(T) == 2 && E * Nb * Kb >= kManyBlocks)
        dequant_mx_kernel<T, kMany><<<static_cast<unsigned>(E * Nb * Kb * (kMxBlock / kMany)), kThreads, 0, s>>>(
            codes, scales, dst, E, N, K, Nb, Kb);
    else if (K % 8 == 0 && sizeof(T) == 2)
        dequant_mx_kernel<T, kFew><<<few, kThreads, 0, s>>>(codes, scales, dst, E, N, K, Nb, Kb);
    else if (K % 4 == 0)
        dequant_mx_rows_kernel<T, true><<<few, kThreads, 0, s>>>(codes, scales, dst, E, N, K, Nb, Kb);
    else
        dequant_mx_rows_kernel<T, false><<<few, kThreads, 0, s>>>(codes, scales, dst, E, N, K, Nb, Kb);
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

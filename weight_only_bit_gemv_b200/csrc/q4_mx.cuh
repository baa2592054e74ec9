// q4_mx.cuh -- the microscaled 4-bit format shared by the pack, product and
// expert kernels: block sizes, element types and exact conversions.
//
// W[n][k] = e2m1(code) * 2^(byte - 127), one exponent byte for 32 weights
// along K.  Storage is in blocks of 128 rows x 128 k, [ceil(N/128)][ceil(K/128)]:
// 128 rows of 64 code bytes (low nibble = even k), and 512 exponent bytes, the
// byte of row r, group g at (r % 32) * 16 + (r / 32) * 4 + g.  A block's codes
// are one contiguous 8 KB copy, and its exponents are already in the order in
// which tensor memory holds the scale factors of 128 rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "q4_internal.cuh"

namespace q4 {

constexpr int kMxBlock = 128;         // rows and k of a block
constexpr int kMxGroup = 32;          // weights per exponent byte
constexpr int kMxCodeBytes = 8192;    // codes of a block
constexpr int kMxScaleBytes = 512;    // exponent bytes of a block
constexpr int kMxMaxSms = 160;        // workspaces hold partial sums for this many CTAs

// Position of row r (0..127), group g (0..3) in a block's exponent bytes.
__host__ __device__ constexpr int mx_scale_at(int r, int g) { return (r % 32) * 16 + (r / 32) * 4 + g; }

__host__ __device__ constexpr int64_t mx_blocks(int64_t n) { return (n + kMxBlock - 1) / kMxBlock; }

// 2^(b - 127) for an exponent byte b; 255 stands for NaN.
__device__ __forceinline__ float mx_scale_value(uint32_t b) {
    return __uint_as_float(b == 255u ? 0x7FFFFFFFu : b == 0u ? 0x00400000u : b << 23);
}

template <typename T>
struct Element;
template <>
struct Element<float> {
    static __device__ __forceinline__ float get(float v) { return v; }
    static __device__ __forceinline__ float put(float v) { return v; }
};
template <>
struct Element<__nv_bfloat16> {
    static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Element<__half> {
    static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
};

inline int type_size(int t) { return t == Q4_F32 ? 4 : 2; }

// ---------------------------------------------------------------------------
// launchers (each validated by q4_api.cu before it is called)
// ---------------------------------------------------------------------------
cudaError_t launch_pack_mx(const void* w, int type, uint8_t* codes, uint8_t* scales, int64_t E, int64_t N,
                           int64_t K, cudaStream_t s);
cudaError_t launch_dequant_mx(const uint8_t* codes, const uint8_t* scales, void* w, int type, int64_t E,
                              int64_t N, int64_t K, cudaStream_t s);
// offsets == nullptr: one matrix (E = 1), T rows of x in order.
// -1: more k blocks of output tiles than 2^31 - 1.  0: none is needed.  Else
// the most that T rows or fewer need: it never falls as T grows.
int64_t gemm_mx_workspace(int64_t T, int64_t E, int64_t N, int64_t K);
cudaError_t launch_gemm_mx(const uint8_t* codes, const uint8_t* scales, const uint16_t* x,
                           const int32_t* rows, const int32_t* offsets, void* y, int y_type, int64_t Mx,
                           int64_t T, int64_t E, int64_t N, int64_t K, void* workspace, cudaStream_t s,
                           const DeviceInfo& dev);
// At most 8 tokens a tile, `split` CTAs of a cluster to a tile, no workspace.
cudaError_t launch_decode_mx(const uint8_t* codes, const uint8_t* scales, const uint16_t* x, const int32_t* rows,
                             const int32_t* offsets, void* y, int y_type, int64_t Mx, int64_t T, int64_t E, int64_t N,
                             int64_t K, int split, int groups, cudaStream_t s, const DeviceInfo& dev);
cudaError_t launch_sort_experts(const void* ids, int wide, int32_t* offsets, int32_t* rows, int32_t* places,
                                int64_t M, int64_t top, int64_t E, cudaStream_t s, const DeviceInfo& dev);
cudaError_t launch_dispatch(const void* x, const int32_t* places, void* xs, int type, int64_t M, int64_t top,
                            int64_t K, cudaStream_t s);
cudaError_t launch_combine(const void* ys, const int32_t* places, const float* weights, void* out, int type,
                           int64_t M, int64_t top, int64_t K, cudaStream_t s);
cudaError_t launch_combine_grad(const void* dout, const void* ys, const int32_t* places, const float* weights,
                                void* dys, float* dweights, int type, int64_t M, int64_t top, int64_t K,
                                cudaStream_t s);

cudaError_t take_gemm_mx_error(unsigned int* out);
cudaError_t take_decode_mx_error(unsigned int* out);
cudaError_t take_bounds_mx_pack(unsigned int* out);
cudaError_t take_bounds_mx_gemm(unsigned int* out);
cudaError_t take_bounds_mx_decode(unsigned int* out);
cudaError_t take_bounds_experts(unsigned int* out);

}  // namespace q4

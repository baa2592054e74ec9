// q4_experts.cu -- tokens sorted by expert and back: q4_sort_experts,
// q4_dispatch, q4_combine and q4_combine_grad.
#include <algorithm>

#include "q4_mx.cuh"

namespace q4 {
namespace {

// ---------------------------------------------------------------------------
// the sort
// ---------------------------------------------------------------------------
// A stable counting sort of the T = M * top choices by expert, in one launch.
// Buckets are the E experts and one more for ids outside [0, E).  Each warp
// owns a run of choices in order; it counts them per bucket, the counts are
// summed over warps, then over the CTAs of a cluster through distributed
// shared memory, and over the buckets; a second pass over the ids hands out
// the positions, lanes with equal ids finding each other by one ballot per bit
// of the bucket (match.any instead took 37 us for 131072 choices of 256
// experts: it goes through the 32 different ids one by one).  Only whole
// numbers are added atomically, so the result is fixed.  Bound by latency: two
// passes and three barriers; a warp has kSortBatch rounds of ids in flight.
// Measured on B200: 24 choices of 8 experts 3.9 us, 131072 of 256 21 us (6.3 and
// 29 to 36 us at the clock that the power cap leaves beside large products).
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortCluster = 8;  // CTAs for more choices than one CTA sorts as fast
constexpr int64_t kSortOneCta = 8192;
constexpr int kSortBatch = 8;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int cluster_load(uint32_t addr, uint32_t rank) {
    uint32_t a;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

template <typename Id>
__global__ void __launch_bounds__(kSortThreads)
    sort_experts_kernel(const Id* __restrict__ ids, int32_t* __restrict__ offsets, int32_t* __restrict__ rows,
                        int32_t* __restrict__ places, int64_t T, int top, int E) {
    extern __shared__ int smem_sort[];
    const int bits = 32 - __clz(E + 1);  // of a bucket number, or of B for no choice
    const int B = E + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int* total = smem_sort;                 // [B] choices of this CTA
    int* sums = total + B;                  // [32]
    int* count = sums + 32 + warp * B;      // [B] of this warp, then its next positions
    const uint32_t rank = cluster_rank(), size = cluster_size();
    for (int i = threadIdx.x; i < kSortWarps * B; i += kSortThreads) sums[32 + i] = 0;
    __syncthreads();

    const int64_t all = static_cast<int64_t>(size) * kSortWarps;
    const int64_t rounds = (T + 32 * all - 1) / (32 * all);  // of 32 choices per warp
    const int64_t first = (static_cast<int64_t>(rank) * kSortWarps + warp) * rounds * 32;
    // buckets of the warp's next kSortBatch rounds; B: no choice
    auto load_buckets = [&](int64_t r, int (&b)[kSortBatch]) {
#pragma unroll
        for (int q = 0; q < kSortBatch; ++q) {
            const int64_t i = first + 32 * (r + q) + lane;
            const bool in = r + q < rounds && i < T && Q4_IN_BOUNDS(i, 1, T);
            const Id id = in ? __ldg(ids + i) : 0;
            b[q] = !in ? B : id >= 0 && id < E ? static_cast<int>(id) : E;
        }
    };
    for (int64_t r = 0; r < rounds && first + 32 * r < T; r += kSortBatch) {
        int b[kSortBatch];
        load_buckets(r, b);
#pragma unroll
        for (int q = 0; q < kSortBatch; ++q)
            if (b[q] < B) atomicAdd(count + b[q], 1);
    }
    __syncthreads();
    for (int b = threadIdx.x; b < B; b += kSortThreads) {
        int sum = 0;
#pragma unroll 8
        for (int w = 0; w < kSortWarps; ++w) {
            int* c = sums + 32 + w * B + b;
            const int v = *c;
            *c = sum;
            sum += v;
        }
        total[b] = sum;
    }
    if (size > 1)
        cluster_sync();
    else
        __syncthreads();

    // threads own consecutive buckets: positions before this CTA's and bucket
    constexpr int kOwn = (Q4_MAX_EXPERTS + 1 + kSortThreads - 1) / kSortThreads;
    const int own = (B + kSortThreads - 1) / kSortThreads;
    int before[kOwn], whole[kOwn], mine = 0;
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
        const int b = threadIdx.x * own + j;
        before[j] = whole[j] = 0;
        if (j < own && b < B)
            for (uint32_t c = 0; c < size; ++c) {
                const int v = size > 1 ? cluster_load(smem_u32(total + b), c) : total[b];
                if (c < rank) before[j] += v;
                whole[j] += v;
            }
        mine += whole[j];
    }
    int scan = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, scan, d);
        if (lane >= d) scan += o;
    }
    if (lane == 31) sums[warp] = scan;
    __syncthreads();
    if (warp == 0) {
        int v = sums[lane];
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int o = __shfl_up_sync(0xFFFFFFFFu, v, d);
            if (lane >= d) v += o;
        }
        sums[lane] = v;
    }
    __syncthreads();
    int at = scan - mine + (warp ? sums[warp - 1] : 0);
    if (size > 1) cluster_sync();  // every CTA has read the others' totals
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
        const int b = threadIdx.x * own + j;
        if (j < own && b < B) {
            if (rank == 0 && Q4_IN_BOUNDS(b, 1, E + 1)) offsets[b] = at;  // offsets[E]: the choices kept
            total[b] = at + before[j];
        }
        at += whole[j];
    }
    __syncthreads();
    for (int b = lane; b < B; b += 32) count[b] += total[b];
    __syncwarp();

    for (int64_t r = 0; r < rounds && first + 32 * r < T; r += kSortBatch) {
        int b[kSortBatch];
        load_buckets(r, b);
#pragma unroll
        for (int q = 0; q < kSortBatch; ++q) {
            if (r + q >= rounds) break;
            uint32_t same = 0xFFFFFFFFu;
            for (int bit = 0; bit < bits; ++bit) {
                const bool set = b[q] >> bit & 1;
                const uint32_t who = __ballot_sync(0xFFFFFFFFu, set);
                same &= set ? who : ~who;
            }
            const int pos = b[q] < B ? count[b[q]] + __popc(same & ((1u << lane) - 1u)) : 0;
            __syncwarp();
            if (b[q] < B) {
                if (__ffs(same) - 1 == lane) count[b[q]] += __popc(same);
                const int64_t i = first + 32 * (r + q) + lane;
                if (Q4_IN_BOUNDS(pos, 1, T)) {
                    rows[pos] = b[q] < E ? static_cast<int32_t>(static_cast<uint32_t>(i) / static_cast<uint32_t>(top)) : -1;
                    places[i] = b[q] < E ? pos : -1 - pos;
                }
            }
            __syncwarp();
        }
    }
}

// ---------------------------------------------------------------------------
// rows to the experts' order and back
// ---------------------------------------------------------------------------
// All three kernels take a token per CTA and walk its row in pieces of the
// widest type that divides a row, every access a whole warp's.  They are bound
// by memory: dispatch reads each row of x once for all its copies, combine
// writes each row of out once, and the gradient reads dout once for all the
// token's choices.  Places outside [-T, T) are skipped.  Measured on B200,
// 16384 tokens x 8 of 256, K = 2048 bfloat16: dispatch 98 us (6.2 TB/s), combine
// 104 us (5.8 TB/s), its gradient 201 us (5.7 TB/s).  (Looking up eight places
// and holding eight pieces first, for more loads in flight, took 104 to 149 us:
// fewer threads fit.)
constexpr int kRowThreads = 256;

// The position a place names, and whether its choice was kept.
__device__ __forceinline__ int64_t place_row(int32_t place, bool* kept) {
    *kept = place >= 0;
    return place >= 0 ? place : -1 - static_cast<int64_t>(place);
}

template <typename V>
__global__ void __launch_bounds__(kRowThreads)
    dispatch_kernel(const V* __restrict__ x, const int32_t* __restrict__ places, V* __restrict__ xs, int64_t M,
                    int top, int64_t vecs) {
    const int64_t m = blockIdx.x, T = M * top;
    for (int64_t v = threadIdx.x; v < vecs; v += blockDim.x) {
        const V value = Q4_IN_BOUNDS(m * vecs + v, 1, M * vecs) ? x[m * vecs + v] : V{};
        for (int j = 0; j < top; ++j) {
            bool kept;
            const int64_t p = place_row(__ldg(places + m * top + j), &kept);
            if (p < T && Q4_IN_BOUNDS(p * vecs + v, 1, T * vecs)) xs[p * vecs + v] = kept ? value : V{};
        }
    }
}

template <typename T, typename V>
union Piece {
    V v;
    T t[sizeof(V) / sizeof(T)];
    __device__ Piece() {}
};

template <typename T, typename V>
__global__ void __launch_bounds__(kRowThreads)
    combine_kernel(const V* __restrict__ ys, const int32_t* __restrict__ places, const float* __restrict__ weights,
                   V* __restrict__ out, int64_t M, int top, int64_t vecs) {
    constexpr int kN = sizeof(V) / sizeof(T);
    const int64_t m = blockIdx.x, rows = M * top;
    for (int64_t v = threadIdx.x; v < vecs; v += blockDim.x) {
        float acc[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) acc[i] = 0.0f;
#pragma unroll 4
        for (int j = 0; j < top; ++j) {
            bool kept;
            const int64_t p = place_row(__ldg(places + m * top + j), &kept);
            if (!kept || p >= rows || !Q4_IN_BOUNDS(p * vecs + v, 1, rows * vecs)) continue;
            const float w = weights ? __ldg(weights + m * top + j) : 1.0f;
            Piece<T, V> y;
            y.v = ys[p * vecs + v];
#pragma unroll
            for (int i = 0; i < kN; ++i) acc[i] = fmaf(w, Element<T>::get(y.t[i]), acc[i]);
        }
        Piece<T, V> o;
#pragma unroll
        for (int i = 0; i < kN; ++i) o.t[i] = Element<T>::put(acc[i]);
        if (Q4_IN_BOUNDS(m * vecs + v, 1, M * vecs)) out[m * vecs + v] = o.v;
    }
}

// kBatch: choices whose dot products a thread holds at a time.
template <typename T, typename V, int kBatch>
__global__ void __launch_bounds__(kRowThreads)
    combine_grad_kernel(const V* __restrict__ dout, const V* __restrict__ ys, const int32_t* __restrict__ places,
                        const float* __restrict__ weights, V* __restrict__ dys, float* __restrict__ dweights,
                        int64_t M, int top, int64_t vecs) {
    constexpr int kN = sizeof(V) / sizeof(T);
    __shared__ float part[kRowThreads / 32][kBatch];
    const int64_t m = blockIdx.x, rows = M * top;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int j0 = 0; j0 < top; j0 += kBatch) {
        float dot[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) dot[j] = 0.0f;
        for (int64_t v = threadIdx.x; v < vecs; v += blockDim.x) {
            Piece<T, V> d;
            d.v = Q4_IN_BOUNDS(m * vecs + v, 1, M * vecs) ? dout[m * vecs + v] : V{};
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (j0 + j >= top) continue;
                bool kept;
                const int64_t p = place_row(__ldg(places + m * top + j0 + j), &kept);
                if (p >= rows || !Q4_IN_BOUNDS(p * vecs + v, 1, rows * vecs)) continue;
                Piece<T, V> o;
                o.v = V{};
                if (kept) {
                    const float w = weights ? __ldg(weights + m * top + j0 + j) : 1.0f;
                    Piece<T, V> y;
                    y.v = ys[p * vecs + v];
#pragma unroll
                    for (int i = 0; i < kN; ++i) {
                        const float g = Element<T>::get(d.t[i]);
                        dot[j] = fmaf(g, Element<T>::get(y.t[i]), dot[j]);
                        o.t[i] = Element<T>::put(w * g);
                    }
                }
                dys[p * vecs + v] = o.v;
            }
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
#pragma unroll
            for (int s = 16; s > 0; s /= 2) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], s);
            if (lane == 0) part[warp][j] = dot[j];
        }
        __syncthreads();
        if (threadIdx.x < kBatch && j0 + static_cast<int>(threadIdx.x) < top) {
            float sum = 0.0f;
            for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w) sum += part[w][threadIdx.x];
            dweights[m * top + j0 + threadIdx.x] = sum;
        }
        __syncthreads();
    }
}

// Threads for rows of `vecs` pieces: whole warps, no more than pieces need.
unsigned row_threads(int64_t vecs) {
    return static_cast<unsigned>(std::min<int64_t>(kRowThreads, (vecs + 31) / 32 * 32));
}

// Calls f(V{}) with the widest of 16, 8, 4, 2 bytes that divides a row.
template <typename F>
void with_vector(int64_t row_bytes, int size, F f) {
    if (row_bytes % 16 == 0)
        f(uint4{});
    else if (row_bytes % 8 == 0)
        f(uint2{});
    else if (row_bytes % 4 == 0 || size == 4)
        f(uint32_t{});
    else
        f(uint16_t{});
}

template <typename T>
cudaError_t combine_as(const void* ys, const int32_t* places, const float* weights, void* out, int64_t M, int top,
                       int64_t K, cudaStream_t s) {
    with_vector(K * sizeof(T), sizeof(T), [&](auto v) {
        using V = decltype(v);
        if constexpr (sizeof(V) >= sizeof(T)) {
            const int64_t vecs = K * static_cast<int64_t>(sizeof(T)) / static_cast<int64_t>(sizeof(V));
            combine_kernel<T, V><<<static_cast<unsigned>(M), row_threads(vecs), 0, s>>>(
                static_cast<const V*>(ys), places, weights, static_cast<V*>(out), M, top, vecs);
        }
    });
    return cudaGetLastError();
}

template <typename T>
cudaError_t combine_grad_as(const void* dout, const void* ys, const int32_t* places, const float* weights, void* dys,
                            float* dweights, int64_t M, int top, int64_t K, cudaStream_t s) {
    with_vector(K * sizeof(T), sizeof(T), [&](auto v) {
        using V = decltype(v);
        if constexpr (sizeof(V) >= sizeof(T)) {
            const int64_t vecs = K * static_cast<int64_t>(sizeof(T)) / static_cast<int64_t>(sizeof(V));
            const auto kernel = top <= 2 ? combine_grad_kernel<T, V, 2>
                                : top <= 4 ? combine_grad_kernel<T, V, 4> : combine_grad_kernel<T, V, 8>;
            kernel<<<static_cast<unsigned>(M), row_threads(vecs), 0, s>>>(
                static_cast<const V*>(dout), static_cast<const V*>(ys), places, weights, static_cast<V*>(dys),
                dweights, M, top, vecs);
        }
    });
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_sort_experts(const void* ids, int wide, int32_t* offsets, int32_t* rows, int32_t* places,
                                int64_t M, int64_t top, int64_t E, cudaStream_t s, const DeviceInfo& dev) {
    const int64_t T = M * top;
    const int smem = static_cast<int>(((E + 1) * (kSortWarps + 1) + 32) * sizeof(int));
    if (smem > dev.smem_optin) return cudaErrorNotSupported;
    const void* fn = wide ? reinterpret_cast<const void*>(sort_experts_kernel<int64_t>)
                          : reinterpret_cast<const void*>(sort_experts_kernel<int32_t>);
    cudaError_t e = ensure_smem_attr(fn, smem, wide ? 106 : 105, dev.device);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = T > kSortOneCta ? kSortCluster : 1;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(attr[0].val.clusterDim.x);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (wide)
        return cudaLaunchKernelEx(&cfg, sort_experts_kernel<int64_t>, static_cast<const int64_t*>(ids), offsets, rows,
                                  places, T, static_cast<int>(top), static_cast<int>(E));
    return cudaLaunchKernelEx(&cfg, sort_experts_kernel<int32_t>, static_cast<const int32_t*>(ids), offsets, rows,
                              places, T, static_cast<int>(top), static_cast<int>(E));
}

cudaError_t launch_dispatch(const void* x, const int32_t* places, void* xs, int type, int64_t M, int64_t top,
                            int64_t K, cudaStream_t s) {
    const int64_t row = K * type_size(type);
    with_vector(row, type_size(type), [&](auto v) {
        using V = decltype(v);
        const int64_t vecs = row / static_cast<int64_t>(sizeof(V));
        dispatch_kernel<V><<<static_cast<unsigned>(M), row_threads(vecs), 0, s>>>(
            static_cast<const V*>(x), places, static_cast<V*>(xs), M, static_cast<int>(top), vecs);
    });
    return cudaGetLastError();
}

cudaError_t launch_combine(const void* ys, const int32_t* places, const float* weights, void* out, int type,
                           int64_t M, int64_t top, int64_t K, cudaStream_t s) {
    const int t = static_cast<int>(top);
    if (type == Q4_F32) return combine_as<float>(ys, places, weights, out, M, t, K, s);
    if (type == Q4_BF16) return combine_as<__nv_bfloat16>(ys, places, weights, out, M, t, K, s);
    return combine_as<__half>(ys, places, weights, out, M, t, K, s);
}

cudaError_t launch_combine_grad(const void* dout, const void* ys, const int32_t* places, const float* weights,
                                void* dys, float* dweights, int type, int64_t M, int64_t top, int64_t K,
                                cudaStream_t s) {
    const int t = static_cast<int>(top);
    if (type == Q4_F32) return combine_grad_as<float>(dout, ys, places, weights, dys, dweights, M, t, K, s);
    if (type == Q4_BF16) return combine_grad_as<__nv_bfloat16>(dout, ys, places, weights, dys, dweights, M, t, K, s);
    return combine_grad_as<__half>(dout, ys, places, weights, dys, dweights, M, t, K, s);
}

Q4_DEFINE_TAKE_BOUNDS(experts)

}  // namespace q4

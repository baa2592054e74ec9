// q4_mx_tc.cuh -- device code shared by the products with microscaled
// matrices (q4_mx_gemm.cu, q4_mx_decode.cu): the block-scaled tensor-core
// instructions, bounded waits, the experts' row table, and the split of x into
// two 8-bit parts.
#pragma once

#include "q4_mx.cuh"
#include "q4_sm100.cuh"
#include "q4_wait.cuh"

namespace q4 {
namespace {

constexpr uint32_t kTmemCols = 512;
constexpr int kMaxExperts = Q4_MAX_EXPERTS;

// ---------------------------------------------------------------------------
// device helpers
// ---------------------------------------------------------------------------
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// tcgen05 instructions of one CTA (kCtas = 1) or of a pair (2): one thread of
// the pair's first CTA then acts for both, each CTA's own shared and tensor
// memory at the same addresses.
#define Q4_TC(one, two, ...)                  \
    do {                                      \
        if constexpr (kCtas == 1)             \
            asm volatile(one __VA_ARGS__);    \
        else                                  \
            asm volatile(two __VA_ARGS__);    \
    } while (0)

// 512 exponent bytes from shared memory to four columns of tensor memory,
// repeated in the four lane quarters.
template <int kCtas>
__device__ __forceinline__ void tc_copy_scales(uint32_t taddr, uint64_t desc) {
    Q4_TC("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;", "tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;",
          ::"r"(taddr), "l"(desc) : "memory");
}

// D[tmem] (+)= (A * sfa) x (B * sfb)^T, both operands in shared memory.
template <int kCtas>
__device__ __forceinline__ void tc_mma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                          uint32_t sfb, uint32_t accumulate) {
    Q4_TC("{\n\t.reg .pred p;\n\t"
          "setp.ne.b32 p, %6, 0;\n\t"
          "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}",
          "{\n\t.reg .pred p;\n\t"
          "setp.ne.b32 p, %6, 0;\n\t"
          "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}",
          ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate) : "memory");
}

// One arrival on `bar`, in every CTA of the group, when all prior MMAs and
// copies of this thread are complete.
template <int kCtas>
__device__ __forceinline__ void tc_commit_all(uint32_t bar) {
    if constexpr (kCtas == 1)
        tc_commit(bar);
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"(static_cast<uint16_t>(3))
            : "memory");
}
template <int kCtas>
__device__ __forceinline__ void tc_commit_own(uint32_t bar) {
    Q4_TC("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];",
          "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];", ::"r"(bar) : "memory");
}
template <int kCtas>
__device__ __forceinline__ void tmem_alloc_all(uint32_t dst) {
    Q4_TC("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;",
          "tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;", ::"r"(dst), "r"(kTmemCols) : "memory");
    Q4_TC("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;",
          "tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;", ::: "memory");
}
template <int kCtas>
__device__ __forceinline__ void tmem_free_all(uint32_t taddr) {
    Q4_TC("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;", "tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;",
          ::"r"(taddr), "r"(kTmemCols) : "memory");
}
#undef Q4_TC

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address in the pair's first CTA of what is at `addr` in this one.
__device__ __forceinline__ uint32_t in_first_cta(uint32_t addr) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(addr));
    return a;
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// TMA loads into this CTA that complete on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2,
                                                 uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

// Descriptor of 32 rows of 16 bytes in a row (no swizzle), for tc_copy_scales.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (1ull << 16) | (static_cast<uint64_t>(128 >> 4) << 32) |
           (1ull << 46);
}

// Instruction descriptor: A e2m1, B e4m3, power-of-two scales; the scale byte
// q of each 32-bit column is taken on both sides.
__host__ __device__ constexpr uint32_t mx_idesc(int M, int N, int q) {
    return (static_cast<uint32_t>(q) << 4) | (5u << 7) | (0u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
           (1u << 23) | (static_cast<uint32_t>(M >> 4) << 24) | (static_cast<uint32_t>(q) << 29);
}

// One lane of a converged warp.  The producer and MMA warps run their loops
// with all lanes, so that addresses and descriptors stay in uniform registers,
// and only issue with one (with `if (lane == 0)` around the loop each MMA took
// 70 cycles to issue and a stage's bookkeeping 450).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0u;
}

// One look of a whole warp at a barrier, its vote included.
__device__ __forceinline__ bool try_wait_all(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "vote.sync.all.pred q, p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0u;
}

// A bounded wait of a whole warp, which also gives up once another role has; the
// result is the same in all lanes.  What is seldom needed is out of line: with
// the loop and its clock in every role a token's product took 1 to 3 % longer.
__device__ __noinline__ bool wait_bar_on(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag) {
    const unsigned long long t0 = globaltimer_ns();
    return wait_together(
        [&] { return try_wait_all(bar, parity); },
        [&] { return __any_sync(0xFFFFFFFFu, *abort_flag != 0u || globaltimer_ns() - t0 > kWaitLimitNs) != 0; });
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag) {
    return try_wait_all(bar, parity) || wait_bar_on(bar, parity, abort_flag);
}

// A ring's slot and the parity of its use, without divisions.
template <int kSlots>
struct Ring {
    int slot = 0;
    uint32_t parity = 0;
    __device__ void next() {
        if (++slot == kSlots) {
            slot = 0;
            parity ^= 1u;
        }
    }
};

// 3-D TMA load of one box into shared memory, completing on `bar`.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

// Barrier of the four epilogue warps; true if `ok` was true in all of them.
// They leave their loop only on its result, so none waits for one that left.
__device__ __forceinline__ bool epilogue_sync(bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(ok ? 1u : 0u)
        : "memory");
    return r != 0u;
}

// Row ranges of the experts and the token tiles before each, in shared
// memory: offset[e], tile[e] for e in [0, E].  Offsets are taken as
// non-decreasing values in [0, T]; anything else is clamped to that.
struct Table {
    int offset[kMaxExperts + 1];
    int tile[kMaxExperts + 1];
};

__device__ void fill_table(Table& t, const int32_t* __restrict__ offsets, int E, int T, int tokens) {
    if (!offsets) {
        if (threadIdx.x == 0) {
            t.offset[0] = 0;
            t.offset[1] = T;
            t.tile[0] = 0;
            t.tile[1] = (T + tokens - 1) / tokens;
        }
    } else if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int high = 0, tiles = 0;  // over the experts before this round
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            int first = e < E && Q4_IN_BOUNDS(e, 2, E + 1) ? min(max(__ldg(offsets + e), 0), T) : 0;
            int last = e < E ? min(max(__ldg(offsets + e + 1), 0), T) : 0;
            // running maxima: first is at least every earlier end
            int top = max(first, last);
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int o = __shfl_up_sync(0xFFFFFFFFu, top, d);
                if (lane >= d) top = max(top, o);
            }
            const int up = __shfl_up_sync(0xFFFFFFFFu, top, 1);
            const int before = max(high, lane ? up : 0);
            first = max(first, before);
            last = max(last, first);
            const int mine = e < E ? (last - first + tokens - 1) / tokens : 0;
            int sum = mine;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
                if (lane >= d) sum += o;
            }
            if (e < E) {
                t.offset[e] = first;
                t.tile[e] = tiles + sum - mine;
                if (e == E - 1) {
                    t.offset[E] = last;
                    t.tile[E] = tiles + sum;
                }
            }
            high = max(high, __shfl_sync(0xFFFFFFFFu, top, 31));
            tiles += __shfl_sync(0xFFFFFFFFu, sum, 31);
        }
    }
    __syncthreads();
}

// The last e with first[e] <= v (first[0] <= v < first[E]).
__device__ __forceinline__ int find_expert(const int* first, int E, int v) {
    int lo = 0, hi = E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (first[mid] <= v)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// ---------------------------------------------------------------------------
// x to its two e4m3 parts
// ---------------------------------------------------------------------------
// Two binary16 values to e4m3 (nearest, saturating) and back.
__device__ __forceinline__ uint32_t to_e4m3x2(__half2 v) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&v)));
    return r;
}
__device__ __forceinline__ __half2 from_e4m3x2(uint32_t v) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
    return *reinterpret_cast<const __half2*>(&h);
}

// A lane's eight consecutive x of a row, a group of 32 in four lanes, as the
// two parts and hi's exponent byte; 255, the byte of NaN, for a group with an
// infinity or NaN.  x / s is exact in bfloat16 (a power of two), and in
// binary16 from 2^-17 on; what is smaller goes to zero in both parts, being
// below half of lo's smallest step, 2^-15.  The remainder x / s - hi has at
// most 8 bits, so two values at a time in binary16 lose nothing.
struct XParts {
    uint2 hi, lo;
    uint32_t byte;
};
__device__ __forceinline__ XParts split_x(const uint4& q) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    uint32_t both = 0;  // magnitudes order as their bits do
#pragma unroll
    for (int j = 0; j < 4; ++j) both = __vmaxu2(both, w[j] & 0x7FFF7FFFu);
    uint32_t top = max(both & 0xFFFFu, both >> 16);
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    // the largest value's exponent field - 7, so that the largest x / s is in
    // [128, 256); at least 5, which leaves lo's byte >= 0
    const uint32_t field = top >> 7;
    const uint32_t byte = field > 12u ? field - 7u : 5u;
    const uint32_t inverse = ((254u - byte) << 7) * 0x10001u;
    uint32_t h[2] = {0, 0}, l[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 scaled = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[j]),
                                              *reinterpret_cast<const __nv_bfloat162*>(&inverse));
        const __half2 a = __float22half2_rn(__bfloat1622float2(scaled));
        const uint32_t c = to_e4m3x2(a);
        const __half2 rest = __hmul2(__hsub2(a, from_e4m3x2(c)), __float2half2_rn(32.0f));
        h[j / 2] |= c << (16 * (j & 1));
        l[j / 2] |= to_e4m3x2(rest) << (16 * (j & 1));
    }
    return {make_uint2(h[0], h[1]), make_uint2(l[0], l[1]), field == 255u ? 255u : byte};
}

// The exponent bytes of the four groups of a k block, held by 16 lanes, in a
// word for hi and one for lo.
__device__ __forceinline__ void gather_bytes(uint32_t byte, int lane, uint32_t& hi, uint32_t& lo) {
    hi = lo = 0;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const uint32_t b = __shfl_sync(0xFFFFFFFFu, byte, (lane & 16) + 4 * g);
        hi |= b << (8 * g);
        lo |= (b == 255u ? 255u : b - 5u) << (8 * g);
    }
}

// A lane's eight x at `x` + first, k being the first's; zeros past K or
// without a row.  kVector: rows are whole pieces of 16 bytes.
template <bool kVector>
__device__ __forceinline__ uint4 load_x8(const uint16_t* __restrict__ x, bool have, int64_t first, int64_t k, int64_t K,
                                         int64_t extent) {
    uint4 q = make_uint4(0, 0, 0, 0);
    if (kVector) {
        if (have && k < K && Q4_IN_BOUNDS(first, 8, extent)) q = __ldg(reinterpret_cast<const uint4*>(x + first));
        return q;
    }
    uint32_t* w = &q.x;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (have && k + j < K && Q4_IN_BOUNDS(first + j, 1, extent))
            w[j / 2] |= static_cast<uint32_t>(x[first + j]) << (16 * (j & 1));
    return q;
}

}  // namespace
}  // namespace q4

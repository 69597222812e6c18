// Blackwell tensor-core building blocks (sm_103a, PTX): mbarriers with bounded waits, TMA
// tile loads, tensor memory and tcgen05.mma, as the attention kernels use them.
//
// Shared-memory tiles are boxes of 64 bf16 columns (128 bytes a row) in the 128-byte
// swizzle, the layout TMA writes and the matrix descriptors name: 8 rows x 128 bytes are a
// swizzle atom of 1024 bytes, and every box starts on a 1024-byte boundary.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fastdiv.cuh"

namespace pvr {

// Waits are bounded in time: after kWaitNs the waiter raises the CTA's abort flag and counts
// one in the device's fault word, the CTA's other waits end when they see the flag, and the CTA drains
// its copies and products, frees its tensor memory and returns.
constexpr unsigned long long kWaitNs = 2000000000ull;
constexpr unsigned long long kDrainNs = 20000000ull;

__device__ __forceinline__ unsigned long long now_ns()
{
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ uint32_t smem_addr(const void *p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n .reg .pred p;\n"
                 " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
                 " selp.b32 %0, 1, 0, p;\n}"
                 : "=r"(done)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return done != 0;
}

// One thread waits for the phase of the given parity; false when the CTA gave up.
static __device__ __noinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity, volatile int *abort_flag, int *fault)
{
    const unsigned long long start = now_ns();
    for (int i = 1;; ++i) {
        if (mbar_try(bar, parity)) return true;
        if (abort_flag != nullptr && *abort_flag != 0) return false;
        if ((i & 63) == 0 && now_ns() - start > kWaitNs) break;
    }
    if (abort_flag != nullptr) *abort_flag = 1;
    atomicAdd(fault, 1);
    return false;
}

__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag, int *fault)
{
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
        if (mbar_try(bar, parity)) return true;
    return mbar_wait_slow(bar, parity, abort_flag, fault);
}

// After an abort: waits a little for copies or products in flight.
static __device__ __noinline__ void mbar_drain(uint32_t bar, uint32_t parity)
{
    const unsigned long long start = now_ns();
    while (!mbar_try(bar, parity) && now_ns() - start < kDrainNs) {}
}

// A converged warp waits; the result is the same in every lane.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag, int *fault)
{
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, fault));
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4}], [%5];"
                 ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar) : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, int c3,
                                            uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4, %5}], [%6];"
                 ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar) : "memory");
}

__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Shared-memory writes of this thread become visible to the tensor core and TMA.
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t columns)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns) : "memory");
}

// Arrives on the barrier when every tcgen05.mma this thread has issued is complete.
__device__ __forceinline__ void tc_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t yes;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.b32 %0, 1, 0, p;\n}" : "=r"(yes));
    return yes != 0;
}

// The value of lane 0, which the compiler then knows to be the same in every lane: what the
// tensor core's instructions take must live in uniform registers, and a value that is not
// known to be uniform costs about 100 cycles an instruction to get there.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// Matrix descriptor of a 128-byte-swizzled bf16 tile at a shared-memory address: strides in
// bytes.  K-major operands (the product's sum runs along the row): `stride` 1024 from one
// group of 8 rows to the next, `lead` unused.  MN-major operands (the sum runs down the
// rows): `stride` 1024 from 8 rows to the next 8, `lead` from one box of 64 columns to the
// next.  The low word holds the address: a step of n bytes adds n >> 4.
__device__ __forceinline__ constexpr uint32_t desc_lo(uint32_t addr, uint32_t lead)
{
    return ((addr & 0x3ffffu) >> 4) | ((lead >> 4) << 16);
}
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);

// Instruction descriptor: bf16 x bf16 -> binary32, M x N, B K-major or MN-major.
__host__ __device__ constexpr uint32_t mma_desc(int m, int n, bool b_mn_major)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

// D[tmem] (+)= A[smem] B[smem], one k step of 16; operands by their descriptors' low words.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate)
{
    asm volatile("{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.u32 p, %4, 0;\n"
                 " mov.b64 x, {%1, %5};\n mov.b64 y, {%2, %5};\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}"
                 ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(kDescHi) : "memory");
}

// D[tmem] (+)= A[tmem] B[smem].
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate)
{
    asm volatile("{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.u32 p, %4, 0;\n mov.b64 y, {%2, %5};\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}"
                 ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(kDescHi) : "memory");
}

#define PVR_R8(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3]), "=r"(a[i + 4]), "=r"(a[i + 5]), \
                     "=r"(a[i + 6]), "=r"(a[i + 7])
#define PVR_W8(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3]), "r"(a[i + 4]), "r"(a[i + 5]), \
                     "r"(a[i + 6]), "r"(a[i + 7])

// 32 consecutive columns of this warp's 32 lanes (one row a lane).
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                 "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : PVR_R8(r, 0), PVR_R8(r, 8), PVR_R8(r, 16), PVR_R8(r, 24)
                 : "r"(addr));
}

__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                 "%14, %15}, [%16];"
                 : PVR_R8(r, 0), PVR_R8(r, 8)
                 : "r"(addr));
}

__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
                 "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
                 ::"r"(addr), PVR_W8(r, 0), PVR_W8(r, 8), PVR_W8(r, 16), PVR_W8(r, 24)
                 : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
                 "%13, %14, %15, %16};"
                 ::"r"(addr), PVR_W8(r, 0), PVR_W8(r, 8)
                 : "memory");
}

#define PVR_RW8(a, i) "+r"(a[i]), "+r"(a[i + 1]), "+r"(a[i + 2]), "+r"(a[i + 3]), "+r"(a[i + 4]), "+r"(a[i + 5]), \
                      "+r"(a[i + 6]), "+r"(a[i + 7])

// The loads before it are complete.  Naming the registers orders every use of them after
// the wait; tmem_loaded does that for further registers of the same wait.
__device__ __forceinline__ void tc_wait_ld(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" : PVR_RW8(r, 0), PVR_RW8(r, 8), PVR_RW8(r, 16), PVR_RW8(r, 24)::"memory");
}

__device__ __forceinline__ void tc_wait_ld16(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" : PVR_RW8(r, 0), PVR_RW8(r, 8)::"memory");
}

__device__ __forceinline__ void tmem_loaded(uint32_t (&r)[32])
{
    asm volatile("" : PVR_RW8(r, 0), PVR_RW8(r, 8), PVR_RW8(r, 16), PVR_RW8(r, 24)::"memory");
}

// 2^x from the special-function unit (subnormal results flush to zero).
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Meets the other warps that name this barrier (ids 1..15), `threads` in all.
__device__ __forceinline__ void named_barrier(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Four floats at a shared-memory address.
__device__ __forceinline__ float4 smem_load4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}

// Both halves of a pair through one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
        " fma.rn.f32x2 w, x, y, z;\n mov.b64 {%0, %1}, w;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{\n .reg .b64 x, y, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 w, x, y;\n"
        " mov.b64 {%0, %1}, w;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("{\n .reg .b64 x, y, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 w, x, y;\n"
        " mov.b64 {%0, %1}, w;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// Thread-block clusters.
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait()
{
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Stores at this CTA's shared address `addr`, in CTA `rank` of the cluster.
__device__ __forceinline__ void cluster_store(uint32_t addr, uint32_t rank, float v)
{
    asm volatile("{\n .reg .u32 p;\n mapa.shared::cluster.u32 p, %0, %1;\n st.shared::cluster.f32 [p], %2;\n}"
                 ::"r"(addr), "r"(rank), "f"(v) : "memory");
}
__device__ __forceinline__ void cluster_store4(uint32_t addr, uint32_t rank, float4 v)
{
    asm volatile("{\n .reg .u32 p;\n mapa.shared::cluster.u32 p, %0, %1;\n"
                 " st.shared::cluster.v4.f32 [p], {%2, %3, %4, %5};\n}"
                 ::"r"(addr), "r"(rank), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

// A warp's 32 rows of COLS bf16, one row a lane, to global memory with whole lines a store: a
// row a lane would touch 32 lines with every 16 bytes a lane, and that alone took 4,000 cycles
// of an attention CTA.  `scratch`: 64 * COLS bytes of shared memory of the warp's own.
// to(row) is where the row's columns go, or NULL; only the first `cols` of them are written.
template <int COLS, typename To>
__device__ __forceinline__ void warp_store_rows(uint32_t scratch, const uint32_t (&v)[COLS / 2], int cols, To to)
{
    constexpr int kChunks = COLS / 8;                        // of 16 bytes
    const int lane = threadIdx.x & 31;
    auto at = [&](int row, int chunk) {                      // spread over the banks
        return scratch + row * (2 * COLS) + ((chunk ^ ((row / (8 / kChunks)) & (kChunks - 1))) << 4);
    };
    __syncwarp();
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at(lane, c)), "r"(v[4 * c]), "r"(v[4 * c + 1]),
                     "r"(v[4 * c + 2]), "r"(v[4 * c + 3]) : "memory");
    __syncwarp();
#pragma unroll 1                                             // run once a CTA: short code, few instruction fetches
    for (int i = 0; i < kChunks; ++i) {
        const int index = 32 * i + lane, row = index / kChunks, chunk = index % kChunks;
        uint4 x;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at(row, chunk)));
        __nv_bfloat16 *dst = to(row);
        if (dst != nullptr && 8 * chunk < cols) *reinterpret_cast<uint4 *>(dst + 8 * chunk) = x;
    }
}

// The sample a tile slot belongs to.  The token axis [0, T) is cut at cu[0..n] into n + 2
// stretches (what lies before the pack, the samples, what lies after it), and stretch s
// owns the slots from floor(start_s / tile) + s on: room for every one of its tiles,
// with no prefix sum over the samples and no size read on the host.  T / tile + n + 2 slots
// cover any pack; those past a stretch's last tile are empty.
struct TileSlot {
    int sample;        // -1 or n: outside the pack
    int start, end;    // the stretch's tokens [start, end), inside [0, T]
    int tile;          // index of the tile in the stretch
    int used;          // the sample's entry of `used` (its length without one); 0 outside the pack
};

// Called by a whole warp.  Whatever cu holds, start and end stay in [0, T].  Short packs
// take one round of loads, the entries of `used` with them.
__device__ __forceinline__ TileSlot find_slot(const int32_t *__restrict__ cu, const int32_t *__restrict__ used, int n,
                                              int T, FastDiv tile, int slot)
{
    const int lane = threadIdx.x & 31;
    auto bound = [&](int s) {                      // first token of stretch s, s in [0, n + 2]
        if (s <= 0) return 0;
        if (s >= n + 2) return T;
        return min(max(__ldg(cu + (s - 1)), 0), T);
    };
    TileSlot r;
    int lo;
    constexpr int kShort = 4;
    if (n + 3 <= 32 * kShort) {
        int b[kShort], u[kShort], count = 0;
#pragma unroll
        for (int j = 0; j < kShort; ++j) {
            const int s = lane + 32 * j;
            b[j] = s <= n + 2 ? bound(s) : T;
            u[j] = used != nullptr && s >= 1 && s <= n ? __ldg(used + (s - 1)) : 0;
        }
#pragma unroll
        for (int j = 0; j < kShort; ++j) {
            const int s = lane + 32 * j;
            count += __popc(__ballot_sync(0xffffffffu, s <= n + 1 && static_cast<int>(fast_div(b[j], tile)) + s <= slot));
        }
        lo = max(count - 1, 0);
        r.start = r.end = r.used = 0;
#pragma unroll
        for (int j = 0; j < kShort; ++j) {
            const int start = __shfl_sync(0xffffffffu, b[j], lo & 31), end = __shfl_sync(0xffffffffu, b[j], (lo + 1) & 31);
            const int entry = __shfl_sync(0xffffffffu, u[j], lo & 31);
            if (lo >> 5 == j) {
                r.start = start;
                r.used = entry;
            }
            if ((lo + 1) >> 5 == j) r.end = end;
        }
    } else {
        lo = 0;
        int len = n + 2;
        while (len > 1) {
            const int step = (len + 31) >> 5;
            const int s = lo + lane * step;
            const bool below = s < lo + len && static_cast<int>(fast_div(bound(s), tile)) + s <= slot;
            const uint32_t vote = __ballot_sync(0xffffffffu, below);
            const int hit = vote == 0xffffffffu ? 31 : __ffs(~vote) - 2;   // last of the leading run
            const int at = lo + max(hit, 0) * step;
            len = min(step, lo + len - at);
            lo = at;
        }
        r.start = bound(lo);
        r.end = bound(lo + 1);
        r.used = used != nullptr && lo >= 1 && lo <= n ? __ldg(used + (lo - 1)) : 0;
    }
    r.sample = lo - 1;
    r.end = max(r.end, r.start);
    r.tile = slot - (static_cast<int>(fast_div(r.start, tile)) + lo);
    if (used == nullptr && lo >= 1 && lo <= n) r.used = r.end - r.start;
    return r;
}

__host__ __device__ inline int slot_count(int T, int n, int tile_tokens) { return T / tile_tokens + n + 2; }

}  // namespace pvr

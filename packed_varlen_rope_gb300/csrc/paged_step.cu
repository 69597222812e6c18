// A serving step's page tables and slots (GB300, sm_103a).
//
// One cluster of CTAs does it all: every thread owns a few consecutive sequences, three prefix
// sums (pages given back, pages wanted, new tokens) run over lanes, warps and the cluster's CTAs,
// and what a warp's sequences give back, take and place is walked flat, a page or a token a
// lane, so that uneven sequences cost what they hold.  Sums are 64 bits wide.  The slots of many
// tokens, which a cluster's few SMs would write at a fraction of HBM's rate, are left to a second
// launch over the whole GPU.
//
// What comes next in the stream reads these arrays, some of it as read-only data: the last
// launch here does not let its successor start early.
//
// Bound by latency: lengths, sums, page ids and the writes follow one another.

#include <cuda_runtime.h>

#include <cstdint>

#include "fastdiv.cuh"
#include "host_checks.h"
#include "paged_step.h"
#include "tensor_core.cuh"

namespace {

using namespace pvr;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int64_t kOwnTokens = 1 << 14;  // slots that the cluster writes itself
constexpr int kFillThreads = 256, kFillTokens = 8;   // of the second launch; tokens a thread
constexpr int kFillStaged = 6144;       // sequences whose cu_seqlens a CTA stages

struct StepArgs {
    paged_kv_step_desc p;
    FastDiv div_page;
    int32_t per_thread;                 // sequences
    int32_t fill;                       // the slots are the second launch's
};

struct Sums {
    int64_t back, take, tokens;         // pages given back, pages taken, new tokens
};

__device__ __forceinline__ Sums operator+(const Sums &a, const Sums &b)
{
    return Sums{a.back + b.back, a.take + b.take, a.tokens + b.tokens};
}

__device__ __forceinline__ Sums shift_up(const Sums &a, int by)
{
    return Sums{__shfl_up_sync(0xffffffffu, a.back, by), __shfl_up_sync(0xffffffffu, a.take, by),
                __shfl_up_sync(0xffffffffu, a.tokens, by)};
}

// Inclusive sums over a warp's lanes.
__device__ __forceinline__ Sums warp_scan(Sums x)
{
    for (int by = 1; by < 32; by *= 2) {
        const Sums y = shift_up(x, by);
        if ((threadIdx.x & 31) >= by) x = x + y;
    }
    return x;
}

__device__ __forceinline__ void cluster_store64(const void *at, uint32_t rank, int64_t v)
{
    asm volatile("{\n .reg .u32 p;\n mapa.shared::cluster.u32 p, %0, %1;\n st.shared::cluster.b64 [p], %2;\n}"
                 ::"r"(smem_addr(at)), "r"(rank), "l"(v) : "memory");
}

// A sequence of the step.
struct Row {
    int past, fresh, held, want;        // tokens, new tokens, pages held before and wanted after
    bool over;                          // its pages go back
    int gives;                          // entries of its row that may go back
};

__device__ __forceinline__ int pages_of(const StepArgs &a, int tokens)
{
    const int whole = static_cast<int>(fast_div(static_cast<uint32_t>(tokens), a.div_page));
    return min(whole + (tokens != whole * a.p.page_size), a.p.max_pages);
}

__device__ __forceinline__ Row load_row(const StepArgs &a, int s, int &status)
{
    Row r{};
    if (s >= a.p.n_seqs) return r;
    r.past = a.p.past_lens[s];
    r.fresh = a.p.new_lens[s];
    r.over = a.p.finished != nullptr && a.p.finished[s] != 0;
    if (r.past < 0 || r.fresh < 0) status |= STEP_NEGATIVE_LENGTH;
    r.past = max(r.past, 0);
    r.fresh = max(r.fresh, 0);
    if (r.over) {
        r.gives = pages_of(a, r.past);
        r.past = 0;
    }
    const int64_t kv = min(static_cast<int64_t>(r.past) + r.fresh, static_cast<int64_t>(INT32_MAX));
    if (kv > static_cast<int64_t>(a.p.max_pages) * a.p.page_size) status |= STEP_TABLE_FULL;
    r.held = pages_of(a, r.past);
    r.want = pages_of(a, static_cast<int>(kv));
    return r;
}

// Walks the items of a warp's lanes flat: lane's items are [0, count), `before` is the sum of the
// counts of the lanes below; act(lane's index, item) for each, 32 at a time.
template <typename Act>
__device__ __forceinline__ void walk(int64_t before, int64_t count, Act act)
{
    const int lane = threadIdx.x & 31;
    const int64_t all = __shfl_sync(0xffffffffu, before + count, 31);
    for (int64_t e0 = 0; e0 < all; e0 += 32) {
        const int64_t e = e0 + lane;
        int owner = 0;                  // last lane whose items begin at or before e
#pragma unroll
        for (int step = 16; step > 0; step /= 2) {
            const int64_t from = __shfl_sync(0xffffffffu, before, owner + step);
            if (from <= e) owner += step;
        }
        const int64_t item = e - __shfl_sync(0xffffffffu, before, owner);
        act(owner, item, e < all);
    }
}

__global__ void __launch_bounds__(kThreads) paged_step_kernel(const __grid_constant__ StepArgs a)
{
    __shared__ Sums s_warp[kWarps], s_rank[kMaxCluster];
    __shared__ int64_t s_status[kMaxCluster];
    __shared__ int s_bits;
    const paged_kv_step_desc &p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank(), ranks = cluster_size();
    if (threadIdx.x == 0) s_bits = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (a.fill) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __syncthreads();
    if (ranks > 1) cluster_arrive();                         // this CTA runs: its memory may be written

    const int first = (static_cast<int>(rank) * kThreads + static_cast<int>(threadIdx.x)) * a.per_thread;
    const int count0 = min(max(*p.free_count, 0), static_cast<int>(p.n_free_max));
    int status = 0;

    // ids of row s that go back: their number, counted by the whole warp for one lane's row
    auto count_back = [&](int s, int entries) {
        int n = 0;
        for (int i0 = 0; i0 < entries; i0 += 32)
            n += __popc(__ballot_sync(0xffffffffu, i0 + lane < entries && p.page_table[s * p.page_table_stride + i0 + lane] >= 0));
        return n;
    };

    // ---- the sums of this thread's sequences
    Sums mine{};
    for (int k = 0; k < a.per_thread; ++k) {
        const Row r = load_row(a, first + k, status);
        mine.take += r.want - r.held;
        mine.tokens += r.fresh;
        uint32_t todo = __ballot_sync(0xffffffffu, r.gives > 0);
        while (todo != 0) {
            const int from = __ffs(todo) - 1;
            todo &= todo - 1;
            const int n = count_back(__shfl_sync(0xffffffffu, first, from) + k, __shfl_sync(0xffffffffu, r.gives, from));
            if (lane == from) mine.back += n;
        }
    }
    const Sums upto = warp_scan(mine);
    if (lane == 31) s_warp[warp] = upto;
    if (status != 0) atomicOr(&s_bits, status);
    __syncthreads();
    Sums before{upto.back - mine.back, upto.take - mine.take, upto.tokens - mine.tokens}, all{};
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp) before = before + all;
        all = all + s_warp[w];
    }
    if (ranks > 1) {
        cluster_wait();
        if (threadIdx.x < ranks) {
            cluster_store64(&s_rank[rank].back, threadIdx.x, all.back);
            cluster_store64(&s_rank[rank].take, threadIdx.x, all.take);
            cluster_store64(&s_rank[rank].tokens, threadIdx.x, all.tokens);
        }
        cluster_arrive();
        cluster_wait();
        all = Sums{};
        for (uint32_t r = 0; r < ranks; ++r) {
            if (r == rank) before = before + all;
            all = all + s_rank[r];
        }
    }

    // ---- pages go back, and are seen by every CTA before any is taken
    if (all.back > 0) {
        int64_t to = count0 + before.back;
        for (int k = 0; k < a.per_thread; ++k) {
            int none = 0;
            const Row r = load_row(a, first + k, none);
            uint32_t todo = __ballot_sync(0xffffffffu, r.gives > 0);
            while (todo != 0) {
                const int from = __ffs(todo) - 1;
                todo &= todo - 1;
                const int64_t row = static_cast<int64_t>(__shfl_sync(0xffffffffu, first, from) + k) * p.page_table_stride;
                const int entries = __shfl_sync(0xffffffffu, r.gives, from);
                int64_t at = __shfl_sync(0xffffffffu, to, from);
                for (int i0 = 0; i0 < entries; i0 += 32) {
                    const int id = i0 + lane < entries ? p.page_table[row + i0 + lane] : -1;
                    const uint32_t valid = __ballot_sync(0xffffffffu, id >= 0);
                    const int64_t place = at + __popc(valid & ((1u << lane) - 1));
                    if (id >= 0 && place < p.n_free_max) p.free_pages[place] = id;
                    at += __popc(valid);
                }
                if (lane == from) to = at;
            }
        }
        if (ranks > 1) {
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
    }
    const int64_t full = count0 + all.back;
    const int64_t count1 = min(full, p.n_free_max);

    // ---- lengths, pages taken, slots
    const bool slots = p.slots != nullptr && !a.fill;
    for (int k = 0; k < a.per_thread; ++k) {
        const int s = first + k;
        int none = 0;
        const Row r = load_row(a, s, none);
        if (s < p.n_seqs) {
            p.kv_lens[s] = static_cast<int>(min(static_cast<int64_t>(r.past) + r.fresh, static_cast<int64_t>(INT32_MAX)));
            p.cu_seqlens[s + 1] = static_cast<int>(min(before.tokens + r.fresh, static_cast<int64_t>(INT32_MAX)));
            if (s == 0) p.cu_seqlens[0] = 0;
        }
        const int takes = r.want - r.held;
        const int64_t top = count1 - 1 - before.take;        // of the stack, for this row's first page
        // whatever the lengths hold, no more tokens are walked than there are slots
        const int64_t placed = max(min(static_cast<int64_t>(r.fresh), p.max_tokens - before.tokens), static_cast<int64_t>(0));
        const Sums lanes = warp_scan(Sums{0, takes, placed});
        walk(lanes.take - takes, takes, [&](int owner, int64_t item, bool in) {
            const int64_t from = __shfl_sync(0xffffffffu, top, owner) - item;
            const int held = __shfl_sync(0xffffffffu, r.held, owner), row = __shfl_sync(0xffffffffu, s, owner);
            if (in) p.page_table[row * p.page_table_stride + held + item] = from >= 0 ? p.free_pages[from] : -1;
        });
        if (slots) {
            walk(lanes.tokens - placed, placed, [&](int owner, int64_t item, bool in) {
                const int64_t to = __shfl_sync(0xffffffffu, before.tokens, owner) + item;
                const int64_t pos = __shfl_sync(0xffffffffu, r.past, owner) + item;
                const int64_t from_top = __shfl_sync(0xffffffffu, top, owner);
                const int held = __shfl_sync(0xffffffffu, r.held, owner), row = __shfl_sync(0xffffffffu, s, owner);
                if (!in) return;
                int64_t slot = -1;
                if (pos < static_cast<int64_t>(p.max_pages) * p.page_size) {
                    const int index = static_cast<int>(fast_div(static_cast<uint32_t>(pos), a.div_page));
                    const int64_t from = from_top - (index - held);
                    const int id = index < held ? p.page_table[row * p.page_table_stride + index]
                                                : from >= 0 ? p.free_pages[from] : -1;
                    if (id >= 0) slot = static_cast<int64_t>(id) * p.page_size + (pos - static_cast<int64_t>(index) * p.page_size);
                }
                p.slots[to] = slot;
            });
        }
        before.take += takes;
        before.tokens += r.fresh;
    }
    if (slots)
        for (int64_t t = all.tokens + rank * kThreads + threadIdx.x; t < p.max_tokens; t += ranks * kThreads) p.slots[t] = -1;
    if (p.n_seqs == 0 && rank == 0 && threadIdx.x == 0) p.cu_seqlens[0] = 0;

    // ---- the count and the bits: every CTA has read the count by now
    if (ranks > 1) {
        if (threadIdx.x == 0) cluster_store64(&s_status[rank], 0, s_bits);
        cluster_arrive();
        cluster_wait();
    } else {
        if (threadIdx.x == 0) s_status[0] = s_bits;
        __syncthreads();
    }
    if (rank == 0 && threadIdx.x == 0) {
        int bits = 0;
        for (uint32_t r = 0; r < ranks; ++r) bits |= static_cast<int>(s_status[r]);
        if (all.take > count1) bits |= STEP_NO_PAGES;
        if (full > p.n_free_max) bits |= STEP_STACK_FULL;
        if (all.tokens > INT32_MAX || (p.slots != nullptr && all.tokens > p.max_tokens)) bits |= STEP_TOKENS_PAST_END;
        *p.count_out = static_cast<int>(max(count1 - all.take, static_cast<int64_t>(0)));
        if (p.status != nullptr) *p.status = bits;
    }
}

// Slots of many tokens, from the arrays that the step has written: the sequence by binary
// search in cu_seqlens, its page from the table.
__global__ void __launch_bounds__(kFillThreads) paged_slots_kernel(const __grid_constant__ StepArgs a)
{
    extern __shared__ int32_t s_cu[];
    const paged_kv_step_desc &p = a.p;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const bool staged = p.n_seqs <= kFillStaged;
    if (staged) {
        for (int i = threadIdx.x; i <= p.n_seqs; i += kFillThreads) s_cu[i] = p.cu_seqlens[i];
        __syncthreads();
    }
    const int32_t *cu = staged ? s_cu : p.cu_seqlens;
    const int total = cu[p.n_seqs];
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * (kFillThreads * kFillTokens) + threadIdx.x;
#pragma unroll
    for (int k = 0; k < kFillTokens; ++k) {
        const int64_t t = t0 + k * kFillThreads;
        if (t >= p.max_tokens) return;
        int64_t slot = -1;
        if (t < total) {
            int lo = 0, hi = p.n_seqs;
            while (hi - lo > 1) {
                const int mid = lo + ((hi - lo) >> 1);
                if (cu[mid] <= t) lo = mid;
                else hi = mid;
            }
            const int64_t pos = static_cast<int64_t>(p.kv_lens[lo]) - (cu[lo + 1] - t);
            if (pos < static_cast<int64_t>(p.max_pages) * p.page_size) {
                const int index = static_cast<int>(fast_div(static_cast<uint32_t>(pos), a.div_page));
                const int id = p.page_table[lo * p.page_table_stride + index];
                if (id >= 0) slot = static_cast<int64_t>(id) * p.page_size + (pos - static_cast<int64_t>(index) * p.page_size);
            }
        }
        p.slots[t] = slot;
    }
}

int check_step(const paged_kv_step_desc &p)
{
    if (p.n_seqs < 0 || p.n_seqs > kMaxTokens || p.max_pages < 0 || p.page_size < 1 || p.page_size > 65536 ||
        p.n_free_max < 0 || p.n_free_max > INT32_MAX || p.max_tokens < 0 || p.max_tokens > INT32_MAX ||
        (p.n_seqs > 1 && p.page_table_stride < p.max_pages) || p.page_table_stride > (int64_t(1) << 40))
        return ROPE_ERR_SHAPE;
    if (p.reserved != 0 || static_cast<int64_t>(p.max_pages) * p.page_size > INT32_MAX / 2) return ROPE_ERR_UNSUPPORTED;
    const int64_t n = p.n_seqs, table = n > 0 && p.max_pages > 0 ? (n - 1) * p.page_table_stride + p.max_pages : 0;
    const int64_t tokens = p.slots != nullptr ? p.max_tokens : 0;
    struct Range {
        const void *at;
        int64_t bytes;
        bool written, needed;
    };
    const Range ranges[] = {
        {p.free_pages, 4 * p.n_free_max, true, true}, {p.count_out, 4, true, true}, {p.page_table, 4 * table, true, true},
        {p.cu_seqlens, 4 * (n + 1), true, true}, {p.kv_lens, 4 * n, true, true}, {p.slots, 8 * tokens, true, false},
        {p.status, p.status != nullptr ? 4 : 0, true, false}, {p.free_count, 4, false, true},
        {p.past_lens, 4 * n, false, true}, {p.new_lens, 4 * n, false, true},
        {p.finished, p.finished != nullptr ? 4 * n : 0, false, false}};
    for (const Range &r : ranges) {
        if (r.needed && r.bytes > 0 && r.at == nullptr) return ROPE_ERR_NULL;
        if (r.bytes > 0 && !aligned(r.at, r.at == p.slots ? 8 : 4)) return ROPE_ERR_ALIGN;
    }
    for (const Range &w : ranges)
        for (const Range &r : ranges)
            // (ranges[1], the count after the step, may be ranges[7], the one before)
            if (&w != &r && w.written && !(&w == ranges + 1 && &r == ranges + 7 && w.at == r.at) &&
                overlap(w.at, w.bytes, r.at, r.bytes))
                return ROPE_ERR_OVERLAP;
    return ROPE_OK;
}

}  // namespace

extern "C" int paged_kv_step(const paged_kv_step_desc *desc, void *stream)
{
    if (desc == nullptr) return ROPE_ERR_NULL;
    const int rc = check_step(*desc);
    if (rc != ROPE_OK) return rc;
    StepArgs a{};
    a.p = *desc;
    a.div_page = make_fastdiv(static_cast<uint32_t>(desc->page_size));
    const int64_t n = desc->n_seqs;
    const int cluster = n <= kThreads ? 1 : n <= 2 * kThreads ? 2 : n <= 4 * kThreads ? 4 : kMaxCluster;
    a.per_thread = static_cast<int32_t>((n + cluster * kThreads - 1) / (cluster * kThreads));
    a.fill = desc->slots != nullptr && desc->max_tokens > kOwnTokens;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, paged_step_kernel, a) != cudaSuccess) return ROPE_ERR_LAUNCH;
    if (!a.fill) return ROPE_OK;
    const int64_t per_cta = kFillThreads * kFillTokens;
    cfg.gridDim = dim3(static_cast<unsigned>((desc->max_tokens + per_cta - 1) / per_cta));
    cfg.blockDim = dim3(kFillThreads);
    cfg.dynamicSmemBytes = n <= kFillStaged ? 4 * static_cast<size_t>(n + 1) : 0;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_slots_kernel, a) == cudaSuccess ? ROPE_OK : ROPE_ERR_LAUNCH;
}

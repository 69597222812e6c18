// A serving step's page tables and slots (GB300, sm_103a).
//
// One cluster of CTAs does it all: every warp owns a stretch of consecutive sequences, a lane each,
// three prefix sums (pages given back, pages taken, new tokens) run over lanes, warps and the
// cluster's CTAs, and what a warp's sequences give back, take and place is walked flat, a page or a
// token a lane and several at a time, so that uneven sequences cost what they hold.  Sums are 64 bits
// wide.  The slots of many tokens, which a cluster's few SMs would write at a fraction of HBM's rate,
// are left to a second launch over the whole GPU.
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

constexpr int kMaxWarps = 32;           // of a CTA
constexpr int kListed = 1024;           // sequences of a CTA up to which those that give back are dealt out
constexpr int kPerWarp = 8;             // sequences a warp, up to what the largest cluster holds
constexpr int kMaxCluster = 8;
constexpr int64_t kOwnTokens = 512;     // slots that the cluster writes itself, or one a sequence up to
constexpr int64_t kMostOwnTokens = 2048;
constexpr int kFillThreads = 256, kFillTokens = 8;   // of the second launch; tokens a thread

struct StepArgs {
    paged_kv_step_desc p;
    FastDiv div_page;
    int32_t per_warp;                   // sequences
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
#pragma unroll
    for (int by = 1; by < 32; by *= 2) {
        const Sums y = shift_up(x, by);
        if ((threadIdx.x & 31) >= by) x = x + y;
    }
    return x;
}

__device__ __forceinline__ Sums from_lane(const Sums &x, int lane)
{
    return Sums{__shfl_sync(0xffffffffu, x.back, lane), __shfl_sync(0xffffffffu, x.take, lane),
                __shfl_sync(0xffffffffu, x.tokens, lane)};
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

// Walks the items of a warp's lanes flat: a lane's items are [0, count), `before` is the sum of the
// counts of the lanes below (all of them fit 31 bits).  get(owner's lane, item, in) is called for 32 *
// kDeep of them before put(its result) is for the first, so that the loads of get are in flight
// together; past the last item in is false.  Both are called by the whole warp.
template <typename Get, typename Put>
__device__ __forceinline__ void walk(int before, int count, Get get, Put put)
{
    constexpr int kDeep = 4;
    const int lane = threadIdx.x & 31;
    const int all = __shfl_sync(0xffffffffu, before + count, 31);
    for (int e0 = 0; e0 < all; e0 += 32 * kDeep) {
        decltype(get(0, 0, false)) got[kDeep];
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            const int e = e0 + 32 * k + lane;
            int owner = 0;              // last lane whose items begin at or before e
#pragma unroll
            for (int step = 16; step > 0; step /= 2)
                if (__shfl_sync(0xffffffffu, before, owner + step) <= e) owner += step;
            got[k] = get(owner, e - __shfl_sync(0xffffffffu, before, owner), e < all);
        }
#pragma unroll
        for (int k = 0; k < kDeep; ++k) put(got[k]);
    }
}

__device__ __forceinline__ int warp_scan_int(int x)
{
#pragma unroll
    for (int by = 1; by < 32; by *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, x, by);
        if ((threadIdx.x & 31) >= by) x += y;
    }
    return x;
}

// The ids of a row that go back, 32 * kRowDeep entries in flight: act(id, how many of the row's before
// it).  Returns their number.  (A row at a time: flat, finding each entry's row cost more than the
// shorter chain of loads saved, 37 against 25 us for 4,096 sequences of which a tenth ended.)
template <typename Act>
__device__ __forceinline__ int walk_row(const int32_t *row, int entries, Act act)
{
    constexpr int kRowDeep = 8;
    const int lane = threadIdx.x & 31;
    int n = 0;
    for (int i0 = 0; i0 < entries; i0 += 32 * kRowDeep) {
        int id[kRowDeep];
#pragma unroll
        for (int k = 0; k < kRowDeep; ++k) {
            const int i = i0 + 32 * k + lane;
            id[k] = i < entries ? row[i] : -1;
        }
#pragma unroll
        for (int k = 0; k < kRowDeep; ++k) {
            if (i0 + 32 * k >= entries) break;
            const uint32_t valid = __ballot_sync(0xffffffffu, id[k] >= 0);
            if (id[k] >= 0) act(id[k], n + __popc(valid & ((1u << lane) - 1)));
            n += __popc(valid);
        }
    }
    return n;
}

__global__ void __launch_bounds__(32 * kMaxWarps) paged_step_kernel(const __grid_constant__ StepArgs a)
{
    __shared__ Sums s_warp[kMaxWarps], s_rank[kMaxCluster];
    __shared__ int64_t s_status[kMaxCluster];
    __shared__ int s_bits[kMaxWarps], s_over[kMaxWarps];
    __shared__ int s_list[kListed], s_gives[kListed], s_back[kListed];   // sequences that give back, their entries, their ids
    const paged_kv_step_desc &p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const uint32_t rank = cluster_rank(), ranks = cluster_size();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (a.fill) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (ranks > 1) cluster_arrive();                         // this CTA runs: its memory may be written

    // this warp's sequences, 32 at a time
    const int64_t first = (static_cast<int64_t>(rank) * warps + warp) * a.per_warp;
    const int begin = static_cast<int>(min(first, static_cast<int64_t>(p.n_seqs)));
    const int end = static_cast<int>(min(first + a.per_warp, static_cast<int64_t>(p.n_seqs)));
    const int count0 = min(max(*p.free_count, 0), static_cast<int>(p.n_free_max));
    int status = 0;
    auto row_at = [&](int s0, int &bits) { return s0 + lane < end ? load_row(a, s0 + lane, bits) : Row{}; };
    // calls act(row's entries, their number) for those of the 32 sequences from s0 on that give pages
    // back, in order
    auto each_back = [&](int s0, const Row &r, auto act) {
        uint32_t todo = __ballot_sync(0xffffffffu, r.gives > 0);
        while (todo != 0) {
            const int from = __ffs(todo) - 1;
            todo &= todo - 1;
            act(p.page_table + (s0 + from) * p.page_table_stride, __shfl_sync(0xffffffffu, r.gives, from));
        }
    };

    // ---- the sums of this warp's sequences
    const bool listed = static_cast<int64_t>(a.per_warp) * warps <= kListed;   // dealt to warps, as few end and long ones take long
    Row r0{};                                                // the first 32, which mostly are all
    Sums mine{};
    int over = 0;
    for (int s0 = begin; s0 < end; s0 += 32) {
        const Row r = row_at(s0, status);
        if (s0 == begin) r0 = r;
        mine.take += r.want - r.held;
        mine.tokens += r.fresh;
        if (listed) {
            over += __popc(__ballot_sync(0xffffffffu, r.gives > 0));
        } else {
            each_back(s0, r, [&](const int32_t *row, int entries) {
                const int n = walk_row(row, entries, [](int, int) {});
                if (lane == 0) mine.back += n;
            });
        }
    }
    Sums total = from_lane(warp_scan(mine), 31);
    status = __reduce_or_sync(0xffffffffu, status);
    if (lane == 0) {
        s_warp[warp] = total;
        s_bits[warp] = status;
        s_over[warp] = over;
    }
    __syncthreads();
    status = __reduce_or_sync(0xffffffffu, lane < warps ? s_bits[lane] : 0);
    const Sums upto = warp_scan(lane < warps ? s_warp[lane] : Sums{});
    const int over_upto = warp_scan_int(lane < warps ? s_over[lane] : 0);
    const int n_over = listed ? __shfl_sync(0xffffffffu, over_upto, 31) : 0;   // sequences in the CTA's list
    Sums all = from_lane(upto, 31), before = from_lane(upto, warp);
    before = Sums{before.back - total.back, before.take - total.take, before.tokens - total.tokens};
    if (n_over > 0) {
        int at = __shfl_sync(0xffffffffu, over_upto, warp) - over;
        for (int s0 = begin; s0 < end; s0 += 32) {
            int none = 0;
            const Row r = s0 == begin ? r0 : row_at(s0, none);
            const uint32_t gives = __ballot_sync(0xffffffffu, r.gives > 0);
            if (r.gives > 0) {
                const int place = at + __popc(gives & ((1u << lane) - 1));
                s_list[place] = s0 + lane;
                s_gives[place] = r.gives;
            }
            at += __popc(gives);
        }
        __syncthreads();
        for (int i = warp; i < n_over; i += warps) {
            const int n = walk_row(p.page_table + s_list[i] * p.page_table_stride, s_gives[i], [](int, int) {});
            if (lane == 0) s_back[i] = n;
        }
        __syncthreads();
        for (int i = lane; i < n_over; i += 32) all.back += s_back[i];   // (0 so far in every lane)
        for (int by = 16; by > 0; by /= 2) all.back += __shfl_xor_sync(0xffffffffu, all.back, by);
    }
    if (ranks > 1) {
        cluster_wait();
        if (threadIdx.x < ranks) {
            cluster_store64(&s_rank[rank].back, threadIdx.x, all.back);
            cluster_store64(&s_rank[rank].take, threadIdx.x, all.take);
            cluster_store64(&s_rank[rank].tokens, threadIdx.x, all.tokens);
            cluster_store64(&s_status[rank], threadIdx.x, status);
        }
        cluster_arrive();
        cluster_wait();
        all = Sums{};
        for (uint32_t r = 0; r < ranks; ++r) {
            if (r == rank) before = before + all;            // (listed: before.back is the CTA's, else the warp's)
            all = all + s_rank[r];
            status |= static_cast<int>(s_status[r]);
        }
    }
    const int64_t full = count0 + all.back;
    const int64_t count1 = min(full, p.n_free_max);
    // every thread of every CTA has read the count by now
    if (rank == 0 && threadIdx.x == 0) {
        if (all.take > count1) status |= STEP_NO_PAGES;
        if (full > p.n_free_max) status |= STEP_STACK_FULL;
        if (all.tokens > INT32_MAX || (p.slots != nullptr && all.tokens > p.max_tokens)) status |= STEP_TOKENS_PAST_END;
        *p.count_out = static_cast<int>(max(count1 - all.take, static_cast<int64_t>(0)));
        if (p.status != nullptr) *p.status = status;
    }

    // ---- pages go back, and are seen by every CTA before any is taken
    if (all.back > 0) {
        int64_t to = count0 + before.back;
        auto give = [&](const int32_t *row, int entries) {
            return walk_row(row, entries, [&](int id, int place) {
                if (to + place < p.n_free_max) p.free_pages[to + place] = id;
            });
        };
        int i0 = 0;                                          // those of the list before it are counted in `to`
        for (int i = warp; i < n_over; i += warps) {
            int64_t between = 0;
            for (int j = i0 + lane; j < i; j += 32) between += s_back[j];
            for (int by = 16; by > 0; by /= 2) between += __shfl_xor_sync(0xffffffffu, between, by);
            to += between;
            i0 = i;
            give(p.page_table + s_list[i] * p.page_table_stride, s_gives[i]);
        }
        for (int s0 = begin; s0 < end && !listed; s0 += 32) {
            int none = 0;
            each_back(s0, s0 == begin ? r0 : row_at(s0, none), [&](const int32_t *row, int entries) { to += give(row, entries); });
        }
        if (ranks > 1) {
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
    }

    // ---- lengths, pages taken, slots
    const bool slots = p.slots != nullptr && !a.fill;
    for (int s0 = begin; s0 < end; s0 += 32) {
        const int s = s0 + lane;
        int none = 0;
        const Row r = s0 == begin ? r0 : row_at(s0, none);
        const int takes = r.want - r.held;
        const Sums upto_lane = warp_scan(Sums{0, takes, r.fresh});
        const int takes_before = static_cast<int>(upto_lane.take) - takes;
        const int64_t tokens = before.tokens + upto_lane.tokens - r.fresh;   // new tokens before this sequence's
        const int64_t taken = before.take + takes_before;
        if (s < end) {
            p.kv_lens[s] = static_cast<int>(min(static_cast<int64_t>(r.past) + r.fresh, static_cast<int64_t>(INT32_MAX)));
            p.cu_seqlens[s + 1] = static_cast<int>(min(tokens + r.fresh, static_cast<int64_t>(INT32_MAX)));
            if (s == 0) p.cu_seqlens[0] = 0;
        }
        const int64_t top = count1 - 1 - taken;              // of the stack, for this sequence's first page
        struct Entry {
            int32_t *to;
            int id;
        };
        walk(takes_before, takes, [&](int owner, int item, bool in) {
            const int64_t from = __shfl_sync(0xffffffffu, top, owner) - item;
            const int held = __shfl_sync(0xffffffffu, r.held, owner);
            Entry e{nullptr, -1};
            if (in) {
                e.to = p.page_table + (s0 + owner) * p.page_table_stride + held + item;
                if (from >= 0) e.id = p.free_pages[from];
            }
            return e;
        }, [](const Entry &e) {
            if (e.to != nullptr) *e.to = e.id;
        });
        if (slots) {
            struct Slot {
                int64_t to, in_page;
                int id;
            };
            // whatever the lengths hold, no more tokens are walked than there are slots
            const int placed = static_cast<int>(max(min(static_cast<int64_t>(r.fresh), p.max_tokens - tokens), static_cast<int64_t>(0)));
            walk(warp_scan_int(placed) - placed, placed, [&](int owner, int item, bool in) {
                const int64_t to = __shfl_sync(0xffffffffu, tokens, owner) + item;
                const int64_t pos = __shfl_sync(0xffffffffu, r.past, owner) + item;
                const int64_t from_top = __shfl_sync(0xffffffffu, top, owner);
                const int held = __shfl_sync(0xffffffffu, r.held, owner);
                Slot e{in ? to : -1, 0, -1};
                if (in && pos < static_cast<int64_t>(p.max_pages) * p.page_size) {
                    const int index = static_cast<int>(fast_div(static_cast<uint32_t>(pos), a.div_page));
                    const int64_t from = from_top - (index - held);
                    e.in_page = pos - static_cast<int64_t>(index) * p.page_size;
                    if (index < held) e.id = p.page_table[(s0 + owner) * p.page_table_stride + index];
                    else if (from >= 0) e.id = p.free_pages[from];
                }
                return e;
            }, [&](const Slot &e) {
                if (e.to >= 0) p.slots[e.to] = e.id >= 0 ? static_cast<int64_t>(e.id) * p.page_size + e.in_page : -1;
            });
        }
        const Sums done = from_lane(upto_lane, 31);
        before.take += done.take;
        before.tokens += done.tokens;
    }
    if (slots)
        for (int64_t t = all.tokens + rank * blockDim.x + threadIdx.x; t < p.max_tokens; t += ranks * blockDim.x) p.slots[t] = -1;
    if (p.n_seqs == 0 && rank == 0 && threadIdx.x == 0) p.cu_seqlens[0] = 0;
}

// Slots of many tokens, from the arrays that the step has written.  A warp has 32 * kFillTokens
// consecutive tokens: it finds the sequence of the first by a 32-ary search in cu_seqlens, keeps that
// and the next 31 sequences' offsets, a lane each, finds every token's sequence among them by
// shuffles, and searches again only where the tokens go on past them.
__global__ void __launch_bounds__(kFillThreads) paged_slots_kernel(const __grid_constant__ StepArgs a)
{
    const paged_kv_step_desc &p = a.p;
    const int lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * (kFillThreads / 32) + (threadIdx.x >> 5)) * (32 * kFillTokens);
    const int n = p.n_seqs, total = p.cu_seqlens[n];
    int lo = 0, start = 0, end = 0, past = 0, past_window = 0;   // past_window: the first token past the sequences kept
    int seq[kFillTokens];
    uint32_t pos[kFillTokens];
#pragma unroll
    for (int k = 0; k < kFillTokens; ++k) {
        const int64_t t = t0 + 32 * k + lane;
        bool pending = t < total && t < p.max_tokens;
        seq[k] = -1;
        pos[k] = 0u;
        for (uint32_t todo; (todo = __ballot_sync(0xffffffffu, pending)) != 0;) {
            const int next = static_cast<int>(t0 + 32 * k + __ffs(todo) - 1);
            if (next >= past_window) {
                int len = n;
                lo = 0;
                while (len > 1) {                            // the last sequence that starts at or before `next`
                    const int step = (len + 31) >> 5, s = lo + lane * step;
                    const uint32_t vote = __ballot_sync(0xffffffffu, s < lo + len && p.cu_seqlens[s] <= next);
                    const int at = lo + (31 - __clz(vote)) * step;   // (the first lane's starts before it)
                    len = min(step, lo + len - at);
                    lo = at;
                }
                start = p.cu_seqlens[min(lo + lane, n)];
                end = p.cu_seqlens[min(lo + lane + 1, n)];
                // (not from kv_lens, which stops at 2^31 - 1)
                const bool fresh = lo + lane >= n || (p.finished != nullptr && p.finished[lo + lane] != 0);
                past = fresh ? 0 : max(p.past_lens[lo + lane], 0);
                past_window = __shfl_sync(0xffffffffu, end, 31);
            }
            const int mine = static_cast<int>(t);
            int owner = 0;
#pragma unroll
            for (int step = 16; step > 0; step /= 2)
                if (__shfl_sync(0xffffffffu, start, owner + step) <= mine) owner += step;
            const int in_new = mine - __shfl_sync(0xffffffffu, start, owner), before = __shfl_sync(0xffffffffu, past, owner);
            if (pending && mine < past_window) {
                seq[k] = lo + owner;
                pos[k] = min(static_cast<uint32_t>(before) + static_cast<uint32_t>(in_new), static_cast<uint32_t>(INT32_MAX));
                pending = false;
            }
        }
    }
    int id[kFillTokens];
    uint32_t in_page[kFillTokens];
#pragma unroll
    for (int k = 0; k < kFillTokens; ++k) {
        const uint32_t index = fast_div(pos[k], a.div_page);
        in_page[k] = pos[k] - index * static_cast<uint32_t>(p.page_size);
        id[k] = seq[k] >= 0 && index < static_cast<uint32_t>(p.max_pages) ? p.page_table[seq[k] * p.page_table_stride + index] : -1;
    }
#pragma unroll
    for (int k = 0; k < kFillTokens; ++k) {
        const int64_t t = t0 + 32 * k + lane;
        if (t < p.max_tokens) p.slots[t] = id[k] >= 0 ? static_cast<int64_t>(id[k]) * p.page_size + in_page[k] : -1;
    }
}

int check_step(const paged_kv_step_desc &p)
{
    if (p.n_seqs < 0 || p.n_seqs > kMaxTokens || p.max_pages < 0 || p.page_size < 1 || p.page_size > 65536 ||
        p.n_free_max < 0 || p.n_free_max > INT32_MAX || p.max_tokens < 0 || p.max_tokens > INT32_MAX ||
        (p.n_seqs > 1 && p.page_table_stride < p.max_pages) || p.page_table_stride > (int64_t(1) << 40))
        return ROPE_ERR_SHAPE;
    if (p.reserved != 0 || p.max_pages > (1 << 24) || static_cast<int64_t>(p.max_pages) * p.page_size > INT32_MAX / 2) return ROPE_ERR_UNSUPPORTED;
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
    // few warps for few sequences, then more CTAs, then more sequences a warp.  64 sequences, a
    // token each, 5.8 us; 4,096 with 940,000 new tokens and a tenth over 25.7 us (lengths and sums 5.6,
    // pages taken 4.2, pages given back 8.7, the slots 7.2)
    int64_t warps = (n + kPerWarp - 1) / kPerWarp;
    int cluster = 1;
    while (cluster < kMaxCluster && warps > kMaxWarps * cluster / 2) cluster *= 2;
    warps = (warps + cluster - 1) / cluster;
    warps = warps < 4 ? 4 : warps > kMaxWarps ? kMaxWarps : warps;
    a.per_warp = static_cast<int32_t>((n + cluster * warps - 1) / (cluster * warps));
    // A sequence's slots are one warp's in the first launch: 512 of one sequence 7.3 us, 513 by the second
    // launch 6.9, 16,384 8.5 (by a warp some 80); one each of 512 sequences 5.1, of 4,096 7.3, but 39 if all
    // 4,096 are one sequence's.
    const int64_t own = n < kOwnTokens ? kOwnTokens : n < kMostOwnTokens ? n : kMostOwnTokens;
    a.fill = desc->slots != nullptr && desc->max_tokens > own;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cluster));
    cfg.blockDim = dim3(static_cast<unsigned>(32 * warps));
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, paged_step_kernel, a) != cudaSuccess) return ROPE_ERR_LAUNCH;
    if (!a.fill) return ROPE_OK;
    const int64_t per_cta = kFillThreads * kFillTokens;
    cfg.gridDim = dim3(static_cast<unsigned>((desc->max_tokens + per_cta - 1) / per_cta));
    cfg.blockDim = dim3(kFillThreads);
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_slots_kernel, a) == cudaSuccess ? ROPE_OK : ROPE_ERR_LAUNCH;
}

// gqa_prefill_plan.cuh -- who computes what in prompt attention: one CTA reads the sequences' offsets and lengths, which
// only the device knows, and writes the work list.
//
// Items (two tiles of query rows each) are sorted by cost, longest first, and workers (one CTA an SM) take whole items in
// rounds, forth and back, as long as no worker passes its share of the total.  What is left is one line of steps that
// fills every worker up to its share: a worker's part of the line may begin and end within an item, and such parts leave
// partial results that a merge kernel joins.  So few rows over a long axis are spread over all SMs, long lists of items run
// whole and in step with one another (which shares K and V tiles in L2), and no SM waits for another at the end.
// The order is a function of the lengths alone (a stable counting sort), so the same call gives the same bits.
#pragma once

#include "gqa_common.cuh"
#include "gqa_prefill.h"

namespace gqa {

constexpr int kPlanThreads = 1024;
constexpr int kPlanBuckets = 64;
constexpr int kPlanExactRounds = 64;  // whose sums every worker works out for itself

// A step's cost with two tiles and with one, and what an item costs beside its steps, for all types and head sizes alike (a 4-bit step
// takes twice a bf16 one, one of d 64 less than one of d 128; only the balance is at stake).  Measured on two (us a call; 24 chunks of
// up to 256 tokens over an int8 cache, mixed step over an FP8 cache): 4, 3 and 4 88 and 1135, 4, 3 and 12 76 and 1129, 4, 4 and 4
// 91 and 1201, 4, 2 and 8 80 and 1184.
constexpr int kPreCostTwo = 4, kPreCostOne = 3, kPreCostItem = 12;

// First and one past the last row of sequence b, clamped into [0, total].
__device__ __forceinline__ void prefill_range(const int32_t *cu, int per, int b, int total, unsigned *err, int *from,
                                              int *to) {
    if (cu == nullptr) {
        *from = b * per, *to = (b + 1) * per;
        return;
    }
    const int f = cu[b], t = cu[b + 1];
    *from = min(max(f, 0), total);
    *to = min(max(t, *from), total);
    if (*from != f || *to != t) flag_error(err, kErrIndex);
}

// Sum of x before this thread, and of all; `sums` is shared memory for 33.  Every warp adds the warps' sums up by itself.
template <typename T, int THREADS>
__device__ __forceinline__ T block_exclusive_scan(T x, T *total, T *sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int WARPS = THREADS / 32;
    T inc = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += y;
    }
    __syncthreads();  // (`sums` may be in use by the scan before)
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    T s = lane < WARPS ? sums[lane] : T(0);
#pragma unroll
    for (int d = 1; d < WARPS; d <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += y;
    }
    *total = __shfl_sync(0xffffffffu, s, WARPS - 1);
    const T before = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
    return (warp > 0 ? before : T(0)) + inc - x;
}

// A sequence's rows and keys.
struct PlanSeq {
    int q_row, n, k_row, L;
};

template <bool PAGED>
__device__ __forceinline__ PlanSeq plan_seq(const PrefillArgs &a, int b, unsigned *err) {
    PlanSeq s;
    int t, kt;
    if constexpr (PAGED) {
        const int n = a.seq_lens[b];
        s.k_row = 0;
        kt = min(max(n, 0), a.pages_per_req * a.page_size);
        if (kt != n) flag_error(err, kErrIndex);
    } else {
        prefill_range(a.cu_k, a.per_k, b, a.Tk, err, &s.k_row, &kt);
    }
    prefill_range(a.cu_q, a.per_q, b, a.Tq, err, &s.q_row, &t);
    s.n = t - s.q_row;
    s.L = kt - s.k_row;
    return s;
}

__device__ __forceinline__ PrefillItem plan_item(const PrefillArgs &a, int b, const PlanSeq &s, int tile) {
    const int first = tile * 2 * a.tok_tile;
    PrefillItem it;
    it.q_row = s.q_row + first;
    it.n_tok = min(2 * a.tok_tile, s.n - first);
    it.req = b;
    it.L = s.L;
    it.k_row = s.k_row;
    it.limit0 = a.causal ? s.L - s.n + first + 1 : s.L;
    const int seen = a.causal ? min(max(it.limit0 + it.n_tok - 1, 0), s.L) : s.L;
    it.steps = (seen + kPreKeys - 1) / kPreKeys;
    it.cost = kPreCostItem + it.steps * (it.n_tok > a.tok_tile ? kPreCostTwo : kPreCostOne);
    return it;
}

__device__ __forceinline__ int plan_bucket(int cost, int top) {
    return kPlanBuckets - 1 - int((unsigned long long)unsigned(cost) * (kPlanBuckets - 1) / unsigned(top));
}

// The last i < n with prefix[i] <= x.
template <typename T, typename X>
__device__ __forceinline__ int plan_search(const T *prefix, int n, X x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (X(prefix[mid]) <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Shares of the sorted items: rounds of whole ones, the cuts of the line of the rest, and the items that several workers hold
// steps of.  prefix[i]: cost before item i (of one head block), prefix[n_items] the sum; in shared memory, or not.
template <typename T, int THREADS>
__device__ __forceinline__ void plan_shares(const PrefillArgs &a, int n_items, int top, const T *prefix, int2 *cuts, long long *sums,
                                            int *isums, int *shared_int) {
    const int tid = threadIdx.x;
    const int W = a.workers, HB = a.head_blocks;
    const int total = n_items * HB;
    const long long all_cost = (long long)prefix[n_items] * HB;
    // number / HB by a product, exact while number x HB < 2^32
    const unsigned inv = unsigned((1ull << 32) / unsigned(HB)) + 1;
    const bool by_product = HB > 1 && (unsigned long long)total * unsigned(HB) < (1ull << 32);
    auto item_of = [&](int number) { return HB == 1 ? number : by_product ? int(__umulhi(unsigned(number), inv)) : number / HB; };
    auto cost_of = [&](int number) {
        const int item = item_of(number);
        return int(prefix[item + 1] - prefix[item]);
    };
    auto number_of = [&](int r, int w) { return r * W + ((r & 1) ? W - 1 - w : w); };
    const int small = min(top, kPreCostItem + kPreMinSplit * kPreCostTwo);  // no part of an item is planned smaller
    const long long goal = max((all_cost + W - 1) / W, (long long)small);
    const int all_rounds = total / W;
    const bool exact = all_rounds <= kPlanExactRounds;
    // Whole rounds, as long as no worker passes its share of the total.
    int rounds = 0;
    long long load = 0;  // this worker's, after them
    if (exact) {
        if (all_rounds > 0) {
            if (tid == 0) *shared_int = all_rounds;
            __syncthreads();
            if (tid < W) {
                int r = 0;
                for (long long sum = 0; r < all_rounds; ++r) {
                    sum += cost_of(number_of(r, tid));
                    if (sum > goal) break;
                }
                atomicMin(shared_int, r);
            }
            __syncthreads();
            rounds = *shared_int;
            if (tid < W)
                for (int r = 0; r < rounds; ++r) load += cost_of(number_of(r, tid));
        }
    } else {
        // Many rounds: two of them, forth and back, are taken as even, as much as their first and last item together.
        long long done = 0;
        for (int r0 = 0;; r0 += THREADS) {
            const int r = r0 + tid;
            const long long c = (long long)(2 * r + 2) * W <= total ? cost_of(2 * r * W) + cost_of((2 * r + 2) * W - 1) : goal + 1;
            long long turn;
            const long long sum = block_exclusive_scan<long long, THREADS>(c, &turn, sums) + c + done;
            const int fit = __syncthreads_count(sum <= goal);
            rounds += 2 * fit;
            done += turn;
            if (fit < THREADS) break;
        }
    }
    // The rest is one line of steps that fills every worker up to its share of the total.
    const int n0 = rounds * W;
    const long long line = n0 < total ? (long long)prefix[item_of(n0)] * HB + (long long)(n0 - item_of(n0) * HB) * cost_of(n0) : all_cost;
    if (!exact) load = line / W;
    const long long need = tid < W ? max(goal - load, (long long)small) : 0;
    long long ignored;
    const long long pos = line + block_exclusive_scan<long long, THREADS>(need, &ignored, sums);
    if (tid < W) {
        int2 cut = make_int2(total, 0);
        if (tid == 0) {
            cut.x = n0;
        } else if (pos < all_cost) {
            // the item whose steps of all head blocks hold the place: prefix x HB <= pos
            int lo = 0, hi = n_items;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if ((long long)prefix[mid] * HB <= pos) lo = mid;
                else hi = mid;
            }
            const int4 *rec = reinterpret_cast<const int4 *>(a.items + lo);
            const int cost = int(prefix[lo + 1] - prefix[lo]);
            const unsigned long long rem = pos - (long long)prefix[lo] * HB;
            const int head = rem >> 32 ? int(rem / unsigned(cost)) : int(unsigned(rem) / unsigned(cost));
            const int y = int(rem - (unsigned long long)unsigned(head) * unsigned(cost));
            const int4 it = rec[0];  // q_row, n_tok, req, steps
            const int steps = it.w;
            int step = max(0, y - kPreCostItem);
            step = it.y > a.tok_tile ? step / kPreCostTwo : step / kPreCostOne;
            if (!a.may_split) step = 2 * y >= cost ? steps : 0;
            cut.x = lo * HB + head;
            if (steps - step < kPreSnap && 2 * y >= cost) cut.x += 1;
            else if (step >= kPreSnap && steps - step >= kPreSnap) cut.y = step;
        }
        cuts[tid] = cut;
        a.cuts[tid] = cut;
    }
    if (tid == 0) a.cuts[W] = cuts[W] = make_int2(total, 0);
    int n_joins = 0;
    if (a.may_split) {
        __syncthreads();
        // Items that several workers hold steps of.  (Cuts within one item are places apart: a worker's share of the line is
        // never less than a few steps.)
        bool first = false;
        int4 join;
        if (tid > 0 && tid < W) {
            const int2 cut = cuts[tid], prev = cuts[tid - 1];
            first = cut.y > 0 && !(prev.x == cut.x && prev.y > 0);
            int lo = tid, hi = W;  // the last worker whose share begins within the item
            while (first && hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cuts[mid].x == cut.x) lo = mid;
                else hi = mid;
            }
            join = make_int4(cut.x, tid - 1, lo, 0);
        }
        const int slot = block_exclusive_scan<int, THREADS>(int(first), &n_joins, isums);
        if (first) a.joins[slot] = join;
    }
    if (tid == 0) *reinterpret_cast<int4 *>(a.plan) = make_int4(n_items, rounds, total, n_joins);
}

// Few sequences and items (THREADS and THREADS x IPT at most, costs that add up in 32 bits): all in shared memory, one thread a
// sequence and IPT items.
template <bool PAGED, int THREADS, int IPT>
__global__ void __launch_bounds__(THREADS, 1) gqa_prefill_plan_small_kernel(const __grid_constant__ PrefillArgs a) {
    constexpr int WARPS = THREADS / 32, HIST = WARPS * kPlanBuckets, PER = HIST / THREADS;
    __shared__ int hist[WARPS][kPlanBuckets];
    __shared__ PlanSeq seq[THREADS];
    __shared__ int2 cuts[THREADS + 1];
    __shared__ int tiles[THREADS + 1];
    __shared__ unsigned prefix[THREADS * IPT + 1];
    __shared__ long long sums[33];
    __shared__ int isums[33], shared_max;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_launch_dependents();
    int mine = 0;
    if (tid < a.B) {
        const PlanSeq s = plan_seq<PAGED>(a, tid, a.err);
        seq[tid] = s;
        mine = (s.n + 2 * a.tok_tile - 1) / (2 * a.tok_tile);
    }
    if (tid == 0) shared_max = 1;
    for (int i = tid; i < HIST; i += THREADS) (&hist[0][0])[i] = 0;
    int n_items;
    const int at = block_exclusive_scan<int, THREADS>(mine, &n_items, isums);
    if (tid < a.B) tiles[tid] = at;
    // overlapping ranges of bad offsets (flagged) may hold more items than any good ones: what is past max_items is left out
    n_items = min(n_items, a.max_items);
    __syncthreads();
    PrefillItem own[IPT];
    int most = 1;
#pragma unroll
    for (int k = 0; k < IPT; ++k) {
        const int i = (warp * IPT + k) * 32 + lane;
        own[k].cost = 0;
        if (i < n_items) {
            const int b = plan_search(tiles, a.B, i);
            own[k] = plan_item(a, b, seq[b], i - tiles[b]);
            most = max(most, own[k].cost);
        }
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0 && most > 1) atomicMax(&shared_max, most);
    __syncthreads();
    const int top = shared_max;
    // stable counting sort, longest first: a warp counts and places a run of items
    const unsigned below = (1u << lane) - 1;
    int bucket[IPT], rank[IPT];
#pragma unroll
    for (int k = 0; k < IPT; ++k) {
        bucket[k] = own[k].cost > 0 ? plan_bucket(own[k].cost, top) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, bucket[k]);
        rank[k] = __popc(same & below);
        if (bucket[k] >= 0) rank[k] += hist[warp][bucket[k]];
        __syncwarp();
        if (bucket[k] >= 0 && (same & below) == 0) hist[warp][bucket[k]] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    {
        int x[PER], sum = 0;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int pos = PER * tid + e;  // bucket-major
            x[e] = hist[pos % WARPS][pos / WARPS];
            sum += x[e];
        }
        int all;
        int base = block_exclusive_scan<int, THREADS>(sum, &all, isums);
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int pos = PER * tid + e;
            hist[pos % WARPS][pos / WARPS] = base;
            base += x[e];
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < IPT; ++k) {
        if (bucket[k] < 0) continue;
        const int pos = hist[warp][bucket[k]] + rank[k];
        a.items[pos] = own[k];
        prefix[pos] = own[k].cost;
    }
    __syncthreads();
    unsigned cost[IPT], sum = 0, all;
#pragma unroll
    for (int k = 0; k < IPT; ++k) {
        const int i = tid * IPT + k;
        cost[k] = i < n_items ? prefix[i] : 0;
        sum += cost[k];
    }
    unsigned before = block_exclusive_scan<unsigned, THREADS>(sum, &all, reinterpret_cast<unsigned *>(isums));
#pragma unroll
    for (int k = 0; k < IPT; ++k) {
        const int i = tid * IPT + k;
        if (i < n_items) prefix[i] = before;
        before += cost[k];
    }
    if (tid == 0) prefix[n_items] = all;
    __syncthreads();
    plan_shares<unsigned, THREADS>(a, n_items, top, prefix, cuts, sums, isums, &shared_max);
}

// Any number of them, through the workspace.
template <bool PAGED>
__global__ void __launch_bounds__(kPlanThreads, 1) gqa_prefill_plan_kernel(const __grid_constant__ PrefillArgs a) {
    __shared__ int hist[kPlanThreads / 32][kPlanBuckets];
    __shared__ int2 cuts[kPlanThreads + 1];
    __shared__ long long sums[33];
    __shared__ int isums[33], shared_max;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_launch_dependents();
    const int tpi = 2 * a.tok_tile;
    const int per_thread = (a.B + kPlanThreads - 1) / kPlanThreads;
    // overlapping ranges of bad offsets (flagged) may hold more items than any good ones: what is past max_items is left out
    long long mine = 0, all_items;
    for (int b = tid * per_thread; b < min((tid + 1) * per_thread, a.B); ++b)
        mine += (plan_seq<PAGED>(a, b, a.err).n + tpi - 1) / tpi;
    if (tid == 0) shared_max = 1;
    for (int i = tid; i < (kPlanThreads / 32) * kPlanBuckets; i += kPlanThreads) (&hist[0][0])[i] = 0;
    long long at = block_exclusive_scan<long long, kPlanThreads>(mine, &all_items, sums);
    for (int b = tid * per_thread; b < min((tid + 1) * per_thread, a.B); ++b) {
        a.tile_prefix[b] = int(min(at, (long long)a.max_items));
        at += (plan_seq<PAGED>(a, b, nullptr).n + tpi - 1) / tpi;
    }
    const int n_items = int(min(all_items, (long long)a.max_items));
    __syncthreads();
    int most = 1;
    for (int i = tid; i < n_items; i += kPlanThreads) {
        const int b = plan_search(a.tile_prefix, a.B, i);
        const PrefillItem it = plan_item(a, b, plan_seq<PAGED>(a, b, nullptr), i - a.tile_prefix[b]);
        a.unsorted[i] = it;
        most = max(most, it.cost);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) atomicMax(&shared_max, most);
    __syncthreads();
    const int top = shared_max;
    const int run = (n_items + kPlanThreads - 1) / kPlanThreads * 32;
    const unsigned below = (1u << lane) - 1;
    for (int i = warp * run + lane; i < (warp + 1) * run; i += 32) {
        const bool there = i < n_items;
        const int bucket = there ? plan_bucket(a.unsorted[i].cost, top) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, bucket);
        if (there && (same & below) == 0) hist[warp][bucket] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    {
        constexpr int WARPS = kPlanThreads / 32, PER = kPlanBuckets / 32;
        int x[PER], sum = 0;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int pos = PER * tid + e;
            x[e] = hist[pos % WARPS][pos / WARPS];
            sum += x[e];
        }
        int all;
        int base = block_exclusive_scan<int, kPlanThreads>(sum, &all, isums);
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int pos = PER * tid + e;
            hist[pos % WARPS][pos / WARPS] = base;
            base += x[e];
        }
    }
    __syncthreads();
    for (int i = warp * run + lane; i < (warp + 1) * run; i += 32) {
        const bool there = i < n_items;
        PrefillItem it = {};
        if (there) it = a.unsorted[i];
        const int bucket = there ? plan_bucket(it.cost, top) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, bucket);
        if (there) a.items[hist[warp][bucket] + __popc(same & below)] = it;
        __syncwarp();
        if (there && (same & below) == 0) hist[warp][bucket] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    const int share = (n_items + kPlanThreads - 1) / kPlanThreads;
    long long cost = 0, all_cost;
    for (int i = tid * share; i < min((tid + 1) * share, n_items); ++i) cost += a.items[i].cost;
    long long before = block_exclusive_scan<long long, kPlanThreads>(cost, &all_cost, sums);
    for (int i = tid * share; i < min((tid + 1) * share, n_items); ++i) {
        a.cost_prefix[i] = before;
        before += a.items[i].cost;
    }
    if (tid == 0) a.cost_prefix[n_items] = all_cost;
    __syncthreads();
    plan_shares<long long, kPlanThreads>(a, n_items, top, a.cost_prefix, cuts, sums, isums, &shared_max);
}

// One piece of a worker's work, as it lies in shared memory for all roles of the CTA.
struct __align__(16) PrefillPiece {
    int q_row, n_tok, req, units;  // units: (tile, step) pairs, in the order of their products; negative behind the last piece
    int limit0, L, k_row, first_limit;  // first_limit: keys that every row sees
    int g, hb, s0, s1;             // KV head, block of its query heads, steps
    int slot;                      // of the partial results; -1: the whole item
    int two;                       // two tiles of rows; one tile otherwise, whose steps the two row groups take in turns
    int spare[2];
};
static_assert(sizeof(PrefillPiece) == 64, "four 16-byte words");

__device__ __forceinline__ PrefillPiece piece_of(const PrefillArgs &a, const PrefillItem &it, int h, int s0, int s1, int slot) {
    const int per = a.head_blocks / a.Hkv;
    PrefillPiece p;
    p.q_row = it.q_row, p.n_tok = it.n_tok, p.req = it.req;
    p.limit0 = it.limit0, p.L = it.L, p.k_row = it.k_row;
    p.g = h / per;
    p.hb = h % per;
    p.s0 = s0;
    p.s1 = s1;
    p.slot = slot;
    p.two = it.n_tok > a.tok_tile;
    p.units = (s1 - s0) * (p.two ? 2 : 1);
    p.first_limit = a.causal ? min(max(it.limit0, 0), it.L) : it.L;
    return p;
}

// Without a plan: the warp works out which item is number `n`, whole.  Returns false past the last one.
template <bool PAGED>
__device__ __forceinline__ bool direct_piece(const PrefillArgs &a, int n, PrefillPiece *p) {
    const int lane = threadIdx.x & 31, item = n / a.head_blocks;
    int before = 0, b = -1, tile = 0;
    PlanSeq found = {};
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        PlanSeq s = {};
        int tiles = 0;
        if (b0 + lane < a.B) {
            s = plan_seq<PAGED>(a, b0 + lane, a.err);
            tiles = (s.n + 2 * a.tok_tile - 1) / (2 * a.tok_tile);
        }
        int inc = tiles;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += y;
        }
        const unsigned here = __ballot_sync(0xffffffffu, before + inc - tiles <= item && item < before + inc);
        if (here != 0) {
            const int src = __ffs(here) - 1;
            b = b0 + src;
            tile = item - __shfl_sync(0xffffffffu, before + inc - tiles, src);
            found = {__shfl_sync(0xffffffffu, s.q_row, src), __shfl_sync(0xffffffffu, s.n, src), __shfl_sync(0xffffffffu, s.k_row, src),
                     __shfl_sync(0xffffffffu, s.L, src)};
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (b < 0) return false;
    const PrefillItem it = plan_item(a, b, found, tile);
    *p = piece_of(a, it, n % a.head_blocks, 0, it.steps, -1);
    return true;
}

// Walks a worker's pieces.  The item after the present one is under way meanwhile.
struct PrefillWalk {
    const PrefillArgs &a;
    int w, r, rounds, n, s0;
    int2 from, end;
    bool line, more;  // in the divided part; there is a piece ahead
    int4 x, y;        // its item
    __device__ __forceinline__ PrefillWalk(const PrefillArgs &args, int worker)
        : a(args), w(worker), r(0), n(0), s0(0), line(false), more(false) {
        rounds = a.plan->rounds;
        from = a.cuts[w];
        end = a.cuts[w + 1];
        ahead();
    }
    __device__ __forceinline__ void ahead() {
        s0 = 0;
        if (line) {
            ++n;
        } else if (r < rounds) {
            n = r * a.workers + ((r & 1) ? a.workers - 1 - w : w);
            ++r;
        } else {
            n = from.x;
            s0 = from.y;
            line = true;
        }
        more = !(line && (n > end.x || (n == end.x && s0 >= end.y)));
        if (more) {
            // (not through the read-only path: the plan may be written while this kernel starts)
            const int4 *src = reinterpret_cast<const int4 *>(a.items + n / a.head_blocks);
            x = src[0];
            y = src[1];
        }
    }
    __device__ __forceinline__ void next(PrefillPiece *p) {
        if (!more) {
            p->units = -1;
            return;
        }
        const PrefillItem it = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        const int s1 = line && n == end.x ? end.y : it.steps;
        *p = piece_of(a, it, n % a.head_blocks, s0, s1, s0 > 0 ? 2 * w : s1 < it.steps ? 2 * w + 1 : -1);
        ahead();
    }
};

constexpr int kPrePieces = 4;  // pieces that are known ahead

// What the roles share to follow the pieces: warp W_LOAD writes them, every other warp reads them and says so.
struct PieceFeed {
    PrefillPiece *ring;
    uint64_t *full, *empty;
    int at;
    uint32_t phase;
    __device__ __forceinline__ PieceFeed(PrefillPiece *r, uint64_t *f, uint64_t *e) : ring(r), full(f), empty(e), at(0), phase(0) {}
    __device__ __forceinline__ bool ready() const { return mbar_test_wait(&full[at], phase); }
    // The next piece, or null: behind the last one, or a wait that ran out (*ok).
    __device__ __forceinline__ const volatile PrefillPiece *next(uint64_t limit, volatile int *abort_flag, bool *ok) {
        *ok = mbar_wait_bounded(&full[at], phase, limit, abort_flag);
        if (!*ok || const_cast<volatile PrefillPiece *>(ring)[at].units < 0) return nullptr;
        return ring + at;
    }
    __device__ __forceinline__ void done() {  // one lane of the warp, once all are
        mbar_arrive(&empty[at]);
    }
    __device__ __forceinline__ void step() {
        if (++at == kPrePieces) at = 0, phase ^= 1;
    }
};

}  // namespace gqa

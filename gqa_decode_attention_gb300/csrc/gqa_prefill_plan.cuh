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

// A step's cost with two tiles and with one, and what an item costs beside its steps.
constexpr int kPreCostTwo = 4, kPreCostOne = 3, kPreCostItem = 4;

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

template <typename T>
__device__ __forceinline__ T block_exclusive_scan(T x, T *total, T *warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T inc = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += y;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        T s = lane < kPlanThreads / 32 ? warp_sums[lane] : T(0);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const T y = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += y;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    const T before = warp > 0 ? warp_sums[warp - 1] : T(0);
    *total = warp_sums[kPlanThreads / 32 - 1];
    __syncthreads();
    return before + inc - x;
}

template <bool PAGED>
__device__ __forceinline__ PrefillItem plan_item(const PrefillArgs &a, int b, int tile, unsigned *err) {
    int f, t, kf = 0, kt;
    prefill_range(a.cu_q, a.per_q, b, a.Tq, nullptr, &f, &t);
    if constexpr (PAGED) {
        const int n = a.seq_lens[b];
        kt = min(max(n, 0), a.pages_per_req * a.page_size);
        if (kt != n) flag_error(err, kErrIndex);
    } else {
        prefill_range(a.cu_k, a.per_k, b, a.Tk, err, &kf, &kt);
    }
    const int tpi = 2 * a.tok_tile;
    PrefillItem it;
    it.q_row = f + tile * tpi;
    it.n_tok = min(tpi, t - it.q_row);
    it.req = b;
    it.L = kt - kf;
    it.k_row = kf;
    it.limit0 = a.causal ? it.L - (t - f) + tile * tpi + 1 : it.L;
    const int seen = a.causal ? min(max(it.limit0 + it.n_tok - 1, 0), it.L) : it.L;
    it.steps = (seen + kPreKeys - 1) / kPreKeys;
    it.cost = kPreCostItem + it.steps * (it.n_tok > a.tok_tile ? kPreCostTwo : kPreCostOne);
    return it;
}

// SMALL: at most one sequence and one item a thread, nothing but the results in global memory.
template <bool PAGED, bool SMALL>
__global__ void __launch_bounds__(kPlanThreads, 1) gqa_prefill_plan_kernel(const __grid_constant__ PrefillArgs a) {
    __shared__ int hist[kPlanThreads / 32][kPlanBuckets];
    __shared__ int tile_prefix_s[SMALL ? kPlanThreads + 1 : 1];
    __shared__ long long cost_prefix_s[SMALL ? kPlanThreads + 1 : 1];
    __shared__ int2 cuts_s[kPlanThreads + 1];
    __shared__ long long sums[32];
    __shared__ int isums[32];
    __shared__ int shared_max;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_launch_dependents();
    const int tpi = 2 * a.tok_tile;
    int *tile_prefix = SMALL ? tile_prefix_s : a.tile_prefix;
    long long *cost_prefix = SMALL ? cost_prefix_s : a.cost_prefix;

    // tiles before each sequence
    const int per_thread = SMALL ? 1 : (a.B + kPlanThreads - 1) / kPlanThreads;
    int mine = 0;
    for (int i = 0; i < per_thread; ++i) {
        const int b = tid * per_thread + i;
        if (b >= a.B) break;
        int f, t;
        prefill_range(a.cu_q, a.per_q, b, a.Tq, a.err, &f, &t);
        mine += (t - f + tpi - 1) / tpi;
    }
    if (tid == 0) shared_max = 1;
    for (int i = tid; i < (kPlanThreads / 32) * kPlanBuckets; i += kPlanThreads) (&hist[0][0])[i] = 0;
    int n_items;
    int at = block_exclusive_scan(mine, &n_items, isums);
    if constexpr (SMALL) {
        if (tid < a.B) tile_prefix[tid] = at;
        if (tid == a.B - 1) tile_prefix[a.B] = at + mine;
    } else {
        for (int i = 0; i < per_thread; ++i) {
            const int b = tid * per_thread + i;
            if (b >= a.B) break;
            int f, t;
            prefill_range(a.cu_q, a.per_q, b, a.Tq, nullptr, &f, &t);
            tile_prefix[b] = at;
            at += (t - f + tpi - 1) / tpi;
            if (b == a.B - 1) tile_prefix[a.B] = at;
        }
    }
    // overlapping ranges of bad offsets (flagged already) may hold more than any good ones
    n_items = min(n_items, a.max_items);
    __syncthreads();

    auto item_at = [&](int i) {
        int lo = 0, hi = a.B;  // the last sequence with tile_prefix <= i
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (tile_prefix[mid] <= i) lo = mid;
            else hi = mid;
        }
        return plan_item<PAGED>(a, lo, i - tile_prefix[lo], a.err);
    };
    PrefillItem own = {};
    int most = 1;
    if constexpr (SMALL) {
        if (tid < n_items) own = item_at(tid);
        most = max(1, own.cost);
    } else {
        for (int i = tid; i < n_items; i += kPlanThreads) {
            const PrefillItem it = item_at(i);
            a.unsorted[i] = it;
            most = max(most, it.cost);
        }
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) atomicMax(&shared_max, most);
    __syncthreads();
    const int top = shared_max;

    // stable counting sort, longest first: a warp counts and places a run of items
    const int run = (n_items + kPlanThreads - 1) / kPlanThreads * 32;
    auto bucket_of = [&](int cost) { return kPlanBuckets - 1 - int((unsigned long long)unsigned(cost) * (kPlanBuckets - 1) / unsigned(top)); };
    const unsigned below = (1u << lane) - 1;
    for (int i = warp * run + lane; i < (warp + 1) * run; i += 32) {
        const bool there = i < n_items;
        const int bucket = there ? bucket_of(SMALL ? own.cost : a.unsorted[i].cost) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, bucket);
        if (there && (same & below) == 0) hist[warp][bucket] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    {
        int x[2], sum = 0;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int pos = 2 * tid + e;  // bucket-major
            x[e] = hist[pos % (kPlanThreads / 32)][pos / (kPlanThreads / 32)];
            sum += x[e];
        }
        int all;
        int base = block_exclusive_scan(sum, &all, isums);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int pos = 2 * tid + e;
            hist[pos % (kPlanThreads / 32)][pos / (kPlanThreads / 32)] = base;
            base += x[e];
        }
    }
    __syncthreads();
    for (int i = warp * run + lane; i < (warp + 1) * run; i += 32) {
        const bool there = i < n_items;
        PrefillItem it = own;
        if (!SMALL && there) it = a.unsorted[i];
        const int bucket = there ? bucket_of(it.cost) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, bucket);
        if (there) {
            const int pos = hist[warp][bucket] + __popc(same & below);
            a.items[pos] = it;
            if (SMALL) cost_prefix[pos] = it.cost;
        }
        __syncwarp();
        if (there && (same & below) == 0) hist[warp][bucket] += __popc(same);
        __syncwarp();
    }
    __syncthreads();

    // cost before each item
    const int share = SMALL ? 1 : (n_items + kPlanThreads - 1) / kPlanThreads;
    long long cost = 0, all_cost;
    if constexpr (SMALL) cost = tid < n_items ? cost_prefix[tid] : 0;
    else
        for (int i = tid * share; i < min((tid + 1) * share, n_items); ++i) cost += a.items[i].cost;
    long long before = block_exclusive_scan(cost, &all_cost, sums);
    for (int i = tid * share; i < min((tid + 1) * share, n_items); ++i) {
        cost_prefix[i] = before;
        if (!SMALL) before += a.items[i].cost;
    }
    if (tid == 0) cost_prefix[n_items] = all_cost;
    __syncthreads();

    // Whole rounds, as long as no worker passes its share of the total.
    const int W = a.workers, HB = a.head_blocks;
    const int total = n_items * HB;
    auto cost_of = [&](int number) {
        const int item = unsigned(number) / unsigned(HB);
        return int(cost_prefix[item + 1] - cost_prefix[item]);
    };
    auto number_of = [&](int r, int w) { return r * W + ((r & 1) ? W - 1 - w : w); };
    const long long goal = max((all_cost * HB + W - 1) / W, (long long)min(top, kPreCostItem + kPreMinSplit * kPreCostTwo));
    const bool exact = total / W <= kPlanExactRounds;
    int rounds = 0;
    long long load = 0;  // this worker's, after them
    if (exact) {
        if (tid == 0) shared_max = total / W;
        __syncthreads();
        if (tid < W) {
            int r = 0;
            for (long long sum = 0; r < total / W; ++r) {
                sum += cost_of(number_of(r, tid));
                if (sum > goal) break;
            }
            atomicMin(&shared_max, r);
        }
        __syncthreads();
        rounds = shared_max;
        if (tid < W)
            for (int r = 0; r < rounds; ++r) load += cost_of(number_of(r, tid));
    } else {
        // Many rounds: two of them, forth and back, are taken as even, as much as their first and last item together.
        long long done = 0;
        for (int r0 = 0;; r0 += kPlanThreads) {
            const int r = r0 + tid;
            const long long c = (long long)(2 * r + 2) * W <= total ? cost_of(2 * r * W) + cost_of((2 * r + 2) * W - 1) : goal + 1;
            long long turn;
            const long long sum = block_exclusive_scan(c, &turn, sums) + c + done;
            const int fit = __syncthreads_count(sum <= goal);
            rounds += 2 * fit;
            done += turn;
            if (fit < kPlanThreads) break;
        }
    }
    // The rest is one line of steps that fills every worker up to its share of the total; no part of it is too small.
    const int n0 = rounds * W;
    const long long line = n0 < total ? cost_prefix[n0 / HB] * HB + (long long)(n0 % HB) * cost_of(n0) : all_cost * HB;
    if (!exact) load = line / W;
    const long long need = tid < W ? max(goal - load, (long long)min(top, kPreCostItem + kPreMinSplit * kPreCostTwo)) : 0;
    long long ignored;
    const long long skip = block_exclusive_scan(need, &ignored, sums);
    if (tid < W) {
        int2 cut = make_int2(total, 0);
        const long long pos = line + skip;
        if (tid == 0) {
            cut.x = n0;
        } else if (pos < all_cost * HB) {
            int lo = 0, hi = n_items;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cost_prefix[mid] * HB <= pos) lo = mid;
                else hi = mid;
            }
            const PrefillItem it = a.items[lo];
            const long long rem = pos - cost_prefix[lo] * HB;
            const int head = int(rem / it.cost), y = int(rem % it.cost);
            int step = max(0, y - kPreCostItem) / (it.n_tok > a.tok_tile ? kPreCostTwo : kPreCostOne);
            if (!a.may_split) step = 2 * y >= it.cost ? it.steps : 0;
            cut.x = lo * HB + head;
            if (it.steps - step < kPreSnap && 2 * y >= it.cost) cut.x += 1;
            else if (step >= kPreSnap && it.steps - step >= kPreSnap) cut.y = step;
        }
        cuts_s[tid] = cut;
        a.cuts[tid] = cut;
    }
    if (tid == 0) a.cuts[W] = cuts_s[W] = make_int2(total, 0);
    __syncthreads();
    // items that several workers hold steps of
    bool first = false;
    int2 join;
    if (tid > 0 && tid < W) {
        const int2 cut = cuts_s[tid], prev = cuts_s[tid - 1];
        first = cut.y > 0 && !(prev.x == cut.x && prev.y > 0);
        int lo = tid, hi = W;  // the last worker whose share begins within the item
        while (first && hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cuts_s[mid].x == cut.x) lo = mid;
            else hi = mid;
        }
        join = make_int2(tid, lo);
    }
    int n_joins;
    const int slot = block_exclusive_scan(int(first), &n_joins, isums);
    if (first) a.joins[slot] = join;
    if (tid == 0) {
        a.plan->n_items = n_items;
        a.plan->rounds = rounds;
        a.plan->total = total;
        a.plan->n_joins = n_joins;
    }
}

// One piece of a worker's work.
struct PrefillPiece {
    PrefillItem item;
    int g, hb;   // KV head, block of its query heads
    int s0, s1;
    int slot;    // of the partial results; -1: the whole item
    bool two;    // two tiles of rows; one tile otherwise, whose steps the two row groups take in turns
    int units;   // (tile, step) pairs, in the order of their products
    int first_limit;  // keys that every row sees
    __device__ __forceinline__ int units_of(int t) const { return two ? s1 - s0 : (s1 - s0 + 1 - t) / 2; }
    __device__ __forceinline__ int step_of(int u) const { return s0 + (two ? u >> 1 : u); }
    // keys past what some row sees lie in this step
    __device__ __forceinline__ bool masked(int step) const { return (step + 1) * kPreKeys > first_limit; }
};

// Walks a worker's pieces; every role of the CTA does so by itself.  The item after the present one is under way meanwhile.
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
    __device__ __forceinline__ bool next(PrefillPiece *p) {
        if (!more) return false;
        p->item = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        const int h = n % a.head_blocks;
        const int per = a.head_blocks / a.Hkv;
        p->g = h / per;
        p->hb = h % per;
        p->s0 = s0;
        p->s1 = line && n == end.x ? end.y : p->item.steps;
        p->slot = s0 > 0 ? 2 * w : p->s1 < p->item.steps ? 2 * w + 1 : -1;
        p->two = p->item.n_tok > a.tok_tile;
        p->units = (p->s1 - p->s0) * (p->two ? 2 : 1);
        p->first_limit = a.causal ? min(max(p->item.limit0, 0), p->item.L) : p->item.L;
        ahead();
        return true;
    }
};

}  // namespace gqa

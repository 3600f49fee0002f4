// tables.cu -- block tables, positions and slot maps of a batch, from the
// lengths of its requests (section 6.3 of "From MLA to CSA + HCA" for the
// compressed slot mapping; the page rules are stated in the header).
//
// One launch.  Where a sequence's tokens, new pages and returned pages start
// is an exclusive prefix sum over the sequences before it: every CTA forms
// all of these sums for itself (at most 4096 sequences of 8 bytes, out of
// L2), which costs less than a second launch or a wait between CTAs.  Half of
// its warps count and add, the others meanwhile copy what does not depend on
// the sums, the tables' old entries; who is done helps with the rest.
// Small batches are bound by latency: the lengths, the sums, the pages, each
// read behind the last, and the code itself, fetched anew by every launch (32
// sequences 4.7 us; 0.3 us more with the counting loop over the groups unrolled).
// Large ones by issuing instructions: the sums that every CTA repeats and the
// rules of each row (2048 sequences of up to 128K tokens, three groups: 14.2 us,
// where writing the tables and reading the pages held takes 4.6 us).
#include <limits.h>

#include <type_traits>

#include "dsv4_common.cuh"
#include "host_once.h"
#include "tmap.h"

namespace dsv4 {

constexpr int kTabThreads = 1024;
constexpr int kTabWarps = kTabThreads / 32;
constexpr int kTabCounters = 512;                       // threads that count
constexpr int kTabMaxSeqs = 4096;
constexpr int kTabSeg = 1024;                           // table entries per warp and unit of work
constexpr int kTabGroups = DSV4_MAX_TABLE_GROUPS;

struct TabGroup {
    int shift;               // log2 of the tokens per entry
    int window;
    int num_pages;
    int stride;
    int segs;                // units of kTabSeg entries per row
    unsigned units;          // of all rows
    int vec;                 // rows of owned and table are 16-byte aligned
    int* owned;
    int* table;
    int* ring;
    unsigned ring_size;
    const long long* pool_in;
    long long* pool_out;
    long long* slots;
};

struct TabParams {
    int num_seqs, max_tokens, num_groups;
    unsigned units;          // table units of all groups
    const int* computed;
    const int* fresh;
    int* offsets;
    int* ctx_len;
    int* positions;
    int* seqs;
    int* row_ctx;
    TabGroup g[kTabGroups];
    int* status;
};

__device__ __forceinline__ int pages_of(int tokens, int shift)
{
    return static_cast<int>((static_cast<unsigned>(tokens >> shift) + kPage - 1) / kPage);   // tokens up to INT_MAX
}

__device__ __forceinline__ int first_live(int tokens, int window)
{
    return (window > 0 && tokens >= window) ? (tokens - window + 1) / kPage : 0;
}

// A sequence's lengths: c tokens computed, n new, done; one that is refused
// counts as done with nothing computed (and nothing to return).
struct SeqLen {
    int c, n;
    bool done;
    int bad;
};

// What every sequence is measured by; groups that are not used measure nothing.
struct TabRules {
    int shift[kTabGroups], window[kTabGroups], stride[kTabGroups];

    __device__ __forceinline__ explicit TabRules(const TabParams& P)
    {
#pragma unroll
        for (int g = 0; g < kTabGroups; ++g) {
            const bool used = g < P.num_groups;
            shift[g] = used ? P.g[g].shift : 0;
            window[g] = used ? P.g[g].window : 0;
            stride[g] = used ? P.g[g].stride : INT_MAX;
        }
    }
};

__device__ __forceinline__ SeqLen seq_len(const TabRules& R, int c, int n)
{
    SeqLen q;
    q.c = c;
    q.n = n;
    q.done = q.n == -1;
    q.bad = 0;
    if (q.c < 0 || q.n < -1 || q.c > INT_MAX - max(q.n, 0)) {
        q.bad = DSV4_DEV_BAD_POSITION;
    } else {
        const int end = q.c + max(q.n, 0);
#pragma unroll
        for (int g = 0; g < kTabGroups; ++g)
            if (pages_of(end, R.shift[g]) > R.stride[g]) q.bad = DSV4_DEV_BAD_PAGE;
    }
    if (q.bad) q.c = 0;
    if (q.bad || q.done) {
        q.n = 0;
        q.done = true;
    }
    return q;
}

// Pages of a group that the sequence has from and to, takes up to and returns
// up to.
__device__ __forceinline__ void seq_pages(int shift, int window, const SeqLen& q, int& lo, int& before, int& after,
                                          int& gone)
{
    lo = first_live(q.c, window);
    before = pages_of(q.c, shift);
    after = pages_of(q.c + q.n, shift);
    gone = q.done ? before : first_live(q.c + q.n, window);
}

// Position base + off of a ring, base < 2 size (a position plus an offset within
// what is taken or returned), off < size: below 3 * 2^31 no sum wraps twice.
__device__ __forceinline__ unsigned ring_at(unsigned base, unsigned off, unsigned size)
{
    unsigned i = base >= size ? base - size : base;
    i += off;
    return i >= size ? i - size : i;
}

// x modulo size, x >= 0; 32-bit unless the counters have run that far.
__device__ __forceinline__ unsigned ring_base(long long x, unsigned size)
{
    if (x <= 0xffffffffll) return static_cast<unsigned>(x) % size;
    return static_cast<unsigned>(x % static_cast<long long>(size));
}

// What a step does with a group's ring: nothing; every CTA with its own rows'
// pages; or one CTA with all of them, where returned pages go to places that the
// step's taken ones are read from.
enum { kRefused = 0, kShared = 1, kAlone = 2 };

struct TabShared {
    int total[2 * kTabGroups + 1];                 // taken and returned pages by group, tokens (at most max_tokens + 1)
    unsigned head[kTabGroups], tail[kTabGroups];   // ring positions
    int ok[kTabGroups];                            // kRefused, kShared or kAlone
    unsigned alone;                                // bit g: group g is kAlone
    unsigned next;                                 // the next of the CTA's units of old entries
};

// Exclusive prefix sums in place of v[0, n), n a multiple of 8 (a whole warp);
// no sum exceeds `most`, where they stay.  Returns the total.
__device__ __forceinline__ int warp_prefix(int* v, int n, int most, int lane)
{
    int base = 0;
    for (int i0 = 0; i0 < n; i0 += 256) {
        const int i = i0 + 8 * lane;
        int4 a = make_int4(0, 0, 0, 0), b = a;
        if (i < n) {
            a = *reinterpret_cast<const int4*>(v + i);
            b = *reinterpret_cast<const int4*>(v + i + 4);
        }
        // each at most `most` <= 2^24 + 1 or, for pages, all together below 2^31
        const int s1 = a.x, s2 = min(s1 + a.y, most), s3 = min(s2 + a.z, most), s4 = min(s3 + a.w, most),
                  s5 = min(s4 + b.x, most), s6 = min(s5 + b.y, most), s7 = min(s6 + b.z, most), sum = min(s7 + b.w, most);
        int x = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        const int at = base + x - sum;
        if (i < n) {
            *reinterpret_cast<int4*>(v + i) = make_int4(at, at + s1, at + s2, at + s3);
            *reinterpret_cast<int4*>(v + i + 4) = make_int4(at + s4, at + s5, at + s6, at + s7);
        }
        base = min(base + __shfl_sync(0xffffffffu, x, 31), most);
    }
    return base;
}

// Unit u of the table rows: kTabSeg entries [j0, j1) of group g's row s.
struct TabUnit {
    int g, s, j0, j1;
};

__device__ __forceinline__ TabUnit table_unit(const TabParams& P, unsigned u)
{
    TabUnit t;
    t.g = 0;
    while (u >= P.g[t.g].units) u -= P.g[t.g++].units;
    const TabGroup& G = P.g[t.g];
    const unsigned row = G.segs == 1 ? u : u / G.segs;
    t.s = row;
    t.j0 = static_cast<int>(u - row * G.segs) * kTabSeg;
    t.j1 = min(t.j0 + kTabSeg, G.stride);
    return t;
}

// The pages that a step takes from and returns to the ring of group g, by one CTA
// (all of its threads): every taken page is read, into `owned`, the table and the
// slot map, ahead of any write to the ring.  Only a windowed group comes here, when
// its chunks pass through more pages than are in use (the first prompts of an idle
// service).  Out of line: other steps do not fetch it, and what they pay for the
// possibility is 0.1, 0.0 and 0.4 us at 32, 200 and 2048 sequences.  A step that
// comes here takes longer: about 12 us for 170 pages of 21,000 new tokens.
__device__ __noinline__ void ring_alone(const TabParams& P, const TabShared& S, int g, const int* len_c, const int* len_n,
                                        const int* take_off, const int* give_off, const int* tok_off, int real)
{
    const TabGroup& G = P.g[g];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int bad = 0;
    for (unsigned u = warp; u < G.units; u += kTabWarps) {
        const int s = u / G.segs, j0 = static_cast<int>(u % G.segs) * kTabSeg;
        const int c = len_c[s], n = max(len_n[s], 0);
        const int before = pages_of(c, G.shift), after = pages_of(c + n, G.shift);
        const int a = max(j0, before), b = min(min(j0 + kTabSeg, G.stride), after);
        const long long row = static_cast<long long>(s) * G.stride;
        for (int k0 = a; k0 < b; k0 += 32) {
            const int k = k0 + lane;
            int v = -1;
            if (k < b) {
                v = G.ring[ring_at(S.head[g] + take_off[s], k - before, G.ring_size)];
                G.owned[row + k] = v;
                if (v < 0 || v >= G.num_pages) {
                    v = -1;
                    bad = 1;
                }
                G.table[row + k] = v;
            }
            if (G.slots == nullptr) continue;
            // the tokens that complete the entries of 32 pages, a page at a time
            for (int i = 0; i < min(32, b - k0); ++i) {
                const long long page = __shfl_sync(0xffffffffu, v, i);
#pragma unroll
                for (int r = lane; r < kPage; r += 32) {
                    const long long off = ((((static_cast<long long>(k0) + i) * kPage + r + 1) << G.shift) - 1) - c;
                    if (off < 0 || off >= n || tok_off[s] + off >= real) continue;
                    G.slots[tok_off[s] + off] = page < 0 ? -1 : page * kPage + r;
                }
            }
        }
    }
    __syncthreads();
    for (unsigned u = warp; u < G.units; u += kTabWarps) {
        const int s = u / G.segs, j0 = static_cast<int>(u % G.segs) * kTabSeg;
        SeqLen q;
        q.c = len_c[s];
        q.done = len_n[s] < 0;
        q.n = max(len_n[s], 0);
        int lo, before, after, gone;
        seq_pages(G.shift, G.window, q, lo, before, after, gone);
        const long long row = static_cast<long long>(s) * G.stride;
        for (int k = max(j0, lo) + lane; k < min(j0 + kTabSeg, gone); k += 32) {
            const int v = G.owned[row + k];
            G.ring[ring_at(S.tail[g] + give_off[s], k - lo, G.ring_size)] = v;
            if (v < 0 || v >= G.num_pages) bad = 1;
        }
    }
    if (bad) flag(P.status, DSV4_DEV_BAD_PAGE);
}

__global__ void __launch_bounds__(kTabThreads) batch_tables_kernel(const __grid_constant__ TabParams P)
{
    extern __shared__ __align__(16) int dyn[];
    __shared__ TabShared S;
    const int nseq = P.num_seqs, ng = P.num_groups, npad = (nseq + 7) & ~7;
    int* len_c = dyn;                                      // [nseq] tokens computed
    int* len_n = len_c + npad;                             // [nseq] new ones, -1: done or refused
    int* counts = len_n + npad;                            // [2 ng][nseq] pages taken and returned by group, then
                                                           // those of the sequences before
    int* tok_off = counts + 2 * ng * npad;                 // [nseq + 1] likewise the new tokens
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool first = blockIdx.x == 0;

    if (tid == 0) S.next = 0;
    __syncthreads();
    // lengths may come from the kernel before
    asm volatile("griddepcontrol.wait;" ::: "memory");
    long long head = 0, tail = 0;                          // thread g: group g's counters, in flight meanwhile
    if (tid < ng) {
        head = P.g[tid].pool_in[0];
        tail = P.g[tid].pool_in[1];
    }

    const TabRules R(P);
    const int cap = P.max_tokens;
    if (tid < kTabCounters) {
        // ---- the sequences' lengths and counts
        for (int i0 = tid; i0 < npad; i0 += 4 * kTabCounters) {
            int c4[4], n4[4];                              // four sequences' reads in flight
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int s = i0 + i * kTabCounters;
                c4[i] = s < nseq ? P.computed[s] : 0;
                n4[i] = s < nseq ? P.fresh[s] : -1;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int s = i0 + i * kTabCounters;
                if (s >= npad) break;
                const SeqLen q = s < nseq ? seq_len(R, c4[i], n4[i]) : SeqLen{0, 0, true, 0};
                len_c[s] = q.c;
                len_n[s] = q.done ? -1 : q.n;
                tok_off[s] = min(q.n, cap + 1);
                if (first && q.bad) flag(P.status, q.bad);
                if (first && P.ctx_len && s < nseq) P.ctx_len[s] = q.done ? 0 : q.c + q.n;
                // not unrolled: a launch fetches its code
#pragma unroll 1
                for (int g = 0; g < ng; ++g) {
                    int lo, before, after, gone;
                    seq_pages(P.g[g].shift, P.g[g].window, q, lo, before, after, gone);
                    counts[2 * g * npad + s] = after - before;
                    counts[(2 * g + 1) * npad + s] = gone - lo;
                }
            }
        }
        // ---- prefix sums: warp i takes sum i; the others need not wait for the counts
        static_assert(kTabCounters == 512 && 2 * kTabGroups < kTabCounters / 32, "a warp for each sum");
        if (warp > 2 * ng) {
            __threadfence_block();
            asm volatile("bar.arrive 1, 512;" ::: "memory");
        } else {
            asm volatile("bar.sync 1, 512;" ::: "memory");
            const bool tokens = warp == 2 * ng;
            const int total =
                warp_prefix(tokens ? tok_off : counts + warp * npad, npad, tokens ? cap + 1 : INT_MAX, lane);
            if (lane == 0) {
                S.total[warp] = total;
                if (tokens) tok_off[nseq] = total;         // npad = nseq: behind the sums; else in their padding
            }
        }
    }

    // ---- the tables' old entries: one warp per unit, 512 entries at a time, all
    // their reads ahead of any write.  New entries are left to who knows their pages.
    while (true) {
        unsigned i = 0;
        if (lane == 0) i = atomicAdd(&S.next, 1u);
        const unsigned u = __shfl_sync(0xffffffffu, i, 0) * gridDim.x + blockIdx.x;
        if (u >= P.units) break;
        const TabUnit t = table_unit(P, u);
        const TabGroup& G = P.g[t.g];
        const SeqLen q = seq_len(R, P.computed[t.s], P.fresh[t.s]);
        const int before = q.done ? 0 : pages_of(q.c, G.shift), lo = first_live(q.c, G.window);
        const int after = q.done ? 0 : pages_of(q.c + q.n, G.shift);
        const int* owned = G.owned + static_cast<long long>(t.s) * G.stride;
        int* table = G.table + static_cast<long long>(t.s) * G.stride;
        int bad = 0;
        // (one comparison: negative ids are large ones)
        auto known = [&](int v) {
            if (static_cast<unsigned>(v) < static_cast<unsigned>(G.num_pages)) return v;
            bad = 1;
            return -1;
        };
        // 16 bytes a lane; `fresh`: the row has new entries
        auto by_chunks = [&](auto fresh) {
            for (int j = t.j0; j < t.j1; j += 512) {
                int4 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = j + 128 * i + 4 * lane;
                    v[i] = make_int4(-1, -1, -1, -1);
                    if (k < t.j1 && k + 3 >= lo && k < before) v[i] = *reinterpret_cast<const int4*>(owned + k);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k0 = j + 128 * i, k = k0 + 4 * lane;
                    // most of a row is behind its sequence's end or ahead of its window
                    if (k0 < before && k0 + 128 > lo) {
                        v[i].x = k >= lo && k < before ? known(v[i].x) : -1;
                        v[i].y = k + 1 >= lo && k + 1 < before ? known(v[i].y) : -1;
                        v[i].z = k + 2 >= lo && k + 2 < before ? known(v[i].z) : -1;
                        v[i].w = k + 3 >= lo && k + 3 < before ? known(v[i].w) : -1;
                    }
                    if (k < t.j1 && (!fresh.value || k + 3 < before || k >= after)) *reinterpret_cast<int4*>(table + k) = v[i];
                }
            }
        };
        // Each of the two loops once more for rows with new entries, not once for
        // both: the conditions cost 0.1 to 0.3 us at 32 and 2048 sequences.
        if (G.vec && after == before) {
            by_chunks(std::false_type{});
        } else if (G.vec) {
            by_chunks(std::true_type{});
            // what shares a chunk with the first or the last new entry
            const int k = ((lane < 4 ? before : after) & ~3) + (lane & 3);
            if (lane < 8 && k >= t.j0 && k < t.j1 && (lane < 4 ? k < before : k >= after))
                table[k] = k >= lo && k < before ? known(owned[k]) : -1;
        } else if (after == before) {
            for (int j = t.j0 + lane; j < t.j1; j += 32) table[j] = j >= lo && j < before ? known(owned[j]) : -1;
        } else {
#pragma unroll 1
            for (int j = t.j0 + lane; j < t.j1; j += 128) {
                int v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = j + 32 * i;
                    v[i] = k >= lo && k < min(t.j1, before) ? owned[k] : -1;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = j + 32 * i;
                    if (k < t.j1 && (k < before || k >= after)) table[k] = k >= lo && k < before ? known(v[i]) : -1;
                }
            }
        }
        if (bad) flag(P.status, DSV4_DEV_BAD_PAGE);
    }

    __syncthreads();
    // ---- the pools: a group that cannot take or return all its pages does neither.
    // The places of the pages that it takes are free for those that it returns.
    if (warp == 0) {
        bool over = false;
        if (lane < ng) {
            const TabGroup& G = P.g[lane];
            const long long taken = S.total[2 * lane], freed = S.total[2 * lane + 1];
            const long long avail = tail - head, size = G.ring_size;
            const bool ok = head >= 0 && tail >= head && avail <= size && taken <= avail &&
                            avail - taken + freed <= size && tail <= LLONG_MAX - freed;
            over = ok && avail + freed > size;
            S.ok[lane] = !ok ? kRefused : (over ? kAlone : kShared);
            // an empty ring is never read or written: nothing to take, nothing to return
            S.head[lane] = ok && G.ring_size ? ring_base(head, G.ring_size) : 0;
            S.tail[lane] = ok && G.ring_size ? ring_base(tail, G.ring_size) : 0;
            if (first) {
                G.pool_out[0] = ok ? head + taken : head;
                G.pool_out[1] = ok ? tail + freed : tail;
                if (!ok) flag(P.status, DSV4_DEV_BAD_PAGE);
            }
        }
        const unsigned alone = __ballot_sync(0xffffffffu, over);
        if (lane == 0) S.alone = alone;
    }
    if (first && tid == 0 && S.total[2 * ng] > cap) flag(P.status, DSV4_DEV_BAD_INDEX);
    __syncthreads();

    const unsigned alone = S.alone;
    // ---- token rows, 32 a warp, from the last warps on (the first ones have more
    // table rows to go on with)
    const int real = min(tok_off[nseq], cap);              // offsets past max_tokens only drop tokens
    for (int t = ((kTabWarps - 1 - warp) * gridDim.x + blockIdx.x) * 32 + lane; t < cap; t += gridDim.x * kTabThreads) {
        int s = -1, p = -1, c = 0;
        if (t < real) {
            int a = 0, b = nseq - 1;               // the last sequence whose offset is <= t
            while (a < b) {
                const int m = (a + b + 1) >> 1;
                if (tok_off[m] <= t) a = m;
                else b = m - 1;
            }
            s = a;
            c = len_c[s];
            p = c + (t - tok_off[s]);
        }
        int page[kTabGroups];                      // -2: the token completes no entry; -3: ring_alone's
#pragma unroll
        for (int g = 0; g < kTabGroups; ++g) {
            page[g] = -2;
            if (g >= ng || P.g[g].slots == nullptr || s < 0) continue;
            const TabGroup& G = P.g[g];
            if ((p + 1) & ((1 << G.shift) - 1)) continue;
            const int j = (p >> G.shift) / kPage, before = pages_of(c, G.shift);
            page[g] = -1;
            if (j < before) page[g] = G.owned[static_cast<long long>(s) * G.stride + j];
            else if (S.ok[g] == kAlone) page[g] = -3;
            else if (S.ok[g] == kShared)
                page[g] = G.ring[ring_at(S.head[g] + counts[2 * g * npad + s], j - before, G.ring_size)];
        }
        if (P.positions) P.positions[t] = p;
        if (P.seqs) P.seqs[t] = s;
        if (P.row_ctx) P.row_ctx[t] = p + 1;
#pragma unroll
        for (int g = 0; g < kTabGroups; ++g) {
            if (g >= ng || P.g[g].slots == nullptr) continue;
            const TabGroup& G = P.g[g];
            if (page[g] == -3) continue;
            long long slot = -1;
            if (page[g] >= 0 && page[g] < G.num_pages)
                slot = static_cast<long long>(page[g]) * kPage + (p >> G.shift) % kPage;
            else if (page[g] != -2) flag(P.status, DSV4_DEV_BAD_PAGE);
            G.slots[t] = slot;
        }
    }

    // ---- the pages that the step takes and returns
    for (unsigned u = warp * gridDim.x + blockIdx.x; u < P.units; u += gridDim.x * kTabWarps) {
        const TabUnit t = table_unit(P, u);
        const TabGroup& G = P.g[t.g];
        SeqLen q;
        q.c = len_c[t.s];
        q.done = len_n[t.s] < 0;
        q.n = max(len_n[t.s], 0);
        int lo, before, after, gone;
        seq_pages(G.shift, G.window, q, lo, before, after, gone);
        if (S.ok[t.g] == kAlone) continue;
        int* owned = G.owned + static_cast<long long>(t.s) * G.stride;
        int* table = G.table + static_cast<long long>(t.s) * G.stride;
        if (S.ok[t.g] == kRefused) {
            // the new entries are unmapped, also for a step that goes on from here: what
            // `owned` has there may be another sequence's by now
#pragma unroll 1
            for (int j = max(t.j0, before) + lane; j < min(t.j1, after); j += 32) owned[j] = table[j] = -1;
            if (after > before && lane == 0 && t.j0 == 0) flag(P.status, DSV4_DEV_BAD_PAGE);
            continue;
        }
        const unsigned take = S.head[t.g] + counts[2 * t.g * npad + t.s],
                       give = S.tail[t.g] + counts[(2 * t.g + 1) * npad + t.s];
        int bad = 0;
        // entries [a, b) of the unit that are taken or returned, four reads ahead
        const int a = max(t.j0, gone > lo ? min(lo, before) : before);
        const int b = min(t.j1, max(after > before ? after : 0, gone > lo ? gone : 0));
        for (int j = a + lane; j < b; j += 128) {
            int v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = j + 32 * i;
                v[i] = -1;
                if (k >= b || (k < before && (k < lo || k >= gone))) continue;
                v[i] = k < before ? owned[k] : G.ring[ring_at(take, k - before, G.ring_size)];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = j + 32 * i;
                if (k >= b || (k < before && (k < lo || k >= gone))) continue;
                if (k < gone) G.ring[ring_at(give, k - lo, G.ring_size)] = v[i];
                // all of these are at lo or behind: a returned one is checked as well
                const bool live = static_cast<unsigned>(v[i]) < static_cast<unsigned>(G.num_pages);
                if (!live) bad = 1;
                if (k < before) continue;
                owned[k] = v[i];
                table[k] = live ? v[i] : -1;
            }
        }
        if (bad) flag(P.status, DSV4_DEV_BAD_PAGE);
    }
    // ---- rings that one CTA takes from and returns to
#pragma unroll 1
    for (int g = 0; alone >> g; ++g)
        if ((alone >> g & 1) && blockIdx.x == gridDim.x - 1 - g % gridDim.x)
            ring_alone(P, S, g, len_c, len_n, counts + 2 * g * npad, counts + (2 * g + 1) * npad, tok_off, real);
    if (first && P.offsets)
        for (int s = tid; s <= nseq; s += kTabThreads) P.offsets[s] = min(tok_off[s], cap);
    // the kernels behind this one may read the tables before their own wait
    // on it (they start once every CTA has ended)
    __threadfence();
}

}  // namespace dsv4

using namespace dsv4;

extern "C" dsv4_status dsv4_build_batch_tables(const dsv4_batch_tables_args* a, dsv4_stream_t stream)
{
    if (a == nullptr || a->num_seqs < 0 || a->max_tokens < 0 || a->num_groups < 0) return DSV4_ERR_INVALID;
    if (a->num_groups < 1 || a->num_groups > DSV4_MAX_TABLE_GROUPS || a->num_seqs > kTabMaxSeqs ||
        a->max_tokens > (1 << 24))
        return DSV4_ERR_UNSUPPORTED;
    if (a->num_seqs > 0 && (!a->computed_dev || !a->new_dev)) return DSV4_ERR_INVALID;
    auto mis = [](const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; };
    if (mis(a->computed_dev, 4) || mis(a->new_dev, 4) || mis(a->offsets_dev, 4) || mis(a->ctx_len_dev, 4) ||
        mis(a->positions_dev, 4) || mis(a->seqs_dev, 4) || mis(a->row_ctx_dev, 4) || mis(a->status_dev, 4))
        return DSV4_ERR_SHAPE;
    TabParams P = {};
    P.num_seqs = a->num_seqs;
    P.max_tokens = a->max_tokens;
    P.num_groups = a->num_groups;
    P.computed = a->computed_dev;
    P.fresh = a->new_dev;
    P.offsets = a->offsets_dev;
    P.ctx_len = a->ctx_len_dev;
    P.positions = a->positions_dev;
    P.seqs = a->seqs_dev;
    P.row_ctx = a->row_ctx_dev;
    P.status = a->status_dev;
    // what is written while it is read elsewhere has to be a buffer of its own
    const void* used[7 + 6 * DSV4_MAX_TABLE_GROUPS];
    int n_used = 0;
    auto own = [&](const void* p) {
        if (p == nullptr) return true;
        for (int k = 0; k < n_used; ++k)
            if (used[k] == p) return false;
        used[n_used++] = p;
        return true;
    };
    const bool rows = a->max_tokens > 0;
    if (a->num_seqs > 0) {
        used[n_used++] = a->computed_dev;                    // read only: both may be the same
        used[n_used++] = a->new_dev;
    }
    if (!own(a->offsets_dev) || (a->num_seqs > 0 && !own(a->ctx_len_dev)) ||
        (rows && (!own(a->positions_dev) || !own(a->seqs_dev) || !own(a->row_ctx_dev))))
        return DSV4_ERR_INVALID;
    for (int i = 0; i < a->num_groups; ++i) {
        const dsv4_table_group& g = a->groups[i];
        if (g.num_pages < 0 || g.stride < 0 || g.ring_size < 0 || g.window < 0) return DSV4_ERR_INVALID;
        if (g.ratio != 1 && g.ratio != 4 && g.ratio != 128) return DSV4_ERR_UNSUPPORTED;
        if (g.window > 0 && g.ratio != 1) return DSV4_ERR_UNSUPPORTED;
        if (!g.pool_in_dev || !g.pool_out_dev) return DSV4_ERR_INVALID;
        if (a->num_seqs > 0 && g.stride > 0 && (!g.owned_dev || !g.table_dev)) return DSV4_ERR_INVALID;
        if (g.ring_size > 0 && !g.ring_dev) return DSV4_ERR_INVALID;
        // the last unit's steps past its row stay below 2^31
        if (static_cast<long long>(a->num_seqs) * g.stride > INT_MAX - 4 * kTabSeg) return DSV4_ERR_UNSUPPORTED;
        if (mis(g.owned_dev, 4) || mis(g.table_dev, 4) || mis(g.ring_dev, 4) || mis(g.pool_in_dev, 8) ||
            mis(g.pool_out_dev, 8) || mis(g.slots_dev, 8))
            return DSV4_ERR_SHAPE;
        if (!own(g.owned_dev) || !own(g.table_dev) || !own(g.ring_dev) || !own(g.pool_in_dev) || !own(g.pool_out_dev) ||
            (rows && !own(g.slots_dev)))
            return DSV4_ERR_INVALID;
        TabGroup& G = P.g[i];
        G.shift = g.ratio == 1 ? 0 : (g.ratio == 4 ? 2 : 7);
        G.window = g.window;
        G.num_pages = g.num_pages;
        G.stride = g.stride;
        G.segs = (g.stride + kTabSeg - 1) / kTabSeg;
        G.units = static_cast<unsigned>(G.segs) * a->num_seqs;
        G.vec = !mis(g.table_dev, 16) && !mis(g.owned_dev, 16) && g.stride % 4 == 0;
        G.owned = g.owned_dev;
        G.table = g.table_dev;
        G.ring = g.ring_dev;
        G.ring_size = static_cast<unsigned>(g.ring_size);
        G.pool_in = g.pool_in_dev;
        G.pool_out = g.pool_out_dev;
        G.slots = g.slots_dev;
        P.units += G.units;
    }
    const size_t smem = (static_cast<size_t>((a->num_seqs + 7) & ~7) * (3 + 2 * a->num_groups) + 1) * sizeof(int);
    static PerDeviceOnce once;
    if (!once.run([] {
            return cudaFuncSetAttribute(batch_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (kTabMaxSeqs * (3 + 2 * kTabGroups) + 1) * sizeof(int)) == cudaSuccess;
        })) {
        (void)cudaGetLastError();
        return DSV4_ERR_CUDA;
    }
    // a unit for each warp that does not count: with two, 32 sequences took 5.2
    // us (4.7 with one), 200 sequences 7.4 (5.6)
    constexpr int other_warps = kTabWarps - kTabCounters / 32;
    const long long by_units = (static_cast<long long>(P.units) + other_warps - 1) / other_warps;
    const long long by_tokens = (a->max_tokens + kTabThreads - 1) / kTabThreads;
    const long long most = sm_count();
    long long ctas = by_units + by_tokens;
    ctas = ctas < 1 ? 1 : (ctas > most ? most : ctas);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(kTabThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, batch_tables_kernel, P) == cudaSuccess) return DSV4_OK;
    (void)cudaGetLastError();
    return DSV4_ERR_CUDA;
}

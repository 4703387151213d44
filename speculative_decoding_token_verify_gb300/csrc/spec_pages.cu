// spec_pages.cu -- the upkeep of a cache held in pages: rows resized, forked and
// compacted, and the walk down a tree of drafts.
//
// The tables are small (megabytes at most) and every decision is a count: which
// entries are dropped, how many pages are wanted before this one, which pages are
// free before that one. One cluster of CTAs makes them in one launch, with a
// cluster barrier between the phases. Each warp owns a contiguous stretch of entries (and later of pages),
// so that a rank is a sum of ballots: over the warp's own stretch, the CTA's earlier
// warps, and the cluster's earlier CTAs. Reference counts change by integer
// atomics, whose order cannot be seen. What bounds them is the chain of five phases with four barriers
// between: 5.5 us for 4 rows of 64 entries, 23 for 512 of 1024; 256 beams of 257 entries forked 13 us with the
// copies (in a graph).
#include <climits>
#include <mutex>

#include "spec_rows.cuh"

namespace sr {

constexpr int NTP = 1024;
constexpr int NWP = NTP / 32;
constexpr int kMaxPagesCluster = 16;
constexpr int U = 4;   // groups of 32 entries whose loads are in flight together (8, 16: more code, and slower)

struct PagesArgs {
    const int32_t *table, *refs, *lengths, *parent;
    int32_t *out_table, *out_refs, *out_lengths, *copies;
    int32_t *list, *claim;   // workspace: free pages in order; the first row that wants a page
    int32_t *status;
    int B, W, N, M, P, page;
};

struct PagesShared {
    int warp[2][NWP];         // two counts per warp
    int cta[2][16];           // and per CTA of the cluster
};

__device__ __forceinline__ void cluster_sync_all(int C) {
    if (C > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
}

// From every warp's counts, in the K slots from `slot` on: how many come before this warp in
// the cluster, and in all. Ends with a cluster barrier, before which the caller's writes
// also count.
template <int K>
__device__ __forceinline__ void ranks(PagesShared &sh, int slot, const int (&mine)[K], int C, int rank, int (&before)[K], int (&total)[K]) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    static_assert(NWP == 32, "a lane per warp");
    if (lane == 0)
        for (int k = 0; k < K; ++k) sh.warp[slot + k][warp] = mine[k];
    __syncthreads();
    for (int k = 0; k < K; ++k) {
        const int n = sh.warp[slot + k][lane];
        before[k] = __reduce_add_sync(kFull, lane < warp ? n : 0);
        if (warp == 0) {
            const int sum = __reduce_add_sync(kFull, n);
            if (C == 1) sh.cta[slot + k][0] = sum;
            else if (lane < C) peer_store_u32(peer(&sh.cta[slot + k][rank], lane), (uint32_t)sum);
        }
    }
    cluster_sync_all(C);
    for (int k = 0; k < K; ++k) {
        const int n = lane < C ? sh.cta[slot + k][lane] : 0;
        before[k] += __reduce_add_sync(kFull, lane < rank ? n : 0);
        total[k] = __reduce_add_sync(kFull, n);
    }
}

// A warp's stretch of n entries, in whole groups of 32 V (of at least U, so that few entries
// are not spread thin).
struct Stretch {
    long long lo, hi;
    __device__ __forceinline__ Stretch(long long n, int warp, int warps, int V = 1) {
        const long long size = 32 * V, groups = (n + size - 1) / size;
        long long per = (groups + warps - 1) / warps;
        if (per < U && per > 1) per = min((long long)U, groups);
        lo = min(n, warp * per * size);
        hi = min(n, (warp + 1) * per * size);
    }
};

// V entries from i on, those past hi as `none`
template <int V>
__device__ __forceinline__ void load_entries(const int32_t *p, long long i, long long hi, int none, int (&e)[V]) {
    if (V == 4 && i + 3 < hi) {
        const int4 v = __ldcg(reinterpret_cast<const int4 *>(p + i));
        e[0] = v.x, e[V / 3] = v.y, e[V / 2] = v.z, e[V - 1] = v.w;
        return;
    }
#pragma unroll
    for (int k = 0; k < V; ++k) e[k] = i + k < hi ? __ldcg(p + i + k) : none;
}

__device__ __forceinline__ int lanes_below(unsigned ballot) {
    return __popc(ballot & ((1u << (threadIdx.x & 31)) - 1));
}

// Whether V pages from i on are free. (A page that a row has claimed is kept by it where nothing
// else names it.)
template <int V, bool kClaims>
__device__ __forceinline__ unsigned free_of(const PagesArgs &a, long long i, long long hi) {
    int refs[V], claim[V];
    load_entries<V>(a.out_refs, i, hi, -1, refs);
    if (kClaims) load_entries<V>(a.claim, i, hi, 0, claim);
    unsigned free = 0;
#pragma unroll
    for (int k = 0; k < V; ++k) free |= (unsigned)(refs[k] == 0 && (!kClaims || claim[k] == INT_MAX)) << k;
    return free;
}
template <int V, bool kClaims>
__device__ __forceinline__ int count_free(const PagesArgs &a, const Stretch &s) {
    int count = 0;
#pragma unroll 4
    for (long long i = s.lo + (threadIdx.x & 31) * V; i < s.hi; i += 32 * V) count += __popc(free_of<V, kClaims>(a, i, s.hi));
    return __reduce_add_sync(kFull, count);
}
// how many of the lower lanes' bits are set, and of all lanes'
template <int V>
__device__ __forceinline__ int bits_below(unsigned bits, int &all) {
    if (V == 1) {
        const unsigned ballot = __ballot_sync(kFull, bits);
        all = __popc(ballot);
        return lanes_below(ballot);
    }
    int upto = __popc(bits);
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int v = __shfl_up_sync(kFull, upto, o);
        if ((threadIdx.x & 31) >= o) upto += v;
    }
    all = __shfl_sync(kFull, upto, 31);
    return upto - __popc(bits);
}
// list[k] = the k-th lowest free page, for k < wanted; `before` free ones lie in front of the stretch
template <int V, bool kClaims>
__device__ __forceinline__ void list_free(const PagesArgs &a, const Stretch &s, int before, int wanted) {
    const int off = (threadIdx.x & 31) * V;
    for (long long i = s.lo + off; i < s.hi + off && before < wanted; i += 32 * V) {
        const unsigned free = free_of<V, kClaims>(a, i, s.hi);
        int all, k = before + bits_below<V>(free, all);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (free >> v & 1) {
                if (k < wanted) a.list[k] = (int)i + v;
                ++k;
            }
        before += all;
    }
}

// a length within [0, M page] (M page < 2^31)
__device__ __forceinline__ int fit(const PagesArgs &a, int length) {
    const int most = a.M * a.page;
    if (length >= 0 && length <= most) return length;
    raise_status(a.status, SPEC_ERR_BAD_LENGTH);
    return length < 0 ? 0 : most;
}
// entry i of a table as (row, place), moved on by 32 without a division most of the time
struct Place {
    int r, m;
    __device__ __forceinline__ Place(long long i, int M) : r((int)(i / max(M, 1))), m((int)(i - (long long)r * M)) {}
    __device__ __forceinline__ void next(int M, int by = 32) {
        m += by;
        if (m >= M) {
            const int q = m / M;
            r += q;
            m -= q * M;
        }
    }
};

// Rows of exactly the pages that their lengths ask for. V = 4: a lane takes four entries
// together, of one row (M is a multiple of 4). A 512 x 1024 table over 315,000 pages takes 23 us
// (one by one 26), twenty times its bytes: 16 SMs, which read the table twice and the counts three times, and
// wait for memory and for the cluster between the phases. Tables that one CTA handles take their entries
// one by one (4 x 64: by fours 1 us more).
template <int V>
__global__ void __launch_bounds__(NTP, 1) resize_kernel(PagesArgs a, int C) {
    __shared__ PagesShared sh;
    const int rank = C > 1 ? blockIdx.x : 0, lane = threadIdx.x & 31, gw = rank * NWP + (threadIdx.x >> 5);
    const Stretch pages(a.P, gw, C * NWP, V), s((long long)a.B * a.W * a.M, gw, C * NWP, V);
    if (a.out_refs != a.refs) {
#pragma unroll 4
        for (long long i = pages.lo + lane * V; i < pages.hi; i += 32 * V) {
            int refs[V];
            load_entries<V>(a.refs, i, pages.hi, 0, refs);
            if (V == 4 && i + 3 < pages.hi) {
                *reinterpret_cast<int4 *>(a.out_refs + i) = make_int4(refs[0], refs[V / 3], refs[V / 2], refs[V - 1]);
            } else {
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (i + k < pages.hi) a.out_refs[i + k] = refs[k];
            }
        }
    }
    cluster_sync_all(C);   // (from here on every CTA of the cluster has shared memory to write to)
    const int most = a.M * a.page;
    int wants = 0, bad = 0;
    {
        Place at(s.lo + lane * V, a.M);
        for (long long i = s.lo + lane * V; i < s.hi; i += 32 * V * U) {
            int e[U][V], len[U], from[U];
#pragma unroll
            for (int u = 0; u < U; ++u, at.next(a.M, 32 * V)) {
                from[u] = at.m * a.page;
                load_entries<V>(a.table, i + 32 * V * u, s.hi, -1, e[u]);
                len[u] = i + 32 * V * u < s.hi ? a.lengths[at.r] : 0;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if ((unsigned)len[u] > (unsigned)most) bad = SPEC_ERR_BAD_LENGTH;
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const bool has = (unsigned)e[u][k] < (unsigned)a.P, in = from[u] + k * a.page < len[u];   // in: m < ceil(len / page)
                    if (!has && e[u][k] != -1) bad = max(bad, SPEC_ERR_BAD_PAGE);
                    if (has && !in) atomicAdd(a.out_refs + e[u][k], -1);
                    wants += !has && in;
                }
            }
        }
        if (bad) raise_status(a.status, bad);
        wants = __reduce_add_sync(kFull, wants);
    }
    int ahead[1], all_wants[1];
    ranks<1>(sh, 0, {wants}, C, rank, ahead, all_wants);
    const int wanted = all_wants[0];
    int before = ahead[0], nfree = 0;
    if (wanted > 0) {   // (the same for the whole cluster)
        int all_free[1];
        ranks<1>(sh, 1, {count_free<V, false>(a, pages)}, C, rank, ahead, all_free);
        nfree = all_free[0];
        list_free<V, false>(a, pages, ahead[0], wanted);
        cluster_sync_all(C);
    }
    if (nfree < wanted && rank == 0 && threadIdx.x == 0) raise_status(a.status, SPEC_ERR_NO_PAGES);
    {
        Place at(s.lo + lane * V, a.M);
        for (long long i = s.lo + lane * V; i < s.hi + lane * V; i += 32 * V * U) {
            int e[U][V], len[U], from[U];
#pragma unroll
            for (int u = 0; u < U; ++u, at.next(a.M, 32 * V)) {
                from[u] = at.m * a.page;
                load_entries<V>(a.table, i + 32 * V * u, s.hi, -1, e[u]);
                len[u] = i + 32 * V * u < s.hi ? a.lengths[at.r] : 0;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const long long at_i = i + 32 * V * u;
                unsigned want = 0;
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const bool has = (unsigned)e[u][k] < (unsigned)a.P, in = from[u] + k * a.page < len[u] && at_i + k < s.hi;
                    if (!has || !in) e[u][k] = -1;
                    want |= (unsigned)(!has && in) << k;
                }
                if (__any_sync(kFull, want)) {   // (few groups want any)
                    int all, rank_of = before + bits_below<V>(want, all);
#pragma unroll
                    for (int k = 0; k < V; ++k)
                        if (want >> k & 1) {
                            if (rank_of < nfree) {
                                e[u][k] = __ldcg(a.list + rank_of);
                                a.out_refs[e[u][k]] = 1;
                            }
                            ++rank_of;
                        }
                    before += all;
                }
                if (V == 4 && at_i + 3 < s.hi) {
                    *reinterpret_cast<int4 *>(a.out_table + at_i) = make_int4(e[u][0], e[u][V / 3], e[u][V / 2], e[u][V - 1]);
                } else {
#pragma unroll
                    for (int k = 0; k < V; ++k)
                        if (at_i + k < s.hi) a.out_table[at_i + k] = e[u][k];
                }
            }
        }
    }
}

// What new row (b, n) continues: its old row's index (-1: none) and length.
__device__ __forceinline__ int source_row(const PagesArgs &a, int r, int b, int n, int &length) {
    int w = a.parent[r];
    if (w < -1 || w >= a.W) {
        raise_status(a.status, SPEC_ERR_BAD_PARENT);
        w = -1;
    }
    if (w < 0) w = n < a.W ? n : -1;
    length = 0;
    if (w < 0) return -1;
    const int src = b * a.W + w;
    length = fit(a, a.lengths[src]);
    return src;
}

__device__ __forceinline__ int entry(const PagesArgs &a, int row, int m) {
    const int e = a.table[(long long)row * a.M + m];
    if (e >= 0 && e < a.P) return e;
    if (e != -1) raise_status(a.status, SPEC_ERR_BAD_PAGE);
    return -1;
}

// Tables in the order of the surviving beams.
__global__ void __launch_bounds__(NTP, 1) fork_kernel(PagesArgs a, int C) {
    __shared__ PagesShared sh;
    const int rank = C > 1 ? blockIdx.x : 0, lane = threadIdx.x & 31, gw = rank * NWP + (threadIdx.x >> 5);
    for (int i = rank * NTP + threadIdx.x; i < a.P; i += C * NTP) a.claim[i] = INT_MAX;
    if (a.out_refs != a.refs) {
#pragma unroll 8
        for (int i = rank * NTP + threadIdx.x; i < a.P; i += C * NTP) a.out_refs[i] = __ldg(a.refs + i);
    }
    cluster_sync_all(C);
    // full pages: the old row's entries lose a reference, the new row's gain one
    {
        const Stretch s((long long)a.B * a.N * a.M, gw, C * NWP);
        Place at(s.lo + lane, a.M);
        int row = -1, length = 0, bad = 0;
        const int32_t *src = nullptr, *own = nullptr;   // the old rows' tables
        for (long long i = s.lo + lane; i < s.hi; i += 32 * U) {
            int e[U], old[U], of[U];
            unsigned in = 0, last = 0;
#pragma unroll
            for (int u = 0; u < U; ++u, at.next(a.M)) {
                e[u] = old[u] = -1;
                if (i + 32 * u < s.hi) {
                    if (at.r != row) {
                        row = at.r;
                        const int b = row / a.N, n = row - b * a.N;
                        src = a.table + (long long)source_row(a, row, b, n, length) * a.M;   // (not read where length is 0)
                        own = n < a.W ? a.table + (long long)(b * a.W + n) * a.M : nullptr;
                    }
                    const int left = length - at.m * a.page;   // tokens from this entry on
                    if (left > 0) {
                        e[u] = src[at.m];
                        in |= 1u << u;
                        last |= (unsigned)(left < a.page) << u;
                    }
                    if (own) old[u] = own[at.m];
                }
                of[u] = row;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (i + 32 * u >= s.hi) continue;
                if ((unsigned)e[u] >= (unsigned)a.P) {
                    if (in >> u & 1) bad = SPEC_ERR_BAD_PAGE;
                    e[u] = -1;
                }
                if ((unsigned)old[u] >= (unsigned)a.P) {
                    if (old[u] != -1) bad = SPEC_ERR_BAD_PAGE;
                    old[u] = -1;
                }
                if (last >> u & 1) {
                    if (e[u] >= 0) atomicMin(a.claim + e[u], of[u]);
                    e[u] = -1;   // (decided below)
                }
                if (old[u] != e[u]) {
                    if (old[u] >= 0) atomicAdd(a.out_refs + old[u], -1);
                    if (e[u] >= 0) atomicAdd(a.out_refs + e[u], 1);
                }
                a.out_table[i + 32 * u] = e[u];
            }
        }
        if (bad) raise_status(a.status, bad);
    }
    if (a.N < a.W) {   // old rows without a new one in their place
        const int gone = a.W - a.N;
        const Stretch s((long long)a.B * gone * a.M, gw, C * NWP);
        Place at(s.lo + lane, a.M);
        for (long long i = s.lo + lane; i < s.hi; i += 32, at.next(a.M)) {
            const int b = at.r / gone, old = entry(a, b * a.W + a.N + at.r - b * gone, at.m);
            if (old >= 0) atomicAdd(a.out_refs + old, -1);
        }
    }
    cluster_sync_all(C);
    // pages that are not full: kept by the first row that wants them, or copied
    const Stretch s((long long)a.B * a.N, gw, C * NWP), pages(a.P, gw, C * NWP);
    int wants = 0;
    for (long long r = s.lo + lane; r < s.hi + lane; r += 32) {
        bool want = false;
        if (r < s.hi) {
            int length;
            const int b = (int)r / a.N, src = source_row(a, (int)r, b, (int)r - b * a.N, length);
            const int full = length / a.page, part = length - full * a.page;
            const int last = src >= 0 && part ? entry(a, src, full) : -1;
            if (last >= 0) {
                want = __ldcg(a.claim + last) != (int)r || __ldcg(a.out_refs + last) != 0;
                if (!want) {
                    a.out_refs[last] = 1;   // (only the first row reads this count)
                    a.out_table[r * a.M + full] = last;
                }
            }
            a.out_lengths[r] = length;
            int32_t *c = a.copies + r * 4;
            c[0] = want ? last : -1;
            c[1] = -1;
            c[2] = want ? part : 0;
            c[3] = 0;
        }
        wants += __popc(__ballot_sync(kFull, want));
    }
    // free pages are counted beside it: those that rows keep are claimed
    int ahead[2], all[2];
    ranks<2>(sh, 0, {wants, count_free<1, true>(a, pages)}, C, rank, ahead, all);
    int before = ahead[0];
    const int wanted = all[0], nfree = all[1];
    if (wanted == 0) return;   // (the same for the whole cluster)
    list_free<1, true>(a, pages, ahead[1], wanted);
    cluster_sync_all(C);
    if (nfree < wanted && rank == 0 && threadIdx.x == 0) raise_status(a.status, SPEC_ERR_NO_PAGES);
    for (long long r = s.lo + lane; r < s.hi + lane; r += 32) {
        int32_t *c = a.copies + r * 4;
        const bool want = r < s.hi && c[0] >= 0;   // (written by this thread)
        const unsigned ballot = __ballot_sync(kFull, want);
        const int k = before + lanes_below(ballot);
        if (want && k < nfree) {
            const int e = __ldcg(a.list + k);
            const int length = a.out_lengths[r];   // (written by this thread, as c)
            c[1] = e;
            a.out_refs[e] = 1;
            a.out_table[r * a.M + length / a.page] = e;
        }
        before += __popc(ballot);
    }
}

// ---- bytes of pages ------------------------------------------------------------------

struct CacheArgs {
    char *cache;
    const int32_t *copies, *table, *lengths, *path;
    int32_t *out_lengths, *status;
    long long unit, ss[3];
    int O, P, H, page, B, N, M;
    long long vecs;   // vectors a segment (copy) or a unit (compact)
};

constexpr int NTC = 256;

// copies[y]: the first slots of a page, CP vectors a thread (4: 16 KB of a page in one CTA's loads)
template <typename Vec, int CP>
__global__ void __launch_bounds__(NTC) copy_kernel(CacheArgs a, int count) {
    asm volatile("griddepcontrol.wait;" ::: "memory");   // (launched while the stream's last kernel, the fork, ends)
    for (int c = blockIdx.y; c < count; c += gridDim.y) {
        const int src = a.copies[c * 4LL], dst = a.copies[c * 4LL + 1], slots = min(a.copies[c * 4LL + 2], a.page);
        if (src < 0 || src >= a.P || dst < 0 || dst >= a.P || slots <= 0) continue;
        const long long n = slots * a.unit / (long long)sizeof(Vec);
        for (long long oh = blockIdx.z; oh < (long long)a.O * a.H; oh += gridDim.z) {
            const long long o = oh / a.H, off = o * a.ss[0] + (oh - o * a.H) * a.ss[2];
            const Vec *from = reinterpret_cast<const Vec *>(a.cache + off + src * a.ss[1]);
            Vec *to = reinterpret_cast<Vec *>(a.cache + off + dst * a.ss[1]);
            for (long long i0 = (long long)blockIdx.x * NTC * CP + threadIdx.x; i0 < n; i0 += (long long)gridDim.x * NTC * CP) {
                Vec v[CP];
#pragma unroll
                for (int k = 0; k < CP; ++k)
                    if (i0 + k * NTC < n) v[k] = from[i0 + k * NTC];
#pragma unroll
                for (int k = 0; k < CP; ++k)
                    if (i0 + k * NTC < n) to[i0 + k * NTC] = v[k];
            }
        }
    }
}

// The kept nodes of row b = blockIdx.y. A thread owns one vector of a unit and
// makes its moves in order, eight loads ahead of their stores: a source path[j]
// lies behind every place i <= j that was written before it is read. 64 rows of 33 nodes,
// 64 KB a node, 67 MB in all: 14.6 us in a graph, 4.6 TB/s; about 4 us of it are the launch and the
// chain of lengths, path and table (16 loads ahead leave one CTA an SM: 28 us; 4, 6 and 12: 14.7 to 15.4).
template <typename Vec>
__global__ void __launch_bounds__(NTC) compact_kernel(CacheArgs a) {
    __shared__ long long s_src[SPEC_MAX_NODES], s_dst[SPEC_MAX_NODES];
    __shared__ int s_kept, s_moves[SPEC_MAX_NODES / 32];
    constexpr int U = 8;
    const bool lead = blockIdx.x == 0;
    for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
        const int L = a.lengths[b];
        const bool bad = L < 0 || L > (long long)a.M * a.page;
        const int32_t *path = a.path + (long long)b * a.N;
        __syncthreads();
        if (threadIdx.x == 0) s_kept = bad ? 0 : a.N;
        __syncthreads();
        if (threadIdx.x < a.N && !bad) {
            const int i = threadIdx.x, p = path[i], q = i ? path[i - 1] : -1;
            if (p <= q || p >= a.N) {   // (ends at the first -1, too)
                atomicMin(&s_kept, i);
            }
        }
        __syncthreads();
        const int kept = s_kept;
        long long so = -1, dof = 0;
        unsigned moves = 0;
        if (threadIdx.x < SPEC_MAX_NODES) {
            const int i = threadIdx.x, p = i < kept ? path[i] : i, from = L + p, to = L + i;
            if (p != i || (lead && i < kept)) {   // (nodes that keep their place need a page, too)
                const int mf = from / a.page, mt = to / a.page;
                const int pf = mf < a.M ? a.table[(long long)b * a.M + mf] : -1;
                const int pt = mt < a.M ? a.table[(long long)b * a.M + mt] : -1;
                if (pf < 0 || pf >= a.P || pt < 0 || pt >= a.P) {
                    if (lead) raise_status(a.status, SPEC_ERR_BAD_PAGE);
                } else if (p != i) {
                    so = pf * a.ss[1] + (from - mf * a.page) * a.unit;
                    dof = pt * a.ss[1] + (to - mt * a.page) * a.unit;
                }
            }
            moves = __ballot_sync(kFull, so >= 0);
            if ((threadIdx.x & 31) == 0) s_moves[threadIdx.x >> 5] = __popc(moves);
        }
        __syncthreads();
        int total = 0;
        for (int w = 0; w < SPEC_MAX_NODES / 32; ++w) {
            if (so >= 0 && w == (int)(threadIdx.x >> 5)) {
                s_src[total + lanes_below(moves)] = so;
                s_dst[total + lanes_below(moves)] = dof;
            }
            total += s_moves[w];
        }
        if (lead && threadIdx.x == 0) {
            a.out_lengths[b] = L + kept;
            if (bad) raise_status(a.status, SPEC_ERR_BAD_LENGTH);
            if (!bad && kept < a.N && path[kept] != -1) raise_status(a.status, SPEC_ERR_BAD_PATH);
        }
        __syncthreads();
        const long long columns = (long long)a.O * a.H * a.vecs;
        for (long long x = (long long)blockIdx.x * NTC + threadIdx.x; x < columns; x += (long long)gridDim.x * NTC) {
            const long long oh = x / a.vecs, o = oh / a.H;
            char *base = a.cache + o * a.ss[0] + (oh - o * a.H) * a.ss[2] + (x - oh * a.vecs) * (long long)sizeof(Vec);
            for (int i = 0; i < total; i += U) {
                Vec v[U];
#pragma unroll
                for (int k = 0; k < U; ++k)
                    if (i + k < total) v[k] = *reinterpret_cast<const Vec *>(base + s_src[i + k]);
#pragma unroll
                for (int k = 0; k < U; ++k)
                    if (i + k < total) *reinterpret_cast<Vec *>(base + s_dst[i + k]) = v[k];
            }
        }
    }
}

// ---- the walk down a tree --------------------------------------------------------------

struct AcceptArgs {
    const int32_t *tokens, *parents, *choice, *counts;
    int32_t *accepted, *out, *path, *status;
    long long ps, cb, cn;
    int B, N;
};

constexpr int kPerLane = SPEC_MAX_NODES / 32;
constexpr int NTA = 128;

// A warp per sequence; lane l holds nodes l, l + 32, ..: a step of the walk is a
// comparison and a ballot for each. 256 trees of 128 nodes 3.1 us in a graph, one of 9 2.1: a launch.
__global__ void __launch_bounds__(NTA) accept_kernel(AcceptArgs a) {
    __shared__ int32_t s_choice[NTA / 32][SPEC_MAX_NODES];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const long long b = (long long)blockIdx.x * (NTA / 32) + w;
    if (b >= a.B) return;
    const int N = a.N;
    int count = a.counts ? a.counts[b] : N;
    int bad = 0;
    if (count < 0 || count > N) {
        bad = SPEC_ERR_BAD_LENGTH;
        count = count < 0 ? 0 : N;
    }
    int tok[kPerLane], par[kPerLane];
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
        const int n = lane + 32 * k;
        tok[k] = 0;
        par[k] = -1;
        if (n < count) {
            tok[k] = a.tokens[b * N + n];
            s_choice[w][n] = a.choice[b * a.cb + n * a.cn];
            par[k] = a.parents ? a.parents[b * a.ps + n] : n - 1;
            if (par[k] < -1 || par[k] >= n) {
                bad = max(bad, SPEC_ERR_BAD_PARENT);
                par[k] = -1;
            }
        }
    }
    if (bad) raise_status(a.status, bad);
    __syncwarp();
    int cur = count > 0 ? 0 : -1, kept = 0;
    while (cur >= 0) {   // parents lie before their children: at most count steps
        const int said = s_choice[w][cur];
        if (lane == 0) {
            a.path[b * N + kept] = cur;
            a.out[b * N + kept] = said;
        }
        ++kept;
        int next = -1;
#pragma unroll
        for (int k = kPerLane - 1; k >= 0; --k) {
            const unsigned hit = __ballot_sync(kFull, par[k] == cur && tok[k] == said);
            if (hit) next = 32 * k + __ffs(hit) - 1;
        }
        cur = next;
    }
    for (int i = kept + lane; i < N; i += 32) a.path[b * N + i] = a.out[b * N + i] = -1;
    if (lane == 0) a.accepted[b] = kept ? kept - 1 : 0;
}

// ---- host ---------------------------------------------------------------------------------

static int check_pages(const spec_pages_params *p, bool fork) {
    if (!p) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "params is NULL");
    if (p->B < 0 || p->W < 0 || p->N < 0 || p->M < 0 || p->P < 0)
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "pages: B, W, N, M and P must be >= 0");
    if (p->page < 1) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "pages: page must be >= 1");
    if (!fork && p->N != p->W) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "pages_resize: N must be W");
    const int64_t rows = (int64_t)p->B * (p->W > p->N ? p->W : p->N);
    if (rows > (1 << 24) || p->P > (1 << 30) || (rows && p->M > (INT32_MAX - 65536) / rows) ||
        (int64_t)p->M * p->page > INT32_MAX)
        return spec_internal_set_error(SPEC_ERR_UNSUPPORTED, "pages: tables, pools or rows outside the supported range");
    return SPEC_OK;
}

// Small tables are one CTA's work, whose barriers cost less; all others the largest cluster's. In a
// graph, one CTA against 16: 8.6 and 10.6 us for rows of 16 x 64 entries, 14.7 and 12.6 for 64 x 128, 58 and
// 16.7 for 256 x 512 (2, 4 and 8 CTAs lie between; 8 are as fast as 16 up to there, and 16 faster beyond).
static int pages_cluster(long long ints) { return ints > 4096 ? kMaxPagesCluster : 1; }

static cudaError_t launch_pages(void (*kernel)(PagesArgs, int), bool *allowed, const PagesArgs &a, int C, cudaStream_t stream) {
    if (C > 1) {   // (clusters of more than 8 CTAs have to be allowed, once for each device)
        static std::mutex mu;
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        std::lock_guard<std::mutex> lk(mu);
        if (!allowed[dev & 63]) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
            allowed[dev & 63] = true;
        }
    }
    return launch_cluster(kernel, C, NTP, C, 0, stream, a, C);
}

static int check_cache(const spec_cache_params *p) {
    if (!p) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "params is NULL");
    if (p->O < 0 || p->P < 0 || p->H < 0 || p->page < 1)
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "cache: O, P and H must be >= 0, page >= 1");
    if (p->O > 65535 || p->H > 65535 || p->P > (1 << 30))
        return spec_internal_set_error(SPEC_ERR_UNSUPPORTED, "cache: O, P or H out of range");
    if (p->unit_bytes < 1 || p->unit_bytes > (1 << 30))
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "cache: unit_bytes must be in [1, 2^30]");
    const int64_t n[3] = {p->O, p->P, p->H};
    for (int i = 0; i < 3; ++i)
        if (p->stride[i] < 0 || (n[i] > 1 && p->stride[i] > (INT64_MAX >> 4) / n[i]))
            return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "cache: strides must be >= 0 and not too large");
    if (p->O == 0 || p->P == 0 || p->H == 0) return SPEC_OK;
    const int64_t bytes = (int64_t)p->page * p->unit_bytes;
    // segments, pages and outer entries that do not overlap: ordered by stride, each
    // axis steps over the whole extent of the smaller ones
    int order[3] = {0, 1, 2};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (p->stride[order[j]] < p->stride[order[i]]) {
                const int t = order[i];
                order[i] = order[j];
                order[j] = t;
            }
    int64_t extent = bytes;
    for (int i = 0; i < 3; ++i) {
        const int k = order[i];
        if (n[k] <= 1) continue;
        if (p->stride[k] < extent) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "cache: pages overlap");
        extent += (n[k] - 1) * p->stride[k];
    }
    return SPEC_OK;
}

static void cache_args(CacheArgs &a, const spec_cache_params *p, void *cache) {
    a.cache = static_cast<char *>(cache);
    a.unit = p->unit_bytes;
    a.O = p->O;
    a.P = p->P;
    a.H = p->H;
    a.page = p->page;
    const int n[3] = {p->O, p->P, p->H};
    for (int i = 0; i < 3; ++i) a.ss[i] = n[i] > 1 ? p->stride[i] : 0;
}

// the widest vector that every unit starts and ends on
static int vec_bytes(const CacheArgs &a) {
    const uint64_t bits = (uint64_t)(a.unit | a.ss[0] | a.ss[1] | a.ss[2]) | reinterpret_cast<uintptr_t>(a.cache);
    return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : bits % 2 == 0 ? 2 : 1;
}

template <typename Vec>
static cudaError_t launch_copy(CacheArgs &a, int count, cudaStream_t st) {
    constexpr int CP = 4;
    const long long n = (long long)a.page * a.unit / (long long)sizeof(Vec), oh = (long long)a.O * a.H;
    const long long gx = (n + NTC * CP - 1) / (NTC * CP);
    const dim3 grid((unsigned)(gx < 1024 ? gx : 1024), (unsigned)(count < 65535 ? count : 65535),
                    (unsigned)(oh < 65535 ? oh : 65535));
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(NTC);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, copy_kernel<Vec, CP>, a, count);
}

template <typename Vec>
static cudaError_t launch_compact(CacheArgs &a, cudaStream_t st) {
    a.vecs = a.unit / (long long)sizeof(Vec);
    const long long columns = (long long)a.O * a.H * a.vecs, gx = (columns + NTC - 1) / NTC;
    const dim3 grid((unsigned)(gx < 65536 ? (gx > 0 ? gx : 1) : 65536), (unsigned)(a.B < 65535 ? a.B : 65535));
    compact_kernel<Vec><<<grid, NTC, 0, st>>>(a);
    return cudaGetLastError();
}

static int done(cudaError_t e) {
    return e == cudaSuccess ? SPEC_OK : spec_internal_set_error(SPEC_ERR_CUDA, cudaGetErrorString(e));
}

}  // namespace sr

extern "C" int spec_pages_resize(const spec_pages_params *p, const int32_t *table, const int32_t *refs,
                                 const int32_t *lengths, int32_t *out_table, int32_t *out_refs, int32_t *workspace,
                                 int32_t *status, void *stream) {
    using namespace sr;
    const int rc = check_pages(p, false);
    if (rc != SPEC_OK) return rc;
    const int64_t rows = (int64_t)p->B * p->W, entries = rows * p->M;
    if (entries == 0 && p->P == 0) return spec_internal_set_error(SPEC_OK, "");
    if ((entries && (!table || !out_table || !lengths)) || (p->P && (!refs || !out_refs || !workspace)))
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "pages_resize: an argument is NULL");
    const int64_t tb = entries * 4, rb = (int64_t)p->P * 4;
    if ((out_table != table && overlap(out_table, tb, table, tb)) || (out_refs != refs && overlap(out_refs, rb, refs, rb)) ||
        overlap(out_table, tb, out_refs, rb) || overlap(out_table, tb, refs, rb) || overlap(out_table, tb, lengths, rows * 4) ||
        overlap(out_refs, rb, table, tb) || overlap(out_refs, rb, lengths, rows * 4) || overlap(workspace, rb, table, tb) ||
        overlap(workspace, rb, refs, rb) || overlap(workspace, rb, lengths, rows * 4) || overlap(workspace, rb, out_table, tb) ||
        overlap(workspace, rb, out_refs, rb))
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "pages_resize: arguments overlap");
    spec_internal_set_error(SPEC_OK, "");
    PagesArgs a{};
    a.table = table;
    a.refs = refs;
    a.lengths = lengths;
    a.out_table = out_table;
    a.out_refs = out_refs;
    a.list = workspace;
    a.status = status;
    a.B = p->B;
    a.W = p->W;
    a.N = p->N;
    a.M = p->M;
    a.P = p->P;
    a.page = p->page;
    const int C = pages_cluster(entries + p->P);
    const uintptr_t all = reinterpret_cast<uintptr_t>(table) | reinterpret_cast<uintptr_t>(refs) | reinterpret_cast<uintptr_t>(out_table) |
                          reinterpret_cast<uintptr_t>(out_refs) | reinterpret_cast<uintptr_t>(workspace);
    static bool allowed[64], allowed4[64];
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (C > 1 && all % 16 == 0 && p->M % 4 == 0) return done(launch_pages(resize_kernel<4>, allowed4, a, C, st));
    return done(launch_pages(resize_kernel<1>, allowed, a, C, st));
}

extern "C" int spec_pages_fork(const spec_pages_params *p, const int32_t *table, const int32_t *refs,
                               const int32_t *lengths, const int32_t *parent, int32_t *out_table, int32_t *out_refs,
                               int32_t *out_lengths, int32_t *copies, int32_t *workspace, int32_t *status,
                               void *stream) {
    using namespace sr;
    const int rc = check_pages(p, true);
    if (rc != SPEC_OK) return rc;
    const int64_t rows = (int64_t)p->B * p->W, out_rows = (int64_t)p->B * p->N;
    if (rows == 0 && out_rows == 0 && p->P == 0) return spec_internal_set_error(SPEC_OK, "");
    if ((rows * p->M && !table) || (rows && !lengths) || (out_rows * p->M && !out_table) ||
        (out_rows && (!parent || !out_lengths || !copies)) || (p->P && (!refs || !out_refs || !workspace)))
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "pages_fork: an argument is NULL");
    const int64_t rb = (int64_t)p->P * 4;
    const void *in[4] = {table, lengths, parent, refs};
    const int64_t in_bytes[4] = {rows * p->M * 4, rows * 4, out_rows * 4, rb};
    const void *out[5] = {out_table, out_lengths, copies, workspace, out_refs};
    const int64_t out_bytes[5] = {out_rows * p->M * 4, out_rows * 4, out_rows * 16, 2 * rb, rb};
    for (int i = 0; i < 5; ++i) {
        for (int j = 0; j < 4; ++j)
            if (overlap(out[i], out_bytes[i], in[j], in_bytes[j]) && !(i == 4 && j == 3 && out_refs == refs))
                return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "pages_fork: an output overlaps an input");
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out_bytes[i], out[j], out_bytes[j]))
                return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "pages_fork: outputs overlap");
    }
    spec_internal_set_error(SPEC_OK, "");
    PagesArgs a{};
    a.table = table;
    a.refs = refs;
    a.lengths = lengths;
    a.parent = parent;
    a.out_table = out_table;
    a.out_refs = out_refs;
    a.out_lengths = out_lengths;
    a.copies = copies;
    a.list = workspace;
    a.claim = workspace + p->P;
    a.status = status;
    a.B = p->B;
    a.W = p->W;
    a.N = p->N;
    a.M = p->M;
    a.P = p->P;
    a.page = p->page;
    const int C = pages_cluster((rows + out_rows) * p->M + p->P);
    static bool allowed[64];
    return done(launch_pages(fork_kernel, allowed, a, C, static_cast<cudaStream_t>(stream)));
}

extern "C" int spec_pages_copy(const spec_cache_params *p, void *cache, const int32_t *copies, int32_t count,
                               void *stream) {
    using namespace sr;
    const int rc = check_cache(p);
    if (rc != SPEC_OK) return rc;
    if (count < 0) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "pages_copy: count must be >= 0");
    if (count == 0 || p->O == 0 || p->H == 0 || p->P == 0) return spec_internal_set_error(SPEC_OK, "");
    if (!cache || !copies) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "pages_copy: cache or copies is NULL");
    spec_internal_set_error(SPEC_OK, "");
    CacheArgs a{};
    cache_args(a, p, cache);
    a.copies = copies;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (vec_bytes(a)) {
        case 16: return done(launch_copy<uint4>(a, count, st));
        case 4: return done(launch_copy<uint32_t>(a, count, st));
        case 2: return done(launch_copy<uint16_t>(a, count, st));
        default: return done(launch_copy<uint8_t>(a, count, st));
    }
}

extern "C" int spec_pages_compact(const spec_cache_params *p, void *cache, int32_t B, int32_t N, int32_t M,
                                  const int32_t *table, const int32_t *lengths, const int32_t *path,
                                  int32_t *out_lengths, int32_t *status, void *stream) {
    using namespace sr;
    const int rc = check_cache(p);
    if (rc != SPEC_OK) return rc;
    if (B < 0 || M < 0) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "pages_compact: B and M must be >= 0");
    if (B > SPEC_MAX_B || N < 1 || N > SPEC_MAX_NODES || (int64_t)M * p->page > INT32_MAX - SPEC_MAX_NODES)
        return spec_internal_set_error(SPEC_ERR_UNSUPPORTED, "pages_compact: B, N or M out of range");
    if (B == 0) return spec_internal_set_error(SPEC_OK, "");
    if (!lengths || !path || !out_lengths || (M && !table) || (p->O && p->H && p->P && !cache))
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "pages_compact: an argument is NULL");
    if (overlap(out_lengths, B * 4LL, lengths, B * 4LL) || overlap(out_lengths, B * 4LL, path, (int64_t)B * N * 4) ||
        overlap(out_lengths, B * 4LL, table, (int64_t)B * M * 4))
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "pages_compact: out_lengths overlaps an input");
    spec_internal_set_error(SPEC_OK, "");
    CacheArgs a{};
    cache_args(a, p, cache);
    a.table = table;
    a.lengths = lengths;
    a.path = path;
    a.out_lengths = out_lengths;
    a.status = status;
    a.B = B;
    a.N = N;
    a.M = M;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (vec_bytes(a)) {
        case 16: return done(launch_compact<uint4>(a, st));
        case 4: return done(launch_compact<uint32_t>(a, st));
        case 2: return done(launch_compact<uint16_t>(a, st));
        default: return done(launch_compact<uint8_t>(a, st));
    }
}

extern "C" int spec_tree_accept(int32_t B, int32_t N, const int32_t *tokens, const int32_t *parents,
                                int64_t parents_stride, const int32_t *choice, int64_t choice_batch_stride,
                                int64_t choice_node_stride, const int32_t *counts, int32_t *accepted_len,
                                int32_t *out_tokens, int32_t *path, int32_t *status, void *stream) {
    using namespace sr;
    if (B < 0) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "tree_accept: B must be >= 0");
    if (B > SPEC_MAX_B || N < 1 || N > SPEC_MAX_NODES)
        return spec_internal_set_error(SPEC_ERR_UNSUPPORTED, "tree_accept: B or N out of range");
    if (parents && parents_stride != 0 && parents_stride < N)
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "tree_accept: parents_stride must be 0 or >= N");
    if (choice_batch_stride < 0 || choice_node_stride < 0 || choice_batch_stride > (INT64_MAX >> 4) / (B + 1) ||
        choice_node_stride > (INT64_MAX >> 12) || parents_stride > (INT64_MAX >> 4) / (B + 1))
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "tree_accept: strides must be >= 0 and not too large");
    if (B == 0) return spec_internal_set_error(SPEC_OK, "");
    if (!tokens || !choice || !accepted_len || !out_tokens || !path)
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "tree_accept: an argument is NULL");
    {
        const int64_t rows = (int64_t)B * N * 4;
        const void *in[4] = {tokens, parents, choice, counts};
        const int64_t in_bytes[4] = {rows, parents ? ((B - 1) * parents_stride + N) * 4 : 0,
                                     ((B - 1) * choice_batch_stride + (N - 1) * choice_node_stride + 1) * 4, counts ? B * 4LL : 0};
        const void *out[3] = {accepted_len, out_tokens, path};
        const int64_t out_bytes[3] = {B * 4LL, rows, rows};
        for (int i = 0; i < 3; ++i) {
            for (int j = 0; j < 4; ++j)
                if (overlap(out[i], out_bytes[i], in[j], in_bytes[j]))
                    return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "tree_accept: an output overlaps an input");
            for (int j = 0; j < i; ++j)
                if (overlap(out[i], out_bytes[i], out[j], out_bytes[j]))
                    return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "tree_accept: outputs overlap");
        }
    }
    spec_internal_set_error(SPEC_OK, "");
    const AcceptArgs a{tokens, parents, choice, counts, accepted_len, out_tokens, path, status,
                       parents_stride, choice_batch_stride, choice_node_stride, B, N};
    const unsigned grid = (unsigned)((B + NTA / 32 - 1) / (NTA / 32));
    accept_kernel<<<grid, NTA, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return done(cudaGetLastError());
}

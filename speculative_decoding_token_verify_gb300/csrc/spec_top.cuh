// spec_top.cuh -- the M largest logits of a part of a row, found while the
// part streams by: device code of the top lists and the beam step.
//
// Beside the softmax sum runs a filter: with T such that at least M logits
// seen so far are >= T, only vectors whose maximum reaches T can hold a listed
// token, and their indices go to a short list in shared memory. T comes from
// the threads' own running maxima: every warp sorts its 32, and with k =
// ceil(M / warps) the smallest of the warps' k-th largest has M logits at or
// above it. It is taken after iterations 1, 2, 4, 8, ... and once more at the
// end, and the part is read in U interleaved streams, so that the first
// iteration samples all of it. About 7 M vectors of a row of 128256 pass; the
// last bound leaves about 1.5 M, whose logits are looked at one by one and
// ranked by counting.
//
// Where more vectors pass than the list holds (runs of equal logits, all large
// logits in one place) a bisection finishes: the M-th largest key by counting
// passes, tokens above it in any order, tokens at it in ascending order. One CTA
// does that for its whole row: 8 rows of 128256 bf16 with ten tokens at large and
// the others at -1e9 take 570 us in place of 11 (M = 64), 256 rows 690 us in place
// of 21. Masked logits never get there (8 us for the same rows masked by -inf).
#pragma once

#include "spec_rows.cuh"

namespace sr {

constexpr int NT = 256;
constexpr int NW = NT / 32;
// 16-byte loads of an iteration per thread. Two iterations are in registers, at
// 64 of them a thread and 4 CTAs per SM: 2048 rows of 128256 bf16 take 110 us;
// 2 loads and 5 CTAs 119 us, 3 loads 120 us, 8 loads and 2 CTAs 133 us.
constexpr int U = 4;
constexpr int CAP = 2048;    // vectors that may pass the filter, per CTA
constexpr int CAPE = 1024;   // logits that may pass the last bound, per row
constexpr int kMaxCluster = 8;

// the k-th largest of the warp's values (k = 1 .. 32)
template <typename V>
__device__ __forceinline__ V warp_kth(V v, int k) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int o = size >> 1; o > 0; o >>= 1) {
            const V w = __shfl_xor_sync(kFull, v, o);
            const bool big = ((lane & o) == 0) == ((lane & size) == 0);   // descending runs
            v = big ? max(v, w) : min(v, w);
        }
    return __shfl_sync(kFull, v, k - 1);
}

// A bound with at least M of the block's `n` values (thread t holds the
// largest of the values t, t + NT, ...) at or above it, or `none`.
// buf: NW values, not written again before another barrier has passed.
template <typename V>
__device__ __forceinline__ V block_bound(V v, int n, int M, V none, V *buf) {
    const int act = min(NW, n >> 5);   // warps whose lanes all hold a value
    const int k = act ? (M + act - 1) / act : 33;
    if (k > 32) return none;           // the same in every thread
    const V t = warp_kth(v, k);
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = t;
    __syncthreads();
    V r = buf[0];
#pragma unroll
    for (int i = 1; i < NW; ++i)
        if (i < act) r = min(r, buf[i]);
    return max(r, none);
}


struct TopShared {
    float c[CAP];        // passing vectors: maximum and code (index in the row, or ~index of a single logit)
    int code[CAP];
    __align__(16) unsigned long long el[CAPE];   // candidates
    int few[CAPE];       // codes of the vectors that pass the last bound
    float b[3][NW], w_mx[NW], w_sum[NW];
    uint32_t kb[NW];
    int n, nf, ne, off, cnt[NW];
};

// places for the lanes that want one, from a shared counter: one addition a warp
__device__ __forceinline__ int take(bool want, int *counter) {
    const unsigned m = __ballot_sync(kFull, want);
    if (m == 0u) return 0;
    const int lane = threadIdx.x & 31, lead = __ffs(m) - 1;
    int at = 0;
    if (lane == lead) at = atomicAdd(counter, __popc(m));
    return __shfl_sync(kFull, at, lead) + __popc(m & ((1u << lane) - 1u));
}

template <typename T, typename F>
__device__ __forceinline__ void each(const Part<T> &p, F f) {
    constexpr int E = Row<T>::E;
    const int e = p.edge(threadIdx.x);
    if (e >= 0) f(load1(p.r.p + e), e);
    for (int k = threadIdx.x; k < p.n; k += NT) {
        float z[E];
        Elem<T>::unpack(__ldg(p.body() + k), z);
#pragma unroll
        for (int j = 0; j < E; ++j) f(z[j], p.r.vec_index(p.k0 + k) + j);
    }
}

// The part's list by bisection; at least M keys of the part are >= t, or t = 1.
// Leaves at most M candidates in s.el, in no order, and returns their number.
template <typename T>
__device__ __noinline__ int bisect(const Part<T> &p, int M, uint32_t t, float mx, TopShared &s) {
    auto count = [&](uint32_t k) {   // tokens of key >= k, k > 0
        int n = 0;
        each(p, [&](float z, int) { n += order_key(z) >= k; });
        n = __reduce_add_sync(kFull, n);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) s.cnt[threadIdx.x >> 5] = n;
        __syncthreads();
        n = 0;
        for (int i = 0; i < NW; ++i) n += s.cnt[i];
        return n;
    };
    // the largest t with count(t) >= M, or 1 when the part has no more tokens
    if (t > 1u || count(1u) > M) {
        uint32_t hi = order_key(mx);   // count(hi + 1) == 0 < M
        while (t < hi) {
            const uint32_t mid = t + (hi - t) / 2 + ((hi - t) & 1u);
            if (count(mid) >= M) t = mid;
            else hi = mid - 1;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) s.n = 0;
    __syncthreads();
    const bool all = t == 1u;
    each(p, [&](float z, int i) {
        const uint32_t key = order_key(z);
        if (all ? key >= 1u : key > t) {
            const int at = atomicAdd(&s.n, 1);
            if (at < M) s.el[at] = cand(key, i);
        }
    });
    __syncthreads();
    int n = min(s.n, M);
    if (!all) {   // tokens at the threshold, lowest index first
        for (int i0 = p.e0; i0 < p.e1 && n < M; i0 += NT) {
            const int i = i0 + threadIdx.x;
            const bool at = i < p.e1 && order_key(load1(p.r.p + i)) == t;
            const unsigned bal = __ballot_sync(kFull, at);
            __syncthreads();
            if ((threadIdx.x & 31) == 0) s.cnt[threadIdx.x >> 5] = __popc(bal);
            __syncthreads();
            int before = n + __popc(bal & ((1u << (threadIdx.x & 31)) - 1u)), total = 0;
            for (int w = 0; w < NW; ++w) {
                before += w < (int)(threadIdx.x >> 5) ? s.cnt[w] : 0;
                total += s.cnt[w];
            }
            if (at && before < M) s.el[before] = cand(t, i);
            n = min(n + total, M);
        }
        __syncthreads();
    }
    return n;
}

// One pass over a part: a bound `thr` with at least M of its logits at or above
// it (or the mask's floor; the same in every thread), the vectors that may hold
// listed tokens in s.c and s.code, every warp's maximum and sum in s.w_mx and
// s.w_sum. The caller's next barrier publishes all of it.
template <typename T>
__device__ __forceinline__ void stream_part(const Part<T> &p, int M, float sL, float rs, TopShared &s, float &thr) {
    constexpr int E = Row<T>::E;
    const int tid = threadIdx.x, n = p.n;
    const uint4 *body = p.body();
    if (tid == 0) s.n = s.nf = s.ne = 0;
    __syncthreads();
    Sum acc = sum_init(sL, rs);
    thr = sv::kMaskFloor;
    const int its = (n + U * NT - 1) / (U * NT), span = its * NT;
    int refresh = 0;
    auto load = [&](uint4 (&w)[U], int it) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = u * span + it * NT + tid;
            w[u] = it < its && i < n ? sv::ldg_stream(body + i) : masked_vec<T>();
        }
    };
    auto work = [&](const uint4 (&w)[U], int it) {
        float c[U], cm;
#pragma unroll
        for (int u = 0; u < U; ++u) c[u] = vec_max<T>(w[u]);
        cm = c[0];
#pragma unroll
        for (int u = 1; u < U; ++u) cm = fmaxf(cm, c[u]);
        sum_see(acc, cm, sL, rs);
        float v = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float z[E];
            Elem<T>::unpack(w[u], z);
            v += sum_terms<E>(acc, z, sL);
        }
        sum_put(acc, v);
        if ((it & (it + 1)) == 0 && (it == 0 || it + 1 < its)) {
            thr = block_bound(acc.mx, n, M, thr, s.b[refresh]);
            refresh ^= 1;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c[u] >= thr) {
                const int at = atomicAdd(&s.n, 1);
                if (at < CAP) {
                    s.c[at] = c[u];
                    s.code[at] = p.k0 + u * span + it * NT + tid;
                }
            }
    };
    // the next iteration's loads are on their way while one is worked on
    uint4 w0[U], w1[U];
    load(w0, 0);
    for (int it = 0; it < its; it += 2) {
        load(w1, it + 1);
        work(w0, it);
        if (it + 1 >= its) break;
        load(w0, it + 2);
        work(w1, it + 1);
    }
    const int e = p.edge(tid);   // the row's ends: single logits
    if (e >= 0) {
        const float z = load1(p.r.p + e);
        sum_add1(acc, z, sL, rs);
        if (z >= thr) {
            const int at = atomicAdd(&s.n, 1);
            if (at < CAP) {
                s.c[at] = z;
                s.code[at] = ~e;
            }
        }
    }
    const float m = warp_max(acc.mx), v = warp_sum(sum_at(acc, m, sL));
    if ((tid & 31) == 0) {
        s.w_mx[tid >> 5] = m;
        s.w_sum[tid >> 5] = v;
    }
    // a last bound, from all of the part (its barrier, or the caller's)
    if (its > 1) thr = block_bound(acc.mx, n, M, thr, s.b[2]);
}

// the part's logits equal to mx; NaN where some are infinite or NaN
template <typename T>
__device__ __forceinline__ float count_equal(const Part<T> &p, float mx, TopShared &s) {
    int n = 0;
    each(p, [&](float z, int) { n = z != z ? n | 1 << 24 : n + (z == mx); });
    n = mx < INFINITY ? __reduce_add_sync(kFull, min(n, 1 << 24)) : 1 << 24;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s.cnt[threadIdx.x >> 5] = n;
    __syncthreads();
    n = 0;
    for (int i = 0; i < NW; ++i) n += min(s.cnt[i], 1 << 24);
    return n < 1 << 24 ? (float)n : NAN;
}

// the part's maximum and sum, after the barrier; where the maximum is far out
// count_equal is the sum
__device__ __forceinline__ void part_sum(const TopShared &s, float sL, float &mx, float &sum) {
    mx = s.w_mx[0];
#pragma unroll
    for (int i = 1; i < NW; ++i) mx = fmaxf(mx, s.w_mx[i]);
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < NW; ++i) sum += moved(s.w_sum[i], s.w_mx[i], mx, sL);
}

// `n` words from this CTA's shared memory to the list `to` of the cluster's
// first CTA, behind what other CTAs have put there; `counter` counts them all,
// past `room` too. One remote addition per CTA: they are slow, and one after
// another. All threads call it; a barrier follows.
template <typename F>
__device__ __forceinline__ void hand_over(int n, F word, unsigned long long *to, int *counter, int room, int *off) {
    if (threadIdx.x == 0) *off = peer_add(peer(counter, 0), n);
    __syncthreads();
    const uint32_t at = peer(to, 0);
    for (int i = threadIdx.x; i < n; i += NT)
        if (*off + i < room) peer_store(at + 8u * (*off + i), word(i));
}

// The passing vectors' logits at or above thr, as candidates in dst[0 .. CAPE),
// counted in *counter past CAPE too. Returns whether more vectors reach thr than
// there is room for. A barrier follows.
template <typename T>
__device__ __forceinline__ bool expand(const Part<T> &p, float thr, TopShared &s, unsigned long long *dst, int *counter) {
    constexpr int E = Row<T>::E, G = 4;   // logits per thread and round, loaded together
    const int np = min(s.n, CAP), lane = threadIdx.x & 31;
    for (int i0 = 0; i0 < np; i0 += NT) {
        const int i = i0 + threadIdx.x;
        const bool want = i < np && s.c[i] >= thr;
        const int at = take(want, &s.nf);
        if (want && at < CAPE) s.few[at] = s.code[i];
    }
    __syncthreads();
    const int nf = s.nf;
    if (nf > CAPE) return true;
    for (int i0 = 0; i0 < nf * E; i0 += G * NT) {
        float z[G];
        int index[G];
#pragma unroll
        for (int k = 0; k < G; ++k) {
            const int i = i0 + k * NT + threadIdx.x, j = i & (E - 1);
            const int code = i < nf * E ? s.few[i / E] : ~0;
            index[k] = code >= 0 ? p.r.vec_index(code) + j : ~code;
            z[k] = i < nf * E && (code >= 0 || j == 0) ? load1(p.r.p + index[k]) : neg_inf();
        }
        unsigned m[G];
        int total = 0;
#pragma unroll
        for (int k = 0; k < G; ++k) {
            m[k] = __ballot_sync(kFull, z[k] >= thr && order_key(z[k]) != 0u);
            total += __popc(m[k]);
        }
        if (total == 0) continue;
        int at = 0;
        if (lane == 0) at = atomicAdd(counter, total);
        at = __shfl_sync(kFull, at, 0);
#pragma unroll
        for (int k = 0; k < G; ++k) {
            const int to = at + __popc(m[k] & ((1u << lane) - 1u));
            if ((m[k] >> lane & 1u) && to < CAPE) dst[to] = cand(order_key(z[k]), index[k]);
            at += __popc(m[k]);
        }
    }
    return false;
}

// The candidates s.el[0 .. ne) cut down to few more than the M best; returns
// their number. Called and left by all threads together.
__device__ __forceinline__ int cut(int ne, int M, TopShared &s) {
    if (ne <= 128) return ne;
    uint32_t k = 0u;
    for (int i = threadIdx.x; i < ne; i += NT) k = max(k, cand_key(s.el[i]));
    const uint32_t bound = block_bound(k, ne, M, 0u, s.kb);
    if (bound == 0u) return ne;
    // s.c holds CAP 32-bit words: room for half as many candidates
    unsigned long long *few = reinterpret_cast<unsigned long long *>(s.c);
    static_assert(CAP >= 2 * CAPE, "the cut's buffer");
    if (threadIdx.x == 0) s.n = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < ne; i += NT)
        if (cand_key(s.el[i]) >= bound) few[atomicAdd(&s.n, 1)] = s.el[i];
    __syncthreads();
    ne = s.n;
    for (int i = threadIdx.x; i < ne; i += NT) s.el[i] = few[i];
    __syncthreads();
    return ne;
}

// f(candidate, rank) for the M best of s.el[0 .. ne): each candidate's rank is
// counted by G neighbouring lanes
template <int G, typename F>
__device__ __forceinline__ void ranked_by(int ne, int M, const TopShared &s, F f) {
    const int g = threadIdx.x & (G - 1);
    for (int i0 = 0; i0 < ne; i0 += NT / G) {
        const int i = i0 + threadIdx.x / G;
        const unsigned long long c = i < ne ? s.el[i] : 0ull;
        int rk = 0;
#pragma unroll 4
        for (int j = g; j < ne; j += G) rk += s.el[j] > c;
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) rk += __shfl_xor_sync(kFull, rk, o);
        if (g == 0 && i < ne && rk < M) f(c, rk);
    }
}
template <typename F>
__device__ __forceinline__ void ranked(int ne, int M, const TopShared &s, F f) {
    if (ne <= NT / 8) ranked_by<8>(ne, M, s, f);
    else if (ne <= NT / 4) ranked_by<4>(ne, M, s, f);
    else if (ne <= NT / 2) ranked_by<2>(ne, M, s, f);
    else ranked_by<1>(ne, M, s, f);
}

}  // namespace sr

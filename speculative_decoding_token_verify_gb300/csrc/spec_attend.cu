// spec_attend.cu -- attention of a tree's nodes over a cache held in pages.
//
// Rows. The query rows of one key head's group, (node, head) in node order, fill
// tiles of 128 rows: floor(128 / G) nodes each. S = Q K^T (128 rows x 128
// keys) and O += P V run on the tensor cores with S, P and O in tensor memory;
// a thread owns a row of S and keeps its running maximum and sum.
//
// Streams. A CTA has two streams, each with an S, an O and a warpgroup for the
// softmax, so that one multiplies while the other exponentiates. A group of one tile
// gives the streams every other tile of keys and merges them at the end; two
// tiles of rows get a stream each and share the keys.
//
// Work. All tiles of keys of all (sequence, head, pair of row tiles) stand in one line that is
// cut into equal parts, one per CTA, from lengths that only the GPU knows; a
// part's ends may lie inside a sequence. Those pieces go to the workspace unnormalised, and a
// second kernel joins them.
//
// What a row must not see. Keys behind the context are masked by a bit per node. A
// probability of 0 does not stop a NaN value, so a warp of its own looks at the values behind the
// context before they are multiplied: slots that no node owns become 0, and of the nodes' own values the NaN and infinities
// do, and are added back at the end to the rows that see them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cmath>
#include <mutex>

#include "spec_rows.cuh"
#include "spec_tc.cuh"

namespace sr {

constexpr int kTile = 128;             // keys a tile, and rows a tile
constexpr int kChunk = kTile * 128;    // bytes of 64 elements of a tile's rows
constexpr int kNT = 384;               // keys, products, values' check, values; two softmax warpgroups
constexpr unsigned kSpin = 1u << 20;   // polls of a wait before it gives up
constexpr int kSegRing = 6;            // segments whose flags of non-finite values are kept
constexpr float kLazy = 8.f;           // a row's reference moves when its maximum is 2^8 above it

struct AttendArgs {
    const void *v;
    const int32_t *table, *lengths, *parents, *counts;
    void *out;
    float *lse;
    int32_t *status;
    float4 *part_o;   // [CTA][2][tile][D padded / 4][row]: unnormalised outputs of a sequence's pieces
    float2 *part_ml;  // [CTA][2][tile][row]: their reference (log2) and sum
    int4 *joins;      // [CTA]: sequence (-1: none), head, pair of tiles, last CTA of what begins here and ends elsewhere
    int B, N, Hq, Hkv, G, D, P, page, M, fill;
    int nodes;        // a tile
    float sL;         // |scale| log2 e
    int neg;          // scale < 0
    long long vs[3], ps;
};

// What a sequence holds: tokens before the nodes, and nodes.
__device__ __forceinline__ void sequence(const AttendArgs &a, int b, int &L, int &count) {
    count = a.counts ? a.counts[b] : a.N;
    L = a.lengths[b];
    int bad = 0;
    if (count < 0 || count > a.N) {
        bad = SPEC_ERR_BAD_LENGTH;
        count = count < 0 ? 0 : a.N;
    }
    const long long most = (long long)a.M * a.page;
    if (count > most) {
        bad = SPEC_ERR_BAD_LENGTH;
        count = (int)most;
    }
    if (L < 0 || L > most - count) {
        bad = SPEC_ERR_BAD_LENGTH;
        L = L < 0 ? 0 : (int)(most - count);
    }
    if (bad) raise_status(a.status, bad);
}

__device__ __forceinline__ int parent_of(const AttendArgs &a, int b, int n) {
    if (!a.parents) return n - 1;
    const int p = a.parents[b * a.ps + n];
    if (p >= -1 && p < n) return p;
    raise_status(a.status, SPEC_ERR_BAD_PARENT);
    return -1;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

template <typename T>
struct Half;
template <>
struct Half<__nv_bfloat16> {
    static constexpr int kBf16 = 1;
    static constexpr uint32_t kExp = 0x7f80;
    __device__ static __forceinline__ uint32_t pack(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    __device__ static __forceinline__ float value(uint32_t h) { return __uint_as_float(h << 16); }
};
template <>
struct Half<__half> {
    static constexpr int kBf16 = 0;
    static constexpr uint32_t kExp = 0x7c00;
    __device__ static __forceinline__ uint32_t pack(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    __device__ static __forceinline__ float value(uint32_t h) { return __half2float(__ushort_as_half((unsigned short)h)); }
};

// (a 64-bit division costs ten times a 32-bit one)
__device__ __forceinline__ long long quotient(long long x, long long y) {
    return ((x | y) >> 32) == 0 ? (long long)((uint32_t)x / (uint32_t)y) : x / y;
}

// One piece of a CTA's work, tiles [t0, t1) of `tiles` of (b, h, pair), and what is left behind
// it. Every warp walks the CTA's segments by itself; its place stands in shared memory,
// which leaves registers to what the warp does.
struct Segment {
    int b, h, pair, t0, t1, tiles, L, count;
    uint8_t act, begun;     // row tiles with nodes; whether next() has given the first one
    long long off, left;    // units of sequence b behind this piece, and of the CTA's part
    __device__ __forceinline__ int keys(int t) const { return min(kTile, L + count - t * kTile); }
    __device__ __forceinline__ bool next(const AttendArgs &a) {
        if (!begun) {
            begun = 1;
            return t1 > t0;
        }
        while (left > 0) {
            sequence(a, b, L, count);
            const int pairs = (count + 2 * a.nodes - 1) / (2 * a.nodes);
            tiles = (L + count + kTile - 1) / kTile;
            const long long head = (long long)pairs * tiles, all = head * a.Hkv;
            if (off >= all) {
                off -= all;
                ++b;
                continue;
            }
            h = (int)quotient(off, head);
            const long long in = off - h * head;
            pair = (int)quotient(in, tiles);
            t0 = (int)(in - (long long)pair * tiles);
            t1 = t0 + (int)min((long long)(tiles - t0), left);
            act = count - pair * 2 * a.nodes > a.nodes ? 2 : 1;
            off += t1 - t0;
            left -= t1 - t0;
            return true;
        }
        return false;
    }
};

template <int DC>
struct AttendSmem {
    static constexpr int kStage = DC * kChunk;
    static constexpr int kStages = DC == 2 ? 5 : 10;
    static constexpr int kQ = 2 * kStage;
    static constexpr int kTiles = kQ + kStages * kStage;
};

// behind the tiles in shared memory
template <int S>
struct AttendShared {
    struct {
        uint64_t full[S], empty[S], fixed[S], s_full[2], p_ready[2], pv_done[2], q_full, q_empty, o_free, merge, drain;
    } bars;
    union {
        float2 ml[2][kTile];
        long long sum[kNT / 32];
    };
    Segment seg[kNT / 32];
    uint32_t tmem, bad[kSegRing][4];
    int abort;
};

template <typename T, int DC>
__global__ void __launch_bounds__(kNT, 1)
    attend_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ CUtensorMap qmap,
                  const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, int box) {
    using SM = AttendSmem<DC>;
    constexpr int S = SM::kStages, DP = DC * 64;
    extern __shared__ __align__(1024) char dyn[];   // (the kernel has no other shared memory, so that this holds)
    AttendShared<S> &sh = *reinterpret_cast<AttendShared<S> *>(dyn + SM::kTiles);
    auto &bars = sh.bars;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = tc::smem(dyn), ring = base + SM::kQ;
    if (threadIdx.x == 0) {
        tc::prefetch_map(&kmap);
        tc::prefetch_map(&qmap);
        tc::prefetch_map(&vmap);
    }

    if (threadIdx.x == 0) {
        sh.abort = 0;
        for (int w = 0; w < kNT / 32; ++w) sh.seg[w].t0 = sh.seg[w].t1 = sh.seg[w].begun = 0;
        for (int i = 0; i < S; ++i) {
            tc::bar_init(tc::smem(&bars.full[i]), 1);
            tc::bar_init(tc::smem(&bars.empty[i]), 2);   // the products and the values' check
            tc::bar_init(tc::smem(&bars.fixed[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::bar_init(tc::smem(&bars.s_full[i]), 1);
            tc::bar_init(tc::smem(&bars.p_ready[i]), 4);
            tc::bar_init(tc::smem(&bars.pv_done[i]), 1);
        }
        tc::bar_init(tc::smem(&bars.q_full), 1);
        tc::bar_init(tc::smem(&bars.q_empty), 1);
        tc::bar_init(tc::smem(&bars.o_free), 8);
        tc::bar_init(tc::smem(&bars.merge), 8);
        tc::bar_init(tc::smem(&bars.drain), 1);
        tc::fence_barrier_init();
    }
    if (warp == 1) tc::tmem_alloc(tc::smem(&sh.tmem), 512);
    // (so far nothing that an earlier kernel of the stream may write has been read)
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- which part of the line is this CTA's ----------------------------------------
    const int G = gridDim.x, me = blockIdx.x;
    const int per_thread = (a.B + kNT - 1) / kNT;
    const int b_lo = min(a.B, (int)threadIdx.x * per_thread), b_hi = min(a.B, b_lo + per_thread);
    auto units = [&](int b) -> long long {
        int L, count;
        sequence(a, b, L, count);
        return (long long)a.Hkv * ((count + 2 * a.nodes - 1) / (2 * a.nodes)) * ((L + count + kTile - 1) / kTile);
    };
    long long mine = 0;
    for (int b = b_lo; b < b_hi; ++b) mine += units(b);
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const long long v = __shfl_up_sync(kFull, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) sh.sum[warp] = upto;
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    long long total = 0;
    for (int w = 0; w < kNT / 32; ++w) {
        if (w < warp) upto += sh.sum[w];
        total += sh.sum[w];
    }
    const long long per = (total + G - 1) / G, u0 = min(total, me * per), u1 = min(total, u0 + per);
    if (u0 < u1 && u0 >= upto - mine && u0 < upto) {   // the thread whose sequences hold u0
        long long at = upto - mine;
        for (int b = b_lo; b < b_hi; ++b) {
            const long long n = units(b);
            if (u0 < at + n) {
                Segment first;
                first.begun = 1;
                first.b = b;
                first.off = u0 - at;
                first.left = u1 - u0;
                first.next(a);
                first.begun = 0;
                for (int w = 0; w < kNT / 32; ++w) sh.seg[w] = first;
                break;
            }
            at += n;
        }
    }
    if (a.fill) {   // rows of nodes that do not exist
        const long long rows = (long long)a.B * a.N * a.Hq;
        for (long long r = (long long)me * kNT + threadIdx.x; r < rows; r += (long long)G * kNT) {
            const int b = (int)(r / ((long long)a.N * a.Hq)), n = (int)(r / a.Hq % a.N);
            int L, count;
            sequence(a, b, L, count);
            if (n < count) continue;
            uint4 *o = reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + r * a.D);
            for (int i = 0; i < a.D / 8; ++i) o[i] = make_uint4(0, 0, 0, 0);
            if (a.lse) a.lse[r] = neg_inf();
        }
    }
    __syncthreads();
    Segment &s = sh.seg[warp];
    auto next_segment = [&]() -> bool {
        bool more = false;
        __syncwarp();
        if (lane == 0) more = s.next(a);
        more = __shfl_sync(kFull, more, 0);   // (the other lanes see the segment from here on)
        __syncwarp();
        return more;
    };
    const uint32_t tmem = sh.tmem;
    const uint32_t tS[2] = {tmem, tmem + 128}, tO[2] = {tmem + 256, tmem + 256 + DP};
    constexpr uint32_t kIdS = tc::shape(Half<T>::kBf16, kTile, false), kIdO = tc::shape(Half<T>::kBf16, DP, true);

    // A wait that gives up: the CTA's other waits then do, too. (The lanes vote, so that the
    // loop does not diverge.)
    auto wait_warp = [&](const uint64_t *bar, uint32_t parity) -> bool {
        const uint32_t addr = tc::smem(bar);
        for (unsigned i = 0; i < kSpin; ++i) {
            if (__all_sync(kFull, tc::bar_try(addr, parity))) return true;
            if (__any_sync(kFull, *(volatile int *)&sh.abort)) return false;
        }
        *(volatile int *)&sh.abort = 1;
        raise_status(a.status, SPEC_ERR_TIMEOUT);
        return false;
    };

    // 168 registers a thread at the launch: 96 for four warps and 200 for eight
    if (warp < 4) {
        tc::fewer_registers<96>();
        if (warp == 0 || warp == 3) {
            // ---- copies: warp 0 the queries and keys, warp 3 the values ----------------------------
            // Both fill one ring of stages, in the order in which the products use them:
            // `ahead` tiles of keys, then values and keys in turn. The products give stages back in
            // that order, so that a warp's wait for a stage is never two phases ahead.
            const bool keys = warp == 0;
            const CUtensorMap *map = keys ? &kmap : &vmap;
            const int bpt = kTile / box, group = 32 / bpt;   // boxes a tile; tiles whose pages the lanes hold (powers of two)
            const int page_bits = 31 - __clz(a.page);
            unsigned n0 = 0, segs = 0, last = 0;
            bool ok = true;
            while (ok && next_segment()) {
                const int t0 = s.t0, nt = s.t1 - t0, ahead = s.act == 2 ? 1 : 2, head = s.h, end = s.L + s.count;
                const int32_t *row = a.table + (long long)s.b * a.M;
                // lane l: the page of box l % bpt of tile l / bpt of the group
                auto pages = [&](int t) -> int {
                    const long long key = (long long)(t0 + t) * kTile + lane * box;
                    if (t + lane / bpt >= nt || key >= end) return -1;
                    return row[key >> page_bits];   // (looked at when it is used)
                };
                int now = pages(0), next = pages(group);
                for (int t = 0; ok && t < nt; ++t) {
                    if (t && (t & (group - 1)) == 0) {
                        now = next;
                        next = pages(t + group);
                    }
                    const unsigned n = n0 + (keys ? (t < ahead ? t : ahead + 2 * (t - ahead) + 1) : (t < nt - ahead ? min(nt, ahead) + 2 * t : nt + t));
                    const int st = n % S;
                    if (n >= S && !(ok = wait_warp(&bars.empty[st], (n / S + 1) & 1))) break;
                    const int boxes = (min(kTile, end - (t0 + t) * kTile) + box - 1) / box;
                    const uint32_t bar = tc::smem(&bars.full[st]), dst = ring + st * SM::kStage;
                    if (lane == 0) tc::bar_expect(bar, (uint32_t)boxes * box * 128 * DC);
                    __syncwarp();
                    const int bx = DC == 2 ? lane >> 1 : lane, c = DC == 2 ? lane & 1 : 0;   // (at most 16 boxes)
                    int p = __shfl_sync(kFull, now, (t & (group - 1)) * bpt + min(bx, bpt - 1));
                    if (bx < boxes) {
                        if (p < 0 || p >= a.P) {
                            raise_status(a.status, SPEC_ERR_BAD_PAGE);
                            p = -1;   // (the copy fills zeros)
                        }
                        tc::load_tile(dst + c * kChunk + bx * box * 128, map, bar, c * 64, head, ((t0 + t) * kTile + bx * box) & (a.page - 1), p);
                    }
                    last = n + 1;
                    if (keys && t == min(nt, ahead) - 1) {
                        if (segs > 0 && !(ok = wait_warp(&bars.q_empty, (segs + 1) & 1))) break;
                        if (lane == 0) {
                            const uint32_t qbar = tc::smem(&bars.q_full);
                            tc::bar_expect(qbar, (uint32_t)a.nodes * a.G * 128 * DC * s.act);
                            for (int m = 0; m < s.act; ++m)
                                for (int x = 0; x < DC; ++x)
                                    tc::load_tile(base + m * SM::kStage + x * kChunk, &qmap, qbar, x * 64, s.h * a.G, (2 * s.pair + m) * a.nodes, s.b);
                        }
                        __syncwarp();
                        ++segs;
                    }
                }
                n0 += 2 * nt;
            }
            // nothing is left in flight when another role has given up
            if (*(volatile int *)&sh.abort) {
                for (unsigned i = last > S ? last - S : 0; i < last; ++i)
                    for (unsigned k = 0; k < kSpin && !tc::bar_try(tc::smem(&bars.full[i % S]), (i / S) & 1); ++k) {}
                if (segs > 0)
                    for (unsigned k = 0; k < kSpin && !tc::bar_try(tc::smem(&bars.q_full), (segs + 1) & 1); ++k) {}
            }
        } else if (warp == 1) {
            // ---- products ---------------------------------------------------------------------
            // The whole warp walks along, so that operands stay in uniform registers; one
            // thread issues.
            const bool lead = tc::elect();
            unsigned n0 = 0, segs = 0, done0 = 0, done1 = 0;
            uint32_t fixed = 0;   // per stage: parity of the next wait for checked values
            bool ok = true;
            while (ok && next_segment()) {
                const int two = s.act == 2, nt = s.t1 - s.t0, ahead = two ? 1 : 2, jobs = two ? 2 * nt : nt;
                const int tails = max(0, s.L / kTile - s.t0);                   // tiles from here on hold nodes' keys
                const int end_steps = (s.keys(s.t1 - 1) + 15) / 16;             // products of the last tile
                // the places of a job's keys and values in the order of copies
                auto kplace = [&](int j) -> unsigned {
                    const int t = two ? j >> 1 : j;
                    return n0 + (t < ahead ? t : 2 * t - ahead + 1);
                };
                auto keys_there = [&](int j) -> bool {
                    const unsigned at = kplace(j);
                    return (two && (j & 1)) || wait_warp(&bars.full[at % S], (at / S) & 1);
                };
                // S of job j
                auto scores = [&](int j, uint32_t q, uint32_t k, uint32_t d) {
                    const int g = j & 1;
#pragma unroll
                    for (int i = 0; i < DC * 4; ++i) {
                        const uint32_t o = ((i >> 2) * kChunk + (i & 3) * 32) >> 4;
                        tc::mma_ss(d, tc::operand(q + o), tc::operand(k + o), kIdS, i > 0);
                    }
                    tc::commit(tc::smem(&bars.s_full[g]));
                    if (!two || g == 1) tc::commit(tc::smem(&bars.empty[kplace(j) % S]));
                    if (j == jobs - 1) tc::commit(tc::smem(&bars.q_empty));
                };
                const uint32_t q0 = tc::operand_lo(base, 16), q1 = two ? q0 + (SM::kStage >> 4) : q0;
                if (!wait_warp(&bars.q_full, segs & 1)) break;
                for (int j = 0; ok && j < min(jobs, 2); ++j) {
                    if (!(ok = keys_there(j))) break;
                    const uint32_t q = tc::uniform(j ? q1 : q0), k = tc::uniform(tc::operand_lo(ring + kplace(j) % S * SM::kStage, 16));
                    const uint32_t d = tc::uniform(tS[0] + (j & 1) * 128);
                    tc::fence_after();
                    if (lead) scores(j, q, k, d);
                    __syncwarp();
                }
                // Job j's P V, then job j + 2's Q K^T into the same columns: all that they wait for but P
                // is waited for before P, so that the tensor cores get both without a pause.
                for (int j = 0; ok && j < jobs; ++j) {
                    const int g = j & 1, t = two ? j >> 1 : j;
                    const unsigned at = n0 + (t < nt - ahead ? min(nt, ahead) + 2 * t : nt + t), st = at % S;
                    const bool more = j + 2 < jobs;
                    if (!two || g == 0) {
                        ok = wait_warp(&bars.full[st], (at / S) & 1);
                        if (ok && t >= tails) {
                            ok = wait_warp(&bars.fixed[st], fixed >> st & 1);
                            fixed ^= 1u << st;
                        }
                        if (!ok) break;
                    }
                    if (more && !(ok = keys_there(j + 2))) break;
                    if (j == 0 && segs > 0 && !(ok = wait_warp(&bars.o_free, (segs + 1) & 1))) break;
                    const uint32_t v = tc::uniform(tc::operand_lo(ring + st * SM::kStage, kChunk));
                    const uint32_t d = tc::uniform(tO[0] + g * DP), p = tc::uniform(tS[0] + g * 128);
                    const uint32_t q = tc::uniform(g ? q1 : q0), k = tc::uniform(tc::operand_lo(ring + kplace(j + 2) % S * SM::kStage, 16));
                    const int steps = t == nt - 1 ? end_steps : kTile / 16;
                    if (!(ok = wait_warp(&bars.p_ready[g], (g ? done1 : done0) & 1))) break;
                    tc::fence_after();
                    if (lead) {
                        if (steps == kTile / 16) {
#pragma unroll
                            for (int i = 0; i < kTile / 16; ++i) tc::mma_ts(d, p + i * 8, tc::operand(v + i * 128), kIdO, j >= 2 || i > 0);
                        } else {
                            for (int i = 0; i < steps; ++i) tc::mma_ts(d, p + i * 8, tc::operand(v + i * 128), kIdO, j >= 2 || i > 0);
                        }
                        tc::commit(tc::smem(&bars.pv_done[g]));
                        if (!two || g == 1) tc::commit(tc::smem(&bars.empty[st]));
                        if (more) scores(j + 2, q, k, p);
                    }
                    __syncwarp();
                    if (g) ++done1;
                    else ++done0;
                }
                n0 += 2 * nt;
                ++segs;
            }
            // (none of the products may still run when the CTA ends)
            if (lead) {
                tc::commit(tc::smem(&bars.drain));
                for (unsigned k = 0; k < kSpin && !tc::bar_try(tc::smem(&bars.drain), 0); ++k) {}
            }
            __syncwarp();
        } else {
            // ---- values behind the context -----------------------------------------------------
            unsigned n = 0, segs = 0;
            int4 join = make_int4(-1, 0, 0, 0);
            long long at_unit = u0;
            bool ok = true;
            while (ok && next_segment()) {
                const int nt = s.t1 - s.t0, ahead = s.act == 2 ? 1 : 2;
                if (s.t0 == 0 && s.t1 < s.tiles) join = make_int4(s.b, s.h, s.pair, (int)((at_unit + s.tiles - 1) / per));
                at_unit += nt;
                bool first = true;
                uint32_t *bad = sh.bad[segs % kSegRing];
                // every tile is waited for and given back in the order of the copies, so that no barrier is
                // ever two phases ahead of this warp or behind it
                for (int x = 0; ok && x < 2 * nt; ++x, ++n) {
                    const unsigned st = n % S;
                    if (!(ok = wait_warp(&bars.full[st], (n / S) & 1))) break;
                    const int v = x < min(nt, ahead) ? -1 : x - min(nt, ahead), lag = nt - min(nt, ahead);
                    // values and keys take turns while there are keys left
                    const int t = v < 0 ? -1 : v < 2 * lag ? (v & 1 ? -1 : v >> 1) : v - lag;
                    if (t < 0 || s.t0 + t < s.L / kTile) {
                        if (lane == 0) tc::bar_arrive(tc::smem(&bars.empty[st]));
                        continue;
                    }
                    if (first && lane < 4) bad[lane] = 0;
                    first = false;
                    __syncwarp();
                    const int at0 = (s.t0 + t) * kTile, keys = s.keys(s.t0 + t), lo = max(0, s.L - at0);
                    char *stage = dyn + SM::kQ + st * SM::kStage;
                    const int rows = ((keys + 15) & ~15) - lo;   // up to the last product's end
                    for (int i = lane; i < rows * DC * 8; i += 32) {
                        const int r = lo + i / (DC * 8), x = i % (DC * 8);
                        uint4 *p = reinterpret_cast<uint4 *>(stage + (x >> 3) * kChunk + r * 128 + (x & 7) * 16);
                        if (r >= keys) {
                            *p = make_uint4(0, 0, 0, 0);
                            continue;
                        }
                        uint4 w = *p;
                        uint32_t *u = &w.x;
                        bool hit = false;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if ((u[e] & Half<T>::kExp) == Half<T>::kExp) u[e] &= 0xffff0000u, hit = true;
                            if ((u[e] >> 16 & Half<T>::kExp) == Half<T>::kExp) u[e] &= 0x0000ffffu, hit = true;
                        }
                        if (hit) {
                            *p = w;
                            const int node = at0 + r - s.L;
                            atomicOr(&bad[node >> 5], 1u << (node & 31));
                        }
                    }
                    tc::fence_async();
                    __syncwarp();
                    if (lane == 0) {
                        tc::bar_arrive(tc::smem(&bars.fixed[st]));
                        tc::bar_arrive(tc::smem(&bars.empty[st]));
                    }
                }
                ++segs;
            }
            if (lane == 0) a.joins[me] = join;
        }
    } else {
        tc::more_registers<200>();
        // ---- softmax: a stream each, a row a thread ------------------------------------------
        const int g = (warp - 4) >> 2, r = threadIdx.x & 127;
        const uint32_t row_lane = (uint32_t)(warp & 3) << 21;   // (lane of tensor memory in bits 16 and up)
        const uint32_t mS = tS[g] + row_lane;
        unsigned segs = 0, merges = 0, own = 0, other = 0;   // jobs of this stream and the other so far
        bool ok = true;
        while (ok && next_segment()) {
            const int first = s.t0, step = s.act == 2, tails = s.L / kTile, jobs = (s.t1 - first) << step;
            // what this row sees of the nodes
            const int tile0 = 2 * s.pair + (s.act == 2 ? g : 0), node = tile0 * a.nodes + r / a.G;
            const bool real = r < a.nodes * a.G && node < s.count;
            uint32_t v0 = 0, v1 = 0, v2 = 0, v3 = 0;
            if (real && s.t1 > tails) {
                for (int j = node; j >= 0; j = parent_of(a, s.b, j)) {
                    const uint32_t bit = 1u << (j & 31);
                    const int w = j >> 5;
                    if (w == 0) v0 |= bit;
                    else if (w == 1) v1 |= bit;
                    else if (w == 2) v2 |= bit;
                    else v3 |= bit;
                }
            }
            const bool idle = !__any_sync(kFull, real);   // a warp without rows: what it leaves in P stays in its rows
            float m = neg_inf(), l = 0.f;
            for (int j = g; j < jobs; j += 2) {
                if (!(ok = wait_warp(&bars.s_full[g], own & 1))) break;
                if (idle) {
                    if (lane == 0) tc::bar_arrive(tc::smem(&bars.p_ready[g]));
                    ++own;
                    continue;
                }
                tc::fence_after();
                float x[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tc::tmem_load(mS + c * 32, x[c]);
                tc::tmem_wait_load();
                if (a.neg)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[c][i] = -x[c][i];
                const int t = first + (step ? j >> 1 : j);
                if (t >= tails) {
                    const int d = t * kTile - s.L;   // node of the tile's first key
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int at = d + 32 * c, w = at >> 5;
                        auto word = [&](int k) -> uint32_t {
                            return k < 0 ? ~0u : k == 0 ? v0 : k == 1 ? v1 : k == 2 ? v2 : k == 3 ? v3 : 0u;
                        };
                        const uint32_t see = __funnelshift_r(word(w), word(w + 1), at & 31);
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[c][i] = see >> i & 1 ? x[c][i] : neg_inf();
                    }
                }
                float mx[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 32; i += 2) mx[c] = max3(mx[c], x[c][i], x[c][i + 1]);
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.sL;
                const bool move = top > m + kLazy;
                if (__any_sync(kFull, move)) {
                    const float to = move ? top : m, keep = move ? ex2(m - to) : 1.f;
                    m = to;
                    l *= keep;
                    if (j >= 2) {   // the output so far
                        if (!(ok = wait_warp(&bars.pv_done[g], (own + 1) & 1))) break;
                        tc::fence_after();
#pragma unroll 1
                        for (int c = 0; c < DP / 32; ++c) {
                            float o[32];
                            tc::tmem_load(tO[g] + row_lane + c * 32, o);
                            tc::tmem_wait_load();
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] *= keep;
                            tc::tmem_store(tO[g] + row_lane + c * 32, o);
                        }
                        tc::tmem_wait_store();
                    }
                }
                const float ref = m == neg_inf() ? 0.f : m;
                const float2 scale = make_float2(a.sL, a.sL), minus = make_float2(-ref, -ref);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t p[16];
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        float2 e = __ffma2_rn(make_float2(x[c][i], x[c][i + 1]), scale, minus);
                        e.x = ex2(e.x);
                        e.y = ex2(e.y);
                        sum[c & 1] = __fadd2_rn(sum[c & 1], e);
                        p[i / 2] = Half<T>::pack(e.x, e.y);
                    }
                    tc::tmem_store16(mS + c * 16, p);
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                tc::tmem_wait_store();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) tc::bar_arrive(tc::smem(&bars.p_ready[g]));
                ++own;
            }
            if (!ok) break;
            other += (jobs + g) / 2;   // (stream 0 has the odd one)
            // ---- the segment's output ---------------------------------------------------------
            const bool two = s.act == 2, both = !two && jobs > 1;
            if (both || two || g == 0) {
                if (!(ok = wait_warp(&bars.pv_done[g], (own + 1) & 1))) break;
            }
            if (!two) {
                if ((g == 1 || both) && !(ok = wait_warp(&bars.pv_done[g ^ 1], (other + 1) & 1))) break;
                sh.ml[g][r] = make_float2(m, l);
                __syncwarp();
                if (lane == 0) tc::bar_arrive(tc::smem(&bars.merge));
                if (!(ok = wait_warp(&bars.merge, merges++ & 1))) break;
            }
            tc::fence_after();
            // one tile: both warpgroups take half of the columns of both streams' outputs
            float w0 = 1.f, w1 = 0.f;
            if (!two) {
                const float2 m0 = sh.ml[0][r], m1 = sh.ml[1][r];
                m = fmaxf(m0.x, m1.x);
                const float ref = m == neg_inf() ? 0.f : m;
                w0 = ex2(m0.x - ref);
                w1 = both ? ex2(m1.x - ref) : 0.f;
                l = m0.y * w0 + (both ? m1.y * w1 : 0.f);
            }
            const bool whole = s.t0 == 0 && s.t1 == s.tiles;
            const float inv = whole ? (l != 0.f ? 1.f / l : 0.f) : 1.f;
            w0 *= inv;
            w1 *= inv;
            uint32_t bad[4] = {0, 0, 0, 0};
            if (s.t1 == s.tiles) {
                const uint32_t *f = sh.bad[segs % kSegRing];
                bad[0] = f[0] & v0;
                bad[1] = f[1] & v1;
                bad[2] = f[2] & v2;
                bad[3] = f[3] & v3;
            }
            const bool spoilt = (bad[0] | bad[1] | bad[2] | bad[3]) != 0;
            const int c0 = two ? 0 : g * (DP / 64), c1 = two ? DP / 32 : c0 + DP / 64;
            const int hq = s.h * a.G + r % a.G;
            const long long row = ((long long)s.b * a.N + node) * a.Hq + hq;
            const long long slot = ((long long)me * 2 + (s.t0 == 0 ? 1 : 0)) * 2 + (two ? g : 0);
#pragma unroll 1
            for (int c = idle ? c1 : c0; c < c1; ++c) {
                float o[32];
                tc::tmem_load(tO[two ? g : 0] + row_lane + c * 32, o);
                tc::tmem_wait_load();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] *= w0;
                if (both) {
                    float q[32];
                    tc::tmem_load(tO[1] + row_lane + c * 32, q);
                    tc::tmem_wait_load();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = fmaf(q[i], w1, o[i]);
                }
                if (!real) continue;
                if (spoilt) {
#pragma unroll 1
                    for (int j = 0; j < a.N; ++j) {
                        const uint32_t bits = j < 32 ? bad[0] : j < 64 ? bad[1] : j < 96 ? bad[2] : bad[3];
                        if (!(bits >> (j & 31) & 1)) continue;
                        const int key = s.L + j, p = a.table[(long long)s.b * a.M + key / a.page];
                        if (p < 0 || p >= a.P) continue;
                        const unsigned short *v = static_cast<const unsigned short *>(a.v) + p * a.vs[0] + key % a.page * a.vs[1] +
                                                  s.h * a.vs[2] + c * 32;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (c * 32 + i < a.D && (v[i] & Half<T>::kExp) == Half<T>::kExp) o[i] += Half<T>::value(v[i]);
                    }
                }
                if (whole) {
                    uint4 *to = reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + row * a.D + c * 32);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (c * 32 + i * 8 < a.D)
                            to[i] = make_uint4(Half<T>::pack(o[8 * i], o[8 * i + 1]), Half<T>::pack(o[8 * i + 2], o[8 * i + 3]),
                                               Half<T>::pack(o[8 * i + 4], o[8 * i + 5]), Half<T>::pack(o[8 * i + 6], o[8 * i + 7]));
                } else {
                    float4 *to = a.part_o + (slot * (DP / 4) + c * 8) * kTile + r;   // (a warp's rows side by side)
#pragma unroll
                    for (int i = 0; i < 8; ++i) to[i * kTile] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                }
            }
            if (real && (two || g == 0)) {
                if (!whole) a.part_ml[slot * kTile + r] = make_float2(m, l);
                else if (a.lse) a.lse[row] = l != 0.f ? sv::kLn2 * (m + log2f(l)) : neg_inf();
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::bar_arrive(tc::smem(&bars.o_free));
            ++segs;
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 1) tc::tmem_free(tmem, 512);
}

// The pieces of what was cut: CTA x joins what begins in CTA x's part and ends in another's. A
// thread per row and four columns, eight rows side by side; the pieces' references
// first, then their outputs.
constexpr int kJoinRows = 8;

template <typename T, int DC>
__global__ void __launch_bounds__(DC * 16 * kJoinRows) join_kernel(const __grid_constant__ AttendArgs a) {
    constexpr int DP = DC * 64;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 join = a.joins[blockIdx.x];
    if (join.x < 0) return;
    const int rr = blockIdx.y * kJoinRows + threadIdx.x % kJoinRows, c4 = threadIdx.x / kJoinRows;
    const int used = a.nodes * a.G, m_tile = rr / used, r = rr - m_tile * used;   // (rows of a tile that are used)
    const int node = (2 * join.z + m_tile) * a.nodes + r / a.G;
    int L, count;
    sequence(a, join.x, L, count);
    if (m_tile > 1 || node >= count) return;
    const int first = blockIdx.x, pieces = join.w - first + 1;
    auto slot = [&](int i) { return ((long long)(first + i) * 2 + (i == 0 ? 1 : 0)) * 2 + m_tile; };
    float m = neg_inf(), l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int U = 16;   // pieces whose loads are in flight together
    for (int i0 = 0; i0 < pieces; i0 += U) {
        float2 ml[U];
        float4 v[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (i0 + i < pieces) {
                ml[i] = a.part_ml[slot(i0 + i) * kTile + r];
                v[i] = a.part_o[(slot(i0 + i) * (DP / 4) + c4) * kTile + r];
            }
        }
        float to = m;
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (i0 + i < pieces) to = fmaxf(to, ml[i].x);
        const float ref = to == neg_inf() ? 0.f : to, keep = ex2(m - ref);
        m = to;
        l *= keep;
        o.x *= keep;
        o.y *= keep;
        o.z *= keep;
        o.w *= keep;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (i0 + i < pieces) {
                const float w = ex2(ml[i].x - ref);
                l = fmaf(ml[i].y, w, l);
                o.x = fmaf(v[i].x, w, o.x);
                o.y = fmaf(v[i].y, w, o.y);
                o.z = fmaf(v[i].z, w, o.z);
                o.w = fmaf(v[i].w, w, o.w);
            }
        }
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    const long long row = ((long long)join.x * a.N + node) * a.Hq + join.y * a.G + r % a.G;
    if (c4 * 4 < a.D)
        *reinterpret_cast<uint2 *>(static_cast<T *>(a.out) + row * a.D + c4 * 4) =
            make_uint2(Half<T>::pack(o.x * inv, o.y * inv), Half<T>::pack(o.z * inv, o.w * inv));
    if (c4 == 0 && a.lse) a.lse[row] = l != 0.f ? sv::kLn2 * (m + log2f(l)) : neg_inf();
}

static bool overlap(const void *a, int64_t na, const void *b, int64_t nb) {
    const char *x = static_cast<const char *>(a), *y = static_cast<const char *>(b);
    return na > 0 && nb > 0 && x < y + nb && y < x + na;
}

static int check_attend(const spec_attend_params *p) {
    if (!p) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "params is NULL");
    if (p->B < 0 || p->N < 0 || p->M < 0 || p->P < 0)
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "tree_attention: B, N, M and P must be >= 0");
    if (p->dtype != SPEC_BF16 && p->dtype != SPEC_F16)
        return spec_internal_set_error(SPEC_ERR_UNSUPPORTED, "tree_attention: dtype must be bf16 or f16");
    if (p->B > 65535 || p->N > SPEC_MAX_NODES || p->P > (1 << 30))
        return spec_internal_set_error(SPEC_ERR_UNSUPPORTED, "tree_attention: B, N or P out of range");
    if (p->Hkv < 1 || p->Hq < 1 || p->Hq % p->Hkv)
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "tree_attention: Hq must be a multiple of Hkv");
    if (p->Hq / p->Hkv > 128 || p->Hq > 65535)
        return spec_internal_set_error(SPEC_ERR_UNSUPPORTED, "tree_attention: too many heads");
    if (p->D < 8 || p->D > 128 || p->D % 8)
        return spec_internal_set_error(SPEC_ERR_UNSUPPORTED, "tree_attention: D must be a multiple of 8 in [8, 128]");
    if (p->page < 8 || p->page > (1 << 20) || (p->page & (p->page - 1)))
        return spec_internal_set_error(SPEC_ERR_UNSUPPORTED, "tree_attention: page must be a power of two in [8, 2^20]");
    if ((int64_t)p->M * p->page > INT32_MAX - 1024 || (int64_t)p->B * p->N * p->Hq > (1 << 30))
        return spec_internal_set_error(SPEC_ERR_UNSUPPORTED, "tree_attention: rows too long or too many");
    if (!(p->scale >= -1e30f && p->scale <= 1e30f))
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "tree_attention: scale must be finite");
    if (p->parents_stride < 0 || (p->parents_stride > 0 && p->parents_stride < p->N) || p->parents_stride > (1LL << 40))
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "tree_attention: parents_stride must be 0 or >= N");
    const int64_t n[3][3] = {{p->B, p->N, p->Hq}, {p->P, p->page, p->Hkv}, {p->P, p->page, p->Hkv}};
    const int64_t *s[3] = {p->q_stride, p->k_stride, p->v_stride};
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < 3; ++j)
            if (n[i][j] > 1 && (s[i][j] <= 0 || s[i][j] % 8 || s[i][j] >= (1LL << 38) || s[i][j] > (INT64_MAX >> 4) / n[i][j]))
                return spec_internal_set_error(SPEC_ERR_INVALID_ARG,
                                               "tree_attention: strides must be multiples of 8 elements, above 0 and below 2^38");
    return SPEC_OK;
}

// ---- launch --------------------------------------------------------------------------------

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                             const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeFn encoder() {
    static const EncodeFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// [n3][n2][n1][D] of 16-bit elements, boxes of 64 elements x b1 x b2
static bool encode(CUtensorMap *map, int bf16, const void *base, int D, const int *n, const int64_t *stride, int b1, int b2) {
    const EncodeFn fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)n[2], (cuuint64_t)n[1], (cuuint64_t)n[0]};
    cuuint64_t st[3];
    for (int i = 0; i < 3; ++i) st[i] = n[2 - i] > 1 ? (cuuint64_t)stride[2 - i] * 2 : (cuuint64_t)(D * 2 + 15) / 16 * 16;
    const cuuint32_t box[4] = {64, (cuuint32_t)b1, (cuuint32_t)b2, 1}, one[4] = {1, 1, 1, 1};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void *>(base), dims, st, box,
              one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return n;
}

constexpr int kMaxCtas = 152;   // one per SM; the workspace's room

static size_t part_floats(int D) { return (size_t)kMaxCtas * 4 * kTile * (D > 64 ? 128 : 64); }
static size_t workspace_bytes_for(const spec_attend_params *p) {
    return part_floats(p->D) * 4 + (size_t)kMaxCtas * 4 * kTile * 8 + (size_t)kMaxCtas * 16;
}

template <typename T, int DC>
static cudaError_t launch_attend(const AttendArgs &a, const CUtensorMap *maps, int box, cudaStream_t st) {
    constexpr size_t smem = AttendSmem<DC>::kTiles + sizeof(AttendShared<AttendSmem<DC>::kStages>);
    static_assert(smem <= 227 * 1024, "shared memory");
    static std::mutex mu;
    static bool done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!done[dev & 63]) {
            e = cudaFuncSetAttribute(attend_kernel<T, DC>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess) return e;
            done[dev & 63] = true;
        }
    }
    int ctas = sm_count();
    if (ctas < 1) return cudaErrorUnknown;
    if (ctas > kMaxCtas) ctas = kMaxCtas;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kNT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, attend_kernel<T, DC>, a, maps[0], maps[1], maps[2], box);
    if (e != cudaSuccess) return e;
    const int tiles = (a.N + a.nodes - 1) / a.nodes, rows = tiles > 1 ? 2 * a.nodes * a.G : a.N * a.G;
    cfg.gridDim = dim3(ctas, (rows + kJoinRows - 1) / kJoinRows);
    cfg.blockDim = dim3(DC * 16 * kJoinRows);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, join_kernel<T, DC>, a);
}

}  // namespace sr

extern "C" size_t spec_tree_attention_workspace_size(const spec_attend_params *p) {
    return sr::check_attend(p) == SPEC_OK ? sr::workspace_bytes_for(p) : 0;
}

extern "C" int spec_tree_attention(const spec_attend_params *p, const void *q, const void *k, const void *v,
                                   const int32_t *table, const int32_t *lengths, const int32_t *parents,
                                   const int32_t *counts, void *out, float *lse, void *workspace,
                                   size_t workspace_bytes, int32_t *status, void *stream) {
    using namespace sr;
    const int rc = check_attend(p);
    if (rc != SPEC_OK) return rc;
    if (p->B == 0 || p->N == 0) return spec_internal_set_error(SPEC_OK, "");
    if (!q || !lengths || !out || (p->M && !table) || (p->P && (!k || !v)))
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "tree_attention: an argument is NULL");
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
         reinterpret_cast<uintptr_t>(out)) % 16)
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "tree_attention: q, k, v and out must be 16-byte aligned");
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16 || workspace_bytes < spec_tree_attention_workspace_size(p))
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "tree_attention: workspace missing, too small or misaligned");
    {
        const int64_t n[3][3] = {{p->B, p->N, p->Hq}, {p->P, p->page, p->Hkv}, {p->P, p->page, p->Hkv}};
        const int64_t *s[3] = {p->q_stride, p->k_stride, p->v_stride};
        const void *in[3] = {q, k, v};
        const int64_t rows = (int64_t)p->B * p->N * p->Hq;
        const void *to[3] = {out, lse, workspace};
        const int64_t size[3] = {rows * p->D * 2, lse ? rows * 4 : 0, (int64_t)workspace_bytes};
        for (int i = 0; i < 3; ++i) {
            int64_t last = 0;
            for (int j = 0; j < 3; ++j) last += n[i][j] > 1 ? (n[i][j] - 1) * s[i][j] : 0;
            for (int o = 0; o < 3; ++o)
                if (n[i][0] > 0 && overlap(to[o], size[o], in[i], (last + p->D) * 2))
                    return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "tree_attention: an output overlaps an input");
        }
        if (overlap(out, size[0], lse, size[1]) || overlap(out, size[0], workspace, size[2]) || overlap(lse, size[1], workspace, size[2]))
            return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "tree_attention: outputs overlap");
    }
    spec_internal_set_error(SPEC_OK, "");
    const int G = p->Hq / p->Hkv;
    AttendArgs a{};
    a.v = v;
    a.table = table;
    a.lengths = lengths;
    a.parents = parents;
    a.counts = counts;
    a.out = out;
    a.lse = lse;
    a.status = status;
    a.part_o = static_cast<float4 *>(workspace);
    a.part_ml = reinterpret_cast<float2 *>(static_cast<float *>(workspace) + part_floats(p->D));
    a.joins = reinterpret_cast<int4 *>(a.part_ml + (size_t)kMaxCtas * 4 * kTile);
    a.B = p->B;
    a.N = p->N;
    a.Hq = p->Hq;
    a.Hkv = p->Hkv;
    a.G = G;
    a.D = p->D;
    a.P = p->P;
    a.page = p->page;
    a.M = p->M;
    a.fill = counts != nullptr || (int64_t)p->M * p->page < p->N;
    a.nodes = kTile / G;
    a.sL = fmaxf(fabsf(p->scale) * sv::kLog2e, FLT_MIN);   // (0 times a masked key's -inf would be NaN)
    a.neg = p->scale < 0.f;
    a.ps = p->parents_stride;
    for (int j = 0; j < 3; ++j) a.vs[j] = p->v_stride[j];
    const int nq[3] = {p->B, p->N, p->Hq}, nk[3] = {p->P > 0 ? p->P : 1, p->page, p->Hkv}, box = p->page < 64 ? p->page : 64;
    const int bf16 = p->dtype == SPEC_BF16;
    const int64_t none[3] = {0, 0, 0};
    CUtensorMap maps[3];
    const int empty[3] = {1, 1, 1};
    if (!encode(&maps[0], bf16, q, p->D, nq, p->q_stride, G, a.nodes) ||
        !encode(&maps[1], bf16, p->P ? k : q, p->D, p->P ? nk : empty, p->P ? p->k_stride : none, 1, box) ||
        !encode(&maps[2], bf16, p->P ? v : q, p->D, p->P ? nk : empty, p->P ? p->v_stride : none, 1, box))
        return spec_internal_set_error(SPEC_ERR_CUDA, "tree_attention: the copies' layout could not be encoded");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (p->D > 64) e = bf16 ? launch_attend<__nv_bfloat16, 2>(a, maps, box, st) : launch_attend<__half, 2>(a, maps, box, st);
    else e = bf16 ? launch_attend<__nv_bfloat16, 1>(a, maps, box, st) : launch_attend<__half, 1>(a, maps, box, st);
    return e == cudaSuccess ? SPEC_OK : spec_internal_set_error(SPEC_ERR_CUDA, cudaGetErrorString(e));
}

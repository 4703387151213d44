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
// Measured (in a graph; bf16, 8 key heads of 128): 64 sequences of up to 8192 tokens, 9 nodes
// of 32 heads, 1.37 GB: 224 us, 6.1 TB/s, 0.90 of a copy's rate; one token for 256 sequences of up
// to 4096: 416 us, 6.5 TB/s. 8 sequences of up to 32768, 64 nodes of 64 heads, 0.37 TFLOP: 292 to 298 us, 1.25
// PFLOP/s (319 in runs so long that the power cap holds); there a job's products take 1440 of the 1800 cycles between two streams' turns (scores
// read both operands from shared memory, at its full rate). One token over 2048: 12 us.
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

extern "C" unsigned spec_internal_wait_limit(void);   // (spec_verify.cu)

namespace sr {

constexpr int kTile = 128;             // keys a tile, and rows a tile
constexpr int kChunk = kTile * 128;    // bytes of 64 elements of a tile's rows
constexpr int kNT = 512;               // warps 0-3 and 12-15 copies and products, 4-7 and 8-11 the streams' softmax
constexpr int kWarpK = 0, kWarpV = 3, kWarpGo = 2, kWarpMma0 = 1, kWarpMma1 = 14;   // (spread over the four schedulers)
constexpr unsigned kDrain = 1u << 20;  // polls for what is in flight at the end
constexpr int kSegRing = 4;            // segments whose flags of non-finite values are kept
constexpr float kLazy = 8.f;           // a row's reference moves when its maximum is 2^8 above it
constexpr float kFarRef = 4096.f;      // (log2) references from which their rounding counts

struct AttendArgs {
    const void *v;
    const int32_t *table, *lengths, *parents, *counts;
    void *out;
    float *lse;
    int32_t *status;
    float4 *part_o;   // [CTA][2][tile][D padded / 4][row]: unnormalised outputs of a sequence's pieces
    float2 *part_ml;  // [CTA][2][tile][row]: their reference score and sum
    int4 *joins;      // [CTA], what begins here and ends elsewhere: sequence (-1: none), head + pair of tiles 2^16, rows, last CTA
    int B, N, Hq, Hkv, G, D, P, page, M, fill;
    int nodes, q_rows;   // a tile, and the rows that a copy of queries brings
    float sL;         // |scale| log2 e
    float lazy;       // kLazy as a difference of scores
    unsigned spin;    // polls of a wait before it gives up
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

// Probabilities are rounded to the inputs' type before they multiply the values, which is what the
// tensor cores take (in fp32 they would have to be split in two, and the product done twice); the sum
// takes them unrounded. A row's reference lies kUp below its maximum (in log2): in fp16 what is
// smaller than 2^-14 loses bits and below 2^-25 everything, so that a long context behind one large
// score would vanish (32767 keys 17 nats below it: their part of the output 44% off, at 18 nats gone; with
// 2^7 times the probabilities 0.1% and 0.9% off). bf16 has fp32's exponents.
template <typename T>
struct Half;
template <>
struct Half<__nv_bfloat16> {
    static constexpr int kBf16 = 1;
    static constexpr uint32_t kExp = 0x7f80;
    static constexpr float kUp = 0.f;
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
    static constexpr float kUp = 7.f;   // (with kLazy: probabilities reach 2^15, and fp16 65504)
    __device__ static __forceinline__ uint32_t pack(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    __device__ static __forceinline__ float value(uint32_t h) { return __half2float(__ushort_as_half((unsigned short)h)); }
};

// A row's sums stand against a reference score mr that its maximum once was. In log2 that is m = mr sL - kUp,
// rounded, and where all use the same m its rounding cancels. But it is half a step of m, which
// beside scores of 2^30 is more than a probability's range: from kFarRef on probabilities and weights are
// taken from differences of scores. Such tiles are read a second time (8 x 64 nodes of 32k 364 us
// in place of 297, 64 x 9 231 and 229 in eager calls); all others take the same time within 1%.
template <typename T>
__device__ __forceinline__ float log2_of(const AttendArgs &a, float mr) {   // (rounded here, whatever it is added to)
    return Half<T>::kUp == 0.f ? __fmul_rn(mr, a.sL) : __fmaf_rn(mr, a.sL, -Half<T>::kUp);
}
struct Reference {
    float base, minus;   // a score's exponent is (score - base) sL + minus
    bool far;
};
template <typename T>
__device__ __forceinline__ Reference reference(const AttendArgs &a, float mr) {
    const float at = mr == neg_inf() ? 0.f : mr, m = log2_of<T>(a, at);   // (-inf: nothing seen)
    Reference r;
    r.far = fabsf(m) > kFarRef && at < INFINITY;
    r.base = r.far ? at : 0.f;
    r.minus = r.far ? Half<T>::kUp : -m;
    return r;
}
// the weight of sums against `from` among those against r, which is no smaller
template <typename T>
__device__ __forceinline__ float weight(const AttendArgs &a, float from, const Reference &r) {
    return ex2(__fadd_rn(log2_of<T>(a, from - r.base), r.minus));
}

// pairs of row tiles that `count` nodes fill
__device__ __forceinline__ int pairs_of(const AttendArgs &a, int count) {
    return a.N <= 2 * a.nodes ? count > 0 : (count + 2 * a.nodes - 1) / (2 * a.nodes);
}

// (a 64-bit division costs ten times a 32-bit one)
__device__ __forceinline__ long long quotient(long long x, long long y) {
    return ((x | y) >> 32) == 0 ? (long long)((uint32_t)x / (uint32_t)y) : x / y;
}

// One piece of a CTA's work, tiles [t0, t1) of `tiles` of (b, h, pair), and what is left behind
// it. Every warp walks the CTA's segments by itself; its place stands in shared memory,
// which leaves registers to what the warp does.
struct Segment {
    int b, h, pair, t0, t1, tiles, L, count;
    int act, begun;         // row tiles with nodes; 1: next() is to give this piece itself
    int off, left;          // units of sequence b behind this piece, and of the CTA's part (below 2^31, the host checks)
    __device__ __forceinline__ int keys(int t) const { return min(kTile, L + count - t * kTile); }
    // the piece that begins at unit `off` of sequence b, of L tokens and `count` nodes
    __device__ __forceinline__ bool begin(const AttendArgs &a) {
        const int pairs = pairs_of(a, count);
        tiles = (L + count + kTile - 1) / kTile;
        const int head = pairs * tiles;
        if (off >= head * a.Hkv) return false;
        h = (int)((unsigned)off / (unsigned)head);
        const int in = off - h * head;
        pair = pairs > 1 ? in / tiles : 0;
        t0 = in - pair * tiles;
        t1 = t0 + min(tiles - t0, left);
        act = count - pair * 2 * a.nodes > a.nodes ? 2 : 1;
        off += t1 - t0;
        left -= t1 - t0;
        return true;
    }
    __device__ __forceinline__ bool next(const AttendArgs &a) {
        if (begun) {
            begun = 0;
            return true;
        }
        Segment s = *this;
        while (s.left > 0) {
            if (s.begin(a)) {
                *this = s;
                return true;
            }
            s.off -= s.tiles * pairs_of(a, s.count) * a.Hkv;
            ++s.b;
            sequence(a, s.b, s.L, s.count);
        }
        return false;
    }
};

// behind the tiles in shared memory
template <int SK, int SV>
struct AttendShared {
    struct {
        uint64_t k_full[SK], k_empty[SK], v_full[SV], v_empty[SV], s_full[2], p_ready[2], pv_done[2], turn[2], q_full[2], q_empty[2], start[2], o_free, merge, drain;
    } bars;
    float2 ml[2][kTile];
    Segment seg[13];   // of warps 0-11 and 14
    uint32_t tmem, bad[kSegRing][4];
    int abort;
};

// FEW: at most 64 rows a sequence and key head (one tile): 64 x 9 nodes of 36 rows take 224 us, 232
// without it, 256 x 1 415 and 431, and 32 x 1 with heads of 64 25.7 and 27.0. Their queries take a quarter of the
// room of two tiles of 128 (the products read what lies behind them, for rows that nobody uses), which
// leaves another stage to the rings.
template <int DC, bool FEW>
struct AttendSmem {
    static constexpr int kStage = DC * kChunk;
    static constexpr int kQChunk = FEW ? kChunk / 2 : kChunk;   // 64 elements of the rows of a tile
    static constexpr int kQ = 2 * DC * kQChunk;
    static constexpr int kKeys = DC == 2 ? 3 : FEW ? 6 : 5, kValues = DC == 2 ? FEW ? 3 : 2 : FEW ? 6 : 5;   // stages of the rings
    using Shared = AttendShared<kKeys, kValues>;
    static constexpr int kTiles = kQ + (kKeys + kValues) * kStage;
};

template <typename T, int DC, bool FEW>
__global__ void __launch_bounds__(kNT, 1)
    attend_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ CUtensorMap qmap,
                  const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, int box) {
    using SM = AttendSmem<DC, FEW>;
    constexpr int SK = SM::kKeys, SV = SM::kValues, DP = DC * 64;
    extern __shared__ __align__(1024) char dyn[];   // (the kernel has no other shared memory, so that this holds)
    typename SM::Shared &sh = *reinterpret_cast<typename SM::Shared *>(dyn + SM::kTiles);
    auto &bars = sh.bars;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = tc::smem(dyn), kring = base + SM::kQ, vring = kring + SK * SM::kStage;
    if (threadIdx.x == 0) {
        sh.abort = 0;
        for (int i = 0; i < SK; ++i) {
            tc::bar_init(tc::smem(&bars.k_full[i]), 1);
            tc::bar_init(tc::smem(&bars.k_empty[i]), 2);   // the streams' products
        }
        for (int i = 0; i < SV; ++i) {
            tc::bar_init(tc::smem(&bars.v_full[i]), 1);
            tc::bar_init(tc::smem(&bars.v_empty[i]), 2);
        }
        for (int i = 0; i < 2; ++i) {
            tc::bar_init(tc::smem(&bars.s_full[i]), 1);
            tc::bar_init(tc::smem(&bars.p_ready[i]), 5);   // four warps, and the copies that the job needs
            tc::bar_init(tc::smem(&bars.pv_done[i]), 1);
            tc::bar_init(tc::smem(&bars.turn[i]), 1);
            tc::bar_init(tc::smem(&bars.q_full[i]), 1);
            tc::bar_init(tc::smem(&bars.q_empty[i]), 2);
            tc::bar_init(tc::smem(&bars.start[i]), 1);
        }
        tc::bar_init(tc::smem(&bars.o_free), 10);          // the softmax's warps and, to keep them in step, the products'
        tc::bar_init(tc::smem(&bars.merge), 8);
        tc::bar_init(tc::smem(&bars.drain), 2);
        tc::fence_barrier_init();
        tc::prefetch_map(&kmap);
        tc::prefetch_map(&qmap);
        tc::prefetch_map(&vmap);
    }
    if (warp == kWarpMma0) tc::tmem_alloc(tc::smem(&sh.tmem), 512);
    // (so far nothing that an earlier kernel of the stream may write has been read)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const int G = gridDim.x, me = blockIdx.x;
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

    // ---- which part of the line is this CTA's: every warp finds it by itself --------------------
    const bool works = warp < 12 || warp == kWarpMma1;
    Segment &s = sh.seg[min(warp, 12)];
    long long per = 1, u0 = 0;
    if (works) {
        // lane l: the units of sequences [l, l + 1) run
        const int run = (a.B + 31) >> 5, b_lo = min(a.B, lane * run), b_hi = min(a.B, b_lo + run);
        auto units = [&](int b, int &L, int &count) -> long long {
            sequence(a, b, L, count);
            return (long long)(a.Hkv * pairs_of(a, count)) * ((L + count + kTile - 1) / kTile);
        };
        long long mine = 0;
        int L, count;
#pragma unroll 8
        for (int b = b_lo; b < b_hi; ++b) mine += units(b, L, count);
        long long upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const long long v = __shfl_up_sync(kFull, upto, o);
            if (lane >= o) upto += v;
        }
        const long long total = __shfl_sync(kFull, upto, 31);
        per = quotient(total + G - 1, G);
        u0 = min(total, me * per);
        const long long u1 = min(total, u0 + per);
        if (lane == 0) s.left = s.begun = 0;
        __syncwarp();
        if (u0 < u1 && u0 >= upto - mine && u0 < upto) {
            long long at = upto - mine;
            for (int b = b_lo; b < b_hi; ++b) {
                const long long n = units(b, L, count);
                if (u0 < at + n) {
                    Segment first;
                    first.b = b;
                    first.L = L;
                    first.count = count;
                    first.off = (int)(u0 - at);
                    first.left = (int)(u1 - u0);
                    first.begin(a);
                    first.begun = 1;
                    s = first;
                    break;
                }
                at += n;
            }
        }
    }
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
        for (unsigned i = 0; i < a.spin; ++i) {
            if (__all_sync(kFull, tc::bar_try(addr, parity))) return true;
            if (__any_sync(kFull, *(volatile int *)&sh.abort)) return false;
        }
        *(volatile int *)&sh.abort = 1;
        raise_status(a.status, SPEC_ERR_TIMEOUT);
        return false;
    };

    // where one tile holds all nodes' rows, the queries' room for two holds the next segment's, too
    const bool twin = FEW || a.N <= a.nodes;

    // 128 registers a thread at the launch: 64 for eight warps and 192 for the eight of the softmax
    if (warp < 4 || warp >= 12) {
        tc::fewer_registers<64>();
        if (warp == kWarpK || warp == kWarpV) {
            // ---- copies: queries and keys, and values ------------------------------------------------
            // A ring of stages each, so that every ring is filled and waited for in one order.
            const bool keys = warp == kWarpK;
            const CUtensorMap *map = keys ? &kmap : &vmap;
            uint64_t *const full = keys ? bars.k_full : bars.v_full, *const empty = keys ? bars.k_empty : bars.v_empty;
            const unsigned S = keys ? SK : SV;
            const uint32_t ring = keys ? kring : vring;
            const int bpt = kTile / box, group = 32 / bpt;   // boxes a tile; tiles whose pages the lanes hold (powers of two)
            const int page_bits = 31 - __clz(a.page);
            unsigned n = 0, segs = 0;
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
                auto queries = [&]() -> bool {
                    const unsigned slot = twin ? segs & 1 : 0, use = twin ? segs >> 1 : segs;
                    if (use > 0 && !wait_warp(&bars.q_empty[slot], (use + 1) & 1)) return false;
                    if (lane == 0) {
                        const uint32_t bar = tc::smem(&bars.q_full[slot]);
                        tc::bar_expect(bar, (uint32_t)a.q_rows * 128 * DC * s.act);
                        for (int m = 0; m < s.act; ++m)
                            for (int x = 0; x < DC; ++x)
                                tc::load_tile(base + ((slot + m) * DC + x) * SM::kQChunk, &qmap, bar, x * 64, head * a.G, (2 * s.pair + m) * a.nodes, s.b);
                    }
                    __syncwarp();
                    ++segs;
                    return true;
                };
                int now = pages(0), next = pages(group);
                const bool first = twin || segs == 0;   // (else the first keys need not wait for the queries' place)
                if (keys && first && !(ok = queries())) break;
                for (int t = 0; ok && t < nt; ++t, ++n) {
                    if (t && (t & (group - 1)) == 0) {
                        now = next;
                        next = pages(t + group);
                    }
                    const unsigned st = n % S;
                    if (n >= S && !(ok = wait_warp(&empty[st], (n / S + 1) & 1))) break;
                    const int boxes = (min(kTile, end - (t0 + t) * kTile) + box - 1) / box;
                    const uint32_t bar = tc::smem(&full[st]), dst = ring + st * SM::kStage;
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
                    if (keys && !first && t == min(nt, ahead) - 1) ok = queries();
                }
            }
            // no copy may still be in flight when the CTA ends, whether or not another role has given up
            for (unsigned i = n > S ? n - S : 0; i < n; ++i)
                for (unsigned k = 0; k < kDrain && !tc::bar_try(tc::smem(&full[i % S]), (i / S) & 1); ++k) {}
            for (unsigned i = segs > (twin ? 1 : 0) ? segs - (twin ? 2 : 1) : 0; keys && i < segs; ++i)
                for (unsigned k = 0; k < kDrain && !tc::bar_try(tc::smem(&bars.q_full[twin ? i & 1 : 0]), (twin ? i >> 1 : i) & 1); ++k) {}
        } else if (warp == kWarpGo) {
            // ---- what a job needs: its copies are there, and its values can be multiplied --------------
            // This warp alone waits for the copies, in their order, and passes a job on when its
            // values and the keys of the stream's next job are there. (A job before on its
            // stream has passed first, so that no barrier gets ahead of its waiters.)
            unsigned kn = 0, vn = 0, segs = 0, sent0 = 0, sent1 = 0;
            int4 join = make_int4(-1, 0, 0, 0);
            long long at_unit = u0;
            bool ok = true;
            auto keys_there = [&]() -> bool {
                const unsigned at = kn++;
                return wait_warp(&bars.k_full[at % SK], (at / SK) & 1);
            };
            auto pass = [&](int g) -> bool {
                const unsigned sent = g ? sent1 : sent0;
                if (sent > 0 && !wait_warp(&bars.p_ready[g], (sent + 1) & 1)) return false;
                if (lane == 0) tc::bar_arrive(tc::smem(&bars.p_ready[g]));
                if (g) ++sent1;
                else ++sent0;
                return true;
            };
            while (ok && next_segment()) {
                const int nt = s.t1 - s.t0, two = s.act == 2, ahead = two ? 1 : 2, tails = s.L / kTile - s.t0;
                if (s.t0 == 0 && s.t1 < s.tiles)
                    join = make_int4(s.b, s.h | s.pair << 16, (s.count - 2 * s.pair * a.nodes) * a.G, (int)quotient(at_unit + s.tiles - 1, per));
                at_unit += nt;
                uint32_t *bad = sh.bad[segs % kSegRing];
                if (lane < 4) bad[lane] = 0;
                const unsigned slot = twin ? segs & 1 : 0;
                ok = wait_warp(&bars.q_full[slot], (twin ? segs >> 1 : segs) & 1);
                for (int t = 0; ok && t < min(nt, ahead); ++t) ok = keys_there();
                if (!ok) break;
                if (lane == 0) tc::bar_arrive(tc::smem(&bars.start[slot]));
                for (int t = 0; t < nt; ++t) {
                    const unsigned st = vn % SV;
                    if (!(ok = wait_warp(&bars.v_full[st], (vn / SV) & 1))) break;
                    ++vn;
                    if (t >= tails) {
                        const int at0 = (s.t0 + t) * kTile, keys = s.keys(s.t0 + t), lo = max(0, s.L - at0);
                        char *stage = dyn + SM::kQ + (SK + st) * SM::kStage;
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
                    }
                    if (t + ahead < nt && !(ok = keys_there())) break;
                    if (!(ok = pass(two ? 0 : t & 1))) break;
                    if (two && !(ok = pass(1))) break;
                }
                ++segs;
            }
            if (lane == 0) a.joins[me] = join;
        } else if (warp == kWarpMma0 || warp == kWarpMma1) {
            // ---- products, a warp per stream -------------------------------------------------------
            // (With one warp the tensor cores paused while it prepared the other stream's job.) Two tiles' streams take
            // turns, so that one's products run while the other exponentiates (8 x 64 nodes of 32k take 4%
            // more without); streams of one tile are faster without (32 x 1 with heads of 64 take 5% more with
            // turns, 44 x 3 with heads of 40 6%). The
            // whole warp walks along, so that operands stay in uniform registers; one thread issues.
            const bool lead = tc::elect();
            const int g = warp == kWarpMma1;
            const uint32_t S_ = tc::uniform(tS[0] + g * 128), O_ = tc::uniform(tO[0] + g * DP);
            unsigned n0 = 0, segs = 0, done = 0, turns = 0;
            auto my_turn = [&]() -> bool {   // (stream 0 begins)
                const unsigned i = turns++;
                return g ? wait_warp(&bars.turn[1], i & 1) : i == 0 || wait_warp(&bars.turn[0], (i + 1) & 1);
            };
            auto pass_on = [&]() {   // (both have as many jobs)
                if (lead) tc::bar_arrive(tc::smem(&bars.turn[g ^ 1]));
                __syncwarp();
            };
            bool ok = true;
            while (ok && next_segment()) {
                const int two = !FEW && s.act == 2, nt = s.t1 - s.t0, step = two ? 1 : 2;
                const int end_steps = (s.keys(s.t1 - 1) + 15) / 16;   // products of the last tile
                const int slot = twin ? segs & 1 : 0;
                const uint32_t q = tc::uniform(tc::operand_lo(base + (two ? g : slot) * DC * SM::kQChunk, 16));
                // S of tile t
                auto scores = [&](int t) {
                    const unsigned st = (n0 + t) % SK;
                    const uint32_t k = tc::uniform(tc::operand_lo(kring + st * SM::kStage, 16));
                    if (lead) {
#pragma unroll
                        for (int i = 0; i < DC * 4; ++i) {
                            const uint32_t x = (i & 3) * 32;
                            tc::mma_ss(S_, tc::operand(q + (((i >> 2) * SM::kQChunk + x) >> 4)), tc::operand(k + (((i >> 2) * kChunk + x) >> 4)),
                                       kIdS, i > 0);
                        }
                        tc::commit(tc::smem(&bars.s_full[g]));
                        tc::commit(tc::smem(&bars.k_empty[st]));
                        if (!two) tc::commit(tc::smem(&bars.k_empty[st]));   // (for the other stream)
                    }
                    __syncwarp();
                };
                const int first = two ? 0 : g;
                if (!(ok = wait_warp(&bars.start[slot], (twin ? segs >> 1 : segs) & 1))) break;
                tc::fence_after();
                if (first < nt) scores(first);
                if (lead && first + step >= nt) tc::commit(tc::smem(&bars.q_empty[slot]));
                if (segs > 0 && !(ok = wait_warp(&bars.o_free, (segs + 1) & 1))) break;
                for (int t = first; t < nt; t += step) {
                    const unsigned st = (n0 + t) % SV;
                    const uint32_t v = tc::uniform(tc::operand_lo(vring + st * SM::kStage, kChunk));
                    const int steps = t == nt - 1 ? end_steps : kTile / 16;
                    if (!(ok = wait_warp(&bars.p_ready[g], done & 1)) || (two && !(ok = my_turn()))) break;
                    tc::fence_after();
                    if (lead) {
                        if (steps == kTile / 16) {
#pragma unroll
                            for (int i = 0; i < kTile / 16; ++i) tc::mma_ts(O_, S_ + i * 8, tc::operand(v + i * 128), kIdO, t > first || i > 0);
                        } else {
                            for (int i = 0; i < steps; ++i) tc::mma_ts(O_, S_ + i * 8, tc::operand(v + i * 128), kIdO, t > first || i > 0);
                        }
                        tc::commit(tc::smem(&bars.pv_done[g]));
                        tc::commit(tc::smem(&bars.v_empty[st]));
                        if (!two) tc::commit(tc::smem(&bars.v_empty[st]));
                    }
                    __syncwarp();
                    ++done;
                    if (t + step < nt) {
                        scores(t + step);
                        if (lead && t + 2 * step >= nt) tc::commit(tc::smem(&bars.q_empty[slot]));
                    }
                    if (two) pass_on();
                }
                n0 += nt;
                ++segs;
                if (lead) tc::bar_arrive(tc::smem(&bars.o_free));
                __syncwarp();
            }
            // (none of the products may still run when the CTA ends)
            if (lead) {
                tc::commit(tc::smem(&bars.drain));
                for (unsigned k = 0; k < kDrain && !tc::bar_try(tc::smem(&bars.drain), 0); ++k) {}
            }
            __syncwarp();
        }
    } else {
        tc::more_registers<192>();
        // ---- softmax: a stream each, a row a thread ------------------------------------------
        const int g = (warp - 4) >> 2, r = threadIdx.x & 127;
        const uint32_t row_lane = (uint32_t)(warp & 3) << 21;   // (lane of tensor memory in bits 16 and up)
        const uint32_t mS = tS[g] + row_lane;
        const int row_node = r / a.G, row_head = r - row_node * a.G;   // within a tile and a key head's group
        unsigned segs = 0, merges = 0, own = 0;   // (own: jobs of this stream so far)
        bool ok = true;
        for (bool more = next_segment(); ok && more;) {
            const int first = s.t0, step = s.act == 2, tails = s.L / kTile, jobs = (s.t1 - first) << step;
            // what this row sees of the nodes
            const int tile0 = 2 * s.pair + (s.act == 2 ? g : 0), node = tile0 * a.nodes + row_node;
            const bool real = row_node < a.nodes && node < s.count;
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
            // lim: a maximum that is not at or below it is looked at (NaN: each, the reference is far;
            // infinity: none, rows that nobody uses may hold anything). minus: what is added to x sL
            float mr = neg_inf(), l = 0.f, lim = real ? neg_inf() : INFINITY, minus = 0.f;
            for (int j = g; j < jobs; j += 2) {
                if (!(ok = wait_warp(&bars.s_full[g], own & 1))) break;
                if (idle) {
                    if (lane == 0) tc::bar_arrive(tc::smem(&bars.p_ready[g]));
                    ++own;
                    continue;
                }
                tc::fence_after();
                const int t = first + (step ? j >> 1 : j);
                float x[4][32];
                // once, and where a reference is far once more, less the reference
                float base = -0.f;
                for (int again = 0;; again = 1) {
                    asm volatile("" : "+r"(again));   // (one copy of this code)
#pragma unroll
                    for (int c = 0; c < 4; ++c) tc::tmem_load(mS + c * 32, x[c]);
                    tc::tmem_wait_load();
#pragma unroll
                    for (int c = 0; c < 4; ++c) tc::loaded(x[c]);
                    if (a.neg | again) {
                        const float sign = a.neg ? -1.f : 1.f;
                        const float2 sign2 = make_float2(sign, sign), base2 = make_float2(base, base);
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int i = 0; i < 32; i += 2) {
                                const float2 d = __ffma2_rn(make_float2(x[c][i], x[c][i + 1]), sign2, base2);
                                x[c][i] = d.x;
                                x[c][i + 1] = d.y;
                            }
                    }
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
                    if (again) break;
                    float mx[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int i = 0; i < 32; i += 2) mx[c] = max3(mx[c], x[c][i], x[c][i + 1]);
                    const float high = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    const bool look = !(high <= lim);
                    if (!__any_sync(kFull, look)) break;
                    const bool move = look && high > mr;
                    const Reference to = reference<T>(a, move ? high : mr);
                    const float keep = move ? weight<T>(a, mr, to) : 1.f;
                    if (move) {
                        mr = high;
                        lim = to.far ? NAN : mr + a.lazy;
                    }
                    l *= keep;
                    minus = to.minus;
                    if (j >= 2 && __any_sync(kFull, move)) {   // the output so far
                        if (!(ok = wait_warp(&bars.pv_done[g], (own + 1) & 1))) break;
                        tc::fence_after();
#pragma unroll 1
                        for (int c = 0; c < DP / 32; ++c) {
                            float o[32];
                            tc::tmem_load(tO[g] + row_lane + c * 32, o);
                            tc::tmem_wait_load();
                            tc::loaded(o);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] *= keep;
                            tc::tmem_store(tO[g] + row_lane + c * 32, o);
                        }
                        tc::tmem_wait_store();
                    }
                    if (!__any_sync(kFull, to.far)) break;
                    base = mr == neg_inf() ? -0.f : -mr;   // (all of the warp's rows, then)
                    minus = Half<T>::kUp;
                }
                if (!ok) break;
                const float2 scale = make_float2(a.sL, a.sL), minus2 = make_float2(minus, minus);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t p[16];
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        float2 e = __ffma2_rn(make_float2(x[c][i], x[c][i + 1]), scale, minus2);
                        e.x = ex2(e.x);
                        e.y = ex2(e.y);
                        sum[c & 1] = __fadd2_rn(sum[c & 1], e);
                        p[i / 2] = Half<T>::pack(e.x, e.y);
                    }
                    tc::tmem_store16(mS + c * 16, p);
                }
                tc::tmem_wait_store();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) tc::bar_arrive(tc::smem(&bars.p_ready[g]));
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                ++own;
            }
            if (!ok) break;
            // ---- the segment's output ---------------------------------------------------------
            const bool two = s.act == 2, both = !two && jobs > 1;
            const bool mine = both || two || g == 0;   // (a stream may have had no job)
            // while the last products run: where the output goes, and the next segment
            const bool whole = s.t0 == 0 && s.t1 == s.tiles, holds_nodes = s.t1 > tails;
            const long long row = ((long long)s.b * a.N + node) * a.Hq + s.h * a.G + row_head;
            const long long slot = ((long long)me * 2 + (s.t0 == 0 ? 1 : 0)) * 2 + (two ? g : 0);
            const int b = s.b, h = s.h, L = s.L;
            __syncwarp();
            more = false;
            if (lane == 0) more = s.next(a);
            if (mine && !(ok = wait_warp(&bars.pv_done[g], (own + 1) & 1))) break;
            if (!two) {
                if (mine) sh.ml[g][r] = make_float2(mr, l);
                __syncwarp();
                if (lane == 0) tc::bar_arrive(tc::smem(&bars.merge));
                if (!(ok = wait_warp(&bars.merge, merges++ & 1))) break;
            }
            tc::fence_after();
            // one tile: both warpgroups take half of the columns of both streams' outputs
            float w0 = 1.f, w1 = 0.f;
            if (!two) {
                const float2 m0 = sh.ml[0][r], m1 = sh.ml[1][r];
                mr = both ? fmaxf(m0.x, m1.x) : m0.x;
                const Reference to = reference<T>(a, mr);
                w0 = weight<T>(a, m0.x, to);
                w1 = both ? weight<T>(a, m1.x, to) : 0.f;   // (ml[1] is not written for a stream without jobs)
                l = m0.y * w0 + (both ? m1.y * w1 : 0.f);
            }
            const float inv = whole ? (l != 0.f ? 1.f / l : 0.f) : 1.f;
            w0 *= inv;
            w1 *= inv;
            uint32_t bad[4] = {0, 0, 0, 0};
            if (holds_nodes) {   // (a node's value is in one piece, and its flag in that piece's alone)
                const uint32_t *f = sh.bad[segs % kSegRing];
                bad[0] = f[0] & v0;
                bad[1] = f[1] & v1;
                bad[2] = f[2] & v2;
                bad[3] = f[3] & v3;
            }
            const bool spoilt = (bad[0] | bad[1] | bad[2] | bad[3]) != 0;
            const int c0 = two ? 0 : g * (DP / 64), c1 = two ? DP / 32 : c0 + DP / 64;
#pragma unroll 1
            for (int c = idle ? c1 : c0; c < c1; ++c) {
                float o[32];
                __syncwarp();
                tc::tmem_load(tO[two ? g : 0] + row_lane + c * 32, o);
                tc::tmem_wait_load();
                tc::loaded(o);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] *= w0;
                if (both) {
                    float q[32];
                    tc::tmem_load(tO[1] + row_lane + c * 32, q);
                    tc::tmem_wait_load();
                    tc::loaded(q);
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = fmaf(q[i], w1, o[i]);
                }
                if (!real) continue;
                if (spoilt) {
#pragma unroll 1
                    for (int j = 0; j < a.N; ++j) {
                        const uint32_t bits = j < 32 ? bad[0] : j < 64 ? bad[1] : j < 96 ? bad[2] : bad[3];
                        if (!(bits >> (j & 31) & 1)) continue;
                        const int key = L + j, p = a.table[(long long)b * a.M + key / a.page];
                        if (p < 0 || p >= a.P) continue;
                        const unsigned short *v = static_cast<const unsigned short *>(a.v) + p * a.vs[0] + key % a.page * a.vs[1] +
                                                  h * a.vs[2] + c * 32;
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
                if (!whole) a.part_ml[slot * kTile + r] = make_float2(mr, l);
                else if (a.lse) a.lse[row] = l != 0.f ? sv::kLn2 * (log2_of<T>(a, mr) + log2f(l)) : neg_inf();
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::bar_arrive(tc::smem(&bars.o_free));
            more = __shfl_sync(kFull, more, 0);
            ++segs;
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == kWarpMma0) tc::tmem_free(tmem, 512);
}

// The pieces of what was cut: CTA x joins what begins in CTA x's part and ends in another's. A
// thread per row and four columns, eight rows side by side; the pieces' references
// first, then their outputs.
constexpr int kJoinRows = 8;

// A piece's part of a sum that came out NaN: an infinity stays one (a weight below fp32's
// range is not 0, and a sequence that is not cut keeps its nodes' infinities, too)
__device__ __forceinline__ float part(float x, float w) { return fabsf(x) == INFINITY ? x : x * w; }

template <typename T, int DC>
__global__ void __launch_bounds__(DC * 16 * kJoinRows) join_kernel(const __grid_constant__ AttendArgs a) {
    constexpr int DP = DC * 64;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 join = a.joins[blockIdx.x];
    if (join.x < 0) return;
    const int rr = blockIdx.y * kJoinRows + threadIdx.x % kJoinRows, c4 = threadIdx.x / kJoinRows;
    const int used = a.nodes * a.G, m_tile = rr / used, r = rr - m_tile * used;   // (rows of a tile that are used)
    const int h = join.y & 0xffff, node = (2 * (join.y >> 16) + m_tile) * a.nodes + r / a.G;
    if (m_tile > 1 || rr >= join.z) return;
    const int first = blockIdx.x, pieces = join.w - first + 1;
    auto slot = [&](int i) { return ((long long)(first + i) * 2 + (i == 0 ? 1 : 0)) * 2 + m_tile; };
    float mr = neg_inf(), l = 0.f;
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
        float to = mr;
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (i0 + i < pieces) to = fmaxf(to, ml[i].x);
        const Reference ref = reference<T>(a, to);
        const float keep = weight<T>(a, mr, ref);
        mr = to;
        l *= keep;
        o.x *= keep;
        o.y *= keep;
        o.z *= keep;
        o.w *= keep;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (i0 + i < pieces) {
                const float w = weight<T>(a, ml[i].x, ref);
                l = fmaf(ml[i].y, w, l);
                o.x = fmaf(v[i].x, w, o.x);
                o.y = fmaf(v[i].y, w, o.y);
                o.z = fmaf(v[i].z, w, o.z);
                o.w = fmaf(v[i].w, w, o.w);
            }
        }
    }
    if (isnan((o.x + o.y) + (o.z + o.w))) {
        const Reference ref = reference<T>(a, mr);
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int i = 0; i < pieces; ++i) {
            const float w = weight<T>(a, a.part_ml[slot(i) * kTile + r].x, ref);
            const float4 v = a.part_o[(slot(i) * (DP / 4) + c4) * kTile + r];
            sum.x += part(v.x, w);
            sum.y += part(v.y, w);
            sum.z += part(v.z, w);
            sum.w += part(v.w, w);
        }
        if (isnan(o.x)) o.x = sum.x;
        if (isnan(o.y)) o.y = sum.y;
        if (isnan(o.z)) o.z = sum.z;
        if (isnan(o.w)) o.w = sum.w;
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    const long long row = ((long long)join.x * a.N + node) * a.Hq + h * a.G + r % a.G;
    if (c4 * 4 < a.D)
        *reinterpret_cast<uint2 *>(static_cast<T *>(a.out) + row * a.D + c4 * 4) =
            make_uint2(Half<T>::pack(o.x * inv, o.y * inv), Half<T>::pack(o.z * inv, o.w * inv));
    if (c4 == 0 && a.lse) a.lse[row] = l != 0.f ? sv::kLn2 * (log2_of<T>(a, mr) + log2f(l)) : neg_inf();
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
    // units of work: of a sequence, and of one CTA of at least 64
    const int64_t nodes = kTile / (p->Hq / p->Hkv), pairs = (p->N + 2 * nodes - 1) / (2 * nodes);
    const int64_t units = ((int64_t)p->M * p->page + kTile - 1) / kTile * pairs * p->Hkv;
    if (units > INT32_MAX || units * p->B > (1LL << 36))
        return spec_internal_set_error(SPEC_ERR_UNSUPPORTED, "tree_attention: rows too long or too many");
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

// [n3][n2][n1][D] of 16-bit elements, boxes of 64 elements x b1 x b2. L2 fetches no more than is asked
// for: a head's 128 or 160 bytes beside other heads' took 131 and 260 us with 256 bytes, 101 and 213 without (60 x
// 10684 tokens of 5 heads of 64, 40 x 12642 of 8 of 80); heads of 128 are 256 bytes and do not care.
static bool encode(CUtensorMap *map, int bf16, const void *base, int D, const int *n, const int64_t *stride, int b1, int b2) {
    const EncodeFn fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)n[2], (cuuint64_t)n[1], (cuuint64_t)n[0]};
    cuuint64_t st[3];
    for (int i = 0; i < 3; ++i) st[i] = n[2 - i] > 1 ? (cuuint64_t)stride[2 - i] * 2 : (cuuint64_t)(D * 2 + 15) / 16 * 16;
    const cuuint32_t box[4] = {64, (cuuint32_t)b1, (cuuint32_t)b2, 1}, one[4] = {1, 1, 1, 1};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void *>(base), dims, st, box,
              one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxCtas = 152;   // one per SM; the workspace's room

static size_t part_floats(int D) { return (size_t)kMaxCtas * 4 * kTile * (D > 64 ? 128 : 64); }
static size_t workspace_bytes_for(const spec_attend_params *p) {
    return part_floats(p->D) * 4 + (size_t)kMaxCtas * 4 * kTile * 8 + (size_t)kMaxCtas * 16;
}

template <typename T, int DC, bool FEW>
static cudaError_t launch_attend(const AttendArgs &a, const CUtensorMap *maps, int box, cudaStream_t st) {
    constexpr size_t smem = AttendSmem<DC, FEW>::kTiles + sizeof(typename AttendSmem<DC, FEW>::Shared);
    static_assert(smem <= 227 * 1024, "shared memory");
    // once for each device: the shared memory allowed, and the number of SMs
    static std::mutex mu;
    static int sms[64];
    int dev = 0, ctas = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (sms[dev & 63] == 0) {
            int n = 0;
            e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(attend_kernel<T, DC, FEW>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess) return e;
            sms[dev & 63] = n < kMaxCtas ? n : kMaxCtas;
        }
        ctas = sms[dev & 63];
    }
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
    e = cudaLaunchKernelEx(&cfg, attend_kernel<T, DC, FEW>, a, maps[0], maps[1], maps[2], box);
    if (e != cudaSuccess) return e;
    const int tiles = (a.N + a.nodes - 1) / a.nodes, rows = tiles > 1 ? 2 * a.nodes * a.G : a.N * a.G;
    cfg.gridDim = dim3(ctas, (rows + kJoinRows - 1) / kJoinRows);
    cfg.blockDim = dim3(DC * 16 * kJoinRows);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, join_kernel<T, DC>, a);
}

template <typename T>
static cudaError_t launch_attend(const AttendArgs &a, const CUtensorMap *maps, int box, cudaStream_t st) {
    const bool few = a.N * a.G <= 64;
    if (a.D > 64) return few ? launch_attend<T, 2, true>(a, maps, box, st) : launch_attend<T, 2, false>(a, maps, box, st);
    return few ? launch_attend<T, 1, true>(a, maps, box, st) : launch_attend<T, 1, false>(a, maps, box, st);
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
    const int q_nodes = p->N < a.nodes ? p->N : a.nodes;
    a.q_rows = q_nodes * G;
    a.sL = fmaxf(fabsf(p->scale) * sv::kLog2e, FLT_MIN);   // (0 times a masked key's -inf would be NaN)
    a.lazy = kLazy / a.sL;   // (infinite for scales next to 0: no score reaches it)
    a.neg = p->scale < 0.f;
    a.spin = spec_internal_wait_limit();
    a.ps = p->parents_stride;
    for (int j = 0; j < 3; ++j) a.vs[j] = p->v_stride[j];
    const int nq[3] = {p->B, p->N, p->Hq}, nk[3] = {p->P > 0 ? p->P : 1, p->page, p->Hkv}, box = p->page < 64 ? p->page : 64;
    const int bf16 = p->dtype == SPEC_BF16;
    const int64_t none[3] = {0, 0, 0};
    CUtensorMap maps[3];
    const int empty[3] = {1, 1, 1};
    if (!encode(&maps[0], bf16, q, p->D, nq, p->q_stride, G, q_nodes) ||
        !encode(&maps[1], bf16, p->P ? k : q, p->D, p->P ? nk : empty, p->P ? p->k_stride : none, 1, box) ||
        !encode(&maps[2], bf16, p->P ? v : q, p->D, p->P ? nk : empty, p->P ? p->v_stride : none, 1, box))
        return spec_internal_set_error(SPEC_ERR_CUDA, "tree_attention: the copies' layout could not be encoded");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    e = bf16 ? launch_attend<__nv_bfloat16>(a, maps, box, st) : launch_attend<__half>(a, maps, box, st);
    return e == cudaSuccess ? SPEC_OK : spec_internal_set_error(SPEC_ERR_CUDA, cudaGetErrorString(e));
}

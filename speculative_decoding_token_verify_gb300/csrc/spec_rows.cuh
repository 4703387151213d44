// spec_rows.cuh -- building blocks of the row operators (top log-probabilities,
// distillation, beam step): a row's layout in 16-byte vectors, the running sum
// of a softmax, ordered keys, block reductions. Internal to the library.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "spec_device.cuh"
#include "spec_verify.h"

namespace sr {

using sv::Elem;
using sv::ex2;
using sv::kLog2e;
using sv::neg_inf;

constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ void raise_status(int32_t *status, int code) {
    if (status) atomicMax(status, code);
}

// ---- a row as scalars, 16-byte vectors, scalars ----------------------------
//
// `head` elements up to the first 16-byte boundary, nvec vectors, `tail`
// elements: any row base that is aligned to its element streams in whole
// vectors, so odd vocabularies and strides cost two partial vectors a row.
template <typename T>
struct Row {
    static constexpr int E = Elem<T>::kPerVec;
    const T *p;
    const uint4 *body;
    int head, nvec, tail;

    __device__ __forceinline__ Row(const T *row, int V) {
        p = row;
        const int mis = (int)(reinterpret_cast<uintptr_t>(row) & 15u);
        head = mis ? min(V, (16 - mis) / (int)sizeof(T)) : 0;
        nvec = (V - head) / E;
        tail = V - head - nvec * E;
        body = reinterpret_cast<const uint4 *>(row + head);
    }
    __device__ __forceinline__ int vec_index(int k) const { return head + k * E; }
    // the element of the head or the tail that slot t (0 .. 2E-1) stands for, or -1
    __device__ __forceinline__ int edge_index(int t) const {
        if (t < head) return t;
        if (t >= E && t - E < tail) return head + nvec * E + t - E;
        return -1;
    }
};

// a CTA's part of a row: vectors [k0, k0 + n), the row's head in the first
// part and its tail in the last, elements [e0, e1) in all
template <typename T>
struct Part {
    static constexpr int E = Row<T>::E;
    Row<T> r;
    int k0, n, e0, e1;
    bool first, last;
    __device__ __forceinline__ Part(const T *row, int V, int rank, int parts)
        : r(row, V), first(rank == 0), last(rank == parts - 1) {
        k0 = (int)((long long)r.nvec * rank / parts);
        n = (int)((long long)r.nvec * (rank + 1) / parts) - k0;
        ends(V);
    }
    // parts of `size` vectors, the last one shorter
    __device__ __forceinline__ Part(const T *row, int V, int rank, int parts, int size)
        : r(row, V), first(rank == 0), last(rank == parts - 1) {
        k0 = min(r.nvec, rank * size);
        n = last ? r.nvec - k0 : min(size, r.nvec - k0);
        ends(V);
    }
    __device__ __forceinline__ void ends(int V) {
        e0 = first ? 0 : r.vec_index(k0);
        e1 = last ? V : r.vec_index(k0 + n);
    }
    // the head's or tail's element of slot t, or -1
    __device__ __forceinline__ int edge(int t) const {
        if (t >= 2 * E) return -1;
        const int i = r.edge_index(t);
        return i >= 0 && (t < E ? first : last) ? i : -1;
    }
    __device__ __forceinline__ const uint4 *body() const { return r.body + k0; }
};

template <typename T>
__device__ __forceinline__ float load1(const T *p) {
    return Elem<T>::load(p);
}

// Loads of logits that the same kernel may overwrite (gradients in place):
// ordered before later stores, and not through the read-only path.
template <typename T>
__device__ __forceinline__ float load1_rw(const T *p) {
    if constexpr (sizeof(T) == 2) {
        unsigned short h;
        asm volatile("ld.global.u16 %0, [%1];" : "=h"(h) : "l"(p) : "memory");
        return __uint_as_float((uint32_t)h << 16);
    } else {
        float f;
        asm volatile("ld.global.f32 %0, [%1];" : "=f"(f) : "l"(p) : "memory");
        return f;
    }
}

// ---- running sum of 2^{(z - mr) sL} ------------------------------------------
//
// One thread's softmax sum against a lazy reference mr that moves only when a
// logit exceeds it by rs (8 processed nats), so that terms stay below e^8.
// The exponent is one FMA, z sL - fl(mr sL); the rounding of mr sL is the
// same factor on every term and is taken out with its exact value eps when
// the reference moves and at the end. Chunks of a few vectors are summed
// apart and added with a compensation, so that a term meets at most about
// twenty roundings on its way into the sum, however long the row.
//
// Beyond |z sL| = 2^30 (masks of -1e9 at a low temperature, of -1e20 at any) eps
// would overflow 2^eps. So the reference starts at -2^30 / sL: logits below add
// nothing. They are 64 or more apart in the exponent, so that a sum against a
// maximum out there is the number of logits equal to it, which a pass of its
// own counts where a part's maximum turns out to lie there, or as far above 0.
struct Sum {
    float mr, mrL, eps, mrh;
    float mx;      // largest logit seen
    float S, lo;   // the sum is S - lo
};

constexpr float kFar = 1073741824.f;
__device__ __forceinline__ bool far_max(float m, float sL) { return m > sv::kMaskFloor && fabsf(m * sL) > kFar; }

__device__ __forceinline__ Sum sum_init(float sL, float rs) {
    Sum a;
    a.mr = rs * (-kFar / (sv::kRescale * kLog2e));   // rs = kRescale / s
    a.mrL = a.mr * sL;
    a.eps = fmaf(a.mr, sL, -a.mrL);
    a.mrh = a.mr + rs;
    a.mx = neg_inf();
    a.S = a.lo = 0.f;
    return a;
}

// before terms are added: c is the largest of their logits
__device__ __forceinline__ void sum_see(Sum &a, float c, float sL, float rs) {
    a.mx = fmaxf(a.mx, c);
    if (c > a.mrh) {
        const float cL = c * sL, ce = fmaf(c, sL, -cL);
        const float al = ex2(fmaf(a.mr - c, sL, ce - a.eps));
        a.S *= al;
        a.lo *= al;
        a.mr = c;
        a.mrL = cL;
        a.eps = ce;
        a.mrh = c + rs;
    }
}

// E logits' terms; masked logits add nothing
template <int E>
__device__ __forceinline__ float sum_terms(const Sum &a, const float (&z)[E], float sL) {
    const float2 L2 = make_float2(sL, sL), ml = make_float2(-a.mrL, -a.mrL);
    float2 e[E / 2];
#pragma unroll
    for (int j = 0; j < E / 2; ++j) {
        const float2 y = sv::pfma(make_float2(z[2 * j], z[2 * j + 1]), L2, ml);
        e[j] = make_float2(ex2(y.x), ex2(y.y));
    }
#pragma unroll
    for (int w = E / 4; w > 0; w >>= 1)
#pragma unroll
        for (int j = 0; j < w; ++j) e[j] = sv::padd(e[j], e[j + w]);
    return e[0].x + e[0].y;
}

// a chunk's sum into the running one (Kahan)
template <typename S>
__device__ __forceinline__ void sum_put(S &a, float v) {
    const float y = __fsub_rn(v, a.lo);
    const float t = __fadd_rn(a.S, y);
    a.lo = __fsub_rn(__fsub_rn(t, a.S), y);
    a.S = t;
}

__device__ __forceinline__ void sum_add1(Sum &a, float z, float sL, float rs) {
    sum_see(a, z, sL, rs);
    sum_put(a, ex2(fmaf(z, sL, -a.mrL)));
}

// the sum against the maximum M
__device__ __forceinline__ float sum_at(const Sum &a, float M, float sL) {
    const float S = a.S - a.lo;
    return S != 0.f ? S * ex2(fmaf(a.mr - M, sL, -a.eps)) : 0.f;
}

// The same sum with the exponent (z - mr) sL, two operations a logit in place of
// one: right for logits of any size without a second pass, and where memory
// bounds the kernel no slower.
struct DiffSum {
    float mr, mrh, mx, S, lo;
};
__device__ __forceinline__ DiffSum diff_init(float rs) {
    const float mr = sv::kMaskFloor * (1.f - 0x1p-23f);   // the least unmasked logit
    return {mr, mr + rs, neg_inf(), 0.f, 0.f};
}
__device__ __forceinline__ void sum_see(DiffSum &a, float c, float sL, float rs) {
    a.mx = fmaxf(a.mx, c);
    if (c > a.mrh) {
        const float al = ex2((a.mr - c) * sL);
        a.S *= al;
        a.lo *= al;
        a.mr = c;
        a.mrh = c + rs;
    }
}
template <int E>
__device__ __forceinline__ float sum_terms(const DiffSum &a, const float (&z)[E], float sL) {
    const float2 L2 = make_float2(sL, sL), ml = make_float2(-a.mr, -a.mr), zero = make_float2(0.f, 0.f);
    float2 e[E / 2];
#pragma unroll
    for (int j = 0; j < E / 2; ++j) {
        const float2 y = sv::pfma(sv::padd(make_float2(z[2 * j], z[2 * j + 1]), ml), L2, zero);
        e[j] = make_float2(ex2(y.x), ex2(y.y));
    }
#pragma unroll
    for (int w = E / 4; w > 0; w >>= 1)
#pragma unroll
        for (int j = 0; j < w; ++j) e[j] = sv::padd(e[j], e[j + w]);
    return e[0].x + e[0].y;
}
__device__ __forceinline__ void sum_add1(DiffSum &a, float z, float sL, float rs) {
    sum_see(a, z, sL, rs);
    sum_put(a, ex2((z - a.mr) * sL));
}
__device__ __forceinline__ float sum_at(const DiffSum &a, float M, float sL) {
    const float S = a.S - a.lo;
    return S != 0.f ? S * ex2((a.mr - M) * sL) : 0.f;
}

// a sum against the maximum m, moved to the larger maximum `to`
__device__ __forceinline__ float moved(float sum, float m, float to, float sL) {
    return sum != 0.f && m != to ? sum * ex2((m - to) * sL) : sum;
}

template <typename T>
__device__ __forceinline__ float vec_max(const uint4 &w) {
    if constexpr (sizeof(T) == 2) {
        const uint32_t m = sv::bmax2(sv::bmax2(w.x, w.y), sv::bmax2(w.z, w.w));
        return fmaxf(sv::bf16_lo(m), sv::bf16_hi(m));
    } else {
        return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
    }
}

// a vector of masked logits
template <typename T>
__device__ __forceinline__ uint4 masked_vec() {
    const uint32_t w = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
    return make_uint4(w, w, w, w);
}

// ---- two-float arithmetic: value = h + l ---------------------------------------

__device__ __forceinline__ void two_sum(float a, float b, float &h, float &l) {
    h = __fadd_rn(a, b);
    const float t = __fsub_rn(h, a);
    l = __fadd_rn(__fsub_rn(a, __fsub_rn(h, t)), __fsub_rn(b, t));
}

// (h, l) += (a, b)
__device__ __forceinline__ void add2f(float &h, float &l, float a, float b) {
    float e;
    two_sum(h, a, h, e);
    l += b + e;
}

// e^x of x = z - M as h + l, relative error at most 2e-10 (0 below e^-87, inf above e^87): x = n ln2 + r with
// ln2 in three floats, then e^r by its Taylor series, whose first terms carry
// their roundings
__device__ __forceinline__ void exp_diff(float z, float M, float &h, float &l) {
    float xh, xl;
    two_sum(z, -M, xh, xl);
    if (!(fabsf(xh) < 87.f)) {
        h = xh > 0.f ? INFINITY : xh == xh ? 0.f : xh;
        l = 0.f;
        return;
    }
    const float n = rintf(xh * kLog2e);
    // ln2 = A + B + rest, A its first 12 bits, so that n A is exact
    constexpr double kL = 0.69314718055994530942;
    constexpr float A = (float)((double)(int)(kL * 4096.0) / 4096.0);
    constexpr float B = (float)(kL - (double)A);
    constexpr double kRest = kL - (double)A - (double)B;
    float rh, rl, t;
    two_sum(__fmaf_rn(-n, A, xh), xl, rh, rl);   // n A and the difference are exact
    float nb = __fmul_rn(n, B), nbl = __fmaf_rn(n, B, -nb);
    two_sum(rh, -nb, rh, t);
    rl = rl + t - nbl - n * (float)kRest;
    two_sum(rh, rl, rh, rl);
    // e^r = 1 + r + r^2/2 + r^3 Q(r), |r| <= 0.35
    const float r = rh;
    float q = 1.f / 3628800.f;
    q = fmaf(q, r, 1.f / 362880.f);
    q = fmaf(q, r, 1.f / 40320.f);
    q = fmaf(q, r, 1.f / 5040.f);
    q = fmaf(q, r, 1.f / 720.f);
    q = fmaf(q, r, 1.f / 120.f);
    q = fmaf(q, r, 1.f / 24.f);
    // r^3 (1/6 + r q): the leading 1/6 in two floats
    const float r2 = __fmul_rn(r, r), r2l = __fmaf_rn(r, r, -r2);
    const float r3 = __fmul_rn(r2, r), r3l = __fmaf_rn(r2, r, -r3) + r2l * r;
    constexpr float s6 = 1.f / 6.f;
    constexpr float s6l = (float)(1.0 / 6.0 - (double)s6);
    const float c3 = __fmul_rn(r3, s6), c3l = __fmaf_rn(r3, s6, -c3) + r3l * s6 + r3 * s6l;
    const float c4 = r2 * r2 * q;   // <= 6e-4: one rounding of 4e-11
    float sh, sl, e1, e2, e3;
    two_sum(1.f, r, sh, e1);
    two_sum(sh, 0.5f * r2, sh, e2);
    two_sum(sh, c3, sh, e3);
    sl = e1 + e2 + e3 + (rl * sh + 0.5f * r2l + c3l + c4);   // rl e^r: sh is e^r but for r^4
    two_sum(sh, sl, sh, sl);
    const float sc = __int_as_float(((int)n + 127) << 23);   // n >= -126
    h = sh * sc;
    l = sl * sc;
}

// a value h + l, |l| <= half a step of h
struct Pair {
    float h, l;
};

// ln S in two floats: one Newton step from logf, S = Sh + Sl
__device__ __forceinline__ Pair ln_pair(float Sh, float Sl) {
    const float g = logf(Sh);
    float eh, el;
    exp_diff(g, 0.f, eh, el);
    const float r = ((Sh - eh) + (Sl - el)) / Sh;
    float h, l;
    two_sum(g, r, h, l);
    return {h, l};
}

// ---- ordered keys --------------------------------------------------------------
//
// Larger logit, larger key; both zeros alike; masked logits (-inf, or below
// -1e29: masks of a type's lowest value) and NaN are key 0.
__device__ __forceinline__ uint32_t order_key(float z) {
    if (!(z > sv::kMaskFloor)) return 0u;
    const int i = __float_as_int(z + 0.f);
    return i < 0 ? ~(uint32_t)i : (uint32_t)i | 0x80000000u;
}

__device__ __forceinline__ float key_value(uint32_t k) {
    if (k == 0u) return neg_inf();
    return __int_as_float(k & 0x80000000u ? (int)(k & 0x7fffffffu) : ~(int)k);
}

// a candidate: the logit's key over the complement of its index, so that the
// larger word ranks first and equal logits rank by ascending index
__device__ __forceinline__ unsigned long long cand(uint32_t key, int index) {
    return ((unsigned long long)key << 32) | (uint32_t)~(uint32_t)index;
}
__device__ __forceinline__ int cand_index(unsigned long long c) { return (int)~(uint32_t)c; }
__device__ __forceinline__ uint32_t cand_key(unsigned long long c) { return (uint32_t)(c >> 32); }

// ---- warp reductions (fixed order) ----------------------------------------------

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// ---- thread-block clusters ----------------------------------------------------------

// (relaxed: by threads that publish nothing)
// The aligned forms want whole warps.
__device__ __forceinline__ void cluster_arrive_relaxed() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the address of a shared variable in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t peer(const void *p, int rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void peer_store(uint32_t a, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void peer_store(uint32_t a, unsigned long long v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ void peer_store_u32(uint32_t a, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ int peer_add(uint32_t a, int v) {
    int r;
    asm volatile("atom.relaxed.cluster.shared::cluster.add.s32 %0, [%1], %2;" : "=r"(r) : "r"(a), "r"(v) : "memory");
    return r;
}

// Launch with clusters of `cluster` CTAs along x (1: none).
template <typename... P, typename... A>
cudaError_t launch_cluster(void (*kernel)(P...), unsigned grid, unsigned nt, unsigned cluster, size_t smem,
                           cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(nt);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---- host-side checks shared by the row and tree operators --------------------------------

int check_rows(const spec_rows_params *p, int max_m, int max_k);
int check_strided(const void *base, int64_t batch_stride, int64_t row_stride, int es, bool out, int B, int K, int V);
// whether na bytes from a on and nb from b on have one in common
inline bool overlap(const void *a, int64_t na, const void *b, int64_t nb) {
    const char *x = static_cast<const char *>(a), *y = static_cast<const char *>(b);
    return na > 0 && nb > 0 && x < y + nb && y < x + na;
}

}  // namespace sr

// defined in spec_verify.cu: sets the thread-local message read by spec_last_error
extern "C" int spec_internal_set_error(int code, const char *msg);

// spec_distill.cu -- distillation of a student's rows from a teacher's top
// lists: loss, gradient by the student's logits, both in one call.
//
// With q = softmax(s y), the list's probabilities p_m, the unlisted tokens'
// teacher mass p_T = 1 - P and student mass q_T:
//   KL = sum_m p_m (l_m - ln q(id_m)) + p_T (ln p_T - ln q_T)
//   dKL / dy_v = s (c q_v - sum_m p_m [id_m = v])   at listed v
//              = s (c q_T - p_T) r_v                at unlisted v,
// r = the softmax over the unlisted tokens alone: their part of q rescaled to
// the teacher's mass; c = P + p_T is the teacher's mass, 1 unless P is more.
//
// The unlisted tokens have a maximum and a sum of their own, so neither q_T =
// 1 - Q (which cancels when the list holds nearly all of the mass) nor q_T /
// p_T (which leaves fp32's range when it holds yet more) is ever formed: the
// list's tokens are marked in a bit map of the row in shared memory, looked up
// once per 16-byte vector. The list's exponentials, their sum P and the loss's
// terms are kept in two floats (p_T = 1 - P, and terms of either sign, cancel):
// in fp64 that work kept GB300's fp64 pipe 53% busy, and the step 1.5 times as
// long.
//
// Loss and step: a cluster of S CTAs per row, each a part of it; a CTA owns the
// list's tokens in its part, and what the CTAs know (maxima, sums, P, the
// loss's terms) meets in one exchange through distributed shared memory. The
// step goes over its part a second time, backwards: the last two iterations
// are still in registers, up to three more in shared memory, the others come
// again from L2, where they were kept by policy, so HBM reads a row once and
// writes its gradient once. The gradient alone needs no exchange: a CTA per 256
// UG vectors.
//
// Measured (bf16, M = 64; shares of the measured copy rate, 6691 GB/s): the loss
// of 1920 rows of 152064 87 us, 6.1 TB/s, 91%; the step of 2048 rows of 128256
// 186 us, 5.4 TB/s of read and written bytes, 81%; the gradient of 2048 rows of
// 128256 151 us, 7.0 TB/s, the rate of a copy; of 320 rows, a tenth of them without
// weight, 25 us in a graph over three input sets (the 82 MB written stay in L2) and
// 28 us called one by one. f32, 2048 rows of 128256: loss 156 us, gradient 297 us, step
// 387 us, the same rates. The step is bound by loads in flight in its second pass
// (issue slots half busy, long-scoreboard stalls first). Without the held
// iterations it takes 190 us, without the L2 policies too 222 us, with S = 8 and
// the whole part in registers 285 us (a part's fixed cost, about 7 us, eight
// times a row), with a persistent CTA per SM fed by bulk copies into a ring of
// chunks 244 us (and the loss 132 to 156 us): 16 warps do not hide the ring's
// waits. 256 threads, 4 loads an iteration and 4 CTAs per SM: 190 us then; 2 or 3
// loads and 5 or 6 CTAs 197 to 217, 128 or 512 threads 214 and 212.
#include <mutex>

#include "spec_rows.cuh"

namespace sr {

constexpr int UG = 8;   // vectors per thread of the gradient alone
constexpr int kMaxCluster = 8;

struct DistillArgs {
    const void *y;
    long long bs, rs;
    void *g;
    long long gbs, grs;
    int B, K, V, M, tail;
    float s, sL, resc;
    const float *logp;
    const int32_t *ids;
    const float *weight, *grad_loss;
    const float4 *stats_in;
    float *loss;
    float4 *stats_out;
    int32_t *status;
};

// one rounding to nearest, the gradient's only one below fp32
template <typename T>
__device__ __forceinline__ T to_elem(float v) {
    if constexpr (sizeof(T) == 2) return __float2bfloat16_rn(v);
    else return v;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
}
template <typename T>
__device__ __forceinline__ uint4 pack_vec(const float (&z)[Elem<T>::kPerVec]) {
    if constexpr (sizeof(T) == 2) return make_uint4(pack2(z[0], z[1]), pack2(z[2], z[3]), pack2(z[4], z[5]), pack2(z[6], z[7]));
    else return make_uint4(__float_as_uint(z[0]), __float_as_uint(z[1]), __float_as_uint(z[2]), __float_as_uint(z[3]));
}

// the part's map of listed tokens: bit 16 + 8 i or 16 + 4 i starts vector i,
// the head lies before it and the tail behind the last vector
template <typename T>
__device__ __forceinline__ int map_bit(const Part<T> &p, int v) {
    return v - p.r.vec_index(p.k0) + 16;
}
template <typename T>
__device__ __forceinline__ uint32_t map_vec(const uint8_t *map, int i) {
    if constexpr (sizeof(T) == 2) return map[i + 2];
    else return (uint32_t)map[(i + 4) >> 1] >> ((i & 1) * 4) & 15u;
}

// the gradient's part: vectors where both rows are aligned alike, else elements
template <typename T>
struct Out {
    T *g;          // the row
    uint4 *body;   // the part's first vector, or null
    __device__ __forceinline__ Out(T *row, const Part<T> &p)
        : g(row),
          body(((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(p.r.p)) & 15u) == 0
                   ? reinterpret_cast<uint4 *>(row + p.r.vec_index(p.k0))
                   : nullptr) {}
    __device__ __forceinline__ void put(const Part<T> &p, int i, const float (&z)[Elem<T>::kPerVec]) const {
        if (body) {
            __stcs(body + i, pack_vec<T>(z));
        } else {
#pragma unroll
            for (int j = 0; j < Elem<T>::kPerVec; ++j) g[p.r.vec_index(p.k0 + i) + j] = to_elem<T>(z[j]);
        }
    }
};

template <typename T, int NT>
__device__ __forceinline__ void zero_part(const Part<T> &p, const Out<T> &o) {
    float z[Part<T>::E];
#pragma unroll
    for (int j = 0; j < Part<T>::E; ++j) z[j] = 0.f;
    for (int i = threadIdx.x; i < p.n; i += NT) o.put(p, i, z);
    const int i = p.edge(threadIdx.x);
    if (i >= 0) o.g[i] = to_elem<T>(0.f);
}

// The unlisted tokens' gradient ku e^{s (y - mo)}; masked logits give 0
struct Factor {
    float ku, mo;
};
__device__ __forceinline__ float grad_one(const Factor &f, float y, float sL) { return f.ku * ex2((y - f.mo) * sL); }

template <typename T>
__device__ __forceinline__ void grad_vec(const Part<T> &p, const Out<T> &o, int i, const uint4 &w, const Factor &f,
                                         float sL) {
    constexpr int E = Part<T>::E;
    float z[E];
    Elem<T>::unpack(w, z);
    const float2 L2 = make_float2(sL, sL), mo = make_float2(-f.mo, -f.mo), k2 = make_float2(f.ku, f.ku);
    const float2 zero = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < E / 2; ++j) {
        const float2 y = sv::pfma(sv::padd(make_float2(z[2 * j], z[2 * j + 1]), mo), L2, zero);
        const float2 g = sv::pfma(make_float2(ex2(y.x), ex2(y.y)), k2, zero);
        z[2 * j] = g.x;
        z[2 * j + 1] = g.y;
    }
    o.put(p, i, z);
}

// L2 policies: rows read twice are kept for the second read, then let go. No
// load takes the read-only path: the step may write over its logits (and the
// path gains nothing, 186 us with it as without).
__device__ __forceinline__ uint64_t l2_keep() {
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ uint64_t l2_drop() {
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ uint4 ld_stream(const uint4 *p, uint64_t policy) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0,%1,%2,%3}, [%4], %5;"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p), "l"(policy));
    return v;
}
__device__ __forceinline__ uint4 ld_rw(const uint4 *p, uint64_t policy) {
    uint4 v;
    asm volatile("ld.global.L2::cache_hint.v4.u32 {%0,%1,%2,%3}, [%4], %5;"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p), "l"(policy)
                 : "memory");
    return v;
}
__device__ __forceinline__ uint4 ld_rw(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

// what a CTA knows of its part, and the row's total of it
struct __align__(16) Known {
    float mo, So;    // unlisted tokens: maximum, sum of 2^{(y - mo) sL}
    float ml, Sl;    // listed tokens: the same, each once
    float Ph, Pl;    // sum of p = e^(l - l0), in two floats
    float Bh, Bl;    // sum of p (l - l0 - s (y - y0)), in two floats
};

// a two-float sum with the lane o away; both lanes get the same bits
__device__ __forceinline__ void pair_total(float &h, float &l, int o) {
    const float a = __shfl_xor_sync(kFull, h, o), b = __shfl_xor_sync(kFull, l, o);
    float e;
    const bool big = fabsf(h) >= fabsf(a);   // one order in both lanes
    const float x = big ? h : a, y = big ? a : h;
    h = __fadd_rn(x, y);
    e = __fsub_rn(y, __fsub_rn(h, x));
    l = fabsf(h) < INFINITY ? (l + b) + e : 0.f;
}

// the total over the first N lanes of a warp, N a power of two
template <int N>
__device__ __forceinline__ void known_total(Known &k, float sL) {
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) {
        const float mo = __shfl_xor_sync(kFull, k.mo, o), So = __shfl_xor_sync(kFull, k.So, o);
        const float ml = __shfl_xor_sync(kFull, k.ml, o), Sl = __shfl_xor_sync(kFull, k.Sl, o);
        const float a = fmaxf(k.mo, mo), c = fmaxf(k.ml, ml);
        k.So = moved(k.So, k.mo, a, sL) + moved(So, mo, a, sL);
        k.Sl = moved(k.Sl, k.ml, c, sL) + moved(Sl, ml, c, sL);
        k.mo = a;
        k.ml = c;
        pair_total(k.Ph, k.Pl, o);
        pair_total(k.Bh, k.Bl, o);
    }
}
__device__ __forceinline__ Known known_nothing() { return {neg_inf(), 0.f, neg_inf(), 0.f, 0.f, 0.f, 0.f, 0.f}; }

// The factor c of q in the gradient: the teacher's mass, P + p_T, and P alone where
// nothing is unlisted. Where P passes 1, p_T is 0, so that c multiplies the unlisted
// tokens' statistic too. P up to 1 + 2^-15 counts as 1: log-probabilities
// s z - lse of two terms up to 256, each rounded to fp32 by at most 2^-17, are off
// by 2^-16, so a list of the whole mass may come with as much more.
constexpr float kMassOne = 1.f + 0x1p-15f;
__device__ __forceinline__ float mass_factor(int tail, bool rest, float P) {
    return tail && (!rest || P > kMassOne) ? P : 1.f;
}

// what the gradient takes from the row's total
struct Row2 {
    float4 st;        // the statistics
    float qscale;     // the factor of q
    float norm;       // factor of p (1 / P with a renormalised list)
    int rest, none;   // unlisted tokens with mass; no unmasked token at all
    int empty;        // nothing to renormalise
};

// a row's list in shared memory: this part's tokens (-1: none), probabilities
// and logits; the warps' largest logits and log-probabilities of the whole row's
// list; dup: some token is listed twice
struct List {
    int ids[SPEC_MAX_TOP];
    float p[SPEC_MAX_TOP], yl[SPEC_MAX_TOP], top[SPEC_MAX_TOP / 32], lmax[SPEC_MAX_TOP / 32];
    int dup;
};

// y0, the largest unmasked logit of the list (or 0): the loss's terms are taken
// against it, so that rows far from 0 lose nothing
__device__ __forceinline__ float list_top(const List &l) {
    const float m = fmaxf(fmaxf(l.top[0], l.top[1]), fmaxf(l.top[2], l.top[3]));
    static_assert(SPEC_MAX_TOP == 128, "four warps hold a list");
    return m > sv::kMaskFloor ? m : 0.f;
}

// l0, what a list's log-probabilities are taken against: 0, or where only their
// differences count (a renormalised list) the largest one, so that no level of
// them leaves fp32's range. lmax: the four warps' largest
__device__ __forceinline__ float list_level(int tail, const float *lmax) {
    const float m = fmaxf(fmaxf(lmax[0], lmax[1]), fmaxf(lmax[2], lmax[3]));
    return !tail && fabsf(m) < INFINITY ? m : 0.f;
}

// whether entry t is the first of its token
__device__ __forceinline__ bool first_entry(const List &l, int t) {
    const int v = l.ids[t];
    bool f = v >= 0;
    if (l.dup)
        for (int i = 0; i < t && f; ++i) f = l.ids[i] != v;
    return f;
}

// what a warp's 32 entries of the list give; l.p of them is written
__device__ __forceinline__ Known list_known(const DistillArgs &a, List &l, int t, int id, float lp) {
    Known k = known_nothing();
    float ph = 0.f, pl = 0.f, yl = neg_inf();
    const float l0 = list_level(a.tail, l.lmax);
    if (id >= 0) {
        exp_diff(lp, l0, ph, pl);
        yl = l.yl[t];
    }
    l.p[t] = ph;
    const bool there = yl > sv::kMaskFloor;
    k.ml = warp_max(yl);
    k.Sl = warp_sum(first_entry(l, t) ? (there ? ex2((yl - k.ml) * a.sL) : yl == yl ? 0.f : yl) : 0.f);
    k.Ph = ph;
    k.Pl = pl;
    if (id >= 0 && lp - l0 > -700.f) {
        if (there) {   // p (l - l0 - s (y - y0)), each product and sum with its rounding
            float dh, dl, lh, ll;
            two_sum(yl, -list_top(l), dh, dl);
            const float sy = __fmul_rn(a.s, dh), syl = __fmaf_rn(a.s, dh, -sy) + a.s * dl;
            two_sum(lp, -l0, lh, ll);
            two_sum(lh, -sy, dh, dl);
            dl += ll - syl;
            k.Bh = __fmul_rn(ph, dh);
            k.Bl = __fmaf_rn(ph, dh, -k.Bh) + (ph * dl + pl * dh);
        } else {
            k.Bh = INFINITY;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        pair_total(k.Ph, k.Pl, o);
        pair_total(k.Bh, k.Bl, o);
    }
    return k;
}

// the vector with its listed tokens masked
template <typename T>
__device__ __forceinline__ void mask_listed(uint4 &w, uint32_t bits) {
    uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(T) == 2) {
            if (bits >> (2 * k) & 1u) v[k] = (v[k] & 0xffff0000u) | 0xff80u;
            if (bits >> (2 * k + 1) & 1u) v[k] = (v[k] & 0xffffu) | 0xff800000u;
        } else {
            if (bits >> k & 1u) v[k] = 0xff800000u;
        }
    }
    w = make_uint4(v[0], v[1], v[2], v[3]);
}

// U vectors' unlisted tokens into the sum; vector u is the part's i0 + u step.
// Listed tokens are masked in w itself: the gradient there comes later. kFull:
// all of the vectors are in the part.
template <typename T, bool kFull, int U>
__device__ __forceinline__ void fold(DiffSum &acc, uint4 (&w)[U], const uint8_t *map, int i0, int step, int n, float sL,
                                     float resc) {
    constexpr int E = Row<T>::E;
    float cm = neg_inf();
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = i0 + u * step;
        const uint32_t bits = kFull || i < n ? map_vec<T>(map, i) : 0u;
        if (bits) mask_listed<T>(w[u], bits);
        cm = fmaxf(cm, vec_max<T>(w[u]));
    }
    sum_see(acc, cm, sL, resc);
    float v = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float z[E];
        Elem<T>::unpack(w[u], z);
        v += sum_terms<E>(acc, z, sL);
    }
    sum_put(acc, v);
}

// the head's or tail's unlisted token of this thread into the sum
template <typename T>
__device__ __forceinline__ void fold_edge(DiffSum &acc, const Part<T> &part, const uint8_t *map, float sL, float resc) {
    const int i = part.edge(threadIdx.x);
    if (i < 0) return;
    const int bit = map_bit(part, i);
    if (!(map[bit >> 3] >> (bit & 7) & 1)) sum_add1(acc, load1_rw(part.r.p + i), sL, resc);
}

__device__ __forceinline__ float row_max(const Known &k) { return fmaxf(k.mo, k.ml); }
__device__ __forceinline__ float row_sum(const DistillArgs &a, const Known &k, float &qo) {
    const float mx = row_max(k);
    qo = moved(k.So, k.mo, mx, a.sL);
    return qo + moved(k.Sl, k.ml, mx, a.sL);
}
__device__ __forceinline__ float tail_mass(const DistillArgs &a, const Known &k) {
    return a.tail ? fmaxf(0.f, (1.f - k.Ph) - k.Pl) : 0.f;   // 1 - Ph is exact near 1
}

__device__ __forceinline__ Row2 row_of(const DistillArgs &a, const Known &k) {
    const float mx = row_max(k);
    float qo;
    const float Z = row_sum(a, k, qo);
    Row2 r;
    r.rest = k.mo > sv::kMaskFloor || k.So != 0.f;
    r.none = !(mx > sv::kMaskFloor) && Z == 0.f;
    r.empty = !a.tail && k.Ph == 0.f;
    r.st = make_float4(mx, 1.f / Z, k.mo, 0.f);
    if (r.rest) r.st.w = (qo / Z - tail_mass(a, k)) / k.So;
    else r.st.z = neg_inf();
    if (r.none || r.empty) r.st = make_float4(0.f, 0.f, 0.f, 0.f);
    r.qscale = mass_factor(a.tail, r.rest, k.Ph);
    r.norm = a.tail ? 1.f : 1.f / k.Ph;
    return r;
}

// the row's divergence, from its totals, in two floats
__device__ float divergence(const DistillArgs &a, const Known &k, const Row2 &r, float y0) {
    if (r.empty) return 0.f;
    if (r.none) return INFINITY;
    const float mx = row_max(k);
    const float qo = moved(k.So, k.mo, mx, a.sL);
    float Z, Zl;   // with its rounding: the tail's term takes qo / Z again
    two_sum(qo, moved(k.Sl, k.ml, mx, a.sL), Z, Zl);
    // lse - s y0 = s (m - y0) + ln Z
    const Pair lnZ = ln_pair(Z, Zl);
    float lh, ll, h, l;
    two_sum(mx, -y0, h, l);
    const float sm = __fmul_rn(a.s, h), sml = __fmaf_rn(a.s, h, -sm) + a.s * l;
    two_sum(sm, lnZ.h, lh, ll);
    ll += sml + lnZ.l;
    if (a.tail) {   // B + P lse
        const float ph = __fmul_rn(k.Ph, lh);
        two_sum(k.Bh, ph, h, l);
        l += __fmaf_rn(k.Ph, lh, -ph) + (k.Ph * ll + k.Pl * lh) + k.Bl;
    } else {        // B / P - ln P + lse
        const float q = k.Bh / k.Ph;
        const float rem = __fmaf_rn(-q, k.Ph, k.Bh) + (k.Bl - q * k.Pl);
        const Pair lnP = ln_pair(k.Ph, k.Pl);
        float e;
        two_sum(q, lh, h, l);
        two_sum(h, -lnP.h, h, e);
        l += e + rem / k.Ph + ll - lnP.l;
    }
    if (!(fabsf(h) < INFINITY)) return h;
    // p_T ln(p_T / q_T): in two floats, or where the list holds little mass and
    // the divergence is small it would be off by 2^-23; by parts where q_T is below
    // fp32's range
    const float pT = tail_mass(a, k);
    if (r.rest && pT > 0.f) {
        if (qo > 1e-30f) {
            float th, tl, e;
            two_sum(1.f, -k.Ph, th, tl);
            tl -= k.Pl;
            two_sum(th, tl, th, tl);
            const float nh = __fmul_rn(th, Z), nl = __fmaf_rn(th, Z, -nh) + (th * Zl + tl * Z);
            const float qh = nh / qo;
            const Pair ln = ln_pair(qh, (__fmaf_rn(-qh, qo, nh) + nl) / qo);
            const float t = __fmul_rn(th, ln.h);
            l += __fmaf_rn(th, ln.h, -t) + (th * ln.l + tl * ln.h);
            two_sum(h, t, h, e);
            l += e;
        } else {
            l += pT * (logf(pT * Z / k.So) + a.s * (mx - k.mo));
        }
    }
    return h + l;
}

__device__ __forceinline__ void put_loss(const DistillArgs &a, int row, float wt, const Known &k, const Row2 &r, float y0) {
    float qo;
    if (!r.empty && (!(row_max(k) > sv::kMaskFloor) || !(row_sum(a, k, qo) > 0.f) || row_max(k) == -neg_inf()))
        raise_status(a.status, SPEC_ERR_BAD_ROW);
    a.loss[row] = wt * divergence(a, k, r, y0);
    if (a.stats_out) a.stats_out[row] = r.st;
}

// the gradient at listed token entry t, over what was written there before
template <typename T>
__device__ __forceinline__ void put_listed(const DistillArgs &a, const List &l, int t, const Row2 &r, float us, T *pg) {
    if (!first_entry(l, t)) return;
    const int v = l.ids[t];
    float p = l.p[t];
    if (l.dup)
        for (int i = t + 1; i < a.M; ++i) p += l.ids[i] == v ? l.p[i] : 0.f;
    const float yl = l.yl[t];
    const float q = yl > sv::kMaskFloor || yl != yl ? ex2((yl - r.st.x) * a.sL) : 0.f;
    pg[v] = to_elem<T>(fmaf(us * r.st.y * r.qscale, q, -us * (p * r.norm)));
}

template <typename T, bool kGrad, int NT, int U>
__global__ void __launch_bounds__(NT, 1024 / NT) distill_kernel(DistillArgs a, int S, int held) {
    constexpr int E = Row<T>::E, NW = NT / 32;
    extern __shared__ __align__(16) uint8_t s_map[];
    __shared__ List s_list;
    __shared__ Known s_warp[NW], s_known[kMaxCluster], s_total;
    __shared__ Row2 s_row;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x / S, rank = blockIdx.x - row * S;
    const int b = row / a.K, kr = row - b * a.K;
    const T *py = static_cast<const T *>(a.y) + b * a.bs + kr * a.rs;
    const Part<T> part(py, a.V, rank, S);
    const int n = part.n, its = (n + U * NT - 1) / (U * NT);
    const uint4 *body = part.body();
    // whether iteration it is full: all but the last are
    auto full = [&](int it) { return (it + 1) * U * NT <= n; };
    auto load = [&](uint4 (&w)[U], int it) {
        const uint4 *p = body + it * U * NT + tid;
        const uint64_t policy = kGrad && it < its - 2 - held ? l2_keep() : l2_drop();
        if (full(it)) {
#pragma unroll
            for (int u = 0; u < U; ++u) w[u] = ld_stream(p + u * NT, policy);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) w[u] = (it * U + u) * NT + tid < n ? ld_stream(p + u * NT, policy) : masked_vec<T>();
        }
    };
    uint4 w0[U], w1[U];   // iterations it and it + 1; the first is on its way during the list's work
    load(w0, 0);

    const float wt = a.weight ? a.weight[row] : 1.f;
    int id = -1;
    float lp = neg_inf();
    if (tid < a.M) {
        id = a.ids[(size_t)row * a.M + tid];
        lp = a.logp[(size_t)row * a.M + tid];
        if (id >= a.V || id < -1) {
            if (rank == 0) raise_status(a.status, SPEC_ERR_BAD_TOKEN);
            id = -1;
        }
    }
    const uint32_t map_words = (16u + (uint32_t)E * n + 8u + 31u) / 32u;
    for (uint32_t i = tid; i < (map_words + 3u) / 4u; i += NT) reinterpret_cast<uint4 *>(s_map)[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) s_list.dup = 0;
    const bool live = __syncthreads_or(id >= 0) && wt != 0.f;
    T *pg = kGrad ? static_cast<T *>(a.g) + b * a.gbs + kr * a.grs : nullptr;
    const Out<T> out(kGrad ? pg : const_cast<T *>(py), part);
    if (!live) {   // the whole cluster alike
        if (rank == 0 && tid == 0) {
            a.loss[row] = 0.f;
            if (a.stats_out) a.stats_out[row] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (kGrad) zero_part<T, NT>(part, out);
        return;
    }

    if (S > 1) cluster_arrive_relaxed();   // waited for before the exchange: by then every CTA of the cluster runs

    // the part's own entries of the list, and while the row's loads arrive the
    // list's part of what this warp knows
    if (tid < SPEC_MAX_TOP) {
        const float y = id >= 0 ? load1_rw(py + id) : neg_inf(), top = warp_max(y);
        const float lmax = warp_max(id >= 0 ? lp : neg_inf());
        if (lane == 0) {
            s_list.top[warp] = top;
            s_list.lmax[warp] = lmax;
        }
        if (!(id >= part.e0 && id < part.e1)) id = -1;
        s_list.ids[tid] = id;
        if (id >= 0) {
            const int bit = map_bit(part, id);
            const uint32_t m = 1u << (bit & 31);
            if (atomicOr(reinterpret_cast<uint32_t *>(s_map) + (bit >> 5), m) & m) s_list.dup = 1;
            s_list.yl[tid] = y;
        }
    }
    __syncthreads();
    {
        const Known k = warp * 32 < a.M ? list_known(a, s_list, tid, id, lp) : known_nothing();
        if (lane == 0) s_warp[warp] = k;
    }

    DiffSum acc = diff_init(a.resc);
    // `held` iterations before the last two go to shared memory for the second pass
    uint4 *s_held = reinterpret_cast<uint4 *>(s_map + (map_words + 3u) / 4u * 16u) + tid;
    const int held0 = max(its - 2 - held, 0);
    auto work = [&](uint4 (&w)[U], int it) {
        if (full(it)) fold<T, true, U>(acc, w, s_map, it * U * NT + tid, NT, n, a.sL, a.resc);
        else fold<T, false, U>(acc, w, s_map, it * U * NT + tid, NT, n, a.sL, a.resc);
        if (kGrad && it >= held0 && it < its - 2) {
#pragma unroll
            for (int u = 0; u < U; ++u) s_held[((it - held0) * U + u) * NT] = w[u];
        }
    };
    for (int it = 0; it < its; it += 2) {   // both buffers end up with the last two iterations
        if (it + 1 < its) load(w1, it + 1);
        work(w0, it);
        if (it + 1 >= its) break;
        if (it + 2 < its) load(w0, it + 2);
        work(w1, it + 1);
    }
    fold_edge(acc, part, s_map, a.sL, a.resc);

    // every warp's part, the CTA's, the row's
    {
        const float m = warp_max(acc.mx), x = warp_sum(sum_at(acc, m, a.sL));
        if (lane == 0) {
            s_warp[warp].mo = m;
            s_warp[warp].So = x;
        }
    }
    __syncthreads();
    Known all = known_nothing();
    if (warp == 0) {
        if (lane < NW) all = s_warp[lane];
        known_total<NW>(all, a.sL);
        if (S > 1) {
            cluster_wait();
            if (lane < S) {   // each lane one destination
                const uint32_t at = peer(&s_known[rank], lane);
                const unsigned long long *v = reinterpret_cast<const unsigned long long *>(&all);
#pragma unroll
                for (int i = 0; i < (int)(sizeof(Known) / 8); ++i) peer_store(at + 8 * i, v[i]);
            }
        }
    }
    if (S > 1) {
        if (warp != 0) {
            cluster_wait();
            cluster_arrive_relaxed();
        } else {
            cluster_arrive();
        }
        cluster_wait();
        if (warp == 0) {
            all = known_nothing();
            if (lane < S) all = s_known[lane];
            known_total<kMaxCluster>(all, a.sL);
        }
    }
    if (warp == 0) {
        const Row2 r = row_of(a, all);
        if (lane == 0) {
            s_row = r;
            s_total = all;
            if (!kGrad && rank == 0) put_loss(a, row, wt, all, r, list_top(s_list));
        }
    }
    if (!kGrad) return;
    __syncthreads();
    const Row2 r2 = s_row;
    if (r2.empty || r2.none) {
        zero_part<T, NT>(part, out);
    } else {
        const float us = wt * a.s;
        const Factor f = {us * r2.st.w * r2.qscale, r2.rest ? r2.st.z : 0.f};
        // backwards, from the two iterations at hand; the others come again, from L2
        auto grad = [&](uint4 (&w)[U], int it) {
            const int i0 = it * U * NT + tid;
            if (full(it)) {
#pragma unroll
                for (int u = 0; u < U; ++u) grad_vec(part, out, i0 + u * NT, w[u], f, a.sL);
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (i0 + u * NT < n) grad_vec(part, out, i0 + u * NT, w[u], f, a.sL);
            }
            if (it < 2) return;
            if (it - 2 >= held0) {
#pragma unroll
                for (int u = 0; u < U; ++u) w[u] = s_held[((it - 2 - held0) * U + u) * NT];
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) w[u] = ld_rw(body + ((it - 2) * U + u) * NT + tid, l2_drop());
            }
        };
        int it = its - 1;
        if (it >= 0 && (it & 1) == 0) grad(w0, it--);
        for (; it > 0; it -= 2) {
            grad(w1, it);
            grad(w0, it - 1);
        }
        const int i = part.edge(tid);
        if (i >= 0) pg[i] = to_elem<T>(grad_one(f, load1_rw(py + i), a.sL));
        __syncthreads();   // the listed tokens' values go over what was just written
        if (tid < a.M) put_listed(a, s_list, tid, r2, us, pg);
    }
    if (rank == 0 && tid == NT - 1) put_loss(a, row, wt, s_total, r2, list_top(s_list));
}

// the gradient from a row's statistics: a CTA per part of a row
template <typename T, int NT>
__global__ void __launch_bounds__(NT, 4) grad_kernel(DistillArgs a, int parts) {
    __shared__ int s_ids[SPEC_MAX_TOP];
    __shared__ float s_p[SPEC_MAX_TOP];
    __shared__ double s_d[SPEC_MAX_TOP / 32];
    __shared__ float s_f[SPEC_MAX_TOP / 32];
    __shared__ uint32_t s_seen[32];   // a hash of the part's tokens: bits met twice may be a token listed twice
    __shared__ int s_dup;
    const int tid = threadIdx.x;
    const int row = blockIdx.x / parts, rank = blockIdx.x - row * parts;
    const int b = row / a.K, kr = row - b * a.K;
    const T *py = static_cast<const T *>(a.y) + b * a.bs + kr * a.rs;
    T *pg = static_cast<T *>(a.g) + b * a.gbs + kr * a.grs;
    const Part<T> part(py, a.V, rank, parts, UG * NT);
    const Out<T> out(pg, part);
    const int n = part.n;
    const uint4 *body = part.body();
    const float4 st = a.stats_in[row];
    const float us = (a.weight ? a.weight[row] : 1.f) * (a.grad_loss ? a.grad_loss[row] : 1.f) * a.s;
    if (us == 0.f || st.y == 0.f) {
        zero_part<T, NT>(part, out);
        return;
    }
    const bool full = n == UG * NT;
    uint4 w[UG];
    if (full) {
#pragma unroll
        for (int u = 0; u < UG; ++u) w[u] = ld_rw(body + u * NT + tid);
    } else {
#pragma unroll
        for (int u = 0; u < UG; ++u)
            if (u * NT + tid < n) w[u] = ld_rw(body + u * NT + tid);
    }
    if (tid < 32) s_seen[tid] = 0u;
    if (tid == 0) s_dup = 0;
    int id = -1;
    float lp = neg_inf();
    if (tid < a.M) {
        id = a.ids[(size_t)row * a.M + tid];
        lp = a.logp[(size_t)row * a.M + tid];
        if (id >= a.V || id < -1) {
            if (rank == 0) raise_status(a.status, SPEC_ERR_BAD_TOKEN);
            id = -1;
        }
    }
    const bool own = id >= part.e0 && id < part.e1;
    // the list's sum: every part sums the whole list, in more bits where P scales
    // every row, in fp32 (relative error 2^-22 and eight roundings, like q's own)
    // where only a mass above 1 does (0.2 us a call; by exp_diff 0.35)
    const bool rest = st.z != neg_inf(), need = !a.tail || !rest;
    double P = 1.0;
    float p = 0.f;
    if (need) {
        float h = 0.f, l = 0.f, l0 = 0.f;
        if (!a.tail) {
            if (tid < SPEC_MAX_TOP) {
                const float m = warp_max(id >= 0 ? lp : neg_inf());
                if ((tid & 31) == 0) s_f[tid >> 5] = m;
            }
            __syncthreads();
            l0 = list_level(0, s_f);
        }
        if (id >= 0) exp_diff(lp, l0, h, l);
        p = h;
        double x = (double)h + (double)l;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
        if (tid < SPEC_MAX_TOP && (tid & 31) == 0) s_d[tid >> 5] = x;
        __syncthreads();
        P = 0.0;
        for (int i = 0; i < SPEC_MAX_TOP / 32; ++i) P += s_d[i];
    } else if (own) {
        float l;
        exp_diff(lp, 0.f, p, l);
    }
    if (tid < SPEC_MAX_TOP) {
        s_ids[tid] = own ? id : -1;
        s_p[tid] = p;
    }
    const float yl = own ? load1_rw(py + id) : neg_inf();
    if (!need) __syncthreads();   // (the sum's barrier, where there was one)
    if (own) {
        const uint32_t m = 1u << (id & 31);
        if (atomicOr(&s_seen[id >> 5 & 31], m) & m) s_dup = 1;
    }
    const int ei = part.edge(tid);
    const float ey = ei >= 0 ? load1_rw(py + ei) : neg_inf();
    if (!need && tid < SPEC_MAX_TOP) {   // (under the loads)
        const float x = warp_sum(id >= 0 ? ex2(lp * kLog2e) : 0.f);
        if ((tid & 31) == 0) s_f[tid >> 5] = x;
    }
    __syncthreads();   // before anything is overwritten
    const float Pf = need ? (float)P : (s_f[0] + s_f[1]) + (s_f[2] + s_f[3]);
    static_assert(SPEC_MAX_TOP == 128, "four warps hold a list");
    const float c = mass_factor(a.tail, rest, Pf);
    const Factor f = {us * st.w * c, rest ? st.z : 0.f};
    if (full) {
#pragma unroll
        for (int u = 0; u < UG; ++u) grad_vec(part, out, u * NT + tid, w[u], f, a.sL);
    } else {
#pragma unroll
        for (int u = 0; u < UG; ++u)
            if (u * NT + tid < n) grad_vec(part, out, u * NT + tid, w[u], f, a.sL);
    }
    if (ei >= 0) pg[ei] = to_elem<T>(grad_one(f, ey, a.sL));
    __syncthreads();   // the listed tokens' values go over what was just written
    if (own) {
        bool once = true;
        float sum = p;
        if (s_dup) {
            sum = 0.f;
            for (int i = 0; i < a.M; ++i)
                if (s_ids[i] == id) {
                    if (i < tid) once = false;
                    sum += s_p[i];
                }
        }
        if (once) {
            const float kl = us * st.y * c;
            const float q = yl > sv::kMaskFloor || yl != yl ? ex2((yl - st.x) * a.sL) : 0.f;
            pg[id] = to_elem<T>(fmaf(kl, q, -us * (a.tail ? sum : sum * (float)(1.0 / P))));
        }
    }
}

template <typename T, bool kGrad, int NT, int U>
static cudaError_t launch_distill(const DistillArgs &a, int S, cudaStream_t stream) {
    const long long nvec = (long long)a.V / Row<T>::E / S + 1;
    size_t smem = (size_t)((16 + Row<T>::E * nvec + 8 + 31) / 32 + 4) / 4 * 16 + 16;
    // iterations held in shared memory, while 1024 / NT CTAs fit an SM (54 KB each)
    int held = 0;
    if (kGrad) {
        const long long its = (nvec + U * NT - 1) / (U * NT);
        while (held < its - 2 && held < 3 && smem + (size_t)(held + 1) * U * NT * 16 <= 54000 * NT / 256) ++held;
        smem += (size_t)held * U * NT * 16;
    }
    if (smem > 40000) {
        static std::mutex mu;
        static bool done[64];
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        std::lock_guard<std::mutex> lk(mu);
        if (!done[dev & 63]) {
            e = cudaFuncSetAttribute(distill_kernel<T, kGrad, NT, U>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     SPEC_MAX_V / 8 + 256);
            if (e != cudaSuccess) return e;
            done[dev & 63] = true;
        }
    }
    return launch_cluster(distill_kernel<T, kGrad, NT, U>, (unsigned)((long long)a.B * a.K * S), NT, S, smem, stream, a, S, held);
}

template <typename T, bool kLoss, bool kGrad>
cudaError_t launch(const DistillArgs &a, cudaStream_t stream) {
    const long long rows = (long long)a.B * a.K, nvec = (long long)a.V / Row<T>::E;
    if constexpr (!kLoss) {
        const long long parts = nvec <= UG * 256 ? 1 : (nvec + UG * 256 - 1) / (UG * 256);
        if (rows * parts > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
        grad_kernel<T, 256><<<(unsigned)(rows * parts), 256, 0, stream>>>(a, (int)parts);
        return cudaGetLastError();
    } else {
        int S = 1;
        // with the gradient, the 608 / S rows in flight are read twice and have to
        // stay in L2 (116 MB of 129): 2048 rows of 128256 bf16 take 241 us at S = 1,
        // 187 at 2, 208 at 4; 1536 rows of 180000 198 at 2, 207 at 4, of 235000 345
        // at 2, 263 at 4; 2048 rows of 32000 57 at 1, 72 at 2
        if (kGrad)
            while (S < kMaxCluster && 608 / S * (long long)a.V * (long long)sizeof(T) > (116ll << 20)) S *= 2;
        // few rows are split while there are SM slots and a part keeps two vectors
        // per thread: 32 rows of 128256 take 8.1 us at S = 8 and 14.6 at 1, 320 rows
        // 18.1 at 2 and 21.7 at 1 (the loss)
        while (S < kMaxCluster && rows * S * 2 <= 640 && nvec >= 2LL * S * 512) S *= 2;
        return launch_distill<T, kGrad, 256, 4>(a, S, stream);
    }
}

template <bool kLoss, bool kGrad>
int run(const spec_rows_params *p, const void *logits, const float *logprobs, const int32_t *ids, const float *weight,
        const float *grad_loss, const float *stats_in, float *loss, float *stats_out, void *dlogits, int64_t dbs,
        int64_t drs, int32_t *status, void *stream) {
    int rc = check_rows(p, SPEC_MAX_TOP, 4096);
    if (rc != SPEC_OK) return rc;
    if ((int64_t)p->B * p->K == 0) return spec_internal_set_error(SPEC_OK, "");
    const int es = p->dtype == SPEC_BF16 ? 2 : 4;
    rc = check_strided(logits, p->batch_stride, p->row_stride, es, false, p->B, p->K, p->V);
    if (rc != SPEC_OK) return rc;
    if (!logprobs || !ids) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "logprobs / ids is NULL");
    if (kLoss && !loss) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "loss is NULL");
    if (kLoss && !kGrad && !stats_out) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "stats is NULL");
    if (kGrad && !kLoss && !stats_in) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "stats is NULL");
    if ((reinterpret_cast<uintptr_t>(stats_in) | reinterpret_cast<uintptr_t>(stats_out)) % 16)
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "stats must be 16-byte aligned");
    if (kGrad) {
        rc = check_strided(dlogits, dbs, drs, es, true, p->B, p->K, p->V);
        if (rc != SPEC_OK) return rc;
        if (dlogits == logits && ((p->B > 1 && dbs != p->batch_stride) || (p->K > 1 && drs != p->row_stride)))
            return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "in place, dlogits needs the logits' strides");
    }
    spec_internal_set_error(SPEC_OK, "");
    DistillArgs a{};
    a.y = logits;
    a.bs = p->batch_stride;
    a.rs = p->row_stride;
    a.g = dlogits;
    a.gbs = dbs;
    a.grs = drs;
    a.B = p->B;
    a.K = p->K;
    a.V = p->V;
    a.M = p->M;
    a.tail = p->tail;
    a.s = p->inv_temperature;
    a.sL = p->inv_temperature * kLog2e;
    a.resc = sv::kRescale / p->inv_temperature;
    a.logp = logprobs;
    a.ids = ids;
    a.weight = weight;
    a.grad_loss = grad_loss;
    a.stats_in = reinterpret_cast<const float4 *>(stats_in);
    a.loss = loss;
    a.stats_out = reinterpret_cast<float4 *>(stats_out);
    a.status = status;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = es == 2 ? launch<__nv_bfloat16, kLoss, kGrad>(a, st) : launch<float, kLoss, kGrad>(a, st);
    return e == cudaSuccess ? SPEC_OK : spec_internal_set_error(SPEC_ERR_CUDA, cudaGetErrorString(e));
}

}  // namespace sr

extern "C" int spec_distill_loss(const spec_rows_params *p, const void *logits, const float *logprobs,
                                 const int32_t *ids, const float *weight, float *loss, float *stats, int32_t *status,
                                 void *stream) {
    return sr::run<true, false>(p, logits, logprobs, ids, weight, nullptr, nullptr, loss, stats, nullptr, 0, 0, status,
                                stream);
}

extern "C" int spec_distill_grad(const spec_rows_params *p, const void *logits, const float *logprobs,
                                 const int32_t *ids, const float *weight, const float *stats, const float *grad_loss,
                                 void *dlogits, int64_t d_batch_stride, int64_t d_row_stride, int32_t *status,
                                 void *stream) {
    return sr::run<false, true>(p, logits, logprobs, ids, weight, grad_loss, stats, nullptr, nullptr, dlogits,
                                d_batch_stride, d_row_stride, status, stream);
}

extern "C" int spec_distill_step(const spec_rows_params *p, const void *logits, const float *logprobs,
                                 const int32_t *ids, const float *weight, float *loss, void *dlogits,
                                 int64_t d_batch_stride, int64_t d_row_stride, int32_t *status, void *stream) {
    return sr::run<true, true>(p, logits, logprobs, ids, weight, nullptr, nullptr, loss, nullptr, dlogits,
                               d_batch_stride, d_row_stride, status, stream);
}

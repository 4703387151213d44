// spec_beam.cu -- one step of beam search.
//
// A sequence's N best continuations over W beams and V tokens are among each
// beam's N best tokens. One launch: a cluster of C CTAs per sequence, which
// splits every beam's row into P parts where whole rows would not share out
// (W P a multiple of C) and streams its parts through the filter of
// spec_top.cuh. The parts' maxima, sums and bounds meet in every CTA: N
// continuations reach the best part's bound as a score, so only vectors that
// reach it too are looked at, a handful in a whole cluster. Their logits go to
// the first CTA, which ranks them by
//   score = cum + ((z - M) - ln S)
// in two floats. What the order rests on in fewer bits is S alone: every S is off
// by at most kTol / 2 relatively, so two candidates of different beams whose
// scores differ by less than kTol may be in the wrong order. Where that
// touches a selected place, all CTAs sum the beams concerned again in two-float
// arithmetic (relative error 2e-10) and the ranking is repeated.
//
// Measured: 64 sequences of 8 beams, V = 128256 bf16, N = 16: 40 us, 2.9 TB/s of
// the live rows; the stream takes 29 us of it (512 rows in one wave, whose CTAs
// start and end together), the exchange, candidates and ranking the rest; f32 59 us,
// a first step (one live beam each) 35 us. With
// scores compared in fp64 the call took 76 to 119 us, with the top lists as a
// launch of their own 53 us.
#include <mutex>

#include "spec_top.cuh"

namespace sr {

// |relative error of S| <= kTol / 2: exponentials of 2^-22 and their
// arguments' rounding (|y| 2^-25 ln 2, |y| <= 24 where the mass is), and
// at most 32 roundings of 2^-24 on the way of a term into the sum
constexpr float kTol = 8.0e-6f;
constexpr int kMaxUnits = SPEC_MAX_BEAMS * kMaxCluster;   // parts of a sequence

struct BeamArgs {
    const void *z;
    long long bs, rs;
    int B, W, V, N;
    const float *scores;
    const int32_t *finished;
    int32_t eos;
    float *out_scores;
    int32_t *out_parent, *out_token, *out_finished;
    int32_t *status;
};

// a part of the row's two-float sum of e^(z - M), as fp64
template <typename T>
__device__ double precise_sum(const Part<T> &p, float M, double *buf) {
    float H = 0.f, L = 0.f;
    each(p, [&](float z, int) {
        float h, l;
        exp_diff(z, M, h, l);
        add2f(H, L, h, l);
    });
    double S = (double)H + (double)L;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) S += __shfl_xor_sync(kFull, S, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = S;
    __syncthreads();
    S = 0.0;
    for (int i = 0; i < NW; ++i) S += buf[i];
    return S;
}

// Pairs are kept in two floats: GB300's fp64 rate makes the same sums in fp64
// many times slower.
// cum + (z - M) - lnS; below fp32's range -inf (the error terms are NaN there)
__device__ __forceinline__ Pair score_sum(float cum, float z, float M, Pair lnS) {
    float h, l, e;
    two_sum(z, -M, h, l);
    two_sum(h, -lnS.h, h, e);
    l += e - lnS.l;
    two_sum(h, cum, h, e);
    l += e;
    two_sum(h, l, h, l);
    if (!(fabsf(h) < INFINITY)) return {neg_inf(), 0.f};
    return {h, l};
}
// as an integer of the same order
__device__ __forceinline__ unsigned long long score_key(Pair s) {
    const auto ordered = [](float x) {
        const int i = __float_as_int(x + 0.f);
        return i < 0 ? ~(uint32_t)i : (uint32_t)i | 0x80000000u;
    };
    return ((unsigned long long)ordered(s.h) << 32) | ordered(s.l);
}
__device__ __forceinline__ float score_diff(Pair a, Pair b) { return (a.h - b.h) + (a.l - b.l); }

constexpr int kKeep = 128;   // vectors kept of a part when a CTA has several

struct BeamShared {
    TopShared top;
    float u_mx[kMaxUnits], u_sum[kMaxUnits], u_thr[kMaxUnits];   // of every part of the sequence
    float cum[SPEC_MAX_BEAMS];
    float mx[SPEC_MAX_BEAMS], sum[SPEC_MAX_BEAMS];               // of every row
    int state[SPEC_MAX_BEAMS];                                   // 0 live, 1 finished, 2 none
    Pair lnS[SPEC_MAX_BEAMS];
    double prec[SPEC_MAX_BEAMS][kMaxCluster], buf[NW];
    Pair sel[SPEC_MAX_BEAM_OUT + 1];
    int selw[SPEC_MAX_BEAM_OUT + 1], selp[SPEC_MAX_BEAM_OUT + 1];
    unsigned need;   // beams to be summed again
    int count;       // candidates at the first CTA
    int many;        // more candidates than room
};

// At the first CTA: the N + 1 best of cands[0 .. n), into s.sel*; with `check` the beams whose order fp32 sums leave open, into s.need.
// All threads call it; s.selw holds -1 before, a barrier follows.
__device__ __forceinline__ void rank_candidates(const BeamArgs &a, BeamShared &s, unsigned long long *cands,
                                                unsigned long long *keys, int n, bool check) {
    const int tid = threadIdx.x, N = a.N;
    auto score_of = [&](unsigned long long c) -> Pair {
        const int w = (int)(uint32_t)c / a.V;
        if (!cand_key(c)) return {s.cum[w], 0.f};
        return score_sum(s.cum[w], key_value(cand_key(c)), s.mx[w], s.lnS[w]);
    };
    if (n > 64 && check) {   // drop what is well below N + 1 others
        float best = neg_inf();
        for (int i = tid; i < n; i += NT) best = fmaxf(best, score_of(cands[i]).h);
        float bound = block_bound(best, n, N + 1, neg_inf(), s.top.b[2]);
        bound -= 1e-3f + 1e-5f * fabsf(bound);
        if (bound > -1e28f) {   // (the same in every thread)
            for (int i0 = 0; i0 < n; i0 += NT) {   // in place: a round's reads come before its writes
                const int i = i0 + tid;
                const unsigned long long c = i < n ? cands[i] : 0ull;
                const bool want = i < n && score_of(c).h >= bound;
                if (i0 == 0 && tid == 0) s.count = 0;
                __syncthreads();
                const int at = take(want, &s.count);
                if (want) cands[at] = c;
                __syncthreads();
            }
            n = s.count;
        }
    }
    for (int i = tid; i < n; i += NT) keys[i] = score_key(score_of(cands[i]));
    __syncthreads();
    // ranks by counting, G neighbouring lanes per candidate
    const int G = n <= NT / 8 ? 8 : n <= NT / 4 ? 4 : n <= NT / 2 ? 2 : 1, g = tid & (G - 1);
    for (int i0 = 0; i0 < n; i0 += NT / G) {
        const int i = i0 + tid / G;
        const unsigned long long k = i < n ? keys[i] : 0ull;
        const uint32_t place = i < n ? (uint32_t)cands[i] : 0u;
        int rk = 0;
#pragma unroll 4
        for (int o = g; o < n; o += G) {
            const unsigned long long ko = keys[o];
            rk += ko > k || (ko == k && (uint32_t)cands[o] < place);
        }
        for (int o = G / 2; o > 0; o >>= 1) rk += __shfl_xor_sync(kFull, rk, o);
        if (g == 0 && i < n && rk <= N) {
            const Pair sc = score_of(cands[i]);
            if (sc.h > neg_inf()) {
                s.sel[rk] = sc;
                s.selw[rk] = (int)place / a.V;
                s.selp[rk] = (int)place;
            }
        }
    }
    if (!check) return;
    __syncthreads();
    // close neighbours among the selected, and all that is as close behind the last one
    auto flag = [&](int w) {
        if (s.state[w] == 0) atomicOr(&s.need, 1u << w);
    };
    if (tid < N && s.selw[tid] >= 0 && s.selw[tid + 1] >= 0 && s.selw[tid] != s.selw[tid + 1] &&
        score_diff(s.sel[tid], s.sel[tid + 1]) < kTol) {
        flag(s.selw[tid]);
        flag(s.selw[tid + 1]);
    }
    const int wl = s.selw[N - 1];
    if (wl >= 0) {
        const Pair last = s.sel[N - 1];
        for (int i = tid; i < n; i += NT) {
            const int w = (int)(uint32_t)cands[i] / a.V;
            if (w == wl) continue;
            const float d = score_diff(last, score_of(cands[i]));
            if (d >= 0.f && d < kTol) {
                flag(w);
                flag(wl);
            }
        }
    }
}

__device__ __forceinline__ void write_beams(const BeamArgs &a, const BeamShared &s, int b) {
    for (int i = threadIdx.x; i < a.N; i += NT) {
        const size_t o = (size_t)b * a.N + i;
        const int w = s.selw[i];
        const int token = w >= 0 ? s.selp[i] - w * a.V : -1;
        a.out_scores[o] = w >= 0 ? s.sel[i].h : neg_inf();
        a.out_parent[o] = w;
        a.out_token[o] = token;
        a.out_finished[o] = w >= 0 && token == a.eos ? 1 : 0;
    }
}

// Dynamic shared memory: with several parts per CTA their kept vectors (maxima,
// codes); at the first CTA `room` candidates (logit's key and place; key 0: a
// finished beam) and their scores.
template <typename T>
__global__ void __launch_bounds__(NT, 4) beam_kernel(BeamArgs a, int C, int P, int room) {
    constexpr int E = Row<T>::E;
    __shared__ BeamShared s;
    extern __shared__ __align__(16) unsigned char dyn[];
    const int tid = threadIdx.x, lane = tid & 31;
    const int b = blockIdx.x / C, rank = blockIdx.x - b * C;
    const int units = a.W * P, N = a.N;
    const int most = (units + C - 1) / C;          // parts a CTA may have, and
    const int mine = (units - rank + C - 1) / C;   // parts this one has (units >= C)
    unsigned long long *cands = reinterpret_cast<unsigned long long *>(dyn);
    unsigned long long *keys = cands + room;
    float *kept_c = reinterpret_cast<float *>(keys + room);                  // [most][kKeep], most > 1
    int *kept_code = reinterpret_cast<int *>(kept_c + (most > 1 ? most : 0) * kKeep);
    int *kept = kept_code + (most > 1 ? most : 0) * kKeep;                    // [most] vectors kept, -1: too many
    if (C > 1) cluster_arrive_relaxed();   // waited for before the exchange: by then every CTA of the cluster runs
    if (tid < a.W) {
        const size_t row = (size_t)b * a.W + tid;
        const float c = a.scores[row];
        const bool good = c < __int_as_float(0x7f800000);
        if (!good && rank == 0) raise_status(a.status, SPEC_ERR_BAD_ROW);
        s.cum[tid] = c;
        s.state[tid] = !good || c == neg_inf() ? 2 : a.finished && a.finished[row] ? 1 : 0;
    }
    if (tid == 0) {
        s.count = 0;
        s.need = 0u;
        s.many = 0;
    }
    __syncthreads();
    auto part_of = [&](int u) {
        const int w = u / P;
        return Part<T>(static_cast<const T *>(a.z) + b * a.bs + w * a.rs, a.V, u - w * P, P);
    };

    // this CTA's parts
    for (int j = 0; j < mine; ++j) {
        const int u = rank + j * C;
        float mx = neg_inf(), sum = 0.f, thr = sv::kMaskFloor;
        int n = 0;
        if (s.state[u / P] == 0) {
            const Part<T> p = part_of(u);
            stream_part(p, N, kLog2e, sv::kRescale, s.top, thr);
            __syncthreads();
            part_sum(s.top, kLog2e, mx, sum);
            if (far_max(mx, kLog2e)) sum = count_equal(p, mx, s.top);
            n = s.top.n > CAP ? -1 : s.top.n;
        }
        if (most > 1) {   // keep what still reaches the bound
            if (n > 0) {
                for (int i0 = 0; i0 < n; i0 += NT) {
                    const int i = i0 + tid;
                    const bool want = i < n && s.top.c[i] >= thr;
                    const int at = take(want, &s.top.nf);
                    if (want && at < kKeep) {
                        kept_c[j * kKeep + at] = s.top.c[i];
                        kept_code[j * kKeep + at] = s.top.code[i];
                    }
                }
                __syncthreads();
                n = s.top.nf > kKeep ? -1 : s.top.nf;
            }
        }
        if (tid == 0) {
            s.u_mx[u] = mx;
            s.u_sum[u] = sum;
            s.u_thr[u] = thr;
            kept[j] = n;
        }
        if (most > 1) __syncthreads();
    }
    if (C > 1) {
        cluster_wait();
        if (most == 1) __syncwarp();   // written by this warp's first lane
        if (tid < 32)
            for (int i = lane; i < mine * C; i += 32) {   // every part to every CTA
                const int u = rank + i / C * C, to = i % C;
                if (to != rank) {
                    peer_store(peer(&s.u_mx[u], to), s.u_mx[u]);
                    peer_store(peer(&s.u_sum[u], to), s.u_sum[u]);
                    peer_store(peer(&s.u_thr[u], to), s.u_thr[u]);
                }
            }
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }

    // rows from their parts, in every warp: lane w has row w
    float base = __int_as_float(0x7fc00000), mag = 0.f;   // score - lse, roughly; NaN: no continuations
    if (lane < a.W && s.state[lane] == 0) {
        float m = neg_inf(), sum = 0.f;
        for (int i = 0; i < P; ++i) m = fmaxf(m, s.u_mx[lane * P + i]);
        for (int i = 0; i < P; ++i) sum += moved(s.u_sum[lane * P + i], s.u_mx[lane * P + i], m, kLog2e);
        const bool bad = !(sum >= 0.f) || m == -neg_inf();
        if (m > sv::kMaskFloor && !bad) {
            base = s.cum[lane] - (m + logf(sum));
            mag = fabsf(s.cum[lane]) + fabsf(m);
        }
        if (tid < 32) {
            if (rank == 0 && bad) raise_status(a.status, SPEC_ERR_BAD_ROW);
            s.mx[lane] = m;
            s.sum[lane] = sum;
            if (rank == 0) s.lnS[lane] = ln_pair(sum, 0.f);
        }
    }
    // a score that N continuations of one part reach, less these scores'
    // roundings many times over
    float bound = neg_inf();
    for (int u0 = 0; u0 < units; u0 += 32) {
        const int u = min(u0 + lane, units - 1);
        const float bw = __shfl_sync(kFull, base, u / P), thr = s.u_thr[u];
        if (thr > sv::kMaskFloor) bound = fmaxf(bound, bw + thr);   // (the floor is no bound)
    }
    bound = warp_max(bound);
    mag = warp_max(mag);
    bound -= 1e-3f + 1e-5f * (mag + fabsf(bound));
    if (!(bound > -1e28f)) bound = neg_inf();

    // candidates are gathered in s.top.el, then handed over
    auto push = [&](int w, float bw, float z, int index) {
        const uint32_t key = order_key(z);
        if (key == 0u || !(bw + z >= bound)) return;
        const int at = atomicAdd(&s.top.ne, 1);
        if (at < CAPE) s.top.el[at] = ((unsigned long long)key << 32) | (uint32_t)(w * a.V + index);
    };
    bool exact = false;   // every part's N best, found by bisection
    for (;;) {
        __syncthreads();
        if (tid == 0) s.top.ne = 0;
        __syncthreads();
        if (rank == 0 && tid < 32) {   // finished beams, key 0
            const bool fin = lane < a.W && s.state[lane] == 1;
            const unsigned m = __ballot_sync(kFull, fin);
            int at = 0;
            if (lane == 0 && m) at = peer_add(peer(&s.count, 0), __popc(m));
            at = __shfl_sync(kFull, at, 0) + __popc(m & ((1u << lane) - 1u));
            if (fin && at < room) cands[at] = (uint32_t)(lane * a.V + a.eos);
        }
        for (int j = 0; j < mine; ++j) {
            const int u = rank + j * C, w = u / P, n = kept[j];
            const float bw = __shfl_sync(kFull, base, w);
            if (!(bw == bw) || exact || n < 0) continue;   // (the same in every thread)
            const Part<T> p = part_of(u);
            const float *lc = most > 1 ? kept_c + j * kKeep : s.top.c;
            const int *lcode = most > 1 ? kept_code + j * kKeep : s.top.code;
            for (int i = tid; i < n; i += NT) {
                const float c = lc[i];
                if (!(bw + c >= bound)) continue;
                const int code = lcode[i];
                if (code < 0) {
                    push(w, bw, c, ~code);
                    continue;
                }
                float z[E];
                Elem<T>::unpack(__ldg(p.r.body + code), z);
#pragma unroll
                for (int k = 0; k < E; ++k) push(w, bw, z[k], p.r.vec_index(code) + k);
            }
        }
        __syncthreads();
        {   // more than there is room for here counts as more than there is room for there
            const int n = s.top.ne > CAPE ? CAPE + room : s.top.ne;
            hand_over(n, [&](int i) { return s.top.el[min(i, CAPE - 1)]; }, cands, &s.count, room, &s.top.off);
        }
        for (int j = 0; j < mine; ++j) {
            const int u = rank + j * C, w = u / P;
            const float bw = __shfl_sync(kFull, base, w);
            if (!(bw == bw) || !(exact || kept[j] < 0)) continue;
            __syncthreads();
            const int ne = bisect(part_of(u), N, 1u, s.u_mx[u], s.top);
            hand_over(ne, [&](int i) {
                const unsigned long long c = s.top.el[i];
                return ((unsigned long long)cand_key(c) << 32) | (uint32_t)(w * a.V + cand_index(c));
            }, cands, &s.count, room, &s.top.off);
        }
        if (C > 1) {
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
        if (rank == 0) {
            const bool many = s.count > room;
            const int n = many ? 0 : s.count;
            if (tid <= N) s.selw[tid] = -1;
            if (many) {
                if (tid == 0) s.many = 1;
                __syncthreads();   // everyone has read the count
                if (tid == 0) s.count = 0;
            } else {
                rank_candidates(a, s, cands, keys, n, true);
            }
            __syncthreads();
            if (C > 1 && tid > 0 && tid < C) {
                peer_store_u32(peer(&s.need, tid), s.need);
                peer_store_u32(peer(&s.many, tid), many ? 1u : 0u);
            }
        }
        if (C > 1) {
            cluster_arrive();
            if (rank == 0 && !s.many && s.need == 0u) write_beams(a, s, b);
            cluster_wait();
        } else {
            __syncthreads();
            if (!s.many && s.need == 0u) write_beams(a, s, b);
        }
        if (!s.many || exact) break;
        exact = true;
        __syncthreads();
        if (tid == 0) s.many = 0;   // (the first CTA publishes it again before it is read again)
        __syncthreads();
    }
    const unsigned need = s.need;
    if (need == 0u) return;

    // the beams concerned once more, every CTA a part of each
    for (int w = 0; w < a.W; ++w) {
        if (!(need >> w & 1u)) continue;
        const Part<T> p(static_cast<const T *>(a.z) + b * a.bs + w * a.rs, a.V, rank, C);
        const double S = precise_sum(p, s.mx[w], s.buf);
        if (tid == 0) peer_store(peer(&s.prec[w][rank], 0), (unsigned long long)__double_as_longlong(S));
    }
    if (C > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (rank != 0) return;
    if (tid < a.W && need >> tid & 1u) {
        double S = 0.0;
        for (int i = 0; i < C; ++i) S += s.prec[tid][i];
        const float h = (float)S;
        s.lnS[tid] = ln_pair(h, (float)(S - (double)h));
    }
    if (tid <= N) s.selw[tid] = -1;
    __syncthreads();
    rank_candidates(a, s, cands, keys, s.count, false);
    __syncthreads();
    write_beams(a, s, b);
}

// CTAs per sequence and parts per row. Clusters as large as fill the SMs' 608
// slots; parts so that the W P units share out evenly, while a part keeps a
// vector per thread and the candidates of all parts fit (4096). V = 128256 bf16, N =
// 2 W: 64 sequences of 8 beams 47 us, of 5, 7 and 11 beams (several parts a CTA,
// one after another) 76, 100 and 170 us; one sequence of 4, 8 and 16 beams 15, 19
// and 35 us. With several parts a CTA and N near 64 more vectors reach a part's
// bound than are kept of it, and bisection takes over: 32 beams, N = 64, 1286 us.
static void beam_plan(const spec_rows_params *p, int es, int &C, int &P) {
    const long long nvec = (long long)p->V * es / 16;
    C = kMaxCluster;
    while (C > 1 && (long long)p->B * C > 608) C /= 2;
    int g = 1;
    while (g < C && p->K % (2 * g) == 0) g *= 2;
    P = C / g;
    while (P > 1 && (nvec < (long long)P * NT || p->K * P * p->M > 4096)) P /= 2;
    while (C > 1 && p->K * P < C) C /= 2;
}

template <typename T>
static cudaError_t launch_beam(const BeamArgs &a, int C, int P, cudaStream_t stream) {
    const int units = a.W * P, most = (units + C - 1) / C;
    const int room = (units * a.N > 1024 ? units * a.N : 1024) + a.W;
    const size_t smem = (size_t)room * 16 + (most > 1 ? (size_t)most * kKeep * 8 : 0) + (size_t)most * 4;
    static std::mutex mu;
    static bool done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (smem > 8 * 1024) {
        std::lock_guard<std::mutex> lk(mu);
        if (!done[dev & 63]) {
            e = cudaFuncSetAttribute(beam_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 1024);
            if (e != cudaSuccess) return e;
            done[dev & 63] = true;
        }
    }
    return launch_cluster(beam_kernel<T>, (unsigned)(a.B * C), NT, C, smem, stream, a, C, P, room);
}

static int check_beam(const spec_rows_params *p) {
    const int rc = check_rows(p, SPEC_MAX_BEAM_OUT, SPEC_MAX_BEAMS);
    if (rc != SPEC_OK) return rc;
    if (p->K < 1) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "beam_step: K (beams) must be >= 1");
    if (p->tail != 0 || p->inv_temperature != 1.f)
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "beam_step: tail must be 0 and inv_temperature 1");
    return SPEC_OK;
}

}  // namespace sr

extern "C" int spec_beam_step(const spec_rows_params *p, const void *logits, const float *scores,
                              const int32_t *finished, int32_t eos, float *out_scores, int32_t *out_parent,
                              int32_t *out_token, int32_t *out_finished, int32_t *status, void *stream) {
    using namespace sr;
    int rc = check_beam(p);
    if (rc != SPEC_OK) return rc;
    if (eos < -1 || eos >= p->V) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "eos must be -1 or in [0, V)");
    if (finished && eos < 0) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "finished beams need an eos token");
    if (p->B == 0) return spec_internal_set_error(SPEC_OK, "");
    const int es = p->dtype == SPEC_BF16 ? 2 : 4;
    rc = check_strided(logits, p->batch_stride, p->row_stride, es, false, p->B, p->K, p->V);
    if (rc != SPEC_OK) return rc;
    if (!scores || !out_scores || !out_parent || !out_token || !out_finished)
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "beam_step: scores or an output is NULL");
    if ((out_scores == scores || out_finished == finished) && p->M != p->K)
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "beam_step: in place needs N = W");
    spec_internal_set_error(SPEC_OK, "");
    BeamArgs a{};
    a.z = logits;
    a.bs = p->batch_stride;
    a.rs = p->row_stride;
    a.B = p->B;
    a.W = p->K;
    a.V = p->V;
    a.N = p->M;
    a.scores = scores;
    a.finished = finished;
    a.eos = eos;
    a.out_scores = out_scores;
    a.out_parent = out_parent;
    a.out_token = out_token;
    a.out_finished = out_finished;
    a.status = status;
    int C, P;
    beam_plan(p, es, C, P);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = es == 2 ? launch_beam<__nv_bfloat16>(a, C, P, st) : launch_beam<float>(a, C, P, st);
    return e == cudaSuccess ? SPEC_OK : spec_internal_set_error(SPEC_ERR_CUDA, cudaGetErrorString(e));
}

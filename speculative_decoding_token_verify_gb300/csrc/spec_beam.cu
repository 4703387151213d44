// spec_beam.cu -- one step of beam search.
//
// A sequence's N best continuations over W beams and V tokens are among each
// beam's N best tokens. One launch: a cluster of C CTAs per sequence, which
// splits every beam's row into P parts where W parts alone would not share out
// (W P a multiple of C), streams its parts through the filter of spec_top.cuh
// and keeps each part's N best logits. The parts' maxima, sums and N-th best
// meet in every CTA; what can still reach the best part's N-th score goes to
// the first CTA, which ranks it by
//   score = cum + ((z - M) - ln S)
// in fp64. What the order rests on in fewer bits is S alone: every S is off
// by at most kTol / 2 relatively, so two candidates of different beams whose
// scores differ by less than kTol may be in the wrong order. Where that
// touches a selected place, all CTAs sum the beams concerned again in two-float
// arithmetic (relative error about 1e-10) and the ranking is repeated.
#include <mutex>

#include "spec_top.cuh"

namespace sr {

// |relative error of S| <= kTol / 2: exponentials of 2^-22 and their
// arguments' rounding (|y| 2^-25 ln 2, |y| <= 24 where the mass is), and
// at most 32 roundings of 2^-24 on the way of a term into the sum
constexpr double kTol = 8.0e-6;
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

// score s at place p ranks before score o at place op
__device__ __forceinline__ bool before(double s, int p, double o, int op) { return s > o || (s == o && p < op); }

struct BeamShared {
    TopShared top;
    float u_mx[kMaxUnits], u_sum[kMaxUnits], u_nth[kMaxUnits];   // of every part of the sequence
    float cum[SPEC_MAX_BEAMS], base[SPEC_MAX_BEAMS];             // score; score - lse, roughly
    float mx[SPEC_MAX_BEAMS], sum[SPEC_MAX_BEAMS];               // of every row
    int state[SPEC_MAX_BEAMS];                                   // 0 live, 1 finished, 2 none
    double lnS[SPEC_MAX_BEAMS], prec[SPEC_MAX_BEAMS][kMaxCluster], buf[NW];
    double sel[SPEC_MAX_BEAM_OUT + 1];
    int selw[SPEC_MAX_BEAM_OUT + 1], selp[SPEC_MAX_BEAM_OUT + 1];
    float red[2][NW];
    unsigned need;   // beams to be summed again
    int count;       // candidates at the first CTA
};

// Dynamic shared memory: lists [units per CTA][N] (logit's key and place), and
// at the first CTA candidates [W P N + W] and their scores.
template <typename T>
__global__ void __launch_bounds__(NT, TOP_OCC) beam_kernel(BeamArgs a, int C, int P) {
    __shared__ BeamShared s;
    extern __shared__ __align__(16) unsigned char dyn[];
    const int tid = threadIdx.x;
    const int b = blockIdx.x / C, rank = blockIdx.x - b * C;
    const int units = a.W * P, N = a.N;
    const int most = (units + C - 1) / C;               // parts a CTA may have, and
    const int mine = (units - rank + C - 1) / C;        // parts this one has (units >= C)
    unsigned long long *list = reinterpret_cast<unsigned long long *>(dyn);
    unsigned long long *cands = list + (size_t)most * N;
    double *score = reinterpret_cast<double *>(cands + (size_t)units * N + a.W);
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
    }
    __syncthreads();
    auto part_of = [&](int u, int w) {
        return Part<T>(static_cast<const T *>(a.z) + b * a.bs + w * a.rs, a.V, u - w * P, P);
    };

    // this CTA's parts
    for (int j = 0; j < mine; ++j) {
        const int u = rank + j * C, w = u / P;
        float mx = neg_inf(), sum = 0.f;
        int ne = 0;
        if (s.state[w] == 0) {
            const Part<T> p = part_of(u, w);
            float thr;
            bool over = stream_part(p, N, kLog2e, sv::kRescale, s.top, mx, sum, thr);
            if (!over) {
                over = expand(p, thr, s.top, [&](bool want, unsigned long long c) {
                    const int at = take(want, &s.top.ne);
                    if (want && at < CAPE) s.top.el[at] = c;
                });
                __syncthreads();
                ne = s.top.ne;
                over |= ne > CAPE;
            }
            if (over) ne = bisect(p, N, max(order_key(thr), 1u), mx, s.top);
            ne = cut(ne, N, s.top);
            ranked(ne, N, s.top, [&](unsigned long long c, int rk) {
                list[(size_t)j * N + rk] = ((unsigned long long)cand_key(c) << 32) | (uint32_t)(w * a.V + cand_index(c));
                if (rk == N - 1) s.u_nth[u] = key_value(cand_key(c));
            });
        }
        for (int i = ne + tid; i < N; i += NT) list[(size_t)j * N + i] = 0ull;
        if (tid == 0) {
            s.u_mx[u] = mx;
            s.u_sum[u] = sum;
            if (ne < N) s.u_nth[u] = neg_inf();
        }
        __syncthreads();
    }
    if (C > 1) {
        cluster_wait();
        for (int i = tid; i < mine * C; i += NT) {   // every part to every CTA
            const int u = rank + i / C * C, to = i % C;
            if (to != rank) {
                peer_store(peer(&s.u_mx[u], to), s.u_mx[u]);
                peer_store(peer(&s.u_sum[u], to), s.u_sum[u]);
                peer_store(peer(&s.u_nth[u], to), s.u_nth[u]);
            }
        }
        cluster_arrive();
        cluster_wait();
    }

    // rows from their parts
    if (tid < a.W) {
        float m = neg_inf(), sum = 0.f;
        for (int i = 0; i < P; ++i) m = fmaxf(m, s.u_mx[tid * P + i]);
        for (int i = 0; i < P; ++i) {
            const float um = s.u_mx[tid * P + i], us = s.u_sum[tid * P + i];
            sum += um == m || !(us > 0.f) ? us : us * ex2((um - m) * kLog2e);
        }
        if (rank == 0 && s.state[tid] == 0 && (!(sum >= 0.f) || m == -neg_inf())) raise_status(a.status, SPEC_ERR_BAD_ROW);
        s.mx[tid] = m;
        s.sum[tid] = sum;
        s.base[tid] = s.cum[tid] - (m + logf(sum));
    }
    __syncthreads();
    // a score that N continuations of one part reach
    float bound = neg_inf(), mag = 0.f;
    for (int u = tid; u < units; u += NT)
        if (s.state[u / P] == 0) {
            bound = fmaxf(bound, s.base[u / P] + s.u_nth[u]);
            mag = fmaxf(mag, fabsf(s.cum[u / P]) + fabsf(s.mx[u / P]));
        }
    bound = block_max<NT>(bound, s.red[0]);
    mag = block_max<NT>(mag, s.red[1]);
    if (mag < INFINITY) bound -= 1e-3f + 1e-5f * (mag + fabsf(bound));   // these scores' roundings, many times over
    else bound = neg_inf();
    {
        const uint32_t c0 = peer(cands, 0), n0 = peer(&s.count, 0);
        for (int i = tid; i < mine * N; i += NT) {
            const unsigned long long c = list[i];
            if (c == 0ull) continue;
            const int w = (int)(uint32_t)c / a.V;
            if (!(s.base[w] + key_value(cand_key(c)) >= bound)) continue;
            const int at = peer_add(n0, 1);   // room for every list of the sequence
            peer_store(c0 + 8u * at, c);
        }
    }
    if (rank == 0 && tid < a.W && s.state[tid] == 1)   // key 0: a finished beam
        cands[atomicAdd(&s.count, 1)] = (uint32_t)(tid * a.V + a.eos);
    if (C > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }

    for (int round = 0; round < 2; ++round) {
        if (rank == 0) {
            const int n = s.count;
            if (round == 0 && tid < a.W) s.lnS[tid] = log((double)s.sum[tid]);
            if (tid <= N) s.selw[tid] = -1;
            __syncthreads();
            for (int i = tid; i < n; i += NT) {
                const unsigned long long c = cands[i];
                const int w = (int)(uint32_t)c / a.V;
                score[i] = cand_key(c) ? (double)s.cum[w] + (((double)key_value(cand_key(c)) - (double)s.mx[w]) - s.lnS[w])
                                       : (double)s.cum[w];
            }
            __syncthreads();
            for (int i = tid; i < n; i += NT) {
                const double sc = score[i];
                const int place = (int)(uint32_t)cands[i];
                int rk = 0;
                for (int o = 0; o < n; ++o) rk += before(score[o], (int)(uint32_t)cands[o], sc, place);
                if (rk <= N) {
                    s.sel[rk] = sc;
                    s.selw[rk] = place / a.V;
                    s.selp[rk] = place;
                }
            }
            __syncthreads();
            if (round == 0) {
                // close neighbours among the selected, and all that is as close behind the last one
                auto flag = [&](int w) {
                    if (s.state[w] == 0) atomicOr(&s.need, 1u << w);
                };
                if (tid < N && s.selw[tid] >= 0 && s.selw[tid + 1] >= 0 && s.selw[tid] != s.selw[tid + 1] &&
                    s.sel[tid] - s.sel[tid + 1] < kTol) {
                    flag(s.selw[tid]);
                    flag(s.selw[tid + 1]);
                }
                const int wl = s.selw[N - 1];
                if (wl >= 0) {
                    const double last = s.sel[N - 1];
                    for (int i = tid; i < n; i += NT) {
                        const int w = (int)(uint32_t)cands[i] / a.V;
                        if (w != wl && score[i] <= last && last - score[i] < kTol) {
                            flag(w);
                            flag(wl);
                        }
                    }
                }
                __syncthreads();
                if (C > 1 && tid < C && tid > 0) {
                    uint32_t at = peer(&s.need, tid);
                    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(s.need) : "memory");
                }
            }
        }
        if (round == 1) break;
        if (C > 1) {
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
        const unsigned need = s.need;
        if (need == 0u) break;
        for (int w = 0; w < a.W; ++w) {
            if (!(need >> w & 1u)) continue;
            const Part<T> p(static_cast<const T *>(a.z) + b * a.bs + w * a.rs, a.V, rank, C);
            const double S = precise_sum(p, s.mx[w], s.buf);
            if (tid == 0) {
                const uint32_t at = peer(&s.prec[w][rank], 0);
                peer_store(at, (unsigned long long)__double_as_longlong(S));
            }
        }
        if (C > 1) {
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
        if (rank != 0) break;
        if (tid < a.W && need >> tid & 1u) {
            double S = 0.0;
            for (int i = 0; i < C; ++i) S += s.prec[tid][i];
            s.lnS[tid] = log(S);
        }
        __syncthreads();
    }
    if (rank != 0) return;
    for (int i = tid; i < N; i += NT) {
        const size_t o = (size_t)b * N + i;
        const int w = s.selw[i];
        const int token = w >= 0 ? s.selp[i] - w * a.V : -1;
        a.out_scores[o] = w >= 0 ? (float)s.sel[i] : neg_inf();
        a.out_parent[o] = w;
        a.out_token[o] = token;
        a.out_finished[o] = w >= 0 && token == a.eos ? 1 : 0;
    }
}

// CTAs per sequence and parts per row. Clusters as large as fill the SMs' 608
// slots; parts so that the W P units share out evenly, while a part keeps a
// vector per thread and the candidates of all parts fit (4096).
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
    const size_t units = (size_t)a.W * P, most = (units + C - 1) / C;
    const size_t smem = (most * a.N + 2 * (units * a.N + a.W)) * 8;
    static std::mutex mu;
    static bool done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (smem > 12 * 1024) {
        std::lock_guard<std::mutex> lk(mu);
        if (!done[dev & 63]) {
            e = cudaFuncSetAttribute(beam_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 1024);
            if (e != cudaSuccess) return e;
            done[dev & 63] = true;
        }
    }
    return launch_cluster(beam_kernel<T>, (unsigned)(a.B * C), NT, C, smem, stream, a, C, P);
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
    rc = check_strided("logits", logits, p->batch_stride, p->row_stride, es, false, p->B, p->K, p->V);
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

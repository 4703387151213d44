// spec_beam.cu -- one step of beam search, and the reordering of the beams'
// states.
//
// Step: a sequence's N best continuations over W beams and V tokens are among
// each beam's N best tokens. The top-list kernel leaves each beam's list of
// raw logits and its (maximum M, sum S) in the workspace; one CTA per
// sequence ranks the at most W N candidates by
//   score = cum + ((z - M) - ln S)
// in fp64. What the order rests on in fewer bits is S alone: every S is off
// by at most kTol / 2 relatively, so two candidates of different beams whose
// scores differ by less than kTol may be in the wrong order. Where that
// touches a selected place, the beams concerned are summed again in two-float
// arithmetic (relative error below 1e-10) and the ranking is repeated.
#include "spec_rows.cuh"
#include "spec_top.cuh"

namespace sr {

constexpr int NTB = 512;
// |relative error of S| <= kTol / 2: exponentials of 2^-22 and their
// arguments' rounding (|y| 2^-25 ln 2, |y| <= 24 where the mass is), and
// at most 32 roundings of 2^-24 on the way of a term into the sum
constexpr double kTol = 8.0e-6;

struct BeamArgs {
    const void *z;
    long long bs, rs;
    int B, W, V, N, n;   // n = min(N, V): entries per beam's list
    const float *scores;
    const int32_t *finished;
    int32_t eos;
    const float *val;     // [B * W][n]
    const int32_t *ids;
    const float2 *stat;
    float *out_scores;
    int32_t *out_parent, *out_token, *out_finished;
    int32_t *status;
};

// ln of the row's sum against M, from two-float sums
template <typename T>
__device__ double precise_sum(const T *p, int V, float M, double *buf) {
    const Row<T> r(p, V);
    float H = 0.f, L = 0.f;
    auto add = [&](float z) {
        float h, l, e;
        exp_diff(z, M, h, l);
        two_sum(H, h, H, e);
        L += l + e;
    };
    constexpr int E = Row<T>::E;
    if (threadIdx.x < 2 * E) {
        const int i = r.edge_index(threadIdx.x);
        if (i >= 0) add(load1(p + i));
    }
    for (int k = threadIdx.x; k < r.nvec; k += NTB) {
        float z[E];
        Elem<T>::unpack(__ldg(r.body + k), z);
#pragma unroll
        for (int j = 0; j < E; ++j) add(z[j]);
    }
    double S = (double)H + (double)L;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) S += __shfl_xor_sync(kFull, S, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = S;
    __syncthreads();
    S = 0.0;
    for (int i = 0; i < NTB / 32; ++i) S += buf[i];
    return S;
}

// the candidate ranks before another of score o, place op
__device__ __forceinline__ bool before(double s, int p, double o, int op) { return s > o || (s == o && p < op); }

template <typename T>
__global__ void __launch_bounds__(NTB) beam_kernel(BeamArgs a) {
    extern __shared__ double s_score[];   // [W * n]
    int *s_place = reinterpret_cast<int *>(s_score + a.W * a.n);   // [W * n], -1: no candidate
    __shared__ double s_lnS[SPEC_MAX_BEAMS], s_buf[NTB / 32];
    __shared__ double s_sel[SPEC_MAX_BEAM_OUT + 1];
    __shared__ int s_selw[SPEC_MAX_BEAM_OUT + 1];
    __shared__ int s_need[SPEC_MAX_BEAMS], s_any;
    const int b = blockIdx.x, tid = threadIdx.x, C = a.W * a.n;
    if (tid < a.W) {
        const float2 st = a.stat[(size_t)b * a.W + tid];
        s_lnS[tid] = log((double)st.y);   // only read for beams whose rows were read
        s_need[tid] = 0;
    }
    if (tid == 0) s_any = 0;
    __syncthreads();
    for (int round = 0; round < 2; ++round) {
        for (int i = tid; i < C; i += NTB) {
            const int w = i / a.n, j = i - w * a.n;
            const size_t row = (size_t)b * a.W + w;
            const float cum = a.scores[row];
            double sc = -INFINITY;
            int place = -1;
            if (!(cum < __int_as_float(0x7f800000))) {
                if (j == 0) raise_status(a.status, SPEC_ERR_BAD_ROW);
            } else if (cum > neg_inf()) {
                if (a.finished && a.finished[row]) {
                    if (j == 0) {
                        sc = cum;
                        place = w * a.V + a.eos;
                    }
                } else {
                    const int id = a.ids[row * a.n + j];
                    if (id >= 0) {
                        sc = (double)cum + (((double)a.val[row * a.n + j] - (double)a.stat[row].x) - s_lnS[w]);
                        place = w * a.V + id;
                        if (!(sc > -INFINITY && sc < INFINITY)) place = -1;   // a spoilt row
                    }
                }
            }
            s_score[i] = sc;
            s_place[i] = place;
        }
        __syncthreads();
        if (tid <= a.N) s_selw[tid] = -1;
        __syncthreads();
        for (int i = tid; i < C; i += NTB) {
            if (s_place[i] < 0) continue;
            int rank = 0;
            for (int o = 0; o < C; ++o)
                rank += s_place[o] >= 0 && before(s_score[o], s_place[o], s_score[i], s_place[i]);
            if (rank <= a.N) {
                s_sel[rank] = s_score[i];
                s_selw[rank] = i / a.n;
            }
            if (rank < a.N) {
                const size_t o = (size_t)b * a.N + rank;
                a.out_parent[o] = i / a.n;
                const int token = s_place[i] - i / a.n * a.V;
                a.out_token[o] = token;
            }
        }
        __syncthreads();
        if (round == 0) {
            // close neighbours among the selected, and everything that close behind the last one
            auto flag = [&](int w) {
                const bool fin = a.finished && a.finished[(size_t)b * a.W + w];
                if (!fin) {
                    s_need[w] = 1;
                    s_any = 1;
                }
            };
            if (tid < a.N && s_selw[tid] >= 0 && tid + 1 <= a.N && s_selw[tid + 1] >= 0 &&
                s_selw[tid] != s_selw[tid + 1] && s_sel[tid] - s_sel[tid + 1] < kTol) {
                flag(s_selw[tid]);
                flag(s_selw[tid + 1]);
            }
            if (s_selw[a.N - 1] >= 0) {
                const double last = s_sel[a.N - 1];
                const int wl = s_selw[a.N - 1];
                for (int i = tid; i < C; i += NTB)
                    if (s_place[i] >= 0 && i / a.n != wl && s_score[i] <= last && last - s_score[i] < kTol) {
                        flag(i / a.n);
                        flag(wl);
                    }
            }
            __syncthreads();
            if (!s_any) break;
            for (int w = 0; w < a.W; ++w) {
                if (!s_need[w]) continue;
                const size_t row = (size_t)b * a.W + w;
                const T *p = static_cast<const T *>(a.z) + b * a.bs + w * a.rs;
                const double S = precise_sum(p, a.V, a.stat[row].x, s_buf);
                if (tid == 0) s_lnS[w] = log(S);
            }
            __syncthreads();
        }
    }
    for (int i = tid; i < a.N; i += NTB) {
        const size_t o = (size_t)b * a.N + i;
        const bool some = s_selw[i] >= 0;
        a.out_scores[o] = some ? (float)s_sel[i] : neg_inf();
        int token = -1;
        if (some) token = a.out_token[o];
        else a.out_parent[o] = a.out_token[o] = -1;
        a.out_finished[o] = some && token == a.eos ? 1 : 0;
    }
}

struct BeamPlan {
    size_t ids, stat, bytes;
    int n;
};

static BeamPlan beam_plan(const spec_rows_params *p) {
    BeamPlan pl;
    const size_t rows = (size_t)p->B * p->K;
    pl.n = p->M < p->V ? p->M : p->V;
    pl.ids = (rows * pl.n * 4 + 15) & ~(size_t)15;
    pl.stat = pl.ids * 2;
    pl.bytes = pl.stat + rows * 8;
    pl.bytes = (pl.bytes + 15) & ~(size_t)15;
    if (pl.bytes == 0) pl.bytes = 16;
    return pl;
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

extern "C" size_t spec_beam_workspace_size(const spec_rows_params *p) {
    if (sr::check_beam(p) != SPEC_OK) return 0;
    return sr::beam_plan(p).bytes;
}

extern "C" int spec_beam_step(const spec_rows_params *p, const void *logits, const float *scores,
                              const int32_t *finished, int32_t eos, float *out_scores, int32_t *out_parent,
                              int32_t *out_token, int32_t *out_finished, int32_t *status, void *workspace,
                              size_t workspace_bytes, void *stream) {
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
    const BeamPlan pl = beam_plan(p);
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16)
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "workspace must be a 16-byte aligned device pointer");
    if (workspace_bytes < pl.bytes) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "workspace too small");
    spec_internal_set_error(SPEC_OK, "");
    char *ws = static_cast<char *>(workspace);
    TopArgs t{};
    t.z = logits;
    t.batch_stride = p->batch_stride;
    t.row_stride = p->row_stride;
    t.B = p->B;
    t.K = p->K;
    t.V = p->V;
    t.M = pl.n;
    t.s = 1.f;
    t.sL = kLog2e;
    t.rs = sv::kRescale;
    t.val = reinterpret_cast<float *>(ws);
    t.ids = reinterpret_cast<int32_t *>(ws + pl.ids);
    t.stat = reinterpret_cast<float2 *>(ws + pl.stat);
    t.scores = scores;
    t.finished = finished;
    t.status = status;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = launch_top(t, es == 2, st);
    if (e != cudaSuccess) return spec_internal_set_error(SPEC_ERR_CUDA, cudaGetErrorString(e));
    BeamArgs a{};
    a.z = logits;
    a.bs = p->batch_stride;
    a.rs = p->row_stride;
    a.B = p->B;
    a.W = p->K;
    a.V = p->V;
    a.N = p->M;
    a.n = pl.n;
    a.scores = scores;
    a.finished = finished;
    a.eos = eos;
    a.val = t.val;
    a.ids = t.ids;
    a.stat = t.stat;
    a.out_scores = out_scores;
    a.out_parent = out_parent;
    a.out_token = out_token;
    a.out_finished = out_finished;
    a.status = status;
    const size_t smem = (size_t)a.W * a.n * 12;   // <= 32 * 64 * 12 = 24 KB
    if (es == 2) beam_kernel<__nv_bfloat16><<<a.B, NTB, smem, st>>>(a);
    else beam_kernel<float><<<a.B, NTB, smem, st>>>(a);
    e = cudaGetLastError();
    return e == cudaSuccess ? SPEC_OK : spec_internal_set_error(SPEC_ERR_CUDA, cudaGetErrorString(e));
}

// spec_top.cu -- the M largest log-probabilities of every row.
//
// lse = s M + ln S with S = sum_v 2^{(z_v - M) s log2e}, M the row's maximum,
// and the list in the order (logit descending, token ascending), which is the
// order of the log-probabilities without their roundings.
//
// One pass over the row by a cluster of S CTAs (S = 1 when there are rows
// enough), each a part of it, with the filter of spec_top.cuh; the parts'
// bounds, maxima and sums meet in one exchange through distributed shared
// memory, and the first CTA ranks what passes the best bound.
//
// Measured: 2048 rows of 128256 bf16, M = 64: 102 us, 5.2 TB/s, 77% of the
// measured copy rate. The stream with its sums alone takes 86 us; the bounds,
// looking at what passed and ranking it the rest (issue slots 66% busy); f32 175 us,
// 6.0 TB/s, 90%. A CTA
// that goes on to further rows with the next one's first loads in flight took
// 110 us, whole iterations without bounds 105 to 110 us.
#include "spec_top.cuh"

namespace sr {

struct TopArgs {
    const void *z;
    long long batch_stride, row_stride;   // elements
    int B, K, V, M;
    float s, sL, rs;   // inverse temperature, s log2(e); how far a logit may exceed the sum's reference
    float *val;        // [B * K][M]
    int32_t *ids;      // [B * K][M]
    float *lse;        // [B * K] or null
    int32_t *status;
};

template <typename T, bool kCluster>
__global__ void __launch_bounds__(NT, 4) top_kernel(TopArgs a, int S) {
    __shared__ TopShared s;
    __shared__ float s_x[4][kMaxCluster];   // per CTA of the cluster: bound, maximum, sum, overflow
    __shared__ int s_ns;
    const int tid = threadIdx.x;
    const int row = kCluster ? blockIdx.x / S : blockIdx.x;
    const int rank = kCluster ? blockIdx.x - row * S : 0;
    if (kCluster) cluster_arrive_relaxed();   // waited for before the exchange: by then every CTA of the cluster runs
    const int b = row / a.K, kr = row - b * a.K;
    const T *z = static_cast<const T *>(a.z) + b * a.batch_stride + kr * a.row_stride;
    const Part<T> part(z, a.V, rank, kCluster ? S : 1);
    float mx, sum, thr;
    stream_part(part, a.M, a.sL, a.rs, s, thr);
    __syncthreads();
    bool over = s.n > CAP;
    part_sum(s, a.sL, mx, sum);
    if (kCluster) {
        cluster_wait();
        if (tid < S) {
            peer_store(peer(&s_x[0][rank], tid), thr);
            peer_store(peer(&s_x[1][rank], tid), mx);
            peer_store(peer(&s_x[2][rank], tid), sum);
            peer_store(peer(&s_x[3][rank], tid), over ? 1.f : 0.f);
        }
        cluster_arrive();
        cluster_wait();
        mx = neg_inf();
        for (int i = 0; i < S; ++i) {
            thr = fmaxf(thr, s_x[0][i]);
            mx = fmaxf(mx, s_x[1][i]);
            over |= s_x[3][i] != 0.f;
        }
        sum = 0.f;
        for (int i = 0; i < S; ++i) sum += moved(s_x[2][i], s_x[1][i], mx, a.sL);
    }
    // to the cluster's first CTA, by way of the list of passing vectors, which
    // is read by then; a part with too many gives up for the row, by a count
    // beyond the room
    if (kCluster && tid == 0) s_ns = 0;
    if (!over) {
        unsigned long long *stage = reinterpret_cast<unsigned long long *>(s.c);
        const bool many = expand(part, thr, s, kCluster ? stage : s.el, kCluster ? &s_ns : &s.ne);
        if (kCluster) {
            __syncthreads();
            hand_over(many ? CAPE + 1 : s_ns, [&](int i) { return stage[min(i, CAPE - 1)]; }, s.el, &s.ne, CAPE, &s.off);
        } else if (many && tid == 0) {
            s.ne = CAPE + 1;
        }
    }
    if (kCluster) {
        cluster_arrive();
        cluster_wait();
        if (rank != 0) return;
    } else {
        __syncthreads();
    }
    int ne = s.ne;
    if (over || ne > CAPE) ne = bisect(Part<T>(z, a.V, 0, 1), a.M, max(order_key(thr), 1u), mx, s);
    ne = cut(ne, a.M, s);
    if (far_max(mx, a.sL)) sum = count_equal(Part<T>(z, a.V, 0, 1), mx, s);
    const bool some = mx > sv::kMaskFloor, bad = !(sum >= 0.f) || mx == -neg_inf();
    const float lnS = logf(sum);
    ranked(ne, a.M, s, [&](unsigned long long c, int rk) {
        a.val[(size_t)row * a.M + rk] = fmaf(key_value(cand_key(c)) - mx, a.s, -lnS);
        a.ids[(size_t)row * a.M + rk] = cand_index(c);
    });
    for (int i = ne + tid; i < a.M; i += NT) {
        a.val[(size_t)row * a.M + i] = neg_inf();
        a.ids[(size_t)row * a.M + i] = -1;
    }
    if (tid == 0) {
        if (a.lse) a.lse[row] = bad ? __int_as_float(0x7fc00000) : some ? fmaf(mx, a.s, lnS) : neg_inf();
        if (bad) raise_status(a.status, SPEC_ERR_BAD_ROW);
    }
}

// CTAs per row: rows are split while half of the SMs' slots (4 CTAs on each of
// 152 SMs) are free and a part keeps four vectors per thread: an exchange
// costs more than it saves beyond. bf16, M = 64, S = 1 / 2 / 4 / 8: 8 rows of
// 128256 16.3 / 13.8 / 12.0 / 10.6 us, 128 rows 16.7 / 16.4 / 19.3 / 24.7 us;
// 128 rows of 32000 10.1 / 11.3 / 14.1 / 20.7 us.
static int top_cluster(long long rows, int V, int es) {
    const long long nvec = (long long)V * es / 16;
    int S = 1;
    while (S < kMaxCluster && rows * S * 2 <= 304 && nvec >= 2LL * S * U * NT) S *= 2;
    return S;
}

template <typename T>
static cudaError_t launch_t(const TopArgs &a, cudaStream_t stream) {
    const long long rows = (long long)a.B * a.K;
    const int S = top_cluster(rows, a.V, sizeof(T));
    if (S > 1) return launch_cluster(top_kernel<T, true>, (unsigned)(rows * S), NT, S, 0, stream, a, S);
    return launch_cluster(top_kernel<T, false>, (unsigned)rows, NT, 1, 0, stream, a, 1);
}

static cudaError_t launch_top(const TopArgs &a, int bf16, cudaStream_t stream) {
    return bf16 ? launch_t<__nv_bfloat16>(a, stream) : launch_t<float>(a, stream);
}

int check_rows(const spec_rows_params *p, int max_m, int max_k) {
    if (!p) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "params is NULL");
    if (p->reserved != 0) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "params.reserved must be 0");
    if (p->B < 0 || p->K < 0) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "B and K must be >= 0");
    if (p->B > SPEC_MAX_B) return spec_internal_set_error(SPEC_ERR_UNSUPPORTED, "B must be <= 2^24");
    if (p->K > max_k) return spec_internal_set_error(SPEC_ERR_UNSUPPORTED, "too many rows per sequence (K)");
    if ((int64_t)p->B * p->K > (1 << 27)) return spec_internal_set_error(SPEC_ERR_UNSUPPORTED, "B * K must be <= 2^27");
    if (p->V < 1 || p->V > SPEC_MAX_V) return spec_internal_set_error(SPEC_ERR_UNSUPPORTED, "V must be in [1, 2^20]");
    if (p->dtype != SPEC_F32 && p->dtype != SPEC_BF16) return spec_internal_set_error(SPEC_ERR_UNSUPPORTED, "unknown dtype");
    if (p->M < 1 || p->M > max_m) return spec_internal_set_error(SPEC_ERR_UNSUPPORTED, "list length (M) out of range");
    if (p->tail != 0 && p->tail != 1) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "tail must be 0 or 1");
    if (!(p->inv_temperature >= SPEC_MIN_INV_TEMPERATURE && p->inv_temperature <= SPEC_MAX_INV_TEMPERATURE))
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "inv_temperature must be in [1e-4, 1e4]");
    return SPEC_OK;
}

// Strides of an input are >= 0. Rows of an output must not overlap: one of the
// two axes steps over the whole extent of the other.
int check_strided(const void *base, int64_t bs, int64_t rs, int es, bool out, int B, int K, int V) {
    if (!base) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "logits / dlogits is NULL");
    if (reinterpret_cast<uintptr_t>(base) % es)
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "logits / dlogits must be aligned to the element size");
    if (bs < 0 || rs < 0) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "strides must be >= 0");
    if ((B > 1 && bs > (INT64_MAX >> 4) / B) || (K > 1 && rs > (INT64_MAX >> 4) / K))
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "strides are too large");
    if (out) {
        const bool rows_inside = (K <= 1 || rs >= V) && (B <= 1 || bs >= (K - 1) * rs + V);
        const bool batch_inside = (B <= 1 || bs >= V) && (K <= 1 || rs >= (B - 1) * bs + V);
        if (!rows_inside && !batch_inside)
            return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "rows of an output overlap");
    }
    return SPEC_OK;
}

}  // namespace sr

extern "C" int spec_top_logprobs(const spec_rows_params *p, const void *logits, float *logprobs, int32_t *ids,
                                 float *lse, int32_t *status, void *stream) {
    using namespace sr;
    int rc = check_rows(p, SPEC_MAX_TOP, 4096);
    if (rc != SPEC_OK) return rc;
    if (p->tail != 0) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "top_logprobs: tail must be 0");
    if ((int64_t)p->B * p->K == 0) return spec_internal_set_error(SPEC_OK, "");
    rc = check_strided(logits, p->batch_stride, p->row_stride, p->dtype == SPEC_BF16 ? 2 : 4, false, p->B,
                       p->K, p->V);
    if (rc != SPEC_OK) return rc;
    if (!logprobs || !ids) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "logprobs / ids is NULL");
    spec_internal_set_error(SPEC_OK, "");
    TopArgs a{};
    a.z = logits;
    a.batch_stride = p->batch_stride;
    a.row_stride = p->row_stride;
    a.B = p->B;
    a.K = p->K;
    a.V = p->V;
    a.M = p->M;
    a.s = p->inv_temperature;
    a.sL = p->inv_temperature * sv::kLog2e;
    a.rs = sv::kRescale / p->inv_temperature;
    a.val = logprobs;
    a.ids = ids;
    a.lse = lse;
    a.status = status;
    const cudaError_t e = launch_top(a, p->dtype == SPEC_BF16, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPEC_OK : spec_internal_set_error(SPEC_ERR_CUDA, cudaGetErrorString(e));
}

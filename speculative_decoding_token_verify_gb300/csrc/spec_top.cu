// spec_top.cu -- the M largest log-probabilities of every row.
//
// lse = s M + ln S with S = sum_v 2^{(z_v - M) s log2e}, M the row's maximum,
// and the list in the order (logit descending, token ascending), which is the
// order of the log-probabilities without their roundings.
//
// One CTA per row. The list's threshold, the M-th largest key, is found by
// bisection over the 32-bit ordered keys: 32 counting passes over the row,
// served by L2 after the first. Tokens above the threshold are collected in
// any order, tokens at the threshold in ascending order until the list is
// full; a rank by counting sorts them.
#include "spec_top.cuh"

#include "spec_rows.cuh"

namespace sr {

constexpr int NT = 512;

template <typename T, typename F>
__device__ __forceinline__ void each(const Row<T> &r, F f) {
    constexpr int E = Row<T>::E;
    if (threadIdx.x < 2 * E) {
        const int i = r.edge_index(threadIdx.x);
        if (i >= 0) f(load1(r.p + i), i);
    }
    for (int k = threadIdx.x; k < r.nvec; k += NT) {
        float z[E];
        Elem<T>::unpack(__ldg(r.body + k), z);
#pragma unroll
        for (int j = 0; j < E; ++j) f(z[j], r.vec_index(k) + j);
    }
}

template <typename T>
__global__ void __launch_bounds__(NT) top_kernel(TopArgs a) {
    __shared__ float fbuf[2][NT / 32];
    __shared__ int s_n;
    __shared__ int s_cnt[NT / 32];
    __shared__ unsigned long long s_cand[SPEC_MAX_TOP];
    const int row = blockIdx.x;
    const int b = row / a.K, k = row - b * a.K;
    if (a.scores) {
        const float sc = a.scores[row];
        if (!(sc > neg_inf()) || sc == -neg_inf() || (a.finished && a.finished[row])) return;
    }
    const Row<T> r(static_cast<const T *>(a.z) + b * a.batch_stride + k * a.row_stride, a.V);
    Sum acc = sum_init(a.sL, a.rs);
    each(r, [&](float z, int) { sum_add1(acc, z, a.sL, a.rs); });
    const float mx = block_max<NT>(acc.mx, fbuf[0]);
    const bool some = mx > sv::kMaskFloor;
    const float S = block_sum<NT>(some || acc.S != 0.f ? sum_at(acc, mx, a.sL) : 0.f, fbuf[1]);
    const bool bad = !(S >= 0.f) || mx == -neg_inf();

    auto count = [&](uint32_t t) {   // tokens of key >= t, t > 0
        int n = 0;
        each(r, [&](float z, int) { n += order_key(z) >= t; });
        n = __reduce_add_sync(kFull, n);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) s_cnt[threadIdx.x >> 5] = n;
        __syncthreads();
        n = 0;
        for (int i = 0; i < NT / 32; ++i) n += s_cnt[i];
        return n;
    };
    // the largest t with count(t) >= M, or 1 when the row has fewer tokens
    uint32_t t = 1;
    if (count(1u) > a.M) {
        uint32_t hi = order_key(mx);   // count(hi + 1) == 0 < M
        while (t < hi) {
            const uint32_t mid = t + (hi - t) / 2 + ((hi - t) & 1u);
            if (count(mid) >= a.M) t = mid;
            else hi = mid - 1;
        }
    }
    if (threadIdx.x == 0) s_n = 0;
    __syncthreads();
    const bool all = t == 1u;
    each(r, [&](float z, int i) {
        const uint32_t key = order_key(z);
        if (all ? key >= 1u : key > t) {
            const int at = atomicAdd(&s_n, 1);
            if (at < a.M) s_cand[at] = cand(key, i);
        }
    });
    __syncthreads();
    int n = min(s_n, a.M);
    if (!all) {   // tokens at the threshold, lowest index first
        for (int i0 = 0; i0 < a.V && n < a.M; i0 += NT) {
            const int i = i0 + threadIdx.x;
            const bool at = i < a.V && order_key(load1(r.p + i)) == t;
            const unsigned bal = __ballot_sync(kFull, at);
            __syncthreads();
            if ((threadIdx.x & 31) == 0) s_cnt[threadIdx.x >> 5] = __popc(bal);
            __syncthreads();
            int before = n + __popc(bal & ((1u << (threadIdx.x & 31)) - 1u)), total = 0;
            for (int w = 0; w < NT / 32; ++w) {
                before += w < (int)(threadIdx.x >> 5) ? s_cnt[w] : 0;
                total += s_cnt[w];
            }
            if (at && before < a.M) s_cand[before] = cand(t, i);
            n = min(n + total, a.M);
        }
        __syncthreads();
    }
    const float lnS = logf(S);
    if (threadIdx.x < a.M) {
        int rank = threadIdx.x;
        float v = neg_inf();
        int id = -1;
        if (threadIdx.x < n) {
            const unsigned long long c = s_cand[threadIdx.x];
            rank = 0;
            for (int i = 0; i < n; ++i) rank += s_cand[i] > c;
            const float z = key_value(cand_key(c));
            v = a.stat ? z : fmaf(z - mx, a.s, -lnS);
            id = cand_index(c);
        }
        a.val[(size_t)row * a.M + rank] = v;
        a.ids[(size_t)row * a.M + rank] = id;
    }
    if (threadIdx.x == 0) {
        if (a.stat) a.stat[row] = make_float2(mx, S);
        if (a.lse) a.lse[row] = bad ? __int_as_float(0x7fc00000) : some ? fmaf(mx, a.s, lnS) : neg_inf();
        if (bad) raise_status(a.status, SPEC_ERR_BAD_ROW);
    }
}

cudaError_t launch_top(const TopArgs &a, int bf16, cudaStream_t stream) {
    if (bf16) top_kernel<__nv_bfloat16><<<a.B * a.K, NT, 0, stream>>>(a);
    else top_kernel<float><<<a.B * a.K, NT, 0, stream>>>(a);
    return cudaGetLastError();
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
int check_strided(const char *name, const void *base, int64_t bs, int64_t rs, int es, bool out, int B, int K, int V) {
    (void)name;
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
    rc = check_strided("logits", logits, p->batch_stride, p->row_stride, p->dtype == SPEC_BF16 ? 2 : 4, false, p->B,
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

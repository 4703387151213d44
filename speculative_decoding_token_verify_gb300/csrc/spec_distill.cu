// spec_distill.cu -- distillation of a student's rows from a teacher's top
// lists: loss, gradient by the student's logits, both in one call.
//
// With q = softmax(s y), the list's probabilities p_m, the unlisted tokens'
// teacher mass p_T = 1 - P and student mass q_T:
//   KL = sum_m p_m (l_m - ln q(id_m)) + p_T (ln p_T - ln q_T)
//   dKL / dy_v = s (q_v - sum_m p_m [id_m = v])   at listed v
//              = s (q_T - p_T) r_v                at unlisted v,
// r = the softmax over the unlisted tokens alone: their part of q rescaled to
// the teacher's mass.
//
// The unlisted tokens have a maximum and a sum of their own, so neither q_T =
// 1 - Q (which cancels when the list holds nearly all of the mass) nor q_T /
// p_T (which leaves fp32's range when it holds yet more) is ever formed: the
// list's tokens are marked in a bit map of the row in shared memory, looked up
// once per 16-byte vector. p_T = 1 - P is formed in fp64, as are the list's
// terms of the loss: fp64 costs M exponentials per row beside V fp32 ones.
#include <mutex>

#include "spec_rows.cuh"

namespace sr {

constexpr int NT = 512;

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

template <typename T>
__device__ __forceinline__ T to_elem(float v);
template <>
__device__ __forceinline__ float to_elem<float>(float v) {
    return v;
}
// one rounding to nearest, the gradient's only one below fp32
template <>
__device__ __forceinline__ __nv_bfloat16 to_elem<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

// bit of element v in the row's map: head and body keep a vector's bits in one word
template <typename T>
__device__ __forceinline__ int map_bit(const Row<T> &r, int v) {
    return v - r.head + Row<T>::E;
}

template <typename T, bool kLoss, bool kGrad>
__global__ void __launch_bounds__(NT) distill_kernel(DistillArgs a) {
    constexpr int E = Row<T>::E;
    extern __shared__ uint32_t s_map[];
    __shared__ float fbuf[4][NT / 32];
    __shared__ double dbuf[2][SPEC_MAX_TOP / 32];
    __shared__ int s_ids[SPEC_MAX_TOP];
    __shared__ float s_p[SPEC_MAX_TOP];
    __shared__ float4 s_stats;
    const int row = blockIdx.x, tid = threadIdx.x;
    const int b = row / a.K, k = row - b * a.K;
    const T *py = static_cast<const T *>(a.y) + b * a.bs + k * a.rs;
    T *pg = kGrad ? static_cast<T *>(a.g) + b * a.gbs + k * a.grs : nullptr;
    const Row<T> r(py, a.V);

    float w = a.weight ? a.weight[row] : 1.f;
    int id = -1;
    float lp = neg_inf();
    if (tid < a.M) {
        id = a.ids[(size_t)row * a.M + tid];
        if (id >= a.V || id < -1) {
            raise_status(a.status, SPEC_ERR_BAD_TOKEN);
            id = -1;
        }
        if (id >= 0) lp = a.logp[(size_t)row * a.M + tid];
    }
    float4 st = make_float4(0.f, 0.f, 0.f, 0.f);
    bool live = __syncthreads_or(id >= 0) && w != 0.f;
    float up = w;   // the gradient's factor
    if (kGrad && !kLoss) {
        if (a.grad_loss) up *= a.grad_loss[row];
        st = a.stats_in[row];
        live = live && up != 0.f && st.y != 0.f;
    }
    auto dead_row = [&] {
        if (kLoss && tid == 0) {
            a.loss[row] = 0.f;
            if (a.stats_out) a.stats_out[row] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (kGrad)
            for (int v = tid; v < a.V; v += NT) pg[v] = to_elem<T>(0.f);
    };
    if (!live) {
        dead_row();
        return;
    }

    // the list: probabilities, their sum, the student's logits there
    const double p64 = id >= 0 ? exp((double)lp) : 0.0;
    double P = p64;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) P += __shfl_xor_sync(kFull, P, o);
    if (tid < SPEC_MAX_TOP && (tid & 31) == 0) dbuf[0][tid >> 5] = P;
    if (tid < SPEC_MAX_TOP) s_ids[tid] = id;
    if (kLoss)
        for (int i = tid; i < (a.V + 2 * E + 31) / 32; i += NT) s_map[i] = 0u;
    __syncthreads();
    P = 0.0;
    for (int i = 0; i < SPEC_MAX_TOP / 32; ++i) P += dbuf[0][i];
    if (!a.tail && P == 0.0) {   // nothing to renormalise: an empty list
        dead_row();
        return;
    }
    const double pn = a.tail ? p64 : p64 / P;
    if (tid < SPEC_MAX_TOP) s_p[tid] = (float)pn;
    const float yl = id >= 0 ? load1_rw(py + id) : neg_inf();
    bool first = id >= 0;   // of the entries with this token
    for (int i = 0; i < tid && i < a.M && first; ++i) first = s_ids[i] != id;

    if (kLoss) {
        if (id >= 0) {
            const int bit = map_bit(r, id);
            atomicOr(&s_map[bit >> 5], 1u << (bit & 31));
        }
        __syncthreads();
        // unlisted tokens' sum, all tokens' maximum
        Sum acc = sum_init(a.sL, a.resc);
        if (tid < 2 * E) {
            const int i = r.edge_index(tid);
            if (i >= 0) {
                const int bit = map_bit(r, i);
                const float z = load1(py + i);
                if (!(s_map[bit >> 5] >> (bit & 31) & 1u)) sum_add1(acc, z, a.sL, a.resc);
            }
        }
        for (int i = tid; i < r.nvec; i += NT) {
            const uint4 v = __ldg(r.body + i);
            float z[E];
            Elem<T>::unpack(v, z);
            float c = vec_max<T>(v);
            const uint32_t bits = s_map[(E * (i + 1)) >> 5] >> ((E * (i + 1)) & 31) & ((1u << E) - 1u);
            if (bits) {
#pragma unroll
                for (int j = 0; j < E; ++j) z[j] = bits >> j & 1u ? neg_inf() : z[j];
                c = z[0];
#pragma unroll
                for (int j = 1; j < E; ++j) c = fmaxf(c, z[j]);
            }
            sum_see(acc, c, a.sL, a.resc);
            sum_put(acc, sum_terms<E>(acc, z, a.sL));
        }
        const float mo = block_max<NT>(acc.mx, fbuf[0]);
        const float So = block_sum<NT>(sum_at(acc, mo, a.sL), fbuf[1]);
        const float mx = fmaxf(mo, block_max<NT>(yl, fbuf[2]));
        const bool rest = mo > sv::kMaskFloor, some = mx > sv::kMaskFloor;
        const float e = first && some ? ex2((yl - mx) * a.sL) : 0.f;
        // a NaN among the unlisted stays in the sum
        const float S = block_sum<NT>(e, fbuf[3]) + (rest ? So * ex2((mo - mx) * a.sL) : So);
        // the list's terms
        const double lnS = log((double)S);
        double t = 0.0;
        if (id >= 0 && pn > 0.0) {
            const double lq = yl > sv::kMaskFloor ? (double)a.s * ((double)yl - (double)mx) - lnS : -INFINITY;
            t = pn * ((a.tail ? (double)lp : (double)lp - log(P)) - lq);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(kFull, t, o);
        if (tid < SPEC_MAX_TOP && (tid & 31) == 0) dbuf[1][tid >> 5] = t;
        __syncthreads();
        if (tid == 0) {
            double kl = 0.0;
            for (int i = 0; i < SPEC_MAX_TOP / 32; ++i) kl += dbuf[1][i];
            const double pT = a.tail ? fmax(0.0, 1.0 - P) : 0.0;
            st = make_float4(mx, 1.f / S, neg_inf(), 0.f);
            if (rest || So != 0.f) {
                const double lqT = (double)a.s * ((double)mo - (double)mx) + log((double)So) - lnS;
                if (pT > 0.0) kl += pT * (log(pT) - lqT);
                st.z = mo;
                st.w = (float)((exp(lqT) - pT) / (double)So);
            }
            if (!some || !(S > 0.f) || mx == -neg_inf()) raise_status(a.status, SPEC_ERR_BAD_ROW);
            if (!some && S == 0.f) {   // no unmasked token
                kl = INFINITY;
                st = make_float4(0.f, 0.f, 0.f, 0.f);
            }
            a.loss[row] = w * (float)kl;
            if (a.stats_out) a.stats_out[row] = st;
            s_stats = st;
        }
        __syncthreads();
        st = s_stats;
    } else {
        __syncthreads();
    }

    if (kGrad) {
        const float us = up * a.s;
        // listed: us (kl e^{s (y - m)} - p); unlisted: ku e^{s (y - m_o)}
        const float kl = us * st.y * (a.tail && st.z == neg_inf() ? (float)P : 1.f), ku = us * st.w;
        if (st.y == 0.f) {
            for (int v = tid; v < a.V; v += NT) pg[v] = to_elem<T>(0.f);
            return;
        }
        for (int v = tid; v < a.V; v += NT) {
            const float y = load1_rw(py + v);
            pg[v] = to_elem<T>(ku * (y > sv::kMaskFloor ? ex2((y - st.z) * a.sL) : 0.f));
        }
        __syncthreads();   // the listed tokens' values go over what was just written
        if (first) {
            float p = 0.f;
            for (int i = tid; i < a.M; ++i) p += s_ids[i] == id ? s_p[i] : 0.f;
            const float q = yl > sv::kMaskFloor ? ex2((yl - st.x) * a.sL) : 0.f;
            pg[id] = to_elem<T>(fmaf(kl, q, -us * p));
        }
    }
}

template <typename T, bool kLoss, bool kGrad>
cudaError_t launch(const DistillArgs &a, cudaStream_t stream) {
    const size_t smem = kLoss ? ((size_t)a.V + 2 * Row<T>::E + 31) / 32 * 4 : 0;
    if (smem > 40000) {
        static std::mutex mu;
        static bool done[64];
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        std::lock_guard<std::mutex> lk(mu);
        if (!done[dev & 63]) {
            e = cudaFuncSetAttribute(distill_kernel<T, kLoss, kGrad>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     SPEC_MAX_V / 8 + 64);
            if (e != cudaSuccess) return e;
            done[dev & 63] = true;
        }
    }
    distill_kernel<T, kLoss, kGrad><<<a.B * a.K, NT, smem, stream>>>(a);
    return cudaGetLastError();
}

template <bool kLoss, bool kGrad>
int run(const spec_rows_params *p, const void *logits, const float *logprobs, const int32_t *ids, const float *weight,
        const float *grad_loss, const float *stats_in, float *loss, float *stats_out, void *dlogits, int64_t dbs,
        int64_t drs, int32_t *status, void *stream) {
    int rc = check_rows(p, SPEC_MAX_TOP, 4096);
    if (rc != SPEC_OK) return rc;
    if ((int64_t)p->B * p->K == 0) return spec_internal_set_error(SPEC_OK, "");
    const int es = p->dtype == SPEC_BF16 ? 2 : 4;
    rc = check_strided("logits", logits, p->batch_stride, p->row_stride, es, false, p->B, p->K, p->V);
    if (rc != SPEC_OK) return rc;
    if (!logprobs || !ids) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "logprobs / ids is NULL");
    if (kLoss && !loss) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "loss is NULL");
    if (kLoss && !kGrad && !stats_out) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "stats is NULL");
    if (kGrad && !kLoss && !stats_in) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "stats is NULL");
    if ((reinterpret_cast<uintptr_t>(stats_in) | reinterpret_cast<uintptr_t>(stats_out)) % 16)
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "stats must be 16-byte aligned");
    if (kGrad) {
        rc = check_strided("dlogits", dlogits, dbs, drs, es, true, p->B, p->K, p->V);
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

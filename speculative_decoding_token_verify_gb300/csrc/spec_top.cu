// spec_top.cu -- the M largest log-probabilities of every row.
//
// lse = s M + ln S with S = sum_v 2^{(z_v - M) s log2e}, M the row's maximum,
// and the list in the order (logit descending, token ascending), which is the
// order of the log-probabilities without their roundings.
//
// One pass. A cluster of S CTAs streams a row (S = 1 when there are rows
// enough), each a stretch of it, and adds the sum as it goes. Beside it runs a
// filter: with T such that at least M logits seen so far are >= T, only
// vectors whose maximum reaches T can hold a listed token, and their indices
// go to a short list in shared memory. T comes from the threads' own running
// maxima: every warp sorts its 32, and with k = ceil(M / warps) the smallest
// of the warps' k-th largest has M logits at or above it. It is taken after
// iterations 1, 2, 4, 8, ..., and a stretch is read in U interleaved streams,
// so that the first iteration samples all of it. About 7 M of a row's vectors
// pass; the same bound over their maxima leaves about 1.5 M, whose logits are
// looked at one by one and ranked by counting.
//
// Rows where more vectors pass than the list holds (runs of equal logits, all
// large logits in one place) are finished by bisection: the M-th largest key
// by counting passes over the row, tokens above it in any order, tokens at it
// in ascending order.
#include "spec_top.cuh"

#include "spec_rows.cuh"

namespace sr {

constexpr int NT = 256;
constexpr int NW = NT / 32;
constexpr int U = 8;         // 16-byte loads in flight per thread
constexpr int CAP = 2048;    // vectors that may pass the filter, per CTA
constexpr int CAPE = 1024;   // logits that may pass the last bound, per row
constexpr int kMaxCluster = 8;

// the k-th largest of the warp's values (k = 1 .. 32)
template <typename V>
__device__ __forceinline__ V warp_kth(V v, int k) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int o = size >> 1; o > 0; o >>= 1) {
            const V w = __shfl_xor_sync(kFull, v, o);
            const bool big = ((lane & o) == 0) == ((lane & size) == 0);   // descending runs
            v = big ? max(v, w) : min(v, w);
        }
    return __shfl_sync(kFull, v, k - 1);
}

// A bound with at least M of the block's `n` values (thread t holds the
// largest of the values t, t + NT, ...) at or above it, or `none`.
// buf: NW values, not written again before another barrier has passed.
template <typename V>
__device__ __forceinline__ V block_bound(V v, int n, int M, V none, V *buf) {
    const int act = min(NW, n >> 5);   // warps whose lanes all hold a value
    const int k = act ? (M + act - 1) / act : 33;
    if (k > 32) return none;           // the same in every thread
    const V t = warp_kth(v, k);
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = t;
    __syncthreads();
    V r = buf[0];
#pragma unroll
    for (int i = 1; i < NW; ++i)
        if (i < act) r = min(r, buf[i]);
    return max(r, none);
}

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

// The list by bisection; at least M keys of the row are >= t, or t = 1.
// Leaves at most M candidates in s_el, in no order, and returns their number.
template <typename T>
__device__ __noinline__ int bisect(const Row<T> &r, int V, int M, uint32_t t, float mx, unsigned long long *s_el,
                                   int *s_cnt, int *s_n) {
    auto count = [&](uint32_t k) {   // tokens of key >= k, k > 0
        int n = 0;
        each(r, [&](float z, int) { n += order_key(z) >= k; });
        n = __reduce_add_sync(kFull, n);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) s_cnt[threadIdx.x >> 5] = n;
        __syncthreads();
        n = 0;
        for (int i = 0; i < NW; ++i) n += s_cnt[i];
        return n;
    };
    // the largest t with count(t) >= M, or 1 when the row has no more tokens
    if (t > 1u || count(1u) > M) {
        uint32_t hi = order_key(mx);   // count(hi + 1) == 0 < M
        while (t < hi) {
            const uint32_t mid = t + (hi - t) / 2 + ((hi - t) & 1u);
            if (count(mid) >= M) t = mid;
            else hi = mid - 1;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) *s_n = 0;
    __syncthreads();
    const bool all = t == 1u;
    each(r, [&](float z, int i) {
        const uint32_t key = order_key(z);
        if (all ? key >= 1u : key > t) {
            const int at = atomicAdd(s_n, 1);
            if (at < M) s_el[at] = cand(key, i);
        }
    });
    __syncthreads();
    int n = min(*s_n, M);
    if (!all) {   // tokens at the threshold, lowest index first
        for (int i0 = 0; i0 < V && n < M; i0 += NT) {
            const int i = i0 + threadIdx.x;
            const bool at = i < V && order_key(load1(r.p + i)) == t;
            const unsigned bal = __ballot_sync(kFull, at);
            __syncthreads();
            if ((threadIdx.x & 31) == 0) s_cnt[threadIdx.x >> 5] = __popc(bal);
            __syncthreads();
            int before = n + __popc(bal & ((1u << (threadIdx.x & 31)) - 1u)), total = 0;
            for (int w = 0; w < NW; ++w) {
                before += w < (int)(threadIdx.x >> 5) ? s_cnt[w] : 0;
                total += s_cnt[w];
            }
            if (at && before < M) s_el[before] = cand(t, i);
            n = min(n + total, M);
        }
        __syncthreads();
    }
    return n;
}

template <typename T, bool kCluster>
__global__ void __launch_bounds__(NT, 4) top_kernel(TopArgs a, int S) {
    constexpr int E = Row<T>::E;
    __shared__ float s_c[CAP];
    __shared__ int s_code[CAP];
    __shared__ __align__(16) unsigned long long s_el[CAPE];
    __shared__ float s_b[3][NW], s_red[2][NW];
    __shared__ uint32_t s_kb[NW];
    __shared__ int s_n, s_ne, s_cnt[NW];
    __shared__ float s_x[4][kMaxCluster];   // per CTA of the cluster: bound, maximum, sum, overflow
    const int tid = threadIdx.x;
    const int row = kCluster ? blockIdx.x / S : blockIdx.x;
    const int rank = kCluster ? blockIdx.x - row * S : 0;
    if (a.scores) {   // dead and finished beams: the whole cluster leaves
        const float sc = a.scores[row];
        if (!(sc > neg_inf()) || sc == -neg_inf() || (a.finished && a.finished[row])) return;
    }
    if (kCluster) cluster_arrive();   // waited for before the exchange: by then every CTA of the cluster runs
    const int b = row / a.K, kr = row - b * a.K;
    const Row<T> r(static_cast<const T *>(a.z) + b * a.batch_stride + kr * a.row_stride, a.V);
    const int k0 = kCluster ? (int)((long long)r.nvec * rank / S) : 0;
    const int n = (kCluster ? (int)((long long)r.nvec * (rank + 1) / S) : r.nvec) - k0;
    const uint4 *body = r.body + k0;
    if (tid == 0) s_n = s_ne = 0;
    __syncthreads();

    Sum acc = sum_init(a.sL, a.rs);
    float thr = sv::kMaskFloor;
    const int its = (n + U * NT - 1) / (U * NT), span = its * NT;
    int refresh = 0;
    for (int it = 0; it < its; ++it) {
        uint4 w[U];
        const int base = it * NT + tid;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = u * span + base;
            w[u] = i < n ? sv::ldg_stream(body + i) : masked_vec<T>();
        }
        float c[U], cm;
#pragma unroll
        for (int u = 0; u < U; ++u) c[u] = vec_max<T>(w[u]);
        cm = c[0];
#pragma unroll
        for (int u = 1; u < U; ++u) cm = fmaxf(cm, c[u]);
        sum_see(acc, cm, a.sL, a.rs);
        float v = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float z[E];
            Elem<T>::unpack(w[u], z);
            v += sum_terms<E>(acc, z, a.sL);
        }
        sum_put(acc, v);
        if ((it & (it + 1)) == 0 && (it == 0 || it + 1 < its)) {
            thr = block_bound(acc.mx, n, a.M, thr, s_b[refresh]);
            refresh ^= 1;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c[u] >= thr) {
                const int at = atomicAdd(&s_n, 1);
                if (at < CAP) {
                    s_c[at] = c[u];
                    s_code[at] = k0 + u * span + base;
                }
            }
    }
    if (tid < 2 * E) {   // the row's ends: single logits, coded by ~index
        const int i = r.edge_index(tid);
        if (i >= 0 && (tid < E ? rank == 0 : rank == S - 1)) {
            const float z = load1(r.p + i);
            sum_add1(acc, z, a.sL, a.rs);
            if (z >= thr) {
                const int at = atomicAdd(&s_n, 1);
                if (at < CAP) {
                    s_c[at] = z;
                    s_code[at] = ~i;
                }
            }
        }
    }
    float mx = block_max<NT>(acc.mx, s_red[0]);
    float sum = block_sum<NT>(sum_at(acc, mx, a.sL), s_red[1]);
    // (the barriers above also publish the list)
    bool over = s_n > CAP;
    const int np = min(s_n, CAP);
    float best = neg_inf();
    for (int i = tid; i < np; i += NT) best = fmaxf(best, s_c[i]);
    thr = block_bound(best, np, a.M, thr, s_b[2]);
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
        float m = neg_inf();
        for (int i = 0; i < S; ++i) {
            thr = fmaxf(thr, s_x[0][i]);
            m = fmaxf(m, s_x[1][i]);
            over |= s_x[3][i] != 0.f;
        }
        sum = 0.f;
        for (int i = 0; i < S; ++i)
            sum += s_x[1][i] == m || !(s_x[2][i] > 0.f) ? s_x[2][i] : s_x[2][i] * ex2((s_x[1][i] - m) * a.sL);
        mx = m;
    }
    // the passing vectors' logits, to the cluster's first CTA
    const uint32_t el0 = kCluster ? peer(s_el, 0) : 0u, ne0 = kCluster ? peer(&s_ne, 0) : 0u;
    auto put = [&](float z, int index) {
        if (!(z >= thr)) return;
        const uint32_t key = order_key(z);
        if (key == 0u) return;
        const int at = kCluster ? peer_add(ne0, 1) : atomicAdd(&s_ne, 1);
        if (at < CAPE) {
            if (kCluster) peer_store(el0 + 8u * at, cand(key, index));
            else s_el[at] = cand(key, index);
        }
    };
    if (!over)
        for (int i = tid; i < np; i += NT) {
            const float c = s_c[i];
            if (!(c >= thr)) continue;
            const int code = s_code[i];
            if (code < 0) {
                put(c, ~code);
                continue;
            }
            float z[E];
            Elem<T>::unpack(__ldg(r.body + code), z);
#pragma unroll
            for (int j = 0; j < E; ++j) put(z[j], r.vec_index(code) + j);
        }
    if (kCluster) {
        cluster_arrive();
        cluster_wait();
        if (rank != 0) return;
    } else {
        __syncthreads();
    }
    int ne = s_ne;
    if (over || ne > CAPE) ne = bisect(r, a.V, a.M, max(order_key(thr), 1u), mx, s_el, s_cnt, &s_n);
    uint32_t bound = 0u;
    if (ne > 128) {   // once more over single logits
        uint32_t k = 0u;
        for (int i = tid; i < ne; i += NT) k = max(k, cand_key(s_el[i]));
        bound = block_bound(k, ne, a.M, 0u, s_kb);
    }
    if (bound) {   // gather what reaches it: s_c holds CAP 32-bit words, half as many candidates
        unsigned long long *s_few = reinterpret_cast<unsigned long long *>(s_c);
        if (tid == 0) s_n = 0;
        __syncthreads();
        for (int i = tid; i < ne; i += NT)
            if (cand_key(s_el[i]) >= bound) s_few[atomicAdd(&s_n, 1)] = s_el[i];
        __syncthreads();
        ne = s_n;
        for (int i = tid; i < ne; i += NT) s_el[i] = s_few[i];
        __syncthreads();
    }
    const bool some = mx > sv::kMaskFloor, bad = !(sum >= 0.f) || mx == -neg_inf();
    const float lnS = logf(sum);
    for (int i = tid; i < ne; i += NT) {
        const unsigned long long c = s_el[i];
        int rk = 0;
        for (int j = 0; j < ne; ++j) rk += s_el[j] > c;
        if (rk < a.M) {
            const float z = key_value(cand_key(c));
            a.val[(size_t)row * a.M + rk] = a.stat ? z : fmaf(z - mx, a.s, -lnS);
            a.ids[(size_t)row * a.M + rk] = cand_index(c);
        }
    }
    for (int i = ne + tid; i < a.M; i += NT) {
        a.val[(size_t)row * a.M + i] = neg_inf();
        a.ids[(size_t)row * a.M + i] = -1;
    }
    if (tid == 0) {
        if (a.stat) a.stat[row] = make_float2(mx, sum);
        if (a.lse) a.lse[row] = bad ? __int_as_float(0x7fc00000) : some ? fmaf(mx, a.s, lnS) : neg_inf();
        if (bad) raise_status(a.status, SPEC_ERR_BAD_ROW);
    }
}

// CTAs per row: rows are split while there are SM slots to fill (4 CTAs on
// each of 152 SMs) and a CTA keeps a vector per thread
static int top_cluster(long long rows, int V, int es) {
    const long long nvec = (long long)V * es / 16;
    int S = 1;
    while (S < kMaxCluster && rows * S * 2 <= 608 && nvec >= 2LL * S * NT) S *= 2;
    return S;
}

template <typename T>
static cudaError_t launch_top_t(const TopArgs &a, cudaStream_t stream) {
    const long long rows = (long long)a.B * a.K;
    const int S = top_cluster(rows, a.V, sizeof(T));
    if (S > 1) return launch_cluster(top_kernel<T, true>, (unsigned)(rows * S), NT, S, 0, stream, a, S);
    return launch_cluster(top_kernel<T, false>, (unsigned)rows, NT, 1, 0, stream, a, 1);
}

cudaError_t launch_top(const TopArgs &a, int bf16, cudaStream_t stream) {
    return bf16 ? launch_top_t<__nv_bfloat16>(a, stream) : launch_top_t<float>(a, stream);
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

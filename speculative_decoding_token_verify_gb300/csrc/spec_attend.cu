// spec_attend.cu -- attention of a tree's nodes over a cache held in pages.
#include <cuda_fp16.h>

#include "spec_rows.cuh"

namespace sr {

struct AttendArgs {
    const void *q, *k, *v;
    const int32_t *table, *lengths, *parents, *counts;
    void *out;
    float *lse;
    int32_t *status;
    int B, N, Hq, Hkv, G, D, P, page, M;
    float sL;   // scale log2 e
    long long qs[3], ks[3], vs[3], ps;
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

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f(float x) { return __float2half_rn(x); }

// A warp per row (b, n, h); lane l holds elements 4 l .. 4 l + 3. One key after
// another, with the running maximum and sum of a softmax.
template <typename T>
__global__ void __launch_bounds__(128) attend_simple_kernel(AttendArgs a) {
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= (long long)a.B * a.N * a.Hq) return;
    const int h = (int)(row % a.Hq), n = (int)(row / a.Hq % a.N), b = (int)(row / a.Hq / a.N), hk = h / a.G;
    int L, count;
    sequence(a, b, L, count);
    const bool mine = 4 * lane < a.D;
    const T *q = static_cast<const T *>(a.q) + b * a.qs[0] + n * a.qs[1] + h * a.qs[2] + 4 * lane;
    float x[4] = {0, 0, 0, 0}, o[4] = {0, 0, 0, 0}, m = neg_inf(), l = 0.f;
    if (mine)
        for (int i = 0; i < 4; ++i) x[i] = to_f(q[i]);
    auto see = [&](int t) {
        const int p = a.table[(long long)b * a.M + t / a.page];
        if (p < 0 || p >= a.P) {
            raise_status(a.status, SPEC_ERR_BAD_PAGE);
            return;
        }
        const int slot = t % a.page;
        const T *k = static_cast<const T *>(a.k) + p * a.ks[0] + slot * a.ks[1] + hk * a.ks[2] + 4 * lane;
        const T *v = static_cast<const T *>(a.v) + p * a.vs[0] + slot * a.vs[1] + hk * a.vs[2] + 4 * lane;
        float s = 0.f;
        if (mine)
            for (int i = 0; i < 4; ++i) s += x[i] * to_f(k[i]);
        s = warp_sum(s) * a.sL;
        const float mx = fmaxf(m, s), w = ex2(s - mx), keep = ex2(m - mx);
        l = l * keep + w;
        m = mx;
        if (mine)
            for (int i = 0; i < 4; ++i) o[i] = o[i] * keep + w * to_f(v[i]);
    };
    if (n < count) {
        for (int t = 0; t < L; ++t) see(t);
        for (int j = n; j >= 0; j = parent_of(a, b, j)) see(L + j);
    }
    T *out = static_cast<T *>(a.out) + row * a.D + 4 * lane;
    if (mine)
        for (int i = 0; i < 4; ++i) out[i] = from_f<T>(l != 0.f ? o[i] / l : 0.f);
    if (lane == 0 && a.lse) a.lse[row] = l != 0.f ? sv::kLn2 * (m + log2f(l)) : neg_inf();
}

static bool overlap(const void *a, int64_t na, const void *b, int64_t nb) {
    const char *x = static_cast<const char *>(a), *y = static_cast<const char *>(b);
    return na > 0 && nb > 0 && x < y + nb && y < x + na;
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
    return SPEC_OK;
}

}  // namespace sr

extern "C" size_t spec_tree_attention_workspace_size(const spec_attend_params *p) {
    return sr::check_attend(p) == SPEC_OK ? 16 : 0;
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
    AttendArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.table = table;
    a.lengths = lengths;
    a.parents = parents;
    a.counts = counts;
    a.out = out;
    a.lse = lse;
    a.status = status;
    a.B = p->B;
    a.N = p->N;
    a.Hq = p->Hq;
    a.Hkv = p->Hkv;
    a.G = p->Hq / p->Hkv;
    a.D = p->D;
    a.P = p->P;
    a.page = p->page;
    a.M = p->M;
    a.sL = p->scale * sv::kLog2e;
    a.ps = p->parents_stride;
    const int n[3][3] = {{p->B, p->N, p->Hq}, {p->P, p->page, p->Hkv}, {p->P, p->page, p->Hkv}};
    for (int j = 0; j < 3; ++j) {
        a.qs[j] = n[0][j] > 1 ? p->q_stride[j] : 0;
        a.ks[j] = n[1][j] > 1 ? p->k_stride[j] : 0;
        a.vs[j] = n[2][j] > 1 ? p->v_stride[j] : 0;
    }
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const unsigned grid = (unsigned)(((long long)a.B * a.N * a.Hq + 3) / 4);
    if (p->dtype == SPEC_BF16) attend_simple_kernel<__nv_bfloat16><<<grid, 128, 0, st>>>(a);
    else attend_simple_kernel<__half><<<grid, 128, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SPEC_OK : spec_internal_set_error(SPEC_ERR_CUDA, cudaGetErrorString(e));
}

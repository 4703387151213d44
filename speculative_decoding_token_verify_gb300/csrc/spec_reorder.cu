// spec_reorder.cu -- the beams' states in the order of the surviving beams.
//
// In place without a second buffer: a column (one vector's place in a row) is
// one thread's alone, which loads that place from every parent before it
// stores any. Rows that keep their place are neither read nor written, and what
// lies behind a sequence's length is skipped by whole tiles.
//
// Measured: a 2 GB bf16 cache, 8 beams of which about a third stay, 280 us: 7.0
// TB/s of moved bytes (parents that go on twice are read from L2 the second
// time), the rate of a plain copy; with one column per thread 308 us. 16 beams
// run at 84% of that, 3 beams at 65%: loads of beams that stay leave their
// registers idle. Random permutations of whole rows, moved bytes against a copy's rate: 2
// beams (half of the rows stay) 63%, 3 beams 91%, 4 and 8 beams all of it, 16 beams
// 92%, 24 beams 91%, 32 beams 80%. Listing the beams that move first, so that few leave room for
// more columns, spilled and was slower throughout (317 us).
#include "spec_rows.cuh"

namespace sr {

constexpr int NTR = 256;

struct ReorderArgs {
    const char *src;
    char *dst;
    const int32_t *parent, *lengths;
    int32_t *status;
    int B, W, N, H, T;
    long long unit, ss[4], ds[4];
    long long seg_tiles;   // tiles of NTR CP vectors per segment, at least 1
    int in_place;
};

// WB: beams a thread has registers for; CP: columns per thread, so that few beams
// too have several loads in flight
template <typename Vec, int WB, int CP>
__global__ void __launch_bounds__(NTR, 2) reorder_kernel(ReorderArgs a) {
    __shared__ int s_par[SPEC_MAX_BEAMS];
    const int o = blockIdx.z;
    const int h = (int)(blockIdx.x / a.seg_tiles);
    const long long tile = blockIdx.x - (long long)h * a.seg_tiles;
    for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
        __syncthreads();
        if (threadIdx.x < a.N) {
            int p = a.parent[(size_t)b * a.N + threadIdx.x];
            if (p < -1 || p >= a.W) {
                if (blockIdx.x == 0 && o == 0) raise_status(a.status, SPEC_ERR_BAD_PARENT);
                p = -1;
            }
            if (a.in_place && p == (int)threadIdx.x) p = -1;   // stays where it is
            s_par[threadIdx.x] = p;
        }
        __syncthreads();
        const long long units = a.lengths ? min(max(a.lengths[b], 0), a.T) : a.T;
        const long long bytes = units * a.unit;
        const char *src = a.src + o * a.ss[0] + b * a.ss[1] + h * a.ss[3];
        char *dst = a.dst + o * a.ds[0] + b * a.ds[1] + h * a.ds[3];
        // bytes up to an aligned address (the same for all beams), vectors, bytes
        const long long head = min(bytes, (long long)(-reinterpret_cast<uintptr_t>(src) & (sizeof(Vec) - 1)));
        const long long vecs = (bytes - head) / (long long)sizeof(Vec);
        const long long i0 = tile * (NTR * CP) + threadIdx.x;
        Vec v[CP][WB];
#pragma unroll
        for (int c = 0; c < CP; ++c)
            if (i0 + c * NTR < vecs) {
                const char *p = src + head + (i0 + c * NTR) * (long long)sizeof(Vec);
#pragma unroll
                for (int n = 0; n < WB; ++n)
                    if (n < a.N && s_par[n] >= 0) v[c][n] = *reinterpret_cast<const Vec *>(p + s_par[n] * a.ss[2]);
            }
#pragma unroll
        for (int c = 0; c < CP; ++c)
            if (i0 + c * NTR < vecs) {
                char *p = dst + head + (i0 + c * NTR) * (long long)sizeof(Vec);
#pragma unroll
                for (int n = 0; n < WB; ++n)
                    if (n < a.N && s_par[n] >= 0) *reinterpret_cast<Vec *>(p + n * a.ds[2]) = v[c][n];
            }
        // head and tail bytes: a segment's first tile has threads for all of them
        const long long rest = bytes - vecs * (long long)sizeof(Vec);
        if (sizeof(Vec) > 1 && tile == 0 && threadIdx.x < rest) {
            const long long at = threadIdx.x < head ? threadIdx.x : bytes - rest + threadIdx.x;
            char w[WB];
#pragma unroll
            for (int n = 0; n < WB; ++n)
                if (n < a.N && s_par[n] >= 0) w[n] = src[at + s_par[n] * a.ss[2]];
#pragma unroll
            for (int n = 0; n < WB; ++n)
                if (n < a.N && s_par[n] >= 0) dst[at + n * a.ds[2]] = w[n];
        }
    }
}

template <typename Vec>
static cudaError_t launch_vec(ReorderArgs &a, int O, cudaStream_t stream) {
    const int cp = a.N <= 4 ? 4 : a.N <= 8 ? 2 : 1;
    const long long seg = (long long)a.T * a.unit / (long long)sizeof(Vec);
    a.seg_tiles = seg > 0 ? (seg + NTR * cp - 1) / (NTR * cp) : 1;
    const long long gx = a.seg_tiles * a.H;
    if (gx > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)gx, (unsigned)(a.B < 65535 ? a.B : 65535), (unsigned)O);
    if (a.N <= 4) reorder_kernel<Vec, 4, 4><<<grid, NTR, 0, stream>>>(a);
    else if (a.N <= 8) reorder_kernel<Vec, 8, 2><<<grid, NTR, 0, stream>>>(a);
    else if (a.N <= 16) reorder_kernel<Vec, 16, 1><<<grid, NTR, 0, stream>>>(a);
    else if constexpr (sizeof(Vec) < 16) reorder_kernel<Vec, 32, 1><<<grid, NTR, 0, stream>>>(a);
    else return cudaErrorInvalidValue;   // (more than 16 beams take narrower vectors)
    return cudaGetLastError();
}

// rows (o, b, beam, segment) of `bytes` bytes that do not overlap: with the
// axes ordered by stride, each steps over the whole extent of the smaller ones
static bool disjoint(const int64_t *stride, const int64_t *count, int64_t bytes) {
    int order[4] = {0, 1, 2, 3};
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 4; ++j)
            if (stride[order[j]] < stride[order[i]]) {
                const int t = order[i];
                order[i] = order[j];
                order[j] = t;
            }
    int64_t extent = bytes;
    for (int i = 0; i < 4; ++i) {
        const int k = order[i];
        if (count[k] <= 1) continue;
        if (stride[k] < extent) return false;
        extent += (count[k] - 1) * stride[k];
    }
    return true;
}

}  // namespace sr

extern "C" int spec_beam_reorder(const spec_reorder_params *p, const void *src, void *dst, const int32_t *parent,
                                 const int32_t *lengths, int32_t *status, void *stream) {
    using namespace sr;
    if (!p) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "params is NULL");
    if (p->O < 0 || p->B < 0 || p->H < 0 || p->T < 0)
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "O, B, H and T must be >= 0");
    if (p->W < 1 || p->W > SPEC_MAX_BEAMS || p->N < 1 || p->N > SPEC_MAX_BEAMS || p->O > 65535 || p->H > 65535 ||
        p->B > SPEC_MAX_B)
        return spec_internal_set_error(SPEC_ERR_UNSUPPORTED, "beam_reorder: O, B, W, N or H out of range");
    if (p->unit_bytes < 1 || p->unit_bytes > (1 << 30))
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "beam_reorder: unit_bytes must be in [1, 2^30]");
    const int64_t sc[4] = {p->O, p->B, p->W, p->H}, dc[4] = {p->O, p->B, p->N, p->H};
    for (int i = 0; i < 4; ++i) {
        if (p->src_stride[i] < 0 || p->dst_stride[i] < 0)
            return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "beam_reorder: strides must be >= 0");
        if ((sc[i] > 1 && p->src_stride[i] > (INT64_MAX >> 4) / sc[i]) ||
            (dc[i] > 1 && p->dst_stride[i] > (INT64_MAX >> 4) / dc[i]))
            return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "beam_reorder: strides are too large");
    }
    if (p->O == 0 || p->B == 0 || p->H == 0 || p->T == 0) return spec_internal_set_error(SPEC_OK, "");
    if (!src || !dst || !parent) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "src / dst / parent is NULL");
    const int64_t bytes = (int64_t)p->T * p->unit_bytes;
    if (!disjoint(p->dst_stride, dc, bytes))
        return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "beam_reorder: rows of dst overlap");
    ReorderArgs a{};
    a.in_place = src == dst;
    if (a.in_place) {
        if (p->N > p->W) return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "beam_reorder: in place needs N <= W");
        for (int i = 0; i < 4; ++i)
            if (sc[i] > 1 && p->src_stride[i] != p->dst_stride[i])
                return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "beam_reorder: in place needs equal strides");
        // beams past N are rows of the state too
        if (!disjoint(p->src_stride, sc, bytes))
            return spec_internal_set_error(SPEC_ERR_INVALID_ARG, "beam_reorder: rows of src overlap");
    }
    a.src = static_cast<const char *>(src);
    a.dst = static_cast<char *>(dst);
    a.parent = parent;
    a.lengths = lengths;
    a.status = status;
    a.B = p->B;
    a.W = p->W;
    a.N = p->N;
    a.H = p->H;
    a.T = p->T;
    a.unit = p->unit_bytes;
    for (int i = 0; i < 4; ++i) {
        a.ss[i] = sc[i] > 1 ? p->src_stride[i] : 0;
        a.ds[i] = dc[i] > 1 ? p->dst_stride[i] : 0;
    }
    // Vectors as wide as all beams of a segment, and its rows in src and dst, are
    // aligned alike; a segment's own alignment, and a length that ends inside a
    // vector, cost bytes at its ends.
    uint64_t bits = (uint64_t)(a.ss[2] | a.ds[2]);
    if (!a.in_place)
        bits |= (uint64_t)((a.ss[0] - a.ds[0]) | (a.ss[1] - a.ds[1]) | (a.ss[3] - a.ds[3])) |
                (reinterpret_cast<uintptr_t>(src) - reinterpret_cast<uintptr_t>(dst));
    spec_internal_set_error(SPEC_OK, "");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (bits % 16 == 0 && a.N <= 16) e = launch_vec<uint4>(a, p->O, st);
    else if (bits % 8 == 0) e = launch_vec<uint2>(a, p->O, st);   // 32 beams' wider vectors leave one CTA an SM
    else if (bits % 4 == 0) e = launch_vec<uint32_t>(a, p->O, st);
    else if (bits % 2 == 0) e = launch_vec<uint16_t>(a, p->O, st);
    else e = launch_vec<uint8_t>(a, p->O, st);
    if (e == cudaErrorInvalidConfiguration)
        return spec_internal_set_error(SPEC_ERR_UNSUPPORTED, "beam_reorder: segments too long");
    return e == cudaSuccess ? SPEC_OK : spec_internal_set_error(SPEC_ERR_CUDA, cudaGetErrorString(e));
}

// Block boxes (pa_block_bounds) and block choice (pa_select_blocks) of the block-sparse
// decode.
#include <cooperative_groups.h>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace cg = cooperative_groups;

namespace pa {

PA_ERROR_WORD_ACCESSOR(error_word_sparse_select)

namespace {

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// ---------------------------------------------------------------------------
// block_bounds: per (block, KV head) tile of 16 keys, per dim the smallest and largest
// value, in eight bits with one scale; rounded outwards, so that the box still holds every
// key.  A tile is read once (16 * D elements) and gives 2 D + 4 bytes: bound by the read.
// One warp per tile, tiles of one block's KV heads next to each other (they are one
// contiguous piece of the cache); every lane keeps the columns of its 16-byte vectors in
// registers, so the 16 rows need only one exchange at the end.  min.NaN / max.NaN carry a
// NaN through to the scale.
// ---------------------------------------------------------------------------
template <typename T, int D>
__global__ void __launch_bounds__(256) block_bounds_kernel(const BoundsArgs a) {
    constexpr int V = 16 / sizeof(T);               // elements per 16-byte vector
    constexpr int LPR = D / V < 32 ? D / V : 32;    // lanes per row
    constexpr int CH = D / V / LPR;                 // vectors of a row per lane
    constexpr int RPL = 32 / LPR;                   // rows per warp load
    pdl_wait();
    pdl_release_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t items = (int64_t)a.B * a.W * a.H, nw = (int64_t)gridDim.x * 8;
    for (int64_t it = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); it < items; it += nw) {
        const int h = (int)(it % a.H);
        const int64_t bw = it / a.H;
        const int w = (int)(bw % a.W), b = (int)(bw / a.W);
        const int first = a.first ? max(a.first[b], 0) / kBlockSize : 0;
        const int end = min(a.lens[b], a.M * kBlockSize) / kBlockSize;
        if (end - first > a.W && w == 0 && h == 0 && lane == 0) raise_flag(PA_EFLAG_BAD_LENGTH);
        const int j = first + w;
        if (j >= end || first < 0) continue;
        const int x = a.tables[(size_t)b * a.M + j];
        if (x < 0 || (int64_t)x >= a.N) {
            if (h == 0 && lane == 0) raise_flag(PA_EFLAG_BAD_BLOCK);
            continue;
        }
        const size_t tile = (size_t)x * a.H + h;
        const T *k = reinterpret_cast<const T *>(a.kc) + tile * (kBlockSize * D) + (lane / LPR) * D + (lane % LPR) * V;
        float lo[CH][V], hi[CH][V];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            uint4 raw[16 / RPL];
#pragma unroll
            for (int i = 0; i < 16 / RPL; ++i)
                raw[i] = __ldg(reinterpret_cast<const uint4 *>(k + i * RPL * D + c * LPR * V));
#pragma unroll
            for (int i = 0; i < 16 / RPL; ++i) {
                const uint32_t wds[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
                float f[V];
                to_float<T, V>(wds, f);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    lo[c][e] = i == 0 ? f[e] : min_nan(lo[c][e], f[e]);
                    hi[c][e] = i == 0 ? f[e] : max_nan(hi[c][e], f[e]);
                }
            }
        }
        const float ks = sizeof(T) == 1 ? a.ks[tile] : 1.f;
        float m = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int e = 0; e < V; ++e) {
#pragma unroll
                for (int o = LPR; o < 32; o <<= 1) {
                    lo[c][e] = min_nan(lo[c][e], __shfl_xor_sync(0xffffffffu, lo[c][e], o));
                    hi[c][e] = max_nan(hi[c][e], __shfl_xor_sync(0xffffffffu, hi[c][e], o));
                }
                if (sizeof(T) == 1) {  // codes: the keys are their products with the tile's scale
                    lo[c][e] = __fmul_rn(lo[c][e], ks);
                    hi[c][e] = __fmul_rn(hi[c][e], ks);
                }
                m = max_nan(m, max_nan(fabsf(lo[c][e]), fabsf(hi[c][e])));
            }
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        const bool fin = m < __int_as_float(0x7f800000);  // false for NaN too
        const float s = fin ? __fdiv_rn(m, 127.0f) : __int_as_float(0x7f800000);
        if (lane == 0) a.scales[tile] = s;
        int8_t *out = a.bounds + tile * (2 * D) + (lane % LPR) * V;
        // lanes of the first row write the lower side, of the second (or the same lanes) the upper
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            if (RPL > 1 ? lane / LPR != side : false) continue;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                uint32_t pk[(V + 3) / 4] = {};
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    int q = 0;
                    if (fin && s > 0.f) {
                        const float r = __fdiv_rn(side ? hi[c][e] : lo[c][e], s);
                        q = (int)fminf(fmaxf(side ? ceilf(r) : floorf(r), -127.f), 127.f);
                    }
                    pk[e / 4] |= (uint32_t)(q & 0xff) << (8 * (e % 4));
                }
                int8_t *o = out + side * D + c * LPR * V;
                if constexpr (V == 16)
                    *reinterpret_cast<uint4 *>(o) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                else if constexpr (V == 8)
                    *reinterpret_cast<uint2 *>(o) = make_uint2(pk[0], pk[1]);
                else
                    *reinterpret_cast<uint32_t *>(o) = pk[0];
            }
        }
    }
}

template <typename T>
int bounds_d(const BoundsArgs &a, cudaStream_t st) {
    const int64_t items = (int64_t)a.B * a.W * a.H;
    const int64_t ctas = (items + 7) / 8;
    const dim3 grid((unsigned)(ctas < 148 * 8 ? ctas : 148 * 8));
    cudaError_t e;
    switch (a.D) {
    case 64: e = launch_pdl(block_bounds_kernel<T, 64>, grid, dim3(256), 0, st, a); break;
    case 128: e = launch_pdl(block_bounds_kernel<T, 128>, grid, dim3(256), 0, st, a); break;
    default: e = launch_pdl(block_bounds_kernel<T, 256>, grid, dim3(256), 0, st, a); break;
    }
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

int launch_block_bounds(const BoundsArgs &a, cudaStream_t st) {
    switch (a.kv_dtype) {
    case PA_F32: return bounds_d<float>(a, st);
    case PA_F16: return bounds_d<__half>(a, st);
    case PA_BF16: return bounds_d<__nv_bfloat16>(a, st);
    default: return bounds_d<int8_t>(a, st);
    }
}

}  // namespace pa

#include "pa_select.cuh"

namespace pa {

namespace {

// One cluster per (query row, KV head).  (256 threads: registers for three CTAs on an SM.)
template <typename T, int D, int NT>
__global__ void __launch_bounds__(NT, NT == 256 && D <= 128 ? 3 : 1) select_kernel(const SparseArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    pdl_wait();
    pdl_release_dependents();
    cg::cluster_group cl = cg::this_cluster();
    const int64_t item = blockIdx.x / cl.num_blocks();
    select_row<T, D, NT>(a, (int)(item / a.H), (int)(item % a.H), (int)cl.block_rank(), (int)cl.num_blocks(), smem);
}

template <typename T, int D, int NT>
int launch_select_n(const SparseArgs &a, int c, size_t smem, cudaStream_t st) {
    auto kern = select_kernel<T, D, NT>;
    if (!set_smem_attr_once(reinterpret_cast<const void *>(kern), 227 * 1024)) return PA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)a.rows * a.H * c));
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = c;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = c > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <typename T, int D>
int launch_select_t(const SparseArgs &a, cudaStream_t st) {
    const int nblk = (a.max_len + kBlockSize - 1) / kBlockSize;
    const int64_t items = (int64_t)a.rows * a.H;
    // CTAs per row: enough of them to fill the GPU, each with at least 128 boxes to score
    int c = 1;
    while (c < 8 && items * c * 2 <= 2 * 148 && nblk / (2 * c) >= 128) c *= 2;
    const size_t smem = SelectSmem<D>::bytes(a.G, nblk);
    if (smem > 227 * 1024) return PA_ERR_UNSUPPORTED;
    // 512 threads where a CTA has many boxes, or few rows leave the SMs to the one that picks
    return nblk / c > 512 || nblk > 1024 ? launch_select_n<T, D, 512>(a, c, smem, st) : launch_select_n<T, D, 256>(a, c, smem, st);
}

template <typename T>
int select_d(const SparseArgs &a, cudaStream_t st) {
    switch (a.D) {
    case 64: return launch_select_t<T, 64>(a, st);
    case 128: return launch_select_t<T, 128>(a, st);
    default: return launch_select_t<T, 256>(a, st);
    }
}

}  // namespace

int launch_select_blocks(const SparseArgs &a, cudaStream_t st) {
    switch (a.q_dtype) {
    case PA_F32: return select_d<float>(a, st);
    case PA_F16: return select_d<__half>(a, st);
    default: return select_d<__nv_bfloat16>(a, st);
    }
}

}  // namespace pa

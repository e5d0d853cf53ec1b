// Block boxes (pa_block_bounds) and block choice (pa_select_blocks) of the block-sparse
// decode.
#include <cooperative_groups.h>

#include "pa_cluster.cuh"
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
// key but for roundings of 2^-24 of the largest (the scale's own, which the clamp to 127 meets,
// and the quotient's).  A tile is read once (16 * D elements) and gives 2 D + 4 bytes: bound by the read.
// One warp per tile, tiles of one block's KV heads next to each other (they are one
// contiguous piece of the cache); every lane keeps the columns of its 16-byte vectors in
// registers, so the 16 rows need only one exchange at the end.  Instructions are the second
// bound, so 16-bit caches are compared two values at a time, and a code's division is done by
// the reciprocal unless the quotient is so near a whole number that only the division itself
// tells on which side it lies.  The comparisons carry a NaN through to the scale.
// 65536 tiles of 16 x 128: fp16 49 us (5.8 TB/s), fp32 86 us (6.4 TB/s); int8 93 us (1.6 TB/s):
// its 32 minima and maxima a lane as fp32 do not fit into the registers of six CTAs on an SM.
// ---------------------------------------------------------------------------
constexpr int kBoundsWarps = 8;  // per CTA

// Two 16-bit values, or one fp32 / int8 value, per register.
template <typename T> struct MinMax {
    static constexpr int PER = 1;  // values per register
    using R = float;
    static __device__ __forceinline__ R lo(R a, R b) { return min_nan(a, b); }
    static __device__ __forceinline__ R hi(R a, R b) { return max_nan(a, b); }
    static __device__ __forceinline__ float get(R a, int) { return a; }
};
template <> struct MinMax<__half> {
    static constexpr int PER = 2;
    using R = uint32_t;
    static __device__ __forceinline__ R lo(R a, R b) {
        asm("min.NaN.f16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
        return a;
    }
    static __device__ __forceinline__ R hi(R a, R b) {
        asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
        return a;
    }
    static __device__ __forceinline__ float get(R a, int e) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&a));
        return e ? f.y : f.x;
    }
};
template <> struct MinMax<__nv_bfloat16> {
    static constexpr int PER = 2;
    using R = uint32_t;
    static __device__ __forceinline__ R lo(R a, R b) {
        asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
        return a;
    }
    static __device__ __forceinline__ R hi(R a, R b) {
        asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
        return a;
    }
    static __device__ __forceinline__ float get(R a, int e) {
        return e ? __uint_as_float(a & 0xffff0000u) : __uint_as_float(a << 16);
    }
};

template <typename T, int D>
__global__ void __launch_bounds__(kBoundsWarps * 32, D == 256 ? 4 : 6) block_bounds_kernel(const BoundsArgs a) {
    using X = MinMax<T>;
    using R = typename X::R;
    constexpr int V = 16 / sizeof(T);               // elements per 16-byte vector
    constexpr int LPR = D / V < 32 ? D / V : 32;    // lanes per row
    constexpr int CH = D / V / LPR;                 // vectors of a row per lane
    constexpr int RPL = 32 / LPR;                   // rows per warp load
    constexpr int NR = V / X::PER;                  // registers per vector
    pdl_wait();
    pdl_release_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t items = (int64_t)a.B * a.W * a.H, nw = (int64_t)gridDim.x * kBoundsWarps;
    for (int64_t it = (int64_t)blockIdx.x * kBoundsWarps + (threadIdx.x >> 5); it < items; it += nw) {
        const int h = (int)(it % a.H);
        const int64_t bw = it / a.H;
        const int w = (int)(bw % a.W), b = (int)(bw / a.W);
        const int len = __ldcg(a.lens + b);
        const int first = a.first ? max(__ldcg(a.first + b), 0) / kBlockSize : 0;
        const int j = first + w;
        // the entry does not wait for the length
        const int x = j < a.M ? __ldcg(a.tables + (size_t)b * a.M + j) : -1;
        const int end = min(len, a.M * kBlockSize) / kBlockSize;
        if (end - first > a.W && w == 0 && h == 0 && lane == 0) raise_flag(PA_EFLAG_BAD_LENGTH);
        if (j >= end) continue;
        if (x < 0 || (int64_t)x >= a.N) {
            if (h == 0 && lane == 0) raise_flag(PA_EFLAG_BAD_BLOCK);
            continue;
        }
        const size_t tile = (size_t)x * a.H + h;
        const T *k = reinterpret_cast<const T *>(a.kc) + tile * (kBlockSize * D) + (lane / LPR) * D + (lane % LPR) * V;
        const float ks = sizeof(T) == 1 ? __ldg(a.ks + tile) : 1.f;
        R lo[CH][NR], hi[CH][NR];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            uint4 raw[16 / RPL];
#pragma unroll
            for (int i = 0; i < 16 / RPL; ++i)
                raw[i] = __ldg(reinterpret_cast<const uint4 *>(k + i * RPL * D + c * LPR * V));
#pragma unroll
            for (int i = 0; i < 16 / RPL; ++i) {
                const uint32_t wds[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
                R f[NR];
                if constexpr (X::PER == 2) {
#pragma unroll
                    for (int e = 0; e < NR; ++e) f[e] = wds[e];
                } else {
                    to_float<T, V>(wds, f);
                }
#pragma unroll
                for (int e = 0; e < NR; ++e) {
                    lo[c][e] = i == 0 ? f[e] : X::lo(lo[c][e], f[e]);
                    hi[c][e] = i == 0 ? f[e] : X::hi(hi[c][e], f[e]);
                }
            }
        }
        float vl[CH][V], vh[CH][V], m = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int r = 0; r < NR; ++r) {
#pragma unroll
                for (int o = LPR; o < 32; o <<= 1) {
                    lo[c][r] = X::lo(lo[c][r], __shfl_xor_sync(0xffffffffu, lo[c][r], o));
                    hi[c][r] = X::hi(hi[c][r], __shfl_xor_sync(0xffffffffu, hi[c][r], o));
                }
#pragma unroll
                for (int p = 0; p < X::PER; ++p) {
                    const int e = r * X::PER + p;
                    vl[c][e] = X::get(lo[c][r], p);
                    vh[c][e] = X::get(hi[c][r], p);
                    if (sizeof(T) == 1) {  // codes: the keys are their products with the tile's scale (of either sign)
                        const float x0 = __fmul_rn(vl[c][e], ks), x1 = __fmul_rn(vh[c][e], ks);
                        vl[c][e] = min_nan(x0, x1);
                        vh[c][e] = max_nan(x0, x1);
                    }
                    m = max_nan(m, max_nan(fabsf(vl[c][e]), fabsf(vh[c][e])));
                }
            }
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        const bool fin = m < __int_as_float(0x7f800000);  // false for NaN too
        const float s = fin ? __fdiv_rn(m, 127.0f) : __int_as_float(0x7f800000);
        if (lane == 0) a.scales[tile] = s;
        const bool some = fin && s > 0.f, safe = s > 1e-30f && s < 1e30f;
        const float inv = some ? __fdividef(1.f, s) : 0.f;
        int8_t *out = a.bounds + tile * (2 * D) + (lane % LPR) * V;
        // lanes of the first row write the lower side, of the second the upper (lanes that hold a
        // whole row write both)
#pragma unroll
        for (int side = 0; side < (RPL > 1 ? 1 : 2); ++side) {
            const bool up = RPL > 1 ? lane >= LPR : side != 0;
            if (RPL > 2 && lane >= 2 * LPR) break;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                uint32_t pk[(V + 3) / 4] = {};
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    // the lower side as the upper one of -x: floor(x) = -ceil(-x)
                    const float y = up ? vh[c][e] : -vl[c][e];
                    float r = y * inv;  // off by less than 127 * 2^-21 < 1e-4 of the quotient
                    if (some && (!safe || fabsf(r - rintf(r)) < 1e-4f)) r = __fdiv_rn(y, s);
                    const int q = some ? (int)fminf(fmaxf(ceilf(r), -127.f), 127.f) : 0;
                    pk[e / 4] |= (uint32_t)((up ? q : -q) & 0xff) << (8 * (e % 4));
                }
                int8_t *o = out + (up ? D : 0) + c * LPR * V;
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
    // a tile per warp (the loop is for the largest grids): the CTAs' own turnover balances the SMs
    // better than a grid of the resident ones that strides over the tiles (49.1 against 55.0 us for
    // 65536 fp16 tiles of 16 x 128)
    const int64_t ctas = (items + kBoundsWarps - 1) / kBoundsWarps;
    const dim3 grid((unsigned)(ctas < (1 << 22) ? ctas : (1 << 22)));
    cudaError_t e;
    switch (a.D) {
    case 64: e = launch_pdl(block_bounds_kernel<T, 64>, grid, dim3(kBoundsWarps * 32), 0, st, a); break;
    case 128: e = launch_pdl(block_bounds_kernel<T, 128>, grid, dim3(kBoundsWarps * 32), 0, st, a); break;
    default: e = launch_pdl(block_bounds_kernel<T, 256>, grid, dim3(kBoundsWarps * 32), 0, st, a); break;
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

// One cluster per (query row, KV head).  (Up to 256 threads: registers for 24 warps on an SM.)
template <typename T, int D, int NT>
__global__ void __launch_bounds__(NT, NT <= 256 && D <= 128 ? 768 / NT : 1) select_kernel(const SparseArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    pdl_wait();
    pdl_release_dependents();
    cg::cluster_group cl = cg::this_cluster();
    const int64_t item = blockIdx.x / cl.num_blocks();
    select_row<T, D, NT>(a, (int)(item / a.H), (int)(item % a.H), (int)cl.block_rank(), (int)cl.num_blocks(), smem);
}

template <typename T, int D, int NT>
int launch_select_n(const SparseArgs &a, int most, size_t smem, cudaStream_t st) {
    auto kern = select_kernel<T, D, NT>;
    if (!set_smem_attr_once(reinterpret_cast<const void *>(kern), 227 * 1024)) return PA_ERR_CUDA;
    const int64_t items = (int64_t)a.rows * a.H;
    static ClusterRoom room;  // of the shared memory that leaves each SM to one CTA of 512 threads anyway
    const int c = NT < 512 ? most : room.largest(kern, items, most, NT, 100 * 1024);
    return launch_cluster(kern, items * c, c, NT, smem, st, a) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <typename T, int D>
int launch_select_t(const SparseArgs &a, cudaStream_t st) {
    const int nblk = (a.max_len + kBlockSize - 1) / kBlockSize;
    const int64_t items = (int64_t)a.rows * a.H;
    static_assert(SelectSmem<D>::bytes(64, PA_SPARSE_MAX_SEQ_LEN / kBlockSize) <= 227 * 1024, "keys of the longest row");
    const size_t smem = SelectSmem<D>::bytes(a.G, nblk);
    // CTAs per row: as many as give every SM one, each with at least 128 boxes to score
    int c = (int)(items < 148 ? 148 / items : 1);
    if (c > 8) c = 8;
    while (c > 1 && nblk / c < 128) --c;
    // Threads: 512 where the SMs have a CTA each at most, with more than a tile for each of 8 warps
    // (128 rows of 256 blocks 5.8 us, with two CTAs of 256 threads a row 7.0; of 512 blocks 7.1 against
    // 9.1), or where a CTA's boxes are many; 128 for very many short rows, whose picking is then
    // spread over more CTAs (1024 rows 15 us, with 256 threads 18.9; but 512 rows, of which half need
    // no choice, 9.9 against 7.9).
    if (items > 6 * 148 && nblk <= 512) return launch_select_n<T, D, 128>(a, c, smem, st);
    if ((items * c <= 148 && nblk / c > 128) || nblk / c > 512) return launch_select_n<T, D, 512>(a, c, smem, st);
    return launch_select_n<T, D, 256>(a, c, smem, st);
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

// pa_decode_selected: decode attention over chosen blocks (pa_attend.cuh).
#include "pa_attend.cuh"
#include "pa_cluster.cuh"

namespace cg = cooperative_groups;

namespace pa {

PA_ERROR_WORD_ACCESSOR(error_word_sparse_decode)

namespace {

// One cluster per (query row, KV head, group of 8 * NT query heads).
template <typename T, typename TKV, int D, int NT, int NW>
__global__ void __launch_bounds__(NW * 32) attend_kernel(const __grid_constant__ CUtensorMap tmK,
                                                     const __grid_constant__ CUtensorMap tmV, const SparseArgs a) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    if (threadIdx.x == 0) {
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    attend_init<AttendCfg<T, TKV, D, NT, NW>>(smem);
    pdl_wait();
    pdl_release_dependents();
    cg::cluster_group cl = cg::this_cluster();
    const int ncta = (int)cl.num_blocks();
    const int64_t item = blockIdx.x / ncta;
    const int grp = (int)(item % a.ng);
    const int64_t rh = item / a.ng;
    attend_row<T, TKV, D, NT, NW>(a, &tmK, &tmV, (int)(rh / a.H), (int)(rh % a.H), grp, (int)cl.block_rank(), ncta, smem);
}

template <int D, int GT>
__global__ void __launch_bounds__(128) attend_f32_kernel(const SparseArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    pdl_wait();
    pdl_release_dependents();
    cg::cluster_group cl = cg::this_cluster();
    const int ncta = (int)cl.num_blocks();
    const int64_t item = blockIdx.x / ncta;
    const int grp = (int)(item % a.ng);
    const int64_t rh = item / a.ng;
    attend_row_f32<D, GT>(a, (int)(rh / a.H), (int)(rh % a.H), grp, (int)cl.block_rank(), ncta, smem);
}

// CTAs per row: as many as the GPU holds at once, each warp with at least two blocks.  (128 rows of 128
// int8 blocks in CTAs of four warps take 25.2 us with one CTA a row, 23.4 with two, 19.8 with three
// and 26.8 with four, which no longer fit at once.)
template <typename K>
int cluster_of(ClusterRoom &room, K *kern, int64_t items, int blocks, int warps, size_t smem) {
    return room.largest(kern, items, blocks / (2 * warps), warps * 32, smem);
}

// Map over a cache as tiles of [16 rows][D], one copy per tile: box (128 bytes of a row, 16 rows,
// the row's 128-byte segments, 1 tile), 128-byte swizzle (64-byte int8 rows at D = 64: none).
bool tile_map(CUtensorMap *m, const void *base, int64_t tiles, int D, int dtype) {
    auto fn = tc_encode_fn();
    if (!fn) return false;
    const int es = dtype == PA_I8 ? 1 : 2, rowb = D * es, segb = rowb < 128 ? rowb : 128;
    const cuuint64_t dims[4] = {(cuuint64_t)(segb / es), 16, (cuuint64_t)(rowb / segb), (cuuint64_t)tiles};
    const cuuint64_t strides[3] = {(cuuint64_t)rowb, (cuuint64_t)segb, (cuuint64_t)rowb * 16};
    const cuuint32_t box[4] = {(cuuint32_t)(segb / es), 16, (cuuint32_t)(rowb / segb), 1};
    const cuuint32_t es1[4] = {1, 1, 1, 1};
    const CUtensorMapDataType dt = dtype == PA_I8     ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : dtype == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    return fn(m, dt, 4, const_cast<void *>(base), dims, strides, box, es1, CU_TENSOR_MAP_INTERLEAVE_NONE,
              segb == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, typename TKV, int D, int NT, int NW = 4>
int launch_attend_t(SparseArgs a, cudaStream_t st) {
    using C = AttendCfg<T, TKV, D, NT, NW>;
    // Many rows: CTAs of three warps, four of which fit on an SM's shared memory where three of
    // four warps do, so that a batch's rows run in fewer waves (512 rows of 64 blocks: 39.9 us
    // against 44.9, 1024 rows 80.8 against 84.8 with their choice; 8 rows 16.7 against 15.6).
    if constexpr (NT == 1 && !C::I8 && D <= 128 && NW == 4)
        if ((int64_t)a.rows * a.H >= 3 * 148) return launch_attend_t<T, TKV, D, NT, 3>(a, st);
    // About a row per SM: one CTA with as many warps as the registers and shared memory hold, instead
    // of a cluster of smaller ones that have to join their shares (128 int8 rows of 128 blocks 19.6 us
    // against 19.8 with three CTAs of four warps; 128 rows of 32 heads 27.8 against 29.2 with their
    // choice).  Fewer rows with long lists: clusters of 8-warp CTAs, so that eight CTAs are 64 warps
    // (8 rows of 128 blocks 5.6 against 6.3 us, of 256 blocks 7.1 against 8.7, but of 64 blocks 5.3
    // against 5.1; with 16 or 32 heads a tile it is the slower form: 9.2 against 8.9).
    constexpr int WIDE = NT == 1 ? 12 : 8;
    if constexpr (D <= 128 && NW == 4) {
        const int64_t items = (int64_t)a.rows * a.H * ((a.G + C::HEADS - 1) / C::HEADS);
        if (items <= 148 && 2 * items > 148 && a.K >= 2 * WIDE) return launch_attend_t<T, TKV, D, NT, WIDE>(a, st);
        if constexpr (NT == 1)
            if (2 * items <= 148 && a.K >= 128) return launch_attend_t<T, TKV, D, NT, 8>(a, st);
    }
    a.ng = (a.G + C::HEADS - 1) / C::HEADS;
    const int64_t items = (int64_t)a.rows * a.H * a.ng;
    auto kern = attend_kernel<T, TKV, D, NT, NW>;
    if (!set_smem_attr_once(reinterpret_cast<const void *>(kern), C::BYTES)) return PA_ERR_CUDA;
    static ClusterRoom room;
    const int c = cluster_of(room, kern, items, a.K, C::NW, C::BYTES);
    CUtensorMap tk, tv;
    if (!tile_map(&tk, a.kc, a.N * a.H, D, a.kv_dtype) || !tile_map(&tv, a.vc, a.N * a.H, D, a.kv_dtype)) return PA_ERR_CUDA;
    return launch_cluster(kern, items * c, c, C::NW * 32, C::BYTES, st, tk, tv, a) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <typename T, typename TKV>
int launch_attend_d(const SparseArgs &a, cudaStream_t st) {
    // n-tiles of 8 heads: as many as the group has and the registers hold, so that a tile is read
    // once for all of them
    switch (a.D) {
    case 64:
        return a.G <= 8 ? launch_attend_t<T, TKV, 64, 1>(a, st)
                        : a.G <= 16 ? launch_attend_t<T, TKV, 64, 2>(a, st) : launch_attend_t<T, TKV, 64, 4>(a, st);
    case 128:
        return a.G <= 8 ? launch_attend_t<T, TKV, 128, 1>(a, st)
                        : a.G <= 16 ? launch_attend_t<T, TKV, 128, 2>(a, st) : launch_attend_t<T, TKV, 128, 4>(a, st);
    default: return a.G <= 8 ? launch_attend_t<T, TKV, 256, 1>(a, st) : launch_attend_t<T, TKV, 256, 2>(a, st);
    }
}

template <int D, int GT>
int launch_attend_f32_t(SparseArgs a, cudaStream_t st) {
    using C = AttendF32Cfg<D, GT>;
    a.ng = (a.G + GT - 1) / GT;
    const int64_t items = (int64_t)a.rows * a.H * a.ng;
    auto kern = attend_f32_kernel<D, GT>;
    if (!set_smem_attr_once(reinterpret_cast<const void *>(kern), C::BYTES)) return PA_ERR_CUDA;
    static ClusterRoom room;
    const int c = cluster_of(room, kern, items, a.K, C::NW, C::BYTES);
    return launch_cluster(kern, items * c, c, C::NW * 32, C::BYTES, st, a) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <int D>
int launch_attend_f32_d(const SparseArgs &a, cudaStream_t st) {
    return a.G == 1   ? launch_attend_f32_t<D, 1>(a, st)
           : a.G == 2 ? launch_attend_f32_t<D, 2>(a, st)
           : a.G <= 4 ? launch_attend_f32_t<D, 4>(a, st)
                      : launch_attend_f32_t<D, 8>(a, st);
}

}  // namespace

int launch_decode_selected(const SparseArgs &a, cudaStream_t st) {
    if (a.q_dtype == PA_F32)
        return a.D == 64    ? launch_attend_f32_d<64>(a, st)
               : a.D == 128 ? launch_attend_f32_d<128>(a, st)
                            : launch_attend_f32_d<256>(a, st);
    if (a.q_dtype == PA_F16)
        return a.kv_dtype == PA_I8 ? launch_attend_d<__half, int8_t>(a, st) : launch_attend_d<__half, __half>(a, st);
    return a.kv_dtype == PA_I8 ? launch_attend_d<__nv_bfloat16, int8_t>(a, st)
                               : launch_attend_d<__nv_bfloat16, __nv_bfloat16>(a, st);
}

}  // namespace pa

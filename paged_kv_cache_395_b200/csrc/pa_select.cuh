// Scoring and choosing the blocks of one (query row, KV head), as device code: the whole
// of pa_select_blocks and the first half of pa_decode_sparse.
//
//   score_j = max_g I_gj * scale_j * s_g,   I_gj = sum_d max(c_gd lo_jd, c_gd hi_jd)
//           = sum_d min(c_gd, 0) lo_jd + max(c_gd, 0) hi_jd
// so the I of 8 heads and 16 blocks is one int8 product of [16 boxes][2 D] with
// [2 D][8 heads] on the tensor cores (mma.sync m16n8k32, whole numbers: exact, any order).
// The boxes are read from global memory once, straight into the A fragments: the
// contraction's order is free, so each lane takes 16 contiguous bytes of its rows and the
// codes of q are read in the same order.  2 D + 4 bytes per block and 16-bit cache's 64 D:
// the score reads 1/32 of what dense attention would.
//
// The row's keys (scores as ordered whole numbers) are gathered in the shared memory of the
// cluster's first CTA, which alone picks: the cut is found by histograms of 256 bins over
// the range that still holds it, starting at the scores' own range (two or three rounds;
// four at most), and the picks are written in index order.
#pragma once
#include <cooperative_groups.h>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

__device__ __forceinline__ void imma(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Shared memory: the codes of q, 8 * ceil(G / 8) heads of 2 D bytes (row stride + 64 bytes: the
// 16-byte reads of 8 rows fall into different banks), their scales, small counters, the keys.
template <int D>
struct SelectSmem {
    static constexpr int QROW = 2 * D + 64;
    static constexpr int MISC = 4 * (256 + 4 * 32 + 16);
    static __host__ __device__ int heads(int G) { return (G + 7) / 8 * 8; }
    static __host__ __device__ size_t bytes(int G, int nblk) {
        return (size_t)heads(G) * (QROW + 4) + MISC + (size_t)((nblk + 31) / 32 * 32) * 4;
    }
};

// Tokens that query row r = (b, t) sees.
__device__ __forceinline__ int sparse_row_len(const SparseArgs &a, int r, int &b) {
    b = r / a.Q;
    return max(min(max(a.lens[b], 0), a.max_len) - a.Q + 1 + (r - b * a.Q), 0);
}

// Every CTA of the cluster calls this with all its threads (a multiple of 32, 256 or more).  On
// return the cluster's first CTA has written the row's list; nothing is synchronised after that.
template <typename T, int D>
__device__ void select_row(const SparseArgs &a, int r, int h, int rank, int ncta, unsigned char *smem) {
    using S = SelectSmem<D>;
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
    const int NH = S::heads(a.G), K = a.K;
    int8_t *qc = reinterpret_cast<int8_t *>(smem);
    float *qs = reinterpret_cast<float *>(smem + NH * S::QROW);
    uint32_t *hist = reinterpret_cast<uint32_t *>(qs + NH);
    uint32_t *wa = hist + 256, *wb = wa + 32, *wc = wb + 32, *misc = wc + 64;
    uint32_t *keys = reinterpret_cast<uint32_t *>(smem + NH * (S::QROW + 4) + S::MISC);

    int b;
    const int L = sparse_row_len(a, r, b), n = (L + kBlockSize - 1) / kBlockSize;
    int32_t *out = a.sel + ((size_t)r * a.H + h) * K;
    if (n <= K) {  // the same in every CTA of the cluster
        if (rank == 0) {
            for (int i = tid; i < K; i += nt) out[i] = i < n ? i : -1;
            if (tid == 0) a.nsel[(size_t)r * a.H + h] = n;
        }
        return;
    }

    // the first CTA's shared memory is written by the others only once that CTA runs: the wait
    // for this is below, before the first score
    if (ncta > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

    // ---- codes of q: [min(c, 0) for every dim][max(c, 0) for every dim] per head ----
    for (int g = warp; g < NH; g += nw) {
        float x[D / 32], m = 0.f;
        const T *q = reinterpret_cast<const T *>(a.q) + ((size_t)r * a.Hq + (size_t)h * a.G + g) * D;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            x[i] = g < a.G ? Cvt<T>::to_f(q[lane * (D / 32) + i]) : 0.f;
            // an infinity or NaN gives m = inf: the codes are then 0
            m = fmaxf(m, fabsf(x[i]) <= 3.402823466e38f ? fabsf(x[i]) : __int_as_float(0x7f800000));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float s = __fdiv_rn(m, 127.0f);
        if (!(s < __int_as_float(0x7f800000))) s = 0.f;
        if (lane == 0) qs[g] = s;
        int8_t *row = qc + g * S::QROW;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            int c = 0;
            if (s > 0.f) c = max(-127, min(127, __float2int_rn(__fdiv_rn(x[i], s))));
            row[lane * (D / 32) + i] = (int8_t)min(c, 0);
            row[D + lane * (D / 32) + i] = (int8_t)max(c, 0);
        }
    }
    __syncthreads();

    // ---- scores of this CTA's blocks ----
    const int per = ((n + ncta - 1) / ncta + 15) / 16 * 16, lo = min(n, rank * per), hi = min(n, lo + per);
    const int g = lane >> 2, c = lane & 3;
    uint32_t *dst = keys;
    if (ncta > 1) {
        dst = cooperative_groups::this_cluster().map_shared_rank(keys, 0);
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    }
    const int32_t *table = a.tables + (size_t)b * a.M;
    for (int j0 = lo + warp * 16; j0 < hi; j0 += nw * 16) {
        int id = -1;
        if (lane < 16 && j0 + lane < hi) {
            id = table[j0 + lane];
            if (id < 0 || (int64_t)id >= a.N) {
                id = -1;
                raise_flag(PA_EFLAG_BAD_BLOCK);
            }
        }
        const int i0 = __shfl_sync(0xffffffffu, id, g), i1 = __shfl_sync(0xffffffffu, id, g + 8);
        const size_t t0 = (size_t)max(i0, 0) * a.H + h, t1 = (size_t)max(i1, 0) * a.H + h;
        const uint4 *p0 = reinterpret_cast<const uint4 *>(a.bounds + t0 * (2 * D)) + c;
        const uint4 *p1 = reinterpret_cast<const uint4 *>(a.bounds + t1 * (2 * D)) + c;
        uint4 u[D / 32], v[D / 32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            u[i] = i0 >= 0 ? __ldg(p0 + 4 * i) : make_uint4(0, 0, 0, 0);
            v[i] = i1 >= 0 ? __ldg(p1 + 4 * i) : make_uint4(0, 0, 0, 0);
        }
        const float s0 = i0 >= 0 ? __ldg(a.bscales + t0) : 0.f, s1 = i1 >= 0 ? __ldg(a.bscales + t1) : 0.f;
        float m0 = __int_as_float(0xff800000), m1 = m0;
        for (int hb = 0; hb < NH; hb += 8) {
            int d[4] = {0, 0, 0, 0};
            const uint4 *bq = reinterpret_cast<const uint4 *>(qc + (hb + g) * S::QROW) + c;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint4 w = bq[4 * i];
                imma(d, u[i].x, v[i].x, u[i].y, v[i].y, w.x, w.y);
                imma(d, u[i].z, v[i].z, u[i].w, v[i].w, w.z, w.w);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int col = hb + 2 * c + e;
                if (col < a.G) {
                    // + 0: a product that underflows to -0 becomes +0
                    m0 = fmaxf(m0, __fmul_rn(__fmul_rn((float)d[e], s0), qs[col]) + 0.f);
                    m1 = fmaxf(m1, __fmul_rn(__fmul_rn((float)d[2 + e], s1), qs[col]) + 0.f);
                }
            }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
            m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
        }
        if (c < 2) {
            const int j = j0 + g + 8 * c;
            const float s = c ? s1 : s0;
            uint32_t k = __float_as_uint(s < __int_as_float(0x7f800000) ? (c ? m1 : m0) : __int_as_float(0x7f800000));
            k ^= (k >> 31) ? 0xffffffffu : 0x80000000u;  // ordered as whole numbers
            if ((c ? i1 : i0) < 0) k = 0;
            if (j < hi) dst[j] = k;
        }
    }
    if (ncta > 1)
        cooperative_groups::this_cluster().sync();
    else
        __syncthreads();
    if (rank != 0) return;

    // ---- the cut: the key of the last of the `need` best unforced blocks ----
    // unforced blocks are [f0, f1); n > K, so there are more than `need` of them
    const int f0 = a.sink, f1 = n - a.recent;
    int need = K - a.sink - a.recent;
    uint32_t cut = 0xffffffffu;  // taken: keys above `cut`, and the first `need` equal to it
    if (need > 0) {
        uint32_t kl = 0xffffffffu, kh = 0;
        for (int j = f0 + tid; j < f1; j += nt) {
            kl = min(kl, keys[j]);
            kh = max(kh, keys[j]);
        }
        kl = __reduce_min_sync(0xffffffffu, kl);
        kh = __reduce_max_sync(0xffffffffu, kh);
        if (lane == 0) {
            wa[warp] = kl;
            wb[warp] = kh;
        }
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int w = 0; w < nw; ++w) {
            kl = min(kl, wa[w]);
            kh = max(kh, wb[w]);
        }
        for (;;) {
            // bins of 2^sh keys over [kl, kh]
            const int sh = max(0, 24 - __clz((int)(kh - kl)));
            for (int j = f0 + tid; j < f1; j += nt) {
                const uint32_t k = keys[j];
                if (k >= kl && k <= kh) atomicAdd(&hist[(k - kl) >> sh], 1u);
            }
            __syncthreads();
            if (warp == 0) {
                // lane l: bins 255 - 8 l .. 248 - 8 l, from the top
                uint32_t s[8], sum = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s[i] = hist[255 - 8 * lane - i];
                    sum += s[i];
                }
                uint32_t up = sum;  // inclusive over the lanes
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, up, o);
                    if (lane >= o) up += y;
                }
                const uint32_t before = up - sum;
                if (before < (uint32_t)need && up >= (uint32_t)need) {
                    uint32_t acc = before;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (acc < (uint32_t)need && acc + s[i] >= (uint32_t)need) {
                            misc[0] = 255 - 8 * lane - i;  // the bin that holds the cut
                            misc[1] = acc;                 // keys above it
                            misc[2] = s[i];
                        }
                        acc += s[i];
                    }
                }
            }
            __syncthreads();
            const uint32_t bin = misc[0], above = misc[1], in = misc[2];
            if (tid < 256) hist[tid] = 0;
            need -= (int)above;
            kl += bin << sh;
            if (in == (uint32_t)need) {  // the whole bin is taken
                cut = kl - 1;            // kl > 0: a key of 0 is a block outside the pool, see below
                need = 0;
                if (kl == 0) {
                    cut = 0;
                    need = 0x7fffffff;
                }
                break;
            }
            if (sh == 0) {
                cut = kl;
                break;
            }
            kh = min(kh, kl + ((1u << sh) - 1));
            __syncthreads();
        }
    }

    // ---- the picks in index order: warp w takes the w-th run of the row ----
    const int run = ((n + nw - 1) / nw + 31) / 32 * 32, j0 = min(n, warp * run), j1 = min(n, j0 + run);
    auto cls = [&](int j) {  // 2: taken, 1: equal to the cut
        if (j >= j1) return 0;
        if (j < f0 || j >= f1) return 2;
        const uint32_t k = keys[j];
        return k > cut ? 2 : k == cut ? 1 : 0;
    };
    uint32_t gt = 0, eq = 0;
    for (int j = j0; j < j1; j += 32) {
        const int k = cls(j + lane);
        gt += __popc(__ballot_sync(0xffffffffu, k == 2));
        eq += __popc(__ballot_sync(0xffffffffu, k == 1));
    }
    __syncthreads();  // wa, wb are read above
    if (lane == 0) {
        wa[warp] = gt;
        wb[warp] = eq;
    }
    __syncthreads();
    uint32_t at = 0, eqs = 0;
    for (int w = 0; w < warp; ++w) {
        at += wa[w];
        eqs += wb[w];
    }
    at += min(eqs, (uint32_t)need);
    const uint32_t below = (1u << lane) - 1;
    for (int j = j0; j < j1; j += 32) {
        const int k = cls(j + lane);
        const uint32_t em = __ballot_sync(0xffffffffu, k == 1);
        const bool take = k == 2 || (k == 1 && eqs + __popc(em & below) < (uint32_t)need);
        const uint32_t tm = __ballot_sync(0xffffffffu, take);
        if (take) out[at + __popc(tm & below)] = j + lane;
        at += __popc(tm);
        eqs += __popc(em);
    }
    if (tid == 0) a.nsel[(size_t)r * a.H + h] = K;
}

}  // namespace pa

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
// cluster's first CTA, which alone picks: a histogram of 256 bins over the scores' range finds
// the bin that holds the cut, that bin's few keys are ranked against each other (or, when equal
// scores make them many, the histogram is taken again over the bin), and every thread writes the
// picks of its run of the row in order.
//
// What bounds it is the latency of dependent loads and barriers, not bytes: so nothing that is
// asked for first (table entries, q) waits for the row's length, the boxes of a warp's first tile
// are on their way while q's codes are made, and later tiles are fetched a step ahead.  64 rows of
// up to 4096 tokens x 8 KV heads take 7.9 us, one row of 131072 tokens 12.7 us (its 17 MB would
// take 2.6 us of DRAM time).
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
    static constexpr int CAND = 512;  // keys of the cut's bin that are ranked directly
    static constexpr int MISC = 4 * (256 + CAND + 2 * 32 + 16);
    static constexpr __host__ __device__ int heads(int G) { return (G + 7) / 8 * 8; }
    static constexpr __host__ __device__ size_t bytes(int G, int nblk) {
        return (size_t)heads(G) * (QROW + 4) + MISC + (size_t)((nblk + 31) / 32 * 32) * 4;
    }
};

// Tokens that query row r = (b, t) sees.
__device__ __forceinline__ int sparse_row_len(const SparseArgs &a, int r, int &b) {
    b = r / a.Q;
    return max(min(max(a.lens[b], 0), a.max_len) - a.Q + 1 + (r - b * a.Q), 0);
}

// Every CTA of the cluster calls this with all its NT threads.  On return the cluster's first CTA has
// written the row's list; nothing is synchronised after that.
template <typename T, int D, int NT>
__device__ void select_row(const SparseArgs &a, int r, int h, int rank, int ncta, unsigned char *smem) {
    using S = SelectSmem<D>;
    constexpr int nw = NT / 32, EL = D / 32;       // warps; dims of q per lane
    constexpr bool AHEAD = NT > 256 && D <= 128;   // boxes of the next tile in registers
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int NH = S::heads(a.G), K = a.K;
    const float kInf = __int_as_float(0x7f800000);
    int8_t *qc = reinterpret_cast<int8_t *>(smem);
    float *qs = reinterpret_cast<float *>(smem + NH * S::QROW);
    uint32_t *hist = reinterpret_cast<uint32_t *>(qs + NH);
    uint32_t *cand = hist + 256, *wa = cand + S::CAND, *wb = wa + 32, *misc = wb + 32;
    uint32_t *keys = reinterpret_cast<uint32_t *>(smem + NH * (S::QROW + 4) + S::MISC);

    // ---- asked for at once: the table entries of the warp's first tile, q's first heads, the length ----
    // tile i of the warp: blocks 16 ((i nw + warp) ncta + rank) on
    const int32_t *table = a.tables + (size_t)(r / a.Q) * a.M;
    const int step = 16 * nw * ncta;
    int j0 = 16 * (warp * ncta + rank);
    auto entries = [&](int j) { return lane < 16 && j + lane < a.M ? __ldcg(table + j + lane) : -1; };
    int id = entries(j0);
    constexpr int QB = 4;  // heads per warp and batch
    const T *q0 = reinterpret_cast<const T *>(a.q) + ((size_t)r * a.Hq + (size_t)h * a.G) * D + lane * EL;
    const bool qvec = ((uintptr_t)a.q & 15) == 0;
    float qx[QB][EL];
    auto q_load = [&](int g0) {
#pragma unroll
        for (int i = 0; i < QB; ++i) {
            const int hd = g0 + warp + i * nw;
            const T *q = q0 + (size_t)hd * D;
            if (hd >= a.G) {
#pragma unroll
                for (int e = 0; e < EL; ++e) qx[i][e] = 0.f;
            } else if (qvec) {
                uint32_t w[EL * sizeof(T) / 4];
#pragma unroll
                for (int e = 0; e < (int)(EL * sizeof(T) / 4); ++e) w[e] = __ldcg(reinterpret_cast<const uint32_t *>(q) + e);
                to_float<T, EL>(w, qx[i]);
            } else {
#pragma unroll
                for (int e = 0; e < EL; ++e) qx[i][e] = Cvt<T>::to_f(q[e]);
            }
        }
    };
    q_load(0);
    int b;
    const int L = sparse_row_len(a, r, b), n = (L + kBlockSize - 1) / kBlockSize;
    int32_t *out = a.sel + ((size_t)r * a.H + h) * K;
    if (n <= K) {  // the same in every CTA of the cluster
        if (rank == 0) {
            for (int i = tid; i < K; i += NT) out[i] = i < n ? i : -1;
            if (tid == 0) a.nsel[(size_t)r * a.H + h] = n;
        }
        return;
    }
    const int f0 = a.sink, f1 = n - a.recent;  // the unforced blocks
    for (int i = tid; i < 256; i += NT) hist[i] = 0;
    if (tid == 0) {
        misc[0] = 0xffffffffu;  // smallest and largest key of the unforced blocks
        misc[1] = 0;
        misc[5] = 0;            // candidates
    }
    // the first CTA's shared memory is written by the others only once that CTA is here: the wait
    // for this is below, before the first score
    if (ncta > 1) asm volatile("barrier.cluster.arrive.release;" ::: "memory");

    // ---- the boxes of 16 blocks: lane (g, c) holds 16-byte pieces c, c + 4, ... of blocks g and g + 8 ----
    struct Box {
        uint4 u[D / 32], v[D / 32];
        float s0, s1;
        int i0, i1;
    };
    auto fetch = [&](int j, int ids, Box &x) {
        if (lane < 16 && j + lane < n && (ids < 0 || (int64_t)ids >= a.N)) {
            ids = -1;
            raise_flag(PA_EFLAG_BAD_BLOCK);
        }
        if (j + lane >= n) ids = -1;
        x.i0 = __shfl_sync(0xffffffffu, ids, g);
        x.i1 = __shfl_sync(0xffffffffu, ids, g + 8);
        const size_t t0 = (size_t)max(x.i0, 0) * a.H + h, t1 = (size_t)max(x.i1, 0) * a.H + h;
        const uint4 *p0 = reinterpret_cast<const uint4 *>(a.bounds + t0 * (2 * D)) + c;
        const uint4 *p1 = reinterpret_cast<const uint4 *>(a.bounds + t1 * (2 * D)) + c;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            x.u[i] = x.i0 >= 0 ? __ldg(p0 + 4 * i) : make_uint4(0, 0, 0, 0);
            x.v[i] = x.i1 >= 0 ? __ldg(p1 + 4 * i) : make_uint4(0, 0, 0, 0);
        }
        x.s0 = x.i0 >= 0 ? __ldg(a.bscales + t0) : 0.f;
        x.s1 = x.i1 >= 0 ? __ldg(a.bscales + t1) : 0.f;
    };
    Box box;
    int id_next = entries(j0 + step);
    if (j0 < n) fetch(j0, id, box);

    // ---- codes of q: [min(c, 0) for every dim][max(c, 0) for every dim] per head ----
    for (int g0 = 0; g0 < NH; g0 += QB * nw) {
        if (g0 > 0) q_load(g0);
#pragma unroll
        for (int i = 0; i < QB; ++i) {
            const int hd = g0 + warp + i * nw;
            if (hd >= NH) break;
            float m = 0.f;
#pragma unroll
            for (int e = 0; e < EL; ++e)  // an infinity or NaN gives m = inf: the codes are then 0
                m = fmaxf(m, fabsf(qx[i][e]) <= 3.402823466e38f ? fabsf(qx[i][e]) : kInf);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            float s = __fdiv_rn(m, 127.0f);
            if (!(s < kInf)) s = 0.f;
            if (lane == 0) qs[hd] = s;
            const float inv = s > 0.f ? __fdividef(1.f, s) : 0.f;
            // x / s by the reciprocal is off by less than 2^-21 * 127 < 1e-4, so its rounding is the
            // quotient's unless it lies that near to a half (or the reciprocal is out of range)
            const bool safe = s > 1e-30f && s < 1e30f;
            uint32_t lo[(EL + 3) / 4] = {}, hi[(EL + 3) / 4] = {};
#pragma unroll
            for (int e = 0; e < EL; ++e) {
                float y = qx[i][e] * inv;
                const float f = fabsf(y) - truncf(fabsf(y));
                if (s > 0.f && (!safe || fabsf(f - 0.5f) < 1e-4f)) y = __fdiv_rn(qx[i][e], s);
                const int k = s > 0.f ? max(-127, min(127, __float2int_rn(y))) : 0;
                lo[e / 4] |= (uint32_t)(min(k, 0) & 0xff) << (8 * (e % 4));
                hi[e / 4] |= (uint32_t)max(k, 0) << (8 * (e % 4));
            }
            int8_t *row = qc + hd * S::QROW + lane * EL;
            if constexpr (EL == 2) {
                *reinterpret_cast<uint16_t *>(row) = (uint16_t)lo[0];
                *reinterpret_cast<uint16_t *>(row + D) = (uint16_t)hi[0];
            } else {
#pragma unroll
                for (int e = 0; e < EL / 4; ++e) {
                    reinterpret_cast<uint32_t *>(row)[e] = lo[e];
                    reinterpret_cast<uint32_t *>(row + D)[e] = hi[e];
                }
            }
        }
    }
    __syncthreads();

    // ---- scores ----
    uint32_t *dst = keys, *range = misc;
    if (ncta > 1) {
        dst = cooperative_groups::this_cluster().map_shared_rank(keys, 0);
        range = cooperative_groups::this_cluster().map_shared_rank(misc, 0);
        asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    }
    uint32_t kl = 0xffffffffu, kh = 0;
    for (; j0 < n; j0 += step) {
        Box next;
        const int id2 = j0 + step < n ? id_next : -1;
        if (j0 + 2 * step < n) id_next = entries(j0 + 2 * step);
        if (AHEAD && j0 + step < n) fetch(j0 + step, id2, next);
        float m0 = -kInf, m1 = m0;
        for (int hb = 0; hb < NH; hb += 8) {
            int d[2][4] = {};
            const uint4 *bq = reinterpret_cast<const uint4 *>(qc + (hb + g) * S::QROW) + c;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint4 w = bq[4 * i];
                imma(d[0], box.u[i].x, box.v[i].x, box.u[i].y, box.v[i].y, w.x, w.y);
                imma(d[1], box.u[i].z, box.v[i].z, box.u[i].w, box.v[i].w, w.z, w.w);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int col = hb + 2 * c + e;
                if (col < a.G) {
                    // + 0: a product that underflows to -0 becomes +0
                    const float sq = qs[col];
                    m0 = fmaxf(m0, __fmul_rn(__fmul_rn((float)(d[0][e] + d[1][e]), box.s0), sq) + 0.f);
                    m1 = fmaxf(m1, __fmul_rn(__fmul_rn((float)(d[0][2 + e] + d[1][2 + e]), box.s1), sq) + 0.f);
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
            uint32_t k = __float_as_uint((c ? box.s1 : box.s0) < kInf ? (c ? m1 : m0) : kInf);
            k ^= (k >> 31) ? 0xffffffffu : 0x80000000u;  // ordered as whole numbers
            if ((c ? box.i1 : box.i0) < 0) k = 0;
            if (j < n) dst[j] = k;
            if (j >= f0 && j < f1) {
                kl = min(kl, k);
                kh = max(kh, k);
            }
        }
        if (AHEAD)
            box = next;
        else if (j0 + step < n)
            fetch(j0 + step, id2, box);
    }
    kl = __reduce_min_sync(0xffffffffu, kl);
    kh = __reduce_max_sync(0xffffffffu, kh);
    if (lane == 0 && kl <= kh) {
        atomicMin(range, kl);
        atomicMax(range + 1, kh);
    }
    if (ncta > 1)
        cooperative_groups::this_cluster().sync();
    else
        __syncthreads();
    if (rank != 0) return;

    // ---- the cut: the key of the last of the `need` best unforced blocks (there are more than `need`) ----
    int need = K - a.sink - a.recent;
    uint32_t cut = 0xffffffffu;  // taken: keys above `cut`, and the first `need` equal to it
    if (need > 0) {
        kl = misc[0];
        kh = misc[1];
        for (;;) {
            // bins of 2^sh keys over [kl, kh]
            const int sh = max(0, 24 - __clz((int)(kh - kl)));
            for (int j = f0 + tid; j < f1; j += NT) {
                const uint32_t k = keys[j];
                if (k >= kl && k <= kh) atomicAdd(&hist[(k - kl) >> sh], 1u);
            }
            __syncthreads();
            if (warp == 0) {
                // lane l: bins 255 - 8 l .. 248 - 8 l, from the top
                const uint4 h1 = reinterpret_cast<const uint4 *>(hist)[63 - 2 * lane],
                            h0 = reinterpret_cast<const uint4 *>(hist)[62 - 2 * lane];
                const uint32_t s[8] = {h1.w, h1.z, h1.y, h1.x, h0.w, h0.z, h0.y, h0.x};
                uint32_t sum = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) sum += s[i];
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
                            misc[2] = 255 - 8 * lane - i;  // the bin that holds the cut
                            misc[3] = acc;                 // keys above it
                            misc[4] = s[i];
                        }
                        acc += s[i];
                    }
                }
            }
            __syncthreads();
            const uint32_t bin = misc[2], above = misc[3], in = misc[4];
            need -= (int)above;
            kl += bin << sh;
            if (in == (uint32_t)need && kl > 0) {  // the whole bin is taken
                cut = kl - 1;
                need = 0;
                break;
            }
            if (sh == 0) {  // one key per bin
                cut = kl;
                break;
            }
            // the bin's end, from the distance: kl + 2^sh - 1 itself may pass 2^32 (bins of 2^24 keys
            // below +inf, the key of every block whose box is not finite)
            kh = kl + min(kh - kl, (1u << sh) - 1);
            if (in <= S::CAND) {
                // the bin's keys, ranked against each other
                for (int j = f0 + tid; j < f1; j += NT) {
                    const uint32_t k = keys[j];
                    if (k >= kl && k <= kh) cand[atomicAdd(&misc[5], 1u)] = k;
                }
                __syncthreads();
                for (int i = tid; i < (int)in; i += NT) {
                    const uint32_t k = cand[i];
                    int gt = 0, ge = 0;
                    for (int x = 0; x < (int)in; ++x) {
                        gt += cand[x] > k;
                        ge += cand[x] >= k;
                    }
                    if (gt < need && need <= ge) {  // equal keys write the same
                        misc[6] = k;
                        misc[7] = (uint32_t)(need - gt);
                    }
                }
                __syncthreads();
                cut = misc[6];
                need = (int)misc[7];
                break;
            }
            for (int i = tid; i < 256; i += NT) hist[i] = 0;
            __syncthreads();
        }
    }

    // ---- the picks in index order: every thread a run of the row (of odd length: the lanes' reads
    // fall into different banks); K of them in all, and none is written past the row's list ----
    const int run = (n + NT - 1) / NT | 1, r0 = min(n, tid * run), r1 = min(n, r0 + run);
    auto cls = [&](int j) {  // 2: taken, 1: equal to the cut
        const uint32_t k = keys[j];
        return j < f0 || j >= f1 || k > cut ? 2 : k == cut ? 1 : 0;
    };
    // of the run: how many, and (up to 32 blocks) which
    uint32_t gt = 0, eq = 0, gm = 0, em = 0;
#pragma unroll 4
    for (int j = r0; j < r1; ++j) {
        const int k = cls(j);
        gt += k == 2;
        eq += k == 1;
        gm |= (uint32_t)(k == 2) << ((j - r0) & 31);
        em |= (uint32_t)(k == 1) << ((j - r0) & 31);
    }
    uint32_t gs = gt, es = eq;  // inclusive over the threads
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, gs, o), z = __shfl_up_sync(0xffffffffu, es, o);
        if (lane >= o) {
            gs += y;
            es += z;
        }
    }
    if (lane == 31) {
        wa[warp] = gs;
        wb[warp] = es;
    }
    __syncthreads();
    uint32_t at = gs - gt, eqs = es - eq;
#pragma unroll
    for (int w = 0; w < nw; ++w)
        if (w < warp) {
            at += wa[w];
            eqs += wb[w];
        }
    at += min(eqs, (uint32_t)need);
    if (run <= 32) {
        for (uint32_t all = gm | em; all; all &= all - 1) {
            const uint32_t bit = all & -all;
            if (((gm & bit) || eqs++ < (uint32_t)need) && at < (uint32_t)K) out[at++] = r0 + __ffs(bit) - 1;
        }
    } else if (gt + eq) {
        for (int j = r0; j < r1; ++j) {
            const int k = cls(j);
            if ((k == 2 || (k == 1 && eqs++ < (uint32_t)need)) && at < (uint32_t)K) out[at++] = j;
        }
    }
    if (tid == 0) a.nsel[(size_t)r * a.H + h] = K;
}

}  // namespace pa

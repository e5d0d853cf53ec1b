// Attention of one (query row, KV head) over its chosen blocks, as device code: the whole of
// pa_decode_selected and the second half of pa_decode_sparse.
//
//   out[g] = sum_t softmax_t(scale q[g] . K[t]) V[t] over the tokens t of the chosen blocks
//
// A cluster of CTAs shares a row: the chosen blocks go round its warps.  Every warp works
// alone on its blocks, with its own ring of (K tile, V tile) stages that TMA fills (one copy
// per tile: a block's tile of one KV head is contiguous), a running maximum and sum per head,
// and its share of the output in registers; the shares are joined once at the end, first the
// CTA's warps through shared memory, then the cluster's CTAs through distributed shared
// memory.  So a row needs no workspace and one launch, and the order of every sum is fixed.
//
// Tensor-core form (mma.sync m16n8k16, fp32 accumulators, NT * 8 query heads): with the tokens
// on the M side for up to 8 heads and for int8 caches (stream_tokens_m), with the heads there for
// 16 or 32 (stream_heads_m); either way a tile is read from shared memory once for all heads.
// bf16 rounds P to 8 bits, too few for the result's own precision, so there P = hi + lo, two
// products.  fp16's 11 bits move the result by at most 2^-11 of the largest |v|, as far as its own
// rounding to fp16 may (as pa_decode does; in an fp32 output it is the largest error left).  An int8 tile's codes become exact fp16 / bf16 fragments in
// registers; the block's K scale multiplies the scores, its V scale the block's product, in fp32.
//
// Bound by DRAM where there are rows enough (512 rows x 64 fp16 blocks of 16 x 128: 45 us, 5.9
// TB/s), by the chain list -> table entry -> tiles -> joining where there are few (8 rows: about
// 5 us), and for int8 by each warp's chain tile -> unpacking -> MMA -> softmax -> unpacking -> MMA,
// with three warps a scheduler and half of the issue slots used (128 rows x 128 blocks 19.6 us, 3.4
// TB/s).  fp32: 512 rows x 64 blocks 142 us, 3.8 TB/s.
#pragma once
#include <cooperative_groups.h>

#include <type_traits>

#include "pa_mma.cuh"
#include "pa_select.cuh"
#include "pa_tc_shared.cuh"

namespace pa {

__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap *map, int tile, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3}], [%4];" ::
            "r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(tile), "r"(bar)
        : "memory");
}

// Bytes b0, b1 of u (int8 values biased by 128) as an exact pair of T.
template <typename T>
__device__ __forceinline__ uint32_t i8_pair(uint32_t u, int b0, int b1) {
    if constexpr (std::is_same<T, __half>::value) {
        return i8x2_to_h2(u, 0x5040u | (uint32_t)(b1 << 8) | (uint32_t)b0);
    } else {
        // 0x4b0000xx is 2^23 + xx: subtracting 2^23 + 128 leaves the value, which bf16's 8 bits hold
        const float lo = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7540u | (uint32_t)b0)) - 8388736.f;
        const float hi = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7540u | (uint32_t)b1)) - 8388736.f;
        return Mma<T>::pack(lo, hi);
    }
}

// Shared-memory layout of the tensor-core form; NWARPS warps per CTA.
template <typename T, typename TKV, int D, int NT, int NWARPS>
struct AttendCfg {
    static constexpr bool I8 = std::is_same<TKV, int8_t>::value;
    static constexpr int NW = NWARPS;
    static constexpr int ROWB = D * (int)sizeof(TKV);                  // bytes per cache row
    static constexpr int SEGB = ROWB < 128 ? ROWB : 128;               // bytes per box row
    static constexpr int TILE = 16 * ROWB;
    static constexpr int STAGE = 2 * TILE;
    // Blocks per step: with two, the step's maximum, its exchanges between lanes and the rescaling
    // are shared by 32 tokens.  The ring holds one step or 16 KB a warp: the warps of several CTAs
    // on an SM take turns at waiting, so a deeper ring would only cost residency.
    static constexpr int NB = TILE > 4096 ? 1 : 2;
    static constexpr int S = STAGE >= 8192 ? 2 : 16384 / STAGE;        // stages per warp
    static constexpr int HEADS = NT * 8;
    static constexpr int QROW = D * 2 + 16;                            // bytes: rows fall into different banks
    static constexpr int OROW = D + 4;                                 // floats
    static constexpr int RING = NW * S * STAGE;
    static constexpr int JOIN = NW * HEADS * OROW * 4;                 // the joining reuses the ring
    static constexpr int Q_OFF = RING > JOIN ? RING : JOIN;
    static constexpr int BAR_OFF = Q_OFF + HEADS * QROW;
    static constexpr int INFO_OFF = BAR_OFF + NW * S * 8;              // int [NW][S]: tokens of the stage's block, 0: none
    static constexpr int ML_OFF = INFO_OFF + NW * S * 4;               // float [NW][2][HEADS], then [2][HEADS]
    static constexpr int BYTES = 1024 + ML_OFF + (NW + 1) * 2 * HEADS * 4;
    static constexpr bool QREG = NT * D <= 256;                        // q fragments kept in registers
};

// Joins the warps' and the CTAs' shares and writes the output.  o: float [NW][HEADS][OROW] shares of
// the CTA's warps; ml: float [NW][2][HEADS] their maxima and sums, then [2][HEADS] for the CTA's own.
template <typename T, int D, int HEADS, int OROW, int NW>
__device__ __forceinline__ void join_shares(const SparseArgs &a, float *o, float *ml, int ncol, size_t out0, int rank,
                                            int ncta) {
    constexpr int Q4 = D / 4;  // vectors of four per head
    const int tid = threadIdx.x, nt = NW * 32;
    const float kNegInf = __int_as_float(0xff800000);
    float *mine = ml + NW * 2 * HEADS;
    __syncthreads();
    if (tid < HEADS) {
        float M = kNegInf, l = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) M = fmaxf(M, ml[w * 2 * HEADS + tid]);
        const float Mu = M == kNegInf ? 0.f : M;
        float f[NW];
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            f[w] = fast_exp2(ml[w * 2 * HEADS + tid] - Mu);
            l += f[w] * ml[w * 2 * HEADS + HEADS + tid];
        }
        // one CTA: the weights are final
        const float inv = ncta > 1 ? 1.f : l == 0.f ? 0.f : __fdividef(1.f, l);
#pragma unroll
        for (int w = 0; w < NW; ++w) ml[w * 2 * HEADS + tid] = f[w] * inv;
        mine[tid] = M;
        mine[HEADS + tid] = l;
    }
    __syncthreads();
    for (int i = tid; i < ncol * Q4; i += nt) {
        const int g = i / Q4, d = i % Q4 * 4;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float f = ml[w * 2 * HEADS + g];
            const float4 v = *reinterpret_cast<const float4 *>(o + (w * HEADS + g) * OROW + d);
            s.x += f * v.x;
            s.y += f * v.y;
            s.z += f * v.z;
            s.w += f * v.w;
        }
        if (ncta == 1) {
            store_out2<T>(a.out, a.out_f32, out0 + (size_t)g * D + d, s.x, s.y);
            store_out2<T>(a.out, a.out_f32, out0 + (size_t)g * D + d + 2, s.z, s.w);
        } else {
            *reinterpret_cast<float4 *>(o + g * OROW + d) = s;
        }
    }
    if (ncta == 1) return;
    cooperative_groups::cluster_group cl = cooperative_groups::this_cluster();
    cl.sync();
    // the CTAs take turns at the row's vectors; a vector's shares, maxima and sums are read together
    for (int i = rank * nt + tid; i < ncol * Q4; i += ncta * nt) {
        const int g = i / Q4, d = i % Q4 * 4;
        float4 v[8], s = make_float4(0.f, 0.f, 0.f, 0.f);
        float m[8], l[8], M = kNegInf, sum = 0.f;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            m[r] = kNegInf;
            l[r] = 0.f;
            if (r < ncta) {
                m[r] = *cl.map_shared_rank(mine + g, r);
                l[r] = *cl.map_shared_rank(mine + HEADS + g, r);
                v[r] = *cl.map_shared_rank(reinterpret_cast<float4 *>(o + g * OROW + d), r);
            }
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) M = fmaxf(M, m[r]);
        if (M == kNegInf) M = 0.f;
#pragma unroll
        for (int r = 0; r < 8; ++r)
            if (r < ncta) {
                const float f = fast_exp2(m[r] - M);
                sum += f * l[r];
                s.x += f * v[r].x;
                s.y += f * v[r].y;
                s.z += f * v[r].z;
                s.w += f * v[r].w;
            }
        const float inv = sum == 0.f ? 0.f : __fdividef(1.f, sum);
        store_out2<T>(a.out, a.out_f32, out0 + (size_t)g * D + d, s.x * inv, s.y * inv);
        store_out2<T>(a.out, a.out_f32, out0 + (size_t)g * D + d + 2, s.z * inv, s.w * inv);
    }
    cl.sync();  // no CTA ends while another reads its shares
}

// Zeroes the V rows behind the last token of a step's blocks: a weight of 0 does not make a NaN
// there 0.
template <typename C, int NB>
__device__ __forceinline__ void zero_rows_past(const uint32_t (&vt)[NB], const int (&valid)[NB], int lane) {
#pragma unroll
    for (int n1 = 0; n1 < NB; ++n1)
        for (int i = lane; i < (kBlockSize - valid[n1]) * (C::ROWB / 16); i += 32) {
            const int row = valid[n1] + i / (C::ROWB / 16), ch = i % (C::ROWB / 16);
            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(swz(vt[n1] + (ch >> 3) * 2048, row, ch & 7)), "r"(0)
                         : "memory");
        }
    fence_proxy_async_smem();
    __syncwarp();
}

// The streaming part of attend_row with the tokens on the MMA's M side, for up to 8 heads per n-tile
// and for int8 caches:
//   S^T[16 tokens x heads] = K[16 x D] . Q^T[D x heads]     (A = K tile, B = q)
//   O^T[D x heads]        += V^T[D x 16] . P^T[16 x heads]  (A = V tile^T, B = p)
// arrived(k, ...): waits for blocks k .. k + NB - 1 of the warp; issue(k): requests block k.
// ks, vs8: the int8 scales of the last two batches of 32 blocks, a block per lane.
template <typename T, typename TKV, int D, int NT, int NWARPS, typename Arrived, typename Issue>
__device__ __forceinline__ void stream_tokens_m(const SparseArgs &a, unsigned char *smem, int cnt, const float (&ks)[2],
                                                const float (&vs8)[2], Arrived arrived, Issue issue) {
    using C = AttendCfg<T, TKV, D, NT, NWARPS>;
    constexpr int S = C::S, NB = C::NB, KS = D / 16, MT = D / 16;
    constexpr bool SPLIT_P = !std::is_same<T, __half>::value;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const uint32_t sb = smem_addr(smem);
    // B fragments of k-steps ks (and, 16-bit caches, ks + 1) of n-tile t, the dims in the order of
    // the K fragments
    auto qfrag = [&](int t, int ks, uint32_t (&f)[4]) {
        if constexpr (!C::I8) {
            ldsm_x4(f, sb + C::Q_OFF + (t * 8 + (lane & 7)) * C::QROW + ks * 32 + (lane >> 3) * 16);
        } else {
            // thread column c reads 32 (D = 64: 16) contiguous bytes per 128-byte segment of a row
            const int d0 = D == 64 ? c * 16 + ks * 4 : (ks / 8) * 128 + c * 32 + (ks % 8) * 4;
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
                         : "r"(sb + C::Q_OFF + (t * 8 + g) * C::QROW + d0 * 2)
                         : "memory");
        }
    };
    uint32_t qb[C::QREG ? NT : 1][C::QREG ? KS / 2 : 1][4];
    if constexpr (C::QREG) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int ks = 0; ks < KS; ks += 2) qfrag(t, ks, qb[t][ks / 2]);
    }

    float o[NT][MT][4] = {};
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        m[t][0] = m[t][1] = __int_as_float(0xff800000);
        l[t][0] = l[t][1] = 0.f;
    }

    int k = 0;  // below cnt after the loop: a copy did not land
    for (; k < cnt; k += NB) {
        int valid[NB];
        uint32_t kt[NB], vt[NB];
        bool whole;
        if (!arrived(k, valid, kt, vt, whole)) break;
        // ---- S^T ----
        float x[NB][NT][4];
#pragma unroll
        for (int n1 = 0; n1 < NB; ++n1)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[n1][t][e] = 0.f;
#pragma unroll
        for (int k2 = 0; k2 < KS; k2 += 2) {
            uint32_t qf[C::QREG ? 1 : NT][4];
            if constexpr (!C::QREG) {
#pragma unroll
                for (int t = 0; t < NT; ++t) qfrag(t, k2, qf[t]);
            }
#pragma unroll
            for (int n1 = 0; n1 < NB; ++n1) {
                uint32_t af[2][4];
                if constexpr (!C::I8) {
                    const int row = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int ch = (k2 + u) * 2 + (lane >> 4);
                        ldsm_x4(af[u], swz(kt[n1] + (ch >> 3) * 2048, row, ch & 7));
                    }
                } else {
                    // 8 bytes of tokens g and g + 8
                    uint32_t wa[2], wb[2];
                    uint32_t pa, pb;
                    if constexpr (D == 64) {
                        pa = kt[n1] + g * 64 + c * 16 + k2 * 4;
                        pb = pa + 8 * 64;
                    } else {
                        const uint32_t seg = kt[n1] + (k2 / 8) * 2048;
                        pa = swz(seg, g, 2 * c + (k2 % 8) / 4) + (k2 % 4) * 4;
                        pb = swz(seg, g + 8, 2 * c + (k2 % 8) / 4) + (k2 % 4) * 4;
                    }
                    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(wa[0]), "=r"(wa[1]) : "r"(pa) : "memory");
                    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(wb[0]), "=r"(wb[1]) : "r"(pb) : "memory");
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint32_t ua = wa[u] ^ 0x80808080u, ub = wb[u] ^ 0x80808080u;
                        af[u][0] = i8_pair<T>(ua, 0, 1);
                        af[u][1] = i8_pair<T>(ub, 0, 1);
                        af[u][2] = i8_pair<T>(ua, 2, 3);
                        af[u][3] = i8_pair<T>(ub, 2, 3);
                    }
                }
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const uint32_t *f = C::QREG ? qb[t][k2 / 2] : qf[t];
                        Mma<T>::mma(x[n1][t], af[u], f[2 * u], f[2 * u + 1]);
                    }
            }
        }
#pragma unroll
        for (int n1 = 0; n1 < NB; ++n1) {
            float sc = a.scale_log2;
            if constexpr (C::I8)
                sc *= __shfl_sync(0xffffffffu, (k + n1) >> 5 & 1 ? ks[1] : ks[0], (k + n1) & 31);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[n1][t][e] *= sc;
        }
        if (!whole) {  // rows past the last token hold anything, NaN among it
#pragma unroll
            for (int n1 = 0; n1 < NB; ++n1)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (g + 8 * (e >> 1) >= valid[n1]) x[n1][t][e] = __int_as_float(0xff800000);
        }
        // ---- running maximum and sum; P ----
        // The reference of the exponentials follows the maximum only when that grew by more than
        // 2^8: weights of up to 2^8 are as exact, and the output is seldom rescaled.
        uint32_t ph[NB][NT][2], pl[SPLIT_P ? NB : 1][SPLIT_P ? NT : 1][2];
        float mx[NT][2];
        bool grew = false;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float v = fmaxf(x[0][t][e], x[0][t][2 + e]);
                if constexpr (NB > 1) v = fmaxf(v, fmaxf(x[1][t][e], x[1][t][2 + e]));
                mx[t][e] = v;
            }
#pragma unroll
        for (int d = 4; d < 32; d <<= 1)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) mx[t][e] = fmaxf(mx[t][e], __shfl_xor_sync(0xffffffffu, mx[t][e], d));
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) grew |= mx[t][e] > m[t][e] + 8.f;
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float al[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float mn = mx[t][e] > m[t][e] + 8.f ? mx[t][e] : m[t][e];
                    al[e] = m[t][e] == mn ? 1.f : fast_exp2(m[t][e] - mn);
                    m[t][e] = mn;
                    l[t][e] *= al[e];
                }
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[t][i][e] *= al[e & 1];
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float mu[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) mu[e] = m[t][e] == __int_as_float(0xff800000) ? 0.f : m[t][e];
#pragma unroll
            for (int n1 = 0; n1 < NB; ++n1) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[n1][t][e] = fast_exp2(x[n1][t][e] - mu[e & 1]);
                    l[t][e & 1] += x[n1][t][e];
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {  // tokens g (e = 0) and g + 8, heads 2c, 2c + 1
                    const uint32_t hi = Mma<T>::pack(x[n1][t][2 * e], x[n1][t][2 * e + 1]);
                    ph[n1][t][e] = movm_t(hi);
                    if constexpr (SPLIT_P) {
                        const float h0 = __uint_as_float(hi << 16), h1 = __uint_as_float(hi & 0xffff0000u);
                        pl[n1][t][e] = movm_t(Mma<T>::pack(x[n1][t][2 * e] - h0, x[n1][t][2 * e + 1] - h1));
                    }
                }
            }
        }
        // ---- O^T ----
        if constexpr (!C::I8) {
            if (!whole) zero_rows_past<C, NB>(vt, valid, lane);
            const int row = (lane & 7) + ((lane >> 4) & 1) * 8;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int ch = i * 2 + ((lane >> 3) & 1);
#pragma unroll
                for (int n1 = 0; n1 < NB; ++n1) {
                    uint32_t af[4];
                    ldsm_x4_t(af, swz(vt[n1] + (ch >> 3) * 2048, row, ch & 7));
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        Mma<T>::mma(o[t][i], af, ph[n1][t][0], ph[n1][t][1]);
                        if constexpr (SPLIT_P) Mma<T>::mma(o[t][i], af, pl[n1][t][0], pl[n1][t][1]);
                    }
                }
            }
        } else {
            constexpr int MS = D == 64 ? 4 : 8, VW = D == 64 ? 2 : 4;  // m-tiles and words per segment
#pragma unroll
            for (int n1 = 0; n1 < NB; ++n1) {
                // a block that is not there: its codes are whatever the stage held, times 0
                const float vb = __shfl_sync(0xffffffffu, (k + n1) >> 5 & 1 ? vs8[1] : vs8[0], (k + n1) & 31);
                const float vs = valid[n1] > 0 ? vb : 0.f;
#pragma unroll
                for (int sg = 0; sg < MT / MS; ++sg) {
                    uint32_t rw[4][4];  // tokens 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int row = 2 * c + (q & 1) + 8 * (q >> 1);
                        if constexpr (D == 64) {
                            asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                                         : "=r"(rw[q][0]), "=r"(rw[q][1])
                                         : "r"(vt[n1] + row * 64 + g * 8)
                                         : "memory");
                        } else {
                            lds_v4(rw[q], swz(vt[n1] + sg * 2048, row, g));
                        }
#pragma unroll
                        for (int e = 0; e < VW; ++e) rw[q][e] ^= 0x80808080u;
                    }
#pragma unroll
                    for (int i = 0; i < MS; ++i) {
                        uint32_t af[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {  // token pair q / 2, dims row (q & 1 ? g + 8 : g)
                            const int p = q >> 1, wd = (q & 1) * (VW / 2) + i / 4;
                            const uint32_t sl = (uint32_t)(i & 3) | (uint32_t)(4 + (i & 3)) << 4;
                            af[q] = i8_pair<T>(__byte_perm(rw[2 * p][wd], rw[2 * p + 1][wd], sl), 0, 1);
                        }
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            float d[4];
                            Mma<T>::mma0(d, af, ph[n1][t][0], ph[n1][t][1]);
                            if constexpr (SPLIT_P) Mma<T>::mma(d, af, pl[n1][t][0], pl[n1][t][1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[t][sg * MS + i][e] += vs * d[e];
                        }
                    }
                }
            }
        }
        __syncwarp();
#pragma unroll
        for (int n1 = 0; n1 < NB; ++n1) issue(k + S + n1);
    }

    // ---- this warp's share, for the joining (after a copy that did not land, a sum that makes the
    // whole row NaN, whatever lands in the shares) ----
    float *os = reinterpret_cast<float *>(smem);
    float *ml = reinterpret_cast<float *>(smem + C::ML_OFF);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (k < cnt) l[t][e] = __int_as_float(0x7fffffff);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], d);
            if (g == 0) {
                ml[warp * 2 * C::HEADS + t * 8 + 2 * c + e] = m[t][e];
                ml[(warp * 2 + 1) * C::HEADS + t * 8 + 2 * c + e] = l[t][e];
            }
        }
    __syncthreads();  // every ring is empty: the shares go there
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                int d;
                if constexpr (!C::I8)
                    d = i * 16 + g + 8 * (e >> 1);
                else if constexpr (D == 64)
                    d = g * 8 + i + 4 * (e >> 1);
                else
                    d = (i / 8) * 128 + g * 16 + i % 8 + 8 * (e >> 1);
                os[(warp * C::HEADS + t * 8 + 2 * c + (e & 1)) * C::OROW + d] = o[t][i][e];
            }
}

// The same with the heads on the M side, for groups of 16 or 32 columns of 16-bit caches:
//   S[16 heads x 8 tokens] = Q[16 x D] . K^T[D x 8]     (A = q, B = K tile)
//   O[16 heads x D]       += P[16 x 16 tokens] . V[16 x D]  (A = p, B = V tile)
// P's fragments are S's accumulators as they stand, a row's maximum lies in four lanes instead of
// eight, and q's fragments take half as many reads, which is what bounded the form above at 32
// heads (shared-memory reads and exchanges between lanes).
template <typename T, int D, int NT, int NWARPS, typename Arrived, typename Issue>
__device__ __forceinline__ void stream_heads_m(const SparseArgs &a, unsigned char *smem, int cnt, Arrived arrived,
                                               Issue issue) {
    using C = AttendCfg<T, T, D, NT, NWARPS>;
    constexpr int S = C::S, NB = C::NB, KS = D / 16, ML = NT / 2, NTK = 2 * NB;  // m-tiles of heads, n-tiles of tokens
    constexpr bool SPLIT_P = !std::is_same<T, __half>::value;
    constexpr bool QR = ML * KS <= 8;  // q fragments in registers
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const uint32_t sb = smem_addr(smem);
    const float kNegInf = __int_as_float(0xff800000);
    auto qfrag = [&](int t, int ks, uint32_t (&f)[4]) {
        ldsm_x4(f, sb + C::Q_OFF + (t * 16 + (lane & 15)) * C::QROW + ks * 32 + (lane >> 4) * 16);
    };
    uint32_t qa[QR ? ML : 1][QR ? KS : 1][4];
    if constexpr (QR) {
#pragma unroll
        for (int t = 0; t < ML; ++t)
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) qfrag(t, ks, qa[t][ks]);
    }
    float o[ML][D / 8][4] = {};
    float m[ML][2], l[ML][2];  // rows g and g + 8
#pragma unroll
    for (int t = 0; t < ML; ++t) {
        m[t][0] = m[t][1] = kNegInf;
        l[t][0] = l[t][1] = 0.f;
    }
    int k = 0;  // below cnt after the loop: a copy did not land
    for (; k < cnt; k += NB) {
        int valid[NB];
        uint32_t kt[NB], vt[NB];
        bool whole;
        if (!arrived(k, valid, kt, vt, whole)) break;
        // ---- S ----
        float x[ML][NTK][4] = {};
        const int krow = (lane & 7) + ((lane >> 4) & 1) * 8;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            uint32_t qf[ML][4];
            if constexpr (!QR) {
#pragma unroll
                for (int t = 0; t < ML; ++t) qfrag(t, ks, qf[t]);
            }
            const int ch = ks * 2 + ((lane >> 3) & 1);
#pragma unroll
            for (int n1 = 0; n1 < NB; ++n1) {
                uint32_t kf[4];
                ldsm_x4(kf, swz(kt[n1] + (ch >> 3) * 2048, krow, ch & 7));
#pragma unroll
                for (int t = 0; t < ML; ++t) {
                    uint32_t af[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if constexpr (QR)
                            af[e] = qa[t][ks][e];
                        else
                            af[e] = qf[t][e];
                    }
                    Mma<T>::mma(x[t][2 * n1], af, kf[0], kf[1]);
                    Mma<T>::mma(x[t][2 * n1 + 1], af, kf[2], kf[3]);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < ML; ++t)
#pragma unroll
            for (int n = 0; n < NTK; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[t][n][e] *= a.scale_log2;
        if (!whole) {  // tokens past the last one hold anything, NaN among it
#pragma unroll
            for (int n = 0; n < NTK; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if ((n & 1) * 8 + 2 * c + e >= valid[n / 2]) {
#pragma unroll
                        for (int t = 0; t < ML; ++t) x[t][n][e] = x[t][n][2 + e] = kNegInf;
                    }
        }
        // ---- running maximum and sum (the reference moves only when it grew by more than 2^8) ----
        float mx[ML][2];
        bool grew = false;
#pragma unroll
        for (int t = 0; t < ML; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                mx[t][r] = fmaxf(x[t][0][2 * r], x[t][0][2 * r + 1]);
#pragma unroll
                for (int n = 1; n < NTK; ++n) mx[t][r] = fmaxf(mx[t][r], fmaxf(x[t][n][2 * r], x[t][n][2 * r + 1]));
            }
#pragma unroll
        for (int d = 1; d < 4; d <<= 1)
#pragma unroll
            for (int t = 0; t < ML; ++t)
#pragma unroll
                for (int r = 0; r < 2; ++r) mx[t][r] = fmaxf(mx[t][r], __shfl_xor_sync(0xffffffffu, mx[t][r], d));
#pragma unroll
        for (int t = 0; t < ML; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) grew |= mx[t][r] > m[t][r] + 8.f;
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
            for (int t = 0; t < ML; ++t) {
                float al[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float mn = mx[t][r] > m[t][r] + 8.f ? mx[t][r] : m[t][r];
                    al[r] = m[t][r] == mn ? 1.f : fast_exp2(m[t][r] - mn);
                    m[t][r] = mn;
                    l[t][r] *= al[r];
                }
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[t][i][e] *= al[e >> 1];
            }
        }
        uint32_t ph[ML][NB][4], pl[SPLIT_P ? ML : 1][SPLIT_P ? NB : 1][4];
#pragma unroll
        for (int t = 0; t < ML; ++t) {
            float mu[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) mu[r] = m[t][r] == kNegInf ? 0.f : m[t][r];
#pragma unroll
            for (int n = 0; n < NTK; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float &p0 = x[t][n][2 * r], &p1 = x[t][n][2 * r + 1];
                    p0 = fast_exp2(p0 - mu[r]);
                    p1 = fast_exp2(p1 - mu[r]);
                    l[t][r] += p0 + p1;
                    const uint32_t hi = Mma<T>::pack(p0, p1);
                    ph[t][n / 2][(n & 1) * 2 + r] = hi;
                    if constexpr (SPLIT_P)
                        pl[t][n / 2][(n & 1) * 2 + r] =
                            Mma<T>::pack(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xffff0000u));
                }
        }
        // ---- O ----
        if (!whole) zero_rows_past<C, NB>(vt, valid, lane);
        const int vrow = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const int ch = i * 2 + (lane >> 4);
#pragma unroll
            for (int n1 = 0; n1 < NB; ++n1) {
                uint32_t vf[4];
                ldsm_x4_t(vf, swz(vt[n1] + (ch >> 3) * 2048, vrow, ch & 7));
#pragma unroll
                for (int t = 0; t < ML; ++t) {
                    Mma<T>::mma(o[t][2 * i], ph[t][n1], vf[0], vf[1]);
                    Mma<T>::mma(o[t][2 * i + 1], ph[t][n1], vf[2], vf[3]);
                    if constexpr (SPLIT_P) {
                        Mma<T>::mma(o[t][2 * i], pl[t][n1], vf[0], vf[1]);
                        Mma<T>::mma(o[t][2 * i + 1], pl[t][n1], vf[2], vf[3]);
                    }
                }
            }
        }
        __syncwarp();
#pragma unroll
        for (int n1 = 0; n1 < NB; ++n1) issue(k + S + n1);
    }
    // ---- this warp's share, for the joining (NaN as above) ----
    float *os = reinterpret_cast<float *>(smem);
    float *ml = reinterpret_cast<float *>(smem + C::ML_OFF);
#pragma unroll
    for (int t = 0; t < ML; ++t)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            if (k < cnt) l[t][r] = __int_as_float(0x7fffffff);
#pragma unroll
            for (int d = 1; d < 4; d <<= 1) l[t][r] += __shfl_xor_sync(0xffffffffu, l[t][r], d);
            if (c == 0) {
                ml[warp * 2 * C::HEADS + t * 16 + g + 8 * r] = m[t][r];
                ml[(warp * 2 + 1) * C::HEADS + t * 16 + g + 8 * r] = l[t][r];
            }
        }
    __syncthreads();  // every ring is empty: the shares go there
#pragma unroll
    for (int t = 0; t < ML; ++t)
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r)
                *reinterpret_cast<float2 *>(os + (warp * C::HEADS + t * 16 + g + 8 * r) * C::OROW + i * 8 + 2 * c) =
                    make_float2(o[t][i][2 * r], o[t][i][2 * r + 1]);
}

// Waits, with a limit, for the copies of blocks k .. end - 1 (out of line: the kernels that call it
// are at their registers, and it runs after a copy that did not land).
__device__ __noinline__ void drain_ring(uint64_t *bars, int S, int k, int end, unsigned long long limit_ns) {
    for (; k < end; ++k) mbar_wait(&bars[k % S], (k / S) & 1, limit_ns);
}

// The barriers of the warps' rings; before attend_row, and before the previous kernel is waited for.
template <typename C>
__device__ __forceinline__ void attend_init(unsigned char *smem) {
    if (threadIdx.x < C::NW * C::S) mbar_init(reinterpret_cast<uint64_t *>(smem + C::BAR_OFF) + threadIdx.x, 1);
    fence_mbar_init();
    __syncthreads();
}

// The chosen blocks of row r and KV head h, 8 * NT query heads from 8 * NT * grp on.
// smem: 1024-byte aligned, AttendCfg bytes, after attend_init.  Called by NW * 32 threads of each CTA.
template <typename T, typename TKV, int D, int NT, int NWARPS>
__device__ void attend_row(const SparseArgs &a, const CUtensorMap *tmK, const CUtensorMap *tmV, int r, int h, int grp,
                           int rank, int ncta, unsigned char *smem) {
    using C = AttendCfg<T, TKV, D, NT, NWARPS>;
    constexpr int NW = C::NW, S = C::S, NB = C::NB;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t sb = smem_addr(smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF) + warp * S;
    int *info = reinterpret_cast<int *>(smem + C::INFO_OFF) + warp * S;
    const uint32_t ring = sb + warp * S * C::STAGE;

    // The first copies wait for a chain of loads: list entry, its table entry.  Neither asks
    // for the row's length or the list's (any entry inside the table is read, and judged
    // later), so those and q are on their way at the same time.
    const size_t list = (size_t)r * a.H + h;
    const int32_t *sel = a.sel + list * a.K, *table = a.tables + (size_t)(r / a.Q) * a.M;
    const int W = ncta * NW, w = rank * NW + warp;
    // the warp's blocks: lane l of a batch of 32 holds the l-th
    int p_j = -1, p_x = -1, p_y = -1;
    // int8 scales of the items of the last two batches, asked for with the batch and used when its
    // blocks are: no copy waits for them
    float b_ks[2] = {0.f, 0.f}, b_vs[2] = {0.f, 0.f};
    auto load_list = [&](int k) {  // items k .. k + 31
        const int64_t i = (int64_t)(k + lane) * W + w;
        p_j = i < a.K ? __ldcg(sel + i) : -1;
        p_x = p_j >= 0 && p_j < a.M ? __ldcg(table + p_j) : -1;
    };
    load_list(0);
    const int ncol = min(C::HEADS, a.G - grp * C::HEADS);
    const size_t row0 = ((size_t)r * a.Hq + (size_t)h * a.G + (size_t)grp * C::HEADS) * D;
    constexpr int QN = (C::HEADS * D / 8 + NW * 32 - 1) / (NW * 32);  // 16-byte vectors of q per thread
    uint4 qv[QN];
    const bool qvec = ((uintptr_t)a.q & 15) == 0;
    if (qvec) {
#pragma unroll
        for (int i = 0; i < QN; ++i) {
            const int e = tid + i * NW * 32;
            qv[i] = e < ncol * (D / 8) ? __ldg(reinterpret_cast<const uint4 *>(reinterpret_cast<const T *>(a.q) + row0) + e)
                                       : make_uint4(0, 0, 0, 0);
        }
    }
    int b;
    const int L = sparse_row_len(a, r, b), nb = (L + kBlockSize - 1) / kBlockSize;
    const int n = min(max(__ldcg(a.nsel + list), 0), a.K);
    const int cnt = n > w ? (n - w + W - 1) / W : 0;

    constexpr int kStalled = -2;
    auto judge = [&](int k) {
        p_y = -1;
        if (k + lane < cnt && p_j >= 0 && p_j < nb) {  // entries outside the row's blocks are skipped
            if (p_x >= 0 && (int64_t)p_x < a.N) {
                p_y = p_x * a.H + h;  // host: num_blocks * H below 2^31
                if constexpr (C::I8) {
                    if (k >> 5 & 1) {
                        b_ks[1] = __ldg(a.ks + p_y);
                        b_vs[1] = __ldg(a.vs + p_y);
                    } else {
                        b_ks[0] = __ldg(a.ks + p_y);
                        b_vs[0] = __ldg(a.vs + p_y);
                    }
                }
            } else {
                raise_flag(PA_EFLAG_BAD_BLOCK);
            }
        }
        // the failure-path self-test leaves one block's copies unissued (never in a normal call)
        if (k + lane == a.stall_at && warp == 0 && blockIdx.x == 0 && p_y >= 0) p_y = kStalled;
    };
    auto issue = [&](int k) {
        if (k >= cnt) return;
        if (k % 32 == 0) {
            if (k > 0) load_list(k);
            judge(k);
        }
        const int y = __shfl_sync(0xffffffffu, p_y, k % 32), j = __shfl_sync(0xffffffffu, p_j, k % 32);
        if (lane == 0) {
            const int s = k % S;
            if (y >= 0) {
                mbar_arrive_expect_tx(&bars[s], C::STAGE);
                tma_tile(ring + s * C::STAGE, tmK, y, smem_addr(&bars[s]));
                tma_tile(ring + s * C::STAGE + C::TILE, tmV, y, smem_addr(&bars[s]));
            } else if (y == kStalled) {
                mbar_arrive_expect_tx(&bars[s], C::STAGE);
            } else {
                mbar_arrive(&bars[s]);
            }
            info[s] = y >= 0 ? min(kBlockSize, L - j * kBlockSize) : 0;
        }
        __syncwarp();
    };
#pragma unroll
    for (int k = 0; k < S; ++k) issue(k);

    // ---- q: rows of 8 * NT heads, zeros past the group ----
    if (qvec) {
#pragma unroll
        for (int i = 0; i < QN; ++i) {
            const int e = tid + i * NW * 32;
            if (e < C::HEADS * (D / 8))
                *reinterpret_cast<uint4 *>(smem + C::Q_OFF + (e / (D / 8)) * C::QROW + (e % (D / 8)) * 16) = qv[i];
        }
    } else {
        uint16_t *qd = reinterpret_cast<uint16_t *>(smem + C::Q_OFF);
        const uint16_t *qsrc = reinterpret_cast<const uint16_t *>(a.q) + row0;
        for (int i = tid; i < C::HEADS * D; i += NW * 32) {
            const int hd = i / D, d = i % D;
            qd[hd * (C::QROW / 2) + d] = hd < ncol ? qsrc[i] : (uint16_t)0;
        }
    }
    __syncthreads();
    // blocks k .. k + NB - 1: waits for their copies; false: give up
    auto arrived = [&](int k, int (&valid)[NB], uint32_t (&kt)[NB], uint32_t (&vt)[NB], bool &whole) -> bool {
        bool landed = true;
#pragma unroll
        for (int n1 = 0; n1 < NB; ++n1)
            if (k + n1 < cnt) landed &= mbar_wait(&bars[(k + n1) % S], ((k + n1) / S) & 1, a.wait_ns);
        if (!__all_sync(0xffffffffu, landed)) {  // (the lanes give up together)
            // every copy still in flight, the late ones among them, is waited for once more, again
            // with a limit: the joining reuses the ring, and the next CTA this memory
            drain_ring(bars, S, k, min(k + S, cnt), a.wait_ns);
            return false;
        }
        whole = true;
#pragma unroll
        for (int n1 = 0; n1 < NB; ++n1) {
            const int s = (k + n1) % S;
            valid[n1] = k + n1 < cnt ? info[s] : 0;
            whole &= valid[n1] == kBlockSize;
            kt[n1] = ring + s * C::STAGE;
            vt[n1] = kt[n1] + C::TILE;
        }
        return true;
    };
    if constexpr (NT >= 2 && !C::I8)
        stream_heads_m<T, D, NT, NWARPS>(a, smem, cnt, arrived, issue);
    else
        stream_tokens_m<T, TKV, D, NT, NWARPS>(a, smem, cnt, b_ks, b_vs, arrived, issue);
    join_shares<T, D, C::HEADS, C::OROW, NW>(a, reinterpret_cast<float *>(smem), reinterpret_cast<float *>(smem + C::ML_OFF),
                                             ncol, row0, rank, ncta);
}

// fp32 caches: the same on the CUDA cores, GT query heads at a time, tiles read from global
// memory.  Lane (token t = lane % 16, half = lane / 16) takes half of the dims of its token's
// product; the output's dims go over the lanes.
template <int D, int GT>
struct AttendF32Cfg {
    static constexpr int NW = 4, OROW = D + 4;
    static constexpr int Q_OFF = NW * GT * OROW * 4;
    static constexpr int ML_OFF = Q_OFF + GT * D * 4;
    static constexpr int BYTES = ML_OFF + (NW + 1) * 2 * GT * 4;
};

template <int D, int GT>
__device__ void attend_row_f32(const SparseArgs &a, int r, int h, int grp, int rank, int ncta, unsigned char *smem) {
    using C = AttendF32Cfg<D, GT>;
    constexpr int NW = C::NW, DL = D / 32, VL = DL < 4 ? DL : 4;  // dims per lane, per vector
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float *os = reinterpret_cast<float *>(smem), *qs = reinterpret_cast<float *>(smem + C::Q_OFF),
          *ml = reinterpret_cast<float *>(smem + C::ML_OFF);
    // as in attend_row: the list and its table entries wait for no length
    const size_t list = (size_t)r * a.H + h;
    const int32_t *sel = a.sel + list * a.K, *table = a.tables + (size_t)(r / a.Q) * a.M;
    const int W = ncta * NW, w = rank * NW + warp;
    int p_j = -1, p_x = -1;
    auto load_list = [&](int k) {  // items k .. k + 31 of the warp, one per lane
        const int64_t i = (int64_t)(k + lane) * W + w;
        p_j = i < a.K ? __ldcg(sel + i) : -1;
        p_x = p_j >= 0 && p_j < a.M ? __ldcg(table + p_j) : -1;
    };
    load_list(0);
    const int ncol = min(GT, a.G - grp * GT);
    const size_t row0 = ((size_t)r * a.Hq + (size_t)h * a.G + (size_t)grp * GT) * D;
    for (int i = tid; i < GT * D; i += NW * 32)
        qs[i] = i < ncol * D ? __ldg(reinterpret_cast<const float *>(a.q) + row0 + i) : 0.f;
    int b;
    const int L = sparse_row_len(a, r, b), nb = (L + kBlockSize - 1) / kBlockSize;
    const int n = min(max(__ldcg(a.nsel + list), 0), a.K);
    const int cnt = n > w ? (n - w + W - 1) / W : 0;
    __syncthreads();
    float o[GT][DL] = {}, m[GT], l[GT];
#pragma unroll
    for (int t = 0; t < GT; ++t) {
        m[t] = __int_as_float(0xff800000);
        l[t] = 0.f;
    }
    const int tok = lane & 15, half = lane >> 4;
    constexpr bool VREG = DL <= 4;  // the 16 rows of V on their way while the scores are made
    for (int k = 0; k < cnt; ++k) {
        if (k > 0 && k % 32 == 0) load_list(k);
        const int j = __shfl_sync(0xffffffffu, p_j, k % 32), x = __shfl_sync(0xffffffffu, p_x, k % 32);
        if (j < 0 || j >= nb) continue;
        if (x < 0 || (int64_t)x >= a.N) {
            if (lane == 0) raise_flag(PA_EFLAG_BAD_BLOCK);
            continue;
        }
        const int valid = min(kBlockSize, L - j * kBlockSize);
        const size_t tile = ((size_t)x * a.H + h) * (kBlockSize * D);
        const float4 *kp = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(a.kc) + tile + tok * D + half * (D / 2));
        const float *vp = reinterpret_cast<const float *>(a.vc) + tile + lane * VL;
        auto vrow = [&](int u, float *v) {
#pragma unroll
            for (int e = 0; e < DL; e += VL) {
                if constexpr (VL == 4) {
                    const float4 f = __ldg(reinterpret_cast<const float4 *>(vp + u * D + e * 32));
                    v[e] = f.x, v[e + 1] = f.y, v[e + 2] = f.z, v[e + 3] = f.w;
                } else {
                    const float2 f = __ldg(reinterpret_cast<const float2 *>(vp + u * D + e * 32));
                    v[e] = f.x, v[e + 1] = f.y;
                }
            }
        };
        float s[GT] = {}, v[VREG ? kBlockSize : 1][DL];
        if constexpr (VREG) {
#pragma unroll
            for (int u = 0; u < kBlockSize; ++u) {
                // rows behind the last token may hold NaN: 0 there
                if (u < valid) {
                    vrow(u, v[u]);
                } else {
#pragma unroll
                    for (int e = 0; e < DL; ++e) v[u][e] = 0.f;
                }
            }
        }
#pragma unroll 8
        for (int i = 0; i < D / 8; ++i) {
            const float4 k4 = __ldg(kp + i);
#pragma unroll
            for (int t = 0; t < GT; ++t) {
                const float4 q4 = *reinterpret_cast<const float4 *>(qs + t * D + half * (D / 2) + 4 * i);
                s[t] += k4.x * q4.x + k4.y * q4.y + k4.z * q4.z + k4.w * q4.w;
            }
        }
#pragma unroll
        for (int t = 0; t < GT; ++t) {
            s[t] += __shfl_xor_sync(0xffffffffu, s[t], 16);
            s[t] = tok < valid ? s[t] * a.scale_log2 : __int_as_float(0xff800000);
            float mx = s[t];
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            const float mn = fmaxf(m[t], mx), mu = mn == __int_as_float(0xff800000) ? 0.f : mn;
            const float al = fast_exp2(m[t] - mu);
            m[t] = mn;
            s[t] = fast_exp2(s[t] - mu);
            l[t] = l[t] * al + (half ? 0.f : s[t]);
#pragma unroll
            for (int e = 0; e < DL; ++e) o[t][e] *= al;
        }
        if constexpr (VREG) {
#pragma unroll
            for (int u = 0; u < kBlockSize; ++u)
#pragma unroll
                for (int t = 0; t < GT; ++t) {
                    const float p = __shfl_sync(0xffffffffu, s[t], u);
#pragma unroll
                    for (int e = 0; e < DL; ++e) o[t][e] += p * v[u][e];
                }
        } else {
#pragma unroll 4
            for (int u = 0; u < valid; ++u) {  // only the tokens that are there: what lies behind may be NaN
                vrow(u, v[0]);
#pragma unroll
                for (int t = 0; t < GT; ++t) {
                    const float p = __shfl_sync(0xffffffffu, s[t], u);
#pragma unroll
                    for (int e = 0; e < DL; ++e) o[t][e] += p * v[0][e];
                }
            }
        }
    }
#pragma unroll
    for (int t = 0; t < GT; ++t) {
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) l[t] += __shfl_xor_sync(0xffffffffu, l[t], d);
        if (lane == 0) {
            ml[warp * 2 * GT + t] = m[t];
            ml[(warp * 2 + 1) * GT + t] = l[t];
        }
#pragma unroll
        for (int e = 0; e < DL; ++e) os[(warp * GT + t) * C::OROW + (e / VL) * 32 * VL + lane * VL + e % VL] = o[t][e];
    }
    join_shares<float, D, GT, C::OROW, NW>(a, os, ml, ncol, row0, rank, ncta);
}

}  // namespace pa

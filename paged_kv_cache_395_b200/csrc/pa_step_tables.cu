// pa_step_tables: block tables, slot map, positions and lengths of one decode step, from
// the lengths of its sequences.
//
//   need_b  = ceil((len_b + new_b) / 16) - ceil(len_b / 16)
//   first_b = sum of the needs before b;   block k of b = F[c - 1 - first_b - k]
//   slot(t) = block(pos / 16) * 16 + pos % 16,   pos = len_b + t - start_b
//
// with F the stack of free blocks after the finished sequences' blocks were pushed and c
// its height.  Everything follows from three prefix sums over the sequences (tokens,
// blocks given back, blocks needed), so the kernel is bound by the latency of a chain of
// dependent loads (lengths -> last block's table entry -> stack entries -> stores), not by
// bytes: one step of 64 sequences moves under 5 KB.
//
// One thread-block cluster: every CTA computes the prefix sums over all sequences for
// itself (8 bytes of input per sequence), and the CTAs share the blocks given back and
// handed out.  Blocks are pushed before they are popped; the cluster's barrier, which also
// makes the pushes visible, stands between the two.  The slots of a step with few tokens are
// written by the same launch.  A step with prompts has so many that a cluster's few SMs
// would be the bound, so a second kernel writes them over the whole GPU, from the tables and
// lengths that the first one left (1024 sequences, 256 of them prompts, 526k slots: 102 us in one
// cluster of 8 CTAs, 24.5 us this way; 64 sequences of one token: 7.5 us).  The blocks given back in
// a step with few tokens are one CTA's too: an ended request of 4096 tokens costs 0.1 us, one of
// 131072 tokens 25 us (50 us with reference counts).
#include <cooperative_groups.h>

#include "pa_cluster.cuh"
#include "pa_common.cuh"
#include "pa_internal.h"

namespace cg = cooperative_groups;

namespace pa {

PA_ERROR_WORD_ACCESSOR(error_word_step_tables)

namespace {

constexpr int kClaim = 1 << 30;  // refs[x] = kClaim + e: entry e is the last one of this call that freed x

// Inclusive prefix sum of one value per thread over the CTA (ws: 32 slots); total: of all threads.
template <typename V>
__device__ __forceinline__ V block_scan(V x, V *ws, V *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const V y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) ws[warp] = x;
    __syncthreads();
    V s = lane < nw ? ws[lane] : 0;  // every warp scans the warps' sums
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const V y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    *total = __shfl_sync(0xffffffffu, s, 31);
    const V before = __shfl_sync(0xffffffffu, s, (warp + 31) & 31);
    __syncthreads();
    return warp ? x + before : x;
}

// Largest b in [lo, B) with start[b] <= t, where start is non-decreasing and start[lo] <= t: doubling
// steps from lo, then halving ones, so that a neighbour of lo is found at once.
__device__ __forceinline__ int row_of(const int *start, int lo, int B, int t) {
    int step = 1;
    while (lo + step < B && start[lo + step] <= t) {
        lo += step;
        step <<= 1;
    }
    for (; step > 0; step >>= 1)
        if (lo + step < B && start[lo + step] <= t) lo += step;
    return lo;
}

__device__ __forceinline__ int blocks_of(int tokens) { return (int)(((unsigned)tokens + kBlockSize - 1) / kBlockSize); }

// Shared memory: per sequence, the exclusive prefix sums (B + 1 entries), the length, the new
// tokens, the table entry of the last, partly filled block (-1: none) and whether it is served.
struct Smem {
    int *tok, *rel, *need, *len, *add, *last;
    uint8_t *ok;
    __device__ Smem(unsigned char *p, int B) {
        tok = reinterpret_cast<int *>(p);
        rel = tok + B + 1;
        need = rel + B + 1;
        len = need + B + 1;
        add = len + B;
        last = add + B;
        ok = reinterpret_cast<uint8_t *>(last + B);
    }
    static size_t bytes(int B) { return (size_t)(3 * (B + 1) + 3 * B) * 4 + B + 16; }
};

// WRITE_SLOTS: this launch also writes the slots and positions; otherwise it only leaves the slot
// of each sequence's first token, -1 if it is not served, for step_slots_kernel.
template <bool WRITE_SLOTS>
__global__ void __launch_bounds__(1024) step_tables_kernel(const StepArgs a) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ long long ws64[32];
    __shared__ int ws32[32];
    __shared__ int2 s_push;  // blocks this CTA pushes; whether it met one that several entries freed
    const Smem s(smem_raw, a.B);
    const int tid = threadIdx.x, nt = blockDim.x, B = a.B, M = a.M, N = a.N, T = a.T;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), ncta = (int)cl.num_blocks();
    const int top = M * kBlockSize;  // host: M <= 2^26
    auto barrier = [&]() {  // of the cluster; its writes are visible after it
        if (ncta > 1)
            cl.sync();
        else
            __syncthreads();
    };

    pdl_wait();
    pdl_release_dependents();

    // ---- lengths, and the prefix sums of new tokens and of blocks given back ----
    int count = __ldcg(a.count);
    const int per = (B + nt - 1) / nt, b0 = min(B, tid * per), b1 = min(B, b0 + per);
    long long tok = 0, tok_all;
    int rel = 0, rel_all;
    for (int b = b0; b < b1; ++b) {
        const int L = __ldcg(a.lens + b), n = __ldcg(a.news + b);
        const bool good = L >= 0 && n >= PA_SEQ_FINISHED && (long long)L + max(n, 0) <= top;
        // the last, partly filled block: asked for now, looked at after the sums
        s.last[b] = good && n > 0 && L % kBlockSize ? __ldcg(a.tables + (size_t)b * M + L / kBlockSize) : -1;
        s.len[b] = L;
        s.add[b] = n;
        if (!good && rank == 0) raise_flag(PA_EFLAG_BAD_LENGTH);
        tok += max(n, 0);
        rel += good && n == PA_SEQ_FINISHED ? blocks_of(L) : 0;
        // 0: nothing to do, 1: to be served, 2: finished
        s.ok[b] = !good ? 0 : n == PA_SEQ_FINISHED ? 2 : n > 0 ? 1 : 0;
    }
    if (count < 0 || count > N) {
        if (tid == 0 && rank == 0) raise_flag(PA_EFLAG_FREE_LIST);
        count = count < 0 ? 0 : N;
    }
    tok = block_scan(tok, ws64, &tok_all) - tok;
    rel = block_scan(rel, ws32, &rel_all) - rel;
    for (int b = b0; b < b1; ++b) {
        const int n = s.add[b];
        s.tok[b] = (int)min(tok, (long long)T + 1);
        s.rel[b] = rel;
        tok += max(n, 0);
        rel += s.ok[b] == 2 ? blocks_of(s.len[b]) : 0;
        if (n > 0 && tok > T) {  // the sequence's tokens do not fit into the slot buffer
            s.ok[b] = 0;
            if (rank == 0) raise_flag(PA_EFLAG_BAD_LENGTH);
        }
    }
    if (tid == 0) {
        s.tok[B] = (int)min(tok_all, (long long)T + 1);
        s.rel[B] = rel_all;
    }
    __syncthreads();

    // ---- push the finished sequences' blocks: entry e of the concatenated rows ----
    if (rel_all > 0) {  // the same in every CTA
        const int chunk = (rel_all + ncta - 1) / ncta, e0 = min(rel_all, rank * chunk), e1 = min(rel_all, e0 + chunk);
        auto entry = [&](int e) {
            const int b = row_of(s.rel, 0, B, e);
            return a.tables[(size_t)b * M + (e - s.rel[b])];
        };
        auto inside = [&](int x) { return x >= 0 && x < N; };
        // a thread's first entries stay in registers (usually they are all)
        constexpr int E = 4;
        const int f0 = e0 + tid;
        int x0[E], old0[E];
        uint32_t k0 = 0;  // which of them are pushed
#pragma unroll
        for (int i = 0; i < E; ++i) {
            x0[i] = f0 + i * nt < e1 ? entry(f0 + i * nt) : -1;
            old0[i] = 0;
        }
        bool claim = false;
        if (a.refs) {
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (inside(x0[i])) old0[i] = atomicSub(a.refs + x0[i], 1);
            for (int e = f0 + E * nt; e < e1; e += nt) {
                const int x = entry(e);
                if (inside(x)) claim |= atomicSub(a.refs + x, 1) > 1;
            }
            barrier();
        }
        // A block whose count reached zero is pushed.  If several entries of this call brought it
        // there (some saw a count above one), the last of them pushes it, which takes another
        // round, as does a count below zero; without such blocks each entry knows by itself.
        int kept = 0, all_kept;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if (f0 + i * nt >= e1) continue;
            if (!inside(x0[i])) {
                raise_flag(PA_EFLAG_BAD_BLOCK);
                continue;
            }
            const int v = a.refs ? __ldcg(a.refs + x0[i]) : 0;
            if (v < 0) raise_flag(PA_EFLAG_FREE_LIST);
            claim |= v < 0 || (v == 0 && old0[i] > 1);
            kept += v == 0;
            k0 |= (uint32_t)(v == 0) << i;
        }
        for (int e = f0 + E * nt; e < e1; e += nt) {
            const int x = entry(e);
            if (!inside(x)) {
                raise_flag(PA_EFLAG_BAD_BLOCK);
                continue;
            }
            const int v = a.refs ? __ldcg(a.refs + x) : 0;
            if (v < 0) raise_flag(PA_EFLAG_FREE_LIST);
            claim |= v < 0;
            kept += v == 0;
        }
        block_scan(kept, ws32, &all_kept);
        claim = __syncthreads_or(claim);
        // lane r of every warp reads CTA r's word
        const int lane = tid & 31;
        auto exchange = [&]() -> int2 {
            if (tid == 0) s_push = make_int2(all_kept, claim);
            barrier();
            if (lane >= ncta) return make_int2(0, 0);
            return ncta > 1 ? *cl.map_shared_rank(&s_push, lane) : s_push;
        };
        int2 theirs = exchange();
        claim = __any_sync(0xffffffffu, theirs.y);
        if (claim) {  // the same in every CTA
            for (int e = f0; e < e1; e += nt) {
                const int x = entry(e);
                if (!inside(x)) continue;
                const int v = __ldcg(a.refs + x);
                if (v == 0 || v >= kClaim) atomicMax(a.refs + x, kClaim + e);
            }
            barrier();
            kept = 0;
            k0 = 0;
            for (int e = f0, i = 0; e < e1; e += nt, ++i) {
                const int x = entry(e);
                const bool k = inside(x) && __ldcg(a.refs + x) == kClaim + e;
                kept += k;
                if (i < E) k0 |= (uint32_t)k << i;
            }
            block_scan(kept, ws32, &all_kept);
            barrier();  // the words of the first exchange are read
            theirs = exchange();
        }
        int at = count + __reduce_add_sync(0xffffffffu, lane < rank ? theirs.x : 0);
        int pushed = __reduce_add_sync(0xffffffffu, theirs.x);
        auto push = [&](int x, bool k) {  // the next nt entries, in order
            int all;
            const int nth = at + block_scan((int)k, ws32, &all) - 1;
            if (k && nth < N) a.free_blocks[nth] = x;
            if (claim && inside(x) && (k || __ldcg(a.refs + x) < 0)) a.refs[x] = 0;
            at += all;
        };
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (e0 + i * nt < e1) push(x0[i], k0 >> i & 1);
        for (int e = e0 + E * nt; e < e1; e += nt) {
            const int f = e + tid, x = f < e1 ? entry(f) : -1;
            push(x, inside(x) && (!a.refs || __ldcg(a.refs + x) == (claim ? kClaim + f : 0)));
        }
        if ((long long)count + pushed > N) {
            if (tid == 0 && rank == 0) raise_flag(PA_EFLAG_FREE_LIST);
            pushed = N - count;
        }
        count += pushed;
        barrier();  // every push is visible before the first pop
    }

    // ---- needs, in order, while the list lasts ----
    int need = 0, need_all;
    for (int b = b0; b < b1; ++b) {
        if (s.ok[b] != 1) continue;
        const int L = s.len[b];
        if (L % kBlockSize) {
            const int x = s.last[b];
            const bool in = x >= 0 && x < N;
            if (!in || (a.refs && __ldcg(a.refs + x) > 1)) {
                s.ok[b] = 0;
                if (rank == 0) raise_flag(in ? PA_EFLAG_BAD_LENGTH : PA_EFLAG_BAD_BLOCK);
                continue;
            }
        }
        need += blocks_of(L + s.add[b]) - blocks_of(L);
    }
    need = block_scan(need, ws32, &need_all) - need;
    int served = 0;  // the most blocks handed out up to a served sequence of this thread
    for (int b = b0; b < b1; ++b) {
        s.need[b] = need;
        if (s.ok[b] != 1) continue;
        const int k = blocks_of(s.len[b] + s.add[b]) - blocks_of(s.len[b]);
        need += k;
        if (k > 0 && need > count) {
            s.ok[b] = 0;
            if (rank == 0) raise_flag(PA_EFLAG_OUT_OF_BLOCKS);
        } else if (k > 0) {
            served = need;
        }
    }
    // the needs grow along the sequences, so those handed out are a prefix of all needs
    served = __reduce_max_sync(0xffffffffu, served);
    if ((tid & 31) == 0) ws32[tid >> 5] = served;
    __syncthreads();
    served = __reduce_max_sync(0xffffffffu, (tid & 31) < nt / 32 ? ws32[tid & 31] : 0);

    // every CTA has read the lengths, the count and the entries that others write below
    if (ncta > 1) cl.sync();

    // ---- results ----
    const int gid = rank * nt + tid, gn = ncta * nt;
    {  // each thread a run of the popped blocks
        const int q = (served + gn - 1) / gn, i0 = min(served, gid * q), i1 = min(served, i0 + q);
        int b = i0 < i1 ? row_of(s.need, 0, B, i0) : 0;
        for (int i = i0; i < i1; i += 4) {
            int x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = i + e < i1 ? __ldcg(a.free_blocks + count - 1 - i - e) : 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (i + e >= i1) break;
                b = row_of(s.need, b, B, i + e);
                a.tables[(size_t)b * M + blocks_of(s.len[b]) + (i + e - s.need[b])] = x[e];
                if (x[e] < 0 || x[e] >= N)
                    raise_flag(PA_EFLAG_BAD_BLOCK);
                else if (a.refs)
                    a.refs[x[e]] = 1;
            }
        }
    }
    // slot of token i of served sequence b
    auto slot_of = [&](int b, int i) {
        const int p = s.len[b] + i, k = p / kBlockSize - blocks_of(s.len[b]);  // k < 0: in the partly filled block
        const int x = k < 0 ? s.last[b] : __ldcg(a.free_blocks + count - 1 - s.need[b] - k);
        return x >= 0 && x < N ? (long long)x * kBlockSize + p % kBlockSize : -1ll;
    };
    for (int b = gid; b < B; b += gn) {
        a.lens_out[b] = s.ok[b] == 2 ? 0 : s.ok[b] == 1 ? s.len[b] + s.add[b] : s.len[b];
        if (!WRITE_SLOTS && s.add[b] > 0 && s.tok[b] < T) a.slots[s.tok[b]] = s.ok[b] == 1 ? slot_of(b, 0) : -1;
    }
    if (a.starts)
        for (int b = gid; b <= B; b += gn) a.starts[b] = min(s.tok[b], T);
    if (gid == 0) a.count_out[0] = count - served;
    if (WRITE_SLOTS) {
        const int live = s.tok[B];
        int row = 0;
        for (int t = gid; t < T; t += gn) {
            long long slot = -1;
            int p = -1;
            if (t < live) {
                row = row_of(s.tok, row, B, t);
                if (s.ok[row] == 1) {
                    p = s.len[row] + t - s.tok[row];
                    slot = slot_of(row, t - s.tok[row]);
                }
            }
            a.slots[t] = slot;
            if (a.pos) a.pos[t] = p;
        }
    }
}

// The slots and positions of a step with many tokens.  Every CTA redoes the prefix sum of the new
// tokens; a sequence's first slot says whether it is served, and its position in its block with the
// length gives the others.  That first slot is written again with the same value, so its readers
// in other CTAs need no order.
__global__ void __launch_bounds__(512) step_slots_kernel(const StepArgs a) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ long long ws64[32];
    int *start = reinterpret_cast<int *>(smem_raw), *base = start + a.B;  // base: position of the first new token, -1: not served
    const int tid = threadIdx.x, nt = blockDim.x, B = a.B, M = a.M, N = a.N, T = a.T;
    pdl_wait();
    pdl_release_dependents();
    const int per = (B + nt - 1) / nt, b0 = min(B, tid * per), b1 = min(B, b0 + per);
    long long tok = 0, all;
    for (int b = b0; b < b1; ++b) tok += max(__ldcg(a.news + b), 0);
    tok = block_scan(tok, ws64, &all) - tok;
    for (int b = b0; b < b1; ++b) {
        const int n = __ldcg(a.news + b);
        start[b] = (int)min(tok, (long long)T + 1);
        base[b] = n > 0 && tok < T && __ldcg(a.slots + tok) >= 0 ? __ldcg(a.lens_out + b) - n : -1;
        tok += max(n, 0);
    }
    __syncthreads();
    const int live = (int)min(all, (long long)T);
    // four tokens per thread and turn, their table entries asked for together
    constexpr int U = 4;
    int row = 0;
    for (int64_t t0 = (int64_t)blockIdx.x * (nt * U) + tid; t0 < T; t0 += (int64_t)gridDim.x * (nt * U)) {
        int p[U], x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t t = t0 + u * nt;
            p[u] = x[u] = -1;
            if (t < live) {
                row = row_of(start, row, B, (int)t);
                if (base[row] >= 0) {
                    p[u] = base[row] + (int)t - start[row];
                    x[u] = __ldcg(a.tables + (size_t)row * M + p[u] / kBlockSize);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t t = t0 + u * nt;
            if (t >= T) break;
            a.slots[t] = x[u] >= 0 && x[u] < N ? (long long)x[u] * kBlockSize + p[u] % kBlockSize : -1;
            if (a.pos) a.pos[t] = p[u];
        }
    }
}

}  // namespace

int launch_step_tables(const StepArgs &a, cudaStream_t st) {
    // A step with few tokens is one launch of one CTA: a cluster's barriers and a second launch
    // would only add latency.
    const bool few = a.T <= 4096;
    const int threads = a.B <= 256 && few ? 256 : 1024;
    const size_t smem = Smem::bytes(a.B);
    auto kern = few ? step_tables_kernel<true> : step_tables_kernel<false>;
    // Always: the 48 KB that a launch has without it count the kernel's static shared memory too.
    // Both kernels' before the first launch, which moves the sequences on: a call that cannot
    // write its slots must not have done that.
    if (!set_smem_attr_once(reinterpret_cast<const void *>(kern), (int)Smem::bytes(PA_STEP_MAX_SEQS))) return PA_ERR_CUDA;
    if (!few && !set_smem_attr_once(reinterpret_cast<const void *>(step_slots_kernel), PA_STEP_MAX_SEQS * 8)) return PA_ERR_CUDA;
    // 16 CTAs, beyond the portable 8 (the steps with prompts hand out thousands of blocks), where a
    // cluster of the largest step's shared memory finds room; half as many, and so on, where not, as
    // on a slice of a GPU.
    int ncta = few ? 1 : 16;
    static ClusterRoom room;
    while (ncta > 1 && room.of(kern, ncta, 1024, Smem::bytes(PA_STEP_MAX_SEQS)) < 1) ncta /= 2;
    if (launch_cluster(kern, ncta, ncta, threads, smem, st, a) != cudaSuccess) return PA_ERR_CUDA;
    if (few) return PA_OK;
    const int64_t ctas = ((int64_t)a.T + 2047) / 2048;
    return launch_pdl(step_slots_kernel, dim3((unsigned)(ctas < 2 * 148 ? ctas : 2 * 148)), dim3(512), (size_t)a.B * 8, st, a) ==
                   cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

}  // namespace pa

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
// One thread-block cluster, so that a step is one launch: every CTA computes the prefix
// sums over all sequences for itself (8 bytes of input per sequence), and the CTAs share
// the blocks given back, the blocks handed out and the token slots.  Blocks are pushed
// before they are popped; the cluster's barrier, which also makes the pushes visible,
// stands between the two.
#include <cooperative_groups.h>

#include <atomic>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace cg = cooperative_groups;

namespace pa {

PA_ERROR_WORD_ACCESSOR(error_word_step_tables)

namespace {

constexpr int kClaim = 1 << 30;  // refs[x] = kClaim + e: entry e is the last one of this call that freed x

// Inclusive prefix sum of one value per thread over the CTA (ws: one slot per warp).
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
    V before = 0, all = 0;
    for (int w = 0; w < nw; ++w) {
        const V s = ws[w];
        if (w < warp) before += s;
        all += s;
    }
    __syncthreads();
    *total = all;
    return x + before;
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

// Shared memory: per sequence, the exclusive prefix sums (B + 1 entries), the length, the
// table entry of the last, partly filled block (-1: none) and whether it is served.
struct Smem {
    int *tok, *rel, *need, *len, *last;
    uint8_t *ok;
    __device__ Smem(unsigned char *p, int B) {
        tok = reinterpret_cast<int *>(p);
        rel = tok + B + 1;
        need = rel + B + 1;
        len = need + B + 1;
        last = len + B;
        ok = reinterpret_cast<uint8_t *>(last + B);
    }
    static size_t bytes(int B) { return (size_t)(3 * (B + 1) + 2 * B) * 4 + B + 16; }
};

__global__ void __launch_bounds__(1024) step_tables_kernel(const StepArgs a) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ long long ws64[32];
    __shared__ int ws32[32];
    __shared__ int s_kept;  // blocks this CTA pushes
    const Smem s(smem_raw, a.B);
    const int tid = threadIdx.x, nt = blockDim.x, B = a.B, M = a.M, N = a.N, T = a.T;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), ncta = (int)cl.num_blocks();
    const int top = M * kBlockSize;  // host: M <= 2^26

    pdl_wait();
    pdl_release_dependents();

    int count = a.count[0];
    if (count < 0 || count > N) {
        if (tid == 0 && rank == 0) raise_flag(PA_EFLAG_FREE_LIST);
        count = count < 0 ? 0 : N;
    }

    // ---- lengths, and the prefix sums of new tokens and of blocks given back ----
    const int per = (B + nt - 1) / nt, b0 = min(B, tid * per), b1 = min(B, b0 + per);
    long long tok = 0, tok_all;
    int rel = 0, rel_all;
    for (int b = b0; b < b1; ++b) {
        const int L = a.lens[b], n = a.news[b];
        s.len[b] = L;
        const bool good = L >= 0 && n >= PA_SEQ_FINISHED && (long long)L + max(n, 0) <= top;
        if (!good && rank == 0) raise_flag(PA_EFLAG_BAD_LENGTH);
        tok += max(n, 0);
        rel += good && n == PA_SEQ_FINISHED ? blocks_of(L) : 0;
        // 0: nothing to do, 1: to be served, 2: finished
        s.ok[b] = !good ? 0 : n == PA_SEQ_FINISHED ? 2 : n > 0 ? 1 : 0;
    }
    tok = block_scan(tok, ws64, &tok_all) - tok;
    rel = block_scan(rel, ws32, &rel_all) - rel;
    for (int b = b0; b < b1; ++b) {
        const int L = s.len[b], n = a.news[b];
        s.tok[b] = (int)min(tok, (long long)T + 1);
        s.rel[b] = rel;
        tok += max(n, 0);
        rel += s.ok[b] == 2 ? blocks_of(L) : 0;
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
        if (a.refs) {
            for (int e = e0 + tid; e < e1; e += nt) {
                const int x = entry(e);
                if (inside(x)) atomicSub(a.refs + x, 1);
            }
            cl.sync();
            // the last entry of a block whose count reached zero claims it
            for (int e = e0 + tid; e < e1; e += nt) {
                const int x = entry(e);
                if (!inside(x)) continue;
                const int v = __ldcg(a.refs + x);
                if (v == 0 || v >= kClaim) atomicMax(a.refs + x, kClaim + e);
            }
            cl.sync();
        }
        auto keep = [&](int e, int x) { return inside(x) && (!a.refs || __ldcg(a.refs + x) == kClaim + e); };
        int mine = 0;
        for (int e = e0 + tid; e < e1; e += nt) {
            const int x = entry(e);
            mine += keep(e, x);
            if (!inside(x)) raise_flag(PA_EFLAG_BAD_BLOCK);
            if (a.refs && inside(x) && __ldcg(a.refs + x) < 0) raise_flag(PA_EFLAG_FREE_LIST);
        }
        int kept;
        block_scan(mine, ws32, &kept);
        if (tid == 0) s_kept = kept;
        cl.sync();
        int at = count, pushed = 0;
        for (int r = 0; r < ncta; ++r) {
            const int k = *cl.map_shared_rank(&s_kept, r);
            if (r < rank) at += k;
            pushed += k;
        }
        for (int e = e0; e < e1; e += nt) {  // in order, nt entries at a time
            const int f = e + tid;
            const int x = f < e1 ? entry(f) : -1;
            const bool k = f < e1 && keep(f, x);
            int all;
            const int nth = at + block_scan((int)k, ws32, &all) - 1;
            if (k) {
                if (nth < N) a.free_blocks[nth] = x;
                if (a.refs) a.refs[x] = 0;
            } else if (f < e1 && a.refs && inside(x) && __ldcg(a.refs + x) < 0) {
                a.refs[x] = 0;
            }
            at += all;
        }
        if ((long long)count + pushed > N) {
            if (tid == 0 && rank == 0) raise_flag(PA_EFLAG_FREE_LIST);
            pushed = N - count;
        }
        count += pushed;
        cl.sync();  // every push is visible before the first pop
    }

    // ---- needs, in order, while the list lasts ----
    int need = 0, need_all;
    for (int b = b0; b < b1; ++b) {
        s.last[b] = -1;
        if (s.ok[b] != 1) continue;
        const int L = s.len[b];
        if (L % kBlockSize) {
            const int x = a.tables[(size_t)b * M + L / kBlockSize];
            s.last[b] = x;
            const bool in = x >= 0 && x < N;
            if (!in || (a.refs && __ldcg(a.refs + x) > 1)) {
                s.ok[b] = 0;
                if (rank == 0) raise_flag(in ? PA_EFLAG_BAD_LENGTH : PA_EFLAG_BAD_BLOCK);
                continue;
            }
        }
        need += blocks_of(L + a.news[b]) - blocks_of(L);
    }
    need = block_scan(need, ws32, &need_all) - need;
    int served = 0;  // the most blocks handed out up to a served sequence of this thread
    for (int b = b0; b < b1; ++b) {
        s.need[b] = need;
        if (s.ok[b] != 1) continue;
        const int k = blocks_of(s.len[b] + a.news[b]) - blocks_of(s.len[b]);
        need += k;
        if (k > 0 && need > count) {
            s.ok[b] = 0;
            if (rank == 0) raise_flag(PA_EFLAG_OUT_OF_BLOCKS);
        } else if (k > 0) {
            served = need;
        }
    }
    if (tid == 0) s.need[B] = need_all;
    // the needs grow along the sequences, so those handed out are a prefix of all needs
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) served = max(served, __shfl_xor_sync(0xffffffffu, served, o));
    if ((tid & 31) == 0) ws32[tid >> 5] = served;
    __syncthreads();
    for (int w = 0; w < nt / 32; ++w) served = max(served, ws32[w]);

    // every CTA has read the lengths, the count and the entries that others write below
    if (ncta > 1) cl.sync();

    // ---- results ----
    if (rank == 0) {
        for (int b = tid; b < B; b += nt)
            a.lens_out[b] = s.ok[b] == 2 ? 0 : s.ok[b] == 1 ? s.len[b] + a.news[b] : s.len[b];
        if (a.starts)
            for (int b = tid; b <= B; b += nt) a.starts[b] = min(s.tok[b], T);
        if (tid == 0) a.count_out[0] = count - served;
    }
    const int gid = rank * nt + tid, gn = ncta * nt;
    for (int i = gid; i < served; i += gn) {
        const int b = row_of(s.need, 0, B, i);
        const int x = __ldcg(a.free_blocks + count - 1 - i);
        a.tables[(size_t)b * M + blocks_of(s.len[b]) + (i - s.need[b])] = x;
        if (a.refs && x >= 0 && x < N) a.refs[x] = 1;
        if (x < 0 || x >= N) raise_flag(PA_EFLAG_BAD_BLOCK);
    }
    const int live = s.tok[B];
    int row = 0;
    for (int t = gid; t < T; t += gn) {
        long long slot = -1;
        int p = -1;
        if (t < live) {
            row = row_of(s.tok, row, B, t);
            if (s.ok[row] == 1) {
                const int L = s.len[row];
                p = L + t - s.tok[row];
                const int k = p / kBlockSize - blocks_of(L);  // < 0: in the block that was partly filled
                const int x = k < 0 ? s.last[row] : __ldcg(a.free_blocks + count - 1 - s.need[row] - k);
                slot = x >= 0 && x < N ? (long long)x * kBlockSize + p % kBlockSize : -1;
            }
        }
        a.slots[t] = slot;
        if (a.pos) a.pos[t] = p;
    }
}

}  // namespace

int launch_step_tables(const StepArgs &a, cudaStream_t st) {
    // A step with few tokens runs on one CTA: a cluster's barriers would only add latency.
    const int ncta = a.T > 4096 ? 8 : 1;
    const int threads = a.B <= 256 && a.T <= 1024 ? 256 : 1024;
    const size_t smem = Smem::bytes(a.B);
    if (smem > 48 * 1024) {
        static std::atomic<unsigned long long> done{0};  // devices whose limit is raised
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return PA_ERR_CUDA;
        const unsigned long long bit = 1ull << (dev & 63);
        if (dev > 63 || !(done.load() & bit)) {
            if (cudaFuncSetAttribute(reinterpret_cast<const void *>(step_tables_kernel),
                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)Smem::bytes(PA_STEP_MAX_SEQS)) != cudaSuccess)
                return PA_ERR_CUDA;
            done.fetch_or(bit);
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ncta);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ncta;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, step_tables_kernel, a) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa

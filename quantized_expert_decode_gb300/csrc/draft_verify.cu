// draft_verify.cu — drafted tokens accepted or rejected from given random numbers, and the token drawn behind the last
// accepted one. A cluster of CTAs per sequence, one launch.
//
// Mathematics. With a draft, the residual after rejections at a node is a multiple of r(x) = max(p(x) - a q(x), 0): with
// a_1 = 0, m_1 = 1 and m_j = sum r_j, r_{j+1} = max(r_j - m_j q, 0) = max(p - (a_j + m_j) q, 0). So a node's state is two
// numbers (a, m), and a child x with random number u is accepted iff (a + u m) q(x) < p(x). Without a draft r is p
// without the rejected tokens.
//
// Sums over the vocabulary are kept as unevaluated pairs of floats (48 bits; 64-bit additions would take 30 times
// an fp32 addition's time) and joined in 64 bits, so that a number falls on the wrong side of a border between two
// tokens with a chance of some 2^-45 times the tokens, whatever the order of the sums.
//
// What bounds it: for few sequences the latency of its steps: nodes, their entries, one or two rows of p and q
// spread over the cluster's CTAs, and the exchange of the CTAs' sums through distributed shared memory. All CTAs of a
// cluster walk the nodes alike; only sums are shared. Nodes that are accepted at their first test need no row at all:
// the entries that the tests need are gathered at the start, all at once.
#include <cooperative_groups.h>

#include "act.cuh"
#include "draft.h"
#include "host.h"
#include "pdl.cuh"

namespace cg = cooperative_groups;

namespace colimoe {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kMaxNodes = 1024;
constexpr int kMaxVocab = 1 << 20;
constexpr int kChunk = 512;  // tokens of a warp's sum
constexpr int kPer = 4;      // tokens of a lane at once
constexpr int kMaxChunks = (kMaxVocab / kCluster + kChunk - 1) / kChunk + 1;

struct Two {
    float hi, lo;
};
// s + x, the rounding error kept
__device__ __forceinline__ void add(Two &s, float x, float rest) {
    const float t = __fadd_rn(s.hi, x), z = __fsub_rn(t, s.hi);
    const float e = __fadd_rn(__fsub_rn(s.hi, __fsub_rn(t, z)), __fsub_rn(x, z));
    s.hi = t;
    s.lo = __fadd_rn(s.lo, __fadd_rn(e, rest));
}
__device__ __forceinline__ double warp_total(Two s) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float hi = __shfl_xor_sync(0xffffffffu, s.hi, o), lo = __shfl_xor_sync(0xffffffffu, s.lo, o);
        add(s, hi, lo);
    }
    return (double)s.hi + (double)s.lo;
}

// max(p - a q, 0) with a = ah + al, as a pair
__device__ __forceinline__ Two residual(float p, float q, float ah, float al) {
    const float h = __fmul_rn(ah, q), e = fmaf(ah, q, -h);  // ah q = h + e
    const float d = __fsub_rn(p, h), z = __fsub_rn(d, p);
    const float f = __fsub_rn(__fsub_rn(p, __fsub_rn(d, z)), __fadd_rn(h, z));  // p - h = d + f
    const float low = __fsub_rn(f, fmaf(al, q, e));
    return __fadd_rn(d, low) > 0.f ? Two{d, low} : Two{0.f, 0.f};
}

struct Shared {
    float p[kMaxNodes], q[kMaxNodes];  // the parent's entries at the node's token
    int32_t parent[kMaxNodes], token[kMaxNodes];
    double chunk[kMaxChunks];
    double warp_sum[kWarps];
    double part[2][kCluster];  // the CTAs' sums, in turn
    float best[2][kCluster];
    int32_t best_at[2][kCluster];
    float warp_best[kWarps];
    int32_t warp_at[kWarps];
    int32_t lost[kMaxNodes];  // rejected tokens at this node (without a draft)
};

template <typename T>
__global__ void __launch_bounds__(kThreads) draft_verify_kernel(const VerifyParams P, int slice, int vec) {
    __shared__ Shared S;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), b = blockIdx.x / kCluster;
    const int tid = threadIdx.x, w = tid / 32, lane = tid % 32;
    wait_for_previous();
    let_next_start();
    int row, n, why;
    draft_rows(P.first[b], P.first[b + 1], P.rows, P.nodes, row, n, why);
    if (why && rank == 0 && tid == 0 && P.err) atomicOr(P.err, COLI_LAYER_BAD_SEQUENCE);
    int32_t *path = P.path + (int64_t)b * P.nodes;
    if (rank == 0)
        for (int i = tid; i < P.nodes; i += kThreads) path[i] = -1;
    if (n == 0) {  // (the whole cluster)
        if (rank == 0 && tid == 0) P.count[b] = 0, P.next[b] = -1;
        return;
    }
    const T *target = (const T *)P.target + (int64_t)row * P.target_stride;
    const T *draft = P.draft ? (const T *)P.draft + (int64_t)row * P.draft_stride : nullptr;
    for (int i = tid; i < n; i += kThreads) {
        int up = P.parent ? P.parent[row + i] : i - 1, x = P.tokens[row + i], flag = 0;
        if (i == 0) up = -1;  // the root
        if (up < -1 || up >= i) up = -1, flag = COLI_DRAFT_BAD_NODE;
        if (i > 0 && (x < 0 || x >= P.vocab)) up = -1, flag = COLI_DRAFT_BAD_NODE;
        S.parent[i] = up;
        S.token[i] = x;
        if (up >= 0 && P.mode == COLI_VERIFY_SAMPLE) {
            S.p[i] = to_f32(target[up * P.target_stride + x]);
            S.q[i] = draft ? to_f32(draft[up * P.draft_stride + x]) : 1.f;
        }
        if (flag && rank == 0 && P.err) atomicOr(P.err, flag);
    }
    cl.sync();  // the CTAs' shared memory may be written to from now on
    if (rank == 0 && tid == 0) path[0] = 0;

    // the cluster's share of a row: tokens [v0, v1) of this CTA, in chunks
    const int v0 = min(rank * slice, P.vocab), v1 = min(v0 + slice, P.vocab);
    const int chunks = (v1 - v0 + kChunk - 1) / kChunk;
    int turn = 0;

    int cur = 0, lost = 0;
    double a = 0.0, m = 1.0;

    // entries [x, x + kPer) of a row, 0 behind `end`
    auto entries = [&](const T *r, int x, int end, float (&e)[kPer]) {
        if (vec && x + kPer <= end) {
            Run<T, kPer> t;
            t.load(r + x);
#pragma unroll
            for (int j = 0; j < kPer; j++) e[j] = to_f32(t.e[j]);
        } else {
#pragma unroll
            for (int j = 0; j < kPer; j++) e[j] = x + j < end ? to_f32(r[x + j]) : 0.f;
        }
    };
    // r at tokens x .. x + kPer - 1 of the current node
    auto left = [&](int x, int end, float ah, float al, bool whole, Two (&r)[kPer]) {
        float p[kPer], q[kPer];
        entries(target + cur * P.target_stride, x, end, p);
        if (draft && !whole && ah > 0.f) {
            entries(draft + cur * P.draft_stride, x, end, q);
#pragma unroll
            for (int j = 0; j < kPer; j++) r[j] = residual(p[j], q[j], ah, al);
        } else {
            if (!whole)
                for (int k = 0; k < lost; k++)
#pragma unroll
                    for (int j = 0; j < kPer; j++)
                        if (S.lost[k] == x + j) p[j] = 0.f;
#pragma unroll
            for (int j = 0; j < kPer; j++) r[j] = Two{p[j], 0.f};
        }
    };
    // sums of r over this CTA's chunks, and over the row: every thread of the cluster gets the same bits
    double before = 0.0;  // of the CTAs before this one
    auto total = [&](bool whole) {
        const float ah = (float)a, al = (float)(a - (double)ah);
        for (int c = w; c < chunks; c += kWarps) {
            Two s{0.f, 0.f};
#pragma unroll
            for (int k = 0; k < kChunk / (32 * kPer); k++) {
                Two r[kPer];
                left(v0 + c * kChunk + (k * 32 + lane) * kPer, v1, ah, al, whole, r);
#pragma unroll
                for (int j = 0; j < kPer; j++) add(s, r[j].hi, r[j].lo);
            }
            const double t = warp_total(s);
            if (lane == 0) S.chunk[c] = t;
        }
        __syncthreads();
        if (w == 0) {
            double t = 0.0;
            for (int c = lane; c < chunks; c += 32) t += S.chunk[c];
#pragma unroll
            for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            if (lane < kCluster) *cl.map_shared_rank(&S.part[turn][rank], lane) = t;
        }
        cl.sync();
        double all = 0.0;
        before = 0.0;
        for (int k = 0; k < kCluster; k++) {
            if (k == rank) before = all;
            all += S.part[turn][k];
        }
        turn ^= 1;
        return all;
    };
    // the index of the current row's largest entry
    auto largest = [&]() {
        float best = -INFINITY;
        int at = INT32_MAX;
        for (int x = v0 + tid * kPer; x < v1; x += kThreads * kPer) {
            float e[kPer];
            entries(target + cur * P.target_stride, x, v1, e);
#pragma unroll
            for (int j = 0; j < kPer; j++)
                if (x + j < v1 && (e[j] > best || (at == INT32_MAX && e[j] == best))) best = e[j], at = x + j;
        }
        auto better = [&](float o, int i) {
            if (i != INT32_MAX && (at == INT32_MAX || o > best || (o == best && i < at))) best = o, at = i;
        };
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float ob = __shfl_xor_sync(0xffffffffu, best, o);
            better(ob, __shfl_xor_sync(0xffffffffu, at, o));
        }
        if (lane == 0) S.warp_best[w] = best, S.warp_at[w] = at;
        __syncthreads();
        if (w == 0) {
            best = lane < kWarps ? S.warp_best[lane] : -INFINITY;
            at = lane < kWarps ? S.warp_at[lane] : INT32_MAX;
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                const float ob = __shfl_xor_sync(0xffffffffu, best, o);
                better(ob, __shfl_xor_sync(0xffffffffu, at, o));
            }
            if (lane < kCluster) {
                *cl.map_shared_rank(&S.best[turn][rank], lane) = best;
                *cl.map_shared_rank(&S.best_at[turn][rank], lane) = at;
            }
        }
        cl.sync();
        best = -INFINITY;
        at = INT32_MAX;
        for (int k = 0; k < kCluster; k++) better(S.best[turn][k], S.best_at[turn][k]);
        turn ^= 1;
        return at == INT32_MAX ? 0 : at;  // nothing but NaN
    };

    int accepted = 1, top = -1;
    if (P.mode == COLI_VERIFY_GREEDY) top = largest();
    // Nodes come behind their parents: one look at each in turn walks down the tree.
    for (int i0 = 0; i0 < n; i0 += 32) {
        int done = i0 == 0 ? 0 : -1;  // nodes of this round up to here are dealt with
        while (true) {
            const int i = i0 + lane;
            const unsigned is = __ballot_sync(0xffffffffu, lane > done && i < n && S.parent[i] == cur);
            if (!is) break;
            done = __ffs(is) - 1;
            const int x = i0 + done;
            bool take;
            if (P.mode == COLI_VERIFY_GREEDY) {
                take = S.token[x] == top;
            } else {
                const double u = (double)P.uniform[row + x];
                bool gone = false;
                for (int k = 0; k < lost; k++) gone |= S.lost[k] == S.token[x];
                take = draft ? (a + u * m) * (double)S.q[x] < (double)S.p[x] : u * m < (gone ? 0.0 : (double)S.p[x]);
            }
            if (take) {
                cur = x;
                if (rank == 0 && tid == 0) path[accepted] = x;
                accepted++;
                a = 0.0;
                m = 1.0;
                lost = 0;
                if (P.mode == COLI_VERIFY_GREEDY) top = largest();
            } else if (P.mode == COLI_VERIFY_SAMPLE) {
                if (draft) {
                    a += m;
                } else {
                    __syncthreads();  // the list is read above
                    if (tid == 0) S.lost[lost] = S.token[x];
                    lost++;
                    __syncthreads();
                }
                m = total(false);
            }
        }
    }
    if (rank == 0 && tid == 0) P.count[b] = accepted;
    if (P.mode == COLI_VERIFY_GREEDY) {
        if (rank == 0 && tid == 0) P.next[b] = top;
        return;
    }
    // the token behind: where the running sum of r passes u * sum r
    double all = total(false);
    bool whole = false;
    if (!(all > 0.0)) {
        whole = true;
        all = total(true);
    }
    double border = (double)P.uniform[row] * all;
    if (!(border >= 0.0)) border = 0.0;  // no number in [0, 1)
    // the last CTA with anything takes what rounding leaves behind the sum
    double mine = 0.0;
    int last = 0;
    for (int k = 0; k < kCluster; k++) {
        const double t = S.part[turn ^ 1][k];
        if (k == rank) mine = t;
        if (t > 0.0) last = k;
    }
    const bool here = mine > 0.0 && before <= border && (border < before + mine || rank == last);
    if (here && w == 0) {
        // the chunk, then the token
        double run = before;
        int found = -1;
        double found_at = 0.0;
        for (int c = 0; c < chunks; c++) {
            const double t = S.chunk[c];
            if (t > 0.0) {
                found = c;
                found_at = run;
                if (border < run + t) break;
                run += t;
            }
        }
        const float ah = (float)a, al = (float)(a - (double)ah);
        int token = -1, fallback = 0;
        run = found_at;
#pragma unroll 1
        for (int k = 0; k < kChunk / (32 * kPer) && token < 0; k++) {
            Two r[kPer];
            const int x = v0 + found * kChunk + (k * 32 + lane) * kPer;
            left(x, v1, ah, al, whole, r);
            double s[kPer], t = 0.0;
            int positive = -1;
#pragma unroll
            for (int j = 0; j < kPer; j++) {
                const double e = (double)r[j].hi + (double)r[j].lo;
                if (e > 0.0) positive = x + j;
                t += e;
                s[j] = t;
            }
            double upto = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            const double base = run + (upto - t);
            int hit = -1;
#pragma unroll
            for (int j = kPer - 1; j >= 0; j--)
                if (base + s[j] > border) hit = x + j;
            const unsigned hits = __ballot_sync(0xffffffffu, hit >= 0);
            const int most = __reduce_max_sync(0xffffffffu, positive);
            if (most >= 0) fallback = most;
            if (hits) token = __shfl_sync(0xffffffffu, hit, __ffs(hits) - 1);
            run += __shfl_sync(0xffffffffu, upto, 31);
        }
        if (lane == 0) P.next[b] = token >= 0 ? token : fallback;
    }
    // a row of nothing (no distribution) gives its first token
    if (!(all > 0.0) && rank == 0 && tid == 0) P.next[b] = 0;
}

template <typename T>
cudaError_t launch_typed(const VerifyParams &P, cudaStream_t s) {
    const int slice = ((P.vocab + kCluster - 1) / kCluster + kChunk - 1) / kChunk * kChunk;
    constexpr int kAlign = sizeof(T) * kPer;
    auto ok = [](const void *p, int64_t stride) {
        return reinterpret_cast<uintptr_t>(p) % kAlign == 0 && stride % kPer == 0;
    };
    const int vec = ok(P.target, P.target_stride) && ok(P.draft, P.draft ? P.draft_stride : 0);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)P.seqs * kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kCluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, draft_verify_kernel<T>, P, slice, vec);
}

}  // namespace

cudaError_t launch_draft_verify(const VerifyParams &P, cudaStream_t s) {
    switch (P.act) {
    case COLI_ACT_F32: return launch_typed<float>(P, s);
    case COLI_ACT_BF16: return launch_typed<__nv_bfloat16>(P, s);
    default: return launch_typed<__half>(P, s);
    }
}

}  // namespace colimoe

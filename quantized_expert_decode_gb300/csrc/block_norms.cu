// block_norms.cu — the norms before and after a block, its gate and the scaled residual, one launch.
//
//   z = y * post_w / sqrt(mean y^2 + e1);  r = a * resid + gate * z;  xn = r * pre_w / sqrt(mean r^2 + e2)
//
// What bounds it: bytes. A row is read once into registers as fp32 and both norms are taken from
// there; the two sums of squares are reduced by shuffles and one exchange through shared memory
// each. Rows wider than a CTA's registers are spread over a cluster, whose CTAs exchange their sums
// through distributed shared memory.
#include <cooperative_groups.h>

#include "act.cuh"
#include "host.h"
#include "layer.h"
#include "pdl.cuh"

namespace cg = cooperative_groups;

namespace colimoe {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxElems = 16;  // elements of a row that a thread holds

// Sum over the CTA, then over the cluster; every thread gets it. `part` is written once per call, so
// that the two sums of a row need no barrier between them.
template <bool kCluster>
__device__ __forceinline__ float row_sum(float v, float *part, float *cta) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int warps = blockDim.x / 32, w = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (lane == 0) part[w] = v;
    __syncthreads();
    float s = lane < warps ? part[lane] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (kCluster) {
        cg::cluster_group cl = cg::this_cluster();
        if (threadIdx.x == 0) *cta = s;
        cl.sync();
        const int n = (int)cl.num_blocks();
        s = 0.f;
        for (int i = 0; i < n; i++) s += *cl.map_shared_rank(cta, i);
    }
    return s;
}

// T the activation type, V elements per access, N accesses per thread. kEarly: the factors are loaded beside the
// row, before the first sum (one row of 6144: 3.1 us against 4.0); else where they are used, which leaves
// registers for a second CTA on the SM (4099 rows: 60 us against 87).
template <typename T, int V, int N, bool kCluster, bool kEarly>
__global__ void __launch_bounds__(kMaxThreads, kEarly ? 1 : 2) block_norms_kernel(const NormsParams P) {
    __shared__ float part[2][32];
    __shared__ float cta[2];
    wait_for_previous();
    let_next_start();
    int row = blockIdx.x, rank = 0, ranks = 1;
    if (kCluster) {
        cg::cluster_group cl = cg::this_cluster();
        ranks = (int)cl.num_blocks();
        rank = (int)cl.block_rank();
        row = blockIdx.x / ranks;
    }
    const int step = blockDim.x * ranks, first = rank * blockDim.x + threadIdx.x;
    const T *y = (const T *)P.y + row * P.y_stride, *r = (const T *)P.resid + row * P.resid_stride;
    const T *g = (const T *)P.gate + (P.gate_kind == COLI_GATE_ELEMENT ? row * P.gate_stride : 0);
    const int runs = P.width / V;  // V divides width
    Run<T, V> yv[N], rv[N];
#pragma unroll
    for (int i = 0; i < N; i++) {
        const int c = first + i * step;
        if (c < runs) {
            yv[i].load(y + (int64_t)c * V);
            rv[i].load(r + (int64_t)c * V);
        }
    }
    const bool channels = P.gate_kind == COLI_GATE_CHANNEL || P.gate_kind == COLI_GATE_ELEMENT;
    Run<float, V> w0[N], w1[N];
    Run<T, V> gv[N];
    auto load_first = [&](int i, int c) {
        if (P.post_w) w0[i].load(P.post_w + (int64_t)c * V);
        if (channels) gv[i].load(g + (int64_t)c * V);
    };
    if constexpr (kEarly) {
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int c = first + i * step;
            if (c >= runs) continue;
            load_first(i, c);
            if (P.pre_w) w1[i].load(P.pre_w + (int64_t)c * V);
        }
    }
    float z[N * V];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < N; i++)
#pragma unroll
        for (int j = 0; j < V; j++) {
            const float v = first + i * step < runs ? to_f32(yv[i].e[j]) : 0.f;
            z[i * V + j] = v;
            ss = fmaf(v, v, ss);
        }
    float grow = 1.f;
    if (P.gate_kind == COLI_GATE_ROW) grow = to_f32(g[row]);
    float rs = 1.f;
    if (P.post_w) rs = rsqrtf(row_sum<kCluster>(ss, part[0], &cta[0]) / (float)P.width + P.post_eps);
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < N; i++) {
        const int c = first + i * step;
        if (c >= runs) continue;
        if constexpr (!kEarly) load_first(i, c);
        Run<T, V> o;
#pragma unroll
        for (int j = 0; j < V; j++) {
            float v = z[i * V + j];
            if (P.post_w) v = v * rs * w0[i].e[j];
            v *= channels ? to_f32(gv[i].e[j]) : grow;
            v = fmaf(P.resid_scale, to_f32(rv[i].e[j]), v);
            z[i * V + j] = v;
            ss = fmaf(v, v, ss);
            o.e[j] = from_f32<T>(v);
        }
        o.store((T *)P.resid_out + row * P.resid_out_stride + (int64_t)c * V);
    }
    if (P.pre_w) {
        rs = rsqrtf(row_sum<kCluster>(ss, part[1], &cta[1]) / (float)P.width + P.pre_eps);
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int c = first + i * step;
            if (c >= runs) continue;
            if constexpr (!kEarly) w1[i].load(P.pre_w + (int64_t)c * V);
            Run<T, V> o;
#pragma unroll
            for (int j = 0; j < V; j++) o.e[j] = from_f32<T>(z[i * V + j] * rs * w1[i].e[j]);
            o.store((T *)P.xn + row * P.xn_stride + (int64_t)c * V);
        }
    }
    // no CTA leaves while another may still read its sums
    if (kCluster) cg::this_cluster().sync();
}

template <typename T, int V, int N>
cudaError_t launch_n(const NormsParams &P, int threads, int ranks, cudaStream_t s) {
    if (ranks == 1)  // a row for every SM or fewer: latency
        return P.rows <= num_sms() ? launch_overlapped(block_norms_kernel<T, V, N, false, true>, dim3(P.rows), threads, 0, s, P)
                                   : launch_overlapped(block_norms_kernel<T, V, N, false, false>, dim3(P.rows), threads, 0, s, P);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)P.rows * ranks);
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ranks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;  // (not overlapped: wait_for_previous returns at once)
    return cudaLaunchKernelEx(&cfg, block_norms_kernel<T, V, N, true, false>, P);
}

// width over threads of at most kMaxElems elements each, over more CTAs where one does not hold it
template <typename T, int V>
cudaError_t launch_v(const NormsParams &P, cudaStream_t s) {
    constexpr int kMaxN = kMaxElems / V;
    const int runs = P.width / V;
    int ranks = 1;
    while ((int64_t)ranks * kMaxThreads * kMaxN < runs) ranks *= 2;
    const int per = (runs + ranks - 1) / ranks;
    // as few accesses per thread as 512 threads allow
    const int n = (per + kMaxThreads - 1) / kMaxThreads;
    auto threads = [&](int k) { return ((per + k - 1) / k + 31) / 32 * 32; };
    if constexpr (V == 1) return launch_n<T, V, kMaxN>(P, threads(kMaxN), ranks, s);
    else if constexpr (kMaxN == 2) return n == 1 ? launch_n<T, V, 1>(P, threads(1), ranks, s) : launch_n<T, V, 2>(P, threads(2), ranks, s);
    else return n == 1   ? launch_n<T, V, 1>(P, threads(1), ranks, s)
                : n == 2 ? launch_n<T, V, 2>(P, threads(2), ranks, s)
                : n == 3 ? launch_n<T, V, 3>(P, threads(3), ranks, s)
                         : launch_n<T, V, 4>(P, threads(4), ranks, s);
}

template <typename T>
cudaError_t launch_t(const NormsParams &P, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    auto ok = [](const void *p, int64_t stride) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % V == 0;
    };
    const bool wide = P.width % V == 0 && ok(P.y, P.y_stride) && ok(P.resid, P.resid_stride) &&
                      ok(P.resid_out, P.resid_out_stride) && ok(P.post_w, 0) && ok(P.pre_w, 0) &&
                      (!P.pre_w || ok(P.xn, P.xn_stride)) &&
                      (P.gate_kind != COLI_GATE_CHANNEL || ok(P.gate, 0)) &&
                      (P.gate_kind != COLI_GATE_ELEMENT || ok(P.gate, P.gate_stride));
    return wide ? launch_v<T, V>(P, s) : launch_v<T, 1>(P, s);
}

}  // namespace

cudaError_t launch_block_norms(const NormsParams &P, cudaStream_t s) {
    switch (P.act) {
    case COLI_ACT_F32: return launch_t<float>(P, s);
    case COLI_ACT_BF16: return launch_t<__nv_bfloat16>(P, s);
    default: return launch_t<__half>(P, s);
    }
}

}  // namespace colimoe

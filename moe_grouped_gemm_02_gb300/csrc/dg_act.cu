// Backward pass of the GEMMs' epilogues: from the gradient dd of D and the kept pre-activations
// z, the gradient dz = dd * act'(z) and the bias gradient, the column sums of dz over an
// expert's rows.  (The residual's gradient is dd itself.)
//
// Bound by HBM: z and dd are read once, dz is written once, ~12 operations per value.  A CTA takes
// one 128-row block and 256 columns: each lane 8 columns (16 bytes of z), each of the 8 warps 16
// rows, four rows' loads in flight.  The column sums stay in FP32 registers over a warp's 16
// rows, are added over the warps in shared memory and leave as one row of partial sums per
// block; a second kernel adds an expert's blocks in a fixed order (no atomics).  The sums take
// the FP32 gradients, before their rounding to BF16 (their accuracy: act_sigmoid in dg_act.cuh).  33152 x 4096, SwiGLU: 671 MB in 106 us, 6.3 TB/s (two
// or eight rows in flight: 112 and 119 us); with GELU 808 MB in 141 us, bound by instruction issue.
#include "dg_act.cuh"
#include "dg_internal.h"
#include "dg_ptx.cuh"

#include <algorithm>
#include <climits>

namespace dg {

namespace {

constexpr int AB_WARPS = 8;
constexpr int AB_COLS = 256;
constexpr int AB_ROWS = 128 / AB_WARPS;
static_assert(AB_COLS == 32 * AB_WARPS, "one thread adds one column over the warps");

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

template <int ACT>
__global__ void __launch_bounds__(32 * AB_WARPS)
    act_backward_kernel(const uint16_t* __restrict__ dd, const uint16_t* __restrict__ z,
                        const int32_t* __restrict__ m_indices, uint16_t* __restrict__ dz, float* __restrict__ part,
                        int rows, int N, int experts, int strips) {
    constexpr bool GATED = ACT == ACT_SWIGLU;
    __shared__ float sums[AB_WARPS][AB_COLS];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int block = blockIdx.x / strips, strip = blockIdx.x - block * strips;
    const int col = strip * AB_COLS + 8 * lane;
    const bool in = col < N;
    const int H = GATED ? N / 2 : N;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
#pragma unroll
    for (int r0 = 0; r0 < AB_ROWS; r0 += 4) {
        uint4 zv[4], dv[4];
        bool live[4], valid[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const long long row = 128LL * block + AB_ROWS * warp + r0 + u;
            live[u] = in && row < rows;
            // (-1 is past every expert as an unsigned number)
            valid[u] = live[u] && (m_indices == nullptr ||
                                   static_cast<uint32_t>(__ldg(m_indices + row)) < static_cast<uint32_t>(experts));
            zv[u] = make_uint4(0u, 0u, 0u, 0u);
            dv[u] = zv[u];
            if (valid[u]) {
                zv[u] = __ldcs(reinterpret_cast<const uint4*>(z + row * N + col));
                if constexpr (GATED) {
                    const uint2 h = __ldcs(reinterpret_cast<const uint2*>(dd + row * H + col / 2));
                    dv[u].x = h.x;
                    dv[u].y = h.y;
                } else {
                    dv[u] = __ldcs(reinterpret_cast<const uint4*>(dd + row * H + col));
                }
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (!live[u]) continue;
            const uint32_t zw[4] = {zv[u].x, zv[u].y, zv[u].z, zv[u].w};
            const uint32_t dw[4] = {dv[u].x, dv[u].y, dv[u].z, dv[u].w};
            uint32_t out[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float a = lo_f(zw[i]), b = hi_f(zw[i]);
                if constexpr (GATED) {
                    // pair i: gate a, up b, one gradient
                    const float d = i & 1 ? hi_f(dw[i >> 1]) : lo_f(dw[i >> 1]);
                    const float t = act_sigmoid(a);
                    const float da = d * b * t * (1.0f + a * (1.0f - t));
                    b = d * a * t;
                    a = da;
                } else {
                    a = lo_f(dw[i]) * act_slope<ACT>(a);
                    b = hi_f(dw[i]) * act_slope<ACT>(b);
                }
                if (!valid[u]) a = b = 0.0f;
                acc[2 * i] += a;
                acc[2 * i + 1] += b;
                out[i] = bf16_pair(a, b);
            }
            const long long row = 128LL * block + AB_ROWS * warp + r0 + u;
            __stcs(reinterpret_cast<uint4*>(dz + row * N + col), make_uint4(out[0], out[1], out[2], out[3]));
        }
    }
    if (part == nullptr) return;
#pragma unroll
    for (int i = 0; i < 8; i += 4)
        *reinterpret_cast<float4*>(&sums[warp][8 * lane + i]) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
    __syncthreads();
    const int c = strip * AB_COLS + static_cast<int>(threadIdx.x);
    if (c < N) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < AB_WARPS; ++w) s += sums[w][threadIdx.x];
        part[static_cast<size_t>(block) * N + c] = s;
    }
}

// dbias[g][c]: the partial sums of g's blocks (all blocks without m_indices).  One CTA takes 128
// columns of one expert, four per lane; its warps take every W-th block each, then the warps' sums are
// added in order.  An expert's blocks are the range from its first to its last block.
constexpr int BR_WARPS = 32;      // the most warps of a CTA
constexpr int BR_COLS = 128;
__global__ void __launch_bounds__(32 * BR_WARPS)
    bias_reduce_kernel(const float* __restrict__ part, const int32_t* __restrict__ m_indices, float* __restrict__ dbias,
                       int blocks, int N, int strips) {
    __shared__ float4 sums[BR_WARPS][32];
    __shared__ int range[2];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5;
    const int g = blockIdx.x / strips, strip = blockIdx.x - g * strips;
    if (threadIdx.x == 0) {
        range[0] = m_indices ? blocks : 0;
        range[1] = m_indices ? -1 : blocks - 1;
    }
    __syncthreads();
    if (m_indices)
        for (int b = threadIdx.x; b < blocks; b += blockDim.x)
            if (__ldg(m_indices + 128LL * b) == g) {
                atomicMin(&range[0], b);
                atomicMax(&range[1], b);
            }
    __syncthreads();
    const int c = BR_COLS * strip + 4 * lane;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (c < N) {
        const int last = range[1];
#pragma unroll 4
        for (int b = range[0] + warp; b <= last; b += W)
            if (m_indices == nullptr || __ldg(m_indices + 128LL * b) == g) {
                const float4 x = *reinterpret_cast<const float4*>(part + static_cast<size_t>(b) * N + c);
                s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
            }
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < N) {
        float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int w = 0; w < W; ++w) {
            const float4 x = sums[w][lane];
            t.x += x.x, t.y += x.y, t.z += x.z, t.w += x.w;
        }
        *reinterpret_cast<float4*>(dbias + static_cast<size_t>(g) * N + c) = t;
    }
}

cudaError_t launch(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, long long blocks, int threads, int pdl,
                   cudaStream_t stream) {
    if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_act_backward(const void* dd, const void* z, const int32_t* m_indices, void* dz, float* dbias,
                                float* part, int rows, int N, int G, int act, int pdl, cudaStream_t stream) {
    const int blocks = (rows + 127) / 128, strips = (N + AB_COLS - 1) / AB_COLS;
    const int experts = dbias ? G : INT_MAX;      // (without dbias nothing says how many there are)
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    cudaError_t e;
    if (blocks > 0) {
        e = launch(cfg, attr, static_cast<long long>(blocks) * strips, 32 * AB_WARPS, pdl, stream);
        if (e != cudaSuccess) return e;
        auto go = [&](auto kernel) {
            return cudaLaunchKernelEx(&cfg, kernel, static_cast<const uint16_t*>(dd), static_cast<const uint16_t*>(z),
                                      m_indices, static_cast<uint16_t*>(dz), dbias ? part : nullptr, rows, N, experts, strips);
        };
        e = act == ACT_RELU     ? go(act_backward_kernel<ACT_RELU>)
            : act == ACT_GELU   ? go(act_backward_kernel<ACT_GELU>)
            : act == ACT_SILU   ? go(act_backward_kernel<ACT_SILU>)
            : act == ACT_SWIGLU ? go(act_backward_kernel<ACT_SWIGLU>)
                                : go(act_backward_kernel<ACT_NONE>);
        if (e != cudaSuccess) return e;
    }
    if (!dbias) return cudaSuccess;
    // a warp for every four blocks an expert has on average
    const int cols = (N + BR_COLS - 1) / BR_COLS;
    const int warps = std::max(2, std::min(BR_WARPS, (blocks / G + 3) / 4));
    e = launch(cfg, attr, static_cast<long long>(cols) * G, 32 * warps, pdl, stream);
    if (e != cudaSuccess) return e;
    return cudaLaunchKernelEx(&cfg, bias_reduce_kernel, static_cast<const float*>(part), m_indices, dbias, blocks, N, cols);
}

}  // namespace dg

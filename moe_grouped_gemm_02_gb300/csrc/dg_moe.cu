// The steps of an MoE layer around its grouped GEMMs: the router's choice of experts, the sort
// of the (token, choice) slots into a grouped layout, the dispatch of the tokens to their
// experts' rows (as BF16/FP32 rows, or quantised to E4M3 with packed scales on the way) and the
// weighted sum of the experts' rows back in token order, with the gradients.
#include "dg_internal.h"
#include "dg_ptx.cuh"
#include "dg_quant.cuh"

#include <algorithm>
#include <cfloat>
#include <climits>
#include <type_traits>

namespace dg {

namespace {

constexpr uint32_t FULL = 0xffffffffu;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two FP32 values rounded to nearest-even BF16, `lo` in the low half.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(FULL, v, off);
    return v;
}

cudaError_t launch_cfg(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, long long blocks, int threads, int pdl,
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

// ---------------------------------------------------------------------------------------------
// Router
// ---------------------------------------------------------------------------------------------
// One warp per token; lane l holds the NV consecutive logits from l * NV on, as keys whose
// unsigned order is the logits' order.  Each lane sorts its keys once and leaves the list in
// shared memory; a choice is then the largest head over the lanes (one redux), and the lane
// that gave it loads its next key.  A BF16 logit and its index share one 32-bit key (16 bits
// each; the complement of the index, so that ties go to the lowest).  FP32 keys take all 32
// bits: ties go to the lowest lane, and the chosen keys' indices are found afterwards, all k at
// once, by searching the row segment of the lane that gave each.
//
// 32768 tokens, 256 BF16 experts, k = 8: 10.2 us; its 19 MB cross HBM in 2.8.  Bound by instructions and by the
// latencies between them: 241 instructions per token take the schedulers 6.8 us of it (59 % of the active cycles), the
// launch 1.8; in between the warps wait for a token's loads, the ALU pipe and the redux of one choice before the next.
constexpr int ROUTE_WARPS = 4;
constexpr int ROUTE_CTAS = 152 * 16;     // CTAs that get one token per warp; with more, warps take several

// A logit as the router sees it: NaN counts as -inf (never chosen), -0 as +0; +inf counts as the
// largest finite value (see finite_value).
__device__ __forceinline__ float canonical(float x) { return fmaxf(x, -INFINITY) + 0.0f; }
__device__ __forceinline__ float finite_value(float x) { return fminf(x, FLT_MAX); }

template <bool F32>
__device__ __forceinline__ const void* logit_row(const void* logits, size_t t, int E) {
    return static_cast<const char*>(logits) + t * E * (F32 ? 4 : 2);
}

template <bool F32>
__device__ __forceinline__ float load_logit(const void* row, int i) {
    const float x = F32 ? __ldg(static_cast<const float*>(row) + i)
                        : __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(row) + i)) << 16);
    return canonical(x);
}

// Words of NV consecutive logits: two BF16 or one FP32 each (the last half of an odd BF16 word: -inf).
template <int NV, bool F32>
constexpr int LOGIT_WORDS = F32 ? NV : (NV + 1) / 2;

// Logits [i0, i0 + NV) of a row of E as they are stored, past its end -inf.  With `vec`, loads of up
// to 16 bytes: every load is aligned and whole or past the end.
template <int NV, bool F32>
__device__ __forceinline__ void load_logit_words(const void* row, int i0, int E, bool vec, uint32_t (&w)[LOGIT_WORDS<NV, F32>]) {
    constexpr int SIZE = F32 ? 4 : 2;
    constexpr int BYTES = NV * SIZE < 16 ? NV * SIZE : 16;     // of a load
    constexpr uint32_t NONE = F32 ? 0xFF800000u : 0xFF80FF80u;
    constexpr int W = LOGIT_WORDS<NV, F32>;
#pragma unroll
    for (int v = 0; v < W; ++v) w[v] = NONE;
    const char* p = static_cast<const char*>(row) + static_cast<size_t>(i0) * SIZE;
    if (BYTES >= 4 && vec) {
#pragma unroll
        for (int v = 0; v < NV; v += BYTES / SIZE) {
            if (i0 + v >= E) continue;
            uint32_t* to = w + v * SIZE / 4;
            if constexpr (BYTES == 16) {
                const uint4 x = __ldg(reinterpret_cast<const uint4*>(p + v * SIZE));
                to[0] = x.x, to[1] = x.y, to[2] = x.z, to[3] = x.w;
            } else if constexpr (BYTES == 8) {
                const uint2 x = __ldg(reinterpret_cast<const uint2*>(p + v * SIZE));
                to[0] = x.x, to[1] = x.y;
            } else {
                to[0] = __ldg(reinterpret_cast<const uint32_t*>(p + v * SIZE));
            }
        }
        return;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        if (i0 + v >= E) continue;
        if constexpr (F32) {
            w[v] = __ldg(reinterpret_cast<const uint32_t*>(p) + v);
        } else {
            const uint32_t x = __ldg(reinterpret_cast<const uint16_t*>(p) + v);
            w[v / 2] = v & 1 ? (w[v / 2] & 0xFFFFu) | (x << 16) : (w[v / 2] & 0xFFFF0000u) | x;
        }
    }
}

// Logit v of those words as a value.
template <int NV, bool F32>
__device__ __forceinline__ float word_logit(const uint32_t (&w)[LOGIT_WORDS<NV, F32>], int v) {
    return canonical(F32 ? __uint_as_float(w[F32 ? v : 0]) : (v & 1 ? bf16_hi(w[v / 2]) : bf16_lo(w[v / 2])));
}

template <int NV, bool F32>
__device__ __forceinline__ void load_logits(const void* row, int i0, int E, bool vec, float (&x)[NV]) {
    uint32_t w[LOGIT_WORDS<NV, F32>];
    load_logit_words<NV, F32>(row, i0, E, vec, w);
#pragma unroll
    for (int v = 0; v < NV; ++v) x[v] = word_logit<NV, F32>(w, v);
}

// Whether a lane's segments of NV logits of rows of E can be loaded and stored in wide units.
__host__ inline int logits_vec(int nv, int f32, int E) { return E % std::min(nv, f32 ? 4 : 8) == 0; }

// Order keys of two BF16 logits, one in each half: -0 becomes +0 and NaN -inf, then the sign
// decides which bits are flipped.
__device__ __forceinline__ uint32_t order_key_bf16x2(uint32_t w) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(0xFF80FF80u));
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(0u));
    return r ^ (prmt(r, r, 0xBB99u) | 0x80008000u);
}

__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k >> 31) ? k ^ 0x80000000u : ~k);
}
// The key of the BF16 logit whose upper half m holds: the lower half is all zeros or all ones, by the sign.
__device__ __forceinline__ uint32_t bf16_key(uint32_t m) { return (m & 0xFFFF0000u) | ((m >> 31) ? 0u : 0xFFFFu); }
constexpr uint32_t KEY_NONE = 0x007FFFFFu;   // order_key(-inf): nothing at or below it is chosen

// Batcher's odd-even merge sort of N (a power of two) keys, descending: for P = 1, 2, .., N / 2 and Q = P, P / 2,
// .., 1 the exchanges of keys Q apart.  The steps are template parameters and each is one flat loop, so that every
// index is a constant and the keys stay in registers (as nested loops they went to local memory at N = 32).
template <int N, int P = 1, int Q = 1>
__device__ __forceinline__ void sort_descending(uint32_t (&e)[N]) {
    if constexpr (P < N) {
#pragma unroll
        for (int i = Q % P; i + Q < N; ++i)
            if ((i - Q % P) % (2 * Q) < Q && i / (2 * P) == (i + Q) / (2 * P)) {
                const uint32_t a = e[i], b = e[i + Q];
                e[i] = max(a, b);
                e[i + Q] = min(a, b);
            }
        if constexpr (Q > 1) sort_descending<N, P, Q / 2>(e);
        else sort_descending<N, 2 * P, 2 * P>(e);
    }
}

// a / b, 0 <= a <= b, b from 1/2 to 1024 (or a = 0): a quotient good to two units and one step of correction by its
// exact remainder, which leaves an error of 2^-20 units before the one rounding.  (An IEEE division, with its
// branch for all other ranges: 3-7 % of the kernel.)
__device__ __forceinline__ float quotient(float a, float b) {
    const float r = __fdividef(1.0f, b), q = a * r;
    return fmaf(fmaf(-b, q, a), r, q);
}

// sigmoid(x) e^-min(top, 0), x <= top: the sigmoid itself with top = 0.  With a token's largest chosen logit as
// top the scores' sum is at least 1/2 and their ratios stay right where the scores themselves underflow (logits
// below about -87).  A logit below SIGMOID_ZERO, such as a mask of the type's lowest value, scores 0.
constexpr float SIGMOID_ZERO = -700.0f;
__device__ __forceinline__ float sigmoid_over(float x, float top) {
    const float up = x >= 0.0f ? 1.0f : x >= SIGMOID_ZERO ? expf(x - fminf(top, 0.0f)) : 0.0f;
    return quotient(up, 1.0f + expf(-fabsf(x)));
}

// group: tokens whose choices share the lanes of the last steps (scores, sums, stores), each
// with slot lanes (a power of two >= k).
// (12 CTAs per SM leave 40 registers: at the compiler's own choice of 31, 32768 x 256 BF16 took 11.1 us instead of 10.2.)
template <int NV, bool F32>
__global__ void __launch_bounds__(32 * ROUTE_WARPS, NV <= 8 ? 12 : 0)
    route_kernel(const void* __restrict__ logits, int32_t* __restrict__ topk_idx, float* __restrict__ topk_w, int T,
                 int E, int k, int sigmoid, int renorm, float scale, int vec, int group, int slot) {
    // row v: every lane's v-th key; the last row is below every key
    __shared__ uint32_t lists[ROUTE_WARPS][NV + 1][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    lists[warp][NV][lane] = 0u;
    uint32_t tag[NV];                                  // BF16: the complement of each logit's index
#pragma unroll
    for (int v = 0; v < NV; ++v) tag[v] = static_cast<uint32_t>(0xFFFF - (lane * NV + v));
    const int my_slot = lane / slot, my_j = lane & (slot - 1);
    griddep_wait();
    griddep_launch_dependents();
    const int t0 = (blockIdx.x * ROUTE_WARPS + warp) * group;
    if (t0 >= T) return;
    uint32_t mine = 0u;                            // the lane's choice: its key, the lane that gave it
    int owner = 0;
    float sum = 0.0f;
    for (int s = 0; s < group && t0 + s < T; ++s) {
        uint32_t w[LOGIT_WORDS<NV, F32>], e[NV];
        load_logit_words<NV, F32>(logit_row<F32>(logits, t0 + s, E), lane * NV, E, vec != 0, w);
#pragma unroll
        for (int v = 0; v < NV; v += 2) {
            if constexpr (F32) {
                e[v] = order_key(word_logit<NV, F32>(w, v));
                if (v + 1 < NV) e[(v + 1) % NV] = order_key(word_logit<NV, F32>(w, (v + 1) % NV));
            } else {
                const uint32_t key = order_key_bf16x2(w[v / 2]);
                e[v] = prmt(tag[v], key, 0x5410u);
                if (v + 1 < NV) e[(v + 1) % NV] = prmt(tag[(v + 1) % NV], key, 0x7610u);
            }
        }
        sort_descending(e);
        __syncwarp();                              // (the last token's reads of the lists are done)
#pragma unroll
        for (int v = 1; v < NV; ++v) lists[warp][v][lane] = e[v];
        const uint32_t* next = &lists[warp][0][lane];
        uint32_t head = e[0];
        if (!sigmoid && !renorm) {
            const uint32_t m = __reduce_max_sync(FULL, head);
            const float top = finite_value(key_value(F32 ? m : bf16_key(m)));
            float part = 0.0f;
#pragma unroll
            for (int v = 0; v < NV; ++v) part += expf(finite_value(word_logit<NV, F32>(w, v)) - top);
            part = warp_sum(part);
            if (my_slot == s) sum = part;
        }
        const int target = s * slot;
#pragma unroll 8
        for (int j = 0; j < k; ++j) {
            const uint32_t m = __reduce_max_sync(FULL, head);
            bool won = head == m;
            if (F32) {
                const uint32_t who = __ballot_sync(FULL, won);
                const int first = __ffs(who) - 1;
                won = lane == first;
                if (lane == target + j) owner = first;
            }
            if (lane == target + j) mine = m;
            if (won) {
                next += 32;
                head = *next;
            }
        }
    }
    const int t = t0 + my_slot;
    const bool have = mine > (F32 ? KEY_NONE : KEY_NONE | 0xFFFFu);
    int index = static_cast<int>(0xFFFFu - (mine & 0xFFFFu));
    const float value = finite_value(key_value(F32 ? mine : bf16_key(mine)));
    if (F32) {
        // the n-th logit with this key in the owner's segment, n counting the token's earlier
        // choices of the same key from the same lane
        const uint32_t same = __match_any_sync(FULL, mine) & __match_any_sync(FULL, owner | (my_slot << 8));
        int n = __popc(same & ((1u << lane) - 1u));
        if (have) {
            float y[NV];
            load_logits<NV, F32>(logit_row<F32>(logits, t, E), owner * NV, E, vec != 0, y);
            index = -1;
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if (order_key(y[v]) == mine && n-- == 0) index = owner * NV + v;
        }
    }
    const float top = __shfl_sync(FULL, value, my_slot * slot);
    float w = 0.0f;
    if (have) w = sigmoid ? sigmoid_over(value, renorm ? top : 0.0f) : expf(value - top);
    if (renorm) {
        sum = w;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const float other = __shfl_xor_sync(FULL, sum, off);
            if (off < slot) sum += other;
        }
    }
    if (!sigmoid || renorm) w = quotient(w, fmaxf(sum, FLT_MIN));
    if (my_j < k && my_slot < group && t < T) {
        topk_idx[static_cast<size_t>(t) * k + my_j] = have ? index : -1;
        topk_w[static_cast<size_t>(t) * k + my_j] = have ? scale * w : 0.0f;
    }
}

// Gradient of the logits from the weights'.  With s the scores, w the returned weights:
//   softmax              dl_i = p_i (g_i - sum_c g_c p_c), g = scale * dw at the chosen, else 0
//   softmax, renorm      dl_c = scale p_c (dw_c - sum_c' dw_c' p_c'), p the softmax of the chosen
//   sigmoid              dl_c = scale s_c (1 - s_c) dw_c
//   sigmoid, renorm      dl_c = scale q_c (1 - s_c) (dw_c - sum_c' dw_c' q_c'), q = s / sum s
// Only the first has a gradient outside the chosen experts.  The row is written once by all
// lanes, then the chosen entries again by the lanes that hold them.
template <bool F32>
__device__ __forceinline__ void store_grad(void* row, int i, float x) {
    if (F32) static_cast<float*>(row)[i] = x;
    else static_cast<uint16_t*>(row)[i] = static_cast<uint16_t>(bf16x2(x, 0.0f));
}

template <int NV, bool F32>
__device__ __forceinline__ void store_grads(void* row, int i0, int E, bool vec, const float (&x)[NV]) {
    constexpr int SIZE = F32 ? 4 : 2;
    constexpr int BYTES = NV * SIZE < 16 ? NV * SIZE : 16;     // of a store
    if constexpr (BYTES >= 4) {
        if (vec) {
            constexpr int PER = BYTES / SIZE;
#pragma unroll
            for (int v = 0; v < NV; v += PER) {
                if (i0 + v >= E) continue;
                uint32_t u[BYTES / 4];
#pragma unroll
                for (int q = 0; q < BYTES / 4; ++q) {
                    if constexpr (F32) u[q] = __float_as_uint(x[v + q]);
                    else u[q] = bf16x2(x[v + 2 * q], x[v + 2 * q + 1]);
                }
                char* to = static_cast<char*>(row) + static_cast<size_t>(i0 + v) * SIZE;
                if constexpr (BYTES == 16) *reinterpret_cast<uint4*>(to) = make_uint4(u[0], u[1], u[2], u[3]);
                else if constexpr (BYTES == 8) *reinterpret_cast<uint2*>(to) = make_uint2(u[0], u[1]);
                else *reinterpret_cast<uint32_t*>(to) = u[0];
            }
            return;
        }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
        if (i0 + v < E) store_grad<F32>(row, i0 + v, x[v]);
}

// One warp per token.  Bound by the chain load, maximum, sums, store (two or four tokens per warp, with
// all their loads first, measured slower: 6.2 and 7.0 us instead of 6.0 at 16381 tokens, 160 FP32 logits).
template <int NV, bool F32>
__global__ void __launch_bounds__(32 * ROUTE_WARPS)
    route_backward_kernel(const void* __restrict__ logits, const int32_t* __restrict__ topk_idx,
                          const float* __restrict__ dw, void* __restrict__ dlogits, int T, int E, int k, int sigmoid,
                          int renorm, float scale, int vec) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * ROUTE_WARPS + (threadIdx.x >> 5);
    if (t >= T) return;
    const void* row = logit_row<F32>(logits, t, E);
    void* out = const_cast<void*>(logit_row<F32>(dlogits, t, E));
    const bool all = !sigmoid && !renorm, normed = !sigmoid || renorm;
    const size_t at = static_cast<size_t>(t) * k + lane;
    int my_i = lane < k ? __ldg(topk_idx + at) : -1;
    float g = lane < k ? __ldg(dw + at) : 0.0f;
    uint32_t w[LOGIT_WORDS<NV, F32>];
    if (all) load_logit_words<NV, F32>(row, lane * NV, E, vec != 0, w);
    if (my_i < 0 || my_i >= E) {
        my_i = -1;
        g = 0.0f;
    }
    const float x = my_i >= 0 ? finite_value(load_logit<F32>(row, my_i)) : -INFINITY;
    float p[NV];
    float m = x;
    if (all) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            p[v] = finite_value(word_logit<NV, F32>(w, v));
            m = fmaxf(m, p[v]);
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, off));
    m = fmaxf(m, -FLT_MAX);      // (a row with nothing available: every term below is 0)
    float s = 0.0f, slope = 1.0f, sum = 0.0f;
    if (sigmoid) {
        // both from e^-|x|: 1 - s of a rounded s would lose the slope of a large logit (all of it from 17 on)
        const float e = expf(-fabsf(x)), r = 1.0f / (1.0f + e);
        // (as sigmoid_over; x is -inf where there is no choice)
        s = x >= 0.0f ? r : x >= SIGMOID_ZERO ? (renorm ? expf(x - fminf(m, 0.0f)) : e) * r : 0.0f;
        slope = x >= 0.0f ? e * r : r;
    } else if (my_i >= 0) {
        s = expf(x - m);
    }
    if (all) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            p[v] = expf(p[v] - m);
            sum += p[v];
        }
    } else {
        sum = s;
    }
    // the scores' sum and sum_c g_c s_c travel together
    float mean = g * s;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        sum += __shfl_xor_sync(FULL, sum, off);
        mean += __shfl_xor_sync(FULL, mean, off);
    }
    const float inv = normed ? 1.0f / fmaxf(sum, FLT_MIN) : 1.0f;
    s *= inv;
    mean = normed ? mean * inv : 0.0f;
    const float f = -scale * inv * mean;
#pragma unroll
    for (int v = 0; v < NV; ++v) p[v] = all ? p[v] * f : 0.0f;
    store_grads<NV, F32>(out, lane * NV, E, vec != 0, p);
    __syncwarp();
    if (my_i >= 0) store_grad<F32>(out, my_i, scale * s * slope * (g - mean));
}

// ---------------------------------------------------------------------------------------------
// Sort
// ---------------------------------------------------------------------------------------------
// A stable counting sort of the n = T * k slots by expert, in one launch: one CTA, or one
// cluster of CTAs for long inputs.  Slots are split in order over the CTAs, their warps and the
// warps' 32-slot steps; within a step a match over the warp gives every slot its rank among
// equal experts, and each warp keeps its own running counts (no atomics: the order of the
// slots decides every position).  The prefix over warps, then over CTAs (distributed shared
// memory), then over the experts' 128-row aligned segments turns those ranks into rows.
// Bound by latencies (memory, barriers, the cluster's) below some 16000 slots, then by the ballots'
// and shared-memory instructions on its 16 SMs: 64 experts, 512 slots 4.3 us, 16384 4.9, 262144 14.7.
// Each slot's rank within its warp's share stays in registers while the counts are formed (shares
// of up to 256 slots), or waits in pos.
struct SortArgs {
    const int32_t* idx;
    int32_t* pos;
    int32_t* m_indices;   // contiguous only
    int32_t* counts;      // contiguous: slots per expert; masked: valid rows per group
    int32_t* ks;          // contiguous only, may be null
    int n, G;
    int rows;             // contiguous: rows of the layout
    int max_m;            // masked: rows per group (0: contiguous)
    int share;            // slots per warp, a multiple of 32
};

__device__ __forceinline__ uint32_t ld_shared_cluster(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

constexpr int SORT_STEPS = 8;    // 32-slot steps of a warp whose loads are in flight together

__host__ __device__ inline int sort_warps(int G) { return G <= 1024 ? 32 : 8; }
inline size_t sort_smem(int G) { return (static_cast<size_t>(sort_warps(G)) * G + 4 * static_cast<size_t>(G) + 32) * 4; }

// The lanes that hold the same v (of BITS bits, or -1): one ballot per bit.  (A match.any of 64
// different values per warp measured several times as long.)
template <int BITS>
__device__ __forceinline__ uint32_t equal_lanes(int v) {
    uint32_t same = __ballot_sync(FULL, v >= 0);
    if (v < 0) same = ~same;
#pragma unroll
    for (int b = 0; b < BITS; ++b) {
        const bool one = (v >> b) & 1;
        const uint32_t ones = __ballot_sync(FULL, one);
        same &= one ? ones : ~ones;
    }
    return same;
}

template <bool CLUSTER, int BITS>
__global__ void __launch_bounds__(1024, 1) sort_kernel(const SortArgs a) {
    extern __shared__ uint32_t sort_sm[];
    const int G = a.G;
    const int W = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t* hist = sort_sm;            // [W][G]: counts of each warp, then their prefix over the warps
    uint32_t* tot = hist + W * G;        // [G]: this CTA's counts (read by the cluster)
    uint32_t* base = tot + G;            // [G]: counts of the CTAs before this one, plus the segment's first row
    uint32_t* count = base + G;          // [G]: counts of all CTAs
    uint32_t* start = count + G;         // [G]: first row of each expert's segment
    uint32_t* scan = start + G;          // [32]
    const uint32_t rank = CLUSTER ? cluster_ctarank() : 0u;
    const uint32_t ctas = CLUSTER ? gridDim.x : 1u;

    // warps of this CTA that have slots: only their counts are cleared and scanned
    const long long ahead = static_cast<long long>(rank) * W * a.share;
    const int used = static_cast<int>(min(static_cast<long long>(W), max(0LL, (a.n - ahead + a.share - 1) / max(a.share, 1))));
    for (int i = threadIdx.x; i < used * G; i += blockDim.x) hist[i] = 0u;
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();

    const long long first = (static_cast<long long>(rank) * W + warp) * a.share;
    const int lo = static_cast<int>(min(first, static_cast<long long>(a.n)));
    const int hi = static_cast<int>(min(first + a.share, static_cast<long long>(a.n)));
    uint32_t* mine = hist + warp * G;
    const bool single = a.share <= 32 * SORT_STEPS;
    int e[SORT_STEPS];            // a batch's experts (-1: none), and the slots' ranks
    uint32_t r[SORT_STEPS];
    for (int i0 = lo; i0 < hi; i0 += 32 * SORT_STEPS) {
#pragma unroll
        for (int u = 0; u < SORT_STEPS; ++u) {
            const int i = i0 + 32 * u + lane;
            e[u] = i < hi ? __ldg(a.idx + i) : -1;
            if (e[u] < 0 || e[u] >= G) e[u] = -1;
        }
#pragma unroll
        for (int u = 0; u < SORT_STEPS; ++u) {
            if (i0 + 32 * u >= hi) break;
            const uint32_t peers = equal_lanes<BITS>(e[u]);
            const uint32_t before = __popc(peers & ((1u << lane) - 1u));
            const uint32_t had = e[u] >= 0 ? mine[e[u]] : 0u;
            __syncwarp();
            if (e[u] >= 0 && before == 0u) mine[e[u]] = had + __popc(peers);
            __syncwarp();
            r[u] = had + before;
            const int i = i0 + 32 * u + lane;
            if (!single && i < hi) a.pos[i] = static_cast<int32_t>(r[u]);
        }
    }
    __syncthreads();
    for (int g = threadIdx.x; g < G; g += blockDim.x) {
        uint32_t sum = 0u;
#pragma unroll 8
        for (int w = 0; w < used; ++w) {
            const uint32_t c = hist[w * G + g];
            hist[w * G + g] = sum;
            sum += c;
        }
        tot[g] = sum;
    }
    if (CLUSTER) cluster_sync_all();
    else __syncthreads();
    for (int g = threadIdx.x; g < G; g += blockDim.x) {
        uint32_t before = 0u, all = tot[g];
        if constexpr (CLUSTER) {
            all = 0u;
            const uint32_t at = smem_u32(tot + g);
#pragma unroll 8
            for (uint32_t c = 0; c < ctas; ++c) {
                const uint32_t v = ld_shared_cluster(map_to_rank(at, c));
                if (c < rank) before += v;
                all += v;
            }
        }
        base[g] = before;
        count[g] = all;
    }
    if (CLUSTER) cluster_arrive();       // this CTA has read the others' counts (waited for at exit)
    __syncthreads();

    if (a.max_m == 0) {
        // exclusive prefix over the experts' aligned counts: a run of experts per thread
        const int per = (G + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x);
        const int g0 = min(G, static_cast<int>(threadIdx.x) * per), g1 = min(G, g0 + per);
        uint32_t run = 0u;
        for (int g = g0; g < g1; ++g) run += (count[g] + 127u) & ~127u;
        uint32_t incl = run;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t v = __shfl_up_sync(FULL, incl, off);
            if (lane >= off) incl += v;
        }
        if (lane == 31) scan[warp] = incl;
        __syncthreads();
        if (warp == 0) {
            uint32_t v = lane < W ? scan[lane] : 0u;
            const uint32_t own = v;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t u = __shfl_up_sync(FULL, v, off);
                if (lane >= off) v += u;
            }
            scan[lane] = v - own;
        }
        __syncthreads();
        uint32_t at = scan[warp] + incl - run;
        for (int g = g0; g < g1; ++g) {
            const uint32_t c = count[g], padded = (c + 127u) & ~127u;
            if (rank == 0u) {
                // segments past the layout's rows are cut there
                const uint32_t room = at < static_cast<uint32_t>(a.rows) ? static_cast<uint32_t>(a.rows) - at : 0u;
                a.counts[g] = static_cast<int32_t>(min(c, room));
                if (a.ks) a.ks[g] = static_cast<int32_t>(min(padded, room));
            }
            start[g] = at;
            base[g] += at;
            at += padded;
        }
    } else {
        for (int g = threadIdx.x; g < G; g += blockDim.x)
            if (rank == 0u) a.counts[g] = static_cast<int32_t>(min(count[g], static_cast<uint32_t>(a.max_m)));
    }
    __syncthreads();
    // each warp's offsets: where its first slot of every expert goes
    if (warp < used)
        for (int g = lane; g < G; g += 32) mine[g] += base[g];
    __syncwarp();

    for (int i0 = lo; i0 < hi; i0 += 32 * SORT_STEPS) {
        if (!single) {
#pragma unroll
            for (int u = 0; u < SORT_STEPS; ++u) {
                const int i = i0 + 32 * u + lane;
                e[u] = i < hi ? __ldg(a.idx + i) : -1;
                r[u] = i < hi ? static_cast<uint32_t>(a.pos[i]) : 0u;
            }
        }
#pragma unroll
        for (int u = 0; u < SORT_STEPS; ++u) {
            const int i = i0 + 32 * u + lane;
            if (i >= hi) continue;
            int32_t p = -1;
            if (e[u] >= 0 && e[u] < G) {
                const uint32_t at = mine[e[u]] + r[u];
                if (a.max_m == 0) {
                    if (at < static_cast<uint32_t>(a.rows)) p = static_cast<int32_t>(at);
                } else if (at < static_cast<uint32_t>(a.max_m)) {
                    p = e[u] * a.max_m + static_cast<int32_t>(at);
                }
            }
            a.pos[i] = p;
        }
    }
    if (a.max_m == 0) {
        // the expert of every row, a 128-row block per warp (four rows per lane): a block lies
        // within one expert's segment, or past the last one
        const int blocks = a.rows / 128;
        for (int b = static_cast<int>(rank) * W + warp; b < blocks; b += static_cast<int>(ctas) * W) {
            const uint32_t r0 = 128u * static_cast<uint32_t>(b);
            int g0 = 0, g1 = G - 1;      // the last expert whose segment starts at or before the block
            while (g0 < g1) {
                const int mid = (g0 + g1 + 1) >> 1;
                if (start[mid] <= r0) g0 = mid; else g1 = mid - 1;
            }
            const uint32_t end = start[g0] + count[g0];
            const uint32_t r = r0 + 4u * lane;
            int4 v;
            v.x = r < end ? g0 : -1;
            v.y = r + 1u < end ? g0 : -1;
            v.z = r + 2u < end ? g0 : -1;
            v.w = r + 3u < end ? g0 : -1;
            *reinterpret_cast<int4*>(a.m_indices + r) = v;
        }
    }
    if (CLUSTER) cluster_wait();
}

// ---------------------------------------------------------------------------------------------
// Dispatch
// ---------------------------------------------------------------------------------------------
// Work unit: one warp takes one token and 512 elements (FP8) or 1 KB (copies) of its row, which
// it reads once and writes to the token's k rows.  Before the tokens' units come those of the
// contiguous layout's rows, 16 rows and one of pad_chunks column ranges per warp, which write the
// padding rows inside segments as zero rows (first, so that they are no tail; a 128-row block whose first
// row is -1 is past the last segment and stays as it is).
//
// Bound by HBM: the token-centric order reads x once, where a row-centric one would read it k times.
// 16384 tokens x 8 to 64 experts, K 7168, FP8: 1.2 GB in 179 us, 6.9 TB/s (a copy: 6.7).  Streaming stores:
// plain ones 1 % slower.
constexpr int DISPATCH_WARPS = 8;
constexpr int PAD_ROWS = 16;
constexpr int DISPATCH_U = 2;        // FP8: 512-element spans per warp

// The padding rows among rows [16 u, 16 u + 16), as bits; none past the last segment.
__device__ __forceinline__ uint32_t padding_bits(const int32_t* m_indices, long long u, int lane) {
    const int first = __ldg(m_indices + u / (128 / PAD_ROWS) * 128);
    const int e = lane < PAD_ROWS ? __ldg(m_indices + PAD_ROWS * u + lane) : 0;
    const uint32_t bits = __ballot_sync(FULL, e < 0);
    return first < 0 ? 0u : bits;
}

// Zeros to column range c of `chunks` of those rows of `out` (n16 16-byte units each); the whole warp.
__device__ __forceinline__ void zero_rows(uint32_t bits, uint4* out, long long u, int n16, int c, int chunks, int lane) {
    uint4* first = out + static_cast<size_t>(PAD_ROWS * u) * n16;
    const int i1 = static_cast<int>(static_cast<long long>(c + 1) * n16 / chunks);
    for (int i = static_cast<int>(static_cast<long long>(c) * n16 / chunks) + lane; i < i1; i += 32)
#pragma unroll
        for (int r = 0; r < PAD_ROWS; ++r)
            if ((bits >> r) & 1u) __stcs(first + static_cast<size_t>(r) * n16 + i, make_uint4(0u, 0u, 0u, 0u));
}

template <int U>
__global__ void __launch_bounds__(32 * DISPATCH_WARPS)
    dispatch_fp8_kernel(const uint16_t* __restrict__ x, const int32_t* __restrict__ pos,
                        const int32_t* __restrict__ m_indices, uint8_t* __restrict__ q, int32_t* __restrict__ sf, int T,
                        int k, int K, int Kb, int Kp, int G, int rows, int rows_al, int pad_chunks) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int lead = m_indices ? rows / PAD_ROWS * pad_chunks : 0;      // padding units
    const long long unit = static_cast<long long>(blockIdx.x) * DISPATCH_WARPS + (threadIdx.x >> 5) - lead;
    // lane l: elements 16l .. 16l + 15 of the unit's 512, in K block l / 8
    if (unit < 0) {
        const int at = static_cast<int>(unit + lead);
        const int u = at / pad_chunks, c = at - u * pad_chunks;
        const uint32_t bits = padding_bits(m_indices, u, lane);
        if (bits == 0u) return;
        zero_rows(bits, reinterpret_cast<uint4*>(q), u, K / 16, c, pad_chunks, lane);
        // an all-zero block has exponent 0: byte 127 in each valid block's place
        if (c == 0 && ((bits >> lane) & 1u))
            for (int kp = 0; kp < Kp; ++kp) {
                const int blocks = min(4, Kb - 4 * kp);
                sf[static_cast<size_t>(kp) * rows_al + PAD_ROWS * u + lane] =
                    static_cast<int32_t>(0x7F7F7F7Fu >> (8 * (4 - blocks)));
            }
        return;
    }
    const int spans = (Kp + U - 1) / U;           // units of a row
    if (unit >= static_cast<long long>(T) * spans) return;
    const int t = static_cast<int>(unit / spans), kp0 = U * static_cast<int>(unit - static_cast<long long>(t) * spans);
    int p = lane < k ? __ldg(pos + static_cast<size_t>(t) * k + lane) : -1;
    if (p >= static_cast<long long>(G) * rows) p = -1;
    uint32_t v[U][8];
    bool valid[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        valid[u] = 4 * (kp0 + u) + (lane >> 3) < Kb;
        uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
        if (valid[u]) {
            const uint4* src = reinterpret_cast<const uint4*>(x + static_cast<size_t>(t) * K + 512 * (kp0 + u) + 16 * lane);
            a = __ldcs(src);
            b = __ldcs(src + 1);
        }
        v[u][0] = a.x, v[u][1] = a.y, v[u][2] = a.z, v[u][3] = a.w;
        v[u][4] = b.x, v[u][5] = b.y, v[u][6] = b.z, v[u][7] = b.w;
    }
    uint32_t c[U][4], word[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max_u16x2(m, v[u][i] & 0x7FFF7FFFu);
        m = max(m & 0xFFFFu, m >> 16);
#pragma unroll
        for (int off = 1; off < 8; off <<= 1) m = max(m, __shfl_xor_sync(FULL, m, off));
        const int e = block_scale_exponent(m << 16);
        const uint32_t s2 = static_cast<uint32_t>(127 - e) * 0x00800080u;      // 2^-e as a BF16 pair
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t y0 = mul_bf16x2(v[u][2 * i], s2), y1 = mul_bf16x2(v[u][2 * i + 1], s2);
            c[u][i] = prmt(cvt_e4m3x2(bf16_lo(y0), bf16_hi(y0)), cvt_e4m3x2(bf16_lo(y1), bf16_hi(y1)), 0x5410u);
        }
        const uint32_t byte = valid[u] ? static_cast<uint32_t>(e + 127) : 0u;
        word[u] = __shfl_sync(FULL, byte, 0) | (__shfl_sync(FULL, byte, 8) << 8) | (__shfl_sync(FULL, byte, 16) << 16) |
                  (__shfl_sync(FULL, byte, 24) << 24);
    }
    if (p >= 0) {        // lane j: the scale words of the token's j-th row
        const int g = p / rows;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (kp0 + u < Kp)
                sf[(static_cast<size_t>(g) * Kp + kp0 + u) * rows_al + (p - g * rows)] = static_cast<int32_t>(word[u]);
    }
    uint8_t* dst = q + 512 * kp0 + 16 * lane;
    for (int j = 0; j < k; ++j) {
        const int r = __shfl_sync(FULL, p, j);
        if (r < 0) continue;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (valid[u])
                __stcs(reinterpret_cast<uint4*>(dst + static_cast<size_t>(r) * K + 512 * u),
                       make_uint4(c[u][0], c[u][1], c[u][2], c[u][3]));
    }
}

// Rows copied as they are (n16 16-byte units each).
__global__ void __launch_bounds__(32 * DISPATCH_WARPS)
    dispatch_copy_kernel(const uint4* __restrict__ x, const int32_t* __restrict__ pos,
                         const int32_t* __restrict__ m_indices, uint4* __restrict__ out, int T, int k, int n16,
                         int chunks, int rows, int pad_chunks) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int lead = m_indices ? rows / PAD_ROWS * pad_chunks : 0;      // padding units
    const long long unit = static_cast<long long>(blockIdx.x) * DISPATCH_WARPS + (threadIdx.x >> 5) - lead;
    if (unit >= static_cast<long long>(T) * chunks) return;
    if (unit < 0) {
        const int at = static_cast<int>(unit + lead);
        const int u = at / pad_chunks, c = at - u * pad_chunks;
        const uint32_t bits = padding_bits(m_indices, u, lane);
        if (bits != 0u) zero_rows(bits, out, u, n16, c, pad_chunks, lane);
        return;
    }
    const long long owner = unit / chunks;                    // token
    const int i0 = 64 * static_cast<int>(unit - owner * chunks) + lane, i1 = i0 + 32;
    int p = lane < k ? __ldg(pos + static_cast<size_t>(owner) * k + lane) : -1;
    if (p >= rows) p = -1;
    const uint4* src = x + static_cast<size_t>(owner) * n16;
    uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
    if (i0 < n16) a = __ldcs(src + i0);
    if (i1 < n16) b = __ldcs(src + i1);
    for (int j = 0; j < k; ++j) {
        const int r = __shfl_sync(FULL, p, j);
        if (r < 0) continue;
        uint4* dst = out + static_cast<size_t>(r) * n16;
        if (i0 < n16) __stcs(dst + i0, a);
        if (i1 < n16) __stcs(dst + i1, b);
    }
}

// ---------------------------------------------------------------------------------------------
// Combine
// ---------------------------------------------------------------------------------------------
// One 16-byte unit of a row as FP32 values (8 of BF16, 4 of FP32), and back.
template <bool F32>
__device__ __forceinline__ void unpack16(const uint4& v, float (&f)[F32 ? 4 : 8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (F32) {
            f[i] = __uint_as_float(w[i]);
        } else {
            f[2 * i] = bf16_lo(w[i]);
            f[2 * i + 1] = bf16_hi(w[i]);
        }
    }
}

template <bool F32>
__device__ __forceinline__ uint4 pack16(const float (&f)[F32 ? 4 : 8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (F32) w[i] = __float_as_uint(f[i]);
        else w[i] = bf16x2(f[2 * i], f[2 * i + 1]);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int COMBINE_WARPS = 8;
constexpr int COMBINE_FEW = 152 * 32;    // warps that hold 64 registers each on all SMs at once

// One warp per token and U x 512 bytes of the row; the k rows' units are summed in j order in FP32 (an output
// element belongs to one thread: no atomics, no order to vary).  Up to ROWS x U units are in flight per lane (the
// FP32 kernel for eight rows compiles to 34 registers, so that some of its loads wait for others' values).
// Bound by HBM: 16384 tokens x 8, N 7168 BF16, 2.1 GB in 303 us, 6.9 TB/s.
template <bool F32, int ROWS, int U>
__global__ void __launch_bounds__(32 * COMBINE_WARPS)
    combine_kernel(const uint4* __restrict__ yp, const int32_t* __restrict__ pos, const float* __restrict__ w,
                   const uint4* __restrict__ residual, uint4* __restrict__ y, int T, int k, int n16, int chunks,
                   int rows) {
    constexpr int V = F32 ? 4 : 8;
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long unit = static_cast<long long>(blockIdx.x) * COMBINE_WARPS + (threadIdx.x >> 5);
    const long long t = unit / chunks;
    if (t >= T) return;
    const int i0 = 32 * U * static_cast<int>(unit - t * chunks) + lane;
    int p = -1;
    float wt = 0.0f;
    if (lane < k) {
        p = __ldg(pos + t * k + lane);
        if (p >= rows) p = -1;
        wt = w ? __ldg(w + t * k + lane) : 1.0f;
    }
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    uint4 res[U];
#pragma unroll
    for (int u = 0; u < U; ++u) res[u] = residual && i0 + 32 * u < n16 ? __ldcs(residual + t * n16 + i0 + 32 * u) : none;
    float acc[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) unpack16<F32>(res[u], acc[u]);
    for (int j0 = 0; j0 < k; j0 += ROWS) {
        uint4 v[ROWS][U];
        int pj[ROWS];
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            pj[j] = __shfl_sync(FULL, p, (j0 + j) & 31);      // lanes at or past k hold -1
            if (j0 + j >= k) pj[j] = -1;
#pragma unroll
            for (int u = 0; u < U; ++u)
                v[j][u] = pj[j] >= 0 && i0 + 32 * u < n16 ? __ldcs(yp + static_cast<size_t>(pj[j]) * n16 + i0 + 32 * u) : none;
        }
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            const float wj = __shfl_sync(FULL, wt, (j0 + j) & 31);
            if (pj[j] < 0) continue;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float f[V];
                unpack16<F32>(v[j][u], f);
#pragma unroll
                for (int c = 0; c < V; ++c) acc[u][c] = fmaf(wj, f[c], acc[u][c]);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (i0 + 32 * u < n16) __stcs(y + t * n16 + i0 + 32 * u, pack16<F32>(acc[u]));
}

// Gradients of the weighted sum: one CTA per token reads dy once and each of the token's rows
// once, writes w_j dy to that row of dyp, and sums dy * yp over the row for dw_j: per thread,
// then over the warp, then over the warps in order (no atomics).  The first CTAs write
// the padding rows, as in the dispatch.  KM: the most choices per token that are held.
// Bound by HBM (reads and writes in equal parts).
constexpr int CB_WARP_TOKENS = 2048;   // tokens from which one warp takes a token
template <bool F32, int KM, int THREADS>
__global__ void __launch_bounds__(THREADS)
    combine_backward_kernel(const uint4* __restrict__ dy, const uint4* __restrict__ yp, const int32_t* __restrict__ pos,
                            const int32_t* __restrict__ m_indices, const float* __restrict__ w, uint4* __restrict__ dyp,
                            float* __restrict__ dw, int T, int k, int n16, int rows, int pad_chunks) {
    constexpr int V = F32 ? 4 : 8;
    __shared__ float part[THREADS / 32][KM];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned lead = gridDim.x - static_cast<unsigned>(T);             // CTAs of padding units
    if (blockIdx.x < lead) {
        const int at = static_cast<int>(blockIdx.x) * (THREADS / 32) + warp;
        const int u = at / pad_chunks, c = at - u * pad_chunks;
        if (u >= rows / PAD_ROWS) return;
        const uint32_t bits = padding_bits(m_indices, u, lane);
        if (bits != 0u) zero_rows(bits, dyp, u, n16, c, pad_chunks, lane);
        return;
    }
    const size_t t = blockIdx.x - lead;
    int p = -1;
    float wt = 0.0f;
    if (lane < k) {
        p = __ldg(pos + t * k + lane);
        if (p >= rows) p = -1;
        wt = __ldg(w + t * k + lane);
    }
    float acc[KM];
#pragma unroll
    for (int j = 0; j < KM; ++j) acc[j] = 0.0f;
    // (whole warps walk the row together: the shuffles below need every lane)
    for (int i0 = 32 * warp; i0 < n16; i0 += THREADS) {
        const int i = i0 + lane;
        const bool in = i < n16;
        float d[V];
        unpack16<F32>(in ? __ldcs(dy + t * n16 + i) : make_uint4(0u, 0u, 0u, 0u), d);
#pragma unroll
        for (int j0 = 0; j0 < KM; j0 += 8) {
            constexpr int B = KM < 8 ? KM : 8;
            uint4 v[B];
            int pj[B];
#pragma unroll
            for (int j = 0; j < B; ++j) {
                pj[j] = __shfl_sync(FULL, p, j0 + j);       // -1 at or past k
                v[j] = pj[j] >= 0 && in ? __ldcs(yp + static_cast<size_t>(pj[j]) * n16 + i) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int j = 0; j < B; ++j) {
                const float wj = __shfl_sync(FULL, wt, j0 + j);
                if (pj[j] < 0 || !in) continue;
                float f[V], o[V];
                unpack16<F32>(v[j], f);
#pragma unroll
                for (int c = 0; c < V; ++c) {
                    acc[j0 + j] = fmaf(d[c], f[c], acc[j0 + j]);
                    o[c] = wj * d[c];
                }
                __stcs(dyp + static_cast<size_t>(pj[j]) * n16 + i, pack16<F32>(o));
            }
        }
    }
#pragma unroll
    for (int j = 0; j < KM; ++j) {
        const float s = warp_sum(acc[j]);
        if (lane == 0) part[warp][j] = s;
    }
    __syncthreads();
    if (threadIdx.x < static_cast<unsigned>(k)) {
        float s = 0.0f;
        for (unsigned q = 0; q < THREADS / 32; ++q) s += part[q][threadIdx.x];
        dw[t * k + threadIdx.x] = s;
    }
}

}  // namespace

// Logits per lane of the router kernels: the power of two that covers E experts.
static int route_width(int E) {
    int nv = 1;
    while (32 * nv < E) nv *= 2;
    return nv;
}

cudaError_t launch_moe_route(const void* logits, int32_t* topk_idx, float* topk_w, int T, int E, int k, int f32,
                             int sigmoid, int renorm, float scale, int pdl, cudaStream_t stream) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    const int nv = route_width(E);
    int slot = 1;
    while (slot < k) slot *= 2;
    // A token per warp up to ROUTE_CTAS, then up to 32 / slot, whose last steps are done together (32768 x 256,
    // k 8: four tokens 10.0 us, two 10.6, one 13.0).
    const int held = ROUTE_WARPS * ROUTE_CTAS;
    const int group = std::min(32 / slot, (T - 1) / held + 1);
    const long long units = (static_cast<long long>(T) + group - 1) / group;
    launch_cfg(cfg, attr, (units + ROUTE_WARPS - 1) / ROUTE_WARPS, 32 * ROUTE_WARPS, pdl, stream);
    const int vec = logits_vec(nv, f32, E);
    auto go = [&](auto kernel) {
        return cudaLaunchKernelEx(&cfg, kernel, logits, topk_idx, topk_w, T, E, k, sigmoid, renorm, scale, vec, group, slot);
    };
    if (nv <= 1) return f32 ? go(route_kernel<1, true>) : go(route_kernel<1, false>);
    if (nv <= 2) return f32 ? go(route_kernel<2, true>) : go(route_kernel<2, false>);
    if (nv <= 4) return f32 ? go(route_kernel<4, true>) : go(route_kernel<4, false>);
    if (nv <= 8) return f32 ? go(route_kernel<8, true>) : go(route_kernel<8, false>);
    if (nv <= 16) return f32 ? go(route_kernel<16, true>) : go(route_kernel<16, false>);
    return f32 ? go(route_kernel<32, true>) : go(route_kernel<32, false>);
}

cudaError_t launch_moe_route_backward(const void* logits, const int32_t* topk_idx, const float* dw, void* dlogits,
                                      int T, int E, int k, int f32, int sigmoid, int renorm, float scale, int pdl,
                                      cudaStream_t stream) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    launch_cfg(cfg, attr, (static_cast<long long>(T) + ROUTE_WARPS - 1) / ROUTE_WARPS, 32 * ROUTE_WARPS, pdl, stream);
    const int nv = route_width(E);
    const int vec = logits_vec(nv, f32, E);
    auto go = [&](auto kernel) {
        return cudaLaunchKernelEx(&cfg, kernel, logits, topk_idx, dw, dlogits, T, E, k, sigmoid, renorm, scale, vec);
    };
    if (nv <= 1) return f32 ? go(route_backward_kernel<1, true>) : go(route_backward_kernel<1, false>);
    if (nv <= 2) return f32 ? go(route_backward_kernel<2, true>) : go(route_backward_kernel<2, false>);
    if (nv <= 4) return f32 ? go(route_backward_kernel<4, true>) : go(route_backward_kernel<4, false>);
    if (nv <= 8) return f32 ? go(route_backward_kernel<8, true>) : go(route_backward_kernel<8, false>);
    if (nv <= 16) return f32 ? go(route_backward_kernel<16, true>) : go(route_backward_kernel<16, false>);
    return f32 ? go(route_backward_kernel<32, true>) : go(route_backward_kernel<32, false>);
}

// f(kernel) of the sort kernel for G experts: the bits of an expert's index, rounded up to 4, 6, 8 or 12.
template <bool CLUSTER, class F>
static cudaError_t with_sort_kernel(int G, const F& f) {
    if (G <= 16) return f(sort_kernel<CLUSTER, 4>);
    if (G <= 64) return f(sort_kernel<CLUSTER, 6>);
    if (G <= 256) return f(sort_kernel<CLUSTER, 8>);
    return f(sort_kernel<CLUSTER, 12>);
}

// *sort_cluster: CTAs of the sort's cluster on this device, 16 where it takes clusters beyond the portable size, else 8.
cudaError_t prepare_moe(int max_smem, int* sort_cluster) {
    auto smem = [&](auto kernel) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem);
    };
    auto wide = [&](auto kernel) { return cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1); };
    cudaError_t e;
    for (int G : {16, 64, 256, 4096}) {
        if ((e = with_sort_kernel<false>(G, smem)) != cudaSuccess) return e;
        if ((e = with_sort_kernel<true>(G, smem)) != cudaSuccess) return e;
        if ((e = with_sort_kernel<true>(G, wide)) != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(16, 1, 1);
    cfg.blockDim = dim3(1024, 1, 1);
    cfg.dynamicSmemBytes = max_smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 16;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, sort_kernel<true, 12>, &cfg) != cudaSuccess) cudaGetLastError();
    *sort_cluster = clusters > 0 ? 16 : 8;
    return cudaSuccess;
}

cudaError_t launch_moe_sort(const int32_t* idx, int32_t* pos, int32_t* m_indices, int32_t* counts, int32_t* ks, int n,
                            int G, int rows, int max_m, int cluster, int pdl, cudaStream_t stream) {
    SortArgs a{idx, pos, m_indices, counts, ks, n, G, rows, max_m, 0};
    const int warps = sort_warps(G);
    // One CTA for decode batches, else a cluster.  Measured (us, one CTA / cluster of 16): 64 experts, 512
    // slots 4.1 / 4.2, 2048 slots 5.2 / 4.9, 16384 slots 13.7 / 4.9, 262144 slots 163 / 14.7; 256 experts (33024
    // rows to fill) 512 slots 7.7 / 4.9.
    const int ctas = n <= 1024 && rows <= 10240 ? 1 : cluster;
    const long long per = (static_cast<long long>(n) + ctas * warps - 1) / (ctas * warps);
    a.share = static_cast<int>((per + 31) / 32 * 32);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, 1, 1);
    cfg.blockDim = dim3(32 * warps, 1, 1);
    cfg.dynamicSmemBytes = sort_smem(G);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int na = 0;
    if (ctas > 1) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = ctas;
        attr[na].val.clusterDim.y = 1;
        attr[na].val.clusterDim.z = 1;
        ++na;
    }
    if (pdl) {
        attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[na].val.programmaticStreamSerializationAllowed = 1;
        ++na;
    }
    cfg.attrs = attr;
    cfg.numAttrs = na;
    auto launch = [&](auto kernel) { return cudaLaunchKernelEx(&cfg, kernel, a); };
    return ctas > 1 ? with_sort_kernel<true>(G, launch) : with_sort_kernel<false>(G, launch);
}

// Column ranges that the padding rows are split into: 1 KB each at the least, and no more than give a few
// thousand units (a decode batch's padding is most of its rows; a prefill's 16-row units suffice).
static int padding_chunks(int rows, int n16) {
    return std::max(1, std::min((n16 + 63) / 64, 4096 * PAD_ROWS / std::max(rows, 1)));
}

cudaError_t launch_moe_dispatch_fp8(const void* x, const int32_t* pos, const int32_t* m_indices, void* q, int32_t* sf,
                                    int T, int k, int K, int G, int rows, int pdl, cudaStream_t stream) {
    const int Kb = K / 128, Kp = (Kb + 3) / 4, rows_al = (rows + 3) / 4 * 4;
    const int pad_chunks = padding_chunks(rows, K / 16);
    // Two spans per warp, and so twice the loads in flight, where few stores follow each load or the spans fill the GPU
    // many times over (us, two / one: 16384 tokens x 1, K 7168 62 / 85; 16384 x 2, K 4096 46 / 57; 16384 x 8,
    // K 7168 190 / 192; 4000 x 3, K 7168 28.7 / 31.3, x 4 30.4 / 31.0, x 5 37.5 / 37.5, x 8 57 / 54; 64 x 8, K 7168
    // 5.1 / 4.5).
    const long long spans = static_cast<long long>(T) * Kp;
    const int U = Kp > 1 && (spans > 65536 || (k <= 4 && spans > 152 * 64)) ? DISPATCH_U : 1;
    const long long units = static_cast<long long>(T) * ((Kp + U - 1) / U) + (m_indices ? static_cast<long long>(rows / PAD_ROWS) * pad_chunks : 0);
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    const cudaError_t e = launch_cfg(cfg, attr, (units + DISPATCH_WARPS - 1) / DISPATCH_WARPS, 32 * DISPATCH_WARPS, pdl, stream);
    if (e != cudaSuccess) return e;
    auto go = [&](auto kernel) {
        return cudaLaunchKernelEx(&cfg, kernel, static_cast<const uint16_t*>(x), pos, m_indices, static_cast<uint8_t*>(q), sf,
                                  T, k, K, Kb, Kp, G, rows, rows_al, pad_chunks);
    };
    return U == 1 ? go(dispatch_fp8_kernel<1>) : go(dispatch_fp8_kernel<DISPATCH_U>);
}

cudaError_t launch_moe_dispatch(const void* x, const int32_t* pos, const int32_t* m_indices, void* out, int T, int k,
                                int n16, int rows, int pdl, cudaStream_t stream) {
    const int chunks = (n16 + 63) / 64;
    const int pad_chunks = padding_chunks(rows, n16);
    const long long units = static_cast<long long>(T) * chunks + (m_indices ? static_cast<long long>(rows / PAD_ROWS) * pad_chunks : 0);
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    const cudaError_t e = launch_cfg(cfg, attr, (units + DISPATCH_WARPS - 1) / DISPATCH_WARPS, 32 * DISPATCH_WARPS, pdl, stream);
    if (e != cudaSuccess) return e;
    return cudaLaunchKernelEx(&cfg, dispatch_copy_kernel, static_cast<const uint4*>(x), pos, m_indices,
                              static_cast<uint4*>(out), T, k, n16, chunks, rows, pad_chunks);
}

cudaError_t launch_moe_combine(const void* yp, const int32_t* pos, const float* w, const void* residual, void* y, int T,
                               int k, int n16, int rows, int f32, int pdl, cudaStream_t stream) {
    // Units in flight per lane: four rows, or as many of fewer rows (16384 tokens: k 1, N 7168, residual 219 us
    // with places for eight rows, 145 for four; k 2, N 4096 106 and 73; k 8, N 7168 310 and 303).
    const int units_per_row = k == 1 ? 4 : k == 2 ? 2 : 1;
    const int chunks = (n16 + 32 * units_per_row - 1) / (32 * units_per_row);
    const long long units = static_cast<long long>(T) * chunks;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    const cudaError_t e = launch_cfg(cfg, attr, (units + COMBINE_WARPS - 1) / COMBINE_WARPS, 32 * COMBINE_WARPS, pdl, stream);
    if (e != cudaSuccess) return e;
    auto go = [&](auto kernel) {
        return cudaLaunchKernelEx(&cfg, kernel, static_cast<const uint4*>(yp), pos, w,
                                  static_cast<const uint4*>(residual), static_cast<uint4*>(y), T, k, n16, chunks, rows);
    };
    if (k == 1) return f32 ? go(combine_kernel<true, 1, 4>) : go(combine_kernel<false, 1, 4>);
    if (k == 2) return f32 ? go(combine_kernel<true, 2, 2>) : go(combine_kernel<false, 2, 2>);
    // (a batch that fills the GPU less than once: one round trip for up to eight rows; 64 tokens x 8, N 7168 3.3 us
    // instead of 3.8)
    if (k > 4 && units <= COMBINE_FEW) return f32 ? go(combine_kernel<true, 8, 1>) : go(combine_kernel<false, 8, 1>);
    return f32 ? go(combine_kernel<true, 4, 1>) : go(combine_kernel<false, 4, 1>);
}

cudaError_t launch_moe_combine_backward(const void* dy, const void* yp, const int32_t* pos, const int32_t* m_indices,
                                        const float* w, void* dyp, float* dw, int T, int k, int n16, int rows, int f32,
                                        int pdl, cudaStream_t stream) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    // A token per warp (no warp waits for another at the end of a row) once the tokens fill the GPU, else a
    // token per eight warps.  us, 32 / 256 threads: 8191 tokens x 4, N 4096 98 / 108; 4096 x 8, N 2048 49 / 53;
    // 2048 x 8, N 7168 91 / 92; 1000 x 8, N 7168 59 / 52; 300 x 4, N 4096 27 / 10; 64 x 8, N 7168 43 / 16.
    const int threads = T >= CB_WARP_TOKENS ? 32 : 256;
    const int pad_chunks = padding_chunks(rows, n16);
    const long long pad_units = m_indices ? static_cast<long long>(rows / PAD_ROWS) * pad_chunks : 0;
    const long long padding = (pad_units + threads / 32 - 1) / (threads / 32);
    const cudaError_t e = launch_cfg(cfg, attr, T + padding, threads, pdl, stream);
    if (e != cudaSuccess) return e;
    auto go = [&](auto kernel) {
        return cudaLaunchKernelEx(&cfg, kernel, static_cast<const uint4*>(dy), static_cast<const uint4*>(yp), pos,
                                  m_indices, w, static_cast<uint4*>(dyp), dw, T, k, n16, rows, pad_chunks);
    };
    auto pick = [&](auto f, auto km) {
        constexpr bool F = decltype(f)::value;
        constexpr int KM = decltype(km)::value;
        return threads == 32 ? go(combine_backward_kernel<F, KM, 32>) : go(combine_backward_kernel<F, KM, 256>);
    };
    auto by_choices = [&](auto f) {
        if (k <= 4) return pick(f, std::integral_constant<int, 4>());
        if (k <= 8) return pick(f, std::integral_constant<int, 8>());
        return pick(f, std::integral_constant<int, 32>());
    };
    return f32 ? by_choices(std::true_type()) : by_choices(std::false_type());
}

}  // namespace dg

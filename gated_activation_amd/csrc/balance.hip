// The router's balance loss with per-expert counts, and its gradient, gfx950.
//
// Over the n tokens that count (below the live count, not masked), with
// p_t = softmax(logits_t) over E experts and the k experts chosen for each:
//     counts_e = number of (t, j) with index[t, j] = e
//     loss     = c E / (k n) sum_e counts_e P_e,   P_e = (1 / n) sum_t p_te
//     dlogits_te = dloss c E / (k n^2) p_te (counts_e - sum_j counts_j p_tj)
// (counts are constants of the gradient; the loss is c where tokens and
// probabilities are spread evenly).  offsets is the running sum of counts:
// expert e's rows in a buffer sorted by expert, offsets[E] its live rows.
// A token whose logits are all -inf has p = 0.
//
// Both passes are bound by reading the logits (the gradient needs every count
// first, so they are read twice), and at small sizes by the launches.  A token
// is held by L lanes, eight experts each (two times eight above 512 experts),
// so a lane owns the same experts for every token and adds their p in
// registers.  Workgroups take contiguous runs of tokens and count indices in
// LDS; with one workgroup the results are formed in the same launch, else
// every workgroup leaves its sums and one workgroup adds them in order.
// Integer counts and a fixed order of the fp32 sums: the same bits every time.
#include "ga_internal.h"
#include "ga_train.h"

namespace ga {

namespace {

constexpr int BAL_BLOCK = 256;
constexpr int FINISH_BLOCK = 1024;

__device__ __forceinline__ float lanes_max(float v, int lanes) {
    for (int s = 1; s < lanes; s <<= 1) v = __builtin_fmaxf(v, __shfl_xor(v, s));
    return v;
}

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
    for (int s = 1; s < lanes; s <<= 1) v += __shfl_xor(v, s);
    return v;
}

// Softmax over E experts of one token, held by L lanes of V octets; lanes past
// E get 0.  A NaN or +inf logit makes the token's probabilities NaN.
template <int DT, int L, int V>
__device__ __forceinline__ void token_softmax(const typename Elem<DT>::storage *row, uint32_t lane, int E,
                                              float (&p)[V][8]) {
    float top = -__builtin_inff();
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (int)(v * L + lane) * 8;
        Oct<DT> o;
        oct_load<DT, false>(o, row + c, E - c);
        oct_unpack<DT>(o, p[v]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (c + e >= E) p[v][e] = -__builtin_inff();
            top = __builtin_fmaxf(top, p[v][e]);
        }
    }
    top = lanes_max(top, L);
    const float base = top == -__builtin_inff() ? 0.0f : top;
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            p[v][e] = __builtin_amdgcn_exp2f((p[v][e] - base) * LOG2_E);
            sum += p[v][e];
        }
    }
    sum = lanes_sum(sum, L);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) p[v][e] *= inv;
}

// counts and sums of E experts (in LDS) -> loss, counts, offsets, tokens.
// All threads of the workgroup call it, after a barrier.
template <int BLOCK>
__device__ void finish(const int32_t *counts, const float *sums, int32_t tokens, int E, int k, float coefficient,
                       float *loss, int32_t *out_counts, int32_t *out_offsets, int32_t *out_tokens) {
    __shared__ float loss_part[BLOCK / 64];
    __shared__ int32_t count_part[BLOCK / 64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    // each thread owns PER consecutive experts
    const int per = (E + BLOCK - 1) / BLOCK, e0 = (int)threadIdx.x * per;
    int32_t own = 0;
    float dot = 0.0f;
    for (int i = 0; i < per; ++i) {
        if (e0 + i < E) {
            own += counts[e0 + i];
            dot = __builtin_fmaf((float)counts[e0 + i], sums[e0 + i], dot);
        }
    }
    int32_t run = own;  // inclusive running sum over the wave
    for (int s = 1; s < 64; s <<= 1) {
        const int32_t o = __shfl_up(run, s);
        if (lane >= s) run += o;
    }
    dot = wave_sum(dot);
    if (lane == 63) count_part[wave] = run;
    if (lane == 0) loss_part[wave] = dot;
    __syncthreads();
    int32_t before = run - own;
    float total = 0.0f;
    for (int w = 0; w < BLOCK / 64; ++w) {
        if (w < wave) before += count_part[w];
        total += loss_part[w];
    }
    for (int i = 0; i < per; ++i) {
        if (e0 + i < E) {
            out_counts[e0 + i] = counts[e0 + i];
            out_offsets[e0 + i] = before;
            before += counts[e0 + i];
            if (e0 + i == E - 1) out_offsets[E] = before;
        }
    }
    if (threadIdx.x == 0) {
        const float n = (float)tokens;
        *loss = tokens == 0 ? 0.0f : coefficient * ((float)E / ((float)k * n)) * (total / n);
        *out_tokens = tokens;
    }
}

template <int DT, int L, int V, typename I>
__global__ __launch_bounds__(BAL_BLOCK) void sums_kernel(
    const typename Elem<DT>::storage *__restrict__ logits, const I *__restrict__ index, const uint8_t *__restrict__ mask,
    float *__restrict__ part_sums, int32_t *__restrict__ part_counts, int32_t *__restrict__ part_tokens, int32_t rows,
    int32_t E, int32_t k, float coefficient, const int32_t *__restrict__ live, float *loss, int32_t *out_counts,
    int32_t *out_offsets, int32_t *out_tokens) {
    constexpr int WAVES = BAL_BLOCK / 64, GROUPS = BAL_BLOCK / L, WIDTH = L * V * 8;
    __shared__ float sums[WAVES][WIDTH];
    __shared__ int32_t counts[WIDTH];
    __shared__ int32_t tokens[WAVES];
    const uint32_t n = live != nullptr ? (uint32_t)clamp_live(live, rows) : (uint32_t)rows;
    // this workgroup's run of tokens
    const uint32_t each = ((uint32_t)rows + gridDim.x - 1) / gridDim.x;
    const uint64_t begin64 = (uint64_t)blockIdx.x * each, end64 = begin64 + each;
    const uint32_t begin = begin64 < n ? (uint32_t)begin64 : n, end = end64 < n ? (uint32_t)end64 : n;
    for (int i = threadIdx.x; i < WIDTH; i += BAL_BLOCK) counts[i] = 0;
    __syncthreads();
    // indices, flat over the run
    const uint64_t first = (uint64_t)begin * k, past = (uint64_t)end * k;
    for (uint64_t i = first + threadIdx.x; i < past; i += BAL_BLOCK) {
        const I e = index[i];
        if (e >= 0 && e < (I)E && (mask == nullptr || mask[begin + (uint32_t)((i - first) / (uint32_t)k)] != 0))
            atomicAdd(&counts[(int)e], 1);
    }
    const uint32_t lane = threadIdx.x % L;
    float acc[V][8];
    int32_t used = 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[v][e] = 0.0f;
    // every lane of a wavefront makes the same number of rounds (shuffles)
    for (uint32_t base = begin; base < end; base += GROUPS) {
        const uint32_t t = base + threadIdx.x / L;
        const bool use = t < end && (mask == nullptr || mask[t] != 0);
        float p[V][8];
        token_softmax<DT, L, V>(logits + (size_t)(t < end ? t : base) * E, lane, E, p);
        if (use) {
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[v][e] += p[v][e];
            used += lane == 0;
        }
    }
    const int wave = threadIdx.x >> 6, wl = threadIdx.x & 63;
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float a = acc[v][e];
            for (int s = L; s < 64; s <<= 1) a += __shfl_xor(a, s);
            if (wl < L) sums[wave][(v * L + wl) * 8 + e] = a;
        }
    }
    for (int s = 1; s < 64; s <<= 1) used += __shfl_xor(used, s);
    if (wl == 0) tokens[wave] = used;
    __syncthreads();
    for (int i = threadIdx.x; i < E; i += BAL_BLOCK) {
        float a = sums[0][i];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) a += sums[w][i];
        sums[0][i] = a;
        if (gridDim.x > 1) {
            part_sums[(size_t)blockIdx.x * E + i] = a;
            part_counts[(size_t)blockIdx.x * E + i] = counts[i];
        }
    }
    int32_t total = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) total += tokens[w];
    if (gridDim.x > 1) {
        if (threadIdx.x == 0) part_tokens[blockIdx.x] = total;
        return;
    }
    __syncthreads();
    finish<BAL_BLOCK>(counts, sums[0], total, E, k, coefficient, loss, out_counts, out_offsets, out_tokens);
}

// The workgroups' sums added in order: the E columns by slices of the groups.
__global__ __launch_bounds__(FINISH_BLOCK) void finish_kernel(const float *__restrict__ part_sums,
                                                              const int32_t *__restrict__ part_counts,
                                                              const int32_t *__restrict__ part_tokens, int32_t groups,
                                                              int32_t E, int32_t k, float coefficient, float *loss,
                                                              int32_t *out_counts, int32_t *out_offsets,
                                                              int32_t *out_tokens) {
    __shared__ float sums[FINISH_BLOCK];
    __shared__ int32_t counts[FINISH_BLOCK];
    __shared__ int32_t tokens[FINISH_BLOCK / 64];
    // columns in a power of two, so that whole slices fit the workgroup
    int width = 1;
    while (width < E) width <<= 1;
    const int slices = FINISH_BLOCK / width;
    const int col = (int)threadIdx.x & (width - 1), slice = (int)threadIdx.x / width;
    float a = 0.0f;
    int32_t c = 0;
    if (col < E) {
#pragma unroll 8
        for (int g = slice; g < groups; g += slices) {
            a += part_sums[(size_t)g * E + col];
            c += part_counts[(size_t)g * E + col];
        }
    }
    sums[threadIdx.x] = a;
    counts[threadIdx.x] = c;
    int32_t used = 0;
    for (int g = threadIdx.x; g < groups; g += FINISH_BLOCK) used += part_tokens[g];
    for (int s = 1; s < 64; s <<= 1) used += __shfl_xor(used, s);
    if ((threadIdx.x & 63) == 0) tokens[threadIdx.x >> 6] = used;
    __syncthreads();
    if (slice == 0 && col < E) {
        for (int s = 1; s < slices; ++s) {
            a += sums[s * width + col];
            c += counts[s * width + col];
        }
        sums[col] = a;  // slot 0 of this column: read by this thread alone
        counts[col] = c;
    }
    __syncthreads();
    int32_t total = 0;
    for (int w = 0; w < FINISH_BLOCK / 64; ++w) total += tokens[w];
    finish<FINISH_BLOCK>(counts, sums, total, E, k, coefficient, loss, out_counts, out_offsets, out_tokens);
}

template <int DT, int L, int V>
__global__ __launch_bounds__(BAL_BLOCK) void gradient_kernel(
    const typename Elem<DT>::storage *__restrict__ logits, const uint8_t *__restrict__ mask,
    const int32_t *__restrict__ counts, const int32_t *__restrict__ offsets, const int32_t *__restrict__ tokens,
    const float *__restrict__ dloss, typename Elem<DT>::storage *__restrict__ dlogits, int32_t rows, int32_t E, int32_t k,
    float coefficient, const int32_t *__restrict__ live) {
    constexpr int GROUPS = BAL_BLOCK / L;
    const uint32_t n = live != nullptr ? (uint32_t)clamp_live(live, rows) : (uint32_t)rows;
    const uint32_t lane = threadIdx.x % L;
    const float m = (float)*tokens;
    const float factor = m == 0.0f ? 0.0f : *dloss * coefficient * ((float)E / ((float)k * m)) / m;
    // sum_j p_j = 1: taken from (about) their mean, the counts cancel less
    const int32_t middle = offsets[E] / E;
    float w[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = (int)(v * L + lane) * 8 + e;
            w[v][e] = c < E ? (float)(counts[c] - middle) : 0.0f;
        }
    }
    for (uint32_t base = blockIdx.x * GROUPS; base < n; base += gridDim.x * GROUPS) {
        const uint32_t t = base + threadIdx.x / L;
        const bool in = t < n;
        float p[V][8];
        token_softmax<DT, L, V>(logits + (size_t)(in ? t : base) * E, lane, E, p);
        float dot = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < 8; ++e) dot = __builtin_fmaf(p[v][e], w[v][e], dot);
        dot = lanes_sum(dot, L);
        if (!in) continue;
        const bool use = mask == nullptr || mask[t] != 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (int)(v * L + lane) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) p[v][e] = use ? factor * p[v][e] * (w[v][e] - dot) : 0.0f;
            if (c < E) oct_store<DT>(dlogits + (size_t)t * E + c, p[v], E - c);
        }
    }
}

struct Sums {
    const void *logits, *index;
    bool wide_index;
    const uint8_t *mask;
    float *part_sums;
    int32_t *part_counts, *part_tokens;
    int32_t rows, E, k;
    float coefficient;
    const int32_t *live;
    int groups;
    float *loss;
    int32_t *counts, *offsets, *tokens;
    hipStream_t stream;
};

template <int DT, int L, int V>
hipError_t sums_as(const Sums &a) {
    using S = typename Elem<DT>::storage;
    if (a.wide_index)
        sums_kernel<DT, L, V, int64_t><<<dim3((uint32_t)a.groups), BAL_BLOCK, 0, a.stream>>>(
            (const S *)a.logits, (const int64_t *)a.index, a.mask, a.part_sums, a.part_counts, a.part_tokens, a.rows,
            a.E, a.k, a.coefficient, a.live, a.loss, a.counts, a.offsets, a.tokens);
    else
        sums_kernel<DT, L, V, int32_t><<<dim3((uint32_t)a.groups), BAL_BLOCK, 0, a.stream>>>(
            (const S *)a.logits, (const int32_t *)a.index, a.mask, a.part_sums, a.part_counts, a.part_tokens, a.rows,
            a.E, a.k, a.coefficient, a.live, a.loss, a.counts, a.offsets, a.tokens);
    return hipGetLastError();
}

struct Gradient {
    const void *logits;
    const uint8_t *mask;
    const int32_t *counts, *offsets, *tokens;
    const float *dloss;
    void *dlogits;
    int32_t rows, E, k;
    float coefficient;
    const int32_t *live;
    int cus;
    hipStream_t stream;
};

template <int DT, int L, int V>
hipError_t gradient_as(const Gradient &a) {
    using S = typename Elem<DT>::storage;
    constexpr int GROUPS = BAL_BLOCK / L;
    const int64_t need = ((int64_t)a.rows + GROUPS - 1) / GROUPS, most = (int64_t)a.cus * 8;
    gradient_kernel<DT, L, V><<<dim3((uint32_t)(need < most ? need : most)), BAL_BLOCK, 0, a.stream>>>(
        (const S *)a.logits, a.mask, a.counts, a.offsets, a.tokens, a.dloss, (S *)a.dlogits, a.rows, a.E, a.k,
        a.coefficient, a.live);
    return hipGetLastError();
}

// The lanes that hold a token, by E: eight experts a lane up to 512.
#define GA_BY_EXPERTS(FN, DT, E, A)                 \
    ((E) <= 8     ? FN<DT, 1, 1>(A)                 \
     : (E) <= 16  ? FN<DT, 2, 1>(A)                 \
     : (E) <= 32  ? FN<DT, 4, 1>(A)                 \
     : (E) <= 64  ? FN<DT, 8, 1>(A)                 \
     : (E) <= 128 ? FN<DT, 16, 1>(A)                \
     : (E) <= 256 ? FN<DT, 32, 1>(A)                \
     : (E) <= 512 ? FN<DT, 64, 1>(A)                \
                  : FN<DT, 64, 2>(A))

}  // namespace

// One workgroup up to 2^15 logits (its launch alone is then most of the time);
// past that a workgroup for every 2^14, at most one a compute unit.
int balance_groups(int64_t rows, int64_t experts, int cus) {
    const int64_t n = rows * experts;
    if (n <= 1 << 15) return 1;
    const int64_t g = (n + (1 << 14) - 1) >> 14;
    return (int)(g < cus ? g : cus);
}

hipError_t launch_balance(int dtype, const void *logits, const void *index, bool wide_index, const uint8_t *mask,
                          float *loss, int32_t *counts, int32_t *offsets, int32_t *tokens, int32_t rows, int32_t experts,
                          int32_t k, float coefficient, const int32_t *live, int groups, void *workspace,
                          hipStream_t stream) {
    float *part_sums = (float *)workspace;
    int32_t *part_counts = groups > 1 ? (int32_t *)(part_sums + (size_t)groups * experts) : nullptr;
    int32_t *part_tokens = groups > 1 ? part_counts + (size_t)groups * experts : nullptr;
    const Sums a{logits, index, wide_index, mask, part_sums, part_counts, part_tokens, rows, experts, k, coefficient,
                 live, groups, loss, counts, offsets, tokens, stream};
    hipError_t e;
    switch (dtype) {
    case DT_F32: e = GA_BY_EXPERTS(sums_as, DT_F32, experts, a); break;
    case DT_F16: e = GA_BY_EXPERTS(sums_as, DT_F16, experts, a); break;
    case DT_BF16: e = GA_BY_EXPERTS(sums_as, DT_BF16, experts, a); break;
    default: return hipErrorInvalidValue;
    }
    if (e != hipSuccess || groups == 1) return e;
    finish_kernel<<<1, FINISH_BLOCK, 0, stream>>>(part_sums, part_counts, part_tokens, groups, experts, k, coefficient,
                                                  loss, counts, offsets, tokens);
    return hipGetLastError();
}

hipError_t launch_balance_backward(int dtype, const void *logits, const uint8_t *mask, const int32_t *counts,
                                   const int32_t *offsets, const int32_t *tokens, const float *dloss, void *dlogits,
                                   int32_t rows, int32_t experts, int32_t k, float coefficient, const int32_t *live,
                                   int cus, hipStream_t stream) {
    const Gradient a{logits, mask, counts, offsets, tokens, dloss, dlogits, rows, experts, k, coefficient, live, cus,
                     stream};
    switch (dtype) {
    case DT_F32: return GA_BY_EXPERTS(gradient_as, DT_F32, experts, a);
    case DT_F16: return GA_BY_EXPERTS(gradient_as, DT_F16, experts, a);
    case DT_BF16: return GA_BY_EXPERTS(gradient_as, DT_BF16, experts, a);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace ga

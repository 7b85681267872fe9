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
//
// Measured (medians of a kernel trace): 16384 tokens of 128 experts, top 8, bf16
// (13 MB): sums 7.2 us, finish 5.4 us, gradient 4.7 us; 64 tokens of 8 experts
// 5.0 us and 2.2 us; 65536 tokens of 128, masked: sums 19.2 us (21 MB), finish 5.0 us,
// gradient 9.8 us (34 MB).  Latency at the smaller sizes: a launch, one or two
// dependent rounds of loads, a finishing workgroup that reads 131 KB by itself; at
// the larger ones the sums run on half of the compute units.
#include "ga_internal.h"
#include "ga_train.h"

namespace ga {

namespace {

constexpr int BAL_BLOCK = 512;
constexpr int FINISH_BLOCK = 1024;

// Over the L lanes (a power of two) that hold a token, the same on each: DPP
// inside 16 lanes, shuffles beyond.
template <int L, typename F>
__device__ __forceinline__ float lanes_reduce(float v, F &&f) {
    if constexpr (L >= 2) v = f(v, dpp_move<0xB1>(v));
    if constexpr (L >= 4) v = f(v, dpp_move<0x4E>(v));
    if constexpr (L >= 8) v = f(v, dpp_move<0x141>(v));
    if constexpr (L >= 16) v = f(v, dpp_move<0x140>(v));
    if constexpr (L >= 32) v = f(v, __shfl_xor(v, 16));
    if constexpr (L >= 64) v = f(v, __shfl_xor(v, 32));
    return v;
}

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
    return lanes_reduce<L>(v, [](float a, float b) { return a + b; });
}

// The lanes that hold a token: L of V octets.  TINY: fewer than eight experts.
template <int L_, int V_, bool TINY_ = false> struct Lanes {
    static constexpr int L = L_, V = V_;
    static constexpr bool TINY = TINY_;
};

template <int DT, typename T> struct Token {
    Oct<DT> o[T::V];
};

template <int DT, typename T>
__device__ __forceinline__ void token_fetch(Token<DT, T> &t, const typename Elem<DT>::storage *row, uint32_t lane, int E) {
#pragma unroll
    for (int v = 0; v < T::V; ++v) oct_fetch<DT, T::TINY, false>(t.o[v], row, (int)(v * T::L + lane) * 8, E);
}

// Softmax over a token's E experts; lanes past E get 0.  A NaN or +inf logit
// makes the token's probabilities NaN.
template <int DT, typename T>
__device__ __forceinline__ void token_softmax(Token<DT, T> &t, uint32_t lane, int E, float (&p)[T::V][8]) {
    constexpr int L = T::L, V = T::V;
    float top = -__builtin_inff();
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (int)(v * L + lane) * 8;
        oct_trim<DT, T::TINY>(t.o[v], c, E);
        oct_unpack<DT>(t.o[v], p[v]);
        if (c + 8 > E) {
#pragma unroll
            for (int e = 0; e < 8; ++e) p[v][e] = c + e < E ? p[v][e] : -__builtin_inff();
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) top = __builtin_fmaxf(top, p[v][e]);
    }
    top = lanes_reduce<L>(top, [](float a, float b) { return __builtin_fmaxf(a, b); });
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
    sum = lanes_sum<L>(sum);
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

template <int DT, typename T, typename I>
__global__ __launch_bounds__(BAL_BLOCK) void sums_kernel(
    const typename Elem<DT>::storage *__restrict__ logits, const I *__restrict__ index, const uint8_t *__restrict__ mask,
    uint2 *__restrict__ parts, int32_t *__restrict__ part_tokens, int32_t rows, int32_t E, int32_t k, float coefficient,
    const int32_t *__restrict__ live, float *loss, int32_t *out_counts, int32_t *out_offsets, int32_t *out_tokens) {
    constexpr int L = T::L, V = T::V;
    constexpr int WAVES = BAL_BLOCK / 64, GROUPS = BAL_BLOCK / L, WIDTH = L * V * 8;
    __shared__ float sums[WAVES][WIDTH];
    __shared__ int32_t counts[WIDTH];
    __shared__ int32_t tokens[WAVES];
    const uint32_t n = live != nullptr ? (uint32_t)clamp_live(live, rows) : (uint32_t)rows;
    // this workgroup's run of tokens
    const uint32_t each = ((uint32_t)rows + gridDim.x - 1) / gridDim.x;
    const uint64_t begin64 = (uint64_t)blockIdx.x * each, end64 = begin64 + each;
    const uint32_t begin = begin64 < n ? (uint32_t)begin64 : n, end = end64 < n ? (uint32_t)end64 : n;
    const uint32_t lane = threadIdx.x % L;
    // a token past the run reads the run's last one, unused
    auto token = [&](uint32_t base) { return base + threadIdx.x / L; };
    auto row_of = [&](uint32_t t) { return logits + (size_t)(t < end ? t : end - 1) * E; };
    Token<DT, T> now, next;
    if (begin < end) token_fetch(next, row_of(token(begin)), lane, E);
    for (int i = threadIdx.x; i < WIDTH; i += BAL_BLOCK) counts[i] = 0;
    __syncthreads();
    // indices, flat over the run
    const uint64_t first = (uint64_t)begin * k, past = (uint64_t)end * k;
    for (uint64_t i = first + threadIdx.x; i < past; i += BAL_BLOCK) {
        const I e = index[i];
        if (e >= 0 && e < (I)E && (mask == nullptr || mask[begin + (uint32_t)((i - first) / (uint32_t)k)] != 0))
            atomicAdd(&counts[(int)e], 1);
    }
    float acc[V][8];
    int32_t used = 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[v][e] = 0.0f;
    // every lane of a wavefront makes the same number of rounds (shuffles)
    for (uint32_t base = begin; base < end; base += GROUPS) {
        const uint32_t t = token(base);
        now = next;
        token_fetch(next, row_of(token(base + GROUPS)), lane, E);
        const bool use = t < end && (mask == nullptr || mask[t < end ? t : begin] != 0);
        float p[V][8];
        token_softmax(now, lane, E, p);
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
        // sum and count side by side: one load of the finishing workgroup
        if (gridDim.x > 1)
            parts[(size_t)blockIdx.x * E + i] = uint2{__builtin_bit_cast(uint32_t, a), (uint32_t)counts[i]};
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
__global__ __launch_bounds__(FINISH_BLOCK) void finish_kernel(const uint2 *__restrict__ parts,
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
    constexpr int AT_ONCE = 16;  // loads in flight
    const int from = col < E ? col : 0;
    for (int g = slice; g < groups; g += slices * AT_ONCE) {
        uint2 v[AT_ONCE];
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j) {
            const int h = g + j * slices;
            v[j] = parts[(size_t)(h < groups ? h : g) * E + from];
        }
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j) {
            const bool in = g + j * slices < groups;
            a += in ? __builtin_bit_cast(float, v[j].x) : 0.0f;
            c += in ? (int32_t)v[j].y : 0;
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

template <int DT, typename T>
__global__ __launch_bounds__(BAL_BLOCK) void gradient_kernel(
    const typename Elem<DT>::storage *__restrict__ logits, const uint8_t *__restrict__ mask,
    const int32_t *__restrict__ counts, const int32_t *__restrict__ offsets, const int32_t *__restrict__ tokens,
    const float *__restrict__ dloss, typename Elem<DT>::storage *__restrict__ dlogits, int32_t rows, int32_t E, int32_t k,
    float coefficient, const int32_t *__restrict__ live) {
    constexpr int L = T::L, V = T::V, GROUPS = BAL_BLOCK / L;
    const uint32_t n = live != nullptr ? (uint32_t)clamp_live(live, rows) : (uint32_t)rows;
    const uint32_t lane = threadIdx.x % L;
    if (blockIdx.x * GROUPS >= n) return;
    // a token past the last reads that one, unused
    auto token = [&](uint32_t base) { return base + threadIdx.x / L; };
    auto row_of = [&](uint32_t t) { return logits + (size_t)(t < n ? t : n - 1) * E; };
    Token<DT, T> now, next;
    token_fetch(next, row_of(token(blockIdx.x * GROUPS)), lane, E);
    Oct<DT_F32> c8[V];  // int32 counts, as raw words
#pragma unroll
    for (int v = 0; v < V; ++v)
        oct_fetch<DT_F32, T::TINY, false>(c8[v], (const uint32_t *)counts, (int)(v * L + lane) * 8, E);
    const float m = (float)*tokens;
    const float factor = m == 0.0f ? 0.0f : *dloss * coefficient * ((float)E / ((float)k * m)) / m;
    // sum_j p_j = 1: taken from (about) their mean, the counts cancel less
    const int32_t middle = offsets[E] / E;
    float w[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (int)(v * L + lane) * 8;
        oct_trim<DT_F32, T::TINY>(c8[v], c, E);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[v][e] = c + e < E ? (float)((int32_t)c8[v].w[e] - middle) : 0.0f;
    }
    for (uint32_t base = blockIdx.x * GROUPS; base < n; base += gridDim.x * GROUPS) {
        const uint32_t t = token(base);
        const bool in = t < n;
        float p[V][8];
        now = next;
        token_fetch(next, row_of(token(base + gridDim.x * GROUPS)), lane, E);
        token_softmax(now, lane, E, p);
        float dot = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < 8; ++e) dot = __builtin_fmaf(p[v][e], w[v][e], dot);
        dot = lanes_sum<L>(dot);
        // the mean of the distances to it, once more: where one p is next to 1 the gradient is a small
        // difference of counts, of which the first mean carries roundings of the counts themselves
        float rest = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < 8; ++e) rest = __builtin_fmaf(p[v][e], w[v][e] - dot, rest);
        rest = lanes_sum<L>(rest);
        if (!in) continue;
        const bool use = mask == nullptr || mask[t] != 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (int)(v * L + lane) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) p[v][e] = use ? factor * p[v][e] * ((w[v][e] - dot) - rest) : 0.0f;
            if (c < E) oct_store<DT>(dlogits + (size_t)t * E + c, p[v], E - c);
        }
    }
}

struct Sums {
    const void *logits, *index;
    bool wide_index;
    const uint8_t *mask;
    uint2 *parts;
    int32_t *part_tokens;
    int32_t rows, E, k;
    float coefficient;
    const int32_t *live;
    int groups;
    float *loss;
    int32_t *counts, *offsets, *tokens;
    hipStream_t stream;
};

template <int DT, typename T, typename I>
hipError_t sums_as(const Sums &a) {
    using S = typename Elem<DT>::storage;
    return launch_kernel(sums_kernel<DT, T, I>, dim3((uint32_t)a.groups), BAL_BLOCK, a.stream, (const S *)a.logits,
                         (const I *)a.index, a.mask, a.parts, a.part_tokens, a.rows, a.E, a.k, a.coefficient,
                         a.live, a.loss, a.counts, a.offsets, a.tokens);
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

template <int DT, typename T>
hipError_t gradient_as(const Gradient &a) {
    using S = typename Elem<DT>::storage;
    constexpr int GROUPS = BAL_BLOCK / T::L;
    const int64_t need = ((int64_t)a.rows + GROUPS - 1) / GROUPS, most = (int64_t)a.cus * 8;
    return launch_kernel(gradient_kernel<DT, T>, dim3((uint32_t)(need < most ? need : most)), BAL_BLOCK, a.stream,
                         (const S *)a.logits, a.mask, a.counts, a.offsets, a.tokens, a.dloss, (S *)a.dlogits, a.rows, a.E,
                         a.k, a.coefficient, a.live);
}

// The lanes that hold a token, by E: eight experts a lane up to 512.
template <typename F>
hipError_t by_experts(int32_t E, F &&f) {
    if (E < 8) return f(Lanes<1, 1, true>());
    if (E == 8) return f(Lanes<1, 1>());
    if (E <= 16) return f(Lanes<2, 1>());
    if (E <= 32) return f(Lanes<4, 1>());
    if (E <= 64) return f(Lanes<8, 1>());
    if (E <= 128) return f(Lanes<16, 1>());
    if (E <= 256) return f(Lanes<32, 1>());
    if (E <= 512) return f(Lanes<64, 1>());
    return f(Lanes<64, 2>());
}

template <int DT>
hipError_t sums_dt(const Sums &a) {
    return by_experts(a.E, [&](auto t) {
        return a.wide_index ? sums_as<DT, decltype(t), int64_t>(a) : sums_as<DT, decltype(t), int32_t>(a);
    });
}

template <int DT>
hipError_t gradient_dt(const Gradient &a) {
    return by_experts(a.E, [&](auto t) { return gradient_as<DT, decltype(t)>(a); });
}

}  // namespace

// One workgroup up to 2^15 logits (its launch alone is then most of the time);
// past that a workgroup for every 2^14, on at most half of the compute units:
// the one that finishes reads 8 E bytes of each (16384 tokens of 128 experts,
// bf16, fastest of a trace: 7.0 us and 4.9 us to finish, 6.6 us and 7.0 us with 256
// workgroups).
int balance_groups(int64_t rows, int64_t experts, int cus) {
    const int64_t n = rows * experts, most = cus > 1 ? cus / 2 : 1;
    if (n <= 1 << 15) return 1;
    const int64_t g = (n + (1 << 14) - 1) >> 14;
    return (int)(g < most ? g : most);
}

hipError_t launch_balance(int dtype, const void *logits, const void *index, bool wide_index, const uint8_t *mask,
                          float *loss, int32_t *counts, int32_t *offsets, int32_t *tokens, int32_t rows, int32_t experts,
                          int32_t k, float coefficient, const int32_t *live, int groups, void *workspace,
                          hipStream_t stream) {
    uint2 *parts = (uint2 *)workspace;
    int32_t *part_tokens = groups > 1 ? (int32_t *)(parts + (size_t)groups * experts) : nullptr;
    const Sums a{logits, index, wide_index, mask, parts, part_tokens, rows, experts, k, coefficient,
                 live, groups, loss, counts, offsets, tokens, stream};
    hipError_t e;
    switch (dtype) {
    case DT_F32: e = sums_dt<DT_F32>(a); break;
    case DT_F16: e = sums_dt<DT_F16>(a); break;
    case DT_BF16: e = sums_dt<DT_BF16>(a); break;
    default: return hipErrorInvalidValue;
    }
    if (e != hipSuccess || groups == 1) return e;
    return launch_kernel(finish_kernel, dim3(1), FINISH_BLOCK, stream, parts, part_tokens, groups, experts,
                         k, coefficient, loss, counts, offsets, tokens);
}

hipError_t launch_balance_backward(int dtype, const void *logits, const uint8_t *mask, const int32_t *counts,
                                   const int32_t *offsets, const int32_t *tokens, const float *dloss, void *dlogits,
                                   int32_t rows, int32_t experts, int32_t k, float coefficient, const int32_t *live,
                                   int cus, hipStream_t stream) {
    const Gradient a{logits, mask, counts, offsets, tokens, dloss, dlogits, rows, experts, k, coefficient, live, cus,
                     stream};
    switch (dtype) {
    case DT_F32: return gradient_dt<DT_F32>(a);
    case DT_F16: return gradient_dt<DT_F16>(a);
    case DT_BF16: return gradient_dt<DT_BF16>(a);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace ga

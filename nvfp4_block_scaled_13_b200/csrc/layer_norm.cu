// layer_norm.cu — layer norm forward (with the amax of its result) and backward on sm_100a.
//
// Forward, per row of x: mean = S x / C, var = S (x - mean)^2 / C, rstd = (var + eps)^-1/2,
// y = (x - mean) rstd w + b. Backward, with xh = (x - mean) rstd and h = dy w:
// dx = rstd (h - S h / C - xh S(h xh) / C), dw = S_rows dy xh, db = S_rows dy.
// Both are bound by memory: 4 bytes an element forward and 6 backward in BF16.
//
// A row belongs to a group of threads: 8, 16 or 32 lanes of a warp (no barrier), or a CTA. A
// thread holds its share of the row in registers from the loads to the result, so x (and dy) are
// read once, and holds its columns' weight and bias (and their gradients' sums) over all the rows
// that its group works through. The variance is summed from the held row after the mean is
// known: no cancellation, at the price of a second reduction.
//
// Rows arrive ahead of their use through a ring in shared memory. Each thread copies (cp.async)
// and later reads its own 16-byte units only, so the ring needs no barrier and no registers.
//
// A row that does not start on 16 bytes is read as if it began at the unit's boundary, `shift`
// elements earlier, and its first and last units are masked. Groups take rows in steps whose
// length in bytes is a multiple of 16, so a group's shift, and with it the columns of each
// thread, stays the same: odd row lengths run on the same vector path.
//
// The column sums of the backward pass stay in registers; each CTA writes one partial row to the
// workspace and a second kernel adds the partial rows in order, so the result does not depend on
// how CTAs were scheduled.
#include <float.h>

#include <algorithm>

#include "../../include/nvfp4_train.h"
#include "train.cuh"

namespace {

using namespace nvfp4_train;

struct NormArgs {
    const void* x;
    const void* weight;
    const void* bias;
    bool w_f32, w_vector;
    int64_t rows;
    int cols;
    float eps;
    void* y;
    float* mean;
    float* rstd;
    uint32_t* amax;
};

struct NormGradArgs {
    const void* dy;
    const void* x;
    const void* weight;
    bool w_f32, w_vector;
    const float* mean;
    const float* rstd;
    int64_t rows;
    int cols;
    void* dx;
    float* sums;   // [2][parts][cols]: partial dweight, partial dbias; or NULL
    int parts;
};

// ---- units ---------------------------------------------------------------------------------

template <typename T>
constexpr int kUnit = 16 / sizeof(T);   // elements of 16 bytes

__device__ __forceinline__ void unpack(const uint4& w, float2 (&v)[4], bf16) {
    v[0] = make_float2(bf16_lo(w.x), bf16_hi(w.x));
    v[1] = make_float2(bf16_lo(w.y), bf16_hi(w.y));
    v[2] = make_float2(bf16_lo(w.z), bf16_hi(w.z));
    v[3] = make_float2(bf16_lo(w.w), bf16_hi(w.w));
}
__device__ __forceinline__ void unpack(const uint4& w, float2 (&v)[2], float) {
    v[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
    v[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
}
__device__ __forceinline__ uint4 pack(const float2 (&v)[4], bf16) {
    return make_uint4(to_bf16x2(v[0].x, v[0].y), to_bf16x2(v[1].x, v[1].y), to_bf16x2(v[2].x, v[2].y),
                      to_bf16x2(v[3].x, v[3].y));
}
__device__ __forceinline__ uint4 pack(const float2 (&v)[2], float) {
    return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
}

// Running maximum of stored magnitudes: two BF16 halves, or one FP32 word.
__device__ __forceinline__ void join_top(uint32_t& top, const uint4& w, bf16) {
    top = __vmaxu2(__vmaxu2(top, w.x & 0x7FFF7FFFu), w.y & 0x7FFF7FFFu);
    top = __vmaxu2(__vmaxu2(top, w.z & 0x7FFF7FFFu), w.w & 0x7FFF7FFFu);
}
__device__ __forceinline__ void join_top(uint32_t& top, const uint4& w, float) {
    top = max(max(top, w.x & 0x7FFFFFFFu), max(w.y & 0x7FFFFFFFu, max(w.z & 0x7FFFFFFFu, w.w & 0x7FFFFFFFu)));
}
__device__ __forceinline__ uint32_t top_bits(uint32_t top, bf16) { return max(top << 16, top & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t top_bits(uint32_t top, float) { return top; }

__device__ __forceinline__ void copy_async(uint4* to, const void* from) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(to))),
                 "l"(from)
                 : "memory");
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// The columns of a thread: unit q holds columns start(q) .. start(q) + E - 1, of which those with
// their bit in mask(q) exist.
template <typename T, int Q, bool SHIFTED>
struct Columns {
    static constexpr int E = kUnit<T>;
    static constexpr uint32_t kAll = (1u << E) - 1u;
    int base, stride, cols;

    __device__ __forceinline__ Columns(int t, int lanes, int shift, int cols_) : base(t * E - shift), stride(lanes * E), cols(cols_) {}
    __device__ __forceinline__ int start(int q) const { return base + q * stride; }
    __device__ __forceinline__ uint32_t mask(int q) const {
        const int c = start(q);
        if (!SHIFTED) return c < cols ? kAll : 0u;
        uint32_t m = kAll;
        if (c < 0) m &= kAll << -c;
        if (c + E > cols) m &= c >= cols ? 0u : kAll >> (c + E - cols);
        return m;
    }
};

template <int H>
__device__ __forceinline__ void keep(float2 (&v)[H], uint32_t mask) {
#pragma unroll
    for (int k = 0; k < H; ++k) {
        if (!(mask >> (2 * k) & 1u)) v[k].x = 0.0f;
        if (!(mask >> (2 * k + 1) & 1u)) v[k].y = 0.0f;
    }
}

// Starts the copy of one unit of a tensor of `total` elements. A unit that reaches over the
// tensor's ends (only where the tensor itself is not aligned) is copied by the element.
template <typename T, bool SHIFTED>
__device__ __forceinline__ void fetch_unit(uint4* slot, const T* tensor, int64_t at, int64_t total, uint32_t mask) {
    constexpr int E = kUnit<T>;
    if (mask == 0) return;
    if (SHIFTED && (at < 0 || at + E > total)) {
        T* to = reinterpret_cast<T*>(slot);
#pragma unroll
        for (int j = 0; j < E; ++j)
            if (mask >> j & 1u) to[j] = tensor[at + j];
    } else {
        copy_async(slot, tensor + at);
    }
}

template <typename T>
__device__ __forceinline__ void store_unit(T* to, const uint4& w, uint32_t mask) {
    constexpr int E = kUnit<T>;
    if (mask == (1u << E) - 1u) {
        *reinterpret_cast<uint4*>(to) = w;
    } else if (mask) {
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < E; ++j) {
            if (!(mask >> j & 1u)) continue;
            if (E == 8) {
                reinterpret_cast<uint16_t*>(to)[j] = static_cast<uint16_t>(a[j / 2] >> (16 * (j & 1)));
            } else {
                reinterpret_cast<uint32_t*>(to)[j] = a[j & 3];
            }
        }
    }
}

__device__ __forceinline__ float param_at(const void* p, bool f32, int c) {
    return f32 ? static_cast<const float*>(p)[c] : to_float(static_cast<const bf16*>(p)[c]);
}

// The weight's (or bias's) values of a unit; `fill` in every existing column where there is no
// parameter, zero in columns that do not exist.
template <int E>
__device__ __forceinline__ void load_param(const void* p, bool f32, bool vector, int c, uint32_t mask, float fill,
                                           float2 (&out)[E / 2]) {
    float v[E];
    if (p == nullptr || mask != (1u << E) - 1u || !vector) {
#pragma unroll
        for (int j = 0; j < E; ++j) v[j] = mask >> j & 1u ? (p ? param_at(p, f32, c + j) : fill) : 0.0f;
    } else if (f32) {
#pragma unroll
        for (int k = 0; k < E / 4; ++k) {
            const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + c + 4 * k);
            v[4 * k] = a.x, v[4 * k + 1] = a.y, v[4 * k + 2] = a.z, v[4 * k + 3] = a.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < E / 4; ++k) {
            const uint2 a = *reinterpret_cast<const uint2*>(static_cast<const bf16*>(p) + c + 4 * k);
            v[4 * k] = bf16_lo(a.x), v[4 * k + 1] = bf16_hi(a.x), v[4 * k + 2] = bf16_lo(a.y), v[4 * k + 3] = bf16_hi(a.y);
        }
    }
#pragma unroll
    for (int k = 0; k < E / 2; ++k) out[k] = make_float2(v[2 * k], v[2 * k + 1]);
}

// ---- sums over a row's threads ------------------------------------------------------------

template <int LANES>
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
    for (int off = (LANES ? LANES : 32) / 2; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
    return v;
}

// Partial sums of a CTA's warps, two sets that alternate: the barrier of the next reduction
// separates this one's reads from the writes after next, so a reduction has one barrier.
struct WarpSums {
    float4 set[2][4];   // 16 warps
    __device__ __forceinline__ void clear() {
        if (threadIdx.x < 8) (&set[0][0])[threadIdx.x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    __device__ __forceinline__ void put(int which, float v) {
        if ((threadIdx.x & 31) == 0) reinterpret_cast<float*>(set[which])[threadIdx.x >> 5] = v;
    }
    __device__ __forceinline__ float total(int which) const {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k * 128 >= blockDim.x) break;
            const float4 p = set[which][k];
            s += (p.x + p.y) + (p.z + p.w);
        }
        return s;
    }
};

// One CTA alone writes its maximum; several join theirs with an (order-free) atomic maximum.
__device__ __forceinline__ void publish_amax(uint32_t top, uint32_t* amax) {
    __shared__ uint32_t best[32];
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    top = __reduce_max_sync(kFull, top);
    if (lane == 0) best[threadIdx.x >> 5] = top;
    __syncthreads();
    if (threadIdx.x < 32) {
        top = __reduce_max_sync(kFull, lane < warps ? best[lane] : 0u);
        if (lane == 0) {
            if (gridDim.x == 1) {
                *amax = top;
            } else {
                atomicMax(amax, top);
            }
        }
    }
}

// ---- forward -------------------------------------------------------------------------------

// Rows in the ring; the longest FP32 rows have room for three.
__host__ __device__ constexpr int forward_stages(int row_bytes_of_thread) { return row_bytes_of_thread > 64 ? 3 : 4; }
constexpr int kBackwardStages = 3;

// Registers of a thread, and with them the CTAs that an SM holds.
constexpr int forward_registers(int elements) { return elements == 32 ? 128 : elements == 16 ? 80 : 64; }
constexpr int backward_registers(int elements) { return elements == 16 ? 128 : 80; }
constexpr int resident(int registers, int threads) { return std::max(1, std::min(32, 65536 / registers / threads)); }

// N elements a thread; LANES threads a row, 0: the CTA.
template <typename T, int N, int LANES, bool SHIFTED>
__global__ void __maxnreg__(forward_registers(N)) norm_kernel(const NormArgs a) {
    constexpr int E = kUnit<T>, Q = N / E, H = E / 2, S = forward_stages(N * sizeof(T));
    extern __shared__ uint4 ring[];   // [S][Q][threads]
    __shared__ WarpSums warp_sums;
    const int threads = blockDim.x, lanes = LANES ? LANES : threads;
    const int t = LANES ? threadIdx.x % (LANES ? LANES : 1) : threadIdx.x;
    const int groups = LANES ? threads / (LANES ? LANES : 1) : 1;
    const int64_t first = int64_t(blockIdx.x) * groups + (LANES ? threadIdx.x / (LANES ? LANES : 1) : 0);
    const int64_t step = int64_t(gridDim.x) * groups, total = a.rows * a.cols;
    const T* x = static_cast<const T*>(a.x);
    const int shift = SHIFTED ? static_cast<int>((reinterpret_cast<uintptr_t>(x + first * a.cols) & 15) / sizeof(T)) : 0;
    const Columns<T, Q, SHIFTED> at(t, lanes, shift, a.cols);
    uint32_t mask[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) mask[q] = at.mask(q);

    const auto fetch = [&](int64_t row, int stage) {
        if (row < a.rows) {
#pragma unroll
            for (int q = 0; q < Q; ++q)
                fetch_unit<T, SHIFTED>(&ring[(stage * Q + q) * threads + threadIdx.x], x, row * a.cols + at.start(q), total, mask[q]);
        }
        commit_copies();
    };
#pragma unroll
    for (int s = 0; s < S - 1; ++s) fetch(first + s * step, s);
    float2 w[Q][H], b[Q][H];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        load_param<E>(a.weight, a.w_f32, a.w_vector, at.start(q), mask[q], 1.0f, w[q]);
        load_param<E>(a.bias, a.w_f32, a.w_vector, at.start(q), mask[q], 0.0f, b[q]);
    }
    if (!LANES) {
        warp_sums.clear();
        __syncthreads();
    }
    const float inv = 1.0f / static_cast<float>(a.cols);
    uint32_t top = 0;
    int stage = 0;
    // Every lane of a warp makes the same number of turns: the shuffles need them all.
    const int64_t turns = LANES ? (a.rows - int64_t(blockIdx.x) * groups + step - 1) / step : (a.rows - first + step - 1) / step;
    int64_t r = first;
    for (int64_t turn = 0; turn < turns; ++turn, r += step) {
        wait_copies<S - 2>();
        float2 v[Q][H];
        float2 sum2 = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            unpack(ring[(stage * Q + q) * threads + threadIdx.x], v[q], T{});
            if (mask[q] != Columns<T, Q, SHIFTED>::kAll) keep(v[q], mask[q]);
#pragma unroll
            for (int k = 0; k < H; ++k) sum2 = add2(sum2, v[q][k]);
        }
        fetch(r + (S - 1) * step, stage == 0 ? S - 1 : stage - 1);
        stage = stage == S - 1 ? 0 : stage + 1;
        float sum = lane_sum<LANES>(sum2.x + sum2.y);
        if (!LANES) {
            warp_sums.put(0, sum);
            __syncthreads();
            sum = warp_sums.total(0);
        }
        const float mean = sum * inv;
        float2 square2 = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
#pragma unroll
            for (int k = 0; k < H; ++k) v[q][k] = add2(v[q][k], make_float2(-mean, -mean));
            if (mask[q] != Columns<T, Q, SHIFTED>::kAll) keep(v[q], mask[q]);
#pragma unroll
            for (int k = 0; k < H; ++k) square2 = fma2(v[q][k], v[q][k], square2);
        }
        float square = lane_sum<LANES>(square2.x + square2.y);
        if (!LANES) {
            warp_sums.put(1, square);
            __syncthreads();
            square = warp_sums.total(1);
        }
        const float rstd = rsqrtf(fmaf(square, inv, a.eps));
        if (r < a.rows) {
            T* y = static_cast<T*>(a.y) + r * a.cols;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
#pragma unroll
                for (int k = 0; k < H; ++k) v[q][k] = fma2(mul2(v[q][k], make_float2(rstd, rstd)), w[q][k], b[q][k]);
                const uint4 out = pack(v[q], T{});
                if (a.amax && mask[q]) join_top(top, out, T{});
                store_unit(y + at.start(q), out, mask[q]);
            }
            if (t == 0) {
                if (a.mean) a.mean[r] = mean;
                if (a.rstd) a.rstd[r] = rstd;
            }
        }
    }
    wait_copies<0>();
    if (a.amax) publish_amax(top_bits(top, T{}), a.amax);
}

// Sum over a CTA of any size; `buffer` alternates as the sets of WarpSums do.
__device__ __forceinline__ float cta_sum(float v, float (*scratch)[32], int& buffer) {
    v = warp_sum(v);
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) scratch[buffer][threadIdx.x >> 5] = v;
    __syncthreads();
    v = warp_sum(lane < warps ? scratch[buffer][lane] : 0.0f);
    buffer ^= 1;
    return v;
}

__device__ __forceinline__ uint32_t stored_magnitude(float v, bf16) {
    return (uint32_t(to_bf16(v)) << 16) & 0x7FFFFFFFu;
}
__device__ __forceinline__ uint32_t stored_magnitude(float v, float) { return magnitude(v); }

// Rows too long for one CTA's registers, and operands whose rows start at different places within
// 16 bytes: three passes by the element, the later two from L1 or L2.
template <typename T>
__global__ void __launch_bounds__(1024) norm_long_kernel(const NormArgs a) {
    __shared__ float scratch[2][32];
    const float count = static_cast<float>(a.cols);
    uint32_t top = 0;
    int buffer = 0;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + r * a.cols;
        float sum = 0.0f, square = 0.0f;
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) sum += to_float(x[c]);
        const float mean = cta_sum(sum, scratch, buffer) / count;
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
            const float d = to_float(x[c]) - mean;
            square = fmaf(d, d, square);
        }
        const float rstd = rsqrtf(cta_sum(square, scratch, buffer) / count + a.eps);
        T* y = static_cast<T*>(a.y) + r * a.cols;
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
            float w = 1.0f, b = 0.0f;
            if (a.weight) w = param_at(a.weight, a.w_f32, c);
            if (a.bias) b = param_at(a.bias, a.w_f32, c);
            const float v = fmaf((to_float(x[c]) - mean) * rstd, w, b);
            y[c] = from_float<T>(v);
            top = max(top, stored_magnitude(v, T{}));
        }
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
    if (a.amax) publish_amax(top, a.amax);
}

// ---- backward ------------------------------------------------------------------------------

// Adds the column sums of the groups of a CTA in their order and writes the CTA's partial row.
template <typename T, int Q, bool SHIFTED>
__device__ __forceinline__ void join_groups(const float2 (&s)[Q][kUnit<T> / 2], const Columns<T, Q, SHIFTED>& at, int group,
                                            int groups, float* shared, float* out) {
    constexpr int E = kUnit<T>;
    for (int g = 0; g < groups; ++g) {
        if (group == g) {
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const uint32_t mask = at.mask(q);
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    const float v = j & 1 ? s[q][j / 2].y : s[q][j / 2].x;
                    float* sum = shared + at.start(q) + j;
                    if (mask >> j & 1u) *sum = g == 0 ? v : *sum + v;
                }
            }
        }
        __syncthreads();
    }
    for (int c = threadIdx.x; c < at.cols; c += blockDim.x) out[c] = shared[c];
    __syncthreads();
}

template <typename T, int N, int LANES, bool SHIFTED>
__global__ void __maxnreg__(backward_registers(N)) norm_grad_kernel(const NormGradArgs a) {
    constexpr int E = kUnit<T>, Q = N / E, H = E / 2, S = kBackwardStages;
    extern __shared__ uint4 ring[];   // [S][x, dy][Q][threads]
    __shared__ WarpSums sums1, sums2;
    __shared__ float joined[LANES ? LANES * N : 1];
    const int threads = blockDim.x, lanes = LANES ? LANES : threads;
    const int t = LANES ? threadIdx.x % (LANES ? LANES : 1) : threadIdx.x;
    const int groups = LANES ? threads / (LANES ? LANES : 1) : 1, group = LANES ? threadIdx.x / (LANES ? LANES : 1) : 0;
    const int64_t first = int64_t(blockIdx.x) * groups + group;
    const int64_t step = int64_t(gridDim.x) * groups, total = a.rows * a.cols;
    const T* x = static_cast<const T*>(a.x);
    const T* dy = static_cast<const T*>(a.dy);
    const int shift = SHIFTED ? static_cast<int>((reinterpret_cast<uintptr_t>(x + first * a.cols) & 15) / sizeof(T)) : 0;
    const Columns<T, Q, SHIFTED> at(t, lanes, shift, a.cols);
    uint32_t mask[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) mask[q] = at.mask(q);

    const auto fetch = [&](int64_t row, int stage) {
        if (row < a.rows) {
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const int64_t place = row * a.cols + at.start(q);
                fetch_unit<T, SHIFTED>(&ring[((stage * 2) * Q + q) * threads + threadIdx.x], x, place, total, mask[q]);
                fetch_unit<T, SHIFTED>(&ring[((stage * 2 + 1) * Q + q) * threads + threadIdx.x], dy, place, total, mask[q]);
            }
        }
        commit_copies();
    };
#pragma unroll
    for (int s = 0; s < S - 1; ++s) fetch(first + s * step, s);
    float2 w[Q][H], sw[Q][H], sb[Q][H];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        load_param<E>(a.weight, a.w_f32, a.w_vector, at.start(q), mask[q], 1.0f, w[q]);
#pragma unroll
        for (int k = 0; k < H; ++k) sw[q][k] = sb[q][k] = make_float2(0.0f, 0.0f);
    }
    if (!LANES) {
        sums1.clear();
        sums2.clear();
        __syncthreads();
    }
    const float inv = 1.0f / static_cast<float>(a.cols);
    int stage = 0, which = 0;
    const int64_t turns = LANES ? (a.rows - int64_t(blockIdx.x) * groups + step - 1) / step : (a.rows - first + step - 1) / step;
    int64_t r = first;
    float next_mean = r < a.rows ? a.mean[r] : 0.0f, next_rstd = r < a.rows ? a.rstd[r] : 0.0f;
    for (int64_t turn = 0; turn < turns; ++turn, r += step) {
        const float mean = next_mean, rstd = next_rstd;
        const bool exists = r < a.rows;   // a group past the last row adds nothing
        wait_copies<S - 2>();
        float2 xh[Q][H], h[Q][H];
        float2 s1 = make_float2(0.0f, 0.0f), s2 = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            unpack(ring[((stage * 2) * Q + q) * threads + threadIdx.x], xh[q], T{});
            unpack(ring[((stage * 2 + 1) * Q + q) * threads + threadIdx.x], h[q], T{});
            const uint32_t m = exists ? mask[q] : 0u;
#pragma unroll
            for (int k = 0; k < H; ++k) xh[q][k] = mul2(add2(xh[q][k], make_float2(-mean, -mean)), make_float2(rstd, rstd));
            if (m != Columns<T, Q, SHIFTED>::kAll) {
                keep(xh[q], m);
                keep(h[q], m);
            }
#pragma unroll
            for (int k = 0; k < H; ++k) {
                sw[q][k] = fma2(h[q][k], xh[q][k], sw[q][k]);
                sb[q][k] = add2(sb[q][k], h[q][k]);
                h[q][k] = mul2(h[q][k], w[q][k]);
                s1 = add2(s1, h[q][k]);
                s2 = fma2(h[q][k], xh[q][k], s2);
            }
        }
        fetch(r + (S - 1) * step, stage == 0 ? S - 1 : stage - 1);
        stage = stage == S - 1 ? 0 : stage + 1;
        if (r + step < a.rows) {
            next_mean = a.mean[r + step];
            next_rstd = a.rstd[r + step];
        }
        float t1 = lane_sum<LANES>(s1.x + s1.y), t2 = lane_sum<LANES>(s2.x + s2.y);
        if (!LANES) {
            sums1.put(which, t1);
            sums2.put(which, t2);
            __syncthreads();
            t1 = sums1.total(which);
            t2 = sums2.total(which);
            which ^= 1;
        }
        t1 *= inv;
        t2 *= inv;
        if (exists) {
            T* dx = static_cast<T*>(a.dx) + r * a.cols;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
#pragma unroll
                for (int k = 0; k < H; ++k)
                    h[q][k] = mul2(add2(h[q][k], fma2(xh[q][k], make_float2(-t2, -t2), make_float2(-t1, -t1))), make_float2(rstd, rstd));
                store_unit(dx + at.start(q), pack(h[q], T{}), mask[q]);
            }
        }
    }
    wait_copies<0>();
    if (a.sums) {
        float* out = a.sums + int64_t(blockIdx.x) * a.cols;
        float* out_b = out + int64_t(a.parts) * a.cols;
        if (LANES) {
            join_groups<T, Q, SHIFTED>(sw, at, group, groups, joined, out);
            join_groups<T, Q, SHIFTED>(sb, at, group, groups, joined, out_b);
        } else {
#pragma unroll
            for (int q = 0; q < Q; ++q)
#pragma unroll
                for (int j = 0; j < E; ++j)
                    if (mask[q] >> j & 1u) {
                        out[at.start(q) + j] = j & 1 ? sw[q][j / 2].y : sw[q][j / 2].x;
                        out_b[at.start(q) + j] = j & 1 ? sb[q][j / 2].y : sb[q][j / 2].x;
                    }
        }
    }
}

// dx where norm_long_kernel runs forward: two passes, the second from L1 or L2.
template <typename T>
__global__ void __launch_bounds__(1024) norm_grad_long_kernel(const NormGradArgs a) {
    __shared__ float scratch[2][2][32];
    const float inv = 1.0f / static_cast<float>(a.cols);
    int b1 = 0, b2 = 0;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + r * a.cols;
        const T* dy = static_cast<const T*>(a.dy) + r * a.cols;
        const float mean = a.mean[r], rstd = a.rstd[r];
        auto scaled = [&](int c) {
            float w = 1.0f;
            if (a.weight) w = param_at(a.weight, a.w_f32, c);
            return to_float(dy[c]) * w;
        };
        float s1 = 0.0f, s2 = 0.0f;
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
            const float h = scaled(c);
            s1 += h;
            s2 = fmaf(h, (to_float(x[c]) - mean) * rstd, s2);
        }
        s1 = cta_sum(s1, scratch[0], b1) * inv;
        s2 = cta_sum(s2, scratch[1], b2) * inv;
        T* dx = static_cast<T*>(a.dx) + r * a.cols;
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x)
            dx[c] = from_float<T>(rstd * (scaled(c) - fmaf((to_float(x[c]) - mean) * rstd, s2, s1)));
    }
}

// Their column sums: one column a thread, one slab of rows a grid row.
template <typename T>
__global__ void __launch_bounds__(256) norm_sums_kernel(const NormGradArgs a) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= a.cols) return;
    const int64_t lo = a.rows * blockIdx.y / gridDim.y, hi = a.rows * (blockIdx.y + 1) / gridDim.y;
    float sw = 0.0f, sb = 0.0f;
    for (int64_t r = lo; r < hi; ++r) {
        const float g = to_float(static_cast<const T*>(a.dy)[r * a.cols + c]);
        const float xh = (to_float(static_cast<const T*>(a.x)[r * a.cols + c]) - a.mean[r]) * a.rstd[r];
        sw = fmaf(g, xh, sw);
        sb += g;
    }
    a.sums[int64_t(blockIdx.y) * a.cols + c] = sw;
    a.sums[int64_t(a.parts + blockIdx.y) * a.cols + c] = sb;
}

// Adds the partial rows: 32 columns a CTA, 8 threads a column, in a fixed order.
template <typename W>
__global__ void __launch_bounds__(256) norm_join_kernel(const float* sums, int parts, int cols, W* dweight, W* dbias) {
    __shared__ float shared[8][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    W* out = blockIdx.y == 0 ? dweight : dbias;
    if (out == nullptr) return;
    const float* in = sums + int64_t(blockIdx.y) * parts * cols;
    float s = 0.0f;
    if (c < cols)
        for (int p = warp; p < parts; p += 8) s += in[int64_t(p) * cols + c];
    shared[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < cols) {
#pragma unroll
        for (int k = 1; k < 8; ++k) s += shared[k][lane];
        out[c] = from_float<W>(s);
    }
}

// ---- host ----------------------------------------------------------------------------------

bool known(nvfp4_type t) { return t == NVFP4_TYPE_BF16 || t == NVFP4_TYPE_F32; }
int type_size(nvfp4_type t) { return t == NVFP4_TYPE_F32 ? 4 : 2; }

bool shape_ok(int64_t rows, int64_t cols) {
    return rows >= 0 && cols >= 1 && cols <= (int64_t(1) << 30) && (rows == 0 || cols <= (int64_t(1) << 60) / rows);
}

nvfp4_status launched() { return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA; }

// How rows are given to threads.
struct Cut {
    int elements;   // of a thread; 0: by norm_long_kernel and its like
    int lanes;      // of a row: 8, 16, 32, or 0 for a CTA
    int threads;    // of a CTA
    bool shifted;
};

// Rows that start on 16 bytes take whole units; others, where all operands' rows start at the same
// place within 16 bytes, are shifted.
Cut cut_rows(int64_t cols, int size, bool aligned, bool congruent, int most_elements) {
    const int unit = 16 / size;
    const bool shifted = !aligned || cols % unit != 0;
    const int64_t need = cols + (shifted ? unit - 1 : 0);
    if (!congruent) return {0, 0, 0, false};
    if (need <= 64) return {8, 8, 128, shifted};
    if (need <= 128) return {8, 16, 128, shifted};
    if (need <= 256) return {8, 32, 128, shifted};
    if (need <= 512) return {16, 32, 128, shifted};
    for (int elements = 16; elements <= most_elements; elements *= 2) {
        const int64_t threads = (need + 32 * elements - 1) / (32 * elements) * 32;
        if (threads <= 512) return {elements, 0, static_cast<int>(threads), shifted};
    }
    return {0, 0, 0, false};
}

// CTAs that share the rows: at most `resident`, and so many that every group keeps its shift.
int64_t grid_of(const Cut& cut, int64_t rows, int64_t resident, int size) {
    const int64_t groups = cut.lanes ? cut.threads / cut.lanes : 1, need = (rows + groups - 1) / groups;
    if (need <= resident) return need;
    const int64_t unit = 16 / size;
    return resident * groups % unit == 0 ? resident : std::max<int64_t>(unit, resident / unit * unit);
}

Cut cut_backward(int64_t cols, int size, bool aligned, bool congruent) { return cut_rows(cols, size, aligned, congruent, 16); }

// CTAs of the backward pass, each of which leaves a partial row.
int64_t backward_parts(const Cut& cut, int64_t rows, int64_t cols, int size) {
    const int64_t sms = sm_count();
    if (cut.elements == 0) {
        const int64_t across = (cols + 255) / 256;
        return std::min<int64_t>(rows, std::max<int64_t>(1, 4 * sms / across));
    }
    return grid_of(cut, rows, sms * resident(backward_registers(cut.elements), cut.threads), size);
}

// Lets `kernel` have `bytes` of dynamic shared memory; without asking it may have 48 KiB with the
// static arrays, which are below 8 KiB.
template <auto kernel>
bool allow_smem(size_t bytes) {
    if (bytes <= 40 * 1024) return true;
    constexpr int kMaxDevices = 64;
    static std::atomic<size_t> allowed[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return false;
    if (dev < kMaxDevices && allowed[dev].load(std::memory_order_acquire) >= bytes) return true;
    if (cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(bytes)) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    if (dev < kMaxDevices) allowed[dev].store(bytes, std::memory_order_release);
    return true;
}

nvfp4_status clear_amax(uint32_t* amax, unsigned grid, cudaStream_t stream) {
    return amax && grid > 1 && cudaMemsetAsync(amax, 0, 4, stream) != cudaSuccess ? NVFP4_ERR_CUDA : NVFP4_OK;
}

template <typename T, int N, int LANES, bool SHIFTED>
nvfp4_status launch_norm(const NormArgs& a, const Cut& cut, cudaStream_t stream) {
    constexpr auto kernel = norm_kernel<T, N, LANES, SHIFTED>;
    const size_t smem = size_t(forward_stages(N * sizeof(T))) * N * sizeof(T) * cut.threads;
    if (!allow_smem<kernel>(smem)) return NVFP4_ERR_CUDA;
    const unsigned grid = static_cast<unsigned>(grid_of(cut, a.rows, int64_t(sm_count()) * resident(forward_registers(N), cut.threads), sizeof(T)));
    if (clear_amax(a.amax, grid, stream) != NVFP4_OK) return NVFP4_ERR_CUDA;
    kernel<<<grid, cut.threads, smem, stream>>>(a);
    return launched();
}

template <typename T, bool SHIFTED>
nvfp4_status dispatch_norm(const NormArgs& a, const Cut& cut, cudaStream_t stream) {
    if (cut.lanes == 8) return launch_norm<T, 8, 8, SHIFTED>(a, cut, stream);
    if (cut.lanes == 16) return launch_norm<T, 8, 16, SHIFTED>(a, cut, stream);
    if (cut.lanes == 32)
        return cut.elements == 8 ? launch_norm<T, 8, 32, SHIFTED>(a, cut, stream) : launch_norm<T, 16, 32, SHIFTED>(a, cut, stream);
    return cut.elements == 16 ? launch_norm<T, 16, 0, SHIFTED>(a, cut, stream) : launch_norm<T, 32, 0, SHIFTED>(a, cut, stream);
}

unsigned long_threads(int64_t cols) { return static_cast<unsigned>(std::min<int64_t>(1024, (cols + 31) / 32 * 32)); }

template <typename T>
nvfp4_status run_norm(const NormArgs& a, const Cut& cut, cudaStream_t stream) {
    if (cut.elements == 0) {
        const unsigned grid = static_cast<unsigned>(std::min<int64_t>(a.rows, sm_count() * 2));
        if (clear_amax(a.amax, grid, stream) != NVFP4_OK) return NVFP4_ERR_CUDA;
        norm_long_kernel<T><<<grid, long_threads(a.cols), 0, stream>>>(a);
        return launched();
    }
    return cut.shifted ? dispatch_norm<T, true>(a, cut, stream) : dispatch_norm<T, false>(a, cut, stream);
}

template <typename T, int N, int LANES, bool SHIFTED>
nvfp4_status launch_grad(const NormGradArgs& a, const Cut& cut, cudaStream_t stream) {
    constexpr auto kernel = norm_grad_kernel<T, N, LANES, SHIFTED>;
    const size_t smem = size_t(kBackwardStages) * 2 * N * sizeof(T) * cut.threads;
    if (!allow_smem<kernel>(smem)) return NVFP4_ERR_CUDA;
    kernel<<<static_cast<unsigned>(a.parts), cut.threads, smem, stream>>>(a);
    return launched();
}

template <typename T, bool SHIFTED>
nvfp4_status dispatch_grad(const NormGradArgs& a, const Cut& cut, cudaStream_t stream) {
    if (cut.lanes == 8) return launch_grad<T, 8, 8, SHIFTED>(a, cut, stream);
    if (cut.lanes == 16) return launch_grad<T, 8, 16, SHIFTED>(a, cut, stream);
    if (cut.lanes == 32)
        return cut.elements == 8 ? launch_grad<T, 8, 32, SHIFTED>(a, cut, stream) : launch_grad<T, 16, 32, SHIFTED>(a, cut, stream);
    return launch_grad<T, 16, 0, SHIFTED>(a, cut, stream);
}

template <typename T>
nvfp4_status run_grad(const NormGradArgs& a, const Cut& cut, cudaStream_t stream) {
    if (cut.elements == 0) {
        norm_grad_long_kernel<T><<<static_cast<unsigned>(std::min<int64_t>(a.rows, sm_count() * 2)), long_threads(a.cols), 0, stream>>>(a);
        if (a.sums)
            norm_sums_kernel<T><<<dim3(static_cast<unsigned>((a.cols + 255) / 256), static_cast<unsigned>(a.parts)), 256, 0,
                                  stream>>>(a);
        return launched();
    }
    return cut.shifted ? dispatch_grad<T, true>(a, cut, stream) : dispatch_grad<T, false>(a, cut, stream);
}

uintptr_t place(const void* p) { return reinterpret_cast<uintptr_t>(p) & 15; }

}  // namespace

extern "C" nvfp4_status nvfp4_layer_norm(const void* x, nvfp4_type x_type, const void* weight, const void* bias,
                                         nvfp4_type w_type, int64_t rows, int64_t cols, float eps, void* y,
                                         float* mean, float* rstd, float* amax, cudaStream_t stream) {
    if (!shape_ok(rows, cols)) return NVFP4_ERR_SHAPE;
    if (!known(x_type) || !known(w_type) || !(eps >= 0.0f) || eps > FLT_MAX) return NVFP4_ERR_VALUE;
    if (rows > 0 && (x == nullptr || y == nullptr)) return NVFP4_ERR_NULL;
    if (!aligned_to(x, type_size(x_type)) || !aligned_to(y, type_size(x_type)) ||
        !aligned_to(weight, type_size(w_type)) || !aligned_to(bias, type_size(w_type)) || !aligned_to(mean, 4) ||
        !aligned_to(rstd, 4) || !aligned_to(amax, 4))
        return NVFP4_ERR_ALIGN;
    if (rows == 0) {
        if (amax && cudaMemsetAsync(amax, 0, 4, stream) != cudaSuccess) return NVFP4_ERR_CUDA;
        return NVFP4_OK;
    }
    const Cut cut = cut_rows(cols, type_size(x_type), place(x) == 0, place(x) == place(y), 32);
    const bool vector = !cut.shifted && place(weight) == 0 && place(bias) == 0;
    const NormArgs a{x, weight, bias, w_type == NVFP4_TYPE_F32, vector, rows, static_cast<int>(cols), eps, y, mean, rstd,
                     reinterpret_cast<uint32_t*>(amax)};
    return x_type == NVFP4_TYPE_F32 ? run_norm<float>(a, cut, stream) : run_norm<bf16>(a, cut, stream);
}

extern "C" int64_t nvfp4_layer_norm_workspace(int64_t rows, int64_t cols) {
    if (!shape_ok(rows, cols)) return -1;
    if (rows == 0) return 0;
    int64_t parts = 0;   // for operands of any type and alignment
    for (const int size : {2, 4})
        for (const bool aligned : {true, false})
            for (const bool congruent : {true, false})
                parts = std::max(parts, backward_parts(cut_backward(cols, size, aligned, congruent), rows, cols, size));
    return 2 * parts * cols * 4;
}

extern "C" nvfp4_status nvfp4_layer_norm_backward(const void* dy, const void* x, nvfp4_type x_type,
                                                  const void* weight, nvfp4_type w_type, const float* mean,
                                                  const float* rstd, int64_t rows, int64_t cols, void* dx,
                                                  void* dweight, void* dbias, void* workspace,
                                                  int64_t workspace_bytes, cudaStream_t stream) {
    if (!shape_ok(rows, cols)) return NVFP4_ERR_SHAPE;
    if (!known(x_type) || !known(w_type)) return NVFP4_ERR_VALUE;
    const bool sums = dweight != nullptr || dbias != nullptr;
    if (rows > 0 && (dy == nullptr || x == nullptr || mean == nullptr || rstd == nullptr || dx == nullptr ||
                     (sums && workspace == nullptr)))
        return NVFP4_ERR_NULL;
    if (!aligned_to(dy, type_size(x_type)) || !aligned_to(x, type_size(x_type)) || !aligned_to(dx, type_size(x_type)) ||
        !aligned_to(weight, type_size(w_type)) || !aligned_to(dweight, type_size(w_type)) ||
        !aligned_to(dbias, type_size(w_type)) || !aligned_to(mean, 4) || !aligned_to(rstd, 4) ||
        (sums && !aligned_to(workspace, 16)))
        return NVFP4_ERR_ALIGN;
    if (rows == 0) {
        for (void* p : {dweight, dbias})
            if (p && cudaMemsetAsync(p, 0, static_cast<size_t>(cols) * type_size(w_type), stream) != cudaSuccess)
                return NVFP4_ERR_CUDA;
        return NVFP4_OK;
    }
    if (sums && workspace_bytes < nvfp4_layer_norm_workspace(rows, cols)) return NVFP4_ERR_SHAPE;
    const int size = type_size(x_type);
    const Cut cut = cut_backward(cols, size, place(x) == 0, place(x) == place(dy) && place(x) == place(dx));
    const bool vector = !cut.shifted && place(weight) == 0;
    const NormGradArgs a{dy, x, weight, w_type == NVFP4_TYPE_F32, vector, mean, rstd, rows, static_cast<int>(cols), dx,
                         sums ? static_cast<float*>(workspace) : nullptr, static_cast<int>(backward_parts(cut, rows, cols, size))};
    const nvfp4_status st = x_type == NVFP4_TYPE_F32 ? run_grad<float>(a, cut, stream) : run_grad<bf16>(a, cut, stream);
    if (st != NVFP4_OK || !sums) return st;
    const dim3 grid(static_cast<unsigned>((cols + 31) / 32), 2);
    if (w_type == NVFP4_TYPE_F32) {
        norm_join_kernel<float><<<grid, 256, 0, stream>>>(a.sums, a.parts, a.cols, static_cast<float*>(dweight),
                                                         static_cast<float*>(dbias));
    } else {
        norm_join_kernel<bf16><<<grid, 256, 0, stream>>>(a.sums, a.parts, a.cols, static_cast<bf16*>(dweight),
                                                        static_cast<bf16*>(dbias));
    }
    return launched();
}

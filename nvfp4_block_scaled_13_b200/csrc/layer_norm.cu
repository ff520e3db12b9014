// layer_norm.cu — layer norm forward (with the amax of its result) and backward on sm_100a.
//
// Forward, per row of x: mean = S x / C, var = S (x - mean)^2 / C, rstd = (var + eps)^-1/2,
// y = (x - mean) rstd w + b. Backward, with xh = (x - mean) rstd and h = dy w:
// dx = rstd (h - S h / C - xh S(h xh) / C), dw = S_rows dy xh, db = S_rows dy.
// Both are bound by memory: 4 bytes an element forward and 6 backward in BF16.
//
// A row is held in registers between its reduction and its result, so x (and dy) are read once.
// Rows of up to 1024 columns forward (512 backward) belong to one warp, which needs no barrier;
// longer ones to one CTA with a column range per thread. The variance is summed from the held
// row after the mean is known: no cancellation, at the price of a second reduction.
// The column sums of the backward pass stay in registers over all rows of a CTA; each CTA
// writes one partial row to the workspace and a second kernel adds the partial rows in order,
// so the result does not depend on how CTAs were scheduled.
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
    bool w_f32;
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
    bool w_f32;
    const float* mean;
    const float* rstd;
    int64_t rows;
    int cols;
    void* dx;
    float* sums;   // [2][parts][cols]: partial dweight, partial dbias
    int parts;
};

// Columns of a thread: V groups of 8. VEC: a group is 8 consecutive columns (one 16-byte load of
// BF16); otherwise column k * T + t for the k-th of its 8 V elements, so that a warp reads
// consecutive elements whatever the row's alignment.
template <bool VEC>
__device__ __forceinline__ int column(int v, int j, int t, int T) {
    return VEC ? (v * T + t) * 8 + j : (v * 8 + j) * T + t;
}

template <bool VEC, typename T>
__device__ __forceinline__ void load_group(const T* row, int cols, int v, int t, int threads, float fill,
                                           float (&out)[8]) {
    if (VEC) {
        const int c = (v * threads + t) * 8;
        if (c < cols) {
            load8(row + c, out);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) out[j] = fill;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = (v * 8 + j) * threads + t;
            out[j] = c < cols ? to_float(row[c]) : fill;
        }
    }
}

template <bool VEC, typename T>
__device__ __forceinline__ void store_group(T* row, int cols, int v, int t, int threads, const float (&in)[8]) {
    if (VEC) {
        const int c = (v * threads + t) * 8;
        if (c < cols) store8(row + c, in);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = (v * 8 + j) * threads + t;
            if (c < cols) row[c] = from_float<T>(in[j]);
        }
    }
}

// The weight's (or bias's) columns of a thread, of either type; `fill` where there is none.
template <bool VEC>
__device__ __forceinline__ void load_param(const void* p, bool f32, int cols, int v, int t, int threads, float fill,
                                           float (&out)[8]) {
    if (p == nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) out[j] = fill;
    } else if (f32) {
        load_group<VEC>(static_cast<const float*>(p), cols, v, t, threads, fill, out);
    } else {
        load_group<VEC>(static_cast<const bf16*>(p), cols, v, t, threads, fill, out);
    }
}

// Sum over the threads of a row. One barrier a reduction: `buffer` alternates, and the barrier
// of the next reduction separates this one's reads from the writes after next.
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float (*scratch)[32], int& buffer) {
    v = warp_sum(v);
    if (!WARP) {
        const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0) scratch[buffer][threadIdx.x >> 5] = v;
        __syncthreads();
        v = warp_sum(lane < warps ? scratch[buffer][lane] : 0.0f);
        buffer ^= 1;
    }
    return v;
}

__device__ __forceinline__ uint32_t stored_magnitude(float v, bf16) {
    return (uint32_t(to_bf16(v)) << 16) & 0x7FFFFFFFu;
}
__device__ __forceinline__ uint32_t stored_magnitude(float v, float) { return magnitude(v); }

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

template <typename T, int V, bool VEC, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 1024) norm_kernel(const NormArgs a) {
    __shared__ float scratch[2][32];
    const int warps = blockDim.x >> 5;
    const int threads = WARP ? 32 : blockDim.x, t = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int64_t first = WARP ? int64_t(blockIdx.x) * warps + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t step = WARP ? int64_t(gridDim.x) * warps : gridDim.x;
    const int cols = a.cols;
    const float count = static_cast<float>(cols);
    uint32_t top = 0;
    int buffer = 0;
    for (int64_t r = first; r < a.rows; r += step) {
        const T* x = static_cast<const T*>(a.x) + r * cols;
        float v[V][8];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) load_group<VEC>(x, cols, i, t, threads, 0.0f, v[i]);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += v[i][j];
        const float mean = row_sum<WARP>(sum, scratch, buffer) / count;
        float square = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] = column<VEC>(i, j, t, threads) < cols ? v[i][j] - mean : 0.0f;
                square = fmaf(v[i][j], v[i][j], square);
            }
        const float rstd = 1.0f / sqrtf(row_sum<WARP>(square, scratch, buffer) / count + a.eps);
        T* y = static_cast<T*>(a.y) + r * cols;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float w[8], b[8];
            load_param<VEC>(a.weight, a.w_f32, cols, i, t, threads, 1.0f, w);
            load_param<VEC>(a.bias, a.w_f32, cols, i, t, threads, 0.0f, b);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] = fmaf(v[i][j] * rstd, w[j], b[j]);
                if (a.amax && column<VEC>(i, j, t, threads) < cols) top = max(top, stored_magnitude(v[i][j], T{}));
            }
            store_group<VEC>(y, cols, i, t, threads, v[i]);
        }
        if (t == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
    if (a.amax) publish_amax(top, a.amax);
}

// Rows too long for the registers of one CTA: three passes, the later two from L2.
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
        const float mean = row_sum<false>(sum, scratch, buffer) / count;
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
            const float d = to_float(x[c]) - mean;
            square = fmaf(d, d, square);
        }
        const float rstd = 1.0f / sqrtf(row_sum<false>(square, scratch, buffer) / count + a.eps);
        T* y = static_cast<T*>(a.y) + r * a.cols;
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
            float w = 1.0f, b = 0.0f;
            if (a.weight) w = a.w_f32 ? static_cast<const float*>(a.weight)[c] : to_float(static_cast<const bf16*>(a.weight)[c]);
            if (a.bias) b = a.w_f32 ? static_cast<const float*>(a.bias)[c] : to_float(static_cast<const bf16*>(a.bias)[c]);
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

// Adds the column sums of the warps of a CTA in warp order and writes the CTA's partial row.
template <int V, bool VEC>
__device__ __forceinline__ void join_warps(const float (&s)[V][8], float* shared, float* out, int cols) {
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int w = 0; w < warps; ++w) {
        if (warp == w) {
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int c = column<VEC>(i, j, lane, 32);
                    if (c < cols) shared[c] = w == 0 ? s[i][j] : shared[c] + s[i][j];
                }
        }
        __syncthreads();
    }
    for (int c = threadIdx.x; c < cols; c += blockDim.x) out[c] = shared[c];
    __syncthreads();
}

template <typename T, int V, bool VEC, bool WARP, bool SUMS>
__global__ void __launch_bounds__(WARP ? 256 : 512) norm_grad_kernel(const NormGradArgs a) {
    __shared__ float scratch[2][2][32];
    __shared__ float joined[WARP ? V * 256 : 1];
    const int warps = blockDim.x >> 5;
    const int threads = WARP ? 32 : blockDim.x, t = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int64_t first = WARP ? int64_t(blockIdx.x) * warps + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t step = WARP ? int64_t(gridDim.x) * warps : gridDim.x;
    const int cols = a.cols;
    const float inv = 1.0f / static_cast<float>(cols);
    float sw[V][8], sb[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) sw[i][j] = sb[i][j] = 0.0f;
    int b1 = 0, b2 = 0;
    for (int64_t r = first; r < a.rows; r += step) {
        const T* x = static_cast<const T*>(a.x) + r * cols;
        const T* dy = static_cast<const T*>(a.dy) + r * cols;
        const float mean = a.mean[r], rstd = a.rstd[r];
        float xh[V][8], h[V][8];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            load_group<VEC>(x, cols, i, t, threads, 0.0f, xh[i]);
            load_group<VEC>(dy, cols, i, t, threads, 0.0f, h[i]);
        }
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float w[8];
            load_param<VEC>(a.weight, a.w_f32, cols, i, t, threads, 1.0f, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                xh[i][j] = column<VEC>(i, j, t, threads) < cols ? (xh[i][j] - mean) * rstd : 0.0f;
                if (SUMS) {
                    sw[i][j] = fmaf(h[i][j], xh[i][j], sw[i][j]);
                    sb[i][j] += h[i][j];
                }
                h[i][j] *= w[j];
                s1 += h[i][j];
                s2 = fmaf(h[i][j], xh[i][j], s2);
            }
        }
        s1 = row_sum<WARP>(s1, scratch[0], b1) * inv;
        s2 = row_sum<WARP>(s2, scratch[1], b2) * inv;
        T* dx = static_cast<T*>(a.dx) + r * cols;
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] = rstd * (h[i][j] - fmaf(xh[i][j], s2, s1));
            store_group<VEC>(dx, cols, i, t, threads, h[i]);
        }
    }
    if (SUMS) {
        float* out = a.sums + int64_t(blockIdx.x) * cols;
        float* out_b = out + int64_t(a.parts) * cols;
        if (WARP) {
            join_warps<V, VEC>(sw, joined, out, cols);
            join_warps<V, VEC>(sb, joined, out_b, cols);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                store_group<VEC>(out, cols, i, t, threads, sw[i]);
                store_group<VEC>(out_b, cols, i, t, threads, sb[i]);
            }
        }
    }
}

// dx of rows too long for the registers of one CTA: two passes, the second from L2.
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
            if (a.weight) w = a.w_f32 ? static_cast<const float*>(a.weight)[c] : to_float(static_cast<const bf16*>(a.weight)[c]);
            return to_float(dy[c]) * w;
        };
        float s1 = 0.0f, s2 = 0.0f;
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
            const float h = scaled(c);
            s1 += h;
            s2 = fmaf(h, (to_float(x[c]) - mean) * rstd, s2);
        }
        s1 = row_sum<false>(s1, scratch[0], b1) * inv;
        s2 = row_sum<false>(s2, scratch[1], b2) * inv;
        T* dx = static_cast<T*>(a.dx) + r * a.cols;
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x)
            dx[c] = from_float<T>(rstd * (scaled(c) - fmaf((to_float(x[c]) - mean) * rstd, s2, s1)));
    }
}

// Column sums of such rows: one column a thread, one slab of rows a grid row.
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
size_t type_size(nvfp4_type t) { return t == NVFP4_TYPE_F32 ? 4 : 2; }

bool shape_ok(int64_t rows, int64_t cols) {
    return rows >= 0 && cols >= 1 && cols <= (int64_t(1) << 30) && (rows == 0 || cols <= (int64_t(1) << 60) / rows);
}

// Rows of a multiple of 8 columns whose every operand starts on 16 bytes take the vector path.
bool vector_rows(int64_t cols, std::initializer_list<const void*> ptrs) {
    if (cols % 8 != 0) return false;
    for (const void* p : ptrs)
        if (!aligned_to(p, 16)) return false;
    return true;
}

nvfp4_status launched() { return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA; }

// How a row is cut: `groups` of 8 columns a thread, `threads` a row (32: one warp, several rows
// a CTA).
struct Cut {
    int groups, threads;
    bool warp, fits;
};

Cut cut_forward(int64_t cols) {
    const int64_t octets = (cols + 7) / 8;
    if (octets <= 128) return {octets <= 32 ? 1 : octets <= 64 ? 2 : 4, 32, true, true};
    const int groups = octets <= 2048 ? 2 : 4;
    const int64_t threads = ((octets + groups - 1) / groups + 31) / 32 * 32;
    return {groups, static_cast<int>(threads), false, threads <= 1024};
}

Cut cut_backward(int64_t cols) {
    const int64_t octets = (cols + 7) / 8;
    if (octets <= 64) return {octets <= 32 ? 1 : 2, 32, true, true};
    const int groups = octets <= 256 ? 1 : 2;
    const int64_t threads = ((octets + groups - 1) / groups + 31) / 32 * 32;
    return {groups, static_cast<int>(threads), false, threads <= 512};
}

// CTAs of the backward pass, each of which leaves a partial row.
int64_t backward_parts(int64_t rows, int64_t cols) {
    const Cut cut = cut_backward(cols);
    const int64_t sms = sm_count();
    if (!cut.fits) {
        const int64_t across = (cols + 255) / 256;
        return std::min<int64_t>(rows, std::max<int64_t>(1, 4 * sms / across));
    }
    const int64_t units = cut.warp ? (rows + 7) / 8 : rows;
    const int64_t per_sm = cut.warp ? 2 : std::max(1, 512 / cut.threads);
    return std::min(units, sms * per_sm);
}

template <typename T, int V, bool VEC>
nvfp4_status launch_norm(const NormArgs& a, const Cut& cut, cudaStream_t stream) {
    const int64_t sms = sm_count();
    if (cut.warp) {
        const unsigned grid = static_cast<unsigned>(std::min<int64_t>((a.rows + 7) / 8, sms * 8));
        if (a.amax && grid > 1 && cudaMemsetAsync(a.amax, 0, 4, stream) != cudaSuccess) return NVFP4_ERR_CUDA;
        norm_kernel<T, V, VEC, true><<<grid, 256, 0, stream>>>(a);
    } else {
        const unsigned grid = static_cast<unsigned>(std::min<int64_t>(a.rows, sms * std::max(1, 2048 / cut.threads)));
        if (a.amax && grid > 1 && cudaMemsetAsync(a.amax, 0, 4, stream) != cudaSuccess) return NVFP4_ERR_CUDA;
        norm_kernel<T, V, VEC, false><<<grid, cut.threads, 0, stream>>>(a);
    }
    return launched();
}

template <typename T>
nvfp4_status dispatch_norm(const NormArgs& a, bool vec, cudaStream_t stream) {
    const Cut cut = cut_forward(a.cols);
    if (!cut.fits) {
        const unsigned grid = static_cast<unsigned>(std::min<int64_t>(a.rows, sm_count() * 2));
        if (a.amax && grid > 1 && cudaMemsetAsync(a.amax, 0, 4, stream) != cudaSuccess) return NVFP4_ERR_CUDA;
        norm_long_kernel<T><<<grid, 1024, 0, stream>>>(a);
        return launched();
    }
    switch (cut.groups) {
        case 1: return vec ? launch_norm<T, 1, true>(a, cut, stream) : launch_norm<T, 1, false>(a, cut, stream);
        case 2: return vec ? launch_norm<T, 2, true>(a, cut, stream) : launch_norm<T, 2, false>(a, cut, stream);
        default: return vec ? launch_norm<T, 4, true>(a, cut, stream) : launch_norm<T, 4, false>(a, cut, stream);
    }
}

template <typename T, int V, bool VEC>
nvfp4_status launch_grad(const NormGradArgs& a, const Cut& cut, bool sums, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>(a.parts);
    if (cut.warp) {
        if (sums) {
            norm_grad_kernel<T, V, VEC, true, true><<<grid, 256, 0, stream>>>(a);
        } else {
            norm_grad_kernel<T, V, VEC, true, false><<<grid, 256, 0, stream>>>(a);
        }
    } else if (sums) {
        norm_grad_kernel<T, V, VEC, false, true><<<grid, cut.threads, 0, stream>>>(a);
    } else {
        norm_grad_kernel<T, V, VEC, false, false><<<grid, cut.threads, 0, stream>>>(a);
    }
    return launched();
}

template <typename T>
nvfp4_status dispatch_grad(const NormGradArgs& a, bool vec, bool sums, cudaStream_t stream) {
    const Cut cut = cut_backward(a.cols);
    if (!cut.fits) {
        norm_grad_long_kernel<T><<<static_cast<unsigned>(std::min<int64_t>(a.rows, sm_count() * 2)), 1024, 0, stream>>>(a);
        if (sums)
            norm_sums_kernel<T><<<dim3(static_cast<unsigned>((a.cols + 255) / 256), static_cast<unsigned>(a.parts)), 256, 0,
                                  stream>>>(a);
        return launched();
    }
    if (cut.groups == 1)
        return vec ? launch_grad<T, 1, true>(a, cut, sums, stream) : launch_grad<T, 1, false>(a, cut, sums, stream);
    return vec ? launch_grad<T, 2, true>(a, cut, sums, stream) : launch_grad<T, 2, false>(a, cut, sums, stream);
}

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
    const NormArgs a{x, weight, bias, w_type == NVFP4_TYPE_F32, rows, static_cast<int>(cols), eps, y, mean, rstd,
                     reinterpret_cast<uint32_t*>(amax)};
    const bool vec = vector_rows(cols, {x, y, weight, bias});
    return x_type == NVFP4_TYPE_F32 ? dispatch_norm<float>(a, vec, stream) : dispatch_norm<bf16>(a, vec, stream);
}

extern "C" int64_t nvfp4_layer_norm_workspace(int64_t rows, int64_t cols) {
    if (!shape_ok(rows, cols)) return -1;
    return rows == 0 ? 0 : 2 * backward_parts(rows, cols) * cols * 4;
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
    const int64_t parts = backward_parts(rows, cols);
    if (sums && workspace_bytes < 2 * parts * cols * 4) return NVFP4_ERR_SHAPE;
    const NormGradArgs a{dy, x, weight, w_type == NVFP4_TYPE_F32, mean, rstd, rows, static_cast<int>(cols), dx,
                         static_cast<float*>(workspace), static_cast<int>(parts)};
    const bool vec = vector_rows(cols, {dy, x, dx, weight});
    const nvfp4_status st =
        x_type == NVFP4_TYPE_F32 ? dispatch_grad<float>(a, vec, sums, stream) : dispatch_grad<bf16>(a, vec, sums, stream);
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

// layer_norm.cu — layer norm forward (with the amax of its result) and backward on sm_100a.
//
// Forward, per row of x: mean = S x / C, var = S (x - mean)^2 / C, rstd = (var + eps)^-1/2,
// y = (x - mean) rstd w + b. Backward, with xh = (x - mean) rstd and h = dy w:
// dx = rstd (h - S h / C - xh S(h xh) / C), dw = S_rows dy xh, db = S_rows dy.
// Both are bound by memory: 4 bytes an element forward and 6 backward in BF16 (8192 x 4096 on the
// device: 25.7 us with the amax, where a copy of the same size takes 22.3; 41.9 us backward, 73% of the
// copy bandwidth. FP32, 4096 x 4096: 24.7 and 36.3 us, 83% and 85%).
//
// A row belongs to a group of threads: 8, 16 or 32 lanes of a warp (no barrier), some warps of a CTA,
// or a cluster of CTAs that exchange their sums through shared memory. A thread holds its share of the row in registers from the loads to the result, so x (and dy) are
// read once, and holds its columns' weight and bias (and their gradients' sums) over all the rows
// that its group works through. The variance is summed from the held row after the mean is
// known: no cancellation, at the price of a second reduction.
//
// Rows arrive ahead of their use through a ring in shared memory. Each thread copies (cp.async)
// and later reads its own 16-byte units only, so the ring needs no barrier and no registers.
//
// A row that does not start on 16 bytes has a head of up to 7 elements, whole units, and a tail; the
// first threads of its group take an element of each beside their units. Groups take rows in steps
// whose length in bytes is a multiple of 16, so a group's head, and with it the columns of each
// thread, stays the same: odd row lengths run on the same vector path. (8192 x 4095 in BF16: 30 us
// forward and 57 backward; with masked first and last units, on which a whole group waits, 35 and 74.)
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
    int row_threads;   // of norm_group_kernel where a row has a CTA or a cluster
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
    int row_threads;
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
    for (const uint32_t v : {w.x, w.y, w.z, w.w})   // NaN stays
        asm("{\n\t.reg .b32 m;\n\tabs.bf16x2 m, %1;\n\tmax.NaN.bf16x2 %0, %0, m;\n\t}" : "+r"(top) : "r"(v));
}
__device__ __forceinline__ void join_top(uint32_t& top, const uint4& w, float) {
    top = max(max(top, w.x & 0x7FFFFFFFu), max(w.y & 0x7FFFFFFFu, max(w.z & 0x7FFFFFFFu, w.w & 0x7FFFFFFFu)));
}
__device__ __forceinline__ void join_top(uint32_t& top, float2 v, bf16) {
    join_top(top, make_uint4(to_bf16x2(v.x, v.y), 0u, 0u, 0u), bf16{});
}
__device__ __forceinline__ void join_top(uint32_t& top, float2 v, float) {
    top = max(top, max(magnitude(v.x), magnitude(v.y)));
}
__device__ __forceinline__ uint32_t top_bits(uint32_t top, bf16) { return max(top << 16, top & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t top_bits(uint32_t top, float) { return top; }

__device__ __forceinline__ void copy_async(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ uint4 read_shared(uint32_t from) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(from) : "memory");
    return v;
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// The columns of a thread: unit q holds columns start(q) .. start(q) + E - 1, if the row has them.
template <typename T, int Q>
struct Columns {
    static constexpr int E = kUnit<T>;
    int base, stride, cols;

    __device__ __forceinline__ Columns(int t, int lanes, int head, int cols_) : base(t * E + head), stride(lanes * E), cols(cols_) {}
    __device__ __forceinline__ int start(int q) const { return base + q * stride; }
    __device__ __forceinline__ bool has(int q) const { return start(q) + E <= cols; }
};

// Elements in front of the first 16-byte boundary of the row at `p`.
template <typename T>
__device__ __forceinline__ int head_of(uintptr_t p, int cols) {
    return min(cols, static_cast<int>((0 - p & 15) / sizeof(T)));
}

// A thread's share of the head and the tail of a shifted row: one element of each, if there is one.
template <typename T, bool SHIFTED>
struct Edge {
    bool any;        // for most threads there is none, and whole warps skip what is done about it
    bool has[2];
    int column[2];

    __device__ __forceinline__ Edge(int t, int head, int cols) {
        const int body = (cols - head) / kUnit<T> * kUnit<T>;
        has[0] = SHIFTED && t < head;
        has[1] = SHIFTED && t < cols - head - body;
        any = has[0] || has[1];
        column[0] = t;
        column[1] = head + body + t;
    }
    __device__ __forceinline__ void load(const void* row, float2& v) const {
        if (!SHIFTED) return;
        v.x = has[0] ? to_float(static_cast<const T*>(row)[column[0]]) : 0.0f;
        v.y = has[1] ? to_float(static_cast<const T*>(row)[column[1]]) : 0.0f;
    }
    __device__ __forceinline__ float2 param(const void* p, bool f32, float fill) const;
    // Zero in the place of an element that does not exist.
    __device__ __forceinline__ float2 keep(float2 v) const { return make_float2(has[0] ? v.x : 0.0f, has[1] ? v.y : 0.0f); }
    __device__ __forceinline__ void store(void* row, float2 v) const {
        if (has[0]) static_cast<T*>(row)[column[0]] = from_float<T>(v.x);
        if (has[1]) static_cast<T*>(row)[column[1]] = from_float<T>(v.y);
    }
};

template <int H>
__device__ __forceinline__ void keep_if(bool has, float2 (&v)[H]) {
#pragma unroll
    for (int k = 0; k < H; ++k) v[k] = has ? v[k] : make_float2(0.0f, 0.0f);
}

__device__ __forceinline__ float param_at(const void* p, bool f32, int c) {
    return f32 ? static_cast<const float*>(p)[c] : to_float(static_cast<const bf16*>(p)[c]);
}

// The weight's (or bias's) values of a unit; `fill` in every existing column where there is no
// parameter, zero in a unit that does not exist.
template <int E>
__device__ __forceinline__ void load_param(const void* p, bool f32, bool vector, int c, bool has, float fill, float2 (&out)[E / 2]) {
    float v[E];
    if (p == nullptr || !has || !vector) {
#pragma unroll
        for (int j = 0; j < E; ++j) v[j] = has ? (p ? param_at(p, f32, c + j) : fill) : 0.0f;
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

template <typename T, bool SHIFTED>
__device__ __forceinline__ float2 Edge<T, SHIFTED>::param(const void* p, bool f32, float fill) const {
    return make_float2(has[0] ? (p ? param_at(p, f32, column[0]) : fill) : 0.0f, has[1] ? (p ? param_at(p, f32, column[1]) : fill) : 0.0f);
}

// ---- sums over a row's threads ------------------------------------------------------------

template <int LANES>
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
    for (int off = (LANES > 0 ? LANES : 32) / 2; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
    return v;
}

// LANES of a row that has a CTA, a cluster of CTAs, or some warps of a CTA (`row_threads`).
constexpr int kCta = 0, kCluster = -1, kRows = -2;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int LANES>
__device__ __forceinline__ void sync_all() {
    if (LANES == kCluster) {
        cluster_sync();
    } else {
        __syncthreads();
    }
}

// Partial sums of the warps of a row, in two sets that alternate: the barrier of the next
// reduction separates this one's reads from the writes after next, so a reduction has one
// barrier. In a cluster every warp leaves its sum in the shared memory of every CTA; row groups
// inside a CTA (kRows, of at most four warps) have 16 places and a barrier each.
template <int LANES>
struct WarpSums {
    static constexpr int kFours = LANES == kCta ? 4 : 32;   // 16 warps; 8 CTAs of 16 warps, or 8 groups of 16 places
    float4 set[2][kFours];

    __device__ __forceinline__ void clear() {
        for (int k = threadIdx.x; k < 2 * kFours; k += blockDim.x) (&set[0][0])[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    __device__ __forceinline__ void put(int which, int group, int t, float v) {
        float* to = reinterpret_cast<float*>(set[which]);
        const int lane = threadIdx.x & 31;
        if (LANES == kCluster) {
            if (lane < static_cast<int>(cluster_size())) {
                const uint32_t at =
                    static_cast<uint32_t>(__cvta_generic_to_shared(to + cluster_rank() * (blockDim.x >> 5) + (threadIdx.x >> 5)));
                uint32_t remote;
                asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(at), "r"(lane));
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(remote), "f"(v) : "memory");
            }
        } else if (lane == 0) {
            to[LANES == kRows ? group * 16 + (t >> 5) : threadIdx.x >> 5] = v;
        }
    }
    static __device__ __forceinline__ void sync(int group, int row_threads) {
        if (LANES == kRows) {
            asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(row_threads) : "memory");
        } else {
            sync_all<LANES>();
        }
    }
    __device__ __forceinline__ float four(int which, int k) const {
        const float4 p = set[which][k];
        return (p.x + p.y) + (p.z + p.w);
    }
    __device__ __forceinline__ float total(int which, int group, int row_threads) const {
        if (LANES == kCluster) return warp_sum(four(which, threadIdx.x & 31));
        if (LANES == kRows) return four(which, group * 4);   // at most four warps
        float s = four(which, 0);
        if (blockDim.x > 128) s += four(which, 1);
        if (blockDim.x > 256) s += four(which, 2) + four(which, 3);
        return s;
    }
};

// Programmatic dependent launch: a kernel launched with it may start while its predecessor runs;
// it waits for the predecessor's end before it touches what that wrote.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

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
                wait_for_previous();   // the kernel that clears it
                atomicMax(amax, top);
            }
        }
    }
}

// ---- forward -------------------------------------------------------------------------------

constexpr int kForwardStages = 4;   // rows in the ring
// Backward: three (four and six were no faster).
constexpr int kBackwardStages = 3;

// Registers of a thread, and with them the CTAs that an SM holds (each of its four quarters has
// 16384 registers).
constexpr int forward_registers(int elements) { return elements == 16 ? 80 : 64; }
constexpr int kBackwardRegisters = 128;   // shifted rows in groups of a CTA (kRows) spill 104 to 116 bytes beside it
constexpr int resident(int registers, int threads) {
    return std::max(1, std::min(32, 16384 / (registers * 32) * 4 / (threads / 32)));
}

// Which rows a thread's group takes: the groups of a CTA take every ctas-th row in turn, which gives
// all of them one head.
template <typename T, int LANES, bool SHIFTED>
struct Group {
    int lanes, t, groups, index;
    int64_t first, step;
    int turns, rows;   // turns of the CTA's loop (the shuffles need every lane of a warp), rows of the group
    int head;
    int part;          // index of the CTA, or cluster, and of its partial row

    __device__ __forceinline__ Group(const void* x, int64_t all_rows, int cols, int row_threads) {
        constexpr unsigned L = LANES > 0 ? LANES : 1;
        int64_t base = blockIdx.x, ctas = gridDim.x;
        const unsigned l = LANES > 0 ? L : LANES == kRows ? row_threads : blockDim.x;
        lanes = static_cast<int>(l);
        index = LANES > 0 || LANES == kRows ? static_cast<int>(threadIdx.x / l) : 0;
        groups = LANES > 0 || LANES == kRows ? static_cast<int>(blockDim.x / l) : 1;
        t = static_cast<int>(threadIdx.x) - index * lanes;
        if (LANES == kCluster) {
            const int size = static_cast<int>(cluster_size());
            t += static_cast<int>(cluster_rank() * blockDim.x);
            lanes *= size;
            base /= size;
            ctas /= size;
        }
        part = static_cast<int>(base);
        first = base + index * ctas;
        step = ctas * groups;
        turns = static_cast<int>((all_rows - base + step - 1) / step);
        rows = first < all_rows ? static_cast<int>((all_rows - first + step - 1) / step) : 0;
        head = SHIFTED ? head_of<T>(reinterpret_cast<uintptr_t>(x) + first * cols * int64_t(sizeof(T)), cols) : 0;
    }
};

// N elements a thread; LANES threads a row, or kCta, or kCluster.
template <typename T, int N, int LANES, bool SHIFTED>
__global__ void __maxnreg__(forward_registers(N)) norm_group_kernel(const __grid_constant__ NormArgs a) {
    constexpr int E = kUnit<T>, Q = N / E, H = E / 2, S = kForwardStages;
    extern __shared__ uint4 ring[];   // [S][Q][threads]
    __shared__ WarpSums<LANES> warp_sums;
    const Group<T, LANES, SHIFTED> group(a.x, a.rows, a.cols, a.row_threads);
    const Columns<T, Q> at(group.t, group.lanes, group.head, a.cols);
    const Edge<T, SHIFTED> edge(group.t, group.head, a.cols);
    bool has[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) has[q] = at.has(q);
    const uint32_t unit_bytes = group.lanes * 16u, slot_bytes = blockDim.x * 16u;
    const uint32_t slots = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + threadIdx.x * 16u;
    const uint32_t slots_end = slots + S * Q * slot_bytes;
    const int64_t row_bytes = group.step * a.cols * int64_t(sizeof(T));
    const char* row = static_cast<const char*>(a.x) + group.first * a.cols * int64_t(sizeof(T));   // for the edges
    const char* next = row + at.start(0) * int(sizeof(T));
    int ahead = 0;   // rows whose copy has been started
    const auto fetch = [&](uint32_t slot) {
        if (ahead < group.rows) {
#pragma unroll
            for (int q = 0; q < Q; ++q)
                if (has[q]) copy_async(slot + q * slot_bytes, next + q * unit_bytes);
        }
        ++ahead;
        next += row_bytes;
        commit_copies();
    };
#pragma unroll
    for (int s = 0; s < S - 1; ++s) fetch(slots + s * Q * slot_bytes);
    float2 w[Q][H], b[Q][H];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        load_param<E>(a.weight, a.w_f32, a.w_vector, at.start(q), has[q], 1.0f, w[q]);
        load_param<E>(a.bias, a.w_f32, a.w_vector, at.start(q), has[q], 0.0f, b[q]);
    }
    const float2 edge_w = edge.param(a.weight, a.w_f32, 1.0f), edge_b = edge.param(a.bias, a.w_f32, 0.0f);
    float2 edge_next = make_float2(0.0f, 0.0f);
    if (group.rows > 0) edge.load(row, edge_next);
    if (LANES <= 0) {
        warp_sums.clear();
        sync_all<LANES>();
    }
    const float inv = 1.0f / static_cast<float>(a.cols), eps = a.eps;
    char* y = static_cast<char*>(a.y) + group.first * a.cols * int64_t(sizeof(T));
    const int y_first = at.start(0) * int(sizeof(T));
    const bool stats = group.t == 0 && (a.mean || a.rstd), tops = a.amax;
    uint32_t top = 0;
    uint32_t slot = slots, refill = slots + (S - 1) * Q * slot_bytes;
    for (int turn = 0; turn < group.turns; ++turn) {
        wait_copies<S - 2>();
        float2 v[Q][H];
        float2 sum2[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            unpack(read_shared(slot + q * slot_bytes), v[q], T{});
            keep_if(has[q], v[q]);
#pragma unroll
            for (int k = 0; k < H; ++k) sum2[k & 1] = add2(sum2[k & 1], v[q][k]);
        }
        float2 e = edge_next;
        if (SHIFTED && edge.any) {
            sum2[0] = add2(sum2[0], e);
            row += row_bytes;
            if (turn + 1 < group.rows) edge.load(row, edge_next);
        }
        fetch(refill);
        refill = slot;
        slot += Q * slot_bytes;
        if (slot == slots_end) slot = slots;
        sum2[0] = add2(sum2[0], sum2[1]);
        float sum = lane_sum<LANES>(sum2[0].x + sum2[0].y);
        if (LANES <= 0) {
            warp_sums.put(0, group.index, group.t, sum);
            warp_sums.sync(group.index, a.row_threads);
            sum = warp_sums.total(0, group.index, a.row_threads);
        }
        const float mean = sum * inv;
        float2 square2[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int q = 0; q < Q; ++q) {
#pragma unroll
            for (int k = 0; k < H; ++k) v[q][k] = add2(v[q][k], make_float2(-mean, -mean));
            keep_if(has[q], v[q]);
#pragma unroll
            for (int k = 0; k < H; ++k) square2[k & 1] = fma2(v[q][k], v[q][k], square2[k & 1]);
        }
        if (SHIFTED && edge.any) {
            e = edge.keep(add2(e, make_float2(-mean, -mean)));
            square2[0] = fma2(e, e, square2[0]);
        }
        square2[0] = add2(square2[0], square2[1]);
        float square = lane_sum<LANES>(square2[0].x + square2[0].y);
        if (LANES <= 0) {
            warp_sums.put(1, group.index, group.t, square);
            warp_sums.sync(group.index, a.row_threads);
            square = warp_sums.total(1, group.index, a.row_threads);
        }
        const float rstd = rsqrtf(fmaf(square, inv, eps));
        if (LANES <= 0 || turn < group.rows) {
#pragma unroll
            for (int q = 0; q < Q; ++q) {
#pragma unroll
                for (int k = 0; k < H; ++k) v[q][k] = fma2(mul2(v[q][k], make_float2(rstd, rstd)), w[q][k], b[q][k]);
                const uint4 out = pack(v[q], T{});
                if (tops) join_top(top, out, T{});   // columns that do not exist hold zero
                if (has[q]) *reinterpret_cast<uint4*>(y + y_first + q * unit_bytes) = out;
            }
            if (SHIFTED && edge.any) {
                e = fma2(mul2(e, make_float2(rstd, rstd)), edge_w, edge_b);
                if (tops) join_top(top, e, T{});
                edge.store(y, e);
            }
            if (stats) {
                const int64_t r = group.first + turn * group.step;
                if (a.mean) a.mean[r] = mean;
                if (a.rstd) a.rstd[r] = rstd;
            }
        }
        y += row_bytes;
    }
    wait_copies<0>();
    if (a.amax) publish_amax(top_bits(top, T{}), a.amax);
}

// Rows of 257 to 10240 columns. With few elements a thread, the two reductions, the barriers and
// the loop cost more instructions than the elements do and bound the kernel (measured at 8192 x
// 4096 in BF16: 16.6 instructions an element and 29 us with 16 elements a thread). Here a row
// belongs to WARPS warps with N elements a lane, one CTA of 16 warps has
// an SM to itself (as many row groups as fit), and weight and bias stay in its shared memory as
// binary32, so that registers hold nothing but the row. The row groups of a CTA take every
// gridDim.x-th row, which gives all of them one head.
template <int WARPS>
constexpr int kWideThreads = 16 / WARPS * WARPS * 32;   // whole row groups
// Rows in the ring: four where a row is so short that two are little to have on the way (BF16 of 257 to
// 512 columns; 30000 x 257 takes 15.7 us, 16384 x 512 9.6 us).
template <typename T, int Q>
constexpr int kWideStages = Q <= 2 ? 4 : sizeof(T) == 2 || Q <= 8 ? 2 : 1;
template <typename T, int Q>
constexpr int kWideCtas = Q * 16 <= 32 ? 2 : 1;                           // CTAs of an SM

// Q units a lane, of which those from K on may not exist.
template <typename T, int Q, int K, int WARPS, bool SHIFTED>
__global__ void __launch_bounds__(kWideThreads<WARPS>, kWideCtas<T, Q>) norm_kernel(const __grid_constant__ NormArgs a) {
    constexpr int E = kUnit<T>, H = E / 2, P = E / 4, S = kWideStages<T, Q>;
    constexpr int kUnits = WARPS * 32 * Q, kGroups = 16 / WARPS;
    constexpr uint32_t kSlot = 512, kStage = Q * kSlot;
    extern __shared__ uint4 ring[];   // rows [warp][S][Q][lane], then weight [P][kUnits], bias [P][kUnits]
    __shared__ float sums[2][kGroups][WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = warp / WARPS, t = (warp % WARPS) * 32 + lane;
    float4* weights = reinterpret_cast<float4*>(ring + 16 * S * Q * 32);
    float4* biases = weights + P * kUnits;
    const uintptr_t place = reinterpret_cast<uintptr_t>(a.x) + blockIdx.x * (a.cols * uintptr_t(sizeof(T)));
    const int head = SHIFTED ? head_of<T>(place, a.cols) : 0;
    const Columns<T, Q> at(t, WARPS * 32, head, a.cols);
    const Edge<T, SHIFTED> edge(t, head, a.cols);
    const auto has = [&](int q) { return q < K || at.has(q); };
    const int64_t first = blockIdx.x + int64_t(group) * gridDim.x, step = int64_t(gridDim.x) * kGroups;
    const int rows = first < a.rows ? static_cast<int>((a.rows - first + step - 1) / step) : 0;
    const int64_t row_bytes = step * a.cols * int64_t(sizeof(T));
    constexpr uint32_t kUnitBytes = WARPS * 512;

    const char* row = static_cast<const char*>(a.x) + first * a.cols * int64_t(sizeof(T));   // for the edges
    const char* next = row + at.start(0) * int(sizeof(T));
    const uint32_t slots = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + warp * (S * kStage) + lane * 16u;
    int ahead = 0;
    const auto fetch = [&](uint32_t slot) {
        if (ahead < rows) {
#pragma unroll
            for (int q = 0; q < Q; ++q)
                if (has(q)) copy_async(slot + q * kSlot, next + q * kUnitBytes);
        }
        ++ahead;
        next += row_bytes;
        commit_copies();
    };
#pragma unroll
    for (int s = 0; s < S; ++s) fetch(slots + s * kStage);
    for (int u = threadIdx.x; u < kUnits; u += kWideThreads<WARPS>) {
        const Columns<T, 1> one(u, 0, head, a.cols);
        float2 w[H], b[H];
        load_param<E>(a.weight, a.w_f32, a.w_vector, one.start(0), one.has(0), 1.0f, w);
        load_param<E>(a.bias, a.w_f32, a.w_vector, one.start(0), one.has(0), 0.0f, b);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            weights[p * kUnits + u] = make_float4(w[2 * p].x, w[2 * p].y, w[2 * p + 1].x, w[2 * p + 1].y);
            biases[p * kUnits + u] = make_float4(b[2 * p].x, b[2 * p].y, b[2 * p + 1].x, b[2 * p + 1].y);
        }
    }
    const float2 edge_w = edge.param(a.weight, a.w_f32, 1.0f), edge_b = edge.param(a.bias, a.w_f32, 0.0f);
    float2 edge_next = make_float2(0.0f, 0.0f);
    if (rows > 0) edge.load(row, edge_next);
    __syncthreads();
    const float inv = 1.0f / static_cast<float>(a.cols), eps = a.eps;
    char* y = static_cast<char*>(a.y) + first * a.cols * int64_t(sizeof(T));
    const int y_first = at.start(0) * int(sizeof(T));
    const bool stats = t == 0 && (a.mean || a.rstd), tops = a.amax;
    // Sum over the row's warps; the two sets alternate as those of WarpSums do.
    const auto row_sum = [&](float v, int which) {
        v = warp_sum(v);
        if (WARPS > 1) {
            if (lane == 0) sums[which][group][warp % WARPS] = v;
            asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(WARPS * 32) : "memory");
            v = sums[which][group][0];
#pragma unroll
            for (int k = 1; k < WARPS; ++k) v += sums[which][group][k];
        }
        return v;
    };
    uint32_t top = 0;
    uint32_t slot = slots;
    for (int turn = 0; turn < rows; ++turn) {
        wait_copies<S - 1>();
        float2 v[Q][H];
        float2 part[4] = {};
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            unpack(read_shared(slot + q * kSlot), v[q], T{});
            keep_if(has(q), v[q]);
#pragma unroll
            for (int k = 0; k < H; ++k) part[k % 4] = add2(part[k % 4], v[q][k]);
        }
        float2 e = edge_next;
        if (SHIFTED && edge.any) {
            part[0] = add2(part[0], e);
            row += row_bytes;
            if (turn + 1 < rows) edge.load(row, edge_next);
        }
        fetch(slot);
        slot += kStage;
        if (slot == slots + S * kStage) slot = slots;
        part[0] = add2(add2(part[0], part[1]), add2(part[2], part[3]));
        const float mean = row_sum(part[0].x + part[0].y, 0) * inv;
        float2 square[4] = {};
#pragma unroll
        for (int q = 0; q < Q; ++q) {
#pragma unroll
            for (int k = 0; k < H; ++k) v[q][k] = add2(v[q][k], make_float2(-mean, -mean));
            keep_if(has(q), v[q]);
#pragma unroll
            for (int k = 0; k < H; ++k) square[k % 4] = fma2(v[q][k], v[q][k], square[k % 4]);
        }
        if (SHIFTED && edge.any) {
            e = edge.keep(add2(e, make_float2(-mean, -mean)));
            square[0] = fma2(e, e, square[0]);
        }
        square[0] = add2(add2(square[0], square[1]), add2(square[2], square[3]));
        const float rstd = rsqrtf(fmaf(row_sum(square[0].x + square[0].y, 1), inv, eps));
#pragma unroll
        for (int q = 0; q < Q; ++q) {
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const float4 w = weights[p * kUnits + q * (WARPS * 32) + t], b = biases[p * kUnits + q * (WARPS * 32) + t];
                v[q][2 * p] = fma2(mul2(v[q][2 * p], make_float2(rstd, rstd)), make_float2(w.x, w.y), make_float2(b.x, b.y));
                v[q][2 * p + 1] = fma2(mul2(v[q][2 * p + 1], make_float2(rstd, rstd)), make_float2(w.z, w.w), make_float2(b.z, b.w));
            }
            const uint4 out = pack(v[q], T{});
            if (tops) join_top(top, out, T{});   // columns that do not exist hold zero
            if (has(q)) *reinterpret_cast<uint4*>(y + y_first + q * kUnitBytes) = out;
        }
        if (SHIFTED && edge.any) {
            e = fma2(mul2(e, make_float2(rstd, rstd)), edge_w, edge_b);
            if (tops) join_top(top, e, T{});
            edge.store(y, e);
        }
        if (stats) {
            const int64_t r = first + turn * step;
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
        y += row_bytes;
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

// Rows of over 65536 columns, and operands whose rows start at different places within 16 bytes: three
// passes by the element, the later two from L1 or L2. The second costs a factor of five: 8192 x 4096
// in BF16 with x one element past a boundary and y on one takes 141 us (25.7 where both lie on one),
// 245 backward (41.9).
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

// Adds the column sums of the row groups of a CTA, first those of a warp, and writes the CTA's
// partial row. `shared`: [warps][cols].
template <typename T, int Q, int LANES, bool SHIFTED>
__device__ __forceinline__ void join_groups(float2 (&s)[Q][kUnit<T> / 2], float2 edges, const Columns<T, Q>& at,
                                            const Edge<T, SHIFTED>& edge, float* shared, float* out) {
    constexpr int E = kUnit<T>;
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();   // nobody uses the shared memory any more
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const bool has = at.has(q);
#pragma unroll
        for (int j = 0; j < E; ++j) {
            float v = j & 1 ? s[q][j / 2].y : s[q][j / 2].x;
#pragma unroll
            for (int off = LANES; off < 32; off *= 2) v += __shfl_xor_sync(kFull, v, off);
            if (lane < LANES && has) shared[(threadIdx.x >> 5) * at.cols + at.start(q) + j] = v;
        }
    }
    if (SHIFTED) {
#pragma unroll
        for (int off = LANES; off < 32; off *= 2) {
            edges.x += __shfl_xor_sync(kFull, edges.x, off);
            edges.y += __shfl_xor_sync(kFull, edges.y, off);
        }
        float* sums = shared + (threadIdx.x >> 5) * at.cols;
        if (lane < LANES && edge.has[0]) sums[edge.column[0]] = edges.x;
        if (lane < LANES && edge.has[1]) sums[edge.column[1]] = edges.y;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < at.cols; c += blockDim.x) {
        float v = shared[c];
        for (int w = 1; w < warps; ++w) v += shared[w * at.cols + c];
        out[c] = v;
    }
}

// Adds the sums of a CTA's row groups, thread by thread (a thread of each has the same columns), to
// those of the first group.
template <int PAIRS, typename Rows>
__device__ __forceinline__ void join_rows(float2* s, const Rows& group, float2* shared) {
    __syncthreads();   // nobody uses the shared memory any more
    if (group.index > 0)
#pragma unroll
        for (int k = 0; k < PAIRS; ++k) shared[k * blockDim.x + threadIdx.x] = s[k];
    __syncthreads();
    if (group.index == 0)
        for (int g = 1; g < group.groups; ++g)
#pragma unroll
            for (int k = 0; k < PAIRS; ++k) s[k] = add2(s[k], shared[k * blockDim.x + g * group.lanes + threadIdx.x]);
}

// A unit's column sums; `vector` where the partial rows lie as the operands' rows do.
template <int E>
__device__ __forceinline__ void store_sums(float* to, const float2 (&s)[E / 2], bool vector) {
    if (vector) {
#pragma unroll
        for (int k = 0; k < E / 4; ++k)
            reinterpret_cast<float4*>(to)[k] = make_float4(s[2 * k].x, s[2 * k].y, s[2 * k + 1].x, s[2 * k + 1].y);
    } else {
#pragma unroll
        for (int j = 0; j < E; ++j) to[j] = j & 1 ? s[j / 2].y : s[j / 2].x;
    }
}

template <typename T, int N, int LANES, bool SHIFTED>
__global__ void __maxnreg__(kBackwardRegisters) norm_grad_kernel(const __grid_constant__ NormGradArgs a) {
    constexpr int E = kUnit<T>, Q = N / E, H = E / 2, P = E / 4, S = kBackwardStages;
    extern __shared__ uint4 ring[];   // [S][Q][x, dy][threads], then the weight [P][Q][lanes of the CTA's rows]
    let_next_start();
    __shared__ WarpSums<LANES> sums1, sums2;
    const Group<T, LANES, SHIFTED> group(a.x, a.rows, a.cols, a.row_threads);
    const Columns<T, Q> at(group.t, group.lanes, group.head, a.cols);
    const Edge<T, SHIFTED> edge(group.t, group.head, a.cols);
    bool has[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) has[q] = at.has(q);
    const uint32_t unit_bytes = group.lanes * 16u, slot_bytes = blockDim.x * 16u;
    const uint32_t slots = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + threadIdx.x * 16u;
    const uint32_t slots_end = slots + S * Q * 2 * slot_bytes;
    const int64_t row_bytes = group.step * a.cols * int64_t(sizeof(T));
    const int64_t first_byte = group.first * a.cols * int64_t(sizeof(T));
    const char *x_row = static_cast<const char*>(a.x) + first_byte, *dy_row = static_cast<const char*>(a.dy) + first_byte;
    const char *x = x_row + at.start(0) * int(sizeof(T)), *dy = dy_row + at.start(0) * int(sizeof(T));
    int ahead = 0;
    const auto fetch = [&](uint32_t slot) {
        if (ahead < group.rows) {
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                if (!has[q]) continue;
                copy_async(slot + 2 * q * slot_bytes, x + q * unit_bytes);
                copy_async(slot + (2 * q + 1) * slot_bytes, dy + q * unit_bytes);
            }
        }
        ++ahead;
        x += row_bytes;
        dy += row_bytes;
        commit_copies();
    };
#pragma unroll
    for (int s = 0; s < S - 1; ++s) fetch(slots + s * Q * 2 * slot_bytes);
    // The weight waits in registers; beside groups of lanes, of which a CTA has many, in shared memory.
    float4* const weights = reinterpret_cast<float4*>(ring + S * Q * 2 * blockDim.x) + group.t;
    float2 held[LANES > 0 ? 1 : Q][H], sw[Q][H], sb[Q][H];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        if constexpr (LANES > 0) {
            if (group.index == 0) {
                float2 w[H];
                load_param<E>(a.weight, a.w_f32, a.w_vector, at.start(q), has[q], 1.0f, w);
#pragma unroll
                for (int p = 0; p < P; ++p)
                    weights[(p * Q + q) * LANES] = make_float4(w[2 * p].x, w[2 * p].y, w[2 * p + 1].x, w[2 * p + 1].y);
            }
        } else {
            load_param<E>(a.weight, a.w_f32, a.w_vector, at.start(q), has[q], 1.0f, held[q]);
        }
#pragma unroll
        for (int k = 0; k < H; ++k) sw[q][k] = sb[q][k] = make_float2(0.0f, 0.0f);
    }
    if (LANES <= 0) {
        sums1.clear();
        sums2.clear();
    }
    sync_all<LANES>();
    const float inv = 1.0f / static_cast<float>(a.cols);
    char* dx = static_cast<char*>(a.dx) + first_byte;
    const int dx_first = at.start(0) * int(sizeof(T));
    const float2 edge_w = edge.param(a.weight, a.w_f32, 1.0f);
    float2 edge_x = make_float2(0.0f, 0.0f), edge_dy = edge_x, edge_sw = edge_x, edge_sb = edge_x;
    const float *means = a.mean + group.first, *rstds = a.rstd + group.first;
    float next_mean = 0.0f, next_rstd = 0.0f;
    if (group.rows > 0) {
        next_mean = *means;
        next_rstd = *rstds;
        edge.load(x_row, edge_x);
        edge.load(dy_row, edge_dy);
    }
    uint32_t slot = slots, refill = slots + (S - 1) * Q * 2 * slot_bytes;
    const int turns = LANES > 0 ? group.turns : group.rows;   // a warp's lanes make the same turns
    for (int turn = 0; turn < turns; ++turn) {
        const float mean = next_mean, rstd = next_rstd;
        const bool exists = LANES <= 0 || turn < group.rows;   // a group past its last row adds nothing
        wait_copies<S - 2>();
        float2 xh[Q][H], h[Q][H];
        float2 s1 = make_float2(0.0f, 0.0f), s2 = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            unpack(read_shared(slot + 2 * q * slot_bytes), xh[q], T{});
            unpack(read_shared(slot + (2 * q + 1) * slot_bytes), h[q], T{});
#pragma unroll
            for (int k = 0; k < H; ++k) xh[q][k] = mul2(add2(xh[q][k], make_float2(-mean, -mean)), make_float2(rstd, rstd));
            keep_if(has[q] && exists, xh[q]);
            keep_if(has[q] && exists, h[q]);
#pragma unroll
            for (int k = 0; k < H; ++k) {
                sw[q][k] = fma2(h[q][k], xh[q][k], sw[q][k]);
                sb[q][k] = add2(sb[q][k], h[q][k]);
                if constexpr (LANES > 0) {
                    const float4 w = weights[(k / 2 * Q + q) * LANES];
                    h[q][k] = mul2(h[q][k], k & 1 ? make_float2(w.z, w.w) : make_float2(w.x, w.y));
                } else {
                    h[q][k] = mul2(h[q][k], held[q][k]);
                }
                s1 = add2(s1, h[q][k]);
                s2 = fma2(h[q][k], xh[q][k], s2);
            }
        }
        float2 edge_xh = make_float2(0.0f, 0.0f), edge_h = edge_xh;
        if (SHIFTED && edge.any) {
            if (exists) {
                edge_xh = edge.keep(mul2(add2(edge_x, make_float2(-mean, -mean)), make_float2(rstd, rstd)));
                edge_h = edge_dy;
            }
            edge_sw = fma2(edge_h, edge_xh, edge_sw);
            edge_sb = add2(edge_sb, edge_h);
            edge_h = mul2(edge_h, edge_w);
            s1 = add2(s1, edge_h);
            s2 = fma2(edge_h, edge_xh, s2);
            x_row += row_bytes;
            dy_row += row_bytes;
            if (turn + 1 < group.rows) {
                edge.load(x_row, edge_x);
                edge.load(dy_row, edge_dy);
            }
        }
        fetch(refill);
        refill = slot;
        slot += Q * 2 * slot_bytes;
        if (slot == slots_end) slot = slots;
        means += group.step;
        rstds += group.step;
        if (turn + 1 < group.rows) {
            next_mean = *means;
            next_rstd = *rstds;
        }
        float t1 = lane_sum<LANES>(s1.x + s1.y), t2 = lane_sum<LANES>(s2.x + s2.y);
        if (LANES <= 0) {
            sums1.put(turn & 1, group.index, group.t, t1);
            sums2.put(turn & 1, group.index, group.t, t2);
            sums1.sync(group.index, a.row_threads);
            t1 = sums1.total(turn & 1, group.index, a.row_threads);
            t2 = sums2.total(turn & 1, group.index, a.row_threads);
        }
        t1 *= -inv;
        t2 *= -inv;
        if (exists) {
#pragma unroll
            for (int q = 0; q < Q; ++q) {
#pragma unroll
                for (int k = 0; k < H; ++k)
                    h[q][k] = mul2(add2(h[q][k], fma2(xh[q][k], make_float2(t2, t2), make_float2(t1, t1))), make_float2(rstd, rstd));
                if (has[q]) *reinterpret_cast<uint4*>(dx + dx_first + q * unit_bytes) = pack(h[q], T{});
            }
            if (SHIFTED && edge.any)
                edge.store(dx, mul2(add2(edge_h, fma2(edge_xh, make_float2(t2, t2), make_float2(t1, t1))), make_float2(rstd, rstd)));
        }
        dx += row_bytes;
    }
    wait_copies<0>();
    if (a.sums) {
        float* out = a.sums + int64_t(group.part) * a.cols;
        float* out_b = out + int64_t(a.parts) * a.cols;
        if (LANES > 0) {
            join_groups<T, Q, LANES, SHIFTED>(sw, edge_sw, at, edge, reinterpret_cast<float*>(ring), out);
            join_groups<T, Q, LANES, SHIFTED>(sb, edge_sb, at, edge, reinterpret_cast<float*>(ring), out_b);
        } else {
            if (LANES == kRows) {   // onto the first group's, in the groups' order
                join_rows<Q * H>(&sw[0][0], group, reinterpret_cast<float2*>(ring));
                join_rows<Q * H>(&sb[0][0], group, reinterpret_cast<float2*>(ring));
                if (SHIFTED) {
                    join_rows<1>(&edge_sw, group, reinterpret_cast<float2*>(ring));
                    join_rows<1>(&edge_sb, group, reinterpret_cast<float2*>(ring));
                }
            }
            if (group.index == 0) {
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    if (!has[q]) continue;
                    store_sums<E>(out + at.start(q), sw[q], !SHIFTED);
                    store_sums<E>(out_b + at.start(q), sb[q], !SHIFTED);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (!edge.has[e]) continue;
                    out[edge.column[e]] = e ? edge_sw.y : edge_sw.x;
                    out_b[edge.column[e]] = e ? edge_sb.y : edge_sb.x;
                }
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

// Adds the partial rows: 32 columns a CTA, 16 threads a column, in a fixed order. It is launched
// while the kernel over the rows still runs and waits for its end here, which hides the launch.
constexpr int kJoinWarps = 16;

template <typename W>
__global__ void __launch_bounds__(kJoinWarps * 32) norm_join_kernel(const float* sums, int parts, int cols, W* dweight, W* dbias) {
    __shared__ float shared[kJoinWarps][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    W* out = blockIdx.y == 0 ? dweight : dbias;
    wait_for_previous();
    if (out == nullptr) return;
    const float* in = sums + int64_t(blockIdx.y) * parts * cols;
    float s = 0.0f;
    if (c < cols) {
        int p = warp;
        for (; p + 7 * kJoinWarps < parts; p += 8 * kJoinWarps) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = in[int64_t(p + k * kJoinWarps) * cols + c];
            s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
        }
#pragma unroll 4
        for (; p < parts; p += kJoinWarps) s += in[int64_t(p) * cols + c];
    }
    shared[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < cols) {
#pragma unroll
        for (int k = 1; k < kJoinWarps; ++k) s += shared[k][lane];
        out[c] = from_float<W>(s);
    }
}

__global__ void clear_kernel(uint32_t* word) {
    if (threadIdx.x == 0) *word = 0;
}

// ---- host ----------------------------------------------------------------------------------

bool known(nvfp4_type t) { return t == NVFP4_TYPE_BF16 || t == NVFP4_TYPE_F32; }
int type_size(nvfp4_type t) { return t == NVFP4_TYPE_F32 ? 4 : 2; }

bool shape_ok(int64_t rows, int64_t cols) {
    return rows >= 0 && cols >= 1 && cols <= (int64_t(1) << 30) && (rows == 0 || cols <= (int64_t(1) << 60) / rows);
}

nvfp4_status launched() { return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA; }

// Threads of a CTA, at most; and forward, where a row has some lanes of a warp.
constexpr int kMostThreads = 512, kLaneThreads = 128;

// How rows are given to threads.
struct Cut {
    int elements;   // of a thread; 0: by norm_long_kernel and its like
    int lanes;      // of a row: 8, 16, 32, kCta, kRows or kCluster
    int threads;    // of a CTA
    int row_threads;   // of those, a row's
    int cluster;    // CTAs of a row
    bool shifted;
};

// Rows that start on 16 bytes take whole units; others, where all operands' rows start at the same
// place within 16 bytes, have heads and tails.
Cut cut_rows(int64_t cols, int size, bool aligned, bool congruent, bool backward) {
    const int unit = 16 / size;
    const bool shifted = !aligned || cols % unit != 0;
    const int64_t need = cols;
    if (!congruent) return {0, 0, 0, 1, 1, false};
    // backward one CTA an SM, so that few partial rows are left
    const int threads = backward ? kMostThreads : kLaneThreads;
    if (need <= 64) return {8, 8, threads, 8, 1, shifted};
    if (need <= 128) return {8, 16, threads, 16, 1, shifted};
    if (need <= 256) return {8, 32, threads, 32, 1, shifted};
    if (need <= 512) return {16, 32, threads, 32, 1, shifted};
    for (int cluster = 1; cluster <= 8; cluster *= 2) {
        const int64_t row = (need + 512 * cluster - 1) / (512 * cluster) * 32;   // 16 elements a thread
        if (row <= kMostThreads) {
            const int groups = backward && row <= 128 ? static_cast<int>(kMostThreads / row) : 1;
            return {16, cluster > 1 ? kCluster : groups > 1 ? kRows : kCta, static_cast<int>(row) * groups, static_cast<int>(row), cluster, shifted};
        }
    }
    return {0, 0, 0, 1, 1, false};
}

// Groups of CTAs (one, or a cluster) that share the rows: at most the `resident` ones, and so many
// that all rows of one keep their head: a multiple of `unit`, unless each has one row only.
int64_t parts_of(const Cut& cut, int64_t rows, int64_t resident_ctas, int size) {
    const int64_t room = std::max<int64_t>(1, resident_ctas / cut.cluster), unit = cut.shifted ? 16 / size : 1;
    return rows <= room ? rows : std::max<int64_t>(unit, room / unit * unit);
}

// Partial rows of the backward pass.
int64_t backward_parts(const Cut& cut, int64_t rows, int64_t cols, int size) {
    const int64_t sms = sm_count();
    if (cut.elements == 0) {
        const int64_t across = (cols + 255) / 256;
        return std::min<int64_t>(rows, std::max<int64_t>(1, 4 * sms / across));
    }
    return parts_of(cut, rows, sms * resident(kBackwardRegisters, cut.threads), size);
}

// Launches a kernel with clusters of CTAs, and, where `after` is true, as one that may start
// before its predecessor in the stream has ended.
template <typename... Args>
nvfp4_status launch(void (*kernel)(Args...), dim3 grid, int threads, int cluster, size_t smem, bool after, cudaStream_t stream,
                    const Args&... args) {
    cudaLaunchConfig_t config{};
    config.gridDim = grid;
    config.blockDim = dim3(threads);
    config.dynamicSmemBytes = smem;
    config.stream = stream;
    cudaLaunchAttribute attributes[2] = {};
    int count = 0;
    if (cluster > 1) {
        attributes[count].id = cudaLaunchAttributeClusterDimension;
        attributes[count].val.clusterDim.x = cluster;
        attributes[count].val.clusterDim.y = attributes[count].val.clusterDim.z = 1;
        ++count;
    }
    if (after) {
        attributes[count].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attributes[count].val.programmaticStreamSerializationAllowed = 1;
        ++count;
    }
    config.attrs = attributes;
    config.numAttrs = count;
    if (cudaLaunchKernelEx(&config, kernel, args...) == cudaSuccess) return launched();
    cudaGetLastError();
    return NVFP4_ERR_CUDA;
}

// Lets `kernel` have MOST bytes of dynamic shared memory, the most that any of its plans asks for:
// threads that get here at once set the same value. Without asking it may have 48 KiB with the static
// arrays, which are below 8 KiB.
template <auto kernel, size_t MOST>
bool allow_smem() {
    static_assert(MOST <= (227 - 8) * 1024, "more than a CTA can have");
    if (MOST <= 40 * 1024) return true;
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> allowed[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return false;
    if (dev < kMaxDevices && allowed[dev].load(std::memory_order_acquire)) return true;
    if (cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(MOST)) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    if (dev < kMaxDevices) allowed[dev].store(true, std::memory_order_release);
    return true;
}

nvfp4_status clear_amax(uint32_t* amax, int64_t grid, cudaStream_t stream) {
    if (amax == nullptr || grid == 1) return NVFP4_OK;
    clear_kernel<<<1, 32, 0, stream>>>(amax);
    return launched();
}

template <typename T, int N, int LANES, bool SHIFTED>
nvfp4_status launch_group(const NormArgs& a, const Cut& cut, cudaStream_t stream) {
    constexpr auto kernel = norm_group_kernel<T, N, LANES, SHIFTED>;
    constexpr size_t kOfThread = size_t(kForwardStages) * N * sizeof(T);
    const size_t smem = kOfThread * cut.threads;
    if (!allow_smem<kernel, kOfThread * (LANES > 0 ? kLaneThreads : kMostThreads)>()) return NVFP4_ERR_CUDA;
    const int64_t parts = parts_of(cut, a.rows, int64_t(sm_count()) * resident(forward_registers(N), cut.threads), sizeof(T));
    if (clear_amax(a.amax, parts * cut.cluster, stream) != NVFP4_OK) return NVFP4_ERR_CUDA;
    return launch<NormArgs>(kernel, dim3(static_cast<unsigned>(parts * cut.cluster)), cut.threads, cut.cluster, smem,
                                  a.amax && parts * cut.cluster > 1, stream, a);
}

template <typename T, int Q, int K, int WARPS, bool SHIFTED>
nvfp4_status launch_norm(const NormArgs& a, cudaStream_t stream) {
    constexpr auto kernel = norm_kernel<T, Q, K, WARPS, SHIFTED>;
    constexpr size_t smem = size_t(16) * Q * 512 * kWideStages<T, Q> + size_t(WARPS) * 32 * Q * kUnit<T> * 8;
    if (!allow_smem<kernel, smem>()) return NVFP4_ERR_CUDA;
    constexpr int64_t unit = 16 / sizeof(T);
    const int64_t ctas = sm_count() * kWideCtas<T, Q>, room = !SHIFTED || ctas % unit == 0 ? ctas : std::max(unit, ctas / unit * unit);
    const int64_t grid = std::min(a.rows, room);
    if (clear_amax(a.amax, grid, stream) != NVFP4_OK) return NVFP4_ERR_CUDA;
    return launch<NormArgs>(kernel, dim3(static_cast<unsigned>(grid)), kWideThreads<WARPS>, 1, smem, a.amax && grid > 1, stream, a);
}

// Rows of WARPS warps whose lanes need FROM to 8 (BF16) units; FP32 rows need twice as many, in
// coarser steps. The units of a shifted row are up to two fewer.
template <typename T, int WARPS, int FROM, bool SHIFTED>
nvfp4_status launch_wide(const NormArgs& a, int need, cudaStream_t stream) {
    constexpr int S = SHIFTED;
    const int units = (need + WARPS * 256 - 1) / (WARPS * 256);
    if constexpr (sizeof(T) == 4) {
        if constexpr (FROM <= 2) if (units <= 2) return launch_norm<T, 4, 2 - S, WARPS, SHIFTED>(a, stream);
        if constexpr (FROM <= 4) if (units <= 4) return launch_norm<T, 8, 4 - S, WARPS, SHIFTED>(a, stream);
        return launch_norm<T, 16, 8 - S, WARPS, SHIFTED>(a, stream);
    } else {
        if constexpr (FROM <= 2) if (units == 2) return launch_norm<T, 2, 1 - S, WARPS, SHIFTED>(a, stream);
        if constexpr (FROM <= 3) if (units == 3) return launch_norm<T, 3, 2 - S, WARPS, SHIFTED>(a, stream);
        if constexpr (FROM <= 4) if (units == 4) return launch_norm<T, 4, 3 - S, WARPS, SHIFTED>(a, stream);
        if constexpr (FROM <= 5) if (units == 5) return launch_norm<T, 5, 4 - S, WARPS, SHIFTED>(a, stream);
        if constexpr (FROM <= 6) if (units == 6) return launch_norm<T, 6, 5 - S, WARPS, SHIFTED>(a, stream);
        if constexpr (FROM <= 7) if (units == 7) return launch_norm<T, 7, 6 - S, WARPS, SHIFTED>(a, stream);
        return launch_norm<T, 8, 7 - S, WARPS, SHIFTED>(a, stream);
    }
}

template <typename T, bool SHIFTED>
nvfp4_status dispatch_norm(const NormArgs& a, const Cut& cut, cudaStream_t stream) {
    if (cut.lanes == 8) return launch_group<T, 8, 8, SHIFTED>(a, cut, stream);
    if (cut.lanes == 16) return launch_group<T, 8, 16, SHIFTED>(a, cut, stream);
    if (cut.lanes == 32 && cut.elements == 8) return launch_group<T, 8, 32, SHIFTED>(a, cut, stream);
    const int need = a.cols;
    if (need <= 2048) return launch_wide<T, 1, 2, SHIFTED>(a, need, stream);
    if (need <= 4096) return launch_wide<T, 2, 5, SHIFTED>(a, need, stream);
    if (need <= 6144) return launch_wide<T, 3, 6, SHIFTED>(a, need, stream);
    if (need <= 8192) return launch_wide<T, 4, 7, SHIFTED>(a, need, stream);
    if (need <= 10240) return launch_wide<T, 5, 7, SHIFTED>(a, need, stream);
    return launch_group<T, 16, kCluster, SHIFTED>(a, cut, stream);
}

unsigned long_threads(int64_t cols) { return static_cast<unsigned>(std::min<int64_t>(1024, (cols + 31) / 32 * 32)); }

template <typename T>
nvfp4_status run_norm(const NormArgs& a, const Cut& cut, cudaStream_t stream) {
    if (cut.elements == 0) {
        const unsigned grid = static_cast<unsigned>(std::min<int64_t>(a.rows, sm_count() * 2));
        if (clear_amax(a.amax, grid, stream) != NVFP4_OK) return NVFP4_ERR_CUDA;
        return launch<NormArgs>(norm_long_kernel<T>, dim3(grid), long_threads(a.cols), 1, 0, a.amax && grid > 1, stream, a);
    }
    return cut.shifted ? dispatch_norm<T, true>(a, cut, stream) : dispatch_norm<T, false>(a, cut, stream);
}

template <typename T, int N, int LANES, bool SHIFTED>
nvfp4_status launch_grad(const NormGradArgs& a, const Cut& cut, cudaStream_t stream) {
    constexpr auto kernel = norm_grad_kernel<T, N, LANES, SHIFTED>;
    constexpr size_t kOfThread = size_t(kBackwardStages) * 2 * N * sizeof(T), kWeight = LANES > 0 ? size_t(4) * N * LANES : 0;
    const size_t smem = kOfThread * cut.threads + kWeight;
    if (!allow_smem<kernel, kOfThread * kMostThreads + kWeight>()) return NVFP4_ERR_CUDA;
    return launch<NormGradArgs>(kernel, dim3(static_cast<unsigned>(a.parts * cut.cluster)), cut.threads, cut.cluster, smem,
                                      false, stream, a);
}

template <typename T, bool SHIFTED>
nvfp4_status dispatch_grad(const NormGradArgs& a, const Cut& cut, cudaStream_t stream) {
    switch (cut.lanes) {
        case 8: return launch_grad<T, 8, 8, SHIFTED>(a, cut, stream);
        case 16: return launch_grad<T, 8, 16, SHIFTED>(a, cut, stream);
        case 32:
            return cut.elements == 8 ? launch_grad<T, 8, 32, SHIFTED>(a, cut, stream) : launch_grad<T, 16, 32, SHIFTED>(a, cut, stream);
        case kCta: return launch_grad<T, 16, kCta, SHIFTED>(a, cut, stream);
        case kRows: return launch_grad<T, 16, kRows, SHIFTED>(a, cut, stream);
        default: return launch_grad<T, 16, kCluster, SHIFTED>(a, cut, stream);
    }
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
    const Cut cut = cut_rows(cols, type_size(x_type), place(x) == 0, place(x) == place(y), false);
    const bool vector = !cut.shifted && place(weight) == 0 && place(bias) == 0;
    const NormArgs a{x, weight, bias, w_type == NVFP4_TYPE_F32, vector, rows, static_cast<int>(cols), eps, y, mean, rstd,
                     reinterpret_cast<uint32_t*>(amax), cut.row_threads};
    return x_type == NVFP4_TYPE_F32 ? run_norm<float>(a, cut, stream) : run_norm<bf16>(a, cut, stream);
}

extern "C" int64_t nvfp4_layer_norm_workspace(int64_t rows, int64_t cols) {
    if (!shape_ok(rows, cols)) return -1;
    if (rows == 0) return 0;
    int64_t parts = 0;   // for operands of any type and alignment
    for (const int size : {2, 4})
        for (const bool aligned : {true, false})
            for (const bool congruent : {true, false})
                parts = std::max(parts, backward_parts(cut_rows(cols, size, aligned, congruent, true), rows, cols, size));
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
    const Cut cut = cut_rows(cols, size, place(x) == 0, place(x) == place(dy) && place(x) == place(dx), true);
    const bool vector = !cut.shifted && place(weight) == 0;
    const NormGradArgs a{dy, x, weight, w_type == NVFP4_TYPE_F32, vector, mean, rstd, rows, static_cast<int>(cols), dx,
                         sums ? static_cast<float*>(workspace) : nullptr, static_cast<int>(backward_parts(cut, rows, cols, size)), cut.row_threads};
    const nvfp4_status st = x_type == NVFP4_TYPE_F32 ? run_grad<float>(a, cut, stream) : run_grad<bf16>(a, cut, stream);
    if (st != NVFP4_OK || !sums) return st;
    const dim3 grid(static_cast<unsigned>((cols + 31) / 32), 2);
    const float* partial = a.sums;
    if (w_type == NVFP4_TYPE_F32)
        return launch<const float*, int, int, float*, float*>(norm_join_kernel<float>, grid, kJoinWarps * 32, 1, 0, true, stream, partial,
                                                              a.parts, a.cols, static_cast<float*>(dweight), static_cast<float*>(dbias));
    return launch<const float*, int, int, bf16*, bf16*>(norm_join_kernel<bf16>, grid, kJoinWarps * 32, 1, 0, true, stream, partial, a.parts,
                                                        a.cols, static_cast<bf16*>(dweight), static_cast<bf16*>(dbias));
}

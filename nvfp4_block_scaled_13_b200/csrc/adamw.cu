// adamw.cu — an AdamW step over a list of tensors, and the norm of their gradients, on sm_100a.
//
// One launch covers the list: the host cuts every tensor into chunks of equal length once (the
// plan, kept in device memory) and the CTAs of a resident grid take chunks in turn. An element
// costs, with BF16 gradients, 28 bytes (BF16 parameter with FP32 master, 32-bit states) or
// 10.125 (BF16 parameter, 8-bit states) and some 40 operations, so memory bounds the step.
//
// The step's arithmetic is binary32 with its fused operations stated one by one, so with 32-bit
// states it has one right answer, bit for bit. 8-bit states are E4M3 codes in blocks of 32 with an E8M0 byte:
// the scale is a power of two, so decoding and scaling are exact and cost one multiplication.
#include <float.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <new>
#include <vector>

#include "../../include/nvfp4_train.h"
#include "train.cuh"

namespace {

using namespace nvfp4_train;

constexpr int kThreads = 256;
constexpr int kTile = kThreads * 8;        // elements of one pass of a CTA: eight a thread
constexpr uint32_t kMagic = 0x4E56504Cu;
constexpr uint32_t kGolden = 0x9E3779B9u;
constexpr int kMaxParts = 2048;            // CTAs of the gradient norm

enum Kind : uint32_t { kGradients = 1, kOptimizer = 2 };

// The plan's image: Header, Tensor[count], Chunk[chunks]; every part a multiple of 16 bytes.
struct Header {
    uint32_t magic, kind;
    uint32_t count, chunks;
    uint32_t chunk_elements, reserved[3];
};
struct Tensor {
    nvfp4_opt_tensor d;
    uint32_t variant;   // Variant bits, and kVector when every pointer suits 16-byte accesses
    uint32_t reserved[3];
};
struct Chunk {
    uint32_t tensor, index;
};
static_assert(sizeof(Header) == 32 && sizeof(nvfp4_opt_tensor) == 88 && sizeof(Chunk) == 8, "plan layout");

enum : uint32_t { kGradF32 = 1, kParamF32 = 2, kMaster = 4, kState8 = 8, kVector = 16 };

struct Image {
    const Header* header;
    const Tensor* tensors;
    const Chunk* chunks;
};

__host__ __device__ inline size_t tensor_offset() { return sizeof(Header); }
__host__ __device__ inline size_t chunk_offset(uint32_t count) { return sizeof(Header) + sizeof(Tensor) * size_t(count); }

__device__ __forceinline__ Image image_of(const void* plan) {
    const char* p = static_cast<const char*>(plan);
    const Header* h = reinterpret_cast<const Header*>(p);
    return {h, reinterpret_cast<const Tensor*>(p + tensor_offset()),
            reinterpret_cast<const Chunk*>(p + chunk_offset(h->count))};
}

// Eight elements from p[i]: one vector access, or the elements below n one by one.
template <typename T>
__device__ __forceinline__ void fetch8(const T* p, int64_t i, int64_t n, bool whole, float (&v)[8]) {
    if (whole) {
        load8(p + i, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = i + j < n ? to_float(p[i + j]) : 0.0f;
    }
}
template <typename T>
__device__ __forceinline__ void put8(T* p, int64_t i, int64_t n, bool whole, const float (&v)[8]) {
    if (whole) {
        store8(p + i, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i + j < n) p[i + j] = from_float<T>(v[j]);
    }
}

// ---- 8-bit states --------------------------------------------------------------------------

__device__ __forceinline__ float power_of_two(uint32_t biased) { return __uint_as_float(biased << 23); }

// Four codes as two pairs, without their scale.
__device__ __forceinline__ void decode4(uint32_t codes, float2* out) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t h2;
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h2) : "r"(codes >> (16 * k)));
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(out[k].x), "=f"(out[k].y)
            : "r"(h2));
    }
}

// The E8M0 byte of a block from its largest magnitude: the significand's carry at 1.75 moves a
// maximum above 448 * 2^(s - 127) to the next power.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) { return max((top + 0x1FFFFFu) >> 23, 9u) - 8u; }

// The largest magnitude of a block, of which four threads hold eight elements each.
__device__ __forceinline__ uint32_t block_top(const float2 (&v)[4]) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) top = max(top, max(magnitude(v[k].x), magnitude(v[k].y)));
    top = max(top, __shfl_xor_sync(kFull, top, 1));
    return max(top, __shfl_xor_sync(kFull, top, 2));
}

__device__ __forceinline__ uint2 encode_nearest(const float2 (&v)[4], float inverse) {
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float2 a = mul2(v[2 * k], make_float2(inverse, inverse)), b = mul2(v[2 * k + 1], make_float2(inverse, inverse));
        asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
            "mov.b32 %0, {lo, hi};\n\t}"
            : "=r"(w[k])
            : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    }
    return make_uint2(w[0], w[1]);
}

// u >= 0. Scaled by 2^-120, a value's exponent field is E4M3's (subnormals included), so its bits
// from bit 20 on are the code, and random bits added below them round it stochastically. The sum
// is taken four bits higher, which leaves the code in the top byte. Codes 0 of positive values,
// NaN and infinity are rare and left to a second look: 0 shows as a byte without a bit, and a
// block with NaN or infinity by its largest magnitude.
__device__ __forceinline__ uint2 encode_stochastic(const float2 (&u)[4], float inverse, uint32_t word, uint32_t top) {
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t sum[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 y = mul2(mul2(u[2 * k + j / 2], make_float2(inverse, inverse)), make_float2(0x1p-120f, 0x1p-120f));
            const uint32_t random = word + (4 * k + j) * kGolden;
            sum[j] = (__float_as_uint(j & 1 ? y.y : y.x) << 4) + __byte_perm(random, 0, 0x4104);
        }
        w[k] = __byte_perm(__byte_perm(sum[0], sum[1], 0x0073), __byte_perm(sum[2], sum[3], 0x0073), 0x5410);
    }
    if (top >= 0x7F800000u || ((w[0] - 0x01010101u) & ~w[0] & 0x80808080u) || ((w[1] - 0x01010101u) & ~w[1] & 0x80808080u)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x = j & 1 ? u[j / 2].y : u[j / 2].x;
            const int at = 8 * (j & 3);
            if (!(x < INFINITY)) {
                w[j >> 2] = (w[j >> 2] & ~(0xFFu << at)) | (0x7Fu << at);
            } else if (x > 0.0f && !(w[j >> 2] >> at & 0xFFu)) {
                w[j >> 2] |= 1u << at;
            }
        }
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint32_t mix(uint32_t a) {
    a ^= a >> 16;
    a *= 0x85EBCA6Bu;
    a ^= a >> 13;
    a *= 0xC2B2AE35u;
    return a ^ (a >> 16);
}

__device__ __forceinline__ void fetch_codes(const uint8_t* p, int64_t i, int64_t n, bool whole, uint2& c) {
    if (whole) {
        c = *reinterpret_cast<const uint2*>(p + i);
    } else {
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i + j < n) w[j >> 2] |= uint32_t(p[i + j]) << (8 * (j & 3));
        c = make_uint2(w[0], w[1]);
    }
}
__device__ __forceinline__ void put_codes(uint8_t* p, int64_t i, int64_t n, bool whole, uint2 c) {
    if (whole) {
        *reinterpret_cast<uint2*>(p + i) = c;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i + j < n) p[i + j] = static_cast<uint8_t>((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
    }
}

// ---- the step --------------------------------------------------------------------------------

struct Factors {
    float beta1, rest1, beta2, rest2, eps;   // rest = 1 - beta
    float lr, rate, root;                    // lr / (1 - beta1^t), (1 - beta2^t)^-1/2
    float scale;
    uint32_t key;
};

struct StepArgs {
    const void* plan;
    nvfp4_adamw_control* control;
    float lr;
    const float* lr_device;
    double beta1, beta2;
    float eps;
    uint32_t seed;
    const float* scale;
    uint32_t* amax;
};

// Root and quotient. 32-bit states take them as IEEE has them. Beside 8-bit states, whose step
// is bound by the instructions, the hardware's approximations do (relative errors of at most 2^-23
// each): u is then rounded to 4 bits, and the update is added to a parameter that it
// changes in its last bits.
template <bool EIGHT>
__device__ __forceinline__ float root_of(float v) {
    if (!EIGHT) return sqrtf(v);
    float r;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
template <bool EIGHT>
__device__ __forceinline__ float quotient(float a, float b) {
    if (!EIGHT) return a / b;
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(b));
    return a * r;
}

// Rounds to BF16 with the high half of each element's random word added to the dropped bits.
__device__ __forceinline__ uint4 round_stochastic(const float2 (&p)[4], uint32_t word) {
    uint32_t w[4];
    float2 finite = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t a = __float_as_uint(p[k].x) + ((word + 2 * k * kGolden) >> 16);
        const uint32_t b = __float_as_uint(p[k].y) + ((word + (2 * k + 1) * kGolden) >> 16);
        w[k] = __byte_perm(a, b, 0x7632);
        finite = fma2(p[k], make_float2(0.0f, 0.0f), finite);
    }
    // NaN and infinity are left to the conversion: adding to their bits could carry into the sign.
    if (!(finite.x + finite.y == 0.0f)) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (!(fabsf(p[k].x) < INFINITY)) w[k] = (w[k] & 0xFFFF0000u) | to_bf16(p[k].x);
            if (!(fabsf(p[k].y) < INFINITY)) w[k] = (w[k] & 0xFFFFu) | (uint32_t(to_bf16(p[k].y)) << 16);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T>
__device__ __forceinline__ void fetch_pairs(const T* p, int64_t i, int64_t n, bool whole, float2 (&v)[4]) {
    float f[8];
    fetch8(p, i, n, whole, f);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = make_float2(f[2 * k], f[2 * k + 1]);
}
__device__ __forceinline__ void put_pairs(float* p, int64_t i, int64_t n, bool whole, const float2 (&v)[4]) {
    const float f[8] = {v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y};
    put8(p, i, n, whole, f);
}
__device__ __forceinline__ void put_bf16(bf16* p, int64_t i, int64_t n, bool whole, const uint4& w) {
    if (whole) {
        *reinterpret_cast<uint4*>(p + i) = w;
    } else {
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i + j < n) p[i + j].bits = static_cast<uint16_t>(a[j / 2] >> (16 * (j & 1)));
    }
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// One chunk; the maximum of the stored parameters is joined to `top`.
template <uint32_t KIND>
__device__ __forceinline__ void step_chunk(const Tensor& t, int64_t lo, int64_t hi, const Factors& f, uint32_t& top) {
    constexpr bool GRAD_F32 = KIND & kGradF32, PARAM_F32 = KIND & kParamF32, MASTER = KIND & kMaster, EIGHT = KIND & kState8;
    const int64_t n = t.d.numel;
    const float keep = 1.0f - t.d.weight_decay * f.lr;
    for (int64_t base = lo; base < hi; base += kTile) {
        const int64_t i = base + threadIdx.x * 8;
        const bool whole = (t.variant & kVector) && i + 8 <= n;
        float2 g[4], p[4], m[4], u[4];
        if (GRAD_F32) {
            fetch_pairs(static_cast<const float*>(t.d.grad), i, n, whole, g);
        } else {
            fetch_pairs(static_cast<const bf16*>(t.d.grad), i, n, whole, g);
        }
        if (MASTER) {
            fetch_pairs(t.d.master, i, n, whole, p);
        } else if (PARAM_F32) {
            fetch_pairs(static_cast<const float*>(t.d.param), i, n, whole, p);
        } else {
            fetch_pairs(static_cast<const bf16*>(t.d.param), i, n, whole, p);
        }
        float sm = 0.0f, su = 0.0f;
        if (EIGHT) {
            uint2 cm, cu;
            fetch_codes(static_cast<const uint8_t*>(t.d.exp_avg), i, n, whole, cm);
            fetch_codes(static_cast<const uint8_t*>(t.d.exp_avg_sq), i, n, whole, cu);
            if (i < n) {
                sm = power_of_two(t.d.exp_avg_scale[i >> 5]);
                su = power_of_two(t.d.exp_avg_sq_scale[i >> 5]);
            }
            decode4(cm.x, m);
            decode4(cm.y, m + 2);
            decode4(cu.x, u);
            decode4(cu.y, u + 2);
        } else {
            fetch_pairs(static_cast<const float*>(t.d.exp_avg), i, n, whole, m);
            fetch_pairs(static_cast<const float*>(t.d.exp_avg_sq), i, n, whole, u);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            g[k] = mul2(g[k], both(f.scale));
            if (EIGHT) {
                m[k] = mul2(m[k], both(sm));
                u[k] = mul2(u[k], both(su));
                u[k] = mul2(u[k], u[k]);
            }
            m[k] = fma2(m[k], both(f.beta1), mul2(g[k], both(f.rest1)));
            u[k] = fma2(u[k], both(f.beta2), mul2(mul2(g[k], g[k]), both(f.rest2)));
            const float2 root = make_float2(root_of<EIGHT>(u[k].x), root_of<EIGHT>(u[k].y));
            const float2 under = fma2(root, both(f.root), both(f.eps));
            const float2 ratio = make_float2(quotient<EIGHT>(m[k].x, under.x), quotient<EIGHT>(m[k].y, under.y));
            p[k] = fma2(ratio, both(-f.rate), mul2(p[k], both(keep)));
            if (EIGHT) u[k] = root;
        }
        const uint32_t word = mix(static_cast<uint32_t>((t.d.first + i) >> 3) ^ f.key);
        if (PARAM_F32) {
            put_pairs(static_cast<float*>(t.d.param), i, n, whole, p);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (i + 2 * k < n) top = max(top, magnitude(p[k].x));
                if (i + 2 * k + 1 < n) top = max(top, magnitude(p[k].y));
            }
        } else {
            uint4 w;
            if (MASTER) {
                put_pairs(t.d.master, i, n, whole, p);
                w = make_uint4(to_bf16x2(p[0].x, p[0].y), to_bf16x2(p[1].x, p[1].y), to_bf16x2(p[2].x, p[2].y), to_bf16x2(p[3].x, p[3].y));
            } else {
                w = round_stochastic(p, word);
            }
            put_bf16(static_cast<bf16*>(t.d.param), i, n, whole, w);
            uint32_t best = 0;   // of two halves
            const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t v = a[k];
                if (i + 2 * k + 1 >= n) v = i + 2 * k >= n ? 0u : v & 0xFFFFu;
                asm("{\n\t.reg .b32 m;\n\tabs.bf16x2 m, %1;\n\tmax.NaN.bf16x2 %0, %0, m;\n\t}" : "+r"(best) : "r"(v));
            }
            top = max(top, max(best << 16, best & 0xFFFF0000u));
        }
        if (EIGHT) {
            const uint32_t tm = block_top(m), tu = block_top(u);
            const uint32_t bm = scale_byte(tm), bu = scale_byte(tu);
            put_codes(static_cast<uint8_t*>(t.d.exp_avg), i, n, whole, encode_nearest(m, power_of_two(254u - bm)));
            put_codes(static_cast<uint8_t*>(t.d.exp_avg_sq), i, n, whole, encode_stochastic(u, power_of_two(254u - bu), word, tu));
            if ((threadIdx.x & 3) == 0 && i < n) {
                t.d.exp_avg_scale[i >> 5] = static_cast<uint8_t>(bm);
                t.d.exp_avg_sq_scale[i >> 5] = static_cast<uint8_t>(bu);
            }
        } else {
            put_pairs(static_cast<float*>(t.d.exp_avg), i, n, whole, m);
            put_pairs(static_cast<float*>(t.d.exp_avg_sq), i, n, whole, u);
        }
    }
}

// A step that does not take place still reports the parameters' maxima.
__device__ __forceinline__ void top_of_chunk(const Tensor& t, int64_t lo, int64_t hi, uint32_t& top) {
    for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads)
        top = max(top, magnitude((t.variant & kParamF32) ? static_cast<const float*>(t.d.param)[i]
                                                         : to_float(static_cast<const bf16*>(t.d.param)[i])));
}

__device__ __forceinline__ void publish_top(uint32_t& top, uint32_t* amax) {
    const uint32_t best = __reduce_max_sync(kFull, top);
    if ((threadIdx.x & 31) == 0 && best != 0) atomicMax(amax, best);
    top = 0;
}

__global__ void __launch_bounds__(kThreads) adamw_kernel(const StepArgs a) {
    __shared__ Factors shared;
    const Image image = image_of(a.plan);
    if (image.header->magic != kMagic || image.header->kind != kOptimizer) return;
    if (threadIdx.x == 0) {
        Factors f;
        f.beta1 = static_cast<float>(a.beta1);
        f.rest1 = static_cast<float>(1.0 - a.beta1);
        f.beta2 = static_cast<float>(a.beta2);
        f.rest2 = static_cast<float>(1.0 - a.beta2);
        f.eps = a.eps;
        f.lr = a.lr_device ? *a.lr_device : a.lr;
        f.rate = static_cast<float>(static_cast<double>(f.lr) / (1.0 - a.control->beta1_t * a.beta1));
        f.root = static_cast<float>(1.0 / sqrt(1.0 - a.control->beta2_t * a.beta2));
        f.scale = a.scale ? *a.scale : 1.0f;
        f.key = mix(a.seed + kGolden * a.control->step);
        shared = f;
    }
    __syncthreads();
    const Factors f = shared;
    const bool takes_place = isfinite(f.scale);
    const uint32_t chunks = image.header->chunks;
    const int64_t length = image.header->chunk_elements;
    uint32_t top = 0, last = 0xFFFFFFFFu;
    for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const Chunk chunk = image.chunks[c];
        const Tensor& t = image.tensors[chunk.tensor];
        if (a.amax && last != 0xFFFFFFFFu && last != chunk.tensor) publish_top(top, a.amax + last);
        last = chunk.tensor;
        const int64_t lo = chunk.index * length, hi = min(t.d.numel, lo + length);
        if (!takes_place) {
            if (a.amax) top_of_chunk(t, lo, hi, top);
            continue;
        }
        switch (t.variant & 15u) {
            case 0: step_chunk<0>(t, lo, hi, f, top); break;
            case kGradF32: step_chunk<kGradF32>(t, lo, hi, f, top); break;
            case kParamF32: step_chunk<kParamF32>(t, lo, hi, f, top); break;
            case kParamF32 | kGradF32: step_chunk<kParamF32 | kGradF32>(t, lo, hi, f, top); break;
            case kMaster: step_chunk<kMaster>(t, lo, hi, f, top); break;
            case kMaster | kGradF32: step_chunk<kMaster | kGradF32>(t, lo, hi, f, top); break;
            case kState8: step_chunk<kState8>(t, lo, hi, f, top); break;
            case kState8 | kGradF32: step_chunk<kState8 | kGradF32>(t, lo, hi, f, top); break;
            case kState8 | kParamF32: step_chunk<kState8 | kParamF32>(t, lo, hi, f, top); break;
            case kState8 | kParamF32 | kGradF32: step_chunk<kState8 | kParamF32 | kGradF32>(t, lo, hi, f, top); break;
            case kState8 | kMaster: step_chunk<kState8 | kMaster>(t, lo, hi, f, top); break;
            case kState8 | kMaster | kGradF32: step_chunk<kState8 | kMaster | kGradF32>(t, lo, hi, f, top); break;
        }
    }
    if (a.amax && last != 0xFFFFFFFFu) publish_top(top, a.amax + last);
    // The last CTA to arrive counts the step: every CTA has read the control block before it
    // arrives.
    __syncthreads();
    if (threadIdx.x == 0 && takes_place && atomicAdd(&a.control->arrived, 1u) == gridDim.x - 1) {
        a.control->arrived = 0;
        a.control->step += 1;
        a.control->beta1_t *= a.beta1;
        a.control->beta2_t *= a.beta2;
    }
}

// ---- gradient norm ---------------------------------------------------------------------------

struct NormWorkspace {
    uint32_t arrived, reserved[3];
    double parts[kMaxParts];
};
static_assert(sizeof(NormWorkspace) == NVFP4_GRAD_NORM_WORKSPACE, "workspace size");

__device__ __forceinline__ double sum_of_squares(const float (&g)[8]) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s = fmaf(g[j], g[j], s);
    // Outside this range a square may have overflowed or lost bits to underflow.
    if (!(s >= 0x1p-90f && s <= FLT_MAX)) {
        double d = 0.0;
#pragma unroll
        for (int j = 0; j < 8; ++j) d = fma(static_cast<double>(g[j]), static_cast<double>(g[j]), d);
        return d;
    }
    return static_cast<double>(s);
}

__device__ __forceinline__ double warp_sum_double(double v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
    return v;
}

// Sum over the CTA, in thread 0.
__device__ __forceinline__ double cta_sum(double v, double* shared) {
    v = warp_sum_double(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x < 32) v = warp_sum_double(threadIdx.x < kThreads / 32 ? shared[threadIdx.x] : 0.0);
    return v;
}

template <typename T>
__device__ __forceinline__ double norm_chunk(const Tensor& t, int64_t lo, int64_t hi) {
    double sum = 0.0;
    const T* g = static_cast<const T*>(t.d.grad);
    const bool vector = t.variant & kVector;
    for (int64_t i = lo + threadIdx.x * 8; i < hi; i += kTile) {
        float v[8];
        fetch8(g, i, t.d.numel, vector && i + 8 <= t.d.numel, v);
        sum += sum_of_squares(v);
    }
    return sum;
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const void* plan, float max_norm, float* norm, float* scale,
                                                             NormWorkspace* work) {
    __shared__ double shared[kThreads / 32];
    __shared__ bool is_last;
    const Image image = image_of(plan);
    if (image.header->magic != kMagic) return;
    const uint32_t chunks = image.header->chunks;
    const int64_t length = image.header->chunk_elements;
    double sum = 0.0;
    for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const Chunk chunk = image.chunks[c];
        const Tensor& t = image.tensors[chunk.tensor];
        const int64_t lo = chunk.index * length, hi = min(t.d.numel, lo + length);
        sum += (t.variant & kGradF32) ? norm_chunk<float>(t, lo, hi) : norm_chunk<bf16>(t, lo, hi);
    }
    sum = cta_sum(sum, shared);
    if (threadIdx.x == 0) {
        work->parts[blockIdx.x] = sum;
        __threadfence();
        is_last = atomicAdd(&work->arrived, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!is_last) return;
    // the last CTA adds the partial sums in their own order
    __threadfence();
    double total = 0.0;
    for (uint32_t p = threadIdx.x; p < gridDim.x; p += kThreads) total += __ldcg(&work->parts[p]);
    total = cta_sum(total, shared);
    if (threadIdx.x == 0) {
        const double n = sqrt(total);
        const float rounded = static_cast<float>(n);
        *norm = rounded;
        *scale = isfinite(rounded) ? static_cast<float>(fmin(1.0, static_cast<double>(max_norm) / (n + 1e-6)))
                                   : __uint_as_float(0x7FC00000u);
        work->arrived = 0;
    }
}

// ---- host --------------------------------------------------------------------------------------

nvfp4_status launched() { return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA; }

constexpr int64_t kMostElements = int64_t(1) << 34;
constexpr int64_t kMostTensors = int64_t(1) << 24;

// Elements of a chunk: eight tiles where the list is long enough for every CTA to get several such
// chunks, fewer for shorter lists, so that they still spread over the SMs.
int64_t chunk_elements(int64_t total) {
    int64_t tiles = 8;
    while (tiles > 1 && total < tiles * kTile * 4096) tiles /= 2;
    return tiles * kTile;
}

bool count_chunks(const nvfp4_opt_tensor* tensors, int64_t count, int64_t* length, int64_t* chunks) {
    if (count < 0 || count >= kMostTensors || (count > 0 && tensors == nullptr)) return false;
    int64_t total = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (tensors[i].numel < 0 || tensors[i].numel >= kMostElements) return false;
        total += tensors[i].numel;
        if (total >= kMostElements) return false;
    }
    *length = chunk_elements(total);
    *chunks = 0;
    for (int64_t i = 0; i < count; ++i) *chunks += (tensors[i].numel + *length - 1) / *length;
    return true;
}

int64_t plan_bytes(int64_t count, int64_t chunks) {
    return static_cast<int64_t>(chunk_offset(static_cast<uint32_t>(count))) + (chunks * static_cast<int64_t>(sizeof(Chunk)) + 15) / 16 * 16;
}

int64_t size_of(int32_t type) { return type == NVFP4_TYPE_F32 ? 4 : 2; }

nvfp4_status check_tensor(const nvfp4_opt_tensor& t, bool gradients) {
    const bool known = (t.grad_type == NVFP4_TYPE_BF16 || t.grad_type == NVFP4_TYPE_F32) &&
                       (gradients || t.param_type == NVFP4_TYPE_BF16 || t.param_type == NVFP4_TYPE_F32);
    if (!known) return NVFP4_ERR_VALUE;
    if (t.numel > 0 && t.grad == nullptr) return NVFP4_ERR_NULL;
    if (!aligned_to(t.grad, size_of(t.grad_type))) return NVFP4_ERR_ALIGN;
    if (gradients) return NVFP4_OK;
    if (t.first < 0 || t.first % 8 != 0 || t.first >= kMostElements) return NVFP4_ERR_SHAPE;
    if ((t.state_bits != 32 && t.state_bits != 8) || !isfinite(t.weight_decay) ||
        (t.master != nullptr && t.param_type != NVFP4_TYPE_BF16))
        return NVFP4_ERR_VALUE;
    if (t.numel > 0 && (t.exp_avg == nullptr || t.exp_avg_sq == nullptr ||
                        (t.state_bits == 8 && (t.exp_avg_scale == nullptr || t.exp_avg_sq_scale == nullptr))))
        return NVFP4_ERR_NULL;
    const uintptr_t state = t.state_bits == 32 ? 4 : 1;
    if (!aligned_to(t.param, size_of(t.param_type)) || !aligned_to(t.master, 4) || !aligned_to(t.exp_avg, state) ||
        !aligned_to(t.exp_avg_sq, state))
        return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

struct Span {
    uintptr_t lo, hi;
    bool written;
};

// Whether memory that is written belongs to two places at once. Reads may share.
bool collides(std::vector<Span>& spans) {
    std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
    uintptr_t end = 0, written_end = 0;
    for (const Span& s : spans) {
        if (s.lo < written_end || (s.written && s.lo < end)) return true;
        end = std::max(end, s.hi);
        if (s.written) written_end = std::max(written_end, s.hi);
    }
    return false;
}

unsigned resident_grid(int64_t chunks, int per_sm) {
    return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(chunks, int64_t(sm_count()) * per_sm)));
}

}  // namespace

extern "C" int64_t nvfp4_tensor_plan_bytes(const nvfp4_opt_tensor* tensors, int64_t count) {
    int64_t length = 0, chunks = 0;
    return count_chunks(tensors, count, &length, &chunks) ? plan_bytes(count, chunks) : -1;
}

extern "C" nvfp4_status nvfp4_tensor_plan(const nvfp4_opt_tensor* tensors, int64_t count, void* image,
                                          int64_t image_bytes, int64_t* chunks_out) {
    int64_t length = 0, chunks = 0;
    if (!count_chunks(tensors, count, &length, &chunks)) return NVFP4_ERR_SHAPE;
    if (image == nullptr || chunks_out == nullptr) return NVFP4_ERR_NULL;
    if (image_bytes < plan_bytes(count, chunks)) return NVFP4_ERR_SHAPE;
    bool gradients = true;   // tensors without an element say nothing
    for (int64_t i = 0; i < count; ++i)
        if (tensors[i].param != nullptr) gradients = false;
    std::vector<Span> spans;
    try {
        for (int64_t i = 0; i < count; ++i) {
            const nvfp4_opt_tensor& t = tensors[i];
            if (!gradients && t.param == nullptr && t.numel > 0) return NVFP4_ERR_VALUE;
            const nvfp4_status st = check_tensor(t, gradients);
            if (st != NVFP4_OK) return st;
            if (t.numel == 0) continue;
            const auto add = [&](const void* p, int64_t bytes, bool written) {
                if (p) spans.push_back({reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + bytes, written});
            };
            add(t.grad, t.numel * size_of(t.grad_type), false);
            if (gradients) continue;
            add(t.param, t.numel * size_of(t.param_type), true);
            add(t.master, t.numel * 4, true);
            add(t.exp_avg, t.numel * t.state_bits / 8, true);
            add(t.exp_avg_sq, t.numel * t.state_bits / 8, true);
            if (t.state_bits == 8) {
                add(t.exp_avg_scale, (t.numel + 31) / 32, true);
                add(t.exp_avg_sq_scale, (t.numel + 31) / 32, true);
            }
        }
        if (collides(spans)) return NVFP4_ERR_VALUE;
    } catch (const std::bad_alloc&) {
        return NVFP4_ERR_CUDA;
    }
    memset(image, 0, static_cast<size_t>(plan_bytes(count, chunks)));
    char* out = static_cast<char*>(image);
    Header header{};
    header.magic = kMagic;
    header.kind = gradients ? kGradients : kOptimizer;
    header.count = static_cast<uint32_t>(count);
    header.chunks = static_cast<uint32_t>(chunks);
    header.chunk_elements = static_cast<uint32_t>(length);
    memcpy(out, &header, sizeof header);
    char* next = out + chunk_offset(header.count);
    for (int64_t i = 0; i < count; ++i) {
        Tensor t{};
        t.d = tensors[i];
        if (gradients) {
            t.variant = (t.d.grad_type == NVFP4_TYPE_F32 ? kGradF32 : 0u) | (aligned_to(t.d.grad, 16) ? kVector : 0u);
        } else {
            const uintptr_t state = t.d.state_bits == 32 ? 16 : 8;
            t.variant = (t.d.grad_type == NVFP4_TYPE_F32 ? kGradF32 : 0u) | (t.d.param_type == NVFP4_TYPE_F32 ? kParamF32 : 0u) |
                        (t.d.master ? kMaster : 0u) | (t.d.state_bits == 8 ? kState8 : 0u);
            if (aligned_to(t.d.grad, 16) && aligned_to(t.d.param, 16) && aligned_to(t.d.master, 16) &&
                aligned_to(t.d.exp_avg, state) && aligned_to(t.d.exp_avg_sq, state))
                t.variant |= kVector;
        }
        memcpy(out + tensor_offset() + sizeof(Tensor) * i, &t, sizeof t);
        for (int64_t c = 0; c * length < t.d.numel; ++c, next += sizeof(Chunk)) {
            const Chunk chunk{static_cast<uint32_t>(i), static_cast<uint32_t>(c)};
            memcpy(next, &chunk, sizeof chunk);
        }
    }
    *chunks_out = chunks;
    return NVFP4_OK;
}

extern "C" nvfp4_status nvfp4_grad_norm(const void* plan, int64_t chunks, float max_norm, float* norm, float* scale,
                                        void* workspace, cudaStream_t stream) {
    if (plan == nullptr || norm == nullptr || scale == nullptr || workspace == nullptr) return NVFP4_ERR_NULL;
    if (chunks < 0) return NVFP4_ERR_SHAPE;
    if (!(max_norm >= 0.0f)) return NVFP4_ERR_VALUE;
    if (!aligned_to(plan, 16) || !aligned_to(norm, 4) || !aligned_to(scale, 4) || !aligned_to(workspace, 16))
        return NVFP4_ERR_ALIGN;
    const unsigned grid = std::min<unsigned>(resident_grid(chunks, 8), kMaxParts);
    grad_norm_kernel<<<grid, kThreads, 0, stream>>>(plan, max_norm, norm, scale, static_cast<NormWorkspace*>(workspace));
    return launched();
}

extern "C" nvfp4_status nvfp4_adamw(const void* plan, int64_t chunks, nvfp4_adamw_control* control, float lr,
                                    const float* lr_device, double beta1, double beta2, float eps, uint32_t seed,
                                    const float* scale, float* amax, int64_t count, cudaStream_t stream) {
    if (plan == nullptr || control == nullptr) return NVFP4_ERR_NULL;
    if (chunks < 0 || count < 0) return NVFP4_ERR_SHAPE;
    if ((lr_device == nullptr && !(lr >= 0.0f && lr <= FLT_MAX)) || !(beta1 >= 0.0 && beta1 < 1.0) ||
        !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0f && eps <= FLT_MAX))
        return NVFP4_ERR_VALUE;
    if (!aligned_to(plan, 16) || !aligned_to(control, 8) || !aligned_to(lr_device, 4) || !aligned_to(scale, 4) ||
        !aligned_to(amax, 4))
        return NVFP4_ERR_ALIGN;
    if (amax && count > 0 && cudaMemsetAsync(amax, 0, static_cast<size_t>(count) * 4, stream) != cudaSuccess)
        return NVFP4_ERR_CUDA;
    const StepArgs a{plan, control, lr, lr_device, beta1, beta2, eps, seed, scale, reinterpret_cast<uint32_t*>(amax)};
    adamw_kernel<<<resident_grid(chunks, 4), kThreads, 0, stream>>>(a);
    return launched();
}

// adamw.cu — an AdamW step over a list of tensors, and the norm of their gradients, on sm_100a.
//
// One launch covers the list: the host cuts every tensor into chunks of equal length once (the
// plan, kept in device memory) and each CTA of a resident grid takes an equal range of them (taken
// in turn, one chunk after another, the pipelines drained at every chunk: 200 M elements with
// 8-bit states took 420 us, against 377).
//
// An element costs, with BF16 gradients, 28 bytes with an FP32 master and 32-bit states: memory
// bounds that step (168 M elements: 802 us, 89% of the copy bandwidth). A BF16 parameter with 8-bit
// states costs 10.125 bytes and 49 instructions: there the issue slots bound it (200 M elements in
// eight tensors: 362 us, 85%; 201 M in fourteen whose gradients differ in scale, the states of three
// plans in turn: 410 us, 76%). Hence paired (f32x2) arithmetic, three-operand maxima, addition of random bits in place
// of a comparison, and rare cases (zero codes, NaN) behind one test for eight elements.
//
// The step's arithmetic is binary32 with its fused operations stated one by one, so with 32-bit
// states it has one right answer, bit for bit. 8-bit states are E4M3 codes in blocks of 32 with an
// E8M0 byte: the scale is a power of two, so decoding and scaling are exact and cost one
// multiplication.
#include <float.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <new>
#include <type_traits>
#include <vector>

#include "../../include/nvfp4_train.h"
#include "train.cuh"

namespace {

using namespace nvfp4_train;

constexpr int kThreads = 256;
constexpr int kTile = kThreads * 8;        // elements of one pass of a CTA: eight a thread
constexpr uint32_t kMagic = 0x4E56504Cu;
constexpr uint32_t kGolden = 0x9E3779B9u;
// CTAs of an SM in a step. 8-bit states need 80 registers: with 64, for four CTAs, they spill (556 us
// for 200 M elements in place of 445 at that stage). 32-bit states spill a little at 80 (36 bytes
// stored, 44 loaded) and more at 64 (48 and 304), and four CTAs stream from more places at once: 168 M
// elements with masters took 835 us with four, 798 with three and 863 with two.
constexpr int kStepCtas = 3;
constexpr int kNormCtas = 4;
// Ring of each CTA (8-bit states), as much as three CTAs can have: 200 M elements took 464 us with
// three tiles in it, 431 with four, and 381 with five and the ranges above.
constexpr int kRingBytes = 74 * 1024;
constexpr int kMaxParts = 2048;            // CTAs of the gradient norm

enum Kind : uint32_t { kGradients = 1, kOptimizer32 = 2, kOptimizer8 = 3 };

// The plan's image: Header, Chunk[chunks], Tensor[count]; every part a multiple of 16 bytes. A kernel
// is given the number of chunks, so that it can look at its first chunk, the header and the control
// block at once: a short list's time is the chain of such reads.
struct Header {
    uint32_t magic, kind;
    uint32_t count, chunks;
    uint32_t chunk_elements, reserved[3];
};
struct Tensor {
    nvfp4_opt_tensor d;
    uint32_t variant;   // kGradF32 and the others below
    uint32_t reserved[3];
};
struct Chunk {
    uint32_t tensor, index;
};
static_assert(sizeof(Header) == 32 && sizeof(nvfp4_opt_tensor) == 88 && sizeof(Chunk) == 8, "plan layout");

// kVector: every pointer suits the step's whole accesses; kGradVector: the gradient the norm's.
enum : uint32_t { kGradF32 = 1, kParamF32 = 2, kMaster = 4, kVector = 8, kGradVector = 16 };

__host__ __device__ inline size_t tensor_offset(uint32_t chunks) {
    return sizeof(Header) + (sizeof(Chunk) * size_t(chunks) + 15) / 16 * 16;
}

struct Image {
    const Header* header;
    const Chunk* chunks;
    const Tensor* tensors;

    __device__ __forceinline__ Image(const void* plan, uint32_t count) {
        const char* p = static_cast<const char*>(plan);
        header = reinterpret_cast<const Header*>(p);
        chunks = reinterpret_cast<const Chunk*>(p + sizeof(Header));
        tensors = reinterpret_cast<const Tensor*>(p + tensor_offset(count));
    }
};

// The chunks of a list, cut into equal ranges for the CTAs, as runs inside one tensor: a CTA streams
// through a long piece of memory and looks at the tables rarely.
struct Runs {
    uint32_t next, end;

    __device__ __forceinline__ explicit Runs(uint64_t chunks) {
        next = static_cast<uint32_t>(chunks * blockIdx.x / gridDim.x);
        end = static_cast<uint32_t>(chunks * (blockIdx.x + 1) / gridDim.x);
    }
    // The elements [lo, hi) of the run that starts with `chunk` in a tensor of `numel`.
    __device__ __forceinline__ void take(const Chunk& chunk, int64_t length, int64_t numel, int64_t& lo, int64_t& hi) {
        lo = chunk.index * length;
        const int64_t of_tensor = (numel - lo + length - 1) / length, run = min(of_tensor, int64_t(end - next));
        hi = min(numel, lo + run * length);
        next += static_cast<uint32_t>(run);
    }
};

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

// The largest magnitude of a block, of which four threads hold eight elements each; NaN stays.
__device__ __forceinline__ uint32_t join_block(uint32_t top) {
    top = max(top, __shfl_xor_sync(kFull, top, 1));
    return max(top, __shfl_xor_sync(kFull, top, 2));
}
__device__ __forceinline__ float max_magnitude(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint32_t top_of(const float2 (&v)[4]) {
    float top = max_magnitude(v[0].x, v[0].y, v[1].x);
    top = max_magnitude(top, v[1].y, v[2].x);
    top = max_magnitude(top, v[2].y, v[3].x);
    return join_block(__float_as_uint(max_magnitude(top, v[3].y, v[3].y)));
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

// The 32-bit finalizer of MurmurHash3 (Austin Appleby, public domain), a bijection.
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

// The step's factors, and for each warp the description of the tensor that it works on: in shared
// memory, because registers are scarce below, and at file scope, so that every function knows it.
__shared__ Factors factors;
__shared__ nvfp4_adamw_control counted;   // the control block after this step
__shared__ Tensor tensors[kThreads / 32];

struct StepArgs {
    const void* plan;
    uint32_t chunks;
    nvfp4_adamw_control* control;
    float lr;
    const float* lr_device;
    double beta1, beta2;
    float eps;
    uint32_t seed;
    const float* scale;
    uint32_t* amax;
    uint32_t count;
};

// Root and reciprocal beside 8-bit states, whose step is bound by the instructions: the hardware's
// approximations (relative errors of at most 2^-23 each; a v below 2^-126 counts as 0). u is then
// rounded to 4 bits, and the update is added to a parameter that it changes in its last bits. A v
// that counts as 0 takes up to 2^-63 from u, which an eps of at least kLeastEps hides (2^-27 of the
// denominator, times 1 / sqrt(1 - beta2^t), which is at most 32 with beta2 = 0.999); and the reciprocal of
// a denominator above 2^126 is 0. Any other eps, 0 among them, takes the rounded root and quotient in
// their place (ROUNDED below), in an instance of its own, because one branch for both spilled in the usual
// one: 201 M BF16 weights take 353 us with the approximations and 592 without.
constexpr float kLeastEps = 0x1p-36f, kMostEps = 0x1p100f;
__device__ __forceinline__ float approximate_root(float v) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float approximate_reciprocal(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Rounds pairs of elements to BF16 with the high half of each element's random word (the first has
// `word`) added to the dropped bits.
template <int PAIRS>
__device__ __forceinline__ void round_stochastic(const float2 (&p)[PAIRS], uint32_t word, uint32_t (&w)[PAIRS]) {
    float2 finite = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < PAIRS; ++k) {
        const uint32_t a = __float_as_uint(p[k].x) + ((word + 2 * k * kGolden) >> 16);
        const uint32_t b = __float_as_uint(p[k].y) + ((word + (2 * k + 1) * kGolden) >> 16);
        w[k] = __byte_perm(a, b, 0x7632);
        finite = fma2(p[k], make_float2(0.0f, 0.0f), finite);
    }
    // NaN and infinity are left to the conversion: adding to their bits could carry into the sign.
    if (!(finite.x + finite.y == 0.0f)) {
#pragma unroll
        for (int k = 0; k < PAIRS; ++k) {
            if (!(fabsf(p[k].x) < INFINITY)) w[k] = (w[k] & 0xFFFF0000u) | to_bf16(p[k].x);
            if (!(fabsf(p[k].y) < INFINITY)) w[k] = (w[k] & 0xFFFFu) | (uint32_t(to_bf16(p[k].y)) << 16);
        }
    }
}

// Joins two stored BF16 parameters, elements i and i + 1 of n (whole: both exist), to a maximum of magnitudes: two
// halves side by side (NaN stays).
__device__ __forceinline__ void join_stored(uint32_t& top, uint32_t w, bool whole, int64_t i, int64_t n) {
    if (!whole && i + 1 >= n) w = i >= n ? 0u : w & 0xFFFFu;
    asm("{\n\t.reg .b32 m;\n\tabs.bf16x2 m, %1;\n\tmax.NaN.bf16x2 %0, %0, m;\n\t}" : "+r"(top) : "r"(w));
}

// ---- a thread's eight elements -------------------------------------------------------------------

template <typename T>
struct Eight {   // as they lie in memory
    uint4 w[sizeof(T) / 2];
};

__device__ __forceinline__ void unpack(const Eight<bf16>& e, float2 (&v)[4]) {
    const uint32_t a[4] = {e.w[0].x, e.w[0].y, e.w[0].z, e.w[0].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = make_float2(bf16_lo(a[k]), bf16_hi(a[k]));
}
__device__ __forceinline__ void unpack(const Eight<float>& e, float2 (&v)[4]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        v[2 * k] = make_float2(__uint_as_float(e.w[k].x), __uint_as_float(e.w[k].y));
        v[2 * k + 1] = make_float2(__uint_as_float(e.w[k].z), __uint_as_float(e.w[k].w));
    }
}
// whole: all eight exist and lie on a boundary of their own size (32 bytes in FP32, one access).
__device__ __forceinline__ void fetch(const bf16* p, int64_t i, int64_t n, bool whole, Eight<bf16>& e) {
    if (whole) {
        e.w[0] = *reinterpret_cast<const uint4*>(p + i);
    } else {
        uint32_t w[4] = {};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i + j < n) w[j / 2] |= uint32_t(p[i + j].bits) << (16 * (j & 1));
        e.w[0] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
__device__ __forceinline__ void fetch(const float* p, int64_t i, int64_t n, bool whole, Eight<float>& e) {
    if (whole) {
        asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(e.w[0].x), "=r"(e.w[0].y), "=r"(e.w[0].z), "=r"(e.w[0].w), "=r"(e.w[1].x), "=r"(e.w[1].y), "=r"(e.w[1].z),
                       "=r"(e.w[1].w)
                     : "l"(p + i)
                     : "memory");
    } else {
        uint32_t w[8] = {};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i + j < n) w[j] = __float_as_uint(p[i + j]);
        e.w[0] = make_uint4(w[0], w[1], w[2], w[3]);
        e.w[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}
__device__ __forceinline__ void put(bf16* p, int64_t i, int64_t n, bool whole, const uint4& w) {
    if (whole) {
        *reinterpret_cast<uint4*>(p + i) = w;
    } else {
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i + j < n) p[i + j].bits = static_cast<uint16_t>(a[j / 2] >> (16 * (j & 1)));
    }
}
__device__ __forceinline__ void put(float* p, int64_t i, int64_t n, bool whole, const float2 (&v)[4]) {
    if (whole) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p + i), "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y),
                     "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y)
                     : "memory");
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (i + 2 * k < n) p[i + 2 * k] = v[k].x;
            if (i + 2 * k + 1 < n) p[i + 2 * k + 1] = v[k].y;
        }
    }
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

template <bool F32>
using Float = typename std::conditional<F32, float, bf16>::type;

// ---- 32-bit states ---------------------------------------------------------------------------------
//
// Four consecutive elements make a unit: 16 bytes in FP32, so that a warp's accesses are
// contiguous. A thread has two units of a tile, all of whose reads are in flight together; with
// 224 to 256 bytes a thread nothing more is needed to keep memory busy.

struct Four {
    float2 v[2];
};

__device__ __forceinline__ void read_four(const float* p, int64_t i, int64_t n, bool whole, Four& f) {
    if (whole) {
        const float4 a = *reinterpret_cast<const float4*>(p + i);
        f.v[0] = make_float2(a.x, a.y);
        f.v[1] = make_float2(a.z, a.w);
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            f.v[k] = make_float2(i + 2 * k < n ? p[i + 2 * k] : 0.0f, i + 2 * k + 1 < n ? p[i + 2 * k + 1] : 0.0f);
    }
}
__device__ __forceinline__ void read_four(const bf16* p, int64_t i, int64_t n, bool whole, Four& f) {
    if (whole) {
        const uint2 a = *reinterpret_cast<const uint2*>(p + i);
        f.v[0] = make_float2(bf16_lo(a.x), bf16_hi(a.x));
        f.v[1] = make_float2(bf16_lo(a.y), bf16_hi(a.y));
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            f.v[k] = make_float2(i + 2 * k < n ? to_float(p[i + 2 * k]) : 0.0f, i + 2 * k + 1 < n ? to_float(p[i + 2 * k + 1]) : 0.0f);
    }
}
__device__ __forceinline__ void write_four(float* p, int64_t i, int64_t n, bool whole, const Four& f) {
    if (whole) {
        *reinterpret_cast<float4*>(p + i) = make_float4(f.v[0].x, f.v[0].y, f.v[1].x, f.v[1].y);
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (i + 2 * k < n) p[i + 2 * k] = f.v[k].x;
            if (i + 2 * k + 1 < n) p[i + 2 * k + 1] = f.v[k].y;
        }
    }
}
__device__ __forceinline__ void write_four(bf16* p, int64_t i, int64_t n, bool whole, uint2 w) {
    if (whole) {
        *reinterpret_cast<uint2*>(p + i) = w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < n) p[i + j].bits = static_cast<uint16_t>((j < 2 ? w.x : w.y) >> (16 * (j & 1)));
    }
}

// A tile that WHOLE says to be all there, on whole accesses; otherwise one in which the tensor ends
// or whose pointers do not suit. The first reads everything before it waits for anything.
template <uint32_t KIND, bool WHOLE>
__device__ __forceinline__ void step_tile_32(const nvfp4_opt_tensor& d, bool vector, int64_t base, float keep, const Factors& f,
                                             uint32_t& top) {
    constexpr bool PARAM_F32 = KIND & kParamF32, MASTER = KIND & kMaster;
    using G = Float<(KIND & kGradF32) != 0>;
    using P = Float<(KIND & (kParamF32 | kMaster)) != 0>;
    P* source = static_cast<P*>(MASTER ? d.master : d.param);
    float *exp_avg = static_cast<float*>(d.exp_avg), *exp_avg_sq = static_cast<float*>(d.exp_avg_sq);
    const int64_t n = d.numel;
    const int64_t at[2] = {base + threadIdx.x * 4, base + kTile / 2 + threadIdx.x * 4};
    Four g[2], p[2], m[2], u[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const bool whole = WHOLE || (vector && at[h] + 4 <= n);
        read_four(static_cast<const G*>(d.grad), at[h], n, whole, g[h]);
        read_four(source, at[h], n, whole, p[h]);
        read_four(exp_avg, at[h], n, whole, m[h]);
        read_four(exp_avg_sq, at[h], n, whole, u[h]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t i = at[h];
        const bool whole = WHOLE || (vector && i + 4 <= n);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float2 &gk = g[h].v[k], &mk = m[h].v[k], &uk = u[h].v[k];
            gk = mul2(gk, both(f.scale));
            mk = fma2(mk, both(f.beta1), mul2(gk, both(f.rest1)));
            uk = fma2(uk, both(f.beta2), mul2(mul2(gk, gk), both(f.rest2)));
            const float2 under = fma2(make_float2(sqrtf(uk.x), sqrtf(uk.y)), both(f.root), both(f.eps));
            const float2 ratio = make_float2(mk.x / under.x, mk.y / under.y);
            p[h].v[k] = fma2(ratio, both(-f.rate), mul2(p[h].v[k], both(keep)));
        }
        write_four(exp_avg, i, n, whole, m[h]);
        write_four(exp_avg_sq, i, n, whole, u[h]);
        if constexpr (PARAM_F32) {
            write_four(source, i, n, whole, p[h]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (whole || i + 2 * k < n) top = max(top, magnitude(p[h].v[k].x));
                if (whole || i + 2 * k + 1 < n) top = max(top, magnitude(p[h].v[k].y));
            }
        } else {
            uint32_t w[2];
            if constexpr (MASTER) {
                write_four(source, i, n, whole, p[h]);
                w[0] = to_bf16x2(p[h].v[0].x, p[h].v[0].y);
                w[1] = to_bf16x2(p[h].v[1].x, p[h].v[1].y);
                write_four(static_cast<bf16*>(d.param), i, n, whole, make_uint2(w[0], w[1]));
            } else {
                const int64_t place = d.first + i;   // below 2^35
                round_stochastic(p[h].v, mix(static_cast<uint32_t>(place >> 3) ^ f.key) + (static_cast<uint32_t>(place) & 4u) * kGolden, w);
                write_four(source, i, n, whole, make_uint2(w[0], w[1]));
            }
            join_stored(top, w[0], whole, i, n);
            join_stored(top, w[1], whole, i + 2, n);
        }
    }
}

template <uint32_t KIND>
__device__ __forceinline__ void step_run_32(const nvfp4_opt_tensor& d, bool vector, int64_t lo, int64_t hi, const Factors& f,
                                              uint32_t& top) {
    const float keep = 1.0f - d.weight_decay * f.lr;
    if (vector)
        for (; lo + kTile <= hi; lo += kTile) step_tile_32<KIND, true>(d, true, lo, keep, f, top);
    for (; lo < hi; lo += kTile) step_tile_32<KIND, false>(d, vector, lo, keep, f, top);
}

// ---- 8-bit states ----------------------------------------------------------------------------------
//
// What a thread reads of the streams of a tensor, eight elements of each, and the ring in shared
// memory through which the tiles after the next one arrive: 50 bytes a thread are too few to keep
// memory busy, and a second set does not fit into the registers. A warp copies (cp.async) and reads
// its own 256 elements only, so the ring needs no barrier beyond the warp's.
template <uint32_t KIND>
struct Read {
    using G = Float<(KIND & kGradF32) != 0>;
    using P = Float<(KIND & (kParamF32 | kMaster)) != 0>;
    // bytes of a stage, by stream
    static constexpr uint32_t kG = 8 * sizeof(G) * kThreads, kP = 8 * sizeof(P) * kThreads, kS = 8 * kThreads;
    static constexpr uint32_t kStage = kG + kP + 2 * kS + kThreads / 32 * 16;
    static constexpr int kStages = kRingBytes / kStage < 8 ? kRingBytes / kStage : 8;
    static_assert(kStages >= 2, "the ring holds two tiles");

    Eight<G> g;
    Eight<P> p;
    uint2 cm, cu;             // codes
    uint32_t sm, su;          // scale bytes

    static __device__ __forceinline__ const P* source(const nvfp4_opt_tensor& d) {
        return static_cast<const P*>((KIND & kMaster) ? d.master : d.param);
    }
    // Without the ring: element by element unless all eight are whole.
    __device__ __forceinline__ void fetch_from(const nvfp4_opt_tensor& d, int64_t i, bool whole) {
        const int64_t n = d.numel;
        fetch(static_cast<const G*>(d.grad), i, n, whole, g);
        fetch(source(d), i, n, whole, p);
        fetch_codes(static_cast<const uint8_t*>(d.exp_avg), i, n, whole, cm);
        fetch_codes(static_cast<const uint8_t*>(d.exp_avg_sq), i, n, whole, cu);
        sm = su = 0;
        if (whole || i < n) {
            sm = d.exp_avg_scale[i >> 5];
            su = d.exp_avg_sq_scale[i >> 5];
        }
    }
    // A warp's part of a stream, BYTES a lane, in contiguous accesses of 8 or 16 bytes a lane.
    template <int BYTES>
    static __device__ __forceinline__ void copy(uint32_t slot, const void* warp_from) {
        const uint32_t to = slot + (threadIdx.x >> 5) * (32 * BYTES), lane = threadIdx.x & 31;
        if (BYTES == 8) {
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to + lane * 8), "l"(static_cast<const char*>(warp_from) + lane * 8)
                         : "memory");
        } else {
#pragma unroll
            for (int k = 0; k < BYTES / 16; ++k)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + k * 512 + lane * 16),
                             "l"(static_cast<const char*>(warp_from) + k * 512 + lane * 16)
                             : "memory");
        }
    }
    template <typename T>
    static __device__ __forceinline__ void take(uint32_t slot, Eight<T>& e) {
#pragma unroll
        for (int k = 0; k < int(sizeof(T)) / 2; ++k)
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(e.w[k].x), "=r"(e.w[k].y), "=r"(e.w[k].z), "=r"(e.w[k].w)
                         : "r"(slot + threadIdx.x * uint32_t(8 * sizeof(T)) + k * 16)
                         : "memory");
    }
    static __device__ __forceinline__ void take(uint32_t slot, uint2& c) {
        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(c.x), "=r"(c.y) : "r"(slot + threadIdx.x * 8) : "memory");
    }
    static __device__ __forceinline__ uint32_t take_byte(uint32_t from) {
        uint16_t b;
        asm volatile("ld.shared.u8 %0, [%1];" : "=h"(b) : "r"(from) : "memory");
        return b;
    }
    // A warp's part of a tile; `i`: the warp's first element.
    static __device__ __forceinline__ void start(const nvfp4_opt_tensor& d, int64_t i, uint32_t slot) {
        copy<8 * sizeof(G)>(slot, static_cast<const G*>(d.grad) + i);
        copy<8 * sizeof(P)>(slot + kG, source(d) + i);
        copy<8>(slot + kG + kP, static_cast<const uint8_t*>(d.exp_avg) + i);
        copy<8>(slot + kG + kP + kS, static_cast<const uint8_t*>(d.exp_avg_sq) + i);
        const uint32_t lane = threadIdx.x & 31;
        if (lane < 4) {   // lanes 0 and 1 copy the eight scale bytes of m, 2 and 3 those of u
            const uint8_t* from = (lane < 2 ? d.exp_avg_scale : d.exp_avg_sq_scale) + (i >> 5) + (lane & 1) * 4;
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(slot + kG + kP + 2 * kS + (threadIdx.x >> 5) * 16 + lane * 4),
                         "l"(from)
                         : "memory");
        }
    }
    __device__ __forceinline__ void collect(uint32_t slot) {
        take(slot, g);
        take(slot + kG, p);
        take(slot + kG + kP, cm);
        take(slot + kG + kP + kS, cu);
        const uint32_t bytes = slot + kG + kP + 2 * kS + (threadIdx.x >> 5) * 16 + ((threadIdx.x & 31) >> 2);
        sm = take_byte(bytes);
        su = take_byte(bytes + 8);
    }
};

// Where a thread's eight elements are written.
template <uint32_t KIND>
struct Write {
    using T = Float<(KIND & kParamF32) != 0>;
    T* param;
    float* master;
    uint8_t *m, *u, *sm, *su;
    int64_t index;   // of the random words

    __device__ __forceinline__ Write(const nvfp4_opt_tensor& d, int64_t i)
        : param(static_cast<T*>(d.param) + i), master((KIND & kMaster) ? d.master + i : nullptr), m(static_cast<uint8_t*>(d.exp_avg) + i),
          u(static_cast<uint8_t*>(d.exp_avg_sq) + i), sm(d.exp_avg_scale + (i >> 5)), su(d.exp_avg_sq_scale + (i >> 5)), index(d.first + i) {}
};

// The step of a thread's eight elements, of which `left` exist where not all do; the maximum of the stored parameters is joined to `top`.
template <uint32_t KIND, bool ROUNDED>
__device__ __forceinline__ void step_eight(const Write<KIND>& to, const Read<KIND>& r, bool whole, int64_t left, float keep,
                                           const Factors& f, uint32_t& top) {
    constexpr bool PARAM_F32 = KIND & kParamF32, MASTER = KIND & kMaster;
    float2 g[4], p[4], m[4], u[4];
    unpack(r.g, g);
    unpack(r.p, p);
    decode4(r.cm.x, m);
    decode4(r.cm.y, m + 2);
    decode4(r.cu.x, u);
    decode4(r.cu.y, u + 2);
    const float sm = power_of_two(r.sm), su = power_of_two(r.su);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        g[k] = mul2(g[k], both(f.scale));
        m[k] = fma2(mul2(m[k], both(sm)), both(f.beta1), mul2(g[k], both(f.rest1)));
        u[k] = mul2(u[k], both(su));
        u[k] = fma2(mul2(u[k], u[k]), both(f.beta2), mul2(mul2(g[k], g[k]), both(f.rest2)));
        u[k] = ROUNDED ? make_float2(sqrtf(u[k].x), sqrtf(u[k].y)) : make_float2(approximate_root(u[k].x), approximate_root(u[k].y));
        const float2 under = fma2(u[k], both(f.root), both(f.eps));
        const float2 ratio = ROUNDED ? make_float2(m[k].x / under.x, m[k].y / under.y)
                                     : mul2(m[k], make_float2(approximate_reciprocal(under.x), approximate_reciprocal(under.y)));
        p[k] = fma2(ratio, both(-f.rate), mul2(p[k], both(keep)));
    }
    const uint32_t word = mix(static_cast<uint32_t>(to.index >> 3) ^ f.key);
    if constexpr (PARAM_F32) {
        put(to.param, 0, left, whole, p);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (whole || 2 * k < left) top = max(top, magnitude(p[k].x));
            if (whole || 2 * k + 1 < left) top = max(top, magnitude(p[k].y));
        }
    } else {
        uint32_t w[4];
        if constexpr (MASTER) {
            put(to.master, 0, left, whole, p);
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = to_bf16x2(p[k].x, p[k].y);
        } else {
            round_stochastic(p, word, w);
        }
        put(to.param, 0, left, whole, make_uint4(w[0], w[1], w[2], w[3]));
#pragma unroll
        for (int k = 0; k < 4; ++k) join_stored(top, w[k], whole, 2 * k, left);
    }
    const uint32_t tm = top_of(m), tu = top_of(u);
    const uint32_t bm = scale_byte(tm), bu = scale_byte(tu);
    put_codes(to.m, 0, left, whole, encode_nearest(m, power_of_two(254u - bm)));
    put_codes(to.u, 0, left, whole, encode_stochastic(u, power_of_two(254u - bu), word, tu));
    if ((threadIdx.x & 3) == 0 && (whole || left > 0)) {
        *to.sm = static_cast<uint8_t>(bm);
        *to.su = static_cast<uint8_t>(bu);
    }
}

// A run: whole tiles through the ring, then the tile in which the tensor ends, or all of it where a
// pointer does not suit whole accesses. A function of its own for each kind: inlined side by side,
// the kinds took registers from one another and spilled.
template <uint32_t KIND, bool ROUNDED>
__device__ __noinline__ uint32_t step_run_8(bool vector, int64_t lo, int64_t hi, uint32_t top) {
    const nvfp4_opt_tensor& d = tensors[threadIdx.x >> 5].d;
    const Factors& f = factors;
    extern __shared__ uint4 ring[];
    constexpr int S = Read<KIND>::kStages;
    const float keep = 1.0f - d.weight_decay * f.lr;
    const uint32_t slots = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
    const int ahead = (threadIdx.x & 31) * 8;   // elements of the warp before this thread's
    int64_t at = lo + threadIdx.x * 8;
    const int whole = vector ? static_cast<int>((hi - lo) / kTile) : 0;
    __syncwarp();   // nothing of an earlier run is still being read by another lane
#pragma unroll
    for (int k = 0; k < S - 1; ++k) {
        if (k < whole) Read<KIND>::start(d, at - ahead + k * kTile, slots + k * Read<KIND>::kStage);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    int stage = 0;
    for (int k = 0; k < whole; ++k, at += kTile) {
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
        __syncwarp();
        const uint32_t slot = slots + stage * Read<KIND>::kStage;
        const int behind = stage == 0 ? S - 1 : stage - 1;   // read by all lanes before the __syncwarp above
        if (k + S - 1 < whole) Read<KIND>::start(d, at - ahead + (S - 1) * kTile, slots + behind * Read<KIND>::kStage);
        asm volatile("cp.async.commit_group;" ::: "memory");
        stage = stage == S - 1 ? 0 : stage + 1;
        Read<KIND> now;
        now.collect(slot);
        step_eight<KIND, ROUNDED>(Write<KIND>(d, at), now, true, 8, keep, f, top);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    for (; at - threadIdx.x * 8 < hi; at += kTile) {
        Read<KIND> now;
        const bool eight = vector && at + 8 <= d.numel;
        now.fetch_from(d, at, eight);
        step_eight<KIND, ROUNDED>(Write<KIND>(d, at), now, eight, d.numel - at, keep, f, top);
    }
    return top;
}

// A step that does not take place still reports the parameters' maxima.
__device__ __forceinline__ void top_of_run(const Tensor& t, int64_t lo, int64_t hi, uint32_t& top) {
    for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) {
        if (t.variant & kParamF32) {
            top = max(top, magnitude(static_cast<const float*>(t.d.param)[i]));
        } else {
            join_stored(top, static_cast<const bf16*>(t.d.param)[i].bits, true, 0, 0);
        }
    }
}

// `top`: the bits of an FP32 magnitude, or the halves of two BF16 ones.
__device__ __forceinline__ void publish_top(uint32_t& top, bool halves, uint32_t* amax) {
    if (halves) top = max(top << 16, top & 0xFFFF0000u);
    const uint32_t best = __reduce_max_sync(kFull, top);
    if ((threadIdx.x & 31) == 0 && best != 0) atomicMax(amax, best);
    top = 0;
}

template <bool EIGHT, bool ROUNDED>
__global__ void __launch_bounds__(kThreads, kStepCtas) adamw_kernel(const StepArgs a) {
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Image image(a.plan, a.chunks);
    Runs runs(a.chunks);
    Chunk chunk{};
    // Each warp keeps the tensor's description in shared memory.
    const auto describe = [&]() {
        if (runs.next < runs.end) {
            chunk = image.chunks[runs.next];
            __syncwarp();
            if (lane < sizeof(Tensor) / 4)
                reinterpret_cast<uint32_t*>(&tensors[warp])[lane] = reinterpret_cast<const uint32_t*>(&image.tensors[chunk.tensor])[lane];
            __syncwarp();
        }
    };
    if (threadIdx.x == 0) {
        Factors f;
        f.beta1 = static_cast<float>(a.beta1);
        f.rest1 = static_cast<float>(1.0 - a.beta1);
        f.beta2 = static_cast<float>(a.beta2);
        f.rest2 = static_cast<float>(1.0 - a.beta2);
        f.eps = a.eps;
        f.lr = a.lr_device ? *a.lr_device : a.lr;
        nvfp4_adamw_control c = *a.control;
        f.key = mix(a.seed + kGolden * c.step);
        c.beta1_t *= a.beta1;
        c.beta2_t *= a.beta2;
        c.step += 1;
        counted = c;
        f.rate = f.lr / static_cast<float>(1.0 - c.beta1_t);
        f.root = 1.0f / sqrtf(static_cast<float>(1.0 - c.beta2_t));
        f.scale = a.scale ? *a.scale : 1.0f;
        factors = f;
    }
    const Header header = *image.header;
    describe();
    __syncthreads();
    if (header.magic != kMagic || header.kind != (EIGHT ? kOptimizer8 : kOptimizer32) || header.chunks != a.chunks ||
        (a.amax && header.count != a.count))
        return;
    const Factors& f = factors;
    const bool takes_place = isfinite(f.scale);
    const int64_t length = header.chunk_elements;
    uint32_t top = 0, last = 0xFFFFFFFFu;
    bool halves = false;
    for (bool described = true; runs.next < runs.end; described = false) {
        if (!described) describe();
        const Tensor& t = tensors[warp];
        if (a.amax && last != 0xFFFFFFFFu && last != chunk.tensor) publish_top(top, halves, a.amax + last);
        last = chunk.tensor;
        halves = !(t.variant & kParamF32);
        int64_t lo, hi;
        runs.take(chunk, length, t.d.numel, lo, hi);
        if (!takes_place) {
            if (a.amax) top_of_run(t, lo, hi, top);
            continue;
        }
        const bool vector = t.variant & kVector;
        if constexpr (EIGHT) {
            switch (t.variant & (kGradF32 | kParamF32 | kMaster)) {
                case 0: top = step_run_8<0, ROUNDED>(vector, lo, hi, top); break;
                case kGradF32: top = step_run_8<kGradF32, ROUNDED>(vector, lo, hi, top); break;
                case kParamF32: top = step_run_8<kParamF32, ROUNDED>(vector, lo, hi, top); break;
                case kParamF32 | kGradF32: top = step_run_8<kParamF32 | kGradF32, ROUNDED>(vector, lo, hi, top); break;
                case kMaster: top = step_run_8<kMaster, ROUNDED>(vector, lo, hi, top); break;
                default: top = step_run_8<kMaster | kGradF32, ROUNDED>(vector, lo, hi, top); break;
            }
        } else {
            switch (t.variant & (kGradF32 | kParamF32 | kMaster)) {
                case 0: step_run_32<0>(t.d, vector, lo, hi, f, top); break;
                case kGradF32: step_run_32<kGradF32>(t.d, vector, lo, hi, f, top); break;
                case kParamF32: step_run_32<kParamF32>(t.d, vector, lo, hi, f, top); break;
                case kParamF32 | kGradF32: step_run_32<kParamF32 | kGradF32>(t.d, vector, lo, hi, f, top); break;
                case kMaster: step_run_32<kMaster>(t.d, vector, lo, hi, f, top); break;
                default: step_run_32<kMaster | kGradF32>(t.d, vector, lo, hi, f, top); break;
            }
        }
    }
    if (a.amax && last != 0xFFFFFFFFu) publish_top(top, halves, a.amax + last);
    // The last CTA to arrive counts the step: every CTA has read the control block before it
    // arrives.
    __syncthreads();
    if (threadIdx.x == 0 && takes_place && atomicAdd(&a.control->arrived, 1u) == gridDim.x - 1) {
        a.control->beta1_t = counted.beta1_t;
        a.control->beta2_t = counted.beta2_t;
        a.control->step = counted.step;
        a.control->arrived = 0;
    }
}

// ---- gradient norm ---------------------------------------------------------------------------

struct NormWorkspace {
    uint32_t arrived, reserved[3];
    double parts[kMaxParts];
};
static_assert(sizeof(NormWorkspace) == NVFP4_GRAD_NORM_WORKSPACE, "workspace size");

__device__ __forceinline__ double sum_of_squares(const float2 (&g)[4]) {
    float2 s2 = mul2(g[0], g[0]);
#pragma unroll
    for (int k = 1; k < 4; ++k) s2 = fma2(g[k], g[k], s2);
    const float s = s2.x + s2.y;
    // Outside this range a square may have overflowed or lost bits to underflow, or there is nothing.
    if (!(s >= 0x1p-90f && s <= FLT_MAX)) {
        float top = max_magnitude(g[0].x, g[0].y, g[1].x);
        top = max_magnitude(top, g[1].y, g[2].x);
        top = max_magnitude(top, g[2].y, g[3].x);
        if (max_magnitude(top, g[3].y, g[3].y) == 0.0f) return 0.0;
        double d = 0.0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            d = fma(static_cast<double>(g[k].x), static_cast<double>(g[k].x), d);
            d = fma(static_cast<double>(g[k].y), static_cast<double>(g[k].y), d);
        }
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

// Four tiles are read before the first is summed: one tile's 16 bytes a thread leave half of the
// memory's bandwidth unused (measured on 400 M BF16 elements: 199 us, against 127).
template <typename T>
__device__ __forceinline__ double norm_run(const Tensor& t, int64_t lo, int64_t hi) {
    constexpr int kAtOnce = 4;
    double sum = 0.0;
    const T* g = static_cast<const T*>(t.d.grad);
    const bool vector = t.variant & kGradVector;
    int64_t i = lo + threadIdx.x * 8;
    if (vector) {
        for (; i + (kAtOnce - 1) * kTile + 8 <= hi; i += kAtOnce * kTile) {
            Eight<T> e[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) fetch(g + k * kTile, i, 0, true, e[k]);
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                float2 v[4];
                unpack(e[k], v);
                sum += sum_of_squares(v);
            }
        }
    }
    for (; i < hi; i += kTile) {
        Eight<T> e;
        float2 v[4];
        fetch(g, i, t.d.numel, vector && i + 8 <= t.d.numel, e);
        unpack(e, v);
        sum += sum_of_squares(v);
    }
    return sum;
}

__global__ void __launch_bounds__(kThreads, kNormCtas) grad_norm_kernel(const void* plan, uint32_t chunks, float max_norm, float* norm, float* scale,
                                                             NormWorkspace* work) {
    __shared__ double shared[kThreads / 32];
    __shared__ bool is_last;
    const Image image(plan, chunks);
    Runs runs(chunks);
    Chunk chunk{};
    if (runs.next < runs.end) chunk = image.chunks[runs.next];
    const Header header = *image.header;
    if (header.magic != kMagic || header.chunks != chunks) return;
    const int64_t length = header.chunk_elements;
    double sum = 0.0;
    for (bool first = true; runs.next < runs.end; first = false) {
        if (!first) chunk = image.chunks[runs.next];
        const Tensor& t = image.tensors[chunk.tensor];
        int64_t lo, hi;
        runs.take(chunk, length, t.d.numel, lo, hi);
        sum += (t.variant & kGradF32) ? norm_run<float>(t, lo, hi) : norm_run<bf16>(t, lo, hi);
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

// Elements of a chunk: one tile, or so many that a list has no more than 65536 full ones. A CTA's
// share is off by at most one chunk.
int64_t chunk_elements(int64_t total) {
    int64_t tiles = 1;
    while (total > tiles * kTile * 65536) tiles *= 2;
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
    return static_cast<int64_t>(tensor_offset(static_cast<uint32_t>(chunks)) + sizeof(Tensor) * static_cast<size_t>(count));
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

// Lets a step's kernel have its ring on the current device (once per device).
template <auto kernel>
bool allow_ring() {
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> allowed[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return false;
    if (dev < kMaxDevices && allowed[dev].load(std::memory_order_acquire)) return true;
    if (cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes) !=
        cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    if (dev < kMaxDevices) allowed[dev].store(true, std::memory_order_release);
    return true;
}

template <bool ROUNDED>
nvfp4_status launch_step_8(const StepArgs& a, cudaStream_t stream) {
    if (!allow_ring<adamw_kernel<true, ROUNDED>>()) return NVFP4_ERR_CUDA;
    adamw_kernel<true, ROUNDED><<<resident_grid(a.chunks, kStepCtas), kThreads, kRingBytes, stream>>>(a);
    return launched();
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
    bool gradients = true;
    for (int64_t i = 0; i < count; ++i)
        if (tensors[i].param != nullptr) gradients = false;
    int32_t bits = 0;
    std::vector<Span> spans;
    try {
        for (int64_t i = 0; i < count; ++i) {
            const nvfp4_opt_tensor& t = tensors[i];
            if (!gradients && t.param == nullptr && t.numel > 0) return NVFP4_ERR_VALUE;
            const nvfp4_status st = check_tensor(t, gradients);
            if (st != NVFP4_OK) return st;
            if (!gradients) {   // of tensors without an element too
                if (bits != 0 && bits != t.state_bits) return NVFP4_ERR_VALUE;
                bits = t.state_bits;
            }
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
    header.kind = gradients ? kGradients : bits == 8 ? kOptimizer8 : kOptimizer32;
    header.count = static_cast<uint32_t>(count);
    header.chunks = static_cast<uint32_t>(chunks);
    header.chunk_elements = static_cast<uint32_t>(length);
    memcpy(out, &header, sizeof header);
    char* next = out + sizeof(Header);
    for (int64_t i = 0; i < count; ++i) {
        Tensor t{};
        t.d = tensors[i];
        t.variant = (t.d.grad_type == NVFP4_TYPE_F32 ? kGradF32 : 0u) | (aligned_to(t.d.grad, 8 * size_of(t.d.grad_type)) ? kGradVector : 0u);
        if (!gradients) {
            t.variant |= (t.d.param_type == NVFP4_TYPE_F32 ? kParamF32 : 0u) | (t.d.master ? kMaster : 0u);
            // whole accesses: of eight elements beside 8-bit states, of four beside 32-bit ones
            const int unit = t.d.state_bits == 8 ? 8 : 4, state = t.d.state_bits == 8 ? 1 : 4;
            const auto suits = [&](const void* p, int64_t element) { return aligned_to(p, unit * element); };
            if (suits(t.d.grad, size_of(t.d.grad_type)) && suits(t.d.param, size_of(t.d.param_type)) && suits(t.d.master, 4) &&
                suits(t.d.exp_avg, state) && suits(t.d.exp_avg_sq, state) &&
                (state == 4 || (aligned_to(t.d.exp_avg_scale, 4) && aligned_to(t.d.exp_avg_sq_scale, 4))))
                t.variant |= kVector;
        }
        memcpy(out + tensor_offset(header.chunks) + sizeof(Tensor) * i, &t, sizeof t);
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
    if (chunks < 0 || chunks > 0xFFFFFFFFll) return NVFP4_ERR_SHAPE;
    if (!(max_norm >= 0.0f)) return NVFP4_ERR_VALUE;
    if (!aligned_to(plan, 16) || !aligned_to(norm, 4) || !aligned_to(scale, 4) || !aligned_to(workspace, 16))
        return NVFP4_ERR_ALIGN;
    const unsigned grid = std::min<unsigned>(resident_grid(chunks, kNormCtas), kMaxParts);
    grad_norm_kernel<<<grid, kThreads, 0, stream>>>(plan, static_cast<uint32_t>(chunks), max_norm, norm, scale, static_cast<NormWorkspace*>(workspace));
    return launched();
}

extern "C" nvfp4_status nvfp4_adamw(const void* plan, int64_t chunks, int32_t state_bits, nvfp4_adamw_control* control, float lr,
                                    const float* lr_device, double beta1, double beta2, float eps, uint32_t seed,
                                    const float* scale, float* amax, int64_t count, cudaStream_t stream) {
    if (plan == nullptr || control == nullptr) return NVFP4_ERR_NULL;
    if (chunks < 0 || chunks > 0xFFFFFFFFll || count < 0) return NVFP4_ERR_SHAPE;
    if ((state_bits != 32 && state_bits != 8) || (lr_device == nullptr && !(lr >= 0.0f && lr <= FLT_MAX)) || !(beta1 >= 0.0 && beta1 < 1.0) ||
        !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0f && eps <= FLT_MAX))
        return NVFP4_ERR_VALUE;
    if (!aligned_to(plan, 16) || !aligned_to(control, 8) || !aligned_to(lr_device, 4) || !aligned_to(scale, 4) ||
        !aligned_to(amax, 4))
        return NVFP4_ERR_ALIGN;
    if (amax && count > 0 && cudaMemsetAsync(amax, 0, static_cast<size_t>(count) * 4, stream) != cudaSuccess)
        return NVFP4_ERR_CUDA;
    const StepArgs a{plan, static_cast<uint32_t>(chunks), control, lr, lr_device, beta1, beta2, eps, seed, scale, reinterpret_cast<uint32_t*>(amax), static_cast<uint32_t>(count)};
    if (state_bits == 8) return eps >= kLeastEps && eps <= kMostEps ? launch_step_8<false>(a, stream) : launch_step_8<true>(a, stream);
    adamw_kernel<false, true><<<resident_grid(chunks, kStepCtas), kThreads, 0, stream>>>(a);
    return launched();
}

// Row operators of a decoding step, between the DF11 matrix products:
// df11_add_rms_norm, df11_silu_mul and df11_logits, and their launchers.
// All three stream rows once and are bound by memory (by launch latency for
// a few rows).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "df11.h"
#include "df11_step.h"

namespace {

using namespace df11_step;

constexpr int kWave = 64;

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// Largest |v| by its bits: a NaN's bits are above infinity's, so it is kept.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)v, d);
        v = v > o ? v : o;
    }
    return v;
}

// ------------------------------------------------------------------ norm
//
// h = x + r, y = h / sqrt(mean(h^2) + eps) * w.  A row stays in the registers
// of its THREADS threads (CHUNKS x 8 elements each) between the sum and the
// scaling, so x and r are read once.  Bound by memory: 8193 x 8192 BF16 rows
// with a BF16 residual into e4m3 83 us, 5.6 TB/s (this card copies at 5.45);
// one row of 4096 2.5 us; 4096 BF16 rows of 4096 26 us and of 4097, whose rows are
// not aligned, 32.

struct NormArgs {
    const void *x, *residual, *weight;
    void *residual_out, *out;
    float *scales;
    uint64_t x_stride, residual_stride, residual_out_stride, out_stride;
    uint32_t row0, rows, width, weight_f32;  // this launch: rows row0 .. rows
    float eps;
};

// e4m3 rows: y * (448 / a) with a the row's largest |y| (at least this, so
// that a row of zeros has a finite factor), scale a / 448
constexpr float kE4m3Max = 448.f, kAmaxFloor = 1e-30f;

struct none_t {};

template <int WAVES>
__device__ __forceinline__ float row_sum(float v, float *lds) {
    v = wave_sum(v);
    if constexpr (WAVES > 1) {
        const int wave = threadIdx.x / kWave;
        if (threadIdx.x % kWave == 0) lds[wave] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) v += lds[i];
    }
    return v;
}

template <int WAVES>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t *lds) {
    v = wave_max(v);
    if constexpr (WAVES > 1) {
        const int wave = threadIdx.x / kWave;
        if (threadIdx.x % kWave == 0) lds[wave] = v;
        __syncthreads();
        v = 0;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) v = v > lds[i] ? v : lds[i];
    }
    return v;
}

template <typename R, bool VEC, uint32_t STEP>
__device__ __forceinline__ void add_residual(const NormArgs &a, uint64_t row, uint32_t col,
                                             uint32_t left, float h[8]) {
    float r[8];
    load8<VEC, STEP>(static_cast<const R *>(a.residual), row * a.residual_stride + col, left, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] += r[j];
}

template <bool VEC, uint32_t STEP>
__device__ __forceinline__ void load_weight(const NormArgs &a, uint32_t col, uint32_t left,
                                            float w[8]) {
    if (a.weight_f32) load8<VEC, STEP>(static_cast<const float *>(a.weight), col, left, w);
    else load8<VEC, STEP>(static_cast<const __bf16 *>(a.weight), col, left, w);
}

// 8 values as e4m3 bytes, to nearest even
template <bool VEC, uint32_t STEP>
__device__ __forceinline__ void store_e4m3(uint8_t *p, uint64_t i, uint32_t count,
                                           const float v[8]) {
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
    global_ptr<uint8_t> g = as_global(p) + i;
    if constexpr (VEC) {
        *(global_ptr<u32x2>)g = u32x2{(uint32_t)lo, (uint32_t)hi};
    } else {
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j)
            if (j * STEP < count) g[j * STEP] = (uint8_t)((uint32_t)(j < 4 ? lo : hi) >> (8 * (j & 3)));
    }
}

// ROWS rows per workgroup, one wave each (ROWS > 1), or one row over all waves.
template <typename X, typename R, bool E4M3, bool VEC, int THREADS, int CHUNKS>
__global__ __launch_bounds__(THREADS < 256 ? 256 : THREADS) void df11_norm_kernel(NormArgs a) {
    constexpr int kWaves = THREADS / kWave;
    constexpr uint32_t kStep = VEC ? 1 : THREADS;  // between a thread's 8 elements
    constexpr bool kResidual = !__is_same(R, none_t);
    __shared__ float lds_sum[16];
    __shared__ uint32_t lds_max[16];
    uint64_t row = (uint64_t)a.row0 + blockIdx.x;
    uint32_t t = threadIdx.x;
    if constexpr (kWaves == 1) {
        row = a.row0 + (uint64_t)blockIdx.x * (blockDim.x / kWave) + threadIdx.x / kWave;
        t = threadIdx.x % kWave;
        if (row >= a.rows) return;  // whole waves; no barrier follows with one wave per row
        // (launches of kNormRows rows end at a multiple of 4)
    }
    float h[CHUNKS][8];
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
        const uint32_t col = VEC ? (c * THREADS + t) * 8 : c * THREADS * 8 + t;
#pragma unroll
        for (int j = 0; j < 8; ++j) h[c][j] = 0.f;
        if (col < a.width) {
            const uint32_t left = a.width - col;
            load8<VEC, kStep>(static_cast<const X *>(a.x), row * a.x_stride + col, left, h[c]);
            if constexpr (kResidual) {
                add_residual<R, VEC, kStep>(a, row, col, left, h[c]);
                store8<VEC, kStep>(static_cast<R *>(a.residual_out), row * a.residual_out_stride + col,
                            left, h[c]);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(h[c][j], h[c][j], ss);
    }
    ss = row_sum<kWaves>(ss, lds_sum);
    const float rstd = 1.f / sqrtf(ss / (float)a.width + a.eps);
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
        const uint32_t col = VEC ? (c * THREADS + t) * 8 : c * THREADS * 8 + t;
        if (col >= a.width) continue;
        float w[8];
        load_weight<VEC, kStep>(a, col, a.width - col, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            h[c][j] = h[c][j] * rstd * w[j];
            const uint32_t mag = __float_as_uint(h[c][j]) & 0x7FFFFFFFu;
            top = top > mag ? top : mag;
        }
        if constexpr (!E4M3)
            store8<VEC, kStep>(static_cast<__bf16 *>(a.out), row * a.out_stride + col, a.width - col, h[c]);
    }
    if constexpr (E4M3) {
        top = row_max<kWaves>(top, lds_max);
        const uint32_t floor_bits = __float_as_uint(kAmaxFloor);
        const float amax = __uint_as_float(top > floor_bits ? top : floor_bits);
        const float inv = kE4m3Max / amax;
        if (t == 0) as_global(a.scales)[row] = amax / kE4m3Max;
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            const uint32_t col = VEC ? (c * THREADS + t) * 8 : c * THREADS * 8 + t;
            if (col >= a.width) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j) h[c][j] *= inv;
            store_e4m3<VEC, kStep>(static_cast<uint8_t *>(a.out), row * a.out_stride + col, a.width - col,
                            h[c]);
        }
    }
}

// Rows too wide for the registers of one workgroup: x and r are read again
// for the scaling (and once more for the e4m3 row's maximum).  The residual is
// written in the last pass, so that it may be updated in place.
template <typename X, typename R, bool E4M3>
__global__ __launch_bounds__(1024) void df11_norm_wide_kernel(NormArgs a) {
    constexpr bool kResidual = !__is_same(R, none_t);
    __shared__ float lds_sum[16];
    __shared__ uint32_t lds_max[16];
    const uint64_t row = (uint64_t)a.row0 + blockIdx.x;
    auto load = [&](uint32_t col, float h[8]) {
        load8<false, 1024>(static_cast<const X *>(a.x), row * a.x_stride + col, a.width - col, h);
        if constexpr (kResidual) add_residual<R, false, 1024>(a, row, col, a.width - col, h);
    };
    float h[8], w[8];
    float ss = 0.f;
    for (uint64_t col = threadIdx.x; col < a.width; col += 1024 * 8) {
        load((uint32_t)col, h);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(h[j], h[j], ss);
    }
    ss = row_sum<16>(ss, lds_sum);
    const float rstd = 1.f / sqrtf(ss / (float)a.width + a.eps);
    float inv = 1.f;
    if constexpr (E4M3) {
        uint32_t top = 0;
        for (uint64_t col = threadIdx.x; col < a.width; col += 1024 * 8) {
            load((uint32_t)col, h);
            load_weight<false, 1024>(a, (uint32_t)col, a.width - (uint32_t)col, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t mag = __float_as_uint(h[j] * rstd * w[j]) & 0x7FFFFFFFu;
                top = top > mag ? top : mag;
            }
        }
        top = row_max<16>(top, lds_max);
        const uint32_t floor_bits = __float_as_uint(kAmaxFloor);
        const float amax = __uint_as_float(top > floor_bits ? top : floor_bits);
        inv = kE4m3Max / amax;
        if (threadIdx.x == 0) as_global(a.scales)[row] = amax / kE4m3Max;
    }
    for (uint64_t col = threadIdx.x; col < a.width; col += 1024 * 8) {
        const uint32_t c = (uint32_t)col, left = a.width - c;
        load(c, h);
        if constexpr (kResidual)
            store8<false, 1024>(static_cast<R *>(a.residual_out), row * a.residual_out_stride + c, left, h);
        load_weight<false, 1024>(a, c, left, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = h[j] * rstd * w[j];
        if constexpr (E4M3) {
#pragma unroll
            for (int j = 0; j < 8; ++j) h[j] *= inv;
            store_e4m3<false, 1024>(static_cast<uint8_t *>(a.out), row * a.out_stride + c, left, h);
        } else {
            store8<false, 1024>(static_cast<__bf16 *>(a.out), row * a.out_stride + c, left, h);
        }
    }
}

// A launch has at most 2^32 - 1 threads: more rows take several.
constexpr uint32_t kNormRows = 1u << 20;

template <typename X, typename R, bool E4M3, bool VEC>
void launch_norm(const NormArgs &a, hipStream_t s) {
    const uint32_t rows = std::min(a.rows - a.row0, kNormRows);
    // threads x chunks of 8 that hold a row
    if (a.width <= 64 * 8)
        hipLaunchKernelGGL((df11_norm_kernel<X, R, E4M3, VEC, 64, 1>), dim3((rows + 3) / 4),
                           dim3(256), 0, s, a);
    else if (a.width <= 256 * 8)
        hipLaunchKernelGGL((df11_norm_kernel<X, R, E4M3, VEC, 256, 1>), dim3(rows), dim3(256), 0,
                           s, a);
    else if (a.width <= 512 * 8)
        hipLaunchKernelGGL((df11_norm_kernel<X, R, E4M3, VEC, 512, 1>), dim3(rows), dim3(512), 0,
                           s, a);
    else if (a.width <= 1024 * 8)
        hipLaunchKernelGGL((df11_norm_kernel<X, R, E4M3, VEC, 512, 2>), dim3(rows), dim3(512), 0,
                           s, a);
    else if (a.width <= 4096 * 8)
        hipLaunchKernelGGL((df11_norm_kernel<X, R, E4M3, VEC, 1024, 4>), dim3(rows), dim3(1024),
                           0, s, a);
    else
        hipLaunchKernelGGL((df11_norm_wide_kernel<X, R, E4M3>), dim3(rows), dim3(1024), 0, s, a);
}

template <typename X, typename R>
void launch_norm(const NormArgs &a, bool e4m3, bool vec, hipStream_t s) {
    if (e4m3) vec ? launch_norm<X, R, true, true>(a, s) : launch_norm<X, R, true, false>(a, s);
    else vec ? launch_norm<X, R, false, true>(a, s) : launch_norm<X, R, false, false>(a, s);
}

template <typename X>
void launch_norm(const NormArgs &a, uint32_t residual_type, bool e4m3, bool vec, hipStream_t s) {
    if (!a.residual) launch_norm<X, none_t>(a, e4m3, vec, s);
    else if (residual_type == DF11_F32) launch_norm<X, float>(a, e4m3, vec, s);
    else launch_norm<X, __bf16>(a, e4m3, vec, s);
}

// ------------------------------------------------------------------ silu * up
//
// g / (1 + exp(-g)) * u, 8 elements a thread, rows down the grid.  Bound by
// memory: 4099 x 14336 BF16 61 us, 5.8 TB/s, x 14335 (rows not aligned) 66; 16
// rows of fp32 2.5 us.

struct ActArgs {
    const void *gate, *up;
    __bf16 *out;
    uint64_t gate_stride, up_stride, out_stride;
    uint32_t rows, width;
};

template <typename X, bool VEC>
__global__ __launch_bounds__(256) void df11_silu_mul_kernel(ActArgs a) {
    constexpr uint32_t kStep = VEC ? 1 : 256;
    const uint64_t at = (uint64_t)blockIdx.x * 2048 + (VEC ? threadIdx.x * 8 : threadIdx.x);
    if (at >= a.width) return;
    const uint32_t col = (uint32_t)at, left = a.width - col;
    for (uint64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        float g[8], u[8];
        load8<VEC, kStep>(static_cast<const X *>(a.gate), row * a.gate_stride + col, left, g);
        load8<VEC, kStep>(static_cast<const X *>(a.up), row * a.up_stride + col, left, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = g[j] / (1.f + __expf(-g[j])) * u[j];
        store8<VEC, kStep>(a.out, row * a.out_stride + col, left, g);
    }
}

// ------------------------------------------------------------------ logits
//
// A workgroup takes kSpan consecutive ids of one row: it counts the row's
// history for those ids in LDS (integer atomics: no order matters), then
// streams its logits through the penalties, the bias and the mask.  Every span
// reads the row's history again (from L2); spans of 2048 ids read it twice as
// often and spans of 8192 leave half as many workgroups per CU (128 x 128001
// fp32 logits, 4096 tokens of history, 64 biases, mask: 55 and 48 us where 4096
// took 45).  Now 38 us for 131 MB (25 at the copy rate): without history 32,
// without biases 34, without all three 28.

constexpr uint32_t kSpan = 4096;
constexpr uint32_t kSeen = 0x80000000u;  // in the prompt; low bits: times in the output

struct LogitsArgs {
    const void *logits;
    float *out;
    const int32_t *tokens, *lens, *prompt_lens, *bias_ids;
    const float *repetition, *frequency, *presence, *bias_values;
    const uint32_t *mask;
    uint64_t stride, out_stride, tokens_stride, bias_stride, mask_stride;
    uint32_t rows, vocab, history, n_bias;
};

// 4 logits as floats from an address aligned to 4 elements.
template <typename X>
__device__ __forceinline__ f32x4 load4(global_ptr<const X> p) {
    if constexpr (__is_same(X, float)) {
        return *(global_ptr<const f32x4>)p;
    } else {
        typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
        const bf16x4 w = *(global_ptr<const bf16x4>)p;
        return f32x4{(float)w[0], (float)w[1], (float)w[2], (float)w[3]};
    }
}

// A thread takes kSpan / 1024 groups of 4 neighbouring ids, loaded before the
// history is counted so that both are in flight together (no branch between
// the loads: a branch makes the compiler wait for those before it).  ALIGNED: the
// span starts at an id that makes its addresses aligned, up to 3 below the id it
// would start with, since rows of any length start anywhere; what that adds in
// front is the row before (rows not aligned themselves have one) and is not
// used, and up to 3 ids at the row's end are done one by one.
template <typename X, bool ALIGNED>
__global__ __launch_bounds__(256) void df11_logits_kernel(LogitsArgs a) {
    constexpr int kGroups = kSpan / 1024;
    constexpr int kAhead = 4;  // ids in flight per thread
    __shared__ uint32_t counts[kSpan];  // then, in spans that a bias falls into: last entry + 1
    __shared__ uint32_t flags[4];
    int32_t *entry = (int32_t *)counts;
    const int tid = threadIdx.x;
    for (uint64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const uint64_t at = row * a.stride;
        const int shift = ALIGNED ? (int)(at & 3) : 0;
        const int lo = blockIdx.x == 0 ? shift : 0;
        // offset d of the span is id first + d; its ids are at offsets lo .. hi - 1
        const int64_t first = (int64_t)blockIdx.x * kSpan - shift;
        if (first >= a.vocab) continue;  // the last span of a row without a shift (no barrier passed)
        const int hi = (int)min((int64_t)kSpan, (int64_t)a.vocab - first);
        const int whole = ALIGNED ? hi & ~3 : hi;  // offsets done in groups
        const uint32_t first32 = (uint32_t)first;
        global_ptr<const X> logits = as_global(static_cast<const X *>(a.logits)) + (int64_t)at + first;
        // everything that does not wait for a count is loaded first
        int32_t said = 0, prompt = 0;
        float rep = 1.f, freq = 0.f, pres = 0.f;
        if (a.history) said = as_global(a.lens)[row];
        if (a.prompt_lens) prompt = as_global(a.prompt_lens)[row];
        if (a.repetition) rep = as_global(a.repetition)[row];
        if (a.frequency) freq = as_global(a.frequency)[row];
        if (a.presence) pres = as_global(a.presence)[row];
        global_ptr<const int32_t> ids = as_global(a.tokens) + row * a.tokens_stride;
        uint32_t d[kAhead];
        auto fetch = [&](uint32_t i0) {  // (past the end: the last id again)
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                d[k] = (uint32_t)ids[min(i0 + k * 256 + tid, a.history - 1)];
        };
        if (a.history) fetch(0);
        global_ptr<const int32_t> bias_ids = as_global(a.bias_ids) + row * a.bias_stride;
        uint32_t bias0 = ~0u;
        if (a.n_bias) bias0 = (uint32_t)bias_ids[min((uint32_t)tid, a.n_bias - 1)];
        f32x4 z[kGroups];
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            const int off = (g * 256 + tid) * 4;
            if constexpr (ALIGNED) {  // (at least 8 ids in a row: the group before a span's start is there)
                z[g] = load4<X>(logits + min(off, whole - 4));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) z[g][e] = (float)logits[min(off + e, hi - 1)];
            }
        }
        // the mask words of each group: its first id's, and its last id's where that is another
        global_ptr<const uint32_t> words = as_global(a.mask) + row * a.mask_stride;
        uint32_t w0[kGroups], w1[kGroups];
        if (a.mask) {
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                const uint32_t id = first32 + max((g * 256 + tid) * 4, lo);
                w0[g] = words[min(id, a.vocab - 1) / 32];
                if (ALIGNED && shift) w1[g] = words[min(id + 3, a.vocab - 1) / 32];
            }
        }
#pragma unroll
        for (int g = 0; g < kGroups; ++g) ((u32x4 *)counts)[g * 256 + tid] = u32x4{0, 0, 0, 0};
        // false for the offset of an id that is not the span's (negative ids
        // wrap to at least 2^31 - 1 away)
        auto inside = [&](uint32_t d) { return d - (uint32_t)lo < (uint32_t)(hi - lo); };
        bool biased = false;  // a bias in this span
        if (a.n_bias) {
            biased = inside(bias0 - first32);
            for (uint32_t i = tid + 256; i < a.n_bias; i += 256)
                biased |= inside((uint32_t)bias_ids[i] - first32);
            biased = __any(biased);
            if (tid % kWave == 0) flags[tid / kWave] = biased;
        }
        __syncthreads();
        if (a.n_bias) biased = (flags[0] | flags[1] | flags[2] | flags[3]) != 0;
        const uint32_t len = said < 0 ? 0 : min((uint32_t)said, a.history);
        const uint32_t old = prompt < 0 ? 0 : (uint32_t)prompt;
        for (uint32_t i0 = 0; i0 < len; i0 += 256 * kAhead) {
            if (i0) fetch(i0);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const uint32_t i = i0 + k * 256 + tid;
                const uint32_t at = d[k] - first32;
                if (inside(at) && i < len) {
                    if (i >= old) atomicAdd(&counts[at], 1u);
                    else atomicOr(&counts[at], kSeen);
                }
            }
        }
        __syncthreads();
        auto penalised = [&](float v, uint32_t c) {
            const uint32_t n = c & ~kSeen;
            if (c) v = v > 0.f ? v / rep : v * rep;
            return v - freq * (float)n - (n ? pres : 0.f);
        };
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            const u32x4 c = ((const u32x4 *)counts)[g * 256 + tid];
            if ((c[0] | c[1] | c[2] | c[3]) == 0) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) z[g][e] = penalised(z[g][e], c[e]);
        }
        const int tail = ALIGNED && tid < hi - whole ? whole + tid : -1;
        float zt = 0.f;
        if (tail >= 0) zt = penalised((float)logits[tail], counts[tail]);
        if (biased) {
            __syncthreads();
#pragma unroll
            for (int g = 0; g < kGroups; ++g) ((u32x4 *)entry)[g * 256 + tid] = u32x4{0, 0, 0, 0};
            __syncthreads();
            for (uint32_t i = tid; i < a.n_bias; i += 256) {
                const uint32_t d = (uint32_t)bias_ids[i] - first32;
                if (inside(d)) atomicMax(&entry[d], (int32_t)i + 1);
            }
            __syncthreads();
            global_ptr<const float> values = as_global(a.bias_values) + row * a.bias_stride;
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int32_t b = entry[(g * 256 + tid) * 4 + e];
                    if (b) z[g][e] += values[b - 1];
                }
            if (tail >= 0 && entry[tail]) zt += values[entry[tail] - 1];
        }
        global_ptr<float> out = as_global(a.out) + (int64_t)(row * a.out_stride) + first;
        const bool inner = lo == 0 && whole == (int)kSpan;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            const int off = (g * 256 + tid) * 4;
            if (!inner && off >= whole) continue;
            if (a.mask) {
                uint32_t bits;
                if (!inner && off < lo) bits = w0[g] << lo;
                else if (ALIGNED && shift)
                    bits = __builtin_amdgcn_alignbit(w1[g], w0[g], (first32 + off) % 32);
                else bits = w0[g] >> (first32 + off) % 32;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!((bits >> e) & 1u)) z[g][e] = -__builtin_inff();
            }
            if (ALIGNED && (inner || off >= lo)) {
                *(global_ptr<f32x4>)(out + off) = z[g];
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (off + e >= lo && off + e < hi) out[off + e] = z[g][e];
            }
        }
        if (tail >= 0) {
            const uint32_t id = first32 + tail;
            if (a.mask && !((words[id / 32] >> (id % 32)) & 1u)) zt = -__builtin_inff();
            out[tail] = zt;
        }
        __syncthreads();  // the next row clears the counts
    }
}

// Rows of a grid of `x` workgroups of 256 threads a row (fewer than 2^32
// threads, at most 65535 rows); the kernels loop over the rest.
uint32_t grid_rows(uint32_t rows, uint32_t x) {
    const uint64_t most = std::max<uint64_t>(1, (1ull << 31) / (256ull * x));
    return (uint32_t)std::min<uint64_t>({rows, 65535, most});
}

int launched() { return hipGetLastError() == hipSuccess ? DF11_OK : DF11_ERR_HIP; }

uint64_t size_of(uint32_t type) { return type == DF11_F32 ? 4 : type == DF11_BF16 ? 2 : 1; }

}  // namespace

extern "C" int df11_add_rms_norm(const void *x, uint32_t x_type, uint64_t x_stride,
                                 const void *residual, void *residual_out, uint32_t residual_type,
                                 uint64_t residual_stride, uint64_t residual_out_stride,
                                 const void *weight, uint32_t weight_type, float eps, void *out,
                                 uint32_t out_type, uint64_t out_stride, float *scales,
                                 uint32_t rows, uint32_t width, void *hip_stream) {
    if (width == 0) return DF11_ERR_ARG;
    if (x_type > DF11_F32 || weight_type > DF11_F32) return DF11_ERR_ARG;
    if (out_type != DF11_BF16 && out_type != DF11_E4M3) return DF11_ERR_ARG;
    if (!(eps >= 0.f)) return DF11_ERR_ARG;
    if (rows == 0) return DF11_OK;  // the arrays may be null
    if (!x || !weight || !out) return DF11_ERR_ARG;
    if ((residual == nullptr) != (residual_out == nullptr)) return DF11_ERR_ARG;
    if (residual && residual_type > DF11_F32) return DF11_ERR_ARG;
    if ((out_type == DF11_E4M3) != (scales != nullptr)) return DF11_ERR_ARG;
    if (x_stride < width || out_stride < width ||
        (residual && (residual_stride < width || residual_out_stride < width)))
        return DF11_ERR_ARG;
    // (updated in place, a row stays where it is)
    if (residual && residual == residual_out && rows > 1 && residual_stride != residual_out_stride)
        return DF11_ERR_ARG;
    if (!aligned(x, size_of(x_type)) || !aligned(weight, size_of(weight_type)) ||
        !aligned(out, size_of(out_type)) || (scales && !aligned(scales, 4)) ||
        (residual && (!aligned(residual, size_of(residual_type)) ||
                      !aligned(residual_out, size_of(residual_type)))))
        return DF11_ERR_ARG;
    // 8 elements at a time where every one of them starts on a 16-byte (e4m3
    // output: 8-byte) boundary; element by element otherwise
    bool vec = width % 8 == 0 && aligned(x, 16) && x_stride % 8 == 0 && aligned(weight, 16) &&
               aligned(out, out_type == DF11_E4M3 ? 8 : 16) && out_stride % 8 == 0;
    if (residual)
        vec = vec && aligned(residual, 16) && residual_stride % 8 == 0 && aligned(residual_out, 16) &&
              residual_out_stride % 8 == 0;
    NormArgs a = {x, residual, weight, residual_out, out, scales, x_stride, residual_stride,
                  residual_out_stride, out_stride, 0, rows, width, weight_type == DF11_F32, eps};
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    for (uint64_t row0 = 0; row0 < rows; row0 += kNormRows) {
        a.row0 = (uint32_t)row0;
        if (x_type == DF11_F32) launch_norm<float>(a, residual_type, out_type == DF11_E4M3, vec, s);
        else launch_norm<__bf16>(a, residual_type, out_type == DF11_E4M3, vec, s);
    }
    return launched();
}

extern "C" int df11_silu_mul(const void *gate, uint64_t gate_stride, const void *up,
                             uint64_t up_stride, uint32_t type, uint16_t *out, uint64_t out_stride,
                             uint32_t rows, uint32_t width, void *hip_stream) {
    if (width == 0 || type > DF11_F32) return DF11_ERR_ARG;
    if (rows == 0) return DF11_OK;  // the arrays may be null
    if (!gate || !up || !out) return DF11_ERR_ARG;
    if (gate_stride < width || up_stride < width || out_stride < width) return DF11_ERR_ARG;
    if (!aligned(gate, size_of(type)) || !aligned(up, size_of(type)) || !aligned(out, 2))
        return DF11_ERR_ARG;
    const bool vec = width % 8 == 0 && aligned(gate, 16) && gate_stride % 8 == 0 &&
                     aligned(up, 16) && up_stride % 8 == 0 && aligned(out, 16) &&
                     out_stride % 8 == 0;
    ActArgs a = {gate, up, reinterpret_cast<__bf16 *>(out), gate_stride, up_stride, out_stride,
                 rows, width};
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    const uint32_t across = (uint32_t)(((uint64_t)width + 2047) / 2048);
    const dim3 grid(across, grid_rows(rows, across));
    if (type == DF11_F32) {
        if (vec) hipLaunchKernelGGL((df11_silu_mul_kernel<float, true>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((df11_silu_mul_kernel<float, false>), grid, dim3(256), 0, s, a);
    } else {
        if (vec) hipLaunchKernelGGL((df11_silu_mul_kernel<__bf16, true>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((df11_silu_mul_kernel<__bf16, false>), grid, dim3(256), 0, s, a);
    }
    return launched();
}

extern "C" int df11_logits(const void *logits, uint32_t type, uint64_t stride, float *out,
                           uint64_t out_stride, const int32_t *tokens, uint64_t tokens_stride,
                           uint32_t history, const int32_t *lens, const int32_t *prompt_lens,
                           const float *repetition, const float *frequency, const float *presence,
                           const int32_t *bias_ids, const float *bias_values, uint64_t bias_stride,
                           uint32_t n_bias, const uint32_t *mask, uint64_t mask_stride,
                           uint32_t rows, uint32_t vocab, void *hip_stream) {
    if (vocab == 0 || vocab > 0x7FFFFFFFu || type > DF11_F32) return DF11_ERR_ARG;
    if (rows == 0) return DF11_OK;  // the arrays may be null
    if (!logits || !out) return DF11_ERR_ARG;
    if (stride < vocab || out_stride < vocab) return DF11_ERR_ARG;
    // (in place, a row stays where it is)
    if (logits == out && (type != DF11_F32 || (rows > 1 && stride != out_stride))) return DF11_ERR_ARG;
    if (history > 0x7FFFFFFFu || (history && (!tokens || !lens || tokens_stride < history)))
        return DF11_ERR_ARG;
    if (n_bias && (!bias_ids || !bias_values || bias_stride < n_bias || n_bias > 0x7FFFFFFEu))
        return DF11_ERR_ARG;
    if (mask && mask_stride < ((uint64_t)vocab + 31) / 32) return DF11_ERR_ARG;
    if (!aligned(logits, size_of(type)) || !aligned(out, 4) || !aligned(tokens, 4) ||
        !aligned(lens, 4) || !aligned(prompt_lens, 4) || !aligned(repetition, 4) ||
        !aligned(frequency, 4) || !aligned(presence, 4) || !aligned(bias_ids, 4) ||
        !aligned(bias_values, 4) || !aligned(mask, 4))
        return DF11_ERR_ARG;
    LogitsArgs a = {logits, out, tokens, lens, prompt_lens, bias_ids, repetition, frequency,
                    presence, bias_values, mask, stride, out_stride, tokens_stride, bias_stride,
                    mask_stride, rows, vocab, history, n_bias};
    // 16-byte accesses where a group of 4 ids is aligned in both arrays
    const bool vec = vocab >= 8 && aligned(logits, type == DF11_F32 ? 16 : 8) && aligned(out, 16) &&
                     stride % 4 == out_stride % 4;
    const uint32_t across = (vocab + (vec && stride % 4 ? 3 : 0) + kSpan - 1) / kSpan;
    const dim3 grid(across, grid_rows(rows, across));
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    if (type == DF11_F32) {
        if (vec) hipLaunchKernelGGL((df11_logits_kernel<float, true>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((df11_logits_kernel<float, false>), grid, dim3(256), 0, s, a);
    } else {
        if (vec) hipLaunchKernelGGL((df11_logits_kernel<__bf16, true>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((df11_logits_kernel<__bf16, false>), grid, dim3(256), 0, s, a);
    }
    return launched();
}

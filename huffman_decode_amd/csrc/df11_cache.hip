// The paged 4-bit cache of keys and values: df11_rope_append turns positions
// into the queries and keys of new tokens and stores keys and values;
// df11_kv_read gives stored tokens back as BF16.
//
// A value is held as a 4-bit float (E2M1) and a power of two shared by 32
// channels of one token (one scale byte s: 2^(s - 127)): the form that
// gfx950 converts to and from in one instruction.  Layout of a block (one
// page of P tokens and one key head, P * D * 17 / 16 bytes):
//   key codes    [P][D/2]   byte: channels 2i (low nibble) and 2i + 1
//   value codes  [D/2][P]   byte: one token's channels 2i and 2i + 1
//   key scales   [D/32][P]
//   value scales [D/32][P]
// Values lie token by token within a channel pair because attention's second
// product sums over tokens: 16 bytes are 16 tokens of one operand row, with no
// transposition.  A byte never holds two tokens, so tokens can be stored by
// different threads.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "df11.h"
#include "df11_step.h"

namespace {

using namespace df11_step;

struct CacheView {
    uint8_t *pages;
    uint64_t page_stride, head_stride;
    uint32_t n_pages, kv_heads, dim, page_log2;
    uint32_t *status;
};

struct AppendArgs {
    CacheView c;
    const void *q, *k, *v;
    uint64_t q_stride, q_head, k_stride, k_head, v_stride, v_head;  // elements
    const float *cos, *sin;
    uint64_t cos_stride, sin_stride;
    const int32_t *positions, *slots;
    __bf16 *q_out;
    uint64_t q_out_stride, q_out_head;
    uint32_t tokens, heads, rot, n_pos, adjacent;
    uint32_t head_log2;  // 2^head_log2 threads a head
};

// The scale byte of a block of 32 values whose largest magnitude has these
// bits: the smallest power of two under which it stays below 7 (the next
// value of the format after 6 would be 8, so 7 is where rounding to 6 ends).
// 2^(s - 127) = 2^(floor(log2(amax * 8 / 7)) - 2) for amax's mantissa below or
// above 1.75, by a carry out of the mantissa.  A block that holds an infinity
// or a NaN gets 255: it reads back as NaN.  252 is the largest used, so that
// 6 * 2^125 is finite.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
    if (amax_bits >= 0x7F800000u) return 255u;
    const int e = (int)((amax_bits + 0x200000u) >> 23) - 2;
    return (uint32_t)(e < 1 ? 1 : e > 252 ? 252 : e);
}

// Largest of a value over groups of 4 lanes.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false);  // 1,0,3,2
    v = v > o ? v : o;
    o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false);  // 2,3,0,1
    return v > o ? v : o;
}

// 8 values as E2M1 codes under scale byte s, to nearest even, saturating at 6
__device__ __forceinline__ uint32_t e2m1x8(const float v[8], uint32_t s) {
    const float scale = __uint_as_float(s << 23);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], scale, 3);
    return c;
}

// 8 channels as they are loaded: conversions wait for the loads, so they come later.
template <typename X>
struct Eight {
    static constexpr int kQuads = sizeof(X) / 2;
    u32x4 raw[kQuads];
    __device__ __forceinline__ void load(global_ptr<const X> p) {
#pragma unroll
        for (int i = 0; i < kQuads; ++i) raw[i] = ((global_ptr<const u32x4>)p)[i];
    }
    __device__ __forceinline__ void widen(float v[8]) const {
        if constexpr (kQuads == 2) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(raw[j / 4][j % 4]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = __uint_as_float(j % 2 ? raw[0][j / 2] & 0xFFFF0000u : raw[0][j / 2] << 16);
        }
    }
};

// Rotation of 8 channels x, with their partners y (adjacent pairs: unused) and
// the cosines and sines of their pairs.  Products and sums are rounded one by
// one (no fused multiply-add), as the formula reads.
__device__ __forceinline__ void rotate8(bool adjacent, bool upper, const float c[8], const float s[8],
                                        const float y[8], float x[8]) {
#pragma clang fp contract(off)
    if (adjacent) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float p = x[2 * j], r = x[2 * j + 1];
            const float pc = p * c[j], rs = r * s[j], rc = r * c[j], ps = p * s[j];
            x[2 * j] = pc - rs;
            x[2 * j + 1] = rc + ps;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float xc = x[j] * c[j], ys = y[j] * s[j];
            x[j] = upper ? xc + ys : xc - ys;
        }
    }
}

// The same, channel by channel from memory: any alignment, any even rot.
template <typename X>
__device__ __forceinline__ void rotate_each(const AppendArgs &a, global_ptr<const X> head, uint32_t ch,
                                            int32_t pos, float x[8]) {
#pragma clang fp contract(off)
    const uint32_t half = a.rot / 2;
    global_ptr<const float> cs = as_global(a.cos) + pos * a.cos_stride;
    global_ptr<const float> sn = as_global(a.sin) + pos * a.sin_stride;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t n = ch + j;
        if (n >= a.rot) break;
        const bool upper = a.adjacent ? n & 1 : n >= half;
        const uint32_t i = a.adjacent ? n / 2 : upper ? n - half : n;
        const uint32_t other = a.adjacent ? n ^ 1u : upper ? n - half : n + half;
        const float y = (float)head[other];
        const float xc = x[j] * cs[i], ys = y * sn[i];
        x[j] = upper ? xc + ys : xc - ys;
    }
}

// One thread takes 8 channels of one token in HEADS heads; 4 threads next to
// each other share a block of 32 channels.  A workgroup has 2048 / dim
// neighbouring tokens (blockIdx.x, then gridDim.x further): they lie side by
// side in the value codes and the scales, and bytes of one line that
// workgroups on different XCDs write are merged in memory, not in an L2 (one
// token per workgroup took 71 us for 8191 tokens of 32 + 8 + 8 heads).
// What bounds it is the chain position -> cosines -> result: all heads'
// channels are loaded first, and a workgroup has several heads (VEC).  8191
// tokens, BF16, pages of 16, three sets of inputs in turn: 53 us for 177 MB (33
// at the copy rate) with 2 heads.  On one set, which stays in the 256 MB cache,
// 36 us; 1, 4, 8 and 12 heads took 9, 1, 7 and 13 us more, and 39 in all where
// neighbouring tiles went to different XCDs.
template <typename X, bool VEC, int HEADS>
__global__ __launch_bounds__(256) void df11_rope_append_kernel(AppendArgs a) {
    constexpr int kMostTokens = 32, kMostWords = 256 + kMostTokens;
    __shared__ uint32_t values[kMostWords];  // [token][dim / 8 + 1] codes of 8 channels
    __shared__ int32_t where[kMostTokens];   // the tokens' slots, -1: not stored
    const uint32_t words = 1u << a.head_log2, tokens_here = 256u >> a.head_log2;
    const uint32_t here = threadIdx.x >> a.head_log2, ch = (threadIdx.x & (words - 1)) * 8;
    const uint32_t page_tokens = 1u << a.c.page_log2;
    const uint32_t half = page_tokens * (a.c.dim / 2), group = page_tokens * (a.c.dim / 32);
    const uint32_t all_heads = a.heads + 2 * a.c.kv_heads, head0 = blockIdx.y * HEADS;
    const bool turned = ch < a.rot, upper = ch >= a.rot / 2;
    // VEC: rot is a multiple of 16, so the 8 channels and their partners lie together
    const int partner = !turned || a.adjacent ? 0 : upper ? -(int)(a.rot / 2) : (int)(a.rot / 2);
    // tiles of neighbouring tokens on one XCD (workgroups go to the 8 in turn)
    const uint32_t tile0 = gridDim.x % 8 ? blockIdx.x : blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8;
    for (uint64_t first = (uint64_t)tile0 * tokens_here; first < a.tokens;
         first += (uint64_t)gridDim.x * tokens_here) {
        const uint64_t t = min(first + here, (uint64_t)a.tokens - 1);
        bool live = first + here < a.tokens;
        int32_t pos = as_global(a.positions)[t], slot = as_global(a.slots)[t];
        auto source = [&](uint32_t head) {  // the head's channels of the token
            return head < a.heads
                       ? as_global(static_cast<const X *>(a.q)) + t * a.q_stride + head * a.q_head
                   : head < a.heads + a.c.kv_heads
                       ? as_global(static_cast<const X *>(a.k)) + t * a.k_stride + (head - a.heads) * a.k_head
                       : as_global(static_cast<const X *>(a.v)) + t * a.v_stride +
                             (head - a.heads - a.c.kv_heads) * a.v_head;
        };
        Eight<X> own[HEADS], other[HEADS];
        if constexpr (VEC) {
#pragma unroll
            for (int h = 0; h < HEADS; ++h) {
                const uint32_t head = min(head0 + h, all_heads - 1);
                global_ptr<const X> p = source(head) + ch;
                own[h].load(p);
                other[h].load(p + (head < a.heads + a.c.kv_heads ? partner : 0));
            }
        }
        if (live && (pos < 0 || (uint32_t)pos >= a.n_pos ||
                     (slot >= 0 && ((uint32_t)slot >> a.c.page_log2) >= a.c.n_pages))) {
            if (blockIdx.y == 0 && ch == 0 && a.c.status) atomicAdd(a.c.status, 1u);
            live = false;
        }
        if (!live) slot = -1, pos = 0;
        float c[8], s[8];
        if constexpr (VEC) {
            if (turned && a.adjacent) {
                const f32x4 cv = *(global_ptr<const f32x4>)(as_global(a.cos) + pos * a.cos_stride + ch / 2);
                const f32x4 sv = *(global_ptr<const f32x4>)(as_global(a.sin) + pos * a.sin_stride + ch / 2);
#pragma unroll
                for (int j = 0; j < 4; ++j) c[j] = cv[j], s[j] = sv[j];
            } else if (turned) {
                const uint32_t i = upper ? ch - a.rot / 2 : ch;
                load8<true>(a.cos, pos * a.cos_stride + i, 8, c);
                load8<true>(a.sin, pos * a.sin_stride + i, 8, s);
            }
        }
        const uint32_t page = (uint32_t)slot >> a.c.page_log2, at = slot & (page_tokens - 1);
#pragma unroll
        for (int h = 0; h < HEADS; ++h) {
            const uint32_t head = head0 + h;
            if (head >= all_heads) break;
            const bool query = head < a.heads, value = head >= a.heads + a.c.kv_heads;
            float x[8];
            if constexpr (VEC) {
                own[h].widen(x);
                if (turned && !value) {
                    float y[8];
                    other[h].widen(y);
                    rotate8(a.adjacent, upper, c, s, y, x);
                }
            } else {
                global_ptr<const X> p = source(head);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = (float)p[ch + j];
                if (!value) rotate_each<X>(a, p, ch, pos, x);
            }
            if (query) {
                if (live)
                    store8<VEC>(a.q_out, t * a.q_out_stride + head * a.q_out_head + ch, 8, x);
                continue;
            }
            const uint32_t kvh = head - a.heads - (value ? a.c.kv_heads : 0);
            uint32_t amax = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t m = __float_as_uint(x[j]) & 0x7FFFFFFFu;
                amax = amax > m ? amax : m;
            }
            const uint32_t scale = scale_byte(quad_max(amax));
            const uint32_t codes = e2m1x8(x, scale);
            if (slot >= 0) {
                global_ptr<uint8_t> block =
                    as_global(a.c.pages) + page * a.c.page_stride + kvh * a.c.head_stride;
                if (!value) *(global_ptr<uint32_t>)(block + at * (a.c.dim / 2) + ch / 2) = codes;
                if (ch % 32 == 0)
                    block[2 * half + (value ? group : 0) + ch / 32 * page_tokens + at] = (uint8_t)scale;
            }
            if (!value) continue;
            // values: 4 neighbouring tokens' bytes of a channel pair per thread
            __syncthreads();
            values[here * (words + 1) + ch / 8] = codes;
            if (ch == 0) where[here] = slot;
            __syncthreads();
            const uint32_t quads = tokens_here / 4;
            const uint32_t t4 = threadIdx.x % quads * 4, pair = threadIdx.x / quads;
            uint32_t bytes = 0;
            int32_t to[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                to[i] = where[t4 + i];
                bytes |= ((values[(t4 + i) * (words + 1) + pair / 4] >> (8 * (pair % 4))) & 255u) << (8 * i);
            }
            global_ptr<uint8_t> v = as_global(a.c.pages) + kvh * a.c.head_stride + half + pair * page_tokens;
            if (to[0] >= 0 && to[0] % 4 == 0 && to[1] == to[0] + 1 && to[2] == to[0] + 2 &&
                to[3] == to[0] + 3) {
                *(global_ptr<uint32_t>)(v + ((uint32_t)to[0] >> a.c.page_log2) * a.c.page_stride +
                                        (to[0] & (page_tokens - 1))) = bytes;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (to[i] >= 0)
                        v[((uint32_t)to[i] >> a.c.page_log2) * a.c.page_stride +
                          (to[i] & (page_tokens - 1))] = (uint8_t)(bytes >> (8 * i));
            }
        }
    }
}

struct ReadArgs {
    CacheView c;
    const int32_t *slots;
    __bf16 *k_out, *v_out;
    uint64_t k_stride, k_head, v_stride, v_head;  // elements
    uint32_t tokens, head_log2;
};

// One thread gives 8 channels of one token; a workgroup has 2048 / dim
// neighbouring tokens of one head, whose value codes it reads 4 tokens at a
// time where their slots follow one another.  Bound by memory's latency (slot,
// then scale and codes): 8191 tokens of 8 heads 15 us for 42 MB (8 at the copy rate).
template <bool VEC>
__global__ __launch_bounds__(256) void df11_kv_read_kernel(ReadArgs a) {
    constexpr int kMostTokens = 32, kMostWords = 256 + kMostTokens;
    __shared__ uint32_t values[kMostWords];  // [token][dim / 8 + 1] codes of 8 channels
    const uint32_t words = 1u << a.head_log2, tokens_here = 256u >> a.head_log2;
    const uint32_t here = threadIdx.x >> a.head_log2, ch = (threadIdx.x & (words - 1)) * 8;
    const uint32_t page_tokens = 1u << a.c.page_log2;
    const uint32_t half = page_tokens * (a.c.dim / 2), group = page_tokens * (a.c.dim / 32);
    const bool value = blockIdx.y >= a.c.kv_heads;
    const uint32_t kvh = blockIdx.y - (value ? a.c.kv_heads : 0);
    global_ptr<const uint8_t> head = as_global((const uint8_t *)a.c.pages) + kvh * a.c.head_stride;
    for (uint64_t first = (uint64_t)blockIdx.x * tokens_here; first < a.tokens;
         first += (uint64_t)gridDim.x * tokens_here) {
        const uint64_t t = first + here;
        const bool live = t < a.tokens;
        const int32_t slot = live ? as_global(a.slots)[t] : -1;
        const uint32_t page = (uint32_t)slot >> a.c.page_log2, at = slot & (page_tokens - 1);
        const bool held = slot >= 0 && page < a.c.n_pages;
        if (slot >= 0 && !held && blockIdx.y == 0 && ch == 0 && a.c.status) atomicAdd(a.c.status, 1u);
        uint32_t codes = 0, s = 127;
        if (held) {
            global_ptr<const uint8_t> block = head + page * a.c.page_stride;
            s = block[2 * half + (value ? group : 0) + ch / 32 * page_tokens + at];
            if (!value) codes = *(global_ptr<const uint32_t>)(block + at * (a.c.dim / 2) + ch / 2);
        }
        if (value) {
            const uint32_t quads = tokens_here / 4;
            const uint32_t t4 = threadIdx.x % quads * 4, pair = threadIdx.x / quads;
            int32_t from[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                from[i] = first + t4 + i < a.tokens ? as_global(a.slots)[first + t4 + i] : -1;
                if (from[i] >= 0 && ((uint32_t)from[i] >> a.c.page_log2) >= a.c.n_pages) from[i] = -1;
            }
            global_ptr<const uint8_t> v = head + half + pair * page_tokens;
            uint32_t bytes = 0;
            if (from[0] >= 0 && from[0] % 4 == 0 && from[1] == from[0] + 1 && from[2] == from[0] + 2 &&
                from[3] == from[0] + 3) {
                bytes = *(global_ptr<const uint32_t>)(v + ((uint32_t)from[0] >> a.c.page_log2) * a.c.page_stride +
                                                      (from[0] & (page_tokens - 1)));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (from[i] >= 0)
                        bytes |= (uint32_t)v[((uint32_t)from[i] >> a.c.page_log2) * a.c.page_stride +
                                             (from[i] & (page_tokens - 1))] << (8 * i);
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i)
                ((uint8_t *)values)[((t4 + i) * (words + 1) + pair / 4) * 4 + pair % 4] = (uint8_t)(bytes >> (8 * i));
            __syncthreads();
            codes = values[here * (words + 1) + ch / 8];
        }
        if (!live) continue;
        const float scale = __uint_as_float(s << 23);  // only its exponent is used
        float x[8];
        const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
        const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
        const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
        const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
        x[0] = (float)p0[0], x[1] = (float)p0[1], x[2] = (float)p1[0], x[3] = (float)p1[1];
        x[4] = (float)p2[0], x[5] = (float)p2[1], x[6] = (float)p3[0], x[7] = (float)p3[1];
        if (value) store8<VEC>(a.v_out, t * a.v_stride + kvh * a.v_head + ch, 8, x);
        else store8<VEC>(a.k_out, t * a.k_stride + kvh * a.k_head + ch, 8, x);
    }
}

int launched() { return hipGetLastError() == hipSuccess ? DF11_OK : DF11_ERR_HIP; }

// Heads of a workgroup where there are workgroups enough without that: from
// kManyGroups (tiles of tokens x heads) on.  Appending and reading back, us with 2
// heads and with 1: 128 channels of 48 heads, BF16, 64 tokens (192) 7.6 and 6.3,
// 1024 (3072) 14.1 and 14.3, 1536 (4608) 16.8 and 18.2, 8191 67 and 77; fp32 19.6
// and 18.8 for 1536, 88 and 89 for 8191.  64 channels, BF16, 4096 tokens (6144)
// 18.9 and 20.6; 256 channels of 24 heads 2048 tokens (6144) 21.3 and 22.9.
constexpr int kHeadsHere = 2;
constexpr uint64_t kManyGroups = 4096;

template <typename X, bool VEC, int HEADS>
void launch_append(const AppendArgs &a, uint32_t tiles, uint32_t heads, hipStream_t s) {
    const uint32_t down = (heads + HEADS - 1) / HEADS;
    uint32_t across = std::min(tiles, std::max<uint32_t>(1, (1u << 23) / down));  // < 2^32 threads
    if (across >= 64) across = (across + 7) / 8 * 8;
    const dim3 grid(across, down);
    hipLaunchKernelGGL((df11_rope_append_kernel<X, VEC, HEADS>), grid, dim3(256), 0, s, a);
}

template <typename X>
void launch_append(const AppendArgs &a, bool vec, hipStream_t s) {
    const uint32_t per = 2048 / a.c.dim, tiles = (uint32_t)(((uint64_t)a.tokens + per - 1) / per);
    const uint32_t heads = a.heads + 2 * a.c.kv_heads;
    if (!vec) launch_append<X, false, 1>(a, tiles, heads, s);
    else if ((uint64_t)tiles * heads < kManyGroups) launch_append<X, true, 1>(a, tiles, heads, s);
    else launch_append<X, true, kHeadsHere>(a, tiles, heads, s);
}

}  // namespace

extern "C" uint64_t df11_kv_block_bytes(uint32_t page_tokens, uint32_t dim) {
    if (page_tokens < 16 || page_tokens > 256 || (page_tokens & (page_tokens - 1))) return 0;
    if (dim != 64 && dim != 128 && dim != 256) return 0;
    return (uint64_t)page_tokens * dim * 17 / 16;
}

int df11_step::check_cache(const df11_kv_cache *c) {
    if (!c || !c->pages || c->n_pages == 0 || c->kv_heads == 0) return DF11_ERR_ARG;
    const uint64_t block = df11_kv_block_bytes(c->page_tokens, c->dim);
    if (block == 0) return DF11_ERR_ARG;
    // slots are int32
    if ((uint64_t)c->n_pages * c->page_tokens > 0x80000000ull) return DF11_ERR_ARG;
    if (!aligned(c->pages, 16) || c->page_stride % 16 || c->head_stride % 16) return DF11_ERR_ARG;
    if (!aligned(c->status, 4)) return DF11_ERR_ARG;
    // the blocks lie apart (pages of heads, or heads of pages) and end inside the buffer
    typedef unsigned __int128 u128;
    const u128 page = c->page_stride, head = c->head_stride;
    if (page < block || head < block) return DF11_ERR_ARG;
    if (page < head * (c->kv_heads - 1) + block && head < page * (c->n_pages - 1) + block)
        return DF11_ERR_ARG;
    if (page * (c->n_pages - 1) + head * (c->kv_heads - 1) + block > c->bytes)
        return DF11_ERR_BUFSIZE;
    return DF11_OK;
}

static CacheView view_of(const df11_kv_cache *c) {
    return {c->pages, c->page_stride, c->head_stride, c->n_pages, c->kv_heads, c->dim,
            (uint32_t)__builtin_ctz(c->page_tokens), c->status};
}

extern "C" int df11_rope_append(const df11_kv_cache *cache, const void *q, uint64_t q_stride,
                                uint64_t q_head_stride, const void *k, uint64_t k_stride,
                                uint64_t k_head_stride, const void *v, uint64_t v_stride,
                                uint64_t v_head_stride, uint32_t type, uint32_t heads,
                                const float *cos, uint64_t cos_stride, const float *sin,
                                uint64_t sin_stride, uint32_t n_pos, uint32_t rot,
                                uint32_t adjacent, const int32_t *positions, const int32_t *slots,
                                uint16_t *q_out, uint64_t q_out_stride,
                                uint64_t q_out_head_stride, uint32_t tokens, void *hip_stream) {
    const int st = check_cache(cache);
    if (st != DF11_OK) return st;
    if (type > DF11_F32) return DF11_ERR_ARG;
    if (tokens == 0) return DF11_OK;  // the arrays may be null
    if (!k || !v || !positions || !slots) return DF11_ERR_ARG;
    if (heads && (!q || !q_out || (const void *)q_out == q)) return DF11_ERR_ARG;
    if (heads > 0x3FFFu || cache->kv_heads > 0x3FFFu) return DF11_ERR_ARG;
    const uint32_t dim = cache->dim;
    if (rot > dim || rot % 2 || (rot && (!cos || !sin || n_pos == 0))) return DF11_ERR_ARG;
    if (rot && (cos_stride < rot / 2 || sin_stride < rot / 2)) return DF11_ERR_ARG;
    if (k_head_stride < dim || v_head_stride < dim ||
        (heads && (q_head_stride < dim || q_out_head_stride < dim)))
        return DF11_ERR_ARG;
    // (inputs may repeat a token's row; outputs may not)
    if (heads && tokens > 1 && q_out_stride < dim) return DF11_ERR_ARG;
    const uint64_t size = type == DF11_F32 ? 4 : 2;
    if (!aligned(q, size) || !aligned(k, size) || !aligned(v, size) || !aligned(cos, 4) ||
        !aligned(sin, 4) || !aligned(positions, 4) || !aligned(slots, 4) || !aligned(q_out, 2))
        return DF11_ERR_ARG;
    // 16-byte accesses where every head's row starts on such a boundary
    bool vec = aligned(k, 16) && aligned(v, 16) && k_stride % 8 == 0 && k_head_stride % 8 == 0 &&
               v_stride % 8 == 0 && v_head_stride % 8 == 0 && aligned(cos, 16) && aligned(sin, 16) &&
              cos_stride % 4 == 0 && sin_stride % 4 == 0 && rot % 16 == 0;
    if (heads)
        vec = vec && aligned(q, 16) && q_stride % 8 == 0 && q_head_stride % 8 == 0 &&
              aligned(q_out, 16) && q_out_stride % 8 == 0 && q_out_head_stride % 8 == 0;
    AppendArgs a = {view_of(cache), q, k, v, q_stride, q_head_stride, k_stride, k_head_stride,
                    v_stride, v_head_stride, cos, sin, cos_stride, sin_stride, positions, slots,
                    reinterpret_cast<__bf16 *>(q_out), q_out_stride, q_out_head_stride, tokens,
                    heads, rot, rot ? n_pos : 0x80000000u, adjacent, (uint32_t)__builtin_ctz(dim / 8)};
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    if (type == DF11_F32) launch_append<float>(a, vec, s);
    else launch_append<__bf16>(a, vec, s);
    return launched();
}

extern "C" int df11_kv_read(const df11_kv_cache *cache, const int32_t *slots, uint16_t *k_out,
                            uint64_t k_stride, uint64_t k_head_stride, uint16_t *v_out,
                            uint64_t v_stride, uint64_t v_head_stride, uint32_t tokens,
                            void *hip_stream) {
    const int st = check_cache(cache);
    if (st != DF11_OK) return st;
    if (tokens == 0) return DF11_OK;  // the arrays may be null
    if (!slots || !k_out || !v_out || cache->kv_heads > 0x3FFFu) return DF11_ERR_ARG;
    if (k_head_stride < cache->dim || v_head_stride < cache->dim) return DF11_ERR_ARG;
    if (tokens > 1 && (k_stride < cache->dim || v_stride < cache->dim)) return DF11_ERR_ARG;
    if (!aligned(slots, 4) || !aligned(k_out, 2) || !aligned(v_out, 2)) return DF11_ERR_ARG;
    const bool vec = aligned(k_out, 16) && aligned(v_out, 16) && k_stride % 8 == 0 &&
                     k_head_stride % 8 == 0 && v_stride % 8 == 0 && v_head_stride % 8 == 0;
    ReadArgs a = {view_of(cache), slots, reinterpret_cast<__bf16 *>(k_out),
                  reinterpret_cast<__bf16 *>(v_out), k_stride, k_head_stride, v_stride,
                  v_head_stride, tokens, (uint32_t)__builtin_ctz(cache->dim / 8)};
    const uint32_t per = 2048 / cache->dim, tiles = (uint32_t)(((uint64_t)tokens + per - 1) / per);
    const uint32_t down = 2 * cache->kv_heads;  // (fewer than 2^32 threads: the kernel loops over the rest)
    const dim3 grid(std::min(tiles, std::max<uint32_t>(1, (1u << 23) / down)), down);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    if (vec) hipLaunchKernelGGL(df11_kv_read_kernel<true>, grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL(df11_kv_read_kernel<false>, grid, dim3(256), 0, s, a);
    return launched();
}

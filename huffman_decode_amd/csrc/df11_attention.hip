// df11_attention: attention of new queries over the paged 4-bit cache, and
// its launcher.
//
// For a query row (one query token and query head) s_t = scale q . k_t,
// p = softmax(s) over the tokens it sees, o = sum_t p_t v_t, in one pass over
// the tokens with a running maximum m and sum l.
//
// A wave works on 16 rows that share a key head (its query heads and
// neighbouring tokens) and on tiles of 64 tokens, with
// v_mfma_f32_16x16x32_bf16 (lane = 16 kg + m holds row m, inputs 8 kg .. 8 kg
// + 7 of an operand; outputs row 4 kg + r, column m):
//  * S^T = K Q^T: operand rows are tokens, columns are query rows.  Row m of
//    product i (0..3) is token 4 m + i, so that a lane's outputs are tokens
//    16 kg .. 16 kg + 15 of one query row: the softmax needs no lane but
//    those 16, 32 and 48 away, and only for m and l.
//  * O^T = V^T P^T: those 16 tokens, rounded to BF16, are the lane's inputs of
//    two products as they stand; its 16 bytes of value codes are the same 16
//    tokens of channels 2 (m + 16 j) and 2 (m + 16 j) + 1, and the products of
//    the even and the odd channels give each lane 8 consecutive channels.
// No operand passes through LDS.  Codes become BF16 in one instruction per
// byte, scale included (exact: 2 significant bits).  Scores, m, l and sums are
// 32-bit floats; p is rounded to BF16 as a matrix operand (its sum l is taken
// before the rounding).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "df11.h"
#include "df11_step.h"

namespace {

using namespace df11_step;

constexpr int kWave = 64;
constexpr int kWaves = 4;      // per workgroup
constexpr int kTile = 64;      // tokens
constexpr int kRows = 16;      // query rows of a wave

struct AttnArgs {
    const uint8_t *pages;
    uint64_t page_stride, head_stride;
    uint32_t n_pages, page_log2;
    uint32_t *status;
    const __bf16 *q;
    uint64_t q_stride, q_head;
    const int32_t *q_start, *kv_lens, *table;
    uint64_t table_stride;
    __bf16 *out;
    uint64_t out_stride, out_head;
    float *lse;           // [tokens][heads]
    float *part_o;        // [splits][tokens * heads][dim]
    float *part_ml;       // [splits][tokens * heads][2]
    uint32_t tokens, heads, kv_heads, group, batch;
    uint32_t max_queries, max_kv, chunk, splits, row_blocks;
    uint32_t causal, window;
    float scale_log2;     // |scale| * log2(e), above 0
    uint32_t q_flip;      // sign bits of two queries where scale is below 0
};

// Maximum and sum over the 4 lanes of one query row (16, 32 and 48 away): the
// swaps exchange rows 1 and 3 of one operand with rows 0 and 2 of the other,
// and the upper with the lower half, here of two copies.
__device__ __forceinline__ float across_max(float v) {
    typedef uint32_t u2 __attribute__((ext_vector_type(2)));
    const u2 a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const u2 b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float across_sum(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

__device__ __forceinline__ uint32_t fp4_pair(uint32_t codes, int byte, float scale) {
    bf16x2 r;
    switch (byte) {
        case 0: r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0); break;
        case 1: r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1); break;
        case 2: r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2); break;
        default: r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3); break;
    }
    return __builtin_bit_cast(uint32_t, r);
}

// Scale byte `i` of a dword as the float operand of the conversion, which
// uses the exponent field alone: the bits around it may be anything.
__device__ __forceinline__ float scale_at(uint32_t bytes, int i) {
    return __uint_as_float(i < 3 ? bytes << (23 - 8 * i) : bytes >> 1);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)lo, (__bf16)hi});
}

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// log of the sum that a maximum (in units of log2) and the sum against it stand for
__device__ __forceinline__ float log_sum(float top, float sum) {
    return sum == 0.f ? -__builtin_inff() : (top + __log2f(sum)) * 0.69314718055994531f;
}

// Queries q0 .. q1 - 1 and the number of tokens of a sequence; false (and
// nothing to do) where they do not fit the stated sizes.
__device__ __forceinline__ bool sequence(const AttnArgs &a, uint32_t seq, int64_t &q0, int64_t &q1,
                                         int64_t &kv) {
    q0 = as_global(a.q_start)[seq], q1 = as_global(a.q_start)[seq + 1];
    kv = as_global(a.kv_lens)[seq];
    if (q0 >= 0 && q1 >= q0 && q1 <= a.tokens && q1 - q0 <= a.max_queries && kv >= 0 &&
        kv <= a.max_kv)
        return true;
    q0 = q1 = kv = 0;
    return false;
}

// Codes and scales of a tile of keys: tokens 4 n + i, this lane's channels.
template <int DIM>
struct KeyTile {
    static constexpr int kParts = DIM >= 128 ? DIM / 128 : 1;
    u32x4 codes[4][kParts];
    uint32_t scales[kParts];
    // block: the keys' block, at: token 4 n in it
    __device__ __forceinline__ void load(global_ptr<const uint8_t> block, uint32_t at,
                                         uint32_t page_tokens, int kg) {
        global_ptr<const uint8_t> sc = block + page_tokens * DIM + at;
        global_ptr<const uint8_t> row = block + at * (DIM / 2) + (DIM >= 128 ? 16 : 8) * kg;
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
            scales[p] = *(global_ptr<const uint32_t>)(sc + (DIM >= 128 ? 4 * p + kg : kg / 2) * page_tokens);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (DIM >= 128) {
                    codes[i][p] = *(global_ptr<const u32x4>)(row + i * (DIM / 2) + 64 * p);
                } else {
                    const u32x2 w = *(global_ptr<const u32x2>)(row + i * (DIM / 2));
                    codes[i][p] = u32x4{w.x, w.y, 0, 0};
                }
            }
        }
    }
};

// A lane's 16 tokens of a channel pair (codes, and the scales of its 32-channel
// group) as operands: the even and the odd channel's tokens 8 s .. 8 s + 7.
__device__ __forceinline__ void value_operands(u32x4 codes, u32x4 scales, u32x4 even[2], u32x4 odd[2]) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        uint32_t c[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) c[b] = fp4_pair(codes[w], b, scale_at(scales[w], b));
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            even[w / 2][2 * (w % 2) + b] = __builtin_amdgcn_perm(c[2 * b + 1], c[2 * b], 0x05040100u);
            odd[w / 2][2 * (w % 2) + b] = __builtin_amdgcn_perm(c[2 * b + 1], c[2 * b], 0x07060302u);
        }
    }
}

// The largest scale byte that appending writes for finite values.  Above it are
// 255 (NaN) and, in slots that nobody wrote, 253 and 254, under which codes become
// infinities: 0 times either is NaN, so a zero weight does not hide them.
constexpr uint32_t kTopScale = 252;

// Not 0 where one of 4 scale bytes is above kTopScale.
__device__ __forceinline__ uint32_t above_top(uint32_t bytes) {
    return bytes & ((bytes & 0x7F7F7F7Fu) + 0x01010101u * (255u - kTopScale)) & 0x80808080u;
}

// Values of a tile: tokens 16 kg .., channel pairs n + 16 j.
template <int DIM>
struct ValueTile {
    u32x4 codes[DIM / 32], scales[DIM / 32];
    __device__ __forceinline__ void load(global_ptr<const uint8_t> block, uint32_t at,
                                         uint32_t page_tokens, int n) {
        global_ptr<const uint8_t> v = block + page_tokens * (DIM / 2) + n * page_tokens + at;
        global_ptr<const uint8_t> s = block + page_tokens * (DIM + DIM / 32) + at;
#pragma unroll
        for (int j = 0; j < DIM / 32; ++j) {
            codes[j] = *(global_ptr<const u32x4>)(v + j * 16 * page_tokens);
            scales[j] = *(global_ptr<const u32x4>)(s + j * page_tokens);
        }
    }
    // Scale bytes above kTopScale of tokens out of the product, and the 32-channel
    // groups in which a token of `seen` (the lane's 16 as bits) has one.
    __device__ __forceinline__ bool any_nan() const {
        uint32_t any = 0;
#pragma unroll
        for (int j = 0; j < DIM / 32; ++j)
#pragma unroll
            for (int w = 0; w < 4; ++w) any |= above_top(scales[j][w]);
        return any != 0;
    }
    __device__ __forceinline__ uint32_t nan_groups(uint32_t seen) const {
        uint32_t groups = 0;
#pragma unroll
        for (int j = 0; j < DIM / 32; ++j)
#pragma unroll
            for (int t = 0; t < 16; ++t)
                if (((scales[j][t / 4] >> (8 * (t % 4))) & 255u) > kTopScale && ((seen >> t) & 1u))
                    groups |= 1u << j;
        return groups;
    }
    __device__ __forceinline__ void clear_nan() {
#pragma unroll
        for (int j = 0; j < DIM / 32; ++j)
#pragma unroll
            for (int t = 0; t < 16; ++t)
                if (((scales[j][t / 4] >> (8 * (t % 4))) & 255u) > kTopScale)
                    scales[j][t / 4] &= ~(255u << (8 * (t % 4)));
    }
};

// A row's scores are taken against a maximum m (scaled, in units of log2) that
// may lag behind the true one by up to a slack: p stays below 2^slack, at the
// same relative precision in BF16 and fp32, and few tiles rescale the sums.  It
// is not free: against the true maximum the largest weight is 1 and exact in
// BF16, which counts where few tokens carry a row (error of the output against
// 64 bits, 2 x 4096 prompt queries: slack 0 0.00206, 2 0.00217, 8 0.00233; its
// own rounding alone 0.00166).  Single tokens wait for memory anyway; prompts
// take 564, 551 and 547 us.
constexpr float kSlackFew = 0.f, kSlackRows = 2.f;

// One tile's scores x of a query row (the lane's 16 tokens) into m, l and the
// operands of the second product; o is rescaled when m moves.
template <int kGroups>
__device__ __forceinline__ void softmax_tile(float slack, float x[16], float scale_log2, float &m, float &l,
                                             f32x4 (&o)[kGroups][2], u32x4 pf[2]) {
    float top = x[0];
#pragma unroll
    for (int j = 1; j < 16; ++j) top = fmaxf(top, x[j]);
    top *= scale_log2;
    if (__any(top > m + slack)) {
        top = fmaxf(m, across_max(top));
        const float alpha = __builtin_amdgcn_exp2f(top == -__builtin_inff() ? 0.f : m - top);
        m = top;
        l *= alpha;
#pragma unroll
        for (int j = 0; j < kGroups; ++j) o[j][0] *= alpha, o[j][1] *= alpha;
    }
    const float base = m == -__builtin_inff() ? 0.f : m;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        x[j] = __builtin_amdgcn_exp2f(fmaf(x[j], scale_log2, -base));
        sum += x[j];
    }
    l += sum;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int b = 0; b < 4; ++b) pf[s][b] = pack_bf16(x[8 * s + 2 * b], x[8 * s + 2 * b + 1]);
}

// What a query row sees: tokens from .. to - 1.
struct Sight {
    int from, to;
};

// Few rows (single tokens, their groups of heads): a workgroup's 4 waves take
// the same NT x 16 rows and every fourth tile of the chunk, and join their sums
// through LDS at the end.  Each byte of the cache is read once, and reading it
// is the bound: 64 sequences of 8192 tokens, 32 heads on 8 of 64, 128 and 256
// channels 56, 101 and 197 us (5.1, 5.65 and 5.8 TB/s; this card reads at 6.0), 4
// of 131071 tokens with 64 heads 107 us with the joining kernel, 64 ragged ones
// (at most 8192) 76 us, where the longest sets the end.
// (Two waves per SIMD where the registers allow it, or nearly: 2 x 16 rows of
// 128 channels spill 27 registers and are 1.2 times as fast as with one.  2 x 16
// rows of 256 channels spill 110 with one wave.)
template <int DIM, int NT>
__global__ __launch_bounds__(kWave *kWaves, DIM + 64 * NT <= 256 ? 2 : 1) void df11_attention_kernel(
    AttnArgs a) {
    constexpr int kGroups = DIM / 32;                   // 32-channel groups
    constexpr int kParts = KeyTile<DIM>::kParts;        // 128-channel parts of a key row
    constexpr int kPartSteps = DIM >= 128 ? 4 : 2;      // products of 32 channels per part
    constexpr int kBlockRows = NT * kRows;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int n = lane % 16, kg = lane / 16;

    uint32_t id = blockIdx.x;
    const uint32_t split = id % a.splits;
    id /= a.splits;
    const uint32_t kvh = id % a.kv_heads;
    id /= a.kv_heads;
    const uint32_t row_block = id % a.row_blocks, seq = id / a.row_blocks;

    // the sequence's queries and tokens: nothing is done for one that does not fit the buffers
    int64_t q0, q1, kv;
    const bool bad = !sequence(a, seq, q0, q1, kv);
    if (bad && a.status && row_block == 0 && split == 0 && kvh == 0 && threadIdx.x == 0)
        atomicAdd(a.status, 1u);
    const int queries = (int)(q1 - q0), len = (int)kv, group = (int)a.group;
    const int rows = queries * group;
    const int row0 = (int)row_block * kBlockRows;
    if (row0 >= rows) return;

    // tokens that the wave's rows see together (lo, hi), and that all of them see
    const int before = len - queries;  // position of the first query
    int lo = 0, hi = len, all_lo = 0, all_hi = len;
    {
        const int first = row0 / group, last = (min(row0 + kBlockRows, rows) - 1) / group;
        if (a.causal) hi = min(hi, before + last + 1), all_hi = min(all_hi, before + first + 1);
        if (a.window) {
            lo = (int)max((int64_t)0, (int64_t)before + first - a.window + 1);
            all_lo = (int)max((int64_t)0, (int64_t)before + last - a.window + 1);
        }
    }
    const int64_t c0 = (int64_t)split * a.chunk;
    if (c0 < hi) {
        lo = max(lo, (int)c0);
        hi = (int)min((int64_t)hi, c0 + a.chunk);
    } else {
        hi = 0;  // nothing of this split is seen
    }
    auto row_of = [&](int nt) { return row0 + nt * kRows + n; };
    auto sight = [&](int nt) {
        Sight s = {0, 0};
        if (row_of(nt) < rows) {
            const int pos = before + row_of(nt) / group;
            s.to = a.causal ? min(len, pos + 1) : len;
            if (a.window) s.from = (int)max((int64_t)0, (int64_t)pos - a.window + 1);
        }
        return s;
    };

    // queries: inputs of product (part, s) are channels 128 part + 32 kg + 8 s (DIM 64: 16 kg + 8 s)
    u32x4 qf[NT][kParts * kPartSteps];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const bool live = row_of(nt) < rows;
        const int r = live ? row_of(nt) : row0;
        global_ptr<const __bf16> q = as_global(a.q) + ((uint64_t)q0 + r / group) * a.q_stride +
                                     (kvh * group + r % group) * a.q_head;
#pragma unroll
        for (int p = 0; p < kParts; ++p)
#pragma unroll
            for (int s = 0; s < kPartSteps; ++s) {
                const int ch = DIM >= 128 ? 128 * p + 32 * kg + 8 * s : 16 * kg + 8 * s;
                u32x4 w = *(global_ptr<const u32x4>)(q + ch);
#pragma unroll
                for (int b = 0; b < 4; ++b) w[b] = live ? w[b] ^ a.q_flip : 0;
                qf[nt][p * kPartSteps + s] = w;
            }
    }

    f32x4 o[NT][kGroups][2];  // [32-channel group][even, odd]: channels 32 j + 8 kg + 2 r + parity
    float m[NT], l[NT];       // l: this lane's tokens only
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < kGroups; ++j) o[nt][j][0] = o[nt][j][1] = f32x4{0.f, 0.f, 0.f, 0.f};
        m[nt] = -__builtin_inff(), l[nt] = 0.f;
    }

    const uint32_t page_tokens = 1u << a.page_log2;
    global_ptr<const int32_t> table = as_global(a.table) + seq * a.table_stride;
    // the page that holds token t, as the table says (past the end: the last token's)
    auto page_of = [&](int t) { return (uint32_t)table[(uint32_t)min(t, len - 1) >> a.page_log2]; };
    auto block = [&](uint32_t page) {  // a page out of range reads page 0; its tokens are hidden
        return as_global(a.pages) + (page < a.n_pages ? page : 0) * a.page_stride + kvh * a.head_stride;
    };
    uint32_t bad_pages = 0;

    constexpr int step = kWaves * kTile;
    int t0 = lo / kTile * kTile + wave * kTile;
    if (t0 < hi) {
        // Keys are loaded one tile ahead, values at the start of their tile,
        // pages two tiles ahead (the last tile is loaded again at the end: a
        // branch around the loads would make the compiler wait for all of them).
        const int k_tok = 4 * n, v_tok = 16 * kg;
        uint32_t k_page = page_of(t0 + k_tok), v_page = page_of(t0 + v_tok);
        int next = t0 + step < hi ? t0 + step : t0;
        uint32_t k_page1 = page_of(next + k_tok), v_page1 = page_of(next + v_tok);
        KeyTile<DIM> keys;
        keys.load(block(k_page), (t0 + k_tok) & (page_tokens - 1), page_tokens, kg);
        for (; t0 < hi; t0 += step) {
            ValueTile<DIM> vals;
            vals.load(block(v_page), (t0 + v_tok) & (page_tokens - 1), page_tokens, n);
            const bool v_ok = v_page < a.n_pages;
            bad_pages += !v_ok && t0 + v_tok < len;
            next = t0 + step < hi ? t0 + step : t0;
            const int next2 = next + step < hi ? next + step : next;
            const uint32_t k_page2 = page_of(next2 + k_tok), v_page2 = page_of(next2 + v_tok);
            KeyTile<DIM> keys1;
            keys1.load(block(k_page1), (next + k_tok) & (page_tokens - 1), page_tokens, kg);

            // S^T
            f32x4 sc[NT][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) sc[nt][i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int p = 0; p < kParts; ++p) {
                    const float scale = scale_at(keys.scales[p], i);
#pragma unroll
                    for (int s = 0; s < kPartSteps; ++s) {
                        u32x4 f;
#pragma unroll
                        for (int b = 0; b < 4; ++b) f[b] = fp4_pair(keys.codes[i][p][s], b, scale);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            sc[nt][i] = mfma(f, qf[nt][p * kPartSteps + s], sc[nt][i]);
                    }
                }
            }
            const bool partial = t0 < all_lo || t0 + kTile > all_hi || __any(!v_ok);
            // A hidden token's value must not count even where it is NaN or infinite
            // (0 times that is not 0): such scales are taken out of the product, and
            // rows that do see one get their NaN afterwards.
            bool nans = false;
            if (partial) nans = __any(vals.any_nan());
            u32x4 pf[NT][2];
            uint32_t poisoned[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float x[16];  // the lane's tokens in order: 16 kg + j
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = sc[nt][j % 4][j / 4];
                poisoned[nt] = 0;
                if (partial) {
                    const Sight sg = sight(nt);
                    uint32_t seen = 0;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const int t = t0 + v_tok + j;
                        const bool see = v_ok && t >= sg.from && t < sg.to;
                        seen |= (uint32_t)see << j;
                        x[j] = see ? x[j] : -__builtin_inff();
                    }
                    if (nans) {
                        uint32_t g = vals.nan_groups(seen);
                        g |= (uint32_t)__shfl_xor((int)g, 16);
                        poisoned[nt] = g | (uint32_t)__shfl_xor((int)g, 32);
                    }
                }
                softmax_tile(kSlackFew, x, a.scale_log2, m[nt], l[nt], o[nt], pf[nt]);
            }
            if (nans) vals.clear_nan();
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                u32x4 even[2], odd[2];
                value_operands(vals.codes[j], vals.scales[j], even, odd);
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        o[nt][j][0] = mfma(even[s], pf[nt][s], o[nt][j][0]);
                        o[nt][j][1] = mfma(odd[s], pf[nt][s], o[nt][j][1]);
                    }
            }
            if (nans) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < kGroups; ++j)
                        if ((poisoned[nt] >> j) & 1u) o[nt][j][0] = o[nt][j][1] = f32x4{} + __builtin_nanf("");
            }
            keys = keys1;
            k_page1 = k_page2;
            v_page = v_page1;
            v_page1 = v_page2;
        }
    }
    if (bad_pages && a.status && n == 0) atomicAdd(a.status, bad_pages);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) l[nt] = across_sum(l[nt]);

    // join the waves' tiles
    constexpr int kPitch = DIM + 4;
    __shared__ float lds_o[kWaves][kRows][kPitch];
    __shared__ float lds_m[kWaves][kRows], lds_l[kWaves][kRows];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        if (nt) __syncthreads();
#pragma unroll
        for (int j = 0; j < kGroups; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float *at = &lds_o[wave][n][32 * j + 8 * kg + 2 * r];
                at[0] = o[nt][j][0][r], at[1] = o[nt][j][1][r];
            }
        if (kg == 0) lds_m[wave][n] = m[nt], lds_l[wave][n] = l[nt];
        __syncthreads();
        // thread: row threadIdx / 16, channels (threadIdx % 16) * DIM / 16 ..
        const int at = threadIdx.x / 16, ch = (threadIdx.x % 16) * (DIM / 16);
        const int row = row0 + nt * kRows + at;
        if (row >= rows) continue;
        float top = lds_m[0][at];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) top = fmaxf(top, lds_m[w][at]);
        const float base = top == -__builtin_inff() ? 0.f : top;
        float sum = 0.f, acc[DIM / 16];
#pragma unroll
        for (int c = 0; c < DIM / 16; ++c) acc[c] = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float f = __builtin_amdgcn_exp2f(lds_m[w][at] - base);
            sum += f * lds_l[w][at];
#pragma unroll
            for (int c = 0; c < DIM / 16; ++c) acc[c] += f * lds_o[w][at][ch + c];
        }
        const uint64_t tok = (uint64_t)q0 + row / group;
        const uint32_t head = kvh * group + row % group;
        const uint64_t to = tok * a.heads + head;
        if (a.splits > 1) {
            const uint64_t p = (uint64_t)split * a.tokens * a.heads + to;
#pragma unroll
            for (int c = 0; c < DIM / 16; c += 4)
                *(global_ptr<f32x4>)(as_global(a.part_o) + p * DIM + ch + c) =
                    f32x4{acc[c], acc[c + 1], acc[c + 2], acc[c + 3]};
            if (ch == 0) as_global(a.part_ml)[2 * p] = top, as_global(a.part_ml)[2 * p + 1] = sum;
            continue;
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int c = 0; c < DIM / 16; c += 2)
            *(global_ptr<uint32_t>)(as_global(a.out) + tok * a.out_stride + head * a.out_head + ch + c) =
                pack_bf16(acc[c] * inv, acc[c + 1] * inv);
        if (ch == 0 && a.lse) as_global(a.lse)[to] = log_sum(top, sum);
    }
}

// Barrier that orders LDS accesses only: global loads stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Many rows (prompts): a workgroup's 4 waves take NT x 16 rows each and every
// tile.  Converting codes costs as many instructions as a row tile's softmax, so
// each wave converts a quarter of the next tile into operands in LDS (double
// buffered, one barrier per tile; an operand is 64 lanes x 16 bytes, written and
// read without conflicts) while all of them work on this one.  4096 queries
// over 8192 tokens, causal, 32 heads on 8 of 128 channels (0.41 TFLOP): 424 us,
// 0.97 PFLOP/s (an 8192^3 library product: 1.26).  Vector instructions bind (55 % of
// the time, the matrix cores 38 %, little of it together): softmax, conversion and the reads
// of LDS operands cost 84, 84 and 108 of 429 us where left out one by one.
// 64 channels have half the products to the same softmax: 309 us, 0.67 PFLOP/s
// (66 and 26 %); 256 channels have one wave per SIMD, and nothing hides the
// conversion: 1404 us, 0.59 PFLOP/s (35 and 24 %).
// WHOLE: pages hold at least a tile, so that a tile's addresses are a scalar base
// and lane offsets that never change.
template <int DIM, int NT, bool WHOLE>
__global__ __launch_bounds__(kWave *kWaves, DIM <= 128 ? 2 : 1) void df11_attention_rows_kernel(
    AttnArgs a) {
    constexpr int kGroups = DIM / 32;
    constexpr int kParts = DIM >= 128 ? DIM / 128 : 1;
    constexpr int kPartSteps = DIM >= 128 ? 4 : 2;
    constexpr int kSteps = kParts * kPartSteps;
    constexpr int kWaveRows = NT * kRows, kBlockRows = kWaves * kWaveRows;
    constexpr int kOperands = 4 * kSteps + 4 * kGroups;  // of a tile: keys [i][step], values [j][parity][s]
    __shared__ u32x4 tile[2][kOperands][kWave];
    // per wave: bits 0..3 the 16-token parts without a page, bit 4 a value scale above kTopScale
    __shared__ uint32_t flags[2][kWaves];
    __shared__ uint16_t nans[2][kGroups][4];  // tokens of a part with such a scale, where bit 4 is set
    // (one value per wave: what follows from it stays in scalar registers)
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int n = lane % 16, kg = lane / 16;

    uint32_t id = blockIdx.x;
    const uint32_t split = id % a.splits;
    id /= a.splits;
    const uint32_t kvh = id % a.kv_heads;
    id /= a.kv_heads;
    // the last rows see the most tokens: they start first
    const uint32_t row_block = a.row_blocks - 1 - id % a.row_blocks, seq = id / a.row_blocks;

    int64_t q0, q1, kv;
    const bool bad = !sequence(a, seq, q0, q1, kv);
    if (bad && a.status && row_block == 0 && split == 0 && kvh == 0 && threadIdx.x == 0)
        atomicAdd(a.status, 1u);
    const int queries = (int)(q1 - q0), len = (int)kv, group = (int)a.group;
    const int rows = queries * group;
    const int block0 = (int)row_block * kBlockRows, row0 = block0 + wave * kWaveRows;
    if (block0 >= rows) return;

    const int before = len - queries;  // position of the first query
    // tokens that rows from .. to - 1 see together, and that all of them see
    struct Range {
        int lo, hi, all_lo, all_hi;
    };
    const int64_t c0 = (int64_t)split * a.chunk;
    auto range = [&](int from, int to) {
        Range r = {0, len, 0, len};
        const int first = from / group, last = (min(to, rows) - 1) / group;
        if (a.causal) r.hi = min(len, before + last + 1), r.all_hi = min(len, before + first + 1);
        if (a.window) {
            r.lo = (int)max((int64_t)0, (int64_t)before + first - a.window + 1);
            r.all_lo = (int)max((int64_t)0, (int64_t)before + last - a.window + 1);
        }
        if (from >= rows || c0 >= r.hi) {
            r.lo = r.hi = 0;
        } else {
            r.lo = max(r.lo, (int)c0);
            r.hi = (int)min((int64_t)r.hi, c0 + a.chunk);
        }
        return r;
    };
    const Range all = range(block0, block0 + kBlockRows), my = range(row0, row0 + kWaveRows);
    auto row_of = [&](int nt) { return row0 + nt * kRows + n; };
    auto sight = [&](int nt) {
        Sight s = {0, 0};
        if (row_of(nt) < rows) {
            const int pos = before + row_of(nt) / group;
            s.to = a.causal ? min(len, pos + 1) : len;
            if (a.window) s.from = (int)max((int64_t)0, (int64_t)pos - a.window + 1);
        }
        return s;
    };

    u32x4 qf[NT][kSteps];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const bool live = row_of(nt) < rows;
        const int r = live ? row_of(nt) : block0;
        global_ptr<const __bf16> q = as_global(a.q) + ((uint64_t)q0 + r / group) * a.q_stride +
                                     (kvh * group + r % group) * a.q_head;
#pragma unroll
        for (int p = 0; p < kParts; ++p)
#pragma unroll
            for (int s = 0; s < kPartSteps; ++s) {
                const int ch = DIM >= 128 ? 128 * p + 32 * kg + 8 * s : 16 * kg + 8 * s;
                u32x4 w = *(global_ptr<const u32x4>)(q + ch);
#pragma unroll
                for (int b = 0; b < 4; ++b) w[b] = live ? w[b] ^ a.q_flip : 0;
                qf[nt][p * kPartSteps + s] = w;
            }
    }
    f32x4 o[NT][kGroups][2];
    float m[NT], l[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < kGroups; ++j) o[nt][j][0] = o[nt][j][1] = f32x4{0.f, 0.f, 0.f, 0.f};
        m[nt] = -__builtin_inff(), l[nt] = 0.f;
    }

    const uint32_t page_tokens = 1u << a.page_log2;
    global_ptr<const int32_t> table = as_global(a.table) + seq * a.table_stride;
    // the page of token `tok` of the tile at t0 (WHOLE: of the tile)
    auto page_of = [&](int t0, int tok) {
        const int t = min(WHOLE ? t0 : t0 + tok, len - 1);
        return (uint32_t)table[(uint32_t)t >> a.page_log2];
    };
    auto block = [&](uint32_t page) {
        return as_global(a.pages) + (page < a.n_pages ? page : 0) * a.page_stride + kvh * a.head_stride;
    };
    uint32_t bad_pages = 0;

    // This wave's quarter of a tile: keys 4 n + wave; value groups wave, wave + 4, ..
    constexpr int kMine = (kGroups + kWaves - 1) / kWaves;
    const int k_tok = 4 * n, v_tok = 16 * kg;
    struct Quarter {
        u32x4 k[kParts], v[kMine], vs[kMine];
        uint32_t ks[kParts];
        bool ok;
    };
    auto load = [&](Quarter &x, int t0, uint32_t k_page, uint32_t v_page) {
        // (made scalar here, a tile after the lookup: it would wait for the lookup there)
        if (WHOLE) k_page = __builtin_amdgcn_readfirstlane(k_page);
        // the lane's token in the tile, and the tile's (or the token's) in the page
        const int k_lane = WHOLE ? k_tok : 0, v_lane = WHOLE ? v_tok : 0;
        const uint32_t k_at = (WHOLE ? t0 : t0 + k_tok) & (page_tokens - 1);
        const uint32_t v_at = (WHOLE ? t0 : t0 + v_tok) & (page_tokens - 1);
        global_ptr<const uint8_t> kb = block(k_page), vb = WHOLE ? kb : block(v_page);
        x.ok = (WHOLE ? k_page : v_page) < a.n_pages;
        global_ptr<const uint8_t> ks = kb + page_tokens * DIM + k_at;
        global_ptr<const uint8_t> row = kb + (k_at + wave) * (DIM / 2);
        global_ptr<const uint8_t> vc = vb + page_tokens * (DIM / 2) + v_at;
        global_ptr<const uint8_t> vs = vb + page_tokens * (DIM + DIM / 32) + v_at;
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
            const uint32_t g = DIM >= 128 ? 4 * p + kg : kg / 2;
            x.ks[p] = *(global_ptr<const uint32_t>)(ks + (g * page_tokens + k_lane));
            if constexpr (DIM >= 128) {
                x.k[p] = *(global_ptr<const u32x4>)(row + (uint32_t)(k_lane * (DIM / 2) + 16 * kg + 64 * p));
            } else {
                const u32x2 w = *(global_ptr<const u32x2>)(row + (uint32_t)(k_lane * (DIM / 2) + 8 * kg));
                x.k[p] = u32x4{w.x, w.y, 0, 0};
            }
        }
#pragma unroll
        for (int g = 0; g < kMine; ++g) {
            const uint32_t j = (wave + kWaves * g) % kGroups;  // (64 channels: two waves convert the same)
            x.v[g] = *(global_ptr<const u32x4>)(vc + ((n + 16 * j) * page_tokens + v_lane));
            x.vs[g] = *(global_ptr<const u32x4>)(vs + j * page_tokens + (uint32_t)v_lane);
        }
    };
    auto convert = [&](Quarter &x, int t0, int buf) {
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
            const float scale = wave == 3 ? scale_at(x.ks[p], 3) : __uint_as_float(x.ks[p] << (23 - 8 * wave));
#pragma unroll
            for (int s = 0; s < kPartSteps; ++s) {
                u32x4 f;
#pragma unroll
                for (int b = 0; b < 4; ++b) f[b] = fp4_pair(x.k[p][s], b, scale);
                tile[buf][wave * kSteps + p * kPartSteps + s][lane] = f;
            }
        }
        uint32_t any = 0;
#pragma unroll
        for (int g = 0; g < kMine; ++g)
#pragma unroll
            for (int w = 0; w < 4; ++w) any |= above_top(x.vs[g][w]);
        const bool nan = __any(any != 0);
        if (nan) {  // out of the product, and noted for the rows that see them
#pragma unroll
            for (int g = 0; g < kMine; ++g) {
                uint32_t tokens = 0;
#pragma unroll
                for (int t = 0; t < 16; ++t)
                    if (((x.vs[g][t / 4] >> (8 * (t % 4))) & 255u) > kTopScale) {
                        x.vs[g][t / 4] &= ~(255u << (8 * (t % 4)));
                        tokens |= 1u << t;
                    }
                if (n == 0) nans[buf][(wave + kWaves * g) % kGroups][kg] = (uint16_t)tokens;
            }
        }
#pragma unroll
        for (int g = 0; g < kMine; ++g) {
            const int j = (wave + kWaves * g) % kGroups;
            u32x4 even[2], odd[2];
            value_operands(x.v[g], x.vs[g], even, odd);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                tile[buf][4 * kSteps + j * 4 + s][lane] = even[s];
                tile[buf][4 * kSteps + j * 4 + 2 + s][lane] = odd[s];
            }
        }
        const uint64_t hidden = __ballot(!x.ok);  // 16 equal bits per part
        if (lane == 0)
            flags[buf][wave] = (uint32_t)(hidden & 1) | (uint32_t)(hidden >> 16 & 1) << 1 |
                               (uint32_t)(hidden >> 32 & 1) << 2 | (uint32_t)(hidden >> 48 & 1) << 3 |
                               (nan ? 16u : 0u);
        if (wave == 0) bad_pages += !x.ok && t0 + v_tok < len;
    };

    const int begin = all.lo / kTile * kTile;
    if (begin < all.hi) {
        auto after = [&](int t) { return t + kTile < all.hi ? t + kTile : t; };  // (the last tile again)
        Quarter x;
        load(x, begin, page_of(begin, k_tok), page_of(begin, v_tok));
        int next = after(begin);
        uint32_t k_page = page_of(next, k_tok), v_page = page_of(next, v_tok);
        convert(x, begin, 0);
        load(x, next, k_page, v_page);
        int next2 = after(next);
        k_page = page_of(next2, k_tok), v_page = page_of(next2, v_tok);
        lds_barrier();
        int buf = 0;
        for (int t0 = begin; t0 < all.hi; t0 += kTile, buf ^= 1) {
            if (t0 < my.hi && t0 + kTile > my.lo) {
                uint32_t flag = flags[buf][0];
#pragma unroll
                for (int w = 1; w < kWaves; ++w) flag |= flags[buf][w];
                f32x4 sc[NT][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) sc[nt][i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int s = 0; s < kSteps; ++s) {
                        const u32x4 f = tile[buf][i * kSteps + s][lane];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) sc[nt][i] = mfma(f, qf[nt][s], sc[nt][i]);
                    }
                }
                const bool partial = t0 < my.all_lo || t0 + kTile > my.all_hi || flag != 0;
                u32x4 pf[NT][2];
                uint32_t poisoned[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float y[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) y[j] = sc[nt][j % 4][j / 4];
                    poisoned[nt] = 0;
                    if (partial) {
                        const Sight sg = sight(nt);
                        const bool ok = !((flag >> kg) & 1u);
                        uint32_t seen = 0;
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const int t = t0 + v_tok + j;
                            const bool see = ok && t >= sg.from && t < sg.to;
                            seen |= (uint32_t)see << j;
                            y[j] = see ? y[j] : -__builtin_inff();
                        }
                        if (flag & 16u) {
                            uint32_t g = 0;
#pragma unroll
                            for (int j = 0; j < kGroups; ++j)  // (group j is wave j % 4's to note)
                                if ((flags[buf][j % kWaves] & 16u) && (nans[buf][j][kg] & seen)) g |= 1u << j;
                            g |= (uint32_t)__shfl_xor((int)g, 16);
                            poisoned[nt] = g | (uint32_t)__shfl_xor((int)g, 32);
                        }
                    }
                    softmax_tile(kSlackRows, y, a.scale_log2, m[nt], l[nt], o[nt], pf[nt]);
                }
#pragma unroll
                for (int j = 0; j < kGroups; ++j)
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const u32x4 even = tile[buf][4 * kSteps + j * 4 + s][lane];
                        const u32x4 odd = tile[buf][4 * kSteps + j * 4 + 2 + s][lane];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            o[nt][j][0] = mfma(even, pf[nt][s], o[nt][j][0]);
                            o[nt][j][1] = mfma(odd, pf[nt][s], o[nt][j][1]);
                        }
                    }
                if (flag & 16u) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < kGroups; ++j)
                            if ((poisoned[nt] >> j) & 1u)
                                o[nt][j][0] = o[nt][j][1] = f32x4{} + __builtin_nanf("");
                }
            }
            if (t0 + kTile < all.hi) {  // the next tile, and loads for the one after
                convert(x, next, buf ^ 1);
                next = next2;
                load(x, next, k_page, v_page);
                next2 = after(next);
                k_page = page_of(next2, k_tok), v_page = page_of(next2, v_tok);
            }
            lds_barrier();
        }
    }
    if (bad_pages && a.status && n == 0) atomicAdd(a.status, bad_pages);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) l[nt] = across_sum(l[nt]);

#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int row = row_of(nt);
        if (row >= rows) continue;
        const uint64_t tok = (uint64_t)q0 + row / group;
        const uint32_t head = kvh * group + row % group;
        const uint64_t to = tok * a.heads + head;
        if (a.splits > 1) {
            const uint64_t p = (uint64_t)split * a.tokens * a.heads + to;
#pragma unroll
            for (int j = 0; j < kGroups; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    *(global_ptr<f32x4>)(as_global(a.part_o) + p * DIM + 32 * j + 8 * kg + 4 * h) =
                        f32x4{o[nt][j][0][2 * h], o[nt][j][1][2 * h], o[nt][j][0][2 * h + 1],
                              o[nt][j][1][2 * h + 1]};
            if (kg == 0) as_global(a.part_ml)[2 * p] = m[nt], as_global(a.part_ml)[2 * p + 1] = l[nt];
            continue;
        }
        const float inv = l[nt] == 0.f ? 0.f : 1.f / l[nt];
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
            u32x4 w;
#pragma unroll
            for (int r = 0; r < 4; ++r) w[r] = pack_bf16(o[nt][j][0][r] * inv, o[nt][j][1][r] * inv);
            *(global_ptr<u32x4>)(as_global(a.out) + tok * a.out_stride + head * a.out_head + 32 * j +
                                 8 * kg) = w;
        }
        if (kg == 0 && a.lse) as_global(a.lse)[to] = log_sum(m[nt], l[nt]);
    }
}

// Joins the splits: one workgroup per query row, its 4 waves take every fourth
// split, each with DIM / 64 channels per lane.  5 us for 256 rows of 16 splits:
// the latency of two chains of loads.
template <int DIM>
__global__ __launch_bounds__(kWave *kWaves) void df11_attention_join_kernel(AttnArgs a) {
    constexpr int kCh = DIM / 64;
    __shared__ float lds_o[kWaves][DIM];
    __shared__ float lds_m[kWaves], lds_l[kWaves];
    const uint64_t n = (uint64_t)a.tokens * a.heads;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    for (uint64_t row = blockIdx.x; row < n; row += gridDim.x) {
        const uint32_t token = (uint32_t)(row / a.heads), head = (uint32_t)(row % a.heads);
        // rows of no sequence are left alone: nobody wrote their parts
        bool mine = false;
        for (uint32_t b = lane; b < a.batch; b += kWave) {
            int64_t q0, q1, kv;
            mine |= sequence(a, b, q0, q1, kv) && token >= q0 && token < q1;
        }
        if (!__any(mine)) continue;  // the same in every wave: no barrier is missed
        float top = -__builtin_inff(), sum = 0.f, acc[kCh];
#pragma unroll
        for (int c = 0; c < kCh; ++c) acc[c] = 0.f;
#pragma unroll 4
        for (uint32_t s = wave; s < a.splits; s += kWaves) {
            const uint64_t p = s * n + row;
            const float ms = as_global(a.part_ml)[2 * p], ls = as_global(a.part_ml)[2 * p + 1];
            float x[kCh];
#pragma unroll
            for (int c = 0; c < kCh; ++c) x[c] = as_global(a.part_o)[p * DIM + kCh * lane + c];
            const float now = fmaxf(top, ms), base = now == -__builtin_inff() ? 0.f : now;
            const float f = __builtin_amdgcn_exp2f(top - base), g = __builtin_amdgcn_exp2f(ms - base);
            top = now;
            sum = sum * f + ls * g;
#pragma unroll
            for (int c = 0; c < kCh; ++c) acc[c] = acc[c] * f + x[c] * g;
        }
#pragma unroll
        for (int c = 0; c < kCh; ++c) lds_o[wave][kCh * lane + c] = acc[c];
        if (lane == 0) lds_m[wave] = top, lds_l[wave] = sum;
        __syncthreads();
        if (wave == 0) {
#pragma unroll
            for (int w = 1; w < kWaves; ++w) top = fmaxf(top, lds_m[w]);
            const float base = top == -__builtin_inff() ? 0.f : top;
            sum = 0.f;
#pragma unroll
            for (int c = 0; c < kCh; ++c) acc[c] = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float f = __builtin_amdgcn_exp2f(lds_m[w] - base);
                sum += f * lds_l[w];
#pragma unroll
                for (int c = 0; c < kCh; ++c) acc[c] += f * lds_o[w][kCh * lane + c];
            }
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
            for (int c = 0; c < kCh; ++c)
                as_global(a.out)[token * a.out_stride + head * a.out_head + kCh * lane + c] =
                    (__bf16)(acc[c] * inv);
            if (lane == 0 && a.lse) as_global(a.lse)[row] = log_sum(top, sum);
        }
        __syncthreads();
    }
}

// How a call is cut: row blocks per sequence and key head, chunks of tokens.
struct Plan {
    bool shared;
    uint32_t nt, row_blocks, chunk, splits;
    uint64_t groups, workspace;
};

// Up to this many rows of a key head, waves split the tokens; above, the rows
// (us with either kernel, 8 key heads; 8 sequences of 8192 tokens: 64 channels
// 64 rows 41 and 44, 80 rows 45 and 46, 128 rows 57 and 52; 128 channels 64 rows
// 51 and 54, 80 rows 78 and 58; 256 channels 64 rows 149 and 151, 80 rows 234 and
// 155; 32 sequences of 4096 tokens: 32 rows 41 and 63, 62 and 76, 149 and 263.
// One sequence alone of 128 or 256 channels is faster over its rows from 20 on:
// 20 and 16, 43 and 26).
constexpr uint32_t kSharedRows = 64;
// Workgroups that are resident at once on 256 compute units: a call's tokens are
// cut to fill them at most once.  A second, partly filled round costs more than
// uneven lengths do (128 channels, 4 x 131071 tokens: 512 workgroups 105 us, 768
// 125, 1024 109, 2048 118; 64 ragged sequences of at most 8192: 78, 90, 86, 98.
// 24 sequences of 8192: 64 channels, 512, 768 and 1024 workgroups 37, 30 and 37;
// 256 channels, 256, 512 and 768 workgroups 89, 103 and 95).
constexpr uint64_t shared_groups(uint32_t dim) { return dim == 64 ? 768 : dim == 128 ? 512 : 256; }
// The same for rows, at the number that is resident for 128 channels (2 prompts
// of 512 queries over 8192 tokens: 256, 512 and 768 workgroups 211, 187 and 200
// us; 1 of 128 queries 45, 44 and 52).  64 channels have 768 resident and 256
// channels 256, but what they gain depends on the rows: 64 channels 174, 155
// and 142, 36, 33 and 35; 256 channels 457, 527 and 538, 84, 101 and 123, but 300
// queries of 40 heads on 8 252, 228 and 235.
constexpr uint64_t kRowGroups = 512;
// The fewest tokens of a chunk.
constexpr uint32_t kSharedChunk = 1024, kRowChunk = 256;
// Up to this many tokens a sequence of single tokens is not cut: a second chunk
// costs the kernel that joins them, as much as 3, 2 and 1 more steps of 256
// tokens (whole and cut, us, 1 sequence of 32 heads on 8: 64 channels 1536 tokens
// 8.7 and 9.7, 1792 9.4 and 9.7, 1900 10.5 and 10.2; 128 channels 1281 11.1 and
// 11.3, 1536 10.8 and 11.3, 1700 12.3 and 11.3; 256 channels 1031 17.2 and 17.3,
// 1281 19.3 and 17.3; 8 sequences cross at the same lengths).
constexpr uint32_t whole_tokens(uint32_t dim) {
    return kSharedChunk + (dim == 64 ? 3 : dim == 128 ? 2 : 1) * kTile * kWaves;
}

int plan_for(uint32_t dim, uint32_t kv_heads, uint32_t tokens, uint32_t heads, uint32_t batch,
             uint32_t max_queries, uint32_t max_kv, Plan *p) {
    const uint64_t rows = (uint64_t)max_queries * (heads / kv_heads);
    if (rows > 0x40000000ull || max_kv > 0x7FFF0000u) return DF11_ERR_ARG;
    p->shared = rows <= kSharedRows;
    p->nt = rows > kRows ? 2 : 1;
    const uint32_t per = p->nt * kRows * (p->shared ? 1 : kWaves);
    p->row_blocks = (uint32_t)((rows + per - 1) / per);
    // a launch has fewer than 2^32 threads (counted in 128 bits: the product may pass 64)
    typedef unsigned __int128 u128;
    const u128 all = (u128)batch * kv_heads * p->row_blocks;
    if (all > 0x00FFFFFFull) return DF11_ERR_ARG;
    const uint64_t units = std::max<uint64_t>(1, (uint64_t)all);
    const uint32_t least = p->shared ? kSharedChunk : kRowChunk;
    const uint64_t most = std::max<uint64_t>(1, ((uint64_t)max_kv + least - 1) / least);
    const uint64_t want = std::max<uint64_t>(
        1, std::min(most, (p->shared ? shared_groups(dim) : kRowGroups) / units));
    const uint32_t unit = p->shared ? kTile * kWaves : kTile;
    p->chunk = (uint32_t)((max_kv + want - 1) / want);
    p->chunk = std::max(p->shared && max_kv <= whole_tokens(dim) ? whole_tokens(dim) : least,
                        (p->chunk + unit - 1) / unit * unit);
    p->splits = (uint32_t)std::max<uint64_t>(1, ((uint64_t)max_kv + p->chunk - 1) / p->chunk);
    p->groups = (uint64_t)all * p->splits;
    p->workspace = p->splits > 1 ? (uint64_t)p->splits * tokens * heads * (dim + 2) * 4 : 0;
    if (p->groups > 0x00FFFFFFull) return DF11_ERR_ARG;
    return DF11_OK;
}

template <int DIM>
void launch(const AttnArgs &a, const Plan &p, hipStream_t s) {
    const dim3 grid((uint32_t)p.groups), block(kWave * kWaves);
    if (p.shared && p.nt == 1)
        hipLaunchKernelGGL((df11_attention_kernel<DIM, 1>), grid, block, 0, s, a);
    else if (p.shared)
        hipLaunchKernelGGL((df11_attention_kernel<DIM, 2>), grid, block, 0, s, a);
    else if ((1u << a.page_log2) >= kTile)
        hipLaunchKernelGGL((df11_attention_rows_kernel<DIM, 2, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((df11_attention_rows_kernel<DIM, 2, false>), grid, block, 0, s, a);
    if (p.splits > 1) {
        const uint64_t rows = (uint64_t)a.tokens * a.heads;
        hipLaunchKernelGGL(df11_attention_join_kernel<DIM>,
                           dim3((uint32_t)std::min<uint64_t>(rows, 1u << 20)), block, 0, s, a);
    }
}

}  // namespace

extern "C" uint64_t df11_attention_workspace_bytes(const df11_kv_cache *cache, uint32_t tokens,
                                                   uint32_t heads, uint32_t batch,
                                                   uint32_t max_queries, uint32_t max_kv) {
    Plan p;
    if (check_cache(cache) != DF11_OK || heads == 0 || heads % cache->kv_heads) return 0;
    if (plan_for(cache->dim, cache->kv_heads, tokens, heads, batch, max_queries, max_kv, &p) !=
        DF11_OK)
        return 0;
    return p.workspace;
}

extern "C" int df11_attention(const df11_kv_cache *cache, const uint16_t *q, uint64_t q_stride,
                              uint64_t q_head_stride, uint32_t tokens, uint32_t heads,
                              const int32_t *q_start, const int32_t *kv_lens, uint32_t batch,
                              const int32_t *page_table, uint64_t table_stride,
                              uint32_t table_cols, uint32_t max_queries, uint32_t max_kv,
                              float scale, uint32_t causal, uint32_t window, uint16_t *out,
                              uint64_t out_stride, uint64_t out_head_stride, float *lse,
                              void *workspace, uint64_t workspace_bytes, void *hip_stream) {
    const int st = check_cache(cache);
    if (st != DF11_OK) return st;
    if (tokens == 0 || batch == 0 || max_queries == 0) return DF11_OK;  // the arrays may be null
    if (!q || !out || !q_start || !kv_lens) return DF11_ERR_ARG;
    if (max_kv && !page_table) return DF11_ERR_ARG;
    if (heads == 0 || heads % cache->kv_heads || heads > 0xFFFFu) return DF11_ERR_ARG;
    if (!std::isfinite(scale) || table_stride < table_cols) return DF11_ERR_ARG;
    if (max_kv > (uint64_t)table_cols * cache->page_tokens) return DF11_ERR_ARG;
    if (q_head_stride < cache->dim || out_head_stride < cache->dim) return DF11_ERR_ARG;
    // (queries may repeat a token's row; outputs may not)
    if (tokens > 1 && out_stride < cache->dim) return DF11_ERR_ARG;
    if (!aligned(q, 16) || q_stride % 8 || q_head_stride % 8 || !aligned(out, 16) ||
        out_stride % 8 || out_head_stride % 8 || !aligned(q_start, 4) || !aligned(kv_lens, 4) ||
        !aligned(page_table, 4) || !aligned(lse, 4))
        return DF11_ERR_ARG;
    if (tokens > 0x7FFFFFFFu) return DF11_ERR_ARG;
    Plan p;
    const int ps = plan_for(cache->dim, cache->kv_heads, tokens, heads, batch, max_queries, max_kv, &p);
    if (ps != DF11_OK) return ps;
    if (p.workspace && (!workspace || !aligned(workspace, 16))) return DF11_ERR_ARG;
    if (workspace_bytes < p.workspace) return DF11_ERR_BUFSIZE;
    AttnArgs a = {};
    a.pages = cache->pages;
    a.page_stride = cache->page_stride;
    a.head_stride = cache->head_stride;
    a.n_pages = cache->n_pages;
    a.page_log2 = (uint32_t)__builtin_ctz(cache->page_tokens);
    a.status = cache->status;
    a.q = reinterpret_cast<const __bf16 *>(q);
    a.q_stride = q_stride;
    a.q_head = q_head_stride;
    a.q_start = q_start;
    a.kv_lens = kv_lens;
    a.table = page_table;
    a.table_stride = table_stride;
    a.out = reinterpret_cast<__bf16 *>(out);
    a.out_stride = out_stride;
    a.out_head = out_head_stride;
    a.lse = lse;
    a.part_o = static_cast<float *>(workspace);
    a.part_ml = a.part_o + (p.splits > 1 ? (uint64_t)p.splits * tokens * heads * cache->dim : 0);
    a.tokens = tokens;
    a.heads = heads;
    a.kv_heads = cache->kv_heads;
    a.group = heads / cache->kv_heads;
    a.batch = batch;
    a.max_queries = max_queries;
    a.max_kv = max_kv;
    a.chunk = p.chunk;
    a.splits = p.splits;
    a.row_blocks = p.row_blocks;
    a.causal = causal;
    a.window = window;
    // (a scale of 0 becomes one that leaves every weight at 1: hidden scores are -inf, and 0 * inf is NaN)
    a.scale_log2 = std::max(std::fabs(scale) * 1.44269504088896341f, 1e-37f);
    a.q_flip = scale < 0.f ? 0x80008000u : 0u;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    if (cache->dim == 64) launch<64>(a, p, s);
    else if (cache->dim == 128) launch<128>(a, p, s);
    else launch<256>(a, p, s);
    return hipGetLastError() == hipSuccess ? DF11_OK : DF11_ERR_HIP;
}

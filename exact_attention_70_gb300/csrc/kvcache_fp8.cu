// kvcache_fp8.cu -- writing the 8-bit paged KV cache and reading it back.
//
// The cache keeps e4m3 codes [num_pages, page_size, Hkv, d] and, per (token, kv head), one
// scale byte b that stands for 2^(b - 127), laid out [num_pages, Hkv, page_size].  A row x of d
// elements is stored with
//   e = the smallest integer >= -126 with max|x| <= 448 2^e,   b = e + 127,
//   code = e4m3(x 2^-e), to the nearest, ties to even;
// an element that is not finite gets the NaN code and does not count for the maximum.  A power
// of two costs e4m3 no precision (only the border of its subnormals moves by less than one
// bit), makes code 2^e exact in bf16, so that reading back is exact, and fits one byte.
//
// Keys are rotated first (kvcache.cu states the rotation), and the rotated value a cos - b sin
// goes to e4m3 as if it were rounded once.  Kahan's fp32 form of it is within 1.5 units in the
// last place (kvcache.cu).  Where the codes of that value less and plus 2^-21 of itself differ (or
// the scales of the row's largest), about one element in 2^16, the warp forms the
// value again as an unevaluated sum of two fp32 numbers (Dekker's and Knuth's error-free product
// and sum), brought to one by rounding to odd, after which rounding to a shorter format gives
// what rounding the exact value would (S. Boldo, G. Melquiond, "Emulation of FMA and correctly
// rounded sums: proved algorithms using rounding to odd", 2008).  Both forms need their products'
// low parts (2^-48 of the product) above fp32's 2^-149: rows below 2^-90 are formed again times 2^64,
// and rows whose rotated elements pass fp32's range (which the cache holds: 448 2^120) times 2^-64.
#include <cuda_bf16.h>

#include "kernels.h"
#include "ptx.cuh"

namespace attn {

namespace {

__device__ __forceinline__ int find_seq(const int* cu, int batch, int t) {
    int lo = 0, hi = batch - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// One block's check that cu_seqlens describe rows of a packed tensor of `total` rows.
__device__ __forceinline__ void check_offsets(const int* cu, int batch, int total, unsigned* status) {
    bool ok = true;
    for (int b = threadIdx.x; b < batch; b += blockDim.x)
        ok = ok && 0 <= cu[b] && cu[b] <= cu[b + 1] && cu[b + 1] <= total;
    if (!ok) atomicOr(status, kStatusBounds);
}

// a b - c d as one fp32 number, rounded to odd.
__device__ __forceinline__ float det2_odd(float a, float b, float c, float d) {
    const float ph = __fmul_rn(a, b), pl = __fmaf_rn(a, b, -ph);
    const float wh = __fmul_rn(c, d), wl = __fmaf_rn(c, d, -wh);
    const float s = __fsub_rn(ph, wh);  // s + t = ph - wh exactly
    const float bb = __fsub_rn(s, ph);
    const float t = __fsub_rn(__fsub_rn(ph, __fsub_rn(s, bb)), __fadd_rn(wh, bb));
    const float r = __fadd_rn(t, __fsub_rn(pl, wl));
    const float hi = __fadd_rn(s, r);  // hi + lo = s + r exactly
    const float z = __fsub_rn(hi, s);
    const float lo = __fadd_rn(__fsub_rn(s, __fsub_rn(hi, z)), __fsub_rn(r, z));
    const int u = __float_as_int(hi);
    const int towards = ((__float_as_int(lo) ^ u) < 0) ? -1 : 1;  // lo's side of hi
    return __int_as_float((lo != 0.f && (u & 1) == 0) ? u + towards : u);
}

// 8 elements as four fp32 pairs.
__device__ __forceinline__ void unpack_pairs(const uint4& w, uint64_t* x) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = f2_make(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
}

// The rotation of 8 elements, in pairs: y = x c + z s, z the partner plane's elements, s signed
// (c and s hold each table entry twice when interleaved).
struct Turn {
    uint64_t c[4], s[4];
};

// Kahan's form: w = z s rounded, e = z s - w exactly, y = (x c + w) + e.
__device__ __forceinline__ uint64_t turn_pair(uint64_t c, uint64_t s, uint64_t x, uint64_t z) {
    const uint64_t w = f2_mul(z, s);
    const uint64_t e = f2_fma(z, s, f2_mul(w, f2_make(-1.f, -1.f)));
    return f2_add(f2_fma(x, c, w), e);
}

// The same to one fp32 number each, rounded to odd.
__device__ __forceinline__ uint64_t turn_pair_odd(uint64_t c, uint64_t s, uint64_t x, uint64_t z) {
    float x0, x1, z0, z1, c0, c1, s0, s1;
    f2_split(x, x0, x1);
    f2_split(z, z0, z1);
    f2_split(c, c0, c1);
    f2_split(s, s0, s1);
    return f2_make(det2_odd(x0, c0, z0, -s0), det2_odd(x1, c1, z1, -s1));
}

// The largest |y| of a lane's 16; NaNs do not count.
__device__ __forceinline__ float lane_top(const uint64_t (&y)[8]) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float a, b;
        f2_split(y[i], a, b);
        top = fmax3(top, fabsf(a), fabsf(b));
    }
    return top;
}

// The bits of the largest |y| of a run of 8.
__device__ __forceinline__ int run_top(const uint64_t* y) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        f2_split(y[i], a, b);
        top = fmax3(top, fabsf(a), fabsf(b));
    }
    return __float_as_int(top);
}

// The largest over the kLanes lanes of a row.
template <int kLanes>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// 448 = 1.75 2^8: the exponent of the largest magnitude (u: its bits) less 8, one more when its
// significand is above 1.75.
__device__ __forceinline__ int scale_exponent(int u) {
    return (u >> 23) - 8 + ((u & 0x7fffff) > 0x600000 ? 1 : 0);
}
__device__ __forceinline__ int scale_byte(int u) { return max(1, scale_exponent(u)); }

// A lane's largest rotated magnitude (its bits) that asks for the row to be formed again with another
// exponent: below 2^-90 (zeros are exact) or beyond fp32's range.
__device__ __forceinline__ bool off_range(int u) {
    return static_cast<unsigned>(u - 1) < static_cast<unsigned>((127 - 90) << 23) - 1 || u >= 0x7f800000;
}

// Multiplies a staged row of bf16 by 2^k so that its products stay clear of both ends of fp32's range,
// and gives k.  Exact but for elements 2^-190 of the row's largest.  (Rare, so in loops.)
template <int kLanes>
__device__ __forceinline__ int scale_row(uint8_t* row, int l) {
    uint32_t* const w = reinterpret_cast<uint32_t*>(row) + l;  // words l, l + kLanes, ...
    int top = 0;
#pragma unroll 1
    for (int j = 0; j < 8; ++j) {
        const int a = (w[j * kLanes] >> 7) & 0xff, b = (w[j * kLanes] >> 23) & 0xff;
        top = max(top, max(a == 255 ? 0 : a, b == 255 ? 0 : b));  // 255: not finite
    }
    top = row_max<kLanes>(top);
    const int k = top >= 127 + 62 ? -64 : top < 127 - 38 ? 64 : 0;
    const float f = exp2_int(k);
#pragma unroll 1
    for (int j = 0; j < 8; ++j)
        w[j * kLanes] = pack_bf16x2(__uint_as_float(w[j * kLanes] << 16) * f,
                                    __uint_as_float(w[j * kLanes] & 0xFFFF0000u) * f);
    __syncwarp();
    return k;
}

// The codes of y times f.
__device__ __forceinline__ uint2 codes8(const uint64_t* y, float f) {
    float z[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) f2_split(f2_mul(y[i], f2_make(f, f)), z[2 * i], z[2 * i + 1]);
    return make_uint2(pack_e4m3x4(z[0], z[1], z[2], z[3]), pack_e4m3x4(z[4], z[5], z[6], z[7]));
}

// The table entries times `unit` of chunk c (8 elements) of a row at position pos; plane: the chunk that
// holds its planes' first elements.
__device__ __forceinline__ Turn turn_of(const AppendFp8Params& p, int pos, int c, int plane,
                                        bool lower, float unit) {
    Turn t;
    const size_t row = static_cast<size_t>(pos) * (p.rot_dim / 2);
    if (p.interleaved) {
        const float4 cv = *reinterpret_cast<const float4*>(p.rot_cos + row + 4 * c);
        const float4 sv = *reinterpret_cast<const float4*>(p.rot_sin + row + 4 * c);
        const float cc[4] = {cv.x, cv.y, cv.z, cv.w}, ss[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            t.c[i] = f2_make(unit * cc[i], unit * cc[i]);
            t.s[i] = f2_make(-unit * ss[i], unit * ss[i]);
        }
        return t;
    }
    const float sign = lower ? -unit : unit;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 cv = *reinterpret_cast<const float4*>(p.rot_cos + row + 8 * plane + 4 * i);
        const float4 sv = *reinterpret_cast<const float4*>(p.rot_sin + row + 8 * plane + 4 * i);
        t.c[2 * i] = f2_make(unit * cv.x, unit * cv.y);
        t.c[2 * i + 1] = f2_make(unit * cv.z, unit * cv.w);
        t.s[2 * i] = f2_make(sign * sv.x, sign * sv.y);
        t.s[2 * i + 1] = f2_make(sign * sv.z, sign * sv.w);
    }
    return t;
}

// A lane's elements of a staged row.
__device__ __forceinline__ void read_row(uint64_t (&x)[8], const uint8_t* row, int l, int lanes) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
        unpack_pairs(*reinterpret_cast<const uint4*>(row + 16 * (l + m * lanes)), &x[4 * m]);
}

// How the keys turn: not at all, whole heads in halves, or otherwise.
constexpr int kNoTurn = 0, kWholeTurn = 1, kAnyTurn = 2;

// x rotated; the partners are the lane's other run, or chunks `from` of the staged row.
template <int kTurn, bool kOdd>
__device__ __forceinline__ void turn_row(uint64_t (&x)[8], const uint8_t* row,
                                         const Turn (&turn)[2], const bool (&turns)[2],
                                         const int (&from)[2], bool interleaved) {
    uint64_t z[8];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        if (kTurn == kWholeTurn) {
#pragma unroll
            for (int j = 0; j < 4; ++j) z[4 * m + j] = x[4 * (1 - m) + j];
        } else {
            uint4 w = *reinterpret_cast<const uint4*>(row + 16 * from[m]);
            if (interleaved)  // the other one of each pair
                w = make_uint4(__byte_perm(w.x, 0, 0x1032), __byte_perm(w.y, 0, 0x1032),
                               __byte_perm(w.z, 0, 0x1032), __byte_perm(w.w, 0, 0x1032));
            unpack_pairs(w, &z[4 * m]);
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint64_t c = turn[j / 4].c[j % 4], s = turn[j / 4].s[j % 4];
        if (kTurn == kWholeTurn || turns[j / 4])
            x[j] = kOdd ? turn_pair_odd(c, s, x[j], z[j]) : turn_pair(c, s, x[j], z[j]);
    }
}

constexpr int kAppendRows = 2;  // rows (heads) of one token a group of lanes takes at a time
constexpr int kAppendThreads = 128;
constexpr int kAppendTokens = 16;  // tokens a block takes at most
constexpr int kAppendStages = 3;
constexpr float kFltMax = 3.402823466e38f;

struct AppendToken {
    long long row;    // of the cache [num_pages * page_size], -1: none
    long long scale;  // of k_scale / v_scale for kv head 0
    int pos;
};

__device__ __forceinline__ AppendToken append_token(const AppendFp8Params& p, int t) {
    AppendToken a{-1, 0, 0};
    if (t >= p.total_q) return a;
    const int b = find_seq(p.cu_q, p.batch, t);
    const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1], ctx = p.cache_seqlens[b];
    if (q0 < 0 || t < q0 || t >= q1) return a;  // tokens outside every sequence are left alone
    const long long pos = static_cast<long long>(ctx) + (t - q0);
    if (ctx >= 0 && pos < static_cast<long long>(p.max_pages) * p.page_size &&
        (p.rot_dim == 0 || pos < p.rot_rows)) {
        const int i = static_cast<int>(pos) / p.page_size;
        const int slot = static_cast<int>(pos) - i * p.page_size;
        const int page = p.block_table[static_cast<size_t>(b) * p.max_pages + i];
        if (page >= 0 && page < p.num_pages)
            return AppendToken{static_cast<long long>(page) * p.page_size + slot,
                               static_cast<long long>(page) * p.Hkv * p.page_size + slot,
                               static_cast<int>(pos)};
    }
    atomicOr(p.status, kStatusBounds);
    return a;
}

// Queries go to the attention kernels as f16 times a power of two a row, rotated ones as the sum
// of two f16 numbers, 22 significant bits: rounding them to bf16 (or to one f16) moved LSE by
// up to 1e-3 (1e-4) of itself where a row sees few keys.
//
// Bound by memory, and by its latency: a block takes a run of tokens, whose places (sequence,
// position, page) its first threads find once, and each group of D / 16 lanes walks its share of
// the tokens' rows, two (heads) at a time, with the loads of the next two steps under way into
// shared memory.  A lane holds elements [8 l, 8 l + 8) and [D / 2 + 8 l, ...) of a row, which are
// each other's partners when the whole head is rotated in halves.  The scale byte is monotone in
// the magnitude, so each lane forms its own and a row's is their maximum.
//
// kKind: keys, values or queries (blockIdx.y): one instruction stream each, since the selects
// that rows of several kinds in one warp cost were a third of all instructions.  kTurn: no
// rotation, the whole head in halves (a lane then has both partners and one set of table
// entries), or any other.
//
// Measured: 16384 tokens of 8 kv heads, d 128, whole head rotated, 25 us, 4.4 TB/s of rows read and
// codes written (a copy: 6.8), with start and end about 5 us of it; 64 single tokens 4.0 us, bound by
// the chain lengths, page, table entries, rows.  Kinds mixed in one warp took 36 us, and two rows
// straight into registers 40.
constexpr int kKeys = 0, kValues = 1, kQueries = 2;

template <int D, int kTurn, int kKind>
__device__ __forceinline__ void append_rows(const AppendFp8Params& p, int tokens,
                                            uint8_t (&stage)[kAppendStages][kAppendThreads * 16 / D]
                                                            [kAppendRows][D * 2],
                                            AppendToken (&place_of)[kAppendTokens]) {
    constexpr int kLanes = D / 16, kGroups = kAppendThreads / kLanes;
    constexpr bool kRotated = kTurn != kNoTurn && kKind != kValues;
    // Queries turn at half their size: their largest rotated elements would pass fp32's range.
    constexpr bool kHalved = kRotated && kKind == kQueries;
    constexpr float kUnit = kHalved ? 0.5f : 1.f;
    const int lane = threadIdx.x & 31, l = lane % kLanes, group = threadIdx.x / kLanes;
    const int t0 = blockIdx.x * tokens;
    const int H = kKind == kQueries ? p.Hq : p.Hkv;
    const __nv_bfloat16* const in = kKind == kKeys ? p.k_new : kKind == kValues ? p.v_new : p.q;
    const int blocks = (H + kAppendRows - 1) / kAppendRows, items = tokens * blocks;
    const float inv_blocks = 1.f / blocks;

    // Item: (token, first head).  The quotient is taken in fp32: (x + 1/2) / n is at least
    // 1 / (2 n) away from an integer, far beyond the error.
    struct Item {
        int tok, h0, n;  // n: rows, 0 for items past the end
    };
    const auto item_of = [&](int item) {
        Item it;
        it.tok = static_cast<int>((item + 0.5f) * inv_blocks);
        it.h0 = (item - it.tok * blocks) * kAppendRows;
        it.n = item < items && t0 + it.tok < p.total_q ? min(kAppendRows, H - it.h0) : 0;
        return it;
    };
    const auto fetch = [&](int step) {
        const Item it = item_of(group + step * kGroups);
        const __nv_bfloat16* src = in + (static_cast<size_t>(t0 + it.tok) * H + it.h0) * D + 8 * l;
#pragma unroll
        for (int i = 0; i < kAppendRows; ++i)
            if (i < it.n) {
                uint8_t* dst = stage[step % kAppendStages][group][i] + 16 * l;
                cp_async16(dst, src + i * D);
                cp_async16(dst + D, src + i * D + D / 2);
            }
        cp_async_commit();
    };
    const int h = p.rot_dim / 16;  // a chunk's partner is h chunks further on, or before
    // (a warp's groups take the same number of steps)
    const int steps = (items - threadIdx.x / 32 * (32 / kLanes) + kGroups - 1) / kGroups;
#pragma unroll
    for (int s = 0; s < kAppendStages - 1; ++s) fetch(s);
    if (threadIdx.x < tokens) place_of[threadIdx.x] = append_token(p, t0 + threadIdx.x);
    __syncthreads();

    for (int step = 0; step < steps; ++step) {
        const Item it = item_of(group + step * kGroups);
        AppendToken place{-1, 0, 0};
        if (it.n > 0) place = place_of[it.tok];
        const int n = place.row >= 0 ? it.n : 0;
        // The lane's two runs of 8 elements (chunks of the row): do they turn, where is their
        // partner, and the rotary tables' entries for them.
        bool turns[2] = {kRotated, kRotated};
        int from[2] = {l, l + kLanes};
        Turn turn[2];
        if (kRotated && kTurn == kWholeTurn && n > 0) {
            turn[0] = turn_of(p, place.pos, l, l, true, kUnit);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                turn[1].c[j] = turn[0].c[j];
                turn[1].s[j] = f2_mul(turn[0].s[j], f2_make(-1.f, -1.f));
            }
        }
        if (kRotated && kTurn == kAnyTurn) {
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int c = l + m * kLanes;
                const bool lower = c < h;
                turns[m] = 8 * c < p.rot_dim;
                if (turns[m] && !p.interleaved) from[m] = lower ? c + h : c - h;
                if (turns[m] && n > 0) turn[m] = turn_of(p, place.pos, c, lower ? c : c - h, lower, kUnit);
            }
        }
        const int most = __reduce_max_sync(0xffffffffu, n);
        cp_async_wait<kAppendStages - 2>();
        __syncwarp();
#pragma unroll 1
        for (int i = 0; i < most; ++i) {
            const bool mine = i < n;  // (other rows' stages hold anything, and ask for nothing)
            uint8_t* const row = stage[step % kAppendStages][group][i];
            uint64_t y[8];
            read_row(y, row, l, kLanes);
            if (kRotated) turn_row<kTurn, false>(y, row, turn, turns, from, p.interleaved);
            const int u = __float_as_int(lane_top(y));
            if (kKind == kQueries) {
                // the row's largest element to [2^13, 2^14) as f16 (kv8_query_shift)
                int e = u >> 23;
                if (kHalved && kTurn == kWholeTurn) e = min(e + 1, 255);
                if (kHalved && kTurn == kAnyTurn)
                    e = min(max((run_top(&y[0]) >> 23) + turns[0], (run_top(&y[4]) >> 23) + turns[1]), 255);
                const int up = kv8_query_shift(row_max<kLanes>(e));
                const float unit = __int_as_float((up + 127) << 23);
                if (!mine) continue;
                const size_t at = static_cast<size_t>(t0 + it.tok) * p.Hq + it.h0 + i;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const float f = kHalved && turns[m] ? 2.f * unit : unit;
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float f0, f1;
                        f2_split(f2_mul(y[4 * m + j], f2_make(f, f)), f0, f1);
                        hi[j] = pack_f16x2(f0, f1);
                        const float2 h = f16x2_to_float2(hi[j]);
                        lo[j] = pack_f16x2(f0 - h.x, f1 - h.y);
                    }
                    const size_t to = at * D + m * (D / 2) + 8 * l;
                    *reinterpret_cast<uint4*>(p.q_rot + to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    if (kRotated)
                        *reinterpret_cast<uint4*>(p.q_lo + to) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                if (l == 0) p.q_unit[at] = __int_as_float((127 - up) << 23);
                continue;
            }
            // Not certain: a row with an element that is not finite (0 times it is NaN); a rotated
            // one near the ends of fp32's range, or whose scale (it changes where the largest's
            // significand passes 1.75) or, below, whose codes change within the rotation's error.
            uint64_t zero = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) zero = f2_fma(y[j], 0, zero);
            float z0, z1;
            f2_split(zero, z0, z1);
            bool redo = z0 + z1 != 0.f || (kRotated && (((u - (0x600000 - 8)) & 0x7fffff) <= 16 || off_range(u)));
            uint32_t sb = row_max<kLanes>(scale_byte(u));
            const float inv = __int_as_float((254 - min(sb, 253u)) << 23);  // 2^-e
            uint2 codes[2];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                codes[m] = codes8(&y[4 * m], turns[m] ? inv * (1.f - 0x1p-21f) : inv);
                if (kRotated) {
                    const uint2 above = codes8(&y[4 * m], turns[m] ? inv * (1.f + 0x1p-21f) : inv);
                    redo = redo || codes[m].x != above.x || codes[m].y != above.y;
                }
            }
            if (__any_sync(0xffffffffu, mine && redo)) {
                const int k =
                    kRotated && __any_sync(0xffffffffu, mine && off_range(u)) ? scale_row<kLanes>(row, l) : 0;
                read_row(y, row, l, kLanes);
                if (kRotated) turn_row<kTurn, true>(y, row, turn, turns, from, p.interleaved);
                float top = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float f[2];
                    f2_split(y[j], f[0], f[1]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (fabsf(f[i]) <= kFltMax)
                            top = fmaxf(top, fabsf(f[i]));
                        else
                            f[i] = __int_as_float(0x7fffffff);  // the NaN code; infinity would saturate
                    }
                    y[j] = f2_make(f[0], f[1]);
                }
                sb = row_max<kLanes>(top == 0.f ? 1 : max(1, scale_exponent(__float_as_int(top)) - k));
                const float inv = __int_as_float(min(254 - static_cast<int>(sb) - k, 254) << 23);
#pragma unroll
                for (int m = 0; m < 2; ++m) codes[m] = codes8(&y[4 * m], inv);
            }
            if (mine) {
                uint8_t* const dst = (kKind == kValues ? p.v_cache : p.k_cache) +
                                     (place.row * p.Hkv + it.h0 + i) * D + 8 * l;
                *reinterpret_cast<uint2*>(dst) = codes[0];
                *reinterpret_cast<uint2*>(dst + D / 2) = codes[1];
                if (l == 0)
                    (kKind == kValues ? p.v_scale : p.k_scale)
                        [place.scale + static_cast<long long>(it.h0 + i) * p.page_size] =
                            static_cast<uint8_t>(sb);
            }
        }
        __syncwarp();  // the stage's rows have been read (by partners too)
        fetch(step + kAppendStages - 1);
    }
    cp_async_wait<0>();
}

template <int D, int kTurn>
__global__ void __launch_bounds__(kAppendThreads, 5)
    kvcache_append_fp8_kernel(const AppendFp8Params p, int tokens) {
    __shared__ __align__(16) uint8_t stage[kAppendStages][kAppendThreads * 16 / D][kAppendRows][D * 2];
    __shared__ AppendToken place_of[kAppendTokens];
    griddep_launch_dependents();  // an attention kernel behind this one may set up
    if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(p.cu_q, p.batch, p.total_q, p.status);
    if (blockIdx.y == kKeys)
        append_rows<D, kTurn, kKeys>(p, tokens, stage, place_of);
    else if (blockIdx.y == kValues)
        append_rows<D, kTurn, kValues>(p, tokens, stage, place_of);
    else
        append_rows<D, kTurn, kQueries>(p, tokens, stage, place_of);
    griddep_wait();  // (attn_fwd_kvcache_fp8 builds its work list beside this grid; what waits for
                     // this grid to finish then waits for the list too)
}

// ---- staging for the tensor-core prefill ----------------------------------------------------
//
// A chunk of many query rows reads each key once per 256 rows, so it pays to turn the codes into
// an MMA operand once, in f16: code 2^(e - E) with E = (the largest e of the sequence and kv head) - 7.
// The largest magnitude is then 448 2^7 = 57344, below f16's 65504, and rows whose e is up to 22
// below the largest stay exact (the smallest code 2^-9 meets f16's smallest 2^-24).  Where a row of the
// pair (of k or v; rows of the smallest scale, zeros, aside) lies further below, one large row,
// perhaps one that most queries do not see, would cost the others their bits: then the codes go in as
// they are, the scale bytes beside them, and the prefill kernel brings them together in fp32.
constexpr int kUnitSpan = 22;
// The same for pairs whose largest value has a scale below 2^-60 (a scale byte): their unit over the
// softmax denominator is no normal number.
constexpr int kUnitLeast = 127 - 60;

// The first key that a new token of a sequence sees, and the keys from there on.
__device__ __forceinline__ int2 staged_keys(const StageFp8Params& p, int b) {
    const int q0 = p.cu_q[b], Lq = p.cu_q[b + 1] - q0, ctx = p.cache_seqlens[b];
    if (Lq <= 0 || q0 < 0 || static_cast<long long>(q0) + Lq > p.total_q || ctx < 0 ||
        static_cast<long long>(ctx) + Lq > static_cast<long long>(p.max_pages) * p.page_size)
        return make_int2(0, 0);
    const int skip = p.wl >= 0 ? max(0, ctx - p.wl) : 0;
    return make_int2(skip, ctx + Lq - skip);
}

// One block per (sequence, kv head): the span of the sequence's rows and the units of k and v.
constexpr int kUnitsThreads = 512;

__global__ void __launch_bounds__(kUnitsThreads)
    kvcache_units_fp8_kernel(const StageFp8Params p) {
    constexpr int kWarps = kUnitsThreads / 32;
    __shared__ int red[2][kWarps], red_low[2][kWarps];
    __shared__ long long sum[kWarps];
    const int b = blockIdx.x / p.Hkv, kvh = blockIdx.x % p.Hkv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    griddep_launch_dependents();
    long long before = 0;
    for (int i = threadIdx.x; i < b; i += blockDim.x)
        before += (staged_keys(p, i).y + kFwdBlockN - 1) / kFwdBlockN * kFwdBlockN;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    if (lane == 0) sum[warp] = before;
    const int2 keys = staged_keys(p, b);
    // scale bytes of K and V, four columns; 255 (NaN) does not count, nor, for the smallest, 0 and 1
    uint32_t top4[2] = {0u, 0u}, low4[2] = {~0u, ~0u};
    griddep_wait();       // the append kernel's scales
    const int* bt = p.block_table + static_cast<size_t>(b) * p.max_pages;
    const int end = keys.x + keys.y;
    for (int g = keys.x / 16 + threadIdx.x; g * 16 < end; g += blockDim.x) {
        const int page = bt[g * 16 / p.page_size];
        if (page < 0 || page >= p.num_pages) continue;  // (reported where the rows are read)
        const size_t at = (static_cast<size_t>(page) * p.Hkv + kvh) * p.page_size + g * 16 % p.page_size;
        const uint4 kw = *reinterpret_cast<const uint4*>(p.k_scale + at);
        const uint4 vw = *reinterpret_cast<const uint4*>(p.v_scale + at);
        const uint32_t w[2][4] = {{kw.x, kw.y, kw.z, kw.w}, {vw.x, vw.y, vw.z, vw.w}};
        const int from = keys.x - g * 16, to = end - g * 16;  // tokens [from, to) count
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t in = ~0u;
            if (from > 4 * i) in = from >= 4 * i + 4 ? 0u : ~0u << (8 * (from - 4 * i));
            if (to < 4 * i + 4) in &= to <= 4 * i ? 0u : ~0u >> (8 * (4 * i + 4 - to));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t x = w[j][i] & in;
                top4[j] = __vmaxu4(top4[j], x & ~__vcmpeq4(x, ~0u));
                low4[j] = __vminu4(low4[j], x | __vcmpleu4(x, 0x01010101u));
            }
        }
    }
    int top[2], low[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        top4[j] = __vmaxu4(top4[j], top4[j] >> 16);
        top[j] = max(1, max(top4[j] & 0xff, (top4[j] >> 8) & 0xff));
        low4[j] = __vminu4(low4[j], low4[j] >> 16 | 0xffff0000u);
        low[j] = min(low4[j] & 0xff, (low4[j] >> 8) & 0xff);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            top[j] = max(top[j], __shfl_xor_sync(0xffffffffu, top[j], o));
            low[j] = min(low[j], __shfl_xor_sync(0xffffffffu, low[j], o));
        }
        if (lane == 0) red[j][warp] = top[j], red_low[j][warp] = low[j];
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        long long first = 0;
        int e[2] = {1, 1}, f[2] = {255, 255};
        for (int i = 0; i < kWarps; ++i) {
            first += sum[i];
            for (int j = 0; j < 2; ++j) e[j] = max(e[j], red[j][i]), f[j] = min(f[j], red_low[j][i]);
        }
        const bool far = e[0] - f[0] > kUnitSpan || e[1] - f[1] > kUnitSpan || e[1] < kUnitLeast;
        const long long padded = (keys.y + kFwdBlockN - 1) / kFwdBlockN * kFwdBlockN;
        const bool fits = first + padded <= p.rows;
        if (!fits) atomicOr(p.status, kStatusBounds);  // more keys than the caller's bound
        if (kvh == 0) p.spans[b] = fits ? make_int2(static_cast<int>(first), keys.y) : make_int2(p.rows, 0);
        if (far && keys.y > 0) *p.by_row = 1;
        p.k_unit[blockIdx.x] = far ? 0.f : e8m0_to_f32(max(1, e[0] - 7));
        p.v_unit[blockIdx.x] = far ? 0.f : e8m0_to_f32(max(1, e[1] - 7));
    }
}

// ---- reading the cache: packed bf16 rows, or the staged f16 ones ---------------------------
//
// Bound by memory: a byte in and two out per element.  A block takes a run of tokens' keys or
// values (blockIdx.y); its first threads find the tokens' places (sequence, page), then every
// thread moves 16 codes at a time, four loads in flight.  158K tokens of 8 kv heads, d 128, to bf16:
// 153 us, 6.35 TB/s read and written (keys and values by the same block: 166 us; a search per thread
// instead of per token: 182).

constexpr int kReadTokens = 128;  // tokens a block takes at most

struct ReadToken {
    long long row;    // of the cache [num_pages * page_size], -1: not written, -2: zeros
    long long scale;  // of k_scale / v_scale for kv head 0
};

// Row t of the packed output.
__device__ __forceinline__ ReadToken read_token(const int* block_table, int b, int pos, int page_size,
                                                int max_pages, int num_pages, int Hkv,
                                                unsigned* status, long long bad) {
    int page = -1;
    if (pos / page_size < max_pages)
        page = block_table[static_cast<size_t>(b) * max_pages + pos / page_size];
    if (page < 0 || page >= num_pages) {
        atomicOr(status, kStatusBounds);
        return ReadToken{bad, 0};
    }
    const int slot = pos % page_size;
    return ReadToken{static_cast<long long>(page) * page_size + slot,
                     static_cast<long long>(page) * Hkv * page_size + slot};
}

__device__ __forceinline__ void check_call(const ReadFp8Params& p) {
    check_offsets(p.cu_k, p.batch, p.total_k, p.status);
}
__device__ __forceinline__ void check_call(const StageFp8Params&) {}  // (the append kernel's)

__device__ __forceinline__ ReadToken place(const ReadFp8Params& p, int t, int& b) {
    b = find_seq(p.cu_k, p.batch, t);
    const int k0 = p.cu_k[b];
    if (k0 < 0 || t < k0 || t >= p.cu_k[b + 1]) return ReadToken{-1, 0};  // outside every sequence
    return read_token(p.block_table, b, t - k0, p.page_size, p.max_pages, p.num_pages, p.Hkv,
                      p.status, -1);
}

__device__ __forceinline__ ReadToken place(const StageFp8Params& p, int t, int& b) {
    int lo = 0, hi = p.batch - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.spans[mid].x <= t) lo = mid; else hi = mid - 1;
    }
    b = lo;
    const int2 span = p.spans[b];
    const int j = t - span.x;
    if (j < 0 || j >= (span.y + kFwdBlockN - 1) / kFwdBlockN * kFwdBlockN) return ReadToken{-1, 0};
    if (j >= span.y) return ReadToken{-2, 0};  // zero rows fill the last key block
    return read_token(p.block_table, b, staged_keys(p, b).x + j, p.page_size, p.max_pages,
                      p.num_pages, p.Hkv, p.status, -2);
}

// 16 codes as bf16: code 2^e, exact but for the smallest scales' subnormals.
__device__ __forceinline__ void convert16(const ReadFp8Params&, const uint4& w, int sb, float,
                                          uint32_t (&out)[8]) {
    const float scale = e8m0_to_f32(sb);
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t h[2];
        e4m3x4_to_f16x2(in[k], h[0], h[1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float2 f = f16x2_to_float2(h[j]);
            out[2 * k + j] = pack_bf16x2(f.x * scale, f.y * scale);
        }
    }
}

// The unit of a (sequence, kv head); where it is 0, rows keep their scale bytes.
__device__ __forceinline__ float unit_of(const ReadFp8Params&, int, bool) { return 1.f; }
__device__ __forceinline__ float unit_of(const StageFp8Params& p, int bh, bool is_v) {
    return (is_v ? p.v_unit : p.k_unit)[bh];
}
__device__ __forceinline__ void keep_scale(const ReadFp8Params&, int, int, int, bool) {}
__device__ __forceinline__ void keep_scale(const StageFp8Params& p, int sb, int row, int kvh, bool is_v) {
    (is_v ? p.v_sb : p.k_sb)[static_cast<size_t>(kvh) * p.rows + row] = sb;
}

// 16 codes as f16 multiples of the (sequence, kv head)'s unit (or as they are).
__device__ __forceinline__ void convert16(const StageFp8Params&, const uint4& w, int sb, float unit,
                                          uint32_t (&out)[8]) {
    const int e = unit == 0.f ? 0 : sb - (__float_as_int(unit) >> 23);  // at most 7
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
    if (e >= -14 && sb != 255) {  // 2^e is a normal f16
        const uint32_t f = static_cast<uint32_t>(e + 15) << 10, ff = f | (f << 16);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t h[2];
            e4m3x4_to_f16x2(in[k], h[0], h[1]);
            out[2 * k] = f16x2_mul(h[0], ff);
            out[2 * k + 1] = f16x2_mul(h[1], ff);
        }
        return;
    }
    const float scale = sb == 255 ? __int_as_float(0x7fffffff) : exp2_int(e);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t h[2];
        e4m3x4_to_f16x2(in[k], h[0], h[1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float2 f = f16x2_to_float2(h[j]);
            out[2 * k + j] = pack_f16x2(f.x * scale, f.y * scale);
        }
    }
}

template <int D, typename Params>
__global__ void __launch_bounds__(256)
    kvcache_read_fp8_kernel(const Params p, uint16_t* k_out, uint16_t* v_out, int rows, int tokens) {
    constexpr int kLanes = D / 16, kUnroll = 4;
    __shared__ ReadToken place_of[kReadTokens];
    __shared__ int seq_of[kReadTokens];
    const int t0 = blockIdx.x * tokens;
    griddep_launch_dependents();  // (staging: the prefill kernel may set up)
    griddep_wait();               // (staging: the spans and units)
    if (blockIdx.x == 0 && blockIdx.y == 0) check_call(p);
    if (threadIdx.x < tokens) {
        int b = 0;
        ReadToken r{-1, 0};
        if (t0 + static_cast<int>(threadIdx.x) < rows) r = place(p, t0 + threadIdx.x, b);
        place_of[threadIdx.x] = r;
        seq_of[threadIdx.x] = b;
    }
    __syncthreads();
    const bool is_v = blockIdx.y != 0;
    const uint8_t* const cache = is_v ? p.v_cache : p.k_cache;
    const uint8_t* const scales = is_v ? p.v_scale : p.k_scale;
    uint16_t* const to = (is_v ? v_out : k_out) + static_cast<size_t>(t0) * p.Hkv * D;
    const int items = tokens * p.Hkv * kLanes;
    // (the quotient in fp32: (x + 1/2) / n is at least 1 / (2 n) away from an integer; x is
    // below 2^22)
    const float inv = 1.f / p.Hkv;
    for (int i0 = threadIdx.x; i0 < items; i0 += 256 * kUnroll) {
        uint4 w[kUnroll];
        int sb[kUnroll], at[kUnroll];  // at: token * Hkv + kv head
        long long row[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + 256 * u;
            row[u] = -1;
            if (i >= items) continue;
            at[u] = i / kLanes;
            const int tok = static_cast<int>((at[u] + 0.5f) * inv), kvh = at[u] - tok * p.Hkv;
            const ReadToken r = place_of[tok];
            row[u] = r.row;
            if (r.row < 0) continue;
            w[u] = *reinterpret_cast<const uint4*>(cache + (r.row * p.Hkv + kvh) * D + i % kLanes * 16);
            sb[u] = scales[r.scale + static_cast<long long>(kvh) * p.page_size];
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (row[u] == -1) continue;
            uint32_t out[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (row[u] >= 0) {
                const int tok = static_cast<int>((at[u] + 0.5f) * inv), kvh = at[u] - tok * p.Hkv;
                const float unit = unit_of(p, seq_of[tok] * p.Hkv + kvh, is_v);
                convert16(p, w[u], sb[u], unit, out);
                if (unit == 0.f) keep_scale(p, sb[u], t0 + tok, kvh, is_v);
            }
            uint4* dst = reinterpret_cast<uint4*>(to + static_cast<size_t>(at[u]) * D +
                                                  (i0 + 256 * u) % kLanes * 16);
            dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
            dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
        }
    }
}

// About 2048 moves of 16 codes a block (158K tokens: 152 us; 178 with half, 151 with twice as many).
int read_tokens(int Hkv, int head_dim) {
    int n = kReadTokens;
    while (n > 8 && n * Hkv * (head_dim / 16) > 2048) n /= 2;
    return n;
}

// `dependent`: may start once every CTA of the kernel before it on the stream has started; the
// kernel waits for that grid itself (griddep_wait).
template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), dim3 grid, int threads, bool dependent,
                   cudaStream_t stream, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename Params>
cudaError_t launch_read(const Params& p, void* k, void* v, int rows, int head_dim, bool dependent,
                        cudaStream_t stream) {
    const int tokens = read_tokens(p.Hkv, head_dim);
    const dim3 grid((rows + tokens - 1) / tokens, 2);
    uint16_t *ko = static_cast<uint16_t*>(k), *vo = static_cast<uint16_t*>(v);
    return launch(head_dim == 128 ? kvcache_read_fp8_kernel<128, Params> : kvcache_read_fp8_kernel<64, Params>,
                  grid, 256, dependent, stream, p, ko, vo, rows, tokens);
}

}  // namespace

cudaError_t launch_kvcache_append_fp8(const AppendFp8Params& p, int head_dim, bool dependent,
                                      cudaStream_t stream) {
    if (p.total_q == 0) return cudaSuccess;
    // Single tokens spread over the GPU, about one step a group of lanes (64 of them: 4.0 us, 6.8 with
    // 16 tokens a block); prompts take up to 16 tokens a block while four blocks an SM remain (16384
    // tokens: 25.0 us, 27.3 with 8 a block, 25.0 with 32).  Whole heads that turn in halves: 25.0 us,
    // 28.9 as any turn.
    const int blocks = (p.Hkv + kAppendRows - 1) / kAppendRows;
    const int groups = kAppendThreads / (head_dim / 16);
    int tokens = 1;
    while (tokens < kAppendTokens &&
           (2 * tokens * blocks <= groups || p.total_q / (2 * tokens) >= 4 * kGb300Sms))
        tokens *= 2;
    const dim3 grid(static_cast<unsigned>((p.total_q + tokens - 1) / tokens), p.q_rot != nullptr ? 3 : 2);
    const int turn = p.rot_dim == 0 ? kNoTurn
                     : p.rot_dim == head_dim && !p.interleaved ? kWholeTurn
                                                               : kAnyTurn;
    const auto go = [&](auto kernel) {
        return launch(kernel, grid, kAppendThreads, dependent, stream, p, tokens);
    };
    if (head_dim == 128)
        return turn == kNoTurn      ? go(kvcache_append_fp8_kernel<128, kNoTurn>)
               : turn == kWholeTurn ? go(kvcache_append_fp8_kernel<128, kWholeTurn>)
                                    : go(kvcache_append_fp8_kernel<128, kAnyTurn>);
    return turn == kNoTurn      ? go(kvcache_append_fp8_kernel<64, kNoTurn>)
           : turn == kWholeTurn ? go(kvcache_append_fp8_kernel<64, kWholeTurn>)
                                : go(kvcache_append_fp8_kernel<64, kAnyTurn>);
}

cudaError_t launch_kvcache_stage_fp8(const StageFp8Params& p, int head_dim, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(p.batch) * p.Hkv);
    const cudaError_t e = launch(kvcache_units_fp8_kernel, grid, kUnitsThreads, true, stream, p);
    return e != cudaSuccess ? e : launch_read(p, p.k, p.v, p.rows, head_dim, true, stream);
}

cudaError_t launch_kvcache_read_fp8(const ReadFp8Params& p, int head_dim, cudaStream_t stream) {
    return p.total_k == 0 ? cudaSuccess : launch_read(p, p.k, p.v, p.total_k, head_dim, false, stream);
}

}  // namespace attn

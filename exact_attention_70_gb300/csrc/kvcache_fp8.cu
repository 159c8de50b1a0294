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
// last place (kvcache.cu); only where that lies within 2 units of a border between two codes (or
// between two scales) is it not certain, about one element in 2^18.  The warp then forms the
// value again as an unevaluated sum of two fp32 numbers (Dekker's and Knuth's error-free product
// and sum), brought to one by rounding to odd, after which rounding to a shorter format gives
// what rounding the exact value would (S. Boldo, G. Melquiond, "Emulation of FMA and correctly
// rounded sums: proved algorithms using rounding to odd", 2008).
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

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
}

// a b - c d within 1.5 units in the last place (Kahan).
__device__ __forceinline__ float det2(float a, float b, float c, float d) {
    const float w = __fmul_rn(c, d);
    return __fadd_rn(__fmaf_rn(a, b, -w), __fmaf_rn(-c, d, w));
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

// The 8 rotated values of a lane; other: the partner plane's elements (rotate-half), c, s: the
// lane's table entries (4 of each when interleaved).
template <bool kOdd>
__device__ __forceinline__ void rotate8(const uint4& own, const uint4& other, const float (&c)[8],
                                        const float (&s)[8], bool interleaved, bool lower,
                                        float (&y)[8]) {
    float x[8], z[8];
    unpack8(own, x);
    unpack8(other, z);
    const auto det = [](float a, float b, float e, float f) {
        return kOdd ? det2_odd(a, b, e, f) : det2(a, b, e, f);
    };
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[2 * i] = det(x[2 * i], c[i], x[2 * i + 1], s[i]);
            y[2 * i + 1] = det(x[2 * i], s[i], -x[2 * i + 1], c[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)  // lower: x cos - z sin; upper (z the lower half): z sin + x cos
            y[i] = det(x[i], c[i], lower ? z[i] : -z[i], s[i]);
    }
}

// The largest |y| of a row (of kLanes lanes), as bits: what is not finite compares above all else.
template <int kLanes>
__device__ __forceinline__ int row_top(const float (&y)[8]) {
    int top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_int(y[i]) & 0x7fffffff);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    return top;
}

// 448 = 1.75 2^8: the exponent of the largest magnitude less 8, one more when its significand
// is above 1.75.
__device__ __forceinline__ int scale_byte(int top) {
    return max(1, (top >> 23) - 8 + ((top & 0x7fffff) > 0x600000 ? 1 : 0));
}

// Is the code of z (a value times 2^-e) uncertain when z may be off by two units in the last
// place?  Normal codes change at values whose 20 low bits are 0x80000, subnormal ones (below
// 2^-6) at odd multiples of 2^-10.
__device__ __forceinline__ bool near_border(float z) {
    const int u = __float_as_int(z) & 0x7fffffff;
    const bool normal = ((u - (0x80000 - 2)) & 0xfffff) <= 4;
    if (u >= 0x3c800000) return normal;  // 2^-6
    const float f = fabsf(z) * 1024.f;
    return fabsf(f - rintf(f)) < 0x1p-12f && f > 0.25f;
}

__device__ __forceinline__ uint2 codes8(const float (&y)[8], float inv) {
    return make_uint2(pack_e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                      pack_e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
}

constexpr int kAppendRows = 4;  // rows (heads) of one token a group of lanes takes

// Rotated queries go to the attention kernel as f16 times a power of two a row: 11 significant
// bits of the rotated value, where bf16's 8 would put up to 2^-9 of a logit's terms on it.
//
// A group of D / 8 lanes, 8 elements a lane, takes up to four rows (heads) of one token: their
// loads go out together and before the token's place is known, the rotary tables are read
// once for the four, and single tokens still spread over many groups.  Keys come first, then
// values, then queries, so that a warp's rows are of one kind.
template <int D>
__global__ void __launch_bounds__(256) kvcache_append_fp8_kernel(const AppendFp8Params p) {
    constexpr int kLanes = D / 8;
    griddep_launch_dependents();  // an attention kernel behind this one may set up
    const int lane = threadIdx.x & 31;
    const int e0 = (lane % kLanes) * 8;
    const int kv_blocks = (p.Hkv + kAppendRows - 1) / kAppendRows;
    const int q_blocks = p.q_rot != nullptr ? (p.Hq + kAppendRows - 1) / kAppendRows : 0;
    const long long kv_items = static_cast<long long>(p.total_q) * kv_blocks;
    const long long items = 2 * kv_items + static_cast<long long>(p.total_q) * q_blocks;
    const long long item = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) / kLanes;
    bool live = item < items;
    const int kind = !live ? 1 : item < kv_items ? 0 : item < 2 * kv_items ? 1 : 2;  // K, V, Q
    const long long at = live ? item - (kind == 0 ? 0 : kind == 1 ? kv_items : 2 * kv_items) : 0;
    const int blocks = kind == 2 ? q_blocks : kv_blocks, H = kind == 2 ? p.Hq : p.Hkv;
    const int t = static_cast<int>(at / blocks);
    const int h0 = static_cast<int>(at - static_cast<long long>(t) * blocks) * kAppendRows;
    const int n = min(kAppendRows, H - h0);
    const __nv_bfloat16* src = (kind == 0 ? p.k_new : kind == 1 ? p.v_new : p.q) +
                               (static_cast<size_t>(t) * H + h0) * D + e0;
    uint4 own[kAppendRows];
#pragma unroll
    for (int i = 0; i < kAppendRows; ++i)
        own[i] = live && i < n ? *reinterpret_cast<const uint4*>(src + i * D) : make_uint4(0, 0, 0, 0);

    // the token's place
    const int b = find_seq(p.cu_q, p.batch, t);
    const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1], ctx = p.cache_seqlens[b];
    live = live && t >= q0 && t < q1;  // tokens outside every sequence are left alone
    const long long pos = static_cast<long long>(ctx) + (t - q0);
    if (live && (ctx < 0 || pos >= static_cast<long long>(p.max_pages) * p.page_size ||
                 (p.rot_dim > 0 && pos >= p.rot_rows))) {
        atomicOr(p.status, kStatusBounds);
        live = false;
    }
    int page = 0, slot = 0;
    if (live && kind != 2) {
        const int i = static_cast<int>(pos) / p.page_size;
        slot = static_cast<int>(pos) - i * p.page_size;
        page = p.block_table[static_cast<size_t>(b) * p.max_pages + i];
        if (page < 0 || page >= p.num_pages) {
            atomicOr(p.status, kStatusBounds);
            live = false;
        }
    }

    const int half = p.rot_dim / 2;
    const bool lower = e0 < half;
    const bool turns = live && kind != 1 && e0 < p.rot_dim;
    float c[8], s[8];
    if (turns) {
        const size_t row = static_cast<size_t>(pos) * half;
        const int plane = p.interleaved ? e0 / 2 : lower ? e0 : e0 - half;
        const float4* cr = reinterpret_cast<const float4*>(p.rot_cos + row + plane);
        const float4* sr = reinterpret_cast<const float4*>(p.rot_sin + row + plane);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (i == 1 && p.interleaved) break;
            const float4 cv = cr[i], sv = sr[i];
            c[4 * i] = cv.x, c[4 * i + 1] = cv.y, c[4 * i + 2] = cv.z, c[4 * i + 3] = cv.w;
            s[4 * i] = sv.x, s[4 * i + 1] = sv.y, s[4 * i + 2] = sv.z, s[4 * i + 3] = sv.w;
        }
    }
    const bool any_turns = __any_sync(0xffffffffu, turns);
#pragma unroll
    for (int i = 0; i < kAppendRows; ++i) {
        if (__all_sync(0xffffffffu, i >= n)) break;
        float y[8];
        unpack8(own[i], y);
        uint4 other = make_uint4(0, 0, 0, 0);
        if (any_turns) {
            // the partner planes of rotate-half live half / 8 lanes further on, or before
            const int from = (lower ? lane + half / 8 : lane - half / 8) & 31;
            other.x = __shfl_sync(0xffffffffu, own[i].x, from);
            other.y = __shfl_sync(0xffffffffu, own[i].y, from);
            other.z = __shfl_sync(0xffffffffu, own[i].z, from);
            other.w = __shfl_sync(0xffffffffu, own[i].w, from);
            if (turns) rotate8<false>(own[i], other, c, s, p.interleaved, lower, y);
        }
        int top = row_top<kLanes>(y);
        const bool mine = live && i < n;
        if (kind == 2) {
            // the row's largest element to [2^13, 2^14) as f16 (kv8_query_shift)
            const int a = kv8_query_shift(top >> 23);
            const float up = __int_as_float((a + 127) << 23);
            if (mine) {
                const size_t row = static_cast<size_t>(t) * p.Hq + h0 + i;
                *reinterpret_cast<uint4*>(p.q_rot + row * D + e0) =
                    make_uint4(pack_f16x2(y[0] * up, y[1] * up), pack_f16x2(y[2] * up, y[3] * up),
                               pack_f16x2(y[4] * up, y[5] * up), pack_f16x2(y[6] * up, y[7] * up));
                if (e0 == 0) p.q_unit[row] = __int_as_float((127 - a) << 23);
            }
        }
        int sb = scale_byte(top);
        float inv = __int_as_float((254 - min(sb, 253)) << 23);  // 2^-e
        // What is certain of the above?  Not a row with an element that is not finite, nor, of
        // a rotated row, codes and scales near a border.
        bool redo = top >= 0x7f800000;
        if (turns && kind == 0) {
            redo = redo || static_cast<unsigned>((top & 0x7fffff) - (0x600000 - 2)) <= 4u;
#pragma unroll
            for (int j = 0; j < 8; ++j) redo = redo || near_border(y[j] * inv);
        }
        if (__any_sync(0xffffffffu, redo && kind != 2)) {
            if (turns) rotate8<true>(own[i], other, c, s, p.interleaved, lower, y);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if ((__float_as_int(y[j]) & 0x7fffffff) >= 0x7f800000) y[j] = 0.f;
            top = row_top<kLanes>(y);  // (of the finite elements)
            if (turns)
                rotate8<true>(own[i], other, c, s, p.interleaved, lower, y);
            else
                unpack8(own[i], y);
            sb = scale_byte(top);
            inv = __int_as_float((254 - sb) << 23);
#pragma unroll
            for (int j = 0; j < 8; ++j)  // the NaN code, where infinity would saturate
                if ((__float_as_int(y[j]) & 0x7fffffff) >= 0x7f800000) y[j] = __int_as_float(0x7fffffff);
        }
        if (mine && kind != 2) {
            const size_t row = (static_cast<size_t>(page) * p.page_size + slot) * p.Hkv + h0 + i;
            *reinterpret_cast<uint2*>((kind == 1 ? p.v_cache : p.k_cache) + row * D + e0) = codes8(y, inv);
            if (e0 == 0)
                (kind == 1 ? p.v_scale : p.k_scale)[
                    (static_cast<size_t>(page) * p.Hkv + h0 + i) * p.page_size + slot] =
                    static_cast<uint8_t>(sb);
        }
    }
}

// ---- staging for the tensor-core prefill ----------------------------------------------------
//
// A chunk of many query rows reads each key once per 256 rows, so it pays to turn the codes into
// an MMA operand once, in f16: code 2^(e - E) with E = (the largest e of the sequence and kv head) - 7.
// The largest magnitude is then 448 2^7 = 57344, below f16's 65504, and rows whose e is up to 22
// below the largest stay exact (the smallest code 2^-9 meets f16's smallest 2^-24).

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
    __shared__ int red[2][kWarps];
    __shared__ long long sum[kWarps];
    const int b = blockIdx.x / p.Hkv, kvh = blockIdx.x % p.Hkv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long before = 0;
    for (int i = threadIdx.x; i < b; i += blockDim.x)
        before += (staged_keys(p, i).y + kFwdBlockN - 1) / kFwdBlockN * kFwdBlockN;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    if (lane == 0) sum[warp] = before;
    const int2 keys = staged_keys(p, b);
    int top[2] = {1, 1};  // scale bytes of K and V; 255 (NaN) does not count
    const int* bt = p.block_table + static_cast<size_t>(b) * p.max_pages;
    const int end = keys.x + keys.y;
    for (int g = keys.x / 16 + threadIdx.x; g * 16 < end; g += blockDim.x) {
        const int page = bt[g * 16 / p.page_size];
        if (page < 0 || page >= p.num_pages) continue;  // (reported where the rows are read)
        const size_t at = (static_cast<size_t>(page) * p.Hkv + kvh) * p.page_size + g * 16 % p.page_size;
        const uint4 kw = *reinterpret_cast<const uint4*>(p.k_scale + at);
        const uint4 vw = *reinterpret_cast<const uint4*>(p.v_scale + at);
        const uint32_t w[2][4] = {{kw.x, kw.y, kw.z, kw.w}, {vw.x, vw.y, vw.z, vw.w}};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (g * 16 + i < keys.x || g * 16 + i >= end) continue;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int e = (w[j][i / 4] >> (8 * (i % 4))) & 0xff;
                if (e != 255) top[j] = max(top[j], e);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top[j] = max(top[j], __shfl_xor_sync(0xffffffffu, top[j], o));
        if (lane == 0) red[j][warp] = top[j];
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        long long first = 0;
        int e[2] = {1, 1};
        for (int i = 0; i < kWarps; ++i) {
            first += sum[i];
            e[0] = max(e[0], red[0][i]);
            e[1] = max(e[1], red[1][i]);
        }
        const long long padded = (keys.y + kFwdBlockN - 1) / kFwdBlockN * kFwdBlockN;
        const bool fits = first + padded <= p.rows;
        if (!fits) atomicOr(p.status, kStatusBounds);  // more keys than the caller's bound
        if (kvh == 0) p.spans[b] = fits ? make_int2(static_cast<int>(first), keys.y) : make_int2(p.rows, 0);
        p.k_unit[blockIdx.x] = e8m0_to_f32(max(1, e[0] - 7));
        p.v_unit[blockIdx.x] = e8m0_to_f32(max(1, e[1] - 7));
    }
}

// ---- reading the cache: packed bf16 rows, or the staged f16 ones ---------------------------
//
// Bound by memory: a byte in and two out per element.  A block takes a run of tokens; its first
// threads find the tokens' places (sequence, page), then every thread moves 16 codes at a time,
// four loads in flight.

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

__device__ __forceinline__ ReadToken place(const ReadFp8Params& p, int t, int& b) {
    b = find_seq(p.cu_k, p.batch, t);
    const int k0 = p.cu_k[b];
    if (t < k0 || t >= p.cu_k[b + 1]) return ReadToken{-1, 0};  // outside every sequence
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
__device__ __forceinline__ void convert16(const ReadFp8Params&, const uint4& w, int sb, int, bool,
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

// 16 codes as f16 multiples of the (sequence, kv head)'s unit.
__device__ __forceinline__ void convert16(const StageFp8Params& p, const uint4& w, int sb, int bh,
                                          bool is_v, uint32_t (&out)[8]) {
    const int e = sb - (__float_as_int((is_v ? p.v_unit : p.k_unit)[bh]) >> 23);  // at most 7
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
    if (threadIdx.x < tokens) {
        int b = 0;
        ReadToken r{-1, 0};
        if (t0 + static_cast<int>(threadIdx.x) < rows) r = place(p, t0 + threadIdx.x, b);
        place_of[threadIdx.x] = r;
        seq_of[threadIdx.x] = b;
    }
    __syncthreads();
    const int per_kind = tokens * p.Hkv * kLanes, items = 2 * per_kind;
    for (int i0 = threadIdx.x; i0 < items; i0 += 256 * kUnroll) {
        uint4 w[kUnroll];
        int sb[kUnroll], tok[kUnroll], kvh[kUnroll];
        long long row[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + 256 * u;
            row[u] = -1;
            if (i >= items) continue;
            const bool is_v = i >= per_kind;
            const int j = (is_v ? i - per_kind : i) / kLanes;
            tok[u] = j / p.Hkv;
            kvh[u] = j - tok[u] * p.Hkv;
            const ReadToken r = place_of[tok[u]];
            row[u] = r.row;
            if (r.row < 0) continue;
            w[u] = *reinterpret_cast<const uint4*>((is_v ? p.v_cache : p.k_cache) +
                                                   (r.row * p.Hkv + kvh[u]) * D + i % kLanes * 16);
            sb[u] = (is_v ? p.v_scale : p.k_scale)[r.scale + static_cast<long long>(kvh[u]) * p.page_size];
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + 256 * u;
            if (row[u] == -1) continue;
            const bool is_v = i >= per_kind;
            uint32_t out[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (row[u] >= 0) convert16(p, w[u], sb[u], seq_of[tok[u]] * p.Hkv + kvh[u], is_v, out);
            uint4* dst = reinterpret_cast<uint4*>(
                (is_v ? v_out : k_out) +
                (static_cast<size_t>(t0 + tok[u]) * p.Hkv + kvh[u]) * D + i % kLanes * 16);
            dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
            dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
        }
    }
}

// About 2048 moves of 16 codes a block.
int read_tokens(int Hkv, int head_dim) {
    int n = kReadTokens;
    while (n > 8 && n * 2 * Hkv * (head_dim / 16) > 2048) n /= 2;
    return n;
}

template <typename Params>
cudaError_t launch_read(const Params& p, void* k, void* v, int rows, int head_dim, cudaStream_t stream) {
    const int tokens = read_tokens(p.Hkv, head_dim);
    const int grid = (rows + tokens - 1) / tokens;
    uint16_t *ko = static_cast<uint16_t*>(k), *vo = static_cast<uint16_t*>(v);
    if (head_dim == 128)
        kvcache_read_fp8_kernel<128><<<grid, 256, 0, stream>>>(p, ko, vo, rows, tokens);
    else
        kvcache_read_fp8_kernel<64><<<grid, 256, 0, stream>>>(p, ko, vo, rows, tokens);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kvcache_append_fp8(const AppendFp8Params& p, int head_dim, cudaStream_t stream) {
    const long long blocks = (p.Hkv + kAppendRows - 1) / kAppendRows * 2 +
                             (p.q_rot != nullptr ? (p.Hq + kAppendRows - 1) / kAppendRows : 0);
    const long long threads = p.total_q * blocks * (head_dim / 8);
    if (threads == 0) return cudaSuccess;
    const unsigned grid = static_cast<unsigned>((threads + 255) / 256);
    if (head_dim == 128)
        kvcache_append_fp8_kernel<128><<<grid, 256, 0, stream>>>(p);
    else
        kvcache_append_fp8_kernel<64><<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_kvcache_stage_fp8(const StageFp8Params& p, int head_dim, cudaStream_t stream) {
    kvcache_units_fp8_kernel<<<static_cast<unsigned>(p.batch) * p.Hkv, kUnitsThreads, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_read(p, p.k, p.v, p.rows, head_dim, stream);
}

cudaError_t launch_kvcache_read_fp8(const ReadFp8Params& p, int head_dim, cudaStream_t stream) {
    return p.total_k == 0 ? cudaSuccess : launch_read(p, p.k, p.v, p.total_k, head_dim, stream);
}

}  // namespace attn

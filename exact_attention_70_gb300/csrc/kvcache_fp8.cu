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
// Keys are rotated first (kvcache.cu states the rotation).  The rotated value a cos - b sin
// goes to e4m3 with one rounding: it is formed as an unevaluated sum of two fp32 numbers
// (Dekker and Knuth's error-free product and sum) and brought to one fp32 number by rounding
// to odd, after which rounding to a shorter format gives what rounding the exact value would
// (S. Boldo, G. Melquiond, "Emulation of FMA and correctly rounded sums: proved algorithms
// using rounding to odd", 2008).
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

// Rotated queries go to the attention kernel as f16 times a power of two a row: 11 significant
// bits of the rotated value, where bf16's 8 would put up to 2^-9 of a logit's terms on it.
//
// One row of D elements per group of D / 8 lanes, 8 elements a lane.  Every lane of a warp
// runs the same trips, so the shuffles inside a group are always complete.
template <int D>
__global__ void __launch_bounds__(256) kvcache_append_fp8_kernel(const AppendFp8Params p) {
    constexpr int kLanes = D / 8;
    griddep_launch_dependents();  // an attention kernel behind this one may set up
    const int lane = threadIdx.x & 31;
    const int e0 = (lane % kLanes) * 8;
    const int rows_per_tok = 2 * p.Hkv + (p.q_rot != nullptr ? p.Hq : 0);
    const long long total = static_cast<long long>(p.total_q) * rows_per_tok;
    const long long stride = static_cast<long long>(gridDim.x) * (blockDim.x / kLanes);
    const long long first = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) / kLanes;
    const int half = p.rot_dim / 2;
    for (long long base = first - first % (32 / kLanes); base < total; base += stride) {
        const long long row = base + lane / kLanes;
        bool live = row < total;
        const int t = live ? static_cast<int>(row / rows_per_tok) : 0;
        const int r = live ? static_cast<int>(row % rows_per_tok) : 0;
        const int b = find_seq(p.cu_q, p.batch, t);
        const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1];
        live = live && t >= q0 && t < q1;  // tokens outside every sequence are left alone
        const int ctx = p.cache_seqlens[b];
        const long long pos = static_cast<long long>(ctx) + (t - q0);
        if (live && (ctx < 0 || pos >= static_cast<long long>(p.max_pages) * p.page_size ||
                     (p.rot_dim > 0 && pos >= p.rot_rows))) {
            atomicOr(p.status, kStatusBounds);
            live = false;
        }
        const bool is_q = r >= 2 * p.Hkv, is_v = !is_q && r >= p.Hkv;
        const int kvh = is_v ? r - p.Hkv : r;
        int page = 0;
        if (live && !is_q) {
            page = p.block_table[static_cast<size_t>(b) * p.max_pages + pos / p.page_size];
            if (page < 0 || page >= p.num_pages) {
                atomicOr(p.status, kStatusBounds);
                live = false;
            }
        }
        const __nv_bfloat16* src =
            is_q ? p.q + (static_cast<size_t>(t) * p.Hq + (r - 2 * p.Hkv)) * D
                 : (is_v ? p.v_new : p.k_new) + (static_cast<size_t>(t) * p.Hkv + kvh) * D;
        const uint4 own = live ? *reinterpret_cast<const uint4*>(src + e0) : make_uint4(0, 0, 0, 0);
        float y[8];
        unpack8(own, y);
        if (p.rot_dim > 0) {
            // the partner planes of rotate-half live half / 8 lanes further on, or before
            const bool lower = e0 < half;
            const int from = lower ? lane + half / 8 : lane - half / 8;
            uint4 other;
            other.x = __shfl_sync(0xffffffffu, own.x, from & 31);
            other.y = __shfl_sync(0xffffffffu, own.y, from & 31);
            other.z = __shfl_sync(0xffffffffu, own.z, from & 31);
            other.w = __shfl_sync(0xffffffffu, own.w, from & 31);
            if (live && !is_v && e0 < p.rot_dim) {
                const size_t at = static_cast<size_t>(pos) * half;
                float x[8];
                unpack8(own, x);
                if (p.interleaved) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float c = p.rot_cos[at + e0 / 2 + i], s = p.rot_sin[at + e0 / 2 + i];
                        y[2 * i] = det2_odd(x[2 * i], c, x[2 * i + 1], s);
                        y[2 * i + 1] = det2_odd(x[2 * i], s, -x[2 * i + 1], c);
                    }
                } else {
                    float z[8];
                    unpack8(other, z);
                    const int plane = lower ? e0 : e0 - half;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float c = p.rot_cos[at + plane + i], s = p.rot_sin[at + plane + i];
                        y[i] = lower ? det2_odd(x[i], c, z[i], s) : det2_odd(z[i], s, -x[i], c);
                    }
                }
            }
        }
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (!(fabsf(y[i]) <= 3.402823466e38f)) y[i] = __int_as_float(0x7fffffff);
            amax = fmaxf(amax, fabsf(y[i]));  // NaN operands are ignored
        }
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const int u = __float_as_int(amax);
        if (is_q) {
            // the row's largest element to [2^13, 2^14) as f16 (kv8_query_shift)
            const int a = kv8_query_shift(u >> 23);
            const float up = __int_as_float((a + 127) << 23);
            if (live) {
                const size_t at = static_cast<size_t>(t) * p.Hq + (r - 2 * p.Hkv);
                *reinterpret_cast<uint4*>(p.q_rot + at * D + e0) =
                    make_uint4(pack_f16x2(y[0] * up, y[1] * up), pack_f16x2(y[2] * up, y[3] * up),
                               pack_f16x2(y[4] * up, y[5] * up), pack_f16x2(y[6] * up, y[7] * up));
                if (e0 == 0) p.q_unit[at] = __int_as_float((127 - a) << 23);
            }
        }
        // 448 = 1.75 2^8: the exponent of amax less 8, one more when its significand is above 1.75
        const int sb = max(1, (u >> 23) - 8 + ((u & 0x7fffff) > 0x600000 ? 1 : 0));
        const float inv = __int_as_float((254 - sb) << 23);  // 2^-e
        if (live && !is_q) {
            const size_t slot = static_cast<size_t>(pos % p.page_size);
            uint8_t* dst = (is_v ? p.v_cache : p.k_cache) +
                           ((static_cast<size_t>(page) * p.page_size + slot) * p.Hkv + kvh) * D + e0;
            *reinterpret_cast<uint2*>(dst) =
                make_uint2(pack_e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                           pack_e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
            if (e0 == 0)
                (is_v ? p.v_scale : p.k_scale)[(static_cast<size_t>(page) * p.Hkv + kvh) * p.page_size +
                                               slot] = static_cast<uint8_t>(sb);
        }
    }
}

// 16 codes a thread: code 2^e, exact in bf16 for all but the smallest scales' subnormals.
template <int D>
__global__ void __launch_bounds__(256) kvcache_read_fp8_kernel(const ReadFp8Params p) {
    constexpr int kLanes = D / 16;
    const long long total = static_cast<long long>(p.total_k) * 2 * p.Hkv * kLanes;
    for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<long long>(gridDim.x) * blockDim.x) {
        const int e0 = static_cast<int>(i % kLanes) * 16;
        const long long row = i / kLanes;
        const int r = static_cast<int>(row % (2 * p.Hkv));
        const int t = static_cast<int>(row / (2 * p.Hkv));
        const int b = find_seq(p.cu_k, p.batch, t);
        const int k0 = p.cu_k[b];
        if (t < k0 || t >= p.cu_k[b + 1]) continue;  // rows outside every sequence are left alone
        const int pos = t - k0;
        int page = -1;
        if (pos / p.page_size < p.max_pages)
            page = p.block_table[static_cast<size_t>(b) * p.max_pages + pos / p.page_size];
        if (page < 0 || page >= p.num_pages) {
            atomicOr(p.status, kStatusBounds);
            continue;
        }
        const bool is_v = r >= p.Hkv;
        const int kvh = is_v ? r - p.Hkv : r;
        const size_t slot = static_cast<size_t>(pos % p.page_size);
        const uint4 w = *reinterpret_cast<const uint4*>(
            (is_v ? p.v_cache : p.k_cache) +
            ((static_cast<size_t>(page) * p.page_size + slot) * p.Hkv + kvh) * D + e0);
        const float scale = e8m0_to_f32((is_v ? p.v_scale : p.k_scale)[
            (static_cast<size_t>(page) * p.Hkv + kvh) * p.page_size + slot]);
        const uint32_t in[4] = {w.x, w.y, w.z, w.w};
        uint32_t out[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float2 f = f16x2_to_float2(e4m3x2_to_f16x2(in[k / 2] >> (16 * (k & 1))));
            out[k] = pack_bf16x2(f.x * scale, f.y * scale);
        }
        uint4* dst = reinterpret_cast<uint4*>((is_v ? p.v : p.k) +
                                              (static_cast<size_t>(t) * p.Hkv + kvh) * D + e0);
        dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
        dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
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

// 16 codes a thread, k and v row by row.
template <int D>
__global__ void __launch_bounds__(256) kvcache_stage_fp8_kernel(const StageFp8Params p) {
    constexpr int kLanes = D / 16;
    const long long total = static_cast<long long>(p.rows) * 2 * p.Hkv * kLanes;
    for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<long long>(gridDim.x) * blockDim.x) {
        const int e0 = static_cast<int>(i % kLanes) * 16;
        const long long row = i / kLanes;
        const int r = static_cast<int>(row % (2 * p.Hkv));
        const int t = static_cast<int>(row / (2 * p.Hkv));
        int lo = 0, hi = p.batch - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.spans[mid].x <= t) lo = mid; else hi = mid - 1;
        }
        const int b = lo;
        const int2 span = p.spans[b];
        const int j = t - span.x;
        if (j < 0 || j >= (span.y + kFwdBlockN - 1) / kFwdBlockN * kFwdBlockN) continue;
        const bool is_v = r >= p.Hkv;
        const int kvh = is_v ? r - p.Hkv : r;
        uint32_t out[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (j < span.y) {
            const int pos = staged_keys(p, b).x + j;
            const int page = p.block_table[static_cast<size_t>(b) * p.max_pages + pos / p.page_size];
            if (page < 0 || page >= p.num_pages) {
                atomicOr(p.status, kStatusBounds);  // zeros
            } else {
                const size_t slot = static_cast<size_t>(pos % p.page_size);
                const uint4 w = *reinterpret_cast<const uint4*>(
                    (is_v ? p.v_cache : p.k_cache) +
                    ((static_cast<size_t>(page) * p.page_size + slot) * p.Hkv + kvh) * D + e0);
                const int sb = (is_v ? p.v_scale : p.k_scale)[
                    (static_cast<size_t>(page) * p.Hkv + kvh) * p.page_size + slot];
                const int eb = __float_as_int((is_v ? p.v_unit : p.k_unit)[b * p.Hkv + kvh]) >> 23;
                const float scale = sb == 255 ? __int_as_float(0x7fffffff) : exp2_int(sb - eb);
                const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 f = f16x2_to_float2(e4m3x2_to_f16x2(in[k / 2] >> (16 * (k & 1))));
                    out[k] = pack_f16x2(f.x * scale, f.y * scale);
                }
            }
        }
        uint4* dst = reinterpret_cast<uint4*>((is_v ? p.v : p.k) +
                                              (static_cast<size_t>(t) * p.Hkv + kvh) * D + e0);
        dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
        dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
    }
}

unsigned grid_for(long long threads, int num_sms) {
    const long long blocks = (threads + 255) / 256, cap = static_cast<long long>(num_sms) * 8;
    return static_cast<unsigned>(blocks < cap ? blocks : cap);
}

}  // namespace

cudaError_t launch_kvcache_append_fp8(const AppendFp8Params& p, int head_dim, int num_sms,
                                      cudaStream_t stream) {
    const long long rows =
        static_cast<long long>(p.total_q) * (2 * p.Hkv + (p.q_rot != nullptr ? p.Hq : 0));
    if (rows == 0) return cudaSuccess;
    const unsigned grid = grid_for(rows * (head_dim / 8), num_sms);
    if (head_dim == 128)
        kvcache_append_fp8_kernel<128><<<grid, 256, 0, stream>>>(p);
    else
        kvcache_append_fp8_kernel<64><<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_kvcache_stage_fp8(const StageFp8Params& p, int head_dim, int num_sms,
                                     cudaStream_t stream) {
    kvcache_units_fp8_kernel<<<static_cast<unsigned>(p.batch) * p.Hkv, kUnitsThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const unsigned grid =
        grid_for(static_cast<long long>(p.rows) * 2 * p.Hkv * (head_dim / 16), num_sms);
    if (head_dim == 128)
        kvcache_stage_fp8_kernel<128><<<grid, 256, 0, stream>>>(p);
    else
        kvcache_stage_fp8_kernel<64><<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_kvcache_read_fp8(const ReadFp8Params& p, int head_dim, int num_sms,
                                    cudaStream_t stream) {
    const long long threads = static_cast<long long>(p.total_k) * 2 * p.Hkv * (head_dim / 16);
    if (threads == 0) return cudaSuccess;
    const unsigned grid = grid_for(threads, num_sms);
    if (head_dim == 128)
        kvcache_read_fp8_kernel<128><<<grid, 256, 0, stream>>>(p);
    else
        kvcache_read_fp8_kernel<64><<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace attn

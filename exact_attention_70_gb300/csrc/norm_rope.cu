// norm_rope.cu -- RMS norms of queries and keys per head and the rotary embedding in one pass, its
// backward pass, and the form that writes keys and values to their slots of the paged cache.
//
// A row x (one token, one head) becomes y = R z, z = x rstd w, rstd = (sum x^2 / d + eps)^-1/2, where
// R turns plane i by the angle whose cosine and sine stand in row positions[axis(i)][token] of the tables.
// Backward: dz = R^T dy, dw = sum over tokens and heads of x rstd dz, and with n = x rstd, h = w dz:
// dx = rstd (h - n sum(n h) / d).  All of it is fp32, rounded once where a tensor in bf16 is written.
//
// Bound by memory: a row is read once and written once (backward: two read, one written).  A row is
// d / 8 lanes wide.  Lane l holds elements 4 l .. 4 l + 3 and those rotary_dim / 2 further on, so
// that the partners of a plane meet in one thread and each table entry is read by one thread of a row,
// once for all of a token's heads that the thread does (interleaved planes and the elements behind
// rotary_dim: 8 l .. 8 l + 7).
#include <cuda_bf16.h>

#include "kernels.h"
#include "ptx.cuh"

namespace attn {

namespace {

constexpr int kNrThreads = 256;
// Sums of squares from kFarSum on are taken again, of x times kFarUnit (128 elements of 2^128 sum to 2^115).
constexpr float kFarSum = 0x1p120f, kFarUnit = 0x1p-70f;

// (a plain load: an output may be its input)
__device__ __forceinline__ uint2 ld_row8(const __nv_bfloat16* p) {
    return *reinterpret_cast<const uint2*>(p);
}

// The four bf16 values of an 8-byte piece.
__device__ __forceinline__ void unpack4(uint2 v, float* f) {
    f[0] = __uint_as_float(v.x << 16);
    f[1] = __uint_as_float(v.x & 0xffff0000u);
    f[2] = __uint_as_float(v.y << 16);
    f[3] = __uint_as_float(v.y & 0xffff0000u);
}

__device__ __forceinline__ uint2 pack4(const float* f) {
    return make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
}

// The sum over a row's lanes.
template <int kLanes>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// What one lane knows of a row's layout.
struct Lane {
    int o0, o1;  // offsets of its two pieces of four elements
    bool turns;  // they lie in planes 4 l .. 4 l + 3
    int plane;
};

template <int D, bool kInter>
__device__ __forceinline__ Lane lane_of(const NormRopeParams& p, int l) {
    Lane s;
    s.turns = 8 * l < p.rot_dim;
    s.plane = 4 * l;
    const bool apart = !kInter && s.turns;
    s.o0 = apart ? 4 * l : 8 * l;
    s.o1 = apart ? p.rot_dim / 2 + 4 * l : 8 * l + 4;
    return s;
}

// Cosines and sines of the lane's four planes at token t (false: a position outside the tables).
__device__ __forceinline__ bool load_turn(const NormRopeParams& p, const Lane& s, int t, float* c, float* sn) {
    if (p.rot_dim == 0) return true;
    int row[4];
    bool ok = true;
#pragma unroll
    for (int a = 0; a < kNrAxes; ++a) {
        row[a] = a < p.axes ? __ldg(p.positions + static_cast<size_t>(a) * p.total + t) : 0;
        ok = ok && row[a] >= 0 && row[a] < p.rot_rows;
    }
    if (!ok || !s.turns) return ok;
    const int half = p.rot_dim / 2;
    const unsigned axes = (p.plane_axis[s.plane >> 4] >> (2 * (s.plane & 15))) & 0xffu;
    if (axes == 0u) {  // (all planes with one axis)
        const size_t at = static_cast<size_t>(row[0]) * half + s.plane;
        const float4 cv = __ldg(reinterpret_cast<const float4*>(p.rot_cos + at));
        const float4 sv = __ldg(reinterpret_cast<const float4*>(p.rot_sin + at));
        c[0] = cv.x, c[1] = cv.y, c[2] = cv.z, c[3] = cv.w;
        sn[0] = sv.x, sn[1] = sv.y, sn[2] = sv.z, sn[3] = sv.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned a = (axes >> (2 * i)) & 3u;
            const int r = a == 0u ? row[0] : a == 1u ? row[1] : row[2];
            const size_t at = static_cast<size_t>(r) * half + s.plane + i;
            c[i] = __ldg(p.rot_cos + at);
            sn[i] = __ldg(p.rot_sin + at);
        }
    }
    return true;
}

// The eight elements (two pieces) turned by their planes' angles, or back.
template <bool kInter, bool kBack>
__device__ __forceinline__ void turn(float (&x)[8], const float* c, const float* sn) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float& a = x[kInter ? 2 * i : i];
        float& b = x[kInter ? 2 * i + 1 : i + 4];
        const float s = kBack ? -sn[i] : sn[i];
        const float ra = a * c[i] - b * s, rb = a * s + b * c[i];
        a = ra;
        b = rb;
    }
}

__device__ __forceinline__ float load_weight(const void* w, bool f32, int i) {
    return f32 ? __ldg(static_cast<const float*>(w) + i)
               : __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(w) + i));
}

// The blocks' division: kind 0 (queries), 1 (keys), 2 (values).
struct Kind {
    int kind, block, blocks, heads, par_log2;
};

__device__ __forceinline__ Kind kind_of(const NormRopeParams& p) {
    Kind k;
    k.kind = 0;
    k.block = blockIdx.x;
    while (k.block >= p.blocks[k.kind]) k.block -= p.blocks[k.kind++];
    k.blocks = p.blocks[k.kind];
    k.heads = k.kind == 0 ? p.Hq : p.Hkv;
    k.par_log2 = p.par_log2[k.kind];
    return k;
}

// A group of D / 8 << par_log2 threads does one token at a time, 1 << par_log2 of its heads side by
// side and kRows of a thread's rows in flight.
template <int D, bool kInter, bool kAppend>
__global__ void __launch_bounds__(kNrThreads) norm_rope_kernel(const NormRopeParams p) {
    constexpr int kLanes = D / 8, kRows = 4;
    const Kind k = kind_of(p);
    const int l = threadIdx.x % kLanes;
    const int group_log2 = (D == 128 ? 4 : 3) + k.par_log2;  // threads a token
    const int par = 1 << k.par_log2, head0 = (threadIdx.x / kLanes) & (par - 1);
    const int t = k.block * (kNrThreads >> group_log2) + (threadIdx.x >> group_log2);
    const Lane s = lane_of<D, kInter>(p, l);
    const bool isv = kAppend && k.kind == 2, isk = k.kind == 1;
    const void* wp = isv ? nullptr : isk ? p.k_weight : p.q_weight;
    bool live = t < p.total;
    float c[4], sn[4];
    __nv_bfloat16* dst = isk ? p.k_out : p.q_out;
    size_t row0 = static_cast<size_t>(live ? t : 0) * k.heads;
    if (live) {
        live = load_turn(p, s, t, c, sn);
        if (!live && head0 == 0 && l == 0) atomicOr(p.status, kStatusBounds);
        if (kAppend) {
            const int slot = __ldg(p.slots + t);
            const bool to_cache = isk || isv;
            if (slot >= p.cache_rows) {
                if (head0 == 0 && l == 0) atomicOr(p.status, kStatusBounds);
                if (to_cache) live = false;
            }
            if (to_cache) {
                if (slot < 0) live = false;
                row0 = static_cast<size_t>(live ? slot : 0) * k.heads;
                dst = isv ? p.v_cache : p.k_cache;
            }
        }
    }
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
    if (wp != nullptr) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = load_weight(wp, p.weight_f32, s.o0 + i);
            w[i + 4] = load_weight(wp, p.weight_f32, s.o1 + i);
        }
    }
    const __nv_bfloat16* src = isv ? p.v : isk ? p.k : p.q;
    src += static_cast<size_t>(live ? t : 0) * (isv ? p.v_stride : isk ? p.k_stride : p.q_stride);
    for (int h0 = 0; h0 < k.heads; h0 += par * kRows) {  // (the same count for a warp's threads)
        uint2 raw[kRows][2];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int h = h0 + u * par + head0;
            const bool on = live && h < k.heads;
            raw[u][0] = on ? ld_row8(src + h * D + s.o0) : make_uint2(0u, 0u);
            raw[u][1] = on ? ld_row8(src + h * D + s.o1) : make_uint2(0u, 0u);
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int h = h0 + u * par + head0;
            float x[8];
            unpack4(raw[u][0], x);
            unpack4(raw[u][1], x + 4);
            if (wp != nullptr) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
                ss = row_sum<kLanes>(ss);
                float eps = p.eps;
                const bool far = !(ss < kFarSum);
                if (__any_sync(0xffffffffu, far)) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] *= far ? kFarUnit : 1.f;
                    float s2 = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) s2 = fmaf(x[i], x[i], s2);
                    s2 = row_sum<kLanes>(s2);
                    if (far) ss = s2, eps = p.eps * kFarUnit * kFarUnit;
                }
                const float r = rsqrtf(fmaf(ss, 1.f / D, eps));
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] *= r * w[i];
            }
            if (!isv && s.turns) turn<kInter, false>(x, c, sn);
            if (live && h < k.heads) {
                __nv_bfloat16* out = dst + (row0 + h) * D;
                if (ATTN_IN_BOUNDS(row0 + h < static_cast<size_t>(kAppend && k.kind != 0 ? p.cache_rows : p.total) * k.heads,
                                   p.status)) {
                    *reinterpret_cast<uint2*>(out + s.o0) = isv ? raw[u][0] : pack4(x);
                    *reinterpret_cast<uint2*>(out + s.o1) = isv ? raw[u][1] : pack4(x + 4);
                }
            }
        }
    }
}

// Persistent blocks: each sums its share of dw in registers, then over its rows in shared memory, into
// a row of its own of part_w; norm_rope_dw_kernel adds the rows.  Fixed shares, so the sums' order too.
template <int D, bool kInter>
__global__ void __launch_bounds__(kNrThreads) norm_rope_bwd_kernel(const NormRopeParams p) {
    constexpr int kLanes = D / 8, kRows = 2;
    __shared__ float sums[kNrThreads / kLanes][D];
    griddep_launch_dependents();
    const Kind k = kind_of(p);
    const int l = threadIdx.x % kLanes;
    const int group_log2 = (D == 128 ? 4 : 3) + k.par_log2;
    const int par = 1 << k.par_log2, head0 = (threadIdx.x / kLanes) & (par - 1);
    const int groups = kNrThreads >> group_log2;
    const Lane s = lane_of<D, kInter>(p, l);
    const bool isk = k.kind == 1;
    const void* wp = isk ? p.k_weight : p.q_weight;
    const __nv_bfloat16* x_all = isk ? p.k : p.q;
    const __nv_bfloat16* g_all = isk ? p.dk_out : p.dq_out;
    __nv_bfloat16* dx_all = isk ? p.dk : p.dq;
    const int x_stride = isk ? p.k_stride : p.q_stride, dx_stride = isk ? p.dk_stride : p.dq_stride;
    float w[8], dw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f, dw[i] = 0.f;
    if (wp != nullptr) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = load_weight(wp, p.weight_f32, s.o0 + i);
            w[i + 4] = load_weight(wp, p.weight_f32, s.o1 + i);
        }
    }
    for (long long t0 = static_cast<long long>(k.block) * groups; t0 < p.total;
         t0 += static_cast<long long>(k.blocks) * groups) {
        const long long tl = t0 + (threadIdx.x >> group_log2);
        bool live = tl < p.total;
        const int t = live ? static_cast<int>(tl) : 0;
        float c[4], sn[4];
        if (live) {
            live = load_turn(p, s, t, c, sn);
            if (!live && head0 == 0 && l == 0) atomicOr(p.status, kStatusBounds);
        }
        const __nv_bfloat16* xt = x_all + static_cast<size_t>(t) * x_stride;
        const __nv_bfloat16* gt = g_all + static_cast<size_t>(t) * k.heads * D;
        __nv_bfloat16* dxt = dx_all + static_cast<size_t>(t) * dx_stride;
        for (int h0 = 0; h0 < k.heads; h0 += par * kRows) {
            uint2 rx[kRows][2], rg[kRows][2];
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const int h = h0 + u * par + head0;
                const bool on = live && h < k.heads;
                const uint2 z = make_uint2(0u, 0u);
                rg[u][0] = on ? ld_row8(gt + h * D + s.o0) : z;
                rg[u][1] = on ? ld_row8(gt + h * D + s.o1) : z;
                rx[u][0] = on && wp != nullptr ? ld_row8(xt + h * D + s.o0) : z;
                rx[u][1] = on && wp != nullptr ? ld_row8(xt + h * D + s.o1) : z;
            }
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const int h = h0 + u * par + head0;
                const bool on = live && h < k.heads;
                float g[8];
                unpack4(rg[u][0], g);
                unpack4(rg[u][1], g + 4);
                if (s.turns && on) turn<kInter, true>(g, c, sn);
                if (wp != nullptr) {
                    float x[8], ss = 0.f, xh = 0.f;
                    unpack4(rx[u][0], x);
                    unpack4(rx[u][1], x + 4);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        ss = fmaf(x[i], x[i], ss);
                        xh = fmaf(x[i], w[i] * g[i], xh);
                    }
                    ss = row_sum<kLanes>(ss);
                    xh = row_sum<kLanes>(xh);
                    float eps = p.eps, unit = 1.f;
                    const bool far = !(ss < kFarSum);
                    if (__any_sync(0xffffffffu, far)) {
                        float s2 = 0.f, xh2 = 0.f;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            x[i] *= far ? kFarUnit : 1.f;
                            s2 = fmaf(x[i], x[i], s2);
                            xh2 = fmaf(x[i], w[i] * g[i], xh2);
                        }
                        s2 = row_sum<kLanes>(s2);
                        xh2 = row_sum<kLanes>(xh2);
                        if (far) ss = s2, xh = xh2, eps = p.eps * kFarUnit * kFarUnit, unit = kFarUnit;
                    }
                    const float r = rsqrtf(fmaf(ss, 1.f / D, eps));
                    const float m = xh * r * (1.f / D);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float n = x[i] * r;
                        dw[i] = fmaf(n, g[i], dw[i]);
                        g[i] = r * (w[i] * g[i] - n * m) * unit;
                    }
                }
                if (on) {
                    *reinterpret_cast<uint2*>(dxt + h * D + s.o0) = pack4(g);
                    *reinterpret_cast<uint2*>(dxt + h * D + s.o1) = pack4(g + 4);
                }
            }
        }
    }
    if (wp == nullptr) return;
    const int r = threadIdx.x / kLanes;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        sums[r][s.o0 + i] = dw[i];
        sums[r][s.o1 + i] = dw[i + 4];
    }
    __syncthreads();
    if (threadIdx.x < D) {
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < kNrThreads / kLanes; ++i) a += sums[i][threadIdx.x];
        p.part_w[static_cast<size_t>(blockIdx.x) * D + threadIdx.x] = a;
    }
}

// dw = the sum of the blocks' rows: 32 columns of one weight a block.
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const NormRopeParams p, int d) {
    __shared__ float sums[32][33];
    griddep_wait();
    const int isk = blockIdx.x / (d / 32), col = blockIdx.x % (d / 32) * 32 + threadIdx.x % 32;
    const int r = threadIdx.x / 32, first = isk ? p.blocks[0] : 0, n = p.blocks[isk];
    float* out = isk ? p.dk_weight : p.dq_weight;
    if (out == nullptr) return;
    float a = 0.f;
    for (int i = r; i < n; i += 32) a += p.part_w[static_cast<size_t>(first + i) * d + col];
    sums[r][threadIdx.x % 32] = a;
    __syncthreads();
    a = sums[threadIdx.x % 32][r];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if (threadIdx.x % 32 == 0) out[blockIdx.x % (d / 32) * 32 + r] = a;
}

// Heads side by side (a power of two): all of a token's where there are few tokens, and fewer, so that
// a thread does up to 8 rows with the same table entries, while threads enough remain.
int par_of(long long total, int heads, int d) {
    const int most = d == 128 ? 4 : 5;
    int par = 0;
    while (par < most && (1 << par) < heads) ++par;
    while (par > 0 && (heads >> par) < 8 && ((total * (d / 8)) << (par - 1)) >= kGb300Sms * 2048ll) --par;
    return par;
}

}  // namespace

cudaError_t launch_norm_rope(NormRopeParams p, int head_dim, bool append, cudaStream_t stream) {
    int grid = 0;
    for (int k = 0; k < 3; ++k) {
        const int heads = k == 0 ? p.Hq : p.Hkv;
        p.par_log2[k] = par_of(p.total, heads, head_dim);
        const int tokens = kNrThreads / (head_dim / 8) >> p.par_log2[k];  // a block
        p.blocks[k] = k == 2 && !append ? 0 : (p.total + tokens - 1) / tokens;
        grid += p.blocks[k];
    }
    const auto go = [&](auto kernel) {
        kernel<<<grid, kNrThreads, 0, stream>>>(p);
        return cudaGetLastError();
    };
    if (head_dim == 128) {
        if (p.interleaved) return append ? go(norm_rope_kernel<128, true, true>) : go(norm_rope_kernel<128, true, false>);
        return append ? go(norm_rope_kernel<128, false, true>) : go(norm_rope_kernel<128, false, false>);
    }
    if (p.interleaved) return append ? go(norm_rope_kernel<64, true, true>) : go(norm_rope_kernel<64, true, false>);
    return append ? go(norm_rope_kernel<64, false, true>) : go(norm_rope_kernel<64, false, false>);
}

cudaError_t launch_norm_rope_bwd(NormRopeParams p, int head_dim, cudaStream_t stream) {
    // the blocks' shares of queries and keys follow their rows
    long long most[2];
    for (int k = 0; k < 2; ++k) {
        const int heads = k == 0 ? p.Hq : p.Hkv;
        p.par_log2[k] = par_of(p.total, heads, head_dim);
        const int tokens = kNrThreads / (head_dim / 8) >> p.par_log2[k];
        most[k] = (static_cast<long long>(p.total) + tokens - 1) / tokens;
    }
    const long long keys = static_cast<long long>(kNrBwdBlocks) * p.Hkv / (p.Hq + p.Hkv);
    p.blocks[1] = static_cast<int>(most[1] < keys ? most[1] : keys > 1 ? keys : 1);
    const long long queries = kNrBwdBlocks - (keys > 1 ? keys : 1);
    p.blocks[0] = static_cast<int>(most[0] < queries ? most[0] : queries);
    p.blocks[2] = 0;
    const int grid = p.blocks[0] + p.blocks[1];
    const auto go = [&](auto kernel) {
        kernel<<<grid, kNrThreads, 0, stream>>>(p);
        return cudaGetLastError();
    };
    const cudaError_t e = head_dim == 128
                              ? (p.interleaved ? go(norm_rope_bwd_kernel<128, true>) : go(norm_rope_bwd_kernel<128, false>))
                              : (p.interleaved ? go(norm_rope_bwd_kernel<64, true>) : go(norm_rope_bwd_kernel<64, false>));
    if (e != cudaSuccess || (p.dq_weight == nullptr && p.dk_weight == nullptr)) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * head_dim / 32);
    cfg.blockDim = dim3(1024);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_rope_dw_kernel, p, head_dim);
}

}  // namespace attn

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

#include <algorithm>

#include "ptx.cuh"
#include "step_kernels.h"

namespace attn {

namespace {

constexpr int kNrThreads = 256;
constexpr int kNrFwdBlocksPerSm = 4, kNrFwdRows = 4;
constexpr int kNrBwdBlocksPerSm = 2, kNrStages = 2;
// Sums of squares from kFarSum on are taken again, of x times kFarUnit (the squares of 128 elements of 2^128 sum to 2^123).
constexpr float kFarSum = 0x1p120f, kFarUnit = 0x1p-70f;

// (a plain load: an output may be its input)
__device__ __forceinline__ uint2 ld_row8(const __nv_bfloat16* p) {
    return *reinterpret_cast<const uint2*>(p);
}

// Asynchronous 16-byte copy of this thread to shared memory; zeros with on = false.
__device__ __forceinline__ void cp_async16z(void* smem_dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(smem_dst)), "l"(src), "r"(on ? 16 : 0)
                 : "memory");
}

// The four bf16 values of an 8-byte piece as two pairs of fp32 for the paired instructions, and back.
__device__ __forceinline__ void unpack_pairs(uint2 v, uint64_t* f) {
    f[0] = f2_make(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u));
    f[1] = f2_make(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
}

__device__ __forceinline__ uint2 pack_pairs(const uint64_t* f) {
    float a, b, c, d;
    f2_split(f[0], a, b);
    f2_split(f[1], c, d);
    return make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
}

__device__ __forceinline__ float f2_sum(uint64_t v) {
    float a, b;
    f2_split(v, a, b);
    return a + b;
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

// A token's positions: fetched a token ahead, since the tables' rows and all that follows wait for them.
struct Rows {
    int r[kNrAxes];
};

__device__ __forceinline__ Rows load_rows(const NormRopeParams& p, long long t) {
    Rows x;
#pragma unroll
    for (int a = 0; a < kNrAxes; ++a)
        x.r[a] = p.rot_dim > 0 && a < p.axes && t < p.total ? __ldg(p.positions + static_cast<size_t>(a) * p.total + t) : 0;
    return x;
}

// Cosines and sines of the lane's four planes.  False: a position outside the tables.
__device__ __forceinline__ bool load_turn(const NormRopeParams& p, const Lane& s, const Rows& x, float* c, float* sn) {
    if (p.rot_dim == 0) return true;
    bool ok = true;
#pragma unroll
    for (int a = 0; a < kNrAxes; ++a) ok = ok && x.r[a] >= 0 && x.r[a] < p.rot_rows;
    if (!ok || !s.turns) return ok;
    const int half = p.rot_dim / 2;
    const unsigned axes = (p.plane_axis[s.plane >> 4] >> (2 * (s.plane & 15))) & 0xffu;
    if (axes == 0u) {  // (all planes with the first axis)
        const size_t at = static_cast<size_t>(x.r[0]) * half + s.plane;
        const float4 cv = __ldg(reinterpret_cast<const float4*>(p.rot_cos + at));
        const float4 sv = __ldg(reinterpret_cast<const float4*>(p.rot_sin + at));
        c[0] = cv.x, c[1] = cv.y, c[2] = cv.z, c[3] = cv.w;
        sn[0] = sv.x, sn[1] = sv.y, sn[2] = sv.z, sn[3] = sv.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned a = (axes >> (2 * i)) & 3u;
            const int r = a == 0u ? x.r[0] : a == 1u ? x.r[1] : x.r[2];
            const size_t at = static_cast<size_t>(r) * half + s.plane + i;
            c[i] = __ldg(p.rot_cos + at);
            sn[i] = __ldg(p.rot_sin + at);
        }
    }
    return true;
}

// The lane's elements, in pairs, turned by their planes' angles, or back.
template <bool kInter, bool kBack>
__device__ __forceinline__ void turn(uint64_t (&x)[4], const float* c, const float* sn) {
    if (kInter) {  // a pair is a plane
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            f2_split(x[i], a, b);
            const float s = kBack ? -sn[i] : sn[i];
            x[i] = f2_make(a * c[i] - b * s, a * s + b * c[i]);
        }
    } else {  // pairs i and i + 2 are two planes
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint64_t c2 = f2_make(c[2 * i], c[2 * i + 1]), s2 = f2_make(sn[2 * i], sn[2 * i + 1]);
            const uint64_t n2 = f2_make(-sn[2 * i], -sn[2 * i + 1]);
            const uint64_t a = f2_fma(x[i], c2, f2_mul(x[i + 2], kBack ? s2 : n2));
            const uint64_t b = f2_fma(x[i], kBack ? n2 : s2, f2_mul(x[i + 2], c2));
            x[i] = a;
            x[i + 2] = b;
        }
    }
}

// The lane's eight weights (ones without a norm).
__device__ __forceinline__ void load_weights(const void* w, bool f32, const Lane& s, uint64_t (&out)[4]) {
    if (w == nullptr) {
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = f2_make(1.f, 1.f);
    } else if (f32) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w) + (i ? s.o1 : s.o0)));
            out[2 * i] = f2_make(x.x, x.y), out[2 * i + 1] = f2_make(x.z, x.w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            unpack_pairs(__ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(w) + (i ? s.o1 : s.o0))),
                         out + 2 * i);
    }
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

// Forward: no block has more than one token a group, so that many small blocks hide one another's latency
// (persistent blocks that ask for a step's rows a step ahead, as the backward's do, took 72.9 us for the 16384
// tokens where these take 56.3).  The rows' loads go out before those of the positions, on which the tables wait.
template <int D, bool kInter, bool kAppend>
__global__ void __launch_bounds__(kNrThreads, kNrFwdBlocksPerSm) norm_rope_kernel(const NormRopeParams p) {
    constexpr int kLanes = D / 8, kRows = kNrFwdRows;
    const Kind k = kind_of(p);
    const int l = threadIdx.x % kLanes;
    const int group_log2 = (D == 128 ? 4 : 3) + k.par_log2;  // threads a token
    const int par = 1 << k.par_log2, head0 = (threadIdx.x / kLanes) & (par - 1);
    const int t = k.block * (kNrThreads >> group_log2) + (threadIdx.x >> group_log2);
    const Lane s = lane_of<D, kInter>(p, l);
    const bool isv = kAppend && k.kind == 2, isk = k.kind == 1, to_cache = kAppend && k.kind != 0;
    const bool here = t < p.total, first = head0 == 0 && l == 0;
    const __nv_bfloat16* src = isv ? p.v : isk ? p.k : p.q;
    src += static_cast<size_t>(here ? t : 0) * (isv ? p.v_stride : isk ? p.k_stride : p.q_stride);
    uint2 raw[kRows][2];
    const auto fetch = [&](int h0) {
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int h = h0 + u * par;
            const bool on = here && h < k.heads;
            raw[u][0] = on ? ld_row8(src + h * D + s.o0) : make_uint2(0u, 0u);
            raw[u][1] = on ? ld_row8(src + h * D + s.o1) : make_uint2(0u, 0u);
        }
    };
    fetch(head0);
    const Rows rows = load_rows(p, t);
    const int slot = kAppend && here ? __ldg(p.slots + t) : 0;
    const void* wp = isv ? nullptr : isk ? p.k_weight : p.q_weight;
    uint64_t w[4];
    load_weights(wp, p.weight_f32, s, w);
    float c[4], sn[4];
    bool live = here;
    if (here) {
        live = load_turn(p, s, rows, c, sn);
        if (!live && first) atomicOr(p.status, kStatusBounds);
    }
    __nv_bfloat16* dst = !to_cache ? (isk ? p.k_out : p.q_out) : isv ? p.v_cache : p.k_cache;
    size_t row0 = static_cast<size_t>(here ? t : 0) * k.heads;
    if (kAppend) {
        if (slot >= p.cache_rows && first) atomicOr(p.status, kStatusBounds);
        if (to_cache) {
            live = live && slot >= 0 && slot < p.cache_rows;
            row0 = static_cast<size_t>(live ? slot : 0) * k.heads;
        }
    }
    dst += row0 * D;
    for (int h0 = head0;;) {  // (the same count for all threads of the block)
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int h = h0 + u * par;
            uint64_t x[4];  // in pairs
            unpack_pairs(raw[u][0], x);
            unpack_pairs(raw[u][1], x + 2);
            if (wp != nullptr) {
                uint64_t s2 = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) s2 = f2_fma(x[i], x[i], s2);
                float ss = row_sum<kLanes>(f2_sum(s2)), eps = p.eps;
                const bool far = !(ss < kFarSum);
                if (__any_sync(0xffffffffu, far)) {
                    const uint64_t f2 = far ? f2_make(kFarUnit, kFarUnit) : f2_make(1.f, 1.f);
                    s2 = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[i] = f2_mul(x[i], f2);
                        s2 = f2_fma(x[i], x[i], s2);
                    }
                    const float t2 = row_sum<kLanes>(f2_sum(s2));
                    if (far) ss = t2, eps = p.eps * kFarUnit * kFarUnit;
                }
                const float r = rsqrtf(fmaf(ss, 1.f / D, eps));
                const uint64_t r2 = f2_make(r, r);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = f2_mul(f2_mul(x[i], r2), w[i]);  // (r w may be past fp32's range)
            }
            if (!isv && s.turns) turn<kInter, false>(x, c, sn);
            if (live && h < k.heads &&
                ATTN_IN_BOUNDS(row0 + h < static_cast<size_t>(to_cache ? p.cache_rows : p.total) * k.heads, p.status)) {
                *reinterpret_cast<uint2*>(dst + h * D + s.o0) = isv ? raw[u][0] : pack_pairs(x);
                *reinterpret_cast<uint2*>(dst + h * D + s.o1) = isv ? raw[u][1] : pack_pairs(x + 2);
            }
        }
        h0 += par * kRows;
        if (h0 - head0 >= k.heads) break;
        fetch(h0);
    }
}

// The walk of a group of D / 8 << par_log2 threads over its tokens: 1 << par_log2 heads side by side, kRows of
// a thread's rows at a time (a step).
struct Walk {
    long long t, stride;  // this group's token; from one token to its next
    long long t0;         // the block's first group's: the same for all threads of the block
    int h;                // the step's first head

    __device__ __forceinline__ bool on(const NormRopeParams& p) const { return t0 < p.total; }
    __device__ __forceinline__ bool step(int heads, int by) {  // true: another token
        h += by;
        if (h < heads) return false;
        h = 0;
        t += stride;
        t0 += stride;
        return true;
    }
};

// Backward: persistent blocks.  Each sums its share of dw in registers, then over its rows in shared memory, into
// a row of its own of part_w; norm_rope_dw_kernel adds the rows.  Fixed shares, so the sums' order too.
// What a step reads comes through shared memory, kNrStages - 1 steps ahead, in 16-byte copies of the row's lanes.
// 16384 tokens of 32:8 heads, d 128: 95 us with the sums behind it, 5.4 TB/s (80% of a copy's rate).  Rows through
// registers a step ahead took 102.7, without looking ahead 112 to 141, copies of 8 bytes 115.  It is
// not the bytes in flight that bound it now: three blocks an SM or three stages took 96 to 105, a block's own
// run of tokens 104, blocks of one token a group 101 to 121.
template <int D, bool kInter>
__global__ void __launch_bounds__(kNrThreads, kNrBwdBlocksPerSm) norm_rope_bwd_kernel(const NormRopeParams p) {
    constexpr int kLanes = D / 8, kRows = 2, kSlots = kNrThreads / kLanes;
    __shared__ __align__(16) __nv_bfloat16 ring[kNrStages][kRows][2][kSlots][D];
    static_assert(sizeof(ring) >= kSlots * D * sizeof(float), "the sums fit in the ring");
    griddep_launch_dependents();
    const Kind k = kind_of(p);
    const int l = threadIdx.x % kLanes;
    const int group_log2 = (D == 128 ? 4 : 3) + k.par_log2;
    const int par = 1 << k.par_log2, head0 = (threadIdx.x / kLanes) & (par - 1), by = par * kRows;
    const int groups = kNrThreads >> group_log2;
    const Lane s = lane_of<D, kInter>(p, l);
    const bool isk = k.kind == 1, first = head0 == 0 && l == 0;
    const void* wp = isk ? p.k_weight : p.q_weight;
    const __nv_bfloat16* x_all = isk ? p.k : p.q;
    const __nv_bfloat16* g_all = isk ? p.dk_out : p.dq_out;
    __nv_bfloat16* dx_all = isk ? p.dk : p.dq;
    const int x_stride = isk ? p.k_stride : p.q_stride, dx_stride = isk ? p.dk_stride : p.dq_stride;
    Walk w;
    w.t0 = static_cast<long long>(k.block) * groups;
    w.t = w.t0 + (threadIdx.x >> group_log2);
    w.stride = static_cast<long long>(k.blocks) * groups;
    w.h = head0;
    const int slot = threadIdx.x / kLanes;
    const auto fetch = [&](const Walk& y, int stage) {
        if (y.on(p)) {
            const bool here = y.t < p.total;
            const size_t t = here ? static_cast<size_t>(y.t) : 0;
            const __nv_bfloat16* xr = x_all + t * x_stride + 8 * l;
            const __nv_bfloat16* gr = g_all + t * k.heads * D + 8 * l;
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const int h = y.h + u * par;
                const bool on = here && h < k.heads;  // (zeros elsewhere)
                const size_t at = on ? static_cast<size_t>(h) * D : 0;
                cp_async16z(&ring[stage][u][0][slot][8 * l], gr + at, on);
                if (wp != nullptr) cp_async16z(&ring[stage][u][1][slot][8 * l], xr + at, on);
            }
        }
        cp_async_commit();
    };
    float c[4], sn[4];
    const auto enter = [&](long long t, const Rows& x) {
        if (t >= p.total) return false;
        const bool live = load_turn(p, s, x, c, sn);
        if (!live && first) atomicOr(p.status, kStatusBounds);
        return live;
    };
    const auto forth = [&](Walk& y) {
        const bool other = y.step(k.heads + head0, by);
        if (other) y.h = head0;
        return other;
    };
    Walk ahead = w;
#pragma unroll
    for (int i = 0; i < kNrStages - 1; ++i) {
        fetch(ahead, i);
        forth(ahead);
    }
    Rows rows = load_rows(p, w.t);
    uint64_t wt[4], dw[4];  // pairs of the lane's elements
    load_weights(wp, p.weight_f32, s, wt);
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[i] = 0;
    bool live = enter(w.t, rows);
    rows = load_rows(p, w.t + w.stride);
    int stage = 0;
    while (w.on(p)) {  // (the same number of steps for all threads of the block)
        cp_async_wait<kNrStages - 2>();
        __syncwarp();  // the row's lanes have copied it, and read the step's before
        fetch(ahead, stage == 0 ? kNrStages - 1 : stage - 1);
        forth(ahead);
        __nv_bfloat16* dxt = dx_all + static_cast<size_t>(w.t < p.total ? w.t : 0) * dx_stride;
        const bool all = __all_sync(0xffffffffu, live || w.t >= p.total);
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int h = w.h + u * par;
            const bool on = live && h < k.heads;
            uint64_t g[4];
            unpack_pairs(*reinterpret_cast<const uint2*>(&ring[stage][u][0][slot][s.o0]), g);
            unpack_pairs(*reinterpret_cast<const uint2*>(&ring[stage][u][0][slot][s.o1]), g + 2);
            if (!all && !live) g[0] = g[1] = g[2] = g[3] = 0;  // (a token outside the tables gives nothing)
            if (s.turns && on) turn<kInter, true>(g, c, sn);
            if (wp != nullptr) {
                uint64_t x[4], hg[4], s2 = 0, d2 = 0;
                unpack_pairs(*reinterpret_cast<const uint2*>(&ring[stage][u][1][slot][s.o0]), x);
                unpack_pairs(*reinterpret_cast<const uint2*>(&ring[stage][u][1][slot][s.o1]), x + 2);
                if (!all && !live) x[0] = x[1] = x[2] = x[3] = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    hg[i] = f2_mul(wt[i], g[i]);
                    s2 = f2_fma(x[i], x[i], s2);
                    d2 = f2_fma(x[i], hg[i], d2);
                }
                float ss = row_sum<kLanes>(f2_sum(s2)), xh = row_sum<kLanes>(f2_sum(d2));
                float eps = p.eps, unit = 1.f;
                const bool far = !(ss < kFarSum);
                if (__any_sync(0xffffffffu, far)) {
                    const uint64_t f2 = far ? f2_make(kFarUnit, kFarUnit) : f2_make(1.f, 1.f);
                    s2 = d2 = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[i] = f2_mul(x[i], f2);
                        s2 = f2_fma(x[i], x[i], s2);
                        d2 = f2_fma(x[i], hg[i], d2);
                    }
                    const float t2 = row_sum<kLanes>(f2_sum(s2)), e2 = row_sum<kLanes>(f2_sum(d2));
                    if (far) ss = t2, xh = e2, eps = p.eps * kFarUnit * kFarUnit, unit = kFarUnit;
                }
                const float r = rsqrtf(fmaf(ss, 1.f / D, eps)), m = -xh * r * (1.f / D), ru = r * unit;
                const uint64_t r2 = f2_make(r, r), m2 = f2_make(m, m), u2 = f2_make(ru, ru);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t n = f2_mul(x[i], r2);
                    dw[i] = f2_fma(n, g[i], dw[i]);
                    g[i] = f2_mul(u2, f2_fma(n, m2, hg[i]));
                }
            }
            if (on) {
                *reinterpret_cast<uint2*>(dxt + static_cast<size_t>(h) * D + s.o0) = pack_pairs(g);
                *reinterpret_cast<uint2*>(dxt + static_cast<size_t>(h) * D + s.o1) = pack_pairs(g + 2);
            }
        }
        stage = stage == kNrStages - 1 ? 0 : stage + 1;
        if (forth(w) && w.on(p)) {
            live = enter(w.t, rows);
            rows = load_rows(p, w.t + w.stride);
        }
    }
    cp_async_wait<0>();
    __syncthreads();
    float(*const sums)[D] = reinterpret_cast<float(*)[D]>(&ring[0][0][0][0][0]);
    if (wp == nullptr) return;
    const int r = threadIdx.x / kLanes;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        *reinterpret_cast<uint64_t*>(&sums[r][s.o0 + 2 * i]) = dw[i];
        *reinterpret_cast<uint64_t*>(&sums[r][s.o1 + 2 * i]) = dw[i + 2];
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
// a thread does up to `most_rows` rows with the same table entries, while threads enough remain.
int par_of(long long total, int heads, int d, int most_rows) {
    const int most = d == 128 ? 4 : 5;
    int par = 0;
    while (par < most && (1 << par) < heads) ++par;
    while (par > 0 && (heads >> par) < most_rows && ((total * (d / 8)) << (par - 1)) >= kGb300Sms * 2048ll) --par;
    return par;
}

// Blocks of the kinds of rows: as many as there are tokens for, or a share of `most` that follows the rows.
int divide(NormRopeParams& p, int kinds, int head_dim, long long most, int most_rows) {
    const long long rows = p.Hq + static_cast<long long>(kinds - 1) * p.Hkv;
    int grid = 0;
    for (int k = 0; k < 3; ++k) {
        const int heads = k == 0 ? p.Hq : p.Hkv;
        p.par_log2[k] = par_of(p.total, heads, head_dim, most_rows);
        const int tokens = kNrThreads / (head_dim / 8) >> p.par_log2[k];  // a block
        const long long need = (static_cast<long long>(p.total) + tokens - 1) / tokens;
        const long long share = std::max(1ll, most * heads / rows);
        p.blocks[k] = k < kinds ? static_cast<int>(std::min(need, share)) : 0;
        grid += p.blocks[k];
    }
    return grid;
}

}  // namespace

cudaError_t launch_norm_rope(NormRopeParams p, int head_dim, bool append, cudaStream_t stream) {
    const int grid = divide(p, append ? 3 : 2, head_dim, 1ll << 31, 16);
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
    const int grid = divide(p, 2, head_dim, kNrBwdBlocks, 8);
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

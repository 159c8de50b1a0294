// attn_kv8_kernel.cu -- attention of few query rows over the 8-bit paged KV cache: split-KV
// partials and their LSE-weighted combine.
//
// The method is decode_kernel.cu's ("Attention kernels: FlashAttention and PagedAttention",
// sections 五.2-五.3, 六.1 and 六.3; "04 · FA4 (CuTeDSL) and engineering interfaces",
// sections 5, 6.1 and 6.2): the keys of a sequence are split into contiguous ranges; each CTA
// gathers one range's K and V through block_table for 16 packed query rows (tokens x the query
// heads of one kv head) and runs the online softmax over it; a second kernel merges the splits.
//
// The arithmetic.  K and V are e4m3 codes times 2^e, one e per (token, kv head).  Codes are exact
// in f16, so both products run on f16 tensor-core MMAs with fp32 sums and the scales
// stay outside of them:
//   * S_ij = 2^ek_j c_i sum_d (2^a_i q_id) k_jd with c_i = scale log2(e) 2^-a_i, where a_i brings
//     row i's largest |q| just below 2^14: the 8 significant bits of bf16 fit f16's 11, and
//     elements down to 2^-28 of the row's largest stay exact (below that the error is less than
//     2^-39 of the largest);
//   * O_i = 2^(E - 15) sum_j (P_ij 2^(15 + ev_j - E)) v_j with E the largest ev_j seen so far:
//     P <= 1, so the f16 factor is at most 2^15, and it loses precision only below 2^-29 of a
//     row's largest term.  When E grows, O is rescaled together with the running maximum.
#include <cuda_bf16.h>

#include "kernels.h"
#include "ptx.cuh"
#include "tile_math.h"

namespace attn {

namespace {

constexpr float kLn2f = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;

template <int D>
struct Kv8Cfg {
    static constexpr int kTileBytes = kKv8Chunk * D;       // K (or V) codes of one chunk
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kStages = D == 128 ? 6 : 12;
    static constexpr int kOffScale = kStages * kStageBytes;  // [stage][K, V][64] scale bytes
    static constexpr int kOffBar = kOffScale + kStages * 2 * kKv8Chunk;
    static constexpr int kMergeStride = D + 4;               // floats a row of the merge buffer
    static constexpr int kMergeBytes = 4 * kKv8Rows * kMergeStride * 4 + 2 * 4 * kKv8Rows * 4;
    static_assert(kMergeBytes <= kOffScale, "merge buffer must fit in the stage ring");
    static constexpr int kSmem = kOffBar + 256 + 1024;
};

struct Kv8Bars {
    uint64_t full[12], empty[12];
    int abort_flag;
};
static_assert(sizeof(Kv8Bars) <= 256, "barrier block");

// Byte offset of the 16-byte unit u of row r in a tile of D-byte rows as TMA swizzles it: the
// unit's index xor the row inside the 8 x 128-byte (D = 128) or 4 x 128-byte (D = 64) pattern.
template <int D>
__device__ __forceinline__ uint32_t kv8_unit(int r, int u) {
    return static_cast<uint32_t>(D == 128 ? r * 128 + ((u ^ (r & 7)) << 4)
                                          : r * 64 + ((u ^ ((r >> 1) & 3)) << 4));
}

template <int D>
__global__ void __launch_bounds__(kKv8Threads, 2)
    kv8_split_kernel(const __grid_constant__ Kv8Params p) {
    using C = Kv8Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    Kv8Bars* bars = reinterpret_cast<Kv8Bars*>(smem + C::kOffBar);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = p.num_splits;
    const int split = blockIdx.x % S, hg = blockIdx.x / S;
    const int kvh = blockIdx.y, b = blockIdx.z;

    // The sequence: its query rows and keys.  A decode call has one query per sequence, at the
    // last of cache_seqlens keys; a chunk's queries follow cache_seqlens cached keys.
    int q0 = b, Lq = 1;
    if (p.cu_q != nullptr) {
        q0 = p.cu_q[b];
        Lq = p.cu_q[b + 1] - q0;
    }
    const int kmax_keys = p.max_pages * p.page_size;
    long long keys = p.seqlens[b];
    bool bad = keys < 0 || q0 < 0 || Lq < 0 || Lq > p.max_seqlen_q ||
               static_cast<long long>(q0) + Lq > p.total_q;
    if (p.cu_q != nullptr) keys += Lq;
    bad = bad || keys > kmax_keys;
    if (bad) {  // the same decision in every thread: nothing of this sequence is computed
        if (threadIdx.x == 0) atomicOr(p.status, kStatusBounds);
        return;
    }
    const int L = static_cast<int>(keys);
    const int row0 = hg * kKv8Rows;                    // first packed row: token r / g, head r % g
    const int rows = min(kKv8Rows, Lq * p.g - row0);   // valid packed rows
    if (rows <= 0) return;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&bars->full[i], 1);
            mbar_init(&bars->empty[i], 4);
        }
        bars->abort_flag = 0;
        mbar_fence_init();
    }
    __syncthreads();
    const Watchdog wd{&bars->abort_flag, p.status};

    const int imin = row0 / p.g, imax = (row0 + rows - 1) / p.g;
    const KvRange range = kv_block_range(imin, imax, Lq, L, kKv8Chunk, p.causal, p.wl, p.wr);
    const int per = (range.hi - range.lo + S - 1) / S;
    const int c0 = min(range.lo + split * per, range.hi), c1 = min(c0 + per, range.hi);

    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
    int e_run = 1;  // E as a scale byte
    float o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;

    if (warp == 4) {
        // ---- producer: lane i gathers piece i of each chunk through block_table ----
        if (lane == 0) {
            tma_prefetch_desc(&p.tm_k);
            tma_prefetch_desc(&p.tm_v);
        }
        const int* bt = p.block_table + static_cast<size_t>(b) * p.max_pages;
        const int pieces = kKv8Chunk / p.box_rows;
        uint32_t issued = 0;
        bool ok = true;
        for (int c = c0; c < c1; ++c, ++issued) {
            const uint32_t st = issued % C::kStages;
            // Pieces wholly past the sequence end (whose table entries are never read) and pieces
            // of a bad page are aimed past the end of the cache: TMA fills them with zeros.
            int page = p.num_pages, slot = 0;
            bool real = false;
            if (lane < pieces) {
                const int key = c * kKv8Chunk + lane * p.box_rows;
                if (key < L) {
                    page = bt[key / p.page_size];
                    slot = key % p.page_size;
                    real = page >= 0 && page < p.num_pages;
                    if (!real) {
                        atomicOr(p.status, kStatusBounds);
                        page = p.num_pages;
                        slot = 0;
                    }
                }
            }
            if (issued >= C::kStages)
                ok = wd.wait(&bars->empty[st], ((issued / C::kStages) - 1) & 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            uint8_t* kdst = smem + st * C::kStageBytes;
            uint8_t* sdst = smem + C::kOffScale + st * 2 * kKv8Chunk;
            if (lane < pieces && !real) {  // no scales to copy: zero bytes (2^-127)
                for (int i = 0; i < p.box_rows; i += 16) {
                    *reinterpret_cast<uint4*>(sdst + lane * p.box_rows + i) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4*>(sdst + kKv8Chunk + lane * p.box_rows + i) =
                        make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
            }
            const int n_real = __popc(__ballot_sync(0xffffffffu, real));
            if (lane == 0)
                mbar_arrive_expect_tx(&bars->full[st], C::kStageBytes + 2 * p.box_rows * n_real);
            __syncwarp();
            if (lane < pieces) {
                const int row = page * p.page_size + slot;
                tma_load_3d(kdst + lane * p.box_rows * D, &p.tm_k, &bars->full[st], 0, kvh, row);
                tma_load_3d(kdst + C::kTileBytes + lane * p.box_rows * D, &p.tm_v, &bars->full[st],
                            0, kvh, row);
                if (real) {
                    const size_t at = (static_cast<size_t>(page) * p.Hkv + kvh) * p.page_size + slot;
                    bulk_load(sdst + lane * p.box_rows, p.k_scale + at, p.box_rows, &bars->full[st]);
                    bulk_load(sdst + kKv8Chunk + lane * p.box_rows, p.v_scale + at, p.box_rows,
                              &bars->full[st]);
                }
            }
        }
        __syncwarp();
        // every load still in flight lands before the ring is reused for the merge; one that
        // never does raises the timeout status and the abort flag
        if (lane == 0) {
            const uint32_t n_st = issued < C::kStages ? issued : C::kStages;
            for (uint32_t st = 0; st < n_st; ++st) {
                const uint32_t last = st + C::kStages * ((issued - 1 - st) / C::kStages);
                const unsigned long long t0 = global_ns();
                bool landed = true;
                while (!mbar_try(&bars->full[st], (last / C::kStages) & 1)) {
                    if (global_ns() - t0 > kWaitLimitNs) {
                        landed = false;
                        break;
                    }
                }
                if (!landed) {
                    wd.fail();
                    break;
                }
            }
        }
        __syncwarp();
    } else {
        // ---- consumers: warp w owns keys [16 w, 16 w + 16) of every chunk ----
        const int gq = lane >> 2, tq = lane & 3;
        // Q as the A operand.  An f16 k-step covers 16 elements of d; the thread's four k slots
        // {2 tq, 2 tq + 1, 2 tq + 8, 2 tq + 9} stand for elements 4 tq .. 4 tq + 3 of them, the
        // four bytes ldmatrix hands it of a key's 16.
        uint32_t qa[D / 16][4];
        float c_row[2];
        int kmin[2], kmax[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = gq + 8 * h;
            const int tok = (row0 + min(r, rows - 1)) / p.g, hd = (row0 + min(r, rows - 1)) % p.g;
            const size_t row = static_cast<size_t>(q0 + tok) * p.Hq + kvh * p.g + hd;
            row_key_interval(tok, Lq, L, p.causal, p.wl, p.wr, kmin[h], kmax[h]);
            if (p.q_rot != nullptr) {  // rotated and scaled by the append kernel
                const uint2* src = reinterpret_cast<const uint2*>(p.q_rot + row * D + 4 * tq);
                c_row[h] = p.scale_log2 * p.q_unit[row];
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint2 w = r < rows ? src[4 * s] : make_uint2(0u, 0u);
                    qa[s][h] = w.x;
                    qa[s][h + 2] = w.y;
                }
                continue;
            }
            const uint2* src = reinterpret_cast<const uint2*>(p.q + row * D + 4 * tq);
            uint2 w[D / 16];
            int top = 0;
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
                w[s] = r < rows ? src[4 * s] : make_uint2(0u, 0u);
                top = max(max(top, static_cast<int>(w[s].x & 0x7fff)),
                          static_cast<int>((w[s].x >> 16) & 0x7fff));
                top = max(max(top, static_cast<int>(w[s].y & 0x7fff)),
                          static_cast<int>((w[s].y >> 16) & 0x7fff));
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int a = kv8_query_shift(top >> 7);
            const float up = __int_as_float((a + 127) << 23);
            c_row[h] = p.scale_log2 * __int_as_float((127 - a) << 23);
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
                qa[s][h] = pack_f16x2(__uint_as_float(w[s].x << 16) * up,
                                      __uint_as_float(w[s].x & 0xffff0000u) * up);
                qa[s][h + 2] = pack_f16x2(__uint_as_float(w[s].y << 16) * up,
                                          __uint_as_float(w[s].y & 0xffff0000u) * up);
            }
        }
        // keys every row of the CTA sees: [full_lo, full_hi]
        int full_lo, full_hi;
        {
            int lo, hi;
            row_key_interval(imin, Lq, L, p.causal, p.wl, p.wr, lo, full_hi);
            row_key_interval(imax, Lq, L, p.causal, p.wl, p.wr, full_lo, hi);
        }
        const int mi = lane >> 3, ri = lane & 7;  // ldmatrix: matrix id, row within matrix
        for (int c = c0; c < c1; ++c) {
            const uint32_t n = c - c0, st = n % C::kStages;
            if (!__all_sync(0xffffffffu, wd.wait(&bars->full[st], (n / C::kStages) & 1))) break;
            const uint8_t* kst = smem + st * C::kStageBytes;
            const uint8_t* sst = smem + C::kOffScale + st * 2 * kKv8Chunk + warp * 16;
            const int key0 = c * kKv8Chunk + warp * 16;
            const int nvalid = min(16, L - key0);
            if (nvalid > 0) {
                // S (16 rows x 16 keys) = Q K^T on the codes
                float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
                const uint32_t kbase = smem_u32(kst);
                const int key = warp * 16 + (mi & 1) * 8 + ri;
#pragma unroll
                for (int u = 0; u < D / 16; u += 2) {
                    uint32_t r0, r1, r2, r3;
                    ldmatrix_x4(kbase + kv8_unit<D>(key, u + (mi >> 1)), r0, r1, r2, r3);
                    mma_f16_16816(s[0], qa[u], e4m3x2_to_f16x2(r0), e4m3x2_to_f16x2(r0 >> 16));
                    mma_f16_16816(s[1], qa[u], e4m3x2_to_f16x2(r1), e4m3x2_to_f16x2(r1 >> 16));
                    mma_f16_16816(s[0], qa[u + 1], e4m3x2_to_f16x2(r2), e4m3x2_to_f16x2(r2 >> 16));
                    mma_f16_16816(s[1], qa[u + 1], e4m3x2_to_f16x2(r3), e4m3x2_to_f16x2(r3 >> 16));
                }
                // the thread's keys are 8 nt + 2 tq + {0, 1}: their scale bytes, and for V
                // the largest of the tile's valid keys
                int kb[4], vb[4], e_tile = 1;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int col = (i >> 1) * 8 + 2 * tq + (i & 1);
                    kb[i] = sst[col];
                    vb[i] = col < nvalid ? sst[kKv8Chunk + col] : 0;
                    e_tile = max(e_tile, vb[i]);
                }
                e_tile = max(e_tile, __shfl_xor_sync(0xffffffffu, e_tile, 1));
                e_tile = max(e_tile, __shfl_xor_sync(0xffffffffu, e_tile, 2));
                const int e_new = max(e_run, e_tile);
                const float e_drop = exp2_int(e_run - e_new);
                e_run = e_new;
                const bool masked = key0 < full_lo || key0 + 15 > full_hi;
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = key0 + nt * 8 + 2 * tq + (e & 1);
                        float x = s[nt][e] * c_row[e >> 1] * e8m0_to_f32(kb[2 * nt + (e & 1)]);
                        if (masked && (j < kmin[e >> 1] || j > kmax[e >> 1])) x = -INFINITY;
                        s[nt][e] = x;
                    }
                float alpha[2], m_use[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float mx = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]),
                                     fmaxf(s[1][2 * r], s[1][2 * r + 1]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    const float m_new = fmaxf(m_run[r], mx);
                    m_use[r] = m_new == -INFINITY ? 0.f : m_new;  // no key seen yet
                    alpha[r] = ex2_approx(m_run[r] - m_use[r]);
                    m_run[r] = m_new;
                }
                uint32_t pa[4];
                float rs[2] = {0.f, 0.f};
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const float f0 = exp2_int(15 + vb[2 * nt] - e_run);
                    const float f1 = exp2_int(15 + vb[2 * nt + 1] - e_run);
                    const float p0 = ex2_approx(s[nt][0] - m_use[0]);
                    const float p1 = ex2_approx(s[nt][1] - m_use[0]);
                    const float p2 = ex2_approx(s[nt][2] - m_use[1]);
                    const float p3 = ex2_approx(s[nt][3] - m_use[1]);
                    rs[0] += p0 + p1;
                    rs[1] += p2 + p3;
                    pa[2 * nt + 0] = pack_f16x2(p0 * f0, p1 * f1);
                    pa[2 * nt + 1] = pack_f16x2(p2 * f0, p3 * f1);
                }
                l_run[0] = l_run[0] * alpha[0] + rs[0];
                l_run[1] = l_run[1] * alpha[1] + rs[1];
                alpha[0] *= e_drop;
                alpha[1] *= e_drop;
#pragma unroll
                for (int x = 0; x < D / 8; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[x][e] *= alpha[e >> 1];
                // O += P V.  A transposed 8 x 8 matrix of byte pairs gives the thread elements
                // 2 gq, 2 gq + 1 of keys 2 tq, 2 tq + 1: the pair of even elements is one n-tile's
                // operand, the odd pair the next one's.  The selector puts them in that order and
                // takes zeros for keys past the end, whose slots may hold anything.
                const uint32_t sel0 = (2 * tq < nvalid ? 0x0100u : 0x0404u) |
                                      (2 * tq + 1 < nvalid ? 0x3020u : 0x4040u);
                const uint32_t sel1 = (2 * tq + 8 < nvalid ? 0x0100u : 0x0404u) |
                                      (2 * tq + 9 < nvalid ? 0x3020u : 0x4040u);
                const uint32_t vbase = kbase + C::kTileBytes;
#pragma unroll
                for (int u = 0; u < D / 16; u += 2) {
                    uint32_t r0, r1, r2, r3;
                    ldmatrix_x4_trans(vbase + kv8_unit<D>(key, u + (mi >> 1)), r0, r1, r2, r3);
                    r0 = __byte_perm(r0, 0u, sel0);
                    r1 = __byte_perm(r1, 0u, sel1);
                    r2 = __byte_perm(r2, 0u, sel0);
                    r3 = __byte_perm(r3, 0u, sel1);
                    mma_f16_16816(o[2 * u], pa, e4m3x2_to_f16x2(r0), e4m3x2_to_f16x2(r1));
                    mma_f16_16816(o[2 * u + 1], pa, e4m3x2_to_f16x2(r0 >> 16), e4m3x2_to_f16x2(r1 >> 16));
                    mma_f16_16816(o[2 * u + 2], pa, e4m3x2_to_f16x2(r2), e4m3x2_to_f16x2(r3));
                    mma_f16_16816(o[2 * u + 3], pa, e4m3x2_to_f16x2(r2 >> 16), e4m3x2_to_f16x2(r3 >> 16));
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->empty[st]);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l_run[r] += __shfl_xor_sync(0xffffffffu, l_run[r], 1);
            l_run[r] += __shfl_xor_sync(0xffffffffu, l_run[r], 2);
        }
    }
    __syncthreads();  // the ring is idle from here on: reuse it for the cross-warp merge
    if (wd.aborted()) return;  // a wait ran out: the status word says so, nothing is stored

    float* mo = reinterpret_cast<float*>(smem);             // [4 warps][16 rows][kMergeStride]
    float* mm = mo + 4 * kKv8Rows * C::kMergeStride;        // [4][16] running max
    float* ml = mm + 4 * kKv8Rows;                          // [4][16] denominators
    if (warp < 4) {
        const int gq = lane >> 2, tq = lane & 3;
        float* w = mo + warp * kKv8Rows * C::kMergeStride;
        const float unit = e8m0_to_f32(e_run) * 0x1p-15f;
#pragma unroll
        for (int u = 0; u < D / 16; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<float4*>(w + (gq + 8 * h) * C::kMergeStride + 16 * u + 4 * tq) =
                    make_float4(o[2 * u][2 * h] * unit, o[2 * u + 1][2 * h] * unit,
                                o[2 * u][2 * h + 1] * unit, o[2 * u + 1][2 * h + 1] * unit);
        if (tq == 0) {
            mm[warp * kKv8Rows + gq] = m_run[0];
            mm[warp * kKv8Rows + gq + 8] = m_run[1];
            ml[warp * kKv8Rows + gq] = l_run[0];
            ml[warp * kKv8Rows + gq + 8] = l_run[1];
        }
    }
    __syncthreads();
    if (threadIdx.x < 128) {
        for (int e = threadIdx.x; e < rows * D; e += 128) {
            const int r = e / D, d = e % D;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < 4; ++w) M = fmaxf(M, mm[w * kKv8Rows + r]);
            if (M == -INFINITY) M = 0.f;  // no key seen, or only NaN scores: l tells which
            float lsum = 0.f, acc = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float sc = ex2_approx(mm[w * kKv8Rows + r] - M);
                lsum += ml[w * kKv8Rows + r] * sc;
                acc += mo[(w * kKv8Rows + r) * C::kMergeStride + d] * sc;
            }
            const float out = lsum == 0.f ? 0.f : acc / lsum;
            const float lse = lsum == 0.f ? -INFINITY : (M + __log2f(lsum)) * kLn2f;
            const int tok = q0 + (row0 + r) / p.g, head = kvh * p.g + (row0 + r) % p.g;
            const size_t at = static_cast<size_t>(tok) * p.Hq + head;
            if (!ATTN_IN_BOUNDS(head < p.Hq && tok < p.total_q, p.status)) continue;
            if (S == 1) {
                p.out[at * D + d] = __float2bfloat16_rn(out);
                if (d == 0) p.lse[static_cast<size_t>(head) * p.lse_head + static_cast<size_t>(tok) * p.lse_tok] = lse;
            } else {
                p.part_o[(at * S + split) * D + d] = out;
                if (d == 0) p.part_lse[at * S + split] = lse;
            }
        }
    }
}

// One warp per (token, head): LSE = log sum_s exp(LSE_s), O = sum_s exp(LSE_s - LSE) O_s (an
// empty split has LSE_s = -inf and weight 0).
template <int D>
__global__ void __launch_bounds__(128) kv8_combine_kernel(const Kv8CombineParams p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = blockIdx.x * 4 + warp;
    if (row >= p.total_q * p.Hq) return;
    const int tok = row / p.Hq, head = row % p.Hq;
    // tokens outside every sequence have no partials and no output
    if (p.cu_q != nullptr && (tok < p.cu_q[0] || tok >= p.cu_q[p.batch])) return;
    const int S = p.num_splits;
    const float* pl = p.part_lse + static_cast<size_t>(row) * S;
    float M = -INFINITY;
    bool nan = false;
    for (int s = lane; s < S; s += 32) {
        M = fmaxf(M, pl[s]);
        nan = nan || pl[s] != pl[s];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (__any_sync(0xffffffffu, nan)) M = __int_as_float(0x7fffffff);
    constexpr int E = D / 32;  // elements per lane
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    float lse = -INFINITY;
    if (M != -INFINITY) {
        float sum = 0.f;
        for (int s = lane; s < S; s += 32) sum += ex2_approx((pl[s] - M) * kLog2e);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        lse = M + __logf(sum);
        const float* po = p.part_o + static_cast<size_t>(row) * S * D + lane * E;
        for (int s = 0; s < S; ++s) {
            const float w = ex2_approx((pl[s] - lse) * kLog2e);
            const float* src = po + static_cast<size_t>(s) * D;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += w * src[e];
        }
    }
    __nv_bfloat16* dst = p.out + static_cast<size_t>(row) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(acc[e], acc[e + 1]);
    if (lane == 0) p.lse[static_cast<size_t>(head) * p.lse_head + static_cast<size_t>(tok) * p.lse_tok] = lse;
}

}  // namespace

cudaError_t configure_kv8_kernels() {
    const cudaFuncAttribute smem = cudaFuncAttributeMaxDynamicSharedMemorySize;
    cudaError_t e = cudaFuncSetAttribute(kv8_split_kernel<128>, smem, Kv8Cfg<128>::kSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kv8_split_kernel<64>, smem, Kv8Cfg<64>::kSmem);
    return e;
}

cudaError_t launch_kv8_attn(const Kv8Params& p, int head_dim, cudaStream_t stream) {
    const long long groups =
        (static_cast<long long>(p.max_seqlen_q) * p.g + kKv8Rows - 1) / kKv8Rows;
    const dim3 grid(static_cast<unsigned>(groups * p.num_splits), p.Hkv, p.batch);
    if (head_dim == 128)
        kv8_split_kernel<128><<<grid, kKv8Threads, Kv8Cfg<128>::kSmem, stream>>>(p);
    else
        kv8_split_kernel<64><<<grid, kKv8Threads, Kv8Cfg<64>::kSmem, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_kv8_combine(const Kv8CombineParams& p, int head_dim, cudaStream_t stream) {
    const unsigned grid = (static_cast<unsigned>(p.total_q) * p.Hq + 3) / 4;
    if (head_dim == 128)
        kv8_combine_kernel<128><<<grid, 128, 0, stream>>>(p);
    else
        kv8_combine_kernel<64><<<grid, 128, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace attn

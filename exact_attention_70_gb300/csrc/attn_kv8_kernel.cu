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
//   * S_ij = 2^ek_j c_i sum_d (2^a_i q_id) k_jd (2^ek_j c_i first where the sum times 2^ek_j would pass
//     fp32's range) with c_i = scale log2(e) 2^-a_i, where a_i brings
//     row i's largest |q| just below 2^14: the 8 significant bits of bf16 fit f16's 11, and
//     elements down to 2^-28 of the row's largest stay exact (below that the error is less than
//     2^-39 of the largest).  A rotated query has no 8 significant bits: it comes as the sum of
//     two f16 numbers, hi + lo, and both parts are multiplied (rounding it to one moved LSE by up to
//     1e-4 of itself where a row sees few keys);
//   * O_i = 2^(E - 5) sum_j (P_ij 2^(5 + ev_j - E)) v_j with P = exp2(x - m), where the references m
//     and E of a row only move when a logit passes m by more than 8 (log2) or an ev_j passes E by
//     more than 2.  E follows the row's largest P 2^ev, and lies above it by 4 at most.  The f16 factor is
//     then at most 2^15 and keeps its 11 bits down to 2^-14, i.e. for P 2^ev down to 2^-15 of the row's
//     largest (2^-19 where the V scales are alike); below that it is off by less than 2^-26.
//     When a reference moves, O is rescaled.
#include <cuda_bf16.h>

#include "kernels.h"
#include "ptx.cuh"
#include "tile_math.h"

namespace attn {

namespace {

constexpr float kLn2f = 0.69314718055994530942f;
constexpr float kMaxScale = 0x1p127f;  // the largest scale; byte 255 reads as infinity before it is NaN
// Scores of the scaled queries with the codes are below 2^30 (2^14 times 448, d times), so they may meet
// key scales up to here before the query's own scale.
constexpr float kFarScale = 0x1p90f;
constexpr int kMinE = 8;  // E as a scale byte; its floor keeps 2^(5 - E) a normal number

template <int D>
struct Kv8Cfg {
    static constexpr int kTileBytes = kKv8Chunk * D;       // K (or V) codes of one chunk
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kOffScale = kStages * kStageBytes;  // [stage][K, V][kKv8Chunk] scale bytes
    static constexpr int kOffMerge = kOffScale + kStages * 2 * kKv8Chunk;
    static constexpr int kMergeStride = D + 16;              // floats a row: [16][kMergeStride] of O,
    static constexpr int kMergeBytes = kKv8Rows * kMergeStride * 4 + 2 * 2 * 4 * kKv8Rows * 4;  // m, l
    // the unit's queries as MMA fragments [high, low][k-step][lane][4], where the merge is later
    static constexpr int kOffQ = kOffMerge;
    static constexpr int kQBytes = D / 16 * 32 * 16;
    static_assert(4 * kKv8Rows * kMergeStride * 4 <= kOffScale, "a buffer a warp fits in the stages");
    static_assert(2 * kQBytes <= kKv8Rows * kMergeStride * 4, "queries fit in the merge buffer's O");
    static constexpr int kOffBar = kOffMerge + kMergeBytes;
    static constexpr int kSmem = kOffBar + 256 + 1024;
    static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs per SM");
};

struct Kv8Bars {
    uint64_t full[6], empty[6];
    int abort_flag;
    int fail[2];       // a consumer warp gave up in a segment of this parity
    // the CTA's share of the work: places [start, start + count) of the list, the first of them
    // number first_off of sequence first_seq's; share: what every CTA but the last ones takes
    int first_seq, first_off, start, count, share;
    int warp_sum[kKv8Threads / 32];
    float unit[kKv8Rows];  // what one unit of the unit's scaled queries stands for
};
static_assert(sizeof(Kv8Bars) <= 256, "barrier block");

// One sequence as the kernel cuts it for a kv head: ng units of 16 packed query rows, each walking
// the same nc chunks from chunk lo on (what any of the sequence's rows sees; at least one, so
// that rows without keys are written too).
struct Kv8Seq {
    int q0, Lq, L, lo, nc, ng;
    bool bad;
};

__device__ __forceinline__ Kv8Seq kv8_seq(const Kv8Params& p, int b) {
    Kv8Seq s;
    s.q0 = b;  // a decode call: one query a sequence, at the last of its keys
    s.Lq = 1;
    if (p.cu_q != nullptr) {
        s.q0 = p.cu_q[b];
        s.Lq = p.cu_q[b + 1] - s.q0;
    }
    long long keys = p.seqlens[b];
    s.bad = keys < 0 || s.q0 < 0 || s.Lq < 0 || s.Lq > p.max_seqlen_q ||
            static_cast<long long>(s.q0) + s.Lq > p.total_q;
    if (p.cu_q != nullptr) keys += s.Lq;
    s.bad = s.bad || keys > static_cast<long long>(p.max_pages) * p.page_size;
    s.L = s.bad ? 0 : static_cast<int>(keys);
    if (s.bad) s.Lq = 0;  // nothing of this sequence is computed
    const KvRange r = kv_block_range(0, s.Lq - 1, s.Lq, s.L, kKv8Chunk, p.causal, p.wl, p.wr);
    s.lo = r.lo;
    s.nc = max(1, r.hi - r.lo);
    s.ng = (s.Lq * p.g + kKv8Rows - 1) / kKv8Rows;
    return s;
}

// Its places in the list: a unit's chunks and, behind them, kKv8SwitchChunks empty places for the
// time that the merge and the next unit's start take (the host has made sure that the whole list
// counts in 31 bits).
__device__ __forceinline__ int kv8_work(const Kv8Seq& s) { return s.ng * (s.nc + kKv8SwitchChunks); }

// The walk over a CTA's share: segments, each a run of chunks of one unit.
struct Kv8Walk {
    int left, off;  // places still to do; the next one's position inside sequence b
    int b;
    Kv8Seq s;
    int row0, rows, c0, c1;  // the current segment: chunks [c0, c1) of the sequence's list
    bool first, last;             // it holds its unit's first / last chunk
    int before;                   // places of the share behind which the unit starts (negative: earlier)

    __device__ __forceinline__ bool next(const Kv8Params& p, int count) {
        while (left > 0) {
            while (off >= kv8_work(s)) {
                off = 0;
                s = kv8_seq(p, ++b);
            }
            const int places = s.nc + kKv8SwitchChunks;
            const int unit = off / places, c = off - unit * places;
            const int len = min(s.nc - c, left);  // not positive: at the unit's empty places
            row0 = unit * kKv8Rows;
            rows = min(kKv8Rows, s.Lq * p.g - row0);
            c0 = s.lo + c;
            c1 = c0 + len;
            first = c == 0;
            last = c + len == s.nc;
            before = count - left - c;
            const int taken = c + len < s.nc ? len : min(places - c, left);
            off += taken;
            left -= taken;
            if (len > 0) return true;
        }
        return false;
    }
};

// Byte offset of the 16-byte unit u of row r in a tile of D-byte rows as TMA swizzles it: the
// unit's index xor the row inside the 8 x 128-byte (D = 128) or 4 x 128-byte (D = 64) pattern.
template <int D>
__device__ __forceinline__ uint32_t kv8_unit(int r, int u) {
    return static_cast<uint32_t>(D == 128 ? r * 128 + ((u ^ (r & 7)) << 4)
                                          : r * 64 + ((u ^ ((r >> 1) & 3)) << 4));
}

// Two scale bytes as floats (byte 0 is 2^-127).
__device__ __forceinline__ void scale_pair(uint32_t w, float (&f)[2]) {
    f[0] = __int_as_float(max(static_cast<int>((w & 0xffu) << 23), 0x00400000));
    f[1] = __int_as_float(max(static_cast<int>((w & 0xff00u) << 15), 0x00400000));
}

// Persistent CTAs, two an SM.  For a kv head, the chunks of all units of all sequences form one
// list, and the CTAs of that head take equal shares of it: every CTA reads the same number of
// bytes whatever the sequences' lengths, and its ring of loads runs on from one segment to the
// next.  CTA i has kv head i % Hkv and share i / Hkv, so that CTAs side by side walk the
// same tokens for all heads and the cache's rows are read whole (with the heads one after the
// other in one list, each access 128 bytes out of 1 KB, 64 sequences took 562 us where they now take
// 345 to 351, one GPU to another).
// A unit cut by a share's border leaves partial results in the CTAs' slots (slot 1 of the CTA
// that starts it, slot 0 of those that go on with it), which kv8_combine_kernel merges.
//
// Long caches: bound by memory.  64 sequences of 1K to 32K tokens, 32:8 heads, d 128: 345 to 351 us
// with the merge, 7.0 TB/s of codes and scales (a plain copy reaches 6.8).  Short ones: bound by latency, about
// 5 us to the first chunk (lengths, page table, keys, one after the other), 1.3 us a chunk, 2 us
// for a unit's merge, 2 us for the kernel behind: 37 sequences up to 3000 tokens, 14:2 heads, 16.0 us.
// kKv8SwitchChunks = 0 took 19.9 us there, 2 to 4 took 15.9; 64 sequences took 352 us with 0 and
// 348.5, 347.6, 348 with 2, 3, 4; 16 sequences of 300 tokens 14.1 us and 11.8, 10.9, 11.9.
// A share of at least kKv8MinShare = 2 chunks: one sequence of 700 tokens, 8:2 heads, d 64, took 7.6 us,
// 8.6 with 1, 9.3 with 4.
// Fetching a unit's queries during the merge before it cost more registers than it gained (64
// sequences 376 us), and so did asking for the first chunks in L2 before the append kernel ends.
template <int D, bool kLo>
__global__ void __launch_bounds__(kKv8Threads, 2)
    kv8_split_kernel(const __grid_constant__ Kv8Params p) {
    using C = Kv8Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    Kv8Bars* bars = reinterpret_cast<Kv8Bars*>(smem + C::kOffBar);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = blockIdx.x, kvh = cta % p.Hkv, at_list = cta / p.Hkv;
    griddep_launch_dependents();
    if (threadIdx.x == 128) {
        tma_prefetch_desc(&p.tm_k);
        tma_prefetch_desc(&p.tm_v);
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&bars->full[i], 1);
            mbar_init(&bars->empty[i], 4);
        }
        bars->abort_flag = bars->fail[0] = bars->fail[1] = 0;
        mbar_fence_init();
    }
    // The list's length, the share, and where this CTA's starts: thread i sums the sequences
    // [i per, (i + 1) per), the sums are scanned, and the thread in whose range the share starts
    // finds the sequence.
    {
        const int per = (p.batch + kKv8Threads - 1) / kKv8Threads;
        const int b0 = threadIdx.x * per, b1 = min(b0 + per, p.batch);
        int mine = 0;
        for (int b = b0; b < b1; ++b) {
            const Kv8Seq s = kv8_seq(p, b);
            if (s.bad && cta == 0) atomicOr(p.status, kStatusBounds);
            mine += kv8_work(s);
        }
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        if (lane == 31) bars->warp_sum[warp] = upto;
        __syncthreads();
        int total = 0, before = upto - mine;
#pragma unroll
        for (int i = 0; i < kKv8Threads / 32; ++i) {
            if (i < warp) before += bars->warp_sum[i];
            total += bars->warp_sum[i];
        }
        total = max(total - kKv8SwitchChunks, 0);  // (no unit follows the last one)
        const int share = max((total - 1) / static_cast<int>(gridDim.x / p.Hkv) + 1, kKv8MinShare);
        const int start = static_cast<int>(min(static_cast<long long>(at_list) * share,
                                               static_cast<long long>(total)));
        const int count = min(share, total - start);
        if (count > 0 && before <= start && start < before + mine) {
            int b = b0, off = start - before;
            for (int n; off >= (n = kv8_work(kv8_seq(p, b))); ++b) off -= n;
            bars->first_seq = b;
            bars->first_off = off;
        }
        if (threadIdx.x == 0) {
            bars->start = start;
            bars->count = count;
            bars->share = share;
            // what kv8_combine_kernel finds of this CTA: nothing, until a segment ends a unit
            // that an earlier CTA started
            p.meta[cta] = make_int4(-1, 0, 0, 0);
        }
    }
    __syncthreads();
    Kv8Walk w;
    const int count = bars->count;
    w.left = count;
    w.off = bars->first_off;
    w.b = bars->first_seq;
    if (w.left > 0) w.s = kv8_seq(p, w.b);
    const Watchdog wd{&bars->abort_flag, p.status};
    griddep_wait();  // what the append kernel before this one wrote
    if (w.left == 0) return;

    if (warp == 4) {
        // ---- producer: lane i gathers piece i of each chunk through block_table ----
        const int pieces = kKv8Chunk / p.box_rows;
        uint32_t issued = 0;
        bool ok = true;
        while (ok && w.next(p, count)) {
            const int* bt = p.block_table + static_cast<size_t>(w.b) * p.max_pages;
            // the first key that any of the sequence's rows sees
            const int key_lo = p.wl >= 0 ? max(0, w.s.L - w.s.Lq - p.wl) : 0;
            for (int c = w.c0; c < w.c1; ++c, ++issued) {
                const uint32_t st = issued % C::kStages;
                // Pieces wholly past the sequence end or before its first key that is seen (whose
                // table entries are never read) and pieces of a bad page are aimed past the end of
                // the cache: TMA fills them with zeros.
                int page = p.num_pages, slot = 0;
                bool real = false;
                if (lane < pieces) {
                    const int key = c * kKv8Chunk + lane * p.box_rows;
                    if (key < w.s.L && key + p.box_rows > key_lo) {
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
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                uint8_t* kdst = smem + st * C::kStageBytes;
                uint8_t* sdst = smem + C::kOffScale + st * 2 * kKv8Chunk;
                if (lane < pieces && !real) {  // no scales to copy: zero bytes
                    for (int i = 0; i < p.box_rows; i += 16) {
                        *reinterpret_cast<uint4*>(sdst + lane * p.box_rows + i) =
                            make_uint4(0, 0, 0, 0);
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
                    tma_load_3d(kdst + lane * p.box_rows * D, &p.tm_k, &bars->full[st], 0, kvh,
                                row);
                    tma_load_3d(kdst + C::kTileBytes + lane * p.box_rows * D, &p.tm_v,
                                &bars->full[st], 0, kvh, row);
                    if (real) {
                        const size_t at =
                            (static_cast<size_t>(page) * p.Hkv + kvh) * p.page_size + slot;
                        bulk_load(sdst + lane * p.box_rows, p.k_scale + at, p.box_rows,
                                  &bars->full[st]);
                        bulk_load(sdst + kKv8Chunk + lane * p.box_rows, p.v_scale + at, p.box_rows,
                                  &bars->full[st]);
                    }
                }
            }
        }
        __syncwarp();
        // every load still in flight lands before the CTA's shared memory goes; one that never
        // does raises the timeout status and the abort flag
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
        return;
    }

    // ---- consumers: warp w owns keys [32 w, 32 w + 32) of every chunk ----
    const int gq = lane >> 2, tq = lane & 3;
    const int mi = lane >> 3, ri = lane & 7;  // ldmatrix: matrix id, row within matrix
    float* const mo = reinterpret_cast<float*>(smem + C::kOffMerge);   // [16 rows][kMergeStride]
    float* const ml_all = mo + kKv8Rows * C::kMergeStride;             // [parity][m, l][4][16]
    const uint32_t qs = smem_u32(smem + C::kOffQ) + lane * 16;  // this lane's fragments
    uint32_t n = 0;  // chunks consumed
    for (int seg = 0; w.next(p, count); ++seg) {
        const int Lq = w.s.Lq, L = w.s.L, q0 = w.s.q0, rows = w.rows, row0 = w.row0;
        float m_run[2] = {-INFINITY, -INFINITY};
        uint64_t l2[2] = {0, 0};  // the rows' denominators, even and odd keys apart
        // 2^(5 - E) of a row (E as a scale byte: 259 less this one's exponent field)
        float inv[2] = {__int_as_float((259 - kMinE) << 23), __int_as_float((259 - kMinE) << 23)};
        float o[D / 8][4];
#pragma unroll
        for (int x = 0; x < D / 8; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.f;
        // Q as the A operand.  An f16 k-step covers 16 elements of d; the thread's four k slots
        // {2 tq, 2 tq + 1, 2 tq + 8, 2 tq + 9} stand for elements 4 tq .. 4 tq + 3 of them, the
        // four bytes ldmatrix hands it of a key's 16.
        // They are the same for all warps and stay in shared memory (in registers they cost spills):
        // each warp brings a quarter of the k-steps.
        float c_row[2];
        int kmin[2], kmax[2];
        size_t q_row[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = row0 + min(gq + 8 * h, rows - 1), tok = r / p.g;
            q_row[h] = static_cast<size_t>(q0 + tok) * p.Hq + kvh * p.g + r % p.g;
            row_key_interval(tok, Lq, L, p.causal, p.wl, p.wr, kmin[h], kmax[h]);
        }
        const bool there[2] = {gq < rows, gq + 8 < rows};
        const uint2 none = make_uint2(0u, 0u);
        float unit[2];
        if (kLo) {  // rotated and scaled by the append kernel
#pragma unroll
            for (int h = 0; h < 2; ++h) unit[h] = p.q_unit[q_row[h]];
            for (int s = warp; s < D / 16; s += 4) {
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    const __half* src = (part ? p.q_lo : p.q_rot) + 16 * s + 4 * tq;
                    uint2 x[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        x[h] = there[h] ? *reinterpret_cast<const uint2*>(src + q_row[h] * D) : none;
                    st_shared_v4(qs + part * C::kQBytes + s * 512, x[0].x, x[1].x, x[0].y, x[1].y);
                }
            }
        } else {
            uint32_t mine[D / 64][4];  // this warp's k-steps
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint2* src = reinterpret_cast<const uint2*>(p.q + q_row[h] * D + 4 * tq);
                uint2 x[D / 16];
                int top = 0;
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    x[s] = there[h] ? src[4 * s] : none;
                    top = max(max(top, static_cast<int>(x[s].x & 0x7fff)),
                              static_cast<int>((x[s].x >> 16) & 0x7fff));
                    top = max(max(top, static_cast<int>(x[s].y & 0x7fff)),
                              static_cast<int>((x[s].y >> 16) & 0x7fff));
                }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int a = kv8_query_shift(top >> 7);
                const float up = __int_as_float((a + 127) << 23);
                unit[h] = __int_as_float((127 - a) << 23);
#pragma unroll
                for (int s = 0; s < D / 16; ++s)
                    if (s % 4 == warp) {
                        mine[s / 4][h] = pack_f16x2(__uint_as_float(x[s].x << 16) * up,
                                                    __uint_as_float(x[s].x & 0xffff0000u) * up);
                        mine[s / 4][h + 2] = pack_f16x2(__uint_as_float(x[s].y << 16) * up,
                                                        __uint_as_float(x[s].y & 0xffff0000u) * up);
                    }
            }
#pragma unroll
            for (int i = 0; i < D / 64; ++i)
                st_shared_v4(qs + (4 * i + warp) * 512, mine[i][0], mine[i][1], mine[i][2], mine[i][3]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            c_row[h] = p.scale_log2 * unit[h];
            if (warp == 0 && tq == 0) bars->unit[gq + 8 * h] = unit[h];
        }
        // A factor c below fp32's normal range (0 times a masked -infinity would be NaN), or a key scale
        // above kFarScale: from that chunk on the three scales meet before the scores, and c is 1.
        float far = fminf(c_row[0], c_row[1]) < 0x1p-126f ? -1.f : kFarScale;
        named_bar_sync(1, 128);
        // keys every row of the unit sees: [full_lo, full_hi]
        int full_lo, full_hi;
        {
            int lo, hi;
            row_key_interval(row0 / p.g, Lq, L, p.causal, p.wl, p.wr, lo, full_hi);
            row_key_interval((row0 + rows - 1) / p.g, Lq, L, p.causal, p.wl, p.wr, full_lo, hi);
        }
        bool ok = true;
        for (int c = w.c0; c < w.c1; ++c, ++n) {
            const uint32_t st = n % C::kStages;
            ok = __all_sync(0xffffffffu, wd.wait(&bars->full[st], (n / C::kStages) & 1));
            if (!ok) break;
            const uint32_t kbase = smem_u32(smem + st * C::kStageBytes);
            const uint32_t sbase =
                smem_u32(smem + C::kOffScale + st * 2 * kKv8Chunk) + warp * 32 + 2 * tq;
            const int key0 = c * kKv8Chunk + warp * 32;
            if (key0 < L) {
                // S (16 rows x 32 keys) = Q K^T on the codes; the thread's keys are
                // 8 nt + 2 tq + {0, 1} of the four n-tiles, whose MMAs are four chains side by side (two
                // at a time, as the fragments come, took 2.5% longer with both parts of the queries)
                float s[4][4];
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
                const int key = warp * 32 + (mi & 1) * 8 + ri;
#pragma unroll
                for (int u = 0; u < D / 16; u += 2) {
                    uint32_t qa[2][4], lo[2][4];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint4 f = ld_shared_v4(qs + (u + i) * 512);
                        qa[i][0] = f.x, qa[i][1] = f.y, qa[i][2] = f.z, qa[i][3] = f.w;
                        if (!kLo) continue;
                        f = ld_shared_v4(qs + C::kQBytes + (u + i) * 512);
                        lo[i][0] = f.x, lo[i][1] = f.y, lo[i][2] = f.z, lo[i][3] = f.w;
                    }
                    uint32_t b[2][8];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t r[4];
                        ldmatrix_x4(kbase + kv8_unit<D>(key + 16 * h, u + (mi >> 1)), r[0], r[1],
                                    r[2], r[3]);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            e4m3x4_to_f16x2(r[i], b[h][2 * i], b[h][2 * i + 1]);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
#pragma unroll
                        for (int nt = 0; nt < 4; ++nt)
                            mma_f16_16816(s[nt], qa[i], b[nt >> 1][4 * i + 2 * (nt & 1)],
                                          b[nt >> 1][4 * i + 2 * (nt & 1) + 1]);
                        if (kLo) {
#pragma unroll
                            for (int nt = 0; nt < 4; ++nt)
                                mma_f16_16816(s[nt], lo[i], b[nt >> 1][4 * i + 2 * (nt & 1)],
                                              b[nt >> 1][4 * i + 2 * (nt & 1) + 1]);
                        }
                    }
                }
                // the keys' scales, in pairs: 2^(b - 127) is the float with exponent field b
                float ks[4][2], vs[4][2];
                float k_top = 0.f, v_top = 0.f;
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    scale_pair(ld_shared_u16(sbase + 8 * nt), ks[nt]);
                    scale_pair(ld_shared_u16(sbase + kKv8Chunk + 8 * nt), vs[nt]);
                }
                uint32_t sel[4] = {0x3120u, 0x3120u, 0x3120u, 0x3120u};
                const bool masked = key0 < full_lo || key0 + 31 > full_hi;
                if (masked) {
                    // keys that no row of the unit sees (past the end, behind the last row's position,
                    // before the first one's window): their slots may hold anything
                    int lo, hi, none;
                    row_key_interval(row0 / p.g, Lq, L, p.causal, p.wl, p.wr, lo, none);
                    row_key_interval((row0 + rows - 1) / p.g, Lq, L, p.causal, p.wl, p.wr, none, hi);
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt) {
                        const int j = key0 + 8 * nt + 2 * tq;
                        const bool see0 = lo <= j && j <= hi, see1 = lo <= j + 1 && j + 1 <= hi;
                        if (!see0) ks[nt][0] = vs[nt][0] = 0.f;
                        if (!see1) ks[nt][1] = vs[nt][1] = 0.f;
                        sel[nt] = (see0 ? 0x0100u : 0x0404u) | (see1 ? 0x3020u : 0x4040u);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    k_top = fmax3(k_top, ks[nt][0], ks[nt][1]);
                    v_top = fmax3(v_top, vs[nt][0], vs[nt][1]);
                }
                if (__any_sync(0xffffffffu, k_top > far)) {
                    far = -1.f;
                    c_row[0] = c_row[1] = 1.f;
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float u = bars->unit[gq + 8 * r];
#pragma unroll
                        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                // (finite: a score may be 0; byte 255 stands for NaN)
                                const float t = fminf(fminf(ks[nt][i] * u, kMaxScale) * p.scale_log2, kMaxScale);
                                s[nt][2 * r + i] *= ks[nt][i] > kMaxScale ? __int_as_float(0x7fffffff) : t;
                            }
                    }
                } else {
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt) {
                        const uint64_t kp = f2_make(ks[nt][0], ks[nt][1]);
                        f2_split(f2_mul(f2_make(s[nt][0], s[nt][1]), kp), s[nt][0], s[nt][1]);
                        f2_split(f2_mul(f2_make(s[nt][2], s[nt][3]), kp), s[nt][2], s[nt][3]);
                    }
                }
                if (masked) {
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int j = key0 + nt * 8 + 2 * tq + (e & 1);
                            if (j < kmin[e >> 1] || j > kmax[e >> 1]) s[nt][e] = -INFINITY;
                        }
                }
                // The references move only when a row's maximum passes m by more than 8 or a V
                // scale passes E by more than 2: the weights stay below 2^8, their f16 form
                // P 2^(5 + ev - E) below 2^15, and most chunks leave O alone.
                float mx[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float x = fmax3(s[0][2 * r], s[0][2 * r + 1], s[1][2 * r]);
                    x = fmax3(x, s[1][2 * r + 1], s[2][2 * r]);
                    x = fmax3(x, s[2][2 * r + 1], s[3][2 * r]);
                    x = fmaxf(x, s[3][2 * r + 1]);
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                    mx[r] = x * c_row[r];
                }
                const bool m_moves = mx[0] > m_run[0] + 8.f || mx[1] > m_run[1] + 8.f;
                const bool e_moves = v_top * fmaxf(inv[0], inv[1]) > 128.f;
                if (__any_sync(0xffffffffu, m_moves || e_moves)) {
                    // E follows the largest P 2^ev that a row has met, and the keys' largest scale by 4 at
                    // most: a scale far above, of a key that the row does not see or that weighs little
                    // in it, leaves the precision to the others.  (By more where 2^(5 + ev - E), which
                    // meets P = 0, would pass fp32's range.)  One E a warp, 4 multiplications less a
                    // step, took 342.9 us for the 64 sequences where this takes 344.7.
                    int v_exp = __float_as_int(v_top) >> 23;
#pragma unroll
                    for (int i = 16; i > 0; i >>= 1)
                        v_exp = max(v_exp, __shfl_xor_sync(0xffffffffu, v_exp, i));
                    float pv[2] = {-INFINITY, -INFINITY};  // the chunk's largest log2 P 2^ev (a scale byte)
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float ev = static_cast<float>(__float_as_int(vs[nt][i]) >> 23);
#pragma unroll
                            for (int r = 0; r < 2; ++r)
                                pv[r] = fmaxf(pv[r], fmaf(s[nt][2 * r + i], c_row[r], ev));
                        }
                    float alpha[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        pv[r] = fmaxf(pv[r], __shfl_xor_sync(0xffffffffu, pv[r], 1));
                        pv[r] = fmaxf(pv[r], __shfl_xor_sync(0xffffffffu, pv[r], 2));
                        const float m_new = fmaxf(m_run[r], mx[r]);
                        const bool none = m_new == -INFINITY;
                        const float drop = none ? 0.f : m_run[r] - m_new;
                        const float top = none ? 0.f : ceilf(pv[r] - m_new);
                        const int e_run = 259 - (__float_as_int(inv[r]) >> 23), least = max(kMinE, v_exp - 120);
                        const int e_new = min(max(max(static_cast<int>(ceilf(drop + e_run)), least),
                                                  max(static_cast<int>(top), min(v_exp, static_cast<int>(top) + 4))),
                                              252);
                        l2[r] = f2_mul(l2[r], f2_make(ex2_approx(drop), ex2_approx(drop)));
                        alpha[r] = ex2_approx(drop + (e_run - e_new));
                        m_run[r] = m_new;
                        inv[r] = __int_as_float((259 - e_new) << 23);
                    }
                    // a V scale byte of 255: every output of the rows becomes NaN
                    if (v_exp == 255) alpha[0] = alpha[1] = __int_as_float(0x7fffffff);
#pragma unroll
                    for (int x = 0; x < D / 8; ++x)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[x][e] *= alpha[e >> 1];
                }
                const uint64_t c2[2] = {f2_make(c_row[0], c_row[0]), f2_make(c_row[1], c_row[1])};
                uint64_t nm[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float m = m_run[r] == -INFINITY ? 0.f : -m_run[r];  // no key seen yet
                    nm[r] = f2_make(m, m);
                }
                uint32_t pa[2][4];  // P as the A operand of two k-steps of 16 keys
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float x0, x1;
                        f2_split(f2_fma(f2_make(s[nt][2 * r], s[nt][2 * r + 1]), c2[r], nm[r]), x0, x1);
                        const uint64_t pp = f2_make(ex2_approx(x0), ex2_approx(x1));
                        l2[r] = f2_add(l2[r], pp);
                        f2_split(f2_mul(pp, f2_mul(f2_make(vs[nt][0], vs[nt][1]), f2_make(inv[r], inv[r]))), x0, x1);
                        pa[nt >> 1][2 * (nt & 1) + r] = pack_f16x2(x0, x1);
                    }
                }
                // O += P V.  A transposed 8 x 8 matrix of byte pairs gives the thread elements
                // 2 gq, 2 gq + 1 of keys 2 tq, 2 tq + 1: the pair of even elements is one n-tile's
                // operand, the odd pair the next one's.  The selector puts them in that order and
                // takes zeros for keys that no row sees.
                const uint32_t vbase = kbase + C::kTileBytes;
#pragma unroll
                for (int u = 0; u < D / 16; u += 2) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t r[4], b[8];
                        ldmatrix_x4_trans(vbase + kv8_unit<D>(key + 16 * h, u + (mi >> 1)), r[0],
                                          r[1], r[2], r[3]);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            e4m3x4_to_f16x2(__byte_perm(r[i], 0u, sel[2 * h + (i & 1)]), b[2 * i],
                                            b[2 * i + 1]);
                        mma_f16_16816(o[2 * u], pa[h], b[0], b[2]);
                        mma_f16_16816(o[2 * u + 1], pa[h], b[1], b[3]);
                        mma_f16_16816(o[2 * u + 2], pa[h], b[4], b[6]);
                        mma_f16_16816(o[2 * u + 3], pa[h], b[5], b[7]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->empty[st]);
        }

        // ---- the warps' results merge, in a fixed order ----
        float* const mm = ml_all + (seg & 1) * 2 * 4 * kKv8Rows;  // [4][16] references m
        float* const ml = mm + 4 * kKv8Rows;                      // [4][16] denominators
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float even, odd;
            f2_split(l2[r], even, odd);
            even += odd;
            even += __shfl_xor_sync(0xffffffffu, even, 1);
            even += __shfl_xor_sync(0xffffffffu, even, 2);
            if (tq == 0) {
                mm[warp * kKv8Rows + gq + 8 * r] = m_run[r];
                ml[warp * kKv8Rows + gq + 8 * r] = even;
            }
        }
        if (!ok && lane == 0) bars->fail[seg & 1] = 1;
        named_bar_sync(1, 128);
        // the same answer in all four warps: the flag of this parity was last written before the
        // barrier, and is written again only behind the next segment's barriers
        if (*reinterpret_cast<volatile int*>(&bars->fail[seg & 1])) return;
        const bool whole = w.first && w.last;
        float sc[2];  // of the warp's O: 2^(m - M) 2^(E - 5) / l
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = gq + 8 * h;
            float M = -INFINITY, lsum = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) M = fmaxf(M, mm[i * kKv8Rows + r]);
            if (M == -INFINITY) M = 0.f;  // no key seen, or only NaN scores: l tells which
#pragma unroll
            for (int i = 0; i < 4; ++i) lsum += ml[i * kKv8Rows + r] * ex2_approx(mm[i * kKv8Rows + r] - M);
            const float over = lsum == 0.f ? 0.f : 1.f / lsum;
            const float un = __int_as_float((254 << 23) - __float_as_int(inv[h]));  // 2^(E - 5)
            const bool tiny = un < 0x1p-60f;
            if (__any_sync(0xffffffffu, tiny)) {  // (un over l may be no normal number)
#pragma unroll
                for (int x = 0; x < D / 8; ++x)
#pragma unroll
                    for (int e = 0; e < 2; ++e) o[x][2 * h + e] *= tiny ? 0x1p-60f : 1.f;
            }
            sc[h] = ex2_approx(m_run[h] - M) * over * (tiny ? un * 0x1p60f : un);
            if (warp == 0 && tq == 0 && r < rows) {
                const float lse = lsum == 0.f ? -INFINITY : M + __log2f(lsum);  // log2
                const int tok = q0 + (row0 + r) / p.g, head = kvh * p.g + (row0 + r) % p.g;
                if (!whole)
                    p.part_lse[(2 * static_cast<size_t>(cta) + (w.first ? 1 : 0)) * kKv8Rows + r] = lse;
                else if (ATTN_IN_BOUNDS(head < p.Hq && tok < p.total_q, p.status))
                    p.lse[static_cast<size_t>(head) * p.lse_head + static_cast<size_t>(tok) * p.lse_tok] =
                        lse * kLn2f;
            }
        }
        // Behind the last segment the stages are free, and each warp has a buffer there; before,
        // the warps add to one buffer in turn.
        const bool apart = w.left == 0;
        float* const buf = apart ? reinterpret_cast<float*>(smem) : mo;
        float* const own = buf + (apart ? warp * kKv8Rows * C::kMergeStride : 0);
        for (int turn = apart ? warp : 0; turn < 4; ++turn) {
            if (turn == warp) {
#pragma unroll
                for (int u = 0; u < D / 16; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float4* dst = reinterpret_cast<float4*>(own + (gq + 8 * h) * C::kMergeStride +
                                                                16 * u + 4 * tq);
                        float4 v = make_float4(o[2 * u][2 * h] * sc[h], o[2 * u + 1][2 * h] * sc[h],
                                               o[2 * u][2 * h + 1] * sc[h],
                                               o[2 * u + 1][2 * h + 1] * sc[h]);
                        if (!apart && turn > 0) {
                            const float4 a = *dst;
                            v = make_float4(a.x + v.x, a.y + v.y, a.z + v.z, a.w + v.w);
                        }
                        *dst = v;
                    }
            }
            if (apart) break;
            named_bar_sync(1, 128);
        }
        if (apart) named_bar_sync(1, 128);
#pragma unroll
        for (int i = 0; i < kKv8Rows * D / 4 / 128; ++i) {
            const int e = threadIdx.x + 128 * i, r = e / (D / 4), d = 4 * (e % (D / 4));
            if (r >= rows) break;
            float4 v = *reinterpret_cast<const float4*>(buf + r * C::kMergeStride + d);
            if (apart) {
#pragma unroll
                for (int j = 1; j < 4; ++j) {
                    const float4 a = *reinterpret_cast<const float4*>(
                        buf + (j * kKv8Rows + r) * C::kMergeStride + d);
                    v = make_float4(v.x + a.x, v.y + a.y, v.z + a.z, v.w + a.w);
                }
            }
            const int tok = q0 + (row0 + r) / p.g, head = kvh * p.g + (row0 + r) % p.g;
            if (!ATTN_IN_BOUNDS(head < p.Hq && tok < p.total_q, p.status)) continue;
            if (whole)
                *reinterpret_cast<uint2*>(p.out + (static_cast<size_t>(tok) * p.Hq + head) * D + d) =
                    make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
            else
                *reinterpret_cast<float4*>(
                    p.part_o + ((2 * static_cast<size_t>(cta) + (w.first ? 1 : 0)) * kKv8Rows + r) * D + d) = v;
        }
        if (w.last && !w.first && threadIdx.x == 0) {
            p.meta[cta] = make_int4((bars->start + w.before) / bars->share, q0, row0, rows);
        }
        named_bar_sync(1, 128);  // the merge buffer has been read: the next segment's queries may come
    }
}

// Merges the units that were cut: a CTA's entry names the share in which the unit it ended started.
// LSE = log2 sum_s 2^LSE_s, O = sum_s 2^(LSE_s - LSE) O_s (a part without keys has LSE_s = -inf
// and weight 0).
template <int D>
__global__ void __launch_bounds__(kKv8Rows * 16) kv8_combine_kernel(const Kv8Params p) {
    griddep_wait();
    const int cta = blockIdx.x;
    const int4 m = p.meta[cta];
    const int kvh = cta % p.Hkv, last = cta / p.Hkv;
    const int r = threadIdx.x / 16, d0 = (threadIdx.x % 16) * 4;
    if (m.x < 0 || r >= m.w) return;
    // parts: slot 1 of the CTA with the head's share m.x, then slot 0 of those up to this one
    const auto part = [&](int s) {
        return (2 * (static_cast<size_t>(s) * p.Hkv + kvh) + (s == m.x ? 1 : 0)) * kKv8Rows + r;
    };
    // One pass, four parts' loads in flight: the sums are kept relative to the running maximum.
    float M = -INFINITY, sum = 0.f;
    float4 acc[D / 64];
#pragma unroll
    for (int i = 0; i < D / 64; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = m.x; s0 <= last; s0 += 4) {
        float x[4], top = M;
        float4 v[4][D / 64];
        bool nan = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const size_t at = part(min(s0 + j, last));
            x[j] = p.part_lse[at];
#pragma unroll
            for (int i = 0; i < D / 64; ++i)
                v[j][i] = *reinterpret_cast<const float4*>(p.part_o + at * D + d0 + 64 * i);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (s0 + j > last) x[j] = -INFINITY;
            nan = nan || x[j] != x[j];
            top = fmaxf(top, x[j]);
        }
        if (top == -INFINITY) continue;  // no keys so far
        if (nan) top = __int_as_float(0x7fffffff);
        const float keep = ex2_approx(M - top);
        M = top;
        sum *= keep;
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
            acc[i] = make_float4(acc[i].x * keep, acc[i].y * keep, acc[i].z * keep, acc[i].w * keep);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float wgt = ex2_approx(x[j] - M);
            sum += wgt;
            if (s0 + j > last) continue;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                acc[i].x += wgt * v[j][i].x;
                acc[i].y += wgt * v[j][i].y;
                acc[i].z += wgt * v[j][i].z;
                acc[i].w += wgt * v[j][i].w;
            }
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int tok = m.y + (m.z + r) / p.g, head = kvh * p.g + (m.z + r) % p.g;
#pragma unroll
    for (int i = 0; i < D / 64; ++i)
        *reinterpret_cast<uint2*>(p.out + (static_cast<size_t>(tok) * p.Hq + head) * D + d0 + 64 * i) =
            make_uint2(pack_bf16x2(acc[i].x * inv, acc[i].y * inv),
                       pack_bf16x2(acc[i].z * inv, acc[i].w * inv));
    if (threadIdx.x % 16 == 0)
        p.lse[static_cast<size_t>(head) * p.lse_head + static_cast<size_t>(tok) * p.lse_tok] =
            sum == 0.f ? -INFINITY : (M + __log2f(sum)) * kLn2f;
}

}  // namespace

cudaError_t configure_kv8_kernels() {
    const cudaFuncAttribute smem = cudaFuncAttributeMaxDynamicSharedMemorySize;
    cudaError_t e = cudaFuncSetAttribute(kv8_split_kernel<128, false>, smem, Kv8Cfg<128>::kSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kv8_split_kernel<128, true>, smem, Kv8Cfg<128>::kSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kv8_split_kernel<64, false>, smem, Kv8Cfg<64>::kSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kv8_split_kernel<64, true>, smem, Kv8Cfg<64>::kSmem);
    return e;
}

namespace {

template <typename Kernel>
cudaError_t launch(Kernel kernel, int grid, int threads, size_t smem, bool dependent,
                   const Kv8Params& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

// Both kernels set up while the one before them finishes (the first only behind the append kernel
// of the same call).
cudaError_t launch_kv8_attn(const Kv8Params& p, int head_dim, int grid, bool after_append,
                            cudaStream_t stream) {
    const bool lo = p.q_lo != nullptr;
    const cudaError_t e =
        head_dim == 128
            ? launch(lo ? kv8_split_kernel<128, true> : kv8_split_kernel<128, false>, grid,
                     kKv8Threads, Kv8Cfg<128>::kSmem, after_append, p, stream)
            : launch(lo ? kv8_split_kernel<64, true> : kv8_split_kernel<64, false>, grid,
                     kKv8Threads, Kv8Cfg<64>::kSmem, after_append, p, stream);
    if (e != cudaSuccess || grid == p.Hkv) return e;  // (one CTA a head cuts nothing)
    return head_dim == 128
               ? launch(kv8_combine_kernel<128>, grid, kKv8Rows * 16, 0, true, p, stream)
               : launch(kv8_combine_kernel<64>, grid, kKv8Rows * 16, 0, true, p, stream);
}

}  // namespace attn

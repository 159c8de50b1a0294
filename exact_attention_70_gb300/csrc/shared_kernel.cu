// shared_kernel.cu -- attention of few query tokens a sequence over the paged cache where sequences share
// prefixes: the keys of a prefix are read once for all the sequences of its group.
//
// The method ("Attention kernels: FlashAttention and PagedAttention", sections 三.2, 五.2-五.3, 六.1 and
// 六.3; "04 · FA4 (CuTeDSL) and engineering interfaces", sections 5 and 6.1-6.2): softmax over two
// disjoint sets of keys is the LSE-weighted sum of the softmax over each.  A group's tokens are neighbours in q,
// so a group against its prefix is what one long sequence is against its keys: its tokens times the g query
// heads of a kv head fill tiles of 128 rows.  Then every sequence meets the keys behind its prefix, and
// a last kernel merges the parts.
//
// Three kernels, each starting while the one before it ends:
//   * shared_units_kernel (one CTA) writes the list of the work: units (query rows that walk the same
//     keys) cut into pieces that keep all CTAs busy to about the same end;
//   * shared_attn_kernel, one CTA an SM, persistent.  Some of its CTAs, as many as the units of more than 16 rows are
//     of the work, do those on tcgen05: two tiles of 128 rows on the same key blocks, roles and barriers as in
//     the prefill kernel (fwd_kernel.cu): warp 16 gathers K and V blocks of 128 keys through block_table, a
//     lane a page, into a ring of shared-memory slots (K_0, K_1, V_0, K_2, V_1, ..., V_{m-1}); warp 17 issues
//     S_t = Q_t K^T, warp 18 O_t += P_t V, accumulators in TMEM; warps 0-7 and 8-15 do the softmax of the
//     two tiles, 16 rows a warp (one whose rows hold no token only keeps the barriers going); warp 19 claims
//     items.  The other CTAs, and these when they are done, do the units of up to 16 rows on mma.sync, each as two.
//     (Where the host can tell that no unit has more, by all tokens of the call or, without groups, by the most of a
//     sequence, shared_small_kernel does them.)
//   * shared_combine_kernel merges the parts (O / l and log2 LSE of a piece, fp32).
// Both sides of the 16 rows (all on tcgen05 / as it is): 4 sequences on 512 keys 16.9 / 12.8 us, 64 sequences of
// 1K to 16K keys of their own, 32:8 heads, 361 / 349 (345 without a group list), 2 of 100K 212 / 131, 5 ragged
// documents 53.9 / 47.7.
//
// Measured in a captured graph, d 128, bf16: 64 requests on 32768 shared and 100 to 2000 own keys, 32:8 heads:
// 84 us (one after the other, by the profiler: list 6, attention 74, merge 5 behind it; 421 MB, 5.0 TB/s over all); 16
// samples of 4 tokens on 100001 keys: 102.5 us (list 6, attention 91, merge 6).  With the two kinds in two kernels one after the other, all SMs on each, the
// first took 97.5 us: the tiles' chain left a seventh of the memory's time idle, and one kernel's last CTAs and the
// other's first loads another 10 us.
// A block of 128 keys under two tiles takes 1.7 to 2.1 us where the memory would take 1.47 (from prefix to prefix, 50K to
// 300K keys on all CTAs; d 64: 1.1 to 1.6, memory 0.74): the chain S, softmax, P V of a tile, 16 warps at half their
// issue rate, is what bounds it, as in the prefill kernel.
// Tried for it and not kept: P in tensor memory over S and five ring slots (the chain gets longer: 122 -> 136 us),
// asking for blocks in L2 ahead of their loads (121 -> 138 us, the TMA unit's work doubles), two pieces a CTA
// (107 -> 120: twice the parts).
#include <cuda_bf16.h>

#include <algorithm>

#include "ptx.cuh"
#include "step_kernels.h"
#include "tile_math.h"

namespace attn {

namespace {

constexpr float kShRescale = 8.0f;  // log2: the reference of a row moves when its maximum passes it by more
constexpr float kShLn2 = 0.69314718055994530942f;
constexpr int kShUnitsThreads = 512;
constexpr int kShFast = 1024;  // groups, and half the units, that the list's kernel keeps in shared memory
constexpr int kShBins = 32;    // lengths that the list tells apart
constexpr int kShLimbs = 3;    // of 20 bits
// Shorter prefixes are read by every sequence.  (Near this size sharing saves little, keys that L2 holds anyway: 64
// sequences, 32:8 heads, on 128 shared keys 25.8 us (26.2 without sharing), on 512 28.1 (34.8), on 1024 28.6 (45.7);
// 4 sequences on 512 12.8 (12.5), on 2048 13.6 (13.8), on 8192 21.6 (25.8).)
// The same calls without a group list, in the kernel for few rows alone: 64 on 128 keys 23.4 us, on 512 30.9, on
// 1024 39.9; 4 on 512 12.5, on 2048 13.9, on 8192 25.2; 16 on 1024 16.6 (18.5 with the list), 2 on 16K 23.9 (25.4),
// on 32K 33.9 (37.5).  So a caller with two sequences, or with little in common, leaves the list out.
constexpr int kShMinPrefix = 128;
// Key blocks a piece takes at least: 2 sequences on 4096 keys, 64:8 heads, 16.2 us (18.0 with 1, 15.5 with 4),
// 4 on 512 12.8 (12.4, 14.2), on 2048 13.6 (15.0, 15.0).
constexpr int kShMinPiece = 2;
// Where there are units of both kinds, those of few rows are not a kernel's only work but fill what the others leave:
// pieces of eight blocks (16 x 4 tokens on 100001 keys, 600 of their own: 105.3 us, 111.9 with two, 106.4 with four).
constexpr int kShMinFewPiece = 8;
// What a block under two tiles costs in blocks under few rows.  The CTAs are divided by it: the tiles' chain leaves
// memory idle that the few rows' loads take (64 requests on 32768 shared and 100 to 2000 own keys: 84.2 us, 90.8 with
// 1.6, 88.8 with 5, 97.8 with all CTAs on tiles first; 5 ragged documents 47.9, 53.2, 48.8, 57.1).  These, and
// the piece above, at d 128; not measured at d 64, where a tile's block takes 1.4 us and its bytes 0.74.
constexpr float kShManyCost = 3.f;
constexpr int kShCombineThreads = 256;
// The merge gives a row eight warps up to kShFewRows rows, four up to kShMostRows (the blocks that are resident at
// once), two beyond.  Few: 64 rows behind 16K shared keys 25.5 us (28.5 with four), 128 rows behind 8K 21.6 (24.5); 512
// rows behind 1K 18.5 (18.2 with eight).  Most: 2048 rows behind 32K 84.4 (86.7 with four, 91.8 with eight), 4096
// rows behind 8K 51.2 (56.0, 65.3), 1204 rows of ragged documents 47.9 (49.2 with two).
constexpr int kShFewRows = kGb300Sms;
constexpr int kShMostRows = 10 * kGb300Sms;
constexpr int kShSoftmaxWarps = 16;

// ---- units and items (one CTA) --------------------------------------------------------------------

struct ShSeq {
    int q0, n, keys;
};

__device__ __forceinline__ ShSeq sh_seq(const SharedParams& p, int b) {
    ShSeq s;
    s.q0 = b;
    s.n = 1;
    if (p.cu_q != nullptr) {
        s.q0 = p.cu_q[b];
        s.n = p.cu_q[b + 1] - s.q0;
    }
    s.keys = p.seqlens[b];
    return s;
}

// Every query of the sequence sees the whole prefix.
__device__ __forceinline__ bool sh_behind(const ShSeq& s, int prefix) {
    return s.n > 0 && prefix > 0 && prefix <= s.keys - s.n + 1;
}

// (of numbers that are not negative: an unsigned division is shorter)
__host__ __device__ __forceinline__ int ceil_div(int a, int b) {
    return static_cast<int>((static_cast<unsigned>(a) + b - 1) / static_cast<unsigned>(b));
}

// This thread's place behind the earlier lanes' n on a counter in shared memory (one atomic a warp).
__device__ __forceinline__ int sh_reserve(int* counter, int n, int lane) {
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    int at = 0;
    if (lane == 31 && x > 0) at = atomicAdd(counter, x);
    return __shfl_sync(0xffffffffu, at, 31) + x - n;
}

// The list is read past L1: kernels that start before the one in front of them has ended could find lines of the
// call before there.
__device__ __forceinline__ SharedUnit sh_unit(const SharedParams& p, int i) {
    SharedUnit u;
    const int4* src = reinterpret_cast<const int4*>(p.units + i);
    int4* dst = reinterpret_cast<int4*>(&u);
#pragma unroll
    for (int x = 0; x < static_cast<int>(sizeof(SharedUnit) / sizeof(int4)); ++x) dst[x] = __ldcg(src + x);
    return u;
}

// All of it but the fields that step 3 of the list's kernel writes: its third 16 bytes.
__device__ __forceinline__ void sh_put(const SharedParams& p, int i, const SharedUnit& u) {
    const int4* src = reinterpret_cast<const int4*>(&u);
    int4* dst = reinterpret_cast<int4*>(p.units + i);
    dst[0] = src[0];
    dst[1] = src[1];
    dst[3] = src[3];
}

__device__ __forceinline__ bool sh_few(int rows) { return rows <= kSharedSmallRows; }

// Writes the list.  Where the parts lie and the order among units of a length depend on the warps' order;
// no result does.  Items of a kind come longest pieces first (kShBins lengths), the kv heads of a piece
// side by side (their keys lie side by side in the cache).
// Bound by the latency of its steps, one after the other: 10,000 to 10,600 clocks (11,300 to 16,400 with idle warps in
// every step, units in 4-byte stores, 64-bit atomics and a thread a unit that wrote its items).
__global__ void __launch_bounds__(kShUnitsThreads) shared_units_kernel(const SharedParams p) {
    __shared__ int4 s_groups[kShFast];  // {first unit or -1, first token, first sequence, prefix}
    __shared__ int2 s_lengths[2 * kShFast];
    __shared__ int s_q0[kShFast], s_n[kShFast], s_keys[kShFast];
    __shared__ __align__(16) int hist[2 * kShBins];
    __shared__ int place[2 * kShBins];
    __shared__ unsigned work[2][kShLimbs];  // key blocks of both kinds, for one kv head
    __shared__ int n_prefix, n_own, n_parts, n_many, s_ctas;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    griddep_launch_dependents();  // (the attention kernels wait for the list, behind their set-up)
    // (generic addresses: shared memory as far as it goes)
    int4* const groups = p.n_groups <= kShFast ? s_groups : p.groups;
    const bool near = p.batch <= kShFast;
    int2* const lengths = p.max_units <= 2 * kShFast ? s_lengths : p.lengths;
    const long long max_keys = static_cast<long long>(p.max_pages) * p.page_size;
    if (tid < 2 * kShBins) hist[tid] = 0;
    if (tid < 2 * kShLimbs) work[0][tid] = 0;
    if (tid == 0) n_prefix = n_own = n_parts = n_many = 0;
    bool bad = false;
    // (here and below a warp that has nothing of it skips a stage: its instructions would hold up the others)
    for (int base = 32 * warp; base < max(p.batch, p.n_groups); base += kShUnitsThreads) {
        const int b = base + lane;
        const bool is_group = b < p.n_groups, is_seq = b < p.batch;
        int s0 = 0, s1 = 0, P = 0;
        ShSeq s = {0, 0, 0};
        if (is_seq) s = sh_seq(p, b);  // (all loads go out together)
        if (is_group) s0 = p.group_starts[b], s1 = p.group_starts[b + 1], P = p.prefix_lens[b];
        bad |= s.q0 < 0 || s.n < 0 || s.n > p.max_seqlen_q || static_cast<long long>(s.q0) + s.n > p.total_q ||
               s.keys < 0 || s.keys > max_keys;
        bad |= is_group && (s0 < 0 || s1 < s0 || s1 > p.batch || (b == 0 && s0 != 0) ||
                            (b == p.n_groups - 1 && s1 != p.batch) || P < 0);
        if (is_seq && near) s_q0[b] = s.q0, s_n[b] = s.n, s_keys[b] = s.keys;
        if (is_group) groups[b] = make_int4(-1, 0, s0, P);
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) {
            atomicOr(p.status, kStatusBounds);
            SharedHeader* h = p.header;
            h->n_items[0] = h->n_items[1] = h->next_item[0] = h->next_item[1] = h->n_own = 0;
            h->bad = 1;
            h->ctas = 0;
        }
        return;
    }
    const auto seq = [&](int b) { return near ? ShSeq{s_q0[b], s_n[b], s_keys[b]} : sh_seq(p, b); };
    const int per = 2 * p.tpt;  // tokens a unit
    const auto units_of = [&](int tokens) { return tokens <= per ? (tokens > 0 ? 1 : 0) : ceil_div(tokens, per); };
    unsigned long long mine[2] = {0, 0};  // this thread's share of work
    int many_units = 0;
    // 1. a warp a group: which row of the table leads to the prefix, which tokens meet it, their units
    for (int i = warp; i < p.n_groups; i += kShUnitsThreads / 32) {
        const int s0 = groups[i].z, P = groups[i].w;
        const int s1 = i + 1 < p.n_groups ? groups[i + 1].z : p.batch;
        int first = -1, count = 0;
        if (P >= kShMinPrefix) {
            for (int b = s0; b < s1; b += 32) {
                const bool on = b + lane < s1 && sh_behind(seq(b + lane), P);
                const unsigned m = __ballot_sync(0xffffffffu, on);
                if (first < 0 && m != 0) first = b + __ffs(m) - 1;
                count += __popc(m);
            }
        }
        if (count > 1) {
            int at = 0;
            const ShSeq a = seq(s0), z = seq(s1 - 1);
            const int q0 = a.q0;
            const int tokens = z.q0 + z.n - q0, n = units_of(tokens), nblk = ceil_div(P, kFwdBlockN);
            if (lane == 0) at = atomicAdd(&n_prefix, n);
            at = __shfl_sync(0xffffffffu, at, 0);
            for (int u = lane; u < n; u += 32) {
                SharedUnit x = {};
                x.q0 = q0 + u * per;
                x.ntok = min(per, tokens - u * per);
                x.row = first;
                x.key_min = 0;
                x.key_end = P;
                x.pos0 = 1 << 30;
                x.blk0 = 0;
                x.nblk = nblk;
                x.rows = x.ntok * p.g;
                x.prefix = -1;
                x.group_q0 = 0;
                mine[sh_few(x.rows)] += nblk;
                many_units += !sh_few(x.rows);
                if (at + u < p.own_base) {
                    sh_put(p, at + u, x);
                    lengths[at + u] = make_int2(nblk, x.rows);
                }
            }
            // (only x and y: other warps read z meanwhile)
            if (lane == 0) *reinterpret_cast<int2*>(&groups[i]) = make_int2(at, q0);
        }
    }
    __syncthreads();
    // 2. a thread a sequence: the keys that its group's prefix leaves to it
    for (int base = 32 * warp; base < p.batch; base += kShUnitsThreads) {
        const int b = base + lane;
        ShSeq s = {0, 0, 0};
        if (b < p.batch) s = seq(b);
        const int n = units_of(s.n);
        int prefix = -1, group_q0 = 0, key_min = 0;
        if (n > 0 && p.n_groups > 0) {
            int lo = 0, hi = p.n_groups - 1;  // the last group that starts at b or before
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (groups[mid].z <= b) lo = mid; else hi = mid - 1;
            }
            const int4 r = groups[lo];
            if (r.x >= 0 && sh_behind(s, r.w)) {
                prefix = r.x;
                group_q0 = r.y;
                key_min = r.w;
            }
        }
        const int at = p.own_base + sh_reserve(&n_own, n, lane);
        for (int u = 0; u < n; ++u) {
            SharedUnit x = {};
            const int t0 = u * per;
            x.q0 = s.q0 + t0;
            x.ntok = min(per, s.n - t0);
            x.row = b;
            x.key_min = key_min;
            x.pos0 = s.keys - s.n + t0;
            x.key_end = max(x.pos0 + x.ntok, 0);
            x.blk0 = key_min / kFwdBlockN;
            x.nblk = x.key_end > key_min ? ceil_div(x.key_end, kFwdBlockN) - x.blk0 : 0;
            x.rows = x.ntok * p.g;
            x.prefix = prefix;
            x.group_q0 = group_q0;
            mine[sh_few(x.rows)] += x.nblk;
            many_units += !sh_few(x.rows) && x.nblk > 0;
            if (at + u < p.max_units) {
                sh_put(p, at + u, x);
                lengths[at + u] = make_int2(x.nblk, x.rows);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (!__any_sync(0xffffffffu, mine[k] > 0)) continue;
        if (k == 0) {
            const int n = __reduce_add_sync(0xffffffffu, many_units);
            if (lane == 0) atomicAdd(&n_many, n);
        }
        for (int i = 0; i < kShLimbs; ++i) {  // (no warp instruction adds 64 bits)
            const unsigned sum = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(mine[k] >> (20 * i)) & 0xfffffu);
            if (lane == 0) atomicAdd(&work[k][i], sum);
            if (!__any_sync(0xffffffffu, mine[k] >> (20 * i + 20) != 0)) break;
        }
    }
    __syncthreads();
    const int n_pre = n_prefix, own = n_own;
    // (the host's bounds hold for every list that passed the checks above)
    const bool fits = n_pre <= p.own_base && p.own_base + own <= p.max_units;
    const int n_units = fits ? n_pre + own : 0;
    int share[2] = {1, 1}, ctas = 1;
    float per_share[2] = {0.f, 0.f};  // bins a key block
    if (32 * warp < n_units) {
        unsigned long long all[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < kShLimbs; ++i) {
            all[0] += static_cast<unsigned long long>(work[0][i]) << (20 * i);
            all[1] += static_cast<unsigned long long>(work[1][i]) << (20 * i);
        }
        if (all[0] > 0) {
            const float a = kShManyCost * static_cast<float>(all[0]);
            const int n = static_cast<int>(ceilf(kSharedShares * __fdividef(a, a + static_cast<float>(all[1]))));
            ctas = min(max(n, 1), kSharedShares);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            // (a unit's last piece is short by half a piece, about: so many more come out than shares)
            const unsigned shares = k ? kSharedSmallShares : ctas == kSharedShares ? ctas : max(ctas - n_many * p.Hkv / 2, (ctas + 1) / 2);
            // (no unit has 2^30 blocks)
            share[k] = max(static_cast<int>(min((all[k] * p.Hkv + shares - 1) / shares, 1ull << 30)),
                           k != 0 && all[0] > 0 ? kShMinFewPiece : kShMinPiece);
            per_share[k] = __fdividef(static_cast<float>(kShBins), static_cast<float>(share[k]));
        }
    }
    // a unit's pieces and the list's bin of their length
    const auto cut = [&](int i, int& u, int& few, int& pieces, int& rows, int& bin) {
        u = i < n_pre ? i : p.own_base + i - n_pre;
        const int2 x = lengths[u];
        few = sh_few(x.y);
        rows = x.y;
        pieces = x.x <= share[few] ? (x.x > 0 ? 1 : 0) : ceil_div(x.x, share[few]);
        bin = 0;
        if (pieces > 0) {
            const int len = pieces == 1 ? x.x : ceil_div(x.x, pieces);  // 1 .. share
            bin = few * kShBins + kShBins - 1 -
                  min(static_cast<int>(static_cast<float>(len - 1) * per_share[few]), kShBins - 1);
        }
    };
    if (tid == 0) s_ctas = ctas;
    // 3. pieces, and the places of their results
    int u = 0, few = 0, pieces = 0, rows = 0, bin = 0;  // of the thread's last unit
    for (int base = 32 * warp; base < n_units; base += kShUnitsThreads) {
        const bool on = base + lane < n_units;
        pieces = 0;
        if (on) cut(base + lane, u, few, pieces, rows, bin);
        const int split = few ? kSharedSmallSplit : 1;
        const int at = sh_reserve(&n_parts, pieces * split * p.Hkv * rows, lane);
        if (on) {
            *reinterpret_cast<int4*>(&p.units[u].pieces) = make_int4(pieces, split, at, rows);
            if (pieces > 0) atomicAdd(&hist[bin], pieces * p.Hkv);
        }
    }
    __syncthreads();
    // 4. the bins' places: a thread a bin adds those before it (as a warp's scan it took 2100 clocks, so 900)
    if (tid < 2 * kShBins) {
        int before = 0, many = 0, all = 0;
#pragma unroll
        for (int i = 0; i < 2 * kShBins; i += 4) {
            const int4 x = *reinterpret_cast<const int4*>(&hist[i]);
            const int v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                before += i + e < tid ? v[e] : 0;
                many += i < kShBins ? v[e] : 0;
                all += v[e];
            }
        }
        place[tid] = before;
        if (tid == 2 * kShBins - 1) {
            const bool ok = fits && n_parts <= p.max_parts && all <= p.max_items;
            if (!ok) atomicOr(p.status, kStatusBounds);
            SharedHeader* h = p.header;
            h->n_items[0] = ok ? many : 0;
            h->n_items[1] = ok ? all - many : 0;
            h->next_item[0] = h->next_item[1] = 0;
            h->n_own = ok ? own : 0;
            h->bad = ok ? 0 : 1;
            h->ctas = many <= kSharedShares ? many : s_ctas;  // (no item waits for another where all can go at once)
            if (!ok) n_parts = -1;
        }
    }
    __syncthreads();
    if (n_parts < 0) return;
    // 5. items: a thread a unit finds their places, a warp or eight lanes a unit write them
    int4* const out = s_groups;
    const int lanes_log2 = n_units <= 128 ? 5 : 3, lanes = 1 << lanes_log2;
    const int sub = tid & (lanes - 1), sub_s = sub / p.Hkv, sub_h = sub - sub_s * p.Hkv;
    const int step_s = lanes / p.Hkv, step_h = lanes - step_s * p.Hkv;
    for (int base = 0; base < n_units; base += kShUnitsThreads) {
        const int n = min(kShUnitsThreads, n_units - base);
        if (tid < n) {
            if (n_units > kShUnitsThreads) cut(base + tid, u, few, pieces, rows, bin);
            const int count = pieces * p.Hkv;
            out[tid] = make_int4(u, count > 0 ? atomicAdd(&place[bin], count) : 0, count, 0);
        }
        __syncthreads();
        for (int i = tid >> lanes_log2; i < n; i += kShUnitsThreads >> lanes_log2) {
            const int4 x = out[i];
            for (int j = sub, s = sub_s, h = sub_h; j < x.z; j += lanes) {
                p.items[x.y + j] = make_int2(x.x, s << 16 | h);
                s += step_s;
                h += step_h;
                if (h >= p.Hkv) h -= p.Hkv, ++s;
            }
        }
        if (base + kShUnitsThreads < n_units) __syncthreads();
    }
}

// ---- attention ------------------------------------------------------------------------------------

template <int D>
struct ShCfg {
    static constexpr int kHalves = D / 64;
    static constexpr int kAtomBytes = 128 * 128;
    static constexpr int kQTile = kHalves * kAtomBytes;
    static constexpr int kKvTile = kHalves * kAtomBytes;
    static constexpr int kPTile = 2 * kAtomBytes;
    static constexpr int kSlots = D == 128 ? 3 : 8;
    static constexpr int kOffQ = 0;
    static constexpr int kOffP = kOffQ + 2 * kQTile;
    static constexpr int kOffKV = kOffP + 2 * kPTile;
    static constexpr int kOffBar = kOffKV + kSlots * kKvTile;
    static constexpr int kOffFew = kOffBar + 768;  // two SmBars
    static constexpr int kSmem = kOffFew + 1024 + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
    static constexpr uint32_t kTmemCols = 512;
    __device__ static constexpr uint32_t col_s(int t) { return 128u * t; }
    __device__ static constexpr uint32_t col_o(int t) { return 256u + D * t; }
};

constexpr uint32_t kShRing = 4;
constexpr uint32_t kShReaders = 19;  // the producer, the two MMA issuers and the 16 softmax warps

// One item as the scheduler hands it to the other roles: a piece of a unit for one kv head.
struct ShItem {
    int q0, ntok;  // ntok = 0: no more items
    int kvh, row, key_min, key_end, pos0;
    int jlo, jhi;   // key blocks
    int part;       // the row of its first result
    uint32_t kv0;   // the ring's loads before its first
    uint32_t vpar;  // per slot the parity of the V loads before its first
};

struct ShBars {
    uint64_t q_full, q_empty;
    uint64_t k_full[8], v_full[8], kv_empty[8];  // (one "full" a kind of block: see fwd_kernel.cu)
    uint64_t s_full[2], s_free[2], p_full[2], pv_done[2], o_free[2];
    uint64_t drain[2];
    uint64_t idx_full[kShRing], idx_empty[kShRing];
    uint64_t near_end;  // the producer is about to be done with its item
    ShItem ring[kShRing];
    uint32_t tmem_base;
    int abort_flag, few_left;
};
static_assert(sizeof(ShBars) <= 768, "barrier block");

// Ring positions, relative to the item's first slot, of K_i and V_i of m blocks.
__device__ __forceinline__ uint32_t sh_pos_k(int i) { return i == 0 ? 0u : 2u * i - 1u; }
__device__ __forceinline__ uint32_t sh_pos_v(int i, int m) { return i == m - 1 ? 2u * m - 1u : 2u * i + 2u; }

__device__ __forceinline__ uint32_t sh_parity(uint32_t bits, uint32_t st) { return (bits >> st) & 1u; }

// Warp 19 claims items and works them out when the producer is about to be done with the one before, so that no
// load waits for it and CTAs take items as they free up (claimed as the one before begins, the CTAs that
// have the longest items take the next longest as well: 64 requests behind 32K keys 105 -> 127 us).  The first
// one is the block's own where `ctas` blocks begin with this half of the list, all others (with 0: all) come off a
// counter.
// kKind: which of the list's two halves.
template <int kKind, int kSlots, typename Bars>
__device__ void sh_scheduler(const SharedParams& p, Bars* bars, const Watchdog& wd, int ctas, int lane) {
    const int first = kKind ? __ldcg(&p.header->n_items[0]) : 0, n_items = __ldcg(&p.header->n_items[kKind]);
    uint32_t kv = 0, vpar = 0;
    for (uint32_t r = 0;; ++r) {
        const uint32_t slot = r % kShRing;
        bool ok = r < kShRing || wd.wait(&bars->idx_empty[slot], ((r / kShRing) - 1) & 1);
        if (r >= 1) ok = ok && wd.wait(&bars->near_end, (r - 1) & 1);
        if (!__all_sync(0xffffffffu, ok)) return;
        int idx = blockIdx.x;
        if (r > 0 || ctas == 0) {
            if (lane == 0) idx = ctas + atomicAdd(&p.header->next_item[kKind], 1);
            idx = __shfl_sync(0xffffffffu, idx, 0);
        }
        ShItem it = {};
        if (idx < n_items) {
            const int2 w = __ldcg(p.items + first + idx);
            const SharedUnit u = sh_unit(p, w.x);
            const int piece = w.y >> 16;
            // (the first nblk % pieces of them have a block more)
            const int len = u.nblk / u.pieces, more = u.nblk - len * u.pieces;
            it.q0 = u.q0;
            it.ntok = u.ntok;
            it.kvh = w.y & 0xffff;
            it.row = u.row;
            it.key_min = u.key_min;
            it.key_end = u.key_end;
            it.pos0 = u.pos0;
            it.jlo = u.blk0 + piece * len + min(piece, more);
            it.jhi = it.jlo + len + (piece < more ? 1 : 0);
            it.part = u.part + (it.kvh * u.pieces + piece) * u.split * u.rows;
            it.kv0 = kv;
            it.vpar = vpar;
        }
        if (lane == 0) {
            bars->ring[slot] = it;
            mbar_arrive(&bars->idx_full[slot]);  // release: the item is visible to the readers
        }
        if (it.ntok == 0) return;
        if (kKind == 0) {
            const int m = it.jhi - it.jlo;
            uint32_t mine = 0;
            for (int i = lane; i < m; i += 32) mine ^= 1u << ((kv + sh_pos_v(i, m)) % kSlots);
            vpar ^= __reduce_xor_sync(0xffffffffu, mine);
            kv += 2 * m;
        }
    }
}

template <typename Bars>
__device__ __forceinline__ bool sh_take(Bars* bars, const Watchdog& wd, uint32_t& r, ShItem& it) {
    const uint32_t slot = r % kShRing;
    if (!wd.wait(&bars->idx_full[slot], (r / kShRing) & 1)) return false;
    it = bars->ring[slot];
    mbar_arrive(&bars->idx_empty[slot]);
    ++r;
    return it.ntok > 0;
}

template <typename Bars>
__device__ __forceinline__ bool sh_take_warp(Bars* bars, const Watchdog& wd, uint32_t& r, ShItem& it, int lane) {
    const uint32_t slot = r % kShRing;
    if (!__all_sync(0xffffffffu, wd.wait(&bars->idx_full[slot], (r / kShRing) & 1))) return false;
    it = bars->ring[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->idx_empty[slot]);
    ++r;
    return it.ntok > 0;
}

// Wait, ignoring the abort flag, for a phase that TMA or the tensor core still owes this CTA.
__device__ void sh_drain(uint64_t* bar, uint32_t parity) {
    const unsigned long long t0 = global_ns();
    while (!mbar_try(bar, parity)) {
        if (global_ns() - t0 > 200000000ull) return;
    }
}

struct ShRingState {
    uint32_t n = 0, kpar = 0, vpar = 0, lastv = 0;
};

// The whole warp: lane i looks up piece i of a block in the table and loads it.
template <int D>
__device__ void sh_producer_loop(const SharedParams& p, uint8_t* smem, ShBars* bars, const Watchdog& wd,
                                 uint32_t& q_cnt, ShRingState& ring, int lane) {
    using C = ShCfg<D>;
    if (lane == 0) {
        tma_prefetch_desc(&p.tm_q);
        tma_prefetch_desc(&p.tm_q1);
        tma_prefetch_desc(&p.tm_k);
        tma_prefetch_desc(&p.tm_v);
    }
    const int boxes = kFwdBlockN / p.box_rows;
    const int oob_row = p.num_pages * p.page_size;
    uint32_t rd = 0;
    ShItem it;
    while (sh_take_warp(bars, wd, rd, it, lane)) {
        if (!__all_sync(0xffffffffu, q_cnt == 0 || wd.wait(&bars->q_empty, (q_cnt - 1) & 1))) return;
        if (lane == 0) {
            uint32_t bytes = 0;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int tokens = it.ntok - t * p.tpt;
                if (tokens > 0) bytes += 128u * p.g * (tokens == 1 ? 1 : p.tpt) * C::kHalves;
            }
            mbar_arrive_expect_tx(&bars->q_full, bytes);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int tokens = it.ntok - t * p.tpt;
                if (tokens <= 0) continue;
#pragma unroll
                for (int h = 0; h < C::kHalves; ++h)
                    tma_load_3d(smem + C::kOffQ + t * C::kQTile + h * C::kAtomBytes, tokens == 1 ? &p.tm_q1 : &p.tm_q,
                                &bars->q_full, h * 64, it.kvh * p.g, it.q0 + t * p.tpt);
            }
        }
        ++q_cnt;
        const int m = it.jhi - it.jlo;
        const int* bt = p.block_table + static_cast<size_t>(it.row) * p.max_pages;
        // The cache's row of this lane's box of block i.  Boxes without a key of this unit (whose table entries
        // are not read) and boxes of a bad page are aimed past the end of the cache: TMA fills them with zeros.
        const auto box_row = [&](int i) {
            int row = oob_row;
            if (lane < boxes) {
                const int key = (it.jlo + i) * kFwdBlockN + lane * p.box_rows;
                if (key < it.key_end && key + p.box_rows > it.key_min) {
                    const int page = bt[key / p.page_size];
                    if (page >= 0 && page < p.num_pages)
                        row = page * p.page_size + key % p.page_size;
                    else
                        atomicOr(p.status, kStatusBounds);
                }
            }
            return row;
        };
        for (int r = 0; r < 2 * m; ++r) {
            // inverse of sh_pos_k / sh_pos_v
            const bool last = r == 2 * m - 1;
            const bool is_v = last || (r > 0 && (r & 1) == 0);
            const int i = is_v ? (last ? m - 1 : (r - 2) / 2) : (r + 1) / 2;
            const int row = box_row(i);
            if (r == max(0, 2 * m - 6) && lane == 0) mbar_arrive(&bars->near_end);
            const uint32_t n = ring.n, st = n % C::kSlots;
            if (!__all_sync(0xffffffffu, n < C::kSlots || wd.wait(&bars->kv_empty[st], ((n / C::kSlots) - 1) & 1)))
                return;
            uint64_t* const full = is_v ? &bars->v_full[st] : &bars->k_full[st];
            if (lane == 0) mbar_arrive_expect_tx(full, C::kKvTile);
            __syncwarp();
            ++ring.n;
            if (is_v) {
                ring.vpar ^= 1u << st;
                ring.lastv |= 1u << st;
            } else {
                ring.kpar ^= 1u << st;
                ring.lastv &= ~(1u << st);
            }
            if (lane < boxes) {
                uint8_t* const dst = smem + C::kOffKV + st * C::kKvTile + lane * p.box_rows * 128;
#pragma unroll
                for (int h = 0; h < C::kHalves; ++h)
                    tma_load_3d(dst + h * C::kAtomBytes, is_v ? &p.tm_v : &p.tm_k, full, h * 64, it.kvh, row);
            }
        }
    }
}

template <int D>
__device__ void sh_producer(const SharedParams& p, uint8_t* smem, ShBars* bars, const Watchdog& wd, int lane) {
    using C = ShCfg<D>;
    uint32_t q_cnt = 0;
    ShRingState ring;
    sh_producer_loop<D>(p, smem, bars, wd, q_cnt, ring, lane);
    __syncwarp();
    // what is in flight lands before the CTA's shared memory goes
    if (q_cnt > 0) sh_drain(&bars->q_full, (q_cnt - 1) & 1);
    for (uint32_t st = 0; st < C::kSlots && st < ring.n; ++st) {
        const bool v = sh_parity(ring.lastv, st) != 0;
        sh_drain(v ? &bars->v_full[st] : &bars->k_full[st], sh_parity(v ? ring.vpar : ring.kpar, st) ^ 1u);
    }
}

template <int D>
__device__ void sh_mma_s(const SharedParams& p, uint8_t* smem, ShBars* bars, uint32_t tmem, const Watchdog& wd) {
    using C = ShCfg<D>;
    constexpr uint32_t kIdesc = idesc_bf16_f32(128, kFwdBlockN, false, false);
    const uint64_t dq = sdesc_sw128(smem_u32(smem + C::kOffQ), 16, 1024);
    const uint64_t dkv = sdesc_sw128(smem_u32(smem + C::kOffKV), 16, 1024);
    const uint32_t q_lo = static_cast<uint32_t>(dq), d_hi = static_cast<uint32_t>(dq >> 32);
    const uint32_t kv_lo = static_cast<uint32_t>(dkv);
    uint32_t q_cnt = 0, kpar = 0, rd = 0;
    uint32_t s_cnt[2] = {0, 0};
    ShItem it;
    while (sh_take(bars, wd, rd, it)) {
        if (!wd.wait(&bars->q_full, q_cnt & 1)) return;
        ++q_cnt;
        const int m = it.jhi - it.jlo;
        const bool two = it.ntok > p.tpt;
        for (int i = 0; i < m; ++i) {
            const uint32_t st = (it.kv0 + sh_pos_k(i)) % C::kSlots;
            if (!wd.wait(&bars->k_full[st], sh_parity(kpar, st))) return;
            kpar ^= 1u << st;
            const uint32_t k_lo = kv_lo + st * (C::kKvTile >> 4);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (t == 1 && !two) continue;
                if (s_cnt[t] > 0 && !wd.wait(&bars->s_free[t], (s_cnt[t] - 1) & 1)) return;
                tc_fence_after();
                const uint32_t a_lo = q_lo + t * (C::kQTile >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * C::kAtomBytes + (kk & 3) * 32) >> 4;
                    umma_ss_lh(tmem + C::col_s(t), a_lo + off, d_hi, k_lo + off, d_hi, kIdesc, kk > 0);
                }
                umma_commit(&bars->s_full[t]);
                ++s_cnt[t];
            }
            umma_commit(&bars->kv_empty[st]);
        }
        umma_commit(&bars->q_empty);
    }
}

template <int D>
__device__ void sh_mma_pv(const SharedParams& p, uint8_t* smem, ShBars* bars, uint32_t tmem, const Watchdog& wd) {
    using C = ShCfg<D>;
    constexpr uint32_t kIdesc = idesc_bf16_f32(128, D, false, true);
    const uint64_t dp = sdesc_sw128(smem_u32(smem + C::kOffP), 16, 1024);
    const uint64_t dv = sdesc_sw128(smem_u32(smem + C::kOffKV), C::kAtomBytes, 1024);
    const uint32_t p_lo = static_cast<uint32_t>(dp), p_hi = static_cast<uint32_t>(dp >> 32);
    const uint32_t v_lo = static_cast<uint32_t>(dv), v_hi = static_cast<uint32_t>(dv >> 32);
    uint32_t vpar = 0, rd = 0;
    uint32_t pv_cnt[2] = {0, 0}, o_items[2] = {0, 0};
    ShItem it;
    while (sh_take(bars, wd, rd, it)) {
        const int m = it.jhi - it.jlo;
        const bool two = it.ntok > p.tpt;
        for (int i = 0; i < m; ++i) {
            const uint32_t st = (it.kv0 + sh_pos_v(i, m)) % C::kSlots;
            if (!wd.wait(&bars->v_full[st], sh_parity(vpar, st))) return;
            vpar ^= 1u << st;
            const uint32_t b_lo = v_lo + st * (C::kKvTile >> 4);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (t == 1 && !two) continue;
                if (i == 0 && o_items[t] > 0 && !wd.wait(&bars->o_free[t], (o_items[t] - 1) & 1)) return;
                if (!wd.wait(&bars->p_full[t], pv_cnt[t] & 1)) return;
                tc_fence_after();
                const uint32_t a_lo = p_lo + t * (C::kPTile >> 4);
#pragma unroll
                for (int kk = 0; kk < kFwdBlockN / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * C::kAtomBytes + (kk & 3) * 32) >> 4;
                    umma_ss_lh(tmem + C::col_o(t), a_lo + off, p_hi, b_lo + kk * (16 * 128 >> 4), v_hi, kIdesc,
                               (i == 0 && kk == 0) ? 0u : 1u);
                }
                umma_commit(&bars->pv_done[t]);
                ++pv_cnt[t];
            }
            umma_commit(&bars->kv_empty[st]);
        }
        ++o_items[0];
        if (two) ++o_items[1];
    }
}

// Softmax of tile t, rows 32 (k % 4) + 16 (k / 4) + [0, 16) of it by warp k, in the layout of an MMA's
// accumulator fragment: thread i holds rows i / 4 and i / 4 + 8, two columns of each 8.
template <int D>
__device__ void sh_softmax(const SharedParams& p, uint8_t* smem, ShBars* bars, uint32_t tmem, const Watchdog& wd,
                           int t, int k, int lane) {
    using C = ShCfg<D>;
    uint64_t* const s_full = &bars->s_full[t];
    uint64_t* const s_free = &bars->s_free[t];
    uint64_t* const p_full = &bars->p_full[t];
    uint64_t* const pv_done = &bars->pv_done[t];
    uint64_t* const o_free = &bars->o_free[t];
    const int rbase = 32 * (k & 3) + 16 * (k >> 2);
    const int ra = rbase + (lane >> 2);
    const int cpair = 2 * (lane & 3);
    const uint32_t tS = tmem + (static_cast<uint32_t>(rbase) << 16) + C::col_s(t);
    const uint32_t tO = tmem + (static_cast<uint32_t>(rbase) << 16) + C::col_o(t);
    const uint32_t p_tile = smem_u32(smem + C::kOffP + t * C::kPTile);
    // stmatrix: this thread addresses row lane % 8 of matrix lane / 8 (see fwd_kernel.cu)
    const int st_row = rbase + 8 * ((lane >> 3) & 1) + (lane & 7);
    const int st_dc = lane >> 4;
    uint32_t st_addr[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) st_addr[c] = p_tile + st_row * 128 + ((((2 * c + st_dc) ^ lane) & 7) << 4);
    const float sl2 = p.scale_log2;
    const uint64_t sl2x2 = f2_make(sl2, sl2);
    const int g = p.g;
    uint32_t blk = 0, rd = 0;
    ShItem it;
    while (sh_take_warp(bars, wd, rd, it, lane)) {
        const int m = it.jhi - it.jlo;
        const int tokens = min(p.tpt, it.ntok - t * p.tpt);
        if (tokens <= 0) continue;
        const int rows = tokens * g;
        const bool busy = rbase < rows;  // a row of this warp holds a token
        // keys [key_min, kmax] of rows ra and ra + 8
        const int tok0 = t * p.tpt;
        const int kmax_a = min(it.key_end - 1, it.pos0 + tok0 + ra / g);
        const int kmax_b = min(it.key_end - 1, it.pos0 + tok0 + (ra + 8) / g);
        const int kmax_first = min(it.key_end - 1, it.pos0 + tok0);
        float m_a = -INFINITY, m_b = -INFINITY, l_a = 0.f, l_b = 0.f;
        for (int j = it.jlo; j < it.jhi; ++j) {
            if (!__all_sync(0xffffffffu, wd.wait(s_full, blk & 1))) return;
            uint32_t pka[16], pkb[16];
            bool moves = false;
            float alpha_a = 1.f, alpha_b = 1.f;
            if (busy) {
                tc_fence_after();
                uint32_t s[64];
                tmem_ld16x256_x8(tS, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
                tmem_ld16x256_x8(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_free);
                if (j * kFwdBlockN < it.key_min || (j + 1) * kFwdBlockN - 1 > kmax_first) {
                    const int key0 = j * kFwdBlockN + cpair;
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int key = key0 + 8 * c + e;
                            if (key < it.key_min || key > kmax_a) s[4 * c + e] = __float_as_uint(-INFINITY);
                            if (key < it.key_min || key > kmax_b) s[4 * c + 2 + e] = __float_as_uint(-INFINITY);
                        }
                    }
                }
                float xa0 = fmaxf(__uint_as_float(s[0]), __uint_as_float(s[4]));
                float xa1 = fmaxf(__uint_as_float(s[1]), __uint_as_float(s[5]));
                float xb0 = fmaxf(__uint_as_float(s[2]), __uint_as_float(s[6]));
                float xb1 = fmaxf(__uint_as_float(s[3]), __uint_as_float(s[7]));
#pragma unroll
                for (int c = 2; c < 16; c += 2) {
                    xa0 = fmax3(xa0, __uint_as_float(s[4 * c]), __uint_as_float(s[4 * c + 4]));
                    xa1 = fmax3(xa1, __uint_as_float(s[4 * c + 1]), __uint_as_float(s[4 * c + 5]));
                    xb0 = fmax3(xb0, __uint_as_float(s[4 * c + 2]), __uint_as_float(s[4 * c + 6]));
                    xb1 = fmax3(xb1, __uint_as_float(s[4 * c + 3]), __uint_as_float(s[4 * c + 7]));
                }
                float mba = fmaxf(xa0, xa1) * sl2, mbb = fmaxf(xb0, xb1) * sl2;
                moves = __any_sync(0xffffffffu, mba > m_a + kShRescale || mbb > m_b + kShRescale);
                if (moves) {  // (a row's maximum is its quad's)
                    mba = fmaxf(mba, __shfl_xor_sync(0xffffffffu, mba, 1));
                    mbb = fmaxf(mbb, __shfl_xor_sync(0xffffffffu, mbb, 1));
                    mba = fmaxf(mba, __shfl_xor_sync(0xffffffffu, mba, 2));
                    mbb = fmaxf(mbb, __shfl_xor_sync(0xffffffffu, mbb, 2));
                    const float mna = mba > m_a + kShRescale ? mba : m_a, mnb = mbb > m_b + kShRescale ? mbb : m_b;
                    alpha_a = mna > m_a ? ex2_approx(m_a - mna) : 1.f;
                    alpha_b = mnb > m_b ? ex2_approx(m_b - mnb) : 1.f;
                    l_a *= alpha_a;
                    l_b *= alpha_b;
                    m_a = mna;
                    m_b = mnb;
                }
                const float na = m_a == -INFINITY ? 0.f : -m_a, nb = m_b == -INFINITY ? 0.f : -m_b;
                const uint64_t nma = f2_make(na, na), nmb = f2_make(nb, nb);
                uint64_t suma = 0, sumb = 0;
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    float a0, a1, b0, b1;
                    f2_split(f2_fma(f2_make(__uint_as_float(s[4 * c]), __uint_as_float(s[4 * c + 1])), sl2x2, nma), a0, a1);
                    f2_split(f2_fma(f2_make(__uint_as_float(s[4 * c + 2]), __uint_as_float(s[4 * c + 3])), sl2x2, nmb), b0, b1);
                    const float pa0 = ex2_approx(a0), pa1 = ex2_approx(a1);
                    const float pb0 = ex2_approx(b0), pb1 = ex2_approx(b1);
                    suma = f2_add(suma, f2_make(pa0, pa1));
                    sumb = f2_add(sumb, f2_make(pb0, pb1));
                    pka[c] = pack_bf16x2(pa0, pa1);  // (operands of the product, at most 2^8; l sums them unrounded)
                    pkb[c] = pack_bf16x2(pb0, pb1);
                }
                float lo, hi;
                f2_split(suma, lo, hi);
                l_a += lo + hi;
                f2_split(sumb, lo, hi);
                l_b += lo + hi;
            } else if (lane == 0) {
                mbar_arrive(s_free);
            }
            // Slots outside [key_min, key_end) may hold anything, and 0 times a NaN would reach O: this
            // tile's warps clear those rows of V.
            const int lo_key = max(it.key_min - j * kFwdBlockN, 0);
            const int hi_key = min(it.key_end - j * kFwdBlockN, kFwdBlockN);
            if (lo_key > 0 || hi_key < kFwdBlockN) {
                uint32_t bits = it.vpar;  // V parities before V_j's load
                for (int i = 0; i < j - it.jlo; ++i) bits ^= 1u << ((it.kv0 + sh_pos_v(i, m)) % C::kSlots);
                const uint32_t st = (it.kv0 + sh_pos_v(j - it.jlo, m)) % C::kSlots;
                if (!__all_sync(0xffffffffu, wd.wait(&bars->v_full[st], sh_parity(bits, st)))) return;
                const uint32_t vslot = smem_u32(smem + C::kOffKV + st * C::kKvTile);
                const int clear = lo_key + kFwdBlockN - hi_key;
                for (int u = k * 32 + lane; u < clear * C::kHalves * 8; u += 8 * 32) {
                    int r = u / (C::kHalves * 8);
                    const int hc = u % (C::kHalves * 8);
                    if (r >= lo_key) r += hi_key - lo_key;
                    st_shared_v4(vslot + (hc >> 3) * C::kAtomBytes + r * 128 + (hc & 7) * 16, 0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
            }
            // the product before this one has read P_t and added to O_t
            if (blk > 0) {
                if (!__all_sync(0xffffffffu, wd.wait(pv_done, (blk - 1) & 1))) return;
                tc_fence_after();
            }
            if (busy) {
                if (moves && j > it.jlo) {
#pragma unroll 1
                    for (int cc = 0; cc < D / 32; ++cc) {
                        uint32_t o[16];
                        tmem_ld16x256_x4(tO + 32 * cc, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            o[4 * c] = __float_as_uint(__uint_as_float(o[4 * c]) * alpha_a);
                            o[4 * c + 1] = __float_as_uint(__uint_as_float(o[4 * c + 1]) * alpha_a);
                            o[4 * c + 2] = __float_as_uint(__uint_as_float(o[4 * c + 2]) * alpha_b);
                            o[4 * c + 3] = __float_as_uint(__uint_as_float(o[4 * c + 3]) * alpha_b);
                        }
                        tmem_st16x256_x4(tO + 32 * cc, o);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                }
#pragma unroll
                for (int cp = 0; cp < 8; ++cp)
                    stmatrix_x4(st_addr[cp & 3] + (cp >> 2) * C::kAtomBytes, pka[2 * cp], pkb[2 * cp], pka[2 * cp + 1],
                                pkb[2 * cp + 1]);
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full);
            ++blk;
        }
        // ---- the rows' parts ----
        if (!__all_sync(0xffffffffu, wd.wait(pv_done, (blk - 1) & 1))) return;
        if (busy) {
            tc_fence_after();
            l_a += __shfl_xor_sync(0xffffffffu, l_a, 1);
            l_b += __shfl_xor_sync(0xffffffffu, l_b, 1);
            l_a += __shfl_xor_sync(0xffffffffu, l_a, 2);
            l_b += __shfl_xor_sync(0xffffffffu, l_b, 2);
            const float inv_a = l_a != 0.f ? 1.f / l_a : 0.f, inv_b = l_b != 0.f ? 1.f / l_b : 0.f;
            const int part_a = it.part + tok0 * g + ra, part_b = part_a + 8;
            const bool on_a = ra < rows && ATTN_IN_BOUNDS(part_a < p.max_parts, p.status);
            const bool on_b = ra + 8 < rows && ATTN_IN_BOUNDS(part_b < p.max_parts, p.status);
            float* const to_a = p.part_o + static_cast<size_t>(part_a) * D + cpair;
            float* const to_b = p.part_o + static_cast<size_t>(part_b) * D + cpair;
#pragma unroll
            for (int cc = 0; cc < D / 64; ++cc) {
                uint32_t o[32];
                tmem_ld16x256_x8(tO + 64 * cc, o);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    if (on_a)
                        *reinterpret_cast<float2*>(to_a + 64 * cc + 8 * c) =
                            make_float2(__uint_as_float(o[4 * c]) * inv_a, __uint_as_float(o[4 * c + 1]) * inv_a);
                    if (on_b)
                        *reinterpret_cast<float2*>(to_b + 64 * cc + 8 * c) =
                            make_float2(__uint_as_float(o[4 * c + 2]) * inv_b, __uint_as_float(o[4 * c + 3]) * inv_b);
                }
            }
            if ((lane & 3) == 0) {
                if (on_a) p.part_lse[part_a] = l_a != 0.f ? m_a + __log2f(l_a) : -INFINITY;
                if (on_b) p.part_lse[part_b] = l_b != 0.f ? m_b + __log2f(l_b) : -INFINITY;
            }
            tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(o_free);
    }
}

// ---- few rows -------------------------------------------------------------------------------------------
//
// Units of up to 16 rows (a sequence's single query, a few sequences' behind a prefix) would fill an eighth of a
// tile, and one warp's softmax over it, 3000 clocks a block, would be slower than the memory.  As in
// decode_kernel.cu four warps take 16 keys each of a chunk of 64, on mma.sync m16n8k16, twice an SM.
// The warps never meet: each leaves a part of its own.

template <int D>
struct SmCfg {
    static constexpr int kChunk = 64;
    static constexpr int kHalves = D / 64;
    static constexpr int kHalfBytes = kChunk * 128;
    static constexpr int kKvBytes = kHalves * kHalfBytes;
    static constexpr int kStageBytes = 2 * kKvBytes;
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kOffBar = kStages * kStageBytes;
    static constexpr int kSmem = kOffBar + 512 + 1024;
    static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs per SM");
};

constexpr int kSmThreads = 192;  // 4 MMA warps, the producer and the scheduler
constexpr uint32_t kSmReaders = 5;

struct SmBars {
    uint64_t full[6], empty[6];
    uint64_t idx_full[kShRing], idx_empty[kShRing];
    uint64_t near_end;
    ShItem ring[kShRing];
    int abort_flag;
};
static_assert(sizeof(SmBars) <= 512, "barrier block");

// The 64-key chunks of an item.
__device__ __forceinline__ int sm_first(const ShItem& it) { return max(2 * it.jlo, it.key_min / 64); }
__device__ __forceinline__ int sm_last(const ShItem& it) { return min(2 * it.jhi, ceil_div(it.key_end, 64)); }

template <int D>
__device__ void sm_producer(const SharedParams& p, uint8_t* smem, SmBars* bars, const Watchdog& wd, int lane) {
    using C = SmCfg<D>;
    const int box = min(p.box_rows, C::kChunk), boxes = C::kChunk / box;
    const int oob_row = p.num_pages * p.page_size;
    uint32_t issued = 0, rd = 0;
    bool ok = true;
    ShItem it;
    while (ok && sh_take_warp(bars, wd, rd, it, lane)) {
        const int* bt = p.block_table + static_cast<size_t>(it.row) * p.max_pages;
        const int c0 = sm_first(it), c1 = sm_last(it);
        for (int c = c0; c < c1; ++c, ++issued) {
            if (c == max(c0, c1 - 3) && lane == 0) mbar_arrive(&bars->near_end);
            // lane i: box i of the chunk (see sh_producer_loop)
            int row = oob_row;
            if (lane < boxes) {
                const int key = c * C::kChunk + lane * box;
                if (key < it.key_end && key + box > it.key_min) {
                    const int page = bt[key / p.page_size];
                    if (page >= 0 && page < p.num_pages)
                        row = page * p.page_size + key % p.page_size;
                    else
                        atomicOr(p.status, kStatusBounds);
                }
            }
            const uint32_t st = issued % C::kStages;
            ok = __all_sync(0xffffffffu, issued < C::kStages ||
                                             wd.wait(&bars->empty[st], ((issued / C::kStages) - 1) & 1));
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&bars->full[st], C::kStageBytes);
            __syncwarp();
            if (lane < boxes) {
                uint8_t* const dst = smem + st * C::kStageBytes + lane * box * 128;
#pragma unroll
                for (int h = 0; h < C::kHalves; ++h) {
                    tma_load_3d(dst + h * C::kHalfBytes, &p.tm_k64, &bars->full[st], h * 64, it.kvh, row);
                    tma_load_3d(dst + C::kKvBytes + h * C::kHalfBytes, &p.tm_v64, &bars->full[st], h * 64, it.kvh, row);
                }
            }
        }
    }
    __syncwarp();
    // what is in flight lands before the CTA's shared memory goes
    const uint32_t n_st = min(issued, static_cast<uint32_t>(C::kStages));
    for (uint32_t st = 0; st < n_st; ++st) {
        const uint32_t last = st + C::kStages * ((issued - 1 - st) / C::kStages);
        sh_drain(&bars->full[st], (last / C::kStages) & 1);
    }
}

__device__ __forceinline__ uint32_t sm_swz(int row, int oct) {
    return static_cast<uint32_t>(row * 128 + ((oct ^ (row & 7)) << 4));
}

// Warp w has keys [16 w, 16 w + 16) of every chunk.
template <int D>
__device__ void sm_consumer(const SharedParams& p, uint8_t* smem, SmBars* bars, const Watchdog& wd, int warp,
                            int lane) {
    using C = SmCfg<D>;
    const int gq = lane >> 2, tq = lane & 3;
    const int mi = lane >> 3, ri = lane & 7;  // ldmatrix: matrix id, row within matrix
    const float sl2 = p.scale_log2;
    uint32_t n = 0, rd = 0;
    ShItem it;
    while (sh_take_warp(bars, wd, rd, it, lane)) {
        const int rows = it.ntok * p.g;
        // rows gq and gq + 8: tokens, the last keys that they see, queries as the A operand
        int kmax[2];
        uint32_t qa[D / 16][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = gq + 8 * h, tok = r / p.g;
            const bool on = r < rows;
            kmax[h] = min(it.key_end - 1, it.pos0 + tok);
            const __nv_bfloat16* src =
                p.q + (static_cast<size_t>(it.q0 + (on ? tok : 0)) * p.Hq + it.kvh * p.g + (on ? r - tok * p.g : 0)) * D;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t* x = reinterpret_cast<const uint32_t*>(src + kk * 16 + 2 * tq);
                qa[kk][h] = on ? x[0] : 0u;
                qa[kk][2 + h] = on ? x[4] : 0u;
            }
        }
        const int kmax_first = min(it.key_end - 1, it.pos0);
        float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
        float o[D / 8][4];
#pragma unroll
        for (int x = 0; x < D / 8; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.f;
        const int c1 = sm_last(it);
        for (int c = sm_first(it); c < c1; ++c, ++n) {
            const uint32_t st = n % C::kStages;
            if (!__all_sync(0xffffffffu, wd.wait(&bars->full[st], (n / C::kStages) & 1))) return;
            uint8_t* const kst = smem + st * C::kStageBytes;
            uint8_t* const vst = kst + C::kKvBytes;
            const int key0 = c * C::kChunk + warp * 16;
            const int lo = max(it.key_min - key0, 0), hi = min(it.key_end - key0, 16);
            if (lo < hi) {
                if (lo > 0 || hi < 16) {
                    // slots outside [key_min, key_end) may hold anything, and 0 times a NaN would reach O
                    for (int i = lane; i < 16 * C::kHalves * 8; i += 32) {
                        const int r = i / (C::kHalves * 8), rest = i % (C::kHalves * 8);
                        if (r < lo || r >= hi)
                            *reinterpret_cast<uint4*>(vst + (rest / 8) * C::kHalfBytes + (warp * 16 + r) * 128 +
                                                      (rest % 8) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
                const uint32_t kbase = smem_u32(kst);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const int key = warp * 16 + (mi >> 1) * 8 + ri, oct = 2 * kk + (mi & 1);
                    uint32_t b0, b1, b2, b3;
                    ldmatrix_x4(kbase + (oct >> 3) * C::kHalfBytes + sm_swz(key, oct & 7), b0, b1, b2, b3);
                    mma_bf16_16816(s[0], qa[kk], b0, b1);
                    mma_bf16_16816(s[1], qa[kk], b2, b3);
                }
                if (lo > 0 || key0 + 15 > kmax_first) {
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = key0 + nt * 8 + 2 * tq + (e & 1);
                            if (key < it.key_min || key > kmax[e >> 1]) s[nt][e] = -INFINITY;
                        }
                }
                float mx[2];
                bool up = false;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    mx[r] = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1])) * sl2;
                    up = up || mx[r] > m_run[r] + kShRescale;
                }
                if (__any_sync(0xffffffffu, up)) {  // a row's reference moves (rarely behind the first chunks)
                    float alpha[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
                        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
                        const bool moves = mx[r] > m_run[r] + kShRescale;
                        alpha[r] = moves ? ex2_approx(m_run[r] - mx[r]) : 1.f;
                        if (moves) m_run[r] = mx[r];
                        l_run[r] *= alpha[r];
                    }
#pragma unroll
                    for (int x = 0; x < D / 8; ++x)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[x][e] *= alpha[e >> 1];
                }
                uint32_t pa[4];
                const float nm[2] = {m_run[0] == -INFINITY ? 0.f : -m_run[0], m_run[1] == -INFINITY ? 0.f : -m_run[1]};
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float p0 = ex2_approx(fmaf(s[nt][2 * r], sl2, nm[r]));
                        const float p1 = ex2_approx(fmaf(s[nt][2 * r + 1], sl2, nm[r]));
                        l_run[r] += p0 + p1;
                        pa[2 * nt + r] = pack_bf16x2(p0, p1);  // (as above: only the product's operand is rounded)
                    }
                const uint32_t vbase = smem_u32(vst);
#pragma unroll
                for (int x = 0; x < D / 8; x += 2) {
                    const int key = warp * 16 + (mi & 1) * 8 + ri, oct = x + (mi >> 1);
                    uint32_t b0, b1, b2, b3;
                    ldmatrix_x4_trans(vbase + (oct >> 3) * C::kHalfBytes + sm_swz(key, oct & 7), b0, b1, b2, b3);
                    mma_bf16_16816(o[x], pa, b0, b1);
                    mma_bf16_16816(o[x + 1], pa, b2, b3);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->empty[st]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float l = l_run[h];
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            const int r = gq + 8 * h, part = it.part + warp * rows + r;
            if (r >= rows || !ATTN_IN_BOUNDS(part < p.max_parts, p.status)) continue;
            const float inv = l != 0.f ? 1.f / l : 0.f;
            float* dst = p.part_o + static_cast<size_t>(part) * D + 2 * tq;
#pragma unroll
            for (int x = 0; x < D / 8; ++x)
                *reinterpret_cast<float2*>(dst + 8 * x) = make_float2(o[x][2 * h] * inv, o[x][2 * h + 1] * inv);
            if (tq == 0) p.part_lse[part] = l != 0.f ? m_run[h] + __log2f(l) : -INFINITY;
        }
    }
}

__device__ void sm_init(SmBars* bars) {
    for (int i = 0; i < 6; ++i) {
        mbar_init(&bars->full[i], 1);
        mbar_init(&bars->empty[i], 4);
    }
    for (uint32_t i = 0; i < kShRing; ++i) {
        mbar_init(&bars->idx_full[i], 1);
        mbar_init(&bars->idx_empty[i], kSmReaders);
    }
    mbar_init(&bars->near_end, 1);
    bars->abort_flag = 0;
}

// Where no unit can have many rows.
template <int D>
__global__ void __launch_bounds__(kSmThreads, 2) shared_small_kernel(const __grid_constant__ SharedParams p) {
    using C = SmCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    SmBars* bars = reinterpret_cast<SmBars*>(smem + C::kOffBar);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        sm_init(bars);
        mbar_fence_init();
        tma_prefetch_desc(&p.tm_k64);
        tma_prefetch_desc(&p.tm_v64);
    }
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    const Watchdog wd{&bars->abort_flag, p.status};
    if (warp < 4)
        sm_consumer<D>(p, smem, bars, wd, warp, lane);
    else if (warp == 4)
        sm_producer<D>(p, smem, bars, wd, lane);
    else
        sh_scheduler<1, 1>(p, bars, wd, gridDim.x, lane);
}

// ---- many rows, then few ----------------------------------------------------------------------------------

template <int D>
__global__ void __launch_bounds__(kFwdThreads, 1) shared_attn_kernel(const __grid_constant__ SharedParams p) {
    using C = ShCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    ShBars* bars = reinterpret_cast<ShBars*>(smem + C::kOffBar);
    SmBars* few = reinterpret_cast<SmBars*>(smem + C::kOffFew);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(&bars->q_full, 1);
        mbar_init(&bars->q_empty, 1);
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(&bars->k_full[i], 1);
            mbar_init(&bars->v_full[i], 1);
            mbar_init(&bars->kv_empty[i], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bars->s_full[t], 1);
            mbar_init(&bars->s_free[t], kShSoftmaxWarps / 2);
            mbar_init(&bars->p_full[t], kShSoftmaxWarps / 2);
            mbar_init(&bars->pv_done[t], 1);
            mbar_init(&bars->o_free[t], kShSoftmaxWarps / 2);
            mbar_init(&bars->drain[t], 1);
        }
        for (uint32_t i = 0; i < kShRing; ++i) {
            mbar_init(&bars->idx_full[i], 1);
            mbar_init(&bars->idx_empty[i], kShReaders);
        }
        mbar_init(&bars->near_end, 1);
        bars->abort_flag = 0;
        for (int v = 0; v < 2; ++v) sm_init(few + v);
        mbar_fence_init();
    }
    if (warp == kShSoftmaxWarps + 1) tmem_alloc(&bars->tmem_base, C::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    const Watchdog wd{&bars->abort_flag, p.status};
    griddep_wait();  // the list, and what stands before this call
    griddep_launch_dependents();  // (from here on the list may be read without waiting)
    const int ctas = min(__ldcg(&p.header->ctas), static_cast<int>(gridDim.x));
    const bool many = static_cast<int>(blockIdx.x) < ctas;
    // registers as in fwd_kernel.cu: 128 * 64 + 512 * 104 = 640 * 96
    if (warp >= kShSoftmaxWarps) {
        regs_decrease<64>();
        if (warp == kShSoftmaxWarps + 3) {
            if (many) sh_scheduler<0, C::kSlots>(p, bars, wd, ctas, lane);
            if (lane == 0)  // (read while the last item is done)
                bars->few_left = __ldcg(&p.header->next_item[1]) < __ldcg(&p.header->n_items[1]);
        } else if (!many) {
        } else if (warp == kShSoftmaxWarps) {
            sh_producer<D>(p, smem, bars, wd, lane);
        } else {
            if (lane == 0) {
                const int w = warp - kShSoftmaxWarps - 1;
                if (w == 0)
                    sh_mma_s<D>(p, smem, bars, tmem, wd);
                else
                    sh_mma_pv<D>(p, smem, bars, tmem, wd);
                umma_commit(&bars->drain[w]);
                sh_drain(&bars->drain[w], 0);
            }
        }
    } else {
        regs_increase<104>();
        if (many) sh_softmax<D>(p, smem, bars, tmem, wd, warp >> 3, warp & 7, lane);
    }
    __syncwarp();
    fence_proxy_async_smem();  // (what has been written here is loaded over below)
    tc_fence_before();
    __syncthreads();
    if (warp == kShSoftmaxWarps + 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
    if (bars->few_left == 0 || bars->abort_flag != 0) return;
    // The CTA becomes two of the other kind: warps 0-3 and 4-7 on mma.sync, 8 and 12 their producers, 9 and 13
    // their schedulers.  Registers: 256 * 168 + 384 * 48 = 640 * 96
    static_assert(2 * SmCfg<D>::kOffBar <= C::kOffBar && 2 * sizeof(SmBars) <= 1024, "both in one CTA's shared memory");
    const int v = warp < 8 ? warp >> 2 : (warp >> 2) & 1, w = warp & 3;
    uint8_t* const half = smem + v * SmCfg<D>::kOffBar;
    const Watchdog wd2{&few[v].abort_flag, p.status};
    if (warp < 8) {
        regs_increase<168>();
        sm_consumer<D>(p, half, few + v, wd2, w, lane);
    } else {
        regs_decrease<48>();
        if (warp >= kShSoftmaxWarps) return;
        if (w == 0)
            sm_producer<D>(p, half, few + v, wd2, lane);
        else if (w == 1)
            sh_scheduler<1, 1>(p, few + v, wd2, 0, lane);
    }
}

// ---- merge --------------------------------------------------------------------------------------------

// Two, four or eight warps have a row, eight parts each at a time, whose loads all go out together: block (i, h, j)
// has rows kRows j .. kRows j + kRows - 1 of sequence unit i for kv head h.  LSE = log2 sum_s 2^LSE_s,
// O = sum_s 2^(LSE_s - LSE) O_s over the parts of the row's prefix and of its own keys; no part, or none with
// a key: O = 0, LSE = -inf.
// Bound by the latency of the parts' loads, and by L2 where there are many: of a call's time 1 us with 32 rows, 3 with
// 1204, 5 with 2048 rows of 37 parts (38 MB); with a warp a row, three times eight parts one after the other, a us more.
template <int D, int kRows>
__global__ void __launch_bounds__(kShCombineThreads) shared_combine_kernel(const SharedParams p) {
    constexpr int E = D / 32, kWarps = kShCombineThreads / 32 / kRows, kBatch = 8;
    __shared__ float4 s_acc[kRows][kWarps][32];
    __shared__ float s_max[kRows][kWarps], s_sum[kRows][kWarps];
    // (the list is there when this kernel starts; the parts are when the one before it has ended)
    const int own = blockIdx.x, kvh = blockIdx.y, lane = threadIdx.x & 31;
    const int half = threadIdx.x / (32 * kWarps), w = (threadIdx.x >> 5) % kWarps, r = kRows * blockIdx.z + half;
    const SharedHeader* h = p.header;
    const bool listed = __ldcg(&h->bad) == 0 && own < __ldcg(&h->n_own);
    SharedUnit u = {};
    if (listed) u = sh_unit(p, p.own_base + own);
    const bool some = listed && kRows * blockIdx.z < u.rows;  // the same for the block
    const bool on = some && r < u.rows;
    int n1 = 0, n2 = 0, base1 = 0, base2 = 0, step1 = 0, step2 = 0, tok = 0;
    if (on) {
        tok = u.q0 + r / p.g;
        n1 = u.pieces * u.split;
        step1 = u.rows;
        base1 = u.part + kvh * n1 * step1 + r;
        if (u.prefix >= 0) {
            const SharedUnit v = sh_unit(p, u.prefix + (tok - u.group_q0) / (2 * p.tpt));
            n2 = v.pieces * v.split;
            step2 = v.rows;
            base2 = v.part + kvh * n2 * step2 + (tok - v.q0) * p.g + r % p.g;
        }
    }
    griddep_wait();
    if (!some) return;
    const int n = n1 + n2;
    float M = -INFINITY, sum = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    bool nan = false;
    for (int s0 = w * kBatch; s0 < n; s0 += kWarps * kBatch) {
        float x[kBatch], v[kBatch][E];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int s = min(s0 + i, n - 1);
            const int at = s < n2 ? base2 + s * step2 : base1 + (s - n2) * step1;
            x[i] = p.part_lse[at];
            const float* src = p.part_o + static_cast<size_t>(at) * D + lane * E;
            if constexpr (E == 4) {
                const float4 y = *reinterpret_cast<const float4*>(src);
                v[i][0] = y.x, v[i][1] = y.y, v[i][2] = y.z, v[i][3] = y.w;
            } else {
                const float2 y = *reinterpret_cast<const float2*>(src);
                v[i][0] = y.x, v[i][1] = y.y;
            }
        }
        float top = M;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (s0 + i >= n) x[i] = -INFINITY;
            nan = nan || x[i] != x[i];
            top = fmaxf(top, x[i]);
        }
        if (top == -INFINITY) continue;  // no keys so far
        const float keep = ex2_approx(M - top);
        M = top;
        sum *= keep;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= keep;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const float wi = ex2_approx(x[i] - M);
            sum += wi;
            if (s0 + i >= n) continue;  // (no part: not even times 0)
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(wi, v[i][e], acc[e]);
        }
    }
    if (nan) sum = __int_as_float(0x7fffffff);  // (the warps' parts are the same in all lanes)
    if (lane == 0) s_max[half][w] = M, s_sum[half][w] = sum;
    float4 mine = make_float4(acc[0], acc[1], 0.f, 0.f);
    if constexpr (E == 4) mine.z = acc[2], mine.w = acc[3];
    s_acc[half][w][lane] = mine;
    __syncthreads();
    if (w != 0 || !on) return;
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) top = fmaxf(top, s_max[half][i]);
    const float ref = top == -INFINITY ? 0.f : top;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        const float wi = ex2_approx(s_max[half][i] - ref);
        const float4 a = s_acc[half][i][lane];
        sum += wi * s_sum[half][i];
        o = make_float4(fmaf(wi, a.x, o.x), fmaf(wi, a.y, o.y), fmaf(wi, a.z, o.z), fmaf(wi, a.w, o.w));
    }
    const int head = kvh * p.g + r % p.g;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // (a NaN stays one)
    if (!ATTN_IN_BOUNDS(tok < p.total_q && head < p.Hq, p.status)) return;
    __nv_bfloat16* dst = p.out + (static_cast<size_t>(tok) * p.Hq + head) * D + lane * E;
    if constexpr (E == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    else
        *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(o.x * inv, o.y * inv);
    if (lane == 0)
        p.lse[static_cast<size_t>(head) * p.lse_head + static_cast<size_t>(tok) * p.lse_tok] =
            sum == 0.f ? -INFINITY : (ref + __log2f(sum)) * kShLn2;
}

template <typename Kernel>
cudaError_t launch_dependent(Kernel kernel, dim3 grid, int threads, size_t smem, const SharedParams& p,
                             cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t configure_shared_kernels() {
    const cudaFuncAttribute smem = cudaFuncAttributeMaxDynamicSharedMemorySize;
    cudaError_t e = cudaFuncSetAttribute(shared_attn_kernel<128>, smem, ShCfg<128>::kSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(shared_attn_kernel<64>, smem, ShCfg<64>::kSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(shared_small_kernel<128>, smem, SmCfg<128>::kSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(shared_small_kernel<64>, smem, SmCfg<64>::kSmem);
    return e;
}

namespace {

template <int D>
cudaError_t launch_shared_attn_d(const SharedParams& p, int num_sms, int own_units, cudaStream_t stream) {
    shared_units_kernel<<<1, kShUnitsThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = p.many ? launch_dependent(shared_attn_kernel<D>, dim3(num_sms), kFwdThreads, ShCfg<D>::kSmem, p, stream)
               : launch_dependent(shared_small_kernel<D>, dim3(2 * num_sms), kSmThreads, SmCfg<D>::kSmem, p, stream);
    if (e != cudaSuccess) return e;
    // a unit's rows, at most (max_seqlen_q may be 0, a grid not)
    const int rows = std::max(std::min(p.max_seqlen_q, 2 * p.tpt), 1) * p.g;
    const bool few = static_cast<long long>(p.total_q) * p.Hq <= kShFewRows;
    const bool most = static_cast<long long>(p.total_q) * p.Hq > kShMostRows;
    const int per = few ? 1 : most ? 4 : 2;
    return launch_dependent(few ? shared_combine_kernel<D, 1> : most ? shared_combine_kernel<D, 4> : shared_combine_kernel<D, 2>,
                            dim3(own_units, p.Hkv, ceil_div(rows, per)), kShCombineThreads, 0, p, stream);
}

}  // namespace

cudaError_t launch_shared_attn(const SharedParams& p, int head_dim, int num_sms, int own_units, cudaStream_t stream) {
    return head_dim == 128 ? launch_shared_attn_d<128>(p, num_sms, own_units, stream)
                           : launch_shared_attn_d<64>(p, num_sms, own_units, stream);
}

}  // namespace attn

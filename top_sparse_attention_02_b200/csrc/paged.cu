// paged.cu -- decode attention of one token per sequence over a paged cache:
// every row of each sequence, or the rows an index list names; optionally on top
// of partials that another pass made over a prefix all sequences share.
//
//   O = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale * <q_h, k_j> - m)
// as flash decoding: running maximum m and sum per head in fp32, one pass over
// the rows, the parts of a unit (sequence, kv-head) joined by
//   O = sum_i 2^(M_i - M) acc_i / sum_i 2^(M_i - M) L_i.
//
// A row is read once for g <= 16 query heads (at most 16 flop a byte), so HBM
// bounds it, and two things decide how near it comes: every SM streaming until
// the end, and enough bytes in flight.
//  - Even work whatever the lengths: the granules (64 rows) of all units, and one
//    empty slot after each unit (ending a unit takes about a granule's time), are
//    laid end to end and each CTA takes the same number of them, so a CTA may end
//    in the middle of one unit and begin in the middle of another.  The lengths
//    are on the device only; each warp adds them up itself.  A unit that lies in
//    one CTA is finished there; otherwise each CTA writes its piece, and a second
//    kernel joins the pieces of each row (with a shared prefix's partials, where
//    there is one), in the order of the CTAs, so that the result does not depend on
//    who was last.  (The last CTA of a unit to arrive, found by a counter, took 3.8 us
//    from its piece to O; a first form of the second kernel, which by then is resident, 3.5.)
//  - Each of a CTA's 4 warps streams its own 16 rows of every granule through
//    its own ring of 8 KB stages (K and V of 16 rows), so a warp never waits for
//    another one until the unit ends.  Two CTAs an SM.  Every row: two 2-D boxes
//    each of K and V (64 elements x 16 rows, 128-byte swizzle) by TMA; a page
//    holds a multiple of 16 rows, so a tile never crosses pages and any order of
//    heads and rows inside the page is a matter of the tensor map's strides.
//    Selected rows: cp.async, 16 bytes a lane, into the same swizzled layout.
//  - The products run on mma.sync with the 16 rows as M and the group's heads as
//    N (8, or 16 for groups above 8): S^T = K Q^T, O^T += V^T P^T.  P is kept as
//    two numbers of the element type (its rounding and the rest), so the weights
//    keep about 16 bits and the output's own rounding is the larger error; the
//    second product costs little in a kernel that waits for memory.
//
// Measured (graph replays): 64 sequences of 8192 to 32768 rows, 64/8 heads (5.18 GB) 805 us =
// 6.44 TB/s, HBM's rate; 17 ragged sequences, 40/8 heads, 139 MB 28.5 us = 4.9 TB/s; one
// sequence of 4096 rows, 2 kv-heads 8.3 us; 2621 selected rows of 8 kv-heads at 131072 (10.7 MB)
// 9.9 us.  The last two are a chain of waits: lengths 0.9 us, pages (or list, then pages) 1 to 2,
// rows 0.4, products and the warps' merge 1.5 (marks of SM time); the second kernel is the rest.
//
// Rows outside the sequence in a tile that is partly valid: their scores become
// -inf, and their V rows are overwritten with zeros in shared memory (0 * NaN in
// memory nobody wrote would be NaN).
#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "paged.cuh"
#include "tma.cuh"

namespace tsa {

constexpr int kPgWarps = 4;
constexpr int kPgThreads = kPgWarps * 32;
constexpr int kPgGranule = kPgWarps * kPageRows;   // rows
constexpr int kPgHalf = kPageRows * 128;           // 64 elements of 16 rows: 2 KB
constexpr int kPgStage = 4 * kPgHalf;              // K halves, V halves: 8 KB
constexpr int kPgCtasPerSm = 2;
constexpr int kPgCtas = kPgCtasPerSm * kPagedSms;  // the grid
constexpr int kPgPieces = 64;  // pieces of a unit that one round of loads joins (8 warps, 8 loads each)
constexpr int kPgEnd = 1;      // empty slots after a unit (17 ragged sequences: none 37.5 us, one 29.9, two 29.6; 400 short ones: 71, 58.5, 59.1)
constexpr int kPgLong = 8;     // granules a CTA above which more pieces pay
constexpr float kNegInf = -INFINITY;

#ifdef TSA_DEBUG_KNOBS
// Debug build only (never in the product library): the granule of CTA 0 whose load
// warp 0 leaves out, so that the wait on it runs out; -1: none.
__device__ int g_debug_paged_skip = -1;
#endif

template <int NT>
struct PgCfg {
    static constexpr int kStages = NT == 1 ? 3 : 2;
    static constexpr int kHeads = NT * 8;
    // all of it dynamic (1024-byte aligned): rings, merge buffer, barriers.
    // Two CTAs of 115,296 B (one n-tile) and their 1 KB each fit an SM's 228 KB.
    static constexpr int kMerge = kPgWarps * kStages * kPgStage;
    static constexpr int kBars = kMerge + kPgWarps * kHeads * kPartFloats * 4;
    static constexpr int kSmem = kBars + kPgWarps * kStages * 8;
};

int paged_ctas() { return kPgCtas; }

// n granules over nc CTAs: the first n % nc take one more
struct Shares {
    int n, nc, each, more;
    __device__ __forceinline__ Shares(int n_, int nc_) : n(n_), nc(nc_), each(0), more(0) {
        if (nc > 0) each = n / nc, more = n - each * nc;
    }
    __device__ __forceinline__ int start(int c) const { return c * each + min(c, more); }
    __device__ __forceinline__ int cta_of(int x) const {
        const int wide = more * (each + 1);
        return x < wide ? x / (each + 1) : more + (x - wide) / each;
    }
};

// Where a sequence's rows begin and end for this pass, in granules of 64 rows; a unit's
// slots are its granules and an empty one.
struct Span {
    int lo, hi;  // rows [lo, hi) (selected rows: entries of the list)
    __device__ __forceinline__ int first() const { return lo / kPgGranule; }
    __device__ __forceinline__ int granules() const { return hi > lo ? (hi + kPgGranule - 1) / kPgGranule - first() : 0; }
    __device__ __forceinline__ int slots() const { return hi > lo ? granules() + kPgEnd : 0; }
};

struct PgArgs {
    Pages c;
    const uint16_t* Q;
    int Hq, G;
    const int32_t *lens, *idx, *kreq;
    int k_max;
    float scale_log2;  // scale * log2(e)
    uint16_t* O;
    float* lse;
    float* pieces;       // [2 * gridDim.x][G][kPartFloats]
    PrefixParts pre;
    float* own;          // over a shared prefix: [B][Hq][kPartFloats], where this pass's partials go
    unsigned* flag;
};

template <bool GATHER>
__device__ __forceinline__ Span span_of(const PgArgs& a, int b, bool report) {
    int len = a.lens[b];
    const int cap = a.c.rows_cap();
    if (len < 0 || len > cap) {
        if (report) atomicOr(a.flag, kFlagBounds);
        len = len < 0 ? 0 : cap;
    }
    Span s;
    s.lo = 0;
    s.hi = len;
    if constexpr (GATHER) {
        int k = a.kreq ? a.kreq[b] : a.k_max;
        if (k < 0 || k > a.k_max) {
            if (report && (k < 0 || min(k, len) > a.k_max)) atomicOr(a.flag, kFlagBounds);
            k = k < 0 ? 0 : a.k_max;
        }
        s.hi = min(k, len);
    } else if (a.pre.splits > 0 && len >= a.pre.prefix_len) {
        s.lo = a.pre.prefix_len;
    }
    return s;
}

// The slots of the sequences b0 + 4 lane .. + 3 (all heads), and the shares of them all.
template <bool GATHER>
__device__ __forceinline__ void slots4(const PgArgs& a, int b0, int lane, bool report, int (&cnt)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int b = b0 + lane * 4 + k;
        cnt[k] = b < a.c.B ? span_of<GATHER>(a, b, report).slots() * a.c.Hkv : 0;
    }
}
// CTAs with work: few units are not spread over more CTAs than it takes to read them
// (joining a unit's pieces costs a round trip for each kPgPieces of them).
__device__ __forceinline__ Shares shares_of(const PgArgs& a, int total) {
    return Shares(total, (int)min((long long)min(kPgCtas, total),
                                  max((long long)a.c.B * a.c.Hkv * (kPgPieces + kPgEnd), (long long)total / kPgLong)));
}

// A row's result out of its sums acc (4 of 128 a lane), maximum M and weight L.
template <class E>
__device__ __forceinline__ void finish_row(const PgArgs& a, long long row, float4 acc, float M, float L, int lane) {
    const float inv = L == 0.f ? 0.f : 1.0f / L;
    uint2 o;
    o.x = E::pack(acc.x * inv, acc.y * inv);
    o.y = E::pack(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(a.O + row * kD + lane * 4) = o;
    if (a.lse && lane == 0) a.lse[row] = L == 0.f ? kNegInf : M + log2f(L);
}

// The same, or (over a shared prefix) one more partial of the row.
template <class E>
__device__ __forceinline__ void put_row(const PgArgs& a, long long row, float4 acc, float M, float L, int lane) {
    if (!a.own) {
        finish_row<E>(a, row, acc, M, L, lane);
        return;
    }
    float* p = a.own + row * kPartFloats;
    __stcg(reinterpret_cast<float4*>(p) + lane, acc);
    if (lane == 0) __stcg(reinterpret_cast<float2*>(p + kD), make_float2(M, L));
}

// The weights of n partials of one row, part(i) for i < n, each kPartFloats with its
// maximum and weight after the 128 sums: wts[i] = 2^(M_i - M), the joint maximum *M
// and weight *L.  All lanes of the warp.
template <class Part>
__device__ __forceinline__ void join_weights(int n, Part part, float* wts, int lane, float* M_out, float* L_out) {
    auto ml_of = [&](int i) { return __ldcg(reinterpret_cast<const float2*>(part(i) + kD)); };
    float2 ml0 = make_float2(kNegInf, 0.f), ml1 = ml0;  // the first 64 stay in registers
    if (lane < n) ml0 = ml_of(lane);
    if (lane + 32 < n) ml1 = ml_of(lane + 32);
    float M = fmaxf(ml0.y > 0.f ? ml0.x : kNegInf, ml1.y > 0.f ? ml1.x : kNegInf);
    for (int i = lane + 64; i < n; i += 32) {
        const float2 ml = ml_of(i);
        if (ml.y > 0.f) M = fmaxf(M, ml.x);
    }
#pragma unroll
    for (int m = 16; m; m >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, m));
    float L = 0.f;
    bool bad = false;  // a NaN weight: the result is NaN, as the softmax's is
    auto take = [&](int i, float2 ml) {
        const float w = ml.y > 0.f ? exp2f(ml.x - M) : 0.f;
        bad |= ml.y != ml.y;
        wts[i] = w;
        L += w * ml.y;
    };
    if (lane < n) take(lane, ml0);
    if (lane + 32 < n) take(lane + 32, ml1);
    for (int i = lane + 64; i < n; i += 32) take(i, ml_of(i));
#pragma unroll
    for (int m = 16; m; m >>= 1) L += __shfl_xor_sync(0xffffffffu, L, m);
    if (__any_sync(0xffffffffu, bad)) L = NAN;
    __syncwarp();
    *M_out = M;
    *L_out = L;
}

// This lane's 4 of the 128 sums over the partials i0, i0 + step, ... < n, with the
// weights that join_weights leaves in wts.  kJoinFlight loads are on their way at a
// time, the first of them before the weights are known (they come out of L2, at
// about a microsecond a round).
constexpr int kJoinFlight = 8;
template <class Part, class Weights>
__device__ __forceinline__ float4 join_sums(int n, int i0, int step, Part part, const float* wts, int lane, Weights weights) {
    float4 v[kJoinFlight], acc = make_float4(0.f, 0.f, 0.f, 0.f);
    bool first = true;
    for (int i = i0; i < n || first; i += kJoinFlight * step) {
#pragma unroll
        for (int k = 0; k < kJoinFlight; ++k)
            if (i + k * step < n) v[k] = __ldcg(reinterpret_cast<const float4*>(part(i + k * step)) + lane);
        if (first) weights();
        first = false;
#pragma unroll
        for (int k = 0; k < kJoinFlight; ++k) {
            const float w = i + k * step < n ? wts[i + k * step] : 0.f;
            if (w == 0.f) continue;  // (a part without a row may hold anything)
            acc.x = fmaf(w, v[k].x, acc.x), acc.y = fmaf(w, v[k].y, acc.y);
            acc.z = fmaf(w, v[k].z, acc.z), acc.w = fmaf(w, v[k].w, acc.w);
        }
    }
    return acc;
}

__device__ __forceinline__ void prefetch_l1(const void* p) { asm volatile("prefetch.global.L1 [%0];\n" ::"l"(p)); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], unsigned addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], unsigned addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t movt(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(x));
    return r;
}

// A place in the walk over the CTA's granules: unit (b, h), granule x of its
// sequence.
struct Cursor {
    int b, h, x, hi;  // x in [span.first(), hi)
    int slot;         // the granule's slot
    Span s;
};

template <class E, int NT, bool GATHER>
__global__ void __launch_bounds__(kPgThreads, kPgCtasPerSm)
paged_attn_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const PgArgs a) {
    using Cfg = PgCfg<NT>;
    extern __shared__ __align__(1024) unsigned char pg_smem[];
    uint64_t* s_full = reinterpret_cast<uint64_t*>(pg_smem + Cfg::kBars);  // per warp and stage
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
    unsigned char* ringp = pg_smem + warp * Cfg::kStages * kPgStage;
    const unsigned ring = su32(ringp);
    float* merge = reinterpret_cast<float*>(pg_smem + Cfg::kMerge);
    if (!GATHER && lane == 0) {
        for (int i = 0; i < Cfg::kStages; ++i) mbar_init(su32(&s_full[warp * Cfg::kStages + i]), 1);
        mbar_init_fence();
    }
    // Over a shared prefix the kernel before this one is the prefix's pass, of which
    // nothing is read here, and which has waited for the kernel before it.
    if (a.pre.splits == 0) griddep_wait();

    griddep_launch();  // the joining kernel may take its place (it waits for this one's end)

    // ---- the CTA's share: slots [g0, g1) of all units' laid end to end.  Every
    // warp adds up the lengths, four sequences a lane at a time (up to 128
    // sequences: all at once, and the second pass finds them in registers)
    const int B = a.c.B, Hkv = a.c.Hkv;
    int cnt[4], total = 0;
#pragma unroll 4
    for (int b0 = 0; b0 < B; b0 += 128) {
        slots4<GATHER>(a, b0, lane, cta == 0 && warp == 0, cnt);
        total += __reduce_add_sync(0xffffffffu, cnt[0] + cnt[1] + cnt[2] + cnt[3]);
    }
    const Shares share = shares_of(a, total);
    const int g0 = cta < share.nc ? share.start(cta) : 0, g1 = cta < share.nc ? share.start(cta + 1) : 0;
    int first_b = 0, first_base = 0;  // the sequence that holds slot g0, and its first slot
    for (int b0 = 0, run = 0; b0 < B && g0 < g1; b0 += 128) {
        if (B > 128) slots4<GATHER>(a, b0, lane, false, cnt);
        const int sum = cnt[0] + cnt[1] + cnt[2] + cnt[3];
        int at = sum;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, at, m);
            if (lane >= m) at += o;
        }
        const int all = __shfl_sync(0xffffffffu, at, 31);
        at += run - sum;  // before this lane's four
        int fb = -1, base = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (cnt[k] > 0 && at <= g0 && g0 < at + cnt[k]) fb = b0 + lane * 4 + k, base = at;
            at += cnt[k];
        }
        const unsigned who = __ballot_sync(0xffffffffu, fb >= 0);
        if (who) {
            first_b = __shfl_sync(0xffffffffu, fb, __ffs(who) - 1);
            first_base = __shfl_sync(0xffffffffu, base, __ffs(who) - 1);
            break;
        }
        run += all;
    }

    if (g0 < g1) {
        auto enter = [&](Cursor& c) {  // c.b is set: the span, its first granule
            c.s = span_of<GATHER>(a, c.b, false);
            c.x = c.s.first();
            c.hi = c.x + c.s.granules();
        };
        auto next_unit = [&](Cursor& c) {
            if (++c.h == Hkv) {
                c.h = 0;
                do {
                    ++c.b;
                    enter(c);
                } while (c.hi == c.x);
            } else {
                c.x = c.s.first();
            }
        };
        auto advance = [&](Cursor& c) {  // to the next granule (the caller knows there is one); true: of another unit
            ++c.slot;
            if (++c.x < c.hi) return false;
            c.slot += kPgEnd;
            next_unit(c);
            return true;
        };
        auto more = [&](const Cursor& c) {  // whether a granule of this CTA's comes after it
            return c.slot + (c.x + 1 < c.hi ? 1 : 1 + kPgEnd) < g1;
        };
        Cursor at;  // of the consumer
        at.b = first_b;
        enter(at);
        at.h = (g0 - first_base) / at.s.slots();
        const int off = g0 - first_base - at.h * at.s.slots(), gap = at.s.slots() - off;
        at.x += off;
        at.slot = g0;
        // (a share may begin with empty slots, and be nothing else)
        const bool empty = gap <= kPgEnd, none = empty && gap >= g1 - g0;
        if (empty && !none) {
            at.slot += gap;
            next_unit(at);
        }
        if (!none) {
            Cursor ld = at;  // of the loads

            // ---- the products' operand of the unit at hand (its loads are issued before its rows')
            uint32_t qf[NT][8][2];
            auto load_q = [&] {
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int head = t * 8 + (lane >> 2);
                    const uint16_t* qp = a.Q + ((long long)at.b * a.Hq + at.h * a.G + head) * kD + (lane & 3) * 2;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        qf[t][k][0] = head < a.G ? *reinterpret_cast<const uint32_t*>(qp + k * 16) : 0u;
                        qf[t][k][1] = head < a.G ? *reinterpret_cast<const uint32_t*>(qp + k * 16 + 8) : 0u;
                    }
                }
            };
            load_q();

            // ---- the loads.  Every row: lane i keeps the page of this warp's tile of
            // granule pg_x + i; the sequence's first 32 are kept apart, since each of its
            // heads begins with them.  A tile that is not there (no row of the sequence in
            // it, or a bad page) is not loaded; `there` says so per stage.
            int pages = -1, pg_b = -1, pg_x = 0, head_pages = -1, head_b = -1;
            unsigned there = 0, pending = 0, phase = 0;  // bits of the stages: holds a tile; on its way; barrier's phase
            bool dead = false;                           // a wait gave up: this warp loads and adds no more
            uint64_t pol = evict_first_policy();
            bool fresh = true;  // (a list) the loads have come to another unit
            int next_e = -1;    // lane i < 16: entry i of the next tile
            auto entry = [&](int x) {
                const int i = x * kPgGranule + warp * kPageRows + lane;
                return lane < kPageRows && i < ld.s.hi ? a.idx[((long long)ld.b * Hkv + ld.h) * a.k_max + i] : -1;
            };
            auto prefetch_q = [&] {  // the unit's queries, G rows of 256 B
                const int line = lane & 31;
                if (line < 2 * a.G)
                    prefetch_l1(a.Q + ((long long)ld.b * a.Hq + ld.h * a.G + (line >> 1)) * kD + (line & 1) * 64);
            };
            auto issue = [&](int slot) {
                const int r0 = ld.x * kPgGranule + warp * kPageRows;  // the tile's first row (or list entry)
                bool ok = r0 < ld.s.hi && r0 + kPageRows > ld.s.lo;
                if constexpr (!GATHER) {
                    if (ld.b != pg_b || ld.x < pg_x || ld.x >= pg_x + 32) {
                        pg_b = ld.b;
                        pg_x = ld.x;
                        const bool head = ld.x == ld.s.first();
                        if (head && ld.b == head_b) {
                            pages = head_pages;
                        } else {
                            const int r = (ld.x + lane) * kPgGranule + warp * kPageRows;
                            pages = -1;
                            if (ld.x + lane < ld.hi && r < ld.s.hi) {
                                pages = a.c.table[(long long)ld.b * a.c.width + r / a.c.page_size];
                                if ((pages < 0 || pages >= a.c.num_pages) && r + kPageRows > ld.s.lo) {
                                    atomicOr(a.flag, kFlagBounds);
                                    pages = -1;
                                }
                            }
                            if (head) head_pages = pages, head_b = ld.b;
                        }
                    }
                    const int page = __shfl_sync(0xffffffffu, pages, ld.x - pg_x);
                    ok = ok && page >= 0;
#ifdef TSA_DEBUG_KNOBS
                    if (ok && lane == 0 && !(cta == 0 && warp == 0 && ld.x == g_debug_paged_skip)) {
#else
                    if (ok && lane == 0) {
#endif
                        const unsigned bar = su32(&s_full[warp * Cfg::kStages + slot]), dst = ring + slot * kPgStage;
                        const int r = r0 % a.c.page_size;
                        mbar_arrive_tx(bar, kPgStage);
                        tma_4d(dst, &kmap, 0, r, ld.h, page, bar, pol);
                        tma_4d(dst + kPgHalf, &kmap, 64, r, ld.h, page, bar, pol);
                        tma_4d(dst + 2 * kPgHalf, &vmap, 0, r, ld.h, page, bar, pol);
                        tma_4d(dst + 3 * kPgHalf, &vmap, 64, r, ld.h, page, bar, pol);
                    }
                    if (ok) pending |= 1u << slot;
                } else {
                    // lane i < 16 finds entry i's row; a missing or bad one is filled with zeros and masked
                    if (fresh) next_e = entry(ld.x);
                    long long off = -1;
                    if (ok && lane < kPageRows && r0 + lane < ld.s.hi) {
                        const int e = next_e;
                        const int len = min(max(a.lens[ld.b], 0), a.c.rows_cap());
                        if (e >= len) {
                            atomicOr(a.flag, kFlagBounds);
                        } else if (e >= 0) {
                            const int pg = e / a.c.page_size, page = a.c.table[(long long)ld.b * a.c.width + pg];
                            if (page < 0 || page >= a.c.num_pages)
                                atomicOr(a.flag, kFlagBounds);
                            else
                                off = page * a.c.page_stride + ld.h * a.c.head_stride +
                                      (long long)(e - pg * a.c.page_size) * a.c.row_stride;
                        }
                    }
                    if (ld.x + 1 < ld.hi) next_e = entry(ld.x + 1);  // on its way while this tile is requested
                    const unsigned valid = __ballot_sync(0xffffffffu, off >= 0);
                    ok = valid != 0;
                    if (ok) {
                        const unsigned dst = ring + slot * kPgStage;
                        const int ch = lane & 15;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int r = (lane >> 4) + 2 * j;
                            const long long o = __shfl_sync(0xffffffffu, off, r);
                            const unsigned d = dst + (ch >> 3) * kPgHalf + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
                            const int n = o >= 0 ? 16 : 0;
                            const long long e = (o >= 0 ? o : 0) + ch * 8;
                            cp_async16(d, static_cast<const uint16_t*>(a.c.K) + e, n);
                            cp_async16(d + 2 * kPgHalf, static_cast<const uint16_t*>(a.c.V) + e, n);
                        }
                        // the rows' mask, for the consumer of this stage
                        if (lane == 0) s_full[warp * Cfg::kStages + slot] = valid;
                    }
                    cp_async_commit();
                }
                there = (there & ~(1u << slot)) | ((ok ? 1u : 0u) << slot);
            };
            bool rest = true;  // granules of this CTA's not yet requested
            auto issue_next = [&](int slot) {
                if (rest && !dead) {
                    issue(slot);
                    rest = more(ld);
                    fresh = rest && advance(ld);
                    if (fresh) prefetch_q();
                } else if (GATHER) {
                    cp_async_commit();
                }
            };
            __syncwarp();
            for (int i = 0; i < Cfg::kStages; ++i) issue_next(i);

            // ---- the products
            float acc[NT][8][4], m[NT][2], l[NT][2];
            bool open = false;  // a unit is being summed
            int seg0 = 0;       // its first granule here
            bool last = false, loaded_q = true;
            for (int slot = 0; !last; slot = slot + 1 == Cfg::kStages ? 0 : slot + 1) {
                if (!open) {
                    open = true;
                    seg0 = at.x;
                    if (!loaded_q) load_q();
                    loaded_q = false;
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) acc[t][k][0] = acc[t][k][1] = acc[t][k][2] = acc[t][k][3] = 0.f;
                        m[t][0] = m[t][1] = kNegInf;
                        l[t][0] = l[t][1] = 0.f;
                    }
                }
                if constexpr (GATHER) {
                    cp_async_wait<Cfg::kStages - 1>();
                    __syncwarp();
                }
                bool here = !dead && (there >> slot & 1u);
                if (!GATHER && here) {
                    dead = !__all_sync(0xffffffffu, mbar_wait(su32(&s_full[warp * Cfg::kStages + slot]), phase >> slot & 1u, a.flag));
                    here = !dead;
                }
                if (here) {
                    const unsigned st = ring + slot * kPgStage;
                    unsigned valid;  // a bit per row of the tile
                    if constexpr (GATHER) {
                        valid = (unsigned)s_full[warp * Cfg::kStages + slot];
                    } else {
                        phase ^= 1u << slot;
                        pending &= ~(1u << slot);
                        const int r0 = at.x * kPgGranule + warp * kPageRows;
                        valid = 0xffffu;
                        if (r0 + kPageRows > at.s.hi) valid &= 0xffffu >> (r0 + kPageRows - at.s.hi);
                        if (r0 < at.s.lo) valid &= 0xffffu << (at.s.lo - r0);
                        valid &= 0xffffu;
                        if (valid != 0xffffu) {
                            unsigned char* vp = ringp + slot * kPgStage + 2 * kPgHalf;
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const int r = (lane >> 4) + 2 * j;
                                if (!(valid >> r & 1u))
                                    *reinterpret_cast<uint4*>(vp + (lane >> 3 & 1) * kPgHalf + r * 128 + (lane & 7) * 16) =
                                        make_uint4(0, 0, 0, 0);
                            }
                            fence_proxy_async();  // before the next copy into this stage
                            __syncwarp();
                        }
                    }
                    float s[NT][4], s2[NT][4];  // two chains of products
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int j = 0; j < 4; ++j) s[t][j] = s2[t][j] = 0.f;
                    const int fr = lane & 15, fc = lane >> 4;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        uint32_t kf[4];
                        ldsm4(kf, st + (k >> 2) * kPgHalf + fr * 128 + ((((k & 3) * 2 + fc) ^ (fr & 7)) << 4));
#pragma unroll
                        for (int t = 0; t < NT; ++t) E::mma(k & 1 ? s2[t] : s[t], kf, qf[t][k][0], qf[t][k][1]);
                    }
                    const int row = lane >> 2;
                    const bool v0 = valid >> row & 1u, v1 = valid >> (row + 8) & 1u;
                    bool up = false;
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) s[t][j] = (j < 2 ? v0 : v1) ? __fmul_rn(s[t][j] + s2[t][j], a.scale_log2) : kNegInf;
                        up |= fmaxf(s[t][0], s[t][2]) > m[t][0] || fmaxf(s[t][1], s[t][3]) > m[t][1];
                    }
                    if (__any_sync(0xffffffffu, up)) {  // a larger maximum: rescale what there is
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                float x = fmaxf(s[t][j], s[t][j + 2]);
                                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                                x = fmaxf(x, m[t][j]);
                                const float f = x == kNegInf ? 1.f : exp2f(lowered<E>(m[t][j]) - lowered<E>(x));
                                m[t][j] = x;
                                l[t][j] *= f;
#pragma unroll
                                for (int k = 0; k < 8; ++k) acc[t][k][j] *= f, acc[t][k][j + 2] *= f;
                            }
                        }
                    }
                    uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        // (no row so far: the scores are -inf and the weights 0)
                        const float ms[2] = {m[t][0] == kNegInf ? 0.f : lowered<E>(m[t][0]), m[t][1] == kNegInf ? 0.f : lowered<E>(m[t][1])};
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            // j = 0: rows 0-7, j = 1: rows 8-15; two heads each
                            const float p0 = exp2f(s[t][2 * j] - ms[0]), p1 = exp2f(s[t][2 * j + 1] - ms[1]);
                            l[t][0] += p0;
                            l[t][1] += p1;
                            const uint32_t hi = E::pack(p0, p1);
                            ph[t][j] = movt(hi);
                            pl[t][j] = movt(E::pack(p0 - E::lo(hi), p1 - E::hi(hi)));
                        }
                    }
                    // V^T fragments: rows of the stage are tokens, 16 dims an m-tile
                    const int vr = (lane & 7) + (lane >> 4) * 8, vc = lane >> 3 & 1;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        uint32_t vf[4];
                        ldsm4t(vf, st + (2 + (k >> 2)) * kPgHalf + vr * 128 + ((((k & 3) * 2 + vc) ^ (vr & 7)) << 4));
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            E::mma(acc[t][k], vf, ph[t][0], ph[t][1]);
                            E::mma(acc[t][k], vf, pl[t][0], pl[t][1]);
                        }
                    }
                }
                __syncwarp();
                issue_next(slot);

                // ---- the end of the unit here
                const Cursor cur = at;
                last = !more(at);
                if (!last && !advance(at)) continue;
                open = false;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float x = l[t][j];
                        x += __shfl_xor_sync(0xffffffffu, x, 4);
                        x += __shfl_xor_sync(0xffffffffu, x, 8);
                        x += __shfl_xor_sync(0xffffffffu, x, 16);
                        const int head = t * 8 + (lane & 3) * 2 + j;
                        float* w = merge + (warp * Cfg::kHeads + head) * kPartFloats;
                        if (lane < 4) {
                            w[kD] = lowered<E>(m[t][j]);
                            w[kD + 1] = x;
                        }
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            w[k * 16 + (lane >> 2)] = acc[t][k][j];
                            w[k * 16 + (lane >> 2) + 8] = acc[t][k][j + 2];
                        }
                    }
                }
                __syncthreads();
                const bool whole = seg0 == cur.s.first() && cur.x + 1 == cur.hi;
                const int u0 = cur.slot - (cur.x - cur.s.first());  // the unit's first slot
                // a CTA's pieces: of the unit it begins in, then of the unit it ends in
                float* piece = a.pieces + (2LL * cta + (u0 > g0 ? 1 : 0)) * a.G * kPartFloats;
                for (int g = warp; g < a.G; g += kPgWarps) {
                    float M = kNegInf, L = 0.f, f[kPgWarps];
                    const float* w = merge + g * kPartFloats;
                    constexpr int S = Cfg::kHeads * kPartFloats;
#pragma unroll
                    for (int k = 0; k < kPgWarps; ++k) M = fmaxf(M, w[k * S + kD]);
#pragma unroll
                    for (int k = 0; k < kPgWarps; ++k) {
                        const float mk = w[k * S + kD];
                        f[k] = mk == kNegInf ? 0.f : exp2f(mk - M);
                        L += (mk == kNegInf ? w[k * S + kD + 1] * 0.f : f[k] * w[k * S + kD + 1]);
                    }
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < kPgWarps; ++k) {
                        const float4 v = *(reinterpret_cast<const float4*>(w + k * S) + lane);
                        o.x = fmaf(f[k], v.x, o.x), o.y = fmaf(f[k], v.y, o.y);
                        o.z = fmaf(f[k], v.z, o.z), o.w = fmaf(f[k], v.w, o.w);
                    }
                    if (whole) {
                        put_row<E>(a, (long long)cur.b * a.Hq + cur.h * a.G + g, o, M, L, lane);
                    } else {
                        float* p = piece + g * kPartFloats;
                        __stcg(reinterpret_cast<float4*>(p) + lane, o);
                        if (lane == 0) __stcg(reinterpret_cast<float2*>(p + kD), make_float2(M, L));
                    }
                }
                __syncthreads();  // the merge buffer is free again
            }
            if (GATHER) cp_async_wait<0>();
            // (only after a wait gave up) nothing lands after the CTA has gone
            for (int i = 0; i < Cfg::kStages; ++i)
                if (pending >> i & 1u) mbar_wait(su32(&s_full[warp * Cfg::kStages + i]), phase >> i & 1u, nullptr);
        }
    }

    if (a.pre.splits > 0) griddep_wait();  // the prefix's pass is over before this one counts as over
}

// Every row's partials into O and lse: a shared prefix's (one of each split, where
// the sequence holds the prefix whole), and the pieces of its own rows.  A row
// whose unit lay in one CTA, without a prefix, is in O already; a sequence without a
// row gets zeros.  W warps a row, each with a part of the partials, whose loads are
// all on their way at once.
//
// Each CTA adds up all lengths, so past kJoinCtas of them a CTA takes several blocks of
// rows in turn: with a CTA for every 8 rows the additions grew with the square of the batch.
// The whole call, us, at 592, 1184, 2368 CTAs and without a limit: 65536 sequences of 16
// rows (8/1 heads) 1409, 1430, 1503, 5477; 4096 of 64 rows (32/8 heads) 327, 326, 330, 402;
// 256 of 612 rows over a prefix of 512 (64/8) 64.0, 62.6, 62.6, 62.7.
constexpr int kJoinWarps = 8;
constexpr int kJoinCtas = 8 * kPagedSms;
template <class E, int W, bool GATHER, bool MANY>
__global__ void __launch_bounds__(32 * kJoinWarps)
paged_join_kernel(const PgArgs a, int rows) {
    __shared__ float wts[kJoinWarps][kMaxPrefixSplits + kPgCtas];
    __shared__ float4 sums[kJoinWarps][32];
    __shared__ int2 red[kJoinWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = warp % W;
    constexpr int kPer = kJoinWarps / W;  // rows of a block
    // (MANY: several blocks a CTA; a kernel of its own, since with the loop the others have fewer loads
    // in flight: one sequence 8.3 us with one block a CTA, 9.6 with the loop)
    const long long blocks = MANY ? (rows + kPer - 1) / kPer : gridDim.x;
    const int blk0 = (int)(blocks * blockIdx.x / gridDim.x), blk1 = (int)(blocks * (blockIdx.x + 1) / gridDim.x);
    // Where the rows' pieces lie follows from the lengths, which the kernels before this
    // one only read: the first block's are found before the wait on them.
    int b_at = blk0 * kPer / a.Hq;  // (the CTA adds up the lengths once)
    int total = 0, u_at = 0;        // u_at: the first slot of sequence b_at
    for (int i = threadIdx.x; i < a.c.B; i += 32 * kJoinWarps) {
        const int v = span_of<GATHER>(a, i, false).slots() * a.c.Hkv;
        total += v;
        if (i < b_at) u_at += v;
    }
    total = __reduce_add_sync(0xffffffffu, total);
    u_at = __reduce_add_sync(0xffffffffu, u_at);
    if (lane == 0) red[warp] = make_int2(total, u_at);
    __syncthreads();
    total = u_at = 0;
#pragma unroll
    for (int i = 0; i < kJoinWarps; ++i) total += red[i].x, u_at += red[i].y;
    const Shares share = shares_of(a, total);
    int blk = blk0;
    do {
        const int row = blk * kPer + warp / W;
        const int b = min(row, rows - 1) / a.Hq, r = min(row, rows - 1) - b * a.Hq, h = r / a.G, g = r - h * a.G;
        for (; b_at < b; ++b_at) u_at += span_of<GATHER>(a, b_at, false).slots() * a.c.Hkv;
        const Span s = span_of<GATHER>(a, b, false);
        const int u0 = u_at + h * s.slots();  // the unit's first slot
        const bool some = s.granules() > 0;
        const int c0 = some ? share.cta_of(u0) : 0, c1 = some ? share.cta_of(u0 + s.granules() - 1) : 0;
        const int first = 2 * c0 + (u0 > share.start(c0) ? 1 : 0);  // its first piece; the others are their CTAs' first
        if (blk == blk0) {
            griddep_wait();
            griddep_launch();
        }
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float M = kNegInf, L = 0.f;
        bool mine = row < rows;
        if (mine) {
            const int n0 = s.lo > 0 ? a.pre.splits : 0;
            const bool own = some && c0 == c1;
            const int n = n0 + (some ? c1 - c0 + 1 : 0);
            auto part = [&](int i) -> const float* {
                if (i < n0) return a.pre.parts + ((long long)i * rows + row) * kPartFloats;
                if (own) return a.own + (long long)row * kPartFloats;
                return a.pieces + ((long long)(i == n0 ? first : (c0 + i - n0) * 2) * a.G + g) * kPartFloats;
            };
            mine = !(own && !a.own);
            __syncwarp();  // (of the block before: the weights have been read)
            if (mine) o = join_sums(n, w, W, part, wts[warp], lane, [&] { join_weights(n, part, wts[warp], lane, &M, &L); });
        }
        static_assert(W == 1 || !MANY);
        if constexpr (W > 1) {
            sums[warp][lane] = o;
            __syncthreads();
#pragma unroll
            for (int i = 1; i < W; ++i) {
                const float4 v = sums[warp + i < kJoinWarps ? warp + i : warp][lane];
                o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
            }
        }
        if (mine && w == 0) finish_row<E>(a, row, o, M, L, lane);
    } while (MANY && ++blk < blk1);
}

template <class E, int W, bool GATHER, bool MANY = false>
static cudaError_t join_launch(const PgArgs& a, cudaStream_t st) {
    const long long rows = (long long)a.c.B * a.Hq, blocks = (rows * W + kJoinWarps - 1) / kJoinWarps;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(MANY ? kJoinCtas : blocks));
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.stream = st;
    cudaLaunchAttribute attr[1] = {pdl_attr()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_join_kernel<E, W, GATHER, MANY>, a, (int)rows);
    note_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

// The fewer rows, the more warps each, as long as the CTAs (8 warps) come to two an SM.
// The whole call with 1, 4 and 8 warps a row, us: 8 rows of 60 pieces 16.3, 10.0, 8.2;
// 256 rows of a shared prefix 20.6, 18.8, 18.9; 320 rows of it 21.2, 19.2, 21.6; 512 rows
// (a prefix of 16384) 35.8, 28.9, 33.4; 768 rows 26.2, 26.6, 30.3, and without a prefix
// 37.7, 41.5, 44.3; 1024 rows 30.1, 33.4, 38.4; 4096 rows 121.7, 136, 157.  (The form with 4
// has 128 registers and spills 8 bytes.)
template <class E, bool GATHER>
static cudaError_t join_pick(const PgArgs& a, cudaStream_t st) {
    const long long rows = (long long)a.c.B * a.Hq;
    if (rows <= 2 * kPagedSms) return join_launch<E, 8, GATHER>(a, st);
    if (rows <= 4 * kPagedSms) return join_launch<E, 4, GATHER>(a, st);
    if (rows <= kJoinWarps * kJoinCtas) return join_launch<E, 1, GATHER>(a, st);
    return join_launch<E, 1, GATHER, true>(a, st);
}

template <class E, int NT, bool GATHER>
static cudaError_t paged_launch(int grid, const CUtensorMap& km, const CUtensorMap& vm, const PgArgs& a, cudaStream_t st) {
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e0 = smem_opt_in((const void*)paged_attn_kernel<E, NT, GATHER>, PgCfg<NT>::kSmem, &done);
    if (e0 != cudaSuccess) return e0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kPgThreads);
    cfg.dynamicSmemBytes = PgCfg<NT>::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1] = {pdl_attr()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_attn_kernel<E, NT, GATHER>, km, vm, a);
    note_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <class E>
static cudaError_t paged_pick(int grid, const CUtensorMap& km, const CUtensorMap& vm, const PgArgs& a, cudaStream_t st) {
    if (a.idx) return a.G <= 8 ? paged_launch<E, 1, true>(grid, km, vm, a, st) : paged_launch<E, 2, true>(grid, km, vm, a, st);
    return a.G <= 8 ? paged_launch<E, 1, false>(grid, km, vm, a, st) : paged_launch<E, 2, false>(grid, km, vm, a, st);
}

cudaError_t launch_paged_attn(const Pages& c, const void* Q, int Hq, const int32_t* lens, const int32_t* idx,
                              const int32_t* kreq, int k_max, float scale, void* O, float* lse, float* pieces,
                              const PrefixParts& pre, unsigned* flag, cudaStream_t st) {
    if (c.B == 0) return cudaSuccess;
    PgArgs a;
    a.c = c;
    a.Q = static_cast<const uint16_t*>(Q);
    a.Hq = Hq;
    a.G = Hq / c.Hkv;
    a.lens = lens;
    a.idx = idx;
    a.kreq = kreq;
    a.k_max = k_max;
    a.scale_log2 = scale * kLog2e;
    a.O = static_cast<uint16_t*>(O);
    a.lse = lse;
    a.pieces = pieces;
    a.pre = pre;
    a.own = pre.splits > 0 ? pre.own : nullptr;
    a.flag = flag;
    CUtensorMap km = {}, vm = {};
    if (!idx) {
        cudaError_t e = page_map(&km, c, c.K, kPageRows);
        if (e == cudaSuccess) e = page_map(&vm, c, c.V, kPageRows);
        if (e != cudaSuccess) return e;
    }
    const int grid = kPgCtas;
    const cudaError_t e = c.half ? paged_pick<F16>(grid, km, vm, a, st) : paged_pick<Bf16>(grid, km, vm, a, st);
    if (e != cudaSuccess) return e;
    if (idx) return c.half ? join_pick<F16, true>(a, st) : join_pick<Bf16, true>(a, st);
    return c.half ? join_pick<F16, false>(a, st) : join_pick<Bf16, false>(a, st);
}

}  // namespace tsa

#ifdef TSA_DEBUG_KNOBS
// Debug build only: the granule (0) of the paged attention or the tile (1) of a shared
// prefix's pass whose load CTA 0 leaves out; -1 for none.  Returns a cudaError_t.
extern "C" int tsa_debug_prefix_skip_tile(int tile);
extern "C" int tsa_debug_paged_skip_tile(int which, int tile) {
    if (which == 1) return tsa_debug_prefix_skip_tile(tile);
    return (int)cudaMemcpyToSymbol(tsa::g_debug_paged_skip, &tile, sizeof tile);
}
#endif

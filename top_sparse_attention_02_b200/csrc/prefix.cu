// prefix.cu -- the pass over a prefix that a batch of sequences shares: for each
// kv-head the queries of all sequences, B * g rows, against the prefix's keys and
// values, read once for all of them.  Its partials (per split of the prefix: the
// sums, maximum and weight of every row) are joined with each sequence's own rows
// by the paged attention that follows (paged.cu).
//
// With R = B g rows a kv-head the pass does 512 R flop for each 512 bytes of a row of
// K and V, so up to about 250 rows HBM bounds it and above the tensor cores do:
// both contractions run on tcgen05, tiles of 128 query rows x 128 prefix rows.
//
// A CTA (one per SM, 20 warps) takes up to 256 rows of one kv-head over one split
// of the prefix, as two streams of 128 rows that take turns on the tensor cores:
// while one stream's softmax runs on its eight warps, the other's products are computed.
//   warp 17  TMA producer: K and V tiles of 128 prefix rows (boxes of as many rows as
//            a page allows, 128-byte swizzle) into a ring of 5 stages of 32 KB;
//   warps 16, 18  MMA issuers of stream 0, 1: S = Q K^T into TMEM (128 columns a
//            stream), then O += P V with P read from TMEM and V as stored (the MN-major
//            operand).  (One warp for both streams spent 2000 cycles a turn on its waits
//            and its issuing, beside 1030 of products: the streams waited for it.)
//   warps 0-7, 8-15  softmax of stream 0, 1: half a row of S a thread, the
//            halves' maxima exchanged through shared memory; P = 2^(S - m) in 16 bits
//            over S's columns, l in fp32.  O is rescaled in TMEM only when the maximum
//            has grown by more than 2^8 (fp16: 2^5; the result is the same: all sums
//            are relative to the reference they were formed with).
//   warp 19  only makes warps 16-19 a warpgroup that hands registers to the softmax
//            (96 a thread at launch; 56 here and 104 there: 4 x 104 + 56 <= 5 x 96).
// TMEM is full: 2 x (S 128 + O 128) columns.  When 128 rows or fewer are left for a
// CTA, both streams take the same rows and every other tile, and are joined at the
// end in shared memory.
//
// P is rounded to the element type once (where paged.cu, which waits for memory, keeps the
// rest as a second number): the second products would take the tensor cores twice as
// long.  The outputs' error is then 1.4 times their own rounding's (2.3e-3 against 1.7e-3 of
// the norm in bf16), the weights' errors being independent.
//
// Measured: 64 sequences x 64/8 heads over 32768 rows (68.7 Gflop, 134 MB) 82 us with the join = 0.84 PFLOP/s,
// 0.51 of the measured matrix rate.  At 96 registers the softmax spills 44 bytes (100 of loads).  With
// fused products of scores (2% faster) a pair of tiles took 3870 cycles where their products take
// 2068: each stream is a chain of softmax (2150, of which the special-function units need
// 1024), turn, products and their waits (1700), and TMEM has no room for S of a third tile.  Half tiles (64 columns) with S two
// halves ahead came to 4140 (one thread a row) and 3870 (two groups in turn); a part of the
// weights by polynomial on the FMA pipe, the maximum found beside
// the weights and a staggered start changed nothing or were slower.
//
// Sequences shorter than the prefix have rows here, too, which nobody reads: no row
// needs a mask of its own.  The prefix's last tile may be partial: its columns past
// the end become -inf and its V rows there are zeroed in shared memory.  A page out
// of range is read as zeros (a box outside the tensor map) and its columns masked.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "common.cuh"
#include "paged.cuh"
#include "tma.cuh"

namespace tsa {

constexpr int kPxSoftWarps = 16;
constexpr int kPxThreads = 32 * (kPxSoftWarps + 4);
constexpr int kPxTile = 128;                  // query rows of a stream, prefix rows of a tile
constexpr int kPxRows = 2 * kPxTile;          // query rows of a CTA
constexpr int kPxHalf = kPxTile * 128;        // 64 elements of 128 rows: 16 KB
constexpr int kPxStage = 2 * kPxHalf;         // 32 KB
constexpr int kPxStages = 5;
constexpr int kPxQ = 0;                       // Q of both streams, 64 KB
constexpr int kPxRing = 2 * kPxStage;
constexpr int kPxBars = kPxRing + kPxStages * kPxStage;
constexpr int kPxMax = kPxBars + 256;            // the halves' maxima: [stream][half][row]
constexpr int kPxSmem = kPxMax + 2 * 2 * kPxTile * 4;
constexpr int kPxTmemCols = 512;
static_assert(kPxRows * kPartFloats * 4 <= kPxStages * kPxStage, "the rows' partials fit the ring");

#ifdef TSA_DEBUG_KNOBS
// Debug build only (never in the product library): the tile of CTA 0 whose K is neither
// armed nor loaded, so that the waits on it run out; -1: none.
__device__ int g_debug_prefix_skip = -1;
#endif

struct PxArgs {
    const uint16_t* Q;
    const int32_t *lens, *table;
    int B, Hq, Hkv, G, width, page_size, num_pages, prefix_len;
    int box_log, groups, splits;  // rows of a TMA box: 16 << box_log
    float scale_log2;
    float* parts;  // [splits][B][Hq][kPartFloats]
    unsigned* flag;
};

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_commit(unsigned bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar) : "memory");
}

// true in one lane of a warp that runs this together: what it issues is then known to be
// issued once (under a test of the lane number an MMA took 100 cycles to issue instead of 64)
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
    return one != 0;
}

__device__ __forceinline__ void tm_ld32(uint32_t (&r)[32], uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tm_st32(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};\n" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};\n" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// Shared-memory operand of a tile stored as two halves of 64 elements (128-byte
// rows, 128-byte swizzle): the descriptor's low word holds the address (in 16
// bytes) and the leading offset, its high word the stride offset (8-row groups
// 1024 B apart), the version and the swizzle.
//   K-major (the contraction runs along the row): no leading offset; 16 elements on = 32 B.
//   MN-major (it runs across the rows): 64-element blocks a half (16 KB) apart; 16 rows on = 2048 B.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k(unsigned saddr) { return (saddr >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mn(unsigned saddr) { return (saddr >> 4) | ((uint32_t)(kPxHalf >> 4) << 16); }

// D (+)= A B, A from shared memory (a low descriptor word) or from TMEM
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 da, db;\n mov.b64 da, {%1, %4};\n mov.b64 db, {%2, %4};\n setp.ne.b32 p, %5, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(kDescHi), "r"((int)add)
        : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 db;\n mov.b64 db, {%2, %4};\n setp.ne.b32 p, %5, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(kDescHi), "r"((int)add)
        : "memory");
}
// instruction descriptor: D f32, A and B bf16 (1) or f16 (0), N and M 128; B MN-major for the second product
template <class E>
__device__ constexpr uint32_t px_idesc(bool b_mn) {
    const uint32_t t = E::kHalf ? 0u : 1u;
    return (1u << 4) | (t << 7) | (t << 10) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(kPxTile >> 3) << 17) |
           ((uint32_t)(kPxTile >> 4) << 24);
}

__device__ __forceinline__ float max3(float a, float b, float c) {  // NaN if one is
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

template <class E>
__global__ void __launch_bounds__(kPxThreads, 1)
prefix_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const PxArgs a) {
    extern __shared__ __align__(1024) unsigned char px_smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t* bars = reinterpret_cast<uint64_t*>(px_smem + kPxBars);
    const unsigned bar0 = su32(bars);
    auto full = [&](int i) { return bar0 + i * 8; };
    auto empty = [&](int i) { return bar0 + (kPxStages + i) * 8; };
    auto sfull = [&](int s) { return bar0 + (2 * kPxStages + s) * 8; };
    auto pfull = [&](int s) { return bar0 + (2 * kPxStages + 2 + s) * 8; };
    auto ofull = [&](int s) { return bar0 + (2 * kPxStages + 4 + s) * 8; };
    auto drain = [&](int s) { return bar0 + (2 * kPxStages + 6 + s) * 8; };
    auto turn = [&](int s) { return bar0 + (2 * kPxStages + 8 + s) * 8; };
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 2 * kPxStages + 10);
    const int box_log = 4 + a.box_log, box = 1 << box_log, chunks = kPxTile >> box_log;

    const int grp = blockIdx.x % a.groups, h = blockIdx.x / a.groups % a.Hkv, split = blockIdx.x / (a.groups * a.Hkv);
    const int nt_all = (a.prefix_len + kPxTile - 1) / kPxTile;  // (2^23 at most, 128 splits)
    const int t0 = nt_all * split / a.splits, nt = nt_all * (split + 1) / a.splits - t0;
    const int R = a.B * a.G, row0 = grp * kPxRows;
    const bool pair = R - row0 > kPxTile;  // two streams of rows; else two streams of tiles
    // set-up that touches no memory of the caller's: before the wait on the kernel before
    if (warp == 16) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(su32(s_tmem)),
                     "r"(kPxTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
    } else if (warp == 17) {
        if (lane == 0) {
            asm volatile("prefetch.tensormap [%0];\n" ::"l"(&kmap) : "memory");
            asm volatile("prefetch.tensormap [%0];\n" ::"l"(&vmap) : "memory");
            for (int i = 0; i < kPxStages; ++i) {
                mbar_init(full(i), 1);
                mbar_init(empty(i), pair ? 2 : 1);  // the streams that use a tile
            }
            for (int s = 0; s < 2; ++s) {
                mbar_init(sfull(s), 1);
                mbar_init(pfull(s), 2 * kPxTile);
                mbar_init(ofull(s), 1);
                mbar_init(drain(s), 1);
                mbar_init(turn(s), 1);
            }
            mbar_init_fence();
        }
        __syncwarp();
    }
    griddep_wait();
    griddep_launch();  // the pass over the sequences' own rows reads nothing of this one
    // Requested first: Q, which needs no length (all of a thread's loads at once; rows past
    // R are zeros), and the first tiles' pages as the first sequence has them, if it holds
    // the prefix (entries past a sequence's rows are not read; without that length in between
    // few streams would take 18.2 us instead of 18.4).
    uint4 qv[kPxRows / 32];
    int pages = 0;
    const int ahead = 32 / chunks;  // tiles whose pages the producer's lanes hold
    if (warp < kPxSoftWarps) {
#pragma unroll
        for (int i = 0; i < kPxRows / 32; ++i) {
            const int gr = row0 + i * 32 + (tid >> 4), b = gr / a.G;
            qv[i] = make_uint4(0, 0, 0, 0);
            if (gr < R)
                qv[i] = *reinterpret_cast<const uint4*>(a.Q + ((long long)b * a.Hq + h * a.G + gr - b * a.G) * kD + (tid & 15) * 8);
        }
    } else if (warp == 17) {
        const int r = (t0 + lane / chunks) * kPxTile + lane % chunks * box;
        if (lane / chunks < nt && r < a.prefix_len && a.lens[0] >= a.prefix_len) pages = a.table[r / a.page_size];
    }
    // the sequence through whose table the prefix is read: the first that holds it whole
    int src = -1;
    for (int b0 = 0; b0 < a.B && src < 0; b0 += 32) {
        const unsigned v = __ballot_sync(0xffffffffu, b0 + lane < a.B && a.lens[b0 + lane] >= a.prefix_len);
        if (v) src = b0 + __ffs(v) - 1;
    }
    if (src < 0) {  // nobody does
        __syncthreads();
        if (warp == 16)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(*s_tmem), "r"(kPxTmemCols) : "memory");
        return;
    }
    const int32_t* table = a.table + (long long)src * a.width;
    // the tiles of stream s: all of the split's, or every other one
    auto count = [&](int s) { return pair ? nt : (nt - s + 1) >> 1; };
    auto tile_of = [&](int s, int i) { return pair ? i : 2 * i + s; };  // (of this CTA's)

    // ---- the producer's loads (warp 17): K of tile t at ring position 2t, V at 2t + 1.
    // The lanes hold the pages of the boxes of the next 32 / chunks tiles.
    const unsigned smem0 = su32(px_smem);
    const uint64_t pol = evict_first_policy();
    int load_pos = 0, pages_t = 0;  // (pages: of the tiles from pages_t on)
    auto load_next = [&] {
        const int t = load_pos >> 1, kv = load_pos & 1, chunk = lane >> 1, half = lane & 1;
        if (!kv && (t == 0 || t - pages_t == ahead)) {
            pages_t = t;
            const int pt = t + lane / chunks, r = (t0 + pt) * kPxTile + lane % chunks * box;
            if (pt < nt && r < a.prefix_len) {
                if (t > 0 || src > 0) pages = table[r / a.page_size];
                if (pages < 0 || pages >= a.num_pages) {
                    atomicOr(a.flag, kFlagBounds);
                    pages = a.num_pages;
                }
            } else {
                pages = a.num_pages;  // outside the map: zeros
            }
        }
#ifdef TSA_DEBUG_KNOBS
        if (blockIdx.x == 0 && !kv && t == g_debug_prefix_skip) {
            ++load_pos;
            return;
        }
#endif
        const int st = load_pos % kPxStages;
        if (lane == 0) mbar_arrive_tx(full(st), kPxStage);
        __syncwarp();
        const int page = __shfl_sync(0xffffffffu, pages, (t - pages_t) * chunks + (chunk < chunks ? chunk : 0));
        if (chunk < chunks)
            tma_4d(smem0 + kPxRing + st * kPxStage + half * kPxHalf + chunk * box * 128, kv ? &vmap : &kmap, half * 64,
                   ((t0 + t) * kPxTile + chunk * box) % a.page_size, h, page, full(st), pol);
        ++load_pos;
    };

    if (warp == 17) {
        load_next();  // the first tile's (the ring is empty: nothing to wait for)
        load_next();
    } else if (warp < kPxSoftWarps) {  // Q: row r of stream s at half * 16 KB + r * 128 B, 16-byte chunks swizzled
        const int c = tid & 15;
#pragma unroll
        for (int i = 0; i < kPxRows / 32; ++i) {
            const int r = i * 32 + (tid >> 4), rr = r & (kPxTile - 1);
            *reinterpret_cast<uint4*>(px_smem + kPxQ + (r >> 7) * kPxStage + (c >> 3) * kPxHalf + rr * 128 +
                                      (((c & 7) ^ (rr & 7)) << 4)) = qv[i];
        }
        fence_proxy_async();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    // TMEM columns: S of stream s at s * 128 (P over its first 64), O at 256 + s * 128

    if (warp >= kPxSoftWarps) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 56;\n");
      if (warp == 17) {
        // ---- TMA producer
        bool ok = true;
        while (load_pos < 2 * nt) {
            if (load_pos >= kPxStages) ok = __all_sync(0xffffffffu, mbar_wait(empty(load_pos % kPxStages), (load_pos / kPxStages - 1) & 1, a.flag));
            if (!ok) break;
            load_next();
        }
        // what was requested has landed before the CTA leaves (at once, unless a wait gave up)
        for (int p = max(0, load_pos - kPxStages); p < load_pos; ++p)
            mbar_wait(full(p % kPxStages), (p / kPxStages) & 1, nullptr);
        __syncwarp();
      } else if (warp != 19) {
        // ---- MMA issuer of stream s: the warp walks and waits together, one lane issues
        const int s = (warp - 16) >> 1, n = count(s);
        const uint32_t ts = tmem + s * 128, to = ts + 256, q = desc_k(smem0 + kPxQ + (pair ? s : 0) * kPxStage);
        bool ok = true;
        auto loaded = [&](int pos) {
            return __all_sync(0xffffffffu, mbar_wait(full(pos % kPxStages), (pos / kPxStages) & 1, a.flag));
        };
        // Per turn: O += P V of tile i, then S of tile i + 1 over the same columns (the tensor
        // core takes a warp's instructions in order).  The streams' turns alternate, so
        // that one's products are computed during the other's softmax: left to
        // themselves the two fall into step, both softmaxes, then both products.
        for (int i = -1; i < n && ok; ++i) {
            const int pv = i >= 0 ? 2 * tile_of(s, i) + 1 : -1, pk = i + 1 < n ? 2 * tile_of(s, i + 1) : -1;
            const int turns = i + 1 + s;  // of the other stream's that came before
            if (pv >= 0) ok = loaded(pv);
            if (pk >= 0) ok = ok && loaded(pk);
            if (turns > 0) ok = ok && __all_sync(0xffffffffu, mbar_wait(turn(s), (turns - 1) & 1, a.flag));
            if (pv >= 0) ok = ok && __all_sync(0xffffffffu, mbar_wait(pfull(s), i & 1, a.flag));
            if (!ok) break;
            tc_fence_after();
            const uint32_t vt = desc_mn(smem0 + kPxRing + pv % kPxStages * kPxStage);
            const uint32_t kt = desc_k(smem0 + kPxRing + pk % kPxStages * kPxStage);
            if (elect_one()) {
                if (pv >= 0) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) tc_mma_ts(to, ts + k * 8, vt + k * (2048 >> 4), px_idesc<E>(true), i + k > 0);
                    tc_commit(empty(pv % kPxStages));
                    if (i + 1 == n) tc_commit(ofull(s));
                }
                if (pk >= 0) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t off = ((k >> 2) * kPxHalf + (k & 3) * 32) >> 4;
                        tc_mma_ss(ts, q + off, kt + off, px_idesc<E>(false), k > 0);
                    }
                    tc_commit(sfull(s));
                    tc_commit(empty(pk % kPxStages));
                }
                mbar_arrive(turn(1 - s));
            }
            __syncwarp();
        }
        // the last products have been computed before TMEM is freed: the softmax
        // warps waited for them, unless a wait gave up
        if (!ok) {
            if (elect_one()) tc_commit(drain(s));
            __syncwarp();
            mbar_wait(drain(s), 0, nullptr);
        }
      }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 104;\n");
        // ---- softmax of stream s: this thread's half (64 columns) of a row
        const int s = warp >> 3, hf = warp >> 2 & 1, q = warp & 3, row = q * 32 + lane;
        const int n = count(s);
        const uint32_t ts = tmem + ((uint32_t)(q * 32) << 16) + s * 128, to = ts + 256 + hf * 64;
        float* maxima = reinterpret_cast<float*>(px_smem + kPxMax) + s * 2 * kPxTile;
        float m = -INFINITY, l = 0.f;
        bool ok = true;  // (after a wait that gave up the barriers below are still kept)
        for (int i = 0; i < n; ++i) {
            const int t = t0 + tile_of(s, i);
            // the tile's columns that are rows of the prefix: a bit per box, and those before the end
            const int r = t * kPxTile + lane * box;
            bool good = false;
            if (lane < chunks && r < a.prefix_len) {
                const int page = table[r / a.page_size];
                good = page >= 0 && page < a.num_pages;
            }
            const unsigned valid = __ballot_sync(0xffffffffu, good);
            const int nv = min(kPxTile, a.prefix_len - t * kPxTile);
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(sfull(s), i & 1, a.flag));
            uint32_t x[2][32];
            if (ok) {
                tc_fence_after();
                tm_ld32(x[0], ts + hf * 64);
                tm_ld32(x[1], ts + hf * 64 + 32);
                tm_wait_ld();
                if (valid != (0xffffffffu >> (32 - chunks)) || nv < kPxTile) {
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const int col = hf * 64 + c * 32 + j;
                            if (col >= nv || !(valid >> (col >> box_log) & 1u)) x[c][j] = 0xff800000u;  // -inf
                        }
                }
                float mq[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t* y = &x[c >> 1][(c & 1) * 16];
                    mq[c] = max3(__uint_as_float(y[0]), __uint_as_float(y[1]), __uint_as_float(y[2]));
#pragma unroll
                    for (int j = 3; j < 15; j += 2) mq[c] = max3(mq[c], __uint_as_float(y[j]), __uint_as_float(y[j + 1]));
                    mq[c] = max3(mq[c], __uint_as_float(y[15]), -INFINITY);
                }
                maxima[hf * kPxTile + row] = max3(max3(mq[0], mq[1], mq[2]), mq[3], -INFINITY);
            }
            // both halves have their S in registers (P goes over it) and each other's maximum
            asm volatile("bar.sync %0, 256;\n" ::"r"(2 + s) : "memory");
            if (!ok) continue;
            float mx = __fmul_rn(max3(maxima[row], maxima[kPxTile + row], -INFINITY), a.scale_log2);
            // a NaN or an infinite score: the row's result is NaN, as the softmax's is
            if (!(mx < INFINITY)) l = NAN, mx = -INFINITY;
            // rescale when some row's maximum has left the range that the sums were formed for
            const bool big = fabsf(mx) >= kBigLogit && mx > -INFINITY;  // (no fraction left: see kBigLogit)
            if (!big) mx -= E::kBiasRef;
            const bool grow = mx > m + (big ? 0.f : E::kGrow) || (m == -INFINITY && mx > m);
            if (__any_sync(0xffffffffu, grow)) {
                const float f = grow ? (m == -INFINITY ? 0.f : ex2(m - mx)) : 1.f;
                if (grow) m = mx;
                l *= f;
                if (i > 0) {
#pragma unroll 1
                    for (int c = 0; c < 2; ++c) {
                        uint32_t o[32];
                        tm_ld32(o, to + c * 32);
                        tm_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                        tm_st32(to + c * 32, o);
                    }
                }
            }
            if (nv < kPxTile) {  // zero V's rows past the end (the boxes past it came as zeros)
                const int pos = 2 * tile_of(s, i) + 1;
                ok = __all_sync(0xffffffffu, mbar_wait(full(pos % kPxStages), (pos / kPxStages) & 1, a.flag));
                if (!ok) continue;
                unsigned char* v = px_smem + kPxRing + pos % kPxStages * kPxStage;
                const int end = min(kPxTile, (nv + box - 1) & -box);
                for (int j = tid & 255; j < (end - nv) * 16; j += 256)
                    *reinterpret_cast<uint4*>(v + (j >> 3 & 1) * kPxHalf + (nv + (j >> 4)) * 128 + (j & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
                fence_proxy_async();
            }
            const float shift = m == -INFINITY ? 0.f : -m;
            float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t p[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    // (a quarter of these by polynomial on the FMA pipe, packed or not, took as long)
                    // (the product is rounded as the maximum's was: a fused one may lie above it by half a
                    // step of the score, 2^4 at 2^28; that would save 2 us of the large batch's 124)
                    const float p0 = ex2(__fmul_rn(__uint_as_float(x[c][2 * j]), a.scale_log2) + shift);
                    const float p1 = ex2(__fmul_rn(__uint_as_float(x[c][2 * j + 1]), a.scale_log2) + shift);
                    ls[2 * j & 3] += p0;
                    ls[(2 * j & 3) + 1] += p1;
                    p[j] = E::pack(p0, p1);
                }
                tm_st16(ts + hf * 32 + c * 16, p);
            }
            tm_wait_st();
            tc_fence_before();
            mbar_arrive(pfull(s));
            l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
        }
        if (ok && n > 0) ok = __all_sync(0xffffffffu, mbar_wait(ofull(s), 0, a.flag));
        tc_fence_after();
        // the row's weight is the sum of its halves'
        asm volatile("bar.sync %0, 256;\n" ::"r"(2 + s) : "memory");
        maxima[hf * kPxTile + row] = l;
        asm volatile("bar.sync %0, 256;\n" ::"r"(2 + s) : "memory");
        l = maxima[row] + maxima[kPxTile + row];
        // The rows' partials are put together in the ring, 528 B each as in memory, and
        // copied out by the copy engine.  (Written from the registers, 16 B a row at a
        // time, they took 2.5 us.)  Without a second stream's rows, stream 1 hands its to stream 0.
        asm volatile("bar.sync 1, 512;\n" ::: "memory");  // no product reads the ring any more
        unsigned char* out = px_smem + kPxRing + (pair ? s * kPxTile * kPartFloats * 4 : 0);
        float* mine = reinterpret_cast<float*>(out) + row * kPartFloats;
        if (ok && (pair || s == 1)) {
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
                uint32_t o[32];
                if (n > 0) {
                    tm_ld32(o, to + c * 32);
                    tm_wait_ld();
                }
#pragma unroll
                for (int j = 0; j < 32; j += 4)
                    *reinterpret_cast<uint4*>(mine + hf * 64 + c * 32 + j) =
                        n > 0 ? make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]) : make_uint4(0, 0, 0, 0);
            }
            if (hf == 0) *reinterpret_cast<float4*>(mine + kD) = make_float4(m, l, 0.f, 0.f);
        }
        if (!pair) {
            asm volatile("bar.sync 1, 512;\n" ::: "memory");
            const float m1 = mine[kD], l1 = mine[kD + 1], M = fmaxf(m, m1);
            const float f0 = m == -INFINITY ? 0.f : ex2(m - M), f1 = m1 == -INFINITY ? 0.f : ex2(m1 - M);
            if (ok && s == 0) {
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    uint32_t o[32];
                    tm_ld32(o, to + c * 32);
                    tm_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        float4* w = reinterpret_cast<float4*>(mine + hf * 64 + c * 32 + j);
                        float4 v = *w;
                        v.x = fmaf(f1, v.x, f0 * __uint_as_float(o[j])), v.y = fmaf(f1, v.y, f0 * __uint_as_float(o[j + 1]));
                        v.z = fmaf(f1, v.z, f0 * __uint_as_float(o[j + 2])), v.w = fmaf(f1, v.w, f0 * __uint_as_float(o[j + 3]));
                        *w = v;
                    }
                }
                l = (m == -INFINITY ? l : f0 * l) + (m1 == -INFINITY ? l1 : f1 * l1);
            }
            asm volatile("bar.sync %0, 256;\n" ::"r"(2 + s) : "memory");  // both halves have read the other's m and l
            if (ok && s == 0 && hf == 0) *reinterpret_cast<float2*>(mine + kD) = make_float2(M, l);
        }
        fence_proxy_async();
        asm volatile("bar.sync %0, 256;\n" ::"r"(2 + s) : "memory");
        if (ok && (pair || s == 0)) {  // a sequence's rows of this head are contiguous: one copy each
            const int lo = row0 + (pair ? s * kPxTile : 0), hi = min(lo + kPxTile, R), b0 = lo / a.G;
            for (int b = b0 + (tid & 255); b * a.G < hi; b += 256) {
                const int r0 = max(b * a.G, lo), r1 = min((b + 1) * a.G, hi);
                bulk_store(a.parts + (((long long)split * a.B + b) * a.Hq + h * a.G + r0 - b * a.G) * kPartFloats,
                           su32(out) + (r0 - lo) * kPartFloats * 4, (r1 - r0) * kPartFloats * 4);
            }
            bulk_store_wait();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(kPxTmemCols) : "memory");
    }
}

// Splits of the prefix: as many as make the fewest rounds of CTAs over the SMs, each
// round as long as its tiles and about three tiles' time of set-up and end.
static int px_groups(int R) { return (R + kPxRows - 1) / kPxRows; }
int prefix_max_splits(int Hkv, int R, int prefix_len) {
    const long long items = (long long)Hkv * px_groups(R), nt = ((long long)prefix_len + kPxTile - 1) / kPxTile;
    return (int)std::min({nt, (long long)kMaxPrefixSplits, std::max(1LL, 2 * kPagedSms / std::max(1LL, items))});
}
static int px_splits(int Hkv, int R, int prefix_len) {
    const long long items = (long long)Hkv * px_groups(R), nt = ((long long)prefix_len + kPxTile - 1) / kPxTile;
    int best = 1;
    long long cost = -1;
    for (int s = 1; s <= prefix_max_splits(Hkv, R, prefix_len); ++s) {
        const long long c = (items * s + kPagedSms - 1) / kPagedSms * ((nt + s - 1) / s + 3);
        if (cost < 0 || c < cost) best = s, cost = c;
    }
    return best;
}

template <class E>
static cudaError_t px_launch(int grid, const CUtensorMap& km, const CUtensorMap& vm, const PxArgs& a, cudaStream_t st) {
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = smem_opt_in((const void*)prefix_kernel<E>, kPxSmem, &done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kPxThreads);
    cfg.dynamicSmemBytes = kPxSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1] = {pdl_attr()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, prefix_kernel<E>, km, vm, a);
    note_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_prefix(const Pages& c, const void* Q, int Hq, const int32_t* lens, int prefix_len, float scale,
                          float* parts, PrefixParts* out, unsigned* flag, cudaStream_t st) {
    PxArgs a;
    a.Q = static_cast<const uint16_t*>(Q);
    a.lens = lens;
    a.table = c.table;
    a.B = c.B;
    a.Hq = Hq;
    a.Hkv = c.Hkv;
    a.G = Hq / c.Hkv;
    a.width = c.width;
    a.page_size = c.page_size;
    a.num_pages = c.num_pages;
    a.prefix_len = prefix_len;
    a.box_log = 0;  // the largest power of two that divides the page, a tile at most
    while ((kPageRows << a.box_log) < kPxTile && c.page_size % (kPageRows << (a.box_log + 1)) == 0) ++a.box_log;
    a.groups = px_groups(c.B * a.G);
    a.splits = px_splits(c.Hkv, c.B * a.G, prefix_len);
    a.scale_log2 = scale * kLog2e;
    a.parts = parts;
    a.flag = flag;
    CUtensorMap km, vm;
    cudaError_t e = page_map(&km, c, c.K, kPageRows << a.box_log);
    if (e == cudaSuccess) e = page_map(&vm, c, c.V, kPageRows << a.box_log);
    if (e != cudaSuccess) return e;
    out->parts = parts;
    out->own = parts + (size_t)a.splits * c.B * Hq * kPartFloats;
    out->splits = a.splits;
    out->prefix_len = prefix_len;
    const int grid = a.splits * c.Hkv * a.groups;
    return c.half ? px_launch<F16>(grid, km, vm, a, st) : px_launch<Bf16>(grid, km, vm, a, st);
}

}  // namespace tsa

#ifdef TSA_DEBUG_KNOBS
extern "C" int tsa_debug_prefix_skip_tile(int tile) {
    return (int)cudaMemcpyToSymbol(tsa::g_debug_prefix_skip, &tile, sizeof tile);
}
#endif

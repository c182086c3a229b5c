// Attention of a tree of drafted tokens (one token, a prompt) over the paged cache.
//
//   x_ij = scale q_i . k_j over the keys j that row i sees,
//   out_i = sum_j 2^(x_ij c - m_i) v_j / l_i,  l_i = sum_j 2^(x_ij c - m_i), c = log2 e,
// in one pass over the keys with a running maximum m (flash form): tiles of
// 128 keys, S = Q K^T and O += P V on the tensor cores (tcgen05, fp32
// accumulators in TMEM), the softmax between them in registers, P back into
// TMEM as the second product's A operand.
//
// Rows: the G = Hq / Hkv query heads of a K/V head share its keys, so a query
// tile's 128 rows are (token, head of the group) pairs, TPT = 128 / G tokens.
// Work: a segment is one request, K/V head and pair of query tiles, over all
// its key tiles.  The segments' key tiles laid end to end are cut into equal
// shares, one a CTA (persistent, one CTA an SM), whatever the lengths; every
// CTA finds its share from the lengths itself.  A segment that a cut divides
// leaves fp32 partial results; at the kernel's end the CTAs that hold parts of
// it wait for one another's and add them in key order, each some of its columns.
//
// Two streams keep the tensor core and the exponentials busy side by side:
// S, P and O exist twice in TMEM (all of its 512 columns), each with a warpgroup of
// softmax threads (a thread a row).  With two query tiles the streams are the tiles,
// and each K/V tile serves both; with one, the streams take alternate key tiles and
// are added at the segment's end.
//
// Warps: 0 and 12 TMA producers (K and V, by page boxes), 13 loads Q (e4m3: makes
// its terms where rows are few), 1 and 3 MMA issuers (one a stream), 2 cleans V tiles
// that hold keys some row does not see, makes f16 of e4m3 ones (with few rows and D = 128
// the softmax warps do) and counts them, 15 counts K tiles, 14 finds the CTA's segments
// and hands them to the others, 4-7 and 8-11 the softmax.
//
// What bounds it.  With few rows the bytes of K and V: 16 requests of 8, bf16: 70 us
// (73 launched from the host), 0.73 of the measured copy bandwidth.  With an e4m3 cache
// and D = 128 a stream's chain comes close to them, and V's codes are a part of it: 128
// requests of one token, contexts to 16384: 625 to 655 us, 0.69 to 0.73, the tensor core
// 57% busy.  With full tiles the chain alone: 1,960 cycles
// of softmax, 910 for the products that follow it (12 MMAs of 128 x 128 x 16), 500 from
// their ends to the next step's start; two such chains keep the tensor core at 54% and
// the exponentials at 27% (prompts of up to 2000 tokens: 435 to 450 us, 0.61 to 0.63 of the
// measured bf16 rate).  S and O leave no room in TMEM for a third chain; S in halves of 64 keys,
// the first made early, was slower (508 us against 442), since an MMA of N = 64 takes as long as
// one of 128.  A call of few tiles is latency, 12.5 us: 2.5 before the first load, 1.5
// a load, then each step of the chain once, at the speed at which code is first
// fetched, which is why what runs once a segment is written as loops.
#include "kv.cuh"
#include "tc_ptx.cuh"

#include <math_constants.h>

#include <atomic>

namespace moe {
namespace {

constexpr int A_THREADS = 512;
constexpr int A_CTAS = 152;                 // CTAs, all running at once: the SMs of a GB300
constexpr int KT = 128;                     // keys a tile
constexpr int A_MISC = 3072;                // barriers and small tables
constexpr int SEGS = 4;                     // segments handed out ahead
constexpr int NAN_SLOTS = 16;

constexpr int least(int a, int b) { return a < b ? a : b; }

template <int D, bool E4M3>
struct ACfg {
    static constexpr int ROWB = E4M3 ? D : 2 * D;            // bytes a key
    static constexpr int SW = ROWB < 128 ? ROWB : 128;       // swizzle width
    static constexpr int HALVES = ROWB / SW;
    static constexpr int SLOT = KT * ROWB;                   // a K or V tile
    static constexpr int QT = 128 * D * 2;                   // a query tile: bf16, or e4m3 hi and lo
    static constexpr int QMISC = E4M3 ? 1024 : 0;            // e4m3: row scales of two query tiles
    // V's slots.  e4m3 codes are made f16 for the second product, and the weights are one
    // f16 term.  (e4m3 terms of the weights have no room for small ones beside a large one;
    // with three e5m2 terms 16 requests of 8 rows take 61 us against 58, 128 of one token
    // 612 to 622 against 622 to 630.)  Warp 2 makes them, but for copies of few rows with D = 128: there K
    // and V come faster than one warp converts (128 requests of one token: 655 us), and the
    // softmax warps make a quarter of a tile each, after their weights (before them: 638).
    // The codes land at RAW in a slot, the f16 rows stand from its begin on, in blocks of
    // 128 bytes a row; with D = 128 the second block takes the codes' own place, row by row.
    static constexpr int RAW = E4M3 ? KT * 128 : 0;
    static constexpr int VSLOT = E4M3 ? KT * (D == 128 ? 256 : 192) : SLOT;
    static constexpr int FIT = 232448 - A_MISC - QMISC - 2 * QT;
    static constexpr int NV = least(8, E4M3 ? FIT / (SLOT + VSLOT) : FIT / SLOT - FIT / SLOT / 2);   // slots of V,
    static constexpr int NK = least(8, E4M3 ? (FIT - NV * VSLOT) / SLOT : FIT / SLOT / 2);           // and of K
    static constexpr int SMEM = 2 * QT + NK * SLOT + NV * VSLOT + QMISC + A_MISC;
    static constexpr int KSTEP = E4M3 ? 32 : 16;             // K of one MMA
    // TMEM columns: S (P in its place) and O of each stream
    static constexpr uint32_t T_S = 0, T_O = 256;
};

// One segment's part in a CTA's share.
struct Seg {
    int b, h, c, n;             // request, K/V head, its cached and new tokens
    int row0, tok0, ntok, kt;   // first row of the batch and token of the request, tokens, key tiles of the whole
    int k0, k1, flags, parts;   // this part's key tiles; SEG_*, SEG_TILES; first CTA << 16 | CTAs that hold parts
};
constexpr int SEG_VALID = 1;    // (0: the share is done)
constexpr int SEG_ONCE = 2;     // the request's only pair: its K and V are read once
constexpr uint32_t SEG_TILES = 4;   // times the tiles of the share before the part's first

// The line that shares are cut on: units a key tile with few rows (tokens up to few_tok,
// which stand in copies), with one and with two query tiles, and a segment's own.
struct Units {
    int few_tok, few, one, two, over;
};

// shared-memory tables behind the tiles
struct AMisc {
    Seg seg[SEGS];
    uint64_t seg_full[SEGS], seg_empty[SEGS];
    uint64_t k_full[8], k_empty[8], v_full[8], v_empty[8], q_full[2], q_empty[2], s_full[2], p_full[2][2],
        o_full, o_free, ml_full, qs_full, wg[2], turn[2], drain[2];
    uint32_t tmem;
    int abort;
    int first_b;
    uint32_t landed[3];         // tiles of K, and of V, that have landed (and are clean), and query tiles whose
                                // buffer is free: in order, never reset
    int nan_seg[NAN_SLOTS];
    long long first_off, total;
    Units units;
    int first_c, first_n, first_r0;
    Seg join[2];                // the divided segments: one that began elsewhere, one that ends elsewhere
    float2 ml[2][128];
};
static_assert(sizeof(AMisc) <= A_MISC, "misc");

struct ATabs {
    int G, tpt;                 // heads a group, tokens a query tile
    uint32_t g_inv;             // ceil(2^16 / G): r / G = r g_inv >> 16 for the rows r < 256 of a pair
    int box;                    // keys a TMA box: gcd(page, 128)
    int rp;                     // rows a partial result holds
    float2* part_ml;            // [2 A_CTAS][rp]: m (log2 units), l
    float* part_o;              // [2 A_CTAS][D / 4][rp][4]
    uint32_t* arrived;          // [A_CTAS][2]: warps that have written, and read, the parts of a
                                // segment that begins in this share; 0 between calls
    StatusBlock* sb;
};

// Shares are cut on a line on which a segment takes `over` units for its start and
// end, then `two`, `one` or `few` units a key tile; a share holds the key tiles whose
// first unit lies in it.  Measured: 2.1 us a key tile for two query tiles (bf16, D = 128),
// 1.0 to 1.3 with copies, 4 to 5 us a segment; 2 : 3 : 4 and 10 against one weight for few
// and one, 2 : 3 and 8: 101 us to 109 (trees of 33, whose last token is a tile of its
// own), 69.6 to 70.5 (trees of 8).  With few key tiles a
// share the line is the key tiles themselves, and a share holds one at least
// (shares past the tiles none).
constexpr int LINE_TILES = 8 * A_CTAS;      // (a share of 16 units or more holds a key tile; by key
                                            // tiles alone 78.7 us against 70.5, 144 against 113)
// first unit of share c, and the share that holds unit x
__device__ __forceinline__ long long share_begin(long long total, int c) {
    return total < A_CTAS ? (c < total ? c : total) : total * c / A_CTAS;
}
__device__ __forceinline__ int share_of(long long total, long long x) {
    return total < A_CTAS ? (int)x
           : total >> 24  ? (int)(((x + 1) * A_CTAS - 1) / total)
                          : (int)(((uint32_t)(x + 1) * A_CTAS - 1) / (uint32_t)total);
}

// A cut that falls next to an end of a segment moves there: the parts of a divided
// segment are written, waited for and added, which with many rows takes as long as
// several key tiles (256 rows, D = 128: 8 us).  Up to two tiles, or as many as a share
// holds: a prompt of 512 after 512, 26 us against 34; three prompts of 302, 36 against 43;
// one of 1973, e4m3, 150 against 160; long ones within 1%.  Every CTA moves a cut the same
// way; shares may be left without tiles.
struct Cuts {
    int low = 0, high = 0;      // cuts up to tile `low` move to 0, the last `high` to the end
    __device__ __forceinline__ Cuts(long long total, int kt, int per_tile, int rows) {
        if (rows <= 64) return;
        const int near = total >= 2 * A_CTAS * per_tile ? 2 : total >= A_CTAS * per_tile ? 1 : 0;
        low = near < kt / 2 ? near : kt / 2;
        high = near < (kt - 1) / 2 ? near : (kt - 1) / 2;
    }
    __device__ __forceinline__ int moved(int k, int kt) const { return k <= low ? 0 : k >= kt - high ? kt : k; }
};

// ---------------------------------------------------------------------------
// bounded waits, whole warps
// ---------------------------------------------------------------------------
// A try suspends the warp for up to a microsecond or so: some seconds in all.
// A wait that runs out, or finds that another one did, leaves its number in
// m->abort, and the kernel's end reports it.
constexpr int WAIT_TRIES = 1 << 22;
constexpr int LANDED_TRIES = 1 << 24;       // polls of a counter in shared memory, a second or so
constexpr int JOIN_TRIES = 1 << 22;         // polls of another CTA's counter, two seconds
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, AMisc* m, int site) {
#pragma unroll 1
    for (int i = 0; i < WAIT_TRIES; ++i) {
        if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity, 1000u))) return true;
        if (*(volatile int*)&m->abort) return false;
    }
    *(volatile int*)&m->abort = site;
    return false;
}

// Waits until tile number `tile` (from 0 on) of a ring has landed.
__device__ __forceinline__ bool wait_landed(const uint32_t* landed, uint32_t tile, AMisc* m, int site) {
#pragma unroll 1
    for (int i = 0; i < LANDED_TRIES; ++i) {
        if ((int32_t)(ptx::ld_acquire_cta(landed) - tile) > 0) return true;
        if (*(volatile int*)&m->abort) return false;
        if (i > 8) __nanosleep(40);
    }
    *(volatile int*)&m->abort = site;
    return false;
}

// ---------------------------------------------------------------------------
// segments
// ---------------------------------------------------------------------------
// key tiles of query-tile pair p of a request
__device__ __forceinline__ int pair_tiles(const KvDims& d, const KvReq& r, int p, int pt) {
    const int upto = d.W || (p + 1) * pt > r.n ? r.n : (p + 1) * pt;
    return (r.c + upto + KT - 1) / KT;
}
// units a key tile of pair p of a request
__device__ __forceinline__ int tile_units(const KvReq& r, int p, int pt, Units u) {
    const int n = r.n - p * pt;
    return n > pt / 2 ? u.two : n > u.few_tok ? u.one : u.few;
}
__device__ __forceinline__ long long pair_units(const KvDims& d, const KvReq& r, int p, int pt, Units u) {
    return u.over + (long long)tile_units(r, p, pt, u) * pair_tiles(d, r, p, pt);
}
// units of a request, a K/V head
__device__ __forceinline__ long long head_units(const KvDims& d, const KvReq& r, int pt, Units u) {
    if (r.n == 0) return 0;
    const int np = (r.n + pt - 1) / pt;
    if (d.W) return (np - 1) * pair_units(d, r, 0, pt, u) + pair_units(d, r, np - 1, pt, u);
    long long s = 0;
#pragma unroll 1
    for (int p = 0; p < np; ++p) s += pair_units(d, r, p, pt, u);
    return s;
}

// The segments of a share, in order, one after the other from a warp that only
// does this; every role takes them from the ring.
struct SegIn {
    uint32_t i = 0;
    __device__ __forceinline__ bool next(AMisc* m, Seg& s) {
        const uint32_t k = i % SEGS;
        if (!wait(&m->seg_full[k], (i / SEGS) & 1, m, 1)) return false;
        const int4* const p = reinterpret_cast<const int4*>(&m->seg[k]);
        const int4 x = p[0], y = p[1], z = p[2];
        s = Seg{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w, z.x, z.y, z.z, z.w};
        __syncwarp();
        if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(&m->seg_empty[k]);
        ++i;
        return s.flags & SEG_VALID;
    }
};
// keys below this one are seen by every row of the segment
__device__ __forceinline__ int all_see(const KvDims& d, const Seg& s) { return d.W ? s.c : s.c + s.tok0 + 1; }

// How often a query tile's rows stand in the 128 rows of the product when they
// are few: with 4 (or 2) copies, each warp of a warpgroup makes the weights of
// a quarter (half) of the keys of its copy, instead of one warp those of all.
// The others' weights in its copy are 0; the copies' O are added at the end.
// That pays where a tile's K and V, 32 KB or less, come faster than one warp makes
// its weights: 128 requests of one token, D = 64: e4m3 412 us against 525 without, bf16 443
// against 476.  Tiles of 64 KB do not (904 us and 906), and the sum at the end costs a
// call of few tiles a microsecond (15.4 us and 14.5).  With e4m3 and D = 128 V's codes weigh
// more: 628 us against 643, 64 requests of 32 heads a group 295 against 313; 48 heads, in two
// copies, 334 against 319, and 16 requests of 8 rows 58.5 to 60 against 56.5.
template <int ROWB>
__device__ __forceinline__ int copies(int ntok, const ATabs& t) {
    const int rows = ntok * t.G;
    return ROWB > 128 || ntok > t.tpt || rows > 64 ? 1 : rows > 32 ? 2 : 4;
}

__device__ __forceinline__ int by_g(int r, const ATabs& t) { return (int)(r * t.g_inv >> 16); }

// A position in a ring of N slots, for whoever goes round it in order.
template <int N>
struct Ring {
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void next() {
        if (++slot == N) {
            slot = 0;
            phase ^= 1;
        }
    }
};

// Whether the softmax warps make V's codes f16 (else warp 2 does).
template <int D, bool E4M3>
__host__ __device__ constexpr bool softmax_converts(bool narrow) { return E4M3 && D == 128 && narrow; }

// The weights are relative to a maximum m (kept as mc = m c) that follows the
// true one only when that is LAZY ahead, so that O is rescaled rarely; P stays
// below 2^(base + LAZY).  With an e4m3 cache P is f16, whose smallest step is 2^-24 and
// largest value 65504.  One key may take nearly all of a row's weight while the output is
// made of the others' (a sink), so the maximum stands high: 2^7, at most 2^15.  A weight has
// f16's 11 bits down to 2^-21 of the largest, and below that an error of at most 2^-32 of it.
template <bool E4M3>
__host__ __device__ constexpr float p_base() { return E4M3 ? 7.f : 0.f; }

// One thread's row and COLS keys: the scores at t_s become weights at t_p (bf16 or f16),
// which may lie over them.  When the maximum moves, the row of O at t_o is rescaled
// (no product into it is under way).  half_done() is called once the first half of the weights has been
// stored.  Sums and maxima run in chains of 32 columns and of pairs, so that
// no chain of dependent operations is longer than 16.
template <int D, bool E4M3, int COLS, class HalfDone>
__device__ __forceinline__ void softmax_cols(uint32_t t_s, uint32_t t_p, uint32_t t_o, float c, bool part,
                                             const uint32_t* vis, bool have_o, HalfDone half_done, float& mc, float& l) {
    constexpr float LAZY = 8.f;
    constexpr int N = COLS / 32;
    float s[N][32], tops[2 * N];
#pragma unroll
    for (int k = 0; k < N; ++k) ptx::tmem_ld32(t_s + 32 * k, s[k]);
#pragma unroll
    for (int k = 0; k < N; ++k) ptx::tmem_ld_wait32(s[k]);
    if (part) {
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int x = 0; x < 32; ++x) s[k][x] = (vis[k] >> x) & 1 ? s[k][x] : -CUDART_INF_F;
    }
#pragma unroll
    for (int k = 0; k < 2 * N; ++k) {
        const float* const r = s[k / 2] + 16 * (k & 1);
        tops[k] = fmaxf(r[0], r[1]);
#pragma unroll
        for (int x = 2; x < 16; x += 2) tops[k] = ptx::max3(tops[k], r[x], r[x + 1]);
    }
    float top = tops[0];
#pragma unroll
    for (int k = 1; k < 2 * N - 1; k += 2) top = ptx::max3(top, tops[k], tops[k + 1]);
    top = fmaxf(top, tops[2 * N - 1]) * c;
    const bool first = mc == -CUDART_INF_F;
    const bool move = first || top > mc + LAZY;
    // (a first maximum finds nothing but zeros in its row of O)
    if (have_o && __any_sync(0xffffffffu, move && !first)) {
        const float f = move && !first ? ptx::ex2(mc - top) : 1.f;
        l *= f;
#pragma unroll 1
        for (int x = 0; x < D; x += 16) {
            uint32_t o[16];
            ptx::tmem_ld16(t_o + x, o);
            ptx::tmem_ld_wait16(o);
#pragma unroll
            for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
            ptx::tmem_st16(t_o + x, o);
        }
    }
    if (move) mc = top;
    const float off = mc == -CUDART_INF_F ? 0.f : p_base<E4M3>() - mc;
    const uint64_t c2 = ptx::pack2(c, c), off2 = ptx::pack2(off, off);
    uint64_t sum[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        uint32_t u[16];
#pragma unroll
        for (int x = 0; x < 32; x += 2) {
            float a, b;
            ptx::unpack2(ptx::fma2(ptx::pack2(s[k][x], s[k][x + 1]), c2, off2), a, b);
            a = ptx::ex2(a);
            b = ptx::ex2(b);
            const uint64_t e = ptx::pack2(a, b);
            sum[k] = x == 0 ? e : ptx::add2(sum[k], e);
            s[k][x] = a;
            s[k][x + 1] = b;
        }
#pragma unroll
        for (int x = 0; x < 16; ++x)
            u[x] = E4M3 ? ptx::cvt_f16x2(s[k][2 * x], s[k][2 * x + 1]) : ptx::cvt_bf16x2(s[k][2 * x], s[k][2 * x + 1]);
        ptx::tmem_st16(t_p + 16 * k, u);
        if (N == 4 && k == 1) half_done();
    }
    uint64_t all = sum[0];
#pragma unroll
    for (int k = 1; k < N; ++k) all = ptx::add2(all, sum[k]);
    float a, b;
    ptx::unpack2(all, a, b);
    l += a + b;
}

// ROWS rows of a tile of V's e4m3 codes, from row0 (a multiple of 8) on, as f16, which
// holds every one of them: rows of D bytes become rows of 2 D, both swizzled (a row's
// 16-byte pieces, by its number).  A lane takes one piece of every STEP-th row; where it goes to
// is the same place in every second (D = 64: every) one of them, so the loop only adds to
// addresses.  A warp's reads are 512 bytes in a row, eight under way together; of its writes,
// eight lanes' pieces lie in different banks (D = 128: the second block's pieces go the
// other way round).
template <int D, int ROWS>
__device__ __forceinline__ void v_to_f16(uint8_t* slot, int row0, int lane) {
    constexpr int PIECES = D / 16, STEP = 32 / PIECES;        // 16-byte pieces a row of codes, rows a warp's reads
    constexpr int BATCH = 8;
    static_assert(ROWS % (BATCH * STEP) == 0, "whole batches");
    const int p = lane % PIECES, r0 = lane / PIECES;          // where the piece lies in its row; the first row
    const uint8_t* from = slot + ACfg<D, true>::RAW + row0 * D + lane * 16;
    // D = 128: in rows r0 + 8 i the pieces p >= 4 belong to the second block, in rows r0 + 4 + 8 i the others
    const bool second = D == 128 && p >= 4;
    const int x = D == 128 ? (p ^ r0) & 3 : p ^ (r0 >> 1);    // the piece's number in its block
    int to[2];                                                // bytes from the slot's begin
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int block = D == 128 ? second ^ q : 0;
        to[q] = block * (KT * 128) + (row0 + r0) * 128 + 16 * ((2 * x ^ r0 ^ (D == 128 ? 4 * q : 0)) ^ block);
    }
#pragma unroll 1
    for (int i = 0; i < ROWS / STEP; i += BATCH) {
        uint4 u[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) u[k] = *reinterpret_cast<const uint4*>(from + k * 512);
        __syncwarp();                                         // (their places are written now)
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int q = D == 128 ? k & 1 : 0;
            const bool turn = D == 128 && second != (q != 0); // the second block's: upper half first
            const uint32_t in[4] = {turn ? u[k].z : u[k].x, turn ? u[k].w : u[k].y, turn ? u[k].x : u[k].z,
                                    turn ? u[k].y : u[k].w};
            uint32_t h[8];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                h[2 * y] = ptx::f16x2_of_e4m3(in[y] & 0xFFFF);
                h[2 * y + 1] = ptx::f16x2_of_e4m3(in[y] >> 16);
            }
            uint8_t* const rows = slot + k * (STEP * 128);
            *reinterpret_cast<uint4*>(rows + to[q]) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(rows + (to[q] ^ 16)) = make_uint4(h[4], h[5], h[6], h[7]);
        }
        from += BATCH * 512;
        to[0] += BATCH * STEP * 128;
        to[1] += BATCH * STEP * 128;
    }
}

// What infinities and NaN 16 bytes of V's columns hold over the keys [k0, k1) that
// row i (row `row` of the batch) sees: what the products, which meet 0 * NaN there,
// cannot give.  Two bits a column: 1 an infinity, 2 a negative one, 3 a NaN (or both
// infinities, whose sum it is).  Page by page, four keys' loads under way together: a
// long cache is looked through in milliseconds.
struct VColumn {                // everything by value: the kernel's parameters stay in constant memory
    const void* v;              // the K/V head's columns in page 0
    const int32_t* pages;       // the request's row of the block table
    const uint32_t* mask;       // the row's mask words (chains: null)
    int64_t page_stride, token_stride;
    int page, n_pages, c, i;    // cached tokens, the row's number in its request
};
template <bool E4M3>
__device__ __forceinline__ uint32_t v_specials(VColumn x, int k0, int k1) {
    constexpr int EL = E4M3 ? 16 : 8, AT_ONCE = 4;
    const int64_t token = x.token_stride * (E4M3 ? 1 : 2);
    // all ones in the elements of a word that are not finite
    auto odd = [](uint32_t v) {
        return E4M3 ? __vcmpeq4(v & 0x7F7F7F7Fu, 0x7F7F7F7Fu) : __vcmpeq2(v & 0x7F807F80u, 0x7F807F80u);
    };
    uint32_t found = 0;
#pragma unroll 1
    for (int key = k0; key < k1;) {
        const int p = key / x.page, end = (p + 1) * x.page < k1 ? (p + 1) * x.page : k1;
        const int pg = ld_dep(x.pages + p);
        const uint8_t* at = reinterpret_cast<const uint8_t*>(x.v) + pg * x.page_stride * (E4M3 ? 1 : 2) +
                            (key - p * x.page) * token;
        if (pg < 0 || pg >= x.n_pages) key = end;
#pragma unroll 1
        for (; key < end; key += AT_ONCE, at += AT_ONCE * token) {
            uint4 u[AT_ONCE];
            uint32_t hit = 0;
#pragma unroll
            for (int y = 0; y < AT_ONCE; ++y)
                u[y] = ld_dep(reinterpret_cast<const uint4*>(at + (key + y < end ? y : 0) * token));
#pragma unroll
            for (int y = 0; y < AT_ONCE; ++y) hit |= odd(u[y].x) | odd(u[y].y) | odd(u[y].z) | odd(u[y].w);
            if (!hit) continue;
#pragma unroll 1
            for (int y = 0; y < AT_ONCE && key + y < end; ++y) {
                const int j = key + y - x.c;
                if (j >= 0 && !(x.mask ? (ld_dep(x.mask + (j >> 5)) >> (j & 31)) & 1 : j <= x.i)) continue;
#pragma unroll 1
                for (int e = 0; e < EL; ++e) {
                    uint32_t bits;
                    if (E4M3) {
                        bits = (ld_dep(at + y * token + e) & 0x7F) == 0x7F ? 3 : 0;
                    } else {
                        const uint32_t v = ld_dep(reinterpret_cast<const unsigned short*>(at + y * token) + e);
                        bits = (v & 0x7F80) != 0x7F80 ? 0 : v & 0x7F ? 3 : v >> 15 ? 2 : 1;
                    }
                    found |= bits << (2 * e);
                }
                if (found == (E4M3 ? 0xFFFFFFFFu : 0xFFFFu)) return found;   // (NaN in all of them: no more to learn)
            }
        }
        key = end;
    }
    return found;
}

// Some of a divided segment's output, from its parts: the running maximum moves
// from part to part as from tile to tile.  U items a thread at once, or one by
// SPLIT threads next to each other, each with every SPLIT-th part.
struct JoinWork {
    int i0, i1;                 // items (4 columns of a row)
    int th, nth;                // this thread of the threads that share them
    int rows, c0, parts;        // rows of the segment, first CTA, CTAs that hold parts
    int row0, h;                // first row of the batch, K/V head
};
template <int D, int U, int SPLIT>
__device__ __forceinline__ void join_items(const KvDims& d, const AttnArgs& a, const ATabs& t, const JoinWork& w,
                                           float v_scale) {
    const int sub = w.th % SPLIT, step = w.nth / SPLIT;
#pragma unroll 1
    for (int base = w.i0; base < w.i1; base += step * U) {
        int r[U], x4[U];
        float mx[U], sum[U];
        float4 o[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            int i = base + w.th / SPLIT + step * u;
            if (i >= w.i1) i = w.i0;   // (past the end: the first is done again)
            x4[u] = i / w.rows;
            r[u] = i - x4[u] * w.rows;
            mx[u] = -CUDART_INF_F;
            sum[u] = 0.f;
            o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        auto add = [&](int u, float m2, float s2, float4 q) {
            const float top = fmaxf(mx[u], m2), zero = top == -CUDART_INF_F ? 0.f : top;
            const float f = ptx::ex2(mx[u] - zero), e = s2 == 0.f ? 0.f : ptx::ex2(m2 - zero);
            mx[u] = top;
            sum[u] = sum[u] * f + s2 * e;
            o[u].x = o[u].x * f + q.x * e;
            o[u].y = o[u].y * f + q.y * e;
            o[u].z = o[u].z * f + q.z * e;
            o[u].w = o[u].w * f + q.w * e;
        };
#pragma unroll 2
        for (int k = sub; k < w.parts; k += SPLIT) {
            const int64_t slot = 2 * (w.c0 + k) + (k == 0);
            const float2* const pm = t.part_ml + slot * t.rp;
            const float4* const po = reinterpret_cast<const float4*>(t.part_o) + slot * (D / 4) * t.rp;
            float2 ml[U];
            float4 q[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                ml[u] = ld_dep(pm + r[u]);
                q[u] = ld_dep(po + x4[u] * t.rp + r[u]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) add(u, ml[u].x, ml[u].y, q[u]);
        }
#pragma unroll 1
        for (int s = 1; s < SPLIT; s <<= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, mx[0], s), s2 = __shfl_xor_sync(0xffffffffu, sum[0], s);
            float4 q;
            q.x = __shfl_xor_sync(0xffffffffu, o[0].x, s);
            q.y = __shfl_xor_sync(0xffffffffu, o[0].y, s);
            q.z = __shfl_xor_sync(0xffffffffu, o[0].z, s);
            q.w = __shfl_xor_sync(0xffffffffu, o[0].w, s);
            add(0, m2, s2, q);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (sub != 0) continue;
            const int tk = by_g(r[u], t);
            const int64_t at = (int64_t)(w.row0 + tk) * d.Hq + w.h * t.G + r[u] - tk * t.G;
            const float sc = (sum[u] == 0.f ? 0.f : __fdividef(1.f, sum[u])) * v_scale;
            *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + at * D + 4 * x4[u]) =
                make_uint2(ptx::cvt_bf16x2(o[u].x * sc, o[u].y * sc), ptx::cvt_bf16x2(o[u].z * sc, o[u].w * sc));
            if (a.lse && x4[u] == 0)
                a.lse[at] = sum[u] == 0.f ? -CUDART_INF_F : (mx[u] + log2f(sum[u])) * 0.69314718055994531f;
        }
    }
}

// A query tile as e4m3 rows hi and lo (leading and next 4 significant bits) under
// one power of two a row, in `nc` copies, into the swizzled K-major layout: 8 (4)
// lanes a row, 16 elements a lane; warp wi of nw.  Chains of dependent steps bound it, so
// a lane has many elements, and two rows' loads are under way ahead of the row that is
// made (a rolled loop: code that runs once a segment is fetched anew).
template <int D>
__device__ __forceinline__ void q_terms(const KvDims& d, const AttnArgs& a, const ATabs& t, const Seg& w, int tile, int rows,
                                        int nc, int wi, int nw, uint8_t* hi, float* scale) {
    constexpr int SW = ACfg<D, true>::SW, QT = ACfg<D, true>::QT;
    constexpr int LPR = D / 16, RPW = 32 / LPR, AHEAD = 2;
    const int lane = threadIdx.x & 31, sub = lane % LPR, rs = 128 / nc;
    uint4 q[AHEAD][2];
    auto load = [&](int r, uint4* x) {
        x[0] = x[1] = make_uint4(0, 0, 0, 0);
        if (r >= rows) return;
        const int tk = by_g(r, t);
        const uint4* const from = reinterpret_cast<const uint4*>(
            reinterpret_cast<const uint16_t*>(a.q) + (int64_t)(w.row0 + tile * t.tpt + tk) * d.q_stride +
            (w.h * t.G + r - tk * t.G) * D + sub * 16);
        x[0] = ld_dep(from);
        x[1] = ld_dep(from + 1);
    };
    const int first = wi * RPW + lane / LPR, step = nw * RPW;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) load(first + i * step, q[i]);
#pragma unroll 1
    for (int r = first; r < (rows + RPW - 1) / RPW * RPW; r += step) {
        const uint32_t u[8] = {q[0][0].x, q[0][0].y, q[0][0].z, q[0][0].w, q[0][1].x, q[0][1].y, q[0][1].z, q[0][1].w};
#pragma unroll
        for (int i = 1; i < AHEAD; ++i) {
            q[i - 1][0] = q[i][0];
            q[i - 1][1] = q[i][1];
        }
        load(r + AHEAD * step, q[AHEAD - 1]);
        float f[16], tops[4];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            tops[i] = fmaxf(fmaxf(fabsf(f[4 * i]), fabsf(f[4 * i + 1])), fmaxf(fabsf(f[4 * i + 2]), fabsf(f[4 * i + 3])));
        float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
#pragma unroll
        for (int o = LPR / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        // 2^(134 - e) brings the row's maximum (exponent field e) to [128, 256)
        // (a row below 2^-87 is as good as 0; one with an infinity has NaN scores)
        int e = (int)(__float_as_uint(top) >> 23);
        const bool inf = e == 255;
        e = e < 40 ? 40 : (e > 250 ? 250 : e);
        const float up = __uint_as_float((uint32_t)(261 - e) << 23);
        if (sub == 0) scale[r] = inf ? CUDART_NAN_F : __uint_as_float((uint32_t)(e - 7) << 23);
        uint32_t vh[4], vl[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float y[4], z[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = f[4 * i + k] * up;
            const uint32_t p0 = ptx::cvt_e4m3x2(y[0], y[1]), p1 = ptx::cvt_e4m3x2(y[2], y[3]);
            ptx::e4m3x2_to_f32(p0, z[0], z[1]);
            ptx::e4m3x2_to_f32(p1, z[2], z[3]);
            vh[i] = p0 | p1 << 16;
            vl[i] = ptx::cvt_e4m3x2(y[0] - z[0], y[1] - z[1]) |
                    ptx::cvt_e4m3x2(y[2] - z[2], y[3] - z[3]) << 16;
        }
        // row r of SW bytes, its 16-byte pieces exchanged by the swizzle
        // (copies are a multiple of 32 rows apart: the same exchange)
        const uint32_t chunk = (uint32_t)sub ^ (SW == 128 ? (r & 7) : ((r >> 1) & 3));
#pragma unroll 1
        for (int k = 0; k < nc; ++k) {
            uint8_t* const to = hi + (k * rs + r) * SW + chunk * 16;
            *reinterpret_cast<uint4*>(to) = make_uint4(vh[0], vh[1], vh[2], vh[3]);
            *reinterpret_cast<uint4*>(to + QT / 2) = make_uint4(vl[0], vl[1], vl[2], vl[3]);
        }
    }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(A_THREADS, 1)
    k_tree_attn(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_q8,
                const __grid_constant__ CUtensorMap tm_q1, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const KvDims d, const AttnArgs a, const ATabs t) {
    using C = ACfg<D, E4M3>;
    extern __shared__ __align__(1024) uint8_t sm[];
    uint8_t* const k_ring = sm + 2 * C::QT;
    uint8_t* const v_ring = k_ring + C::NK * C::SLOT;
    float* const q_scale = reinterpret_cast<float*>(v_ring + C::NV * C::VSLOT);   // e4m3: [2][128]
    AMisc* const m = reinterpret_cast<AMisc*>(v_ring + C::NV * C::VSLOT + C::QMISC);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int pt = 2 * t.tpt;
    KT_MARK(K_TREE_ATTN, 0);
    if (ptx::smem_u32(sm) & 1023u) {   // the swizzled tiles need it
        if (tid == 0) latch_status(t.sb, MOE_ERR_CUDA, 0);
        return;
    }
    if (warp == 0) {
        // the barriers, seg_full .. drain, lie one after the other: 1 arrival each but for these
        constexpr int N = (offsetof(AMisc, tmem) - offsetof(AMisc, seg_full)) / 8;
        auto at = [&](const uint64_t* b) { return (int)(b - m->seg_full); };
#pragma unroll 1
        for (int i = lane; i < N; i += 32) {
            uint32_t n = 1;
            if (i >= at(m->seg_empty) && i < at(m->k_full)) n = 15;                          // roles
            if (i >= at(m->k_empty) && i < at(m->v_full)) n = 2;                             // issuers
            if (i >= at(m->v_empty) && i < at(m->q_full)) n = 2;
            if (E4M3 && i >= at(m->q_full) && i < at(m->q_empty)) n = 8;                     // softmax warps
            if (i >= at(m->q_empty) && i < at(m->s_full)) n = 8;                             // softmax warps, or 4 an issuer
            if (i >= at(&m->p_full[0][0]) && i < at(&m->o_full)) n = 4;
            if (i == at(&m->o_full)) n = 2;
            if (i >= at(&m->o_free) && i < at(m->wg)) n = 8;
            if (i >= at(m->wg) && i < at(m->drain)) n = 4;                                   // and turn
            ptx::mbar_init(&m->seg_full[i], n);
        }
        if (lane < NAN_SLOTS) m->nan_seg[lane] = 0;
        if (lane < 2) m->join[lane].parts = 0;
        if (lane < 3) m->landed[lane] = 0;
        if (lane == 0) {
            m->abort = 0;
            ptx::prefetch_tensormap(&tm_k);
            ptx::prefetch_tensormap(&tm_v);
            if (!E4M3) ptx::prefetch_tensormap(&tm_q);
        }
        ptx::fence_mbar_init();
    }
    if (warp == 1) ptx::tmem_alloc(&m->tmem, 512);
    pdl_wait();
    KT_MARK(K_TREE_ATTN, 1);

    // this CTA's share: a scan of the requests' key tiles
    {
        const int per = (d.B + A_THREADS - 1) / A_THREADS;
        const int b0 = tid * per, b1 = b0 + per < d.B ? b0 + per : d.B;
        long long sum = 0, upto = 0, total = 0;       // this thread's requests, those up to them, all
        KvReq r{0, 0, 0, true};
        long long* const part = reinterpret_cast<long long*>(m->ml);   // free until the first segment's end
        Units u{0, 1, 1, 1, 0};
        // first in key tiles; again in the line's units if there are enough of them
#pragma unroll 1
        for (int round = 0;; ++round) {
            sum = 0;
#pragma unroll 1
            for (int b = b0; b < b1; ++b) {
                r = kv_request(d, a.ctx_len, a.row_start, b);
                if (!r.ok && blockIdx.x == 0) latch_status(t.sb, MOE_ERR_BAD_LENGTHS, b);
                sum += head_units(d, r, pt, u) * d.Hkv;
            }
            auto scan = [&](long long v) {
#pragma unroll 1
                for (int o = 1; o < 32; o <<= 1) {
                    const long long x = __shfl_up_sync(0xffffffffu, v, o);
                    if (lane >= o) v += x;
                }
                return v;
            };
            const long long s = scan(sum);
            if (lane == 31) part[16 * round + warp] = s;
            __syncthreads();
            const long long w = scan(lane < A_THREADS / 32 ? part[16 * round + lane] : 0);
            const long long before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
            total = __shfl_sync(0xffffffffu, w, 31);
            upto = (warp > 0 ? before : 0) + s;
            if (round == 1 || total < LINE_TILES) break;
            u = Units{C::ROWB <= 128 ? 64 / t.G : 0, 2, 3, 4, 10};
        }
        long long base = upto - sum;
        const long long pos = share_begin(total, blockIdx.x);
        if (tid == 0) {
            m->total = total;
            m->units = u;
        }
        if (pos >= base && pos < base + sum) {
            int b = b0;
#pragma unroll 1
            for (; per > 1; ++b) {
                r = kv_request(d, a.ctx_len, a.row_start, b);
                const long long n = head_units(d, r, pt, u) * d.Hkv;
                if (pos < base + n) break;
                base += n;
            }
            m->first_b = b;
            m->first_c = r.c;
            m->first_n = r.n;
            m->first_r0 = r.r0;
            m->first_off = pos - base;
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = m->tmem;

    if (warp < 4 || warp >= 12) {
        ptx::reg_dec<72>();
        SegIn in;
        Seg w;
        if (warp == 14) {
            // ---- the share's segments -----------------------------------------
            const long long total = m->total, begin = share_begin(total, blockIdx.x);
            const long long end = share_begin(total, blockIdx.x + 1);
            const Units u = m->units;
            long long at = begin;                         // first unit of the segment
            int b = 0, h = 0, p = 0, np = 1, kt = 0, k0 = 0, per_tile = 1;
            KvReq r{0, 0, 0, true};
            if (begin < end) {
                b = m->first_b;
                r = KvReq{m->first_c, m->first_n, m->first_r0, true};
                np = (r.n + pt - 1) / pt;
                const long long per_head = head_units(d, r, pt, u);
                long long off = m->first_off;
                h = (off | per_head) >> 32 ? (int)(off / per_head) : (int)((uint32_t)off / (uint32_t)per_head);
                off -= h * per_head;
                if (d.W && np > 1) {                      // all pairs but the last are alike
                    const uint32_t n = (uint32_t)pair_units(d, r, 0, pt, u);
                    p = off >> 32 ? (int)(off / n) : (int)((uint32_t)off / n);
                    if (p > np - 1) p = np - 1;
                    off -= (long long)p * n;
                }
#pragma unroll 1
                for (long long n; off >= (n = pair_units(d, r, p, pt, u)); ++p) off -= n;
                at -= off;
                per_tile = tile_units(r, p, pt, u);
                kt = pair_tiles(d, r, p, pt);
                if (off > u.over) k0 = (int)((uint32_t)(off - u.over + per_tile - 1) / (uint32_t)per_tile);
            }
#pragma unroll 1
            for (uint32_t i = 0, tiles = 0;;) {
                const long long left = end - at - u.over;   // units from the segment's first tile to the share's end
                const bool more = begin < end && left > 0;
                const int ntok = r.n - p * pt < pt ? r.n - p * pt : pt;
                const Cuts cuts(total, kt, per_tile, ntok * t.G);
                k0 = cuts.moved(k0, kt);
                const int k1 = cuts.moved(left >= (long long)kt * per_tile
                                              ? kt
                                              : (int)((uint32_t)(left + per_tile - 1) / (uint32_t)per_tile), kt);
                if (!more || k0 < k1) {
                    if (!wait(&m->seg_empty[i % SEGS], ((i / SEGS) & 1) ^ 1, m, 2)) break;
                    if (lane == 0) {
                        Seg* const s = &m->seg[i % SEGS];
                        s->b = b;
                        s->h = h;
                        s->c = r.c;
                        s->n = r.n;
                        s->row0 = r.r0 + p * pt;
                        s->tok0 = p * pt;
                        s->ntok = ntok;
                        s->kt = kt;
                        s->k0 = k0;
                        s->k1 = k1;
                        s->flags = (more ? SEG_VALID : 0) | (np == 1 ? SEG_ONCE : 0) | (int)(tiles * SEG_TILES);
                        s->parts = 0;
                        if (more && (k0 > 0 || k1 < kt)) {   // divided: where its first and last tile are
                            const long long first = at + u.over;
                            const int c0 = share_of(total, first + cuts.low * per_tile);
                            s->parts =
                                c0 << 16 | (share_of(total, first + (long long)(kt - 1 - cuts.high) * per_tile) - c0 + 1);
                        }
                        ptx::mbar_arrive(&m->seg_full[i % SEGS]);
                    }
                    __syncwarp();
                    ++i;
                    tiles += k1 - k0;
                    if (!more) break;
                }
                // (no tiles: the share begins or ends so that they are another's)
                at += u.over + (long long)kt * per_tile;
                k0 = 0;
                if (at + u.over < end) {
                    if (++p == np) {
                        p = 0;
                        if (++h == d.Hkv) {
                            h = 0;
                            do {
                                r = kv_request(d, a.ctx_len, a.row_start, ++b);
                            } while (r.n == 0);
                            np = (r.n + pt - 1) / pt;
                        }
                    }
                    per_tile = tile_units(r, p, pt, u);
                    kt = pair_tiles(d, r, p, pt);
                }
            }
        } else if (warp == 0 || warp == 12) {
            // ---- producers: warp 0 for K, warp 12 for V -------------------------
            // The keys of a part come in boxes of t.box; lane x holds the page of
            // box 32 r + x, so that pages are looked up once for 32 boxes, one
            // round ahead.
            const bool is_v = warp == 12;
            const CUtensorMap* const tm = is_v ? &tm_v : &tm_k;
            uint64_t* const full = is_v ? m->v_full : m->k_full;
            uint64_t* const empty = is_v ? m->v_empty : m->k_empty;
            const uint32_t slots = is_v ? C::NV : C::NK;
            uint8_t* const ring = is_v ? v_ring + C::RAW : k_ring;
            const uint32_t slot_bytes = is_v ? C::VSLOT : C::SLOT;
            uint32_t slot = 0, phase = 0, loads = 0;
            const int nb = KT / t.box;
            bool ok = true;
#pragma unroll 1
            while (ok && in.next(m, w)) {
                const int total = w.c + w.n, mt = w.k1 - w.k0;
                const int32_t* const table = a.block_table + (int64_t)w.b * d.max_pages;
                // (K and V that later segments of the request read again are kept in L2;
                // first out always: prompts 460 us against 432, last out always: 16
                // requests of 8 rows 75.5 us against 70.7)
                const uint64_t pol = w.flags & SEG_ONCE ? ptx::policy_evict_first() : ptx::policy_evict_last();
                const int key_end = total < w.k1 * KT ? total : w.k1 * KT;
                int pg = 0, off = 0, pg2 = 0, off2 = 0;
                int at = 32;                              // first box of the tile in its round; 32: a new round
                int first = w.k0 * KT;                    // key of the next round's look-up
#pragma unroll 1
                for (int j = -1; j < mt; ++j, at += nb) {
                    if (at == 32 || j < 0) {
                        pg = pg2;
                        off = off2;
                        const int key = first + lane * t.box;
                        pg2 = 0;
                        if (key < key_end) {
                            const int q = key / d.page;
                            off2 = key - q * d.page;
                            pg2 = ld_dep(table + q);
                        }
                        first += 32 * t.box;
                        if (j < 0) {                      // the first look-up; the next one follows at once
                            at = 32 - nb;
                            continue;
                        }
                        at = 0;
                        if (pg < 0 || pg >= d.n_pages) {
                            latch_status(t.sb, MOE_ERR_BAD_PAGE, pg);
                            pg = d.n_pages;               // outside: the copy fills zeros
                        }
                    }
                    const int left = total - (w.k0 + j) * KT;
                    const int boxes = left >= KT ? nb : (left + t.box - 1) / t.box;
                    ok = wait(&empty[slot], phase ^ 1, m, 3);
                    if (!ok) break;
                    if (lane == 0) ptx::mbar_arrive_expect_tx(&full[slot], boxes * t.box * C::ROWB);
                    __syncwarp();
                    const int i = lane - at;
                    if (i >= 0 && i < boxes) {
                        uint8_t* const to = ring + slot * slot_bytes + i * t.box * C::SW;
#pragma unroll
                        for (int hf = 0; hf < C::HALVES; ++hf)
                            ptx::tma_load_4d(to + hf * (KT * C::SW), tm, hf * (C::SW / (E4M3 ? 1 : 2)), off, w.h, pg,
                                             &full[slot], pol);
                    }
                    __syncwarp();
                    ++loads;
                    if (++slot == slots) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
            }
            // after a wait ran out, copies in flight land before the CTA's memory is given up
            const int none = 0;
            if (!ok) {
#pragma unroll 1
                for (uint32_t i = loads > slots ? loads - slots : 0; i < loads; ++i)
                    ptx::mbar_wait_warp(&full[i % slots], (i / slots) & 1, &none, 10000000ull);
            }
        } else if (warp == 13 && E4M3) {
            // ---- query tiles of few rows but the first, and leave to make the others' terms
            uint32_t nq = 0;
            bool ok = true;
#pragma unroll 1
            while (ok && in.next(m, w)) {
                const int nt = w.ntok > t.tpt ? 2 : 1, nc = copies<C::ROWB>(w.ntok, t);
#pragma unroll 1
                for (int i = 0; i < nt; ++i, ++nq) {
                    const uint32_t qb = nq & 1;
                    ok = wait(&m->q_empty[qb], ((nq >> 1) & 1) ^ 1, m, 4);
                    if (!ok) break;
                    if (nc > 1 && nq > 0) {
                        q_terms<D>(d, a, t, w, 0, w.ntok * t.G, nc, 0, 1, sm + qb * C::QT, q_scale + qb * 128);
                        ptx::fence_proxy_async_shared();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive_n(&m->q_full[qb], 8);
                    }
                    if (lane == 0) ptx::st_release_cta(&m->landed[2], nq + 1);
                    __syncwarp();
                }
            }
        } else if (warp == 13) {
            // ---- query tiles ----------------------------------------------------
            uint32_t nq = 0;
            bool ok = true;
#pragma unroll 1
            while (ok && in.next(m, w)) {
                const int nt = w.ntok > t.tpt ? 2 : 1, nc = copies<C::ROWB>(w.ntok, t);
#pragma unroll 1
                for (int i = 0; i < nt; ++i, ++nq) {
                    const uint32_t qb = nq & 1;
                    ok = wait(&m->q_empty[qb], ((nq >> 1) & 1) ^ 1, m, 4);
                    if (!ok) break;
                    const int ntok = w.ntok - i * t.tpt < t.tpt ? w.ntok - i * t.tpt : t.tpt;
                    const int row = w.row0 + i * t.tpt, head = w.h * t.G;
                    uint8_t* const dst = sm + qb * C::QT;
                    // whole tiles (rows past ntok are not used), or copies 128 / nc
                    // rows apart, by 8 tokens and by one
                    const int n8 = ntok / 8, per = nc == 1 ? 1 : n8 + ntok % 8;   // boxes of a copy and half
                    if (lane == 0)
                        ptx::mbar_arrive_expect_tx(&m->q_full[qb],
                                                   (nc == 1 ? t.tpt : nc * ntok) * t.G * C::SW * C::HALVES);
                    __syncwarp();
#pragma unroll 1
                    for (int x = lane; x < per * nc * C::HALVES; x += 32) {
                        const int k = x % per, cp = x / per % nc, hf = x / per / nc;
                        const int tk = nc == 1 ? 0 : k < n8 ? 8 * k : 8 * n8 + (k - n8);
                        const CUtensorMap* const tm = nc == 1 ? &tm_q : k < n8 ? &tm_q8 : &tm_q1;
                        ptx::tma_load_3d(dst + (hf * 128 + cp * (128 / nc) + tk * t.G) * C::SW, tm, hf * 64, head,
                                         row + tk, &m->q_full[qb], ptx::policy_evict_last());
                    }
                    __syncwarp();
                }
            }
            const int none = 0;
            if (!ok) {
#pragma unroll 1
                for (uint32_t i = nq > 2 ? nq - 2 : 0; i < nq; ++i)
                    ptx::mbar_wait_warp(&m->q_full[i & 1], (i >> 1) & 1, &none, 10000000ull);
            }
        } else if (warp == 1 || warp == 3) {
            // ---- MMA issuers: warp 1 for stream 0, warp 3 for stream 1 ---------
            // The whole warp walks and waits, one lane issues: descriptors built
            // from values that are the same in the whole warp stay in uniform
            // registers, and a product costs a few instructions.  Tiles are waited for
            // by count, not by their barriers' phases, so that an issuer can pass over
            // the tiles of the other stream (a phase may be two ahead, which a parity
            // wait takes for none); who uses a tile alone releases it for both.
            // S of the stream's next tile is begun right after the product with
            // this one's weights, in whose place it lies; that product in two
            // halves, the first while the weights of the second are made (one go
            // where rows are few).  Waits come before the one for P, which ends a
            // tile's critical path.
            constexpr uint32_t id_s = ptx::idesc_attn(E4M3, 128, KT, false);
            constexpr uint32_t id_o = ptx::idesc_attn(E4M3, 128, D, true);   // (f16 has e4m3's number)
            const int s = warp >> 1;
            uint32_t nq = 0, n_p0 = 0, n_p1 = 0, n_seg = 0;
            uint32_t base = 0;                                                 // the segment's first tile in the rings
            bool ok = true;
            const uint32_t sm0 = ptx::smem_u32(sm), k0 = ptx::smem_u32(k_ring), v0 = ptx::smem_u32(v_ring);
            const uint32_t t_s = tmem + C::T_S + s * 128, t_o = tmem + C::T_O + s * 128;
            auto same = [](uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); };
#pragma unroll 1
            for (; ok && in.next(m, w); ++n_seg) {
                const int mt = w.k1 - w.k0;
                const bool two = w.ntok > t.tpt, narrow = copies<C::ROWB>(w.ntok, t) > 1;
                const int step = two ? 1 : 2, first = two ? 0 : s;             // own tiles: first, first + step, ...
                const uint32_t nq_s = nq + (two ? s : 0), qb = same(nq_s & 1);
                const uint32_t qd = ptx::smem_desc_lo(sm0 + qb * C::QT, 16);
                ok = wait(&m->q_full[qb], (nq_s >> 1) & 1, m, 5);
                // the previous segment's O is read before the first product into it
                bool o_free = n_seg == 0, add = false;
                // step j: V of tile j and K of the stream's next one
#pragma unroll 1
                for (int j = first - step; j < mt && ok; j += step) {
                    const bool nx = j + step < mt;
                    const uint32_t ks = same((base + j + step) % C::NK), vs = same((base + j) % C::NV);
                    if (nx) ok = wait_landed(&m->landed[0], base + j + step, m, 6);
                    if (j >= 0) ok = ok && wait_landed(&m->landed[1], base + j, m, 7);
                    if (j >= 0 && !o_free && ok) {
                        ok = wait(&m->o_free, (n_seg - 1) & 1, m, 8);
                        o_free = true;
                    }
                    const uint32_t vd = ptx::smem_desc_lo(v0 + vs * C::VSLOT, KT * 128);
                    const uint32_t kd = ptx::smem_desc_lo(k0 + ks * C::SLOT, 16);
#pragma unroll 1
                    for (uint32_t half = j < 0 ? 1 : 0; half < 2 && ok; ++half) {
                        if (j >= 0 && (half == 0 || !narrow)) {
                            ok = wait(&m->p_full[s][half], (half ? n_p1 : n_p0) & 1, m, 9);
                            if (!ok) break;
                            if (half)
                                ++n_p1;
                            else
                                ++n_p0;
                        }
                        ptx::tc_fence_after();
                        const uint32_t more_o = same(add);
                        if (ptx::elect_one()) {
                            if (j >= 0) {   // O += P V, 64 keys
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    ptx::mma_ts(t_o, t_s + half * 32 + e * 8,
                                                ptx::smem_desc<128>(vd + (half * 64 + e * 16) * 128 / 16), id_o,
                                                e ? 1u : more_o);
                                if (half) {
                                    ptx::mma_commit(&m->v_empty[vs]);
                                    if (!two) ptx::mma_commit(&m->v_empty[vs]);
                                }
                            }
                            if (half && nx) {       // S = Q K^T
#pragma unroll
                                for (int part = 0; part < (E4M3 ? 2 : 1); ++part) {
#pragma unroll
                                    for (int e = 0; e < D / C::KSTEP; ++e) {
                                        const uint32_t o = ((e * 32) / C::SW * (128 * C::SW) + (e * 32) % C::SW) >> 4;
                                        ptx::mma_ss<E4M3>(t_s, ptx::smem_desc<C::SW>(qd + part * (C::QT / 2 >> 4) + o),
                                                          ptx::smem_desc<C::SW>(kd + o), id_s, (part | e) ? 1u : 0u);
                                    }
                                }
                                ptx::mma_commit(&m->s_full[s]);
                                ptx::mma_commit(&m->k_empty[ks]);
                                if (!two) ptx::mma_commit(&m->k_empty[ks]);
                            }
                        }
                        __syncwarp();
                        add = j >= 0;
                    }
                }
                // (a stream without tiles keeps step with the segments)
                if (ok && !o_free) ok = wait(&m->o_free, (n_seg - 1) & 1, m, 12);
                if (!ok) break;
                if (ptx::elect_one()) {
                    ptx::mma_commit(&m->o_full);
                    // every product of this stream is issued, those that read Q among them
                    // (of few rows, the epilogue uses Q's memory and releases it)
                    if (!narrow) {
#pragma unroll 1
                        for (int i = 0; i < 4; ++i) {
                            ptx::mma_commit(&m->q_empty[nq & 1]);
                            if (two) ptx::mma_commit(&m->q_empty[(nq + 1) & 1]);
                        }
                    }
                }
                __syncwarp();
                nq += two ? 2 : 1;
                base += mt;
            }
            if (!ok) {
                // products in flight end before TMEM and shared memory are given up
                const int none = 0;
                if (ptx::elect_one()) ptx::mma_commit(&m->drain[s]);
                __syncwarp();
                ptx::mbar_wait_warp(&m->drain[s], 0, &none, 10000000ull);
            }
        } else if (warp == 2) {
            // ---- V tiles with keys that some row does not see ------------------
            // A key past the end, or one that holds NaN or an infinity, must not
            // reach rows whose weight for it is 0 (0 * NaN).  Rows of V past the end
            // are zeroed; non-finite entries of new tokens too, and the segment is
            // flagged, so that its epilogue puts them where they are seen.
            // Every V tile passes through this warp, which counts them.
            uint32_t tiles = 0;
            Ring<C::NV> vr;
            bool ok = true;
#pragma unroll 1
            for (int seg = 0; ok && in.next(m, w); ++seg) {
                const int mt = w.k1 - w.k0, total = w.c + w.n, see = all_see(d, w);
                const bool convert = E4M3 && !softmax_converts<D, E4M3>(copies<C::ROWB>(w.ntok, t) > 1);
#pragma unroll 1
                for (int j = 0; j < mt; ++j, vr.next()) {
                    const int key0 = (w.k0 + j) * KT;
                    ok = wait(&m->v_full[vr.slot], vr.phase, m, 13);
                    if (!ok) break;
                    if (key0 + KT > see) {
                        const int r0 = see > key0 ? see - key0 : 0, r1 = total - key0 < KT ? total - key0 : KT;
                        uint32_t bad = 0;
#pragma unroll 1
                        for (int hf = 0; hf < C::HALVES; ++hf) {
                            uint8_t* const v = v_ring + vr.slot * C::VSLOT + C::RAW + hf * (KT * C::SW);
#pragma unroll 1
                            for (int o = r1 * C::SW + lane * 16; o < KT * C::SW; o += 512)
                                *reinterpret_cast<uint4*>(v + o) = make_uint4(0, 0, 0, 0);
#pragma unroll 1
                            for (int o = r0 * C::SW + lane * 16; o < r1 * C::SW; o += 512) {
                                uint4 x = *reinterpret_cast<uint4*>(v + o);
                                uint32_t* const u = reinterpret_cast<uint32_t*>(&x);
                                uint32_t hit = 0;
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    // all ones in the elements that are not finite
                                    const uint32_t z = E4M3 ? __vcmpeq4(u[i] & 0x7F7F7F7Fu, 0x7F7F7F7Fu)
                                                            : __vcmpeq2(u[i] & 0x7F807F80u, 0x7F807F80u);
                                    u[i] &= ~z;
                                    hit |= z;
                                }
                                if (hit) *reinterpret_cast<uint4*>(v + o) = x;
                                bad |= hit;
                            }
                        }
                        ptx::fence_proxy_async_shared();
                        bad = __any_sync(0xffffffffu, bad != 0);
                        if (bad && lane == 0) *(volatile int*)&m->nan_seg[seg % NAN_SLOTS] = seg + 1;
                        __syncwarp();
                    }
                    if (convert) {
                        v_to_f16<D, KT>(v_ring + vr.slot * C::VSLOT, 0, lane);
                        ptx::fence_proxy_async_shared();
                        __syncwarp();
                    }
                    if (lane == 0) ptx::st_release_cta(&m->landed[1], ++tiles);
                    __syncwarp();
                }
            }
        } else if (warp == 15) {
            // ---- K tiles are counted ---------------------------------------------
            Ring<C::NK> kr;
            uint32_t tiles = 0;
            bool ok = true;
#pragma unroll 1
            while (ok && in.next(m, w)) {
#pragma unroll 1
                for (int j = w.k0; j < w.k1; ++j, kr.next()) {
                    ok = wait(&m->k_full[kr.slot], kr.phase, m, 10);
                    if (!ok) break;
                    if (lane == 0) ptx::st_release_cta(&m->landed[0], ++tiles);
                    __syncwarp();
                }
            }
        }
    } else {
        // ---- softmax: warpgroup g, thread = row -------------------------------
        ptx::reg_inc<184>();
        SegIn in;
        Seg w;
        const int g = (warp - 4) >> 2, wq = warp & 3, row = 32 * wq + lane;
        const uint32_t lanes = (uint32_t)(32 * wq) << 16;
        const uint32_t t_s = tmem + lanes + C::T_S + g * 128, t_o = tmem + lanes + C::T_O + g * 128;
        uint32_t n_s = 0, nq = 0, n_seg = 0, n_ml = 0, n_wg = 0, n_qs = 0, n_turn = 0;
        bool ok = true;
#pragma unroll 1
        for (; ok && in.next(m, w); ++n_seg) {
            const int mt = w.k1 - w.k0, see = all_see(d, w);
            const bool two = w.ntok > t.tpt;
            const int nc = copies<C::ROWB>(w.ntok, t), rs = 128 / nc;             // copies of the rows, lanes each has
            const int cp = row / rs, rl = row % rs;                      // this thread's copy, and row in it
            const int qs = two ? g : 0;                                  // this stream's query tile
            const int ntok = w.ntok - qs * t.tpt < t.tpt ? w.ntok - qs * t.tpt : t.tpt;
            const int rows = ntok * t.G;
            const bool live = 32 * wq % rs < rows;                       // a warp without rows only keeps step
            const int tok = qs * t.tpt + by_g(rl, t);                     // token of the segment (rl < rows)
            const uint32_t qb = (nq + qs) & 1;
            float c = d.scale * 1.4426950408889634f;
            if (E4M3) {
                // wide tiles, and a CTA's first: these warps make the e4m3 terms, once the
                // buffer is free; else warp 13 does, ahead of them
                c *= ld_dep(a.k_scale + w.h);
                if (nc == 1 || n_seg == 0) {
                    ok = wait_landed(&m->landed[2], nq + qs, m, 14);
                    if (!ok) break;
                    q_terms<D>(d, a, t, w, qs, rows, nc, two ? wq : warp - 4, two ? 4 : 8, sm + qb * C::QT,
                               q_scale + qb * 128);
                    ptx::fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        ptx::mbar_arrive_n(&m->q_full[qb], two ? 2 : 1);
                        ptx::mbar_arrive(&m->qs_full);
                    }
                    ok = wait(&m->qs_full, n_qs & 1, m, 15);             // the row scales are there
                    ++n_qs;
                } else {
                    ok = wait(&m->q_full[qb], (nq >> 1) & 1, m, 15);
                }
                if (!ok) break;
                c *= q_scale[qb * 128 + rl];
            }
            float mc = -CUDART_INF_F, l = 0.f;
            const int step = two ? 1 : 2;
#pragma unroll 1
            for (int j = two ? 0 : g; j < mt; j += step) {
                const int key0 = (w.k0 + j) * KT;
                const bool part = key0 + KT > see;
                uint32_t vis[4] = {~0u, ~0u, ~0u, ~0u};
                if (part && live) {
                    if (d.W == 0) {
                        const int n = w.c + w.tok0 + tok + 1 - key0;     // keys of the tile the row sees
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            vis[k] = n >= 32 * k + 32 ? ~0u : (n <= 32 * k ? 0u : (1u << (n - 32 * k)) - 1u);
                    } else {
                        // bit x of the tile is new token key0 + x - c
                        uint32_t words[5];
                        const int j0 = key0 - w.c, word0 = j0 >> 5;
                        const uint32_t* const mr = a.mask + (int64_t)(w.row0 + tok) * d.W;
#pragma unroll
                        for (int k = 0; k < 5; ++k) {
                            const int x = word0 + k, n = w.n - 32 * x;
                            uint32_t v = x < 0 ? ~0u : 0u;
                            if (x >= 0 && n > 0 && rl < rows) {
                                v = ld_dep(mr + x);
                                if (n < 32) v &= (1u << n) - 1u;
                            }
                            words[k] = v;
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) vis[k] = __funnelshift_r(words[k], words[k + 1], j0 & 31);
                    }
                }
                ok = wait(&m->s_full[g], n_s & 1, m, 16);
                if (!ok) break;
                ++n_s;
                ptx::tc_fence_after();
                const bool have_o = j >= step;
                auto stored = [&](int half) {
                    ptx::tmem_st_wait();
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&m->p_full[g][half]);
                };
                auto nothing = [] {};
                int last_half = 0;
                // The warpgroups take turns: two at once would each take longer, and
                // reach the tensor core together, which then waits for both.
                if (g == 1 || n_turn > 0) ok = wait(&m->turn[g], (n_turn - (g ^ 1)) & 1, m, 20);
                if (!ok) break;
                ++n_turn;
                auto hand_over = [&] {
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&m->turn[g ^ 1]);
                };
                if (nc == 4) {
                    // this warp's quarter of the keys; the other quarters' weights are 0 in its rows
                    const uint32_t v = cp == 0 ? vis[0] : cp == 1 ? vis[1] : cp == 2 ? vis[2] : vis[3];
                    softmax_cols<D, E4M3, 32>(t_s + 32 * cp, t_s + 16 * cp, t_o, c, part, &v, have_o, nothing, mc, l);
                    hand_over();
#pragma unroll 1
                    for (int k = 1; k < 4; ++k) ptx::tmem_st16_rep(t_s + 16 * ((cp + k) & 3), 0);
                } else if (nc == 2) {
                    const uint32_t v[2] = {cp ? vis[2] : vis[0], cp ? vis[3] : vis[1]};
                    softmax_cols<D, E4M3, 64>(t_s + 64 * cp, t_s + 32 * cp, t_o, c, part, v, have_o, nothing, mc, l);
                    hand_over();
                    const uint32_t other = t_s + 32 * (cp ^ 1);
                    ptx::tmem_st16_rep(other, 0);
                    ptx::tmem_st16_rep(other + 16, 0);
                } else {
                    last_half = 1;
                    auto half_done = [&] {
                        stored(0);
                        if (lane == 0) ptx::mbar_arrive(&m->turn[g ^ 1]);
                    };
                    if (live)
                        softmax_cols<D, E4M3, 128>(t_s, t_s, t_o, c, part, vis, have_o, half_done, mc, l);
                    else
                        half_done();
                }
                if constexpr (softmax_converts<D, E4M3>(true)) {
                    if (nc > 1) {
                        // this warp's quarter of V's tile, handed over with the weights
                        const uint32_t tile = (uint32_t)w.flags / SEG_TILES + j;
                        ok = wait_landed(&m->landed[1], tile, m, 22);
                        if (!ok) break;
                        v_to_f16<D, KT / 4>(v_ring + tile % C::NV * C::VSLOT, 32 * wq, lane);
                        ptx::fence_proxy_async_shared();
                        __syncwarp();
                    }
                }
                stored(last_half);
            }
            if (!ok) break;
            if (!two && g == 1 && mt % 2) {                   // the turn of a tile that stream 1 does not have
                ok = wait(&m->turn[1], n_turn & 1, m, 21);
                if (!ok) break;
                ++n_turn;
                if (lane == 0) ptx::mbar_arrive(&m->turn[0]);
            }
            nq += two ? 2 : 1;
            ok = wait(&m->o_full, n_seg & 1, m, 17);
            if (!ok) break;
            ptx::tc_fence_after();
            // ---- the segment's end ------------------------------------------
            const bool whole = w.k0 == 0 && w.k1 == w.kt;
            const int slot = 2 * blockIdx.x + (w.k0 == 0 ? 1 : 0);       // of a partial result
            const bool flagged = *(volatile int*)&m->nan_seg[n_seg % NAN_SLOTS] == (int)n_seg + 1;
            const float v_scale = E4M3 ? ld_dep(a.v_scale + w.h) : 1.f;
            if (!two) {
                m->ml[g][row] = make_float2(mc, l);
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&m->ml_full);
                ok = wait(&m->ml_full, n_ml & 1, m, 18);
                if (!ok) break;
                ++n_ml;
            }
            // a part that saw nothing adds nothing (its O may never have been written)
            auto factor = [](float2 x, float top) {
                return x.x == -CUDART_INF_F && !(x.y != x.y) ? 0.f : ptx::ex2(x.x - top);
            };
            // where row r (of tile qs) and column x of this segment go
            auto out_at = [&](int tk, int r, int x) {
                return ((int64_t)(w.row0 + tk) * d.Hq + w.h * t.G + r - by_g(r, t) * t.G) * D + x;
            };
            // a partial result's O stands by 4 columns: [slot][D / 4][rows][4], so that a
            // warp's rows are written next to each other
            auto part_row = [&](int r) { return (int64_t)slot * t.rp + qs * t.tpt * t.G + r; };
            auto part_at = [&](int r, int x) {
                return t.part_o + (((int64_t)slot * (D / 4) + x / 4) * t.rp + qs * t.tpt * t.G + r) * 4;
            };
            auto put_ml = [&](int tk, int r, float top, float zero, float sum) {
                // log2 of the sum, without the weights' 2^base
                if (!whole)
                    t.part_ml[part_row(r)] = make_float2(top - p_base<E4M3>(), sum);
                else if (a.lse)
                    a.lse[out_at(tk, r, 0) / D] =
                        sum == 0.f ? -CUDART_INF_F : (zero - p_base<E4M3>() + log2f(sum)) * 0.69314718055994531f;
            };
            uint32_t odd = 0;                                            // copies: pieces that are not finite
            if (nc == 1) {
                // one query tile: both streams' O of a row, half its columns a warpgroup
                float2 x0 = make_float2(mc, l), x1 = make_float2(-CUDART_INF_F, 0.f);
                if (!two) x1 = m->ml[g ^ 1][row];
                const float top = fmaxf(x0.x, x1.x), zero = top == -CUDART_INF_F ? 0.f : top;
                float f0 = factor(x0, zero), f1 = factor(x1, zero);
                const float sum = x0.y * f0 + x1.y * f1;
                const float scale = whole ? (sum == 0.f ? 0.f : 1.f / sum) * v_scale : 1.f;
                f0 *= scale;
                f1 *= scale;
                if (live) {
                    const int c0 = two ? 0 : g * (D / 2), c1 = two ? D : c0 + D / 2;
#pragma unroll 1
                    for (int x = c0; x < c1; x += 16) {
                        uint32_t u[16], v[16];
                        ptx::tmem_ld16(t_o + x, u);
                        ptx::tmem_ld16((two ? t_o : tmem + lanes + C::T_O + (g ^ 1) * 128) + x, v);
                        ptx::tmem_ld_wait16(u);
                        ptx::tmem_ld_wait16(v);
                        float o[16];
#pragma unroll
                        for (int y = 0; y < 16; ++y)
                            o[y] = (f0 != 0.f ? __uint_as_float(u[y]) * f0 : 0.f) +
                                   (f1 != 0.f ? __uint_as_float(v[y]) * f1 : 0.f);
                        if (row < rows && whole) {
                            uint32_t z[8];
#pragma unroll
                            for (int y = 0; y < 8; ++y) z[y] = ptx::cvt_bf16x2(o[2 * y], o[2 * y + 1]);
                            uint4* const to =
                                reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.out) + out_at(tok, row, x));
                            to[0] = make_uint4(z[0], z[1], z[2], z[3]);
                            to[1] = make_uint4(z[4], z[5], z[6], z[7]);
                        } else if (row < rows) {
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                *reinterpret_cast<float4*>(part_at(row, x + 4 * y)) =
                                    make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
                        }
                    }
                    if (row < rows && (two || g == 0)) put_ml(tok, row, top, zero, sum);
                }
            } else {
                // few rows: the copies' and streams' O of a row are added through the
                // memory of Q, half the columns a warpgroup, in two passes (one where
                // all of them fit)
                auto group_sync = [&] {
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&m->wg[g]);
                    return wait(&m->wg[g], n_wg++ & 1, m, 19);
                };
                const int passes = nc * rows > 64 ? 2 : 1, cols = D / 2 / passes, w4 = cols / 4;
                const int srow = cp * (passes == 1 ? rows : rs) + rl;    // this thread's row in the stage
                float4* const stage = reinterpret_cast<float4*>(sm + qb * C::QT + g * (C::QT / 2));
                auto piece = [&](int r, int k) { return r * w4 + (k ^ (r & (w4 - 1))); };   // spread over the banks
                float top = -CUDART_INF_F, sum = 0.f;
#pragma unroll 1
                for (int k = 0; k < nc; ++k) top = ptx::max3(top, m->ml[0][k * rs + rl].x, m->ml[1][k * rs + rl].x);
                const float zero = top == -CUDART_INF_F ? 0.f : top;
#pragma unroll 1
                for (int k = 0; k < nc; ++k) {
                    const float2 x0 = m->ml[0][k * rs + rl], x1 = m->ml[1][k * rs + rl];
                    sum += x0.y * factor(x0, zero) + x1.y * factor(x1, zero);
                }
                const float scale = whole ? (sum == 0.f ? 0.f : 1.f / sum) * v_scale : 1.f;
                const float f0 = factor(m->ml[0][row], zero) * scale, f1 = factor(m->ml[1][row], zero) * scale;
                if (g == 0 && row < rows) put_ml(tok, row, top, zero, sum);
#pragma unroll 1
                for (int pass = 0; pass < passes && ok; ++pass) {
                    const int x0 = g * (D / 2) + pass * cols;
                    if (pass == 1) ok = group_sync();                    // the first pass has been read
                    if (!ok) break;
#pragma unroll 1
                    for (int x = 0; x < cols; x += 16) {
                        uint32_t u[16], v[16];
                        ptx::tmem_ld16(tmem + lanes + C::T_O + x0 + x, u);
                        ptx::tmem_ld16(tmem + lanes + C::T_O + 128 + x0 + x, v);
                        ptx::tmem_ld_wait16(u);
                        ptx::tmem_ld_wait16(v);
                        if (rl < rows) {
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                float o[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    o[e] = (f0 != 0.f ? __uint_as_float(u[4 * y + e]) * f0 : 0.f) +
                                           (f1 != 0.f ? __uint_as_float(v[4 * y + e]) * f1 : 0.f);
                                stage[piece(srow, x / 4 + y)] = make_float4(o[0], o[1], o[2], o[3]);
                            }
                        }
                        __syncwarp();
                    }
                    ok = group_sync();
                    if (!ok) break;
                    const int next = passes == 1 ? rows : rs, sh = passes == 1 ? (D == 128 ? 4 : 3) : (D == 128 ? 3 : 2);
#pragma unroll 1
                    for (int i = row, item = 1 << 4 * pass; i < rows << sh; i += 128, item <<= 1) {
                        const int r = i >> sh, k = i & (w4 - 1), x = x0 + 4 * k, tk = by_g(r, t);
                        float4 z = stage[piece(r, k)];
#pragma unroll 1
                        for (int e = 1; e < nc; ++e) {
                            const float4 q = stage[piece(e * next + r, k)];
                            z.x += q.x; z.y += q.y; z.z += q.z; z.w += q.w;
                        }
                        if (whole)
                            *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + out_at(tk, r, x)) =
                                make_uint2(ptx::cvt_bf16x2(z.x, z.y), ptx::cvt_bf16x2(z.z, z.w));
                        else
                            *reinterpret_cast<float4*>(part_at(r, x)) = z;
                        if (!E4M3 && !isfinite(z.x + z.y + z.z + z.w)) odd |= item;
                    }
                }
                if (!ok) break;
                ptx::fence_proxy_async_shared();                         // Q's next tile comes by TMA
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&m->q_empty[qb]);
            }
            // Entries of V that were cleaned and are seen; and, with copies, whose weights of 0 make NaN of
            // a seen infinity, all that are not finite.  (e4m3 has no infinity, and a NaN that every row
            // sees is right as it is.)  This warp's pieces of four columns one after the other, the keys
            // shared among the lanes.
            if (flagged || (!E4M3 && C::ROWB <= 128 && __any_sync(0xffffffffu, odd != 0))) {
                constexpr int EL = E4M3 ? 16 : 8;
                const int key_0 = w.k0 * KT, key_1 = w.c + w.n < w.k1 * KT ? w.c + w.n : w.k1 * KT;
                const int cleaned = see < key_0 ? key_0 : see;           // the first key that was cleaned
                const int passes = nc * rows > 64 ? 2 : 1, sh = (D == 128 ? 5 : 4) - passes;
                const int items = nc > 1 ? 8 : two ? D / 4 : D / 8;
#pragma unroll 1
                for (int item = 0; item < items; ++item) {
                    int r = row, x = (two ? 0 : g * (D / 2)) + 4 * item;
                    bool special = row < rows;
                    if (nc > 1) {                                        // as the loop above goes
                        const int i = row + 128 * (item & 3), pass = item >> 2;
                        r = i >> sh;
                        x = g * (D / 2) + pass * (D / 4) + 4 * (i & ((1 << sh) - 1));
                        special = r < rows && pass < passes && (flagged || (odd >> item & 1));
                    }
                    if (special) {                                       // (scores that are NaN have a NaN sum)
                        float sum = two ? l : 0.f;
                        for (int e = 0; !two && e < nc; ++e) sum += m->ml[0][e * rs + r].y + m->ml[1][e * rs + r].y;
                        special = !(sum != sum);
                    }
                    const int tk = nc > 1 ? by_g(r, t) : tok;
#pragma unroll 1
                    for (uint32_t left = __ballot_sync(0xffffffffu, special); left; left &= left - 1) {
                        const int from = __ffs(left) - 1;
                        const int sx = __shfl_sync(0xffffffffu, x, from), stk = __shfl_sync(0xffffffffu, tk, from);
                        const int first = __shfl_sync(0xffffffffu, odd >> item & 1, from) ? key_0 : cleaned;
                        const int each = (key_1 - first + 31) / 32, mine = first + lane * each;
                        VColumn col;
                        col.v = reinterpret_cast<const uint8_t*>(a.v_cache) +
                                (w.h * d.head_stride + sx / EL * EL) * (E4M3 ? 1 : 2);
                        col.pages = a.block_table + (int64_t)w.b * d.max_pages;
                        col.mask = d.W ? a.mask + (int64_t)(w.row0 + stk) * d.W : nullptr;
                        col.page_stride = d.page_stride;
                        col.token_stride = d.token_stride;
                        col.page = d.page;
                        col.n_pages = d.n_pages;
                        col.c = w.c;
                        col.i = w.tok0 + stk;
                        const uint32_t found = __reduce_or_sync(
                            0xffffffffu, v_specials<E4M3>(col, mine, mine + each < key_1 ? mine + each : key_1));
                        if (lane != from) continue;
#pragma unroll 1
                        for (int y = 0; y < 4; ++y) {
                            const uint32_t bits = found >> (2 * (x % EL + y)) & 3;
                            if (bits == 0) continue;
                            const float e = bits == 3 ? CUDART_NAN_F : bits == 2 ? -CUDART_INF_F : CUDART_INF_F;
                            if (whole)
                                reinterpret_cast<__nv_bfloat16*>(a.out)[out_at(tk, r, x + y)] = __float2bfloat16_rn(e);
                            else
                                part_at(r, x)[y] = e;
                        }
                    }
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive(&m->o_free);
                if (!whole) {
                    // (every warp leaves the same, and reads what it has left)
                    m->join[w.k0 == 0] = w;
                    // this warp's rows of the part are written: who counts them sees them
                    ptx::red_release_gpu_add(t.arrived + 2 * (w.parts >> 16), 1);
                }
            }
        }
        // ---- divided segments --------------------------------------------------
        // The CTAs that hold parts of a segment are few and all run (the launch is
        // cooperative); each has written all its parts before it waits here.
        __syncwarp();
        const Seg* const mine = m->join;
        if (ok && lane < 2 && mine[lane].parts) {
            const int parts = mine[lane].parts;
            const uint32_t* const arrived = t.arrived + 2 * (parts >> 16);
#pragma unroll 1
            for (int i = 0; ptx::ld_acquire_gpu(arrived) != 8u * (parts & 0xFFFF); ++i) {
                if (i == JOIN_TRIES || *(volatile int*)&m->abort) {
                    *(volatile int*)&m->abort = 23;
                    ok = false;
                    break;
                }
                __nanosleep(i < 16 ? 32 : 500);
            }
        }
        __syncwarp();
        ok = __all_sync(0xffffffffu, ok);
        // two segments: one a warpgroup; one: both take it
        const bool both = mine[0].parts && mine[1].parts;
#pragma unroll 1
        for (int x = 0; x < 2 && ok; ++x) {
            w = mine[x];
            if (w.parts == 0) continue;
            const int c0 = w.parts >> 16, parts = w.parts & 0xFFFF;
            uint32_t* const arrived = t.arrived + 2 * c0;
            const int rows = w.ntok * t.G, at = blockIdx.x - c0;
            const float v_scale = E4M3 ? ld_dep(a.v_scale + w.h) : 1.f;
            if (!both || x == g) {
                // 4 columns of a row an item.  Where a thread has several, four at once: the
                // loads of a part for all of them, and of the next part, are under way
                // together (256 rows and 3 parts: 10 us against 18 us one by one).  Where
                // there are few, four threads an item, each with every fourth part.
                const int all = rows * (D / 4), th = both ? row : tid - 128, nth = both ? 128 : 256;
                const JoinWork jw{(int)((long long)all * at / parts), (int)((long long)all * (at + 1) / parts),
                                  th, nth, rows, c0, parts, w.row0, w.h};
                if (jw.i1 - jw.i0 > nth)
                    join_items<D, 4, 1>(d, a, t, jw, v_scale);
                else
                    join_items<D, 1, 4>(d, a, t, jw, v_scale);
            }
            // the last warp past the wait leaves the counters as it found them
            __syncwarp();
            if (lane == 0 && atomicAdd(arrived + 1, 1u) == 8u * parts - 1) {
                arrived[0] = 0;
                arrived[1] = 0;
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_dealloc(tmem, 512);
    if (tid == 0 && m->abort) latch_status(t.sb, MOE_ERR_TIMEOUT, 200 + m->abort);
    KT_MARK(K_TREE_ATTN, 2);
}

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

ATabs attn_tabs(const KvDims& d, char* ws, size_t* bytes) {
    ATabs t{};
    t.G = d.Hq / d.Hkv;
    t.tpt = 128 / t.G;
    t.g_inv = (65536u + t.G - 1) / t.G;
    t.box = gcd(d.page, KT);
    const int64_t tokens = d.T < 2 * t.tpt ? d.T : 2 * t.tpt;
    t.rp = (int)(tokens * t.G);
    size_t o = sizeof(StatusBlock);
    auto take = [&](size_t n) { const size_t at = o; o = (o + n + 255) & ~(size_t)255; return at; };
    const size_t arrived = take(A_CTAS * 2 * sizeof(uint32_t));   // in the prefix that moe_workspace_init clears
    static_assert(sizeof(StatusBlock) + A_CTAS * 2 * sizeof(uint32_t) <= WS_ZERO_PREFIX, "zeroed prefix");
    if (o < WS_ZERO_PREFIX) o = (WS_ZERO_PREFIX + 255) & ~(size_t)255;
    const size_t ml = take((size_t)2 * A_CTAS * t.rp * sizeof(float2));
    const size_t po = take((size_t)2 * A_CTAS * t.rp * d.D * sizeof(float));
    if (bytes) *bytes = o;
    t.arrived = reinterpret_cast<uint32_t*>(ws + arrived);
    t.part_ml = reinterpret_cast<float2*>(ws + ml);
    t.part_o = reinterpret_cast<float*>(ws + po);
    t.sb = reinterpret_cast<StatusBlock*>(ws);
    return t;
}

// The CTAs of a launch wait for one another's parts, so it is cooperative: all of
// them run at once or none does yet, whatever other streams have on the SMs.
template <typename... KArgs, typename... Args>
cudaError_t launch_together(void (*kern)(KArgs...), size_t smem, cudaStream_t st, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(A_CTAS);
    cfg.blockDim = dim3(A_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

template <int D, bool E4M3>
cudaError_t launch_attn(const KvDims& d, const AttnArgs& a, cudaStream_t st) {
    using C = ACfg<D, E4M3>;
    const ATabs t = attn_tabs(d, a.ws, nullptr);
    CUtensorMap tm_q, tm_q8, tm_q1, tm_k, tm_v;
    const uint64_t el = E4M3 ? 1 : 2;
    const CUtensorMapDataType dt = E4M3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUtensorMapSwizzle sw = C::SW == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)d.page, (uint64_t)d.Hkv, (uint64_t)d.n_pages};
    const uint64_t str[3] = {d.token_stride * el, d.head_stride * el, d.page_stride * el};
    const uint32_t box[4] = {(uint32_t)(C::SW / el), (uint32_t)t.box, 1, 1};
    if (!make_map(&tm_k, dt, a.k_cache, 4, dims, str, box, sw) || !make_map(&tm_v, dt, a.v_cache, 4, dims, str, box, sw))
        return cudaErrorInvalidValue;
    tm_q = tm_q8 = tm_q1 = tm_k;
    if (!E4M3) {
        const uint64_t qd[3] = {(uint64_t)D, (uint64_t)d.Hq, (uint64_t)d.T};
        const uint64_t qs[2] = {(uint64_t)D * 2, (uint64_t)d.q_stride * 2};
        // boxes of a whole tile; for copies, of 8 tokens (where they fit 64 rows) and of one
        auto q_map = [&](CUtensorMap* m, int tokens) {
            const uint32_t qb[3] = {64, (uint32_t)t.G, (uint32_t)tokens};
            return make_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, 3, qd, qs, qb, CU_TENSOR_MAP_SWIZZLE_128B);
        };
        if (!q_map(&tm_q, t.tpt)) return cudaErrorInvalidValue;
        if (C::ROWB <= 128 && (!q_map(&tm_q8, 8 * t.G <= 64 ? 8 : 1) || !q_map(&tm_q1, 1))) return cudaErrorInvalidValue;
    }
    if (num_sms() < A_CTAS) return cudaErrorNotSupported;
    static std::atomic<bool> attribute_set[64];   // (a device's kernel attribute: set once)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !attribute_set[dev])) {
        e = cudaFuncSetAttribute(k_tree_attn<D, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e == cudaSuccess && dev < 64) attribute_set[dev] = true;
    }
    if (e != cudaSuccess) return e;
    timing_begin(K_TREE_ATTN, st);
    e = launch_together(k_tree_attn<D, E4M3>, C::SMEM, st, tm_q, tm_q8, tm_q1, tm_k, tm_v, d, a, t);
    timing_end(st);
    return e;
}

}  // namespace

size_t tree_attn_ws_bytes(const KvDims& d) {
    size_t n = 0;
    attn_tabs(d, nullptr, &n);
    return n;
}

cudaError_t launch_tree_attn(const KvDims& d, const AttnArgs& a, cudaStream_t st) {
    KT_BIND();
    if (d.D == 128) return d.e4m3 ? launch_attn<128, true>(d, a, st) : launch_attn<128, false>(d, a, st);
    return d.e4m3 ? launch_attn<64, true>(d, a, st) : launch_attn<64, false>(d, a, st);
}

}  // namespace moe

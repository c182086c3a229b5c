// out[t, n] = sum_k x[t, k] w[n, k] with MXFP4 weights, on the tensor cores.
//
// The weights are the MMA's A (M = 128 of their rows), the tokens its B.  With MXFP4 x
// both stay packed (tcgen05.mma kind::mxf4, K = 64).  A bf16 x enters as
// in the experts' kernel (experts_mx.cu): as two e4m3 terms a row, hi and lo, under
// a power of two a block of 32, which the scale warps make in shared memory (up to 8 tokens) or a
// small kernel (k_mx_split) writes first; the TMA
// unpacks the weights' codes for kind::mxf8f6f4.  Either way the tensor core applies the
// block scales.  (Two terms are fewer bits than a bf16 has where a block's magnitudes are far apart: exact to 2^-9 of the
// largest, within 2^-17 of it below.  It is the price of weights that go in as codes and scales: for a
// product in bf16 they are decoded first, to twice the bytes in shared memory.)
//
// Few tokens: one CTA a tile of 128 weight rows x NT tokens; a token of a bf16 x takes
// two columns of the MMA, added at the end.  Many: a pair of CTAs (cta_group::2) a tile of
// 256 weight rows x up to 256 tokens, of which each holds half of either operand (half the bytes a
// product that two single CTAs would copy); the terms of a bf16 x are two MMAs into one accumulator.
//
// How the tiles' stages (KS elements of K) are shared out (mx_cut chooses):
//   - few tiles: a cluster of up to eight CTAs a tile, each a part of K; every CTA sends its part by fours of tokens to
//     the CTA that adds them, in the order of K (T = 8, N = 7168, K = 4096, MXFP4 x: 4.7 us; by way of global memory 4 us more;
//     parts that the adding CTA reads: T = 64 8.1 us against 6.7);
//   - else the persistent CTAs (pairs) take whole tiles in turn; pairs take fewer tokens where that fills their
//     rounds.  (The last tiles cut anywhere and joined by way of global memory were slower for 50 of 52 products, by
//     half for most; for the others, T = 16, N = 20480, K = 4096 and T = 40, N = 39680, bf16 x, 14.8 and 25.7 us against 15.5 and 28.7.)
//
// What bounds it: up to some dozen tokens the weights' bytes from HBM (N = 16384, K = 8192: 71 MB in 12.7 us) and, for small
// products, the chain of a launch (1.2 us from the wait for earlier kernels to the first MMA, 1.2 for the sum over a
// cluster) and the stages' own pace (some 500 cycles: barrier, fences, four MMAs and their commit, whatever the tokens);
// with many tokens and a bf16 x the tensor cores (4096 x 4864 x 4096: 92 us, 1770 TFLOP/s, 0.91 of the
// measured bf16 rate); with both operands at 4 bits the K = 64 MMAs, which alone take 197 of 257 us, and the copies,
// scales and stores beside them (8192 x 14336 x 7168: 6550 TFLOP/s).
//
// Warps: 0 TMA, 1 MMA, 2-5 scales (global memory -> shared memory or registers -> TMEM), from 6 on the accumulators' way
// out (four, or eight of a pair's CTA), then a second set of scale warps.
#include "mx.cuh"
#include "quant.cuh"
#include "tc_ptx.cuh"

#include <atomic>
#include <math.h>
#include <type_traits>

namespace moe {
namespace {

template <int N>
using Int = std::integral_constant<int, N>;

constexpr int LM = 128;                       // weight rows a CTA
#ifndef MOE_WAIT_TEST
constexpr uint64_t L_WAIT_NS = 2000000000ull;
#else
constexpr uint64_t L_WAIT_NS = 1000000ull;    // test-only build: waits give up after 1 ms
#endif
constexpr int L_SITE = 300;                   // detail of MOE_ERR_TIMEOUT: site of the wait

// what a CTA of a cluster of up to 8 gets at most of n groups, each in as many parts
constexpr int most_parts(int n) {
    int most = 0;
    for (int c = 2; c <= 8; ++c) most = (n + c - 1) / c * c > most ? (n + c - 1) / c * c : most;
    return most;
}

// NT tokens a tile, CG CTAs a tile.
template <bool XMX, int NT, int CG>
struct LCfg {
    static constexpr bool FUSED = !XMX && CG == 1 && NT == 8;     // the terms of x are made here (K % 512 == 0)
    static constexpr bool FIRST = XMX || FUSED;                   // the call's first kernel: it reads nothing before its wait
    static constexpr int TERMS = !XMX && CG == 2 ? 2 : 1;         // MMAs of a K step
    static constexpr int PER = !XMX && CG == 1 ? 2 : 1;           // accumulator columns a token
    static constexpr int NB = PER * NT;                           // MMA N
    static constexpr int KS = TERMS == 2 ? 128 : 256;             // K a stage
    static constexpr int WORDS = KS / 128;                        // 32-bit words of scale bytes a row and stage
    static constexpr int B_ROWS = NB / CG;                        // rows of one term of x in this CTA
    static constexpr int A_BYTES = XMX ? LM * KS / 2 : LM * KS;   // a stage's weights in shared memory
    static constexpr int B_BYTES = XMX ? B_ROWS * KS / 2 : TERMS * B_ROWS * KS;
    static constexpr int EW = CG == 2 ? 8 : 4;                    // warps of the way out, and tokens of each
    static constexpr int EN = NT / (EW / 4);
    // sets of four scale warps (2-5, and behind the others), which take turns where a stage has little else (T = 16, N = 16384,
    // K = 8192, bf16 x: 17.7 us with one, 16.0 with two; with wider tiles the registers of more warps cost more than they
    // gain: T = 128, N = 9216, K = 7168, MXFP4 x 10.8 and 11.9)
    static constexpr int SETS = CG == 1 && NT <= (XMX ? 64 : 32) ? 2 : 1;
    static constexpr int THREADS = 32 * (2 + 4 * SETS + EW);
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int TX = CG * (LM * KS / 2 + (FUSED ? 0 : B_BYTES));   // bytes of a stage that its barrier counts
    static constexpr int ACC = NB <= 128 ? 2 : 1;                 // accumulators
    // a stage's scales in TMEM: weight words of 128 K each at SF_A, SF_A + 16, the token words behind them
    // (every scale address is a multiple of 16 columns)
    static constexpr int SF_SLOT = WORDS * 32, SF_B = WORDS * 16;
    static constexpr int SF_COL0 = (ACC * NB + 63) / 64 * 64;
    static constexpr int S_TMEM = (512 - SF_COL0) / SF_SLOT;
    // scales on their way to TMEM: a pair's groups of 1024 K, [8 words][rows], twice; else RING
    // groups of 512 K (RING / SETS a set), a row of weights or tokens 16 bytes (or half as many of twice the bytes, where the rows in
    // memory are not 16-byte aligned: the two aligned pieces that hold them)
    static constexpr int RING = SETS == 2 && !FUSED ? 8 : 4;
    static constexpr int XCH_BYTES = CG == 2 ? 2 * 8 * (LM + NT + 8) * 4 : RING * (LM + NT) * 16 + (FUSED ? SETS * 2 * NT * 8 : 0);
    static constexpr int S_FIT = (232448 - 1024 - 512 - XCH_BYTES) / STAGE;
    // (a ring of their own for the scales, which leaves a pair's MXFP4 tiles six stages of copies under way
    // instead of four, made T = 8192, N = 14336, K = 7168 slower: 335 us against 296)
    // (FUSED: five leave ROOM, see below: T = 1, N = 6144, K = 4096 7.05 us, with six 7.4)
    static constexpr int S = TERMS == 2 ? 4 : FUSED ? 5 : S_FIT < S_TMEM ? S_FIT : S_TMEM;
    // where a cluster's parts of a tile meet: a CTA's groups of four tokens, of each [part][LM] float4, behind the rest where
    // there is room, so that they need not wait for this CTA's stages, else in those
    static constexpr int MEET = most_parts(NT / 4) * LM * 16;
    static constexpr bool ROOM = CG == 1 && 1024 + S * STAGE + XCH_BYTES + 512 + MEET <= 232448;
    static constexpr int SMEM = 1024 + S * STAGE + XCH_BYTES + 512 + (ROOM ? MEET : 0);
    static_assert(CG == 2 || ROOM || S * STAGE >= MEET, "a place for the parts");
    static_assert(S >= 2 && S <= S_FIT && SMEM <= 232448, "stages");
    static_assert(CG == 1 || NT == 256, "a pair's tile is 256 x 256");
};

// n / d for 0 <= n < 2^31 as a product and a shift: with s = ceil(log2 d) and m = ceil(2^(31 + s) / d), n m 2^-(31 + s)
// exceeds n / d by n e / (d 2^(31 + s)), 0 <= e < d <= 2^s, which is less than 1 / d.  (Divisions on the way
// to the first MMA took 0.6 us of a launch's 6.7, with the code they needed 1.2.)
struct Div {
    uint32_t mul;
    int shift;
    Div() = default;
    explicit Div(uint32_t d) : shift(31) {
        while (((uint32_t)1 << (shift - 31)) < d) ++shift;
        mul = (uint32_t)((((uint64_t)1 << shift) + d - 1) / d);
    }
    __device__ __forceinline__ int of(int n) const { return (int)(((uint64_t)(uint32_t)n * mul) >> shift); }
};

struct LArgs {
    const uint8_t *w_scales, *xs;             // [N][K/32], [T][K/32]
    __nv_bfloat16* out;
    StatusBlock* sb;
    int T, N, K;
    int64_t out_stride;
    int nt;                                   // tokens of a pair's tile: a multiple of 32 up to NT
    int nk, tt, mt;                           // stages a tile, token tiles, weight tiles
    int under_way;                            // stages of a pair with a bf16 x that are used: S or fewer
    int split;                                // CTAs of a cluster that share a tile, or 1
    int tiles;
    int vec;                                  // scale rows are 16-byte aligned
    int w_once;
    Div workers, by_split, by_band, by_last;   // (by_band: tiles of a band, by_last: weight tiles of the last one)
};

// Token t's (low half) and t + 1's value of this lane's row of weights, to out[0] and out[stride] while below `end`: lanes 2i and
// 2i + 1 exchange, so that each stores both rows of one of the tokens (2-byte stores: T = 8192, N = 14336,
// K = 7168 in 311 us against 289; rows of 256 bytes through shared memory: 330, by TMA: 371).
__device__ __forceinline__ void store_rows(__nv_bfloat16* out, int64_t stride, bool row, int t, int end, uint32_t v) {
    const int odd = threadIdx.x & 1;
    const uint32_t u = __shfl_xor_sync(0xffffffffu, v, 1);
    if (row && t + odd < end)
        *reinterpret_cast<uint32_t*>(out + (odd ? stride - 1 : 0)) = odd ? __byte_perm(u, v, 0x7632) : __byte_perm(v, u, 0x5410);
}

// A worker's segments: stages [k0, k1) of tile (m, t), one after the other: every n-th tile of n workers, or a cluster's CTA's
// share of one.  Tiles are numbered through bands of GM weight tiles, so that those that are worked on at one
// time share their rows of w and of x.
template <int CG>
struct Segment {
    static constexpr int GM = 8;
    int left;                    // segments to go, this one too
    int tile, m, t, k0, k1;
    const LArgs& a;
    __device__ __forceinline__ explicit Segment(const LArgs& args) : k0(0), k1(args.nk), a(args) {
        if (CG == 1 && a.split > 1) {
            const int part = ptx::cluster_rank();
            tile = ptx::cluster_id();
            left = 1;
            k0 = a.by_split.of(a.nk * part);
            k1 = a.by_split.of(a.nk * (part + 1));
        } else {
            tile = blockIdx.x / CG;
            left = a.workers.of(a.tiles - tile + gridDim.x / CG - 1);
        }
        place();
    }
    __device__ __forceinline__ void place() {
        m = tile;
        t = 0;
        if (a.tt > 1) {
            const int band = a.by_band.of(tile), in = tile - band * GM * a.tt;
            const bool whole = (band + 1) * GM <= a.mt;
            t = whole ? in / GM : a.by_last.of(in);
            m = band * GM + in - t * (whole ? GM : a.mt - band * GM);
        }
    }
    __device__ __forceinline__ bool more() const { return left > 0; }
    __device__ __forceinline__ void next() {
        tile += gridDim.x / CG;
        if (--left > 0) place();
    }
};

template <bool XMX, int NT, int CG>
__global__ void __launch_bounds__(LCfg<XMX, NT, CG>::THREADS, 1)
    k_mx_linear(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, const LArgs a) {
    using C = LCfg<XMX, NT, CG>;
    constexpr int S = C::S, NB = C::NB, ACC = C::ACC, WORDS = C::WORDS;
    constexpr bool PAIR = CG == 2;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int stages = C::TERMS == 2 ? a.under_way : S;
    // scales: a pair's two buffers of 8 x (LM + 4) words of the weights and 8 x (NT + 4) of the tokens, else [RING][LM + NT] rows
    uint8_t* xch = sm + stages * C::STAGE;
    // a pair's stages are counted on the even CTA's `full`, and its MMAs' ends on both CTAs' barriers
    uint64_t* full = reinterpret_cast<uint64_t*>(xch + C::XCH_BYTES);
    uint64_t* empty = full + S;          // the stage's MMAs are done
    uint64_t* acc_full = empty + S;
    uint64_t* acc_empty = acc_full + ACC;
    uint64_t* x_full = acc_empty + ACC;  // FUSED: the stage's rows of x are there
    uint64_t* fin = x_full + (C::FUSED ? S : 0);
    uint32_t* holder = reinterpret_cast<uint32_t*>(fin + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(holder + 1);
    volatile int* last_flag = abort_flag + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = PAIR ? blockIdx.x & 1 : 0;
    KT_MARK(K_MX_LINEAR, 0);
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            ptx::mbar_init(&full[i], 1 + 4 * CG);      // TMA, the scale warps
            ptx::mbar_init(&empty[i], 1);
            if (C::FUSED) ptx::mbar_init(&x_full[i], 1);
        }
        for (int i = 0; i < ACC; ++i) {
            ptx::mbar_init(&acc_full[i], 1);
            ptx::mbar_init(&acc_empty[i], C::EW * CG);
        }
        ptx::mbar_init(fin, 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&tm_w);
        ptx::prefetch_tensormap(&tm_x);
    }
    if (warp == 1) {
        if (PAIR) ptx::tmem2_alloc(holder, 512);
        else ptx::tmem_alloc(holder, 512);
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (PAIR) ptx::cluster_sync_all();   // both CTAs' barriers exist
    // the cluster's CTAs run (and, without ROOM, are done with their stages): parts may be sent to them
    bool met = PAIR || a.split == 1;
    if (!PAIR && C::ROOM && a.split > 1) ptx::cluster_arrive_relaxed();
    auto meet = [&] {
        if (met) return;
        met = true;
        if (!C::ROOM) ptx::cluster_arrive_relaxed();
        ptx::cluster_wait();
    };
    float4* parts = reinterpret_cast<float4*>(C::ROOM ? xch + C::XCH_BYTES + 512 : sm);
    ptx::tc_fence_after();
    const uint32_t tmem = *holder;
    // (with what needs no input done, each role waits for the kernels before)

    auto fail = [&](int site) {
        latch_status(a.sb, MOE_ERR_TIMEOUT, L_SITE + site);
        *abort_flag = 1;
    };
    if (warp == 0) {
        // ------------------------------------------------------------ TMA
        const uint64_t pol_w = a.w_once ? ptx::policy_evict_first() : ptx::policy_evict_last();
        const uint64_t pol_x = ptx::policy_evict_last();
        const uint32_t full0 = PAIR ? ptx::map_cluster(full, 0) : 0;
        const uint32_t pair_tx = C::TX - C::B_BYTES / (NT / 2) * (NT - a.nt);
        auto weights = [&](const Segment<CG>& g, int k, int s) {
            uint8_t* st = sm + s * C::STAGE;
            const int row = (g.m * CG + rank) * LM;
            if (rank == 0) ptx::mbar_arrive_expect_tx(&full[s], PAIR ? pair_tx : C::TX);
            if (PAIR) {
                if (XMX) ptx::tma2_load_2d(st, &tm_w, 128 * k, row, full0 + 8 * s, pol_w);
                else ptx::tma2_load_3d(st, &tm_w, 0, row, WORDS * k, full0 + 8 * s, pol_w);
            } else {
                if (XMX) ptx::tma_load_2d(st, &tm_w, 128 * k, row, &full[s], pol_w);
                else ptx::tma_load_3d(st, &tm_w, 0, row, WORDS * k, &full[s], pol_w);
            }
        };
        auto tokens = [&](const Segment<CG>& g, int k, int s) {
            uint8_t* st = sm + s * C::STAGE + C::A_BYTES;
            const int row = PAIR ? g.t * a.nt + rank * (a.nt / 2) : g.t * NB;
            if (PAIR) {
                if (XMX) ptx::tma2_load_2d(st, &tm_x, 128 * k, row, full0 + 8 * s, pol_x);
                else ptx::tma2_load_4d(st, &tm_x, 0, row, 0, k, full0 + 8 * s, pol_x);
            } else {
                if (C::FUSED) {
                    // x itself, NT rows of 512 bytes
                    ptx::mbar_arrive_expect_tx(&x_full[s], C::B_BYTES);
                    ptx::tma_load_2d(st, &tm_x, 256 * k, g.t * NT, &x_full[s], pol_x);
                } else if (XMX) {
                    ptx::tma_load_2d(st, &tm_x, 128 * k, row, &full[s], pol_x);
                } else {
                    ptx::tma_load_3d(st, &tm_x, 0, row, 2 * k, &full[s], pol_x);
                }
            }
        };
        if (lane == 0) {
            int pre = 0;
            if (!C::FIRST) {
                // the first stages' weights, inputs of the call, before the wait for the tokens' terms
                int i = 0;
                for (Segment<CG> g(a); g.more() && i < stages; g.next())
                    for (int k = g.k0; k < g.k1 && i < stages; ++k, ++i) weights(g, k, i);
                pre = i;
                pdl_wait();
            }
            bool ok = true;
            int it = 0, s = 0;
            uint32_t par = 1;
            Segment<CG> g(a);
            if (C::FIRST) pdl_wait();
            for (; ok && g.more(); g.next()) {
                for (int k = g.k0; k < g.k1; ++k, ++it) {
                    if (it >= pre) {
                        if (!(PAIR ? ptx::mbar_wait(&empty[s], par, abort_flag, L_WAIT_NS)
                                   : ptx::mbar_wait_spin(&empty[s], par, abort_flag, L_WAIT_NS))) {
                            fail(1);
                            ok = false;
                            break;
                        }
                        weights(g, k, s);
                    }
                    tokens(g, k, s);
                    if (++s == stages) s = 0, par ^= 1;
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA
        // (one thread goes through the stages by itself, its waits without suspension: what it does between two stages'
        // MMAs sets the pace)
        if (rank == 0 && ptx::elect_one()) {
            int s = 0, seg = 0;
            uint32_t par = 0;
            bool ok = true;
            // descriptors of stage 0; a stage further is STAGE / 16 more
            const uint64_t a_desc = ptx::smem_desc_sw128(ptx::smem_u32(sm)), b_desc = a_desc + C::A_BYTES / 16;
            const int n_mma = PAIR ? a.nt : NB;
            // (it reads nothing that they wrote, but its waits' limit must not count their time)
            pdl_wait();
            for (Segment<CG> g(a); ok && g.more(); g.next(), ++seg) {
                const int ab = seg % ACC;
                if (!ptx::mbar_wait_spin(&acc_empty[ab], ((seg / ACC) & 1) ^ 1, abort_flag, L_WAIT_NS)) {
                    fail(2);
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t d_tmem = tmem + ab * NB;
                for (int k = g.k0; k < g.k1; ++k) {
                    if (!ptx::mbar_wait_spin(&full[s], par, abort_flag, L_WAIT_NS)) {
                        fail(3);
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint64_t a0 = a_desc + (uint32_t)(s * (C::STAGE / 16)), b0 = b_desc + (uint32_t)(s * (C::STAGE / 16));
                    const uint32_t sfa = tmem + C::SF_COL0 + s * C::SF_SLOT, sfb = sfa + C::SF_B;
                    if constexpr (XMX) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint64_t ad = a0 + 2 * j, bd = b0 + 2 * j;
                            const uint32_t id = ptx::idesc_mxf4(LM * CG, n_mma, 2 * (j & 1), 2 * (j & 1));
                            const uint32_t acc = k > g.k0 || j > 0, fa = sfa + 16 * (j >> 1), fb = sfb + 16 * (j >> 1);
                            if (PAIR) ptx::mma2_mxf4_ss(d_tmem, ad, bd, id, acc, fa, fb);
                            else ptx::mma_mxf4_ss(d_tmem, ad, bd, id, acc, fa, fb);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 4 * WORDS * C::TERMS; ++j) {
                            // 128-K slab, K step within it, term
                            const int h = WORDS == 2 ? j >> 2 : 0, q = j & 3, e = C::TERMS == 2 ? j >> 2 : 0;
                            const uint64_t ad = a0 + (h * LM * 8 + 2 * q);
                            const uint64_t bd = b0 + (uint32_t)((h * C::B_ROWS + e * (a.nt / 2)) * 8 + 2 * q);
                            const uint32_t id = ptx::idesc_mx_e2m1_e4m3(LM * CG, n_mma, q, q);
                            const uint32_t acc = k > g.k0 || j > 0, fa = sfa + 16 * h, fb = sfb + 16 * h;
                            if (PAIR) ptx::mma2_mx_ss(d_tmem, ad, bd, id, acc, fa, fb);
                            else ptx::mma_mx_ss(d_tmem, ad, bd, id, acc, fa, fb);
                        }
                    }
                    if (PAIR) {
                        ptx::mma2_commit(&empty[s]);
                        if (k + 1 == g.k1) ptx::mma2_commit(&acc_full[ab]);
                    } else {
                        ptx::mma_commit(&empty[s]);
                        if (k + 1 == g.k1) ptx::mma_commit(&acc_full[ab]);
                    }
                    if (++s == stages) s = 0, par ^= 1;
                }
            }
            // every MMA issued above has completed before TMEM is released
            if (PAIR) ptx::mma2_commit(fin);
            else ptx::mma_commit(fin);
        }
        __syncwarp();
        ptx::mbar_wait_all(fin, 0, abort_flag, L_WAIT_NS);
    } else if (warp < 6 && PAIR) {
        // ------------------------------------------------------------ scales of a pair: groups of 1024 K, the next one ahead
        // in registers.  Eight lanes load a row's 32 bytes: a lane a row, which takes two to eight requests a
        // row instead of one, held up the TMA's (T = 4096, N = 6144, K = 4096, MXFP4 x: 51 us against 46)
        const int q = warp & 3, word = lane & 7, sub = lane >> 3;
        const uint32_t lane_base = (uint32_t)(32 * q) << 16;
        const int kb = a.K / 32;
        constexpr int PG = 8 / WORDS;                                 // stages of a group
        constexpr int PT = 256;                                       // (NT)
        constexpr int NA = LM / 16, NR = PT / 16;                     // rows of weights, tokens a thread loads a word of
        constexpr int SA = LM + 4, SB = PT + 4;                       // (4: the lanes' stores fall into different banks)
        const uint32_t full0 = ptx::map_cluster(full, 0);
        uint32_t na[NA], nb[NR];
        // bytes 32 grp + 4 word .. + 3 of rows 4 i + sub of this warp's part; past the tensor's ends 127 (its codes are zeros)
        auto load = [&](const uint8_t* from, int row0, int rows, int grp, auto& to) {
            const bool in = 32 * grp + 4 * word < kb;
            const int n = rows - row0 - sub;     // rows from this lane's first one on
            uint32_t at = (uint32_t)(row0 + sub) * kb + 32 * grp + 4 * word;   // (rows * kb <= 2^31)
#pragma unroll
            for (int i = 0; i < (int)(sizeof(to) / 4); ++i, at += 4 * kb)
                to[i] = in && 4 * i < n ? ld_dep(reinterpret_cast<const uint32_t*>(from + at)) : 0x7F7F7F7Fu;
        };
        auto load_a = [&](const Segment<CG>& g, int grp) { load(a.w_scales, (g.m * CG + rank) * LM + q * (LM / 4), a.N, grp, na); };
        auto load_b = [&](const Segment<CG>& g, int grp) { load(a.xs, g.t * a.nt + q * (PT / 4), a.T, grp, nb); };
        Segment<CG> g(a);
        if (C::FIRST) pdl_wait();
        if (g.more()) load_a(g, 0);
        if (!C::FIRST) pdl_wait();
        if (g.more()) load_b(g, 0);
        // a warp whose wait gave up goes on without waiting: the four share the barrier below
        int s = 0, buf = 0;
        uint32_t par = 1;
        bool ok = true;
        for (; g.more(); g.next()) {
            for (int grp = 0; PG * grp < g.k1; ++grp) {
                uint32_t* xa = reinterpret_cast<uint32_t*>(xch) + buf * 8 * (SA + SB);
                uint32_t* xb = xa + 8 * SA;
                uint32_t nan = 0;
#pragma unroll
                for (int i = 0; i < NA; ++i) {
                    nan |= __vcmpeq4(na[i], 0xFFFFFFFFu);
                    xa[word * SA + q * (LM / 4) + 4 * i + sub] = na[i];
                }
#pragma unroll
                for (int i = 0; i < NR; ++i) xb[word * SB + q * (PT / 4) + 4 * i + sub] = nb[i];
                if (nan) latch_status(a.sb, MOE_ERR_BAD_SCALE, 255);
                // the next group's, under way while this one's stages go through
                Segment<CG> n = g;
                int ngrp = grp + 1;
                if (PG * ngrp >= g.k1) n.next(), ngrp = 0;
                if (n.more()) {
                    load_a(n, ngrp);
                    load_b(n, ngrp);
                }
                // (one barrier a group: a buffer is written again two groups later)
                ptx::named_bar_sync(1, 128);
                buf ^= 1;
#pragma unroll 1
                for (int i = 0; i < PG; ++i) {
                    if (!ok || PG * grp + i >= g.k1) break;
                    uint32_t w[WORDS], v[WORDS][PT / 32];
#pragma unroll
                    for (int h = 0; h < WORDS; ++h) {
                        w[h] = xa[(WORDS * i + h) * SA + 32 * q + lane];
#pragma unroll
                        for (int c = 0; c < PT / 32; ++c) v[h][c] = xb[(WORDS * i + h) * SB + 32 * c + lane];
                    }
                    if (!ptx::mbar_wait_all(&empty[s], par, abort_flag, L_WAIT_NS)) {
                        if (lane == 0) fail(4);
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint32_t col = tmem + lane_base + C::SF_COL0 + s * C::SF_SLOT;
#pragma unroll
                    for (int h = 0; h < WORDS; ++h) {
                        // row r is read at lane r mod 32 of this quarter, column + q; column n of B:
                        // lane n mod 32 of every quarter, column + n / 32
                        ptx::tmem_st1(col + 16 * h + q, w[h]);
                        ptx::tmem_st8(col + C::SF_B + 16 * h, v[h]);
                    }
                    ptx::tmem_st_wait();
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive_cluster(full0 + 8 * s);
                    if (++s == stages) s = 0, par ^= 1;
                }
            }
        }
    } else if (warp < 6 || warp >= 6 + C::EW) {
        // ------------------------------------------------------------ scales: groups of 512 K, ahead in shared memory
        // (a set of four warps takes every SETS-th group, of which it has `ring` - 1 under way)
        const int set = warp < 6 ? 0 : 1;
        const int q = warp & 3, r = 32 * q + lane;      // TMEM lane quarter; weight row and token of this thread
        const uint32_t lane_base = (uint32_t)(32 * q) << 16;
        const int kb = a.K / 32;
        constexpr int RING_BYTES = C::RING * (LM + NT) * 16;
        const int ring = (a.vec ? C::RING : C::RING / 2) / C::SETS, bytes = a.vec ? 16 : 32;
        uint8_t* mine = xch + set * (C::RING / C::SETS) * (LM + NT) * 16;
        // a group's scale bytes of row `n` of `rows`; zeros past the tensor's ends, where the codes are zeros too
        auto fetch = [&](const uint8_t* src, int n, int rows, int grp, uint8_t* dst) {
            const int64_t at = (int64_t)min(n, rows - 1) * kb + 16 * grp, end = (int64_t)rows * kb;
            if (a.vec) {
                ptx::cp_async_16(dst, src + at, n < rows ? 16 : 0);
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int64_t p = (at & ~(int64_t)15) + 16 * i;
                    ptx::cp_async_16(dst + 16 * i, src + min(p, end & ~(int64_t)15),
                                     n < rows ? (uint32_t)max((int64_t)0, min((int64_t)16, end - p)) : 0u);
                }
            }
        };
        // its 8 bytes of stage k.  Where K ends in half a stage the second word is the next row's first scales: a 0 in
        // its place, because the codes there are zeros, but a 255 (NaN) of that row times zero is NaN
        auto words = [&](const uint8_t* p, int n, int rows, int k) {
            if (a.vec) return *reinterpret_cast<const uint2*>(p + 8 * (k & 1));
            const uint32_t* w = reinterpret_cast<const uint32_t*>(p + ((int64_t)min(n, rows - 1) * kb & 15) + 8 * (k & 1));
            return make_uint2(w[0], 8 * k + 4 < kb ? w[1] : 0u);
        };
        auto fetch_a = [&](const Segment<CG>& g, int grp, int buf) {
            fetch(a.w_scales, g.m * LM + r, a.N, grp, mine + (buf * (LM + NT) + r) * bytes);
        };
        auto fetch_b = [&](const Segment<CG>& g, int grp, int buf) {
            if (!C::FUSED && r < NT) fetch(a.xs, g.t * NT + r, a.T, grp, mine + (buf * (LM + NT) + LM + r) * bytes);
        };
        auto advance = [&](Segment<CG>& g, int& grp) {
            if (2 * ++grp >= g.k1) {
                g.next();
                grp = g.k0 / 2;
            }
        };
        // to the set's next group
        auto skip = [&](Segment<CG>& g, int& grp) {
#pragma unroll
            for (int i = 0; i < C::SETS; ++i)
                if (g.more()) advance(g, grp);
        };
        Segment<CG> g(a), ahead = g;
        int grp = g.k0 / 2, agrp = grp;
        if (set == 1 && ahead.more()) advance(ahead, agrp);
        if (!C::FIRST) {
            // the weights' scales, inputs of the call, before the wait for the tokens'
            Segment<CG> n = ahead;
            int ngrp = agrp;
#pragma unroll 1
            for (int i = 0; i < ring - 1 && n.more(); ++i, skip(n, ngrp)) fetch_a(n, ngrp, i);
        }
        pdl_wait();
#pragma unroll 1
        for (int i = 0; i < ring - 1; ++i) {
            if (ahead.more()) {
                if (C::FIRST) fetch_a(ahead, agrp, i);
                fetch_b(ahead, agrp, i);
                skip(ahead, agrp);
            }
            ptx::cp_async_commit();
        }
        // a warp whose wait gave up goes on without waiting: the four share the barrier below
        int s = 0, buf = 0, turn = 0;
        uint32_t par = C::FUSED ? 0 : 1;
        uint2* made = reinterpret_cast<uint2*>(xch + RING_BYTES) + set * 2 * NT;   // FUSED: [2][NT] scale words of the stage's tokens
        int turn_of = 0;                           // whose group it is
        bool ok = true;
#pragma unroll 1
        for (; g.more(); advance(g, grp)) {
            const int k0 = max(2 * grp, g.k0), k1 = min(2 * grp + 2, g.k1);
            if (C::SETS == 2) {
                const bool other = turn_of != set;
                turn_of ^= 1;
                if (other) {
                    s += k1 - k0;
                    if (s >= S) s -= S, par ^= 1;
                    continue;
                }
            }
            if (ring == 4) ptx::cp_async_wait<2>();
            else ptx::cp_async_wait<0>();
            ptx::named_bar_sync(1 + 2 * set, 128);
            // (behind the barrier every warp is done with the group before this one)
            if (ahead.more()) {
                const int to = buf == 0 ? ring - 1 : buf - 1;
                fetch_a(ahead, agrp, to);
                fetch_b(ahead, agrp, to);
                skip(ahead, agrp);
            }
            ptx::cp_async_commit();
            const uint8_t* rows = mine + buf * (LM + NT) * bytes;
            buf = buf + 1 == ring ? 0 : buf + 1;
#pragma unroll 1
            for (int k = k0; k < k1; ++k) {
                const uint2 w = words(rows + bytes * r, g.m * LM + r, a.N, k);
                if (__vcmpeq4(w.x, 0xFFFFFFFFu) | __vcmpeq4(w.y, 0xFFFFFFFFu)) latch_status(a.sb, MOE_ERR_BAD_SCALE, 255);
                uint2 v[(NB + 31) / 32];
                uint64_t* free = C::FUSED ? &x_full[s] : &empty[s];
                if (ok && !__all_sync(0xffffffffu, ptx::mbar_test_wait(free, par)) && !ptx::mbar_wait_all(free, par, abort_flag, L_WAIT_NS)) {
                    if (lane == 0) fail(4);
                    ok = false;
                }
                ptx::tc_fence_after();
                if constexpr (C::FUSED) {
                    // warp q takes tokens q, q + 4, ..., a lane 8 elements of each: x out of the stage, then its
                    // terms in place of it (row 2t hi, 2t + 1 lo, two slabs of 128 K, 128-byte swizzle)
                    uint8_t* st = sm + s * C::STAGE + C::A_BYTES;
                    QuantChunk qc[NT / 4];
#pragma unroll
                    for (int i = 0; i < NT / 4; ++i) {
                        if (g.t * NT + 4 * i + q >= a.T) {      // (the arithmetic is what a stage takes longest for)
                            qc[i].hi = qc[i].lo = make_uint2(0, 0);
                            qc[i].e = 1;
                            qc[i].amax = 0;
                        } else {
                            qc[i] = quantize_vals(*reinterpret_cast<const uint4*>(st + (4 * i + q) * 512 + 16 * lane));
                        }
                        if (qc[i].amax >= 0x7F800000u) {
                            qc[i].hi = qc[i].lo = make_uint2(0, 0);
                            qc[i].e = 255;
                        }
                        // lanes 0-15: the scale bytes of the first 128 K, lanes 16-31: of the second
                        uint32_t e = (uint32_t)qc[i].e << (8 * (lane >> 2 & 3));
                        e |= __shfl_xor_sync(0xffffffffu, e, 4);
                        e |= __shfl_xor_sync(0xffffffffu, e, 8);
                        if ((lane & 15) == 0) reinterpret_cast<uint32_t*>(made + turn * NT + 4 * i + q)[lane >> 4] = e;
                    }
                    ptx::named_bar_sync(1 + 2 * set, 128);
#pragma unroll
                    for (int i = 0; i < NT / 4; ++i) {
                        const int row = 2 * (4 * i + q), unit = lane >> 1 & 7;
                        uint8_t* to = st + (lane >> 4) * NB * 128 + row * 128 + 8 * (lane & 1);
                        *reinterpret_cast<uint2*>(to + ((unit ^ (row & 7)) << 4)) = qc[i].hi;
                        *reinterpret_cast<uint2*>(to + 128 + ((unit ^ (row + 1 & 7)) << 4)) = qc[i].lo;
                    }
                    ptx::fence_proxy_async_shared();
                    v[0] = made[turn * NT + (lane >> 1) % NT];
                    turn ^= 1;                     // (written again only behind the next stage's barrier)
                } else {
#pragma unroll
                    for (int c = 0; c < (NB + 31) / 32; ++c) {
                        const int t = (C::PER == 1 ? 32 * c + lane : 16 * c + (lane >> 1)) % NT;
                        v[c] = words(rows + bytes * (LM + t), g.t * NT + t, a.T, k);
                    }
                }
                if (!ok) continue;
                const uint32_t col = tmem + lane_base + C::SF_COL0 + s * C::SF_SLOT;
                // row r is read at lane r mod 32 of this quarter, column + q
                ptx::tmem_st1(col + q, w.x);
                ptx::tmem_st1(col + 16 + q, w.y);
                // column n of B: lane n mod 32 of every quarter, column + n / 32
                const uint32_t to = col + C::SF_B;
                if constexpr (NB <= 32) {
                    ptx::tmem_st4_rep(to, v[0].x);
                    ptx::tmem_st4_rep(to + 16, v[0].y);
                } else if constexpr (NB == 64) {
                    ptx::tmem_st2(to, v[0].x, v[1].x);
                    ptx::tmem_st2(to + 16, v[0].y, v[1].y);
                } else if constexpr (NB == 128) {
                    ptx::tmem_st4(to, v[0].x, v[1].x, v[2].x, v[3].x);
                    ptx::tmem_st4(to + 16, v[0].y, v[1].y, v[2].y, v[3].y);
                }
                ptx::tmem_st_wait();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&full[s]);
                if (++s == S) s = 0, par ^= 1;
            }
        }
        ptx::cp_async_wait<0>();
    } else {
        // ------------------------------------------------------------ accumulators
        const int q = warp & 3, r = 32 * q + lane;
        const uint32_t lane_base = (uint32_t)(32 * q) << 16;
        const uint32_t acc_empty0 = PAIR ? ptx::map_cluster(acc_empty, 0) : 0;
        pdl_wait();
        pdl_trigger();
        // G tokens' sums, a token's columns added
        constexpr int G = C::EN < 32 ? C::EN : 32;
        const int first = PAIR ? (warp - 6) / 4 * (a.nt / 2) : 0;       // this warp's tokens: from here, at most EN
        auto read = [&](int ab, int t, float (&y)[G]) {
            const uint32_t from = tmem + lane_base + ab * NB + C::PER * t;
            if constexpr (C::PER * G == 16) {
                uint32_t v[16];
                ptx::tmem_ld16(from, v);
                ptx::tmem_ld_wait16(v);
#pragma unroll
                for (int j = 0; j < G; ++j)
                    y[j] = C::PER == 1 ? __uint_as_float(v[j]) : __uint_as_float(v[2 * j]) + __uint_as_float(v[2 * j + 1]);
            } else if constexpr (C::PER == 1) {
                ptx::tmem_ld32(from, y);
                ptx::tmem_ld_wait32(y);
            } else {
#pragma unroll
                for (int b = 0; b < C::PER * G / 32; ++b) {
                    float v[32];
                    ptx::tmem_ld32(from + 32 * b, v);
                    ptx::tmem_ld_wait32(v);
#pragma unroll
                    for (int j = 0; j < 16; ++j) y[16 * b + j] = v[2 * j] + v[2 * j + 1];
                }
            }
        };
        auto release = [&](int ab) {
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (PAIR) ptx::mbar_arrive_cluster(acc_empty0 + 8 * ab);
                else ptx::mbar_arrive(&acc_empty[ab]);
            }
        };
        int seg = 0;
        for (Segment<CG> g(a); g.more(); g.next(), ++seg) {
            const int ab = seg % ACC;
            if (C::ROOM) meet();
            if (!ptx::mbar_wait_all(&acc_full[ab], (seg / ACC) & 1, abort_flag, L_WAIT_NS) && lane == 0) fail(5);
            // the warps decide together (they share barriers below)
            if (threadIdx.x == 6 * 32) last_flag[1 + (seg & 1)] = *abort_flag;
            ptx::named_bar_sync(2, 32 * C::EW);
            meet();
            if (last_flag[1 + (seg & 1)]) break;
            ptx::tc_fence_after();
            const int row0 = (g.m * CG + rank) * LM, row = row0 + r, t0 = g.t * (PAIR ? a.nt : NT);
            const int n_tok = min(PAIR ? a.nt : NT, a.T - t0), mine = PAIR ? min(first + a.nt / 2, n_tok) : n_tok;
            if constexpr (!PAIR) {
                if (a.split > 1) {
                    // the cluster's CTAs take four tokens in turn to add: their parts go there
                    uint32_t at = ptx::smem_u32(parts + ptx::cluster_rank() * LM + r), to = 0;
#pragma unroll 1
                    for (int t = 0; t < n_tok; t += G) {
                        float y[G];
                        read(ab, t, y);
#pragma unroll
                        for (int j = 0; j < G; j += 4) {
                            if (t + j < n_tok)
                                ptx::st_cluster(ptx::map_cluster(at, to), make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]));
                            if (++to == a.split) to = 0, at += a.split * LM * 16;
                        }
                    }
                    break;
                }
            }
            auto store = [&](int t, uint32_t v) {
                store_rows(a.out + (t0 + first + t) * a.out_stride + row, a.out_stride, row < a.N, first + t, mine, v);
            };
            if constexpr (PAIR) {
                // its one accumulator is read out first, so that the next tile's MMAs may begin
                uint32_t y2[C::EN / 2];
#pragma unroll
                for (int t = 0; t < C::EN; t += G) {
                    float y[G];
                    read(ab, first + t, y);
#pragma unroll
                    for (int j = 0; j < G; j += 2) y2[(t + j) / 2] = ptx::cvt_bf16x2(y[j], y[j + 1]);
                }
                release(ab);
                __nv_bfloat16* out = a.out + (t0 + first) * a.out_stride + row;
#pragma unroll
                for (int t = 0; t < C::EN; t += 2, out += 2 * a.out_stride)
                    store_rows(out, a.out_stride, row < a.N, first + t, mine, y2[t / 2]);
            } else {
#pragma unroll 1
                for (int t = 0; t < n_tok; t += G) {
                    float y[G];
                    read(ab, t, y);
#pragma unroll
                    for (int j = 0; j < G; j += 2) store(t + j, ptx::cvt_bf16x2(y[j], y[j + 1]));
                }
                release(ab);
            }
        }
    }
    if constexpr (!PAIR) {
        if (a.split > 1) {
            const Segment<CG> g(a);
            const int c = ptx::cluster_rank(), t0 = g.t * NT, n_tok = min(NT, a.T - t0);
            const int groups = a.by_split.of((n_tok + 3) / 4 - c + a.split - 1);
            __syncwarp();
            meet();
            ptx::cluster_sync_all();
            // added in the order of K, four tokens of a row at a time
            auto add = [&](auto most) {
                constexpr int P = decltype(most)::value;
#pragma unroll 1
                for (int i = warp; i < 4 * groups; i += C::THREADS / 32) {
                    const int r = 32 * (i & 3) + lane, row = g.m * LM + r;
                    const float4* from = parts + (i >> 2) * a.split * LM + r;
                    float4 v[P];
#pragma unroll
                    for (int p = 0; p < P; ++p) v[p] = p < a.split ? from[p * LM] : make_float4(0.f, 0.f, 0.f, 0.f);
                    float4 y = v[0];
#pragma unroll
                    for (int p = 1; p < P; ++p) y.x += v[p].x, y.y += v[p].y, y.z += v[p].z, y.w += v[p].w;
                    const int t = 4 * ((i >> 2) * a.split + c);
                    __nv_bfloat16* out = a.out + (t0 + t) * a.out_stride + row;
                    store_rows(out, a.out_stride, row < a.N, t, n_tok, ptx::cvt_bf16x2(y.x, y.y));
                    store_rows(out + 2 * a.out_stride, a.out_stride, row < a.N, t + 2, n_tok, ptx::cvt_bf16x2(y.z, y.w));
                }
            };
            if (a.split == 2) add(Int<2>());
            else add(Int<8>());
        }
    }
    __syncthreads();
    KT_MARK(K_MX_LINEAR, 2);
    if (*abort_flag) {
        // let copies still in flight into this CTA's shared memory land
        const uint64_t t0 = ptx::globaltimer();
        while (ptx::globaltimer() - t0 < 200000ull) {
        }
    }
    if (PAIR) ptx::cluster_sync_all();   // the other CTA reads this one's shared memory and arrives on its barriers
    ptx::tc_fence_after();
    if (warp == 1) {
        if (PAIR) ptx::tmem2_dealloc(tmem, 512);
        else ptx::tmem_dealloc(tmem, 512);
    }
}

// A bf16 x as two e4m3 terms a row (rows 2t and 2t + 1 of xq) and a scale byte a
// block (quant.cuh); a block with a NaN or an infinity has byte 255 and codes 0.
// PIECES of 16 bytes a thread, their loads under way together: with many rows four in blocks of 128 (bound by HBM; the product
// with 4096 rows of 4096 takes 118 us, in blocks of 256 119.5, with one piece 128), with few one in blocks of 256 (latency; 512 rows of
// 4096 21.7 us, in blocks of 128 22.3; 128 rows of 7168 19.6, with four pieces 21).
constexpr int split_threads(int pieces) { return pieces == 1 ? 256 : 128; }
template <int PIECES>
__global__ void __launch_bounds__(split_threads(PIECES)) k_mx_split(const __nv_bfloat16* x, int64_t stride, int K, uint8_t* xq, uint8_t* xs) {
    constexpr int THREADS = split_threads(PIECES);
    const int t = blockIdx.x, first = blockIdx.y * THREADS * PIECES + threadIdx.x, n = K / 8;
    const uint4* row = reinterpret_cast<const uint4*>(x + t * stride);
    KT_MARK(K_MX_SPLIT, 0);
    pdl_wait();
    pdl_trigger();   // (after the wait: the product reads the weights as soon as it starts)
    KT_MARK(K_MX_SPLIT, 1);
    uint4 v[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int c = first + i * THREADS;
        v[i] = c < n ? ld_dep(row + c) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int c = first + i * THREADS;
        QuantChunk q = quantize_vals(v[i]);
        if (q.amax >= 0x7F800000u) {
            q.hi = q.lo = make_uint2(0, 0);
            q.e = 255;
        }
        if (c >= n) continue;
        uint8_t* to = xq + (size_t)2 * t * K + 8 * c;
        *reinterpret_cast<uint2*>(to) = q.hi;
        *reinterpret_cast<uint2*>(to + K) = q.lo;
        if ((c & 3) == 0) xs[(size_t)t * (K / 32) + (c >> 2)] = (uint8_t)q.e;
    }
    KT_MARK(K_MX_SPLIT, 2);
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

constexpr int L_CTAS = 152;   // a GB300's SMs (with fewer the cuts are right all the same, but chosen for these)
// How many clusters of 0 .. 8 such CTAs (one an SM) a GB300 runs at once (cudaOccupancyMaxActiveClusters)
constexpr int CLUSTERS[9] = {0, 152, 76, 46, 36, 28, 23, 15, 15};
}  // namespace

// The cut with the least estimated time: a launch costs `start`, a round of tiles a stage's time for each of its
// stages, every round behind the first `round` more, and sharing K `join` (us).  The numbers were fitted to 591 measured
// cuts of 58 products, T = 1 .. 2048, operands in L2; of 70 products, T = 1 .. 8192, measured since, what it takes is 0.5% slower than
// the best cut on average, 8% at most.  For instance T = 256, N = 6144, K = 4096, MXFP4 x: pairs with 128 tokens 9.1 us, tiles of
// 128 tokens 11.6; bf16 x, T = 8, N = 16384, K = 8192: tiles of 16 tokens 15.3, of 8 18.5; T = 4096: pairs with 224
// tokens 117, with 256 128.
void mx_cut(MxDims& d) {
    struct Single {
        int nt;
        float start, stage, join, round;
    };
    static const Single mx[4] = {{16, 3.05f, 0.273f, 0.22f, 0.57f}, {32, 3.48f, 0.287f, 0.05f, 0.13f}, {64, 4.45f, 0.307f, -0.28f, 0.21f},
                                 {128, 5.23f, 0.431f, -0.13f, 0.96f}};
    static const Single bf[4] = {{8, 3.11f, 0.485f, 0.46f, 0.1f}, {16, 4.48f, 0.339f, 0.71f, 0.25f}, {32, 5.34f, 0.364f, 0.32f, 0.f},
                                 {64, 6.17f, 0.491f, -0.27f, 0.57f}};
    float least = INFINITY;
    auto take = [&](float t, int cg, int nt, int split) {
        if (t < least) least = t, d.cg = cg, d.nt = nt, d.split = split;
    };
    const int64_t nk = (d.K + 255) / 256;
    for (const Single& c : d.x_mx ? mx : bf) {
        if (c.nt == 8 && d.K % 512) continue;   // its kernel takes the scales by 16 bytes
        const int64_t tiles = (int64_t)((d.N + LM - 1) / LM) * ((d.T + c.nt - 1) / c.nt);
        const int64_t rounds = (tiles + L_CTAS - 1) / L_CTAS;
        for (int n = 2; n <= 8 && n <= nk; ++n)
            if (tiles <= CLUSTERS[n]) take(c.start + c.join + c.stage * ((nk + n - 1) / n), 1, c.nt, n);
        take(c.start + c.round * (rounds - 1) + c.stage * (rounds * nk), 1, c.nt, 1);
    }
    for (int nt = 64; nt <= 256; nt += 32) {
        const int64_t tiles = (int64_t)((d.N + 2 * LM - 1) / (2 * LM)) * ((d.T + nt - 1) / nt);
        const int64_t rounds = (tiles + L_CTAS / 2 - 1) / (L_CTAS / 2);
        if (d.x_mx) take(4.72f + 0.0043f * nt + 0.69f * (rounds - 1) + (0.312f + 0.00022f * nt) * (rounds * nk), 2, nt, 1);
        else take(7.11f + 0.0014f * nt + 0.37f * (rounds - 1) + (0.227f + 0.00138f * nt) * (rounds * (d.K / 128)), 2, nt, 1);
    }
}

namespace {

struct LLayout {
    size_t xq, xs, total;
};
LLayout layout(const MxDims& d) {
    LLayout L;
    L.xq = align256(WS_ZERO_PREFIX);
    // k_mx_split's terms of a bf16 x, room for them also where the cut makes them in the product's kernel: which cut that is
    // does not follow T alone, and a workspace for many tokens has to serve fewer
    L.xs = L.xq + (d.x_mx ? 0 : align256((size_t)2 * d.T * d.K));
    L.total = L.xs + (d.x_mx ? 0 : align256((size_t)d.T * (d.K / 32)));
    return L;
}

template <bool XMX, int NT, int CG>
cudaError_t launch_tiles(const MxDims& d, const MxArgs& p, cudaStream_t st) {
    using C = LCfg<XMX, NT, CG>;
    const LLayout L = layout(d);
    const int nt = d.nt;
    CUtensorMap tm_w, tm_x;
    const uint64_t N = d.N, T = d.T, K = d.K;
    const CUtensorMapDataType U8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    bool ok;
    if (XMX) {
        // packed rows of K / 2 bytes, 128 bytes (256 K) a stage
        const uint64_t w_d[2] = {K / 2, N}, x_d[2] = {K / 2, T}, s[1] = {K / 2};
        const uint32_t w_b[2] = {128, LM}, x_b[2] = {128, CG == 2 ? (uint32_t)nt / 2 : (uint32_t)NT};
        ok = make_map(&tm_w, U8, p.w, 2, w_d, s, w_b, CU_TENSOR_MAP_SWIZZLE_128B) &&
             make_map(&tm_x, U8, p.x, 2, x_d, s, x_b, CU_TENSOR_MAP_SWIZZLE_128B);
    } else {
        // codes {128, N rows, K/128 slabs}; xq {128 bytes, 2T rows, K/128 slabs}, or its terms apart
        // {128 bytes, T rows, 2 terms, K/128 slabs}
        const uint64_t w_d[3] = {128, N, K / 128}, w_s[2] = {K / 2, 64}, x_d[3] = {128, 2 * T, K / 128}, x_s[2] = {K, 128};
        const uint64_t t_d[4] = {128, T, 2, K / 128}, t_s[3] = {2 * K, K, 128};
        const uint32_t w_b[3] = {128, LM, C::WORDS}, x_b[3] = {128, (uint32_t)C::NB, 2}, t_b[4] = {128, (uint32_t)nt / 2, 2, 1};
        const uint64_t r_d[2] = {K, T}, r_s[1] = {2 * (uint64_t)d.x_stride};
        const uint32_t r_b[2] = {256, (uint32_t)NT};
        ok = make_map(&tm_w, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, p.w, 3, w_d, w_s, w_b, CU_TENSOR_MAP_SWIZZLE_128B) &&
             (C::FUSED ? make_map(&tm_x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.x, 2, r_d, r_s, r_b, CU_TENSOR_MAP_SWIZZLE_NONE)
              : CG == 2 ? make_map(&tm_x, U8, p.ws + L.xq, 4, t_d, t_s, t_b, CU_TENSOR_MAP_SWIZZLE_128B)
                        : make_map(&tm_x, U8, p.ws + L.xq, 3, x_d, x_s, x_b, CU_TENSOR_MAP_SWIZZLE_128B));
    }
    if (!ok) return cudaErrorInvalidValue;
    static std::atomic<bool> attribute_set[64];   // (a device's kernel attribute: set once, 0.3 us of a call)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !attribute_set[dev])) {
        e = cudaFuncSetAttribute(k_mx_linear<XMX, NT, CG>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e == cudaSuccess && dev < 64) attribute_set[dev] = true;
    }
    if (e != cudaSuccess) return e;
    LArgs a;
    a.w_scales = p.w_scales;
    a.xs = XMX ? p.xs : reinterpret_cast<const uint8_t*>(p.ws + L.xs);
    a.out = reinterpret_cast<__nv_bfloat16*>(p.out);
    a.sb = reinterpret_cast<StatusBlock*>(p.ws);
    a.T = d.T;
    a.N = d.N;
    a.K = d.K;
    a.out_stride = d.out_stride;
    a.nk = (d.K + C::KS - 1) / C::KS;
    a.mt = (d.N + CG * LM - 1) / (CG * LM);
    a.nt = nt;
    a.tt = (d.T + nt - 1) / nt;
    const int64_t tiles = (int64_t)a.mt * a.tt;
    const int workers = (num_sms() < L_CTAS ? num_sms() : L_CTAS) / CG;
    a.tiles = (int)tiles;
    a.split = d.split;
    const int ctas = d.split > 1 ? (int)tiles * d.split : (int)(tiles < workers ? tiles : workers);
    a.vec = d.K % 512 == 0;
    a.w_once = a.tt == 1;
    // with most of a tile's tokens copies further ahead only get in the way of the others (T = 4096, N = 4864,
    // K = 4096, 256 tokens: three 91.8 us, four 93.5; T = 512, N = 6144, 192 tokens: 23.4 and 22.2)
    a.under_way = nt > 192 ? 3 : 4;
    const int gm = Segment<CG>::GM;
    a.workers = Div(ctas);
    a.by_split = Div(a.split);
    a.by_band = Div(gm * a.tt);
    a.by_last = Div(a.mt % gm ? a.mt % gm : gm);
    if (!C::FIRST) {
        timing_begin(K_MX_SPLIT, st);
        const bool many = (int64_t)d.T * (d.K / 8) > (int64_t)num_sms() * 4096;   // more than two rounds of the SMs' threads
        const int pieces = many ? 4 : 1, threads = split_threads(pieces), per = threads * pieces;
        e = launch_pdl(many ? k_mx_split<4> : k_mx_split<1>, dim3(d.T, (d.K / 8 + per - 1) / per), dim3(threads), 0, st,
                       reinterpret_cast<const __nv_bfloat16*>(p.x), d.x_stride, d.K,
                       reinterpret_cast<uint8_t*>(p.ws + L.xq), reinterpret_cast<uint8_t*>(p.ws + L.xs));
        timing_end(st);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(ctas * CG));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM - (C::TERMS == 2 ? (C::S - a.under_way) * C::STAGE : 0);   // (what is left is L1's)
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG * a.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CG * a.split > 1 ? 2 : 1;
    timing_begin(K_MX_LINEAR, st);
    e = cudaLaunchKernelEx(&cfg, k_mx_linear<XMX, NT, CG>, tm_w, tm_x, a);
    timing_end(st);
    return e;
}

}  // namespace

size_t mx_linear_ws_bytes(const MxDims& d) { return layout(d).total; }

cudaError_t launch_mx_linear(const MxDims& d, const MxArgs& a, cudaStream_t st) {
    KT_BIND();
    if (d.x_mx) {
        if (d.cg == 2) return launch_tiles<true, 256, 2>(d, a, st);
        switch (d.nt) {
            case 16: return launch_tiles<true, 16, 1>(d, a, st);
            case 32: return launch_tiles<true, 32, 1>(d, a, st);
            case 64: return launch_tiles<true, 64, 1>(d, a, st);
            default: return launch_tiles<true, 128, 1>(d, a, st);
        }
    }
    if (d.cg == 2) return launch_tiles<false, 256, 2>(d, a, st);
    switch (d.nt) {
        case 8: return launch_tiles<false, 8, 1>(d, a, st);
        case 16: return launch_tiles<false, 16, 1>(d, a, st);
        case 32: return launch_tiles<false, 32, 1>(d, a, st);
        default: return launch_tiles<false, 64, 1>(d, a, st);
    }
}

}  // namespace moe

#ifdef MOE_WAIT_TEST
// Test-only export of the wait-test build: a kernel of one warp that lets its successor start at once and ends `us`
// microseconds later, for calls whose waits have a shorter limit.
__global__ void k_test_early(int us) {
    moe::pdl_trigger();
    const uint64_t t0 = moe::ptx::globaltimer();
    while (moe::ptx::globaltimer() - t0 < 1000ull * us) {
    }
}
extern "C" int moe_test_early_kernel(int us, void* stream) {
    if (us < 0 || us > 100000) return MOE_ERR_INVALID_ARG;
    k_test_early<<<1, 32, 0, (cudaStream_t)stream>>>(us);
    return moe::cuda_rc(cudaGetLastError());
}
#endif

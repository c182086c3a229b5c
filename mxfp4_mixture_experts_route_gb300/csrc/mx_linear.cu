// out[t, n] = sum_k x[t, k] w[n, k] with MXFP4 weights, on the tensor cores.
//
// The weights are the MMA's A (M = 128 of their rows), the tokens its B.  With MXFP4 x
// both stay packed (tcgen05.mma kind::mxf4, K = 64).  A bf16 x enters as
// in the experts' kernel (experts_mx.cu): as two e4m3 terms a row, hi and lo, under
// a power of two a block of 32, which a small kernel (k_mx_split) writes first; the TMA
// unpacks the weights' codes for kind::mxf8f6f4 and a token takes two columns of the
// MMA, added at the end.  Either way the tensor core applies the block scales.
//
// All tiles (128 weight rows x NT tokens) stand one after the other on a line, cut into
// stages of 256 K; each of the persistent CTAs takes an equal share of the line.
// A tile that a cut divides is joined without waiting: every CTA writes its
// part to the workspace and counts itself, and the one that comes last adds the
// parts in the order of the line (so the sum does not depend on who came last).
//
// Warps: 0 TMA, 1 MMA, 2-5 scales (global memory -> TMEM, 1024 K ahead in
// registers), 6-9 the accumulators' way out.
#include "mx.cuh"
#include "quant.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int LM = 128;                       // weight rows a tile
constexpr int LKS = 256;                      // K a stage
constexpr int L_THREADS = 320;
constexpr int SF_SLOT = 64;                   // TMEM columns of a stage's scales
constexpr int SF_A1 = 16, SF_B0 = 32, SF_B1 = 48;
constexpr uint64_t L_WAIT_NS = 2000000000ull;
constexpr int L_SITE = 300;                   // detail of MOE_ERR_TIMEOUT: site of the wait

template <bool XMX, int NT>
struct LCfg {
    static constexpr int NB = XMX ? NT : 2 * NT;                  // MMA N
    static constexpr int A_BYTES = XMX ? LM * 128 : LM * 256;     // a stage's weights in shared memory
    static constexpr int B_BYTES = XMX ? NB * 128 : NB * 256;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int ACC = NB <= 128 ? 2 : 1;                 // accumulators
    static constexpr int SF_COL0 = (ACC * NB + 63) / 64 * 64;
    static constexpr int S_TMEM = (512 - SF_COL0) / SF_SLOT;
    static constexpr bool XCH = NB > 32;                          // token scales exchanged through shared memory
    static constexpr int XCH_BYTES = XCH ? 2 * 8 * NT * 4 : 0;
    static constexpr int S_FIT = (232448 - 1024 - 512 - XCH_BYTES) / STAGE;
    static constexpr int S = S_FIT < S_TMEM ? S_FIT : S_TMEM;
    static constexpr int SMEM = 1024 + S * STAGE + XCH_BYTES + 512;
    static_assert(S >= 2 && SMEM <= 232448, "stages");
};

struct LArgs {
    const uint8_t *w_scales, *xs;             // [N][K/32], [T][K/32]
    __nv_bfloat16* out;
    float* parts;                             // [CTA][2][NT][LM]
    uint32_t* count;                          // [CTA]: parts of the tile that CTA began and did not finish
    StatusBlock* sb;
    int T, N, K;
    int64_t out_stride;
    int nk, tt;                               // stages a tile, token tiles
    int64_t total;                            // stages on the line
    int vec;                                  // scale rows are 16-byte aligned
    int w_once;
};

// [first, last) of CTA c's share of the line, and the CTA that holds stage p
__device__ __forceinline__ int64_t share(int64_t total, int c, int n) { return total * c / n; }
__device__ __forceinline__ int holder_of(int64_t p, int64_t total, int n) { return (int)(((p + 1) * n - 1) / total); }

// A CTA's segments: stages [k0, k1) of a tile, one tile after the other.
struct Segment {
    int64_t at, end, tile;
    int k0, k1, nk;
    __device__ __forceinline__ Segment(const LArgs& a)
        : at(share(a.total, blockIdx.x, gridDim.x)), end(share(a.total, blockIdx.x + 1, gridDim.x)), nk(a.nk) {
        tile = at / nk;
        k0 = (int)(at - tile * nk);
        cut();
    }
    __device__ __forceinline__ void cut() { k1 = (int)min((int64_t)nk, k0 + (end - at)); }
    __device__ __forceinline__ bool more() const { return at < end; }
    __device__ __forceinline__ void next() {
        at += k1 - k0;
        ++tile;
        k0 = 0;
        cut();
    }
};

// Scale bytes 32 g .. 32 g + 31 of a row (1024 K); past the row's end 127 (its codes are zeros).
__device__ __forceinline__ void load_scales(const uint8_t* row, int g, int kb, bool vec, uint32_t (&w)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0x7F7F7F7Fu;
    if (row == nullptr) return;
    row += 32 * g;
    const int n = kb - 32 * g;
    if (vec) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (16 * i < n) {
                const uint4 v = ld_dep(reinterpret_cast<const uint4*>(row) + i);
                w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
            }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (4 * i < n) w[i] = ld_dep(reinterpret_cast<const uint32_t*>(row) + i);
    }
}

template <bool XMX, int NT>
__global__ void __launch_bounds__(L_THREADS, 1)
    k_mx_linear(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, const LArgs a) {
    using C = LCfg<XMX, NT>;
    constexpr int S = C::S, NB = C::NB, ACC = C::ACC;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint32_t* xch = reinterpret_cast<uint32_t*>(sm + S * C::STAGE);     // [2][8 words][NT] token scales
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + S * C::STAGE + C::XCH_BYTES);
    uint64_t* empty = full + S;          // the stage's MMAs are done
    uint64_t* acc_full = empty + S;
    uint64_t* acc_empty = acc_full + ACC;
    uint64_t* fin = acc_empty + ACC;
    uint32_t* holder = reinterpret_cast<uint32_t*>(fin + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(holder + 1);
    volatile int* last_flag = abort_flag + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    KT_MARK(K_MX_LINEAR, 0);
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            ptx::mbar_init(&full[i], 1 + 4);      // TMA, the four scale warps
            ptx::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < ACC; ++i) {
            ptx::mbar_init(&acc_full[i], 1);
            ptx::mbar_init(&acc_empty[i], 4);
        }
        ptx::mbar_init(fin, 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&tm_w);
        ptx::prefetch_tensormap(&tm_x);
    }
    if (warp == 1) ptx::tmem_alloc(holder, 512);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *holder;
    // with MXFP4 x this is the call's first kernel: it reads nothing before its wait
    if (XMX) pdl_wait();

    auto fail = [&](int site) {
        latch_status(a.sb, MOE_ERR_TIMEOUT, L_SITE + site);
        *abort_flag = 1;
    };
    if (warp == 0) {
        // ------------------------------------------------------------ TMA
        const uint64_t pol_w = a.w_once ? ptx::policy_evict_first() : ptx::policy_evict_last();
        const uint64_t pol_x = ptx::policy_evict_last();
        auto weights = [&](int64_t tile, int k, int s) {
            uint8_t* st = sm + s * C::STAGE;
            const int row = (int)(tile / a.tt) * LM;
            ptx::mbar_arrive_expect_tx(&full[s], LM * 128 + C::B_BYTES);
            if (XMX)
                ptx::tma_load_2d(st, &tm_w, 128 * k, row, &full[s], pol_w);
            else
                ptx::tma_load_3d(st, &tm_w, 0, row, 2 * k, &full[s], pol_w);
        };
        auto tokens = [&](int64_t tile, int k, int s) {
            uint8_t* st = sm + s * C::STAGE + C::A_BYTES;
            const int row = (int)(tile % a.tt) * NB;
            if (XMX)
                ptx::tma_load_2d(st, &tm_x, 128 * k, row, &full[s], pol_x);
            else
                ptx::tma_load_3d(st, &tm_x, 0, row, 2 * k, &full[s], pol_x);
        };
        if (lane == 0) {
            int pre = 0;
            if (!XMX) {
                // the first stages' weights, inputs of the call, before the wait for the tokens' terms
                int i = 0;
                for (Segment g(a); g.more() && i < S; g.next())
                    for (int k = g.k0; k < g.k1 && i < S; ++k, ++i) weights(g.tile, k, i);
                pre = i;
                pdl_wait();
            }
            bool ok = true;
            int it = 0;
            for (Segment g(a); ok && g.more(); g.next()) {
                for (int k = g.k0; k < g.k1; ++k, ++it) {
                    const int s = it % S;
                    if (it >= pre) {
                        if (!ptx::mbar_wait(&empty[s], ((it / S) & 1) ^ 1, abort_flag, L_WAIT_NS)) {
                            fail(1);
                            ok = false;
                            break;
                        }
                        weights(g.tile, k, s);
                    }
                    tokens(g.tile, k, s);
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA
        int it = 0, seg = 0;
        bool ok = true;
        for (Segment g(a); ok && g.more(); g.next(), ++seg) {
            const int ab = seg % ACC;
            if (!ptx::mbar_wait_warp(&acc_empty[ab], ((seg / ACC) & 1) ^ 1, abort_flag, L_WAIT_NS)) {
                if (lane == 0) fail(2);
                ok = false;
            }
            const uint32_t d_tmem = tmem + ab * NB;
            for (int k = g.k0; ok && k < g.k1; ++k, ++it) {
                const int s = it % S;
                if (!ptx::mbar_wait_warp(&full[s], (it / S) & 1, abort_flag, L_WAIT_NS)) {
                    if (lane == 0) fail(3);
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t a0 = ptx::smem_u32(sm + s * C::STAGE), b0 = a0 + C::A_BYTES;
                const uint32_t col = tmem + C::SF_COL0 + s * SF_SLOT;
                if (ptx::elect_one()) {
                    if constexpr (XMX) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            ptx::mma_mxf4_ss(d_tmem, ptx::smem_desc_sw128(a0 + 32 * j), ptx::smem_desc_sw128(b0 + 32 * j),
                                             ptx::idesc_mxf4(LM, NB, 2 * (j & 1), 2 * (j & 1)), k > g.k0 || j > 0,
                                             col + SF_A1 * (j >> 1), col + SF_B0 + (SF_B1 - SF_B0) * (j >> 1));
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int h = j >> 2, q = j & 3;   // 128-K slab, K step within it
                            ptx::mma_mx_ss(d_tmem, ptx::smem_desc_sw128(a0 + h * LM * 128 + 32 * q),
                                           ptx::smem_desc_sw128(b0 + h * NB * 128 + 32 * q),
                                           ptx::idesc_mx_e2m1_e4m3(LM, NB, q, q), k > g.k0 || j > 0,
                                           col + SF_A1 * h, col + SF_B0 + (SF_B1 - SF_B0) * h);
                        }
                    }
                    ptx::mma_commit(&empty[s]);
                    if (k + 1 == g.k1) ptx::mma_commit(&acc_full[ab]);
                }
                __syncwarp();
            }
        }
        // every MMA issued above has completed before TMEM is released
        if (ptx::elect_one()) ptx::mma_commit(fin);
        __syncwarp();
        ptx::mbar_wait(fin, 0, abort_flag, L_WAIT_NS);
    } else if (warp < 6) {
        // ------------------------------------------------------------ scales
        const int q = warp & 3, r = 32 * q + lane;      // TMEM lane quarter; weight row of this thread
        const uint32_t lane_base = (uint32_t)(32 * q) << 16;
        const int kb = a.K / 32;
        constexpr int OWN = !C::XCH ? 1 : NT > 128 ? NT / 128 : 1;    // tokens whose scales this thread loads
        uint32_t wa[8], wb[OWN][8], na[8], nb[OWN][8];
        auto load_a = [&](int64_t tile, int grp) {
            const int64_t row = tile / a.tt * LM + r;
            load_scales(row < a.N ? a.w_scales + row * kb : nullptr, grp, kb, a.vec, na);
        };
        auto load_b = [&](int64_t tile, int grp) {
#pragma unroll
            for (int u = 0; u < OWN; ++u) {
                const int j = !C::XCH ? (XMX ? lane : lane >> 1) % NT : r + 128 * u;
                const int64_t t = tile % a.tt * NT + j;
                load_scales(j < NT && t < a.T ? a.xs + t * kb : nullptr, grp, kb, a.vec, nb[u]);
            }
        };
        Segment g(a);
        if (g.more()) load_a(g.tile, g.k0 >> 2);
        if (!XMX) pdl_wait();
        if (g.more()) load_b(g.tile, g.k0 >> 2);
        // a warp whose wait gave up goes on without waiting: the four share the barrier below
        int it = 0, buf = 0;
        bool ok = true;
        for (; g.more(); g.next()) {
            for (int grp = g.k0 >> 2; 4 * grp < g.k1; ++grp) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    wa[i] = na[i];
#pragma unroll
                    for (int u = 0; u < OWN; ++u) wb[u][i] = nb[u][i];
                }
                // the next group's, under way while this one's stages go through
                if (4 * (grp + 1) < g.k1) {
                    load_a(g.tile, grp + 1);
                    load_b(g.tile, grp + 1);
                } else {
                    Segment n = g;
                    n.next();
                    if (n.more()) {
                        load_a(n.tile, 0);
                        load_b(n.tile, 0);
                    }
                }
                uint32_t* xb = xch + buf * 8 * NT;
                if constexpr (C::XCH) {
#pragma unroll
                    for (int u = 0; u < OWN; ++u)
                        if (r + 128 * u < NT)
#pragma unroll
                            for (int i = 0; i < 8; ++i) xb[i * NT + r + 128 * u] = wb[u][i];
                    // (one barrier a group: a buffer is written again two groups later)
                    ptx::named_bar_sync(1, 128);
                    buf ^= 1;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = 4 * grp + i;
                    if (!ok || k < g.k0 || k >= g.k1) continue;
                    const int s = it % S;
                    if (!ptx::mbar_wait_warp(&empty[s], ((it / S) & 1) ^ 1, abort_flag, L_WAIT_NS)) {
                        if (lane == 0) fail(4);
                        ok = false;
                        continue;
                    }
                    if (__vcmpeq4(wa[2 * i], 0xFFFFFFFFu) | __vcmpeq4(wa[2 * i + 1], 0xFFFFFFFFu))
                        latch_status(a.sb, MOE_ERR_BAD_SCALE, 255);
                    const uint32_t col = tmem + lane_base + C::SF_COL0 + s * SF_SLOT;
                    // row r is read at lane r mod 32 of this quarter, column col + q (a warp writes
                    // its word into all four columns; the other quarters' are never read)
                    ptx::tmem_st4_rep(col, wa[2 * i]);
                    ptx::tmem_st4_rep(col + SF_A1, wa[2 * i + 1]);
                    // column n of B: lane n mod 32 of every quarter, column + n / 32
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t to = col + SF_B0 + (SF_B1 - SF_B0) * h;
                        if constexpr (!C::XCH) {
                            ptx::tmem_st4_rep(to, wb[0][2 * i + h]);
                        } else {
                            uint32_t v[NB / 32];
#pragma unroll
                            for (int c = 0; c < NB / 32; ++c)
                                v[c] = xb[(2 * i + h) * NT + (XMX ? 32 * c + lane : 16 * c + (lane >> 1))];
                            if constexpr (NB == 64)
                                ptx::tmem_st2(to, v[0], v[1]);
                            else if constexpr (NB == 128)
                                ptx::tmem_st4(to, v[0], v[1], v[2], v[3]);
                            else
                                ptx::tmem_st8(to, v);
                        }
                    }
                    ptx::tmem_st_wait();
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&full[s]);
                    ++it;
                }
            }
        }
    } else {
        // ------------------------------------------------------------ accumulators
        const int q = warp & 3, r = 32 * q + lane;
        const uint32_t lane_base = (uint32_t)(32 * q) << 16;
        if (!XMX) pdl_wait();   // (the workspace's parts: an earlier call may still read its own)
        pdl_trigger();
        int seg = 0;
        for (Segment g(a); g.more(); g.next(), ++seg) {
            const int ab = seg % ACC;
            const bool got = ptx::mbar_wait_warp(&acc_full[ab], (seg / ACC) & 1, abort_flag, L_WAIT_NS);
            if (!got && lane == 0) fail(5);
            // the four warps decide together (they share barriers below)
            if (threadIdx.x == 6 * 32) last_flag[1 + (seg & 1)] = *abort_flag;
            ptx::named_bar_sync(2, 128);
            if (last_flag[1 + (seg & 1)]) break;
            ptx::tc_fence_after();
            const int row = (int)(g.tile / a.tt) * LM + r, t0 = (int)(g.tile % a.tt) * NT;
            const bool whole = g.k0 == 0 && g.k1 == g.nk;
            float* part = a.parts + ((int64_t)blockIdx.x * 2 + (g.k0 == 0 ? 1 : 0)) * NT * LM + r;
            const int n_tok = min(NT, a.T - t0);
#pragma unroll 1
            for (int c = 0; c < NB; c += 16) {
                uint32_t v[16];
                ptx::tmem_ld16(tmem + lane_base + ab * NB + c, v);
                ptx::tmem_ld_wait16(v);
#pragma unroll
                for (int j = 0; j < (XMX ? 16 : 8); ++j) {
                    const int t = (XMX ? c : c / 2) + j;
                    const float y = XMX ? __uint_as_float(v[j])
                                        : __uint_as_float(v[2 * j]) + __uint_as_float(v[2 * j + 1]);
                    if (t >= n_tok) continue;
                    if (!whole)
                        part[t * LM] = y;
                    else if (row < a.N)
                        a.out[(t0 + t) * a.out_stride + row] = __float2bfloat16_rn(y);
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&acc_empty[ab]);
            if (whole) continue;
            // the tile's parts: those of CTAs c0 .. c1
            const int64_t p0 = g.tile * g.nk;
            const int c0 = holder_of(p0, a.total, gridDim.x), c1 = holder_of(p0 + g.nk - 1, a.total, gridDim.x);
            __threadfence();
            ptx::named_bar_sync(2, 128);
            if (threadIdx.x == 6 * 32) {
                const uint32_t was = atomicAdd(&a.count[c0], 1u);
                const bool last = was == (uint32_t)(c1 - c0);
                if (last) a.count[c0] = 0;
                __threadfence();
                last_flag[0] = last;
            }
            ptx::named_bar_sync(2, 128);
            if (!last_flag[0]) continue;
            // four rows a lane, a token a warp at a time; J tokens' loads under way together
            constexpr int J = NT / 4 < 8 ? NT / 4 : 8;
            const int row4 = (int)(g.tile / a.tt) * LM + 4 * lane;
            const float* p = a.parts + ((int64_t)c0 * 2 + 1) * NT * LM + 4 * lane;
#pragma unroll 1
            for (int tb = warp - 6; tb < n_tok; tb += 4 * J) {
                float4 y[J];
#pragma unroll
                for (int j = 0; j < J; ++j) y[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
                for (int c = c0; c <= c1; ++c) {
                    const float* from = c == c0 ? p : p + ((int64_t)(c - c0) * 2 - 1) * NT * LM;
                    float4 v[J];
#pragma unroll
                    for (int j = 0; j < J; ++j)
                        v[j] = tb + 4 * j < n_tok ? ld_dep(reinterpret_cast<const float4*>(from + (tb + 4 * j) * LM))
                                                  : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int j = 0; j < J; ++j)
                        y[j].x += v[j].x, y[j].y += v[j].y, y[j].z += v[j].z, y[j].w += v[j].w;
                }
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if (tb + 4 * j < n_tok && row4 < a.N)
                        *reinterpret_cast<uint2*>(a.out + (t0 + tb + 4 * j) * a.out_stride + row4) =
                            make_uint2(ptx::cvt_bf16x2(y[j].x, y[j].y), ptx::cvt_bf16x2(y[j].z, y[j].w));
            }
            ptx::named_bar_sync(2, 128);   // the flag is written again
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
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_dealloc(tmem, 512);
}

// A bf16 x as two e4m3 terms a row (rows 2t and 2t + 1 of xq) and a scale byte a
// block (quant.cuh); a block with a NaN or an infinity has byte 255 and codes 0.
constexpr int SPLIT_THREADS = 128;
__global__ void __launch_bounds__(SPLIT_THREADS) k_mx_split(const __nv_bfloat16* x, int64_t stride, int K, uint8_t* xq, uint8_t* xs) {
    const int t = blockIdx.x, c = blockIdx.y * SPLIT_THREADS + threadIdx.x, n = K / 8;
    KT_MARK(K_MX_SPLIT, 0);
    pdl_wait();
    pdl_trigger();   // (after the wait: the product reads the weights as soon as it starts)
    KT_MARK(K_MX_SPLIT, 1);
    QuantChunk q = quantize_chunk_dep(reinterpret_cast<const uint4*>(x + t * stride), c, c < n);
    if (q.amax >= 0x7F800000u) {
        q.hi = q.lo = make_uint2(0, 0);
        q.e = 255;
    }
    if (c < n) {
        uint8_t* row = xq + (size_t)2 * t * K + 8 * c;
        *reinterpret_cast<uint2*>(row) = q.hi;
        *reinterpret_cast<uint2*>(row + K) = q.lo;
        if ((c & 3) == 0) xs[(size_t)t * (K / 32) + (c >> 2)] = (uint8_t)q.e;
    }
    KT_MARK(K_MX_SPLIT, 2);
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// Tokens a tile: the fewest that hold T, up to 256 (MXFP4 x) or 64.
int tile_tokens(const MxDims& d) {
    const int most = d.x_mx ? 256 : 64;
    int n = d.x_mx ? 16 : 8;
    while (n < most && n < d.T) n *= 2;
    return d.x_mx && n == 32 ? 32 : n;
}

constexpr int L_CTAS = 160;   // at most as many CTAs as the workspace has parts for

struct LLayout {
    size_t count, parts, xq, xs, total;
};
LLayout layout(const MxDims& d) {
    LLayout L;
    L.count = sizeof(StatusBlock);            // in the zeroed prefix
    L.parts = align256(WS_ZERO_PREFIX);
    L.xq = L.parts + align256((size_t)L_CTAS * 2 * tile_tokens(d) * LM * 4);
    L.xs = L.xq + (d.x_mx ? 0 : align256((size_t)2 * d.T * d.K));
    L.total = L.xs + (d.x_mx ? 0 : align256((size_t)d.T * (d.K / 32)));
    return L;
}

template <bool XMX, int NT>
cudaError_t launch_tiles(const MxDims& d, const MxArgs& p, cudaStream_t st) {
    using C = LCfg<XMX, NT>;
    const LLayout L = layout(d);
    CUtensorMap tm_w, tm_x;
    const uint64_t N = d.N, T = d.T, K = d.K;
    const CUtensorMapDataType U8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    bool ok;
    if (XMX) {
        // packed rows of K / 2 bytes, 128 bytes (256 K) a stage
        const uint64_t w_d[2] = {K / 2, N}, x_d[2] = {K / 2, T}, s[1] = {K / 2};
        const uint32_t w_b[2] = {128, LM}, x_b[2] = {128, (uint32_t)C::NB};
        ok = make_map(&tm_w, U8, p.w, 2, w_d, s, w_b, CU_TENSOR_MAP_SWIZZLE_128B) &&
             make_map(&tm_x, U8, p.x, 2, x_d, s, x_b, CU_TENSOR_MAP_SWIZZLE_128B);
    } else {
        // codes {128, N rows, K/128 slabs}; xq {128 bytes, 2T rows, K/128 slabs}
        const uint64_t w_d[3] = {128, N, K / 128}, w_s[2] = {K / 2, 64}, x_d[3] = {128, 2 * T, K / 128}, x_s[2] = {K, 128};
        const uint32_t w_b[3] = {128, LM, 2}, x_b[3] = {128, (uint32_t)C::NB, 2};
        ok = make_map(&tm_w, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, p.w, 3, w_d, w_s, w_b, CU_TENSOR_MAP_SWIZZLE_128B) &&
             make_map(&tm_x, U8, p.ws + L.xq, 3, x_d, x_s, x_b, CU_TENSOR_MAP_SWIZZLE_128B);
    }
    if (!ok) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(k_mx_linear<XMX, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    LArgs a;
    a.w_scales = p.w_scales;
    a.xs = XMX ? p.xs : reinterpret_cast<const uint8_t*>(p.ws + L.xs);
    a.out = reinterpret_cast<__nv_bfloat16*>(p.out);
    a.parts = reinterpret_cast<float*>(p.ws + L.parts);
    a.count = reinterpret_cast<uint32_t*>(p.ws + L.count);
    a.sb = reinterpret_cast<StatusBlock*>(p.ws);
    a.T = d.T;
    a.N = d.N;
    a.K = d.K;
    a.out_stride = d.out_stride;
    a.nk = (d.K + LKS - 1) / LKS;
    a.tt = (d.T + NT - 1) / NT;
    a.total = (int64_t)((d.N + LM - 1) / LM) * a.tt * a.nk;
    a.vec = d.K % 512 == 0;
    a.w_once = a.tt == 1;
    if (!XMX) {
        timing_begin(K_MX_SPLIT, st);
        e = launch_pdl(k_mx_split, dim3(d.T, (d.K / 8 + SPLIT_THREADS - 1) / SPLIT_THREADS), dim3(SPLIT_THREADS), 0, st,
                       reinterpret_cast<const __nv_bfloat16*>(p.x), d.x_stride, d.K,
                       reinterpret_cast<uint8_t*>(p.ws + L.xq), reinterpret_cast<uint8_t*>(p.ws + L.xs));
        timing_end(st);
        if (e != cudaSuccess) return e;
    }
    const int sms = num_sms() < L_CTAS ? num_sms() : L_CTAS;
    timing_begin(K_MX_LINEAR, st);
    e = launch_pdl(k_mx_linear<XMX, NT>, dim3((unsigned)(a.total < sms ? a.total : sms)), dim3(L_THREADS), C::SMEM, st, tm_w,
                   tm_x, a);
    timing_end(st);
    return e;
}

}  // namespace

size_t mx_linear_ws_bytes(const MxDims& d) { return layout(d).total; }

cudaError_t launch_mx_linear(const MxDims& d, const MxArgs& a, cudaStream_t st) {
    KT_BIND();
    const int nt = tile_tokens(d);
    if (d.x_mx) {
        switch (nt) {
            case 16: return launch_tiles<true, 16>(d, a, st);
            case 32: return launch_tiles<true, 32>(d, a, st);
            case 64: return launch_tiles<true, 64>(d, a, st);
            case 128: return launch_tiles<true, 128>(d, a, st);
            default: return launch_tiles<true, 256>(d, a, st);
        }
    }
    switch (nt) {
        case 8: return launch_tiles<false, 8>(d, a, st);
        case 16: return launch_tiles<false, 16>(d, a, st);
        case 32: return launch_tiles<false, 32>(d, a, st);
        default: return launch_tiles<false, 64>(d, a, st);
    }
}

}  // namespace moe

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
// leaves fp32 partial results, which k_tree_join adds in key order.
//
// Two streams keep the tensor core and the exponentials busy side by side:
// S, P and O exist twice in TMEM, each with a warpgroup of softmax threads
// (a thread a row).  With two query tiles the streams are the tiles, and each
// K/V tile serves both; with one, the streams take alternate key tiles and are
// added at the segment's end.
//
// Warps: 0 TMA producer (K, V by page boxes; Q), 1 and 3 MMA issuers (one a
// stream), 2 cleans V tiles that hold keys some row does not see, 4-7 and 8-11
// the softmax.
#include "kv.cuh"
#include "tc_ptx.cuh"

#include <math_constants.h>

namespace moe {
namespace {

constexpr int A_THREADS = 384;
constexpr int A_CTAS = 152;                 // shares (SMs of a GB300)
constexpr int KT = 128;                     // keys a tile
constexpr int A_MISC = 3072;                // barriers and small tables
constexpr uint64_t A_WAIT_NS = 2000000000ull;
constexpr int SAN_SLOTS = 16;

template <int D, bool E4M3>
struct ACfg {
    static constexpr int ROWB = E4M3 ? D : 2 * D;            // bytes a key
    static constexpr int SW = ROWB < 128 ? ROWB : 128;       // swizzle width
    static constexpr int HALVES = ROWB / SW;
    static constexpr int SLOT = KT * ROWB;                   // a K or V tile
    static constexpr int QT = 128 * D * 2;                   // a query tile: bf16, or e4m3 hi and lo
    static constexpr int QMISC = E4M3 ? 1024 : 0;            // e4m3: row scales of two query tiles
    static constexpr int FIT = (232448 - A_MISC - QMISC - 2 * QT) / SLOT;
    static constexpr int NS = FIT < 16 ? FIT : 16;           // ring slots
    static constexpr int SMEM = 2 * QT + NS * SLOT + QMISC + A_MISC;
    static constexpr int KSTEP = E4M3 ? 32 : 16;             // K of one MMA
    // TMEM columns: S (P in its place) and O of each stream
    static constexpr uint32_t T_S = 0, T_O = 256;
};

// shared-memory tables behind the tiles
struct AMisc {
    uint64_t full[16], empty[16], q_full[2], q_empty[2], s_full[2], p_full[2], o_full, o_free, san[16], ml_full, qs_full, drain[2];
    uint32_t tmem;
    int abort;
    int first_b;
    int nan_seg[SAN_SLOTS];
    long long first_base, total;
    long long warp_sum[A_THREADS / 32];
    float2 ml[2][128];
};
static_assert(sizeof(AMisc) <= A_MISC, "misc");

struct ATabs {
    int G, tpt;                 // heads a group, tokens a query tile
    int box;                    // keys a TMA box: gcd(page, 128)
    int qbox;                   // tokens of the small query box
    int rp;                     // rows a partial result holds
    float2* part_ml;            // [2 A_CTAS][rp]: m (log2 units), l
    float* part_o;              // [2 A_CTAS][rp][D]
    struct Joint* joint;        // [A_CTAS]
    StatusBlock* sb;
};

// A divided segment, left by the CTA that holds its first key tile.
struct Joint {
    int rows;                   // 0: none
    int row0;                   // row of its first token
    int kvh;
    int last;                   // last CTA that holds a part
    long long total;
    int pad[2];
};

__device__ __forceinline__ long long share_begin(long long total, int c) { return total * c / A_CTAS; }

// key tiles of query-tile pair p of a request
__device__ __forceinline__ int pair_tiles(const KvDims& d, const KvReq& r, int p, int pt) {
    const int upto = d.W || (p + 1) * pt > r.n ? r.n : (p + 1) * pt;
    return (r.c + upto + KT - 1) / KT;
}
__device__ __forceinline__ long long request_tiles(const KvDims& d, const KvReq& r, int pt) {
    if (r.n == 0) return 0;
    const int np = (r.n + pt - 1) / pt;
    long long s = 0;
    if (d.W) {
        s = (long long)np * pair_tiles(d, r, 0, pt);
    } else {
        for (int p = 0; p < np; ++p) s += pair_tiles(d, r, p, pt);
    }
    return s * d.Hkv;
}

// The walk of one CTA over its share's segments; every role walks by itself.
struct Walk {
    long long pos, end;
    KvReq r;
    int b, h, p, np, kt;
    int k0, k1;                 // key tiles of the current segment's part
    __device__ __forceinline__ bool start(const KvDims& d, const AttnArgs& a, const AMisc* m, int pt) {
        pos = share_begin(m->total, blockIdx.x);
        end = share_begin(m->total, blockIdx.x + 1);
        if (pos >= end) return false;
        b = m->first_b;
        r = kv_request(d, a.ctx_len, a.row_start, b);
        np = (r.n + pt - 1) / pt;
        long long off = pos - m->first_base;
        const long long a_head = request_tiles(d, r, pt) / d.Hkv;
        h = (int)(off / a_head);
        off -= h * a_head;
        p = 0;
        while (off >= (kt = pair_tiles(d, r, p, pt))) {
            off -= kt;
            ++p;
        }
        k0 = (int)off;
        k1 = (int)(kt - k0 < end - pos ? kt : k0 + (end - pos));
        return true;
    }
    __device__ __forceinline__ bool next(const KvDims& d, const AttnArgs& a, int pt) {
        pos += k1 - k0;
        if (pos >= end) return false;
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
        kt = pair_tiles(d, r, p, pt);
        k0 = 0;
        k1 = (int)(kt < end - pos ? kt : end - pos);
        return true;
    }
    // the pair's tokens, and whether it has two query tiles
    __device__ __forceinline__ int tok0(int pt) const { return p * pt; }
    __device__ __forceinline__ int ntok(int pt) const { return r.n - p * pt < pt ? r.n - p * pt : pt; }
    // keys below this one are seen by every row of the segment
    __device__ __forceinline__ int all_see(const KvDims& d, int pt) const { return d.W ? r.c : r.c + p * pt + 1; }
};

// ring position of K tile j and V tile j of a segment of m tiles:
// K0 K1 V0 K2 V1 ... K(m-1) V(m-2) V(m-1), the order in which they are used
__device__ __forceinline__ uint32_t seq_k(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ uint32_t seq_v(int j, int m) { return j == m - 1 ? 2 * m - 1 : 2 * j + 2; }

__device__ __forceinline__ bool row_sees(const KvDims& d, const AttnArgs& a, int row, int i, int j) {
    if (d.W == 0) return j <= i;
    return (ld_dep(a.mask + (int64_t)row * d.W + (j >> 5)) >> (j & 31)) & 1;
}

// The weights are relative to a maximum m (kept as mc = m c) that follows the
// true one only when that is LAZY ahead, so that O is rescaled rarely; P stays
// below 2^(base + LAZY).  An e4m3 P is held above that format's smallest steps
// (2^-9): 2^5 at the maximum, at most 2^8 of 448.
template <bool E4M3>
__host__ __device__ constexpr float p_base() { return E4M3 ? 5.f : 0.f; }

// One thread's row of a tile: its 128 scores at t_s become weights in their
// place, o (the row of O at t_o) is rescaled when the maximum moves.  Sums and
// maxima run in four chains of pairs, so that no chain of dependent
// operations is longer than 16.
template <int D, bool E4M3>
__device__ __forceinline__ void softmax_tile(uint32_t t_s, uint32_t t_o, float c, bool part, const uint32_t* vis,
                                             bool have_o, float& mc, float& l) {
    constexpr float LAZY = E4M3 ? 3.f : 8.f;
    float s[4][32];
#pragma unroll
    for (int k = 0; k < 4; ++k) ptx::tmem_ld32(t_s + 32 * k, s[k]);
#pragma unroll
    for (int k = 0; k < 4; ++k) ptx::tmem_ld_wait32(s[k]);
    if (part) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int x = 0; x < 32; ++x) s[k][x] = (vis[k] >> x) & 1 ? s[k][x] : -CUDART_INF_F;
    }
    float tops[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        tops[k] = fmaxf(s[k][0], s[k][1]);
#pragma unroll
        for (int x = 2; x < 32; x += 2) tops[k] = ptx::max3(tops[k], s[k][x], s[k][x + 1]);
    }
    const float top = fmaxf(ptx::max3(tops[0], tops[1], tops[2]), tops[3]) * c;
    const bool first = mc == -CUDART_INF_F;
    const bool move = first || top > mc + LAZY;
    // (a first maximum finds nothing but zeros in its row of O)
    const float f = move && !first ? ptx::ex2(mc - top) : 1.f;
    if (move) mc = top;
    if (have_o && __any_sync(0xffffffffu, move && !first)) {
#pragma unroll
        for (int x = 0; x < D; x += 16) {
            uint32_t o[16];
            ptx::tmem_ld16(t_o + x, o);
            ptx::tmem_ld_wait16(o);
#pragma unroll
            for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
            ptx::tmem_st16(t_o + x, o);
        }
    }
    const float off = mc == -CUDART_INF_F ? 0.f : p_base<E4M3>() - mc;
    const uint64_t c2 = ptx::pack2(c, c), off2 = ptx::pack2(off, off);
    uint64_t sum[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
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
        if (E4M3) {
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                uint32_t h0, h1, l0, l1;
                ptx::split_e4m3x2(s[k][4 * x], s[k][4 * x + 1], h0, l0);
                ptx::split_e4m3x2(s[k][4 * x + 2], s[k][4 * x + 3], h1, l1);
                u[x] = h0 | h1 << 16;
                u[8 + x] = l0 | l1 << 16;
            }
            ptx::tmem_st8(t_s + 8 * k, u);
            ptx::tmem_st8(t_s + 32 + 8 * k, u + 8);
        } else {
#pragma unroll
            for (int x = 0; x < 16; ++x) u[x] = ptx::cvt_bf16x2(s[k][2 * x], s[k][2 * x + 1]);
            ptx::tmem_st16(t_s + 16 * k, u);
        }
    }
    float a, b;
    ptx::unpack2(ptx::add2(ptx::add2(sum[0], sum[1]), ptx::add2(sum[2], sum[3])), a, b);
    l = l * f + (a + b);
    ptx::tmem_st_wait();
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(A_THREADS, 1)
    k_tree_attn(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_q1,
                const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const KvDims d,
                const AttnArgs a, const ATabs t) {
    using C = ACfg<D, E4M3>;
    extern __shared__ __align__(1024) uint8_t sm[];
    AMisc* const m = reinterpret_cast<AMisc*>(sm + 2 * C::QT + C::NS * C::SLOT + C::QMISC);
    uint8_t* const ring = sm + 2 * C::QT;
    float* const q_scale = reinterpret_cast<float*>(ring + C::NS * C::SLOT);   // e4m3: [2][128]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int pt = 2 * t.tpt;
    KT_MARK(K_TREE_ATTN, 0);
    if (ptx::smem_u32(sm) & 1023u) {   // the swizzled tiles need it
        if (tid == 0) latch_status(t.sb, MOE_ERR_CUDA, 0);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < C::NS; ++i) {
            ptx::mbar_init(&m->full[i], 1);
            ptx::mbar_init(&m->empty[i], 2);
            ptx::mbar_init(&m->san[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&m->q_full[i], E4M3 ? 8 : 1);
            ptx::mbar_init(&m->q_empty[i], 2);
            ptx::mbar_init(&m->drain[i], 1);
            ptx::mbar_init(&m->s_full[i], 1);
            ptx::mbar_init(&m->p_full[i], 4);
        }
        ptx::mbar_init(&m->o_full, 2);
        ptx::mbar_init(&m->o_free, 8);
        ptx::mbar_init(&m->ml_full, 8);
        ptx::mbar_init(&m->qs_full, 8);
        m->abort = 0;
        for (int i = 0; i < SAN_SLOTS; ++i) m->nan_seg[i] = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) ptx::tmem_alloc(&m->tmem, 512);
    if (warp == 0 && lane == 0) {
        ptx::prefetch_tensormap(&tm_k);
        ptx::prefetch_tensormap(&tm_v);
        if (!E4M3) ptx::prefetch_tensormap(&tm_q);
    }
    pdl_wait();
    KT_MARK(K_TREE_ATTN, 1);
    pdl_trigger();   // k_tree_join, which waits for this grid before it reads anything

    // this CTA's share: a scan of the requests' key tiles
    {
        const int per = (d.B + A_THREADS - 1) / A_THREADS;
        const int b0 = tid * per, b1 = b0 + per < d.B ? b0 + per : d.B;
        long long sum = 0;
        for (int b = b0; b < b1; ++b) {
            const KvReq r = kv_request(d, a.ctx_len, a.row_start, b);
            if (!r.ok && blockIdx.x == 0) latch_status(t.sb, MOE_ERR_BAD_LENGTHS, b);
            sum += request_tiles(d, r, pt);
        }
        long long s = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += u;
        }
        if (lane == 31) m->warp_sum[warp] = s;
        __syncthreads();
        long long total = 0, before = 0;
        for (int w = 0; w < A_THREADS / 32; ++w) {
            if (w == warp) before = total;
            total += m->warp_sum[w];
        }
        long long base = before + s - sum;
        const long long pos = share_begin(total, blockIdx.x);
        if (tid == 0) m->total = total;
        if (pos >= base && pos < base + sum) {
            for (int b = b0; b < b1; ++b) {
                const long long n = request_tiles(d, kv_request(d, a.ctx_len, a.row_start, b), pt);
                if (pos < base + n) {
                    m->first_b = b;
                    m->first_base = base;
                    break;
                }
                base += n;
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = m->tmem;
    volatile int* const abort_flag = &m->abort;
    auto fail = [&](int site) {
        latch_status(t.sb, MOE_ERR_TIMEOUT, 200 + site);
        *abort_flag = 1;
    };

    if (tid == 0) t.joint[blockIdx.x].rows = 0;
    if (warp < 4) {
    ptx::reg_dec<88>();
    Walk w;
    bool more = w.start(d, a, m, pt);
    if (warp == 0) {
        // ---- producer -----------------------------------------------------
        uint32_t seq = 0, nq = 0;
        const int nb = KT / t.box;
        const int bi = lane / C::HALVES, half = lane % C::HALVES;
        bool ok = true;
        for (; more && ok; more = w.next(d, a, pt)) {
            const int total = w.r.c + w.r.n, mt = w.k1 - w.k0;
            const int64_t table = (int64_t)w.b * d.max_pages;
            const uint64_t pol = w.np == 1 ? ptx::policy_evict_first() : ptx::policy_evict_last();
            // the page (and offset in it) of this lane's box of key tile j
            auto page = [&](int j, int& off) {
                const int key = (w.k0 + j) * KT + bi * t.box;
                if (j >= mt || bi >= nb || key >= total) return -1;
                const int pg = key / d.page;
                off = key - pg * d.page;
                return ld_dep(a.block_table + table + pg);
            };
            auto load = [&](const CUtensorMap* tm, int j, int pg, int off) {
                const uint32_t s = seq % C::NS;
                const int key = (w.k0 + j) * KT + bi * t.box;
                if (!ptx::mbar_wait_warp_fast(&m->empty[s], ((seq / C::NS) & 1) ^ 1, abort_flag, A_WAIT_NS)) return false;
                if (lane == 0) {
                    const int left = total - (w.k0 + j) * KT;
                    const int boxes = left >= KT ? nb : (left + t.box - 1) / t.box;
                    ptx::mbar_arrive_expect_tx(&m->full[s], boxes * t.box * C::ROWB);
                }
                __syncwarp();
                if (bi < nb && key < total) {
                    if (pg < 0 || pg >= d.n_pages) {
                        latch_status(t.sb, MOE_ERR_BAD_PAGE, pg);
                        pg = d.n_pages;   // outside: the copy fills zeros
                    }
                    ptx::tma_load_4d(ring + s * C::SLOT + half * (KT * C::SW) + bi * t.box * C::SW, tm,
                                     half * (C::SW / (E4M3 ? 1 : 2)), off, w.h, pg, &m->full[s], pol);
                }
                ++seq;
                return true;
            };
            if (!E4M3) {
                const int nt = w.ntok(pt) > t.tpt ? 2 : 1;
                for (int i = 0; i < nt && ok; ++i, ++nq) {
                    const uint32_t qb = nq & 1;
                    ok = ptx::mbar_wait_warp_fast(&m->q_empty[qb], ((nq >> 1) & 1) ^ 1, abort_flag, A_WAIT_NS);
                    const int ntok = w.ntok(pt) - i * t.tpt;
                    const bool small = ntok <= t.qbox;
                    if (ok && lane == 0) {
                        ptx::mbar_arrive_expect_tx(&m->q_full[qb],
                                                   (small ? t.qbox : t.tpt) * t.G * C::SW * C::HALVES);
                        const int row = w.r.r0 + w.tok0(pt) + i * t.tpt;
                        for (int hf = 0; hf < C::HALVES; ++hf)
                            ptx::tma_load_3d(sm + qb * C::QT + hf * (128 * C::SW), small ? &tm_q1 : &tm_q, hf * 64,
                                             w.h * t.G, row, &m->q_full[qb], ptx::policy_evict_last());
                    }
                    __syncwarp();
                }
            }
            int off0 = 0, off1 = 0, off2 = 0;
            int pg0 = page(0, off0), pg1 = page(1, off1);
            ok = ok && load(&tm_k, 0, pg0, off0);
            for (int j = 0; j < mt && ok; ++j) {
                const int pg2 = page(j + 2, off2);
                if (j + 1 < mt) ok = load(&tm_k, j + 1, pg1, off1);
                ok = ok && load(&tm_v, j, pg0, off0);
                pg0 = pg1;
                off0 = off1;
                pg1 = pg2;
                off1 = off2;
            }
            if (!ok) break;
        }
        if (!ok) {
            if (lane == 0) fail(1);
            // copies in flight land before the CTA's memory is given up
            const int none = 0;
            for (uint32_t i = seq > C::NS ? seq - C::NS : 0; i < seq; ++i)
                ptx::mbar_wait_warp_fast(&m->full[i % C::NS], (i / C::NS) & 1, &none, 10000000ull);
            for (uint32_t i = nq > 2 ? nq - 2 : 0; i < nq && !E4M3; ++i)
                ptx::mbar_wait_warp_fast(&m->q_full[i & 1], (i >> 1) & 1, &none, 10000000ull);
        }
    } else if (warp == 1 || warp == 3) {
        // ---- MMA issuers: warp 1 for stream 0, warp 3 for stream 1 ---------
        // The whole warp walks and waits, one lane issues: descriptors built
        // from values that are the same in the whole warp stay in uniform
        // registers, and a product costs a few instructions.  An issuer waits
        // for, and releases, every tile of the ring, also those that only the
        // other stream uses, so that neither can be two phases ahead of or
        // behind a barrier (a parity wait takes two phases for none).
        constexpr uint32_t id_s = ptx::idesc_attn(E4M3, 128, KT, false);
        constexpr uint32_t id_o = ptx::idesc_attn(E4M3, 128, D, true);
        const int s = warp >> 1;
        uint32_t base = 0, nq = 0, n_p = 0, n_seg = 0, san_phase = 0;   // san_phase: a bit a ring slot
        bool ok = true;
        const uint32_t sm0 = ptx::smem_u32(sm), ring0 = ptx::smem_u32(ring);
        const uint32_t t_s = tmem + C::T_S + s * 128, t_o = tmem + C::T_O + s * 128;
        auto same = [](uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); };
        // Waits come before the one for P, which ends a tile's critical path:
        // after it the products go out one after the other.
        for (; more && ok; more = w.next(d, a, pt), ++n_seg) {
            const int mt = w.k1 - w.k0;
            const bool two = same(w.ntok(pt) > t.tpt);
            bool first = true;
            const uint32_t qb = same((nq + (two ? s : 0)) & 1);
            const uint32_t qd = ptx::smem_desc_lo(sm0 + qb * C::QT, 16);
            ok = ptx::mbar_wait_warp_fast(&m->q_full[qb], ((nq + (two ? s : 0)) >> 1) & 1, abort_flag, A_WAIT_NS);
            // the previous segment's O is read before the first product into it
            auto k_ready = [&](int j, uint32_t& slot) {
                const uint32_t q = base + seq_k(j);
                slot = same(q % C::NS);
                return ptx::mbar_wait_warp_fast(&m->full[slot], (q / C::NS) & 1, abort_flag, A_WAIT_NS);
            };
            auto v_ready = [&](int j, uint32_t& slot) {   // landed and clean
                slot = same((base + seq_v(j, mt)) % C::NS);
                const bool r =
                    ptx::mbar_wait_warp_fast(&m->san[slot], (san_phase >> slot) & 1, abort_flag, A_WAIT_NS);
                san_phase ^= 1u << slot;
                return r;
            };
            // (one lane) S = Q K^T, and the slot's release
            auto qk = [&](uint32_t slot, bool mine) {
                if (mine) {
                    const uint32_t kd = ptx::smem_desc_lo(ring0 + slot * C::SLOT, 16);
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
                }
                ptx::mma_commit(&m->empty[slot]);
            };
            // two query tiles: both streams take K0 V0 K1 V1 ...; one: stream j % 2
            // takes tile j, in the order K0 K1 V0 K2 V1 ...
            const int ahead = two ? 1 : 2;
            uint32_t ks = 0, vs = 0;
            for (int j = 0; j < ahead && j < mt && ok; ++j) {
                ok = k_ready(j, ks);
                ptx::tc_fence_after();
                const bool mine = same(two || (j & 1) == s);
                if (ok && ptx::elect_one()) qk(ks, mine);
                __syncwarp();
            }
            if (ok && n_seg > 0) ok = ptx::mbar_wait_warp_fast(&m->o_free, (n_seg - 1) & 1, abort_flag, A_WAIT_NS);
            for (int j = 0; j < mt && ok; ++j) {
                const bool mine = same(two || (j & 1) == s);
                const bool nx = same(j + ahead < mt);
                ok = v_ready(j, vs) && (!nx || k_ready(j + ahead, ks));
                const uint32_t vd = ptx::smem_desc_lo(ring0 + vs * C::SLOT, KT * C::SW);
                const uint32_t add = same(!first);
                if (mine && ok) {
                    ok = ptx::mbar_wait_warp_fast(&m->p_full[s], n_p & 1, abort_flag, A_WAIT_NS);
                    ++n_p;
                    first = false;
                }
                if (!ok) break;
                ptx::tc_fence_after();
                if (ptx::elect_one()) {
                    if (mine) {   // O += P V
#pragma unroll
                        for (int part = 0; part < (E4M3 ? 2 : 1); ++part) {
#pragma unroll
                            for (int e = 0; e < KT / C::KSTEP; ++e)
                                ptx::mma_ts<E4M3>(t_o, t_s + part * 32 + e * 8,
                                                  ptx::smem_desc<C::SW>(vd + (e * C::KSTEP * C::SW >> 4)), id_o,
                                                  (part | e) ? 1u : add);
                        }
                    }
                    ptx::mma_commit(&m->empty[vs]);
                    if (nx) qk(ks, mine);
                }
                __syncwarp();
            }
            if (!ok) break;
            if (ptx::elect_one()) {
                ptx::mma_commit(&m->o_full);
                // (every product of this stream is issued, those that read Q among them)
                ptx::mma_commit(&m->q_empty[nq & 1]);
                if (two) ptx::mma_commit(&m->q_empty[(nq + 1) & 1]);
            }
            __syncwarp();
            nq += two ? 2 : 1;
            base += 2 * mt;
        }
        if (!ok) {
            if (lane == 0) fail(2);
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
        // Every V tile passes through this warp (it waits for every load in ring
        // order, the MMA issuer waits for it): a warp that looked only at the tiles
        // it cleans could be two phases ahead of or behind their barriers, which a
        // parity wait takes for complete, or waits on for ever.
        uint32_t base = 0, seen = 0;
        int seg = 0;
        bool ok = true;
        for (; more && ok; more = w.next(d, a, pt), ++seg) {
            const int mt = w.k1 - w.k0, total = w.r.c + w.r.n, see = w.all_see(d, pt);
            for (int j = 0; j < mt; ++j) {
                const int key0 = (w.k0 + j) * KT;
                const uint32_t q = base + seq_v(j, mt), slot = q % C::NS;
                for (; seen <= q && ok; ++seen)
                    ok = ptx::mbar_wait_warp_fast(&m->full[seen % C::NS], (seen / C::NS) & 1, abort_flag, A_WAIT_NS);
                if (!ok) {
                    if (lane == 0) fail(3);
                    break;
                }
                if (key0 + KT <= see) {
                    if (lane == 0) ptx::mbar_arrive(&m->san[slot]);
                    continue;
                }
                const int r0 = see > key0 ? see - key0 : 0, r1 = total - key0 < KT ? total - key0 : KT;
                uint32_t bad = 0;
                for (int hf = 0; hf < C::HALVES; ++hf) {
                    uint8_t* const v = ring + slot * C::SLOT + hf * (KT * C::SW);
                    for (int o = r1 * C::SW + lane * 16; o < KT * C::SW; o += 512)
                        *reinterpret_cast<uint4*>(v + o) = make_uint4(0, 0, 0, 0);
                    for (int o = r0 * C::SW + lane * 16; o < r1 * C::SW; o += 512) {
                        uint4 x = *reinterpret_cast<uint4*>(v + o);
                        uint32_t* const u = reinterpret_cast<uint32_t*>(&x);
                        uint32_t hit = 0;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t z;   // all ones in the elements that are not finite
                            if (E4M3) {
                                z = __vcmpeq4(u[i] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                            } else {
                                z = __vcmpeq2(u[i] & 0x7F807F80u, 0x7F807F80u);
                            }
                            u[i] &= ~z;
                            hit |= z;
                        }
                        if (hit) *reinterpret_cast<uint4*>(v + o) = x;
                        bad |= hit;
                    }
                }
                ptx::fence_proxy_async_shared();
                bad = __any_sync(0xffffffffu, bad != 0);
                if (lane == 0) {
                    if (bad) *(volatile int*)&m->nan_seg[seg % SAN_SLOTS] = seg + 1;
                    ptx::mbar_arrive(&m->san[slot]);
                }
                __syncwarp();
            }
            base += 2 * mt;
        }
    }
    } else {
        ptx::reg_inc<208>();
        Walk w;
        bool more = w.start(d, a, m, pt);
        // ---- softmax: warpgroup g, thread = row ---------------------------
        const int g = (warp - 4) >> 2, wq = warp & 3, row = 32 * wq + lane;
        const uint32_t lanes = (uint32_t)(32 * wq) << 16;
        const uint32_t t_s = tmem + lanes + C::T_S + g * 128;
        uint32_t n_s = 0, nq = 0, n_seg = 0, n_ml = 0;
        bool ok = true;
        for (; more && ok; more = w.next(d, a, pt), ++n_seg) {
            const int mt = w.k1 - w.k0, total = w.r.c + w.r.n, see = w.all_see(d, pt);
            const bool two = w.ntok(pt) > t.tpt;
            const int qs = two ? g : 0;                                  // this stream's query tile
            const int ntok = w.ntok(pt) - qs * t.tpt < t.tpt ? w.ntok(pt) - qs * t.tpt : t.tpt;
            const int rows = ntok * t.G;
            const bool live = 32 * wq < rows;                            // a warp without rows only keeps step
            const int tok = w.tok0(pt) + qs * t.tpt + row / t.G;         // token of the request (row < rows)
            const int cnt = two ? mt : (g == 0 ? (mt + 1) / 2 : mt / 2);
            float c = d.scale * 1.4426950408889634f;
            if (E4M3) {
                // the query tile as e4m3 rows hi and lo (leading and next 4
                // significant bits) under one power of two a row, into the
                // swizzled K-major layout: 16 (8) lanes a row, 8 elements a lane
                c *= ld_dep(a.k_scale + w.h);
                constexpr int LPR = D / 8, RPW = 32 / LPR;
                const uint32_t qb = (nq + qs) & 1;
                uint8_t* const hi = sm + qb * C::QT;
                const int nw = two ? 4 : 8, wi = two ? wq : warp - 4;    // warps that share the tile
                const int sub = lane % LPR;
                for (int r = wi * RPW + lane / LPR; r < (rows + RPW - 1) / RPW * RPW; r += nw * RPW) {
                    const int tk = w.tok0(pt) + qs * t.tpt + r / t.G, hh = w.h * t.G + r % t.G;
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (r < rows)
                        x = ld_dep(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.q) +
                                                                  (int64_t)(w.r.r0 + tk) * d.q_stride +
                                                                  (int64_t)hh * D) + sub);
                    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
                    float f[8], top = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        f[2 * i] = __uint_as_float(u[i] << 16);
                        f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
                        top = fmaxf(top, fmaxf(fabsf(f[2 * i]), fabsf(f[2 * i + 1])));
                    }
#pragma unroll
                    for (int o = LPR / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    // 2^(134 - e) brings the row's maximum (exponent field e) to [128, 256)
                    int e = (int)(__float_as_uint(top) >> 23);
                    // (a row below 2^-87 is as good as 0; one with an infinity has NaN scores)
                    const bool inf = e == 255;
                    e = e < 40 ? 40 : (e > 250 ? 250 : e);
                    const float up = __uint_as_float((uint32_t)(261 - e) << 23);
                    if (sub == 0) q_scale[qb * 128 + r] = inf ? CUDART_NAN_F : __uint_as_float((uint32_t)(e - 7) << 23);
                    uint32_t vh[2], vl[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
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
                    const uint32_t chunk = (uint32_t)(sub >> 1) ^ (C::SW == 128 ? (r & 7) : ((r >> 1) & 3));
                    uint8_t* const to = hi + r * C::SW + chunk * 16 + (sub & 1) * 8;
                    *reinterpret_cast<uint2*>(to) = make_uint2(vh[0], vh[1]);
                    *reinterpret_cast<uint2*>(to + C::QT / 2) = make_uint2(vl[0], vl[1]);
                }
                ptx::fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_n(&m->q_full[qb], two ? 2 : 1);
                if (lane == 0) ptx::mbar_arrive(&m->qs_full);
                if (!ptx::mbar_wait_warp_fast(&m->qs_full, n_seg & 1, abort_flag, A_WAIT_NS)) {   // the row scales are there
                    if (lane == 0) fail(6);
                    break;
                }
                c *= q_scale[qb * 128 + row];
            }
            float mc = -CUDART_INF_F, l = 0.f;
            for (int i = 0; i < cnt && ok; ++i) {
                const int key0 = (w.k0 + (two ? i : 2 * i + g)) * KT;
                const bool part = key0 + KT > see;
                uint32_t vis[4] = {~0u, ~0u, ~0u, ~0u};
                if (part && live) {
                    if (d.W == 0) {
                        const int n = w.r.c + tok + 1 - key0;            // keys of the tile the row sees
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            vis[k] = n >= 32 * k + 32 ? ~0u : (n <= 32 * k ? 0u : (1u << (n - 32 * k)) - 1u);
                    } else {
                        // bit x of the tile is new token key0 + x - c
                        uint32_t words[5];
                        const int j0 = key0 - w.r.c, word0 = j0 >> 5;
                        const uint32_t* const mr = a.mask + (int64_t)(w.r.r0 + tok) * d.W;
#pragma unroll
                        for (int k = 0; k < 5; ++k) {
                            const int x = word0 + k, n = w.r.n - 32 * x;
                            uint32_t v = x < 0 ? ~0u : 0u;
                            if (x >= 0 && n > 0 && row < rows) {
                                v = ld_dep(mr + x);
                                if (n < 32) v &= (1u << n) - 1u;
                            }
                            words[k] = v;
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) vis[k] = __funnelshift_r(words[k], words[k + 1], j0 & 31);
                    }
                }
                if (!ptx::mbar_wait_warp_fast(&m->s_full[g], n_s & 1, abort_flag, A_WAIT_NS)) {
                    if (lane == 0) fail(4);
                    ok = false;
                    break;
                }
                ++n_s;
                ptx::tc_fence_after();
                if (live)
                    softmax_tile<D, E4M3>(t_s, tmem + lanes + C::T_O + g * 128, c, part, vis, i > 0, mc, l);
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&m->p_full[g]);
            }
            if (!ok) break;
            nq += two ? 2 : 1;
            if (!ptx::mbar_wait_warp_fast(&m->o_full, n_seg & 1, abort_flag, A_WAIT_NS)) {
                if (lane == 0) fail(5);
                break;
            }
            ptx::tc_fence_after();
            // ---- the segment's end ------------------------------------------
            // one query tile: both streams' O of a row, half its columns a warpgroup
            float m1 = -CUDART_INF_F, l1 = 0.f;
            if (!two) {
                m->ml[g][row] = make_float2(mc, l);
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&m->ml_full);
                if (!ptx::mbar_wait_warp_fast(&m->ml_full, n_ml & 1, abort_flag, A_WAIT_NS)) {
                    if (lane == 0) fail(7);
                    break;
                }
                ++n_ml;
                const float2 o = m->ml[g ^ 1][row];
                m1 = o.x;
                l1 = o.y;
            }
            const float top = fmaxf(mc, m1), zero = top == -CUDART_INF_F ? 0.f : top;
            // a stream that saw nothing adds nothing (its O may never have been written)
            const float f0 = mc == -CUDART_INF_F && !(l != l) ? 0.f : ptx::ex2(mc - zero);
            const float f1 = m1 == -CUDART_INF_F && !(l1 != l1) ? 0.f : ptx::ex2(m1 - zero);
            const float sum = l * f0 + l1 * f1;
            const bool whole = w.k0 == 0 && w.k1 == w.kt;
            const bool mine = row < rows;
            const int grow = w.r.r0 + tok;                               // row of the batch
            const int head = w.h * t.G + row % t.G;
            const int slot = 2 * blockIdx.x + (w.k0 == 0 ? 1 : 0);
            const int prow = qs * t.tpt * t.G + row;                     // row of the partial result
            const bool flagged = *(volatile int*)&m->nan_seg[n_seg % SAN_SLOTS] == (int)n_seg + 1;
            if (live) {
                const int x0 = two ? 0 : g * (D / 2), x1 = two ? D : x0 + D / 2;
                const float scale = whole ? (sum == 0.f ? 0.f : 1.f / sum) * (E4M3 ? ld_dep(a.v_scale + w.h) : 1.f) : 1.f;
                const bool have0 = f0 != 0.f, have1 = f1 != 0.f;
                for (int x = x0; x < x1; x += 16) {
                    uint32_t u[16], v[16];
                    ptx::tmem_ld16(tmem + lanes + C::T_O + g * 128 + x, u);
                    if (!two) ptx::tmem_ld16(tmem + lanes + C::T_O + (g ^ 1) * 128 + x, v);
                    ptx::tmem_ld_wait16(u);
                    if (!two) ptx::tmem_ld_wait16(v);
                    float o[16];
#pragma unroll
                    for (int y = 0; y < 16; ++y) {
                        o[y] = have0 ? __uint_as_float(u[y]) * f0 : 0.f;
                        if (!two) o[y] += have1 ? __uint_as_float(v[y]) * f1 : 0.f;
                        o[y] *= scale;
                    }
                    if (flagged && mine) {
                        const int kb = see > w.k0 * KT ? see : w.k0 * KT, ke = total < w.k1 * KT ? total : w.k1 * KT;
                        for (int key = kb; key < ke; ++key) {
                            const int j = key - w.r.c;
                            if (j >= 0 && !row_sees(d, a, grow, tok, j)) continue;
                            const int pg = ld_dep(a.block_table + (int64_t)w.b * d.max_pages + key / d.page);
                            if (pg < 0 || pg >= d.n_pages) continue;
                            const int64_t at = pg * d.page_stride + w.h * d.head_stride +
                                               (key % d.page) * d.token_stride + x;
#pragma unroll
                            for (int y = 0; y < 16; ++y) {
                                float e;
                                if (E4M3) {
                                    const uint8_t q8 = reinterpret_cast<const uint8_t*>(a.v_cache)[at + y];
                                    e = (q8 & 0x7F) == 0x7F ? CUDART_NAN_F : 0.f;
                                } else {
                                    e = __uint_as_float(
                                        (uint32_t) reinterpret_cast<const uint16_t*>(a.v_cache)[at + y] << 16);
                                }
                                if (!isfinite(e)) o[y] += e;
                            }
                        }
                    }
                    if (mine && whole) {
                        uint32_t z[8];
#pragma unroll
                        for (int y = 0; y < 8; ++y) z[y] = ptx::cvt_bf16x2(o[2 * y], o[2 * y + 1]);
                        uint4* const to = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.out) +
                                                                   ((int64_t)grow * d.Hq + head) * D + x);
                        to[0] = make_uint4(z[0], z[1], z[2], z[3]);
                        to[1] = make_uint4(z[4], z[5], z[6], z[7]);
                    } else if (mine) {
                        float4* const to = reinterpret_cast<float4*>(t.part_o + ((int64_t)slot * t.rp + prow) * D + x);
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            to[y] = make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
                    }
                }
                if (mine && (two || g == 0)) {
                    // log2 of the sum, without the weights' 2^BASE
                    if (!whole)
                        t.part_ml[(int64_t)slot * t.rp + prow] = make_float2(top - p_base<E4M3>(), sum);
                    else if (a.lse)
                        a.lse[(int64_t)grow * d.Hq + head] =
                            sum == 0.f ? -CUDART_INF_F : (zero - p_base<E4M3>() + log2f(sum)) * 0.69314718055994531f;
                }
            }
            if (warp == 4 && lane == 0 && w.k0 == 0 && !whole) {
                Joint jn;
                jn.rows = w.ntok(pt) * t.G;
                jn.row0 = w.r.r0 + w.tok0(pt);
                jn.kvh = w.h;
                // the CTA that holds the segment's last tile
                jn.last = (int)(((w.pos + w.kt) * A_CTAS - 1) / m->total);
                jn.total = m->total;
                jn.pad[0] = jn.pad[1] = 0;
                t.joint[blockIdx.x] = jn;
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&m->o_free);
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_dealloc(tmem, 512);
    KT_MARK(K_TREE_ATTN, 2);
}

// The parts of the divided segments: CTA x of the first grid axis joins the
// segment whose first tile share x holds, a warp a row, parts in key order.
constexpr int JOIN_WARPS = 8;

template <int D>
__global__ void __launch_bounds__(32 * JOIN_WARPS) k_tree_join(const KvDims d, const AttnArgs a, const ATabs t) {
    constexpr int V = D / 32;
    const int lane = threadIdx.x & 31, row = blockIdx.y * JOIN_WARPS + (threadIdx.x >> 5), cta = blockIdx.x;
    KT_MARK(K_TREE_JOIN, 0);
    pdl_wait();
    KT_MARK(K_TREE_JOIN, 1);
    const Joint* const jp = t.joint + cta;
    if (row >= ld_dep(&jp->rows)) return;
    const int last = ld_dep(&jp->last);
    const long long total = ld_dep(&jp->total);
    // part slots: 2 cta + 1 (the first), then 2 c of the CTAs that hold any tile
    float top = -CUDART_INF_F;
    for (int c = cta + lane; c <= last; c += 32) {
        if (c > cta && share_begin(total, c) == share_begin(total, c + 1)) continue;
        top = fmaxf(top, ld_dep(t.part_ml + (int64_t)(2 * c + (c == cta)) * t.rp + row).x);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float zero = top == -CUDART_INF_F ? 0.f : top;
    float sum = 0.f, o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = 0.f;
#pragma unroll 4
    for (int c = cta; c <= last; ++c) {
        if (c > cta && share_begin(total, c) == share_begin(total, c + 1)) continue;
        const int64_t at = (int64_t)(2 * c + (c == cta)) * t.rp + row;
        const float2 ml = ld_dep(t.part_ml + at);
        float p[V];
        if (V == 4) {
            const float4 x = ld_dep(reinterpret_cast<const float4*>(t.part_o + at * D) + lane);
            p[0] = x.x; p[1] = x.y; p[2 % V] = x.z; p[3 % V] = x.w;
        } else {
            const float2 x = ld_dep(reinterpret_cast<const float2*>(t.part_o + at * D) + lane);
            p[0] = x.x; p[1] = x.y;
        }
        const float f = ml.y == 0.f ? 0.f : ptx::ex2(ml.x - zero);
        sum += ml.y * f;
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] += p[v] * f;
    }
    const int G = t.G, kvh = ld_dep(&jp->kvh), grow = ld_dep(&jp->row0) + row / G, head = kvh * G + row % G;
    const float s = (sum == 0.f ? 0.f : 1.f / sum) * (d.e4m3 ? ld_dep(a.v_scale + kvh) : 1.f);
    uint32_t* const to = reinterpret_cast<uint32_t*>(reinterpret_cast<__nv_bfloat16*>(a.out) +
                                                     ((int64_t)grow * d.Hq + head) * D) + lane * (V / 2);
#pragma unroll
    for (int v = 0; v < V; v += 2) to[v / 2] = ptx::cvt_bf16x2(o[v] * s, o[v + 1] * s);
    if (a.lse && lane == 0)
        a.lse[(int64_t)grow * d.Hq + head] =
            sum == 0.f ? -CUDART_INF_F : (zero + log2f(sum)) * 0.69314718055994531f;
    KT_MARK(K_TREE_JOIN, 2);
}

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

ATabs attn_tabs(const KvDims& d, char* ws, size_t* bytes) {
    ATabs t{};
    t.G = d.Hq / d.Hkv;
    t.tpt = 128 / t.G;
    t.box = gcd(d.page, KT);
    t.qbox = t.tpt < 8 ? t.tpt : 8;
    const int64_t tokens = d.T < 2 * t.tpt ? d.T : 2 * t.tpt;
    t.rp = (int)(tokens * t.G);
    size_t o = sizeof(StatusBlock);
    auto take = [&](size_t n) { const size_t at = o; o = (o + n + 255) & ~(size_t)255; return at; };
    const size_t joint = take(A_CTAS * sizeof(Joint));
    const size_t ml = take((size_t)2 * A_CTAS * t.rp * sizeof(float2));
    const size_t po = take((size_t)2 * A_CTAS * t.rp * d.D * sizeof(float));
    if (bytes) *bytes = o;
    t.joint = reinterpret_cast<Joint*>(ws + joint);
    t.part_ml = reinterpret_cast<float2*>(ws + ml);
    t.part_o = reinterpret_cast<float*>(ws + po);
    t.sb = reinterpret_cast<StatusBlock*>(ws);
    return t;
}

template <int D, bool E4M3>
cudaError_t launch_attn(const KvDims& d, const AttnArgs& a, cudaStream_t st) {
    using C = ACfg<D, E4M3>;
    const ATabs t = attn_tabs(d, a.ws, nullptr);
    CUtensorMap tm_q, tm_q1, tm_k, tm_v;
    const uint64_t el = E4M3 ? 1 : 2;
    const CUtensorMapDataType dt = E4M3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUtensorMapSwizzle sw = C::SW == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)d.page, (uint64_t)d.Hkv, (uint64_t)d.n_pages};
    const uint64_t str[3] = {d.token_stride * el, d.head_stride * el, d.page_stride * el};
    const uint32_t box[4] = {(uint32_t)(C::SW / el), (uint32_t)t.box, 1, 1};
    if (!make_map(&tm_k, dt, a.k_cache, 4, dims, str, box, sw) || !make_map(&tm_v, dt, a.v_cache, 4, dims, str, box, sw))
        return cudaErrorInvalidValue;
    tm_q = tm_q1 = tm_k;
    if (!E4M3) {
        const uint64_t qd[3] = {(uint64_t)D, (uint64_t)d.Hq, (uint64_t)d.T};
        const uint64_t qs[2] = {(uint64_t)D * 2, (uint64_t)d.q_stride * 2};
        const uint32_t qb[3] = {64, (uint32_t)t.G, (uint32_t)t.tpt}, qb1[3] = {64, (uint32_t)t.G, (uint32_t)t.qbox};
        if (!make_map(&tm_q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, 3, qd, qs, qb, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !make_map(&tm_q1, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, 3, qd, qs, qb1, CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    }
    cudaError_t e = cudaFuncSetAttribute(k_tree_attn<D, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    timing_begin(K_TREE_ATTN, st);
    e = launch_pdl(k_tree_attn<D, E4M3>, dim3(A_CTAS), dim3(A_THREADS), C::SMEM, st, tm_q, tm_q1, tm_k, tm_v, d, a, t);
    timing_end(st);
    if (e != cudaSuccess) return e;
    timing_begin(K_TREE_JOIN, st);
    e = launch_pdl(k_tree_join<D>, dim3(A_CTAS, (t.rp + JOIN_WARPS - 1) / JOIN_WARPS), dim3(32 * JOIN_WARPS), 0, st, d, a,
                   t);
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

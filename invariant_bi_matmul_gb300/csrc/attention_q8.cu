// attention_q8.cu -- decode / verify / prefill attention over the 8-bit paged KV cache
// (kv_q8.cu has its format), causal, for blocks of any width.
//
// Mathematics.  With the codes a_i, b_i of key i, its scales 2^x_i (K) and 2^y_i (V), and a
// query row q:
//   t_i = scale * log2(e) * 2^x_i * (q . a_i) + y_i,   p_i = 2^(t_i - m),
//   sum_i p_i b_i  and  l = sum_i p_i 2^-y_i,   out = sum p b / l
// -- the V scale rides in the exponent, so the tensor cores see codes only, and the row sum
// takes it out again (2^-y is exact).  m is a reference maximum of the t_i seen so far.
//
// Both products run on the codes as they lie in the cache (tcgen05 kind::f8f6f4, e4m3 x e4m3,
// fp32 accumulators).  The other operand is split into two e4m3 pieces, so nothing of its
// precision is lost to 8 bits:
//   * q * 2^s (s puts the row's largest value in [128, 256)) = hi + lo, each rounded to
//     nearest: exact for bf16 q down to 2^-9 of the row's largest value, off by at most
//     2^-18 of it below;
//   * p = hi + lo / 32: p <= 2^8; hi has four bits, lo the next four, so p is held to
//     2^-9 of itself (bf16 would hold 2^-8) or to 2^-15 absolute, whichever is more; the
//     largest p of a row is 2^3 at least.
//
// Reduction of one (query, head) -- a function of its position alone, as in attention.cu:
// chunks of 512 keys from key 0; a chunk in tiles of 128 keys, ascending; per tile the exact
// maximum of the row's t, m raised to (maximum - 3) only when the maximum exceeds m + 8 (O and
// the sums then scaled by 2^(m_old - m_new)); each of 128 threads sums its key of every tile,
// and the 128 sums are added by a fixed tree; the chunk partials (m, l, o) go through the
// merge of attention.cu.  A tile that a row does not see changes none of its numbers, and a
// row's place in the MMA tile, the other rows and the block's width enter nowhere.
//
// Orientation.  S^T = K Q^T (M = 128 keys, N = 32 query rows) and O^T = V^T P^T (M = head
// dim, N = 32 hi + 32 lo rows): the cache is the operand that the tensor core reads 128 rows
// at a time, whatever the number of query rows, and a softmax thread owns one key, so it does
// as many exponentials as there are query rows (rounded up to 8, 16 or 32), reads its key's
// two scale bytes once, and writes its P values as 16-byte pieces.
//
// Warps: one or two softmax groups of four (one key of the tile per thread; two groups share
// the query rows), four epilogue warps (they also split the next item's Q), the TMA producer
// (it also finds the work items and publishes them), the S issuer (and TMEM owner), the P V
// issuer.  One persistent CTA per SM; work items (sequence, chunk, query tile, KV head) are
// enumerated on the device.  All waits are bounded; the one barrier that warps meet in, a
// softmax group's, is left by all of them together.
//
// Bound by memory: 2 * (D + 1) bytes per key and KV head against 4 * 32 * D operations.
#include "attn_common.cuh"

#include <cuda_fp8.h>

namespace bi {
namespace {

constexpr int QR = 32;                    // query rows of a tile
constexpr int TK = 128;                   // keys of a tile: two pages
constexpr int TPAGES = TK / PAGE;
constexpr int NQ = 4;                     // warps of a softmax group: 32 keys each
constexpr int NDESC = 16;                 // item descriptors in flight
constexpr int NSB = 4;                    // S buffers in tensor memory
constexpr int TMEM_COLS = 256;
constexpr int S_COL = 0;                  // S buffers: 32 columns each
constexpr int O_COL = NSB * QR;           // O buffers (by item): 32 hi + 32 lo columns each
constexpr float kNoMax = -1e30f;          // m before any visible key: every finite t exceeds it
// A raised m leaves p = 2^3 at the maximum and holds until p would exceed 2^8 (the second
// piece of such a p is at most 8: 8 * kLoScale fits e4m3's 448).  More headroom means fewer
// raises, which cost an exchange between the group's warps and a rescale of O; less, a finer
// floor of the small weights (2^-15 absolute against the maximum).
constexpr float kHeadroom = 3.f;
constexpr float kRaise = 8.f;
constexpr float kLoScale = 32.f;          // the second piece of p is held times this
constexpr int MAX_BATCH = BI_ATTN_MAX_BATCH;

static_assert(CHUNK % TK == 0 && TK == NQ * 32, "a thread per key");
static_assert(O_COL + 2 * 2 * QR <= TMEM_COLS, "tensor memory columns");

template <int D>
struct Cfg {
    static constexpr int NST = D == 64 ? 8 : 5;          // tile stages in the ring
    static constexpr int PAGE_BYTES = PAGE * D;
    static constexpr int SIDE_BYTES = TK * D;            // K or V of a tile
    static constexpr int STAGE_BYTES = 2 * SIDE_BYTES;
    static constexpr int Q_PIECE = QR * D;               // hi or lo of a Q tile
    static constexpr int Q_BYTES = 2 * Q_PIECE;
    static constexpr int P_BYTES = TK * 2 * QR;          // [key][32 hi | 32 lo]
    static constexpr int Q_OFF = 0;                      // two Q buffers
    static constexpr int P_OFF = Q_OFF + 2 * Q_BYTES;    // two P buffers
    static constexpr int RING_OFF = P_OFF + 2 * P_BYTES;
    static constexpr int SCALE_OFF = RING_OFF + NST * STAGE_BYTES;  // [NST][K 128 | V 128]
    static constexpr int BAR_OFF = SCALE_OFF + NST * 2 * TK;
    static constexpr int NBARS = 2 * NST + 2 * NSB + 4 + 4 + 2 + 2 + NDESC + 2;
    static constexpr int DESC_OFF = (BAR_OFF + NBARS * 8 + 8 + 15) / 16 * 16;
    static constexpr int XS_OFF = DESC_OFF + NDESC * 32;
    // per item buffer: four warps' row sums and the row maxima; per Q buffer the row factors;
    // the maxima exchanged within the softmax groups
    static constexpr int XS_FLOATS = 2 * (NQ + 1) * QR + 2 * QR + NQ * QR;
    static constexpr int MISC_OFF = XS_OFF + XS_FLOATS * 4;
    static constexpr int MISC_INTS = NST + (MAX_BATCH + 1) + 4 + 1;
    static constexpr size_t SMEM = 1024 + size_t(MISC_OFF) + MISC_INTS * 4;
    // K-major and MN-major rows of D bytes: the 128- or 64-byte swizzle, groups of 8 rows
    static constexpr uint32_t LAYOUT = D == 128 ? 2 : 4;
    static constexpr uint32_t SBO = 8 * D;
    static_assert(P_OFF % 1024 == 0 && RING_OFF % 1024 == 0 && STAGE_BYTES % 1024 == 0, "");
    static_assert(SMEM <= 232448, "shared memory per CTA");
};

// byte offset of 16-byte piece `ch` of row `row` in a tile of D-byte rows (the TMA patterns
// SWIZZLE_128B and SWIZZLE_64B)
template <int ROW>
__device__ __forceinline__ uint32_t swz_row(int row, int ch) {
    return ROW == 128 ? uint32_t(row) * 128u + uint32_t((ch ^ (row & 7)) << 4)
                      : uint32_t(row) * 64u + uint32_t((ch ^ ((row >> 1) & 3)) << 4);
}

// D[tmem] (+)= A[smem desc] * B[smem desc], 8-bit floats (e4m3 here), 32 of K per instruction
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor for kind::f8f6f4, e4m3 operands, fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n, int a_mn, int b_mn) {
    return (1u << 4) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) |
           (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}

// Untiled bulk copy global -> shared (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
        ::"r"(smem_addr(dst)), "l"(src), "r"(bytes), "r"(smem_addr(bar))
        : "memory");
}

// RP consecutive columns of this warp's 32 lanes, with the wait.
__device__ __forceinline__ void tmem_cols(uint32_t ta, uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(ta)
        : "memory");
}
__device__ __forceinline__ void tmem_store_x8(uint32_t ta, const uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(ta),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
        : "memory");
}
__device__ __forceinline__ void tmem_cols(uint32_t ta, uint32_t (&r)[16]) {
    tmem_load_32x32b_x16_sync(ta, r);
}
__device__ __forceinline__ void tmem_cols(uint32_t ta, uint32_t (&r)[32]) {
    tmem_load_32x32b_x32_sync(ta, r);
}

// Combines v[r] over the 32 lanes for each of N rows (max, or a sum over a fixed tree: lanes
// that differ in bit 4, then bit 3, .. bit 0 -- the same for every N).  Every lane gets row
// lane * N / 32: at each step a lane keeps one half of its rows while it has several.
template <int N, bool MAX, int OFF = 16>
__device__ __forceinline__ float combine_lanes(const float (&v)[N], int lane) {
    auto op = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
    if constexpr (OFF == 0) {
        return v[0];
    } else if constexpr (N == 1) {
        const float w[1] = {op(v[0], __shfl_xor_sync(0xffffffffu, v[0], OFF))};
        return combine_lanes<1, MAX, OFF / 2>(w, lane);
    } else {
        const bool up = (lane & OFF) != 0;
        float w[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float got = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + N / 2], OFF);
            w[i] = op(up ? v[i + N / 2] : v[i], got);
        }
        return combine_lanes<N / 2, MAX, OFF / 2>(w, lane);
    }
}

// Two e4m3 codes of (a, b), a in the low byte; and the values they stand for.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 e4m3x2_values(uint32_t c) {
    return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(c), __NV_E4M3)));
}

// 2^(s - 127) of an E8M0 byte (255: NaN), and its inverse (255: 1, its row is NaN anyway).
__device__ __forceinline__ float e8m0(uint32_t s) {
    return __uint_as_float(s == 0 ? 0x00400000u : s == 255 ? 0x7fc00000u : s << 23);
}
__device__ __forceinline__ float e8m0_inv(uint32_t s) {
    return s == 255 ? 1.f : e8m0(254 - s);
}

// True in every thread of a softmax group (named barrier `id`, 128 threads) when `v` is true
// in one of them.  The group's warps leave their loop only on a common decision taken here,
// so none is left waiting: a warp whose bounded wait ran out runs on (its later waits return
// at once) to the next such point.
__device__ __forceinline__ bool group_or(int id, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(v ? 1u : 0u), "r"(id)
        : "memory");
    return r != 0;
}

// A work item as the producer publishes it: chunk c of the keys for one query tile of
// sequence b, KV head h.
struct alignas(16) Item {
    int npages;  // pages of the chunk that the tile's last token sees (0: no more items)
    int key0;    // first key of the chunk
    int L;       // the sequence's length
    int pos0;    // position of the tile's first token
    int t0;      // its row in q and out
    int ntok;    // the tile's tokens
    int h;
    int b;
};
static_assert(sizeof(Item) == 32, "two 16-byte pieces");

// RPW query rows per softmax group, NWG groups (each with its own rows of every tile).
template <int D, int RPW, int NWG>
__global__ void __launch_bounds__((NQ * NWG + 7) * 32, 1)
attn_q8_kernel(const __grid_constant__ CUtensorMap tmap_k,
               const __grid_constant__ CUtensorMap tmap_v, const __nv_bfloat16* __restrict__ q,
               const uint8_t* __restrict__ k_scale, const uint8_t* __restrict__ v_scale,
               const int32_t* __restrict__ block_table, int max_pages, int num_pages,
               const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ cu_q, int B,
               int total_q, int max_q, int max_seq_len, int Hq, int Hkv, float scale_log2,
               float* __restrict__ ws_o, float* __restrict__ ws_ml, int maxC,
               unsigned int* __restrict__ cnt, unsigned int* err) {
    using C = Cfg<D>;
    constexpr int NST = C::NST;
    constexpr int RP = RPW * NWG;
    constexpr int EPI = NQ * NWG;  // first epilogue warp (a multiple of 4: its lane quarter is 0)
    constexpr int PRODUCER = EPI + 4, S_WARP = EPI + 5, PV_WARP = EPI + 6;
    constexpr int THREADS = (EPI + 7) * 32;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    uint8_t* sQ = smem + C::Q_OFF;
    uint8_t* sP = smem + C::P_OFF;
    uint8_t* sStage = smem + C::RING_OFF;
    uint8_t* sScale = smem + C::SCALE_OFF;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
    uint64_t* empty = full + NST;
    uint64_t* s_full = empty + NST;     // scores of tile g in S buffer g % NSB
    uint64_t* s_empty = s_full + NSB;   // ... read by the softmax warps
    uint64_t* p_full = s_empty + NSB;   // P of tile g in P buffer g & 1
    uint64_t* p_empty = p_full + 2;     // P V of tile g has completed (MMA commit)
    uint64_t* o_full = p_empty + 2;     // item k's O (buffer k & 1) is complete (MMA commit)
    uint64_t* o_empty = o_full + 2;     // ... and read out by the epilogue warps
    uint64_t* xs_bar = o_empty + 2;     // item k's row sums and maxima are in xs[k & 1]
    uint64_t* q_full = xs_bar + 2;      // item k's Q tile and row factors are in buffer k & 1
    uint64_t* d_full = q_full + 2;      // item k's descriptor is in items[k % NDESC]
    uint64_t* drain = d_full + NDESC;   // [2]: S issuer, P V issuer
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
    Item* items = reinterpret_cast<Item*>(smem + C::DESC_OFF);
    float* xs = reinterpret_cast<float*>(smem + C::XS_OFF);  // [2][NQ + 1][QR]
    float* q_fac = xs + 2 * (NQ + 1) * QR;                   // [2][QR]
    float* x_max = q_fac + 2 * QR;                           // [NQ][QR]
    int* stage_valid = reinterpret_cast<int*>(smem + C::MISC_OFF);  // [NST], a bit per page
    int* prefix = stage_valid + NST;                         // [B + 1]
    int* done = prefix + MAX_BATCH + 1;                      // [4]: epilogue warps per item
    volatile int* abort_flag = reinterpret_cast<volatile int*>(done + 4);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = Hq / Hkv;
    const int TQ = QR / G;  // tokens of a query tile

    if (warp == S_WARP) {
        tmem_alloc(tmem_slot, TMEM_COLS);
        tmem_relinquish();
    }
    // With item counters the grid before this one is the call's own counter reset, which
    // waited for everything before it: the inputs are final, and only the counters need the
    // epilogue's wait (see attention.cu).  Without, this grid waits for the previous one.
    if (!cnt) {
        pdl_wait();
        pdl_trigger();
    }
    const unsigned long long wait_ns = wait_budget_ns(err);
    if (tid == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < NSB; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], NQ * NWG);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&p_full[i], NQ * NWG);
            mbar_init(&p_empty[i], 1);
            mbar_init(&o_full[i], 1);
            mbar_init(&o_empty[i], 4);
            mbar_init(&xs_bar[i], NQ * NWG);
            mbar_init(&q_full[i], 4);
            mbar_init(&drain[i], 1);
        }
        for (int i = 0; i < NDESC; ++i) mbar_init(&d_full[i], 1);
        for (int i = 0; i < 4; ++i) done[i] = 0;
        *abort_flag = 0;
        fence_barrier_init();
    }
    for (int b = tid; b < B; b += THREADS) {
        const SeqInfo si = seq_info(seq_lens, cu_q, b);
        const bool ok = seq_ok(si, max_q, max_seq_len, total_q);
        if (!ok) latch_error(err, kErrDeviceArg);
        prefix[b + 1] = ok ? ((si.L + CHUNK - 1) >> CHUNK_LOG2) * ((si.qb + TQ - 1) / TQ) * Hkv : 0;
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 0) {  // inclusive scan of prefix[1..B], 32 at a time
        int carry = 0;
        for (int base = 0; base < B; base += 32) {
            const int i = base + lane;
            int v = i < B ? prefix[i + 1] : 0;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, off);
                if (lane >= off) v += u;
            }
            if (i < B) prefix[i + 1] = v + carry;
            carry += __shfl_sync(0xffffffffu, v, 31);
        }
        if (lane == 0) prefix[0] = 0;
    }
    __syncthreads();
    const uint32_t tmem_base = *tmem_slot;

    auto give_up = [&]() {
        if (!*abort_flag) {
            *abort_flag = 1;
            latch_error(err, kErrTimeout);
        }
    };
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (ok && !mbar_wait_warp(bar, parity, abort_flag, wait_ns)) ok = false;
        return ok;
    };
    // the descriptor of item k; npages = 0 after the last one (or when the wait ran out)
    auto item_at = [&](int k) {
        Item it;
        it.npages = 0;
        if (wait(&d_full[k % NDESC], uint32_t(k / NDESC) & 1u)) {
            const uint4* src = reinterpret_cast<const uint4*>(&items[k % NDESC]);
            const uint4 a = src[0], b = src[1];
            it = Item{int(a.x), int(a.y), int(a.z), int(a.w),
                      int(b.x), int(b.y), int(b.z), int(b.w)};
        }
        return it;
    };

    if (warp == PRODUCER) {
        // ------------------------------------------------------------------ producer
        // The whole warp runs the loop; one elected lane issues the copies.  It also finds
        // the items and publishes them one item ahead: item k's slot was last read for item
        // k - NDESC, and no reader is that far behind (the ring holds the producer at most
        // NST <= 8 tiles, so as many items, ahead of P V, and P V is at most two items ahead
        // of the epilogue).
        static_assert(NST + 4 < NDESC, "descriptors in flight");
        const int total = prefix[B];
        int w = blockIdx.x, pub = 0;
        // publishes the next item of this CTA that is not empty; lane k returns the physical
        // page of the item's page k
        auto publish = [&](Item& it, int& phys) {
            it.npages = 0;
            phys = -1;
            for (; w < total && it.npages == 0; w += gridDim.x) {
                int lo = 0, hi = B;
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (prefix[mid] <= w) lo = mid; else hi = mid;
                }
                const SeqInfo si = seq_info(seq_lens, cu_q, lo);
                const int U = (si.qb + TQ - 1) / TQ;
                const int r = w - prefix[lo];
                const int cu = r / Hkv;
                const int c = cu / U, u = cu - c * U;
                it.b = lo;
                it.h = r - cu * Hkv;
                it.L = si.L;
                it.key0 = c * CHUNK;
                it.t0 = si.t0 + u * TQ;
                it.ntok = min(TQ, si.qb - u * TQ);
                it.pos0 = si.L - si.qb + u * TQ;
                const int seen = it.pos0 + it.ntok - it.key0;
                it.npages = seen <= 0 ? 0 : min(CHUNK / PAGE, (seen + PAGE - 1) / PAGE);
            }
            if (lane < it.npages) {
                const int pidx = it.key0 / PAGE + lane;
                if (pidx < max_pages) phys = block_table[int64_t(it.b) * max_pages + pidx];
            }
            if (lane == 0) {
                items[pub % NDESC] = it;
                mbar_arrive(&d_full[pub % NDESC]);
            }
            ++pub;
        };
        if (lane == 0) {
            tma_prefetch_desc(&tmap_k);
            tma_prefetch_desc(&tmap_v);
        }
        // blocks of one query tile read K and V once; wider ones read them again from L2
        const uint64_t policy = max_q <= TQ ? l2_policy_evict_first() : l2_policy_evict_last();
        uint32_t g = 0;
        Item it, nx;
        int phys_l, phys_n;
        publish(it, phys_l);
        while (ok && it.npages > 0) {
            publish(nx, phys_n);
            for (int i = 0; i < it.npages; i += TPAGES, ++g) {
                const int s = int(g % NST);
                if (!wait(&empty[s], ((g / NST) & 1u) ^ 1u)) break;
                int phys[TPAGES], valid = 0;
#pragma unroll
                for (int k = 0; k < TPAGES; ++k) {
                    phys[k] = __shfl_sync(0xffffffffu, phys_l, i + k);
                    const bool there = i + k < it.npages;
                    const bool v = there && phys[k] >= 0 && phys[k] < num_pages;
                    if (v) valid |= 1 << k;
                    if (there && !v && lane == 0) latch_error(err, kErrDeviceArg);
                }
                if (elect_one()) {
                    stage_valid[s] = valid;
                    uint8_t* st = sStage + s * C::STAGE_BYTES;
                    if (valid)
                        mbar_arrive_expect_tx(&full[s], uint32_t(__popc(valid)) *
                                                            (2 * C::PAGE_BYTES + 2 * PAGE));
                    else
                        mbar_arrive(&full[s]);
#pragma unroll
                    for (int k = 0; k < TPAGES; ++k) {
                        if (valid & (1 << k)) {
                            const int row = (phys[k] * Hkv + it.h) * PAGE;
                            tma_load_2d_hint(st + k * C::PAGE_BYTES, &tmap_k, &full[s], 0, row,
                                             policy);
                            tma_load_2d_hint(st + C::SIDE_BYTES + k * C::PAGE_BYTES, &tmap_v,
                                             &full[s], 0, row, policy);
                            uint8_t* sc = sScale + s * 2 * TK + k * PAGE;
                            bulk_load(sc, k_scale + row, PAGE, &full[s]);
                            bulk_load(sc + TK, v_scale + row, PAGE, &full[s]);
                        }
                    }
                }
                __syncwarp();
            }
            it = nx;
            phys_l = phys_n;
        }
        if (!ok) {
            if (lane == 0) give_up();
            // copies already issued land before the CTA exits (bounded)
            for (int k = 1; k <= NST && k <= int(g); ++k) {
                const uint32_t gg = g - k;
                mbar_wait(&full[gg % NST], (gg / NST) & 1u, nullptr, 100000000ull);
            }
        }
    } else if (warp == S_WARP) {
        // ------------------------------------------------- S^T = K (Q_hi + Q_lo)^T
        constexpr uint32_t idesc = idesc_e4m3(TK, QR, 0, 0);
        const uint64_t q_desc0 = umma_smem_desc(smem_addr(sQ), 16, C::SBO, C::LAYOUT);
        const uint64_t k_desc0 = umma_smem_desc(smem_addr(sStage), 16, C::SBO, C::LAYOUT);
        uint32_t g = 0;
        for (int item = 0; ok; ++item) {
            const int npages = item_at(item).npages;
            if (npages == 0) break;
            const int qbuf = item & 1;
            if (!wait(&q_full[qbuf], uint32_t(item >> 1) & 1u)) break;
            for (int i = 0; i < npages; i += TPAGES, ++g) {
                const int s = int(g % NST), sb = int(g % NSB);
                if (!wait(&full[s], (g / NST) & 1u) ||
                    !wait(&s_empty[sb], ((g / NSB) & 1u) ^ 1u))
                    break;
                tc_fence_after_sync();
                if (elect_one()) {
                    const uint64_t k_desc = k_desc0 + uint64_t((s * C::STAGE_BYTES) >> 4);
                    const uint64_t q_desc = q_desc0 + uint64_t((qbuf * C::Q_BYTES) >> 4);
                    const uint32_t d = tmem_base + uint32_t(S_COL + sb * QR);
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) {  // head dims 32k .. 32k+31: +32 B
                        tc_mma_f8(d, k_desc + uint64_t(k * 2), q_desc + uint64_t(k * 2), idesc,
                                  k != 0 ? 1u : 0u);
                        tc_mma_f8(d, k_desc + uint64_t(k * 2),
                                  q_desc + uint64_t((C::Q_PIECE >> 4) + k * 2), idesc, 1u);
                    }
                    tc_commit(&s_full[sb]);
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) give_up();
        if (elect_one()) tc_commit(&drain[0]);
        __syncwarp();
        mbar_wait(&drain[0], 0, nullptr, 100000000ull);
    } else if (warp == PV_WARP) {
        // ------------------------------------------------- O^T += V^T [P_hi | P_lo]^T
        constexpr uint32_t idesc = idesc_e4m3(D, 2 * QR, 1, 1);
        const uint64_t v_desc0 =
            umma_smem_desc(smem_addr(sStage + C::SIDE_BYTES), 16, C::SBO, C::LAYOUT);
        const uint64_t p_desc0 = umma_smem_desc(smem_addr(sP), 16, 512, 4);
        uint32_t g = 0;
        for (int item = 0; ok; ++item) {
            const int npages = item_at(item).npages;
            if (npages == 0) break;
            const int ob = item & 1;
            // the O buffer of this item was read out for item-2
            if (!wait(&o_empty[ob], (uint32_t(item >> 1) & 1u) ^ 1u)) break;
            for (int i = 0; i < npages; i += TPAGES, ++g) {
                const int s = int(g % NST), pb = int(g & 1u);
                if (!wait(&p_full[pb], (g >> 1) & 1u)) break;
                tc_fence_after_sync();
                if (elect_one()) {
                    const uint64_t v_desc = v_desc0 + uint64_t((s * C::STAGE_BYTES) >> 4);
                    const uint64_t p_desc = p_desc0 + uint64_t((pb * C::P_BYTES) >> 4);
                    const uint32_t d = tmem_base + uint32_t(O_COL + ob * 2 * QR);
#pragma unroll
                    for (int k = 0; k < TK / 32; ++k)  // keys 32k .. 32k+31
                        tc_mma_f8(d, v_desc + uint64_t(k * 32 * D / 16),
                                  p_desc + uint64_t(k * 32 * 2 * QR / 16), idesc,
                                  (i | k) != 0 ? 1u : 0u);
                    tc_commit(&p_empty[pb]);
                    tc_commit(&empty[s]);  // K, V and scales of the tile are no longer read
                    if (i + TPAGES >= npages) tc_commit(&o_full[ob]);
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) give_up();
        if (elect_one()) tc_commit(&drain[1]);
        __syncwarp();
        mbar_wait(&drain[1], 0, nullptr, 100000000ull);
    } else if (warp >= EPI) {
        // ------------------------------------------------- Q split and epilogue
        const int ew = warp - EPI;  // tensor-memory lane quarter
        // Q tile of an item: four neighbouring threads split one row.
        auto split_q = [&](const Item& it, int buf) {
            constexpr int PER = D / 4;  // elements per thread
            const int r = ew * 8 + (lane >> 2), part = lane & 3;
            const int j = r / G;
            uint4 v[PER / 8];
#pragma unroll
            for (int k = 0; k < PER / 8; ++k) v[k] = make_uint4(0, 0, 0, 0);
            if (j < it.ntok && r < TQ * G) {
                const __nv_bfloat16* src =
                    q + (int64_t(it.t0 + j) * Hq + it.h * G + (r - j * G)) * D + part * PER;
#pragma unroll
                for (int k = 0; k < PER / 8; ++k)
                    v[k] = *reinterpret_cast<const uint4*>(src + k * 8);
            }
            uint32_t amax = 0;  // of bf16 magnitudes, which order as their bits
#pragma unroll
            for (int k = 0; k < PER / 8; ++k) {
                const uint32_t x[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    amax = max(amax, max(x[n] & 0x7fffu, (x[n] >> 16) & 0x7fffu));
            }
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // s = 7 - floor(log2(amax)), held where 2^s and 2^-s are normal
            const int s = max(-120, min(120, 134 - int(amax >> 7)));
            const float mul = __uint_as_float(uint32_t(127 + s) << 23);
            uint8_t* hi = sQ + buf * C::Q_BYTES;
            uint8_t* lo = hi + C::Q_PIECE;
#pragma unroll
            for (int k = 0; k < PER / 16; ++k) {
                uint32_t h[4], l[4];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const uint4& src = v[2 * k + (n >> 1)];
                    const uint32_t x0 = n & 1 ? src.z : src.x, x1 = n & 1 ? src.w : src.y;
                    float f[4] = {__uint_as_float(x0 << 16) * mul,
                                  __uint_as_float(x0 & 0xffff0000u) * mul,
                                  __uint_as_float(x1 << 16) * mul,
                                  __uint_as_float(x1 & 0xffff0000u) * mul};
                    const uint32_t c0 = e4m3x2(f[0], f[1]), c1 = e4m3x2(f[2], f[3]);
                    const float2 b0 = e4m3x2_values(c0), b1 = e4m3x2_values(c1);
                    h[n] = c0 | (c1 << 16);
                    l[n] = e4m3x2(f[0] - b0.x, f[1] - b0.y) |
                           (e4m3x2(f[2] - b1.x, f[3] - b1.y) << 16);
                }
                const uint32_t at = swz_row<D>(r, part * (PER / 16) + k);
                *reinterpret_cast<uint4*>(hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4*>(lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
            }
            // a query with an infinity or NaN scores NaN throughout
            if (part == 0)
                q_fac[buf * QR + r] = amax >= 0x7f80u
                                          ? __int_as_float(0x7fc00000)
                                          : scale_log2 * __uint_as_float(uint32_t(127 - s) << 23);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[buf]);
        };
        bool reset_done = cnt == nullptr;  // griddepcontrol.wait passed
        // Item k's stores are counted an item later, when the fence finds them done.  The last
        // of the four warps counts; done[k & 3] holds no other item's arrivals, since a warp
        // that counts item k has seen O of item k, so every warp has read O of item k - 2 and
        // counted item k - 3.
        auto count = [&](int k, int at) {
            if (!cnt) return;
            __threadfence();
            __syncwarp();
            if (!reset_done) {
                pdl_wait();
                pdl_trigger();
                reset_done = true;
            }
            if (lane == 0 && (atomicAdd(&done[k & 3], 1) & 3) == 3) {
                __threadfence();
                atomicAdd(cnt + at, 1u);
            }
        };
        Item it = item_at(0), nx;
        if (it.npages > 0) split_q(it, 0);
        int item = 0, prev = -1;
        for (; ok && it.npages > 0; ++item) {
            nx = item_at(item + 1);
            // (this buffer's item-1 is complete: its O was waited for)
            if (nx.npages > 0) split_q(nx, (item + 1) & 1);
            if (prev >= 0) count(item - 1, prev);
            const int ob = item & 1;
            const uint32_t par = uint32_t(item >> 1) & 1u;
            if (!wait(&xs_bar[ob], par) || !wait(&o_full[ob], par)) break;
            tc_fence_after_sync();
            uint32_t vh[RP], vl[RP];
            const uint32_t ta =
                tmem_base + (uint32_t(32 * ew) << 16) + uint32_t(O_COL + ob * 2 * QR);
            tmem_cols(ta, vh);
            tmem_cols(ta + QR, vl);
            tc_fence_before_sync();
            // rows (token j, head gg) are stored when their token sees the chunk
            const int rows = it.ntok * G;
            const int first = max(0, it.key0 - it.pos0) * G;
            const int c = it.key0 >> CHUNK_LOG2;
            const int64_t row0 = int64_t(it.t0) * Hq + int64_t(it.h) * G;
            if (ew == 0) {
                const int r = lane, j = r / G;
                if (r < rows && r >= first) {
                    const float* x = xs + ob * ((NQ + 1) * QR);
                    const float l = ((x[r] + x[QR + r]) + x[2 * QR + r]) + x[3 * QR + r];
                    const int64_t idx = (row0 + int64_t(j) * (Hq - G) + r) * maxC + c;
                    *reinterpret_cast<float2*>(ws_ml + idx * 2) = make_float2(x[NQ * QR + r], l);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_empty[ob]);
            // O^T: lane = head dim (M = 128), or dims 16 ew .. 16 ew + 15 in lanes 0..15 (M = 64)
            const int d = D == 128 ? ew * 32 + lane : ew * 16 + lane;
            if (D == 128 || lane < 16) {
                float* dst = ws_o + (row0 * maxC + c) * D + d;
                const int64_t step = int64_t(maxC) * D, skip = step * (Hq - G);
                int gg = 0;
#pragma unroll
                for (int r = 0; r < RP; ++r) {
                    if (r < rows && r >= first)
                        *dst = fmaf(__uint_as_float(vl[r]), 1.f / kLoScale, __uint_as_float(vh[r]));
                    dst += step;
                    if (++gg == G) {
                        gg = 0;
                        dst += skip;
                    }
                }
            }
            prev = it.b * Hkv + it.h;
            it = nx;
        }
        if (ok && prev >= 0) count(item - 1, prev);
        if (!ok && lane == 0) give_up();
        // a CTA with no item (or one that gave up) still waits before it completes
        if (!reset_done) {
            pdl_wait();
            pdl_trigger();
        }
    } else {
        // ------------------------------------------------------------------- softmax
        // Group wg owns query rows wg * RPW .. of every tile; each thread one key.
        const int wg = warp / NQ, wq = warp % NQ;
        const int key = wq * 32 + lane;
        const int row0 = wg * RPW;
        const uint32_t lane_base = uint32_t(32 * wq) << 16;
        uint32_t g = 0;
        float m[RPW], l[RPW];
        for (int item = 0;; ++item) {
            const Item it = item_at(item);
            const int ob = item & 1;
            const uint32_t ipar = uint32_t(item >> 1) & 1u;
            if (it.npages > 0) wait(&q_full[ob], ipar);
            if (!ok && lane == 0) give_up();
            if (group_or(1 + wg, !ok) || it.npages == 0) break;
            const float* fac = q_fac + ob * QR + row0;
#pragma unroll
            for (int r = 0; r < RPW; ++r) {
                m[r] = kNoMax;
                l[r] = 0.f;
            }
            bool left = false;
            for (int i = 0; i < it.npages; i += TPAGES, ++g) {
                const int s = int(g % NST), sb = int(g % NSB), pb = int(g & 1u);
                const int kp = it.key0 + i * PAGE + key;  // this key's position
                wait(&full[s], (g / NST) & 1u);
                const bool live = ((stage_valid[s] >> (key / PAGE)) & 1) && kp < it.L;
                const uint32_t ksc = sScale[s * 2 * TK + key], vsc = sScale[s * 2 * TK + TK + key];
                wait(&s_full[sb], (g / NSB) & 1u);
                tc_fence_after_sync();
                uint32_t sv[RPW];
                tmem_cols(tmem_base + lane_base + uint32_t(S_COL + sb * QR + row0), sv);
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_empty[sb]);
                const float ka = e8m0(ksc);
                const float vb = vsc == 255 ? __int_as_float(0x7fc00000) : float(int(vsc) - 127);
                const float vinv = live ? e8m0_inv(vsc) : 0.f;
                float t[RPW];
#pragma unroll
                for (int r = 0; r < RPW; r += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(fac + r);
                    t[r] = fmaf(__uint_as_float(sv[r]) * ka, f.x, vb);
                    t[r + 1] = fmaf(__uint_as_float(sv[r + 1]) * ka, f.y, vb);
                    t[r + 2] = fmaf(__uint_as_float(sv[r + 2]) * ka, f.z, vb);
                    t[r + 3] = fmaf(__uint_as_float(sv[r + 3]) * ka, f.w, vb);
                }
                // causal mask: row r (token r / G) sees the key when r / G >= kp - pos0
                if (!__all_sync(0xffffffffu, live && kp <= it.pos0)) {
                    const int first = live ? max(0, kp - it.pos0) * G : QR;  // first row seeing it
#pragma unroll
                    for (int r = 0; r < RPW; ++r) t[r] = row0 + r >= first ? t[r] : -INFINITY;
                }
                // does any row's maximum exceed its reference by more than 2^8?
                bool slow = i == 0;
                if (!slow) {
                    float over[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int r = 0; r < RPW; ++r) over[r & 3] = fmaxf(over[r & 3], t[r] - m[r]);
                    slow = group_or(1 + wg, !ok || fmaxf(fmaxf(over[0], over[1]),
                                                         fmaxf(over[2], over[3])) > kRaise);
                }
                if (slow) {
                    // the tile's maximum of every row, over the four warps
                    const float mine = combine_lanes<RPW, true>(t, lane);
                    if (lane % (32 / RPW) == 0) x_max[wq * QR + row0 + lane / (32 / RPW)] = mine;
                    if (!ok && lane == 0) give_up();
                    if (group_or(1 + wg, !ok)) {
                        ok = false;
                        left = true;
                        break;
                    }
                    // O of this warp's lanes may be scaled once P V of the tile before is done
                    const uint32_t gp = g - 1u;
                    if (i > 0) wait(&p_empty[gp & 1u], (gp >> 1) & 1u);
                    tc_fence_after_sync();
#pragma unroll
                    for (int r0 = 0; r0 < RPW; r0 += 8) {
                        float fa[8];
#pragma unroll
                        for (int k = 0; k < 8; k += 4) {
                            float4 x = *reinterpret_cast<const float4*>(x_max + row0 + r0 + k);
#pragma unroll
                            for (int n = 1; n < NQ; ++n) {
                                const float4 y = *reinterpret_cast<const float4*>(
                                    x_max + n * QR + row0 + r0 + k);
                                x = make_float4(fmaxf(x.x, y.x), fmaxf(x.y, y.y),
                                                fmaxf(x.z, y.z), fmaxf(x.w, y.w));
                            }
                            const float mt[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int n = 0; n < 4; ++n) {
                                const int r = r0 + k + n;
                                const bool raise = mt[n] > m[r] + kRaise;
                                const float mn = raise ? mt[n] - kHeadroom : m[r];
                                fa[k + n] = raise ? ex2(m[r] - mn) : 1.f;
                                m[r] = mn;
                                l[r] *= fa[k + n];
                            }
                        }
                        if (i > 0) {
                            uint32_t o[8];
                            const uint32_t ta = tmem_base + lane_base +
                                                uint32_t(O_COL + ob * 2 * QR + row0 + r0);
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                tmem_cols(ta + half * QR, o);
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    o[k] = __float_as_uint(__uint_as_float(o[k]) * fa[k]);
                                tmem_store_x8(ta + half * QR, o);
                            }
                        }
                    }
                    tc_fence_before_sync();
                }
                uint32_t hi[RPW / 4], lo[RPW / 4];
#pragma unroll
                for (int r = 0; r < RPW; r += 4) {
                    float p[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        p[k] = ex2(t[r + k] - m[r + k]);
                        l[r + k] = fmaf(p[k], vinv, l[r + k]);
                    }
                    const uint32_t c0 = e4m3x2(p[0], p[1]), c1 = e4m3x2(p[2], p[3]);
                    const float2 b0 = e4m3x2_values(c0), b1 = e4m3x2_values(c1);
                    hi[r / 4] = c0 | (c1 << 16);
                    lo[r / 4] = e4m3x2((p[0] - b0.x) * kLoScale, (p[1] - b0.y) * kLoScale) |
                                (e4m3x2((p[2] - b1.x) * kLoScale, (p[3] - b1.y) * kLoScale) << 16);
                }
                // P buffer pb is free once P V of tile g-2 has completed
                wait(&p_empty[pb], ((g >> 1) & 1u) ^ 1u);
                if (!ok) continue;  // (to the group's next common decision)
                uint8_t* pbuf = sP + pb * C::P_BYTES;
                if (RPW == 8) {
                    const int at = wg * 8;
                    *reinterpret_cast<uint2*>(pbuf + swz_row<64>(key, 0) + at) =
                        make_uint2(hi[0], hi[1]);
                    *reinterpret_cast<uint2*>(pbuf + swz_row<64>(key, 2) + at) =
                        make_uint2(lo[0], lo[1]);
                } else {
                    *reinterpret_cast<uint4*>(pbuf + swz_row<64>(key, wg)) =
                        make_uint4(hi[0], hi[1], hi[RPW / 4 - 2], hi[RPW / 4 - 1]);
                    *reinterpret_cast<uint4*>(pbuf + swz_row<64>(key, 2 + wg)) =
                        make_uint4(lo[0], lo[1], lo[RPW / 4 - 2], lo[RPW / 4 - 1]);
                }
                // V rows past the sequence's end or of an invalid page are zeroed, so that
                // unwritten codes (NaN) cannot reach O through 0 * v
                if (wg == 0 && !live) {
                    uint4* vr = reinterpret_cast<uint4*>(sStage + s * C::STAGE_BYTES +
                                                         C::SIDE_BYTES + key * D);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) vr[k] = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[pb]);
            }
            if (left) break;
            // the warp's row sums (and the maxima) for the epilogue, once it has read this
            // buffer's previous contents (item-2)
            wait(&o_empty[ob], ipar ^ 1u);
            float* x = xs + ob * ((NQ + 1) * QR) + row0;
            const float sum = combine_lanes<RPW, false>(l, lane);
            if (ok) {
                if (wq == 0 && lane == 0) {
#pragma unroll
                    for (int r = 0; r < RPW; ++r) x[NQ * QR + r] = m[r];
                }
                if (lane % (32 / RPW) == 0) x[wq * QR + lane / (32 / RPW)] = sum;
                __syncwarp();
                if (lane == 0) mbar_arrive(&xs_bar[ob]);
            }
        }
        if (!ok && lane == 0) give_up();
    }
    // every warp is done with tensor memory and shared memory past this barrier
    tc_fence_before_sync();
    __syncthreads();
    if (warp == S_WARP) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

template <int D, int RPW, int NWG>
cudaError_t launch_q8_t(const DeviceInfo& dev, const void* q, const PagedArgs& a,
                        const void* k_scale, const void* v_scale, float scale, void* out,
                        float* lse, void* workspace, cudaStream_t stream) {
    using Cf = Cfg<D>;
    const uint64_t rows = uint64_t(a.num_pages) * uint64_t(a.hkv) * PAGE;
    CUtensorMap tk, tv;
    if (!tmap_2d_u8_swizzled(&tk, a.k_cache, D, rows, PAGE) ||
        !tmap_2d_u8_swizzled(&tv, a.v_cache, D, rows, PAGE))
        return cudaErrorNotSupported;
    auto kern = attn_q8_kernel<D, RPW, NWG>;
    static bool attr_done[64] = {};
    if (dev.device >= 0 && dev.device < 64 && !attr_done[dev.device]) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             int(Cf::SMEM));
        if (e != cudaSuccess) return e;
        attr_done[dev.device] = true;
    }
    const int maxC = int((a.max_seq_len + CHUNK - 1) / CHUNK);
    const int64_t TQ = QR / (a.hq / a.hkv);
    const int64_t tiles = (a.max_q + TQ - 1) / TQ;
    const int64_t items_bound = a.batch * int64_t(maxC) * tiles * a.hkv;
    if (items_bound > 0x7fffffffLL - dev.num_sms) return cudaErrorNotSupported;
    const int grid = int(items_bound < dev.num_sms ? items_bound : dev.num_sms);
    float* ws_o = static_cast<float*>(workspace);
    float* ws_ml = ws_o + a.total_q * a.hq * int64_t(maxC) * D;
    // one query tile per sequence: the merge of a (sequence, KV head) starts when its chunks
    // are counted; more: it waits for the whole grid
    unsigned int* cnt = nullptr;
    if (tiles == 1) {
        cnt = attn_item_counters(a, workspace, CHUNK_LOG2);
        cudaError_t e = launch_attn_count_reset(cnt, int(a.batch * a.hkv), stream);
        if (e != cudaSuccess) return e;
    }
    cudaError_t e = launch_pdl(
        kern, dim3(grid), dim3((NQ * NWG + 7) * 32), Cf::SMEM, stream, tk, tv,
        static_cast<const __nv_bfloat16*>(q), static_cast<const uint8_t*>(k_scale),
        static_cast<const uint8_t*>(v_scale), a.block_table, int(a.max_pages), int(a.num_pages),
        a.seq_lens, a.cu_q, int(a.batch), int(a.total_q), int(a.max_q), int(a.max_seq_len),
        int(a.hq), int(a.hkv), scale * kLog2e, ws_o, ws_ml, maxC, cnt, dev.err_word);
    if (e != cudaSuccess) return e;
    return launch_attn_merge(a, workspace, CHUNK_LOG2, out, lse, cnt, dev.err_word, stream);
}

}  // namespace

cudaError_t launch_attention_q8(const DeviceInfo& dev, const void* q, const PagedArgs& a,
                                const void* k_scale, const void* v_scale, float scale, void* out,
                                float* lse, void* workspace, cudaStream_t stream) {
    // query rows of the fullest tile: up to 8 in one softmax group, 16 or 32 over two
    const int64_t G = a.hq / a.hkv, TQ = QR / G;
    const int64_t rows = (a.max_q < TQ ? a.max_q : TQ) * G;
    auto run = [&](auto f) {
        return f(dev, q, a, k_scale, v_scale, scale, out, lse, workspace, stream);
    };
    if (a.head_dim == 64)
        return run(rows <= 8    ? launch_q8_t<64, 8, 1>
                   : rows <= 16 ? launch_q8_t<64, 8, 2>
                                : launch_q8_t<64, 16, 2>);
    return run(rows <= 8    ? launch_q8_t<128, 8, 1>
               : rows <= 16 ? launch_q8_t<128, 8, 2>
                            : launch_q8_t<128, 16, 2>);
}

}  // namespace bi

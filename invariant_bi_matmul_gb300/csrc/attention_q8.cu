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
//   * q * 2^s (s puts the row's largest value in [128, 256) where that is 2^-113 or more) =
//     hi + lo, each rounded to nearest: exact for bf16 q down to 2^-9 of the row's largest
//     value, off by at most 2^-17 of it below (2^-10 beside 128);
//   * p = hi + lo / 32: p <= 2^8, rounded to binary16 first; hi has four bits, lo the next
//     four, so p is held to 2^-9 + 2^-11 of itself (bf16 would hold 2^-8) or, in place of the
//     2^-9, to 2^-15 absolute (2^-23 of the row's largest), whichever is more.
//
// Reduction of one (query, head) -- a function of its position alone, as in attention.cu:
// chunks of 512 keys from key 0; m is the exact maximum of the row's t over the chunk, less 8
// (so p <= 2^8); a chunk is four tiles of 128 keys, each of 128 threads sums its key of every
// tile in ascending order, and the 128 sums are added by a fixed tree; the chunk partials
// (m, l, o) go through the merge of attention.cu.  Keys that a row does not see have t = -inf and
// add +0, and a row's place in the MMA tile, the other rows and the block's width enter nowhere.
//
// A softmax thread holds its four t of every row in registers between the maximum and the
// exponentials, so a chunk needs one exchange between warps and O is never rescaled.  (With a
// running maximum per tile, every tile cost an exchange, and rows whose maximum kept rising a
// rescale of O: 299 us where this form took 230, 64 ragged sequences of up to 16,388 keys.)
// K and V have rings of their own: K runs an item ahead of V, so the scores of the next chunk
// are ready when this one's P is done.
//
// Orientation.  S^T = K Q^T (M = 128 keys, N = 32 query rows) and O^T = V^T P^T (M = head
// dim, N = 32 hi + 32 lo rows): the cache is the operand that the tensor core reads 128 rows
// at a time, whatever the number of query rows, and a softmax thread owns one key of a tile, so
// it does as many exponentials as there are query rows (rounded up to 4, 8, 16 or 32), reads its
// key's two scale bytes once, and writes its P values in pieces of 4 or 8 bytes.
//
// Warps: one, two or four softmax groups of four warps (4 or 8 query rows each), four epilogue
// warps, the scheduler, a TMA producer for K and one for V, the S issuer (and TMEM owner), the
// P V issuer, the counter, one or two warps that split Q and fetch the scale bytes.  One
// persistent CTA per SM; work items (sequence, chunk, query tile, KV head) are enumerated on
// the device.  All waits are bounded; the one barrier that warps meet in, a softmax group's,
// is left by all of them together.
//
// Bound by memory: 2 * (D + 1) bytes per key and KV head against 4 * 32 * D operations.  One query
// row per KV group of four: eight sequences of 65,540 keys 165 us (97% of the copy rate), 64 ragged
// ones of up to 16,388 220 us (98%), one of 1,028 9.6 us (launches, one chunk's chain, the merge).
// 32 query rows: 64 of 8,196 keys 240 us (67%: 4 us an item where one row takes 3.2, and a merge
// of 145 MB), one of 65,540 38.8 us (51%: seven rounds of items).  The two instances of 32 rows
// have 28 warps at 72 registers and spill 40 bytes.
#include "attn_common.cuh"

#include <cuda_fp8.h>

namespace bi {
namespace {

constexpr int QR = 32;                    // query rows of a tile
constexpr int TK = 128;                   // keys of a tile: two pages
constexpr int TPAGES = TK / PAGE;
constexpr int NQ = 4;                     // warps of a softmax group: 32 keys each
constexpr int NDESC = 64;                 // item descriptors in flight
constexpr int LEAD = 16;                  // items found ahead of the K copies, at most
constexpr int NT = CHUNK / TK;            // tiles of a chunk
constexpr int TMEM_COLS = 512;
constexpr int S_COL = 0;                  // two S sets (by item) of NT tiles, 32 columns each
constexpr int O_COL = 2 * NT * QR;          // O buffers (by item): 32 hi + 32 lo columns each
constexpr uint32_t kOddScale = 224;       // scale bytes from here on take the longer way
constexpr float kLowest = -3.402823466e38f;  // the maximum, where a row sees no key of a chunk
constexpr float kHeadroom = 8.f;          // p = 2^8 at the row's maximum (e4m3 holds 448)
constexpr float kLoScale = 32.f;          // the second piece of p (at most 8) times this
constexpr int MAX_BATCH = BI_ATTN_MAX_BATCH;

static_assert(CHUNK % TK == 0 && TK == NQ * 32, "a thread per key");
static_assert(O_COL + 2 * 2 * QR <= TMEM_COLS, "tensor memory columns");

template <int D>
struct Cfg {
    static constexpr int NSLOT = D == 64 ? 10 : 5;       // tiles in the K ring, and in V's
    static constexpr int PAGE_BYTES = PAGE * D;
    static constexpr int SLOT_BYTES = TK * D;
    static constexpr int Q_PIECE = QR * D;               // hi or lo of a Q tile
    static constexpr int Q_BYTES = 2 * Q_PIECE;
    static constexpr int P_BYTES = TK * 2 * QR;          // [key][32 hi | 32 lo]
    static constexpr int Q_OFF = 0;                      // two Q buffers
    static constexpr int P_OFF = Q_OFF + 2 * Q_BYTES;
    static constexpr int RING_OFF = P_OFF + NT * P_BYTES;
    static constexpr int V_OFF = RING_OFF + NSLOT * SLOT_BYTES;
    static constexpr int SCALE_OFF = V_OFF + NSLOT * SLOT_BYTES;  // two sets of scale bytes,
    static constexpr int SCALE_BYTES = 2 * TK * NT;               // [K | V][key][tile]
    static constexpr int BAR_OFF = SCALE_OFF + 2 * SCALE_BYTES;
    static constexpr int NBARS = 4 * NSLOT + 4 + 2 + 4 + 4 + 2 + 4 + NDESC + LEAD + 2;
    static constexpr int DESC_OFF = (BAR_OFF + NBARS * 8 + 8 + 15) / 16 * 16;
    static constexpr int XS_OFF = DESC_OFF + NDESC * 64;
    // per item (four buffers): four warps' row sums and the row maxima; per Q buffer the row
    // factors; the maxima exchanged within the softmax groups (two buffers: a warp may be an
    // item ahead)
    static constexpr int XS_FLOATS = 4 * (NQ + 1) * QR + 2 * QR + 2 * NQ * QR;
    static constexpr int MISC_OFF = XS_OFF + XS_FLOATS * 4;
    static constexpr int MISC_INTS = (MAX_BATCH + 1) + 1 + 4;
    static constexpr size_t SMEM = 1024 + size_t(MISC_OFF) + MISC_INTS * 4;
    // K-major and MN-major rows of D bytes: the 128- or 64-byte swizzle, groups of 8 rows
    static constexpr uint32_t LAYOUT = D == 128 ? 2 : 4;
    static constexpr uint32_t SBO = 8 * D;
    // swizzled tiles start on their pattern's boundary, what is read and written 16 bytes at a
    // time (scale bytes, descriptors, row factors, sums and maxima) and the barriers on theirs
    static_assert(Q_OFF % 1024 == 0 && Q_PIECE % 1024 == 0 && P_OFF % 1024 == 0 &&
                      P_BYTES % 1024 == 0 && RING_OFF % 1024 == 0 && V_OFF % 1024 == 0 &&
                      SLOT_BYTES % 1024 == 0 && PAGE_BYTES % 1024 == 0,
                  "tiles");
    static_assert(SCALE_OFF % 16 == 0 && SCALE_BYTES % 16 == 0 && TK * NT % 16 == 0 &&
                      BAR_OFF % 8 == 0 && DESC_OFF % 16 == 0 && XS_OFF % 16 == 0 &&
                      (NQ + 1) * QR % 4 == 0 && QR % 4 == 0 && MISC_OFF % 4 == 0,
                  "regions");
    static_assert(DESC_OFF >= BAR_OFF + NBARS * 8 + 4, "the tensor memory's address fits");
    static_assert(LEAD + NSLOT + 6 < NDESC, "descriptors in flight (see the scheduler)");
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

// RP consecutive columns of this warp's 32 lanes, with the wait.
__device__ __forceinline__ void tmem_cols(uint32_t ta, uint32_t (&r)[4]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(ta)
        : "memory");
}
__device__ __forceinline__ void tmem_cols(uint32_t ta, uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(ta)
        : "memory");
}
__device__ __forceinline__ void tmem_cols(uint32_t ta, uint32_t (&r)[16]) {
    tmem_load_32x32b_x16_sync(ta, r);
}
// RPW columns of each of a set's four S tiles (QR columns apart), with one wait.
__device__ __forceinline__ void tmem_tiles(uint32_t ta, uint32_t (&r)[NT][8]) {
    static_assert(NT == 4, "four loads");
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%33];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%16, %17, %18, %19, %20, %21, %22, %23}, [%34];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%24, %25, %26, %27, %28, %29, %30, %31}, [%35];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0][0]), "=r"(r[0][1]), "=r"(r[0][2]), "=r"(r[0][3]), "=r"(r[0][4]), "=r"(r[0][5]),
          "=r"(r[0][6]), "=r"(r[0][7]), "=r"(r[1][0]), "=r"(r[1][1]), "=r"(r[1][2]), "=r"(r[1][3]),
          "=r"(r[1][4]), "=r"(r[1][5]), "=r"(r[1][6]), "=r"(r[1][7]), "=r"(r[2][0]), "=r"(r[2][1]),
          "=r"(r[2][2]), "=r"(r[2][3]), "=r"(r[2][4]), "=r"(r[2][5]), "=r"(r[2][6]), "=r"(r[2][7]),
          "=r"(r[3][0]), "=r"(r[3][1]), "=r"(r[3][2]), "=r"(r[3][3]), "=r"(r[3][4]), "=r"(r[3][5]),
          "=r"(r[3][6]), "=r"(r[3][7])
        : "r"(ta), "r"(ta + QR), "r"(ta + 2 * QR), "r"(ta + 3 * QR)
        : "memory");
}
__device__ __forceinline__ void tmem_tiles(uint32_t ta, uint32_t (&r)[NT][4]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%16];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%4, %5, %6, %7}, [%17];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%8, %9, %10, %11}, [%18];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%12, %13, %14, %15}, [%19];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0][0]), "=r"(r[0][1]), "=r"(r[0][2]), "=r"(r[0][3]), "=r"(r[1][0]), "=r"(r[1][1]),
          "=r"(r[1][2]), "=r"(r[1][3]), "=r"(r[2][0]), "=r"(r[2][1]), "=r"(r[2][2]), "=r"(r[2][3]),
          "=r"(r[3][0]), "=r"(r[3][1]), "=r"(r[3][2]), "=r"(r[3][3])
        : "r"(ta), "r"(ta + QR), "r"(ta + 2 * QR), "r"(ta + 3 * QR)
        : "memory");
}

// The sum of v[r] over the 32 lanes for each of N rows, over a fixed tree: lanes that differ in
// bit 4, then bit 3, .. bit 0 -- the same for every N.  Every lane gets row lane * N / 32: at
// each step a lane keeps one half of its rows while it has several.
template <int N, int OFF = 16>
__device__ __forceinline__ float sum_lanes(const float (&v)[N], int lane) {
    if constexpr (OFF == 0) {
        return v[0];
    } else if constexpr (N == 1) {
        const float w[1] = {v[0] + __shfl_xor_sync(0xffffffffu, v[0], OFF)};
        return sum_lanes<1, OFF / 2>(w, lane);
    } else {
        const bool up = (lane & OFF) != 0;
        float w[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float got = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + N / 2], OFF);
            w[i] = (up ? v[i + N / 2] : v[i]) + got;
        }
        return sum_lanes<N / 2, OFF / 2>(w, lane);
    }
}

// Two fp32 operations in one instruction, each rounded as its scalar form.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// The largest of 32 lanes' values (a NaN is ignored beside a number).
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// The two e4m3 pieces of (a, b), both in [0, 2^8]: hi in the low half of the result, lo (times
// kLoScale) in the high half.  By way of binary16, whose eleven bits lose 2^-11 of a value.
__device__ __forceinline__ uint32_t split_p(float a, float b) {
    const __half2 p = __floats2half2_rn(a, b);
    const uint32_t hi = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(p), __NV_SATFINITE, __NV_E4M3);
    const __half2 h(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(hi), __NV_E4M3));
    const __half2 l = __hmul2(__hsub2(p, h), __float2half2_rn(kLoScale));  // exact
    const uint32_t lo = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(l), __NV_SATFINITE, __NV_E4M3);
    return hi | (lo << 16);
}

// The two e4m3 pieces of two bf16 values times `mul`: hi in the low half of the result, lo in
// the high half.  Binary16 holds the products (below 2^8) but for bits under 2^-24.
__device__ __forceinline__ uint32_t split_q(uint32_t x, float mul) {
    const __half2 p = __floats2half2_rn(__uint_as_float(x << 16) * mul,
                                        __uint_as_float(x & 0xffff0000u) * mul);
    const uint32_t hi = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(p), __NV_SATFINITE, __NV_E4M3);
    const __half2 h(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(hi), __NV_E4M3));
    const uint32_t lo =
        __nv_cvt_halfraw2_to_fp8x2(__half2_raw(__hsub2(p, h)), __NV_SATFINITE, __NV_E4M3);
    return hi | (lo << 16);
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

// A work item as the scheduler publishes it: chunk c of the keys for one query tile of
// sequence b, KV head h.
struct alignas(16) Item {
    int npages;  // pages of the chunk that the tile's last token sees (0: no more items)
    int key0;    // first key of the chunk
    int L;       // the sequence's length
    int pos0;    // position of the tile's first token
    int t0;      // its row in q and out
    int ntok;    // the tile's tokens
    int h;
    int bq;      // 4 * b + 2 when every row sees every key of the chunk + its Q tile's buffer
};
struct alignas(16) ItemSlot {
    Item it;
    int phys[CHUNK / PAGE];  // physical pages, -1 for those that are not there or out of range
};
static_assert(sizeof(ItemSlot) == 64 && CHUNK / PAGE == 8, "four 16-byte pieces");

__device__ __forceinline__ int tiles_of(int npages) { return (npages + TPAGES - 1) / TPAGES; }

// NWG softmax groups of RPW query rows.
// softmax, epilogue, scheduler, K, V, S, P V, counter, one or two preparing warps
template <int NWG>
constexpr int kWarps = NQ * NWG + 4 + 6 + (NWG == 4 ? 2 : 1);

template <int D, int RPW, int NWG>
__global__ void __launch_bounds__(kWarps<NWG> * 32, 1)
attn_q8_kernel(const __grid_constant__ CUtensorMap tmap_k,
               const __grid_constant__ CUtensorMap tmap_v, const __nv_bfloat16* __restrict__ q,
               const uint8_t* __restrict__ k_scale, const uint8_t* __restrict__ v_scale,
               const int32_t* __restrict__ block_table, int max_pages, int num_pages,
               const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ cu_q, int B,
               int total_q, int max_q, int max_seq_len, int Hq, int Hkv, float scale_log2,
               float* __restrict__ ws_o, float* __restrict__ ws_ml, int maxC, int run,
               unsigned int* __restrict__ cnt, unsigned int* err) {
    using C = Cfg<D>;
    constexpr int NSLOT = C::NSLOT;
    constexpr int RP = RPW * NWG;
    constexpr int EPI = NQ * NWG;  // first epilogue warp (a multiple of 4: its lane quarter is 0)
    constexpr int SCHED = EPI + 4, K_WARP = EPI + 5, V_WARP = EPI + 6;
    constexpr int S_WARP = EPI + 7, PV_WARP = EPI + 8, COUNTER = EPI + 9, PREP = EPI + 10;
    constexpr int THREADS = kWarps<NWG> * 32;
    constexpr int NPREP = kWarps<NWG> - PREP;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    uint8_t* sQ = smem + C::Q_OFF;
    uint8_t* sP = smem + C::P_OFF;
    uint8_t* sK = smem + C::RING_OFF;
    uint8_t* sV = smem + C::V_OFF;
    uint8_t* sScale = smem + C::SCALE_OFF;
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
    uint64_t* k_empty = k_full + NSLOT;
    uint64_t* v_full = k_empty + NSLOT;
    uint64_t* v_empty = v_full + NSLOT;
    uint64_t* s_full = v_empty + NSLOT; // item k's scores are in S set k & 1
    uint64_t* s_empty = s_full + 2;     // ... and read by the softmax
    uint64_t* p_full = s_empty + 2;     // item k's P is written
    uint64_t* p_empty = p_full + 1;     // P V of item k has completed (MMA commit)
    uint64_t* o_full = p_empty + 1;     // item k's O (buffer k & 1) is complete (MMA commit)
    uint64_t* o_empty = o_full + 2;     // ... and read out by the epilogue warps
    uint64_t* xs_bar = o_empty + 2;     // item k's row sums and maxima are in xs[k & 3]
    uint64_t* q_full = xs_bar + 4;      // item k's scale bytes (set k & 1) and its Q are there
    uint64_t* st_bar = q_full + 2;      // item k's partials are stored by the epilogue warps
    uint64_t* c_done = st_bar + 2;      // ... and counted
    uint64_t* d_full = c_done + 2;      // item k's descriptor is in items[k % NDESC]
    uint64_t* d_used = d_full + NDESC;  // the K copies of item k are issued (k % LEAD)
    uint64_t* drain = d_used + LEAD;    // [2]: S issuer, P V issuer
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
    ItemSlot* items = reinterpret_cast<ItemSlot*>(smem + C::DESC_OFF);
    float* xs = reinterpret_cast<float*>(smem + C::XS_OFF);  // [4][NQ + 1][QR]
    float* q_fac = xs + 4 * (NQ + 1) * QR;                   // [2][QR]
    float* x_max = q_fac + 2 * QR;                           // [2][NQ][QR]
    int* prefix = reinterpret_cast<int*>(smem + C::MISC_OFF);  // [B + 1]
    int* scale_odd = prefix + MAX_BATCH + 1;  // [2 sets][2]: a scale byte from kOddScale on
    volatile int* abort_flag = reinterpret_cast<volatile int*>(scale_odd + 4);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = Hq / Hkv;
    const int TQ = QR / G;  // tokens of a query tile

    if (warp == S_WARP) {
        tmem_alloc(tmem_slot, TMEM_COLS);
        tmem_relinquish();
    }
    // every barrier, one per thread (one thread after the other took longer than the rest of the
    // prologue): arrivals of its phase
    static_assert(C::NBARS <= THREADS, "a thread per barrier");
    if (tid < C::NBARS) {
        uint64_t* bar = k_full + tid;
        int count = 1;
        if ((bar >= s_empty && bar < p_empty) || (bar >= xs_bar && bar < q_full)) count = NQ * NWG;
        if (bar >= o_empty && bar < xs_bar) count = 4;
        if (bar >= q_full && bar < st_bar) count = NPREP;
        if (bar >= st_bar && bar < c_done) count = 4;
        mbar_init(bar, uint32_t(count));
        fence_barrier_init();
    }
    if (tid == 0) *abort_flag = 0;
    if (tid < 4) scale_odd[tid] = 0;
    // With item counters the grid before this one is the call's own counter reset, which
    // waited for everything before it: the inputs are final, and only the counters need the
    // counter's wait (see attention.cu).  Without, this grid waits for the previous one.
    if (!cnt) {
        pdl_wait();
        pdl_trigger();
    }
    const unsigned long long wait_ns = wait_budget_ns(err);
    for (int b = tid; b < B; b += THREADS) {
        const SeqInfo si = seq_info(seq_lens, cu_q, b);
        const bool ok = seq_ok(si, max_q, max_seq_len, total_q);
        if (!ok) latch_error(err, kErrDeviceArg);
        // units: runs of up to `run` chunks of one query tile and KV head
        const int chunks = (si.L + CHUNK - 1) >> CHUNK_LOG2;
        prefix[b + 1] = ok ? ((chunks + run - 1) / run) * ((si.qb + TQ - 1) / TQ) * Hkv : 0;
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
    // tile g's slot of a ring has landed (flip 0) or is free again (flip 1)
    auto wait_slot = [&](uint64_t* bars, uint32_t g, uint32_t flip) {
        return wait(&bars[g % NSLOT], ((g / NSLOT) & 1u) ^ flip);
    };
    // the descriptor of item k; npages = 0 after the last one (or when the wait ran out)
    auto item_at = [&](int k) {
        Item it;
        it.npages = 0;
        if (wait(&d_full[k % NDESC], uint32_t(k / NDESC) & 1u)) {
            const uint4* src = reinterpret_cast<const uint4*>(&items[k % NDESC].it);
            const uint4 a = src[0], b = src[1];
            it = Item{int(a.x), int(a.y), int(a.z), int(a.w),
                      int(b.x), int(b.y), int(b.z), int(b.w)};
        }
        return it;
    };

    if (warp == SCHED) {
        // ----------------------------------------------------------------- scheduler
        // Finds this CTA's items and publishes them, at most LEAD ahead of the K copies.  Item
        // j takes the descriptor of item j - NDESC.  When the K copies of item x are issued,
        // the scores of item x - NSLOT at least are done, so the softmax has finished the item
        // three before that, the epilogue has read the O of the item two before that one, and
        // the counter is at most two items behind it: no reader is as far back as NDESC.
        // A unit's chunks follow one another, so they share a Q tile, which is split once.
        const int total = prefix[B];
        int w = blockIdx.x, b = 0, left = 0, qgen = 0, last_t0 = -1, last_h = -1;
        Item it;
        for (int j = 0;; ++j) {
            if (!wait(&d_used[j % LEAD], (uint32_t(j / LEAD) & 1u) ^ 1u)) break;
            if (left > 0) {  // the unit's next chunk
                it.key0 += CHUNK;
            } else {         // the next unit that has a chunk its tile sees
                for (; w < total && left == 0; w += gridDim.x) {
                    int lo = 0, hi = B;
                    while (hi - lo > 1) {
                        const int mid = (lo + hi) >> 1;
                        if (prefix[mid] <= w) lo = mid; else hi = mid;
                    }
                    b = lo;
                    const SeqInfo si = seq_info(seq_lens, cu_q, lo);
                    const int U = (si.qb + TQ - 1) / TQ;
                    const int r = w - prefix[lo];
                    const int cu = r / Hkv;
                    const int c = cu / U, u = cu - c * U;
                    it.h = r - cu * Hkv;
                    it.L = si.L;
                    it.key0 = c * run * CHUNK;
                    it.t0 = si.t0 + u * TQ;
                    it.ntok = min(TQ, si.qb - u * TQ);
                    it.pos0 = si.L - si.qb + u * TQ;
                    const int keys = it.pos0 + it.ntok - it.key0;
                    left = keys <= 0 ? 0 : min(run, (keys + CHUNK - 1) >> CHUNK_LOG2);
                }
                if (left > 0 && (it.t0 != last_t0 || it.h != last_h)) {
                    ++qgen;
                    last_t0 = it.t0;
                    last_h = it.h;
                }
            }
            it.bq = 4 * b + (qgen & 1);
            it.npages = 0;
            if (left > 0) {
                it.npages = min(CHUNK / PAGE, (it.pos0 + it.ntok - it.key0 + PAGE - 1) / PAGE);
                --left;
            }
            ItemSlot* slot = &items[j % NDESC];
            int phys = -1;
            if (lane < it.npages) {
                const int pidx = it.key0 / PAGE + lane;
                if (pidx < max_pages) phys = block_table[int64_t(b) * max_pages + pidx];
                if (phys < 0 || phys >= num_pages) {
                    phys = -1;
                    latch_error(err, kErrDeviceArg);
                }
            }
            if (lane < CHUNK / PAGE) slot->phys[lane] = phys;
            if ((__ballot_sync(0xffffffffu, phys >= 0) & 0xffu) == 0xffu &&
                it.key0 + CHUNK - 1 <= it.pos0)
                it.bq |= 2;
            if (lane == 0) slot->it = it;
            __syncwarp();
            if (lane == 0) mbar_arrive(&d_full[j % NDESC]);
            if (it.npages == 0) break;
        }
        if (!ok && lane == 0) give_up();
    } else if (warp == K_WARP || warp == V_WARP) {
        // ----------------------------------------------------------------- producers
        // One warp copies K, one V: the copies' issue takes about as long as their data.  The
        // whole warp runs the loop; one elected lane issues.
        const bool is_k = warp == K_WARP;
        const CUtensorMap* map = is_k ? &tmap_k : &tmap_v;
        uint64_t* full = is_k ? k_full : v_full;
        uint64_t* empty = is_k ? k_empty : v_empty;
        uint8_t* ring = is_k ? sK : sV;
        if (lane == 0) tma_prefetch_desc(map);
        // blocks of one query tile read K and V once; wider ones read them again from L2
        const uint64_t policy = max_q <= TQ ? l2_policy_evict_first() : l2_policy_evict_last();
        uint32_t g = 0;
        for (int item = 0; ok; ++item) {
            const Item it = item_at(item);
            if (it.npages == 0) break;
            const int phys_l = lane < CHUNK / PAGE ? items[item % NDESC].phys[lane] : -1;
            for (int i = 0; i < it.npages; i += TPAGES, ++g) {
                if (!wait_slot(empty, g, 1u)) break;
                int phys[TPAGES], there = 0;
#pragma unroll
                for (int k = 0; k < TPAGES; ++k) {
                    phys[k] = __shfl_sync(0xffffffffu, phys_l, i + k);
                    there += phys[k] >= 0 ? 1 : 0;
                }
                if (elect_one()) {
                    const int slot = int(g % NSLOT);
                    if (there)
                        mbar_arrive_expect_tx(&full[slot], uint32_t(there * C::PAGE_BYTES));
                    else
                        mbar_arrive(&full[slot]);
#pragma unroll
                    for (int k = 0; k < TPAGES; ++k)
                        if (phys[k] >= 0)
                            tma_load_2d_hint(ring + slot * C::SLOT_BYTES + k * C::PAGE_BYTES, map,
                                             &full[slot], 0, (phys[k] * Hkv + it.h) * PAGE, policy);
                }
                __syncwarp();
            }
            if (is_k && lane == 0) mbar_arrive(&d_used[item % LEAD]);
        }
        if (!ok) {
            if (lane == 0) give_up();
            // copies already issued land before the CTA exits (bounded)
            for (uint32_t k = 1; k <= NSLOT && k <= g; ++k) {
                const uint32_t p = g - k;
                mbar_wait(&full[p % NSLOT], (p / NSLOT) & 1u, nullptr, 100000000ull);
            }
        }
    } else if (warp == S_WARP) {
        // ------------------------------------------------- S^T = K (Q_hi + Q_lo)^T
        constexpr uint32_t idesc = idesc_e4m3(TK, QR, 0, 0);
        const uint64_t q_desc0 = umma_smem_desc(smem_addr(sQ), 16, C::SBO, C::LAYOUT);
        const uint64_t k_desc0 = umma_smem_desc(smem_addr(sK), 16, C::SBO, C::LAYOUT);
        uint32_t g = 0;
        for (int item = 0; ok; ++item) {
            const Item it = item_at(item);
            const int nt = tiles_of(it.npages);
            if (nt == 0) break;
            const int buf = item & 1, qbuf = it.bq & 1;
            const uint32_t par = uint32_t(item >> 1) & 1u;
            if (!wait(&q_full[buf], par) || !wait(&s_empty[buf], par ^ 1u)) break;
            for (int i = 0; i < nt; ++i, ++g) {
                if (!wait_slot(k_full, g, 0u)) break;
                tc_fence_after_sync();
                if (elect_one()) {
                    const uint64_t k_desc = k_desc0 + uint64_t(((g % NSLOT) * C::SLOT_BYTES) >> 4);
                    const uint64_t q_desc = q_desc0 + uint64_t((qbuf * C::Q_BYTES) >> 4);
                    const uint32_t d = tmem_base + uint32_t(S_COL + (buf * NT + i) * QR);
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) {  // head dims 32k .. 32k+31: +32 B
                        tc_mma_f8(d, k_desc + uint64_t(k * 2), q_desc + uint64_t(k * 2), idesc,
                                  k != 0 ? 1u : 0u);
                        tc_mma_f8(d, k_desc + uint64_t(k * 2),
                                  q_desc + uint64_t((C::Q_PIECE >> 4) + k * 2), idesc, 1u);
                    }
                    tc_commit(&k_empty[g % NSLOT]);  // K of the tile is no longer read
                    if (i == nt - 1) tc_commit(&s_full[buf]);
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
        const uint64_t v_desc0 = umma_smem_desc(smem_addr(sV), 16, C::SBO, C::LAYOUT);
        const uint64_t p_desc0 = umma_smem_desc(smem_addr(sP), 16, 512, 4);
        uint32_t g = 0;
        for (int item = 0; ok; ++item) {
            const int nt = tiles_of(item_at(item).npages);
            if (nt == 0) break;
            const int ob = item & 1;
            // the O buffer of this item was read out for item-2
            if (!wait(&o_empty[ob], (uint32_t(item >> 1) & 1u) ^ 1u) ||
                !wait(p_full, uint32_t(item) & 1u))
                break;
            for (int i = 0; i < nt; ++i, ++g) {
                if (!wait_slot(v_full, g, 0u)) break;
                tc_fence_after_sync();
                if (elect_one()) {
                    const uint64_t v_desc = v_desc0 + uint64_t(((g % NSLOT) * C::SLOT_BYTES) >> 4);
                    const uint64_t p_desc = p_desc0 + uint64_t((i * C::P_BYTES) >> 4);
                    const uint32_t d = tmem_base + uint32_t(O_COL + ob * 2 * QR);
#pragma unroll
                    for (int k = 0; k < TK / 32; ++k)  // keys 32k .. 32k+31
                        tc_mma_f8(d, v_desc + uint64_t(k * 32 * D / 16),
                                  p_desc + uint64_t(k * 32 * 2 * QR / 16), idesc,
                                  (i | k) != 0 ? 1u : 0u);
                    tc_commit(&v_empty[g % NSLOT]);
                    if (i == nt - 1) {
                        tc_commit(p_empty);
                        tc_commit(&o_full[ob]);
                    }
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) give_up();
        if (elect_one()) tc_commit(&drain[1]);
        __syncwarp();
        mbar_wait(&drain[1], 0, nullptr, 100000000ull);
    } else if (warp >= PREP) {
        // ------------------------------------------------- scale bytes and Q of an item
        // As soon as the softmax has read item k - 2's from the same buffers.
        const int pw = warp - PREP;
        int last_q = -1;
        for (int item = 0; ok; ++item) {
            const Item it = item_at(item);
            if (it.npages == 0) break;
            const int buf = item & 1, qbuf = it.bq & 1;
            // scale bytes of page pp of every tile: lanes 0..15 read K's as words, 16..31 V's
            uint32_t sw[2 / NPREP][NT];
            uint32_t odd = 0;
#pragma unroll
            for (int n = 0; n < 2 / NPREP; ++n) {
                const int pp = NPREP == 2 ? pw : n;
                const uint32_t* src =
                    reinterpret_cast<const uint32_t*>(lane < 16 ? k_scale : v_scale);
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const int phys = items[item % NDESC].phys[i * TPAGES + pp];
                    sw[n][i] = 0x7f7f7f7fu;
                    if (phys >= 0)
                        sw[n][i] = src[(int64_t(phys) * Hkv + it.h) * (PAGE / 4) + (lane & 15)];
                }
            }
            bool free = false;
            const int rows = qbuf != last_q ? RP : 0;  // (else the item before has this Q tile)
            last_q = qbuf;
#pragma unroll 1
            for (int r0 = pw * 8; r0 < rows; r0 += NPREP * 8) {
                // four neighbouring lanes split one query row
                constexpr int PER = D / 4;  // elements per lane
                const int r = r0 + (lane >> 2), part = lane & 3;
                const int j = r / G;
                uint4 v[PER / 8];
#pragma unroll
                for (int n = 0; n < PER / 8; ++n) v[n] = make_uint4(0, 0, 0, 0);
                if (j < it.ntok && r < TQ * G) {
                    const __nv_bfloat16* src =
                        q + (int64_t(it.t0 + j) * Hq + it.h * G + (r - j * G)) * D + part * PER;
#pragma unroll
                    for (int n = 0; n < PER / 8; ++n)
                        v[n] = *reinterpret_cast<const uint4*>(src + n * 8);
                }
                uint32_t amax = 0;  // of bf16 magnitudes, which order as their bits
#pragma unroll
                for (int n = 0; n < PER / 8; ++n) {
                    const uint32_t x[4] = {v[n].x, v[n].y, v[n].z, v[n].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        amax = max(amax, max(x[e] & 0x7fffu, (x[e] >> 16) & 0x7fffu));
                }
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                // s = 7 - floor(log2(amax)), held where 2^s and 2^-s are normal
                const int s = max(-120, min(120, 134 - int(amax >> 7)));
                const float mul = __uint_as_float(uint32_t(127 + s) << 23);
                // item k-2's scores are read: the Q before the last, in this buffer, is not needed
                if (!free) {
                    if (!wait(&s_empty[buf], (uint32_t(item >> 1) & 1u) ^ 1u)) break;
                    free = true;
                }
                uint8_t* hi = sQ + qbuf * C::Q_BYTES;
                uint8_t* lo = hi + C::Q_PIECE;
#pragma unroll
                for (int n = 0; n < PER / 16; ++n) {
                    uint32_t h[4], l[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint4& src = v[2 * n + (e >> 1)];
                        const uint32_t x0 = e & 1 ? src.z : src.x, x1 = e & 1 ? src.w : src.y;
                        const uint32_t a = split_q(x0, mul), b = split_q(x1, mul);
                        h[e] = __byte_perm(a, b, 0x5410);
                        l[e] = __byte_perm(a, b, 0x7632);
                    }
                    const uint32_t at = swz_row<D>(r, part * (PER / 16) + n);
                    *reinterpret_cast<uint4*>(hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
                    *reinterpret_cast<uint4*>(lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
                }
                // a query with an infinity or NaN scores NaN throughout
                if (part == 0)
                    q_fac[qbuf * QR + r] =
                        amax >= 0x7f80u ? __int_as_float(0x7fc00000)
                                        : scale_log2 * __uint_as_float(uint32_t(127 - s) << 23);
            }
            if (!ok) break;
            if (!free && !wait(&s_empty[buf], (uint32_t(item >> 1) & 1u) ^ 1u)) break;
            // stored key by key, the tiles' four bytes in one word
#pragma unroll
            for (int n = 0; n < 2 / NPREP; ++n) {
                const int pp = NPREP == 2 ? pw : n;
#pragma unroll
                for (int i = 0; i < NT; ++i)  // a byte from kOddScale on?
                    odd |= sw[n][i] & (sw[n][i] << 1) & (sw[n][i] << 2) & 0x80808080u;
                const uint32_t a = __byte_perm(sw[n][0], sw[n][1], 0x5140);
                const uint32_t b = __byte_perm(sw[n][2], sw[n][3], 0x5140);
                const uint32_t c = __byte_perm(sw[n][0], sw[n][1], 0x7362);
                const uint32_t d = __byte_perm(sw[n][2], sw[n][3], 0x7362);
                *reinterpret_cast<uint4*>(sScale + buf * C::SCALE_BYTES + (lane >> 4) * (TK * NT) +
                                          (pp * PAGE + (lane & 15) * 4) * NT) =
                    make_uint4(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632),
                               __byte_perm(c, d, 0x5410), __byte_perm(c, d, 0x7632));
            }
            odd = __any_sync(0xffffffffu, odd != 0) ? 1u : 0u;
            if (lane == 0) scale_odd[buf * 2 + pw] = int(odd);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[buf]);
        }
        if (!ok && lane == 0) give_up();
    } else if (warp == COUNTER) {
        // ----------------------------------------------------------------- counter
        // Counts each stored item for its (sequence, KV head), which the merge waits on: the
        // epilogue warps release their stores to the CTA, the fence takes them to the GPU.
        if (cnt) {
            pdl_wait();  // the counters are zeroed
            pdl_trigger();
            for (int item = 0; ok; ++item) {
                const Item it = item_at(item);
                if (it.npages == 0) break;
                if (!wait(&st_bar[item & 1], uint32_t(item >> 1) & 1u)) break;
                if (lane == 0) {
                    asm volatile("fence.acq_rel.gpu;" ::: "memory");
                    atomicAdd(cnt + (it.bq >> 2) * Hkv + it.h, 1u);
                    mbar_arrive(&c_done[item & 1]);
                }
                __syncwarp();
            }
            if (!ok && lane == 0) give_up();
        }
    } else if (warp >= EPI && warp < EPI + 4) {
        // ------------------------------------------------------------------- epilogue
        const int ew = warp - EPI;  // tensor-memory lane quarter
        // O^T: lane = head dim (M = 128), or dims 16 ew .. 16 ew + 15 in lanes 0..15 (M = 64)
        const int d = D == 128 ? ew * 32 + lane : ew * 16 + lane;
        const bool mine = D == 128 || lane < 16;
        for (int item = 0; ok; ++item) {
            const Item it = item_at(item);
            if (it.npages == 0) break;
            const int ob = item & 1;
            const uint32_t par = uint32_t(item >> 1) & 1u;
            // rows (token j, head gg) are stored when their token sees the chunk; row r = lane's
            // place among the partials, or -1
            const int j = lane / G;
            const int c = it.key0 >> CHUNK_LOG2;
            const bool store = j < it.ntok && lane < TQ * G && it.pos0 + j >= it.key0;
            const int64_t idx =
                store ? (int64_t(it.t0 + j) * Hq + int64_t(it.h) * G + (lane - j * G)) * maxC + c
                      : -1;
            if (!wait(&xs_bar[item & 3], uint32_t(item >> 2) & 1u) || !wait(&o_full[ob], par))
                break;
            tc_fence_after_sync();
            if (ew == 0 && store) {
                const float* x = xs + (item & 3) * ((NQ + 1) * QR);
                const float l =
                    ((x[lane] + x[QR + lane]) + x[2 * QR + lane]) + x[3 * QR + lane];
                *reinterpret_cast<float2*>(ws_ml + idx * 2) = make_float2(x[NQ * QR + lane], l);
            }
            const uint32_t ta =
                tmem_base + (uint32_t(32 * ew) << 16) + uint32_t(O_COL + ob * 2 * QR);
            constexpr int PART = RP < 16 ? RP : 16;
#pragma unroll
            for (int r0 = 0; r0 < RP; r0 += PART) {
                uint32_t vh[PART], vl[PART];
                tmem_cols(ta + r0, vh);
                tmem_cols(ta + QR + r0, vl);
                if (r0 + PART == RP) {  // O is read
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&o_empty[ob]);
                }
#pragma unroll
                for (int k = 0; k < PART; ++k) {
                    const int64_t at = __shfl_sync(0xffffffffu, idx, r0 + k);
                    if (at >= 0 && mine)
                        ws_o[at * D + d] =
                            fmaf(__uint_as_float(vl[k]), 1.f / kLoScale, __uint_as_float(vh[k]));
                }
            }
            // (item-2 is counted: the counter never falls a phase of st_bar behind)
            if (cnt && !wait(&c_done[ob], par ^ 1u)) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(&st_bar[ob]);
        }
        if (!ok && lane == 0) give_up();
    } else {
        // ------------------------------------------------------------------- softmax
        // Group wg owns query rows wg * RPW .. of every tile; each thread one key.
        const int wg = warp / NQ, wq = warp % NQ;
        const int key = wq * 32 + lane;
        const int row0 = wg * RPW;
        const uint32_t lane_base = uint32_t(32 * wq) << 16;
        uint32_t g = 0;
        for (int item = 0;; ++item) {
            const int ob = item & 1;
            const uint32_t ipar = uint32_t(item >> 1) & 1u;
            const Item it = item_at(item);
            if (it.npages > 0) wait(&q_full[ob], ipar);
            if (it.npages == 0) {  // no more items, or this warp gave up: one barrier either way
                if (!ok && lane == 0) give_up();
                if (group_or(1 + wg, !ok)) ok = false;
                break;
            }
            const int nt = tiles_of(it.npages);
            float2 f[RPW / 2];
#pragma unroll
            for (int r = 0; r < RPW; r += 4) {
                const float4 x =
                    *reinterpret_cast<const float4*>(q_fac + (it.bq & 1) * QR + row0 + r);
                f[r / 2] = make_float2(x.x, x.y);
                f[r / 2 + 1] = make_float2(x.z, x.w);
            }
            // t of this thread's keys (one of each tile), and each row's maximum
            const uint32_t* sc =
                reinterpret_cast<const uint32_t*>(sScale + ob * C::SCALE_BYTES) + key;
            const uint32_t kw = sc[0], vw = sc[TK];
            const bool odd = (scale_odd[ob * 2] | scale_odd[ob * 2 + 1]) != 0;
            const bool all_seen = (it.bq & 2) != 0;  // every row sees every key
            wait(&s_full[ob], ipar);
            tc_fence_after_sync();
            uint32_t sv[NT][RPW];
            tmem_tiles(tmem_base + lane_base + uint32_t(S_COL + ob * NT * QR + row0), sv);
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_empty[ob]);
            // the scales of this thread's keys: 2^x, y, 2^-y
            float ka[NT], vb[NT], vinv[NT], t[NT][RPW], mx[RPW];
            auto score = [&](int i, int r) {
                const float2 s2 = make_float2(__uint_as_float(sv[i][r]),
                                              __uint_as_float(sv[i][r + 1]));
                return fma2(mul2(s2, make_float2(ka[i], ka[i])), f[r / 2],
                            make_float2(vb[i], vb[i]));
            };
            if (!odd) {
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const int up = 23 - 8 * i;  // byte i to the exponent's place
                    const uint32_t ks = up > 0 ? kw << (up & 31) : kw >> (-up & 31);
                    const uint32_t vs = up > 0 ? vw << (up & 31) : vw >> (-up & 31);
                    // (a byte of 0 is 2^-127)
                    ka[i] = __uint_as_float(max(ks & 0x7f800000u, 0x00400000u));
                    // 2^23 + byte, less 2^23 + 127
                    vb[i] = __uint_as_float(__byte_perm(vw, 0x4b000000u, 0x7650 | i)) - 8388735.f;
                    vinv[i] = __uint_as_float(0x7f000000u - (vs & 0x7f800000u));
#pragma unroll
                    for (int r = 0; r < RPW; r += 2) {
                        const float2 x = score(i, r);
                        t[i][r] = x.x;
                        t[i][r + 1] = x.y;
                    }
                }
            } else {
                // Products of codes are below 2^24: times a key scale below 2^97 they are finite.
                // With a larger one t is formed as 2^24 * (t * 2^-24), whose factors are finite
                // where t is, and whose rounding is the same.
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const uint32_t ks = (kw >> (8 * i)) & 0xffu, vs = (vw >> (8 * i)) & 0xffu;
                    const bool big = ks >= kOddScale;
                    ka[i] = e8m0(ks) * (big ? 0x1p-24f : 1.f);
                    vb[i] = vs == 255 ? __int_as_float(0x7fc00000)
                                      : float(int(vs) - 127) * (big ? 0x1p-24f : 1.f);
                    vinv[i] = e8m0_inv(vs);
#pragma unroll
                    for (int r = 0; r < RPW; r += 2) {
                        const float2 x = score(i, r);
                        t[i][r] = x.x * (big ? 0x1p24f : 1.f);
                        t[i][r + 1] = x.y * (big ? 0x1p24f : 1.f);
                    }
                }
            }
            // causal mask: row r (token r / G) sees the key that is `ahead` of the first token
            // when r / G >= ahead; none sees a key past the sequence's end or of an invalid page
            uint32_t dead = 0;  // a bit per tile
            if (!all_seen) {
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const int kp = it.key0 + i * TK + key, ahead = kp - it.pos0;
                    const bool live =
                        items[item % NDESC].phys[i * TPAGES + key / PAGE] >= 0 && kp < it.L;
                    if (!live) {
                        dead |= 1u << i;
                        vinv[i] = 0.f;
                    }
                    const int first = live ? max(0, ahead) * G : QR;
#pragma unroll
                    for (int r = 0; r < RPW; ++r)
                        t[i][r] = row0 + r >= first ? t[i][r] : -INFINITY;
                }
            }
#pragma unroll
            for (int r = 0; r < RPW; ++r)
                mx[r] = fmaxf(fmax3(t[0][r], t[1][r], t[2][r]), t[3][r]);
            // the rows' maxima over the group's four warps
#pragma unroll
            for (int r = 0; r < RPW; ++r) mx[r] = warp_max(mx[r]);
            float* xm = x_max + ob * (NQ * QR) + row0;
            if (lane == 0) {
#pragma unroll
                for (int r = 0; r < RPW; r += 4)
                    *reinterpret_cast<float4*>(xm + wq * QR + r) =
                        make_float4(mx[r], mx[r + 1], mx[r + 2], mx[r + 3]);
                if (!ok) give_up();
            }
            if (group_or(1 + wg, !ok)) {
                ok = false;
                break;
            }
            float m[RPW], l[RPW];
#pragma unroll
            for (int r = 0; r < RPW; r += 4) {
                const float4 x0 = *reinterpret_cast<const float4*>(xm + 0 * QR + r);
                const float4 x1 = *reinterpret_cast<const float4*>(xm + 1 * QR + r);
                const float4 x2 = *reinterpret_cast<const float4*>(xm + 2 * QR + r);
                const float4 x3 = *reinterpret_cast<const float4*>(xm + 3 * QR + r);
                m[r] = fmax3(fmax3(x0.x, x1.x, x2.x), x3.x, kLowest) - kHeadroom;
                m[r + 1] = fmax3(fmax3(x0.y, x1.y, x2.y), x3.y, kLowest) - kHeadroom;
                m[r + 2] = fmax3(fmax3(x0.z, x1.z, x2.z), x3.z, kLowest) - kHeadroom;
                m[r + 3] = fmax3(fmax3(x0.w, x1.w, x2.w), x3.w, kLowest) - kHeadroom;
            }
#pragma unroll
            for (int r = 0; r < RPW; ++r) l[r] = 0.f;
            // P's buffers are free once P V of item-1 has completed
            wait(p_empty, (uint32_t(item) & 1u) ^ 1u);
            uint8_t* pbuf = sP + (row0 & 15);
#pragma unroll
            for (int i = 0; i < NT; ++i) {  // (tiles past the item's last write zeros)
                const float vi = vinv[i];
                uint32_t hi[RPW / 4], lo[RPW / 4];
#pragma unroll
                for (int r = 0; r < RPW; r += 4) {
                    float p[4];
#pragma unroll
                    for (int k = 0; k < 4; k += 2) {
                        const float2 e = add2(make_float2(t[i][r + k], t[i][r + k + 1]),
                                              make_float2(-m[r + k], -m[r + k + 1]));
                        p[k] = ex2(e.x);
                        p[k + 1] = ex2(e.y);
                        const float2 s2 = fma2(make_float2(p[k], p[k + 1]), make_float2(vi, vi),
                                               make_float2(l[r + k], l[r + k + 1]));
                        l[r + k] = s2.x;
                        l[r + k + 1] = s2.y;
                    }
                    const uint32_t a = split_p(p[0], p[1]), b = split_p(p[2], p[3]);
                    hi[r / 4] = __byte_perm(a, b, 0x5410);
                    lo[r / 4] = __byte_perm(a, b, 0x7632);
                }
                uint8_t* ph = pbuf + i * C::P_BYTES + swz_row<64>(key, row0 >> 4);
                uint8_t* pl = pbuf + i * C::P_BYTES + swz_row<64>(key, 2 + (row0 >> 4));
                if (RPW == 8) {
                    *reinterpret_cast<uint2*>(ph) = make_uint2(hi[0], hi[RPW / 4 - 1]);
                    *reinterpret_cast<uint2*>(pl) = make_uint2(lo[0], lo[RPW / 4 - 1]);
                } else {
                    *reinterpret_cast<uint32_t*>(ph) = hi[0];
                    *reinterpret_cast<uint32_t*>(pl) = lo[0];
                }
            }
            // V rows past the sequence's end or of an invalid page are zeroed, so that
            // unwritten codes (NaN) cannot reach O through 0 * v
            if (wg == 0 && __any_sync(0xffffffffu, dead != 0)) {
                for (int i = 0; i < nt; ++i) {
                    wait_slot(v_full, g + i, 0u);
                    if (ok && ((dead >> i) & 1u)) {
                        uint4* vr = reinterpret_cast<uint4*>(
                            sV + ((g + i) % NSLOT) * C::SLOT_BYTES + key * D);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) vr[k] = make_uint4(0, 0, 0, 0);
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(p_full);
            // the warp's row sums (and the maxima) for the epilogue.  The buffer held those of
            // item-4, and the barrier its phase: P V of item-1 has completed, so that of item-2
            // has begun, for which the epilogue had read O and the sums of item-4.
            const float sum = sum_lanes<RPW>(l, lane);
            if (ok) {
                float* x = xs + (item & 3) * ((NQ + 1) * QR) + row0;
                if (wq == 0 && lane == 0) {
#pragma unroll
                    for (int r = 0; r < RPW; r += 4)
                        *reinterpret_cast<float4*>(x + NQ * QR + r) =
                            make_float4(m[r], m[r + 1], m[r + 2], m[r + 3]);
                }
                if (lane % (32 / RPW) == 0) x[wq * QR + lane / (32 / RPW)] = sum;
                __syncwarp();
                if (lane == 0) mbar_arrive(&xs_bar[item & 3]);
            }
            g += uint32_t(nt);
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
    // Chunks of a unit (consecutive items of a CTA with one Q tile, split once): as many as
    // leave each CTA eight units or more, so that the dealing stays even -- where the items'
    // turn-around is what binds (64 sequences of 8,196 keys, blocks of 8: 245 us with runs, 276
    // without; one-token blocks at head_dim 64, 16,388 keys: 178 and 194; 512 tokens after 65,028:
    // 1.56 ms and 1.96).  One-token blocks at head_dim 128 are bound by memory and keep the finer
    // dealing (ragged batch of 64: 230 us without, 246 with).
    int run = 1;
    auto units = [&](int r) { return a.batch * ((maxC + r - 1) / r) * tiles * a.hkv; };
    while (run < 8 && (D == 64 || RPW * NWG > 4) && units(2 * run) >= 8 * int64_t(dev.num_sms))
        run *= 2;
    float* ws_o = static_cast<float*>(workspace);
    float* ws_ml = ws_o + a.total_q * a.hq * int64_t(maxC) * D;
    // The merge of a (sequence, KV head) may start when its chunks are counted, beside the chunks
    // of others: 64 sequences of 8,196 keys, blocks of 8, 245 us with counts and 280 without; two
    // of 65,540 keys 65.9 and 67.8.  The counters' reset costs a launch, which a call of few items
    // does not earn back (one of 65,540 keys 39.5 and 38.2).  With few query rows there is little
    // to merge (64 at head_dim 64 205 with and 178 without), and the tiles of a wide block are not
    // counted apart: there the merge waits for the whole grid.
    unsigned int* cnt = nullptr;
    if (tiles == 1 && RPW * NWG > 4) {
        cnt = attn_item_counters(a, workspace, CHUNK_LOG2);
        cudaError_t e = launch_attn_count_reset(cnt, int(a.batch * a.hkv), stream);
        if (e != cudaSuccess) return e;
    }
    cudaError_t e = launch_pdl(
        kern, dim3(grid), dim3(kWarps<NWG> * 32), Cf::SMEM, stream, tk, tv,
        static_cast<const __nv_bfloat16*>(q), static_cast<const uint8_t*>(k_scale),
        static_cast<const uint8_t*>(v_scale), a.block_table, int(a.max_pages), int(a.num_pages),
        a.seq_lens, a.cu_q, int(a.batch), int(a.total_q), int(a.max_q), int(a.max_seq_len),
        int(a.hq), int(a.hkv), scale * kLog2e, ws_o, ws_ml, maxC, run, cnt, dev.err_word);
    if (e != cudaSuccess) return e;
    return launch_attn_merge(a, workspace, CHUNK_LOG2, out, lse, cnt, dev.err_word, stream,
                             Shape{});
}

}  // namespace

cudaError_t launch_attention_q8(const DeviceInfo& dev, const void* q, const PagedArgs& a,
                                const void* k_scale, const void* v_scale, float scale, void* out,
                                float* lse, void* workspace, cudaStream_t stream) {
    // softmax groups of four or eight query rows for those of the fullest tile
    const int64_t G = a.hq / a.hkv, TQ = QR / G;
    const int64_t rows = (a.max_q < TQ ? a.max_q : TQ) * G;
    auto run = [&](auto f) {
        return f(dev, q, a, k_scale, v_scale, scale, out, lse, workspace, stream);
    };
    if (a.head_dim == 64)
        return run(rows <= 4    ? launch_q8_t<64, 4, 1>
                   : rows <= 8  ? launch_q8_t<64, 4, 2>
                   : rows <= 16 ? launch_q8_t<64, 8, 2>
                                : launch_q8_t<64, 8, 4>);
    return run(rows <= 4    ? launch_q8_t<128, 4, 1>
               : rows <= 8  ? launch_q8_t<128, 4, 2>
               : rows <= 16 ? launch_q8_t<128, 8, 2>
                            : launch_q8_t<128, 8, 4>);
}

}  // namespace bi

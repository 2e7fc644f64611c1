// sage_extend.cu -- attention of several new tokens a sequence over the paged key-value cache: a prompt's
// chunk, a conversation's next turn, drafted tokens.
//
//   s_tk = q_t . K_k / sqrt(d),  O_t = sum_k softmax(s_t)_k V_k,  L_t = log sum_k exp s_tk,
//   over the slots k <= start[b] + t  (token t's own slot is start[b] + t),  t < count[b].
//
// Work.  4 d multiply-adds a query head, new token and visible slot against a cache that is read once a
// tile of rows: bound by the tensor cores from a few hundred rows a kv head on.  The rows of a kv head, its G query
// heads times T tokens, are consecutive in Q (B,Hq,T,d): a tile is 128 consecutive ones, whatever heads
// they belong to, so that grouped heads fill tiles when T is small, and row r's token is r mod T.
// (Few rows, up to kExtendFewRows a kv head, go to the one-token kernel's warps instead: sage_decode.cu.)
//
// One CTA takes two tiles (256 rows) of one kv head and walks the slots in steps of 128:
//   warps 8-11  load K's rows by page, widen codes to 16 bits, and store them as swizzled operands, two
//               stages; warps 12-15 V's.  8-bit rows come through registers, one step ahead; 16-bit
//               rows by cp.async.
//   warp 16     issues every MMA: S_t = Q_t K^T and O_t += P_t V, M = 128, N = 128 and d
//   warps 0-3   softmax of tile 0, warps 4-7 of tile 1: a thread a row.  P goes back to TMEM over S,
//               as the A operand of the second product, 64 slots at a time, so that their product runs
//               beside the other 64's softmax; O stays in TMEM over the whole walk and is rescaled only where a
//               row's reference, its largest logit when it last moved, lags too far behind.
// Measured (INT8 with scales of blocks / bf16 pool, 2 sequences of 2048 new tokens over 6144, 32 query heads on 8, d = 128):
// 508 / 387 us, 947 / 1243 TFLOP/s of the 1903 that a library product reaches.  A step of 128 slots takes 3050 cycles over a
// bf16 pool where the MMAs alone take 2540 (their operands fill shared memory's bandwidth): what is left is the chain
// from a tile's last P to its next S.  In 8 bits 3900: the loaders share schedulers and instruction cache with the softmax.
// And the last wave: these 512 CTAs of 50 to 64 steps are 192 steps an SM, and the SM that ends last has 224.
// TMEM: columns 256 t + [0, 128) S_t and P_t, 256 t + 128 + [0, d) O_t.
//
// Scales.  Codes are exact in fp16 and bf16, so a logit x is acc * (sK log2(e) / sqrt(d)); with one scale a
// block that is one factor for 16 or more columns.  q = 2^(x - m) goes into l, and p' = q sV feeds the second product,
// where m follows the running maximum of x + log2 sV, so that the largest p' stays near 1 whatever the scales are.  For
// m a scale counts as at least 2^-60, so that q stays below 2^80 (and as at most 2^20 in bf16, whose p' can grow): l
// then loses nothing above 2^-46 of a row's largest weight, and no scale, however small or not finite, reaches it.
// A scale a row is multiplied on; scales of blocks go into the exponent with x, in the rare steps with one outside
// [2^-60, 2^20] or with hidden slots by a pass over S of their own.
// Roundings: p' is rounded to Q's type, half a step of the output's own type each, and they average over the slots: bf16
// (8 bits, down to 2^-100 of the row's largest), or fp16, the running maximum's at 2^11, so that all 11 bits are there
// down to 2^-25 of it and below in steps of 2^-35.  A row whose weight lies on slots of little value can be made of
// those.  Where what fp16 may have lost (half a step a slot, times the largest V) exceeds 2^-12 of a row's largest
// output, its CTA walks the slots twice more, under the references that the first walk left: once for the small p',
// 2^24 times, and once for the others.  That takes 3.3 times as long where every row needs it (chunk over an fp16 pool
// 390 -> 1288 us); the largest V of a 16-bit pool is found beside the first walk.
// K's codes meet Q in fp16 (4 of them take 5 or 2 instructions, to bf16 8 or 10), Q in bf16 under a power of two a row.
// Sums, statistics and O are float32.
//
// Up to 128 rows a kv head there is one tile: its steps go to the two softmax groups in turn, so that one's MMAs
// run beside the other's softmax here too, and the two parts are joined like ranges.
// Few CTAs are given more to do by cutting the slots into up to kExtMaxSplits ranges; a second kernel joins
// their O, m and l in order, so results do not depend on the order in which CTAs run.
//
// What a row does not see never reaches it.  Logits of hidden slots are replaced (not added to); hidden
// V rows are multiplied by 0, so a V that is not finite in the steps that only some rows see is set
// to 0 in the operand, and added at the end to the rows that do see it.
#include "sage_kv.cuh"
#include "sage_decode.h"

namespace sage {

__device__ unsigned int g_ext_err = 0;      // bounded waits that gave up
__device__ unsigned int g_ext_index = 0;    // 1: a page, start or count was out of range

namespace ext {

constexpr int kThreads = 640;
constexpr int kKeyWarp = 8, kValueWarp = 12;    // 8 .. 11, 12 .. 15
constexpr int kMmaWarp = 16;                // (17 .. 19 are idle)
// Launched at 96 registers a thread (640 x 96 = 61440): 256 x 128 + 256 x 80 + 128 x 64 = 61440.
constexpr uint32_t kRegsSoftmax = 128, kRegsLoad = 80, kRegsControl = 64;
constexpr int kRows = 256;                  // of a CTA
constexpr int kStep = 128;                  // slots a step
constexpr int kExtMaxSplits = 16;
constexpr int kWalks = 3;                   // over the slots: one, and where fp16 may have lost too much two more
constexpr int kMinSteps = 8;                // of a range of slots
constexpr int kCtaSteps = 6;                // what a CTA costs besides its steps, in steps (512 tokens over 65536: 9 ranges 229 us, 14 242)

struct Args {
    KvView c;
    const void *Q;
    void *O;
    float *L;
    const int *start, *count;
    int T, rows;                            // new tokens; rows of a kv head (heads a kv head times T)
    int tiles, splits;                      // CTAs a kv head's rows and slots are cut into
    int order_heads, order_tiles;           // T a multiple of 256: heads a kv head, tiles a head; else 0
    float sl2;                              // log2(e) / sqrt(d)
    float *part_O, *part_ml;                // splits > 1 or one tile: (items, splits, 256, d), (items, splits, 256, 2)
};

// Barriers of one walk over the slots.
struct Bars {
    uint64_t k_full[2], k_free[2], v_full[2], v_free[2], mma_done;
    uint64_t s_full[2], p_full[2][2], o_full[2], o_done[2];   // p_full[tile][half of the step]; o_full: a half's PV, o_done: a tile's last
};

template <int D>
struct Smem {
    alignas(1024) uint8_t q[2][D / 64][128 * 128];   // [tile][64 channels][row][128 bytes], 128-byte swizzle
    alignas(1024) uint8_t k[2][D / 64][128 * 128];   // two stages: step j's rows in stage j & 1
    alignas(1024) uint8_t v[2][D / 64][128 * 128];
    // of step j in place j & 3 (a place is written again when the step before the last has been read):
    // factor of the products, V's scale and its log2 as the reference follows it, a slot or a group of 16 slots each;
    // the scales' reciprocals, a group
    alignas(16) float kc[4][128], sv[4][128], lv[4][128], rv[4][8];
    float qs[256];                                   // the rows' factors of Q (8-bit pools, Q in bf16)
    uint32_t holes[4];                               // groups of 16 slots whose page is none; kOdd: scales of V out of the ordinary
    uint64_t q_full;
    Bars bars[kWalks];
    uint32_t tmem_base, v_most;                      // v_most: the largest |V| of the CTA's slots, its bits (16-bit pools, fp16)
    int abort_flag, not_finite, ask, again;
};

// log2 of V's scale as the reference follows it.  Held to 2^-60, so that the probabilities before their scales stay
// below 2^80, and in bf16, where P itself can grow, to 2^20, so that they stay above 2^-126 where they count.  A scale of 0
// counts as 2^-60 too (its codes are 0): a slot of no value, however large its weight, does not hold the reference above
// those that have one.  A scale that is not finite reaches O by itself.
constexpr float kLeastScale = 0x1p-60f, kMostScale = 0x1p20f;
template <bool BF16>
__device__ __forceinline__ float followed_log2(float sv) {
    const float x = fabsf(sv);
    if (!(x < INFINITY)) return 0.0f;
    const float l = x < kLeastScale ? -60.0f : log2f(x);
    return BF16 ? fminf(l, 20.0f) : l;
}
// Scales of groups of 16 go into the exponent as they are where all of a step are 0 or from 2^-60 to 2^20.
constexpr uint32_t kOdd = 4u;                        // in the word of a step's holes
__device__ __forceinline__ bool ordinary(float sv) { return sv == 0.0f || (sv >= kLeastScale && sv <= kMostScale); }

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        return pack_half2(lo, hi);
    }
}

// To fp16, 65504 at most (a NaN stays one).
__device__ __forceinline__ uint32_t pack_finite(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// max(|a|, |b|) of two pairs of fp16, under some sign
__device__ __forceinline__ uint32_t larger_halves(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Place of 16-byte chunk c of row r in an operand of 64-channel parts.
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    return static_cast<uint32_t>((c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ void sts128(uint32_t at, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 lds128u(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}

// 16 codes of each of N rows (r, r + STEP, ..), chunk c of 16 of them, to chunks 2 c and 2 c + 1 of the operand;
// lanes of the second 64 channels store theirs the other way round, so that a row's eight stores meet eight
// different 16-byte bank groups.
template <bool BF16, bool FP8, int N, int STEP>
__device__ __forceinline__ void store_codes(uint32_t to, const uint4 (&from)[N], int r, int c) {
    const int flip = c >> 2 & 1;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        uint4 lo, hi;
        widen4<BF16, FP8>(from[i].x, lo.x, lo.y);
        widen4<BF16, FP8>(from[i].y, lo.z, lo.w);
        widen4<BF16, FP8>(from[i].z, hi.x, hi.y);
        widen4<BF16, FP8>(from[i].w, hi.z, hi.w);
        sts128(to + chunk_at(r + i * STEP, 2 * c + flip), flip ? hi : lo);
        sts128(to + chunk_at(r + i * STEP, 2 * c + 1 - flip), flip ? lo : hi);
    }
}

// Bounded wait of a warp until K of a step has been stored.  S of the step says so too: by then K's barrier may have
// gone on to the phase after the next, whose parity is that of one not yet over.
__device__ __forceinline__ bool wait_either(uint64_t *k_full, uint32_t k_parity, uint64_t *s_full, uint32_t s_parity, volatile int *abort_flag) {
    bool ok = true;
    const unsigned long long t0 = clock64();
    for (uint32_t it = 1; !mbar_try_wait(k_full, k_parity) && !mbar_try_wait(s_full, s_parity); ++it) {
        if ((it & 15u) == 0u && (*abort_flag || clock64() - t0 > SAGE_WAIT_CYCLES)) {
            if (!*abort_flag) {
                *abort_flag = 1;
                atomicOr(&g_ext_err, 1u | (10u << 8));
            }
            ok = false;
            break;
        }
    }
    return __all_sync(0xffffffffu, ok);
}

// What a sequence brings: its first new slot, its new tokens and its slots in all, held to what exists.
struct Seq {
    int start, count, len;
};
__device__ __forceinline__ Seq sequence(const Args &a, int b) {
    Seq s;
    s.start = kv_len(a.c, a.start, b, &g_ext_index);
    s.count = a.T;
    if (a.count) {
        s.count = __ldg(a.count + b);
        if (s.count < 0 || s.count > a.T) {
            atomicOr(&g_ext_index, 1u);
            s.count = s.count < 0 ? 0 : a.T;
        }
    }
    s.len = s.count > 0 ? s.start + s.count : 0;
    if (s.len > a.c.cap) {
        atomicOr(&g_ext_index, 1u);
        s.len = a.c.cap;
    }
    return s;
}
// the slots that row r sees
__device__ __forceinline__ int row_limit(const Args &a, const Seq &s, int r) {
    const int t = r % a.T;
    return r < a.rows && t < s.count ? min(s.start + t + 1, s.len) : 0;
}
// the first and the last token of rows [r0, r1) of a kv head that exist
__device__ __forceinline__ int first_token(const Args &a, int r0, int r1) {
    const int t0 = r0 % a.T;
    return t0 + (r1 - r0) > a.T ? 0 : t0;
}
__device__ __forceinline__ int last_token(const Args &a, int r0, int r1) {
    const int t0 = r0 % a.T;
    return t0 + (r1 - r0) > a.T ? a.T - 1 : t0 + (r1 - r0) - 1;
}
// slots that any row of [r0, r0 + n) sees
__device__ __forceinline__ int tile_end(const Args &a, const Seq &s, int r0, int n) {
    const int r1 = min(r0 + n, a.rows);
    if (r0 >= r1 || s.len == 0) return 0;
    const int t = min(last_token(a, r0, r1), s.count - 1);
    // (a range of one head's tokens that all lie behind the count)
    if (first_token(a, r0, r1) >= s.count) return 0;
    return min(s.start + t + 1, s.len);
}

// K's or V's rows, step after step, by 128 threads; first Q's rows of a tile, 0 by K's threads and 1 by V's.
template <int D, bool BF16, int SC, bool FP8>
struct Loader {
    const Args &a;
    Smem<D> &s;
    Bars &z;
    int walk;
    int b, hk, j0, j1, kv_end, mixed, tid, r0, n_q;
    size_t out0;

    static constexpr int ROW = SC ? D : 2 * D;                       // bytes of a row
    static constexpr int CPR = ROW / 16, RPI = 128 / CPR, ITS = 128 / RPI;   // 16-byte chunks a row, rows at a time
    static constexpr uint32_t kNone = 0xFFFFFFFFu;                   // (a pool in memory has fewer rows)

    // this warp's part of an operand is stored
    __device__ __forceinline__ void done(uint64_t *bar) const {
        fence_view_async_shared();
        __syncwarp();
        if ((tid & 31) == 0) mbar_arrive(bar);
    }
    // the stage of step j0 + i has been read
    __device__ __forceinline__ bool free_of(uint64_t *bar, int i) const {
        return i < 2 || mbar_wait_warp(&bar[i & 1], ((i >> 1) - 1) & 1, &s.abort_flag, &g_ext_err, 6);
    }

    // zeros behind the last row
    __device__ __forceinline__ void query(int t) const {
        const uint4 *Q = static_cast<const uint4 *>(a.Q) + out0 * (D / 8);
        constexpr int QC = D / 8, QR = 128 / QC;
        if (j0 < n_q) {
#pragma unroll 8
            for (int r = tid / QC; r < 128; r += QR) {
                const int row = r0 + 128 * t + r;
                uint4 w = row < a.rows ? __ldg(Q + static_cast<size_t>(row) * QC + tid % QC) : make_uint4(0u, 0u, 0u, 0u);
                if constexpr (BF16 && SC != 0) {
                    // to fp16 under a power of two a row: the largest value lands in [2^14, 2^15); the 8 bits of others are
                    // all there down to 2^-31 of it (fp16's steps end at 2^-24), and from 2^-39 on they are gone
                    float2 f[4];
                    float mx = 0.0f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        f[e] = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162 *>(&w)[e]);
                        mx = max3f(mx, fabsf(f[e].x), fabsf(f[e].y));
                    }
#pragma unroll
                    for (int o = 1; o < QC; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    // exponent of the largest, held to [-100, 127] so that both factors are normal
                    const int e0 = max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -100);
                    const float up = __uint_as_float(static_cast<uint32_t>(14 - e0 + 127) << 23);
                    w = make_uint4(pack_half2(f[0].x * up, f[0].y * up), pack_half2(f[1].x * up, f[1].y * up),
                                   pack_half2(f[2].x * up, f[2].y * up), pack_half2(f[3].x * up, f[3].y * up));
                    if (tid % QC == 0) s.qs[128 * t + r] = __uint_as_float(static_cast<uint32_t>(e0 - 14 + 127) << 23);
                }
                sts128(smem_u32(s.q[t][0]) + chunk_at(r, tid % QC), w);
            }
        }
        done(&s.q_full);
    }

    template <bool VALUES>
    __device__ __forceinline__ void run() const {
        const int lane = tid & 31;
        const int rr = tid / CPR, cc = tid % CPR;                    // rows rr + i RPI, chunk cc
        const void *pool = VALUES ? a.c.V : a.c.K;
        uint64_t *full = VALUES ? z.v_full : z.k_full, *free = VALUES ? z.v_free : z.k_free;
        // Pages are asked for two steps ahead, by lane g of every warp (mod 8) for its step's group g of 16 slots,
        // and become the group's first row of the pool, kNone where it has no page, a step ahead.
        const int *table = a.c.table + static_cast<size_t>(b) * a.c.max_pages;
        int page = 0;
        uint32_t base = kNone;
        bool plain = false;                                          // every group has its page and all of its slots
        auto look = [&](int j) {
            const int slot = j * kStep + (lane & 7) * 16;
            page = slot < kv_end ? __ldg(table + kv_page_of(a.c, slot)) : 0;
        };
        auto find = [&](int j) {
            const int slot = j * kStep + (lane & 7) * 16;
            base = kNone;
            if (slot < kv_end) {
                if (static_cast<unsigned>(page) < static_cast<unsigned>(a.c.pages)) base = static_cast<uint32_t>(kv_row(a.c, page, hk, slot));
                else atomicOr(&g_ext_index, 1u);
            }
            plain = (j + 1) * kStep <= kv_end && __all_sync(0xffffffffu, base != kNone);
        };
        // row r of the step: its row of the pool (whole warps call it)
        auto row_of = [&](int r) -> uint32_t {
            const uint32_t first = __shfl_sync(0xffffffffu, base, r >> 4);
            return first == kNone ? kNone : first + (r & 15);
        };
        // ---- scales, by K's threads, one step ahead
        float sk = 0.0f, sv = 0.0f;
        bool hole = false;
        auto load_scales = [&](int j) {
            // a thread a slot (SC = 1), or threads 0 .. 7 a group of 16 each; of a 16-bit pool the holes alone
            const int slot = j * kStep + (SC == 1 ? tid : (lane & 7) * 16);
            const uint32_t r = SC == 1 ? row_of(tid) : base;
            sk = sv = 0.0f;
            hole = slot < kv_end && r == kNone && (SC == 1 || lane < 8);
            if (SC != 0 && r != kNone && slot < kv_end && (SC == 1 || tid < 8)) {
                sk = __ldg(a.c.sK + (r >> a.c.block_shift));
                sv = __ldg(a.c.sV + (r >> a.c.block_shift));
            }
        };
        auto store_scales = [&](int i) {
            const int at = i & 3;
            if (SC == 1 || (SC == 2 && tid < 8)) {
                s.kc[at][tid] = sk * a.sl2;
                s.sv[at][tid] = sv;
                s.lv[at][tid] = followed_log2<BF16>(sv);
                if (SC == 2) s.rv[at][tid] = 1.0f / (sv == 0.0f ? kLeastScale : sv);   // (not read where a scale is odd)
            }
            if constexpr (SC == 1) {
                // slots 32 w .. of warp w: two groups
                const uint32_t h = __ballot_sync(0xffffffffu, hole);
                if (lane == 0) {
                    const uint32_t two = (h & 0xFFFFu ? 1u : 0u) | (h >> 16 ? 2u : 0u);
                    reinterpret_cast<uint8_t *>(&s.holes[at])[tid >> 5] = static_cast<uint8_t>(two);
                }
            } else if (tid < 32) {
                const uint32_t h = __ballot_sync(0xffffffffu, hole);
                const bool odd = SC == 2 && __any_sync(0xffffffffu, !ordinary(sv));
                // groups 2 w and 2 w + 1 in byte w, as above
                if (lane == 0) s.holes[at] = (h & 3u) | ((h >> 2) & 3u) << 8 | ((h >> 4) & 3u) << 16 | ((h >> 6) & 3u) << 24 | (odd ? kOdd : 0u);
            }
        };
        if constexpr (SC != 0) {
            // 8-bit rows, half a step (64 rows) at a time, a step ahead
            constexpr int HALF = ITS / 2;
            uint4 x[2][HALF];
            auto load = [&](int j, const int h) {
                uint32_t rows[HALF];
#pragma unroll
                for (int i = 0; i < HALF; ++i) rows[i] = row_of(64 * h + rr + i * RPI);
                const uint4 *from = static_cast<const uint4 *>(pool) + cc;
                if (plain) {
#pragma unroll
                    for (int i = 0; i < HALF; ++i) x[h][i] = __ldg(from + static_cast<size_t>(rows[i]) * CPR);
                } else {
#pragma unroll
                    for (int i = 0; i < HALF; ++i) {
                        x[h][i] = make_uint4(0u, 0u, 0u, 0u);
                        if (rows[i] != kNone && j * kStep + 64 * h + rr + i * RPI < kv_end) x[h][i] = __ldg(from + static_cast<size_t>(rows[i]) * CPR);
                    }
                }
            };
            auto store = [&](int j, const int h) {
                const int st = (j - j0) & 1;
                if constexpr (VALUES && FP8) {
                    if (j >= mixed) {
#pragma unroll
                        for (int y = 0; y < HALF; ++y) {
                            uint32_t *w = &x[h][y].x;
                            uint32_t bad = 0;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t m = not_finite_mask<BF16, true>(w[e]);
                                w[e] &= ~m;
                                bad |= m;
                            }
                            if (bad) s.not_finite = 1;
                        }
                    }
                }
                store_codes<VALUES && BF16, FP8, HALF, RPI>(smem_u32(VALUES ? s.v[st][0] : s.k[st][0]), x[h], 64 * h + rr, cc);
            };
            look(j0);
            find(j0);
            look(j0 + 1);
            if (!VALUES) load_scales(j0);
            load(j0, 0);
            load(j0, 1);
            if (walk == 0) query(VALUES);
#pragma unroll 1
            for (int j = j0; j < j1; ++j) {
                const int i = j - j0;
                if (!free_of(free, i)) break;
                store(j, 0);
                if (!VALUES) store_scales(i);
                if (j + 1 < j1) {
                    find(j + 1);
                    look(j + 2);
                    if (!VALUES) load_scales(j + 1);
                    load(j + 1, 0);
                }
                store(j, 1);
                done(&full[i & 1]);
                if (j + 1 < j1) load(j + 1, 1);
            }
        } else {
            auto load = [&](int j) {
                const uint32_t to = smem_u32(VALUES ? s.v[(j - j0) & 1][0] : s.k[(j - j0) & 1][0]);
                // this thread has ITS / 8 rows of each of the 8 groups
                const uint8_t *from[8];
                bool there[8];
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    const uint32_t row = row_of(16 * g + rr);
                    there[g] = row != kNone;
                    from[g] = static_cast<const uint8_t *>(pool) + (row == kNone ? 0 : static_cast<size_t>(row) * ROW + cc * 16);
                }
                if (plain) {
#pragma unroll
                    for (int i = 0; i < ITS; ++i) cp_async16(to + chunk_at(rr + i * RPI, cc), from[i * RPI / 16] + i * RPI % 16 * ROW);
                } else {
#pragma unroll
                    for (int i = 0; i < ITS; ++i) {
                        const bool is = there[i * RPI / 16] && j * kStep + rr + i * RPI < kv_end;
                        cp_async16(to + chunk_at(rr + i * RPI, cc), is ? from[i * RPI / 16] + i * RPI % 16 * ROW : static_cast<const uint8_t *>(pool), is);
                    }
                }
                cp_commit();
            };
            look(j0);
            find(j0);
            look(j0 + 1);
            load(j0);
            if (!VALUES) load_scales(j0);
            if (walk == 0) query(VALUES);
            [[maybe_unused]] uint32_t most = 0;                      // |V|, pairs of fp16
            for (int j = j0; j < j1; ++j) {
                const int i = j - j0, st = i & 1;
                if (!VALUES) store_scales(i);
                cp_wait<0>();
                if (VALUES && j >= mixed) {                          // the chunks this thread has copied itself
#pragma unroll 4
                    for (int y = 0; y < ITS; ++y) {
                        const uint32_t at = smem_u32(s.v[st][0]) + chunk_at(rr + y * RPI, cc);
                        uint4 w = lds128u(at);
                        const uint32_t m0 = not_finite_mask<BF16, false>(w.x), m1 = not_finite_mask<BF16, false>(w.y);
                        const uint32_t m2 = not_finite_mask<BF16, false>(w.z), m3 = not_finite_mask<BF16, false>(w.w);
                        if (m0 | m1 | m2 | m3) {
                            sts128(at, make_uint4(w.x & ~m0, w.y & ~m1, w.z & ~m2, w.w & ~m3));
                            s.not_finite = 1;
                        }
                    }
                }
                done(&full[st]);
                if (j + 1 < j1) {
                    find(j + 1);
                    look(j + 2);
                    if (!free_of(free, i + 1)) break;
                    load(j + 1);
                    if (!VALUES) load_scales(j + 1);
                }
                if constexpr (VALUES && !BF16) {
                    // the largest |V|, from the chunks this thread has copied itself, while the next step's are on their way
                    if (walk == 0) {
#pragma unroll 4
                        for (int y = 0; y < ITS; ++y) {
                            const uint4 w = lds128u(smem_u32(s.v[st][0]) + chunk_at(rr + y * RPI, cc));
                            most = larger_halves(larger_halves(most, w.x), larger_halves(larger_halves(w.y, w.z), w.w));
                        }
                    }
                }
            }
            if constexpr (VALUES && !BF16) {
                if (walk == 0) atomicMax(&s.v_most, min(max(most & 0x7FFFu, most >> 16 & 0x7FFFu), 0x7BFFu));
            }
            cp_wait<0>();                                            // no copy outlives the CTA's shared memory
        }
    }
};

// SC: 0 a 16-bit pool, 1 a scale a row, 2 a scale a block
template <int D, bool BF16, int SC, bool FP8>
__global__ void __launch_bounds__(kThreads, 1) extend_kernel(const __grid_constant__ Args a) {
    extern __shared__ uint8_t smem_raw[];
    Smem<D> &s = *reinterpret_cast<Smem<D> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    // Results are referred to 2^kShift of the running maximum, which lags by up to 2^kSlack.
    constexpr float kSlack = 4.0f, kShift = BF16 ? 0.0f : 11.0f, kMost = BF16 ? 0x1p15f : 65504.0f;
    // fp16: below kLow a p' has fewer than 11 bits.
    [[maybe_unused]] constexpr float kLow = 0x1p-14f, kLift = 0x1p24f;
    const int warp = threadIdx.x >> 5;
    const int BH = a.c.B * a.c.H;
    // item: tiles with many slots first, all heads of a rank after one another
    int x = blockIdx.x;
    const int split = x % a.splits;
    x /= a.splits;
    // One tile of rows: its steps are dealt out to the two softmax groups in turn, as two parts of the slots.
    const bool dealt = a.rows <= 128;
    const int bh = x % BH, rank = x / BH, b = bh / a.c.H, hk = bh - b * a.c.H;
    const int tile = a.order_heads ? (rank % a.order_heads) * a.order_tiles + a.order_tiles - 1 - rank / a.order_heads : a.tiles - 1 - rank;
    const int r0 = tile * kRows;
    const Seq seq = sequence(a, b);
    int end[2];                                       // slots a tile's rows see
    end[0] = tile_end(a, seq, r0, 128);
    end[1] = dealt ? end[0] : tile_end(a, seq, r0 + 128, 128);
    const int all = (max(end[0], end[1]) + kStep - 1) / kStep;
    // (a short sequence is cut into fewer ranges than the plan has: what a CTA costs besides its steps is worth several)
    const int ranges = max(1, min(a.splits, all / kMinSteps));
    const int j0 = static_cast<int>(static_cast<long long>(all) * min(split, ranges) / ranges);
    const int j1 = static_cast<int>(static_cast<long long>(all) * min(split + 1, ranges) / ranges);
    const int kv_end = max(end[0], end[1]);
    int n_t[2];                                       // a tile's steps: j0 .. n_t - 1
    n_t[0] = min(j1, (end[0] + kStep - 1) / kStep);
    n_t[1] = min(j1, (end[1] + kStep - 1) / kStep);
    const size_t item = (static_cast<size_t>(bh) * a.tiles + tile) * a.splits + split;
    const size_t out0 = static_cast<size_t>(bh) * a.rows;            // first row of the kv head in O and L
    // steps from here on hold slots that not every row sees
    const int mixed = seq.len == 0 ? 0 : (seq.start + first_token(a, r0, min(r0 + kRows, a.rows)) + 1) / kStep;

    if (j0 >= j1) {                                   // nothing to see: the whole CTA alike
        const int row = threadIdx.x >> 1, half = threadIdx.x & 1;
        if (row >= kRows || (dealt ? (row & 127) : r0 + row) >= a.rows) return;
        if (a.splits > 1 || dealt) {
            if (half == 0) reinterpret_cast<float2 *>(a.part_ml)[item * kRows + row] = make_float2(-INFINITY, 0.0f);
        } else {
            uint4 *O = static_cast<uint4 *>(a.O) + (out0 + r0 + row) * (D / 8) + half * (D / 16);
#pragma unroll
            for (int c = 0; c < D / 16; ++c) O[c] = make_uint4(0u, 0u, 0u, 0u);
            if (half == 0) a.L[out0 + r0 + row] = -INFINITY;
        }
        return;
    }

    if (warp == kMmaWarp) {
        tmem_alloc(&s.tmem_base, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        s.abort_flag = 0;
        s.not_finite = 0;
        s.ask = s.again = 0;
        s.v_most = 0;
        mbar_init(&s.q_full, 8);
        for (int w = 0; w < (BF16 ? 1 : kWalks); ++w) {
            Bars &z = s.bars[w];
            mbar_init(&z.mma_done, 1);
            for (int t = 0; t < 2; ++t) {
                mbar_init(&z.k_full[t], 4);
                mbar_init(&z.k_free[t], 1);
                mbar_init(&z.v_full[t], 4);
                mbar_init(&z.v_free[t], 1);
                mbar_init(&z.s_full[t], 1);
                mbar_init(&z.p_full[t][0], 4);
                mbar_init(&z.p_full[t][1], 4);
                mbar_init(&z.o_full[t], 1);
                mbar_init(&z.o_done[t], 1);
            }
        }
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem_base;
    volatile int *abort_flag = &s.abort_flag;
    // step j is the (j - j0)th: stage (j - j0) & 1, its barriers' phase ((j - j0) >> 1) & 1
    // All warps of the CTA, each at the end of a walk, also of one that gave up: whether there is another one.
    // `bearable`: the largest |V| (8 bits: code) with which fp16 cannot have lost too much of this thread's row.
    auto all_warps = [&]() {
        __syncwarp();
        tc_fence_before();
        asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
        tc_fence_after();
    };
    auto another = [&](int walk, float bearable) -> bool {
        if constexpr (BF16) {
            return false;
        } else {
            if (walk + 1 == kWalks) return false;
            constexpr float top = SC == 0 ? 65504.0f : FP8 ? 448.0f : 127.0f;
            if (walk == 0 && bearable < top) s.ask = 1;
            all_warps();
            if (*static_cast<volatile int *>(&s.ask) == 0) return false;
            if (SC != 0 || walk > 0) return SC != 0 || *static_cast<volatile int *>(&s.again) != 0;
            const uint32_t v = *static_cast<volatile uint32_t *>(&s.v_most);
            if (bearable < __half2float(__ushort_as_half(static_cast<unsigned short>(v)))) s.again = 1;
            all_warps();
            return *static_cast<volatile int *>(&s.again) != 0;
        }
    };

    if (warp >= kMmaWarp) {
        regs_dec<kRegsControl>();
        for (int walk = 0;; ++walk) {
            Bars &z = s.bars[walk];
            if (warp == kMmaWarp && elect_one()) {
                // ------------------------------------------------------------------ MMA issuer
                constexpr uint32_t idS = idesc_f16(128, 128, BF16 && SC == 0, false, false);
                constexpr uint32_t idPV = idesc_f16(128, D, BF16, false, true);
                auto issue_s = [&](const int t, int st) {
                    const uint32_t q_addr = smem_u32(s.q[dealt ? 0 : t][0]), k_addr = smem_u32(s.k[st][0]);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk / 4) * 16384 + (kk % 4) * 32;
                        umma_ss(tmem + 256 * t, sdesc_sw128(q_addr + off, 16, 1024), sdesc_sw128(k_addr + off, 16, 1024), idS, kk > 0);
                    }
                    umma_commit(&z.s_full[t]);
                };
                // O_t += P_t V of a step, the tile's u-th, half by half
                auto issue_pv = [&](const int t, int u, int st, bool last) -> bool {
                    const uint32_t v_addr = smem_u32(s.v[st][0]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (!mbar_wait(&z.p_full[t][h], u & 1, abort_flag, &g_ext_err, 4)) return false;
                        tc_fence_after();
#pragma unroll
                        for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
                            umma_ts(tmem + 256 * t + 128, tmem + 256 * t + 8 * kk, sdesc_sw128(v_addr + 16 * kk * 128, 16384, 1024), idPV, (walk == 2 || u > 0 || kk > 0) ? 1u : 0u);
                        umma_commit(&z.o_full[t]);
                    }
                    if (last) umma_commit(&z.o_done[t]);
                    return true;
                };
                const int n = j1 - j0;
                bool ok = mbar_wait(&s.q_full, 0, abort_flag, &g_ext_err, 1) && mbar_wait(&z.k_full[0], 0, abort_flag, &g_ext_err, 2);
                // As in the forward kernel a tile's next S follows its PV in issue order and overwrites the P that the
                // PV reads: the tensor pipe runs MMAs in that order.
                if (dealt) {
                    // step i is group i & 1's: its S once that group's last PV has been issued
                    if (ok) {
                        tc_fence_after();
                        issue_s(0, 0);
                        umma_commit(&z.k_free[0]);
                    }
                    if (ok && n > 1 && (ok = mbar_wait(&z.k_full[1], 0, abort_flag, &g_ext_err, 2))) {
                        tc_fence_after();
                        issue_s(1, 1);
                        umma_commit(&z.k_free[1]);
                    }
                    auto step = [&](const int t, int i) -> bool {
                        if (!mbar_wait(&z.v_full[t], (i >> 1) & 1, abort_flag, &g_ext_err, 3)) return false;
                        if (!issue_pv(t, i >> 1, t, i + 2 >= n)) return false;
                        umma_commit(&z.v_free[t]);
                        if (i + 2 < n) {
                            if (!mbar_wait(&z.k_full[t], ((i + 2) >> 1) & 1, abort_flag, &g_ext_err, 2)) return false;
                            tc_fence_after();
                            issue_s(t, t);
                            umma_commit(&z.k_free[t]);
                        }
                        return true;
                    };
                    for (int i = 0; i < n && ok; i += 2) ok = step(0, i) && (i + 1 >= n || step(1, i + 1));
                } else {
                    if (ok) {
                        tc_fence_after();
                        if (j0 < n_t[0]) issue_s(0, 0);
                        if (j0 < n_t[1]) issue_s(1, 0);
                        umma_commit(&z.k_free[0]);
                    }
                    for (int j = j0; j < j1 && ok; ++j) {
                        const int i = j - j0, st = i & 1, nst = st ^ 1;
                        if (!(ok = mbar_wait(&z.v_full[st], (i >> 1) & 1, abort_flag, &g_ext_err, 3))) break;
                        // (the next K too, which has been there for long: nothing then stands between a tile's PV and its next S)
                        if (j + 1 < j1 && !(ok = mbar_wait(&z.k_full[nst], ((i + 1) >> 1) & 1, abort_flag, &g_ext_err, 2))) break;
                        auto tile_step = [&](const int t) -> bool {
                            if (j >= n_t[t]) return true;
                            if (!issue_pv(t, i, st, j + 1 == n_t[t])) return false;
                            if (t == 1 || j >= n_t[1]) umma_commit(&z.v_free[st]);
                            if (j + 1 < n_t[t]) issue_s(t, nst);
                            return true;
                        };
                        ok = tile_step(0) && tile_step(1);
                        if (!ok) break;
                        if (j + 1 < j1) umma_commit(&z.k_free[nst]);
                    }
                }
                // every MMA must have finished before the tensor memory is released
                umma_commit(&z.mma_done);
                mbar_wait_drain(&z.mma_done, 0, &g_ext_err, 5);
            }
            if (!another(walk, INFINITY)) break;
        }
    } else if (warp >= kKeyWarp) {
        regs_dec<kRegsLoad>();
        for (int walk = 0;; ++walk) {
            const Loader<D, BF16, SC, FP8> load{a, s, s.bars[walk], walk, b, hk, j0, j1, kv_end, mixed, static_cast<int>(threadIdx.x) & 127, r0,
                                                warp >= kValueWarp && dealt ? 0 : n_t[warp >= kValueWarp], out0};
            if (warp < kValueWarp) load.template run<false>();
            else load.template run<true>();
            if (!another(walk, INFINITY)) break;
        }
    } else {
        regs_inc<kRegsSoftmax>();
        // ------------------------------------------------------------------ softmax
        const int t = warp >> 2, quarter = warp & 3, lane = static_cast<int>(lane_id());
        const int row = (dealt ? 0 : 128 * t) + 32 * quarter + lane;
        const int limit = row_limit(a, seq, r0 + row);               // slots this row sees
        const int steps = t ? n_t[1] : n_t[0];
        const uint32_t lane_base = tmem_addr(tmem, 32 * quarter, 256 * t);
        float m = -INFINITY, l = 0.0f;                               // reference of O and l; l
        bool ok = steps <= j0 || mbar_wait_warp(&s.q_full, 0, abort_flag, &g_ext_err, 11);
        const float qs = BF16 && SC != 0 ? s.qs[row] : 1.0f;
        const int deal = dealt ? 1 : 0, first = dealt ? j0 + t : j0;
        const bool any = steps > first;
        Bars &z = s.bars[0];
        for (int j = first; j < steps && ok; j += 1 + deal) {
            const int i = j - j0, u = i >> deal, at = i & 3;         // u: of this group's steps
            // What the step's scales say is read ahead of its S, not a group at a time: shared memory answers slowly beside
            // the products' operands and the loaders' stores.
            if (!(ok = wait_either(&z.k_full[i & 1], (i >> 1) & 1, &z.s_full[t], u & 1, abort_flag))) break;
            const uint32_t holes = s.holes[at];
            const int seen = limit > 0 ? limit - j * kStep : kStep;  // of this step's slots, from the first; rows that are none take all
            const bool whole = holes == 0u && !__any_sync(0xffffffffu, seen < kStep);
            uint32_t raw[2][16];                                     // S, 16 slots a group, a group ahead
            // Logits of slots k .. k + 3 of the step (hidden ones: -inf), `scaled`: and V's scales on them.
            auto four = [&](const uint32_t *r, int k, float (&v)[4], auto scaled) {
                float4 kc = make_float4(a.sl2, a.sl2, a.sl2, a.sl2), lv = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if constexpr (SC == 1) {
                    kc = lds128(smem_u32(&s.kc[at][k]));
                    if (decltype(scaled)::value) lv = lds128(smem_u32(&s.lv[at][k]));
                } else if constexpr (SC == 2) {
                    kc.x = kc.y = kc.z = kc.w = s.kc[at][k / 16];
                    if (decltype(scaled)::value) lv.x = lv.y = lv.z = lv.w = s.lv[at][k / 16];
                }
                if constexpr (BF16 && SC != 0) {
                    kc.x *= qs; kc.y *= qs; kc.z *= qs; kc.w *= qs;
                }
                const f2 lo = fma2(f2{__uint_as_float(r[0]), __uint_as_float(r[1])}, f2{kc.x, kc.y}, f2{lv.x, lv.y});
                const f2 hi = fma2(f2{__uint_as_float(r[2]), __uint_as_float(r[3])}, f2{kc.z, kc.w}, f2{lv.z, lv.w});
                v[0] = lo.x; v[1] = lo.y; v[2] = hi.x; v[3] = hi.y;
                if (!whole) {
                    const bool none = (holes >> (k / 32 * 8 + (k / 16 & 1))) & 1u;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (none || k + e >= seen) v[e] = -INFINITY;
                }
            };
            [[maybe_unused]] float4 kc4, lv4, rv4, kc4n, lv4n, rv4n; // of this half and of the next
            if constexpr (SC == 2) {
                kc4 = lds128(smem_u32(&s.kc[at][0])); kc4n = lds128(smem_u32(&s.kc[at][4]));
                lv4 = lds128(smem_u32(&s.lv[at][0])); lv4n = lds128(smem_u32(&s.lv[at][4]));
                rv4 = lds128(smem_u32(&s.rv[at][0])); rv4n = lds128(smem_u32(&s.rv[at][4]));
                if (!whole) {                                        // prepare() puts the factors on
                    kc4 = kc4n = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
                    lv4 = lv4n = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                }
            }
            [[maybe_unused]] const float qs4 = whole ? qs : 1.0f;
            if (!(ok = mbar_wait_warp(&z.s_full[t], u & 1, abort_flag, &g_ext_err, 7))) break;
            tc_fence_after();
            // Half h of the step, 64 slots: p' = 2^(x - ref) sV, packed, and their l, sums of 2^(x - ref); the largest sum of
            // 16 p', or infinity.  Scales of groups go into the exponent, and a group's sum times its scale's reciprocal is
            // its part of l.
            uint32_t pk[32];
            float add;
            auto probabilities = [&](const int h, float ref, auto plain) -> float {
                constexpr bool PLAIN = decltype(plain)::value;       // no slot is hidden
                static_assert(PLAIN || SC != 2, "prepare() has been there");
                constexpr bool SCALED = SC == 1;                     // p' = q sV after q = 2^(x - ref)
                const uint32_t from = lane_base + 64 * h;
                float most = 0.0f;
                [[maybe_unused]] float sums[4];
                add = 0.0f;
                tmem_ld16(from, raw[0]);
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    tmem_wait_ld_regs(raw[g & 1]);
                    if (g < 3) tmem_ld16(from + 16 * (g + 1), raw[(g + 1) & 1]);
                    uint32_t(&r)[16] = raw[g & 1];
                    f2 sum{0.0f, 0.0f};
                    [[maybe_unused]] f2 l2{0.0f, 0.0f};
                    f2 f{a.sl2, a.sl2}, off{-ref, -ref};
                    if constexpr (SC == 2) {
                        f.x = f.y = (g == 0 ? kc4.x : g == 1 ? kc4.y : g == 2 ? kc4.z : kc4.w) * (BF16 ? qs4 : 1.0f);
                        off.x = off.y = (g == 0 ? lv4.x : g == 1 ? lv4.y : g == 2 ? lv4.z : lv4.w) - ref;
                    }
#pragma unroll
                    for (int k = 0; k < 16; k += 4) {
                        const int col = 64 * h + 16 * g + k;
                        f2 x[2];
                        [[maybe_unused]] float v[4];
                        if constexpr (PLAIN) {
                            [[maybe_unused]] float4 kc;
                            if constexpr (SC == 1) {
                                kc = lds128(smem_u32(&s.kc[at][col]));
                                if constexpr (BF16) {
                                    kc.x *= qs; kc.y *= qs; kc.z *= qs; kc.w *= qs;
                                }
                            }
                            x[0] = fma2(f2{__uint_as_float(r[k]), __uint_as_float(r[k + 1])}, SC == 1 ? f2{kc.x, kc.y} : f, off);
                            x[1] = fma2(f2{__uint_as_float(r[k + 2]), __uint_as_float(r[k + 3])}, SC == 1 ? f2{kc.z, kc.w} : f, off);
                        } else {
                            four(&r[k], col, v, std::false_type());
                            x[0] = add2(f2{v[0], v[1]}, off);
                            x[1] = add2(f2{v[2], v[3]}, off);
                        }
                        [[maybe_unused]] float4 sv;
                        if constexpr (SCALED) sv = lds128(smem_u32(&s.sv[at][col]));
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            f2 p{ex2_approx(x[e].x), ex2_approx(x[e].y)};
                            if constexpr (SCALED) {
                                l2 = add2(l2, p);
                                p = mul2(p, e ? f2{sv.z, sv.w} : f2{sv.x, sv.y});
                                if constexpr (!PLAIN) {              // (a hidden slot's scale may be anything)
                                    if (v[2 * e] == -INFINITY) p.x = 0.0f;
                                    if (v[2 * e + 1] == -INFINITY) p.y = 0.0f;
                                }
                            }
                            sum = add2(sum, p);
                            pk[8 * g + k / 2 + e] = pack2<BF16>(p.x, p.y);
                        }
                    }
                    const float both = sum.x + sum.y;
                    most = fmaxf(most, both);
                    if constexpr (SCALED) add += l2.x + l2.y;
                    else if constexpr (SC == 2) sums[g] = both;
                    else add += both;
                }
                if constexpr (SC == 2) {
                    const float rvs[4] = {rv4.x, rv4.y, rv4.z, rv4.w};
#pragma unroll
                    for (int g = 0; g < 4; ++g) add += sums[g] * rvs[g];
                }
                // (slots of little scale, far above the reference: it has to follow before their q overflows)
                if constexpr (SC == 1 && PLAIN) most = add > 0x1p90f ? INFINITY : most;
                return most;
            };
            // The reference follows half h's largest x + lv where it lags.  False: a wait gave up.
            auto follow = [&](const int h, float most) __attribute__((always_inline)) -> bool {
                float mx = -INFINITY;
#pragma unroll 1
                for (int g = 4 * h; g < 4 * h + 4; ++g) {
                    uint32_t(&r)[16] = raw[0];
                    tmem_ld16(lane_base + 16 * g, r);
                    tmem_wait_ld_regs(r);
#pragma unroll
                    for (int k = 0; k < 16; k += 4) {
                        float v[4];
                        four(r + k, 16 * g + k, v, std::true_type());
                        mx = max3f(mx, v[0], v[1]);
                        mx = max3f(mx, v[2], v[3]);
                    }
                }
                const bool moves = mx > m + kSlack || (most > kMost && mx > m);
                if (!__any_sync(0xffffffffu, moves)) return true;
                const float to = moves ? mx : m, alpha = moves ? ex2_approx(m - to) : 1.0f;    // (m = -inf: 0)
                m = to;
                l *= alpha;
                if (u == 0 && h == 0) return true;
                // The half before has to be in O.  (s_full says that of all halves of the steps before, so the
                // barrier is in the phase of the half before or in the next.)
                if (!mbar_wait_warp(&z.o_full[t], h ^ 1, abort_flag, &g_ext_err, 8)) return false;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                    uint32_t o[16];
                    tmem_ld16(lane_base + 128 + c, o);
                    tmem_wait_ld_regs(o);
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                    tmem_st16(lane_base + 128 + c, o);
                }
                tmem_wait_st();
                return true;
            };
            // Scales of groups, a step with hidden slots or odd scales: half h's logits take their factors here, a group at a
            // time, and go back to TMEM with V's scales on them, hidden ones as -inf, for the code of the whole steps.  Their part
            // of l.
            [[maybe_unused]] auto prepare = [&](const int h, float ref) __attribute__((always_inline)) -> float {
                float part = 0.0f;
#pragma unroll 1
                for (int g = 4 * h; g < 4 * h + 4; ++g) {
                    uint32_t(&r)[16] = raw[0];
                    tmem_ld16(lane_base + 16 * g, r);
                    tmem_wait_ld_regs(r);
                    const float sv = s.sv[at][g], lv = sv == 0.0f ? s.lv[at][g] : log2f(sv);
#pragma unroll
                    for (int k = 0; k < 16; k += 4) {
                        float v[4];
                        four(r + k, 16 * g + k, v, std::false_type());
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            part += ex2_approx(v[e] - ref);
                            r[k + e] = __float_as_uint(v[e] == -INFINITY ? v[e] : v[e] + lv);
                        }
                    }
                    tmem_st16(lane_base + 16 * g, r);
                }
                tmem_wait_st();
                return part;
            };
            // Most halves keep the reference that they find: the row's largest x then lies so little above it that no p'
            // exceeds kMost, which the sums of 16 show without a maximum.
            auto half_step = [&](const int h) __attribute__((always_inline)) -> bool {
                bool known = whole && !__any_sync(0xffffffffu, m == -INFINITY);
                float most = 0.0f;
                if constexpr (SC == 2) {
                    // (at most twice round)
                    float ref = m - kShift, part = 0.0f;
                    bool sure = false;
#pragma unroll 1
                    for (;;) {
                        if (known) {
                            most = probabilities(h, ref, std::true_type());
                            if (sure || !__any_sync(0xffffffffu, most > kMost)) break;
                        }
                        if (!follow(h, most)) return false;
                        ref = m == -INFINITY ? 0.0f : m - kShift;    // (nothing seen yet: all terms are 0)
                        if (!whole) part = prepare(h, ref);
                        known = sure = true;
                    }
                    l += whole ? add : part;
                } else {
                    if (known) {
                        most = probabilities(h, m - kShift, std::true_type());
                        known = !__any_sync(0xffffffffu, most > kMost);
                    }
                    if (!known) {
                        if (!follow(h, most)) return false;
                        const float ref = m == -INFINITY ? 0.0f : m - kShift;
                        if (whole) probabilities(h, ref, std::true_type());
                        else probabilities(h, ref, std::false_type());
                    }
                    l += add;
                }
                // ---- to TMEM over slots of S that have been read: 32 columns a half, behind which half 1 finds its own
                tmem_st32(lane_base + 32 * h, pk);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&z.p_full[t][h]);
                if constexpr (SC == 2) {
                    kc4 = kc4n;
                    lv4 = lv4n;
                    rv4 = rv4n;
                }
                return true;
            };
            // One copy of the code where the loaders widen codes beside it, whose instruction cache it shares; with a scale a
            // row, whose vectors are read at constant places, and over 16-bit pools two.
            if constexpr (SC == 2) {
#pragma unroll 1
                for (int h = 0; h < 2 && ok; ++h) ok = half_step(h);
            } else {
                ok = half_step(0) && half_step(1);
            }
            if (!ok) break;
        }
        if (ok && any) ok = mbar_wait_warp(&z.o_done[t], 0, abort_flag, &g_ext_err, 9);
        tc_fence_after();
        if constexpr (!BF16) {
            // Each p' was off by at most half of fp16's smallest step, 2^-25, besides its rounding.  Where that, times the
            // slots and the largest V, may be above 2^-12 of the row's largest output, the CTA walks twice more under the
            // references that it has now, for the p' below kLow, 2^24 times, and for the others.  (Loops of their own: within
            // the first walk's they cost it a fifth of its time.)
            float bearable = INFINITY;
            if (ok && any) {                                         // (whole warps)
                float top = 0.0f;
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                    uint32_t o[16];
                    tmem_ld16(lane_base + 128 + c, o);
                    tmem_wait_ld_regs(o);
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float x = fabsf(__uint_as_float(o[k]));
                        top = x < INFINITY ? fmaxf(top, x) : top;
                    }
                }
                const int slots = min(limit, j1 * kStep) - j0 * kStep;
                if (slots > 0) bearable = top * 0x1p13f / static_cast<float>(slots);
            }
            const float ref = m == -INFINITY ? 0.0f : m - kShift;
            for (int walk = 1; another(walk - 1, bearable); ++walk) {
                Bars &z = s.bars[walk];
                const float for_low = walk == 1 ? kLift : 0.0f, for_others = walk == 1 ? 0.0f : 1.0f;
                for (int j = first; j < steps && ok; j += 1 + deal) {
                    const int i = j - j0, u = i >> deal, at = i & 3;
                    if (!(ok = wait_either(&z.k_full[i & 1], (i >> 1) & 1, &z.s_full[t], u & 1, abort_flag))) break;
                    const uint32_t holes = s.holes[at];
                    const int seen = limit > 0 ? limit - j * kStep : kStep;
                    const bool whole = (holes & ~kOdd) == 0u && !__any_sync(0xffffffffu, seen < kStep);
                    if (!(ok = mbar_wait_warp(&z.s_full[t], u & 1, abort_flag, &g_ext_err, 12))) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < kStep; c += 32) {            // 32 slots at a time, two groups
                        uint32_t r[2][16], pk[16];
                        tmem_ld16(lane_base + c, r[0]);
                        tmem_ld16(lane_base + c + 16, r[1]);
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            tmem_wait_ld_regs(r[g]);
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const int col = c + 16 * g + k, place = SC == 1 ? col : col / 16;
                                float p = ex2_approx(fmaf(__uint_as_float(r[g][k]), SC == 0 ? a.sl2 : s.kc[at][place], -ref));
                                if constexpr (SC != 0) p *= s.sv[at][place];
                                r[g][k] = __float_as_uint(p);
                            }
                            if (!whole) {
#pragma unroll
                                for (int k = 0; k < 16; ++k)
                                    if (((holes >> (c / 4 + g)) & 1u) || c + 16 * g + k >= seen) r[g][k] = 0u;
                            }
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                // (rounded otherwise than in the first walk a p' can lie just above what that allowed; one that is
                                // infinite, of a scale that is, leaves a NaN)
                                const float p = __uint_as_float(r[g][k]), f = fabsf(p) < kLow ? for_low : for_others;
                                r[g][k] = __float_as_uint(SC == 0 ? p * f : fmaf(p, f, p * 0.0f));
                            }
#pragma unroll
                            for (int k = 0; k < 16; k += 2) pk[8 * g + k / 2] = pack_finite(__uint_as_float(r[g][k]), __uint_as_float(r[g][k + 1]));
                        }
                        tmem_st16(lane_base + c / 2, pk);
                        if (c % 64 == 32) {
                            tmem_wait_st();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&z.p_full[t][c / 64]);
                        }
                    }
                }
                if (ok && any) ok = mbar_wait_warp(&z.o_done[t], 0, abort_flag, &g_ext_err, 13);
                tc_fence_after();
                if (walk == 1 && ok && any) {                        // to the others' units
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t o[16];
                        tmem_ld16(lane_base + 128 + c, o);
                        tmem_wait_ld_regs(o);
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * (1.0f / kLift));
                        tmem_st16(lane_base + 128 + c, o);
                    }
                    tmem_wait_st();
                }
            }
        }
        const bool there = r0 + row < a.rows;
        const bool empty = limit == 0 || l == 0.0f;                  // saw nothing (a NaN is no 0)
        const bool part = a.splits > 1 || dealt;
        const size_t part_row = item * kRows + (dealt ? 128 * t : 0) + row;
        if (ok && !*abort_flag) {
            const float inv = empty ? 0.0f : 1.0f / l;
            if (there) {
                const float ref = m - kShift;
                if (part) reinterpret_cast<float2 *>(a.part_ml)[part_row] = empty ? make_float2(-INFINITY, 0.0f) : make_float2(ref, l);
                else a.L[out0 + r0 + row] = empty ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
            }
            // V values that are not finite and were taken out of the products: added for the rows that see them
            const bool fix = s.not_finite != 0;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = 0u;
                if (any) {
                    tmem_ld16(lane_base + 128 + c, *reinterpret_cast<uint32_t(*)[16]>(&o[0]));
                    tmem_ld16(lane_base + 128 + c + 16, *reinterpret_cast<uint32_t(*)[16]>(&o[16]));
                    tmem_wait_ld_regs(*reinterpret_cast<uint32_t(*)[16]>(&o[0]));
                    tmem_wait_ld_regs(*reinterpret_cast<uint32_t(*)[16]>(&o[16]));
                }
                float v[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) v[k] = empty ? 0.0f : __uint_as_float(o[k]) * (part ? 1.0f : inv);
                if (fix) {
                    const int *table = a.c.table + static_cast<size_t>(b) * a.c.max_pages;
                    for (int slot = max(j0, mixed) * kStep; slot < min(limit, j1 * kStep); ++slot) {
                        const int p = __ldg(table + kv_page_of(a.c, slot));
                        if (static_cast<unsigned>(p) >= static_cast<unsigned>(a.c.pages)) continue;
                        const size_t from = kv_row(a.c, p, hk, slot) * D + c;
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            float z = 0.0f;
                            if constexpr (SC != 0) {
                                if (FP8 && (static_cast<const uint8_t *>(a.c.V)[from + k] & 0x7Fu) == 0x7Fu) z = __int_as_float(0x7FC00000);
                            } else if constexpr (BF16) {
                                z = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.c.V)[from + k]);
                            } else {
                                z = __half2float(static_cast<const __half *>(a.c.V)[from + k]);
                            }
                            if (!(fabsf(z) < INFINITY)) v[k] += z;
                        }
                    }
                }
                if (!there) continue;
                if (part) {
                    if (empty) continue;                             // not read
                    float4 *to = reinterpret_cast<float4 *>(a.part_O + part_row * D + c);
#pragma unroll
                    for (int k = 0; k < 8; ++k) to[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                } else {
                    uint4 *to = static_cast<uint4 *>(a.O) + ((out0 + r0 + row) * D + c) / 8;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        to[k] = make_uint4(pack2<BF16>(v[8 * k], v[8 * k + 1]), pack2<BF16>(v[8 * k + 2], v[8 * k + 3]),
                                           pack2<BF16>(v[8 * k + 4], v[8 * k + 5]), pack2<BF16>(v[8 * k + 6], v[8 * k + 7]));
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// A row's parts under their common reference, in their order.  A warp a row.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) extend_join_kernel(const __grid_constant__ Args a) {
    const int lane = threadIdx.x & 31;
    const size_t row = static_cast<size_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);     // of all kv heads
    const size_t total = static_cast<size_t>(a.c.B) * a.c.H * a.rows;
    if (row >= total) return;
    const size_t bh = row / a.rows;
    const int r = static_cast<int>(row - bh * a.rows), tile = r / kRows;
    const bool dealt = a.rows <= 128;                                // two parts a CTA
    const int parts = dealt ? 2 * a.splits : a.splits, stride = dealt ? 128 : kRows;
    const size_t first = ((bh * a.tiles + tile) * a.splits) * kRows + (r - tile * kRows);   // part k: + k * stride
    float2 ml = make_float2(-INFINITY, 0.0f);
    if (lane < parts) ml = reinterpret_cast<const float2 *>(a.part_ml)[first + static_cast<size_t>(lane) * stride];
    float M = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float mine = ml.y == 0.0f ? 0.0f : ex2_approx(ml.x - M);
    float l = mine * ml.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    constexpr int V = D / 32;                                        // channels a lane: 2 or 4
    float o[V] = {};
    for (int k = 0; k < parts; ++k) {
        const float f = __shfl_sync(0xffffffffu, mine, k), lk = __shfl_sync(0xffffffffu, ml.y, k);
        if (lk == 0.0f) continue;                                    // saw nothing: not written
        const float *from = a.part_O + (first + static_cast<size_t>(k) * stride) * D + lane * V;
        if constexpr (V == 4) {
            const float4 x = *reinterpret_cast<const float4 *>(from);
            o[0] += f * x.x; o[1] += f * x.y; o[2] += f * x.z; o[3] += f * x.w;
        } else {
            const float2 x = *reinterpret_cast<const float2 *>(from);
            o[0] += f * x.x; o[1] += f * x.y;
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint32_t *to = static_cast<uint32_t *>(a.O) + (row * D + lane * V) / 2;
#pragma unroll
    for (int k = 0; k < V / 2; ++k) to[k] = pack2<BF16>(o[2 * k] * inv, o[2 * k + 1] * inv);
    if (lane == 0) a.L[row] = l == 0.0f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
}

// ---- host -------------------------------------------------------------------------------------
struct Plan {
    int tiles, splits;
    size_t off_ml, bytes;
};

static Plan plan(const sage_kv &c, int Hq, int T) {
    Plan p;
    const long long rows = static_cast<long long>(Hq / c.H) * T;
    p.tiles = static_cast<int>((rows + kRows - 1) / kRows);
    const long long items = static_cast<long long>(c.B) * c.H * p.tiles;
    // The slots are cut where CTAs are fewer than SMs: into as many ranges as end first, by waves of CTAs and the steps of
    // each, if every sequence fills its capacity.
    const long long steps = (static_cast<long long>(c.max_pages) * c.page + kStep - 1) / kStep;
    p.splits = 1;
    if (items < kSMs) {
        double best = 1e30;
        for (int k = 1; k <= kExtMaxSplits && (k == 1 || steps / k >= kMinSteps); ++k) {
            const double cost = static_cast<double>((items * k + kSMs - 1) / kSMs) * (static_cast<double>(steps) / k + kCtaSteps);
            if (cost < best) {
                best = cost;
                p.splits = k;
            }
        }
    }
    const size_t parts = p.splits > 1 || rows <= 128 ? static_cast<size_t>(items) * p.splits * kRows : 0;
    p.off_ml = parts * c.d * sizeof(float);
    p.bytes = p.off_ml + parts * 2 * sizeof(float);
    return p;
}

template <int D, bool BF16, int SC, bool FP8>
static cudaError_t launch_k(const Args &a, cudaStream_t st) {
    auto kernel = extend_kernel<D, BF16, SC, FP8>;
    const size_t smem = sizeof(Smem<D>) + 1024;
    static bool raised[16] = {false};
    cudaError_t e = raise_smem(reinterpret_cast<const void *>(kernel), smem, raised);
    if (e != cudaSuccess) return e;
    // the register split must fit in what the block is launched with, or an increase could never be granted
    static int regs = 0;
    if (regs == 0) {
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, kernel);
        if (e != cudaSuccess) return e;
        regs = fa.numRegs;
    }
    if (regs * kThreads < 256 * static_cast<int>(kRegsSoftmax + kRegsLoad) + 128 * static_cast<int>(kRegsControl)) return cudaErrorInvalidConfiguration;
    const long long grid = static_cast<long long>(a.c.B) * a.c.H * a.tiles * a.splits;
    kernel<<<static_cast<unsigned>(grid), kThreads, smem, st>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess || (a.splits == 1 && a.rows > 128)) return e;
    const size_t rows = static_cast<size_t>(a.c.B) * a.c.H * a.rows;
    extend_join_kernel<D, BF16><<<static_cast<unsigned>((rows + 7) / 8), 256, 0, st>>>(a);
    return cudaGetLastError();
}

template <int D, bool BF16>
static cudaError_t launch(const sage_kv &c, const Args &a, cudaStream_t st) {
    const bool fp8 = kv_format(c) == SAGE_KV_FP8;
    if (kv_format(c) == SAGE_KV_16) return launch_k<D, BF16, 0, false>(a, st);
    if (kv_block(c)) return fp8 ? launch_k<D, BF16, 2, true>(a, st) : launch_k<D, BF16, 2, false>(a, st);
    return fp8 ? launch_k<D, BF16, 1, true>(a, st) : launch_k<D, BF16, 1, false>(a, st);
}

}  // namespace ext

unsigned int take_extend_error() {
    unsigned int v = 0;
    const unsigned int zero = 0;
    cudaMemcpyFromSymbol(&v, g_ext_err, sizeof(v));
    if (v) cudaMemcpyToSymbol(g_ext_err, &zero, sizeof(zero));
    return v;
}
unsigned int take_extend_index() {
    unsigned int v = 0;
    const unsigned int zero = 0;
    cudaMemcpyFromSymbol(&v, g_ext_index, sizeof(v));
    if (v) cudaMemcpyToSymbol(g_ext_index, &zero, sizeof(zero));
    return v;
}

}  // namespace sage

using namespace sage;

// Rows a kv head up to which the one-token kernel takes the call.
constexpr int kExtendFewRows = 32;

static int check_extend(const sage_kv *c, int Hq, int T) {
    const int st = check_kv(c, false);
    if (st != SAGE_OK) return st;
    if (Hq <= 0 || Hq % c->H != 0 || T <= 0) return SAGE_ERR_ARG;
    if (static_cast<long long>(c->B) * Hq > (1 << 24) || static_cast<long long>(c->B) * Hq * T > (1 << 28)) return SAGE_ERR_UNSUPPORTED;
    return SAGE_OK;
}

extern "C" {

size_t sage_extend_workspace_bytes(const sage_kv *c, int Hq, int T) {
    if (check_extend(c, Hq, T) != SAGE_OK) return 0;
    return static_cast<long long>(Hq / c->H) * T <= kExtendFewRows ? decode_rows_bytes(*c, Hq, T) : ext::plan(*c, Hq, T).bytes;
}

int sage_attn_extend(const sage_kv *c, int Hq, int T, const void *Q, const int *start, const int *count, void *O, float *L,
                     void *workspace, size_t workspace_bytes, sage_stream_t stream) {
    int st = check_extend(c, Hq, T);
    if (st != SAGE_OK) return st;
    st = check_kv(c, true);
    if (st != SAGE_OK) return st;
    if (!Q || !start || !O || !L || O == Q) return SAGE_ERR_ARG;
    if (misaligned(Q, 16) || misaligned(O, 16) || misaligned(L, 16) || misaligned(start, 4) || misaligned(count, 4)) return SAGE_ERR_ALIGN;
    const size_t bytes = sage_extend_workspace_bytes(c, Hq, T);
    if (bytes) {                                 // else it is not looked at
        if (!workspace || workspace_bytes < bytes) return SAGE_ERR_WORKSPACE;
        if (misaligned(workspace, 256)) return SAGE_ERR_ALIGN;
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int G = Hq / c->H;
    cudaError_t e;
    if (static_cast<long long>(G) * T <= kExtendFewRows) {
        e = decode_rows(*c, Hq, T, Q, start, count, O, L, workspace, s);
    } else {
        const ext::Plan p = ext::plan(*c, Hq, T);
        ext::Args a;
        a.c = kv_view(*c);
        a.Q = Q; a.O = O; a.L = L; a.start = start; a.count = count;
        a.T = T; a.rows = G * T; a.tiles = p.tiles; a.splits = p.splits;
        const bool whole = T % ext::kRows == 0;
        a.order_heads = whole ? G : 0;
        a.order_tiles = whole ? T / ext::kRows : 0;
        a.sl2 = scale_log2(c->d);
        a.part_O = static_cast<float *>(workspace);
        a.part_ml = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + p.off_ml);
        const bool bf16 = c->dtype == SAGE_BF16;
        if (c->d == 64) e = bf16 ? ext::launch<64, true>(*c, a, s) : ext::launch<64, false>(*c, a, s);
        else e = bf16 ? ext::launch<128, true>(*c, a, s) : ext::launch<128, false>(*c, a, s);
    }
    return e == cudaSuccess ? SAGE_OK : SAGE_ERR_CUDA;
}

}  // extern "C"

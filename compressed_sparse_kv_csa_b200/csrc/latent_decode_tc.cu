// latent_decode_tc.cu -- latent attention in its absorbed form on tcgen05 for rows of 512 + 64
// channels: every operand of the cache goes to the tensor cores as it is stored, FP8 latent part and
// BF16 rotated part, with nothing converted on the way.
//
// The queries and the probabilities are what has to meet the FP8 codes, so each is split into two
// 8-bit terms whose products add up in the fp32 accumulators:
//   q 2^k = hi + lo, both E4M3 (2^k brings the row's largest latent entry to [128, 256)): 8 bits of
//     bf16 split into 4 + 4, exact down to 2^-10 of the largest entry, then off by at most 2^-18 of it;
//   v = hi + lo / 16, both E4M3 (the two have accumulators of their own): off by at most 2^-8 relative
//     for v >= 2^-6, as a bf16 probability is, and by 2^-14 absolute below.
// With s the scale of a key's row, S_n = sum_r (q 2^k)_r code_r and S_r = sum_r (q 2^k)_r rope_r,
//   z = (S_n s + S_r) scale log2e 2^-k,  p = 2^(z - ref),  l = sum p,  v = p s,  O = sum v code
// and o = O / l.  A row's ref is kept so that its v stay in E4M3's range: it is moved (and O and l
// rescaled) when a tile's largest v leaves it at the top (448), or falls below 1/16 while what is
// still to come could matter beside what has been summed: behind a key that outweighs all others the
// reference comes down again, and the many small ones keep their 8 bits.
//
// A work item's rows are 32 (head, token) pairs, stacked to the 64 rows of a weight-stationary MMA
// (tcgen05.mma.ws), rows 32 g + 16 part + r with part 0 = hi, 1 = lo: one pass over the keys serves both
// terms, and hi and lo of a score lie in lanes l and l + 16 of one warp.  M = 64 with .ws spreads the
// accumulator's column halves over all 128 lanes and reads 10 KB of shared memory for N = 256 in 80
// cycles (3273 multiply-adds a cycle at 16 bits, measured; without .ws 128 cycles, 2045).
// Per tile of 128 keys: S_n (N = 128, K = 512, FP8), S_r (N = 128, K = 64, BF16), O (+)= v code (two N = 256,
// K = 128, FP8, the codes read MN-major): 28 MMAs.
//
// Roles: warps 0-7 softmax and output, warps 8-9 copy the keys (cp.async, 16 bytes a lane, any page
// size; rows that are not to be seen arrive as zeros), warp 10 MMA.  Two stages of 80 KB.  Bound by HBM for up to 32 query rows a key.
#include "latent.cuh"
#include "tc_common.cuh"

namespace csa {

namespace {

using namespace tc;

constexpr int kR = 512, kRd = 64, kRB = 32, kKT = 128, kStages = 2;
constexpr int kSoftThreads = 256, kProdWarp0 = 8, kMmaWarp = 10, kThreads = 11 * 32;
// operand tiles of 128-byte rows, 128-byte swizzle: 64 query rows, 128 keys
constexpr uint32_t kQSlice = 8192, kSlice = 16384;
constexpr uint32_t OFF_Q = 0;                         // 4 slices of 128 latent channels, 1 of the rotated ones
constexpr uint32_t OFF_P = 5 * kQSlice;               // v: two buffers
constexpr uint32_t OFF_K = 7 * kQSlice;               // kStages x 5 slices
constexpr uint32_t OFF_SC = OFF_K + kStages * 5 * kSlice;
constexpr uint32_t OFF_XCH = OFF_SC + kStages * kKT * 4;     // [2 buffers][4 key quarters][32 rows] float2
constexpr uint32_t OFF_BAR = OFF_XCH + 2 * 4 * 32 * 8;
constexpr uint32_t OFF_AT = OFF_BAR + 160;            // where the CTA's walk begins (3 x int64)
constexpr uint32_t OFF_TMEM = OFF_AT + 32;
constexpr uint32_t SMEM_ALLOC = OFF_TMEM + 64 + 1024;
static_assert(SMEM_ALLOC <= 232448, "shared memory per block");
enum { B_KFULL = 0, B_KEMPTY = B_KFULL + kStages, B_S = B_KEMPTY + kStages, B_P = B_S + 2, B_Q = B_P + 2, B_ALL, B_ROWS, B_FINAL = B_ROWS + 2, NUM_BARS };
static_assert(8 * NUM_BARS <= 160, "barrier space");
// TMEM columns: O (two N = 256 accumulators, 128 columns each), S_n and S_r (two buffers of 64 each)
constexpr uint32_t kColO = 0, kColSn = 256, kColSr = 384, kTmemCols = 512;
constexpr uint32_t IDESC_SN = (1u << 4) | ((uint32_t)(kKT >> 3) << 17) | (4u << 24);                              // E4M3 x E4M3
constexpr uint32_t IDESC_SR = idesc_bf16_f32(64, kKT, false, false);
constexpr uint32_t IDESC_O = (1u << 4) | (1u << 16) | ((uint32_t)(256 >> 3) << 17) | (4u << 24); // B MN-major
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr uint32_t kNoKey = 0xffffffffu; // in place of a row's scale: the key is not to be seen
constexpr float kTop = 448.f, kLow = 1.f / 16.f, kSmallestScale = 7.8886090522101181e-31f; // 2^-100

using Split = LatentSplit<kRB, kKT>;

template <bool F8> __device__ __forceinline__ void mma_ws(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    if constexpr (F8)
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "setp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.ws.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
                     "r"(accumulate));
    else
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "setp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.ws.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
                     "r"(accumulate));
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void sts4(uint32_t addr, const uint32_t (&v)[4])
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

// Byte `byte` of row `row` in a 128-byte-swizzled tile of 128-byte rows.
__device__ __forceinline__ uint32_t sw128(uint32_t row, uint32_t byte)
{
    return row * 128u + ((((byte >> 4) ^ row) & 7u) << 4) + (byte & 15u);
}

// Two values as E4M3 codes (low byte first), and what the codes stand for.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b)
{
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 e4m3x2_value(uint32_t c)
{
    return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c, __NV_E4M3)));
}

// 16 values as hi and lo * lo_scale, 16 E4M3 codes each.
__device__ __forceinline__ void split16(const float (&v)[16], float lo_scale, uint32_t (&hi)[4], uint32_t (&lo)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        hi[i] = lo[i] = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float a = v[4 * i + 2 * h], b = v[4 * i + 2 * h + 1];
            const uint32_t c = e4m3x2(a, b);
            const float2 x = e4m3x2_value(c);
            hi[i] |= c << (16 * h);
            lo[i] |= e4m3x2((a - x.x) * lo_scale, (b - x.y) * lo_scale) << (16 * h);
        }
    }
}

// The runs of a CTA, one after another; every role walks them by itself.
struct Walk {
    int64_t at, end, b, before, nrb;
    __device__ __forceinline__ bool next(const LatentDecodeArgs &a, LatentRun &r)
    {
        if (at >= end || b >= a.B) return false;
        const int64_t tiles = Split::tiles(a, b);
        r.b = b;
        r.rb = (int)((at - before) / tiles);
        r.t0 = (at - before) - r.rb * tiles;
        r.t1 = min(tiles, r.t0 + (end - at));
        r.first = r.t0 == 0;
        r.whole = r.first && r.t1 == tiles;
        at += r.t1 - r.t0;
        if (r.t1 == tiles && r.rb + 1 == nrb) {
            before += tiles * nrb;
            ++b;
        }
        return true;
    }
};

struct Ctx {
    uint32_t base, tmem;
    __device__ __forceinline__ uint32_t bar(int b) const { return base + OFF_BAR + 8u * (uint32_t)b; }
    __device__ __forceinline__ uint32_t stage(uint32_t n) const { return base + OFF_K + (n % kStages) * 5u * kSlice; }
};

// Keys (warps 8-9): warp w copies rows 64 w .. 64 w + 63 of a tile, 8 lanes a row of 128 bytes.
__device__ __forceinline__ bool producer_role(const LatentDecodeArgs &a, const Ctx &c, Walk walk, int warp, int lane)
{
    LatentRun run;
    uint32_t n = 0; // tiles so far
    bool ok = true;
    while (ok && walk.next(a, run)) {
        const int64_t seen = latent_visible(a, run.b, a.Lq - 1);
        auto resolve = [&](int64_t t, int h) { // row of the key that this lane looks up
            const int64_t s = t * kKT + 64 * warp + 32 * h + lane;
            if (s >= seen) return (int64_t)-1;
            const int64_t row = a.map.row(run.b, s);
            if (row < 0) flag_error(a.err, CSA_DEVERR_INDEX);
            return row;
        };
        int64_t mine[2] = {resolve(run.t0, 0), resolve(run.t0, 1)};
        for (int64_t t = run.t0; t < run.t1; ++t, ++n) {
            const int64_t cur[2] = {mine[0], mine[1]};
            if (t + 1 < run.t1) mine[0] = resolve(t + 1, 0), mine[1] = resolve(t + 1, 1); // page lookups beside this tile's copies
            if (n >= kStages && !__all_sync(0xffffffffu, mbar_wait(c.bar(B_KEMPTY + n % kStages), ((n / kStages) & 1) ^ 1))) {
                ok = false;
                break;
            }
            const uint32_t st = c.stage(n), sc = c.base + OFF_SC + (n % kStages) * kKT * 4;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int r = 64 * warp + 4 * i + (lane >> 3);
                const int64_t row = __shfl_sync(0xffffffffu, cur[i >> 3], 4 * (i & 7) + (lane >> 3));
                const int64_t src = row < 0 ? 0 : row;
                const uint32_t bytes = row < 0 ? 0u : 16u, dst = st + sw128((uint32_t)r, 16u * (uint32_t)(lane & 7));
                const uint8_t *f8 = a.rows.fp8 + src * kR + 16 * (lane & 7);
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + (uint32_t)s * kSlice), "l"(f8 + 128 * s), "r"(bytes)
                                 : "memory");
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + 4 * kSlice),
                             "l"(a.rows.rope + src * kRd + 8 * (lane & 7)), "r"(bytes)
                             : "memory");
                if ((lane & 7) == 0) {
                    if (row < 0) asm volatile("st.shared.u32 [%0], %1;" ::"r"(sc + 4u * (uint32_t)r), "r"(kNoKey) : "memory");
                    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(sc + 4u * (uint32_t)r), "l"(a.rows.scale + row) : "memory");
                }
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(c.bar(B_KFULL + n % kStages)) : "memory");
            mbar_arrive(c.bar(B_KFULL + n % kStages)); // and for the plain stores
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory"); // nothing is in flight when the block ends
    return ok;
}

// Waits until either barrier's phase is complete; true when the second's is and the first's is not.
__device__ __forceinline__ bool mbar_wait_either(uint32_t a, uint32_t pa, uint32_t b, uint32_t pb)
{
    const uint64_t t0 = globaltimer();
    for (uint32_t it = 1;; ++it) {
        if (mbar_test_wait(a, pa)) return false;
        if (mbar_test_wait(b, pb)) return true;
        if ((it & 255u) == 0 && globaltimer() - t0 > 2000000000ull) return false; // the caller's own wait reports it
    }
}

// MMA issue (one thread).  S of tile n goes before O of tile n - 1, so that the softmax of one runs beside
// the MMAs of the other; at a run's first tile O of the run before goes first, since its output has to
// be read before the new queries are there.
__device__ __forceinline__ bool mma_role(const LatentDecodeArgs &a, const Ctx &c, Walk walk)
{
    LatentRun run;
    uint32_t n = 0, runs = 0;
    bool pending = false, pending_first = false;
    auto output = [&](uint32_t k, bool first) { // O (+)= v code of tile k
        if (!mbar_wait(c.bar(B_P + (k & 1)), (k >> 1) & 1)) return false;
        tc_fence_after();
        const uint32_t st = c.stage(k);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                mma_ws<true>(c.tmem + kColO + 128u * h, sdesc_sw128(c.base + OFF_P + kQSlice * (k & 1) + 32u * kk, 16, 1024),
                             sdesc_sw128(st + 2u * h * kSlice + 4096u * kk, kSlice, 1024), IDESC_O, !first || kk > 0);
        mma_commit(c.bar(B_KEMPTY + k % kStages));
        return true;
    };
    while (walk.next(a, run)) {
        for (int64_t t = run.t0; t < run.t1; ++t, ++n) {
            const bool first = t == run.t0;
            if (first) {
                if (pending && !output(n - 1, pending_first)) return false;
                pending = false;
                if (!mbar_wait(c.bar(B_Q), runs & 1)) return false;
                ++runs;
            }
            const uint32_t full = c.bar(B_KFULL + n % kStages), full_ph = (n / kStages) & 1;
            if (pending && !mbar_test_wait(full, full_ph) && mbar_wait_either(full, full_ph, c.bar(B_P + ((n - 1) & 1)), ((n - 1) >> 1) & 1)) {
                // the keys are late: O of the tile before goes first, so that its stage is free the sooner
                if (!output(n - 1, pending_first)) return false;
                pending = false;
            }
            if (!mbar_wait(full, full_ph)) return false;
            fence_proxy_async_smem(); // the copies were the generic proxy's
            tc_fence_after();
            const uint32_t st = c.stage(n);
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_ws<true>(c.tmem + kColSn + 64u * (n & 1), sdesc_sw128(c.base + OFF_Q + s * kQSlice + 32u * kk, 16, 1024),
                                 sdesc_sw128(st + s * kSlice + 32u * kk, 16, 1024), IDESC_SN, (s | kk) != 0);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_ws<false>(c.tmem + kColSr + 64u * (n & 1), sdesc_sw128(c.base + OFF_Q + 4 * kQSlice + 32u * kk, 16, 1024),
                              sdesc_sw128(st + 4 * kSlice + 32u * kk, 16, 1024), IDESC_SR, kk != 0);
            mma_commit(c.bar(B_S + (n & 1)));
            if (pending && !output(n - 1, pending_first)) return false;
            pending = true;
            pending_first = first;
        }
    }
    return !pending || output(n - 1, pending_first);
}

// A barrier between softmax warps, with the bound of every other wait.
struct Meet {
    uint32_t bar, phase;
    __device__ __forceinline__ bool sync()
    {
        mbar_arrive(bar);
        const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, phase));
        phase ^= 1;
        return ok;
    }
};

// Queries of a run into shared memory, as hi and lo rows; *factor is the factor that takes a score of this lane's
// row (16 (warp & 1) + (lane & 15)) to the log2 domain.
__device__ __forceinline__ bool load_queries(const LatentDecodeArgs &a, const Ctx &c, const LatentRun &run, int warp, int lane,
                                             Meet &all, float *factor)
{
    const int n_rows = min(kRB, a.Lq * a.H - run.rb * kRB);
    const uint16_t *q = a.q + (run.b * a.Lq * a.H + run.rb * kRB) * (int64_t)(kR + kRd);
    uint4 u[4][2];
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) { // all loads of the warp's 4 rows in flight together
        const int r = 4 * warp + i;
        u[i][0] = u[i][1] = make_uint4(0, 0, 0, 0);
        w[i] = 0;
        if (r < n_rows) {
            const uint16_t *p = q + (int64_t)r * (kR + kRd);
            u[i][0] = __ldg(reinterpret_cast<const uint4 *>(p + 16 * lane));
            u[i][1] = __ldg(reinterpret_cast<const uint4 *>(p + 16 * lane + 8));
            w[i] = __ldg(reinterpret_cast<const uint32_t *>(p + kR + 2 * lane));
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * warp + i;
        float x[16];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t y[4] = {u[i][h].x, u[i][h].y, u[i][h].z, u[i][h].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[8 * h + 2 * e] = __uint_as_float(y[e] << 16);
                x[8 * h + 2 * e + 1] = __uint_as_float(y[e] & 0xffff0000u);
            }
        }
        float am = 0.f;
        bool finite = true;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            am = fmaxf(am, fabsf(x[e]));
            finite = finite && fabsf(x[e]) < INFINITY;
        }
        const float rx = __uint_as_float(w[i] << 16), ry = __uint_as_float(w[i] & 0xffff0000u);
        am = warp_max(am);
        const float ar = warp_max(fmaxf(fabsf(rx), fabsf(ry)));
        finite = __all_sync(0xffffffffu, finite);
        // the largest latent entry to [128, 256), as far as the rotated entries stay far inside bf16's range
        const int en = (int)(__float_as_uint(am) >> 23) - 127, er = (int)(__float_as_uint(ar) >> 23) - 127;
        int k = am > 0.f && finite ? min(7 - en, 126) : 0;
        if (ar < INFINITY) k = min(k, 100 - er);
        const float up = exp2i(k);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] *= up;
        uint32_t hi[4], lo[4];
        split16(x, 1.f, hi, lo);
        const uint32_t row = 32u * (uint32_t)(r >> 4) + (uint32_t)(r & 15);
        // lane holds channels 16 lane .. 16 lane + 15: byte 16 (lane & 7) of slice lane / 8
        sts4(c.base + OFF_Q + (uint32_t)(lane >> 3) * kQSlice + sw128(row, 16u * (uint32_t)(lane & 7)), hi);
        sts4(c.base + OFF_Q + (uint32_t)(lane >> 3) * kQSlice + sw128(row + 16, 16u * (uint32_t)(lane & 7)), lo);
        const uint32_t rr = uint32_t(f32_to_bf16_bits(rx * up)) | (uint32_t(f32_to_bf16_bits(ry * up)) << 16);
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(c.base + OFF_Q + 4 * kQSlice + sw128(row, 4u * (uint32_t)lane)), "r"(rr) : "memory");
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(c.base + OFF_Q + 4 * kQSlice + sw128(row + 16, 4u * (uint32_t)lane)), "r"(0) : "memory");
        // a row that is not finite makes NaN of its scores
        const float f = finite ? a.scale * kLog2e * exp2i(-k) : NAN;
        if (lane == 0) asm volatile("st.shared.f32 [%0], %1;" ::"r"(c.base + OFF_XCH + 4u * (uint32_t)r), "f"(f) : "memory");
    }
    fence_proxy_async_smem();
    if (!all.sync()) return false;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(*factor) : "r"(c.base + OFF_XCH + 4u * (uint32_t)(16 * (warp & 1) + (lane & 15))) : "memory");
    return all.sync(); // the factors are read before the place is used again
}

// Softmax and output (warps 0-7).  Warp w has rows 16 g .. 16 g + 15 (g = w & 1) and quarter `kq` of a tile's 128
// keys; its lanes l and l + 16 hold the hi and lo parts of row 16 g + (l & 15) for the 32 keys, and after an
// exchange the whole scores of 16 keys each.  Warps w and w + 4 reach the same lanes of TMEM, and take one
// half of O's columns each.
__device__ __forceinline__ bool softmax_role(const LatentDecodeArgs &a, const Ctx &c, Walk walk, int warp, int lane)
{
    const int g = warp & 1, half = (warp >> 1) & 1, sub = warp >> 2, kq = 2 * half + sub;
    const int part = lane >> 4, r16 = lane & 15, row = 16 * g + r16;
    const uint32_t tw = c.tmem + ((uint32_t)(32 * (warp & 3)) << 16), tO = tw + kColO + 128u * (uint32_t)sub;
    Meet all{c.bar(B_ALL), 0}, four{c.bar(B_ROWS + g), 0}; // the eight warps; those that share the rows
    struct Others {
        float2 v[3];
    };
    auto swap_row = [&](uint32_t buf, float2 v, Others &o) { // a value of the row from the warps with its other keys
        const uint32_t at = c.base + OFF_XCH + 8u * (uint32_t)row + 1024u * buf;
        if (part == 0) asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(at + 256u * (uint32_t)kq), "f"(v.x), "f"(v.y) : "memory");
        if (!four.sync()) return false;
#pragma unroll
        for (int i = 0; i < 3; ++i)
            asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(o.v[i].x), "=f"(o.v[i].y) : "r"(at + 256u * (uint32_t)((kq + 1 + i) & 3)) : "memory");
        return true;
    };
    LatentRun run;
    uint32_t n = 0;
    while (walk.next(a, run)) {
        float cq;
        if (!load_queries(a, c, run, warp, lane, all, &cq)) return false;
        mbar_arrive(c.bar(B_Q));
        const int rr = run.rb * kRB + row, n_rows = a.Lq * a.H;
        const bool valid = rr < n_rows;
        const int64_t seen = valid ? latent_visible(a, run.b, rr / a.H) : 0;
        float ref = 0.f, l = 0.f, vs = 0.f; // reference, sum of p and of v over this thread's keys
        bool begun = seen <= run.t0 * kKT;  // the row has a reference, or needs none here
        for (int64_t t = run.t0; t < run.t1; ++t, ++n) {
            const uint32_t buf = n & 1;
            if (!__all_sync(0xffffffffu, mbar_wait(c.bar(B_S + buf), (n >> 1) & 1))) return false;
            tc_fence_after();
            uint32_t sn[32], sr[32];
            tmem_ld32(tw + kColSn + 64u * buf + 32u * (uint32_t)sub, sn);
            tmem_ld32(tw + kColSr + 64u * buf + 32u * (uint32_t)sub, sr);
            const uint32_t sc = c.base + OFF_SC + (n % kStages) * kKT * 4 + 128u * (uint32_t)kq;
            float s[32];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(s[4 * e]), "=f"(s[4 * e + 1]), "=f"(s[4 * e + 2]), "=f"(s[4 * e + 3])
                             : "r"(sc + 16u * e)
                             : "memory");
            tmem_ld_wait();
            // this thread's 16 keys: 32 kq + 16 part + e
            float z[16], sk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float t0 = fmaf(__uint_as_float(sn[e]), s[e], __uint_as_float(sr[e]));
                const float t1 = fmaf(__uint_as_float(sn[16 + e]), s[16 + e], __uint_as_float(sr[16 + e]));
                z[e] = (part ? t1 : t0) + __shfl_xor_sync(0xffffffffu, part ? t0 : t1, 16);
                sk[e] = part ? s[16 + e] : s[e];
            }
            const int n_seen = (int)max((int64_t)0, min((int64_t)16, seen - (t * kKT + 32 * kq + 16 * part)));
            uint32_t open = 0; // bit e: key e is seen
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                z[e] *= cq;
                const bool ok = __float_as_uint(sk[e]) != kNoKey && e < n_seen;
                open |= ok ? 1u << e : 0u;
                sk[e] = ok ? sk[e] : 0.f;
            }
            float v[16], top = 0.f, pt = 0.f, vt = 0.f;
            auto weigh = [&]() {
                top = pt = vt = 0.f;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float p = (open >> e & 1u) ? ex2(z[e] - ref) : 0.f;
                    pt += p;
                    v[e] = p * sk[e];
                    vt += v[e];
                    top = fmaxf(top, p * fmaxf(sk[e], kSmallestScale));
                }
            };
            weigh();
            float2 mine = make_float2(begun ? top : INFINITY, vs);
            mine.x = fmaxf(mine.x, __shfl_xor_sync(0xffffffffu, mine.x, 16));
            mine.y += __shfl_xor_sync(0xffffffffu, mine.y, 16);
            Others other;
            if (!swap_row(buf, mine, other)) return false;
            // (in the order of the quarters' pairs, so that all four warps get the same sum)
            const float row_top = fmaxf(fmaxf(mine.x, other.v[0].x), fmaxf(other.v[1].x, other.v[2].x));
            const float row_vs = kq & 1 ? (mine.y + other.v[2].y) + (other.v[0].y + other.v[1].y) : (mine.y + other.v[0].y) + (other.v[1].y + other.v[2].y);
            const float left = (float)(run.t1 - t) * kKT;
            const bool raise = row_top > kTop;
            const bool lower = row_top < kLow && row_top > 1e-30f && left * row_top > row_vs * (1.f / 256.f);
            // (the warps of the rows see the same values, so they take this branch together)
            if (__any_sync(0xffffffffu, raise || lower)) {
                float zt = -INFINITY; // the row's largest z + log2 s of this tile
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (open >> e & 1u) zt = fmaxf(zt, z[e] + __log2f(fmaxf(sk[e], kSmallestScale)));
                zt = fmaxf(zt, __shfl_xor_sync(0xffffffffu, zt, 16));
                if (!four.sync() || !swap_row(buf, make_float2(zt, 0.f), other)) return false; // (the place is read before it is used again)
                zt = fmaxf(fmaxf(zt, other.v[0].x), fmaxf(other.v[1].x, other.v[2].x));
                float f = 1.f;
                if ((raise || lower) && zt > -INFINITY) {
                    const float next = rintf(zt) - 3.f; // a whole number: O and the sums move by an exact power of two
                    f = begun ? ex2(ref - next) : 0.f;
                    ref = next;
                    begun = true;
                    l *= f;
                    vs *= f;
                }
                if (t > run.t0 && __any_sync(0xffffffffu, f != 1.f)) { // O of the tiles before this one
                    if (!__all_sync(0xffffffffu, mbar_wait(c.bar(B_KEMPTY + (n - 1) % kStages), ((n - 1) / kStages) & 1))) return false;
                    tc_fence_after();
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) {
                        uint32_t o[32];
                        tmem_ld32(tO + 32u * k, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st32(tO + 32u * k, o);
                    }
                    tmem_st_wait();
                }
                weigh();
            }
            l += pt;
            vs += vt;
            uint32_t hi[4], lo[4];
            split16(v, 16.f, hi, lo);
            const uint32_t col = 32u * (uint32_t)kq + 16u * (uint32_t)part;
            sts4(c.base + OFF_P + kQSlice * buf + sw128((uint32_t)(32 * g + r16), col), hi);
            sts4(c.base + OFF_P + kQSlice * buf + sw128((uint32_t)(32 * g + 16 + r16), col), lo);
            fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive(c.bar(B_P + buf));
        }
        // the run's last O, and the row's sum over the eight threads that share it
        if (!__all_sync(0xffffffffu, mbar_wait(c.bar(B_KEMPTY + (n - 1) % kStages), ((n - 1) / kStages) & 1))) return false;
        tc_fence_after();
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        Others other;
        if (!four.sync() || !swap_row(0, make_float2(l, 0.f), other)) return false;
        l = kq & 1 ? (l + other.v[2].x) + (other.v[0].x + other.v[1].x) : (l + other.v[0].x) + (other.v[1].x + other.v[2].x);
        const int64_t out_row = run.b * n_rows + rr;
        const float inv = l != 0.f ? 1.f / l : 0.f;
        float *rec = a.part + ((2 * (int64_t)blockIdx.x + run.first) * kRB + row) * (kR + 4);
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
            uint32_t o[32];
            tmem_ld32(tO + 32u * k, o);
            tmem_ld_wait();
            float x[16]; // channels 256 sub + 128 half + 32 k + 16 part + e
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float a0 = __uint_as_float(o[e]), a1 = __uint_as_float(o[16 + e]);
                const float got = __shfl_xor_sync(0xffffffffu, part ? a0 : a1, 16);
                x[e] = part ? fmaf(a1, 1.f / 16.f, got) : fmaf(got, 1.f / 16.f, a0); // hi + lo / 16
            }
            const int ch = 256 * sub + 128 * half + 32 * k + 16 * part;
            if (!valid) continue;
            if (run.whole) {
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    w[e] = uint32_t(f32_to_bf16_bits(x[2 * e] * inv)) | (uint32_t(f32_to_bf16_bits(x[2 * e + 1] * inv)) << 16);
                uint4 *d = reinterpret_cast<uint4 *>(a.o + out_row * kR + ch);
                d[0] = make_uint4(w[0], w[1], w[2], w[3]);
                d[1] = make_uint4(w[4], w[5], w[6], w[7]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    *reinterpret_cast<float4 *>(rec + 4 + ch + 4 * e) = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
            }
        }
        if (valid && kq == 0 && part == 0) {
            if (run.whole) {
                if (a.lse) a.lse[out_row] = l != 0.f ? (ref + log2f(l)) * kLn2 : -INFINITY;
            } else {
                rec[0] = l != 0.f ? ref : -INFINITY;
                rec[1] = l;
            }
        }
        tc_fence_before();
        if (!all.sync()) return false; // the sums are read before the place is used again
    }
    return true;
}

__global__ void __launch_bounds__(kThreads, 1) latent_decode_tc_kernel(LatentDecodeArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *sp = smem_raw + (base - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int64_t *s_at = reinterpret_cast<int64_t *>(sp + OFF_AT);
    const int64_t nrb = Split::row_blocks(a.Lq, a.H), G = gridDim.x;
    if (warp == 0) {
        const int64_t T = Split::warp_total(a, 0, a.B, lane) * nrb;
        int64_t b, before;
        Split::warp_find(a, T * blockIdx.x / G, nrb, lane, &b, &before);
        if (lane == 0) s_at[0] = b, s_at[1] = before, s_at[2] = T;
    } else if (tid == 32) {
        for (int b = 0; b < NUM_BARS; ++b) {
            uint32_t count = 1;
            if (b >= B_KFULL && b < B_KFULL + kStages) count = 128; // each producer thread's copies, and itself
            if (b == B_P || b == B_P + 1 || b == B_Q || b == B_ALL) count = kSoftThreads;
            if (b == B_ROWS || b == B_ROWS + 1) count = kSoftThreads / 2;
            mbar_init(base + OFF_BAR + 8u * (uint32_t)b, count);
        }
        mbar_init_fence();
    }
    if (warp == kMmaWarp) tmem_alloc(base + OFF_TMEM, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const Ctx c{base, *reinterpret_cast<volatile uint32_t *>(sp + OFF_TMEM)};
    const int64_t T = s_at[2];
    const Walk walk{T * blockIdx.x / G, T * (blockIdx.x + 1) / G, s_at[0], s_at[1], nrb};
    bool ok = true;
    if (warp < kProdWarp0) ok = softmax_role(a, c, walk, warp, lane);
    else if (warp < kMmaWarp) ok = producer_role(a, c, walk, warp - kProdWarp0, lane);
    else if (lane == 0) ok = mma_role(a, c, walk);
    if (!ok) flag_error(a.err, CSA_DEVERR_TIMEOUT);
    if (warp == kMmaWarp && lane == 0) { // every MMA completes before TMEM is released
        mma_commit(c.bar(B_FINAL));
        if (!mbar_wait(c.bar(B_FINAL), 0)) flag_error(a.err, CSA_DEVERR_TIMEOUT);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(c.tmem, kTmemCols);
}

} // namespace

bool latent_decode_tc_eligible(int R, int rd) { return R == kR && rd == kRd; }

size_t latent_decode_tc_workspace(int64_t B, int Lq, int H, int64_t max_len, int *grid)
{
    const int64_t tiles = (max_len + kKT - 1) / kKT, work = B * Split::row_blocks(Lq, H) * (tiles < 1 ? 1 : tiles);
    const int64_t most = device_sms();
    *grid = (int)(work < most ? work : most);
    return (size_t)*grid * 2 * kRB * (kR + 4) * sizeof(float);
}

cudaError_t launch_latent_decode_tc(const LatentDecodeArgs &a, cudaStream_t st)
{
    cudaError_t e = cudaFuncSetAttribute(latent_decode_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_ALLOC);
    if (e != cudaSuccess) return e;
    latent_decode_tc_kernel<<<(unsigned)a.grid, kThreads, SMEM_ALLOC, st>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_latent_merge_32x128(a, st);
}

} // namespace csa

// latent_decode_tc.cu -- latent attention in its absorbed form on tcgen05 for rows of 512 + 64
// channels: every operand of the cache goes to the tensor cores as it is stored, FP8 latent part and
// BF16 rotated part, with nothing converted on the way.
//
// The queries and the probabilities are what has to meet the FP8 codes, so each is split into two
// 8-bit terms whose products add up in the fp32 accumulators:
//   q 2^k = hi + lo, both E4M3 (2^k brings the row's largest latent entry to [128, 256)): 8 bits of
//     bf16 split into 4 + 4, exact down to 2^-10 of the largest entry, then off by at most 2^-18 of it;
//   v = hi + lo, hi E4M3 and lo E5M2, or E4M3 of 16 times itself where the two have accumulators of their own: off by
//     at most 2^-8 relative for v >= 2^-6, as a bf16 probability is, and by 2^-14 absolute below.
// With s the scale of a key's row, S_n = sum_r (q 2^k)_r code_r and S_r = sum_r (q 2^k)_r rope_r,
//   z = (S_n s + S_r) scale log2e 2^-k,  p = 2^(z - ref),  l = sum p,  v = p s,  O = sum v code
// and o = O / l.  A row's ref is kept so that its v stay in E4M3's range: it is moved (and O and l
// rescaled) when a tile's v leave it at the top, and when they are so small that the 2^-14 which rounding may take
// off each comes to more than 2^-9 of the row's sum of v.  With a sum of kLost / kAllowed a key (4 for 128
// keys) a tile's loss is within that by itself, below it is added up and held against the sum so far.  So behind
// a key that outweighs all others the reference comes down again, as far as the many small ones matter beside
// it: an output is off by at most 2^-8 of its terms and 2^-8 of the mean of 448 s, weighted by p.  A key
// whose codes are all zero would spoil that -- its scale stands for nothing, and is 1 as such rows are written
// -- so its v is taken as 0 (of 4,096 keys one without a value and e^12 above the others: 0.74 of the output's norm was
// lost with its scale).
//
// A work item's rows are RB = 32 or 64 (head, token) pairs.  The MMAs are bound by what they read of shared memory,
// 128 bytes a cycle, behind 46 cycles each for the issue; those with M = 64 are weight-stationary (tcgen05.mma.ws),
// which spread an accumulator over all 128 lanes (M = 64, N = 256 at 16 bits: 80 cycles, measured; without .ws 128).
//   RB = 32, tiles of 128 keys, two stages of 80 KB: hi and lo are rows of one operand with M = 64.  S_n (N = 128,
//     K = 512, FP8), S_r (N = 128, K = 64, BF16), O (+)= v code (two N = 256, K = 128; the codes read MN-major): 28
//     MMAs, 1,600 cycles.  Rows 32 g + 16 part + r of an operand are part 0 (hi) and 1 (lo) of row 16 g + r, so the
//     two parts of a score lie in lanes l and l + 16 of one warp and meet by shuffle.  (Two passes with M = 32 need
//     no shuffle, but 680 more cycles of the chain below; measured 5,100 cycles a tile.)  3,050 to 3,400 cycles a
//     tile, which is HBM's rate.
//   RB = 64, tiles of 64 keys, three stages of 40 KB: S_n with M = 128, hi over lo, whose parts meet through shared
//     memory (two passes with M = 64 read the keys twice: 1,650 cycles for S instead of 930, and as long a tile;
//     4 x 1M keys x 64 rows in a loop of seconds 0.79 ms, so 0.77 ms); S_r with M = 64; O from hi, then from lo.
//     2,300 cycles a tile: the chain load (2,000 cycles) - S (1,200) - softmax (1,700) - O (1,200) over the stages.
//     At that rate the chip is at its power limit too (990 W, 1.5 GHz).
// One exchange a tile, of the threads' sums of a row's v, lets the softmax warps decide alike whether a reference moves.
//
// Roles: warps 0-7 softmax and output; warp 8 copies the keys by TMA, in boxes of a page or of a tile, and warp 9
// brings the tiles after into L2 (with pages that no box fits, both copy by cp.async); warp 10 MMA.  Rows that are
// not to be seen are zeros in shared memory, or not read: the probability 0 times whatever they held would not be 0.
// Measured: 64 sequences of 1k to 16k keys x 16 heads 66 us (3.6 TB/s), 32 of 3k to 12k x 128 heads x 2 tokens 178 us (of
// contiguous rows 158), 4 x 1M keys x 64 heads 0.65 to 0.68 ms in a short run (4 TB/s), 0.78 in a loop of seconds.
#include "latent.cuh"
#include "tc_common.cuh"
#include "tma_host.cuh"

namespace csa {

namespace {

using namespace tc;

constexpr int kR = 512, kRd = 64;
constexpr int kSoftThreads = 256, kProdWarp0 = 8, kMmaWarp = 10, kThreads = 384; // whole warpgroups, for the register split
// Of the registers that the block is launched with (168 a thread, checked on the host), the two softmax warpgroups take 192
// a thread and the other leaves 120.
constexpr int kRegs = 168, kRegsSoft = 192, kRegsRest = 120;
static_assert(256 * kRegsSoft + 128 * kRegsRest <= kThreads * kRegs, "register split");
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr uint32_t kNoKey = 0xbf800000u; // -1 in place of a row's scale (scales are positive): the key is not to be seen
constexpr float kTop = 448.f, kSmallestScale = 7.8886090522101181e-31f; // 2^-100
constexpr float kLost = 6.103515625e-5f;         // 2^-14: what rounding may take off a small v
constexpr float kAllowed = 1.f / 512.f;          // share of a row's sum of v that this may come to
constexpr float kMostP = 3.2451855365842673e32f; // 2^108, of a thread's p in a tile; a row's sum of p stays in fp32's range
constexpr float kAbove = 2.f;                    // a tile's largest v is 4 to 8 when it sets the reference
constexpr float kMostL = 104.f;                 // log2 of a row's sum of p that a reference may be brought down to

template <bool F8, bool WS = true> __device__ __forceinline__ void mma(uint32_t d, Desc a, Desc b, uint32_t idesc, uint32_t accumulate)
{
    if constexpr (F8 && !WS)
        asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
                     "setp.ne.b32 p, %6, 0;\n\tmov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\t"
                     "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %5, p;\n\t}" ::"r"(d), "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi),
                     "r"(idesc), "r"(accumulate));
    else if constexpr (F8)
        asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
                     "setp.ne.b32 p, %6, 0;\n\tmov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\t"
                     "tcgen05.mma.ws.cta_group::1.kind::f8f6f4 [%0], x, y, %5, p;\n\t}" ::"r"(d), "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi),
                     "r"(idesc), "r"(accumulate));
    else
        asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
                     "setp.ne.b32 p, %6, 0;\n\tmov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\t"
                     "tcgen05.mma.ws.cta_group::1.kind::f16 [%0], x, y, %5, p;\n\t}" ::"r"(d), "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi),
                     "r"(idesc), "r"(accumulate));
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

// 16 values as two terms, 16 codes each: hi in E4M3, and what is left either 16 times as large in E4M3 or as it is in
// E5M2 (which has the range for it).
template <bool E5M2> __device__ __forceinline__ void split16(const float2 (&v)[8], float lo_scale, uint32_t (&hi)[4], uint32_t (&lo)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        hi[i] = lo[i] = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float2 a = v[2 * i + h];
            const uint32_t c = e4m3x2(a.x, a.y);
            const float2 x = e4m3x2_value(c);
            hi[i] |= c << (16 * h);
            lo[i] |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2((a.x - x.x) * lo_scale, (a.y - x.y) * lo_scale), __NV_SATFINITE,
                                                        E5M2 ? __NV_E5M2 : __NV_E4M3)
                     << (16 * h);
        }
    }
}

struct Maps {
    CUtensorMap lat, rope;
    int box;             // rows of a box; 0: copied by cp.async
    int shift;           // pages of less than a tile: log2 of their rows
    uint32_t page_tiles; // pages of whole tiles: how many
    uint32_t n_pages;    // pages that lie in the cache in full
    // the latent part of a stage: bytes between slices of 128 channels and between groups of 8 rows.  Boxes of pages
    // put the four slices of 8 rows side by side (one box whatever the page's size, 8 rows on an 8-row boundary);
    // a contiguous run, which may begin anywhere, and cp.async put the rows of a slice side by side
    uint32_t slice, group;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, uint32_t bytes) // 16 bytes, or zeros
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void sts1(uint32_t dst, uint32_t v) { asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst), "r"(v) : "memory"); }

__device__ __forceinline__ void tmem_ld32_pairs(uint32_t taddr, float2 (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=f"(r[0].x), "=f"(r[0].y), "=f"(r[1].x), "=f"(r[1].y), "=f"(r[2].x), "=f"(r[2].y), "=f"(r[3].x), "=f"(r[3].y),
                   "=f"(r[4].x), "=f"(r[4].y), "=f"(r[5].x), "=f"(r[5].y), "=f"(r[6].x), "=f"(r[6].y), "=f"(r[7].x), "=f"(r[7].y),
                   "=f"(r[8].x), "=f"(r[8].y), "=f"(r[9].x), "=f"(r[9].y), "=f"(r[10].x), "=f"(r[10].y), "=f"(r[11].x), "=f"(r[11].y),
                   "=f"(r[12].x), "=f"(r[12].y), "=f"(r[13].x), "=f"(r[13].y), "=f"(r[14].x), "=f"(r[14].y), "=f"(r[15].x), "=f"(r[15].y)
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16_pairs(uint32_t taddr, float2 (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=f"(r[0].x), "=f"(r[0].y), "=f"(r[1].x), "=f"(r[1].y), "=f"(r[2].x), "=f"(r[2].y), "=f"(r[3].x), "=f"(r[3].y),
                   "=f"(r[4].x), "=f"(r[4].y), "=f"(r[5].x), "=f"(r[5].y), "=f"(r[6].x), "=f"(r[6].y), "=f"(r[7].x), "=f"(r[7].y)
                 : "r"(taddr));
}

__device__ __forceinline__ void lds4(uint32_t addr, float2 &a, float2 &b)
{
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(a.x), "=f"(a.y), "=f"(b.x), "=f"(b.y) : "r"(addr) : "memory");
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

// A barrier between softmax warps, with the bound of every other wait.
struct Meet {
    uint32_t bar, phase;
    __device__ __forceinline__ bool sync()
    {
        mbar_arrive(bar);
        return wait();
    }
    __device__ __forceinline__ bool wait() // after the arrival
    {
        const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, phase));
        phase ^= 1;
        return ok;
    }
};

// The kernel for blocks of RB query rows.
template <int RB> struct Decode {

static constexpr int kRB = RB, kKT = RB == 32 ? 128 : 64, kStages = RB == 32 ? 2 : 3;
static constexpr bool kStacked = RB == 32; // hi and lo as rows of one operand
// operand tiles of 128-byte rows, 128-byte swizzle: 64 rows of q and v, kKT keys
static constexpr uint32_t kQSlice = 2 * kRB * 128, kQRope = 4 * kQSlice, kPTile = 8192, kSlice = kKT * 128, kStage = 5 * kSlice;
static constexpr uint32_t kPBufs = kStacked ? 2 : 1, kExch = kStacked ? 0 : 16384;
static constexpr uint32_t OFF_P = 0;                         // v
static constexpr uint32_t OFF_K = kPBufs * kPTile;           // stages of 5 slices: 4 of 128 latent channels, 1 of the rotated ones
static constexpr uint32_t OFF_Q = OFF_K + kStages * kStage;
static constexpr uint32_t OFF_EX = OFF_Q + kQRope + 8192;       // after q: 4 slices (hi and lo rows), the rotated channels
static constexpr uint32_t OFF_SC = OFF_EX + kExch;              // parts of scores that change hands
static constexpr uint32_t OFF_XCH = OFF_SC + kStages * kKT * 4; // [4 places][4 key quarters][rows]
static constexpr uint32_t OFF_BAR = OFF_XCH + 4 * 4 * kRB * 4;
static constexpr uint32_t OFF_AT = OFF_BAR + 160; // where the CTA's walk begins (4 x int64)
static constexpr uint32_t OFF_TMEM = OFF_AT + 32;
static constexpr uint32_t SMEM_ALLOC = OFF_TMEM + 64 + 1024;
static_assert(SMEM_ALLOC <= 232448, "shared memory per block");
enum { B_KFULL = 0, B_KEMPTY = B_KFULL + kStages, B_S = B_KEMPTY + kStages, B_P = B_S + 2, B_Q = B_P + 2, B_ALL, B_ROWS, B_TAIL = B_ROWS + 2, B_FINAL, NUM_BARS };
static_assert(8 * NUM_BARS <= 160, "barrier space");
// TMEM columns: O (two N = 256 accumulators, 128 columns each), S_n and S_r (two buffers each)
static constexpr uint32_t kSrCols = kKT / 2, kColO = 0, kColSn = 256, kColSr = 384, kTmemCols = 512;
static constexpr uint32_t IDESC_SN = (1u << 4) | ((uint32_t)(kKT >> 3) << 17) | ((uint32_t)(2 * kRB >> 4) << 24); // M = 2 RB, E4M3 x E4M3
static constexpr uint32_t IDESC_SR = idesc_bf16_f32(64, kKT, false, false);
static constexpr uint32_t IDESC_O = (1u << 4) | (1u << 16) | ((uint32_t)(256 >> 3) << 17) | (4u << 24); // M = 64, B MN-major
static constexpr uint32_t IDESC_O_LO = IDESC_O | (kStacked ? 0u : 1u << 7);                             // lo in E5M2

using Split = LatentSplit<kRB, kKT, 4>;
using Walk = LatentWalk<Split>;

struct Ctx {
    uint32_t base, tmem;
    __device__ __forceinline__ uint32_t bar(int b) const { return base + OFF_BAR + 8u * (uint32_t)b; }
    __device__ __forceinline__ bool wait(int b, uint32_t parity) const { return mbar_wait(bar(b), parity); }
    __device__ __forceinline__ uint32_t stage(uint32_t n) const { return base + OFF_K + (n % kStages) * kStage; }
};

// Steps of 32 keys that O (+)= v code takes of tile t: up to the last key that is to be seen.  Rows behind it are not read
// (a score that they gave is not used, whatever it is); of those before, the ones that are not there are zeros.
static __device__ __forceinline__ int output_steps(int64_t seen, int64_t t)
{
    const int64_t n = seen - t * kKT;
    return n >= kKT ? kKT / 32 : n <= 32 ? 1 : (int)(n + 31) / 32;
}

// The boxes of a run's tiles: lane i has box i.  Everything here is on the way between a free stage and its copies,
// so a tile costs a lane one page number, loaded two tiles ahead and untouched before (behind a busy memory a
// lookup takes as long as a tile).
struct Boxes {
    const LatentDecodeArgs &a;
    const Maps &M;
    const int32_t *table;
    int64_t base, seen, t1;
    int lane, n; // boxes of a tile
    __device__ __forceinline__ Boxes(const LatentDecodeArgs &a_, const Maps &M_, int lane_) : a(a_), M(M_), lane(lane_), n(kKT / M_.box) {}
    __device__ __forceinline__ void begin(const LatentRun &run)
    {
        table = a.map.pages + (a.map.pages ? run.b * a.map.max_pages : 0);
        base = a.map.first(run.b); // without pages: the row of position 0
        seen = latent_visible(a, run.b, a.Lq - 1);
        t1 = run.t1;
    }
    __device__ __forceinline__ int32_t page(int64_t t) const
    {
        int32_t p = -1;
        if (a.map.pages && lane < n && t < t1) {
            const uint32_t i = M.box == kKT ? (uint32_t)t / M.page_tiles : ((uint32_t)t * kKT + lane * M.box) >> M.shift;
            if (i < (uint32_t)a.map.max_pages) p = __ldg(table + i);
        }
        return p;
    }
    // First row of this lane's box, or -1 when not all of its rows are there to be seen.
    __device__ __forceinline__ int32_t row(int64_t t, int32_t page) const
    {
        int64_t r = base + t * kKT;
        bool ok = seen >= t * kKT + (lane + 1) * M.box;
        if (a.map.pages) {
            r = (int64_t)(uint32_t)page * a.map.page_rows + (M.box == kKT ? (uint32_t)t % M.page_tiles * kKT : 0u);
            ok = ok && (uint32_t)page < M.n_pages;
        } else {
            ok = ok && r >= 0 && r + kKT <= a.rows.n;
        }
        return ok ? (int32_t)r : -1;
    }
    __device__ __forceinline__ bool whole(int32_t row) const { return !__any_sync(0xffffffffu, lane < n && row < 0); }
};

static __device__ __forceinline__ bool any_row(const int64_t (&r)[kKT / 32])
{
    bool any = false;
#pragma unroll
    for (int k = 0; k < kKT / 32; ++k) any |= r[k] >= 0;
    return any;
}
static __device__ __forceinline__ int64_t pick(const int64_t (&r)[kKT / 32], int k) // without an address
{
    int64_t v = r[0];
#pragma unroll
    for (int i = 1; i < kKT / 32; ++i) v = k == i ? r[i] : v;
    return v;
}

// Keys by TMA (warp 8).
static __device__ __forceinline__ bool tma_role(const LatentDecodeArgs &a, const Maps &M, const Ctx &c, Walk walk, volatile uint32_t *issued, int lane)
{
    LatentRun run;
    uint32_t n = 0, tails = 0; // tiles so far, those with rows that are not to be seen
    bool ok = true;
    Boxes B(a, M, lane);
    const bool paged = a.map.pages != nullptr;
    while (ok && walk.next(a, run)) {
        B.begin(run);
        auto scales = [&](int64_t t, float (&s)[kKT / 32]) { // contiguous: a tile ahead, in registers
#pragma unroll
            for (int k = 0; k < kKT / 32; ++k) {
                const int64_t r = B.base + t * kKT + 32 * k + lane;
                s[k] = 0.f;
                if (!paged && t < run.t1 && r >= 0 && r < a.rows.n) s[k] = __ldg(a.rows.scale + r);
            }
        };
        int32_t now = B.page(run.t0), next = B.page(run.t0 + 1);
        float sc_next[kKT / 32];
        scales(run.t0, sc_next);
        for (int64_t t = run.t0; t < run.t1; ++t, ++n) {
            const int32_t page = now, row = B.row(t, now), row0 = __shfl_sync(0xffffffffu, row, 0);
            const bool whole = B.whole(row);
            float sc_now[kKT / 32];
#pragma unroll
            for (int k = 0; k < kKT / 32; ++k) sc_now[k] = sc_next[k];
            now = next;
            next = B.page(t + 2);
            scales(t + 1, sc_next);
            int64_t tail_row[kKT / 32];
            uint32_t tail_scale[kKT / 32];
            if (!whole) { // row by row
                const int64_t n_seen = B.seen - t * kKT;
                bool refused = false;
#pragma unroll
                for (int k = 0; k < kKT / 32; ++k) {
                    const int j = 32 * k + lane;
                    const int32_t p = __shfl_sync(0xffffffffu, page, j / M.box);
                    tail_row[k] = j < n_seen ? a.map.row(p, B.base, (uint32_t)(t * kKT + j)) : -1;
                    tail_scale[k] = tail_row[k] < 0 ? kNoKey : __float_as_uint(__ldg(a.rows.scale + tail_row[k]));
                    refused |= j < n_seen && tail_row[k] < 0;
                }
                if (refused) flag_error(a.err, CSA_DEVERR_INDEX);
            }
            if (n >= kStages && !__all_sync(0xffffffffu, mbar_wait(c.bar(B_KEMPTY + n % kStages), ((n / kStages) & 1) ^ 1, a.wait_ns))) {
                ok = false;
                break;
            }
            const uint32_t st = c.stage(n), full = c.bar(B_KFULL + n % kStages), sc = c.base + OFF_SC + (n % kStages) * kKT * 4;
            if (whole && paged && B.n == 1) {
                if (elect_one()) {
                    mbar_arrive_expect_tx(full, (uint32_t)kKT * 644u);
                    tma_load_4d(st, &M.lat, 0, 0, 0, row0 >> 3, full);
                    tma_load_2d(st + 4 * kSlice, &M.rope, 0, row0, full);
                    bulk_load(sc, a.rows.scale + row0, (uint32_t)kKT * 4u, full);
                }
            } else if (whole && paged) {
                if (elect_one()) mbar_arrive_expect_tx(full, (uint32_t)kKT * 644u);
                for (int i = 0; i < B.n; ++i) {
                    const int32_t r = __shfl_sync(0xffffffffu, row, i);
                    if (elect_one()) {
                        tma_load_4d(st + (uint32_t)(i * M.box) * 512u, &M.lat, 0, 0, 0, r >> 3, full);
                        tma_load_2d(st + 4 * kSlice + (uint32_t)(i * M.box) * 128u, &M.rope, 0, r, full);
                        bulk_load(sc + (uint32_t)(i * M.box) * 4u, a.rows.scale + r, (uint32_t)M.box * 4u, full);
                    }
                }
            } else if (whole) {
#pragma unroll
                for (int k = 0; k < kKT / 32; ++k) sts1(sc + 4u * (uint32_t)(32 * k + lane), __float_as_uint(sc_now[k]));
                __syncwarp(); // every lane's scales before the one arrival that stands for them
                if (elect_one()) {
                    mbar_arrive_expect_tx(full, (uint32_t)kKT * 640u);
                    tma_load_3d(st, &M.lat, 0, row0, 0, full);
                    tma_load_2d(st + 4 * kSlice, &M.rope, 0, row0, full);
                }
            } else {
                // some rows are not to be seen, or not there: their places are zeroed once no box is on its way
                const int64_t(&key_row)[kKT / 32] = tail_row;
                uint32_t bytes = 0;
                if (!paged && __any_sync(0xffffffffu, any_row(key_row))) {
                    bytes = (uint32_t)kKT * 640u; // the run may begin or end outside the cache: zeros
                    if (elect_one()) {
                        tma_load_3d(st, &M.lat, 0, (int32_t)(B.base + t * kKT), 0, c.bar(B_TAIL));
                        tma_load_2d(st + 4 * kSlice, &M.rope, 0, (int32_t)(B.base + t * kKT), c.bar(B_TAIL));
                    }
                }
                for (int i = 0; paged && i < B.n; ++i) { // boxes whose first row is there; the rest of them may reach past the cache (zeros)
                    const int j = i * M.box, k = j >> 5;
                    const int64_t r = __shfl_sync(0xffffffffu, pick(key_row, k), j & 31);
                    if (r < 0) continue;
                    bytes += (uint32_t)M.box * 640u;
                    if (elect_one()) {
                        tma_load_4d(st + (uint32_t)j * 512u, &M.lat, 0, 0, 0, (int32_t)(r >> 3), c.bar(B_TAIL));
                        tma_load_2d(st + 4 * kSlice + (uint32_t)j * 128u, &M.rope, 0, (int32_t)r, c.bar(B_TAIL));
                    }
                }
                if (elect_one()) mbar_arrive_expect_tx(c.bar(B_TAIL), bytes);
#pragma unroll
                for (int k = 0; k < kKT / 32; ++k) sts1(sc + 4u * (uint32_t)(32 * k + lane), tail_scale[k]);
                if (!__all_sync(0xffffffffu, mbar_wait(c.bar(B_TAIL), tails & 1, a.wait_ns))) {
                    mbar_wait(c.bar(B_TAIL), tails & 1);
                    ok = false;
                    break;
                }
                ++tails;
                const uint32_t zero[4] = {0, 0, 0, 0};
                const int steps = output_steps(B.seen, t);
#pragma unroll 1
                for (int k = 0; k < steps; ++k) {
                    uint32_t bad = __ballot_sync(0xffffffffu, (pick(key_row, k)) < 0);
                    while (bad) { // a row at a time: 32 chunks of 16 bytes
                        const uint32_t j = (uint32_t)(32 * k + __ffs(bad) - 1), e = (uint32_t)lane;
                        bad &= bad - 1;
                        sts4(st + (e >> 3) * M.slice + (j >> 3) * M.group + (j & 7u) * 128u + 16u * (e & 7u), zero);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (elect_one()) mbar_arrive(full);
            }
            if (lane == 0) *issued = n + 1;
        }
    }
    if (lane == 0) *issued = 0xffffffffu;
    // nothing is on its way when the block ends, whatever the others waited for
    for (uint32_t k = n - min(n, (uint32_t)kStages); k < n; ++k) ok = mbar_wait(c.bar(B_KFULL + k % kStages), (k / kStages) & 1) && ok;
    return ok;
}

// The next kAhead tiles into L2 (warp 9): their stages are not free yet, and the way from HBM is most of what a load
// takes.  It follows the tiles that warp 8 has asked for, and nothing waits for it: what it is too late for it
// leaves out.
static constexpr int kAhead = kStages;
static __device__ __forceinline__ void prefetch_role(const LatentDecodeArgs &a, const Maps &M, Walk walk, const volatile uint32_t *issued, int lane)
{
    LatentRun run;
    uint32_t n = 0; // the run's first tile
    Boxes B(a, M, lane);
    while (walk.next(a, run)) {
        B.begin(run);
        int32_t next = B.page(run.t0 + 1);
        for (int64_t t = run.t0 + 1; t < run.t1; ++t) {
            const uint32_t k = n + (uint32_t)(t - run.t0); // this tile, counted as warp 8 counts
            const int32_t row = B.row(t, next);
            next = B.page(t + 1);
            uint32_t at = *issued;
            const uint64_t t0 = globaltimer();
            while (at + kAhead <= k && at <= k) { // (it ends at 2^32 - 1)
                __nanosleep(100);
                if (globaltimer() - t0 > 2000000000ull) return;
                at = *issued;
            }
            if (!__all_sync(0xffffffffu, at <= k) || !B.whole(row)) continue;
            if (lane < B.n) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.rows.scale + row));
            for (int i = 0; i < B.n; ++i) {
                const int32_t r = __shfl_sync(0xffffffffu, row, i);
                if (elect_one()) {
                    if (a.map.pages) tma_prefetch_4d(&M.lat, 0, 0, 0, r >> 3);
                    else tma_prefetch_3d(&M.lat, 0, r, 0);
                    tma_prefetch_2d(&M.rope, 0, r);
                }
            }
        }
        n += (uint32_t)(run.t1 - run.t0);
    }
}

// Keys by cp.async (warps 8-9): each warp copies half the rows of a tile, 8 lanes a row of 128 bytes.
static __device__ __forceinline__ bool copy_role(const LatentDecodeArgs &a, const Ctx &c, Walk walk, int warp, int lane)
{
    constexpr int kHalf = kKT / 2;
    LatentRun run;
    uint32_t n = 0;
    bool ok = true;
    while (ok && walk.next(a, run)) {
        const int64_t seen = latent_visible(a, run.b, a.Lq - 1);
        const int64_t first = a.map.first(run.b);
        auto resolve = [&](int64_t t, int h) { // row of the key that this lane looks up
            const int64_t s = t * kKT + kHalf * warp + 32 * h + lane;
            if (s >= seen) return (int64_t)-1;
            const int64_t row = a.map.row(a.map.page(run.b, (uint32_t)s), first, (uint32_t)s);
            if (row < 0) flag_error(a.err, CSA_DEVERR_INDEX);
            return row;
        };
        int64_t mine[kHalf / 32];
        for (int h = 0; h < kHalf / 32; ++h) mine[h] = resolve(run.t0, h);
        for (int64_t t = run.t0; t < run.t1; ++t, ++n) {
            int64_t cur[kHalf / 32];
#pragma unroll
            for (int h = 0; h < kHalf / 32; ++h) {
                cur[h] = mine[h];
                if (t + 1 < run.t1) mine[h] = resolve(t + 1, h);
            }
            if (n >= kStages && !__all_sync(0xffffffffu, mbar_wait(c.bar(B_KEMPTY + n % kStages), ((n / kStages) & 1) ^ 1, a.wait_ns))) {
                ok = false;
                break;
            }
            const uint32_t st = c.stage(n);
#pragma unroll
            for (int i = 0; i < kHalf / 4; ++i) {
                const int r = kHalf * warp + 4 * i + (lane >> 3);
                const int64_t row = __shfl_sync(0xffffffffu, cur[i >> 3], 4 * (i & 7) + (lane >> 3));
                const int64_t src = row < 0 ? 0 : row;
                const uint32_t bytes = row < 0 ? 0u : 16u, dst = st + sw128((uint32_t)r, 16u * (uint32_t)(lane & 7));
                const uint8_t *f8 = a.rows.fp8 + src * kR + 16 * (lane & 7);
#pragma unroll
                for (int s = 0; s < 4; ++s) copy16(dst + (uint32_t)s * kSlice, f8 + 128 * s, bytes);
                copy16(dst + 4 * kSlice, a.rows.rope + src * kRd + 8 * (lane & 7), bytes);
            }
#pragma unroll
            for (int h = 0; h < kHalf / 32; ++h) {
                const uint32_t dst = c.base + OFF_SC + (n % kStages) * kKT * 4 + 4u * (uint32_t)(kHalf * warp + 32 * h + lane);
                if (cur[h] < 0) sts1(dst, kNoKey);
                else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(a.rows.scale + cur[h]) : "memory");
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(c.bar(B_KFULL + n % kStages)) : "memory");
            mbar_arrive(c.bar(B_KFULL + n % kStages)); // and for the plain stores
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory"); // nothing is in flight when the block ends
    return ok;
}

// MMA issue (one thread).  S of tile n goes before O of tile n - 1, so that the softmax of one runs beside
// the MMAs of the other; at a run's first tile O of the run before goes first, since its output has to
// be read before the new queries are there.
static __device__ __forceinline__ bool mma_role(const LatentDecodeArgs &a, const Maps &M, const Ctx &c, Walk walk)
{
    LatentRun run;
    uint32_t n = 0, runs = 0;
    bool pending = false, pending_first = false;
    int pending_steps = 0;
    const Desc q_desc(sdesc_sw128(c.base + OFF_Q, 16, 1024)), k_desc(sdesc_sw128(c.base + OFF_K, 16, M.group)), r_desc(sdesc_sw128(c.base + OFF_K, 16, 1024));
    const Desc p_desc(sdesc_sw128(c.base + OFF_P, 16, 1024)), v_desc(sdesc_sw128(c.base + OFF_K, M.slice, M.group));
    auto output = [&](uint32_t k, bool first, int steps) { // O (+)= v code of tile k
        if (!c.wait(B_P + (k & 1), (k >> 1) & 1)) return false;
        tc_fence_after();
        const Desc dp = p_desc.at(kPTile * (k % kPBufs)), dv = v_desc.at((k % kStages) * kStage);
#pragma unroll
        for (int kk = 0; kk < kKT / 32; ++kk)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (kk < steps) {
                    const Desc b = dv.at(2u * h * M.slice + 4u * kk * M.group);
                    mma<true>(c.tmem + kColO + 128u * h, dp.at(32u * kk), b, IDESC_O, !first || kk > 0);
                    if constexpr (!kStacked) mma<true>(c.tmem + kColO + 128u * h, dp.at(64u + 32u * kk), b, IDESC_O_LO, 1);
                }
        mma_commit(c.bar(B_KEMPTY + k % kStages));
        return true;
    };
    while (walk.next(a, run)) {
        const int64_t seen = latent_visible(a, run.b, a.Lq - 1);
        for (int64_t t = run.t0; t < run.t1; ++t, ++n) {
            const bool first = t == run.t0;
            if (first) {
                if (pending && !output(n - 1, pending_first, pending_steps)) return false;
                pending = false;
                if (!c.wait(B_Q, runs & 1)) return false;
                ++runs;
            }
            const uint32_t full = c.bar(B_KFULL + n % kStages), full_ph = (n / kStages) & 1;
            if (pending && !mbar_test_wait(full, full_ph) && mbar_wait_either(full, full_ph, c.bar(B_P + ((n - 1) & 1)), ((n - 1) >> 1) & 1)) {
                // the keys are late: O of the tile before goes first, so that its stage is free the sooner
                if (!output(n - 1, pending_first, pending_steps)) return false;
                pending = false;
            }
            if (!mbar_wait(full, full_ph)) return false;
            fence_proxy_async_smem(); // cp.async writes for the generic proxy
            tc_fence_after();
            const Desc dk = k_desc.at((n % kStages) * kStage), dr = r_desc.at((n % kStages) * kStage + 4 * kSlice);
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma<true, kStacked>(c.tmem + kColSn + 64u * (n & 1), q_desc.at(s * kQSlice + 32u * kk), dk.at(s * M.slice + 32u * kk), IDESC_SN, (s | kk) != 0);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma<false>(c.tmem + kColSr + kSrCols * (n & 1), q_desc.at(kQRope + 32u * kk), dr.at(32u * kk), IDESC_SR, kk != 0);
            mma_commit(c.bar(B_S + (n & 1)));
            if (pending && !output(n - 1, pending_first, pending_steps)) return false;
            pending = true;
            pending_first = first;
            pending_steps = output_steps(seen, t);
        }
    }
    return !pending || output(n - 1, pending_first, pending_steps);
}

// 4 rows of a run's queries (of the kRB / 8 that a warp has), on their way from memory.
struct Queries {
    uint4 u[4][2];
    uint32_t w[4];
    __device__ __forceinline__ void fetch(const LatentDecodeArgs &a, const LatentRun &run, int row0, int lane)
    {
        const int n_rows = min(kRB, a.Lq * a.H - run.rb * kRB);
        const uint16_t *q = a.q + (run.b * a.Lq * a.H + run.rb * kRB) * (int64_t)(kR + kRd);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = row0 + i;
            u[i][0] = u[i][1] = make_uint4(0, 0, 0, 0);
            w[i] = 0;
            if (r < n_rows) {
                const uint16_t *p = q + (int64_t)r * (kR + kRd);
                u[i][0] = __ldg(reinterpret_cast<const uint4 *>(p + 16 * lane));
                u[i][1] = __ldg(reinterpret_cast<const uint4 *>(p + 16 * lane + 8));
                w[i] = __ldg(reinterpret_cast<const uint32_t *>(p + kR + 2 * lane));
            }
        }
    }
};

// Into shared memory, as hi and lo, with the factor that takes a row's scores to the log2 domain.  (Rows one after
// another: code that runs once a run comes from far away, and its length is what it costs.)
static __device__ __forceinline__ void store_queries(const LatentDecodeArgs &a, const Ctx &c, Queries &in, int row0, int lane)
{
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        const int r = row0 + i;
        float2 x[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t y[4] = {in.u[0][h].x, in.u[0][h].y, in.u[0][h].z, in.u[0][h].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) x[4 * h + e] = make_float2(__uint_as_float(y[e] << 16), __uint_as_float(y[e] & 0xffff0000u));
        }
        float am = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) am = fmaxf(am, fmaxf(fabsf(x[e].x), fabsf(x[e].y)));
        float nan = 0.f; // NaN where an entry is not finite
#pragma unroll
        for (int e = 0; e < 8; ++e) nan = fmaf(x[e].x, 0.f, fmaf(x[e].y, 0.f, nan));
        const float rx = __uint_as_float(in.w[0] << 16), ry = __uint_as_float(in.w[0] & 0xffff0000u);
        am = warp_max(am);
        const float ar = warp_max(fmaxf(fabsf(rx), fabsf(ry)));
        const bool finite = __all_sync(0xffffffffu, nan == 0.f);
        // the largest latent entry to [128, 256), as far as the rotated entries stay far inside bf16's range
        const int en = (int)(__float_as_uint(am) >> 23) - 127, er = (int)(__float_as_uint(ar) >> 23) - 127;
        int k = am > 0.f && finite ? min(7 - en, 126) : 0;
        if (ar < INFINITY) k = min(k, 100 - er);
        const float up = exp2i(k);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e].x *= up, x[e].y *= up;
        uint32_t hi[4], lo[4];
        split16<false>(x, 1.f, hi, lo);
        // lane holds channels 16 lane .. 16 lane + 15: byte 16 (lane & 7) of slice lane / 8
        const uint32_t row = kStacked ? 32u * (uint32_t)(r >> 4) + (uint32_t)(r & 15) : (uint32_t)r, q = c.base + OFF_Q, at = q + (uint32_t)(lane >> 3) * kQSlice;
        sts4(at + sw128(row, 16u * (uint32_t)(lane & 7)), hi);
        sts4(at + sw128(row + (kStacked ? 16 : 64), 16u * (uint32_t)(lane & 7)), lo);
        const uint32_t rot = q + kQRope;
        sts1(rot + sw128(row, 4u * (uint32_t)lane), uint32_t(f32_to_bf16_bits(rx * up)) | (uint32_t(f32_to_bf16_bits(ry * up)) << 16));
        if constexpr (kStacked) sts1(rot + sw128(row + 16, 4u * (uint32_t)lane), 0);
        // a row that is not finite makes NaN of its scores
        const float f = finite ? a.scale * kLog2e * exp2i(-k) : NAN;
        if (lane == 0) sts1(c.base + OFF_XCH + 4u * (uint32_t)r, __float_as_uint(f));
#pragma unroll
        for (int n = 0; n < 3; ++n) in.u[n][0] = in.u[n + 1][0], in.u[n][1] = in.u[n + 1][1], in.w[n] = in.w[n + 1];
    }
}

// Softmax and output (warps 0-7).  The rows lie in two halves g, and of a tile's keys a warp has quarter kq.  Warps w and
// w + 4 reach the same lanes of TMEM, and take one of O's two accumulators each.
//   Stacked: lanes l and l + 16 hold the hi and lo parts of row 16 g + (l & 15) for the quarter's 32 keys, and after
//   an exchange the whole scores of 16 keys each.
//   Otherwise lane l has row 32 g + l, warps with half 0 its hi and with half 1 its lo part for all keys; they exchange what
//   the other finishes, and hold the whole scores of the quarter's 16 keys.
static __device__ __forceinline__ bool softmax_role(const LatentDecodeArgs &a, const Maps &M, const Ctx &c, Walk walk, int warp, int lane)
{
    const int g = warp & 1, half = (warp >> 1) & 1, sub = warp >> 2, kq = 2 * half + sub;
    const int part = kStacked ? lane >> 4 : 0, r16 = lane & 15, row = kStacked ? 16 * g + r16 : 32 * g + lane;
    const int key = kStacked ? 32 * kq + 16 * part : 16 * kq;
    const uint32_t tw = c.tmem + ((uint32_t)(32 * (warp & 3)) << 16), tO = tw + kColO + 128u * (uint32_t)sub;
    Meet all{c.bar(B_ALL), 0}, rows{c.bar(B_ROWS + g), 0}; // the eight warps; those that share the rows
    // one value of the row from each quarter of the keys, in the quarters' order, so that all reduce them alike
    const uint32_t xch = c.base + OFF_XCH + 4u * (uint32_t)row;
    auto put_part = [&](uint32_t buf, float v) {
        if (part == 0) asm volatile("st.shared.f32 [%0], %1;" ::"r"(xch + 16u * kRB * buf + 4u * kRB * (uint32_t)kq), "f"(v) : "memory");
        mbar_arrive(rows.bar);
    };
    auto put = [&](uint32_t buf, float v) {
        put_part(buf, v);
        return rows.wait();
    };
    auto get = [&](uint32_t buf, float (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[i]) : "r"(xch + 16u * kRB * buf + 4u * kRB * i) : "memory");
    };
    auto max4 = [](const float (&v)[4]) { return fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])); };
    auto sum4 = [](const float (&v)[4]) { return (v[0] + v[1]) + (v[2] + v[3]); };
    auto other_part = [](float v) { return __shfl_xor_sync(0xffffffffu, v, 16); };
    auto row_max = [&](float v) { // over the lanes that share the row
        if constexpr (kStacked) v = fmaxf(v, other_part(v));
        return v;
    };
    auto row_sum = [&](float v) {
        if constexpr (kStacked) v += other_part(v);
        return v;
    };
    // Bit e: key e of this thread's has no value -- a scale of 1 and no code but +0 and -0.  Of the quarter's keys a lane looks
    // at one's scale and 16 of its codes, and the warp at all codes of those that may be such.
    auto no_value = [&](uint32_t st, uint32_t sc) {
        constexpr uint32_t kKeys = kKT / 4;
        auto row = [&](uint32_t i) {
            const uint32_t j = kKeys * (uint32_t)kq + i;
            return st + (j >> 3) * M.group + (j & 7u) * 128u;
        };
        auto any_code = [](uint32_t at) {
            uint32_t c[4];
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3]) : "r"(at) : "memory");
            return ((c[0] | c[1] | c[2] | c[3]) & 0x7f7f7f7fu) != 0;
        };
        const uint32_t mine = (uint32_t)lane % kKeys;
        float x;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(sc + 4u * mine) : "memory");
        uint32_t none = __ballot_sync(0xffffffffu, x == 1.f && (uint32_t)lane < kKeys && !any_code(row(mine) + 16u * (mine & 7u)));
#pragma unroll 1
        for (uint32_t left = none; left; left &= left - 1) {
            const uint32_t i = (uint32_t)__ffs(left) - 1, e = (uint32_t)lane;
            if (__any_sync(0xffffffffu, any_code(row(i) + (e >> 3) * M.slice + 16u * (e & 7u)))) none &= ~(1u << i);
        }
        return none >> (16 * part);
    };
    LatentRun run, next_run;
    uint32_t n = 0;
    float cq = 0.f, ref = 0.f, l = 0.f; // factor; reference and sum of p over this thread's keys
    // the run's last O, and the row's sum over the eight threads that share it
    auto output = [&](uint32_t n) {
        float other[4];
        const int rr = run.rb * kRB + row, n_rows = a.Lq * a.H;
        const bool valid = rr < n_rows;
        // the run's last O, and the row's sum over the eight warps
        if (!__all_sync(0xffffffffu, c.wait(B_KEMPTY + n % kStages, (n / kStages) & 1))) return false;
        tc_fence_after();
        if (!rows.sync() || !put(0, row_sum(l))) return false;
        get(0, other);
        l = sum4(other);
        const int64_t out_row = run.b * n_rows + rr;
        const float inv = l != 0.f ? 1.f / l : 0.f;
        float *rec = latent_part<kRB>(a.part, kR, 2 * (int64_t)blockIdx.x + run.first);
        auto put_out = [&](const auto &x, int ch) { // consecutive channels of the row
            constexpr int n = sizeof(x) / 4;
            if (run.whole) {
#pragma unroll
                for (int e = 0; e < n; e += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        w[u] = uint32_t(f32_to_bf16_bits(x[e + 2 * u] * inv)) | (uint32_t(f32_to_bf16_bits(x[e + 2 * u + 1] * inv)) << 16);
                    *reinterpret_cast<uint4 *>(a.o + out_row * kR + ch + e) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < n; e += 4)
                    *reinterpret_cast<float4 *>(rec + latent_part_at<kRB>(row, ch + e)) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
            }
        };
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
            uint32_t o[32];
            tmem_ld32(tO + 32u * k, o);
            tmem_ld_wait();
            if constexpr (kStacked) { // hi + lo / 16 of channels 256 sub + 128 half + 32 k + 16 part + e
                float x[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float a0 = __uint_as_float(o[e]), a1 = __uint_as_float(o[16 + e]), got = other_part(part ? a0 : a1);
                    x[e] = part ? fmaf(a1, 1.f / 16.f, got) : fmaf(got, 1.f / 16.f, a0);
                }
                if (valid) put_out(x, 256 * sub + 128 * half + 32 * k + 16 * part);
            } else if (valid) {
                put_out(*reinterpret_cast<float(*)[32]>(o), 256 * sub + 128 * half + 32 * k);
            }
        }
        if (valid && kq == 0 && part == 0) {
            if (run.whole) {
                if (a.lse) a.lse[out_row] = l != 0.f ? (ref + log2f(l)) * kLn2 : -INFINITY;
            } else {
                rec[2 * row] = l != 0.f ? ref : -INFINITY;
                rec[2 * row + 1] = l;
            }
        }
        tc_fence_before();
        return rows.sync(); // the sums are read before the place is used again
    };
    bool have = false;
    for (;;) {
        // every S of the run behind is there, so the next one's queries may go in, and its first S beside the output
        const bool more = walk.next(a, next_run);
        float cq_next = 0.f;
        if (more) {
            if (have && !all.sync()) return false; // the last exchange has been read
#pragma unroll 1
            for (int r = 0; r < kRB / 8; r += 4) {
                Queries queries;
                queries.fetch(a, next_run, kRB / 8 * warp + r, lane);
                store_queries(a, c, queries, kRB / 8 * warp + r, lane);
            }
            fence_proxy_async_smem();
            if (!all.sync()) return false;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(cq_next) : "r"(c.base + OFF_XCH + 4u * (uint32_t)row) : "memory");
            if (!all.sync()) return false; // the factors are read before the place is used again
            mbar_arrive(c.bar(B_Q));
        }
        if (have && !output(n - 1)) return false;
        if (!more) break;
        have = true;
        run = next_run;
        cq = cq_next;
        ref = l = 0.f;
        float other[4];
        const int rr = run.rb * kRB + row, n_rows = a.Lq * a.H;
        const bool valid = rr < n_rows;
        constexpr float kFew = kLost / kAllowed * kKT;
        const int64_t seen = valid ? latent_visible(a, run.b, rr / a.H) : 0;
        const int64_t seen_least = latent_visible(a, run.b, run.rb * kRB / a.H); // by every row of the block
        float vs = 0.f, vs_row = 0.f;      // sum of v over this thread's keys; and over the row's, at least
        float spent = 0.f;                 // what rounding may have taken off it
        bool begun = seen <= run.t0 * kKT;  // the row has a reference, or needs none here
        for (int64_t t = run.t0; t < run.t1; ++t, ++n) {
            const uint32_t buf = n & 1;
            if (!__all_sync(0xffffffffu, c.wait(B_KFULL + n % kStages, (n / kStages) & 1))) return false;
            float2 z[8], s[8], v[8];
            bool odd = false; // some key may not be seen by some row
            const uint32_t sc = c.base + OFF_SC + (n % kStages) * kKT * 4 + (kStacked ? 128u : 64u) * (uint32_t)kq;
            if constexpr (kStacked) {
                float2 sn[16], sr[16], sk[16];
#pragma unroll
                for (int e = 0; e < 8; ++e) lds4(sc + 16u * e, sk[2 * e], sk[2 * e + 1]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    s[e] = part ? sk[8 + e] : sk[e];
                    odd |= fabsf(s[e].x) == 1.f || fabsf(s[e].y) == 1.f;
                }
                if (!__all_sync(0xffffffffu, c.wait(B_S + buf, (n >> 1) & 1))) return false;
                tc_fence_after();
                tmem_ld32_pairs(tw + kColSn + 64u * buf + 32u * (uint32_t)sub, sn);
                tmem_ld32_pairs(tw + kColSr + kSrCols * buf + 32u * (uint32_t)sub, sr);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) sn[e] = fma2(sn[e], sk[e], sr[e]);
                // hi and lo of a score meet: this lane takes the first or the last 16 keys
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 send = part ? sn[e] : sn[8 + e], keep = part ? sn[8 + e] : sn[e];
                    z[e] = add2(keep, make_float2(other_part(send.x), other_part(send.y)));
                }
            } else {
                float2 sn[8], give[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) lds4(sc + 16u * e, s[2 * e], s[2 * e + 1]);
#pragma unroll
                for (int e = 0; e < 8; ++e) odd |= fabsf(s[e].x) == 1.f || fabsf(s[e].y) == 1.f;
                if (!__all_sync(0xffffffffu, c.wait(B_S + buf, (n >> 1) & 1))) return false;
                tc_fence_after();
                // this warp has hi or lo of all 64 keys, and gives the warp with the other part what that one has to finish
                tmem_ld16_pairs(tw + kColSn + 64u * buf + 32u * (uint32_t)(half ^ 1) + 16u * (uint32_t)sub, give);
                tmem_ld16_pairs(tw + kColSn + 64u * buf + 32u * (uint32_t)half + 16u * (uint32_t)sub, sn);
                tmem_ld16_pairs(tw + kColSr + kSrCols * buf + 16u * (uint32_t)sub, z);
                tmem_ld_wait();
                const uint32_t ex = c.base + OFF_EX + 16u * (uint32_t)lane;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(ex + 2048u * (uint32_t)(warp ^ 2) + 512u * e), "f"(give[2 * e].x),
                                 "f"(give[2 * e].y), "f"(give[2 * e + 1].x), "f"(give[2 * e + 1].y)
                                 : "memory");
                if (!rows.sync()) return false;
#pragma unroll
                for (int e = 0; e < 4; ++e) lds4(ex + 2048u * (uint32_t)warp + 512u * e, give[2 * e], give[2 * e + 1]);
#pragma unroll
                for (int e = 0; e < 8; ++e) z[e] = fma2(add2(sn[e], give[e]), s[e], z[e]);
            }
            odd |= (t + 1) * kKT > seen_least;
            uint32_t open = 0xffffu; // bit e: key e is seen
            if (__any_sync(0xffffffffu, odd)) {
                const int n_seen = (int)max((int64_t)0, min((int64_t)16, seen - (t * kKT + key)));
                open = (1u << n_seen) - 1u;
                const uint32_t none = no_value(c.stage(n), sc); // a key without a value has its share of l, and its v is 0
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (__float_as_uint(s[e].x) == kNoKey) open &= ~(1u << (2 * e)), s[e].x = 0.f;
                    if (__float_as_uint(s[e].y) == kNoKey) open &= ~(2u << (2 * e)), s[e].y = 0.f;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    // an unseen key's score: finite, whatever it was
                    if (!(open >> (2 * e) & 1u)) z[e].x = 0.f;
                    if (!(open >> (2 * e) & 2u)) z[e].y = 0.f;
                    if (none >> (2 * e) & 1u) s[e].x = 0.f;
                    if (none >> (2 * e) & 2u) s[e].y = 0.f;
                }
            }
            float pt, vt;
            auto weigh = [&]() {
                const float2 mul = make_float2(cq, cq), sub2 = make_float2(-ref, -ref);
                float2 ps = make_float2(0.f, 0.f), ws = ps;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float2 p = fma2(z[e], mul, sub2);
                    p.x = ex2(p.x);
                    p.y = ex2(p.y);
                    if (odd) {
                        p.x = open >> (2 * e) & 1u ? p.x : 0.f;
                        p.y = open >> (2 * e) & 2u ? p.y : 0.f;
                    }
                    ps = add2(ps, p);
                    v[e] = mul2(p, s[e]);
                    ws = add2(ws, v[e]);
                }
                pt = ps.x + ps.y;
                vt = ws.x + ws.y;
            };
            auto largest = [&]() { // the row's largest z + log2 s of this tile, in this thread
                float zt = -INFINITY;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (open >> (2 * e) & 1u) zt = fmaxf(zt, fmaf(z[e].x, cq, __log2f(fmaxf(s[e].x, kSmallestScale))));
                    if (open >> (2 * e) & 2u) zt = fmaxf(zt, fmaf(z[e].y, cq, __log2f(fmaxf(s[e].y, kSmallestScale))));
                }
                return row_max(zt);
            };
            // weigh with the reference as it is, and again if that turns out to move; a run's first tile sets it first
            uint32_t hi[4], lo[4];
            bool move = true, set = true; // the row's reference; that of some row of the warp
            float least = -INFINITY;      // lower bound of the reference
            if (t > run.t0) {
                weigh();
                // the largest sum of v in a thread of the row, in place of the largest v.  A row without a reference, or whose p
                // grow too large (scales far below those that it was set by), takes one
                put_part(buf, row_max(begun && !(pt > kMostP) ? vt : INFINITY));
                split16<!kStacked>(v, kStacked ? 16.f : 1.f, hi, lo); // while the others arrive; seldom in vain
                if (!rows.wait()) return false;
                get(buf, other);
                const float most = max4(other), some = sum4(other); // (the tile's sum, or at least half of it)
                const bool raise = most > kTop;
                // What rounding may take off this tile's v counts as spent where they are few; with kFew or more, it is at
                // most kAllowed of them.
                const bool few = some < kFew;
                const float lost = few ? fminf(kStacked ? 2.f * some : some, kLost * kKT) : 0.f;
                if (!raise) vs_row += some;
                spent += lost;
                bool low = few && spent > kAllowed * vs_row;
                set = __any_sync(0xffffffffu, raise || low); // (alike in the warps of the rows)
                if (set && __any_sync(0xffffffffu, low)) {
                    if (!put(2, row_sum(vs))) return false;
                    get(2, other);
                    vs_row = sum4(other);
                    low = few && spent > kAllowed * vs_row;
                    if (__any_sync(0xffffffffu, low)) { // the sum of p, which keys without a value may make large, has to stay finite
                        if (!put(buf, row_sum(l))) return false;
                        get(buf, other);
                        least = ref + rintf(__log2f(sum4(other))) - kMostL;
                        low = some < 4.f * kFew && 4.f * spent > kAllowed * vs_row; // rows that are near it come along
                        if (low) spent -= lost;
                    }
                    set = __any_sync(0xffffffffu, raise || low);
                }
                move = raise || low;
            }
            if (set) {
                if (!put(3, largest())) return false;
                get(3, other);
                const float zt = max4(other);
                float f = 1.f;
                if (move && zt > -INFINITY) {
                    const float next = fmaxf(floorf(zt) - kAbove, least); // a whole number: O and the sums move by an exact power of two
                    f = begun ? ex2(ref - next) : 0.f;
                    ref = next;
                    begun = true;
                    l *= f;
                    vs *= f;
                    vs_row *= f;
                    spent *= f;
                }
                if (t > run.t0 && __any_sync(0xffffffffu, f != 1.f)) { // O of the tiles before this one
                    if (!__all_sync(0xffffffffu, c.wait(B_KEMPTY + (n - 1) % kStages, ((n - 1) / kStages) & 1))) return false;
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
                split16<!kStacked>(v, kStacked ? 16.f : 1.f, hi, lo);
            }
            l += pt;
            vs += vt;
            const uint32_t at = c.base + OFF_P + kPTile * (n % kPBufs);
            if constexpr (!kStacked) { // one buffer: O of the tile before has read it
                if (n > 0 && !__all_sync(0xffffffffu, c.wait(B_KEMPTY + (n - 1) % kStages, ((n - 1) / kStages) & 1))) return false;
            }
            if constexpr (kStacked) {
                sts4(at + sw128((uint32_t)(32 * g + r16), (uint32_t)key), hi);
                sts4(at + sw128((uint32_t)(32 * g + 16 + r16), (uint32_t)key), lo);
            } else {
                sts4(at + sw128((uint32_t)row, (uint32_t)key), hi);
                sts4(at + sw128((uint32_t)row, 64u + (uint32_t)key), lo);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive(c.bar(B_P + buf));
        }
    }
    return true;
}

static __device__ __forceinline__ void run(const LatentDecodeArgs &a, const Maps &maps, uint8_t *smem_raw)
{
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *sp = smem_raw + (base - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int64_t(&s_at)[4] = *reinterpret_cast<int64_t(*)[4]>(sp + OFF_AT);
    if (warp == 0) {
        Walk::begin(a, lane, s_at);
    } else if (tid == 64 && maps.box) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.lat));
        asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.rope));
    } else if (tid == 32) {
        for (int b = 0; b < NUM_BARS; ++b) {
            uint32_t count = 1;
            if (b >= B_KFULL && b < B_KFULL + kStages) count = maps.box ? 1 : 128; // TMA; each copying thread's copies, and itself
            if (b == B_P || b == B_P + 1 || b == B_Q || b == B_ALL) count = kSoftThreads;
            if (b == B_ROWS || b == B_ROWS + 1) count = kSoftThreads / 2;
            mbar_init(base + OFF_BAR + 8u * (uint32_t)b, count);
        }
        mbar_init_fence();
        *reinterpret_cast<volatile uint32_t *>(sp + OFF_TMEM + 16) = 0;
    }
    if (warp == kMmaWarp) tmem_alloc(base + OFF_TMEM, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const Ctx c{base, *reinterpret_cast<volatile uint32_t *>(sp + OFF_TMEM)};
    cudaTriggerProgrammaticLaunchCompletion(); // the merge may come up
    const Walk walk(a, s_at);
    volatile uint32_t *issued = reinterpret_cast<volatile uint32_t *>(sp + OFF_TMEM + 16); // tiles asked for
    bool ok = true;
    if (warp < kProdWarp0) {
        regs_inc<kRegsSoft>();
        ok = softmax_role(a, maps, c, walk, warp, lane);
    } else {
        regs_dec<kRegsRest>();
        if (warp == kMmaWarp) {
            if (elect_one()) ok = mma_role(a, maps, c, walk);
        } else if (!maps.box) {
            if (warp < kMmaWarp) ok = copy_role(a, c, walk, warp - kProdWarp0, lane);
        } else if (warp == kProdWarp0) {
            ok = tma_role(a, maps, c, walk, issued, lane);
        } else if (warp == kProdWarp0 + 1) {
            prefetch_role(a, maps, walk, issued, lane);
        }
    }
    if (!ok) flag_error(a.err, CSA_DEVERR_TIMEOUT);
    if (warp == kMmaWarp && elect_one()) { // every MMA completes before TMEM is released
        mma_commit(c.bar(B_FINAL));
        if (!mbar_wait(c.bar(B_FINAL), 0)) flag_error(a.err, CSA_DEVERR_TIMEOUT);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(c.tmem, kTmemCols);
}

};

template <int RB> __global__ void __launch_bounds__(kThreads, 1) latent_decode_tc_kernel(LatentDecodeArgs a, const __grid_constant__ Maps maps)
{
    extern __shared__ uint8_t smem_raw[];
    Decode<RB>::run(a, maps, smem_raw);
}

} // namespace

bool latent_decode_tc_eligible(int R, int rd) { return R == kR && rd == kRd; }

// Blocks of 32 rows where that is all there are, else of 64.  A tile of 128 keys takes 3,050 to 3,400 cycles for 32 rows
// and, as two tiles of 64, 4,600 for 64.
static bool one_block(int Lq, int H) { return Lq * H <= 32; }

size_t latent_decode_tc_workspace(int64_t B, int Lq, int H, int64_t max_len, int *grid, int *par)
{
    if (one_block(Lq, H)) Decode<32>::Split::plan(B, Lq, H, max_len, device_sms(), grid, par);
    else Decode<64>::Split::plan(B, Lq, H, max_len, device_sms(), grid, par);
    return (size_t)*grid * 2 * (one_block(Lq, H) ? latent_part_size<32>(kR) : latent_part_size<64>(kR)) * sizeof(float);
}

// Boxes with the 128-byte swizzle; what lies outside reads as zeros.
static bool encode_u8(CUtensorMap *m, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tma::encoder();
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)rank, const_cast<void *>(base), dims, strides, box, estr,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int RB> static cudaError_t launch(const LatentDecodeArgs &a, cudaStream_t st)
{
    constexpr int kKT = Decode<RB>::kKT;
    // a box is 128 rows of a contiguous run or of pages of whole tiles, or a page of 8, 16, 32 or 64 rows (in groups of 8,
    // as the swizzle has them); other pages are copied row by row: 3,700 cycles of issue a tile where a box takes one
    Maps maps{};
    const int pr = a.map.page_rows;
    const uint64_t n = (uint64_t)a.rows.n;
    maps.page_tiles = 1;
    maps.slice = Decode<RB>::kSlice;
    maps.group = 1024;
    if (n >= 1 && n < (1ull << 31)) { // TMA coordinates are int32
        if (!a.map.pages) maps.box = kKT;
        else if (n % 8 == 0 && (reinterpret_cast<uintptr_t>(a.rows.scale) & 15u) == 0) // whole groups; scales as bulk copies
            maps.box = pr % kKT == 0 ? kKT : (pr == 8 || pr == 16 || pr == 32 || pr == 64) ? pr : 0;
    }
    if (maps.box) {
        const uint32_t rows = (uint32_t)maps.box;
        bool ok;
        if (a.map.pages) {
            maps.n_pages = (uint32_t)(n / pr);
            if (maps.box == kKT) maps.page_tiles = (uint32_t)(pr / kKT);
            else maps.shift = pr == 8 ? 3 : pr == 16 ? 4 : pr == 32 ? 5 : 6;
            maps.slice = 1024;
            maps.group = 4096;
            const cuuint64_t dims[4] = {128, 8, kR / 128, n / 8}, strides[3] = {kR, 128, 8 * kR};
            const cuuint32_t box[4] = {128, 8, kR / 128, rows / 8};
            ok = encode_u8(&maps.lat, a.rows.fp8, 4, dims, strides, box);
        } else {
            const cuuint64_t dims[3] = {128, n, kR / 128}, strides[2] = {kR, 128};
            const cuuint32_t box[3] = {128, rows, kR / 128};
            ok = encode_u8(&maps.lat, a.rows.fp8, 3, dims, strides, box);
        }
        const cuuint64_t dims[2] = {2 * kRd, n}, strides[1] = {2 * kRd};
        const cuuint32_t box[2] = {2 * kRd, rows};
        if (!ok || !encode_u8(&maps.rope, a.rows.rope, 2, dims, strides, box)) return cudaErrorNotSupported;
    }
    static std::atomic<bool> done[64];
    cudaError_t e = prepare_kernel(latent_decode_tc_kernel<RB>, Decode<RB>::SMEM_ALLOC, kRegs, done);
    if (e != cudaSuccess) return e;
    latent_decode_tc_kernel<RB><<<(unsigned)a.grid, kThreads, Decode<RB>::SMEM_ALLOC, st>>>(a, maps);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_latent_merge_tc(a, RB, st);
}

cudaError_t launch_latent_decode_tc(const LatentDecodeArgs &a, cudaStream_t st) { return one_block(a.Lq, a.H) ? launch<32>(a, st) : launch<64>(a, st); }

} // namespace csa

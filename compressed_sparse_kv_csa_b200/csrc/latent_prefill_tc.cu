// latent_prefill_tc.cu -- latent attention in its expanded form on tcgen05, for bf16 heads of
// 128 + 64 key channels and 128 value channels over packed sequences.
//
// One pass over the keys with the running maximum and sum of the softmax (log2 domain, fp32).  A CTA
// takes 256 consecutive queries of one head as two tiles of 128: while one tile's scores are turned
// into probabilities, the tensor cores work on the other's.  Per tile of 128 keys and queries:
//   S = Q K^T   M = 128, N = 128, K = 192, in TMEM (the key's last 64 channels come from k_rope,
//               which all heads share)
//   P = 2^(S scale log2e - m) in bf16, written over the first half of S in TMEM
//   O += P V    M = 128, N = 128, K = 128, P read from TMEM, V read MN-major
// TMEM: S0, S1, O0, O1 of 128 columns each.  The running maximum moves, and O is rescaled in TMEM, only
// when a tile raises it by more than 8 (2^8 fits any of the sums' fp32); S of tile i complete implies
// P V of tile i - 1 complete, since one thread issues both in order, so the rescale needs no wait.
// Rounding P to bf16 (the type of V, which one MMA shares) costs 2^-9 relative a term; the sum is
// taken over the unrounded fp32 values.
//
// Shared memory: Q 96 KB, and a ring of eight 16 KB slots of [128 rows x 64 channels] that the key
// (three slots a tile) and value (two) boxes pass through in order, so that the loads run up to 1.6
// tiles ahead.  Everything arrives by TMA.
// P is handed over in two halves, and one instruction takes the maximum of three: 16k queries and keys of 16 heads 3%
// faster than without.  Where query blocks do not fill the SMs to the end, keys are split (latent_prefill_tc_parts).
// Roles: warps 0-3 and 4-7 softmax, rescale and output of the two query tiles (one row a thread), warp 8
// TMA, warp 9 MMA.  Per pair of query tiles and tile of keys the tensor cores need 2,560 cycles and the chain S - softmax - P V
// of each, beside the other's MMAs, 3,800; in long calls the chip's power limits what is left (990 W, 1.5 GHz): 16k
// x 16 heads causal 0.99 to 1.05 ms in a short run (1.3 PFLOP/s), 1.13 to 1.16 ms in a loop of seconds; 4k 72 us.
// The threads that issue copies and MMAs index a tile's slot numbers at run time, which lie in a stack of 64 to 72 bytes.
#include "latent.cuh"
#include "tc_common.cuh"
#include "tma_host.cuh"

namespace csa {

namespace {

using namespace tc;

constexpr int kDn = 128, kDr = 64, kDv = 128, kT = 128; // kT: queries and keys of a tile
constexpr int kTmaWarp = 8, kMmaWarp = 9, kThreads = 384; // whole warpgroups, for the register split
// A softmax thread holds a row of 128 scores.  Of the registers that the block is launched with (168 a
// thread, checked on the host), the two softmax warpgroups take 208 a thread and the other leaves 88.
constexpr int kRegs = 168, kRegsSoft = 208, kRegsRest = 88;
static_assert(256 * kRegsSoft + 128 * kRegsRest <= kThreads * kRegs, "register split");
constexpr uint32_t kSlot = 16384;
constexpr int kSlots = 8;
constexpr int kParts = 2; // P is handed over in halves, so that P V begins while the rest is computed
constexpr uint32_t OFF_Q = 0, OFF_RING = 2 * 3 * kSlot, OFF_BAR = OFF_RING + kSlots * kSlot, OFF_TMEM = OFF_BAR + 256;
constexpr uint32_t SMEM_ALLOC = OFF_TMEM + 64 + 1024; // slack to align the base to 1024 bytes
static_assert(SMEM_ALLOC <= 232448, "shared memory per block");
enum { B_Q = 0, B_FULL, B_EMPTY = B_FULL + kSlots, B_S = B_EMPTY + kSlots, B_P = B_S + 2, B_O = B_P + 2 * kParts, B_VTAIL = B_O + 2,
       B_FINAL, NUM_BARS };
static_assert(8 * NUM_BARS <= 256, "barrier space");
constexpr uint32_t IDESC_S = idesc_bf16_f32(128, 128, false, false), IDESC_PV = idesc_bf16_f32(128, 128, false, true);
constexpr uint32_t kColS = 0, kColO = 256; // + 128 t
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct Maps {
    CUtensorMap q, kv, kr;
};

// What a CTA does: queries i0 .. of sequence rows [q0, q0 + nq), keys [k0, k0 + nk).
struct Job {
    int64_t q0, k0;
    int h, i0, nq, nk, lag, n[2], tiles; // n[t]: key tiles of query tile t
    int c0;                              // the first of them, behind those of the parts before
};

__device__ __forceinline__ bool find_job(const LatentPrefillArgs &a, int64_t id, int part, int parts, Job &j)
{
    // the query blocks that see the most keys first
    const int per = (int)((a.max_q + 2 * kT - 1) / (2 * kT));
    const int64_t bh = a.B * a.H;
    const int64_t r = id % bh, b = r / a.H;
    j.h = (int)(r % a.H);
    j.i0 = (per - 1 - (int)(id / bh)) * 2 * kT;
    int64_t q1, k1;
    packed_range(a.cu_q, b, a.Tq, &j.q0, &q1);
    packed_range(a.cu_k, b, a.Tk, &j.k0, &k1);
    const int nq = (int)(q1 - j.q0);
    j.nk = (int)(k1 - j.k0);
    j.lag = j.nk - nq;
    j.nq = nq < a.max_q ? nq : (int)a.max_q;
    j.tiles = 0;
    for (int t = 0; t < 2; ++t) {
        const int first = j.i0 + t * kT, last = min(first + kT, j.nq); // queries of the tile
        int64_t seen = first >= j.nq ? 0 : j.nk;
        if (a.causal && first < j.nq) seen = min((int64_t)j.nk, (int64_t)last + j.lag);
        j.n[t] = seen <= 0 ? 0 : (int)((seen + kT - 1) / kT);
        j.tiles = max(j.tiles, j.n[t]);
    }
    j.c0 = 0;
    if (part >= 0) {
        const int c1 = (int)((int64_t)j.tiles * (part + 1) / parts);
        j.c0 = (int)((int64_t)j.tiles * part / parts);
        j.tiles = c1 - j.c0;
#pragma unroll
        for (int t = 0; t < 2; ++t) j.n[t] = max(0, min(j.n[t], c1) - j.c0);
    }
    return j.i0 < j.nq;
}

__device__ __forceinline__ uint32_t pk_bf16(float lo, float hi)
{
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&h);
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

struct Ring { // slot and phase of the next 16 KB box
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next()
    {
        if (++slot == kSlots) slot = 0, phase ^= 1;
    }
};

// TMA (one warp).  The ring's order is K0 V0 K1 V1 ...
__device__ __forceinline__ bool tma_role(const Job &j, const Maps &M, uint32_t base, int lane, uint64_t wait_ns)
{
    const uint32_t bars = base + OFF_BAR;
    auto bar = [&](int b) { return bars + 8u * (uint32_t)b; };
    // nothing is on its way when the block ends, whatever the others waited for: Q, and the last boxes of the `boxes`
    // that went into the ring
    auto drain = [&](uint32_t boxes) {
        bool ok = mbar_wait(bar(B_Q), 0);
        for (uint32_t p = boxes - min(boxes, (uint32_t)kSlots); p < boxes; ++p) ok = mbar_wait(bar(B_FULL + p % kSlots), (p / kSlots) & 1) && ok;
        return ok;
    };
    if (lane == 0) {
        const int nt = j.i0 + kT < j.nq ? 2 : 1;
        mbar_arrive_expect_tx(bar(B_Q), (uint32_t)nt * 3 * kSlot);
        for (int t = 0; t < nt; ++t)
            for (int s = 0; s < 3; ++s)
                tma_load_3d(base + OFF_Q + (uint32_t)(3 * t + s) * kSlot, &M.q, 64 * s, j.h, (int)(j.q0 + j.i0 + t * kT), bar(B_Q));
    }
    Ring r;
    uint32_t lap = 0; // the first lap's slots are empty
    for (int i = 0; i < j.tiles; ++i) {
        const int y = (int)(j.k0 + (int64_t)(j.c0 + i) * kT);
        const int tail = j.nk - (j.c0 + i) * kT; // rows of the sequence in this tile, when less than kT
        int v_slot[2];
        for (int s = 0; s < 5; ++s) {
            const int slot = r.slot;
            if (lap && !__all_sync(0xffffffffu, mbar_wait(bar(B_EMPTY + slot), r.phase ^ 1, wait_ns))) {
                drain(5u * (uint32_t)i + (uint32_t)min(s, 3)); // (the values' boxes go when both their slots are empty)
                return false;
            }
            const uint32_t dst = base + OFF_RING + (uint32_t)slot * kSlot;
            if (s < 3) {
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar(B_FULL + slot), kSlot);
                    if (s < 2) tma_load_3d(dst, &M.kv, 64 * s, j.h, y, bar(B_FULL + slot));
                    else tma_load_2d(dst, &M.kr, 0, y, bar(B_FULL + slot));
                }
            } else {
                v_slot[s - 3] = slot;
            }
            r.next();
            if (r.slot == 0) lap = 1;
        }
        // the lower slot takes channels 0-63, so that the pair reads with one positive stride
        const int lo = min(v_slot[0], v_slot[1]), hi = max(v_slot[0], v_slot[1]);
        const uint32_t vlo = base + OFF_RING + (uint32_t)lo * kSlot, vhi = base + OFF_RING + (uint32_t)hi * kSlot;
        if (tail >= kT) {
            if (lane == 0) {
                mbar_arrive_expect_tx(bar(B_FULL + lo), kSlot);
                tma_load_3d(vlo, &M.kv, kDn, j.h, y, bar(B_FULL + lo));
                mbar_arrive_expect_tx(bar(B_FULL + hi), kSlot);
                tma_load_3d(vhi, &M.kv, kDn + 64, j.h, y, bar(B_FULL + hi));
            }
        } else {
            // the sequence ends in this tile: the values behind it carry probability 0, but may hold
            // anything (0 x NaN is NaN), so they are zeroed before the MMAs may read them
            if (lane == 0) {
                mbar_arrive_expect_tx(bar(B_VTAIL), 2 * kSlot);
                tma_load_3d(vlo, &M.kv, kDn, j.h, y, bar(B_VTAIL));
                tma_load_3d(vhi, &M.kv, kDn + 64, j.h, y, bar(B_VTAIL));
            }
            __syncwarp();
            if (!__all_sync(0xffffffffu, mbar_wait(bar(B_VTAIL), 0, wait_ns))) {
                mbar_wait(bar(B_VTAIL), 0);
                drain(5u * (uint32_t)i + 3u);
                return false;
            }
            for (int e = 8 * tail + lane; e < 8 * kT; e += 32)
                for (int s = 0; s < 2; ++s)
                    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"((s ? vhi : vlo) + 16u * (uint32_t)e), "r"(0) : "memory");
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(B_FULL + lo));
                mbar_arrive(bar(B_FULL + hi));
            }
        }
        __syncwarp();
    }
    return drain(5u * (uint32_t)j.tiles);
}

// MMA issue (one thread).
__device__ __forceinline__ bool mma_role(const Job &j, uint32_t base, uint32_t tmem)
{
    const uint32_t bars = base + OFF_BAR;
    auto bar = [&](int b) { return bars + 8u * (uint32_t)b; };
    if (!mbar_wait(bar(B_Q), 0)) return false;
    tc_fence_after();
    const Desc q_desc(sdesc_sw128(base + OFF_Q, 16, 1024)), ring_desc(sdesc_sw128(base + OFF_RING, 16, 1024));
    Ring r;
    struct Box {
        int slot[3];
    };
    auto take = [&](int n, Box &b) { // the ring's next n slots, loaded
        for (int s = 0; s < n; ++s) {
            if (!mbar_wait(bar(B_FULL + r.slot), r.phase)) return false;
            b.slot[s] = r.slot;
            r.next();
        }
        tc_fence_after();
        return true;
    };
    auto free_slots = [&](int n, const Box &b) { // when the MMAs issued so far have read them
        for (int s = 0; s < n; ++s) mma_commit(bar(B_EMPTY + b.slot[s]));
    };
    auto scores = [&](int t, const Box &k) {
#pragma unroll
        for (int s = 0; s < 3; ++s)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_bf16(tmem + kColS + 128u * t, q_desc.at((uint32_t)(3 * t + s) * kSlot + 32u * kk),
                         ring_desc.at((uint32_t)k.slot[s] * kSlot + 32u * kk), IDESC_S, (s | kk) != 0);
        mma_commit(bar(B_S + t));
    };
    Box k, v;
    if (j.tiles > 0) {
        if (!take(3, k)) return false;
        for (int t = 0; t < 2; ++t)
            if (j.n[t] > 0) scores(t, k);
        free_slots(3, k);
    }
    for (int i = 0; i < j.tiles; ++i) {
        const uint32_t ph = (uint32_t)(i & 1);
        if (!take(2, v)) return false;
        const int lo = min(v.slot[0], v.slot[1]), hi = max(v.slot[0], v.slot[1]);
        const Desc dv(sdesc_sw128(base + OFF_RING + (uint32_t)lo * kSlot, (uint32_t)(hi - lo) * kSlot, 1024));
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (i < j.n[t]) {
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    if (kk % (8 / kParts) == 0) {
                        if (!mbar_wait(bar(B_P + kParts * t + kk / (8 / kParts)), ph)) return false;
                        tc_fence_after();
                    }
                    mma_bf16_ts(tmem + kColO + 128u * t, tmem + kColS + 128u * t + 8u * kk,
                                dv.at(2048u * kk), IDESC_PV, (i | kk) != 0);
                }
                if (i + 1 == j.n[t]) mma_commit(bar(B_O + t));
            }
            if (t == 1) free_slots(2, v);
            if (t == 0 && i + 1 < j.tiles && !take(3, k)) return false;
            if (i + 1 < j.n[t]) scores(t, k);
        }
        if (i + 1 < j.tiles) free_slots(3, k);
    }
    return true;
}

// What a grid's blocks are: none of them split, all, or those behind the first.
enum Keys { kWhole, kSplit, kSome };

// Softmax, rescale and output of query tile t: one row per thread.  Of a part of the keys, the maximum, the sum and O as
// it is go to the part's record.
template <Keys KEYS> __device__ __forceinline__ bool softmax_role(const LatentPrefillArgs &a, const LatentKeyParts &parts, const Job &j, uint32_t base, uint32_t tmem, int warp, int lane)
{
    const uint32_t bars = base + OFF_BAR;
    auto bar = [&](int b) { return bars + 8u * (uint32_t)b; };
    const int t = warp >> 2;
    const uint32_t tw = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t tS = tw + kColS + 128u * t, tO = tw + kColO + 128u * t;
    const int first = j.i0 + t * kT, i = first + 32 * (warp & 3) + lane; // this thread's query
    // the last key it sees, and the last that every query of its tile sees
    const int last = a.causal ? min(j.nk - 1, i + j.lag) : j.nk - 1;
    const int last_all = a.causal ? min(j.nk - 1, first + j.lag) : j.nk - 1;
    // scores are compared before they are scaled: a negative scale turns them round first, and a scale
    // of 0 becomes one that is lost in any score (a hidden score is -inf, and 0 x -inf is NaN)
    const bool turn = a.scale < 0.f;
    const float sl2 = fmaxf(fabsf(a.scale) * kLog2e, 1e-37f);
    float m = -INFINITY, l = 0.f; // maximum in use (scaled, log2 domain), sum
    const int c0 = KEYS != kWhole ? j.c0 : 0;
    for (int c = 0; c < j.n[t]; ++c) {
        if (!__all_sync(0xffffffffu, mbar_wait(bar(B_S + t), (uint32_t)(c & 1)))) return false;
        tc_fence_after();
        float s[kT];
#pragma unroll
        for (int g = 0; g < 4; ++g) tmem_ld32(tS + 32u * g, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * g]));
        tmem_ld_wait();
        if (turn) {
#pragma unroll
            for (int e = 0; e < kT; ++e) s[e] = -s[e];
        }
        if ((c + c0) * kT + kT - 1 > last_all) {
            const int n = last - (c + c0) * kT; // the last visible key of the tile
#pragma unroll
            for (int e = 0; e < kT; ++e) s[e] = e <= n ? s[e] : -INFINITY;
        }
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int e = 4; e + 8 <= kT; e += 8)
#pragma unroll
            for (int u = 0; u < 4; ++u) mx[u] = max3(mx[u], s[e + u], s[e + 4 + u]);
#pragma unroll
        for (int u = 0; u < 4; ++u) mx[u] = fmaxf(mx[u], s[kT - 4 + u]);
        const float mt = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * sl2;
        float f = 1.f;
        if (mt > m + 8.f || m == -INFINITY) {
            f = m == -INFINITY ? 0.f : ex2(m - mt); // O of a row that has seen nothing is 0 (or not yet written)
            m = mt;
        }
        if (c > 0 && __any_sync(0xffffffffu, f != 1.f)) {
            const float fo = l == 0.f ? 1.f : f; // a row without a key so far has O = 0: nothing to scale
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                uint32_t o[32];
                tmem_ld32(tO + 32u * g, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * fo);
                tmem_st32(tO + 32u * g, o);
            }
            tmem_st_wait();
        }
        const float sub = m == -INFINITY ? 0.f : -m;
        const float2 sl2v = make_float2(sl2, sl2), subv = make_float2(sub, sub);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int g = 0; g < kParts; ++g) {
            uint32_t p[64 / kParts];
#pragma unroll
            for (int e = 0; e < 64 / kParts; ++e) {
                const int k = kT / kParts * g + 2 * e;
                float2 z = fma2(make_float2(s[k], s[k + 1]), sl2v, subv);
                z.x = ex2(z.x);
                z.y = ex2(z.y);
                sum[e & 1] = add2(sum[e & 1], z);
                p[e] = pk_bf16(z.x, z.y);
            }
            tmem_st32(tS + (uint32_t)(64 / kParts) * g, p);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(bar(B_P + kParts * t + g));
        }
        l = fmaf(l, f, (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y));
    }
    if (j.n[t] > 0) {
        if (!__all_sync(0xffffffffu, mbar_wait(bar(B_O + t), 0))) return false;
        tc_fence_after();
    }
    if (KEYS == kSplit || (KEYS == kSome && blockIdx.x >= (uint32_t)parts.whole)) {
        float *rec = latent_part<2 * kT>(parts.part, kDv, KEYS == kSplit ? blockIdx.x : blockIdx.x - (uint32_t)parts.whole);
        const int row = t * kT + 32 * (warp & 3) + lane;
        if (i < j.nq) *reinterpret_cast<float2 *>(rec + 2 * row) = make_float2(l == 0.f ? -INFINITY : m == -INFINITY ? 0.f : m, l);
        if (j.n[t] > 0) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                uint32_t o[32];
                tmem_ld32(tO + 32u * g, o);
                tmem_ld_wait();
                if (i < j.nq)
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<uint4 *>(rec + latent_part_at<2 * kT>(row, 32 * g + e)) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
        }
        tc_fence_before();
        return true;
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    const int64_t row = (j.q0 + i) * a.H + j.h;
    uint4 *out = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.o) + row * kDv);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        uint32_t o[32];
        if (j.n[t] > 0) {
            tmem_ld32(tO + 32u * g, o);
            tmem_ld_wait();
        }
        if (i < j.nq) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t w[4] = {0, 0, 0, 0};
                if (l != 0.f) {
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        w[u] = pk_bf16(__uint_as_float(o[8 * e + 2 * u]) * inv, __uint_as_float(o[8 * e + 2 * u + 1]) * inv);
                }
                out[4 * g + e] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
    if (a.lse && i < j.nq) a.lse[row] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
    tc_fence_before();
    return true;
}

template <Keys KEYS>
__global__ void __launch_bounds__(kThreads, 1) latent_prefill_tc_kernel(LatentPrefillArgs a, const __grid_constant__ Maps maps, LatentKeyParts parts)
{
    extern __shared__ uint8_t smem_raw[];
    if constexpr (KEYS != kWhole) cudaTriggerProgrammaticLaunchCompletion(); // the merge may come up
    Job j;
    int64_t block = blockIdx.x;
    int part = -1;
    if (KEYS == kSplit || (KEYS == kSome && block >= parts.whole)) {
        const uint32_t i = (uint32_t)(KEYS == kSplit ? block : block - parts.whole);
        part = (int)(i % (uint32_t)parts.n);
        block = (KEYS == kSplit ? 0 : parts.whole) + i / (uint32_t)parts.n;
    }
    if (!find_job(a, block, part, parts.n, j)) return; // no queries here (the same on every thread)
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *sp = smem_raw + (base - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int b = 0; b < NUM_BARS; ++b) mbar_init(base + OFF_BAR + 8u * (uint32_t)b, b >= B_P && b < B_O ? 128u : 1u);
        mbar_init_fence();
    }
    if (warp == kMmaWarp) tmem_alloc(base + OFF_TMEM, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(sp + OFF_TMEM);
    bool ok = true;
    if (warp < kTmaWarp) {
        regs_inc<kRegsSoft>();
        ok = softmax_role<KEYS>(a, parts, j, base, tmem, warp, lane);
    } else {
        regs_dec<kRegsRest>();
        if (warp == kTmaWarp) ok = tma_role(j, maps, base, lane, parts.wait_ns);
        else if (warp == kMmaWarp && elect_one()) ok = mma_role(j, base, tmem);
    }
    if (!ok) flag_error(a.err, CSA_DEVERR_TIMEOUT);
    if (warp == kMmaWarp && elect_one()) { // every MMA completes before TMEM is released
        mma_commit(base + OFF_BAR + 8u * B_FINAL);
        if (!mbar_wait(base + OFF_BAR + 8u * B_FINAL, 0)) flag_error(a.err, CSA_DEVERR_TIMEOUT);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// Merge of a block's key parts, 16 rows x 128 channels a CTA: with part i holding the maximum m_i, the sum l_i and O_i,
// o = sum 2^(m_i - m) O_i / l, l = sum 2^(m_i - m) l_i, m = max m_i.  Bound by the latency of its loads.
constexpr int kMergeRows = 16;
__global__ void __launch_bounds__(32 * kMergeRows) latent_prefill_merge_kernel(LatentPrefillArgs a, LatentKeyParts parts)
{
    constexpr int kBlocks = 2 * kT / kMergeRows;
    // four rows of eight fours of channels a warp
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = (int)(blockIdx.x % kBlocks) * kMergeRows + 4 * (warp >> 2) + (lane & 3), ch = 32 * (warp & 3) + 4 * (lane >> 2);
    const int64_t block = blockIdx.x / kBlocks; // of those that are split
    Job j;
    const bool there = find_job(a, parts.whole + block, -1, 1, j) && j.i0 + r < j.nq;
    cudaGridDependencySynchronize(); // every block waits: what follows in the stream waits for this kernel alone
    if (!there) return;
    const int64_t step = latent_part_size<2 * kT>(kDv);
    const float *rec = latent_part<2 * kT>(parts.part, kDv, block * parts.n);
    float m = -INFINITY, l = 0.f;
#pragma unroll 8
    for (int k = 0; k < parts.n; ++k) m = fmaxf(m, __ldcg(rec + k * step + 2 * r));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const int at = latent_part_at<2 * kT>(r, ch);
    for (int k0 = 0; k0 < parts.n; k0 += 4) {
        float2 ml[4];
        float4 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float *p = rec + min(k0 + e, parts.n - 1) * step;
            ml[e] = __ldcg(reinterpret_cast<const float2 *>(p + 2 * r));
            v[e] = __ldcg(reinterpret_cast<const float4 *>(p + at));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (k0 + e >= parts.n || ml[e].x == -INFINITY) continue; // nothing was seen there, or nothing was written
            const float w = exp2f(ml[e].x - m);
            l = fmaf(w, ml[e].y, l);
            acc.x = fmaf(w, v[e].x, acc.x);
            acc.y = fmaf(w, v[e].y, acc.y);
            acc.z = fmaf(w, v[e].z, acc.z);
            acc.w = fmaf(w, v[e].w, acc.w);
        }
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    const int64_t row = (j.q0 + j.i0 + r) * a.H + j.h;
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.o) + row * kDv + ch) =
        make_uint2(pk_bf16(acc.x * inv, acc.y * inv), pk_bf16(acc.z * inv, acc.w * inv));
    if (a.lse && ch == 0) a.lse[row] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

// A packed bf16 array [rows, heads, cols] read in boxes of 64 columns of one head x 128 rows with the
// 128-byte swizzle; rows outside read as zeros.
bool encode_heads(CUtensorMap *m, const void *base, int64_t rows, int heads, int cols)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tma::encoder();
    if (!enc || rows <= 0) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)cols * 2, (cuuint64_t)cols * 2 * heads};
    const cuuint32_t box[3] = {64, 1, kT}, estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

} // namespace

bool latent_prefill_tc_eligible(const LatentPrefillArgs &a, int dtype)
{
    return dtype == CSA_BF16 && a.dn == kDn && a.dr == kDr && a.dv == kDv && a.Tk > 0;
}

static int64_t query_blocks(const LatentPrefillArgs &a) { return a.B * a.H * ((a.max_q + 2 * kT - 1) / (2 * kT)); }

// Which blocks' keys are split, and into how many parts, so that the SMs are busy to the end: of the blocks behind the last
// full round of all SMs the keys are cut into the number of parts that takes the least time, by the time of a key tile,
// what a CTA takes beside its tiles, and what the partials cost to write, read and merge.  The lengths are
// taken as the average's.  With as many queries as keys, causal blocks differ so much that the short ones fill the last
// round by themselves: full rounds are then followed by none that is split.
//   256 queries of 16 heads (16 blocks) after 64k keys: 150 us in 9 parts, 914 whole; after 2k: 20 in 4, 36 whole;
//   80 blocks after 8k: 116 in 3, 126 whole; 100 blocks: 129 whole, 141 in 4;
//   2,560 queries of 16 heads, the last of 8k keys (148 blocks whole, 12 in 12): 147 us, 191 whole;
//   3 x 1,024, the last of 4k (148 whole, 44 in 3): 105, 118 whole; 2 x 2,048 after 14k: 487 whole, 505 with 108 blocks in 4.
LatentKeyParts latent_prefill_tc_parts(const LatentPrefillArgs &a)
{
    constexpr double kTile = 1.9, kCta = 10, kMerge = 6, kPartial = 0.06; // us
    const int64_t blocks = query_blocks(a), sms = device_sms(), nk = a.Tk / a.B, nq = a.Tq / a.B;
    const LatentKeyParts none{nullptr, 0, 1, 0};
    const int64_t whole = blocks / sms * sms, rest = blocks - whole;
    if (blocks >= ((int64_t)1 << 31) || rest == 0 || (whole > 0 && 2 * nq > nk) || whole > 8 * sms) return none;
    const double tiles = (double)(nk > nq ? nk - nq / 2 : nk) / kT;
    LatentKeyParts best = none;
    double least = 0.95 * (tiles * kTile + kCta);
    for (int n = 2; n <= sms && 3.5 * n <= tiles; ++n) {
        const double rounds = (double)((rest * n + sms - 1) / sms), t = rounds * (tiles / n * kTile + kCta) + kMerge + kPartial * (double)(rest * n);
        if (t < least) least = t, best.whole = (int)whole, best.n = n;
    }
    return best;
}
size_t latent_prefill_tc_workspace(const LatentPrefillArgs &a)
{
    const LatentKeyParts p = latent_prefill_tc_parts(a);
    return p.n < 2 ? 0 : (size_t)((query_blocks(a) - p.whole) * p.n * latent_part_size<2 * kT>(kDv)) * sizeof(float);
}

template <Keys KEYS> static cudaError_t launch(const LatentPrefillArgs &a, const Maps &maps, const LatentKeyParts &parts, int64_t ctas, cudaStream_t st)
{
    static std::atomic<bool> done[64];
    cudaError_t e = prepare_kernel(latent_prefill_tc_kernel<KEYS>, SMEM_ALLOC, kRegs, done);
    if (e != cudaSuccess) return e;
    latent_prefill_tc_kernel<KEYS><<<(unsigned)ctas, kThreads, SMEM_ALLOC, st>>>(a, maps, parts);
    return cudaGetLastError();
}

cudaError_t launch_latent_prefill_tc(const LatentPrefillArgs &a, const LatentKeyParts &parts, cudaStream_t st)
{
    Maps maps;
    if (!encode_heads(&maps.q, a.q, a.Tq, a.H, kDn + kDr) || !encode_heads(&maps.kv, a.kv, a.Tk, a.H, kDn + kDv) ||
        !tma::encode_bf16_rows(&maps.kr, a.k_rope, (uint64_t)a.Tk, kDr, kT))
        return cudaErrorNotSupported;
    const int64_t blocks = query_blocks(a);
    if (blocks >= ((int64_t)1 << 31)) return cudaErrorInvalidValue;
    if (parts.n < 2) return launch<kWhole>(a, maps, parts, blocks, st);
    const int64_t ctas = parts.whole + (blocks - parts.whole) * parts.n;
    cudaError_t e = parts.whole ? launch<kSome>(a, maps, parts, ctas, st) : launch<kSplit>(a, maps, parts, ctas, st);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{}; // its blocks come up while the parts are written, and wait for them
    cfg.gridDim = dim3((unsigned)((blocks - parts.whole) * (2 * kT / kMergeRows)));
    cfg.blockDim = dim3(32 * kMergeRows);
    cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, latent_prefill_merge_kernel, a, parts);
}

} // namespace csa

// latent.cuh -- arguments and the work schedule shared by the latent attention kernels: a cache of
// one row per token (R latent channels in FP8 with a row scale, rd rotated channels in BF16;
// csa_kv_rows with c = R + rd, rope_dims = rd), written by latent_append, read back by
// latent_gather and attended by latent_attn_decode (absorbed form); latent_attn_prefill attends
// the expanded keys and values.
#pragma once

#include <atomic>

#include "common.cuh"

namespace csa {

// Where the row of position s of sequence b lies: through a page table, or at off[b] + s.
struct RowMap {
    const int32_t *pages; // [B, max_pages] or null
    const int64_t *off;   // [B] when pages is null
    int max_pages, page_rows;
    int64_t n; // rows of the cache

    // Row of position s, or -1 when the table or the cache does not hold it.
    __device__ __forceinline__ int64_t row(int64_t b, int64_t s) const
    {
        const int64_t r = paged_row(pages, max_pages, page_rows, b, s, pages ? 0 : off[b]);
        return r >= 0 && r < n ? r : -1;
    }
    // The same in two steps for positions below 2^31 (32-bit division), the load apart from its use: nothing touches
    // the loaded page number, so nothing waits for it.  `first` is the sequence's off[b] (0 with pages).
    __device__ __forceinline__ int64_t first(int64_t b) const { return pages ? 0 : off[b]; }
    __device__ __forceinline__ int32_t page(int64_t b, uint32_t s) const
    {
        int32_t p = -1;
        if (pages) {
            const uint32_t i = s / (uint32_t)page_rows;
            if (i < (uint32_t)max_pages) p = __ldg(pages + b * max_pages + i);
        }
        return p;
    }
    __device__ __forceinline__ int64_t row(int32_t page, int64_t first, uint32_t s) const
    {
        const int64_t r = pages ? (page < 0 ? -1 : (int64_t)page * page_rows + s % (uint32_t)page_rows) : first + s;
        return r >= 0 && r < n ? r : -1;
    }
};

struct LatentAppendArgs {
    const void *x;
    int64_t n, B;
    const float *g;
    float eps;
    double base; // 0: the rotated part is stored as given
    const int64_t *pos;
    const int32_t *seq; // null: row i belongs to sequence i
    RowMap map;
    KvRowsDev out;
    int *err;
};
cudaError_t launch_latent_append(const LatentAppendArgs &a, int in_dtype, cudaStream_t st);

struct LatentGatherArgs {
    KvRowsDev rows;
    const int64_t *cu, *start;
    int64_t B, n_out;
    RowMap map;
    void *lat, *rope;
    int *err;
};
cudaError_t launch_latent_gather(const LatentGatherArgs &a, int out_dtype, cudaStream_t st);

struct LatentDecodeArgs {
    const uint16_t *q; // [B, Lq, H, R + rd] bf16
    KvRowsDev rows;
    const int64_t *pos; // position of each sequence's first new token
    RowMap map;
    float scale;
    int64_t B;
    int Lq, H;
    int64_t max_len;
    uint16_t *o; // [B, Lq, H, R] bf16
    float *lse;  // [B, Lq, H] or null
    float *part; // partials: 2 slots per CTA (latent_part)
    int grid;    // CTAs of the split
    int par;     // CTAs side by side on the same keys, one for each row block; 1: a CTA's runs may be of any row block
    int *err;
    uint64_t wait_ns; // limit of the waits of the warps that copy (one in the other roles too cost up to 10%)
};

// Positions token j of a sequence sees (0 .. result - 1).
__device__ __forceinline__ int64_t latent_visible(const LatentDecodeArgs &a, int64_t b, int j)
{
    int64_t p = a.pos[b];
    p = (p < a.max_len ? p : a.max_len) + j + 1;
    return p < 0 ? 0 : (p < a.max_len ? p : a.max_len);
}

// A partial: the rows' (maximum, sum), then their outputs, four channels of all rows beside one another, so that the lanes
// of a warp write whole sectors where they hold rows, and read them where they hold four rows of eight such fours.
template <int RB> __host__ __device__ __forceinline__ int64_t latent_part_size(int R) { return (int64_t)RB * (R + 4); } // floats
template <int RB> __device__ __forceinline__ float *latent_part(float *part, int R, int64_t slot) { return part + slot * latent_part_size<RB>(R); }
template <int RB> __device__ __forceinline__ int latent_part_at(int row, int ch) { return 4 * RB + ((ch >> 2) * RB + row) * 4 + (ch & 3); }

// x / y of numbers that are not negative, in 32 bits where they fit (a fifth of the time).
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y)
{
    return ((x | y) >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
}

// The split of a decode call: every (sequence, block of RB query rows) is a run of key tiles, and all runs lie one
// behind another.  With par = 1 CTA i of G takes the tiles [i T / G, (i + 1) T / G) of them.  With par =
// the row blocks of a sequence, the runs are those of one row block, G / par groups of CTAs share them
// so, and CTA rb of a group has row block rb: the row blocks walk the same keys at the same time, so that
// memory is read once for all of them (one after another, a long sequence's keys have left L2 in
// between: 4 x 1M keys x 64 heads, two row blocks, read 5.4 GB instead of 2.7).  Either way the work is even
// whatever the lengths are, and a CTA cuts at most the two runs at its ends: its run that starts inside
// goes to slot 2i, the one that starts at its first tile but does not end here to slot 2i + 1; a run that
// lies in one CTA is finished there.  A sequence that sees nothing has one (empty) tile, so its rows are
// written too.  What a run costs beside its tiles -- queries in, output out, the first tile's references -- counts as
// COST tiles in front of its own (64 sequences of 1k to 16k keys: the CTAs with the short ones took 80 us where
// the median took 54).
template <int RB, int KT, int COST> struct LatentSplit {
    static constexpr int kCost = COST;
    static __device__ __forceinline__ int64_t tiles(const LatentDecodeArgs &a, int64_t b)
    {
        const int64_t t = (latent_visible(a, b, a.Lq - 1) + KT - 1) / KT;
        return t < 1 ? 1 : t;
    }
    static __host__ __device__ __forceinline__ int64_t row_blocks(int Lq, int H) { return ((int64_t)Lq * H + RB - 1) / RB; }
    // Grid and par for at most `most` CTAs; side by side where that leaves at most a tenth of them idle.  Of short work only as
    // many CTAs as keep the largest share as it is: the SMs left over bring up the merge meanwhile, and it has fewer
    // parts to read (1 x 32k keys x 16 heads: 31 us with 148 CTAs, 21 with 130).
    static void plan(int64_t B, int Lq, int H, int64_t max_len, int most, int *grid, int *par)
    {
        const int64_t nrb = row_blocks(Lq, H), t = (max_len + KT - 1) / KT, tiles = B * (t < 1 ? 1 : t); // a CTA for each tile at most
        const bool side = nrb <= most && most / nrb * nrb * 10 >= 9 * (int64_t)most;
        *par = side ? (int)nrb : 1;
        const int64_t runs = side ? B : B * nrb, work = side ? tiles : tiles * nrb, groups = most / *par;
        const int64_t places = work + COST * runs, share = (places + groups - 1) / groups, few = share <= 8 ? (places + share - 1) / share : groups;
        const int64_t n = work < few ? work : few;
        *grid = (int)((n < groups ? n : groups) * *par);
    }
    static __device__ __forceinline__ int64_t length(const LatentDecodeArgs &a, int64_t b) { return tiles(a, b) + COST; }
    // Lengths of the runs of the sequences [b0, b1), one warp.
    static __device__ __forceinline__ int64_t warp_total(const LatentDecodeArgs &a, int64_t b0, int64_t b1, int lane)
    {
        int64_t s = 0;
        for (int64_t b = b0 + lane; b < b1; b += 32) s += length(a, b);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        return s;
    }
    // The sequence whose nrb runs hold place `at`, and the length before them; one warp, every lane returns the same.
    static __device__ __forceinline__ void warp_find(const LatentDecodeArgs &a, int64_t at, int64_t nrb, int lane,
                                                     int64_t *b_out, int64_t *before)
    {
        int64_t base = 0;
        for (int64_t b0 = 0; b0 < a.B; b0 += 32) {
            int64_t v = b0 + lane < a.B ? length(a, b0 + lane) * nrb : 0, inc = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t u = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += u;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, base + inc > at);
            if (hit) {
                const int l = __ffs(hit) - 1;
                *b_out = b0 + l;
                *before = base + __shfl_sync(0xffffffffu, inc - v, l);
                return;
            }
            base += __shfl_sync(0xffffffffu, inc, 31);
        }
        *b_out = a.B;
        *before = base;
    }
};

// A part of a run.
struct LatentRun {
    int64_t b, t0, t1; // sequence, first tile and end of the part that lies here
    int rb;            // row block
    bool whole, first; // the run lies here entirely; its first tile lies here
};

// A CTA's walk over its runs.  One warp finds where it begins (begin()); then every role walks by itself.
template <class Split> struct LatentWalk {
    int64_t at, end, b, before, nrb; // nrb: row blocks within the runs (1 side by side)
    int rb0;                         // the CTA's row block side by side
    static __device__ __forceinline__ void begin(const LatentDecodeArgs &a, int lane, int64_t (&out)[4])
    {
        const int64_t nrb = a.par > 1 ? 1 : Split::row_blocks(a.Lq, a.H), G = gridDim.x / a.par, i = blockIdx.x / a.par;
        const int64_t T = Split::warp_total(a, 0, a.B, lane) * nrb, at = quotient(T * i, G);
        int64_t b, before;
        Split::warp_find(a, at, nrb, lane, &b, &before);
        if (lane == 0) out[0] = b, out[1] = before, out[2] = at, out[3] = quotient(T * (i + 1), G);
    }
    __device__ __forceinline__ LatentWalk(const LatentDecodeArgs &a, const int64_t (&from)[4])
    {
        nrb = a.par > 1 ? 1 : Split::row_blocks(a.Lq, a.H);
        rb0 = (int)(blockIdx.x % a.par);
        b = from[0];
        before = from[1];
        at = from[2];
        end = from[3];
    }
    __device__ __forceinline__ bool next(const LatentDecodeArgs &a, LatentRun &r)
    {
        while (at < end && b < a.B) {
            const int64_t tiles = Split::tiles(a, b), length = tiles + Split::kCost;
            int64_t in = at - before;
            r.b = b;
            r.rb = rb0;
            if (nrb > 1) {
                r.rb = (int)quotient(in, length);
                in -= r.rb * length;
            }
            const int64_t out = min(length, in + (end - at));
            r.t0 = max((int64_t)0, in - Split::kCost);
            r.t1 = max((int64_t)0, out - Split::kCost);
            r.first = r.t0 == 0;
            r.whole = r.first && r.t1 == tiles;
            at += out - in;
            if (out == length && (nrb == 1 || r.rb + 1 == nrb)) {
                before += length * nrb;
                ++b;
            }
            if (r.t0 < r.t1) return true; // else only of what counts in front of the tiles
        }
        return false;
    }
};

// Shared memory and, for a kernel that splits its registers between warpgroups (regs > 0), the registers that
// it was compiled to (another number would let the split wait for ever): set and checked once for each device.
template <class Kernel> inline cudaError_t prepare_kernel(Kernel kernel, size_t smem, int regs, std::atomic<bool> (&done)[64])
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (regs > 0) {
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, kernel);
        if (e != cudaSuccess) return e;
        if (fa.numRegs != regs) return cudaErrorInvalidConfiguration;
    }
    if (dev < 64) done[dev].store(true, std::memory_order_release);
    return cudaSuccess;
}

cudaError_t launch_latent_decode_generic(LatentDecodeArgs a, cudaStream_t st);
size_t latent_decode_generic_workspace(int64_t B, int Lq, int H, int R, int64_t max_len, int *grid, int *par);

// 512 + 64 channels on the tensor cores (blocks of 32 rows with tiles of 128 keys, or of 64 with 64).
bool latent_decode_tc_eligible(int R, int rd);
size_t latent_decode_tc_workspace(int64_t B, int Lq, int H, int64_t max_len, int *grid, int *par);
cudaError_t launch_latent_decode_tc(const LatentDecodeArgs &a, cudaStream_t st);
cudaError_t launch_latent_merge_tc(const LatentDecodeArgs &a, int rows, cudaStream_t st);

struct LatentPrefillArgs {
    const void *q, *kv, *k_rope; // [Tq, H, dn + dr], [Tk, H, dn + dv], [Tk, dr]
    const int64_t *cu_q, *cu_k;  // [B + 1]
    int64_t B, Tq, Tk, max_q;
    int H, dn, dr, dv;
    float scale;
    int causal;
    void *o;    // [Tq, H, dv]
    float *lse; // [Tq, H] or null
    int *err;
};
struct LatentKeyParts {
    float *part; // their partials (latent_part of 256 rows), block after block
    int whole;   // blocks of queries whose keys are not split
    int n;       // parts of each of the others; 1: there are none
    uint64_t wait_ns; // as above (here, since two words more in the arguments above slowed the kernel by 7%)
};

// The rows of sequence b in a packed array of T rows.
__device__ __forceinline__ void packed_range(const int64_t *cu, int64_t b, int64_t T, int64_t *beg, int64_t *end)
{
    const int64_t s = cu[b], e = cu[b + 1];
    *beg = s < 0 ? 0 : (s < T ? s : T);
    *end = e < *beg ? *beg : (e < T ? e : T);
}

bool latent_prefill_tc_eligible(const LatentPrefillArgs &a, int dtype);
LatentKeyParts latent_prefill_tc_parts(const LatentPrefillArgs &a);
size_t latent_prefill_tc_workspace(const LatentPrefillArgs &a);
cudaError_t launch_latent_prefill_tc(const LatentPrefillArgs &a, const LatentKeyParts &parts, cudaStream_t st);
cudaError_t launch_latent_prefill_generic(const LatentPrefillArgs &a, int dtype, cudaStream_t st);

} // namespace csa

// latent_rows.cu -- writing and reading back the latent cache: latent_append (RMSNorm of the latent
// part, rotary embedding of the rest, quantise on write at (sequence, position)) and latent_gather
// (rows of ragged runs of positions, dequantised, packed for the expanded form's projection).
//
// Both are HBM-bound: append reads 2c bytes (bf16) and writes R + 2 rd + 4 a row, gather the other
// way round.  A lane holds 8 consecutive channels of a row, so that loads and stores of bf16 are 16 bytes a
// lane beside its neighbour's.  Measured, 512 + 64 channels in pages of 128: append of 65,536 bf16 rows 34 us
// (3.5 TB/s), fp32 39 us; gather of 190,000 rows 61 us (5.6 TB/s), to fp32 95 us (5.9 TB/s).  The append is bound by latency: a
// warp's next rows are asked for when the last are done (285 instructions a row, issued in 52% of the cycles).
#include "latent.cuh"
#include "tc_common.cuh"

namespace csa {

namespace {

using namespace tc;

constexpr double kTwoPi = 6.283185307179586476925287;

// 8 channels as they are stored.
template <typename T> struct Raw8;
template <> struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = __ldcs(reinterpret_cast<const float4 *>(p));
        b = __ldcs(reinterpret_cast<const float4 *>(p + 4));
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float2 (&v)[4]) const
    {
        v[0] = make_float2(a.x, a.y), v[1] = make_float2(a.z, a.w), v[2] = make_float2(b.x, b.y), v[3] = make_float2(b.z, b.w);
    }
};
template <> struct Raw8<uint16_t> {
    uint4 u;
    __device__ __forceinline__ void load(const uint16_t *p) { u = __ldcs(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float2 (&v)[4]) const
    {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
};

__device__ __forceinline__ float2 pair_of(const float *p) { return __ldcs(reinterpret_cast<const float2 *>(p)); }
__device__ __forceinline__ float2 pair_of(const uint16_t *p)
{
    const uint32_t w = __ldcs(reinterpret_cast<const uint32_t *>(p));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// 8 values over the row's scale as E4M3 codes, each the code of the IEEE quotient v / sc, as the library's other
// quantisers take it.  One reciprocal serves the row: with inv = 1 / sc rounded to nearest, q = v inv, r = v - q sc (exact
// in a fused multiply-add) and q + r inv is the correctly rounded quotient (Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990) as long as nothing leaves the normal range: scales outside
// 2^-90 .. 2^90 are divided one by one.
__device__ __forceinline__ uint2 encode8(const float2 (&v)[4], float sc, float inv, bool plain)
{
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float2 q;
        if (plain) {
            const float2 i2 = make_float2(inv, inv);
            q = mul2(v[e], i2);
            q = fma2(fma2(q, make_float2(-sc, -sc), v[e]), i2, q);
        } else {
            q = make_float2(__fdiv_rn(v[e].x, sc), __fdiv_rn(v[e].y, sc));
        }
        w[e >> 1] |= (uint32_t)__nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3) << (16 * (e & 1));
    }
    // -0 is stored as +0: a sign stays where the other seven bits are not all zero
    auto plus0 = [](uint32_t c) { return c & ((((c & 0x7f7f7f7fu) + 0x7f7f7f7fu) & 0x80808080u) | 0x7f7f7f7fu); };
    return make_uint2(plus0(w[0]), plus0(w[1]));
}

// Sums (or maxima) over the warp of four values, one a row: lane l returns that of row 2 (l / 16) + (l / 8) % 2.  Six
// shuffles for the four.
template <class Op> __device__ __forceinline__ float reduce(const float (&v)[4], int lane, Op op)
{
    const bool hi = lane & 16, odd = lane & 8;
    const float a = op(hi ? v[2] : v[0], __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], 16));
    const float b = op(hi ? v[3] : v[1], __shfl_xor_sync(0xffffffffu, hi ? v[1] : v[3], 16));
    float c = op(odd ? b : a, __shfl_xor_sync(0xffffffffu, odd ? a : b, 8));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) c = op(c, __shfl_xor_sync(0xffffffffu, c, o));
    return c;
}
template <class Op> __device__ __forceinline__ float reduce(const float (&v)[1], int, Op op)
{
    float c = v[0];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) c = op(c, __shfl_xor_sync(0xffffffffu, c, o));
    return c;
}
template <int N> __device__ __forceinline__ float of_row(float v, int r) { return N == 1 ? v : __shfl_sync(0xffffffffu, v, 16 * (r >> 1) + 8 * (r & 1)); }

// A warp takes `per` rows, kBatch = 4 at once (or one, where that is all): their loads are in flight together, their
// places are looked up side by side (a lane each), what a row needs once -- a root, three divisions -- is computed by
// different lanes for the four, and no branch between the rows keeps their chains apart.  Lane l holds channels
// 8 l + 256 k .. + 7, k < NV.  64k rows of 512 + 64 bf16 channels: 63 us one row at a time, 38 with a branch a row, 34.
//
// The rotation of pair i at position p is by p * base^(-2i/rd).  The frequency of a lane's pair is computed once for all
// rows, in 64-bit floating point, as a fraction of a turn of 64 bits; a 64-bit product with the position drops
// the whole turns by itself, and the sine and cosine of what is left are taken in 32 bits.
template <typename Tin, int NV, int kBatch> __global__ void __launch_bounds__(256, NV > 2 ? 1 : 2) latent_append_kernel(LatentAppendArgs a, double log_base, int per)
{
    const int lane = threadIdx.x & 31;
    const int64_t i0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * per;
    const int cnt = (int)min((int64_t)per, a.n - i0), rd = a.out.rope_dims, R = a.out.c - rd;
    if (cnt <= 0) return;
    const Tin *x = static_cast<const Tin *>(a.x) + i0 * a.out.c;
    int64_t my_pos = -1, my_row = -1;
    if (lane < cnt) {
        my_pos = a.pos[i0 + lane];
        const int64_t b = a.seq ? a.seq[i0 + lane] : i0 + lane;
        if (my_pos >= 0) {
            if (b >= 0 && b < a.B) {
                // (a position below 2^31 is divided in 32 bits)
                my_row = my_pos >> 31 ? a.map.row(b, my_pos) : a.map.row(a.map.page(b, (uint32_t)my_pos), a.map.first(b), (uint32_t)my_pos);
            }
            if (my_row < 0) flag_error(a.err, CSA_DEVERR_INDEX);
        }
    }
    auto turns_of = [&](int k) { return (uint64_t)(exp(-(2.0 * k / rd) * log_base) / kTwoPi * 18446744073709551616.0); }; // pair k, a position
    uint64_t turns = 0;
    if (a.base > 0 && 2 * lane < rd) turns = turns_of(lane);
    for (int r0 = 0; r0 < cnt; r0 += kBatch) {
        Raw8<Tin> raw[kBatch][NV];
        float2 pair[kBatch];
#pragma unroll
        for (int r = 0; r < kBatch; ++r) {
            const Tin *xr = x + (int64_t)(r0 + r) * a.out.c;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int j = 8 * (lane + 32 * k);
                if (r0 + r < cnt && j < R) raw[r][k].load(xr + j);
                else raw[r][k].zero();
            }
            pair[r] = make_float2(0.f, 0.f);
            if (r0 + r < cnt && 2 * lane < rd) pair[r] = pair_of(xr + R + 2 * lane);
        }
        int64_t row[kBatch]; // negative: skipped, refused or not there
#pragma unroll
        for (int r = 0; r < kBatch; ++r) row[r] = r0 + r < cnt ? __shfl_sync(0xffffffffu, my_row, (r0 + r) & 31) : -1;
        // (no branch a row: the four rows' chains run beside one another)
        uint64_t p[kBatch];
#pragma unroll
        for (int r = 0; r < kBatch; ++r) p[r] = (uint64_t)__shfl_sync(0xffffffffu, my_pos, (r0 + r) & 31);
        auto rotate = [](float2 v, uint64_t t) {
            float sn, cs;
            sincospif((float)(int32_t)(t >> 32) * 4.656612873077393e-10f, &sn, &cs); // half turns, -1 .. 1
            return make_float2(fmaf(v.x, cs, -v.y * sn), fmaf(v.x, sn, v.y * cs));
        };
        auto put = [&](int r, int k, float2 v) {
            if (row[r] >= 0)
                *reinterpret_cast<uint32_t *>(a.out.rope + row[r] * rd + 2 * k) = uint32_t(f32_to_bf16_bits(v.x)) | (uint32_t(f32_to_bf16_bits(v.y)) << 16);
        };
        if (2 * lane < rd) {
            if (a.base > 0) {
#pragma unroll
                for (int r = 0; r < kBatch; ++r) pair[r] = rotate(pair[r], p[r] * turns);
            }
#pragma unroll
            for (int r = 0; r < kBatch; ++r) put(r, lane, pair[r]);
        }
        for (int k = lane + 32; 2 * k < rd; k += 32) { // more than 64 rotated channels
            const uint64_t t = a.base > 0 ? turns_of(k) : 0;
#pragma unroll
            for (int r = 0; r < kBatch; ++r) {
                if (row[r] < 0) continue;
                const float2 u = pair_of(x + (int64_t)(r0 + r) * a.out.c + R + 2 * k);
                put(r, k, a.base > 0 ? rotate(u, p[r] * t) : u);
            }
        }
        float2 v[kBatch][NV][4];
#pragma unroll
        for (int r = 0; r < kBatch; ++r)
#pragma unroll
            for (int k = 0; k < NV; ++k) raw[r][k].get(v[r][k]);
        auto row_amax = [&](float (&m)[kBatch]) { // this lane's share
#pragma unroll
            for (int r = 0; r < kBatch; ++r) {
                m[r] = 0.f;
#pragma unroll
                for (int k = 0; k < NV; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) m[r] = fmaxf(m[r], fmaxf(fabsf(v[r][k][e].x), fabsf(v[r][k][e].y)));
            }
        };
        float s[kBatch];
        if (a.g) {
            auto mean_square = [&]() { // of this lane's row
#pragma unroll
                for (int r = 0; r < kBatch; ++r) {
                    float2 ss = make_float2(0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < NV; ++k)
#pragma unroll
                        for (int e = 0; e < 4; ++e) ss = fma2(v[r][k][e], v[r][k][e], ss);
                    s[r] = ss.x + ss.y;
                }
                return reduce(s, lane, [](float x, float y) { return x + y; }) / (float)R;
            };
            float ms = mean_square() + a.eps;
            // squares that overflow, or fall among the subnormals where eps does not cover them: the row is brought near 1
            // by a power of two first, and eps by its square, which leaves the quotient as it is
            const bool far = !(ms < 1e38f && ms > 8.0779357e-28f); // 2^-90
            if (__any_sync(0xffffffffu, far)) {
                row_amax(s);
                const float am = reduce(s, lane, [](float x, float y) { return fmaxf(x, y); });
                const int ea = (int)(__float_as_uint(am) >> 23) - 127, ee = (int)(__float_as_uint(a.eps) >> 23) - 127;
                const int up = far ? max(-126, min(-ea, (100 - ee) / 2)) : 0;
                const float f = exp2i(up);
#pragma unroll
                for (int r = 0; r < kBatch; ++r) {
                    const float fr = of_row<kBatch>(f, r);
#pragma unroll
                    for (int k = 0; k < NV; ++k)
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[r][k][e] = mul2(v[r][k][e], make_float2(fr, fr));
                }
                ms = mean_square() + a.eps * f * f;
            }
            const float f = 1.f / sqrtf(ms);
#pragma unroll
            for (int r = 0; r < kBatch; ++r) s[r] = of_row<kBatch>(f, r);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int j = 8 * (lane + 32 * k);
                if (j >= R) continue;
                const float4 u = __ldg(reinterpret_cast<const float4 *>(a.g + j)), w = __ldg(reinterpret_cast<const float4 *>(a.g + j + 4));
                const float2 g[4] = {make_float2(u.x, u.y), make_float2(u.z, u.w), make_float2(w.x, w.y), make_float2(w.z, w.w)};
#pragma unroll
                for (int r = 0; r < kBatch; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[r][k][e] = mul2(mul2(v[r][k][e], make_float2(s[r], s[r])), g[e]);
            }
        }
        row_amax(s);
        float my_sc = __fdiv_rn(reduce(s, lane, [](float x, float y) { return fmaxf(x, y); }), 448.f);
        if (!(my_sc > 0.f)) my_sc = 1.f;
        const float my_inv = 1.f / my_sc;
        const bool plain = __all_sync(0xffffffffu, my_sc > 8.0779357e-28f && my_sc < 1.2379400e27f); // 2^-90 .. 2^90
        uint2 code[kBatch][NV];
#pragma unroll
        for (int r = 0; r < kBatch; ++r) {
            const float sc = of_row<kBatch>(my_sc, r), inv = of_row<kBatch>(my_inv, r);
#pragma unroll
            for (int k = 0; k < NV; ++k) code[r][k] = encode8(v[r][k], sc, inv, plain);
            s[r] = sc;
        }
#pragma unroll
        for (int r = 0; r < kBatch; ++r) {
            if (row[r] < 0) continue;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int j = 8 * (lane + 32 * k);
                if (j < R) *reinterpret_cast<uint2 *>(a.out.fp8 + row[r] * R + j) = code[r][k];
            }
            if (lane == 0) a.out.scale[row[r]] = s[r];
        }
    }
}

__device__ __forceinline__ void st8(uint16_t *p, const float2 (&v)[4])
{
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = uint32_t(f32_to_bf16_bits(v[e].x)) | (uint32_t(f32_to_bf16_bits(v[e].y)) << 16);
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
}
__device__ __forceinline__ void st8(float *p, const float2 (&v)[4])
{
    __stcs(reinterpret_cast<float4 *>(p), make_float4(v[0].x, v[0].y, v[1].x, v[1].y));
    __stcs(reinterpret_cast<float4 *>(p + 4), make_float4(v[2].x, v[2].y, v[3].x, v[3].y));
}

constexpr int kGatherRows = 4; // rows per warp (200k rows: 8 at once 69 us, 4 60 us, 16 77 us)

template <typename Tout> __global__ void __launch_bounds__(256) latent_gather_kernel(LatentGatherArgs a)
{
    const int lane = threadIdx.x & 31;
    const int64_t n0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * kGatherRows;
    const int rd = a.rows.rope_dims, R = a.rows.c - rd;
    // lane l < kGatherRows resolves row n0 + l: -2 outside the runs (left as it is), -1 refused
    int64_t mine = -2;
    if (lane < kGatherRows) {
        const int64_t n = n0 + lane;
        if (n < a.n_out && n >= a.cu[0] && n < a.cu[a.B]) {
            int64_t lo = 0, hi = a.B; // the last b with cu[b] <= n
            while (hi - lo > 1) {
                const int64_t mid = (lo + hi) / 2;
                if (a.cu[mid] <= n) lo = mid;
                else hi = mid;
            }
            const int64_t s = n - a.cu[lo] + (a.start ? a.start[lo] : 0);
            mine = s >= 0 ? a.map.row(lo, s) : -1;
            if (mine < 0) {
                mine = -1;
                flag_error(a.err, CSA_DEVERR_INDEX);
            }
        }
    }
    for (int j0 = 0; a.lat && j0 < R; j0 += 256) { // 8 channels a lane: its store is 16 bytes (bf16) beside its neighbour's
        const int j = j0 + 8 * lane;
        uint2 u[kGatherRows];
        float s[kGatherRows];
        int64_t row[kGatherRows];
#pragma unroll
        for (int r = 0; r < kGatherRows; ++r) {
            row[r] = __shfl_sync(0xffffffffu, mine, r);
            u[r] = make_uint2(0, 0);
            s[r] = 0.f;
            if (row[r] >= 0 && j < R) {
                u[r] = __ldg(reinterpret_cast<const uint2 *>(a.rows.fp8 + row[r] * R + j));
                s[r] = __ldg(a.rows.scale + row[r]);
            }
        }
#pragma unroll
        for (int r = 0; r < kGatherRows; ++r) {
            if (row[r] < -1 || j >= R) continue;
            const uint32_t w[2] = {u[r].x, u[r].y};
            float2 v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 x = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[e >> 1] >> (16 * (e & 1))), __NV_E4M3)));
                v[e] = make_float2(x.x * s[r], x.y * s[r]);
            }
            st8(static_cast<Tout *>(a.lat) + (n0 + r) * R + j, v);
        }
    }
    if (a.rope) {
        const int per = rd / 8; // 16-byte vectors a row
        for (int e = lane; e - lane < kGatherRows * per; e += 32) {
            const int r = e / per < kGatherRows ? e / per : kGatherRows - 1;
            const int64_t row = __shfl_sync(0xffffffffu, mine, r);
            if (e >= kGatherRows * per || row < -1) continue;
            const int j = 8 * (e % per);
            float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (row >= 0) {
                const uint4 q = __ldg(reinterpret_cast<const uint4 *>(a.rows.rope + row * rd + j));
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
            Tout *dst = static_cast<Tout *>(a.rope) + (n0 + r) * rd + j;
            st4(dst, 0, make_float4(v[0], v[1], v[2], v[3]));
            st4(dst, 4, make_float4(v[4], v[5], v[6], v[7]));
        }
    }
}

} // namespace

template <typename Tin> static void append(const LatentAppendArgs &a, cudaStream_t st)
{
    // as many rows a warp as make one wave of 16 warps an SM, at most 32 (a lane looks up each)
    const int64_t warps = 16 * (int64_t)device_sms(), p = (a.n + warps - 1) / warps;
    const int per = p < 2 ? 1 : p > 32 ? 32 : (int)(p + 3) / 4 * 4;
    const unsigned grid = (unsigned)((a.n + 8 * per - 1) / (8 * per));
    const double lb = a.base > 0 ? log(a.base) : 0.0;
    const int R = a.out.c - a.out.rope_dims;
    auto run = [&](auto kernel) { kernel<<<grid, 256, 0, st>>>(a, lb, per); };
    if (per == 1) // (64 rows: 4.0 us, for four at once 6.8)
        R <= 256 ? run(latent_append_kernel<Tin, 1, 1>) : R <= 512 ? run(latent_append_kernel<Tin, 2, 1>) : run(latent_append_kernel<Tin, 4, 1>);
    else
        R <= 256 ? run(latent_append_kernel<Tin, 1, 4>) : R <= 512 ? run(latent_append_kernel<Tin, 2, 4>) : run(latent_append_kernel<Tin, 4, 4>);
}

cudaError_t launch_latent_append(const LatentAppendArgs &a, int in_dtype, cudaStream_t st)
{
    if (in_dtype == CSA_F32) append<float>(a, st);
    else append<uint16_t>(a, st);
    return cudaGetLastError();
}

cudaError_t launch_latent_gather(const LatentGatherArgs &a, int out_dtype, cudaStream_t st)
{
    const unsigned grid = (unsigned)((a.n_out + 8 * kGatherRows - 1) / (8 * kGatherRows));
    if (out_dtype == CSA_F32) latent_gather_kernel<float><<<grid, 256, 0, st>>>(a);
    else latent_gather_kernel<uint16_t><<<grid, 256, 0, st>>>(a);
    return cudaGetLastError();
}

} // namespace csa
